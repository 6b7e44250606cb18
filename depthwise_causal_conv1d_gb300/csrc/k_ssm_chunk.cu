// Selective scan in chunks of 128 tokens on the tensor cores (ccu_selective_scan,
// CCU_SCAN_CHUNKED).
//
// With c_t the running sum of d A over a chunk's tokens (so exp(c_t - c_s) is the decay from
// token s to token t) and h the state before the chunk,
//
//   y_t = exp(c_t) C_t h  +  sum_{s <= t} exp(c_t - c_s) d_s (C_t . B_s) x_s
//   h'  = exp(c_end) h    +  sum_s exp(c_end - c_s) d_s  B_s (x) x_s
//
// A CTA walks the chunks of one (sequence, head, 64 channels) and keeps h on the SM. Per chunk,
// four products, all BF16 in and FP32 out (t, s tokens; k states; p channels):
//
//   S[t,s] = C B^T          C, B from shared memory
//   Y[t,p] = C h^T          h in two BF16 terms; the rows are then scaled by exp(c_t) in FP32
//   Y     += M x            M = S with decays, steps and the causal mask, in two BF16 terms, in TMEM
//   U[k,p] = B^T (w x)      w_s = exp(c_end - c_s) d_s
//
// Rounding. M and the h that Y sees are split into two BF16 terms (16 bits in all), so a term of an output is off by 2^-16
// or less and what the outputs are off is their own rounding. (Rounded to BF16 once, at 2^-9 a term, the outputs
// of the batch below were off by 0.0018 of their size instead of 0.0017; the second terms take 430 -> 489 us.) The
// state may not lose that much either: w x is split into three BF16 terms (24 bits in all) and U accumulated over
// all three, and h itself stays FP32 (in registers) and is only added to by FP32 instructions.
//
// Decays are exponentials of differences of running sums; a difference of sums over a whole chunk
// would lose what the steps' sizes vary by, and a product exp(c_t) exp(-c_s) would overflow. So the sums run
// over 32 tokens: within such a block the difference is taken, between blocks the decay is
// a product of two that are both at most 1, exp(c_t - c_r) exp(c_r - c_s), r the token before t's block.
// The state's weights come from sums taken from the chunk's end.
//
// One CTA an SM, its warps in roles that meet at mbarriers, so that the products of one chunk run
// under the element work of its neighbours (in lock step, eight warps doing every phase in turn, a chunk
// took 13 thousand cycles of which the products were 2.3):
//
//   4 warps   M: S from TMEM, decays and mask, split, back over S
//   4 warps   w x: x from shared memory, split, to shared memory
//   8 warps   out: exp(c_t) Y0 + Y, skip, gate, store
//   8 warps   h: FP32 in registers (a thread a state, 32 of its channels), U added, split, to shared memory: the
//             second term over the first, once its product is done (there is no room for both)
//   1 warp    the products, by one thread, in the order Y0(c) in two terms, U(c+1), S(c+1), Y(c): U needs neither S
//             nor h, so the state runs a chunk ahead of the outputs, and M(c) is made under Y0(c) and U(c+1)
//   1 warp    the copies (TMA, zero-filled past P and K)
//   2 warps   the decays, of every other chunk each
//
// TMEM (512 columns): S, later M, 2 x 128; Y 64; Y0 2 x 64; U 64. Shared memory 222 KB: B 2 x 32,
// C 32, x 3 x 16, w x 48, h 16, decays of 4 chunks.
//
// 8 x 4096 tokens, 64 heads of 64 channels, 128 states: 489 us (1.72 TB/s of the bytes it cannot do without; token by token
// 9.8 ms); one sequence of 16384: 356 us, in 7 segments. Neither HBM (21 %) nor the tensor cores (31 %) bound it: a
// chunk takes 7.5 thousand cycles, which the element work's roles share at 1.8 instructions a cycle, waiting for
// TMEM and for each other. Every wait has a limit; a role that runs into it
// reports CCU_DEVERR_TIMEOUT and ends, and so do the others.
#include <atomic>
#include <cstddef>

#include "ssm_tensor.cuh"

namespace ccu {

int current_device();
int device_sm_count();

__device__ int32_t g_scan_error = 0;        // CCU_DEVERR_* bits of calls without a status word
__device__ int32_t g_scan_error_taken = 0;  // the value the last exchange read

__global__ void k_exchange_scan_error() {
  grid_dependency_boundary();
  g_scan_error_taken = atomicExch(&g_scan_error, 0);
}

namespace {

using namespace tensor;

constexpr int kQ = 128;       // tokens a chunk
constexpr int kTile = kQ * 128;             // a block of 128 rows: 16 KB
constexpr int kWarpsW = 4 /* M: warps 0..3 */, kWarpsOut = 8, kWarpsH = 16, kWarpMma = 24, kWarpCopy = 25, kWarpDecay = 26;
constexpr int kThreads = 28 * 32;            // 72 registers a thread
constexpr int kColS = 0, kColY = 256, kColY0 = 320, kColU = 448, kColumns = 512;
constexpr int kStages = 4;    // chunks of decays
constexpr float kLog2e = 1.4426950408889634f;
// exp2 of anything below -150 is zero in FP32; sums of steps stay finite and small with this floor.
constexpr float kLeast = -300.0f;

struct alignas(16) Decays {   // read in 16-byte vectors
  float sum[kQ], step[kQ];    // running sum of log2 decays in its block of 32; d
  float from[3][kQ];          // [r - 1][s]: decay from s to the token before block r, times d_s
  float in[kQ], weight[kQ];   // exp(c_t); w
  float total[4];             // sums of the blocks
  int bad[64];                // first token with a non-finite x, a channel
  int any_bad;
  float decay;                // exp(c_end)
};

// What a CTA works on. Read from shared memory by the roles: held in registers from the start, it made them spill.
struct Job {
  int64_t begin, length, s, h, b, p0, segment;
  int g, np, first, last, whole;
};

struct alignas(16) Shared {
  Decays decays[kStages];
  uint64_t d_full[kStages], d_empty[kStages];
  uint64_t b_full[2], b_empty[2], c_full, c_done, x_full[3], x_empty[3];
  uint64_t s_full[2], m_ready[2], w_ready, u_full[2], u_empty[2], h_ready, h_read, rest_ready, y_full, y_empty, drained;
  Job job;
  uint32_t tmem;
};

constexpr int kSmemB = 0, kSmemC = 4 * kTile, kSmemX = 6 * kTile, kSmemW = 9 * kTile, kSmemH = 12 * kTile, kSmemShared = 13 * kTile;
constexpr size_t kSmemBytes = kSmemShared + sizeof(Shared) + 1024;
static_assert(sizeof(Decays) % 16 == 0 && offsetof(Decays, from) % 16 == 0 && offsetof(Decays, step) % 16 == 0, "vectors");
static_assert(kSmemBytes <= 227 * 1024, "shared memory of a CTA");

__device__ __forceinline__ float first_of(uint32_t pair) { return __uint_as_float(pair << 16); }
__device__ __forceinline__ float second_of(uint32_t pair) { return __uint_as_float(pair & 0xffff0000u); }

// A pair as three BF16 pairs whose sums are the pair to 24 bits.
__device__ __forceinline__ void split3(float2 v, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
  const float2 minus = make_float2(-1.0f, -1.0f);
  hi = pack_bf16x2(v.x, v.y);
  v = __ffma2_rn(make_float2(first_of(hi), second_of(hi)), minus, v);
  mid = pack_bf16x2(v.x, v.y);
  v = __ffma2_rn(make_float2(first_of(mid), second_of(mid)), minus, v);
  lo = pack_bf16x2(v.x, v.y);
}

// A pair as two BF16 pairs whose sums are the pair to 16 bits.
__device__ __forceinline__ void split2(float2 v, uint32_t &hi, uint32_t &lo) {
  hi = pack_bf16x2(v.x, v.y);
  v = __ffma2_rn(make_float2(first_of(hi), second_of(hi)), make_float2(-1.0f, -1.0f), v);
  lo = pack_bf16x2(v.x, v.y);
}

// The kernel's instructions have to fit the caches: with every loop and wait unrolled in place
// they were 192 KB, and all roles waited for their own code (8 x 4096 tokens 1286 us). So loops are
// rolled where no register array needs them unrolled, a wait is a loop of a few instructions, and what
// is long and rare stands once.
__device__ __forceinline__ bool wait_phase(uint64_t *bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
      "mov.u32 n, %3;\n\t"
      "AGAIN:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra DONE;\n\t"
      "sub.u32 n, n, 1;\n\t"
      "setp.ne.u32 q, n, 0;\n\t"
      "@q bra AGAIN;\n\t"
      "DONE:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bulk::smem_addr(bar)), "r"(parity), "n"(bulk::kMaxSpins)
      : "memory");
  return done != 0;
}

// How sequences are cut when there are too few of them, and heads, to fill the card: segments of
// `tokens` (a multiple of the chunk). A first launch (STATES) computes what every segment but a sequence's last
// adds to the state and how it decays it, U and the state alone; the second starts every segment from the
// states before it.
//
// The lengths are on the device, so segments are numbered from the offsets: sequence b has the numbers from
// first_segment(b) on, of which it needs ceil(length / tokens), or one when it is empty, and never more than there are up to
// first_segment(b + 1). `count` = T / tokens + sequences bounds them all: the grid and the workspace grow with
// the tokens and the sequences, not with their product.
struct Segments {
  int64_t count, tokens;
  float *states;  // [segment][H, P, K]
  float *decays;  // [segment][H]
};

__device__ __forceinline__ int64_t first_segment(const ScanParams &p, const Segments &seg, int64_t b) {
  const int64_t t = __ldg(p.cu_seqlens + b);
  return (t < 0 ? 0 : t > p.T ? p.T : t) / seg.tokens + b;
}

// The states before the segments, from what each segment adds and how it decays what comes before it:
// one thread a state, its sequence's segments in order.
__global__ void __launch_bounds__(256) k_scan_join(ScanParams p, Segments seg) {
  grid_dependency_boundary();
  const int64_t inner = p.H * p.P * p.K, i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, b = blockIdx.y;
  if (i >= inner) return;
  if (slot_of(p.indices, b, p.S, nullptr, false) < 0) return;  // padding: nothing was written
  const Bounds q = sequence_bounds(p.cu_seqlens, b, p.T);
  const int64_t h = i / (p.P * p.K), parts = (q.end - q.begin + seg.tokens - 1) / seg.tokens;
  if (parts < 3) return;
  const int64_t first = first_segment(p, seg, b);
  float *entry = seg.states + first * inner + i;
  const float *decay = seg.decays + first * p.H + h;
  float v = entry[inner];
  for (int64_t j = 2; j < parts; ++j) {
    v = fmaf(v, decay[(j - 1) * p.H], entry[j * inner]);
    entry[j * inner] = v;
  }
}

// A chunk's decays, by one warp: lane l takes token l of each block of 32; `raw` are their dt, and
// tokens from `rows` on are past the sequence's end: no step. What goes into the state (weight, decay) takes
// exp2f, what is rounded to BF16 with its output the approximation (2^-22).
__device__ __forceinline__ void fill_decays(Decays &t, const uint16_t (&raw)[4], float bias, int softplus_on, int rows, float A2, int lane) {
  uint32_t pair = raw[0] | ((uint32_t)raw[1] << 16), later = raw[2] | ((uint32_t)raw[3] << 16);
#pragma unroll 1
  for (int j = 0; j < 4; ++j) {
    const int row = 32 * j + lane;
    const float d = row < rows ? step_of(first_of(pair) + bias, softplus_on) : 0.0f;
    pair = (pair >> 16) | (later << 16);
    later >>= 16;
    float a = d * A2;
    a = a < kLeast ? kLeast : a;
    float sum = a, after = a;  // over the block up to this token, and from this token on
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float u = __shfl_up_sync(0xffffffffu, sum, o), w = __shfl_down_sync(0xffffffffu, after, o);
      if (lane >= o) sum += u;
      if (lane + o < 32) after += w;
    }
    after = __shfl_down_sync(0xffffffffu, after, 1);
    t.sum[row] = sum;
    t.step[row] = d;
    t.weight[row] = lane == 31 ? 0.0f : after;  // for now
    if (lane == 31) t.total[j] = sum;
  }
  __syncwarp();
  const float4 total = *reinterpret_cast<const float4 *>(t.total);
  float before = 0.0f, rest = (total.y + total.z) + total.w;  // of the blocks before and after this one
#pragma unroll 1
  for (int j = 0; j < 4; ++j) {
    const int row = 32 * j + lane;
    const float d = t.step[row], after = t.weight[row];
    t.in[row] = ex2_approx_ftz(before + t.sum[row]);
    // the decay from this token to the token before block r: the rest of its block, and the blocks between
    if (j < 1) t.from[0][row] = ex2_approx_ftz(after) * d;
    if (j < 2) t.from[1][row] = ex2_approx_ftz(after + (j < 1 ? total.y : 0.0f)) * d;
    if (j < 3) t.from[2][row] = ex2_approx_ftz(after + (j < 1 ? total.y + total.z : j < 2 ? total.z : 0.0f)) * d;
    t.weight[row] = exp2f(after + rest) * d;
    before += t.total[j];
    rest = j < 1 ? total.z + total.w : j < 2 ? total.w : 0.0f;
  }
  t.bad[lane] = t.bad[32 + lane] = kQ;
  if (lane == 0) {
    t.any_bad = 0;
    t.decay = exp2f(before);
  }
}

template <bool STATES>
__global__ void __launch_bounds__(kThreads, 1) k_scan_chunked(ScanParams p, int blocks_p, Segments seg, const __grid_constant__ CUtensorMap map_x,
                                                              const __grid_constant__ CUtensorMap map_b,
                                                              const __grid_constant__ CUtensorMap map_c,
                                                              const __grid_constant__ CUtensorMap map_z) {
  grid_dependency_boundary();
  extern __shared__ unsigned char raw[];
  const uint32_t base = (bulk::smem_addr(raw) + 1023) & ~1023u;
  Shared &sh = *reinterpret_cast<Shared *>(raw + (base - bulk::smem_addr(raw)) + kSmemShared);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int quarter = warp & 3, row = quarter * 32 + lane;  // token (state) of a thread in the first four roles
  int64_t item = blockIdx.x;
  const int64_t p0 = item % blocks_p * 64;
  item /= blocks_p;
  const int64_t h = item % p.H;
  item /= p.H;
  int64_t b = item, part = 0;                        // this CTA's segment, of sequence b
  if (seg.tokens < p.T) {
    int64_t past = p.n_seq;
    for (b = 0; past - b > 1;) {
      const int64_t mid = (b + past) >> 1;
      if (first_segment(p, seg, mid) <= item) b = mid; else past = mid;
    }
    part = item - first_segment(p, seg, b);
    if (part < 0) return;                            // rows before the first sequence
  }
  const int g = (int)(h / (p.H / p.G));
  const int np = (int)(p.P - p0 < 64 ? p.P - p0 : 64), K = (int)p.K;
  Bounds q = sequence_bounds(p.cu_seqlens, b, p.T);
  const bool whole = q.end - q.begin <= seg.tokens;  // the sequence is one segment
  q.begin += part * seg.tokens;
  if (part > 0 && q.begin >= q.end) return;
  const bool last = q.end - q.begin <= seg.tokens;
  if (!last) q.end = q.begin + seg.tokens;
  if (STATES && last) return;  // nothing starts from its state
  const int64_t s = slot_of(p.indices, b, p.S, p.status_dev, !STATES && tid == 0 && h == 0 && p0 == 0 && part == 0);
  uint16_t *out = static_cast<uint16_t *>(p.out) + h * p.out_stride_h + p0;
  if (s < 0) {
    if (STATES) return;
    const int piece = tid & 7;
    if (8 * piece < np)
      for (int64_t t = q.begin + (tid >> 3); t < q.end; t += kThreads / 8) st_stream(out + t * p.out_stride_t + 8 * piece, make_uint4(0, 0, 0, 0));
    return;
  }
  if (warp == kWarpMma) tmem_alloc(&sh.tmem, kColumns);
  if (tid == 0) {
    sh.job = {q.begin, q.end - q.begin, s, h, b, p0, item, g, np, part == 0, last, whole};
    for (int i = 0; i < kStages; ++i) {
      bulk::mbar_init(&sh.d_full[i], 32);
      bulk::mbar_init(&sh.d_empty[i], STATES ? 12 : 24);
    }
    for (int i = 0; i < 2; ++i) {
      bulk::mbar_init(&sh.b_full[i], 1);
      bulk::mbar_init(&sh.b_empty[i], 1);
      bulk::mbar_init(&sh.s_full[i], 1);
      bulk::mbar_init(&sh.m_ready[i], kQ);
      bulk::mbar_init(&sh.u_full[i], 1);
      bulk::mbar_init(&sh.u_empty[i], 2 * kQ);
    }
    for (int i = 0; i < 3; ++i) {
      bulk::mbar_init(&sh.x_full[i], 1);
      bulk::mbar_init(&sh.x_empty[i], STATES ? 4 : 9);  // Y's product, and the eight warps that read x for the skip
    }
    bulk::mbar_init(&sh.c_full, 1);
    bulk::mbar_init(&sh.c_done, 1);
    bulk::mbar_init(&sh.w_ready, kQ);
    bulk::mbar_init(&sh.h_ready, 2 * kQ);
    bulk::mbar_init(&sh.h_read, 1);
    bulk::mbar_init(&sh.rest_ready, 2 * kQ);
    bulk::mbar_init(&sh.y_full, 1);
    bulk::mbar_init(&sh.drained, 1);
    bulk::mbar_init(&sh.y_empty, 2 * kQ);
    bulk::fence_mbar_init();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const Job &job = sh.job;
  const int chunks = (int)((job.length + kQ - 1) / kQ);
  const uint32_t tmem = sh.tmem, mine = tmem + ((uint32_t)(quarter * 32) << 16);
  // U of two chunks where TMEM has room for it: without outputs
  constexpr int kU = STATES ? 2 : 1;
  auto col_u = [](int c) { return STATES ? kColS + (c & 1) * 64 : kColU; };
  bool fine = true;
  // Waits for a barrier's phase number n (counted from 0); false when it gave up, now or before.
  auto wait = [&](uint64_t &bar, int n) { return fine = fine && wait_phase(&bar, n & 1); };
  auto wait2 = [&](uint64_t &bar, int n, uint64_t &also, int m) { return fine = fine && wait_phases(&bar, n & 1, &also, m & 1); };
  auto done_with = [&](int c) {  // a warp has read the decays of chunk c
    __syncwarp();
    if (lane == 0) bulk::mbar_arrive(&sh.d_empty[c % kStages]);
  };

  if (warp < kWarpsW) {
    // ---------------------------------------------------------------- M
    for (int c = 0; !STATES && c < chunks; ++c) {
      const Decays &now = sh.decays[c % kStages];
      if (!wait2(sh.d_full[c % kStages], c / kStages, sh.s_full[c & 1], c >> 1)) break;
      __syncwarp();
      fence_after_sync();
      const uint32_t at = mine + kColS + (c & 1) * 128;
      const float sum = now.sum[row], local = ex2_approx_ftz(sum);
#pragma unroll 1
      for (int block = 0; block < 4; ++block) {
        // 16 tokens s of M take the place of 16 columns of S: 8 columns of the first terms, 8 of the second.
        if (block > quarter) {
          uint32_t m[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) m[i] = 0;
          tmem_store16(at + 32 * block, m);
          tmem_store16(at + 32 * block + 16, m);
        } else {
          float v[32];
          tmem_load32(at + 32 * block, v);
          wait_loads();
          loaded(v);
          if (block < quarter) {
            const float4 *from = reinterpret_cast<const float4 *>(&now.from[quarter - 1][block * 32]);
            const float2 scale = make_float2(local, local);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint32_t m[16];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float4 f = from[4 * half + i];
                const float *e = v + 16 * half + 4 * i;
                const float2 u = __fmul2_rn(make_float2(e[0], e[1]), __fmul2_rn(scale, make_float2(f.x, f.y)));
                const float2 w = __fmul2_rn(make_float2(e[2], e[3]), __fmul2_rn(scale, make_float2(f.z, f.w)));
                split2(u, m[2 * i], m[8 + 2 * i]);
                split2(w, m[2 * i + 1], m[9 + 2 * i]);
              }
              tmem_store16(at + 32 * block + 16 * half, m);
            }
          } else {
            const float4 *sums = reinterpret_cast<const float4 *>(&now.sum[block * 32]);
            const float4 *steps = reinterpret_cast<const float4 *>(&now.step[block * 32]);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint32_t m[16];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float4 e = sums[4 * half + i], d = steps[4 * half + i];
                const int s = 16 * half + 4 * i;  // in the block: token s counts for those from it on
                const float w0 = ex2_approx_ftz(sum - e.x) * d.x, w1 = ex2_approx_ftz(sum - e.y) * d.y;
                const float w2 = ex2_approx_ftz(sum - e.z) * d.z, w3 = ex2_approx_ftz(sum - e.w) * d.w;
                split2(make_float2(s <= lane ? v[s] * w0 : 0.0f, s + 1 <= lane ? v[s + 1] * w1 : 0.0f), m[2 * i], m[8 + 2 * i]);
                split2(make_float2(s + 2 <= lane ? v[s + 2] * w2 : 0.0f, s + 3 <= lane ? v[s + 3] * w3 : 0.0f), m[2 * i + 1], m[9 + 2 * i]);
              }
              tmem_store16(at + 32 * block + 16 * half, m);
            }
          }
        }
      }
      wait_stores();
      fence_before_sync();
      bulk::mbar_arrive(&sh.m_ready[c & 1]);
      done_with(c);
    }
  } else if (warp < kWarpsOut) {
    // ---------------------------------------------------------------- w x
    for (int c = 0; c < chunks; ++c) {
      Decays &now = sh.decays[c % kStages];
      const int rows = (int)(job.length - (int64_t)c * kQ < kQ ? job.length - (int64_t)c * kQ : kQ);
      if (!wait2(sh.d_full[c % kStages], c / kStages, sh.x_full[c % 3], c / 3)) break;
      // a partial chunk's B is in place before its rows are zeroed
      if (rows < kQ && !wait(sh.b_full[c & 1], c >> 1)) break;
      const uint32_t tile = base + kSmemX + c % 3 * kTile;
      if (row >= rows) {  // a row of another sequence
        const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
          const uint32_t at = swizzled(row, i);
          sts128(tile + at, zero);
          sts128(base + kSmemB + (c & 1) * 2 * kTile + at, zero);
          sts128(base + kSmemB + (c & 1) * 2 * kTile + kTile + at, zero);
        }
      }
      const float2 w = make_float2(now.weight[row], now.weight[row]);
      float2 probe = make_float2(0.0f, 0.0f);  // 0 x, summed: NaN if any x is not finite
#pragma unroll 1
      for (int i = 0; i < 8; i += 2) {
        uint32_t term[3][8];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint4 x = lds128(tile + swizzled(row, i + k));
          const uint32_t e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 v = make_float2(first_of(e[j]), second_of(e[j]));
            probe = __ffma2_rn(v, make_float2(0.0f, 0.0f), probe);
            split3(__fmul2_rn(w, v), term[0][4 * k + j], term[1][4 * k + j], term[2][4 * k + j]);
          }
        }
        // w x of the last chunk has been used
        if (i == 0 && c > 0) wait(sh.u_full[(c - 1) % kU], (c - 1) / kU);
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int j = 0; j < 3; ++j)
            sts128(base + kSmemW + j * kTile + swizzled(row, i + k),
                   make_uint4(term[j][4 * k], term[j][4 * k + 1], term[j][4 * k + 2], term[j][4 * k + 3]));
      }
      if (!fine) break;
      if (!(probe.x + probe.y == 0.0f)) {
        // A non-finite value goes into the first term alone. In M's product it would reach earlier tokens
        // through the zeros of M: it is taken out of the tile, and its channel's outputs from there on are NaN.
        now.any_bad = 1;
#pragma unroll 1
        for (int i = 0; i < 32; ++i) {
          const uint32_t at = swizzled(row, i >> 2) + (i & 3) * 4, e = lds32(tile + at);
          const bool f = (e & 0x7f80u) == 0x7f80u, l = (e & 0x7f800000u) == 0x7f800000u;
          const uint32_t keep = (f ? 0u : 0xffffu) | (l ? 0u : 0xffff0000u);
          if (f) atomicMin(&now.bad[2 * i], row);
          if (l) atomicMin(&now.bad[2 * i + 1], row);
          sts32(tile + at, e & keep);
          sts32(base + kSmemW + kTile + at, lds32(base + kSmemW + kTile + at) & keep);
          sts32(base + kSmemW + 2 * kTile + at, lds32(base + kSmemW + 2 * kTile + at) & keep);
        }
      }
      bulk::fence_proxy_async();
      bulk::mbar_arrive(&sh.w_ready);
      done_with(c);
      if (STATES && lane == 0) bulk::mbar_arrive(&sh.x_empty[c % 3]);
    }
  } else if (warp < kWarpsH) {
    // ---------------------------------------------------------------- out
    const uint16_t *z = p.z != nullptr ? static_cast<const uint16_t *>(p.z) + job.h * p.z_stride_h + job.p0 : nullptr;
    const float skip = p.D != nullptr ? __ldg(p.D + job.h) : 0.0f;
    const int side = (warp - kWarpsOut) >> 2;  // 32 channels a warp: 0..31 or 32..63
    // T < 2^31: what is left of the sequence from this token on is an int.
    int left = (int)job.length - row;
    const int pieces = (job.np - 32 * side) >> 3;  // 8 channels each; 4 or more: all of them
    uint16_t *to = out + (job.begin + row) * p.out_stride_t + 32 * side;
    const bool gated = z != nullptr;
    if (gated) z += (job.begin + row) * p.z_stride_t + 32 * side;
    for (int c = 0; !STATES && c < chunks; ++c, left -= kQ, to += kQ * p.out_stride_t, z += kQ * p.z_stride_t) {
      // The gate comes from L2 (the copying warp asked for it) while Y is on its way. No register of it
      // lives from one round to the next: a copy of a load in flight would wait for it.
      uint4 zv[4];
      if (gated && left > 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < pieces) zv[i] = ld_stream(z + 8 * i);
      }
      const Decays &now = sh.decays[c % kStages];
      if (!wait2(sh.d_full[c % kStages], c / kStages, sh.y_full, c)) break;
      __syncwarp();
      fence_after_sync();
      const float2 in = make_float2(now.in[row], now.in[row]), skips = make_float2(skip, skip);
      const bool any_bad = now.any_bad != 0;
      const uint32_t tile = base + kSmemX + c % 3 * kTile;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int channel = 32 * side + 8 * i;
        float y[8], y0[8];
        tmem_load8(mine + kColY0 + (c & 1) * 64 + channel, y0);
        tmem_load8(mine + kColY + channel, y);
        uint4 x = make_uint4(0, 0, 0, 0);  // without a D it must not count (0 x NaN)
        if (p.D != nullptr) x = lds128(tile + swizzled(row, channel >> 3));
        const uint32_t e[4] = {x.x, x.y, x.z, x.w}, f[4] = {zv[i].x, zv[i].y, zv[i].z, zv[i].w};
        wait_loads();
        loaded(y0);
        loaded(y);
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float2 r = __ffma2_rn(in, make_float2(y0[2 * j], y0[2 * j + 1]), make_float2(y[2 * j], y[2 * j + 1]));
          r = __ffma2_rn(skips, make_float2(first_of(e[j]), second_of(e[j])), r);
          if (gated) r = __fmul2_rn(r, activate2<1>(make_float2(first_of(f[j]), second_of(f[j]))));
          o[j] = pack_bf16x2(r.x, r.y);
        }
        if (any_bad) {
#pragma unroll 1
          for (int j = 0; j < 8; ++j)
            if (now.bad[channel + j] <= row) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (j >> 1 == k) o[k] = j & 1 ? (o[k] & 0xffffu) | 0x7fff0000u : (o[k] & 0xffff0000u) | 0x7fffu;
            }
        }
        if (left > 0 && i < pieces) st_stream(to + 8 * i, make_uint4(o[0], o[1], o[2], o[3]));
      }
      fence_before_sync();
      bulk::mbar_arrive(&sh.y_empty);
      done_with(c);
      if (lane == 0) bulk::mbar_arrive(&sh.x_empty[c % 3]);
    }
  } else if (warp < kWarpMma) {
    // ---------------------------------------------------------------- h
    const int first = ((warp - kWarpsH) >> 2) * 32, mine_of = job.np - first;  // 32 channels, as many as there are
    const int64_t at_h = (job.h * p.P + job.p0 + first) * p.K, inner = p.H * p.P * p.K;
    float *state = p.state + job.s * p.state_stride_s + at_h;
    // A segment's entry of the workspace: the state before it (from a sequence's third on what the segment before adds to
    // it, until the joining kernel has been through).
    float *entry = seg.states + job.segment * inner + at_h;
    const bool initial = p.has_initial != nullptr && __ldg(p.has_initial + job.b) != 0;
    float v[32];
    auto read = [&](const float *from) {  // (zeros past the channels and states there are)
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        v[i] = i < mine_of && row < K ? from[i * K + row] : 0.0f;
        if (i % 8 == 7) asm volatile("" ::: "memory");  // eight loads at a time: their addresses take registers
      }
    };
    auto write = [&](float *to) {
      asm volatile("" : "+l"(to));  // else the addresses of the first reads are kept for it, spilled
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        if (i < mine_of && row < K) to[i * K + row] = v[i];
        if (i % 8 == 7) asm volatile("" ::: "memory");
      }
    };
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = 0.0f;
    if (STATES || job.whole) {
      if (job.first && initial) read(state);
      if (STATES && job.first) write(entry);
    } else {
      read(entry);
    }
    float through = 1.0f;  // decay of the segment
    // The state's place in the operand tile of Y0's product: row channel, K-major in k.
    const uint32_t at = base + kSmemH + (row >> 6) * (kTile / 2) + first * 128 + (row & 7) * 2;
    const int piece = (row >> 3) & 7;
    auto put = [&](int i, uint32_t pair) {  // channels i and i + 1
      sts16(at + i * 128 + ((piece ^ (i & 7)) << 4), (uint16_t)pair);
      sts16(at + (i + 1) * 128 + ((piece ^ ((i + 1) & 7)) << 4), (uint16_t)(pair >> 16));
    };
    for (int c = 0; c <= chunks; ++c) {
      if (!STATES && c < chunks) {
#pragma unroll
        for (int i = 0; i < 32; i += 2) put(i, pack_bf16x2(v[i], v[i + 1]));
        bulk::fence_proxy_async();
        bulk::mbar_arrive(&sh.h_ready);
        // the second term goes over the first once its product is done
        if (!wait(sh.h_read, c)) break;
        loaded(v);  // else the first terms are kept for it, in registers that there are not
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          uint32_t first_term, rest;
          split2(make_float2(v[i], v[i + 1]), first_term, rest);
          put(i, rest);
        }
        bulk::fence_proxy_async();
        bulk::mbar_arrive(&sh.rest_ready);
      }
      if (c == chunks) break;
      const Decays &now = sh.decays[c % kStages];
      if (!wait2(sh.d_full[c % kStages], c / kStages, sh.u_full[c % kU], c / kU)) break;
      __syncwarp();
      fence_after_sync();
      const float2 decay = make_float2(now.decay, now.decay);
      if (STATES) through *= decay.x;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float u[16];
        tmem_load16(mine + col_u(c) + first + 16 * i, u);
        wait_loads();
        loaded(u);
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          const float2 r = __ffma2_rn(make_float2(v[16 * i + j], v[16 * i + j + 1]), decay, make_float2(u[j], u[j + 1]));
          v[16 * i + j] = r.x;
          v[16 * i + j + 1] = r.y;
        }
      }
      fence_before_sync();
      bulk::mbar_arrive(&sh.u_empty[c % kU]);
      done_with(c);
      if (!STATES && !wait(sh.c_done, c)) break;  // Y0's product has read the old h
    }
    if (fine) {
      if (STATES) {
        write(entry + inner);
        if (warp == kWarpsH && lane == 0 && job.p0 == 0) seg.decays[job.segment * p.H + job.h] = through;
      } else if (job.last) {
        write(state);
      }
    }
  } else {
    if (warp == kWarpMma) {
      // The whole warp walks the loop, so that addresses stay in uniform registers; one lane issues.
      const bool leader = elect_one();
      // ---------------------------------------------------------------- products
      uint64_t b_mn = desc_mn_major(base + kSmemB, kTile), w_mn = desc_mn_major(base + kSmemW, kTile);
      uint64_t b_k = desc_k_major(base + kSmemB), c_k = desc_k_major(base + kSmemC), h_k = desc_k_major(base + kSmemH);
      uint64_t x_mn = desc_mn_major(base + kSmemX, kTile);
      // Opaque to the compiler from here on: with their constant parts in sight some builds of this kernel had channels 8 and up of
      // every output wrong, the same in every run. The cause was not found (their fields and sums, all below a field's size,
      // are right by hand); the tests compare every channel.
      asm volatile("" : "+l"(b_mn), "+l"(w_mn), "+l"(x_mn), "+l"(b_k), "+l"(c_k), "+l"(h_k));
      constexpr uint64_t kTile16 = kTile >> 4;  // descriptors count in 16 bytes: 16 K are 2 along rows, 128 across them
      auto product_u = [&](int c) {  // U = B^T (w x)
        // the first U find their places empty
        uint64_t &place = c >= kU ? sh.u_empty[c % kU] : sh.b_full[c & 1];
        fine = fine && wait_phases(&sh.w_ready, c & 1, &sh.b_full[c & 1], (c >> 1) & 1, &place, (c >= kU ? c / kU - 1 : c >> 1) & 1);
        if (!fine) return;
        fence_after_sync();
        if (leader) {
          const uint64_t bt = b_mn + (c & 1) * 2 * kTile16;
  #pragma unroll
          for (int term = 0; term < 3; ++term)
  #pragma unroll
            for (int k = 0; k < 8; ++k)
              mma_ss(tmem + col_u(c), bt + 128 * k, w_mn + term * kTile16 + 128 * k, instruction(128, 64, true, true), term + k > 0);
          mma_commit(&sh.u_full[c % kU]);
          if (STATES) mma_commit(&sh.b_empty[c & 1]);
        }
      };
      auto product_y0 = [&](int c, bool add) {
        fence_after_sync();
        if (leader) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_ss(tmem + kColY0 + (c & 1) * 64, c_k + (k >> 2) * kTile16 + (k & 3) * 2, h_k + (k >> 2) * (kTile16 / 2) + (k & 3) * 2,
                   instruction(128, 64, false, false), add || k > 0);
        }
      };
      auto product_s = [&](int c) {  // S = C B^T, over M of two chunks before, whose product is done
        fine = fine && wait_phases(&sh.c_full, c & 1, c >= 2 ? &sh.y_full : &sh.c_full, c & 1);
        if (!fine) return;
        fence_after_sync();
        if (leader) {
          const uint64_t bt = b_k + (c & 1) * 2 * kTile16;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint64_t at = (k >> 2) * kTile16 + (k & 3) * 2;
            mma_ss(tmem + kColS + (c & 1) * 128, c_k + at, bt + at, instruction(128, 128, false, false), k > 0);
          }
          mma_commit(&sh.s_full[c & 1]);
        }
      };
      if (chunks > 0) product_u(0);
      if (!STATES && chunks > 0) product_s(0);
#pragma unroll 1
      for (int c = 0; fine && c < chunks; ++c) {
        if (STATES) {
          if (c + 1 < chunks) product_u(c + 1);
          continue;
        }
        // Y0 = C h^T, the first term of h, and the second when the state's warps have put it into the first one's place
        // (Y0 of two chunks before is out: Y of the last one waited for that)
        if (!wait(sh.h_ready, c)) break;
        product_y0(c, false);
        if (leader) {
          mma_commit(&sh.h_read);
          mma_commit(&sh.b_empty[c & 1]);
        }
        if (!wait(sh.rest_ready, c)) break;
        product_y0(c, true);
        if (leader) mma_commit(&sh.c_done);
        if (c + 1 < chunks) {
          product_u(c + 1);
          product_s(c + 1);
        }
        // Y = M x, both terms of M; Y of the last chunk is out
        if (!wait2(sh.m_ready[c & 1], c >> 1, c > 0 ? sh.y_empty : sh.m_ready[c & 1], c > 0 ? c - 1 : c >> 1)) break;
        fence_after_sync();
        if (leader) {
          const uint64_t xt = x_mn + c % 3 * kTile16;
          const uint32_t m = tmem + kColS + (c & 1) * 128;
#pragma unroll
          for (int term = 0; term < 2; ++term)
#pragma unroll
            for (int k = 0; k < 8; ++k)
              mma_ts(tmem + kColY, m + 16 * k + 8 * term, xt + 128 * k, instruction(128, 64, false, true), term + k > 0);
          mma_commit(&sh.y_full);
          mma_commit(&sh.x_empty[c % 3]);
        }
      }
      // No product reads shared memory or TMEM, and no barrier is to be arrived at, once the CTA leaves: also
      // where a wait ran out and what was issued is left behind.
      if (leader) mma_commit(&sh.drained);
      fine &= wait_phase(&sh.drained, 0);
    } else if (warp == kWarpCopy && lane == 0) {
      // ---------------------------------------------------------------- copies
      int issued_x = 0, issued_b = 0, issued_c = 0;
      auto load_x = [&](int c) {
        if (c >= 3 && !wait(sh.x_empty[c % 3], c / 3 - 1)) return;
        issued_x = c + 1;
        bulk::mbar_arrive_expect_tx(&sh.x_full[c % 3], kTile);
        tile_load(base + kSmemX + c % 3 * kTile, &map_x, (int)job.p0, (int)job.h, (int)(job.begin + (int64_t)c * kQ), &sh.x_full[c % 3]);
        if (!STATES && p.z != nullptr) tile_prefetch(&map_z, (int)job.p0, (int)job.h, (int)(job.begin + (int64_t)c * kQ));  // used about two chunks later
      };
      auto load_b = [&](int c) {
        if (c >= 2 && !wait(sh.b_empty[c & 1], (c >> 1) - 1)) return;
        issued_b = c + 1;
        bulk::mbar_arrive_expect_tx(&sh.b_full[c & 1], 2 * kTile);
        for (int i = 0; i < 2; ++i)
          tile_load(base + kSmemB + ((c & 1) * 2 + i) * kTile, &map_b, 64 * i, job.g, (int)(job.begin + (int64_t)c * kQ), &sh.b_full[c & 1]);
      };
      auto load_c = [&](int c) {
        if (STATES) return;
        if (c >= 1 && !wait(sh.c_done, c - 1)) return;
        issued_c = c + 1;
        bulk::mbar_arrive_expect_tx(&sh.c_full, 2 * kTile);
        for (int i = 0; i < 2; ++i)
          tile_load(base + kSmemC + i * kTile, &map_c, 64 * i, job.g, (int)(job.begin + (int64_t)c * kQ), &sh.c_full);
      };
      if (chunks > 0) {
        load_x(0);
        load_b(0);
      }
      for (int c = 0; fine && c < chunks; ++c) {
        load_c(c);
        if (fine && c + 1 < chunks) {
          load_b(c + 1);
          if (fine) load_x(c + 1);
        }
      }
      // The last copies into every place have landed before anybody leaves.
      for (int c = issued_x > 3 ? issued_x - 3 : 0; c < issued_x; ++c) fine &= wait_phase(&sh.x_full[c % 3], (c / 3) & 1);
      for (int c = issued_b > 2 ? issued_b - 2 : 0; c < issued_b; ++c) fine &= wait_phase(&sh.b_full[c & 1], (c >> 1) & 1);
      if (issued_c > 0) fine &= wait_phase(&sh.c_full, (issued_c - 1) & 1);
    } else if (warp >= kWarpDecay) {
      // ---------------------------------------------------------------- decays
      const uint16_t *dt = static_cast<const uint16_t *>(p.dt) + job.h;
      const float A2 = __ldg(p.A + job.h) * kLog2e, bias = p.dt_bias != nullptr ? __ldg(p.dt_bias + job.h) : 0.0f;
      uint16_t next[4];
      auto fetch = [&](int c) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t t = job.begin + (int64_t)c * kQ + 32 * j + lane;
          next[j] = t < (job.begin + job.length) ? __ldg(dt + t * p.dt_stride_t) : (uint16_t)0;
        }
      };
      int c = warp - kWarpDecay;  // two warps take the chunks in turn
      if (c < chunks) fetch(c);
      for (; c < chunks; c += 2) {
        const uint16_t raw_dt[4] = {next[0], next[1], next[2], next[3]};
        const int rows = (int)(job.length - (int64_t)c * kQ < kQ ? job.length - (int64_t)c * kQ : kQ);
        if (c + 2 < chunks) fetch(c + 2);
        if (c >= kStages && !wait(sh.d_empty[c % kStages], c / kStages - 1)) break;
        __syncwarp();
        fill_decays(sh.decays[c % kStages], raw_dt, bias, p.dt_softplus, rows, A2, lane);
        bulk::mbar_arrive(&sh.d_full[c % kStages]);
      }
    }
  }
  if (!fine) atomicOr(p.status_dev != nullptr ? p.status_dev : &g_scan_error, kDevErrTimeout);
  __syncwarp();
  fence_before_sync();
  __syncthreads();
  if (warp == kWarpMma) {
    fence_after_sync();
    tmem_free(tmem, kColumns);
  }
}

}  // namespace

cudaError_t take_scan_error(int32_t *bits) {
  cudaError_t e = launch_overlapped(k_exchange_scan_error, dim3(1), dim3(1), 0, (cudaStream_t)0);
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(bits, g_scan_error_taken, sizeof(int32_t));
  return e;
}

cudaError_t encode_tiles(CUtensorMap *map, const void *data, int64_t inner, int64_t groups, int64_t rows, int64_t stride_group,
                         int64_t stride_row, int box_inner, int box_rows, CUtensorMapSwizzle swizzle) {
  using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                              const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                              CUtensorMapFloatOOBfill);
  static const Encode fn = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess) {
      (void)cudaGetLastError();
      return static_cast<Encode>(nullptr);
    }
    return reinterpret_cast<Encode>(f);
  }();
  if (fn == nullptr) return cudaErrorNotSupported;
  // A stride is a multiple of 16 bytes and counts only where there is more than one.
  const cuuint64_t any = (cuuint64_t)(inner * 2 + 15) / 16 * 16;
  const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)groups, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {groups > 1 ? (cuuint64_t)stride_group * 2 : any, rows > 1 ? (cuuint64_t)stride_row * 2 : any};
  const cuuint32_t box[3] = {(cuuint32_t)box_inner, 1, (cuuint32_t)box_rows}, ones[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(data), dims, strides, box, ones,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

namespace {

// Boxes of a chunk's rows x 64.
cudaError_t encode(CUtensorMap *map, const void *data, int64_t inner, int64_t groups, int64_t rows, int64_t stride_group,
                   int64_t stride_row) {
  return encode_tiles(map, data, inner, groups, rows, stride_group, stride_row, 64, kQ, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Segments of the sequences for these arguments; as many as sequences is not to cut. Cutting costs the first launch, which
// takes about half a chunk's time again, so it starts where less than half of the SMs would have work;
// segments are at least 4 chunks, and enough for about three CTAs an SM (whole waves matter less then).
Segments segments_of(const ScanParams &p, int sms) {
  const int64_t items = p.n_seq * p.H * ((p.P + 63) / 64), chunks = (p.T + kQ - 1) / kQ;
  Segments seg = {p.n_seq, INT64_MAX / 4, nullptr, nullptr};
  if (items * 2 > sms || items < 1 || chunks < 8) return seg;
  const int64_t want = 3 * sms / items * p.n_seq;   // segments in all, were all sequences alike
  int64_t length = (chunks + want - 1) / want;
  if (length < 4) length = 4;
  if (length >= chunks) return seg;
  seg.tokens = length * kQ;
  seg.count = p.T / seg.tokens + p.n_seq;
  return seg;
}

bool cut(const ScanParams &p, const Segments &seg) { return seg.count > p.n_seq; }

template <bool STATES>
cudaError_t launch_segments(const ScanParams &p, const Segments &seg, const CUtensorMap (&maps)[4], int dev, cudaStream_t stream) {
  static std::atomic<bool> opted_in[64];
  if (!opted_in[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(k_scan_chunked<STATES>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
    if (e != cudaSuccess) return e;
    opted_in[dev].store(true, std::memory_order_release);
  }
  const int blocks_p = (int)((p.P + 63) / 64);
  return launch_overlapped(k_scan_chunked<STATES>, dim3((unsigned)(seg.count * p.H * blocks_p)), dim3(kThreads), kSmemBytes,
                           stream, p, blocks_p, seg, maps[0], maps[1], maps[2], maps[3]);
}

}  // namespace

int64_t scan_chunked_workspace(const ScanParams &p, int sms) {
  const Segments seg = segments_of(p, sms);
  return cut(p, seg) ? 4 * seg.count * (p.H * p.P * p.K + p.H) : 0;
}

cudaError_t launch_scan_chunked(const ScanParams &p, cudaStream_t stream) {
  const int dev = current_device();
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  alignas(64) CUtensorMap maps[4] = {};
  if (p.T > 0) {
    cudaError_t e = encode(&maps[0], p.x, p.P, p.H, p.T, p.x_stride_h, p.x_stride_t);
    if (e == cudaSuccess) e = encode(&maps[1], p.b, p.K, p.G, p.T, p.b_stride_g, p.b_stride_t);
    if (e == cudaSuccess) e = encode(&maps[2], p.c, p.K, p.G, p.T, p.c_stride_g, p.c_stride_t);
    if (e == cudaSuccess && p.z != nullptr) e = encode(&maps[3], p.z, p.P, p.H, p.T, p.z_stride_h, p.z_stride_t);
    if (e != cudaSuccess) return e;
  }
  Segments seg = segments_of(p, device_sm_count());
  if (cut(p, seg)) {
    seg.states = static_cast<float *>(p.workspace);
    seg.decays = seg.states + seg.count * p.H * p.P * p.K;
    cudaError_t e = launch_segments<true>(p, seg, maps, dev, stream);
    const dim3 grid((unsigned)((p.H * p.P * p.K + 255) / 256), (unsigned)p.n_seq);
    if (e == cudaSuccess) e = launch_overlapped(k_scan_join, grid, dim3(256), 0, stream, p, seg);
    if (e != cudaSuccess) return e;
  }
  return launch_segments<false>(p, seg, maps, dev, stream);
}

}  // namespace ccu
