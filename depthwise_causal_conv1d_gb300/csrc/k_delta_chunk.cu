// Gated delta rule in chunks of 64 tokens on the tensor cores (ccu_gated_delta_rule, CCU_SCAN_CHUNKED).
//
// Within a chunk let c_t be the running sum of the log decays (exp(c_t - c_s) is the decay from token s to token t), b_t the strengths,
// kn and qn the keys and queries of unit length, and s the state before the chunk. A token's write u_t sees the
// writes before it:
//
//   u_t = b_t (v_t - exp(c_t) s kn_t - sum_{s<t} exp(c_t - c_s) (kn_t . kn_s) u_s)
//
// so with A[t,s] = b_t exp(c_t - c_s) (kn_t . kn_s) below the diagonal, and T = (1 + A)^-1 diag(b),
//
//   u    = T r,             r_t = v_t - exp(c_t) s kn_t
//   y_t  = exp(c_t) s qn_t + sum_{s<=t} M[t,s] u_s,     M[t,s] = exp(c_t - c_s) (qn_t . kn_s)
//   s'   = exp(c_end) s + sum_t exp(c_end - c_t) u_t (x) kn_t
//
// A CTA walks the chunks of one (sequence, head, 128 value channels). Everything is laid out with the value channels along
// the lanes of TMEM, so that what one product gives is the next one's operand after a pass through registers, and no
// tile is turned around:
//
//   G[q|k, s]  = [Q; K] K^T          128 x 64, from shared memory: both (q . k) and (k . k)
//   KS[v, t]   = s K^T               s in three BF16 terms, in TMEM
//   QS[v, t]   = s Q^T               the same terms
//   U[v, t]    = V^T T^T + R T^T     T in three terms in shared memory; R = -exp(c_t) KS in three, in TMEM
//   D[v, k]    = (w U) K             w_t = exp(c_end - c_t), w U in three terms, in TMEM
//   O[v, t]    = QS exp(c_t) + U M^T U and M in three terms each
//
// K and Q stay as they came: their lengths are a token's factor, like the decays, and go into T, M, r and w.
//
// Rounding. The state is FP32, in registers, and everything that goes into it (s K^T, T, r, w U) is split into three BF16 terms (24
// bits), products of two such factors being six products. So is what only an output sees (s Q^T, M, U):
// an output can be the small difference of two large sums (a write that replaces what a large state holds along a key), where 16 bits of the factors
// show: 64 tokens of one key on a state 16384 times the values, two terms 62 steps of 2^-24 of the state off in the mean square, three 5. They cost 5 to
// 7 % (8 x 4096 tokens 564 us with two, 16384 tokens 884).
// Running sums are held in two floats each: a difference of sums over many fast decays would lose what neighbours differ by.
//
// The inverse: blocks of 8 on the diagonal by rows (T[t] = e_t - sum_{s<t} A[t,s] T[s], a column a lane), then two blocks to one, three times:
// the lower left of (X 0; A Y)^-1 is -Y^-1 A X^-1.
//
// What is not finite must reach no earlier token, and in the products every token meets every other through zeros: such values of V are
// taken out of the tile and their channel's outputs made NaN from there on; a key (or a gate that is NaN) ends all channels so. An infinity
// thus gives NaN where the formula may give an infinity.
//
// One CTA an SM, its 24 warps in roles that meet at mbarriers:
//
//   0..7    the chunk ahead, two groups of four that take the chunks in turn: lengths of k, M and A from G, the inverse, to shared memory as operands
//   8..15   the chain s -> KS -> R -> U -> w U -> D -> s: 64 states or 32 tokens of a channel a thread
//   16..19  the outputs, turned to rows of tokens through the place of V
//   20      the products but G, by one thread
//   21      the copies (TMA, zero-filled past P and K), and the next ones into L2
//   22      the decays and strengths, a chunk ahead, and the check of V
//   23      G, as early as Q and K are there, and the queries' lengths
//
// TMEM (512 columns): s in three terms 192, where w U (96), the third term of U (32) and U (64) come later; O 64; KS, later two terms of U, 64; D, before it R, 128;
// G 64. Shared memory 224 KB of 227: Q and K 2 x 32, V 2 x 16, T 2 x 24 (A waits in its place), M 2 x 24, the inverse's halves 2 x 9 (the corner between them goes
// from registers into T), four chunks' decays and the barriers 13, alignment 1.
//
// What bounds it: the chain of a chunk, six products and five passes through registers one after the other, some 10 thousand cycles; on a full
// card also fetching instructions (one request of nine, with two turns of six, misses the cache; loops here are rolled where a role has time, which made
// the batch faster and a single CTA slower). 8 sequences of 4096 tokens, 32 heads of 128 channels, 128 states: 597 us, 1010 TFLOP/s of
// issued BF16 products, 1.4 TB/s. One sequence of 16384 tokens: 949 us in segments (below), 1259 without.
//
// Left out, each built and timed at those two sizes (then 699 and 1206 us): all eight warps of the first role on one chunk, 1285 us the long one; the inverse in one loop over its block sizes,
// to save code, 1334 and 699; 16 warps for the chain, slower in both; KS and QS as one product of 128 columns, which holds
// KS back; mma.sync for the inverse's products (a block of 32 takes 1400 cycles instead of 240, waiting for tcgen05).
//
// Every wait has a limit; a role that runs into it reports CCU_DEVERR_TIMEOUT and ends, and so do the others.
#include <atomic>
#include <cstddef>

#include "ssm_tensor.cuh"

namespace ccu {

int current_device();
int device_sm_count();

__device__ int32_t g_delta_error = 0;        // CCU_DEVERR_* bits of calls without a status word
__device__ int32_t g_delta_error_taken = 0;  // the value the last exchange read

__global__ void k_exchange_delta_error() {
  grid_dependency_boundary();
  g_delta_error_taken = atomicExch(&g_delta_error, 0);
}

namespace {

using namespace tensor;

constexpr int kC = 64;                       // tokens a chunk
constexpr int kV = 128;                      // value channels a CTA
constexpr int kPad = kC + 4, kPadInv = 36;   // floats a row of A and of the inverse's halves: rows 4 banks apart, 8 of them for 16-byte accesses
constexpr int kTile = kC * 128;              // 64 rows of 128 bytes: 8 KB
constexpr int kWarpsPrep = 8 /* 0..7 */, kWarpsChain = 16 /* 8..15 */, kWarpMma = 20 /* out: 16..19 */, kWarpCopy = 21, kWarpDecay = 22, kWarpG = 23;
constexpr int kThreads = 24 * 32;
// Registers a thread: the launch's, and after the roles have parted; two of the six warpgroups are the chain.
constexpr int kRegs = 80, kRegsChain = 112, kRegsOther = 64;
static_assert(2 * kRegsChain + 4 * kRegsOther <= 6 * kRegs, "a share above the launch's total would be waited for forever");
// TMEM: the terms of s, where w U (96), the third term of U (32) and U (the last 64) come later; O; KS, later two terms of U; D, before it R; G.
constexpr int kColA = 0, kColUThird = 96, kColU = 128, kColO = 192, kColKS = 256, kColD = 320, kColG = 448, kColumns = 512;
constexpr int kStages = 4;                   // chunks of decays
constexpr int kSorted = 64;                  // sequences that are put in order by length
constexpr int kMaxCuts = 256;
constexpr float kLog2e = 1.4426950408889634f;
// exp2 of anything below -150 is zero in FP32; sums of steps stay finite and small with this floor.
constexpr float kLeast = -300.0f;

struct alignas(16) Tokens {                  // read in 16-byte vectors
  float sum[kC], rest[kC];                   // running sum of log2 decays: sum + rest
  float beta[kC], in[kC], left[kC];          // strength; exp(c_t); exp(c_end - c_t)
  float half[kC];                            // exp(c_31 - c_t) of the first 32, exp(c_t - c_31) of the others
  float key[kC];                             // 1 / |k_t|
  float near[kC / 2];                        // half / |k_t|
  float minus[kC], weight[kC];               // -exp(c_t) / |k_t|; exp(c_end - c_t) / |k_t|
  float query[kC];                           // 1 / |q_t|; the scale comes after it: their product need not be a float
  int bad[kV];                               // first token with a non-finite v, a channel
  int bad_all;                               // first token whose key or gates are not finite
  float decay;                               // exp(c_end)
};

// What a CTA works on. Read from shared memory by the roles: held in registers from the start, it would make them spill.
struct Job {
  int64_t begin, length, h, p0;
  const float *from;            // the state to start from, or NULL: zeros, or with `unit` the unit matrix
  float *to;                    // where the state goes, or NULL: nowhere
  int g, np;                    // group; rows of the state (value channels)
  bool unit, outputs;
};

// A part of an item that a CTA does at a time; as the plan has it, in 16-byte vectors.
struct alignas(16) Piece {
  int b, j, cut;         // sequence, item of it (head and block of channels); where its state is handed on, -1: a whole item
  int first, count;      // chunks; none: there is no such piece
  int late;              // the last tokens: waits for the first ones
  int unused[2];
};

struct alignas(16) Shared {
  Tokens tokens[kStages];
  uint64_t d_full[kStages], d_empty[kStages];
  uint64_t qk_full[2], v_full[2], qk_empty[2], v_empty[2], norm_ready[2], q_ready[2], t_ready[2], m_ready[2], g_full[2], o_done[2], v_ready[2], s_ready[2], s_full[2];
  uint64_t g_empty, ks_full, r_ready, u_full, wu_ready, u_ready, qs_full, qs_scaled, o_full, o_empty, drained, g_drained;
  Job job;
  uint32_t tmem;
  int lengths[kSorted], found, arrived;
};

constexpr int kSmemQK = 0, kSmemV = 8 * kTile, kSmemT = 12 * kTile, kSmemM = 18 * kTile, kSmemInv = 24 * kTile,
              kSmemShared = kSmemInv + 2 * 2 * 32 * kPadInv * 4;
constexpr size_t kSmemBytes = kSmemShared + sizeof(Shared) + 1024;
static_assert(sizeof(Tokens) % 16 == 0, "vectors");
static_assert(kSmemBytes <= 227 * 1024, "shared memory of a CTA");

// The warps of the first and of the third role meet at named barriers, which all of them reach whatever became of their waits; they leave
// their loops together.
__device__ __forceinline__ void meet(int id, int threads) {
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ bool meet_and(int id, int threads, bool v) {  // whether it is true for all of them
  uint32_t all;
  __syncwarp();
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
               : "=r"(all)
               : "r"((uint32_t)v), "r"(id), "r"(threads)
               : "memory");
  return all != 0;
}

__device__ __forceinline__ float4 read4(const float *p) { return *reinterpret_cast<const float4 *>(p); }

// 16 columns of a lane, times `f` (or as they are), as three BF16 terms (8 columns each, `stride` apart, the third at `third`). Eight at a time:
// registers are scarce.
__device__ __forceinline__ void put_terms(uint32_t addr, uint32_t stride, uint32_t third, const float *v, const float *f = nullptr) {
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t a[4], b[4], c[4];
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const float *e = v + 8 * half + 2 * i;
      float2 x = make_float2(e[0], e[1]), y = make_float2(e[2], e[3]);
      if (f != nullptr) {
        const float4 m = read4(f + 8 * half + 2 * i);
        x = __fmul2_rn(x, make_float2(m.x, m.y));
        y = __fmul2_rn(y, make_float2(m.z, m.w));
      }
      split3_signs(x, a[i], b[i], c[i]);
      split3_signs(y, a[i + 1], b[i + 1], c[i + 1]);
    }
    tmem_store4(addr + 4 * half, a);
    tmem_store4(addr + stride + 4 * half, b);
    tmem_store4(third + 4 * half, c);
  }
}

// A B for blocks of floats in shared memory, of ROWS rows and 8 columns, K from `first` to `last` (multiples of 4): a lane has a row (the first
// lanes of ROWS) and ROWS / 4 columns. A is a part of the chunk's A, B of the inverse: A[m][k] is at a[k * kPad + m], B[k][n] at b[k * kPadInv + n]; or, with
// INVERSE, A of the inverse and B what was put into A's place: a[m * kPadInv + k], b[k * kPad + n]. In FP32 on the
// ordinary pipes: mma.sync has to wait for what tcgen05 is at (a block of 32 took 1400 cycles instead of 240).
template <int ROWS, bool INVERSE>
__device__ __forceinline__ void block_product(float2 (&d)[ROWS / 8], const float *a, const float *b, int first, int last, int lane) {
  constexpr int N = ROWS / 8;  // pairs of columns
  constexpr int kPadB = INVERSE ? kPad : kPadInv;
  const int m = lane % ROWS;
  b += lane / ROWS * 2 * N;
#pragma unroll
  for (int i = 0; i < N; ++i) d[i] = make_float2(0.0f, 0.0f);
#pragma unroll 2
  for (int k = first; k < last; k += 4) {
    float e[4];
    if (INVERSE) {
      const float4 x = read4(a + m * kPadInv + k);
      e[0] = x.x, e[1] = x.y, e[2] = x.z, e[3] = x.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) e[j] = a[(k + j) * kPad + m];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float *q = b + (k + j) * kPadB;
      const float2 x = make_float2(e[j], e[j]);
      if constexpr (N == 1) {
        d[0] = __ffma2_rn(x, *reinterpret_cast<const float2 *>(q), d[0]);
      } else {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          const float4 y = read4(q + 2 * i);
          d[i] = __ffma2_rn(x, make_float2(y.x, y.y), d[i]);
          d[i + 1] = __ffma2_rn(x, make_float2(y.z, y.w), d[i + 1]);
        }
      }
    }
  }
}
// Its result, times `sign`, to rows of PAD floats.
template <int ROWS, int PAD>
__device__ __forceinline__ void put_block(float *to, const float2 (&d)[ROWS / 8], float sign, int lane) {
  to += lane % ROWS * PAD + lane / ROWS * (ROWS / 4);
  if constexpr (ROWS == 8) {
    *reinterpret_cast<float2 *>(to) = make_float2(sign * d[0].x, sign * d[0].y);
  } else {
#pragma unroll
    for (int i = 0; i < ROWS / 8; i += 2)
      *reinterpret_cast<float4 *>(to + 2 * i) = make_float4(sign * d[i].x, sign * d[i].y, sign * d[i + 1].x, sign * d[i + 1].y);
  }
}

// A sum in two floats plus another.
__device__ __forceinline__ void add_exact(float &hi, float &lo, float hi2, float lo2) {
  const float s = hi + hi2, t = s - hi;
  lo = (lo + lo2) + ((hi - (s - t)) + (hi2 - t));
  hi = s;
}

// A chunk's decays and strengths, by one warp: lane l takes tokens 2 l and 2 l + 1; tokens from `rows` on are past the sequence's end: no
// step, and no strength.
__device__ __forceinline__ void fill_tokens(Tokens &t, uint32_t a, uint32_t b, float bias, float A2, int rows, int lane) {
  const unsigned full = 0xffffffffu;
  int bad = kC;
#pragma unroll 1
  for (int row = 2 * lane; row < 2 * lane + 2; ++row, a >>= 16, b >>= 16) {
    float step = step_of(first_of(a) + bias, 1) * A2, beta = sigmoid(first_of(b));
    if (row >= rows) step = beta = 0.0f;
    if (step != step || beta != beta) {  // this token's, and all later outputs are NaN
      bad = bad < row ? bad : row;
      step = beta = 0.0f;
    }
    t.sum[row] = step < kLeast ? kLeast : step;
    t.beta[row] = beta;
  }
  const float2 own = *reinterpret_cast<const float2 *>(t.sum + 2 * lane);
  float hi = own.x, lo = 0.0f;  // up to this lane's second token
  add_exact(hi, lo, own.y, 0.0f);
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const float u = __shfl_up_sync(full, hi, o), w = __shfl_up_sync(full, lo, o);
    if (lane >= o) add_exact(hi, lo, u, w);
  }
  const float mid_hi = __shfl_sync(full, hi, 15), mid_lo = __shfl_sync(full, lo, 15), end = __shfl_sync(full, hi, 31), end_lo = __shfl_sync(full, lo, 31);
#pragma unroll 1
  for (int row = 2 * lane + 1; row >= 2 * lane; --row) {
    t.sum[row] = hi;
    t.rest[row] = lo;
    t.in[row] = ex2_approx_ftz(hi + lo);
    t.left[row] = ex2_approx_ftz((end - hi) + (end_lo - lo));
    const float mid = (hi - mid_hi) + (lo - mid_lo);
    t.half[row] = ex2_approx_ftz(lane < 16 ? -mid : mid);
    add_exact(hi, lo, -own.y, 0.0f);  // up to its first token
  }
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) bad = min(bad, __shfl_xor_sync(full, bad, o));
#pragma unroll 1
  for (int i = lane; i < kV; i += 32) t.bad[i] = kC;
  if (lane == 0) {
    t.bad_all = bad;
    t.decay = ex2_approx_ftz(end + end_lo);
  }
}

// How sequences are cut when there are too few of them, and heads, to fill the card: segments of `tokens` (a multiple of the chunk). A
// segment's writes are linear in the state before it: after it, the state is s Phi + W, with W what it makes of no state and Phi (K x K) what it
// makes of the unit matrix, with no values. So a first launch runs every sequence's first segment, W of the ones between and Phi of
// them, a small one joins them to the states before the segments, and a second runs all segments but the first.
//
// The lengths are on the device, so segments are numbered from the offsets: sequence b has the numbers from
// first_segment(b) on, of which it needs ceil(length / tokens), or one when it is empty, and never more than there are up to
// first_segment(b + 1). `count` = T / tokens + sequences bounds them all.
struct Segments {
  int64_t count, tokens;
  float *states;  // [segment][H, P, K]: before the segment (from a sequence's third on W of the one before, until they are joined)
  float *maps;    // [segment][H, K, K]: Phi
};
enum Pass { kFirst, kRest };

__device__ __forceinline__ int64_t first_segment(const DeltaParams &p, const Segments &seg, int64_t b) {
  const int64_t t = __ldg(p.cu_seqlens + b);
  return (t < 0 ? 0 : t > p.T ? p.T : t) / seg.tokens + b;
}

// The states before the segments, a sequence's in order: 16 rows of one head a CTA, a column a thread (two threads share one, 8 rows each).
// 3 segments of 32 heads, 128 x 128: the products are 1 us of the card's FP32 work, the chain of loads under them more.
constexpr int kJoinRows = 16;
__global__ void __launch_bounds__(2 * kV) k_delta_join(DeltaParams p, Segments seg) {
  grid_dependency_boundary();
  __shared__ float before[kJoinRows][kV];
  const int64_t row0 = (int64_t)blockIdx.x * kJoinRows, h = blockIdx.y, b = blockIdx.z;
  if (slot_of(p.indices, b, p.S, nullptr, false) < 0) return;  // padding: nothing was written
  const Bounds q = sequence_bounds(p.cu_seqlens, b, p.T);
  const int64_t parts = (q.end - q.begin + seg.tokens - 1) / seg.tokens, first = first_segment(p, seg, b);
  const int k = threadIdx.x & (kV - 1), r0 = (threadIdx.x >> 7) * (kJoinRows / 2), K = (int)p.K;
  auto entry = [&](int64_t j, int r) { return seg.states + (((first + j) * p.H + h) * p.P + row0 + r) * p.K + k; };
  float v[kJoinRows / 2];
  for (int64_t j = 1; j + 1 < parts; ++j) {
    if (j == 1) {
#pragma unroll
      for (int r = 0; r < kJoinRows / 2; ++r) v[r] = row0 + r0 + r < p.P && k < K ? *entry(1, r0 + r) : 0.0f;
    }
#pragma unroll
    for (int r = 0; r < kJoinRows / 2; ++r) before[r0 + r][k] = v[r];
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kJoinRows / 2; ++r) v[r] = row0 + r0 + r < p.P && k < K ? *entry(j + 1, r0 + r) : 0.0f;
    const float *map = seg.maps + ((first + j) * p.H + h) * p.K * p.K + k;
    for (int i0 = 0; i0 < K; i0 += 32) {  // K is a multiple of 8
      float m[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) m[i] = i0 + i < K && k < K ? map[(int64_t)(i0 + i) * K] : 0.0f;
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (i0 + i < K) {
#pragma unroll
          for (int r = 0; r < kJoinRows / 2; ++r) v[r] = fmaf(before[r0 + r][i0 + i], m[i], v[r]);
        }
    }
#pragma unroll
    for (int r = 0; r < kJoinRows / 2; ++r)
      if (row0 + r0 + r < p.P && k < K) *entry(j + 1, r0 + r) = v[r];
    __syncthreads();
  }
}

// The sequence that comes `at`th by length, longest first: CTAs start in the order of their numbers, and a long sequence that starts
// last is waited for by an idle card. Equal lengths keep their order.
__device__ int longest(const DeltaParams &p, int at, int *lengths, int *found) {
  const int i = threadIdx.x, n = (int)p.n_seq;
  if (i < n) {
    const Bounds q = sequence_bounds(p.cu_seqlens, i, p.T);
    lengths[i] = (int)(q.end - q.begin);
  }
  __syncthreads();
  if (i < n) {
    const int mine = lengths[i];
    int before = 0;
    for (int j = 0; j < n; ++j) before += lengths[j] > mine || (lengths[j] == mine && j < i);
    if (before == at) *found = i;
  }
  __syncthreads();
  return *found;
}

// Even shares, where there are more items (sequence, head, block of channels) than SMs, and not a multiple of them. Think of all items one
// after the other on a line, longest sequences first, cut into as many equal shares as there are SMs (a share is no shorter than the longest
// sequence). With clusters an item is two of one sequence, and a share that of two SMs. An item over a border is done in two pieces: its
// first tokens at the start of one SM's time, its last ones at the end of another's, and since it is no longer than a share, one piece is
// done before the other begins. So CTAs take, in this order: the first pieces; whole items; the last pieces, longest first. They take them by a ticket, so that whoever waits for a first piece knows it to be on an SM
// already, and hand the state on through the workspace. The same chunks give the same bits, cut or not. A kernel of one CTA makes the plan:
// made by every CTA for itself it took 6 us each.
struct Shares {
  int *ticket, *flags;  // of the workspace: zeros when the kernel starts
  Piece *plan;          // [items + SMs - 1]
  float *states;        // [cut][kV, K]
  int sms, pair;        // CTAs of a cluster: items that go together
};
constexpr int kMaxItems = 2048;  // more have so many turns that the last one's idle SMs do not count
constexpr int kShareHeader = 2048;  // bytes: the ticket, and flags from its 64th on; then the plan
constexpr int kLeastPiece = 2;      // chunks: a shorter one is not worth a CTA's start
static_assert(256 + 4 * kMaxCuts <= kShareHeader, "the ticket and the flags");

__global__ void __launch_bounds__(1024) k_delta_plan(DeltaParams p, int blocks_p, Shares sharing) {
  grid_dependency_boundary();
  __shared__ int given[kSorted], lengths[kSorted], order[kSorted], left_of[kMaxCuts], number_of[kMaxCuts];
  const int tid = threadIdx.x, n = (int)p.n_seq, pair = sharing.pair;
  const int each = (int)p.H * blocks_p / pair, items = n * each, sms = sharing.sms / pair, most = sms - 1;  // counted in pairs
  for (int i = tid; i < kShareHeader / 4; i += 1024) sharing.ticket[i] = 0;
  if (tid < n) {
    const Bounds q = sequence_bounds(p.cu_seqlens, tid, p.T);
    given[tid] = q.end > q.begin ? (int)((q.end - q.begin + kC - 1) / kC) : 1;
  }
  __syncthreads();
  if (tid < n) {
    const int mine = given[tid];
    int place = 0;
    for (int j = 0; j < n; ++j) place += given[j] > mine || (given[j] == mine && j < tid);
    order[place] = tid;
    lengths[place] = mine;
  }
  __syncthreads();
  int total = 0;
  for (int r = 0; r < n; ++r) total += lengths[r];
  total *= each;
  const int even = (total + sms - 1) / sms, share = even > lengths[0] ? even : lengths[0];
  // A cut a thread: the item on the line over the end of its share, and how much of that is left of it
  int r = 0, left = 0, j = 0, length = 0;
  if (tid < most) {
    int where = (tid + 1) * share;
    if (where < total) {
      for (; r < n - 1 && where >= lengths[r] * each; ++r) where -= lengths[r] * each;
      length = lengths[r];
      j = where / length;
      left = where - j * length;
      if (left < kLeastPiece || length - left < kLeastPiece) left = 0;
    }
    left_of[tid] = left;
    number_of[tid] = r * each + j;
  }
  const int cuts = __syncthreads_count(left > 0);
  if (left > 0) {
    int before = 0, longer = 0;
    for (int i = 0; i < most; ++i) {
      before += left_of[i] > 0 && i < tid;
      longer += left_of[i] > left || (left_of[i] == left && i < tid);
    }
    sharing.plan[before] = {order[r], pair * j, pair * tid, 0, length - left, 0};
    sharing.plan[items + longer] = {order[r], pair * j, pair * tid, length - left, left, 1};
  }
  for (int item = tid; item < items; item += 1024) {  // whole ones, in the order of the line
    int before = 0;
    bool cut = false;
    for (int i = 0; i < most; ++i) {
      before += left_of[i] > 0 && number_of[i] < item;
      cut |= left_of[i] > 0 && number_of[i] == item;
    }
    r = item / each;
    j = item - r * each;
    if (!cut) sharing.plan[cuts + item - before] = {order[r], pair * j, -1, 0, lengths[r], 0};
  }
  for (int i = items + cuts + tid; i < items + most; i += 1024) sharing.plan[i] = {};
}

// The two CTAs of a cluster: rank, a word into the other's shared memory (of a CTA that has started: behind a barrier), a barrier after which
// it is seen there.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void put_in_cluster(const void *here, uint32_t rank, int v) {
  uint32_t there;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(bulk::smem_addr(here)), "r"(rank));
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(there), "r"(v) : "memory");
}
__device__ __forceinline__ void meet_cluster() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Waits until the first piece has left its state; false: it gave up, after some seconds.
__device__ int wait_flag(const int *flag) {
  for (uint32_t i = 0; i < 1u << 22; ++i) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(flag) : "memory");
    if (v != 0) return 1;
    __nanosleep(1000);
  }
  return 0;
}

// Kinds of launches: whole sequences; one of the two over segments; even shares.
enum Mode { kWhole, kSegments, kShares };
template <int MODE>
__global__ void __launch_bounds__(kThreads, 1) k_delta_chunked(DeltaParams p, int blocks_p, Segments seg, Shares sharing, int pass,
                                                               const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                                                               const __grid_constant__ CUtensorMap map_v) {
  grid_dependency_boundary();
  constexpr bool PARTS = MODE == kSegments, SHARES = MODE == kShares;
  extern __shared__ unsigned char raw[];
  const uint32_t base = (bulk::smem_addr(raw) + 1023) & ~1023u;
  unsigned char *aligned_raw = raw + (base - bulk::smem_addr(raw));
  Shared &sh = *reinterpret_cast<Shared *>(aligned_raw + kSmemShared);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int quarter = warp & 3, row = quarter * 32 + lane;  // lane of TMEM of a thread in the first three roles
  int64_t item = blockIdx.x;
  Piece piece = {};
  if constexpr (SHARES) {
    const int rank = sharing.pair > 1 ? (int)cluster_rank() : 0;
    if (sharing.pair > 1) meet_cluster();  // the other CTA has started: until then its shared memory is not to be written
    if (tid == 0 && rank == 0) {
      const int at = atomicAdd(sharing.ticket, 1);  // as many as there are places in the plan
      sh.found = at;
      if (sharing.pair > 1) put_in_cluster(&sh.found, 1, at);
    }
    if (sharing.pair > 1) meet_cluster();
    __syncthreads();
    piece = sharing.plan[sh.found];
    if (piece.count == 0) return;
    piece.j += rank;
    piece.cut += piece.cut >= 0 ? rank : 0;
  }
  // A block of channels, or Phi. Over segments heads come first: a pair of CTAs is two heads of one kind, which come and go together
  const int kinds = PARTS && pass == kFirst ? blocks_p + 1 : blocks_p;
  const int kind = SHARES ? piece.j % blocks_p : (int)(PARTS ? item / p.H % kinds : item % kinds);
  const int64_t h = SHARES ? piece.j / blocks_p : PARTS ? item % p.H : item / kinds % p.H;
  item /= kinds * p.H;
  int64_t b = SHARES ? piece.b : item, part = 0;     // this CTA's segment, of sequence b
  if constexpr (PARTS) {
    int64_t past = p.n_seq;
    for (b = 0; past - b > 1;) {
      const int64_t mid = (b + past) >> 1;
      if (first_segment(p, seg, mid) <= item) b = mid; else past = mid;
    }
    part = item - first_segment(p, seg, b);
    if (part < (pass == kRest)) return;              // rows before the first sequence; first segments are done
  } else if (!SHARES && p.n_seq > 1 && p.n_seq <= kSorted) {
    b = longest(p, (int)b, sh.lengths, &sh.found);
  }
  const bool unit = PARTS && kind == blocks_p;
  const int K = (int)p.K;
  const int64_t p0 = unit ? 0 : (int64_t)kind * kV;
  const int np = unit ? K : (int)(p.P - p0 < kV ? p.P - p0 : kV);
  Bounds bounds = sequence_bounds(p.cu_seqlens, b, p.T);
  bool last = true;
  if constexpr (PARTS) {
    bounds.begin += part * seg.tokens;
    if (part > 0 && bounds.begin >= bounds.end) return;
    last = bounds.end - bounds.begin <= seg.tokens;
    if (!last) bounds.end = bounds.begin + seg.tokens;
    if (pass == kFirst && (part > 0 ? last : unit)) return;  // nothing starts from its state; the first state is known
  }
  if constexpr (SHARES) {
    if (piece.cut >= 0 && !piece.late) bounds.end = bounds.begin + (int64_t)piece.count * kC;
    bounds.begin += (int64_t)piece.first * kC;
  }
  const bool outputs = !PARTS || pass != kFirst || part == 0;
  const int64_t s = slot_of(p.indices, b, p.S, p.status_dev, tid == 0 && h == 0 && kind == 0 && part == 0 && !piece.late);
  uint16_t *out = static_cast<uint16_t *>(p.out) + h * p.out_stride_h + p0;
  if (s < 0) {
    const int piece = tid & 15;
    if (outputs && 8 * piece < np)
      for (int64_t t = bounds.begin + (tid >> 4); t < bounds.end; t += kThreads / 16) st_stream(out + t * p.out_stride_t + 8 * piece, make_uint4(0, 0, 0, 0));
    return;
  }
  if (warp == kWarpMma) tmem_alloc(&sh.tmem, kColumns);
  if (tid == 0) {
    const int64_t at = (h * p.P + p0) * p.K;
    float *slot = p.state + s * p.state_stride_s + at, *entry = seg.states + item * p.H * p.P * p.K + at;  // the state before this segment
    const bool initial = p.has_initial != nullptr && __ldg(p.has_initial + b) != 0;
    const float *from = part == 0 ? (initial ? slot : nullptr) : PARTS && pass == kRest ? entry : nullptr;
    float *to = unit ? seg.maps + (item * p.H + h) * p.K * p.K : last ? slot : entry + p.H * p.P * p.K;
    if (PARTS && pass == kRest && !last) to = nullptr;  // the next segment's CTA starts from the joined state that stands there, at any time of this launch
    if constexpr (SHARES) {
      sh.arrived = 1;
      if (piece.cut >= 0) {
        float *handed = sharing.states + (int64_t)piece.cut * kV * p.K;
        if (!piece.late) to = handed;
        else from = handed, sh.arrived = wait_flag(sharing.flags + piece.cut);
      }
    }
    sh.job = {bounds.begin, bounds.end - bounds.begin, h, p0, from, to, (int)(h / (p.H / p.G)), np, unit, outputs};
    for (int i = 0; i < kStages; ++i) {
      bulk::mbar_init(&sh.d_full[i], 32);
      bulk::mbar_init(&sh.d_empty[i], 16);  // the warps of the first three roles
    }
    for (int i = 0; i < 2; ++i) {
      bulk::mbar_init(&sh.qk_full[i], 1);
      bulk::mbar_init(&sh.v_full[i], 1);
      bulk::mbar_init(&sh.qk_empty[i], 1);
      bulk::mbar_init(&sh.v_empty[i], 4);
      bulk::mbar_init(&sh.norm_ready[i], 4);
      bulk::mbar_init(&sh.q_ready[i], 1);
      bulk::mbar_init(&sh.o_done[i], 1);
      bulk::mbar_init(&sh.t_ready[i], 4);
      bulk::mbar_init(&sh.m_ready[i], 2);
    }
    uint64_t *ones[] = {&sh.g_full[0], &sh.g_full[1], &sh.ks_full, &sh.u_full, &sh.s_full[0], &sh.s_full[1], &sh.v_ready[0], &sh.v_ready[1], &sh.qs_full, &sh.o_full, &sh.drained, &sh.g_drained};
    for (uint64_t *bar : ones) bulk::mbar_init(bar, 1);
    bulk::mbar_init(&sh.g_empty, 4);
    uint64_t *fours[] = {&sh.s_ready[0], &sh.s_ready[1], &sh.qs_scaled, &sh.o_empty};
    for (uint64_t *bar : fours) bulk::mbar_init(bar, 4);
    uint64_t *chain[] = {&sh.r_ready, &sh.wu_ready, &sh.u_ready};
    for (uint64_t *bar : chain) bulk::mbar_init(bar, 8);
    bulk::fence_mbar_init();
  }
  // The columns from 32 on of M are zero in its first 32 rows, and the inverse above its blocks of 8: nobody writes them again.
  for (int i = tid; i < 6 * kTile / 16; i += kThreads) sts128(base + kSmemM + 16 * i, make_uint4(0, 0, 0, 0));
  for (int i = tid; i < 2 * 2 * 32 * kPadInv / 4; i += kThreads) sts128(base + kSmemInv + 16 * i, make_uint4(0, 0, 0, 0));
  if (PARTS && unit)  // no values
    for (int i = tid; i < 4 * kTile / 16; i += kThreads) sts128(base + kSmemV + 16 * i, make_uint4(0, 0, 0, 0));
  bulk::fence_proxy_async();
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const Job &job = sh.job;
  const int chunks = (int)((job.length + kC - 1) / kC);
  const uint32_t tmem = sh.tmem, mine = tmem + ((uint32_t)(quarter * 32) << 16);
  bool fine = !SHARES || sh.arrived != 0;
  // Waits for a barrier's phase number n (counted from 0); false when it gave up, now or before.
  auto wait = [&](uint64_t &bar, int n) { return fine = fine && wait_phase(&bar, n & 1); };
  auto wait2 = [&](uint64_t &bar, int n, uint64_t &also, int m) { return fine = fine && wait_phases(&bar, n & 1, &also, m & 1); };
  auto arrive = [&](uint64_t &bar) {  // one arrival a warp, for what all its lanes have done
    __syncwarp();
    if (lane == 0) bulk::mbar_arrive(&bar);
  };
  auto rows_of = [&](int c) { return (int)(job.length - (int64_t)c * kC < kC ? job.length - (int64_t)c * kC : kC); };

  if (warp >= kWarpsPrep && warp < kWarpsChain)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsChain));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
  if (warp < kWarpsPrep) {
    // ---------------------------------------------------------------- the chunk ahead
    const bool keys = row >= kC;           // this thread's row of [Q; K]
    const int t = row & (kC - 1);
    const int group = warp >> 2, part = warp & 3;  // two groups of four warps take the chunks in turn: one's work takes longer than a chunk
    const int diagonal = t >> 5;
    // A waits in the place of T that will be made from it, the halves of the inverse (two blocks of 32 on its diagonal) in the group's own. The
    // corner between the halves goes into T from registers.
    float *at = reinterpret_cast<float *>(aligned_raw + kSmemT + group * 3 * kTile), *inv = reinterpret_cast<float *>(aligned_raw + kSmemInv) + group * 2 * 32 * kPadInv;
    static_assert(kC * kPad * 4 <= 3 * kTile, "A in the place of T");
    auto meet_group = [&] { meet(2 + group, 128); };
    // A wait that ran out is noted, and all warps of the group leave together at the next turn.
    for (int c = group; c < chunks && meet_and(2 + group, 128, fine); c += 2) {
      Tokens &now = sh.tokens[c % kStages];
      const int rows = rows_of(c);
      wait2(sh.d_full[c % kStages], c / kStages, sh.g_full[c & 1], c >> 1);
      // M of two chunks before has been read, and nobody waits any more for what that chunk's role had to say
      if (c >= 2) wait(sh.o_done[c & 1], (c >> 1) - 1);
      __syncwarp();
      fence_after_sync();
      if (keys) {  // a key's squares are on the diagonal of G
        float sum = 0.0f;
#pragma unroll 1
        for (int i = 0; i < 32; i += 8) {
          float v[8];
          tmem_load8(mine + kColG + 32 * diagonal + i, v);
          wait_loads();
          loaded(v);
#pragma unroll
          for (int j = 0; j < 8; ++j) sum = lane == i + j ? v[j] : sum;
        }
        if (t >= rows || !(sum < INFINITY)) {
          // A row of another sequence, or a key that is not finite or whose squares overflow (products of two such would): it would reach
          // earlier tokens through the zeros of T, so it is taken out of the tile, and all outputs from there on are NaN.
          if (t < rows) atomicMin(&now.bad_all, t);
          sum = 0.0f;
          wait(sh.qk_full[c & 1], c >> 1);
          const uint32_t tile = base + kSmemQK + (c & 1) * 4 * kTile + kTile;  // blocks of 64 entries are 2 kTile apart
#pragma unroll 1
          for (int i = 0; i < K / 8; ++i) sts128(tile + (i >> 3) * 2 * kTile + swizzled(t, i & 7), make_uint4(0, 0, 0, 0));
          bulk::fence_proxy_async();
        }
        const float length = p.qk_norm ? rsqrtf(sum + kUnitEps) : 1.0f;
        now.key[t] = length;
        now.minus[t] = -now.in[t] * length;
        now.weight[t] = now.left[t] * length;
        if (t < kC / 2) now.near[t] = now.half[t] * length;
      }
      arrive(sh.norm_ready[c & 1]);
      meet_group();
      const float factor = keys ? now.beta[t] * now.key[t] : 1.0f;
      // Rows past the sequence's end, and from a token on whose key or gates are not finite, are left out: G holds what came there.
      const int cut = min(rows, now.bad_all), before = t < cut ? t + (keys ? 0 : 1) : 0;
      const uint32_t m_row = base + kSmemM + (c & 1) * 3 * kTile;
      const float2 sum_t = make_float2(now.sum[t], now.sum[t]), rest_t = make_float2(now.rest[t], now.rest[t]), minus = make_float2(-1.0f, -1.0f);
      const float far = before > 0 ? now.half[t] * factor : 0.0f;
      const float2 factors = make_float2(factor, factor), fars = make_float2(far, far);
      // 8 columns at a time. The first 32 rows have nothing in the others: zeros since the start.
#pragma unroll 1
      for (int s0 = 0; (!PARTS || keys || job.outputs) && s0 < 32 * (1 + diagonal); s0 += 8) {
        float v[8];
        tmem_load8(mine + kColG + s0, v);
        wait_loads();
        loaded(v);
        if (s0 >= 32 * diagonal) {
#pragma unroll
          for (int i = 0; i < 8; i += 4) {
            const float4 hi = read4(now.sum + s0 + i), lo = read4(now.rest + s0 + i), len = read4(now.key + s0 + i);
            const float2 a = __fadd2_rn(__ffma2_rn(make_float2(hi.x, hi.y), minus, sum_t), __ffma2_rn(make_float2(lo.x, lo.y), minus, rest_t));
            const float2 b = __fadd2_rn(__ffma2_rn(make_float2(hi.z, hi.w), minus, sum_t), __ffma2_rn(make_float2(lo.z, lo.w), minus, rest_t));
            float2 x = __fmul2_rn(make_float2(ex2_approx_ftz(a.x), ex2_approx_ftz(a.y)), __fmul2_rn(make_float2(len.x, len.y), factors));
            float2 y = __fmul2_rn(make_float2(ex2_approx_ftz(b.x), ex2_approx_ftz(b.y)), __fmul2_rn(make_float2(len.z, len.w), factors));
            x = __fmul2_rn(x, make_float2(v[i], v[i + 1]));
            y = __fmul2_rn(y, make_float2(v[i + 2], v[i + 3]));
            const int least = before - s0 - i;  // columns that count
            v[i] = 0 < least ? x.x : 0.0f, v[i + 1] = 1 < least ? x.y : 0.0f;
            v[i + 2] = 2 < least ? y.x : 0.0f, v[i + 3] = 3 < least ? y.y : 0.0f;
          }
        } else {  // decays over the middle are products of two
#pragma unroll
          for (int i = 0; i < 8; i += 4) {
            const float4 g = read4(now.near + s0 + i);
            const float2 x = __fmul2_rn(make_float2(v[i], v[i + 1]), __fmul2_rn(make_float2(g.x, g.y), fars));
            const float2 y = __fmul2_rn(make_float2(v[i + 2], v[i + 3]), __fmul2_rn(make_float2(g.z, g.w), fars));
            v[i] = before > 0 ? x.x : 0.0f, v[i + 1] = before > 0 ? x.y : 0.0f, v[i + 2] = before > 0 ? y.x : 0.0f, v[i + 3] = before > 0 ? y.y : 0.0f;
          }
        }
        if (keys) {
#pragma unroll
          for (int i = 0; i < 8; ++i) at[(s0 + i) * kPad + t] = v[i];
        } else {
          uint32_t hi[4], mid[4], lo[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) split3_signs(make_float2(v[2 * j], v[2 * j + 1]), hi[j], mid[j], lo[j]);
          const uint32_t where = m_row + swizzled(t, s0 / 8);
          sts128(where, make_uint4(hi[0], hi[1], hi[2], hi[3]));
          sts128(where + kTile, make_uint4(mid[0], mid[1], mid[2], mid[3]));
          sts128(where + 2 * kTile, make_uint4(lo[0], lo[1], lo[2], lo[3]));
        }
      }
      fence_before_sync();
      arrive(sh.g_empty);
      if (!keys) {
        bulk::fence_proxy_async();
        arrive(sh.m_ready[c & 1]);
      }
      meet_group();
      // ---- the inverse. Two blocks of 8 on the diagonal a warp, by rows, a column a lane (both halves of the warp do the same); then two
      // blocks to one: the lower left of (X 0; A Y)^-1 is -Y^-1 A X^-1. A warp does 8 of its columns; A X^-1 goes through the corner of A
      // that is above the diagonal, which nobody else uses.
      float2 corner[4];
      {
        const int first = 16 * part, block = first + (lane & 8), column = block + (lane & 7);
        float *half = inv + (part >> 1) * 32 * kPadInv;
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = i == (lane & 7) ? 1.0f : 0.0f;
#pragma unroll
        for (int r = 0; r < 7; ++r) {
#pragma unroll
          for (int i = (r + 1) / 4; i < 2; ++i) {
            const float4 e = read4(at + (block + r) * kPad + block + 4 * i);
            const float f[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (4 * i + k > r) x[4 * i + k] = fmaf(-f[k], x[r], x[4 * i + k]);
          }
        }
        if (lane < 16) {
#pragma unroll
          for (int i = 0; i < 8; ++i) half[((block & 31) + i) * kPadInv + (column & 31)] = x[i];
        }
        __syncwarp();
        float *mid = at + 32 * kPad + 8 * part;
        {
          float2 d[1];
          float *own = half + (first & 31) * (kPadInv + 1);
          block_product<8, false>(d, at + first * kPad + first + 8, own, 0, 8, lane);
          put_block<8, kPad>(mid, d, 1.0f, lane);
          __syncwarp();
          block_product<8, true>(d, own + 8 * kPadInv + 8, mid, 0, 8, lane);
          put_block<8, kPadInv>(own + 8 * kPadInv, d, -1.0f, lane);
        }
        meet(4 + 2 * group + (part >> 1), 64);
        {
          const int x0 = 32 * (part >> 1), y0 = x0 + 16, n = 8 * (part & 1);
          float2 d[2];
          block_product<16, false>(d, at + x0 * kPad + y0, half + n, 0, 16, lane);
          put_block<16, kPad>(mid, d, 1.0f, lane);
          __syncwarp();
          block_product<16, true>(d, half + 16 * kPadInv + 16, mid, 0, 16, lane);
          put_block<16, kPadInv>(half + 16 * kPadInv + n, d, -1.0f, lane);
        }
        meet_group();
        block_product<32, false>(corner, at + 32, inv + 8 * part, 8 * part, 32, lane);  // rows of X^-1 above these columns are zero
        put_block<32, kPad>(mid, corner, 1.0f, lane);
        __syncwarp();
        block_product<32, true>(corner, inv + 32 * kPadInv, mid, 0, 32, lane);
      }
      meet_group();
      // T = inverse diag(b), as an operand: 8 entries of a row at a time; those above the diagonal are zero. First the corner, a row a lane
      const uint32_t t_tile = base + kSmemT + (c & 1) * 3 * kTile;
#pragma unroll 1
      for (int i = -128 + row; i < 3 * 128; i += 128) {
        // the first 32 rows, then the last four pieces of the others
        const int line = i < 0 ? 32 + lane : i < 256 ? (i & 7) + 8 * (i >> 6) : 32 + (i & 7) + 8 * ((i - 256) >> 5);
        const int piece = i < 0 ? part : i < 256 ? (i >> 3) & 7 : 4 + ((i >> 3) & 3);
        uint32_t term[3][4] = {};
        if (8 * piece <= line) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float4 f = read4(now.beta + 8 * piece + 4 * j);
            float4 e = make_float4(-corner[2 * j].x, -corner[2 * j].y, -corner[2 * j + 1].x, -corner[2 * j + 1].y);
            if (i >= 0) e = read4(inv + line * kPadInv + 8 * (piece & 3) + 4 * j);
            split3_signs(make_float2(e.x * f.x, e.y * f.y), term[0][2 * j], term[1][2 * j], term[2][2 * j]);
            split3_signs(make_float2(e.z * f.z, e.w * f.w), term[0][2 * j + 1], term[1][2 * j + 1], term[2][2 * j + 1]);
          }
        }
#pragma unroll
        for (int j = 0; j < 3; ++j) sts128(t_tile + j * kTile + swizzled(line, piece), make_uint4(term[j][0], term[j][1], term[j][2], term[j][3]));
      }
      bulk::fence_proxy_async();
      arrive(sh.t_ready[c & 1]);
      arrive(sh.d_empty[c % kStages]);
    }
  } else if (warp < kWarpsChain) {
    // ---------------------------------------------------------------- the chain
    const int part = (warp - kWarpsPrep) >> 2, first = 64 * part, tokens = 32 * part;  // 64 states, 32 tokens of a channel
    const bool mine_v = row < job.np;
    const int mine_k = K - first < 0 ? 0 : K - first < 64 ? K - first : 64;
    float v[64];
    const float *from = job.from + row * p.K + first;
#pragma unroll
    for (int i = 0; i < 64; i += 4) {
      float4 e = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (job.from != nullptr && mine_v && i < mine_k) e = *reinterpret_cast<const float4 *>(from + i);
      if (PARTS && job.unit) e = make_float4(row == first + i, row == first + i + 1, row == first + i + 2, row == first + i + 3);
      v[i] = e.x, v[i + 1] = e.y, v[i + 2] = e.z, v[i + 3] = e.w;
    }
    for (int c = 0; c <= chunks; ++c) {
      if (c > 0) {
        const Tokens &last = sh.tokens[(c - 1) % kStages];
        if (!wait(sh.s_full[part], c - 1)) break;
        __syncwarp();
        fence_after_sync();
        const float2 decay = make_float2(last.decay, last.decay);
        const bool lost = min(last.bad_all, last.bad[row]) < kC;
#pragma unroll
        for (int i = 0; i < 64; i += 32) {
          float d[32];
          tmem_load32(mine + kColD + first + i, d);
          wait_loads();
          loaded(d);
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float2 r = __ffma2_rn(make_float2(v[i + j], v[i + j + 1]), decay, make_float2(d[j], d[j + 1]));
            v[i + j] = r.x;
            v[i + j + 1] = r.y;
          }
        }
        if (lost) {
#pragma unroll
          for (int i = 0; i < 64; ++i) v[i] = __int_as_float(0x7fffffff);
        }
        arrive(sh.d_empty[(c - 1) % kStages]);
        // the terms of s take the place of U, which everybody has read, and of w U
        if (!wait(sh.o_full, c - 1)) break;
      }
      if (c == chunks) break;
#pragma unroll
      for (int i = 0; i < 64; i += 16) put_terms(mine + kColA + (first + i) / 2, 64, mine + kColA + 128 + (first + i) / 2, v + i);
      wait_stores();
      fence_before_sync();
      arrive(sh.s_ready[part]);
      // R = -exp(c_t) / |k_t| KS, where D will be; then w U for the state where the terms of s were
      const Tokens &now = sh.tokens[c % kStages];
#pragma unroll 1
      for (int turn = 0; turn < 2; ++turn) {
        if (!wait2(turn == 0 ? sh.norm_ready[c & 1] : sh.v_ready[c & 1], c >> 1, turn == 0 ? sh.ks_full : sh.u_full, c)) break;
        __syncwarp();
        fence_after_sync();
        const uint32_t from = mine + (turn == 0 ? kColKS : kColU) + tokens, to = mine + (turn == 0 ? kColD : kColA) + tokens / 2;
        const float *factor = (turn == 0 ? now.minus : now.weight) + tokens;
#pragma unroll 1
        for (int i = 0; i < 32; i += 16) {
          float u[16];
          tmem_load16(from + i, u);
          wait_loads();
          loaded(u);
          put_terms(to + i / 2, 32, to + 64 + i / 2, u, factor + i);
        }
        wait_stores();
        fence_before_sync();
        arrive(turn == 0 ? sh.r_ready : sh.wu_ready);
      }
      if (!fine) break;
      // U for the outputs where KS was; its third term behind w U
#pragma unroll 1
      for (int i = 0; i < 32; i += 16) {
        float u[16];
        tmem_load16(mine + kColU + tokens + i, u);
        wait_loads();
        loaded(u);
        put_terms(mine + kColKS + (tokens + i) / 2, 32, mine + kColUThird + (tokens + i) / 2, u);
      }
      wait_stores();
      fence_before_sync();
      arrive(sh.u_ready);
    }
    if (fine && mine_v && job.to != nullptr) {
      float *to = job.to + row * p.K + first;
#pragma unroll
      for (int i = 0; i < 64; i += 4)
        if (i < mine_k) *reinterpret_cast<float4 *>(to + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
  } else if (warp < kWarpMma) {
    // ---------------------------------------------------------------- the outputs
    // a thread writes 8 channels of every eighth token
    const int i_out = tid - 32 * kWarpsChain, piece = i_out & 15;
    uint16_t *to = out + (job.begin + (i_out >> 4)) * p.out_stride_t + 8 * piece;
    for (int c = 0; c < chunks; ++c) {
      const Tokens &now = sh.tokens[c % kStages];
      const int rows = rows_of(c);
      // Everything of the chunk is waited for here: once O is on its way, what is two chunks on may come to the same barriers.
      fine = fine && wait_phases(&sh.norm_ready[c & 1], (c >> 1) & 1, &sh.qs_full, c & 1, &sh.q_ready[c & 1], (c >> 1) & 1);
      __syncwarp();
      fence_after_sync();
#pragma unroll 1
      for (int i = 0; (!PARTS || job.outputs) && i < kC; i += 16) {
        float v[16];
        uint32_t r[16];
        tmem_load16(mine + kColO + i, v);
        wait_loads();
        loaded(v);
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const float4 f = read4(now.in + i + j);
          const float2 x = __fmul2_rn(make_float2(v[j], v[j + 1]), make_float2(f.x, f.y)), y = __fmul2_rn(make_float2(v[j + 2], v[j + 3]), make_float2(f.z, f.w));
          r[j] = __float_as_uint(x.x), r[j + 1] = __float_as_uint(x.y), r[j + 2] = __float_as_uint(y.x), r[j + 3] = __float_as_uint(y.y);
        }
        tmem_store16(mine + kColO + i, r);
      }
      wait_stores();
      fence_before_sync();
      arrive(sh.qs_scaled);
      wait2(sh.o_full, c, sh.v_ready[c & 1], c >> 1);
      __syncwarp();
      fence_after_sync();
      // A lane has a channel, a row of memory is a token: through the place of V, which nothing reads any more.
      const uint32_t tile = base + kSmemV + (c & 1) * 2 * kTile;
#pragma unroll 1
      for (int i = 0; (!PARTS || job.outputs) && i < kC; i += 16) {
        float v[16];
        tmem_load16(mine + kColO + i, v);
        wait_loads();
        loaded(v);
        const uint32_t at = tile + i * 256 + 2 * row;
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const float4 f = read4(now.query + i + j);
          const float2 scale = make_float2(p.scale, p.scale), g = __fmul2_rn(__fmul2_rn(make_float2(v[j], v[j + 1]), make_float2(f.x, f.y)), scale);
          const float2 h = __fmul2_rn(__fmul2_rn(make_float2(v[j + 2], v[j + 3]), make_float2(f.z, f.w)), scale);
          const uint32_t x = pack_bf16x2(g.x, g.y), y = pack_bf16x2(h.x, h.y);
          sts16(at + j * 256, (uint16_t)x);
          sts16(at + (j + 1) * 256, (uint16_t)(x >> 16));
          sts16(at + (j + 2) * 256, (uint16_t)y);
          sts16(at + (j + 3) * 256, (uint16_t)(y >> 16));
        }
      }
      fence_before_sync();
      arrive(sh.o_empty);
      for (int t = min(now.bad_all, now.bad[row]); (!PARTS || job.outputs) && t < kC; ++t) sts16(tile + t * 256 + 2 * row, (uint16_t)0x7fff);
      arrive(sh.d_empty[c % kStages]);
      if (!meet_and(1, 128, fine)) break;
#pragma unroll 2
      for (int i = 0; (!PARTS || job.outputs) && i < 8; ++i) {
        if (8 * i + (i_out >> 4) < rows && 8 * piece < job.np) st_stream(to, lds128(tile + 16 * (i_out + 128 * i)));
        to += 8 * p.out_stride_t;
      }
      bulk::fence_proxy_async();
      arrive(sh.v_empty[c & 1]);
    }
  } else if (warp == kWarpMma) {
    // ---------------------------------------------------------------- products
    // The whole warp walks the loop, so that addresses stay in uniform registers; one lane issues.
    const bool leader = elect_one();
    const bool wide = K > 64;
    uint64_t qk_k = desc_k_major(base + kSmemQK), k_mn = desc_mn_major(base + kSmemQK + kTile, 2 * kTile);
    uint64_t v_mn = desc_mn_major(base + kSmemV, kTile), t_k = desc_k_major(base + kSmemT), m_k = desc_k_major(base + kSmemM);
    asm volatile("" : "+l"(qk_k), "+l"(k_mn), "+l"(v_mn), "+l"(t_k), "+l"(m_k));  // constant parts out of the compiler's sight, as in the scan
    constexpr uint64_t kTile16 = kTile >> 4;  // descriptors count in 16 bytes: 16 K are 2 along rows, 128 across them
#pragma unroll 1
    for (int c = 0; fine && c < chunks; ++c) {
      const uint64_t q_at = qk_k + (c & 1) * 4 * kTile16, k_at = q_at + kTile16, t_at = t_k + (c & 1) * 3 * kTile16;
      // KS, a half of the states after the other; rows of K that do not count are zero
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        if (!wait2(sh.s_ready[half], c, sh.norm_ready[c & 1], c >> 1)) break;
        fence_after_sync();
        if (leader && (half == 0 || wide)) {
          const uint64_t kt = k_at + half * 2 * kTile16;
          const uint32_t s_at = tmem + kColA + 32 * half;
#pragma unroll
          for (int term = 0; term < 3; ++term)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ts(tmem + kColKS, s_at + 64 * term + 8 * k, kt + 2 * k, instruction(128, 64, false, false, term == 1), half + term + k > 0);
        }
      }
      if (!fine) break;
      if (leader) mma_commit(&sh.ks_full);
      // QS
      if (c > 0 && !wait(sh.o_empty, c - 1)) break;
      fence_after_sync();
      if (leader) {
#pragma unroll 1
        for (int half = 0; (!PARTS || job.outputs) && half < (wide ? 2 : 1); ++half) {
          const uint64_t qt = q_at + half * 2 * kTile16;
          const uint32_t s_at = tmem + kColA + 32 * half;
#pragma unroll
          for (int term = 0; term < 3; ++term)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ts(tmem + kColO, s_at + 64 * term + 8 * k, qt + 2 * k, instruction(128, 64, false, false, term == 1), half + term + k > 0);
        }
        mma_commit(&sh.qs_full);
      }
      // U = V^T T^T, over the third terms of s, while R is made, then R T^T. The products that read those terms are waited for: the order of
      // products with other accumulators is not promised
      fine = fine && wait_phases(&sh.t_ready[c & 1], (c >> 1) & 1, &sh.v_ready[c & 1], (c >> 1) & 1, &sh.qs_full, c & 1);
      if (!fine) break;
      fence_after_sync();
      if (leader) {
        const uint64_t vt = v_mn + (c & 1) * 2 * kTile16;
#pragma unroll
        for (int term = 0; term < 3; ++term)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ss(tmem + kColU, vt + 128 * k, t_at + term * kTile16 + 2 * k, instruction(128, 64, true, false, false, term == 1), term + k > 0);
      }
      if (!wait(sh.r_ready, c)) break;
      fence_after_sync();
      if (leader) {
#pragma unroll
        for (int pair = 0; pair < 6; ++pair) {  // terms (0,0) (0,1) (0,2) (1,0) (1,1) (2,0)
          const int of_r = pair < 3 ? 0 : pair < 5 ? 1 : 2, of_t = pair < 3 ? pair : pair < 5 ? pair - 3 : 0;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ts(tmem + kColU, tmem + kColD + 32 * of_r + 8 * k, t_at + of_t * kTile16 + 2 * k,
                   instruction(128, 64, false, false, of_r == 1, of_t == 1), true);
        }
        mma_commit(&sh.u_full);
      }
      // D = (w U) K, a half of the states after the other, the last to read Q and K (the queries' lengths are known)
      if (!wait2(sh.wu_ready, c, sh.q_ready[c & 1], c >> 1)) break;
      fence_after_sync();
      if (leader) {
        const uint64_t kt = k_mn + (c & 1) * 4 * kTile16;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          const uint64_t k_half = kt + half * 2 * kTile16;
          if (half == 0 || wide) {
#pragma unroll
            for (int term = 0; term < 3; ++term)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_ts(tmem + kColD + 64 * half, tmem + kColA + 32 * term + 8 * k, k_half + 128 * k, instruction(128, 64, false, true, term == 1), term + k > 0);
          }
          mma_commit(&sh.s_full[half]);
        }
        mma_commit(&sh.qk_empty[c & 1]);
      }
      // O = QS, scaled, + U M^T
      fine = fine && wait_phases(&sh.m_ready[c & 1], (c >> 1) & 1, &sh.qs_scaled, c & 1, &sh.u_ready, c & 1);
      if (!fine) break;
      fence_after_sync();
      if (leader) {
        const uint64_t mt = m_k + (c & 1) * 3 * kTile16;
        if (!PARTS || job.outputs) {
#pragma unroll
          for (int pair = 0; pair < 6; ++pair) {  // as above
            const int of_u = pair < 3 ? 0 : pair < 5 ? 1 : 2, of_m = pair < 3 ? pair : pair < 5 ? pair - 3 : 0;
            const uint32_t u_at = tmem + (of_u < 2 ? kColKS + 32 * of_u : kColUThird);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ts(tmem + kColO, u_at + 8 * k, mt + of_m * kTile16 + 2 * k, instruction(128, 64, false, false, of_u == 1, of_m == 1), true);
          }
        }
        mma_commit(&sh.o_full);
        mma_commit(&sh.o_done[c & 1]);
      }
    }
    // No product reads shared memory or TMEM, and no barrier is to be arrived at, once the CTA leaves: also
    // where a wait ran out and what was issued is left behind.
    if (leader) mma_commit(&sh.drained);
    fine &= wait_phase(&sh.drained, 0);
  } else if (warp == kWarpCopy) {
    // ---------------------------------------------------------------- copies
    if (lane == 0) {
      int issued = 0, issued_v = 0;
      const int blocks_k = K > 64 ? 2 : 1, blocks_v = job.np > 64 ? 2 : 1;
#pragma unroll 1
      for (int c = 0; c < chunks; ++c) {
        if (c >= 2 && !wait(sh.qk_empty[c & 1], (c >> 1) - 1)) break;
        const int t0 = (int)(job.begin + (int64_t)c * kC);
        const uint32_t qk = base + kSmemQK + (c & 1) * 4 * kTile, vt = base + kSmemV + (c & 1) * 2 * kTile;
        bulk::mbar_arrive_expect_tx(&sh.qk_full[c & 1], 2 * blocks_k * kTile);
#pragma unroll 1
        for (int i = 0; i < blocks_k; ++i) {
          tile_load(qk + 2 * i * kTile, &map_q, 64 * i, job.g, t0, &sh.qk_full[c & 1]);
          tile_load(qk + (2 * i + 1) * kTile, &map_k, 64 * i, job.g, t0, &sh.qk_full[c & 1]);
        }
        issued = c + 1;
        if (c >= 2 && !wait(sh.v_empty[c & 1], (c >> 1) - 1)) break;
        if (PARTS && job.unit) {
          bulk::mbar_arrive(&sh.v_full[c & 1]);
          issued_v = c + 1;
          continue;
        }
        bulk::mbar_arrive_expect_tx(&sh.v_full[c & 1], blocks_v * kTile);
#pragma unroll 1
        for (int i = 0; i < blocks_v; ++i) tile_load(vt + i * kTile, &map_v, (int)job.p0 + 64 * i, (int)job.h, t0, &sh.v_full[c & 1]);
        issued_v = c + 1;
        // the chunk after the next one into L2: there is no place for it here yet
        const int t2 = t0 + 2 * kC;
        if (c + 2 < chunks) {
#pragma unroll 1
          for (int i = 0; i < blocks_k; ++i) {
            tile_prefetch(&map_q, 64 * i, job.g, t2);
            tile_prefetch(&map_k, 64 * i, job.g, t2);
          }
#pragma unroll 1
          for (int i = 0; i < blocks_v; ++i) tile_prefetch(&map_v, (int)job.p0 + 64 * i, (int)job.h, t2);
        }
      }
      // The last copies into every place have landed before anybody leaves.
#pragma unroll 1
      for (int c = issued > 2 ? issued - 2 : 0; c < issued; ++c) fine &= wait_phase(&sh.qk_full[c & 1], (c >> 1) & 1);
#pragma unroll 1
      for (int c = issued_v > 2 ? issued_v - 2 : 0; c < issued_v; ++c) fine &= wait_phase(&sh.v_full[c & 1], (c >> 1) & 1);
    }
  } else if (warp == kWarpG) {
    // ---------------------------------------------------------------- G, ahead of the other products
    const bool leader = elect_one();
    const int steps_k = (K + 15) / 16;
    uint64_t qk_k = desc_k_major(base + kSmemQK);
    asm volatile("" : "+l"(qk_k));
    constexpr uint64_t kTile16 = kTile >> 4;
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {  // G = [Q; K] K^T
      if (!wait(sh.qk_full[c & 1], c >> 1)) break;
      if (c > 0 && !wait(sh.g_empty, c - 1)) break;
      fence_after_sync();
      if (leader) {
        const uint64_t at = qk_k + (c & 1) * 4 * kTile16;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint64_t along = (k >> 2) * 2 * kTile16 + (k & 3) * 2;
          if (k < steps_k) mma_ss(tmem + kColG, at + along, at + kTile16 + along, instruction(128, 64, false, false), k > 0);
        }
        mma_commit(&sh.g_full[c & 1]);
      }
      // The queries' lengths, two rows a lane, for the outputs
      if (c >= 2 && !wait(sh.o_done[c & 1], (c >> 1) - 1)) break;
      if (c >= kStages && !wait(sh.d_empty[c % kStages], c / kStages - 1)) break;
      __syncwarp();
      Tokens &now = sh.tokens[c % kStages];
#pragma unroll 1
      for (int t = lane; t < kC; t += 32) {
        float2 squares[2] = {};
        if (p.qk_norm) {
#pragma unroll 2
          for (int i = 0; i < K / 8; ++i) {
            const uint4 x = lds128(base + kSmemQK + (c & 1) * 4 * kTile + (i >> 3) * 2 * kTile + swizzled(t, i & 7));
            const uint32_t e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 v = make_float2(first_of(e[j]), second_of(e[j]));
              squares[j & 1] = __ffma2_rn(v, v, squares[j & 1]);
            }
          }
        }
        const float sum = (squares[0].x + squares[0].y) + (squares[1].x + squares[1].y);
        now.query[t] = p.qk_norm ? rsqrtf(sum + kUnitEps) : 1.0f;
      }
      arrive(sh.q_ready[c & 1]);
    }
    // As with the other products: its last ones are done before it leaves.
    if (leader) mma_commit(&sh.g_drained);
    fine &= wait_phase(&sh.g_drained, 0);
  } else if (warp == kWarpDecay) {
    // ---------------------------------------------------------------- decays and strengths
    const uint16_t *a = static_cast<const uint16_t *>(p.a) + job.h, *b = static_cast<const uint16_t *>(p.b) + job.h;
    const float A2 = __ldg(p.A + job.h) * kLog2e, bias = p.dt_bias != nullptr ? __ldg(p.dt_bias + job.h) : 0.0f;
    uint32_t next_a = 0, next_b = 0;  // two tokens
    auto fetch = [&](int c) {
      next_a = next_b = 0;
#pragma unroll 1
      for (int j = 1; j >= 0; --j) {
        const int64_t t = (int64_t)c * kC + 2 * lane + j;
        next_a <<= 16, next_b <<= 16;
        if (t < job.length) {
          next_a |= __ldg(a + (job.begin + t) * p.a_stride_t);
          next_b |= __ldg(b + (job.begin + t) * p.b_stride_t);
        }
      }
    };
    if (chunks > 0) fetch(0);
#pragma unroll 1
    for (int ahead = 0; ahead <= chunks; ++ahead) {
      if (ahead < chunks) {
        const uint32_t raw_a = next_a, raw_b = next_b;
        if (ahead + 1 < chunks) fetch(ahead + 1);
        if (ahead >= kStages && !wait(sh.d_empty[ahead % kStages], ahead / kStages - 1)) break;
        __syncwarp();
        fill_tokens(sh.tokens[ahead % kStages], raw_a, raw_b, bias, A2, rows_of(ahead), lane);
        bulk::mbar_arrive(&sh.d_full[ahead % kStages]);
      }
      if (ahead == 0) continue;
      const int c = ahead - 1, rows = rows_of(c);
      Tokens &now = sh.tokens[c % kStages];
      // The rows of V: those of other sequences are zeroed, and what is not finite is taken out and noted, by what 0 v gives
      if (!wait(sh.v_full[c & 1], c >> 1)) break;
      __syncwarp();
      const uint32_t vt = base + kSmemV + (c & 1) * 2 * kTile + (lane >> 3) * 128 + (lane & 7) * 16;
      const int quads = job.np > 64 ? 32 : 16;  // of rows of 64 channels
      const __nv_bfloat162 zero = __floats2bfloat162_rn(0.0f, 0.0f);
      __nv_bfloat162 probe[2] = {zero, zero};
      if (rows < kC) {
        const int t = lane >> 3;
#pragma unroll 1
        for (int i = 0; i < quads; ++i)
          if (4 * (i & 15) + t >= rows) sts128(vt + 512 * i, make_uint4(0, 0, 0, 0));
        bulk::fence_proxy_async();
      }
#pragma unroll 2
      for (int i = 0; i < quads; ++i) {
        const uint4 x = lds128(vt + 512 * i);
        const uint32_t e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) probe[j & 1] = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&e[j]), zero, probe[j & 1]);
      }
      const __nv_bfloat162 both = __hadd2(probe[0], probe[1]);
      if (!(__low2float(both) + __high2float(both) == 0.0f)) {
#pragma unroll 1
        for (int i = 0; i < 4 * quads; ++i) {
          const uint32_t where = vt + 512 * (i >> 2) + 4 * (i & 3), e = lds32(where);
          const int t = 4 * ((i >> 2) & 15) + (lane >> 3), channel = 64 * (i >> 6) + 8 * ((lane & 7) ^ (t & 7)) + 2 * (i & 3);
          const bool f = (e & 0x7f80u) == 0x7f80u, l = (e & 0x7f800000u) == 0x7f800000u;
          if (f) atomicMin(&now.bad[channel], t);
          if (l) atomicMin(&now.bad[channel + 1], t);
          sts32(where, e & ((f ? 0u : 0xffffu) | (l ? 0u : 0xffff0000u)));
        }
        bulk::fence_proxy_async();
      }
      arrive(sh.v_ready[c & 1]);
    }
  }
  if (!fine) atomicOr(p.status_dev != nullptr ? p.status_dev : &g_delta_error, kDevErrTimeout);
  __syncwarp();
  fence_before_sync();
  __syncthreads();
  if (warp == kWarpMma) {
    fence_after_sync();
    tmem_free(tmem, kColumns);
  }
  if (SHARES && tid == 0 && piece.cut >= 0 && !piece.late) {  // the state is written (the barrier above): whoever waits for it may read it
    __threadfence();
    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(sharing.flags + piece.cut), "r"(1) : "memory");
  }
}

// Boxes of a chunk's rows x 64.
cudaError_t encode(CUtensorMap *map, const void *data, int64_t inner, int64_t groups, int64_t rows, int64_t stride_group, int64_t stride_row) {
  return encode_tiles(map, data, inner, groups, rows, stride_group, stride_row, 64, kC, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

cudaError_t take_delta_error(int32_t *bits) {
  cudaError_t e = launch_overlapped(k_exchange_delta_error, dim3(1), dim3(1), 0, (cudaStream_t)0);
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(bits, g_delta_error_taken, sizeof(int32_t));
  return e;
}

namespace {

// Segments of the sequences for these arguments; as many as sequences is not to cut. The first launch runs the first segments and, of
// those between, W and Phi: as many segments as its CTAs find SMs for, three at least (two would run one after the other). A segment is
// 8 chunks or more: below that the second launch's start takes what the shorter chains give. In microseconds, not cut against cut: 8 heads of 128 channels, 128 states, 2048
// tokens 166 and 130, 4096 tokens 319 and 222, 16384 1248 and 442; 32 heads 4096 tokens 322 and 273, 16384 1259 and 937; 48 heads of 64 channels, 64 states, 16384 1185 and 893. With
// floors of 4 and of 16 chunks, and two terms in the outputs' factors, the 2048 tokens took 177 and 156 (8: 123), the 4096 of 8 heads 242 and 199 (215).
Segments segments_of(const DeltaParams &p, int sms) {
  const int64_t heads = p.n_seq * p.H, items = heads * ((p.P + kV - 1) / kV), chunks = (p.T + kC - 1) / kC;
  Segments seg = {p.n_seq, INT64_MAX / 4, nullptr, nullptr};
  if (items < 1 || items + items + heads > sms) return seg;
  int64_t most = 2 + (sms - items) / (items + heads), length = (chunks + p.n_seq * most - 1) / (p.n_seq * most);
  if (length < 8) length = 8;
  if (chunks <= 2 * length * p.n_seq) return seg;
  seg.tokens = length * kC;
  seg.count = p.T / seg.tokens + p.n_seq;
  return seg;
}

bool cut(const DeltaParams &p, const Segments &seg) { return seg.count > p.n_seq; }

template <int MODE>
cudaError_t launch_pass(const DeltaParams &p, const Segments &seg, const Shares &sharing, int64_t ctas, int pair, int pass, int blocks_p,
                        const CUtensorMap (&maps)[3], int dev, cudaStream_t stream) {
  static std::atomic<bool> opted_in[64];
  if (!opted_in[dev].load(std::memory_order_acquire)) {
    cudaError_t e = cudaFuncSetAttribute(k_delta_chunked<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
    cudaFuncAttributes has;
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&has, k_delta_chunked<MODE>);
    if (e != cudaSuccess) return e;
    if (has.numRegs < kRegs) return cudaErrorInvalidConfiguration;  // the roles' shares are taken from the launch's registers
    opted_in[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas), cfg.blockDim = dim3(kThreads), cfg.dynamicSmemBytes = kSmemBytes, cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // as launch_overlapped
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)pair, attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr, cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_delta_chunked<MODE>, p, blocks_p, seg, sharing, pass, maps[0], maps[1], maps[2]);
}

// CTAs of a cluster, which work on one sequence: two heads or blocks of channels, that start together on the same number of chunks. They share
// no data, and the SMs' mean time stays (304 items: the same instructions, active cycles within 0.5 %, instruction misses 18.5 and 17.5 %; the gain is the
// same with q and k of their own for every head): what goes is the spread, the slowest SMs were 10 % behind the mean. Why is not known. With two terms in the outputs' factors 8 x 4096 tokens, 32 heads 664 us without, 633 with, 304 items of 64 chunks 691 and 638, 16384 tokens in segments 937 and 889
// (the pairs two heads: a head's W and its Phi in a pair leave half of it empty at the first segment, 48 heads of 64 channels 1167 against 825).
int pair_of(const DeltaParams &p, int64_t per_head, int sms) { return p.H * per_head % 2 == 0 && sms % 2 == 0 ? 2 : 1; }

// Whether items are shared out evenly: where whole ones would leave the SMs of their last turn idle for longer than the pieces' starts take. n turns of
// whole items against w = items / SMs shares of all chunks: chunks (n - w) > 4. In microseconds, whole against shared out, items of 128 channels, 128 states:
//   of 8 chunks  160 items 102 and 81, 200 103 and 91, 320 155 and 134, 512 210 and 200
//   of 16        160 180 and 122, 200 184 and 154, 240 185 and 175, 256 186 and 183, 320 273 and 218, 512 370 and 342
//   of 64        160 650 and 378, 200 653 and 474, 240 658 and 556, 256 663 and 589, 288 666 and 660, 320 977 and 730, 512 1312 and 1146
// and, left whole, before the outputs' factors had three terms: of 8 chunks 240 102 and 108, 256 104 and 113; of 16 288 182 and 194; of 64 304 638 and 641.
// Without pairs (measured then too) the SMs' times spread (pieces of 60 chunks 304 to 369 us), and less is gained: chunks (n - 1.25 w) > 4. Of 64 chunks 160 items 622 and 458, 240 637 and 631, 256
// 646 and 684, 320 933 and 841.
bool shared_out(const DeltaParams &p, int sms) {
  const int64_t blocks_p = (p.P + kV - 1) / kV, items = p.n_seq * p.H * blocks_p, turns = (items + sms - 1) / sms, chunks = p.T / p.n_seq / kC;
  if (items <= sms || items > kMaxItems || p.n_seq > kSorted || sms - 1 > kMaxCuts || p.T / kC >= INT32_MAX / (2 * items) / p.n_seq) return false;
  return chunks * (4 * turns * sms - (pair_of(p, blocks_p, sms) == 2 ? 4 : 5) * items) > 16 * (int64_t)sms;
}

// Bytes of the workspace before the states: the header and the plan.
int64_t plan_bytes(const DeltaParams &p, int sms) {
  return kShareHeader + (int64_t)sizeof(Piece) * (p.n_seq * p.H * ((p.P + kV - 1) / kV) + sms - 1);
}

}  // namespace

int64_t delta_chunked_workspace(const DeltaParams &p, int sms) {
  if (shared_out(p, sms)) return plan_bytes(p, sms) + 4 * (int64_t)(sms - 1) * kV * p.K;
  const Segments seg = segments_of(p, sms);
  return cut(p, seg) ? 4 * seg.count * p.H * p.K * (p.P + p.K) : 0;
}

cudaError_t launch_delta_chunked(const DeltaParams &p, cudaStream_t stream) {
  const int dev = current_device();
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  alignas(64) CUtensorMap maps[3] = {};
  if (p.T > 0) {
    cudaError_t e = encode(&maps[0], p.q, p.K, p.G, p.T, p.q_stride_g, p.q_stride_t);
    if (e == cudaSuccess) e = encode(&maps[1], p.k, p.K, p.G, p.T, p.k_stride_g, p.k_stride_t);
    if (e == cudaSuccess) e = encode(&maps[2], p.v, p.P, p.H, p.T, p.v_stride_h, p.v_stride_t);
    if (e != cudaSuccess) return e;
  }
  const int blocks_p = (int)((p.P + kV - 1) / kV), sms = device_sm_count();
  const int64_t items = p.n_seq * p.H * blocks_p;
  const int pair = pair_of(p, blocks_p, sms);
  Shares sharing = {};
  Segments seg = segments_of(p, sms);
  if (shared_out(p, sms)) {
    char *work = static_cast<char *>(p.workspace);
    sharing = {reinterpret_cast<int *>(work), reinterpret_cast<int *>(work) + 64, reinterpret_cast<Piece *>(work + kShareHeader),
               reinterpret_cast<float *>(work + plan_bytes(p, sms)), sms, pair};
    const cudaError_t e = launch_overlapped(k_delta_plan, dim3(1), dim3(1024), 0, stream, p, blocks_p, sharing);
    return e == cudaSuccess ? launch_pass<kShares>(p, seg, sharing, items + sms - pair, pair, 0, blocks_p, maps, dev, stream) : e;
  }
  if (!cut(p, seg)) return launch_pass<kWhole>(p, seg, sharing, items, pair, 0, blocks_p, maps, dev, stream);
  seg.states = static_cast<float *>(p.workspace);
  seg.maps = seg.states + seg.count * p.H * p.P * p.K;
  cudaError_t e = launch_pass<kSegments>(p, seg, sharing, seg.count * p.H * (blocks_p + 1), pair_of(p, 1, sms), kFirst, blocks_p, maps, dev, stream);
  const dim3 grid((unsigned)((p.P + kJoinRows - 1) / kJoinRows), (unsigned)p.H, (unsigned)p.n_seq);
  if (e == cudaSuccess) e = launch_overlapped(k_delta_join, grid, dim3(2 * kV), 0, stream, p, seg);
  return e == cudaSuccess ? launch_pass<kSegments>(p, seg, sharing, seg.count * p.H * blocks_p, pair_of(p, 1, sms), kRest, blocks_p, maps, dev, stream) : e;
}

}  // namespace ccu
