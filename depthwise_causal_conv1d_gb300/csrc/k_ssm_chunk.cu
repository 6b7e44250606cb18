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
//   Y[t,p] = C h^T          h rounded to BF16; the rows are then scaled by exp(c_t) in FP32
//   Y     += M x            M = S with decays, steps and the causal mask, rounded to BF16, in TMEM
//   U[k,p] = B^T (w x)      w_s = exp(c_end - c_s) d_s
//
// Rounding. M and the h that Y sees are rounded to BF16 once: each term of an output carries 2^-9
// or less, as the BF16 output itself does. The state may not lose that much: w x is split into three
// BF16 terms (24 bits in all) and U accumulated over all three, and h itself stays FP32
// (in TMEM) and is only added to by FP32 instructions.
//
// Decays are exponentials of differences of running sums; a difference of sums over a whole chunk
// would lose what the steps' sizes vary by, and a product exp(c_t) exp(-c_s) would overflow. So the sums run
// over 32 tokens: within such a block the difference is taken, between blocks the decay is
// a product of two that are both at most 1, exp(c_t - c_r) exp(c_r - c_s), r the token before t's block.
// The state's weights come from sums taken from the chunk's end.
//
// TMEM (256 columns; two CTAs share an SM's 512): S at 0..127, then, when S has been read, M at
// 0..63 and U at 64..127; Y at 128..191; h at 192..255 (lane k, column p).
// Shared memory (96 KB and tables, so that two CTAs fit): B 32 KB, x 16 KB, C 32 KB (then the
// first two terms of w x), h 16 KB (then the third term of w x). One thread copies the tiles with TMA
// (which zero-fills past P and K) and issues the products; the tiles' other rows past a
// sequence's end belong to the next sequence and are zeroed here.
#include <atomic>

#include "ssm_tensor.cuh"

namespace ccu {

int current_device();

__device__ int32_t g_scan_error = 0;        // CCU_DEVERR_* bits of calls without a status word
__device__ int32_t g_scan_error_taken = 0;  // the value the last exchange read

__global__ void k_exchange_scan_error() {
  grid_dependency_boundary();
  g_scan_error_taken = atomicExch(&g_scan_error, 0);
}

namespace {

using namespace tensor;

constexpr int kQ = 128;       // tokens a chunk
constexpr int kThreads = 256;
constexpr int kTile = kQ * 128;             // a block of 128 rows: 16 KB
constexpr int kColS = 0, kColM = 0, kColU = 64, kColY = 128, kColH = 192, kColumns = 256;
constexpr float kLog2e = 1.4426950408889634f;
// exp2 of anything below -150 is zero in FP32; sums of steps stay finite and small with this floor.
constexpr float kLeast = -300.0f;

struct Decays {
  float sum[kQ], step[kQ];    // running sum of log2 decays in its block of 32; d
  float from[3][kQ];          // [r - 1][s]: decay from s to the token before block r, times d_s
  float in[kQ], weight[kQ];   // exp(c_t); w
  float total[4];
};
struct Tables {
  Decays decays[2];           // this chunk's and the next one's
  int bad[64];                // first token with a non-finite x, a channel
  uint64_t full, first, second, third;  // tiles in place; S and Y0, Y, U ready
  uint32_t tmem;
};

constexpr int kSmemB = 0, kSmemX = 2 * kTile, kSmemC = 3 * kTile, kSmemH = 5 * kTile, kSmemTables = 6 * kTile;
constexpr size_t kSmemBytes = kSmemTables + sizeof(Tables) + 1024;

__device__ __forceinline__ float first_of(uint32_t pair) { return __uint_as_float(pair << 16); }
__device__ __forceinline__ float second_of(uint32_t pair) { return __uint_as_float(pair & 0xffff0000u); }

// a and b as three BF16 pairs whose sum is a (b) to 24 bits; a non-finite value goes into the first alone.
__device__ __forceinline__ void split3(float a, float b, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
  hi = pack_bf16x2(a, b);
  const float ra = a - first_of(hi), rb = b - second_of(hi);
  mid = pack_bf16x2(ra, rb);
  lo = pack_bf16x2(ra - first_of(mid), rb - second_of(mid));
}
__device__ __forceinline__ bool finite_pair(uint32_t v) { return (v & 0x7f80u) != 0x7f80u && (v & 0x7f800000u) != 0x7f800000u; }

// A chunk's decays, a token a thread (128 threads; `dt` of a row past the sequence's end is not read: d = 0).
__device__ __forceinline__ void fill_decays(Decays &t, float d, float A2, int row) {
  const int lane = row & 31, block = row >> 5;
  float a = d * A2;
  a = a < kLeast ? kLeast : a;
  float sum = a, after = a;  // over the block up to this token, and from this token on
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float u = __shfl_up_sync(0xffffffffu, sum, o), w = __shfl_down_sync(0xffffffffu, after, o);
    if (lane >= o) sum += u;
    if (lane + o < 32) after += w;
  }
  if (lane == 31) t.total[block] = sum;
  after = __shfl_down_sync(0xffffffffu, after, 1);
  if (lane == 31) after = 0.0f;
  bar_sync(1, kQ);
  float before = 0.0f, reach = after;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < block) before += t.total[j];
  t.sum[row] = sum;
  t.step[row] = d;
  t.in[row] = exp2f(before + sum);
#pragma unroll
  for (int r = 1; r < 4; ++r)
    if (r > block) {
      t.from[r - 1][row] = exp2f(reach) * d;
      reach += t.total[r];
    }
  t.weight[row] = exp2f(reach) * d;
}

// WIDE: rows of z and out on 32-byte boundaries.
template <bool WIDE>
__global__ void __launch_bounds__(kThreads, 2) k_scan_chunked(ScanParams p, int blocks_p, const __grid_constant__ CUtensorMap map_x,
                                                              const __grid_constant__ CUtensorMap map_b,
                                                              const __grid_constant__ CUtensorMap map_c) {
  grid_dependency_boundary();
  extern __shared__ unsigned char raw[];
  const uint32_t base = (bulk::smem_addr(raw) + 1023) & ~1023u;
  Tables &tab = *reinterpret_cast<Tables *>(raw + (base - bulk::smem_addr(raw)) + kSmemTables);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int quarter = warp & 3, half = warp >> 2;
  const int row = quarter * 32 + lane;              // token (k for the state) of this thread
  int64_t item = blockIdx.x;
  const int pb = (int)(item % blocks_p);
  item /= blocks_p;
  const int64_t h = item % p.H, b = item / p.H;
  const int64_t g = h / (p.H / p.G);
  const int64_t p0 = (int64_t)pb * 64;
  const int np = (int)(p.P - p0 < 64 ? p.P - p0 : 64), K = (int)p.K;
  const Bounds q = sequence_bounds(p.cu_seqlens, b, p.T);
  const int64_t s = slot_of(p.indices, b, p.S, p.status_dev, tid == 0 && h == 0 && pb == 0);
  const int column = half * 32;                     // this thread's 32 channels of the block
  const int columns = np - column < 32 ? np - column : 32;
  uint16_t *out = static_cast<uint16_t *>(p.out) + h * p.out_stride_h + p0 + column;
  // 64 bytes of a row of out, or the whole 16-byte pieces of them that there are.
  auto put_row = [&](int64_t t, const uint4 (&v)[4]) {
    uint16_t *at = out + t * p.out_stride_t;
    if (columns == 32) {
      store64<WIDE>(at, v);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (8 * c < columns) st_stream(at + 8 * c, v[c]);
    }
  };
  if (s < 0) {
    const uint4 zero[4] = {};
    for (int64_t t = q.begin + row; t < q.end; t += kQ) put_row(t, zero);
    return;
  }
  const uint16_t *z = p.z != nullptr ? static_cast<const uint16_t *>(p.z) + h * p.z_stride_h + p0 + column : nullptr;
  const uint16_t *dt = static_cast<const uint16_t *>(p.dt) + h;
  float *state = p.state + s * p.state_stride_s + (h * p.P + p0) * p.K;
  const int64_t length = q.end - q.begin;

  if (warp == 0) tmem_alloc(&tab.tmem, kColumns);
  if (tid == 0) {
    bulk::mbar_init(&tab.full, 1);
    bulk::mbar_init(&tab.first, 1);
    bulk::mbar_init(&tab.second, 1);
    bulk::mbar_init(&tab.third, 1);
    bulk::fence_mbar_init();
  }
  if (tid < 64) tab.bad[tid] = kQ;
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = tab.tmem, mine = tmem + ((uint32_t)(quarter * 32) << 16);

  auto load_tiles = [&](int64_t t0) {  // one thread
    bulk::mbar_arrive_expect_tx(&tab.full, 5 * kTile);
    tile_load(base + kSmemB, &map_b, 0, (int)g, (int)t0, &tab.full);
    tile_load(base + kSmemB + kTile, &map_b, 64, (int)g, (int)t0, &tab.full);
    tile_load(base + kSmemC, &map_c, 0, (int)g, (int)t0, &tab.full);
    tile_load(base + kSmemC + kTile, &map_c, 64, (int)g, (int)t0, &tab.full);
    tile_load(base + kSmemX, &map_x, (int)p0, (int)h, (int)t0, &tab.full);
  };
  // The step of this thread's token in the chunk at t0 (half 0's threads), 0 past the sequence's end.
  auto step_at = [&](int64_t t0) {
    const int64_t t = t0 + row;
    return t < q.end ? step_size(__ldg(dt + t * p.dt_stride_t), p.dt_bias, h, p.dt_softplus) : 0.0f;
  };
  // The state's place in the operand tile of Y's product: row channel, K-major in k.
  auto put_h = [&](const float (&v)[32]) {
    const uint32_t at = base + kSmemH + (row >> 6) * (kTile / 2) + column * 128 + (row & 7) * 2;
    const int chunk = (row >> 3) & 7;
#pragma unroll
    for (int i = 0; i < 32; ++i) sts16(at + i * 128 + ((chunk ^ (i & 7)) << 4), round_bf16(v[i]));
  };

  const float A2 = __ldg(p.A + h) * kLog2e, skip = p.D != nullptr ? __ldg(p.D + h) : 0.0f;
  if (tid == 0 && length > 0) load_tiles(q.begin);
  {
    float v[32];
    const bool initial = p.has_initial != nullptr && __ldg(p.has_initial + b) != 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = initial && i < columns && row < K ? state[(int64_t)(column + i) * K + row] : 0.0f;
    tmem_store32(mine + kColH + column, v);
    wait_stores();
    put_h(v);
  }
  if (half == 0) fill_decays(tab.decays[0], step_at(q.begin), A2, row);

  uint32_t phase = 0;
  bool fine = true;
  for (int64_t done = 0; done < length; done += kQ) {
    const int64_t t0 = q.begin + done;
    const int rows = (int)(length - done < kQ ? length - done : kQ);
    const Decays &now = tab.decays[phase];
    // ---- tiles in place; what a partial chunk read of other sequences goes
    fine &= bulk::mbar_wait(&tab.full, phase);
    if (row >= rows) {
      const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        sts128(base + kSmemB + half * kTile + swizzled(row, c), zero);
        sts128(base + kSmemC + half * kTile + swizzled(row, c), zero);
        if (c < 4) sts128(base + kSmemX + swizzled(row, half * 4 + c), zero);
      }
    }
    __syncwarp();
    bulk::fence_proxy_async();
    fence_before_sync();
    fine = __syncthreads_and(fine);
    if (!fine) break;
    // ---- S = C B^T, Y = C h^T
    if (tid == 0) {
      fence_after_sync();
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t at = (k >> 2) * kTile + (k & 3) * 32;
        mma_ss(tmem + kColS, desc_k_major(base + kSmemC + at), desc_k_major(base + kSmemB + at), instruction(128, 128, false, false), k > 0);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k)
        mma_ss(tmem + kColY, desc_k_major(base + kSmemC + (k >> 2) * kTile + (k & 3) * 32),
               desc_k_major(base + kSmemH + (k >> 2) * (kTile / 2) + (k & 3) * 32), instruction(128, 64, false, false), k > 0);
      mma_commit(&tab.first);
    }
    // ---- meanwhile: this thread's x (32 channels of its token)
    uint4 xv[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) xv[c] = lds128(base + kSmemX + swizzled(row, half * 4 + c));
    // A non-finite x would reach earlier tokens through the zeros of M: it is taken out of the tile, and its
    // channel's outputs from there on are set to NaN.
    bool all_finite = true;
#pragma unroll
    for (int c = 0; c < 4; ++c) all_finite &= finite_pair(xv[c].x) && finite_pair(xv[c].y) && finite_pair(xv[c].z) && finite_pair(xv[c].w);
    if (!all_finite) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t e[4] = {xv[c].x, xv[c].y, xv[c].z, xv[c].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int channel = column + 8 * c + 2 * i;
          if ((e[i] & 0x7f80u) == 0x7f80u) e[i] &= 0xffff0000u, atomicMin(&tab.bad[channel], row);
          if ((e[i] & 0x7f800000u) == 0x7f800000u) e[i] &= 0xffffu, atomicMin(&tab.bad[channel + 1], row);
        }
        sts128(base + kSmemX + swizzled(row, half * 4 + c), make_uint4(e[0], e[1], e[2], e[3]));
      }
    }
    fine &= bulk::mbar_wait(&tab.first, phase);
    __syncwarp();
    fence_after_sync();
    // ---- the rows of Y by exp(c_t)
    {
      float v[32];
      tmem_load32(mine + kColY + column, v);
      wait_loads();
      const float e = now.in[row];
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] *= e;
      tmem_store32(mine + kColY + column, v);
    }
    // ---- M: this thread's token against 64 earlier ones, two blocks of 32
    {
      float v[2][32];
      tmem_load32(mine + kColS + half * 64, v[0]);
      tmem_load32(mine + kColS + half * 64 + 32, v[1]);
      wait_loads();
      fence_before_sync();
      bar_sync(2 + quarter, 64);  // both warps of these lanes have read S: M may overwrite it
      fence_after_sync();
      const float sum = now.sum[row], local = exp2f(sum);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int block = half * 2 + j;
        uint32_t m[16];
        if (block > quarter) {
#pragma unroll
          for (int i = 0; i < 16; ++i) m[i] = 0;
        } else if (block < quarter) {
          const float4 *from = reinterpret_cast<const float4 *>(&now.from[quarter - 1][block * 32]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 f = from[i];
            m[2 * i] = pack_bf16x2(v[j][4 * i] * (local * f.x), v[j][4 * i + 1] * (local * f.y));
            m[2 * i + 1] = pack_bf16x2(v[j][4 * i + 2] * (local * f.z), v[j][4 * i + 3] * (local * f.w));
          }
        } else {
          const float4 *sums = reinterpret_cast<const float4 *>(&now.sum[block * 32]);
          const float4 *steps = reinterpret_cast<const float4 *>(&now.step[block * 32]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 c = sums[i], d = steps[i];
            const float w0 = ex2_approx_ftz(sum - c.x) * d.x, w1 = ex2_approx_ftz(sum - c.y) * d.y;
            const float w2 = ex2_approx_ftz(sum - c.z) * d.z, w3 = ex2_approx_ftz(sum - c.w) * d.w;
            m[2 * i] = pack_bf16x2(4 * i <= lane ? v[j][4 * i] * w0 : 0.0f, 4 * i + 1 <= lane ? v[j][4 * i + 1] * w1 : 0.0f);
            m[2 * i + 1] = pack_bf16x2(4 * i + 2 <= lane ? v[j][4 * i + 2] * w2 : 0.0f, 4 * i + 3 <= lane ? v[j][4 * i + 3] * w3 : 0.0f);
          }
        }
        tmem_store16(mine + kColM + half * 32 + 16 * j, m);
      }
    }
    // ---- w x in three terms, over C and h
    {
      const float w = now.weight[row];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t e[4] = {xv[c].x, xv[c].y, xv[c].z, xv[c].w};
        uint32_t hi[4], mid[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) split3(w * first_of(e[i]), w * second_of(e[i]), hi[i], mid[i], lo[i]);
        if (!all_finite) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t keep = ((e[i] & 0x7f80u) == 0x7f80u ? 0u : 0xffffu) | ((e[i] & 0x7f800000u) == 0x7f800000u ? 0u : 0xffff0000u);
            mid[i] &= keep;
            lo[i] &= keep;
          }
        }
        const uint32_t at = swizzled(row, half * 4 + c);
        sts128(base + kSmemC + at, make_uint4(hi[0], hi[1], hi[2], hi[3]));
        sts128(base + kSmemC + kTile + at, make_uint4(mid[0], mid[1], mid[2], mid[3]));
        sts128(base + kSmemH + at, make_uint4(lo[0], lo[1], lo[2], lo[3]));
      }
    }
    wait_stores();
    bulk::fence_proxy_async();
    fence_before_sync();
    __syncthreads();
    // ---- Y += M x, U = B^T (w x)
    if (tid == 128) {
      fence_after_sync();
#pragma unroll
      for (int k = 0; k < 8; ++k)
        mma_ts(tmem + kColY, tmem + kColM + 8 * k, desc_mn_major(base + kSmemX + k * 2048, kTile), instruction(128, 64, false, true), true);
      mma_commit(&tab.second);
#pragma unroll
      for (int term = 0; term < 3; ++term) {
        const uint32_t wx = base + (term == 2 ? kSmemH : kSmemC + term * kTile);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_ss(tmem + kColU, desc_mn_major(base + kSmemB + k * 2048, kTile), desc_mn_major(wx + k * 2048, kTile),
                 instruction(128, 64, true, true), term + k > 0);
      }
      mma_commit(&tab.third);
    }
    // ---- meanwhile: the gate, and the next chunk's decays
    const bool live = row < rows && columns > 0;
    uint4 zv[4] = {};
    if (z != nullptr && live) {
      const uint16_t *at = z + (t0 + row) * p.z_stride_t;
      if (columns == 32) {
        load64<WIDE>(at, zv);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (8 * c < columns) zv[c] = ld_stream(at + 8 * c);
      }
    }
    if (half == 0 && done + kQ < length) fill_decays(tab.decays[phase ^ 1], step_at(t0 + kQ), A2, row);
    // ---- out: skip, gate, round, store
    __syncwarp();
    fine &= bulk::mbar_wait(&tab.second, phase);
    __syncwarp();
    fence_after_sync();
    {
      float v[32];
      tmem_load32(mine + kColY + column, v);
      wait_loads();
      uint4 y[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t e[4] = {xv[c].x, xv[c].y, xv[c].z, xv[c].w}, f[4] = {zv[c].x, zv[c].y, zv[c].z, zv[c].w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2 r = make_float2(v[8 * c + 2 * i], v[8 * c + 2 * i + 1]);
          if (p.D != nullptr) r = __ffma2_rn(make_float2(skip, skip), make_float2(first_of(e[i]), second_of(e[i])), r);
          if (z != nullptr) r = __fmul2_rn(r, activate2<1>(make_float2(first_of(f[i]), second_of(f[i]))));
          o[i] = pack_bf16x2(r.x, r.y);
        }
        y[c] = make_uint4(o[0], o[1], o[2], o[3]);
      }
      if (live) {
        const int4 *bad = reinterpret_cast<const int4 *>(&tab.bad[column]);
        bool hit = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int4 f = bad[i];
          hit |= min(min(f.x, f.y), min(f.z, f.w)) <= row;
        }
        if (hit) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t o[4] = {y[c].x, y[c].y, y[c].z, y[c].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (tab.bad[column + 8 * c + 2 * i] <= row) o[i] = (o[i] & 0xffff0000u) | 0x7fffu;
              if (tab.bad[column + 8 * c + 2 * i + 1] <= row) o[i] = (o[i] & 0xffffu) | 0x7fff0000u;
            }
            y[c] = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
        put_row(t0 + row, y);
      }
    }
    // ---- the state; the next tiles are on their way meanwhile
    __syncwarp();
    fine &= bulk::mbar_wait(&tab.third, phase);
    if (tid == 0 && done + kQ < length) load_tiles(t0 + kQ);
    __syncwarp();
    fence_after_sync();
    {
      float v[32], u[32];
      tmem_load32(mine + kColH + column, v);
      tmem_load32(mine + kColU + column, u);
      wait_loads();
      const float decay = now.in[kQ - 1];
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = fmaf(v[i], decay, u[i]);
      tmem_store32(mine + kColH + column, v);
      wait_stores();
      put_h(v);
    }
    phase ^= 1;
  }
  fine = __syncthreads_and(fine);
  if (fine) {
    float v[32];
    tmem_load32(mine + kColH + column, v);
    wait_loads();
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < columns && row < K) state[(int64_t)(column + i) * K + row] = v[i];
  } else if (tid == 0) {
    atomicOr(p.status_dev != nullptr ? p.status_dev : &g_scan_error, kDevErrTimeout);
  }
  fence_before_sync();
  __syncthreads();
  if (warp == 0) {
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

namespace {

// Tensor map of a BF16 tensor [rows, groups, inner] (inner contiguous), boxes of 128 rows x 64.
cudaError_t encode(CUtensorMap *map, const void *data, int64_t inner, int64_t groups, int64_t rows, int64_t stride_group,
                   int64_t stride_row) {
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
  const cuuint32_t box[3] = {64, 1, kQ}, ones[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(data), dims, strides, box, ones,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <bool WIDE>
cudaError_t launch_wide(const ScanParams &p, const CUtensorMap (&maps)[3], cudaStream_t stream) {
  static std::atomic<bool> opted_in[64];
  const int dev = current_device();
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!opted_in[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(k_scan_chunked<WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
    if (e != cudaSuccess) return e;
    opted_in[dev].store(true, std::memory_order_release);
  }
  const int blocks_p = (int)((p.P + 63) / 64);
  return launch_overlapped(k_scan_chunked<WIDE>, dim3((unsigned)(p.n_seq * p.H * blocks_p)), dim3(kThreads), kSmemBytes, stream, p,
                           blocks_p, maps[0], maps[1], maps[2]);
}

}  // namespace

cudaError_t launch_scan_chunked(const ScanParams &p, cudaStream_t stream) {
  alignas(64) CUtensorMap maps[3];
  if (p.T > 0) {
    cudaError_t e = encode(&maps[0], p.x, p.P, p.H, p.T, p.x_stride_h, p.x_stride_t);
    if (e == cudaSuccess) e = encode(&maps[1], p.b, p.K, p.G, p.T, p.b_stride_g, p.b_stride_t);
    if (e == cudaSuccess) e = encode(&maps[2], p.c, p.K, p.G, p.T, p.c_stride_g, p.c_stride_t);
    if (e != cudaSuccess) return e;
  }
  auto on32 = [](const void *v, int64_t t, int64_t h) {
    return v == nullptr || (reinterpret_cast<uintptr_t>(v) % 32 == 0 && t % 16 == 0 && h % 16 == 0);
  };
  return on32(p.z, p.z_stride_t, p.z_stride_h) && on32(p.out, p.out_stride_t, p.out_stride_h) ? launch_wide<true>(p, maps, stream)
                                                                                            : launch_wide<false>(p, maps, stream);
}

}  // namespace ccu
