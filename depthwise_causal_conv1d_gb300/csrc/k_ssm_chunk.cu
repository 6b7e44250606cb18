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
// first two terms of w x, then Y's way out), h 16 KB (then the third term of w x).
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

struct Tables {
  float sum[kQ], step[kQ];    // running sum of log2 decays in its block of 32; d
  float from[4][kQ];          // [r][s]: decay from s to the token before block r, times d_s
  float in[kQ], weight[kQ];   // exp(c_t); w
  float total[4];
  float decay;                // exp(c_end)
  int bad[64];                // first token with a non-finite x, a channel
  uint64_t done;
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

__global__ void __launch_bounds__(kThreads, 2) k_scan_chunked(ScanParams p, int blocks_p) {
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
  uint16_t *out = static_cast<uint16_t *>(p.out) + h * p.out_stride_h + p0;
  const int out_row = tid >> 3, out_chunk = tid & 7;  // the 16 bytes of 32 rows this thread stores
  if (s < 0) {
    if (8 * out_chunk < np)
      for (int64_t t = q.begin + out_row; t < q.end; t += 32)
        *reinterpret_cast<uint4 *>(out + t * p.out_stride_t + 8 * out_chunk) = make_uint4(0, 0, 0, 0);
    return;
  }
  const uint16_t *x = static_cast<const uint16_t *>(p.x) + h * p.x_stride_h + p0;
  const uint16_t *bm = static_cast<const uint16_t *>(p.b) + g * p.b_stride_g;
  const uint16_t *cm = static_cast<const uint16_t *>(p.c) + g * p.c_stride_g;
  const uint16_t *z = p.z != nullptr ? static_cast<const uint16_t *>(p.z) + h * p.z_stride_h + p0 : nullptr;
  const uint16_t *dt = static_cast<const uint16_t *>(p.dt) + h;
  float *state = p.state + s * p.state_stride_s + (h * p.P + p0) * p.K;

  if (warp == 0) tmem_alloc(&tab.tmem, kColumns);
  if (tid == 0) {
    bulk::mbar_init(&tab.done, 1);
    bulk::fence_mbar_init();
  }
  if (tid < 64) tab.bad[tid] = kQ;
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = tab.tmem, mine = tmem + ((uint32_t)(quarter * 32) << 16);

  // 64 columns x rows of a tile: chunk c of row r, zero past the sequence's end and past `columns`.
  auto load_rows = [&](uint32_t tile, const uint16_t *from, int64_t stride, int64_t t0, int rows, int columns, int wide) {
    const int per_row = wide >> 3;  // 16-byte chunks a row
    for (int i = tid; i < kQ * per_row; i += kThreads) {
      const int r = i / per_row, c = i % per_row;
      const bool valid = r < rows && 8 * c < columns;
      copy16(base + tile + (c >> 3) * kTile + swizzled(r, c & 7), from + (valid ? (t0 + r) * stride + 8 * c : 0), valid);
    }
  };
  // The state's place in the operand tile of Y's product: row channel, K-major in k.
  auto put_h = [&](const float (&v)[32]) {
    const uint32_t at = base + kSmemH + (row >> 6) * (kTile / 2) + (half * 32) * 128 + (row & 7) * 2;
    const int chunk = (row >> 3) & 7;
#pragma unroll
    for (int i = 0; i < 32; ++i) sts16(at + i * 128 + ((chunk ^ (i & 7)) << 4), round_bf16(v[i]));
  };

  {
    float v[32];
    const bool initial = p.has_initial != nullptr && __ldg(p.has_initial + b) != 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const int pp = half * 32 + i;
      v[i] = initial && pp < np && row < K ? state[(int64_t)pp * K + row] : 0.0f;
    }
    tmem_store32(mine + kColH + half * 32, v);
    wait_stores();
    put_h(v);
  }

  const float A2 = __ldg(p.A + h) * kLog2e, skip = p.D != nullptr ? __ldg(p.D + h) : 0.0f;
  uint32_t phase = 0;
  bool fine = true;
  const int64_t length = q.end - q.begin;
  if (length > 0) {
    const int rows = (int)(length < kQ ? length : kQ);
    load_rows(kSmemB, bm, p.b_stride_t, q.begin, rows, K, 128);
    load_rows(kSmemX, x, p.x_stride_t, q.begin, rows, np, 64);
    load_rows(kSmemC, cm, p.c_stride_t, q.begin, rows, K, 128);
    copy_commit();
  }
  for (int64_t done = 0; done < length; done += kQ) {
    const int64_t t0 = q.begin + done;
    const int rows = (int)(length - done < kQ ? length - done : kQ);
    // ---- decays: warps 0..3, a token a thread
    if (half == 0) {
      const float d = row < rows ? step_size(__ldg(dt + (t0 + row) * p.dt_stride_t), p.dt_bias, h, p.dt_softplus) : 0.0f;
      float a = d * A2;
      a = a < kLeast ? kLeast : a;
      float sum = a, after = a;  // over the block up to this token, and from this token on
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float u = __shfl_up_sync(0xffffffffu, sum, o), w = __shfl_down_sync(0xffffffffu, after, o);
        if (lane >= o) sum += u;
        if (lane + o < 32) after += w;
      }
      if (lane == 31) tab.total[quarter] = sum;
      after = __shfl_down_sync(0xffffffffu, after, 1);
      if (lane == 31) after = 0.0f;
      bar_sync(1, 128);
      float before = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < quarter) before += tab.total[j];
      tab.sum[row] = sum;
      tab.step[row] = d;
      tab.in[row] = exp2f(before + sum);
      float reach = after;
#pragma unroll
      for (int r = 1; r < 4; ++r)
        if (r > quarter) {
          tab.from[r][row] = exp2f(reach) * d;
          reach += tab.total[r];
        }
      tab.weight[row] = exp2f(reach) * d;
      if (tid == 0) tab.decay = exp2f(tab.total[0] + tab.total[1] + tab.total[2] + tab.total[3]);
    }
    copy_wait_all();
    bulk::fence_proxy_async();
    fence_before_sync();
    __syncthreads();
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
      mma_commit(&tab.done);
    }
    // ---- meanwhile: this thread's x (32 channels of its token) and the gate it will store with
    uint4 xv[4], zv[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) xv[c] = lds128(base + kSmemX + swizzled(row, half * 4 + c));
    if (z != nullptr) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        zv[i] = make_uint4(0, 0, 0, 0);
        if (i * 32 + out_row < rows && 8 * out_chunk < np)
          zv[i] = ld_stream(z + (t0 + i * 32 + out_row) * p.z_stride_t + 8 * out_chunk);
      }
    }
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
          const int channel = half * 32 + 8 * c + 2 * i;
          if ((e[i] & 0x7f80u) == 0x7f80u) e[i] &= 0xffff0000u, atomicMin(&tab.bad[channel], row);
          if ((e[i] & 0x7f800000u) == 0x7f800000u) e[i] &= 0xffffu, atomicMin(&tab.bad[channel + 1], row);
        }
        sts128(base + kSmemX + swizzled(row, half * 4 + c), make_uint4(e[0], e[1], e[2], e[3]));
      }
    }
    fine &= bulk::mbar_wait(&tab.done, phase);
    phase ^= 1;
    __syncwarp();
    fence_after_sync();
    // ---- the rows of Y by exp(c_t)
    {
      float v[32];
      tmem_load32(mine + kColY + half * 32, v);
      wait_loads();
      const float e = tab.in[row];
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] *= e;
      tmem_store32(mine + kColY + half * 32, v);
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
      const float sum = tab.sum[row], local = exp2f(sum);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int block = half * 2 + j;
        uint32_t m[16];
        if (block > quarter) {
#pragma unroll
          for (int i = 0; i < 16; ++i) m[i] = 0;
        } else if (block < quarter) {
          const float4 *from = reinterpret_cast<const float4 *>(&tab.from[quarter][block * 32]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 f = from[i];
            m[2 * i] = pack_bf16x2(v[j][4 * i] * (local * f.x), v[j][4 * i + 1] * (local * f.y));
            m[2 * i + 1] = pack_bf16x2(v[j][4 * i + 2] * (local * f.z), v[j][4 * i + 3] * (local * f.w));
          }
        } else {
          const float4 *sums = reinterpret_cast<const float4 *>(&tab.sum[block * 32]);
          const float4 *steps = reinterpret_cast<const float4 *>(&tab.step[block * 32]);
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
      const float w = tab.weight[row];
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
    if (tid == 0) {
      fence_after_sync();
#pragma unroll
      for (int k = 0; k < 8; ++k)
        mma_ts(tmem + kColY, tmem + kColM + 8 * k, desc_mn_major(base + kSmemX + k * 2048, kTile), instruction(128, 64, false, true), true);
#pragma unroll
      for (int term = 0; term < 3; ++term) {
        const uint32_t wx = base + (term == 2 ? kSmemH : kSmemC + term * kTile);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_ss(tmem + kColU, desc_mn_major(base + kSmemB + k * 2048, kTile), desc_mn_major(wx + k * 2048, kTile),
                 instruction(128, 64, true, true), term + k > 0);
      }
      mma_commit(&tab.done);
    }
    fine &= bulk::mbar_wait(&tab.done, phase);
    phase ^= 1;
    __syncwarp();
    fence_after_sync();
    // ---- the next chunk's B and x; C's place is Y's way out first
    const int64_t next = done + kQ;
    const int next_rows = (int)(length - next < kQ ? length - next : kQ);
    if (next < length) {
      load_rows(kSmemB, bm, p.b_stride_t, q.begin + next, next_rows, K, 128);
      load_rows(kSmemX, x, p.x_stride_t, q.begin + next, next_rows, np, 64);
    }
    {
      float v[32];
      tmem_load32(mine + kColY + half * 32, v);
      wait_loads();
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t e[4] = {xv[c].x, xv[c].y, xv[c].z, xv[c].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = 8 * c + 2 * i;
          if (p.D != nullptr) {
            v[at] = fmaf(skip, first_of(e[i]), v[at]);
            v[at + 1] = fmaf(skip, second_of(e[i]), v[at + 1]);
          }
        }
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const int chunk = (half * 8 + c) ^ (row & 7);
        sts128(base + kSmemC + row * 256 + (chunk << 4),
               make_uint4(__float_as_uint(v[4 * c]), __float_as_uint(v[4 * c + 1]), __float_as_uint(v[4 * c + 2]), __float_as_uint(v[4 * c + 3])));
      }
    }
    {
      float v[32], u[32];
      tmem_load32(mine + kColH + half * 32, v);
      tmem_load32(mine + kColU + half * 32, u);
      wait_loads();
      const float decay = tab.decay;
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = fmaf(v[i], decay, u[i]);
      tmem_store32(mine + kColH + half * 32, v);
      wait_stores();
      put_h(v);
    }
    fine = __syncthreads_and(fine);
    if (!fine) break;
    // ---- out: gate, round, store
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = i * 32 + out_row;
      if (r < rows && 8 * out_chunk < np) {
        // even chunks first in one half of the row's threads, odd ones in the other: no bank twice
        const int flip = out_chunk >> 2;
        const uint4 a = lds128(base + kSmemC + r * 256 + (((2 * out_chunk + flip) ^ (r & 7)) << 4));
        const uint4 c = lds128(base + kSmemC + r * 256 + (((2 * out_chunk + 1 - flip) ^ (r & 7)) << 4));
        const uint4 lo = flip ? c : a, hi = flip ? a : c;
        float y[8] = {__uint_as_float(lo.x), __uint_as_float(lo.y), __uint_as_float(lo.z), __uint_as_float(lo.w),
                      __uint_as_float(hi.x), __uint_as_float(hi.y), __uint_as_float(hi.z), __uint_as_float(hi.w)};
        if (z != nullptr) {
          float2 f[4];
          widen8(zv[i], f);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 w = activate2<1>(f[e]);
            y[2 * e] *= w.x;
            y[2 * e + 1] *= w.y;
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (tab.bad[8 * out_chunk + e] <= r) y[e] = __uint_as_float(0x7fffffffu);
        st_stream(out + (t0 + r) * p.out_stride_t + 8 * out_chunk,
                  make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7])));
      }
    }
    __syncthreads();
    if (tid < 64) tab.bad[tid] = kQ;
    if (next < length) load_rows(kSmemC, cm, p.c_stride_t, q.begin + next, next_rows, K, 128);
    copy_commit();
  }
  copy_wait_all();
  if (fine) {
    float v[32];
    tmem_load32(mine + kColH + half * 32, v);
    wait_loads();
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const int pp = half * 32 + i;
      if (pp < np && row < K) state[(int64_t)pp * K + row] = v[i];
    }
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

cudaError_t launch_scan_chunked(const ScanParams &p, cudaStream_t stream) {
  static std::atomic<bool> opted_in[64];
  const int dev = current_device();
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!opted_in[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(k_scan_chunked, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
    if (e != cudaSuccess) return e;
    opted_in[dev].store(true, std::memory_order_release);
  }
  const int blocks_p = (int)((p.P + 63) / 64);
  return launch_overlapped(k_scan_chunked, dim3((unsigned)(p.n_seq * p.H * blocks_p)), dim3(kThreads), kSmemBytes, stream, p, blocks_p);
}

}  // namespace ccu
