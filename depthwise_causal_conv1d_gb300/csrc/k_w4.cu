// Products of a few rows with 4-bit weights (ccu_w4_matmul).
//
// The weights are read once and bound the call (0.5 bytes each; every other operand is small), so
// what has to be kept low is the work a weight costs on its way to the multiplier: it is widened
// to BF16 as q - 8, which is exact, in 1.4 instructions, and multiplied on the tensor cores: up to 8 rows
// from registers (mma.sync m16n8k16: 16 outputs, 8 token rows, 16 inputs), more rows through TMEM (tcgen05).
// The boundary: 8 rows 8192 x 16384 30 us there, 9 rows 29 here; at 16768 x 4096 22 and 30. A group's sums stay in 32 bits, are scaled in 32 bits, and added up in 32 bits; zero points other
// than 8 enter as (8 - zero) * (sum of the group's inputs).
#include <atomic>
#include <cfloat>
#include <type_traits>

#include "ssm_tensor.cuh"

namespace ccu {

int device_sm_count();
int current_device();

__device__ int32_t g_w4_error = 0;        // CCU_DEVERR_* bits
__device__ int32_t g_w4_error_taken = 0;  // the value the last exchange read

__global__ void k_exchange_w4_error() {
  grid_dependency_boundary();
  g_w4_error_taken = atomicExch(&g_w4_error, 0);
}

namespace {

// ------------------------------------------------------------------ any alignment

// One warp per (output, row of x): the lanes walk the inputs eight at a time. For operands that
// are not on 16-byte boundaries; the anchor of the kernel below.
__global__ void __launch_bounds__(256) k_w4_scalar(W4Params p) {
  grid_dependency_boundary();
  const int lane = threadIdx.x & 31;
  const int64_t o = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (o >= p.O) return;
  const uint32_t *q = static_cast<const uint32_t *>(p.qweight) + o * (p.I / 8);
  const uint16_t *scales = static_cast<const uint16_t *>(p.scales) + o * (p.I / p.group);
  const uint16_t *zeros = static_cast<const uint16_t *>(p.zeros);
  if (zeros != nullptr) zeros += o * (p.I / p.group);
  for (int64_t m = blockIdx.y; m < p.M; m += gridDim.y) {
    const uint16_t *x = static_cast<const uint16_t *>(p.x) + m * p.ld_x;
    float acc = 0.0f;
    for (int64_t i = lane * 8; i < p.I; i += 256) {
      const uint32_t word = __ldg(q + i / 8);
      const int64_t g = i / p.group;
      const float zero = zeros != nullptr ? bf16_bits(__ldg(zeros + g)) : 8.0f;
      float part = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        part = fmaf((float)((word >> (4 * e)) & 15u) - zero, bf16_bits(__ldg(x + i + e)), part);
      acc = fmaf(part, bf16_bits(__ldg(scales + g)), acc);
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, s);
    if (lane == 0) static_cast<uint16_t *>(p.out)[m * p.ld_out + o] = round_bf16(acc);
  }
}

// One output as it is defined, a product (q - zero) x at a time, in one thread: its rows of weights, scales, zero points and x.
__device__ __noinline__ float by_definition(const uint32_t *q, const uint16_t *scales, const uint16_t *zeros, const uint16_t *x, int groups,
                                            int group) {
  float acc = 0.0f;
  for (int g = 0; g < groups && acc == acc; ++g) {  // a NaN stays one
    const float zero = bf16_bits(__ldg(zeros + g));
    float part = 0.0f;
    for (int64_t i = (int64_t)g * group; i < (int64_t)(g + 1) * group; i += 8) {
      const uint32_t word = __ldg(q + i / 8);
#pragma unroll
      for (int e = 0; e < 8; ++e) part = fmaf((float)((word >> (4 * e)) & 15u) - zero, bf16_bits(__ldg(x + i + e)), part);
    }
    acc = fmaf(part, bf16_bits(__ldg(scales + g)), acc);
  }
  return acc;
}

// An output on its way out. With zero points its sum came from the sums of (q - 8) x and (8 - zero) x, which an
// infinite x can make infinities of opposite signs where (q - zero) x is one infinity: what is not finite is summed again.
// (5 rows 16768 x 4096, weights not in L2: 21.5 us with the test, 20.9 without.)
template <bool ZEROS>
__device__ __forceinline__ uint16_t finish(const W4Params &p, float sum, int64_t o, int64_t m) {
  if (ZEROS && !(fabsf(sum) <= FLT_MAX)) {
    const int groups = (int)(p.I / p.group);
    sum = by_definition(static_cast<const uint32_t *>(p.qweight) + o * (p.I / 8), static_cast<const uint16_t *>(p.scales) + o * groups,
                        static_cast<const uint16_t *>(p.zeros) + o * groups, static_cast<const uint16_t *>(p.x) + m * p.ld_x, groups,
                        (int)p.group);
  }
  return round_bf16(sum);
}

// ------------------------------------------------------------------ matrix instructions

// D[16 x 8] += A[16 x 16] B[16 x 8], BF16 in, FP32 out. Lane l = 4 r + t holds A's rows r and
// r + 8, B's column r and D's columns 2t, 2t + 1; along the 16 inputs it holds four, the pairs
// (2t, 2t + 1) and (2t + 8, 2t + 9). Which inputs of the group these stand for is free, as long as A and B agree.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Nibbles e and e + 4 of a word as a BF16 pair q - 8: 0x4300 | q is 128 + q.
template <int E>
__device__ __forceinline__ uint32_t widen_pair(uint32_t word) {
  const uint32_t v = ((word >> (4 * E)) & 0x000f000fu) | 0x43004300u;
  const __nv_bfloat162 minus = __halves2bfloat162(__ushort_as_bfloat16(0xc308), __ushort_as_bfloat16(0xc308));  // -136
  const __nv_bfloat162 r = __hadd2(*reinterpret_cast<const __nv_bfloat162 *>(&v), minus);
  return *reinterpret_cast<const uint32_t *>(&r);
}

template <int GROUP>
struct Words;  // a lane's quarter of a group: GROUP / 4 nibbles
template <> struct Words<128> { uint4 v; __device__ uint32_t get(int i) const { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; } };
template <> struct Words<64> { uint2 v; __device__ uint32_t get(int i) const { return i == 0 ? v.x : v.y; } };
template <> struct Words<32> { uint32_t v; __device__ uint32_t get(int) const { return v; } };

// Eight inputs of a token row in the pairs (0,4) (1,5) (2,6) (3,7) that the nibbles of a word come in.
__device__ __forceinline__ uint4 pair_up(uint4 e) {
  return make_uint4(__byte_perm(e.x, e.z, 0x5410), __byte_perm(e.x, e.z, 0x7632), __byte_perm(e.y, e.w, 0x5410), __byte_perm(e.y, e.w, 0x7632));
}

// A CTA's rows of scales and zero points that a lane needs (its outputs r and r + 8).
struct Rows {
  const uint16_t *sa, *sb, *za, *zb;
};

// ------------------------------------------------------------------ up to 8 token rows
//
// A CTA computes 16 outputs; its 8 warps take the groups of inputs in turn and join their sums in
// shared memory; where the outputs are too few to fill the card the inputs are split over a cluster as well
// (8 rows 1024 x 8192, groups of 32: 8.2 us, 23.7 unsplit). A lane reads the quarter t of a group of
// rows r and r + 8 (16, 8 or 4 bytes each: four lanes cover a row's group), kPre groups ahead of their use.
// What bounds it are the instructions between a load and its use: 1 row 8512 x 2048 4.7 us, 5 rows 16768 x 4096 (zero
// points, groups of 64) 19, 1 row 8192 x 16384 26 (2.6 TB/s of weights). Left out, for the second: x, scales and zero points as far ahead as the
// weights (146 registers instead of 72) 23.6 us; x one group ahead 22.0; scales and zero points alone 21.9; weights and x in
// asynchronous copies to shared memory, 32 outputs a CTA, 20.3 (52 % of the issue slots taken; 25 for the third, 5.2 for the first).
constexpr int kWarps = 8;

// SPLIT apart: the split's registers cost the unsplit kernel a CTA an SM (26 -> 35 us for the third). Groups of 128 without zero
// points spill 16 bytes at the 64 registers the compiler picks (four CTAs an SM).
template <int GROUP, bool ZEROS, bool SPLIT>
__global__ void __launch_bounds__(32 * kWarps) k_w4_few(W4Params p, int split) {
  grid_dependency_boundary();
  constexpr int kWords = GROUP / 32;             // 32-bit words a lane and row of a group
  constexpr int kPre = GROUP == 128 ? 2 : 4;
  __shared__ float joined[kWarps][16][9], sums_of[SPLIT ? 8 : 1][16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, t = lane & 3;
  const int rank = SPLIT ? (int)blockIdx.x % split : 0;  // place in the cluster
  const int64_t o0 = (int64_t)(SPLIT ? blockIdx.x / split : blockIdx.x) * 16;
  const int groups = (int)(p.I / GROUP);
  const int from = SPLIT ? (int)((int64_t)groups * rank / split) : 0, to = SPLIT ? (int)((int64_t)groups * (rank + 1) / split) : groups;
  const int64_t oa = o0 + r < p.O ? o0 + r : p.O - 1, ob = o0 + r + 8 < p.O ? o0 + r + 8 : p.O - 1;
  using Vec = Words<GROUP>;
  const Vec *qa = reinterpret_cast<const Vec *>(static_cast<const uint32_t *>(p.qweight) + oa * (p.I / 8)) + t;
  const Vec *qb = reinterpret_cast<const Vec *>(static_cast<const uint32_t *>(p.qweight) + ob * (p.I / 8)) + t;
  const uint16_t *scales = static_cast<const uint16_t *>(p.scales), *zeros = static_cast<const uint16_t *>(p.zeros);
  const Rows rows = {scales + oa * groups, scales + ob * groups, ZEROS ? zeros + oa * groups : nullptr, ZEROS ? zeros + ob * groups : nullptr};
  const uint16_t *x = r < p.M ? static_cast<const uint16_t *>(p.x) + r * p.ld_x + t * (GROUP / 4) : nullptr;
  float total[4] = {};
  Vec wa[kPre], wb[kPre];
  auto fetch = [&](int slot, int g) {
    if (g >= to) return;
    wa[slot].v = __ldcs(&qa[4 * g].v);
    wb[slot].v = __ldcs(&qb[4 * g].v);
  };
#pragma unroll
  for (int i = 0; i < kPre; ++i) fetch(i, from + warp + i * kWarps);
  for (int g0 = from + warp; g0 < to; g0 += kPre * kWarps) {
#pragma unroll
    for (int i = 0; i < kPre; ++i) {
      const int g = g0 + i * kWarps;
      if (g >= to) break;
      const Vec va = wa[i], vb = wb[i];
      fetch(i, g + kPre * kWarps);
      const float fa = bf16_bits(__ldg(rows.sa + g)), fb = bf16_bits(__ldg(rows.sb + g));
      float acc[4] = {}, sums[4] = {};
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        const uint32_t u = va.get(w), v = vb.get(w);
        const uint32_t a0[4] = {widen_pair<0>(u), widen_pair<0>(v), widen_pair<1>(u), widen_pair<1>(v)};
        const uint32_t a1[4] = {widen_pair<2>(u), widen_pair<2>(v), widen_pair<3>(u), widen_pair<3>(v)};
        const uint32_t ones[4] = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
        uint4 e = make_uint4(0, 0, 0, 0);
        if (x != nullptr) e = pair_up(__ldg(reinterpret_cast<const uint4 *>(x + (int64_t)g * GROUP + 8 * w)));
        mma16816(acc, a0, e.x, e.y);
        mma16816(acc, a1, e.z, e.w);
        if (ZEROS) {
          mma16816(sums, ones, e.x, e.y);
          mma16816(sums, ones, e.z, e.w);
        }
      }
      float ca = 0.0f, cb = 0.0f;
      if (ZEROS) ca = 8.0f - bf16_bits(__ldg(rows.za + g)), cb = 8.0f - bf16_bits(__ldg(rows.zb + g));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float v = ZEROS ? fmaf(j < 2 ? ca : cb, sums[j], acc[j]) : acc[j];
        total[j] = fmaf(j < 2 ? fa : fb, v, total[j]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) joined[warp][r + (j >> 1) * 8][2 * t + (j & 1)] = total[j];
  __syncthreads();
  const int o = threadIdx.x & 15, m = threadIdx.x >> 4;
  uint16_t *out = static_cast<uint16_t *>(p.out) + m * p.ld_out + o0 + o;
  const bool there = o0 + o < p.O && m < p.M;
  if (threadIdx.x < 128) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += joined[w][o][m];
    if (SPLIT) sums_of[m][o] = v;
    else if (there) *out = finish<ZEROS>(p, v, o0 + o, m);
  }
  if (SPLIT) {
    cluster_sync();
    if (o / (16 / split) == rank && there) {     // each CTA adds up a part of the outputs, in rank order
      float sum = 0.0f;
      for (int i = 0; i < split; ++i) sum += cluster_load(&sums_of[m][o], i);
      *out = finish<ZEROS>(p, sum, o0 + o, m);
    }
    cluster_sync();  // nobody leaves while its sums may be read
  }
}

// ------------------------------------------------------------------ more token rows
//
// A CTA computes 128 outputs for N token rows on the fifth-generation tensor cores (tcgen05), 128 inputs a
// step: a warp copies the step's weights and x with tiled copies (kRing steps ahead), two sets of four warps
// take the steps in turn and widen the weights into TMEM (a thread a row), one warp issues the products, with one
// accumulator for every group of the step, and eight warps scale the accumulators and add them up in registers.
// The weights go through TMEM because shared memory is what a step fills most: widened there, 32 KB written
// and 32 KB read a step beside x. Two warps issue products, for their three waits a step. 64 rows 8192 x 16384: 35 us, a step
// of 128 inputs some 750 cycles, half of a widening set's turn (55 us with the widened tile in shared memory, 50 with
// waits one after the other and one issuing warp, 85 with one set of warps for everything, 95 on mma.sync; three sets of widening warps 35 too, and
// registers for them spill with groups of 64: 65 us instead of 42 at 16768 x 4096). The inputs are split over the CTAs of a cluster, which
// join their 32-bit sums through distributed shared memory in rank order (the same bits in every run): 8192
// outputs are only 64 CTAs otherwise. All waits have a limit.
//
// Barriers: full (a step's copies have landed; the copying warp refills a place of the ring once the
// products that read it are done: empty), widened, read (the products that read a widened tile are done), done (the
// same for their accumulators), added (the accumulators are free), summed (the sums of x are). Each barrier's
// next phase needs what every waiter of the present one does after its wait, so no waiter falls behind by two phases.
//
// A CTA takes an SM's whole TMEM, and shared memory enough that no second one is placed beside it: CTAs of
// two clusters could otherwise wait for each other's TMEM.
constexpr int kStep = 128;                       // inputs a step
constexpr int kTileO = 128;                      // outputs a CTA
constexpr int kRawW = kTileO * kStep / 2;        // a step's weights as they come
constexpr int kSets = 2, kWiden = 4 * kSets, kAdd = 8;  // sets of widening warps; warps
constexpr int kTiles = 4;                        // widened tiles in TMEM, kStep / 2 columns each
constexpr int kColumns = 512;
constexpr int kMma = 2;                          // warps that issue products, taking the steps in turn
constexpr int kTileThreads = 32 * (kWiden + kAdd + kMma + 1);

template <int N>
struct Smem {
  static constexpr int kRing = N == 64 ? 8 : N == 32 ? 12 : 16;
  static constexpr int kBlockX = N * 128, kPlace = kRawW + 2 * kBlockX;   // of the ring: x, weights
  static constexpr int kSums = kRing * kPlace;
  static constexpr size_t kBytes = kSums + kTiles * 4 * N * sizeof(float) + 1024;
  static_assert(2 * kBytes > 227 * 1024, "one CTA an SM");
};

// Eight weights of a word as BF16 q - 8, in their order.
__device__ __forceinline__ uint4 widen8(uint32_t word) {
  const uint32_t even = word & 0x0f0f0f0fu, odd = (word >> 4) & 0x0f0f0f0fu;
  const uint32_t low = __byte_perm(even, odd, 0x5140), high = __byte_perm(even, odd, 0x7362);
  const uint32_t v[4] = {__byte_perm(low, 0x43u, 0x4140), __byte_perm(low, 0x43u, 0x4342), __byte_perm(high, 0x43u, 0x4140),
                         __byte_perm(high, 0x43u, 0x4342)};
  const __nv_bfloat162 minus = __halves2bfloat162(__ushort_as_bfloat16(0xc308), __ushort_as_bfloat16(0xc308));  // -136
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 d = __hadd2(*reinterpret_cast<const __nv_bfloat162 *>(&v[i]), minus);
    r[i] = *reinterpret_cast<const uint32_t *>(&d);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

template <int GROUP, int N, bool ZEROS>
__global__ void __launch_bounds__(kTileThreads, 1) k_w4_tile(W4Params p, int split, const __grid_constant__ CUtensorMap map_w,
                                                             const __grid_constant__ CUtensorMap map_x) {
  grid_dependency_boundary();
  using S = Smem<N>;
  constexpr int kGroups = kStep / GROUP, kHalf = N / 2, kRing = S::kRing;
  constexpr int kTilesAt = 2 * kGroups * N;      // TMEM column of the widened tiles, behind two steps' accumulators
  constexpr int kPieces = N * 16 / 128;          // 16-byte pieces of x a widening thread and step
  static_assert(kTilesAt + kTiles * kStep / 2 <= kColumns, "an SM's TMEM");
  extern __shared__ __align__(16) unsigned char raw[];
  __shared__ uint64_t full[kRing], empty[kRing], widened[kTiles], read[kTiles], summed[kTiles], done[2], added[2];
  __shared__ uint32_t tmem_at;
  const uint32_t base = (bulk::smem_addr(raw) + 1023) & ~1023u;
  float *sums = reinterpret_cast<float *>(raw + (base - bulk::smem_addr(raw)) + S::kSums);  // [step % kTiles][group][N]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)blockIdx.x % split;      // place in the cluster
  const int64_t o0 = (int64_t)(blockIdx.x / split) * kTileO, m0 = (int64_t)blockIdx.y * N;
  const int groups = (int)(p.I / GROUP), all = (int)((p.I + kStep - 1) / kStep);
  const int from = (int)((int64_t)all * rank / split), steps = (int)((int64_t)all * (rank + 1) / split) - from;

  if (warp == 0) tensor::tmem_alloc(&tmem_at, kColumns);
  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) bulk::mbar_init(&full[i], 1), bulk::mbar_init(&empty[i], 1);
    for (int i = 0; i < kTiles; ++i) bulk::mbar_init(&widened[i], 4), bulk::mbar_init(&read[i], 1), bulk::mbar_init(&summed[i], kAdd);
    for (int i = 0; i < 2; ++i) bulk::mbar_init(&done[i], 1), bulk::mbar_init(&added[i], kAdd);
    bulk::fence_mbar_init();
  }
  tensor::fence_before_sync();
  __syncthreads();
  tensor::fence_after_sync();
  const uint32_t tmem = tmem_at;
  bool fine = true;
  // the output and the rows whose sums this thread keeps
  const int quarter = warp & 3, half = (warp >> 2) & 1, mine = quarter * 32 + lane;
  float total[kHalf];

  if (warp < kWiden) {
    for (int i = warp >> 2; i < steps; i += kSets) {
      const int tile = i % kTiles, place = i % kRing;
      const uint32_t at_x = base + place * S::kPlace, at_w = at_x + 2 * S::kBlockX + mine * (kStep / 2);
      const uint32_t landed = (i / kRing) & 1, before = i >= kTiles ? (i / kTiles - 1) & 1 : landed;
      uint64_t &room = i >= kTiles ? read[tile] : full[place];   // the first steps find their tiles free
      if (ZEROS) fine = tensor::wait_phases(&full[place], landed, &room, before, i >= kTiles ? &summed[tile] : &full[place], before);
      else fine = tensor::wait_phases(&full[place], landed, &room, before);
      fine = __all_sync(0xffffffffu, fine);
      if (!fine) break;
      tensor::fence_after_sync();
      uint4 v[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = tensor::lds128(at_w + ((c ^ (mine >> 1 & 3)) << 4));  // the 64-byte swizzle
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t words[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
        uint32_t out[16];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint4 e = widen8(words[k]);
          out[4 * k] = e.x, out[4 * k + 1] = e.y, out[4 * k + 2] = e.z, out[4 * k + 3] = e.w;
        }
        tensor::tmem_store16(tmem + ((uint32_t)(quarter * 32) << 16) + kTilesAt + tile * (kStep / 2) + c * 16, out);
      }
      if (ZEROS) {  // a group's sum of x: GROUP / 8 neighbouring threads hold it
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
          const int at = (tid & 127) + j * 128, n = at >> 4, c = at & 15;
          const uint4 e = tensor::lds128(at_x + (c >> 3) * S::kBlockX + tensor::swizzled(n, c & 7));
          float sum = ((bf16_lo(e.x) + bf16_hi(e.x)) + (bf16_lo(e.y) + bf16_hi(e.y))) +
                      ((bf16_lo(e.z) + bf16_hi(e.z)) + (bf16_lo(e.w) + bf16_hi(e.w)));
#pragma unroll
          for (int o = 1; o < GROUP / 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          if (c % (GROUP / 8) == 0) sums[(tile * 4 + c / (GROUP / 8)) * N + n] = sum;
        }
      }
      tensor::wait_stores();
      tensor::fence_before_sync();
      __syncwarp();
      if (lane == 0) bulk::mbar_arrive(&widened[tile]);
    }
  } else if (warp < kWiden + kAdd) {
    const uint32_t sums_at = tmem + ((uint32_t)(quarter * 32) << 16) + half * kHalf;
    const int64_t os = o0 + mine < p.O ? o0 + mine : p.O - 1;
    const uint16_t *scales = static_cast<const uint16_t *>(p.scales) + os * groups;
    const uint16_t *zeros = ZEROS ? static_cast<const uint16_t *>(p.zeros) + os * groups : nullptr;
    uint16_t sc[2][kGroups], ze[2][kGroups];     // of two steps
    auto fetch = [&](auto which, int i) {
      constexpr int kBuffer = decltype(which)::value;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const int at = (from + i) * kGroups + g < groups ? (from + i) * kGroups + g : groups - 1;
        sc[kBuffer][g] = __ldg(scales + at);
        if (ZEROS) ze[kBuffer][g] = __ldg(zeros + at);
      }
    };
    // Scales the accumulators of a step and adds them up; `which` is i % 2. False: a wait ran out.
    auto add = [&](auto which, int i) {
      constexpr int kBuffer = decltype(which)::value;
      const int tile = i % kTiles;
      if (ZEROS) fine = bulk::mbar_wait(&widened[tile], (i / kTiles) & 1);  // the sums of x
      fine &= bulk::mbar_wait(&done[kBuffer], (i >> 1) & 1);
      if (!__all_sync(0xffffffffu, fine)) return fine = false;
      tensor::fence_after_sync();
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        if ((from + i) * kGroups + g >= groups) break;
        const float2 scale = make_float2(bf16_bits(sc[kBuffer][g]), bf16_bits(sc[kBuffer][g]));
        const float shift = ZEROS ? 8.0f - bf16_bits(ze[kBuffer][g]) : 0.0f;
#pragma unroll
        for (int k = 0; k < kHalf; k += 8) {
          float v[8];
          tensor::tmem_load8(sums_at + (kBuffer * kGroups + g) * N + k, v);
          tensor::wait_loads();
          tensor::loaded(v);
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            float2 u = make_float2(v[j], v[j + 1]);
            if (ZEROS) {
              const float *s = &sums[(tile * 4 + g) * N + half * kHalf + k + j];
              u = __ffma2_rn(make_float2(shift, shift), make_float2(s[0], s[1]), u);
            }
            const float2 r = __ffma2_rn(scale, u, make_float2(total[k + j], total[k + j + 1]));
            total[k + j] = r.x;
            total[k + j + 1] = r.y;
          }
        }
      }
      tensor::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        bulk::mbar_arrive(&added[kBuffer]);
        if (ZEROS) bulk::mbar_arrive(&summed[tile]);
      }
      if (i + 2 < steps) fetch(which, i + 2);
      return true;
    };
    using Even = std::integral_constant<int, 0>;
    using Odd = std::integral_constant<int, 1>;
#pragma unroll
    for (int k = 0; k < kHalf; ++k) total[k] = 0.0f;
    if (steps > 0) fetch(Even(), 0);
    if (steps > 1) fetch(Odd(), 1);
    for (int i = 0; i < steps; i += 2) {
      if (!add(Even(), i)) break;
      if (i + 1 < steps && !add(Odd(), i + 1)) break;
    }
  } else if (warp < kWiden + kAdd + kMma) {
    uint64_t x_k = tensor::desc_k_major(base);
    asm volatile("" : "+l"(x_k));  // opaque, as in the chunked scan
    int last = -1;
    for (int i = warp - kWiden - kAdd; i < steps; i += kMma) {
      const int buffer = i & 1, tile = i % kTiles, place = i % kRing;
      uint64_t &room = i >= 2 ? added[buffer] : full[place];   // the first two steps find their accumulators free
      fine = tensor::wait_phases(&full[place], (i / kRing) & 1, &widened[tile], (i / kTiles) & 1, &room,
                                 i >= 2 ? ((i >> 1) - 1) & 1 : (i / kRing) & 1);
      fine = __all_sync(0xffffffffu, fine);
      if (!fine) break;
      tensor::fence_after_sync();
      if (tensor::elect_one()) {
        const uint64_t x = x_k + place * (S::kPlace >> 4);
#pragma unroll
        for (int k = 0; k < kStep / 16; ++k)
          if ((from + i) * kGroups + k * 16 / GROUP < groups)
            tensor::mma_ts(tmem + (buffer * kGroups + k * 16 / GROUP) * N, tmem + kTilesAt + tile * (kStep / 2) + k * 8,
                           x + (k >> 2) * (S::kBlockX >> 4) + (k & 3) * 2, tensor::instruction(128, N, false, false), k * 16 % GROUP != 0);
        tensor::mma_commit(&empty[place]);
        tensor::mma_commit(&read[tile]);
        tensor::mma_commit(&done[buffer]);
      }
      __syncwarp();
      last = i;
    }
    // its products are done before anybody leaves
    if (last >= 0) fine &= bulk::mbar_wait(&done[last & 1], (last >> 1) & 1);
  } else if (lane == 0) {
    int issued = 0;
    for (int i = 0; i < steps; ++i) {
      const int place = i % kRing;
      if (i >= kRing) fine = bulk::mbar_wait(&empty[place], (i / kRing - 1) & 1);
      if (!fine) break;
      const uint32_t at_x = base + place * S::kPlace;
      bulk::mbar_arrive_expect_tx(&full[place], S::kPlace);
      tensor::tile_load(at_x, &map_x, (from + i) * kStep, 0, (int)m0, &full[place]);
      tensor::tile_load(at_x + S::kBlockX, &map_x, (from + i) * kStep + 64, 0, (int)m0, &full[place]);
      tensor::tile_load(at_x + 2 * S::kBlockX, &map_w, (from + i) * (kStep / 4), 0, (int)o0, &full[place]);
      issued = i + 1;
    }
    // its copies have landed before anybody leaves
    for (int i = issued > kRing ? issued - kRing : 0; i < issued; ++i) fine &= bulk::mbar_wait(&full[i % kRing], (i / kRing) & 1);
  }
  __syncwarp();
  fine = __syncthreads_and(fine);
  if (!fine && tid == 0) atomicOr(&g_w4_error, kDevErrTimeout);
  // Join: every CTA puts its sums into its shared memory and adds up a part of the outputs over all of them.
  constexpr int kRow = N + 1;
  float *joined = reinterpret_cast<float *>(raw);
  if (warp >= kWiden && warp < kWiden + kAdd) {
#pragma unroll
    for (int k = 0; k < kHalf; ++k) joined[mine * kRow + half * kHalf + k] = total[k];
  }
  cluster_sync();
  const int part = kTileO / split;               // outputs a CTA adds up
  for (int i = tid; i < part * N; i += kTileThreads) {
    const int o = rank * part + i % part, m = i / part;
    if (o0 + o >= p.O || m0 + m >= p.M) continue;
    float v = 0.0f;
    for (int s = 0; s < split; ++s) v += cluster_load(joined + o * kRow + m, s);
    static_cast<uint16_t *>(p.out)[(m0 + m) * p.ld_out + o0 + o] = finish<ZEROS>(p, v, o0 + o, m0 + m);
  }
  cluster_sync();  // nobody leaves while its sums may be read
  if (warp == 0) {
    tensor::fence_after_sync();
    tensor::tmem_free(tmem, kColumns);
  }
}

template <int GROUP, bool ZEROS>
cudaError_t launch_few(const W4Params &p, cudaStream_t stream) {
  // About three CTAs an SM; the inputs are split while all of them fit and every warp keeps two groups.
  const int64_t tiles = (p.O + 15) / 16;
  int split = 1;
  while (split < 8 && tiles * split * 2 <= 3 * device_sm_count() && p.I / GROUP >= 4 * kWarps * split) split *= 2;
  if (split == 1) return launch_overlapped(k_w4_few<GROUP, ZEROS, false>, dim3((unsigned)tiles), dim3(32 * kWarps), 0, stream, p, 1);
  return launch_cluster(k_w4_few<GROUP, ZEROS, true>, dim3((unsigned)(tiles * split)), dim3(32 * kWarps), 0, split, stream, p, split);
}

template <int GROUP, int N, bool ZEROS>
cudaError_t launch_tile(const W4Params &p, cudaStream_t stream) {
  constexpr size_t kBytes = Smem<N>::kBytes;
  static std::atomic<bool> opted_in[64];
  const int dev = current_device();
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!opted_in[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(k_w4_tile<GROUP, N, ZEROS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kBytes);
    if (e != cudaSuccess) return e;
    opted_in[dev].store(true, std::memory_order_release);
  }
  alignas(64) CUtensorMap map_w = {}, map_x = {};
  cudaError_t e = encode_tiles(&map_w, p.qweight, p.I / 4, 1, p.O, 0, p.I / 4, kStep / 4, kTileO, CU_TENSOR_MAP_SWIZZLE_64B);
  if (e == cudaSuccess) e = encode_tiles(&map_x, p.x, p.I, 1, p.M, 0, p.ld_x, 64, N, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  const int64_t tiles_o = (p.O + kTileO - 1) / kTileO, tiles_m = (p.M + N - 1) / N;
  // One CTA an SM; the inputs are split while that gives every CTA an SM of its own and two steps at least.
  // Clusters of 8 leave SMs of their GPCs out, so they count for more (64 rows 1024 x 8192, groups of 32: 16 clusters 28 us).
  int split = 1;
  const auto fits = [&](int n) { return tiles_o * tiles_m * n <= (n == 8 ? device_sm_count() * 3 / 4 : device_sm_count()); };
  while (split < 8 && fits(split * 2) && p.I / kStep >= 4 * split) split *= 2;
  return launch_cluster(k_w4_tile<GROUP, N, ZEROS>, dim3((unsigned)(tiles_o * split), (unsigned)tiles_m), dim3(kTileThreads), kBytes, split,
                        stream, p, split, map_w, map_x);
}

template <int GROUP, bool ZEROS>
cudaError_t launch_rows(const W4Params &p, cudaStream_t stream) {
  if (p.M <= 8) return launch_few<GROUP, ZEROS>(p, stream);
  if (p.M <= 16) return launch_tile<GROUP, 16, ZEROS>(p, stream);
  // four accumulators a step with groups of 32: 32 rows are what TMEM holds beside the weights
  if (p.M <= 32 || GROUP == 32) return launch_tile<GROUP, 32, ZEROS>(p, stream);
  return launch_tile<GROUP, GROUP == 32 ? 32 : 64, ZEROS>(p, stream);
}

template <int GROUP>
cudaError_t launch_group(const W4Params &p, cudaStream_t stream) {
  return p.zeros != nullptr ? launch_rows<GROUP, true>(p, stream) : launch_rows<GROUP, false>(p, stream);
}

bool on16(const void *v) { return reinterpret_cast<uintptr_t>(v) % 16 == 0; }

}  // namespace

cudaError_t take_w4_error(int32_t *bits) {
  cudaError_t e = launch_overlapped(k_exchange_w4_error, dim3(1), dim3(1), 0, (cudaStream_t)0);
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(bits, g_w4_error_taken, sizeof(int32_t));
  return e;
}

cudaError_t launch_w4(const W4Params &p, cudaStream_t stream) {
  // 16-byte loads of x and of the weights (a row of weights is a multiple of 16 bytes); the tiled copies'
  // coordinates are 32-bit and their strides below 2^40 bytes; the token tiles go along the grid's y axis.
  constexpr int64_t kMost = INT32_MAX - 1024;
  const bool vectors = on16(p.x) && (p.M == 1 || p.ld_x % 8 == 0) && on16(p.qweight) && p.I > 0 && (p.M + 31) / 32 <= 65535 &&
                       (p.M <= 8 || (p.O <= kMost && p.I <= kMost && p.ld_x < (int64_t(1) << 39)));
  if (vectors) {
    if (p.group == 128) return launch_group<128>(p, stream);
    if (p.group == 64) return launch_group<64>(p, stream);
    return launch_group<32>(p, stream);
  }
  const dim3 grid((unsigned)((p.O + 7) / 8), (unsigned)(p.M < 64 ? p.M : 64));
  return launch_overlapped(k_w4_scalar, grid, dim3(256), 0, stream, p);
}

}  // namespace ccu
