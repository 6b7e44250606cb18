// Products of a few rows with 4-bit weights (ccu_w4_matmul).
//
// The weights are read once and bound the call (0.5 bytes each; every other operand is small), so
// what has to be kept low is the work a weight costs on its way to the multiplier: it is widened
// to BF16 as q - 8, which is exact, in 1.4 instructions, and multiplied on the tensor cores
// (mma.sync m16n8k16: 16 outputs, 8 token rows, 16 inputs) whatever the number of rows up to 8.
// A group's sums stay in 32 bits, are scaled in 32 bits, and added up in 32 bits; zero points other
// than 8 enter as (8 - zero) * (sum of the group's inputs).
#include <atomic>
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
// shared memory, so that few outputs still fill the card. A lane reads the quarter t of a group of
// rows r and r + 8 (16, 8 or 4 bytes each: four lanes cover a row's group), kPre groups ahead of their use.
// (x, scales and zero points as far ahead as the weights: 146 registers instead of 72, 5 rows 16768 x 4096 23.6 us
// against 19.2 on the GPU; x one group ahead in 80 registers: 22.0; scales and zero points alone: 21.9.)
constexpr int kWarps = 8;

template <int GROUP, bool ZEROS>
__global__ void __launch_bounds__(32 * kWarps) k_w4_few(W4Params p) {
  grid_dependency_boundary();
  constexpr int kWords = GROUP / 32;             // 32-bit words a lane and row of a group
  constexpr int kPre = GROUP == 128 ? 2 : 4;
  __shared__ float joined[kWarps][16][9];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, t = lane & 3;
  const int64_t o0 = (int64_t)blockIdx.x * 16;
  const int groups = (int)(p.I / GROUP);
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
    if (g >= groups) return;
    wa[slot].v = __ldcs(&qa[4 * g].v);
    wb[slot].v = __ldcs(&qb[4 * g].v);
  };
#pragma unroll
  for (int i = 0; i < kPre; ++i) fetch(i, warp + i * kWarps);
  for (int g0 = warp; g0 < groups; g0 += kPre * kWarps) {
#pragma unroll
    for (int i = 0; i < kPre; ++i) {
      const int g = g0 + i * kWarps;
      if (g >= groups) break;
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
  if (threadIdx.x < 128) {
    const int o = threadIdx.x & 15, m = threadIdx.x >> 4;
    if (o0 + o < p.O && m < p.M) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += joined[w][o][m];
      static_cast<uint16_t *>(p.out)[m * p.ld_out + o0 + o] = round_bf16(v);
    }
  }
}

// ------------------------------------------------------------------ more token rows
//
// A CTA computes 128 outputs for N token rows on the fifth-generation tensor cores (tcgen05). A step is
// 128 inputs: the threads widen its weights into a 128 x 128 BF16 tile in shared memory and put x beside it (both in
// the order in which a word's nibbles come), one thread issues the products, one accumulator in TMEM for
// every group of the step, and while they run the threads scale and add up the step before.
// (The same tile on mma.sync, weights widened into registers: 64 rows 8192 x 16384 95 us against 85.) The inputs are split
// over the CTAs of a cluster, which join their 32-bit sums through distributed shared memory in rank
// order (the same bits in every run): 8192 outputs are only 64 CTAs otherwise. Waits have a limit.
constexpr int kStep = 128;                       // inputs a step
constexpr int kTileO = 128;                      // outputs a CTA
constexpr int kBlockA = kTileO * 128;            // 64 inputs of the weights' tile

template <int N>
struct Smem {
  static constexpr int kA = 0, kBlockX = N * 128, kX = 4 * kBlockA, kSums = kX + 4 * kBlockX;  // two of each
  static constexpr size_t kBytes = kSums + 3 * 4 * N * sizeof(float) + 1024;
};

template <int GROUP, int N, bool ZEROS>
__global__ void __launch_bounds__(256, 2) k_w4_tile(W4Params p, int split) {
  grid_dependency_boundary();
  constexpr int kGroups = kStep / GROUP, kHalf = N / 2;
  constexpr int kColumns = 2 * kGroups * N < 32 ? 32 : 2 * kGroups * N;   // two steps' accumulators
  constexpr int kPieces = (N * 16 + 255) / 256;  // 16-byte pieces of x a thread and step
  using S = Smem<N>;
  extern __shared__ __align__(16) unsigned char raw[];
  __shared__ uint64_t done[2];
  __shared__ uint32_t tmem_at;
  const uint32_t base = (bulk::smem_addr(raw) + 1023) & ~1023u;
  float *sums = reinterpret_cast<float *>(raw + (base - bulk::smem_addr(raw)) + S::kSums);  // [step % 3][group][N]: a step's are read until the barrier of the next but one
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int quarter = warp & 3, half = warp >> 2;
  const int rank = (int)blockIdx.x % split;      // place in the cluster
  const int64_t o0 = (int64_t)(blockIdx.x / split) * kTileO, m0 = (int64_t)blockIdx.y * N;
  const int groups = (int)(p.I / GROUP), steps = (int)((p.I + kStep - 1) / kStep);
  const int from = (int)((int64_t)steps * rank / split), to = (int)((int64_t)steps * (rank + 1) / split);
  // the row and 64 inputs whose weights this thread widens; the row whose sums it keeps
  const int row = tid >> 1, side = tid & 1, mine = quarter * 32 + lane;
  const int64_t ow = o0 + row < p.O ? o0 + row : p.O - 1, os = o0 + mine < p.O ? o0 + mine : p.O - 1;
  const unsigned char *q = static_cast<const unsigned char *>(p.qweight) + ow * (p.I / 2);
  const uint16_t *scales = static_cast<const uint16_t *>(p.scales) + os * groups;
  const uint16_t *zeros = ZEROS ? static_cast<const uint16_t *>(p.zeros) + os * groups : nullptr;

  if (warp == 0) tensor::tmem_alloc(&tmem_at, kColumns);
  if (tid == 0) {
    bulk::mbar_init(&done[0], 1);
    bulk::mbar_init(&done[1], 1);
    bulk::fence_mbar_init();
  }
  tensor::fence_before_sync();
  __syncthreads();
  tensor::fence_after_sync();
  const uint32_t tmem = tmem_at, sums_at = tmem + ((uint32_t)(quarter * 32) << 16) + half * kHalf;
  uint64_t a_k = tensor::desc_k_major(base + S::kA), x_k = tensor::desc_k_major(base + S::kX);
  asm volatile("" : "+l"(a_k), "+l"(x_k));

  // Piece j (16 bytes, 32 inputs) of this thread's weights: the other way round in every other thread, so that
  // a warp's stores meet all banks.
  uint4 w[2][2], xs[2][kPieces];                 // of the next two steps
  auto fetch = [&](auto buffer, int step) {
    constexpr int kBuffer = decltype(buffer)::value;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t at = (int64_t)step * (kStep / 2) + side * 32 + (j ^ side) * 16;
      w[kBuffer][j] = make_uint4(0, 0, 0, 0);
      if (at < p.I / 2) w[kBuffer][j] = __ldcs(reinterpret_cast<const uint4 *>(q + at));
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int at = tid + i * 256, n = at >> 4;
      const int64_t m = m0 + n, input = (int64_t)step * kStep + 8 * (at & 15);
      xs[kBuffer][i] = make_uint4(0, 0, 0, 0);
      if (n < N && m < p.M && input < p.I)
        xs[kBuffer][i] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.x) + m * p.ld_x + input));
    }
  };
  uint16_t sc[2][kGroups], ze[2][kGroups];       // of the step before and this one
  auto fetch_scales = [&](auto buffer, int step) {
    constexpr int kBuffer = decltype(buffer)::value;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const int at = step * kGroups + g < groups ? step * kGroups + g : groups - 1;
      sc[kBuffer][g] = __ldg(scales + at);
      if (ZEROS) ze[kBuffer][g] = __ldg(zeros + at);
    }
  };
  auto place = [&](auto buffer, int step) {
    constexpr int kBuffer = decltype(buffer)::value;
    const uint32_t at_a = base + S::kA + (2 * kBuffer + side) * kBlockA, at_x = base + S::kX + 2 * kBuffer * S::kBlockX;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint4 v = w[kBuffer][j];
      const uint32_t words[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        tensor::sts128(at_a + tensor::swizzled(row, (j ^ side) * 4 + i),
                       make_uint4(widen_pair<0>(words[i]), widen_pair<1>(words[i]), widen_pair<2>(words[i]), widen_pair<3>(words[i])));
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int at = tid + i * 256, n = at >> 4, c = at & 15;
      const uint4 v = xs[kBuffer][i];
      if (n < N) tensor::sts128(at_x + (c >> 3) * S::kBlockX + tensor::swizzled(n, c & 7), pair_up(v));
      if (ZEROS) {  // a group's sum of x: GROUP / 8 neighbouring threads hold it
        float s = ((bf16_lo(v.x) + bf16_hi(v.x)) + (bf16_lo(v.y) + bf16_hi(v.y))) +
                  ((bf16_lo(v.z) + bf16_hi(v.z)) + (bf16_lo(v.w) + bf16_hi(v.w)));
#pragma unroll
        for (int o = 1; o < GROUP / 8; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (n < N && c % (GROUP / 8) == 0) sums[((step - from) % 3 * 4 + c / (GROUP / 8)) * N + n] = s;
      }
    }
  };
  float total[kHalf];
#pragma unroll
  for (int i = 0; i < kHalf; ++i) total[i] = 0.0f;
  bool fine = true;
  // Scales the accumulators of a step and adds them up.
  auto add_up = [&](auto buffer, int step) {
    constexpr int kBuffer = decltype(buffer)::value;
    fine &= bulk::mbar_wait(&done[kBuffer], ((step - from) >> 1) & 1);
    __syncwarp();
    tensor::fence_after_sync();
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      if (step * kGroups + g >= groups) break;
      const float2 scale = make_float2(bf16_bits(sc[kBuffer][g]), bf16_bits(sc[kBuffer][g]));
      const float shift = ZEROS ? 8.0f - bf16_bits(ze[kBuffer][g]) : 0.0f;
#pragma unroll
      for (int i = 0; i < kHalf; i += 8) {
        float v[8];
        tensor::tmem_load8(sums_at + (kBuffer * kGroups + g) * N + i, v);
        tensor::wait_loads();
        tensor::loaded(v);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          float2 u = make_float2(v[j], v[j + 1]);
          if (ZEROS) {
            const float *s = &sums[((step - from) % 3 * 4 + g) * N + half * kHalf + i + j];
            u = __ffma2_rn(make_float2(shift, shift), make_float2(s[0], s[1]), u);
          }
          const float2 r = __ffma2_rn(scale, u, make_float2(total[i + j], total[i + j + 1]));
          total[i + j] = r.x;
          total[i + j + 1] = r.y;
        }
      }
    }
    tensor::fence_before_sync();
  };
  using Even = std::integral_constant<int, 0>;
  using Odd = std::integral_constant<int, 1>;
  // One step; `buffer` is (step - from) % 2. False: a wait ran out.
  auto advance = [&](auto buffer, auto other, int step) {
    constexpr int kBuffer = decltype(buffer)::value;
    place(buffer, step);  // the products of two steps before are done: their sums have been added up
    bulk::fence_proxy_async();
    tensor::fence_before_sync();
    fine = __syncthreads_and(fine);
    if (!fine) return false;
    if (warp == 0 && tensor::elect_one()) {
      tensor::fence_after_sync();
      const uint64_t a = a_k + kBuffer * 2 * (kBlockA >> 4), x = x_k + kBuffer * 2 * (S::kBlockX >> 4);
#pragma unroll
      for (int k = 0; k < kStep / 16; ++k)
        if (step * kGroups + k * 16 / GROUP < groups)
          tensor::mma_ss(tmem + (kBuffer * kGroups + k * 16 / GROUP) * N, a + (k >> 2) * (kBlockA >> 4) + (k & 3) * 2,
                         x + (k >> 2) * (S::kBlockX >> 4) + (k & 3) * 2, tensor::instruction(128, N, false, false), k * 16 % GROUP != 0);
      tensor::mma_commit(&done[kBuffer]);
    }
    __syncwarp();
    if (step + 2 < to) fetch(buffer, step + 2);
    if (step > from) add_up(other, step - 1);
    if (step + 1 < to) fetch_scales(other, step + 1);
    return true;
  };

  if (from < to) fetch(Even(), from), fetch_scales(Even(), from);
  if (from + 1 < to) fetch(Odd(), from + 1);
  for (int step = from; step < to; step += 2) {
    if (!advance(Even(), Odd(), step)) break;
    if (step + 1 < to && !advance(Odd(), Even(), step + 1)) break;
  }
  if (fine && from < to) {
    if ((to - from) & 1) add_up(Even(), to - 1);
    else add_up(Odd(), to - 1);
  }
  fine = __syncthreads_and(fine);
  if (!fine && tid == 0) atomicOr(&g_w4_error, kDevErrTimeout);
  // Join: every CTA puts its sums into its shared memory and adds up a part of the outputs over all of them.
  constexpr int kRow = N + 1;
  float *joined = reinterpret_cast<float *>(raw);
#pragma unroll
  for (int i = 0; i < kHalf; ++i) joined[mine * kRow + half * kHalf + i] = total[i];
  cluster_sync();
  const int part = kTileO / split;               // outputs a CTA adds up
  for (int i = tid; i < part * N; i += 256) {
    const int o = rank * part + i % part, m = i / part;
    if (o0 + o >= p.O || m0 + m >= p.M) continue;
    float v = 0.0f;
    for (int s = 0; s < split; ++s) v += cluster_load(joined + o * kRow + m, s);
    static_cast<uint16_t *>(p.out)[(m0 + m) * p.ld_out + o0 + o] = round_bf16(v);
  }
  cluster_sync();  // nobody leaves while its sums may be read
  if (warp == 0) {
    tensor::fence_after_sync();
    tensor::tmem_free(tmem, kColumns);
  }
}

template <int GROUP, bool ZEROS>
cudaError_t launch_few(const W4Params &p, cudaStream_t stream) {
  return launch_overlapped(k_w4_few<GROUP, ZEROS>, dim3((unsigned)((p.O + 15) / 16)), dim3(32 * kWarps), 0, stream, p);
}

template <int GROUP, int N, bool ZEROS>
cudaError_t launch_tile(const W4Params &p, cudaStream_t stream) {
  static_assert(2 * kStep / GROUP * N <= 256, "two CTAs' accumulators in an SM's TMEM");
  constexpr size_t kBytes = Smem<N>::kBytes;
  static std::atomic<bool> opted_in[64];
  const int dev = current_device();
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!opted_in[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(k_w4_tile<GROUP, N, ZEROS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kBytes);
    if (e != cudaSuccess) return e;
    opted_in[dev].store(true, std::memory_order_release);
  }
  const int64_t tiles_o = (p.O + kTileO - 1) / kTileO, tiles_m = (p.M + N - 1) / N;
  // Two CTAs an SM fit; the inputs are split until there is one for each place, at least two steps each.
  int split = 1;
  while (split < 8 && tiles_o * tiles_m * split * 2 <= 2 * device_sm_count() && p.I / kStep >= 4 * split) split *= 2;
  return launch_cluster(k_w4_tile<GROUP, N, ZEROS>, dim3((unsigned)(tiles_o * split), (unsigned)tiles_m), dim3(256), kBytes, split, stream,
                        p, split);
}

template <int GROUP, bool ZEROS>
cudaError_t launch_rows(const W4Params &p, cudaStream_t stream) {
  if (p.M <= 8) return launch_few<GROUP, ZEROS>(p, stream);
  if (p.M <= 16) return launch_tile<GROUP, 16, ZEROS>(p, stream);
  // four accumulators a step with groups of 32: 32 rows are what two CTAs' TMEM holds
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
  // 16-byte loads of x and of the weights (a row of weights is a multiple of 16 bytes); the token
  // tiles go along the grid's y axis.
  const bool vectors = on16(p.x) && (p.M == 1 || p.ld_x % 8 == 0) && on16(p.qweight) && (p.M + 31) / 32 <= 65535 && p.I > 0;
  if (vectors) {
    if (p.group == 128) return launch_group<128>(p, stream);
    if (p.group == 64) return launch_group<64>(p, stream);
    return launch_group<32>(p, stream);
  }
  const dim3 grid((unsigned)((p.O + 7) / 8), (unsigned)(p.M < 64 ? p.M : 64));
  return launch_overlapped(k_w4_scalar, grid, dim3(256), 0, stream, p);
}

}  // namespace ccu
