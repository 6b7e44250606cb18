// Products of a few rows with 4-bit weights (ccu_w4_matmul).
//
// The weights are read once and bound the call (0.5 bytes each; every other operand is small), so
// what has to be kept low is the work a weight costs on its way to the multiplier: it is widened
// to BF16 as q - 8, which is exact, in 1.4 instructions, and multiplied on the tensor cores
// (mma.sync m16n8k16: 16 outputs, 8 token rows, 16 inputs) whatever the number of rows up to 8.
// A group's sums stay in 32 bits, are scaled in 32 bits, and added up in 32 bits; zero points other
// than 8 enter as (8 - zero) * (sum of the group's inputs), which a product with a matrix of
// ones gives in the same lanes.
#include "ssm_internal.cuh"

namespace ccu {

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

// A CTA computes 16 outputs for 8 NT token rows; its 8 warps take the groups of inputs in
// turn and join their sums in shared memory, so that few outputs still fill the card. A lane reads the
// quarter t of a group of rows r and r + 8 (16, 8 or 4 bytes each: four lanes cover a row's group),
// PRE groups ahead of their use.
constexpr int kWarps = 8;

template <int GROUP, int NT, bool ZEROS>
__global__ void __launch_bounds__(32 * kWarps) k_w4_mma(W4Params p) {
  grid_dependency_boundary();
  constexpr int kWords = GROUP / 32;             // 32-bit words a lane and row of a group
  constexpr int kPre = GROUP == 128 ? 2 : 4;
  __shared__ float joined[kWarps][16][8 * NT + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, t = lane & 3;
  const int64_t o0 = (int64_t)blockIdx.x * 16, m0 = (int64_t)blockIdx.y * 8 * NT;
  const int groups = (int)(p.I / GROUP);
  const int64_t oa = o0 + r < p.O ? o0 + r : p.O - 1, ob = o0 + r + 8 < p.O ? o0 + r + 8 : p.O - 1;
  using Vec = Words<GROUP>;
  const Vec *qa = reinterpret_cast<const Vec *>(static_cast<const uint32_t *>(p.qweight) + oa * (p.I / 8)) + t;
  const Vec *qb = reinterpret_cast<const Vec *>(static_cast<const uint32_t *>(p.qweight) + ob * (p.I / 8)) + t;
  const uint16_t *sa = static_cast<const uint16_t *>(p.scales) + oa * groups, *sb = static_cast<const uint16_t *>(p.scales) + ob * groups;
  const uint16_t *za = nullptr, *zb = nullptr;
  if (ZEROS) za = static_cast<const uint16_t *>(p.zeros) + oa * groups, zb = static_cast<const uint16_t *>(p.zeros) + ob * groups;
  const uint16_t *x[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int64_t m = m0 + 8 * n + r;
    x[n] = m < p.M ? static_cast<const uint16_t *>(p.x) + m * p.ld_x + t * (GROUP / 4) : nullptr;
  }
  float total[NT][4] = {};
  Vec wa[kPre], wb[kPre];
  auto fetch = [&](int slot, int g) {
    if (g < groups) {
      wa[slot].v = __ldcs(&qa[4 * g].v);
      wb[slot].v = __ldcs(&qb[4 * g].v);
    }
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
      const float fa = bf16_bits(__ldg(sa + g)), fb = bf16_bits(__ldg(sb + g));
      float acc[NT][4] = {}, sums[NT][4] = {};
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        const uint32_t u = va.get(w), v = vb.get(w);
        const uint32_t a0[4] = {widen_pair<0>(u), widen_pair<0>(v), widen_pair<1>(u), widen_pair<1>(v)};
        const uint32_t a1[4] = {widen_pair<2>(u), widen_pair<2>(v), widen_pair<3>(u), widen_pair<3>(v)};
        const uint32_t ones[4] = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          uint4 e = make_uint4(0, 0, 0, 0);  // eight inputs of a token row
          if (x[n] != nullptr) e = __ldg(reinterpret_cast<const uint4 *>(x[n] + (int64_t)g * GROUP + 8 * w));
          // the pairs (0,4) (1,5) (2,6) (3,7) that the nibbles come in
          const uint32_t b0 = __byte_perm(e.x, e.z, 0x5410), b1 = __byte_perm(e.x, e.z, 0x7632);
          const uint32_t b2 = __byte_perm(e.y, e.w, 0x5410), b3 = __byte_perm(e.y, e.w, 0x7632);
          mma16816(acc[n], a0, b0, b1);
          mma16816(acc[n], a1, b2, b3);
          if (ZEROS) {
            mma16816(sums[n], ones, b0, b1);
            mma16816(sums[n], ones, b2, b3);
          }
        }
      }
      float ca = 0.0f, cb = 0.0f;
      if (ZEROS) ca = 8.0f - bf16_bits(__ldg(za + g)), cb = 8.0f - bf16_bits(__ldg(zb + g));
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float v = ZEROS ? fmaf(j < 2 ? ca : cb, sums[n][j], acc[n][j]) : acc[n][j];
          total[n][j] = fmaf(j < 2 ? fa : fb, v, total[n][j]);
        }
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) joined[warp][r + (j >> 1) * 8][8 * n + 2 * t + (j & 1)] = total[n][j];
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * 8 * NT; i += 32 * kWarps) {
    const int o = i & 15, m = i >> 4;
    if (o0 + o >= p.O || m0 + m >= p.M) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += joined[w][o][m];
    static_cast<uint16_t *>(p.out)[(m0 + m) * p.ld_out + o0 + o] = round_bf16(v);
  }
}

template <int GROUP, int NT>
cudaError_t launch_nt(const W4Params &p, cudaStream_t stream) {
  const int64_t tiles = (p.M + 8 * NT - 1) / (8 * NT);
  const dim3 grid((unsigned)((p.O + 15) / 16), (unsigned)tiles);
  return p.zeros != nullptr ? launch_overlapped(k_w4_mma<GROUP, NT, true>, grid, dim3(32 * kWarps), 0, stream, p)
                            : launch_overlapped(k_w4_mma<GROUP, NT, false>, grid, dim3(32 * kWarps), 0, stream, p);
}

template <int GROUP>
cudaError_t launch_group(const W4Params &p, cudaStream_t stream) {
  if (p.M <= 8) return launch_nt<GROUP, 1>(p, stream);
  if (p.M <= 16) return launch_nt<GROUP, 2>(p, stream);
  return launch_nt<GROUP, 4>(p, stream);
}

bool on16(const void *v) { return reinterpret_cast<uintptr_t>(v) % 16 == 0; }

}  // namespace

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
