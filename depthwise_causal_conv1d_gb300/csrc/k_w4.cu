// Products of a few rows with 4-bit weights (ccu_w4_matmul).
//
// The weights are read once and bound the call (0.5 bytes each; every other operand is small), so
// what has to be kept low is the work a weight costs on its way to the multiplier: it is widened
// to BF16 as q - 8, which is exact, in 1.4 instructions, and multiplied on the tensor cores
// (mma.sync m16n8k16: 16 outputs, 8 token rows, 16 inputs) whatever the number of rows up to 8.
// A group's sums stay in 32 bits, are scaled in 32 bits, and added up in 32 bits; zero points other
// than 8 enter as (8 - zero) * (sum of the group's inputs).
#include "ssm_internal.cuh"

namespace ccu {

int device_sm_count();

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
// against 19.2 on the GPU; x one group ahead in 80 registers: 22.0.)
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
// A CTA computes 128 outputs (16 a warp) for 8 NT token rows; x goes through shared memory,
// 128 inputs at a time, already in the order the lanes read it, with the groups' sums of x beside it. The
// weights go straight to the lanes that widen them. The inputs are split over the CTAs of a cluster, which
// join their 32-bit sums through distributed shared memory in rank order (the same bits in every run):
// 8192 outputs are only 64 CTAs otherwise.
constexpr int kStep = 128;                       // inputs a step
constexpr int kTileO = 16 * kWarps;

template <int NT>
struct Tile {
  uint4 x[2][8 * NT][16];
  float sums[2][8 * NT][4];
};

// Where the 16-byte piece c (inputs 8c..8c+7 of a step) of a token row stands: the pieces that four lanes of a
// row read together are neighbours, and every other row is turned by half of the eight that span the banks.
template <int GROUP>
__device__ __forceinline__ int piece_at(int row, int c) {
  constexpr int kWords = GROUP / 32;
  const int g = c / (4 * kWords), t = c / kWords % 4, w = c % kWords;
  return (((g * kWords + w) * 4) + t) ^ ((row & 1) << 2);
}

template <int GROUP, int NT, bool ZEROS>
__global__ void __launch_bounds__(32 * kWarps, 2) k_w4_tile(W4Params p, int split) {
  grid_dependency_boundary();
  constexpr int kWords = GROUP / 32, kGroups = kStep / GROUP;
  constexpr int kPieces = 8 * NT * 16 / (32 * kWarps);  // pieces of x a thread and step
  extern __shared__ __align__(16) unsigned char raw[];
  Tile<NT> &tile = *reinterpret_cast<Tile<NT> *>(raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, t = lane & 3;
  const int rank = (int)blockIdx.x % split;      // place in the cluster
  const int64_t o0 = (int64_t)(blockIdx.x / split) * kTileO, ow = o0 + 16 * warp, m0 = (int64_t)blockIdx.y * 8 * NT;
  const int groups = (int)(p.I / GROUP), steps = (int)((p.I + kStep - 1) / kStep);
  const int from = (int)((int64_t)steps * rank / split), to = (int)((int64_t)steps * (rank + 1) / split);
  const int64_t oa = ow + r < p.O ? ow + r : p.O - 1, ob = ow + r + 8 < p.O ? ow + r + 8 : p.O - 1;
  using Vec = Words<GROUP>;
  const Vec *qa = reinterpret_cast<const Vec *>(static_cast<const uint32_t *>(p.qweight) + oa * (p.I / 8)) + t;
  const Vec *qb = reinterpret_cast<const Vec *>(static_cast<const uint32_t *>(p.qweight) + ob * (p.I / 8)) + t;
  const uint16_t *scales = static_cast<const uint16_t *>(p.scales), *zeros = static_cast<const uint16_t *>(p.zeros);
  const Rows rows = {scales + oa * groups, scales + ob * groups, ZEROS ? zeros + oa * groups : nullptr, ZEROS ? zeros + ob * groups : nullptr};
  Vec wa[kGroups], wb[kGroups];
  uint16_t sa[kGroups], sb[kGroups], za[kGroups], zb[kGroups];
  uint4 xs[kPieces];
  auto fetch = [&](int step) {
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const int g = step * kGroups + i;
      if (g >= groups) break;
      wa[i].v = __ldcs(&qa[4 * g].v);
      wb[i].v = __ldcs(&qb[4 * g].v);
      sa[i] = __ldg(rows.sa + g);
      sb[i] = __ldg(rows.sb + g);
      if (ZEROS) za[i] = __ldg(rows.za + g), zb[i] = __ldg(rows.zb + g);
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int at = tid + i * 32 * kWarps, row = at >> 4, c = at & 15;
      const int64_t m = m0 + row, input = (int64_t)step * kStep + 8 * c;
      xs[i] = make_uint4(0, 0, 0, 0);
      if (m < p.M && input < p.I) xs[i] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.x) + m * p.ld_x + input));
    }
  };
  auto place = [&](int buffer) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int at = tid + i * 32 * kWarps, row = at >> 4, c = at & 15;
      tile.x[buffer][row][piece_at<GROUP>(row, c)] = pair_up(xs[i]);
      if (ZEROS) {  // a group's sum of x: GROUP / 8 neighbouring threads hold it
        float s = ((bf16_lo(xs[i].x) + bf16_hi(xs[i].x)) + (bf16_lo(xs[i].y) + bf16_hi(xs[i].y))) +
                  ((bf16_lo(xs[i].z) + bf16_hi(xs[i].z)) + (bf16_lo(xs[i].w) + bf16_hi(xs[i].w)));
#pragma unroll
        for (int o = 1; o < GROUP / 8; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (c % (GROUP / 8) == 0) tile.sums[buffer][row][c / (GROUP / 8)] = s;
      }
    }
  };
  float total[NT][4] = {};
  if (from < to) {
    fetch(from);
    place(0);
  }
  for (int step = from; step < to; ++step) {
    const int buffer = (step - from) & 1;
    Vec va[kGroups], vb[kGroups];
    float fa[kGroups], fb[kGroups], ca[kGroups], cb[kGroups];
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      va[i] = wa[i];
      vb[i] = wb[i];
      fa[i] = bf16_bits(sa[i]);
      fb[i] = bf16_bits(sb[i]);
      if (ZEROS) ca[i] = 8.0f - bf16_bits(za[i]), cb[i] = 8.0f - bf16_bits(zb[i]);
    }
    __syncthreads();  // this step's x is in place, and the other buffer has been read
    if (step + 1 < to) fetch(step + 1);
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      if (step * kGroups + i >= groups) break;
      float acc[NT][4] = {};
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        const uint32_t u = va[i].get(w), v = vb[i].get(w);
        const uint32_t a0[4] = {widen_pair<0>(u), widen_pair<0>(v), widen_pair<1>(u), widen_pair<1>(v)};
        const uint32_t a1[4] = {widen_pair<2>(u), widen_pair<2>(v), widen_pair<3>(u), widen_pair<3>(v)};
        constexpr int kAtOnce = NT < 4 ? NT : 4;  // independent products between the two on one accumulator
#pragma unroll
        for (int n0 = 0; n0 < NT; n0 += kAtOnce) {
          uint4 e[kAtOnce];
#pragma unroll
          for (int n = 0; n < kAtOnce; ++n) e[n] = tile.x[buffer][8 * (n0 + n) + r][(((i * kWords + w) * 4) + t) ^ ((r & 1) << 2)];
#pragma unroll
          for (int n = 0; n < kAtOnce; ++n) mma16816(acc[n0 + n], a0, e[n].x, e[n].y);
#pragma unroll
          for (int n = 0; n < kAtOnce; ++n) mma16816(acc[n0 + n], a1, e[n].z, e[n].w);
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float v = acc[n][j];
          if (ZEROS) v = fmaf(j < 2 ? ca[i] : cb[i], tile.sums[buffer][8 * n + 2 * t + (j & 1)][i], v);
          total[n][j] = fmaf(j < 2 ? fa[i] : fb[i], v, total[n][j]);
        }
    }
    if (step + 1 < to) place(buffer ^ 1);
  }
  // Join: every CTA puts its sums into its shared memory and adds up a part of the outputs over all of them.
  __syncthreads();
  constexpr int kRow = 8 * NT + 1;
  float *mine = reinterpret_cast<float *>(raw);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) mine[(16 * warp + r + (j >> 1) * 8) * kRow + 8 * n + 2 * t + (j & 1)] = total[n][j];
  cluster_sync();
  const int part = kTileO / split;               // outputs a CTA adds up
  for (int i = tid; i < part * 8 * NT; i += 32 * kWarps) {
    const int o = rank * part + i % part, m = i / part;
    if (o0 + o >= p.O || m0 + m >= p.M) continue;
    float v = 0.0f;
    for (int s = 0; s < split; ++s) v += cluster_load(mine + o * kRow + m, s);
    static_cast<uint16_t *>(p.out)[(m0 + m) * p.ld_out + o0 + o] = round_bf16(v);
  }
  cluster_sync();  // nobody leaves while its sums may be read
}

template <int GROUP, bool ZEROS>
cudaError_t launch_few(const W4Params &p, cudaStream_t stream) {
  return launch_overlapped(k_w4_few<GROUP, ZEROS>, dim3((unsigned)((p.O + 15) / 16)), dim3(32 * kWarps), 0, stream, p);
}

template <int GROUP, int NT, bool ZEROS>
cudaError_t launch_tile(const W4Params &p, cudaStream_t stream) {
  constexpr size_t kSums = sizeof(float) * kTileO * (8 * NT + 1), kBytes = sizeof(Tile<NT>) > kSums ? sizeof(Tile<NT>) : kSums;
  static_assert(kBytes <= 48 * 1024, "no opt-in needed");
  const int64_t tiles_o = (p.O + kTileO - 1) / kTileO, tiles_m = (p.M + 8 * NT - 1) / (8 * NT);
  // Two CTAs an SM fit; the inputs are split until there is one for each place, at least two steps each.
  int split = 1;
  while (split < 8 && tiles_o * tiles_m * split * 2 <= 2 * device_sm_count() && p.I / kStep >= 4 * split) split *= 2;
  return launch_cluster(k_w4_tile<GROUP, NT, ZEROS>, dim3((unsigned)(tiles_o * split), (unsigned)tiles_m), dim3(32 * kWarps), kBytes,
                        split, stream, p, split);
}

template <int GROUP, bool ZEROS>
cudaError_t launch_rows(const W4Params &p, cudaStream_t stream) {
  if (p.M <= 8) return launch_few<GROUP, ZEROS>(p, stream);
  if (p.M <= 16) return launch_tile<GROUP, 2, ZEROS>(p, stream);
  if (p.M <= 32) return launch_tile<GROUP, 4, ZEROS>(p, stream);
  return launch_tile<GROUP, 8, ZEROS>(p, stream);
}

template <int GROUP>
cudaError_t launch_group(const W4Params &p, cudaStream_t stream) {
  return p.zeros != nullptr ? launch_rows<GROUP, true>(p, stream) : launch_rows<GROUP, false>(p, stream);
}

bool on16(const void *v) { return reinterpret_cast<uintptr_t>(v) % 16 == 0; }

}  // namespace

cudaError_t launch_w4(const W4Params &p, cudaStream_t stream) {
  // 16-byte loads of x and of the weights (a row of weights is a multiple of 16 bytes); the token
  // tiles go along the grid's y axis.
  const bool vectors = on16(p.x) && (p.M == 1 || p.ld_x % 8 == 0) && on16(p.qweight) && (p.M + 63) / 64 <= 65535 && p.I > 0;
  if (vectors) {
    if (p.group == 128) return launch_group<128>(p, stream);
    if (p.group == 64) return launch_group<64>(p, stream);
    return launch_group<32>(p, stream);
  }
  const dim3 grid((unsigned)((p.O + 7) / 8), (unsigned)(p.M < 64 ? p.M : 64));
  return launch_overlapped(k_w4_scalar, grid, dim3(256), 0, stream, p);
}

}  // namespace ccu
