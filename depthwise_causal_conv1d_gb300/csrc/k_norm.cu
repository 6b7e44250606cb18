// Norms around a layer (ccu_gated_rms_norm, ccu_residual_rms_norm).
//
// A row is read once: a team of threads (a part of a warp, warps, or a whole CTA) holds it in registers, V accesses of E
// entries a thread, sums its squares in 32 bits and writes the results. Bound by HBM where there are many rows, by a launch and one
// or two sums over the team where there are few. Gated: 32768 tokens x 32 heads x 128 127.9 us, 6.3 TB/s; 2377 x 8 x 1024 23.3 us, 5.0 TB/s;
// one token of 16 heads 1.8 us. Residual: 32768 rows of 4096 in FP32 with both norms 249 us, 6.5 TB/s; 64 rows of 16384 in BF16 3.8 us.
//
// E is what the boundaries of rows allow (8: 16-byte accesses; 2; 1), V the fewest accesses with which up to
// 1024 threads hold the row. Rows that are longer than that go through a kernel that reads them again for every pass.
#include <atomic>

#include "ssm_internal.cuh"

namespace ccu {

int current_device();
int device_sm_count();

namespace {

constexpr int kBlock = 256;     // threads of a CTA whose teams are smaller

// E entries of a BF16 tensor, as they are in memory; FP32 tensors are two of them.
template <int E>
struct Raw {
  uint32_t e[E == 1 ? 1 : E / 2];
};
template <int E>
__device__ __forceinline__ Raw<E> nothing() {
  Raw<E> r;
#pragma unroll
  for (int i = 0; i < (E == 1 ? 1 : E / 2); ++i) r.e[i] = 0;
  return r;
}
template <int E>
__device__ __forceinline__ Raw<E> read16(const uint16_t *p) {
  Raw<E> r;
  if constexpr (E == 8) {
    const uint4 w = ld_stream(p);
    r.e[0] = w.x, r.e[1] = w.y, r.e[2] = w.z, r.e[3] = w.w;
  } else if constexpr (E == 2) {
    r.e[0] = __ldcs(reinterpret_cast<const uint32_t *>(p));
  } else {
    r.e[0] = __ldcs(p);
  }
  return r;
}
// Entries in pairs (one of E = 1 in the first place of a pair whose second is zero): the instructions on two floats halve the count.
template <int E>
struct Pairs {
  static constexpr int N = E == 1 ? 1 : E / 2;
  float2 v[N];
};
template <int E>
__device__ __forceinline__ Pairs<E> widen(const Raw<E> &r) {
  Pairs<E> p;
  if constexpr (E == 1) {
    p.v[0] = make_float2(bf16_bits(r.e[0]), 0.0f);
  } else {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) p.v[i] = make_float2(bf16_lo(r.e[i]), bf16_hi(r.e[i]));
  }
  return p;
}
template <int E>
__device__ __forceinline__ Pairs<E> read32(const float *p) {
  Pairs<E> r;
  if constexpr (E == 8) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 w = __ldcs(reinterpret_cast<const float4 *>(p) + i);
      r.v[2 * i] = make_float2(w.x, w.y), r.v[2 * i + 1] = make_float2(w.z, w.w);
    }
  } else if constexpr (E == 2) {
    r.v[0] = __ldcs(reinterpret_cast<const float2 *>(p));
  } else {
    r.v[0] = make_float2(__ldcs(p), 0.0f);
  }
  return r;
}
template <int E>
__device__ __forceinline__ void write16(uint16_t *p, const Pairs<E> &r) {
  if constexpr (E == 8)
    st_stream(p, make_uint4(pack_bf16x2(r.v[0].x, r.v[0].y), pack_bf16x2(r.v[1].x, r.v[1].y), pack_bf16x2(r.v[2].x, r.v[2].y), pack_bf16x2(r.v[3].x, r.v[3].y)));
  else if constexpr (E == 2)
    __stcs(reinterpret_cast<uint32_t *>(p), pack_bf16x2(r.v[0].x, r.v[0].y));
  else
    __stcs(p, round_bf16(r.v[0].x));
}
template <int E>
__device__ __forceinline__ void write32(float *p, const Pairs<E> &r) {
  if constexpr (E == 8) {
    __stcs(reinterpret_cast<float4 *>(p), make_float4(r.v[0].x, r.v[0].y, r.v[1].x, r.v[1].y));
    __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(r.v[2].x, r.v[2].y, r.v[3].x, r.v[3].y));
  } else if constexpr (E == 2) {
    __stcs(reinterpret_cast<float2 *>(p), r.v[0]);
  } else {
    __stcs(p, r.v[0].x);
  }
}
// Weights are on any boundary of their type, and shared by many rows: cached reads, one by one where vectors do not fit.
template <int E>
__device__ __forceinline__ Pairs<E> read_weight(const void *w, int type, int64_t at) {
  Pairs<E> r;
  float *v = &r.v[0].x;
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = 1.0f;
  } else if (type == CCU_DTYPE_BF16) {
    const uint16_t *p = static_cast<const uint16_t *>(w) + at;
    if (E == 8 && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
      const uint4 u = ld_keep(p);
      const uint32_t e[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = i & 1 ? bf16_hi(e[(i / 2) % 4]) : bf16_lo(e[(i / 2) % 4]);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = bf16_bits(__ldg(p + i));
    }
  } else {
    const float *p = static_cast<const float *>(w) + at;
    if (E == 8 && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
      const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
      const float u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = u[i % 8];
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = __ldg(p + i);
    }
  }
  if (E == 1) r.v[0].y = 0.0f;
  return r;
}
template <int E>
__device__ __forceinline__ void times(Pairs<E> &a, const Pairs<E> &b) {
#pragma unroll
  for (int i = 0; i < Pairs<E>::N; ++i) a.v[i] = __fmul2_rn(a.v[i], b.v[i]);
}
template <int E>
__device__ __forceinline__ void times(Pairs<E> &a, float b) {
#pragma unroll
  for (int i = 0; i < Pairs<E>::N; ++i) a.v[i] = __fmul2_rn(a.v[i], make_float2(b, b));
}
template <int E>
__device__ __forceinline__ void add_squares(const Pairs<E> &a, float2 &sum) {
#pragma unroll
  for (int i = 0; i < Pairs<E>::N; ++i) sum = __ffma2_rn(a.v[i], a.v[i], sum);
}
// z sigmoid(z).
template <int E>
__device__ __forceinline__ void gates(Pairs<E> &a) {
#pragma unroll
  for (int i = 0; i < Pairs<E>::N; ++i) a.v[i] = activate2<1>(a.v[i]);
}

// Sum over a team of `team` threads (a power of two; a CTA's teams are all in step). `part`: 32 floats of shared memory
// for every sum of a kernel.
__device__ __forceinline__ float team_sum(float v, int team, float *part) {
  for (int o = (team < 32 ? team : 32) >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (team > 32) {
    const int warp = threadIdx.x >> 5, warps = team >> 5, first = warp & ~(warps - 1);
    if ((threadIdx.x & 31) == 0) part[warp] = v;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    v = lane < warps ? part[first + lane] : 0.0f;
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  }
  return v;
}

// Reciprocal of the root mean square of `n` entries whose squares add up to `squares`.
__device__ __forceinline__ float inverse_rms(float squares, int64_t n, float eps) { return rsqrtf(squares / (float)n + eps); }

// The gated norm. A CTA goes through the rows in turns of as many as it has teams; a turn's rows are loaded one turn ahead (AHEAD), so
// that a team's sum runs under the next row's loads.
template <int E, int V, int BLOCK>
__global__ void __launch_bounds__(BLOCK) k_gated_norm(GatedNormParams p, int team) {
  grid_dependency_boundary();
  constexpr bool AHEAD = V <= 2;
  __shared__ float part[2][32];
  const int per = blockDim.x / team, of = threadIdx.x / team, rank = threadIdx.x - of * team;
  const int64_t rows = p.T * p.H, step = (int64_t)gridDim.x * per;  // below 2^31, as T * H is, and 2^31
  const uint16_t *x = static_cast<const uint16_t *>(p.x), *z = static_cast<const uint16_t *>(p.z);
  Raw<E> rx[V], rz[V];
  uint32_t t_next = 0, h_next = 0;
  auto fetch = [&](int64_t r) {
    const bool live = r < rows;
    t_next = live ? (uint32_t)r / (uint32_t)p.H : 0;
    h_next = live ? (uint32_t)r - t_next * (uint32_t)p.H : 0;
    const int64_t t = t_next, h = h_next;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int64_t at = (int64_t)E * (rank + j * team);
      const bool in = live && at < p.P;
      rx[j] = in ? read16<E>(x + t * p.x_stride_t + h * p.x_stride_h + at) : nothing<E>();
      rz[j] = in && z != nullptr ? read16<E>(z + t * p.z_stride_t + h * p.z_stride_h + at) : nothing<E>();
    }
  };
  int64_t base = (int64_t)blockIdx.x * per;
  if (AHEAD) fetch(base + of);
  for (int turn = 0; base < rows; base += step, turn ^= 1) {
    const int64_t r = base + of;
    const bool live = r < rows;
    if (!AHEAD) fetch(r);
    const int64_t t = t_next, h = h_next;
    Pairs<E> v[V], gate[V];
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = widen<E>(rx[j]), gate[j] = widen<E>(rz[j]);
    if (AHEAD) fetch(r + step);
    float2 squares = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (z != nullptr) gates<E>(gate[j]);
      if (p.gate_first && z != nullptr) times<E>(v[j], gate[j]);
      add_squares<E>(v[j], squares);
    }
    const float scale = inverse_rms(team_sum(squares.x + squares.y, team, part[turn]), p.P, p.eps);
    uint16_t *out = static_cast<uint16_t *>(p.out) + t * p.out_stride_t + h * p.out_stride_h;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int64_t at = (int64_t)E * (rank + j * team);
      if (!live || at >= p.P) continue;
      const Pairs<E> w = read_weight<E>(p.weight, p.weight_type, h * p.weight_stride_h + at);
      times<E>(v[j], scale);
      times<E>(v[j], w);
      if (!p.gate_first && z != nullptr) times<E>(v[j], gate[j]);
      write16<E>(out + at, v[j]);
    }
  }
}

// The residual norm, in the same way. Registers for three of the smaller CTAs an SM: 32768 rows of 4096 in FP32 249 us, with the
// two CTAs that fit by themselves 280, with four, which spill, 352.
template <int E, int V, bool WIDE, int BLOCK>
__global__ void __launch_bounds__(BLOCK, BLOCK == kBlock ? 3 : 1) k_residual_norm(ResidualNormParams p, int team) {
  grid_dependency_boundary();
  constexpr bool AHEAD = V <= (BLOCK == 1024 ? 1 : 2);
  __shared__ float part[3][32];
  const int per = blockDim.x / team, of = threadIdx.x / team, rank = threadIdx.x - of * team;
  const int64_t step = (int64_t)gridDim.x * per;
  const uint16_t *x = static_cast<const uint16_t *>(p.x);
  uint16_t *r16 = static_cast<uint16_t *>(p.residual);
  float *r32 = static_cast<float *>(p.residual);
  Raw<E> rx[V], rr[V];
  Pairs<E> wide[V];
  auto fetch = [&](int64_t t) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int64_t at = (int64_t)E * (rank + j * team);
      const bool in = t < p.T && at < p.D;
      rx[j] = in ? read16<E>(x + t * p.ld_x + at) : nothing<E>();
      if constexpr (WIDE) {
        wide[j] = widen<E>(nothing<E>());
        if (in) wide[j] = read32<E>(r32 + t * p.ld_residual + at);
      } else {
        rr[j] = in ? read16<E>(r16 + t * p.ld_residual + at) : nothing<E>();
      }
    }
  };
  int64_t base = (int64_t)blockIdx.x * per;
  if (AHEAD) fetch(base + of);
  for (int turn = 0; base < p.T; base += step, turn ^= 1) {
    const int64_t t = base + of;
    const bool live = t < p.T;
    if (!AHEAD) fetch(t);
    Pairs<E> v[V], r[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      v[j] = widen<E>(rx[j]);
      if constexpr (WIDE) r[j] = wide[j];
      else r[j] = widen<E>(rr[j]);
    }
    if (AHEAD) fetch(t + step);
    if (p.post_weight != nullptr) {
      float2 squares = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int j = 0; j < V; ++j) add_squares<E>(v[j], squares);
      const float scale = inverse_rms(team_sum(squares.x + squares.y, team, part[2]), p.D, p.eps);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int64_t at = (int64_t)E * (rank + j * team);
        if (!live || at >= p.D) continue;
        times<E>(v[j], scale);
        times<E>(v[j], read_weight<E>(p.post_weight, p.weight_type, at));
      }
    }
    float2 squares = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int64_t at = (int64_t)E * (rank + j * team);
      if (!live || at >= p.D) continue;
#pragma unroll
      for (int i = 0; i < Pairs<E>::N; ++i) r[j].v[i] = __ffma2_rn(make_float2(p.scale, p.scale), v[j].v[i], r[j].v[i]);
      add_squares<E>(r[j], squares);
      if constexpr (WIDE) write32<E>(r32 + t * p.ld_residual + at, r[j]);
      else write16<E>(r16 + t * p.ld_residual + at, r[j]);
    }
    const float scale = inverse_rms(team_sum(squares.x + squares.y, team, part[turn]), p.D, p.eps);
    uint16_t *out = static_cast<uint16_t *>(p.out) + t * p.ld_out;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int64_t at = (int64_t)E * (rank + j * team);
      if (!live || at >= p.D) continue;
      times<E>(r[j], scale);
      times<E>(r[j], read_weight<E>(p.weight, p.weight_type, at));
      write16<E>(out + at, r[j]);
    }
  }
}

// Rows of any length, a CTA each: read again for every pass, entry by entry. The residual's second pass forms the sum again
// from the old residual, and stores it.
__global__ void __launch_bounds__(1024) k_gated_norm_long(GatedNormParams p) {
  grid_dependency_boundary();
  __shared__ float part[32];
  const int64_t t = blockIdx.x / (uint64_t)p.H, h = blockIdx.x - t * p.H;
  const uint16_t *x = static_cast<const uint16_t *>(p.x) + t * p.x_stride_t + h * p.x_stride_h;
  const uint16_t *z = static_cast<const uint16_t *>(p.z) + t * p.z_stride_t + h * p.z_stride_h;
  uint16_t *out = static_cast<uint16_t *>(p.out) + t * p.out_stride_t + h * p.out_stride_h;
  float squares = 0.0f;
  for (int64_t i = threadIdx.x; i < p.P; i += blockDim.x) {
    float v = bf16_bits(x[i]);
    if (p.gate_first && p.z != nullptr) v *= activate<1>(bf16_bits(z[i]));
    squares = fmaf(v, v, squares);
  }
  const float scale = inverse_rms(team_sum(squares, blockDim.x, part), p.P, p.eps);
  for (int64_t i = threadIdx.x; i < p.P; i += blockDim.x) {
    const float gate = p.z != nullptr ? activate<1>(bf16_bits(z[i])) : 1.0f;
    const float w = read_weight<1>(p.weight, p.weight_type, h * p.weight_stride_h + i).v[0].x;
    float v = bf16_bits(x[i]);
    if (p.gate_first) v *= gate;
    v = v * scale * w;
    if (!p.gate_first) v *= gate;
    out[i] = round_bf16(v);
  }
}

__global__ void __launch_bounds__(1024) k_residual_norm_long(ResidualNormParams p) {
  grid_dependency_boundary();
  __shared__ float part[64];
  const int64_t t = blockIdx.x;
  const bool wide = p.residual_type == CCU_DTYPE_FP32, post = p.post_weight != nullptr;
  const uint16_t *x = static_cast<const uint16_t *>(p.x) + t * p.ld_x;
  uint16_t *r16 = static_cast<uint16_t *>(p.residual) + t * p.ld_residual, *out = static_cast<uint16_t *>(p.out) + t * p.ld_out;
  float *r32 = static_cast<float *>(p.residual) + t * p.ld_residual;
  float first = 1.0f, squares = 0.0f;
  if (post) {
    for (int64_t i = threadIdx.x; i < p.D; i += blockDim.x) {
      const float v = bf16_bits(x[i]);
      squares = fmaf(v, v, squares);
    }
    first = inverse_rms(team_sum(squares, blockDim.x, part), p.D, p.eps);
  }
  auto sum = [&](int64_t i) {  // not contracted differently in the two passes
    const float y = post ? bf16_bits(x[i]) * first * read_weight<1>(p.post_weight, p.weight_type, i).v[0].x : bf16_bits(x[i]);
    return fmaf(p.scale, y, wide ? r32[i] : bf16_bits(r16[i]));
  };
  squares = 0.0f;
  for (int64_t i = threadIdx.x; i < p.D; i += blockDim.x) {
    const float v = sum(i);
    squares = fmaf(v, v, squares);
  }
  const float scale = inverse_rms(team_sum(squares, blockDim.x, part + 32), p.D, p.eps);
  for (int64_t i = threadIdx.x; i < p.D; i += blockDim.x) {
    const float v = sum(i);
    const float w = read_weight<1>(p.weight, p.weight_type, i).v[0].x;
    if (wide) r32[i] = v;
    else r16[i] = round_bf16(v);
    out[i] = round_bf16(v * scale * w);
  }
}

bool multiples(int64_t e, std::initializer_list<int64_t> strides, std::initializer_list<const void *> bases16, const void *base32) {
  for (int64_t s : strides)
    if (s % e != 0) return false;
  for (const void *b : bases16)
    if (reinterpret_cast<uintptr_t>(b) % (2 * e) != 0) return false;
  return reinterpret_cast<uintptr_t>(base32) % (e == 8 ? 16 : 4 * e) == 0;
}

// How a row of n entries is spread: accesses a thread, threads a team and a CTA. One access a thread where there are few rows, so that
// many threads share a row; two where there are rows for all of them, so that a sum over the team serves twice the entries (gated, 2^20 rows of
// 128 152 us with one and 130 with two, 19016 rows of 1024 27 and 24; residual, 32768 rows of 4096 in FP32 274 and 249);
// more where 1024 threads need them.
struct Spread {
  int v, team, block;
};
Spread spread_of(int64_t n, int e, int64_t rows) {
  const int64_t pieces = (n + e - 1) / e;
  int v = pieces > 4 && rows * pieces >= (int64_t)device_sm_count() * 2048 ? 2 : 1;
  while (v < 8 && pieces > 1024 * (int64_t)v) v *= 2;
  int team = 1;
  while (team < 1024 && (int64_t)team * v < pieces) team *= 2;
  return {(int64_t)team * v < pieces ? 0 : v, team, team > kBlock ? team : kBlock};
}

// CTAs for so many rows: no more than the device holds at once, which then go through the rows in turns.
template <auto KERNEL>
unsigned ctas_for(const Spread &s, int64_t rows) {
  static std::atomic<int> held[64][4];  // CTAs an SM, by device and by threads a CTA (256, 512, 1024)
  const int per = s.block / s.team, dev = current_device();
  const int64_t need = (rows + per - 1) / per, sms = device_sm_count();
  if (need <= sms * (1024 / s.block) || dev < 0 || dev >= 64) return (unsigned)need;
  std::atomic<int> &slot = held[dev][s.block / 512];
  int each = slot.load(std::memory_order_relaxed);
  if (each == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&each, KERNEL, s.block, 0) != cudaSuccess || each < 1) {
      (void)cudaGetLastError();
      each = 1;
    }
    slot.store(each, std::memory_order_relaxed);
  }
  return (unsigned)(need < sms * each ? need : sms * each);
}

template <int E, int V>
cudaError_t launch_gated_v(const GatedNormParams &p, const Spread &s, cudaStream_t stream) {
  if constexpr (V <= 2) {  // more only with 1024 threads
    if (s.block <= kBlock)
      return launch_overlapped(k_gated_norm<E, V, kBlock>, dim3(ctas_for<k_gated_norm<E, V, kBlock>>(s, p.T * p.H)), dim3(s.block), 0, stream, p, s.team);
  }
  return launch_overlapped(k_gated_norm<E, V, 1024>, dim3(ctas_for<k_gated_norm<E, V, 1024>>(s, p.T * p.H)), dim3(s.block), 0, stream, p, s.team);
}
template <int E>
cudaError_t launch_gated(const GatedNormParams &p, const Spread &s, cudaStream_t stream) {
  switch (s.v) {
    case 1: return launch_gated_v<E, 1>(p, s, stream);
    case 2: return launch_gated_v<E, 2>(p, s, stream);
    case 4: return launch_gated_v<E, 4>(p, s, stream);
    default: return launch_gated_v<E, 8>(p, s, stream);
  }
}

template <int E, int V, bool WIDE>
cudaError_t launch_residual_v(const ResidualNormParams &p, const Spread &s, cudaStream_t stream) {
  if constexpr (V <= 2) {
    if (s.block <= kBlock)
      return launch_overlapped(k_residual_norm<E, V, WIDE, kBlock>, dim3(ctas_for<k_residual_norm<E, V, WIDE, kBlock>>(s, p.T)), dim3(s.block), 0, stream, p,
                               s.team);
  }
  return launch_overlapped(k_residual_norm<E, V, WIDE, 1024>, dim3(ctas_for<k_residual_norm<E, V, WIDE, 1024>>(s, p.T)), dim3(s.block), 0, stream, p, s.team);
}
template <int E, bool WIDE>
cudaError_t launch_residual(const ResidualNormParams &p, const Spread &s, cudaStream_t stream) {
  switch (s.v) {
    case 1: return launch_residual_v<E, 1, WIDE>(p, s, stream);
    case 2: return launch_residual_v<E, 2, WIDE>(p, s, stream);
    case 4: return launch_residual_v<E, 4, WIDE>(p, s, stream);
    default: return launch_residual_v<E, 8, WIDE>(p, s, stream);
  }
}

}  // namespace

cudaError_t launch_gated_norm(const GatedNormParams &p, cudaStream_t stream) {
  int e = 1;
  for (int c : {8, 2}) {
    if (e == 1 && multiples(c, {p.P, p.x_stride_t, p.x_stride_h, p.z_stride_t, p.z_stride_h, p.out_stride_t, p.out_stride_h},
                            {p.x, p.z, p.out}, nullptr))
      e = c;
  }
  const Spread s = spread_of(p.P, e, p.T * p.H);
  if (s.v == 0) return launch_overlapped(k_gated_norm_long, dim3((unsigned)(p.T * p.H)), dim3(1024), 0, stream, p);
  return e == 8 ? launch_gated<8>(p, s, stream) : e == 2 ? launch_gated<2>(p, s, stream) : launch_gated<1>(p, s, stream);
}

cudaError_t launch_residual_norm(const ResidualNormParams &p, cudaStream_t stream) {
  const bool wide = p.residual_type == CCU_DTYPE_FP32;
  int e = 1;
  for (int c : {8, 2})
    if (e == 1 && multiples(c, {p.D, p.ld_x, p.ld_residual, p.ld_out}, {p.x, p.out, wide ? nullptr : p.residual}, wide ? p.residual : nullptr))
      e = c;
  const Spread s = spread_of(p.D, e, p.T);
  if (s.v == 0) return launch_overlapped(k_residual_norm_long, dim3((unsigned)p.T), dim3(1024), 0, stream, p);
  if (wide) return e == 8 ? launch_residual<8, true>(p, s, stream) : e == 2 ? launch_residual<2, true>(p, s, stream) : launch_residual<1, true>(p, s, stream);
  return e == 8 ? launch_residual<8, false>(p, s, stream) : e == 2 ? launch_residual<2, false>(p, s, stream) : launch_residual<1, false>(p, s, stream);
}

}  // namespace ccu
