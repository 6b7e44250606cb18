// Selective state update of one token per row (ccu_selective_state_update).
//
// Two launches: the convolution step of all H*P + 2*G*K channels (sums kept in 32 bits, in the
// caller's workspace), then the state step. The heads of a group share B and C, whose
// convolution state is shifted in place, so one kernel has to have read it before any writes it.
//
// The state step reads and writes 8 bytes a state and does five operations on it: it is bound by
// HBM, and by latency when there are few rows. (Left out: one kernel that takes the convolution of
// its own channels and of its group's B and C itself, with the states already on their way. Every
// CTA then repeats 2 K channels of 4 taps: 256 paged rows 527 us against 303.) 256 rows, 230 of them with a
// slot, of 128 heads x 64 channels x 128 states: 303 us, 6.5 TB/s; 64 rows of 96 x 64 x 64: 37 us, 5.7 TB/s; one row
// of 32 x 64 x 128: 4.5 us, both launches.
#include "ssm_internal.cuh"

namespace ccu {

int device_sm_count();

namespace {

// One thread per (row, channel): window sum, activation, and the slot's L entries shifted
// by one in place. Up to 8 entries are loaded at once; longer states in a loop.
template <int ACT>
__global__ void __launch_bounds__(128) k_step_conv(StepParams p, int64_t channels) {
  grid_dependency_boundary();
  const uint16_t *x = static_cast<const uint16_t *>(p.xbc), *w = static_cast<const uint16_t *>(p.conv_weight);
  const uint16_t *bias = static_cast<const uint16_t *>(p.conv_bias);
  float *done = static_cast<float *>(p.workspace);
  const int L = (int)(p.L < 9 ? p.L : 9), W = (int)(p.W < 9 ? p.W : 9);
  for (int64_t n = blockIdx.y; n < p.N; n += gridDim.y) {
    const int64_t d = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (d >= channels) return;
    const int64_t s = slot_of(p.indices, n, p.S, p.status_dev, d == 0);
    if (s < 0) continue;
    uint16_t *st = static_cast<uint16_t *>(p.conv_state) + s * p.conv_stride_s + d * p.conv_stride_d;
    const uint16_t v = x[n * p.ld_xbc + d];
    float acc = 0.0f;
    if (L <= 8) {
      uint16_t e[8], window[8], f[8];
      const uint16_t *first = st + (L - (W - 1)) * p.conv_stride_l;
#pragma unroll
      for (int l = 0; l < 8; ++l) e[l] = l < L ? st[l * p.conv_stride_l] : 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        window[j] = j < W - 1 ? first[j * p.conv_stride_l] : 0;
        f[j] = j < W - 1 ? w[d * p.W + j] : 0;
      }
      const uint16_t newest = w[d * p.W + W - 1];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < W - 1) acc = __fmaf_rn(bf16_bits(window[j]), bf16_bits(f[j]), acc);
      acc = __fmaf_rn(bf16_bits(v), bf16_bits(newest), acc);
#pragma unroll
      for (int l = 0; l < 8; ++l)
        if (l < L) st[l * p.conv_stride_l] = l + 1 < L ? e[l < 7 ? l + 1 : 7] : v;
    } else {
      for (int64_t j = 0; j < p.W - 1; ++j)
        acc = __fmaf_rn(bf16_bits(st[(p.L - (p.W - 1) + j) * p.conv_stride_l]), bf16_bits(w[d * p.W + j]), acc);
      acc = __fmaf_rn(bf16_bits(v), bf16_bits(w[d * p.W + p.W - 1]), acc);
      for (int64_t l = 0; l + 1 < p.L; ++l) st[l * p.conv_stride_l] = st[(l + 1) * p.conv_stride_l];
      st[(p.L - 1) * p.conv_stride_l] = v;
    }
    if (bias != nullptr) acc += bf16_bits(bias[d]);
    done[n * channels + d] = activate<ACT>(acc);
  }
}

constexpr int kRows = 8;
constexpr int kWarps = 4;

// The state step for any K, P and alignment: a warp owns 8 channels of one (row, head), K spread
// over its lanes one by one.
template <int NV>
__global__ void __launch_bounds__(32 * kWarps) k_step_state(StepParams p, int64_t channels, int64_t blocks_p) {
  grid_dependency_boundary();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t item = blockIdx.x;
  const int64_t pb = item % blocks_p;
  item /= blocks_p;
  const int64_t h = item % p.H, n = item / p.H;
  const int64_t row0 = (pb * kWarps + warp) * kRows;
  if (row0 >= p.P) return;
  const int64_t row = row0 + (lane >> 2);
  const bool writes = (lane & 3) == 0 && row < p.P;
  uint16_t *out = static_cast<uint16_t *>(p.out) + n * p.out_stride_n + h * p.out_stride_h + row;
  const int64_t s = slot_of(p.indices, n, p.S, p.status_dev, lane == 0 && h == 0 && row0 == 0);
  if (s < 0) {
    if (writes) *out = 0;
    return;
  }
  const bool conv = p.conv_weight != nullptr;
  const float *done = static_cast<const float *>(p.workspace) + n * channels;
  const uint16_t *raw = static_cast<const uint16_t *>(p.xbc) + n * p.ld_xbc;
  auto value = [&](int64_t d) { return conv ? done[d] : bf16_bits(raw[d]); };
  const int64_t at_b = p.H * p.P + h / (p.H / p.G) * p.K, at_c = at_b + p.G * p.K;
  float *st = p.state + s * p.state_stride_s + (h * p.P + row0) * p.K;
  const float x = row < p.P ? value(h * p.P + row) : 0.0f;
  const float d = step_size(static_cast<const uint16_t *>(p.dt)[n * p.dt_stride_n + h], p.dt_bias, h, p.dt_softplus);
  const float decay = expf(d * __ldg(p.A + h)), dx = d * x;
  float y[kRows] = {};
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int k = lane + 32 * j;
    const float b = k < p.K ? value(at_b + k) : 0.0f, c = k < p.K ? value(at_c + k) : 0.0f;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const float xr = __shfl_sync(0xffffffffu, dx, 4 * r);
      if (row0 + r < p.P && k < p.K) {
        const float v = fmaf(st[r * p.K + k], decay, xr * b);
        st[r * p.K + k] = v;
        y[r] = fmaf(v, c, y[r]);
      }
    }
  }
  float sum = sum8_over<32>(y, lane);
  if (p.D != nullptr) sum = fmaf(__ldg(p.D + h), x, sum);
  if (writes) {
    if (p.z != nullptr) sum *= activate<1>(bf16_bits(static_cast<const uint16_t *>(p.z)[n * p.z_stride_n + h * p.z_stride_h + row]));
    *out = round_bf16(sum);
  }
}

// The state step for K % 4 == 0 and states on 16-byte boundaries. LANES lanes hold a channel's K
// states as NV float4 each (LANES * 4 * NV >= K), so a warp's load covers 32 / LANES channels,
// and every warp has 8 of them in flight: 4 KB of the state a warp at K = 128.
template <int LANES, int NV, bool CONV>
__global__ void __launch_bounds__(32 * kWarps) k_step_state_v(StepParams p, int64_t channels, int64_t blocks_p) {
  grid_dependency_boundary();
  constexpr int kSub = 32 / LANES;          // channels a load
  constexpr int kRowsW = kRows * kSub;      // channels a warp
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane / LANES, l = lane % LANES;
  const uint32_t items = blockIdx.x;
  const uint32_t pb = items % (uint32_t)blocks_p, hn = items / (uint32_t)blocks_p;
  const uint32_t h = hn % (uint32_t)p.H;
  const int64_t n = hn / (uint32_t)p.H;
  const int64_t row0 = ((int64_t)pb * kWarps + warp) * kRowsW;
  if (row0 >= p.P) return;
  const int64_t row = row0 + (l / (LANES / 8)) * kSub + sub;  // the channel whose x and y this lane handles
  const bool mine = row < p.P, writes = mine && l % (LANES / 8) == 0;
  uint16_t *out = static_cast<uint16_t *>(p.out) + n * p.out_stride_n + h * p.out_stride_h + row;
  const int64_t s = slot_of(p.indices, n, p.S, p.status_dev, lane == 0 && h == 0 && row0 == 0);
  if (s < 0) {
    if (writes) *out = 0;
    return;
  }
  float4 v[kRows][NV];
  float *st = p.state + s * p.state_stride_s + ((int64_t)h * p.P + row0 + sub) * p.K + 4 * l;
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      v[r][j] = make_float4(0, 0, 0, 0);
      if (row0 + r * kSub + sub < p.P && 4 * (l + LANES * j) < p.K)
        v[r][j] = *reinterpret_cast<const float4 *>(st + (int64_t)r * kSub * p.K + 4 * LANES * j);
    }
  float z = 0.0f;
  if (p.z != nullptr && mine) z = bf16_bits(__ldg(static_cast<const uint16_t *>(p.z) + n * p.z_stride_n + h * p.z_stride_h + row));
  const float skip = p.D != nullptr ? __ldg(p.D + h) : 0.0f;
  const float d = step_size(__ldg(static_cast<const uint16_t *>(p.dt) + n * p.dt_stride_n + h), p.dt_bias, h, p.dt_softplus);
  const float decay = expf(d * __ldg(p.A + h));
  const int64_t at_b = p.H * p.P + h / (uint32_t)(p.H / p.G) * p.K, at_c = at_b + p.G * p.K;
  float x = 0.0f;
  float4 b[NV], c[NV];
  if (CONV) {
    const float *done = static_cast<const float *>(p.workspace) + n * channels;
    if (mine) x = done[(int64_t)h * p.P + row];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int k = 4 * (l + LANES * j);
      const bool in = k < p.K;  // whole vectors: K % 4 == 0 (and H*P need not be a multiple of 4: scalar loads)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        (&b[j].x)[e] = in ? done[at_b + k + e] : 0.0f;
        (&c[j].x)[e] = in ? done[at_c + k + e] : 0.0f;
      }
    }
  } else {
    const uint16_t *raw = static_cast<const uint16_t *>(p.xbc) + n * p.ld_xbc;
    if (mine) x = bf16_bits(raw[(int64_t)h * p.P + row]);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int k = 4 * (l + LANES * j);
      const bool in = k < p.K;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        (&b[j].x)[e] = in ? bf16_bits(raw[at_b + k + e]) : 0.0f;
        (&c[j].x)[e] = in ? bf16_bits(raw[at_c + k + e]) : 0.0f;
      }
    }
  }
  const float dx = d * x;
  float y[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const float xr = __shfl_sync(0xffffffffu, dx, sub * LANES + r * (LANES / 8));
    y[r] = 0.0f;
    const bool in_p = row0 + r * kSub + sub < p.P;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float4 &q = v[r][j];
      q.x = fmaf(q.x, decay, xr * b[j].x);
      q.y = fmaf(q.y, decay, xr * b[j].y);
      q.z = fmaf(q.z, decay, xr * b[j].z);
      q.w = fmaf(q.w, decay, xr * b[j].w);
      y[r] = fmaf(q.x, c[j].x, fmaf(q.y, c[j].y, fmaf(q.z, c[j].z, fmaf(q.w, c[j].w, y[r]))));
      if (in_p && 4 * (l + LANES * j) < p.K)
        *reinterpret_cast<float4 *>(st + (int64_t)r * kSub * p.K + 4 * LANES * j) = q;
    }
  }
  float sum = sum8_over<LANES>(y, lane);
  sum = p.D != nullptr ? fmaf(skip, x, sum) : sum;
  if (p.z != nullptr) sum *= activate<1>(z);
  if (writes) *out = round_bf16(sum);
}

template <int LANES, int NV>
cudaError_t launch_state_v(const StepParams &p, int64_t channels, cudaStream_t stream) {
  const int64_t rows = kRows * (32 / LANES) * kWarps;
  const int64_t blocks_p = (p.P + rows - 1) / rows;
  const dim3 grid((unsigned)(p.N * p.H * blocks_p)), block(32 * kWarps);
  return p.conv_weight != nullptr ? launch_overlapped(k_step_state_v<LANES, NV, true>, grid, block, 0, stream, p, channels, blocks_p)
                                  : launch_overlapped(k_step_state_v<LANES, NV, false>, grid, block, 0, stream, p, channels, blocks_p);
}

}  // namespace

cudaError_t launch_step(const StepParams &p, cudaStream_t stream) {
  const int64_t channels = p.H * p.P + 2 * p.G * p.K;
  cudaError_t e = cudaSuccess;
  if (p.conv_weight != nullptr) {
    const dim3 grid((unsigned)((channels + 127) / 128), (unsigned)(p.N < 65535 ? p.N : 65535));
    e = p.act == CCU_ACT_SILU ? launch_overlapped(k_step_conv<1>, grid, dim3(128), 0, stream, p, channels)
                              : launch_overlapped(k_step_conv<0>, grid, dim3(128), 0, stream, p, channels);
    if (e != cudaSuccess) return e;
  }
  // 16-byte vectors of the state need whole ones in every channel, slot and the base.
  if (p.K % 4 == 0 && p.state_stride_s % 4 == 0 && reinterpret_cast<uintptr_t>(p.state) % 16 == 0) {
    if (p.K <= 32) return launch_state_v<8, 1>(p, channels, stream);
    if (p.K <= 64) return launch_state_v<16, 1>(p, channels, stream);
    if (p.K <= 128) return launch_state_v<32, 1>(p, channels, stream);
    return launch_state_v<32, 2>(p, channels, stream);
  }
  const int64_t blocks_p = (p.P + kRows * kWarps - 1) / (kRows * kWarps);
  const dim3 grid((unsigned)(p.N * p.H * blocks_p)), block(32 * kWarps);
  if (p.K <= 32) return launch_overlapped(k_step_state<1>, grid, block, 0, stream, p, channels, blocks_p);
  if (p.K <= 64) return launch_overlapped(k_step_state<2>, grid, block, 0, stream, p, channels, blocks_p);
  if (p.K <= 128) return launch_overlapped(k_step_state<4>, grid, block, 0, stream, p, channels, blocks_p);
  return launch_overlapped(k_step_state<8>, grid, block, 0, stream, p, channels, blocks_p);
}

}  // namespace ccu
