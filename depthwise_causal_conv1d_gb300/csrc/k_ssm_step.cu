// Selective state update of one token per row (ccu_selective_state_update).
//
// Two launches: the convolution step of all H*P + 2*G*K channels (sums kept in 32 bits, in the
// caller's workspace), then the state step. The heads of a group share B and C, whose
// convolution state is shifted in place, so one kernel has to have read it before any writes it.
#include "ssm_internal.cuh"

namespace ccu {

int device_sm_count();

namespace {

// One thread per (row, channel): window sum, activation, and the slot's L entries shifted
// by one in place.
template <int ACT>
__global__ void __launch_bounds__(256) k_step_conv(StepParams p, int64_t channels) {
  grid_dependency_boundary();
  const uint16_t *x = static_cast<const uint16_t *>(p.xbc), *w = static_cast<const uint16_t *>(p.conv_weight);
  const uint16_t *bias = static_cast<const uint16_t *>(p.conv_bias);
  float *done = static_cast<float *>(p.workspace);
  const int64_t total = p.N * channels;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t n = i / channels, d = i - n * channels;
    const int64_t s = slot_of(p.indices, n, p.S, p.status_dev, d == 0);
    if (s < 0) continue;
    uint16_t *st = static_cast<uint16_t *>(p.conv_state) + s * p.conv_stride_s + d * p.conv_stride_d;
    const uint16_t v = x[n * p.ld_xbc + d];
    float acc = 0.0f;
    for (int64_t j = 0; j < p.W - 1; ++j)
      acc = __fmaf_rn(bf16_bits(st[(p.L - (p.W - 1) + j) * p.conv_stride_l]), bf16_bits(w[d * p.W + j]), acc);
    acc = __fmaf_rn(bf16_bits(v), bf16_bits(w[d * p.W + p.W - 1]), acc);
    if (bias != nullptr) acc += bf16_bits(bias[d]);
    done[i] = activate<ACT>(acc);
    for (int64_t l = 0; l + 1 < p.L; ++l) st[l * p.conv_stride_l] = st[(l + 1) * p.conv_stride_l];
    st[(p.L - 1) * p.conv_stride_l] = v;
  }
}

constexpr int kRows = 8;
constexpr int kWarps = 4;

// A warp owns 8 channels of one (row, head), K spread over its lanes.
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
  float sum = sum8_over_warp(y, lane);
  if (p.D != nullptr) sum = fmaf(__ldg(p.D + h), x, sum);
  if (writes) {
    if (p.z != nullptr) sum *= activate<1>(bf16_bits(static_cast<const uint16_t *>(p.z)[n * p.z_stride_n + h * p.z_stride_h + row]));
    *out = round_bf16(sum);
  }
}

}  // namespace

cudaError_t launch_step(const StepParams &p, cudaStream_t stream) {
  const int64_t channels = p.H * p.P + 2 * p.G * p.K;
  cudaError_t e = cudaSuccess;
  if (p.conv_weight != nullptr) {
    const int64_t blocks = (p.N * channels + 255) / 256, cap = (int64_t)device_sm_count() * 16;
    const dim3 grid((unsigned)(blocks < cap ? blocks : cap));
    e = p.act == CCU_ACT_SILU ? launch_overlapped(k_step_conv<1>, grid, dim3(256), 0, stream, p, channels)
                              : launch_overlapped(k_step_conv<0>, grid, dim3(256), 0, stream, p, channels);
    if (e != cudaSuccess) return e;
  }
  const int64_t blocks_p = (p.P + kRows * kWarps - 1) / (kRows * kWarps);
  const dim3 grid((unsigned)(p.N * p.H * blocks_p)), block(32 * kWarps);
  if (p.K <= 32) return launch_overlapped(k_step_state<1>, grid, block, 0, stream, p, channels, blocks_p);
  if (p.K <= 64) return launch_overlapped(k_step_state<2>, grid, block, 0, stream, p, channels, blocks_p);
  if (p.K <= 128) return launch_overlapped(k_step_state<4>, grid, block, 0, stream, p, channels, blocks_p);
  return launch_overlapped(k_step_state<8>, grid, block, 0, stream, p, channels, blocks_p);
}

}  // namespace ccu
