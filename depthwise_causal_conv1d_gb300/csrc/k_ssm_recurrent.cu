// Selective scan, token by token (ccu_selective_scan, CCU_SCAN_RECURRENT): the kernel for every
// size (any P, K <= 256, any alignment) and the anchor of the chunked kernel.
//
// A warp owns 8 channels of one (sequence, head) and keeps their 8 x K states in registers,
// K spread over the lanes, for the whole sequence; the state is read and written once. A token
// costs the decay (one exponential a warp), 2 fused multiply-adds and one multiply a state
// and one joint warp sum of the 8 outputs. It is bound by the latency of that chain, token after token, so
// long prompts belong to the chunked kernel (8 x 4096 tokens, 64 heads x 64 channels x 128 states: 9.8 ms, there 0.49).
// The next token's inputs are loaded one token ahead.
#include "ssm_internal.cuh"

namespace ccu {

namespace {

constexpr int kRows = 8;    // channels a warp
constexpr int kWarps = 4;

template <int NV>  // states a lane: k = lane + 32 j
struct Token {
  float x, z, b[NV], c[NV];
  uint16_t dt;
};

template <int NV>
__device__ __forceinline__ void load_token(const ScanParams &p, int64_t t, int64_t h, int64_t g, int64_t row, int lane,
                                           Token<NV> &v) {
  const uint16_t *b = static_cast<const uint16_t *>(p.b) + t * p.b_stride_t + g * p.b_stride_g;
  const uint16_t *c = static_cast<const uint16_t *>(p.c) + t * p.c_stride_t + g * p.c_stride_g;
  v.dt = __ldg(static_cast<const uint16_t *>(p.dt) + t * p.dt_stride_t + h);
  v.x = v.z = 0.0f;
  if (row < p.P) {
    v.x = bf16_bits(__ldg(static_cast<const uint16_t *>(p.x) + t * p.x_stride_t + h * p.x_stride_h + row));
    if (p.z != nullptr) v.z = bf16_bits(__ldg(static_cast<const uint16_t *>(p.z) + t * p.z_stride_t + h * p.z_stride_h + row));
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int k = lane + 32 * j;
    v.b[j] = k < p.K ? bf16_bits(__ldg(b + k)) : 0.0f;
    v.c[j] = k < p.K ? bf16_bits(__ldg(c + k)) : 0.0f;
  }
}

template <int NV>
__global__ void __launch_bounds__(32 * kWarps) k_scan_recurrent(ScanParams p, int64_t blocks_p) {
  grid_dependency_boundary();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t item = blockIdx.x;
  const int64_t pb = item % blocks_p;
  item /= blocks_p;
  const int64_t h = item % p.H, b = item / p.H;
  const int64_t row0 = (pb * kWarps + warp) * kRows;
  if (row0 >= p.P) return;
  const int64_t row = row0 + (lane >> 2);  // the channel whose x and y this lane handles
  const int64_t g = h / (p.H / p.G);
  const Bounds q = sequence_bounds(p.cu_seqlens, b, p.T);
  const int64_t s = slot_of(p.indices, b, p.S, p.status_dev, lane == 0 && h == 0 && row0 == 0);
  uint16_t *out = static_cast<uint16_t *>(p.out) + h * p.out_stride_h + row;
  const bool writes = (lane & 3) == 0 && row < p.P;
  if (s < 0) {
    for (int64_t t = q.begin; t < q.end; ++t)
      if (writes) out[t * p.out_stride_t] = 0;
    return;
  }
  float *st = p.state + s * p.state_stride_s + (h * p.P + row0) * p.K;
  const bool initial = p.has_initial != nullptr && __ldg(p.has_initial + b) != 0;
  float v[kRows][NV];
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int k = lane + 32 * j;
      v[r][j] = initial && row0 + r < p.P && k < p.K ? st[r * p.K + k] : 0.0f;
    }
  const float A = __ldg(p.A + h), D = p.D != nullptr ? __ldg(p.D + h) : 0.0f;
  Token<NV> now, next;
  if (q.begin < q.end) load_token(p, q.begin, h, g, row, lane, next);
  for (int64_t t = q.begin; t < q.end; ++t) {
    now = next;
    if (t + 1 < q.end) load_token(p, t + 1, h, g, row, lane, next);
    const float d = step_size(now.dt, p.dt_bias, h, p.dt_softplus);
    const float decay = expf(d * A);
    const float dx = d * now.x;
    float y[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const float xr = __shfl_sync(0xffffffffu, dx, 4 * r);
      y[r] = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        v[r][j] = fmaf(v[r][j], decay, xr * now.b[j]);
        y[r] = fmaf(v[r][j], now.c[j], y[r]);
      }
    }
    float sum = sum8_over<32>(y, lane);
    if (p.D != nullptr) sum = fmaf(D, now.x, sum);
    if (p.z != nullptr) sum *= activate<1>(now.z);
    if (writes) out[t * p.out_stride_t] = round_bf16(sum);
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int k = lane + 32 * j;
      if (row0 + r < p.P && k < p.K) st[r * p.K + k] = v[r][j];
    }
}

}  // namespace

cudaError_t launch_scan_recurrent(const ScanParams &p, cudaStream_t stream) {
  const int64_t blocks_p = (p.P + kRows * kWarps - 1) / (kRows * kWarps);
  const dim3 grid((unsigned)(p.n_seq * p.H * blocks_p)), block(32 * kWarps);
  if (p.K <= 32) return launch_overlapped(k_scan_recurrent<1>, grid, block, 0, stream, p, blocks_p);
  if (p.K <= 64) return launch_overlapped(k_scan_recurrent<2>, grid, block, 0, stream, p, blocks_p);
  if (p.K <= 128) return launch_overlapped(k_scan_recurrent<4>, grid, block, 0, stream, p, blocks_p);
  return launch_overlapped(k_scan_recurrent<8>, grid, block, 0, stream, p, blocks_p);
}

}  // namespace ccu
