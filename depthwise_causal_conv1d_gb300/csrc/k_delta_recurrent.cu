// The gated delta rule, token by token (ccu_gated_delta_rule, CCU_SCAN_RECURRENT): the kernel for every
// size (any P, K <= 256, any alignment).
//
// A warp owns 8 channels of one (sequence, head) and keeps their 8 x K states in registers,
// K spread over the lanes, for the whole sequence; the state is read and written once. With h = decay s, both sums of a
// token are taken over h: out = h q + u (k . q) is the sum over the new state, and waits for no second round.
//
// Bound by a token's chain of sums over the warp (0.70 us: 1 sequence of 32 heads x 128 channels x 128 states takes 14.0 us for 16 tokens, 47.5 for 64),
// and by the instructions of all warps where they fill the card: 128 such sequences of 64 tokens 2022 us, 14.9 TFLOP/s at 7 operations a
// state. Such calls go to the chunked kernel (424 us) where it serves.
#include "ssm_internal.cuh"

namespace ccu {

namespace {

constexpr int kRows = 8;    // channels a warp
constexpr int kWarps = 4;

template <int NV>  // states a lane: k = lane + 32 j
struct Token {
  float v, k[NV], q[NV];
  uint16_t a, b;
};

template <int NV>
__device__ __forceinline__ void load_token(const DeltaParams &p, int64_t t, int64_t h, int64_t g, int64_t row, int lane, Token<NV> &n) {
  const uint16_t *k = static_cast<const uint16_t *>(p.k) + t * p.k_stride_t + g * p.k_stride_g;
  const uint16_t *q = static_cast<const uint16_t *>(p.q) + t * p.q_stride_t + g * p.q_stride_g;
  n.a = __ldg(static_cast<const uint16_t *>(p.a) + t * p.a_stride_t + h);
  n.b = __ldg(static_cast<const uint16_t *>(p.b) + t * p.b_stride_t + h);
  n.v = row < p.P ? bf16_bits(__ldg(static_cast<const uint16_t *>(p.v) + t * p.v_stride_t + h * p.v_stride_h + row)) : 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = lane + 32 * j;
    n.k[j] = i < p.K ? bf16_bits(__ldg(k + i)) : 0.0f;
    n.q[j] = i < p.K ? bf16_bits(__ldg(q + i)) : 0.0f;
  }
}

template <int NV>
__global__ void __launch_bounds__(32 * kWarps) k_delta_recurrent(DeltaParams p, int64_t blocks_p) {
  grid_dependency_boundary();
  const unsigned full = 0xffffffffu;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t item = blockIdx.x;
  const int64_t pb = item % blocks_p;
  item /= blocks_p;
  const int64_t h = item % p.H, b = item / p.H;
  const int64_t row0 = (pb * kWarps + warp) * kRows;
  if (row0 >= p.P) return;
  const int64_t row = row0 + (lane >> 2);  // the channel whose v and output this lane handles
  const int64_t g = h / (p.H / p.G);
  const Bounds bounds = sequence_bounds(p.cu_seqlens, b, p.T);
  const int64_t s = slot_of(p.indices, b, p.S, p.status_dev, lane == 0 && h == 0 && row0 == 0);
  uint16_t *out = static_cast<uint16_t *>(p.out) + h * p.out_stride_h + row;
  const bool writes = (lane & 3) == 0 && row < p.P;
  if (s < 0) {
    for (int64_t t = bounds.begin; t < bounds.end; ++t)
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
      const int i = lane + 32 * j;
      v[r][j] = initial && row0 + r < p.P && i < p.K ? st[r * p.K + i] : 0.0f;
    }
  const float A = __ldg(p.A + h);
  Token<NV> now, next;
  if (bounds.begin < bounds.end) load_token(p, bounds.begin, h, g, row, lane, next);
  for (int64_t t = bounds.begin; t < bounds.end; ++t) {
    now = next;
    if (t + 1 < bounds.end) load_token(p, t + 1, h, g, row, lane, next);
    const float decay = expf(A * step_size(now.a, p.dt_bias, h, 1)), beta = sigmoid(bf16_bits(now.b));
    float kk = 0.0f, qq = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      kk = fmaf(now.k[j], now.k[j], kk);
      qq = fmaf(now.q[j], now.q[j], qq);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      kk += __shfl_xor_sync(full, kk, o);
      qq += __shfl_xor_sync(full, qq, o);
    }
    const float rk = p.qk_norm ? rsqrtf(kk + kUnitEps) : 1.0f, rq = p.qk_norm ? rsqrtf(qq + kUnitEps) : 1.0f;
    float kq = 0.0f, old[kRows], y[kRows];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      now.k[j] *= rk;
      now.q[j] *= rq;
      kq = fmaf(now.k[j], now.q[j], kq);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) kq += __shfl_xor_sync(full, kq, o);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      old[r] = y[r] = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        v[r][j] *= decay;
        old[r] = fmaf(v[r][j], now.k[j], old[r]);
        y[r] = fmaf(v[r][j], now.q[j], y[r]);
      }
    }
    const float u = beta * (now.v - sum8_over<32>(old, lane));
    const float sum = fmaf(u, kq, sum8_over<32>(y, lane));
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const float ur = __shfl_sync(full, u, 4 * r);
#pragma unroll
      for (int j = 0; j < NV; ++j) v[r][j] = fmaf(ur, now.k[j], v[r][j]);
    }
    if (writes) out[t * p.out_stride_t] = round_bf16(p.scale * sum);
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = lane + 32 * j;
      if (row0 + r < p.P && i < p.K) st[r * p.K + i] = v[r][j];
    }
}

}  // namespace

cudaError_t launch_delta_recurrent(const DeltaParams &p, cudaStream_t stream) {
  const int64_t blocks_p = (p.P + kRows * kWarps - 1) / (kRows * kWarps);
  const dim3 grid((unsigned)(p.n_seq * p.H * blocks_p)), block(32 * kWarps);
  if (p.K <= 32) return launch_overlapped(k_delta_recurrent<1>, grid, block, 0, stream, p, blocks_p);
  if (p.K <= 64) return launch_overlapped(k_delta_recurrent<2>, grid, block, 0, stream, p, blocks_p);
  if (p.K <= 128) return launch_overlapped(k_delta_recurrent<4>, grid, block, 0, stream, p, blocks_p);
  return launch_overlapped(k_delta_recurrent<8>, grid, block, 0, stream, p, blocks_p);
}

}  // namespace ccu
