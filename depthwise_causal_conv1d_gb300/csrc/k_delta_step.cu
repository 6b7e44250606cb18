// Gated delta update of one token per row (ccu_gated_delta_update).
//
// Two launches, as in the selective state update: the convolution step of all 2*G*K + H*P channels (sums kept in
// 32 bits, in the caller's workspace), then the state step; the heads of a group share q and k, whose convolution state is
// shifted in place, so one launch has to have read it before any other writes it.
//
// The state step reads and writes 8 bytes a state and does seven operations on it: it is bound by HBM, and by
// latency when there are few rows. A warp holds its channels' states in registers between the sum over the old state and
// the update, so the state passes once each way; both sums (with k and with q) are taken in one round, from h = decay s:
// out = h q + u (k . q). 256 rows, 230 of them with a slot, of 64 heads x 128 channels x 128 states, with
// the convolution of 16384 channels: 298 us, 6.7 TB/s of its bytes; 64 strided rows of 96 heads x 64 x 64: 33.5 us, 6.2 TB/s; one row of
// 16 heads x 128 x 128: 4.9 us, both launches: two launches and the latency of their loads.
#include "ssm_internal.cuh"

namespace ccu {

namespace {

constexpr int kRows = 8;
constexpr int kWarps = 4;

// The state step for any K, P and alignment: a warp owns 8 channels of one (row, head), K spread
// over its lanes one by one.
template <int NV>
__global__ void __launch_bounds__(32 * kWarps) k_delta_state(DeltaStepParams p, int64_t channels, int64_t blocks_p) {
  grid_dependency_boundary();
  const unsigned full = 0xffffffffu;
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
  const uint16_t *raw = static_cast<const uint16_t *>(p.qkv) + n * p.ld_qkv;
  auto value = [&](int64_t d) { return conv ? done[d] : bf16_bits(raw[d]); };
  const int64_t at_q = h / (p.H / p.G) * p.K, at_k = p.G * p.K + at_q;
  float *st = p.state + s * p.state_stride_s + (h * p.P + row0) * p.K;
  const float v = row < p.P ? value(2 * p.G * p.K + h * p.P + row) : 0.0f;
  const float decay = expf(__ldg(p.A + h) * step_size(static_cast<const uint16_t *>(p.a)[n * p.a_stride_n + h], p.dt_bias, h, 1));
  const float beta = sigmoid(bf16_bits(static_cast<const uint16_t *>(p.b)[n * p.b_stride_n + h]));
  float w[kRows][NV], k[NV], q[NV], kk = 0.0f, qq = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = lane + 32 * j;
    q[j] = i < p.K ? value(at_q + i) : 0.0f;
    k[j] = i < p.K ? value(at_k + i) : 0.0f;
    kk = fmaf(k[j], k[j], kk);
    qq = fmaf(q[j], q[j], qq);
#pragma unroll
    for (int r = 0; r < kRows; ++r) w[r][j] = row0 + r < p.P && i < p.K ? st[r * p.K + i] : 0.0f;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    kk += __shfl_xor_sync(full, kk, o);
    qq += __shfl_xor_sync(full, qq, o);
  }
  const float rk = p.qk_norm ? rsqrtf(kk + kUnitEps) : 1.0f, rq = p.qk_norm ? rsqrtf(qq + kUnitEps) : 1.0f;
  float kq = 0.0f, old[kRows] = {}, y[kRows] = {};
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    k[j] *= rk;
    q[j] *= rq;
    kq = fmaf(k[j], q[j], kq);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      w[r][j] *= decay;
      old[r] = fmaf(w[r][j], k[j], old[r]);
      y[r] = fmaf(w[r][j], q[j], y[r]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) kq += __shfl_xor_sync(full, kq, o);
  const float u = beta * (v - sum8_over<32>(old, lane));
  const float sum = fmaf(u, kq, sum8_over<32>(y, lane));
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const float ur = __shfl_sync(full, u, 4 * r);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = lane + 32 * j;
      if (row0 + r < p.P && i < p.K) st[r * p.K + i] = fmaf(ur, k[j], w[r][j]);
    }
  }
  if (writes) *out = round_bf16(p.scale * sum);
}

// The state step for K % 4 == 0 and states on 16-byte boundaries. LANES lanes hold a channel's K
// states as NV float4 each (LANES * 4 * NV >= K), so a warp's load covers 32 / LANES channels,
// and every warp has 8 of them in flight.
template <int LANES, int NV, bool CONV>
__global__ void __launch_bounds__(32 * kWarps, NV == 1 ? 8 : 4) k_delta_state_v(DeltaStepParams p, int64_t channels, int64_t blocks_p) {
  grid_dependency_boundary();
  constexpr int kSub = 32 / LANES;          // channels a load
  constexpr int kRowsW = kRows * kSub;      // channels a warp
  const unsigned full = 0xffffffffu;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane / LANES, l = lane % LANES;
  const uint32_t items = blockIdx.x;
  const uint32_t pb = items % (uint32_t)blocks_p, hn = items / (uint32_t)blocks_p;
  const int64_t h = hn % (uint64_t)p.H, n = hn / (uint64_t)p.H;
  const int64_t row0 = ((int64_t)pb * kWarps + warp) * kRowsW;
  if (row0 >= p.P) return;
  const int64_t row = row0 + (l / (LANES / 8)) * kSub + sub;  // the channel whose v and output this lane handles
  const bool mine = row < p.P, writes = mine && l % (LANES / 8) == 0;
  uint16_t *out = static_cast<uint16_t *>(p.out) + n * p.out_stride_n + h * p.out_stride_h + row;
  const int64_t s = slot_of(p.indices, n, p.S, p.status_dev, lane == 0 && h == 0 && row0 == 0);
  if (s < 0) {
    if (writes) *out = 0;
    return;
  }
  float4 w[kRows][NV];
  float *st = p.state + s * p.state_stride_s + (h * p.P + row0 + sub) * p.K + 4 * l;
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      w[r][j] = make_float4(0, 0, 0, 0);
      if (row0 + r * kSub + sub < p.P && 4 * (l + LANES * j) < p.K)
        w[r][j] = *reinterpret_cast<const float4 *>(st + (int64_t)r * kSub * p.K + 4 * LANES * j);
    }
  const float *done = static_cast<const float *>(p.workspace) + n * channels;
  const uint16_t *raw = static_cast<const uint16_t *>(p.qkv) + n * p.ld_qkv;
  auto value = [&](int64_t d) { return CONV ? done[d] : bf16_bits(raw[d]); };
  const int64_t at_q = h / (p.H / p.G) * p.K, at_k = p.G * p.K + at_q;
  const float v = mine ? value(2 * p.G * p.K + h * p.P + row) : 0.0f;
  const float step = step_size(__ldg(static_cast<const uint16_t *>(p.a) + n * p.a_stride_n + h), p.dt_bias, h, 1);
  const float decay = expf(__ldg(p.A + h) * step);
  const float beta = sigmoid(bf16_bits(__ldg(static_cast<const uint16_t *>(p.b) + n * p.b_stride_n + h)));
  float k[4 * NV], q[4 * NV], kk = 0.0f, qq = 0.0f, kq = 0.0f;
#pragma unroll
  for (int j = 0; j < 4 * NV; ++j) {
    const int i = 4 * (l + LANES * (j / 4)) + j % 4;
    q[j] = i < p.K ? value(at_q + i) : 0.0f;
    k[j] = i < p.K ? value(at_k + i) : 0.0f;
    kk = fmaf(k[j], k[j], kk);
    qq = fmaf(q[j], q[j], qq);
  }
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) {
    kk += __shfl_xor_sync(full, kk, o);
    qq += __shfl_xor_sync(full, qq, o);
  }
  const float rk = p.qk_norm ? rsqrtf(kk + kUnitEps) : 1.0f, rq = p.qk_norm ? rsqrtf(qq + kUnitEps) : 1.0f;
#pragma unroll
  for (int j = 0; j < 4 * NV; ++j) {
    k[j] *= rk;
    q[j] *= rq;
    kq = fmaf(k[j], q[j], kq);
  }
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) kq += __shfl_xor_sync(full, kq, o);
  // Both sums over the old state, two states an instruction; the decay is one factor of either
  float old[kRows], y[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    float2 a = make_float2(0.0f, 0.0f), c = a;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const float2 lo = make_float2(w[r][j].x, w[r][j].y), hi = make_float2(w[r][j].z, w[r][j].w);
      a = __ffma2_rn(lo, make_float2(k[4 * j], k[4 * j + 1]), a);
      c = __ffma2_rn(lo, make_float2(q[4 * j], q[4 * j + 1]), c);
      a = __ffma2_rn(hi, make_float2(k[4 * j + 2], k[4 * j + 3]), a);
      c = __ffma2_rn(hi, make_float2(q[4 * j + 2], q[4 * j + 3]), c);
    }
    old[r] = a.x + a.y;
    y[r] = c.x + c.y;
  }
  const float u = beta * fmaf(-decay, sum8_over<LANES>(old, lane), v);
  const float sum = fmaf(u, kq, decay * sum8_over<LANES>(y, lane));
  const float2 decays = make_float2(decay, decay);
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const float ur = __shfl_sync(full, u, sub * LANES + r * (LANES / 8));
    const float2 us = make_float2(ur, ur);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const float2 lo = __ffma2_rn(us, make_float2(k[4 * j], k[4 * j + 1]), __fmul2_rn(make_float2(w[r][j].x, w[r][j].y), decays));
      const float2 hi = __ffma2_rn(us, make_float2(k[4 * j + 2], k[4 * j + 3]), __fmul2_rn(make_float2(w[r][j].z, w[r][j].w), decays));
      if (row0 + r * kSub + sub < p.P && 4 * (l + LANES * j) < p.K)
        *reinterpret_cast<float4 *>(st + (int64_t)r * kSub * p.K + 4 * LANES * j) = make_float4(lo.x, lo.y, hi.x, hi.y);
    }
  }
  if (writes) *out = round_bf16(p.scale * sum);
}

template <int LANES, int NV>
cudaError_t launch_state_v(const DeltaStepParams &p, int64_t channels, cudaStream_t stream) {
  const int64_t rows = kRows * (32 / LANES) * kWarps;
  const int64_t blocks_p = (p.P + rows - 1) / rows;
  const dim3 grid((unsigned)(p.N * p.H * blocks_p)), block(32 * kWarps);
  return p.conv_weight != nullptr ? launch_overlapped(k_delta_state_v<LANES, NV, true>, grid, block, 0, stream, p, channels, blocks_p)
                                  : launch_overlapped(k_delta_state_v<LANES, NV, false>, grid, block, 0, stream, p, channels, blocks_p);
}

}  // namespace

cudaError_t launch_delta_step(const DeltaStepParams &p, cudaStream_t stream) {
  const int64_t channels = 2 * p.G * p.K + p.H * p.P;
  if (p.conv_weight != nullptr) {
    StepParams c = {};
    c.xbc = p.qkv, c.ld_xbc = p.ld_qkv;
    c.conv_weight = p.conv_weight, c.conv_bias = p.conv_bias, c.conv_state = p.conv_state;
    c.conv_stride_s = p.conv_stride_s, c.conv_stride_d = p.conv_stride_d, c.conv_stride_l = p.conv_stride_l;
    c.indices = p.indices, c.workspace = p.workspace, c.status_dev = p.status_dev;
    c.N = p.N, c.S = p.S, c.L = p.L, c.W = p.W, c.act = p.act;
    const cudaError_t e = launch_step_conv(c, channels, true, stream);
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
  if (p.K <= 32) return launch_overlapped(k_delta_state<1>, grid, block, 0, stream, p, channels, blocks_p);
  if (p.K <= 64) return launch_overlapped(k_delta_state<2>, grid, block, 0, stream, p, channels, blocks_p);
  if (p.K <= 128) return launch_overlapped(k_delta_state<4>, grid, block, 0, stream, p, channels, blocks_p);
  return launch_overlapped(k_delta_state<8>, grid, block, 0, stream, p, channels, blocks_p);
}

}  // namespace ccu
