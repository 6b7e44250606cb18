// C-ABI entry points of the gated delta rule and of the norms around a layer: argument checks (typed declines) and
// kernel choice.
#include <cmath>

#include "ssm_checks.cuh"
#include "ssm_internal.cuh"

namespace ccu {

int device_sm_count();

namespace {

ccu_status_t check_rule(const DeltaParams &a, bool *noop) {
  ccu_status_t st = check_heads(a.H, a.P, a.K, a.G, a.S);
  if (st != CCU_OK) return st;
  CCU_DECLINE(a.T < 0 || a.n_seq < 0, "T and n_seq must be >= 0");
  CCU_DECLINE(a.route < 0 || a.route >= CCU_SCAN_ROUTE_COUNT, "unknown route %d", a.route);
  CCU_DECLINE(!std::isfinite(a.scale), "scale must be finite");
  if (a.T > INT32_MAX) return fail(CCU_ERR_NOT_IMPLEMENTED, "T < 2^31 rows are served");
  *noop = a.n_seq == 0 || a.H == 0 || a.P == 0;
  if (*noop) return CCU_OK;
  CCU_DECLINE(a.cu_seqlens == nullptr, "cu_seqlens must not be NULL");
  CCU_DECLINE(a.A == nullptr, "A must not be NULL");
  CCU_DECLINE(a.T > 0 && (a.q == nullptr || a.k == nullptr || a.v == nullptr || a.a == nullptr || a.b == nullptr || a.out == nullptr),
              "q, k, v, a, b and out must not be NULL");
  CCU_DECLINE(!aligned(a.q, 2) || !aligned(a.k, 2) || !aligned(a.v, 2) || !aligned(a.a, 2) || !aligned(a.b, 2) || !aligned(a.out, 2),
              "BF16 tensors must be 2-byte aligned");
  CCU_DECLINE(!aligned(a.A, 4) || !aligned(a.dt_bias, 4), "FP32 tensors must be 4-byte aligned");
  CCU_DECLINE(!aligned(a.cu_seqlens, 4) || !aligned(a.indices, 4) || !aligned(a.has_initial, 4) || !aligned(a.status_dev, 4),
              "int32 tensors must be 4-byte aligned");
  CCU_DECLINE(!aligned(a.workspace, 16), "workspace must be 16-byte aligned");
  const int64_t strides[] = {a.q_stride_t, a.q_stride_g, a.k_stride_t, a.k_stride_g, a.v_stride_t, a.v_stride_h,
                             a.a_stride_t, a.b_stride_t, a.out_stride_t, a.out_stride_h};
  for (int64_t v : strides) {
    CCU_DECLINE(v < 0, "strides must be >= 0");
    int64_t u;
    if (!mul(a.T, v, &u) || !mul(a.H, v, &u)) return overflow();
  }
  CCU_DECLINE(a.indices == nullptr && a.S < a.n_seq,
              "without indices sequence b uses slot b, so S must be >= n_seq (S=%lld, n_seq=%lld)", (long long)a.S,
              (long long)a.n_seq);
  st = check_state(a.state, a.state_stride_s, a.H * a.P * a.K, a.S);
  if (st != CCU_OK) return st;
  int64_t v;
  if (!mul(a.n_seq, a.H, &v) || !mul(v, (a.P + 31) / 32, &v) || v > kMaxGrid)
    return fail(CCU_ERR_NOT_IMPLEMENTED, "n_seq * H * ceil(P / 32) must be < 2^31");
  return CCU_OK;
}

// The chunked kernel copies tiles of rows in 16-byte pieces and holds up to 128 states a channel.
bool chunked_rule_serves(const DeltaParams &a) {
  if (a.P % 8 != 0 || a.K % 8 != 0 || a.K > kChunkMaxStates) return false;
  if (!aligned(a.q, 16) || !aligned(a.k, 16) || !aligned(a.v, 16) || !aligned(a.out, 16) || a.out_stride_t % 8 != 0 || a.out_stride_h % 8 != 0)
    return false;
  if (!aligned(a.state, 16) || a.state_stride_s % 4 != 0) return false;
  const int64_t steps[][2] = {{a.q_stride_t, a.T}, {a.q_stride_g, a.G}, {a.k_stride_t, a.T}, {a.k_stride_g, a.G}, {a.v_stride_t, a.T}, {a.v_stride_h, a.H}};
  // What a tensor map describes: real strides (no row or head shared by a stride of 0), multiples of 16 bytes below 2^40.
  for (const auto &v : steps)
    if (v[0] % 8 != 0 || (v[1] > 1 && (v[0] < 8 || v[0] >= (int64_t(1) << 39)))) return false;
  return a.H <= INT32_MAX && a.P <= INT32_MAX;
}

// From this many tokens a sequence (on average: the lengths are on the device) AUTO takes the chunked kernel, times the channels of a
// CTA's 128 that it fills: a chunk costs the same however few tokens it holds. Token by token against chunked, in microseconds:
//   32 heads of 128 channels, 128 states: 1 sequence of 12 tokens 11.2 against 16.0, of 16 14.0 against 16.0, of 24 19.5 against
//   16.1; 16 sequences of 12 54.5 against 64.7, of 16 69.5 against 64.7; 128 of 8 309 against 421, of 12 432 against 423, of 16 554 against 422
//   48 heads of 64 channels, 64 states: 16 sequences of 24 tokens 59 against 80, of 32 77 against 80; 128 of 24 420 against 531, of 32 550
//   against 531. 16 heads of 32 channels, 64 states: 128 sequences of 48 tokens 142 against 179, of 64 187 against 176
constexpr int64_t kChunkedRuleMinTokens = 16;

bool long_enough(const DeltaParams &a) {
  const int64_t filled = a.P < 128 ? a.P : 128;
  return a.T / kChunkedRuleMinTokens >= a.n_seq && a.T / a.n_seq * filled >= kChunkedRuleMinTokens * 128;
}

ccu_status_t choose_rule(const DeltaParams &a, int *route) {
  if (a.route == CCU_SCAN_CHUNKED && !chunked_rule_serves(a))
    return fail(CCU_ERR_NOT_IMPLEMENTED,
                "the chunked delta rule needs P and K in multiples of 8, K <= %lld, and rows of q, k, v and out and slots on 16-byte boundaries",
                (long long)kChunkMaxStates);
  if (a.route != CCU_SCAN_AUTO) *route = a.route;
  else *route = chunked_rule_serves(a) && long_enough(a) ? CCU_SCAN_CHUNKED : CCU_SCAN_RECURRENT;
  return CCU_OK;
}

ccu_status_t check_delta_update(const DeltaStepParams &a, bool *noop) {
  ccu_status_t st = check_heads(a.H, a.P, a.K, a.G, a.S);
  if (st != CCU_OK) return st;
  CCU_DECLINE(a.N < 0, "N must be >= 0");
  CCU_DECLINE(!std::isfinite(a.scale), "scale must be finite");
  const bool conv = a.conv_weight != nullptr;
  if (conv) {
    CCU_DECLINE(a.act != CCU_ACT_IDENTITY && a.act != CCU_ACT_SILU,
                "act must be CCU_ACT_IDENTITY or CCU_ACT_SILU, got %d", a.act);
    CCU_DECLINE(a.W < 1, "W must be >= 1, got %lld", (long long)a.W);
    CCU_DECLINE(a.L < a.W - 1, "L must be >= W - 1 (L=%lld, W=%lld)", (long long)a.L, (long long)a.W);
    if (a.L < 1) return fail(CCU_ERR_NOT_IMPLEMENTED, "an empty state (L = 0) is not served");
  }
  *noop = a.N == 0 || a.H == 0 || a.P == 0;
  if (*noop) return CCU_OK;
  CCU_DECLINE(a.qkv == nullptr || a.a == nullptr || a.b == nullptr || a.A == nullptr || a.out == nullptr,
              "qkv, a, b, A and out must not be NULL");
  CCU_DECLINE(!aligned(a.qkv, 2) || !aligned(a.conv_weight, 2) || !aligned(a.conv_bias, 2) || !aligned(a.conv_state, 2) ||
                  !aligned(a.a, 2) || !aligned(a.b, 2) || !aligned(a.out, 2),
              "BF16 tensors must be 2-byte aligned");
  CCU_DECLINE(!aligned(a.A, 4) || !aligned(a.dt_bias, 4), "FP32 tensors must be 4-byte aligned");
  CCU_DECLINE(!aligned(a.indices, 4) || !aligned(a.status_dev, 4), "int32 tensors must be 4-byte aligned");
  const int64_t channels = 2 * a.G * a.K + a.H * a.P;
  CCU_DECLINE(a.N > 1 && a.ld_qkv < channels, "ld_qkv must be >= 2*G*K + H*P");
  const int64_t strides[] = {a.ld_qkv, a.a_stride_n, a.b_stride_n, a.out_stride_n, a.out_stride_h};
  int64_t v;
  for (int64_t s : strides) {
    CCU_DECLINE(s < 0, "strides must be >= 0");
    if (!mul(a.N, s, &v) || !mul(a.H, s, &v)) return overflow();
  }
  if (!mul(a.N, channels, &v)) return overflow();
  CCU_DECLINE(a.indices == nullptr && a.S < a.N,
              "without indices row n uses slot n, so S must be >= N (S=%lld, N=%lld)", (long long)a.S, (long long)a.N);
  st = check_state(a.state, a.state_stride_s, a.H * a.P * a.K, a.S);
  if (st != CCU_OK) return st;
  if (conv) {
    CCU_DECLINE(a.conv_state == nullptr && a.S > 0, "conv_state must not be NULL");
    CCU_DECLINE(a.conv_stride_s < 0 || a.conv_stride_d < 0 || a.conv_stride_l < 0, "strides must be >= 0");
    if (!mul(a.S, a.conv_stride_s, &v) || !mul(channels, a.conv_stride_d, &v) || !mul(a.L, a.conv_stride_l, &v) ||
        !mul(channels, a.W, &v))
      return overflow();
    CCU_DECLINE(a.workspace == nullptr || !aligned(a.workspace, 16) || a.workspace_bytes < 4 * a.N * channels,
                "the convolution needs a 16-byte aligned workspace of 4 * N * (2*G*K + H*P) = %lld bytes, got %lld",
                (long long)(4 * a.N * channels), (long long)a.workspace_bytes);
  }
  if (!mul(a.N, a.H, &v) || !mul(v, (a.P + 7) / 8, &v) || v > kMaxGrid)
    return fail(CCU_ERR_NOT_IMPLEMENTED, "N * H * ceil(P / 8) must be < 2^31");
  return CCU_OK;
}

bool known_type(int32_t t) { return t == CCU_DTYPE_BF16 || t == CCU_DTYPE_FP32; }

ccu_status_t check_gated_norm(const GatedNormParams &a, bool *noop) {
  CCU_DECLINE(a.T < 0 || a.H < 0 || a.P < 0, "T, H and P must be >= 0");
  CCU_DECLINE(!known_type(a.weight_type), "unknown type %d of the weight", a.weight_type);
  CCU_DECLINE(!(a.eps >= 0.0f) || std::isinf(a.eps), "eps must be finite and >= 0");
  *noop = a.T == 0 || a.H == 0 || a.P == 0;
  if (*noop) return CCU_OK;
  CCU_DECLINE(a.x == nullptr || a.out == nullptr, "x and out must not be NULL");
  CCU_DECLINE(!aligned(a.x, 2) || !aligned(a.z, 2) || !aligned(a.out, 2), "BF16 tensors must be 2-byte aligned");
  CCU_DECLINE(!aligned(a.weight, a.weight_type == CCU_DTYPE_FP32 ? 4 : 2), "weight must be aligned to its type");
  const int64_t strides[] = {a.x_stride_t, a.x_stride_h, a.z_stride_t, a.z_stride_h, a.out_stride_t, a.out_stride_h};
  int64_t v;
  for (int64_t s : strides) {
    CCU_DECLINE(s < 0, "strides must be >= 0");
    if (!mul(a.T, s, &v) || !mul(a.H, s, &v)) return overflow();
  }
  CCU_DECLINE(a.weight_stride_h < 0, "strides must be >= 0");
  if (!mul(a.H, a.weight_stride_h, &v) || !mul(a.T, a.H, &v) || !mul(v, a.P, &v)) return overflow();
  if (a.T * a.H > kMaxGrid) return fail(CCU_ERR_NOT_IMPLEMENTED, "T * H must be < 2^31");
  return CCU_OK;
}

ccu_status_t check_residual_norm(const ResidualNormParams &a, bool *noop) {
  CCU_DECLINE(a.T < 0 || a.D < 0, "T and D must be >= 0");
  CCU_DECLINE(!known_type(a.weight_type), "unknown type %d of the weights", a.weight_type);
  CCU_DECLINE(!known_type(a.residual_type), "unknown type %d of the residual", a.residual_type);
  CCU_DECLINE(!(a.eps >= 0.0f) || std::isinf(a.eps), "eps must be finite and >= 0");
  CCU_DECLINE(!std::isfinite(a.scale), "scale must be finite");
  *noop = a.T == 0 || a.D == 0;
  if (*noop) return CCU_OK;
  CCU_DECLINE(a.x == nullptr || a.residual == nullptr || a.out == nullptr, "x, residual and out must not be NULL");
  CCU_DECLINE(!aligned(a.x, 2) || !aligned(a.out, 2), "BF16 tensors must be 2-byte aligned");
  CCU_DECLINE(!aligned(a.residual, a.residual_type == CCU_DTYPE_FP32 ? 4 : 2), "residual must be aligned to its type");
  const uintptr_t w = a.weight_type == CCU_DTYPE_FP32 ? 4 : 2;
  CCU_DECLINE(!aligned(a.weight, w) || !aligned(a.post_weight, w), "weights must be aligned to their type");
  CCU_DECLINE(a.T > 1 && (a.ld_x < 0 || a.ld_residual < a.D || a.ld_out < a.D),
              "row strides must be >= D (of x: >= 0)");
  int64_t v;
  if (a.T > 1 && (!mul(a.T, a.ld_x, &v) || !mul(a.T, a.ld_residual, &v) || !mul(a.T, a.ld_out, &v))) return overflow();
  if (!mul(a.T, a.D, &v)) return overflow();
  if (a.T > kMaxGrid) return fail(CCU_ERR_NOT_IMPLEMENTED, "T must be < 2^31");
  return CCU_OK;
}

template <typename Params>
Params with_scale(const Params &a) {
  Params p = a;
  if (p.scale == 0.0f) p.scale = (float)(1.0 / std::sqrt((double)p.K));
  return p;
}

}  // namespace
}  // namespace ccu

extern "C" {

ccu_status_t ccu_gated_delta_rule(const ccu_gated_delta_rule_args_t *args, ccu_stream_t stream) {
  ccu::record_error("");
  if (args == nullptr) return ccu::fail(CCU_ERR_INVALID_ARGUMENT, "args must not be NULL");
  bool noop = false;
  ccu_status_t st = ccu::check_rule(*args, &noop);
  if (st != CCU_OK || noop) return st;
  int route = CCU_SCAN_AUTO;
  st = ccu::choose_rule(*args, &route);
  if (st != CCU_OK) return st;
  if (route == CCU_SCAN_CHUNKED) {
    const int64_t need = ccu::delta_chunked_workspace(*args, ccu::device_sm_count());
    if (need > 0 && (args->workspace == nullptr || args->workspace_bytes < need))
      return ccu::fail(CCU_ERR_INVALID_ARGUMENT, "the delta rule needs a 16-byte aligned workspace of %lld bytes, got %lld", (long long)need,
                       (long long)(args->workspace == nullptr ? 0 : args->workspace_bytes));
  }
  const auto p = ccu::with_scale(*args);
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  return ccu::launched(route == CCU_SCAN_CHUNKED ? ccu::launch_delta_chunked(p, cs) : ccu::launch_delta_recurrent(p, cs), "gated delta rule");
}

int64_t ccu_gated_delta_rule_workspace_bytes(const ccu_gated_delta_rule_args_t *args) {
  ccu::record_error("");
  bool noop = false;
  int route = CCU_SCAN_AUTO;
  if (args == nullptr || ccu::check_rule(*args, &noop) != CCU_OK) return -1;
  if (noop) return 0;
  if (ccu::choose_rule(*args, &route) != CCU_OK) return -1;
  return route == CCU_SCAN_CHUNKED ? ccu::delta_chunked_workspace(*args, ccu::device_sm_count()) : 0;
}

int32_t ccu_gated_delta_rule_select_route(const ccu_gated_delta_rule_args_t *args) {
  ccu::record_error("");
  bool noop = false;
  int route = CCU_SCAN_AUTO;
  if (args == nullptr || ccu::check_rule(*args, &noop) != CCU_OK) return -1;
  if (noop) return CCU_SCAN_AUTO;
  return ccu::choose_rule(*args, &route) == CCU_OK ? route : -1;
}

ccu_status_t ccu_gated_delta_update(const ccu_gated_delta_update_args_t *args, ccu_stream_t stream) {
  ccu::record_error("");
  if (args == nullptr) return ccu::fail(CCU_ERR_INVALID_ARGUMENT, "args must not be NULL");
  bool noop = false;
  const ccu_status_t st = ccu::check_delta_update(*args, &noop);
  if (st != CCU_OK || noop) return st;
  return ccu::launched(ccu::launch_delta_step(ccu::with_scale(*args), reinterpret_cast<cudaStream_t>(stream)), "gated delta update");
}

int64_t ccu_gated_delta_update_workspace_bytes(int64_t N, int64_t H, int64_t P, int64_t K, int64_t G, int32_t has_conv) {
  return ccu_selective_state_update_workspace_bytes(N, H, P, K, G, has_conv);
}

ccu_status_t ccu_gated_rms_norm(const ccu_gated_rms_norm_args_t *args, ccu_stream_t stream) {
  ccu::record_error("");
  if (args == nullptr) return ccu::fail(CCU_ERR_INVALID_ARGUMENT, "args must not be NULL");
  bool noop = false;
  const ccu_status_t st = ccu::check_gated_norm(*args, &noop);
  if (st != CCU_OK || noop) return st;
  return ccu::launched(ccu::launch_gated_norm(*args, reinterpret_cast<cudaStream_t>(stream)), "gated norm");
}

ccu_status_t ccu_residual_rms_norm(const ccu_residual_rms_norm_args_t *args, ccu_stream_t stream) {
  ccu::record_error("");
  if (args == nullptr) return ccu::fail(CCU_ERR_INVALID_ARGUMENT, "args must not be NULL");
  bool noop = false;
  const ccu_status_t st = ccu::check_residual_norm(*args, &noop);
  if (st != CCU_OK || noop) return st;
  return ccu::launched(ccu::launch_residual_norm(*args, reinterpret_cast<cudaStream_t>(stream)), "residual norm");
}

}  // extern "C"
