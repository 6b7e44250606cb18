// C-ABI entry points of the state-space operators: argument checks (typed declines) and kernel
// choice. Declines follow the rules of the convolution's entry points (api.cu).
#include <cstdarg>
#include <cstdio>

#include "ssm_internal.cuh"

namespace ccu {

int device_sm_count();

namespace {

ccu_status_t fail(ccu_status_t st, const char *fmt, ...) {
  char msg[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof msg, fmt, ap);
  va_end(ap);
  record_error(msg);
  return st;
}

bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

constexpr int64_t kLimit = INT64_MAX / 16;      // elements: byte offsets stay in 64 bits
constexpr int64_t kMaxGrid = INT32_MAX;         // CTAs along the grid's x axis

// a * b <= kLimit (and sets *out), for a, b >= 0.
bool mul(int64_t a, int64_t b, int64_t *out) {
  if (a != 0 && b > kLimit / a) return false;
  *out = a * b;
  return true;
}

#define CCU_DECLINE(cond, ...) \
  if (cond) return fail(CCU_ERR_INVALID_ARGUMENT, __VA_ARGS__)

ccu_status_t overflow() { return fail(CCU_ERR_INVALID_ARGUMENT, "tensor sizes overflow 64-bit indexing"); }

ccu_status_t check_conv_packed(const ConvPackedParams &a, bool *noop) {
  CCU_DECLINE(a.act != CCU_ACT_IDENTITY && a.act != CCU_ACT_SILU,
              "act must be CCU_ACT_IDENTITY or CCU_ACT_SILU, got %d", a.act);
  CCU_DECLINE(a.T < 0 || a.B < 0 || a.D < 0 || a.S < 0, "T, B, D and S must be >= 0");
  CCU_DECLINE(a.W < 1, "W must be >= 1, got %lld", (long long)a.W);
  if (a.W < 2 || a.W > kW) return fail(CCU_ERR_NOT_IMPLEMENTED, "widths 2 to 4 are served, got %lld", (long long)a.W);
  if (a.T > INT32_MAX) return fail(CCU_ERR_NOT_IMPLEMENTED, "T < 2^31 rows are served");
  *noop = a.D == 0 || a.B == 0 || (a.T == 0 && a.conv_state == nullptr);
  if (*noop) return CCU_OK;
  CCU_DECLINE(a.cu_seqlens == nullptr, "cu_seqlens must not be NULL");
  CCU_DECLINE(a.weight == nullptr || (a.T > 0 && (a.x == nullptr || a.out == nullptr)), "x, weight and out must not be NULL");
  CCU_DECLINE(!aligned(a.x, 2) || !aligned(a.weight, 2) || !aligned(a.bias, 2) || !aligned(a.out, 2) || !aligned(a.conv_state, 2),
              "BF16 tensors must be 2-byte aligned");
  CCU_DECLINE(!aligned(a.cu_seqlens, 4) || !aligned(a.indices, 4) || !aligned(a.has_initial, 4) || !aligned(a.status_dev, 4),
              "int32 tensors must be 4-byte aligned");
  CCU_DECLINE(a.T > 1 && (a.ld_x < a.D || a.ld_out < a.D), "row strides must be >= D");
  CCU_DECLINE(a.conv_state == nullptr && (a.indices != nullptr || a.has_initial != nullptr),
              "indices and has_initial need a conv_state");
  int64_t v;
  if (!mul(a.T, a.ld_x < a.D ? a.D : a.ld_x, &v) || !mul(a.T, a.ld_out < a.D ? a.D : a.ld_out, &v) || !mul(a.B, a.D, &v) ||
      !mul(a.D, a.W, &v))
    return overflow();
  if (a.conv_state != nullptr) {
    CCU_DECLINE(a.L < a.W - 1, "L must be >= W - 1 (L=%lld, W=%lld)", (long long)a.L, (long long)a.W);
    CCU_DECLINE(a.stride_s < 0 || a.stride_d < 0 || a.stride_l < 0, "strides must be >= 0");
    CCU_DECLINE(a.indices == nullptr && a.S < a.B,
                "without indices sequence b uses slot b, so S must be >= B (S=%lld, B=%lld)", (long long)a.S, (long long)a.B);
    int64_t s, d, l;
    if (!mul(a.S, a.stride_s, &s) || !mul(a.D, a.stride_d, &d) || !mul(a.L, a.stride_l, &l)) return overflow();
  }
  return CCU_OK;
}

// Sizes and heads that the scan and the update share.
ccu_status_t check_heads(int64_t H, int64_t P, int64_t K, int64_t G, int64_t S) {
  CCU_DECLINE(H < 0 || P < 0 || K < 0 || G < 0 || S < 0, "sizes must be >= 0");
  CCU_DECLINE(G < 1 || H % G != 0, "H must be a multiple of G >= 1 (H=%lld, G=%lld)", (long long)H, (long long)G);
  CCU_DECLINE(K < 1, "K must be >= 1");
  if (K > kMaxStates) return fail(CCU_ERR_NOT_IMPLEMENTED, "K <= %lld states are served, got %lld", (long long)kMaxStates, (long long)K);
  int64_t v;
  if (!mul(H, P, &v) || !mul(v, K, &v) || !mul(S, v, &v) || !mul(G, K, &v)) return overflow();
  return CCU_OK;
}

ccu_status_t check_state(const float *state, int64_t stride_s, int64_t inner, int64_t S) {
  CCU_DECLINE(state == nullptr && S > 0, "state must not be NULL");
  CCU_DECLINE(!aligned(state, 4), "FP32 tensors must be 4-byte aligned");
  CCU_DECLINE(S > 1 && stride_s < inner, "slots must not overlap: state_stride_s must be >= H * P * K");
  int64_t v;
  if (!mul(S, stride_s < inner ? inner : stride_s, &v)) return overflow();
  return CCU_OK;
}

ccu_status_t check_scan(const ScanParams &a, bool *noop) {
  ccu_status_t st = check_heads(a.H, a.P, a.K, a.G, a.S);
  if (st != CCU_OK) return st;
  CCU_DECLINE(a.T < 0 || a.n_seq < 0, "T and n_seq must be >= 0");
  CCU_DECLINE(a.route < 0 || a.route >= CCU_SCAN_ROUTE_COUNT, "unknown route %d", a.route);
  if (a.T > INT32_MAX) return fail(CCU_ERR_NOT_IMPLEMENTED, "T < 2^31 rows are served");
  *noop = a.n_seq == 0 || a.H == 0 || a.P == 0;
  if (*noop) return CCU_OK;
  CCU_DECLINE(a.cu_seqlens == nullptr, "cu_seqlens must not be NULL");
  CCU_DECLINE(a.A == nullptr, "A must not be NULL");
  CCU_DECLINE(a.T > 0 && (a.x == nullptr || a.dt == nullptr || a.b == nullptr || a.c == nullptr || a.out == nullptr),
              "x, dt, B, C and out must not be NULL");
  CCU_DECLINE(!aligned(a.x, 2) || !aligned(a.dt, 2) || !aligned(a.b, 2) || !aligned(a.c, 2) || !aligned(a.z, 2) || !aligned(a.out, 2),
              "BF16 tensors must be 2-byte aligned");
  CCU_DECLINE(!aligned(a.A, 4) || !aligned(a.D, 4) || !aligned(a.dt_bias, 4), "FP32 tensors must be 4-byte aligned");
  CCU_DECLINE(!aligned(a.cu_seqlens, 4) || !aligned(a.indices, 4) || !aligned(a.has_initial, 4) || !aligned(a.status_dev, 4),
              "int32 tensors must be 4-byte aligned");
  CCU_DECLINE(!aligned(a.workspace, 16), "workspace must be 16-byte aligned");
  const int64_t strides[] = {a.x_stride_t, a.x_stride_h, a.dt_stride_t, a.b_stride_t, a.b_stride_g, a.c_stride_t, a.c_stride_g,
                             a.z_stride_t, a.z_stride_h, a.out_stride_t, a.out_stride_h};
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
bool chunked_serves(const ScanParams &a) {
  if (a.P % 8 != 0 || a.K % 8 != 0 || a.K > kChunkMaxStates) return false;
  const void *rows[] = {a.x, a.b, a.c, a.z, a.out};
  for (const void *v : rows)
    if (!aligned(v, 16)) return false;
  const int64_t strides[] = {a.x_stride_t, a.x_stride_h, a.b_stride_t, a.b_stride_g, a.c_stride_t, a.c_stride_g,
                             a.z_stride_t, a.z_stride_h, a.out_stride_t, a.out_stride_h};
  for (int64_t v : strides)
    if (v % 8 != 0) return false;
  // What a tensor map describes: real strides (no row or head shared by a stride of 0) below 2^40 bytes.
  const bool gated = a.z != nullptr;
  const int64_t steps[][2] = {{a.x_stride_t, a.T}, {a.x_stride_h, a.H}, {a.b_stride_t, a.T}, {a.b_stride_g, a.G}, {a.c_stride_t, a.T},
                              {a.c_stride_g, a.G}, {a.z_stride_t, gated ? a.T : 0}, {a.z_stride_h, gated ? a.H : 0}};
  for (const auto &v : steps)
    if (v[1] > 1 && (v[0] < 8 || v[0] >= (int64_t(1) << 39))) return false;
  return a.H <= INT32_MAX && a.P <= INT32_MAX;
}

// From this many tokens a sequence (on average: the lengths are on the device) AUTO takes the
// chunked kernel. A chunk costs the same however few tokens it holds: 64 heads x 64 channels x 128 states, token
// by token against chunked, 14 tokens a sequence: 1 sequence 12.6 us against 10.7, 16 sequences 56 against 71, 128 sequences 513 against
// 532; 16 tokens: 14.0 / 10.6, 63 / 71, 610 / 532. 48 heads x 128 channels x 64 states: 15.6 / 11.1, 60 / 106, 554 / 790 at 16 tokens,
// even at 11, 30 and 24.
constexpr int64_t kChunkedMinTokens = 16;

ccu_status_t choose_scan(const ScanParams &a, int *route) {
  if (a.route == CCU_SCAN_CHUNKED && !chunked_serves(a))
    return fail(CCU_ERR_NOT_IMPLEMENTED,
                "the chunked scan needs P and K in multiples of 8, K <= %lld, and rows on 16-byte boundaries",
                (long long)kChunkMaxStates);
  if (a.route != CCU_SCAN_AUTO) *route = a.route;
  else *route = chunked_serves(a) && a.T / kChunkedMinTokens >= a.n_seq ? CCU_SCAN_CHUNKED : CCU_SCAN_RECURRENT;
  return CCU_OK;
}

ccu_status_t check_update(const StepParams &a, bool *noop) {
  ccu_status_t st = check_heads(a.H, a.P, a.K, a.G, a.S);
  if (st != CCU_OK) return st;
  CCU_DECLINE(a.N < 0, "N must be >= 0");
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
  CCU_DECLINE(a.xbc == nullptr || a.dt == nullptr || a.A == nullptr || a.out == nullptr, "xbc, dt, A and out must not be NULL");
  CCU_DECLINE(!aligned(a.xbc, 2) || !aligned(a.conv_weight, 2) || !aligned(a.conv_bias, 2) || !aligned(a.conv_state, 2) ||
                  !aligned(a.dt, 2) || !aligned(a.z, 2) || !aligned(a.out, 2),
              "BF16 tensors must be 2-byte aligned");
  CCU_DECLINE(!aligned(a.A, 4) || !aligned(a.D, 4) || !aligned(a.dt_bias, 4), "FP32 tensors must be 4-byte aligned");
  CCU_DECLINE(!aligned(a.indices, 4) || !aligned(a.status_dev, 4), "int32 tensors must be 4-byte aligned");
  const int64_t channels = a.H * a.P + 2 * a.G * a.K;
  CCU_DECLINE(a.N > 1 && a.ld_xbc < channels, "ld_xbc must be >= H*P + 2*G*K");
  const int64_t strides[] = {a.ld_xbc, a.dt_stride_n, a.z_stride_n, a.z_stride_h, a.out_stride_n, a.out_stride_h};
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
                "the convolution needs a 16-byte aligned workspace of 4 * N * (H*P + 2*G*K) = %lld bytes, got %lld",
                (long long)(4 * a.N * channels), (long long)a.workspace_bytes);
  }
  if (!mul(a.N, a.H, &v) || !mul(v, (a.P + 7) / 8, &v) || v > kMaxGrid)
    return fail(CCU_ERR_NOT_IMPLEMENTED, "N * H * ceil(P / 8) must be < 2^31");
  return CCU_OK;
}

ccu_status_t check_w4(const W4Params &a, bool *noop) {
  CCU_DECLINE(a.M < 0 || a.I < 0 || a.O < 0, "M, I and O must be >= 0");
  CCU_DECLINE(a.group < 1, "group must be >= 1");
  if (a.group != 32 && a.group != 64 && a.group != 128)
    return fail(CCU_ERR_NOT_IMPLEMENTED, "groups of 32, 64 and 128 are served, got %lld", (long long)a.group);
  CCU_DECLINE(a.I % a.group != 0, "I must be a multiple of group (I=%lld, group=%lld)", (long long)a.I, (long long)a.group);
  *noop = a.M == 0 || a.O == 0;
  if (*noop) return CCU_OK;
  CCU_DECLINE(a.out == nullptr || (a.I > 0 && (a.x == nullptr || a.qweight == nullptr || a.scales == nullptr)),
              "x, qweight, scales and out must not be NULL");
  CCU_DECLINE(!aligned(a.x, 2) || !aligned(a.scales, 2) || !aligned(a.zeros, 2) || !aligned(a.out, 2),
              "BF16 tensors must be 2-byte aligned");
  CCU_DECLINE(!aligned(a.qweight, 4), "qweight must be 4-byte aligned");
  CCU_DECLINE(a.M > 1 && (a.ld_x < a.I || a.ld_out < a.O), "row strides must be >= I and >= O");
  int64_t v;
  if (!mul(a.O, a.I, &v) || !mul(a.M, a.ld_x < a.I ? a.I : a.ld_x, &v) || !mul(a.M, a.ld_out < a.O ? a.O : a.ld_out, &v))
    return overflow();
  if ((a.O + 7) / 8 > kMaxGrid) return fail(CCU_ERR_NOT_IMPLEMENTED, "O < 2^34 outputs are served");
  return CCU_OK;
}

ccu_status_t launched(cudaError_t e, const char *what) {
  if (e == cudaSuccess) return CCU_OK;
  return fail(CCU_ERR_CUDA, "launch of the %s failed: %s", what, cudaGetErrorString(e));
}

}  // namespace
}  // namespace ccu

extern "C" {

ccu_status_t ccu_causal_conv1d_packed(const ccu_conv1d_packed_args_t *args, ccu_stream_t stream) {
  ccu::record_error("");
  if (args == nullptr) return ccu::fail(CCU_ERR_INVALID_ARGUMENT, "args must not be NULL");
  bool noop = false;
  const ccu_status_t st = ccu::check_conv_packed(*args, &noop);
  if (st != CCU_OK || noop) return st;
  return ccu::launched(ccu::launch_conv_packed(*args, reinterpret_cast<cudaStream_t>(stream)), "packed convolution");
}

ccu_status_t ccu_selective_scan(const ccu_selective_scan_args_t *args, ccu_stream_t stream) {
  ccu::record_error("");
  if (args == nullptr) return ccu::fail(CCU_ERR_INVALID_ARGUMENT, "args must not be NULL");
  bool noop = false;
  ccu_status_t st = ccu::check_scan(*args, &noop);
  if (st != CCU_OK || noop) return st;
  int route = CCU_SCAN_AUTO;
  st = ccu::choose_scan(*args, &route);
  if (st != CCU_OK) return st;
  if (route == CCU_SCAN_CHUNKED) {
    const int64_t need = ccu::scan_chunked_workspace(*args, ccu::device_sm_count());
    if (need > 0 && (args->workspace == nullptr || args->workspace_bytes < need))
      return ccu::fail(CCU_ERR_INVALID_ARGUMENT, "the scan needs a 16-byte aligned workspace of %lld bytes, got %lld", (long long)need,
                       (long long)(args->workspace == nullptr ? 0 : args->workspace_bytes));
  }
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  return ccu::launched(route == CCU_SCAN_CHUNKED ? ccu::launch_scan_chunked(*args, cs) : ccu::launch_scan_recurrent(*args, cs),
                       "selective scan");
}

int64_t ccu_selective_scan_workspace_bytes(const ccu_selective_scan_args_t *args) {
  ccu::record_error("");
  bool noop = false;
  int route = CCU_SCAN_AUTO;
  if (args == nullptr || ccu::check_scan(*args, &noop) != CCU_OK) return -1;
  if (noop) return 0;
  if (ccu::choose_scan(*args, &route) != CCU_OK) return -1;
  return route == CCU_SCAN_CHUNKED ? ccu::scan_chunked_workspace(*args, ccu::device_sm_count()) : 0;
}

int32_t ccu_selective_scan_select_route(const ccu_selective_scan_args_t *args) {
  ccu::record_error("");
  bool noop = false;
  int route = CCU_SCAN_AUTO;
  if (args == nullptr || ccu::check_scan(*args, &noop) != CCU_OK) return -1;
  if (noop) return CCU_SCAN_AUTO;
  return ccu::choose_scan(*args, &route) == CCU_OK ? route : -1;
}

ccu_status_t ccu_selective_state_update(const ccu_selective_state_update_args_t *args, ccu_stream_t stream) {
  ccu::record_error("");
  if (args == nullptr) return ccu::fail(CCU_ERR_INVALID_ARGUMENT, "args must not be NULL");
  bool noop = false;
  const ccu_status_t st = ccu::check_update(*args, &noop);
  if (st != CCU_OK || noop) return st;
  return ccu::launched(ccu::launch_step(*args, reinterpret_cast<cudaStream_t>(stream)), "selective state update");
}

int64_t ccu_selective_state_update_workspace_bytes(int64_t N, int64_t H, int64_t P, int64_t K, int64_t G,
                                                   int32_t has_conv) {
  ccu::record_error("");
  int64_t inner, bc, v;
  if (N < 0 || H < 0 || P < 0 || K < 0 || G < 0 || !ccu::mul(H, P, &inner) || !ccu::mul(G, K, &bc) ||
      !ccu::mul(N, inner + 2 * bc, &v))
    return -1;
  return has_conv ? 4 * v : 0;
}

ccu_status_t ccu_w4_matmul(const ccu_w4_matmul_args_t *args, ccu_stream_t stream) {
  ccu::record_error("");
  if (args == nullptr) return ccu::fail(CCU_ERR_INVALID_ARGUMENT, "args must not be NULL");
  bool noop = false;
  const ccu_status_t st = ccu::check_w4(*args, &noop);
  if (st != CCU_OK || noop) return st;
  return ccu::launched(ccu::launch_w4(*args, reinterpret_cast<cudaStream_t>(stream)), "4-bit product");
}

}  // extern "C"
