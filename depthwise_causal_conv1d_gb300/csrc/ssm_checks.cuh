// Argument checks that the entry points of the state-space operators share (ssm_api.cu, delta_api.cu): typed
// declines with a message, sizes whose products stay in 64 bits.
#pragma once

#include <cstdarg>
#include <cstdio>

#include "ssm_internal.cuh"

namespace ccu {
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

// Sizes and heads that prompts and single tokens share.
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

ccu_status_t launched(cudaError_t e, const char *what) {
  if (e == cudaSuccess) return CCU_OK;
  return fail(CCU_ERR_CUDA, "launch of the %s failed: %s", what, cudaGetErrorString(e));
}

}  // namespace
}  // namespace ccu
