// What the kernels of the state-space operators share (ccu_ssm.h): the arguments as the
// kernels take them, the device helpers, and the launchers.
#pragma once

#include "ccu_internal.cuh"
#include "ccu_ssm.h"

namespace ccu {

using ConvPackedParams = ccu_conv1d_packed_args_t;
using ScanParams = ccu_selective_scan_args_t;
using StepParams = ccu_selective_state_update_args_t;
using W4Params = ccu_w4_matmul_args_t;

// Most states a channel the register-resident kernels hold.
constexpr int64_t kMaxStates = 256;

// softplus(v) = max(v, 0) + log1p(exp(-|v|)): the exponential never overflows, and small
// results (v << 0, where steps live) keep their relative accuracy. Two library functions
// per token and head, shared by its P * K states.
__device__ __forceinline__ float softplus(float v) { return fmaxf(v, 0.0f) + log1pf(expf(-fabsf(v))); }

// The step of a token from dt + bias. A NaN stays one (fmaxf would drop it).
__device__ __forceinline__ float step_of(float v, int softplus_on) { return softplus_on && v == v ? softplus(v) : v; }

__device__ __forceinline__ float step_size(uint16_t dt, const float *bias, int64_t h, int softplus_on) {
  float v = bf16_bits(dt);
  if (bias != nullptr) v += __ldg(bias + h);
  return step_of(v, softplus_on);
}

// Sequence bounds from cu_seqlens, clamped so that no value can reach outside the T rows.
struct Bounds {
  int64_t begin, end;
};
__device__ __forceinline__ Bounds sequence_bounds(const int32_t *cu, int64_t b, int64_t T) {
  int64_t s = __ldg(cu + b), e = __ldg(cu + b + 1);
  s = s < 0 ? 0 : (s > T ? T : s);
  e = e < s ? s : (e > T ? T : e);
  return {s, e};
}

// Slot of sequence (row) i, or -1: padding, or out of range (reported when `report`).
__device__ __forceinline__ int64_t slot_of(const int32_t *indices, int64_t i, int64_t S, int32_t *status, bool report) {
  if (indices == nullptr) return i;
  const int64_t s = __ldg(indices + i);
  if (s >= -1 && s < S) return s;
  if (report && status != nullptr) atomicOr(status, CCU_DEVERR_RANGE);
  return -1;
}

// Sums each of v[0..7] over groups of LANES lanes (8, 16 or 32) of a warp; a lane gets the sum
// of v[its place in the group / (LANES / 8)]. Every round sends half of what a lane still holds to
// the partner that keeps it: 4 + 2 + 1 exchanges, then one a round, instead of 8 a round.
template <int LANES>
__device__ __forceinline__ float sum8_over(const float (&v)[8], int lane) {
  const unsigned full = 0xffffffffu;
  float a[4], b[2], c;
  const bool h1 = lane & (LANES / 2), h2 = lane & (LANES / 4), h3 = lane & (LANES / 8);
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = (h1 ? v[i + 4] : v[i]) + __shfl_xor_sync(full, h1 ? v[i] : v[i + 4], LANES / 2);
#pragma unroll
  for (int i = 0; i < 2; ++i) b[i] = (h2 ? a[i + 2] : a[i]) + __shfl_xor_sync(full, h2 ? a[i] : a[i + 2], LANES / 4);
  c = (h3 ? b[1] : b[0]) + __shfl_xor_sync(full, h3 ? b[0] : b[1], LANES / 8);
#pragma unroll
  for (int o = LANES / 16; o > 0; o >>= 1) c += __shfl_xor_sync(full, c, o);
  return c;
}

// Clusters of CTAs: a barrier over the cluster, and a float of CTA `rank`'s shared memory at the
// place that p has in this CTA's.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ float cluster_load(const float *p, int rank) {
  uint32_t at;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}

// launch_overlapped with clusters of `cluster` CTAs along x (the grid a multiple of it).
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, int cluster, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)cluster, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

cudaError_t launch_conv_packed(const ConvPackedParams &p, cudaStream_t stream);
cudaError_t launch_scan_recurrent(const ScanParams &p, cudaStream_t stream);
// Chunks of 128 tokens on the tensor cores; what it serves is checked in ssm_api.cu.
constexpr int64_t kChunkMaxStates = 128;
cudaError_t launch_scan_chunked(const ScanParams &p, cudaStream_t stream);
// Bytes of workspace it needs on a device of so many SMs (for sizes that do not overflow).
int64_t scan_chunked_workspace(const ScanParams &p, int sms);
cudaError_t launch_step(const StepParams &p, cudaStream_t stream);
cudaError_t launch_w4(const W4Params &p, cudaStream_t stream);

}  // namespace ccu
