// Products of a few rows with 4-bit weights (ccu_w4_matmul).
#include "ssm_internal.cuh"

namespace ccu {

namespace {

// One warp per (output, row of x): the lanes walk the inputs eight at a time.
__global__ void __launch_bounds__(256) k_w4_scalar(W4Params p) {
  grid_dependency_boundary();
  const int lane = threadIdx.x & 31;
  const int64_t o = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (o >= p.O) return;
  const uint32_t *q = static_cast<const uint32_t *>(p.qweight) + o * (p.I / 8);
  const uint16_t *scales = static_cast<const uint16_t *>(p.scales) + o * (p.I / p.group);
  const uint16_t *zeros = static_cast<const uint16_t *>(p.zeros);
  if (zeros != nullptr) zeros += o * (p.I / p.group);
  for (int64_t m = blockIdx.y; m < p.M; m += gridDim.y) {
    const uint16_t *x = static_cast<const uint16_t *>(p.x) + m * p.ld_x;
    float acc = 0.0f;
    for (int64_t i = lane * 8; i < p.I; i += 256) {
      const uint32_t word = __ldg(q + i / 8);
      const int64_t g = i / p.group;
      const float zero = zeros != nullptr ? bf16_bits(__ldg(zeros + g)) : 8.0f;
      float part = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        part = fmaf((float)((word >> (4 * e)) & 15u) - zero, bf16_bits(__ldg(x + i + e)), part);
      acc = fmaf(part, bf16_bits(__ldg(scales + g)), acc);
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, s);
    if (lane == 0) static_cast<uint16_t *>(p.out)[m * p.ld_out + o] = round_bf16(acc);
  }
}

}  // namespace

cudaError_t launch_w4(const W4Params &p, cudaStream_t stream) {
  const dim3 grid((unsigned)((p.O + 7) / 8), (unsigned)(p.M < 64 ? p.M : 64));
  return launch_overlapped(k_w4_scalar, grid, dim3(256), 0, stream, p);
}

}  // namespace ccu
