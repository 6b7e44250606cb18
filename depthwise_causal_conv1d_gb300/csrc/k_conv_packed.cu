// Causal convolution over packed prompts (ccu_causal_conv1d_packed).
//
// Two launches: the outputs, then the states. A sequence's first W - 1 outputs read the old
// state of its slot, and any number of CTAs work on one sequence, so the state is written by a
// kernel of its own, after all of them (stream order; the launch overlaps the first kernel's
// end). One thread of it owns a (sequence, channel) and reads what it needs before it writes.
#include "ssm_internal.cuh"

namespace ccu {

int device_sm_count();

namespace {

// Sequence of row t: the last b with cu_seqlens[b] <= t whose end is past t; -1 for a row
// outside every sequence.
__device__ __forceinline__ int64_t sequence_of(const ConvPackedParams &p, int64_t t) {
  int64_t lo = 0, hi = p.B;  // cu[lo] <= t (or no sequence begins at or before t), cu[hi] > t (or hi == B)
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) >> 1;
    if (__ldg(p.cu_seqlens + mid) <= t) lo = mid; else hi = mid;
  }
  const Bounds s = sequence_bounds(p.cu_seqlens, lo, p.T);
  return t >= s.begin && t < s.end ? lo : -1;
}

// One thread per (row, channel).
template <int ACT>
__global__ void __launch_bounds__(256) k_conv_packed_scalar(ConvPackedParams p) {
  grid_dependency_boundary();
  const uint16_t *x = static_cast<const uint16_t *>(p.x), *w = static_cast<const uint16_t *>(p.weight);
  const uint16_t *bias = static_cast<const uint16_t *>(p.bias);
  const uint16_t *state = static_cast<const uint16_t *>(p.conv_state);
  uint16_t *out = static_cast<uint16_t *>(p.out);
  const int64_t total = p.T * p.D;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t t = i / p.D, d = i - t * p.D;
    const int64_t b = sequence_of(p, t);
    if (b < 0) continue;
    const int64_t begin = sequence_bounds(p.cu_seqlens, b, p.T).begin;
    const int64_t s = p.conv_state != nullptr ? slot_of(p.indices, b, p.S, p.status_dev, t == begin) : 0;
    if (s < 0) {
      out[t * p.ld_out + d] = 0;
      continue;
    }
    const bool initial = p.conv_state != nullptr && p.has_initial != nullptr && __ldg(p.has_initial + b) != 0;
    float acc = 0.0f;
    for (int64_t j = 0; j < p.W; ++j) {
      const int64_t u = t - (p.W - 1) + j - begin;  // place in the sequence
      uint16_t v = 0;
      if (u >= 0) v = x[(begin + u) * p.ld_x + d];
      else if (initial) v = state[s * p.stride_s + d * p.stride_d + (p.L + u) * p.stride_l];
      acc = __fmaf_rn(bf16_bits(v), bf16_bits(w[d * p.W + j]), acc);
    }
    if (bias != nullptr) acc += bf16_bits(bias[d]);
    out[t * p.ld_out + d] = round_bf16(activate<ACT>(acc));
  }
}

// One thread per (sequence, channel): entry l of the new state is input len - L + l of the
// sequence, or an older entry of the old state. Ascending l reads each old entry (L + u >= l,
// as len >= 0) before it is overwritten.
__global__ void __launch_bounds__(256) k_conv_packed_state(ConvPackedParams p) {
  grid_dependency_boundary();
  const uint16_t *x = static_cast<const uint16_t *>(p.x);
  const int64_t total = p.B * p.D;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t b = i / p.D, d = i - b * p.D;
    const int64_t s = slot_of(p.indices, b, p.S, p.status_dev, true);
    if (s < 0) continue;
    const Bounds q = sequence_bounds(p.cu_seqlens, b, p.T);
    const bool initial = p.has_initial != nullptr && __ldg(p.has_initial + b) != 0;
    uint16_t *st = static_cast<uint16_t *>(p.conv_state) + s * p.stride_s + d * p.stride_d;
    for (int64_t l = 0; l < p.L; ++l) {
      const int64_t u = q.end - q.begin - p.L + l;
      uint16_t v = 0;
      if (u >= 0) v = x[(q.begin + u) * p.ld_x + d];
      else if (initial) v = st[(p.L + u) * p.stride_l];
      st[l * p.stride_l] = v;
    }
  }
}

unsigned grid_for(int64_t work) {
  const int64_t blocks = (work + 255) / 256, cap = (int64_t)device_sm_count() * 16;
  return (unsigned)(blocks < cap ? (blocks > 0 ? blocks : 1) : cap);
}

}  // namespace

cudaError_t launch_conv_packed(const ConvPackedParams &p, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (p.T > 0)
    e = p.act == CCU_ACT_SILU
            ? launch_overlapped(k_conv_packed_scalar<1>, dim3(grid_for(p.T * p.D)), dim3(256), 0, stream, p)
            : launch_overlapped(k_conv_packed_scalar<0>, dim3(grid_for(p.T * p.D)), dim3(256), 0, stream, p);
  if (e == cudaSuccess && p.conv_state != nullptr)
    e = launch_overlapped(k_conv_packed_state, dim3(grid_for(p.B * p.D)), dim3(256), 0, stream, p);
  return e;
}

}  // namespace ccu
