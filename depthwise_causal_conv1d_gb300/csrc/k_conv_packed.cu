// Causal convolution over packed prompts (ccu_causal_conv1d_packed).
//
// Two launches: the outputs, then the states. A sequence's first W - 1 outputs read the old
// state of its slot, and any number of CTAs work on one sequence, so the state is written by a
// kernel of its own, after all of them (stream order; the launch overlaps the first kernel's
// end). One thread of it owns a (sequence, channel) and reads what it needs before it writes.
//
// The outputs move 4 bytes an element and do nine operations on it: bound by HBM.
#include "ssm_internal.cuh"

namespace ccu {

int device_sm_count();

namespace {

// Sequence of row t: the last b with cu_seqlens[b] <= t. (The caller checks that t is inside it:
// a row before the first sequence or past the last one is in none.)
__device__ __forceinline__ int64_t sequence_at(const ConvPackedParams &p, int64_t t) {
  int64_t lo = 0, hi = p.B;
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) >> 1;
    if (__ldg(p.cu_seqlens + mid) <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// One thread per (row, channel): any D and any alignment.
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
    const int64_t b = sequence_at(p, t);
    const Bounds q = sequence_bounds(p.cu_seqlens, b, p.T);
    if (t < q.begin || t >= q.end) continue;
    const int64_t s = p.conv_state != nullptr ? slot_of(p.indices, b, p.S, p.status_dev, t == q.begin) : 0;
    if (s < 0) {
      out[t * p.ld_out + d] = 0;
      continue;
    }
    const bool initial = p.conv_state != nullptr && p.has_initial != nullptr && __ldg(p.has_initial + b) != 0;
    float acc = 0.0f;
    for (int64_t j = 0; j < p.W; ++j) {
      const int64_t u = t - (p.W - 1) + j - q.begin;  // place in the sequence
      uint16_t v = 0;
      if (u >= 0) v = x[(q.begin + u) * p.ld_x + d];
      else if (initial) v = state[s * p.stride_s + d * p.stride_d + (p.L + u) * p.stride_l];
      acc = __fmaf_rn(bf16_bits(v), bf16_bits(w[d * p.W + j]), acc);
    }
    if (bias != nullptr) acc += bf16_bits(bias[d]);
    out[t * p.ld_out + d] = round_bf16(activate<ACT>(acc));
  }
}

// A thread owns 8 channels and walks a run of kRun rows with the window in registers, kAhead
// rows' 16-byte loads in flight. A run may cross sequences: at a sequence's first row the
// window is filled from its slot (or zeroed), and a run that starts inside a sequence reads the
// rows before it, or the slot for those before the sequence. Halo: W - 1 rows of kRun.
// 32672 rows of 4352 channels: 125 us, 4.5 TB/s at 4 bytes an element (16 rows 139, 64 rows 124, 128 rows 132;
// 16 rows ahead 146, 4 ahead 128). Runs of 32 leave more threads than 64 to a single prompt.
constexpr int kRun = 32;
constexpr int kAhead = 8;

// Inputs of 8 channels at place u (may be negative) of the sequence that begins at row `begin`.
__device__ __forceinline__ uint4 input8(const ConvPackedParams &p, int64_t begin, int64_t u, int64_t slot, bool initial,
                                        int64_t c0) {
  if (u >= 0) return ld_keep(static_cast<const uint16_t *>(p.x) + (begin + u) * p.ld_x + c0);
  if (!initial) return make_uint4(0, 0, 0, 0);
  const uint16_t *st = static_cast<const uint16_t *>(p.conv_state) + slot * p.stride_s + (p.L + u) * p.stride_l;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = st[(c0 + 2 * i) * p.stride_d] | ((uint32_t)st[(c0 + 2 * i + 1) * p.stride_d] << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int ACT, int W>
__global__ void __launch_bounds__(128) k_conv_packed_vector(ConvPackedParams p, int64_t groups) {
  grid_dependency_boundary();
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, run = i / groups, g = i - run * groups;
  const int64_t c0 = g * 8;
  const int64_t first = run * kRun;
  if (first >= p.T) return;
  const int64_t last = first + kRun < p.T ? first + kRun : p.T;
  float2 wf[kW][4], bf[4] = {};
  load_weights_f<W>(static_cast<const uint16_t *>(p.weight), c0, wf);
  const bool has_bias = p.bias != nullptr;
  if (has_bias) widen8(ld_keep(static_cast<const uint16_t *>(p.bias) + c0), bf);
  const uint16_t *x = static_cast<const uint16_t *>(p.x) + c0;
  uint16_t *out = static_cast<uint16_t *>(p.out) + c0;
  int64_t b = sequence_at(p, first);
  int64_t t = first;
  while (t < last && b < p.B) {
    const Bounds q = sequence_bounds(p.cu_seqlens, b, p.T);
    if (q.begin > t) t = q.begin;  // rows of no sequence
    const int64_t end = q.end < last ? q.end : last;
    if (t >= end) {
      ++b;
      continue;
    }
    const int64_t s = p.conv_state != nullptr ? slot_of(p.indices, b, p.S, p.status_dev, t == q.begin && g == 0) : 0;
    if (s < 0) {
      for (; t < end; ++t) st_stream(out + t * p.ld_out, make_uint4(0, 0, 0, 0));
      ++b;
      continue;
    }
    const bool initial = p.conv_state != nullptr && p.has_initial != nullptr && __ldg(p.has_initial + b) != 0;
    float2 h0[4] = {}, h1[4] = {}, h2[4];
    if (W >= 4) widen8(input8(p, q.begin, t - q.begin - 3, s, initial, c0), h0);
    if (W >= 3) widen8(input8(p, q.begin, t - q.begin - 2, s, initial, c0), h1);
    widen8(input8(p, q.begin, t - q.begin - 1, s, initial, c0), h2);
    for (; t < end; t += kAhead) {
      uint4 v[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (t + i < end) v[i] = ld_stream(x + (t + i) * p.ld_x);
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (t + i < end) {
          float2 xf[4];
          widen8(v[i], xf);
          st_stream(out + (t + i) * p.ld_out, outputs8f<ACT, W>(wf, bf, has_bias, h0, h1, h2, xf));
          slide(h0, h1, h2, xf);
        }
    }
    t = end;
    ++b;
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

bool on16(const void *v) { return reinterpret_cast<uintptr_t>(v) % 16 == 0; }

template <int ACT>
cudaError_t launch_outputs(const ConvPackedParams &p, cudaStream_t stream) {
  const int64_t runs = (p.T + kRun - 1) / kRun;
  const bool rows = p.T == 1 || (p.ld_x % 8 == 0 && p.ld_out % 8 == 0);
  const int64_t groups = p.D / 8, blocks = (runs * groups + 127) / 128;
  if (p.D % 8 == 0 && rows && on16(p.x) && on16(p.weight) && on16(p.bias) && on16(p.out) && blocks <= INT32_MAX) {
    const dim3 grid((unsigned)blocks);  // (run, channels) in a row: no lane idles at the end of the channels
    if (p.W == 4) return launch_overlapped(k_conv_packed_vector<ACT, 4>, grid, dim3(128), 0, stream, p, groups);
    if (p.W == 3) return launch_overlapped(k_conv_packed_vector<ACT, 3>, grid, dim3(128), 0, stream, p, groups);
    return launch_overlapped(k_conv_packed_vector<ACT, 2>, grid, dim3(128), 0, stream, p, groups);
  }
  return launch_overlapped(k_conv_packed_scalar<ACT>, dim3(grid_for(p.T * p.D)), dim3(256), 0, stream, p);
}

}  // namespace

cudaError_t launch_conv_packed(const ConvPackedParams &p, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (p.T > 0) e = p.act == CCU_ACT_SILU ? launch_outputs<1>(p, stream) : launch_outputs<0>(p, stream);
  if (e == cudaSuccess && p.conv_state != nullptr)
    e = launch_overlapped(k_conv_packed_state, dim3(grid_for(p.B * p.D)), dim3(256), 0, stream, p);
  return e;
}

}  // namespace ccu
