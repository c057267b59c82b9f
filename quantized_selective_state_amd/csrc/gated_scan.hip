// Gated linear recurrence h_t = a_t h_{t-1} + b_t with a gate per channel, its gradient and its
// single-token step (Ternary Mamba, Section 1, states the recurrence).
#include "gated_types.h"

namespace ssdq {
namespace {

constexpr int kBlock = SSDQ_CHECKPOINT_BLOCK;

__device__ __forceinline__ void sequence_rows(const GatedArgs& g, int s, int64_t& first, int64_t& last) {
  if (g.offsets == nullptr) {
    const int64_t len = g.tokens / g.sequences;
    first = s * len;
    last = first + len;
    return;
  }
  // whatever the offsets hold, the rows stay inside the tensors
  first = min(max(int64_t(g.offsets[s]), int64_t(0)), g.tokens);
  last = min(max(int64_t(g.offsets[s + 1]), first), g.tokens);
}

// One thread per (sequence, channel), one wave per checkpoint block, tokens in order.
template <typename T, int KIND>
__global__ void __launch_bounds__(64) gated_scan_kernel(GatedArgs g) {
  const int blocks = (g.channels + kBlock - 1) / kBlock;
  const int s = int(blockIdx.x / unsigned(blocks)), blk = int(blockIdx.x % unsigned(blocks));
  const int c = blk * kBlock + int(threadIdx.x);
  const bool in = c < g.channels;
  int64_t first, last;
  sequence_rows(g, s, first, last);
  float h = in && g.h0 ? g.h0[int64_t(s) * g.channels + c] : 0.f;
  for (int64_t t = first; t < last; ++t) {
    float seen = 0.f;
    const int64_t at = t * g.channels + c;
    if (in) {
      float a, m;
      gate_terms<KIND>(to_f32(static_cast<const T*>(g.gate)[at]), a, m);
      const float u = to_f32(static_cast<const T*>(g.u)[at]);
      h = fmaf(a, h, KIND == SSDQ_GATE_LOG ? u : m * u);
      const T r = from_f32<T>(h);
      static_cast<T*>(g.h)[at] = r;
      seen = to_f32(r);
    }
    if (g.codes) {
      uint32_t most = __float_as_uint(fabsf(seen));
#pragma unroll
      for (int o = 32; o >= 1; o >>= 1) most = max(most, uint32_t(__shfl_xor(int(most), o, 64)));
      const float sc = checkpoint_scale(most);
      if (in) g.codes[at] = int8_t(code_of(seen, code_scale(sc)));
      if (threadIdx.x == 0) g.scale[t * blocks + blk] = sc;
    }
  }
  if (in && g.h_final) g.h_final[int64_t(s) * g.channels + c] = h;
}

template <typename T, int KIND>
__global__ void __launch_bounds__(64) gated_backward_kernel(GatedArgs g) {
  const int blocks = (g.channels + kBlock - 1) / kBlock;
  const int s = int(blockIdx.x / unsigned(blocks)), blk = int(blockIdx.x % unsigned(blocks));
  const int c = blk * kBlock + int(threadIdx.x);
  if (c >= g.channels) return;
  int64_t first, last;
  sequence_rows(g, s, first, last);
  const int64_t sc = int64_t(s) * g.channels + c;
  float k = g.dh_final ? g.dh_final[sc] : 0.f;
  const float h0 = g.h0 ? g.h0[sc] : 0.f;
  for (int64_t t = last - 1; t >= first; --t) {
    const int64_t at = t * g.channels + c;
    float a, m, before;
    gate_terms<KIND>(to_f32(static_cast<const T*>(g.gate)[at]), a, m);
    if (t == first) before = h0;
    else if (g.codes) before = float(g.codes[at - g.channels]) * g.scale[(t - 1) * blocks + blk];
    else before = to_f32(static_cast<const T*>(g.h)[at - g.channels]);
    const float d = to_f32(static_cast<const T*>(g.dh)[at]) + k;
    k = a * d;
    float dg, du;
    if (KIND == SSDQ_GATE_LOG) {
      dg = k * before;
      du = d;
    } else {
      dg = k * m * (before - to_f32(static_cast<const T*>(g.u)[at]));
      du = m * d;
    }
    static_cast<T*>(g.dgate)[at] = from_f32<T>(dg);
    static_cast<T*>(g.du)[at] = from_f32<T>(du);
  }
  if (g.dh0) g.dh0[sc] = k;
}

template <typename T, int KIND>
__global__ void __launch_bounds__(256) gated_step_kernel(float* state, const T* gate, const T* u, T* h, int64_t n) {
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) {
    float a, m;
    gate_terms<KIND>(to_f32(gate[i]), a, m);
    const float v = to_f32(u[i]);
    const float s = fmaf(a, state[i], KIND == SSDQ_GATE_LOG ? v : m * v);
    state[i] = s;
    h[i] = from_f32<T>(s);
  }
}

// f(T, KIND) for the runtime dtype and gate kind
template <template <typename, int> class F, typename... A>
hipError_t dispatch(int32_t dtype, int32_t kind, A... args) {
  const bool log = kind == SSDQ_GATE_LOG;
  switch (dtype) {
    case SSDQ_DTYPE_F32: return log ? F<float, SSDQ_GATE_LOG>::run(args...) : F<float, SSDQ_GATE_LOGIT>::run(args...);
    case SSDQ_DTYPE_F16:
      return log ? F<_Float16, SSDQ_GATE_LOG>::run(args...) : F<_Float16, SSDQ_GATE_LOGIT>::run(args...);
    default: return log ? F<__bf16, SSDQ_GATE_LOG>::run(args...) : F<__bf16, SSDQ_GATE_LOGIT>::run(args...);
  }
}

template <typename T, int KIND>
struct Forward {
  static hipError_t run(const GatedArgs* g, hipStream_t stream) {
    const int blocks = (g->channels + kBlock - 1) / kBlock;
    hipLaunchKernelGGL((gated_scan_kernel<T, KIND>), dim3(uint32_t(g->sequences * int64_t(blocks))), dim3(64), 0, stream, *g);
    return hipGetLastError();
  }
};
template <typename T, int KIND>
struct Backward {
  static hipError_t run(const GatedArgs* g, hipStream_t stream) {
    const int blocks = (g->channels + kBlock - 1) / kBlock;
    hipLaunchKernelGGL((gated_backward_kernel<T, KIND>), dim3(uint32_t(g->sequences * int64_t(blocks))), dim3(64), 0, stream,
                       *g);
    return hipGetLastError();
  }
};
template <typename T, int KIND>
struct Step {
  static hipError_t run(float* state, const void* gate, const void* u, void* h, int64_t n, hipStream_t stream) {
    hipLaunchKernelGGL((gated_step_kernel<T, KIND>), dim3(uint32_t(min((n + 255) / 256, int64_t(1) << 20))), dim3(256), 0, stream, state,
                       static_cast<const T*>(gate), static_cast<const T*>(u), static_cast<T*>(h), n);
    return hipGetLastError();
  }
};

}  // namespace

size_t gated_workspace_bytes(int32_t sequences, int64_t tokens, int32_t channels, bool packed) {
  (void)tokens;
  (void)packed;
  const int64_t blocks = (int64_t(channels) + kBlock - 1) / kBlock;
  return sequences * blocks < (int64_t(1) << 24) ? 256 : 0;   // a grid holds 2^32 threads
}

hipError_t launch_gated_scan(const GatedArgs& a, hipStream_t stream) {
  return dispatch<Forward>(a.dtype, a.gate_kind, &a, stream);
}
hipError_t launch_gated_backward(const GatedArgs& a, hipStream_t stream) {
  return dispatch<Backward>(a.dtype, a.gate_kind, &a, stream);
}
hipError_t launch_gated_step(int32_t dtype, int32_t gate_kind, float* state, const void* gate, const void* u, void* h,
                             int64_t n, hipStream_t stream) {
  return dispatch<Step>(dtype, gate_kind, state, gate, u, h, n, stream);
}

}  // namespace ssdq
