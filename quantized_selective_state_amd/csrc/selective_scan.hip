// Selective state space scan: a decay for every (channel, state) and a step size for every channel, for prompts (dense
// or packed) and for single tokens.
//
//   d = softplus(delta + bias);  h[n] = exp(d A[n]) h[n] + d u B[n];  y = (sum_n C[n] h[n] + D u) silu(z)
//
// A lane holds one channel with its N states in registers and walks a chunk of rows; B and C, the same for all channels,
// are staged as binary32 in LDS for the block's 256 channels.  Chunks run side by side: a first kernel forms what every
// chunk makes of a zero state, a second one carries states from chunk to chunk, h <- exp(A sum d) h + that, and a third
// walks the chunks again from the states that enter them and writes y.
#include "block_internal.h"
#include "gated_types.h"
#include "sequences.h"

namespace ssdq {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 16;            // rows of B and C in LDS at a time
constexpr float kLog2e = 1.44269502e+00f;

// softplus(v) = max(v, 0) + log(1 + e), e = exp(-|v|), to a few 2^-24 of itself also where it is small: there by the
// series of log(1 + e), else by the hardware's logarithm of w = 1 + e with the rounding of that sum put back.
__device__ __forceinline__ float softplus(float v) {
  const float e = exp_f32<true>(-fabsf(v));
  const float w = 1.f + e, lost = e - (w - 1.f);
  const float large = fmaf(__builtin_amdgcn_logf(w), 0.693147182f, lost * __builtin_amdgcn_rcpf(w));
  const float small = e * fmaf(-e, fmaf(-e, fmaf(-e, 0.25f, 0.333333343f), 0.5f), 1.f);
  const float log1p = e < 0.015625f ? small : large;
  return fmaxf(v, 0.f) + log1p;
}
__device__ __forceinline__ float gated(float y, float z) {
  return y * z * __builtin_amdgcn_rcpf(1.f + exp_f32<true>(-z));
}

struct ScanKernelArgs {
  Sequences seq;
  const void* u;
  const void* delta;
  const float* A;
  const void* B;
  const void* C;
  const float* D;
  const void* z;
  const float* delta_bias;
  const float* h0;
  void* y;
  float* h_final;
  float* states;       // (chunks, N, channels): after the first kernel a chunk's own, after the second what leaves it
  float* sums;         // (chunks, channels): sum of d over the chunk
  int32_t* resets;     // (chunks): what leaves the chunk does not depend on what enters it
  int32_t channels, dstate;
  int32_t chunk;       // rows
  int32_t per_sequence;   // chunks of a dense sequence; packed: all
  int32_t chunks;
  bool softplus;
};

// the rows of a chunk: dense chunks are cut within their sequence, packed ones at multiples of the chunk
__device__ __forceinline__ Span chunk_rows(const ScanKernelArgs& a, int32_t k) {
  if (a.seq.offsets != nullptr) return Span{k * a.chunk, int32_t(min(int64_t(k + 1) * a.chunk, int64_t(a.seq.tokens)))};
  const int32_t s = k / a.per_sequence, i = k - s * a.per_sequence;
  const Span span = a.seq.span(s);
  return Span{span.begin + i * a.chunk, int32_t(min(int64_t(span.begin) + int64_t(i + 1) * a.chunk, int64_t(span.end)))};
}

template <typename T, int N, bool OUTPUT>
__global__ void __launch_bounds__(kThreads) chunk_kernel(ScanKernelArgs a) {
  __shared__ float Bs[kRows][N], Cs[OUTPUT ? kRows : 1][N];
  const int32_t c = int32_t(blockIdx.y) * kThreads + int32_t(threadIdx.x);
  const bool live = c < a.channels;
  if (int32_t(blockIdx.x) >= a.chunks) {   // sequences without rows: their state passes through
    const int32_t step = int32_t(gridDim.x) - a.chunks;
    for (int32_t s = int32_t(blockIdx.x) - a.chunks; s < a.seq.sequences; s += step) {
      const Span span = a.seq.span(s);
      if (span.begin < span.end || !live) continue;
      for (int n = 0; n < a.dstate; ++n) {
        const int64_t at = (int64_t(s) * a.channels + c) * a.dstate + n;
        a.h_final[at] = a.h0 != nullptr ? a.h0[at] : 0.f;
      }
    }
    return;
  }
  const int32_t k = int32_t(blockIdx.x);
  const Span rows = chunk_rows(a, k);
  int32_t s = a.seq.at(rows.begin);
  Span span = a.seq.span(s);
  int32_t from = rows.begin;
  if constexpr (!OUTPUT) {
    // only what leaves the chunk is wanted: the sequence that goes on behind its last row
    while (s < a.seq.sequences) {
      span = a.seq.span(s);
      if (span.end > rows.end) break;
      ++s;
    }
    const bool leaves = s < a.seq.sequences && span.begin < rows.end;
    if (c == 0) a.resets[k] = !leaves || span.begin >= rows.begin;
    if (!leaves) return;
    from = max(from, span.begin);
  }
  float A2[N], h[N], sum = 0.f;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    A2[n] = live && n < a.dstate ? a.A[int64_t(c) * a.dstate + n] * kLog2e : 0.f;
    h[n] = 0.f;
  }
  const float bias = live && a.delta_bias != nullptr ? a.delta_bias[c] : 0.f;
  const float skip = OUTPUT && live && a.D != nullptr ? a.D[c] : 0.f;
  const T* u = static_cast<const T*>(a.u);
  const T* delta = static_cast<const T*>(a.delta);
  const T* z = static_cast<const T*>(a.z);
  const T* B = static_cast<const T*>(a.B);
  const T* C = static_cast<const T*>(a.C);
  T* y = static_cast<T*>(a.y);

  const auto enter = [&](int32_t row) {   // the state ahead of `row`, which is in sequence s
    if (!live) return;
    if (row == span.begin) {
#pragma unroll
      for (int n = 0; n < N; ++n)
        h[n] = a.h0 != nullptr && n < a.dstate ? a.h0[(int64_t(s) * a.channels + c) * a.dstate + n] : 0.f;
    } else if (OUTPUT && k > 0) {   // (k is 0 here only with offsets out of order)
#pragma unroll
      for (int n = 0; n < N; ++n)
        h[n] = n < a.dstate ? a.states[(int64_t(k - 1) * a.dstate + n) * a.channels + c] : 0.f;
    }
  };
  bool inside = false;
  for (int32_t tile = from; tile < rows.end; tile += kRows) {
    __syncthreads();
    const int32_t count = min(kRows, rows.end - tile);
    for (int i = threadIdx.x; i < kRows * N; i += kThreads) {
      const int r = i / N, n = i % N;
      const bool some = r < count && n < a.dstate;
      Bs[r][n] = some ? to_f32(B[int64_t(tile + r) * a.dstate + n]) : 0.f;
      if constexpr (OUTPUT) Cs[r][n] = some ? to_f32(C[int64_t(tile + r) * a.dstate + n]) : 0.f;
    }
    __syncthreads();
    for (int r = 0; r < count; ++r) {
      const int32_t row = tile + r;
      while (s < a.seq.sequences && span.end <= row) {
        if (++s < a.seq.sequences) span = a.seq.span(s);
        inside = false;
      }
      if (s >= a.seq.sequences || row < span.begin) continue;
      if (!inside) {
        enter(row);
        inside = true;
      }
      if (live) {
        const int64_t at = int64_t(row) * a.channels + c;
        float d = to_f32(delta[at]) + bias;
        if (a.softplus) d = softplus(d);
        const float v = to_f32(u[at]), dv = d * v;
        float out = skip * v;
#pragma unroll
        for (int n = 0; n < N; ++n) {
          h[n] = fmaf(__builtin_amdgcn_exp2f(d * A2[n]), h[n], dv * Bs[r][n]);
          if constexpr (OUTPUT) out = fmaf(Cs[r][n], h[n], out);
        }
        sum += d;
        if constexpr (OUTPUT) y[at] = from_f32<T>(z != nullptr ? gated(out, to_f32(z[at])) : out);
      }
      if (OUTPUT && live && row + 1 == span.end && a.h_final != nullptr) {
#pragma unroll
        for (int n = 0; n < N; ++n)
          if (n < a.dstate) a.h_final[(int64_t(s) * a.channels + c) * a.dstate + n] = h[n];
      }
    }
  }
  if constexpr (!OUTPUT) {
    if (!live) return;
#pragma unroll
    for (int n = 0; n < N; ++n)
      if (n < a.dstate) a.states[(int64_t(k) * a.dstate + n) * a.channels + c] = h[n];
    a.sums[int64_t(k) * a.channels + c] = sum;
  }
}

// chunk by chunk along every chain (a dense sequence, or all packed rows), one thread per channel and state
__global__ void __launch_bounds__(kThreads) carry_kernel(ScanKernelArgs a) {
  const int32_t c = int32_t(blockIdx.x) * kThreads + int32_t(threadIdx.x);
  const int32_t n = int32_t(blockIdx.y);
  if (c >= a.channels) return;
  const float A2 = a.A[int64_t(c) * a.dstate + n] * kLog2e;
  for (int32_t first = int32_t(blockIdx.z) * a.per_sequence; first < a.chunks;
       first += int32_t(gridDim.z) * a.per_sequence) {
    const int32_t last = first + a.per_sequence - 1;
    float h = 0.f;
    for (int32_t k = first; k < last; ++k) {   // nothing enters a chain's first chunk; nothing reads what leaves its last
      float* at = a.states + (int64_t(k) * a.dstate + n) * a.channels + c;
      const float own = *at;
      h = a.resets[k] ? own : fmaf(__builtin_amdgcn_exp2f(a.sums[int64_t(k) * a.channels + c] * A2), h, own);
      *at = h;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) step_kernel(float* __restrict__ state, const T* __restrict__ u,
                                                        const T* __restrict__ delta, const float* __restrict__ A,
                                                        const T* __restrict__ B, const T* __restrict__ C,
                                                        const float* __restrict__ D, const T* __restrict__ z,
                                                        const float* __restrict__ delta_bias, T* __restrict__ y,
                                                        int64_t items, int32_t channels, int32_t dstate, int32_t lanes,
                                                        bool use_softplus) {
  // `lanes` neighbouring lanes per channel, four states each
  const int64_t step = int64_t(gridDim.x) * (kThreads / lanes);
  const int first = int(threadIdx.x % lanes) * 4, count = dstate - first;
  for (int64_t item = int64_t(blockIdx.x) * (kThreads / lanes) + threadIdx.x / lanes; item < items; item += step) {
    const int64_t s = item / channels;
    const int32_t c = int32_t(item - s * channels);
    float d = to_f32(delta[item]) + (delta_bias != nullptr ? delta_bias[c] : 0.f);
    if (use_softplus) d = softplus(d);
    const float v = to_f32(u[item]), dv = d * v;
    float out = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < count) {
        const int n = first + i;
        float* at = state + item * dstate + n;
        const float h = fmaf(__builtin_amdgcn_exp2f(d * A[int64_t(c) * dstate + n] * kLog2e), *at, dv * to_f32(B[s * dstate + n]));
        *at = h;
        out = fmaf(to_f32(C[s * dstate + n]), h, out);
      }
    }
    for (int k = 1; k < lanes; k <<= 1) out += __shfl_xor(out, k);
    if (threadIdx.x % lanes == 0) {
      if (D != nullptr) out = fmaf(D[c], v, out);
      y[item] = from_f32<T>(z != nullptr ? gated(out, to_f32(z[item])) : out);
    }
  }
}

// ---- host ----

constexpr int32_t kChunk = 256;

struct Plan {
  int32_t chunk, per_sequence, chunks;
  size_t sums, resets, bytes;   // byte offsets behind the states, and the total
};

bool make_plan(int32_t sequences, int64_t tokens, int32_t channels, int32_t dstate, bool packed, Plan* p) {
  p->chunk = kChunk;
  const int64_t length = packed ? tokens : tokens / sequences;
  const int64_t per = (length + p->chunk - 1) / p->chunk, chunks = packed ? per : per * sequences;
  if (chunks >= int64_t(1) << 23) return false;   // a grid's threads along x in 32 bits
  p->per_sequence = int32_t(per);
  p->chunks = int32_t(chunks);
  const double need = double(chunks) * channels * (dstate + 1) * 4.0;
  if (need >= double(int64_t(1) << 40)) return false;
  const auto round = [](size_t n) { return (n + 255) & ~size_t(255); };
  p->sums = round(size_t(chunks) * dstate * channels * 4);
  p->resets = p->sums + round(size_t(chunks) * channels * 4);
  p->bytes = std::max<size_t>(256, p->resets + round(size_t(chunks) * 4));
  return true;
}

template <typename T, int N>
hipError_t launch_states(const ScanKernelArgs& a, hipStream_t stream) {
  const uint32_t blocks = uint32_t((a.channels + kThreads - 1) / kThreads);
  // grid.x: the chunks, and where packed sequences may have no rows some blocks that look for those
  const bool empty = a.h_final != nullptr && (a.seq.offsets != nullptr || a.seq.tokens == 0);
  const uint32_t extra = empty ? uint32_t(std::min(a.seq.sequences, 64)) : 0u;
  if (a.per_sequence > 1) {
    chunk_kernel<T, N, false><<<dim3(a.chunks, blocks), kThreads, 0, stream>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const uint32_t chains = uint32_t(std::min(a.chunks / a.per_sequence, 32768));
    carry_kernel<<<dim3(blocks, a.dstate, chains), kThreads, 0, stream>>>(a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.chunks + extra == 0) return hipSuccess;
  chunk_kernel<T, N, true><<<dim3(a.chunks + extra, blocks), kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_scan(const ScanKernelArgs& a, hipStream_t stream) {
  if (a.dstate <= 8) return launch_states<T, 8>(a, stream);
  if (a.dstate <= 16) return launch_states<T, 16>(a, stream);
  if (a.dstate <= 32) return launch_states<T, 32>(a, stream);
  return launch_states<T, 64>(a, stream);
}

template <typename T>
hipError_t launch_step(float* state, const void* u, const void* delta, const float* A, const void* B, const void* C,
                       const float* D, const void* z, const float* delta_bias, void* y, int32_t batch, int32_t channels,
                       int32_t dstate, bool softplus, hipStream_t stream) {
  int32_t lanes = 1;
  while (lanes * 4 < dstate) lanes *= 2;
  const int64_t items = int64_t(batch) * channels, per = kThreads / lanes;
  const int64_t blocks = std::min<int64_t>((items + per - 1) / per, 1 << 20);
  step_kernel<T><<<dim3(uint32_t(blocks)), kThreads, 0, stream>>>(
      state, static_cast<const T*>(u), static_cast<const T*>(delta), A, static_cast<const T*>(B),
      static_cast<const T*>(C), D, static_cast<const T*>(z), delta_bias, static_cast<T*>(y), items, channels, dstate,
      lanes, softplus);
  return hipGetLastError();
}

}  // namespace

size_t selective_workspace_bytes(int32_t sequences, int64_t tokens, int32_t channels, int32_t dstate, bool packed) {
  Plan p;
  return make_plan(sequences, tokens, channels, dstate, packed, &p) ? p.bytes : 0;
}

hipError_t launch_selective_scan(const SelectiveArgs& s, hipStream_t stream) {
  Plan p;
  if (!make_plan(s.sequences, s.tokens, s.channels, s.dstate, s.offsets != nullptr, &p)) return hipErrorInvalidValue;
  ScanKernelArgs a = {};
  a.seq = make_sequences(s.offsets, s.sequences, s.tokens);
  a.u = s.u;
  a.delta = s.delta;
  a.A = s.A;
  a.B = s.B;
  a.C = s.C;
  a.D = s.D;
  a.z = s.z;
  a.delta_bias = s.delta_bias;
  a.h0 = s.h0;
  a.y = s.y;
  a.h_final = s.h_final;
  char* base = static_cast<char*>(s.workspace);
  a.states = reinterpret_cast<float*>(base);
  a.sums = reinterpret_cast<float*>(base + p.sums);
  a.resets = reinterpret_cast<int32_t*>(base + p.resets);
  a.channels = s.channels;
  a.dstate = s.dstate;
  a.chunk = p.chunk;
  a.per_sequence = p.per_sequence;
  a.chunks = p.chunks;
  a.softplus = s.softplus;
  switch (s.dtype) {
    case SSDQ_DTYPE_F32: return launch_scan<float>(a, stream);
    case SSDQ_DTYPE_F16: return launch_scan<_Float16>(a, stream);
    default: return launch_scan<__bf16>(a, stream);
  }
}

hipError_t launch_selective_step(int32_t dtype, float* state, const void* u, const void* delta, const float* A,
                                 const void* B, const void* C, const float* D, const void* z, const float* delta_bias,
                                 void* y, int32_t batch, int32_t channels, int32_t dstate, bool softplus,
                                 hipStream_t stream) {
  switch (dtype) {
    case SSDQ_DTYPE_F32:
      return launch_step<float>(state, u, delta, A, B, C, D, z, delta_bias, y, batch, channels, dstate, softplus, stream);
    case SSDQ_DTYPE_F16:
      return launch_step<_Float16>(state, u, delta, A, B, C, D, z, delta_bias, y, batch, channels, dstate, softplus, stream);
    default:
      return launch_step<__bf16>(state, u, delta, A, B, C, D, z, delta_bias, y, batch, channels, dstate, softplus, stream);
  }
}

}  // namespace ssdq
