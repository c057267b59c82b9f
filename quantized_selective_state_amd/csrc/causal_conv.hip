// Short causal convolution along the tokens of every channel with SiLU, for prompts (dense or packed) and for single
// tokens.
//
// HBM-bound: one read and one write per element (out of memory 4 x 2048 x 4096 bf16 30 us, 4.5 TB/s; 16384 x 5120 fp16 62
// us, 5.4 TB/s, a copy of it 63; small ones by the latency of a wave, 9001 x 1536 bf16 21 us).  A lane holds 4 neighbouring channels of a run of 16 rows and the width - 1 rows before it, all loaded before the
// first is used, so a row is read once and (width - 1) / 16 times more, from cache (rows loaded one by one: 136 us at
// 16384 x 5120; with a branch at every row's end 111).  Runs are cut at multiples of their rows in the whole tensor,
// whatever the sequences are; those that a sequence begins or ends within decide row by row (9001 x 1536 in 2 or 37 sequences
// 26 and 27 us).
#include "block_internal.h"
#include "gated_types.h"
#include "sequences.h"

namespace ssdq {
namespace {

constexpr int V = 4;
constexpr int kRun = 16;       // rows of a wave
constexpr int kThreads = 256;
constexpr int kWaveChannels = kWave * V;
constexpr int kNoLoads = 0x0F70;   // s_waitcnt: no memory operation under way, whatever LDS has

struct ConvKernelArgs {
  Sequences seq;
  const void* x;
  const float* weight;
  const float* bias;
  const void* state;
  void* out;
  void* state_out;
  int32_t channels;
  uint32_t runs;      // then one item per sequence that writes its state
  uint32_t items;
  FastDiv blocks;     // of kWaveChannels channels
  bool silu;
};

template <typename T>
struct Taps { T e[V]; };

template <typename T>
__device__ __forceinline__ Taps<T> load_taps(const T* __restrict__ p, int count) {
  Taps<T> t = {};
  if (count >= V) {
    __builtin_memcpy(&t, p, sizeof(t));
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < count) t.e[i] = p[i];
  }
  return t;
}
// PAST: the caches are not to keep it
template <bool PAST = false, typename T>
__device__ __forceinline__ void store_taps(T* __restrict__ p, int count, const Taps<T>& t) {
  if (count >= V) {
    typedef typename Bytes<sizeof(t)>::type Word;
    typedef Word Anywhere __attribute__((aligned(sizeof(T))));
    if constexpr (PAST) __builtin_nontemporal_store(__builtin_bit_cast(Word, t), reinterpret_cast<Anywhere*>(p));
    else *reinterpret_cast<Anywhere*>(p) = __builtin_bit_cast(Word, t);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < count) p[i] = t.e[i];
  }
}

template <int W>
__device__ __forceinline__ void load_weights(const float* __restrict__ weight, const float* __restrict__ bias, int c,
                                             int count, float (&w)[V][W], float (&b)[V]) {
  if (count >= V) {
    __builtin_memcpy(&w, weight + int64_t(c) * W, sizeof(w));
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int k = 0; k < W; ++k) w[i][k] = i < count ? weight[int64_t(c + i) * W + k] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) b[i] = bias != nullptr && i < count ? bias[c + i] : 0.f;
}

// the output of one row: the window holds the W - 1 rows before `now`, oldest first
template <typename T, int W>
__device__ __forceinline__ Taps<T> convolve(const Taps<T> (&window)[W - 1], const Taps<T>& now, const float (&w)[V][W],
                                            const float (&b)[V], bool activate) {
  Taps<T> r;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float a = b[i];
#pragma unroll
    for (int k = 0; k + 1 < W; ++k) a = fmaf(w[i][k], to_f32(window[k].e[i]), a);
    a = fmaf(w[i][W - 1], to_f32(now.e[i]), a);
    if (activate) a = silu<__is_same(T, float)>(a);
    r.e[i] = from_f32<T>(a);
  }
  return r;
}

template <typename T, int W>
__device__ __forceinline__ Taps<T> state_row(const ConvKernelArgs& a, int64_t s, int k, int c, int count) {
  if (a.state == nullptr) return Taps<T>{};
  return load_taps(static_cast<const T*>(a.state) + (s * (W - 1) + k) * a.channels + c, count);
}

template <typename T, int W, bool PAST>
__global__ void __launch_bounds__(kThreads) causal_conv_kernel(ConvKernelArgs a) {
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x / kWave));
  const uint32_t unit = blockIdx.x * uint32_t(kThreads / kWave) + uint32_t(wave);
  const uint32_t item = fdiv(unit, a.blocks);
  if (item >= a.items) return;
  int c = int(unit - item * a.blocks.d) * kWaveChannels + int(threadIdx.x % kWave) * V;
  if (c >= a.channels) return;
  // a last lane with fewer channels moves back and writes some of its neighbour's too, the same values
  if (a.channels >= V) c = min(c, a.channels - V);
  const int count = a.channels - c;
  const T* x = static_cast<const T*>(a.x);
  if (item >= a.runs) {   // the inputs of a sequence's last W - 1 tokens
    const int64_t s = item - a.runs;
    const Span span = a.seq.span(s);
#pragma unroll
    for (int k = 0; k + 1 < W; ++k) {
      const int64_t row = int64_t(span.end) - (W - 1) + k;
      const int from = int(row - span.begin) + W - 1;   // before the first token: of the state
      const Taps<T> t = row >= span.begin ? load_taps(x + row * a.channels + c, count)
                                          : state_row<T, W>(a, s, from, c, count);
      store_taps(static_cast<T*>(a.state_out) + (s * (W - 1) + k) * a.channels + c, count, t);
    }
    return;
  }
  const int32_t first = int32_t(item) * kRun, last = min(first + kRun, a.seq.tokens);
  float w[V][W], b[V];
  load_weights<W>(a.weight, a.bias, c, count, w, b);
  T* out = static_cast<T*>(a.out);
  Taps<T> x_of[kRun + W - 1];
  int32_t s = a.seq.at(first);
  Span span = a.seq.span(s);
  if (a.channels >= V && last - first == kRun && span.begin <= first && last <= span.end) {
    // One sequence: straight through.  Behind a branch a wave would wait for its earlier stores too.
#pragma unroll
    for (int i = W - 1; i < kRun + W - 1; ++i) x_of[i] = load_taps(x + int64_t(first - (W - 1) + i) * a.channels + c, V);
    if (span.begin <= first - (W - 1)) {
#pragma unroll
      for (int i = 0; i + 1 < W; ++i) x_of[i] = load_taps(x + int64_t(first - (W - 1) + i) * a.channels + c, V);
    } else {
#pragma unroll
      for (int i = 0; i + 1 < W; ++i) {
        const int32_t source = first - (W - 1) + i;
        if (source >= span.begin) x_of[i] = load_taps(x + int64_t(source) * a.channels + c, V);
        else x_of[i] = state_row<T, W>(a, s, source - span.begin + W - 1, c, V);
      }
    }
#pragma unroll
    for (int r = 0; r < kRun; ++r) {
      Taps<T> window[W - 1];
#pragma unroll
      for (int k = 0; k + 1 < W; ++k) window[k] = x_of[r + k];
      store_taps<PAST>(out + int64_t(first + r) * a.channels + c, V, convolve<T, W>(window, x_of[r + W - 1], w, b, a.silu));
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < kRun + W - 1; ++i)   // (rows of other sequences too, and the tensor's first and last ones again)
    x_of[i] = load_taps(x + int64_t(min(max(first - (W - 1) + i, 0), last - 1)) * a.channels + c, count);
  if (span.begin < first && first < span.end) {
#pragma unroll
    for (int k = 0; k + 1 < W; ++k) {
      const int32_t source = first - (W - 1) + k;
      if (source < span.begin) x_of[k] = state_row<T, W>(a, s, source - span.begin + W - 1, c, count);
    }
  }
  __builtin_amdgcn_s_waitcnt(kNoLoads);
#pragma unroll
  for (int r = 0; r < kRun; ++r) {
    const int32_t row = first + r;
    if (s < a.seq.sequences && span.end <= row) a.seq.advance(row, s, span);
    if (row >= last || s >= a.seq.sequences) break;
    if (row < span.begin) continue;
    if (row == span.begin) {   // its state in the place of the rows ahead, which are done with
#pragma unroll
      for (int k = 0; k + 1 < W; ++k) x_of[r + k] = state_row<T, W>(a, s, k, c, count);
      __builtin_amdgcn_s_waitcnt(kNoLoads);   // here, so that rows without a beginning wait for nothing
    }
    Taps<T> window[W - 1];
#pragma unroll
    for (int k = 0; k + 1 < W; ++k) window[k] = x_of[r + k];
    store_taps<PAST>(out + int64_t(row) * a.channels + c, count, convolve<T, W>(window, x_of[r + W - 1], w, b, a.silu));
  }
}

template <typename T, int W>
__global__ void __launch_bounds__(kThreads) causal_conv_step_kernel(T* __restrict__ state, const T* __restrict__ x,
                                                                    const float* __restrict__ weight,
                                                                    const float* __restrict__ bias, T* __restrict__ out,
                                                                    uint32_t units, FastDiv packs, int32_t channels,
                                                                    bool activate) {
  const uint32_t unit = blockIdx.x * kThreads + threadIdx.x;
  if (unit >= units) return;
  const uint32_t s = fdiv(unit, packs);
  const int c = int(unit - s * packs.d) * V, count = channels - c;
  float w[V][W], b[V];
  load_weights<W>(weight, bias, c, count, w, b);
  T* rows = state + int64_t(s) * (W - 1) * channels + c;
  Taps<T> window[W - 1];
#pragma unroll
  for (int k = 0; k + 1 < W; ++k) window[k] = load_taps(rows + int64_t(k) * channels, count);
  const Taps<T> now = load_taps(x + int64_t(s) * channels + c, count);
  store_taps(out + int64_t(s) * channels + c, count, convolve<T, W>(window, now, w, b, activate));
#pragma unroll
  for (int k = 0; k + 1 < W; ++k) store_taps(rows + int64_t(k) * channels, count, k + 2 < W ? window[k + 1] : now);
}

template <typename T>
hipError_t launch_conv(const ConvArgs& c, hipStream_t stream) {
  ConvKernelArgs a = {};
  a.seq = make_sequences(c.offsets, c.sequences, c.tokens);
  a.x = c.x;
  a.weight = c.weight;
  a.bias = c.bias;
  a.state = c.state;
  a.out = c.out;
  a.state_out = c.state_out;
  a.channels = c.channels;
  a.runs = uint32_t((c.tokens + kRun - 1) / kRun);
  a.items = a.runs + (c.state_out != nullptr ? uint32_t(c.sequences) : 0u);
  a.blocks = make_fastdiv(uint32_t((c.channels + kWaveChannels - 1) / kWaveChannels));
  a.silu = c.silu;
  const int64_t units = int64_t(a.items) * a.blocks.d;
  if (units == 0) return hipSuccess;
  constexpr int kWaves = kThreads / kWave;
  const dim3 grid(uint32_t((units + kWaves - 1) / kWaves));
  // Stores pass the caches by once a call touches more than the 256 MiB of the Infinity Cache (16384 x 8192 bf16: 92 us
  // against 95, its input in the caches 79 against 94).  Below that it would gain up to 2 us, and what reads the output
  // next would lose more.
  const bool past = c.tokens * c.channels * int64_t(2 * sizeof(T)) > int64_t(256) << 20;
  switch (c.width * 2 + past) {
    case 4: causal_conv_kernel<T, 2, false><<<grid, kThreads, 0, stream>>>(a); break;
    case 5: causal_conv_kernel<T, 2, true><<<grid, kThreads, 0, stream>>>(a); break;
    case 6: causal_conv_kernel<T, 3, false><<<grid, kThreads, 0, stream>>>(a); break;
    case 7: causal_conv_kernel<T, 3, true><<<grid, kThreads, 0, stream>>>(a); break;
    case 8: causal_conv_kernel<T, 4, false><<<grid, kThreads, 0, stream>>>(a); break;
    default: causal_conv_kernel<T, 4, true><<<grid, kThreads, 0, stream>>>(a);
  }
  return hipGetLastError();
}

template <typename T>
hipError_t launch_step(void* state, const void* x, const float* weight, const float* bias, void* out, int32_t batch,
                       int32_t channels, int32_t width, bool silu, hipStream_t stream) {
  const FastDiv packs = make_fastdiv(uint32_t((channels + V - 1) / V));
  const uint32_t units = uint32_t(batch) * packs.d;      // below 2^31: no more than batch * channels
  const dim3 grid((units + kThreads - 1) / kThreads);
  T* st = static_cast<T*>(state);
  const T* in = static_cast<const T*>(x);
  T* o = static_cast<T*>(out);
  const auto kernel = width == 2   ? causal_conv_step_kernel<T, 2>
                      : width == 3 ? causal_conv_step_kernel<T, 3>
                                   : causal_conv_step_kernel<T, 4>;
  kernel<<<grid, kThreads, 0, stream>>>(st, in, weight, bias, o, units, packs, channels, silu);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_causal_conv(const ConvArgs& a, hipStream_t stream) {
  switch (a.dtype) {
    case SSDQ_DTYPE_F32: return launch_conv<float>(a, stream);
    case SSDQ_DTYPE_F16: return launch_conv<_Float16>(a, stream);
    default: return launch_conv<__bf16>(a, stream);
  }
}

hipError_t launch_causal_conv_step(int32_t dtype, void* state, const void* x, const float* weight, const float* bias,
                                   void* out, int32_t batch, int32_t channels, int32_t width, bool silu,
                                   hipStream_t stream) {
  switch (dtype) {
    case SSDQ_DTYPE_F32: return launch_step<float>(state, x, weight, bias, out, batch, channels, width, silu, stream);
    case SSDQ_DTYPE_F16: return launch_step<_Float16>(state, x, weight, bias, out, batch, channels, width, silu, stream);
    default: return launch_step<__bf16>(state, x, weight, bias, out, batch, channels, width, silu, stream);
  }
}

}  // namespace ssdq
