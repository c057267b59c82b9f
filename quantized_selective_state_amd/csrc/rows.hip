// Root-mean-square norm of rows with the residual's addition or a gate, output in the inputs' type or as 8-bit codes
// with a scale per row; rows as codes without a norm; and their values.
//
// One pass: n = (v w) / sqrt(mean(v^2) + eps), and since multiplying by the positive root is monotone in binary32,
// max |n| is max |v w| times it.  So the sum of squares and the largest |v w| are reduced together, the row stays in
// registers between, and a block has one barrier per row (none where a row fits one wave).
//
// Squares below 2^-149 are lost.  That is nothing beside an eps of 2^-64 or more; with a smaller one (kSmall) a group's
// values are first scaled by a power of two to a largest magnitude near 1, which changes no other digit and takes one
// reduction more (32768 x 4096 with eps 0, fp32: norm 238 us and 244 so, to codes 124 and 129).
//
// HBM-bound: every tensor once (32768 x 4096 bf16: norm 82 us, 6.5 TB/s; to codes 73, with a residual in bf16 to codes 172,
// 5.5 TB/s; 32768 x 8192 fp16 gated to codes 256, 5.2 TB/s; rows as codes 70 and back 61 at 32768 x 4096).  A lane's 16
// bytes are neighbours and a lane holds up to four such pieces, so that a row has some waves and a compute unit many
// rows: their loads cover each other's latency, and no row is loaded ahead by its own block.
#include <algorithm>
#include <cmath>

#include "block_internal.h"
#include "gated_types.h"

namespace ssdq {
namespace {

constexpr int V = 8;              // neighbouring channels of a lane
constexpr int kMostThreads = 1024;
enum Source { kPlain, kResidual, kGate };
enum Output { kValues, kDynamic, kStatic };

template <typename T>
struct Eight { T e[V]; };

// Rows start at any element, so the loads and stores are of 16 bytes (or 32, or 8) at any alignment; the last channels
// of a group one by one.
template <int kBytes> struct Words;
template <> struct Words<32> { typedef uint32_t type __attribute__((ext_vector_type(8))); };
template <> struct Words<16> { typedef v4u type; };
template <> struct Words<8> { typedef v2u type; };

template <typename T>
__device__ __forceinline__ void load_some(const T* __restrict__ p, int count, float (&v)[V]) {
  typedef typename Words<sizeof(Eight<T>)>::type W;
  typedef W Anywhere __attribute__((aligned(sizeof(T))));
  Eight<T> raw = {};
  if (count >= V) {
    raw = __builtin_bit_cast(Eight<T>, W(*reinterpret_cast<const Anywhere*>(p)));
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < count) raw.e[i] = p[i];
  }
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = to_f32(raw.e[i]);
}
// PAST: the caches are not to keep it
template <bool PAST, typename T>
__device__ __forceinline__ void store_some(T* __restrict__ p, int count, const Eight<T>& raw) {
  typedef typename Words<sizeof(Eight<T>)>::type W;
  typedef W Anywhere __attribute__((aligned(sizeof(T))));
  if (count >= V) {
    if constexpr (PAST) __builtin_nontemporal_store(__builtin_bit_cast(W, raw), reinterpret_cast<Anywhere*>(p));
    else *reinterpret_cast<Anywhere*>(p) = __builtin_bit_cast(W, raw);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < count) p[i] = raw.e[i];
  }
}
template <typename T>
__device__ __forceinline__ Eight<T> rounded(const float (&v)[V]) {
  Eight<T> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.e[i] = from_f32<T>(v[i]);
  return r;
}

struct NormKernelArgs {
  const void* x;
  const void* other;        // residual or gate
  const float* weight;
  const float* static_scale;
  void* out;
  int8_t* codes;
  float* scale;
  void* residual_out;
  int64_t rows;
  int32_t channels, groups, size;   // size = channels / groups
  int32_t lanes;                    // threads of a group, a power of two
  int32_t per_block;                // rows of a block
  float eps, inverse_size;
  int32_t most_shift;               // kSmall: of the scaling, so that eps stays finite under it
};

// sum and most over the `lanes` (at most 64) neighbouring lanes of a group, in all of them
__device__ __forceinline__ void reduce_lanes(float& sum, uint32_t& most, int lanes) {
  for (int d = 1; d < lanes && d < kWave; d <<= 1) {
    sum += __shfl_xor(sum, d);
    most = max(most, uint32_t(__shfl_xor(int(most), d)));
  }
}

__device__ __forceinline__ float root(float sum, float eps, const NormKernelArgs& a) {
  return sum < __builtin_inff() ? 1.f / sqrtf(fmaf(sum, a.inverse_size, eps)) : __builtin_nanf("");
}

// kSmall: 2^shift for a group with this largest magnitude, 1 where that is 1 or more (or not finite)
__device__ __forceinline__ float scaling(uint32_t most, const NormKernelArgs& a) {
  const int shift = min(max(127 - int(most >> 23), 0), a.most_shift);
  return __uint_as_float(uint32_t(127 + shift) << 23);
}

template <typename T, typename R, int SOURCE, bool NORM, int OUT, int SLOTS, bool PAST, bool kSmall>
__global__ void __launch_bounds__(kMostThreads) norm_kernel(NormKernelArgs a) {
  __shared__ float sums[2][kMostThreads];       // of a wave, or of a group with fewer lanes; two rows in turn
  __shared__ uint32_t mosts[2][kMostThreads];
  __shared__ uint32_t tops[2][kSmall ? kMostThreads : 1];
  const int sub = int(threadIdx.x) / a.lanes, lane = int(threadIdx.x) % a.lanes;
  const int in_block = sub / a.groups, group = sub % a.groups;
  const int unit = a.lanes < kWave ? a.lanes : kWave;            // threads that share one entry of sums
  const int entry = int(threadIdx.x) / unit;
  const int per_group = a.lanes / unit;
  const int first = in_block * a.groups * per_group;             // the row's entries
  const int start = group * a.size;

  float w[SLOTS][V];
  if constexpr (NORM) {
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      const int c = (s * a.lanes + lane) * V;
      load_some(a.weight + start + c, in_block < a.per_block ? a.size - c : 0, w[s]);
    }
  }
  int parity = 0;
  for (int64_t row0 = int64_t(blockIdx.x) * a.per_block; row0 < a.rows; row0 += int64_t(gridDim.x) * a.per_block) {
    const int64_t row = row0 + in_block;
    const bool live = in_block < a.per_block && row < a.rows;
    const int64_t at = row * a.channels + start;
    float v[SLOTS][V], sum = 0.f, eps = a.eps;
    uint32_t most = 0;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      const int c = (s * a.lanes + lane) * V, count = live ? a.size - c : 0;
      load_some(static_cast<const T*>(a.x) + at + c, count, v[s]);
      if constexpr (SOURCE != kPlain) {
        float o[V];
        load_some(static_cast<const R*>(a.other) + at + c, count, o);
#pragma unroll
        for (int i = 0; i < V; ++i)
          v[s][i] = SOURCE == kResidual ? v[s][i] + o[i] : v[s][i] * silu<sizeof(T) == 4>(o[i]);
        if constexpr (SOURCE == kResidual)
          store_some<false>(static_cast<R*>(a.residual_out) + at + c, count, rounded<R>(v[s]));
      }
      if constexpr (kSmall) {
#pragma unroll
        for (int i = 0; i < V; ++i) most = max(most, __float_as_uint(fabsf(v[s][i])));
        continue;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if constexpr (NORM) {
          sum = fmaf(v[s][i], v[s][i], sum);
          v[s][i] *= w[s][i];
        }
        if constexpr (OUT == kDynamic) most = max(most, __float_as_uint(fabsf(v[s][i])));
      }
    }
    const auto scale_of = [&](int g) {   // kSmall: of the row's group g, once tops has its largest magnitudes
      uint32_t top = 0;
      for (int k = 0; k < per_group; ++k) top = max(top, tops[parity][kSmall ? first + g * per_group + k : 0]);
      return scaling(top, a);
    };
    if constexpr (kSmall) {
      reduce_lanes(sum, most, a.lanes);
      float up;
      if (per_group == 1) {
        up = scaling(most, a);
      } else {
        tops[parity][entry] = most;
        __syncthreads();
        up = scale_of(group);
      }
      most = 0;
      eps = a.eps * up * up;
#pragma unroll
      for (int s = 0; s < SLOTS; ++s) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          v[s][i] *= up;
          sum = fmaf(v[s][i], v[s][i], sum);
          v[s][i] *= w[s][i];
          if constexpr (OUT == kDynamic) most = max(most, __float_as_uint(fabsf(v[s][i])));
        }
      }
    }
    reduce_lanes(sum, most, a.lanes);
    float r = 1.f;
    if (per_group == 1) {   // a group's lanes have its sums
      if constexpr (NORM) {
        r = root(sum, eps, a);
        most = __float_as_uint(fabsf(__uint_as_float(most) * r));
      }
      if (OUT == kDynamic && a.groups > 1) {
        mosts[parity][entry] = most;
        __syncthreads();
        for (int g = 0; g < a.groups; ++g) most = max(most, mosts[parity][first + g]);
        parity ^= 1;
      }
    } else {
      sums[parity][entry] = sum;
      mosts[parity][entry] = most;
      __syncthreads();
      most = 0;
      for (int g = 0, e = first; g < a.groups; ++g) {   // the row's largest value needs every group's root
        float total = 0.f;
        uint32_t top = 0;
        for (int k = 0; k < per_group; ++k, ++e) {
          total += sums[parity][e];
          top = max(top, mosts[parity][e]);
        }
        if constexpr (NORM) {
          if (OUT != kDynamic && g != group) continue;
          float its_eps = eps;
          if constexpr (kSmall) {
            const float up = scale_of(g);
            its_eps = a.eps * up * up;
          }
          const float its = root(total, its_eps, a);
          if (g == group) r = its;
          top = __float_as_uint(fabsf(__uint_as_float(top) * its));
        }
        most = max(most, top);
      }
      parity ^= 1;
    }
    float s = 0.f;
    if constexpr (OUT == kDynamic) {
      s = checkpoint_scale(most);
      if (live && group == 0 && lane == 0) a.scale[row] = s;
    } else if constexpr (OUT == kStatic) {
      s = a.static_scale[0];
    }
#pragma unroll
    for (int k = 0; k < SLOTS; ++k) {
      const int c = (k * a.lanes + lane) * V, count = live ? a.size - c : 0;
      float n[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        n[i] = NORM ? v[k][i] * r : v[k][i];
        // beyond 127 scales a code is 127, and a NaN has the code 0; the bound is within a rounding of 127 s
        if constexpr (OUT == kStatic) n[i] = n[i] != n[i] ? 0.f : fminf(fmaxf(n[i], -127.f * s), 127.f * s);
      }
      if constexpr (OUT == kValues) {
        store_some<PAST>(static_cast<T*>(a.out) + at + c, count, rounded<T>(n));
      } else {
        const auto packed = codes_of<V>(n, s);
        store_some<PAST>(a.codes + at + c, count, __builtin_bit_cast(Eight<int8_t>, packed));
      }
    }
  }
}

template <typename T, bool PAST>
__global__ void __launch_bounds__(256) dequantize_rows_kernel(const int8_t* __restrict__ codes,
                                                              const float* __restrict__ scale, T* __restrict__ x,
                                                              int64_t rows, int32_t channels, int32_t lanes) {
  // kAtOnce rows of a thread, so that their loads are under way together (32768 x 8192 fp16 121 us, 230 with one)
  constexpr int kAtOnce = 4;
  const int per_block = 256 / lanes, lane = int(threadIdx.x) % lanes;
  const int64_t step = int64_t(gridDim.x) * per_block;
  for (int64_t row0 = int64_t(blockIdx.x) * per_block + threadIdx.x / lanes; row0 < rows; row0 += step * kAtOnce) {
    float s[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) s[k] = scale[min(row0 + k * step, rows - 1)];
    for (int64_t c = int64_t(lane) * V; c < channels; c += int64_t(lanes) * V) {
      const int count = int(min(int64_t(V), channels - c));
      float v[kAtOnce][V];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) load_some(codes + min(row0 + k * step, rows - 1) * channels + c, count, v[k]);
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        if (row0 + k * step >= rows) break;
#pragma unroll
        for (int i = 0; i < V; ++i) v[k][i] *= s[k];
        store_some<PAST>(x + (row0 + k * step) * channels + c, count, rounded<T>(v[k]));
      }
    }
  }
}

int32_t power_of_two(int32_t n) {
  int32_t p = 1;
  while (p < n) p <<= 1;
  return p;
}

// Stores pass the caches by once a call touches more than the 256 MiB of the Infinity Cache (32768 x 4096 bf16: norm 98
// us and 82 with it, norm to codes 86 and 72, values of codes 82 and 61; below, 100000 x 256 fp16 gated to codes, 29
// and 44).
// The residual stays an ordinary store (fp32 residual to codes, 32768 x 4096: 275 us, 285 with all stores).
constexpr int64_t kInfinityCache = int64_t(256) << 20;
constexpr float kSmallEps = 5.42101086e-20f;   // 2^-64

template <typename T, typename R, int SOURCE, bool NORM, int OUT, bool PAST>
hipError_t launch_slots(const NormArgs& n, hipStream_t stream) {
  NormKernelArgs a = {};
  a.x = n.x;
  a.other = SOURCE == kResidual ? n.residual : n.gate;
  a.weight = n.weight;
  a.static_scale = n.static_scale;
  a.out = n.out;
  a.codes = n.codes;
  a.scale = n.scale;
  a.residual_out = n.residual_out;
  a.rows = n.rows;
  a.channels = n.channels;
  a.groups = n.groups;
  a.size = n.channels / n.groups;
  a.eps = n.eps;
  a.inverse_size = 1.f / float(a.size);
  // (numbers of binary16, down to 2^-24, have squares that do not underflow)
  constexpr bool kUnderflows = NORM && !(__is_same(T, _Float16) && (SOURCE == kPlain || (SOURCE == kResidual && __is_same(R, T))));
  const bool small = kUnderflows && a.eps < kSmallEps;
  if (small) a.most_shift = a.eps > 0.f ? std::min(126, (59 - std::ilogb(a.eps)) / 2) : 126;
  const int32_t packs = (a.size + V - 1) / V;
  // Up to four packs a lane, so that a compute unit has several rows (the limits on sizes keep all groups within
  // kMostThreads); one where there is not a row for every compute unit.
  const bool few = a.rows < compute_units() && power_of_two(packs) * a.groups <= kMostThreads;
  a.lanes = power_of_two(few ? packs : (packs + 3) / 4);
  const int32_t threads = a.lanes * a.groups;
  a.per_block = threads >= 256 ? 1 : 256 / threads;
  const int32_t block = (threads * a.per_block + kWave - 1) / kWave * kWave;
  const int64_t items = (a.rows + a.per_block - 1) / a.per_block;
  const int64_t most = int64_t(compute_units()) * (2048 / block);
  const dim3 grid(uint32_t(items < most ? items : most));
  const int32_t slots = (packs + a.lanes - 1) / a.lanes;
  if (small) norm_kernel<T, R, SOURCE, NORM, OUT, 4, PAST, kUnderflows><<<grid, block, 0, stream>>>(a);
  else if (slots <= 1) norm_kernel<T, R, SOURCE, NORM, OUT, 1, PAST, false><<<grid, block, 0, stream>>>(a);
  else if (slots <= 2) norm_kernel<T, R, SOURCE, NORM, OUT, 2, PAST, false><<<grid, block, 0, stream>>>(a);
  else norm_kernel<T, R, SOURCE, NORM, OUT, 4, PAST, false><<<grid, block, 0, stream>>>(a);
  return hipGetLastError();
}

template <typename T, typename R, int SOURCE, bool NORM, int OUT>
hipError_t launch_past(const NormArgs& a, hipStream_t stream) {
  const int64_t per = sizeof(T) + (OUT == kValues ? sizeof(T) : 1) +
                      (SOURCE == kGate ? sizeof(T) : SOURCE == kResidual ? 2 * sizeof(R) : 0);
  if (a.rows * a.channels * per > kInfinityCache) return launch_slots<T, R, SOURCE, NORM, OUT, true>(a, stream);
  return launch_slots<T, R, SOURCE, NORM, OUT, false>(a, stream);
}

template <typename T, typename R, int SOURCE>
hipError_t launch_output(const NormArgs& a, hipStream_t stream) {
  if (a.out != nullptr) return launch_past<T, R, SOURCE, true, kValues>(a, stream);
  if (a.scale != nullptr) return launch_past<T, R, SOURCE, true, kDynamic>(a, stream);
  return launch_past<T, R, SOURCE, true, kStatic>(a, stream);
}

template <typename T>
hipError_t launch_source(const NormArgs& a, hipStream_t stream) {
  if (a.weight == nullptr) return launch_past<T, T, kPlain, false, kDynamic>(a, stream);
  if (a.gate != nullptr) return launch_output<T, T, kGate>(a, stream);
  if (a.residual == nullptr) return launch_output<T, T, kPlain>(a, stream);
  if (a.residual_dtype == a.dtype) return launch_output<T, T, kResidual>(a, stream);
  return launch_output<T, float, kResidual>(a, stream);
}

template <typename T>
hipError_t launch_values(const int8_t* codes, const float* scale, void* x, int64_t rows, int32_t channels,
                         hipStream_t stream) {
  const int32_t packs = int32_t((int64_t(channels) + V - 1) / V);
  const int32_t lanes = packs >= 256 ? 256 : power_of_two(packs);
  const int64_t items = (rows + 256 / lanes - 1) / (256 / lanes), most = int64_t(compute_units()) * 16;
  const dim3 grid(uint32_t(items < most ? items : most));
  T* to = static_cast<T*>(x);
  if (rows * channels * int64_t(1 + sizeof(T)) > kInfinityCache)
    dequantize_rows_kernel<T, true><<<grid, 256, 0, stream>>>(codes, scale, to, rows, channels, lanes);
  else
    dequantize_rows_kernel<T, false><<<grid, 256, 0, stream>>>(codes, scale, to, rows, channels, lanes);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t stream) {
  switch (a.dtype) {
    case SSDQ_DTYPE_F32: return launch_source<float>(a, stream);
    case SSDQ_DTYPE_F16: return launch_source<_Float16>(a, stream);
    default: return launch_source<__bf16>(a, stream);
  }
}

hipError_t launch_dequantize_rows(int32_t dtype, const int8_t* codes, const float* scale, void* x, int64_t rows,
                                  int32_t channels, hipStream_t stream) {
  switch (dtype) {
    case SSDQ_DTYPE_F32: return launch_values<float>(codes, scale, x, rows, channels, stream);
    case SSDQ_DTYPE_F16: return launch_values<_Float16>(codes, scale, x, rows, channels, stream);
    default: return launch_values<__bf16>(codes, scale, x, rows, channels, stream);
  }
}

}  // namespace ssdq
