// 8-bit activation checkpoints: codes and one scale per 64 channels of a row, and their values.
//
// HBM-bound: 2 or 4 bytes in and 1 + 1/16 out per element, or the other way (8192 x 4096 bf16: both together 39 us,
// 5.3 TB/s; one channel per lane and one block per wave took 158; a row length that 8 does not divide, one channel per
// lane and four blocks in flight, takes 61 and 33 us at 8192 x 4095).  An item is one block of
// 64 channels of a row.  Its 64 / V lanes hold V neighbouring channels each (16 bytes of x, where the
// row length is a multiple of V: else one channel per lane), take the block's largest magnitude over the
// lanes in registers, and a thread has the loads of kItems items in flight before it works on the first.
#include "gated_types.h"

namespace ssdq {
namespace {

constexpr int kBlock = SSDQ_CHECKPOINT_BLOCK;
constexpr int kThreads = 256;
constexpr int kItems = 4;
constexpr int64_t kMostItems = int64_t(1) << 27;   // of one launch: 16 threads each where rows are ragged, 2^31 in all

// the channels of lane `col` and item number of its k-th item; an item past the end has no channels
template <int V>
struct Place {
  uint32_t item;
  int64_t at;    // element offset of the lane's first channel
  bool in;
  __device__ __forceinline__ Place(int k, uint32_t items, FastDiv blocks, int32_t channels) {
    constexpr int LPR = kBlock / V, kPer = kThreads / LPR;   // items side by side in a block of threads
    item = (blockIdx.x * kItems + uint32_t(k)) * kPer + threadIdx.x / LPR;
    const uint32_t row = fdiv(item, blocks);
    const int32_t c = int32_t(item - row * blocks.d) * kBlock + int32_t(threadIdx.x % LPR) * V;
    in = item < items && c < channels;
    at = int64_t(row) * channels + c;
  }
};

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) checkpoint_save_kernel(const T* __restrict__ x, int8_t* __restrict__ codes,
                                                                   float* __restrict__ scale, uint32_t items,
                                                                   FastDiv blocks, int32_t channels) {
  constexpr int LPR = kBlock / V;
  typedef typename Bytes<sizeof(T) * V>::type Raw;
  Raw raw[kItems];
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const Place<V> p(k, items, blocks, channels);
    raw[k] = Raw{};
    if (p.in) raw[k] = *reinterpret_cast<const Raw*>(x + p.at);
  }
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const Place<V> p(k, items, blocks, channels);
    const Pack<T, V> v{raw[k]};
    const float s = checkpoint_scale(row_umax<LPR>(largest<T, V>(v, V)));   // (elements past the row are 0)
    if (p.in) *reinterpret_cast<typename Bytes<V>::type*>(codes + p.at) = codes_of<V>(v, s);
    if (threadIdx.x % LPR == 0 && p.item < items) scale[p.item] = s;
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) checkpoint_load_kernel(const int8_t* __restrict__ codes,
                                                                   const float* __restrict__ scale, T* __restrict__ x,
                                                                   uint32_t items, FastDiv blocks, int32_t channels) {
  typedef typename Bytes<V>::type Raw;
  Raw raw[kItems];
  float s[kItems];
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const Place<V> p(k, items, blocks, channels);
    raw[k] = Raw{};
    s[k] = 0.f;
    if (p.in) {
      raw[k] = *reinterpret_cast<const Raw*>(codes + p.at);
      s[k] = scale[p.item];
    }
  }
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const Place<V> p(k, items, blocks, channels);
    const Pack<int8_t, V> q{raw[k]};
    struct { T e[V]; } out;
#pragma unroll
    for (int e = 0; e < V; ++e) out.e[e] = from_f32<T>(q[e] * s[k]);
    if (p.in) {
      if constexpr (sizeof(out) > 16) {   // 8 values of 4 bytes: two stores
        const auto half = __builtin_bit_cast(Halves, out);
        reinterpret_cast<v4u*>(x + p.at)[0] = half.h[0];
        reinterpret_cast<v4u*>(x + p.at)[1] = half.h[1];
      } else {
        *reinterpret_cast<typename Bytes<sizeof(out)>::type*>(x + p.at) =
            __builtin_bit_cast(typename Bytes<sizeof(out)>::type, out);
      }
    }
  }
}

// f(rows of this launch, row offset) over as many launches as the threads need: one, but for more than 2^27 blocks
// of 64 channels
template <typename F>
hipError_t over_rows(int64_t rows, int32_t blocks, F f) {
  const int64_t most = kMostItems / blocks > 0 ? kMostItems / blocks : 1;
  for (int64_t r = 0; r < rows; r += most) {
    f(rows - r < most ? rows - r : most, r);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// blocks of a row: up to 2^25 (channels + 63 may pass 31 bits)
constexpr int32_t blocks_of(int32_t channels) { return int32_t((int64_t(channels) + kBlock - 1) / kBlock); }
static_assert(blocks_of(0x7FFFFFFF) == 1 << 25 && blocks_of(65) == 2, "any row length has its blocks");

template <int V>
dim3 grid_of(int64_t items) {
  constexpr int64_t kPer = int64_t(kItems) * kThreads / (kBlock / V);
  return dim3(uint32_t((items + kPer - 1) / kPer));
}

template <typename T, int V>
hipError_t save(const void* x, int8_t* codes, float* scale, int64_t rows, int32_t channels, hipStream_t stream) {
  const int32_t blocks = blocks_of(channels);
  return over_rows(rows, blocks, [&](int64_t n, int64_t r) {
    hipLaunchKernelGGL((checkpoint_save_kernel<T, V>), grid_of<V>(n * blocks), dim3(kThreads), 0, stream,
                       static_cast<const T*>(x) + r * channels, codes + r * channels, scale + r * blocks,
                       uint32_t(n * blocks), make_fastdiv(uint32_t(blocks)), channels);
  });
}
template <typename T, int V>
hipError_t load(const int8_t* codes, const float* scale, void* x, int64_t rows, int32_t channels, hipStream_t stream) {
  const int32_t blocks = blocks_of(channels);
  return over_rows(rows, blocks, [&](int64_t n, int64_t r) {
    hipLaunchKernelGGL((checkpoint_load_kernel<T, V>), grid_of<V>(n * blocks), dim3(kThreads), 0, stream,
                       codes + r * channels, scale + r * blocks, static_cast<T*>(x) + r * channels,
                       uint32_t(n * blocks), make_fastdiv(uint32_t(blocks)), channels);
  });
}

template <typename T>
hipError_t save_any(const void* x, int8_t* codes, float* scale, int64_t rows, int32_t channels, hipStream_t stream) {
  constexpr int V = 16 / int(sizeof(T));
  return channels % V == 0 ? save<T, V>(x, codes, scale, rows, channels, stream)
                           : save<T, 1>(x, codes, scale, rows, channels, stream);
}
template <typename T>
hipError_t load_any(const int8_t* codes, const float* scale, void* x, int64_t rows, int32_t channels,
                    hipStream_t stream) {
  return channels % 8 == 0 ? load<T, 8>(codes, scale, x, rows, channels, stream)
                           : load<T, 1>(codes, scale, x, rows, channels, stream);
}

}  // namespace

hipError_t launch_checkpoint_save(int32_t dtype, const void* x, int8_t* codes, float* scale, int64_t rows,
                                  int32_t channels, hipStream_t stream) {
  if (dtype == SSDQ_DTYPE_F32) return save_any<float>(x, codes, scale, rows, channels, stream);
  if (dtype == SSDQ_DTYPE_F16) return save_any<_Float16>(x, codes, scale, rows, channels, stream);
  return save_any<__bf16>(x, codes, scale, rows, channels, stream);
}
hipError_t launch_checkpoint_load(int32_t dtype, const int8_t* codes, const float* scale, void* x, int64_t rows,
                                  int32_t channels, hipStream_t stream) {
  if (dtype == SSDQ_DTYPE_F32) return load_any<float>(codes, scale, x, rows, channels, stream);
  if (dtype == SSDQ_DTYPE_F16) return load_any<_Float16>(codes, scale, x, rows, channels, stream);
  return load_any<__bf16>(codes, scale, x, rows, channels, stream);
}

}  // namespace ssdq
