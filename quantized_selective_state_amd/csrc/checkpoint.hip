// 8-bit activation checkpoints: codes and one scale per 64 channels of a row, and their values.
#include "gated_types.h"

namespace ssdq {
namespace {

constexpr int kBlock = SSDQ_CHECKPOINT_BLOCK;
constexpr int64_t kMostBlocks = 1 << 20;   // further work is reached by striding (a grid holds 2^32 threads)

// One wave per block of 64 channels, a lane per channel.
template <typename T>
__global__ void __launch_bounds__(256) checkpoint_save_kernel(const T* x, int8_t* codes, float* scale, int64_t rows,
                                                              int32_t channels, int32_t blocks) {
  for (int64_t w = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6); w < rows * blocks; w += int64_t(gridDim.x) * 4) {
    const int64_t row = w / blocks;
    const int c = int(w - row * blocks) * kBlock + int(threadIdx.x & 63);
    const bool in = c < channels;
    const float v = in ? to_f32(x[row * channels + c]) : 0.f;
    uint32_t most = __float_as_uint(fabsf(v));
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) most = max(most, uint32_t(__shfl_xor(int(most), o, 64)));
    const float s = checkpoint_scale(most);
    if (in) codes[row * channels + c] = int8_t(code_of(v, code_scale(s)));
    if ((threadIdx.x & 63) == 0) scale[w] = s;
  }
}

template <typename T>
__global__ void __launch_bounds__(256) checkpoint_load_kernel(const int8_t* codes, const float* scale, T* x,
                                                              int64_t rows, int32_t channels, int32_t blocks) {
  for (int64_t w = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6); w < rows * blocks; w += int64_t(gridDim.x) * 4) {
    const int64_t row = w / blocks;
    const int c = int(w - row * blocks) * kBlock + int(threadIdx.x & 63);
    if (c < channels) x[row * channels + c] = from_f32<T>(float(codes[row * channels + c]) * scale[w]);
  }
}

template <typename T>
hipError_t save(const void* x, int8_t* codes, float* scale, int64_t rows, int32_t channels, hipStream_t stream) {
  const int32_t blocks = (channels + kBlock - 1) / kBlock;
  hipLaunchKernelGGL((checkpoint_save_kernel<T>), dim3(uint32_t(min((rows * blocks + 3) / 4, kMostBlocks))), dim3(256), 0, stream,
                     static_cast<const T*>(x), codes, scale, rows, channels, blocks);
  return hipGetLastError();
}
template <typename T>
hipError_t load(const int8_t* codes, const float* scale, void* x, int64_t rows, int32_t channels, hipStream_t stream) {
  const int32_t blocks = (channels + kBlock - 1) / kBlock;
  hipLaunchKernelGGL((checkpoint_load_kernel<T>), dim3(uint32_t(min((rows * blocks + 3) / 4, kMostBlocks))), dim3(256), 0, stream, codes,
                     scale, static_cast<T*>(x), rows, channels, blocks);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_checkpoint_save(int32_t dtype, const void* x, int8_t* codes, float* scale, int64_t rows,
                                  int32_t channels, hipStream_t stream) {
  if (dtype == SSDQ_DTYPE_F32) return save<float>(x, codes, scale, rows, channels, stream);
  if (dtype == SSDQ_DTYPE_F16) return save<_Float16>(x, codes, scale, rows, channels, stream);
  return save<__bf16>(x, codes, scale, rows, channels, stream);
}
hipError_t launch_checkpoint_load(int32_t dtype, const int8_t* codes, const float* scale, void* x, int64_t rows,
                                  int32_t channels, hipStream_t stream) {
  if (dtype == SSDQ_DTYPE_F32) return load<float>(codes, scale, x, rows, channels, stream);
  if (dtype == SSDQ_DTYPE_F16) return load<_Float16>(codes, scale, x, rows, channels, stream);
  return load<__bf16>(codes, scale, x, rows, channels, stream);
}

}  // namespace ssdq
