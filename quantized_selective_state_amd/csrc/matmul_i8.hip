// Matrix product of 8-bit codes with a scale per token and per output channel, on INT8 MFMA.
//
// Both operands have their inner axis contiguous, as the matrix instructions take them (a lane's 16 codes are
// neighbours).  The weights are the instruction's first operand, so that a lane of the result holds 4 neighbouring output
// channels of one token and stores them together.
#include "block_internal.h"
#include "gated_types.h"

namespace ssdq {
namespace {

struct Epilogue {
  const float* a_scale;
  const float* b_scale;
  const float* bias;
  bool per_row;
};

// (float(sum) * a_scale) * b_scale + bias
__device__ __forceinline__ float finish(int32_t sum, float sa, float sb, float bias) {
  return fmaf(float(sum) * sa, sb, bias);
}

// 128 x 128 tiles over any sizes: rows may start at any byte, and a row's last codes are loaded one by one.
constexpr int kTile = 128, kDepth = 64, kThreads = 256;

__device__ __forceinline__ v4i load_codes(const int8_t* __restrict__ row, int32_t k, int32_t depth) {
  v4i r = {0, 0, 0, 0};
  if (k + 16 <= depth) {
    __builtin_memcpy(&r, row + k, 16);
  } else if (k < depth) {
    int8_t e[16] = {};
    for (int i = 0; i < 16; ++i)
      if (k + i < depth) e[i] = row[k + i];
    __builtin_memcpy(&r, e, 16);
  }
  return r;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) matmul_kernel(const int8_t* __restrict__ a, const int8_t* __restrict__ b,
                                                          Epilogue ep, T* __restrict__ out, int64_t m, int32_t k,
                                                          int32_t n, int32_t n_tiles) {
  __shared__ v4i as[kTile][4], bs[kTile][4];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int64_t m0 = int64_t(blockIdx.x / n_tiles) * kTile;
  const int32_t n0 = int32_t(blockIdx.x % n_tiles) * kTile;
  const int wm = (wave & 1) * 64, wn = (wave >> 1) * 64;
  v4i acc[4][4] = {};   // [n][m]
  for (int32_t k0 = 0; k0 < k; k0 += kDepth) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = int(threadIdx.x) + i * kThreads, r = at / 4, chunk = at % 4;
      v4i va = {0, 0, 0, 0}, vb = {0, 0, 0, 0};
      if (m0 + r < m) va = load_codes(a + (m0 + r) * k, k0 + chunk * 16, k);
      if (n0 + r < n) vb = load_codes(b + int64_t(n0 + r) * k, k0 + chunk * 16, k);
      as[r][chunk ^ ((r >> 1) & 3)] = va;
      bs[r][chunk ^ ((r >> 1) & 3)] = vb;
    }
    __syncthreads();
    v4i fa[4], fb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ra = wm + i * 16 + lane % 16, rb = wn + i * 16 + lane % 16;
      fa[i] = as[ra][(lane / 16) ^ ((ra >> 1) & 3)];
      fb[i] = bs[rb][(lane / 16) ^ ((rb >> 1) & 3)];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j], fa[i], acc[j][i], 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = m0 + wm + i * 16 + lane % 16;
    if (row >= m) continue;
    const float sa = ep.a_scale[ep.per_row ? row : 0];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int32_t col = n0 + wn + j * 16 + (lane / 16) * 4;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (col + e < n)
          out[row * n + col + e] = from_f32<T>(finish(acc[j][i][e], sa, ep.b_scale[col + e],
                                                      ep.bias != nullptr ? ep.bias[col + e] : 0.f));
    }
  }
}

template <typename T>
hipError_t launch(const MatmulArgs& a, hipStream_t stream) {
  const Epilogue ep = {a.a_scale, a.b_scale, a.bias, a.per_row};
  const int64_t n_tiles = (int64_t(a.n) + kTile - 1) / kTile, tiles = (a.m + kTile - 1) / kTile * n_tiles;
  matmul_kernel<T><<<dim3(uint32_t(tiles)), kThreads, 0, stream>>>(a.a, a.b, ep, static_cast<T*>(a.out), a.m, a.k, a.n,
                                                                   int32_t(n_tiles));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_matmul_i8(const MatmulArgs& a, hipStream_t stream) {
  switch (a.dtype) {
    case SSDQ_DTYPE_F32: return launch<float>(a, stream);
    case SSDQ_DTYPE_F16: return launch<_Float16>(a, stream);
    default: return launch<__bf16>(a, stream);
  }
}

}  // namespace ssdq
