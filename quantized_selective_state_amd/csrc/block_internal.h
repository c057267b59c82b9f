// What the block's norms, its 8-bit product and the selective scan share between the C ABI and their kernels.
#pragma once

#include "ssdq_internal.h"

namespace ssdq {

// Compute units of the current device.
int32_t compute_units();

// ssdq_rms_norm, ssdq_quantize_rows after validation (weight null: no norm).
struct NormArgs {
  int32_t dtype, residual_dtype;
  const void* x;
  const void* residual;
  const void* gate;
  const float* weight;
  const float* static_scale;
  void* out;
  int8_t* codes;
  float* scale;
  void* residual_out;
  int64_t rows;
  int32_t channels, groups;
  float eps;
};
hipError_t launch_norm(const NormArgs& a, hipStream_t stream);
hipError_t launch_dequantize_rows(int32_t dtype, const int8_t* codes, const float* scale, void* x, int64_t rows,
                                  int32_t channels, hipStream_t stream);

struct MatmulArgs {
  int32_t dtype;
  const int8_t* a;
  const float* a_scale;
  bool per_row;
  const int8_t* b;
  const float* b_scale;
  const float* bias;
  void* out;
  int64_t m;
  int32_t k, n;
};
hipError_t launch_matmul_i8(const MatmulArgs& a, hipStream_t stream);
int32_t matmul_i8_plan(int64_t m, int32_t k, int32_t n);   // of valid sizes, m > 0

struct ConvArgs {
  int32_t dtype;
  const void* x;
  const float* weight;
  const float* bias;
  const void* state;
  const int32_t* offsets;
  void* out;
  void* state_out;
  int32_t sequences;
  int64_t tokens;
  int32_t channels, width;
  bool silu;
};
hipError_t launch_causal_conv(const ConvArgs& a, hipStream_t stream);
hipError_t launch_causal_conv_step(int32_t dtype, void* state, const void* x, const float* weight, const float* bias,
                                   void* out, int32_t batch, int32_t channels, int32_t width, bool silu,
                                   hipStream_t stream);

struct SelectiveArgs {
  int32_t dtype;
  const void* u;
  const void* delta;
  const float* A;
  const void* B;
  const void* C;
  const float* D;
  const void* z;
  const float* delta_bias;
  const float* h0;
  const int32_t* offsets;
  void* y;
  float* h_final;
  int32_t sequences;
  int64_t tokens;
  int32_t channels, dstate;
  bool softplus;
  void* workspace;
};
// 0: sizes that the kernels do not take
size_t selective_workspace_bytes(int32_t sequences, int64_t tokens, int32_t channels, int32_t dstate, bool packed);
int32_t selective_scan_plan(int32_t sequences, int64_t tokens, int32_t channels, int32_t dstate, bool packed);   // of such
int32_t selective_step_plan(int32_t batch, int32_t channels, int32_t dstate);   // of valid sizes
hipError_t launch_selective_scan(const SelectiveArgs& a, hipStream_t stream);
hipError_t launch_selective_step(int32_t dtype, float* state, const void* u, const void* delta, const float* A,
                                 const void* B, const void* C, const float* D, const void* z, const float* delta_bias,
                                 void* y, int32_t batch, int32_t channels, int32_t dstate, bool softplus,
                                 hipStream_t stream);

}  // namespace ssdq
