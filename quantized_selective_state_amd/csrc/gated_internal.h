// What the gated scan and the activation checkpoints share between the C ABI and their kernels.
#pragma once

#include "ssdq_internal.h"

namespace ssdq {

// Gated scan and its gradient after validation (pointers as in the public calls; unused ones null).
struct GatedArgs {
  int32_t dtype, gate_kind;
  const void* gate;
  const void* u;
  const float* h0;
  const int32_t* offsets;
  void* h;            // forward: written; backward: the saved states or nullptr
  float* h_final;
  int8_t* codes;      // forward: written or nullptr; backward: read or nullptr
  float* scale;
  const void* dh;
  const float* dh_final;
  void* dgate;
  void* du;
  float* dh0;
  int32_t sequences;
  int64_t tokens;
  int32_t channels;
  void* workspace;
};
size_t gated_workspace_bytes(int32_t sequences, int64_t tokens, int32_t channels, bool packed);
hipError_t launch_gated_scan(const GatedArgs& a, hipStream_t stream);
hipError_t launch_gated_backward(const GatedArgs& a, hipStream_t stream);
hipError_t launch_gated_step(int32_t dtype, int32_t gate_kind, float* state, const void* gate, const void* u, void* h,
                             int64_t n, hipStream_t stream);
hipError_t launch_checkpoint_save(int32_t dtype, const void* x, int8_t* codes, float* scale, int64_t rows,
                                  int32_t channels, hipStream_t stream);
hipError_t launch_checkpoint_load(int32_t dtype, const int8_t* codes, const float* scale, void* x, int64_t rows,
                                  int32_t channels, hipStream_t stream);

}  // namespace ssdq
