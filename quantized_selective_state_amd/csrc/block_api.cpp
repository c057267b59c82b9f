// C ABI of the block's norms, its 8-bit product and the selective scan: validation on the host, then one launcher each.
// No HIP runtime call is made before every argument has been validated.
#include <math.h>
#include <stdint.h>

#include "block_internal.h"

namespace ssdq {

int32_t compute_units() {
  int device = 0, count = 0;
  if (hipGetDevice(&device) != hipSuccess ||
      hipDeviceGetAttribute(&count, hipDeviceAttributeMultiprocessorCount, device) != hipSuccess || count <= 0)
    return 256;
  return count;
}

}  // namespace ssdq

using namespace ssdq;

namespace {

bool ok_ptr(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool ok_opt(const void* p) { return p == nullptr || ok_ptr(p); }
bool ok_dtype(int32_t d) { return d == SSDQ_DTYPE_F32 || d == SSDQ_DTYPE_F16 || d == SSDQ_DTYPE_BF16; }
ssdq_status launched(hipError_t e) { return e == hipSuccess ? SSDQ_SUCCESS : SSDQ_ERROR_LAUNCH; }

constexpr int64_t kMostRows = (int64_t(1) << 31) - (int64_t(1) << 16);   // rows in 32 bits, a tile past the end too
constexpr int32_t kMostSequences = 1 << 24;
constexpr int32_t kMostChannels = 1 << 20;

ssdq_status check_sequences(int32_t sequences, int64_t tokens, int32_t channels, bool packed) {
  if (sequences <= 0 || tokens < 0 || channels <= 0) return SSDQ_ERROR_INVALID_VALUE;
  if (!packed && tokens % sequences != 0) return SSDQ_ERROR_INVALID_VALUE;
  if (tokens >= kMostRows || sequences >= kMostSequences || channels > kMostChannels) return SSDQ_ERROR_UNSUPPORTED;
  return SSDQ_SUCCESS;
}

ssdq_status check_selective(int32_t sequences, int64_t tokens, int32_t channels, int32_t dstate, bool packed) {
  if (dstate <= 0) return SSDQ_ERROR_INVALID_VALUE;
  const ssdq_status st = check_sequences(sequences, tokens, channels, packed);
  if (st != SSDQ_SUCCESS) return st;
  if (dstate > 64 || selective_workspace_bytes(sequences, tokens, channels, dstate, packed) == 0)
    return SSDQ_ERROR_UNSUPPORTED;
  return SSDQ_SUCCESS;
}

bool ok_matmul(int64_t m, int32_t k, int32_t n) {
  // a grid's threads in 32 bits, at 256 for each 128 x 128 of out
  return k <= 131071 && m < kMostRows && ((m + 127) / 128) * ((int64_t(n) + 127) / 128) < (int64_t(1) << 24);
}

bool ok_selective_step(int32_t batch, int32_t channels, int32_t dstate) {
  // a grid's threads in 32 bits, at up to 256 for each 16 channels
  return dstate <= 64 && (int64_t(channels) + 15) / 16 * batch < int64_t(1) << 24;
}

}  // namespace

extern "C" {

ssdq_status ssdq_rms_norm(int32_t dtype, int32_t residual_dtype, const void* x, const void* residual, const void* gate,
                          const float* weight, const float* static_scale, void* out, int8_t* codes, float* scale,
                          void* residual_out, int64_t rows, int32_t channels, int32_t groups, float eps,
                          hipStream_t stream) {
  if (!ok_dtype(dtype) || (residual_dtype != dtype && residual_dtype != SSDQ_DTYPE_F32) || rows < 0 || channels <= 0 ||
      groups <= 0 || channels % groups != 0 || !(eps >= 0.f) || isinf(eps))
    return SSDQ_ERROR_INVALID_VALUE;
  if (rows >= (int64_t(1) << 31) || groups > 256 || channels > (groups == 1 ? 32768 : 16384))
    return SSDQ_ERROR_UNSUPPORTED;
  if (rows == 0) return SSDQ_SUCCESS;
  if (!ok_ptr(x) || !ok_ptr(weight) || !ok_opt(residual) || !ok_opt(residual_out) || !ok_opt(gate) || !ok_opt(out) ||
      !ok_opt(codes) || !ok_opt(scale) || !ok_opt(static_scale))
    return SSDQ_ERROR_INVALID_VALUE;
  if ((residual == nullptr) != (residual_out == nullptr) || (residual != nullptr && gate != nullptr))
    return SSDQ_ERROR_INVALID_VALUE;
  if ((out == nullptr) == (codes == nullptr)) return SSDQ_ERROR_INVALID_VALUE;
  // codes go with exactly one of the two scales, out with neither
  if (int(scale != nullptr) + int(static_scale != nullptr) != int(codes != nullptr)) return SSDQ_ERROR_INVALID_VALUE;
  NormArgs a = {};
  a.dtype = dtype;
  a.residual_dtype = residual_dtype;
  a.x = x;
  a.residual = residual;
  a.gate = gate;
  a.weight = weight;
  a.static_scale = static_scale;
  a.out = out;
  a.codes = codes;
  a.scale = scale;
  a.residual_out = residual_out;
  a.rows = rows;
  a.channels = channels;
  a.groups = groups;
  a.eps = eps;
  return launched(launch_norm(a, stream));
}

ssdq_status ssdq_quantize_rows(int32_t dtype, const void* x, int8_t* codes, float* scale, int64_t rows,
                               int32_t channels, hipStream_t stream) {
  if (!ok_dtype(dtype) || rows < 0 || channels <= 0) return SSDQ_ERROR_INVALID_VALUE;
  if (rows >= (int64_t(1) << 31) || channels > 32768) return SSDQ_ERROR_UNSUPPORTED;
  if (rows == 0) return SSDQ_SUCCESS;
  if (!ok_ptr(x) || !ok_ptr(codes) || !ok_ptr(scale)) return SSDQ_ERROR_INVALID_VALUE;
  NormArgs a = {};
  a.dtype = dtype;
  a.residual_dtype = dtype;
  a.x = x;
  a.codes = codes;
  a.scale = scale;
  a.rows = rows;
  a.channels = channels;
  a.groups = 1;
  return launched(launch_norm(a, stream));
}

ssdq_status ssdq_dequantize_rows(int32_t dtype, const int8_t* codes, const float* scale, void* x, int64_t rows,
                                 int32_t channels, hipStream_t stream) {
  if (!ok_dtype(dtype) || rows < 0 || channels <= 0) return SSDQ_ERROR_INVALID_VALUE;
  if (rows >= (int64_t(1) << 31)) return SSDQ_ERROR_UNSUPPORTED;
  if (rows == 0) return SSDQ_SUCCESS;
  if (!ok_ptr(x) || !ok_ptr(codes) || !ok_ptr(scale)) return SSDQ_ERROR_INVALID_VALUE;
  return launched(launch_dequantize_rows(dtype, codes, scale, x, rows, channels, stream));
}

ssdq_status ssdq_matmul_i8(int32_t dtype, const int8_t* a, const float* a_scale, int32_t a_scale_per_row,
                           const int8_t* b, const float* b_scale, const float* bias, void* out, int64_t m, int32_t k,
                           int32_t n, hipStream_t stream) {
  if (!ok_dtype(dtype) || m < 0 || k <= 0 || n <= 0) return SSDQ_ERROR_INVALID_VALUE;
  if (!ok_matmul(m, k, n)) return SSDQ_ERROR_UNSUPPORTED;
  if (m == 0) return SSDQ_SUCCESS;
  if (!ok_ptr(a) || !ok_ptr(a_scale) || !ok_ptr(b) || !ok_ptr(b_scale) || !ok_opt(bias) || !ok_ptr(out))
    return SSDQ_ERROR_INVALID_VALUE;
  const MatmulArgs args = {dtype, a, a_scale, a_scale_per_row != 0, b, b_scale, bias, out, m, k, n};
  return launched(launch_matmul_i8(args, stream));
}

int32_t ssdq_matmul_i8_plan(int64_t m, int32_t k, int32_t n) {
  return m > 0 && k > 0 && n > 0 && ok_matmul(m, k, n) ? matmul_i8_plan(m, k, n) : -1;
}

ssdq_status ssdq_causal_conv(int32_t dtype, const void* x, const float* weight, const float* bias, const void* state,
                             const int32_t* offsets, void* out, void* state_out, int32_t sequences, int64_t tokens,
                             int32_t channels, int32_t width, int32_t silu, hipStream_t stream) {
  if (!ok_dtype(dtype) || width < 2 || width > 4) return SSDQ_ERROR_INVALID_VALUE;
  const ssdq_status st = check_sequences(sequences, tokens, channels, offsets != nullptr);
  if (st != SSDQ_SUCCESS) return st;
  // a grid's threads in 31 bits, at 64 for each 16 rows x 256 channels and for each sequence's state
  if ((int64_t(channels) + 255) / 256 * (sequences + tokens / 16 + 1) >= int64_t(1) << 25) return SSDQ_ERROR_UNSUPPORTED;
  if (!ok_ptr(weight) || !ok_opt(bias) || !ok_opt(state) || !ok_opt(offsets) || !ok_opt(state_out))
    return SSDQ_ERROR_INVALID_VALUE;
  if (tokens > 0 && (!ok_ptr(x) || !ok_ptr(out))) return SSDQ_ERROR_INVALID_VALUE;
  // neighbouring waves read the rows ahead of their own
  if ((tokens > 0 && x == out) || (state != nullptr && state == state_out)) return SSDQ_ERROR_INVALID_VALUE;
  const ConvArgs a = {dtype, x, weight, bias, state, offsets, out, state_out, sequences, tokens, channels, width,
                      silu != 0};
  return launched(launch_causal_conv(a, stream));
}

ssdq_status ssdq_causal_conv_step(int32_t dtype, void* state, const void* x, const float* weight, const float* bias,
                                  void* out, int32_t batch, int32_t channels, int32_t width, int32_t silu,
                                  hipStream_t stream) {
  if (!ok_dtype(dtype) || width < 2 || width > 4 || batch <= 0 || channels <= 0) return SSDQ_ERROR_INVALID_VALUE;
  if (int64_t(batch) * channels >= (int64_t(1) << 31)) return SSDQ_ERROR_UNSUPPORTED;
  if (!ok_ptr(state) || !ok_ptr(x) || !ok_ptr(weight) || !ok_opt(bias) || !ok_ptr(out)) return SSDQ_ERROR_INVALID_VALUE;
  return launched(launch_causal_conv_step(dtype, state, x, weight, bias, out, batch, channels, width, silu != 0, stream));
}

size_t ssdq_selective_scan_workspace_size(int32_t sequences, int64_t tokens, int32_t channels, int32_t dstate,
                                          int32_t packed) {
  if (check_selective(sequences, tokens, channels, dstate, packed != 0) != SSDQ_SUCCESS) return 0;
  return selective_workspace_bytes(sequences, tokens, channels, dstate, packed != 0);
}

int32_t ssdq_selective_scan_plan(int32_t sequences, int64_t tokens, int32_t channels, int32_t dstate, int32_t packed) {
  if (check_selective(sequences, tokens, channels, dstate, packed != 0) != SSDQ_SUCCESS) return -1;
  return selective_scan_plan(sequences, tokens, channels, dstate, packed != 0);
}

ssdq_status ssdq_selective_scan(int32_t dtype, const void* u, const void* delta, const float* A, const void* B,
                                const void* C, const float* D, const void* z, const float* delta_bias, const float* h0,
                                const int32_t* offsets, void* y, float* h_final, int32_t sequences, int64_t tokens,
                                int32_t channels, int32_t dstate, int32_t softplus, void* workspace,
                                size_t workspace_bytes, hipStream_t stream) {
  if (!ok_dtype(dtype)) return SSDQ_ERROR_INVALID_VALUE;
  const ssdq_status st = check_selective(sequences, tokens, channels, dstate, offsets != nullptr);
  if (st != SSDQ_SUCCESS) return st;
  if (!ok_ptr(A) || !ok_opt(D) || !ok_opt(delta_bias) || !ok_opt(h0) || !ok_opt(offsets) || !ok_opt(h_final) ||
      !ok_ptr(workspace))
    return SSDQ_ERROR_INVALID_VALUE;
  if (tokens > 0 && (!ok_ptr(u) || !ok_ptr(delta) || !ok_ptr(B) || !ok_ptr(C) || !ok_opt(z) || !ok_ptr(y)))
    return SSDQ_ERROR_INVALID_VALUE;
  if (h0 != nullptr && h0 == h_final) return SSDQ_ERROR_INVALID_VALUE;
  if (workspace_bytes < selective_workspace_bytes(sequences, tokens, channels, dstate, offsets != nullptr))
    return SSDQ_ERROR_WORKSPACE_TOO_SMALL;
  const SelectiveArgs a = {dtype, u, delta, A, B, C, D, z, delta_bias, h0, offsets, y, h_final, sequences, tokens,
                           channels, dstate, softplus != 0, workspace};
  return launched(launch_selective_scan(a, stream));
}

ssdq_status ssdq_selective_step(int32_t dtype, float* state, const void* u, const void* delta, const float* A,
                                const void* B, const void* C, const float* D, const void* z, const float* delta_bias,
                                void* y, int32_t batch, int32_t channels, int32_t dstate, int32_t softplus,
                                hipStream_t stream) {
  if (!ok_dtype(dtype) || batch <= 0 || channels <= 0 || dstate <= 0) return SSDQ_ERROR_INVALID_VALUE;
  if (!ok_selective_step(batch, channels, dstate)) return SSDQ_ERROR_UNSUPPORTED;
  if (!ok_ptr(state) || !ok_ptr(u) || !ok_ptr(delta) || !ok_ptr(A) || !ok_ptr(B) || !ok_ptr(C) || !ok_opt(D) ||
      !ok_opt(z) || !ok_opt(delta_bias) || !ok_ptr(y))
    return SSDQ_ERROR_INVALID_VALUE;
  return launched(launch_selective_step(dtype, state, u, delta, A, B, C, D, z, delta_bias, y, batch, channels, dstate,
                                        softplus != 0, stream));
}

int32_t ssdq_selective_step_plan(int32_t batch, int32_t channels, int32_t dstate) {
  if (batch <= 0 || channels <= 0 || dstate <= 0 || !ok_selective_step(batch, channels, dstate)) return -1;
  return selective_step_plan(batch, channels, dstate);
}

}  // extern "C"
