/*
 * ssdq.h -- C ABI of the INT8-input Mamba-2 SSD scan for AMD MI355X (gfx950).
 *
 * The library evaluates the selective state-space recurrence of Mamba-2
 * (stated in Ternary Mamba, Section 1, as h_t = Abar_t h_{t-1} + Bbar_t x_t)
 * with the zero-order-hold decay Abar_t = exp(dt_t A_h), Bbar_t = dt_t B_t and
 * the readout y_t = C_t . h_t + D_h x_t, where x, B and C arrive as INT8 codes
 * with static scales: one fp32 scale per head for x and one per state group
 * for B and C (Quamba2 rebuttal: 8-bit SSD inputs B, C, x and per-state-group
 * quantization; SSDi8 Table 10: per-H(G) scales; Quamba project page: static
 * scales).  Prefill uses the chunked state-space-duality evaluation (SSDi8
 * abstract and Figure 1b: chunk state, chunk-level C.B^T on INT8, state
 * passing); decode is one recurrence step per call (Quamba2 rebuttal: the SSD
 * update is the decode-time latency and memory bottleneck).
 *
 * Conventions for every call:
 *  - Pointers are DEVICE pointers unless stated otherwise, must be 16-byte
 *    aligned, and address contiguous row-major tensors in the layouts given.
 *  - The caller owns every buffer, including the workspace.  The library never
 *    allocates or frees device memory, never synchronizes the device, keeps no
 *    global state and is safe to call from several host threads.
 *  - Work is enqueued asynchronously on `stream` (0 = the null stream) of the
 *    current HIP device.
 *  - Arguments are validated on the host before anything is enqueued; any
 *    status other than SSDQ_SUCCESS means nothing was enqueued.  Validation
 *    cannot read device memory, so NaN/Inf or out-of-range VALUES in device
 *    buffers are not detected (see each call for what they produce).
 *  - y (fp16) never aliases an input.  The only aliases allowed are the ones
 *    each call names.
 */
#ifndef SSDQ_H_
#define SSDQ_H_

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SSDQ_SUCCESS = 0,
  SSDQ_ERROR_INVALID_VALUE = 1,       /* null / misaligned pointer, non-positive size, H % G != 0 */
  SSDQ_ERROR_UNSUPPORTED = 2,         /* a shape the kernels do not handle (see each call) */
  SSDQ_ERROR_WORKSPACE_TOO_SMALL = 3, /* workspace_bytes below ssdq_chunk_scan_workspace_size() */
  SSDQ_ERROR_LAUNCH = 4,              /* the HIP runtime rejected a kernel launch */
  SSDQ_ERROR_SCRATCH_LIMIT = 5        /* ssdq_chunk_scan_noalloc: the shape needs more than the static scratch */
} ssdq_status;

/* Human-readable name of a status (host; static storage; never NULL). */
const char* ssdq_status_string(ssdq_status status);

/*
 * Static INT8 quantizer (the 8-bit SSD inputs of the Quamba2 rebuttal; static
 * per-head / per-group scales of SSDi8 Table 10).
 *
 *   q[r, k, i] = clamp(round_half_even(float(x[r, k, i]) / scale[k]), -127, 127)
 *
 * with the fp32 quotient correctly rounded (not a reciprocal multiply).
 * A NaN quotient gives 0 and +-Inf gives +-127; -128 is never produced.
 *   x_f16 : (rows, nscale, inner) IEEE binary16, device
 *   q     : (rows, nscale, inner) int8, device, written
 *   scale : [nscale] fp32, device (positive finite for meaningful codes)
 * Use for x (b, L, H, P): rows = b*L, nscale = H, inner = P; for B or C
 * (b, L, G, N): rows = b*L, nscale = G, inner = N.  Any rows >= 0 (0 = no-op),
 * nscale >= 1, inner >= 1.  q must not overlap x_f16.
 */
ssdq_status ssdq_quantize(const void* x_f16, int8_t* q, const float* scale, int64_t rows, int32_t nscale,
                          int32_t inner, hipStream_t stream);

/* One tensor of a batched quantize: the arguments of ssdq_quantize. */
typedef struct {
  const void* x_f16;   /* (rows, nscale, inner) IEEE binary16, device */
  int8_t* q;           /* (rows, nscale, inner) int8, device, written */
  const float* scale;  /* [nscale] fp32, device */
  int64_t rows;
  int32_t nscale;
  int32_t inner;
} ssdq_quantize_job;

#define SSDQ_QUANTIZE_MAX_JOBS 8

/*
 * The same static INT8 quantizer applied to several tensors (x, B and C of one step) in
 * one kernel launch where their shapes allow it: each job's codes equal those of
 * ssdq_quantize with the same arguments.  Jobs whose inner is a multiple of 16 share one
 * launch; any other job is launched on its own (same stream, same result).
 *   jobs  : host array of `count` jobs, read during the call only
 *   count : 1 .. SSDQ_QUANTIZE_MAX_JOBS
 * Every job is validated as ssdq_quantize validates its arguments before anything is
 * launched (one invalid job: nothing runs).  Jobs with rows == 0 are skipped.  No output
 * may overlap another job's output or any job's input.
 */
ssdq_status ssdq_quantize_batch(const ssdq_quantize_job* jobs, int32_t count, hipStream_t stream);

/*
 * The static INT8 quantizer with one scale per (k, i) instead of one per k: B or C with a scale per
 * (group, state), the finer granularity of SSDi8 Table 10 (per-P(N) together with per-H(G)), or x
 * with a scale per (head, channel) (rows = b*L, nscale = H, inner = P, scale (H, P)).
 *
 *   q[r, k, i] = clamp(round_half_even(float(x[r, k, i]) / scale[k, i]), -127, 127)
 *
 *   scale : (nscale, inner) fp32, device (each positive finite)
 * Arguments, layout, rounding, special values and validation otherwise as ssdq_quantize (B or C
 * (b, L, G, N): rows = b*L, nscale = G, inner = N, scale (G, N)); codes bit-exact to the
 * correctly rounded quotient.
 */
ssdq_status ssdq_quantize_per_channel(const void* x_f16, int8_t* q, const float* scale, int64_t rows,
                                      int32_t nscale, int32_t inner, hipStream_t stream);

/* Bytes of workspace ssdq_chunk_scan needs for this shape (host; 0 on invalid shapes).
 * Layout (stable, used by the stage-level tests), with nchunks = ceil(seqlen / chunk) and
 * each region starting at a 256-byte boundary:
 *   Acs     fp32 (batch, nheads, nchunks, chunk): within-chunk inclusive cumsum of dt * A
 *           (padded past the sequence end with the last value)           -- written by stage 0
 *   Dtc     fp32 (batch, nheads, nchunks, chunk): dt in the same chunk order, 0 past the
 *           sequence end (one contiguous row per chunk for stage 2)      -- written by stage 0
 *   S       fp32 (batch, nchunks, nheads, headdim, dstate): chunk states  -- written by stage 0
 *   Hprev   int8 (batch, nchunks, nheads, 2, headdim, dstate) and
 *   Hscale  fp32 (batch, nchunks, nheads, headdim): the state entering each chunk is
 *           (Hprev[..., 0, p, n] + Hprev[..., 1, p, n] / 256) * Hscale[..., p], two INT8
 *           limbs with a power-of-two scale per state row           -- written by stage 1
 *           Within each full 64-state block of a row, the 4 bytes of states
 *           64 blk + 16 t + 4 k + (0..3) are stored at 64 blk + 16 k + 4 t + (0..3) (a 4x4
 *           transpose of 4-byte groups: the writing lanes store 16 contiguous bytes); a
 *           partial last block (dstate % 64 != 0) is stored in natural order.
 * When ssdq_chunk_scan_state_fused(batch, nheads) is 1, stage 0 writes Acs, Dtc, Hprev, Hscale
 * (and h_final) itself, stage 1 does nothing, and S is not written. */
size_t ssdq_chunk_scan_workspace_size(int32_t batch, int64_t seqlen, int32_t nheads, int32_t headdim,
                                      int32_t dstate, int32_t chunk);

/*
 * Prefill: the chunked SSD scan over INT8 inputs (SSDi8 Figure 1b pipeline).
 *
 *   for every (b, h):  h_{-1} = h0[b, h] (or 0),
 *     h_t = exp(dt[b,t,h] A[h]) h_{t-1} + dt[b,t,h] * xhat[b,t,h,:] (x) Bhat[b,t,g,:]
 *     y[b,t,h,:] = h_t . Chat[b,t,g,:] + D[h] * xhat[b,t,h,:]
 *   with xhat = x_scale[h] * x, Bhat = B_scale[g] * B, Chat = C_scale[g] * C and
 *   g = h / (nheads / ngroups).
 *
 *   x  : (batch, seqlen, nheads, headdim) int8      x_scale : [nheads] fp32
 *   B  : (batch, seqlen, ngroups, dstate) int8      B_scale : [ngroups] fp32
 *   C  : (batch, seqlen, ngroups, dstate) int8      C_scale : [ngroups] fp32
 *   (every scale finite and > 0: the output kernel divides by them, and a zero or non-finite
 *   scale gives non-finite y; calibration gives a zero-absmax group the scale 1)
 *   dt : (batch, seqlen, nheads) fp32, > 0, already passed through softplus
 *   A  : [nheads] fp32, finite, <= 0          D : [nheads] fp32 or NULL (= 0)
 *   h0 : (batch, nheads, headdim, dstate) fp32 or NULL (= 0)
 *   y  : (batch, seqlen, nheads, headdim) fp16, written
 *   h_final : (batch, nheads, headdim, dstate) fp32 or NULL; may alias h0
 *   workspace : device scratch of at least ssdq_chunk_scan_workspace_size() bytes,
 *               owned by the caller, not shared with a concurrent call
 * Supported shapes: headdim % 16 == 0 and headdim <= 64; dstate % 16 == 0 and
 * dstate <= 128; chunk in {64, 128, 256}; any seqlen >= 1 (a ragged last chunk
 * is masked); nheads % ngroups == 0; nheads * headdim * chunk < 2^30,
 * ngroups * dstate * chunk < 2^31 and batch * seqlen * nheads < 2^31.  Others
 * return SSDQ_ERROR_UNSUPPORTED.
 * Accuracy: y within 2e-3 * max|y| and h_final within 1e-4 * max|h| of the exact
 * recurrence over the same codes (fp32 accumulation, fp16 y).
 */
ssdq_status ssdq_chunk_scan(const int8_t* x, const float* x_scale, const int8_t* B, const float* B_scale,
                            const int8_t* C, const float* C_scale, const float* dt, const float* A,
                            const float* D, const float* h0, void* y, float* h_final, int32_t batch,
                            int64_t seqlen, int32_t nheads, int32_t headdim, int32_t dstate, int32_t ngroups,
                            int32_t chunk, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Number of stages ssdq_chunk_scan runs, in order: 0 chunk cumsum + chunk state,
 * 1 state passing, 2 chunk output. */
#define SSDQ_CHUNK_SCAN_STAGES 3

/*
 * 1 if, on the current device, ssdq_chunk_scan folds state passing into stage 0 for this
 * batch and head count, else 0 (also for non-positive arguments or without a device).
 * Folding applies when batch * nheads is at least the device's CU count: one block per
 * (batch, head) sequence then walks its chunks in order (Mamba-2 SSD state passing,
 * Ternary Mamba sec. 1 recurrence per chunk) and the fp32 chunk states never reach memory.
 */
int32_t ssdq_chunk_scan_state_fused(int32_t batch, int32_t nheads);

/*
 * The form of stage 0 that ssdq_chunk_scan (scale_layout 0) or ssdq_chunk_scan_scaled takes on
 * the current device for this batch and head count (host; informational, the results do not
 * depend on it beyond fp32 rounding):
 *   0 : three kernels (chunk states in parallel, then state passing; ssdq_chunk_scan_state_fused 0)
 *   8 : the folded state kernel in blocks of eight waves, one block per CU at a time
 *   4 : the folded state kernel in blocks of four waves, two blocks per CU (many more sequences
 *       than CUs)
 *  -1 : non-positive sizes or unknown scale_layout bits.
 */
int32_t ssdq_chunk_scan_plan(int32_t batch, int32_t nheads, uint32_t scale_layout);

/*
 * One stage of ssdq_chunk_scan, with the same arguments and validation.
 * Running stages 0..2 in order on one stream is exactly ssdq_chunk_scan; the
 * intermediate results are in the workspace layout documented above.  This
 * lets a caller time each kernel with its own events and lets tests inspect
 * the intermediates.  stage outside [0, SSDQ_CHUNK_SCAN_STAGES) is INVALID_VALUE.
 */
ssdq_status ssdq_chunk_scan_stage(int32_t stage, const int8_t* x, const float* x_scale, const int8_t* B,
                                  const float* B_scale, const int8_t* C, const float* C_scale,
                                  const float* dt, const float* A, const float* D, const float* h0, void* y,
                                  float* h_final, int32_t batch, int64_t seqlen, int32_t nheads,
                                  int32_t headdim, int32_t dstate, int32_t ngroups, int32_t chunk,
                                  void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * ssdq_chunk_scan with SSDi8's output correction: every output also receives a per-(head,
 * channel) term (the SSDi8 abstract describes a correction derived from error statistics gathered
 * per channel, Figure 1b labels it a mean correction; Tables 6 and 16).  The pages give no algebra for it; the reading
 * taken is the plainest they support: an additive term, calibrated offline (like the static
 * scales) as the mean over a calibration set of the unquantized scan's y minus the quantized
 * scan's y, channel by channel.  Calibration is the caller's; the library only applies it:
 *
 *   y[b,t,h,p] = (the output of ssdq_chunk_scan) + y_corr[h, p]     (added in fp32 before the fp16 rounding)
 *
 *   y_corr : (nheads, headdim) fp32, device, 16-byte aligned (NULL: SSDQ_ERROR_INVALID_VALUE)
 * Every other argument, the shapes, the accuracy and the validation are those of ssdq_chunk_scan,
 * and h_final does not depend on y_corr.
 */
ssdq_status ssdq_chunk_scan_corrected(const int8_t* x, const float* x_scale, const int8_t* B, const float* B_scale,
                                      const int8_t* C, const float* C_scale, const float* dt, const float* A,
                                      const float* D, const float* y_corr, const float* h0, void* y, float* h_final,
                                      int32_t batch, int64_t seqlen, int32_t nheads, int32_t headdim, int32_t dstate,
                                      int32_t ngroups, int32_t chunk, void* workspace, size_t workspace_bytes,
                                      hipStream_t stream);

/*
 * ssdq_chunk_scan with B and C scales per (group, state) (SSDi8 Table 10: per-P(N) together with
 * per-H(G)) and an optional output correction:
 *
 *   Bhat[b,t,g,n] = B_scale[g, n] B[b,t,g,n],   Chat[b,t,g,n] = C_scale[g, n] C[b,t,g,n]
 *   (the recurrence and readout of ssdq_chunk_scan over these), plus y_corr[h, p] on every y
 *
 *   B_scale, C_scale : (ngroups, dstate) fp32, device, each finite and > 0
 *   y_corr           : (nheads, headdim) fp32 or NULL (no correction)
 * Everything else as ssdq_chunk_scan, except:
 *  - C.B^T over the per-state scales runs on the INT8 matrix cores with the product
 *    B_scale C_scale of each state folded into the B codes as a 16-bit fixed-point number (two
 *    INT8 limbs) relative to the group's largest product: each term of the sum carries at most
 *    2^-9 of that largest product times |C code|, well inside the stated y accuracy;
 *  - the workspace regions of the chunk states and the carried state hold those states times
 *    C_scale[g, n] of each state column (h_final is unscaled).
 */
ssdq_status ssdq_chunk_scan_per_state(const int8_t* x, const float* x_scale, const int8_t* B, const float* B_scale,
                                      const int8_t* C, const float* C_scale, const float* dt, const float* A,
                                      const float* D, const float* y_corr, const float* h0, void* y, float* h_final,
                                      int32_t batch, int64_t seqlen, int32_t nheads, int32_t headdim, int32_t dstate,
                                      int32_t ngroups, int32_t chunk, void* workspace, size_t workspace_bytes,
                                      hipStream_t stream);

/* Scale layouts for ssdq_chunk_scan_scaled and ssdq_state_update_scaled (bit flags; 0 is the
 * layout of ssdq_chunk_scan: one x scale per head, one B and one C scale per group). */
#define SSDQ_SCALES_BC_PER_STATE 1u  /* B_scale, C_scale: (ngroups, dstate) */
#define SSDQ_SCALES_X_PER_CHANNEL 2u /* x_scale: (nheads, headdim) */

/*
 * ssdq_chunk_scan under any of the static scale layouts, with an optional output correction.
 * With SSDQ_SCALES_X_PER_CHANNEL, x has one static scale per (head, channel):
 *
 *   xhat[b,t,h,p] = x_scale[h, p] x[b,t,h,p]
 *
 * the granularity that Quamba2's sort-and-cluster of the x channels produces (its rebuttal names
 * the sort-and-cluster and the per-state-group quantization as the two steps; each channel cluster
 * of a head shares one scale, given here expanded to every channel of the cluster, so any
 * clustering, sorted or not, is one (nheads, headdim) table).  Such a scale factors out of every
 * contraction of the scan (they sum over tokens and states, never over channels), and is applied
 * in fp32 per output channel and per state row.  With SSDQ_SCALES_BC_PER_STATE, B and C have
 * one scale per (group, state) as in ssdq_chunk_scan_per_state.  Both bits may be set.
 *
 *   x_scale      : (nheads) fp32, or (nheads, headdim) with SSDQ_SCALES_X_PER_CHANNEL; each
 *                  finite and > 0
 *   B_scale, C_scale : (ngroups) fp32, or (ngroups, dstate) with SSDQ_SCALES_BC_PER_STATE
 *   y_corr       : (nheads, headdim) fp32 or NULL (no correction)
 *   scale_layout : SSDQ_SCALES_* bits (other bits: SSDQ_ERROR_INVALID_VALUE)
 * Everything else (shapes, workspace, accuracy, validation) as ssdq_chunk_scan; the codes of x are
 * those of ssdq_quantize_per_channel under the (nheads, headdim) table.
 */
ssdq_status ssdq_chunk_scan_scaled(const int8_t* x, const float* x_scale, const int8_t* B, const float* B_scale,
                                   const int8_t* C, const float* C_scale, const float* dt, const float* A,
                                   const float* D, const float* y_corr, const float* h0, void* y, float* h_final,
                                   int32_t batch, int64_t seqlen, int32_t nheads, int32_t headdim, int32_t dstate,
                                   int32_t ngroups, int32_t chunk, uint32_t scale_layout, void* workspace,
                                   size_t workspace_bytes, hipStream_t stream);

/* Bytes of the library's static device scratch that ssdq_chunk_scan_noalloc uses (per device). */
#define SSDQ_NOALLOC_SCRATCH_BYTES (64u << 20)

/*
 * ssdq_chunk_scan without a workspace argument, for callers that cannot allocate device memory
 * (code under HIP graph capture, tight serving loops, harnesses that forbid allocation).  The
 * intermediates (Acs, the chunk-ordered dt, the chunk states of the three-kernel plan, the
 * carried-state limbs and their row scales) live in one static device array of SSDQ_NOALLOC_SCRATCH_BYTES that the
 * library holds on every device it runs on until the process ends; the call allocates and
 * frees nothing.  Arguments, shapes, accuracy and validation are those of ssdq_chunk_scan, and
 * the results are those of ssdq_chunk_scan with the same arguments (the same kernels run).
 *   - A shape whose intermediates exceed the scratch (ssdq_chunk_scan_noalloc_scratch_size()
 *     above SSDQ_NOALLOC_SCRATCH_BYTES) returns SSDQ_ERROR_SCRATCH_LIMIT and launches nothing.
 *   - Every call on a device shares that device's scratch, and it keeps the last call's contents:
 *     calls that overlap on one device (concurrent streams, or several host threads without
 *     ordering) race on it and must be serialized by the caller.  Calls on one stream are
 *     ordered and safe.  Nothing in the scratch needs to start at zero.
 *   - The first call on a device looks up the scratch's device address (hipGetSymbolAddress);
 *     if that fails the call returns SSDQ_ERROR_LAUNCH.
 */
ssdq_status ssdq_chunk_scan_noalloc(const int8_t* x, const float* x_scale, const int8_t* B, const float* B_scale,
                                    const int8_t* C, const float* C_scale, const float* dt, const float* A,
                                    const float* D, const float* h0, void* y, float* h_final, int32_t batch,
                                    int64_t seqlen, int32_t nheads, int32_t headdim, int32_t dstate,
                                    int32_t ngroups, int32_t chunk, hipStream_t stream);

/* Scratch bytes ssdq_chunk_scan_noalloc needs for this shape on the current device (host; 0 on
 * invalid shapes): the Acs, Dtc, carried-state and row-scale regions, plus the fp32 chunk states when
 * the three-kernel plan runs, each rounded up to 256 bytes. */
size_t ssdq_chunk_scan_noalloc_scratch_size(int32_t batch, int64_t seqlen, int32_t nheads, int32_t headdim,
                                            int32_t dstate, int32_t chunk);

/*
 * Decode: one recurrence step per sequence, state updated IN PLACE (the
 * decode-time SSD update of the Quamba2 rebuttal, Tables R7/R8).
 *
 *   state[b,h,p,n] <- exp(dt[b,h] A[h]) state[b,h,p,n] + dt[b,h] xhat[b,h,p] Bhat[b,g,n]
 *   y[b,h,p] = sum_n Chat[b,g,n] state[b,h,p,n] (updated) + D[h] xhat[b,h,p]
 *
 *   state : (batch, nheads, headdim, dstate) fp32, read and written
 *   x : (batch, nheads, headdim) int8     B, C : (batch, ngroups, dstate) int8
 *   dt : (batch, nheads) fp32   A : [nheads]   D : [nheads] or NULL   y : (batch, nheads, headdim) fp16
 * Supported: dstate == 128 or dstate == 64, headdim <= 64, nheads % ngroups == 0.
 */
ssdq_status ssdq_state_update(float* state, const int8_t* x, const float* x_scale, const int8_t* B,
                              const float* B_scale, const int8_t* C, const float* C_scale, const float* dt,
                              const float* A, const float* D, void* y, int32_t batch, int32_t nheads,
                              int32_t headdim, int32_t dstate, int32_t ngroups, hipStream_t stream);

/*
 * The decode step with the state cached in IEEE binary16: half the bytes per step of the fp32
 * state on the HBM-bound update (a lower-precision cached SSM state, as the Quamba2
 * rebuttal's Tables R7/R8 discuss for decode-time memory and latency).
 *
 *   u[b,h,p,n] = exp(dt[b,h] A[h]) state[b,h,p,n] + dt[b,h] xhat[b,h,p] Bhat[b,g,n]   (fp32)
 *   y[b,h,p]   = sum_n Chat[b,g,n] u[b,h,p,n] + D[h] xhat[b,h,p]                   (from u)
 *   state[b,h,p,n] <- u rounded to the nearest binary16 (ties to even; |u| beyond the
 *                     format's range gives +-inf)
 *
 *   state : (batch, nheads, headdim, dstate) IEEE binary16, read and written
 * Every other argument, the shapes supported and the validation are those of
 * ssdq_state_update.  Each step rounds the state once (2^-11 relative at most), so after T
 * steps the cached state is within T * 2^-11 of the largest state magnitude of the fp32
 * recurrence; the caller chooses it where that is acceptable.
 */
ssdq_status ssdq_state_update_f16(void* state, const int8_t* x, const float* x_scale, const int8_t* B,
                                  const float* B_scale, const int8_t* C, const float* C_scale, const float* dt,
                                  const float* A, const float* D, void* y, int32_t batch, int32_t nheads,
                                  int32_t headdim, int32_t dstate, int32_t ngroups, hipStream_t stream);

/*
 * The decode step with the state cached as 8-bit codes and one binary32 scale per state row
 * (b, h, p): a quarter of the fp32 state's bytes per step (the 8-bit cached SSM states of the
 * Quamba2 rebuttal, Tables R7/R8; the pages do not fix the scale granularity, one scale per
 * row and the symmetric max/127 rule are the choice made here).
 *
 *   u[b,h,p,n] = exp(dt[b,h] A[h]) scale[b,h,p] state[b,h,p,n] + dt[b,h] xhat[b,h,p] Bhat[b,g,n]  (fp32)
 *   y[b,h,p]   = sum_n Chat[b,g,n] u[b,h,p,n] + D[h] xhat[b,h,p]                               (from u)
 *   scale[b,h,p] <- max_n |u[b,h,p,n]| / 127     (binary32; 0, with zero codes, when that is below 2^-126)
 *   state[b,h,p,n] <- u / scale rounded to nearest, ties to even, within [-127, 127] (0 if scale is 0)
 *
 *   state       : (batch, nheads, headdim, dstate) int8 codes, read and written
 *   state_scale : (batch, nheads, headdim) float32, read and written; 16-byte aligned
 * Every other argument, the shapes supported and the validation are those of
 * ssdq_state_update; a NULL or misaligned state_scale gives SSDQ_ERROR_INVALID_VALUE.  Each step
 * moves every element by at most half a code step (max|row| / 254), so after T steps the cached
 * state is within T/254 of the largest row magnitude of the fp32 recurrence; the values must
 * stay finite (a non-finite update makes its row's scale non-finite).  Codes where the update
 * falls within fp32 rounding of a midpoint between two codes may take either neighbour.
 */
ssdq_status ssdq_state_update_i8(int8_t* state, float* state_scale, const int8_t* x, const float* x_scale,
                                 const int8_t* B, const float* B_scale, const int8_t* C, const float* C_scale,
                                 const float* dt, const float* A, const float* D, void* y, int32_t batch,
                                 int32_t nheads, int32_t headdim, int32_t dstate, int32_t ngroups,
                                 hipStream_t stream);

/* Formats of the decode state for ssdq_state_update_corrected. */
typedef enum {
  SSDQ_STATE_F32 = 0,   /* fp32 state, as ssdq_state_update */
  SSDQ_STATE_F16 = 1,   /* IEEE binary16 cache, as ssdq_state_update_f16 */
  SSDQ_STATE_I8 = 2     /* 8-bit codes + row scales, as ssdq_state_update_i8 */
} ssdq_state_format;

/*
 * The decode step with the output correction of ssdq_chunk_scan_corrected: the step of the given
 * state format (its arguments, layout, validation and in-place update unchanged) whose y also
 * receives y_corr[h, p]:
 *
 *   y[b,h,p] = (the y of the plain step) + y_corr[h, p]
 *
 *   state_format : SSDQ_STATE_F32, SSDQ_STATE_F16 or SSDQ_STATE_I8 (else SSDQ_ERROR_INVALID_VALUE)
 *   state        : (batch, nheads, headdim, dstate) fp32, binary16 or int8 codes, read and written
 *   state_scale  : (batch, nheads, headdim) fp32 row scales for SSDQ_STATE_I8, read and written;
 *                  ignored (may be NULL) for the other formats
 *   y_corr       : (nheads, headdim) fp32, device, 16-byte aligned (NULL: SSDQ_ERROR_INVALID_VALUE)
 * The state does not depend on y_corr.
 */
ssdq_status ssdq_state_update_corrected(int32_t state_format, void* state, float* state_scale, const int8_t* x,
                                        const float* x_scale, const int8_t* B, const float* B_scale, const int8_t* C,
                                        const float* C_scale, const float* dt, const float* A, const float* D,
                                        const float* y_corr, void* y, int32_t batch, int32_t nheads, int32_t headdim,
                                        int32_t dstate, int32_t ngroups, hipStream_t stream);

/*
 * The decode step of ssdq_state_update_corrected with B and C scales per (group, state):
 * B_scale, C_scale (ngroups, dstate) fp32; y_corr (nheads, headdim) fp32 or NULL (no correction).
 * Formats, arguments, layouts and validation otherwise as ssdq_state_update_corrected.  (On the
 * 8-bit cached state, y is then summed in fp32 over the per-state C values instead of by integer
 * dot products.)
 */
ssdq_status ssdq_state_update_per_state(int32_t state_format, void* state, float* state_scale, const int8_t* x,
                                        const float* x_scale, const int8_t* B, const float* B_scale, const int8_t* C,
                                        const float* C_scale, const float* dt, const float* A, const float* D,
                                        const float* y_corr, void* y, int32_t batch, int32_t nheads, int32_t headdim,
                                        int32_t dstate, int32_t ngroups, hipStream_t stream);

/*
 * The decode step of ssdq_state_update_corrected under any of the static scale layouts of
 * ssdq_chunk_scan_scaled (scale_layout: SSDQ_SCALES_* bits; x_scale (nheads, headdim) with
 * SSDQ_SCALES_X_PER_CHANNEL, B_scale and C_scale (ngroups, dstate) with
 * SSDQ_SCALES_BC_PER_STATE); y_corr (nheads, headdim) fp32 or NULL.  Formats, arguments, layouts
 * and validation otherwise as ssdq_state_update_corrected; other bits: SSDQ_ERROR_INVALID_VALUE.
 */
ssdq_status ssdq_state_update_scaled(int32_t state_format, void* state, float* state_scale, const int8_t* x,
                                     const float* x_scale, const int8_t* B, const float* B_scale, const int8_t* C,
                                     const float* C_scale, const float* dt, const float* A, const float* D,
                                     const float* y_corr, void* y, int32_t batch, int32_t nheads, int32_t headdim,
                                     int32_t dstate, int32_t ngroups, uint32_t scale_layout, hipStream_t stream);

/*
 * Front end of the SSD block, fused with the static quantizer: the causal convolution that the
 * pages keep in FP16 ahead of the SSD box (Quamba2 rebuttal Tables R6/R7; SSDi8 Table 16, Conv
 * column), read as Mamba-2's depthwise convolution of width 4 over the tokens of every channel
 * of the in-projection output, with a per-channel bias and SiLU; its binary16 output is
 * quantized as ssdq_quantize does, straight into the scan's layouts; and dt = softplus(dt_raw
 * + dt_bias), the positive step size the scan takes.
 *
 *   xbc    : (batch, seqlen, nheads*headdim + 2*ngroups*dstate) binary16, channels [x | B | C]
 *            (x channel h*headdim + p, then B channel g*dstate + n, then C likewise)
 *   conv_w : (channels, d_conv) float32; tap k multiplies token t - d_conv + 1 + k (zero before 0)
 *   conv_b : (channels) float32, or NULL for no bias
 *   a[b,t,c] = binary16( SiLU( conv_b[c] + sum_k conv_w[c,k] xbc[b, t-3+k, c] ) ),  SiLU(v) = v / (1 + e^-v)
 *   x      : (batch, seqlen, nheads, headdim) int8 = quantize(a[.., x channels], x_scale (nheads))
 *   B, C   : (batch, seqlen, ngroups, dstate) int8 = quantize(a[.., B / C channels], B_scale / C_scale (ngroups))
 *   dt_raw : (batch, seqlen, nheads) float32; dt_bias: (nheads) float32 or NULL
 *   dt     : (batch, seqlen, nheads) float32 = softplus(dt_raw + dt_bias) = max(v,0) + log1p(e^-|v|)
 * The codes are those of ssdq_quantize applied to a (bit-exact); a is formed in fp32, so an
 * element whose exact SiLU value lies within fp32 rounding of a binary16 midpoint may take the
 * other neighbour (and its code).  seqlen 0 is a no-op (after the size checks; pointers are not
 * looked at then).  Errors: NULL or misaligned (16-byte) pointers, non-positive sizes or nheads % ngroups != 0 -> SSDQ_ERROR_INVALID_VALUE; d_conv other
 * than 4, headdim or dstate not a multiple of 8, or batch * ceil(channels / 256) * ceil(seqlen / 16)
 * >= 2^31 ->
 * SSDQ_ERROR_UNSUPPORTED.  All pointers are device memory owned by the caller.
 */
ssdq_status ssdq_frontend(const void* xbc, const float* conv_w, const float* conv_b, int32_t d_conv,
                          const float* x_scale, const float* B_scale, const float* C_scale, const float* dt_raw,
                          const float* dt_bias, int8_t* x, int8_t* B, int8_t* C, float* dt, int32_t batch,
                          int64_t seqlen, int32_t nheads, int32_t headdim, int32_t dstate, int32_t ngroups,
                          hipStream_t stream);

/*
 * ssdq_frontend for one decode token per sequence, with the convolution's history carried in a
 * conv state: the same output, codes and dt as ssdq_frontend gives for the last token of a
 * sequence whose three previous tokens are the state's rows (the cached convolution states of
 * the Quamba2 rebuttal, Table R7).
 *
 *   conv_state : (batch, 3, channels) binary16, read and written: rows are the inputs of tokens
 *                t-3, t-2, t-1 before the call and t-2, t-1, t after it (zeros at the start)
 *   xbc        : (batch, channels) binary16, token t
 *   x (batch, nheads, headdim), B and C (batch, ngroups, dstate) int8; dt_raw, dt (batch, nheads)
 * Every other argument, its layout and the validation are those of ssdq_frontend (d_conv 4;
 * headdim and dstate multiples of 8); all pointers are device memory owned by the caller.
 */
ssdq_status ssdq_frontend_step(void* conv_state, const void* xbc, const float* conv_w, const float* conv_b,
                               int32_t d_conv, const float* x_scale, const float* B_scale, const float* C_scale,
                               const float* dt_raw, const float* dt_bias, int8_t* x, int8_t* B, int8_t* C, float* dt,
                               int32_t batch, int32_t nheads, int32_t headdim, int32_t dstate, int32_t ngroups,
                               hipStream_t stream);

/* Element types of the gated scan, of activation checkpoints, of the norms and of the selective scan. */
typedef enum {
  SSDQ_DTYPE_F32 = 0,   /* binary32 */
  SSDQ_DTYPE_F16 = 1,   /* IEEE binary16 */
  SSDQ_DTYPE_BF16 = 2   /* bfloat16 */
} ssdq_dtype;

/* Channels that share one scale of an 8-bit activation checkpoint. */
#define SSDQ_CHECKPOINT_BLOCK 64

/*
 * 8-bit activation checkpoint: an activation kept between the forward and the backward pass as one
 * signed code per element and one binary32 scale per 64 consecutive channels of a row (1.0625
 * bytes per element).  As in the 8-bit decode state the largest magnitude takes the code 127; its scale is
 * a product here and the rounded quotient m / 127 there, so the two may differ in the last place.
 *
 *   m[r,k]     = max over i in block k of |x[r,i]|
 *   scale[r,k] = m * (1/127), one product of binary32 numbers, 1/127 rounded to binary32 (within
 *                2^-23 of m / 127); 0, with zero codes, when m < 127 * 2^-126
 *   codes[r,i] = the integer nearest to the exact quotient x[r,i] / scale[r,k], ties to even
 *                (within [-127, 127]; -128 is never produced)
 * A block that holds a NaN or an infinity gets the scale NaN and zero codes, so that it reads back
 * as NaN and the fault is not hidden.
 *   dtype : ssdq_dtype of x          x : (rows, channels)
 *   codes : (rows, channels) int8, written     scale : (rows, ceil(channels / 64)) fp32, written
 * Any rows >= 0 (0 = no-op) and channels >= 1 (the last block of a row may be partial) with
 * rows * ceil(channels / 64) < 2^36; else SSDQ_ERROR_UNSUPPORTED.  No output overlaps x.
 */
ssdq_status ssdq_checkpoint_save(int32_t dtype, const void* x, int8_t* codes, float* scale, int64_t rows,
                                 int32_t channels, hipStream_t stream);

/*
 * The values of an 8-bit checkpoint: x[r,i] = codes[r,i] * scale[r,k], formed in binary32 and rounded
 * once to dtype.  Arguments and limits as ssdq_checkpoint_save; codes of -128 read as such.
 */
ssdq_status ssdq_checkpoint_load(int32_t dtype, const int8_t* codes, const float* scale, void* x, int64_t rows,
                                 int32_t channels, hipStream_t stream);

/* What the gate tensor of the gated scan holds. */
typedef enum {
  SSDQ_GATE_LOG = 0,    /* log a:      a = exp(gate),                b = u   (-inf: a = 0) */
  SSDQ_GATE_LOGIT = 1   /* logit of a: a = 1 / (1 + exp(-gate)),     b = (1 - a) u              */
} ssdq_gate_kind;

/* Bytes of workspace that ssdq_gated_scan and ssdq_gated_scan_backward need (host; the same for
 * both, any dtype; packed is nonzero for calls with offsets; 0 on invalid or unsupported sizes,
 * else at least 256). */
size_t ssdq_gated_scan_workspace_size(int32_t sequences, int64_t tokens, int32_t channels, int32_t packed);

/*
 * Gated linear recurrence: the recurrence h_t = Abar_t h_{t-1} + Bbar_t x_t (Ternary Mamba,
 * Section 1) with a gate of its own for every channel,
 *
 *   h_t[c] = a_t[c] h_{t-1}[c] + b_t[c],   h_{-1} = h0 (or 0),   a and b from gate and u by gate_kind,
 *
 * over every token of every sequence, in binary32 whatever the types.
 *   dtype   : ssdq_dtype of gate, u and h         gate, u, h : (tokens, channels); h is written
 *   offsets : NULL: tokens = sequences * L, sequence s holds rows s*L .. s*L + L - 1 (dense).
 *             Otherwise (sequences + 1) int32, device, nondecreasing, within [0, tokens]: sequence s
 *             holds rows offsets[s] .. offsets[s+1] - 1 (packed; none, one or many each).  Rows in no
 *             sequence are neither read nor written.  Offsets out of range or out of order give
 *             unspecified results but no access outside the tensors.
 *   h0      : (sequences, channels) fp32 or NULL (= 0)
 *   h_final : (sequences, channels) fp32 or NULL: the state after each sequence's last token (the
 *             unrounded one; h0 for a sequence without tokens); may alias h0
 *   codes, scale : both NULL, or the 8-bit checkpoint of the written h (that of
 *             ssdq_checkpoint_save(dtype, h, ...), bit for bit): (tokens, channels) int8 and
 *             (tokens, ceil(channels / 64)) fp32
 *   workspace : device scratch of at least ssdq_gated_scan_workspace_size() bytes, owned by the
 *             caller, not shared with a concurrent call; it need not start at any value
 * Any sequences >= 1, tokens >= 0 and 1 <= channels <= 2^20 with tokens < 2^31 - 2^16 and
 * ceil(channels / 64) * tiles < 2^24 (else SSDQ_ERROR_UNSUPPORTED), where tiles is, dense, sequences *
 * max(1, ceil(L / 128)) and, packed, sequences, plus floor(tokens / 128) if tokens > 128; dense tokens must be
 * a multiple of sequences.  With tokens == 0 the (tokens, ...) pointers are not looked at.  No output overlaps
 * an input or another output, but for h_final on h0.
 * A NaN or infinity in gate, u or h0 makes the rows after it in its sequence and channel non-finite
 * or NaN (a = 0 does not clear it: 0 times infinity is NaN), and nothing else.  Products of a over up to
 * 256 neighbouring tokens of a sequence are formed on the way: where one is past binary32's range (only log
 * gates above 0 can reach that) h may be infinite or NaN though the recurrence is not.  The result does not
 * depend on timing: calls with the same arguments give the same bits.
 */
ssdq_status ssdq_gated_scan(int32_t dtype, int32_t gate_kind, const void* gate, const void* u, const float* h0,
                            const int32_t* offsets, void* h, float* h_final, int8_t* codes, float* scale,
                            int32_t sequences, int64_t tokens, int32_t channels, void* workspace,
                            size_t workspace_bytes, hipStream_t stream);

/*
 * Gradients of ssdq_gated_scan.  With dh the gradient of every h_t and dh_final that of h_final,
 *
 *   d_t = dh_t + k_{t+1},  k_t = a_t d_t   (k after a sequence's last token: dh_final or 0)
 *   SSDQ_GATE_LOG   : dgate_t = k_t h_{t-1}                        du_t = d_t
 *   SSDQ_GATE_LOGIT : dgate_t = k_t (1 - a_t) (h_{t-1} - u_t)      du_t = (1 - a_t) d_t
 *   dh0 = k of the first token (dh_final, or 0, for a sequence without tokens)
 *
 * where h_{t-1} is read from the saved h of the forward pass, or from its 8-bit checkpoint (codes *
 * scale), and is h0 (or 0) for a first token.
 *   gate, dh, dgate, du : (tokens, channels) of dtype; dgate and du are written
 *   u       : (tokens, channels) of dtype; needed with SSDQ_GATE_LOGIT, not looked at otherwise
 *   h       : (tokens, channels) of dtype, or NULL with codes and scale given (exactly one of them)
 *   dh_final, dh0 : (sequences, channels) fp32 or NULL each; dh0 is written and may alias dh_final
 * Everything else as ssdq_gated_scan; no output overlaps an input (h0 among them) or another output, but for
 * dh0 on dh_final.
 */
ssdq_status ssdq_gated_scan_backward(int32_t dtype, int32_t gate_kind, const void* gate, const void* u, const void* h,
                                     const int8_t* codes, const float* scale, const float* h0, const void* dh,
                                     const float* dh_final, const int32_t* offsets, void* dgate, void* du, float* dh0,
                                     int32_t sequences, int64_t tokens, int32_t channels, void* workspace,
                                     size_t workspace_bytes, hipStream_t stream);

/*
 * One token of ssdq_gated_scan for every sequence of a decode batch, the state updated in place:
 *   state <- a state + b;   h = the updated state rounded to dtype
 *   state : (batch, channels) fp32, read and written     gate, u, h : (batch, channels) of dtype
 * batch, channels >= 1 with batch * channels < 2^36; no workspace.  h and state overlap no other tensor.
 */
ssdq_status ssdq_gated_step(int32_t dtype, int32_t gate_kind, float* state, const void* gate, const void* u, void* h,
                            int32_t batch, int32_t channels, hipStream_t stream);

/*
 * Root-mean-square norm of rows, the step ahead of a block's projections, with its output rounded to dtype or as
 * 8-bit codes (the W8A8 projections of the Quamba project page and of the Quamba2 rebuttal).
 *
 *   v[r,c] = x[r,c]                                       plain
 *            x[r,c] + residual[r,c]                       with residual (residual_out receives v, rounded)
 *            x[r,c] * z / (1 + exp(-z)), z = gate[r,c]    with gate
 *   n[r,c] = v[r,c] * weight[c] / sqrt(mean over the group of c of v[r,:]^2 + eps)
 *
 * in binary32; groups equal parts of a row's channels are normalized each by itself.  v is not rounded to dtype
 * before it is squared and scaled.  The output is one of
 *   out          : (rows, channels) of dtype = n, rounded to nearest even
 *   codes, scale : (rows, channels) int8 and (rows) fp32: the row's scale is m * (1/127) with m = max |n[r,:]| (0, with
 *                  zero codes, when m < 127 * 2^-126), a code the integer nearest to n / scale, ties to even
 *   codes, static_scale : static_scale [1] fp32, device, from 2^-126 to 2^115; a code is the integer nearest to
 *                  n / static_scale, within [-127, 127] (NaN gives 0); scale is NULL then
 * -128 is never produced.  A row whose sum of squares is not finite in binary32 (a NaN or an infinity in it, or
 * magnitudes near 2^64) is NaN: out is NaN throughout, the scale is NaN and the codes 0, so that the fault is not hidden;
 * with a static scale its codes are 0.  So is a row of zeros with eps 0.  A row whose squares underflow is none of these: its
 * n is that of the formula, whatever eps.  (With groups: out is NaN in that group, scale
 * and codes over the row; under a static scale the codes are 0 in that group.)
 *   dtype    : ssdq_dtype of x, gate and out     x, gate, out : (rows, channels)
 *   residual_dtype : ssdq_dtype of residual and residual_out: dtype, or SSDQ_DTYPE_F32
 *   residual, residual_out : (rows, channels) or both NULL; residual_out may be residual
 *   gate     : (rows, channels) or NULL; not together with residual
 *   weight   : (channels) fp32, device           eps : not negative, finite
 * Any rows >= 0 (0 = no-op, pointers not looked at) below 2^31; 1 <= channels <= 16384, or 32768 with one group;
 * 1 <= groups <= 256 and channels % groups == 0 (a remainder: SSDQ_ERROR_INVALID_VALUE; sizes beyond:
 * SSDQ_ERROR_UNSUPPORTED).  No output overlaps an input or another output, but residual_out on residual.
 */
ssdq_status ssdq_rms_norm(int32_t dtype, int32_t residual_dtype, const void* x, const void* residual, const void* gate,
                          const float* weight, const float* static_scale, void* out, int8_t* codes, float* scale,
                          void* residual_out, int64_t rows, int32_t channels, int32_t groups, float eps,
                          hipStream_t stream);

/*
 * Rows as 8-bit codes with one scale each: activations per token, or weights per output channel, as the operands of
 * ssdq_matmul_i8.  Codes and scales are those of ssdq_rms_norm for n = x, bit-exact: scale = m * (1/127), codes the
 * integers nearest to the exact quotient x / scale, ties to even.  A row that holds a NaN or an infinity gets the scale
 * NaN and zero codes.
 *   x : (rows, channels) of dtype     codes : (rows, channels) int8, written     scale : (rows) fp32, written
 * Any rows >= 0 (0 = no-op) below 2^31 and 1 <= channels <= 32768 (else SSDQ_ERROR_UNSUPPORTED).
 */
ssdq_status ssdq_quantize_rows(int32_t dtype, const void* x, int8_t* codes, float* scale, int64_t rows,
                               int32_t channels, hipStream_t stream);

/*
 * The values of such rows: x[r,c] = codes[r,c] * scale[r], formed in binary32 and rounded once to dtype.  Any codes
 * (-128 reads as such) and any channels >= 1; everything else as ssdq_quantize_rows.
 */
ssdq_status ssdq_dequantize_rows(int32_t dtype, const int8_t* codes, const float* scale, void* x, int64_t rows,
                                 int32_t channels, hipStream_t stream);

/*
 * Matrix product of 8-bit codes, the block's projections in W8A8:
 *
 *   out[m,n] = (float(sum_k a[m,k] b[n,k]) * a_scale[m]) * b_scale[n] + bias[n]
 *
 * The sum is exact in int32; the conversion, the two products and the sum with the bias are binary32 operations, each
 * rounded to nearest even (the last product and the sum may be one fused operation), and out is rounded once more.
 *   dtype   : ssdq_dtype of out
 *   a       : (m, k) int8, a row per token            b    : (n, k) int8, a row per output channel
 *   a_scale : (m) fp32 with a_scale_per_row nonzero, else [1]     b_scale : (n) fp32
 *   bias    : (n) fp32 or NULL                         out  : (m, n) of dtype, written
 * Any codes, -128 among them.  Any m >= 0 (0 = no-op, pointers not looked at), n >= 1, 1 <= k <= 131071 (above, a
 * sum could leave int32) with m < 2^31 - 2^16 and ceil(m/128) * ceil(n/128) < 2^24 (else SSDQ_ERROR_UNSUPPORTED).  A NaN
 * or an infinity in a scale or in bias makes the outputs that it enters non-finite or NaN, and no others.  out overlaps
 * no input.
 */
ssdq_status ssdq_matmul_i8(int32_t dtype, const int8_t* a, const float* a_scale, int32_t a_scale_per_row,
                           const int8_t* b, const float* b_scale, const float* bias, void* out, int64_t m, int32_t k,
                           int32_t n, hipStream_t stream);

/*
 * The kernel that ssdq_matmul_i8 takes for these sizes on the current device (host; informational: the sums are exact in
 * all of them); -1 for sizes without work, invalid or unsupported ones.
 */
typedef enum {
  SSDQ_MATMUL_STREAM_16 = 0,            /* weights streamed, up to 16 tokens */
  SSDQ_MATMUL_STREAM_32 = 1,            /* the same, up to 32 */
  SSDQ_MATMUL_TILES_256X256 = 2,        /* tiles of tokens x output channels */
  SSDQ_MATMUL_TILES_128X128 = 3,
  SSDQ_MATMUL_TILES_128X64 = 4,
  SSDQ_MATMUL_TILES_64X64 = 5,
  SSDQ_MATMUL_TILES_64X64_HALVES = 6,   /* in two halves of the inner axis */
  SSDQ_MATMUL_ODD_STREAM_16 = 7,        /* inner sizes that no 16 divides, the same kinds */
  SSDQ_MATMUL_ODD_128X128 = 8,
  SSDQ_MATMUL_ODD_64X64 = 9,
  SSDQ_MATMUL_ODD_64X64_HALVES = 10,
} ssdq_matmul_plan;
int32_t ssdq_matmul_i8_plan(int64_t m, int32_t k, int32_t n);

/*
 * Short causal convolution along the tokens of every channel, ahead of the selective scan (the convolution of the
 * Mamba block; ssdq_frontend holds the Mamba-2 block's, fused with its quantizer):
 *
 *   a[t,c] = bias[c] + sum_k weight[c,k] x[t - width + 1 + k, c];    out = a, or a / (1 + exp(-a)) with silu nonzero
 *
 * in binary32, rounded once to dtype; rows before a sequence's first token are those of its state (or 0).
 *   x, out    : (tokens, channels) of dtype; dense or packed by offsets exactly as in ssdq_gated_scan
 *   weight    : (channels, width) fp32, tap width - 1 multiplies the token itself     bias : (channels) fp32 or NULL
 *   state     : (sequences, width - 1, channels) of dtype or NULL (= 0): the inputs ahead of the first token, oldest
 *               first
 *   state_out : (sequences, width - 1, channels) of dtype or NULL, written: the inputs of each sequence's last width - 1
 *               tokens, oldest first (of state where it has fewer); it must not be state
 * width 2, 3 or 4; sequences, channels >= 1; tokens >= 0, dense a multiple of sequences (else SSDQ_ERROR_INVALID_VALUE);
 * tokens < 2^31 - 2^16, sequences < 2^24, channels <= 2^20 and ceil(channels / 256) * (sequences + tokens / 16 + 1) <
 * 2^25 (else SSDQ_ERROR_UNSUPPORTED).  With tokens == 0 x and out are not looked at.  Offsets out of range or out of
 * order give unspecified results but no access outside the tensors.  No output overlaps an input (out on x is refused).
 */
ssdq_status ssdq_causal_conv(int32_t dtype, const void* x, const float* weight, const float* bias, const void* state,
                             const int32_t* offsets, void* out, void* state_out, int32_t sequences, int64_t tokens,
                             int32_t channels, int32_t width, int32_t silu, hipStream_t stream);

/*
 * One token of ssdq_causal_conv for every sequence of a decode batch, the state updated in place:
 *   state : (batch, width - 1, channels) of dtype, read and written     x, out : (batch, channels) of dtype
 * batch, channels >= 1 with batch * channels < 2^31 (else SSDQ_ERROR_UNSUPPORTED).  No output overlaps an input.
 */
ssdq_status ssdq_causal_conv_step(int32_t dtype, void* state, const void* x, const float* weight, const float* bias,
                                  void* out, int32_t batch, int32_t channels, int32_t width, int32_t silu,
                                  hipStream_t stream);

/* Bytes of workspace that ssdq_selective_scan needs (host; packed is nonzero for calls with offsets; 0 on invalid or
 * unsupported sizes, else at least 256). */
size_t ssdq_selective_scan_workspace_size(int32_t sequences, int64_t tokens, int32_t channels, int32_t dstate,
                                          int32_t packed);

/* How ssdq_selective_scan walks sequences of these sizes (host; informational, results differ in binary32 rounding
 * only): 0 whole, else in chunks of so many tokens; -1 on invalid or unsupported sizes. */
int32_t ssdq_selective_scan_plan(int32_t sequences, int64_t tokens, int32_t channels, int32_t dstate, int32_t packed);

/*
 * Selective state space scan with a decay for every channel and state and a step size for every channel (the recurrence
 * h_t = Abar_t h_{t-1} + Bbar_t x_t of Ternary Mamba, Section 1, in the form of the first Mamba block, which the Quamba
 * project page quantizes beside the second):
 *
 *   d_t[c]   = softplus(delta_t[c] + delta_bias[c])      (softplus nonzero; else delta_t[c] + delta_bias[c])
 *   h_t[c,n] = exp(d_t[c] A[c,n]) h_{t-1}[c,n] + d_t[c] u_t[c] B_t[n],        h_{-1} = h0 (or 0)
 *   y_t[c]   = (sum_n C_t[n] h_t[c,n] + D[c] u_t[c]) * z_t[c] / (1 + exp(-z_t[c]))      (without z: the bracket)
 *
 * over every token of every sequence, in binary32 whatever the types; y is rounded once.
 *   dtype        : ssdq_dtype of u, delta, B, C, z and y
 *   u, delta, y  : (tokens, channels); z the same or NULL     B, C : (tokens, dstate)
 *   A            : (channels, dstate) fp32     D, delta_bias : (channels) fp32 or NULL (= 0) each
 *   offsets      : NULL (dense) or (sequences + 1) int32, exactly as in ssdq_gated_scan
 *   h0, h_final  : (sequences, channels, dstate) fp32 or NULL each; h_final is the state after each sequence's last token
 *                  (h0, or 0, for one without tokens) and must not be h0
 *   workspace    : device scratch of at least ssdq_selective_scan_workspace_size() bytes, owned by the caller, not
 *                  shared with a concurrent call; it need not start at any value
 * sequences >= 1, tokens >= 0, channels >= 1, 1 <= dstate <= 64; dense tokens a multiple of sequences (else
 * SSDQ_ERROR_INVALID_VALUE); tokens < 2^31 - 2^16, sequences < 2^24, channels <= 2^20, a workspace below 2^40 bytes and
 * fewer than 2^23 pieces that the kernels walk the sequences in: 16 to 256 tokens of a sequence each, or a whole one
 * (else SSDQ_ERROR_UNSUPPORTED; the workspace's size is 0 then).  With tokens == 0 the (tokens, ...) pointers are not
 * looked at.  No output overlaps an input or another output.  A NaN or an infinity in u, delta or h0 stays in its sequence
 * and channel, one in B or C in its sequence, one in z in its element; behind an infinity (or where d u overflows) y may be a
 * NaN where the formula has an infinity.  exp(d A) above 1 (A above 0) is allowed as long as
 * products of it over 256 neighbouring tokens stay finite.  The result does not depend on timing: calls with the same
 * arguments give the same bits.
 */
ssdq_status ssdq_selective_scan(int32_t dtype, const void* u, const void* delta, const float* A, const void* B,
                                const void* C, const float* D, const void* z, const float* delta_bias, const float* h0,
                                const int32_t* offsets, void* y, float* h_final, int32_t sequences, int64_t tokens,
                                int32_t channels, int32_t dstate, int32_t softplus, void* workspace,
                                size_t workspace_bytes, hipStream_t stream);

/*
 * One token of ssdq_selective_scan for every sequence of a decode batch, the state updated in place:
 *   state : (batch, channels, dstate) fp32, read and written     u, delta, z, y : (batch, channels)
 *   B, C  : (batch, dstate)
 * batch, channels >= 1; 1 <= dstate <= 64 and batch * ceil(channels / 16) < 2^24 (else SSDQ_ERROR_UNSUPPORTED); no
 * workspace.  No output overlaps another tensor.
 */
ssdq_status ssdq_selective_step(int32_t dtype, float* state, const void* u, const void* delta, const float* A,
                                const void* B, const void* C, const float* D, const void* z, const float* delta_bias,
                                void* y, int32_t batch, int32_t channels, int32_t dstate, int32_t softplus,
                                hipStream_t stream);

/* How many sequences a lane of ssdq_selective_step takes at these sizes, 4 or 1 (host; informational, the results do not
 * depend on it); -1 on invalid or unsupported sizes. */
int32_t ssdq_selective_step_plan(int32_t batch, int32_t channels, int32_t dstate);

#ifdef __cplusplus
}
#endif

#endif /* SSDQ_H_ */
