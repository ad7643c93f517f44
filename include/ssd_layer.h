/*
 * ssd_layer.h -- C ABI of libssd, second part: the operators around the scan
 * in a state-space layer, on one AMD Instinct MI355X (gfx950).
 *
 *   ssd_conv_*        the short depthwise causal convolution (with bias and
 *                     SiLU) that makes x, B and C from a layer's projection;
 *   ssd_selscan_*     the selective scan of first-generation layers, with a
 *                     decay of its own for every channel and state, beside
 *                     ssd_fwd (ssd.h), whose decay is one per head;
 *   ssd_gated_norm_*  the grouped RMS norm with a SiLU gate that follows it.
 *
 * A second-generation layer is ssd_conv_fwd -> ssd_fwd_ex -> ssd_gated_norm_fwd,
 * a first-generation one ssd_conv_fwd -> ssd_selscan_fwd; for single tokens
 * ssd_conv_step -> ssd_step -> ssd_gated_norm_fwd, or ssd_conv_step ->
 * ssd_selscan_step; in training the _bwd calls in reverse.
 *
 * Everything ssd.h says of ownership, streams, determinism, graph capture
 * and errors holds here.  In particular: pointers are device memory owned by
 * the caller, work is enqueued on `stream` without synchronising, nothing is allocated, kernels
 * only are enqueued (so every call can be captured into a HIP graph), the
 * same call gives the same bits, and no exception crosses the interface.
 * `stream` belongs to the current device.  Outputs must not overlap inputs or
 * each other (a final_state that overlaps init_state, which ssd_fwd allows, is
 * SSD_ERR_BAD_VALUE here: chunks of the sequence run side by side).  One workspace serves one call at a
 * time; its contents on entry do not matter.
 *
 * io dtype is SSD_BF16 or SSD_F32.  Sums, states and statistics are fp32;
 * outputs in the io dtype are rounded once.
 *
 * Operands with strides.  An operand marked (strided) is [batch, seqlen, width]
 * with its last axis contiguous and an ssd_strides for the other two, in
 * elements: a slice of a wider projection is read or written in place.  A NULL
 * ssd_strides means contiguous.  Strides of inputs may be any values >= 0 (0
 * repeats a row); strides of outputs must keep rows apart.  The stride between
 * tokens (batches) of a call with one token (batch) separates nothing: any value
 * >= 0 does, of an output too.  A strided pointer needs the alignment of its
 * element only; every other pointer is 16-byte aligned.  Where pointers, strides
 * and sizes allow accesses of several elements they are used.
 *
 * Errors, in this order: SSD_ERR_NULL_POINTER, SSD_ERR_BAD_SHAPE (a size <= 0, sizes
 * that do not divide or add up, or a product overflowing int64),
 * SSD_ERR_BAD_DTYPE (io_dtype, or a reserved field not 0), SSD_ERR_BAD_VALUE
 * (an invalid option, transform or stride), SSD_ERR_MISALIGNED, SSD_ERR_UNSUPPORTED,
 * SSD_ERR_WORKSPACE, SSD_ERR_HIP.  Nothing is enqueued when a call returns an
 * error other than SSD_ERR_HIP.
 */
#ifndef LIBSSD_SSD_LAYER_H
#define LIBSSD_SSD_LAYER_H

#include "ssd.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SSD_LAYER_ABI_VERSION 1

/* SSD_LAYER_ABI_VERSION of the loaded library. */
int ssd_layer_abi_version(void);

/* Elements between batches and between tokens of a strided operand. */
typedef struct {
  int64_t batch;
  int64_t token;
} ssd_strides;

/* ---------------------------------------------------------------- convolution
 *
 * For every batch b, channel c and token t, with width W:
 *     u[t] = bias[c] + sum_{k < W} weight[c, k] x[t - (W - 1) + k]
 *     y[t] = u[t]                      activation 0
 *          = u[t] / (1 + exp(-u[t]))   activation 1 (SiLU)
 * where x at t < 0 comes from init_state, zero without one.
 *
 * The outputs can be split along the channels into up to three contiguous
 * tensors [batch, seqlen, split[i]], the layouts that ssd_fwd takes as x, B and C.
 */
typedef struct {
  int64_t batch;
  int64_t seqlen;
  int64_t channels;
  int64_t width;      /* W: 2, 3 or 4 */
  int64_t nsplit;     /* outputs: 1, 2 or 3 */
  int64_t split[3];   /* channels of each output (first nsplit entries; sum = channels) */
  int32_t io_dtype;
  int32_t activation; /* 0 none, 1 SiLU */
  int64_t reserved;   /* must be 0 */
} ssd_conv_problem;

/* Prompt.
 *   x           : (strided) [batch, seqlen, channels] io dtype.
 *   weight      : [channels, width] fp32;  bias: [channels] fp32 or NULL.
 *   init_state  : [batch, width - 1, channels] io dtype: the inputs before the first
 *                 token, oldest first; or NULL for zeros.
 *   y           : nsplit outputs, y[i] [batch, seqlen, split[i]] io dtype (a host
 *                 array of device pointers).
 *   final_state : [batch, width - 1, channels] io dtype: the last width - 1 inputs
 *                 (earlier ones from init_state where seqlen < width - 1), or NULL.
 * Errors: UNSUPPORTED for a width outside 2..4, batch > 65535, or sizes past a
 * launch's 2^32 threads. */
ssd_status ssd_conv_fwd(const ssd_conv_problem* prob, const void* x, const ssd_strides* x_strides,
                        const float* weight, const float* bias, const void* init_state,
                        void* const* y, void* final_state, void* stream);

/* Single tokens: as ssd_conv_fwd over seqlen tokens with init_state = state,
 * and `state` (required) then holds the last width - 1 inputs. */
ssd_status ssd_conv_step(const ssd_conv_problem* prob, void* state, const void* x,
                         const ssd_strides* x_strides, const float* weight, const float* bias,
                         void* const* y, void* stream);

/* Workspace bytes of ssd_conv_bwd (part sums of the weight gradients). */
ssd_status ssd_conv_bwd_workspace_size(const ssd_conv_problem* prob, size_t* bytes);

/* Gradients, given dy[i] = dLoss/dy[i] and optionally dfinal = dLoss/dfinal_state.
 *   dx      : (strided output) [batch, seqlen, channels] io dtype.
 *   dweight : [channels, width] fp32;  dbias: [channels] fp32 or NULL.
 *   dinit   : [batch, width - 1, channels] io dtype, or NULL. */
ssd_status ssd_conv_bwd(const ssd_conv_problem* prob, const void* x, const ssd_strides* x_strides,
                        const float* weight, const float* bias, const void* init_state,
                        const void* const* dy, const void* dfinal, void* dx,
                        const ssd_strides* dx_strides, float* dweight, float* dbias, void* dinit,
                        void* workspace, size_t workspace_bytes, void* stream);

/* -------------------------------------------------------------- selective scan
 *
 * For every batch b, channel c and state n, with group g = c / (channels /
 * ngroups) and dt' from dt as ssd_dt_transform says (dt itself without one):
 *     h_t = exp(dt'_t A[c, n]) h_{t-1} + dt'_t x_t B_t[g, n]
 *     s_t = sum_n C_t[g, n] h_t[n] + D[c] x_t
 *     y_t = s_t                        without z
 *         = s_t z_t / (1 + exp(-z_t))  with z
 * dt_bias, where given, is [channels].  Preconditions, not checked: dt' >= 0 and
 * A <= 0, inputs finite.
 */
typedef struct {
  int64_t batch;
  int64_t seqlen;
  int64_t channels;
  int64_t dstate;   /* N, at most 64 */
  int64_t ngroups;  /* divides channels */
  int32_t io_dtype;
  int32_t reserved; /* must be 0 */
} ssd_selscan_problem;

ssd_status ssd_selscan_fwd_workspace_size(const ssd_selscan_problem* prob, size_t* bytes);

/* Prompt.
 *   x, dt, y    : [batch, seqlen, channels] io dtype.
 *   A           : [channels, dstate] fp32;  D: [channels] fp32 or NULL.
 *   B, C        : (strided) [batch, seqlen, ngroups * dstate] io dtype.
 *   z           : (strided) [batch, seqlen, channels] io dtype, or NULL.
 *   init_state, final_state : [batch, channels, dstate] fp32, or NULL.
 *   workspace   : ssd_selscan_fwd_workspace_size bytes (which may be 0: then it
 *                 may be NULL).
 * Errors: UNSUPPORTED for dstate > 64, batch > 65535, several tokens of z 2^28 bytes
 * or more apart, or sizes past a launch's 2^32 threads. */
ssd_status ssd_selscan_fwd(const ssd_selscan_problem* prob, const ssd_dt_transform* dtx,
                           const void* x, const void* dt, const float* A, const void* B,
                           const ssd_strides* b_strides, const void* C,
                           const ssd_strides* c_strides, const float* D, const void* z,
                           const ssd_strides* z_strides, const float* init_state, void* y,
                           float* final_state, void* workspace, size_t workspace_bytes,
                           void* stream);

/* Single tokens: advances `state` [batch, channels, dstate] fp32 in place
 * through seqlen tokens, one at a time. */
ssd_status ssd_selscan_step(const ssd_selscan_problem* prob, const ssd_dt_transform* dtx,
                            float* state, const void* x, const void* dt, const float* A,
                            const void* B, const ssd_strides* b_strides, const void* C,
                            const ssd_strides* c_strides, const float* D, const void* z,
                            const ssd_strides* z_strides, void* y, void* stream);

ssd_status ssd_selscan_bwd_workspace_size(const ssd_selscan_problem* prob, size_t* bytes);

/* Gradients, given dy = dLoss/dy and optionally dfinal = dLoss/dfinal_state.
 *   dx, ddt   : [batch, seqlen, channels] io dtype; ddt with respect to the dt
 *               argument (through bias, softplus and clamp, whose ends pass it).
 *   dA        : [channels, dstate] fp32.
 *   dB, dC    : [batch, seqlen, ngroups, dstate] io dtype, contiguous.
 *   dD, ddt_bias : [channels] fp32, or NULL.
 *   dz        : (strided output) [batch, seqlen, channels] io dtype, required
 *               with z and ignored without.
 *   dinit     : [batch, channels, dstate] fp32, or NULL.
 * Everything between is fp32.  Errors as for ssd_selscan_fwd. */
ssd_status ssd_selscan_bwd(const ssd_selscan_problem* prob, const ssd_dt_transform* dtx,
                           const void* x, const void* dt, const float* A, const void* B,
                           const ssd_strides* b_strides, const void* C,
                           const ssd_strides* c_strides, const float* D, const void* z,
                           const ssd_strides* z_strides, const float* init_state, const void* dy,
                           const float* dfinal, void* dx, void* ddt, float* dA, void* dB, void* dC,
                           float* dD, void* dz, const ssd_strides* dz_strides, float* dinit,
                           float* ddt_bias, void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------ gated norm
 *
 * A token's channels fall into ngroups groups of S.  With s(z) = z / (1 + exp(-z))
 * (1 without z) and, in each group, r = (sum(u^2) / S + eps)^(-1/2):
 *     norm_before_gate 0:  u = x s(z),  y = weight u r
 *     norm_before_gate 1:  u = x,       y = weight u r s(z)
 * The sums of u^2 and, for the gradients, of weight dy u (dy s(z) u where the norm
 * comes first) are fp32 and have to fit it; with eps 0 a group has to have an u that
 * is not 0.
 */
typedef struct {
  int64_t batch;
  int64_t seqlen;
  int64_t channels;
  int64_t ngroups;          /* divides channels; at most 8192 channels per group */
  float eps;                /* finite, >= 0 */
  int32_t norm_before_gate; /* 0 or 1 */
  int32_t io_dtype;
  int32_t reserved;         /* must be 0 */
} ssd_gated_norm_problem;

/*   x, y   : [batch, seqlen, channels] io dtype.
 *   z      : (strided) [batch, seqlen, channels] io dtype, or NULL.
 *   weight : [channels] fp32. */
ssd_status ssd_gated_norm_fwd(const ssd_gated_norm_problem* prob, const void* x, const void* z,
                              const ssd_strides* z_strides, const float* weight, void* y,
                              void* stream);

ssd_status ssd_gated_norm_bwd_workspace_size(const ssd_gated_norm_problem* prob, size_t* bytes);

/* Gradients, given dy [batch, seqlen, channels] io dtype.
 *   dx      : [batch, seqlen, channels] io dtype.
 *   dz      : (strided output), required with z and ignored without.
 *   dweight : [channels] fp32. */
ssd_status ssd_gated_norm_bwd(const ssd_gated_norm_problem* prob, const void* x, const void* z,
                              const ssd_strides* z_strides, const float* weight, const void* dy,
                              void* dx, void* dz, const ssd_strides* dz_strides, float* dweight,
                              void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBSSD_SSD_LAYER_H */
