/*
 * ssd_block.h -- C ABI of libssd, third part: what stands around a layer in a
 * model and in its training step, on one AMD Instinct MI355X (gfx950).
 *
 *   ssd_add_norm_*           the residual addition with the RMS norm before a layer,
 *                            with an output in the io dtype, in 8 bits, or both;
 *   ssd_gated_norm_fwd_8bit  ssd_gated_norm_fwd (ssd_layer.h) with its output in 8
 *                            bits, for the output projection;
 *   ssd_quant8               values in 8 bits with a scale for each block: weights,
 *                            upstream gradients, by rows, transposed, or both;
 *   ssd_matmul8              the matrix product of two such operands: projections, and
 *                            the gradients of their inputs and weights;
 *   ssd_clip_grads           the global norm over many gradients, and clipping by it.
 *
 * A second-generation block is ssd_add_norm_fwd -> ssd_matmul8 -> ssd_conv_fwd ->
 * ssd_fwd_ex -> ssd_gated_norm_fwd_8bit -> ssd_matmul8; the next block adds the result to
 * the residual.  Single tokens take the same calls with few rows.
 *
 * 8-bit operands.  A matrix [rows, depth] that a product sums over depth is held as
 *     q     [rows, P] bytes, e4m3 (1 sign, 4 exponent, 3 mantissa bits, largest value 448,
 *           no infinities), P = depth rounded up to whole blocks of 128; zeros past depth;
 *     scale [P / 128, rows] fp32: a scale for each row and block ("by row"), or
 *           [P / 128, ceil(rows / 128)]: one for each 128 x 128 ("by tile");
 * and stands for q * scale.  The calls here make, for a block with magnitudes up to a,
 *     m = max(a, 2^-100),  q = e4m3(v * (448 / m)) to nearest, ties to even,  scale = m / 448.
 * A NaN is left out of a and gives a NaN; with an infinity the scale is infinite, and the
 * block stands for NaN.
 *
 * Everything ssd.h and ssd_layer.h say of ownership, streams, determinism, graph capture,
 * strided operands and errors (their kinds and their order) holds here.  8-bit
 * tensors and scales are 16-byte aligned.
 */
#ifndef LIBSSD_SSD_BLOCK_H
#define LIBSSD_SSD_BLOCK_H

#include "ssd_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SSD_BLOCK_ABI_VERSION 1

/* SSD_BLOCK_ABI_VERSION of the loaded library. */
int ssd_block_abi_version(void);

/* ----------------------------------------------------------- residual and norm
 *
 * For every token, over its C channels:
 *     h = x + residual, rounded to the residual's dtype (x without a residual)
 *     r = (sum(h^2) / C + eps)^(-1/2),  y = weight h r
 * The norm is taken of h as it is stored, so that the gradients, which read h, are
 * those of the forward pass.  The sum of h^2 is fp32 and has to fit it; with eps 0 a
 * token has to have an h that is not 0.
 */
typedef struct {
  int64_t batch;
  int64_t seqlen;
  int64_t channels;       /* at most 8192 */
  float eps;              /* finite, >= 0 */
  int32_t io_dtype;       /* of x, y, dy, dx */
  int32_t residual_dtype; /* of residual, h, dresidual; SSD_F32 where io_dtype is */
  int32_t reserved;       /* must be 0 */
} ssd_add_norm_problem;

/*   x        : (strided) [batch, seqlen, channels] io dtype.
 *   residual : [batch, seqlen, channels] residual dtype, or NULL.
 *   weight   : [channels] fp32.
 *   h        : [batch, seqlen, channels] residual dtype, or NULL; may be `residual`.
 *   y        : [batch, seqlen, channels] io dtype, or NULL.
 *   q, scale : the 8-bit y by row (rows = batch * seqlen, depth = channels), or both NULL.
 * One of y and q at least.  Errors: UNSUPPORTED for more than 8192 channels or 2^31 - 1 tokens, or
 * sizes past a launch's 2^32 threads: a token of up to 128 channels takes 16, of up to 256 takes 32,
 * beyond that at most 64 for each 512 channels. */
ssd_status ssd_add_norm_fwd(const ssd_add_norm_problem* prob, const void* x,
                            const ssd_strides* x_strides, const void* residual,
                            const float* weight, void* h, void* y, void* q, float* scale,
                            void* stream);

/* Workspace bytes of ssd_add_norm_bwd (part sums of the weight's gradient). */
ssd_status ssd_add_norm_bwd_workspace_size(const ssd_add_norm_problem* prob, size_t* bytes);

/* Gradients, given h as ssd_add_norm_fwd left it, dy = dLoss/dy [batch, seqlen, channels] io
 * dtype and optionally dh = dLoss/dh (residual dtype; what comes back along the residual).
 *   dx        : [batch, seqlen, channels] io dtype, or NULL.
 *   dresidual : [batch, seqlen, channels] residual dtype, or NULL; may be `dh`.  The same
 *               gradient as dx, rounded to its own type.
 *   dweight   : [channels] fp32.
 * One of dx and dresidual at least.  Errors: UNSUPPORTED for more than 8192 channels or 2^31 - 1
 * tokens. */
ssd_status ssd_add_norm_bwd(const ssd_add_norm_problem* prob, const void* h, const float* weight,
                            const void* dy, const void* dh, void* dx, void* dresidual,
                            float* dweight, void* workspace, size_t workspace_bytes, void* stream);

/* ssd_gated_norm_fwd with the output in 8 bits, by row (rows = batch * seqlen, depth =
 * channels).  Errors beside those of ssd_gated_norm_fwd: UNSUPPORTED for more than one
 * group whose channels are not whole blocks of 128, and past ssd_add_norm_fwd's limits of tokens
 * and threads (a group's channels in place of a token's). */
ssd_status ssd_gated_norm_fwd_8bit(const ssd_gated_norm_problem* prob, const void* x,
                                   const void* z, const ssd_strides* z_strides,
                                   const float* weight, void* q, float* scale, void* stream);

/* ------------------------------------------------------------------ quantising
 *
 * A matrix of rows = batch * seqlen and channels columns, in 8 bits:
 *   q,  scale   : as it is (depth = channels);
 *   qt, scale_t : transposed (rows of its own = channels, depth = batch * seqlen).
 * tile 0 scales by row, each form along its own depth; tile 1 by tile, and both
 * forms then hold the same values.
 */
typedef struct {
  int64_t batch;
  int64_t seqlen;
  int64_t channels;
  int32_t io_dtype;
  int32_t tile;     /* 0 or 1 */
  int64_t reserved; /* must be 0 */
} ssd_quant8_problem;

/*   x : (strided) [batch, seqlen, channels] io dtype.
 * q with scale, or qt with scale_t, or all four; the others NULL.
 * Errors: UNSUPPORTED for more than 2^31 - 1 rows or columns, or sizes past a launch's 2^32
 * threads: 16 for each block of a row where q is made alone with tile 0, else 256 for each 128 x
 * 128. */
ssd_status ssd_quant8(const ssd_quant8_problem* prob, const void* x, const ssd_strides* x_strides,
                      void* q, float* scale, void* qt, float* scale_t, void* stream);

/* -------------------------------------------------------------- matrix product
 *
 *     y[m, n] = sum over blocks b of  xs[b, m] ws[b, n] sum_{k in block b} x[m, k] w[n, k]
 * with ws by row, or by tile (ws[b, n / 128]); xs is by row.  Products and sums of a
 * block are those of the matrix cores, scaled and added in fp32; y is rounded once.
 * Products of two scales have to fit fp32.
 *
 * A projection takes x by row and the weight [cols, depth] by tile; the gradient of its input
 * takes the upstream gradient by row and the weight's transposed form; the gradient of the
 * weight takes both transposed forms by row (rows and cols the channels, depth the tokens).
 */
typedef struct {
  int64_t rows;          /* of x and y */
  int64_t cols;          /* rows of w, columns of y */
  int64_t depth;         /* a multiple of 128: the padded one */
  int32_t w_tile;        /* w scaled 1: by tile, 0: by row */
  int32_t out_dtype;     /* ssd_dtype of y */
  int64_t reserved;      /* must be 0 */
} ssd_matmul8_problem;

/* Workspace bytes (0 where the product is not split along its depth). */
ssd_status ssd_matmul8_workspace_size(const ssd_matmul8_problem* prob, size_t* bytes);

/*   x, xs : [rows, depth] e4m3, [depth / 128, rows] fp32.
 *   w, ws : [cols, depth] e4m3, [depth / 128, cols or ceil(cols / 128)] fp32.
 *   y     : [rows, cols] out dtype.
 *   workspace : ssd_matmul8_workspace_size bytes (which may be 0: then it may be NULL).
 * Errors: BAD_SHAPE for a depth that is not a multiple of 128; UNSUPPORTED for more than
 * 2^31 - 1 rows or cols, a depth above 2^23, or sizes past a launch's 2^32 threads (up to 16 rows
 * 2^27 cols, beyond that 2^24 tiles of 64 x 64 of y or larger ones). */
ssd_status ssd_matmul8(const ssd_matmul8_problem* prob, const void* x, const float* xs,
                       const void* w, const float* ws, void* y, void* workspace,
                       size_t workspace_bytes, void* stream);

/* -------------------------------------------------------------------- clipping
 *
 * Over all n tensors together:
 *     norm = grad_scale sqrt(sum g^2)
 *     c    = grad_scale min(1, max_norm / (norm + eps)), grad_scale where norm is not finite
 *     out  = g c
 * The sum is 64-bit; c is rounded to fp32, and out once to its type.  Whether the norm is
 * finite goes by its rounding to fp32, which is what `norm` holds: a caller that skips a step
 * whose norm is not finite finds that there.
 */
typedef struct {
  const void* grad;  /* contiguous, aligned to its element */
  void* out;         /* the same number of elements; may be grad where the dtypes agree */
  int64_t elements;  /* >= 0; 0: both pointers are ignored */
  int32_t dtype;     /* of grad */
  int32_t out_dtype;
} ssd_grad;

typedef struct {
  double max_norm;   /* > 0; INFINITY: nothing is clipped */
  double eps;        /* finite, >= 0 */
  double grad_scale; /* finite, > 0: 1 / the loss scale or the number of micro-batches */
  int64_t reserved;  /* must be 0 */
} ssd_clip_options;

/* Workspace bytes (part sums) for these tensors; only their elements are read. */
ssd_status ssd_clip_grads_workspace_size(const ssd_grad* grads, int64_t n, size_t* bytes);

/*   grads : a host array of n >= 1 tensors, read before the call returns.
 *   norm  : [1] fp32.
 * Errors: BAD_VALUE also where an out overlaps another tensor's grad or out, its own grad but
 * not wholly, or `norm`; UNSUPPORTED, ahead of that, for more than 2^20 tensors or 2^40 elements. */
ssd_status ssd_clip_grads(const ssd_grad* grads, int64_t n, const ssd_clip_options* options,
                          float* norm, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBSSD_SSD_BLOCK_H */
