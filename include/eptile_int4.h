/*
 * eptile -- 4-bit group-scaled weights and 8-bit activation checkpoints (sm_100a).
 *
 * C ABI of libeptile.so beside eptile.h, with its rules: plain pointers and sizes, no exceptions, an
 * ep_status from every call, every buffer the caller's.
 *
 * A weight layout that needs no entropy decode, for linear layers that are served token by token or
 * whose scales are trained (no counterpart in the EntroPack pages; it stands beside the INT8 / FP8
 * code containers):
 *
 *   W[o, k] = s[o, k / group] q[o, k],  q in -8 .. 7, group 32, 64 or 128 inputs.
 *
 *   codes   n rows of ceil(k / 32) * 16 bytes, 16-byte aligned.  A 32-bit little-endian word holds eight
 *           consecutive inputs, each q + 8 in four bits: inputs 0, 2, 4, 6 of the eight in bits 0, 4, 8, 12,
 *           inputs 1, 3, 5, 7 in bits 16, 20, 24, 28.  Padding inputs hold q = 0 (the word 0x88888888).
 *   scales  n x ceil(k / group), row-major, of `dtype` (EP_BF16 or EP_FP16), which is also the type of
 *           the activations, gradients, bias and outputs of the products below.
 *
 * Activations and gradients are row-major with rows `ld` elements apart (ld >= the row's length; not
 * read for one row); outputs are contiguous and overlap no input.  Products are summed in fp32 and
 * rounded once to `dtype`.  ep_int4_linear of up to 16 tokens takes q, s and x exactly; above that, and in
 * ep_int4_linear_dx, the weight s q is rounded to `dtype` first, as is the checkpoint's a c in
 * ep_int4_scale_grad: an FP16 |s q| from 65520 on (scales from 8192 on) is then infinite, one up to 2^-25
 * zero.  On what is so rounded, NaN and infinities propagate as in the formulas.
 * m = 0 does nothing (ep_int4_scale_grad: writes zeros).
 *
 * Every call is asynchronous on `stream`, allocates nothing, needs no workspace, keeps nothing between
 * calls and gives the same bits on every call on one GPU; calls may overlap and be captured into graphs.
 * d_status (nullable device uint32): EP_DEC_TIMEOUT is ORed in if a copy into shared memory does not
 * complete within the kernels' poll limit (the output is then not valid).
 * EP_ERR_INVALID_ARG: a null or misaligned pointer, sizes below 1 (m below 0) or above 2^30, another group
 * or dtype; EP_ERR_UNSUPPORTED: the launch would exceed the grid's limits; EP_ERR_CUDA: the launch failed.
 */
#ifndef EPTILE_INT4_H
#define EPTILE_INT4_H

#include "eptile.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The weight from n x k elements of BF16, FP16 or FP32, rows ldw apart: per group s = max |w| / 7
 * (rounded to fp32, then to scale_dtype; 1 where that is 0) and q = w / s rounded to the nearest
 * integer, ties to even, in -7 .. 7.  A group that holds a NaN or an infinity, or whose scale overflows
 * scale_dtype, gets s = NaN and q = 0. */
int ep_int4_quantize(const void *d_w, int32_t dtype, int64_t n, int64_t k, int64_t ldw, int32_t group,
                     void *d_codes, void *d_scales, int32_t scale_dtype, ep_stream_t stream);

/* n x k elements of dtype: s q, rounded once. */
int ep_int4_dequantize(const void *d_codes, const void *d_scales, int32_t dtype, int64_t n, int64_t k,
                       int32_t group, void *d_out, ep_stream_t stream);

/* A linear layer's forward: y[t, o] = sum_k x[t, k] W[o, k] (+ bias[o], nullable), t < m. */
int ep_int4_linear(const void *d_codes, const void *d_scales, int64_t n, int64_t k, int32_t group, int32_t dtype,
                   const void *d_x, int64_t m, int64_t ldx, const void *d_bias, void *d_y, uint32_t *d_status,
                   ep_stream_t stream);

/* Its input gradient: dx[t, k] = sum_o dy[t, o] W[o, k]. */
int ep_int4_linear_dx(const void *d_codes, const void *d_scales, int64_t n, int64_t k, int32_t group, int32_t dtype,
                      const void *d_dy, int64_t m, int64_t lddy, void *d_dx, uint32_t *d_status,
                      ep_stream_t stream);

/* An 8-bit checkpoint of m x k activations (BF16, FP16 or FP32, rows ldx apart): per token and group of
 * 128 features a = max |x| / 127 (fp32; 1 where that is 0) and c = x / a rounded to the nearest integer,
 * ties to even, in -127 .. 127.  codes: m rows of ceil(k / 16) * 16 bytes (padding 0), 16-byte aligned;
 * scales: m x ceil(k / 128) fp32.  A group that holds a NaN or an infinity gets a = NaN and c = 0. */
int ep_act8_pack(const void *d_x, int32_t dtype, int64_t m, int64_t k, int64_t ldx, void *d_codes, float *d_scales,
                 ep_stream_t stream);

/* m x k elements of dtype (BF16, FP16 or FP32): a c, rounded once. */
int ep_act8_unpack(const void *d_codes, const float *d_scales, int64_t m, int64_t k, void *d_out, int32_t dtype,
                   ep_stream_t stream);

/* The gradient of every group scale from the output's gradient and the forward's checkpointed input:
 * ds[o, g] = sum over k in group g of q[o, k] sum_t dy[t, o] a[t, k / 128] c[t, k], n x ceil(k / group) of
 * dtype.  The weight gradient itself is never written.  dtype EP_FP16 holds a c in FP16 whatever the checkpoint
 * was made of: of activations that were BF16 or FP32, a group with one from about 65504 on makes its sums
 * infinite or NaN, and values up to 2^-25 add nothing (up to 2^-14 they lose digits). */
int ep_int4_scale_grad(const void *d_dy, int64_t lddy, const void *d_act, const float *d_act_scales, int64_t m,
                       const void *d_codes, int64_t n, int64_t k, int32_t group, int32_t dtype, void *d_ds,
                       uint32_t *d_status, ep_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif
