/*
 * gdn_train.h -- training entry points of libgdn.so: the gradients of the
 * gated delta rule, the norm of its outputs with its gradients, and activation
 * checkpoints in 8 bits, which both backward passes read.
 *
 * The conventions are those of gdn.h: device pointers owned by the caller, no
 * allocation and no synchronisation inside, work enqueued on `stream` (whose
 * device must be the current one), host-side validation that launches nothing
 * on a refusal, status codes of gdn_status, and gdn_last_route() naming what
 * ran.  Entry points are reentrant; a workspace is used in the stream's order
 * only, needs no initialisation, and is not to be shared by calls that may
 * overlap (two streams, two captured graphs replayed at once).  Every entry
 * point launches kernels only, so all can be captured into a HIP graph.
 * Results are the same bits run to run (no atomics).  Outputs must not overlap
 * inputs or each other.
 *
 * One training step of a layer: gdn_ckpt8_store of q, k, v; gdn_chunk_prefill;
 * gdn_norm_forward (which can write the checkpoints of its inputs); and on the
 * way back gdn_norm_backward, then gdn_chunk_backward.
 */
#ifndef GDN_TRAIN_H
#define GDN_TRAIN_H

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of activations held as 8-bit checkpoints (next to gdn_dtype's
 * GDN_F32 = 0 and GDN_BF16 = 1): OCP e4m3 codes with scale bytes. */
#define GDN_E4M3 2

/* Consecutive values of a row that share one scale byte. */
#define GDN_CKPT8_GROUP 128

/* ------------------------------------------------------------------------ */
/* Activation checkpoints in 8 bits.
 *
 * A row of d values is cut into groups of 128 (the last one may be shorter).
 * Group g of row r has one byte exps[r * ceil(d/128) + g] standing for the
 * scale 2^(byte - 127), the smallest power of two (from 2^-126) that brings
 * the group's largest finite magnitude to 448 or less (1 where all are zero),
 * and one e4m3 code per value, codes[r * d + j], the value over the scale
 * rounded to nearest even; infinities and NaN become the NaN code.  A code
 * times its scale is exactly a bf16 value, down to bf16's own smallest.
 * Groups whose largest magnitude is above 448 * 2^119 have byte 247, which
 * stands for 255 * 2^112 instead of 2^120: like this the largest finite value's
 * code, 256, is bf16's largest finite value and not infinity.  A code times that
 * one scale has 12 bits, and is rounded where bf16 takes it.
 *
 * store: x [rows][x_stride] (io_dtype F32 or BF16) -> codes, exps.
 * load:  codes, exps -> y [rows][y_stride] (out_dtype F32 or BF16).
 * codes [rows][d] and exps are dense.  rows >= 0 (0 launches nothing);
 * 1 <= d <= 2^30; a stride >= d.  Returns GDN_OK, GDN_ERR_NULL, GDN_ERR_SHAPE,
 * GDN_ERR_DIM_LIMIT (d), GDN_ERR_DTYPE, GDN_ERR_STRIDE or GDN_ERR_HIP.
 */
int gdn_ckpt8_store(const void* x, uint8_t* codes, uint8_t* exps, int64_t rows, int d,
                    int64_t x_stride, int io_dtype, hipStream_t stream);
int gdn_ckpt8_load(const uint8_t* codes, const uint8_t* exps, void* y, int64_t rows, int d,
                   int64_t y_stride, int out_dtype, hipStream_t stream);
int gdn_ckpt8_store_plan(const void* x, uint8_t* codes, uint8_t* exps, int64_t rows, int d,
                         int64_t x_stride, int io_dtype);
int gdn_ckpt8_load_plan(const uint8_t* codes, const uint8_t* exps, void* y, int64_t rows, int d,
                        int64_t y_stride, int out_dtype);

/* ------------------------------------------------------------------------ */
/* Norm of the recurrence's outputs, forward and backward.
 *
 * Row (t, h), t < T tokens and h < H heads, is the d values at
 * x + t * x_stride + h * d; z, y, dy, dx and dz likewise with their own token
 * strides (elements, each >= H * d), so that z may be a column block of a
 * fused projection.  H = 1 is the norm of a hidden row.
 *   n = (x - mean) / sqrt(var + eps)   (center != 0: layer norm)
 *   n = x / sqrt(mean(x^2) + eps)      (center == 0: RMS norm)
 *   a = n * w + b,   y = a * silu(z),  silu(z) = z / (1 + exp(-z))
 * with w [d] fp32, b [d] fp32 or NULL (no bias), z NULL for no gate.
 * Statistics and sums are fp32; each output is rounded once.
 *
 * gdn_norm_forward can also write the 8-bit checkpoints of its inputs (as
 * gdn_ckpt8_store does, rows = T * H): x_codes with x_exps, z_codes with
 * z_exps, each pair NULL or both given.
 *
 * gdn_norm_backward: with g = dy * silu(z) (g = dy without a gate),
 *   dw = sum over rows of g * n,   db = sum over rows of g   (fp32 [d])
 *   dx = (dn - n mean(dn n) - [center] mean(dn)) / sqrt(var + eps),  dn = g * w
 *   dz = dy * a * (s + z s (1 - s)),  s = 1 / (1 + exp(-z))
 * The statistics are formed again from x.  act_dtype is the type of x and z:
 * io_dtype, or GDN_E4M3, where x and z are code arrays (dense, x_stride =
 * z_stride = H * d) with x_exps and z_exps, and the gradients are those at the
 * values the codes stand for.  io_dtype is the type of dy, dx, dz.  dw is
 * required; db is required exactly when b is given, dz exactly when z is.
 * T == 0 writes zeros to dw and db.
 * workspace: gdn_norm_workspace_bytes(T, H, d) bytes (fp32 partial sums),
 * aligned to 16 bytes.
 *
 * Limits: T >= 0, H >= 1, 1 <= d <= 8192, T * H < 2^31, eps >= 0 and finite.
 * Returns GDN_OK, GDN_ERR_NULL, GDN_ERR_SHAPE, GDN_ERR_DIM_LIMIT (d),
 * GDN_ERR_DTYPE, GDN_ERR_STRIDE, GDN_ERR_WORKSPACE or GDN_ERR_HIP.
 */
size_t gdn_norm_workspace_bytes(int T, int H, int d);

int gdn_norm_forward(const void* x, const void* z, const float* w, const float* b, void* y,
                     uint8_t* x_codes, uint8_t* x_exps, uint8_t* z_codes, uint8_t* z_exps, int T,
                     int H, int d, int64_t x_stride, int64_t z_stride, int64_t y_stride, float eps,
                     int center, int io_dtype, hipStream_t stream);
int gdn_norm_forward_plan(const void* x, const void* z, const float* w, const float* b, void* y,
                          uint8_t* x_codes, uint8_t* x_exps, uint8_t* z_codes, uint8_t* z_exps, int T,
                          int H, int d, int64_t x_stride, int64_t z_stride, int64_t y_stride, float eps,
                          int center, int io_dtype);

int gdn_norm_backward(const void* x, const uint8_t* x_exps, const void* z, const uint8_t* z_exps,
                      const float* w, const float* b, const void* dy, void* dx, void* dz, float* dw,
                      float* db, int T, int H, int d, int64_t x_stride, int64_t z_stride,
                      int64_t dy_stride, int64_t dx_stride, int64_t dz_stride, float eps, int center,
                      int act_dtype, int io_dtype, void* workspace, size_t workspace_bytes,
                      hipStream_t stream);
int gdn_norm_backward_plan(const void* x, const uint8_t* x_exps, const void* z, const uint8_t* z_exps,
                           const float* w, const float* b, const void* dy, void* dx, void* dz, float* dw,
                           float* db, int T, int H, int d, int64_t x_stride, int64_t z_stride,
                           int64_t dy_stride, int64_t dx_stride, int64_t dz_stride, float eps, int center,
                           int act_dtype, int io_dtype, void* workspace, size_t workspace_bytes);

/* ------------------------------------------------------------------------ */
/* Gradients of the chunked gated delta rule (gdn_chunk_prefill).
 *
 * Given dout, the gradient of the outputs, and dh_final, the gradient of the
 * final states (NULL: zero), the gradients with respect to q, k, v, log_g,
 * beta and h0.  The states are formed again from q, k, v and the gates; the
 * forward call's outputs are not needed.  Layouts are gdn_chunk_prefill's:
 * dense [B][T][heads][d] or packed rows with cu_seqlens; dq, dk like q (summed
 * over the v-heads of a k-head), dv and dout like v, dlog_g and dbeta like
 * log_g; h0, dh_final, dh0: [B][Hv][dk][dv] fp32.  h0 NULL means zero initial
 * states, and dh0 may be NULL (not wanted) or given in either case.  Packed
 * rows behind the last sequence are left as they were; an empty sequence's dh0
 * is its dh_final.
 *
 * io_dtype: the type of q, k and v: GDN_F32, GDN_BF16, or GDN_E4M3, where they
 * are the code arrays of gdn_ckpt8_store with rows = tokens * heads, and
 * q_exps, k_exps, v_exps their scale bytes (one per row, as d <= 128; NULL
 * otherwise).  grad_dtype: the type of dout, dq, dk, dv, dlog_g and dbeta.
 * With GDN_BF16 the gates' gradients are rounded to bf16 too: they go into the
 * bf16 product with the gate projection's weight.
 *
 * Kernels: bf16 or 8-bit inputs with grad_dtype GDN_BF16, dk == dv == 128 and
 * 16-byte aligned pointers run on bf16 MFMA (fp32 accumulation and states);
 * everything else (dk, dv <= 128) on the generic fp32 kernels.
 * gdn_last_route() names what ran.
 * workspace: gdn_backward_workspace_bytes() bytes, asked with the same sizes,
 * types and packed = (cu_seqlens != NULL), aligned to 16 bytes; it covers
 * either route.
 *
 * Limits: B, Hk, Hv, dk, dv >= 1, T >= 0, B and Hv <= 65535, Hv a multiple of
 * Hk, dk, dv <= 128; any finite gates with log_g <= 0 (one under -104, whose decay
 * is zero in fp32, counts as -104).
 * Returns GDN_OK, GDN_ERR_NULL, GDN_ERR_SHAPE, GDN_ERR_HEAD_GROUPS,
 * GDN_ERR_DIM_LIMIT, GDN_ERR_DTYPE, GDN_ERR_WORKSPACE or GDN_ERR_HIP.
 */
size_t gdn_backward_workspace_bytes(int B, int T, int Hk, int Hv, int dk, int dv, int io_dtype,
                                    int grad_dtype, int packed);

int gdn_chunk_backward(const void* q, const void* k, const void* v, const uint8_t* q_exps,
                       const uint8_t* k_exps, const uint8_t* v_exps, const float* log_g,
                       const float* beta, const float* h0, const void* dout, const float* dh_final,
                       void* dq, void* dk_out, void* dv_out, void* dlog_g, void* dbeta, float* dh0,
                       int B, int T, int Hk, int Hv, int dk, int dv, const int32_t* cu_seqlens,
                       int io_dtype, int grad_dtype, void* workspace, size_t workspace_bytes,
                       hipStream_t stream);
int gdn_chunk_backward_plan(const void* q, const void* k, const void* v, const uint8_t* q_exps,
                            const uint8_t* k_exps, const uint8_t* v_exps, const float* log_g,
                            const float* beta, const float* h0, const void* dout, const float* dh_final,
                            void* dq, void* dk_out, void* dv_out, void* dlog_g, void* dbeta, float* dh0,
                            int B, int T, int Hk, int Hv, int dk, int dv, const int32_t* cu_seqlens,
                            int io_dtype, int grad_dtype, void* workspace, size_t workspace_bytes);

#ifdef __cplusplus
}
#endif

#endif /* GDN_TRAIN_H */
