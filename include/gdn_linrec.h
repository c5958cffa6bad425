/*
 * gdn_linrec.h -- the gated linear recurrence with a vector state (libgdn.so):
 * whole sequences, their gradients, and one token in place.
 *
 * Each channel has its own decay at each token, a_t = exp(log_a_t), log_a <= 0:
 *
 *     h_t = a_t h_{t-1} + c(a_t) x_t,   y_t = h_t
 *
 * input_scale chooses c: GDN_LINREC_PLAIN 1, GDN_LINREC_COMPLEMENT 1 - a,
 * GDN_LINREC_ROOT sqrt(1 - a^2).  Hybrid stacks put such layers next to the
 * gated delta rule's; the decays come from the same kind of gates.
 *
 * The conventions are those of gdn.h and gdn_train.h: device pointers owned by
 * the caller, no allocation and no synchronisation inside, work enqueued on
 * `stream` (whose device must be the current one), host-side validation that
 * launches nothing on a refusal, status codes of gdn_status, gdn_last_route()
 * naming what ran.  Entry points are reentrant; a workspace is used in the
 * stream's order only, needs no initialisation, and is not to be shared by
 * calls that may overlap (two streams, two captured graphs replayed at once;
 * results are then wrong or NaN).
 * Kernels only, so all can be captured into a HIP graph.  The same bits run to
 * run.  Outputs must not overlap inputs or each other (equal pointers are refused;
 * gdn_linrec_step_plan compares no addresses).
 */
#ifndef GDN_LINREC_H
#define GDN_LINREC_H

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum gdn_linrec_scale { GDN_LINREC_PLAIN = 0, GDN_LINREC_COMPLEMENT = 1, GDN_LINREC_ROOT = 2 } gdn_linrec_scale;

/* Rows.  dense (cu_seqlens == NULL): B sequences of T rows, B * T rows in all;
 * packed: T rows in all, cu_seqlens device int32 [B+1], cu[0] = 0,
 * non-decreasing, cu[B] <= T (values outside [0, T] are clamped into it).
 * Sequences may be empty.  Rows behind cu[B] belong to no sequence: nothing
 * there is used (infinities and NaN neither), and outputs are left as they were.
 * Row r of a tensor is the D values at base + r * stride (elements, each
 * stride >= D).  io_dtype is the type of x, y, dy and dx, gate_dtype that of
 * log_a and dlog_a: GDN_F32 or GDN_BF16 each, but F32 rows take F32 gates only.
 * h0, h_final, dh_final, dh0: [B][D] fp32, each may be NULL (zero, or not
 * wanted).  States, decays and sums are fp32; each output is rounded once.
 * A state that is infinite or NaN is one of both from there on until its sequence
 * ends (runs of rows are joined by the products of their decays), no further.
 *
 * log_a <= 0, finite or -infinity (a reset: a = 0).  With PLAIN a positive one makes
 * the state grow: decays are multiplied over runs of rows of one sequence, and no such
 * product may pass fp32's range.  The other scales have no value there.
 *
 * gdn_linrec_backward: with D_t the gradient of h_t (dy_t plus what the later
 * rows hand back; dh_final enters behind the last row),
 *   D_t = dy_t + a_{t+1} D_{t+1},   dx_t = c D_t,   dh0 = a_1 D_1,
 *   dlog_a_t = D_t (a_t h_{t-1} + c'(a_t) x_t),  c' = dc/dlog_a: 0, -a, -a^2 / c.
 * y is the forward call's output, from which h_{t-1} is read as it was stored
 * (with bf16 rows rounded to bf16: 2^-9 of the term, as dlog_a's own rounding);
 * h0 the forward call's (NULL: zero).  x is read where input_scale is not PLAIN
 * and may be NULL otherwise.  Where c is 0 (log_a = 0) c' x, which is infinite
 * with ROOT, counts as 0.
 * An empty sequence's h_final is its h0, its dh0 its dh_final.
 *
 * workspace: gdn_linrec_workspace_bytes() bytes, asked with the same sizes and
 * packed = (cu_seqlens != NULL), aligned to 16 bytes; it covers both directions.
 *
 * Limits: B, D >= 1, T >= 0, B <= 65535, D <= 2^20, at most 2^30 rows, and
 * ceil(rows / 64) * ceil(D / 64) < 2^23 (2^35 values).
 * Returns GDN_OK, GDN_ERR_NULL, GDN_ERR_SHAPE, GDN_ERR_DIM_LIMIT (D),
 * GDN_ERR_DTYPE, GDN_ERR_STRIDE, GDN_ERR_WORKSPACE or GDN_ERR_HIP.
 */
size_t gdn_linrec_workspace_bytes(int B, int T, int D, int packed);

int gdn_linrec_forward(const void* x, const void* log_a, const float* h0, void* y, float* h_final, int B,
                       int T, int D, int64_t x_stride, int64_t a_stride, int64_t y_stride,
                       const int32_t* cu_seqlens, int input_scale, int io_dtype, int gate_dtype,
                       void* workspace, size_t workspace_bytes, hipStream_t stream);
int gdn_linrec_forward_plan(const void* x, const void* log_a, const float* h0, void* y, float* h_final, int B,
                            int T, int D, int64_t x_stride, int64_t a_stride, int64_t y_stride,
                            const int32_t* cu_seqlens, int input_scale, int io_dtype, int gate_dtype,
                            void* workspace, size_t workspace_bytes);

int gdn_linrec_backward(const void* x, const void* log_a, const void* y, const float* h0, const void* dy,
                        const float* dh_final, void* dx, void* dlog_a, float* dh0, int B, int T, int D,
                        int64_t x_stride, int64_t a_stride, int64_t y_stride, int64_t dy_stride,
                        int64_t dx_stride, int64_t da_stride, const int32_t* cu_seqlens, int input_scale,
                        int io_dtype, int gate_dtype, void* workspace, size_t workspace_bytes,
                        hipStream_t stream);
int gdn_linrec_backward_plan(const void* x, const void* log_a, const void* y, const float* h0, const void* dy,
                             const float* dh_final, void* dx, void* dlog_a, float* dh0, int B, int T, int D,
                             int64_t x_stride, int64_t a_stride, int64_t y_stride, int64_t dy_stride,
                             int64_t dx_stride, int64_t da_stride, const int32_t* cu_seqlens, int input_scale,
                             int io_dtype, int gate_dtype, void* workspace, size_t workspace_bytes);

/* One token of B sequences, in place: h_table[b] (device array of device
 * pointers, as in gdn_decode_step) points at sequence b's state [D] fp32, read
 * and written once; row b of x, log_a and y is its token.  A NULL entry is a
 * padding row: nothing of it is read, and its row of y is left as it was.  The
 * entries that are not NULL must differ, and point at multiples of 4 bytes.
 * Limits: 1 <= B <= 65535, 1 <= D <= 2^20.  Returns GDN_OK, GDN_ERR_NULL,
 * GDN_ERR_SHAPE, GDN_ERR_DIM_LIMIT (D), GDN_ERR_DTYPE, GDN_ERR_STRIDE or GDN_ERR_HIP.
 */
int gdn_linrec_step(float* const* h_table, const void* x, const void* log_a, void* y, int B, int D,
                    int64_t x_stride, int64_t a_stride, int64_t y_stride, int input_scale, int io_dtype,
                    int gate_dtype, hipStream_t stream);
int gdn_linrec_step_plan(float* const* h_table, const void* x, const void* log_a, void* y, int B, int D,
                         int64_t x_stride, int64_t a_stride, int64_t y_stride, int input_scale, int io_dtype,
                         int gate_dtype);

#ifdef __cplusplus
}
#endif

#endif /* GDN_LINREC_H */
