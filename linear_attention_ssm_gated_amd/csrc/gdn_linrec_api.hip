// C ABI of the vector-state recurrence (include/gdn_linrec.h): host-side
// validation that names every refusal, the route line, and the launches.
#include "../../include/gdn_linrec.h"
#include "gdn_linrec_internal.h"

namespace {

using gdn::refuse_call;

constexpr int kMaxD = 1 << 20;
constexpr int64_t kMaxRows = 1 << 30;
constexpr int64_t kMaxTiles = (1 << 23) - 1;   // of 64 rows and 64 channels: the grid's threads stay under 2^32

int64_t rows_of(int B, int T, bool packed) { return packed ? T : (int64_t)B * T; }
bool too_many(int64_t rows, int D) { return (rows + 63) / 64 * ((D + 63) / 64) > kMaxTiles; }

// what the types and sizes of every entry point have in common
int check_common(const char* who, int B, int D, int scale, int io, int gate)
{
    if ((io != GDN_F32 && io != GDN_BF16) || (gate != GDN_F32 && gate != GDN_BF16))
        return refuse_call(GDN_ERR_DTYPE, who, "io_dtype and gate_dtype must be GDN_F32 or GDN_BF16");
    if (io == GDN_F32 && gate != GDN_F32) return refuse_call(GDN_ERR_DTYPE, who, "F32 rows take F32 gates");
    if (scale < GDN_LINREC_PLAIN || scale > GDN_LINREC_ROOT)
        return refuse_call(GDN_ERR_SHAPE, who, "input_scale must be one of gdn_linrec_scale");
    if (B < 1 || D < 1) return refuse_call(GDN_ERR_SHAPE, who, "need B, D >= 1");
    if (B > 65535) return refuse_call(GDN_ERR_SHAPE, who, "B > 65535 (grid limits)");
    if (D > kMaxD) return refuse_call(GDN_ERR_DIM_LIMIT, who, "D <= 2^20");
    return GDN_OK;
}

int check_rows(const char* who, const gdn::LinrecArgs& a)
{
    if (const int st = check_common(who, a.B, a.D, a.scale, a.io_dtype, a.gate_dtype)) return st;
    if (a.T < 0) return refuse_call(GDN_ERR_SHAPE, who, "need T >= 0");
    const int64_t rows = rows_of(a.B, a.T, a.cu != nullptr);
    if (rows > kMaxRows || too_many(rows, a.D))
        return refuse_call(GDN_ERR_SHAPE, who, "more than 2^30 rows, or ceil(rows / 64) * ceil(D / 64) >= 2^23");
    if (a.a_stride < a.D || a.y_stride < a.D) return refuse_call(GDN_ERR_STRIDE, who, "a row stride is shorter than its row");
    if ((!a.backward || a.scale != GDN_LINREC_PLAIN) && a.x_stride < a.D)
        return refuse_call(GDN_ERR_STRIDE, who, "a row stride is shorter than its row");
    if (a.backward && (a.dy_stride < a.D || a.dx_stride < a.D || a.da_stride < a.D))
        return refuse_call(GDN_ERR_STRIDE, who, "a row stride is shorter than its row");
    if (rows > 0) {
        if (!a.log_a || !a.y) return refuse_call(GDN_ERR_NULL, who, "log_a and y are required when there are rows");
        if ((!a.backward || a.scale != GDN_LINREC_PLAIN) && !a.x)
            return refuse_call(GDN_ERR_NULL, who, a.backward ? "x is required where input_scale is not PLAIN" : "x is required when there are rows");
        if (a.backward && (!a.dy || !a.dx || !a.dlog_a))
            return refuse_call(GDN_ERR_NULL, who, "dy, dx and dlog_a are required when there are rows");
    }
    if ((a.h0 && a.h0 == a.h_final) || (a.dh_final && a.dh_final == a.dh0) || (a.h0 && a.h0 == a.dh0))
        return refuse_call(GDN_ERR_SHAPE, who, "the states handed in and out must not share memory");
    const auto read = [&](const void* out) {
        return out && (out == a.x || out == a.log_a || (a.backward && (out == a.y || out == a.dy)));
    };
    if (rows > 0 && (a.backward ? read(a.dx) || read(a.dlog_a) || a.dx == a.dlog_a : read(a.y)))
        return refuse_call(GDN_ERR_SHAPE, who, "outputs must not share memory with inputs or each other");
    const size_t need = gdn::linrec_workspace_bytes(rows, a.D);
    if (need > 0 && (!a.workspace || a.workspace_bytes < need))
        return refuse_call(GDN_ERR_WORKSPACE, who, "workspace smaller than gdn_linrec_workspace_bytes()");
    if (reinterpret_cast<uintptr_t>(a.workspace) % 16 != 0)
        return refuse_call(GDN_ERR_WORKSPACE, who, "workspace must be 16-byte aligned");
    return GDN_OK;
}

gdn::LinrecArgs forward_args(const void* x, const void* log_a, const float* h0, void* y, float* h_final, int B,
                             int T, int D, int64_t x_stride, int64_t a_stride, int64_t y_stride,
                             const int32_t* cu_seqlens, int input_scale, int io_dtype, int gate_dtype,
                             void* workspace, size_t workspace_bytes)
{
    gdn::LinrecArgs a{};
    a.x = x; a.log_a = log_a; a.h0 = h0; a.y = y; a.h_final = h_final;
    a.B = B; a.T = T; a.D = D; a.x_stride = x_stride; a.a_stride = a_stride; a.y_stride = y_stride;
    a.cu = cu_seqlens; a.scale = input_scale; a.io_dtype = io_dtype; a.gate_dtype = gate_dtype;
    a.workspace = workspace; a.workspace_bytes = workspace_bytes;
    return a;
}

gdn::LinrecArgs backward_args(const void* x, const void* log_a, const void* y, const float* h0, const void* dy,
                              const float* dh_final, void* dx, void* dlog_a, float* dh0, int B, int T, int D,
                              int64_t x_stride, int64_t a_stride, int64_t y_stride, int64_t dy_stride,
                              int64_t dx_stride, int64_t da_stride, const int32_t* cu_seqlens, int input_scale,
                              int io_dtype, int gate_dtype, void* workspace, size_t workspace_bytes)
{
    gdn::LinrecArgs a = forward_args(x, log_a, h0, const_cast<void*>(y), nullptr, B, T, D, x_stride, a_stride,
                                     y_stride, cu_seqlens, input_scale, io_dtype, gate_dtype, workspace,
                                     workspace_bytes);
    a.dy = dy; a.dh_final = dh_final; a.dx = dx; a.dlog_a = dlog_a; a.dh0 = dh0;
    a.dy_stride = dy_stride; a.dx_stride = dx_stride; a.da_stride = da_stride;
    a.backward = true;
    return a;
}

gdn::LinrecStepArgs step_args(float* const* h_table, const void* x, const void* log_a, void* y, int B, int D,
                              int64_t x_stride, int64_t a_stride, int64_t y_stride, int input_scale, int io_dtype,
                              int gate_dtype)
{
    return gdn::LinrecStepArgs{h_table, x, log_a, y, B, D, x_stride, a_stride, y_stride, input_scale, io_dtype, gate_dtype};
}

}  // namespace

extern "C" {

size_t gdn_linrec_workspace_bytes(int B, int T, int D, int packed)
{
    if (B < 1 || T < 0 || D < 1 || B > 65535 || D > kMaxD) return 0;
    const int64_t rows = rows_of(B, T, packed != 0);
    return rows > kMaxRows || too_many(rows, D) ? 0 : gdn::linrec_workspace_bytes(rows, D);
}

int gdn_linrec_forward_plan(const void* x, const void* log_a, const float* h0, void* y, float* h_final, int B,
                            int T, int D, int64_t x_stride, int64_t a_stride, int64_t y_stride,
                            const int32_t* cu_seqlens, int input_scale, int io_dtype, int gate_dtype,
                            void* workspace, size_t workspace_bytes)
{
    const gdn::LinrecArgs a = forward_args(x, log_a, h0, y, h_final, B, T, D, x_stride, a_stride, y_stride, cu_seqlens,
                                           input_scale, io_dtype, gate_dtype, workspace, workspace_bytes);
    const int st = check_rows("gdn_linrec_forward", a);
    if (st != GDN_OK) return st;
    gdn::route_call(gdn::linrec_geometry(a), "");
    return GDN_OK;
}

int gdn_linrec_forward(const void* x, const void* log_a, const float* h0, void* y, float* h_final, int B, int T,
                       int D, int64_t x_stride, int64_t a_stride, int64_t y_stride, const int32_t* cu_seqlens,
                       int input_scale, int io_dtype, int gate_dtype, void* workspace, size_t workspace_bytes,
                       hipStream_t stream)
{
    const int st = gdn_linrec_forward_plan(x, log_a, h0, y, h_final, B, T, D, x_stride, a_stride, y_stride, cu_seqlens,
                                           input_scale, io_dtype, gate_dtype, workspace, workspace_bytes);
    if (st != GDN_OK) return st;
    return gdn::launch_status(gdn::launch_linrec(
        forward_args(x, log_a, h0, y, h_final, B, T, D, x_stride, a_stride, y_stride, cu_seqlens, input_scale,
                     io_dtype, gate_dtype, workspace, workspace_bytes),
        stream));
}

int gdn_linrec_backward_plan(const void* x, const void* log_a, const void* y, const float* h0, const void* dy,
                             const float* dh_final, void* dx, void* dlog_a, float* dh0, int B, int T, int D,
                             int64_t x_stride, int64_t a_stride, int64_t y_stride, int64_t dy_stride,
                             int64_t dx_stride, int64_t da_stride, const int32_t* cu_seqlens, int input_scale,
                             int io_dtype, int gate_dtype, void* workspace, size_t workspace_bytes)
{
    const gdn::LinrecArgs a = backward_args(x, log_a, y, h0, dy, dh_final, dx, dlog_a, dh0, B, T, D, x_stride,
                                            a_stride, y_stride, dy_stride, dx_stride, da_stride, cu_seqlens,
                                            input_scale, io_dtype, gate_dtype, workspace, workspace_bytes);
    const int st = check_rows("gdn_linrec_backward", a);
    if (st != GDN_OK) return st;
    gdn::route_call(gdn::linrec_geometry(a), "");
    return GDN_OK;
}

int gdn_linrec_backward(const void* x, const void* log_a, const void* y, const float* h0, const void* dy,
                        const float* dh_final, void* dx, void* dlog_a, float* dh0, int B, int T, int D,
                        int64_t x_stride, int64_t a_stride, int64_t y_stride, int64_t dy_stride,
                        int64_t dx_stride, int64_t da_stride, const int32_t* cu_seqlens, int input_scale,
                        int io_dtype, int gate_dtype, void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    const int st = gdn_linrec_backward_plan(x, log_a, y, h0, dy, dh_final, dx, dlog_a, dh0, B, T, D, x_stride,
                                            a_stride, y_stride, dy_stride, dx_stride, da_stride, cu_seqlens,
                                            input_scale, io_dtype, gate_dtype, workspace, workspace_bytes);
    if (st != GDN_OK) return st;
    return gdn::launch_status(gdn::launch_linrec(
        backward_args(x, log_a, y, h0, dy, dh_final, dx, dlog_a, dh0, B, T, D, x_stride, a_stride, y_stride, dy_stride,
                      dx_stride, da_stride, cu_seqlens, input_scale, io_dtype, gate_dtype, workspace, workspace_bytes),
        stream));
}

int gdn_linrec_step_plan(float* const* h_table, const void* x, const void* log_a, void* y, int B, int D,
                         int64_t x_stride, int64_t a_stride, int64_t y_stride, int input_scale, int io_dtype,
                         int gate_dtype)
{
    const char* who = "gdn_linrec_step";
    if (const int st = check_common(who, B, D, input_scale, io_dtype, gate_dtype)) return st;
    if (x_stride < D || a_stride < D || y_stride < D)
        return refuse_call(GDN_ERR_STRIDE, who, "a row stride is shorter than its row");
    if (!h_table || !x || !log_a || !y) return refuse_call(GDN_ERR_NULL, who, "h_table, x, log_a and y are required");
    gdn::route_call(gdn::linrec_step_geometry(step_args(h_table, x, log_a, y, B, D, x_stride, a_stride, y_stride,
                                                        input_scale, io_dtype, gate_dtype)),
                    "");
    return GDN_OK;
}

int gdn_linrec_step(float* const* h_table, const void* x, const void* log_a, void* y, int B, int D,
                    int64_t x_stride, int64_t a_stride, int64_t y_stride, int input_scale, int io_dtype,
                    int gate_dtype, hipStream_t stream)
{
    const int st = gdn_linrec_step_plan(h_table, x, log_a, y, B, D, x_stride, a_stride, y_stride, input_scale,
                                        io_dtype, gate_dtype);
    if (st != GDN_OK) return st;
    // (the plan compares no addresses; a row of y written over x or log_a of another workgroup would be read there)
    if (y == x || y == log_a || y == static_cast<const void*>(h_table))
        return refuse_call(GDN_ERR_SHAPE, "gdn_linrec_step", "y must not share memory with h_table, x or log_a");
    return gdn::launch_status(gdn::launch_linrec_step(
        step_args(h_table, x, log_a, y, B, D, x_stride, a_stride, y_stride, input_scale, io_dtype, gate_dtype), stream));
}

}  // extern "C"
