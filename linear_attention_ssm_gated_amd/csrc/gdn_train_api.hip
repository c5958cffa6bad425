// C ABI of the training entry points (include/gdn_train.h): host-side
// validation that names every refusal, the route line, and the launches.
#include "../../include/gdn_train.h"
#include "gdn_train_internal.h"

#include <math.h>

#include <mutex>
#include <set>
#include <utility>

namespace gdn {
hipError_t allow_lds(const void* kernel, size_t bytes)
try {
    static std::mutex mu;
    static std::set<std::pair<int, const void*>> allowed;
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    if (allowed.count({dev, kernel})) return hipSuccess;
    e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == hipSuccess) allowed.insert({dev, kernel});
    return e;
} catch (...) {          // the set's memory: nothing leaves a C entry point
    return hipErrorOutOfMemory;
}
}  // namespace gdn

namespace {

using gdn::refuse_call;

bool wide_dtype(int d) { return d == GDN_F32 || d == GDN_BF16; }

int check_ckpt(const gdn::CkptArgs& a, bool store)
{
    const char* who = store ? "gdn_ckpt8_store" : "gdn_ckpt8_load";
    if (!wide_dtype(a.dtype)) return refuse_call(GDN_ERR_DTYPE, who, "dtype must be GDN_F32 or GDN_BF16");
    if (a.rows < 0 || a.d < 1) return refuse_call(GDN_ERR_SHAPE, who, "need rows >= 0 and d >= 1");
    if (a.d > (1 << 30)) return refuse_call(GDN_ERR_DIM_LIMIT, who, "d <= 2^30");
    if (a.stride < a.d) return refuse_call(GDN_ERR_STRIDE, who, "a row stride is shorter than its row");
    const bool all = store ? a.x && a.codes && a.exps_out : a.x && a.exps_in && a.y;
    if (a.rows > 0 && !all)
        return refuse_call(GDN_ERR_NULL, who, store ? "x, codes and exps are required" : "codes, exps and y are required");
    return GDN_OK;
}

int check_norm(const gdn::NormArgs& a, bool backward)
{
    const char* who = backward ? "gdn_norm_backward" : "gdn_norm_forward";
    if (!wide_dtype(a.io_dtype)) return refuse_call(GDN_ERR_DTYPE, who, "io_dtype must be GDN_F32 or GDN_BF16");
    if (backward && a.act_dtype != a.io_dtype && a.act_dtype != GDN_E4M3)
        return refuse_call(GDN_ERR_DTYPE, who, "act_dtype must be io_dtype or GDN_E4M3");
    if (a.T < 0 || a.H < 1 || a.d < 1) return refuse_call(GDN_ERR_SHAPE, who, "need T >= 0, H >= 1 and d >= 1");
    if ((int64_t)a.T * a.H >= (1LL << 31)) return refuse_call(GDN_ERR_SHAPE, who, "T * H must stay below 2^31");
    if (a.d > 8192) return refuse_call(GDN_ERR_DIM_LIMIT, who, "d <= 8192");
    if (!(a.eps >= 0.0f) || !isfinite(a.eps)) return refuse_call(GDN_ERR_SHAPE, who, "eps must be finite and not negative");
    const int64_t row = (int64_t)a.H * a.d;
    if (a.x_stride < row || a.y_stride < row || (a.z && a.z_stride < row) || (backward && a.dx_stride < row) ||
        (backward && a.z && a.dz_stride < row))
        return refuse_call(GDN_ERR_STRIDE, who, "a token stride is shorter than its H * d values");
    if (!a.w) return refuse_call(GDN_ERR_NULL, who, "w is required");
    if (!backward) {
        if (a.T > 0 && (!a.x || !a.y)) return refuse_call(GDN_ERR_NULL, who, "x and y are required");
        if (!a.x_codes != !a.x_exps_out || !a.z_codes != !a.z_exps_out)
            return refuse_call(GDN_ERR_NULL, who, "codes and exps come together");
        if (a.T > 0 && a.z_codes && !a.z) return refuse_call(GDN_ERR_NULL, who, "z_codes without z");
        return GDN_OK;
    }
    if (!a.dw) return refuse_call(GDN_ERR_NULL, who, "dw is required");
    if (!a.b != !a.db) return refuse_call(GDN_ERR_NULL, who, "b and db come together");
    if (a.T == 0) return GDN_OK;
    if (!a.x || !a.dy || !a.dx) return refuse_call(GDN_ERR_NULL, who, "x, dy and dx are required when T > 0");
    if (!a.z != !a.dz) return refuse_call(GDN_ERR_NULL, who, "z and dz come together");
    if (a.act_dtype == GDN_E4M3) {
        if (!a.x_exps || (a.z && !a.z_exps))
            return refuse_call(GDN_ERR_NULL, who, "8-bit activations need their exps");
        if (a.x_stride != row || (a.z && a.z_stride != row))
            return refuse_call(GDN_ERR_STRIDE, who, "8-bit activations are dense: stride H * d");
    }
    if (!a.workspace || a.workspace_bytes < gdn::norm_workspace_bytes(a.T, a.H, a.d))
        return refuse_call(GDN_ERR_WORKSPACE, who, "workspace smaller than gdn_norm_workspace_bytes()");
    if (reinterpret_cast<uintptr_t>(a.workspace) % 16 != 0)
        return refuse_call(GDN_ERR_WORKSPACE, who, "workspace must be 16-byte aligned");
    return GDN_OK;
}

gdn::NormArgs forward_args(const void* x, const void* z, const float* w, const float* b, void* y,
                           uint8_t* x_codes, uint8_t* x_exps, uint8_t* z_codes, uint8_t* z_exps, int T,
                           int H, int d, int64_t x_stride, int64_t z_stride, int64_t y_stride, float eps,
                           int center, int io_dtype)
{
    gdn::NormArgs a{};
    a.x = x; a.z = z; a.w = w; a.b = b; a.y = y;
    a.x_codes = x_codes; a.x_exps_out = x_exps; a.z_codes = z_codes; a.z_exps_out = z_exps;
    a.T = T; a.H = H; a.d = d; a.x_stride = x_stride; a.z_stride = z_stride; a.y_stride = y_stride;
    a.eps = eps; a.center = center != 0; a.io_dtype = a.act_dtype = io_dtype;
    return a;
}

gdn::NormArgs backward_args(const void* x, const uint8_t* x_exps, const void* z, const uint8_t* z_exps,
                            const float* w, const float* b, const void* dy, void* dx, void* dz, float* dw,
                            float* db, int T, int H, int d, int64_t x_stride, int64_t z_stride,
                            int64_t dy_stride, int64_t dx_stride, int64_t dz_stride, float eps, int center,
                            int act_dtype, int io_dtype, void* workspace, size_t workspace_bytes)
{
    gdn::NormArgs a{};
    a.x = x; a.x_exps = x_exps; a.z = z; a.z_exps = z_exps; a.w = w; a.b = b;
    a.dy = dy; a.dx = dx; a.dz = dz; a.dw = dw; a.db = db;
    a.T = T; a.H = H; a.d = d; a.x_stride = x_stride; a.z_stride = z_stride; a.y_stride = dy_stride;
    a.dx_stride = dx_stride; a.dz_stride = dz_stride;
    a.eps = eps; a.center = center != 0; a.act_dtype = act_dtype; a.io_dtype = io_dtype;
    a.workspace = workspace; a.workspace_bytes = workspace_bytes;
    return a;
}

gdn::CkptArgs store_args(const void* x, uint8_t* codes, uint8_t* exps, int64_t rows, int d, int64_t stride, int dtype)
{
    gdn::CkptArgs a{};
    a.x = x; a.codes = codes; a.exps_out = exps; a.rows = rows; a.d = d; a.stride = stride; a.dtype = dtype;
    return a;
}

gdn::CkptArgs load_args(const uint8_t* codes, const uint8_t* exps, void* y, int64_t rows, int d, int64_t stride, int dtype)
{
    gdn::CkptArgs a{};
    a.x = codes; a.exps_in = exps; a.y = y; a.rows = rows; a.d = d; a.stride = stride; a.dtype = dtype;
    return a;
}

gdn::BackwardArgs chunk_args(const void* q, const void* k, const void* v, const uint8_t* q_exps,
                             const uint8_t* k_exps, const uint8_t* v_exps, const float* log_g,
                             const float* beta, const float* h0, const void* dout, const float* dh_final,
                             void* dq, void* dk_out, void* dv_out, void* dlog_g, void* dbeta, float* dh0,
                             int B, int T, int Hk, int Hv, int dk, int dv, const int32_t* cu_seqlens,
                             int io_dtype, int grad_dtype, void* workspace, size_t workspace_bytes)
{
    gdn::BackwardArgs a{};
    a.q = q; a.k = k; a.v = v; a.q_exps = q_exps; a.k_exps = k_exps; a.v_exps = v_exps;
    a.log_g = log_g; a.beta = beta; a.h0 = h0; a.dout = dout; a.dh_final = dh_final;
    a.dq = dq; a.dk_out = dk_out; a.dv_out = dv_out; a.dlog_g = dlog_g; a.dbeta = dbeta; a.dh0 = dh0;
    a.B = B; a.T = T; a.Hk = Hk; a.Hv = Hv; a.dk = dk; a.dv = dv; a.cu = cu_seqlens;
    a.io_dtype = io_dtype; a.grad_dtype = grad_dtype;
    a.workspace = workspace; a.workspace_bytes = workspace_bytes;
    return a;
}

bool chunk_sizes_fine(int B, int T, int Hk, int Hv, int dk, int dv)
{
    return B >= 1 && T >= 0 && Hk >= 1 && Hv >= 1 && dk >= 1 && dv >= 1 && B <= 65535 && Hv <= 65535 &&
           Hv % Hk == 0 && dk <= 128 && dv <= 128;
}

int check_chunk(const gdn::BackwardArgs& a)
{
    const char* who = "gdn_chunk_backward";
    if (!wide_dtype(a.grad_dtype) || (!wide_dtype(a.io_dtype) && a.io_dtype != GDN_E4M3))
        return refuse_call(GDN_ERR_DTYPE, who, "io_dtype: GDN_F32, GDN_BF16 or GDN_E4M3; grad_dtype: GDN_F32 or GDN_BF16");
    if (a.B < 1 || a.T < 0 || a.Hk < 1 || a.Hv < 1 || a.dk < 1 || a.dv < 1)
        return refuse_call(GDN_ERR_SHAPE, who, "need B, Hk, Hv, dk, dv >= 1 and T >= 0");
    if (a.B > 65535 || a.Hv > 65535) return refuse_call(GDN_ERR_SHAPE, who, "B or Hv > 65535 (grid limits)");
    if (a.Hv % a.Hk != 0) return refuse_call(GDN_ERR_HEAD_GROUPS, who, "Hv must be a multiple of Hk");
    if (a.dk > 128 || a.dv > 128) return refuse_call(GDN_ERR_DIM_LIMIT, who, "dk, dv <= 128");
    if (a.T > 0) {
        if (!a.q || !a.k || !a.v || !a.log_g || !a.beta || !a.dout)
            return refuse_call(GDN_ERR_NULL, who, "q, k, v, log_g, beta and dout are required when T > 0");
        if (!a.dq || !a.dk_out || !a.dv_out || !a.dlog_g || !a.dbeta)
            return refuse_call(GDN_ERR_NULL, who, "dq, dk, dv, dlog_g and dbeta are required when T > 0");
        if (a.io_dtype == GDN_E4M3 && (!a.q_exps || !a.k_exps || !a.v_exps))
            return refuse_call(GDN_ERR_NULL, who, "8-bit activations need their exps");
    }
    const size_t need = gdn::backward_workspace_need(a);
    if (need > 0 && (!a.workspace || a.workspace_bytes < need))
        return refuse_call(GDN_ERR_WORKSPACE, who, "workspace smaller than gdn_backward_workspace_bytes()");
    if (reinterpret_cast<uintptr_t>(a.workspace) % 16 != 0)
        return refuse_call(GDN_ERR_WORKSPACE, who, "workspace must be 16-byte aligned");
    return GDN_OK;
}

const gdn::Geometry kNothing{"nothing to launch", {0, 0, 0}, 0, 0};

}  // namespace

extern "C" {

int gdn_ckpt8_store_plan(const void* x, uint8_t* codes, uint8_t* exps, int64_t rows, int d,
                         int64_t x_stride, int io_dtype)
{
    const gdn::CkptArgs a = store_args(x, codes, exps, rows, d, x_stride, io_dtype);
    const int st = check_ckpt(a, true);
    if (st != GDN_OK) return st;
    gdn::route_call(rows ? gdn::ckpt_store_geometry(a) : kNothing, "");
    return GDN_OK;
}

int gdn_ckpt8_store(const void* x, uint8_t* codes, uint8_t* exps, int64_t rows, int d, int64_t x_stride,
                    int io_dtype, hipStream_t stream)
{
    const int st = gdn_ckpt8_store_plan(x, codes, exps, rows, d, x_stride, io_dtype);
    if (st != GDN_OK) return st;
    return gdn::launch_status(
        gdn::launch_ckpt_store(store_args(x, codes, exps, rows, d, x_stride, io_dtype), stream));
}

int gdn_ckpt8_load_plan(const uint8_t* codes, const uint8_t* exps, void* y, int64_t rows, int d,
                        int64_t y_stride, int out_dtype)
{
    const gdn::CkptArgs a = load_args(codes, exps, y, rows, d, y_stride, out_dtype);
    const int st = check_ckpt(a, false);
    if (st != GDN_OK) return st;
    gdn::route_call(rows ? gdn::ckpt_load_geometry(a) : kNothing, "");
    return GDN_OK;
}

int gdn_ckpt8_load(const uint8_t* codes, const uint8_t* exps, void* y, int64_t rows, int d,
                   int64_t y_stride, int out_dtype, hipStream_t stream)
{
    const int st = gdn_ckpt8_load_plan(codes, exps, y, rows, d, y_stride, out_dtype);
    if (st != GDN_OK) return st;
    return gdn::launch_status(
        gdn::launch_ckpt_load(load_args(codes, exps, y, rows, d, y_stride, out_dtype), stream));
}

size_t gdn_norm_workspace_bytes(int T, int H, int d)
{
    if (T < 1 || H < 1 || d < 1 || d > 8192 || (int64_t)T * H >= (1LL << 31)) return 0;
    return gdn::norm_workspace_bytes(T, H, d);
}

int gdn_norm_forward_plan(const void* x, const void* z, const float* w, const float* b, void* y,
                          uint8_t* x_codes, uint8_t* x_exps, uint8_t* z_codes, uint8_t* z_exps, int T,
                          int H, int d, int64_t x_stride, int64_t z_stride, int64_t y_stride, float eps,
                          int center, int io_dtype)
{
    const gdn::NormArgs a = forward_args(x, z, w, b, y, x_codes, x_exps, z_codes, z_exps, T, H, d, x_stride,
                                         z_stride, y_stride, eps, center, io_dtype);
    const int st = check_norm(a, false);
    if (st != GDN_OK) return st;
    gdn::route_call(T ? gdn::norm_forward_geometry(a) : kNothing, "");
    return GDN_OK;
}

int gdn_norm_forward(const void* x, const void* z, const float* w, const float* b, void* y,
                     uint8_t* x_codes, uint8_t* x_exps, uint8_t* z_codes, uint8_t* z_exps, int T, int H,
                     int d, int64_t x_stride, int64_t z_stride, int64_t y_stride, float eps, int center,
                     int io_dtype, hipStream_t stream)
{
    const int st = gdn_norm_forward_plan(x, z, w, b, y, x_codes, x_exps, z_codes, z_exps, T, H, d, x_stride,
                                         z_stride, y_stride, eps, center, io_dtype);
    if (st != GDN_OK) return st;
    return gdn::launch_status(gdn::launch_norm_forward(
        forward_args(x, z, w, b, y, x_codes, x_exps, z_codes, z_exps, T, H, d, x_stride, z_stride, y_stride,
                     eps, center, io_dtype),
        stream));
}

int gdn_norm_backward_plan(const void* x, const uint8_t* x_exps, const void* z, const uint8_t* z_exps,
                           const float* w, const float* b, const void* dy, void* dx, void* dz, float* dw,
                           float* db, int T, int H, int d, int64_t x_stride, int64_t z_stride,
                           int64_t dy_stride, int64_t dx_stride, int64_t dz_stride, float eps, int center,
                           int act_dtype, int io_dtype, void* workspace, size_t workspace_bytes)
{
    const gdn::NormArgs a = backward_args(x, x_exps, z, z_exps, w, b, dy, dx, dz, dw, db, T, H, d, x_stride,
                                          z_stride, dy_stride, dx_stride, dz_stride, eps, center, act_dtype,
                                          io_dtype, workspace, workspace_bytes);
    const int st = check_norm(a, true);
    if (st != GDN_OK) return st;
    gdn::route_call(gdn::norm_backward_geometry(a), T ? "" : "(no rows: the weight kernel writes zeros)");
    return GDN_OK;
}

int gdn_norm_backward(const void* x, const uint8_t* x_exps, const void* z, const uint8_t* z_exps,
                      const float* w, const float* b, const void* dy, void* dx, void* dz, float* dw,
                      float* db, int T, int H, int d, int64_t x_stride, int64_t z_stride,
                      int64_t dy_stride, int64_t dx_stride, int64_t dz_stride, float eps, int center,
                      int act_dtype, int io_dtype, void* workspace, size_t workspace_bytes,
                      hipStream_t stream)
{
    const int st = gdn_norm_backward_plan(x, x_exps, z, z_exps, w, b, dy, dx, dz, dw, db, T, H, d, x_stride,
                                          z_stride, dy_stride, dx_stride, dz_stride, eps, center, act_dtype,
                                          io_dtype, workspace, workspace_bytes);
    if (st != GDN_OK) return st;
    return gdn::launch_status(gdn::launch_norm_backward(
        backward_args(x, x_exps, z, z_exps, w, b, dy, dx, dz, dw, db, T, H, d, x_stride, z_stride, dy_stride,
                      dx_stride, dz_stride, eps, center, act_dtype, io_dtype, workspace, workspace_bytes),
        stream));
}

size_t gdn_backward_workspace_bytes(int B, int T, int Hk, int Hv, int dk, int dv, int io_dtype,
                                    int grad_dtype, int packed)
{
    if (!chunk_sizes_fine(B, T, Hk, Hv, dk, dv)) return 0;
    const int32_t* cu = packed ? reinterpret_cast<const int32_t*>(static_cast<uintptr_t>(16)) : nullptr;
    return gdn::backward_workspace_need(chunk_args(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                                                   nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                                                   nullptr, nullptr, nullptr, B, T, Hk, Hv, dk, dv, cu, io_dtype,
                                                   grad_dtype, nullptr, 0));
}

int gdn_chunk_backward_plan(const void* q, const void* k, const void* v, const uint8_t* q_exps,
                            const uint8_t* k_exps, const uint8_t* v_exps, const float* log_g,
                            const float* beta, const float* h0, const void* dout, const float* dh_final,
                            void* dq, void* dk_out, void* dv_out, void* dlog_g, void* dbeta, float* dh0,
                            int B, int T, int Hk, int Hv, int dk, int dv, const int32_t* cu_seqlens,
                            int io_dtype, int grad_dtype, void* workspace, size_t workspace_bytes)
{
    const gdn::BackwardArgs a = chunk_args(q, k, v, q_exps, k_exps, v_exps, log_g, beta, h0, dout, dh_final, dq,
                                           dk_out, dv_out, dlog_g, dbeta, dh0, B, T, Hk, Hv, dk, dv, cu_seqlens,
                                           io_dtype, grad_dtype, workspace, workspace_bytes);
    const int st = check_chunk(a);
    if (st != GDN_OK) return st;
    const char* why = gdn::backward_mfma_refuses(a);
    gdn::route_call(why ? gdn::backward_generic_geometry(a) : gdn::backward_mfma_geometry(a), why ? why : "");
    return GDN_OK;
}

int gdn_chunk_backward(const void* q, const void* k, const void* v, const uint8_t* q_exps,
                       const uint8_t* k_exps, const uint8_t* v_exps, const float* log_g,
                       const float* beta, const float* h0, const void* dout, const float* dh_final,
                       void* dq, void* dk_out, void* dv_out, void* dlog_g, void* dbeta, float* dh0, int B,
                       int T, int Hk, int Hv, int dk, int dv, const int32_t* cu_seqlens, int io_dtype,
                       int grad_dtype, void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    const int st = gdn_chunk_backward_plan(q, k, v, q_exps, k_exps, v_exps, log_g, beta, h0, dout, dh_final, dq,
                                           dk_out, dv_out, dlog_g, dbeta, dh0, B, T, Hk, Hv, dk, dv, cu_seqlens,
                                           io_dtype, grad_dtype, workspace, workspace_bytes);
    if (st != GDN_OK) return st;
    const gdn::BackwardArgs a = chunk_args(q, k, v, q_exps, k_exps, v_exps, log_g, beta, h0, dout, dh_final, dq,
                                           dk_out, dv_out, dlog_g, dbeta, dh0, B, T, Hk, Hv, dk, dv, cu_seqlens,
                                           io_dtype, grad_dtype, workspace, workspace_bytes);
    return gdn::launch_status(gdn::backward_mfma_refuses(a) ? gdn::launch_backward_generic(a, stream)
                                                            : gdn::launch_backward_mfma(a, stream));
}

}  // extern "C"
