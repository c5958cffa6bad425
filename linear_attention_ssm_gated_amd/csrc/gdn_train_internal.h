// Declarations shared by the training sources of libgdn.so (not part of the C
// ABI; include/gdn_train.h is).
#pragma once

#include "gdn_internal.h"

namespace gdn {

constexpr int kCkptGroup = 128;   // values per scale byte

struct CkptArgs {
    const void* x;         // store: input; load: codes
    uint8_t* codes;        // store: output
    const uint8_t* exps_in;
    uint8_t* exps_out;
    void* y;               // load: output
    int64_t rows;
    int d;
    int64_t stride;        // of the wide side, in elements
    int dtype;             // of the wide side
};

struct NormArgs {
    const void* x;
    const void* z;         // NULL: no gate
    const float* w;
    const float* b;        // NULL: no bias
    void* y;               // forward
    uint8_t *x_codes, *x_exps_out, *z_codes, *z_exps_out;   // forward's checkpoints or NULL
    const uint8_t *x_exps, *z_exps;                         // backward from codes
    const void* dy;
    void *dx, *dz;
    float *dw, *db;
    int T, H, d;
    int64_t x_stride, z_stride, y_stride;                   // y_stride: dy's in the backward
    int64_t dx_stride, dz_stride;
    float eps;
    int center, act_dtype, io_dtype;
    void* workspace;
    size_t workspace_bytes;
};

struct BackwardArgs {
    const void *q, *k, *v;
    const uint8_t *q_exps, *k_exps, *v_exps;
    const float *log_g, *beta, *h0;
    const void* dout;
    const float* dh_final;
    void *dq, *dk_out, *dv_out, *dlog_g, *dbeta;
    float* dh0;
    int B, T, Hk, Hv, dk, dv;
    const int32_t* cu;
    int io_dtype, grad_dtype;
    void* workspace;
    size_t workspace_bytes;
};

Geometry ckpt_store_geometry(const CkptArgs& a);
Geometry ckpt_load_geometry(const CkptArgs& a);
hipError_t launch_ckpt_store(const CkptArgs& a, hipStream_t s);
// rows = tokens * heads, a.stride the token stride (the wide side)
hipError_t launch_ckpt_store_heads(const CkptArgs& a, int heads, hipStream_t s);
hipError_t launch_ckpt_load(const CkptArgs& a, hipStream_t s);

size_t norm_workspace_bytes(int T, int H, int d);
Geometry norm_forward_geometry(const NormArgs& a);
Geometry norm_backward_geometry(const NormArgs& a);
hipError_t launch_norm_forward(const NormArgs& a, hipStream_t s);
hipError_t launch_norm_backward(const NormArgs& a, hipStream_t s);

// Bytes either route needs for these sizes and types (pointers are only
// compared with NULL).
size_t backward_workspace_need(const BackwardArgs& a);
// The guard that keeps a call off the MFMA route, NULL where it takes it.
const char* backward_mfma_refuses(const BackwardArgs& a);
Geometry backward_mfma_geometry(const BackwardArgs& a);
hipError_t launch_backward_mfma(const BackwardArgs& a, hipStream_t s);
Geometry backward_generic_geometry(const BackwardArgs& a);
hipError_t launch_backward_generic(const BackwardArgs& a, hipStream_t s);

// Lets a kernel take `bytes` of dynamic LDS on the current device (beyond the
// runtime's default limit); the runtime is asked once per kernel and device.
hipError_t allow_lds(const void* kernel, size_t bytes);

// Route-line helpers of the C ABI layer (gdn_api.hip): a named refusal, the line
// of an accepted call, and the status of its launches.
int refuse_call(int status, const char* who, const char* why);
void route_call(const Geometry& g, const char* note);
int launch_status(hipError_t e);

// ---- 8-bit checkpoints ----------------------------------------------------
// Scale byte of a group whose largest finite magnitude is top (>= 0, finite):
// the smallest power of two 2^e with top <= 448 * 2^e, i.e. with top = m 2^x,
// 1 <= m < 2: e = x - 8 where m <= 1.75, else x - 7; at least 2^-126 (its
// reciprocal is finite, and a smaller group keeps fewer bits), 1 for zero.
__device__ __forceinline__ int ckpt_exp_byte(float top)
{
    const uint32_t u = __float_as_uint(top);
    int byte = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    byte = byte < 1 ? 1 : byte;
    return u == 0 ? 127 : byte;
}
// 2^(byte - 127) for bytes 1..246, and its reciprocal.  The last byte, 247, stands for
// 255 2^112 instead of 2^120: the largest float is 256.99 of it and rounds to code 256,
// which is 255 2^120, bf16's largest finite value, where 256 2^120 would be infinity.
// (A select; bringing back the one code behind the product took 4 to 8 us of the
// 274 of a packed backward call from codes.)
constexpr int kCkptTopByte = 247;
__device__ __forceinline__ float ckpt_scale(int byte)
{
    return byte == kCkptTopByte ? 0x1.fep119f : __uint_as_float((uint32_t)byte << 23);
}
__device__ __forceinline__ float ckpt_inverse(int byte)
{
    return byte == kCkptTopByte ? 0x1.010102p-120f : __uint_as_float((uint32_t)(254 - byte) << 23);
}

// |x| where finite, 0 for infinities and NaN
__device__ __forceinline__ float ckpt_magnitude(float x)
{
    const float a = fabsf(x);
    return a < __builtin_inff() ? a : 0.0f;
}
// infinities leave as NaN
__device__ __forceinline__ float ckpt_finite(float x) { return fabsf(x) < __builtin_inff() ? x : __builtin_nanf(""); }

// four scaled values as e4m3 codes (round to nearest even), the first lowest
__device__ __forceinline__ uint32_t ckpt_pack4(float a, float b, float c, float d)
{
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
}
typedef float f32x2v __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void ckpt_unpack4(uint32_t codes, float* f)
{
    const f32x2v lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, false);
    const f32x2v hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, true);
    f[0] = lo.x; f[1] = lo.y; f[2] = hi.x; f[3] = hi.y;
}
__device__ __forceinline__ float ckpt_unpack1(uint8_t code)
{
    return __builtin_amdgcn_cvt_f32_fp8((int)code, 0);
}

}  // namespace gdn
