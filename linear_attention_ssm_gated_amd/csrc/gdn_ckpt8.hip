// Activation checkpoints in 8 bits: e4m3 codes with one power-of-two scale
// byte per 128 values of a row (include/gdn_train.h).
//
// The scale is the smallest power of two that brings the group's largest
// finite magnitude to 448 or less: a power of two costs a floating code no
// precision that another scale would keep (only the range at its subnormals,
// 2^-9 of 448 * 2^-e below), needs one byte, and leaves every decoded value
// exactly representable in bf16, so that a bf16 matrix product takes it
// without a second rounding.  The code is rounded to nearest even: relative
// error at most 2^-4.  (The last scale byte is not a power of two: ckpt_scale.)
//
// Both kernels are bound by HBM: store moves (element size + 1) bytes a value
// in one pass, the group's maximum formed in registers across the 8 lanes
// that hold it.  Measured, bf16 rows of 128: store 14.2 us for 4576 x 48 rows
// (84.8 MB, 5.9 TB/s), load 9.7 us for 2371 x 48 (43.8 MB, 4.5 TB/s; a 1 GiB copy
// reaches 5.15 TB/s on this card, and part of these sizes comes from the caches).
#include "gdn_train_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr unsigned kMaxGrid = 256 * 32;   // 32 workgroups a compute unit: the rest by grid stride

typedef uint32_t u4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ void load16(const float* p, float* f)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 v = *reinterpret_cast<const float4*>(p + 4 * i);
        f[4 * i] = v.x; f[4 * i + 1] = v.y; f[4 * i + 2] = v.z; f[4 * i + 3] = v.w;
    }
}
__device__ __forceinline__ void load16(const uint16_t* p, float* f)
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const u4 v = *reinterpret_cast<const u4*>(p + 8 * i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[8 * i + 2 * j] = __uint_as_float(v[j] << 16);
            f[8 * i + 2 * j + 1] = __uint_as_float(v[j] & 0xffff0000u);
        }
    }
}
__device__ __forceinline__ void store16(float* p, const float* f)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(p + 4 * i) = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
}
__device__ __forceinline__ void store16(uint16_t* p, const float* f)
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        u4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = (uint32_t)f32_to_bf16_bits(f[8 * i + 2 * j]) |
                   ((uint32_t)f32_to_bf16_bits(f[8 * i + 2 * j + 1]) << 16);
        *reinterpret_cast<u4*>(p + 8 * i) = v;
    }
}

// Row r of the wide side: rows of `heads` heads share a token stride.
__device__ __forceinline__ int64_t row_offset(int64_t row, int heads, int d, int64_t stride)
{
    if (heads == 1) return row * stride;
    const int64_t t = row / heads;
    return t * stride + (row - t * heads) * d;
}

// Aligned rows, d a multiple of 16: 16 values a lane, LPG lanes a group.
template <typename T, int LPG>
__global__ void __launch_bounds__(kThreads)
gdn_ckpt8_store_kernel(const T* __restrict__ x, uint8_t* __restrict__ codes, uint8_t* __restrict__ exps,
                       int64_t units, int ng, int heads, int d, int64_t stride)
{
    const int l = threadIdx.x % LPG;
    const int64_t step = (int64_t)gridDim.x * (kThreads / LPG);
    for (int64_t u = (int64_t)blockIdx.x * (kThreads / LPG) + threadIdx.x / LPG; u < units; u += step) {
        const int64_t row = ng == 1 ? u : u / ng;
        const int g = (int)(u - row * ng);
        const int j = g * kCkptGroup + 16 * l;
        const bool live = j < d;
        float f[16];
        float top = 0.f;
        if (live) {
            load16(x + row_offset(row, heads, d, stride) + j, f);
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, ckpt_magnitude(f[i]));
        }
#pragma unroll
        for (int o = LPG / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
        const int byte = ckpt_exp_byte(top);
        const float inv = ckpt_inverse(byte);
        if (live) {
            u4 c;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                c[i] = ckpt_pack4(ckpt_finite(f[4 * i]) * inv, ckpt_finite(f[4 * i + 1]) * inv,
                                  ckpt_finite(f[4 * i + 2]) * inv, ckpt_finite(f[4 * i + 3]) * inv);
            *reinterpret_cast<u4*>(codes + row * d + j) = c;
        }
        if (l == 0) exps[u] = (uint8_t)byte;
    }
}

// Any width, stride and alignment: a wave per group, values lane and lane + 64.
template <typename T>
__global__ void __launch_bounds__(kThreads)
gdn_ckpt8_store_any_kernel(const T* __restrict__ x, uint8_t* __restrict__ codes,
                           uint8_t* __restrict__ exps, int64_t units, int ng, int heads, int d,
                           int64_t stride)
{
    const int l = threadIdx.x & 63;
    const int64_t step = (int64_t)gridDim.x * 4;
    for (int64_t u = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); u < units; u += step) {
        const int64_t row = ng == 1 ? u : u / ng;
        const int j = (int)(u - row * ng) * kCkptGroup + l;
        const T* p = x + row_offset(row, heads, d, stride);
        const float a = j < d ? Elem<T>::load(p + j) : 0.f;
        const float b = j + 64 < d ? Elem<T>::load(p + j + 64) : 0.f;
        float top = fmaxf(ckpt_magnitude(a), ckpt_magnitude(b));
#pragma unroll
        for (int o = 32; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
        const int byte = ckpt_exp_byte(top);
        const float inv = ckpt_inverse(byte);
        const uint32_t c = ckpt_pack4(ckpt_finite(a) * inv, ckpt_finite(b) * inv, 0.f, 0.f);
        if (j < d) codes[row * d + j] = (uint8_t)c;
        if (j + 64 < d) codes[row * d + j + 64] = (uint8_t)(c >> 8);
        if (l == 0) exps[u] = (uint8_t)byte;
    }
}

// 16 codes a lane (d a multiple of 16, aligned rows).
template <typename T>
__global__ void __launch_bounds__(kThreads)
gdn_ckpt8_load_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ exps,
                      T* __restrict__ y, int64_t items, int per_row, int ng, int d, int64_t stride)
{
    const int64_t step = (int64_t)gridDim.x * kThreads;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < items; i += step) {
        const int64_t row = items < (1LL << 31) ? (int64_t)((uint32_t)i / (uint32_t)per_row) : i / per_row;
        const int j = (int)(i - row * per_row) * 16;
        const u4 c = *reinterpret_cast<const u4*>(codes + i * 16);
        const float s = ckpt_scale(exps[row * ng + (j >> 7)]);
        float f[16];
#pragma unroll
        for (int e = 0; e < 4; ++e) ckpt_unpack4(c[e], f + 4 * e);
#pragma unroll
        for (int e = 0; e < 16; ++e) f[e] *= s;
        store16(y + row * stride + j, f);
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
gdn_ckpt8_load_any_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ exps,
                          T* __restrict__ y, int64_t n, int ng, int d, int64_t stride)
{
    const int64_t step = (int64_t)gridDim.x * kThreads;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += step) {
        const int64_t row = n < (1LL << 31) ? (int64_t)((uint32_t)i / (uint32_t)d) : i / d;
        const int j = (int)(i - row * d);
        Elem<T>::store(y + row * stride + j,
                       ckpt_unpack1(codes[i]) * ckpt_scale(exps[row * ng + (j >> 7)]));
    }
}

int groups(int d) { return (d + kCkptGroup - 1) / kCkptGroup; }
size_t elem(int dtype) { return dtype == 0 ? 4 : 2; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The 16-wide kernels take rows of a multiple of 16 values that start on 16
// bytes (4576 x 48 rows of 128 in bf16: store 14.6 us against 38.1 us value by
// value, load 15.8 us against 43.5 us).
bool wide(const CkptArgs& a, const void* side, const void* codes)
{
    return a.d % 16 == 0 && (a.stride * (int64_t)elem(a.dtype)) % 16 == 0 && aligned16(side) && aligned16(codes);
}
// lanes a group takes: a power of two of at least min(d, 128) / 16
int lanes(int d)
{
    const int need = ((d < kCkptGroup ? d : kCkptGroup) + 15) / 16;
    return need <= 1 ? 1 : need <= 2 ? 2 : need <= 4 ? 4 : 8;
}
unsigned grid_of(int64_t blocks) { return (unsigned)(blocks < (int64_t)kMaxGrid ? blocks : (int64_t)kMaxGrid); }

template <typename T>
void store_typed(const CkptArgs& a, int heads, hipStream_t s)
{
    const int ng = groups(a.d);
    const int64_t units = a.rows * ng;
    const T* x = static_cast<const T*>(a.x);
    if (!wide(a, a.x, a.codes)) {
        hipLaunchKernelGGL((gdn_ckpt8_store_any_kernel<T>), dim3(grid_of((units + 3) / 4)), dim3(kThreads), 0, s,
                           x, a.codes, a.exps_out, units, ng, heads, a.d, a.stride);
        return;
    }
    const int lpg = lanes(a.d);
    const dim3 grid(grid_of((units * lpg + kThreads - 1) / kThreads));
#define GDN_STORE(N)                                                                                   \
    hipLaunchKernelGGL((gdn_ckpt8_store_kernel<T, N>), grid, dim3(kThreads), 0, s, x, a.codes, a.exps_out, \
                       units, ng, heads, a.d, a.stride)
    if (lpg == 1) GDN_STORE(1);
    else if (lpg == 2) GDN_STORE(2);
    else if (lpg == 4) GDN_STORE(4);
    else GDN_STORE(8);
#undef GDN_STORE
}

template <typename T>
void load_typed(const CkptArgs& a, hipStream_t s)
{
    const int ng = groups(a.d);
    const uint8_t* codes = static_cast<const uint8_t*>(a.x);
    T* y = static_cast<T*>(a.y);
    if (!wide(a, a.y, codes)) {
        const int64_t n = a.rows * a.d;
        hipLaunchKernelGGL((gdn_ckpt8_load_any_kernel<T>), dim3(grid_of((n + kThreads - 1) / kThreads)),
                           dim3(kThreads), 0, s, codes, a.exps_in, y, n, ng, a.d, a.stride);
        return;
    }
    const int per_row = a.d / 16;
    const int64_t items = a.rows * per_row;
    hipLaunchKernelGGL((gdn_ckpt8_load_kernel<T>), dim3(grid_of((items + kThreads - 1) / kThreads)),
                       dim3(kThreads), 0, s, codes, a.exps_in, y, items, per_row, ng, a.d, a.stride);
}

Geometry geometry(const char* entry, unsigned grid)
{
    return Geometry{entry, {grid, 1, 1}, kThreads, 0};
}

}  // namespace

Geometry ckpt_store_geometry(const CkptArgs& a)
{
    const int64_t units = a.rows * groups(a.d);
    if (!wide(a, a.x, a.codes)) return geometry("gdn_ckpt8_store_any_kernel", grid_of((units + 3) / 4));
    return geometry("gdn_ckpt8_store_kernel", grid_of((units * lanes(a.d) + kThreads - 1) / kThreads));
}

Geometry ckpt_load_geometry(const CkptArgs& a)
{
    if (!wide(a, a.y, a.x))
        return geometry("gdn_ckpt8_load_any_kernel", grid_of((a.rows * a.d + kThreads - 1) / kThreads));
    return geometry("gdn_ckpt8_load_kernel", grid_of((a.rows * (a.d / 16) + kThreads - 1) / kThreads));
}

hipError_t launch_ckpt_store_heads(const CkptArgs& a, int heads, hipStream_t s)
{
    if (a.rows == 0) return hipSuccess;
    if (a.dtype == 0) store_typed<float>(a, heads, s);
    else store_typed<uint16_t>(a, heads, s);
    return hipGetLastError();
}

hipError_t launch_ckpt_store(const CkptArgs& a, hipStream_t s) { return launch_ckpt_store_heads(a, 1, s); }

hipError_t launch_ckpt_load(const CkptArgs& a, hipStream_t s)
{
    if (a.rows == 0) return hipSuccess;
    if (a.dtype == 0) load_typed<float>(a, s);
    else load_typed<uint16_t>(a, s);
    return hipGetLastError();
}

}  // namespace gdn
