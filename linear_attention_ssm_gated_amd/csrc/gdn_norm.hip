// Layer norm / RMS norm of the recurrence's outputs times silu of a gate,
// forward and backward, with the reduction of the weight's and the bias's
// gradients (include/gdn_train.h).
//
// One row of d values is held in the registers of TPR threads (TPR <= 64: part
// of a wave, reduced by lane exchanges; TPR >= 256: a workgroup, reduced
// through LDS), so each input is read once and each output written once.  The
// statistics take two steps over the registers (mean, then the squares of the
// differences), which loses nothing where the mean is large.  Both passes are
// bound by HBM: 4576 x 48 rows of 128 in bf16 with a gate take 50 us forward with
// both checkpoints written (225 MB, 4.5 TB/s) and 61 us backward (281 MB, 4.6
// TB/s; 56 of them in the pass over the rows), where a 1 GiB copy reaches 5.15.
// At a decode step's 16 x 48 rows the 3.5 us of the launch itself are the time.
//
// Backward: a workgroup walks rows by grid stride and keeps its columns' sums
// of g n and g in registers; at the end its row groups are added through LDS
// into one partial row of the workspace, and a second kernel adds the partial
// rows in a fixed order: no atomics, the same bits run to run.
#include "gdn_train_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxWaves = 16;
// threads of a workgroup whose rows take tpr threads each
__host__ __device__ constexpr int wg_threads(int tpr) { return tpr > kThreads ? tpr : kThreads; }

typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

// ---- VEC consecutive values ------------------------------------------------
template <int VEC> __device__ __forceinline__ void load_vec(const float* p, float* f)
{
    if constexpr (VEC == 8) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 v = *reinterpret_cast<const float4*>(p + 4 * i);
            f[4 * i] = v.x; f[4 * i + 1] = v.y; f[4 * i + 2] = v.z; f[4 * i + 3] = v.w;
        }
    } else {
        f[0] = *p;
    }
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2v{lo, hi}, b2));
}
template <int VEC> __device__ __forceinline__ void store_vec(float* p, const float* f)
{
    if constexpr (VEC == 8) {
        *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        *p = f[0];
    }
}
template <int VEC> __device__ __forceinline__ void store_vec(uint16_t* p, const float* f)
{
    if constexpr (VEC == 8)
        *reinterpret_cast<u4*>(p) = u4{bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]),
                                       bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7])};
    else
        *p = f32_to_bf16_bits(f[0]);
}

// The same values as they lie in memory, fetched ahead of their use.
template <int VEC, typename T> struct RawVec {
    static constexpr int W = VEC * sizeof(T) >= 4 ? VEC * sizeof(T) / 4 : 1;
    uint32_t w[W];
    __device__ __forceinline__ void load(const T* p)
    {
        if constexpr (VEC == 1) {
            if constexpr (sizeof(T) == 4) w[0] = __float_as_uint(*reinterpret_cast<const float*>(p));
            else w[0] = (uint32_t)*p;
        } else if constexpr (W >= 4) {
#pragma unroll
            for (int i = 0; i < W / 4; ++i) {
                const u4 v = *reinterpret_cast<const u4*>(reinterpret_cast<const uint32_t*>(p) + 4 * i);
#pragma unroll
                for (int j = 0; j < 4; ++j) w[4 * i + j] = v[j];
            }
        } else {
            const u2 v = *reinterpret_cast<const u2*>(p);
            w[0] = v[0];
            w[1] = v[1];
        }
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void widen(float* f) const
    {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) f[i] = __uint_as_float(w[i]);
        } else if constexpr (sizeof(T) == 2) {
            if constexpr (VEC == 1) f[0] = __uint_as_float(w[0] << 16);
            else
#pragma unroll
                for (int i = 0; i < VEC / 2; ++i) {
                    f[2 * i] = __uint_as_float(w[i] << 16);
                    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
                }
        } else {
            if constexpr (VEC == 1) f[0] = ckpt_unpack1((uint8_t)w[0]);
            else {
                ckpt_unpack4(w[0], f);
                ckpt_unpack4(w[1], f + 4);
            }
        }
    }
};

// ---- sums over the TPR threads of a row --------------------------------------
// slot: a different one for each reduction of a row (LDS, TPR > 64 only); two
// reductions a row keep a slot's readers ahead of its next writers.
template <int TPR> __device__ __forceinline__ float row_sum(float x, float* red, int slot)
{
    constexpr int W = TPR < 64 ? TPR : 64;
#pragma unroll
    for (int o = W / 2; o; o >>= 1) x += __shfl_xor(x, o);
    if constexpr (TPR > 64) {
        float* r = red + slot * kMaxWaves;
        if ((threadIdx.x & 63) == 0) r[threadIdx.x >> 6] = x;
        __syncthreads();
        x = 0.f;
#pragma unroll
        for (int i = 0; i < TPR / 64; ++i) x += r[i];
    }
    return x;
}

// two sums at once, in slots slot and slot + 1
template <int TPR> __device__ __forceinline__ void row_sum2(float& x, float& y, float* red, int slot)
{
    constexpr int W = TPR < 64 ? TPR : 64;
#pragma unroll
    for (int o = W / 2; o; o >>= 1) {
        x += __shfl_xor(x, o);
        y += __shfl_xor(y, o);
    }
    if constexpr (TPR > 64) {
        float *r = red + slot * kMaxWaves, *t = r + kMaxWaves;
        if ((threadIdx.x & 63) == 0) {
            r[threadIdx.x >> 6] = x;
            t[threadIdx.x >> 6] = y;
        }
        __syncthreads();
        x = y = 0.f;
#pragma unroll
        for (int i = 0; i < TPR / 64; ++i) {
            x += r[i];
            y += t[i];
        }
    }
}

// The hardware's exp2 and reciprocal, within one unit in the last place each: a
// relative error of a few 2^-24, far below the output's rounding to bf16 and
// without the instructions of a correctly rounded division.  (fp32 gradients are off
// by 1.1e-7 in the 2-norm, 5.8e-8 for a form in fp32 that rounds each step once.)
__device__ __forceinline__ float sigmoid(float z)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
}

struct Shape {
    int64_t rows;
    int H, d, ng;
    float inv_d, eps;
    int center;
};

// Where a row group is: token and head, moved on by a fixed number of rows
// without a division.
struct Place {
    int64_t row;
    int t, h;
    __device__ __forceinline__ Place(int64_t r, const Shape& s) : row(r), t((int)r), h(0)
    {
        if (s.H > 1) {
            t = (int)((uint32_t)r / (uint32_t)s.H);
            h = (int)((uint32_t)r - (uint32_t)t * (uint32_t)s.H);
        }
    }
    __device__ __forceinline__ void move(int rows, int dt, int dh, const Shape& s)
    {
        row += rows;
        t += dt;
        h += dh;
        if (h >= s.H) {
            h -= s.H;
            ++t;
        }
    }
    // (the heads of one token alone may hold more than 2^31 values)
    __device__ __forceinline__ int64_t at(int64_t stride, const Shape& s) const
    {
        return (int64_t)t * stride + (int64_t)h * s.d;
    }
};

// The row's values minus their mean (center), and 1 / sqrt(var + eps).  The
// mean of a row far from zero is known to 2^-24 of itself only; what is left of
// it in the differences, which lose nothing, is taken out with the sum that the
// variance's pass forms beside the squares.
template <int TPR, int NV, int VEC>
__device__ __forceinline__ float normalise(float* x, const Shape& s, int l, float* red)
{
    auto minus = [&](float m) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if ((i * TPR + l) * VEC < s.d)
#pragma unroll
                for (int e = 0; e < VEC; ++e) x[i * VEC + e] -= m;
    };
    if (s.center) {
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < NV * VEC; ++e) m += x[e];
        minus(row_sum<TPR>(m, red, 0) * s.inv_d);
    }
    float q = 0.f, c = 0.f;
#pragma unroll
    for (int e = 0; e < NV * VEC; ++e) q = fmaf(x[e], x[e], q);
    if (s.center) {
#pragma unroll
        for (int e = 0; e < NV * VEC; ++e) c += x[e];
        row_sum2<TPR>(q, c, red, 1);
        c *= s.inv_d;
        minus(c);
        q = fmaf(-c, c, q * s.inv_d);
    } else {
        q = row_sum<TPR>(q, red, 1) * s.inv_d;
    }
    // (a centred row's may round below zero; fmaxf would make a NaN row's zero too)
    return __builtin_amdgcn_rsqf((q < 0.f ? 0.f : q) + s.eps);
}

// Codes and scale byte of the VEC = 8 values of each lane, a group's 128 lying
// in 16 consecutive lanes (or in all of a narrower row's).
template <int TPR, int NV>
__device__ __forceinline__ void write_codes(const float* x, uint8_t* codes, uint8_t* exps, int64_t row,
                                            const Shape& s, int l)
{
    constexpr int W = TPR < 16 ? TPR : 16;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = (i * TPR + l) * 8;
        const float* f = x + 8 * i;
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, ckpt_magnitude(f[e]));
#pragma unroll
        for (int o = W / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
        const int byte = ckpt_exp_byte(top);
        const float inv = ckpt_inverse(byte);
        if (j < s.d) {
            *reinterpret_cast<u2*>(codes + row * s.d + j) =
                u2{ckpt_pack4(ckpt_finite(f[0]) * inv, ckpt_finite(f[1]) * inv, ckpt_finite(f[2]) * inv,
                              ckpt_finite(f[3]) * inv),
                   ckpt_pack4(ckpt_finite(f[4]) * inv, ckpt_finite(f[5]) * inv, ckpt_finite(f[6]) * inv,
                              ckpt_finite(f[7]) * inv)};
            if ((j & (kCkptGroup - 1)) == 0) exps[row * s.ng + (j >> 7)] = (uint8_t)byte;
        }
    }
}

// ---- forward -----------------------------------------------------------------
template <typename T, int TPR, int NV, int VEC, bool GATE>
__global__ void __launch_bounds__(wg_threads(TPR))
gdn_norm_forward_kernel(const T* __restrict__ x, const T* __restrict__ z, const float* __restrict__ w,
                        const float* __restrict__ b, T* __restrict__ y, uint8_t* __restrict__ x_codes,
                        uint8_t* __restrict__ x_exps, uint8_t* __restrict__ z_codes,
                        uint8_t* __restrict__ z_exps, Shape s, int64_t x_stride, int64_t z_stride,
                        int64_t y_stride)
{
    __shared__ float red[TPR > 64 ? 6 * kMaxWaves : 1];
    constexpr int RPW = wg_threads(TPR) / TPR;
    const int l = threadIdx.x % TPR;
    const int step = (int)gridDim.x * RPW, dt = step / s.H, dh = step - dt * s.H;
    Place p((int64_t)blockIdx.x * RPW + threadIdx.x / TPR, s);
    int turn = 0;
    for (int64_t base = (int64_t)blockIdx.x * RPW; base < s.rows; base += step, p.move(step, dt, dh, s)) {
        const bool live = p.row < s.rows;   // a dead row group still takes part in the lane exchanges
        float xv[NV * VEC], zv[GATE ? NV * VEC : 1];
        RawVec<VEC, T> rx[NV], rz[GATE ? NV : 1];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = (i * TPR + l) * VEC;
            rx[i].zero();
            if constexpr (GATE) rz[i].zero();
            if (live && j < s.d) {
                rx[i].load(x + p.at(x_stride, s) + j);
                if constexpr (GATE) rz[i].load(z + p.at(z_stride, s) + j);
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            rx[i].widen(xv + i * VEC);
            if constexpr (GATE) rz[i].widen(zv + i * VEC);
        }
        if constexpr (VEC == 8) {
            if (live && x_codes) write_codes<TPR, NV>(xv, x_codes, x_exps, p.row, s, l);
            if constexpr (GATE)
                if (live && z_codes) write_codes<TPR, NV>(zv, z_codes, z_exps, p.row, s, l);
        }
        // LDS slots by turns: an RMS norm's one reduction a row would let the
        // next row's writers overtake this row's readers
        const float r = normalise<TPR, NV, VEC>(xv, s, l, red + 3 * kMaxWaves * turn);
        turn = TPR > 64 ? turn ^ 1 : 0;
        if (!live) continue;
        T* py = y + p.at(y_stride, s);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = (i * TPR + l) * VEC;
            if (j >= s.d) continue;
            float wv[VEC], bv[VEC], o[VEC];
            load_vec<VEC>(w + j, wv);
            if (b) load_vec<VEC>(b + j, bv);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                float a = xv[i * VEC + e] * r * wv[e];
                if (b) a += bv[e];
                if constexpr (GATE) {
                    const float zz = zv[i * VEC + e];
                    a *= zz * sigmoid(zz);
                }
                o[e] = a;
            }
            store_vec<VEC>(py + j, o);
        }
    }
}

// ---- backward ----------------------------------------------------------------
// The next row's values are fetched while the present one's are worked on.
template <typename A, typename T, int TPR, int NV, int VEC, bool GATE>
__global__ void __launch_bounds__(wg_threads(TPR), TPR <= 64 && NV == 1 ? 4 : 1)
gdn_norm_backward_kernel(const A* __restrict__ x, const uint8_t* __restrict__ x_exps,
                         const A* __restrict__ z, const uint8_t* __restrict__ z_exps,
                         const float* __restrict__ w, const float* __restrict__ b,
                         const T* __restrict__ dy, T* __restrict__ dx, T* __restrict__ dz,
                         float* __restrict__ part, Shape s, int64_t x_stride, int64_t z_stride,
                         int64_t dy_stride, int64_t dx_stride, int64_t dz_stride)
{
    constexpr int RPW = wg_threads(TPR) / TPR;     // rows a workgroup takes at a time
    constexpr int N = NV * VEC, NG = GATE ? N : 1, NR = GATE ? NV : 1;
    constexpr bool codes = sizeof(A) == 1;
    __shared__ float red[TPR > 64 ? 6 * kMaxWaves : 1];
    __shared__ float sums[RPW > 1 ? kThreads * N : 1];
    const int l = threadIdx.x % TPR, rg = threadIdx.x / TPR;
    const int step = (int)gridDim.x * RPW, dt = step / s.H, dh = step - dt * s.H;

    float wv[N], bv[NG], dw[N], db[N];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = (i * TPR + l) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            wv[i * VEC + e] = dw[i * VEC + e] = db[i * VEC + e] = 0.f;
            if constexpr (GATE) bv[i * VEC + e] = 0.f;
        }
        if (j < s.d) {
            load_vec<VEC>(w + j, wv + i * VEC);
            if constexpr (GATE)
                if (b) load_vec<VEC>(b + j, bv + i * VEC);
        }
    }

    struct Row {
        RawVec<VEC, A> x[NV], z[NR];
        RawVec<VEC, T> g[NV];
        uint8_t ex[NV], ez[NR];
    } next;
    Place p((int64_t)blockIdx.x * RPW + rg, s);
    auto fetch = [&]() {
        const bool live = p.row < s.rows;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = (i * TPR + l) * VEC;
            next.x[i].zero();
            if constexpr (GATE) next.z[i].zero();
            next.g[i].zero();
            next.ex[i] = 127;
            if constexpr (GATE) next.ez[i] = 127;
            if (live && j < s.d) {
                next.x[i].load(x + p.at(x_stride, s) + j);
                if constexpr (GATE) next.z[i].load(z + p.at(z_stride, s) + j);
                next.g[i].load(dy + p.at(dy_stride, s) + j);
                if constexpr (codes) {
                    next.ex[i] = x_exps[p.row * s.ng + (j >> 7)];
                    if constexpr (GATE) next.ez[i] = z_exps[p.row * s.ng + (j >> 7)];
                }
            }
        }
    };
    fetch();
    for (int64_t base = (int64_t)blockIdx.x * RPW; base < s.rows; base += step) {
        const Place at = p;
        const bool live = at.row < s.rows;
        float xv[N], zv[NG], gv[N];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            next.x[i].widen(xv + i * VEC);
            if constexpr (GATE) next.z[i].widen(zv + i * VEC);
            next.g[i].widen(gv + i * VEC);
            if constexpr (codes) {
                const float sx = ckpt_scale(next.ex[i]);
#pragma unroll
                for (int e = 0; e < VEC; ++e) xv[i * VEC + e] *= sx;
                if constexpr (GATE) {
                    const float sz = ckpt_scale(next.ez[i]);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) zv[i * VEC + e] *= sz;
                }
            }
        }
        p.move(step, dt, dh, s);
        fetch();
        float r = normalise<TPR, NV, VEC>(xv, s, l, red);
        if (!live) r = 0.f;    // a dead row adds nothing to the sums, whatever eps is
        float dot = 0.f, sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = (i * TPR + l) * VEC;
            float o[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int c = i * VEC + e;
                const float n = xv[c] * r;
                xv[c] = n;
                if constexpr (GATE) {
                    // silu' = s + z s (1 - s); where s rounds to 1 the second term is
                    // zero at once (z s - z s s, with s added to z s, loses the s
                    // beside a large z)
                    const float sg = sigmoid(zv[c]), d = gv[c], si = zv[c] * sg;
                    gv[c] = d * si;
                    o[e] = d * fmaf(n, wv[c], bv[c]) * fmaf(si, 1.0f - sg, sg);
                }
                dw[c] = fmaf(gv[c], n, dw[c]);
            }
            if constexpr (GATE)
                if (live && j < s.d) store_vec<VEC>(dz + at.at(dz_stride, s) + j, o);
        }
        if (b) {
#pragma unroll
            for (int c = 0; c < N; ++c) db[c] += gv[c];
        }
#pragma unroll
        for (int c = 0; c < N; ++c) {
            gv[c] *= wv[c];            // dn
            dot = fmaf(gv[c], xv[c], dot);
        }
        if (s.center) {
#pragma unroll
            for (int c = 0; c < N; ++c) sum += gv[c];
            row_sum2<TPR>(dot, sum, red, 3);
            sum *= s.inv_d;
        } else {
            dot = row_sum<TPR>(dot, red, 3);
        }
        dot *= s.inv_d;
        if (live) {
            T* pdx = dx + at.at(dx_stride, s);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int j = (i * TPR + l) * VEC;
                if (j >= s.d) continue;
                float o[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const int c = i * VEC + e;
                    o[e] = (gv[c] - fmaf(xv[c], dot, sum)) * r;
                }
                store_vec<VEC>(pdx + j, o);
            }
        }
    }

    // this workgroup's partial row of dw, then of db
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        if (half && !b) break;
        float* a = half ? db : dw;
        if constexpr (RPW > 1) {
            __syncthreads();
#pragma unroll
            for (int c = 0; c < N; ++c) sums[c * kThreads + threadIdx.x] = a[c];
            __syncthreads();
            if (rg == 0) {
#pragma unroll
                for (int c = 0; c < N; ++c) {
                    float t = 0.f;
                    for (int k = 0; k < RPW; ++k) t += sums[c * kThreads + k * TPR + l];
                    a[c] = t;
                }
            }
        }
        if (rg == 0) {
            float* q = part + ((int64_t)half * gridDim.x + blockIdx.x) * s.d;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int j = (i * TPR + l) * VEC;
                if (j < s.d) store_vec<VEC>(q + j, a + i * VEC);
            }
        }
    }
}

// Sums of the partial rows, in a fixed order: COLS columns a workgroup, 256 /
// COLS threads a column, eight partial rows in flight each.  parts == 0 writes
// zeros.  Eight columns spread a narrow row over more workgroups (d = 128: 5.3 us,
// 7.8 with 32; d = 1024: 3.9 and 6.4), 32 read whole 128-byte lines of a wide one
// (d = 5120: 8.0 us, 10.6 with eight; d = 2048 takes 6 with either).
template <int COLS>
__global__ void __launch_bounds__(kThreads)
gdn_norm_weight_kernel(const float* __restrict__ part, int parts, int d, float* __restrict__ dw,
                       float* __restrict__ db)
{
    constexpr int K = kThreads / COLS;
    __shared__ float sums[K][COLS + 1];
    const int c = threadIdx.x % COLS, k = threadIdx.x / COLS;
    const int j = blockIdx.x * COLS + c, half = blockIdx.y;
    float a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (j < d) {
        const float* p = part + (int64_t)half * parts * d + j;
        int i = k;
        for (; i + 7 * K < parts; i += 8 * K)
#pragma unroll
            for (int u = 0; u < 8; ++u) a[u] += p[(int64_t)(i + K * u) * d];
        for (; i < parts; i += K) a[0] += p[(int64_t)i * d];
    }
    sums[k][c] = ((a[0] + a[1]) + (a[2] + a[3])) + ((a[4] + a[5]) + (a[6] + a[7]));
    __syncthreads();
    if (k == 0 && j < d) {
        float t = 0.f;
        for (int i = 0; i < K; ++i) t += sums[i][c];
        (half ? db : dw)[j] = t;
    }
}

// ---- choice --------------------------------------------------------------------
// Threads a row takes and vectors a thread: eight values a thread while d fits
// a wave (16 lanes hold d = 128), two up to 1024, a workgroup beyond (d = 2048
// backward: 23.1 us, 29.8 with four in a wave).  Value by value where a row is not
// a multiple of eight or not aligned (4576 x 48 rows of 128 in bf16: 33 us forward
// and 57 backward by eights, 71 and 121 by single values; 2371 rows of 5120 in
// fp32: 26 and 57, 34 and 66).
struct Choice { int tpr, nv, vec; };
Choice choose(int d, bool vec8)
{
    if (vec8) {
        if (d <= 32) return {4, 1, 8};
        if (d <= 64) return {8, 1, 8};
        if (d <= 128) return {16, 1, 8};
        if (d <= 256) return {32, 1, 8};
        if (d <= 512) return {64, 1, 8};
        if (d <= 1024) return {64, 2, 8};
        if (d <= 2048) return {256, 1, 8};
        if (d <= 4096) return {256, 2, 8};
        if (d <= 6144) return {256, 3, 8};
        return {256, 4, 8};
    }
    if (d <= 64) return {64, 1, 1};
    if (d <= 128) return {64, 2, 1};
    if (d <= 256) return {64, 4, 1};
    if (d <= 1024) return {256, 4, 1};
    if (d <= 2048) return {256, 8, 1};
    if (d <= 4096) return {1024, 4, 1};
    return {1024, 8, 1};
}

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool stride8(int64_t s) { return s % 8 == 0; }
bool forward_vec8(const NormArgs& a)
{
    return a.d % 8 == 0 && aligned(a.x, 16) && aligned(a.z, 16) && aligned(a.y, 16) && aligned(a.w, 16) &&
           aligned(a.b, 16) && aligned(a.x_codes, 8) && aligned(a.z_codes, 8) && stride8(a.x_stride) &&
           (!a.z || stride8(a.z_stride)) && stride8(a.y_stride);
}
bool backward_vec8(const NormArgs& a)
{
    return a.d % 8 == 0 && aligned(a.x, 16) && aligned(a.z, 16) && aligned(a.dy, 16) && aligned(a.dx, 16) &&
           aligned(a.dz, 16) && aligned(a.w, 16) && aligned(a.b, 16) && stride8(a.x_stride) &&
           (!a.z || (stride8(a.z_stride) && stride8(a.dz_stride))) && stride8(a.y_stride) &&
           stride8(a.dx_stride);
}

// Workgroups of the backward pass, and so partial rows: enough to fill 256
// compute units several times over, few enough that the partial rows stay
// small next to the data (both kernels, 1024 against 512 workgroups: 4576 x 48
// rows of 128 in bf16 54 and 62 us; 4576 rows of 5120 in fp32 119 and 108; of 1024
// or 2048 in bf16 alike).
int backward_parts(int64_t rows, int d)
{
    const int64_t most = d <= 1024 ? 1024 : 512;
    const int tpr = choose(d, true).tpr, rpw = wg_threads(tpr) / tpr;
    const int64_t need = (rows + rpw - 1) / rpw;
    if (need <= most) return (int)need;
    const int64_t each = (need + most - 1) / most;   // turns a workgroup takes, the same for all but the last
    return (int)((need + each - 1) / each);
}
// Workgroups of the forward pass: one row a row group, more by grid stride.
unsigned forward_grid(int64_t rows, int tpr)
{
    const int rpw = wg_threads(tpr) / tpr;
    const int64_t need = (rows + rpw - 1) / rpw;
    return (unsigned)(need < (1 << 20) ? need : (1 << 20));
}

Shape shape_of(const NormArgs& a)
{
    return Shape{(int64_t)a.T * a.H, a.H, a.d, (a.d + kCkptGroup - 1) / kCkptGroup, 1.0f / (float)a.d,
                 a.eps, a.center};
}

#define GDN_NORM_CHOICES(X)                                                                  \
    X(4, 1, 8) X(8, 1, 8) X(16, 1, 8) X(32, 1, 8) X(64, 1, 8) X(64, 2, 8) X(256, 1, 8)       \
    X(256, 2, 8) X(256, 3, 8) X(256, 4, 8) X(64, 1, 1) X(64, 2, 1) X(64, 4, 1) X(256, 4, 1)  \
    X(256, 8, 1) X(1024, 4, 1) X(1024, 8, 1)

template <typename T, bool GATE>
void forward_gated(const NormArgs& a, bool vec8, hipStream_t s)
{
    const Choice c = choose(a.d, vec8);
    const Shape sh = shape_of(a);
    const dim3 grid(forward_grid(sh.rows, c.tpr));
#define GDN_RUN(TPR, NV, VEC)                                                                             \
    if (c.tpr == TPR && c.nv == NV && c.vec == VEC)                                                       \
        hipLaunchKernelGGL((gdn_norm_forward_kernel<T, TPR, NV, VEC, GATE>), grid, dim3(wg_threads(TPR)), 0, s,        \
                           (const T*)a.x, (const T*)a.z, a.w, a.b, (T*)a.y, a.x_codes, a.x_exps_out,      \
                           a.z_codes, a.z_exps_out, sh, a.x_stride, a.z_stride, a.y_stride);
    GDN_NORM_CHOICES(GDN_RUN)
#undef GDN_RUN
}

template <typename A, typename T, bool GATE>
void backward_gated(const NormArgs& a, hipStream_t s)
{
    const Choice c = choose(a.d, backward_vec8(a));
    const Shape sh = shape_of(a);
    const dim3 grid((unsigned)backward_parts(sh.rows, a.d));
#define GDN_RUN(TPR, NV, VEC)                                                                              \
    if (c.tpr == TPR && c.nv == NV && c.vec == VEC)                                                        \
        hipLaunchKernelGGL((gdn_norm_backward_kernel<A, T, TPR, NV, VEC, GATE>), grid, dim3(wg_threads(TPR)), 0, s,     \
                           (const A*)a.x, a.x_exps, (const A*)a.z, a.z_exps, a.w, a.b, (const T*)a.dy,     \
                           (T*)a.dx, (T*)a.dz, (float*)a.workspace, sh, a.x_stride, a.z_stride,            \
                           a.y_stride, a.dx_stride, a.dz_stride);
    GDN_NORM_CHOICES(GDN_RUN)
#undef GDN_RUN
}

template <typename T>
void forward_typed(const NormArgs& a, bool vec8, hipStream_t s)
{
    if (a.z) forward_gated<T, true>(a, vec8, s);
    else forward_gated<T, false>(a, vec8, s);
}
template <typename A, typename T>
void backward_typed(const NormArgs& a, hipStream_t s)
{
    if (a.z) backward_gated<A, T, true>(a, s);
    else backward_gated<A, T, false>(a, s);
}

}  // namespace

size_t norm_workspace_bytes(int T, int H, int d)
{
    return (size_t)backward_parts((int64_t)T * H, d) * 2 * d * sizeof(float);
}

Geometry norm_forward_geometry(const NormArgs& a)
{
    const Choice c = choose(a.d, forward_vec8(a));
    return Geometry{c.vec == 8 ? "gdn_norm_forward_kernel<8>" : "gdn_norm_forward_kernel<1>",
                    {forward_grid((int64_t)a.T * a.H, c.tpr), 1, 1}, (unsigned)wg_threads(c.tpr),
                    c.tpr > 64 ? (unsigned)(6 * kMaxWaves * sizeof(float)) : 4u};
}

Geometry norm_backward_geometry(const NormArgs& a)
{
    const Choice c = choose(a.d, backward_vec8(a));
    return Geometry{c.vec == 8 ? "gdn_norm_backward_kernel<8>+gdn_norm_weight_kernel"
                               : "gdn_norm_backward_kernel<1>+gdn_norm_weight_kernel",
                    {(unsigned)backward_parts((int64_t)a.T * a.H, a.d), 1, 1}, (unsigned)wg_threads(c.tpr),
                    (unsigned)(c.tpr > 64 ? 6 * kMaxWaves * sizeof(float)
                                          : kThreads * c.nv * c.vec * sizeof(float))};
}

hipError_t launch_norm_forward(const NormArgs& a, hipStream_t s)
{
    if (a.T == 0) return hipSuccess;
    const bool v8 = forward_vec8(a);
    if (a.io_dtype == 0) forward_typed<float>(a, v8, s);
    else forward_typed<uint16_t>(a, v8, s);
    hipError_t e = hipGetLastError();
    // value by value, the lanes of a row do not hold whole groups: the
    // checkpoints are passes of their own
    for (int i = 0; i < 2 && !v8 && e == hipSuccess; ++i) {
        CkptArgs c{};
        c.x = i ? a.z : a.x;
        c.codes = i ? a.z_codes : a.x_codes;
        c.exps_out = i ? a.z_exps_out : a.x_exps_out;
        if (!c.codes) continue;
        c.rows = (int64_t)a.T * a.H;
        c.d = a.d;
        c.stride = i ? a.z_stride : a.x_stride;
        c.dtype = a.io_dtype;
        e = launch_ckpt_store_heads(c, a.H, s);
    }
    return e;
}

hipError_t launch_norm_backward(const NormArgs& a, hipStream_t s)
{
    if (a.T > 0) {
        if (a.act_dtype == 2) {
            if (a.io_dtype == 0) backward_typed<uint8_t, float>(a, s);
            else backward_typed<uint8_t, uint16_t>(a, s);
        } else if (a.io_dtype == 0) {
            backward_typed<float, float>(a, s);
        } else {
            backward_typed<uint16_t, uint16_t>(a, s);
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const int parts = a.T > 0 ? backward_parts((int64_t)a.T * a.H, a.d) : 0;
    const unsigned halves = a.db ? 2 : 1;
    if (a.d <= 1024)
        hipLaunchKernelGGL((gdn_norm_weight_kernel<8>), dim3((a.d + 7) / 8, halves), dim3(kThreads), 0, s,
                           (const float*)a.workspace, parts, a.d, a.dw, a.db);
    else
        hipLaunchKernelGGL((gdn_norm_weight_kernel<32>), dim3((a.d + 31) / 32, halves), dim3(kThreads), 0, s,
                           (const float*)a.workspace, parts, a.d, a.dw, a.db);
    return hipGetLastError();
}

}  // namespace gdn
