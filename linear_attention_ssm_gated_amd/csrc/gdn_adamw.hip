// One AdamW step over many tensors, states in fp32 or in 8 bits
// (include/gdn_adamw.h): the kernel, the host-side validation and the launches.
//
// Every value is read once and written once.  A lane has 8 neighbouring values,
// so that 16 lanes hold a group of 128 and find its largest magnitude by lane
// exchanges.  The tensors' descriptions travel in the kernel's arguments (no
// table in device memory to fill before the call or to keep valid behind it), up
// to 64 (with 8-bit states 48) a launch; a workgroup finds its tensor among them by one compare a
// lane.  Addresses need the alignment of their element type only: global memory
// takes 16-byte accesses on any address.
//
// Measured for 115.8 M values in 8 tensors, bf16 weights and gradients.  fp32 masters and
// states: 604 us (3.2 GB, 5.35 TB/s: bound by HBM; a 1 GiB copy reaches 5.12).  States in 8
// bits, chance rounding, no masters: 255 to 262 us (1.17 GB, 4.5 TB/s); bound by the vector units,
// about 80 instructions a value (26 of them the random bits), which keep every SIMD busy
// nine tenths of the time.  120 tensors of up to 5120 values: 10 us, two launches on the
// host's side.
#include "../../include/gdn_adamw.h"
#include "gdn_train_internal.h"

#include <math.h>

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;                    // values of a lane
constexpr int kStep = kThreads * kPer;     // values of a workgroup's step: whole groups
constexpr int kMaxBlocks = 1 << 20;

struct Entry {
    void* w;
    float* master;
    const void* g;
    void *m, *v;
    int64_t n;
    float weight_decay, decay;             // decay = 1 - lr weight_decay, without a control
};
struct Scales {
    float *m, *v;
};
// A launch's tensors: as many as 4 KB of arguments take.
template <bool E8> struct Pack {
    static constexpr int kTensors = E8 ? 48 : 64;
    Entry t[kTensors];
    Scales s[E8 ? kTensors : 1];
    int first[kTensors + 1];               // first workgroup of each tensor; behind the last: the grid
    int count, place;                      // tensors, and the first one's place in the call
    int64_t chunk;                         // values of a workgroup
    float factor, beta1, gain1, beta2, gain2, eps, rate, root;   // gain = 1 - beta, rate = lr / (1 - beta1^t), root = 1 / sqrt(1 - beta2^t)
    uint32_t seed;
    const float* control;
};
static_assert(sizeof(Pack<true>) <= 4096 && sizeof(Pack<false>) <= 4096, "kernel arguments");

typedef uint32_t u4 __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u2 __attribute__((ext_vector_type(2), aligned(1)));

// n of 8 values (fewer at a tensor's end; the rest are zero)
__device__ __forceinline__ void load8(const float* p, int n, float* f)
{
    if (n >= kPer) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const u4 v = *reinterpret_cast<const u4*>(p + 4 * i);
#pragma unroll
            for (int j = 0; j < 4; ++j) f[4 * i + j] = __uint_as_float(v[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j) f[j] = j < n ? p[j] : 0.0f;
    }
}
__device__ __forceinline__ void load8(const uint16_t* p, int n, float* f)
{
    if (n >= kPer) {
        const u4 v = *reinterpret_cast<const u4*>(p);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[2 * j] = __uint_as_float(v[j] << 16);
            f[2 * j + 1] = __uint_as_float(v[j] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j) f[j] = j < n ? bf16_bits_to_f32(p[j]) : 0.0f;
    }
}
__device__ __forceinline__ void load8(const uint8_t* p, int n, float* f)
{
    if (n >= kPer) {
        const u2 v = *reinterpret_cast<const u2*>(p);
        ckpt_unpack4(v[0], f);
        ckpt_unpack4(v[1], f + 4);
    } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j) f[j] = j < n ? ckpt_unpack1(p[j]) : 0.0f;
    }
}
__device__ __forceinline__ void store8(float* p, int n, const float* f)
{
    if (n >= kPer) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            *reinterpret_cast<u4*>(p + 4 * i) = u4{__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]),
                                                   __float_as_uint(f[4 * i + 2]), __float_as_uint(f[4 * i + 3])};
    } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (j < n) p[j] = f[j];
    }
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2v{lo, hi}, b2));
}
__device__ __forceinline__ void store8(uint16_t* p, int n, const float* f)
{
    if (n >= kPer) {
        *reinterpret_cast<u4*>(p) = u4{bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]),
                                       bf16_pair(f[6], f[7])};
    } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (j < n) p[j] = f32_to_bf16_bits(f[j]);
    }
}

// 32 bits mixed: multiplications by odd numbers (the fractions of sqrt(2) and
// sqrt(3)) carry bits up, shifts bring them down.
__device__ __forceinline__ uint32_t mix(uint32_t x)
{
    x ^= x >> 16;
    x *= 0x6a09e667u;
    x ^= x >> 15;
    x *= 0xbb67ae85u;
    return x ^ (x >> 16);
}

// sqrt(v), correctly rounded: v 1/sqrt(v) with its remainder added, which is what IEEE's
// square root gives for every float from 2^-100 to 2^100 (all of them compared).  Where
// some value of the wave lies outside (zeros among them) all go through sqrtf, and the
// result is false.
__device__ __forceinline__ bool roots(const float* v, float* r)
{
    float least = v[0], most = v[0];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        least = fminf(least, v[j]);
        most = fmaxf(most, v[j]);                    // (NaN is passed over, and stays NaN)
        const float y = __builtin_amdgcn_rsqf(v[j]), s = v[j] * y;
        r[j] = fmaf(fmaf(-s, s, v[j]), 0.5f * y, s);
    }
    if (!__any(!(least >= 0x1p-100f && most <= 0x1p100f))) return true;
#pragma unroll
    for (int j = 0; j < kPer; ++j) r[j] = sqrtf(v[j]);
    return false;
}

// m / d by the reciprocal and the remainder: a division's result save where the quotient is
// within 2^-45 of the middle of two floats.  Where there is no remainder (infinities, NaN,
// d = 0) the product has the right value.
__device__ __forceinline__ float quotient(float m, float d)
{
    const float y = __builtin_amdgcn_rcpf(d), q = m * y, r = fmaf(-q, d, m);
    return fabsf(r) < __builtin_inff() ? fmaf(r, y, q) : q;
}

// 1 in place of the bytes that are 0
__device__ __forceinline__ uint32_t bytes_above_zero(uint32_t c)
{
    return c | (((c & 0x7f7f7f7fu) + 0x7f7f7f7fu) & 0x80808080u ^ 0x80808080u) >> 7;
}

// the largest of 16 lanes' values, in all of them
template <int CTRL> __device__ __forceinline__ float max_with(float x)
{
    return fmaxf(x, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true)));
}
__device__ __forceinline__ float max16(float x)
{
    x = max_with<0x128>(x);   // rotations by 8, 4, 2, 1 within a row of 16 lanes
    x = max_with<0x124>(x);
    x = max_with<0x122>(x);
    return max_with<0x121>(x);
}

// 8 values as codes with their group's scale.  By chance: the conversion adds the upper 20
// of the bits it is given to the 20 that it cuts off (below 2^-6, e4m3's subnormals, to
// those below 2^-9), 16 random ones and zeros.  A root's code is at least 1 where the root
// is above zero; positive: all of the wave's are.
template <bool ROOT, bool SR>
__device__ __forceinline__ void keep8(uint8_t* codes, float* scales, int64_t at, int n, float* f, const uint32_t* bits,
                                      bool positive)
{
#pragma clang fp contract(off)
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < kPer; ++j) top = fmaxf(top, fabsf(f[j]));   // (NaN is passed over)
    top = max16(top);
    if (__any(top == __builtin_inff())) {            // infinities become NaN, and the scale is the rest's
        top = 0.0f;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            top = fmaxf(top, ckpt_magnitude(f[j]));
            f[j] = ckpt_finite(f[j]);
        }
        top = max16(top);
    }
    float scale = top * (1.0f / 448.0f);
    if (top > 0.0f) scale = fmaxf(scale, 0x1p-126f);
    const float inv = scale > 0.0f ? 1.0f / scale : 0.0f;
    float y[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        y[j] = f[j] * inv;
        if (ROOT && !positive) y[j] = f[j] > 0.0f && y[j] < 0x1p-9f ? 0x1p-9f : y[j];
    }
    uint32_t lo, hi;
    if constexpr (SR) {
        int c[2] = {0, 0};
        const auto random = [&](int j) { return ROOT ? bits[j] & 0xffff0000u : bits[j] << 16; };
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            c[k] = __builtin_amdgcn_cvt_sr_fp8_f32(y[4 * k], random(4 * k), c[k], 0);
            c[k] = __builtin_amdgcn_cvt_sr_fp8_f32(y[4 * k + 1], random(4 * k + 1), c[k], 1);
            c[k] = __builtin_amdgcn_cvt_sr_fp8_f32(y[4 * k + 2], random(4 * k + 2), c[k], 2);
            c[k] = __builtin_amdgcn_cvt_sr_fp8_f32(y[4 * k + 3], random(4 * k + 3), c[k], 3);
        }
        lo = (uint32_t)c[0];
        hi = (uint32_t)c[1];
    } else {
        lo = ckpt_pack4(y[0], y[1], y[2], y[3]);
        hi = ckpt_pack4(y[4], y[5], y[6], y[7]);
    }
    if (ROOT && positive) {
        lo = bytes_above_zero(lo);
        hi = bytes_above_zero(hi);
    }
    if (n >= kPer) {
        *reinterpret_cast<u2*>(codes + at) = u2{lo, hi};
    } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (j < n) codes[at + j] = (uint8_t)((j < 4 ? lo : hi) >> (8 * (j & 3)));
    }
    if (n > 0 && (threadIdx.x & 15) == 0) scales[at / GDN_ADAMW_GROUP] = scale;
}

// fp32 onto bf16's grid, up with the probability of the part cut off
__device__ __forceinline__ float chance_bf16(float w, uint32_t bits16)
{
    return w == w ? __uint_as_float((__float_as_uint(w) + bits16) & 0xffff0000u) : w;
}

// W: 0 fp32 weights, 1 bf16, 2 bf16 with fp32 masters
template <int W, typename TG, bool E8, bool SR>
__global__ void __launch_bounds__(kThreads)
gdn_adamw_kernel(Pack<E8> pk)
{
#pragma clang fp contract(off)
    // the tensor of this workgroup: as many as end ahead of it
    const int lane = threadIdx.x & 63;
    const bool behind = lane < pk.count && (int)blockIdx.x >= pk.first[lane + 1];
    const int i = __builtin_amdgcn_readfirstlane(__popcll(__ballot(behind)));
    const Entry& t = pk.t[i];
    float factor = pk.factor, rate = pk.rate, root = pk.root, decay = t.decay;
    uint32_t seed = pk.seed;
    if (pk.control) {
        const float lr = pk.control[0];
        rate = lr / pk.control[1];
        root = 1.0f / sqrtf(pk.control[2]);
        factor = pk.control[3];
        seed = __float_as_uint(pk.control[4]);
        decay = 1.0f - lr * t.weight_decay;
        if (!(factor > 0.0f && factor < __builtin_inff())) return;
    }
    const uint32_t key0 = mix(mix(seed ^ 0x3c6ef372u) + (uint32_t)(pk.place + i));
    const int64_t begin = (int64_t)((int)blockIdx.x - pk.first[i]) * pk.chunk;
    const int64_t end = begin + pk.chunk < t.n ? begin + pk.chunk : t.n;
    for (int64_t base = begin; base < end; base += kStep) {
        const int64_t at = base + threadIdx.x * kPer;
        const int64_t left = t.n - at;
        const int n = left >= kPer ? kPer : left > 0 ? (int)left : 0;
        float g[kPer], m[kPer], v[kPer], w[kPer];
        if (n > 0) {
            load8(static_cast<const TG*>(t.g) + at, n, g);
            if constexpr (W == 0) load8(static_cast<const float*>(t.w) + at, n, w);
            else if constexpr (W == 1) load8(static_cast<const uint16_t*>(t.w) + at, n, w);
            else load8(t.master + at, n, w);
            if constexpr (E8) {
                load8(static_cast<const uint8_t*>(t.m) + at, n, m);
                load8(static_cast<const uint8_t*>(t.v) + at, n, v);
                const float sm = pk.s[i].m[at / GDN_ADAMW_GROUP], sv = pk.s[i].v[at / GDN_ADAMW_GROUP];
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    m[j] = m[j] * sm;
                    const float r = v[j] * sv;
                    v[j] = r * r;
                }
            } else {
                load8(static_cast<const float*>(t.m) + at, n, m);
                load8(static_cast<const float*>(t.v) + at, n, v);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kPer; ++j) g[j] = m[j] = v[j] = w[j] = 0.0f;
        }
        float r[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const float gj = g[j] * factor;
            m[j] = m[j] * pk.beta1 + gj * pk.gain1;
            v[j] = v[j] * pk.beta2 + (gj * gj) * pk.gain2;
        }
        // With 8-bit states the arithmetic is what bounds the kernel: square roots by one
        // correction, and quotients from the hardware's reciprocal (r is zero or above 2^-75, so
        // that none is lost below the normal floats).  Weights in bf16 alone, rounded to 2^-9 at
        // once, take it as it is, within 2^-22 (115.8 M values 262 us; corrected 270, divided 281);
        // the others corrected (fp32 weights 350 us, as without; divided 353).
        bool positive = false;
        if constexpr (E8) {
            positive = roots(v, r);
        } else {
#pragma unroll
            for (int j = 0; j < kPer; ++j) r[j] = sqrtf(v[j]);
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const float d = r[j] * root + pk.eps;
            const float u = !E8 ? m[j] / d : W == 1 ? m[j] * __builtin_amdgcn_rcpf(d) : quotient(m[j], d);
            w[j] = w[j] * decay - u * rate;
        }
        uint32_t bits[kPer];
        if constexpr (SR) {
            const uint32_t hi = (uint32_t)((uint64_t)at >> 32);
            const uint32_t key = key0 ^ (hi * 0x9e3779b1u);
#pragma unroll
            for (int j = 0; j < kPer; ++j) bits[j] = mix(((uint32_t)at + j) ^ key);
        }
        if (n > 0) {
            if constexpr (W == 0) {
                store8(static_cast<float*>(t.w) + at, n, w);
            } else {
                if constexpr (W == 2) store8(t.master + at, n, w);
                if constexpr (W == 1 && SR)
#pragma unroll
                    for (int j = 0; j < kPer; ++j) w[j] = chance_bf16(w[j], mix(bits[j] ^ 0x510e527fu) & 0xffffu);
                store8(static_cast<uint16_t*>(t.w) + at, n, w);
            }
            if constexpr (!E8) {
                store8(static_cast<float*>(t.m) + at, n, m);
                store8(static_cast<float*>(t.v) + at, n, v);
            }
        }
        if constexpr (E8) {      // all 16 lanes of a group come here
            keep8<false, SR>(static_cast<uint8_t*>(t.m), pk.s[i].m, at, n, m, bits, false);
            keep8<true, SR>(static_cast<uint8_t*>(t.v), pk.s[i].v, at, n, r, bits, positive);
        }
    }
}

struct Call {
    const gdn_adamw_tensor* tensors;
    int count;
    double lr, beta1, beta2, eps;
    int64_t step;
    double factor;
    const float* control;
    int w_dtype, g_dtype, state_dtype;
    bool stochastic;
    uint32_t seed;
};

// what the kernel multiplies by, in fp32
float rate_of(const Call& a) { return (float)(a.lr / (1 - pow(a.beta1, (double)a.step))); }
float decay_of(const Call& a, const gdn_adamw_tensor& t) { return (float)(1.0 - a.lr * (double)t.weight_decay); }

int check(const Call& a)
{
    const char* who = "gdn_adamw_step";
    if ((a.w_dtype != GDN_F32 && a.w_dtype != GDN_BF16) || (a.g_dtype != GDN_F32 && a.g_dtype != GDN_BF16))
        return refuse_call(GDN_ERR_DTYPE, who, "w_dtype and g_dtype must be GDN_F32 or GDN_BF16");
    if (a.state_dtype != GDN_F32 && a.state_dtype != GDN_E4M3)
        return refuse_call(GDN_ERR_DTYPE, who, "state_dtype must be GDN_F32 or GDN_E4M3");
    if (a.count < 0) return refuse_call(GDN_ERR_SHAPE, who, "need count >= 0");
    if (a.count > 0 && !a.tensors) return refuse_call(GDN_ERR_NULL, who, "tensors is required");
    if (!(a.beta1 >= 0 && a.beta1 < 1 && a.beta2 >= 0 && a.beta2 < 1)) return refuse_call(GDN_ERR_SHAPE, who, "need 0 <= beta1, beta2 < 1");
    if (!(a.eps >= 0) || !isfinite((float)a.eps)) return refuse_call(GDN_ERR_SHAPE, who, "eps must be finite in fp32 and not negative");
    // (the quotient's reciprocal takes a divisor under that as zero)
    if (a.state_dtype == GDN_E4M3 && a.eps > 0 && a.eps < 0x1p-126)
        return refuse_call(GDN_ERR_SHAPE, who, "with 8-bit states eps must be 0 or at least 2^-126");
    if (!a.control && (!isfinite((float)a.lr) || !isfinite((float)a.factor) || a.step < 1))
        return refuse_call(GDN_ERR_SHAPE, who, "lr and grad_factor must be finite in fp32, step >= 1");
    if (!a.control && !isfinite(rate_of(a)))
        return refuse_call(GDN_ERR_SHAPE, who, "lr / (1 - beta1^step) must be finite in fp32");
    int master = -1;      // not known yet
    for (int i = 0; i < a.count; ++i) {
        const gdn_adamw_tensor& t = a.tensors[i];
        if (t.n < 0 || t.n > (1LL << 40)) return refuse_call(GDN_ERR_SHAPE, who, "need 0 <= n <= 2^40");
        if (!(t.weight_decay >= 0) || !isfinite(t.weight_decay))
            return refuse_call(GDN_ERR_SHAPE, who, "weight_decay must be finite and not negative");
        if (t.reserved != 0) return refuse_call(GDN_ERR_SHAPE, who, "reserved must be 0");
        if (t.n == 0) continue;
        if (!a.control && !isfinite(decay_of(a, t)))
            return refuse_call(GDN_ERR_SHAPE, who, "1 - lr weight_decay must be finite in fp32");
        if (!t.w || !t.g || !t.m || !t.v) return refuse_call(GDN_ERR_NULL, who, "w, g, m and v are required");
        if ((a.state_dtype == GDN_E4M3) != (t.m_scale && t.v_scale) || (a.state_dtype == GDN_F32 && (t.m_scale || t.v_scale)))
            return refuse_call(GDN_ERR_NULL, who, "8-bit states need both scales, fp32 states take none");
        if (t.master && a.w_dtype != GDN_BF16) return refuse_call(GDN_ERR_DTYPE, who, "masters go with BF16 weights");
        if (master >= 0 && master != (t.master != nullptr))
            return refuse_call(GDN_ERR_NULL, who, "all tensors of a call have masters, or none");
        master = t.master != nullptr;
    }
    return GDN_OK;
}

bool has_master(const Call& a)
{
    for (int i = 0; i < a.count; ++i)
        if (a.tensors[i].n > 0) return a.tensors[i].master != nullptr;
    return false;
}

// Packs the tensors from `from` on, as many as a launch takes, and returns the
// next one; pk->first[pk->count] workgroups (0: nothing to do).
template <bool E8> int fill(const Call& a, int from, Pack<E8>* pk)
{
    int64_t total = 0;
    pk->count = 0;
    int at = from;
    // Tensors without values are left out, but a launch's places in the call are
    // consecutive (place + i): one ends the launch where others are in it already.
    while (at < a.count && a.tensors[at].n == 0) ++at;
    pk->place = at;
    for (; at < a.count && pk->count < Pack<E8>::kTensors && a.tensors[at].n > 0; ++at) {
        const gdn_adamw_tensor& t = a.tensors[at];
        if constexpr (E8) pk->s[pk->count] = Scales{t.m_scale, t.v_scale};
        Entry& e = pk->t[pk->count++];
        e.w = t.w; e.master = t.master; e.g = t.g; e.m = t.m; e.v = t.v; e.n = t.n;
        e.weight_decay = t.weight_decay;
        e.decay = decay_of(a, t);
        total += t.n;
    }
    // One step a workgroup (115.8 M values, fp32 states: 603 us, with two 618), or with 8-bit
    // states two, where these are still many rounds of workgroups: there the arithmetic
    // counts, and what a workgroup does ahead of its steps (260 us, with one 266); more
    // where the grid would not take them.
    const int64_t steps = (total + kStep - 1) / kStep;
    const int64_t least = E8 && steps > 16384 ? 2 : 1, most = (steps + kMaxBlocks - 1) / kMaxBlocks;
    pk->chunk = kStep * (most > least ? most : least);
    int64_t blocks = 0;
    for (int i = 0; i < pk->count; ++i) {
        pk->first[i] = (int)blocks;
        blocks += (pk->t[i].n + pk->chunk - 1) / pk->chunk;
    }
    pk->first[pk->count] = (int)blocks;
    return at;
}

template <bool E8> void scalars(const Call& a, Pack<E8>* pk)
{
    const double c2 = 1 - pow(a.beta2, (double)a.step);
    pk->factor = (float)a.factor;
    pk->beta1 = (float)a.beta1; pk->gain1 = (float)(1 - a.beta1);
    pk->beta2 = (float)a.beta2; pk->gain2 = (float)(1 - a.beta2);
    pk->eps = (float)a.eps;
    pk->rate = rate_of(a);
    pk->root = (float)(1 / sqrt(c2));
    pk->seed = a.seed;
    pk->control = a.control;
}

template <int W, typename TG, bool E8>
void launch_form(const Pack<E8>& pk, bool sr, hipStream_t s)
{
    const dim3 grid((unsigned)pk.first[pk.count]);
    if constexpr (W == 1 || E8) {
        if (sr) {
            hipLaunchKernelGGL((gdn_adamw_kernel<W, TG, E8, true>), grid, dim3(kThreads), 0, s, pk);
            return;
        }
    }
    hipLaunchKernelGGL((gdn_adamw_kernel<W, TG, E8, false>), grid, dim3(kThreads), 0, s, pk);
}
template <int W, bool E8> void launch_grad(const Call& a, const Pack<E8>& pk, hipStream_t s)
{
    if (a.g_dtype == GDN_F32) launch_form<W, float, E8>(pk, a.stochastic, s);
    else launch_form<W, uint16_t, E8>(pk, a.stochastic, s);
}

// The route line names the first launch, and whether there are more.
template <bool E8> void route(const Call& a)
{
    Pack<E8> pk;
    const int at = fill<E8>(a, 0, &pk);
    if (!pk.count) {
        route_call(Geometry{"nothing to launch", {0, 0, 0}, 0, 0}, "");
        return;
    }
    bool more = false;
    for (int i = at; i < a.count; ++i) more = more || a.tensors[i].n > 0;
    route_call(Geometry{"gdn_adamw_kernel", {(unsigned)pk.first[pk.count], 1, 1}, kThreads, 0},
               more ? "(the first of several launches)" : "");
}
template <bool E8> hipError_t launch(const Call& a, hipStream_t s)
{
    Pack<E8> pk;
    scalars<E8>(a, &pk);
    const bool master = has_master(a);
    for (int at = 0; at < a.count;) {
        at = fill<E8>(a, at, &pk);
        if (pk.count == 0) break;
        if (a.w_dtype == GDN_F32) launch_grad<0, E8>(a, pk, s);
        else if (master) launch_grad<2, E8>(a, pk, s);
        else launch_grad<1, E8>(a, pk, s);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

int plan(const Call& a)
{
    const int st = check(a);
    if (st != GDN_OK) return st;
    if (a.state_dtype == GDN_E4M3) route<true>(a);
    else route<false>(a);
    return GDN_OK;
}

int run(const Call& a, hipStream_t s)
{
    const int st = plan(a);
    if (st != GDN_OK) return st;
    return launch_status(a.state_dtype == GDN_E4M3 ? launch<true>(a, s) : launch<false>(a, s));
}

}  // namespace
}  // namespace gdn

extern "C" {

int gdn_adamw_step_plan(const gdn_adamw_tensor* tensors, int count, double lr, double beta1, double beta2, double eps,
                        int64_t step, double grad_factor, const float* control, int w_dtype, int g_dtype,
                        int state_dtype, int stochastic, uint32_t seed)
{
    return gdn::plan(gdn::Call{tensors, count, lr, beta1, beta2, eps, step, grad_factor, control, w_dtype, g_dtype,
                               state_dtype, stochastic != 0, seed});
}

int gdn_adamw_step(const gdn_adamw_tensor* tensors, int count, double lr, double beta1, double beta2, double eps,
                   int64_t step, double grad_factor, const float* control, int w_dtype, int g_dtype, int state_dtype,
                   int stochastic, uint32_t seed, hipStream_t stream)
{
    return gdn::run(gdn::Call{tensors, count, lr, beta1, beta2, eps, step, grad_factor, control, w_dtype, g_dtype,
                              state_dtype, stochastic != 0, seed},
                    stream);
}

}  // extern "C"
