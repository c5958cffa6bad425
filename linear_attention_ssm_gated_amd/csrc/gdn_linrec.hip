// The gated linear recurrence with a vector state, h_t = a_t h_{t-1} + c(a_t) x_t
// per channel, over sequences, its gradients, and one token of it
// (include/gdn_linrec.h).
//
// Walks.  A run of rows maps the state before it to the state behind it by
// h -> A h + B, A the product of its decays, and such maps compose.  The rows
// are cut into segments of R; a lane walks Lt rows of V channels, the lanes of
// a workgroup compose their maps through LDS, and the segments' maps are
// composed over the workspace: one pass over the rows, with the states between the
// segments handed on while all rows are in registers.  Backward is the same walk from the last row to
// the first, of G_t = a_t D_t: G_t = a_t G_{t+1} + a_t dy_t, D_t = dy_t + G_{t+1}.
// Where a sequence begins (for backward: ends) the walk's state is replaced by
// h0 (dh_final), so dense and packed rows are one axis of rows, and the maps of
// such runs do not depend on what is before: A is not used there, not even as a
// zero, which would carry an infinity of one sequence into the next as NaN.
//
// Bound by HBM and by the latency of a segment's steps (ticket 1 us, loads and first walk
// 4, waiting for the waves and for the state before 3.5, stores and the next workgroup's
// start 3; two workgroups a compute unit overlap them).  Measured, bf16: 4576 x 6144 with the
// root scale 42 us (169 MB, 4.0 TB/s; reading and writing the same tiles and nothing else
// takes 37, a 1 GiB copy reaches 5.1 TB/s), its gradients 76 us (337 MB, 4.5 TB/s), 40000 x 768
// 47.5 us (184 MB, 3.9 TB/s: 157 segments one behind the other).  Reading the rows twice, first
// for the maps, took 85, 103 and 85 us.
#include "gdn_linrec_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;        // of the single token and the clearing
constexpr int kWaves = 8;            // of a workgroup of the rows
constexpr int kRowThreads = 64 * kWaves;
constexpr int kChannels = 64;        // channels of a workgroup
constexpr int kOutside = -2;         // marks of a row: belongs to no sequence,
constexpr int kInside = -1;          // or is neither first nor last of one

// Global memory takes vector accesses on any address; rows may start on odd ones.
typedef uint32_t u2 __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u4 __attribute__((ext_vector_type(4), aligned(1)));

// The map of a segment for one channel, in one word that is read and written at
// once: B below, above it A with the sign bit set (a decay has none), or kReset
// where the map does not depend on the state before.  Zero: not there yet.
constexpr uint32_t kReset = 0xffffffffu;
__device__ __forceinline__ uint64_t map_word(float A, float B, bool reset)
{
    const uint32_t hi = reset ? kReset : __float_as_uint(A) | 0x80000000u;
    return (uint64_t)hi << 32 | __float_as_uint(B);
}
__device__ __forceinline__ bool map_resets(uint64_t w) { return (uint32_t)(w >> 32) == kReset; }
__device__ __forceinline__ float map_apply(uint64_t w, float h)
{
    const float B = __uint_as_float((uint32_t)w);
    return map_resets(w) ? B : fmaf(__uint_as_float((uint32_t)(w >> 32) & 0x7fffffffu), h, B);
}

// V values as they lie in memory.
template <int V, typename T> struct Raw {
    static constexpr int W = V * sizeof(T) >= 4 ? V * sizeof(T) / 4 : 1;
    uint32_t w[W];
    __device__ __forceinline__ void load(const T* p)
    {
        if constexpr (V == 1) {
            if constexpr (sizeof(T) == 4) w[0] = __float_as_uint(*p);
            else w[0] = (uint32_t)*p;
        } else if constexpr (W == 4) {
            const u4 v = *reinterpret_cast<const u4*>(p);
            w[0] = v[0]; w[1] = v[1]; w[2] = v[2]; w[3] = v[3];
        } else {
            static_assert(W == 2, "8 or 16 bytes a lane");
            const u2 v = *reinterpret_cast<const u2*>(p);
            w[0] = v[0]; w[1] = v[1];
        }
    }
    __device__ __forceinline__ float get(int j) const
    {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[j]);
        else if (V > 1 && (j & 1)) return __uint_as_float(w[j / 2] & 0xffff0000u);
        else return __uint_as_float(w[j / 2] << 16);
    }
};

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2v{lo, hi}, b2));
}
// Outputs go past the caches, which the inputs' lines need until all their parts are read
// (4576 x 4096 in bf16: 26 us, through them 31; 2000 x 4096 in fp32: 20, 24).  Inputs do not:
// past the caches too, 4576 x 6144 takes 41.6 us for 42.2, but 4576 x 4096 30 for 26, and rows
// off 16 bytes, whose lines two lanes share, 37 for 30.
template <int V> __device__ __forceinline__ void store_vec(float* p, const float* f)
{
    if constexpr (V == 4)
        __builtin_nontemporal_store(u4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                                       __float_as_uint(f[3])},
                                    reinterpret_cast<u4*>(p));
    else
#pragma unroll
        for (int j = 0; j < V; ++j) p[j] = f[j];
}
template <int V> __device__ __forceinline__ void store_vec(uint16_t* p, const float* f)
{
    if constexpr (V == 8)
        __builtin_nontemporal_store(u4{bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]),
                                       bf16_pair(f[6], f[7])},
                                    reinterpret_cast<u4*>(p));
    else if constexpr (V == 4)
        __builtin_nontemporal_store(u2{bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3])}, reinterpret_cast<u2*>(p));
    else
        *p = f32_to_bf16_bits(f[0]);
}

// a = exp(l), and with an input scale u = 1 - a with its own digits: sqrt(1 - a^2) =
// sqrt((1 - a)(1 + a)) is formed from it.  Near 0, for -1/4 < l < 0, 1 - a is -expm1(l) =
// -(l + l^2 p(l)), p the cubic whose largest error there, relative to expm1, is least (2^-28,
// with its coefficients rounded; the Taylor polynomial of as many terms is 2^-19 off at -1/4):
// 1 - a within 1.5 2^-24 of itself, and a within (1 + 3 |l|) 2^-25.  Else a is off by
// (2 + |l|) 2^-23 of itself, and 1 - a, at least 0.22, by 2^-20 of itself at most.  Without an
// input scale a alone is wanted, and for |l| < 1/64 a cubic gives it (2^-28.6 off there, and
// rounded once): the hardware's exp2 is up to 0.69 2^-24 off near 0 and 2^-27 too low on the
// average, which adds up over the 1 / (1 - a) tokens that a state lasts.  (Five instructions a
// value: 1168 x 5120 in bf16 takes 11.9 us for 11.3.)  S: 0 plain, 1 complement, 2 root.
template <int S> struct Decay {
    float a, u;
    __device__ __forceinline__ explicit Decay(float l)
    {
        const float far = __builtin_amdgcn_exp2f(l * 1.44269504f);
        if constexpr (S == 0) {
            const float q = fmaf(l, fmaf(l, fmaf(l, 1.0f / 6, 0.5f), 1.0f), 1.0f);
            a = fabsf(l) < 0x1p-6f ? q : far;
            u = 1.0f;
        } else {
            float q = fmaf(l, 0x1.ed7c28p-8f, 0x1.53f7d6p-5f);
            q = fmaf(l, q, 0x1.554e1ap-3f);
            q = fmaf(l, q, 0x1.ffffe8p-2f);
            q = fmaf(l * l, q, l);
            const bool near = __float_as_uint(l) - 0x80000000u < 0x3e800000u;
            a = near ? 1.0f + q : far;
            u = near ? -q : 1.0f - far;
        }
    }
    // 2^96 (1 - a^2): the roots' instructions take values under 2^-126 as zeros
    __device__ __forceinline__ float raised() const { return u * fmaf(a, 0x1p96f, 0x1p96f); }
    __device__ __forceinline__ float scale() const
    {
        return S == 0 ? 1.0f : S == 1 ? u : __builtin_amdgcn_sqrtf(raised()) * 0x1p-48f;
    }
    // scale(), and c' = dc/dlog_a (0 where c is)
    __device__ __forceinline__ void scale_and_slope(float& c, float& dc) const
    {
        if constexpr (S == 0) {
            c = 1.0f;
            dc = 0.0f;
        } else if constexpr (S == 1) {
            c = u;
            dc = -a;
        } else {
            const float w = raised(), r = w > 0.0f ? __builtin_amdgcn_rsqf(w) : 0.0f;
            c = w * 0x1p-48f * r;
            dc = -a * 0x1p48f * a * r;
        }
    }
};

constexpr int kTicketWords = 32;     // from one block's ticket to the next: lines of their own

// Rows of a lane's run, by its channels and the direction, and R of the segment: what
// 128 registers a lane take, so that two workgroups share a compute unit.  A forward call
// of few rows and channels takes one segment with longer runs, a workgroup to a compute
// unit: no maps to clear and to wait for.  200 and 380 rows in fp32 take 8.7 and 9.5 us with
// 768 channels, in segments 10.3 and 10.4; 8.8 and 9.7 for 10.5 and 10.2 with 2048, the last
// that the rule lets in; 10.0 for 10.2 with 2560 and 10.5 for 10.4 with 5120, where the
// segments fill the chip.  bf16 rows and gates gain with the plain scale (300 x 768: 7.8 us for
// 9.8); with the root 300 or 500 rows take 10.2 to 10.4 either way up to 2048 channels, 10.9
// for 10.2 with 5120.  Backward, whose runs need three times the registers, 380 x 768 took
// 12.8 for 11.0 in segments, and has no such form.
template <int V, bool BACK> struct RowsOf {
    static constexpr int kRuns = 64 / (kChannels / V) * kWaves;
    static constexpr int LT = V == 1 ? 8 : V == 8 ? (BACK ? 2 : 4) : BACK ? 3 : 4;
    static constexpr int R = kRuns * LT;
    static constexpr int kBriefLT = V == 1 || BACK ? LT : V == 8 ? 8 : 12;
    static constexpr int kBriefR = kRuns * kBriefLT;
    static bool brief(int rows, int blocks) { return rows > R && rows <= kBriefR && blocks <= 32; }
    static int rows(int all, int blocks) { return brief(all, blocks) ? kBriefR : R; }
};
template <int V, int LT, bool BACK> constexpr int waves_a_simd() { return LT > RowsOf<V, BACK>::LT ? 2 : 4; }

struct Launch {
    LinrecArgs p;
    int rows;          // all rows
    int blocks;        // of 64 channels
    int segments;
    unsigned* tickets; // segments > 1: workgroups that have started, for each block
    uint64_t* maps;    // [segments][blocks * 64]
};

__device__ __forceinline__ int clamped_row(const LinrecArgs& p, int b)
{
    // (nothing writes the offsets while the call runs: read as constants, through the scalar cache
    // where b is the same for all lanes)
    const int v = ((const __attribute__((address_space(4))) int32_t*)p.cu)[b];
    return v < 0 ? 0 : v > p.T ? p.T : v;
}

// Whether the n places of the walk from `first` on, a wave's, lie inside one sequence,
// neither its first nor its last row among them.  Where they do not, enter[k] becomes the
// sequence that the walk enters at place first + k, leave[k] the one it leaves there
// (kInside: none), and kOutside in enter where no sequence has the row.  A row that is
// inside is its sequence's first, or there is a row before it: row 0 is inside only where
// a sequence begins there, whatever the offsets.
template <bool BACK>
__device__ __forceinline__ bool wave_marks(const Launch& g, int first, int n, int* enter, int* leave)
{
    const LinrecArgs& p = g.p;
    const int low = BACK ? g.rows - first - n : first;    // the rows low .. low + n - 1 (some may not be there)
    int b = 0;                                            // the first sequence that ends behind low
    if (g.rows > 0) {
        if (!p.cu) {
            b = low > 0 ? low / p.T : 0;
            if (b < p.B && low > b * p.T && low + n < (b + 1) * p.T) return true;
        } else {
            int hi = p.B;
            while (b < hi) {
                const int mid = (b + hi) / 2;
                if (clamped_row(p, mid + 1) > low) hi = mid;
                else b = mid + 1;
            }
            if (b < p.B && low > clamped_row(p, b) && low + n < clamped_row(p, b + 1)) return true;
        }
    }
    for (int k = threadIdx.x % 64; k < n; k += 64) {
        const int row = BACK ? low + n - 1 - k : low + k;
        int e = kOutside, l = kInside;
        if (row >= 0 && row < g.rows) {
            int q = b, s, end;                            // the row's sequence, its first row and its end
            if (!p.cu) {
                q = row / p.T;
                s = q * p.T;
                end = s + p.T;
            } else {
                int hi = p.B;
                while (q < hi) {
                    const int mid = (q + hi) / 2;
                    if (clamped_row(p, mid + 1) > row) hi = mid;
                    else q = mid + 1;
                }
                s = q < p.B ? clamped_row(p, q) : g.rows;
                end = q < p.B ? clamped_row(p, q + 1) : g.rows;
            }
            if (s <= row && row < end) {
                e = row == (BACK ? end - 1 : s) ? q : kInside;
                l = row == (BACK ? s : end - 1) ? q : kInside;
            }
        }
        enter[k] = e;
        leave[k] = l;
    }
    return false;
}

// The state before segment seg for a channel (one lane each), from the maps of the
// segments before it, word[p * pitch].  Walks back to the nearest map that does not
// depend on what is before it and composes from there on in the rows' order, so that
// the result does not depend on how far the others are.
//
// Every wait ends: a block's segments are handed out in order, by a ticket, to
// workgroups that run, and a workgroup writes its own map without waiting for anything.
// Where the workspace is not the call's own, against the contract, a map may never come:
// after kPatience readings (seconds) the state is taken as NaN.
constexpr int kPatience = 1 << 22;
__device__ __forceinline__ float state_before(const uint64_t* word, int64_t pitch, int seg)
{
    constexpr int K = 6;                  // maps that are read at a time
    uint64_t w[K];
    int top = seg - 1, left = kPatience;
    for (;;) {
        bool ready = true, found = false;
#pragma unroll
        for (int j = 0; j < K; ++j)
            w[j] = top - j >= 0 ? __hip_atomic_load(word + (top - j) * pitch, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)
                                : (uint64_t)kReset << 32;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            ready = ready && (found || w[j] != 0);
            found = found || map_resets(w[j]);
        }
        if (!__all(ready)) {
            if (--left == 0) return __builtin_nanf("");
            __builtin_amdgcn_s_sleep(1);
            continue;
        }
        if (__all(found)) break;
        top -= K;
    }
    float h = 0.0f;
#pragma unroll
    for (int j = K - 1; j >= 0; --j) h = map_apply(w[j], h);
    for (int p = top + 1; p < seg; ++p)
        h = map_apply(__hip_atomic_load(word + p * pitch, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT), h);
    return h;
}

// LDS operations of one wave are done in order: this keeps the compiler to it.
__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// One pass over the rows: a workgroup reads a segment of R rows of 64 channels
// into registers, forms the segment's map, hands it on, takes the state before
// the segment from the maps before it, and writes the rows.
template <typename TX, typename TG, int V, int LT, int S, bool BACK>
__global__ void __launch_bounds__(kRowThreads, (waves_a_simd<V, LT, BACK>()))
gdn_linrec_kernel(Launch g)
{
    constexpr int CL = kChannels / V;                 // lanes of a row
    constexpr int WL = 64 / CL;                       // runs of LT rows in a wave
    constexpr int TL = WL * kWaves;
    constexpr int R = TL * LT;
    __shared__ float sA[TL][kChannels], sB[TL][kChannels], sState[kChannels];
    __shared__ uint64_t sMap[kWaves][kChannels];
    __shared__ int sReset[TL], sEnter[R], sLeave[R], sTicket;
    const LinrecArgs& p = g.p;
    // the workgroups of one XCD (every eighth) take neighbouring blocks, whose rows lie next to each other
    int cb = blockIdx.x % (unsigned)g.blocks;
    if (g.blocks % 8 == 0) cb = cb % 8 * (g.blocks / 8) + cb / 8;
    int seg = 0;
    if (g.segments > 1) {
        if (threadIdx.x == 0)
            sTicket = (int)__hip_atomic_fetch_add(g.tickets + cb * kTicketWords, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        seg = __builtin_amdgcn_readfirstlane(sTicket);
        seg = seg < g.segments ? seg : g.segments - 1;    // (beyond only where another call uses the workspace too)
    }
    const int first = seg * R;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
    const int run = threadIdx.x / CL;                 // the thread's place among the runs
    const int cl = (threadIdx.x % CL) * V;            // its first channel in the block
    const bool live = cb * kChannels + cl < p.D;
    // a row's last lane takes its last V channels: some twice, with the same results
    const int ch = cb * kChannels + cl < p.D - V ? cb * kChannels + cl : p.D - V;

    // The rows' values: x, or backward dy with h_{t-1} and x.  Places behind the last
    // row take that row's values, and are not used; nor is row 0's h_{t-1}.
    Raw<V, TX> rb[LT], ry[BACK ? LT : 1], rx[BACK && S != 0 ? LT : 1];
    Raw<V, TG> rl[LT];
    const TX* const in = static_cast<const TX*>(BACK ? p.dy : p.x) + ch;
    const int64_t in_stride = BACK ? p.dy_stride : p.x_stride;
    const TG* const gate = static_cast<const TG*>(p.log_a) + ch;
    const TX* const y = static_cast<const TX*>(p.y) + ch;
    const TX* const x = static_cast<const TX*>(p.x) + ch;
    const int start = first + run * LT;
    const auto fetch = [&](int i, int64_t row, int64_t row_before) {
        rb[i].load(in + row * in_stride);
        rl[i].load(gate + row * p.a_stride);
        if constexpr (BACK) {
            ry[i].load(y + row_before * p.y_stride);
            if constexpr (S != 0) rx[i].load(x + row * p.x_stride);
        }
    };
    if (first + R < g.rows) {                         // all there, row 0 not among them in backward
        const int64_t row = BACK ? g.rows - 1 - start : start;
#pragma unroll
        for (int i = 0; i < LT; ++i) fetch(i, BACK ? row - i : row + i, row - i - 1);
    } else if (g.rows > 0) {
#pragma unroll
        for (int i = 0; i < LT; ++i) {
            const int at = start + i < g.rows ? start + i : g.rows - 1;
            const int64_t row = BACK ? g.rows - 1 - at : at;
            fetch(i, row, row > 0 ? row - 1 : 0);
        }
    }
    // (LDS arrays by run or row belong to the run's wave alone)
    const bool quiet = wave_marks<BACK>(g, first + wave * WL * LT, WL * LT, sEnter + wave * WL * LT, sLeave + wave * WL * LT);
    const int *enter = sEnter + run * LT, *leave = sLeave + run * LT;
    wave_fence();

    // the run's map; the decays and forward the inputs stay in registers for the second walk
    const float* fresh = BACK ? p.dh_final : p.h0;    // the state a sequence is entered with
    float A[V], h[V], a[LT][V], u[BACK && S != 0 ? LT : 1][V], b[BACK ? 1 : LT][V];
    bool reset = false;
#pragma unroll
    for (int j = 0; j < V; ++j) { A[j] = 1.0f; h[j] = 0.0f; }
    const auto first_walk = [&](int i) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const Decay<S> k(rl[i].get(j));
            a[i][j] = k.a;
            A[j] *= k.a;
            if constexpr (BACK) {
                if constexpr (S != 0) u[i][j] = k.u;
                h[j] = k.a * (h[j] + rb[i].get(j));
            } else {
                b[i][j] = S == 0 ? rb[i].get(j) : k.scale() * rb[i].get(j);
                h[j] = fmaf(k.a, h[j], b[i][j]);
            }
        }
    };
    const auto enter_state = [&](int sequence) {
#pragma unroll
        for (int j = 0; j < V; ++j) h[j] = fresh ? fresh[(int64_t)sequence * p.D + ch + j] : 0.0f;
    };
    if (quiet) {
#pragma unroll
        for (int i = 0; i < LT; ++i) first_walk(i);
    } else {
#pragma unroll
        for (int i = 0; i < LT; ++i) {
            const int e = enter[i];
            if (e == kOutside) continue;
            if (e >= 0) {
                reset = true;
                enter_state(e);
            }
            first_walk(i);
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        sA[run][cl + j] = A[j];
        sB[run][cl + j] = h[j];
    }
    if (cl == 0) sReset[run] = reset;
    wave_fence();

    // the maps of the wave's runs one behind the other, a lane a channel
    uint64_t maps[WL];
    {
        float aa = 1.0f, s = 0.0f;
        bool r = false;
#pragma unroll
        for (int k = 0; k < WL; ++k) {
            const float ak = sA[wave * WL + k][lane];
            maps[k] = map_word(ak, sB[wave * WL + k][lane], sReset[wave * WL + k]);
            s = map_apply(maps[k], s);
            aa *= ak;
            r = r || map_resets(maps[k]);
        }
        sMap[wave][lane] = map_word(aa, s, r);
    }
    const int64_t pitch = (int64_t)g.blocks * kChannels;
    uint64_t* const word = g.maps + cb * kChannels + lane;
    __syncthreads();
    if (wave == 0) {
        float aa = 1.0f, s = 0.0f, before = 0.0f;
        bool r = seg == 0;                            // nothing is before the first segment
#pragma unroll
        for (int k = 0; k < kWaves; ++k) {
            const uint64_t w = sMap[k][lane];
            s = map_apply(w, s);
            aa *= __uint_as_float((uint32_t)(w >> 32) & 0x7fffffffu);
            r = r || map_resets(w);
        }
        if (seg + 1 < g.segments)
            __hip_atomic_store(word + seg * pitch, map_word(aa, s, r), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (seg > 0 && (quiet || sEnter[0] < 0)) {
            before = state_before(word, pitch, seg);
            if (seg + 1 < g.segments && !r)
                __hip_atomic_store(word + seg * pitch, map_word(0.0f, fmaf(aa, before, s), true), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        sState[lane] = before;
    }
    __syncthreads();
    // the state before each run of the wave
    {
        float s = sState[lane];
        for (int k = 0; k < wave; ++k) s = map_apply(sMap[k][lane], s);
#pragma unroll
        for (int k = 0; k < WL; ++k) {
            sB[wave * WL + k][lane] = s;
            s = map_apply(maps[k], s);
        }
    }
    wave_fence();

    // sequences without rows, 64 at a time
    float* const last = BACK ? p.dh0 : p.h_final;
    if (seg == 0 && last && (p.cu || p.T == 0)) {
        const int c = cb * kChannels + lane;
        for (int q0 = wave * 64; q0 < p.B; q0 += kRowThreads) {
            const int q = q0 + lane;
            uint64_t empty = __ballot(q < p.B && (!p.cu || clamped_row(p, q + 1) <= clamped_row(p, q)));
            for (; empty; empty &= empty - 1) {
                const int64_t at = (int64_t)(q0 + __builtin_ctzll(empty)) * p.D + c;
                if (c < p.D) last[at] = fresh ? fresh[at] : 0.0f;
            }
        }
    }
    if (!live) return;

    // the rows once more, from the state before the run
#pragma unroll
    for (int j = 0; j < V; ++j) h[j] = sB[run][cl + j];
    const auto second_walk = [&](int i, int64_t row, int out) {
        if constexpr (!BACK) {
#pragma unroll
            for (int j = 0; j < V; ++j) h[j] = fmaf(a[i][j], h[j], b[i][j]);
            store_vec<V>(static_cast<TX*>(p.y) + row * p.y_stride + ch, h);
        } else {
            float dx[V], dl[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float before = ry[i].get(j);
                if (out >= 0) before = p.h0 ? p.h0[(int64_t)out * p.D + ch + j] : 0.0f;
                const float D = h[j] + rb[i].get(j);
                if constexpr (S == 0) {
                    dx[j] = D;
                    dl[j] = D * (a[i][j] * before);
                } else {
                    Decay<S> k(0.0f);
                    float c, dc;
                    k.a = a[i][j];
                    k.u = u[i][j];
                    k.scale_and_slope(c, dc);
                    dx[j] = c * D;
                    dl[j] = D * fmaf(dc, rx[i].get(j), k.a * before);
                }
                h[j] = a[i][j] * D;
            }
            store_vec<V>(static_cast<TX*>(p.dx) + row * p.dx_stride + ch, dx);
            store_vec<V>(static_cast<TG*>(p.dlog_a) + row * p.da_stride + ch, dl);
        }
    };
    const int64_t row = BACK ? g.rows - 1 - (int64_t)start : start;
    if (quiet) {
#pragma unroll
        for (int i = 0; i < LT; ++i) second_walk(i, BACK ? row - i : row + i, kInside);
    } else {
#pragma unroll
        for (int i = 0; i < LT; ++i) {
            const int e = enter[i], out = leave[i];
            if (e == kOutside) continue;
            if (e >= 0) enter_state(e);
            second_walk(i, BACK ? row - i : row + i, out);
            if (out >= 0 && last) {
#pragma unroll
                for (int j = 0; j < V; ++j) last[(int64_t)out * p.D + ch + j] = h[j];
            }
        }
    }
}

// Ahead of a call of several segments: no ticket taken, no map there.
__global__ void __launch_bounds__(kThreads)
gdn_linrec_clear_kernel(u4* p, int64_t n)
{
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads)
        p[i] = u4{0, 0, 0, 0};
}

// ---- one token ---------------------------------------------------------------
// V channels a lane; the last lane of a row may have fewer (the state changes in
// place, so no channel is taken twice here).  16 sequences of 6144: a few microseconds on the
// GPU, less than the 6 of the host's call.
template <typename TX, typename TG, int V, int S>
__global__ void __launch_bounds__(kThreads)
gdn_linrec_step_kernel(LinrecStepArgs p)
{
    typedef float f4 __attribute__((ext_vector_type(4), aligned(4)));   // states on any 4 bytes
    const int b = blockIdx.y;
    const int ch = (blockIdx.x * kThreads + threadIdx.x) * V;
    if (ch >= p.D) return;
    float* const state = p.h_table[b];
    if (!state) return;
    const TX* x = static_cast<const TX*>(p.x) + b * p.x_stride + ch;
    const TG* l = static_cast<const TG*>(p.log_a) + b * p.a_stride + ch;
    TX* y = static_cast<TX*>(p.y) + b * p.y_stride + ch;
    GDN_GLOBAL float* at = (GDN_GLOBAL float*)state + ch;
    if (p.D - ch < V) {
        for (int j = 0; j < p.D - ch; ++j) {
            const Decay<S> k(Elem<TG>::load(l + j));
            const float h = fmaf(k.a, at[j], S == 0 ? Elem<TX>::load(x + j) : k.scale() * Elem<TX>::load(x + j));
            at[j] = h;
            Elem<TX>::store(y + j, h);
        }
        return;
    }
    Raw<V, TX> rx;
    Raw<V, TG> rl;
    rx.load(x);
    rl.load(l);
    float h[V];
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        const f4 v = *(GDN_GLOBAL f4*)(at + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[i + j] = v[j];
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const Decay<S> k(rl.get(j));
        h[j] = fmaf(k.a, h[j], S == 0 ? rx.get(j) : k.scale() * rx.get(j));
    }
#pragma unroll
    for (int i = 0; i < V; i += 4) *(GDN_GLOBAL f4*)(at + i) = f4{h[i], h[i + 1], h[i + 2], h[i + 3]};
    store_vec<V>(y, h);
}

// ---- launches ----------------------------------------------------------------
constexpr int kLeastRows = 64;   // the smallest segment of any form
static_assert(RowsOf<8, false>::R >= kLeastRows && RowsOf<4, false>::R >= kLeastRows && RowsOf<1, false>::R >= kLeastRows &&
              RowsOf<8, true>::R >= kLeastRows && RowsOf<4, true>::R >= kLeastRows && RowsOf<1, true>::R >= kLeastRows, "workspace");

// Channels of a lane: 16 bytes of the rows' type, or of the gates' where these are wider.
// Narrower rows than that take one.
int lane_channels(int io, int gate) { return io == 1 && gate == 1 ? 8 : 4; }
int channels_of(const LinrecArgs& a)
{
    const int v = lane_channels(a.io_dtype, a.gate_dtype);
    return a.D < v ? 1 : v;
}
int rows_of(const LinrecArgs& a) { return a.cu ? a.T : a.B * a.T; }
template <bool BACK> int segment_rows(int v, int rows, int blocks)
{
    return v == 8 ? RowsOf<8, BACK>::rows(rows, blocks)
           : v == 4 ? RowsOf<4, BACK>::rows(rows, blocks) : RowsOf<1, BACK>::rows(rows, blocks);
}
int segments(int rows, int r) { return rows ? (rows - 1) / r + 1 : 1; }
int blocks_of(int D) { return (D + kChannels - 1) / kChannels; }
size_t ticket_bytes(int D) { return (size_t)blocks_of(D) * kTicketWords * sizeof(unsigned); }

template <typename TX, typename TG, int V, int S, bool BACK>
hipError_t launch_form(const LinrecArgs& a, hipStream_t s)
{
    using Rows = RowsOf<V, BACK>;
    const int rows = rows_of(a), n = segments(rows, Rows::rows(rows, blocks_of(a.D)));
    char* ws = static_cast<char*>(a.workspace);
    const Launch g{a, rows, blocks_of(a.D), n, reinterpret_cast<unsigned*>(ws),
                   reinterpret_cast<uint64_t*>(ws + (n > 1 ? ticket_bytes(a.D) : 0))};
    if (n > 1) {
        const int64_t words = (ticket_bytes(a.D) + (int64_t)(n - 1) * g.blocks * kChannels * sizeof(uint64_t)) / 16;
        const int64_t grid = (words + kThreads - 1) / kThreads;
        hipLaunchKernelGGL(gdn_linrec_clear_kernel, dim3((unsigned)(grid < 1024 ? grid : 1024)), dim3(kThreads), 0, s,
                           reinterpret_cast<u4*>(ws), words);
    }
    const dim3 grid((unsigned)n * g.blocks);
    if constexpr (Rows::kBriefLT != Rows::LT) {
        if (Rows::brief(rows, g.blocks)) {
            hipLaunchKernelGGL((gdn_linrec_kernel<TX, TG, V, Rows::kBriefLT, S, BACK>), grid, dim3(kRowThreads), 0, s, g);
            return hipGetLastError();
        }
    }
    hipLaunchKernelGGL((gdn_linrec_kernel<TX, TG, V, Rows::LT, S, BACK>), grid, dim3(kRowThreads), 0, s, g);
    return hipGetLastError();
}
template <typename TX, typename TG, int V, int S>
hipError_t launch_way(const LinrecArgs& a, hipStream_t s)
{
    return a.backward ? launch_form<TX, TG, V, S, true>(a, s) : launch_form<TX, TG, V, S, false>(a, s);
}
template <typename TX, typename TG, int V>
hipError_t launch_scale(const LinrecArgs& a, hipStream_t s)
{
    return a.scale == 0 ? launch_way<TX, TG, V, 0>(a, s)
           : a.scale == 1 ? launch_way<TX, TG, V, 1>(a, s) : launch_way<TX, TG, V, 2>(a, s);
}

template <typename TX, typename TG, int V>
hipError_t launch_step_scale(const LinrecStepArgs& a, hipStream_t s)
{
    const dim3 grid((unsigned)((a.D + kThreads * V - 1) / (kThreads * V)), (unsigned)a.B);
    if (a.scale == 0) hipLaunchKernelGGL((gdn_linrec_step_kernel<TX, TG, V, 0>), grid, dim3(kThreads), 0, s, a);
    else if (a.scale == 1) hipLaunchKernelGGL((gdn_linrec_step_kernel<TX, TG, V, 1>), grid, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((gdn_linrec_step_kernel<TX, TG, V, 2>), grid, dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace

size_t linrec_workspace_bytes(int64_t rows, int D)
{
    const int64_t n = rows ? (rows - 1) / kLeastRows + 1 : 1;
    return n > 1 ? ticket_bytes(D) + (size_t)(n - 1) * blocks_of(D) * kChannels * sizeof(uint64_t) : 0;
}

Geometry linrec_geometry(const LinrecArgs& a)
{
    const int v = channels_of(a);
    const int rows = rows_of(a), blocks = blocks_of(a.D);
    const int n = segments(rows, a.backward ? segment_rows<true>(v, rows, blocks) : segment_rows<false>(v, rows, blocks));
    const char* name = a.backward ? (n > 1 ? "gdn_linrec_clear_kernel+gdn_linrec_kernel<backward>" : "gdn_linrec_kernel<backward>")
                                  : (n > 1 ? "gdn_linrec_clear_kernel+gdn_linrec_kernel<forward>" : "gdn_linrec_kernel<forward>");
    return Geometry{name, {(unsigned)n * (unsigned)blocks_of(a.D), 1, 1}, kRowThreads, 0};
}

hipError_t launch_linrec(const LinrecArgs& a, hipStream_t s)
{
    const int v = channels_of(a);
    if (a.io_dtype == 0)
        return v == 1 ? launch_scale<float, float, 1>(a, s) : launch_scale<float, float, 4>(a, s);
    if (a.gate_dtype == 0)
        return v == 1 ? launch_scale<uint16_t, float, 1>(a, s) : launch_scale<uint16_t, float, 4>(a, s);
    return v == 1 ? launch_scale<uint16_t, uint16_t, 1>(a, s) : launch_scale<uint16_t, uint16_t, 8>(a, s);
}

Geometry linrec_step_geometry(const LinrecStepArgs& a)
{
    const int per = kThreads * lane_channels(a.io_dtype, a.gate_dtype);
    return Geometry{"gdn_linrec_step_kernel", {(unsigned)((a.D + per - 1) / per), (unsigned)a.B, 1}, kThreads, 0};
}

hipError_t launch_linrec_step(const LinrecStepArgs& a, hipStream_t s)
{
    if (a.io_dtype == 0) return launch_step_scale<float, float, 4>(a, s);
    if (a.gate_dtype == 0) return launch_step_scale<uint16_t, float, 4>(a, s);
    return launch_step_scale<uint16_t, uint16_t, 8>(a, s);
}

}  // namespace gdn
