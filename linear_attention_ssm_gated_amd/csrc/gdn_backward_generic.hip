// Generic backward pass of the gated delta rule: fp32 arithmetic on fp32, bf16
// or 8-bit inputs, any dk, dv <= 128.  The formulas are in
// gdn_backward_common.h.  Three kernels:
//   prep    one workgroup per (chunk, v-head): B, P, T, W, U, Qt
//   spine   one workgroup per (sequence, v-head, 16 or 32 dv columns, direction): the
//           states walked forwards and their gradients backwards, both in the
//           same launch, every chunk's start state and end gradient written
//   grads   one workgroup per (chunk, v-head): the chunk's gradients; dq and dk
//           of v-heads that share a k-head go to the workspace and
//   sum     adds them in the v-heads' order
// Products run on fp32 MFMA (16x16x4: exact fp32 operands); the chunk's running
// sums of log_g and their differences are fp64, since a difference of two large
// sums would lose the decay's digits.  Head sizes are padded with zeros to 32, 64
// or 128, or 96 of dv, in the workspace, which the kernels know at compile time: with
// tile counts of the call, every tile stood behind a branch of its own and its LDS
// reads were waited for one by one (85 us for the gradients of 16 chunks x 6 heads
// of 64 x 96; 58 with constants and 64 x 128, 51 with 64 x 96, 43 with eight waves for
// four; 128 x 128 takes the same with either).  2 x 500 tokens of 2 / 6 heads, 64 x
// 96, with both end states take 98 us back to back (prep 32, spine 22, grads 42, sum
// 5): 96 workgroups for 256 compute units, bound by the latency of their chains of
// fp32 products.
#include "gdn_backward_common.h"

#include <type_traits>

namespace gdn {
namespace {

using bwd::C;
using bwd::ChunkAt;

constexpr int kThreads = 256;
constexpr int kMP = bwd::kBP;        // pitch of a 64 x 64 matrix in LDS

using bwd::f32x4;
using bwd::mfma4;

// Lane (g, n) = (lane / 16, lane % 16) supplies A[n][k] and B[k][n] of a 16 x 16
// tile's product with k = 16 kb + 4 g + s at step s (any order of k is one sum)
// and holds rows 4g .. 4g + 3 of column n.
// acc[j] += A B_j for NT column tiles that share A's rows: a(kb) gives A[n][kb +
// 4 g .. + 3] of this lane, b(j, k) B_j[k][n].  A step's operands are read before
// the products of the step before.
template <int K, int NT, typename FA, typename FB>
__device__ __forceinline__ void mm_tiles(f32x4 (&acc)[NT], FA&& a, FB&& b)
{
    const int g = (threadIdx.x & 63) >> 4;
    f32x4 av[2];
    float bv[2][NT][4];
    auto read = [&](int t) {
        av[t & 1] = a(16 * t);
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int s = 0; s < 4; ++s) bv[t & 1][j][s] = b(j, 16 * t + 4 * g + s);
    };
    read(0);
#pragma unroll
    for (int t = 0; t < K / 16; ++t) {
        if (t + 1 < K / 16) read(t + 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[j] = mfma4(av[t & 1][s], bv[t & 1][j][s], acc[j]);
    }
}
template <int NT> __device__ __forceinline__ void clear(f32x4 (&acc)[NT])
{
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j] = f32x4{0, 0, 0, 0};
}
__device__ __forceinline__ f32x4 four(const float* p) { return *reinterpret_cast<const f32x4*>(p); }

// Workspace of one (chunk, v-head) and of one (chunk, k-head), in floats.
struct Sizes {
    int dkp, dvp;
    __host__ __device__ size_t mats() const { return 3 * (size_t)C * C; }                  // T, B, P
    __host__ __device__ size_t head() const { return mats() + 2 * (size_t)C * dkp + 2 * (size_t)C * dvp + 2 * C; }   // + W, Qt, U, V, G
    __host__ __device__ size_t state() const { return (size_t)dkp * dvp; }
    __host__ __device__ size_t group() const { return 2 * (size_t)C * dkp; }               // K, Q
};

struct Ws {
    int32_t* base;     // chunk table (packed)
    float* heads;      // [chunk][Hv] head()
    float* groups;     // [chunk][Hk] group()
    float* h;          // [chunk][Hv] start states
    float* dh;         // [chunk][Hv] end gradients
    float* part;       // [chunk][Hv] dq, dk of a v-head, where heads share
};

struct Args {
    const void *q, *k, *v, *dout;
    const uint8_t *q_exps, *k_exps, *v_exps;
    const float *log_g, *beta, *h0, *dht;
    void *dq, *dk, *dv, *dg, *db;
    float* dh0;
    int B, T, Hk, Hv, dk_, dv_;
    const int32_t* cu;
    int nc_dense;
    Sizes sz;
    Ws ws;
};

// value j of row r (token * heads + head) of an activation
template <typename T> __device__ __forceinline__ float act(const void* p, const uint8_t* exps, int64_t r, int d, int j)
{
    if constexpr (sizeof(T) == 1)
        return ckpt_unpack1(static_cast<const uint8_t*>(p)[r * d + j]) * ckpt_scale(exps[r]);
    else
        return Elem<T>::load(static_cast<const T*>(p) + r * d + j);
}

__global__ void __launch_bounds__(kThreads)
gdn_backward_table_kernel(const int32_t* __restrict__ cu, int B, int T, int32_t* __restrict__ base)
{
    __shared__ int32_t part[256];
    bwd::chunk_table(cu, B, T, base, part);
}

// The chunk's gates: G (running sum, fp64), beta, ga = exp(G), E = exp(G_L - G).
struct alignas(16) Gates {
    double G[C];
    float beta[C], ga[C], E[C];
};
__device__ __forceinline__ void load_gates(const Args& a, const ChunkAt& at, int vh, Gates* s)
{
    const int tid = threadIdx.x;
    if (tid < C) {
        const bool live = tid < at.rows;
        const int64_t r = (at.row0 + tid) * a.Hv + vh;
        s->G[tid] = live ? (double)bounded_log_decay(a.log_g[r]) : 0.0;   // (fp64 too has no digits left behind -1e38)
        s->beta[tid] = live ? a.beta[r] : 0.f;
    }
    __syncthreads();
    if (tid < C) {                            // one wave: the running sum, and the decays
        double G = s->G[tid];
#pragma unroll
        for (int o = 1; o < C; o <<= 1) {
            const double before = __shfl_up(G, o);
            if (tid >= o) G += before;
        }
        const double GL = __shfl(G, C - 1);
        s->G[tid] = G;
        s->ga[tid] = (float)exp(G);
        s->E[tid] = (float)exp(GL - G);
    }
    __syncthreads();
}
__device__ __forceinline__ float decay(const Gates& s, int r, int c) { return expf((float)(s.G[r] - s.G[c])); }

// ---- prep ----------------------------------------------------------------------
extern __shared__ __attribute__((aligned(16))) float lds_dyn[];

template <int NK, int NV, typename TA>
__global__ void __launch_bounds__(kThreads)
gdn_backward_prep_kernel(Args a)
{
    __shared__ Gates sg;
    constexpr int dkp = 16 * NK, dvp = 16 * NV, dp = dkp + 4, vp = dvp + 4;
    float* sK = lds_dyn;              // [C][dp]
    float* sQ = sK + C * dp;          // [C][dp], then T (ga K)
    float* sV = sQ + C * dp;          // [C][vp]
    float* sB = sV + C * vp;          // [C][kMP]
    float* sP = sB + C * kMP;
    float* sT = sP + C * kMP;

    ChunkAt at;
    const int x = blockIdx.x, vh = blockIdx.y, kh = vh / (a.Hv / a.Hk);
    if (!bwd::chunk_at(x, a.cu, a.ws.base, a.B, a.T, a.nc_dense, &at)) return;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, g = lane >> 4, n = lane & 15;
    float* head = a.ws.heads + ((size_t)x * a.Hv + vh) * a.sz.head();
    float *gT = head, *gB = gT + C * C, *gP = gB + C * C, *gW = gP + C * C, *gQt = gW + C * dkp,
          *gU = gQt + C * dkp, *gV = gU + C * dvp, *gG = gV + C * dvp;
    float* gK = a.ws.groups + ((size_t)x * a.Hk + kh) * a.sz.group();

    for (int e = tid; e < C * dkp; e += kThreads) {
        const int r = e / dkp, j = e % dkp;
        const bool live = r < at.rows && j < a.dk_;
        const int64_t row = (at.row0 + r) * a.Hk + kh;
        sK[r * dp + j] = live ? act<TA>(a.k, a.k_exps, row, a.dk_, j) : 0.f;
        sQ[r * dp + j] = live ? act<TA>(a.q, a.q_exps, row, a.dk_, j) : 0.f;
    }
    for (int e = tid; e < C * dvp; e += kThreads) {
        const int r = e / dvp, j = e % dvp;
        const float v = r < at.rows && j < a.dv_ ? act<TA>(a.v, a.v_exps, (at.row0 + r) * a.Hv + vh, a.dv_, j) : 0.f;
        sV[r * vp + j] = v;
        gV[e] = v;
    }
    load_gates(a, at, vh, &sg);
    if (vh % (a.Hv / a.Hk) == 0)
        for (int e = tid; e < C * dkp; e += kThreads) {
            const int r = e / dkp, j = e % dkp;
            gK[e] = sK[r * dp + j];
            gK[C * dkp + e] = sQ[r * dp + j];
        }
    if (tid < C) reinterpret_cast<double*>(gG)[tid] = sg.G[tid];

    // B and P: wave w forms rows 16 w .. + 15
    {
        f32x4 kk[4], qk[4];
        clear(kk);
        clear(qk);
        mm_tiles<dkp>(kk, [&](int kb) { return four(sK + (16 * w + n) * dp + kb + 4 * g); },
                 [&](int j, int k) { return sK[(16 * j + n) * dp + k]; });
        mm_tiles<dkp>(qk, [&](int kb) { return four(sQ + (16 * w + n) * dp + kb + 4 * g); },
                 [&](int j, int k) { return sK[(16 * j + n) * dp + k]; });
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int r = 16 * w + 4 * g + s, c = 16 * j + n;
                const float e = c <= r ? decay(sg, r, c) : 0.f;
                const float bv = c < r ? e * kk[j][s] : 0.f, pv = c <= r ? e * qk[j][s] : 0.f;
                sB[r * kMP + c] = bv;
                sP[r * kMP + c] = pv;
                gB[r * C + c] = bv;
                gP[r * C + c] = pv;
            }
    }
    __syncthreads();

    {
        if (w == 0) bwd::solve_diagonal(sB, sg.beta, sT);     // sT's place takes the diagonal blocks
        __syncthreads();
        f32x4 Tc[4];
        bwd::solve_column(sB, sg.beta, sT, w, Tc);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int s = 0; s < 4; ++s) sT[(16 * i + 4 * g + s) * kMP + 16 * w + n] = Tc[i][s];
    }
    __syncthreads();
    for (int e = tid; e < C * C; e += kThreads) gT[e] = sT[(e >> 6) * kMP + (e & 63)];

    // Z = T (ga K), W = E beta Z; U = E beta T V
    f32x4 z[NK], u[NV], t[NK], qv[NK];
    clear(z);
    clear(u);
    clear(t);
    auto row_of_T = [&](int kb) { return four(sT + (16 * w + n) * kMP + kb + 4 * g); };
    mm_tiles<C>(u, row_of_T, [&](int j, int k) { return sV[k * vp + 16 * j + n]; });
    mm_tiles<C>(z, row_of_T, [&](int j, int k) { return sg.ga[k] * sK[k * dp + 16 * j + n]; });
    // Q to registers, then Z in its place as the operand of P beta Z
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int r = 16 * w + 4 * g + s;
            gU[r * dvp + 16 * j + n] = sg.E[r] * sg.beta[r] * u[j][s];
        }
#pragma unroll
    for (int j = 0; j < NK; ++j)
#pragma unroll
        for (int s = 0; s < 4; ++s) qv[j][s] = sQ[(16 * w + 4 * g + s) * dp + 16 * j + n];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NK; ++j)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int r = 16 * w + 4 * g + s;
            gW[r * dkp + 16 * j + n] = sg.E[r] * sg.beta[r] * z[j][s];
            sQ[r * dp + 16 * j + n] = sg.beta[r] * z[j][s];
        }
    __syncthreads();
    mm_tiles<C>(t, [&](int kb) { return four(sP + (16 * w + n) * kMP + kb + 4 * g); },
                [&](int j, int k) { return sQ[k * dp + 16 * j + n]; });
#pragma unroll
    for (int j = 0; j < NK; ++j)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int r = 16 * w + 4 * g + s;
            gQt[r * dkp + 16 * j + n] = sg.ga[r] * qv[j][s] - t[j][s];
        }
}

// ---- spine -----------------------------------------------------------------------
// grid (Hv * column slices, B, 2): z = 0 walks the states, z = 1 their gradients.
// A step's operands come from memory as they are, fetched while the step before
// runs (two register sets): wave w needs rows 16 w .. + 15 of the left matrix (W,
// or K) and columns of state tiles w and w + 4 of the right ones (K, or W and Qt).
template <int NK, int NC, typename TG, bool REV>
__device__ __forceinline__ void spine_walk(const Args& a, int slices, float (&sS)[16 * NK][16 * NC + 4],
                                           float (&sD)[C][16 * NC + 4], float (&sO)[C][16 * NC + 4])
{
    constexpr int dkp = 16 * NK, NI = NK > 4 ? 2 : 1, kCols = 16 * NC;   // NI: row tiles of the state that a wave holds
    const int dvp = a.sz.dvp;
    const int vh = blockIdx.x / slices, col0 = (blockIdx.x % slices) * kCols, b = blockIdx.y;
    const int kh = vh / (a.Hv / a.Hk);
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, g = lane >> 4, n = lane & 15;
    const bool some = w < NK;                // wave w has a state tile

    int64_t row0, len;
    bwd::seq_rows(a.cu, b, a.T, &row0, &len);
    const int nc = bwd::walk_chunks(a.cu, a.ws.base, b, len);
    const int64_t x0 = a.cu ? a.ws.base[b] : (int64_t)b * a.nc_dense;
    const float* from = REV ? a.dht : a.h0;
    const size_t hoff = ((size_t)b * a.Hv + vh) * a.dk_ * a.dv_;

    // wave w holds state rows of tiles w and w + 4, every column tile
    f32x4 st[NI][NC];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int r = 16 * (w + 4 * i) + 4 * g + s, c = col0 + 16 * j + n;
                st[i][j][s] = from && r < a.dk_ && c < a.dv_ ? from[hoff + (size_t)r * a.dv_ + c] : 0.f;
            }

    struct Regs {
        f32x4 left[NK];      // row 16 w + n, k = 16 t + 4 g .. + 3
        float right[NI][16], qt[NI][16];   // column 16 (w + 4 i) + n, rows 16 (e / 4) + 4 g + e % 4
        float add[NC][4];           // U (rows 16 w + 4 g + s), or do (this thread's 4 NC)
        double gl;
    } in0, in1;
    auto chunk_of = [&](int i) { return (size_t)(x0 + (REV ? nc - 1 - i : i)); };
    auto fetch = [&](Regs& in, int i) {
        const size_t x = chunk_of(i);
        const float* head = a.ws.heads + (x * a.Hv + vh) * a.sz.head();
        const float *gW = head + a.sz.mats(), *gQt = gW + C * dkp, *gU = gQt + C * dkp;
        const float* gK = a.ws.groups + (x * a.Hk + kh) * a.sz.group();
        const float *left = REV ? gK : gW, *right = REV ? gW : gK;
#pragma unroll
        for (int t = 0; t < NK; ++t) in.left[t] = four(left + (16 * w + n) * dkp + 16 * t + 4 * g);
#pragma unroll
        for (int i2 = 0; i2 < NI; ++i2)
            if (some)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int k = 16 * (e >> 2) + 4 * g + (e & 3), m = 16 * (w + 4 * i2) + n;
                    in.right[i2][e] = right[k * dkp + m];
                    if constexpr (REV) in.qt[i2][e] = gQt[k * dkp + m];
                }
        if constexpr (REV) {
            const int64_t first = row0 + (int64_t)(nc - 1 - i) * C;
#pragma unroll
            for (int e = 0; e < 4 * NC; ++e) {
                const int r = (tid + kThreads * e) / kCols, j = (tid + kThreads * e) % kCols;
                in.add[e >> 2][e & 3] = first + r < row0 + len && col0 + j < a.dv_
                                            ? Elem<TG>::load(static_cast<const TG*>(a.dout) + ((first + r) * a.Hv + vh) * a.dv_ + col0 + j)
                                            : 0.f;
            }
        } else {
#pragma unroll
            for (int j = 0; j < NC; ++j)
#pragma unroll
                for (int s = 0; s < 4; ++s) in.add[j][s] = gU[(16 * w + 4 * g + s) * dvp + col0 + 16 * j + n];
        }
        in.gl = reinterpret_cast<const double*>(gU + 2 * C * dvp)[C - 1];
    };
    auto step = [&](int i, Regs& in, Regs& next) {
        const size_t x = chunk_of(i);
        float* out = (REV ? a.ws.dh : a.ws.h) + (x * a.Hv + vh) * a.sz.state();
        fetch(next, min(i + 1, nc - 1));
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i2 = 0; i2 < NI; ++i2)
#pragma unroll
            for (int j = 0; j < NC; ++j)
                if (some)
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const int r = 16 * (w + 4 * i2) + 4 * g + s;
                        sS[r][16 * j + n] = st[i2][j][s];
                        out[(size_t)r * dvp + col0 + 16 * j + n] = st[i2][j][s];
                    }
        if constexpr (REV)
#pragma unroll
            for (int e = 0; e < 4 * NC; ++e) sO[(tid + kThreads * e) / kCols][(tid + kThreads * e) % kCols] = in.add[e >> 2][e & 3];
        bwd::lds_barrier();
        // rows 16 w .. + 15 of W h (of K dh')
        f32x4 d[NC];
        clear(d);
#pragma unroll
        for (int kt = 0; kt < NK; ++kt)
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int j = 0; j < NC; ++j) d[j] = mfma4(in.left[kt][s], sS[16 * kt + 4 * g + s][16 * j + n], d[j]);
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
            for (int s = 0; s < 4; ++s) sD[16 * w + 4 * g + s][16 * j + n] = REV ? -d[j][s] : in.add[j][s] - d[j][s];
        bwd::lds_barrier();
        const float gL = (float)exp(in.gl);
        if (some) {
#pragma unroll
            for (int i2 = 0; i2 < NI; ++i2)
#pragma unroll
                for (int j = 0; j < NC; ++j) st[i2][j] *= gL;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int k = 16 * (e >> 2) + 4 * g + (e & 3);
#pragma unroll
                for (int j = 0; j < NC; ++j) {
                    const float dv = sD[k][16 * j + n], ov = REV ? sO[k][16 * j + n] : 0.f;
#pragma unroll
                    for (int i2 = 0; i2 < NI; ++i2) {
                        st[i2][j] = mfma4(in.right[i2][e], dv, st[i2][j]);
                        if constexpr (REV) st[i2][j] = mfma4(in.qt[i2][e], ov, st[i2][j]);
                    }
                }
            }
        }
        bwd::lds_barrier();   // sS, sD and sO have been read
    };
    if (nc > 0) fetch(in0, 0);
    for (int i = 0; i < nc; i += 2) {
        step(i, in0, in1);
        if (i + 1 < nc) step(i + 1, in1, in0);
    }
    if (REV && a.dh0)
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < NC; ++j)
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int r = 16 * (w + 4 * i) + 4 * g + s, c = col0 + 16 * j + n;
                    if (r < a.dk_ && c < a.dv_) a.dh0[hoff + (size_t)r * a.dv_ + c] = st[i][j][s];
                }
}

template <int NK, int NC, typename TG>
__global__ void __launch_bounds__(kThreads, 1)
gdn_backward_spine_kernel(Args a, int slices)
{
    __shared__ float sS[16 * NK][16 * NC + 4];   // the state's columns
    __shared__ float sD[C][16 * NC + 4];         // U - W h, or -K dh'
    __shared__ float sO[C][16 * NC + 4];         // do
    if (blockIdx.z == 0) spine_walk<NK, NC, TG, false>(a, slices, sS, sD, sO);
    else spine_walk<NK, NC, TG, true>(a, slices, sS, sD, sO);
}

// ---- grads -----------------------------------------------------------------------
// sum over the 16 lanes of a row's columns
__device__ __forceinline__ float sum16(float x)
{
#pragma unroll
    for (int o = 8; o; o >>= 1) x += __shfl_xor(x, o);
    return x;
}

// Eight waves: wave w of half p has rows 16 w .. + 15 of half the columns of dv, then
// of Zu (p = 0) or do u^T (1), then of half the columns of dk.
constexpr int kGradThreads = 512;

template <int NK, int NV, typename TG>
__global__ void __launch_bounds__(kGradThreads)
gdn_backward_grads_kernel(Args a)
{
    __shared__ Gates sg;
    __shared__ float s_dG[2][C], s_db[2][C], s_Y[2][C];   // row sums of a half
    __shared__ float s_colX[8][C], s_colZ[4][C];
    __shared__ float s_sum[8];
    constexpr int dkp = 16 * NK, dvp = 16 * NV, vp = dvp + 4, NH = NV / 2;
    float* s1 = lds_dyn;              // x, then u           [C][vp]
    float* s2 = s1 + C * vp;          // do
    float* s3 = s2 + C * vp;          // h, then dh' [dkp][vp], then beta ddelta, then dx
    float* sN = s3 + C * vp;          // N  [C][kMP]
    float* sM = sN + C * kMP;         // dP o Gam

    ChunkAt at;
    const int x = blockIdx.x, vh = blockIdx.y, rep = a.Hv / a.Hk, kh = vh / rep;
    if (!bwd::chunk_at(x, a.cu, a.ws.base, a.B, a.T, a.nc_dense, &at)) return;
    const int tid = threadIdx.x, lane = tid & 63, w = (tid >> 6) & 3, g = lane >> 4, n = lane & 15;
    const int p = __builtin_amdgcn_readfirstlane(tid >> 8), cn = 16 * NH * p + n;   // this lane's first column of dv
    const float* gK = a.ws.groups + ((size_t)x * a.Hk + kh) * a.sz.group();
    const float* gQ = gK + C * dkp;
    const float* head = a.ws.heads + ((size_t)x * a.Hv + vh) * a.sz.head();
    const float *gT = head, *gB = gT + C * C, *gP = gB + C * C, *gV = gP + C * C + 2 * C * dkp + C * dvp;
    const float* h = a.ws.h + ((size_t)x * a.Hv + vh) * a.sz.state();
    const float* dh = a.ws.dh + ((size_t)x * a.Hv + vh) * a.sz.state();
    const int ra = 16 * w + n;                // this lane's row as an A operand

    f32x4 kr[NK];                             // this lane's row of K
#pragma unroll
    for (int t = 0; t < NK; ++t) kr[t] = four(gK + ra * dkp + 16 * t + 4 * g);
    load_gates(a, at, vh, &sg);
    for (int e = tid; e < C * dvp; e += kGradThreads) {
        const int r = e / dvp, j = e % dvp;
        s2[r * vp + j] = r < at.rows && j < a.dv_
                             ? Elem<TG>::load(static_cast<const TG*>(a.dout) + ((at.row0 + r) * a.Hv + vh) * a.dv_ + j)
                             : 0.f;
    }
    // K h and K dh': the states through LDS
    f32x4 rG = {0, 0, 0, 0}, rB = {0, 0, 0, 0}, rY = {0, 0, 0, 0};
    f32x4 gkh[NH], ek[NH], u[NH], dx[NH], dd[NH];
    clear(gkh);
    clear(ek);
    clear(u);
    clear(dx);
    clear(dd);
    float part = 0.f;                         // <h, dh'>
    {
        // vectors of a state a thread holds (32 x 32 and 32 x 96: the last one not in every thread)
        constexpr int all = dkp * dvp / 4, per = (all + kGradThreads - 1) / kGradThreads;
        auto held = [&](int i) { return all % kGradThreads == 0 || tid + kGradThreads * i < all; };
        f32x4 hv[per];
#pragma unroll
        for (int i = 0; i < per; ++i) hv[i] = held(i) ? four(h + 4 * (tid + kGradThreads * i)) : f32x4{0, 0, 0, 0};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < per; ++i) {
                const int e = 4 * (tid + kGradThreads * i);
                if (!held(i)) break;
                f32x4* at_e = reinterpret_cast<f32x4*>(s3 + (e / dvp) * vp + e % dvp);
                if (half) {
                    const f32x4 o = *at_e;
#pragma unroll
                    for (int s = 0; s < 4; ++s) part = fmaf(o[s], hv[i][s], part);
                }
                *at_e = hv[i];
            }
            if (!half)
#pragma unroll
                for (int i = 0; i < per; ++i)
                    if (held(i)) hv[i] = four(dh + 4 * (tid + kGradThreads * i));
            __syncthreads();
            mm_tiles<dkp>(half ? ek : gkh, [&](int kb) { return kr[kb / 16]; },
                          [&](int j, int k) { return s3[k * vp + cn + 16 * j]; });
        }
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) part += __shfl_xor(part, o);
    if (lane == 0) s_sum[tid >> 6] = part;
    // this lane's row of T, and columns of T and P
    f32x4 tr[4], tc[4], pc[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        tr[t] = four(gT + ra * C + 16 * t + 4 * g);
        const float *ct = gT + (16 * t + 4 * g) * C + ra, *cp = gP + (16 * t + 4 * g) * C + ra;
        tc[t] = f32x4{ct[0], ct[C], ct[2 * C], ct[3 * C]};
        pc[t] = f32x4{cp[0], cp[C], cp[2 * C], cp[3 * C]};
    }
    // x = V - ga K h; ga K h and E K dh' stay in registers
#pragma unroll
    for (int j = 0; j < NH; ++j) {
        const int col = cn + 16 * j;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int r = 16 * w + 4 * g + s;
            gkh[j][s] *= sg.ga[r];
            ek[j][s] *= sg.E[r];
            s1[r * vp + col] = gV[r * dvp + col] - gkh[j][s];
        }
    }
    __syncthreads();
    // u = T x
    mm_tiles<C>(u, [&](int kb) { return tr[kb / 16]; }, [&](int j, int k) { return s1[k * vp + cn + 16 * j]; });
    // ddelta = P^T do + E K dh'
    mm_tiles<C>(dd, [&](int kb) { return pc[kb / 16]; }, [&](int j, int k) { return s2[k * vp + cn + 16 * j]; });
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NH; ++j)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int r = 16 * w + 4 * g + s;
            const float d = dd[j][s] + ek[j][s];
            rY[s] = fmaf(sg.beta[r] * u[j][s], ek[j][s], rY[s]);
            rB[s] = fmaf(d, u[j][s], rB[s]);
            s1[r * vp + cn + 16 * j] = u[j][s];
            s3[r * vp + cn + 16 * j] = sg.beta[r] * d;
        }
    __syncthreads();
    mm_tiles<C>(dx, [&](int kb) { return tc[kb / 16]; }, [&](int j, int k) { return s3[k * vp + cn + 16 * j]; });
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NH; ++j) {
        const int col = cn + 16 * j;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int r = 16 * w + 4 * g + s;
            s3[r * vp + col] = dx[j][s];
            rG[s] = fmaf(-dx[j][s], gkh[j][s], rG[s]);
            if (r < at.rows && col < a.dv_)
                Elem<TG>::store(static_cast<TG*>(a.dv) + ((at.row0 + r) * a.Hv + vh) * a.dv_ + col, dx[j][s]);
        }
    }
    __syncthreads();
    // Zu = dx u^T or do u^T on and below the diagonal: X, N or dP o Gam
    f32x4 rX = {0, 0, 0, 0}, z[4];
    clear(z);
    const float *sA = p ? s2 : s3, *gBP = p ? gP : gB;
    float* sNM = p ? sM : sN;
    mm_tiles<dvp>(z, [&](int kb) { return four(sA + ra * vp + kb + 4 * g); },
                  [&](int j, int k) { return s1[(16 * j + n) * vp + k]; });
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float cx = 0.f, cz = 0.f;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int r = 16 * w + 4 * g + s, c = 16 * j + n;
            float v = 0.f;
            if (p ? c <= r : c < r) {
                v = p ? z[j][s] * sg.beta[c] : -z[j][s] * sg.beta[c];
                if (c < r) {
                    const float b = gBP[r * C + c], X = v * b;
                    rX[s] += X;
                    cx += X;
                    cz = fmaf(b, z[j][s], cz);
                }
                v *= decay(sg, r, c);
            }
            sNM[r * kMP + c] = v;
        }
        cx += __shfl_xor(cx, 16); cx += __shfl_xor(cx, 32);
        cz += __shfl_xor(cz, 16); cz += __shfl_xor(cz, 32);
        if (g == 0) {
            s_colX[4 * p + w][16 * j + n] = cx;
            if (p == 0) s_colZ[w][16 * j + n] = cz;
        }
    }
    __syncthreads();

    // dq and dk, a tile of columns at a time: the rows of h and dh' that it needs
    // are fetched whole ahead of the products
    float* parts = a.ws.part + ((size_t)x * a.Hv + vh) * 2 * C * dkp;
    struct Cols {
        f32x4 h[NV], dh[NV];
        float k[16], q[16];
    } now, next;
    auto fetch = [&](Cols& c, int j) {
        const int col = 16 * j + n;
#pragma unroll
        for (int t = 0; t < NV; ++t) {
            c.h[t] = four(h + col * dvp + 16 * t + 4 * g);
            c.dh[t] = four(dh + col * dvp + 16 * t + 4 * g);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int k = 16 * (e >> 2) + 4 * g + (e & 3);
            c.k[e] = gK[k * dkp + col];
            c.q[e] = gQ[k * dkp + col];
        }
    };
    constexpr bool ahead = NV < 6;            // a wide tile's columns fill the registers once
    const int j0 = NK / 2 * p;
    if (ahead) fetch(now, j0);
    for (int j = j0; j < j0 + NK / 2; ++j) {
        const int col = 16 * j + n;
        if (!ahead) fetch(now, j);
        else fetch(next, min(j + 1, j0 + NK / 2 - 1));
        __builtin_amdgcn_sched_barrier(0);
        f32x4 dq = {0, 0, 0, 0}, dk = {0, 0, 0, 0}, dxh = {0, 0, 0, 0}, udh = {0, 0, 0, 0}, doh = {0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < NV; ++t) {
            const f32x4 o4 = four(s2 + ra * vp + 16 * t + 4 * g), x4 = four(s3 + ra * vp + 16 * t + 4 * g),
                        u4 = four(s1 + ra * vp + 16 * t + 4 * g);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                doh = mfma4(o4[s], now.h[t][s], doh);
                dxh = mfma4(x4[s], now.h[t][s], dxh);
                udh = mfma4(u4[s], now.dh[t][s], udh);
            }
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int k = 16 * (e >> 2) + 4 * g + (e & 3);
            dq = mfma4(sM[ra * kMP + k], now.k[e], dq);
            dk = mfma4(sM[k * kMP + ra], now.q[e], dk);
            dk = mfma4(sN[ra * kMP + k] + sN[k * kMP + ra], now.k[e], dk);
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int r = 16 * w + 4 * g + s;
            const float d = sg.ga[r] * doh[s];
            rG[s] = fmaf(d, gQ[r * dkp + col], rG[s]);
            const float q1 = dq[s] + d, k1 = dk[s] + sg.E[r] * sg.beta[r] * udh[s] - sg.ga[r] * dxh[s];
            if (rep > 1) {
                parts[r * dkp + col] = q1;
                parts[(C + r) * dkp + col] = k1;
            } else if (r < at.rows && col < a.dk_) {
                const int64_t o = ((at.row0 + r) * a.Hk + kh) * a.dk_ + col;
                Elem<TG>::store(static_cast<TG*>(a.dq) + o, q1);
                Elem<TG>::store(static_cast<TG*>(a.dk) + o, k1);
            }
        }
        if (ahead) now = next;
    }
    // row sums over the columns' 16 lanes
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const float G = sum16(rG[s] + rX[s]), Bt = sum16(rB[s]), Y = sum16(rY[s]);
        const int r = 16 * w + 4 * g + s;
        if (n == 0) {
            s_dG[p][r] = G - Y;
            s_db[p][r] = Bt;
            s_Y[p][r] = Y;
        }
    }
    __syncthreads();
    if (tid < C) {                            // one wave: column sums, the last row's terms, the running sum
        float cx = 0.f, cz = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) cx += s_colX[i][tid];
#pragma unroll
        for (int i = 0; i < 4; ++i) cz += s_colZ[i][tid];
        double d = (double)(s_dG[0][tid] + s_dG[1][tid]) - (double)cx;
        double Y = s_Y[0][tid] + s_Y[1][tid];
#pragma unroll
        for (int o = 32; o; o >>= 1) Y += __shfl_xor(Y, o);
        if (tid == C - 1) {
            double hd = 0.0;
#pragma unroll
            for (int i = 0; i < 8; ++i) hd += s_sum[i];
            d += Y + (double)sg.ga[C - 1] * hd;
        }
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const double up = __shfl_down(d, o);
            if (tid + o < 64) d += up;
        }
        if (tid < at.rows) {
            const int64_t r = (at.row0 + tid) * a.Hv + vh;
            Elem<TG>::store(static_cast<TG*>(a.dg) + r, (float)d);
            Elem<TG>::store(static_cast<TG*>(a.db) + r, s_db[0][tid] + s_db[1][tid] - cz);
        }
    }
}

// dq and dk of a k-head: its v-heads' parts, added in order.
template <typename TG>
__global__ void __launch_bounds__(kThreads)
gdn_backward_sum_kernel(Args a)
{
    ChunkAt at;
    const int x = blockIdx.x, kh = blockIdx.y, rep = a.Hv / a.Hk, dkp = a.sz.dkp;
    if (!bwd::chunk_at(x, a.cu, a.ws.base, a.B, a.T, a.nc_dense, &at)) return;
    const float* p = a.ws.part + ((size_t)x * a.Hv + (size_t)kh * rep) * 2 * C * dkp;
    // 16 rows of dq (z = 0 .. 3) or of dk (4 .. 7); a thread's row is tid / 16
    const int r = 16 * (blockIdx.z & 3) + (threadIdx.x >> 4);
    if (r >= at.rows) return;
    p += (size_t)(blockIdx.z >> 2) * C * dkp + r * dkp;
    TG* out = static_cast<TG*>(blockIdx.z < 4 ? a.dq : a.dk) + ((at.row0 + r) * a.Hk + kh) * a.dk_;
    for (int j = 4 * (threadIdx.x & 15); j < a.dk_; j += 64) {
        f32x4 t = four(p + j);
        for (int i = 1; i < rep; ++i) t += four(p + (size_t)i * 2 * C * dkp + j);
#pragma unroll
        for (int s = 0; s < 4; ++s)
            if (j + s < a.dk_) Elem<TG>::store(out + j + s, t[s]);
    }
}

int padded(int d) { return d <= 32 ? 32 : d <= 64 ? 64 : 128; }
Sizes sizes(int dk, int dv) { return Sizes{padded(dk), dv > 64 && dv <= 96 ? 96 : padded(dv)}; }

struct Layout {
    size_t base, heads, groups, h, dh, part, total;
};
Layout layout(const BackwardArgs& a)
{
    const Sizes sz = sizes(a.dk, a.dv);
    const size_t n = (size_t)bwd::max_chunks(a.B, a.T, a.cu != nullptr);
    Layout l;
    size_t at = 0;
    l.base = at; at += bwd::round_up(a.cu ? (size_t)(a.B + 1) * sizeof(int32_t) : 0);
    l.heads = at; at += bwd::round_up(n * a.Hv * sz.head() * sizeof(float));
    l.groups = at; at += bwd::round_up(n * a.Hk * sz.group() * sizeof(float));
    l.h = at; at += bwd::round_up(n * a.Hv * sz.state() * sizeof(float));
    l.dh = at; at += bwd::round_up(n * a.Hv * sz.state() * sizeof(float));
    l.part = at; at += bwd::round_up(a.Hv > a.Hk ? n * a.Hv * sz.group() * sizeof(float) : 0);
    l.total = at;
    return l;
}

size_t prep_lds(const Sizes& s)
{
    return (2 * (size_t)C * (s.dkp + 4) + (size_t)C * (s.dvp + 4) + 3 * (size_t)C * kMP) * sizeof(float);
}
size_t grads_lds(const Sizes& s)
{
    const size_t row = s.dvp + 4, tail = C * row + 2 * (size_t)C * kMP, state = s.dkp * row;
    return (2 * C * row + (tail > state ? tail : state)) * sizeof(float);
}
// 16-column tiles of dv that a spine workgroup walks: two, or one where twice the
// workgroups still find a compute unit each (2 x 500 tokens of 6 heads, 64 x 96:
// 31 us with two, 22 with one).  Either gives the same bits.
int spine_tiles(const Sizes& s, int Hv, int B) { return (int64_t)Hv * (s.dvp / 32) * B * 2 <= 128 ? 1 : 2; }

// The head sizes' tile counts as compile-time constants: 2, 4 or 8 of dk, whose
// state tiles the spine's four waves share out evenly, and also 6 of dv.
template <typename F>
hipError_t with_dk(int n, F&& f)
{
    if (n == 32) return f(std::integral_constant<int, 2>());
    if (n == 64) return f(std::integral_constant<int, 4>());
    return f(std::integral_constant<int, 8>());
}
template <typename F>
hipError_t with_dv(int n, F&& f)
{
    return n == 96 ? f(std::integral_constant<int, 6>()) : with_dk(n, f);
}

template <typename K>
hipError_t run(K kernel, dim3 grid, unsigned threads, size_t lds, hipStream_t s, const Args& k)
{
    const hipError_t e = lds > 0 ? allow_lds(reinterpret_cast<const void*>(kernel), lds) : hipSuccess;
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, grid, dim3(threads), lds, s, k);
    return hipGetLastError();
}

template <typename TA>
hipError_t launch_prep(const Args& k, unsigned chunks, hipStream_t s)
{
    return with_dk(k.sz.dkp, [&](auto nk) {
        return with_dv(k.sz.dvp, [&](auto nv) {
            return run(gdn_backward_prep_kernel<nk.value, nv.value, TA>, dim3(chunks, k.Hv), kThreads, prep_lds(k.sz), s, k);
        });
    });
}

template <typename TG>
hipError_t launch_walk(const Args& k, unsigned chunks, hipStream_t s)
{
    const int tiles = spine_tiles(k.sz, k.Hv, k.B), slices = k.sz.dvp / (16 * tiles);
    hipError_t e = with_dk(k.sz.dkp, [&](auto nk) {
        const dim3 grid(k.Hv * slices, k.B, 2);
        if (tiles == 1)
            hipLaunchKernelGGL((gdn_backward_spine_kernel<nk.value, 1, TG>), grid, dim3(kThreads), 0, s, k, slices);
        else
            hipLaunchKernelGGL((gdn_backward_spine_kernel<nk.value, 2, TG>), grid, dim3(kThreads), 0, s, k, slices);
        return hipGetLastError();
    });
    if (e != hipSuccess || chunks == 0) return e;
    e = with_dk(k.sz.dkp, [&](auto nk) {
        return with_dv(k.sz.dvp, [&](auto nv) {
            return run(gdn_backward_grads_kernel<nk.value, nv.value, TG>, dim3(chunks, k.Hv), kGradThreads, grads_lds(k.sz), s,
                       k);
        });
    });
    if (e != hipSuccess || k.Hv == k.Hk) return e;
    return run(gdn_backward_sum_kernel<TG>, dim3(chunks, k.Hk, 8), kThreads, 0, s, k);
}

}  // namespace

size_t backward_workspace_need(const BackwardArgs& a)
{
    // the generic route's, which a call of the MFMA route's types takes too where a
    // pointer is not aligned; at 128 x 128 it is the larger one (304 KiB and more a
    // chunk and v-head, the MFMA route's 138 KiB)
    return layout(a).total;
}

Geometry backward_generic_geometry(const BackwardArgs& a)
{
    const Sizes sz = sizes(a.dk, a.dv);
    return Geometry{"gdn_backward_prep_kernel+gdn_backward_spine_kernel+gdn_backward_grads_kernel",
                    {(unsigned)(a.Hv * (sz.dvp / (16 * spine_tiles(sz, a.Hv, a.B)))), (unsigned)a.B, 2}, kThreads, (unsigned)grads_lds(sz)};
}

hipError_t launch_backward_generic(const BackwardArgs& a, hipStream_t s)
{
    const Layout l = layout(a);
    unsigned char* w = static_cast<unsigned char*>(a.workspace);
    Args k{};
    k.q = a.q; k.k = a.k; k.v = a.v; k.dout = a.dout;
    k.q_exps = a.q_exps; k.k_exps = a.k_exps; k.v_exps = a.v_exps;
    k.log_g = a.log_g; k.beta = a.beta; k.h0 = a.h0; k.dht = a.dh_final;
    k.dq = a.dq; k.dk = a.dk_out; k.dv = a.dv_out; k.dg = a.dlog_g; k.db = a.dbeta; k.dh0 = a.dh0;
    k.B = a.B; k.T = a.T; k.Hk = a.Hk; k.Hv = a.Hv; k.dk_ = a.dk; k.dv_ = a.dv;
    k.cu = a.cu;
    k.nc_dense = a.T > 0 ? (a.T + C - 1) / C : 1;
    k.sz = sizes(a.dk, a.dv);
    k.ws = Ws{reinterpret_cast<int32_t*>(w + l.base), reinterpret_cast<float*>(w + l.heads),
              reinterpret_cast<float*>(w + l.groups), reinterpret_cast<float*>(w + l.h),
              reinterpret_cast<float*>(w + l.dh), reinterpret_cast<float*>(w + l.part)};
    const int64_t chunks = bwd::max_chunks(a.B, a.T, a.cu != nullptr);
    if (k.cu) {
        hipLaunchKernelGGL(gdn_backward_table_kernel, dim3(1), dim3(256), 0, s, k.cu, k.B, k.T, k.ws.base);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (chunks > 0) {
        const hipError_t e = a.io_dtype == 0   ? launch_prep<float>(k, (unsigned)chunks, s)
                             : a.io_dtype == 1 ? launch_prep<uint16_t>(k, (unsigned)chunks, s)
                                               : launch_prep<uint8_t>(k, (unsigned)chunks, s);
        if (e != hipSuccess) return e;
    }
    return a.grad_dtype == 0 ? launch_walk<float>(k, (unsigned)chunks, s) : launch_walk<uint16_t>(k, (unsigned)chunks, s);
}

}  // namespace gdn
