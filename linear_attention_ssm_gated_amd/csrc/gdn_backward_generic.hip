// Generic backward pass of the gated delta rule: fp32 arithmetic on fp32, bf16
// or 8-bit inputs, any dk, dv <= 128.  The formulas are in
// gdn_backward_common.h.  Three kernels:
//   prep    one workgroup per (chunk, v-head): B, P, T, W, U, Qt
//   spine   one workgroup per (sequence, v-head, 32 dv columns, direction): the
//           states walked forwards and their gradients backwards, both in the
//           same launch, every chunk's start state and end gradient written
//   grads   one workgroup per (chunk, k-head): the chunk's gradients, the
//           v-heads of the k-head in turn, dq and dk summed in registers
// Products run on fp32 MFMA (16x16x4: exact fp32 operands); the chunk's running
// sums of log_g and their differences are fp64, since a difference of two large
// sums would lose the decay's digits.  Head sizes are padded with zeros to
// multiples of 16 in the workspace.
#include "gdn_backward_common.h"

namespace gdn {
namespace {

using bwd::C;
using bwd::ChunkAt;

constexpr int kThreads = 256;
constexpr int kMaxTiles = 8;        // 16-wide tiles of a padded head size
constexpr int kMP = C + 4;          // pitch of a 64 x 64 matrix in LDS
constexpr int kCols = 32;           // dv columns of a spine workgroup
constexpr int kSP = kCols + 4;

typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4 mfma4(float a, float b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// acc += A (16 x K) B (K x 16) for one tile: lane (g, n) = (lane / 16, lane %
// 16) supplies A[n][k] and B[k][n] with k = 16 kb + 4 g + s at step s (any
// order of k is one sum), and holds rows 4g .. 4g + 3 of column n.  Row and k
// strides are in elements; the pointers may be LDS or global.
template <typename FA, typename FB>
__device__ __forceinline__ void mm(f32x4& acc, int K, FA&& a, FB&& b)
{
    const int g = (threadIdx.x & 63) >> 4;
    for (int kb = 0; kb < K; kb += 16) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int k = kb + 4 * g + s;
            acc = mfma4(a(k), b(k), acc);
        }
    }
}

// Workspace of one (chunk, v-head) and of one (chunk, k-head), in floats.
struct Sizes {
    int dkp, dvp;
    __host__ __device__ size_t mats() const { return 3 * (size_t)C * C; }                  // T, B, P
    __host__ __device__ size_t head() const { return mats() + 2 * (size_t)C * dkp + (size_t)C * dvp + 2 * C; }   // + W, Qt, U, G
    __host__ __device__ size_t state() const { return (size_t)dkp * dvp; }
    __host__ __device__ size_t group() const { return 2 * (size_t)C * dkp; }               // K, Q
};

struct Ws {
    int32_t* base;     // chunk table (packed)
    float* heads;      // [chunk][Hv] head()
    float* groups;     // [chunk][Hk] group()
    float* h;          // [chunk][Hv] start states
    float* dh;         // [chunk][Hv] end gradients
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
struct Gates {
    double G[C];
    float beta[C], ga[C], E[C];
};
__device__ __forceinline__ void load_gates(const Args& a, const ChunkAt& at, int vh, Gates* s)
{
    const int tid = threadIdx.x;
    if (tid < C) {
        const bool live = tid < at.rows;
        const int64_t r = (at.row0 + tid) * a.Hv + vh;
        s->G[tid] = live ? (double)a.log_g[r] : 0.0;
        s->beta[tid] = live ? a.beta[r] : 0.f;
    }
    __syncthreads();
    if (tid == 0) {
        double acc = 0.0;
        for (int r = 0; r < C; ++r) { acc += s->G[r]; s->G[r] = acc; }
    }
    __syncthreads();
    if (tid < C) {
        s->ga[tid] = (float)exp(s->G[tid]);
        s->E[tid] = (float)exp(s->G[C - 1] - s->G[tid]);
    }
    __syncthreads();
}
__device__ __forceinline__ float decay(const Gates& s, int r, int c) { return expf((float)(s.G[r] - s.G[c])); }

// ---- prep ----------------------------------------------------------------------
extern __shared__ __attribute__((aligned(16))) float lds_dyn[];

template <typename TA>
__global__ void __launch_bounds__(kThreads)
gdn_backward_prep_kernel(Args a)
{
    __shared__ Gates sg;
    const int dkp = a.sz.dkp, dvp = a.sz.dvp, dp = dkp + 4;
    float* sK = lds_dyn;              // [C][dp]
    float* sQ = sK + C * dp;          // [C][dp], then T (ga K)
    float* sB = sQ + C * dp;          // [C][kMP]
    float* sP = sB + C * kMP;
    float* sT = sP + C * kMP;

    ChunkAt at;
    const int x = blockIdx.x, vh = blockIdx.y, kh = vh / (a.Hv / a.Hk);
    if (!bwd::chunk_at(x, a.cu, a.ws.base, a.B, a.T, a.nc_dense, &at)) return;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, g = lane >> 4, n = lane & 15;
    float* head = a.ws.heads + ((size_t)x * a.Hv + vh) * a.sz.head();
    float *gT = head, *gB = gT + C * C, *gP = gB + C * C, *gW = gP + C * C, *gQt = gW + C * dkp,
          *gU = gQt + C * dkp, *gG = gU + C * dvp;
    float* gK = a.ws.groups + ((size_t)x * a.Hk + kh) * a.sz.group();

    for (int e = tid; e < C * dkp; e += kThreads) {
        const int r = e / dkp, j = e % dkp;
        const bool live = r < at.rows && j < a.dk_;
        const int64_t row = (at.row0 + r) * a.Hk + kh;
        sK[r * dp + j] = live ? act<TA>(a.k, a.k_exps, row, a.dk_, j) : 0.f;
        sQ[r * dp + j] = live ? act<TA>(a.q, a.q_exps, row, a.dk_, j) : 0.f;
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
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f32x4 kk = {0, 0, 0, 0}, qk = {0, 0, 0, 0};
        if (j <= w) {
            mm(kk, dkp, [&](int k) { return sK[(16 * w + n) * dp + k]; }, [&](int k) { return sK[(16 * j + n) * dp + k]; });
            mm(qk, dkp, [&](int k) { return sQ[(16 * w + n) * dp + k]; }, [&](int k) { return sK[(16 * j + n) * dp + k]; });
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int r = 16 * w + 4 * g + s, c = 16 * j + n;
            const float e = c <= r ? decay(sg, r, c) : 0.f;
            const float bv = c < r ? e * kk[s] : 0.f, pv = c <= r ? e * qk[s] : 0.f;
            sB[r * kMP + c] = bv;
            sP[r * kMP + c] = pv;
            gB[r * C + c] = bv;
            gP[r * C + c] = pv;
        }
    }
    __syncthreads();

    // T = (I + B diag(beta))^-1: thread c forms column c; once t_m is final it
    // is taken out of every later row
    if (tid < C) {
        float t[C];
#pragma unroll
        for (int r = 0; r < C; ++r) t[r] = r == tid ? 1.f : 0.f;
#pragma unroll
        for (int m = 0; m < C - 1; ++m) {
            const float f = sg.beta[m] * t[m];
#pragma unroll
            for (int r = m + 1; r < C; ++r) t[r] = fmaf(-sB[r * kMP + m], f, t[r]);
        }
#pragma unroll
        for (int r = 0; r < C; ++r) sT[r * kMP + tid] = t[r];
    }
    __syncthreads();
    for (int e = tid; e < C * C; e += kThreads) gT[e] = sT[(e >> 6) * kMP + (e & 63)];

    // Z = T (ga K), W = E beta Z
    f32x4 z[kMaxTiles];
#pragma unroll
    for (int j = 0; j < kMaxTiles; ++j) {
        z[j] = f32x4{0, 0, 0, 0};
        if (16 * j < dkp)
            mm(z[j], C, [&](int k) { return sT[(16 * w + n) * kMP + k]; },
               [&](int k) { return sg.ga[k] * sK[k * dp + 16 * j + n]; });
    }
    // U = E beta T V
    for (int j = 0; j < dvp / 16; ++j) {
        f32x4 u = {0, 0, 0, 0};
        const int col = 16 * j + n;
        mm(u, C, [&](int k) { return sT[(16 * w + n) * kMP + k]; },
           [&](int k) {
               return k < at.rows && col < a.dv_ ? act<TA>(a.v, a.v_exps, (at.row0 + k) * a.Hv + vh, a.dv_, col) : 0.f;
           });
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int r = 16 * w + 4 * g + s;
            gU[r * dvp + col] = sg.E[r] * sg.beta[r] * u[s];
        }
    }
    // Q to registers, then Z in its place as the operand of P beta Z
    f32x4 qv[kMaxTiles];
#pragma unroll
    for (int j = 0; j < kMaxTiles; ++j)
        if (16 * j < dkp)
#pragma unroll
            for (int s = 0; s < 4; ++s) qv[j][s] = sQ[(16 * w + 4 * g + s) * dp + 16 * j + n];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kMaxTiles; ++j)
        if (16 * j < dkp)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int r = 16 * w + 4 * g + s;
                gW[r * dkp + 16 * j + n] = sg.E[r] * sg.beta[r] * z[j][s];
                sQ[r * dp + 16 * j + n] = sg.beta[r] * z[j][s];
            }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kMaxTiles; ++j)
        if (16 * j < dkp) {
            f32x4 t = {0, 0, 0, 0};
            mm(t, C, [&](int k) { return sP[(16 * w + n) * kMP + k]; }, [&](int k) { return sQ[k * dp + 16 * j + n]; });
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int r = 16 * w + 4 * g + s;
                gQt[r * dkp + 16 * j + n] = sg.ga[r] * qv[j][s] - t[s];
            }
        }
}

// ---- spine -----------------------------------------------------------------------
// grid (Hv * column slices, B, 2): z = 0 walks the states, z = 1 their gradients.
template <typename TG>
__global__ void __launch_bounds__(kThreads)
gdn_backward_spine_kernel(Args a, int slices)
{
    __shared__ float sS[kMaxTiles * 16][kSP];   // the state's columns
    __shared__ float sD[C][kSP];                // U - W h, or K dh'
    __shared__ float sO[C][kSP];                // do
    const int dkp = a.sz.dkp, dvp = a.sz.dvp;
    const int vh = blockIdx.x / slices, col0 = (blockIdx.x % slices) * kCols, b = blockIdx.y;
    const int kh = vh / (a.Hv / a.Hk);
    const bool rev = blockIdx.z == 1;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, g = lane >> 4, n = lane & 15;
    const int nkt = dkp / 16, nct = min(2, (dvp - col0) / 16);

    int64_t row0, len;
    bwd::seq_rows(a.cu, b, a.T, &row0, &len);
    const int nc = (int)((len + C - 1) / C);
    const int64_t x0 = a.cu ? a.ws.base[b] : (int64_t)b * a.nc_dense;
    const float* from = rev ? a.dht : a.h0;
    const size_t hoff = ((size_t)b * a.Hv + vh) * a.dk_ * a.dv_;

    // wave w holds state rows of tiles w and w + 4, both column tiles
    f32x4 st[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int r = 16 * (w + 4 * i) + 4 * g + s, c = col0 + 16 * j + n;
                st[i][j][s] = from && r < a.dk_ && c < a.dv_ ? from[hoff + (size_t)r * a.dv_ + c] : 0.f;
            }

    for (int i0 = 0; i0 < nc; ++i0) {
        const int c = rev ? nc - 1 - i0 : i0;
        const size_t x = x0 + c;
        const float* head = a.ws.heads + (x * a.Hv + vh) * a.sz.head();
        const float *gW = head + a.sz.mats(), *gQt = gW + C * dkp, *gU = gQt + C * dkp;
        const double* gG = reinterpret_cast<const double*>(gU + C * dvp);
        const float* gK = a.ws.groups + (x * a.Hk + kh) * a.sz.group();
        float* out = (rev ? a.ws.dh : a.ws.h) + (x * a.Hv + vh) * a.sz.state();
        const float gL = (float)exp(gG[C - 1]);

        __syncthreads();   // the step before has read sS and sD
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (w + 4 * i < nkt && j < nct)
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const int r = 16 * (w + 4 * i) + 4 * g + s;
                        sS[r][16 * j + n] = st[i][j][s];
                        out[(size_t)r * dvp + col0 + 16 * j + n] = st[i][j][s];
                    }
        if (rev)
            for (int e = tid; e < C * kCols; e += kThreads) {
                const int r = e / kCols, j = e % kCols;
                const int64_t row = row0 + (int64_t)c * C + r;
                sO[r][j] = row < row0 + len && col0 + j < a.dv_
                               ? Elem<TG>::load(static_cast<const TG*>(a.dout) + (row * a.Hv + vh) * a.dv_ + col0 + j)
                               : 0.f;
            }
        __syncthreads();
        // rows 16 w .. + 15 of W h (of K dh')
        const float* left = rev ? gK : gW;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (j < nct) {
                f32x4 t = {0, 0, 0, 0};
                mm(t, dkp, [&](int k) { return left[(16 * w + n) * dkp + k]; }, [&](int k) { return sS[k][16 * j + n]; });
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int r = 16 * w + 4 * g + s;
                    sD[r][16 * j + n] = rev ? -t[s] : gU[r * dvp + col0 + 16 * j + n] - t[s];
                }
            }
        __syncthreads();
        const float* right = rev ? gW : gK;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (w + 4 * i < nkt)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (j < nct) {
                        f32x4 t = st[i][j] * gL;
                        const int m = 16 * (w + 4 * i) + n;
                        mm(t, C, [&](int k) { return right[k * dkp + m]; }, [&](int k) { return sD[k][16 * j + n]; });
                        if (rev)
                            mm(t, C, [&](int k) { return gQt[k * dkp + m]; }, [&](int k) { return sO[k][16 * j + n]; });
                        st[i][j] = t;
                    }
    }
    if (rev && a.dh0)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int r = 16 * (w + 4 * i) + 4 * g + s, c = col0 + 16 * j + n;
                    if (r < a.dk_ && c < a.dv_) a.dh0[hoff + (size_t)r * a.dv_ + c] = st[i][j][s];
                }
}

// ---- grads -----------------------------------------------------------------------
// sum over the 16 lanes of a row's columns
__device__ __forceinline__ float sum16(float x)
{
#pragma unroll
    for (int o = 8; o; o >>= 1) x += __shfl_xor(x, o);
    return x;
}

template <typename TA, typename TG>
__global__ void __launch_bounds__(kThreads)
gdn_backward_grads_kernel(Args a)
{
    __shared__ Gates sg;
    __shared__ float s_dG[C], s_db[C];        // row sums, later with the column sums
    __shared__ float s_colX[4][C], s_colZ[4][C];
    __shared__ float s_sum[8];
    const int dkp = a.sz.dkp, dvp = a.sz.dvp, vp = dvp + 4;
    float* s1 = lds_dyn;              // x, then u           [C][vp]
    float* s2 = s1 + C * vp;          // do
    float* s3 = s2 + C * vp;          // beta ddelta, then dx
    float* sN = s3 + C * vp;          // N  [C][kMP]
    float* sM = sN + C * kMP;         // dP o Gam

    ChunkAt at;
    const int x = blockIdx.x, kh = blockIdx.y, rep = a.Hv / a.Hk;
    if (!bwd::chunk_at(x, a.cu, a.ws.base, a.B, a.T, a.nc_dense, &at)) return;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, g = lane >> 4, n = lane & 15;
    const float* gK = a.ws.groups + ((size_t)x * a.Hk + kh) * a.sz.group();
    const float* gQ = gK + C * dkp;
    const int ra = 16 * w + n;                // this lane's row as an A operand
    f32x4 dq[kMaxTiles], dk[kMaxTiles];
#pragma unroll
    for (int j = 0; j < kMaxTiles; ++j) dq[j] = dk[j] = f32x4{0, 0, 0, 0};

    for (int vh = kh * rep; vh < (kh + 1) * rep; ++vh) {
        const float* head = a.ws.heads + ((size_t)x * a.Hv + vh) * a.sz.head();
        const float *gT = head, *gB = gT + C * C, *gP = gB + C * C;
        const float* h = a.ws.h + ((size_t)x * a.Hv + vh) * a.sz.state();
        const float* dh = a.ws.dh + ((size_t)x * a.Hv + vh) * a.sz.state();
        __syncthreads();                      // the v-head before has read the LDS
        load_gates(a, at, vh, &sg);
        for (int e = tid; e < C * dvp; e += kThreads) {
            const int r = e / dvp, j = e % dvp;
            s2[r * vp + j] = r < at.rows && j < a.dv_
                                 ? Elem<TG>::load(static_cast<const TG*>(a.dout) + ((at.row0 + r) * a.Hv + vh) * a.dv_ + j)
                                 : 0.f;
        }
        float part = 0.f;                     // <h, dh'>
        for (int e = tid; e < dkp * dvp; e += kThreads) part = fmaf(h[e], dh[e], part);
#pragma unroll
        for (int o = 32; o; o >>= 1) part += __shfl_xor(part, o);
        if (lane == 0) s_sum[w] = part;

        // x = V - ga K h; ga K h stays in registers
        f32x4 gkh[kMaxTiles], u[kMaxTiles];
        f32x4 rG = {0, 0, 0, 0}, rB = {0, 0, 0, 0}, rY = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < kMaxTiles; ++j)
            if (16 * j < dvp) {
                f32x4 t = {0, 0, 0, 0};
                mm(t, dkp, [&](int k) { return gK[ra * dkp + k]; }, [&](int k) { return h[k * dvp + 16 * j + n]; });
                const int col = 16 * j + n;
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int r = 16 * w + 4 * g + s;
                    gkh[j][s] = sg.ga[r] * t[s];
                    const float v = r < at.rows && col < a.dv_ ? act<TA>(a.v, a.v_exps, (at.row0 + r) * a.Hv + vh, a.dv_, col) : 0.f;
                    s1[r * vp + col] = v - gkh[j][s];
                }
            }
        __syncthreads();
        // u = T x
#pragma unroll
        for (int j = 0; j < kMaxTiles; ++j)
            if (16 * j < dvp) {
                u[j] = f32x4{0, 0, 0, 0};
                mm(u[j], C, [&](int k) { return gT[ra * C + k]; }, [&](int k) { return s1[k * vp + 16 * j + n]; });
            }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kMaxTiles; ++j)
            if (16 * j < dvp) {
                // ddelta = P^T do + E K dh'
                f32x4 kdh = {0, 0, 0, 0}, dd = {0, 0, 0, 0};
                mm(kdh, dkp, [&](int k) { return gK[ra * dkp + k]; }, [&](int k) { return dh[k * dvp + 16 * j + n]; });
                mm(dd, C, [&](int k) { return gP[k * C + ra]; }, [&](int k) { return s2[k * vp + 16 * j + n]; });
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int r = 16 * w + 4 * g + s;
                    const float ek = sg.E[r] * kdh[s];
                    const float d = dd[s] + ek;
                    rY[s] = fmaf(sg.beta[r] * u[j][s], ek, rY[s]);
                    rB[s] = fmaf(d, u[j][s], rB[s]);
                    s1[r * vp + 16 * j + n] = u[j][s];
                    s3[r * vp + 16 * j + n] = sg.beta[r] * d;
                }
            }
        __syncthreads();
        f32x4 dx[kMaxTiles];
#pragma unroll
        for (int j = 0; j < kMaxTiles; ++j)
            if (16 * j < dvp) {
                dx[j] = f32x4{0, 0, 0, 0};
                mm(dx[j], C, [&](int k) { return gT[k * C + ra]; }, [&](int k) { return s3[k * vp + 16 * j + n]; });
            }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kMaxTiles; ++j)
            if (16 * j < dvp) {
                const int col = 16 * j + n;
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
        // Zu = dx u^T and do u^T on and below the diagonal: X, N, dP o Gam
        f32x4 rX = {0, 0, 0, 0};
        float cX[4], cZ[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f32x4 zu = {0, 0, 0, 0}, du = {0, 0, 0, 0};
            if (j <= w) {
                mm(zu, dvp, [&](int k) { return s3[ra * vp + k]; }, [&](int k) { return s1[(16 * j + n) * vp + k]; });
                mm(du, dvp, [&](int k) { return s2[ra * vp + k]; }, [&](int k) { return s1[(16 * j + n) * vp + k]; });
            }
            float cx = 0.f, cz = 0.f;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int r = 16 * w + 4 * g + s, c = 16 * j + n;
                float nv = 0.f, mv = 0.f;
                if (c <= r) {
                    const float e = decay(sg, r, c), bt = sg.beta[c];
                    mv = du[s] * bt;
                    if (c < r) {
                        const float bb = gB[r * C + c];
                        nv = -zu[s] * bt;
                        const float X = nv * bb + mv * gP[r * C + c];
                        rX[s] += X;
                        cx += X;
                        cz = fmaf(bb, zu[s], cz);
                        nv *= e;
                    }
                    mv *= e;
                }
                sN[r * kMP + c] = nv;
                sM[r * kMP + c] = mv;
            }
            cx += __shfl_xor(cx, 16); cx += __shfl_xor(cx, 32);
            cz += __shfl_xor(cz, 16); cz += __shfl_xor(cz, 32);
            cX[j] = cx;
            cZ[j] = cz;
        }
        if (g == 0)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s_colX[w][16 * j + n] = cX[j];
                s_colZ[w][16 * j + n] = cZ[j];
            }
        __syncthreads();

        // dq, dk of this v-head
#pragma unroll
        for (int j = 0; j < kMaxTiles; ++j)
            if (16 * j < dkp) {
                const int col = 16 * j + n;
                f32x4 dohT = {0, 0, 0, 0}, dxh = {0, 0, 0, 0}, udh = {0, 0, 0, 0};
                mm(dohT, dvp, [&](int k) { return s2[ra * vp + k]; }, [&](int k) { return h[col * dvp + k]; });
                mm(dxh, dvp, [&](int k) { return s3[ra * vp + k]; }, [&](int k) { return h[col * dvp + k]; });
                mm(udh, dvp, [&](int k) { return s1[ra * vp + k]; }, [&](int k) { return dh[col * dvp + k]; });
                mm(dq[j], C, [&](int k) { return sM[ra * kMP + k]; }, [&](int k) { return gK[k * dkp + col]; });
                mm(dk[j], C, [&](int k) { return sM[k * kMP + ra]; }, [&](int k) { return gQ[k * dkp + col]; });
                mm(dk[j], C, [&](int k) { return sN[ra * kMP + k] + sN[k * kMP + ra]; }, [&](int k) { return gK[k * dkp + col]; });
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int r = 16 * w + 4 * g + s;
                    const float d = sg.ga[r] * dohT[s];
                    rG[s] = fmaf(d, gQ[r * dkp + col], rG[s]);
                    dq[j][s] += d;
                    dk[j][s] += sg.E[r] * sg.beta[r] * udh[s] - sg.ga[r] * dxh[s];
                }
            }
        // row sums over the columns' 16 lanes
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const float G = sum16(rG[s] + rX[s]), Bt = sum16(rB[s]), Y = sum16(rY[s]);
            const int r = 16 * w + 4 * g + s;
            if (n == 0) {
                s_dG[r] = G - Y;
                s_db[r] = Bt;
                sg.E[r] = Y;                  // E is not used again
            }
        }
        __syncthreads();
        if (tid < C) {                        // one wave: column sums, the last row's terms, the running sum
            float cx = 0.f, cz = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) { cx += s_colX[i][tid]; cz += s_colZ[i][tid]; }
            double d = (double)s_dG[tid] - (double)cx;
            double Y = sg.E[tid];
#pragma unroll
            for (int o = 32; o; o >>= 1) Y += __shfl_xor(Y, o);
            if (tid == C - 1) {
                const double hd = (double)s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3];
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
                Elem<TG>::store(static_cast<TG*>(a.db) + r, s_db[tid] - cz);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kMaxTiles; ++j)
        if (16 * j < dkp) {
            const int col = 16 * j + n;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int r = 16 * w + 4 * g + s;
                if (r < at.rows && col < a.dk_) {
                    const int64_t o = ((at.row0 + r) * a.Hk + kh) * a.dk_ + col;
                    Elem<TG>::store(static_cast<TG*>(a.dq) + o, dq[j][s]);
                    Elem<TG>::store(static_cast<TG*>(a.dk) + o, dk[j][s]);
                }
            }
        }
}

Sizes sizes(int dk, int dv) { return Sizes{(dk + 15) / 16 * 16, (dv + 15) / 16 * 16}; }

struct Layout {
    size_t base, heads, groups, h, dh, total;
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
    l.total = at;
    return l;
}

size_t prep_lds(const Sizes& s) { return (2 * (size_t)C * (s.dkp + 4) + 3 * (size_t)C * kMP) * sizeof(float); }
size_t grads_lds(const Sizes& s) { return (3 * (size_t)C * (s.dvp + 4) + 2 * (size_t)C * kMP) * sizeof(float); }
int slices_of(const Sizes& s) { return (s.dvp + kCols - 1) / kCols; }

template <typename K>
hipError_t allow_lds(K kernel, size_t bytes)
{
    return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename TA, typename TG>
hipError_t launch_typed(const Args& k, int64_t chunks, hipStream_t s)
{
    hipError_t e;
    const size_t lp = prep_lds(k.sz), lg = grads_lds(k.sz);
    if ((e = allow_lds(gdn_backward_prep_kernel<TA>, lp)) != hipSuccess) return e;
    if ((e = allow_lds(gdn_backward_grads_kernel<TA, TG>, lg)) != hipSuccess) return e;
    if (k.cu)
        hipLaunchKernelGGL(gdn_backward_table_kernel, dim3(1), dim3(256), 0, s, k.cu, k.B, k.T, k.ws.base);
    if (chunks > 0)
        hipLaunchKernelGGL((gdn_backward_prep_kernel<TA>), dim3((unsigned)chunks, k.Hv), dim3(kThreads), lp, s, k);
    const int slices = slices_of(k.sz);
    hipLaunchKernelGGL((gdn_backward_spine_kernel<TG>), dim3(k.Hv * slices, k.B, 2), dim3(kThreads), 0, s, k, slices);
    if (chunks > 0)
        hipLaunchKernelGGL((gdn_backward_grads_kernel<TA, TG>), dim3((unsigned)chunks, k.Hk), dim3(kThreads), lg, s, k);
    return hipGetLastError();
}

template <typename TA>
hipError_t launch_act(const Args& k, int grad, int64_t chunks, hipStream_t s)
{
    return grad == 0 ? launch_typed<TA, float>(k, chunks, s) : launch_typed<TA, uint16_t>(k, chunks, s);
}

}  // namespace

size_t backward_generic_workspace_bytes(const BackwardArgs& a) { return layout(a).total; }

size_t backward_workspace_need(const BackwardArgs& a)
{
    // the generic route's is the larger one, and an unaligned call of the MFMA
    // route's types falls back to it
    return backward_generic_workspace_bytes(a);
}

Geometry backward_generic_geometry(const BackwardArgs& a)
{
    const Sizes sz = sizes(a.dk, a.dv);
    return Geometry{"gdn_backward_prep_kernel+gdn_backward_spine_kernel+gdn_backward_grads_kernel",
                    {(unsigned)(a.Hv * slices_of(sz)), (unsigned)a.B, 2}, kThreads, (unsigned)grads_lds(sz)};
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
              reinterpret_cast<float*>(w + l.dh)};
    const int64_t chunks = bwd::max_chunks(a.B, a.T, a.cu != nullptr);
    if (a.io_dtype == 0) return launch_act<float>(k, a.grad_dtype, chunks, s);
    if (a.io_dtype == 1) return launch_act<uint16_t>(k, a.grad_dtype, chunks, s);
    return launch_act<uint8_t>(k, a.grad_dtype, chunks, s);
}

}  // namespace gdn
