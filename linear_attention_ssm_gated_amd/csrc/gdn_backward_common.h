// What the two routes of the delta rule's backward pass share: the chunk
// table, the rows of a chunk and its gates.
//
// Notation, per chunk of C = 64 rows of one v-head, with start state h
// (dk x dv) and the gradient dh' of its end state; G the running sum of log_g
// in the chunk, ga_r = exp(G_r), E_s = exp(G_L - G_s), Gam_rs = exp(G_r - G_s):
//   B = strict_lower(Gam o K K^T),  P = lower(Gam o Q K^T)
//   T = (I + B diag(beta))^-1,  u = T (V - ga K h),  delta = beta u
//   o = ga Q h + P delta,  h' = ga_L h + K^T E delta
// (with beta on the right of B, beta = 0 needs no division anywhere).  With
//   W = E beta T (ga K),  U = E beta T V,  Qt = ga Q - P beta T (ga K)
// the states and their gradients walk the chunks by
//   h' = ga_L h + K^T (U - W h),   dh = ga_L dh' + Qt^T do - W^T (K dh')
// and each chunk's gradients follow from h and dh' alone:
//   ddelta = P^T do + E K dh',  dx = T^T (beta ddelta),  dv = dx
//   Zu = strict_lower(dx u^T),  dB = -Zu beta_s,  dP = lower(do u^T) beta_s
//   dq = ga (do h^T) + (dP o Gam) K
//   dk = E beta (u dh'^T) - ga (dx h^T) + (dP o Gam)^T Q + (N + N^T) K,  N = dB o Gam
//   dbeta_r = ddelta_r . u_r - sum_m B_mr Zu_mr
//   X = strict_lower(dB o B + dP o P),  Y_r = E_r delta_r . (K dh')_r
//   dG_r = ga_r q_r . (do h^T)_r - dx_r . (ga K h)_r - Y_r + sum_s X_rs - sum_m X_mr
//   dG_L += sum Y + ga_L <h, dh'>,   dlog_g_t = sum_{r >= t} dG_r
// A pair (r, s) enters dG_r and dG_s with the same X_rs, so that the running
// sum cancels what does not cross t exactly; the diagonal of P, which no decay
// touches, is left out of X for the same reason.
#pragma once

#include "gdn_train_internal.h"

namespace gdn {
namespace bwd {

constexpr int C = 64;

// Work item of this workgroup.  Workgroups go to the eight XCDs in turn, each
// with an L2 of its own; numbered like this, neighbouring items (which share
// rows of k, q and of the workspace) meet in one L2.
constexpr int kXcds = 8;
__device__ __forceinline__ int64_t xcd_item()
{
    const int64_t n = (int64_t)gridDim.x * gridDim.y * gridDim.z;
    const int64_t id = blockIdx.x + (int64_t)gridDim.x * (blockIdx.y + (int64_t)gridDim.y * blockIdx.z);
    const int64_t each = n / kXcds, more = n % kXcds, xcd = id % kXcds;
    return xcd * each + (xcd < more ? xcd : more) + id / kXcds;
}

struct ChunkAt {
    int b;          // sequence
    int c;          // chunk within it
    int64_t row0;   // first row of the chunk
    int rows;       // rows of the chunk, 1..64
};

// Rows of sequence b: [row0, row0 + len); offsets outside [0, T] are clamped
// into it, as in the forward pass.
__device__ __forceinline__ void seq_rows(const int32_t* cu, int b, int T, int64_t* row0, int64_t* len)
{
    if (cu) {
        const int64_t a = min(max((int64_t)cu[b], (int64_t)0), (int64_t)T);
        const int64_t e = min(max((int64_t)cu[b + 1], a), (int64_t)T);
        *row0 = a;
        *len = e - a;
    } else {
        *row0 = (int64_t)b * T;
        *len = T;
    }
}

// First chunk of each sequence, base[0 .. B] (one workgroup of 256 threads), at
// most the T / C + B chunks that sequences one behind the other have: offsets out
// of order can overlap, and their further chunks are left out (walk_chunks).
__device__ __forceinline__ void chunk_table(const int32_t* cu, int B, int T, int32_t* base, int32_t* part)
{
    const int tid = threadIdx.x;
    const int per = (B + 255) / 256;
    const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
    const int64_t most = (int64_t)T / C + B;
    int64_t s = 0;
    for (int b = b0; b < b1; ++b) {
        int64_t r0, len;
        seq_rows(cu, b, T, &r0, &len);
        s = min(s + (len + C - 1) / C, most);
    }
    part[tid] = (int32_t)s;
    __syncthreads();
    int64_t before = 0;
    for (int i = 0; i < tid; ++i) before += part[i];
    if (tid == 255) base[B] = (int32_t)min(before + part[255], most);
    s = min(before, most);
    for (int b = b0; b < b1; ++b) {
        base[b] = (int32_t)s;
        int64_t r0, len;
        seq_rows(cu, b, T, &r0, &len);
        s = min(s + (len + C - 1) / C, most);
    }
}

// Chunks of sequence b, len rows, that have a place in the workspace.
__device__ __forceinline__ int walk_chunks(const int32_t* cu, const int32_t* base, int b, int64_t len)
{
    const int n = (int)((len + C - 1) / C);
    return cu ? min(n, base[b + 1] - base[b]) : n;
}

// Chunk x of the call; false beyond the last one (packed grids are sized for
// the most chunks that B sequences of T rows can have).
__device__ __forceinline__ bool chunk_at(int x, const int32_t* cu, const int32_t* base, int B, int T,
                                         int nc_dense, ChunkAt* at)
{
    int b, c;
    if (!cu) {
        b = x / nc_dense;
        c = x % nc_dense;
    } else {
        if (x >= base[B]) return false;
        int lo = 0, hi = B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (base[mid] <= x) lo = mid; else hi = mid - 1;
        }
        b = lo;
        c = x - base[b];
    }
    int64_t row0, len;
    seq_rows(cu, b, T, &row0, &len);
    at->b = b;
    at->c = c;
    at->row0 = row0 + (int64_t)c * C;
    at->rows = (int)min((int64_t)C, len - (int64_t)c * C);
    return true;
}

// Most chunks of a call.
inline int64_t max_chunks(int B, int T, bool packed)
{
    return packed ? (int64_t)T / C + B : (int64_t)B * ((T + C - 1) / C);
}

// T = (I + B diag(beta))^-1 in fp32, by 16 x 16 blocks, 256 threads.  B's lower
// part is in LDS at sB (pitch kBP floats), sD takes the diagonal blocks (4 x 16 x
// 17 floats).  solve_diagonal is one wave's: lane (g, n) forms column n of block g
// by forward substitution.  After a barrier solve_column gives wave w the blocks
// T_iw as accumulators (rows 16 i + 4 g + s of column 16 w + n, zero above the
// diagonal): T_iw = -T_ii sum_{m = w}^{i-1} B_im beta_m T_mw on fp32 MFMA
// (16x16x4), k of step s being 4 g + s, so that an accumulator is the next
// product's right operand as it is.
constexpr int kBP = 68;
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4 mfma4(float a, float b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ void solve_diagonal(const float* sB, const float* sBt, float* sD)
{
    const int lane = threadIdx.x & 63, g = lane >> 4, n = lane & 15;
    const float* blk = sB + (16 * g) * kBP + 16 * g;
    f32x4 br[16][4], bt[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) bt[m] = *reinterpret_cast<const f32x4*>(sBt + 16 * g + 4 * m);
#pragma unroll
    for (int r = 1; r < 16; ++r)
#pragma unroll
        for (int m = 0; m < 4; ++m)
            if (4 * m < r) br[r][m] = *reinterpret_cast<const f32x4*>(blk + r * kBP + 4 * m);
    __builtin_amdgcn_sched_barrier(0);
    float t[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) t[r] = r == n ? 1.f : 0.f;
#pragma unroll
    for (int m = 0; m < 15; ++m) {
        const float f = bt[m >> 2][m & 3] * t[m];
#pragma unroll
        for (int r = m + 1; r < 16; ++r) t[r] = fmaf(-br[r][m >> 2][m & 3], f, t[r]);
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) sD[(16 * g + r) * 17 + n] = t[r];
}

__device__ __forceinline__ void solve_column(const float* sB, const float* sBt, const float* sD, int w, f32x4 (&Tc)[4])
{
    const int lane = threadIdx.x & 63, g = lane >> 4, n = lane & 15;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        Tc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (i == w) {
#pragma unroll
            for (int s = 0; s < 4; ++s) Tc[i][s] = sD[(16 * i + 4 * g + s) * 17 + n];
        } else if (i > w) {
            f32x4 M = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int m = 0; m < i; ++m)
                if (m >= w) {
                    const f32x4 b = *reinterpret_cast<const f32x4*>(sB + (16 * i + n) * kBP + 16 * m + 4 * g);
                    const f32x4 bt = *reinterpret_cast<const f32x4*>(sBt + 16 * m + 4 * g);
#pragma unroll
                    for (int s = 0; s < 4; ++s) M = mfma4(b[s] * bt[s], Tc[m][s], M);
                }
            f32x4 t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < 4; ++s) t = mfma4(sD[(16 * i + n) * 17 + 4 * g + s], M[s], t);
            Tc[i] = -t;
        }
    }
}

// A workgroup barrier that orders LDS alone: __syncthreads would also wait for
// every global load and store in flight.
__device__ __forceinline__ void lds_barrier()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

inline size_t round_up(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace bwd
}  // namespace gdn
