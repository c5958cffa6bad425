// bf16 MFMA backward pass of the gated delta rule for dk = dv = 128 (gfx950):
// bf16 or 8-bit q, k, v and bf16 gradients, fp32 accumulation, states in fp32.
// The formulas are in gdn_backward_common.h.  Three kernels:
//   prep    one workgroup per (chunk, v-head): B, P, T; W, U, Qt
//   spine   one workgroup per (sequence, v-head, 64 dv columns, direction):
//           the states forwards and their gradients backwards in one launch
//   grads   one workgroup per (chunk, k-head): the gradients of the chunk, the
//           v-heads of the k-head in turn, dq and dk summed in registers (short
//           calls: one per v-head, and a sum over the k-head's)
// 4576 tokens of 16 / 48 heads in bf16 take 466 us back to back (traced, which slows
// each kernel a little: prep 91 to 92, spine 159, grads 231 to 233), where the inputs and gradients
// alone would take 48 us at a large copy's rate and the products 64 us at a large
// matrix product's; the generic route takes 2.8 ms.  The matrices that the three hand
// on set a floor of their own: 1482 MB moved, 288 us at a copy's rate.
// Matrices are rounded to bf16 where a product takes them (T, P, W, U, Qt; h and dh',
// which the gradients read as such; u, dx and the masked products), as the matrix units
// need; the walked states, sums, gates and statistics stay fp32.  Of an error of 3.3e-3
// in the 2-norm the outputs' own rounding is 1.7e-3; P, x = V - ga K h, u, beta ddelta
// and dP o Gam add 1.2e-3 to 1.7e-3 each to the gradients behind them, all others under
// 6e-4 (each rounded alone in 64 bits).  dlog_g's sums take B, P, h and dh' as rounded:
// fp32 copies of h and dh' beside the bf16 ones would move 906 MB more for 5e-4 of it.
//
// Operands.  v_mfma_f32_16x16x32_bf16: lane 16 g + n supplies A[n][8g .. 8g+7]
// and B[8g .. 8g+7][n] of a 32-wide k-step and holds rows 4g .. 4g+3 of column
// n.  Where an accumulator's rows become the next product's k, row m of tile t
// stands for index sig(t, m) = 32 (t/2) + 8 (m/4) + 4 (t%2) + m%4: tiles 2j and
// 2j+1, rounded to bf16, are then k-step j's operand as they are.
// Every matrix in LDS is row-major bf16 in swizzled 16-byte granules; an operand
// whose k runs along a row is one 16-byte read, one whose k runs down a column
// two transposing reads (lane i of a group of 16 names the 8 bytes of row i/4,
// columns 4 (i%4) .. + 3 of a 4 x 16 block and receives column i).
#include "gdn_backward_common.h"

namespace gdn {
namespace {

using bwd::C;
using bwd::ChunkAt;

constexpr int D = 128;
constexpr int kTile = C * D * 2;        // a 64 x 128 matrix
constexpr int kSquare = C * C * 2;      // a 64 x 64 matrix
constexpr int kState = D * D * 2;       // a bf16 state
constexpr float kLog2e = 1.4426950408889634f;

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
using bwd::f32x4;
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef unsigned char byte;

__device__ __forceinline__ f32x4 mfma(s16x8 a, s16x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                   c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 zero4() { return f32x4{0.f, 0.f, 0.f, 0.f}; }
__device__ __forceinline__ uint32_t pair(float lo, float hi)
{
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}
__device__ __forceinline__ u32x2 pack4(f32x4 a) { return u32x2{pair(a[0], a[1]), pair(a[2], a[3])}; }
__device__ __forceinline__ u32x4 pack8(f32x4 a, f32x4 b)
{
    return u32x4{pair(a[0], a[1]), pair(a[2], a[3]), pair(b[0], b[1]), pair(b[2], b[3])};
}
__device__ __forceinline__ s16x8 frag(f32x4 a, f32x4 b) { return __builtin_bit_cast(s16x8, pack8(a, b)); }
__device__ __forceinline__ f32x4 widen(s16x4 v)
{
    const u32x2 u = __builtin_bit_cast(u32x2, v);
    return f32x4{__uint_as_float(u[0] << 16), __uint_as_float(u[0] & 0xffff0000u), __uint_as_float(u[1] << 16),
                 __uint_as_float(u[1] & 0xffff0000u)};
}
__device__ __forceinline__ f32x4 widen_lo(s16x8 v) { return widen(s16x4{v[0], v[1], v[2], v[3]}); }
__device__ __forceinline__ f32x4 widen_hi(s16x8 v) { return widen(s16x4{v[4], v[5], v[6], v[7]}); }

// first index of tile t under sig, and sig's row for m
__device__ __forceinline__ constexpr int sig0(int t) { return 32 * (t >> 1) + 4 * (t & 1); }

// ---- LDS matrices ------------------------------------------------------------
// 256-byte rows (128 columns): granule q of row r at q ^ swz16(r); rows r .. r + 3
// differ in the upper two bits (a transposing read's 4 x 4 granules fall in 16
// different places), and the 16 rows of a direct read, natural or sig, in all
// four.  128-byte rows (64 columns): swz8, two rows covering the banks once.
__device__ __forceinline__ int swz16(int r)
{
    return ((r & 3) << 2) | (((r >> 3) & 3) ^ (((r >> 2) & 1) << 1));
}
__device__ __forceinline__ int swz8(int r)
{
    return (((r >> 1) & 1) << 2) | (((r >> 3) & 1) << 1) | (((r >> 2) ^ (r >> 4)) & 1);
}
template <int ROW> __device__ __forceinline__ int granule(int r, int q)
{
    if constexpr (ROW == 256) return r * 256 + 16 * (q ^ swz16(r));
    else return r * 128 + 16 * (q ^ swz8(r));
}
// The i-th 16-byte granule of thread tid (of 256) of a matrix in row order.
template <int ROW> __device__ __forceinline__ int staged(int tid, int i)
{
    if constexpr (ROW == 256) return (granule<256>(tid >> 4, tid & 15) ^ (32 * (i & 1))) + 4096 * i;
    else return granule<128>(tid >> 3, tid & 7) + 4096 * i;
}
// The same for a matrix that lies in memory as products leave it ("tile order":
// 1 KiB for 16 rows x 32 columns, lane 16 g + n's eight columns 8 g .. of row n at
// byte 16 lane, four of these a 16-row tile): whole 1 KiB stores and loads, where
// rows of 256 bytes took 64 bytes of 16 rows a store.
__device__ __forceinline__ int staged_tile(int tid, int i)
{
    return (granule<256>(tid & 15, tid >> 4) ^ (32 * (i & 1))) + 4096 * i;
}
// Operand reads.  A lane's address of an operand differs from tile to tile and
// k-step to k-step by an exclusive or of constant swizzle bits and a constant
// offset, so that eight lane bases, one for each way of reading, serve them all.
// fresh() keeps the compiler from forming every address ahead of a loop and
// spilling them.
typedef const __attribute__((address_space(3))) byte* lds_ptr;
__device__ __forceinline__ lds_ptr at_lds(uint32_t a) { return (lds_ptr)(uintptr_t)a; }
struct Lane {
    uint32_t rn, rs;    // 256-byte rows: a row of 16 i + n, of sig(t, n)
    uint32_t cs, cn;    // 256-byte rows, down a column: sig columns, natural ones
    uint32_t hn, hs;    // 128-byte rows: rows
    uint32_t ds, dn;    // 128-byte rows: columns
    __device__ __forceinline__ Lane(uint32_t base)
    {
        const int lane = threadIdx.x & 63, g = lane >> 4, n = lane & 15, kr = n >> 2, qq = n & 3;
        const int sr = 8 * (n >> 2) + (n & 3);
        rn = base + granule<256>(n, g);
        rs = base + granule<256>(sr, g);
        cs = base + granule<256>(8 * g + kr, qq);
        cn = base + granule<256>(8 * g + kr, qq >> 1) + 8 * (qq & 1);
        hn = base + granule<128>(n, g);
        hs = base + granule<128>(sr, g);
        ds = base + granule<128>(8 * g + kr, qq);
        dn = base + granule<128>(8 * g + kr, qq >> 1) + 8 * (qq & 1);
    }
    __device__ __forceinline__ void fresh()
    {
        asm volatile("" : "+v"(rn), "+v"(rs), "+v"(cs), "+v"(cn), "+v"(hn), "+v"(hs), "+v"(ds), "+v"(dn));
    }
};
__device__ __forceinline__ s16x8 rd16(uint32_t a, uint32_t off)
{
    return *reinterpret_cast<const __attribute__((address_space(3))) s16x8*>(at_lds(a) + off);
}
__device__ __forceinline__ s16x4 rdtr(uint32_t a, uint32_t off)
{
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at_lds(a) + off));
}
__device__ __forceinline__ s16x8 join(s16x4 a, s16x4 b)
{
    return s16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}
// columns 32 ks + 8 g .. + 7 of row 16 i + n, or of row sig(i, n)
template <int ROW> __device__ __forceinline__ s16x8 row8(const Lane& l, int m, int i, int ks)
{
    if constexpr (ROW == 256) return rd16(l.rn ^ (64 * ks) ^ (32 * (i & 1)), m + 4096 * i);
    else return rd16(l.hn ^ (64 * ks) ^ (16 * (i & 1)), m + 2048 * i);
}
template <int ROW> __device__ __forceinline__ s16x8 row8_sig(const Lane& l, int m, int i, int ks)
{
    if constexpr (ROW == 256) return rd16(l.rs ^ (64 * ks) ^ (32 * (i & 1)), m + 256 * sig0(i));
    else return rd16(l.hs ^ (64 * ks) ^ (16 * (i & 1)), m + 128 * sig0(i));
}
// rows 32 j + 8 g + 4 h .. + 3 of column sig(t, n), or 16 t + n
template <int ROW> __device__ __forceinline__ s16x4 col4_sig(const Lane& l, int m, int j, int h, int t)
{
    if constexpr (ROW == 256) return rdtr(l.cs ^ (64 * (t >> 1)) ^ (32 * h), m + 8192 * j + 1024 * h + 8 * (t & 1));
    else return rdtr(l.ds ^ (64 * (t >> 1)) ^ (16 * h), m + 4096 * j + 512 * h + 8 * (t & 1));
}
template <int ROW> __device__ __forceinline__ s16x4 col4(const Lane& l, int m, int j, int h, int t)
{
    if constexpr (ROW == 256) return rdtr(l.cn ^ (32 * t) ^ (32 * h), m + 8192 * j + 1024 * h);
    else return rdtr(l.dn ^ (32 * t) ^ (16 * h), m + 4096 * j + 512 * h);
}
// rows 32 j + 8 g .. + 7
template <int ROW> __device__ __forceinline__ s16x8 down_sig(const Lane& l, int m, int j, int t)
{
    return join(col4_sig<ROW>(l, m, j, 0, t), col4_sig<ROW>(l, m, j, 1, t));
}
template <int ROW> __device__ __forceinline__ s16x8 down(const Lane& l, int m, int j, int t)
{
    return join(col4<ROW>(l, m, j, 0, t), col4<ROW>(l, m, j, 1, t));
}
using bwd::lds_barrier;
// Nothing is moved across: a batch of operand reads is issued whole ahead of the
// products of the batch before, not one by one in front of each product.
__device__ __forceinline__ void sched_fence() { __builtin_amdgcn_sched_barrier(0); }

// ---- global operands -----------------------------------------------------------
// Rows of a chunk through a buffer resource whose range ends with the chunk:
// rows past it read as zero, without a branch.
typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ __forceinline__ uint64_t uniform(uint64_t v)
{
    // (the builtin's int must not be sign-extended into the upper half)
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)v);
    return ((uint64_t)hi << 32) | lo;
}
__device__ __forceinline__ rsrc_t make_rsrc(const void* base, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc((void*)uniform((uint64_t)base), (short)0,
                                             (int)__builtin_amdgcn_readfirstlane(bytes), 0x00020000);
}
// soff: a wave-uniform offset in an SGPR, so that a thread's loads share one
// address register
__device__ __forceinline__ u32x4 load16(rsrc_t r, uint32_t voff, uint32_t soff)
{
    return __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, 0);
}
// Eight values of an activation as they lie in memory (bf16, or codes with the
// row's scale byte), and as bf16: a code times a power of two is exact in bf16.
template <typename TA> struct Raw;
template <> struct Raw<uint16_t> {
    u32x4 v;
    __device__ __forceinline__ u32x4 bits() const { return v; }
};
template <> struct Raw<uint8_t> {
    u32x2 c;
    uint32_t e;
    __device__ __forceinline__ u32x4 bits() const
    {
        const float s = ckpt_scale((int)e);
        float f[8];
        ckpt_unpack4(c[0], f);
        ckpt_unpack4(c[1], f + 4);
        return u32x4{pair(f[0] * s, f[1] * s), pair(f[2] * s, f[3] * s), pair(f[4] * s, f[5] * s), pair(f[6] * s, f[7] * s)};
    }
};
// One head's rows of a chunk of an activation [tokens][heads][128].
template <typename TA> struct Rows {
    rsrc_t data, exps;
    uint32_t stride, heads;
    __device__ __forceinline__ Rows(const void* p, const uint8_t* e, int64_t row0, int rows, int H, int head)
    {
        const int64_t first = row0 * H + head;
        stride = (uint32_t)H * D * (uint32_t)sizeof(TA);
        heads = (uint32_t)H;
        data = make_rsrc(static_cast<const TA*>(p) + first * D, (uint32_t)rows * stride);
        if constexpr (sizeof(TA) == 1) exps = make_rsrc(e + first, (uint32_t)rows * heads);
    }
    // granule q (eight values) of row r + dr, dr wave-uniform
    __device__ __forceinline__ Raw<TA> load(int r, int q, int dr = 0) const
    {
        Raw<TA> x;
        if constexpr (sizeof(TA) == 1) {
            x.c = __builtin_amdgcn_raw_buffer_load_b64(data, (uint32_t)r * stride + 8 * q, (uint32_t)dr * stride, 0);
            x.e = __builtin_amdgcn_raw_buffer_load_b8(exps, (uint32_t)r * heads, (uint32_t)dr * heads, 0);
        } else {
            x.v = load16(data, (uint32_t)r * stride + 16 * q, (uint32_t)dr * stride);
        }
        return x;
    }
};

// Workspace of one (chunk, v-head), in bytes.
constexpr int W_W = 0;                       // [64][128] in tile order
constexpr int W_QT = W_W + kTile;            // likewise
constexpr int W_U = W_QT + kTile;            // likewise
constexpr int W_TT = W_U + kTile;            // T^T [64][64]
constexpr int W_PT = W_TT + kSquare;         // P^T [64][64]
constexpr int W_B = W_PT + kSquare;          // B's ten lower tiles in accumulator order, 512 bytes each
constexpr int W_P = W_B + 10 * 512;          // P's
constexpr int W_G = W_P + 10 * 512;          // G log2(e), 64 floats; beta, 64 floats
constexpr int W_BYTES = W_G + 512;

struct Args {
    const void *q, *k, *v, *dout;
    const uint8_t *q_exps, *k_exps, *v_exps;
    const float *log_g, *beta, *h0, *dht;
    uint16_t *dq, *dk, *dv, *dg, *db;
    float* dh0;
    int B, T, Hk, Hv;
    const int32_t* cu;
    int nc_dense;
    int32_t* base;       // chunk table (packed)
    byte* heads;         // [chunk][Hv] W_BYTES
    byte* h;             // [chunk][Hv] start states, bf16, transposed [dv][dk], in tile order
    byte* dh;            // [chunk][Hv] end gradients, likewise
};

__global__ void __launch_bounds__(256)
gdn_bwd_table_kernel(const int32_t* __restrict__ cu, int B, int T, int32_t* __restrict__ base)
{
    __shared__ int32_t part[256];
    bwd::chunk_table(cu, B, T, base, part);
}

// sum over the 16 lanes of a row of lanes
__device__ __forceinline__ float sum16(float x)
{
#define GDN_ROR(n) x += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x120 | n, 0xf, 0xf, false))
    GDN_ROR(8); GDN_ROR(4); GDN_ROR(2); GDN_ROR(1);
#undef GDN_ROR
    return x;
}
__device__ __forceinline__ float wave_scan(float x, int lane)
{
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const float y = __shfl_up(x, o);
        if (lane >= o) x += y;
    }
    return x;
}

extern __shared__ __attribute__((aligned(1024))) byte lds[];

// ---- prep ------------------------------------------------------------------------
// Four waves, two workgroups a compute unit.  T by 16 x 16 blocks in fp32; P diag(beta)
// T, W, U and Qt are products with T's and (P beta T ga)'s columns as they lie
// transposed in LDS.  Bound by the workspace it writes: 4576 tokens, 48 v-heads: 263
// MB written and 106 MB read (counters) in 91 to 92 us, 4.0 TB/s.
using bwd::kBP;                                // pitch of the fp32 matrix B
constexpr int P_K = 0;                         // K
constexpr int P_Q = P_K + kTile;               // Q, then V
constexpr int P_B = P_Q + kTile;               // B (fp32), then T^T and (T ga)^T
constexpr int P_BBYTES = C * kBP * 4;
constexpr int P_D = P_B + P_BBYTES;            // T's diagonal blocks (fp32, 16 x 17 each)
constexpr int P_TBG = P_D + 4 * 16 * 17 * 4;   // (beta T ga)^T
constexpr int P_PT = P_TBG + kSquare;          // P^T
constexpr int P_PTG = P_PT + kSquare;          // (P beta T ga)^T
constexpr int P_G = P_PTG + kSquare;           // G log2(e), beta, ga, E beta
constexpr int kPrepLds = P_G + 4 * C * 4;
static_assert(2 * kSquare <= P_BBYTES && 2 * kPrepLds <= 160 * 1024, "two prep workgroups a compute unit");

template <typename TA>
__global__ void __launch_bounds__(256, 2)
gdn_bwd_prep_kernel(Args a)
{
    ChunkAt at;
    // the v-heads of a k-head, which share k and q, are neighbours
    const int64_t item = bwd::xcd_item();
    const int vh = (int)(item % a.Hv), x = (int)(item / a.Hv), kh = vh / (a.Hv / a.Hk);
    if (!bwd::chunk_at(x, a.cu, a.base, a.B, a.T, a.nc_dense, &at)) return;
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, n = lane & 15;
    byte* out = a.heads + ((size_t)x * a.Hv + vh) * W_BYTES;
    byte *sK = lds + P_K, *sQ = lds + P_Q, *sTT = lds + P_B, *sTG = lds + P_B + kSquare, *sTBG = lds + P_TBG,
         *sPT = lds + P_PT, *sPTG = lds + P_PTG;
    float *sB = reinterpret_cast<float*>(lds + P_B), *sD = reinterpret_cast<float*>(lds + P_D),
          *sG = reinterpret_cast<float*>(lds + P_G), *sBt = sG + C, *sGa = sBt + C, *sEb = sGa + C;

    const Lane L((uint32_t)(uintptr_t)(lds_ptr)lds);

    // K and Q rows to LDS, V rows to registers (rows past the chunk are zero)
    const Rows<TA> rq(a.q, a.q_exps, at.row0, at.rows, a.Hk, kh);
    Raw<TA> vr[4];
    {
        const Rows<TA> rk(a.k, a.k_exps, at.row0, at.rows, a.Hk, kh), rv(a.v, a.v_exps, at.row0, at.rows, a.Hv, vh);
        Raw<TA> kr[4], qr[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            kr[i] = rk.load(tid >> 4, tid & 15, 16 * i);
            qr[i] = rq.load(tid >> 4, tid & 15, 16 * i);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) vr[i] = rv.load(tid >> 4, tid & 15, 16 * i);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int o = staged<256>(tid, i);
            *reinterpret_cast<u32x4*>(sK + o) = kr[i].bits();
            *reinterpret_cast<u32x4*>(sQ + o) = qr[i].bits();
        }
    }
    if (w == 0) {
        const bool live = lane < at.rows;
        const int64_t r = (at.row0 + lane) * a.Hv + vh;
        const float G = wave_scan(live ? bounded_log_decay(a.log_g[r]) : 0.f, lane) * kLog2e;
        const float GL = __shfl(G, 63);
        const float bt = live ? a.beta[r] : 0.f;
        sG[lane] = G;
        sBt[lane] = bt;
        sGa[lane] = __builtin_amdgcn_exp2f(G);
        sEb[lane] = __builtin_amdgcn_exp2f(GL - G) * bt;
        float* gG = reinterpret_cast<float*>(out + W_G);
        gG[lane] = G;
        gG[C + lane] = bt;
    }
    lds_barrier();

    // lower tiles: wave w forms row tile w of B and row tile 3 - w of P
    {
        s16x8 kf[4][4], lf[2][4];
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            lf[0][ks] = row8<256>(L, P_K, w, ks);
            lf[1][ks] = row8<256>(L, P_Q, 3 - w, ks);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) kf[j][ks] = row8<256>(L, P_K, j, ks);
        sched_fence();
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int i = half ? 3 - w : w;
            const f32x4 Gr = *reinterpret_cast<const f32x4*>(sG + 16 * i + 4 * g);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f32x4 t = zero4();
                const int c = 16 * j + n;
                if (j <= i) {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) t = mfma(lf[half][ks], kf[j][ks], t);
                    const float Gc = sG[c];
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const int r = 16 * i + 4 * g + s;
                        t[s] = (half ? c <= r : c < r) ? t[s] * __builtin_amdgcn_exp2f(Gr[s] - Gc) : 0.f;
                    }
                    const int tile = i * (i + 1) / 2 + j;
                    *reinterpret_cast<u32x2*>(out + (half ? W_P : W_B) + 512 * tile + 8 * lane) = pack4(t);
                }
                if (half)
                    *reinterpret_cast<u32x2*>(sPT + granule<128>(c, 2 * i + (g >> 1)) + 8 * (g & 1)) = pack4(t);
                else if (j <= i)
#pragma unroll
                    for (int s = 0; s < 4; ++s) sB[(16 * i + 4 * g + s) * kBP + c] = t[s];
            }
        }
    }
    lds_barrier();
    // V takes Q's place; T = (I + B diag(beta))^-1
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        *reinterpret_cast<u32x4*>(sQ + staged<256>(tid, i)) = vr[i].bits();
    }
    if (w == 0) bwd::solve_diagonal(sB, sBt, sD);
    lds_barrier();
    f32x4 Tc[4];
    bwd::solve_column(sB, sBt, sD, w, Tc);
    lds_barrier();   // every read of B is done
    {
        const int c = 16 * w + n;
        const float ga = sGa[c];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x4 bt = *reinterpret_cast<const f32x4*>(sBt + 16 * i + 4 * g);
            const int o = granule<128>(c, 2 * i + (g >> 1)) + 8 * (g & 1);
            const u32x2 tt = pack4(Tc[i]);
            *reinterpret_cast<u32x2*>(sTT + o) = tt;
            *reinterpret_cast<u32x2*>(sTG + o) = pack4(Tc[i] * ga);
            *reinterpret_cast<u32x2*>(sTBG + o) = pack4(Tc[i] * bt * ga);
        }
    }
    lds_barrier();
    // (P beta T ga)^T, row tile i of the product by wave i: A = P down P^T, B =
    // (beta T ga)^T's rows
    {
        const s16x8 p0 = down<128>(L, P_PT, 0, w), p1 = down<128>(L, P_PT, 1, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f32x4 t = mfma(p0, row8<128>(L, P_TBG, j, 0), zero4());
            t = mfma(p1, row8<128>(L, P_TBG, j, 1), t);
            *reinterpret_cast<u32x2*>(sPTG + granule<128>(16 * j + n, 2 * w + (g >> 1)) + 8 * (g & 1)) = pack4(t);
        }
    }
    // T^T and P^T as they are, rows in order
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int e = tid + 256 * i, r = e >> 3, q = e & 7;
        *reinterpret_cast<u32x4*>(out + W_TT + 16 * e) = *reinterpret_cast<const u32x4*>(sTT + granule<128>(r, q));
        *reinterpret_cast<u32x4*>(out + W_PT + 16 * e) = *reinterpret_cast<const u32x4*>(sPT + granule<128>(r, q));
    }
    lds_barrier();
    // W, Qt and U formed transposed (dk or dv down, chunk rows across): wave w
    // takes columns 32 w .. + 31, and each lane ends with eight consecutive
    // columns of its row
    s16x8 kf[2][2], vf[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            kf[i][j] = down_sig<256>(L, P_K, j, 2 * w + i);
            vf[i][j] = down_sig<256>(L, P_Q, j, 2 * w + i);
        }
    Raw<TA> q8[4];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) q8[rt] = rq.load(16 * rt + n, 4 * w + g);
    s16x8 tg[2][2], tt[2][2], pg[2][2];        // by turns: row tile rt, k-step
    auto read = [&](int rt) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (2 * j <= rt) {                  // T and P are lower triangular
                tg[rt & 1][j] = down<128>(L, P_B + kSquare, j, rt);
                tt[rt & 1][j] = down<128>(L, P_B, j, rt);
                pg[rt & 1][j] = down<128>(L, P_PTG, j, rt);
            }
    };
    read(0);
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
        if (rt < 3) read(rt + 1);
        sched_fence();
        const int r = 16 * rt + n;
        f32x4 ww[2] = {zero4(), zero4()}, uu[2] = {zero4(), zero4()}, qq[2] = {zero4(), zero4()};
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (2 * j <= rt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    ww[i] = mfma(kf[i][j], tg[rt & 1][j], ww[i]);
                    uu[i] = mfma(vf[i][j], tt[rt & 1][j], uu[i]);
                    qq[i] = mfma(kf[i][j], pg[rt & 1][j], qq[i]);
                }
        const float eb = sEb[r], ga = sGa[r];
        const int o = 4096 * rt + 1024 * w + 16 * lane;
        *reinterpret_cast<u32x4*>(out + W_W + o) = pack8(ww[0] * eb, ww[1] * eb);
        *reinterpret_cast<u32x4*>(out + W_U + o) = pack8(uu[0] * eb, uu[1] * eb);
        const s16x8 qb = __builtin_bit_cast(s16x8, q8[rt].bits());
        *reinterpret_cast<u32x4*>(out + W_QT + o) = pack8(widen_lo(qb) * ga - qq[0], widen_hi(qb) * ga - qq[1]);
        sched_fence();
    }
}

// ---- spine -------------------------------------------------------------------------
// Eight waves.  Four walk: each owns 16 dv columns of the state, so that a step's
// two products follow each other in its registers.  Four load: the next chunks'
// matrices through registers (three steps ahead) into the LDS stage that is not
// being read, so that a load or an LDS write that waits for the compute unit's
// memory path holds up no product.  72 steps of 48 v-heads take 159 us (316 MB read
// and 226 MB written by the counters, 3.4 TB/s), 197 us with four waves that did
// both and without the XCD order of Walk.  A step's latency is the time: 4800 cycles
// backwards, of which the products fill 770, the LDS reads about 2000 and the 72 KB
// of matrices through the compute unit's memory path 2200.  Loading waves that also
// wrote the states out (two barriers a step) took 172 us.
// One stage of LDS holds a chunk's matrices: forwards W, K and U's columns,
// backwards K, W, Qt and do's columns.
constexpr int kCols = 64;
constexpr int kSpineThreads = 512;
constexpr int S_L = 0;                     // W, or K
constexpr int S_R = S_L + kTile;           // K, or W
constexpr int S_X = S_R + kTile;           // Qt (backwards)
constexpr int S_C = S_X + kTile;           // U, or do: [64][64]
constexpr int S_G = S_C + kSquare;         // G_L log2(e)
constexpr int kStage = S_G + 1024;
constexpr int kSpineLds = 2 * kStage;

// Where a workgroup walks.
struct Walk {
    int vh, kh, half, b, nc;
    bool rev;
    int64_t row0, len, x0;
    __device__ __forceinline__ explicit Walk(const Args& a)
    {
        // the halves of a v-head, which read the same W, Qt and K step by step, are
        // neighbours, then the v-heads of a k-head; the two directions, which meet
        // only half way, come one after the other; each XCD has all sequences,
        // whose lengths differ
        int64_t i = bwd::xcd_item();
        half = (int)(i & 1);
        i >>= 1;
        const int rep = a.Hv / a.Hk;
        const int g = (int)(i % rep);
        i /= rep;
        rev = (i & 1) != 0;
        i >>= 1;
        b = (int)(i % a.B);
        kh = (int)(i / a.B);
        vh = kh * rep + g;
        bwd::seq_rows(a.cu, b, a.T, &row0, &len);
        nc = bwd::walk_chunks(a.cu, a.base, b, len);
        x0 = a.cu ? a.base[b] : (int64_t)b * a.nc_dense;
    }
};

template <typename TA, bool REV>
__device__ __forceinline__ void spine_load(const Args& a, const Walk& k)
{
    const int tid = threadIdx.x & 255;
    struct Regs {
        u32x4 W[4], x[4], c[2];
        Raw<TA> K[4];
        float gl;
    } in[3];
    auto fetch = [&](Regs& in, int i) {      // the i-th chunk of the walk
        i = min(i, k.nc - 1);
        const int c = REV ? k.nc - 1 - i : i;
        const byte* head = a.heads + ((size_t)(k.x0 + c) * a.Hv + k.vh) * W_BYTES;
        const int64_t r0 = k.row0 + (int64_t)c * C;
        const int rows = (int)min((int64_t)C, k.len - (int64_t)c * C);
        const Rows<TA> rk(a.k, a.k_exps, r0, rows, a.Hk, k.kh);
        const rsrc_t rh = make_rsrc(head, W_BYTES);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            in.W[j] = load16(rh, 16 * tid, W_W + 4096 * j);
            if (REV) in.x[j] = load16(rh, 16 * tid, W_QT + 4096 * j);
            in.K[j] = rk.load(tid >> 4, tid & 15, 16 * j);
        }
        const Rows<uint16_t> ro(a.dout, nullptr, r0, REV ? rows : 0, a.Hv, k.vh);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            // do: rows; U: the two 1 KiB pieces of this half's columns in two row tiles
            in.c[j] = REV ? ro.load(tid >> 3, 8 * k.half + (tid & 7), 32 * j).v
                          : load16(rh, 4096 * (tid >> 7) + 16 * (tid & 127), W_U + 2048 * k.half + 8192 * j);
        }
        in.gl = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rh, 0, W_G + 4 * (C - 1), 0));
    };
    auto put = [&](const Regs& in, int S) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            byte* o = lds + S + staged_tile(tid, j);
            *reinterpret_cast<u32x4*>(o + (REV ? S_R : S_L)) = in.W[j];
            if (REV) *reinterpret_cast<u32x4*>(o + S_X) = in.x[j];
            *reinterpret_cast<u32x4*>(lds + S + staged<256>(tid, j) + (REV ? S_L : S_R)) = in.K[j].bits();
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int row = 16 * (2 * j + (tid >> 7)) + (tid & 15), q = 4 * ((tid >> 6) & 1) + ((tid >> 4) & 3);
            *reinterpret_cast<u32x4*>(lds + S + S_C + (REV ? staged<128>(tid, j) : granule<128>(row, q))) = in.c[j];
        }
        *reinterpret_cast<float*>(lds + S + S_G) = in.gl;      // the same value from every thread
    };
    // chunk i's set is i % 3; past the end the last chunk is fetched again and
    // written to a stage that nobody reads (no branches)
    fetch(in[0], 0);
    fetch(in[1], 1);
    fetch(in[2], 2);
    put(in[0], 0);
    fetch(in[0], 3);
    lds_barrier();
    auto step = [&](int i, Regs& r) {
        put(r, ((i + 1) & 1) * kStage);
        __builtin_amdgcn_sched_barrier(0);
        fetch(r, i + 4);
        __builtin_amdgcn_sched_barrier(0);
        lds_barrier();
    };
    // whole turns of three, so that no path skips a fetch: the compiler's waits,
    // which count the loads behind the one that is needed, serve every path
    for (int i = 0; i < k.nc; i += 3) {
        step(i, in[1]);
        step(i + 1, in[2]);
        step(i + 2, in[0]);
    }
}

template <bool REV>
__device__ __forceinline__ void spine_step(const Args& a, const Walk& k)
{
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 4, n = lane & 15;
    const int col = k.half * kCols + 16 * w + n;     // this lane's dv column
    const float* from = REV ? a.dht : a.h0;
    const size_t hoff = ((size_t)k.b * a.Hv + k.vh) * D * D;

    f32x4 st[8];                                     // dk index sig(t, 4g + s)
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int s = 0; s < 4; ++s)
            st[t][s] = from ? from[hoff + (size_t)(sig0(t) + 8 * g + s) * D + col] : 0.f;
    // the start state has arrived: else the loop's waits, which serve its first
    // pass too, would wait for the stores in flight each time
#pragma unroll
    for (int t = 0; t < 8; ++t) asm volatile("" : "+v"(st[t]));
    const Lane L((uint32_t)(uintptr_t)(lds_ptr)lds);
    if (k.nc > 0) lds_barrier();
    for (int i = 0; i < k.nc; ++i) {
        const int S = (i & 1) * kStage;
        s16x8 lf[4][4];
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) lf[rt][ks] = row8_sig<256>(L, S + S_L, rt, ks);
        const float gl = __builtin_amdgcn_exp2f(*reinterpret_cast<const float*>(lds + S + S_G));
        sched_fence();
        s16x8 sb[4];
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) sb[ks] = frag(st[2 * ks], st[2 * ks + 1]);
        f32x4 d[4];
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) d[rt] = zero4();
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) d[rt] = mfma(lf[rt][ks], sb[ks], d[rt]);
        sched_fence();
        // the second product's operands, half its rows at a time, while the first
        // product runs
        s16x8 rf[2][8], xf[2][8], ob[2];
        s16x4 uf[4];
        auto read = [&](int j) {
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                if (REV) xf[j][t] = down_sig<256>(L, S + S_X, j, t);
                rf[j][t] = down_sig<256>(L, S + S_R, j, t);
            }
        };
        if (REV) {
#pragma unroll
            for (int j = 0; j < 2; ++j) ob[j] = down<128>(L, S + S_C, j, w);
        } else {
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) uf[rt] = col4<128>(L, S + S_C, rt >> 1, rt & 1, w);
        }
        read(0);
        sched_fence();
#pragma unroll
        for (int ks = 2; ks < 4; ++ks)
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) d[rt] = mfma(lf[rt][ks], sb[ks], d[rt]);
        sched_fence();
        read(1);
        const int c = REV ? k.nc - 1 - i : i;
        byte* out = (REV ? a.dh : a.h) + ((size_t)(k.x0 + c) * a.Hv + k.vh) * kState + 4096 * (4 * k.half + w) + 16 * lane;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) *reinterpret_cast<s16x8*>(out + 1024 * ks) = sb[ks];
        sched_fence();
#pragma unroll
        for (int t = 0; t < 8; ++t) st[t] *= gl;
        if (REV) {
#pragma unroll
            for (int t = 0; t < 8; ++t) st[t] = mfma(xf[0][t], ob[0], st[t]);
        }
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) d[rt] = REV ? -d[rt] : widen(uf[rt]) - d[rt];
        const s16x8 db[2] = {frag(d[0], d[1]), frag(d[2], d[3])};
#pragma unroll
        for (int t = 0; t < 8; ++t) st[t] = mfma(rf[0][t], db[0], st[t]);
        if (REV) {
#pragma unroll
            for (int t = 0; t < 8; ++t) st[t] = mfma(xf[1][t], ob[1], st[t]);
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) st[t] = mfma(rf[1][t], db[1], st[t]);
        sched_fence();
        lds_barrier();
    }
    for (int i = k.nc; i % 3 != 0; ++i) lds_barrier();   // the loading waves' last turn
    if (REV && a.dh0)
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int s = 0; s < 4; ++s) a.dh0[hoff + (size_t)(sig0(t) + 8 * g + s) * D + col] = st[t][s];
}

template <typename TA>
__global__ void __launch_bounds__(kSpineThreads)
gdn_bwd_spine_kernel(Args a)
{
    const Walk k(a);
    const bool loads = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8) != 0;
    if (loads) {
        if (k.nc == 0) return;
        if (k.rev) spine_load<TA, true>(a, k);
        else spine_load<TA, false>(a, k);
    } else {
        if (k.rev) spine_step<true>(a, k);
        else spine_step<false>(a, k);
    }
}

// ---- grads -------------------------------------------------------------------------
// Eight waves, two to a SIMD, so that one's products run under the other's vector
// work and LDS reads; the LDS holds a v-head whole (K, Q, do, V, h, dh', T, P), so one
// workgroup a compute unit.  72 x 16 chunks and k-heads of three v-heads: 231 to 233 us (471
// MB read, 100 MB written by the counters, 2.5 TB/s).  Nothing is full: LDS 35 % of
// the cycles (a third more in bank conflicts), vector units 35 %, matrix units 14 %;
// the time is the five barriers of a v-head, each behind a chain of reads, products
// and rounding, and 4.5 rounds of workgroups, the last half empty; the matrices that it
// reads would take 111 us at a large copy's rate.  Taken and dropped: four
// waves with the next v-head in registers (250 us), eight with it (250 to 270 us, as
// registers spill), h, dh', T and P by asynchronous loads to LDS under the last products
// (no gain: the loads' time moves into the phases that they run under).
constexpr int kGradThreads = 512;
constexpr int G_K = 0;
constexpr int G_Q = G_K + kTile;
constexpr int G_DO = G_Q + kTile;
constexpr int G_H = G_DO + kTile;          // h^T [dv][dk]
constexpr int G_DH = G_H + kState;         // dh'^T, then N^T and (dP o Gam)^T
constexpr int G_U = G_DH + kState;         // V, then u^T [dv][64]
constexpr int G_X = G_U + kTile;           // T^T and P^T, then dx^T [dv][64]
constexpr int G_S = G_X + kTile;           // small arrays
struct Small {
    float G[C], beta[C], ga[C], E[C];      // G in units of log2
    float rowG[8][C], rowB[8][C];          // by wave
    float rowX[2][C], colX[8][C], colZ[4][C];
    float rowQ[4][C];
    float sumY[8], hd[8];
};
constexpr int kGradLds = G_S + (int)sizeof(Small);
static_assert(kGradLds <= 160 * 1024, "the grads kernel's LDS");

// SPLIT: a workgroup takes one v-head and leaves its part of dq and dk, in fp32,
// where the v-head's h and dh' were, which only it reads.
template <typename TA, bool SPLIT>
__global__ void __launch_bounds__(kGradThreads)
gdn_bwd_grads_kernel(Args a)
{
    ChunkAt at;
    const int x = blockIdx.x, rep = a.Hv / a.Hk, kh = SPLIT ? blockIdx.y / rep : blockIdx.y;
    const int vh0 = SPLIT ? blockIdx.y : kh * rep, vh1 = SPLIT ? vh0 + 1 : vh0 + rep;
    if (!bwd::chunk_at(x, a.cu, a.base, a.B, a.T, a.nc_dense, &at)) return;
    int tid = threadIdx.x;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    byte *sK = lds + G_K, *sQ = lds + G_Q, *sO = lds + G_DO, *sH = lds + G_H, *sDH = lds + G_DH, *sU = lds + G_U,
         *sX = lds + G_X, *sTT = sX, *sPT = sX + kSquare, *sV = sU, *sN = sDH, *sM = sDH + kSquare;
    Small& sm = *reinterpret_cast<Small*>(lds + G_S);

    // a v-head's matrices on their way to LDS; B's or P's tiles of the rows that
    // this wave forms of Zu (waves 0-3, row tile w) or do u^T (row tile 7 - w)
    struct Regs {
        u32x4 h[4], dh[4], o[2], tt, pt;
        Raw<TA> v[2];
        s16x4 bp[4];
        float G, beta;
    } in;
    const int ti = w >= 4 ? 7 - w : w;     // row tile of Zu or do u^T: with its SIMD's other wave, five tiles
    auto fetch = [&](int vh) {
        const byte* head = a.heads + ((size_t)x * a.Hv + vh) * W_BYTES;
        const byte* hT = a.h + ((size_t)x * a.Hv + vh) * kState;
        const byte* dhT = a.dh + ((size_t)x * a.Hv + vh) * kState;
        const Rows<TA> rv(a.v, a.v_exps, at.row0, at.rows, a.Hv, vh);
        const Rows<uint16_t> ro(a.dout, nullptr, at.row0, at.rows, a.Hv, vh);
        const rsrc_t rw = make_rsrc(head, W_BYTES), rh = make_rsrc(hT, kState), rd = make_rsrc(dhT, kState);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            in.h[i] = load16(rh, 16 * tid, 8192 * i);
            in.dh[i] = load16(rd, 16 * tid, 8192 * i);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            in.v[i] = rv.load(tid >> 4, tid & 15, 32 * i);
            in.o[i] = ro.load(tid >> 4, tid & 15, 32 * i).v;
        }
        in.tt = load16(rw, 16 * tid, W_TT);
        in.pt = load16(rw, 16 * tid, W_PT);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            in.bp[j] = __builtin_bit_cast(s16x4, __builtin_amdgcn_raw_buffer_load_b64(
                rw, 8 * (tid & 63), (w >= 4 ? W_P : W_B) + 512 * (ti * (ti + 1) / 2 + min(ti, j)), 0));
        }
        in.G = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rw, 4 * (tid & 63), W_G, 0));
        in.beta = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rw, 4 * (tid & 63), W_G + 4 * C, 0));
    };
    {
        const Rows<TA> rk(a.k, a.k_exps, at.row0, at.rows, a.Hk, kh), rq(a.q, a.q_exps, at.row0, at.rows, a.Hk, kh);
        Raw<TA> kr[2], qr[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            kr[i] = rk.load(tid >> 4, tid & 15, 32 * i);
            qr[i] = rq.load(tid >> 4, tid & 15, 32 * i);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int o = granule<256>(tid >> 4, tid & 15) + 8192 * i;
            *reinterpret_cast<u32x4*>(sK + o) = kr[i].bits();
            *reinterpret_cast<u32x4*>(sQ + o) = qr[i].bits();
        }
    }
    Lane L((uint32_t)(uintptr_t)(lds_ptr)lds);
    // dq and dk, transposed: dk columns 32 wc .. + 31 down (two tiles under sig),
    // rows 32 wr + 16 j + n
    const int wc = w & 3, wr = w >> 2;
    f32x4 dq[2][2], dk[2][2];              // [dk tile][row tile]
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) dq[i][j] = dk[i][j] = zero4();

    for (int vh = vh0; vh < vh1; ++vh) {
        L.fresh();
        asm volatile("" : "+v"(tid));      // likewise for all that is formed from it
        const int lane = tid & 63, g = lane >> 4, n = lane & 15;
        fetch(vh);
        lds_barrier();                     // the v-head before has read the LDS
        float hd = 0.f;                    // <h, dh'>
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int o = granule<256>(16 * (tid >> 8) + (tid & 15), (tid >> 4) & 15) + 8192 * i;
            *reinterpret_cast<u32x4*>(sH + o) = in.h[i];
            *reinterpret_cast<u32x4*>(sDH + o) = in.dh[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                hd = fmaf(__uint_as_float(in.h[i][j] << 16), __uint_as_float(in.dh[i][j] << 16), hd);
                hd = fmaf(__uint_as_float(in.h[i][j] & 0xffff0000u), __uint_as_float(in.dh[i][j] & 0xffff0000u), hd);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int o = granule<256>(tid >> 4, tid & 15) + 8192 * i;
            *reinterpret_cast<u32x4*>(sO + o) = in.o[i];
            *reinterpret_cast<u32x4*>(sV + o) = in.v[i].bits();
        }
        *reinterpret_cast<u32x4*>(sTT + granule<128>(tid >> 3, tid & 7)) = in.tt;
        *reinterpret_cast<u32x4*>(sPT + granule<128>(tid >> 3, tid & 7)) = in.pt;
        s16x4 bp4[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) bp4[j] = in.bp[j];
        if (w == 0) {
            const float GL = __shfl(in.G, 63);
            sm.G[lane] = in.G;
            sm.beta[lane] = in.beta;
            sm.ga[lane] = __builtin_amdgcn_exp2f(in.G);
            sm.E[lane] = __builtin_amdgcn_exp2f(GL - in.G);
        }
#pragma unroll
        for (int o = 32; o; o >>= 1) hd += __shfl_xor(hd, o);
        if (lane == 0) sm.hd[w] = hd;
        lds_barrier();

        // columns 16 w .. + 15 of dv: x, u, ddelta, dx, rows under sig
        f32x4 u[4], dx[4];
        {
            f32x4 kh4[4], kd[4];
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) kh4[rt] = kd[rt] = zero4();
            s16x8 hb[2], db[2], kf[2][4];    // by turns of the k-steps
            auto read = [&](int ks) {
                hb[ks & 1] = row8<256>(L, G_H, w, ks);
                db[ks & 1] = row8<256>(L, G_DH, w, ks);
#pragma unroll
                for (int rt = 0; rt < 4; ++rt) kf[ks & 1][rt] = row8_sig<256>(L, G_K, rt, ks);
            };
            s16x8 tf[4][2], pf[4][2], ob[2];
            s16x4 vf[4];
            read(0);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                if (ks < 3) {
                    read(ks + 1);
                } else {
#pragma unroll
                    for (int rt = 0; rt < 4; ++rt) vf[rt] = col4<256>(L, G_U, rt >> 1, rt & 1, w);
#pragma unroll
                    for (int rt = 0; rt < 4; ++rt) {
                        tf[rt][0] = down_sig<128>(L, G_X, 0, rt);            // T lower triangular
                        if (rt >= 2) tf[rt][1] = down_sig<128>(L, G_X, 1, rt);
                    }
                }
                sched_fence();
#pragma unroll
                for (int rt = 0; rt < 4; ++rt) {
                    kh4[rt] = mfma(kf[ks & 1][rt], hb[ks & 1], kh4[rt]);
                    kd[rt] = mfma(kf[ks & 1][rt], db[ks & 1], kd[rt]);
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) ob[j] = down<256>(L, G_DO, j, w);
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) {                                 // P^T upper triangular
                pf[rt][1] = row8_sig<128>(L, G_X + kSquare, rt, 1);
                if (rt < 2) pf[rt][0] = row8_sig<128>(L, G_X + kSquare, rt, 0);
            }
            sched_fence();
            f32x4 dd[4];
            f32x4 xv[4];
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) {
                kh4[rt] *= *reinterpret_cast<const f32x4*>(sm.ga + sig0(rt) + 8 * g);      // ga K h
                xv[rt] = widen(vf[rt]) - kh4[rt];
            }
            const s16x8 xb[2] = {frag(xv[0], xv[1]), frag(xv[2], xv[3])};
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) {
                u[rt] = mfma(tf[rt][0], xb[0], zero4());
                if (rt >= 2) u[rt] = mfma(tf[rt][1], xb[1], u[rt]);
                dd[rt] = mfma(pf[rt][1], ob[1], zero4());
                if (rt < 2) dd[rt] = mfma(pf[rt][0], ob[0], dd[rt]);
            }
            // T^T's rows, in the place of P^T's
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) {
                pf[rt][1] = row8_sig<128>(L, G_X, rt, 1);
                if (rt < 2) pf[rt][0] = row8_sig<128>(L, G_X, rt, 0);
            }
            sched_fence();
            float sumY = 0.f;
            f32x4 rG[4], rB[4];
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) rG[rt] = rB[rt] = zero4();
            f32x4 yv[4];
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) {
                const int r = sig0(rt) + 8 * g;
                const f32x4 E = *reinterpret_cast<const f32x4*>(sm.E + r), bt = *reinterpret_cast<const f32x4*>(sm.beta + r);
                const f32x4 ek = E * kd[rt];
                dd[rt] += ek;
                yv[rt] = bt * dd[rt];
                rB[rt] += dd[rt] * u[rt];
                const f32x4 Y = bt * u[rt] * ek;
                rG[rt] -= Y;
                sumY += (Y[0] + Y[1]) + (Y[2] + Y[3]);
            }
            const s16x8 yb[2] = {frag(yv[0], yv[1]), frag(yv[2], yv[3])};
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) {
                dx[rt] = mfma(pf[rt][1], yb[1], zero4());
                if (rt < 2) dx[rt] = mfma(pf[rt][0], yb[0], dx[rt]);
            }
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) {
                f32x4 rg, rb;
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    rg[s] = sum16(rG[rt][s] - dx[rt][s] * kh4[rt][s]);
                    rb[s] = sum16(rB[rt][s]);
                }
                if (n == 0) {
                    *reinterpret_cast<f32x4*>(&sm.rowG[w][sig0(rt) + 8 * g]) = rg;
                    *reinterpret_cast<f32x4*>(&sm.rowB[w][sig0(rt) + 8 * g]) = rb;
                }
            }
#pragma unroll
            for (int o = 32; o; o >>= 1) sumY += __shfl_xor(sumY, o);
            if (lane == 0) sm.sumY[w] = sumY;
        }
        lds_barrier();                     // V, T^T and P^T have been read
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int o = granule<128>(16 * w + n, 4 * j + g);
            *reinterpret_cast<u32x4*>(sU + o) = pack8(u[2 * j], u[2 * j + 1]);
            *reinterpret_cast<u32x4*>(sX + o) = pack8(dx[2 * j], dx[2 * j + 1]);
        }
        lds_barrier();

        // u dh'^T, then do h^T and dx h^T; after them h and dh' are not needed any more
        const int rn[2] = {32 * wr + n, 32 * wr + 16 + n};
        const float ga_n[2] = {sm.ga[rn[0]], sm.ga[rn[1]]};
        {
            const float eb[2] = {sm.E[rn[0]] * sm.beta[rn[0]], sm.E[rn[1]] * sm.beta[rn[1]]};
            f32x4 z[2][2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) z[i][j] = zero4();
            s16x8 df[2][2], uf[2][2];      // [turn][tile]
            auto read = [&](int ks) {
#pragma unroll
                for (int i = 0; i < 2; ++i) df[ks & 1][i] = down_sig<256>(L, G_DH, ks, 2 * wc + i);
#pragma unroll
                for (int j = 0; j < 2; ++j) uf[ks & 1][j] = down<128>(L, G_U, ks, 2 * wr + j);
            };
            read(0);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                if (ks < 3) read(ks + 1);
                sched_fence();
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) z[i][j] = mfma(df[ks & 1][i], uf[ks & 1][j], z[i][j]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) dk[i][j] += z[i][j] * eb[j];
        }
        {
            f32x4 t[2][2], y[2][2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) t[i][j] = y[i][j] = zero4();
            s16x8 hf[2][2], of[2][2], xf[2][2];
            auto read = [&](int ks) {
#pragma unroll
                for (int i = 0; i < 2; ++i) hf[ks & 1][i] = down_sig<256>(L, G_H, ks, 2 * wc + i);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    of[ks & 1][j] = row8<256>(L, G_DO, 2 * wr + j, ks);
                    xf[ks & 1][j] = down<128>(L, G_X, ks, 2 * wr + j);
                }
            };
            read(0);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                if (ks < 3) read(ks + 1);
                sched_fence();
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        t[i][j] = mfma(hf[ks & 1][i], of[ks & 1][j], t[i][j]);
                        y[i][j] = mfma(hf[ks & 1][i], xf[ks & 1][j], y[i][j]);
                    }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float s = 0.f;
                const s16x8 q8 = row8<256>(L, G_Q, 2 * wr + j, wc);
                const f32x4 q0 = widen_lo(q8), q1 = widen_hi(q8);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s = fmaf(t[0][j][e], q0[e], s);
                    s = fmaf(t[1][j][e], q1[e], s);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    dq[i][j] += t[i][j] * ga_n[j];
                    dk[i][j] -= y[i][j] * ga_n[j];
                }
                s += __shfl_xor(s, 16);
                s += __shfl_xor(s, 32);
                if (g == 0) sm.rowQ[wc][rn[j]] = s * ga_n[j];
            }
        }
        lds_barrier();                     // h and dh' have been read

        // dv = dx: row tile w % 4, dv columns 64 (w / 4) .. + 63, eight columns at a time from transposing reads of dx^T
        {
            const int r = 16 * (w & 3) + n;
            s16x8 v8[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) v8[j] = down<128>(L, G_X, 2 * (w >> 2) + j, w & 3);
            if (r < at.rows)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    *reinterpret_cast<s16x8*>(a.dv + ((at.row0 + r) * a.Hv + vh) * D + 64 * (w >> 2) + 32 * j + 8 * g) = v8[j];
        }
        // rows 16 ti .. + 15 of Zu or do u^T on and below the diagonal: N or dP o
        // Gam, and X's row and column sums
        {
            const bool isP = w >= 4;
            s16x8 af[4], uf[2][4];
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) af[ks] = isP ? row8<256>(L, G_DO, ti, ks) : down<128>(L, G_X, ks, ti);
            auto read = [&](int j) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) uf[j & 1][ks] = down<128>(L, G_U, ks, j);
            };
            read(0);
            const f32x4 Gr = *reinterpret_cast<const f32x4*>(sm.G + 16 * ti + 4 * g);
            f32x4 rx = zero4();
            byte* dst = isP ? sM : sN;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f32x4 t = zero4();
                const int c = 16 * j + n;
                float cx = 0.f, cz = 0.f;
                if (j <= ti) {
                    if (j < 3) read(j + 1);
                    sched_fence();
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) t = mfma(af[ks], uf[j & 1][ks], t);
                    const f32x4 bp = widen(bp4[j]);
                    const float bt = isP ? sm.beta[c] : -sm.beta[c], Gc = sm.G[c];
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const int r = 16 * ti + 4 * g + s;
                        // B's and, in the mask, P's entries from the diagonal on are zero
                        const float b = c < r ? bp[s] : 0.f, val = t[s] * bt;
                        cz = fmaf(b, t[s], cz);
                        rx[s] = fmaf(val, b, rx[s]);
                        cx = fmaf(val, b, cx);
                        t[s] = (isP ? c <= r : c < r) ? val * __builtin_amdgcn_exp2f(Gr[s] - Gc) : 0.f;
                    }
                }
                *reinterpret_cast<u32x2*>(dst + granule<128>(c, 2 * ti + (g >> 1)) + 8 * (g & 1)) = pack4(t);
                cx += __shfl_xor(cx, 16); cx += __shfl_xor(cx, 32);
                if (g == 0) sm.colX[w][c] = cx;
                if (!isP) {
                    cz += __shfl_xor(cz, 16); cz += __shfl_xor(cz, 32);
                    if (g == 0) sm.colZ[w][c] = cz;
                }
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const float v = sum16(rx[s]);
                if (n == 0) sm.rowX[isP][16 * ti + 4 * g + s] = v;
            }
        }
        lds_barrier();

        // (dP o Gam) K to dq; (dP o Gam)^T Q + (N + N^T) K to dk
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            s16x8 kf[2], qf[2], m0[2], m1[2], n0[2], n1[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                m0[j] = down<128>(L, G_DH + kSquare, ks, 2 * wr + j);
                n0[j] = down<128>(L, G_DH, ks, 2 * wr + j);
                n1[j] = row8<128>(L, G_DH, 2 * wr + j, ks);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) kf[i] = down_sig<256>(L, G_K, ks, 2 * wc + i);
#pragma unroll
            for (int j = 0; j < 2; ++j) m1[j] = row8<128>(L, G_DH + kSquare, 2 * wr + j, ks);
#pragma unroll
            for (int i = 0; i < 2; ++i) qf[i] = down_sig<256>(L, G_Q, ks, 2 * wc + i);
            sched_fence();
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    dq[i][j] = mfma(kf[i], m0[j], dq[i][j]);
                    dk[i][j] = mfma(kf[i], n0[j], dk[i][j]);
                }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) dk[i][j] = mfma(kf[i], n1[j], dk[i][j]);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) dk[i][j] = mfma(qf[i], m1[j], dk[i][j]);
        }
        // the gates' gradients
        if (w == 0) {
            float r = 0.f, bt = 0.f, cx = 0.f, cz = 0.f, Y = 0.f, hds = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                r += sm.rowG[i][lane];
                bt += sm.rowB[i][lane];
                Y += sm.sumY[i];
                hds += sm.hd[i];
                cx += sm.colX[i][lane];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                cz += sm.colZ[i][lane];
                r += sm.rowQ[i][lane];
            }
            float d = r + ((sm.rowX[0][lane] + sm.rowX[1][lane]) - cx);
            if (lane == C - 1) d += Y + sm.ga[C - 1] * hds;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const float up = __shfl_down(d, o);
                if (lane + o < 64) d += up;
            }
            if (lane < at.rows) {
                const int64_t row = (at.row0 + lane) * a.Hv + vh;
                a.dg[row] = f32_to_bf16_bits(d);
                a.db[row] = f32_to_bf16_bits(bt - cz);
            }
        }
    }
    const int g = (tid & 63) >> 4, n = tid & 15;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int r = 32 * wr + 16 * j + n;
        if constexpr (SPLIT) {
            const size_t o = ((size_t)x * a.Hv + vh0) * kState + 512 * r + 4 * (32 * wc + 8 * g);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                *reinterpret_cast<f32x4*>(a.h + o + 16 * i) = dq[i][j];
                *reinterpret_cast<f32x4*>(a.dh + o + 16 * i) = dk[i][j];
            }
        } else if (r < at.rows) {
            const int64_t o = ((at.row0 + r) * a.Hk + kh) * D + 32 * wc + 8 * g;
            *reinterpret_cast<u32x4*>(a.dq + o) = pack8(dq[0][j], dq[1][j]);
            *reinterpret_cast<u32x4*>(a.dk + o) = pack8(dk[0][j], dk[1][j]);
        }
    }
}

// dq (z = 0, 1) and dk (2, 3) of a k-head's chunk, 32 rows a workgroup: the parts of
// its v-heads, added in their order.
__global__ void __launch_bounds__(256)
gdn_bwd_sum_kernel(Args a)
{
    ChunkAt at;
    const int x = blockIdx.x, kh = blockIdx.y, rep = a.Hv / a.Hk, q = threadIdx.x & 7;
    if (!bwd::chunk_at(x, a.cu, a.base, a.B, a.T, a.nc_dense, &at)) return;
    const int r = 32 * (blockIdx.z & 1) + (threadIdx.x >> 3);
    if (r >= at.rows) return;
    const byte* p = (blockIdx.z < 2 ? a.h : a.dh) + ((size_t)x * a.Hv + (size_t)kh * rep) * kState + 512 * r + 64 * q;
    f32x4 t[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) t[e] = reinterpret_cast<const f32x4*>(p)[e];
    for (int i = 1; i < rep; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] += reinterpret_cast<const f32x4*>(p + (size_t)i * kState)[e];
    uint16_t* out = (blockIdx.z < 2 ? a.dq : a.dk) + ((at.row0 + r) * a.Hk + kh) * D + 16 * q;
    reinterpret_cast<u32x4*>(out)[0] = pack8(t[0], t[1]);
    reinterpret_cast<u32x4*>(out)[1] = pack8(t[2], t[3]);
}

// Whether the gradients' workgroups take one v-head each: where every v-head finds a
// compute unit (256) of its own, a k-head's v-heads need not wait for each other
// (8 chunks x 2 k-heads x 3 v-heads: 34 us whole, 15 + 4 with the sum). From there on
// the parts cost more than the turns: 8 x 16 x 3 takes 40 us whole and 37 + 5 split,
// 16 x 16 x 3 takes 50 and 61 + 9, 72 x 16 x 3 takes 239 and 270 + 42.
bool split_heads(int64_t chunks, int Hk, int Hv) { return Hv > Hk && chunks * Hv <= 256; }

struct Layout {
    size_t base, heads, h, dh, total;
};
Layout layout(int B, int T, int Hv, bool packed)
{
    const size_t n = (size_t)bwd::max_chunks(B, T, packed) * Hv;
    Layout l;
    size_t at = 0;
    l.base = at; at += bwd::round_up(packed ? (size_t)(B + 1) * sizeof(int32_t) : 0);
    l.heads = at; at += bwd::round_up(n * W_BYTES);
    l.h = at; at += bwd::round_up(n * kState);
    l.dh = at; at += bwd::round_up(n * kState);
    l.total = at;
    return l;
}

template <typename TA>
hipError_t launch_typed(const Args& k, int64_t chunks, hipStream_t s)
{
    hipError_t e;
    if ((e = allow_lds(reinterpret_cast<const void*>(gdn_bwd_prep_kernel<TA>), kPrepLds)) != hipSuccess) return e;
    if ((e = allow_lds(reinterpret_cast<const void*>(gdn_bwd_spine_kernel<TA>), kSpineLds)) != hipSuccess) return e;
    if ((e = allow_lds(reinterpret_cast<const void*>(gdn_bwd_grads_kernel<TA, false>), kGradLds)) != hipSuccess) return e;
    if ((e = allow_lds(reinterpret_cast<const void*>(gdn_bwd_grads_kernel<TA, true>), kGradLds)) != hipSuccess) return e;
    if (k.cu) hipLaunchKernelGGL(gdn_bwd_table_kernel, dim3(1), dim3(256), 0, s, k.cu, k.B, k.T, k.base);
    if (chunks > 0)
        hipLaunchKernelGGL((gdn_bwd_prep_kernel<TA>), dim3((unsigned)chunks, k.Hv), dim3(256), kPrepLds, s, k);
    hipLaunchKernelGGL((gdn_bwd_spine_kernel<TA>), dim3(k.Hv * 2, k.B, 2), dim3(kSpineThreads), kSpineLds, s, k);
    if (chunks > 0 && split_heads(chunks, k.Hk, k.Hv)) {
        hipLaunchKernelGGL((gdn_bwd_grads_kernel<TA, true>), dim3((unsigned)chunks, k.Hv), dim3(kGradThreads), kGradLds, s, k);
        hipLaunchKernelGGL(gdn_bwd_sum_kernel, dim3((unsigned)chunks, k.Hk, 4), dim3(256), 0, s, k);
    } else if (chunks > 0) {
        hipLaunchKernelGGL((gdn_bwd_grads_kernel<TA, false>), dim3((unsigned)chunks, k.Hk), dim3(kGradThreads), kGradLds, s, k);
    }
    return hipGetLastError();
}

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

const char* backward_mfma_refuses(const BackwardArgs& a)
{
    if (a.io_dtype == 0 || a.grad_dtype != 1) return "(generic: the MFMA route takes bf16 or 8-bit activations and bf16 gradients)";
    if (a.dk != D || a.dv != D) return "(generic: the MFMA route takes dk = dv = 128)";
    const size_t n = a.io_dtype == 2 ? 8 : 16;
    if (!aligned(a.q, n) || !aligned(a.k, n) || !aligned(a.v, n) || !aligned(a.dout, 16) || !aligned(a.dq, 16) ||
        !aligned(a.dk_out, 16) || !aligned(a.dv_out, 16))
        return "(generic: the MFMA route takes 16-byte aligned pointers)";
    return nullptr;
}

Geometry backward_mfma_geometry(const BackwardArgs& a)
{
    return Geometry{"gdn_bwd_prep_kernel+gdn_bwd_spine_kernel+gdn_bwd_grads_kernel",
                    {(unsigned)(a.Hv * 2), (unsigned)a.B, 2}, kSpineThreads, (unsigned)kSpineLds};
}

hipError_t launch_backward_mfma(const BackwardArgs& a, hipStream_t s)
{
    const Layout l = layout(a.B, a.T, a.Hv, a.cu != nullptr);
    byte* w = static_cast<byte*>(a.workspace);
    Args k{};
    k.q = a.q; k.k = a.k; k.v = a.v; k.dout = a.dout;
    k.q_exps = a.q_exps; k.k_exps = a.k_exps; k.v_exps = a.v_exps;
    k.log_g = a.log_g; k.beta = a.beta; k.h0 = a.h0; k.dht = a.dh_final;
    k.dq = static_cast<uint16_t*>(a.dq); k.dk = static_cast<uint16_t*>(a.dk_out); k.dv = static_cast<uint16_t*>(a.dv_out);
    k.dg = static_cast<uint16_t*>(a.dlog_g); k.db = static_cast<uint16_t*>(a.dbeta); k.dh0 = a.dh0;
    k.B = a.B; k.T = a.T; k.Hk = a.Hk; k.Hv = a.Hv; k.cu = a.cu;
    k.nc_dense = a.T > 0 ? (a.T + C - 1) / C : 1;
    k.base = reinterpret_cast<int32_t*>(w + l.base);
    k.heads = w + l.heads; k.h = w + l.h; k.dh = w + l.dh;
    const int64_t chunks = bwd::max_chunks(a.B, a.T, a.cu != nullptr);
    if (a.io_dtype == 1) return launch_typed<uint16_t>(k, chunks, s);
    return launch_typed<uint8_t>(k, chunks, s);
}

}  // namespace gdn
