// Gradients of the GDN recurrence (gdn_backward), chunk by chunk, in fp32.
//
// The recurrence per head, state H (dk x dv), scan order t = 1 .. T:
//     w_t = v_t - a_t H_{t-1}^T k_t,   u_t = b_t w_t,   H_t = a_t H_{t-1} + k_t u_t^T,   o_t = H_t^T q_t.
// Over a chunk of C = 64 tokens with entry state H0, G the running sum of log2 a in the chunk,
// D_ij = 2^(G_i - G_j) for j <= i, gam_i = 2^G_i, e_j = 2^(G_C - G_j):
//     X = strict-lower[D_ij k_i.k_j],  P = lower[D_ij q_i.k_j],  N = (I + X diag(b))^-1 X,
//     R = V - diag(gam) K H0,   W = R - N diag(b) R,   U = diag(b) W,
//     H1 = gam_C H0 + K^T diag(e) U.
// N serves both triangular inverses the gradients need: (I + X diag(b))^-1 = I - N diag(b) and
// (I + diag(b) X)^-1 = I - diag(b) N, and no division by b occurs, so b = 0 is an ordinary value.
// With dO and the gradient dH1 of the chunk's final state:
//     dU = P^T dO + diag(e) K dH1,   Z = dU - N^T diag(b) dU,   Y = diag(b) Z,
//     dH0 = gam_C dH1 + Q^T diag(gam) dO - K^T diag(gam) Y,
//     dV = Y,   db_i = Z_i . W_i,   dP = lower[dO U^T],   dX = -strict-lower[Y U^T],
//     E = dP o D,  F = dX o D,
//     dQ = diag(gam) dO H0^T + E K,
//     dK = (F + F^T) K + E^T Q - diag(gam) Y H0^T + diag(e) U dH1^T.
// The gradient of a decay is the sum of every product that contains it, divided by it: with
//     M_ij = dX_ij X_ij + dP_ij P_ij (j < i),  M_i0 = gam_i (q_i.H0 dO_i - k_i.H0 Y_i),
//     M_Ej = e_j k_j.dH1 U_j,  M_E0 = gam_C <H0, dH1>      (0: the entry, E: the end of the chunk)
//     da_t = (sum over i >= t, j < t of M_ij) / a_t.
// The sums are taken as prefix sums along j and then over i, never as differences, so a strong decay
// loses nothing to cancellation.
//
// Kernels: prepare (X, P, N of every chunk, all chunks at once); chains (two serial walks, forward for
// H0 and W, backward for dH1 and Z, which need nothing of one another and run side by side, each split
// over 32-column slices of dv, whose columns are independent); gradients (every chunk at once, both
// scan directions of a tile in one block, so that a bidirectional call's sums are rounded once).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int kC = 64;         // tokens per chunk
constexpr int kThreads = 256;
constexpr int kSl = 32;        // dv columns per slice
constexpr int kLdC = kC + 4;   // row pitch of 64-wide fp32 tiles in shared memory
constexpr int kLdS = kSl + 4;  // row pitch of 32-wide tiles

__device__ __forceinline__ float ldf(const float *p) { return *p; }
__device__ __forceinline__ float ldf(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void stf(float *p, float x) { *p = x; }
__device__ __forceinline__ void stf(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

struct BwdParams {
    const void *q, *k, *v, *dout;
    const float *beta, *decay, *state_in, *dstate;
    void *dq, *dk_, *dv_;
    float *dbeta, *ddecay, *dstate_in;
    // workspace of this launch's heads, one entry per (direction, head, chunk)
    float *X, *P, *N, *H0, *dH1, *W, *Z;
    int head0, heads;          // the heads [head0, head0 + heads) of B*H
    int BH, T, nc, dk, dv, dirs;
};

// A chunk of one scan: its tokens in scan order.  Chunks are tiles [64 c, 64 c + n) of the sequence for
// both directions; the reverse scan walks tiles and tokens downwards.
struct Tile {
    int dir, head, c, n;       // head: index in B*H
    size_t ws;                 // index of the (direction, head, chunk) entry in the workspace
    __device__ __forceinline__ int tok(int i) const { return c * kC + (dir ? n - 1 - i : i); }
};

__device__ __forceinline__ Tile make_tile(const BwdParams &p, int dir, int local_head, int c)
{
    Tile t;
    t.dir = dir;
    t.head = p.head0 + local_head;
    t.c = c;
    t.n = min(kC, p.T - c * kC);
    t.ws = ((size_t)dir * p.heads + local_head) * p.nc + c;
    return t;
}

// Gates of a tile: b, a (clamped as in the forward kernels; 1 behind the sequence's end, where b = 0) and the
// running sums of log2 a.  The sums are held in 64 bits: a strong decay brings them to several
// hundred within a chunk, where 32 bits would leave differences of neighbours 1e-5 off.
struct Gates {
    double G[kC];
    float a[kC], b[kC], gam[kC], e[kC];
};

__device__ __forceinline__ void load_gates(const BwdParams &p, const Tile &t, Gates &g)
{
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        double l[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = 2 * lane + h;
            float a = 1.f, b = 0.f;
            if (i < t.n) {
                const size_t at = (size_t)t.head * p.T + t.tok(i);
                a = fmaxf(p.decay[at], 7.52316385e-37f);   // 2^-120
                b = p.beta[at];
            }
            g.a[i] = a;
            g.b[i] = b;
            l[h] = (double)log2f(a);
        }
        double s = l[0] + l[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        const double end = __shfl_sync(0xffffffffu, s, 31);
        g.G[2 * lane] = s - l[1];
        g.G[2 * lane + 1] = s;
        g.gam[2 * lane] = exp2f((float)(s - l[1]));
        g.gam[2 * lane + 1] = exp2f((float)s);
        g.e[2 * lane] = exp2f((float)(end - (s - l[1])));
        g.e[2 * lane + 1] = exp2f((float)(end - s));
    }
}

// rows i < 64 of x (row length `len` in memory, columns [c0, c0 + COLS)), zero where there is nothing
template <int COLS, typename T>
__device__ __forceinline__ void load_rows(const T *x, int len, int c0, const Tile &t, int T_, float *dst, int ld)
{
    const T *base = x + (size_t)t.head * T_ * len + c0;
    for (int e = threadIdx.x; e < kC * COLS; e += kThreads) {
        const int i = e / COLS, j = e % COLS;
        dst[i * ld + j] = (i < t.n && c0 + j < len) ? ldf(base + (size_t)t.tok(i) * len + j) : 0.f;
    }
}

// acc[i][j] += sum_k A[m_i][k] B[k][n_j]  (TA: A[k][m_i]),  m_i = ty + TY i,  n_j = 4 tx + j;
// the block's threads are TX x TY with TX = N / 4.
template <int M, int N, bool TA, int RM>
__device__ __forceinline__ void gemm(float (&acc)[RM][4], const float *A, int lda, const float *B, int ldb, int K)
{
    constexpr int TX = N / 4, TY = kThreads / TX;
    static_assert(RM * TY == M, "tile");
    const int tx = threadIdx.x % TX, ty = threadIdx.x / TX;
    for (int k = 0; k < K; k += 4) {
        float4 b[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) b[u] = *reinterpret_cast<const float4 *>(B + (k + u) * ldb + 4 * tx);
#pragma unroll
        for (int i = 0; i < RM; ++i) {
            const int m = ty + TY * i;
            float a[4];
            if (TA) {
#pragma unroll
                for (int u = 0; u < 4; ++u) a[u] = A[(k + u) * lda + m];
            } else {
                const float4 x = *reinterpret_cast<const float4 *>(A + m * lda + k);
                a[0] = x.x; a[1] = x.y; a[2] = x.z; a[3] = x.w;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                acc[i][0] = fmaf(a[u], b[u].x, acc[i][0]);
                acc[i][1] = fmaf(a[u], b[u].y, acc[i][1]);
                acc[i][2] = fmaf(a[u], b[u].z, acc[i][2]);
                acc[i][3] = fmaf(a[u], b[u].w, acc[i][3]);
            }
        }
    }
}

template <int M, int N, int RM, typename F>
__device__ __forceinline__ void each(const float (&acc)[RM][4], F f)
{
    constexpr int TX = N / 4, TY = kThreads / TX;
    const int tx = threadIdx.x % TX, ty = threadIdx.x / TX;
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) f(ty + TY * i, 4 * tx + j, acc[i][j]);
}

template <int RM>
__device__ __forceinline__ void zero(float (&acc)[RM][4])
{
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
}

// ---------------------------------------------------------------- prepare
// X, P, N of one chunk: grid (chunks, heads, directions).
template <int DK>
struct PrepSmem {
    float K[kC * (DK + 4)];
    float Q[kC * (DK + 4)];
    float KT[DK * kLdC];
    float X[kC * kLdC];        // X, then X diag(b)
    float N[kC * kLdC];
    Gates g;
};

template <int DK, typename T>
__global__ void __launch_bounds__(kThreads) bwd_prepare_kernel(BwdParams p)
{
    extern __shared__ __align__(16) unsigned char raw[];
    PrepSmem<DK> &s = *reinterpret_cast<PrepSmem<DK> *>(raw);
    const Tile t = make_tile(p, blockIdx.z, blockIdx.y, blockIdx.x);
    constexpr int ld = DK + 4;
    load_gates(p, t, s.g);
    load_rows<DK>(static_cast<const T *>(p.k), p.dk, 0, t, p.T, s.K, ld);
    load_rows<DK>(static_cast<const T *>(p.q), p.dk, 0, t, p.T, s.Q, ld);
    __syncthreads();
    for (int e = threadIdx.x; e < kC * DK; e += kThreads) s.KT[(e / kC) * kLdC + e % kC] = s.K[(e % kC) * ld + e / kC];
    __syncthreads();
    float kk[4][4], qk[4][4];
    zero(kk);
    zero(qk);
    gemm<kC, kC, false>(kk, s.K, ld, s.KT, kLdC, DK);
    gemm<kC, kC, false>(qk, s.Q, ld, s.KT, kLdC, DK);
    float *Xg = p.X + t.ws * kC * kC, *Pg = p.P + t.ws * kC * kC, *Ng = p.N + t.ws * kC * kC;
    each<kC, kC>(kk, [&](int i, int j, float x) {
        const float y = j < i ? x * exp2f((float)(s.g.G[i] - s.g.G[j])) : 0.f;
        Xg[i * kC + j] = y;
        s.N[i * kLdC + j] = y;
        s.X[i * kLdC + j] = y * s.g.b[j];
    });
    each<kC, kC>(qk, [&](int i, int j, float x) {
        Pg[i * kC + j] = j <= i ? x * exp2f((float)(s.g.G[i] - s.g.G[j])) : 0.f;
    });
    __syncthreads();
    // N <- X - (X diag(b)) N in block rows of 16: the rows above by all threads, the 16 x 16 triangle by one
    // thread per column
    for (int r = 0; r < kC; r += 16) {
        for (int e = threadIdx.x; e < 16 * kC; e += kThreads) {
            const int i = r + e / kC, j = e % kC;
            float y = s.N[i * kLdC + j];
            for (int l = 0; l < r; ++l) y = fmaf(-s.X[i * kLdC + l], s.N[l * kLdC + j], y);
            s.N[i * kLdC + j] = y;
        }
        __syncthreads();
        if (threadIdx.x < kC) {
            const int j = threadIdx.x;
            float y[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                y[i] = s.N[(r + i) * kLdC + j];
#pragma unroll
                for (int l = 0; l < i; ++l) y[i] = fmaf(-s.X[(r + i) * kLdC + r + l], y[l], y[i]);
                s.N[(r + i) * kLdC + j] = y[i];
            }
        }
        __syncthreads();
    }
    for (int e = threadIdx.x; e < kC * kC; e += kThreads) Ng[e] = s.N[(e / kC) * kLdC + e % kC];
}

// ---------------------------------------------------------------- chains
// Grid (slices, heads, 2 directions-and-walks): the forward walk stores H0 and W of every chunk, the backward
// walk dH1 and Z.  The state slice (dk x 32) stays in registers and is mirrored in shared memory, where the
// products read it.
template <int DK>
struct ChainSmem {
    float K[kC * (DK + 4)];
    float Q[kC * (DK + 4)];    // backward walk
    float H[DK * kLdS];
    float V[kC * kLdS];        // V or dO
    float R[kC * kLdS];
    float S[kC * kLdS];        // second 64 x 32 operand
    float N[kC * kLdC];
    float P[kC * kLdC];
    Gates g;
};

template <int DK, typename T>
__global__ void __launch_bounds__(kThreads) bwd_chain_kernel(BwdParams p)
{
    extern __shared__ __align__(16) unsigned char raw[];
    ChainSmem<DK> &s = *reinterpret_cast<ChainSmem<DK> *>(raw);
    constexpr int ld = DK + 4, RH = DK / 32;
    const int dir = blockIdx.z >> 1, walk = blockIdx.z & 1, local = blockIdx.y, c0 = blockIdx.x * kSl;
    const int head = p.head0 + local;
    const size_t st = (size_t)p.dk * p.dv;
    float h[RH][4];
    zero(h);
    const float *init = nullptr;
    if (walk == 0 && dir == 0 && p.state_in) init = p.state_in + head * st;
    if (walk == 1 && p.dstate) init = p.dstate + ((size_t)dir * p.BH + head) * st;
    {
        const int tx = threadIdx.x % 8, ty = threadIdx.x / 8;
#pragma unroll
        for (int i = 0; i < RH; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (init && ty + 32 * i < p.dk) h[i][j] = init[(size_t)(ty + 32 * i) * p.dv + c0 + 4 * tx + j];
    }
    for (int step = 0; step < p.nc; ++step) {
        const int c = (dir ^ walk) ? p.nc - 1 - step : step;
        const Tile t = make_tile(p, dir, local, c);
        float *keep = (walk ? p.dH1 : p.H0) + t.ws * st + c0;
        each<DK, kSl>(h, [&](int i, int j, float x) {
            s.H[i * kLdS + j] = x;
            if (i < p.dk) keep[(size_t)i * p.dv + j] = x;
        });
        load_gates(p, t, s.g);
        load_rows<DK>(static_cast<const T *>(p.k), p.dk, 0, t, p.T, s.K, ld);
        load_rows<kSl>(static_cast<const T *>(walk ? p.dout : p.v), p.dv, c0, t, p.T, s.V, kLdS);
        if (walk) load_rows<DK>(static_cast<const T *>(p.q), p.dk, 0, t, p.T, s.Q, ld);
        const float *Ng = p.N + t.ws * kC * kC, *Pg = p.P + t.ws * kC * kC;
        for (int e = threadIdx.x; e < kC * kC; e += kThreads) {
            s.N[(e / kC) * kLdC + e % kC] = Ng[e];
            if (walk) s.P[(e / kC) * kLdC + e % kC] = Pg[e];
        }
        __syncthreads();
        float r[2][4], m[2][4];
        zero(r);
        gemm<kC, kSl, false>(r, s.K, ld, s.H, kLdS, DK);
        float *out = (walk ? p.Z : p.W) + t.ws * kC * p.dv + c0;
        const float gend = s.g.gam[kC - 1];
        if (walk == 0) {
            each<kC, kSl>(r, [&](int i, int j, float x) { s.R[i * kLdS + j] = s.V[i * kLdS + j] - s.g.gam[i] * x; });
            __syncthreads();
            each<kC, kSl>(r, [&](int i, int j, float) { s.S[i * kLdS + j] = s.g.b[i] * s.R[i * kLdS + j]; });
            __syncthreads();
            zero(m);
            gemm<kC, kSl, false>(m, s.N, kLdC, s.S, kLdS, kC);
            __syncthreads();
            each<kC, kSl>(m, [&](int i, int j, float x) {
                const float w = s.R[i * kLdS + j] - x;
                out[(size_t)i * p.dv + j] = w;
                s.S[i * kLdS + j] = s.g.e[i] * s.g.b[i] * w;
            });
            __syncthreads();
#pragma unroll
            for (int i = 0; i < RH; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) h[i][j] *= gend;
            gemm<DK, kSl, true>(h, s.K, ld, s.S, kLdS, kC);
        } else {
            zero(m);
            gemm<kC, kSl, true>(m, s.P, kLdC, s.V, kLdS, kC);
            each<kC, kSl>(r, [&](int i, int j, float x) { s.R[i * kLdS + j] = s.g.e[i] * x; });
            __syncthreads();
            each<kC, kSl>(m, [&](int i, int j, float x) {
                const float du = s.R[i * kLdS + j] + x;
                s.R[i * kLdS + j] = du;
                s.S[i * kLdS + j] = s.g.b[i] * du;
            });
            __syncthreads();
            zero(m);
            gemm<kC, kSl, true>(m, s.N, kLdC, s.S, kLdS, kC);
            __syncthreads();
            each<kC, kSl>(m, [&](int i, int j, float x) {
                const float z = s.R[i * kLdS + j] - x;
                out[(size_t)i * p.dv + j] = z;
                s.S[i * kLdS + j] = -s.g.gam[i] * s.g.b[i] * z;
                s.V[i * kLdS + j] *= s.g.gam[i];
            });
            __syncthreads();
#pragma unroll
            for (int i = 0; i < RH; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) h[i][j] *= gend;
            gemm<DK, kSl, true>(h, s.K, ld, s.S, kLdS, kC);
            gemm<DK, kSl, true>(h, s.Q, ld, s.V, kLdS, kC);
        }
        __syncthreads();
    }
    if (walk == 1 && dir == 0 && p.dstate_in) {
        float *out = p.dstate_in + head * st + c0;
        each<DK, kSl>(h, [&](int i, int j, float x) {
            if (i < p.dk) out[(size_t)i * p.dv + j] = x;
        });
    }
}

// ---------------------------------------------------------------- gradients
// Grid (chunks, heads).  Walks the slices of dv, summing dO H0^T, Y H0^T, U dH1^T (64 x dk) and dO U^T, Y U^T
// (64 x 64) in registers, then finishes dQ, dK and the gates.
template <int DK>
struct GradSmem {
    float K[kC * (DK + 4)];
    float Q[kC * (DK + 4)];
    float dq[kC * (DK + 4)];   // sums over the directions, rows by token
    float dk[kC * (DK + 4)];
    // during the walk: HT, GT (32 x dk: slices of H0 and dH1, transposed); behind it M (64 x 65)
    static constexpr int kHT = kSl * (DK + 4);
    float states[2 * kHT];
    // during the walk: dO, Y = diag(b) Z, U = diag(b) W (64 x 32 each) and U^T; behind it E, F (64 x 64)
    static constexpr int kRow = kC * kLdS;
    float rows[3 * kRow + kSl * kLdC];
    float m0[kC], m1[kC], db[2][kC], da[2][kC], red[kThreads / 32];
    Gates g;
};

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

template <int DK, typename T>
__global__ void __launch_bounds__(kThreads, 1) bwd_grad_kernel(BwdParams p)
{
    extern __shared__ __align__(16) unsigned char raw[];
    GradSmem<DK> &s = *reinterpret_cast<GradSmem<DK> *>(raw);
    static_assert(2 * kC * kLdC <= 3 * kC * kLdS + kSl * kLdC, "E and F fit in the slices' tiles");
    static_assert(kC * (kC + 1) <= 2 * kSl * (DK + 4), "M fits in the state tiles");
    float *const sHT = s.states, *const sGT = s.states + s.kHT, *const sM = s.states;
    float *const sO = s.rows, *const sY = s.rows + s.kRow, *const sU = s.rows + 2 * s.kRow;
    float *const sUT = s.rows + 3 * s.kRow, *const sE = s.rows, *const sF = s.rows + kC * kLdC;
    constexpr int ld = DK + 4, RG = kC * DK / 4 / kThreads;
    const size_t st = (size_t)p.dk * p.dv;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    for (int e = threadIdx.x; e < kC * ld; e += kThreads) s.dq[e] = s.dk[e] = 0.f;
    if (threadIdx.x < kC) s.db[1][threadIdx.x] = s.da[1][threadIdx.x] = 0.f;

    for (int dir = 0; dir < p.dirs; ++dir) {
        const Tile t = make_tile(p, dir, blockIdx.y, blockIdx.x);
        const float *H0 = p.H0 + t.ws * st, *dH1 = p.dH1 + t.ws * st;
        const float *Wg = p.W + t.ws * kC * p.dv, *Zg = p.Z + t.ws * kC * p.dv;
        __syncthreads();
        load_gates(p, t, s.g);
        load_rows<DK>(static_cast<const T *>(p.k), p.dk, 0, t, p.T, s.K, ld);
        load_rows<DK>(static_cast<const T *>(p.q), p.dk, 0, t, p.T, s.Q, ld);
        float hdo[RG][4], hy[RG][4], du1[RG][4], dp[4][4], dx[4][4];
        zero(hdo);
        zero(hy);
        zero(du1);
        zero(dp);
        zero(dx);
        float hh = 0.f, db[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) db[i] = 0.f;
        for (int c0 = 0; c0 < p.dv; c0 += kSl) {
            __syncthreads();
            load_rows<kSl>(static_cast<const T *>(p.dout), p.dv, c0, t, p.T, sO, kLdS);
            // one warp per row, one lane per column: the row's part of db = Z . W is a warp sum
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const int i = warp + 8 * r;
                const float w = Wg[(size_t)i * p.dv + c0 + lane], z = Zg[(size_t)i * p.dv + c0 + lane];
                const float b = s.g.b[i];
                sU[i * kLdS + lane] = b * w;
                sUT[lane * kLdC + i] = b * w;
                sY[i * kLdS + lane] = b * z;
                db[r] = fmaf(z, w, db[r]);
            }
            for (int e = threadIdx.x; e < DK * kSl; e += kThreads) {
                const int i = e / kSl, j = e % kSl;
                float x = 0.f, y = 0.f;
                if (i < p.dk) {
                    x = H0[(size_t)i * p.dv + c0 + j];
                    y = dH1[(size_t)i * p.dv + c0 + j];
                }
                sHT[j * ld + i] = x;
                sGT[j * ld + i] = y;
                hh = fmaf(x, y, hh);
            }
            __syncthreads();
            gemm<kC, DK, false>(hdo, sO, kLdS, sHT, ld, kSl);
            gemm<kC, DK, false>(hy, sY, kLdS, sHT, ld, kSl);
            gemm<kC, DK, false>(du1, sU, kLdS, sGT, ld, kSl);
            gemm<kC, kC, false>(dp, sO, kLdS, sUT, kLdC, kSl);
            gemm<kC, kC, false>(dx, sY, kLdS, sUT, kLdC, kSl);
            // dv = Y: a bidirectional call adds the second direction to what the first one keeps in Z
            for (int e = threadIdx.x; e < kC * kSl; e += kThreads) {
                const int i = e / kSl, j = e % kSl;
                if (i >= t.n) continue;
                const size_t at = ((size_t)t.head * p.T + t.tok(i)) * p.dv + c0 + j;
                float y = sY[i * kLdS + j];
                if (dir == 1) {
                    const Tile f = make_tile(p, 0, blockIdx.y, blockIdx.x);
                    const float b = p.beta[(size_t)t.head * p.T + t.tok(i)];
                    y += b * p.Z[f.ws * kC * p.dv + (size_t)(t.n - 1 - i) * p.dv + c0 + j];
                }
                if (dir == p.dirs - 1) stf(static_cast<T *>(p.dv_) + at, y);
            }
        }
        const float *Xg = p.X + t.ws * kC * kC, *Pg = p.P + t.ws * kC * kC;
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const float x = warp_sum(db[r]);
            if (lane == 0) s.db[0][warp + 8 * r] = x;
        }
        hh = warp_sum(hh);
        if (lane == 0) s.red[warp] = hh;
        each<kC, kC>(dp, [&](int i, int j, float x) {
            const bool on = j <= i;
            sE[i * kLdC + j] = on ? x * exp2f((float)(s.g.G[i] - s.g.G[j])) : 0.f;
            sM[i * (kC + 1) + j] = j < i ? x * Pg[i * kC + j] : 0.f;
        });
        each<kC, kC>(dx, [&](int i, int j, float x) {
            sF[i * kLdC + j] = j < i ? -x * exp2f((float)(s.g.G[i] - s.g.G[j])) : 0.f;
            if (j < i) sM[i * (kC + 1) + j] -= x * Xg[i * kC + j];
        });
        // m0_i = gam_i (q_i . hdo_i - k_i . hy_i), m1_i = e_i k_i . du1_i: sums over the row's threads
        {
            constexpr int TX = DK / 4, TY = kThreads / TX;
            const int tx = threadIdx.x % TX, ty = threadIdx.x / TX;
#pragma unroll
            for (int i = 0; i < RG; ++i) {
                const int m = ty + TY * i;
                float x = 0.f, y = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float k = s.K[m * ld + 4 * tx + j];
                    x = fmaf(s.Q[m * ld + 4 * tx + j], hdo[i][j], x);
                    x = fmaf(-k, hy[i][j], x);
                    y = fmaf(k, du1[i][j], y);
                    hdo[i][j] *= s.g.gam[m];
                    hy[i][j] = s.g.e[m] * du1[i][j] - s.g.gam[m] * hy[i][j];
                }
#pragma unroll
                for (int o = TX / 2; o; o >>= 1) {
                    x += __shfl_xor_sync(0xffffffffu, x, o);
                    y += __shfl_xor_sync(0xffffffffu, y, o);
                }
                if (tx == 0) {
                    s.m0[m] = s.g.gam[m] * x;
                    s.m1[m] = s.g.e[m] * y;
                }
            }
        }
        __syncthreads();
        gemm<kC, DK, false>(hdo, sE, kLdC, s.K, ld, kC);
        gemm<kC, DK, true>(hy, sE, kLdC, s.Q, ld, kC);
        gemm<kC, DK, false>(hy, sF, kLdC, s.K, ld, kC);
        gemm<kC, DK, true>(hy, sF, kLdC, s.K, ld, kC);
        each<kC, DK>(hdo, [&](int i, int j, float x) {
            if (i < t.n) s.dq[(t.tok(i) - t.c * kC) * ld + j] += x;
        });
        each<kC, DK>(hy, [&](int i, int j, float x) {
            if (i < t.n) s.dk[(t.tok(i) - t.c * kC) * ld + j] += x;
        });
        // prefix sums along j from the entry, one thread per row; then sums over the rows i >= t
        if (threadIdx.x < kC) {
            const int i = threadIdx.x;
            float x = s.m0[i];
            for (int j = 0; j < i; ++j) {
                const float y = sM[i * (kC + 1) + j];
                sM[i * (kC + 1) + j] = x;      // the sum over columns before token j (0-based)
                x += y;
            }
            sM[i * (kC + 1) + i] = x;
        }
        __syncthreads();
        if (threadIdx.x < kC) {
            const int u = threadIdx.x;
            float x = 0.f;
            for (int w = 0; w < kThreads / 32; ++w) x += s.red[w];
            x *= s.g.gam[kC - 1];
            for (int j = 0; j < u; ++j) x += s.m1[j];
            for (int i = kC - 1; i >= u; --i) x += sM[i * (kC + 1) + u];
            if (u < t.n) {
                const int at = t.tok(u) - t.c * kC;
                s.da[1][at] += x / s.g.a[u];
                s.db[1][at] += s.db[0][u];
            }
        }
    }
    __syncthreads();
    const int head = p.head0 + blockIdx.y, base = blockIdx.x * kC, n = min(kC, p.T - base);
    for (int e = threadIdx.x; e < n * p.dk; e += kThreads) {
        const int i = e / p.dk, j = e % p.dk;
        const size_t at = ((size_t)head * p.T + base + i) * p.dk + j;
        stf(static_cast<T *>(p.dq) + at, s.dq[i * ld + j]);
        stf(static_cast<T *>(p.dk_) + at, s.dk[i * ld + j]);
    }
    if (threadIdx.x < n) {
        const size_t at = (size_t)head * p.T + base + threadIdx.x;
        p.dbeta[at] = s.db[1][threadIdx.x];
        p.ddecay[at] = s.da[1][threadIdx.x];
    }
}

template <typename F>
cudaError_t launch(F kernel, dim3 grid, size_t smem, const BwdParams &p, cudaStream_t stream)
{
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess) return err;
    kernel<<<grid, kThreads, smem, stream>>>(p);
    err = cudaGetLastError();
    if (err == cudaSuccess) count_launches(1);
    return err;
}

template <int DK, typename T>
cudaError_t run(const BwdParams &p, cudaStream_t stream)
{
    cudaError_t err = launch(bwd_prepare_kernel<DK, T>, dim3(p.nc, p.heads, p.dirs), sizeof(PrepSmem<DK>), p, stream);
    if (err == cudaSuccess)
        err = launch(bwd_chain_kernel<DK, T>, dim3(p.dv / kSl, p.heads, 2 * p.dirs), sizeof(ChainSmem<DK>), p, stream);
    if (err == cudaSuccess) err = launch(bwd_grad_kernel<DK, T>, dim3(p.nc, p.heads), sizeof(GradSmem<DK>), p, stream);
    return err;
}

// The workspace holds both chains' states of every chunk of the heads that one pass takes; passes are cut so
// that it stays under this, unless one head alone needs more.
constexpr size_t kMaxWorkspace = (size_t)6 << 30;

}  // namespace

cudaError_t launch_backward(const BwdArgs &a, cudaStream_t stream)
{
    BwdParams p;
    p.q = a.f.q; p.k = a.f.k; p.v = a.f.v; p.dout = a.dout;
    p.beta = a.f.beta; p.decay = a.f.decay; p.state_in = a.f.state_in; p.dstate = a.dstate;
    p.dq = a.dq; p.dk_ = a.dk; p.dv_ = a.dv; p.dbeta = a.dbeta; p.ddecay = a.ddecay; p.dstate_in = a.dstate_in;
    p.BH = a.f.B * a.f.H; p.T = a.f.T; p.nc = (a.f.T + kC - 1) / kC; p.dk = a.f.dk; p.dv = a.f.dv;
    p.dirs = a.f.bidi ? 2 : 1;
    const size_t sq = kC * kC, st = (size_t)p.dk * p.dv, rows = (size_t)kC * p.dv;
    const size_t per_head = (3 * sq + 2 * st + 2 * rows) * p.nc * p.dirs * sizeof(float);
    const int most = (int)std::min<size_t>((size_t)p.BH, std::max<size_t>(1, kMaxWorkspace / per_head));
    const int passes = (p.BH + most - 1) / most, each_pass = (p.BH + passes - 1) / passes;
    float *ws = nullptr;
    cudaError_t err = ws_alloc(reinterpret_cast<void **>(&ws), per_head * each_pass, stream);
    if (err != cudaSuccess) return err;
    for (int h = 0; h < p.BH && err == cudaSuccess; h += each_pass) {
        p.head0 = h;
        p.heads = std::min(each_pass, p.BH - h);
        const size_t n = (size_t)p.nc * p.dirs * p.heads;
        p.X = ws;
        p.P = p.X + n * sq;
        p.N = p.P + n * sq;
        p.H0 = p.N + n * sq;
        p.dH1 = p.H0 + n * st;
        p.W = p.dH1 + n * st;
        p.Z = p.W + n * rows;
        if (a.f.fp32) err = p.dk <= 64 ? run<64, float>(p, stream) : run<128, float>(p, stream);
        else err = p.dk <= 64 ? run<64, __nv_bfloat16>(p, stream) : run<128, __nv_bfloat16>(p, stream);
    }
    const cudaError_t e2 = ws_free(ws, stream);
    return err != cudaSuccess ? err : e2;
}

}  // namespace gdn
