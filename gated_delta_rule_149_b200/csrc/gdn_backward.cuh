// What the kernels of gdn_backward share: the workspace's layout, the three-term bf16 form of fp32 values, swizzled
// tiles, and tensor-core products over terms.  The mathematics is at the top of gdn_backward.cu.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gdn_internal.h"
#include "sm100_ptx.cuh"

namespace gdn {
namespace bwd {

constexpr int kC = 64;             // tokens per chunk
constexpr int kSlice = 32;         // dv columns of a V or dO tile
constexpr int kTri = kC * kC * 2;  // bytes of one term plane of N or P

__device__ __forceinline__ float ldf(const float *p) { return *p; }
__device__ __forceinline__ float ldf(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st2(float *p, float x, float y) { *reinterpret_cast<float2 *>(p) = make_float2(x, y); }
__device__ __forceinline__ void st2(__nv_bfloat16 *p, float x, float y)
{
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(x, y);
}

// Gates of a chunk in scan order, as prepare leaves them for the other kernels.  a is clamped as in the
// forward kernels; behind the sequence's end a = 1 and b = 0.  The running sums G of log2 a are formed in 64 bits and
// held as a whole number and a fraction in [-1/2, 1/2]: a strong decay brings them to several hundred within a chunk,
// where one float would leave 2^G 1e-5 off.  2^(G_i - G_j) adds 2^-22 to what the logarithms
// are off, and is 0 under 2^-126.

// 2^(n + f), |f| <= 1
__device__ __forceinline__ float power2(int n, float f)
{
    float x;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(x) : "f"(f));
    return x * __int_as_float((min(max(n, -127), 128) + 127) << 23);
}

struct Gates {
    float gam[kC], e[kC], b[kC], a[kC];
    int whole[kC];
    float frac[kC];
    // 2^shift D_ij = 2^(G_i - G_j + shift) for j <= i, and 2^shift gam_i
    __device__ __forceinline__ float decay(int i, int j, int shift = 0) const { return power2(whole[i] - whole[j] + shift, frac[i] - frac[j]); }
    __device__ __forceinline__ float from_entry(int i, int shift) const { return power2(whole[i] + shift, frac[i]); }
};

// log2 of a decay (no less than 2^-120, or not finite): the exponent exactly, and a fraction of at most 1/2, which log2f
// leaves 2^-25 off.  log2f of the whole would leave 1e-5 of a decay of 1e-35.
__device__ __forceinline__ double log2_of(float a)
{
    const int bits = __float_as_int(a);
    int n = (bits >> 23) - 127;
    float m = __int_as_float((bits & 0x7fffff) | 0x3f800000);
    if (n == 128) return (double)a;
    if (m > 1.41421356f) {
        m *= 0.5f;
        ++n;
    }
    return (double)n + (double)log2f(m);
}

// The products that a decay's gradient sums up (M) are the size of the decay, down to 2^-120 of the gradients given, and
// would leave fp32's range before the division by it.  A chunk with a decay under 2^-40 holds them 2^60 times larger (an
// exact factor): 24 bits then down to given gradients of 2^-42 at a decay of 2^-120, and of 2^-62 where none is under
// 2^-40, without bringing products of ordinary decays, up to 2^67, out of range at the other end.
struct Lift {
    int shift;
    float up, down;
};
// by whole warps
__device__ __forceinline__ Lift lift_of(const Gates &g)
{
    const int lane = threadIdx.x & 31;
    const bool strong = __any_sync(0xffffffffu, fminf(g.a[lane], g.a[lane + 32]) < 0x1p-40f);
    return strong ? Lift{60, 0x1p60f, 0x1p-60f} : Lift{0, 1.f, 1.f};
}

// Workspace of one (direction, head, chunk), in bytes.  Tiles are row-major with the 16-byte pieces of a
// row XOR-ed by the row's number, so that eight rows' pieces of one column lie in eight bank groups.
template <int DK, int NI>
struct Unit {
    static constexpr size_t kKey = (size_t)kC * DK * 2;    // one term plane of K or Q
    static constexpr size_t gates = 0;
    static constexpr size_t N = sizeof(Gates);             // three planes [i][j]
    static constexpr size_t K = N + 3 * kTri;              // NI planes [token][dk]
    static constexpr size_t Q = K + NI * kKey;
    static constexpr size_t P = Q + NI * kKey;             // three planes [i][j]
    static constexpr size_t size = P + 3 * kTri;
    static_assert(N % 128 == 0 && size % 128 == 0, "tiles start on 128-byte boundaries");
};

struct BwdParams {
    const void *q, *k, *v, *dout;
    const float *beta, *decay, *state_in, *dstate;
    void *dq, *dk_, *dv_;
    float *dbeta, *ddecay, *dstate_in;
    // workspace of this launch's heads, one entry per (direction, head, chunk)
    unsigned char *unit;       // Unit<DK, NI>
    unsigned char *vt;         // [slice][64 tokens][32 columns] of the input type
    unsigned char *ot;         // [slice][NI planes][64 tokens][32 columns]
    float *HT, *GT;            // [dv][DK]: H0 and dH1, transposed
    float *WT, *ZT;            // [dv][64 tokens]
    int head0, heads;          // the heads [head0, head0 + heads) of B*H
    int BH, T, nc, dk, dv, dirs, slices;
    int *err;                  // the device error word of bounded waits
    int stall;                 // testing: the first waits of head 0's walks and of the first chunk's gradients run out
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

// ---------------------------------------------------------------- terms, fragments, products
// two values as packed bf16 pairs (x in the low half): terms of x and y
template <int NT>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&out)[NT])
{
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
        out[t] = *reinterpret_cast<const uint32_t *>(&v);
        if (t + 1 < NT) {
            x -= __uint_as_float(out[t] << 16);
            y -= __uint_as_float(out[t] & 0xffff0000u);
        }
    }
}

__device__ __forceinline__ float lo16(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi16(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// byte offset of the 16-byte piece `piece` of row `row` in a swizzled tile with RB-byte rows.  kHalves: 64 rows of 256
// bytes as two tiles of 128-byte rows, columns 0 - 63 and 64 - 127 (the widest row a tcgen05 operand tile can have).
constexpr int kHalves = 512;
template <int RB>
__device__ __forceinline__ uint32_t sw(int row, int piece)
{
    if (RB == kHalves) return (piece >> 3) * (kC * 128) + row * 128 + (((piece & 7) ^ (row & 7)) << 4);
    return row * RB + ((piece ^ (RB == 64 ? (row >> 1) & 3 : row & 7)) << 4);
}
template <int DK> constexpr int kKeyRow = DK == 128 ? kHalves : DK * 2;   // the layout of a plane of K or Q

__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// c += A B.  The tensor core's fp32 sums are truncated, not rounded.
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Fragments of a 16 x 16 block of a tile at shared address `tile`.  A from [m][k] storage, A from [k][m] storage; B
// (two n8 halves: r[0], r[1] and r[2], r[3]) from [n][k] storage, B from [k][n] storage.
template <int RB>
__device__ __forceinline__ void frag_a(uint32_t (&r)[4], uint32_t tile, int m, int k)
{
    const int l = threadIdx.x & 31;
    ldsm(r, tile + sw<RB>(m + (l & 15), (k >> 3) + (l >> 4)));
}
template <int RB>
__device__ __forceinline__ void frag_at(uint32_t (&r)[4], uint32_t tile, int m, int k)
{
    const int l = threadIdx.x & 31;
    ldsm_t(r, tile + sw<RB>(k + (l & 7) + ((l >> 4) << 3), (m >> 3) + ((l >> 3) & 1)));
}
template <int RB>
__device__ __forceinline__ void frag_b(uint32_t (&r)[4], uint32_t tile, int k, int n)
{
    const int l = threadIdx.x & 31;
    ldsm(r, tile + sw<RB>(n + (l & 7) + ((l >> 4) << 3), (k >> 3) + ((l >> 3) & 1)));
}
template <int RB>
__device__ __forceinline__ void frag_bt(uint32_t (&r)[4], uint32_t tile, int k, int n)
{
    const int l = threadIdx.x & 31;
    ldsm_t(r, tile + sw<RB>(k + (l & 15), (n >> 3) + (l >> 4)));
}

// c (m16 x 16 G: 2 G tiles of n8) += the sum of KS products A B over the terms: products of order i + j < 3 (one term
// each: 0), the small ones first and all into sums of their own, which an ordinary addition, rounded to nearest, adds to
// c: the truncation of the tensor core's sums then touches every 16 KS products once and does not pile up over k.  The
// 2 G sums are independent; a product waits for the one before it in its own sum only.
template <int G, int KS, int NA, int NB>
__device__ __forceinline__ void mma_terms(float (*c)[4], const uint32_t (&a)[KS][NA][4], const uint32_t (&b)[G][KS][NB][4])
{
    float d[2 * G][4] = {};
#pragma unroll
    for (int order = NA + NB - 2 < 2 ? NA + NB - 2 : 2; order >= 0; --order)
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int i = 0; i < NA; ++i) {
                const int j = order - i;
                if (j < 0 || j >= NB) continue;
#pragma unroll
                for (int n = 0; n < G; ++n) {
                    mma(d[2 * n], a[k][i], b[n][k][j][0], b[n][k][j][1]);
                    mma(d[2 * n + 1], a[k][i], b[n][k][j][2], b[n][k][j][3]);
                }
            }
#pragma unroll
    for (int n = 0; n < 2 * G; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) c[n][x] += d[n][x];
}

// the same for one product of one n16 block
template <int NA, int NB>
__device__ __forceinline__ void mma_terms(float (*c)[4], const uint32_t (&a)[NA][4], const uint32_t (&b)[NB][4])
{
    mma_terms<1, 1, NA, NB>(c, reinterpret_cast<const uint32_t (&)[1][NA][4]>(a), reinterpret_cast<const uint32_t (&)[1][1][NB][4]>(b));
}

// the left operand whose columns k .. k + 15 are the accumulator tiles x, y times per-column factors
// f[0..1] (columns 2 t, 2 t + 1 of x) and f[2..3] (of y)
template <int NT>
__device__ __forceinline__ void acc_to_a(uint32_t (&a)[NT][4], const float (&x)[4], const float (&y)[4], const float (&f)[4])
{
    uint32_t u[NT];
    split2<NT>(x[0] * f[0], x[1] * f[1], u);
#pragma unroll
    for (int t = 0; t < NT; ++t) a[t][0] = u[t];
    split2<NT>(x[2] * f[0], x[3] * f[1], u);
#pragma unroll
    for (int t = 0; t < NT; ++t) a[t][1] = u[t];
    split2<NT>(y[0] * f[2], y[1] * f[3], u);
#pragma unroll
    for (int t = 0; t < NT; ++t) a[t][2] = u[t];
    split2<NT>(y[2] * f[2], y[3] * f[3], u);
#pragma unroll
    for (int t = 0; t < NT; ++t) a[t][3] = u[t];
}

__device__ __forceinline__ void copy16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void copy_tile(uint32_t dst, const unsigned char *src, int bytes, int threads)
{
    for (int o = threadIdx.x * 16; o < bytes; o += threads * 16) copy16(dst + o, src + o);
}

__device__ __forceinline__ void copy_block(uint32_t dst, const unsigned char *src, int bytes)
{
    copy_tile(dst, src, bytes, blockDim.x);
}

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// 8 floats to term planes in a swizzled tile
template <int RB>
__device__ __forceinline__ void planes8(const float (&x)[8], int row, int piece, unsigned char *to, int plane)
{
    uint32_t w[3][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t u[3];
        split2<3>(x[2 * i], x[2 * i + 1], u);
#pragma unroll
        for (int t = 0; t < 3; ++t) w[t][i] = u[t];
    }
#pragma unroll
    for (int t = 0; t < 3; ++t)
        *reinterpret_cast<uint4 *>(to + t * plane + sw<RB>(row, piece)) = make_uint4(w[t][0], w[t][1], w[t][2], w[t][3]);
}

__device__ __forceinline__ void get8f(const float *p, float (&x)[8])
{
    const float4 u = reinterpret_cast<const float4 *>(p)[0], v = reinterpret_cast<const float4 *>(p)[1];
    x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
    x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
}

// The gradients kernel for bf16, dk of 96 or 128: on tcgen05 tensor cores (gdn_backward_tc.cu).
cudaError_t launch_grad_tc(const BwdParams &p, cudaStream_t stream);
cudaError_t set_wait_limit_tc(unsigned long long ns);   // of this kernel's module

}  // namespace bwd
}  // namespace gdn
