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
// Products run on the tensor cores with bf16 operands and fp32 sums, at fp32 grade: an fp32 operand is three bf16
// terms, x = h + m + l (24 bits of significand), and of the products of terms those of total order under three are
// taken; a bf16 input is one term and exact.  Two terms would halve the products and leave 3e-6 (rel-L2) in the fp32
// gradients where three leave 2e-7.
//
// Kernels:
// * prepare (a block per chunk and direction): brings K, Q, V, dO into scan order as term planes in the
//   layout that the other two load without conversion, forms N and P likewise.
// * chains (two serial walks, forward for H0 and W, backward for dH1 and Z, which need nothing of one another
//   and run side by side): the columns of dv are independent, and two or four warps carry 16 of them through the
//   whole sequence.  They hold H^T (16 x dk) as accumulator fragments, which are, split into terms, the left
//   operands of the next product; so no state goes through shared memory, only sums over dk and over tokens meet
//   there, and the block's barrier paces the double-buffered operands.
// * gradients (a block per chunk, both scan directions, so that a bidirectional call's sums are rounded once).
#include <algorithm>
#include <cstdint>

#include "gdn_backward.cuh"
#include "gdn_chunk_common.cuh"

namespace gdn {

extern int g_stall_chunk;      // gdn_debug_stall

namespace {

using namespace bwd;

// ---------------------------------------------------------------- prepare
// Grid (chunks, heads, directions), 256 threads.
template <int DK, int NI>
struct PrepSmem {
    struct Keys {
        unsigned char K[NI * Unit<DK, NI>::kKey];
        unsigned char Q[NI * Unit<DK, NI>::kKey];
    };
    struct Solve {
        float X[kC * (kC + 4)];    // X diag(b)
        float N[kC * (kC + 4)];
        float inv[4 * 16 * 20];    // the inverses of the 16 x 16 diagonal blocks of I + X diag(b)
        float rows[16 * (kC + 4)];
    };
    union {                        // K and Q are done with when X is there: small blocks, four to an SM
        Keys k;
        Solve n;
    };
    Gates g;
};

constexpr int kPrepThreads = 256;

// eight values of a row as term planes in a swizzled tile (and its copy in the workspace)
template <int NI, int RB, typename T>
__device__ __forceinline__ void put8(const float (&x)[8], int row, int piece, unsigned char *smem, unsigned char *ws, size_t plane)
{
    uint32_t w[NI][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t u[NI];
        split2<NI>(x[2 * i], x[2 * i + 1], u);
#pragma unroll
        for (int t = 0; t < NI; ++t) w[t][i] = u[t];
    }
    const uint32_t o = sw<RB>(row, piece);
#pragma unroll
    for (int t = 0; t < NI; ++t) {
        const uint4 v = make_uint4(w[t][0], w[t][1], w[t][2], w[t][3]);
        if (smem) *reinterpret_cast<uint4 *>(smem + t * plane + o) = v;
        *reinterpret_cast<uint4 *>(ws + t * plane + o) = v;
    }
}

// eight consecutive values of a row of `len`, zero behind its end (len is a multiple of 32)
template <typename T>
__device__ __forceinline__ void get8(const T *row, bool on, int c, int len, float (&x)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
    if (!on || c >= len) return;
    if constexpr (sizeof(T) == 2) {
        const uint4 u = __ldg(reinterpret_cast<const uint4 *>(row + c));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = lo16(w[i]);
            x[2 * i + 1] = hi16(w[i]);
        }
    } else {
        const float4 u = __ldg(reinterpret_cast<const float4 *>(row + c)), v = __ldg(reinterpret_cast<const float4 *>(row + c) + 1);
        x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
        x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
    }
}

template <int DK, int NI, typename T>
__global__ void __launch_bounds__(kPrepThreads, NI == 1 ? 4 : 1) bwd_prepare_kernel(const __grid_constant__ BwdParams p)
{
    extern __shared__ __align__(128) unsigned char raw[];
    using U = Unit<DK, NI>;
    PrepSmem<DK, NI> &s = *reinterpret_cast<PrepSmem<DK, NI> *>(raw);
    constexpr int ld = kC + 4;
    const Tile t = make_tile(p, blockIdx.z, blockIdx.y, blockIdx.x);
    unsigned char *unit = p.unit + t.ws * U::size;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    auto gates = [&] {
        if (warp == 0) {
            double l[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = 2 * lane + h;
                float a = 1.f, b = 0.f;
                if (i < t.n) {
                    const size_t at = (size_t)t.head * p.T + t.tok(i);
                    a = p.decay[at];
                    a = a < 7.52316385e-37f ? 7.52316385e-37f : a;   // 2^-120; a NaN stays one
                    b = p.beta[at];
                }
                s.g.a[i] = a;
                s.g.b[i] = b;
                l[h] = log2_of(a);
            }
            double sum = l[0] + l[1];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double y = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += y;
            }
            const double end = __shfl_sync(0xffffffffu, sum, 31), G[2] = {sum - l[1], sum};
            const double end_whole = rint(end);
            const float end_frac = (float)(end - end_whole);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const double whole = rint(G[h]);
                const int n = (int)whole;
                const float f = (float)(G[h] - whole);
                s.g.whole[2 * lane + h] = n;
                s.g.frac[2 * lane + h] = f;
                s.g.gam[2 * lane + h] = power2(n, f);
                s.g.e[2 * lane + h] = power2((int)end_whole - n, end_frac - f);
            }
        }
    };
    const T *kb = static_cast<const T *>(p.k) + (size_t)t.head * p.T * p.dk;
    const T *qb = static_cast<const T *>(p.q) + (size_t)t.head * p.T * p.dk;
    const T *vb = static_cast<const T *>(p.v) + (size_t)t.head * p.T * p.dv;
    const T *ob = static_cast<const T *>(p.dout) + (size_t)t.head * p.T * p.dv;
    unsigned char *const ot = p.ot + t.ws * p.slices * (NI * kC * 64), *const vt = p.vt + t.ws * p.slices * (kC * kSlice * sizeof(T));
    if constexpr (NI == 1) {
        // bf16 is its own term: the pieces move as they are, all loads of a tensor pair in flight together
        auto piece = [&](const T *x, int len, int i, int c) {
            return i < t.n && c < len ? __ldg(reinterpret_cast<const uint4 *>(x + (size_t)t.tok(i) * len + c)) : make_uint4(0, 0, 0, 0);
        };
        constexpr int IT = kC * DK / 8 / kPrepThreads;
        uint4 x[4], y[4];
#pragma unroll
        for (int u = 0; u < IT; ++u) {
            const int e = tid + u * kPrepThreads, i = e / (DK / 8), c = e % (DK / 8);
            x[u] = piece(kb, p.dk, i, 8 * c);
            y[u] = piece(qb, p.dk, i, 8 * c);
        }
        gates();                                               // beside the loads
#pragma unroll
        for (int u = 0; u < IT; ++u) {
            const int e = tid + u * kPrepThreads;
            const uint32_t o = sw<kKeyRow<DK>>(e / (DK / 8), e % (DK / 8));
            *reinterpret_cast<uint4 *>(s.k.K + o) = x[u];
            *reinterpret_cast<uint4 *>(s.k.Q + o) = y[u];
            *reinterpret_cast<uint4 *>(unit + U::K + o) = x[u];
            *reinterpret_cast<uint4 *>(unit + U::Q + o) = y[u];
        }
        const int i = tid >> 2, c = tid & 3;
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (u < p.slices) {
                x[u] = piece(ob, p.dv, i, u * kSlice + 8 * c);
                y[u] = piece(vb, p.dv, i, u * kSlice + 8 * c);
            }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (u < p.slices) {
                *reinterpret_cast<uint4 *>(ot + u * (kC * 64) + sw<64>(i, c)) = x[u];
                *reinterpret_cast<uint4 *>(vt + u * (kC * 64) + sw<64>(i, c)) = y[u];
            }
    } else {
        gates();
        for (int e = tid; e < kC * (DK / 8); e += kPrepThreads) {
            const int i = e / (DK / 8), c = e % (DK / 8);
            const bool on = i < t.n;
            const size_t row = on ? (size_t)t.tok(i) * p.dk : 0;
            float x[8], y[8];
            get8(kb + row, on, 8 * c, p.dk, x);
            get8(qb + row, on, 8 * c, p.dk, y);
            put8<NI, kKeyRow<DK>, T>(x, i, c, s.k.K, unit + U::K, U::kKey);
            put8<NI, kKeyRow<DK>, T>(y, i, c, s.k.Q, unit + U::Q, U::kKey);
        }
        for (int e = tid; e < p.slices * kC * 4; e += kPrepThreads) {
            const int sl = e / (kC * 4), i = e / 4 % kC, c = e % 4;
            const bool on = i < t.n;
            const size_t row = on ? (size_t)t.tok(i) * p.dv : 0;
            float x[8], y[8];
            get8(ob + row, on, sl * kSlice + 8 * c, p.dv, x);
            get8(vb + row, on, sl * kSlice + 8 * c, p.dv, y);
            put8<NI, 64, T>(x, i, c, nullptr, ot + sl * (NI * kC * 64), kC * 64);
            unsigned char *to = vt + sl * (kC * kSlice * sizeof(T));
            *reinterpret_cast<float4 *>(to + sw<128>(i, 2 * c)) = make_float4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<float4 *>(to + sw<128>(i, 2 * c + 1)) = make_float4(y[4], y[5], y[6], y[7]);
        }
    }
    __syncthreads();
    if (tid < (int)sizeof(Gates) / 16)
        reinterpret_cast<uint4 *>(unit + U::gates)[tid] = reinterpret_cast<const uint4 *>(&s.g)[tid];

    // K K^T and Q K^T: warp w has rows 16 (w % 4) .. and columns 32 (w / 4) .., lower triangle only
    const int wm = warp & 3, wn = warp >> 2;
    const uint32_t ks = ptx::smem_u32(s.k.K), qs = ptx::smem_u32(s.k.Q);
    float kk[4][4] = {}, qk[4][4] = {};
#pragma unroll 2
    for (int k = 0; k < DK; k += 16) {
        uint32_t ka[NI][4], qa[NI][4];
#pragma unroll
        for (int x = 0; x < NI; ++x) {
            frag_a<kKeyRow<DK>>(ka[x], ks + x * U::kKey, 16 * wm, k);
            frag_a<kKeyRow<DK>>(qa[x], qs + x * U::kKey, 16 * wm, k);
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int nb = 32 * wn + 16 * n;
            if (nb > 16 * wm) continue;
            uint32_t b[NI][4];
#pragma unroll
            for (int x = 0; x < NI; ++x) frag_b<kKeyRow<DK>>(b[x], ks + x * U::kKey, k, nb);
            mma_terms(kk + 2 * n, ka, b);
            mma_terms(qk + 2 * n, qa, b);
        }
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = 16 * wm + (lane >> 2) + 8 * h, j = 32 * wn + 8 * n + 2 * (lane & 3);
            float x[2], y[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float d = j + c <= i ? s.g.decay(i, j + c) : 0.f;
                x[c] = j + c < i ? kk[n][2 * h + c] * d : 0.f;
                y[c] = j + c <= i ? qk[n][2 * h + c] * d : 0.f;
                s.n.N[i * ld + j + c] = x[c];
                s.n.X[i * ld + j + c] = x[c] * s.g.b[j + c];
            }
            uint32_t u[3];
            split2<3>(y[0], y[1], u);
#pragma unroll
            for (int x3 = 0; x3 < 3; ++x3)
                *reinterpret_cast<uint32_t *>(unit + U::P + x3 * kTri + sw<128>(i, j >> 3) + (j & 7) * 2) = u[x3];
        }
    __syncthreads();
    // N = (I + L)^-1 X, L = X diag(b), in block rows of 16: the inverses of the diagonal blocks first, all four at once by
    // a thread per column; then each block row, N_I = (I + L_II)^-1 (X_I - L_I N), by all threads
    if (tid < kC) {
        const int r = 16 * (tid >> 4), c = tid & 15;
        float y[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            y[i] = i == c ? 1.f : 0.f;
#pragma unroll
            for (int l = 0; l < i; ++l) y[i] = fmaf(-s.n.X[(r + i) * ld + r + l], y[l], y[i]);
            s.n.inv[((tid >> 4) * 16 + i) * 20 + c] = y[i];
        }
    }
    for (int r = 0; r < kC; r += 16) {
        const int i = tid >> 4, j = 4 * (tid & 15);
        float4 y = *reinterpret_cast<float4 *>(&s.n.N[(r + i) * ld + j]);
        for (int l = 0; l < r; l += 4) {
            const float4 x = *reinterpret_cast<const float4 *>(&s.n.X[(r + i) * ld + l]);
            const float xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float4 n = *reinterpret_cast<const float4 *>(&s.n.N[(l + u) * ld + j]);
                y.x = fmaf(-xs[u], n.x, y.x);
                y.y = fmaf(-xs[u], n.y, y.y);
                y.z = fmaf(-xs[u], n.z, y.z);
                y.w = fmaf(-xs[u], n.w, y.w);
            }
        }
        *reinterpret_cast<float4 *>(&s.n.rows[i * ld + j]) = y;
        __syncthreads();
        y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int l = 0; l < 16; l += 4) {
            const float4 x = *reinterpret_cast<const float4 *>(&s.n.inv[(r + i) * 20 + l]);
            const float xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float4 n = *reinterpret_cast<const float4 *>(&s.n.rows[(l + u) * ld + j]);
                y.x = fmaf(xs[u], n.x, y.x);
                y.y = fmaf(xs[u], n.y, y.y);
                y.z = fmaf(xs[u], n.z, y.z);
                y.w = fmaf(xs[u], n.w, y.w);
            }
        }
        *reinterpret_cast<float4 *>(&s.n.N[(r + i) * ld + j]) = y;
        __syncthreads();
    }
    for (int e = tid; e < kC * kC / 8; e += kPrepThreads) {
        const int i = e / (kC / 8), c = e % (kC / 8);
        float x[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) x[u] = s.n.N[i * ld + 8 * c + u];
        put8<3, 128, T>(x, i, c, nullptr, unit + U::N, kTri);
    }
}

// ---------------------------------------------------------------- chains
// Grid (groups of 16 PAIRS columns of dv, heads, directions and walks).  A pair of warps carries 16 columns: each holds
// half of dk of H^T; their partial H^T K^T meet in shared memory, and again their halves of the triangular product, and
// both go on with the whole of W (or Z).  One warp per 16 columns would spare the exchanges, but takes 8.9 us for a
// chunk of 64 tokens (dk = dv = 128, bf16, one warp to a scheduler) where the pairs take 6.2 with two: a walk is bound by
// its own dependent steps.  The products are at 62 % of what mma.sync reaches here (970 multiply-adds a cycle and SM).

// A stage's two bulk copies, issued by one thread (sixteen-byte copies by all threads took 1000 of a chunk's 7300 cycles)
// and awaited by all.
struct Loads {
    uint64_t bar[2];
    int abort;
    // stall (testing): the first stage waits for an arrival more than it gets
    __device__ __forceinline__ void init(bool stall)
    {
        if (threadIdx.x == 0) {
            mbar_init(&bar[0], stall ? 2 : 1);
            mbar_init(&bar[1], 1);
            abort = 0;
            fence_mbar_init();
        }
        __syncthreads();
    }
    __device__ __forceinline__ void fetch(unsigned char *to, const unsigned char *unit, int head, const unsigned char *tile, int bytes, int b)
    {
        if (threadIdx.x) return;
        fence_proxy_async_smem();                              // behind the reads of what the stage held
        mbar_arrive_expect_tx(&bar[b], head + bytes);
        bulk_load(to, unit, head, &bar[b]);
        bulk_load(to + head, tile, bytes, &bar[b]);
    }
    // whether the stage is there; when a wait ran out, not before its copies have landed (or a second limit has passed): the
    // block leaves then
    __device__ __forceinline__ bool wait(int b, uint32_t parity, int *err) { return wait_copies(&bar[b], parity, &abort, err, 128); }
};

// bytes of one stage: the unit's tiles from its start (forward: gates, N, K; backward: all) and V or dO
template <int DK, int NI, typename T, int WALK, int PAIRS>
struct Stage {
    using U = Unit<DK, NI>;
    static constexpr int head = WALK ? (int)U::size : (int)U::Q;
    static constexpr int tile = WALK ? NI * kC * 64 : kC * kSlice * (int)sizeof(T);
    static constexpr int size = head + PAIRS / 2 * tile;
    static constexpr int meet = PAIRS * 2 * 8 * 32 * 16;       // the pairs' partial products
    static constexpr int buffers = meet + 2 * size <= 227 * 1024 ? 2 : 1;
    static constexpr int bytes = meet + buffers * size;
};

// c (16 x 64) += A B with B the triangular tile at tB (N or P, three terms), tokens 16 k .. of the contraction against
// tokens n0 .. n1 - 1 (in sixteens); TRANS: B is stored [k][n]
template <bool TRANS, int NA>
__device__ __forceinline__ void triangle(float (*c)[4], const uint32_t (&a)[NA][4], uint32_t tB, int k, int n0, int n1)
{
#pragma unroll
    for (int n = 0; n < 4; n += 2) {
        if (n + 1 < n0 || n >= n1) continue;
        uint32_t b[2][1][3][4];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int x = 0; x < 3; ++x) {
                if (n + u < n0 || n + u >= n1) continue;
                if (TRANS) frag_bt<128>(b[u][0][x], tB + x * kTri, 16 * k, 16 * (n + u));
                else frag_b<128>(b[u][0][x], tB + x * kTri, 16 * k, 16 * (n + u));
            }
        const auto &a1 = reinterpret_cast<const uint32_t (&)[1][NA][4]>(a);
        if (n >= n0 && n + 1 < n1) mma_terms<2, 1, NA, 3>(c + 2 * n, a1, b);
        else if (n >= n0) mma_terms<1, 1, NA, 3>(c + 2 * n, a1, reinterpret_cast<const uint32_t (&)[1][1][3][4]>(b[0]));
        else mma_terms<1, 1, NA, 3>(c + 2 * n + 2, a1, reinterpret_cast<const uint32_t (&)[1][1][3][4]>(b[1]));
    }
}

template <int DK, int NI, typename T, int WALK, int PAIRS>
__device__ __forceinline__ void chain(const BwdParams &p, int dir, unsigned char *raw)
{
    using U = Unit<DK, NI>;
    using S = Stage<DK, NI, T, WALK, PAIRS>;
    constexpr int HK = DK / 2, NT = HK / 8, KP = (int)U::kKey; // a warp's half of dk, its n8 tiles, a plane of K
    const int lane = threadIdx.x & 31, half = (threadIdx.x >> 5) & 1, pair = threadIdx.x >> 6;
    const int g = lane >> 2, q2 = 2 * (lane & 3), k0 = half * HK;
    const int local = blockIdx.y, head = p.head0 + local, sl = blockIdx.x * (PAIRS / 2);
    const int row = 16 * (blockIdx.x * PAIRS + pair);          // this pair's columns of dv: rows of H^T
    const bool on = row < p.dv;
    const int tiles = min(PAIRS / 2, p.slices - sl) * S::tile;
    const size_t st = (size_t)p.dk * p.dv;
    float h[NT][4];
    const float *init = nullptr;
    if (WALK == 0 && dir == 0 && p.state_in) init = p.state_in + head * st;
    if (WALK == 1 && p.dstate) init = p.dstate + ((size_t)dir * p.BH + head) * st;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int kx = k0 + 8 * n + q2 + (x & 1), vx = row + g + 8 * (x >> 1);
            h[n][x] = init && on && kx < p.dk ? init[(size_t)kx * p.dv + vx] : 0.f;
        }

    float4 *const meets = reinterpret_cast<float4 *>(raw) + pair * 512 + lane;
    unsigned char *const stages = raw + S::meet;
    __shared__ Loads loads;
    const uint32_t base = ptx::smem_u32(stages);
    auto fetch = [&](int step) {
        const int c = (dir ^ WALK) ? p.nc - 1 - step : step;
        const size_t ws = ((size_t)dir * p.heads + local) * p.nc + c;
        loads.fetch(stages + (step % S::buffers) * S::size, p.unit + ws * U::size, S::head,
                    (WALK ? p.ot : p.vt) + (ws * p.slices + sl) * S::tile, tiles, step % S::buffers);
    };
    // r (16 x 64, columns tokens) += the warp's part of H^T K^T
    auto state_times_keys = [&](float (&r)[8][4], uint32_t tK) {
        const float one[4] = {1.f, 1.f, 1.f, 1.f};
#pragma unroll
        for (int k = 0; k < HK / 16; k += 2) {
            uint32_t a[2][3][4];
            acc_to_a<3>(a[0], h[2 * k], h[2 * k + 1], one);
            acc_to_a<3>(a[1], h[2 * k + 2], h[2 * k + 3], one);
#pragma unroll
            for (int n = 0; n < 4; n += 2) {
                uint32_t b[2][2][NI][4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int x = 0; x < NI; ++x)
                        frag_b<kKeyRow<DK>>(b[u >> 1][u & 1][x], tK + x * KP, k0 + 16 * (k + (u & 1)), 16 * (n + (u >> 1)));
                mma_terms<2, 2, 3, NI>(r + 2 * n, a, b);
            }
        }
    };
    // h += A X: A the left operands of tokens 16 k .. 16 k + 31, X the tile K or Q
    auto add_outer = [&](const uint32_t (&a)[2][3][4], uint32_t tX, int k) {
#pragma unroll
        for (int n = 0; n < HK / 16; n += 2) {
            uint32_t b[2][2][NI][4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int x = 0; x < NI; ++x)
                    frag_bt<kKeyRow<DK>>(b[u >> 1][u & 1][x], tX + x * KP, 16 * (k + (u & 1)), k0 + 16 * (n + (u >> 1)));
            mma_terms<2, 2, 3, NI>(h + 2 * n, a, b);
        }
    };
    // adds the other warp's part of r to this one's.  The first exchange writes the warp's own room and reads the other's, the
    // second the other way round: what a warp overwrites it has read itself
    auto meet = [&](float (&r)[8][4], int second) {
        float4 *const to = meets + (half ^ second) * 256;
        const float4 *const from = meets + (half ^ second ^ 1) * 256;
#pragma unroll
        for (int n = 0; n < 8; ++n) to[32 * n] = make_float4(r[n][0], r[n][1], r[n][2], r[n][3]);
        asm volatile("bar.sync %0, 64;" ::"r"(pair + 1) : "memory");
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const float4 y = from[32 * n];
            r[n][0] += y.x;
            r[n][1] += y.y;
            r[n][2] += y.z;
            r[n][3] += y.w;
        }
    };

    loads.init(p.stall && head == 0);
    if (S::buffers == 2) fetch(0);
    for (int step = 0; step < p.nc; ++step) {
        const int c = (dir ^ WALK) ? p.nc - 1 - step : step;
        const size_t ws = ((size_t)dir * p.heads + local) * p.nc + c;
        if (S::buffers == 1) {
            __syncthreads();
            fetch(step);
        }
        const bool ok = loads.wait(step % S::buffers, step / S::buffers & 1, p.err);
        if (__syncthreads_or(!ok)) return;
        if (S::buffers == 2 && step + 1 < p.nc) fetch(step + 1);   // into the stage that all warps have left
        if (!on) continue;
        const int so = (step % S::buffers) * S::size;
        const Gates &gt = *reinterpret_cast<const Gates *>(stages + so);
        const uint32_t tN = base + so + (uint32_t)U::N, tK = base + so + (uint32_t)U::K;
        {
            float *keep = (WALK ? p.GT : p.HT) + (ws * p.dv + row) * DK + k0;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                st2(keep + (size_t)g * DK + 8 * n + q2, h[n][0], h[n][1]);
                st2(keep + (size_t)(g + 8) * DK + 8 * n + q2, h[n][2], h[n][3]);
            }
        }
        float r[8][4] = {}, w[8][4];
        state_times_keys(r, tK);
        const float gend = gt.gam[kC - 1];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) h[n][x] *= gend;
        // per-token factors at the fragment's columns of tokens 16 k ..
        auto factors = [&](float (&f)[4], int k, auto of) {
#pragma unroll
            for (int x = 0; x < 4; ++x) f[x] = of(16 * k + q2 + (x & 1) + 8 * (x >> 1));
        };
        if (WALK == 0) {
            meet(r, 0);
            // R = V - gam (H^T K^T)
            const unsigned char *vt = stages + so + S::head + (pair >> 1) * S::tile;
#pragma unroll
            for (int n = 0; n < 8; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int i = 8 * n + q2 + (x & 1), v = 16 * (pair & 1) + g + 8 * (x >> 1);
                    constexpr int RB = kSlice * sizeof(T), per = 16 / sizeof(T);
                    const float y = ldf(reinterpret_cast<const T *>(vt + sw<RB>(i, v / per)) + v % per);
                    r[n][x] = y - gt.gam[i] * r[n][x];
                    w[n][x] = half ? 0.f : r[n][x];
                }
            // W = R - N diag(b) R: tokens j = 16 k .. feed tokens i >= j; the warps take two k each
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if ((k == 0 || k == 3) != (half == 0)) continue;
                float f[4];
                uint32_t a[3][4];
                factors(f, k, [&](int i) { return -gt.b[i]; });
                acc_to_a<3>(a, r[2 * k], r[2 * k + 1], f);
                triangle<false>(w, a, tN, k, k, 4);
            }
        } else {
            const uint32_t tQ = base + so + (uint32_t)U::Q, tP = base + so + (uint32_t)U::P;
            const uint32_t tX = base + so + S::head + (pair >> 1) * S::tile;
            // dU = diag(e) K dH1 + P^T dO, tokens i = 16 k .. feeding tokens j <= i: the warps take two k each
#pragma unroll
            for (int n = 0; n < 8; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x) r[n][x] *= gt.e[8 * n + q2 + (x & 1)];
            // and dH += Q^T diag(gam) dO
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
                uint32_t a[2][3][4];
#pragma unroll
                for (int kk = k; kk < k + 2; ++kk) {
                    uint32_t o[NI][4];
#pragma unroll
                    for (int x = 0; x < NI; ++x) frag_at<64>(o[x], tX + x * (kC * 64), 16 * (pair & 1), 16 * kk);
                    if ((kk == 0 || kk == 3) == (half == 0)) {
                        triangle<true>(r, o, tP, kk, 0, kk + 1);
                    }
                    float f[4], u[4] = {}, v[4] = {};
                    factors(f, kk, [&](int i) { return gt.gam[i]; });
#pragma unroll
                    for (int x = NI - 1; x >= 0; --x) {
                        u[0] += lo16(o[x][0]); u[1] += hi16(o[x][0]); u[2] += lo16(o[x][1]); u[3] += hi16(o[x][1]);
                        v[0] += lo16(o[x][2]); v[1] += hi16(o[x][2]); v[2] += lo16(o[x][3]); v[3] += hi16(o[x][3]);
                    }
                    acc_to_a<3>(a[kk - k], u, v, f);
                }
                add_outer(a, tQ, k);
            }
            meet(r, 0);
            // Z = dU - N^T diag(b) dU: tokens i = 16 k .. feed tokens j <= i; the warps take two k each
#pragma unroll
            for (int n = 0; n < 8; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x) w[n][x] = half ? 0.f : r[n][x];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if ((k == 0 || k == 3) != (half == 0)) continue;
                float f[4];
                uint32_t a[3][4];
                factors(f, k, [&](int i) { return -gt.b[i]; });
                acc_to_a<3>(a, r[2 * k], r[2 * k + 1], f);
                triangle<true>(w, a, tN, k, 0, k + 1);
            }
        }
        meet(w, 1);
        float *out = (WALK ? p.ZT : p.WT) + (ws * p.dv + row) * kC;
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            if ((n >> 2) != half) continue;
            st2(out + (size_t)g * kC + 8 * n + q2, w[n][0], w[n][1]);
            st2(out + (size_t)(g + 8) * kC + 8 * n + q2, w[n][2], w[n][3]);
        }
        // H <- gam_C H + K^T diag(e b) W, or dH <- ... - K^T diag(gam b) Z
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
            uint32_t a[2][3][4];
#pragma unroll
            for (int kk = k; kk < k + 2; ++kk) {
                float f[4];
                factors(f, kk, [&](int i) { return WALK ? -gt.gam[i] * gt.b[i] : gt.e[i] * gt.b[i]; });
                acc_to_a<3>(a[kk - k], w[2 * kk], w[2 * kk + 1], f);
            }
            add_outer(a, tK, k);
        }
    }
    if (WALK == 1 && dir == 0 && on && p.dstate_in) {
        float *to = p.dstate_in + head * st;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int kx = k0 + 8 * n + q2 + (x & 1), vx = row + g + 8 * (x >> 1);
                if (kx < p.dk) to[(size_t)kx * p.dv + vx] = h[n][x];
            }
    }
}

// The same walks with four warps to 16 columns, for calls whose blocks leave SMs idle: the walk's latency is then what
// counts.  A warp holds a quarter of dk of H^T.  Its partial H^T K^T goes to the others by tokens: warp q adds up tokens
// 16 q .. 16 q + 15, multiplies them into its part of the triangular product, whose sums by tokens meet the same way,
// and shares the finished W (or Z) of its tokens as left operands; nothing but the shared operands' loads is done twice.
// (480p chunk, 16 heads of 74 chunks, dk = dv = 128, bf16: 3.8 us a chunk, 4.7 with pairs of warps.)
template <int DK, int NI, typename T, int WALK>
struct StageNarrow {
    using U = Unit<DK, NI>;
    static constexpr int head = WALK ? (int)U::size : (int)U::Q;
    static constexpr int tile = WALK ? NI * kC * 64 : kC * kSlice * (int)sizeof(T);
    static constexpr int size = head + tile;
    static constexpr int sums = 16 * 1024, share = 6 * 1024;    // a group's partial sums; its left operands of three terms
    static constexpr int meet = 2 * (sums + share);
    static constexpr int buffers = meet + 2 * size <= 227 * 1024 ? 2 : 1;
    static constexpr int bytes = meet + buffers * size;
};

template <int DK, int NI, typename T, int WALK>
__device__ __forceinline__ void chain_narrow(const BwdParams &p, int dir, unsigned char *raw)
{
    using U = Unit<DK, NI>;
    using S = StageNarrow<DK, NI, T, WALK>;
    constexpr int HK = DK / 4, NT = HK / 8, KS = HK / 16, KP = (int)U::kKey;   // a warp's quarter of dk, its n8 tiles, its k16 steps
    const int lane = threadIdx.x & 31, me = (threadIdx.x >> 5) & 3, group = threadIdx.x >> 7;
    const int g = lane >> 2, q2 = 2 * (lane & 3), k0 = me * HK;
    const int local = blockIdx.y, head = p.head0 + local, sl = blockIdx.x;
    const int row = 32 * sl + 16 * group;                      // this group's columns of dv: rows of H^T
    const size_t st = (size_t)p.dk * p.dv;
    float h[NT][4];
    const float *init = nullptr;
    if (WALK == 0 && dir == 0 && p.state_in) init = p.state_in + head * st;
    if (WALK == 1 && p.dstate) init = p.dstate + ((size_t)dir * p.BH + head) * st;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int kx = k0 + 8 * n + q2 + (x & 1), vx = row + g + 8 * (x >> 1);
            h[n][x] = init && kx < p.dk ? init[(size_t)kx * p.dv + vx] : 0.f;
        }

    // sums[a][b][tile][lane]: warp a's part of the first product for warp b's tokens, and then, in the slot that b has
    // read, b's part of the second product for a's tokens
    float4 *const sums = reinterpret_cast<float4 *>(raw + group * (S::sums + S::share)) + lane;
    uint4 *const share = reinterpret_cast<uint4 *>(raw + group * (S::sums + S::share) + S::sums) + lane;   // [tokens / 16][term][lane]
    auto slot = [&](int a, int b, int tile) -> float4 & { return sums[((a * 4 + b) * 2 + tile) * 32]; };
    auto barrier = [&] { asm volatile("bar.sync %0, 128;" ::"r"(group + 1) : "memory"); };
    unsigned char *const stages = raw + S::meet;
    __shared__ Loads loads;
    const uint32_t base = ptx::smem_u32(stages);
    auto fetch = [&](int step) {
        const int c = (dir ^ WALK) ? p.nc - 1 - step : step;
        const size_t ws = ((size_t)dir * p.heads + local) * p.nc + c;
        loads.fetch(stages + (step % S::buffers) * S::size, p.unit + ws * U::size, S::head,
                    (WALK ? p.ot : p.vt) + (ws * p.slices + sl) * S::tile, S::tile, step % S::buffers);
    };
    auto give = [&](const uint32_t (&a)[3][4]) {
#pragma unroll
        for (int x = 0; x < 3; ++x) share[(me * 3 + x) * 32] = make_uint4(a[x][0], a[x][1], a[x][2], a[x][3]);
    };
    // h += A X over all tokens, A the shared left operands, X the tile K or Q
    auto add_outer = [&](uint32_t tX) {
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
            uint32_t a[2][3][4];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int x = 0; x < 3; ++x) {
                    const uint4 v = share[((k + u) * 3 + x) * 32];
                    a[u][x][0] = v.x; a[u][x][1] = v.y; a[u][x][2] = v.z; a[u][x][3] = v.w;
                }
            uint32_t b[HK / 16][2][NI][4];
#pragma unroll
            for (int n = 0; n < HK / 16; ++n)
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int x = 0; x < NI; ++x) frag_bt<kKeyRow<DK>>(b[n][u][x], tX + x * KP, 16 * (k + u), k0 + 16 * n);
            mma_terms<HK / 16, 2, 3, NI>(h, a, b);
        }
    };

    loads.init(p.stall && head == 0);
    if (S::buffers == 2) fetch(0);
    for (int step = 0; step < p.nc; ++step) {
        const int c = (dir ^ WALK) ? p.nc - 1 - step : step;
        const size_t ws = ((size_t)dir * p.heads + local) * p.nc + c;
        if (S::buffers == 1) {
            __syncthreads();
            fetch(step);
        }
        const bool ok = loads.wait(step % S::buffers, step / S::buffers & 1, p.err);
        if (__syncthreads_or(!ok)) return;
        if (S::buffers == 2 && step + 1 < p.nc) fetch(step + 1);   // into the stage that all warps have left
        const int so = (step % S::buffers) * S::size;
        const Gates &gt = *reinterpret_cast<const Gates *>(stages + so);
        const uint32_t tN = base + so + (uint32_t)U::N, tK = base + so + (uint32_t)U::K, tQ = base + so + (uint32_t)U::Q;
        const uint32_t tP = base + so + (uint32_t)U::P, tX = base + so + S::head;
        {
            float *keep = (WALK ? p.GT : p.HT) + (ws * p.dv + row) * DK + k0;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                st2(keep + (size_t)g * DK + 8 * n + q2, h[n][0], h[n][1]);
                st2(keep + (size_t)(g + 8) * DK + 8 * n + q2, h[n][2], h[n][3]);
            }
        }
        // this warp's part of H^T K^T
        float r[8][4] = {};
        {
            const float one[4] = {1.f, 1.f, 1.f, 1.f};
            uint32_t a[KS][3][4];
#pragma unroll
            for (int k = 0; k < KS; ++k) acc_to_a<3>(a[k], h[2 * k], h[2 * k + 1], one);
#pragma unroll
            for (int n = 0; n < 4; n += 2) {
                uint32_t b[2][KS][NI][4];
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int k = 0; k < KS; ++k)
#pragma unroll
                        for (int x = 0; x < NI; ++x) frag_b<kKeyRow<DK>>(b[u][k][x], tK + x * KP, k0 + 16 * k, 16 * (n + u));
                mma_terms<2, KS, 3, NI>(r + 2 * n, a, b);
            }
        }
        const float gend = gt.gam[kC - 1];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) h[n][x] *= gend;
        auto factors = [&](float (&f)[4], int k, auto of) {
#pragma unroll
            for (int x = 0; x < 4; ++x) f[x] = of(16 * k + q2 + (x & 1) + 8 * (x >> 1));
        };
        if (WALK == 1) {
            // dU = diag(e) K dH1 + P^T dO, tokens i = 16 k .. feeding tokens j <= i: k = 3 - me here, k = me below, so that the two
            // triangles together are the same work for every warp; and the terms of diag(gam) dO for Q^T
#pragma unroll
            for (int n = 0; n < 8; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x) r[n][x] *= gt.e[8 * n + q2 + (x & 1)];
            uint32_t o[NI][4], a[3][4];
#pragma unroll
            for (int x = 0; x < NI; ++x) frag_at<64>(o[x], tX + x * (kC * 64), 16 * group, 16 * (3 - me));
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                if (n > 3 - me) continue;
                uint32_t b[3][4];
#pragma unroll
                for (int x = 0; x < 3; ++x) frag_bt<128>(b[x], tP + x * kTri, 16 * (3 - me), 16 * n);
                mma_terms(r + 2 * n, o, b);
            }
#pragma unroll
            for (int x = 0; x < NI; ++x) frag_at<64>(o[x], tX + x * (kC * 64), 16 * group, 16 * me);
            float f[4], u[4] = {}, v[4] = {};
            factors(f, me, [&](int i) { return gt.gam[i]; });
#pragma unroll
            for (int x = NI - 1; x >= 0; --x) {
                u[0] += lo16(o[x][0]); u[1] += hi16(o[x][0]); u[2] += lo16(o[x][1]); u[3] += hi16(o[x][1]);
                v[0] += lo16(o[x][2]); v[1] += hi16(o[x][2]); v[2] += lo16(o[x][3]); v[3] += hi16(o[x][3]);
            }
            acc_to_a<3>(a, u, v, f);
            give(a);
        }
#pragma unroll
        for (int n = 0; n < 8; ++n) slot(me, n >> 1, n & 1) = make_float4(r[n][0], r[n][1], r[n][2], r[n][3]);
        barrier();
        // R (or dU) of this warp's tokens
        float rr[2][4], w[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const float4 a = slot(0, me, n), b = slot(1, me, n), x = slot(2, me, n), y = slot(3, me, n);
            rr[n][0] = (a.x + b.x) + (x.x + y.x);
            rr[n][1] = (a.y + b.y) + (x.y + y.y);
            rr[n][2] = (a.z + b.z) + (x.z + y.z);
            rr[n][3] = (a.w + b.w) + (x.w + y.w);
        }
        if (WALK == 0) {
            const unsigned char *vt = stages + so + S::head;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int i = 16 * me + 8 * n + q2 + (x & 1), v = 16 * group + g + 8 * (x >> 1);
                    constexpr int RB = kSlice * sizeof(T), per = 16 / sizeof(T);
                    rr[n][x] = ldf(reinterpret_cast<const T *>(vt + sw<RB>(i, v / per)) + v % per) - gt.gam[i] * rr[n][x];
                }
        }
        // its part of N diag(b) R for the tokens behind (or N^T diag(b) dU for those before)
        {
            float f[4];
            uint32_t a[3][4];
            factors(f, me, [&](int i) { return -gt.b[i]; });
            acc_to_a<3>(a, rr[0], rr[1], f);
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                if (WALK ? n > me : n < me) continue;
                uint32_t b[3][4];
#pragma unroll
                for (int x = 0; x < 3; ++x) {
                    if (WALK) frag_bt<128>(b[x], tN + x * kTri, 16 * me, 16 * n);
                    else frag_b<128>(b[x], tN + x * kTri, 16 * me, 16 * n);
                }
                float part[2][4] = {};
                mma_terms(part, a, b);
                if (n == me) {
#pragma unroll
                    for (int x = 0; x < 8; ++x) w[x >> 2][x & 3] = rr[x >> 2][x & 3] + part[x >> 2][x & 3];
                } else {
                    slot(n, me, 0) = make_float4(part[0][0], part[0][1], part[0][2], part[0][3]);
                    slot(n, me, 1) = make_float4(part[1][0], part[1][1], part[1][2], part[1][3]);
                }
            }
        }
        if (WALK == 1) add_outer(tQ);                          // dH += Q^T diag(gam) dO
        barrier();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (WALK ? q <= me : q >= me) continue;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const float4 y = slot(me, q, n);
                w[n][0] += y.x;
                w[n][1] += y.y;
                w[n][2] += y.z;
                w[n][3] += y.w;
            }
        }
        {
            float f[4];
            uint32_t a[3][4];
            factors(f, me, [&](int i) { return WALK ? -gt.gam[i] * gt.b[i] : gt.e[i] * gt.b[i]; });
            acc_to_a<3>(a, w[0], w[1], f);
            give(a);
        }
        barrier();
        add_outer(tK);                                         // H <- gam_C H + K^T diag(e b) W, or dH <- ... - K^T diag(gam b) Z
        float *out = (WALK ? p.ZT : p.WT) + (ws * p.dv + row) * kC + 16 * me;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            st2(out + (size_t)g * kC + 8 * n + q2, w[n][0], w[n][1]);
            st2(out + (size_t)(g + 8) * kC + 8 * n + q2, w[n][2], w[n][3]);
        }
    }
    if (WALK == 1 && dir == 0 && p.dstate_in) {
        float *to = p.dstate_in + head * st;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int kx = k0 + 8 * n + q2 + (x & 1), vx = row + g + 8 * (x >> 1);
                if (kx < p.dk) to[(size_t)kx * p.dv + vx] = h[n][x];
            }
    }
}

template <int DK, int NI, typename T>
__global__ void __launch_bounds__(256, 1) bwd_chain_narrow_kernel(const __grid_constant__ BwdParams p)
{
    extern __shared__ __align__(128) unsigned char raw[];
    if (blockIdx.z < p.dirs) chain_narrow<DK, NI, T, 1>(p, blockIdx.z, raw);
    else chain_narrow<DK, NI, T, 0>(p, blockIdx.z - p.dirs, raw);
}

template <int DK, int NI, typename T, int PAIRS>
__global__ void __launch_bounds__(64 * PAIRS, 1) bwd_chain_kernel(const __grid_constant__ BwdParams p)
{
    extern __shared__ __align__(128) unsigned char raw[];
    // the backward walks, the longer ones, come first
    if (blockIdx.z < p.dirs) chain<DK, NI, T, 1, PAIRS>(p, blockIdx.z, raw);
    else chain<DK, NI, T, 0, PAIRS>(p, blockIdx.z - p.dirs, raw);
}

// ---------------------------------------------------------------- gradients
// Grid (chunks, heads), eight warps: warp w has the tokens 16 (w % 4) .. of every result and its columns' half w / 4.
constexpr int kGradThreads = 256;
constexpr int kStep = kSlice;          // dv columns per step of the walk over dv
constexpr int kLdT = kC + 4;           // pitch of 64-wide fp32 rows

template <int DK, int NI>
struct GradSmem {
    using U = Unit<DK, NI>;
    static constexpr bool kStage = NI == 1;                    // room for the next step's fp32 tiles
    static constexpr int NE = 3;                               // terms of E and S
    static constexpr int kOTiles = NI == 1 ? 4 : 1;            // dO: every slice, or the step's
    static constexpr int kState = kStep * DK * 2, kVal = kStep * kC * 2;
    struct Walk {                                              // term planes of the step's H0, dH1, U, Y: rows dv
        unsigned char H[3 * kState], G[3 * kState], U[3 * kVal], Y[3 * kVal];
    };
    struct Tail {
        unsigned char E[NE * kTri], S[NE * kTri];              // [i][j]
        float F[kC * kLdT], M[kC * (kC + 1)];
    };
    Gates g;
    unsigned char K[NI * U::kKey], Q[NI * U::kKey];
    unsigned char O[kOTiles * NI * kC * 64];
    union {
        Walk walk;
        Tail tail;
    };
    float Z[kStep * kLdT], Z0[kStep * kLdT];                   // the step's Z; the first direction's
    float W[kStage ? kStep * kLdT : 4];
    float H[kStage ? kStep * DK : 4], GT[kStage ? kStep * DK : 4];
    float db[kC], da[kC];                                      // over the directions, by token
    float m0[2][kC], m1[2][kC], dbw[8][kC], col[8][kC], hh[8];
};

// 32 rows of `len` floats to rows of pitch `ld`
__device__ __forceinline__ void copy_rows(float *dst, int ld, const float *src, int len)
{
    const int per = len / 4;
    for (int e = threadIdx.x; e < kStep * per; e += kGradThreads)
        copy16(ptx::smem_u32(dst + (e / per) * ld + 4 * (e % per)), src + (size_t)(e / per) * len + 4 * (e % per));
}

// columns j, j + 1 of row i of a tile of term planes
template <int NI, int RB>
__device__ __forceinline__ float2 pair_at(const unsigned char *tile, int plane, int i, int j)
{
    float2 r = make_float2(0.f, 0.f);
#pragma unroll
    for (int x = NI - 1; x >= 0; --x) {
        const uint32_t u = *reinterpret_cast<const uint32_t *>(tile + x * plane + sw<RB>(i, j >> 3) + (j & 7) * 2);
        r.x += lo16(u);
        r.y += hi16(u);
    }
    return r;
}

template <int DK, int NI, typename T>
__global__ void __launch_bounds__(kGradThreads, 1) bwd_grad_kernel(const __grid_constant__ BwdParams p)
{
    extern __shared__ __align__(128) unsigned char raw[];
    using U = Unit<DK, NI>;
    using Sm = GradSmem<DK, NI>;
    Sm &s = *reinterpret_cast<Sm *>(raw);
    constexpr int NT = DK / 16, NE = Sm::NE;                   // n8 tiles of a warp's half of dk
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, wm = warp & 3, wn = warp >> 2;
    const int g = lane >> 2, q2 = 2 * (lane & 3);
    const uint32_t aK = ptx::smem_u32(s.K), aQ = ptx::smem_u32(s.Q), aO = ptx::smem_u32(s.O);
    const uint32_t aH = ptx::smem_u32(s.walk.H), aG = ptx::smem_u32(s.walk.G), aU = ptx::smem_u32(s.walk.U), aY = ptx::smem_u32(s.walk.Y);
    const uint32_t aE = ptx::smem_u32(s.tail.E), aS = ptx::smem_u32(s.tail.S);
    const size_t first = ((size_t)blockIdx.y) * p.nc + blockIdx.x;   // this chunk in the first direction
    float *const part = reinterpret_cast<float *>(p.unit + first * U::size);   // bidirectional: its dQ, dK sums
    static_assert(2 * kC * DK * sizeof(float) <= U::size, "the first direction's sums fit in its unit");
    if (tid < kC) s.db[tid] = s.da[tid] = 0.f;

    for (int dir = 0; dir < p.dirs; ++dir) {
        const Tile t = make_tile(p, dir, blockIdx.y, blockIdx.x);
        const unsigned char *unit = p.unit + t.ws * U::size;
        const float *HT = p.HT + t.ws * p.dv * DK, *GT = p.GT + t.ws * p.dv * DK;
        const float *WT = p.WT + t.ws * p.dv * kC, *ZT = p.ZT + t.ws * p.dv * kC, *ZT0 = p.ZT + first * p.dv * kC;
        const bool last = dir == p.dirs - 1;
        __syncthreads();
        auto fetch = [&](int c0) {
            if constexpr (Sm::kStage) {
                copy_rows(s.H, DK, HT + (size_t)c0 * DK, DK);
                copy_rows(s.GT, DK, GT + (size_t)c0 * DK, DK);
                copy_rows(s.W, kLdT, WT + (size_t)c0 * kC, kC);
            }
            copy_rows(s.Z, kLdT, ZT + (size_t)c0 * kC, kC);
            if (dir == 1) copy_rows(s.Z0, kLdT, ZT0 + (size_t)c0 * kC, kC);
            if (!Sm::kStage) copy_block(aO, p.ot + (t.ws * p.slices + c0 / kSlice) * (NI * kC * 64), NI * kC * 64);
            copy_commit();
        };
        copy_block(ptx::smem_u32(&s.g), unit, sizeof(Gates));
        copy_block(aK, unit + U::K, NI * (int)U::kKey);
        copy_block(aQ, unit + U::Q, NI * (int)U::kKey);
        if (Sm::kStage) copy_block(aO, p.ot + t.ws * p.slices * (NI * kC * 64), p.slices * NI * kC * 64);
        fetch(0);

        float hdo[NT][4] = {}, hy[NT][4] = {}, du[NT][4] = {}, dp[4][4] = {}, dx[4][4] = {}, db[8] = {}, hh = 0.f;
        for (int c0 = 0; c0 < p.dv; c0 += kStep) {
            copy_wait<0>();
            __syncthreads();           // the step's tiles are here, and every warp has left the last step's planes
            for (int e = tid; e < kStep * (DK / 8); e += kGradThreads) {
                const int r = e / (DK / 8), c = e % (DK / 8);
                float x[8], y[8];
                get8f(Sm::kStage ? s.H + r * DK + 8 * c : HT + (size_t)(c0 + r) * DK + 8 * c, x);
                get8f(Sm::kStage ? s.GT + r * DK + 8 * c : GT + (size_t)(c0 + r) * DK + 8 * c, y);
#pragma unroll
                for (int i = 0; i < 8; ++i) hh = fmaf(x[i], y[i], hh);
                planes8<DK * 2>(x, r, c, s.walk.H, Sm::kState);
                planes8<DK * 2>(y, r, c, s.walk.G, Sm::kState);
            }
            {
                const int r = tid >> 3, c = tid & 7;           // a column of dv, eight tokens
                float w[8], z[8];
                get8f(Sm::kStage ? s.W + r * kLdT + 8 * c : WT + (size_t)(c0 + r) * kC + 8 * c, w);
                get8f(s.Z + r * kLdT + 8 * c, z);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    db[i] = fmaf(w[i], z[i], db[i]);
                    w[i] *= s.g.b[8 * c + i];
                    z[i] *= s.g.b[8 * c + i];
                }
                planes8<128>(w, r, c, s.walk.U, Sm::kVal);
                planes8<128>(z, r, c, s.walk.Y, Sm::kVal);
            }
            if (last) {                // dV = Y, of both directions
                for (int e = tid; e < t.n * (kStep / 2); e += kGradThreads) {
                    const int i = e / (kStep / 2), j = 2 * (e % (kStep / 2));
                    float x = s.Z[j * kLdT + i], y = s.Z[(j + 1) * kLdT + i];
                    if (dir == 1) {
                        x += s.Z0[j * kLdT + t.n - 1 - i];
                        y += s.Z0[(j + 1) * kLdT + t.n - 1 - i];
                    }
                    st2(static_cast<T *>(p.dv_) + ((size_t)t.head * p.T + t.tok(i)) * p.dv + c0 + j, s.g.b[i] * x, s.g.b[i] * y);
                }
            }
            __syncthreads();
            if (Sm::kStage && c0 + kStep < p.dv) fetch(c0 + kStep);
#pragma unroll
            for (int k = 0; k < kStep; k += 16) {
                uint32_t o[NI][4], u[3][4], y[3][4];
                const uint32_t ot = aO + (Sm::kStage ? c0 / kSlice : 0) * (NI * kC * 64);
#pragma unroll
                for (int x = 0; x < NI; ++x) frag_a<64>(o[x], ot + x * (kC * 64), 16 * wm, k);
#pragma unroll
                for (int x = 0; x < 3; ++x) {
                    frag_at<128>(u[x], aU + x * Sm::kVal, 16 * wm, k);
                    frag_at<128>(y[x], aY + x * Sm::kVal, 16 * wm, k);
                }
#pragma unroll
                for (int n = 0; n < NT / 2; ++n) {
                    uint32_t b[3][4];
#pragma unroll
                    for (int x = 0; x < 3; ++x) frag_bt<DK * 2>(b[x], aH + x * Sm::kState, k, wn * (DK / 2) + 16 * n);
                    mma_terms(hdo + 2 * n, o, b);
                    mma_terms(hy + 2 * n, y, b);
#pragma unroll
                    for (int x = 0; x < 3; ++x) frag_bt<DK * 2>(b[x], aG + x * Sm::kState, k, wn * (DK / 2) + 16 * n);
                    mma_terms(du + 2 * n, u, b);
                }
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    if (32 * wn + 16 * n > 16 * wm) continue;
                    uint32_t b[3][4];
#pragma unroll
                    for (int x = 0; x < 3; ++x) frag_bt<128>(b[x], aU + x * Sm::kVal, k, 32 * wn + 16 * n);
                    mma_terms(dp + 2 * n, o, b);
                    mma_terms(dx + 2 * n, y, b);
                }
            }
            if (!Sm::kStage && c0 + kStep < p.dv) {
                __syncthreads();
                fetch(c0 + kStep);
            }
        }

        // db_i = Z_i . W_i: over a warp's four columns of dv here, over the warps below; <H0, dH1> likewise
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            db[i] += __shfl_xor_sync(0xffffffffu, db[i], 8);
            db[i] += __shfl_xor_sync(0xffffffffu, db[i], 16);
            if (lane < 8) s.dbw[warp][8 * lane + i] = db[i];
        }
        hh = warp_sum(hh);
        if (lane == 0) s.hh[warp] = hh;
        // X and P again, in the layout of dX and dP
        float kk[4][4] = {}, qk[4][4] = {};
#pragma unroll 2
        for (int k = 0; k < DK; k += 16) {
            uint32_t ka[NI][4], qa[NI][4];
#pragma unroll
            for (int x = 0; x < NI; ++x) {
                frag_a<kKeyRow<DK>>(ka[x], aK + x * (int)U::kKey, 16 * wm, k);
                frag_a<kKeyRow<DK>>(qa[x], aQ + x * (int)U::kKey, 16 * wm, k);
            }
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int nb = 32 * wn + 16 * n;
                if (nb > 16 * wm) continue;
                uint32_t b[NI][4];
#pragma unroll
                for (int x = 0; x < NI; ++x) frag_b<kKeyRow<DK>>(b[x], aK + x * (int)U::kKey, k, nb);
                mma_terms(kk + 2 * n, ka, b);
                mma_terms(qk + 2 * n, qa, b);
            }
        }
        __syncthreads();               // the walk's planes are done with: E, F, M take their place
        const Lift lift = lift_of(s.g);
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = 16 * wm + g + 8 * h, j = 32 * wn + 8 * n + q2;
                float x[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float d = j + c <= i ? s.g.decay(i, j + c, lift.shift) : 0.f;
                    const float f = j + c < i ? -d * dx[n][2 * h + c] : 0.f;
                    x[c] = j + c <= i ? d * dp[n][2 * h + c] : 0.f;
                    s.tail.F[i * kLdT + j + c] = f * lift.down;
                    s.tail.M[i * (kC + 1) + j + c] = j + c < i ? f * kk[n][2 * h + c] + x[c] * qk[n][2 * h + c] : 0.f;
                    x[c] *= lift.down;
                }
                uint32_t u[NE];
                split2<NE>(x[0], x[1], u);
#pragma unroll
                for (int z = 0; z < NE; ++z)
                    *reinterpret_cast<uint32_t *>(s.tail.E + z * kTri + sw<128>(i, j >> 3) + (j & 7) * 2) = u[z];
            }
        // m0_i = gam_i (q_i . H0 dO_i - k_i . H0 Y_i), m1_i = e_i k_i . dH1 U_i: this warp's half of dk
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = 16 * wm + g + 8 * h;
            const float gam = s.g.gam[i], e = s.g.e[i];
            float x = 0.f, y = 0.f;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int j = wn * (DK / 2) + 8 * n + q2;
                const float2 k = pair_at<NI, kKeyRow<DK>>(s.K, (int)U::kKey, i, j), q = pair_at<NI, kKeyRow<DK>>(s.Q, (int)U::kKey, i, j);
                float *a = &hdo[n][2 * h], *b = &hy[n][2 * h], *c = &du[n][2 * h];
                x = fmaf(q.x, a[0], fmaf(q.y, a[1], fmaf(-k.x, b[0], fmaf(-k.y, b[1], x))));
                y = fmaf(k.x, c[0], fmaf(k.y, c[1], y));
                a[0] *= gam;
                a[1] *= gam;
                b[0] = e * c[0] - gam * b[0];
                b[1] = e * c[1] - gam * b[1];
            }
            x += __shfl_xor_sync(0xffffffffu, x, 1);
            x += __shfl_xor_sync(0xffffffffu, x, 2);
            y += __shfl_xor_sync(0xffffffffu, y, 1);
            y += __shfl_xor_sync(0xffffffffu, y, 2);
            if ((lane & 3) == 0) {
                s.m0[wn][i] = s.g.from_entry(i, lift.shift) * x;
                s.m1[wn][i] = s.g.decay(kC - 1, i, lift.shift) * y;
            }
        }
        __syncthreads();
        for (int e = tid; e < kC * kC / 2; e += kGradThreads) {   // S = F + F^T
            const int i = e / (kC / 2), j = 2 * (e % (kC / 2));
            uint32_t u[NE];
            split2<NE>(s.tail.F[i * kLdT + j] + s.tail.F[j * kLdT + i], s.tail.F[i * kLdT + j + 1] + s.tail.F[(j + 1) * kLdT + i], u);
#pragma unroll
            for (int z = 0; z < NE; ++z)
                *reinterpret_cast<uint32_t *>(s.tail.S + z * kTri + sw<128>(i, j >> 3) + (j & 7) * 2) = u[z];
        }
        // sums of M over the rows i >= t of their sums over the columns before t; the lane has t = 2 lane, 2 lane + 1.
        // Row 64 is the chunk's end.
        float col[2] = {};
        for (int i = warp; i <= kC; i += 8) {
            float x, y, from;
            if (i < kC) {
                x = s.tail.M[i * (kC + 1) + 2 * lane];
                y = s.tail.M[i * (kC + 1) + 2 * lane + 1];
                from = s.m0[0][i] + s.m0[1][i];
            } else {
                x = s.m1[0][2 * lane] + s.m1[1][2 * lane];
                y = s.m1[0][2 * lane + 1] + s.m1[1][2 * lane + 1];
                from = 0.f;
#pragma unroll
                for (int w = 0; w < 8; ++w) from += s.hh[w];
                from *= s.g.from_entry(kC - 1, lift.shift);
            }
            float sum = x + y;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float z = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += z;
            }
            float before = __shfl_up_sync(0xffffffffu, sum, 1);
            before = (lane ? before : 0.f) + from;
            if (i >= 2 * lane) col[0] += before;
            if (i >= 2 * lane + 1) col[1] += before + x;
        }
        s.col[warp][2 * lane] = col[0];
        s.col[warp][2 * lane + 1] = col[1];
        __syncthreads();
        if (tid < t.n) {
            float a = 0.f, b = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                a += s.col[w][tid];
                b += s.dbw[w][tid];
            }
            const int at = t.tok(tid) - t.c * kC;
            s.da[at] += a / (s.g.a[tid] * lift.up);
            s.db[at] += b;
        }
        // dQ = gam hdo + E K;  dK = e du - gam hy + S K + E^T Q
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t a[NE][4], b[NI][4];
#pragma unroll
            for (int n = 0; n < NT / 2; ++n) {
                const int nb = wn * (DK / 2) + 16 * n;
#pragma unroll
                for (int x = 0; x < NI; ++x) frag_bt<kKeyRow<DK>>(b[x], aK + x * (int)U::kKey, 16 * k, nb);
                if (k <= wm) {
#pragma unroll
                    for (int x = 0; x < NE; ++x) frag_a<128>(a[x], aE + x * kTri, 16 * wm, 16 * k);
                    mma_terms(hdo + 2 * n, a, b);
                }
#pragma unroll
                for (int x = 0; x < NE; ++x) frag_a<128>(a[x], aS + x * kTri, 16 * wm, 16 * k);
                mma_terms(hy + 2 * n, a, b);
                if (k >= wm) {
#pragma unroll
                    for (int x = 0; x < NI; ++x) frag_bt<kKeyRow<DK>>(b[x], aQ + x * (int)U::kKey, 16 * k, nb);
#pragma unroll
                    for (int x = 0; x < NE; ++x) frag_at<128>(a[x], aE + x * kTri, 16 * wm, 16 * k);
                    mma_terms(hy + 2 * n, a, b);
                }
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = 16 * wm + g + 8 * h;
            if (i >= t.n) continue;
            const int tok = t.tok(i), at = tok - t.c * kC;
            const size_t row = ((size_t)t.head * p.T + tok) * p.dk;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int j = wn * (DK / 2) + 8 * n + q2;
                if (j >= p.dk) continue;
                float2 x = make_float2(hdo[n][2 * h], hdo[n][2 * h + 1]), y = make_float2(hy[n][2 * h], hy[n][2 * h + 1]);
                float2 *px = reinterpret_cast<float2 *>(part + at * DK + j), *py = reinterpret_cast<float2 *>(part + (kC + at) * DK + j);
                if (!last) {
                    __stcg(px, x);
                    __stcg(py, y);
                    continue;
                }
                if (dir == 1) {
                    const float2 u = __ldcg(px), v = __ldcg(py);
                    x.x += u.x; x.y += u.y;
                    y.x += v.x; y.y += v.y;
                }
                st2(static_cast<T *>(p.dq) + row + j, x.x, x.y);
                st2(static_cast<T *>(p.dk_) + row + j, y.x, y.y);
            }
        }
    }
    __syncthreads();
    const int base = blockIdx.x * kC, n = min(kC, p.T - base);
    if (tid < n) {
        const size_t at = (size_t)(p.head0 + blockIdx.y) * p.T + base + tid;
        p.dbeta[at] = s.db[tid];
        p.ddecay[at] = s.da[tid];
    }
}

// ---------------------------------------------------------------- launches
template <typename F>
cudaError_t launch(F kernel, dim3 grid, int threads, size_t smem, const BwdParams &p, cudaStream_t stream)
{
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess) return err;
    kernel<<<grid, threads, smem, stream>>>(p);
    err = cudaGetLastError();
    if (err == cudaSuccess) count_launches(1);
    return err;
}

template <int DK, int NI, typename T>
cudaError_t launch_chains(const BwdParams &p, bool wide, cudaStream_t stream)
{
    constexpr int kPairs = 4;
    constexpr int smem = std::max(Stage<DK, NI, T, 0, kPairs>::bytes, Stage<DK, NI, T, 1, kPairs>::bytes);
    constexpr int narrow = std::max(StageNarrow<DK, NI, T, 0>::bytes, StageNarrow<DK, NI, T, 1>::bytes);
    static_assert(smem <= 227 * 1024 && narrow <= 227 * 1024, "shared memory");
    if (!wide) return launch(bwd_chain_narrow_kernel<DK, NI, T>, dim3(p.slices, p.heads, 2 * p.dirs), 256, narrow, p, stream);
    return launch(bwd_chain_kernel<DK, NI, T, kPairs>, dim3((p.slices + kPairs / 2 - 1) / (kPairs / 2), p.heads, 2 * p.dirs), 64 * kPairs,
                  smem, p, stream);
}

// The workspace holds the operands and both chains' states of every chunk of the heads that one pass takes; passes are
// cut so that it stays under this, unless one head alone needs more.
constexpr size_t kMaxWorkspace = (size_t)6 << 30;

template <int DK, int NI, typename T>
cudaError_t run(BwdParams p, cudaStream_t stream)
{
    using U = Unit<DK, NI>;
    static_assert(sizeof(GradSmem<DK, NI>) <= 227 * 1024 && sizeof(PrepSmem<DK, NI>) <= 227 * 1024, "shared memory");
    p.slices = (p.dv + kSlice - 1) / kSlice;
    const size_t vt = (size_t)p.slices * kC * kSlice * sizeof(T), ot = (size_t)p.slices * NI * kC * 64;
    const size_t state = (size_t)p.dv * DK * sizeof(float), rows = (size_t)p.dv * kC * sizeof(float);
    const size_t per_head = (U::size + vt + ot + 2 * state + 2 * rows) * p.nc * p.dirs;
    const int most = (int)std::min<size_t>((size_t)p.BH, std::max<size_t>(1, kMaxWorkspace / per_head));
    const int passes = (p.BH + most - 1) / most, each_pass = (p.BH + passes - 1) / passes;
    int dev = 0, sms = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (err == cudaSuccess) err = device_error_word(&p.err);
    unsigned char *ws = nullptr;
    if (err == cudaSuccess) err = ws_alloc(reinterpret_cast<void **>(&ws), per_head * each_pass, stream);
    if (err != cudaSuccess) return err;
    for (int h = 0; h < p.BH && err == cudaSuccess; h += each_pass) {
        p.head0 = h;
        p.heads = std::min(each_pass, p.BH - h);
        const size_t n = (size_t)p.nc * p.dirs * p.heads;
        // a chain block fills an SM's shared memory: 32 columns a block, four warps to 16 of them, while those blocks fit the
        // SMs; 64 columns, two warps to 16, beyond
        const bool wide = (long long)p.slices * p.heads * 2 * p.dirs > sms;
        p.unit = ws;
        p.vt = p.unit + n * U::size;
        p.ot = p.vt + n * vt;
        p.HT = reinterpret_cast<float *>(p.ot + n * ot);
        p.GT = p.HT + n * p.dv * DK;
        p.WT = p.GT + n * p.dv * DK;
        p.ZT = p.WT + n * p.dv * kC;
        err = launch(bwd_prepare_kernel<DK, NI, T>, dim3(p.nc, p.heads, p.dirs), kPrepThreads, sizeof(PrepSmem<DK, NI>), p, stream);
        if (err == cudaSuccess)
            err = launch_chains<DK, NI, T>(p, wide, stream);
        if (err == cudaSuccess) {
            if constexpr (DK == 128 && NI == 1) err = launch_grad_tc(p, stream);
            else err = launch(bwd_grad_kernel<DK, NI, T>, dim3(p.nc, p.heads), kGradThreads, sizeof(GradSmem<DK, NI>), p, stream);
        }
    }
    const cudaError_t e2 = ws_free(ws, stream);
    return err != cudaSuccess ? err : e2;
}

}  // namespace

cudaError_t set_wait_limit_backward(unsigned long long ns)
{
    const cudaError_t err = set_module_wait_limit(ns);
    return err == cudaSuccess ? bwd::set_wait_limit_tc(ns) : err;
}

cudaError_t launch_backward(const BwdArgs &a, cudaStream_t stream)
{
    BwdParams p = {};
    p.q = a.f.q; p.k = a.f.k; p.v = a.f.v; p.dout = a.dout;
    p.beta = a.f.beta; p.decay = a.f.decay; p.state_in = a.f.state_in; p.dstate = a.dstate;
    p.dq = a.dq; p.dk_ = a.dk; p.dv_ = a.dv; p.dbeta = a.dbeta; p.ddecay = a.ddecay; p.dstate_in = a.dstate_in;
    p.BH = a.f.B * a.f.H; p.T = a.f.T; p.nc = (a.f.T + bwd::kC - 1) / bwd::kC; p.dk = a.f.dk; p.dv = a.f.dv;
    p.dirs = a.f.bidi ? 2 : 1;
    p.stall = g_stall_chunk >= 0;
    if (a.f.fp32) return p.dk <= 64 ? run<64, 3, float>(p, stream) : run<128, 3, float>(p, stream);
    return p.dk <= 64 ? run<64, 1, __nv_bfloat16>(p, stream) : run<128, 1, __nv_bfloat16>(p, stream);
}

}  // namespace gdn
