// The gradients of one chunk for bf16 inputs and dk of 96 or 128, on tcgen05 tensor cores: the last kernel of
// gdn_backward, whose mathematics is at the top of gdn_backward.cu.
//
// A block takes a chunk of 64 tokens and both scan directions.  Results stand transposed, lanes of tensor memory for
// dk (128) or for the token j of the contracted pair, columns for tokens, so that every product has M = 128:
//     HD = H0 dO^T, HY = H0 Y^T, DU = dH1 U^T            (dk x 64, summed over dv)
//     PP = U dO^T, XX = U Y^T                            (64 x 64; the terms of U stacked: lanes j and 64 + j add up)
//     KK = K K^T, QK = K Q^T                             (64 x 64, lanes 0 - 63)
//     EK = K^T E^T,  SK = K^T S + Q^T E                  (dk x 64)
// The states and W, Z come as fp32 rows of dv; a step of 32 of them is split into three bf16 terms each on the way to
// shared memory, as operands with the contraction's index as their row (MN-major), in two buffers, so that the next
// step's loads and splitting run beside the tensor core.  One warp issues the products: a product of 128 x 64 x 16 takes
// the tensor core 48 cycles, its issue as long, and a step has 42 of them, which the splitting must not wait for.  (1184
// chunks, dv = 128: 170 us, where mma.sync tiles took 280; the tensor core is busy for a third of that, the rest is the
// latency of loads, splitting and epilogue with sixteen warps of 96 registers.)  Products of terms are those of order
// i + j < 3, the small ones first in each step.  The tensor core truncates its fp32 sums, and a result's run over all of dv here,
// up to 48 products: 3e-7 to 1e-6 (rel-L2) in the gradient of the decay, where the other kernel, which adds every few products by a
// rounded addition, leaves 2e-7 and elementary fp32 operations 2 - 3e-7.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gdn_backward.cuh"
#include "gdn_chunk_common.cuh"

namespace gdn {
namespace {

using bwd::BwdParams;
using bwd::Gates;
using bwd::Tile;

constexpr int kWorkers = 512, kThreads = kWorkers + 32;   // sixteen warps that work, and one that issues products
constexpr int kRows = 32;                       // dv rows per step
constexpr int kHalf = kRows * 128;              // one 64-wide half of a plane of the states
constexpr int kPlane = 2 * kHalf;               // a term of H0 or dH1: 32 x 128
constexpr int kVal = kRows * 128;               // a term of U or Y: 32 x 64 tokens
constexpr int kBuf = 6 * kPlane + 7 * kVal;     // H0, dH1, U, a tile of zeros, Y
constexpr int oH = 0, oG = 3 * kPlane, oU = 6 * kPlane, oZero = oU + 3 * kVal, oY = oZero + kVal;
constexpr int kSq = 64 * 128;                   // a 64 x 64 tile of one term
constexpr int kKeys = 64 * 256;                 // K or Q
constexpr int kLd = 65;
using U1 = bwd::Unit<128, 1>;

// columns of tensor memory; EK and SK take the place of PP and XX once these are read
enum { cHD = 0, cHY = 64, cDU = 128, cPP = 192, cXX = 256, cKK = 320, cQK = 384, cEK = cPP, cSK = cXX, kCols = 512 };

struct Smem {
    // Offsets from a 1024-byte boundary.  Behind the walk over dv the first buffer holds what two threads of PP, XX, KK
    // and QK exchange (the place of H0, dH1 and some of U; F^T over PP's; KK and QK of half the tokens) and the warps'
    // parts of db (the rest of U), the second the terms of E^T and S (H0 and dH1); and then the first dQ and dK.  V
    // collects dV.
    static constexpr int K = 0, Q = K + kKeys, O = Q + kKeys, V = O + 4 * 64 * 64, buf = V + kKeys, end = buf + 2 * kBuf;
    static constexpr int dbw = buf + oU + 2 * kVal;
    static constexpr int xP = buf, xX = xP + 64 * kLd * 4, xK = xX + 64 * kLd * 4, E = buf + kBuf, S = E + 3 * kSq, out = buf;
    static_assert(xK + 2 * 64 * 32 * 4 <= dbw && dbw + 16 * 64 * 4 <= buf + oZero && S + 3 * kSq <= buf + kBuf + oZero,
                  "the walk's zeros stay");
    struct Small {
        Gates g;
        float db[64], da[64];                   // over the directions, by token
        float m0[4][64], m1[4][64], col[2][64], whole[8][64], hh[16];
        uint64_t full[3], done[3];              // a buffer's operands are there, its products are done; the last products'
        uint64_t drain;                         // behind a wait that ran out: every product issued is done
        uint32_t tmem;
        int abort;
    };
    static constexpr int bytes = end + (int)sizeof(Small) + 1024;
};
static_assert(Smem::bytes <= 227 * 1024, "shared memory");

constexpr uint32_t kIdMK = idesc_bf16(128, 64, true, false);    // A MN-major, B K-major
constexpr uint32_t kIdMM = idesc_bf16(128, 64, true, true);
constexpr uint32_t kIdKK = idesc_bf16(128, 64, false, false);

// Operand descriptors are formed as two words, and one product's differ from another's by a constant in the low word
// alone: the issuing thread spends one addition a product, not a descriptor.
constexpr uint32_t kDesc128 = (1024u >> 4) | (1u << 14) | (2u << 29);   // high word: groups of 8 rows 1024 bytes apart, 128-byte swizzle
constexpr uint32_t kDesc64 = (512u >> 4) | (1u << 14) | (4u << 29);     // rows of 64 bytes, 64-byte swizzle
// low word: the address, and the distance of two 64-wide halves of an MN-major tile
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t halves) { return (saddr >> 4) | (halves >> 4) << 16; }
__host__ __device__ constexpr uint32_t step_of(uint32_t bytes) { return bytes >> 4; }

__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t a_hi, uint32_t b, uint32_t b_hi, uint32_t idesc, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
                 "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
                 "setp.ne.b32 p, %6, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}"
                 ::"r"(d), "r"(a), "r"(a_hi), "r"(b), "r"(b_hi), "r"(idesc), "r"(acc)
                 : "memory");
}

// lane l gets the sum over the warp's lanes of their v[l % N]
template <int N>
__device__ __forceinline__ float sum_across(float (&v)[N])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = N / 2; o; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float mine = up ? v[i + o] : v[i], theirs = up ? v[i] : v[i + o];
            v[i] = mine + __shfl_xor_sync(0xffffffffu, theirs, o);
        }
    }
    float x = v[0];
#pragma unroll
    for (int o = N; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ void prefetch_l2(const void *p, uint32_t bytes)
{
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

__device__ __forceinline__ void read4(const float *p, float *x)
{
    const float4 u = __ldcg(reinterpret_cast<const float4 *>(p));
    x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
}

// a thread's share of a step: eight values of a row of H0^T and dH1^T, four of W^T, Z^T and the first direction's Z^T
struct Step {
    float h[8], g[8], w[4], z[4], z0[4];
};

// four floats as term planes: half a 16-byte piece of a tile of 128-byte rows
__device__ __forceinline__ void planes4(const float (&x)[4], int row, int c4, unsigned char *to, int plane)
{
    uint32_t u[3], v[3];
    bwd::split2<3>(x[0], x[1], u);
    bwd::split2<3>(x[2], x[3], v);
#pragma unroll
    for (int t = 0; t < 3; ++t)
        *reinterpret_cast<uint2 *>(to + t * plane + bwd::sw<128>(row, c4 >> 1) + (c4 & 1) * 8) = make_uint2(u[t], v[t]);
}

// the issuing thread's products of one step
__device__ __forceinline__ void issue_step(uint32_t tmem, uint32_t base, int at, int step)
{
    if (step == 0) {                                            // K K^T, K Q^T: lanes 64 - 127 multiply what follows K
        const uint32_t k = desc_lo(base + Smem::K, 16);
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            const uint32_t o = k + step_of((x >> 2) * 8192 + (x & 3) * 32);
            mma(tmem + cKK, o, kDesc128, o, kDesc128, kIdKK, x > 0);
            mma(tmem + cQK, o, kDesc128, o + step_of(Smem::Q - Smem::K), kDesc128, kIdKK, x > 0);
        }
    }
    static_assert(kHalf == kVal, "one distance serves the states' halves and the stacked terms of U");
    const uint32_t w0 = desc_lo(base + at, kHalf), o0 = desc_lo(base + Smem::O + step * 4096, 16);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t acc = k > 0 ? 1 : step > 0, O = o0 + step_of(k * 32);
        const auto H = [&](int i) { return w0 + step_of(oH + i * kPlane + k * 2048); };
        const auto G = [&](int i) { return w0 + step_of(oG + i * kPlane + k * 2048); };
        const auto U = [&](int i) { return w0 + step_of(oU + i * kVal + k * 2048); };
        const auto Y = [&](int i) { return w0 + step_of(oY + i * kVal + k * 2048); };
        mma(tmem + cHD, H(2), kDesc128, O, kDesc64, kIdMK, acc);
        mma(tmem + cHD, H(1), kDesc128, O, kDesc64, kIdMK, 1);
        mma(tmem + cHD, H(0), kDesc128, O, kDesc64, kIdMK, 1);
#pragma unroll
        for (int order = 2; order >= 0; --order)
#pragma unroll
            for (int i = 2; i >= 0; --i) {
                const int j = order - i;
                if (j < 0) continue;
                mma(tmem + cHY, H(i), kDesc128, Y(j), kDesc128, kIdMM, order == 2 && i == 2 ? acc : 1);
                mma(tmem + cDU, G(i), kDesc128, U(j), kDesc128, kIdMM, order == 2 && i == 2 ? acc : 1);
            }
        // A of two terms: U(0) over U(1), and U(2) over zeros
        mma(tmem + cPP, U(2), kDesc128, O, kDesc64, kIdMK, acc);
        mma(tmem + cPP, U(0), kDesc128, O, kDesc64, kIdMK, 1);
        mma(tmem + cXX, U(2), kDesc128, Y(0), kDesc128, kIdMM, acc);
        mma(tmem + cXX, U(0), kDesc128, Y(2), kDesc128, kIdMM, 1);
        mma(tmem + cXX, U(0), kDesc128, Y(1), kDesc128, kIdMM, 1);
        mma(tmem + cXX, U(0), kDesc128, Y(0), kDesc128, kIdMM, 1);
    }
}

// EK = K^T E^T, SK = K^T S + Q^T E, of three terms of E and S
__device__ __forceinline__ void issue_tail(uint32_t tmem, uint32_t base)
{
    const uint32_t k0 = desc_lo(base + Smem::K, 8192), q0 = desc_lo(base + Smem::Q, 8192);
    const uint32_t e0 = desc_lo(base + Smem::E, 16), s0 = desc_lo(base + Smem::S, 16);
#pragma unroll
    for (int x = 2; x >= 0; --x)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t acc = x < 2 || k > 0, o = step_of(k * 2048), e = e0 + step_of(x * kSq);
            mma(tmem + cEK, k0 + o, kDesc128, e + o, kDesc128, kIdMM, acc);
            mma(tmem + cSK, k0 + o, kDesc128, s0 + step_of(x * kSq) + o, kDesc128, kIdMM, acc);
            mma(tmem + cSK, q0 + o, kDesc128, e + step_of(k * 32), kDesc128, kIdMK, 1);
        }
}

// The products of every chunk of this block, as the workers hand their operands over.
__device__ __forceinline__ void issuer(const BwdParams &p, Smem::Small &s, uint32_t tmem, uint32_t base)
{
    uint32_t phase[3] = {0, 0, 0};
    const int steps = p.dv / kRows;
    for (int u = blockIdx.x; u < p.nc * p.heads; u += gridDim.x)
        for (int dir = 0; dir < p.dirs; ++dir) {
            for (int step = 0; step < steps; ++step) {
                const int b = step & 1;
                if (!wait_bar(&s.full[b], phase[b], &s.abort, p.err, 64)) return;
                phase[b] ^= 1;
                tc_fence_after();
                issue_step(tmem, base, Smem::buf + b * kBuf, step);
                mma_commit(&s.done[b]);
            }
            if (!wait_bar(&s.full[2], phase[2], &s.abort, p.err, 64)) return;
            phase[2] ^= 1;
            tc_fence_after();
            issue_tail(tmem, base);
            mma_commit(&s.done[2]);
        }
}

// a warp's operands are written: hands them to the issuer
__device__ __forceinline__ void hand_over(uint64_t *bar)
{
    fence_proxy_async_smem();
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

template <bool BIDI>
__device__ __forceinline__ void workers(const BwdParams &p, Smem::Small &s, uint32_t tmem, unsigned char *sm)
{
    const uint32_t base = smem_u32(sm);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int quad = warp & 3, group = warp >> 2, t0 = 16 * group;   // this warp's lanes of tensor memory, its tokens t0 .. t0 + 15
    const int r = tid >> 4, c = tid & 15;                       // this thread's row of a step, its sixteenth of the columns
    const uint32_t mine = tmem + ((uint32_t)(32 * quad) << 16) + t0;
    uint32_t phase[3] = {0, 0, 0};
    const int steps = p.dv / kRows;
    bool ok = true;

    for (int u = blockIdx.x; u < p.nc * p.heads; u += gridDim.x) {
        const size_t first = u;                                 // the chunk's entry in the first direction
        float *const part = reinterpret_cast<float *>(p.unit + first * U1::size);   // bidirectional: the first direction's dQ, dK
        static_assert(2 * 64 * 128 * sizeof(float) <= U1::size, "the first direction's sums fit in its unit");
        if (tid < 64) s.db[tid] = s.da[tid] = 0.f;
        for (int dir = 0; dir < (BIDI ? 2 : 1); ++dir) {
            const Tile t = bwd::make_tile(p, dir, u / p.nc, u % p.nc);
            const unsigned char *unit = p.unit + t.ws * U1::size;
            const float *HT = p.HT + t.ws * p.dv * 128 + r * 128 + 8 * c, *GT = p.GT + t.ws * p.dv * 128 + r * 128 + 8 * c;
            const float *WT = p.WT + t.ws * p.dv * 64 + r * 64 + 4 * c, *ZT = p.ZT + t.ws * p.dv * 64 + r * 64 + 4 * c;
            const float *ZT0 = p.ZT + first * p.dv * 64 + r * 64;
            const bool last = !BIDI || dir == 1;
            bwd::copy_tile(smem_u32(&s.g), unit, sizeof(Gates), kWorkers);
            bwd::copy_tile(base + Smem::K, unit + U1::K, kKeys, kWorkers);
            bwd::copy_tile(base + Smem::Q, unit + U1::Q, kKeys, kWorkers);
            bwd::copy_tile(base + Smem::O, p.ot + t.ws * p.slices * (64 * 64), p.slices * 64 * 64, kWorkers);
            bwd::copy_commit();
            Step now;
            auto fetch = [&](Step &x, int step) {
                const size_t st = (size_t)step * kRows * 128, rw = (size_t)step * kRows * 64;
                read4(HT + st, x.h);
                read4(HT + st + 4, x.h + 4);
                read4(GT + st, x.g);
                read4(GT + st + 4, x.g + 4);
                read4(WT + rw, x.w);
                read4(ZT + rw, x.z);
                if (BIDI && dir == 1) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int i0 = t.n - 1 - 4 * c - i;     // the token's place in the first direction
                        x.z0[i] = i0 >= 0 ? __ldcg(ZT0 + rw + i0) : 0.f;
                    }
                }
            };
            bwd::copy_wait<0>();
            named_bar(1, kWorkers);

            float db[4] = {}, hh = 0.f;
            for (int step = 0; step < steps; ++step) {
                const int b = step & 1;
                unsigned char *const at = sm + Smem::buf + b * kBuf;
                fetch(now, step);
                if (step >= 2) {
                    ok = ok && wait_bar(&s.done[b], phase[b], &s.abort, p.err, 64);
                    phase[b] ^= 1;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) hh = fmaf(now.h[i], now.g[i], hh);
                bwd::planes8<128>(now.h, r, c & 7, at + oH + (c >> 3) * kHalf, kPlane);
                bwd::planes8<128>(now.g, r, c & 7, at + oG + (c >> 3) * kHalf, kPlane);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int ti = 4 * c + i;
                    const float beta = s.g.b[ti];
                    db[i] = fmaf(now.w[i], now.z[i], db[i]);
                    now.w[i] *= beta;
                    now.z[i] *= beta;
                    // dV = Y, of both directions: pairs of columns swizzled by the sixteenth of the tokens
                    if (last)
                        *reinterpret_cast<__nv_bfloat16 *>(sm + Smem::V + ti * 256 + (((step * 16 + (r >> 1)) ^ (2 * c)) * 4) + (r & 1) * 2) =
                            __float2bfloat16_rn(BIDI ? fmaf(beta, now.z0[i], now.z[i]) : now.z[i]);
                }
                planes4(now.w, r, c, at + oU, kVal);
                planes4(now.z, r, c, at + oY, kVal);
                hand_over(&s.full[b]);
            }
            hh = bwd::warp_sum(hh);
            if (lane == 0) s.hh[warp] = hh;
            // the walk after this one reads its states from L2
            if (tid < 6 && (!last || u + (int)gridDim.x < p.nc * p.heads)) {
                const size_t ws = last ? u + gridDim.x : first + (size_t)p.heads * p.nc;
                const size_t bytes = (size_t)p.dv * (tid < 2 ? 128 : 64) * 4;
                const char *from = tid == 0 ? reinterpret_cast<const char *>(p.HT) : tid == 1 ? reinterpret_cast<const char *>(p.GT)
                                 : tid == 2 ? reinterpret_cast<const char *>(p.WT) : reinterpret_cast<const char *>(p.ZT);
                if (tid < 4) prefetch_l2(from + ws * bytes, (uint32_t)bytes);
                else if (tid == 4) prefetch_l2(p.unit + ws * U1::size + U1::K, 2 * kKeys);
                else prefetch_l2(p.ot + ws * p.slices * 4096, p.slices * 4096);
            }
            // each buffer has one phase open
#pragma unroll
            for (int b = 0; b < 2; ++b)
                if (steps > b) {
                    ok = ok && wait_bar(&s.done[b], phase[b], &s.abort, p.err, 64);
                    phase[b] ^= 1;
                }
            tc_fence_after();
            ok = !named_bar_any(1, kWorkers, !ok);
            if (!ok) return;

            // db_i = Z_i . W_i: over a warp's two columns of dv here
            float *const dbw = reinterpret_cast<float *>(sm + Smem::dbw);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                db[i] += __shfl_xor_sync(0xffffffffu, db[i], 16);
                if (lane < 16) dbw[warp * 64 + 4 * lane + i] = db[i];
            }
            const bwd::Lift lift = bwd::lift_of(s.g);
            // m0_i = gam_i (q_i . H0 dO_i - k_i . H0 Y_i), m1_i = e_i k_i . dH1 U_i over this quadrant's dk
            const int d = 32 * quad + lane;                     // dk
            {
                const unsigned char *kq = sm + (d >> 6) * 8192 + (d & 7) * 2;
                float a[16], b[16], du[16];
                tmem_ld16(mine + cHD, a);
                tmem_ld16(mine + cHY, b);
                tmem_ld16(mine + cDU, du);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int o = (t0 + i) * 128 + ((((d & 63) >> 3) ^ (i & 7)) << 4);
                    const float k = __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(kq + Smem::K + o));
                    const float q = __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(kq + Smem::Q + o));
                    a[i] = fmaf(q, a[i], -k * b[i]);
                    b[i] = k * du[i];
                }
                const float m0 = sum_across(a), m1 = sum_across(b);
                if (lane < 16) {
                    s.m0[quad][t0 + lane] = s.g.from_entry(t0 + lane, lift.shift) * m0;
                    s.m1[quad][t0 + lane] = s.g.decay(63, t0 + lane, lift.shift) * m1;
                }
            }
            // PP and XX stand as two parts, in lanes j and 64 + j: the two threads take eight tokens each, give the
            // other its part of the rest, and the lower one its KK and QK of them
            const int upper = quad >> 1, j = 32 * (quad & 1) + lane, ti0 = t0 + 8 * upper, g8 = 2 * group + upper;
            float *const xP = reinterpret_cast<float *>(sm + Smem::xP) + j * kLd, *const xX = reinterpret_cast<float *>(sm + Smem::xX) + j * kLd;
            float *const xK = reinterpret_cast<float *>(sm + Smem::xK) + j * 32, *const xQ = xK + 64 * 32;
            float pp[8], xx[8], kk[8], qk[8];
            {
                float a[16], b[16];
                tmem_ld16(mine + cPP, a);
                tmem_ld16(mine + cXX, b);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    pp[i] = upper ? a[8 + i] : a[i];
                    xx[i] = upper ? b[8 + i] : b[i];
                    xP[t0 + 8 - 8 * upper + i] = upper ? a[i] : a[8 + i];
                    xX[t0 + 8 - 8 * upper + i] = upper ? b[i] : b[8 + i];
                }
                if (!upper) {
                    tmem_ld16(mine + cKK, a);
                    tmem_ld16(mine + cQK, b);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        kk[i] = a[i];
                        qk[i] = b[i];
                        xK[(8 * group + i) ^ lane] = a[8 + i];
                        xQ[(8 * group + i) ^ lane] = b[8 + i];
                    }
                }
            }
            named_bar(1, kWorkers);
            // the contracted token j is this thread's row of E^T, F^T, M^T
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int ti = ti0 + i;
                if (upper) {
                    kk[i] = xK[(8 * group + i) ^ lane];
                    qk[i] = xQ[(8 * group + i) ^ lane];
                }
                const float dc = j <= ti ? s.g.decay(ti, j, lift.shift) : 0.f;
                const float x = j <= ti ? dc * (pp[i] + xP[ti]) : 0.f;                   // E
                const float f = j < ti ? -dc * (xx[i] + xX[ti]) : 0.f;                   // F
                xP[ti] = f * lift.down;
                kk[i] = j < ti ? f * kk[i] + x * qk[i] : 0.f;                            // M
                pp[i] = x * lift.down;
            }
            {
                uint32_t v[4][3];
#pragma unroll
                for (int i = 0; i < 4; ++i) bwd::split2<3>(pp[2 * i], pp[2 * i + 1], v[i]);
#pragma unroll
                for (int x = 0; x < 3; ++x)
                    *reinterpret_cast<uint4 *>(sm + Smem::E + x * kSq + bwd::sw<128>(j, g8)) = make_uint4(v[0][x], v[1][x], v[2][x], v[3][x]);
            }
            // sums of M over this warp's i >= t for each of its t, then over its lanes j < t; its tokens' whole sum for each
            // j goes to the earlier tokens
            {
                float run = 0.f;
#pragma unroll
                for (int i = 7; i >= 0; --i) {
                    run += kk[i];
                    kk[i] = j < ti0 + i ? run : 0.f;
                }
                s.whole[g8][j] = run;
                const float sum = sum_across(kk);
                if (lane < 8) s.col[quad & 1][ti0 + lane] = sum;
            }
            named_bar(1, kWorkers);
            {                                                   // S = F + F^T
                const int row = tid >> 3, c2 = tid & 7;
                const float *f = reinterpret_cast<const float *>(sm + Smem::xP);
                uint32_t v[4][3];
#pragma unroll
                for (int i = 0; i < 8; i += 2)
                    bwd::split2<3>(f[row * kLd + 8 * c2 + i] + f[(8 * c2 + i) * kLd + row],
                                   f[row * kLd + 8 * c2 + i + 1] + f[(8 * c2 + i + 1) * kLd + row], v[i / 2]);
#pragma unroll
                for (int x = 0; x < 3; ++x)
                    *reinterpret_cast<uint4 *>(sm + Smem::S + x * kSq + bwd::sw<128>(row, c2)) = make_uint4(v[0][x], v[1][x], v[2][x], v[3][x]);
            }
            hand_over(&s.full[2]);                              // PP and XX are read: EK and SK may take their place
            if (quad == 3) {
                // da_t = (sum over i >= t, j < t of M with its entry column and end row) / a_t: the lane has j (or i) = lane
                // and lane + 32
                float v[16], from[2], m0[2], more[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int jj = lane + 32 * x;
                    from[x] = (s.m1[0][jj] + s.m1[1][jj]) + (s.m1[2][jj] + s.m1[3][jj]);
                    m0[x] = (s.m0[0][jj] + s.m0[1][jj]) + (s.m0[2][jj] + s.m0[3][jj]);
                    for (int y = 2 * group + 2; y < 8; ++y) from[x] += s.whole[y][jj];
                    more[x] = from[x] + s.whole[2 * group + 1][jj];
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int ti = t0 + i;
                    const float lo = i < 8 ? more[0] : from[0], hi = i < 8 ? more[1] : from[1];
                    v[i] = (lane < ti ? lo : m0[0]) + (lane + 32 < ti ? hi : m0[1]);
                }
                float x = sum_across(v), end = 0.f, b = 0.f;
                const int ti = t0 + (lane & 15);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    end += s.hh[i];
                    b += dbw[i * 64 + ti];
                }
                x += fmaf(end, s.g.from_entry(63, lift.shift), s.col[0][ti] + s.col[1][ti]);
                if (lane < 16 && ti < t.n) {
                    const int tok = t.tok(ti) - t.c * 64;
                    s.da[tok] += x / (s.g.a[ti] * lift.up);
                    s.db[tok] += b;
                }
            }
            ok = ok && wait_bar(&s.done[2], phase[2], &s.abort, p.err, 64);
            phase[2] ^= 1;
            tc_fence_after();
            ok = !named_bar_any(1, kWorkers, !ok);
            if (!ok) return;
            // dQ = gam HD + EK;  dK = e DU - gam HY + SK: rows by token, in shared memory on their way out.  The reverse
            // walk's token i is row 63 - i, so that rows behind the sequence's end need no test
            auto put = [&](const float (&v)[16], int which) {
                if (!last) {
                    float *at = part + which * 64 * 128 + t0 * 128 + d;
#pragma unroll
                    for (int i = 0; i < 16; ++i) __stcg(at + i * 128, v[i]);
                    return;
                }
                __nv_bfloat16 *to = reinterpret_cast<__nv_bfloat16 *>(sm + Smem::out + which * kKeys) + d;
                if (BIDI) {
                    const float *at = part + which * 64 * 128 + d;
                    float x[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = __ldcg(at + max(t.n - 1 - t0 - i, 0) * 128);
#pragma unroll
                    for (int i = 0; i < 16; ++i) to[(63 - t0 - i) * 128] = __float2bfloat16_rn(v[i] + x[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) to[(t0 + i) * 128] = __float2bfloat16_rn(v[i]);
                }
            };
            {
                float a[16], b[16], e[16];
                tmem_ld16(mine + cHD, a);
                tmem_ld16(mine + cEK, b);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) a[i] = fmaf(s.g.gam[t0 + i], a[i], b[i]);
                put(a, 0);
                tmem_ld16(mine + cHY, a);
                tmem_ld16(mine + cSK, b);
                tmem_ld16(mine + cDU, e);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) a[i] = fmaf(s.g.e[t0 + i], e[i], fmaf(-s.g.gam[t0 + i], a[i], b[i]));
                put(a, 1);
            }
            named_bar(1, kWorkers);
            if (last) {
                for (int e = tid; e < 2 * t.n * 16; e += kWorkers) {
                    const int which = e >= t.n * 16, row = (e - which * t.n * 16) >> 4, piece = e & 15;
                    if (8 * piece >= p.dk) continue;            // dk = 96 is padded to 128
                    __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(which ? p.dk_ : p.dq);
                    *reinterpret_cast<uint4 *>(to + ((size_t)t.head * p.T + t.c * 64 + row) * p.dk + 8 * piece) =
                        *reinterpret_cast<const uint4 *>(sm + Smem::out + which * kKeys + (BIDI ? 64 - t.n + row : row) * 256 + piece * 16);
                }
                for (int e = tid; e < t.n * 32; e += kWorkers) {
                    const int row = e >> 5, two = 2 * (e & 31);                 // four columns of a token
                    if (2 * two >= p.dv) continue;
                    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.dv_) + ((size_t)t.head * p.T + t.tok(row)) * p.dv + 2 * two) =
                        *reinterpret_cast<const uint2 *>(sm + Smem::V + row * 256 + (two ^ (2 * (row >> 2))) * 4);
                }
                if (tid < t.n) {
                    const size_t at = (size_t)t.head * p.T + t.c * 64 + tid;
                    p.dbeta[at] = s.db[tid];
                    p.ddecay[at] = s.da[tid];
                }
            }
        }
    }
}

template <bool BIDI>
__global__ void __launch_bounds__(kThreads, 1) bwd_grad_tc_kernel(const __grid_constant__ BwdParams p)
{
    extern __shared__ unsigned char dyn[];
    unsigned char *const sm = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~(uintptr_t)1023);
    Smem::Small &s = *reinterpret_cast<Smem::Small *>(sm + Smem::end);
    const int tid = threadIdx.x, warp = tid >> 5;
    if (warp == 0) tmem_alloc(&s.tmem, kCols);
    if (tid == 0) {
        for (int i = 0; i < 3; ++i) {
            mbar_init(&s.full[i], kWorkers / 32 + (p.stall && p.head0 + blockIdx.x + i == 0));
            mbar_init(&s.done[i], 1);
        }
        mbar_init(&s.drain, 1);
        s.abort = 0;
        fence_mbar_init();
    }
    for (int e = tid; e < 2 * kVal / 16; e += kThreads)
        *reinterpret_cast<uint4 *>(sm + Smem::buf + (e / (kVal / 16)) * kBuf + oZero + (e % (kVal / 16)) * 16) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem;
    if (tid < kWorkers) workers<BIDI>(p, s, tmem, sm);
    else if (tid == kWorkers) issuer(p, s, tmem, smem_u32(sm));
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (*static_cast<volatile int *>(&s.abort)) {
        // products still in flight read shared memory and write tensor memory: none may outlive the block
        if (tid == kWorkers) {
            mma_commit(&s.drain);
            drain_copies(&s.drain, 0);
        }
        __syncthreads();
    }
    if (warp == 0) {
        tmem_relinquish();
        tmem_dealloc(tmem, kCols);
    }
}

}  // namespace

namespace bwd {

cudaError_t set_wait_limit_tc(unsigned long long ns) { return set_module_wait_limit(ns); }

cudaError_t launch_grad_tc(const BwdParams &p, cudaStream_t stream)
{
    auto *kernel = p.dirs == 2 ? bwd_grad_tc_kernel<true> : bwd_grad_tc_kernel<false>;
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem::bytes);
    if (err != cudaSuccess) return err;
    // a block fills an SM (shared and tensor memory): one for each, walking the chunks
    int dev = 0, sms = 0;
    err = cudaGetDevice(&dev);
    if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (err != cudaSuccess) return err;
    const long long units = (long long)p.nc * p.heads;
    kernel<<<(unsigned)(units < sms ? units : sms), kThreads, Smem::bytes, stream>>>(p);
    err = cudaGetLastError();
    if (err == cudaSuccess) count_launches(1);
    return err;
}

}  // namespace bwd
}  // namespace gdn
