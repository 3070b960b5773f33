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
// step's loads and splitting run beside the tensor core.  Products of terms are those of order i + j < 3, the small
// ones first.
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

constexpr int kThreads = 512;
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
    // Offsets from a 1024-byte boundary.  Behind the walk over dv the buffers hold the exchanged halves of PP and
    // XX (the place of H0 and dH1 of the first), F^T over PP's, and the terms of E^T and S (of the second).
    static constexpr int K = 0, Q = K + kKeys, O = Q + kKeys, buf = O + 4 * 64 * 64, end = buf + 2 * kBuf;
    static constexpr int xP = buf, xX = xP + 64 * kLd * 4, E = buf + kBuf, S = E + 2 * kSq;
    static_assert(xX + 64 * kLd * 4 <= buf + oU && S + 2 * kSq <= buf + kBuf + oU, "the walk's zeros stay");
    struct Small {
        Gates g;
        float z[kRows * kLd], z0[kRows * kLd];  // the step's b Z, and the first direction's
        float db[64], da[64];                   // over the directions, by token
        float m0[4][64], m1[4][64], dbw[16][64], col[2][64], whole[4][64], hh[16];
        uint64_t bar[3];                        // a buffer's products are done; the chunk's other products
        uint32_t tmem;
        int abort;
    };
    static constexpr int bytes = end + (int)sizeof(Small) + 1024;
};
static_assert(Smem::bytes <= 227 * 1024, "shared memory");

constexpr uint32_t kIdMK = idesc_bf16(128, 64, true, false);    // A MN-major, B K-major
constexpr uint32_t kIdMM = idesc_bf16(128, 64, true, true);
constexpr uint32_t kIdKK = idesc_bf16(128, 64, false, false);

// K-major tile of 64-byte rows, 64-byte swizzle
__device__ __forceinline__ uint64_t sw64_desc(uint32_t saddr)
{
    return (uint64_t)((saddr >> 4) & 0x3FFF) | (uint64_t)1 << 16 | (uint64_t)(512 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)4 << 61;
}

// lanes l and l + 16 get the sum over the warp's lanes of their v[l]
__device__ __forceinline__ float sum_across(float (&v)[16])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 8; o; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float mine = up ? v[i + o] : v[i], theirs = up ? v[i] : v[i + o];
            v[i] = mine + __shfl_xor_sync(0xffffffffu, theirs, o);
        }
    }
    return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
}

__device__ __forceinline__ void read4(const float *p, float *x)
{
    const float4 u = __ldcg(reinterpret_cast<const float4 *>(p));
    x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
}

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

__global__ void __launch_bounds__(kThreads, 1) bwd_grad_tc_kernel(const __grid_constant__ BwdParams p, int *err)
{
    extern __shared__ unsigned char dyn[];
    unsigned char *const sm = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~(uintptr_t)1023);
    Smem::Small &s = *reinterpret_cast<Smem::Small *>(sm + Smem::end);
    const uint32_t base = smem_u32(sm);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int quad = warp & 3, group = warp >> 2, t0 = 16 * group;   // this warp's lanes of tensor memory, its tokens t0 .. t0 + 15
    const int r = tid >> 4, c = tid & 15;                       // this thread's row of a step, its sixteenth of the columns
    const size_t first = (size_t)blockIdx.y * p.nc + blockIdx.x;
    float *const part = reinterpret_cast<float *>(p.unit + first * U1::size);   // bidirectional: the first direction's dQ, dK
    static_assert(2 * 64 * 128 * sizeof(float) <= U1::size, "the first direction's sums fit in its unit");

    if (warp == 0) tmem_alloc(&s.tmem, kCols);
    if (tid == 0) {
        for (int i = 0; i < 3; ++i) mbar_init(&s.bar[i], 1);
        s.abort = 0;
        fence_mbar_init();
    }
    if (tid < 64) s.db[tid] = s.da[tid] = 0.f;
    for (int e = tid; e < 2 * kVal / 16; e += kThreads)
        *reinterpret_cast<uint4 *>(sm + Smem::buf + (e / (kVal / 16)) * kBuf + oZero + (e % (kVal / 16)) * 16) = make_uint4(0, 0, 0, 0);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem, mine = tmem + ((uint32_t)(32 * quad) << 16) + t0;
    uint32_t phase[3] = {0, 0, 0};
    const int steps = p.dv / kRows;
    bool ok = true;

    for (int dir = 0; dir < p.dirs; ++dir) {
        const Tile t = bwd::make_tile(p, dir, blockIdx.y, blockIdx.x);
        const unsigned char *unit = p.unit + t.ws * U1::size;
        const float *HT = p.HT + t.ws * p.dv * 128 + r * 128 + 8 * c, *GT = p.GT + t.ws * p.dv * 128 + r * 128 + 8 * c;
        const float *WT = p.WT + t.ws * p.dv * 64 + r * 64 + 4 * c, *ZT = p.ZT + t.ws * p.dv * 64 + r * 64 + 4 * c;
        const float *ZT0 = p.ZT + first * p.dv * 64 + r * 64 + 4 * c;
        const bool last = dir == p.dirs - 1;
        bwd::copy_block(smem_u32(&s.g), unit, sizeof(Gates));
        bwd::copy_block(base + Smem::K, unit + U1::K, kKeys);
        bwd::copy_block(base + Smem::Q, unit + U1::Q, kKeys);
        bwd::copy_block(base + Smem::O, p.ot + t.ws * p.slices * (64 * 64), p.slices * 64 * 64);
        bwd::copy_commit();
        float h[8], g[8], w[4], z[4], z0[4];
        auto fetch = [&](int step) {
            const size_t st = (size_t)step * kRows * 128, rw = (size_t)step * kRows * 64;
            read4(HT + st, h);
            read4(HT + st + 4, h + 4);
            read4(GT + st, g);
            read4(GT + st + 4, g + 4);
            read4(WT + rw, w);
            read4(ZT + rw, z);
            if (dir == 1) read4(ZT0 + rw, z0);
        };
        fetch(0);
        bwd::copy_wait<0>();
        fence_proxy_async_smem();
        __syncthreads();

        float db[4] = {}, hh = 0.f;
        for (int step = 0; step < steps; ++step) {
            const int b = step & 1, at = Smem::buf + b * kBuf;
            if (step >= 2) {
                ok = ok && wait_bar(&s.bar[b], phase[b], &s.abort, err, 64);
                phase[b] ^= 1;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) hh = fmaf(h[i], g[i], hh);
            bwd::planes8<128>(h, r, c & 7, sm + at + oH + (c >> 3) * kHalf, kPlane);
            bwd::planes8<128>(g, r, c & 7, sm + at + oG + (c >> 3) * kHalf, kPlane);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float beta = s.g.b[4 * c + i];
                db[i] = fmaf(w[i], z[i], db[i]);
                w[i] *= beta;
                z[i] *= beta;
                s.z[r * kLd + 4 * c + i] = z[i];
                if (dir == 1) s.z0[r * kLd + 4 * c + i] = z0[i];
            }
            planes4(w, r, c, sm + at + oU, kVal);
            planes4(z, r, c, sm + at + oY, kVal);
            fence_proxy_async_smem();
            ok = !__syncthreads_or(!ok);
            if (!ok) break;
            if (tid == 0) {
                tc_fence_after();
                if (step == 0) {                                // K K^T, K Q^T: lanes 64 - 127 multiply what follows K
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint32_t o = (k >> 2) * 8192 + (k & 3) * 32;
                        const uint64_t a = sw128_desc(base + Smem::K + o, 16, 1024);
                        mma_bf16(tmem + cKK, a, a, kIdKK, k > 0);
                        mma_bf16(tmem + cQK, a, sw128_desc(base + Smem::Q + o, 16, 1024), kIdKK, k > 0);
                    }
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t k0 = base + at + k * 2048, acc = step > 0 || k > 0;
                    const uint64_t O = sw64_desc(base + Smem::O + step * 4096 + k * 32);
                    uint64_t H[3], G[3], U[3], Y[3];
#pragma unroll
                    for (int i = 0; i < 3; ++i) {
                        H[i] = sw128_desc(k0 + oH + i * kPlane, kHalf, 1024);
                        G[i] = sw128_desc(k0 + oG + i * kPlane, kHalf, 1024);
                        U[i] = sw128_desc(k0 + oU + i * kVal, kVal, 1024);
                        Y[i] = sw128_desc(k0 + oY + i * kVal, kVal, 1024);
                    }
                    mma_bf16(tmem + cHD, H[2], O, kIdMK, acc);
                    mma_bf16(tmem + cHD, H[1], O, kIdMK, 1);
                    mma_bf16(tmem + cHD, H[0], O, kIdMK, 1);
#pragma unroll
                    for (int order = 2; order >= 0; --order)
#pragma unroll
                        for (int i = 2; i >= 0; --i) {
                            const int j = order - i;
                            if (j < 0) continue;
                            mma_bf16(tmem + cHY, H[i], Y[j], kIdMM, order == 2 && i == 2 ? acc : 1);
                            mma_bf16(tmem + cDU, G[i], U[j], kIdMM, order == 2 && i == 2 ? acc : 1);
                        }
                    // A of two terms: U[0] over U[1], and U[2] over zeros
                    mma_bf16(tmem + cPP, U[2], O, kIdMK, acc);
                    mma_bf16(tmem + cPP, U[0], O, kIdMK, 1);
                    mma_bf16(tmem + cXX, U[2], Y[0], kIdMM, acc);
                    mma_bf16(tmem + cXX, U[0], Y[2], kIdMM, 1);
                    mma_bf16(tmem + cXX, U[0], Y[1], kIdMM, 1);
                    mma_bf16(tmem + cXX, U[0], Y[0], kIdMM, 1);
                }
                mma_commit(&s.bar[b]);
            }
            if (step + 1 < steps) fetch(step + 1);
            if (last) {                                         // dV = Y, of both directions
                for (int e = tid; e < t.n * (kRows / 2); e += kThreads) {
                    const int i = e / (kRows / 2), j = 2 * (e % (kRows / 2));
                    float x = s.z[j * kLd + i], y = s.z[(j + 1) * kLd + i];
                    if (dir == 1) {
                        x = fmaf(s.g.b[i], s.z0[j * kLd + t.n - 1 - i], x);
                        y = fmaf(s.g.b[i], s.z0[(j + 1) * kLd + t.n - 1 - i], y);
                    }
                    bwd::st2(static_cast<__nv_bfloat16 *>(p.dv_) + ((size_t)t.head * p.T + t.tok(i)) * p.dv + step * kRows + j, x, y);
                }
            }
            __syncthreads();                                    // z is free again
        }
        if (!ok) break;
        // db_i = Z_i . W_i: over a warp's two rows of dv here, over the warps below; <H0, dH1> likewise
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            db[i] += __shfl_xor_sync(0xffffffffu, db[i], 16);
            if (lane < 16) s.dbw[warp][4 * lane + i] = db[i];
        }
        hh = bwd::warp_sum(hh);
        if (lane == 0) s.hh[warp] = hh;
        // a buffer's last products: with an even number of steps both buffers have one phase open
#pragma unroll
        for (int b = 0; b < 2; ++b)
            if (steps > b) {
                ok = ok && wait_bar(&s.bar[b], phase[b], &s.abort, err, 64);
                phase[b] ^= 1;
            }
        tc_fence_after();
        ok = !__syncthreads_or(!ok);
        if (!ok) break;

        // lanes 64 - 127 of PP and XX hand their half over; m0_i = gam_i (q_i . H0 dO_i - k_i . H0 Y_i), m1_i = e_i
        // k_i . dH1 U_i over this quadrant's dk
        float *const xP = reinterpret_cast<float *>(sm + Smem::xP), *const xX = reinterpret_cast<float *>(sm + Smem::xX);
        float pp[16], xx[16];
        tmem_ld16(mine + cPP, pp);
        tmem_ld16(mine + cXX, xx);
        tmem_wait_ld();
        if (quad >= 2) {
            const int j = 32 * (quad - 2) + lane;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                xP[j * kLd + t0 + i] = pp[i];
                xX[j * kLd + t0 + i] = xx[i];
            }
        }
        {
            const int d = 32 * quad + lane;                     // dk
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
                s.m0[quad][t0 + lane] = s.g.gam[t0 + lane] * m0;
                s.m1[quad][t0 + lane] = s.g.e[t0 + lane] * m1;
            }
        }
        __syncthreads();
        if (quad < 2) {
            const int j = 32 * quad + lane;                     // the contracted token: this lane's row of E^T, F^T, M^T
            float kk[16], qk[16];
            tmem_ld16(mine + cKK, kk);
            tmem_ld16(mine + cQK, qk);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int ti = t0 + i;
                const float d = j <= ti ? exp2f((float)(s.g.G[ti] - s.g.G[j])) : 0.f;
                const float x = d * (pp[i] + xP[j * kLd + ti]);                          // E
                const float f = j < ti ? -d * (xx[i] + xX[j * kLd + ti]) : 0.f;          // F
                xP[j * kLd + ti] = f;
                kk[i] = j < ti ? f * kk[i] + x * qk[i] : 0.f;                            // M
                pp[i] = x;
            }
#pragma unroll
            for (int c2 = 0; c2 < 2; ++c2) {
                uint32_t u[2][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t v[2];
                    bwd::split2<2>(pp[8 * c2 + 2 * i], pp[8 * c2 + 2 * i + 1], v);
                    u[0][i] = v[0];
                    u[1][i] = v[1];
                }
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    *reinterpret_cast<uint4 *>(sm + Smem::E + x * kSq + bwd::sw<128>(j, t0 / 8 + c2)) = make_uint4(u[x][0], u[x][1], u[x][2], u[x][3]);
            }
            // sums of M over this warp's i >= t for each of its t, then over its lanes j < t; its tokens' whole sum
            // for each j goes to the earlier groups
            float run = 0.f;
#pragma unroll
            for (int i = 15; i >= 0; --i) {
                run += kk[i];
                kk[i] = j < t0 + i ? run : 0.f;
            }
            s.whole[group][j] = run;
            const float sum = sum_across(kk);
            if (lane < 16) s.col[quad][t0 + lane] = sum;
        }
        __syncthreads();
        {                                                       // S = F + F^T
            const int j = tid >> 3, c2 = tid & 7;
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = xP[j * kLd + 8 * c2 + i] + xP[(8 * c2 + i) * kLd + j];
            uint32_t u[2][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t v[2];
                bwd::split2<2>(x[2 * i], x[2 * i + 1], v);
                u[0][i] = v[0];
                u[1][i] = v[1];
            }
#pragma unroll
            for (int y = 0; y < 2; ++y)
                *reinterpret_cast<uint4 *>(sm + Smem::S + y * kSq + bwd::sw<128>(j, c2)) = make_uint4(u[y][0], u[y][1], u[y][2], u[y][3]);
        }
        tc_fence_before();                                      // PP and XX are read
        fence_proxy_async_smem();
        __syncthreads();
        if (tid == 0) {
            tc_fence_after();
#pragma unroll
            for (int x = 1; x >= 0; --x)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint64_t K = sw128_desc(base + Smem::K + k * 2048, 8192, 1024), Q = sw128_desc(base + Smem::Q + k * 2048, 8192, 1024);
                    const uint32_t e = base + Smem::E + x * kSq, sy = base + Smem::S + x * kSq;
                    const uint32_t acc = x == 0 || k > 0;
                    mma_bf16(tmem + cEK, K, sw128_desc(e + k * 2048, 8192, 1024), kIdMM, acc);
                    mma_bf16(tmem + cSK, K, sw128_desc(sy + k * 2048, 8192, 1024), kIdMM, acc);
                    mma_bf16(tmem + cSK, Q, sw128_desc(e + k * 32, 16, 1024), kIdMK, 1);
                }
            mma_commit(&s.bar[2]);
        }
        if (quad == 3) {
            // da_t = (sum over i >= t, j < t of M with its entry column and end row) / a_t: the lane has j (or i) = lane
            // and lane + 32
            float v[16], from[2], m0[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int j = lane + 32 * u;
                from[u] = (s.m1[0][j] + s.m1[1][j]) + (s.m1[2][j] + s.m1[3][j]);
                m0[u] = (s.m0[0][j] + s.m0[1][j]) + (s.m0[2][j] + s.m0[3][j]);
                for (int x = group + 1; x < 4; ++x) from[u] += s.whole[x][j];
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int ti = t0 + i;
                v[i] = (lane < ti ? from[0] : m0[0]) + (lane + 32 < ti ? from[1] : m0[1]);
            }
            float x = sum_across(v), end = 0.f, b = 0.f;
            const int ti = t0 + (lane & 15);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                end += s.hh[i];
                b += s.dbw[i][ti];
            }
            x += fmaf(end, s.g.gam[63], s.col[0][ti] + s.col[1][ti]);
            if (lane < 16 && ti < t.n) {
                const int at = t.tok(ti) - t.c * 64;
                s.da[at] += x / s.g.a[ti];
                s.db[at] += b;
            }
        }
        ok = ok && wait_bar(&s.bar[2], phase[2], &s.abort, err, 64);
        phase[2] ^= 1;
        ok = !__syncthreads_or(!ok);
        if (!ok) break;
        tc_fence_after();
        // dQ = gam HD + EK;  dK = e DU - gam HY + SK
        const int d = 32 * quad + lane;
        auto put = [&](const float (&v)[16], void *to, float *sum) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if (t0 + i >= t.n || d >= p.dk) break;          // dk = 96 is padded to 128
                const int tok = t.tok(t0 + i);
                float x = v[i], *at = sum + (tok - t.c * 64) * 128 + d;
                if (!last) {
                    __stcg(at, x);
                    continue;
                }
                if (dir == 1) x += __ldcg(at);
                static_cast<__nv_bfloat16 *>(to)[((size_t)t.head * p.T + tok) * p.dk + d] = __float2bfloat16_rn(x);
            }
        };
        float a[16], b[16], e[16];
        tmem_ld16(mine + cHD, a);
        tmem_ld16(mine + cEK, b);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) a[i] = fmaf(s.g.gam[t0 + i], a[i], b[i]);
        put(a, p.dq, part);
        tmem_ld16(mine + cHY, a);
        tmem_ld16(mine + cSK, b);
        tmem_ld16(mine + cDU, e);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) a[i] = fmaf(s.g.e[t0 + i], e[i], fmaf(-s.g.gam[t0 + i], a[i], b[i]));
        put(a, p.dk_, part + 64 * 128);
        tc_fence_before();
        __syncthreads();                                        // tensor memory and the buffers are free again
        tc_fence_after();
    }
    if (ok) {
        const int start = blockIdx.x * 64, n = min(64, p.T - start);
        if (tid < n) {
            const size_t at = (size_t)(p.head0 + blockIdx.y) * p.T + start + tid;
            p.dbeta[at] = s.db[tid];
            p.ddecay[at] = s.da[tid];
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tmem_relinquish();
        tmem_dealloc(tmem, kCols);
    }
}

}  // namespace

namespace bwd {

cudaError_t launch_grad_tc(const BwdParams &p, cudaStream_t stream)
{
    int *word = nullptr;
    cudaError_t err = device_error_word(&word);
    if (err == cudaSuccess) err = cudaFuncSetAttribute(bwd_grad_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem::bytes);
    if (err != cudaSuccess) return err;
    bwd_grad_tc_kernel<<<dim3(p.nc, p.heads), kThreads, Smem::bytes, stream>>>(p, word);
    err = cudaGetLastError();
    if (err == cudaSuccess) count_launches(1);
    return err;
}

}  // namespace bwd
}  // namespace gdn
