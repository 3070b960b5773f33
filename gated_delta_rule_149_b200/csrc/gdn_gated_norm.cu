// The read-out of the recurrence, normalised per head, scaled and gated, and the gradients of that:
//     n = o / sqrt(mean(o^2) + eps),   y = n w silu(g)                 per row of dv values
//     dn = dy w silu(g),   do = r (dn - n mean(dn n)),   r = 1 / sqrt(mean(o^2) + eps)
//     dg = dy n w (s + g s (1 - s)),   s = sigmoid(g),   dw = sum over rows of dy silu(g) n
//
// One pass over the data, which bounds it: o is read head-major as the recurrence writes it, gate and y are
// token-major as the projections around it take them; a row's 16-byte pieces lie in one group of lanes and its
// sums are shuffles.  A block keeps one head and walks tokens, so that a thread's columns of the weight, and its
// sums for dw, stay in registers; the blocks' sums of dw go to a workspace and a second small kernel adds them in
// a fixed order, so that dw is the same every time.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;            // values of a row per lane

struct NormParams {
    View o, gate, y, dy, dout, dgate;
    const float *weight;
    long long w_head;              // elements between two heads' weights (0: shared)
    float *part;                   // [head][batch][block][dv] sums for dw, or nullptr
    int T, dv, per_block;          // tokens per block
    float eps;
};

// A lane's values of a row: VEC, values 8 l .. 8 l + 7 by 16-byte accesses; otherwise l, l + LPR, ...  (16 x 12000 rows of 80
// bf16 values: 32 us, off 16-byte boundaries 56; of 33 values, 1 x 16 x 32000: 124 us, 32 values by pieces 30)
template <bool VEC, int LPR>
__device__ __forceinline__ int column(int l, int i) { return VEC ? kPer * l + i : l + LPR * i; }

template <bool VEC, int LPR>
__device__ __forceinline__ void load(const __nv_bfloat16 *p, int l, int dv, float *f)
{
    if (VEC) {
        const uint4 u = *reinterpret_cast<const uint4 *>(p + 8 * l);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) f[i] = l + LPR * i < dv ? __bfloat162float(p[l + LPR * i]) : 0.f;
    }
}

template <bool VEC, int LPR>
__device__ __forceinline__ void load(const float *p, int l, int dv, float *f)
{
    if (VEC) {
        const float4 a = reinterpret_cast<const float4 *>(p + 8 * l)[0], b = reinterpret_cast<const float4 *>(p + 8 * l)[1];
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) f[i] = l + LPR * i < dv ? p[l + LPR * i] : 0.f;
    }
}

template <bool VEC, int LPR>
__device__ __forceinline__ void store(__nv_bfloat16 *p, int l, int dv, const float *f)
{
    if (VEC) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&v);
        }
        *reinterpret_cast<uint4 *>(p + 8 * l) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (l + LPR * i < dv) p[l + LPR * i] = __float2bfloat16_rn(f[i]);
    }
}

template <bool VEC, int LPR>
__device__ __forceinline__ void store(float *p, int l, int dv, const float *f)
{
    if (VEC) {
        reinterpret_cast<float4 *>(p + 8 * l)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4 *>(p + 8 * l)[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (l + LPR * i < dv) p[l + LPR * i] = f[i];
    }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float x)
{
#pragma unroll
    for (int o = LPR / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// 1 / (1 + 2^(-x log2 e)) by the hardware's approximations of 2^y (2^-22 of itself) and of the reciprocal (2^-23); results under
// 2^-126 go to 0.  The rounding of x log2 e costs another 2^-24 |x| of the power.  For fp32 it is taken in two parts,
// 2^(high + low) = 2^high (1 + low ln 2 + ..), which leaves 2^-21 of the result at either end.
template <typename T> __device__ __forceinline__ float sigmoid(float x);
template <> __device__ __forceinline__ float sigmoid<float>(float x)
{
    // between these bounds the parts are finite; beyond them it is 1, or 0.  (NaN as one of them: callers multiply by x.)
    const float t = fminf(fmaxf(x, -88.f), 80.f), high = t * -1.442695022f;
    const float low = fmaf(t, -1.925963034e-8f, fmaf(t, -1.442695022f, -high));
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(high));
    e = fmaf(e, low * 0.6931471806f, e);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}
// For bf16 it is left: 7e-8 |x| of the power, 6e-6 at a gate of -87, where results are rounded to 2^-9.  (Taken in two parts, the
// 720p clip's backward takes 544 us, not 533; with the bounds as for fp32, 564.)
template <> __device__ __forceinline__ float sigmoid<__nv_bfloat16>(float x)
{
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.442695041f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}

// Grid (token tiles, heads, batches).  Blocks to an SM: enough warps to cover the loads' latency count for more than rows
// in flight per thread.  (720p clip, 2 x 16 x 75600 rows of 128 bf16 values: backward 532 us with four blocks, 551 us with four
// and two rows in flight, 607 us with three and two; 650 us with five, which spill.)
template <typename T, bool VEC, int LPR, bool GATE, bool BACK>
__global__ void __launch_bounds__(kThreads, BACK ? 4 : 6) gated_norm_kernel(const __grid_constant__ NormParams p)
{
    constexpr int kGroups = kThreads / LPR;
    const int l = threadIdx.x % LPR, group = threadIdx.x / LPR;
    const int h = blockIdx.y, b = blockIdx.z;
    const bool lane_on = column<VEC, LPR>(l, 0) < p.dv;
    const float inv = 1.f / p.dv;
    float w[kPer], dw[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int c = column<VEC, LPR>(l, i);
        w[i] = p.weight && c < p.dv ? p.weight[h * p.w_head + c] : 1.f;
        dw[i] = 0.f;
    }
    const long long t0 = (long long)blockIdx.x * p.per_block;
    const int count = (int)min((long long)p.per_block, p.T - t0), rounds = (count + kGroups - 1) / kGroups;
    // a thread's rows, kGroups tokens apart
    auto rows = [&](const View &v) { return const_cast<T *>(static_cast<const T *>(v.p)) + b * v.sb + h * v.sh + (t0 + group) * v.st; };
    const T *o = rows(p.o), *gate = rows(p.gate), *dy = rows(p.dy);
    T *y = rows(p.y), *dout = rows(p.dout), *dgate = rows(p.dgate);
#pragma unroll 1
    for (int k = 0; k < rounds; ++k) {
        const bool act = lane_on && group + k * kGroups < count;
        float x[kPer], g[kPer], z[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) x[i] = g[i] = z[i] = 0.f;
        if (act) {
            load<VEC, LPR>(o, l, p.dv, x);
            if (GATE) load<VEC, LPR>(gate, l, p.dv, g);
            if (BACK) load<VEC, LPR>(dy, l, p.dv, z);
        }
        o += kGroups * p.o.st;
        if (GATE) gate += kGroups * p.gate.st;
        if (BACK) dy += kGroups * p.dy.st;
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) sq = fmaf(x[i], x[i], sq);
        const float r = rsqrtf(fmaf(row_sum<LPR>(sq), inv, p.eps));
        if (!BACK) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                x[i] = x[i] * r * w[i];
                if (GATE) x[i] *= g[i] * sigmoid<T>(g[i]);
            }
            if (act) store<VEC, LPR>(y, l, p.dv, x);
            y += kGroups * p.y.st;
        } else {
            float dot = 0.f, dg[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const float n = x[i] * r, zn = z[i] * n;
                float act_ = 1.f;
                if (GATE) {
                    const float s = sigmoid<T>(g[i]);
                    act_ = g[i] * s;
                    dg[i] = zn * (w[i] * fmaf(act_, 1.f - s, s));
                }
                dw[i] = fmaf(zn, act_, dw[i]);
                z[i] *= w[i] * act_;
                x[i] = n;
                dot = fmaf(z[i], n, dot);
            }
            dot = row_sum<LPR>(dot) * inv;
#pragma unroll
            for (int i = 0; i < kPer; ++i) x[i] = r * fmaf(-x[i], dot, z[i]);
            if (act) {
                store<VEC, LPR>(dout, l, p.dv, x);
                if (GATE) store<VEC, LPR>(dgate, l, p.dv, dg);
            }
            dout += kGroups * p.dout.st;
            if (GATE) dgate += kGroups * p.dgate.st;
        }
    }
    if (BACK && p.part) {
        __shared__ float sum[kThreads * kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) sum[group * LPR * kPer + column<VEC, LPR>(l, i)] = dw[i];
        __syncthreads();
        float *out = p.part + (((size_t)h * gridDim.z + b) * gridDim.x + blockIdx.x) * p.dv;
        for (int c = threadIdx.x; c < p.dv; c += kThreads) {
            float x = 0.f;
            for (int q = 0; q < kGroups; ++q) x += sum[q * LPR * kPer + c];
            out[c] = x;
        }
    }
}

// dw[block y][c] = the sum of n consecutive partial rows: grid (columns / 32, sets), 32 columns x 32 parts of the
// rows per block
__global__ void __launch_bounds__(1024) weight_sum_kernel(const float *part, float *dw, int n, int dv)
{
    __shared__ float sum[32][33];
    const int c = blockIdx.x * 32 + threadIdx.x;
    const float *in = part + (size_t)blockIdx.y * n * dv;
    float x = 0.f;
    if (c < dv)
        for (int i = threadIdx.y; i < n; i += 32) x += in[(size_t)i * dv + c];
    sum[threadIdx.y][threadIdx.x] = x;
    __syncthreads();
    x = sum[threadIdx.x][threadIdx.y];
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (threadIdx.x == 0 && blockIdx.x * 32 + threadIdx.y < dv) dw[(size_t)blockIdx.y * dv + blockIdx.x * 32 + threadIdx.y] = x;
}

bool rows_aligned(const View &v, int esize)
{
    const long long per = 16 / esize;
    return !v.p || ((reinterpret_cast<uintptr_t>(v.p) & 15u) == 0 && v.sb % per == 0 && v.sh % per == 0 && v.st % per == 0);
}

template <typename T, bool VEC, int LPR>
cudaError_t run(const GatedNormArgs &a, const NormParams &p, dim3 grid, cudaStream_t stream)
{
    if (a.back) {
        if (a.gate.p) gated_norm_kernel<T, VEC, LPR, true, true><<<grid, kThreads, 0, stream>>>(p);
        else gated_norm_kernel<T, VEC, LPR, false, true><<<grid, kThreads, 0, stream>>>(p);
    } else {
        if (a.gate.p) gated_norm_kernel<T, VEC, LPR, true, false><<<grid, kThreads, 0, stream>>>(p);
        else gated_norm_kernel<T, VEC, LPR, false, false><<<grid, kThreads, 0, stream>>>(p);
    }
    const cudaError_t err = cudaGetLastError();
    if (err == cudaSuccess) count_launches(1);
    return err;
}

template <typename T>
cudaError_t run_typed(const GatedNormArgs &a, const NormParams &p, bool vec, int lanes, dim3 grid, cudaStream_t stream)
{
    if (!vec) return run<T, false, 32>(a, p, grid, stream);
    switch (lanes) {
        case 4: return run<T, true, 4>(a, p, grid, stream);
        case 8: return run<T, true, 8>(a, p, grid, stream);
        case 16: return run<T, true, 16>(a, p, grid, stream);
        default: return run<T, true, 32>(a, p, grid, stream);
    }
}

}  // namespace

cudaError_t launch_gated_norm(const GatedNormArgs &a, cudaStream_t stream)
{
    const int esize = a.fp32 ? 4 : 2;
    bool vec = a.dv % kPer == 0;
    for (const View *v : {&a.o, &a.gate, &a.y, &a.dy, &a.dout, &a.dgate}) vec = vec && rows_aligned(*v, esize);
    int lanes = vec ? 4 : 32;
    while (lanes * kPer < a.dv) lanes *= 2;
    int dev = 0, sms = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (err != cudaSuccess) return err;
    // tokens per block: whole rounds of the block's groups, as many as leave every SM eight blocks; the backward
    // pass, whose blocks each end in a sum over their threads, takes up to 64 rounds, the forward pass up to 8
    const int groups = kThreads / lanes;
    const long long rows = (long long)a.B * a.H * a.T, want = rows / ((long long)sms * 8 * groups);
    const int rounds = (int)std::max<long long>(1, std::min<long long>(want, a.back ? 64 : 8));
    NormParams p;
    p.o = a.o; p.gate = a.gate; p.y = a.y; p.dy = a.dy; p.dout = a.dout; p.dgate = a.dgate;
    p.weight = a.weight;
    p.w_head = a.per_head ? a.dv : 0;
    p.part = nullptr;
    p.T = a.T; p.dv = a.dv; p.per_block = rounds * groups; p.eps = a.eps;
    const int tiles = (int)(((long long)a.T + p.per_block - 1) / p.per_block);
    const dim3 grid(tiles, a.H, a.B);
    if (a.back && a.dweight) {
        err = ws_alloc(reinterpret_cast<void **>(&p.part), (size_t)a.H * a.B * tiles * a.dv * sizeof(float), stream);
        if (err != cudaSuccess) return err;
    }
    err = a.fp32 ? run_typed<float>(a, p, vec, lanes, grid, stream) : run_typed<__nv_bfloat16>(a, p, vec, lanes, grid, stream);
    if (p.part) {
        if (err == cudaSuccess) {
            const int sets = a.per_head ? a.H : 1, n = a.B * tiles * (a.per_head ? 1 : a.H);
            weight_sum_kernel<<<dim3((a.dv + 31) / 32, sets), dim3(32, 32), 0, stream>>>(p.part, a.dweight, n, a.dv);
            err = cudaGetLastError();
            if (err == cudaSuccess) count_launches(1);
        }
        const cudaError_t e2 = ws_free(p.part, stream);
        if (err == cudaSuccess) err = e2;
    }
    return err;
}

}  // namespace gdn
