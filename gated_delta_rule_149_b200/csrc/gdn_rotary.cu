// Rotary positions with up to three axes (time, height, width) on q and k, with an optional L2 normalisation of
// each row before the rotation, and the gradients of both.
//
// Pair p of a head's d/2 pairs belongs to one axis, as the i-th of its d_axis/2 pairs, and turns by
//     angle = position on that axis * theta^(-2 i / d_axis).
// Interleaved form: pair p is elements (2p, 2p+1); half form: (p, p + d/2).
//     y = Rot(angle) x r,   r = 1 / sqrt(|x|^2 + eps)   (r = 1 without the normalisation)
// Gradient, with z = Rot(angle)^T g:   dx = r (z - x r^2 (x . z)).
// Positions come from the token's place in a frames x height x width grid, or from an int32 tensor.
//
// One pass over the data, which bounds it: q and k are read in whatever strides the projection left them and
// written in whatever strides the next operator takes.  The angles are formed in 64 bits as turns
// (position * frequency / 2 pi), whose fraction alone goes to the 32-bit sine and cosine.  The turns are within 2^-50 of
// themselves (the frequency and four roundings): nothing beside fp32 up to 2^24 radians, 2^-19 at 2^31, where positions end
// (int32 ones, and by the check of the arguments those of a grid).  A block takes a tile of tokens, forms their sines and
// cosines once in shared memory, and all heads of q and k use them; a thread keeps those of its eight pairs in
// registers over its heads.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;
constexpr int kPer = 8;            // pairs per thread
constexpr int kMaxTokens = 16;     // tokens per block

struct RotParams {
    View x[2], g[2], y[2];
    const int *positions;
    long long pos_sb;
    double slope[3], slope_lo[3];  // log2 of the i-th frequency of an axis is i (slope + slope_lo)
    int end_t, end_h;              // pairs below end_t: time; below end_h: height; the others: width
    int H, T, d, rows;             // rows: heads of q and k together
    int tokens;                    // tokens per block
    int grid_h, grid_w;
    long long start;
    float eps;
};

// eight pairs of a row as two runs of eight elements: interleaved, elements [16 l, 16 l + 16) of it; half form,
// [8 l, 8 l + 8) and the same d/2 further
template <typename T> struct Run8;
template <> struct Run8<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { u = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void get(float *f) const
    {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float *f)
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&v);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <> struct Run8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = reinterpret_cast<const float4 *>(p)[0];
        b = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ void get(float *f) const
    {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    static __device__ __forceinline__ void store(float *p, const float *f)
    {
        reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// A thread's part of one row: a[i], b[i] are the two elements of its i-th pair.  VEC: pairs 8 l .. 8 l + 7 by
// 16-byte accesses; otherwise pairs l, l + LPR, ... element by element, so that neighbouring lanes still touch
// neighbouring elements.  (2 x 16 x 12000 rows of 96 bf16 values: 48 us, off 16-byte boundaries 75)
template <typename T, bool HALF, bool VEC, int LPR>
struct Row {
    float a[kPer], b[kPer];
    static __device__ __forceinline__ int pair(int l, int i) { return VEC ? kPer * l + i : l + LPR * i; }
    __device__ __forceinline__ void load(const T *p, int l, int d)
    {
        if (VEC) {
            float f[16];
            Run8<T> u, v;
            if (HALF) {
                u.load(p + 8 * l);
                v.load(p + d / 2 + 8 * l);
            } else {
                u.load(p + 16 * l);
                v.load(p + 16 * l + 8);
            }
            u.get(f);
            v.get(f + 8);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                a[i] = HALF ? f[i] : f[2 * i];
                b[i] = HALF ? f[8 + i] : f[2 * i + 1];
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int q = pair(l, i);
                const bool on = q < d / 2;
                a[i] = on ? to_f(p[HALF ? q : 2 * q]) : 0.f;
                b[i] = on ? to_f(p[HALF ? q + d / 2 : 2 * q + 1]) : 0.f;
            }
        }
    }
    __device__ __forceinline__ void store(T *p, int l, int d) const
    {
        if (VEC) {
            float f[16];
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                f[HALF ? i : 2 * i] = a[i];
                f[HALF ? 8 + i : 2 * i + 1] = b[i];
            }
            Run8<T>::store(HALF ? p + 8 * l : p + 16 * l, f);
            Run8<T>::store(HALF ? p + d / 2 + 8 * l : p + 16 * l + 8, f + 8);
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int q = pair(l, i);
                if (q >= d / 2) continue;
                put(p + (HALF ? q : 2 * q), a[i]);
                put(p + (HALF ? q + d / 2 : 2 * q + 1), b[i]);
            }
        }
    }
};

template <int LPR>
__device__ __forceinline__ float row_sum(float x)
{
#pragma unroll
    for (int o = LPR / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Grid (token tiles, head splits, batches).  LPR lanes hold a row; a block's threads are LPR x tokens x the rest,
// which walks the rows (heads of q, then of k).
template <typename T, bool HALF, bool VEC, int LPR, bool L2, bool BACK>
__global__ void __launch_bounds__(kThreads, 4) rotary_kernel(const __grid_constant__ RotParams p)
{
    extern __shared__ float2 cs[];                    // [tokens][d/2]: cosine, sine
    __shared__ double at[kMaxTokens][3], freq[kMaxPairs];
    const int pairs = p.d / 2, t0 = blockIdx.x * p.tokens, b = blockIdx.z;
    // the frequencies, in turns per position (formed here: as a table in the kernel's arguments they cost every block a
    // string of constant-cache misses), and the tokens' positions
    if (threadIdx.x < pairs) {
        const int q = threadIdx.x, axis = q < p.end_t ? 0 : q < p.end_h ? 1 : 2;
        const double i = q - (axis == 0 ? 0 : axis == 1 ? p.end_t : p.end_h);
        freq[q] = exp2(i * p.slope[axis]) * fma(i * p.slope_lo[axis], 0.693147180559945309, 1.0) * 0.159154943091895336;
    } else if (threadIdx.x >= kMaxPairs && threadIdx.x - kMaxPairs < p.tokens && t0 + (int)threadIdx.x - kMaxPairs < p.T) {
        const int tl = threadIdx.x - kMaxPairs, t = t0 + tl;
        if (p.positions) {
#pragma unroll
            for (int i = 0; i < 3; ++i) at[tl][i] = (double)p.positions[b * p.pos_sb + (long long)t * 3 + i];
        } else {
            const long long n = p.start + t, row = n / p.grid_w, frame = row / p.grid_h;
            at[tl][0] = (double)frame;
            at[tl][1] = (double)(row - frame * p.grid_h);
            at[tl][2] = (double)(n - row * p.grid_w);
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.tokens * pairs; e += kThreads) {
        const int tl = e / pairs, q = e - tl * pairs;
        if (t0 + tl >= p.T) break;
        const double turns = at[tl][q < p.end_t ? 0 : q < p.end_h ? 1 : 2] * freq[q];
        float s, c;
        sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
        cs[e] = make_float2(c, s);
    }
    __syncthreads();

    const int l = threadIdx.x % LPR, group = threadIdx.x / LPR;
    const int tl = group % p.tokens, t = t0 + tl, first = group / p.tokens + blockIdx.y * (kThreads / LPR / p.tokens);
    const int step = kThreads / LPR / p.tokens * gridDim.y;
    const bool lane_on = VEC ? kPer * l < pairs : l < pairs;
    const bool on = t < p.T && lane_on;
    float c[kPer], s[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int q = Row<T, HALF, VEC, LPR>::pair(l, i);
        const bool in = t < p.T && q < pairs;
        const float2 v = in ? cs[tl * pairs + q] : make_float2(1.f, 0.f);
        c[i] = v.x;
        s[i] = BACK ? -v.y : v.y;
    }
    // every lane takes every step, so that the row sums see whole warps
    const int rounds = (p.rows + step - 1) / step;
#pragma unroll 1
    for (int k = 0; k < rounds; ++k) {
        const int r = first + k * step;
        const bool act = on && r < p.rows;
        const int which = r >= p.H, h = which ? r - p.H : r;
        Row<T, HALF, VEC, LPR> x, z;
#pragma unroll
        for (int i = 0; i < kPer; ++i) x.a[i] = x.b[i] = z.a[i] = z.b[i] = 0.f;
        if (act) {
            const View &vx = p.x[which], &vg = p.g[which];
            if (!BACK || L2) x.load(static_cast<const T *>(vx.p) + b * vx.sb + h * vx.sh + t * vx.st, l, p.d);
            if (BACK) z.load(static_cast<const T *>(vg.p) + b * vg.sb + h * vg.sh + t * vg.st, l, p.d);
        }
        float rn = 1.f;
        if (L2) {
            float sq = 0.f;
#pragma unroll
            for (int i = 0; i < kPer; ++i) sq = fmaf(x.a[i], x.a[i], fmaf(x.b[i], x.b[i], sq));
            rn = rsqrtf(row_sum<LPR>(sq) + p.eps);
        }
        Row<T, HALF, VEC, LPR> y;
        const Row<T, HALF, VEC, LPR> &in = BACK ? z : x;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const float u = in.a[i], v = in.b[i];
            y.a[i] = u * c[i] - v * s[i];
            y.b[i] = u * s[i] + v * c[i];
        }
        if (L2 && BACK) {
            float dot = 0.f;
#pragma unroll
            for (int i = 0; i < kPer; ++i) dot = fmaf(x.a[i], y.a[i], fmaf(x.b[i], y.b[i], dot));
            dot = row_sum<LPR>(dot) * rn * rn;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                y.a[i] = rn * (y.a[i] - x.a[i] * dot);
                y.b[i] = rn * (y.b[i] - x.b[i] * dot);
            }
        } else if (L2) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                y.a[i] *= rn;
                y.b[i] *= rn;
            }
        }
        if (act) {
            const View &vy = p.y[which];
            y.store(const_cast<T *>(static_cast<const T *>(vy.p)) + b * vy.sb + h * vy.sh + t * vy.st, l, p.d);
        }
    }
}

// whether every row of the view starts on a 16-byte boundary
bool rows_aligned(const View &v, int esize)
{
    const long long per = 16 / esize;
    return !v.p || ((reinterpret_cast<uintptr_t>(v.p) & 15u) == 0 && v.sb % per == 0 && v.sh % per == 0 && v.st % per == 0);
}

template <typename T, bool HALF, bool VEC, int LPR>
cudaError_t run(const RotaryArgs &a, const RotParams &p, dim3 grid, cudaStream_t stream)
{
    const size_t smem = (size_t)p.tokens * (p.d / 2) * sizeof(float2);
    if (a.back) {
        if (a.l2) rotary_kernel<T, HALF, VEC, LPR, true, true><<<grid, kThreads, smem, stream>>>(p);
        else rotary_kernel<T, HALF, VEC, LPR, false, true><<<grid, kThreads, smem, stream>>>(p);
    } else {
        if (a.l2) rotary_kernel<T, HALF, VEC, LPR, true, false><<<grid, kThreads, smem, stream>>>(p);
        else rotary_kernel<T, HALF, VEC, LPR, false, false><<<grid, kThreads, smem, stream>>>(p);
    }
    const cudaError_t err = cudaGetLastError();
    if (err == cudaSuccess) count_launches(1);
    return err;
}

template <typename T, bool HALF, bool VEC>
cudaError_t run_lanes(const RotaryArgs &a, const RotParams &p, int lanes, dim3 grid, cudaStream_t stream)
{
    if constexpr (VEC) {
        if (lanes == 2) return run<T, HALF, VEC, 2>(a, p, grid, stream);
        if (lanes == 4) return run<T, HALF, VEC, 4>(a, p, grid, stream);
        if (lanes == 8) return run<T, HALF, VEC, 8>(a, p, grid, stream);
    }
    return run<T, HALF, VEC, 16>(a, p, grid, stream);
}

template <typename T>
cudaError_t run_typed(const RotaryArgs &a, const RotParams &p, bool vec, int lanes, dim3 grid, cudaStream_t stream)
{
    if (a.half) return vec ? run_lanes<T, true, true>(a, p, lanes, grid, stream) : run_lanes<T, true, false>(a, p, lanes, grid, stream);
    return vec ? run_lanes<T, false, true>(a, p, lanes, grid, stream) : run_lanes<T, false, false>(a, p, lanes, grid, stream);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs &a, cudaStream_t stream)
{
    RotParams p;
    const int esize = a.fp32 ? 4 : 2;
    bool vec = a.d % 16 == 0;
    for (int i = 0; i < 2; ++i) {
        p.x[i] = i < a.n ? a.x[i] : View{};
        p.g[i] = i < a.n ? a.g[i] : View{};
        p.y[i] = i < a.n ? a.y[i] : View{};
        vec = vec && rows_aligned(p.x[i], esize) && rows_aligned(p.g[i], esize) && rows_aligned(p.y[i], esize);
    }
    p.positions = a.positions;
    p.pos_sb = a.pos_sb;
    // theta^(-2 i / n): the slope's first part has 40 bits, so that its multiples are exact
    for (int x = 0; x < 3; ++x) {
        const long double slope = a.axes[x] ? -2.0L * std::log2((long double)a.theta) / a.axes[x] : 0.0L;
        int e = 0;
        const double m = std::frexp((double)slope, &e);
        p.slope[x] = std::ldexp(std::rint(std::ldexp(m, 40)), e - 40);
        p.slope_lo[x] = (double)(slope - p.slope[x]);
    }
    p.end_t = a.axes[0] / 2;
    p.end_h = p.end_t + a.axes[1] / 2;
    p.H = a.H; p.T = a.T; p.d = a.d; p.rows = a.H * a.n;
    p.grid_h = a.grid_h; p.grid_w = a.grid_w; p.start = a.start; p.eps = a.eps;
    int lanes = vec ? 2 : 16;
    while (lanes * 2 * kPer < a.d) lanes *= 2;
    int dev = 0, sms = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (err != cudaSuccess) return err;
    // 16 tokens a block where that leaves every SM eight blocks (720p clip, backward: 611 us; 14 more with 8), else 8 (480p
    // chunk: 20.5 us; 2 more with 16)
    p.tokens = (long long)((a.T + 15) / 16) * a.B >= 8LL * sms ? 16 : 8;
    // a short sequence leaves SMs idle: its heads are split over blocks as well, though each forms the sines again (the
    // 480p chunk, which fills the SMs, takes 20.5 us unsplit, 22.7 in two)
    const long long tiles = (a.T + p.tokens - 1) / p.tokens;
    const int side = kThreads / lanes / p.tokens, most = (p.rows + side - 1) / side;
    int splits = 1;
    while (splits < most && tiles * a.B * splits < 2 * sms) splits *= 2;
    const dim3 grid((unsigned)tiles, splits, a.B);
    return a.fp32 ? run_typed<float>(a, p, vec, lanes, grid, stream)
                  : run_typed<__nv_bfloat16>(a, p, vec, lanes, grid, stream);
}

}  // namespace gdn
