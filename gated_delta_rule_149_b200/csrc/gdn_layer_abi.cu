// C ABI of the operators around the recurrence: argument checks of gdn_rotary and gdn_gated_norm and of their
// gradients.  Every argument error is caught before anything is launched; no C++ exception crosses.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/gdn.h"
#include "gdn_internal.h"

using gdn::fail;
using gdn::ok;

namespace {

gdn::View to_view(const gdn_view *v)
{
    return v ? gdn::View{v->data, v->stride_b, v->stride_h, v->stride_t} : gdn::View{};
}

// One strided tensor: data there, on an element boundary, strides that stay in the 64-bit range; an output's
// steps must also be at least one row.
int check_view(const gdn_view *v, const char *name, int B, int H, int T, int d, int esize, bool output)
{
    if (!v || !v->data) return fail(GDN_ERR_INVALID_ARG, "%s must be non-NULL", name);
    if (reinterpret_cast<uintptr_t>(v->data) % esize)
        return fail(GDN_ERR_MISALIGNED, "%s is not aligned to its element size", name);
    const long long st[] = {v->stride_b, v->stride_h, v->stride_t};
    const int n[] = {B, H, T};
    for (int i = 0; i < 3; ++i) {
        if (n[i] == 1) continue;
        if (st[i] < (output ? d : 0) || st[i] > (1ll << 60) / n[i])
            return fail(GDN_ERR_INVALID_ARG, "%s: stride %lld of dimension %d is out of range", name, st[i], i);
    }
    return GDN_OK;
}

int check_sizes(int B, int H, int T, int d, int least, int step, const char *d_name)
{
    if (B <= 0 || H <= 0 || T <= 0)
        return fail(GDN_ERR_INVALID_ARG, "B, H and T must be positive (got %d, %d, %d)", B, H, T);
    if (T > INT_MAX - 64) return fail(GDN_ERR_UNSUPPORTED, "T = %d is too long", T);
    if ((long long)B * H > 65535) return fail(GDN_ERR_UNSUPPORTED, "B*H = %lld exceeds 65535", (long long)B * H);
    if (d < least || d % step || d > 256)
        return fail(GDN_ERR_UNSUPPORTED, "%s must be a multiple of %d in [%d, 256] (got %d)", d_name, step, least, d);
    return GDN_OK;
}

int launched(cudaError_t err)
{
    if (err == cudaSuccess) return ok();
    (void)cudaGetLastError();   // reported here alone
    return fail(GDN_ERR_CUDA, "launch failed: %s", cudaGetErrorString(err));
}

int rotary(bool back, const gdn_view *dq, const gdn_view *dk, const gdn_view *q, const gdn_view *k, const gdn_view *yq,
           const gdn_view *yk, const int *positions, long long pos_stride_b, int B, int H, int T, int d, int axis_t,
           int axis_h, int axis_w, int grid_h, int grid_w, long long start, double theta, float eps, int mode,
           void *stream)
{
    int rc = check_sizes(B, H, T, d, 2, 2, "d");
    if (rc != GDN_OK) return rc;
    if (mode & ~(GDN_FP32 | GDN_ROTARY_HALF | GDN_ROTARY_L2))
        return fail(GDN_ERR_INVALID_ARG, "unknown mode bits 0x%x", mode);
    const int esize = (mode & GDN_FP32) ? 4 : 2;
    const bool l2 = (mode & GDN_ROTARY_L2) != 0;
    const int axes[] = {axis_t, axis_h, axis_w};
    long long sum = 0;
    for (int n : axes) {
        if (n < 0 || n % 2) return fail(GDN_ERR_INVALID_ARG, "axis dims must be even and >= 0 (got %d)", n);
        sum += n;
    }
    if (sum != d) return fail(GDN_ERR_INVALID_ARG, "axis dims sum to %lld, not d = %d", sum, d);
    if (!(theta > 0) || !std::isfinite(theta)) return fail(GDN_ERR_INVALID_ARG, "theta must be positive and finite");
    if (l2 && (!(eps > 0) || !std::isfinite(eps))) return fail(GDN_ERR_INVALID_ARG, "eps must be positive and finite");
    if (positions) {
        if (reinterpret_cast<uintptr_t>(positions) % 4) return fail(GDN_ERR_MISALIGNED, "positions is not 4-byte aligned");
        if (pos_stride_b < 0 || pos_stride_b > (1ll << 60) / B)
            return fail(GDN_ERR_INVALID_ARG, "pos_stride_b = %lld is out of range", pos_stride_b);
    } else if (grid_h <= 0 || grid_w <= 0 || start < 0 || start > (1ll << 52)) {
        return fail(GDN_ERR_INVALID_ARG, "without positions, grid_h and grid_w must be positive and start in [0, 2^52] "
                    "(got %d, %d, %lld)", grid_h, grid_w, start);
    } else if ((start + T - 1) / ((long long)grid_h * grid_w) > INT_MAX) {
        return fail(GDN_ERR_INVALID_ARG, "the last token's frame, token %lld of frames of %d x %d, is beyond 2^31",
                    start + T - 1, grid_h, grid_w);
    }
    const bool two = k || dk || yk;
    gdn::RotaryArgs a = {};
    a.n = two ? 2 : 1;
    const gdn_view *x[] = {q, k}, *g[] = {dq, dk}, *y[] = {yq, yk};
    for (int i = 0; i < a.n; ++i) {
        if (back && (rc = check_view(g[i], i ? "dk" : "dq", B, H, T, d, esize, false)) != GDN_OK) return rc;
        if (!back || l2) {
            if ((rc = check_view(x[i], i ? "k" : "q", B, H, T, d, esize, false)) != GDN_OK) return rc;
            a.x[i] = to_view(x[i]);
        }
        if ((rc = check_view(y[i], i ? "k's output" : "q's output", B, H, T, d, esize, true)) != GDN_OK) return rc;
        a.g[i] = to_view(g[i]);
        a.y[i] = to_view(y[i]);
    }
    a.positions = positions; a.pos_sb = pos_stride_b;
    a.B = B; a.H = H; a.T = T; a.d = d;
    for (int i = 0; i < 3; ++i) a.axes[i] = axes[i];
    a.grid_h = grid_h; a.grid_w = grid_w; a.start = start; a.theta = theta; a.eps = eps;
    a.half = (mode & GDN_ROTARY_HALF) != 0;
    a.l2 = l2;
    a.back = back;
    a.fp32 = esize == 4;
    return launched(gdn::launch_rotary(a, static_cast<cudaStream_t>(stream)));
}

int gated_norm(bool back, const gdn_view *dy, const gdn_view *o, const gdn_view *gate, const float *weight, int per_head,
               const gdn_view *y, const gdn_view *dout, const gdn_view *dgate, float *dweight, int B, int H, int T,
               int dv, float eps, int mode, void *stream)
{
    int rc = check_sizes(B, H, T, dv, 1, 1, "dv");
    if (rc != GDN_OK) return rc;
    if (mode & ~GDN_FP32) return fail(GDN_ERR_INVALID_ARG, "unknown mode bits 0x%x", mode);
    const int esize = (mode & GDN_FP32) ? 4 : 2;
    if (!(eps > 0) || !std::isfinite(eps)) return fail(GDN_ERR_INVALID_ARG, "eps must be positive and finite");
    if (reinterpret_cast<uintptr_t>(weight) % 4 || reinterpret_cast<uintptr_t>(dweight) % 4)
        return fail(GDN_ERR_MISALIGNED, "weight is not aligned to its element size");
    if (dweight && !weight) return fail(GDN_ERR_INVALID_ARG, "dweight without weight");
    if ((rc = check_view(o, "o", B, H, T, dv, esize, false)) != GDN_OK) return rc;
    if (gate && (rc = check_view(gate, "gate", B, H, T, dv, esize, false)) != GDN_OK) return rc;
    if (back) {
        if ((rc = check_view(dy, "dy", B, H, T, dv, esize, false)) != GDN_OK) return rc;
        if ((rc = check_view(dout, "dout", B, H, T, dv, esize, true)) != GDN_OK) return rc;
        if ((gate != nullptr) != (dgate != nullptr))
            return fail(GDN_ERR_INVALID_ARG, "dgate must be given exactly when gate is");
        if (dgate && (rc = check_view(dgate, "dgate", B, H, T, dv, esize, true)) != GDN_OK) return rc;
    } else if ((rc = check_view(y, "y", B, H, T, dv, esize, true)) != GDN_OK) {
        return rc;
    }
    gdn::GatedNormArgs a = {};
    a.o = to_view(o); a.gate = to_view(gate); a.y = to_view(y); a.dy = to_view(dy);
    a.dout = to_view(dout); a.dgate = to_view(dgate);
    a.weight = weight; a.dweight = dweight; a.per_head = per_head != 0;
    a.B = B; a.H = H; a.T = T; a.dv = dv; a.eps = eps;
    a.back = back;
    a.fp32 = esize == 4;
    return launched(gdn::launch_gated_norm(a, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int gdn_rotary(const gdn_view *q, const gdn_view *k, const gdn_view *q_out, const gdn_view *k_out, const int *positions,
               long long pos_stride_b, int B, int H, int T, int d, int axis_t, int axis_h, int axis_w, int grid_h,
               int grid_w, long long start, double theta, float eps, int mode, void *stream)
{
    try {
        return rotary(false, nullptr, nullptr, q, k, q_out, k_out, positions, pos_stride_b, B, H, T, d, axis_t, axis_h,
                      axis_w, grid_h, grid_w, start, theta, eps, mode, stream);
    } catch (...) {
        return fail(GDN_ERR_CUDA, "internal error in gdn_rotary");
    }
}

int gdn_rotary_backward(const gdn_view *dq, const gdn_view *dk, const gdn_view *q, const gdn_view *k,
                        const gdn_view *q_grad, const gdn_view *k_grad, const int *positions, long long pos_stride_b,
                        int B, int H, int T, int d, int axis_t, int axis_h, int axis_w, int grid_h, int grid_w,
                        long long start, double theta, float eps, int mode, void *stream)
{
    try {
        return rotary(true, dq, dk, q, k, q_grad, k_grad, positions, pos_stride_b, B, H, T, d, axis_t, axis_h, axis_w,
                      grid_h, grid_w, start, theta, eps, mode, stream);
    } catch (...) {
        return fail(GDN_ERR_CUDA, "internal error in gdn_rotary_backward");
    }
}

int gdn_gated_norm(const gdn_view *o, const gdn_view *gate, const float *weight, int per_head, const gdn_view *y, int B,
                   int H, int T, int dv, float eps, int mode, void *stream)
{
    try {
        return gated_norm(false, nullptr, o, gate, weight, per_head, y, nullptr, nullptr, nullptr, B, H, T, dv, eps, mode,
                          stream);
    } catch (...) {
        return fail(GDN_ERR_CUDA, "internal error in gdn_gated_norm");
    }
}

int gdn_gated_norm_backward(const gdn_view *dy, const gdn_view *o, const gdn_view *gate, const float *weight,
                            int per_head, const gdn_view *dout, const gdn_view *dgate, float *dweight, int B, int H,
                            int T, int dv, float eps, int mode, void *stream)
{
    try {
        return gated_norm(true, dy, o, gate, weight, per_head, nullptr, dout, dgate, dweight, B, H, T, dv, eps, mode,
                          stream);
    } catch (...) {
        return fail(GDN_ERR_CUDA, "internal error in gdn_gated_norm_backward");
    }
}

}  // extern "C"
