// RMS norms before and after a block, fused with the block's gate, the residual scale and the residual sum, and their
// gradient.
//
//   n  = y * r_y * w_post,  r_y = 1 / sqrt(mean(y^2) + eps)     (n = y without w_post)
//   x' = x + alpha * gate * n                                   (x' = x without y; gate 1 without gate)
//   h  = x' * r_x * w,      r_x = 1 / sqrt(mean(x'^2) + eps)
//
//   d_x  = d_x' + r_x * (w d_h - x' r_x^2 mean(w d_h x')),      d_w = sum_t d_h x' r_x
//   d_n  = alpha * gate * d_x,                                  d_gate = alpha * n * d_x (summed over t for [H])
//   d_y  = r_y * (w_post d_n - y r_y^2 mean(w_post d_n y)),     d_w_post = sum_t d_n y r_y
//
// Bound by HBM: one pass over every tensor.  A row stays in the registers of one CTA between its sums, which are kept
// in fp32, as are x' before h and everything else until its one rounding.
#pragma once
#include "rowwise.cuh"

namespace dg {

constexpr int NORM_MAX_H = 16384;
constexpr int NORM_MAX_THREADS = 512;
enum GateKind { GATE_NONE = 0, GATE_ROW = 1, GATE_TOKEN = 2 };

struct NormParams {
    const void *x, *y;                 // forward: x; gradient: x' as stored
    const void *w, *w_post, *gate;     // w, w_post and a gate [H]: param_f32 ? float : bf16; a gate [T][H]: type of y
    void *x_out, *h;
    ScaleLayout sf;                    // h in e4m3 if sf.sf
    float *rstd, *rstd_post;           // [T]; forward: may be null
    const void *d_x_out, *d_h;         // gradient; d_x_out may be null (0)
    void *d_x, *d_y, *d_gate_token;
    float *partial;                    // gradient: [CTAs][3][H]: d_w, d_w_post, d_gate [H]
    float alpha, eps;
    int T, H, param_f32, gate_kind;
};

__device__ __forceinline__ void load_param8(const void *p, int f32, int i, float (&v)[VEC]) {
    if (f32) load8(static_cast<const float *>(p) + i, v);
    else load8(static_cast<const bf16 *>(p) + i, v);
}

// Sum over the CTA, the same in every thread.  `part` is read until the next barrier: two buffers in turn.
__device__ __forceinline__ float cta_sum(float v, float *part) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < warps ? part[lane] : 0.f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

template <typename X, typename Y, int ITERS>
__global__ void __launch_bounds__(NORM_MAX_THREADS) rms_norm_kernel(const NormParams p) {
    __shared__ float part[2][32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int row = blockIdx.x;
    const long long at = static_cast<long long>(row) * p.H;
    float x[ITERS][VEC];
#pragma unroll
    for (int j = 0; j < ITERS; ++j) {
        const int col = (j * blockDim.x + threadIdx.x) * VEC;
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[j][i] = 0.f;
        if (col < p.H) load8(static_cast<const X *>(p.x) + at + col, x[j]);
    }
    if (p.y) {
        float n[ITERS][VEC];
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < ITERS; ++j) {
            const int col = (j * blockDim.x + threadIdx.x) * VEC;
#pragma unroll
            for (int i = 0; i < VEC; ++i) n[j][i] = 0.f;
            if (col < p.H) load8(static_cast<const Y *>(p.y) + at + col, n[j]);
#pragma unroll
            for (int i = 0; i < VEC; ++i) sum = fmaf(n[j][i], n[j][i], sum);
        }
        float r = 1.f;
        if (p.w_post) {
            r = rsqrtf(cta_sum(sum, part[0]) / p.H + p.eps);
            if (threadIdx.x == 0 && p.rstd_post) p.rstd_post[row] = r;
        }
#pragma unroll
        for (int j = 0; j < ITERS; ++j) {
            const int col = (j * blockDim.x + threadIdx.x) * VEC;
            if (col >= p.H) continue;
            float c[VEC];
            if (p.w_post) {
                load_param8(p.w_post, p.param_f32, col, c);
#pragma unroll
                for (int i = 0; i < VEC; ++i) n[j][i] *= r * c[i];
            }
            if (p.gate_kind != GATE_NONE) {
                if (p.gate_kind == GATE_ROW) load_param8(p.gate, p.param_f32, col, c);
                else load8(static_cast<const Y *>(p.gate) + at + col, c);
#pragma unroll
                for (int i = 0; i < VEC; ++i) n[j][i] *= c[i];
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) x[j][i] = fmaf(p.alpha, n[j][i], x[j][i]);
            store8(static_cast<X *>(p.x_out) + at + col, x[j]);
        }
    }
    if (!p.w) return;
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < ITERS; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) sum = fmaf(x[j][i], x[j][i], sum);
    const float r = rsqrtf(cta_sum(sum, part[1]) / p.H + p.eps);
    if (threadIdx.x == 0 && p.rstd) p.rstd[row] = r;
#pragma unroll
    for (int j = 0; j < ITERS; ++j) {
        const int col = (j * blockDim.x + threadIdx.x) * VEC;
        const bool in = col < p.H;  // (the same in a block's 16 lanes where h is e4m3)
        float c[VEC] = {};
        if (in) load_param8(p.w, p.param_f32, col, c);
#pragma unroll
        for (int i = 0; i < VEC; ++i) c[i] *= x[j][i] * r;
        if (p.sf.sf) {
            float scale;
            const uint2 q = quantise8(c, block_amax(c), scale);
            if (in) {
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.h) + at + col) = q;
                if ((threadIdx.x & 15) == 0) *p.sf.at(row, col >> 7) = scale;
            }
        } else if (in) {
            store8(static_cast<Y *>(p.h) + at + col, c);
        }
    }
}

// CTA b takes rows b, b + CTAs, ...: the parameters' sums over its rows stay in registers and go to `partial` once.
template <typename X, typename Y, int ITERS>
__global__ void __launch_bounds__(NORM_MAX_THREADS) rms_norm_backward_kernel(const NormParams p) {
    __shared__ float part[2][32];
    grid_dependency_wait();
    grid_launch_dependents();
    float sum_w[ITERS][VEC] = {}, sum_post[ITERS][VEC] = {}, sum_gate[ITERS][VEC] = {};
    for (int row = blockIdx.x; row < p.T; row += gridDim.x) {
        const long long at = static_cast<long long>(row) * p.H;
        float dx[ITERS][VEC];
#pragma unroll
        for (int j = 0; j < ITERS; ++j) {
            const int col = (j * blockDim.x + threadIdx.x) * VEC;
#pragma unroll
            for (int i = 0; i < VEC; ++i) dx[j][i] = 0.f;
            if (p.d_x_out && col < p.H) load8(static_cast<const X *>(p.d_x_out) + at + col, dx[j]);
        }
        if (p.w) {
            const float r = *(p.rstd + row);
            float x[ITERS][VEC], e[ITERS][VEC], sum = 0.f;
#pragma unroll
            for (int j = 0; j < ITERS; ++j) {
                const int col = (j * blockDim.x + threadIdx.x) * VEC;
                float c[VEC] = {};
#pragma unroll
                for (int i = 0; i < VEC; ++i) x[j][i] = e[j][i] = 0.f;
                if (col < p.H) {
                    load8(static_cast<const X *>(p.x) + at + col, x[j]);
                    load8(static_cast<const Y *>(p.d_h) + at + col, e[j]);
                    load_param8(p.w, p.param_f32, col, c);
                }
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    x[j][i] *= r;
                    sum_w[j][i] = fmaf(e[j][i], x[j][i], sum_w[j][i]);
                    e[j][i] *= c[i];
                    sum = fmaf(e[j][i], x[j][i], sum);
                }
            }
            const float mean = cta_sum(sum, part[0]) / p.H;
#pragma unroll
            for (int j = 0; j < ITERS; ++j)
#pragma unroll
                for (int i = 0; i < VEC; ++i) dx[j][i] = fmaf(r, e[j][i] - x[j][i] * mean, dx[j][i]);
        }
#pragma unroll
        for (int j = 0; j < ITERS; ++j) {
            const int col = (j * blockDim.x + threadIdx.x) * VEC;
            if (col < p.H) store8(static_cast<X *>(p.d_x) + at + col, dx[j]);
        }
        if (!p.y) {
            __syncthreads();  // part[0] is written again in the next row
            continue;
        }
        const float r = p.w_post ? *(p.rstd_post + row) : 1.f;
        float y[ITERS][VEC], sum = 0.f;
#pragma unroll
        for (int j = 0; j < ITERS; ++j) {
            const int col = (j * blockDim.x + threadIdx.x) * VEC;
            float post[VEC], gate[VEC], d_gate[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) y[j][i] = 0.f, post[i] = gate[i] = 1.f;
            if (col < p.H) {
                load8(static_cast<const Y *>(p.y) + at + col, y[j]);
                if (p.w_post) load_param8(p.w_post, p.param_f32, col, post);
                if (p.gate_kind == GATE_ROW) load_param8(p.gate, p.param_f32, col, gate);
                if (p.gate_kind == GATE_TOKEN) load8(static_cast<const Y *>(p.gate) + at + col, gate);
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                y[j][i] *= r;
                const float d = p.alpha * dx[j][i];
                d_gate[i] = d * y[j][i] * post[i];
                sum_gate[j][i] += d_gate[i];
                const float dn = d * gate[i];
                sum_post[j][i] = fmaf(dn, y[j][i], sum_post[j][i]);
                dx[j][i] = dn * post[i];
                sum = fmaf(dx[j][i], y[j][i], sum);
            }
            if (p.gate_kind == GATE_TOKEN && col < p.H) store8(static_cast<Y *>(p.d_gate_token) + at + col, d_gate);
        }
        float mean = 0.f;
        if (p.w_post) mean = cta_sum(sum, part[1]) / p.H;
#pragma unroll
        for (int j = 0; j < ITERS; ++j) {
            const int col = (j * blockDim.x + threadIdx.x) * VEC;
            if (col >= p.H) continue;
#pragma unroll
            for (int i = 0; i < VEC; ++i) dx[j][i] = r * (dx[j][i] - y[j][i] * mean);
            store8(static_cast<Y *>(p.d_y) + at + col, dx[j]);
        }
        __syncthreads();
    }
    float *partial = p.partial + static_cast<long long>(blockIdx.x) * 3 * p.H;
#pragma unroll
    for (int j = 0; j < ITERS; ++j) {
        const int col = (j * blockDim.x + threadIdx.x) * VEC;
        if (col >= p.H) continue;
        if (p.w) store8(partial + col, sum_w[j]);
        if (p.w_post) store8(partial + p.H + col, sum_post[j]);
        if (p.gate_kind == GATE_ROW) store8(partial + 2 * p.H + col, sum_gate[j]);
    }
}

constexpr int NORM_SUM_COLS = 64, NORM_SUM_PARTS = 16;

// d[z][col] = sum over the CTAs' partial sums, in an order that does not change.  blockIdx.y: which of the three.
__global__ void __launch_bounds__(NORM_SUM_COLS *NORM_SUM_PARTS)
    rms_norm_sum_kernel(const float *partial, int ctas, int H, float *d0, float *d1, float *d2) {
    __shared__ float part[NORM_SUM_PARTS][NORM_SUM_COLS];
    grid_dependency_wait();
    grid_launch_dependents();
    float *d = blockIdx.y == 0 ? d0 : blockIdx.y == 1 ? d1 : d2;
    if (!d) return;
    const int col = blockIdx.x * NORM_SUM_COLS + threadIdx.x;
    float sum = 0.f;
    if (col < H)
        for (int b = threadIdx.y; b < ctas; b += NORM_SUM_PARTS)
            sum += partial[(static_cast<long long>(b) * 3 + blockIdx.y) * H + col];
    part[threadIdx.y][threadIdx.x] = sum;
    __syncthreads();
    if (threadIdx.y == 0 && col < H) {
        sum = 0.f;
        for (int i = 0; i < NORM_SUM_PARTS; ++i) sum += part[i][threadIdx.x];
        d[col] = sum;
    }
}

}  // namespace dg
