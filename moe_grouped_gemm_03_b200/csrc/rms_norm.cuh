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
// Bound by HBM: one pass over every tensor.  A row belongs to one CTA, a thread to eight of its columns.  Between a row's
// loads and its stores lie one or two sums over the CTA, so a CTA that loads, sums and stores in turn leaves the memory
// idle most of the time.  The CTAs therefore stay (as many as fit on the SMs, each taking every CTAs-th row) and copy
// their next rows to shared memory ahead of use; the parameters lie there too, copied once.  Every thread copies what it
// will read itself, so no barrier goes with the copies.  Rows of more than 8192 columns do not fit and go without.
// Sums are fp32, as are x' before h and everything else until its one rounding.
#pragma once
#include "rowwise.cuh"

namespace dg {

constexpr int NORM_MAX_H = 16384;
constexpr int NORM_MAX_THREADS = 1024;                  // of a CTA whose rows go through shared memory, a vector each
constexpr int NORM_RING_H = NORM_MAX_THREADS * VEC;     // widest row of such a CTA
constexpr int NORM_WIDE_THREADS = 512;                  // of a CTA for wider rows
constexpr int NORM_ROW_WARPS = 8;                       // rows of a forward CTA that takes a row a warp
constexpr int NORM_MAX_STAGES = 4;
constexpr int NORM_SHARED_BYTES = 226 * 1024;           // of an SM, for the CTAs' parameters and stages
constexpr int NORM_CTA_BYTES = 1024 + 256;              // of them a CTA's for the system and its static ones
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
    int stages;                        // rows of a CTA under way in shared memory
};

__device__ __forceinline__ void load_param(const void *p, int f32, int i, float (&v)[VEC]) {
    if (f32) load_vec(static_cast<const float *>(p) + i, v);
    else load_vec(static_cast<const bf16 *>(p) + i, v);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// Sum over the CTA, the same in every thread.  `part` is read until the next barrier: two buffers in turn.
__device__ __forceinline__ float cta_sum(float v, float *part) {
    v = warp_sum(v);
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    if (warps == 1) return v;
    if (lane == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum(lane < warps ? part[lane] : 0.f);
}

// A thread's vectors in shared memory: the parameters (w, w_post, a gate [H]) and the stages of a row's tensors, in planes of
// one 16-byte unit a thread; a bf16 vector is a unit, an fp32 vector two.  A thread copies what it will read itself, but for
// the rows in fp32: copies are 16 bytes a lane, and so that the lanes of a warp copy runs of memory its 64 units are copied
// in memory order, 32 to a plane (in an order that lets eight lanes reading every other unit meet eight banks; each lane
// copying its own two units took 159 us where this takes 110).
struct NormSlots {
    uint4 *mine;
    int stage;  // first unit of the stage in use

    __device__ __forceinline__ uint4 *unit(int n) const { return mine + n * static_cast<int>(blockDim.x); }
    static __device__ __forceinline__ int turned(int unit) { return unit ^ (unit >> 3 & 1); }

    // the vector at `src`, columns col .. col + 7 (of `width`) of a row; `in`: whether they exist
    __device__ __forceinline__ void copy(int n, const bf16 *src, int, int, bool in) const {
        if (in) copy_async16(unit(n), src);
    }
    __device__ __forceinline__ void copy(int n, const float *src, int col, int width, bool) const {
        const int lane = threadIdx.x & 31, c = col - 4 * lane, place = turned(lane) - lane;
        if (c < width) copy_async16(unit(n) + place, src - 4 * lane);
        if (c + 128 < width) copy_async16(unit(n + 1) + place, src - 4 * lane + 128);
    }
    __device__ __forceinline__ void get(int n, const bf16 *, float (&v)[VEC]) const {
        Raw<bf16> raw;
        raw.a = *unit(n);
        raw.get(v);
    }
    __device__ __forceinline__ void get(int n, const float *, float (&v)[VEC]) const {
        const int lane = threadIdx.x & 31, first = 2 * lane & 31;
        const uint4 *s = unit(n + (lane >> 4)) - lane;
        halves(s[turned(first)], s[turned(first + 1)], v);
    }
    template <typename T> __device__ __forceinline__ void get(int n, float (&v)[VEC]) const {
        get(n, static_cast<const T *>(nullptr), v);
    }
    static __device__ __forceinline__ void halves(uint4 a, uint4 b, float (&v)[VEC]) {
        v[0] = __uint_as_float(a.x), v[1] = __uint_as_float(a.y), v[2] = __uint_as_float(a.z), v[3] = __uint_as_float(a.w);
        v[4] = __uint_as_float(b.x), v[5] = __uint_as_float(b.y), v[6] = __uint_as_float(b.z), v[7] = __uint_as_float(b.w);
    }
    // parameter number i; through L1: up to 32 CTAs of an SM start on the same few lines, and all SMs' requests for them meet in
    // a few slices of L2 (8192 x 640 with w in fp32: 16 us, 32 when the copies pass L1 by; 8192 x 1024, all parameters: 27, 42)
    __device__ __forceinline__ void copy_param(int i, const void *src, int f32, int col) const {
        if (f32) {
            copy_async16_ca(unit(2 * i), static_cast<const float *>(src) + col);
            copy_async16_ca(unit(2 * i + 1), static_cast<const float *>(src) + col + 4);
        } else {
            copy_async16_ca(unit(i), static_cast<const bf16 *>(src) + col);
        }
    }
    __device__ __forceinline__ void get_param(int i, int f32, float (&v)[VEC]) const {
        if (f32) halves(*unit(2 * i), *unit(2 * i + 1), v);
        else get<bf16>(i, v);
    }
};

// Waits until the oldest of `stages` groups of copies has come.
__device__ __forceinline__ void wait_stage(int stages) {
    switch (stages) {
        case 1: copy_async_wait<0>(); break;
        case 2: copy_async_wait<1>(); break;
        case 3: copy_async_wait<2>(); break;
        default: copy_async_wait<3>(); break;
    }
}

// Units of a thread: parameters (w, w_post and a gate [H]), and one stage.
__host__ __device__ constexpr int norm_param_units(int param_f32, int gate_kind) {
    return (gate_kind == GATE_ROW ? 3 : 2) * (param_f32 ? 2 : 1);
}
__host__ __device__ constexpr int norm_stage_units(int x, int y, bool has_w, bool has_y, bool gate_token) {
    return x + (has_w ? x + y : 0) + (has_y ? y : 0) + (gate_token ? y : 0);
}

// The parameters' sums over the CTA's rows stay in registers and go to `partial` once.  A call without y has a kernel of its own
// (4603 x 7168 in bf16: 50 us, 58 in the general one).  That there is a y stays a question of the run in the others: where the
// compiler knows it, it orders a row's work so that the same rows with y and a gate [H] take 105 us in place of 88.
template <typename X, typename Y, int GATE, bool HAS_Y>
__global__ void __launch_bounds__(NORM_MAX_THREADS) rms_norm_backward_kernel(const NormParams p) {
    extern __shared__ uint4 norm_smem[];
    __shared__ float part[2][32];
    constexpr int UX = Raw<X>::UNITS, UY = Raw<Y>::UNITS;
    const int col = threadIdx.x * VEC;
    const bool in = col < p.H, has_y = HAS_Y && p.y != nullptr, has_w = p.w != nullptr;
    const float inv_h = 1.f / p.H;
    const int first_stage = norm_param_units(p.param_f32, GATE);
    const int stage_units = norm_stage_units(UX, UY, has_w, has_y, GATE == GATE_TOKEN);
    const int y_unit = UX + (has_w ? UX + UY : 0);  // units of a stage: d_x_out, x', d_h, y, gate
    NormSlots s{norm_smem + threadIdx.x, first_stage};
    grid_dependency_wait();
    grid_launch_dependents();
    auto fill = [&](long long row, int stage) {
        if (row < p.T && (UX > 1 || in)) {  // (in fp32 a lane copies other columns than its own)
            const long long at = row * p.H + col;
            if (has_w) {
                s.copy(stage + UX, static_cast<const X *>(p.x) + at, col, p.H, UX == 1 || in);
                s.copy(stage + 2 * UX, static_cast<const Y *>(p.d_h) + at, col, p.H, UX == 1 || in);
            }
            if (p.d_x_out) s.copy(stage, static_cast<const X *>(p.d_x_out) + at, col, p.H, UX == 1 || in);
            if (has_y) s.copy(stage + y_unit, static_cast<const Y *>(p.y) + at, col, p.H, UX == 1 || in);
            if (GATE == GATE_TOKEN) s.copy(stage + y_unit + UY, static_cast<const Y *>(p.gate) + at, col, p.H, UX == 1 || in);
        }
        copy_async_commit();  // (a group for every stage, empty past the last row: the waits count them)
    };
    if (in) {  // (with the first stage's group)
        if (has_w) s.copy_param(0, p.w, p.param_f32, col);
        if (p.w_post) s.copy_param(1, p.w_post, p.param_f32, col);
        if (GATE == GATE_ROW) s.copy_param(2, p.gate, p.param_f32, col);
    }
    for (int i = 0; i < p.stages; ++i) fill(blockIdx.x + static_cast<long long>(i) * gridDim.x, first_stage + i * stage_units);
    // sum_n: of alpha d_x y r_post, times w_post the gradient of a gate [H] and times that gate the one of w_post; of alpha
    // d_x gate y r_post with a gate [T][H]
    float sum_w[VEC] = {}, sum_n[VEC] = {};
    float r = 0.f, r_post = 1.f;  // of the row to come, loaded a row ahead
    if (has_w) r = p.rstd[blockIdx.x];
    if (p.w_post) r_post = p.rstd_post[blockIdx.x];
    int turn = 0;  // the buffer of the next sum, where there is one a row
    for (int row = blockIdx.x; row < p.T; row += gridDim.x) {
        const long long at = static_cast<long long>(row) * p.H + col;
        const int next = row + static_cast<int>(gridDim.x) < p.T ? row + gridDim.x : row;
        float r_next = 0.f, r_post_next = 1.f;
        if (has_w) r_next = p.rstd[next];
        if (p.w_post) r_post_next = p.rstd_post[next];
        wait_stage(p.stages);
        if (UX > 1) __syncwarp();  // fp32 rows are copied by other lanes
        float dx[VEC] = {}, t[VEC] = {}, c[VEC] = {};
        if (has_w) {
            float sum[2] = {};
            if (in) {
                s.get<X>(s.stage + UX, t);
                s.get<Y>(s.stage + 2 * UX, dx);
                s.get_param(0, p.param_f32, c);
                mul_vec(t, r);
                fma_vec(sum_w, dx, t);
                mul_vec(dx, c);
                dot_vec(sum, dx, t);  // dx: w d_h, t: x' r
            }
            const float mean = cta_sum(sum[0] + sum[1], part[HAS_Y ? 0 : turn]) * inv_h;
            fma_vec(dx, t, -mean);
            if (p.d_x_out) {
                if (in) s.get<X>(s.stage, t);
                fma_vec(t, dx, r);
#pragma unroll
                for (int i = 0; i < VEC; ++i) dx[i] = t[i];
            } else {
                mul_vec(dx, r);
            }
        } else if (in) {
            s.get<X>(s.stage, dx);
        }
        if (in) store_vec(static_cast<X *>(p.d_x) + at, dx);
        if (has_y) {
            float sum[2] = {};
            if (in) {
                s.get<Y>(s.stage + y_unit, t);
                mul_vec(t, r_post);
                mul_vec(dx, p.alpha);
                if (GATE == GATE_TOKEN) {  // d_gate = alpha d_x n, n = t w_post
#pragma unroll
                    for (int i = 0; i < VEC; ++i) c[i] = t[i];
                    mul_vec(c, dx);
                    if (p.w_post) {
                        float post[VEC];
                        s.get_param(1, p.param_f32, post);
                        mul_vec(c, post);
                    }
                    store_vec(static_cast<Y *>(p.d_gate_token) + at, c);
                    s.get<Y>(s.stage + y_unit + UY, c);
                    mul_vec(dx, c);
                }
                fma_vec(sum_n, dx, t);
                if (GATE == GATE_ROW) {
                    s.get_param(2, p.param_f32, c);
                    mul_vec(dx, c);
                }
                if (p.w_post) {
                    s.get_param(1, p.param_f32, c);
                    mul_vec(dx, c);
                    dot_vec(sum, dx, t);
                }
            }
            if (p.w_post) {
                const float mean = cta_sum(sum[0] + sum[1], part[1]) * inv_h;
                fma_vec(dx, t, -mean);
                mul_vec(dx, r_post);
            }
            if (in) store_vec(static_cast<Y *>(p.d_y) + at, dx);
        }
        if (UX > 1) __syncwarp();  // every lane has read the stage
        fill(row + static_cast<long long>(p.stages) * gridDim.x, s.stage);
        s.stage += stage_units;
        if (s.stage == first_stage + p.stages * stage_units) s.stage = first_stage;
        r = r_next;
        r_post = r_post_next;
        if (!HAS_Y) turn ^= 1;
        else if (!(has_w && p.w_post)) __syncthreads();
    }
    if (!in) return;
    float *partial = p.partial + static_cast<long long>(blockIdx.x) * 3 * p.H + col;
    if (has_w) store_vec(partial, sum_w);
    float c[VEC];
    if (p.w_post) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) sum_w[i] = sum_n[i];
        if (GATE == GATE_ROW) {
            s.get_param(2, p.param_f32, c);
            mul_vec(sum_w, c);
        }
        store_vec(partial + p.H, sum_w);
    }
    if (GATE == GATE_ROW) {
        if (p.w_post) {
            s.get_param(1, p.param_f32, c);
            mul_vec(sum_n, c);
        }
        store_vec(partial + 2 * p.H, sum_n);
    }
}

// A row waits for the sums in registers, ITERS vectors a thread: a row a CTA or, up to 512 columns, a row a WARP, without
// barriers.
template <typename X, typename Y, bool FP8, int ITERS, bool WARP>
__global__ void __launch_bounds__(ITERS == 1 ? NORM_MAX_THREADS : NORM_MAX_H / 32) rms_norm_kernel(const NormParams p) {
    __shared__ float part[2][32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int row = WARP ? blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    if (WARP && row >= p.T) return;
    const int lane = WARP ? threadIdx.x & 31 : threadIdx.x, lanes = WARP ? 32 : blockDim.x;  // of the row
    auto row_sum = [&](float v, float *part) {
        if constexpr (WARP) return warp_sum(v);
        else return cta_sum(v, part);
    };
    const long long at = static_cast<long long>(row) * p.H;
    const float inv_h = 1.f / p.H;
    Raw<X> rx[ITERS];
    Raw<Y> ry[ITERS];
#pragma unroll
    for (int j = 0; j < ITERS; ++j) {
        const int col = (j * lanes + lane) * VEC;
        if (col < p.H) {
            rx[j].load(static_cast<const X *>(p.x) + at + col);
            if (p.y) ry[j].load(static_cast<const Y *>(p.y) + at + col);
        }
    }
    float r_post = 1.f;
    if (p.w_post) {
        float sum[2] = {};
#pragma unroll
        for (int j = 0; j < ITERS; ++j)
            if ((j * lanes + lane) * VEC < p.H) {
                float n[VEC];
                ry[j].get(n);
                dot_vec(sum, n, n);
            }
        r_post = rsqrtf(fmaf(row_sum(sum[0] + sum[1], part[0]), inv_h, p.eps));
        if (lane == 0 && p.rstd_post) p.rstd_post[row] = r_post;
    }
    float x[ITERS][VEC], sum[2] = {};
#pragma unroll
    for (int j = 0; j < ITERS; ++j) {
        const int col = (j * lanes + lane) * VEC;
        if (col >= p.H) continue;
        rx[j].get(x[j]);
        if (p.y) {
            float n[VEC], c[VEC];
            ry[j].get(n);
            if (p.w_post) {
                load_param(p.w_post, p.param_f32, col, c);
                mul_vec(n, r_post);
                mul_vec(n, c);
            }
            if (p.gate_kind != GATE_NONE) {
                if (p.gate_kind == GATE_ROW) load_param(p.gate, p.param_f32, col, c);
                else load_vec(static_cast<const Y *>(p.gate) + at + col, c);
                mul_vec(n, c);
            }
            fma_vec(x[j], n, p.alpha);
            store_vec(static_cast<X *>(p.x_out) + at + col, x[j]);
        }
        dot_vec(sum, x[j], x[j]);
    }
    if (!p.w) return;
    const float r = rsqrtf(fmaf(row_sum(sum[0] + sum[1], part[1]), inv_h, p.eps));
    if (lane == 0 && p.rstd) p.rstd[row] = r;
#pragma unroll
    for (int j = 0; j < ITERS; ++j) {
        const int col = (j * lanes + lane) * VEC;
        if (col >= p.H) continue;  // (a block's lanes are in or out together)
        float c[VEC];
        load_param(p.w, p.param_f32, col, c);
        mul_vec(x[j], r);
        mul_vec(c, x[j]);
        if constexpr (FP8) {
            float scale;
            *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.h) + at + col) = quantise(c, block_amax(c, col, p.H), scale);
            if ((threadIdx.x & (BLOCK_LANES - 1)) == 0) p.sf.sf[static_cast<long long>(col >> 7) * p.sf.ld + row] = scale;
        } else {
            store_vec(static_cast<Y *>(p.h) + at + col, c);
        }
    }
}

// Rows past NORM_RING_H columns, read from memory as they are needed.
template <typename X, typename Y, int ITERS>
__global__ void __launch_bounds__(NORM_WIDE_THREADS) rms_norm_backward_wide_kernel(const NormParams p) {
    __shared__ float part[2][32];
    grid_dependency_wait();
    grid_launch_dependents();
    const float inv_h = 1.f / p.H;
    float sum_w[ITERS][VEC] = {}, sum_post[ITERS][VEC] = {}, sum_gate[ITERS][VEC] = {};
    for (int row = blockIdx.x; row < p.T; row += gridDim.x) {
        const long long at = static_cast<long long>(row) * p.H;
        float dx[ITERS][VEC];
        float r = 0.f, r_post = 1.f;
        if (p.w) r = p.rstd[row];
        if (p.w_post) r_post = p.rstd_post[row];
        if (p.w) {
            float x[ITERS][VEC], sum[2] = {};  // x r, and w d_h in dx
#pragma unroll
            for (int j = 0; j < ITERS; ++j) {
                const int col = (j * blockDim.x + threadIdx.x) * VEC;
                if (col < p.H) {
                    float c[VEC];
                    load_vec(static_cast<const X *>(p.x) + at + col, x[j]);
                    load_vec(static_cast<const Y *>(p.d_h) + at + col, dx[j]);
                    load_param(p.w, p.param_f32, col, c);
                    mul_vec(x[j], r);
                    fma_vec(sum_w[j], dx[j], x[j]);
                    mul_vec(dx[j], c);
                    dot_vec(sum, dx[j], x[j]);
                }
            }
            const float mean = cta_sum(sum[0] + sum[1], part[0]) * inv_h;
#pragma unroll
            for (int j = 0; j < ITERS; ++j) {
                const int col = (j * blockDim.x + threadIdx.x) * VEC;
                if (col < p.H) {
                    fma_vec(dx[j], x[j], -mean);
                    if (p.d_x_out) {
                        load_vec(static_cast<const X *>(p.d_x_out) + at + col, x[j]);
                        fma_vec(x[j], dx[j], r);
#pragma unroll
                        for (int i = 0; i < VEC; ++i) dx[j][i] = x[j][i];
                    } else {
                        mul_vec(dx[j], r);
                    }
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < ITERS; ++j) {
                const int col = (j * blockDim.x + threadIdx.x) * VEC;
                if (col < p.H) load_vec(static_cast<const X *>(p.d_x_out) + at + col, dx[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < ITERS; ++j) {
            const int col = (j * blockDim.x + threadIdx.x) * VEC;
            if (col < p.H) store_vec(static_cast<X *>(p.d_x) + at + col, dx[j]);
        }
        if (p.y) {
            float n[ITERS][VEC], sum[2] = {};  // y r_post; from here on dx is the gradient of w_post n
#pragma unroll
            for (int j = 0; j < ITERS; ++j) {
                const int col = (j * blockDim.x + threadIdx.x) * VEC;
                if (col >= p.H) continue;
                float c[VEC];
                load_vec(static_cast<const Y *>(p.y) + at + col, n[j]);
                mul_vec(n[j], r_post);
                mul_vec(dx[j], p.alpha);
                if (p.gate_kind != GATE_NONE) {  // d_gate = d n post, then d gate
                    float d_gate[VEC];
#pragma unroll
                    for (int i = 0; i < VEC; ++i) d_gate[i] = n[j][i];
                    mul_vec(d_gate, dx[j]);
                    if (p.w_post) {
                        load_param(p.w_post, p.param_f32, col, c);
                        mul_vec(d_gate, c);
                    }
                    if (p.gate_kind == GATE_ROW) {
#pragma unroll
                        for (int i = 0; i < VEC; ++i) sum_gate[j][i] += d_gate[i];
                        load_param(p.gate, p.param_f32, col, c);
                    } else {
                        store_vec(static_cast<Y *>(p.d_gate_token) + at + col, d_gate);
                        load_vec(static_cast<const Y *>(p.gate) + at + col, c);
                    }
                    mul_vec(dx[j], c);
                }
                if (p.w_post) {
                    fma_vec(sum_post[j], dx[j], n[j]);
                    load_param(p.w_post, p.param_f32, col, c);
                    mul_vec(dx[j], c);
                    dot_vec(sum, dx[j], n[j]);
                }
            }
            const float mean = p.w_post ? cta_sum(sum[0] + sum[1], part[1]) * inv_h : 0.f;
#pragma unroll
            for (int j = 0; j < ITERS; ++j) {
                const int col = (j * blockDim.x + threadIdx.x) * VEC;
                if (col >= p.H) continue;
                if (p.w_post) {
                    fma_vec(dx[j], n[j], -mean);
                    mul_vec(dx[j], r_post);
                }
                store_vec(static_cast<Y *>(p.d_y) + at + col, dx[j]);
            }
        }
        if (!(p.w && p.w_post)) __syncthreads();
    }
    float *partial = p.partial + static_cast<long long>(blockIdx.x) * 3 * p.H;
#pragma unroll
    for (int j = 0; j < ITERS; ++j) {
        const int col = (j * blockDim.x + threadIdx.x) * VEC;
        if (col >= p.H) continue;
        if (p.w) store_vec(partial + col, sum_w[j]);
        if (p.w_post) store_vec(partial + p.H + col, sum_post[j]);
        if (p.gate_kind == GATE_ROW) store_vec(partial + 2 * p.H + col, sum_gate[j]);
    }
}

constexpr int NORM_SUM_THREADS = 1024;

// d[z][col] = sum over the CTAs' partial sums, in an order that does not change.  blockIdx.y: which of the three.  LANES lanes
// of four columns, the CTAs' sums in 1024 / LANES parts.
template <int LANES>
__global__ void __launch_bounds__(NORM_SUM_THREADS)
    rms_norm_sum_kernel(const float *partial, int ctas, int H, float *d0, float *d1, float *d2) {
    constexpr int kParts = NORM_SUM_THREADS / LANES;
    __shared__ float4 part[NORM_SUM_THREADS / 32][LANES];
    grid_dependency_wait();
    grid_launch_dependents();
    float *d = blockIdx.y == 0 ? d0 : blockIdx.y == 1 ? d1 : d2;
    if (!d) return;
    const int lane = threadIdx.x % LANES;
    const int col = (blockIdx.x * LANES + lane) * 4;  // (H is a multiple of 8)
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    if (col < H)
#pragma unroll 4
        for (int b = threadIdx.x / LANES; b < ctas; b += kParts) {
            const float4 v = *reinterpret_cast<const float4 *>(partial + (static_cast<long long>(b) * 3 + blockIdx.y) * H + col);
            sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
        }
#pragma unroll
    for (int i = LANES; i < 32; i *= 2) {
        sum.x += __shfl_xor_sync(0xffffffffu, sum.x, i);
        sum.y += __shfl_xor_sync(0xffffffffu, sum.y, i);
        sum.z += __shfl_xor_sync(0xffffffffu, sum.z, i);
        sum.w += __shfl_xor_sync(0xffffffffu, sum.w, i);
    }
    if ((threadIdx.x & 31) < LANES) part[threadIdx.x >> 5][lane] = sum;
    __syncthreads();
    const int out = blockIdx.x * LANES * 4 + threadIdx.x;  // a thread a column
    if (threadIdx.x < LANES * 4 && out < H) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < NORM_SUM_THREADS / 32; ++w) s += reinterpret_cast<const float *>(part[w])[threadIdx.x];
        d[out] = s;
    }
}

}  // namespace dg
