// Rows to the experts and back: dispatch (gather of the tokens into the operand of a grouped GEMM, quantised on the
// way), combine (weighted sum of a token's expert rows) and the combine's gradient.  All three go by tokens and read
// row_of_slot [T][k]; a slot without a row (-1) takes no part.
//
//   permute            a[row(t, s)] = x[t]                       (e4m3: codes and scales of the token, made once)
//   unpermute          out[t] = sum_s w(t, s) * rows[row(t, s)]
//   its gradient       d_rows[row(t, s)] = w(t, s) * d_out[t],  d_w(t, s) = <d_out[t], rows[row(t, s)]>
//
// All are bound by HBM.  Permute reads a token's row once, whatever k is, and unpermute each expert row once; the gradient
// reads d_out's row, and finds its blocks' largest values, once for every 8 slots of the token (the second time from L2).
#pragma once
#include "rowwise.cuh"

namespace dg {

constexpr int MAX_TOPK = 32;     // one lane of a warp for each slot of a token
constexpr int ROWS_WARPS = 8;    // warps of a CTA (permute, unpermute)
constexpr int STEP = 32 * VEC;   // elements of one step of a warp

struct RowsParams {
    const void *x;           // permute: x [T][H]; unpermute and gradient: rows [rows][H]
    const void *d_out;       // gradient: [T][H]
    const int *row_of_slot;  // [T][k]
    const float *weights;    // [T][k]; null: 1 (unpermute)
    void *out;               // permute, gradient: [rows][H]; unpermute: [T][H]
    float *d_weights;        // gradient: [T][k]
    ScaleLayout sf;
    long long T;
    int k, H, rows, segments;  // segments: parts of a row, each a warp's work
    unsigned *err;
};

// Lane s's row of slot s of the token: -1 if there is none (or it is out of range, which is recorded).
__device__ __forceinline__ int slot_row(const RowsParams &p, long long token, int s) {
    if (s >= p.k) return -1;
    const int row = *(p.row_of_slot + token * p.k + s);
    if (row >= p.rows || row < -1) raise_bad_group(p.err);
    return row < p.rows ? row : -1;
}

constexpr int PERMUTE_COLS = 1024;  // of a token, a warp's work

// All loads first, then each block is quantised once, then the slots in turn, so that a slot's address is made once for all
// of its stores.
template <typename T, bool FP8>
__global__ void __launch_bounds__(32 * ROWS_WARPS) permute_kernel(const RowsParams p) {
    constexpr int kSteps = PERMUTE_COLS / STEP;
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long item = static_cast<long long>(blockIdx.x) * ROWS_WARPS + (threadIdx.x >> 5);
    const long long token = item / p.segments;
    if (token >= p.T) return;
    const int row = slot_row(p, token, lane);
    const unsigned live = __ballot_sync(0xffffffffu, row >= 0);
    if (!live) return;
    const int begin = static_cast<int>(item - token * p.segments) * PERMUTE_COLS + lane * VEC;
    const T *x = static_cast<const T *>(p.x) + token * p.H;
    Raw<T> r[kSteps];
#pragma unroll
    for (int j = 0; j < kSteps; ++j)
        if (begin + j * STEP < p.H) r[j].load(x + begin + j * STEP);
    if constexpr (FP8) {
        uint2 q[kSteps];
        float scale[kSteps];
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
            if (begin + j * STEP >= p.H) continue;  // (a block's lanes are in or out together)
            float v[VEC];
            r[j].get(v);
            q[j] = quantise(v, block_amax(v, begin + j * STEP, p.H), scale[j]);
        }
        for (unsigned m = live; m; m &= m - 1) {
            const long long at = __shfl_sync(0xffffffffu, row, __ffs(m) - 1);
            uint8_t *out = static_cast<uint8_t *>(p.out) + at * p.H + begin;
#pragma unroll
            for (int j = 0; j < kSteps; ++j)
                if (begin + j * STEP < p.H) *reinterpret_cast<uint2 *>(out + j * STEP) = q[j];
        }
        // lane s of each block's lanes writes slot s's scale of the block, 16 slots at a time
        for (int s = 0; s < p.k; s += BLOCK_LANES) {
            const int at = __shfl_sync(0xffffffffu, row, s + (lane & (BLOCK_LANES - 1)));
            if (at < 0) continue;
            float *sf = p.sf.at(at, begin >> 7);
#pragma unroll
            for (int j = 0; j < kSteps; ++j)
                if (begin + j * STEP < p.H) sf[static_cast<long long>(j) * (STEP / 128) * p.sf.ld] = scale[j];
        }
    } else {
        for (unsigned m = live; m; m &= m - 1) {
            const long long at = __shfl_sync(0xffffffffu, row, __ffs(m) - 1);
            T *out = static_cast<T *>(p.out) + at * p.H + begin;
#pragma unroll
            for (int j = 0; j < kSteps; ++j)
                if (begin + j * STEP < p.H) r[j].store(out + j * STEP);
        }
    }
}

// The sum is taken in fp32 in the slots' order and rounded once; U rows' loads are in flight at a time.
template <typename T, int U>
__global__ void __launch_bounds__(32 * ROWS_WARPS) unpermute_kernel(const RowsParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long item = static_cast<long long>(blockIdx.x) * ROWS_WARPS + (threadIdx.x >> 5);
    const long long token = item / p.segments;
    if (token >= p.T) return;
    const int row = slot_row(p, token, lane);
    const float w = row >= 0 && p.weights ? *(p.weights + token * p.k + lane) : 1.f;
    const int col = static_cast<int>(item - token * p.segments) * STEP + lane * VEC;
    const bool in = col < p.H;
    const T *rows = static_cast<const T *>(p.x) + (in ? col : 0);
    float acc[VEC] = {};
    unsigned m = __ballot_sync(0xffffffffu, row >= 0);
    while (m) {
        Raw<T> r[U];
        float weight[U];
        int n = 0;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (m) {
                const int s = __ffs(m) - 1;
                m &= m - 1;
                const long long at = __shfl_sync(0xffffffffu, row, s);
                weight[u] = __shfl_sync(0xffffffffu, w, s);
                r[u].load(rows + at * p.H);
                n = u + 1;
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (u < n) {
                float v[VEC];
                r[u].get(v);
#pragma unroll
                for (int i = 0; i < VEC; ++i) acc[i] = fmaf(weight[u], v[i], acc[i]);
            }
    }
    if (in) store_vec(static_cast<T *>(p.out) + token * p.H + col, acc);
}

constexpr int GRAD_MAX_WARPS = 16;

// The inner products need whole rows: a CTA a token or, with many tokens, a WARP a token, which needs no barrier and lets a
// short row's latency be covered by other tokens.  SLOTS of a token at a time, their loads together.  fp32 sums, in an order
// that does not change.
template <typename T, bool FP8, int SLOTS, bool WARP>
__global__ void __launch_bounds__(32 * (WARP ? ROWS_WARPS : GRAD_MAX_WARPS), WARP ? 2 : 1)
    unpermute_backward_kernel(const RowsParams p) {
    __shared__ float part[SLOTS][GRAD_MAX_WARPS];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = WARP ? 0 : threadIdx.x >> 5, warps = WARP ? 1 : blockDim.x >> 5;
    const long long token = WARP ? static_cast<long long>(blockIdx.x) * ROWS_WARPS + (threadIdx.x >> 5) : blockIdx.x;
    if (WARP && token >= p.T) return;
    const int row = slot_row(p, token, lane);
    const float w = lane < p.k ? p.weights[token * p.k + lane] : 0.f;
    const T *d_out = static_cast<const T *>(p.d_out) + token * p.H;
    const T *rows = static_cast<const T *>(p.x);
    for (int first = 0; first < p.k; first += SLOTS) {
        int at[SLOTS];
        float weight[SLOTS], acc[SLOTS][2] = {};
#pragma unroll
        for (int u = 0; u < SLOTS; ++u) {
            at[u] = __shfl_sync(0xffffffffu, row, (first + u) & 31);
            if (first + u >= p.k) at[u] = -1;
            weight[u] = __shfl_sync(0xffffffffu, w, (first + u) & 31);
        }
        // lanes u and 16 + u write slot first + u's scales: this is where the row's first one goes
        float *sf = nullptr;
        if constexpr (FP8) {
            const int mine = __shfl_sync(0xffffffffu, row, (first + (lane & 15)) & 31);
            if ((lane & 15) < SLOTS && first + (lane & 15) < p.k && mine >= 0) sf = p.sf.at(mine, 0);
        }
        for (int col = warp * STEP + lane * VEC; col < p.H; col += warps * STEP) {  // (a block's lanes end together)
            Raw<T> r[SLOTS];
#pragma unroll
            for (int u = 0; u < SLOTS; ++u)
                if (at[u] >= 0) r[u].load(rows + static_cast<long long>(at[u]) * p.H + col);
            float d[VEC], amax = 0.f, keep = 0.f;
            load_vec(d_out + col, d);
            if constexpr (FP8) amax = block_amax(d, col, p.H);
#pragma unroll
            for (int u = 0; u < SLOTS; ++u)
                if (at[u] >= 0) {
                    float v[VEC];
                    r[u].get(v);
                    dot_vec(acc[u], d, v);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) v[i] = d[i];
                    mul_vec(v, weight[u]);
                    if constexpr (FP8) {
                        // rounding keeps order: the largest of the rounded products is the product of the largest
                        float scale;
                        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.out) + static_cast<long long>(at[u]) * p.H + col) =
                            quantise(v, fabsf(weight[u]) * amax, scale);
                        if ((lane & 15) == u) keep = scale;
                    } else {
                        store_vec(static_cast<T *>(p.out) + static_cast<long long>(at[u]) * p.H + col, v);
                    }
                }
            if constexpr (FP8)
                if (sf) sf[static_cast<long long>(col >> 7) * p.sf.ld] = keep;
        }
        __syncwarp();
#pragma unroll
        for (int u = 0; u < SLOTS; ++u) {
            float sum = acc[u][0] + acc[u][1];
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            if (WARP) {
                if (lane == 0 && first + u < p.k) p.d_weights[token * p.k + first + u] = sum;
            } else if (lane == 0) {
                part[u][warp] = sum;
            }
        }
        if (!WARP) {
            __syncthreads();
            if (threadIdx.x < SLOTS && first + threadIdx.x < p.k) {
                float sum = 0.f;
                for (int i = 0; i < warps; ++i) sum += part[threadIdx.x][i];
                p.d_weights[token * p.k + first + threadIdx.x] = sum;
            }
            __syncthreads();
        }
    }
}

}  // namespace dg
