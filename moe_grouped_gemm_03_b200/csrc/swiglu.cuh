// SwiGLU between the two expert GEMMs, on the rows that the groups own, and its gradient.
//
//   h = g * sigmoid(g) * u,  gate_up = [g | u]
//   d_g = d_h * u * sigmoid(g) * (1 + g * (1 - sigmoid(g))),  d_u = d_h * g * sigmoid(g)
//
// Bound by HBM: forward 4 bytes in and 1 (e4m3) or 2 (bf16) out an element.  The warps of a CTA lie side by side on 2048
// columns of the same rows, so that a CTA reads and writes runs of kilobytes (a warp a row, walking along it, was 8% slower),
// and a warp takes ROWS rows at once: ROWS times two (backward: three) vector loads in flight, and scales that lie next to
// each other written together.  An e4m3 output adds the block's largest value (two reductions over the warp for 8 elements
// of each lane), its scale and the conversion: with the two special functions of an element they take as long as the memory
// (two thirds of the issue slots at 69632 x 2048).
#pragma once
#include "rowwise.cuh"

namespace dg {

constexpr int SWIGLU_WARPS = 8;
constexpr int STEP_COLS = 32 * VEC;  // columns of a warp
enum OwnedRows { OWN_ALL = 0, OWN_M_INDICES = 1, OWN_COUNTS = 2, OWN_MASKED = 3 };

struct SwigluParams {
    const void *gate_up;  // [R][2 * I]
    const void *d_out;    // gradient: [R][I]
    void *out;            // [R][I]; gradient: [R][2 * I]
    ScaleLayout sf;
    const int *own;       // m_indices [R], counts [G] or masked_m [G]
    int own_kind, G, R, I, rows_per_group;
    int cta_rows;         // rows of a CTA, at most 32
    int across;           // warps side by side in a row: 1, 2, 4 or 8
};

// s = sigmoid(g).  FAST, for bf16 and e4m3 results: exp and the reciprocal by their approximating instructions, off by (2 + |g|)
// 2^-23 of s, far below half a step of the result, 2^-8 or 2^-4 (fp32 to e4m3, 16976 x 4608: 86 us, 107 without).  The reciprocal
// is that of a quarter of 1 + exp(-g): the instruction has no results below 2^-126, which s falls to at g = -87.3 (the factor makes
// bf16 results 0.5% slower and e4m3 ones 0.5 to 2%, 69632 x 2048 124.6 us in place of 122.2).  From g = -88.7 down exp(-g) is
// infinite, in both forms, and s is 0.
template <bool FAST> __device__ __forceinline__ void sigmoid(const float (&g)[VEC], float (&s)[VEC]) {
    if constexpr (FAST) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) s[i] = g[i];
        mul_vec(s, -1.4426950408889634f);
#pragma unroll
        for (int i = 0; i < VEC; ++i) asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(s[i]));
        one_plus_times(s, 0.25f);
#pragma unroll
        for (int i = 0; i < VEC; ++i) asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(s[i]));
        mul_vec(s, 0.25f);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) s[i] = 1.f / (1.f + expf(-g[i]));
    }
}

template <typename T, bool FP8, bool BACKWARD, int ROWS>
__global__ void __launch_bounds__(32 * SWIGLU_WARPS, BACKWARD ? 3 : 4) swiglu_kernel(const SwigluParams p) {
    __shared__ int part[SWIGLU_WARPS];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int valid = p.R;  // no padding: rows that the counts cover (negative counts are none)
    if (p.own_kind == OWN_COUNTS) {
        int n = 0;
        for (int g = threadIdx.x; g < p.G; g += blockDim.x) n += min(max(p.own[g], 0), p.R - n);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) n += min(__shfl_xor_sync(0xffffffffu, n, d), p.R - n);
        if (lane == 0) part[warp] = n;
        __syncthreads();
        valid = 0;
        for (int i = 0; i < SWIGLU_WARPS; ++i) valid += min(part[i], p.R - valid);
    }
    // The CTA's rows, and which of them are rows of a group (a bit each).
    const int row0 = blockIdx.x * p.cta_rows;
    bool owned = false;
    if (lane < p.cta_rows && row0 + lane < p.R) {
        const int row = row0 + lane;
        if (p.own_kind == OWN_M_INDICES) owned = p.own[row] >= 0;
        else if (p.own_kind == OWN_MASKED) owned = row % p.rows_per_group < p.own[row / p.rows_per_group];
        else owned = row < valid;
    }
    const unsigned owned_rows = __ballot_sync(0xffffffffu, owned);
    if (!owned_rows) return;
    // `across` warps side by side cover a row's columns (or 2048 of them), the others take the next rows
    const int col = (blockIdx.y * SWIGLU_WARPS + (warp & (p.across - 1))) * STEP_COLS + lane * VEC;
    const bool in = col < p.I;
    const int stride = SWIGLU_WARPS / p.across * ROWS;
    int first = warp / p.across * ROWS;
    Raw<T> rg[ROWS], ru[ROWS], rd[BACKWARD ? ROWS : 1];
    auto load = [&](int r) {
        const T *gu = static_cast<const T *>(p.gate_up) + static_cast<long long>(row0 + first + r) * 2 * p.I + col;
        rg[r].load(gu);
        ru[r].load(gu + p.I);
        if constexpr (BACKWARD)
            rd[r].load(static_cast<const T *>(p.d_out) + static_cast<long long>(row0 + first + r) * p.I + col);
    };
    for (; first < p.cta_rows; first += stride) {
        const unsigned live = owned_rows >> first & ((1u << ROWS) - 1);
        if (!live || !in) continue;  // (`in` is the same in the lanes of a block where the output is e4m3)
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
            if (live >> r & 1) load(r);
        float keep = 0.f, keep_u = 0.f;  // lane r of a block's lanes: the scale of the block in row r
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
            if (live >> r & 1) {
                float g[VEC], u[VEC], a[VEC], b[VEC], d[VEC];
                rg[r].get(g);
                ru[r].get(u);
                if constexpr (BACKWARD) rd[r].get(d);
                sigmoid<sizeof(T) == 2 || FP8>(g, a);
                if constexpr (!BACKWARD) {
                    mul_vec(a, g);
                    mul_vec(a, u);
                } else {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) b[i] = 1.f - a[i];
#pragma unroll
                    for (int i = 0; i < VEC; ++i) b[i] = fmaf(g[i], b[i], 1.f);
                    // s is 0 where g is far below zero, so it comes first: u (1 + g (1 - s)) may pass the largest number
                    mul_vec(a, d);  // d s
                    mul_vec(b, a);
                    mul_vec(b, u);  // d_g
                    mul_vec(a, g);  // d_u
                }
                auto &left = BACKWARD ? b : a, &right = a;  // the output's columns from 0 and (gradient) from I on
                const long long at = static_cast<long long>(row0 + first + r) * (BACKWARD ? 2 : 1) * p.I + col;
                if constexpr (FP8) {
                    float scale;
                    uint8_t *out = static_cast<uint8_t *>(p.out) + at;
                    *reinterpret_cast<uint2 *>(out) = quantise(left, block_amax(left, col, p.I), scale);
                    if ((lane & (BLOCK_LANES - 1)) == r) keep = scale;
                    if constexpr (BACKWARD) {
                        *reinterpret_cast<uint2 *>(out + p.I) = quantise(right, block_amax(right, col, p.I), scale);
                        if ((lane & (BLOCK_LANES - 1)) == r) keep_u = scale;
                    }
                } else {
                    store_vec(static_cast<T *>(p.out) + at, left);
                    if constexpr (BACKWARD) store_vec(static_cast<T *>(p.out) + at + p.I, right);
                }
            }
        if constexpr (FP8) {
            const int r = lane & (BLOCK_LANES - 1);
            if (r < ROWS && (live >> r & 1)) {
                float *sf = p.own_kind == OWN_MASKED ? p.sf.at(row0 + first + r, 0) : p.sf.sf + row0 + first + r;
                sf[static_cast<long long>(col >> 7) * p.sf.ld] = keep;
                if constexpr (BACKWARD) sf[static_cast<long long>((p.I + col) >> 7) * p.sf.ld] = keep_u;
            }
        }
    }
}

}  // namespace dg
