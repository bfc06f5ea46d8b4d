// SwiGLU between the two expert GEMMs, on the rows that the groups own, and its gradient.
//
//   h = g * sigmoid(g) * u,  gate_up = [g | u]
//   d_g = d_h * u * sigmoid(g) * (1 + g * (1 - sigmoid(g))),  d_u = d_h * g * sigmoid(g)
//
// Bound by HBM: forward 4 bytes in and 1 (e4m3) or 2 (bf16) out an element.  A warp takes ROWS consecutive rows, 256
// columns at a time, so that ROWS times two (backward: three) vector loads are in flight and the rows' scales, which
// lie next to each other, are written together.
#pragma once
#include "rowwise.cuh"

namespace dg {

constexpr int SWIGLU_WARPS = 8;
enum OwnedRows { OWN_ALL = 0, OWN_M_INDICES = 1, OWN_COUNTS = 2, OWN_MASKED = 3 };

struct SwigluParams {
    const void *gate_up;  // [R][2 * I]
    const void *d_out;    // gradient: [R][I]
    void *out;            // [R][I]; gradient: [R][2 * I]
    ScaleLayout sf;
    const int *own;       // m_indices [R], counts [G] or masked_m [G]
    int own_kind, G, R, I, rows_per_group;
    int segment;          // columns of a warp's work, a multiple of 256
};

// bf16: exp and the reciprocal by their approximating instructions, each within a few 2^-23 (|g| < 20), far below half a
// step of the result, 2^-8.  exp(-g) of a large negative g is infinite and its reciprocal 0, as it should be.
template <typename T> __device__ __forceinline__ float sigmoid(float g);
template <> __device__ __forceinline__ float sigmoid<bf16>(float g) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}
template <> __device__ __forceinline__ float sigmoid<float>(float g) { return 1.f / (1.f + expf(-g)); }

template <typename T, bool FP8, bool BACKWARD, int ROWS>
__global__ void __launch_bounds__(32 * SWIGLU_WARPS, BACKWARD ? 3 : 4) swiglu_kernel(const SwigluParams p) {
    __shared__ int part[SWIGLU_WARPS];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int valid = p.R;  // no padding: rows that the counts cover (negative counts are none)
    if (p.own_kind == OWN_COUNTS) {
        int n = 0;
        for (int g = threadIdx.x; g < p.G; g += blockDim.x) n = min(n + max(*(p.own + g), 0), p.R);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) n = min(n + __shfl_xor_sync(0xffffffffu, n, d), p.R);
        if (lane == 0) part[warp] = n;
        __syncthreads();
        valid = 0;
        for (int i = 0; i < SWIGLU_WARPS; ++i) valid = min(valid + part[i], p.R);
    }
    const int row0 = (blockIdx.x * SWIGLU_WARPS + warp) * ROWS;
    bool owned = false;  // lane r: whether row0 + r is a row of a group
    if (lane < ROWS && row0 + lane < p.R) {
        const int row = row0 + lane;
        if (p.own_kind == OWN_M_INDICES) owned = *(p.own + row) >= 0;
        else if (p.own_kind == OWN_MASKED)
            owned = row % p.rows_per_group < *(p.own + row / p.rows_per_group);
        else owned = row < valid;
    }
    const unsigned live = __ballot_sync(0xffffffffu, owned);
    if (!live) return;
    const int end = min(p.I, (static_cast<int>(blockIdx.y) + 1) * p.segment);
    for (int base = blockIdx.y * p.segment; base < end; base += 32 * VEC) {
        const int col = base + lane * VEC;
        const bool in = col < end;
        Raw8<T> rg[ROWS], ru[ROWS], rd[BACKWARD ? ROWS : 1];
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
            if (in && (live >> r & 1)) {
                const T *gu = static_cast<const T *>(p.gate_up) + static_cast<long long>(row0 + r) * 2 * p.I + col;
                rg[r].load(gu);
                ru[r].load(gu + p.I);
                if constexpr (BACKWARD)
                    rd[r].load(static_cast<const T *>(p.d_out) + static_cast<long long>(row0 + r) * p.I + col);
            }
        float keep = 0.f, keep_u = 0.f;  // lanes r and 16 + r: the scales of row r's two blocks
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
            if (live >> r & 1) {
                float g[VEC] = {}, u[VEC] = {}, a[VEC], b[VEC];
                if (in) {
                    rg[r].get(g);
                    ru[r].get(u);
                }
                if constexpr (!BACKWARD) {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) a[i] = g[i] * sigmoid<T>(g[i]) * u[i];
                } else {
                    float d[VEC] = {};
                    if (in) rd[r].get(d);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const float s = sigmoid<T>(g[i]), silu = g[i] * s;
                        a[i] = d[i] * u[i] * s * (1.f + g[i] * (1.f - s));
                        b[i] = d[i] * silu;
                    }
                }
                const long long at = static_cast<long long>(row0 + r) * (BACKWARD ? 2 : 1) * p.I + col;
                if constexpr (FP8) {
                    float scale;
                    uint8_t *out = static_cast<uint8_t *>(p.out) + at;
                    const uint2 q = quantise8(a, block_amax(a), scale);
                    if ((lane & 15) == r) keep = scale;
                    if (in) *reinterpret_cast<uint2 *>(out) = q;
                    if constexpr (BACKWARD) {
                        const uint2 qu = quantise8(b, block_amax(b), scale);
                        if ((lane & 15) == r) keep_u = scale;
                        if (in) *reinterpret_cast<uint2 *>(out + p.I) = qu;
                    }
                } else if (in) {
                    store8(static_cast<T *>(p.out) + at, a);
                    if constexpr (BACKWARD) store8(static_cast<T *>(p.out) + at + p.I, b);
                }
            }
        if constexpr (FP8) {
            const int r = lane & 15;
            if (in && r < ROWS && (live >> r & 1)) {
                *p.sf.at(row0 + r, col >> 7) = keep;
                if constexpr (BACKWARD) *p.sf.at(row0 + r, (p.I + col) >> 7) = keep_u;
            }
        }
    }
}

}  // namespace dg
