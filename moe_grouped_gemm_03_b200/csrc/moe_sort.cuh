// Rows of the routed slots in the grouped GEMMs' layouts: a stable counting sort of the slots (token-major, k slots a
// token) by expert, in one launch.
//
//   rank(i)  = number of slots j < i with the same expert
//   row(i)   = start[expert(i)] + rank(i)
//
// start: exclusive sums of the counts (no padding), of the counts rounded up to the M alignment (contiguous), or
// g * M_max (masked).  Slots with expert -1 get row -1.
//
// The work is latency: 4 bytes in and 4 out a slot.  A histogram needs every slot before any row is known, so the
// kernel is one cluster of up to 8 CTAs whose histograms meet in distributed shared memory: a second launch or a
// grid-wide barrier would cost more than the slots' arithmetic.  Every warp takes a consecutive run of slots, 32 at a
// time: match.any gives the lanes with the same expert, the warp's own histogram (no atomics: the order is fixed) the
// earlier ones.  The rank waits in row_of_slot, read back by the lane that wrote it.
#pragma once
#include "rowwise.cuh"

namespace dg {

constexpr int SORT_MAX_GROUPS = 1024;
constexpr int SORT_MAX_WARPS = 32;
enum SortLayout { SORT_CONTIGUOUS = 0, SORT_NOPAD = 1, SORT_MASKED = 2 };

struct SortParams {
    const void *ids;      // [slots], 32 or 64 bits
    int slots, G, layout;
    int align;            // contiguous: rows of a group are padded to a multiple of this
    int M_total;          // contiguous: rows of m_indices
    int M_max;            // masked: rows of a group
    int per_warp;         // slots of a warp, a multiple of 32
    int *row_of_slot;     // [slots]
    int *m_indices;       // [M_total] (contiguous)
    int *counts;          // [G]
    unsigned *err;
};

// Words of dynamic shared memory: a histogram for each warp (odd stride: a column read by 32 lanes meets 32 banks),
// the CTA's totals, every group's first row and row count, and the CTA's first rank in every group.
__host__ __device__ constexpr int sort_smem_words(int warps, int G) { return warps * (G | 1) + 4 * G + 1 + 32; }

__device__ __forceinline__ int sort_id(const SortParams &p, const int *ids, int i, bool &bad) {
    const int id = __ldg(ids + i);
    bad |= id < -1 || id >= p.G;
    return id >= 0 && id < p.G ? id : -1;
}
__device__ __forceinline__ int sort_id(const SortParams &p, const long long *ids, int i, bool &bad) {
    const long long id = __ldg(ids + i);
    bad |= id < -1 || id >= p.G;
    return id >= 0 && id < p.G ? static_cast<int>(id) : -1;
}

__device__ __forceinline__ int load_shared_rank(const int *p, int rank) {
    int v;
    asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(map_shared_rank(smem_u32(p), rank)) : "memory");
    return v;
}

template <typename Id>
__global__ void __launch_bounds__(32 * SORT_MAX_WARPS) moe_sort_kernel(const SortParams p) {
    extern __shared__ int sort_smem[];
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ctas = gridDim.x, cta = blockIdx.x;  // one cluster
    const int stride = p.G | 1;
    int *hist = sort_smem, *total = hist + warps * stride, *start = total + p.G, *rows = start + p.G + 1,
        *first = rows + p.G, *part = first + p.G;
    grid_dependency_wait();
    grid_launch_dependents();
    for (int i = threadIdx.x; i < warps * stride; i += blockDim.x) hist[i] = 0;
    __syncthreads();

    // ranks within the warp's run
    const Id *ids = static_cast<const Id *>(p.ids);
    const long long begin64 = static_cast<long long>(cta * warps + warp) * p.per_warp;
    const int begin = static_cast<int>(begin64 < p.slots ? begin64 : p.slots);
    const int end = static_cast<int>(begin64 + p.per_warp < p.slots ? begin64 + p.per_warp : p.slots);
    int *mine = hist + warp * stride;
    bool bad = false;
    for (int base = begin; base < end; base += 32) {
        const int i = base + lane;
        const int id = i < end ? sort_id(p, ids, i, bad) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, id);
        const int before = __popc(same & ((1u << lane) - 1));
        int rank = 0;
        if (id >= 0) rank = mine[id] + before;
        __syncwarp();
        if (id >= 0 && before == 0) mine[id] += __popc(same);
        __syncwarp();
        if (i < end) p.row_of_slot[i] = rank;
    }
    if (bad) raise_bad_group(p.err);
    __syncthreads();

    // hist: earlier warps' counts of the CTA; total: the CTA's counts
    for (int g = warp; g < p.G; g += warps) {
        const int n = lane < warps ? hist[lane * stride + g] : 0;
        int sum = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, sum, d);
            if (lane >= d) sum += up;
        }
        if (lane < warps) hist[lane * stride + g] = sum - n;
        if (lane == 31) total[g] = sum;
    }
    __syncthreads();
    if (ctas > 1) cluster_sync();
    for (int g = threadIdx.x; g < p.G; g += blockDim.x) {
        int before = 0, all = 0;
        for (int r = 0; r < ctas; ++r) {
            const int n = ctas > 1 ? load_shared_rank(total + g, r) : total[g];
            before += r < cta ? n : 0;
            all += n;
        }
        first[g] = before;
        rows[g] = all;
    }
    if (ctas > 1) cluster_sync();  // no CTA leaves while another reads its totals
    __syncthreads();

    // start: exclusive sums over the groups, 32 to a warp step and the steps' sums in turn
    if (p.layout == SORT_MASKED) {
        for (int g = threadIdx.x; g < p.G; g += blockDim.x) start[g] = g * p.M_max;
    } else {
        const int steps = (p.G + 31) / 32;
        const int a = p.layout == SORT_CONTIGUOUS ? p.align : 1;
        for (int s = warp; s < steps; s += warps) {
            const int g = s * 32 + lane;
            const int n = g < p.G ? (rows[g] + a - 1) / a * a : 0;
            int sum = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, sum, d);
                if (lane >= d) sum += up;
            }
            if (g < p.G) start[g] = sum - n;
            if (lane == 31) part[s] = sum;
        }
        __syncthreads();
        for (int g = threadIdx.x; g < p.G; g += blockDim.x) {
            int add = 0;
            for (int s = 0; s < g / 32; ++s) add += part[s];
            start[g] += add;
            if (g == p.G - 1) start[p.G] = start[g] + (rows[g] + a - 1) / a * a;
        }
    }
    __syncthreads();

    // rows of the slots
    const int limit = p.layout == SORT_CONTIGUOUS ? p.M_total : 0x7fffffff;
    bool over = false;
    bad = false;
    for (int base = begin; base < end; base += 32) {
        const int i = base + lane;
        if (i >= end) break;
        const int id = sort_id(p, ids, i, bad);
        int row = -1;
        if (id >= 0) {
            const int rank = first[id] + mine[id] + p.row_of_slot[i];
            row = start[id] + rank;
            if (row >= limit || (p.layout == SORT_MASKED && rank >= p.M_max)) {
                row = -1;
                over = true;
            }
        }
        p.row_of_slot[i] = row;
    }
    if (over) raise_bad_group(p.err);

    // counts of the rows that were placed; groups of the rows
    if (cta == 0)
        for (int g = threadIdx.x; g < p.G; g += blockDim.x) {
            int n = rows[g];
            if (p.layout == SORT_MASKED) n = min(n, p.M_max);
            if (p.layout == SORT_CONTIGUOUS) n = min(n, max(0, p.M_total - start[g]));
            p.counts[g] = n;
        }
    if (p.layout == SORT_CONTIGUOUS) {
        // a warp writes 128 rows at a time: they belong to one group (the alignment is 128 or 256)
        for (int b = cta * warps + warp; b < p.M_total / 128; b += ctas * warps) {
            const int row = b * 128;
            int g = -1;
            if (row < start[p.G]) {
                int lo = 0, hi = p.G;  // the last group that starts at or before the row
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (start[mid] <= row) lo = mid; else hi = mid;
                }
                g = lo;
            }
            const int last = g >= 0 ? start[g] + rows[g] : 0, r = row + 4 * lane;
            int4 v;
            v.x = r < last ? g : -1;
            v.y = r + 1 < last ? g : -1;
            v.z = r + 2 < last ? g : -1;
            v.w = r + 3 < last ? g : -1;
            *reinterpret_cast<int4 *>(p.m_indices + r) = v;
        }
    }
}

}  // namespace dg
