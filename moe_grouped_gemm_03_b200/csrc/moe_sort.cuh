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
// kernel is one cluster of up to 16 CTAs whose histograms meet in distributed shared memory: a second launch or a
// grid-wide barrier would cost more than the slots' arithmetic.  Every warp takes a consecutive run of slots, 32 at a
// time: match.any gives the lanes with the same expert, the warp's own histogram (no atomics: the order is fixed) the
// earlier ones.  Ranks wait in registers, or, past 256 slots a warp, in row_of_slot, read back by the lane that wrote them.
#pragma once
#include "rowwise.cuh"

namespace dg {

constexpr int SORT_MAX_GROUPS = 1024;
constexpr int SORT_MAX_WARPS = 32;
constexpr int SORT_MAX_CTAS = 16;
constexpr int SORT_BATCHES = 8;  // 32 slots each, loaded together
enum SortLayout { SORT_CONTIGUOUS = 0, SORT_NOPAD = 1, SORT_MASKED = 2 };

struct SortParams {
    const void *ids;      // [slots], 32 or 64 bits
    int slots, G, layout;
    int align;            // contiguous: rows of a group are padded to a multiple of this
    int M_total;          // contiguous: rows of m_indices
    int M_max;            // masked: rows of a group
    int slot_warps;       // warps of a CTA that take slots (the first ones), each a row of the histogram
    int per_warp;         // slots of such a warp, a multiple of 32
    int id_bits;          // bits that tell the groups apart
    int *row_of_slot;     // [slots]
    int *m_indices;       // [M_total] (contiguous)
    int *counts;          // [G]
    unsigned *err;
};

// Words of dynamic shared memory: a histogram for each warp with slots, the CTA's totals, every group's first row (and the
// end of the last), its row count and the CTA's first row in it, and the warps' parts of a sum.
__host__ __device__ constexpr int sort_smem_words(int slot_warps, int G) { return slot_warps * G + 4 * G + 1 + 32; }

__device__ __forceinline__ int sort_id(const SortParams &p, const int *ids, int i, bool &bad) {
    const int id = *(ids + i);
    bad |= id < -1 || id >= p.G;
    return id >= 0 && id < p.G ? id : -1;
}
__device__ __forceinline__ int sort_id(const SortParams &p, const long long *ids, int i, bool &bad) {
    const long long id = *(ids + i);
    bad |= id < -1 || id >= p.G;
    return id >= 0 && id < p.G ? static_cast<int>(id) : -1;
}

// Lanes whose slot has the same expert (none for a slot without one): one vote a bit of the expert's number.  match.any
// says the same in one instruction, but takes about 64 cycles of the SM each time: 65536 slots
// take 7 us with votes and took 14 with it (8 CTAs).
__device__ __forceinline__ unsigned same_expert(int id, int bits) {
    unsigned same = __ballot_sync(0xffffffffu, id >= 0);
    for (int b = 0; b < bits; ++b) {
        const bool one = (id >> b) & 1;
        const unsigned ones = __ballot_sync(0xffffffffu, one);
        same &= one ? ones : ~ones;
    }
    return same;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ int load_shared_rank(const int *p, int rank) {
    int v;
    asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(map_shared_rank(smem_u32(p), rank)) : "memory");
    return v;
}

// ONE: no warp has more than SORT_BATCHES * 32 slots, whose experts and ranks then stay in registers.
template <typename Id, bool ONE>
__global__ void __launch_bounds__(32 * SORT_MAX_WARPS) moe_sort_kernel(const SortParams p) {
    extern __shared__ int sort_smem[];
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ctas = gridDim.x, cta = blockIdx.x;  // one cluster
    int *hist = sort_smem, *total = hist + p.slot_warps * p.G, *start = total + p.G, *rows = start + p.G + 1,
        *base = rows + p.G, *part = base + p.G;
    for (int i = threadIdx.x; i < p.slot_warps * p.G; i += blockDim.x) hist[i] = 0;
    grid_dependency_wait();
    grid_launch_dependents();
    __syncthreads();

    // ranks within the warp's run
    const Id *ids = static_cast<const Id *>(p.ids);
    const long long begin64 = warp < p.slot_warps ? static_cast<long long>(cta * p.slot_warps + warp) * p.per_warp : p.slots;
    const int begin = static_cast<int>(begin64 < p.slots ? begin64 : p.slots);
    const int end = static_cast<int>(begin64 + p.per_warp < p.slots ? begin64 + p.per_warp : p.slots);
    constexpr int kChunk = 32 * SORT_BATCHES;
    int *mine = hist + warp * p.G;
    int id[SORT_BATCHES], rank[SORT_BATCHES];
    bool bad = false;
    for (int at = begin; at < end; at += kChunk) {
#pragma unroll
        for (int b = 0; b < SORT_BATCHES; ++b) {
            const int i = at + 32 * b + lane;
            id[b] = i < end ? sort_id(p, ids, i, bad) : -1;
        }
#pragma unroll
        for (int b = 0; b < SORT_BATCHES; ++b) {
            if (at + 32 * b >= end) break;
            const unsigned same = same_expert(id[b], p.id_bits);
            const int before = __popc(same & ((1u << lane) - 1));
            rank[b] = id[b] >= 0 ? mine[id[b]] + before : 0;
            __syncwarp();
            if (id[b] >= 0 && before == 0) mine[id[b]] += __popc(same);
            __syncwarp();
            if (!ONE && at + 32 * b + lane < end) p.row_of_slot[at + 32 * b + lane] = rank[b];
        }
        if (ONE) break;
    }
    if (bad) raise_bad_group(p.err);
    __syncthreads();

    // One thread a group (the CTA has at least G).  hist: earlier warps' counts of the CTA; total: the CTA's counts, which
    // the other CTAs read to find the group's rows and this CTA's first one among them.
    const int g = threadIdx.x;
    int all = 0, before = 0;
    if (g < p.G) {
        for (int w = 0; w < p.slot_warps; w += 8) {
            int n[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) n[i] = w + i < p.slot_warps ? hist[(w + i) * p.G + g] : 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (w + i < p.slot_warps) hist[(w + i) * p.G + g] = all;
                all += n[i];
            }
        }
        total[g] = all;
    }
    if (ctas > 1) {
        cluster_sync();
        if (g < p.G) {
            int n[SORT_MAX_CTAS];
            all = 0;
#pragma unroll
            for (int r = 0; r < SORT_MAX_CTAS; ++r) n[r] = r < ctas ? load_shared_rank(total + g, r) : 0;
#pragma unroll
            for (int r = 0; r < SORT_MAX_CTAS; ++r) {
                before += r < cta ? n[r] : 0;
                all += n[r];
            }
        }
        cluster_arrive();  // no CTA leaves while another reads its totals (the wait is at the end)
    }
    // start: the groups' exclusive sums
    const int a = p.layout == SORT_CONTIGUOUS ? p.align : 1;
    const int room = g >= p.G ? 0 : p.layout == SORT_MASKED ? p.M_max : (all + a - 1) / a * a;
    int sum = room;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += up;
    }
    if (lane == 31) part[warp] = sum;
    __syncthreads();
    int add = lane < warp ? part[lane] : 0;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) add += __shfl_xor_sync(0xffffffffu, add, d);
    if (g < p.G) {
        start[g] = sum - room + add;
        base[g] = start[g] + before;
        rows[g] = all;
        if (g == p.G - 1) start[p.G] = sum + add;
    }
    __syncthreads();

    // rows of the slots
    const int limit = p.layout == SORT_CONTIGUOUS ? p.M_total : 0x7fffffff;
    bool over = false;
    for (int at = begin; at < end; at += kChunk) {
        if (!ONE) {
#pragma unroll
            for (int b = 0; b < SORT_BATCHES; ++b) {
                const int i = at + 32 * b + lane;
                id[b] = i < end ? sort_id(p, ids, i, bad) : -1;
                rank[b] = i < end ? p.row_of_slot[i] : 0;
            }
        }
#pragma unroll
        for (int b = 0; b < SORT_BATCHES; ++b) {
            const int i = at + 32 * b + lane;
            if (i >= end) break;
            int row = -1;
            if (id[b] >= 0) {
                row = base[id[b]] + mine[id[b]] + rank[b];
                if (row >= (p.layout == SORT_MASKED ? (id[b] + 1) * p.M_max : limit)) {
                    row = -1;
                    over = true;
                }
            }
            p.row_of_slot[i] = row;
        }
        if (ONE) break;
    }
    if (over) raise_bad_group(p.err);

    // counts of the rows that were placed; groups of the rows
    if (cta == 0 && g < p.G) {
        int n = all;
        if (p.layout == SORT_MASKED) n = min(n, p.M_max);
        if (p.layout == SORT_CONTIGUOUS) n = min(n, max(0, p.M_total - start[g]));
        p.counts[g] = n;
    }
    if (p.layout == SORT_CONTIGUOUS) {
        // A warp writes 128 rows at a time: they belong to one group (the alignment is 128 or 256), the last one that starts
        // at or before them, found in two votes: over every 32nd group, then over the 32 from there.
        for (int b = cta * warps + warp; b < p.M_total / 128; b += ctas * warps) {
            const int row = b * 128;
            int h = -1;
            if (row < start[p.G]) {
                h = 32 * (__popc(__ballot_sync(0xffffffffu, 32 * lane < p.G && start[32 * lane] <= row)) - 1);
                h += __popc(__ballot_sync(0xffffffffu, h + lane < p.G && start[h + lane] <= row)) - 1;
            }
            const int last = h >= 0 ? start[h] + rows[h] : 0, r = row + 4 * lane;
            int4 v;
            v.x = r < last ? h : -1;
            v.y = r + 1 < last ? h : -1;
            v.z = r + 2 < last ? h : -1;
            v.w = r + 3 < last ? h : -1;
            *reinterpret_cast<int4 *>(p.m_indices + r) = v;
        }
    }
    if (ctas > 1) cluster_wait();
}

}  // namespace dg
