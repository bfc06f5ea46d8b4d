// Host side of the operators around the grouped GEMMs (include/dg.h): argument validation and launches of dispatch,
// combine, SwiGLU and the norms on the caller's stream.  Compiled behind dg_api.cu (libdg.cu), whose errors, device
// information, scratch pool and settings it uses.
#pragma once
#include "moe_rows.cuh"
#include "moe_sort.cuh"
#include "rms_norm.cuh"
#include "swiglu.cuh"

namespace {

using dg::bf16;

constexpr int kMaxRows = 1 << 30;  // rows and tokens of a call: row arithmetic stays within 32 bits

// Vectors of eight elements: 16 bytes of bf16, 32 of fp32.
bool vec_aligned(const void *p, int type) { return aligned(p, type == DG_F32 ? 32 : 16); }
bool is_type(int t) { return t == DG_BF16 || t == DG_F32; }
int aligned_rows(int rows) { return (rows + 3) / 4 * 4; }

// The current device (an sm_100) and its SMs under the cap of dg_set_num_sms.
int current_device(int &device, int &num_sms) {
    DeviceInfo info;
    if (int rc = device_info(info)) return rc;
    device = info.device;
    num_sms = effective_sms(info);
    return DG_OK;
}

// Launches `kernel` as a programmatic dependent: it may be set up while the kernel before it on the stream ends, and
// waits for that one (griddepcontrol.wait) before it touches memory.  Every kernel of this file does so at its start.
template <typename... Params, typename... Args>
int launch(const char *name, void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, int cluster, dg_stream_t stream,
           Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e == cudaSuccess ? DG_OK : cuda_fail(e, name);
}

// Lets `Kernel` have `bytes` of dynamic shared memory, the most that any call of it asks for, once per kernel and device.  The
// attribute belongs to the function and is shared by all host threads: set by each call to its own size, it could be lowered by
// another thread's smaller call before the launch, which the runtime then refuses.
template <auto Kernel> int allow_shared(int device, int bytes, const char *what) {
    static std::atomic<bool> set[64];
    if (device < 64 && set[device].load(std::memory_order_acquire)) return DG_OK;
    const cudaError_t e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return cuda_fail(e, what);
    if (device < 64) set[device].store(true, std::memory_order_release);
    return DG_OK;
}

// ------------------------------------------------------------------------------------------------ dispatch: rows
int check_sort(const void *topk_ids, int id_bytes, int T, int k, int G, const int *row_of_slot, const int *counts) {
    if (!counts || (T > 0 && (!topk_ids || !row_of_slot))) return fail(DG_ERR_INVALID_ARG, "null pointer argument");
    if (id_bytes != 4 && id_bytes != 8) return fail(DG_ERR_INVALID_ARG, "id_bytes=%d must be 4 or 8", id_bytes);
    if (topk_ids && topk_ids == row_of_slot) return fail(DG_ERR_INVALID_ARG, "row_of_slot must not be topk_ids");
    if (!aligned(topk_ids, id_bytes) || !aligned(row_of_slot, 4) || !aligned(counts, 4))
        return fail(DG_ERR_ALIGNMENT, "topk_ids, row_of_slot and counts must be aligned to their elements");
    if (T < 0) return fail(DG_ERR_INVALID_ARG, "T=%d must be non-negative", T);
    if (k < 1 || k > dg::MAX_TOPK) return fail(DG_ERR_INVALID_ARG, "k=%d must be in [1, %d]", k, dg::MAX_TOPK);
    if (G < 1 || G > dg::SORT_MAX_GROUPS)
        return fail(DG_ERR_INVALID_ARG, "G=%d must be in [1, %d]", G, dg::SORT_MAX_GROUPS);
    if (static_cast<long long>(T) * k > kMaxRows) return fail(DG_ERR_INVALID_ARG, "T*k exceeds 2^30");
    return DG_OK;
}

// Makes one of the sort's kernels ready on the current device: its shared memory, and clusters of more than 8 CTAs.  `most`
// becomes the largest of 16, 8 and 1 CTAs (or stays, if smaller) whose cluster the device can place with the most shared memory
// and threads that a call asks for: 16 CTAs need as many free SMs in one GPC, which a part of a GPU may not have.
template <typename Id, bool ONE> int prepare_sort(int device, int &most) {
    constexpr auto kernel = dg::moe_sort_kernel<Id, ONE>;
    constexpr int kMostShared = static_cast<int>(sizeof(int)) * dg::sort_smem_words(dg::SORT_MAX_WARPS, dg::SORT_MAX_GROUPS);
    if (int rc = allow_shared<kernel>(device, kMostShared, "cudaFuncSetAttribute (sort)")) return rc;
    if (most > 8 && cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
        cudaGetLastError();  // (what the runtime refuses here is no error of the call)
        most = 8;
    }
    for (; most > 1; most = most > 8 ? 8 : 1) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(most);
        cfg.blockDim = dim3(32 * dg::SORT_MAX_WARPS);
        cfg.dynamicSmemBytes = kMostShared;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = static_cast<unsigned>(most);
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int clusters = 0;
        if (cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) != cudaSuccess) cudaGetLastError();
        else if (clusters > 0) break;
    }
    return DG_OK;
}

// The most CTAs of a sort's cluster on this device, found by its first sort.
int sort_most_ctas(int device, int &most) {
    static std::atomic<int> cache[64];
    if (device < 64 && (most = cache[device].load(std::memory_order_acquire)) > 0) return DG_OK;
    most = dg::SORT_MAX_CTAS;
    int rc = prepare_sort<int, true>(device, most);
    if (!rc) rc = prepare_sort<int, false>(device, most);
    if (!rc) rc = prepare_sort<long long, true>(device, most);
    if (!rc) rc = prepare_sort<long long, false>(device, most);
    if (!rc && device < 64) cache[device].store(most, std::memory_order_release);
    return rc;
}

template <typename Id, bool ONE> int launch_sort(const dg::SortParams &p, int warps, int ctas, dg_stream_t stream) {
    return launch("sort launch", dg::moe_sort_kernel<Id, ONE>, dim3(ctas), dim3(32 * warps),
                  sizeof(int) * dg::sort_smem_words(p.slot_warps, p.G), ctas, stream, p);
}

int sort_call(dg::SortParams p, int id_bytes, int T, int k, dg_stream_t stream) {
    int device, sms;
    if (int rc = current_device(device, sms)) return rc;
    p.slots = T * k;
    p.err = device_error_word();
    if (!p.err) return fail(DG_ERR_CUDA, "device error word is not available");
    int warps = (p.slots + 31) / 32;
    // Measured (us, 256 groups, one CTA / 8 / 16): 256 slots 2.9 / 3.8 / -, 1024 slots 6.2 / 3.8 / -, 2048 slots
    // 7.0 / 3.9 / 3.9, 8192 slots - / 5.3 / 4.3, 65536 slots - / 10.4 / 7.9.
    int ctas = warps > 32 ? 16 : warps > 8 ? 8 : 1, most;
    if (int rc = sort_most_ctas(device, most)) return rc;
    if (most > sms) most = sms;  // (the cap of dg_set_num_sms: a sort's CTAs take an SM each)
    if (ctas > most) ctas = most >= 8 ? 8 : 1;
    static const bool debug = getenv("DG_DEBUG") && getenv("DG_DEBUG")[0] == '1';
    if (debug) fprintf(stderr, "[dg] sort layout=%d slots=%d G=%d ctas=%d\n", p.layout, p.slots, p.G, ctas);
    warps = (warps + ctas - 1) / ctas;
    p.slot_warps = warps < 1 ? 1 : warps > dg::SORT_MAX_WARPS ? dg::SORT_MAX_WARPS : warps;
    const int all = p.slot_warps * ctas;
    p.per_warp = ((p.slots + all - 1) / all + 31) / 32 * 32;
    while ((1 << p.id_bits) < p.G) ++p.id_bits;
    // a thread for each group's column too
    const int group_warps = (p.G + 31) / 32;
    warps = p.slot_warps > group_warps ? p.slot_warps : group_warps;
    const bool one = p.per_warp <= 32 * dg::SORT_BATCHES;
    if (id_bytes == 8)
        return one ? launch_sort<long long, true>(p, warps, ctas, stream) : launch_sort<long long, false>(p, warps, ctas, stream);
    return one ? launch_sort<int, true>(p, warps, ctas, stream) : launch_sort<int, false>(p, warps, ctas, stream);
}

// ----------------------------------------------------------------------------------------- dispatch and combine
int check_rows(const void *x, const int *row_of_slot, const void *out, const float *out_sf, int type, int T, int k, int H,
               int rows) {
    // (a tensor without elements may be null)
    if (T > 0 && (!x || !row_of_slot || !out)) return fail(DG_ERR_INVALID_ARG, "null pointer argument");
    if (!is_type(type)) return fail(DG_ERR_INVALID_ARG, "unknown element type %d", type);
    if (T < 0 || T > kMaxRows || rows < 0 || rows > kMaxRows)
        return fail(DG_ERR_INVALID_ARG, "T=%d and rows=%d must be in [0, 2^30]", T, rows);
    if (k < 1 || k > dg::MAX_TOPK) return fail(DG_ERR_INVALID_ARG, "k=%d must be in [1, %d]", k, dg::MAX_TOPK);
    if (H <= 0 || H > (1 << 24)) return fail(DG_ERR_INVALID_ARG, "H=%d must be in [1, 2^24]", H);
    if (H % dg::VEC) return fail(DG_ERR_ALIGNMENT, "H=%d must be a multiple of %d", H, dg::VEC);
    if (!vec_aligned(x, type) || !vec_aligned(out, out_sf ? DG_BF16 : type))
        return fail(DG_ERR_ALIGNMENT, "row operands must be 16-byte (fp32: 32-byte) aligned");
    if (!aligned(row_of_slot, 4)) return fail(DG_ERR_ALIGNMENT, "row_of_slot must be 4-byte aligned");
    return DG_OK;
}

// An e4m3 output's scales: rows in groups of rows_per_group, cols a multiple of 128.
int scale_layout(dg::ScaleLayout &sf, float *out_sf, int rows, int rows_per_group, int cols) {
    sf = dg::ScaleLayout{out_sf, 1, 4, 1};
    if (!out_sf) return DG_OK;
    if (cols % 128) return fail(DG_ERR_ALIGNMENT, "an e4m3 output's width %d must be a multiple of 128", cols);
    if (!aligned(out_sf, 16)) return fail(DG_ERR_ALIGNMENT, "the scales must be 16-byte aligned");
    if (rows > 0 && (rows_per_group < 1 || rows % rows_per_group))
        return fail(DG_ERR_INVALID_ARG, "rows=%d must be a multiple of rows_per_group=%d", rows, rows_per_group);
    if (rows > 0) sf = dg::ScaleLayout{out_sf, rows_per_group, aligned_rows(rows_per_group), cols / 128};
    return DG_OK;
}

int rows_params(dg::RowsParams &p, const void *x, const int *row_of_slot, int T, int k, int H, int rows, void *out) {
    int device, sms;
    if (int rc = current_device(device, sms)) return rc;
    p.x = x;
    p.row_of_slot = row_of_slot;
    p.T = T;
    p.k = k;
    p.H = H;
    p.rows = rows;
    p.out = out;
    p.err = device_error_word();
    return p.err ? DG_OK : fail(DG_ERR_CUDA, "device error word is not available");
}

unsigned row_ctas(long long items) { return static_cast<unsigned>((items + dg::ROWS_WARPS - 1) / dg::ROWS_WARPS); }
int check_items(long long items) {
    return items <= 0x7fffffffLL * dg::ROWS_WARPS ? DG_OK : fail(DG_ERR_INVALID_ARG, "T*H is out of range");
}

template <typename T, bool FP8> int launch_permute(dg::RowsParams p, dg_stream_t stream) {
    p.segments = (p.H + dg::PERMUTE_COLS - 1) / dg::PERMUTE_COLS;
    if (int rc = check_items(p.T * p.segments)) return rc;
    return launch("permute launch", dg::permute_kernel<T, FP8>, dim3(row_ctas(p.T * p.segments)),
                  dim3(32 * dg::ROWS_WARPS), 0, 1, stream, p);
}

template <typename T, bool FP8, int SLOTS> int launch_unpermute_backward(const dg::RowsParams &p, int sms, dg_stream_t stream) {
    // a warp a token from 8 tokens an SM on (e4m3, 4099 x 7168, top 8: 136 us, 155 with a CTA a token; 7725 x 1152, top 1: 18
    // and 32; but 600 x 2048, top 8: 14.4 and 11.0)
    if (p.T >= 8LL * sms)
        return launch("combine gradient launch", dg::unpermute_backward_kernel<T, FP8, SLOTS, true>, dim3(row_ctas(p.T)),
                      dim3(32 * dg::ROWS_WARPS), 0, 1, stream, p);
    const int steps = (p.H + dg::STEP - 1) / dg::STEP;
    const int iters = (steps + 7) / 8;
    int warps = (steps + iters - 1) / iters;
    warps = warps > dg::GRAD_MAX_WARPS ? dg::GRAD_MAX_WARPS : warps;
    return launch("combine gradient launch", dg::unpermute_backward_kernel<T, FP8, SLOTS, false>,
                  dim3(static_cast<unsigned>(p.T)), dim3(32 * warps), 0, 1, stream, p);
}

template <typename T, bool FP8> int launch_unpermute_backward(const dg::RowsParams &p, dg_stream_t stream) {
    int device, sms;
    if (int rc = current_device(device, sms)) return rc;
    if (p.k <= 2) return launch_unpermute_backward<T, FP8, 2>(p, sms, stream);
    return p.k <= 4 ? launch_unpermute_backward<T, FP8, 4>(p, sms, stream) : launch_unpermute_backward<T, FP8, 8>(p, sms, stream);
}

// -------------------------------------------------------------------------------------------------------- SwiGLU
template <typename T, bool FP8, bool BACKWARD> int launch_swiglu(dg::SwigluParams p, dg_stream_t stream) {
    constexpr int kRows = (BACKWARD ? 2 : 4) / (static_cast<int>(sizeof(T)) / 2);
    const int steps = (p.I + dg::STEP_COLS - 1) / dg::STEP_COLS;
    for (p.across = 1; p.across < dg::SWIGLU_WARPS && p.across < steps;) p.across *= 2;
    // two turns of the CTA's warps (I = 2048: 8 rows; 16 or 32 leave short calls too few CTAs, 4 are too short a life)
    p.cta_rows = 2 * kRows * dg::SWIGLU_WARPS / p.across;
    if (p.cta_rows > 32) p.cta_rows = 32;
    return launch("swiglu launch", dg::swiglu_kernel<T, FP8, BACKWARD, kRows>,
                  dim3((p.R + p.cta_rows - 1) / p.cta_rows, (steps + p.across - 1) / p.across), dim3(32 * dg::SWIGLU_WARPS), 0,
                  1, stream, p);
}

int swiglu_call(dg::SwigluParams p, int type, bool backward, const int *m_indices, const int *counts, const int *masked_m,
                float *out_sf, dg_stream_t stream) {
    if (p.R != 0 && (!p.gate_up || !p.out || (backward && !p.d_out))) return fail(DG_ERR_INVALID_ARG, "null pointer argument");
    if (!is_type(type)) return fail(DG_ERR_INVALID_ARG, "unknown element type %d", type);
    if (p.R < 0 || p.R > kMaxRows) return fail(DG_ERR_INVALID_ARG, "R=%d must be in [0, 2^30]", p.R);
    if (p.I <= 0 || p.I > (1 << 24)) return fail(DG_ERR_INVALID_ARG, "I=%d must be in [1, 2^24]", p.I);
    if (p.I % dg::VEC) return fail(DG_ERR_ALIGNMENT, "I=%d must be a multiple of %d", p.I, dg::VEC);
    if (out_sf && p.I % 128) return fail(DG_ERR_ALIGNMENT, "I=%d must be a multiple of 128 for an e4m3 output", p.I);
    if (!vec_aligned(p.gate_up, type) || !vec_aligned(p.out, out_sf ? DG_BF16 : type) ||
        !vec_aligned(p.d_out, type))
        return fail(DG_ERR_ALIGNMENT, "row operands must be 16-byte (fp32: 32-byte) aligned");
    if ((m_indices != nullptr) + (counts != nullptr) + (masked_m != nullptr) > 1)
        return fail(DG_ERR_INVALID_ARG, "at most one of m_indices, counts and masked_m may be given");
    p.own = m_indices ? m_indices : counts ? counts : masked_m;
    p.own_kind = m_indices ? dg::OWN_M_INDICES : counts ? dg::OWN_COUNTS : masked_m ? dg::OWN_MASKED : dg::OWN_ALL;
    if (!aligned(p.own, 4)) return fail(DG_ERR_ALIGNMENT, "m_indices, counts and masked_m must be 4-byte aligned");
    if ((counts || masked_m) && (p.G < 1 || p.G > dg::SORT_MAX_GROUPS))
        return fail(DG_ERR_INVALID_ARG, "G=%d must be in [1, %d]", p.G, dg::SORT_MAX_GROUPS);
    if (masked_m && p.R % p.G) return fail(DG_ERR_INVALID_ARG, "R=%d must be a multiple of G=%d", p.R, p.G);
    p.rows_per_group = masked_m && p.R > 0 ? p.R / p.G : p.R;
    if (int rc = scale_layout(p.sf, out_sf, p.R, p.rows_per_group, (backward ? 2 : 1) * p.I)) return rc;
    if (p.R == 0) return DG_OK;
    int device, sms;
    if (int rc = current_device(device, sms)) return rc;
    if (type == DG_BF16) {
        if (backward) return out_sf ? launch_swiglu<bf16, true, true>(p, stream) : launch_swiglu<bf16, false, true>(p, stream);
        return out_sf ? launch_swiglu<bf16, true, false>(p, stream) : launch_swiglu<bf16, false, false>(p, stream);
    }
    if (backward) return out_sf ? launch_swiglu<float, true, true>(p, stream) : launch_swiglu<float, false, true>(p, stream);
    return out_sf ? launch_swiglu<float, true, false>(p, stream) : launch_swiglu<float, false, false>(p, stream);
}

// --------------------------------------------------------------------------------------------------------- norms
int check_norm(const dg::NormParams &p, int x_type, int y_type, int param_type) {
    if (!is_type(x_type) || !is_type(y_type) || !is_type(param_type))
        return fail(DG_ERR_INVALID_ARG, "unknown element type (%d, %d, %d)", x_type, y_type, param_type);
    if (x_type == DG_BF16 && y_type == DG_F32)
        return fail(DG_ERR_UNSUPPORTED, "a bf16 residual stream takes bf16 block outputs and norms only");
    if (p.T < 0 || p.T > kMaxRows) return fail(DG_ERR_INVALID_ARG, "T=%d must be in [0, 2^30]", p.T);
    if (p.H <= 0) return fail(DG_ERR_INVALID_ARG, "H=%d must be positive", p.H);
    if (p.H > dg::NORM_MAX_H) return fail(DG_ERR_UNSUPPORTED, "H=%d exceeds %d", p.H, dg::NORM_MAX_H);
    if (p.H % dg::VEC) return fail(DG_ERR_ALIGNMENT, "H=%d must be a multiple of %d", p.H, dg::VEC);
    if (p.T != 0 && (p.gate_kind < dg::GATE_NONE || p.gate_kind > dg::GATE_TOKEN))
        return fail(DG_ERR_INVALID_ARG, "gate_kind must be 0 without a gate, 1 ([H]) or 2 ([T][H]) with one");
    const int gate_type = p.gate_kind == dg::GATE_ROW ? param_type : y_type;
    auto bad = [&](const void *q, int type) { return !vec_aligned(q, type); };
    if (bad(p.x, x_type) || bad(p.x_out, x_type) || bad(p.d_x_out, x_type) || bad(p.d_x, x_type) || bad(p.y, y_type) ||
        bad(p.d_h, y_type) || bad(p.d_y, y_type) || bad(p.d_gate_token, y_type) || bad(p.w, param_type) ||
        bad(p.w_post, param_type) || bad(p.gate, gate_type) || !vec_aligned(p.h, p.sf.sf ? DG_BF16 : y_type))
        return fail(DG_ERR_ALIGNMENT,
                    "tensors of the norms must be 16-byte (fp32: 32-byte) aligned");
    if (!aligned(p.rstd, 4) || !aligned(p.rstd_post, 4))
        return fail(DG_ERR_ALIGNMENT, "rstd and rstd_post must be 4-byte aligned");
    return DG_OK;
}

// -1 where the kind and the pointer do not go together (refused by check_norm).
int gate_of(const void *gate, int kind) {
    if (!gate) return kind == dg::GATE_NONE ? dg::GATE_NONE : -1;
    return kind == dg::GATE_ROW || kind == dg::GATE_TOKEN ? kind : -1;
}

// Launch of the kernels whose rows go through shared memory: CTAs of a vector a thread, as many an SM as `per_sm` and the
// shared memory allow, with up to four stages each.  More than four CTAs: one fewer where that gives a second stage (fp32, 512
// columns, y and a gate for each token: 168 us, 187 without); of up to four none is given up for it (fp32 stream with y and a gate
// [H], 4096 columns: 107 us, 154 with one CTA and more stages; 2048 columns: 102 and 112; but with bf16 and fp32 parameters 85
// and 80).
struct NormShape {
    int threads, ctas, stages;
    size_t smem;
};

NormShape norm_shape(const dg::NormParams &p, int stage_units, int per_sm, int sms) {
    NormShape s{};
    s.threads = (p.H / dg::VEC + 31) / 32 * 32;
    const int unit = 16 * s.threads, param_bytes = dg::norm_param_units(p.param_f32, p.gate_kind) * unit, stage_bytes = stage_units * unit;
    // (with NORM_CTA_BYTES left out, 32 CTAs an SM did not all fit, 128905 x 256 in fp32 98 us in place of 80)
    auto stages = [&](int n) { return (dg::NORM_SHARED_BYTES / n - dg::NORM_CTA_BYTES - param_bytes) / stage_bytes; };
    while (per_sm > 1 && stages(per_sm) < (per_sm > 4 ? 2 : 1)) --per_sm;
    s.ctas = p.T < per_sm * sms ? p.T : per_sm * sms;
    s.stages = stages(per_sm);
    const int rows = (p.T + s.ctas - 1) / s.ctas;  // (of a CTA: more stages would stay empty)
    s.stages = s.stages > dg::NORM_MAX_STAGES ? dg::NORM_MAX_STAGES : s.stages < 1 ? 1 : s.stages;
    s.stages = s.stages > rows ? rows : s.stages;
    s.smem = static_cast<size_t>(param_bytes) + static_cast<size_t>(s.stages) * stage_bytes;
    return s;
}

template <auto Kernel> int launch_norm_ring(const dg::NormParams &p, const NormShape &s, int device, dg_stream_t stream) {
    if (int rc = allow_shared<Kernel>(device, dg::NORM_SHARED_BYTES - dg::NORM_CTA_BYTES, "cudaFuncSetAttribute (norm)")) return rc;
    return launch("norm gradient launch", Kernel, dim3(s.ctas), dim3(s.threads), s.smem, 1, stream, p);
}

template <typename X, typename Y, bool FP8> int launch_norm(const dg::NormParams &p, int sms, dg_stream_t stream) {
    // 8 elements a thread while all rows' vectors fit on the SMs together (the call is then one row long); with many rows 32, so
    // that fewer warps take part in the sums, but 16 up to 16 times what fits, and with fp32 outputs, whose rows wait longer for
    // memory.  Residual norm with w_post and a gate [H] (rms_norm alone), us with 16 and with 32: bf16 8192 x 8192 109 and 95
    // (64, 48), 4000 x 4096 29 and 29 (16.5, 13.5), 1344 x 5888 17 and 20 (6.7, 6.5), 16000 x 1024 27 and 29 (18, 18); all
    // fp32 8192 x 8192 163 and 169, 1344 x 5888 25 and 31.
    const int vecs = p.H / dg::VEC;
    const long long vecs_per_sm = (p.T * static_cast<long long>(vecs) + sms - 1) / sms;
    const int iters = vecs > dg::NORM_MAX_THREADS                   ? 4
                      : vecs_per_sm <= 1024 || p.T <= sms           ? 1
                      : vecs_per_sm <= 16 * 1024 || sizeof(Y) == 4 ? 2 : 4;
    if (vecs > 64 || iters == 1) {
        auto kernel = iters == 1   ? dg::rms_norm_kernel<X, Y, FP8, 1, false>
                      : iters == 2 ? dg::rms_norm_kernel<X, Y, FP8, 2, false> : dg::rms_norm_kernel<X, Y, FP8, 4, false>;
        return launch("norm launch", kernel, dim3(static_cast<unsigned>(p.T)), dim3(((vecs + iters - 1) / iters + 31) / 32 * 32),
                      0, 1, stream, p);
    }
    // a row a warp: 16384 rows in bf16, rms_norm of 256 columns 3.9 us (17.5 with a row a CTA), of 512 6.0 (17.7); residual norm
    // with w_post and a gate [H] 6.1 (17.6) and 15.6 (20.3).  1024 columns gained 3% in bf16 and lost 9% to e4m3.
    auto kernel = vecs <= 32 ? dg::rms_norm_kernel<X, Y, FP8, 1, true> : dg::rms_norm_kernel<X, Y, FP8, 2, true>;
    return launch("norm launch", kernel, dim3((p.T + dg::NORM_ROW_WARPS - 1) / dg::NORM_ROW_WARPS),
                  dim3(32 * dg::NORM_ROW_WARPS), 0, 1, stream, p);
}
template <typename X, typename Y> int launch_norm(const dg::NormParams &p, int sms, dg_stream_t stream) {
    return p.sf.sf ? launch_norm<X, Y, true>(p, sms, stream) : launch_norm<X, Y, false>(p, sms, stream);
}

int norm_call(const dg::NormParams &p, int x_type, int y_type, int param_type, dg_stream_t stream) {
    if (int rc = check_norm(p, x_type, y_type, param_type)) return rc;
    if (p.T == 0) return DG_OK;
    int device, sms;
    if (int rc = current_device(device, sms)) return rc;
    if (x_type == DG_BF16) return launch_norm<bf16, bf16>(p, sms, stream);
    return y_type == DG_BF16 ? launch_norm<float, bf16>(p, sms, stream) : launch_norm<float, float>(p, sms, stream);
}

// (wide rows: one CTA an SM)
template <typename X, typename Y> NormShape norm_backward_shape(const dg::NormParams &p, int sms) {
    if (p.H > dg::NORM_RING_H) return NormShape{dg::NORM_WIDE_THREADS, p.T < sms ? p.T : sms, 0, 0};
    const int units = dg::norm_stage_units(dg::Raw<X>::UNITS, dg::Raw<Y>::UNITS, p.w != nullptr, p.y != nullptr,
                                           p.gate_kind == dg::GATE_TOKEN);
    const int threads = (p.H / dg::VEC + 31) / 32 * 32;
    const int per_sm = dg::NORM_MAX_THREADS / threads;  // (at 64 registers)
    return norm_shape(p, units, per_sm, sms);
}

template <typename X, typename Y>
int launch_norm_backward(const dg::NormParams &p, const NormShape &s, int device, dg_stream_t stream) {
    if (p.H > dg::NORM_RING_H)
        return launch("norm gradient launch", dg::rms_norm_backward_wide_kernel<X, Y, 4>, dim3(s.ctas), dim3(s.threads), 0, 1,
                      stream, p);
    if (!p.y) return launch_norm_ring<dg::rms_norm_backward_kernel<X, Y, dg::GATE_NONE, false>>(p, s, device, stream);
    if (p.gate_kind == dg::GATE_NONE)
        return launch_norm_ring<dg::rms_norm_backward_kernel<X, Y, dg::GATE_NONE, true>>(p, s, device, stream);
    if (p.gate_kind == dg::GATE_ROW)
        return launch_norm_ring<dg::rms_norm_backward_kernel<X, Y, dg::GATE_ROW, true>>(p, s, device, stream);
    return launch_norm_ring<dg::rms_norm_backward_kernel<X, Y, dg::GATE_TOKEN, true>>(p, s, device, stream);
}

int norm_backward_call(dg::NormParams p, int x_type, int y_type, int param_type, float *d_w, float *d_w_post,
                       float *d_gate_row, dg_stream_t stream) {
    if (int rc = check_norm(p, x_type, y_type, param_type)) return rc;
    for (const float *q : {d_w, d_w_post, d_gate_row})
        if (!aligned(q, 4)) return fail(DG_ERR_ALIGNMENT, "parameter gradients must be 4-byte aligned");
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (p.T == 0) {  // sums over no rows
        for (float *q : {d_w, d_w_post, d_gate_row})
            if (q && (e = cudaMemsetAsync(q, 0, sizeof(float) * p.H, s)) != cudaSuccess)
                return cuda_fail(e, "cudaMemsetAsync (parameter gradients)");
        return DG_OK;
    }
    int device, sms;
    if (int rc = current_device(device, sms)) return rc;
    const NormShape shape = x_type == DG_BF16   ? norm_backward_shape<bf16, bf16>(p, sms)
                            : y_type == DG_BF16 ? norm_backward_shape<float, bf16>(p, sms)
                                                : norm_backward_shape<float, float>(p, sms);
    const int ctas = shape.ctas;
    p.stages = shape.stages;
    cudaMemPool_t pool;
    if (int rc = scratch_pool(device, pool)) return rc;
    void *partial = nullptr;
    e = cudaMallocFromPoolAsync(&partial, sizeof(float) * 3 * p.H * static_cast<size_t>(ctas), pool, s);
    if (e != cudaSuccess) return cuda_fail(e, "cudaMallocFromPoolAsync (parameter gradients)");
    p.partial = static_cast<float *>(partial);
    int rc = x_type == DG_BF16   ? launch_norm_backward<bf16, bf16>(p, shape, device, stream)
             : y_type == DG_BF16 ? launch_norm_backward<float, bf16>(p, shape, device, stream)
                                 : launch_norm_backward<float, float>(p, shape, device, stream);
    if (rc == DG_OK && (d_w || d_w_post || d_gate_row)) {
        // columns of a CTA: 64, or 16 for short rows, whose sums would be the work of a few SMs (1184 partial sums of 288: 11 us)
        const bool narrow = p.H <= 2048;
        const int cols = narrow ? 16 : 64;
        rc = launch("norm gradient sum launch", narrow ? dg::rms_norm_sum_kernel<4> : dg::rms_norm_sum_kernel<16>,
                    dim3((p.H + cols - 1) / cols, 3), dim3(dg::NORM_SUM_THREADS), 0, 1, stream,
                    static_cast<const float *>(p.partial), ctas, p.H, d_w, d_w_post, d_gate_row);
    }
    e = cudaFreeAsync(partial, s);
    if (rc == DG_OK && e != cudaSuccess) rc = cuda_fail(e, "cudaFreeAsync (parameter gradients)");
    return rc;
}

}  // namespace

extern "C" {

long long dg_moe_m_total_bound(long long num_slots, int G) {
    if (num_slots < 0 || G < 1) return fail(DG_ERR_INVALID_ARG, "num_slots=%lld and G=%d are out of range", num_slots, G);
    const long long a = dg_get_m_alignment_for_contiguous_layout();
    return (num_slots + (num_slots < G ? num_slots : G) * (a - 1)) / a * a;
}

int dg_moe_sort_contiguous(const void *topk_ids, int id_bytes, int T, int k, int G, int M_total, int *row_of_slot,
                           int *m_indices, int *counts, dg_stream_t stream) {
    if (int rc = check_sort(topk_ids, id_bytes, T, k, G, row_of_slot, counts)) return rc;
    if (!m_indices && M_total > 0) return fail(DG_ERR_INVALID_ARG, "m_indices is null");
    if (!aligned(m_indices, 16)) return fail(DG_ERR_ALIGNMENT, "m_indices must be 16-byte aligned");
    const int a = dg_get_m_alignment_for_contiguous_layout();
    if (M_total < 0 || M_total > kMaxRows) return fail(DG_ERR_INVALID_ARG, "M_total=%d must be in [0, 2^30]", M_total);
    if (M_total % a) return fail(DG_ERR_ALIGNMENT, "M_total=%d must be a multiple of %d", M_total, a);
    dg::SortParams p{};
    p.ids = topk_ids;
    p.G = G;
    p.layout = dg::SORT_CONTIGUOUS;
    p.align = a;
    p.M_total = M_total;
    p.row_of_slot = row_of_slot;
    p.m_indices = m_indices;
    p.counts = counts;
    return sort_call(p, id_bytes, T, k, stream);
}

int dg_moe_sort_nopad(const void *topk_ids, int id_bytes, int T, int k, int G, int *row_of_slot, int *counts,
                      dg_stream_t stream) {
    if (int rc = check_sort(topk_ids, id_bytes, T, k, G, row_of_slot, counts)) return rc;
    dg::SortParams p{};
    p.ids = topk_ids;
    p.G = G;
    p.layout = dg::SORT_NOPAD;
    p.row_of_slot = row_of_slot;
    p.counts = counts;
    return sort_call(p, id_bytes, T, k, stream);
}

int dg_moe_sort_masked(const void *topk_ids, int id_bytes, int T, int k, int G, int M_max, int *row_of_slot, int *masked_m,
                       dg_stream_t stream) {
    if (int rc = check_sort(topk_ids, id_bytes, T, k, G, row_of_slot, masked_m)) return rc;
    if (M_max < 1 || static_cast<long long>(G) * M_max > kMaxRows)
        return fail(DG_ERR_INVALID_ARG, "M_max=%d must be positive and G*M_max at most 2^30", M_max);
    dg::SortParams p{};
    p.ids = topk_ids;
    p.G = G;
    p.layout = dg::SORT_MASKED;
    p.M_max = M_max;
    p.row_of_slot = row_of_slot;
    p.counts = masked_m;
    return sort_call(p, id_bytes, T, k, stream);
}

int dg_moe_permute(const void *x, int type, const int *row_of_slot, int T, int k, int H, int rows, int rows_per_group,
                   void *out, float *out_sf, dg_stream_t stream) {
    dg::RowsParams p{};
    if (rows == 0) T = 0;  // nowhere to write
    if (int rc = check_rows(x, row_of_slot, out, out_sf, type, T, k, H, rows)) return rc;
    if (int rc = scale_layout(p.sf, out_sf, rows, rows_per_group, H)) return rc;
    if (T == 0) return DG_OK;
    if (int rc = rows_params(p, x, row_of_slot, T, k, H, rows, out)) return rc;
    if (type == DG_BF16) return out_sf ? launch_permute<bf16, true>(p, stream) : launch_permute<bf16, false>(p, stream);
    return out_sf ? launch_permute<float, true>(p, stream) : launch_permute<float, false>(p, stream);
}

int dg_moe_unpermute(const void *rows_in, int type, const int *row_of_slot, const float *weights, int T, int k, int H,
                     int rows, void *out, dg_stream_t stream) {
    dg::RowsParams p{};
    if (rows == 0) rows_in = out;  // (no row is read)
    if (int rc = check_rows(rows_in, row_of_slot, out, nullptr, type, T, k, H, rows)) return rc;
    if (!aligned(weights, 4)) return fail(DG_ERR_ALIGNMENT, "weights must be 4-byte aligned");
    if (T == 0) return DG_OK;
    if (int rc = rows_params(p, rows_in, row_of_slot, T, k, H, rows, out)) return rc;
    p.weights = weights;
    p.segments = (H + dg::STEP - 1) / dg::STEP;
    if (int rc = check_items(p.T * p.segments)) return rc;
    const dim3 grid(row_ctas(p.T * p.segments)), block(32 * dg::ROWS_WARPS);
    if (type == DG_BF16) return launch("combine launch", dg::unpermute_kernel<bf16, 8>, grid, block, 0, 1, stream, p);
    return launch("combine launch", dg::unpermute_kernel<float, 4>, grid, block, 0, 1, stream, p);
}

int dg_moe_unpermute_backward(const void *d_out, const void *rows_in, int type, const int *row_of_slot,
                              const float *weights, int T, int k, int H, int rows, int rows_per_group, void *d_rows,
                              float *d_rows_sf, float *d_weights, dg_stream_t stream) {
    dg::RowsParams p{};
    if (rows == 0) rows_in = d_rows = const_cast<void *>(d_out);  // (no row is read or written)
    if (int rc = check_rows(rows_in, row_of_slot, d_rows, d_rows_sf, type, T, k, H, rows)) return rc;
    if (T > 0 && (!d_out || !weights || !d_weights)) return fail(DG_ERR_INVALID_ARG, "null pointer argument");
    if (!vec_aligned(d_out, type)) return fail(DG_ERR_ALIGNMENT, "row operands must be 16-byte (fp32: 32-byte) aligned");
    if (!aligned(weights, 4) || !aligned(d_weights, 4))
        return fail(DG_ERR_ALIGNMENT, "weights and d_weights must be 4-byte aligned");
    if (int rc = scale_layout(p.sf, d_rows_sf, rows, rows_per_group, H)) return rc;
    if (T == 0) return DG_OK;
    if (int rc = rows_params(p, rows_in, row_of_slot, T, k, H, rows, d_rows)) return rc;
    p.d_out = d_out;
    p.weights = weights;
    p.d_weights = d_weights;
    if (type == DG_BF16)
        return d_rows_sf ? launch_unpermute_backward<bf16, true>(p, stream) : launch_unpermute_backward<bf16, false>(p, stream);
    return d_rows_sf ? launch_unpermute_backward<float, true>(p, stream) : launch_unpermute_backward<float, false>(p, stream);
}

int dg_swiglu(const void *gate_up, int type, int R, int I, const int *m_indices, const int *counts, const int *masked_m,
              int G, void *out, float *out_sf, dg_stream_t stream) {
    dg::SwigluParams p{};
    p.gate_up = gate_up;
    p.out = out;
    p.G = G;
    p.R = R;
    p.I = I;
    return swiglu_call(p, type, false, m_indices, counts, masked_m, out_sf, stream);
}

int dg_swiglu_backward(const void *d_out, const void *gate_up, int type, int R, int I, const int *m_indices,
                       const int *counts, const int *masked_m, int G, void *d_gate_up, float *d_gate_up_sf,
                       dg_stream_t stream) {
    dg::SwigluParams p{};
    p.gate_up = gate_up;
    p.d_out = d_out;
    p.out = d_gate_up;
    p.G = G;
    p.R = R;
    p.I = I;
    return swiglu_call(p, type, true, m_indices, counts, masked_m, d_gate_up_sf, stream);
}

int dg_residual_rms_norm(const void *x, int x_type, const void *y, int y_type, const void *weight, const void *weight_post,
                         const void *gate, int gate_kind, int param_type, float alpha, float eps, int T, int H, void *x_out,
                         void *out, float *out_sf, float *rstd, float *rstd_post, dg_stream_t stream) {
    dg::NormParams p{};
    if (T != 0 && (!x || !y || !x_out)) return fail(DG_ERR_INVALID_ARG, "null pointer argument");
    if (T != 0 && (weight != nullptr) != (out != nullptr)) return fail(DG_ERR_INVALID_ARG, "weight and out go together");
    if (T != 0 && out_sf && !out) return fail(DG_ERR_INVALID_ARG, "scales without an output");
    if (rstd && !weight) return fail(DG_ERR_INVALID_ARG, "rstd without weight");
    if (rstd_post && !weight_post) return fail(DG_ERR_INVALID_ARG, "rstd_post without weight_post");
    if (int rc = scale_layout(p.sf, out_sf, T, T, H)) return rc;
    p.x = x;
    p.y = y;
    p.w = weight;
    p.w_post = weight_post;
    p.gate = gate;
    p.gate_kind = gate_of(gate, gate_kind);
    p.x_out = x_out;
    p.h = out;
    p.rstd = rstd;
    p.rstd_post = rstd_post;
    p.alpha = alpha;
    p.eps = eps;
    p.T = T;
    p.H = H;
    p.param_f32 = param_type == DG_F32;
    return norm_call(p, x_type, y_type, param_type, stream);
}

int dg_rms_norm(const void *x, int x_type, const void *weight, int param_type, float eps, int T, int H, void *out,
                int out_type, float *out_sf, float *rstd, dg_stream_t stream) {
    dg::NormParams p{};
    if (!weight || (T != 0 && (!x || !out))) return fail(DG_ERR_INVALID_ARG, "null pointer argument");
    if (int rc = scale_layout(p.sf, out_sf, T, T, H)) return rc;
    p.x = x;
    p.w = weight;
    p.h = out;
    p.rstd = rstd;
    p.eps = eps;
    p.T = T;
    p.H = H;
    p.param_f32 = param_type == DG_F32;
    return norm_call(p, x_type, out_type, param_type, stream);
}

int dg_residual_rms_norm_backward(const void *d_x_out, const void *d_out, const void *x_out, int x_type, const void *y,
                                  int y_type, const void *weight, const void *weight_post, const void *gate, int gate_kind,
                                  int param_type, float alpha, const float *rstd, const float *rstd_post, int T, int H,
                                  void *d_x, void *d_y, float *d_weight, float *d_weight_post, void *d_gate,
                                  dg_stream_t stream) {
    dg::NormParams p{};
    if (T != 0 && (!y || !d_x || !d_y)) return fail(DG_ERR_INVALID_ARG, "null pointer argument");
    if (weight && (!d_weight || (T != 0 && (!d_out || !x_out || !rstd))))
        return fail(DG_ERR_INVALID_ARG, "weight needs d_out, x_out, rstd and d_weight");
    if (!weight && (d_out || d_weight)) return fail(DG_ERR_INVALID_ARG, "d_out and d_weight need weight");
    if (weight_post && (!d_weight_post || (T != 0 && !rstd_post)))
        return fail(DG_ERR_INVALID_ARG, "weight_post needs rstd_post and d_weight_post");
    if (!weight_post && d_weight_post) return fail(DG_ERR_INVALID_ARG, "d_weight_post needs weight_post");
    if (T != 0 && (gate != nullptr) != (d_gate != nullptr)) return fail(DG_ERR_INVALID_ARG, "gate and d_gate go together");
    if (T != 0 && !d_x_out && !weight) return fail(DG_ERR_INVALID_ARG, "no gradient comes in: give d_x_out or weight and d_out");
    p.x = x_out;
    p.y = y;
    p.w = weight;
    p.w_post = weight_post;
    p.gate = gate;
    p.gate_kind = gate_of(gate, gate_kind);
    p.rstd = const_cast<float *>(rstd);
    p.rstd_post = const_cast<float *>(rstd_post);
    p.d_x_out = d_x_out;
    p.d_h = d_out;
    p.d_x = d_x;
    p.d_y = d_y;
    p.d_gate_token = p.gate_kind == dg::GATE_TOKEN ? d_gate : nullptr;
    p.alpha = alpha;
    p.T = T;
    p.H = H;
    p.param_f32 = param_type == DG_F32;
    return norm_backward_call(p, x_type, y_type, param_type, d_weight, d_weight_post,
                              p.gate_kind == dg::GATE_ROW ? static_cast<float *>(d_gate) : nullptr, stream);
}

int dg_rms_norm_backward(const void *d_out, const void *d_skip, const void *x, int x_type, int out_type, const void *weight,
                         int param_type, const float *rstd, int T, int H, void *d_x, float *d_weight, dg_stream_t stream) {
    dg::NormParams p{};
    if (!weight || !d_weight || (T != 0 && (!d_out || !x || !rstd || !d_x))) return fail(DG_ERR_INVALID_ARG, "null pointer argument");
    p.x = x;
    p.w = weight;
    p.rstd = const_cast<float *>(rstd);
    p.d_x_out = d_skip;
    p.d_h = d_out;
    p.d_x = d_x;
    p.T = T;
    p.H = H;
    p.param_f32 = param_type == DG_F32;
    return norm_backward_call(p, x_type, out_type, param_type, d_weight, nullptr, nullptr, stream);
}

}  // extern "C"
