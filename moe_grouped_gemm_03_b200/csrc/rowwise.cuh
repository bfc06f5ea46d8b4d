// Building blocks of the row-wise operators (dispatch, combine, SwiGLU, norms): 8-element vectors in fp32, and the
// quantisation of a block of 128 values to e4m3 with a power-of-two scale.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"

namespace dg {

using bf16 = __nv_bfloat16;
constexpr int VEC = 8;  // elements a lane handles at a time: 16 bytes of bf16
constexpr int BLOCK_LANES = 128 / VEC;  // lanes that hold one block of 128 (half a warp)
constexpr unsigned ERR_WORD_BAD_GROUP = 2u;    // device error word of DG_ERR_BAD_GROUP

__device__ __forceinline__ void raise_bad_group(unsigned *err) { atomicCAS(err, 0u, ERR_WORD_BAD_GROUP); }

__device__ __forceinline__ void unpack_bf16x2(uint32_t w, float &lo, float &hi) {
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xffff0000u);
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Asynchronous copies of 16 bytes to shared memory, past L1, waited for in groups by the thread that made them.
__device__ __forceinline__ void copy_async16(void *s, const void *p) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(s)), "l"(p) : "memory");
}
// (through L1: what several CTAs of an SM read)
__device__ __forceinline__ void copy_async16_ca(void *s, const void *p) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(smem_u32(s)), "l"(p) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_async_wait() {  // until at most N groups are under way
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Loads are ordinary ones, not the non-coherent kind (__ldg): a kernel here may start before the one that writes its
// inputs has ended, and memory that changes during a kernel's life is not for that path.

// One lane's vector of eight elements as it lies in memory, at a multiple of its size (at most 32 bytes).  Loads and stores of
// 32 bytes are single 256-bit accesses: as two of 128 bits, half of each request's sectors went unused.
__device__ __forceinline__ void load256(uint32_t (&w)[8], const void *p) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
}
__device__ __forceinline__ void store256(void *p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

template <typename T> struct Raw;
template <> struct Raw<bf16> {
    uint4 a;
    __device__ __forceinline__ void load(const bf16 *p) { a = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void store(bf16 *p) const { *reinterpret_cast<uint4 *>(p) = a; }
    static constexpr int UNITS = 1;  // of 16 bytes
    __device__ __forceinline__ void get(float (&v)[VEC]) const {
        unpack_bf16x2(a.x, v[0], v[1]);
        unpack_bf16x2(a.y, v[2], v[3]);
        unpack_bf16x2(a.z, v[4], v[5]);
        unpack_bf16x2(a.w, v[6], v[7]);
    }
    __device__ __forceinline__ void set(const float (&v)[VEC]) {  // round to nearest even
        a = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                       pack_bf16x2(v[6], v[7]));
    }
};
template <> struct Raw<float> {
    uint32_t w[VEC];
    __device__ __forceinline__ void load(const float *p) { load256(w, p); }
    __device__ __forceinline__ void store(float *p) const { store256(p, w); }
    static constexpr int UNITS = 2;
    __device__ __forceinline__ void get(float (&v)[VEC]) const {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = __uint_as_float(w[i]);
    }
    __device__ __forceinline__ void set(const float (&v)[VEC]) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) w[i] = __float_as_uint(v[i]);
    }
};

template <typename T> __device__ __forceinline__ void load_vec(const T *p, float (&v)[VEC]) {
    Raw<T> r;
    r.load(p);
    r.get(v);
}
template <typename T> __device__ __forceinline__ void store_vec(T *p, const float (&v)[VEC]) {
    Raw<T> r;
    r.set(v);
    r.store(p);
}

// Two fp32 operations an instruction, on the pairs of a vector (the kernels here run out of issue slots before they run out
// of arithmetic): a *= b, a *= s, a += b * c, a = a * s + b.
__device__ __forceinline__ void mul2(float &a0, float &a1, float b0, float b1) {
    asm("{.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\tmul.rn.f32x2 a, a, b;\n\t"
        "mov.b64 {%0, %1}, a;}"
        : "+f"(a0), "+f"(a1)
        : "f"(b0), "f"(b1));
}
__device__ __forceinline__ void fma2(float &c0, float &c1, float a0, float a1, float b0, float b1) {  // c += a * b
    asm("{.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%0, %1};\n\t"
        "fma.rn.f32x2 c, a, b, c;\n\tmov.b64 {%0, %1}, c;}"
        : "+f"(c0), "+f"(c1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void mul_vec(float (&a)[VEC], const float (&b)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; i += 2) mul2(a[i], a[i + 1], b[i], b[i + 1]);
}
__device__ __forceinline__ void mul_vec(float (&a)[VEC], float s) {
#pragma unroll
    for (int i = 0; i < VEC; i += 2) mul2(a[i], a[i + 1], s, s);
}
__device__ __forceinline__ void fma_vec(float (&c)[VEC], const float (&a)[VEC], const float (&b)[VEC]) {  // c += a * b
#pragma unroll
    for (int i = 0; i < VEC; i += 2) fma2(c[i], c[i + 1], a[i], a[i + 1], b[i], b[i + 1]);
}
__device__ __forceinline__ void fma_vec(float (&c)[VEC], const float (&a)[VEC], float s) {  // c += a * s
#pragma unroll
    for (int i = 0; i < VEC; i += 2) fma2(c[i], c[i + 1], a[i], a[i + 1], s, s);
}
__device__ __forceinline__ void one_plus_times(float (&a)[VEC], float s) {  // a = (1 + a) * s for a power of two s
#pragma unroll
    for (int i = 0; i < VEC; i += 2)
        asm("{.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %2};\n\tfma.rn.f32x2 a, a, b, b;\n\t"
            "mov.b64 {%0, %1}, a;}"
            : "+f"(a[i]), "+f"(a[i + 1])
            : "f"(s));
}
// Sum of products of a vector, onto a pair of partial sums.
__device__ __forceinline__ void dot_vec(float (&sum)[2], const float (&a)[VEC], const float (&b)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; i += 2) fma2(sum[0], sum[1], a[i], a[i + 1], b[i], b[i + 1]);
}

__device__ __forceinline__ float absmax3(float a, float b, float c) {  // NaN is passed over
    float m;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {  // a in the lowest byte
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

__device__ __forceinline__ float vec_amax(const float (&v)[VEC]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < VEC; i += 2) m = absmax3(m, v[i], v[i + 1]);
    return m;
}

// Largest |v| of a block of 128 over its 16 lanes; NaN is passed over, an infinity gives infinity.  A warp's lanes hold 256
// columns from a multiple of 256 on, `col` is the calling lane's; those at or past `width`, a multiple of 128, do not call.
// Each half's largest by one reduction over the warp, in the order of the bits since no sign is set: against four shuffles the
// contiguous SwiGLU takes 108 us (112), its gradient of 23424 x 1536 68 (72), the norm of 8192 x 7168 110.5 (113).
__device__ __forceinline__ float block_amax(const float (&v)[VEC], int col, int width) {
    const unsigned lanes = (col & ~(32 * VEC - 1)) + 128 < width ? 0xffffffffu : 0xffffu;
    const uint32_t m = __float_as_uint(vec_amax(v));
    const bool upper = threadIdx.x & BLOCK_LANES;
    const uint32_t lo = __reduce_max_sync(lanes, upper ? 0u : m), hi = __reduce_max_sync(lanes, upper ? m : 0u);
    return __uint_as_float(upper ? hi : lo);
}

// Quantises one lane's values of a block whose largest |v| is `amax` (the same in the block's lanes, which all call this).
// scale = 2^ceil(log2(amax / 448)), the smallest power of two that brings every value within e4m3's +-448 (at least
// 2^-126; 1 for a block of zeros); codes = e4m3 RNE(v / scale), where the division is an exact multiplication by the
// inverse power.  A value that is not finite gets e4m3's NaN code, and the scale goes by the block's finite values, so that
// it does not flatten its neighbours.
__device__ __forceinline__ uint2 quantise(float (&v)[VEC], float amax, float &scale) {
    if (__builtin_expect(!(amax < __int_as_float(0x7f800000)), 0)) {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (!(fabsf(v[i]) < __int_as_float(0x7f800000))) v[i] = __int_as_float(0x7fffffff);
        amax = vec_amax(v);
        const unsigned lanes = 0xffffu << (threadIdx.x & BLOCK_LANES);  // (the other half of the warp may not come here)
#pragma unroll
        for (int d = BLOCK_LANES / 2; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(lanes, amax, d));
    }
    // 448 = 1.75 * 2^8: adding 2^23 - 1 - 0.75 * 2^23 to the bits carries into the exponent where the mantissa is
    // above 1.75
    int e = static_cast<int>((__float_as_uint(amax) + 0x1fffffu) >> 23) - 8;
    e = amax == 0.f ? 127 : max(e, 1);
    scale = __uint_as_float(static_cast<uint32_t>(e) << 23);
    mul_vec(v, __uint_as_float(static_cast<uint32_t>(254 - e) << 23));  // (e <= 247)
    return make_uint2(e4m3x4(v[0], v[1], v[2], v[3]), e4m3x4(v[4], v[5], v[6], v[7]));
}

// Scales of an e4m3 operand, MN-major: [groups][cols / 128][ld], rows_per_group rows in each group.
struct ScaleLayout {
    float *sf;
    int rows_per_group, ld, blocks;  // blocks = cols / 128
    __device__ __forceinline__ float *at(int row, int block) const {
        const int g = row / rows_per_group;
        return sf + (static_cast<long long>(g) * blocks + block) * ld + (row - g * rows_per_group);
    }
};

}  // namespace dg
