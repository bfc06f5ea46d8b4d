// Building blocks of the row-wise operators (dispatch, combine, SwiGLU, norms): 8-element vectors in fp32, and the
// quantisation of a block of 128 values to e4m3 with a power-of-two scale.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"

namespace dg {

using bf16 = __nv_bfloat16;
constexpr int VEC = 8;                         // elements a lane handles at a time: 16 bytes of bf16
constexpr int BLOCK_LANES = 128 / VEC;         // lanes that hold one block of 128 (half a warp)
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

// Loads are ordinary ones, not the non-coherent kind (__ldg): a kernel here may start before the one that writes its
// inputs has ended, and memory that changes during a kernel's life is not for that path.

// One lane's vector of eight elements as it lies in memory (bf16: 16 bytes, fp32: 32 bytes, each at a multiple of that).
template <typename T> struct Raw8;
template <> struct Raw8<bf16> {
    uint4 a;
    __device__ __forceinline__ void load(const bf16 *p) { a = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void store(bf16 *p) const { *reinterpret_cast<uint4 *>(p) = a; }
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
template <> struct Raw8<float> {  // one 256-bit access: as two of 128 bits, half of each request's sectors went unused
    float v8[VEC];
    __device__ __forceinline__ void load(const float *p) {
        asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=f"(v8[0]), "=f"(v8[1]), "=f"(v8[2]), "=f"(v8[3]), "=f"(v8[4]), "=f"(v8[5]), "=f"(v8[6]), "=f"(v8[7])
                     : "l"(p));
    }
    __device__ __forceinline__ void store(float *p) const {
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v8[0]), "f"(v8[1]), "f"(v8[2]),
                     "f"(v8[3]), "f"(v8[4]), "f"(v8[5]), "f"(v8[6]), "f"(v8[7])
                     : "memory");
    }
    __device__ __forceinline__ void get(float (&v)[VEC]) const {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = v8[i];
    }
    __device__ __forceinline__ void set(const float (&v)[VEC]) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v8[i] = v[i];
    }
};

template <typename T> __device__ __forceinline__ void load8(const T *p, float (&v)[VEC]) {
    Raw8<T> r;
    r.load(p);
    r.get(v);
}
template <typename T> __device__ __forceinline__ void store8(T *p, const float (&v)[VEC]) {
    Raw8<T> r;
    r.set(v);
    r.store(p);
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {  // a in the lowest byte
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// Largest |v| of a block of 128 over its 16 lanes; NaN is passed over, an infinity gives infinity.
__device__ __forceinline__ float block_amax(const float (&v)[VEC]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) m = fmaxf(m, fabsf(v[i]));
    const unsigned lanes = 0xffffu << (threadIdx.x & 16);
#pragma unroll
    for (int d = BLOCK_LANES / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(lanes, m, d));
    return m;
}

// Quantises one lane's eight values of a block whose largest |v| is `amax` (the same in the block's 16 lanes, which
// all call this).  scale = 2^ceil(log2(amax / 448)), the smallest power of two that brings every value within e4m3's
// +-448 (at least 2^-126; 1 for a block of zeros); codes = e4m3 RNE(v / scale), where the division is an exact
// multiplication by the inverse power.  A value that is not finite gets e4m3's NaN code, and the scale goes by the
// block's finite values, so that it does not flatten its neighbours.
__device__ __forceinline__ uint2 quantise8(float (&v)[VEC], float amax, float &scale) {
    if (__builtin_expect(!(amax < __int_as_float(0x7f800000)), 0)) {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (!(fabsf(v[i]) < __int_as_float(0x7f800000))) v[i] = __int_as_float(0x7fffffff);
        amax = block_amax(v);
    }
    // 448 = 1.75 * 2^8: adding 2^23 - 1 - 0.75 * 2^23 to the bits carries into the exponent where the mantissa is
    // above 1.75
    int e = static_cast<int>((__float_as_uint(amax) + 0x1fffffu) >> 23) - 8;
    e = amax == 0.f ? 127 : max(e, 1);
    scale = __uint_as_float(static_cast<uint32_t>(e) << 23);
    const float inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);  // (e <= 247)
    return make_uint2(e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                      e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
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
