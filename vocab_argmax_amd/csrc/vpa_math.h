// vpa_math.h -- device helpers of the head's operators: element conversion,
// base-2 exponentials, and sums over a wavefront or workgroup.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "vpa_device.h"

namespace vpa {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Element types by size: bf16 is a uint16_t pattern in memory.
template <int ESIZE>
struct elem;
template <>
struct elem<2> {
    using type = uint16_t;
};
template <>
struct elem<4> {
    using type = float;
};

__device__ __forceinline__ float to_f32(uint16_t h) {
    return __builtin_bit_cast(float, (uint32_t)h << 16);
}
__device__ __forceinline__ float to_f32(float f) {
    return f;
}
// fp32 to bf16, round to nearest even (NaN stays NaN).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const f32x2 f = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
}
__device__ __forceinline__ void from_f32(uint16_t& d, float f) {
    d = __builtin_bit_cast(uint16_t, (__bf16)f);
}
__device__ __forceinline__ void from_f32(float& d, float f) {
    d = f;
}

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

// 16 bytes at any element address: global memory takes such accesses at every
// alignment of the element.
struct __attribute__((packed, aligned(2))) Loose16 {
    u32x4_t v;
};

// Element e of a 16-byte vector as fp32.
template <int ESIZE>
__device__ __forceinline__ float vec_elem(u32x4_t v, int e) {
    if constexpr (ESIZE == 4)
        return __builtin_bit_cast(float, (uint32_t)v[e]);
    const uint32_t w = v[e / 2];
    return __builtin_bit_cast(float, e % 2 ? w & 0xFFFF0000u : w << 16);
}

// 2^x by the hardware instruction: within 1 ulp, results below 2^-126 are 0.
__device__ __forceinline__ float exp2_fast(float x) {
    return __builtin_amdgcn_exp2f(x);
}

// Sum over the 64 lanes of a wavefront by lane moves (vpa_device.h); every
// lane holds the result.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ float add_move(float v) {
    return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                                             0, __builtin_bit_cast(int, v), CTRL, ROW_MASK, 0xF,
                                             false));
}
__device__ __forceinline__ float wave_sum(float v) {
    v = add_move<dpp::kSwap1, 0xF>(v);
    v = add_move<dpp::kSwap2, 0xF>(v);
    v = add_move<dpp::kHalfMirror, 0xF>(v);
    v = add_move<dpp::kMirror, 0xF>(v);
    v = add_move<dpp::kBcast15, 0xA>(v);
    v = add_move<dpp::kBcast31, 0xC>(v);
    return __builtin_bit_cast(float,
                              __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}
// The maximum, alike; a NaN counts as nothing.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ float max_move(float v) {
    const int i = __builtin_bit_cast(int, v);
    return fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(i, i, CTRL, ROW_MASK, 0xF,
                                                                          false)));
}
__device__ __forceinline__ float wave_max(float v) {
    v = max_move<dpp::kSwap1, 0xF>(v);
    v = max_move<dpp::kSwap2, 0xF>(v);
    v = max_move<dpp::kHalfMirror, 0xF>(v);
    v = max_move<dpp::kMirror, 0xF>(v);
    v = max_move<dpp::kBcast15, 0xA>(v);
    v = max_move<dpp::kBcast31, 0xC>(v);
    return __builtin_bit_cast(float,
                              __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// Two sums over a workgroup of WAVES wavefronts through `lds`; every thread
// holds the results.  Callers leave a barrier between two uses of an lds.
template <int WAVES>
__device__ __forceinline__ void block_sum2(float& a, float& b, float (&lds)[WAVES][2]) {
    a = wave_sum(a);
    b = wave_sum(b);
    if constexpr (WAVES > 1) {
        if ((threadIdx.x & 63) == 0) {
            lds[threadIdx.x >> 6][0] = a;
            lds[threadIdx.x >> 6][1] = b;
        }
        __syncthreads();
        a = b = 0.0f;
#pragma unroll
        for (int i = 0; i < WAVES; ++i) {
            a += lds[i][0];
            b += lds[i][1];
        }
    }
}

}  // namespace vpa
