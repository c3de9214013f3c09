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
struct elem<1> {
    using type = uint8_t;             // e4m3 patterns
};
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

// Sums over a wavefront in 64 bits: v plus its partner's of a DPP move, 0 where a lane
// has none.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ double add_move_f64(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROW_MASK, 0xF, false);
    const uint32_t hi =
        __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROW_MASK, 0xF, false);
    return v + __builtin_bit_cast(double, lo | (uint64_t)hi << 32);
}
// The running sum over the lanes of a wavefront, the lane's own included.
__device__ __forceinline__ double wave_scan_f64(double v) {
    constexpr int kRight = 0x110;                  // row_shr:0
    v = add_move_f64<kRight + 1, 0xF>(v);
    v = add_move_f64<kRight + 2, 0xF>(v);
    v = add_move_f64<kRight + 4, 0xF>(v);
    v = add_move_f64<kRight + 8, 0xF>(v);
    v = add_move_f64<dpp::kBcast15, 0xA>(v);
    return add_move_f64<dpp::kBcast31, 0xC>(v);
}
__device__ __forceinline__ double lane63_f64(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, 63);
    const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), 63);
    return __builtin_bit_cast(double, lo | (uint64_t)hi << 32);
}
__device__ __forceinline__ double wave_sum_f64(double v) {
    return lane63_f64(wave_scan_f64(v));
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

// (value, id) in the argmax order; 0 is below every real column.
__device__ __forceinline__ uint64_t order_of(float x, int32_t id) {
    return ((uint64_t)key_f32(__builtin_bit_cast(uint32_t, x)) << 32) | (uint32_t)~id;
}
__device__ __forceinline__ float value_of_key(uint32_t key) {
    if (key == kKeyNanF32)
        return __builtin_nanf("");
    if (key == kKeyZeroF32)
        return 0.0f;
    return __builtin_bit_cast(float, bits_of_key_f32(key));
}
__device__ __forceinline__ float value_of(uint64_t order) {
    return value_of_key((uint32_t)(order >> 32));
}
__device__ __forceinline__ int32_t id_of(uint64_t order) {
    return (int32_t)~(uint32_t)order;
}

__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
        const uint64_t o = __shfl_xor((unsigned long long)v, off, 64);
        v = o > v ? o : v;
    }
    return v;
}

}  // namespace vpa
