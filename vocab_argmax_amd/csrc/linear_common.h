// linear_common.h -- the epilogue of the head's products: activations with
// their slopes, and the stores of finished results.
#pragma once

#include "vpa_head_internal.h"
#include "vpa_math.h"

namespace vpa {

// Activations and their slopes, in fp32.
template <int ACT>
__device__ __forceinline__ float act(float z) {
    if constexpr (ACT == VPA_ACT_RELU)
        return z < 0.0f ? 0.0f : z;                // NaN stays
    if constexpr (ACT == VPA_ACT_GELU)
        return 0.5f * z * (1.0f + erff(z * 0.70710678118654752440f));
    if constexpr (ACT == VPA_ACT_SILU)
        return z * __builtin_amdgcn_rcpf(1.0f + exp2_fast(-z * kLog2e));   // within 1 ulp
    return z;
}
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    if constexpr (ACT == VPA_ACT_RELU)
        return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
    if constexpr (ACT == VPA_ACT_GELU)
        return 0.5f * (1.0f + erff(z * 0.70710678118654752440f)) +
               z * exp2_fast(-0.5f * kLog2e * z * z) * 0.39894228040143267794f;
    if constexpr (ACT == VPA_ACT_SILU) {
        const float q = __builtin_amdgcn_rcpf(1.0f + exp2_fast(-z * kLog2e));
        return q * (1.0f + z * (1.0f - q));
    }
    return 1.0f;
}

template <int ACT>
__device__ __forceinline__ f32x4 act4(f32x4 z) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        z[i] = act<ACT>(z[i]);
    return z;
}

// The activation of an epilogue, chosen at run time: a uniform branch.
__device__ __forceinline__ float act_any(int32_t a, float z) {
    switch (a) {
    case VPA_ACT_RELU:
        return act<VPA_ACT_RELU>(z);
    case VPA_ACT_GELU:
        return act<VPA_ACT_GELU>(z);
    case VPA_ACT_SILU:
        return act<VPA_ACT_SILU>(z);
    default:
        return z;
    }
}

// One finished product of the epilogue.
template <typename T>
__device__ __forceinline__ void store_result(const GemmTask& t, int64_t m, int64_t n, float acc) {
    const float z = acc + (t.bias ? to_f32(((const T*)t.bias)[n]) : 0.0f);
    if (t.pre)
        from_f32(((T*)t.pre)[m * t.ldp + n], z);
    float y = act_any(t.act, z);
    if (t.residual)
        y += to_f32(((const T*)t.residual)[m * t.ldr + n]);
    if (t.out_f32)
        ((float*)t.y)[m * t.ldy + n] = y;
    else
        from_f32(((T*)t.y)[m * t.ldy + n], y);
}

// Four elements at any element address: global memory takes accesses of 8 or
// 16 bytes at every alignment of the element.
template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) Loose4 {
    T e[4];
};
template <typename T>
__device__ __forceinline__ f32x4 load4(const T* p) {
    const Loose4<T> v = *(const Loose4<T>*)p;
    return f32x4{to_f32(v.e[0]), to_f32(v.e[1]), to_f32(v.e[2]), to_f32(v.e[3])};
}
// Results are stored past the L2, which keeps the operands in it (nt; 32 x
// 2048 x 151936 to fp32 122 -> 118 us, 2048 x 50257 x 2048 412 -> 404, 128 x
// 2048 x 151936 160 -> 151).  A slice's sums, which the next kernel reads, are
// kept.
__device__ __forceinline__ void keep4(float* p, f32x4 v) {
    *(Loose4<float>*)p = Loose4<float>{{v[0], v[1], v[2], v[3]}};
}
__device__ __forceinline__ void store4(float* p, f32x4 v) {
    typedef float f32x4_loose __attribute__((ext_vector_type(4), aligned(4)));
    __builtin_nontemporal_store((f32x4_loose)v, (f32x4_loose*)p);
}
__device__ __forceinline__ void store4(uint16_t* p, f32x4 v) {
    typedef uint32_t u32x2_loose __attribute__((ext_vector_type(2), aligned(2)));
    const u32x2_loose u = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    __builtin_nontemporal_store(u, (u32x2_loose*)p);
}

// Four results of consecutive n; `res` holds the residual's, where there is one.
template <typename T>
__device__ __forceinline__ void store_results(const GemmTask& t, int64_t m, int64_t n, f32x4 acc,
                                              f32x4 res) {
    if (t.bias)
        acc += load4((const T*)t.bias + n);
    if (t.pre)
        store4((T*)t.pre + m * t.ldp + n, acc);
    switch (t.act) {                               // one uniform branch for the four
    case VPA_ACT_RELU:
        acc = act4<VPA_ACT_RELU>(acc);
        break;
    case VPA_ACT_GELU:
        acc = act4<VPA_ACT_GELU>(acc);
        break;
    case VPA_ACT_SILU:
        acc = act4<VPA_ACT_SILU>(acc);
        break;
    default:
        break;
    }
    acc += res;
    if (t.out_f32)
        store4((float*)t.y + m * t.ldy + n, acc);
    else
        store4((T*)t.y + m * t.ldy + n, acc);
}
template <typename T>
__device__ __forceinline__ void store_results(const GemmTask& t, int64_t m, int64_t n, f32x4 acc) {
    const f32x4 none = {-0.0f, -0.0f, -0.0f, -0.0f};    // keeps a result's sign of zero
    store_results<T>(t, m, n, acc,
                     t.residual ? load4((const T*)t.residual + m * t.ldr + n) : none);
}

// A wavefront's 64 x 64 results from accumulators to memory, through its own
// 16 KiB of LDS so that a store instruction covers 4 rows of 64, 4 results a
// lane; the lane that n ends in stores its one by one (a row at a time, a
// result a lane, cost 512 x 784 x 10240's gradient of W 44 us, 27 so).
// Rows of LDS have 16 chunks of 16 bytes, chunk c of row r at c ^ (r & 15).
template <typename T>
__device__ __forceinline__ void store_block(const GemmTask& t, float* part, char* lds,
                                            int64_t m0, int64_t n0, const f32x4 (&acc)[4][4]) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = i * 16 + (lane & 15), c = j * 4 + (lane >> 4);
            *(f32x4*)(lds + r * 256 + ((c ^ (r & 15)) << 4)) = acc[i][j];
        }
    // this LDS is the wavefront's alone and its accesses execute in order; the
    // fences keep the compiler to it
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int64_t n = n0 + (lane & 15) * 4;
    const int left = t.n - n < 4 ? (int)(t.n - n) : 4;          // results of this lane, or < 1
    if (n0 < t.n) {
        // the residual of a pass of 4 x 4 rows is on its way during the last
        const bool res = t.residual && !part;
        f32x4 next[4];
        auto fetch = [&](int r0) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t m = m0 + r0 + k * 4 + (lane >> 4);
                next[k] = f32x4{-0.0f, -0.0f, -0.0f, -0.0f};
                if (res && m < t.m && left == 4)
                    next[k] = load4((const T*)t.residual + m * t.ldr + n);
            }
        };
        fetch(0);
#pragma unroll 1
        for (int r0 = 0; r0 < 64; r0 += 16) {
            f32x4 v[4], r4[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = r0 + k * 4 + (lane >> 4), c = lane & 15;
                v[k] = *(const f32x4*)(lds + r * 256 + ((c ^ (r & 15)) << 4));
                r4[k] = next[k];
            }
            if (r0 < 48)
                fetch(r0 + 16);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t m = m0 + r0 + k * 4 + (lane >> 4);
                if (m >= t.m)
                    continue;
                if (left == 4) {
                    if (part)
                        keep4(part + m * t.n + n, v[k]);
                    else
                        store_results<T>(t, m, n, v[k], r4[k]);
                    continue;
                }
#pragma unroll
                for (int e = 0; e < 3; ++e)
                    if (e < left) {
                        if (part)
                            part[m * t.n + n + e] = v[k][e];
                        else
                            store_result<T>(t, m, n + e, v[k][e]);
                    }
            }
        }
    }
}

}  // namespace vpa
