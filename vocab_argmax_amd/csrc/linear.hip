// linear.hip -- the head's products: y = residual + act(x W^T + bias) and the
// products of its backward pass, on the matrix cores with fp32 accumulation.
#include "vpa_head_internal.h"
#include "vpa_math.h"

namespace vpa {
namespace {

constexpr int kThreads = 256;

// Activations and their slopes, in fp32.
template <int ACT>
__device__ __forceinline__ float act(float z) {
    if constexpr (ACT == VPA_ACT_RELU)
        return z < 0.0f ? 0.0f : z;                // NaN stays
    if constexpr (ACT == VPA_ACT_GELU)
        return 0.5f * z * (1.0f + erff(z * 0.70710678118654752440f));
    if constexpr (ACT == VPA_ACT_SILU)
        return z / (1.0f + exp2_fast(-z * kLog2e));
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
        const float q = 1.0f / (1.0f + exp2_fast(-z * kLog2e));
        return q * (1.0f + z * (1.0f - q));
    }
    return 1.0f;
}

// One finished product of the epilogue.
template <typename T, int ACT>
__device__ __forceinline__ void store_result(const GemmTask& t, int64_t m, int64_t n, float acc) {
    const float z = acc + (t.bias ? to_f32(((const T*)t.bias)[n]) : 0.0f);
    if (t.pre)
        from_f32(((T*)t.pre)[m * t.ldp + n], z);
    float y = act<ACT>(z);
    if (t.residual)
        y += to_f32(((const T*)t.residual)[m * t.ldr + n]);
    if (t.out_f32)
        ((float*)t.y)[m * t.ldy + n] = y;
    else
        from_f32(((T*)t.y)[m * t.ldy + n], y);
}

constexpr int kTile = 64;

// Any strides and sizes: a 64x64 tile per workgroup, a wavefront per 16 rows
// of it, operands staged element by element.  MFMA operand layout: lane l
// holds row l % 16, k = (l / 16) * E + e for its E elements; of the result,
// column l % 16 and rows (l / 16) * 4 + i.
template <int ESIZE, int ACT>
__global__ __launch_bounds__(kThreads) void gemm_any_kernel(GemmTask t) {
    using T = typename elem<ESIZE>::type;
    constexpr int KB = 32;
    constexpr int LD = KB + 16 / ESIZE;
    __shared__ T as[kTile][LD], bs[kTile][LD];
    const int64_t tiles_n = (t.n + kTile - 1) / kTile;
    const int64_t m0 = blockIdx.x / tiles_n * kTile, n0 = blockIdx.x % tiles_n * kTile;
    const T* a = (const T*)t.a;
    const T* b = (const T*)t.b;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    f32x4 acc[4] = {};
    for (int64_t k0 = 0; k0 < t.k; k0 += KB) {
        for (int i = threadIdx.x; i < kTile * KB; i += kThreads) {
            // consecutive threads along the operand's contiguous direction
            const int ra = t.a_k == 1 ? i / KB : i % kTile, ka = t.a_k == 1 ? i % KB : i / kTile;
            const int rb = t.b_k == 1 ? i / KB : i % kTile, kb = t.b_k == 1 ? i % KB : i / kTile;
            as[ra][ka] = m0 + ra < t.m && k0 + ka < t.k
                             ? a[(m0 + ra) * t.a_m + (k0 + ka) * t.a_k] : (T)0;
            bs[rb][kb] = n0 + rb < t.n && k0 + kb < t.k
                             ? b[(n0 + rb) * t.b_n + (k0 + kb) * t.b_k] : (T)0;
        }
        __syncthreads();
        const int r = lane & 15, q = lane >> 4;
        if constexpr (ESIZE == 2) {
            const bf16x8 av = *(const bf16x8*)&as[wave * 16 + r][q * 8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bf16x8 bv = *(const bf16x8*)&bs[j * 16 + r][q * 8];
                acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, bv, acc[j], 0, 0, 0);
            }
        } else {
            for (int k = 0; k < KB; k += 4) {
                const float av = as[wave * 16 + r][k + q];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(av, bs[j * 16 + r][k + q],
                                                                  acc[j], 0, 0, 0);
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t m = m0 + wave * 16 + (lane >> 4) * 4 + i, n = n0 + j * 16 + (lane & 15);
            if (m < t.m && n < t.n)
                store_result<T, ACT>(t, m, n, acc[j][i]);
        }
}

template <typename T, int ACT>
__global__ __launch_bounds__(kThreads) void dz_kernel(DzTask t, int32_t splits) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (c >= t.cols)
        return;
    const int64_t per = (t.rows + splits - 1) / splits;
    const int64_t r0 = per * blockIdx.y, r1 = r0 + per < t.rows ? r0 + per : t.rows;
    float sum = 0.0f;
    for (int64_t r = r0; r < r1; ++r) {
        float d = to_f32(((const T*)t.grad)[r * t.ldg + c]);
        if constexpr (ACT != VPA_ACT_NONE)
            d *= act_slope<ACT>(to_f32(((const T*)t.pre)[r * t.ldp + c]));
        sum += d;
        if (t.dz)
            from_f32(((T*)t.dz)[r * t.ldz + c], d);
    }
    if (t.part)
        t.part[(int64_t)blockIdx.y * t.cols + c] = sum;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void bias_finish_kernel(DzTask t, int32_t splits) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (c >= t.cols)
        return;
    float sum = 0.0f;
    for (int32_t s = 0; s < splits; ++s)
        sum += t.part[(int64_t)s * t.cols + c];
    from_f32(((T*)t.bias)[c], sum);
}

template <int ESIZE>
hipError_t launch_gemm_any(const GemmTask& t, hipStream_t stream) {
    const dim3 grid((uint32_t)(gemm_threads(t.m, t.n) / kThreads)), block(kThreads);
    switch (t.act) {
    case VPA_ACT_RELU:
        return launch(gemm_any_kernel<ESIZE, VPA_ACT_RELU>, grid, block, 0, stream, t);
    case VPA_ACT_GELU:
        return launch(gemm_any_kernel<ESIZE, VPA_ACT_GELU>, grid, block, 0, stream, t);
    case VPA_ACT_SILU:
        return launch(gemm_any_kernel<ESIZE, VPA_ACT_SILU>, grid, block, 0, stream, t);
    default:
        return launch(gemm_any_kernel<ESIZE, VPA_ACT_NONE>, grid, block, 0, stream, t);
    }
}

template <typename T>
hipError_t launch_dz_typed(const DzTask& t, hipStream_t stream) {
    const int32_t splits = dz_splits(t.rows, t.cols);
    const dim3 grid((uint32_t)((t.cols + kThreads - 1) / kThreads), (uint32_t)splits);
    const dim3 block(kThreads);
    hipError_t e;
    switch (t.act) {
    case VPA_ACT_RELU:
        e = launch(dz_kernel<T, VPA_ACT_RELU>, grid, block, 0, stream, t, splits);
        break;
    case VPA_ACT_GELU:
        e = launch(dz_kernel<T, VPA_ACT_GELU>, grid, block, 0, stream, t, splits);
        break;
    case VPA_ACT_SILU:
        e = launch(dz_kernel<T, VPA_ACT_SILU>, grid, block, 0, stream, t, splits);
        break;
    default:
        e = launch(dz_kernel<T, VPA_ACT_NONE>, grid, block, 0, stream, t, splits);
    }
    if (e != hipSuccess || !t.bias)
        return e;
    return launch(bias_finish_kernel<T>, dim3(grid.x), block, 0, stream, t, t.part ? splits : 0);
}

}  // namespace

size_t gemm_workspace(int, int64_t, int64_t, int64_t, bool, bool) {
    return 0;
}

int64_t gemm_threads(int64_t m, int64_t n) {
    return ((m + kTile - 1) / kTile) * ((n + kTile - 1) / kTile) * kThreads;
}

hipError_t launch_gemm(int esize, const GemmTask& t, hipStream_t stream) {
    return esize == 2 ? launch_gemm_any<2>(t, stream) : launch_gemm_any<4>(t, stream);
}

int32_t dz_splits(int64_t rows, int64_t) {
    const int64_t s = (rows + 63) / 64;
    return (int32_t)(s < 1 ? 1 : s > 64 ? 64 : s);
}

int64_t dz_threads(int64_t rows, int64_t cols) {
    return (cols + kThreads - 1) / kThreads * kThreads * dz_splits(rows, cols);
}

hipError_t launch_dz(int esize, const DzTask& t, hipStream_t stream) {
    return esize == 2 ? launch_dz_typed<uint16_t>(t, stream) : launch_dz_typed<float>(t, stream);
}

}  // namespace vpa
