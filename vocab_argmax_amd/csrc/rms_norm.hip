// rms_norm.hip -- root-mean-square norm over the rows of a matrix, with the
// residual's addition before it and, where asked for, an output in 8 bits with
// a scale for each block of 128 columns; its backward pass; and the same 8-bit
// form of a matrix as it is.
//
// The sum of squares is fp32.  The norm is taken of the sum as it is stored
// (rounded to its type), which is what the backward pass reads.
#include "norm_rows.h"
#include "vpa_draft_internal.h"

namespace vpa {
namespace {

constexpr int kThreads = 256;
constexpr float kFp8Max = 448.0f;
constexpr uint32_t kAmaxLeast = 0x0D800000u;       // 2^-100

// A block's scale and its inverse from the largest |y| as fp32 bits, which sort
// as the values do, infinity and NaN last.
struct BlockScale {
    float scale, inverse;
};
__device__ __forceinline__ BlockScale block_scale(uint32_t amax_bits) {
    if (amax_bits >= 0x7F800000u)
        return {__builtin_nanf(""), __builtin_nanf("")};
    const float amax = __builtin_bit_cast(float, amax_bits < kAmaxLeast ? kAmaxLeast : amax_bits);
    return {amax / kFp8Max, kFp8Max / amax};
}
__device__ __forceinline__ uint32_t abs_bits(float f) {
    return __builtin_bit_cast(uint32_t, f) & 0x7FFFFFFFu;
}
// Two values in 8 bits, to nearest even (NaN stays NaN): bits 0-7 and 8-15.
// Values above 448 by the inverse's rounding are 448.
__device__ __forceinline__ uint32_t pack_fp8(float a, float b) {
    a = a > kFp8Max ? kFp8Max : a < -kFp8Max ? -kFp8Max : a;
    b = b > kFp8Max ? kFp8Max : b < -kFp8Max ? -kFp8Max : b;
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false) & 0xFFFFu;
}

// A row to a workgroup, several passes over it.
template <typename T, typename W>
__global__ __launch_bounds__(kLongThreads) void rms_long_kernel(RmsTask t) {
    __shared__ float lds[kLongWaves][2];
    const int64_t row = blockIdx.x;
    const T* x = (const T*)t.x + row * t.ldx;
    const T* r = t.residual ? (const T*)t.residual + row * t.ldr : nullptr;
    T* s = t.residual ? (T*)t.summed + row * t.lds : nullptr;
    const W* w = (const W*)t.weight;
    float q = 0.0f, none = 0.0f;
    for (int64_t c = threadIdx.x; c < t.cols; c += kLongThreads) {
        float v = to_f32(x[c]);
        if (r) {
            T sum;
            from_f32(sum, v + to_f32(r[c]));
            s[c] = sum;
            v = to_f32(sum);
        }
        q = __builtin_fmaf(v, v, q);
    }
    block_sum2<kLongWaves>(q, none, lds);
    const float rstd = 1.0f / sqrtf(q / (float)t.cols + t.eps);
    if (t.rstd && threadIdx.x == 0)
        t.rstd[row] = rstd;
    auto value = [&](int64_t c) {
        const float v = to_f32(s ? s[c] : x[c]);
        return v * rstd * (w ? to_f32(w[c]) : 1.0f);
    };
    if (!t.scale) {
        for (int64_t c = threadIdx.x; c < t.cols; c += kLongThreads)
            from_f32(((T*)t.y)[row * t.ldy + c], value(c));
        return;
    }
    if (s)
        __syncthreads();                   // other threads' sums
    // a wavefront a block of 128 columns, two a lane
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint8_t* y = (uint8_t*)t.y + row * t.ldy;
    for (int64_t b = wave; b * kScaleBlock < t.cols; b += kLongWaves) {
        const int64_t c = b * kScaleBlock + lane * 2;
        const float v0 = c < t.cols ? value(c) : 0.0f, v1 = c + 1 < t.cols ? value(c + 1) : 0.0f;
        uint32_t amax = abs_bits(v0) > abs_bits(v1) ? abs_bits(v0) : abs_bits(v1);
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) {
            const uint32_t o = __shfl_xor(amax, off, 64);
            amax = o > amax ? o : amax;
        }
        const BlockScale sc = block_scale(amax);
        const uint32_t p = pack_fp8(v0 * sc.inverse, v1 * sc.inverse);
        if (c < t.cols)
            y[c] = (uint8_t)p;
        if (c + 1 < t.cols)
            y[c + 1] = (uint8_t)(p >> 8);
        if (lane == 0)
            t.scale[row * t.ld_scale + b] = sc.scale;
    }
}

template <typename T, typename W>
__global__ __launch_bounds__(kLongThreads) void rms_long_dx_kernel(RmsGradTask t) {
    __shared__ float lds[kLongWaves][2];
    const int64_t row = blockIdx.x;
    const T* x = (const T*)t.summed + row * t.lds;
    const T* g = (const T*)t.grad + row * t.ldg;
    const T* gs = t.grad_summed ? (const T*)t.grad_summed + row * t.ldgs : nullptr;
    T* dx = (T*)t.dx + row * t.lddx;
    const W* w = (const W*)t.weight;
    const float rstd = t.rstd[row];
    float b = 0.0f, none = 0.0f;
    for (int64_t c = threadIdx.x; c < t.cols; c += kLongThreads) {
        const float u = to_f32(g[c]) * (w ? to_f32(w[c]) : 1.0f);
        b = __builtin_fmaf(u, to_f32(x[c]) * rstd, b);
    }
    block_sum2<kLongWaves>(b, none, lds);
    b /= (float)t.cols;
    for (int64_t c = threadIdx.x; c < t.cols; c += kLongThreads) {
        const float u = to_f32(g[c]) * (w ? to_f32(w[c]) : 1.0f);
        const float d = rstd * (u - to_f32(x[c]) * rstd * b);
        from_f32(dx[c], gs ? d + to_f32(gs[c]) : d);
    }
}

// The column sums of one slice of rows, a thread a column.
template <typename T>
__global__ __launch_bounds__(kThreads) void rms_long_columns_kernel(RmsGradTask t,
                                                                    int32_t splits) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int32_t split = blockIdx.y;
    if (c >= t.cols)
        return;
    const int64_t per = (t.rows + splits - 1) / splits;
    const int64_t r1 = per * (split + 1) < t.rows ? per * (split + 1) : t.rows;
    float dw = 0.0f;
    for (int64_t r = per * split; r < r1; ++r)
        dw = __builtin_fmaf(to_f32(((const T*)t.grad)[r * t.ldg + c]),
                            to_f32(((const T*)t.summed)[r * t.lds + c]) * t.rstd[r], dw);
    t.part[(int64_t)split * t.cols + c] = dw;
}

// The slices' column sums, added in a fixed order: 64 columns a workgroup, 16
// wavefronts with every sixteenth sum each.
constexpr int kJoinWaves = 16;

template <typename W>
__global__ __launch_bounds__(kJoinWaves * 64) void rms_join_kernel(RmsGradTask t, int32_t splits) {
    __shared__ float sums[kJoinWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    float s = 0.0f;
    if (c < t.cols) {
#pragma unroll 8
        for (int32_t i = wave; i < splits; i += kJoinWaves)
            s += t.part[(int64_t)i * t.cols + c];
    }
    sums[wave][lane] = s;
    __syncthreads();
    if (wave != 0 || c >= t.cols)
        return;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < kJoinWaves; ++i)
        s += sums[i][lane];
    from_f32(((W*)t.dweight)[c], s);
}

// A workgroup a block of block_rows x 128.
template <typename T>
__global__ __launch_bounds__(kThreads) void quant_kernel(QuantTask t, int64_t blocks_across) {
    __shared__ uint32_t lds[4];
    const int64_t br = blockIdx.x / blocks_across, bc = blockIdx.x % blocks_across;
    const int64_t r0 = br * t.block_rows, c = bc * kScaleBlock + threadIdx.x % kScaleBlock;
    const int64_t r1 = r0 + t.block_rows < t.rows ? r0 + t.block_rows : t.rows;
    const int64_t first = r0 + threadIdx.x / kScaleBlock;
    uint32_t amax = 0;
    if (c < t.cols)
        for (int64_t r = first; r < r1; r += kThreads / kScaleBlock) {
            const uint32_t b = abs_bits(to_f32(((const T*)t.x)[r * t.ldx + c]));
            amax = b > amax ? b : amax;
        }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
        const uint32_t o = __shfl_xor(amax, off, 64);
        amax = o > amax ? o : amax;
    }
    if ((threadIdx.x & 63) == 0)
        lds[threadIdx.x >> 6] = amax;
    __syncthreads();
    for (int i = 0; i < 4; ++i)
        amax = lds[i] > amax ? lds[i] : amax;
    const BlockScale sc = block_scale(amax);
    if (c < t.cols)
        for (int64_t r = first; r < r1; r += kThreads / kScaleBlock)
            ((uint8_t*)t.y)[r * t.ldy + c] =
                (uint8_t)pack_fp8(to_f32(((const T*)t.x)[r * t.ldx + c]) * sc.inverse, 0.0f);
    if (threadIdx.x == 0)
        t.scale[br * t.ld_scale + bc] = sc.scale;
}

template <typename T, typename W>
hipError_t launch_rms_typed(const RmsTask& t, hipStream_t stream) {
    return launch(rms_long_kernel<T, W>, dim3((uint32_t)t.rows), dim3(kLongThreads), 0, stream, t);
}

template <typename T, typename W>
hipError_t launch_rms_grad_typed(const RmsGradTask& t, hipStream_t stream) {
    // no rows: no sums, and the joining kernel writes 0
    const int32_t splits = t.rows > 0 ? rms_splits((int)sizeof(T), t.rows, t.cols) : 0;
    hipError_t e = hipSuccess;
    if (t.dx)
        e = launch(rms_long_dx_kernel<T, W>, dim3((uint32_t)t.rows), dim3(kLongThreads), 0, stream,
                   t);
    if (e != hipSuccess || !t.dweight)
        return e;
    if (splits > 0)
        e = launch(rms_long_columns_kernel<T>,
                   dim3((uint32_t)((t.cols + kThreads - 1) / kThreads), (uint32_t)splits),
                   dim3(kThreads), 0, stream, t, splits);
    if (e != hipSuccess)
        return e;
    return launch(rms_join_kernel<W>, dim3((uint32_t)((t.cols + 63) / 64)), dim3(kJoinWaves * 64), 0,
                  stream, t, splits);
}

}  // namespace

int64_t rms_threads(int, int64_t rows, int64_t) {
    return rows * kLongThreads;
}

hipError_t launch_rms(int esize, const RmsTask& t, hipStream_t stream) {
    if (esize == 4)
        return launch_rms_typed<float, float>(t, stream);
    return t.wsize == 4 ? launch_rms_typed<uint16_t, float>(t, stream)
                        : launch_rms_typed<uint16_t, uint16_t>(t, stream);
}

int32_t rms_splits(int, int64_t rows, int64_t) {
    const int64_t s = (rows + 63) / 64;
    return (int32_t)(s < 1 ? 1 : s > 64 ? 64 : s);
}

int64_t rms_grad_threads(int esize, int64_t rows, int64_t cols, bool dx, bool sums) {
    int64_t most = dx ? rows * kLongThreads : 0;
    if (sums) {
        const int64_t columns = (cols + kThreads - 1) / kThreads * kThreads *
                                rms_splits(esize, rows, cols);
        const int64_t join = (cols + 63) / 64 * 64 * kJoinWaves;
        most = columns > most ? columns : most;
        most = join > most ? join : most;
    }
    return most;
}

hipError_t launch_rms_grad(int esize, const RmsGradTask& t, hipStream_t stream) {
    if (esize == 4)
        return launch_rms_grad_typed<float, float>(t, stream);
    return t.wsize == 4 ? launch_rms_grad_typed<uint16_t, float>(t, stream)
                        : launch_rms_grad_typed<uint16_t, uint16_t>(t, stream);
}

int64_t quant_threads(int64_t rows, int64_t cols, int32_t block_rows) {
    return (rows + block_rows - 1) / block_rows * ((cols + kScaleBlock - 1) / kScaleBlock) *
           kThreads;
}

hipError_t launch_quant(int esize, const QuantTask& t, hipStream_t stream) {
    const int64_t across = (t.cols + kScaleBlock - 1) / kScaleBlock;
    const dim3 grid((uint32_t)((t.rows + t.block_rows - 1) / t.block_rows * across));
    return esize == 2 ? launch(quant_kernel<uint16_t>, grid, dim3(kThreads), 0, stream, t, across)
                      : launch(quant_kernel<float>, grid, dim3(kThreads), 0, stream, t, across);
}

}  // namespace vpa
