// layer_norm.hip -- layer norm over the rows of a matrix and its backward
// pass.  Statistics and sums are fp32 whatever the element type; the variance
// comes from the squared distances from the mean, so that a large mean costs
// no digits.
#include "vpa_head_internal.h"
#include "vpa_math.h"

namespace vpa {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

template <typename T, typename W>
__global__ __launch_bounds__(kThreads) void norm_kernel(NormTask t) {
    __shared__ float lds[3][kWaves];
    const int64_t row = blockIdx.x;
    const T* x = (const T*)t.x + row * t.ldx;
    T* y = (T*)t.y + row * t.ldy;
    const W* w = (const W*)t.weight;
    const W* b = (const W*)t.bias;
    float s = 0.0f;
    for (int64_t c = threadIdx.x; c < t.cols; c += kThreads)
        s += to_f32(x[c]);
    // a first mean, then its correction beside the variance: the sum of a row
    // far from 0 loses bits that the sum of its distances keeps
    const float mean0 = block_sum<kWaves>(s, lds[0]) / (float)t.cols;
    float p = 0.0f, q = 0.0f;
    for (int64_t c = threadIdx.x; c < t.cols; c += kThreads) {
        const float d = to_f32(x[c]) - mean0;
        p += d;
        q += d * d;
    }
    const float delta = block_sum<kWaves>(p, lds[1]) / (float)t.cols;
    const float var = block_sum<kWaves>(q, lds[2]) / (float)t.cols - delta * delta;
    const float rstd = 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + t.eps);
    for (int64_t c = threadIdx.x; c < t.cols; c += kThreads) {
        float v = ((to_f32(x[c]) - mean0) - delta) * rstd;
        v = v * (w ? to_f32(w[c]) : 1.0f) + (b ? to_f32(b[c]) : 0.0f);
        from_f32(y[c], v);
    }
    const float mean = mean0 + delta;
    if (threadIdx.x == 0) {
        if (t.mean)
            t.mean[row] = mean;
        if (t.rstd)
            t.rstd[row] = rstd;
    }
}

template <typename T, typename W>
__global__ __launch_bounds__(kThreads) void norm_dx_kernel(NormGradTask t) {
    __shared__ float lds[2][kWaves];
    const int64_t row = blockIdx.x;
    const T* x = (const T*)t.x + row * t.ldx;
    const T* g = (const T*)t.grad + row * t.ldg;
    T* dx = (T*)t.dx + row * t.lddx;
    const W* w = (const W*)t.weight;
    const float mean = t.mean[row], rstd = t.rstd[row];
    float a = 0.0f, b = 0.0f;
    for (int64_t c = threadIdx.x; c < t.cols; c += kThreads) {
        const float u = to_f32(g[c]) * (w ? to_f32(w[c]) : 1.0f);
        a += u;
        b += u * ((to_f32(x[c]) - mean) * rstd);
    }
    a = block_sum<kWaves>(a, lds[0]) / (float)t.cols;
    b = block_sum<kWaves>(b, lds[1]) / (float)t.cols;
    for (int64_t c = threadIdx.x; c < t.cols; c += kThreads) {
        const float u = to_f32(g[c]) * (w ? to_f32(w[c]) : 1.0f);
        const float xh = (to_f32(x[c]) - mean) * rstd;
        from_f32(dx[c], rstd * (u - a - xh * b));
    }
}

// Column sums of one slice of rows: part[0][split][c] = sum grad * xh,
// part[1][split][c] = sum grad.
template <typename T>
__global__ __launch_bounds__(kThreads) void norm_columns_kernel(NormGradTask t, int32_t splits) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int32_t split = blockIdx.y;
    if (c >= t.cols)
        return;
    const int64_t per = (t.rows + splits - 1) / splits;
    const int64_t r1 = per * (split + 1) < t.rows ? per * (split + 1) : t.rows;
    float dw = 0.0f, db = 0.0f;
    for (int64_t r = per * split; r < r1; ++r) {
        const float g = to_f32(((const T*)t.grad)[r * t.ldg + c]);
        dw += g * ((to_f32(((const T*)t.x)[r * t.ldx + c]) - t.mean[r]) * t.rstd[r]);
        db += g;
    }
    t.part[(int64_t)split * t.cols + c] = dw;
    t.part[((int64_t)splits + split) * t.cols + c] = db;
}

template <typename W>
__global__ __launch_bounds__(kThreads) void norm_columns_finish_kernel(NormGradTask t,
                                                                       int32_t splits) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (c >= t.cols)
        return;
    float dw = 0.0f, db = 0.0f;
    for (int32_t s = 0; s < splits; ++s) {
        dw += t.part[(int64_t)s * t.cols + c];
        db += t.part[((int64_t)splits + s) * t.cols + c];
    }
    if (t.dweight)
        from_f32(((W*)t.dweight)[c], dw);
    if (t.dbias)
        from_f32(((W*)t.dbias)[c], db);
}

}  // namespace

int64_t norm_threads(int64_t rows, int64_t) {
    return rows * kThreads;
}

hipError_t launch_norm(int esize, const NormTask& t, hipStream_t stream) {
    const dim3 grid((uint32_t)t.rows), block(kThreads);
    if (esize == 4)
        return launch(norm_kernel<float, float>, grid, block, 0, stream, t);
    return t.wsize == 4 ? launch(norm_kernel<uint16_t, float>, grid, block, 0, stream, t)
                        : launch(norm_kernel<uint16_t, uint16_t>, grid, block, 0, stream, t);
}

int32_t norm_splits(int64_t rows, int64_t) {
    const int64_t s = (rows + 63) / 64;
    return (int32_t)(s < 1 ? 1 : s > 64 ? 64 : s);
}

int64_t norm_grad_threads(int64_t rows, int64_t cols) {
    const int64_t a = rows * kThreads;
    const int64_t b = (cols + kThreads - 1) / kThreads * kThreads * norm_splits(rows, cols);
    return a > b ? a : b;
}

hipError_t launch_norm_grad(int esize, const NormGradTask& t, hipStream_t stream) {
    const dim3 block(kThreads);
    hipError_t e = hipSuccess;
    if (t.dx && t.rows > 0) {
        const dim3 grid((uint32_t)t.rows);
        if (esize == 4)
            e = launch(norm_dx_kernel<float, float>, grid, block, 0, stream, t);
        else if (t.wsize == 4)
            e = launch(norm_dx_kernel<uint16_t, float>, grid, block, 0, stream, t);
        else
            e = launch(norm_dx_kernel<uint16_t, uint16_t>, grid, block, 0, stream, t);
        if (e != hipSuccess)
            return e;
    }
    if (!t.dweight && !t.dbias)
        return e;
    const int32_t splits = norm_splits(t.rows, t.cols);
    const uint32_t tiles = (uint32_t)((t.cols + kThreads - 1) / kThreads);
    e = esize == 4
            ? launch(norm_columns_kernel<float>, dim3(tiles, splits), block, 0, stream, t, splits)
            : launch(norm_columns_kernel<uint16_t>, dim3(tiles, splits), block, 0, stream, t,
                     splits);
    if (e != hipSuccess)
        return e;
    return t.wsize == 4
               ? launch(norm_columns_finish_kernel<float>, dim3(tiles), block, 0, stream, t, splits)
               : launch(norm_columns_finish_kernel<uint16_t>, dim3(tiles), block, 0, stream, t,
                        splits);
}

}  // namespace vpa
