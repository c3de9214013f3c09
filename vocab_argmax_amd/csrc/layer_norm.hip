// layer_norm.hip -- layer norm over the rows of a matrix and its backward
// pass.  Statistics and sums are fp32 whatever the element type; the variance
// comes from the squared distances from the mean, so that a large mean costs
// no digits.
//
// Both directions are bound by memory: a row is read once, into registers.
// A workgroup of WAVES wavefronts holds NV 16-byte vectors a thread and walks
// over rows blockIdx.x, blockIdx.x + gridDim.x, ...; the next row is on its
// way while one is worked on, and the weights stay in registers.  The
// backward pass adds its rows' weight and bias gradients up in registers too
// (a thread always has the same columns), so x and grad are read once for all
// three gradients; a second kernel joins the workgroups' sums in order.
// Measured, kernels alone: 8192 x 4096 bf16 forward 24 us (5.7 TB/s of reads
// and writes), backward 34 + 4.5 us (6.0); 32768 x 4096 forward 87 us (6.2);
// 3001 x 1601 fp32 10 and 13.4 + 4.5 us; 32 x 4096 forward 5.1 us, a launch's
// latency and two sums over a row.
#include "norm_rows.h"
#include "vpa_head_internal.h"

namespace vpa {
namespace {

template <typename T, typename W, int WAVES, int NV>
__global__ __launch_bounds__(WAVES == 1 ? 256 : WAVES * 64) void norm_kernel(NormTask t) {
    using P = RowPart<T, WAVES, NV>;
    constexpr int VEC = P::VEC, ESIZE = (int)sizeof(T);
    __shared__ float lds[2][2][WAVES][2];
    const int cols = (int)t.cols;
    float w[NV][VEC], b[NV][VEC];
    P::load_weights((const W*)t.weight, cols, 1.0f, w);
    P::load_weights((const W*)t.bias, cols, 0.0f, b);
    u32x4_t next[NV];
    int64_t row = P::first_row();
    if (row < t.rows)
        P::load((const T*)t.x + row * t.ldx, cols, next);
    for (int turn = 0; row < t.rows; row += P::row_step(), turn ^= 1) {
        u32x4_t v[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i)
            v[i] = next[i];
        const int64_t after = row + P::row_step();
        // (y may be x: the next row is read before any of it is written)
        if (after < t.rows)
            P::load((const T*)t.x + after * t.ldx, cols, next);
        float s = 0.0f, none = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                s += vec_elem<ESIZE>(v[i], e);       // 0 past the row
        block_sum2<WAVES>(s, none, lds[turn][0]);
        // a first mean, then its correction beside the variance: the sum of a
        // row far from 0 loses bits that the sum of its distances keeps
        const float mean0 = s / (float)cols;
        float p = 0.0f, q = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int n = P::count(i, cols);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float d = e < n ? vec_elem<ESIZE>(v[i], e) - mean0 : 0.0f;
                p += d;
                q = __builtin_fmaf(d, d, q);
            }
        }
        block_sum2<WAVES>(p, q, lds[turn][1]);
        const float delta = p / (float)cols;
        const float var = q / (float)cols - delta * delta;
        const float rstd = 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + t.eps);
        T* y = (T*)t.y + row * t.ldy;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float f[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                f[e] = __builtin_fmaf(((vec_elem<ESIZE>(v[i], e) - mean0) - delta) * rstd, w[i][e],
                                      b[i][e]);
            P::store(y, cols, i, f);
        }
        if (P::column(0) == 0) {
            if (t.mean)
                t.mean[row] = mean0 + delta;
            if (t.rstd)
                t.rstd[row] = rstd;
        }
    }
}

template <typename T, typename W, int WAVES, int NV>
__global__ __launch_bounds__(WAVES == 1 ? 256 : WAVES * 64) void norm_grad_kernel(NormGradTask t) {
    using P = RowPart<T, WAVES, NV>;
    constexpr int VEC = P::VEC, ESIZE = (int)sizeof(T);
    __shared__ float lds[2][WAVES][2];
    const int cols = (int)t.cols;
    float w[NV][VEC], dw[NV][VEC] = {}, db[NV][VEC] = {};
    P::load_weights((const W*)t.weight, cols, 1.0f, w);
    u32x4_t next_g[NV], next_x[NV];
    float next_mean = 0.0f, next_rstd = 0.0f;
    auto fetch = [&](int64_t r) {
        P::load((const T*)t.grad + r * t.ldg, cols, next_g);
        P::load((const T*)t.x + r * t.ldx, cols, next_x);
        next_mean = t.mean[r];
        next_rstd = t.rstd[r];
    };
    int64_t row = P::first_row();
    if (row < t.rows)
        fetch(row);
    for (int turn = 0; row < t.rows; row += P::row_step(), turn ^= 1) {
        u32x4_t g[NV], x[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            g[i] = next_g[i];
            x[i] = next_x[i];
        }
        const float mean = next_mean, rstd = next_rstd;
        const int64_t after = row + P::row_step();
        if (after < t.rows)
            fetch(after);
        // The xh of the 0 past the row meets grad's 0 there, and has to be finite:
        // where it is not, which takes elements that hardly differ, the mean
        // stands for it.
        if (!(fabsf(mean) * rstd < __builtin_inff())) {
            T value;
            from_f32(value, mean);
            P::fill_past(value, cols, x);
        }
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float gr = vec_elem<ESIZE>(g[i], e);          // 0 past the row
                const float xh = (vec_elem<ESIZE>(x[i], e) - mean) * rstd;
                const float u = gr * w[i][e];
                a += u;
                b = __builtin_fmaf(u, xh, b);
                dw[i][e] = __builtin_fmaf(gr, xh, dw[i][e]);
                db[i][e] += gr;
            }
        if (!t.dx)
            continue;
        block_sum2<WAVES>(a, b, lds[turn]);
        a /= (float)cols;
        b /= (float)cols;
        T* dx = (T*)t.dx + row * t.lddx;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float f[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float xh = (vec_elem<ESIZE>(x[i], e) - mean) * rstd;
                const float u = vec_elem<ESIZE>(g[i], e) * w[i][e];
                f[e] = rstd * ((u - a) - xh * b);
            }
            P::store(dx, cols, i, f);
        }
    }
    if (!t.part)
        return;
    if constexpr (P::ROWS > 1) {
        // the workgroup's rows' sums, added in order
        static_assert(NV == 1, "a wavefront a row");
        __shared__ float sums[P::ROWS][2][64 * VEC];
        const int group = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            sums[group][0][lane * VEC + e] = dw[0][e];
            sums[group][1][lane * VEC + e] = db[0][e];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * 64 * VEC; i += P::THREADS) {
            const int c = i % (64 * VEC), which = i / (64 * VEC);
            float s = 0.0f;
#pragma unroll
            for (int r = 0; r < P::ROWS; ++r)
                s += sums[r][which][c];
            if (c < cols)
                t.part[((int64_t)which * gridDim.x + blockIdx.x) * cols + c] = s;
        }
        return;
    }
    // part[0][workgroup][column]: weight's, part[1]: bias's
    float* pw = t.part + (int64_t)blockIdx.x * cols;
    float* pb = pw + (int64_t)gridDim.x * cols;
    typedef float f32x4_loose __attribute__((ext_vector_type(4), aligned(4)));
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VEC; e += 4) {
            const int c = P::column(i) + e;
            if (c + 4 <= cols) {
                *(f32x4_loose*)(pw + c) = f32x4_loose{dw[i][e], dw[i][e + 1], dw[i][e + 2],
                                                      dw[i][e + 3]};
                *(f32x4_loose*)(pb + c) = f32x4_loose{db[i][e], db[i][e + 1], db[i][e + 2],
                                                      db[i][e + 3]};
                continue;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (c + k < cols) {
                    pw[c + k] = dw[i][e + k];
                    pb[c + k] = db[i][e + k];
                }
        }
}

// Rows too long for a workgroup's registers: several passes over the row,
// which the caches hold.
template <typename T, typename W>
__global__ __launch_bounds__(kLongThreads) void norm_long_kernel(NormTask t) {
    __shared__ float lds[2][kLongWaves][2];
    const int64_t row = blockIdx.x;
    const T* x = (const T*)t.x + row * t.ldx;
    T* y = (T*)t.y + row * t.ldy;
    const W* w = (const W*)t.weight;
    const W* b = (const W*)t.bias;
    float s = 0.0f, none = 0.0f;
    for (int64_t c = threadIdx.x; c < t.cols; c += kLongThreads)
        s += to_f32(x[c]);
    block_sum2<kLongWaves>(s, none, lds[0]);
    const float mean0 = s / (float)t.cols;
    float p = 0.0f, q = 0.0f;
    for (int64_t c = threadIdx.x; c < t.cols; c += kLongThreads) {
        const float d = to_f32(x[c]) - mean0;
        p += d;
        q = __builtin_fmaf(d, d, q);
    }
    block_sum2<kLongWaves>(p, q, lds[1]);
    const float delta = p / (float)t.cols;
    const float var = q / (float)t.cols - delta * delta;
    const float rstd = 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + t.eps);
    for (int64_t c = threadIdx.x; c < t.cols; c += kLongThreads) {
        const float v = ((to_f32(x[c]) - mean0) - delta) * rstd;
        from_f32(y[c], __builtin_fmaf(v, w ? to_f32(w[c]) : 1.0f, b ? to_f32(b[c]) : 0.0f));
    }
    if (threadIdx.x == 0) {
        if (t.mean)
            t.mean[row] = mean0 + delta;
        if (t.rstd)
            t.rstd[row] = rstd;
    }
}

template <typename T, typename W>
__global__ __launch_bounds__(kLongThreads) void norm_long_dx_kernel(NormGradTask t) {
    __shared__ float lds[kLongWaves][2];
    const int64_t row = blockIdx.x;
    const T* x = (const T*)t.x + row * t.ldx;
    const T* g = (const T*)t.grad + row * t.ldg;
    T* dx = (T*)t.dx + row * t.lddx;
    const W* w = (const W*)t.weight;
    const float mean = t.mean[row], rstd = t.rstd[row];
    float a = 0.0f, b = 0.0f;
    for (int64_t c = threadIdx.x; c < t.cols; c += kLongThreads) {
        const float u = to_f32(g[c]) * (w ? to_f32(w[c]) : 1.0f);
        a += u;
        b = __builtin_fmaf(u, (to_f32(x[c]) - mean) * rstd, b);
    }
    block_sum2<kLongWaves>(a, b, lds);
    a /= (float)t.cols;
    b /= (float)t.cols;
    for (int64_t c = threadIdx.x; c < t.cols; c += kLongThreads) {
        const float u = to_f32(g[c]) * (w ? to_f32(w[c]) : 1.0f);
        const float xh = (to_f32(x[c]) - mean) * rstd;
        from_f32(dx[c], rstd * ((u - a) - xh * b));
    }
}

// The column sums of one slice of long rows, a thread a column.
constexpr int kThreads = 256;

template <typename T>
__global__ __launch_bounds__(kThreads) void norm_long_columns_kernel(NormGradTask t,
                                                                     int32_t splits) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int32_t split = blockIdx.y;
    if (c >= t.cols)
        return;
    const int64_t per = (t.rows + splits - 1) / splits;
    const int64_t r1 = per * (split + 1) < t.rows ? per * (split + 1) : t.rows;
    float dw = 0.0f, db = 0.0f;
    for (int64_t r = per * split; r < r1; ++r) {
        const float g = to_f32(((const T*)t.grad)[r * t.ldg + c]);
        const float xh = (to_f32(((const T*)t.x)[r * t.ldx + c]) - t.mean[r]) * t.rstd[r];
        dw = __builtin_fmaf(g, xh, dw);
        db += g;
    }
    t.part[(int64_t)split * t.cols + c] = dw;
    t.part[((int64_t)splits + split) * t.cols + c] = db;
}

// The workgroups' column sums, added in a fixed order: 64 columns a
// workgroup, 16 wavefronts with every sixteenth sum each.
constexpr int kJoinWaves = 16;

template <typename W>
__global__ __launch_bounds__(kJoinWaves * 64) void norm_join_kernel(NormGradTask t,
                                                                    int32_t splits) {
    __shared__ float sums[kJoinWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    const float* part = t.part + (int64_t)blockIdx.y * splits * t.cols;
    float s = 0.0f;
    if (c < t.cols) {
#pragma unroll 8
        for (int32_t i = wave; i < splits; i += kJoinWaves)
            s += part[(int64_t)i * t.cols + c];
    }
    sums[wave][lane] = s;
    __syncthreads();
    void* out = blockIdx.y == 0 ? t.dweight : t.dbias;
    if (wave != 0 || c >= t.cols || !out)
        return;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < kJoinWaves; ++i)
        s += sums[i][lane];
    from_f32(((W*)out)[c], s);
}

template <typename T, typename W>
hipError_t launch_norm_typed(const NormTask& t, hipStream_t stream) {
    const NormForm form = norm_form((int)sizeof(T), t.cols, false);
    const dim3 grid((uint32_t)norm_blocks(form, t.rows));
    if (form.waves == 0)
        return launch(norm_long_kernel<T, W>, grid, dim3(kLongThreads), 0, stream, t);
    return with_form<(int)sizeof(T), false>(form, [&](auto waves, auto nv) {
        return launch(norm_kernel<T, W, waves(), nv()>, grid,
                      dim3(RowPart<T, waves(), nv()>::THREADS), 0, stream, t);
    });
}

template <typename T, typename W>
hipError_t launch_norm_grad_typed(const NormGradTask& task, hipStream_t stream) {
    NormGradTask t = task;
    const bool sums = t.dweight || t.dbias;
    t.part = sums ? t.part : nullptr;
    const int32_t splits = norm_splits((int)sizeof(T), t.rows, t.cols);
    const NormForm form = norm_form((int)sizeof(T), t.cols, true);
    hipError_t e = hipSuccess;
    if (form.waves != 0) {
        if (t.rows > 0 || sums)
            e = with_form<(int)sizeof(T), true>(form, [&](auto waves, auto nv) {
                return launch(norm_grad_kernel<T, W, waves(), nv()>, dim3((uint32_t)splits),
                              dim3(RowPart<T, waves(), nv()>::THREADS), 0, stream, t);
            });
    } else {
        if (t.dx && t.rows > 0)
            e = launch(norm_long_dx_kernel<T, W>, dim3((uint32_t)t.rows), dim3(kLongThreads), 0,
                       stream, t);
        if (e == hipSuccess && sums)
            e = launch(norm_long_columns_kernel<T>,
                       dim3((uint32_t)((t.cols + kThreads - 1) / kThreads), (uint32_t)splits),
                       dim3(kThreads), 0, stream, t, splits);
    }
    if (e != hipSuccess || !sums)
        return e;
    return launch(norm_join_kernel<W>, dim3((uint32_t)((t.cols + 63) / 64), 2),
                  dim3(kJoinWaves * 64), 0, stream, t, splits);
}

}  // namespace

int64_t norm_threads(int esize, int64_t rows, int64_t cols) {
    const NormForm form = norm_form(esize, cols, false);
    return norm_blocks(form, rows) * (form.waves == 0 ? kLongThreads : form.threads());
}

hipError_t launch_norm(int esize, const NormTask& t, hipStream_t stream) {
    if (esize == 4)
        return launch_norm_typed<float, float>(t, stream);
    return t.wsize == 4 ? launch_norm_typed<uint16_t, float>(t, stream)
                        : launch_norm_typed<uint16_t, uint16_t>(t, stream);
}

// Workgroups of the backward pass, each of which leaves a row of sums: 2 a CU,
// for long rows slices of 64 rows.
int32_t norm_splits(int esize, int64_t rows, int64_t cols) {
    const NormForm form = norm_form(esize, cols, true);
    int64_t s = form.waves == 0 ? (rows + 63) / 64 : form.waves == 1 ? (rows + 3) / 4 : rows;
    const int64_t most = form.waves == 0 ? 64 : 512;
    s = s > most ? most : s;
    return (int32_t)(s < 1 ? 1 : s);
}

int64_t norm_grad_threads(int esize, int64_t rows, int64_t cols, bool dx, bool sums) {
    const NormForm form = norm_form(esize, cols, true);
    const int64_t splits = norm_splits(esize, rows, cols);
    int64_t most = form.waves != 0 ? splits * form.threads() : dx ? rows * kLongThreads : 0;
    if (sums) {
        const int64_t columns = form.waves == 0 ? (cols + kThreads - 1) / kThreads * kThreads * splits
                                                : 0;
        const int64_t join = (cols + 63) / 64 * 64 * kJoinWaves * 2;
        most = columns > most ? columns : most;
        most = join > most ? join : most;
    }
    return most;
}

hipError_t launch_norm_grad(int esize, const NormGradTask& t, hipStream_t stream) {
    if (esize == 4)
        return launch_norm_grad_typed<float, float>(t, stream);
    return t.wsize == 4 ? launch_norm_grad_typed<uint16_t, float>(t, stream)
                        : launch_norm_grad_typed<uint16_t, uint16_t>(t, stream);
}

}  // namespace vpa
