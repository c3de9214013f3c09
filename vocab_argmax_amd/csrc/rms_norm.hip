// rms_norm.hip -- root-mean-square norm over the rows of a matrix, with the
// residual's addition before it and, where asked for, an output in 8 bits with
// a scale for each block of 128 columns; its backward pass; and the same 8-bit
// form of a matrix as it is.
//
// The sum of squares is of 64 bits: squares leave fp32 for values past 1.8e19, or a
// row's sum of them well before, and for values below 1e-23.  The norm is taken of
// the sum as it is stored (rounded to its type), which is what the backward pass
// reads.
#include "norm_rows.h"
#include "vpa_draft_internal.h"

namespace vpa {
namespace {

constexpr int kThreads = 256;
constexpr float kFp8Max = 448.0f;
constexpr uint32_t kAmaxLeast = 0x0D800000u;       // 2^-100

// Quotients by d, those of a division rounded once: a product with a rounded inverse
// puts a tie of e4m3 in fourteen on the wrong side.  The inverse is in two parts, the
// second what the first one's rounding left: together they give y / d to 2^-46, so q
// within its last place, and one step by the remainder, which a multiply-add has
// exactly, the nearest fp32 value.
struct Divisor {
    float d, inverse, rest;
    __device__ __forceinline__ float quotient(float y) const {
        const float q = __builtin_fmaf(y, inverse, y * rest);
        return copysignf(__builtin_fmaf(__builtin_fmaf(-d, q, y), inverse, q), y);
    }
};
constexpr Divisor kByFp8Max = {kFp8Max, (float)(1.0 / kFp8Max),
                               (float)(1.0 / kFp8Max - (double)(float)(1.0 / kFp8Max))};

// A block's scale from the largest |y| as fp32 bits, which sort as the values do,
// infinity and NaN last.
__device__ __forceinline__ Divisor block_scale(uint32_t amax_bits) {
    if (amax_bits >= 0x7F800000u)
        return {__builtin_nanf(""), __builtin_nanf(""), 0.0f};
    const Divisor by = kByFp8Max;
    const float scale = by.quotient(
        __builtin_bit_cast(float, amax_bits < kAmaxLeast ? kAmaxLeast : amax_bits));
    const float inverse = 1.0f / scale;
    return {scale, inverse, __builtin_fmaf(-scale, inverse, 1.0f) * inverse};
}
__device__ __forceinline__ uint32_t abs_bits(float f) {
    return __builtin_bit_cast(uint32_t, f) & 0x7FFFFFFFu;
}
// Two values in 8 bits, to nearest even (NaN stays NaN): bits 0-7 and 8-15.  The
// instruction makes 448 of everything up to 464 (measured), so quotients that the
// scale's rounding leaves above 448, by a step or two of fp32, need no clamp.
__device__ __forceinline__ uint32_t pack_fp8(float a, float b) {
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false) & 0xFFFFu;
}

// Sum over a workgroup of WAVES wavefronts through `lds`; every thread holds it.
// Callers leave a barrier between two uses of an lds.
template <int WAVES, typename S>
__device__ __forceinline__ S block_sum(S a, S (&lds)[WAVES]) {
    if constexpr (std::is_same_v<S, double>)
        a = wave_sum_f64(a);
    else
        a = wave_sum(a);
    if constexpr (WAVES > 1) {
        if ((threadIdx.x & 63) == 0)
            lds[threadIdx.x >> 6] = a;
        __syncthreads();
        a = 0;
#pragma unroll
        for (int i = 0; i < WAVES; ++i)
            a += lds[i];
    }
    return a;
}

// 1 / sqrt(v), within 2.5 steps of 2^-24: in fp32, of v's part in [1/2, 2).
__device__ __forceinline__ float inverse_root(double v) {
    const int half = __builtin_amdgcn_frexp_exp(v) >> 1;            // 0 for 0, infinity and NaN
    const float part = (float)__builtin_amdgcn_ldexp(v, -2 * half);
    return __builtin_amdgcn_ldexpf(1.0f / sqrtf(part), -half);
}

// The largest over aligned groups of LANES (16 or 32) lanes.
template <int LANES>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
    const auto step = [&](uint32_t o) { v = o > v ? o : v; };
    step(dpp_move<dpp::kSwap1, 0xF>(v));
    step(dpp_move<dpp::kSwap2, 0xF>(v));
    step(dpp_move<dpp::kHalfMirror, 0xF>(v));
    step(dpp_move<dpp::kMirror, 0xF>(v));
    if constexpr (LANES == 32)
        step(__shfl_xor(v, 16, 64));
    return v;
}

// N bytes at any address.
template <int N>
struct __attribute__((packed, aligned(1))) LooseBytes {
    uint32_t w[N / 4];
};

// A row in registers: x and the residual of the next one on their way, the weights
// kept over a workgroup's rows.  With FP8, the 128 columns of a scale lie in 16
// (bf16) or 32 (fp32) lanes side by side.  Bound by memory: 8192 x 4096 bf16 with
// a residual 45 us (6.0 TB/s), with y in 8 bits 40 (5.9); 32 rows 4.4, latency.
template <typename T, typename W, int WAVES, int NV, bool FP8>
__global__ __launch_bounds__(WAVES == 1 ? 256 : WAVES * 64) void rms_kernel(RmsTask t) {
    using P = RowPart<T, WAVES, NV>;
    constexpr int VEC = P::VEC, ESIZE = (int)sizeof(T), LANES = kScaleBlock / VEC;
    __shared__ double lds[2][WAVES];
    const int cols = (int)t.cols;
    const double inv_cols = 1.0 / (double)cols;
    const bool res = t.residual != nullptr;
    float w[NV][VEC];
    P::load_weights((const W*)t.weight, cols, 1.0f, w);
    u32x4_t next[NV], next_r[NV];
    int64_t row = P::first_row();
    const auto fetch = [&](int64_t r) {
        P::load((const T*)t.x + r * t.ldx, cols, next);
        if (res)
            P::load((const T*)t.residual + r * t.ldr, cols, next_r);
    };
    if (row < t.rows)
        fetch(row);
    for (int turn = 0; row < t.rows; row += P::row_step(), turn ^= 1) {
        u32x4_t v[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i)
            v[i] = next[i];
        if (res) {
            T* s = (T*)t.summed + row * t.lds;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float f[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    f[e] = vec_elem<ESIZE>(v[i], e) + vec_elem<ESIZE>(next_r[i], e);
                v[i] = P::pack(f);
                P::store_packed(s, cols, i, v[i]);
            }
        }
        const int64_t after = row + P::row_step();
        // (outputs may take the inputs' places: the next row is another)
        if (after < t.rows)
            fetch(after);
        double q = 0.0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const double f = vec_elem<ESIZE>(v[i], e);          // 0 past the row
                q = __builtin_fma(f, f, q);
            }
        q = block_sum<WAVES>(q, lds[turn]);
        const float rstd = inverse_root(__builtin_fma(q, inv_cols, (double)t.eps));
        if (t.rstd && P::column(0) == 0)
            t.rstd[row] = rstd;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float f[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                f[e] = vec_elem<ESIZE>(v[i], e) * rstd * w[i][e];
            if constexpr (!FP8) {
                P::store((T*)t.y + row * t.ldy, cols, i, f);
            } else {
                const int n = P::count(i, cols);
                uint32_t amax = 0;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const uint32_t b = e < n ? abs_bits(f[e]) : 0;
                    amax = b > amax ? b : amax;
                }
                const Divisor sc = block_scale(group_max<LANES>(amax));
                LooseBytes<VEC> o;
#pragma unroll
                for (int e = 0; e < VEC; e += 4)
                    o.w[e / 4] = pack_fp8(sc.quotient(f[e]), sc.quotient(f[e + 1])) |
                                 pack_fp8(sc.quotient(f[e + 2]), sc.quotient(f[e + 3])) << 16;
                uint8_t* y = (uint8_t*)t.y + row * t.ldy + P::column(i);
                if (n == VEC) {
                    *(LooseBytes<VEC>*)y = o;
                } else {
#pragma unroll
                    for (int e = 0; e < VEC - 1; ++e)
                        if (e < n)
                            y[e] = (uint8_t)(o.w[e / 4] >> (e % 4 * 8));
                }
                if (n > 0 && P::column(i) % kScaleBlock == 0)
                    t.scale[row * t.ld_scale + P::column(i) / kScaleBlock] = sc.d;
            }
        }
    }
}

// The gradients of a workgroup's rows from one read of grad, s and grad_summed,
// the weight's in registers until the end (a thread always has the same columns).
// Bound by memory: 8192 x 4096 bf16 with grad_summed 45 us, 6.2 TB/s.
template <typename T, typename W, int WAVES, int NV>
__global__ __launch_bounds__(WAVES == 1 ? 256 : WAVES * 64) void rms_grad_kernel(RmsGradTask t) {
    using P = RowPart<T, WAVES, NV>;
    constexpr int VEC = P::VEC, ESIZE = (int)sizeof(T);
    __shared__ float lds[2][WAVES];
    const int cols = (int)t.cols;
    const bool along = t.grad_summed != nullptr && t.dx != nullptr;
    float w[NV][VEC], dw[NV][VEC] = {};
    P::load_weights((const W*)t.weight, cols, 1.0f, w);
    u32x4_t next_g[NV], next_x[NV], next_s[NV];
    float next_rstd = 0.0f;
    const auto fetch = [&](int64_t r) {
        P::load((const T*)t.grad + r * t.ldg, cols, next_g);
        P::load((const T*)t.summed + r * t.lds, cols, next_x);
        if (along)
            P::load((const T*)t.grad_summed + r * t.ldgs, cols, next_s);
        next_rstd = t.rstd[r];
    };
    int64_t row = P::first_row();
    if (row < t.rows)
        fetch(row);
    for (int turn = 0; row < t.rows; row += P::row_step(), turn ^= 1) {
        u32x4_t g[NV], x[NV], gs[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            g[i] = next_g[i];
            x[i] = next_x[i];
            gs[i] = next_s[i];
        }
        const float rstd = next_rstd;
        const int64_t after = row + P::row_step();
        // (grad_x may take grad's or grad_summed's place: the next row is another)
        if (after < t.rows)
            fetch(after);
        float b = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float gr = vec_elem<ESIZE>(g[i], e);          // 0 past the row
                const float xh = vec_elem<ESIZE>(x[i], e) * rstd;
                b = __builtin_fmaf(gr * w[i][e], xh, b);
                dw[i][e] = __builtin_fmaf(gr, xh, dw[i][e]);
            }
        if (!t.dx)
            continue;
        b = block_sum<WAVES>(b, lds[turn]) / (float)cols;
        T* dx = (T*)t.dx + row * t.lddx;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float f[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float xh = vec_elem<ESIZE>(x[i], e) * rstd;
                f[e] = rstd * (vec_elem<ESIZE>(g[i], e) * w[i][e] - xh * b);
                if (along)
                    f[e] += vec_elem<ESIZE>(gs[i], e);
            }
            P::store(dx, cols, i, f);
        }
    }
    if (!t.part)
        return;
    if constexpr (P::ROWS > 1) {
        // the workgroup's rows' sums, added in order
        static_assert(NV == 1, "a wavefront a row");
        __shared__ float sums[P::ROWS][64 * VEC];
        const int group = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            sums[group][lane * VEC + e] = dw[0][e];
        __syncthreads();
        for (int c = threadIdx.x; c < 64 * VEC && c < cols; c += P::THREADS) {
            float s = 0.0f;
#pragma unroll
            for (int r = 0; r < P::ROWS; ++r)
                s += sums[r][c];
            t.part[(int64_t)blockIdx.x * cols + c] = s;
        }
        return;
    }
    float* pw = t.part + (int64_t)blockIdx.x * cols;
    typedef float f32x4_loose __attribute__((ext_vector_type(4), aligned(4)));
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VEC; e += 4) {
            const int c = P::column(i) + e;
            if (c + 4 <= cols) {
                *(f32x4_loose*)(pw + c) = f32x4_loose{dw[i][e], dw[i][e + 1], dw[i][e + 2],
                                                      dw[i][e + 3]};
                continue;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (c + k < cols)
                    pw[c + k] = dw[i][e + k];
        }
}

// Rows too long for a workgroup's registers: several passes over the row, which the
// caches hold, an element a lane: 4096 x 12288 bf16 backward 284 us, 1.8 TB/s.
template <typename T, typename W>
__global__ __launch_bounds__(kLongThreads) void rms_long_kernel(RmsTask t) {
    __shared__ double lds[kLongWaves];
    const int64_t row = blockIdx.x;
    const T* x = (const T*)t.x + row * t.ldx;
    const T* r = t.residual ? (const T*)t.residual + row * t.ldr : nullptr;
    T* s = t.residual ? (T*)t.summed + row * t.lds : nullptr;
    const W* w = (const W*)t.weight;
    double q = 0.0;
    for (int64_t c = threadIdx.x; c < t.cols; c += kLongThreads) {
        float v = to_f32(x[c]);
        if (r) {
            T sum;
            from_f32(sum, v + to_f32(r[c]));
            s[c] = sum;
            v = to_f32(sum);
        }
        q = __builtin_fma((double)v, (double)v, q);
    }
    q = block_sum<kLongWaves>(q, lds);
    const float rstd = inverse_root(q / (double)t.cols + (double)t.eps);
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
        const Divisor sc = block_scale(amax);
        const uint32_t p = pack_fp8(sc.quotient(v0), sc.quotient(v1));
        if (c < t.cols)
            y[c] = (uint8_t)p;
        if (c + 1 < t.cols)
            y[c + 1] = (uint8_t)(p >> 8);
        if (lane == 0)
            t.scale[row * t.ld_scale + b] = sc.d;
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
// wavefronts with every sixteenth sum each.  512 x 4096 sums 4.2 us, a launch and
// two rounds of loads.
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

// A matrix as it is in 8 bits.  LANES lanes side by side hold 128 columns of a row,
// 16 bytes each; a workgroup takes kThreads / LANES rows of one block of columns at
// a time, or with SQUARE the 128 rows that share a scale, in registers.  Bound by
// memory: 151936 x 2048 bf16 179 us (5.3 TB/s), in blocks of 128 x 128 165 (5.7).
template <typename T, bool SQUARE>
__global__ __launch_bounds__(kThreads) void quant_kernel(QuantTask t, int64_t blocks_across) {
    constexpr int VEC = 16 / (int)sizeof(T), LANES = kScaleBlock / VEC;
    constexpr int ROWS = kThreads / LANES, NV = SQUARE ? kScaleBlock / ROWS : 1;
    __shared__ uint32_t lds[kThreads / 64];
    const int64_t down = blockIdx.x / blocks_across, across = blockIdx.x % blocks_across;
    const int64_t r0 = down * (SQUARE ? kScaleBlock : ROWS) + threadIdx.x / LANES;
    const int64_t c = across * kScaleBlock + threadIdx.x % LANES * VEC;
    const int n = t.cols - c < VEC ? (int)(t.cols - c) : VEC;   // columns of this lane, or < 1
    u32x4_t v[NV];
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t r = r0 + i * ROWS;
        const T* x = (const T*)t.x + r * t.ldx + c;
        v[i] = u32x4_t{0, 0, 0, 0};
        if (r < t.rows && n == VEC) {
            v[i] = ((const Loose16*)x)->v;
        } else if (r < t.rows) {
            union {
                T e[VEC];
                u32x4_t v;
            } u;
            u.v = v[i];
#pragma unroll
            for (int e = 0; e < VEC - 1; ++e)
                if (e < n)
                    u.e[e] = x[e];
            v[i] = u.v;
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const uint32_t b = abs_bits(vec_elem<(int)sizeof(T)>(v[i], e));
            amax = b > amax ? b : amax;
        }
    }
    amax = group_max<LANES>(amax);
    if constexpr (SQUARE) {
#pragma unroll
        for (int off = LANES; off < 64; off <<= 1) {
            const uint32_t o = __shfl_xor(amax, off, 64);
            amax = o > amax ? o : amax;
        }
        if ((threadIdx.x & 63) == 0)
            lds[threadIdx.x >> 6] = amax;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kThreads / 64; ++i)
            amax = lds[i] > amax ? lds[i] : amax;
    }
    const Divisor sc = block_scale(amax);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t r = r0 + i * ROWS;
        if (r >= t.rows)
            continue;
        LooseBytes<VEC> o;
        const auto f = [&](int e) { return sc.quotient(vec_elem<(int)sizeof(T)>(v[i], e)); };
#pragma unroll
        for (int e = 0; e < VEC; e += 4)
            o.w[e / 4] = pack_fp8(f(e), f(e + 1)) | pack_fp8(f(e + 2), f(e + 3)) << 16;
        uint8_t* y = (uint8_t*)t.y + r * t.ldy + c;
        if (n == VEC) {
            *(LooseBytes<VEC>*)y = o;
        } else {
#pragma unroll
            for (int e = 0; e < VEC - 1; ++e)
                if (e < n)
                    y[e] = (uint8_t)(o.w[e / 4] >> (e % 4 * 8));
        }
        if (!SQUARE && threadIdx.x % LANES == 0)
            t.scale[r * t.ld_scale + across] = sc.d;
    }
    if (SQUARE && threadIdx.x == 0)
        t.scale[down * t.ld_scale + across] = sc.d;
}

template <typename T, typename W>
hipError_t launch_rms_typed(const RmsTask& t, hipStream_t stream) {
    const NormForm form = norm_form((int)sizeof(T), t.cols, false);
    const dim3 grid((uint32_t)norm_blocks(form, t.rows));
    if (form.waves == 0)
        return launch(rms_long_kernel<T, W>, grid, dim3(kLongThreads), 0, stream, t);
    return with_form<(int)sizeof(T), false>(form, [&](auto waves, auto nv) {
        const dim3 block(RowPart<T, waves(), nv()>::THREADS);
        return t.scale ? launch(rms_kernel<T, W, waves(), nv(), true>, grid, block, 0, stream, t)
                       : launch(rms_kernel<T, W, waves(), nv(), false>, grid, block, 0, stream, t);
    });
}

template <typename T, typename W>
hipError_t launch_rms_grad_typed(const RmsGradTask& task, hipStream_t stream) {
    RmsGradTask t = task;
    t.part = t.dweight && t.rows > 0 ? t.part : nullptr;
    // no rows: no sums, and the joining kernel writes 0
    const int32_t splits = t.rows > 0 ? rms_splits((int)sizeof(T), t.rows, t.cols) : 0;
    const NormForm form = norm_form((int)sizeof(T), t.cols, true);
    hipError_t e = hipSuccess;
    if (t.rows > 0 && form.waves != 0) {
        e = with_form<(int)sizeof(T), true>(form, [&](auto waves, auto nv) {
            return launch(rms_grad_kernel<T, W, waves(), nv()>, dim3((uint32_t)splits),
                          dim3(RowPart<T, waves(), nv()>::THREADS), 0, stream, t);
        });
    } else if (t.rows > 0) {
        if (t.dx)
            e = launch(rms_long_dx_kernel<T, W>, dim3((uint32_t)t.rows), dim3(kLongThreads), 0,
                       stream, t);
        if (e == hipSuccess && t.dweight)
            e = launch(rms_long_columns_kernel<T>,
                       dim3((uint32_t)((t.cols + kThreads - 1) / kThreads), (uint32_t)splits),
                       dim3(kThreads), 0, stream, t, splits);
    }
    if (e != hipSuccess || !t.dweight)
        return e;
    return launch(rms_join_kernel<W>, dim3((uint32_t)((t.cols + 63) / 64)), dim3(kJoinWaves * 64), 0,
                  stream, t, splits);
}

}  // namespace

int64_t rms_threads(int esize, int64_t rows, int64_t cols) {
    const NormForm form = norm_form(esize, cols, false);
    return norm_blocks(form, rows) * (form.waves == 0 ? kLongThreads : form.threads());
}

hipError_t launch_rms(int esize, const RmsTask& t, hipStream_t stream) {
    if (esize == 4)
        return launch_rms_typed<float, float>(t, stream);
    return t.wsize == 4 ? launch_rms_typed<uint16_t, float>(t, stream)
                        : launch_rms_typed<uint16_t, uint16_t>(t, stream);
}

// Workgroups of the backward pass, each of which leaves a row of sums: 2 a CU (8192 x
// 4096 bf16 53 us, with 1 52, with 4 61); up to 4 of those with one vector a lane,
// as long as each has 16 rows (16384 x 1600 45 us, with 2 50; 8192 x 1024 fp32, 512
// of them, 29, with 4 32) or, where they leave half of the lanes idle, 8 (8192 x 513
// 24, with 2 33).  For long rows slices of 64 rows.
int32_t rms_splits(int esize, int64_t rows, int64_t cols) {
    const NormForm form = norm_form(esize, cols, true);
    int64_t s = form.waves == 0 ? (rows + 63) / 64 : form.waves == 1 ? (rows + 3) / 4 : rows;
    int64_t most = form.waves == 0 ? 64 : 512;
    if (form.nv == 1) {
        const int64_t each = rows / (cols * esize <= form.threads() * 8 ? 8 : 16);
        most = each > 1024 ? 1024 : each > most ? each : most;
    }
    s = s > most ? most : s;
    return (int32_t)(s < 1 ? 1 : s);
}

int64_t rms_grad_threads(int esize, int64_t rows, int64_t cols, bool dx, bool sums) {
    const NormForm form = norm_form(esize, cols, true);
    const int64_t splits = rms_splits(esize, rows, cols);
    int64_t most = form.waves != 0 ? splits * form.threads() : dx ? rows * kLongThreads : 0;
    if (sums) {
        const int64_t columns =
            form.waves == 0 ? (cols + kThreads - 1) / kThreads * kThreads * splits : 0;
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

namespace {

// Workgroups down the rows.
int64_t quant_down(int esize, int64_t rows, int32_t block_rows) {
    const int64_t per = block_rows == 1 ? kThreads / (kScaleBlock * esize / 16) : block_rows;
    return (rows + per - 1) / per;
}

template <typename T>
hipError_t launch_quant_typed(const QuantTask& t, hipStream_t stream) {
    const int64_t across = (t.cols + kScaleBlock - 1) / kScaleBlock;
    const dim3 grid((uint32_t)(quant_down((int)sizeof(T), t.rows, t.block_rows) * across));
    return t.block_rows == 1
               ? launch(quant_kernel<T, false>, grid, dim3(kThreads), 0, stream, t, across)
               : launch(quant_kernel<T, true>, grid, dim3(kThreads), 0, stream, t, across);
}

}  // namespace

int64_t quant_threads(int esize, int64_t rows, int64_t cols, int32_t block_rows) {
    return quant_down(esize, rows, block_rows) * ((cols + kScaleBlock - 1) / kScaleBlock) * kThreads;
}

hipError_t launch_quant(int esize, const QuantTask& t, hipStream_t stream) {
    return esize == 2 ? launch_quant_typed<uint16_t>(t, stream) : launch_quant_typed<float>(t, stream);
}

}  // namespace vpa
