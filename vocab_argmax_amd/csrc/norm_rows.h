// norm_rows.h -- what the norms (layer_norm.hip, rms_norm.hip) share: a row of a
// matrix in the registers of one or several wavefronts, and which of these
// forms a row takes.
#pragma once

#include <type_traits>

#include "vpa_internal.h"
#include "vpa_math.h"

namespace vpa {
namespace {

// A thread's part of a row: NV vectors of VEC elements, vector i at column
// (i * WAVES * 64 + thread) * VEC, and how many elements of each exist.
template <typename T, int WAVES, int NV>
struct RowPart {
    static constexpr int VEC = 16 / (int)sizeof(T);
    // a workgroup of single wavefronts works on 4 rows at a time
    static constexpr int ROWS = WAVES == 1 ? 4 : 1;
    static constexpr int THREADS = WAVES * 64 * ROWS;

    static __device__ __forceinline__ int column(int i) {
        return (i * WAVES * 64 + (int)threadIdx.x % (WAVES * 64)) * VEC;
    }
    static __device__ __forceinline__ int64_t first_row() {
        return (int64_t)blockIdx.x * ROWS + threadIdx.x / (WAVES * 64);
    }
    static __device__ __forceinline__ int64_t row_step() {
        return (int64_t)gridDim.x * ROWS;
    }
    static __device__ __forceinline__ int count(int i, int cols) {
        const int n = cols - column(i);
        return n < 0 ? 0 : n > VEC ? VEC : n;
    }
    static __device__ __forceinline__ void load(const T* row, int cols, u32x4_t (&v)[NV]) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int n = count(i, cols);
            if (n == VEC) {
                v[i] = ((const Loose16*)(row + column(i)))->v;
            } else {
                union {
                    T e[VEC];
                    u32x4_t v;
                } u;
                u.v = u32x4_t{0, 0, 0, 0};
#pragma unroll
                for (int e = 0; e < VEC - 1; ++e)
                    if (e < n)
                        u.e[e] = row[column(i) + e];
                v[i] = u.v;
            }
        }
    }
    // `value` in every place past the row's end
    static __device__ __forceinline__ void fill_past(T value, int cols, u32x4_t (&v)[NV]) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            union {
                T e[VEC];
                u32x4_t v;
            } u;
            u.v = v[i];
            const int n = count(i, cols);
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                u.e[e] = e < n ? u.e[e] : value;
            v[i] = u.v;
        }
    }
    // rounded to T
    static __device__ __forceinline__ u32x4_t pack(const float (&f)[VEC]) {
        u32x4_t v;
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = pack_bf16(f[2 * e], f[2 * e + 1]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = __builtin_bit_cast(uint32_t, f[e]);
        }
        return v;
    }
    static __device__ __forceinline__ void store_packed(T* row, int cols, int i, u32x4_t v) {
        const int n = count(i, cols);
        if (n == VEC) {
            // past the L2 (32768 x 4096 forward 105 -> 87 us; loads past it are slower)
            __builtin_nontemporal_store(v, &((Loose16*)(row + column(i)))->v);
        } else {
            union {
                T e[VEC];
                u32x4_t v;
            } u;
            u.v = v;
#pragma unroll
            for (int e = 0; e < VEC - 1; ++e)
                if (e < n)
                    row[column(i) + e] = u.e[e];
        }
    }
    static __device__ __forceinline__ void store(T* row, int cols, int i,
                                                 const float (&f)[VEC]) {
        store_packed(row, cols, i, pack(f));
    }
    // weights or biases: `none` where there are none
    template <typename W>
    static __device__ __forceinline__ void load_weights(const W* w, int cols, float none,
                                                        float (&f)[NV][VEC]) {
        constexpr int WVEC = 16 / (int)sizeof(W);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = column(i);
            if (w && c + VEC <= cols) {
#pragma unroll
                for (int h = 0; h < VEC / WVEC; ++h) {
                    const u32x4_t v = ((const Loose16*)(w + c + h * WVEC))->v;
#pragma unroll
                    for (int e = 0; e < WVEC; ++e)
                        f[i][h * WVEC + e] = vec_elem<(int)sizeof(W)>(v, e);
                }
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    f[i][e] = w && c + e < cols ? to_f32(w[c + e]) : none;
            }
        }
    }
};

constexpr int kLongWaves = 16;
constexpr int kLongThreads = kLongWaves * 64;

// The smallest form that holds a row: one wavefront with 1 vector a lane, 4
// with 1 or 2, 8 with 2 or 4; 0 where none does.  8 wavefronts with 4 vectors
// of bf16 leave the backward pass's sums no registers.
struct NormForm {
    int waves, nv;
    // of a workgroup (as RowPart's): single wavefronts work on 4 rows at a time
    int rows() const { return waves == 1 ? 4 : 1; }
    int threads() const { return waves * rows() * 64; }
};
inline NormForm norm_form(int esize, int64_t cols, bool grad) {
    const int64_t vecs = (cols * esize + 15) / 16;      // 16-byte vectors of a row
    if (vecs <= 64)
        return {1, 1};
    if (vecs <= 512)
        return {4, vecs <= 256 ? 1 : 2};
    if (vecs <= 1024)
        return {8, 2};
    return vecs <= 2048 && !(grad && esize == 2) ? NormForm{8, 4} : NormForm{0, 0};
}

// Workgroups of the forward pass: 16 wavefronts a CU, which walk over the rows,
// so that each has several for its weights; long rows have a workgroup each.
inline int64_t norm_blocks(NormForm form, int64_t rows) {
    if (form.waves == 0)
        return rows;
    const int64_t most = 4096 * 64 / form.threads();
    const int64_t need = (rows + form.rows() - 1) / form.rows();
    return need < most ? need : most;
}

// Calls f(WAVES, NV), as types, for the form.
template <int ESIZE, bool GRAD, typename F>
hipError_t with_form(NormForm form, F f) {
    using std::integral_constant;
    if (form.waves == 1)
        return f(integral_constant<int, 1>{}, integral_constant<int, 1>{});
    if (form.waves == 4)
        return form.nv == 1 ? f(integral_constant<int, 4>{}, integral_constant<int, 1>{})
                            : f(integral_constant<int, 4>{}, integral_constant<int, 2>{});
    if constexpr (!GRAD || ESIZE == 4)
        if (form.nv == 4)
            return f(integral_constant<int, 8>{}, integral_constant<int, 4>{});
    return f(integral_constant<int, 8>{}, integral_constant<int, 2>{});
}

}  // namespace
}  // namespace vpa
