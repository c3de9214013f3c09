// linear.hip -- the head's products: y = residual + act(x W^T + bias) and the
// products of its backward pass.  This file plans a product (which kernel,
// tile and split of k), joins the slices of a split one and computes dz.
#include "linear_common.h"
#include "vpa_head_internal.h"
#include "vpa_math.h"

namespace vpa {
namespace {

constexpr int kThreads = 256;

// The slices of a split product, added in order, and its epilogue: 4 results
// of a row a thread (one where a row is not a multiple of 4).
template <typename T, bool FOUR>
__global__ __launch_bounds__(kThreads) void gemm_join_kernel(GemmTask t, int32_t slices) {
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const float* part = (const float*)t.ws;
    const int64_t slice = t.m * t.n;
    if constexpr (FOUR) {
        if (id * 4 >= slice)
            return;
        f32x4 v = *(const f32x4*)(part + id * 4);
        for (int32_t s = 1; s < slices; ++s)
            v += *(const f32x4*)(part + s * slice + id * 4);
        const int64_t m = id / (t.n / 4);
        store_results<T>(t, m, id * 4 - m * t.n, v);
    } else {
        if (id >= slice)
            return;
        float v = part[id];
        for (int32_t s = 1; s < slices; ++s)
            v += part[s * slice + id];
        const int64_t m = id / t.n;
        store_result<T>(t, m, id - m * t.n, v);
    }
}

// 8 consecutive elements of a row, as loaded and stored (past the L2) in
// 16-byte accesses.
template <typename T>
struct Eight {
    static constexpr int CHUNKS = (int)sizeof(T) / 2, VEC = 16 / (int)sizeof(T);
    u32x4_t v[CHUNKS];
    // the first n of them, 0 after them
    __device__ __forceinline__ void load(const T* p, int n) {
        if (n == 8) {
#pragma unroll
            for (int h = 0; h < CHUNKS; ++h)
                v[h] = ((const Loose16*)(p + h * VEC))->v;
            return;
        }
        union {
            T e[8];
            u32x4_t v[CHUNKS];
        } u;
#pragma unroll
        for (int h = 0; h < CHUNKS; ++h)
            u.v[h] = u32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n)
                u.e[i] = p[i];
#pragma unroll
        for (int h = 0; h < CHUNKS; ++h)
            v[h] = u.v[h];
    }
    __device__ __forceinline__ float operator[](int i) const {
        return vec_elem<(int)sizeof(T)>(v[i / VEC], i % VEC);
    }
    static __device__ __forceinline__ void store(T* p, int n, const float (&d)[8]) {
        if (n == 8) {
            if constexpr (sizeof(T) == 2) {
                const u32x4_t u = {pack_bf16(d[0], d[1]), pack_bf16(d[2], d[3]),
                                   pack_bf16(d[4], d[5]), pack_bf16(d[6], d[7])};
                __builtin_nontemporal_store(u, &((Loose16*)p)->v);
            } else {
                store4(p, f32x4{d[0], d[1], d[2], d[3]});
                store4(p + 4, f32x4{d[4], d[5], d[6], d[7]});
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n)
                from_f32(p[i], d[i]);
    }
};

// dz = grad * act'(pre), rounded to the operands' type as the matrix cores
// take it, and the slices of its column sums, which are of the values before
// that rounding.  For bf16 that rounding and pre's are half a step each, as in
// a bf16 training step whose saved tensors are bf16: with silu at 4096^3 the
// gradients of x and the weight are 0.0024 off 64 bits, of which the rounding
// of the results alone is 0.0017; an fp32 pre would make it 0.00235, and a
// second product with what dz's rounding dropped would double the time.
//
// A workgroup takes 512 columns, 8 a lane, and each of its 4 wavefronts every
// fourth row of its slice of rows, kDzRows of them loaded at a time.  Bound by
// memory: 2048 x 50257 bf16 copied in 85 us, 4.9 TB/s, as a large copy (93
// with a row at a time).
constexpr int kDzCols = 512, kDzRows = 4;

template <typename T, typename G, int ACT>
__global__ __launch_bounds__(kThreads) void dz_kernel(DzTask t, int32_t splits) {
    __shared__ float sums[4][kDzCols];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * kDzCols + lane * 8;
    const int64_t per = (t.rows + splits - 1) / splits;
    const int64_t r0 = per * blockIdx.y, r1 = r0 + per < t.rows ? r0 + per : t.rows;
    const int n = t.cols - c < 8 ? (int)(t.cols - c) : 8;       // columns of this lane, or < 1
    float sum[8] = {};
    for (int64_t r = r0 + wave; r < r1; r += 4 * kDzRows) {
        Eight<G> g[kDzRows];
        Eight<T> z[kDzRows];
#pragma unroll
        for (int k = 0; k < kDzRows; ++k)
            if (r + 4 * k < r1) {
                g[k].load((const G*)t.grad + (r + 4 * k) * t.ldg + c, n);
                if constexpr (ACT != VPA_ACT_NONE)
                    z[k].load((const T*)t.pre + (r + 4 * k) * t.ldp + c, n);
            }
#pragma unroll
        for (int k = 0; k < kDzRows; ++k) {
            if (r + 4 * k >= r1)
                break;
            float d[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                d[i] = g[k][i];
                if constexpr (ACT != VPA_ACT_NONE)
                    d[i] *= act_slope<ACT>(z[k][i]);
                sum[i] += d[i];
            }
            if (t.dz && n > 0)
                Eight<T>::store((T*)t.dz + (r + 4 * k) * t.ldz + c, n, d);
        }
    }
    if (!t.part)
        return;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        sums[wave][lane * 8 + i] = sum[i];
    __syncthreads();
    for (int i = threadIdx.x; i < kDzCols; i += kThreads) {
        const int64_t col = (int64_t)blockIdx.x * kDzCols + i;
        if (col < t.cols)
            t.part[(int64_t)blockIdx.y * t.cols + col] =
                ((sums[0][i] + sums[1][i]) + sums[2][i]) + sums[3][i];
    }
}

// The slices' column sums, added in a fixed order: 64 columns a workgroup, 16
// wavefronts with every sixteenth slice each (4096 x 4096, 256 slices: a
// thread a column took 50 us).
constexpr int kFinishWaves = 16;

template <typename T>
__global__ __launch_bounds__(kFinishWaves * 64) void bias_finish_kernel(DzTask t, int32_t splits) {
    __shared__ float sums[kFinishWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    float sum = 0.0f;
    if (c < t.cols) {
#pragma unroll 4
        for (int32_t s = wave; s < splits; s += kFinishWaves)
            sum += t.part[(int64_t)s * t.cols + c];
    }
    sums[wave][lane] = sum;
    __syncthreads();
    if (wave != 0 || c >= t.cols)
        return;
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kFinishWaves; ++i)
        sum += sums[i][lane];
    from_f32(((T*)t.bias)[c], sum);
}

// Direct loads move 16 bytes at a time: an operand with contiguous k needs
// rows at 16-byte aligned addresses, one with contiguous rows a multiple of
// 16 bytes of them too.  Offsets within a tile are 32 bits.
bool direct_operand(int esize, const void* p, int64_t ld, bool k1, int64_t rows) {
    const int64_t vec = 16 / esize;
    return (uintptr_t)p % 16 == 0 && ld % vec == 0 && ld <= ((int64_t)1 << 21) &&
           (k1 || rows % vec == 0);
}

// Stages of 128 bytes of k (no k: one, which stores zeros).
int64_t stages_of(int esize, int64_t k) {
    return k > 0 ? (k * esize + 127) / 128 : 1;
}

template <typename T, typename G>
hipError_t launch_dz_typed(const DzTask& t, hipStream_t stream) {
    const int32_t splits = dz_splits(t.rows, t.cols);
    const dim3 grid((uint32_t)((t.cols + kDzCols - 1) / kDzCols), (uint32_t)splits);
    const dim3 block(kThreads);
    hipError_t e;
    switch (t.act) {
    case VPA_ACT_RELU:
        e = launch(dz_kernel<T, G, VPA_ACT_RELU>, grid, block, 0, stream, t, splits);
        break;
    case VPA_ACT_GELU:
        e = launch(dz_kernel<T, G, VPA_ACT_GELU>, grid, block, 0, stream, t, splits);
        break;
    case VPA_ACT_SILU:
        e = launch(dz_kernel<T, G, VPA_ACT_SILU>, grid, block, 0, stream, t, splits);
        break;
    default:
        e = launch(dz_kernel<T, G, VPA_ACT_NONE>, grid, block, 0, stream, t, splits);
    }
    if (e != hipSuccess || !t.bias)
        return e;
    return launch(bias_finish_kernel<T>, dim3((uint32_t)((t.cols + 63) / 64)),
                  dim3(kFinishWaves * 64), 0, stream, t, t.part ? splits : 0);
}

}  // namespace

namespace {

// The best tile and number of slices of k for one launch, and its modelled
// time in us: rounds of workgroups over the CUs times a stage's time, plus
// what slices cost to write and join.  The constants are measured (bf16: a
// 256-tile alone on a CU needs 1.5 to 1.6 us a stage, two 128-tiles on a CU 1.1 us;
// fp32's matrix instructions take 16 times as long for the same k).
double plan_tiles(int esize, int64_t m, int64_t n, int64_t k, GemmPlan& p) {
    const int64_t stages = stages_of(esize, k);
    double best = 0;
    for (int32_t tile = esize == 2 ? 256 : 128; tile >= 128; tile /= 2) {
        const double stage_us = esize == 4 ? 7.0 : tile == 256 ? 1.6 : 1.1;
        const int64_t at_once = tile == 256 ? 256 : 512;
        const int64_t tiles = ((m + tile - 1) / tile) * ((n + tile - 1) / tile);
        for (int32_t s = 1; s <= 16; s *= 2) {
            const int64_t per = (stages + s - 1) / s, blocks = tiles * s;
            if (s > 1 && per < 4)
                break;
            const double rounds = (double)((blocks + at_once - 1) / at_once);
            double us = rounds * ((double)per * stage_us + 2.0);
            if (s > 1)
                us += 4.0 + (double)s * (double)m * (double)n * 8.0 / 4.0e6;
            if (best == 0 || us < best) {
                best = us;
                p.tile = tile;
                p.slices = (int32_t)((stages + per - 1) / per);
                p.stages_per_slice = per;
            }
        }
    }
    return best;
}

size_t slices_bytes(const GemmPlan& p, int64_t m, int64_t n) {
    return p.slices > 1 ? (size_t)p.slices * (size_t)m * (size_t)n * 4 : 0;
}

}  // namespace

// The 256-tiles of a product seldom fill the last round: 272 of them take as
// long as 512.  Where the model says so, a first launch takes as many columns
// (or rows) of tiles as fill whole rounds, and a second one, of smaller tiles
// or slices of k, the rest: 4096 x 4352 x 4096 192 -> 135 us, 2048 x 50257 x
// 2048 434 -> 417, its gradient of the weight 653 -> 607.
GemmPlan plan_gemm(int esize, int64_t m, int64_t n, int64_t k, bool a_k1, bool b_k1) {
    GemmPlan p{};
    p.slices = 1;
    const int64_t stages = stages_of(esize, k);
    p.stages_per_slice = stages;
    if (a_k1 && b_k1 && m <= 64) {
        const int64_t tiles = (n + kFewRowsCols - 1) / kFewRowsCols;
        // Wavefronts alone while the ring's tiles do not give every CU one
        // (K = 4096, 8 rows: n = 8192 17 us against 20 for the ring, 16384 39
        // and 33, 32000 68 and 44).
        if (m <= kRowsKernelMost && tiles < 256) {
            p.rows_kernel = true;
            return p;
        }
        // Slices as long as all workgroups run at once, two a CU, and have at
        // least 8 stages (32 x 4096 x 32000 bf16, 500 tiles: 59 us in 2 slices,
        // 44 in one; 32 x 4096 x 25600 51 and 41; 32 x 4096 x 11008, 172 tiles:
        // 26.6 in 3, 26.1 in 2).
        p.tile = m <= 32 ? 32 : 64;
        int64_t s = 512 / tiles;
        s = s > stages / 8 ? stages / 8 : s;
        s = s < 1 ? 1 : s;
        p.stages_per_slice = (stages + s - 1) / s;
        p.slices = (int32_t)((stages + p.stages_per_slice - 1) / p.stages_per_slice);
        return p;
    }
    double best = plan_tiles(esize, m, n, k, p);
    if (esize != 2)
        return p;
    const int64_t tm = (m + 255) / 256, tn = (n + 255) / 256, whole = tm * tn / 256 * 256;
    for (int axis = 0; axis < 2; ++axis) {
        const int64_t first = (axis ? whole / tm : whole / tn) * 256;
        if (first == 0 || first >= (axis ? n : m))
            continue;
        GemmPlan f{}, r{};
        const double us = axis ? plan_tiles(esize, m, first, k, f) +
                                     plan_tiles(esize, m, n - first, k, r)
                               : plan_tiles(esize, first, n, k, f) +
                                     plan_tiles(esize, m - first, n, k, r);
        if (f.tile == 256 && us + 3.0 < best) {
            best = us + 3.0;
            p.first_m = axis ? m : first;
            p.first_n = axis ? first : n;
            p.tile = f.tile;
            p.slices = f.slices;
            p.stages_per_slice = f.stages_per_slice;
        }
    }
    return p;
}

namespace {

// The second launch of a plan that has one: m and n become its part's sizes.
GemmPlan plan_rest(int esize, const GemmPlan& first, int64_t& m, int64_t& n, int64_t k) {
    m -= first.first_m < m ? first.first_m : 0;
    n -= first.first_n < n ? first.first_n : 0;
    GemmPlan r{};
    plan_tiles(esize, m, n, k, r);
    return r;
}

// Most work-items of one of a plan's dispatches, the join among them.
int64_t planned_threads(const GemmPlan& p, int64_t m, int64_t n) {
    const auto blocks = [&](int64_t rows, int64_t cols) {
        return ((m + rows - 1) / rows) * ((n + cols - 1) / cols) * p.slices;
    };
    // rows that are not aligned take 128-tiles whatever the plan says
    int64_t most = blocks(128, 128) * 256;
    const int64_t own = p.tile <= 64    ? blocks(64, kFewRowsCols) * 256
                        : p.tile == 256 ? blocks(256, 256) * 512
                                        : most;
    most = own > most ? own : most;
    const int64_t join = p.slices > 1 ? (m * n + kThreads - 1) / kThreads * kThreads : 0;
    return join > most ? join : most;
}

}  // namespace

size_t gemm_workspace(int esize, int64_t m, int64_t n, int64_t k, bool a_k1, bool b_k1) {
    const GemmPlan p = plan_gemm(esize, m, n, k, a_k1, b_k1);
    if (!p.first_m)
        return slices_bytes(p, m, n);
    const GemmPlan q = plan_rest(esize, p, m, n, k);
    const size_t first = slices_bytes(p, p.first_m, p.first_n), rest = slices_bytes(q, m, n);
    return first > rest ? first : rest;
}

int64_t gemm_threads(int esize, int64_t m, int64_t n, int64_t k, bool a_k1, bool b_k1) {
    const GemmPlan p = plan_gemm(esize, m, n, k, a_k1, b_k1);
    if (p.rows_kernel)
        return linear_rows_threads(n);
    if (!p.first_m)
        return planned_threads(p, m, n);
    const GemmPlan q = plan_rest(esize, p, m, n, k);
    const int64_t first = planned_threads(p, p.first_m, p.first_n);
    const int64_t rest = planned_threads(q, m, n);
    return first > rest ? first : rest;
}

namespace {

hipError_t launch_planned(int esize, const GemmTask& t, const GemmPlan& p, hipStream_t stream) {
    hipError_t e = esize == 2 ? launch_gemm_tiles_bf16(t, p, stream)
                              : launch_gemm_tiles_f32(t, p, stream);
    if (e != hipSuccess || p.slices == 1)
        return e;
    const bool join4 = t.n % 4 == 0;
    const int64_t items = t.m * t.n / (join4 ? 4 : 1);
    const dim3 grid((uint32_t)((items + kThreads - 1) / kThreads)), block(kThreads);
    if (esize == 2)
        return join4 ? launch(gemm_join_kernel<uint16_t, true>, grid, block, 0, stream, t, p.slices)
                     : launch(gemm_join_kernel<uint16_t, false>, grid, block, 0, stream, t,
                              p.slices);
    return join4 ? launch(gemm_join_kernel<float, true>, grid, block, 0, stream, t, p.slices)
                 : launch(gemm_join_kernel<float, false>, grid, block, 0, stream, t, p.slices);
}

}  // namespace

hipError_t launch_gemm(int esize, const GemmTask& t, hipStream_t stream) {
    const bool ak = t.a_k1, bk = t.b_k1;
    GemmPlan p = plan_gemm(esize, t.m, t.n, t.k, ak, bk);
    if (p.rows_kernel)
        return launch_linear_rows(esize, t, stream);
    p.direct = direct_operand(esize, t.a, ak ? t.a_m : t.a_k, ak, t.m_readable) &&
               direct_operand(esize, t.b, bk ? t.b_n : t.b_k, bk, t.n_readable);
    if (!p.first_m)
        return launch_planned(esize, t, p, stream);
    GemmTask f = t, r = t;                          // the first part and the rest
    const int out = t.out_f32 ? 4 : esize;
    auto past = [](const void* q, int64_t bytes) { return q ? (char*)q + bytes : nullptr; };
    f.m = p.first_m;
    f.n = p.first_n;
    const int64_t dm = f.m < t.m ? f.m : 0, dn = f.n < t.n ? f.n : 0;
    r.m -= dm;
    r.m_readable -= dm;
    r.n -= dn;
    r.n_readable -= dn;
    r.a = past(t.a, dm * t.a_m * esize);
    r.b = past(t.b, dn * t.b_n * esize);
    r.bias = past(t.bias, dn * esize);
    r.residual = past(t.residual, (dm * t.ldr + dn) * esize);
    r.pre = past(t.pre, (dm * t.ldp + dn) * esize);
    r.y = past(t.y, (dm * t.ldy + dn) * out);
    int64_t m = t.m, n = t.n;
    GemmPlan q = plan_rest(esize, p, m, n, t.k);
    q.direct = p.direct;
    hipError_t e = launch_planned(esize, f, p, stream);
    return e != hipSuccess ? e : launch_planned(esize, r, q, stream);
}

// Slices of rows: enough workgroups for 8 a CU, at least 16 rows each.
int32_t dz_splits(int64_t rows, int64_t cols) {
    const int64_t tiles = (cols + kDzCols - 1) / kDzCols;
    int64_t s = (2048 + tiles - 1) / tiles;
    s = s > (rows + 15) / 16 ? (rows + 15) / 16 : s;
    return (int32_t)(s < 1 ? 1 : s > 256 ? 256 : s);
}

int64_t dz_threads(int64_t rows, int64_t cols, bool bias) {
    const int64_t finish = bias ? (cols + 63) / 64 * 64 * kFinishWaves : 0;
    const int64_t dz = (cols + kDzCols - 1) / kDzCols * kThreads * dz_splits(rows, cols);
    return dz > finish ? dz : finish;
}

hipError_t launch_dz(int esize, const DzTask& t, hipStream_t stream) {
    if (esize == 4)
        return launch_dz_typed<float, float>(t, stream);
    return t.grad_f32 ? launch_dz_typed<uint16_t, float>(t, stream)
                      : launch_dz_typed<uint16_t, uint16_t>(t, stream);
}

}  // namespace vpa
