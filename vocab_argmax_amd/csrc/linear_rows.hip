// linear_rows.hip -- y = residual + act(x W^T + bias) for at most 64 rows of x:
// a decode batch, down to a single token.
//
// Every element of W is used a few times at most, so the kernel is bound by
// reading W once from memory.  A wavefront takes 16 * NW rows of W and a
// share of k; W goes straight from memory into the matrix instruction's
// operand registers, and x, which all wavefronts share, comes from the
// caches.  Where W has too few rows to fill the chip with wavefronts, KS of
// a workgroup's 8 wavefronts split the k of one block of rows and join their
// sums in LDS, in order: one launch, no workspace.
#include "gemm_tile.h"
#include "linear_common.h"

namespace vpa {
namespace {

constexpr int kWaves = 8;

// 16 bytes of row `p` at element e, 0 past n.
template <int ESIZE>
__device__ __forceinline__ u32x4_t load16(const char* p, int64_t e, int64_t n) {
    using T = typename elem<ESIZE>::type;
    constexpr int VEC = 16 / ESIZE;
    if (e + VEC <= n)
        return ((const Loose16*)(p + e * ESIZE))->v;
    union {
        T x[VEC];
        u32x4_t v;
    } u;
    u.v = u32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < VEC; ++i)
        if (e + i < n)
            u.x[i] = ((const T*)p)[e + i];
    return u.v;
}

template <int ESIZE, int MT, int NW>
__global__ __launch_bounds__(kWaves * 64) void linear_rows_kernel(GemmTask t, int32_t ks) {
    using T = typename elem<ESIZE>::type;
    constexpr int KB = 128 / ESIZE;                 // k of a step: 128 bytes of a row
    constexpr int VEC = 16 / ESIZE;
    constexpr int M = MT * 16, N = NW * 16;
    constexpr int D = MT == 4 ? 1 : 2;
    __shared__ f32x4 sums[kWaves][NW * MT][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t block = (int64_t)blockIdx.x * (kWaves / ks) + wave / ks;
    const int share = wave % ks;
    const int64_t n0 = block * N;
    const int r = lane & 15, q = lane >> 4;
    const char* w[NW];
    const char* x[MT];
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        // rows past the end repeat the last one: their sums are not stored
        const int64_t n = n0 + i * 16 + r < t.n ? n0 + i * 16 + r : t.n - 1;
        w[i] = (const char*)t.b + n * t.b_n * ESIZE;
    }
#pragma unroll
    for (int j = 0; j < MT; ++j) {
        const int64_t m = j * 16 + r < t.m ? j * 16 + r : t.m - 1;
        x[j] = (const char*)t.a + m * t.a_m * ESIZE;
    }
    f32x4 acc[NW][MT] = {};
    const int64_t whole = t.k / KB, steps = (t.k + KB - 1) / KB;
    auto multiply = [&](const u32x4_t (&wv)[NW][2], const u32x4_t (&xv)[MT][2]) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < NW; ++i)
#pragma unroll
                for (int j = 0; j < MT; ++j)
                    acc[i][j] = mma<ESIZE>(wv[i][h], xv[j][h], acc[i][j]);
    };
    if (n0 < t.n) {
        // D steps at a time, the next D on their way
        u32x4_t wn[D][NW][2], xn[D][MT][2];
        auto fetch = [&](int64_t s) {
#pragma unroll
            for (int d = 0; d < D; ++d)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int64_t o = (s + d * ks) * 128 + h * 64 + q * 16;
#pragma unroll
                    for (int i = 0; i < NW; ++i)
                        wn[d][i][h] = ((const Loose16*)(w[i] + o))->v;
#pragma unroll
                    for (int j = 0; j < MT; ++j)
                        xn[d][j][h] = ((const Loose16*)(x[j] + o))->v;
                }
        };
        int64_t s = share;
        const int64_t last = whole - (int64_t)(D - 1) * ks;     // the last start of D steps, + 1
        if (s < last)
            fetch(s);
        for (; s < last; s += (int64_t)D * ks) {
            u32x4_t wv[D][NW][2], xv[D][MT][2];
#pragma unroll
            for (int d = 0; d < D; ++d)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int i = 0; i < NW; ++i)
                        wv[d][i][h] = wn[d][i][h];
#pragma unroll
                    for (int j = 0; j < MT; ++j)
                        xv[d][j][h] = xn[d][j][h];
                }
            if (s + (int64_t)D * ks < last)
                fetch(s + (int64_t)D * ks);
#pragma unroll
            for (int d = 0; d < D; ++d)
                multiply(wv[d], xv[d]);
        }
        for (; s < whole; s += ks) {
            u32x4_t wv[NW][2], xv[MT][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t o = s * 128 + h * 64 + q * 16;
#pragma unroll
                for (int i = 0; i < NW; ++i)
                    wv[i][h] = ((const Loose16*)(w[i] + o))->v;
#pragma unroll
                for (int j = 0; j < MT; ++j)
                    xv[j][h] = ((const Loose16*)(x[j] + o))->v;
            }
            multiply(wv, xv);
        }
        if (whole < steps && share == whole % ks) {
            u32x4_t wv[NW][2], xv[MT][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t e = whole * KB + (h * 4 + q) * VEC;
#pragma unroll
                for (int i = 0; i < NW; ++i)
                    wv[i][h] = load16<ESIZE>(w[i], e, t.k);
#pragma unroll
                for (int j = 0; j < MT; ++j)
                    xv[j][h] = load16<ESIZE>(x[j], e, t.k);
            }
            multiply(wv, xv);
        }
    }
#pragma unroll
    for (int i = 0; i < NW; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j)
            sums[wave][i * MT + j][lane] = acc[i][j];
    __syncthreads();
    // results of the workgroup's blocks, n fastest; in a 16 x 16 piece n is
    // (lane / 16) * 4 + e and m is lane % 16
    const int blocks = kWaves / ks;
    for (int id = threadIdx.x; id < blocks * M * N; id += kWaves * 64) {
        const int b = id / (M * N), rest = id % (M * N);
        const int m = rest / N, n = rest % N;
        const int64_t col = ((int64_t)blockIdx.x * blocks + b) * N + n;
        if (m >= t.m || col >= t.n)
            continue;
        const int piece = (n >> 4) * MT + (m >> 4), at = (m & 15) + ((n & 15) >> 2) * 16;
        float v = sums[b * ks][piece][at][n & 3];
        for (int s = 1; s < ks; ++s)
            v += sums[b * ks + s][piece][at][n & 3];
        store_result<T>(t, m, col, v);
    }
}

// Rows of W per wavefront and wavefronts that share a block's k: 32 rows
// where that still leaves 8 wavefronts a CU, else 16, and k is split until
// there are as many.
struct RowsPlan {
    int32_t nw, ks;
    int64_t groups;
};
RowsPlan plan_rows(int64_t n) {
    RowsPlan p;
    p.nw = n >= 32 * 2048 ? 2 : 1;
    const int64_t blocks = (n + 16 * p.nw - 1) / (16 * p.nw);
    p.ks = 1;
    while (p.ks < kWaves && blocks * p.ks < 2048)
        p.ks *= 2;
    const int64_t per = kWaves / p.ks;
    p.groups = (blocks + per - 1) / per;
    return p;
}

template <int ESIZE, int MT>
hipError_t launch_rows(const GemmTask& t, hipStream_t stream) {
    const RowsPlan p = plan_rows(t.n);
    const dim3 grid((uint32_t)p.groups), block(kWaves * 64);
    return p.nw == 2 ? launch(linear_rows_kernel<ESIZE, MT, 2>, grid, block, 0, stream, t, p.ks)
                     : launch(linear_rows_kernel<ESIZE, MT, 1>, grid, block, 0, stream, t, p.ks);
}

template <int ESIZE>
hipError_t launch_rows_any(const GemmTask& t, hipStream_t stream) {
    if (t.m <= 16)
        return launch_rows<ESIZE, 1>(t, stream);
    return t.m <= 32 ? launch_rows<ESIZE, 2>(t, stream) : launch_rows<ESIZE, 4>(t, stream);
}

}  // namespace

int64_t linear_rows_threads(int64_t, int64_t n) {
    return plan_rows(n).groups * kWaves * 64;
}

hipError_t launch_linear_rows(int esize, const GemmTask& t, hipStream_t stream) {
    return esize == 2 ? launch_rows_any<2>(t, stream) : launch_rows_any<4>(t, stream);
}

}  // namespace vpa
