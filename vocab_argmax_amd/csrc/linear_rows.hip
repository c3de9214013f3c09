// linear_rows.hip -- y = residual + act(x W^T + bias) for at most 16 rows of
// x: a small decode batch, down to a single token.
//
// Every element of W is used a few times at most, so the kernel is bound by
// reading W once from memory.  A wavefront takes 16 rows of W and a
// share of k; W goes straight from memory into the matrix instruction's
// operand registers, D steps of 128 bytes a row at a time, and x, which all
// wavefronts share, comes from the caches.  The WAVES wavefronts of a
// workgroup split the k of one block of rows and join their sums in LDS, in
// order: one launch, no workspace.  1 x 4096 x 4096 bf16 8.2 us, 4.1 TB/s (a launch of this size
// alone takes about 3); with rows at 16 bytes past a line 14, at 2 bytes 16.
#include <type_traits>

#include "gemm_tile.h"
#include "linear_common.h"

namespace vpa {
namespace {

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

template <int ESIZE, int D, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void linear_rows_kernel(GemmTask t) {
    using T = typename elem<ESIZE>::type;
    constexpr int KB = 128 / ESIZE;                 // k of a step: 128 bytes of a row
    constexpr int VEC = 16 / ESIZE;
    __shared__ f32x4 sums[WAVES][64];
    // The wavefront's number as a scalar: what depends on it has to be branched
    // over, not masked, since a matrix instruction ignores the mask.
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int r = lane & 15, q = lane >> 4;
    // rows past the end repeat the last one: their sums are not stored
    const char* w = (const char*)t.b + (n0 + r < t.n ? n0 + r : t.n - 1) * t.b_n * ESIZE;
    const char* x = (const char*)t.a + (r < t.m ? r : t.m - 1) * t.a_m * ESIZE;
    f32x4 acc = {};
    const int64_t whole = t.k / KB, steps = (t.k + KB - 1) / KB;
    // COUNT whole steps from s
    auto run = [&](int64_t s, auto count) {
        constexpr int COUNT = count();
        u32x4_t wv[COUNT][2], xv[COUNT][2];
#pragma unroll
        for (int d = 0; d < COUNT; ++d)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t o = (s + d) * 128 + h * 64 + q * 16;
                wv[d][h] = __builtin_nontemporal_load(&((const Loose16*)(w + o))->v);
                xv[d][h] = ((const Loose16*)(x + o))->v;
            }
        __builtin_amdgcn_sched_barrier(0);          // all loads before the first wait
#pragma unroll
        for (int d = 0; d < COUNT; ++d)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                acc = mma<ESIZE>(wv[d][h], xv[d][h], acc);
    };
    const int64_t batches = whole / D;
    for (int64_t b = wave; b < batches; b += WAVES)
        run(b * D, std::integral_constant<int, D>{});
    for (int64_t s = batches * D + wave; s < whole; s += WAVES)
        run(s, std::integral_constant<int, 1>{});
    if (whole < steps && wave == WAVES - 1) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t e = whole * KB + (h * 4 + q) * VEC;
            acc = mma<ESIZE>(load16<ESIZE>(w, e, t.k), load16<ESIZE>(x, e, t.k), acc);
        }
    }
    sums[wave][lane] = acc;
    __syncthreads();
    // n fastest; in a block n is (lane / 16) * 4 + e and m is lane % 16
    const int m = threadIdx.x / 16, n = threadIdx.x % 16;
    if (m >= t.m || n0 + n >= t.n)
        return;
    const int at = m + (n >> 2) * 16;
    float v = sums[0][at][n & 3];
#pragma unroll
    for (int s = 1; s < WAVES; ++s)
        v += sums[s][at][n & 3];
    store_result<T>(t, m, n0 + n, v);
}

// 8 wavefronts a workgroup while each has a CU to itself, which its registers
// allow, else 4 (K = 4096, one row: n = 4800 14.6 us with 8, 14.4 with 4; 4112
// of K = 1600 8.9 and 7.6; 4096 of K = 4096 9.3 with 8).
int rows_waves(int64_t n) {
    return n <= 16 * 256 ? 8 : 4;
}

template <int ESIZE>
hipError_t launch_rows(const GemmTask& t, hipStream_t stream) {
    constexpr int D = 8;
    const int waves = rows_waves(t.n);
    const dim3 grid((uint32_t)((t.n + 15) / 16)), block((uint32_t)waves * 64);
    return waves == 8 ? launch(linear_rows_kernel<ESIZE, D, 8>, grid, block, 0, stream, t)
                      : launch(linear_rows_kernel<ESIZE, D, 4>, grid, block, 0, stream, t);
}

}  // namespace

int64_t linear_rows_threads(int64_t n) {
    return (n + 15) / 16 * rows_waves(n) * 64;
}

hipError_t launch_linear_rows(int esize, const GemmTask& t, hipStream_t stream) {
    return esize == 2 ? launch_rows<2>(t, stream) : launch_rows<4>(t, stream);
}

}  // namespace vpa
