// linear_fp8.hip -- y = residual + act(x W^T + bias) of 8-bit operands with a
// scale for each block of 128 columns (of W: and 128 rows).
//
// A block of k is summed from 0 in fp32, and the result is scaled and added to
// the accumulators with one multiply-add: W's fragment is given to the matrix
// instruction first, so a lane's four results have consecutive n and one m, and
// one factor.  A lane's operand registers hold 32 bytes of a row, 16 of each
// half of the block; which k a byte has does not matter as long as both
// operands agree.
//
// The matrix cores' 8-bit instruction cuts, in every group of 8 products, what
// lies below 2^-13 of the largest (measured; random normal operands end 1.4e-5
// off in the 2-norm).  Widened to bf16, which holds every e4m3 value, products
// are summed in full fp32 at half the rate.
#include "gemm_tile.h"
#include "linear_common.h"
#include "vpa_draft_internal.h"

namespace vpa {
namespace {

// 8 bytes as bf16.
__device__ __forceinline__ bf16x8 widen(uint32_t lo, uint32_t hi) {
    union {
        bf16x2 h[4];
        bf16x8 v;
    } u;
    u.h[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    u.h[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    u.h[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    u.h[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    return u.v;
}

// P Q^T for 16 rows of P and of Q over 128 k: bytes q*16.. of both halves.
__device__ __forceinline__ f32x4 mma_exact(const u32x4_t (&p)[2], const u32x4_t (&q)[2]) {
    f32x4 d = {0, 0, 0, 0};
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; e += 2)
            d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen(p[h][e], p[h][e + 1]),
                                                        widen(q[h][e], q[h][e + 1]), d, 0, 0, 0);
    return d;
}

// 16 bytes at column k of a row of n, 0 past its end.
__device__ __forceinline__ u32x4_t load16(const uint8_t* row, int64_t k, int64_t n) {
    if (k + 16 <= n)
        return *(const u32x4_t*)(row + k);
    union {
        uint8_t e[16];
        u32x4_t v;
    } u;
    u.v = u32x4_t{0, 0, 0, 0};
    for (int i = 0; i < 16; ++i)
        if (k + i < n)
            u.e[i] = row[k + i];
    return u.v;
}

// A wavefront a 16 x 16 tile.
__global__ __launch_bounds__(64) void fp8_simple_kernel(Fp8Task f, uint32_t tiles_m) {
    const GemmTask& t = f.g;
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int64_t m0 = (int64_t)(blockIdx.x % tiles_m) * 16, n0 = (int64_t)(blockIdx.x / tiles_m) * 16;
    const int64_t m = m0 + r < t.m ? m0 + r : t.m - 1, n = n0 + r < t.n ? n0 + r : t.n - 1;
    const uint8_t* x = (const uint8_t*)t.a + m * t.a_m;
    const uint8_t* w = (const uint8_t*)t.b + n * t.b_n;
    const float* xs = f.a_scale + m * f.lda_scale;
    const float* ws = f.b_scale + n0 / kScaleBlock * f.ldb_scale;
    f32x4 acc = {};
    for (int64_t b = 0; b * kScaleBlock < t.k; ++b) {
        const int64_t k = b * kScaleBlock + q * 16;
        const u32x4_t p[2] = {load16(w, k, t.k), load16(w, k + 64, t.k)};
        const u32x4_t v[2] = {load16(x, k, t.k), load16(x, k + 64, t.k)};
        acc += mma_exact(p, v) * (xs[b] * ws[b]);
    }
    if (m0 + r >= t.m)
        return;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (n0 + q * 4 + e < t.n)
            store_result<uint16_t>(t, m0 + r, n0 + q * 4 + e, acc[e]);
}

}  // namespace

size_t fp8_workspace(int64_t, int64_t, int64_t) {
    return 0;
}

int64_t fp8_threads(int64_t m, int64_t n, int64_t) {
    return (m + 15) / 16 * ((n + 15) / 16) * 64;
}

hipError_t launch_fp8(const Fp8Task& t, hipStream_t stream) {
    const int64_t tm = (t.g.m + 15) / 16, tn = (t.g.n + 15) / 16;
    return launch(fp8_simple_kernel, dim3((uint32_t)(tm * tn)), dim3(64), 0, stream, t,
                  (uint32_t)tm);
}

}  // namespace vpa
