// linear.hip -- the head's products: y = residual + act(x W^T + bias) and the
// products of its backward pass, on the matrix cores with fp32 accumulation.
#include "gemm_tile.h"
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

// Four results of consecutive n: 16- or 8-byte accesses (every row of the
// outputs and the residual is aligned for them).
template <typename T, int ACT>
__device__ __forceinline__ void store_results(const GemmTask& t, int64_t m, int64_t n, f32x4 acc) {
    using V = T __attribute__((ext_vector_type(4)));
    if (t.bias)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            acc[i] += to_f32(((const T*)t.bias)[n + i]);
    auto put = [](T* p, f32x4 v) {
        if constexpr (sizeof(T) == 2)
            *(uint2*)p = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
        else
            *(f32x4*)p = v;
    };
    if (t.pre)
        put((T*)t.pre + m * t.ldp + n, acc);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        acc[i] = act<ACT>(acc[i]);
    if (t.residual) {
        const V r = *(const V*)((const T*)t.residual + m * t.ldr + n);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            acc[i] += to_f32((T)r[i]);
    }
    if (t.out_f32)
        *(f32x4*)((float*)t.y + m * t.ldy + n) = acc;
    else
        put((T*)t.y + m * t.ldy + n, acc);
}

// A wavefront's 64 x 64 results from accumulators to memory, through its own
// 16 KiB of LDS so that a store instruction covers whole rows: 4 rows of 64
// where `vec` says that rows are aligned for 4 elements, else one row, an
// element a lane.  Rows of LDS have 16 chunks of 16 bytes, chunk c of row r
// at c ^ (r & 15).
template <typename T, int ACT>
__device__ __forceinline__ void store_block(const GemmTask& t, bool vec, float* part, char* lds,
                                            int64_t m0, int64_t n0, const f32x4 (&acc)[4][4]) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = i * 16 + (lane & 15), c = j * 4 + (lane >> 4);
            *(f32x4*)(lds + r * 256 + ((c ^ (r & 15)) << 4)) = acc[i][j];
        }
    // this LDS is the wavefront's alone and its accesses execute in order; the
    // fences keep the compiler to it
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (vec && n0 + 64 <= t.n) {
#pragma unroll 1
        for (int r0 = 0; r0 < 64; r0 += 16) {
            f32x4 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = r0 + k * 4 + (lane >> 4), c = lane & 15;
                v[k] = *(const f32x4*)(lds + r * 256 + ((c ^ (r & 15)) << 4));
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t m = m0 + r0 + k * 4 + (lane >> 4), n = n0 + (lane & 15) * 4;
                if (m >= t.m)
                    continue;
                if (part)
                    *(f32x4*)(part + m * t.n + n) = v[k];
                else
                    store_results<T, ACT>(t, m, n, v[k]);
            }
        }
        return;
    }
    const int64_t n = n0 + lane;
#pragma unroll 4
    for (int r = 0; r < 64; ++r) {
        const float v = *(const float*)(lds + r * 256 + (((lane >> 2) ^ (r & 15)) << 4) +
                                        (lane & 3) * 4);
        const int64_t m = m0 + r;
        if (m >= t.m || n >= t.n)
            continue;
        if (part)
            part[m * t.n + n] = v;
        else
            store_result<T, ACT>(t, m, n, v);
    }
}

// The tiled product (gemm_tile.h): WM x WN wavefronts, each with BM/WM x
// BN/WN of the tile in its accumulators.  With part set, blockIdx.y is a
// slice of k and the raw sums go to part[slice][m][n].
template <int ESIZE, bool AK, bool BK, int BM, int BN, int WM, int WN, int ACT>
__global__ __launch_bounds__(WM* WN * 64) void gemm_tile_kernel(GemmTask t, uint32_t tiles_m,
                                                                uint32_t tiles_n,
                                                                int64_t stages_per_slice,
                                                                bool vec, float* part) {
    using T = typename elem<ESIZE>::type;
    constexpr int NT = WM * WN * 64;
    constexpr int IM = BM / WM / 16, JN = BN / WN / 16;
    static_assert(IM % 4 == 0 && JN == 4, "the epilogue stores blocks of 64 x 64");
    using LA = TileLoader<ESIZE, AK, BM, NT>;
    using LB = TileLoader<ESIZE, BK, BN, NT>;
    __shared__ __align__(1024) char lds0[LA::BYTES + LB::BYTES];
    __shared__ __align__(1024) char lds1[LA::BYTES + LB::BYTES];
    uint32_t tm, tn;
    tile_of_block(blockIdx.x, tiles_m, tiles_n, tm, tn);
    const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = wave / WN * (BM / WM), wn = wave % WN * (BN / WN);
    LA la;
    LB lb;
    la.init(t.a, AK ? t.a_m : t.a_k, m0, t.m);
    lb.init(t.b, BK ? t.b_n : t.b_k, n0, t.n);
    const int64_t whole = t.k / LA::KB, all = (t.k + LA::KB - 1) / LA::KB;
    const int64_t s0 = blockIdx.y * stages_per_slice;
    const int64_t end = s0 + stages_per_slice < all ? s0 + stages_per_slice : all;
    f32x4 acc[IM][JN] = {};
    auto stage = [&](int64_t s, char* lds) {
        la.load(s, lds);
        lb.load(s, lds + LA::BYTES);
    };
    auto multiply = [&](const char* lds) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            u32x4_t av[IM], bv[JN];
#pragma unroll
            for (int j = 0; j < JN; ++j)
                bv[j] = LB::fragment(lds + LA::BYTES, wn + j * 16, s);
#pragma unroll
            for (int i = 0; i < IM; ++i)
                av[i] = LA::fragment(lds, wm + i * 16, s);
#pragma unroll
            for (int i = 0; i < IM; ++i)
#pragma unroll
                for (int j = 0; j < JN; ++j)
                    acc[i][j] = mma<ESIZE>(bv[j], av[i], acc[i][j]);
            __builtin_amdgcn_sched_barrier(0);      // one step's fragments at a time
        }
    };
    // a stage that k ends in comes first, so that the loop has whole ones only
    const int64_t s1 = end < whole ? end : whole;
    if (end > whole) {
        la.load_tail(whole, t.k, lds1);
        lb.load_tail(whole, t.k, lds1 + LA::BYTES);
    }
    if (s0 < s1)
        stage(s0, lds0);
    if (end > whole) {
        __syncthreads();
        multiply(lds1);
    }
    for (int64_t s = s0; s < s1; s += 2) {
        __syncthreads();
        if (s + 1 < s1)
            stage(s + 1, lds1);
        multiply(lds0);
        if (s + 1 >= s1)
            break;
        __syncthreads();
        if (s + 2 < s1)
            stage(s + 2, lds0);
        multiply(lds1);
    }
    __syncthreads();
    if (part)
        part += (int64_t)blockIdx.y * t.m * t.n;
    char* mine = wave * 16384 < LA::BYTES + LB::BYTES
                     ? lds0 + wave * 16384 : lds1 + (wave * 16384 - LA::BYTES - LB::BYTES);
#pragma unroll
    for (int h = 0; h < IM / 4; ++h) {
        f32x4 block[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                block[i][j] = acc[h * 4 + i][j];
        store_block<T, ACT>(t, vec, part, mine, m0 + wm + h * 64, n0 + wn, block);
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
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

// The tiled kernel moves 16 bytes at a time: an operand with contiguous k
// needs rows of 16-byte aligned address, one with contiguous rows a multiple
// of 16 bytes of them too.  Offsets within a tile are 32 bits.
bool tile_operand(int esize, const void* p, int64_t ld, bool k1, int64_t rows) {
    const int64_t vec = 16 / esize;
    return (uintptr_t)p % 16 == 0 && ld % vec == 0 && ld <= ((int64_t)1 << 21) &&
           (k1 || rows % vec == 0);
}

bool vec4(const void* p, int64_t ld, int esize) {
    return !p || ((uintptr_t)p % (4 * esize) == 0 && ld % 4 == 0);
}

template <int ESIZE, bool AK, bool BK, int ACT>
hipError_t launch_tile(const GemmTask& t, hipStream_t stream) {
    // fp32's instructions take 8 times as long for the same bytes, so half the
    // tile feeds them, and its fragments leave registers free
    constexpr int BM = ESIZE == 2 ? 256 : 128, BN = BM, WM = 2, WN = BN / 64;
    const uint32_t tm = (uint32_t)((t.m + BM - 1) / BM), tn = (uint32_t)((t.n + BN - 1) / BN);
    const int64_t stages = (t.k * ESIZE + 127) / 128;
    const bool vec = vec4(t.y, t.ldy, t.out_f32 ? 4 : ESIZE) && vec4(t.pre, t.ldp, ESIZE) &&
                     vec4(t.residual, t.ldr, ESIZE);
    return launch(gemm_tile_kernel<ESIZE, AK, BK, BM, BN, WM, WN, ACT>, dim3(tm * tn),
                  dim3(WM * WN * 64), 0, stream, t, tm, tn, stages, vec, nullptr);
}

template <int ESIZE>
hipError_t launch_tile_any(const GemmTask& t, hipStream_t stream) {
    const bool ak = t.a_k == 1, bk = t.b_k == 1;
    if (!ak)
        return launch_tile<ESIZE, false, false, VPA_ACT_NONE>(t, stream);
    if (!bk)
        return launch_tile<ESIZE, true, false, VPA_ACT_NONE>(t, stream);
    switch (t.act) {
    case VPA_ACT_RELU:
        return launch_tile<ESIZE, true, true, VPA_ACT_RELU>(t, stream);
    case VPA_ACT_GELU:
        return launch_tile<ESIZE, true, true, VPA_ACT_GELU>(t, stream);
    case VPA_ACT_SILU:
        return launch_tile<ESIZE, true, true, VPA_ACT_SILU>(t, stream);
    default:
        return launch_tile<ESIZE, true, true, VPA_ACT_NONE>(t, stream);
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
    const bool ak = t.a_k == 1, bk = t.b_k == 1;
    if (t.m >= 128 && t.n >= 128 && t.k >= 64 &&
        tile_operand(esize, t.a, ak ? t.a_m : t.a_k, ak, t.m) &&
        tile_operand(esize, t.b, bk ? t.b_n : t.b_k, bk, t.n))
        return esize == 2 ? launch_tile_any<2>(t, stream) : launch_tile_any<4>(t, stream);
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
