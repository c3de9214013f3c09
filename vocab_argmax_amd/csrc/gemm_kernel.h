// gemm_kernel.h -- the tiled product's kernel (see gemm_tile.h) and its
// launch, instantiated for one element size by gemm_bf16.hip and gemm_f32.hip.
#pragma once

#include <type_traits>

#include "gemm_tile.h"
#include "linear_common.h"

namespace vpa {
namespace {

// WM x WN wavefronts, each with BM/WM x BN/WN of the tile in its
// accumulators.  With part set, the raw sums of a slice of k go to
// part[slice][m][n].
//
// Bound by the matrix cores and the card's power: they are busy for 74 % of the
// clocks of 8192^3 bf16 (747 us, 1472 TFLOP/s, at the 1.9 GHz that the card
// then holds; at 66 % it held 2.0; 672 us by the library in turn with it);
// 4096^3 104 us, with bias, silu and a residual 123.
// A 256-tile needs 32 KiB of each operand a stage, so that two stages fill
// 128 of 160 KiB of LDS, and reads 24 KiB of LDS a wavefront and stage; a
// 256-tile of 4 wavefronts spills (729 TFLOP/s); 128-tiles need 2.2 us for the
// area and k that a 256-tile takes 1.5 for, but fill the chip with small
// products.  fp32: 4096^3 957 us, 144 TFLOP/s, 96 % of the library's, at the
// rate of fp32's matrix instruction.
template <int ESIZE, bool AK, bool BK, bool DIRECT, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM* WN * 64) void gemm_tile_kernel(GemmTask t, uint32_t tiles_m,
                                                                uint32_t tiles_n,
                                                                int64_t stages_per_slice,
                                                                float* part) {
    using T = typename elem<ESIZE>::type;
    constexpr int NT = WM * WN * 64;
    constexpr int IM = BM / WM / 16, JN = BN / WN / 16;
    static_assert(IM % 4 == 0 && JN % 4 == 0 && JN <= IM, "the epilogue stores blocks of 64 x 64");
    using LA = TileLoader<ESIZE, AK, DIRECT, BM, NT>;
    using LB = TileLoader<ESIZE, BK, DIRECT, BN, NT>;
    __shared__ __align__(1024) char lds0[LA::BYTES + LB::BYTES];
    __shared__ __align__(1024) char lds1[LA::BYTES + LB::BYTES];
    uint32_t slice, tm, tn;
    tile_of_block(blockIdx.x, gridDim.x, tiles_m, tiles_n, slice, tm, tn);
    const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = wave / WN * (BM / WM), wn = wave % WN * (BN / WN);
    LA la;
    LB lb;
    la.init(t.a, AK ? t.a_m : t.a_k, m0, t.m_readable);
    lb.init(t.b, BK ? t.b_n : t.b_k, n0, t.n_readable);
    const int64_t whole = t.k / LA::KB, all = (t.k + LA::KB - 1) / LA::KB;
    const int64_t s0 = slice * stages_per_slice;
    const int64_t end = s0 + stages_per_slice < all ? s0 + stages_per_slice : all;
    const typename LA::Place pa = LA::place(wm);
    const typename LB::Place pb = LB::place(wn);
    f32x4 acc[IM][JN] = {};
    auto multiply = [&](const char* lds) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            u32x4_t av[IM], bv[JN];
#pragma unroll
            for (int j = 0; j < JN; ++j)
                bv[j] = LB::fragment(lds + LA::BYTES, pb, j, s);
#pragma unroll
            for (int i = 0; i < IM; ++i)
                av[i] = LA::fragment(lds, pa, i, s);
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
    if constexpr (DIRECT) {
        // While a step's products run, from fragments in registers, the next
        // step's fragments are read into the registers that they free.  One
        // barrier a stage says both that the next stage has landed and that
        // every wavefront has read this one, whose buffer the stage after
        // next then fills.  It stands after the first products of a step, so
        // that nothing waits for the reads issued just before it; half of the
        // wavefronts, one of the two on a SIMD, issue their loads there and
        // half a stage later the others, since a wavefront that issues them is
        // held up by the 64 bytes a clock that the loads can be taken in
        // (8192^3 800 us with all loads and the barrier before a step, 790
        // with halves, 775 so; 679 by the library on the same card).  A
        // wavefront that issues loads gives way to the other one on its SIMD
        // until it has done its first products after the next barrier (757 ->
        // 747 us on a card where the library needs 672).
        const typename LA::Direct da = la.direct();
        const typename LB::Direct db = lb.direct();
        auto stage = [&](int64_t s, char* lds) {
            __builtin_amdgcn_s_setprio(0);
            la.load(da, s, lds);
            lb.load(db, s, lds + LA::BYTES);
        };
        u32x4_t av[IM], bv0[JN], bv1[JN];
        // multiplies av and bv and reads the next fragments into av and bn,
        // from iteration FIRST on, which between() precedes
        auto step = [&](const u32x4_t (&bv)[JN], u32x4_t (&bn)[JN], const char* next,
                        int next_step, auto first, auto between) {
            const typename LA::Place a = pa.again();
            const typename LB::Place b = pb.again();
            constexpr int FIRST = first();
#pragma unroll
            for (int i = 0; i < IM; ++i) {
                if (i == FIRST)
                    between();
#pragma unroll
                for (int j = 0; j < JN; ++j)
                    acc[i][j] = mma<ESIZE>(bv[j], av[i], acc[i][j]);
                if (i == FIRST)
                    __builtin_amdgcn_s_setprio(1);
#pragma unroll
                for (int r = i == FIRST ? 0 : i; r <= i && i >= FIRST; ++r)
                    av[r] = LA::fragment(next, a, r, next_step);
                if (i == IM - 1)
#pragma unroll
                    for (int j = 0; j < JN; ++j)
                        bn[j] = LB::fragment(next + LA::BYTES, b, j, next_step);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        const std::integral_constant<int, 0> at_once{};
        const std::integral_constant<int, 1> after_one{};
        const bool early =
            (int)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6) < WM * WN / 2;
        if (end > whole) {
            stage_barrier();
            multiply(lds1);
            stage_barrier();
        }
        if (s0 < s1) {
            stage(s0, lds0);
            if (s0 + 1 < s1)
                stage(s0 + 1, lds1);
            stage_barrier();
#pragma unroll
            for (int j = 0; j < JN; ++j)
                bv0[j] = LB::fragment(lds0 + LA::BYTES, pb, j, 0);
#pragma unroll
            for (int i = 0; i < IM; ++i)
                av[i] = LA::fragment(lds0, pa, i, 0);
            step(bv0, bv1, lds0, 1, at_once, [] {});
        }
        // stage s's second step and stage s + 1's first
        for (int64_t s = s0; s + 1 < s1; ++s) {
            char* now = (s - s0) & 1 ? lds1 : lds0;
            char* next = (s - s0) & 1 ? lds0 : lds1;
            step(bv1, bv0, next, 0, after_one, [&] {
                stage_barrier();
                if (early && s + 2 < s1)
                    stage(s + 2, now);
            });
            if (!early && s + 2 < s1)
                stage(s + 2, now);
            step(bv0, bv1, next, 1, at_once, [] {});
        }
        if (s0 < s1) {
#pragma unroll
            for (int i = 0; i < IM; ++i)
#pragma unroll
                for (int j = 0; j < JN; ++j)
                    acc[i][j] = mma<ESIZE>(bv1[j], av[i], acc[i][j]);
        }
    } else {
        u32x4_t va[LA::LOADS], vb[LB::LOADS];
        auto fetch = [&](int64_t s) {
            la.fetch(s, va);
            lb.fetch(s, vb);
        };
        auto put = [&](char* lds) {
            LA::put(va, lds);
            LB::put(vb, lds + LA::BYTES);
        };
        if (end > whole) {
            stage_barrier();
            multiply(lds1);
        }
        if (s0 < s1) {
            fetch(s0);
            put(lds0);
        }
        for (int64_t s = s0; s < s1; s += 2) {
            stage_barrier();
            if (s + 1 < s1)
                fetch(s + 1);
            multiply(lds0);
            if (s + 1 >= s1)
                break;
            put(lds1);
            stage_barrier();
            if (s + 2 < s1)
                fetch(s + 2);
            multiply(lds1);
            if (s + 2 < s1)
                put(lds0);
        }
    }
    stage_barrier();
    if (part)
        part += slice * t.m * t.n;
    char* mine = wave * 16384 < LA::BYTES + LB::BYTES
                     ? lds0 + wave * 16384 : lds1 + (wave * 16384 - LA::BYTES - LB::BYTES);
#pragma unroll
    for (int h = 0; h < IM / 4; ++h)
#pragma unroll
        for (int g = 0; g < JN / 4; ++g) {
            f32x4 block[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    block[i][j] = acc[h * 4 + i][g * 4 + j];
            store_block<T>(t, part, mine, m0 + wm + h * 64, n0 + wn + g * 64, block);
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
}

// Few rows of A (BM = 32 or 64), k contiguous in both: bound by reading B, so
// the tile is 64 rows of B by all of A's, and STAGES - 1 stages are on their
// way at a time: 5 for 32 rows, 4 for 64, which with two workgroups a CU is 80
// or 64 KiB of B in flight (two stages of a 128 x 128 tile, 32 KiB, reached
// 3.6 TB/s).  B is read once and past the L2 (nt).  32 x 2048 x 151936 to fp32:
// 118 us, of which reading B alone takes 95 in the same pattern; a weight row
// more costs nothing until the output shows (1 row 102 us, 64 rows 134).
template <int ESIZE, int BM, int STAGES>
__global__ __launch_bounds__(256) void gemm_few_rows_kernel(GemmTask t, int64_t stages_per_slice,
                                                            float* part) {
    using T = typename elem<ESIZE>::type;
    constexpr int BN = kFewRowsCols, NT = 256;
    constexpr int IM = BM / 16, JN = BN / 64;       // a wavefront: BM x BN / 4 results
    using LA = TileLoader<ESIZE, true, true, BM, NT>;
    using LB = TileLoader<ESIZE, true, true, BN, NT>;
    constexpr int BYTES = LA::BYTES + LB::BYTES, LOADS = LA::LOADS + LB::LOADS;
    __shared__ __align__(1024) char lds[STAGES * BYTES];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t n0 = (int64_t)blockIdx.x * BN;
    LA la;
    LB lb;
    la.init(t.a, t.a_m, 0, t.m);
    lb.init(t.b, t.b_n, n0, t.n);
    const typename LA::Place pa = LA::place(0);
    const typename LB::Place pb = LB::place(wave * (BN / 4));
    const typename LA::Direct da = la.direct();
    const typename LB::Direct db = lb.direct();
    const int64_t whole = t.k / LA::KB, all = (t.k + LA::KB - 1) / LA::KB;
    const int64_t s0 = blockIdx.y * stages_per_slice;
    const int64_t end = s0 + stages_per_slice < all ? s0 + stages_per_slice : all;
    const int64_t s1 = end < whole ? end : whole;
    f32x4 acc[IM][JN] = {};
    // Workgroups begin at different stages: rows a power of two apart would
    // otherwise be read at one place of each by all workgroups at once, from
    // few of the memory's channels (32 x 4096 x 151936 258 us, so 231).
    const int64_t shift = s0 < s1 ? blockIdx.x % (s1 - s0) : 0;
    auto stage = [&](int64_t s) {
        char* p = lds + (s - s0) % STAGES * BYTES;
        const int64_t at = s + shift < s1 ? s + shift : s + shift - (s1 - s0);
        la.load(da, at, p);
        lb.template load<true>(db, at, p + LA::BYTES);
    };
    auto multiply = [&](const char* p) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            u32x4_t av[IM], bv[JN];
#pragma unroll
            for (int j = 0; j < JN; ++j)
                bv[j] = LB::fragment(p + LA::BYTES, pb, j, s);
#pragma unroll
            for (int i = 0; i < IM; ++i)
                av[i] = LA::fragment(p, pa, i, s);
#pragma unroll
            for (int i = 0; i < IM; ++i)
#pragma unroll
                for (int j = 0; j < JN; ++j)
                    acc[i][j] = mma<ESIZE>(bv[j], av[i], acc[i][j]);
        }
    };
    // a stage that k ends in comes first
    if (end > whole) {
        la.load_tail(whole, t.k, lds);
        lb.load_tail(whole, t.k, lds + LA::BYTES);
        stage_barrier();
        multiply(lds);
        stage_barrier();
    }
    for (int64_t s = s0; s < s0 + STAGES - 1 && s < s1; ++s)
        stage(s);
    for (int64_t s = s0; s < s1; ++s) {
        // stage s has landed when only the later ones are outstanding
        if (s + STAGES - 1 <= s1)
            wait_loads<(STAGES - 2) * LOADS>();
        else
            wait_loads<0>();
        // every wavefront's has, and all have read the stage before
        bare_barrier();
        if (s + STAGES - 1 < s1)
            stage(s + STAGES - 1);
        multiply(lds + (s - s0) % STAGES * BYTES);
    }
    // the tile through LDS, 4 results of a row a thread
    constexpr int LD = BN + 4;
    static_assert(BM * LD * 4 <= STAGES * BYTES, "the results fit");
    float* c = (float*)lds;
    stage_barrier();
#pragma unroll
    for (int i = 0; i < IM; ++i)
#pragma unroll
        for (int j = 0; j < JN; ++j)
            *(f32x4*)(c + (i * 16 + (lane & 15)) * LD + wave * (BN / 4) + j * 16 + (lane >> 4) * 4) =
                acc[i][j];
    __syncthreads();
    constexpr int ACROSS = BN / 4;                  // threads of a row
    const int64_t n = n0 + threadIdx.x % ACROSS * 4;
    for (int m = threadIdx.x / ACROSS; m < BM && m < t.m; m += NT / ACROSS) {
        const f32x4 v = *(const f32x4*)(c + m * LD + threadIdx.x % ACROSS * 4);
        float* p = part ? part + ((int64_t)blockIdx.y * t.m + m) * t.n + n : nullptr;
        if (n + 4 <= t.n) {
            if (part)
                keep4(p, v);
            else
                store_results<T>(t, m, n, v);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < t.n) {
                    if (part)
                        p[e] = v[e];
                    else
                        store_result<T>(t, m, n + e, v[e]);
                }
        }
    }
}

template <int ESIZE, bool AK, bool BK, bool DIRECT, int BM, int BN, int WM, int WN>
hipError_t launch_tile(const GemmTask& t, const GemmPlan& p, hipStream_t stream) {
    const uint32_t tm = (uint32_t)((t.m + BM - 1) / BM), tn = (uint32_t)((t.n + BN - 1) / BN);
    return launch(gemm_tile_kernel<ESIZE, AK, BK, DIRECT, BM, BN, WM, WN>,
                  dim3(tm * tn * (uint32_t)p.slices), dim3(WM * WN * 64), 0, stream, t, tm, tn,
                  p.stages_per_slice, p.slices > 1 ? (float*)t.ws : nullptr);
}

template <int ESIZE, bool AK, bool BK>
hipError_t launch_layout(const GemmTask& t, const GemmPlan& p, hipStream_t stream) {
    if (!p.direct)
        return launch_tile<ESIZE, AK, BK, false, 128, 128, 2, 2>(t, p, stream);
    if constexpr (AK && BK)
        if (p.tile <= 64) {
            const dim3 grid((uint32_t)((t.n + kFewRowsCols - 1) / kFewRowsCols), (uint32_t)p.slices);
            const dim3 block(256);
            float* part = p.slices > 1 ? (float*)t.ws : nullptr;
            return p.tile == 32 ? launch(gemm_few_rows_kernel<ESIZE, 32, 6>, grid, block, 0,
                                         stream, t, p.stages_per_slice, part)
                                : launch(gemm_few_rows_kernel<ESIZE, 64, 5>, grid, block, 0,
                                         stream, t, p.stages_per_slice, part);
        }
    if constexpr (ESIZE == 2)
        if (p.tile == 256)
            return launch_tile<ESIZE, AK, BK, true, 256, 256, 2, 4>(t, p, stream);
    return launch_tile<ESIZE, AK, BK, true, 128, 128, 2, 2>(t, p, stream);
}

template <int ESIZE>
hipError_t launch_tiles(const GemmTask& t, const GemmPlan& p, hipStream_t stream) {
    if (!t.a_k1)
        return launch_layout<ESIZE, false, false>(t, p, stream);
    return t.b_k1 ? launch_layout<ESIZE, true, true>(t, p, stream)
                  : launch_layout<ESIZE, true, false>(t, p, stream);
}

}  // namespace
}  // namespace vpa
