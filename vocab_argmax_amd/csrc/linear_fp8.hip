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
// off in the 2-norm; +-448 * 448 that cancel leave nothing of products of 1 beside
// them).  Widened to bf16, which holds every e4m3 value, products are summed in full
// fp32 at half the rate: EXACT, which is what callers get who do not ask for the
// other.
#include <type_traits>

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

// The first n bytes at p (n may be 0 or negative), 0 after them; p at 16 bytes.
__device__ __forceinline__ u32x4_t first_bytes(const char* p, int64_t n) {
    if (n >= 16)
        return *(const u32x4_t*)p;
    union {
        uint8_t e[16];
        u32x4_t v;
    } u;
    u.v = u32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 15; ++i)
        if (i < n)
            u.e[i] = ((const uint8_t*)p)[i];
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

// The same by the 8-bit instruction (see above).
__device__ __forceinline__ f32x4 mma_fast(const u32x4_t (&p)[2], const u32x4_t (&q)[2]) {
    typedef int i32x8 __attribute__((ext_vector_type(8)));
    const i32x8 a = {(int)p[0][0], (int)p[0][1], (int)p[0][2], (int)p[0][3],
                     (int)p[1][0], (int)p[1][1], (int)p[1][2], (int)p[1][3]};
    const i32x8 b = {(int)q[0][0], (int)q[0][1], (int)q[0][2], (int)q[0][3],
                     (int)q[1][0], (int)q[1][1], (int)q[1][2], (int)q[1][3]};
    // e4m3 in both, and no scales of the instruction's own
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{0, 0, 0, 0}, 0, 0, 0, 0, 0,
                                                            0);
}

// A row's 128 bytes widened, for products with several others.
struct Wide {
    bf16x8 v[4];
    __device__ __forceinline__ Wide() {}
    __device__ __forceinline__ explicit Wide(const u32x4_t (&p)[2]) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = widen(p[e / 2][e % 2 * 2], p[e / 2][e % 2 * 2 + 1]);
    }
};
__device__ __forceinline__ f32x4 mma_wide(const Wide& p, const Wide& q) {
    f32x4 d = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(p.v[e], q.v[e], d, 0, 0, 0);
    return d;
}

// A row's 128 bytes as an operand of either product.
template <bool EXACT>
struct Operand : Wide {
    __device__ __forceinline__ explicit Operand(const u32x4_t (&p)[2]) : Wide(p) {}
};
template <>
struct Operand<false> {
    u32x4_t v[2];
    __device__ __forceinline__ explicit Operand(const u32x4_t (&p)[2]) : v{p[0], p[1]} {}
};
__device__ __forceinline__ f32x4 mma(const Operand<true>& p, const Operand<true>& q) {
    return mma_wide(p, q);
}
__device__ __forceinline__ f32x4 mma(const Operand<false>& p, const Operand<false>& q) {
    return mma_fast(p.v, q.v);
}

// Weight scales of a workgroup's columns, one for each block of k: the same in
// all lanes, read through the scalar cache.
typedef const float __attribute__((address_space(4))) * scalar_floats;
__device__ __forceinline__ scalar_floats weight_scales(const Fp8Task& f, int64_t n) {
    return (scalar_floats)uniform(f.b_scale + n / kScaleBlock * f.ldb_scale);
}

// The scales of up to 64 rows (of x, or of blocks of W's rows) for one block of k,
// straight to LDS; rows past the last repeat it.
struct ScaleLoader {
    const float* base;
    uint32_t off, size;
    // rows `first` and up to 63 more of `rows`; none where first is past them
    __device__ __forceinline__ void init(const float* p, int64_t ld, int64_t first, int64_t rows) {
        first = first < rows ? first : rows - 1;
        const int left = rows - first < 64 ? (int)(rows - first) : 64;
        const int r = (int)(threadIdx.x & 63);
        base = p + first * ld;
        off = (uint32_t)((r < left ? r : left - 1) * ld * 4);
        size = (uint32_t)((left - 1) * ld * 4 + 4);
    }
    // to `lds` and the 255 bytes after it
    __device__ __forceinline__ void load(int64_t block, char* lds) const {
#ifdef __HIP_DEVICE_COMPILE__
        const auto buf = __builtin_amdgcn_make_buffer_rsrc(
            uniform(base + block), 0, __builtin_amdgcn_readfirstlane(size), 0x00020000);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(buf, (lds_ptr)lds, 4, off, 0, 0, 0);
#endif
    }
};

// What a wavefront of the tile kernel adds to its results: a pass is 32 rows of 64
// columns, 8 columns of a row a lane, and is loaded while the one before is stored.
// (store_block's passes are 16 rows, 8 waits for memory where this has 4: with it
// 4096^3 with a residual took 92 us and 77 so, 2048 x 2048 x 8192 60 and 44.)
struct ResidualAhead {
    u32x4_t v[4];
    const uint16_t* p;
    int64_t ld, rows;
    bool any;
    // rows m0 and on, columns n0 and on; `none`: sums of a slice take no residual
    __device__ __forceinline__ void init(const GemmTask& t, int64_t m0, int64_t n0, bool none) {
        const int lane = threadIdx.x & 63;
        const int64_t n = n0 + (lane & 7) * 8, m = m0 + (lane >> 3);
        any = t.residual && !none && n + 8 <= t.n;
        ld = t.ldr;
        rows = t.m - m;
        p = (const uint16_t*)t.residual + m * ld + n;
    }
    __device__ __forceinline__ void fetch(int pass) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t row = pass * 32 + k * 8;
            v[k] = u32x4_t{0x80008000u, 0x80008000u, 0x80008000u, 0x80008000u};   // -0
            if (any && row < rows)
                v[k] = ((const Loose16*)(p + row * ld))->v;
        }
    }
};

// 8 finished results of a row.
__device__ __forceinline__ void store8(const GemmTask& t, int64_t m, int64_t n, f32x4 (&v)[2],
                                       u32x4_t res) {
    if (t.bias)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            v[h] += load4((const uint16_t*)t.bias + n + h * 4);
    const auto each = [&](auto a) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            v[h] = act4<a()>(v[h]);
    };
    using std::integral_constant;
    if (t.act == VPA_ACT_RELU)
        each(integral_constant<int, VPA_ACT_RELU>{});
    else if (t.act == VPA_ACT_GELU)
        each(integral_constant<int, VPA_ACT_GELU>{});
    else if (t.act == VPA_ACT_SILU)
        each(integral_constant<int, VPA_ACT_SILU>{});
#pragma unroll
    for (int e = 0; e < 8; ++e)
        v[e / 4][e % 4] += vec_elem<2>(res, e);
    if (t.out_f32) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            store4((float*)t.y + m * t.ldy + n + h * 4, v[h]);
        return;
    }
    const u32x4_t o = {pack_bf16(v[0][0], v[0][1]), pack_bf16(v[0][2], v[0][3]),
                       pack_bf16(v[1][0], v[1][1]), pack_bf16(v[1][2], v[1][3])};
    __builtin_nontemporal_store(o, &((Loose16*)((uint16_t*)t.y + m * t.ldy + n))->v);
}

// store_block with 8 results of a row a lane: block `block` of those that a
// wavefront stores one below the other, the first at row m0.
__device__ __forceinline__ void store_block8(const GemmTask& t, float* part, char* lds, int64_t m0,
                                             int64_t n0, int block, int blocks,
                                             const f32x4 (&acc)[4][4], ResidualAhead& res) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = i * 16 + (lane & 15), c = j * 4 + (lane >> 4);
            *(f32x4*)(lds + r * 256 + ((c ^ (r & 15)) << 4)) = acc[i][j];
        }
    // the wavefront's own LDS, in order (see store_block)
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int64_t n = n0 + (lane & 7) * 8;
    const int left = t.n - n < 8 ? (int)(t.n - n) : 8;          // results of this lane, or < 1
    if (n0 >= t.n)
        return;
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
        u32x4_t now[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            now[k] = res.v[k];
        const int pass = block * 2 + half;
        if (pass + 1 < blocks * 2)
            res.fetch(pass + 1);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int r = half * 32 + k * 8 + (lane >> 3), c = (lane & 7) * 2;
            const int64_t m = m0 + block * 64 + r;
            f32x4 v[2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
                v[h] = *(const f32x4*)(lds + r * 256 + (((c + h) ^ (r & 15)) << 4));
            if (m >= t.m)
                continue;
            float* p = part ? part + m * t.n + n : nullptr;
            if (left == 8) {
                if (part) {
                    keep4(p, v[0]);
                    keep4(p + 4, v[1]);
                } else {
                    store8(t, m, n, v, now[k]);
                }
                continue;
            }
            // the lane that n ends in: its results once more, one by one
#pragma unroll 1
            for (int e = 0; e < left; ++e) {
                const float one = *(const float*)(lds + r * 256 +
                                                  (((c + e / 4) ^ (r & 15)) << 4) + e % 4 * 4);
                if (part)
                    p[e] = one;
                else
                    store_result<uint16_t>(t, m, n + e, one);
            }
        }
    }
}

// WM x WN wavefronts, each with BM/WM x BN/WN of the tile in its accumulators.
// With part set, the raw sums of a slice of k go to part[slice][m][n].
//
// As in the 16-bit products, a stage is 128 bytes of k, here one block of scales,
// and BUFS of them lie in LDS.  A wavefront holds the stage's fragments of W, and of
// x a ring of 4 that are read 4 products ahead, so that the accumulators, which
// the scaling keeps in ordinary registers, leave room.
// The barrier that says that the next stage has landed, and that every wavefront has
// read this one, stands before the first read from the next.
//
// The fast form: 8192^3 475-490 us, 2240-2310 TFLOP/s, the matrix cores busy half of
// the clocks: a product's 4 multiply-adds take issue slots beside it (a tenth of the
// time with everything else left in), and operands come at the rate of LDS and the
// caches (a fifth).  4096^3 63-67 us.  EXACT has four bf16 instructions for one of
// those, the widening (an instruction for 2 values) and smaller tiles, whose operands
// come twice as often: 916-937 and 120-130.  The 16-bit product of these sizes takes 790
// and 105.
template <bool EXACT, int BM, int BN, int WM, int WN, int BUFS>
__global__ __launch_bounds__(WM* WN * 64, 2) void fp8_tile_kernel(Fp8Task f, uint32_t tiles_m,
                                                               uint32_t tiles_n,
                                                               int64_t stages_per_slice,
                                                               float* part) {
    constexpr int NT = WM * WN * 64, RING = 4;
    constexpr int IM = BM / WM / 16, JN = BN / WN / 16;
    static_assert(IM % RING == 0 && JN == 4, "a ring of fragments, blocks of 64 columns");
    static_assert(BN / WN <= kScaleBlock && kScaleBlock % (BN / WN) == 0, "one scale of W");
    using LA = TileLoader<1, true, true, BM, NT>;
    using LB = TileLoader<1, true, true, BN, NT>;
    // x's scales, then W's; where stages are counted every wavefront loads some, past
    // the first of them W's again
    constexpr int SCALES = LA::BYTES + LB::BYTES, XWAVES = BM / 64;
    constexpr int SWAVES = BUFS > 2 ? WM * WN : XWAVES + 1;
    constexpr int STAGE = (SCALES + SWAVES * 256 + 1023) / 1024 * 1024;
    constexpr int LOADS = LA::LOADS + LB::LOADS + 1;
    static_assert(XWAVES < WM * WN, "a wavefront for each 64 scales");
    static_assert((BUFS & (BUFS - 1)) == 0, "a mask for stages");
    __shared__ __align__(1024) char lds[BUFS * STAGE];
    const GemmTask& t = f.g;
    uint32_t slice, tm, tn;
    tile_of_block(blockIdx.x, gridDim.x, tiles_m, tiles_n, slice, tm, tn);
    const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN * (BM / WM), wn = wave % WN * (BN / WN);
    LA la;
    LB lb;
    la.init(t.a, t.a_m, m0, t.m);
    lb.init(t.b, t.b_n, n0, t.n);
    ScaleLoader ls;
    if (wave < XWAVES)
        ls.init(f.a_scale, f.lda_scale, m0 + wave * 64, t.m);
    else
        ls.init(f.b_scale, f.ldb_scale, n0 / kScaleBlock, (t.n + kScaleBlock - 1) / kScaleBlock);
    const int64_t whole = t.k / 128, all = (t.k + 127) / 128;
    const int64_t s0 = slice * stages_per_slice;
    const int64_t end = s0 + stages_per_slice < all ? s0 + stages_per_slice : all;
    const int64_t s1 = end < whole ? end : whole;
    const typename LA::Place pa = LA::place(wm);
    const typename LB::Place pb = LB::place(wn);
    const int scale_at = SCALES + (wm + (lane & 15)) * 4;
    const int wscale_at = SCALES + XWAVES * 256 + wn / kScaleBlock * 4;
    f32x4 acc[IM][JN] = {};
    const typename LA::Direct da = la.direct();
    const typename LB::Direct db = lb.direct();
    auto stage = [&](int64_t s, char* lds) {
        __builtin_amdgcn_s_setprio(0);
        la.load(da, s, lds);
        lb.load(db, s, lds + LA::BYTES);
        if (wave < SWAVES)
            ls.load(s, lds + SCALES + wave * 256);
    };
    const auto buffer = [&](int64_t s) { return lds + ((int)(s - s0) & (BUFS - 1)) * STAGE; };
    // stage s is in LDS and every wavefront has come here; `more` stages of those
    // after it may be on their way, if so many there are
    const auto landed = [&](int64_t s, auto more) {
        if constexpr (BUFS == 2) {
            stage_barrier();
        } else {
            if (s + more() < s1)
                wait_loads<more() * LOADS>();
            else
                wait_loads<0>();
            bare_barrier();
        }
    };
    using std::integral_constant;
    u32x4_t av[RING][2], bv[JN][2];
    float sx[RING];
    auto read_a = [&](const char* lds, const typename LA::Place& p, int i) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            av[i % RING][h] = LA::fragment(lds, p, i, h);
        sx[i % RING] = *(const float*)(lds + scale_at + i * 64);
    };
    auto read_b = [&](const char* lds, const typename LB::Place& p, int j) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            bv[j][h] = LB::fragment(lds + LA::BYTES, p, j, h);
    };
    Wide wide[EXACT ? JN : 1];
    // A product's scaling, 4 multiply-adds, runs four products later: row i's follow row
    // i + 1's products one by one, and the last row's the next stage's first.
    f32x4 p[2][JN] = {};
    float scale[2] = {};
    auto add = [&](int i, int j) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            acc[i][j][e] = __builtin_fmaf(p[i % 2][j][e], scale[i % 2], acc[i][j][e]);
        // here, not at the end of the stage with all of its products kept
        asm volatile("" : "+v"(acc[i][j]));
    };
    static_assert(IM % 2 == 0, "rows take turns");
    auto products = [&](int i, float sw, auto after) {
        Wide a;
        if constexpr (EXACT)
            a = Wide(av[i % RING]);
        scale[i % 2] = sx[i % RING] * sw;
#pragma unroll
        for (int j = 0; j < JN; ++j) {
            if constexpr (EXACT)
                p[i % 2][j] = mma_wide(wide[j], a);
            else
                p[i % 2][j] = mma_fast(bv[j], av[i % RING]);
            add((i + IM - 1) % IM, j);
            after(j);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    const auto nothing = [](int) {};
    auto finish = [&] {
#pragma unroll
        for (int j = 0; j < JN; ++j)
            add(IM - 1, j);
    };
    auto widen_b = [&] {
        if constexpr (EXACT)
#pragma unroll
            for (int j = 0; j < JN; ++j)
                wide[j] = Wide(bv[j]);
    };
    // a stage that k ends in comes first, so that the loop has whole ones only
    if (end > whole) {
        la.load_tail(whole, t.k, buffer(s0 + 1));
        lb.load_tail(whole, t.k, buffer(s0 + 1) + LA::BYTES);
        if (wave < SWAVES)
            ls.load(whole, buffer(s0 + 1) + SCALES + wave * 256);
        stage_barrier();
#pragma unroll
        for (int j = 0; j < JN; ++j)
            read_b(buffer(s0 + 1), pb, j);
        widen_b();
#pragma unroll
        for (int i = 0; i < IM; ++i) {
            read_a(buffer(s0 + 1), pa, i);
            products(i, *(const float*)(buffer(s0 + 1) + wscale_at), nothing);
        }
        stage_barrier();
    }
    if (s0 < s1) {
#pragma unroll
        for (int i = 0; i < BUFS; ++i)
            if (s0 + i < s1)
                stage(s0 + i, buffer(s0 + i));
        landed(s0, integral_constant<int, BUFS - 1>{});
#pragma unroll
        for (int j = 0; j < JN; ++j)
            read_b(buffer(s0), pb, j);
#pragma unroll
        for (int i = 0; i < RING; ++i)
            read_a(buffer(s0), pa, i);
    }
    const bool early = wave < WM * WN / 2;
    // (scalar loads of it would make every wait one for all of LDS's answers)
    float sw = *(const float*)(lds + wscale_at);
    for (int64_t s = s0; s + 1 < s1; ++s) {
        char *now = buffer(s), *next = buffer(s + 1);
        float sw_next = 0.0f;
        widen_b();
        const typename LA::Place a = pa.again();
        const typename LB::Place b = pb.again();
#pragma unroll
        for (int i = 0; i < IM; ++i) {
            // the last row's products are the last to use a fragment of W
            products(i, sw, [&](int j) {
                if (i == IM - 1)
                    read_b(next, b, j);
            });
            if (i == 0)
                __builtin_amdgcn_s_setprio(1);
            if (i == IM - RING) {
                // the next stage has landed, and this one has been read
                landed(s + 1, integral_constant<int, BUFS - 2>{});
                if (early && s + BUFS < s1)
                    stage(s + BUFS, now);
            }
            if (i == IM - RING + 2 && !early && s + BUFS < s1)
                stage(s + BUFS, now);
            if (i < IM - RING)
                read_a(now, a, i + RING);
            else
                read_a(next, a, i + RING - IM);
            if (i == IM - RING)
                sw_next = *(const float*)(next + wscale_at);
            __builtin_amdgcn_sched_barrier(0);
        }
        sw = sw_next;
    }
    if (s0 < s1) {
        const char* now = buffer(s1 - 1);
        widen_b();
#pragma unroll
        for (int i = 0; i < IM; ++i) {
            products(i, sw, nothing);
            if (i < IM - RING)
                read_a(now, pa, i + RING);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    ResidualAhead res;
    res.init(t, m0 + wm, n0 + wn, part != nullptr);
    res.fetch(0);
    finish();
    bare_barrier();                                // this stage's fragments have been read
    if (part)
        part += slice * t.m * t.n;
    static_assert(WM * WN * 16384 <= BUFS * STAGE, "a block of results for each wavefront");
    char* mine = lds + wave * 16384;
#pragma unroll
    for (int h = 0; h < IM / 4; ++h) {
        f32x4 block[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                block[i][j] = acc[h * 4 + i][j];
        store_block8(t, part, mine, m0 + wm, n0 + wn, h, IM / 4, block, res);
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

// Few rows of x: bound by reading W, so the tile is 64 rows of W by 32 or 64 of x,
// which has as many or (see plan_fp8) a few times those, with STAGES - 1 stages on
// their way (as in the 16-bit products).  Up to 64 rows products are exact: the
// matrix cores and the widening have time to spare (with the 8-bit instruction 64 x
// 4096 x 11008 took 24 us for 26), in the fast form too.
//
// Workgroups on a CU beside one another hide more than stages on their way: 32 x
// 2048 x 151936 62 us (5.1 TB/s) with 4 stages, 3 workgroups a CU, and 73 with 6,
// two; 64 x 2048 x 151936 79 with 2, 84 with 3, 93 with 4.  64 rows keep 4 stages
// where no CU gets a second workgroup (64 x 4096 x 4096 13.4 us, with 3 14.0).
template <bool EXACT, int BM, int STAGES>
__global__ __launch_bounds__(256) void fp8_few_rows_kernel(Fp8Task f, int64_t stages_per_slice,
                                                           float* part) {
    constexpr int BN = kFewRowsCols, NT = 256, WAVES = 4;
    constexpr int IM = BM / 16;                     // a wavefront: BM x 16 results
    using LA = TileLoader<1, true, true, BM, NT>;
    using LB = TileLoader<1, true, true, BN, NT>;
    // x's scales: every wavefront loads its own copy, so that each has as many
    // loads under way
    constexpr int SCALES = LA::BYTES + LB::BYTES, BYTES = SCALES + WAVES * 256;
    constexpr int LOADS = LA::LOADS + LB::LOADS + 1;
    __shared__ __align__(1024) char lds[STAGES * BYTES];
    const GemmTask& t = f.g;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * BN, m0 = (int64_t)blockIdx.z * BM;
    LA la;
    LB lb;
    la.init(t.a, t.a_m, m0, t.m);
    lb.init(t.b, t.b_n, n0, t.n);
    ScaleLoader ls;
    ls.init(f.a_scale, f.lda_scale, m0, t.m);
    const scalar_floats ws = weight_scales(f, n0);
    const typename LA::Place pa = LA::place(0);
    const typename LB::Place pb = LB::place(wave * 16);
    const typename LA::Direct da = la.direct();
    const typename LB::Direct db = lb.direct();
    const int64_t whole = t.k / 128, all = (t.k + 127) / 128;
    const int64_t s0 = blockIdx.y * stages_per_slice;
    const int64_t end = s0 + stages_per_slice < all ? s0 + stages_per_slice : all;
    const int64_t s1 = end < whole ? end : whole;
    f32x4 acc[IM] = {};
    // workgroups begin at different stages (see the 16-bit kernel)
    const int64_t shift = s0 < s1 ? blockIdx.x % (s1 - s0) : 0;
    auto at = [&](int64_t s) { return s + shift < s1 ? s + shift : s + shift - (s1 - s0); };
    auto stage = [&](int64_t s) {
        char* p = lds + (s - s0) % STAGES * BYTES;
        la.load(da, at(s), p);
        lb.template load<true>(db, at(s), p + LA::BYTES);
        ls.load(at(s), p + SCALES + wave * 256);
    };
    auto multiply = [&](const char* p, float sw) {
        u32x4_t v[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            v[h] = LB::fragment(p + LA::BYTES, pb, 0, h);
        const Operand<EXACT> w(v);
#pragma unroll
        for (int i = 0; i < IM; ++i) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                v[h] = LA::fragment(p, pa, i, h);
            const float sc = *(const float*)(p + SCALES + wave * 256 + (i * 16 + (lane & 15)) * 4) * sw;
            const f32x4 d = mma(w, Operand<EXACT>(v));
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[i][e] = __builtin_fmaf(d[e], sc, acc[i][e]);
        }
    };
    // a stage that k ends in comes first
    if (end > whole) {
        la.load_tail(whole, t.k, lds);
        lb.load_tail(whole, t.k, lds + LA::BYTES);
        ls.load(whole, lds + SCALES + wave * 256);
        stage_barrier();
        multiply(lds, ws[whole]);
        stage_barrier();
    }
    for (int64_t s = s0; s < s0 + STAGES - 1 && s < s1; ++s)
        stage(s);
    for (int64_t s = s0; s < s1; ++s) {
        const float sw = ws[at(s)];
        // stage s has landed when only the later ones are outstanding
        if (s + STAGES - 1 <= s1)
            wait_loads<(STAGES - 2) * LOADS>();
        else
            wait_loads<0>();
        // every wavefront's has, and all have read the stage before
        bare_barrier();
        if (s + STAGES - 1 < s1)
            stage(s + STAGES - 1);
        multiply(lds + (s - s0) % STAGES * BYTES, sw);
    }
    // the tile through LDS, 4 results of a row a thread
    constexpr int LD = BN + 4;
    static_assert(BM * LD * 4 <= STAGES * BYTES, "the results fit");
    float* c = (float*)lds;
    stage_barrier();
#pragma unroll
    for (int i = 0; i < IM; ++i)
        *(f32x4*)(c + (i * 16 + (lane & 15)) * LD + wave * 16 + (lane >> 4) * 4) = acc[i];
    __syncthreads();
    constexpr int ACROSS = BN / 4;                  // threads of a row
    const int64_t n = n0 + threadIdx.x % ACROSS * 4;
    for (int r = threadIdx.x / ACROSS; r < BM && m0 + r < t.m; r += NT / ACROSS) {
        const int64_t m = m0 + r;
        const f32x4 v = *(const f32x4*)(c + r * LD + threadIdx.x % ACROSS * 4);
        float* p = part ? part + ((int64_t)blockIdx.y * t.m + m) * t.n + n : nullptr;
        if (n + 4 <= t.n) {
            if (part)
                keep4(p, v);
            else
                store_results<uint16_t>(t, m, n, v);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < t.n) {
                    if (part)
                        p[e] = v[e];
                    else
                        store_result<uint16_t>(t, m, n + e, v[e]);
                }
        }
    }
}

// At most 16 rows of x and too few columns for the ring: a workgroup of WAVES
// wavefronts takes 16 rows of W, whose k they split and whose sums they join in
// LDS, in order; W goes straight from memory to the wavefronts' registers, D
// blocks at a time (as in the 16-bit products).  1 x 4096 x 4096 6 us, latency; 8 x
// 4096 x 16000 17.8, in the ring 19.1; past 256 tiles of it the ring is faster (8 x
// 4096 x 32000 28.8 and 33.3).
template <int D, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void fp8_rows_kernel(Fp8Task f) {
    __shared__ f32x4 sums[WAVES][64];
    const GemmTask& t = f.g;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int r = lane & 15, q = lane >> 4;
    // rows past the end repeat the last one: their sums are not stored
    const int64_t xr = r < t.m ? r : t.m - 1;
    const char* w = (const char*)t.b + (n0 + r < t.n ? n0 + r : t.n - 1) * t.b_n;
    const char* x = (const char*)t.a + xr * t.a_m;
    const float* xs = f.a_scale + xr * f.lda_scale;
    const scalar_floats ws = weight_scales(f, n0);
    f32x4 acc = {};
    auto add = [&](const u32x4_t (&wv)[2], const u32x4_t (&xv)[2], float sc) {
        const f32x4 d = mma_exact(wv, xv);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            acc[e] = __builtin_fmaf(d[e], sc, acc[e]);
    };
    // COUNT whole blocks from s
    auto run = [&](int64_t s, auto count) {
        constexpr int COUNT = count();
        u32x4_t wv[COUNT][2], xv[COUNT][2];
        float sx[COUNT];
#pragma unroll
        for (int d = 0; d < COUNT; ++d) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t o = (s + d) * 128 + h * 64 + q * 16;
                wv[d][h] = __builtin_nontemporal_load((const u32x4_t*)(w + o));
                xv[d][h] = *(const u32x4_t*)(x + o);
            }
            sx[d] = xs[s + d];
        }
        __builtin_amdgcn_sched_barrier(0);          // all loads before the first wait
#pragma unroll
        for (int d = 0; d < COUNT; ++d)
            add(wv[d], xv[d], sx[d] * ws[s + d]);
    };
    const int64_t whole = t.k / 128, batches = whole / D;
    for (int64_t b = wave; b < batches; b += WAVES)
        run(b * D, std::integral_constant<int, D>{});
    for (int64_t s = batches * D + wave; s < whole; s += WAVES)
        run(s, std::integral_constant<int, 1>{});
    if (t.k > whole * 128 && wave == WAVES - 1) {
        u32x4_t wv[2], xv[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t k = whole * 128 + h * 64 + q * 16;
            wv[h] = first_bytes(w + k, t.k - k);
            xv[h] = first_bytes(x + k, t.k - k);
        }
        add(wv, xv, xs[whole] * ws[whole]);
    }
    sums[wave][lane] = acc;
    __syncthreads();
    // n fastest; in a block n is (lane / 16) * 4 + e and m is lane % 16
    const int m = threadIdx.x / 16, n = threadIdx.x % 16;
    if (m >= t.m || m >= 16 || n0 + n >= t.n)
        return;
    const int place = m + (n >> 2) * 16;
    float v = sums[0][place][n & 3];
#pragma unroll
    for (int i = 1; i < WAVES; ++i)
        v += sums[i][place][n & 3];
    store_result<uint16_t>(t, m, n0 + n, v);
}

int64_t as_16_bits(int64_t k) {
    return (k + 1) / 2;
}
// A plan of `blocks` tiles, fewer than there are CUs: slices of at least 8 stages
// until every CU has one.
GemmPlan plan_a_round(int tile, int64_t blocks, int64_t k) {
    GemmPlan p{};
    const int64_t stages = (k + 127) / 128;
    int64_t s = 256 / blocks;
    s = s > stages / 8 ? stages / 8 : s;
    s = s < 1 ? 1 : s;
    p.tile = tile;
    p.stages_per_slice = (stages + s - 1) / s;
    p.slices = (int32_t)((stages + p.stages_per_slice - 1) / p.stages_per_slice);
    return p;
}
// More than 64 rows in 64-tiles while a round of workgroups holds them (128 x 4096 x
// 4096 18.5 us, in 128-tiles 21.9, fast 15.8 and 18.5; 100 x 2048 x 8192 15.3 and 20.4,
// fast 11.8 and 16.5; 256 x 4096 x 4096 26.5 and 26.9, fast 19.9 and 22.0; but 128 x
// 8192 x 8192 48 and 33, fast 35.7 and 29.9), then in 128-tiles while a round holds
// those (fast, 512 x 8192 x 8192 61 us, in two slices or two rounds 75; 512 x 4096 x 4096
// 25.6 in the two slices that fit, 28.7 in one, 26.6 in four).  Else the plan of a 16-bit
// product whose rows have as many bytes, whose stages, tiles and costs are alike.
// Exact products have no 256-tiles: widening takes the registers of more.
// They take up to twice the time from 1024 rows on (4096^3 121 us, by the 8-bit
// instruction 64; 2048 x 2048 x 50257 400 and 257; 512 x 4096 x 4096 30.5 and 25.5),
// which is what the fast form is for.
GemmPlan plan_fp8(int64_t m, int64_t n, int64_t k, bool exact) {
    const auto blocks = [&](int64_t tile) {
        return ((m + tile - 1) / tile) * ((n + tile - 1) / tile);
    };
    if (m > 64 && blocks(64) <= 256)
        return plan_a_round(64, blocks(64), k);
    if (m > 64 && blocks(128) <= 256)
        return plan_a_round(128, blocks(128), k);
    GemmPlan p = plan_gemm(2, m, n, as_16_bits(k), true, true);
    if (exact && !p.rows_kernel && p.tile == 256) {
        p = GemmPlan{};
        p.tile = 128;
        p.slices = 1;
        p.stages_per_slice = (k + 127) / 128;
    }
    return p;
}
static_assert(kFewRowsCols == 64, "64-tiles");
size_t slices_bytes(const GemmPlan& p, int64_t m, int64_t n) {
    return p.slices > 1 ? (size_t)p.slices * (size_t)m * (size_t)n * 4 : 0;
}

template <bool EXACT, int TILE, int WM, int WN, int BUFS>
hipError_t launch_tile(const Fp8Task& f, const GemmPlan& p, hipStream_t stream) {
    const uint32_t tm = (uint32_t)((f.g.m + TILE - 1) / TILE);
    const uint32_t tn = (uint32_t)((f.g.n + TILE - 1) / TILE);
    return launch(fp8_tile_kernel<EXACT, TILE, TILE, WM, WN, BUFS>, dim3(tm * tn * (uint32_t)p.slices),
                  dim3(WM * WN * 64), 0, stream, f, tm, tn, p.stages_per_slice,
                  p.slices > 1 ? (float*)f.g.ws : nullptr);
}

hipError_t launch_planned(const Fp8Task& f, const GemmPlan& p, hipStream_t stream) {
    hipError_t e;
    // The fast form's 128-tiles of which no CU gets a second workgroup have its LDS for
    // 4 stages (512 x 8192 x 8192 61 us, with two 85; 128 x 2048 x 32000 21.8 and 25.8).
    // Exact products, which take longer over a stage, have two (512 x 8192 x 8192 72 us,
    // with four 78; 1024 x 4096 x 4096 40 and 43; 128 x 2048 x 32000 24 and 26).
    const bool deep = ((f.g.m + 127) / 128) * ((f.g.n + 127) / 128) * p.slices <= 256;
    if (p.tile <= 64) {
        const dim3 grid((uint32_t)((f.g.n + kFewRowsCols - 1) / kFewRowsCols), (uint32_t)p.slices,
                        (uint32_t)((f.g.m + p.tile - 1) / p.tile));
        float* part = p.slices > 1 ? (float*)f.g.ws : nullptr;
        const bool one = grid.x * grid.y * grid.z <= 256u;
        const auto kernel = f.g.m > 64 && !f.exact ? fp8_few_rows_kernel<false, 64, 4>
                            : p.tile == 32         ? fp8_few_rows_kernel<true, 32, 4>
                            : one                  ? fp8_few_rows_kernel<true, 64, 4>
                                                   : fp8_few_rows_kernel<true, 64, 2>;
        e = launch(kernel, grid, dim3(256), 0, stream, f, p.stages_per_slice, part);
    } else if (f.exact) {
        e = launch_tile<true, 128, 2, 2, 2>(f, p, stream);
    } else if (p.tile == 256) {
        e = launch_tile<false, 256, 2, 4, 2>(f, p, stream);
    } else {
        e = deep ? launch_tile<false, 128, 2, 2, 4>(f, p, stream)
                 : launch_tile<false, 128, 2, 2, 2>(f, p, stream);
    }
    return e != hipSuccess || p.slices == 1 ? e : launch_gemm_join(2, f.g, p.slices, stream);
}

}  // namespace

size_t fp8_workspace(int64_t m, int64_t n, int64_t k, bool exact) {
    const GemmPlan p = plan_fp8(m, n, k, exact);
    if (!p.first_m)
        return slices_bytes(p, m, n);
    const GemmPlan q = plan_rest(2, p, m, n, as_16_bits(k));
    const size_t first = slices_bytes(p, p.first_m, p.first_n), rest = slices_bytes(q, m, n);
    return first > rest ? first : rest;
}

// The 16-bit plan's launches, in smaller tiles at most.
int64_t fp8_threads(int64_t m, int64_t n, int64_t k, bool exact) {
    const int64_t planned = gemm_threads(2, m, n, as_16_bits(k), true, true);
    const int64_t tiles = (m + 127) / 128 * ((n + 127) / 128) * 256;
    return exact && m > 64 && tiles > planned ? tiles : planned;
}

hipError_t launch_fp8(const Fp8Task& f, hipStream_t stream) {
    const GemmTask& t = f.g;
    const GemmPlan p = plan_fp8(t.m, t.n, t.k, f.exact);
    if (p.rows_kernel) {
        const int waves = linear_rows_waves(t.n);
        const dim3 grid((uint32_t)((t.n + 15) / 16)), block((uint32_t)waves * 64);
        return waves == 8 ? launch(fp8_rows_kernel<8, 8>, grid, block, 0, stream, f)
                          : launch(fp8_rows_kernel<8, 4>, grid, block, 0, stream, f);
    }
    if (!p.first_m)
        return launch_planned(f, p, stream);
    Fp8Task a = f, r = f;                           // the first part and the rest
    auto past = [](const void* q, int64_t bytes) { return q ? (char*)q + bytes : nullptr; };
    a.g.m = p.first_m;
    a.g.n = p.first_n;
    const int64_t dm = a.g.m < t.m ? a.g.m : 0, dn = a.g.n < t.n ? a.g.n : 0;
    r.g.m -= dm;
    r.g.n -= dn;
    r.g.a = past(t.a, dm * t.a_m);
    r.g.b = past(t.b, dn * t.b_n);
    r.g.bias = past(t.bias, dn * 2);
    r.g.residual = past(t.residual, (dm * t.ldr + dn) * 2);
    r.g.y = past(t.y, (dm * t.ldy + dn) * (t.out_f32 ? 4 : 2));
    r.a_scale += dm * f.lda_scale;
    r.b_scale += dn / kScaleBlock * f.ldb_scale;    // (dn is a multiple of 256)
    int64_t m = t.m, n = t.n;
    const GemmPlan q = plan_rest(2, p, m, n, as_16_bits(t.k));
    const hipError_t e = launch_planned(a, p, stream);
    return e != hipSuccess ? e : launch_planned(r, q, stream);
}

}  // namespace vpa
