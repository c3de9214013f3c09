// gemm_tile.h -- the tiled matrix product on the matrix cores: one workgroup
// computes a BM x BN tile of C[m][n] = sum_k A(m, k) B(n, k).
//
// Operands are moved from memory to LDS by direct loads (16 bytes a lane, no
// registers), two stages deep: while one stage of 128 bytes of k per row is
// multiplied, the next is on its way; one barrier a stage.  An operand is
// stored either with its k contiguous ([row][k], AK / BK true) or with its
// rows contiguous ([k][row]); the latter is read from LDS with the
// transposing read, so all four layouts run on the same loop.
//
// Direct loads need addresses aligned to 16 bytes (and whole chunks of rows).
// Where an operand has other strides, its stages go through registers
// (DIRECT false): 16-byte loads of any alignment before the product, LDS
// writes after it.
//
// LDS layout, k contiguous: row r has 8 chunks of 16 bytes; chunk c lies at
// position c ^ ((r >> 1) & 7), so that the 16 rows a fragment read touches
// fall into different banks.  Rows contiguous: row k has chunks of 32 bytes;
// chunk c lies at position c ^ swizzle(k), so that the 16 k rows of one
// transposing read do.  The direct load writes lanes side by side, so the
// permutation is applied to the address that each lane reads from.
//
// The matrix instruction is given B's fragment first: its result then has 4
// consecutive n of one m in a lane, which is what row-major stores want.
#pragma once

#include "vpa_head_internal.h"
#include "vpa_math.h"

namespace vpa {

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef i16x4 __attribute__((address_space(3))) * lds_i16x4;
typedef __attribute__((address_space(3))) void* lds_ptr;
typedef const __attribute__((address_space(1))) void* global_ptr;

// A pointer that is the same in every lane, as one.
__device__ __forceinline__ void* uniform(const void* p) {
    const uint64_t v = (uint64_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return (void*)(((uint64_t)hi << 32) | lo);
}

// One operand's tile of ROWS rows and one stage of k, for NT threads.
template <int ESIZE, bool K1, bool DIRECT, int ROWS, int NT>
struct TileLoader {
    using T = typename elem<ESIZE>::type;
    static constexpr int VEC = 16 / ESIZE;              // elements of a 16-byte chunk
    static constexpr int KB = 128 / ESIZE;              // k of a stage
    static constexpr int BYTES = ROWS * 128;
    static constexpr int LOADS = BYTES / 16 / NT;       // 16-byte chunks of a thread
    static constexpr int ROW_CHUNKS = K1 ? 8 : ROWS / VEC;   // of an LDS row
    static constexpr int ROWS_PER_LOAD = NT / ROW_CHUNKS;    // LDS rows from load to load
    // loads after which the swizzle of a thread's LDS row repeats
    static constexpr int PERIOD = K1 ? (ROWS_PER_LOAD % 16 == 0 ? 1 : LOADS)
                                     : (32 / ROWS_PER_LOAD < LOADS ? 32 / ROWS_PER_LOAD : LOADS);
    static_assert(NT % ROW_CHUNKS == 0 && LOADS % PERIOD == 0, "whole rows a load");

    const char* base;            // the tile's first row at k = 0
    int64_t ld;                  // bytes from LDS row to LDS row
    int32_t left;                // rows of the operand from the tile's first (at most ROWS)
    bool narrow;                 // rows contiguous, and fewer than a chunk

    static __device__ __forceinline__ int swizzle(int k) {
        constexpr int n = ROWS * ESIZE / 32;            // 32-byte chunks of a row
        return ((k & 3) | (((k >> 3) & 3) << 2)) & (n - 1);
    }
    // operand element (from the LDS row's first) of the chunk at position pos of LDS row r
    static __device__ __forceinline__ int element(int r, int pos) {
        if constexpr (K1)
            return (pos ^ ((r >> 1) & 7)) * VEC;
        else
            return ((pos >> 1) ^ swizzle(r)) * (32 / ESIZE) + (pos & 1) * VEC;
    }
    static __device__ __forceinline__ int lds_row(int i) {
        return i * ROWS_PER_LOAD + threadIdx.x / ROW_CHUNKS;
    }
    static __device__ __forceinline__ int position() {
        return threadIdx.x % ROW_CHUNKS;
    }
    // bytes from base (+ k) of this thread's chunk of load i
    __device__ __forceinline__ int64_t offset(int i) const {
        const int r = lds_row(i);
        // rows past the operand repeat its last one: their products are not stored
        const int row = K1 && r >= left ? left - 1 : r;
        return row * ld + element(r, position()) * ESIZE;
    }
    // first row, and the operand's row count and stride in elements; with
    // DIRECT and rows contiguous, `rows` may count readable padding
    __device__ __forceinline__ void init(const void* p, int64_t stride, int64_t row0,
                                         int64_t rows) {
        base = (const char*)p + (K1 ? row0 * stride : row0) * ESIZE;
        ld = stride * ESIZE;
        left = rows - row0 < ROWS ? (int32_t)(rows - row0) : ROWS;
        narrow = !K1 && rows < VEC;
    }
    __device__ __forceinline__ const char* at_stage(int64_t stage) const {
        return base + stage * (K1 ? 128 : KB * ld);
    }

    // This thread's 32-bit offsets for direct loads, which see the tile's
    // stage as a buffer that ends with the operand's last element: a chunk
    // past it is not read (its products are not stored).
    struct Direct {
        uint32_t off[PERIOD];
        uint32_t step;           // bytes of PERIOD loads
        uint32_t size;           // of the buffer
    };
    __device__ __forceinline__ Direct direct() const {
        Direct d;
#pragma unroll
        for (int i = 0; i < PERIOD; ++i)
            d.off[i] = (uint32_t)(lds_row(i) * ld + element(lds_row(i), position()) * ESIZE);
        d.step = (uint32_t)(PERIOD * ROWS_PER_LOAD * ld);
        d.size = (uint32_t)(K1 ? (left - 1) * ld + 128 : (KB - 1) * ld + left * ESIZE);
        return d;
    }
    // a whole stage, straight to LDS; ONCE for an operand that nothing else reads
    template <bool ONCE = false>
    __device__ __forceinline__ void load(const Direct& d, int64_t stage, char* lds) const {
#ifdef __HIP_DEVICE_COMPILE__    // the host pass has no buffer type
        const auto buf = __builtin_amdgcn_make_buffer_rsrc(
            uniform(at_stage(stage)), 0, __builtin_amdgcn_readfirstlane(d.size), 0x00020000);
        const int wave_base = __builtin_amdgcn_readfirstlane((threadIdx.x & ~63) * 16);
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(buf, (lds_ptr)(lds + i * NT * 16 + wave_base),
                                                     16, d.off[i % PERIOD] + i / PERIOD * d.step,
                                                     0, 0, ONCE ? 2 : 0);   // 2: nt
#endif
    }
    // a whole stage to registers, and from there to LDS
    __device__ __forceinline__ void fetch(int64_t stage, u32x4_t (&v)[LOADS]) const {
        const char* p = at_stage(stage);
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int64_t o = offset(i);
            if constexpr (!K1) {
                const int col = element(lds_row(i), position());
                if (col + VEC > left) {                 // the operand's last columns
                    v[i] = part(p + o, left - col);
                    continue;
                }
            }
            v[i] = ((const Loose16*)(p + o))->v;
        }
    }
    static __device__ __forceinline__ void put(const u32x4_t (&v)[LOADS], char* lds) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            *(u32x4_t*)(lds + (i * NT + threadIdx.x) * 16) = v[i];
    }
    // the first n elements of a chunk (n may be 0 or negative), 0 after them
    static __device__ __forceinline__ u32x4_t part(const char* p, int n) {
        union {
            T e[VEC];
            u32x4_t v;
        } u;
        u.v = u32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if (e < n)
                u.e[e] = ((const T*)p)[e];
        return u.v;
    }
    // v without its first n elements, 0 after the others (n >= 0)
    static __device__ __forceinline__ u32x4_t moved_down(u32x4_t v, int n) {
        const uint64_t lo = v[0] | (uint64_t)v[1] << 32, hi = v[2] | (uint64_t)v[3] << 32;
        const int bits = n < VEC ? n * ESIZE * 8 : 128, in = bits & 63;
        const uint64_t both = lo >> in | (hi << 1) << (63 - in);
        const uint64_t l = bits < 64 ? both : bits < 128 ? hi >> in : 0;
        const uint64_t h = bits < 64 ? hi >> in : 0;
        return u32x4_t{(uint32_t)l, (uint32_t)(l >> 32), (uint32_t)h, (uint32_t)(h >> 32)};
    }
    // The stage that k ends in: 0 past k, and past the operand's contiguous
    // rows.  A chunk that reaches past an end is the one that stops there,
    // moved down, so that all loads are under way before the first is waited
    // for (464 x 785 x 10240 bf16 element by element 47 us, 41 so); what has
    // fewer elements than a chunk goes one by one.
    __device__ __forceinline__ void load_tail(int64_t stage, int64_t k, char* lds) const {
        if (narrow || (K1 && k < VEC)) {
            const char* p = at_stage(stage);
            const int k_left = (int)(k - stage * KB);
#pragma unroll 1
            for (int i = 0; i < LOADS; ++i) {
                const int r = lds_row(i), e = element(r, position());
                const int n = K1 ? k_left - e : (r < k_left ? left - e : 0);
                *(u32x4_t*)(lds + (i * NT + threadIdx.x) * 16) = part(p + offset(i), n);
            }
            return;
        }
        u32x4_t v[LOADS];
        int skip[LOADS];
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int r = lds_row(i), e = element(r, position());
            int64_t row, at;                        // of the chunk that is loaded
            if constexpr (K1) {
                const int64_t want = stage * KB + e;
                at = want < k - VEC ? want : k - VEC;
                skip[i] = (int)(want - at);
                row = r < left ? r : left - 1;
            } else {
                const int64_t want = stage * KB + r;
                at = e < left - VEC ? e : left - VEC;
                skip[i] = want < k ? (int)(e - at) : VEC;
                row = want < k ? want : k - 1;
            }
            v[i] = ((const Loose16*)(base + row * ld + at * ESIZE))->v;
        }
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            *(u32x4_t*)(lds + (i * NT + threadIdx.x) * 16) = moved_down(v[i], skip[i]);
    }
    // Fragments: 16 rows, 64 bytes of k (step 0 or 1 of a stage).  A lane's
    // LDS address is worked out once for the wavefront's first row (a multiple
    // of 64); fragment i, 16 i rows on, is a constant distance away (k
    // contiguous), or differs in the bits of the 32-byte chunk (k strided).
    struct Place {
        uint32_t at[K1 ? 2 : 1];
        // The same places, unknown to the compiler: it would otherwise keep
        // the sums with every fragment's and buffer's distance in registers
        // around the loop, which do not fit.
        __device__ __forceinline__ Place again() const {
            Place p = *this;
#pragma unroll
            for (int i = 0; i < (K1 ? 2 : 1); ++i)
                asm volatile("" : "+v"(p.at[i]));
            return p;
        }
    };
    static __device__ __forceinline__ Place place(int row) {
        const int lane = threadIdx.x & 63, q = lane >> 4;
        Place p;
        if constexpr (K1) {
            const int f = (lane >> 1) & 7;              // ((row + lane % 16) >> 1) & 7
#pragma unroll
            for (int s = 0; s < 2; ++s)
                p.at[s] = (row + (lane & 15)) * 128 + (((s * 4 + q) ^ f) << 4);
        } else if constexpr (ESIZE == 2) {
            // a transposing read: lane i of a group of 16 reads 8 bytes of row
            // k = i / 4 and is given column i of rows k..k+3
            const int k = q * 8 + ((lane >> 2) & 3);
            p.at[0] = k * ROWS * 2 + (((row >> 4) ^ swizzle(k)) << 5) + (lane & 3) * 8;
        } else {
            p.at[0] = row + (lane & 15);
        }
        return p;
    }
    static __device__ __forceinline__ u32x4_t fragment(const char* lds, const Place& p, int i,
                                                       int s) {
        if constexpr (K1) {
            return *(const u32x4_t*)(lds + p.at[s] + i * 2048);
        } else if constexpr (ESIZE == 2) {
            union {
                i16x4 h[2];
                u32x4_t v;
            } u;
            const char* c = lds + (p.at[0] ^ (i << 5));
#pragma unroll
            for (int h = 0; h < 2; ++h)
                u.h[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (lds_i16x4)(lds_ptr)(c + (s * 32 + h * 4) * ROWS * 2));
            return u.v;
        } else {
            const int q = (threadIdx.x & 63) >> 4;
            const int col = p.at[0] + i * 16;
            u32x4_t v;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int k = s * 16 + q * 4 + e;
                v[e] = *(const uint32_t*)(lds + k * ROWS * 4 + (((col >> 3) ^ swizzle(k)) << 5) +
                                          (col & 7) * 4);
            }
            return v;
        }
    }
};

// The barrier between stages.  A direct load to LDS is counted as a memory
// load, which a workgroup barrier does not wait for by itself: each wavefront
// waits for its own loads (and its LDS accesses), then for the others.
__device__ __forceinline__ void stage_barrier() {
    __builtin_amdgcn_s_waitcnt(0x0070);             // vmcnt(0) lgkmcnt(0)
    __syncthreads();
}

// A barrier that leaves memory loads outstanding: LDS accesses are done before
// it, and the compiler moves none across it.
__device__ __forceinline__ void bare_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);             // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Waits until at most N memory loads of this wavefront are outstanding.
template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N >= 0 && N < 64, "six bits of vmcnt");
    __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4 << 14) | 0x0F70);
}

// D += P Q^T for 16 rows of P and of Q over 64 bytes of k.
template <int ESIZE>
__device__ __forceinline__ f32x4 mma(u32x4_t p, u32x4_t q, f32x4 d) {
    if constexpr (ESIZE == 2) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, p),
                                                       __builtin_bit_cast(bf16x8, q), d, 0, 0, 0);
    } else {
        // element e of every lane is one step of 4 k; both operands hold the same k there
#pragma unroll
        for (int e = 0; e < 4; ++e)
            d = __builtin_amdgcn_mfma_f32_16x16x4f32(__builtin_bit_cast(float, (uint32_t)p[e]),
                                                     __builtin_bit_cast(float, (uint32_t)q[e]), d,
                                                     0, 0, 0);
        return d;
    }
}

// Block -> slice of k and tile: blocks are dealt to the 8 XCDs in turn, so
// each XCD is given a contiguous run of (slice, tile), ordered in columns of 4
// m tiles: the run's operands then share that XCD's L2, and a slice's are read
// by few XCDs (the gradient of x, 2048 x 50264 x 2048 in 4 slices: 453 us with
// every slice's tiles over all XCDs, 445 so).
__device__ __forceinline__ void tile_of_block(uint32_t block, uint32_t blocks, uint32_t tiles_m,
                                              uint32_t tiles_n, uint32_t& slice, uint32_t& tm,
                                              uint32_t& tn) {
    const uint32_t tiles = tiles_m * tiles_n, q = blocks / 8, r = blocks % 8, x = block % 8;
    uint32_t id = (x < r ? x * (q + 1) : r * (q + 1) + (x - r) * q) + block / 8;
    slice = blocks == tiles ? 0 : id / tiles;
    id -= slice * tiles;
    constexpr uint32_t G = 4;
    const uint32_t group = id / (G * tiles_n), first = group * G;
    const uint32_t size = tiles_m - first < G ? tiles_m - first : G;
    const uint32_t in = id - group * G * tiles_n;
    tm = first + in % size;
    tn = in / size;
}

}  // namespace vpa
