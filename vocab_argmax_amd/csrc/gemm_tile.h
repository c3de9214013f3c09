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
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

// 16 bytes at any element address.
struct __attribute__((packed, aligned(2))) Loose16 {
    u32x4_t v;
};

template <bool DIRECT>
struct tile_offset {
    using type = uint32_t;
};
template <>
struct tile_offset<false> {
    using type = int64_t;
};

// One operand's tile of ROWS rows and one stage of k, for NT threads.
template <int ESIZE, bool K1, bool DIRECT, int ROWS, int NT>
struct TileLoader {
    using T = typename elem<ESIZE>::type;
    static constexpr int VEC = 16 / ESIZE;              // elements of a 16-byte chunk
    static constexpr int KB = 128 / ESIZE;              // k of a stage
    static constexpr int BYTES = ROWS * 128;
    static constexpr int LOADS = BYTES / 16 / NT;
    static constexpr int ROW_CHUNKS = K1 ? 8 : ROWS / VEC;   // 16-byte chunks of an LDS row

    const char* base;            // the tile's first row at k = 0
    int64_t k_step;              // bytes from a stage to the next
    int32_t left;                // rows from the tile's first
    // bytes from base (+ k) of each of this thread's chunks; direct loads are
    // given operands whose tiles span less than 4 GiB
    using Offset = typename tile_offset<DIRECT>::type;
    Offset off[LOADS];

    static __device__ __forceinline__ int swizzle(int k) {
        constexpr int n = ROWS * ESIZE / 32;            // 32-byte chunks of a row
        return ((k & 3) | (((k >> 3) & 3) << 2)) & (n - 1);
    }
    // first row of the tile's chunk at position pos of LDS row r (k strided)
    static __device__ __forceinline__ int column(int r, int pos) {
        return ((pos >> 1) ^ swizzle(r)) * (32 / ESIZE) + (pos & 1) * VEC;
    }
    // first row, and the operand's row count and stride in elements; with
    // DIRECT and rows contiguous, `rows` may count readable padding
    __device__ __forceinline__ void init(const void* p, int64_t ld, int64_t row0, int64_t rows) {
        base = (const char*)p + (K1 ? row0 * ld : row0) * ESIZE;
        k_step = (K1 ? KB : KB * ld) * ESIZE;
        left = rows - row0 < ROWS ? (int32_t)(rows - row0) : ROWS;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int id = i * NT + threadIdx.x;
            const int r = id / ROW_CHUNKS, pos = id % ROW_CHUNKS;
            int64_t o;
            if constexpr (K1) {
                // rows past the operand repeat its last one: their products are not stored
                const int row = r < left ? r : left - 1;
                o = row * ld + (pos ^ ((r >> 1) & 7)) * VEC;
            } else {
                const int col = column(r, pos);
                o = r * ld + (DIRECT && col + VEC > left ? left - VEC : col);
            }
            off[i] = (Offset)(o * ESIZE);
        }
    }
    // a whole stage, straight to LDS
    __device__ __forceinline__ void load(int64_t stage, char* lds) const {
        const char* p = base + stage * k_step;
        const int wave_base = (threadIdx.x & ~63) * 16;
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            __builtin_amdgcn_global_load_lds((global_ptr)(p + off[i]),
                                             (lds_ptr)(lds + i * NT * 16 + wave_base), 16, 0, 0);
    }
    // a whole stage to registers, and from there to LDS
    __device__ __forceinline__ void fetch(int64_t stage, u32x4_t (&v)[LOADS]) const {
        const char* p = base + stage * k_step;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            if constexpr (!K1) {
                const int id = i * NT + threadIdx.x;
                const int col = column(id / ROW_CHUNKS, id % ROW_CHUNKS);
                if (col + VEC > left) {                 // the operand's last columns
                    v[i] = part(p + off[i], left - col);
                    continue;
                }
            }
            v[i] = ((const Loose16*)(p + off[i]))->v;
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
    // the stage that k ends in: 0 past k
    __device__ __forceinline__ void load_tail(int64_t stage, int64_t k, char* lds) const {
        const char* p = base + stage * k_step;
        const int k_left = (int)(k - stage * KB);
#pragma unroll 1
        for (int i = 0; i < LOADS; ++i) {
            const int id = i * NT + threadIdx.x;
            const int r = id / ROW_CHUNKS, pos = id % ROW_CHUNKS;
            Offset o = 0;
#pragma unroll
            for (int j = 0; j < LOADS; ++j)
                o = j == i ? off[j] : o;
            int n;
            if constexpr (K1)
                n = k_left - (pos ^ ((r >> 1) & 7)) * VEC;
            else
                n = r >= k_left ? 0 : (DIRECT ? VEC : left - column(r, pos));
            *(u32x4_t*)(lds + id * 16) = part(p + o, n);
        }
    }
    // the fragment of 16 rows from `row`, 64 bytes of k from chunk s * 4
    static __device__ __forceinline__ u32x4_t fragment(const char* lds, int row, int s) {
        const int lane = threadIdx.x & 63;
        if constexpr (K1) {
            const int r = row + (lane & 15), c = s * 4 + (lane >> 4);
            return *(const u32x4_t*)(lds + r * 128 + ((c ^ ((r >> 1) & 7)) << 4));
        } else if constexpr (ESIZE == 2) {
            // lane i of a group of 16 reads 8 bytes of row k = i / 4 and is
            // given column i of rows k..k+3
            union {
                i16x4 h[2];
                u32x4_t v;
            } u;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = s * 32 + (lane >> 4) * 8 + h * 4 + ((lane >> 2) & 3);
                const int c = (row >> 4) ^ swizzle(k);
                const char* p = lds + k * ROWS * 2 + c * 32 + (lane & 3) * 8;
                u.h[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4)(lds_ptr)p);
            }
            return u.v;
        } else {
            u32x4_t v;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int k = s * 16 + (lane >> 4) * 4 + e;
                const int col = row + (lane & 15);
                const int c = (col >> 3) ^ swizzle(k);
                v[e] = *(const uint32_t*)(lds + k * ROWS * 4 + c * 32 + (col & 7) * 4);
            }
            return v;
        }
    }
};

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

// Block -> tile: blocks are dealt to the 8 XCDs in turn, so each XCD is given
// a contiguous run of tiles, ordered in columns of 4 m tiles: the run's
// operands then share that XCD's L2.
__device__ __forceinline__ void tile_of_block(uint32_t block, uint32_t tiles_m, uint32_t tiles_n,
                                              uint32_t& tm, uint32_t& tn) {
    const uint32_t total = tiles_m * tiles_n, q = total / 8, r = total % 8, x = block % 8;
    const uint32_t id = (x < r ? x * (q + 1) : r * (q + 1) + (x - r) * q) + block / 8;
    constexpr uint32_t G = 4;
    const uint32_t group = id / (G * tiles_n), first = group * G;
    const uint32_t size = tiles_m - first < G ? tiles_m - first : G;
    const uint32_t in = id - group * G * tiles_n;
    tm = first + in % size;
    tn = in / size;
}

}  // namespace vpa
