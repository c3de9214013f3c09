// row_scan.h -- one pass over a segment of a row of logits for a sum of
// exponentials (and, where asked for, the first column in the argmax order), as
// sampled.hip and distill.hip need it.
//
// A workgroup walks its segment in chunks of U 16-byte vectors a thread, held in
// registers, that begin at aligned columns.  Every lane keeps s = sum 2^z of its
// own columns, z = (x - M) scale, from an M that its wavefront shares: the first
// chunk's maximum, moved to a later chunk's where that is more than kLag (of z)
// above it.  A later chunk is one pass: for bf16 an element costs 1.5
// instructions to unpack it and take the maximum, a multiply-add, 2 slots for
// 2^z and an add.
//
// A vector's terms and a chunk's vectors, 20 at most, are added in fp32, chunks in 64
// bits: equal terms are rounded in the same direction in every lane, so in fp32
// alone a row's error would grow with its length (2^21 equal logits in one segment
// 1e-5 off, 2^24 1e-4).
#pragma once

#include "vpa_math.h"

namespace vpa {
namespace {

constexpr float kMinusInf = -__builtin_inff();
// most (of z) that a chunk's maximum may exceed M by: an exponent further off is
// rounded to fewer digits, and ln s is a large number of which a loss needs the last
constexpr float kLag = 6.0f;

// The largest of three (a NaN among them: any of them or NaN), one instruction.
__device__ __forceinline__ float largest3(float a, float b, float c) {
    float d;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "v"(c));
    return d;
}

template <int ESIZE>
__device__ __forceinline__ float vec_largest(u32x4_t w) {
    constexpr int VEC = 16 / ESIZE;
    float v = largest3(vec_elem<ESIZE>(w, 0), vec_elem<ESIZE>(w, 1), vec_elem<ESIZE>(w, 2));
#pragma unroll
    for (int e = 3; e + 1 < VEC; e += 2)
        v = largest3(v, vec_elem<ESIZE>(w, e), vec_elem<ESIZE>(w, e + 1));
    return largest3(v, vec_elem<ESIZE>(w, VEC - 1), vec_elem<ESIZE>(w, VEC - 1));
}

template <int ESIZE>
__device__ __forceinline__ u32x4_t vec_minus_inf() {
    constexpr uint32_t w = ESIZE == 2 ? 0xFF80FF80u : 0xFF800000u;
    return u32x4_t{w, w, w, w};
}

// 16 bytes as one number, and back.
struct Bits128 {
    uint64_t lo, hi;
    __device__ __forceinline__ explicit Bits128(u32x4_t v)
        : lo(v[0] | (uint64_t)v[1] << 32), hi(v[2] | (uint64_t)v[3] << 32) {}
    __device__ __forceinline__ Bits128(uint64_t l, uint64_t h) : lo(l), hi(h) {}
    __device__ __forceinline__ u32x4_t vec() const {
        return u32x4_t{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
    }
    // by n bits, 0 <= n <= 128
    __device__ __forceinline__ Bits128 right(int n) const {
        const int in = n & 63;
        const uint64_t both = lo >> in | (hi << 1) << (63 - in);
        return {n < 64 ? both : n < 128 ? hi >> in : 0, n < 64 ? hi >> in : 0};
    }
    __device__ __forceinline__ Bits128 left(int n) const {
        const int in = n & 63;
        const uint64_t both = hi << in | (lo >> 1) >> (63 - in);
        return {n < 64 ? lo << in : 0, n < 64 ? both : n < 128 ? lo << in : 0};
    }
};

// Columns c .. c+VEC-1 of a row, those outside [lo, hi) as -inf.  A vector that
// reaches past an end is the one that stops there, moved: with a load for each
// element a row's registers would be as many again.
template <int ESIZE, typename T>
__device__ __forceinline__ u32x4_t load_columns(const T* x, int c, int lo, int hi) {
    constexpr int VEC = 16 / ESIZE;
    if (c >= lo && c + VEC <= hi)
        return __builtin_nontemporal_load((const u32x4_t*)(x + c));
    if (c + VEC <= lo || c >= hi)
        return vec_minus_inf<ESIZE>();
    Bits128 v(0, 0), in(0, 0);                     // values, and where they are
    if (hi - lo >= VEC) {
        const int at = c < lo ? lo : hi - VEC;
        v = Bits128(((const Loose16*)(x + at))->v);
        const int n = (c < at ? at - c : c - at) * ESIZE * 8;
        const Bits128 all(~0ull, ~0ull);
        v = c < at ? v.left(n) : v.right(n);
        in = c < at ? all.left(n) : all.right(n);
        // (both ends in one vector: hi - lo >= VEC leaves one of them to each)
    } else {
#pragma unroll 1
        for (int e = lo > c ? lo - c : 0; e < VEC && c + e < hi; ++e) {
            uint64_t one;
            if constexpr (ESIZE == 2)
                one = x[c + e];
            else
                one = __builtin_bit_cast(uint32_t, x[c + e]);
            const Bits128 put = Bits128(one, 0).left(e * ESIZE * 8);
            const Bits128 all = Bits128(ESIZE == 2 ? 0xFFFFull : 0xFFFFFFFFull, 0).left(e * ESIZE * 8);
            v = Bits128(v.lo | put.lo, v.hi | put.hi);
            in = Bits128(in.lo | all.lo, in.hi | all.hi);
        }
    }
    const Bits128 none(vec_minus_inf<ESIZE>());
    return Bits128(v.lo | (none.lo & ~in.lo), v.hi | (none.hi & ~in.hi)).vec();
}

// Stores those of columns c .. c+VEC-1 that lie in [lo, hi), past the L2.
template <int ESIZE, typename T>
__device__ __forceinline__ void store_columns(T* d, int c, int lo, int hi, u32x4_t o) {
    constexpr int VEC = 16 / ESIZE;
    if (c >= lo && c + VEC <= hi) {
        __builtin_nontemporal_store(o, &((Loose16*)(d + c))->v);
        return;
    }
    const Bits128 v(o);
#pragma unroll 1
    for (int e = lo > c ? lo - c : 0; e < VEC && c + e < hi; ++e) {
        const uint64_t one = v.right(e * ESIZE * 8).lo;
        if constexpr (ESIZE == 2)
            d[c + e] = (uint16_t)one;
        else
            d[c + e] = __builtin_bit_cast(float, (uint32_t)one);
    }
}

// Makes element e (the same in all lanes) of lane `at`'s vector -inf.
template <int ESIZE>
__device__ __forceinline__ void mask_element(u32x4_t& w, int e, int at) {
    const Bits128 one = Bits128(ESIZE == 2 ? 0xFFFFull : 0xFFFFFFFFull, 0).left(e * ESIZE * 8);
    const u32x4_t m = one.vec(), none = vec_minus_inf<ESIZE>();
    const bool mine = (int)(threadIdx.x & 63) == at;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const uint32_t in = mine ? m[d] : 0;
        w[d] = (w[d] & ~in) | (none[d] & in);
    }
}

// z = (x - M) scale as one multiply-add, x scale - b with b = M scale rounded:
// what the rounding took off, 2^-24 of b at most, is put right on the sum.  From
// 2^20 on, where that would leave a power's range before long (a low temperature,
// logits of 1e6), `apart` says that the difference comes first.
struct ScaledFrom {
    float m, b, fix;
    bool apart;
    __device__ __forceinline__ void set(float m_, float scale) {
        m = m_;
        b = m * scale;
        apart = !(fabsf(b) < 0x1p20f);
        fix = apart ? 1.0f : exp2_fast(-__builtin_fmaf(m, scale, -b));
    }
};

// Sum of 2^z over a chunk in registers.  `base` holds a finite M.
template <int ESIZE, int U>
__device__ __forceinline__ float chunk_sum(const u32x4_t (&w)[U], const ScaledFrom& base,
                                           float scale) {
    constexpr int VEC = 16 / ESIZE;
    float sum = 0.0f;
    // (one branch around both loops would have all of the values unpacked before it)
#pragma unroll
    for (int i = 0; i < U; ++i) {
        float s = 0.0f;
        if (base.apart) {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                s += exp2_fast((vec_elem<ESIZE>(w[i], e) - base.m) * scale);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                s += exp2_fast(__builtin_fmaf(vec_elem<ESIZE>(w[i], e), scale, -base.b));
        }
        sum += s;
        asm volatile("" : "+v"(sum));           // not all vectors' sums first
        __builtin_amdgcn_sched_barrier(0);         // registers for one vector at a time
    }
    return sum * base.fix;
}

// (m, s) of a set of columns: m near its largest, s = sum 2^((x - m) scale); the
// empty set is (-inf, 0).  A NaN or +inf among the columns makes s NaN.
struct ExpSum {
    float m, s;
};
__device__ __forceinline__ ExpSum join(ExpSum a, ExpSum b, float scale) {
    const float m = fmaxf(a.m, b.m);
    if (m == kMinusInf)
        return {m, a.s + b.s};
    return {m, a.s * exp2_fast((a.m - m) * scale) + b.s * exp2_fast((b.m - m) * scale)};
}
// Over the lanes of a wavefront, each with its own m.
__device__ __forceinline__ ExpSum wave_join(ExpSum v, float scale) {
    const float m = wave_max(v.m);
    return {m, wave_sum(m == kMinusInf ? v.s : v.s * exp2_fast((v.m - m) * scale))};
}

// The scan of columns [lo, hi) of the row x, whose chunks of a workgroup of
// THREADS begin at column `begin` (aligned, at most VEC - 1 below lo).
template <int ESIZE, int U, int THREADS, bool BEST>
struct SegmentScan {
    using T = typename elem<ESIZE>::type;
    static constexpr int VEC = 16 / ESIZE;
    static constexpr int CHUNK = THREADS * U * VEC;

    ScaledFrom base = {kMinusInf, 0.0f, 1.0f, false};
    double s = 0.0;                                // the lane's
    float best = kMinusInf;                        // the lane's largest value
    int best_at = -1;                              // and its vector's first column

    // `masked` is called with a chunk and its first column before it is summed.
    template <typename Mask>
    __device__ __forceinline__ void run(const T* x, int begin, int lo, int hi, float scale,
                                        Mask masked) {
        for (int c0 = begin; c0 < hi; c0 += CHUNK) {
            u32x4_t w[U];
            const int mine = c0 + (int)threadIdx.x * VEC;
            if (c0 >= lo && c0 + CHUNK <= hi) {
#pragma unroll
                for (int i = 0; i < U; ++i)
                    w[i] = __builtin_nontemporal_load((const u32x4_t*)(x + mine + i * THREADS * VEC));
            } else {
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    w[i] = load_columns<ESIZE>(x, mine + i * THREADS * VEC, lo, hi);
                    asm volatile("" : "+v"(w[i]));
                    __builtin_amdgcn_sched_barrier(0);     // registers for one at a time
                }
            }
            masked(w, c0);
            float mx = kMinusInf;
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const float g = vec_largest<ESIZE>(w[i]);
                if constexpr (BEST) {
                    if (g > best) {
                        best = g;
                        best_at = mine + i * THREADS * VEC;
                    }
                }
                mx = fmaxf(mx, g);
            }
            // values are unpacked anew in every use: held as fp32 they would
            // cost half the wavefronts
#pragma unroll
            for (int i = 0; i < U; ++i)
                asm volatile("" : "+v"(w[i]));
            if (base.m == kMinusInf || __ballot((mx - base.m) * scale > kLag)) {
                const float m = fmaxf(base.m, wave_max(mx));
                if (m == kMinusInf) {              // nothing but masked columns, or NaN
                    ScaledFrom zero;
                    zero.set(0.0f, scale);
                    s += (double)chunk_sum<ESIZE, U>(w, zero, scale);
                    continue;
                }
                if (base.m != kMinusInf)
                    s *= (double)exp2_fast((base.m - m) * scale);
                base.set(m, scale);
            }
            s += (double)chunk_sum<ESIZE, U>(w, base, scale);
        }
    }
    // of the wavefront's columns
    __device__ __forceinline__ ExpSum wave() const {
        return {base.m, (float)wave_sum_f64(s)};
    }
    // The first of the wavefront's columns in the argmax order as one number (0:
    // no columns).  A wavefront with a NaN or +inf goes through its columns again.
    __device__ __forceinline__ uint64_t wave_best(const T* x, int begin, int lo, int hi) const {
        uint64_t order = 0;
        if (__ballot(!(s < __builtin_inff()))) {
            for (int c0 = begin; c0 < hi; c0 += THREADS * VEC)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const int c = c0 + (int)threadIdx.x * VEC + e;
                    if (c >= lo && c < hi) {
                        const uint64_t o = order_of(to_f32(x[c]), c);
                        order = o > order ? o : order;
                    }
                }
            return wave_max_u64(order);
        }
        const float top = wave_max(best);
        if (top == kMinusInf) {                    // masked: the lowest column
            const int c = begin + (int)threadIdx.x * VEC;
            const int first = c > lo ? c : lo;
            if (c + VEC > lo && first < hi)
                order = order_of(kMinusInf, first);
        } else if (best == top) {
#pragma unroll
            for (int e = VEC - 1; e >= 0; --e) {
                const int c = best_at + e;
                if (c >= lo && c < hi && to_f32(x[c]) == top)
                    order = order_of(top, c);
            }
        }
        return wave_max_u64(order);
    }
};

}  // namespace
}  // namespace vpa
