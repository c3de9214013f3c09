// logprob.hip -- log probabilities of given tokens with entropy and the top
// alternatives, over one or several vocabulary shards, and their gradient.
//
// A set of columns is described by a logit M near its maximum and by s = sum
// 2^z and u = sum z 2^z with z = (x - M) log2(e); two sets join as
//   M = max(Ma, Mb),  s = sum_i s_i 2^di,  u = sum_i (u_i + di s_i) 2^di,
//   di = (Mi - M) log2(e),
// so a row is one pass over its columns, cut into chunks that workgroups
// reduce independently.  At the end the log probability of a logit x is
// (x - M) - ln s, which keeps its digits where lse = M + ln s is large (a
// row of the type's lowest value still has -log V), and the entropy is
// (log2 s - u/s) ln 2.
//
// Top alternatives carry the argmax order as one 64-bit number, the value's
// key (vpa_device.h) above the inverted column id: every comparison is one
// unsigned compare, and no two columns are equal.
//
// Large batches are bound by reading the logits once, small ones by the
// latency of a chunk and of two launches.  Measured, kernels alone in a trace:
// 1024 x 200064 bf16 with 8 alternatives 78 us, 5.2 TB/s; 2048 x 50257 bf16
// 44 us (4.9; rows that are not aligned); 512 x 50257 fp32 21 + 4 us; 32 x
// 151936 bf16 with 20 alternatives 11.0 + 5.4 us; one row 6.9 + 3.6 us.
// Calls: records of one of 8 shards of 1024 x 200064 26 us, their combination
// 7 us; of 32 rows with 20 alternatives 13.8 and 7.2 us.
#include "vpa_device.h"
#include "vpa_head_internal.h"
#include "vpa_math.h"

namespace vpa {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kCandidates = 2048;                 // LDS list of a workgroup's candidates
constexpr int kMostSegments = 64;                 // of a part of a row

// Columns of a chunk: U 16-byte vectors a thread.
constexpr int chunk_cols(int esize, int u) {
    return kThreads * u * (16 / esize);
}

constexpr float kNegInf = -__builtin_inff();
constexpr float kLag = 4.0f;                      // most that a chunk's maximum may exceed M by

// M, s, u of a set of columns; the empty set is (-inf, 0, 0).
struct Sums {
    float m, s, u;
};
// (x - m) log2(e), held at -1000, where 2^z is 0 already: its products with
// 2^z and with the sum of a set that it moves (d s, before 2^d = 0 takes it
// away) are finite, whatever the logits; a NaN stays.
__device__ __forceinline__ float scaled_distance(float x, float m) {
    const float z = (x - m) * kLog2e;
    return z < -1000.0f ? -1000.0f : z;
}
__device__ __forceinline__ void join(Sums& a, const Sums& b) {
    const float m = fmaxf(a.m, b.m);
    const float da = a.m == m ? 0.0f : scaled_distance(a.m, m);
    const float db = b.m == m ? 0.0f : scaled_distance(b.m, m);
    const float fa = exp2_fast(da), fb = exp2_fast(db);
    a.u = (a.u + da * a.s) * fa + (b.u + db * b.s) * fb;
    a.s = a.s * fa + b.s * fb;
    a.m = m;
}
// One step of a join with the partner lane of a DPP move (vpa_device.h); rows
// outside ROW_MASK join the empty set.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ void join_step(Sums& v) {
    const auto move = [](float x, float none) {
        return __builtin_bit_cast(
            float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, none),
                                               __builtin_bit_cast(int, x), CTRL, ROW_MASK, 0xF,
                                               false));
    };
    join(v, Sums{move(v.m, kNegInf), move(v.s, 0.0f), move(v.u, 0.0f)});
}
__device__ __forceinline__ float lane63(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 63));
}
// Over the wavefront; every lane holds the result.
__device__ __forceinline__ Sums wave_join(Sums v) {
    join_step<dpp::kSwap1, 0xF>(v);
    join_step<dpp::kSwap2, 0xF>(v);
    join_step<dpp::kHalfMirror, 0xF>(v);
    join_step<dpp::kMirror, 0xF>(v);
    join_step<dpp::kBcast15, 0xA>(v);
    join_step<dpp::kBcast31, 0xC>(v);
    return Sums{lane63(v.m), lane63(v.s), lane63(v.u)};
}
// Over the workgroup, of sums that are the same in all lanes of a wavefront,
// through `lds`; every thread holds the result.
__device__ __forceinline__ Sums block_join(Sums v, Sums* lds) {
    if ((threadIdx.x & 63) == 0)
        lds[threadIdx.x >> 6] = v;
    __syncthreads();
    static_assert(kWaves == 4, "two steps of the first four lanes");
    v = lds[threadIdx.x & 3];
    join_step<dpp::kSwap1, 0xF>(v);
    join_step<dpp::kSwap2, 0xF>(v);
    return v;
}

// Partial results in the workspace: the Sums of every segment first, then the
// segments' top lists.
__host__ __device__ inline size_t sums_bytes(int64_t n) {
    return ((size_t)n * sizeof(Sums) + 255) / 256 * 256;
}

// A row's max and ln s from its joined sums; no finite column: (-inf, 0).
struct RowScale {
    float max, log_sum;
    bool empty;
    __device__ __forceinline__ float logprob(float x) const {
        return empty ? kNegInf : (x - max) - log_sum;
    }
};
__device__ __forceinline__ RowScale scale_of(const Sums& r) {
    const bool empty = r.m == kNegInf && r.s == 0.0f;
    return RowScale{r.m, empty ? 0.0f : log2f(r.s) * kLn2, empty};
}

// Writes the outputs of one row other than its alternatives; `logit(j, id)`
// is the logit of given token j.
template <typename Logit>
__device__ __forceinline__ void write_row(const Sums& r, const RowScale& sc, int64_t row,
                                          int32_t vocab, const LogprobOut& o, Logit logit) {
    if (threadIdx.x == 0) {
        if (o.lse)
            o.lse[row] = sc.max + sc.log_sum;
        o.row_stats[3 * row] = sc.max;
        o.row_stats[3 * row + 1] = sc.log_sum;
        o.row_stats[3 * row + 2] = sc.empty ? 0.0f : (log2f(r.s) - r.u / r.s) * kLn2;
    }
    for (int j = threadIdx.x; j < o.n_tokens; j += kThreads) {
        const int32_t id = o.token_ids[row * o.n_tokens + j];
        float lp = __builtin_nanf("");
        if (id == -1)
            lp = 0.0f;
        else if (id >= 0 && id < vocab)
            lp = sc.logprob(logit(j, id));
        o.logprobs[row * o.n_tokens + j] = lp;
    }
}

// n of a wavefront's 64 keys are at least the result, cut to its upper 16
// bits: the n-th largest key from below.
__device__ __forceinline__ uint32_t wave_nth_key(uint32_t key, int n) {
    uint32_t nth = 0;
#pragma unroll
    for (int b = 31; b >= 16; --b) {
        const uint32_t t = nth | (1u << b);
        nth = __popcll(__ballot(key >= t)) >= n ? t : nth;
    }
    return nth;
}

// The largest n_top of the n orders cand[] (0: none), by the whole workgroup,
// in order into out[]: each candidate's place is the number of larger ones.
// Places past n are left as they are.
__device__ __forceinline__ void rank_candidates(const uint64_t* cand, int n, int n_top,
                                                uint64_t* out) {
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const uint64_t mine = cand[i];
        int larger = 0;
#pragma unroll 8
        for (int j = 0; j < n; ++j)
            larger += cand[j] > mine;
        if (larger < n_top)
            out[larger] = mine;
    }
}

// The largest of three (a NaN among them: any of them or NaN): one
// instruction, where fmaxf would first quiet inputs that come from bit
// operations.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "v"(c));
    return d;
}

// z = (x - M) log2(e) as one multiply-add, x log2(e) - b with b = M log2(e)
// rounded: what the rounding took off is put right on a chunk's sums.
struct LaneScale {
    float b, off, fix;
    __device__ __forceinline__ void set(float m) {
        b = m * kLog2e;
        off = __builtin_fmaf(m, kLog2e, -b);
        fix = exp2_fast(-off);
    }
};

template <int ESIZE>
__device__ __forceinline__ u32x4_t all_neg_inf() {
    constexpr uint32_t w = ESIZE == 2 ? 0xFF80FF80u : 0xFF800000u;
    return u32x4_t{w, w, w, w};
}

// One segment of a row: its Sums and its first n_top columns.
//
// The workgroup walks the segment in chunks of U 16-byte vectors a thread,
// held in registers.  Every lane keeps s and u of its own columns, measured
// from an M that its wavefront shares and that follows the maximum: it is the
// first chunk's, and moves to a later chunk's that is more than kLag above it.
// s is then at least 1 and 2^z at most e^kLag, so that ln s and u / s lose no
// digits to a large z: the log probability of a token that the model is sure
// of is right to a few steps at kLag, and where nothing comes within kLag of
// it, its row's entropy to a few steps at 1 (with M up to 40 behind both were
// off by 4e-6).  A later chunk is one pass: for bf16 an element costs 1.5
// instructions to unpack it and take the maximum, 2 slots for 2^z, a
// multiply-add, an add and a multiply-add, 6.5 slots; where M moves it is two
// passes (1024 x 200064 with a sure token in half of the rows: 76.7 us, 81.4
// with a kLag of 1, 76.1 with one of 40).
//
// Alternatives: T is a lower bound of the n_top-th largest value, from the
// largest values of the lanes on the first chunk (in each of the W
// wavefronts with columns at least ceil(n_top / W) lanes reach T, so n_top
// columns do, unless the mask leaves fewer), then the n_top-th value found so
// far; columns reaching T go to a list in LDS, and the list is cut to its first
// n_top by counting for each the larger ones.  Few columns pass T, so the scan
// costs one maximum and one comparison a vector.  A chunk with a NaN, an
// infinity or more candidates than the list holds takes n_top maxima over the
// registers.
template <int ESIZE, int U>
__global__ __launch_bounds__(kThreads) void logprob_part_kernel(LogprobTask t, LogprobCut cut,
                                                                LogprobOut o, void* ws) {
    using T = typename elem<ESIZE>::type;
    constexpr int VEC = 16 / ESIZE;
    constexpr int N = U * VEC;
    constexpr int CHUNK = chunk_cols(ESIZE, U);
    __shared__ Sums lds_s[kWaves];
    __shared__ uint32_t lds_key[kWaves];
    __shared__ uint64_t lds_best[2][kWaves];
    __shared__ uint64_t cand[kCandidates];
    __shared__ uint64_t list[VPA_MAX_TOP];
    __shared__ uint32_t added[3];
    const int32_t seg = blockIdx.x % cut.segments;
    const int32_t rest = blockIdx.x / cut.segments;
    const int32_t row = rest % t.n_rows, part = rest / t.n_rows;
    const int64_t first = t.col0 + part * t.part_stride;
    const int64_t part_end = first + t.part_width < t.vocab ? first + t.part_width : t.vocab;
    const T* x = (const T*)t.logits + (int64_t)row * t.ld - t.col0;
    // chunks start at a 16-byte aligned column, up to VEC - 1 before the part
    const int back = (int)(((uintptr_t)(x + first) & 15) / ESIZE);
    const int64_t from = first - back + (int64_t)seg * cut.chunks_per_segment * CHUNK;
    const int64_t to = from + (int64_t)cut.chunks_per_segment * CHUNK;
    // columns stay below 2^24 (but a part may begin past the vocabulary)
    const int begin = (int)(from < part_end ? from : part_end);
    const int hi = (int)(to < part_end ? to : part_end);
    const int lo = begin < first ? (int)first : begin;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;

    Sums r = {kNegInf, 0.0f, 0.0f};                 // M is the wavefront's, s and u the lane's
    LaneScale scale = {0.0f, 0.0f, 1.0f};
    int kept = 0;                                   // of cand[]: the best so far, in order
    float bound = kNegInf;                          // T
    if (t.n_top && threadIdx.x < 3)
        added[threadIdx.x] = 0;
    int turn = 0;                                   // of added[]
    for (int c0 = begin; c0 < hi; c0 += CHUNK) {
        u32x4_t w[U];                               // columns mine + i * kThreads * VEC + e
        float g[U];                                 // a vector's maximum
        const int mine = c0 + threadIdx.x * VEC;
        auto column = [&](int i) { return mine + (i / VEC) * kThreads * VEC + i % VEC; };
        auto value = [&](int i) { return vec_elem<ESIZE>(w[i / VEC], i % VEC); };
        const bool whole = c0 >= lo && c0 + CHUNK <= hi;
        // whether vector i has columns of the segment
        auto has = [&](int i) { return column(i * VEC) + VEC > lo && column(i * VEC) < hi; };
        if (whole) {
#pragma unroll
            for (int i = 0; i < U; ++i)
                w[i] = __builtin_nontemporal_load((const u32x4_t*)(x + column(i * VEC)));
        } else {
            // the segment's ends: columns outside hold -inf
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int c = column(i * VEC);
                w[i] = all_neg_inf<ESIZE>();
                if (c >= lo && c + VEC <= hi) {
                    w[i] = *(const u32x4_t*)(x + c);
                } else if (has(i)) {
                    union {
                        T e[VEC];
                        u32x4_t v;
                    } part;
                    part.v = w[i];
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        if (c + e >= lo && c + e < hi)
                            part.e[e] = x[c + e];
                    w[i] = part.v;
                }
            }
        }
        // values are unpacked anew in every use: held as fp32, 64 of them
        // would cost half the wavefronts
        auto anew = [&] {
#pragma unroll
            for (int i = 0; i < U; ++i)
                asm volatile("" : "+v"(w[i]));
        };
        // the largest of vector i
        auto largest = [&](int i) {
            float v = max3(value(i * VEC), value(i * VEC + 1), value(i * VEC + 2));
#pragma unroll
            for (int e = 3; e + 1 < VEC; e += 2)
                v = max3(v, value(i * VEC + e), value(i * VEC + e + 1));
            return max3(v, value(i * VEC + VEC - 1), value(i * VEC + VEC - 1));
        };
        if (r.m == kNegInf) {
            float v = kNegInf;
#pragma unroll
            for (int i = 0; i < U; ++i)
                v = fmaxf(v, largest(i));
            scale.set(r.m = wave_max(v));
            anew();
        }
        float s = 0.0f, u = 0.0f, mx = kNegInf;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            g[i] = largest(i);
            mx = fmaxf(mx, g[i]);
            if (whole || has(i)) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float z = __builtin_fmaf(value(i * VEC + e), kLog2e, -scale.b);
                    const float p = exp2_fast(z);
                    s += p;
                    u = __builtin_fmaf(z, p, u);
                }
            }
            __builtin_amdgcn_sched_barrier(0);      // registers for one vector at a time
        }
        u = __builtin_fmaf(-scale.off, s, u) * scale.fix;
        s *= scale.fix;
        // masked columns (0 * -inf), infinities and NaN, values whose product
        // with log2(e) is not finite, a maximum that M has to follow: once
        // more, with care, from the larger of M and the chunk's maximum
        const bool odd = !(fabsf(u) < __builtin_inff()) || mx > r.m + kLag;
        if (__ballot(odd)) {
            anew();
            const float m = fmaxf(r.m, wave_max(mx));
            if (m != r.m) {
                const float d = scaled_distance(r.m, m);
                const float f = exp2_fast(d);
                r.u = (r.u + d * r.s) * f;
                r.s *= f;
                scale.set(r.m = m);
            }
            const float base = m == kNegInf ? 0.0f : m;
            s = u = 0.0f;
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (whole || has(i)) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float z = scaled_distance(value(i * VEC + e), base);
                        const float p = exp2_fast(z);
                        s += p;
                        u = __builtin_fmaf(z, p, u);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        r.s += s;
        r.u += u;
        if (t.n_top == 0)
            continue;

        {
            if (c0 == begin) {
                const int lanes = (hi - begin + VEC - 1) / VEC;    // with columns
                const int waves = lanes >= kThreads ? kWaves : (lanes + 63) / 64;
                const uint32_t nth = wave_nth_key(key_f32(__builtin_bit_cast(uint32_t, mx)),
                                                  (t.n_top + waves - 1) / waves);
                if (lane == 0)
                    lds_key[wave] = nth;
                __syncthreads();
                uint32_t least = lds_key[0];
                for (int i = 1; i < waves; ++i)
                    least = lds_key[i] < least ? lds_key[i] : least;
                bound = value_of_key(least ? least : 1);        // -inf is below it
            }
            // The first chunk lists its first n_top columns whatever their
            // values: where the mask leaves fewer than n_top, the rest are
            // -inf by the lowest ids.
            const int head = c0 == begin ? lo + t.n_top : lo;
            // NaN and +inf make the lane's s NaN: such a chunk is not listed
            if (s != s)
                atomicAdd(&added[turn], (uint32_t)kCandidates);
            else if (__ballot(mx >= bound || mine < head)) {
                anew();
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    if (!__ballot(g[i] >= bound || column(i * VEC) < head))
                        continue;
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const int c = column(i * VEC + e);
                        if ((value(i * VEC + e) >= bound || c < head) && c >= lo && c < hi) {
                            const uint32_t at = kept + atomicAdd(&added[turn], 1u);
                            if (at < kCandidates)
                                cand[at] = order_of(value(i * VEC + e), c);
                        }
                    }
                }
            }
            __syncthreads();
        }
        int total = kept + (int)added[turn];
        const bool slow = total >= kCandidates;
        // the counter after next was last read before the barrier above
        if (threadIdx.x == 0)
            added[turn == 0 ? 2 : turn - 1] = 0;
        turn = turn == 2 ? 0 : turn + 1;
        if (!slow && total == kept)
            continue;
        if (!slow) {
            rank_candidates(cand, total, t.n_top, list);
        } else {
            // the best of the kept ones and of every column, n_top times
            uint64_t below = ~0ull;
            total = 0;
            for (int k = 0; k < t.n_top; ++k) {
                uint64_t best = 0;
                if ((int)threadIdx.x < kept && cand[threadIdx.x] < below)
                    best = cand[threadIdx.x];
                anew();                             // nor keep their orders around the loop
                int at = mine;
                asm volatile("" : "+v"(at));
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int c = at + column(i) - mine;
                    const uint64_t o = order_of(value(i), c);
                    if (c >= lo && c < hi && o < below && o > best)
                        best = o;
                    if (i % VEC == VEC - 1)
                        __builtin_amdgcn_sched_barrier(0);
                }
                best = wave_max_u64(best);
                if (lane == 0)
                    lds_best[k & 1][wave] = best;
                __syncthreads();
                for (int i = 0; i < kWaves; ++i)
                    best = lds_best[k & 1][i] > best ? lds_best[k & 1][i] : best;
                if (threadIdx.x == 0)
                    list[k] = best;
                total += best != 0;
                below = best;
            }
        }
        __syncthreads();
        kept = total < t.n_top ? total : t.n_top;
        if ((int)threadIdx.x < kept)
            cand[threadIdx.x] = list[threadIdx.x];
        // later columns have larger ids: they have to be above the last value
        if (kept == t.n_top) {
            const uint32_t key = (uint32_t)(list[kept - 1] >> 32);
            bound = key >= kKeyNanF32 ? __builtin_nanf("") : value_of_key(key + 1);
        }
    }
    r.s = wave_sum(r.s);
    r.u = wave_sum(r.u);
    r = block_join(r, lds_s);
    const uint64_t top = (int)threadIdx.x < kept ? cand[threadIdx.x] : 0;
    if (o.row_stats) {                              // the segment is the row
        const RowScale sc = scale_of(r);
        write_row(r, sc, row, t.vocab, o, [&](int, int32_t id) { return to_f32(x[id]); });
        if ((int)threadIdx.x < t.n_top) {
            o.top_ids[(int64_t)row * t.n_top + threadIdx.x] = id_of(top);
            o.top_logprobs[(int64_t)row * t.n_top + threadIdx.x] = sc.logprob(value_of(top));
        }
        return;
    }
    if (threadIdx.x == 0)
        ((Sums*)ws)[blockIdx.x] = r;
    uint64_t* tops = (uint64_t*)((char*)ws + sums_bytes(cut.total)) + (int64_t)blockIdx.x * t.n_top;
    if ((int)threadIdx.x < t.n_top)
        tops[threadIdx.x] = top;
}

// The n_top largest of n orders (0: none), by the whole workgroup: take(k,
// order) is called for the k-th by one thread.  Lists of n_top orders begin at
// multiples of n_top, largest first.  With j = ceil(n_top / lists), the
// ceil(n_top / j)-th largest of the lists' j-th orders is reached by n_top
// orders; the orders whose keys reach its key go to LDS to be ranked.  Where
// they do not fit, the largest is taken n_top times.
template <typename Order, typename Take>
__device__ __forceinline__ void select_top(int64_t lists, int32_t n_top, uint64_t* cand,
                                           uint64_t* list, Order order, Take take) {
    __shared__ uint64_t best_of[2][kWaves];
    __shared__ uint32_t count;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t n = lists * n_top;
    const int some = lists < 64 ? (int)lists : 64;  // lists, one a lane
    const int j = (n_top + some - 1) / some;
    const uint64_t jth = lane < some ? order((int64_t)lane * n_top + j - 1) : 0;
    const uint32_t key = wave_nth_key((uint32_t)(jth >> 32), (n_top + j - 1) / j);
    // (empty places are not candidates)
    const uint64_t least = key ? (uint64_t)key << 32 : 1;
    if (threadIdx.x == 0)
        count = 0;
    __syncthreads();
    for (int64_t i = threadIdx.x; i < n; i += kThreads) {
        const uint64_t o = order(i);
        if (o >= least) {
            const uint32_t at = atomicAdd(&count, 1u);
            if (at < kCandidates)
                cand[at] = o;
        }
    }
    if ((int)threadIdx.x < n_top)
        list[threadIdx.x] = 0;
    __syncthreads();
    if (count <= kCandidates) {
        rank_candidates(cand, (int)count, n_top, list);
        __syncthreads();
        if ((int)threadIdx.x < n_top)
            take((int)threadIdx.x, list[threadIdx.x]);
        return;
    }
    uint64_t below = ~0ull;
    for (int k = 0; k < n_top; ++k) {
        uint64_t best = 0;
        for (int64_t i = threadIdx.x; i < n; i += kThreads) {
            const uint64_t o = order(i);
            if (o < below && o > best)
                best = o;
        }
        best = wave_max_u64(best);
        if (lane == 0)
            best_of[k & 1][wave] = best;
        __syncthreads();
        for (int i = 0; i < kWaves; ++i)
            best = best_of[k & 1][i] > best ? best_of[k & 1][i] : best;
        if (threadIdx.x == 0)
            take(k, best);
        below = best;
    }
}

// Joins sums(0) ... sums(n - 1); every thread holds the result.
template <typename Get>
__device__ __forceinline__ Sums join_all(int64_t n, Get sums) {
    __shared__ Sums lds[kWaves];
    Sums r = {kNegInf, 0.0f, 0.0f};
    for (int64_t i = threadIdx.x; i < n; i += kThreads)
        join(r, sums(i));
    return block_join(wave_join(r), lds);
}

template <int ESIZE>
__global__ __launch_bounds__(kThreads) void logprob_finish_kernel(LogprobTask t, LogprobCut cut,
                                                                  const void* ws, LogprobOut o) {
    using T = typename elem<ESIZE>::type;
    __shared__ uint64_t cand[kCandidates], list[VPA_MAX_TOP];
    const int64_t row = blockIdx.x;
    const Sums* sums = (const Sums*)ws + row * cut.segments;
    const Sums r = join_all(cut.segments, [&](int64_t i) { return sums[i]; });
    const T* x = (const T*)t.logits + row * t.ld - t.col0;
    const RowScale sc = scale_of(r);
    write_row(r, sc, row, t.vocab, o, [&](int, int32_t id) { return to_f32(x[id]); });
    if (t.n_top == 0)
        return;
    const uint64_t* tops = (const uint64_t*)((const char*)ws + sums_bytes(cut.total)) +
                           row * cut.segments * t.n_top;
    select_top(cut.segments, t.n_top, cand, list, [&](int64_t i) { return tops[i]; },
               [&](int k, uint64_t best) {
                   o.top_ids[row * t.n_top + k] = id_of(best);
                   o.top_logprobs[row * t.n_top + k] = sc.logprob(value_of(best));
               });
}

template <int ESIZE>
__global__ __launch_bounds__(kThreads) void logprob_record_kernel(LogprobTask t, LogprobCut cut,
                                                                  const void* ws,
                                                                  const int32_t* token_ids,
                                                                  int32_t n_tokens,
                                                                  int32_t* stats) {
    using T = typename elem<ESIZE>::type;
    __shared__ uint64_t cand[kCandidates], list[VPA_MAX_TOP];
    const int64_t slot = blockIdx.x;
    const int64_t row = slot % t.n_rows, part = slot / t.n_rows;
    int32_t* rec = stats + slot * (3 + n_tokens + 2 * t.n_top);
    const Sums* sums = (const Sums*)ws + slot * cut.segments;
    const Sums r = join_all(cut.segments, [&](int64_t i) { return sums[i]; });
    if (threadIdx.x == 0) {
        rec[0] = __builtin_bit_cast(int32_t, r.m);
        rec[1] = __builtin_bit_cast(int32_t, r.s);
        rec[2] = __builtin_bit_cast(int32_t, r.u);
    }
    const int64_t first = t.col0 + part * t.part_stride;
    const int64_t end = first + t.part_width < t.vocab ? first + t.part_width : t.vocab;
    const T* x = (const T*)t.logits + row * t.ld - t.col0;
    for (int j = threadIdx.x; j < n_tokens; j += kThreads) {
        const int32_t id = token_ids[row * n_tokens + j];
        const float v = id >= first && id < end ? to_f32(x[id]) : 0.0f;
        rec[3 + j] = __builtin_bit_cast(int32_t, v);
    }
    if (t.n_top == 0)
        return;
    const uint64_t* tops = (const uint64_t*)((const char*)ws + sums_bytes(cut.total)) +
                           slot * cut.segments * t.n_top;
    select_top(cut.segments, t.n_top, cand, list, [&](int64_t i) { return tops[i]; },
               [&](int k, uint64_t best) {
                   int32_t* p = rec + 3 + n_tokens + 2 * k;
                   p[0] = best ? __builtin_bit_cast(int32_t, value_of(best))
                               : (int32_t)VPA_EMPTY_BITS;
                   p[1] = best ? id_of(best) : VPA_EMPTY_ID;
               });
}

__global__ __launch_bounds__(kThreads) void logprob_combine_kernel(const int32_t* stats,
                                                                   int32_t n_shards,
                                                                   int64_t shard_width,
                                                                   int32_t vocab, int32_t n_rows,
                                                                   int32_t n_top, LogprobOut o) {
    __shared__ uint64_t cand[kCandidates], list[VPA_MAX_TOP];
    const int64_t row = blockIdx.x;
    const int64_t words = 3 + o.n_tokens + 2 * (int64_t)n_top;
    const int32_t* rec = stats + row * words;
    const int64_t step = n_rows * words;           // from shard to shard
    const Sums r = join_all(n_shards, [&](int64_t s) {
        const int32_t* p = rec + s * step;
        return Sums{__builtin_bit_cast(float, p[0]), __builtin_bit_cast(float, p[1]),
                    __builtin_bit_cast(float, p[2])};
    });
    const RowScale sc = scale_of(r);
    write_row(r, sc, row, vocab, o, [&](int j, int32_t id) {
        return __builtin_bit_cast(float, rec[(id / shard_width) * step + 3 + j]);
    });
    if (n_top == 0)
        return;
    const int32_t* top0 = rec + 3 + o.n_tokens;
    select_top(n_shards, n_top, cand, list,
               [&](int64_t i) {
                   const int32_t* p = top0 + (i / n_top) * step + 2 * (i % n_top);
                   return p[1] == VPA_EMPTY_ID
                              ? 0ull
                              : order_of(__builtin_bit_cast(float, p[0]), p[1]);
               },
               [&](int k, uint64_t best) {
                   o.top_ids[row * n_top + k] = id_of(best);
                   o.top_logprobs[row * n_top + k] = sc.logprob(value_of(best));
               });
}

constexpr int kGradVecs = 4;                       // 16-byte vectors a thread

// grad_c = sum_j g_j [c = t_j] - p_c (G + gH (log p_c + H)), G = sum_j g_j.
// A workgroup writes one chunk of a row without the given tokens' own terms,
// then the few elements that have them, from logits read before the chunk
// was written (the gradient may replace the logits).  Equal tokens all write
// the same sum.  Bound by memory: 2048 x 50257 bf16 74 us in a trace, 5.7 TB/s
// of reads and writes; 77 us a call with other logits each time, 64 with the
// same ones, which the Infinity Cache then holds in part.
template <int ESIZE, bool ENTROPY>
__global__ __launch_bounds__(kThreads) void logprob_grad_kernel(LogprobGradTask t,
                                                                int32_t chunks) {
    using T = typename elem<ESIZE>::type;
    constexpr int VEC = 16 / ESIZE;
    constexpr int CHUNK = chunk_cols(ESIZE, kGradVecs);
    const int64_t row = blockIdx.x / chunks;
    const int64_t lo = (int64_t)(blockIdx.x % chunks) * CHUNK;
    const int64_t hi = lo + CHUNK < t.grad_cols ? lo + CHUNK : t.grad_cols;
    const T* x = (const T*)t.logits + row * t.ld;
    T* d = (T*)t.grad + row * t.grad_ld;
    const float max = t.row_stats[3 * row], log_sum = t.row_stats[3 * row + 1];
    const float h = t.row_stats[3 * row + 2];
    const bool empty = max == kNegInf && log_sum == 0.0f;
    const float gh = ENTROPY ? t.grad_entropy[row] : 0.0f;
    const int32_t* tok = t.token_ids + row * t.n_tokens;
    const float* g = t.grad_logprobs + row * t.n_tokens;
    float sum = 0.0f;
    for (int j = 0; j < t.n_tokens; ++j)
        sum += tok[j] >= 0 && tok[j] < t.vocab ? g[j] : 0.0f;
    // -p (G + gH (log p + H))
    auto slope = [&](float v) {
        const float lp = (v - max) - log_sum;
        const float p = exp2f(lp * kLog2e);        // keeps p below 2^-126
        const float w = ENTROPY ? __builtin_fmaf(gh, lp + h, sum) : sum;
        return empty || p == 0.0f ? 0.0f : -p * w;
    };
    // this workgroup's given token, one a thread
    const int32_t mine = threadIdx.x < (uint32_t)t.n_tokens ? tok[threadIdx.x] : -1;
    const int64_t at = (int64_t)mine - t.col0;
    const bool here = mine >= 0 && mine < t.vocab && at >= lo && at < hi && at < t.cols;
    const float own = here ? to_f32(x[at]) : 0.0f;
    __syncthreads();
    u32x4_t w[kGradVecs];
#pragma unroll
    for (int i = 0; i < kGradVecs; ++i) {
        const int64_t c = lo + (i * kThreads + threadIdx.x) * VEC;
        if (c + VEC <= t.cols)
            w[i] = ((const Loose16*)(x + c))->v;
    }
#pragma unroll
    for (int i = 0; i < kGradVecs; ++i) {
        const int64_t c = lo + (i * kThreads + threadIdx.x) * VEC;
        if (c + VEC <= t.cols) {
            u32x4_t o;
            if constexpr (ESIZE == 2) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[e] = pack_bf16(slope(vec_elem<2>(w[i], 2 * e)),
                                     slope(vec_elem<2>(w[i], 2 * e + 1)));
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[e] = __builtin_bit_cast(uint32_t, slope(vec_elem<4>(w[i], e)));
            }
            __builtin_nontemporal_store(o, &((Loose16*)(d + c))->v);   // past the L2: 83 -> 66 us (same logits)
        } else {
            for (int e = 0; e < VEC; ++e)
                if (c + e < hi)
                    from_f32(d[c + e], c + e < t.cols ? slope(to_f32(x[c + e])) : 0.0f);
        }
    }
    __syncthreads();
    if (here) {
        float hot = 0.0f;
        for (int j = 0; j < t.n_tokens; ++j)
            hot += tok[j] == mine ? g[j] : 0.0f;
        from_f32(d[at], empty ? 0.0f : hot + slope(own));
    }
}

}  // namespace

// Chunks of 8 vectors a thread where that still gives every CU 4 workgroups
// and fills at least half of them, else of 2 (a decode batch, a small
// vocabulary); a part is cut into segments of whole chunks until there are 4
// workgroups a CU, or 8 of the smaller ones.
LogprobCut logprob_cut(int esize, int64_t part_width, int64_t n_parts, int64_t n_rows) {
    LogprobCut c;
    const int64_t rows = n_parts * n_rows;
    const int64_t width = part_width + 16 / esize - 1;       // with the columns before it
    const int64_t big = chunk_cols(esize, 8);
    c.vecs = 2 * width > big && rows * ((width + big - 1) / big) >= 1024 ? 8 : 2;
    const int64_t chunks = (width + chunk_cols(esize, c.vecs) - 1) / chunk_cols(esize, c.vecs);
    const int64_t groups = c.vecs == 8 ? 1024 : 2048;
    int64_t want = (groups + rows - 1) / rows;
    want = want > chunks ? chunks : want;
    want = want > kMostSegments ? kMostSegments : want;
    c.chunks_per_segment = (int32_t)((chunks + want - 1) / want);
    c.segments = (int32_t)((chunks + c.chunks_per_segment - 1) / c.chunks_per_segment);
    c.total = rows * c.segments;
    return c;
}

size_t logprob_workspace(const LogprobCut& c, int32_t n_top) {
    return sums_bytes(c.total) + ((size_t)c.total * n_top * 8 + 255) / 256 * 256;
}

int64_t logprob_threads(const LogprobCut& c) {
    return c.total * kThreads;
}

namespace {

hipError_t launch_parts(int esize, const LogprobTask& t, const LogprobCut& c, const LogprobOut& o,
                        void* ws, hipStream_t stream) {
    const dim3 grid((uint32_t)c.total), block(kThreads);
    if (esize == 2)
        return c.vecs == 8 ? launch(logprob_part_kernel<2, 8>, grid, block, 0, stream, t, c, o, ws)
                           : launch(logprob_part_kernel<2, 2>, grid, block, 0, stream, t, c, o, ws);
    return c.vecs == 8 ? launch(logprob_part_kernel<4, 8>, grid, block, 0, stream, t, c, o, ws)
                       : launch(logprob_part_kernel<4, 2>, grid, block, 0, stream, t, c, o, ws);
}

}  // namespace

hipError_t launch_token_logprobs(int esize, const LogprobTask& t, void* ws, const LogprobOut& o,
                                 hipStream_t stream) {
    const LogprobCut c = logprob_cut(esize, t.part_width, t.n_parts, t.n_rows);
    if (c.segments == 1)
        return launch_parts(esize, t, c, o, ws, stream);
    hipError_t e = launch_parts(esize, t, c, LogprobOut{}, ws, stream);
    if (e != hipSuccess)
        return e;
    const dim3 grid((uint32_t)t.n_rows), block(kThreads);
    return esize == 2 ? launch(logprob_finish_kernel<2>, grid, block, 0, stream, t, c, ws, o)
                      : launch(logprob_finish_kernel<4>, grid, block, 0, stream, t, c, ws, o);
}

hipError_t launch_logprob_records(int esize, const LogprobTask& t, void* ws,
                                  const int32_t* token_ids, int32_t n_tokens, int32_t* stats,
                                  hipStream_t stream) {
    const LogprobCut c = logprob_cut(esize, t.part_width, t.n_parts, t.n_rows);
    hipError_t e = launch_parts(esize, t, c, LogprobOut{}, ws, stream);
    if (e != hipSuccess)
        return e;
    const dim3 grid((uint32_t)((int64_t)t.n_rows * t.n_parts)), block(kThreads);
    return esize == 2 ? launch(logprob_record_kernel<2>, grid, block, 0, stream, t, c, ws,
                               token_ids, n_tokens, stats)
                      : launch(logprob_record_kernel<4>, grid, block, 0, stream, t, c, ws,
                               token_ids, n_tokens, stats);
}

hipError_t launch_logprob_combine(const int32_t* stats, int32_t n_shards, int64_t shard_width,
                                  int32_t vocab, int32_t n_rows, int32_t n_top,
                                  const LogprobOut& o, hipStream_t stream) {
    return launch(logprob_combine_kernel, dim3((uint32_t)n_rows), dim3(kThreads), 0, stream, stats,
                  n_shards, shard_width, vocab, n_rows, n_top, o);
}

int64_t logprob_grad_threads(int esize, int64_t grad_cols, int64_t n_rows) {
    const int64_t chunk = chunk_cols(esize, kGradVecs);
    return (grad_cols + chunk - 1) / chunk * n_rows * kThreads;
}

hipError_t launch_logprob_grad(int esize, const LogprobGradTask& t, hipStream_t stream) {
    const int64_t chunk = chunk_cols(esize, kGradVecs);
    const int32_t chunks = (int32_t)((t.grad_cols + chunk - 1) / chunk);
    const dim3 grid((uint32_t)((int64_t)chunks * t.n_rows)), block(kThreads);
    if (esize == 2)
        return t.grad_entropy
                   ? launch(logprob_grad_kernel<2, true>, grid, block, 0, stream, t, chunks)
                   : launch(logprob_grad_kernel<2, false>, grid, block, 0, stream, t, chunks);
    return t.grad_entropy
               ? launch(logprob_grad_kernel<4, true>, grid, block, 0, stream, t, chunks)
               : launch(logprob_grad_kernel<4, false>, grid, block, 0, stream, t, chunks);
}

}  // namespace vpa
