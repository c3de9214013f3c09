// sampled.hip -- verification of drafted tokens against the target's
// probabilities, from given random numbers.
//
// Three or four launches: partial sums of exponentials and the argmax of every
// row's segments; a request's acceptance tests, which give the row it draws
// from, and that row's exponentials summed in 64 bits by blocks of columns; the
// sums of the weights max(p - q, 0), where a draft distribution is subtracted;
// the column where the running sum passes the random number.
//
// The draw is in 64 bits because a border lies between any two of up to 2^24
// columns: with sums that are off by 2^-24 one draw in a hundred over a flat
// row of 2e5 columns would come out a column off.  With e = exp((x - m) / T) and
// Z its sum, the weights are e - q Z, so nothing is divided.  An acceptance has one
// border: the row's fp32 sum decides it, and where that is too near to say, a sum in
// 64 bits.
#include <type_traits>

#include "row_scan.h"
#include "vpa_draft_internal.h"

namespace vpa {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMostSegments = 64;
constexpr int kDrawCols = 1024;                    // columns of a block of the drawn row

// A segment of a row of logits: m near its largest, s = sum exp((x - m) / T), and
// the first column in the argmax order.  s is NaN where it holds a NaN or +inf;
// m = -inf where nothing is finite.
struct RowStat {
    float m, s;
    uint64_t order;
};

// The row a request draws from, as the acceptance tests leave it.
enum DrawKind : int32_t { kDrawn, kPlain, kWithout, kMinus };
struct Draw {
    double scale;              // log2(e) / T
    float m;
    int32_t kind;              // kDrawn: the token stands; weights e, e without `id`, e - q Z
    int32_t row, q_row, id, pos;
};
// Sums over a block of that row's columns: of e, and of the weights.
struct DrawSum {
    double e, w;
};

// 2^((x - m) scale) as 2^n (1 + f q(f)): n the nearest whole number, which 1.5 2^52
// leaves in the last bits of a sum, and q the interpolation of (2^f - 1) / f at the
// 9 Chebyshev nodes of [-1/2, 1/2], off by 4e-14 at most.  From `least` down (and
// for -inf) x is taken for one whose power is below every number.
struct Power {
    double m, scale, least, top;
    __device__ __forceinline__ Power(double m_, double scale_)
        : m(m_), scale(scale_), least(-1100.0 / scale_), top(0x1.b63880a30e9ffp-24) {
        asm("" : "+v"(top));                       // in registers, not moved there each time
    }
    __device__ __forceinline__ double of(float x) const {
        constexpr double kWhole = 0x1.8p52;
        // (one multiply-add of x scale - m scale loses every digit where m is 1e30)
        const double d = fmax((double)x - m, least);
        const double t = __builtin_fma(d, scale, kWhole);
        const double f = __builtin_fma(d, scale, -(t - kWhole));
        double q = __builtin_fma(top, f, 0x1.63d136366db24p-20);
        q = __builtin_fma(q, f, 0x1.ffcb9515a8016p-17);
        q = __builtin_fma(q, f, 0x1.4308ac85aa947p-13);
        q = __builtin_fma(q, f, 0x1.5d87fe86fe88ep-10);
        q = __builtin_fma(q, f, 0x1.3b2ab7181b755p-7);
        q = __builtin_fma(q, f, 0x1.c6b08d7047e52p-5);
        q = __builtin_fma(q, f, 0x1.ebfbdff823cedp-3);
        q = __builtin_fma(q, f, 0x1.62e42fefa39efp-1);
        return __builtin_amdgcn_ldexp(__builtin_fma(q, f, 1.0),
                                      (int)__builtin_bit_cast(uint64_t, t));
    }
};

__device__ __forceinline__ float temperature_of(const SampleTask& t, int32_t req) {
    return t.temperature ? t.temperature[req] : 1.0f;
}
__device__ __forceinline__ bool is_greedy(float temperature) {
    return !(temperature >= 0x1p-100f && temperature < __builtin_inff());
}
__device__ __forceinline__ bool is_draft(const SampleTask& t, int32_t id) {
    return id >= 0 && id < t.vocab;
}

// A workgroup a segment of a row.  Bound by reading: 170 x 6 x 200064 bf16 68 us, 6.0
// TB/s; 1 x 5 x 151936 5.3 us, latency.  A chunk is 2 vectors a thread: 170 x 6 x
// 200064 bf16 110 us for the whole call, 117 with 8 and 108-117 with 1; 64 x 4 x
// 151936 37, 39 and 42; 24 x 4 x 32000 14.5, 17.3 and 15.0.
constexpr int kRowVecs = 2;

template <int ESIZE>
__global__ __launch_bounds__(kThreads) void sample_rows_kernel(SampleTask t, SampleCut cut,
                                                               RowStat* stats) {
    using T = typename elem<ESIZE>::type;
    using Scan = SegmentScan<ESIZE, kRowVecs, kThreads, true>;
    __shared__ ExpSum lds_s[kWaves];
    __shared__ uint64_t lds_o[kWaves];
    const int32_t row = blockIdx.x / cut.row_segments, seg = blockIdx.x % cut.row_segments;
    const int32_t req = row / (t.k + 1), pos = row % (t.k + 1);
    // rows after a placeholder are not needed
    const int32_t* ids = t.draft_ids + (int64_t)req * t.k;
    bool ended = false;
    if (pos <= 16) {                               // the same loads in every lane
        for (int j = 0; j < pos; ++j)
            ended |= !is_draft(t, ids[j]);
    } else {
        for (int j = threadIdx.x; j < pos; j += kThreads)
            ended |= !is_draft(t, ids[j]);
        ended = __syncthreads_or(ended);
    }
    if (ended)
        return;
    const T* x = (const T*)t.logits + (int64_t)row * t.ld;
    const float temp = temperature_of(t, req);
    const float scale = is_greedy(temp) ? kLog2e : kLog2e / temp;
    const int first = -(int)(((uintptr_t)x & 15) / ESIZE);
    const int begin = first + seg * cut.row_chunks * Scan::CHUNK;
    const int end = begin + cut.row_chunks * Scan::CHUNK;
    const int lo = begin < 0 ? 0 : begin, hi = end < t.vocab ? end : t.vocab;
    Scan scan;
    scan.run(x, begin, lo, hi, scale, [](auto&, int) {});
    const ExpSum s = scan.wave();
    const uint64_t best = scan.wave_best(x, begin, lo, hi);
    if ((threadIdx.x & 63) == 0) {
        lds_s[threadIdx.x >> 6] = s;
        lds_o[threadIdx.x >> 6] = best;
    }
    __syncthreads();
    if (threadIdx.x != 0)
        return;
    ExpSum all = lds_s[0];
    uint64_t order = lds_o[0];
#pragma unroll
    for (int i = 1; i < kWaves; ++i) {
        all = join(all, lds_s[i], scale);
        order = lds_o[i] > order ? lds_o[i] : order;
    }
    stats[blockIdx.x] = RowStat{all.m, all.s, order};
}

// Sum over a workgroup of kThreads, of each thread's own, in a fixed order.
__device__ __forceinline__ double block_sum_f64(double v, double (&lds)[kWaves]) {
    v = wave_sum_f64(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        lds[threadIdx.x >> 6] = v;
    __syncthreads();
    return ((lds[0] + lds[1]) + lds[2]) + lds[3];
}

// Sum of a row's exponentials in 64 bits, by a workgroup.
template <int ESIZE>
__device__ __forceinline__ double row_sum_f64(const SampleTask& t, int32_t row, const Power& e,
                                              double (&lds)[kWaves]) {
    constexpr int VEC = 16 / ESIZE;
    const auto* x = (const typename elem<ESIZE>::type*)t.logits + (int64_t)row * t.ld;
    // whole aligned vectors, and what lies before and after them
    int first = (int)(((16 - ((uintptr_t)x & 15)) & 15) / ESIZE);
    first = first < t.vocab ? first : t.vocab;
    const int vecs = (t.vocab - first) / VEC, tail = first + vecs * VEC;
    double s = 0.0;
#pragma unroll 1
    for (int i = threadIdx.x; i < vecs; i += kThreads) {
        const u32x4_t v = *(const u32x4_t*)(x + first + i * VEC);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            s += e.of(vec_elem<ESIZE>(v, k));
            asm volatile("" : "+v"(s));            // registers for one at a time
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    const int c = (int)threadIdx.x < first ? (int)threadIdx.x : tail + (int)threadIdx.x - first;
    if (c < t.vocab && c - tail < VEC)
        s += e.of(to_f32(x[c]));
    return block_sum_f64(s, lds);
}

// How near to its border, relatively, an acceptance is decided again in 64 bits.
// The rows' fp32 sums are off by less than 2^-17: of the exponents, up to kLag above
// M and ln V below the maximum on average, a step's half and the rounded scale take
// 0.5 and 2.2e-6, their joining over wavefronts and segments 2.2e-6 again, the sums
// themselves 1e-6.  One position in 2^15 or so takes that long: 60 us for 200064
// columns.
constexpr double kNear = 0x1p-16;

// The acceptance tests of a request by a workgroup, a wavefront a position, until
// one is not accepted: the row that the request draws from.  `token` is the argmax
// where that is what it draws, else -1.
template <int ESIZE, int QSIZE>
__device__ __forceinline__ Draw accept_request(const SampleTask& t, const SampleCut& cut,
                                               const RowStat* stats, int32_t req, int32_t& token) {
    using T = typename elem<ESIZE>::type;
    using Q = typename elem<QSIZE>::type;
    enum { kAccepted, kEnds, kOpen };
    __shared__ Draw ends[kWaves];
    __shared__ int32_t tokens[kWaves], states[kWaves];
    __shared__ float logits[kWaves];               // of the open ones: x, and u q
    __shared__ double borders[kWaves], lds[kWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const float temp = temperature_of(t, req);
    const float scale = is_greedy(temp) ? kLog2e : kLog2e / temp;
    for (int first = 0;; first += kWaves) {
        const int pos = first + wave;
        int32_t state = kEnds;
        if (pos <= t.k) {
            const int32_t row = req * (t.k + 1) + pos;
            RowStat st = {kMinusInf, 0.0f, 0};
            if (lane < cut.row_segments)
                st = stats[(int64_t)row * cut.row_segments + lane];
            // the draft's logit and probability are on their way meanwhile
            const int32_t id = pos < t.k ? t.draft_ids[(int64_t)req * t.k + pos] : -1;
            const int32_t q_row = req * t.k + pos;
            float x = 0.0f, q = 1.0f, u = 0.0f;
            if (is_draft(t, id)) {
                x = to_f32(((const T*)t.logits)[(int64_t)row * t.ld + id]);
                u = t.accept_u[q_row];
                if (t.probs)
                    q = to_f32(((const Q*)t.probs)[(int64_t)q_row * t.ldq + id]);
            }
            const ExpSum sum = wave_join(ExpSum{st.m, st.s}, scale);
            const uint64_t order = wave_max_u64(st.order);
            const bool greedy = is_greedy(temp) || !(fabsf(sum.m) < __builtin_inff()) ||
                                !(sum.s < __builtin_inff());
            Draw d;
            d.scale = 1.4426950408889634074 / (double)temp;
            d.m = sum.m;
            d.kind = kPlain;
            d.row = row;
            d.q_row = 0;
            d.id = -1;
            d.pos = pos;
            if (is_draft(t, id)) {
                double p;
                if (greedy)
                    p = id == id_of(order) ? 1.0 : 0.0;
                else
                    p = Power((double)sum.m, d.scale).of(x) / (double)sum.s;
                const double border = (double)u * (double)q;
                state = border < p ? kAccepted : kEnds;
                if (!greedy && fabs(border - p) < kNear * p)
                    state = kOpen;
                if (lane == 0) {
                    logits[wave] = x;
                    borders[wave] = border;
                }
                d.q_row = q_row;
                d.kind = t.probs ? kMinus : kWithout;
                d.id = id;
            }
            if (greedy)
                d.kind = kDrawn;
            if (lane == 0) {
                ends[wave] = d;
                tokens[wave] = greedy ? id_of(order) : -1;
            }
        }
        if (lane == 0)
            states[wave] = state;
        __syncthreads();
        for (int i = 0; i < kWaves; ++i) {         // (the same in all threads)
            bool end = states[i] == kEnds;
            if (states[i] == kOpen) {
                const Power e((double)ends[i].m, ends[i].scale);
                end = !(borders[i] < e.of(logits[i]) / row_sum_f64<ESIZE>(t, ends[i].row, e, lds));
            }
            if (end) {
                token = tokens[i];
                return ends[i];
            }
        }
        __syncthreads();
    }
}

// What is known of a request's outputs before its draw; by a workgroup.
__device__ __forceinline__ void write_request(const SampleTask& t, int32_t req, const Draw& d,
                                              int32_t token, Draw* draws) {
    int32_t* out = t.out_tokens + (int64_t)req * (t.k + 1);
    for (int j = threadIdx.x; j <= t.k; j += kThreads)
        out[j] = j < d.pos ? t.draft_ids[(int64_t)req * t.k + j] : j == d.pos ? token : -1;
    if (threadIdx.x == 0) {
        t.num_sampled[req] = d.pos + 1;
        t.num_rejected[req] = t.k - d.pos;
        draws[req] = d;
    }
}

// The weights of the columns of the row that is drawn from, by KIND, or with kAny
// by the kind that a call is given: a few columns, for which three copies of the
// code would take longer to fetch than to run.
constexpr int kAny = -1;

template <int ESIZE, int QSIZE, int KIND>
struct Weights {
    using T = typename elem<ESIZE>::type;
    using Q = typename elem<QSIZE>::type;
    const T* x;
    const Q* q;
    Power e;
    double z;
    int32_t id, kind;

    __device__ __forceinline__ Weights(const SampleTask& t, const Draw& d, int32_t k, double sum)
        : e((double)d.m, d.scale) {
        kind = KIND == kAny ? k : KIND;
        x = (const T*)t.logits + (int64_t)d.row * t.ld;
        q = (const Q*)t.probs + (int64_t)d.q_row * t.ldq;
        z = sum;
        id = d.id;
    }
    // what N consecutive columns hold
    template <int N>
    struct Columns {
        struct __attribute__((packed, aligned(sizeof(T)))) {
            T v[N];
        } x;
        struct __attribute__((packed, aligned(sizeof(Q)))) {
            Q v[N];
        } q;
    };
    // columns from c on, masked from `hi` on
    template <int N>
    __device__ __forceinline__ void load(int c, int hi, Columns<N>& o) const {
        if (c + N <= hi) {
            o.x = *(const decltype(o.x)*)(x + c);
            if (kind == kMinus)
                o.q = *(const decltype(o.q)*)(q + c);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                from_f32(o.x.v[i], c + i < hi ? to_f32(x[c + i]) : kMinusInf);
                o.q.v[i] = 0;
                if (kind == kMinus && c + i < hi)
                    o.q.v[i] = q[c + i];
            }
        }
    }
    // their weights
    template <int N>
    __device__ __forceinline__ void of(int c, const Columns<N>& o, double (&w)[N]) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            w[i] = e.of(to_f32(o.x.v[i]));
            if (kind == kMinus)
                w[i] = fmax(__builtin_fma(-(double)to_f32(o.q.v[i]), z, w[i]), 0.0);
            if (kind == kWithout)
                w[i] = c + i == id ? 0.0 : w[i];
        }
    }
};

// Calls f with the kind as a type.
template <typename F>
__device__ __forceinline__ void with_kind(int32_t kind, F f) {
    using std::integral_constant;
    if (kind == kMinus)
        f(integral_constant<int, kMinus>{});
    else if (kind == kWithout)
        f(integral_constant<int, kWithout>{});
    else
        f(integral_constant<int, kPlain>{});
}

__device__ __forceinline__ double sum_of_e(const DrawSum* sums, int blocks, double (&lds)[kWaves]) {
    double v = 0.0;
    for (int i = threadIdx.x; i < blocks; i += kThreads)
        v += sums[i].e;
    return block_sum_f64(v, lds);
}

// The acceptance tests alone; a workgroup a request.  5.8 us for 170 of 6 positions,
// latency: the segments' sums, the draft's logit, 64-bit divisions.
template <int ESIZE, int QSIZE>
__global__ __launch_bounds__(kThreads) void sample_accept_kernel(SampleTask t, SampleCut cut,
                                                                 const RowStat* stats,
                                                                 Draw* draws) {
    int32_t token;
    const Draw d = accept_request<ESIZE, QSIZE>(t, cut, stats, blockIdx.x, token);
    write_request(t, blockIdx.x, d, token, draws);
}

// Sums of the weights over blocks of kDrawCols columns of each request's row, a
// wavefront a block at a time; of e alone for the requests that subtract a draft
// distribution, whose weights are summed by a second launch (kSecond).  With
// kAccept each of a request's workgroups makes its acceptance tests, and the
// first writes what they say: while the workgroups run at once, 6 a CU, that costs
// less than a launch (1 x 5 x 151936 14.4 us with a launch of its own, 13.1 so; 24 x 4
// 23.2 and 21.7; 40 x 4, 1520 workgroups, 28.5 and 27.8; 300 x 3 x 4000 19.4 and 17.5),
// more of them take as long or longer (48 x 4 x 151936, 1824 of them, 31.8 and 32.0;
// 64 x 6 x 200064 52.2 and 54.6).
//
// Bound by instructions: 18 an element for e, 24 for e - q Z, most of them 64-bit
// ones, of 5 clocks of a SIMD each: for 170 x 200064 bf16 20 and 27 us of 30 and
// 32 (the loads alone take 14 and 28).  The next block's loads ahead of a block's
// sums made it no faster.
enum SumsStep { kAccept, kFirst, kSecond };
constexpr int64_t kAcceptInSums = 6 * 256;         // workgroups

// (6 wavefronts a SIMD: kAccept's second look at an acceptance would leave 5, with which
// 64 x 4 x 151936 took 37.7 us for 36.8)
template <int ESIZE, int QSIZE, int STEP>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(6))) void
sample_sums_kernel(SampleTask t, SampleCut cut, const RowStat* stats, Draw* draws, DrawSum* sums) {
    constexpr int VEC = 16 / ESIZE;
    constexpr bool SECOND = STEP == kSecond;
    __shared__ double lds[kWaves];
    const int32_t req = blockIdx.x / cut.draw_groups, group = blockIdx.x % cut.draw_groups;
    Draw d;
    if constexpr (STEP == kAccept) {
        int32_t token;
        d = accept_request<ESIZE, QSIZE>(t, cut, stats, req, token);
        if (group == 0)
            write_request(t, req, d, token, draws);
    } else {
        d = draws[req];
    }
    if (d.kind == kDrawn || (SECOND && d.kind != kMinus))
        return;
    DrawSum* mine = sums + (int64_t)req * cut.draw_blocks;
    const double z = SECOND ? sum_of_e(mine, cut.draw_blocks, lds) : 0.0;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    with_kind(!SECOND && d.kind == kMinus ? (int32_t)kPlain : d.kind, [&](auto kind) {
        const Weights<ESIZE, QSIZE, kind()> w(t, d, kind(), z);
        for (int b = group * kWaves + wave; b < cut.draw_blocks; b += cut.draw_groups * kWaves) {
            double s = 0.0;
#pragma unroll
            for (int i = 0; i < kDrawCols / 64 / VEC; ++i) {
                const int c = b * kDrawCols + (i * 64 + lane) * VEC;
                typename Weights<ESIZE, QSIZE, kind()>::template Columns<VEC> columns;
                double v[VEC];
                w.load(c, t.vocab, columns);
                w.of(c, columns, v);
#pragma unroll
                for (int k = 0; k < VEC; ++k)
                    s += v[k];
            }
            s = wave_sum_f64(s);
            if (lane != 0)
                continue;
            if (!SECOND && d.kind == kMinus)
                mine[b].e = s;
            else
                mine[b].w = s;
        }
    });
}

// The running sum over a workgroup's threads, each with its own v: what is
// before the thread's, and the whole.
__device__ __forceinline__ double block_scan_f64(double v, double& all, double (&lds)[kWaves]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const double upto = wave_scan_f64(v);
    double before = __shfl_up(upto, 1, 64);
    before = lane == 0 ? 0.0 : before;
    __syncthreads();
    if (lane == 63)
        lds[wave] = upto;
    __syncthreads();
    all = ((lds[0] + lds[1]) + lds[2]) + lds[3];
#pragma unroll
    for (int i = 0; i < kWaves - 1; ++i)
        before += i < wave ? lds[i] : 0.0;
    return before;
}

// The first of a workgroup's items, in the order of its threads, that the running
// sum passes at; as long as none does, the last one with a weight.  (Atomics on
// LDS go through a wavefront's lanes one by one.)
struct PassingWave {
    double before;
    int32_t index;
    int32_t kind;              // 2: passed, 1: has a weight, 0: neither
};
template <int WAVES>
struct Passing {
    PassingWave* lds;
    bool passed = false;
    int32_t index = 0;
    double before = 0.0;
    __device__ __forceinline__ explicit Passing(PassingWave* l) : lds(l) {}

    // every thread: whether it passes at item `at`, whether it has a weight and its
    // last one, and the sum before
    __device__ __forceinline__ void take(bool passes, bool weight, int32_t at, int32_t top,
                                         double sum) {
        const uint64_t p = __ballot(passes), w = __ballot(weight);
        const int from = p ? (int)__builtin_ctzll(p) : w ? 63 - (int)__builtin_clzll(w) : 0;
        __syncthreads();
        if ((int)(threadIdx.x & 63) == from)
            lds[threadIdx.x >> 6] = PassingWave{sum, p ? at : top, p ? 2 : w ? 1 : 0};
        __syncthreads();
#pragma unroll
        for (int i = 0; i < WAVES; ++i) {
            const PassingWave o = lds[i];
            if (!passed && o.kind != 0) {
                passed = o.kind == 2;
                index = o.index;
                before = o.before;
            }
        }
    }
};

// The column where the running sum passes the random number: its block from the
// blocks' sums, then its 4 columns a thread.  Where rounding lets none pass, and
// for random numbers from 1 on, the last one with a weight.  Bound by latency (loads,
// scans and barriers one after another): 3.4 us for one request, 4.3 for 170.
template <int ESIZE, int QSIZE>
__global__ __launch_bounds__(kThreads) void sample_pick_kernel(SampleTask t, SampleCut cut,
                                                               const Draw* draws,
                                                               const DrawSum* sums) {
    constexpr int N = kDrawCols / kThreads;
    __shared__ double lds[kWaves];
    __shared__ PassingWave found[kWaves];
    const int32_t req = blockIdx.x;
    const DrawSum* mine = sums + (int64_t)req * cut.draw_blocks;
    // loaded together: a kernel's first loads take a microsecond
    const Draw d = draws[req];
    const double u = t.sample_u[req];
    DrawSum first = {0.0, 0.0};
    if ((int)threadIdx.x < cut.draw_blocks)
        first = mine[threadIdx.x];
    __builtin_amdgcn_sched_barrier(0);
    if (d.kind == kDrawn)
        return;
    double total = first.w, z = d.kind == kMinus ? first.e : 0.0;
    for (int i = threadIdx.x + kThreads; i < cut.draw_blocks; i += kThreads) {
        const DrawSum s = mine[i];
        total += s.w;
        z += d.kind == kMinus ? s.e : 0.0;
    }
    total = block_sum_f64(total, lds);
    if (d.kind == kMinus)
        z = block_sum_f64(z, lds);
    int32_t kind = d.kind;
    if (!(total > 0.0)) {
        // no weight: p itself, which has the draft's column alone where nothing else is left
        if (kind != kMinus) {
            if (threadIdx.x == 0)
                t.out_tokens[(int64_t)req * (t.k + 1) + d.pos] = d.id;
            return;
        }
        kind = kPlain;
        total = z;
    }
    const bool of_e = kind != d.kind;
    // (from 1 on nothing passes: the sums' orders differ, and the last columns may be too
    // small to change one)
    const double target = u >= 1.0 ? (double)__builtin_inff() : (u > 0.0 ? u : 0.0) * total;
    // the block
    Passing<kWaves> at(found);
    double run = 0.0;
    for (int b0 = 0; b0 < cut.draw_blocks; b0 += kThreads) {
        const int b = b0 + (int)threadIdx.x;
        double v = 0.0, all;
        if (b0 == 0)
            v = of_e ? first.e : first.w;
        else if (b < cut.draw_blocks)
            v = of_e ? mine[b].e : mine[b].w;
        const double before = run + block_scan_f64(v, all, lds);
        at.take(v > 0.0 && before + v > target, v > 0.0, b, b, before);
        run += all;
        if (at.passed)
            break;
    }
    const int block = at.index;
    const double from = at.before;
    // the column
    const Weights<ESIZE, QSIZE, kAny> w(t, d, kind, z);
    const int c = block * kDrawCols + (int)threadIdx.x * N;
    double v[N], own = 0.0, all;
    typename Weights<ESIZE, QSIZE, kAny>::template Columns<N> columns;
    w.load(c, t.vocab, columns);
    w.of(c, columns, v);
    int top = -1;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        own += v[i];
        top = v[i] > 0.0 ? c + i : top;
    }
    double sum = from + block_scan_f64(own, all, lds);
    int32_t token = t.vocab;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        sum += v[i];
        token = v[i] > 0.0 && sum > target && token == t.vocab ? c + i : token;
    }
    Passing<kWaves> column(found);
    column.take(token < t.vocab, top >= 0, token, top, 0.0);
    if (threadIdx.x == 0)
        t.out_tokens[(int64_t)req * (t.k + 1) + d.pos] = column.index;
}

size_t align16(size_t n) {
    return (n + 15) / 16 * 16;
}

// Where the parts of the workspace lie.
struct Layout {
    size_t draws, sums, total;
};
Layout layout_of(const SampleCut& c, int64_t n_req, int32_t k) {
    Layout l;
    l.draws = align16((size_t)n_req * (k + 1) * c.row_segments * sizeof(RowStat));
    l.sums = l.draws + align16((size_t)n_req * sizeof(Draw));
    l.total = l.sums + (size_t)n_req * c.draw_blocks * sizeof(DrawSum);
    return l;
}

}  // namespace

// Rows in segments of whole chunks until there are 4 workgroups a CU (65 x 4 x
// 151936: 40.7 us with 4, 42.5 with 8, 41.1 with 16; 24 x 4 23.5, 23.7, 27.3).
// A drawn row has a wavefront for each block of columns, 16 workgroups a CU at
// most over all requests (64 x 4 x 151936: 43.0 us with 8, 38.6 with 16, 38.2 with 32).
SampleCut sample_cut(int esize, int64_t vocab, int64_t n_req, int32_t k) {
    SampleCut c;
    const int64_t rows = n_req * (k + 1), vec = 16 / esize;
    const int64_t width = vocab + vec - 1;         // with the columns before an aligned one
    const int64_t chunk = kThreads * kRowVecs * vec, chunks = (width + chunk - 1) / chunk;
    int64_t want = (1024 + rows - 1) / rows;
    want = want > chunks ? chunks : want;
    want = want > kMostSegments ? kMostSegments : want;
    c.row_chunks = (int32_t)((chunks + want - 1) / want);
    c.row_segments = (int32_t)((chunks + c.row_chunks - 1) / c.row_chunks);
    c.draw_blocks = (int32_t)((vocab + kDrawCols - 1) / kDrawCols);
    const int64_t groups = (4096 + n_req - 1) / n_req, enough = (c.draw_blocks + kWaves - 1) / kWaves;
    c.draw_groups = (int32_t)(groups < enough ? groups : enough);
    return c;
}

size_t sample_workspace(const SampleCut& c, int64_t n_req, int32_t k) {
    return layout_of(c, n_req, k).total;
}

int64_t sample_threads(const SampleCut& c, int64_t n_req, int32_t k) {
    const int64_t rows = n_req * (k + 1) * c.row_segments * kThreads;
    const int64_t sums = n_req * c.draw_groups * kThreads;
    return rows > sums ? rows : sums;
}

namespace {

template <int ESIZE, int QSIZE>
hipError_t launch_typed(const SampleTask& t, void* ws, hipStream_t stream) {
    const SampleCut c = sample_cut(ESIZE, t.vocab, t.n_req, t.k);
    const Layout l = layout_of(c, t.n_req, t.k);
    RowStat* stats = (RowStat*)ws;
    Draw* draws = (Draw*)((char*)ws + l.draws);
    DrawSum* sums = (DrawSum*)((char*)ws + l.sums);
    const dim3 rows((uint32_t)((int64_t)t.n_req * (t.k + 1) * c.row_segments));
    const dim3 groups((uint32_t)((int64_t)t.n_req * c.draw_groups)), reqs((uint32_t)t.n_req);
    const dim3 block(kThreads);
    hipError_t e = launch(sample_rows_kernel<ESIZE>, rows, block, 0, stream, t, c, stats);
    if (e == hipSuccess && groups.x <= kAcceptInSums) {
        e = launch(sample_sums_kernel<ESIZE, QSIZE, kAccept>, groups, block, 0, stream, t, c, stats,
                   draws, sums);
    } else if (e == hipSuccess) {
        e = launch(sample_accept_kernel<ESIZE, QSIZE>, reqs, block, 0, stream, t, c, stats, draws);
        if (e == hipSuccess)
            e = launch(sample_sums_kernel<ESIZE, QSIZE, kFirst>, groups, block, 0, stream, t, c,
                       stats, draws, sums);
    }
    if (e == hipSuccess && t.probs)
        e = launch(sample_sums_kernel<ESIZE, QSIZE, kSecond>, groups, block, 0, stream, t, c, stats,
                   draws, sums);
    if (e == hipSuccess)
        e = launch(sample_pick_kernel<ESIZE, QSIZE>, reqs, dim3(kThreads), 0, stream, t, c,
                   draws, sums);
    return e;
}

}  // namespace

hipError_t launch_sample(int esize, int probs_esize, const SampleTask& t, void* ws,
                         hipStream_t stream) {
    if (esize == 2)
        return probs_esize == 2 ? launch_typed<2, 2>(t, ws, stream)
                                : launch_typed<2, 4>(t, ws, stream);
    return probs_esize == 2 ? launch_typed<4, 2>(t, ws, stream) : launch_typed<4, 4>(t, ws, stream);
}

}  // namespace vpa
