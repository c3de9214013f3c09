// sampled.hip -- verification of drafted tokens against the target's
// probabilities, from given random numbers.
//
// Five steps: partial sums of exponentials and the argmax of every row's
// segments; a request's acceptance tests, which give the row it draws from;
// that row's exponentials summed in 64 bits by segments; the sums of the
// weights max(p - q, 0), where a draft distribution is subtracted; the column
// where the running sum passes the random number.
//
// The draw is in 64 bits because a border lies between any two of up to 2^24
// columns: with sums that are off by 2^-24 one draw in a hundred over a flat
// row of 2e5 columns would come out a column off.  With e = exp((x - m) / T) and
// Z its sum, the weights are e - q Z, so nothing is divided.
#include "row_scan.h"
#include "vpa_draft_internal.h"

namespace vpa {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMostSegments = 64;

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
// Sums over a segment of that row: of e, and of the weights.
struct DrawSum {
    double e, w;
};

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1)
        v += __shfl_xor(v, off, 64);
    return v;
}

// 2^z for z <= 1000, 0 below 2^-1000 (a masked column): 2^n (1 + f q(f)) with n
// the nearest whole number and q the interpolation of (2^f - 1) / f at the 9
// Chebyshev nodes of [-1/2, 1/2], off by 4e-14 at most.
__device__ __forceinline__ double exp2_f64(double z) {
    const double n = __builtin_rint(z);
    const double f = z - n;
    double q = 0x1.b63880a30e9ffp-24;
    q = __builtin_fma(q, f, 0x1.63d136366db24p-20);
    q = __builtin_fma(q, f, 0x1.ffcb9515a8016p-17);
    q = __builtin_fma(q, f, 0x1.4308ac85aa947p-13);
    q = __builtin_fma(q, f, 0x1.5d87fe86fe88ep-10);
    q = __builtin_fma(q, f, 0x1.3b2ab7181b755p-7);
    q = __builtin_fma(q, f, 0x1.c6b08d7047e52p-5);
    q = __builtin_fma(q, f, 0x1.ebfbdff823cedp-3);
    q = __builtin_fma(q, f, 0x1.62e42fefa39efp-1);
    return z < -1000.0 ? 0.0 : __builtin_amdgcn_ldexp(__builtin_fma(q, f, 1.0), (int)n);
}

__device__ __forceinline__ float temperature_of(const SampleTask& t, int32_t req) {
    return t.temperature ? t.temperature[req] : 1.0f;
}
__device__ __forceinline__ bool is_greedy(float temperature) {
    return !(temperature >= 0x1p-100f && temperature < __builtin_inff());
}
__device__ __forceinline__ bool is_draft(const SampleTask& t, int32_t id) {
    return id >= 0 && id < t.vocab;
}

// A workgroup a segment of a row.
template <int ESIZE, int U>
__global__ __launch_bounds__(kThreads) void sample_rows_kernel(SampleTask t, SampleCut cut,
                                                               RowStat* stats) {
    using T = typename elem<ESIZE>::type;
    using Scan = SegmentScan<ESIZE, U, kThreads, true>;
    __shared__ ExpSum lds_s[kWaves];
    __shared__ uint64_t lds_o[kWaves];
    const int32_t row = blockIdx.x / cut.row_segments, seg = blockIdx.x % cut.row_segments;
    const int32_t req = row / (t.k + 1), pos = row % (t.k + 1);
    // rows after a placeholder are not needed
    bool ended = false;
    for (int j = threadIdx.x; j < pos; j += kThreads)
        ended |= !is_draft(t, t.draft_ids[(int64_t)req * t.k + j]);
    if (__syncthreads_or(ended))
        return;
    const T* x = (const T*)t.logits + (int64_t)row * t.ld;
    const float temp = temperature_of(t, req);
    const float scale = is_greedy(temp) ? kLog2e : kLog2e / temp;
    const int first = -(int)(((uintptr_t)x & 15) / ESIZE);
    const int begin = first + seg * cut.row_chunks * Scan::CHUNK;
    const int end = begin + cut.row_chunks * Scan::CHUNK;
    const int lo = begin < 0 ? 0 : begin, hi = end < t.vocab ? end : t.vocab;
    Scan scan;
    scan.run(x, begin, lo, hi, scale, 60.0f, [](auto&, int) {});
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

// A workgroup a request, a wavefront a position, until one is not accepted.
constexpr int kAcceptWaves = 8;

template <int ESIZE, int QSIZE>
__global__ __launch_bounds__(kAcceptWaves * 64) void sample_accept_kernel(SampleTask t,
                                                                          SampleCut cut,
                                                                          const RowStat* stats,
                                                                          Draw* draws) {
    using T = typename elem<ESIZE>::type;
    using Q = typename elem<QSIZE>::type;
    __shared__ Draw ends[kAcceptWaves];
    __shared__ int32_t tokens[kAcceptWaves];         // the argmax where it is drawn, else -1
    __shared__ int32_t at_end[kAcceptWaves];
    const int32_t req = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const float temp = temperature_of(t, req);
    const float scale = is_greedy(temp) ? kLog2e : kLog2e / temp;
    const int32_t* ids = t.draft_ids + (int64_t)req * t.k;
    for (int first = 0;; first += kAcceptWaves) {
        const int pos = first + wave;
        bool last = true;
        if (pos <= t.k) {
            const int32_t row = req * (t.k + 1) + pos;
            RowStat st = {kMinusInf, 0.0f, 0};
            if (lane < cut.row_segments)
                st = stats[(int64_t)row * cut.row_segments + lane];
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
            const int32_t id = pos < t.k ? ids[pos] : -1;
            if (is_draft(t, id)) {
                double p;
                if (greedy)
                    p = id == id_of(order) ? 1.0 : 0.0;
                else
                    p = exp2_f64(((double)to_f32(((const T*)t.logits)[(int64_t)row * t.ld + id]) -
                                  (double)sum.m) * d.scale) / (double)sum.s;
                d.q_row = req * t.k + pos;
                const double q =
                    t.probs ? (double)to_f32(((const Q*)t.probs)[(int64_t)d.q_row * t.ldq + id]) : 1.0;
                last = !((double)t.accept_u[d.q_row] * q < p);
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
            at_end[wave] = last;
        __syncthreads();
        int found = 0;
        while (found < kAcceptWaves && !at_end[found])
            ++found;
        if (found < kAcceptWaves) {
            const Draw d = ends[found];
            int32_t* out = t.out_tokens + (int64_t)req * (t.k + 1);
            for (int j = threadIdx.x; j <= t.k; j += kAcceptWaves * 64)
                out[j] = j < d.pos ? ids[j] : j == d.pos ? tokens[found] : -1;
            if (threadIdx.x == 0) {
                t.num_sampled[req] = d.pos + 1;
                t.num_rejected[req] = t.k - d.pos;
                draws[req] = d;
            }
            return;
        }
        __syncthreads();
    }
}

// The weights of VEC columns of the row that is drawn from.
template <int ESIZE, int QSIZE>
struct Weights {
    using T = typename elem<ESIZE>::type;
    using Q = typename elem<QSIZE>::type;
    const T* x;
    const Q* q;
    double scale, m;           // e = 2^((x - m) scale)
    double z;
    int32_t kind, id;

    __device__ __forceinline__ Weights(const SampleTask& t, const Draw& d) {
        x = (const T*)t.logits + (int64_t)d.row * t.ld;
        q = (const Q*)t.probs + (int64_t)d.q_row * t.ldq;
        scale = d.scale;
        m = (double)d.m;
        z = 0.0;
        kind = d.kind;
        id = d.id;
    }
    __device__ __forceinline__ double e(T v) const {
        // (one multiply-add of x scale - m scale loses every digit where m is 1e30)
        return exp2_f64(((double)to_f32(v) - m) * scale);
    }
    __device__ __forceinline__ double of(int c, double e) const {
        if (kind == kWithout)
            return c == id ? 0.0 : e;
        if (kind == kMinus) {
            const double r = __builtin_fma(-(double)to_f32(q[c]), z, e);
            return r > 0.0 ? r : 0.0;
        }
        return e;
    }
};

// Sums over the segments of each request's row; a workgroup a segment.  With
// SECOND, the sums of e - q Z for the requests that need them.
template <int ESIZE, int QSIZE, bool SECOND>
__global__ __launch_bounds__(kThreads) void sample_sums_kernel(SampleTask t, SampleCut cut,
                                                               const Draw* draws, DrawSum* sums) {
    __shared__ double lds[2][kWaves];
    const int32_t req = blockIdx.x / cut.draw_segments, seg = blockIdx.x % cut.draw_segments;
    const Draw d = draws[req];
    if (d.kind == kDrawn || (SECOND && d.kind != kMinus))
        return;
    Weights<ESIZE, QSIZE> w(t, d);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if constexpr (SECOND) {
        const DrawSum* mine = sums + (int64_t)req * cut.draw_segments;
        w.z = wave_sum_f64(lane < cut.draw_segments ? mine[lane].e : 0.0);
    } else if (d.kind == kMinus) {
        w.kind = kPlain;
    }
    const int lo = seg * cut.draw_cols;
    const int hi = lo + cut.draw_cols < t.vocab ? lo + cut.draw_cols : t.vocab;
    double se = 0.0, sw = 0.0;
    for (int c = lo + (int)threadIdx.x; c < hi; c += kThreads) {
        const double e = w.e(w.x[c]);
        se += e;
        sw += w.of(c, e);
    }
    se = wave_sum_f64(se);
    sw = wave_sum_f64(sw);
    if (lane == 0) {
        lds[0][wave] = se;
        lds[1][wave] = sw;
    }
    __syncthreads();
    if (threadIdx.x != 0)
        return;
    DrawSum* out = sums + blockIdx.x;
    if constexpr (!SECOND)
        out->e = ((lds[0][0] + lds[0][1]) + lds[0][2]) + lds[0][3];
    out->w = ((lds[1][0] + lds[1][1]) + lds[1][2]) + lds[1][3];
}

// The column where the running sum passes the random number: its segment from
// the segments' sums, then a workgroup's threads sum consecutive columns of it,
// and the thread that the border lies in goes through its own.
constexpr int kPickThreads = 1024;

template <int ESIZE, int QSIZE>
__global__ __launch_bounds__(kPickThreads) void sample_pick_kernel(SampleTask t, SampleCut cut,
                                                                   const Draw* draws,
                                                                   const DrawSum* sums) {
    __shared__ double lds[kPickThreads / 64];
    __shared__ int32_t passed, last;
    const int32_t req = blockIdx.x;
    const Draw d = draws[req];
    if (d.kind == kDrawn)
        return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    Weights<ESIZE, QSIZE> w(t, d);
    const DrawSum* all = sums + (int64_t)req * cut.draw_segments;
    if (threadIdx.x == 0) {
        passed = kPickThreads;
        last = 0;
    }
    // every thread goes through the (at most 64) sums in the same order
    double total = 0.0, plain = 0.0;
    for (int i = 0; i < cut.draw_segments; ++i) {
        total += all[i].w;
        plain += all[i].e;
    }
    w.z = wave_sum_f64(lane < cut.draw_segments ? all[lane].e : 0.0);
    const bool fall_back = !(total > 0.0);
    if (fall_back) {
        total = plain;
        w.kind = kPlain;
    }
    const double u = t.sample_u[req];
    const double target = (u > 0.0 ? u : 0.0) * total;
    double before = 0.0, run = 0.0;
    int seg = 0;
    bool inside = false;
    for (int i = 0; i < cut.draw_segments && !inside; ++i) {
        const double s = fall_back ? all[i].e : all[i].w;
        if (s > 0.0) {                             // the last such one, if none passes
            seg = i;
            before = run;
            inside = run + s > target;
        }
        run += s;
    }
    const int lo = seg * cut.draw_cols;
    const int hi = lo + cut.draw_cols < t.vocab ? lo + cut.draw_cols : t.vocab;
    const int per = (hi - lo + kPickThreads - 1) / kPickThreads;
    const int c0 = lo + (int)threadIdx.x * per;
    const int c1 = c0 + per < hi ? c0 + per : hi;
    double mine = 0.0;
    int top = -1;                                  // the thread's last column with a weight
    for (int c = c0; c < c1; ++c) {
        const double v = w.of(c, w.e(w.x[c]));
        mine += v;
        top = v > 0.0 ? c : top;
    }
    double upto = mine;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const double o = __shfl_up(upto, off, 64);
        upto += lane >= off ? o : 0.0;
    }
    if (lane == 63)
        lds[wave] = upto;
    __syncthreads();
    for (int i = 0; i < wave; ++i)
        before += lds[i];
    if (mine > 0.0 && before + upto > target)
        atomicMin(&passed, (int32_t)threadIdx.x);
    if (top >= 0)
        atomicMax(&last, top);
    __syncthreads();
    int32_t* out = t.out_tokens + (int64_t)req * (t.k + 1) + d.pos;
    if (passed == kPickThreads) {
        if (threadIdx.x == 0)
            *out = last;
        return;
    }
    if ((int32_t)threadIdx.x != passed)
        return;
    double sum = before + upto - mine;
    int32_t token = top;
    for (int c = c0; c < c1; ++c) {
        const double v = w.of(c, w.e(w.x[c]));
        sum += v;
        if (v > 0.0 && sum > target) {
            token = c;
            break;
        }
    }
    *out = token;
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
    l.total = l.sums + (size_t)n_req * c.draw_segments * sizeof(DrawSum);
    return l;
}

}  // namespace

// Rows in chunks of 8 vectors a thread where that gives every CU 4 workgroups,
// else of 2, and segments of whole chunks until there are 4 (8) workgroups a CU.
// The drawn rows in segments of at least 2048 columns.
SampleCut sample_cut(int esize, int64_t vocab, int64_t n_req, int32_t k) {
    SampleCut c;
    const int64_t rows = n_req * (k + 1), vec = 16 / esize;
    const int64_t width = vocab + vec - 1;         // with the columns before an aligned one
    const int64_t big = kThreads * 8 * vec;
    c.vecs = 2 * width > big && rows * ((width + big - 1) / big) >= 1024 ? 8 : 2;
    const int64_t chunk = kThreads * c.vecs * vec, chunks = (width + chunk - 1) / chunk;
    int64_t want = ((c.vecs == 8 ? 1024 : 2048) + rows - 1) / rows;
    want = want > chunks ? chunks : want;
    want = want > kMostSegments ? kMostSegments : want;
    c.row_chunks = (int32_t)((chunks + want - 1) / want);
    c.row_segments = (int32_t)((chunks + c.row_chunks - 1) / c.row_chunks);
    int64_t segs = (2048 + n_req - 1) / n_req;
    const int64_t most = (vocab + 2047) / 2048;
    segs = segs > most ? most : segs;
    segs = segs > kMostSegments ? kMostSegments : segs;
    c.draw_cols = (int32_t)(((vocab + segs - 1) / segs + 7) / 8 * 8);
    c.draw_segments = (int32_t)((vocab + c.draw_cols - 1) / c.draw_cols);
    return c;
}

size_t sample_workspace(const SampleCut& c, int64_t n_req, int32_t k) {
    return layout_of(c, n_req, k).total;
}

int64_t sample_threads(const SampleCut& c, int64_t n_req, int32_t k) {
    const int64_t rows = n_req * (k + 1) * c.row_segments * kThreads;
    const int64_t sums = n_req * c.draw_segments * kThreads, pick = n_req * kPickThreads;
    return rows > sums ? (rows > pick ? rows : pick) : (sums > pick ? sums : pick);
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
    const dim3 segs((uint32_t)((int64_t)t.n_req * c.draw_segments)), reqs((uint32_t)t.n_req);
    hipError_t e = c.vecs == 8 ? launch(sample_rows_kernel<ESIZE, 8>, rows, dim3(kThreads), 0,
                                        stream, t, c, stats)
                               : launch(sample_rows_kernel<ESIZE, 2>, rows, dim3(kThreads), 0,
                                        stream, t, c, stats);
    if (e == hipSuccess)
        e = launch(sample_accept_kernel<ESIZE, QSIZE>, reqs, dim3(kAcceptWaves * 64), 0, stream, t,
                   c, stats, draws);
    if (e == hipSuccess)
        e = launch(sample_sums_kernel<ESIZE, QSIZE, false>, segs, dim3(kThreads), 0, stream, t, c,
                   draws, sums);
    if (e == hipSuccess && t.probs)
        e = launch(sample_sums_kernel<ESIZE, QSIZE, true>, segs, dim3(kThreads), 0, stream, t, c,
                   draws, sums);
    if (e == hipSuccess)
        e = launch(sample_pick_kernel<ESIZE, QSIZE>, reqs, dim3(kPickThreads), 0, stream, t, c,
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
