// sampled.hip -- verification of drafted tokens against the target's
// probabilities, from given random numbers.
//
// Five steps: every row's maximum, sum of exponentials and argmax; a request's
// acceptance tests, which give the row it draws from; that row's sum of
// exponentials in 64 bits (where a draft distribution is subtracted); the sums
// of its weights; the column where the running sum passes the random number.
// The draw is in 64 bits because a border lies between any two of up to 2^24
// columns: with sums that are off by 2^-24 one draw in a hundred over a flat
// row of 2e5 columns would come out a column off.
#include "vpa_draft_internal.h"
#include "vpa_math.h"

namespace vpa {
namespace {

constexpr int kThreads = 256;

// A row's statistics: m near the largest logit, s = sum exp((x - m) / T), and
// the first column in the argmax order.  s is NaN where the row holds a NaN or
// +inf; m = -inf where nothing is finite.
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

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1)
        v += __shfl_xor(v, off, 64);
    return v;
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

template <int ESIZE>
__global__ __launch_bounds__(kThreads) void sample_rows_kernel(SampleTask t, RowStat* stats) {
    using T = typename elem<ESIZE>::type;
    __shared__ float lds_m[4], lds_s[4];
    __shared__ uint64_t lds_o[4];
    const int32_t row = blockIdx.x, req = row / (t.k + 1), pos = row % (t.k + 1);
    // rows after a placeholder are not needed
    for (int j = 0; j < pos; ++j)
        if (!is_draft(t, t.draft_ids[(int64_t)req * t.k + j]))
            return;
    const T* x = (const T*)t.logits + (int64_t)row * t.ld;
    const float temp = temperature_of(t, req);
    const float scale = is_greedy(temp) ? kLog2e : kLog2e / temp;
    float m = -__builtin_inff(), s = 0.0f;
    uint64_t best = 0;
    for (int c = threadIdx.x; c < t.vocab; c += kThreads) {
        const uint64_t o = order_of(to_f32(x[c]), c);
        best = o > best ? o : best;
    }
    best = wave_max_u64(best);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (lane == 0)
        lds_o[wave] = best;
    __syncthreads();
    for (int i = 0; i < 4; ++i)
        best = lds_o[i] > best ? lds_o[i] : best;
    m = value_of(best);
    if (m > -__builtin_inff())
        for (int c = threadIdx.x; c < t.vocab; c += kThreads)
            s += exp2_fast((to_f32(x[c]) - m) * scale);
    s = wave_sum(s);
    if (lane == 0)
        lds_s[wave] = s;
    __syncthreads();
    if (threadIdx.x == 0)
        stats[row] = RowStat{m, lds_s[0] + lds_s[1] + lds_s[2] + lds_s[3], best};
    (void)lds_m;
}

template <int ESIZE, int QSIZE>
__global__ __launch_bounds__(64) void sample_accept_kernel(SampleTask t, const RowStat* stats,
                                                           Draw* draws) {
    using T = typename elem<ESIZE>::type;
    using Q = typename elem<QSIZE>::type;
    const int32_t req = blockIdx.x;
    if (threadIdx.x != 0)
        return;
    const float temp = temperature_of(t, req);
    Draw d{};
    d.kind = kPlain;
    d.scale = 1.4426950408889634074 / (double)temp;
    int pos = 0;
    int32_t greedy_id = 0;
    bool greedy = false;
    for (;; ++pos) {
        const int32_t row = req * (t.k + 1) + pos;
        const RowStat st = stats[row];
        d.row = row;
        d.m = st.m;
        greedy = is_greedy(temp) || !(fabsf(st.m) < __builtin_inff()) || !(st.s < __builtin_inff());
        greedy_id = id_of(st.order);
        if (pos == t.k)
            break;
        const int32_t id = t.draft_ids[(int64_t)req * t.k + pos];
        if (!is_draft(t, id))
            break;
        double p;
        if (greedy)
            p = id == greedy_id ? 1.0 : 0.0;
        else
            p = exp2(((double)to_f32(((const T*)t.logits)[(int64_t)row * t.ld + id]) - st.m) *
                     d.scale) / (double)st.s;
        const int64_t q_row = (int64_t)req * t.k + pos;
        const double q = t.probs ? (double)to_f32(((const Q*)t.probs)[q_row * t.ldq + id]) : 1.0;
        if ((double)t.accept_u[q_row] * q < p)
            continue;
        d.kind = t.probs ? kMinus : kWithout;
        d.q_row = (int32_t)q_row;
        d.id = id;
        break;
    }
    d.pos = pos;
    int32_t* out = t.out_tokens + (int64_t)req * (t.k + 1);
    for (int j = 0; j <= t.k; ++j)
        out[j] = j < pos ? t.draft_ids[(int64_t)req * t.k + j] : -1;
    if (greedy) {
        out[pos] = greedy_id;
        d.kind = kDrawn;
    }
    t.num_sampled[req] = pos + 1;
    t.num_rejected[req] = t.k - pos;
    draws[req] = d;
}

// exp((x - m) / T) in 64 bits.
template <typename T>
__device__ __forceinline__ double weight(T x, const Draw& d) {
    return exp2(((double)to_f32(x) - (double)d.m) * d.scale);
}

template <int ESIZE, int QSIZE>
__global__ __launch_bounds__(kThreads) void sample_draw_kernel(SampleTask t, const Draw* draws) {
    using T = typename elem<ESIZE>::type;
    using Q = typename elem<QSIZE>::type;
    __shared__ double sums[4];
    __shared__ int32_t found;
    const int32_t req = blockIdx.x;
    const Draw d = draws[req];
    if (d.kind == kDrawn)
        return;
    const T* x = (const T*)t.logits + (int64_t)d.row * t.ld;
    const Q* q = (const Q*)t.probs + (int64_t)d.q_row * t.ldq;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    auto total = [&](auto f) {
        double s = 0.0;
        for (int c = threadIdx.x; c < t.vocab; c += kThreads)
            s += f(c);
        s = wave_sum_f64(s);
        __syncthreads();
        if (lane == 0)
            sums[wave] = s;
        __syncthreads();
        return ((sums[0] + sums[1]) + sums[2]) + sums[3];
    };
    auto plain = [&](int c) { return weight(x[c], d); };
    const double z = d.kind == kMinus ? total(plain) : 0.0;
    int32_t kind = d.kind;
    auto w = [&](int c) {
        const double e = plain(c);
        if (kind == kWithout)
            return c == d.id ? 0.0 : e;
        if (kind == kMinus) {
            const double r = e - (double)to_f32(q[c]) * z;
            return r > 0.0 ? r : 0.0;
        }
        return e;
    };
    double all = total(w);
    if (!(all > 0.0)) {
        kind = kPlain;
        all = total(w);
    }
    const double u = t.sample_u[req];
    const double target = (u > 0.0 ? u : 0.0) * all;
    // the running sum, a workgroup's columns at a time
    double before = 0.0;
    int32_t last = 0;
    if (threadIdx.x == 0)
        found = t.vocab;
    for (int c0 = 0; c0 < t.vocab; c0 += kThreads) {
        const int c = c0 + threadIdx.x;
        const double mine = c < t.vocab ? w(c) : 0.0;
        double run = mine;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const double o = __shfl_up(run, off, 64);
            run += lane >= off ? o : 0.0;
        }
        __syncthreads();
        if (lane == 63)
            sums[wave] = run;
        __syncthreads();
        double mine_before = before;
        for (int i = 0; i < wave; ++i)
            mine_before += sums[i];
        if (mine > 0.0 && mine_before + run > target)
            atomicMin(&found, c);
        last = mine > 0.0 ? c : last;
        before += ((sums[0] + sums[1]) + sums[2]) + sums[3];
        __syncthreads();
        if (found < t.vocab)
            break;
    }
    int32_t token = found;
    if (token == t.vocab) {
        __syncthreads();
        if (threadIdx.x == 0)
            found = 0;
        __syncthreads();
        atomicMax(&found, last);
        __syncthreads();
        token = found;
    }
    if (threadIdx.x == 0)
        t.out_tokens[(int64_t)req * (t.k + 1) + d.pos] = token;
}

size_t align16(size_t n) {
    return (n + 15) / 16 * 16;
}

}  // namespace

SampleCut sample_cut(int64_t, int64_t, int32_t) {
    return SampleCut{1, 1};
}

size_t sample_workspace(const SampleCut& c, int64_t n_req, int32_t k) {
    return align16((size_t)n_req * (k + 1) * c.row_segments * sizeof(RowStat)) +
           (size_t)n_req * sizeof(Draw);
}

int64_t sample_threads(const SampleCut& c, int64_t n_req, int32_t k) {
    return n_req * (k + 1) * c.row_segments * kThreads;
}

namespace {

template <int ESIZE, int QSIZE>
hipError_t launch_typed(const SampleTask& t, void* ws, hipStream_t stream) {
    const int64_t rows = (int64_t)t.n_req * (t.k + 1);
    RowStat* stats = (RowStat*)ws;
    Draw* draws = (Draw*)((char*)ws + align16((size_t)rows * sizeof(RowStat)));
    hipError_t e = launch(sample_rows_kernel<ESIZE>, dim3((uint32_t)rows), dim3(kThreads), 0,
                          stream, t, stats);
    if (e == hipSuccess)
        e = launch(sample_accept_kernel<ESIZE, QSIZE>, dim3((uint32_t)t.n_req), dim3(64), 0, stream,
                   t, stats, draws);
    if (e == hipSuccess)
        e = launch(sample_draw_kernel<ESIZE, QSIZE>, dim3((uint32_t)t.n_req), dim3(kThreads), 0,
                   stream, t, draws);
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
