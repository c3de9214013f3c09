// distill.hip -- the loss of a student's logits against a teacher's top tokens,
// and its gradient.
//
// A row's columns are summed in two sets, the named ones and the others, each
// as M near its maximum and s = sum exp((x - M) / t).  The others' sum is
// formed without the named columns, not by taking them off a total: a student
// that is sure of the teacher's tokens leaves so little to the others that the
// difference would have no digits.  With r(c) = exp((x_c - M_o) / t) / s_o the
// distribution over the others and q_0 their share, the gradient of a column
// not named is r(c) (q_0 P - p_0) / t: one exponential, and right where q(c)
// itself is too small for fp32.
#include <type_traits>

#include "row_scan.h"
#include "vpa_draft_internal.h"

namespace vpa {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMostSegments = 64;
constexpr float kInf = __builtin_inff();

// A row's statistics as the backward pass takes them.  (Of the sums 1 / s: from
// ln s in fp32 a probability would be off by half a step of ln s, 4e-7 for 2e5
// columns.)
struct DistillStats {
    float m_out, inv_out;      // of the columns not named (of all, without a tail)
    float f_out;               // q_0 P - p_0 (P, without a tail)
    float m, inv_s;            // of all columns
    float norm, log_norm;      // of the teacher: p_j = exp((l_j - norm) - log_norm)
    float mass;                // P; 0 where the gradient is 0
};
static_assert(sizeof(DistillStats) == VPA_DISTILL_STATS * sizeof(float), "as the header says");

// A row's named tokens, one a lane: the id (-1 for none) and log probability.
struct Named {
    int32_t id;
    float lp;
    bool bad;
};
__device__ __forceinline__ Named named_of(const DistillTask& t, int64_t row) {
    const int lane = threadIdx.x & 63;
    Named n{-1, -kInf, false};
    if (lane < t.n_top) {
        n.id = t.ids[row * t.n_top + lane];
        n.lp = t.logprobs[row * t.n_top + lane];
    }
    n.bad = n.id < -1 || n.id >= t.vocab || (n.id >= 0 && !(n.lp < kInf));
    if (n.id < 0 || n.id >= t.vocab)
        n.id = -1;
    return n;
}
// Calls f(lane, id) for each lane of `lanes`, in order.
template <typename F>
__device__ __forceinline__ void each_id(uint64_t lanes, int32_t id, F f) {
    for (; lanes; lanes &= lanes - 1) {
        const int j = (int)__builtin_ctzll(lanes);
        f(j, __builtin_amdgcn_readlane(id, j));
    }
}

// What the teacher says of a row, in every lane of a wavefront but p and lp,
// which are the lane's: the few terms in 64 bits, since what they leave of 1 may
// be small.
struct Teacher {
    double p, lp;
    double mass, left;         // sum p, and what it leaves (with a tail)
    float norm;
    double log_norm;
    bool has, bad;
};
__device__ __forceinline__ Teacher teacher_of(const DistillTask& t, const Named& n) {
    Teacher r;
    r.has = __ballot(n.id >= 0 || n.bad) != 0;
    r.bad = __ballot(n.bad) != 0;
    const float best = wave_max(n.id >= 0 ? n.lp : -kInf);
    r.norm = !t.tail && best > -kInf ? best : 0.0f;
    r.log_norm = 0.0;
    const double e = n.id >= 0 ? exp((double)n.lp - r.norm) : 0.0;
    const double sum = wave_sum_f64(e);
    r.lp = (double)n.lp - r.norm;
    r.p = e;
    r.mass = sum;
    if (!t.tail && best > -kInf) {
        r.log_norm = log(sum);
        r.lp -= r.log_norm;
        r.p = e / sum;
        r.mass = 1.0;
    }
    r.left = t.tail && r.mass < 1.0 ? 1.0 - r.mass : 0.0;
    return r;
}

// The loss and statistics of a row from the sums of its columns not named (of all
// columns without a tail), by one wavefront; v is the lane's named logit.  Every
// lane holds the statistics.
__device__ __forceinline__ DistillStats finish_row(const DistillTask& t, int64_t row, float v,
                                                   const Named& n, const Teacher& te,
                                                   ExpSum out) {
    const float scale = kLog2e / t.temperature;
    float m = out.m, s = out.s;
    if (t.tail) {
        bool first = n.id >= 0;                    // an id that is named twice counts once
        each_id(__ballot(first), n.id, [&](int j, int32_t id) {
            first = first && !(id == n.id && j < (int)(threadIdx.x & 63));
        });
        const float add = first ? v : -kInf;
        const float mx = fmaxf(m, wave_max(add));
        s = wave_sum(add == -kInf ? 0.0f : exp2_fast((add - mx) * scale)) +
            (mx == -kInf || m == mx ? s : s * exp2_fast((m - mx) * scale));
        m = mx;
    }
    const bool empty = m == -kInf && s == 0.0f;
    const bool bad = te.bad || !(s < kInf) || m == kInf;
    const double inv_t = 1.0 / (double)t.temperature;
    const double log_s = empty ? 0.0 : log((double)s);
    const double log_out = !t.tail ? log_s : out.s > 0.0f ? log((double)out.s) : 0.0;
    // log q of the named column, and of the others together
    const double lq = ((double)v - (double)m) * inv_t - log_s;
    const double lq0 =
        out.s > 0.0f ? ((double)out.m - (double)m) * inv_t + log_out - log_s : -INFINITY;
    double loss = wave_sum_f64(te.p > 0.0 ? te.p * (te.lp - lq) : 0.0);
    if (te.left > 0.0)
        loss += te.left * (log(te.left) - lq0);
    const double all = te.mass + te.left;
    DistillStats st;
    st.m_out = out.m == -kInf ? 0.0f : out.m;      // r of a masked column is 0
    st.inv_out = !t.tail ? 1.0f / s : out.s > 0.0f ? 1.0f / out.s : 0.0f;
    st.f_out = (float)(t.tail ? exp(lq0) * all - te.left : all);
    st.m = m;
    st.inv_s = 1.0f / s;
    st.norm = te.norm;
    st.log_norm = (float)te.log_norm;
    st.mass = (float)all;
    if (empty) {
        loss = all > 0.0 ? INFINITY : 0.0;
        st.mass = 0.0f;
    }
    if (bad) {
        loss = NAN;
        st.f_out = st.mass = NAN;
    }
    if (!te.has) {
        loss = 0.0;
        st.mass = 0.0f;
    }
    if ((threadIdx.x & 63) == 0) {
        t.loss[row] = (float)loss;
        *(DistillStats*)(t.row_stats + row * VPA_DISTILL_STATS) = st;
    }
    return st;
}
template <typename T>
__device__ __forceinline__ float named_logit(const T* x, const Named& n) {
    return n.id >= 0 ? to_f32(x[n.id]) : -kInf;
}

// Masks the named columns of a chunk: of THREADS threads with U vectors each,
// from column c0.  A wavefront does those of its own lanes, vector by vector and
// one at a time.
template <int ESIZE, int U, int THREADS>
__device__ __forceinline__ void mask_named(u32x4_t (&w)[U], int c0, int32_t id) {
    constexpr int VEC = 16 / ESIZE;
    const int at = id >= 0 ? id - c0 : -1;         // (>= 0: c0 may be below 0)
    const bool here = at >= 0 && at / VEC % THREADS / 64 == (int)threadIdx.x / 64;
    if (!__ballot(here && at < THREADS * U * VEC))
        return;
#pragma unroll
    for (int i = 0; i < U; ++i)
        each_id(__ballot(here && at / VEC / THREADS == i), at, [&](int, int32_t a) {
            mask_element<ESIZE>(w[i], a % VEC, a / VEC % 64);
        });
}

// How the loss's launch is cut: segments of whole chunks.
struct Cut {
    int32_t segments, chunks;
};

// A workgroup a segment of a row; with one segment, the whole of it.  Bound by
// reading: 512 x 50257 fp32 18 us, 1024 x 151936 bf16 54-56 (5.7-5.9 TB/s).  A chunk is 2
// vectors a thread (2048 x 50257 bf16 40.8 us, with 1 40.9, 4 41.5, 8 46.3; 8192 x
// 16000 57, 61, 58, 77; 64 x 151936 11.2, 11.6, 11.2, 12.1).
constexpr int kScanVecs = 2;

template <int ESIZE>
__global__ __launch_bounds__(kThreads) void distill_kernel(DistillTask t, Cut cut, ExpSum* sums) {
    using T = typename elem<ESIZE>::type;
    using Scan = SegmentScan<ESIZE, kScanVecs, kThreads, false>;
    __shared__ ExpSum lds[kWaves];
    const int64_t row = blockIdx.x / cut.segments;
    const int32_t seg = blockIdx.x % cut.segments;
    const T* x = (const T*)t.logits + row * t.ld;
    const float scale = kLog2e / t.temperature;
    const Named n = named_of(t, row);
    const int32_t id = t.tail ? n.id : -1;
    const int begin = -(int)(((uintptr_t)x & 15) / ESIZE) + seg * cut.chunks * Scan::CHUNK;
    const int end = begin + cut.chunks * Scan::CHUNK;
    const int lo = begin < 0 ? 0 : begin, hi = end < t.vocab ? end : t.vocab;
    Scan scan;
    scan.run(x, begin, lo, hi, scale, [&](u32x4_t (&w)[kScanVecs], int c0) {
        mask_named<ESIZE, kScanVecs, kThreads>(w, c0, id);
    });
    const ExpSum s = scan.wave();
    if ((threadIdx.x & 63) == 0)
        lds[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x >= 64)
        return;
    ExpSum all = lds[0];
#pragma unroll
    for (int i = 1; i < kWaves; ++i)
        all = join(all, lds[i], scale);
    if (cut.segments == 1)
        finish_row(t, row, named_logit(x, n), n, teacher_of(t, n), all);
    else if (threadIdx.x == 0)
        sums[blockIdx.x] = all;
}

// The segments' sums joined; a wavefront a row.  Bound by latency, of its loads and
// of the 64-bit logarithms: 4 us for 512 rows of 4 segments.
template <int ESIZE>
__global__ __launch_bounds__(64) void distill_finish_kernel(DistillTask t, Cut cut,
                                                            const ExpSum* sums) {
    using T = typename elem<ESIZE>::type;
    const int64_t row = blockIdx.x;
    ExpSum s = {kMinusInf, 0.0f};
    if ((int)threadIdx.x < cut.segments)
        s = sums[row * cut.segments + threadIdx.x];
    const Named n = named_of(t, row);
    const float v = named_logit((const T*)t.logits + row * t.ld, n);
    finish_row(t, row, v, n, teacher_of(t, n), wave_join(s, kLog2e / t.temperature));
}

// The gradient of a row: of its columns not named, r(c) f with r(c) = 2^z / s_o,
// and of the lane's named one.
struct Slope {
    float scale, f, g;
    ScaledFrom base;
    bool zero;
    __device__ __forceinline__ Slope(const DistillTask& t, int64_t row, const DistillStats& st) {
        scale = kLog2e / t.temperature;
        g = t.grad_loss[row] / t.temperature;
        zero = st.mass == 0.0f;
        base.set(st.m_out, scale);
        f = g * st.f_out * (st.inv_out * base.fix);
    }
    // 16 bytes of columns
    template <int ESIZE>
    __device__ __forceinline__ u32x4_t of(u32x4_t w) const {
        constexpr int VEC = 16 / ESIZE;
        u32x4_t o = {0, 0, 0, 0};
        if (zero)                                  // whatever the logits hold
            return o;
        float d[VEC];
        if (base.apart) {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                d[e] = exp2_fast((vec_elem<ESIZE>(w, e) - base.m) * scale) * f;
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                d[e] = exp2_fast(__builtin_fmaf(vec_elem<ESIZE>(w, e), scale, -base.b)) * f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = ESIZE == 2 ? pack_bf16(d[2 * i % VEC], d[(2 * i + 1) % VEC])
                              : __builtin_bit_cast(uint32_t, d[i]);
        return o;
    }
    // by a whole wavefront, for the lanes whose tokens are `here`, with logits v;
    // equal ids get the same sum
    __device__ __forceinline__ float named(const DistillStats& st, const Named& n, bool here,
                                           float v) const {
        const float mine = exp2f(((n.lp - st.norm) - st.log_norm) * kLog2e);
        float p = 0.0f;
        each_id(__ballot(here), n.id, [&](int j, int32_t id) {
            const float other = __builtin_bit_cast(
                float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, mine), j));
            p += id == n.id ? other : 0.0f;
        });
        const float q = exp2f((v - st.m) * scale) * st.inv_s;
        return zero ? 0.0f : g * (q * st.mass - p);
    }
};

constexpr int kGradVecs = 4;                       // 16-byte vectors a thread
constexpr int grad_chunk(int esize) {
    return kThreads * kGradVecs * (16 / esize);
}

// The gradient of one chunk of a row: every column as one that is not named,
// then the named ones, from logits read before the chunk was written (the
// gradient may replace the logits).  A workgroup's stores keep their order, so
// what the first wavefront stores after the barrier is what stays.  Bound by
// memory: 1024 x 151936 bf16 107 us, 5.8 TB/s read and written.
template <int ESIZE>
__global__ __launch_bounds__(kThreads) void distill_grad_kernel(DistillTask t, int32_t chunks) {
    using T = typename elem<ESIZE>::type;
    constexpr int VEC = 16 / ESIZE;
    constexpr int CHUNK = grad_chunk(ESIZE);
    const int64_t row = blockIdx.x / chunks;
    const int64_t lo = (int64_t)(blockIdx.x % chunks) * CHUNK;
    const int64_t hi = lo + CHUNK < t.grad_cols ? lo + CHUNK : t.grad_cols;
    const T* x = (const T*)t.logits + row * t.ld;
    T* d = (T*)t.grad + row * t.grad_ld;
    u32x4_t w[kGradVecs];
#pragma unroll
    for (int i = 0; i < kGradVecs; ++i) {
        const int64_t c = lo + (i * kThreads + threadIdx.x) * VEC;
        if (c + VEC <= t.vocab)
            w[i] = ((const Loose16*)(x + c))->v;
        else
            w[i] = load_columns<ESIZE>(x, (int)c, 0, t.vocab);
    }
    const DistillStats st = *(const DistillStats*)(t.row_stats + row * VPA_DISTILL_STATS);
    const Slope sl(t, row, st);
    // this workgroup's named columns, one a lane of the first wavefront
    float own = 0.0f;
    int64_t at = -1;
    if (threadIdx.x < 64) {
        const Named n = named_of(t, row);
        const bool here = n.id >= lo && n.id < hi;
        if (__ballot(here)) {
            own = sl.named(st, n, here, here ? to_f32(x[n.id]) : 0.0f);
            at = here ? n.id : -1;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kGradVecs; ++i) {
        const int64_t c = lo + (i * kThreads + threadIdx.x) * VEC;
        if (c < t.vocab)
            store_columns<ESIZE>(d, (int)c, 0, t.vocab, sl.of<ESIZE>(w[i]));
        if (c + VEC > t.vocab)
#pragma unroll 1
            for (int64_t z = c > t.vocab ? c : t.vocab; z < c + VEC && z < hi; ++z)
                from_f32(d[z], 0.0f);
    }
    __syncthreads();
    if (at >= 0)
        from_f32(d[at], own);
}

// Loss and gradient of a row that a workgroup holds in registers, NV vectors a
// lane: the logits are read once.  Bound by memory: 2048 x 50257 bf16 89 us, 4.8
// TB/s read and written, where a large copy has 4.9; the two passes of rows that
// are read twice have more bandwidth and a third more bytes (121 us).
template <int ESIZE, int NV, int THREADS>
__global__ __launch_bounds__(THREADS) void distill_row_kernel(DistillTask t) {
    using T = typename elem<ESIZE>::type;
    constexpr int VEC = 16 / ESIZE;
    constexpr int ROW_WAVES = THREADS / 64;
    __shared__ float lds_m[ROW_WAVES], lds_s[ROW_WAVES];
    __shared__ DistillStats lds_st;
    __shared__ Teacher lds_te[64];                 // registers are short
    const int64_t row = blockIdx.x;
    const T* x = (const T*)t.logits + row * t.ld;
    T* d = (T*)t.grad + row * t.grad_ld;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const float scale = kLog2e / t.temperature;
    const int begin = -(int)(((uintptr_t)x & 15) / ESIZE);
    const int mine = begin + (int)threadIdx.x * VEC;
    // whether all of the workgroup's i-th vectors are columns of the row
    const auto whole = [&](int i) {
        return (i > 0 || begin == 0) && begin + (i + 1) * THREADS * VEC <= t.vocab;
    };
    u32x4_t w[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = mine + i * THREADS * VEC;
        if (whole(i))
            w[i] = __builtin_nontemporal_load((const u32x4_t*)(x + c));
        else
            w[i] = load_columns<ESIZE>(x, c, 0, t.vocab);
    }
    const Named n = named_of(t, row);
    const float v = named_logit(x, n);
    if (wave == 0)
        lds_te[lane] = teacher_of(t, n);
    // the named columns stay out of the sums; their own slopes are stored at the end
    if (t.tail)
        mask_named<ESIZE, NV, THREADS>(w, begin, n.id);
    float m = kMinusInf;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        m = fmaxf(m, vec_largest<ESIZE>(w[i]));
    m = wave_max(m);
    if (lane == 0)
        lds_m[wave] = m;
    __syncthreads();
    m = wave_max(lds_m[lane % ROW_WAVES]);
    ScaledFrom base;
    base.set(m == kMinusInf ? 0.0f : m, scale);
#pragma unroll
    for (int i = 0; i < NV; ++i)
        asm volatile("" : "+v"(w[i]));
    const float s = wave_sum(chunk_sum<ESIZE, NV>(w, base, scale));
    if (lane == 0)
        lds_s[wave] = s;
    __syncthreads();
    if (wave == 0) {
        const float all = wave_sum(lane < ROW_WAVES ? lds_s[lane] : 0.0f);
        const DistillStats st = finish_row(t, row, v, n, lds_te[lane], ExpSum{m, all});
        if (lane == 0)
            lds_st = st;
    }
    __syncthreads();
    const DistillStats st = lds_st;
    const Slope sl(t, row, st);
    float own = 0.0f;
    if (wave == 0)
        own = sl.named(st, n, n.id >= 0, v);
#pragma unroll
    for (int i = 0; i < NV; ++i)
        asm volatile("" : "+v"(w[i]));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = mine + i * THREADS * VEC;
        const u32x4_t o = sl.of<ESIZE>(w[i]);
        if (whole(i))
            __builtin_nontemporal_store(o, &((Loose16*)(d + c))->v);   // past the L2
        else
            store_columns<ESIZE>(d, c, 0, t.vocab, o);
        __builtin_amdgcn_sched_barrier(0);
    }
    for (int64_t c = t.vocab + threadIdx.x; c < t.grad_cols; c += THREADS)
        from_f32(d[c], 0.0f);
    __syncthreads();
    if (wave == 0 && n.id >= 0)
        from_f32(d[n.id], own);
}

// Segments of whole chunks until there are 8 workgroups a CU (64 x 151936 bf16 11.2
// us, with 4 a CU 11.9, with 16 11.5); whole rows where those alone are 4 a CU (1024
// x 200064 fp32 123 us, in two segments 130; the launch that joins them is saved).
Cut distill_cut(int esize, int64_t vocab, int64_t n_rows) {
    Cut c;
    const int64_t vec = 16 / esize, width = vocab + vec - 1;
    const int64_t chunk = kThreads * kScanVecs * vec, chunks = (width + chunk - 1) / chunk;
    int64_t want = n_rows >= 1024 ? 1 : (2048 + n_rows - 1) / n_rows;
    want = want > chunks ? chunks : want;
    want = want > kMostSegments ? kMostSegments : want;
    c.chunks = (int32_t)((chunks + want - 1) / want);
    c.segments = (int32_t)((chunks + c.chunks - 1) / c.chunks);
    return c;
}

// Threads and vectors a lane that hold a row of `vocab` columns (one vector more
// for what lies before the first aligned column); 0 where a row is too long.
struct RowForm {
    int threads, vectors;
};
RowForm row_form(int esize, int64_t vocab) {
    const int64_t vec = 16 / esize, need = (vocab + vec - 1 + vec - 1) / vec;
    constexpr RowForm forms[] = {{256, 1}, {256, 4}, {256, 8}, {512, 7},
                                 {512, 13}, {1024, 10}, {1024, 14}, {1024, 20}};
    for (const RowForm& f : forms)
        if (need <= f.threads * f.vectors)
            return f;
    return {0, 0};
}

// Whether a call takes its rows whole: up to 64 KB (32 x 28000 bf16 10.4 us, in two
// launches 12.1; 8 x 1000 8.3 and 11.0; 8192 x 16000 105 and 178).  Longer ones leave
// most of the chip idle where they are few: from 64 rows on with 512 threads (50257
// columns, 16 rows 13.7 and 12.2, 64 14.6 and 15.3, 2048 90 and 121), from 128 on
// with 1024 (151936 columns, 64 rows 31.7 and 19.0, 128 33.3 and 32.7, 256 42.8 and
// 51.1, 1024 163 and 168; 100000 columns, 96 rows 21.2 and 19.1, 128 21.5 and 22.4).
bool rows_whole(RowForm f, int64_t n_rows) {
    return f.threads != 0 && (f.threads * f.vectors <= 4096 || n_rows >= f.threads / 8);
}

size_t sums_bytes(const Cut& c, int64_t n_rows) {
    return c.segments == 1 ? 0 : (size_t)n_rows * c.segments * sizeof(ExpSum);
}

}  // namespace

size_t distill_workspace(int64_t vocab, int64_t n_rows) {
    const size_t b2 = sums_bytes(distill_cut(2, vocab, n_rows), n_rows);
    const size_t b4 = sums_bytes(distill_cut(4, vocab, n_rows), n_rows);
    return b2 > b4 ? b2 : b4;
}

int64_t distill_threads(int esize, int64_t vocab, int64_t n_rows) {
    const int64_t cut = n_rows * distill_cut(esize, vocab, n_rows).segments * kThreads;
    const RowForm f = row_form(esize, vocab);
    const int64_t rows = rows_whole(f, n_rows) ? n_rows * f.threads : 0;
    return cut > rows ? cut : rows;
}

int64_t distill_grad_threads(int esize, int64_t grad_cols, int64_t n_rows) {
    const int64_t chunk = grad_chunk(esize);
    return (grad_cols + chunk - 1) / chunk * n_rows * kThreads;
}

namespace {

template <int ESIZE>
hipError_t launch_loss(const DistillTask& t, void* ws, hipStream_t stream) {
    const Cut c = distill_cut(ESIZE, t.vocab, t.n_rows);
    const dim3 grid((uint32_t)((int64_t)t.n_rows * c.segments)), block(kThreads);
    ExpSum* sums = (ExpSum*)ws;
    const hipError_t e = launch(distill_kernel<ESIZE>, grid, block, 0, stream, t, c, sums);
    if (e != hipSuccess || c.segments == 1)
        return e;
    return launch(distill_finish_kernel<ESIZE>, dim3((uint32_t)t.n_rows), dim3(64), 0, stream, t, c,
                  sums);
}

template <int ESIZE>
hipError_t launch_rows(const DistillTask& t, RowForm f, hipStream_t stream) {
    const dim3 grid((uint32_t)t.n_rows), block((uint32_t)f.threads);
    if (f.threads == 256) {
        if (f.vectors == 1)
            return launch(distill_row_kernel<ESIZE, 1, 256>, grid, block, 0, stream, t);
        return f.vectors == 4 ? launch(distill_row_kernel<ESIZE, 4, 256>, grid, block, 0, stream, t)
                              : launch(distill_row_kernel<ESIZE, 8, 256>, grid, block, 0, stream, t);
    }
    if (f.threads == 512) {
        if (f.vectors == 7)
            return launch(distill_row_kernel<ESIZE, 7, 512>, grid, block, 0, stream, t);
        return launch(distill_row_kernel<ESIZE, 13, 512>, grid, block, 0, stream, t);
    }
    if (f.vectors == 10)
        return launch(distill_row_kernel<ESIZE, 10, 1024>, grid, block, 0, stream, t);
    return f.vectors == 14 ? launch(distill_row_kernel<ESIZE, 14, 1024>, grid, block, 0, stream, t)
                           : launch(distill_row_kernel<ESIZE, 20, 1024>, grid, block, 0, stream, t);
}

}  // namespace

hipError_t launch_distill(int esize, const DistillTask& t, void* ws, hipStream_t stream) {
    return esize == 2 ? launch_loss<2>(t, ws, stream) : launch_loss<4>(t, ws, stream);
}

hipError_t launch_distill_grad(int esize, const DistillTask& t, hipStream_t stream) {
    const int64_t chunk = grad_chunk(esize);
    const int32_t chunks = (int32_t)((t.grad_cols + chunk - 1) / chunk);
    const dim3 grid((uint32_t)((int64_t)chunks * t.n_rows)), block(kThreads);
    return esize == 2 ? launch(distill_grad_kernel<2>, grid, block, 0, stream, t, chunks)
                      : launch(distill_grad_kernel<4>, grid, block, 0, stream, t, chunks);
}

hipError_t launch_distill_both(int esize, const DistillTask& t, void* ws, hipStream_t stream) {
    const RowForm f = row_form(esize, t.vocab);
    if (rows_whole(f, t.n_rows))
        return esize == 2 ? launch_rows<2>(t, f, stream) : launch_rows<4>(t, f, stream);
    const hipError_t e = launch_distill(esize, t, ws, stream);
    return e != hipSuccess ? e : launch_distill_grad(esize, t, stream);
}

}  // namespace vpa
