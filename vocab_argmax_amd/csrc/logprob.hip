// logprob.hip -- log probabilities of given tokens with entropy and the top
// alternatives, over one or several vocabulary shards, and their gradient.
//
// A set of columns is described by M = max x, s = sum 2^z and u = sum z 2^z
// with z = (x - M) log2(e), and two sets join as
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
#include "vpa_device.h"
#include "vpa_head_internal.h"
#include "vpa_math.h"

namespace vpa {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kVecs = 8;                          // 16-byte vectors per thread and chunk

constexpr int chunk_cols(int esize) {
    return kThreads * kVecs * (16 / esize);
}

constexpr float kNegInf = -__builtin_inff();

// (value, id) in the argmax order; 0 is below every real column.
__device__ __forceinline__ uint64_t order_of(float x, int32_t id) {
    return ((uint64_t)key_f32(__builtin_bit_cast(uint32_t, x)) << 32) | (uint32_t)~id;
}
__device__ __forceinline__ float value_of(uint64_t order) {
    const uint32_t key = (uint32_t)(order >> 32);
    if (key == kKeyNanF32)
        return __builtin_nanf("");
    if (key == kKeyZeroF32)
        return 0.0f;
    return __builtin_bit_cast(float, bits_of_key_f32(key));
}
__device__ __forceinline__ int32_t id_of(uint64_t order) {
    return (int32_t)~(uint32_t)order;
}

__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
        const uint64_t o = __shfl_xor((unsigned long long)v, off, 64);
        v = o > v ? o : v;
    }
    return v;
}

// M, s, u of a set of columns; the empty set is (-inf, 0, 0).
struct Sums {
    float m, s, u;
};
// (x - m) log2(e), held above -inf so that its product with 2^z = 0 is 0;
// a NaN stays.
__device__ __forceinline__ float scaled_distance(float x, float m) {
    const float z = (x - m) * kLog2e;
    return z < -1e30f ? -1e30f : z;
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
__device__ __forceinline__ Sums wave_join(Sums v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
        const Sums o = {__shfl_xor(v.m, off, 64), __shfl_xor(v.s, off, 64),
                        __shfl_xor(v.u, off, 64)};
        join(v, o);
    }
    return v;
}

// A chunk's partial result in the workspace: Sums of every chunk first, then
// the chunks' top lists.
__device__ __forceinline__ Sums* sums_of(void* ws) {
    return (Sums*)ws;
}
__host__ __device__ inline size_t sums_bytes(int64_t n) {
    return ((size_t)n * sizeof(Sums) + 255) / 256 * 256;
}

template <int ESIZE>
__global__ __launch_bounds__(kThreads) void logprob_part_kernel(LogprobTask t, int32_t chunks,
                                                                void* ws) {
    using T = typename elem<ESIZE>::type;
    constexpr int VEC = 16 / ESIZE;
    constexpr int N = kVecs * VEC;
    __shared__ float lds_m[kWaves];
    __shared__ Sums lds_s[kWaves];
    __shared__ uint64_t lds_top[2][kWaves];
    const int32_t chunk = blockIdx.x % chunks;
    const int32_t rest = blockIdx.x / chunks;
    const int32_t row = rest % t.n_rows, part = rest / t.n_rows;
    const int64_t first = t.col0 + part * t.part_stride;
    const int64_t end = first + t.part_width < t.vocab ? first + t.part_width : t.vocab;
    const int64_t lo = first + (int64_t)chunk * chunk_cols(ESIZE);
    const T* x = (const T*)t.logits + (int64_t)row * t.ld - t.col0;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;

    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int64_t c = lo + ((i / VEC) * kThreads + threadIdx.x) * VEC + i % VEC;
        v[i] = c < end ? to_f32(x[c]) : kNegInf;
    }
    float mx = kNegInf;
#pragma unroll
    for (int i = 0; i < N; ++i)
        mx = fmaxf(mx, v[i]);
    mx = wave_max(mx);
    if (lane == 0)
        lds_m[wave] = mx;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWaves; ++i)
        mx = fmaxf(mx, lds_m[i]);
    // a chunk of -inf alone: measured from 0, every term is 2^-1e30 = 0
    const float base = mx == kNegInf ? 0.0f : mx;
    float s = 0.0f, u = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float z = scaled_distance(v[i], base);
        const float e = exp2_fast(z);
        s += e;
        u += z * e;
    }
    s = wave_sum(s);
    u = wave_sum(u);
    if (lane == 0)
        lds_s[wave] = Sums{mx, s, u};
    __syncthreads();
    const int64_t slot = blockIdx.x;
    if (threadIdx.x == 0) {
        Sums r = lds_s[0];
        for (int i = 1; i < kWaves; ++i) {
            r.s += lds_s[i].s;
            r.u += lds_s[i].u;
        }
        sums_of(ws)[slot] = r;
    }
    if (t.n_top == 0)
        return;
    uint64_t* tops = (uint64_t*)((char*)ws + sums_bytes((int64_t)chunks * t.n_rows * t.n_parts)) +
                     slot * t.n_top;
    uint64_t below = ~0ull;
    for (int k = 0; k < t.n_top; ++k) {
        uint64_t best = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int64_t c = lo + ((i / VEC) * kThreads + threadIdx.x) * VEC + i % VEC;
            const uint64_t o = order_of(v[i], (int32_t)c);
            if (c < end && o < below && o > best)
                best = o;
        }
        best = wave_max_u64(best);
        if (lane == 0)
            lds_top[k & 1][wave] = best;
        __syncthreads();
        for (int i = 0; i < kWaves; ++i)
            best = lds_top[k & 1][i] > best ? lds_top[k & 1][i] : best;
        if (threadIdx.x == 0)
            tops[k] = best;
        below = best;
    }
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
    for (int j = threadIdx.x; j < o.n_tokens; j += 64) {
        const int32_t id = o.token_ids[row * o.n_tokens + j];
        float lp = __builtin_nanf("");
        if (id == -1)
            lp = 0.0f;
        else if (id >= 0 && id < vocab)
            lp = sc.logprob(logit(j, id));
        o.logprobs[row * o.n_tokens + j] = lp;
    }
}

// The n_top largest of n orders, one after the other, by one wavefront.
template <typename Order, typename Take>
__device__ __forceinline__ void select_top(int64_t n, int32_t n_top, Order order, Take take) {
    uint64_t below = ~0ull;
    for (int k = 0; k < n_top; ++k) {
        uint64_t best = 0;
        for (int64_t i = threadIdx.x; i < n; i += 64) {
            const uint64_t o = order(i);
            if (o < below && o > best)
                best = o;
        }
        best = wave_max_u64(best);
        if (threadIdx.x == 0)
            take(k, best);
        below = best;
    }
}

// One wavefront per (part, row): joins the chunks.
__device__ __forceinline__ Sums join_chunks(const void* ws, int64_t first, int32_t chunks) {
    Sums r = {kNegInf, 0.0f, 0.0f};
    for (int32_t c = threadIdx.x; c < chunks; c += 64)
        join(r, ((const Sums*)ws)[first + c]);
    return wave_join(r);
}

template <int ESIZE>
__global__ __launch_bounds__(64) void logprob_finish_kernel(LogprobTask t, int32_t chunks,
                                                            const void* ws, LogprobOut o) {
    using T = typename elem<ESIZE>::type;
    const int64_t row = blockIdx.x;
    const Sums r = join_chunks(ws, row * chunks, chunks);
    const T* x = (const T*)t.logits + row * t.ld - t.col0;
    const RowScale sc = scale_of(r);
    write_row(r, sc, row, t.vocab, o, [&](int, int32_t id) { return to_f32(x[id]); });
    if (t.n_top == 0)
        return;
    const uint64_t* tops =
        (const uint64_t*)((const char*)ws + sums_bytes((int64_t)chunks * t.n_rows * t.n_parts)) +
        row * chunks * t.n_top;
    select_top((int64_t)chunks * t.n_top, t.n_top, [&](int64_t i) { return tops[i]; },
               [&](int k, uint64_t best) {
                   o.top_ids[row * t.n_top + k] = id_of(best);
                   o.top_logprobs[row * t.n_top + k] = sc.logprob(value_of(best));
               });
}

template <int ESIZE>
__global__ __launch_bounds__(64) void logprob_record_kernel(LogprobTask t, int32_t chunks,
                                                            const void* ws,
                                                            const int32_t* token_ids,
                                                            int32_t n_tokens, int32_t* stats) {
    using T = typename elem<ESIZE>::type;
    const int64_t slot = blockIdx.x;
    const int64_t row = slot % t.n_rows, part = slot / t.n_rows;
    int32_t* rec = stats + slot * (3 + n_tokens + 2 * t.n_top);
    const Sums r = join_chunks(ws, slot * chunks, chunks);
    if (threadIdx.x == 0) {
        rec[0] = __builtin_bit_cast(int32_t, r.m);
        rec[1] = __builtin_bit_cast(int32_t, r.s);
        rec[2] = __builtin_bit_cast(int32_t, r.u);
    }
    const int64_t first = t.col0 + part * t.part_stride;
    const int64_t end = first + t.part_width < t.vocab ? first + t.part_width : t.vocab;
    const T* x = (const T*)t.logits + row * t.ld - t.col0;
    for (int j = threadIdx.x; j < n_tokens; j += 64) {
        const int32_t id = token_ids[row * n_tokens + j];
        const float v = id >= first && id < end ? to_f32(x[id]) : 0.0f;
        rec[3 + j] = __builtin_bit_cast(int32_t, v);
    }
    if (t.n_top == 0)
        return;
    const uint64_t* tops =
        (const uint64_t*)((const char*)ws + sums_bytes((int64_t)chunks * t.n_rows * t.n_parts)) +
        slot * chunks * t.n_top;
    select_top((int64_t)chunks * t.n_top, t.n_top, [&](int64_t i) { return tops[i]; },
               [&](int k, uint64_t best) {
                   int32_t* p = rec + 3 + n_tokens + 2 * k;
                   p[0] = best ? __builtin_bit_cast(int32_t, value_of(best))
                               : (int32_t)VPA_EMPTY_BITS;
                   p[1] = best ? id_of(best) : VPA_EMPTY_ID;
               });
}

__global__ __launch_bounds__(64) void logprob_combine_kernel(const int32_t* stats,
                                                             int32_t n_shards,
                                                             int64_t shard_width, int32_t vocab,
                                                             int32_t n_rows, int32_t n_top,
                                                             LogprobOut o) {
    const int64_t row = blockIdx.x;
    const int64_t words = 3 + o.n_tokens + 2 * (int64_t)n_top;
    const int32_t* rec = stats + row * words;
    const int64_t step = n_rows * words;           // from shard to shard
    Sums r = {kNegInf, 0.0f, 0.0f};
    for (int32_t s = threadIdx.x; s < n_shards; s += 64) {
        const int32_t* p = rec + s * step;
        join(r, Sums{__builtin_bit_cast(float, p[0]), __builtin_bit_cast(float, p[1]),
                     __builtin_bit_cast(float, p[2])});
    }
    r = wave_join(r);
    const RowScale sc = scale_of(r);
    write_row(r, sc, row, vocab, o, [&](int j, int32_t id) {
        return __builtin_bit_cast(float, rec[(id / shard_width) * step + 3 + j]);
    });
    const int32_t* top0 = rec + 3 + o.n_tokens;
    select_top((int64_t)n_shards * n_top, n_top,
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

// grad_c = sum_j g_j [c = t_j] - p_c (G + gH (log p_c + H)), G = sum_j g_j.
// A workgroup writes one chunk of a row without the given tokens' own terms,
// then the few elements that have them, from logits read before the chunk
// was written (the gradient may replace the logits).  Equal tokens all write
// the same sum.
template <int ESIZE>
__global__ __launch_bounds__(kThreads) void logprob_grad_kernel(LogprobGradTask t,
                                                                int32_t chunks) {
    using T = typename elem<ESIZE>::type;
    constexpr int VEC = 16 / ESIZE;
    const int64_t row = blockIdx.x / chunks;
    const int64_t lo = (int64_t)(blockIdx.x % chunks) * chunk_cols(ESIZE);
    const int64_t hi = lo + chunk_cols(ESIZE) < t.grad_cols ? lo + chunk_cols(ESIZE) : t.grad_cols;
    const T* x = (const T*)t.logits + row * t.ld;
    T* d = (T*)t.grad + row * t.grad_ld;
    const float max = t.row_stats[3 * row], log_sum = t.row_stats[3 * row + 1];
    const float h = t.row_stats[3 * row + 2];
    const bool empty = max == kNegInf && log_sum == 0.0f;
    const float gh = t.grad_entropy ? t.grad_entropy[row] : 0.0f;
    const int32_t* tok = t.token_ids + row * t.n_tokens;
    const float* g = t.grad_logprobs + row * t.n_tokens;
    float sum = 0.0f;
    for (int j = 0; j < t.n_tokens; ++j)
        sum += tok[j] >= 0 && tok[j] < t.vocab ? g[j] : 0.0f;
    // -p (G + gH (log p + H))
    auto slope = [&](float v) {
        const float lp = (v - max) - log_sum;
        const float p = exp2f(lp * kLog2e);        // keeps p below 2^-126
        return empty || p == 0.0f ? 0.0f : -p * (sum + gh * (lp + h));
    };
    // this workgroup's given token, one a thread
    const int32_t mine = threadIdx.x < (uint32_t)t.n_tokens ? tok[threadIdx.x] : -1;
    const int64_t at = (int64_t)mine - t.col0;
    const bool here = mine >= 0 && mine < t.vocab && at >= lo && at < hi && at < t.cols;
    const float own = here ? to_f32(x[at]) : 0.0f;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kVecs * VEC; ++i) {
        const int64_t c = lo + ((i / VEC) * kThreads + threadIdx.x) * VEC + i % VEC;
        if (c < hi)
            from_f32(d[c], c < t.cols ? slope(to_f32(x[c])) : 0.0f);
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

int32_t logprob_chunks(int esize, int64_t part_width, int64_t, int64_t) {
    return (int32_t)((part_width + chunk_cols(esize) - 1) / chunk_cols(esize));
}

size_t logprob_workspace(int64_t n_chunks, int64_t n_parts, int64_t n_rows, int32_t n_top) {
    const int64_t n = n_chunks * n_parts * n_rows;
    return sums_bytes(n) + ((size_t)n * n_top * 8 + 255) / 256 * 256;
}

int64_t logprob_threads(int64_t n_chunks, int64_t n_parts, int64_t n_rows) {
    return n_chunks * n_parts * n_rows * kThreads;
}

hipError_t launch_logprob_parts(int esize, const LogprobTask& t, void* ws, hipStream_t stream) {
    const int32_t chunks = logprob_chunks(esize, t.part_width, t.n_parts, t.n_rows);
    const dim3 grid((uint32_t)((int64_t)chunks * t.n_rows * t.n_parts));
    return esize == 2
               ? launch(logprob_part_kernel<2>, grid, dim3(kThreads), 0, stream, t, chunks, ws)
               : launch(logprob_part_kernel<4>, grid, dim3(kThreads), 0, stream, t, chunks, ws);
}

hipError_t launch_logprob_finish(int esize, const LogprobTask& t, const void* ws,
                                 const LogprobOut& o, hipStream_t stream) {
    const int32_t chunks = logprob_chunks(esize, t.part_width, t.n_parts, t.n_rows);
    const dim3 grid((uint32_t)t.n_rows);
    return esize == 2
               ? launch(logprob_finish_kernel<2>, grid, dim3(64), 0, stream, t, chunks, ws, o)
               : launch(logprob_finish_kernel<4>, grid, dim3(64), 0, stream, t, chunks, ws, o);
}

hipError_t launch_logprob_records(int esize, const LogprobTask& t, const void* ws,
                                  const int32_t* token_ids, int32_t n_tokens, int32_t* stats,
                                  hipStream_t stream) {
    const int32_t chunks = logprob_chunks(esize, t.part_width, t.n_parts, t.n_rows);
    const dim3 grid((uint32_t)((int64_t)t.n_rows * t.n_parts));
    return esize == 2 ? launch(logprob_record_kernel<2>, grid, dim3(64), 0, stream, t, chunks, ws,
                               token_ids, n_tokens, stats)
                      : launch(logprob_record_kernel<4>, grid, dim3(64), 0, stream, t, chunks, ws,
                               token_ids, n_tokens, stats);
}

hipError_t launch_logprob_combine(const int32_t* stats, int32_t n_shards, int64_t shard_width,
                                  int32_t vocab, int32_t n_rows, int32_t n_top,
                                  const LogprobOut& o, hipStream_t stream) {
    return launch(logprob_combine_kernel, dim3((uint32_t)n_rows), dim3(64), 0, stream, stats,
                  n_shards, shard_width, vocab, n_rows, n_top, o);
}

int64_t logprob_grad_threads(int esize, int64_t grad_cols, int64_t n_rows) {
    return (grad_cols + chunk_cols(esize) - 1) / chunk_cols(esize) * n_rows * kThreads;
}

hipError_t launch_logprob_grad(int esize, const LogprobGradTask& t, hipStream_t stream) {
    const int32_t chunks = (int32_t)((t.grad_cols + chunk_cols(esize) - 1) / chunk_cols(esize));
    const dim3 grid((uint32_t)((int64_t)chunks * t.n_rows));
    return esize == 2 ? launch(logprob_grad_kernel<2>, grid, dim3(kThreads), 0, stream, t, chunks)
                      : launch(logprob_grad_kernel<4>, grid, dim3(kThreads), 0, stream, t, chunks);
}

}  // namespace vpa
