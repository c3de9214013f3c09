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
#include "vpa_draft_internal.h"
#include "vpa_math.h"

namespace vpa {
namespace {

constexpr int kThreads = 256;
constexpr float kInf = __builtin_inff();

// A row's statistics as the backward pass takes them.
struct DistillStats {
    float m_out, log_out;      // of the columns not named (of all, without a tail)
    float f_out;               // q_0 P - p_0 (P, without a tail)
    float m, log_s;            // of all columns
    float norm, log_norm;      // of the teacher: p_j = exp((l_j - norm) - log_norm)
    float mass;                // P; 0 where the gradient is 0
};
static_assert(sizeof(DistillStats) == VPA_DISTILL_STATS * sizeof(float), "as the header says");

// A row's named tokens, one a lane: the id (-1 for none), log probability, and
// whether the lane is the first with its id.
struct Named {
    int32_t id;
    float lp;
    bool first, bad;
};
__device__ __forceinline__ Named named_of(const DistillTask& t, int64_t row) {
    const int lane = threadIdx.x & 63;
    Named n{-1, -kInf, false, false};
    if (lane < t.n_top) {
        n.id = t.ids[row * t.n_top + lane];
        n.lp = t.logprobs[row * t.n_top + lane];
    }
    n.bad = n.id < -1 || n.id >= t.vocab || (n.id >= 0 && !(n.lp < kInf));
    if (n.id < 0 || n.id >= t.vocab)
        n.id = -1;
    n.first = n.id >= 0;
    for (int j = 0; j < t.n_top; ++j) {
        const int32_t other = __builtin_amdgcn_readlane(n.id, j);
        n.first = n.first && !(j < lane && other == n.id);
    }
    return n;
}

// (m, s) of a set of columns; the empty set is (-inf, 0).
__device__ __forceinline__ void join(float& m, float& s, float om, float os, float scale) {
    const float mx = fmaxf(m, om);
    if (mx == -kInf)
        return;                            // (a NaN in s stays)
    s = s * exp2_fast((m - mx) * scale) + os * exp2_fast((om - mx) * scale);
    m = mx;
}

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1)
        v += __shfl_xor(v, off, 64);
    return v;
}

// The loss and statistics of a row from (m, s) of its columns not named (of all
// columns without a tail), by one wavefront.
template <typename T>
__device__ __forceinline__ void finish_row(const DistillTask& t, int64_t row, const T* x,
                                           const Named& n, float m_out, float s_out) {
    const float scale = kLog2e / t.temperature;
    const float v = n.id >= 0 ? to_f32(x[n.id]) : -kInf;
    float m = m_out, s = s_out;
    if (t.tail) {
        const float add = n.first ? v : -kInf;
        const float mx = fmaxf(m_out, wave_max(add));
        const float in = add == -kInf ? 0.0f : exp2_fast((add - mx) * scale);
        s = wave_sum(in);
        m = mx;
        if (mx > -kInf)
            s += m_out == -kInf ? s_out : s_out * exp2_fast((m_out - mx) * scale);
        else
            s += s_out;
    }
    // the teacher's few terms in 64 bits: what they leave of 1 may be small
    const bool has = __ballot(n.id >= 0 || n.bad) != 0;
    const bool empty = m == -kInf && s == 0.0f;
    const bool bad = __ballot(n.bad) != 0 || !(s < kInf) || m == kInf;
    const float best = wave_max(n.id >= 0 ? n.lp : -kInf);
    const float norm = !t.tail && best > -kInf ? best : 0.0f;
    double log_norm = 0.0;
    if (!t.tail && best > -kInf)
        log_norm = log(wave_sum_f64(n.id >= 0 ? exp((double)n.lp - norm) : 0.0));
    const double lp = ((double)n.lp - norm) - log_norm;
    const double p = n.id >= 0 ? exp(lp) : 0.0;
    const double mass = wave_sum_f64(p);
    const double left = t.tail && mass < 1.0 ? 1.0 - mass : 0.0;
    const double inv_t = 1.0 / (double)t.temperature;
    const double log_s = empty ? 0.0 : log((double)s);
    const double log_out = s_out > 0.0f ? log((double)s_out) : 0.0;
    // log q of the named column, and of the others together
    const double lq = ((double)v - (double)m) * inv_t - log_s;
    const double lq0 = s_out > 0.0f ? ((double)m_out - (double)m) * inv_t + log_out - log_s : -INFINITY;
    double loss = wave_sum_f64(p > 0.0 ? p * (lp - lq) : 0.0);
    if (left > 0.0)
        loss += left * (log(left) - lq0);
    const double all = mass + left;
    DistillStats st;
    st.m_out = m_out == -kInf ? 0.0f : m_out;      // r of a masked column is 0
    st.log_out = (float)log_out;
    st.f_out = (float)(t.tail ? exp(lq0) * all - left : all);
    st.m = m;
    st.log_s = (float)log_s;
    st.norm = norm;
    st.log_norm = (float)log_norm;
    st.mass = (float)all;
    if (empty) {
        loss = all > 0.0 ? INFINITY : 0.0;
        st.mass = 0.0f;
    }
    if (bad) {
        loss = NAN;
        st.f_out = st.mass = NAN;
    }
    if (!has) {
        loss = 0.0;
        st.mass = 0.0f;
    }
    if ((threadIdx.x & 63) == 0) {
        t.loss[row] = (float)loss;
        *(DistillStats*)(t.row_stats + row * VPA_DISTILL_STATS) = st;
    }
}

template <int ESIZE>
__global__ __launch_bounds__(kThreads) void distill_kernel(DistillTask t) {
    using T = typename elem<ESIZE>::type;
    __shared__ float lds[4][2];
    __shared__ int32_t ids[64];
    const int64_t row = blockIdx.x;
    const T* x = (const T*)t.logits + row * t.ld;
    const Named n = named_of(t, row);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (wave == 0)
        ids[lane] = t.tail ? n.id : -1;
    __syncthreads();
    auto value = [&](int c) {
        for (int j = 0; j < t.n_top; ++j)
            if (ids[j] == c)
                return -kInf;
        return to_f32(x[c]);
    };
    const float scale = kLog2e / t.temperature;
    float m = -kInf;
    for (int c = threadIdx.x; c < t.vocab; c += kThreads)
        m = fmaxf(m, value(c));
    float s = 0.0f;
    const float base = m == -kInf ? 0.0f : m;
    for (int c = threadIdx.x; c < t.vocab; c += kThreads)
        s += exp2_fast((value(c) - base) * scale);
    const float mx = wave_max(m);
    s = wave_sum(m == -kInf ? s : s * exp2_fast((m - mx) * scale));
    if (lane == 0) {
        lds[wave][0] = mx;
        lds[wave][1] = s;
    }
    __syncthreads();
    if (wave != 0)
        return;
    m = -kInf;
    s = 0.0f;
    for (int i = 0; i < 4; ++i) {
        if (lds[i][0] == -kInf)
            s += lds[i][1];
        else
            join(m, s, lds[i][0], lds[i][1], scale);
    }
    finish_row(t, row, x, n, m, s);
}

constexpr int kGradVecs = 4;                       // 16-byte vectors a thread
constexpr int grad_chunk(int esize) {
    return kThreads * kGradVecs * (16 / esize);
}

// The gradient of one chunk of a row: every column as one that is not named,
// then the named ones, from logits read before the chunk was written (the
// gradient may replace the logits).
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
    const DistillStats st = *(const DistillStats*)(t.row_stats + row * VPA_DISTILL_STATS);
    const float scale = kLog2e / t.temperature;
    const float g = t.grad_loss[row] / t.temperature;
    const bool zero = st.mass == 0.0f;
    const float f = g * st.f_out;
    const float log2_out = st.log_out * kLog2e;
    auto slope = [&](float v) {
        const float r = exp2f((v - st.m_out) * scale - log2_out);
        return zero ? 0.0f : r * f;
    };
    // this workgroup's named tokens, one a lane of the first wavefront
    float own = 0.0f;
    int64_t at = -1;
    if (threadIdx.x < 64) {
        const Named n = named_of(t, row);
        if (n.first && n.id >= lo && n.id < hi) {
            at = n.id;
            own = to_f32(x[at]);
        }
        float p = 0.0f;
        for (int j = 0; j < t.n_top; ++j) {
            const int32_t other = __builtin_amdgcn_readlane(n.id, j);
            const float lp = __builtin_bit_cast(
                float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, n.lp), j));
            p += other == n.id ? exp2f(((lp - st.norm) - st.log_norm) * kLog2e) : 0.0f;
        }
        const float q = exp2f((own - st.m) * scale - st.log_s * kLog2e);
        own = zero ? 0.0f : g * (q * st.mass - p);
    }
    __syncthreads();
    u32x4_t w[kGradVecs];
#pragma unroll
    for (int i = 0; i < kGradVecs; ++i) {
        const int64_t c = lo + (i * kThreads + threadIdx.x) * VEC;
        if (c + VEC <= t.vocab)
            w[i] = ((const Loose16*)(x + c))->v;
    }
#pragma unroll
    for (int i = 0; i < kGradVecs; ++i) {
        const int64_t c = lo + (i * kThreads + threadIdx.x) * VEC;
        if (c + VEC <= t.vocab) {
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
            __builtin_nontemporal_store(o, &((Loose16*)(d + c))->v);
        } else {
            for (int e = 0; e < VEC; ++e)
                if (c + e < hi)
                    from_f32(d[c + e], c + e < t.vocab ? slope(to_f32(x[c + e])) : 0.0f);
        }
    }
    __syncthreads();
    if (at >= 0)
        from_f32(d[at], own);
}

}  // namespace

size_t distill_workspace(int64_t, int64_t) {
    return 0;
}

int64_t distill_threads(int, int64_t, int64_t n_rows) {
    return n_rows * kThreads;
}

int64_t distill_grad_threads(int esize, int64_t grad_cols, int64_t n_rows) {
    const int64_t chunk = grad_chunk(esize);
    return (grad_cols + chunk - 1) / chunk * n_rows * kThreads;
}

hipError_t launch_distill(int esize, const DistillTask& t, void*, hipStream_t stream) {
    const dim3 grid((uint32_t)t.n_rows), block(kThreads);
    return esize == 2 ? launch(distill_kernel<2>, grid, block, 0, stream, t)
                      : launch(distill_kernel<4>, grid, block, 0, stream, t);
}

hipError_t launch_distill_grad(int esize, const DistillTask& t, hipStream_t stream) {
    const int64_t chunk = grad_chunk(esize);
    const int32_t chunks = (int32_t)((t.grad_cols + chunk - 1) / chunk);
    const dim3 grid((uint32_t)((int64_t)chunks * t.n_rows)), block(kThreads);
    return esize == 2 ? launch(distill_grad_kernel<2>, grid, block, 0, stream, t, chunks)
                      : launch(distill_grad_kernel<4>, grid, block, 0, stream, t, chunks);
}

hipError_t launch_distill_both(int esize, const DistillTask& t, void* ws, hipStream_t stream) {
    const hipError_t e = launch_distill(esize, t, ws, stream);
    return e != hipSuccess ? e : launch_distill_grad(esize, t, stream);
}

}  // namespace vpa
