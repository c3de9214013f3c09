// vpa_draft_internal.h -- declarations shared by the HIP sources of the draft
// head's operators (include/vpa_draft.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "vpa_draft.h"
#include "vpa_head_internal.h"

namespace vpa {

constexpr int kScaleBlock = 128;       // columns (a weight's: and rows) of a scale

// ---- sampled verification (sampled.hip) ----

struct SampleTask {
    const void* logits;
    int64_t ld;
    int32_t vocab;
    int32_t n_req, k;
    const int32_t* draft_ids;
    const void* probs;                 // or null
    int64_t ldq;
    const float* accept_u;
    const double* sample_u;
    const float* temperature;          // or null
    int32_t* out_tokens;
    int32_t* num_sampled;
    int32_t* num_rejected;
};
// How the launches are cut: segments of a row of logits for its statistics, of
// whole chunks; blocks of columns of the row that a request draws from, and
// workgroups that share them.
struct SampleCut {
    int32_t row_segments, row_chunks;
    int32_t draw_blocks, draw_groups;
};
SampleCut sample_cut(int esize, int64_t vocab, int64_t n_req, int32_t k);
size_t sample_workspace(const SampleCut& c, int64_t n_req, int32_t k);
// Most work-items of one of the launches.
int64_t sample_threads(const SampleCut& c, int64_t n_req, int32_t k);
// probs_esize: 2 or 4 (any without probs).
hipError_t launch_sample(int esize, int probs_esize, const SampleTask& t, void* ws,
                         hipStream_t stream);

// ---- distillation (distill.hip) ----

struct DistillTask {
    const void* logits;
    int64_t ld;
    int32_t vocab;
    int32_t n_rows;
    const int32_t* ids;
    const float* logprobs;
    int32_t n_top;
    bool tail;
    float temperature;
    float* loss;
    float* row_stats;
    // the gradient
    const float* grad_loss;
    void* grad;
    int64_t grad_ld, grad_cols;
};
size_t distill_workspace(int64_t vocab, int64_t n_rows);
int64_t distill_threads(int esize, int64_t vocab, int64_t n_rows);
int64_t distill_grad_threads(int esize, int64_t grad_cols, int64_t n_rows);
hipError_t launch_distill(int esize, const DistillTask& t, void* ws, hipStream_t stream);
hipError_t launch_distill_grad(int esize, const DistillTask& t, hipStream_t stream);
hipError_t launch_distill_both(int esize, const DistillTask& t, void* ws, hipStream_t stream);

// ---- root-mean-square norm and 8-bit rows (rms_norm.hip) ----

struct RmsTask {
    const void* x;
    int64_t ldx;
    const void* residual;
    int64_t ldr;
    const void* weight;
    int wsize;
    int64_t rows, cols;
    float eps;
    void* summed;
    int64_t lds;
    void* y;                           // of x's type, or e4m3 where scale is set
    int64_t ldy;
    float* rstd;
    float* scale;
    int64_t ld_scale;
};
int64_t rms_threads(int esize, int64_t rows, int64_t cols);
hipError_t launch_rms(int esize, const RmsTask& t, hipStream_t stream);

struct RmsGradTask {
    const void* grad;
    int64_t ldg;
    const void* summed;
    int64_t lds;
    const void* weight;
    int wsize;
    const float* rstd;
    const void* grad_summed;
    int64_t ldgs;
    int64_t rows, cols;
    void* dx;
    int64_t lddx;
    void* dweight;
    float* part;                       // [rms_splits(esize, rows, cols)][cols]
};
int32_t rms_splits(int esize, int64_t rows, int64_t cols);
int64_t rms_grad_threads(int esize, int64_t rows, int64_t cols, bool dx, bool sums);
hipError_t launch_rms_grad(int esize, const RmsGradTask& t, hipStream_t stream);

struct QuantTask {
    const void* x;
    int64_t ldx;
    int64_t rows, cols;
    int32_t block_rows;
    void* y;
    int64_t ldy;
    float* scale;
    int64_t ld_scale;
};
int64_t quant_threads(int esize, int64_t rows, int64_t cols, int32_t block_rows);
hipError_t launch_quant(int esize, const QuantTask& t, hipStream_t stream);

// ---- products of 8-bit operands (linear_fp8.hip) ----

// g: operands, sizes and epilogue as for a bf16 product whose k is contiguous
// in both, a and b in 8 bits.
struct Fp8Task {
    GemmTask g;
    const float* a_scale;
    int64_t lda_scale;
    const float* b_scale;
    int64_t ldb_scale;
    bool exact;                        // products in full fp32
};
size_t fp8_workspace(int64_t m, int64_t n, int64_t k, bool exact);
int64_t fp8_threads(int64_t m, int64_t n, int64_t k, bool exact);
hipError_t launch_fp8(const Fp8Task& t, hipStream_t stream);

}  // namespace vpa
