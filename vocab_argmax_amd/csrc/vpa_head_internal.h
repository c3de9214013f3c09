// vpa_head_internal.h -- declarations shared by the HIP sources of the
// language-model head's operators (include/vpa_head.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "vpa_head.h"
#include "vpa_internal.h"

namespace vpa {

// ---- token log probabilities (logprob.hip) ----

// The columns of a launch: n_parts parts of part_width columns each, part p
// holding global columns [col0 + p*part_width, ...) cut to vocab.  A call on
// one GPU uses one part of V columns, a sharded one a part per local shard.
struct LogprobTask {
    const void* logits;       // column 0 = global column col0
    int64_t ld;
    int32_t vocab;
    int32_t col0;
    int32_t part_width;       // at most vocab
    int64_t part_stride;      // shard width: global columns from part to part
    int32_t n_parts;
    int32_t n_rows;
    int32_t n_top;
};

// How a launch is cut: one workgroup per (part, row, segment of columns).
struct LogprobCut {
    int32_t vecs;             // 16-byte vectors of a thread and chunk
    int32_t segments;         // of a part of a row
    int32_t chunks_per_segment;
    int64_t total;            // workgroups, and partial results
};
LogprobCut logprob_cut(int esize, int64_t part_width, int64_t n_parts, int64_t n_rows);
size_t logprob_workspace(const LogprobCut& c, int32_t n_top);
int64_t logprob_threads(const LogprobCut& c);

struct LogprobOut {
    const int32_t* token_ids;
    int32_t n_tokens;
    float* logprobs;
    float* lse;               // or null
    float* row_stats;
    int32_t* top_ids;
    float* top_logprobs;
};

// The outputs of whole rows (one part): one launch where a row is one segment,
// else the segments' partial results into `ws` and a second one.
hipError_t launch_token_logprobs(int esize, const LogprobTask& t, void* ws, const LogprobOut& o,
                                 hipStream_t stream);
// One record per (part, row), through partial results in `ws`.
hipError_t launch_logprob_records(int esize, const LogprobTask& t, void* ws,
                                  const int32_t* token_ids, int32_t n_tokens, int32_t* stats,
                                  hipStream_t stream);
// Records of every shard -> the outputs.
hipError_t launch_logprob_combine(const int32_t* stats, int32_t n_shards, int64_t shard_width,
                                  int32_t vocab, int32_t n_rows, int32_t n_top,
                                  const LogprobOut& o, hipStream_t stream);

struct LogprobGradTask {
    const void* logits;
    int64_t ld;
    int32_t vocab;
    int32_t col0;
    int32_t cols;             // valid local columns
    int64_t grad_cols;
    int64_t grad_ld;
    int32_t n_rows;
    const int32_t* token_ids;
    int32_t n_tokens;
    const float* row_stats;
    const float* grad_logprobs;
    const float* grad_entropy;
    void* grad;
};
int64_t logprob_grad_threads(int esize, int64_t grad_cols, int64_t n_rows);
hipError_t launch_logprob_grad(int esize, const LogprobGradTask& t, hipStream_t stream);

// ---- the head's products (linear.hip) ----

// C[m][n] = sum_k A(m, k) B(n, k), A(m, k) = a[m*a_m + k*a_k] (one of the two
// strides is 1), B alike, then the epilogue y = residual + act(C + bias[n]).
// The layouts used: k contiguous in both (a product with a weight), in A
// alone (grad_x) and in neither (grad_weight).  The caller names the layout:
// strides do not tell it (a matrix of one column has 1 both ways), and the
// workspace was sized for it.
struct GemmTask {
    const void* a;
    const void* b;
    int64_t a_m, a_k, b_n, b_k;
    bool a_k1, b_k1;          // k is contiguous in A, in B
    int64_t m, n, k;
    int64_t m_readable;       // columns of A that may be read where k is not contiguous (>= m)
    int64_t n_readable;       // columns of B, alike (>= n)
    const void* bias;
    const void* residual;
    int64_t ldr;
    void* y;
    int64_t ldy;
    bool out_f32;
    void* pre;
    int64_t ldp;
    int32_t act;
    void* ws;                 // gemm_workspace() bytes
};
constexpr int kFewRowsCols = 64;  // columns of a tile of few rows
// How a product is cut; everything but `direct` follows from sizes.
struct GemmPlan {
    bool rows_kernel;         // few rows: linear_rows.hip
    int32_t tile;             // 256 or 128: rows and columns of a workgroup's tile; 64 or
                              // 32: the rows, of kFewRowsCols columns
    int32_t slices;           // of k, joined by a second kernel
    int64_t stages_per_slice; // stages of 128 bytes of k
    int64_t first_m, first_n; // the plan is for these, the rest has its own; 0: for all
    bool direct;              // operands' strides allow direct loads to LDS
};
GemmPlan plan_gemm(int esize, int64_t m, int64_t n, int64_t k, bool a_k1, bool b_k1);
size_t gemm_workspace(int esize, int64_t m, int64_t n, int64_t k, bool a_k1, bool b_k1);
// Most work-items of one of the product's dispatches.
int64_t gemm_threads(int esize, int64_t m, int64_t n, int64_t k, bool a_k1, bool b_k1);
hipError_t launch_gemm(int esize, const GemmTask& t, hipStream_t stream);

hipError_t launch_gemm_tiles_bf16(const GemmTask& t, const GemmPlan& p, hipStream_t stream);
hipError_t launch_gemm_tiles_f32(const GemmTask& t, const GemmPlan& p, hipStream_t stream);

// The product for few rows of A (linear_rows.hip), k contiguous in both.
constexpr int kRowsKernelMost = 16;
int64_t linear_rows_threads(int64_t n);
hipError_t launch_linear_rows(int esize, const GemmTask& t, hipStream_t stream);

// dz = grad * act'(pre) (of the operands' type, skipped if dz is null), and
// the column sums of dz (before rounding) into `bias` (skipped if null).
struct DzTask {
    const void* grad;         // of the operands' type or, with grad_f32, fp32
    int64_t ldg;
    bool grad_f32;
    const void* pre;
    int64_t ldp;
    int32_t act;
    int64_t rows, cols;
    void* dz;                 // [rows][ldz]
    int64_t ldz;
    void* bias;
    float* part;              // [dz_splits(rows, cols)][cols]
};
int32_t dz_splits(int64_t rows, int64_t cols);
int64_t dz_threads(int64_t rows, int64_t cols, bool bias);
hipError_t launch_dz(int esize, const DzTask& t, hipStream_t stream);

// ---- layer norm (layer_norm.hip) ----

struct NormTask {
    const void* x;
    int64_t ldx;
    const void* weight;
    const void* bias;
    int wsize;                // element size of weight and bias
    int64_t rows, cols;
    float eps;
    void* y;
    int64_t ldy;
    float* mean;
    float* rstd;
};
int64_t norm_threads(int esize, int64_t rows, int64_t cols);
hipError_t launch_norm(int esize, const NormTask& t, hipStream_t stream);

struct NormGradTask {
    const void* grad;
    int64_t ldg;
    const void* x;
    int64_t ldx;
    const void* weight;
    int wsize;
    const float* mean;
    const float* rstd;
    int64_t rows, cols;
    void* dx;
    int64_t lddx;
    void* dweight;
    void* dbias;
    float* part;              // [2][norm_splits(esize, rows, cols)][cols]
};
int32_t norm_splits(int esize, int64_t rows, int64_t cols);
// Most work-items of one dispatch, for grad_x (dx) and the sums over rows.
int64_t norm_grad_threads(int esize, int64_t rows, int64_t cols, bool dx, bool sums);
hipError_t launch_norm_grad(int esize, const NormGradTask& t, hipStream_t stream);

}  // namespace vpa
