// What the C entry points hand to the sampling-control and block-scaled kernels.
#pragma once

#include "lpd_internal.cuh"

namespace lpd {

// ---------------------------------------------------------------- sampling controls
// One side's controls as the kernels take them (include/lpd.h, lpd_controls);
// all zero: no controls.
struct CtlSide {
    const int32_t *history;
    int64_t n_history;
    const int64_t *hist_begin, *hist_split, *hist_end;
    int counts;  // a history and at least one penalty
    const float *repetition, *frequency, *presence, *scale;
    const int32_t *bias_ids;
    const float *bias;
    int n_bias;
    const uint32_t *mask;
    int64_t n_masks, mask_stride;
    const int32_t *mask_row;
};

// One call of lpd_score_controlled behind the row selection.
struct CtlScoreCall {
    CtlSide t, r;
    const void *xt, *xr;
    int dtype_t, dtype_r;
    int64_t t_stride, r_stride;  // bytes
    int64_t n_rows, vocab;
    const WsHeader *hdr;
    const int2 *rowid;
    float4 *part_a;              // [active row][warp state] (mt, st, dd, mr)
    float *part_b;               // [active row][warp state] sr
    double2 *pick;               // selected controlled logits, before the scale
    float *out_lt, *out_lr, *out_d;
    double *dval;
    uint32_t *keys, *status;
};

int controls_states(int64_t vocab);  // warp states a row of the scoring form
cudaError_t launch_controls_apply(const CtlSide &c, const void *x, int x_dtype, int64_t x_stride_elems, void *out,
                                  int out_dtype, int64_t out_stride_elems, int64_t n_rows, int64_t vocab,
                                  cudaStream_t stream);
cudaError_t launch_controls_gradient(const CtlSide &c, const void *x, int x_dtype, int64_t x_stride_elems, void *out,
                                     int out_dtype, int64_t out_stride_elems, int64_t n_rows, int64_t vocab,
                                     const int32_t *ids, const uint8_t *mask, const float *logp, const float *grad,
                                     cudaStream_t stream);
cudaError_t launch_controls_score(const CtlScoreCall &c, cudaStream_t stream);

// ---------------------------------------------------------------- block-scaled 8-bit operands
struct BlockOperand {
    const void *ptr;
    int64_t row_stride;
    bool e5m2, block;      // 128 x 128 scales, else 1 x 128
    const float *scales;
    int64_t scale_stride;
};

// How a product is cut: output tiles, k blocks of 128, splits of the k axis.
struct BlockPlan {
    int64_t n_tm, n_tn, kb_total, kb_per_split, n_splits;
    int64_t part_stride;   // floats a row of a partial result
    size_t bytes;          // workspace
};
BlockPlan block_plan(int64_t m, int64_t n, int64_t k);
cudaError_t launch_block_quantize(const void *x, int x_dtype, int64_t x_stride_elems, int64_t rows, int64_t cols,
                                  bool block, bool transpose, bool pow2, bool e5m2, void *out, int64_t out_stride,
                                  float *scales, int64_t scale_stride, cudaStream_t stream);
cudaError_t launch_block_matmul(const BlockOperand &x, const BlockOperand &y, int64_t m, int64_t n, int64_t k,
                                void *out, int out_dtype, int64_t out_stride_elems, void *workspace,
                                cudaStream_t stream);

}  // namespace lpd
