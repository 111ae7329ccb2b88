/*
 * mamba_block.h - C ABI of the operators that make a Mamba block and its language model complete around
 * the selective scan: the short causal convolution, the block's step from one token to the next, the norms
 * before and after a block, and the cross entropy over the vocabulary. Built into the same library as
 * mamba_scan.h, whose dtypes, error codes and mamba_scan_strerror() they share; the conventions are those
 * of mamba_layers.h:
 *  - All pointers are DEVICE pointers of the GPU that is current when the call is made. The caller owns
 *    every buffer; the library never allocates, frees or synchronises. Work is enqueued on `stream`.
 *    Errors are returned before anything is enqueued.
 *  - dtype is the storage type of activations (and of the projections' and the output matrix's weights);
 *    convolution weights, norm weights, biases, A, D, scan states, statistics, losses and their gradients
 *    are fp32. Arithmetic is fp32. An activation's gradient has the activation's dtype, a parameter's the
 *    parameter's; each is rounded once, at its store.
 *  - Strides are in elements and >= 0; a tensor's innermost stride is 1 and is not given.
 *  - Outputs must not overlap any input or each other (MAMBA_SCAN_ERR_ARGS), except where said.
 *  - Sizes may be 0: tensors without elements are never touched and may be NULL; gradients that are sums
 *    over nothing are written as zeros.
 *  - Workspaces are 256-byte aligned. Results are bitwise deterministic.
 */
#ifndef MAMBA_BLOCK_H
#define MAMBA_BLOCK_H

#include "mamba_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MAMBA_BLOCK_ABI_VERSION 1

/*
 * Short causal convolution over each channel (depthwise), with its activation:
 *
 *   pre_t = bias + sum_{k < width} weight[d,k] v_{t - width + 1 + k},   y_t = silu(pre_t)  (or pre_t)
 *
 * v_t = x_t for t >= 0; v_{-1}, v_{-2}, ... are the initial state's rows from its last one back (zeros without
 * one). Where reset[b,t] is set, a sequence begins at t: steps from t on see zeros in place of what lies
 * before it. last_state receives the width - 1 values that a step at len would see, so that a sequence can
 * be continued: last_state[b,j] = v_{len - width + 1 + j}, or 0 where a reset lies after it.
 *  - width 1 to 4. x and y in either layout: rows of channels at each step (x_steps = 0: strides {batch, step},
 *    unit stride over channels), or rows of steps of each channel (x_steps = 1: strides {batch, channel}, unit
 *    stride over steps: the scan's). y_steps = 0 with x_steps = 1 is MAMBA_SCAN_ERR_UNSUPPORTED.
 *  - weight (dim, width), bias (dim) or NULL; initial_state, last_state: (batch, width - 1, dim) dtype
 *    contiguous, or NULL; last_state may be initial_state's own buffer. reset: (batch, len) bytes or NULL.
 *  - batch * ceil(len / 8), or batch where len is 0, below 2^31, len below 2^30 and dim up to 2^22
 *    (MAMBA_SCAN_ERR_UNSUPPORTED).
 */
#define MAMBA_CONV_NONE 0
#define MAMBA_CONV_SILU 1

typedef struct mamba_conv_shape {
    int64_t batch, len, dim, width;
} mamba_conv_shape;

typedef struct mamba_conv_ptrs {
    const void* x;
    const float* weight;
    const float* bias;           /* or NULL */
    const void* initial_state;   /* or NULL */
    const uint8_t* reset;        /* or NULL */
    void* y;
    void* last_state;            /* or NULL */
    int64_t x_batch, x_row, y_batch, y_row;
    int32_t x_steps, y_steps;
} mamba_conv_ptrs;

int mamba_conv_fwd(const mamba_conv_ptrs* p, const mamba_conv_shape* s, int act, mamba_scan_dtype dtype, void* stream);

/*
 * Its gradient for incoming dy (in y's layout) and, optionally, dlast_state. pre is recomputed from x. With
 * dpre_t = dy_t silu'(pre_t):
 *   dv_s = sum_k weight[d,k] dpre_{s + width - 1 - k} over the steps that see s, + dlast_state where it holds s
 *   dx_s = dv_s (s >= 0), dinitial_state = dv_s (s < 0);  dweight[d,k] = sum dpre_t v_{t-width+1+k};  dbias = sum dpre
 *  - dx in x's layout with strides of its own; dweight (dim, width), dbias (dim) or NULL, fp32;
 *    dinitial_state (batch, width - 1, dim) dtype or NULL. The workspace depends on the current device's compute-unit
 *    count.
 */
typedef struct mamba_conv_bwd_ptrs {
    const void* x;
    const float* weight;
    const float* bias;
    const void* initial_state;
    const uint8_t* reset;
    const void* dy;
    const void* dlast_state;     /* or NULL */
    void* dx;
    float* dweight;
    float* dbias;                /* or NULL */
    void* dinitial_state;        /* or NULL */
    int64_t x_batch, x_row, dy_batch, dy_row, dx_batch, dx_row;
    int32_t x_steps, dy_steps;
    void* workspace;             /* mamba_conv_bwd_workspace_bytes() */
    int64_t workspace_bytes;
} mamba_conv_bwd_ptrs;

int mamba_conv_bwd(const mamba_conv_bwd_ptrs* p, const mamba_conv_shape* s, int act, mamba_scan_dtype dtype, void* stream);
int64_t mamba_conv_bwd_workspace_bytes(const mamba_conv_shape* s, mamba_scan_dtype dtype, int x_steps);

/*
 * One token of each stream through a Mamba block's path from the convolution to the gate:
 *
 *   u = silu(conv_b + sum_k conv_w[d,k] v_k),  v = the conv state's rows, then x
 *   (dt rows, B, C) = w_x u;  delta = w_dt dt;  s = softplus(delta + dt_bias)
 *   h' = exp(s A) h + s B u;  y = (sum_n C h' + D u) silu(z)
 *
 * what mamba_conv_fwd, the projections and mamba_scan_fwd (delta_softplus) compute for one step, with u, the
 * projections and delta kept in fp32.
 *  - x, z (batch, dim) dtype, row strides free; z may be NULL. conv_w (dim, width), conv_b (dim) or NULL,
 *    dt_bias (dim) or NULL, A (dim, dstate), D (dim) or NULL: fp32. w_x (dt_rank + 2 dstate, dim), w_dt (dim,
 *    dt_rank): dtype, contiguous.
 *  - conv_state (batch, width - 1, dim) dtype, ssm_state (batch, dim, dstate) fp32, contiguous; the new states
 *    go to conv_state_out and ssm_state_out, which may be the old ones' own buffers. y (batch, dim) fp32
 *    contiguous.
 *  - width 2 to 4, dstate 1 to 256, dt_rank 1 to 512, batch * ceil(dim / 64) up to 2^23 (MAMBA_SCAN_ERR_UNSUPPORTED).
 */
typedef struct mamba_step_shape {
    int64_t batch, dim, dstate, dt_rank, width;
} mamba_step_shape;

typedef struct mamba_step_ptrs {
    const void* x;
    const void* z;            /* or NULL */
    const void* conv_state;
    const float* ssm_state;
    const float* conv_w;
    const float* conv_b;      /* or NULL */
    const void* w_x;
    const void* w_dt;
    const float* dt_bias;     /* or NULL */
    const float* A;
    const float* D;           /* or NULL */
    void* conv_state_out;
    float* ssm_state_out;
    float* y;
    int64_t x_stride, z_stride;
    void* workspace;          /* mamba_block_step_workspace_bytes() */
    int64_t workspace_bytes;
} mamba_step_ptrs;

int mamba_block_step(const mamba_step_ptrs* p, const mamba_step_shape* s, mamba_scan_dtype dtype, void* stream);
int64_t mamba_block_step_workspace_bytes(const mamba_step_shape* s);

/*
 * Root-mean-square norm over the last dimension of (rows, dim), with the scaled residual added on the way:
 *
 *   t = residual + scale x, rounded to dtype (t = x without a residual); `sum` receives t
 *   y = t rstd weight,   rstd = 1 / sqrt(mean(t^2) + eps)
 *
 *  - x, residual, y, sum: dtype, row strides free (>= dim for what is written). weight (dim) fp32 or NULL (1).
 *    stats: (rows) fp32 rstd, or NULL. sum is written exactly when residual is given; scale is not used
 *    without one. y or sum may be x's or residual's own buffer with the same stride, but not each other's.
 *  - eps must be finite and >= 0, scale finite.
 *
 * The gradient at t (the forward's x, or its sum) with the forward's stats; n = t rstd, g = dy weight:
 *   dt = rstd (g - n mean(g n)) + dsum;   dx = scale dt;   dresidual = dt;   dweight = sum_rows dy n
 * dsum: the gradient that reaches t through the residual stream, or NULL. dx and dresidual are written where
 * they are not NULL.
 */
typedef struct mamba_rms_shape {
    int64_t rows, dim;
} mamba_rms_shape;

typedef struct mamba_rms_ptrs {
    const void* x;
    const void* residual;   /* or NULL */
    const float* weight;    /* or NULL */
    void* y;
    void* sum;              /* iff residual */
    float* stats;           /* (rows) or NULL */
    int64_t x_stride, residual_stride, y_stride, sum_stride;
} mamba_rms_ptrs;

typedef struct mamba_rms_bwd_ptrs {
    const void* t;
    const float* weight;    /* or NULL */
    const float* stats;
    const void* dy;
    const void* dsum;       /* or NULL */
    void* dx;               /* or NULL */
    void* dresidual;        /* or NULL */
    float* dweight;         /* or NULL */
    int64_t t_stride, dy_stride, dsum_stride, dx_stride, dresidual_stride;
    void* workspace;        /* mamba_rms_norm_bwd_workspace_bytes() */
    int64_t workspace_bytes;
} mamba_rms_bwd_ptrs;

int mamba_rms_norm_fwd(const mamba_rms_ptrs* p, const mamba_rms_shape* s, float scale, float eps, mamba_scan_dtype dtype,
                       void* stream);
int mamba_rms_norm_bwd(const mamba_rms_bwd_ptrs* p, const mamba_rms_shape* s, float scale, mamba_scan_dtype dtype, void* stream);
int64_t mamba_rms_norm_bwd_workspace_bytes(const mamba_rms_shape* s);

/*
 * The norm after a block's scan, with its gate z; each of `groups` stretches of dim / groups values has its
 * own rstd = 1 / sqrt(mean(v^2) + eps):
 *
 *   gate_first:  v = x silu(z),  y = v rstd weight         otherwise:  v = x,  y = v rstd weight silu(z)
 *
 *  - x, z, y: dtype, row strides free; weight (dim) fp32 or NULL; stats: (rows, groups) fp32 or NULL.
 *    y may be x's or z's own buffer with the same stride. groups, 1 to 65536, divides dim.
 *  - The gradients dx, dz (row strides free) and dweight (or NULL) come from x, z and the stats.
 */
typedef struct mamba_gated_rms_shape {
    int64_t rows, dim, groups;
} mamba_gated_rms_shape;

typedef struct mamba_gated_rms_ptrs {
    const void* x;
    const void* z;
    const float* weight;    /* or NULL */
    void* y;
    float* stats;           /* or NULL */
    int64_t x_stride, z_stride, y_stride;
} mamba_gated_rms_ptrs;

typedef struct mamba_gated_rms_bwd_ptrs {
    const void* x;
    const void* z;
    const float* weight;    /* or NULL */
    const float* stats;
    const void* dy;
    void* dx;
    void* dz;
    float* dweight;         /* or NULL */
    int64_t x_stride, z_stride, dy_stride, dx_stride, dz_stride;
    void* workspace;        /* mamba_gated_rms_norm_bwd_workspace_bytes() */
    int64_t workspace_bytes;
} mamba_gated_rms_bwd_ptrs;

int mamba_gated_rms_norm_fwd(const mamba_gated_rms_ptrs* p, const mamba_gated_rms_shape* s, int gate_first, float eps,
                             mamba_scan_dtype dtype, void* stream);
int mamba_gated_rms_norm_bwd(const mamba_gated_rms_bwd_ptrs* p, const mamba_gated_rms_shape* s, int gate_first,
                             mamba_scan_dtype dtype, void* stream);
int64_t mamba_gated_rms_norm_bwd_workspace_bytes(const mamba_gated_rms_shape* s);

/*
 * Softmax cross entropy of rows of hidden states against a large output matrix, the logits never stored:
 *
 *   l = scale x weight^T;  lse = log sum_v exp(l_v);  loss = lse - l[target]   (0 for a target outside [0, vocab))
 *
 * and its gradient for incoming dloss and, optionally, dlse (rows, or one value for all with stride 0). With
 * a = dloss where the target is inside [0, vocab), else 0:
 *   dl_v = (a + dlse) exp(l_v - lse) - a [v = target], rounded to bf16 as the operand of the products (where all rows
 *   with a target have the same a, as in a mean, without that factor, which then multiplies the fp32 sums)
 *   dx = scale dl weight;   dweight = scale dl^T x
 * A row with a + dlse = a = 0 takes no part in the gradients, whatever x holds there. The gradient works on
 * pieces of the vocabulary whose dl fit the workspace.
 *  - x (rows, dim), weight (vocab, dim): bf16, row strides free (MAMBA_SCAN_ERR_UNSUPPORTED for F32); dx, dweight
 *    contiguous bf16. target: (rows) int64 or int32 (target64). loss, lse: (rows) fp32, each may be NULL in the
 *    forward (not both); a loss needs target.
 *  - rows, vocab < 2^30, vocab >= 1 where there are rows; dim and row strides up to 2^21, and (rows / 128 + 1) (vocab /
 *    128 + 1) up to 2^23 (MAMBA_SCAN_ERR_UNSUPPORTED).
 */
typedef struct mamba_xent_shape {
    int64_t rows, dim, vocab;
} mamba_xent_shape;

typedef struct mamba_xent_ptrs {
    const void* x;
    const void* weight;
    const void* target;
    float* loss;
    float* lse;
    float* total;           /* {sum of the losses, number of targets inside [0, vocab)}, or NULL; needs loss */
    int64_t x_stride, weight_stride;
    void* workspace;        /* mamba_xent_workspace_bytes() */
    int64_t workspace_bytes;
} mamba_xent_ptrs;

typedef struct mamba_xent_bwd_ptrs {
    const void* x;
    const void* weight;
    const void* target;
    const float* lse;
    const float* dloss;     /* or NULL */
    const float* dlse;      /* or NULL */
    void* dx;               /* or NULL */
    void* dweight;          /* or NULL */
    int64_t x_stride, weight_stride, dloss_stride, dlse_stride; /* the last two 0 or 1 */
    void* workspace;        /* mamba_xent_bwd_workspace_bytes() */
    int64_t workspace_bytes;
} mamba_xent_bwd_ptrs;

int mamba_xent_fwd(const mamba_xent_ptrs* p, const mamba_xent_shape* s, int target64, float scale, mamba_scan_dtype dtype,
                   void* stream);
int mamba_xent_bwd(const mamba_xent_bwd_ptrs* p, const mamba_xent_shape* s, int target64, float scale, mamba_scan_dtype dtype,
                   void* stream);
/* Workspace bytes, or a negative error code. They depend on the operands' pointers and strides (rows that are not
 * 16-byte aligned are copied), on which gradients are asked for, and on the current device's compute-unit count. */
int64_t mamba_xent_workspace_bytes(const mamba_xent_ptrs* p, const mamba_xent_shape* s);
int64_t mamba_xent_bwd_workspace_bytes(const mamba_xent_bwd_ptrs* p, const mamba_xent_shape* s);

/* MAMBA_BLOCK_ABI_VERSION of the built library. */
int mamba_block_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA_BLOCK_H */
