/*
 * mamba_layers.h - C ABI of the layer operators that stand around the selective scan in a recurrent
 * language model: the gated linear recurrence, layer norm, the token embedding and the gated
 * feed-forward block, each with its gradient. Built into the same library as mamba_scan.h, whose
 * dtypes, error codes and mamba_scan_strerror() they share.
 *
 * Conventions (as in mamba_scan.h)
 *  - All pointers are DEVICE pointers of the GPU that is current when the call is made. The caller
 *    owns every buffer; the library never allocates, frees or synchronises.
 *  - Work is enqueued on `stream` (a hipStream_t; NULL = the default stream); the call returns
 *    without waiting. Errors are returned before anything is enqueued; the library never aborts.
 *  - dtype is the storage type of activations (and of the embedding's and the feed-forward block's
 *    weights); lam, weight and bias of the recurrence and the norm, states, statistics and their
 *    gradients are fp32. Arithmetic is fp32 in every case. An activation's gradient has the
 *    activation's dtype, a parameter's gradient the parameter's: each is rounded once, at its store.
 *  - Strides are in elements; a tensor's innermost stride is 1 and is not given.
 *  - Outputs must not overlap any input or each other (MAMBA_SCAN_ERR_ARGS), except where said.
 *  - Sizes may be 0: tensors without elements are never touched and may be NULL; gradients that are
 *    sums over nothing are written as zeros.
 *  - Results are bitwise deterministic: no sum depends on the order in which work is executed.
 */
#ifndef MAMBA_LAYERS_H
#define MAMBA_LAYERS_H

#include "mamba_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MAMBA_LAYERS_ABI_VERSION 1

/*
 * Gated linear recurrence over (batch, len, dim), one state per channel:
 *
 *   log a = -c * softplus(lam[d]) * sigmoid(r[b,t,d])          a = 0 where reset[b,t] != 0
 *   h_t   = a * h_{t-1} + sqrt(1 - a^2) * sigmoid(i[b,t,d]) * x[b,t,d]     (h starts at h0 or 0)
 *   y[b,t,d] = h_t;   last_state[b,d] = h after the last step
 *
 * A reset forgets the state before that step: sequences packed one after another do not see each
 * other. Nothing else forgets a NaN: one in x, r, i, lam or h0 reaches every state from there to the next
 * reset (a reset step does not use its r). The recurrence's associative form, (a1, b1) then (a2, b2) =
 * (a1 a2, a2 b1 + b2), is that of the parallel scan of "手把手用PyTorch实现Mamba的SSM层从HiPPO矩阵到
 * 选择性扫描算法" §3.2.
 *  - x, r, i, y: `dtype`, strides {batch, len} free and >= 0 (slices of a projection's output are
 *    fine). h0, last_state: (batch, dim) fp32 contiguous; last_state may be h0's own buffer (a
 *    decoder's state updated in place). reset: (batch, len) bytes, contiguous, or NULL.
 *  - checkpoints: NULL, or (batch, ceil(len / MAMBA_GATED_CHECKPOINT), dim) fp32 that receives the
 *    state before steps 0, 128, 256, ... for the backward pass.
 *  - workspace: mamba_gated_workspace_bytes(), 256-byte aligned (0 bytes unless several workgroups share
 *    a row's sequence, as for few long rows: they pass the state on through it).
 *  - Row strides up to 2^22 elements or so (64 stride + dim < 2^28), dim < 2^28, and batch * ceil(dim / 64)
 *    below 2^23 - 8; MAMBA_SCAN_ERR_UNSUPPORTED otherwise.
 *  - c must be finite and >= 0.
 */
#define MAMBA_GATED_CHECKPOINT 128

typedef struct mamba_gated_shape {
    int64_t batch, len, dim;
} mamba_gated_shape;

typedef struct mamba_gated_ptrs {
    const void* x;          /* (batch, len, dim) dtype */
    const void* r;
    const void* i;
    const float* lam;       /* (dim) */
    const float* h0;        /* (batch, dim) or NULL */
    const uint8_t* reset;   /* (batch, len) or NULL */
    void* y;                /* (batch, len, dim) dtype, written */
    float* last_state;      /* (batch, dim) written, or NULL */
    float* checkpoints;     /* written, or NULL */
    void* workspace;
    int64_t workspace_bytes;
} mamba_gated_ptrs;

typedef struct mamba_gated_strides {
    int64_t x[2], r[2], i[2], y[2]; /* {batch, len} */
} mamba_gated_strides;

int mamba_gated_scan_fwd(const mamba_gated_ptrs* p, const mamba_gated_shape* s, const mamba_gated_strides* st,
                         float c, mamba_scan_dtype dtype, void* stream);

/*
 * Its gradient for incoming dy (batch, len, dim; dtype) and, optionally, dlast_state (batch, dim; fp32).
 * The states are recomputed inside stretches of 128 steps from `checkpoints` (the forward's, on the
 * same inputs; NULL: recomputed first, into the workspace). With s = -log a, m = sqrt(1 - a^2),
 * g_t = dy_t + a_{t+1} g_{t+1} (dlast_state is added at the last step):
 *   dx = g m sigmoid(i);  di = g m x sigmoid'(i);  dh0 = a_0 g_0
 *   q  = s dLoss/ds = -a s g h_{t-1} + (s / m) a^2 sigmoid(i) x g     (0 at a reset; s / m -> 0 as s -> 0)
 *   dr = q (1 - sigmoid(r));   dlam[d] = sigmoid(lam) / softplus(lam) * sum_{b,t} q
 *  - dx, dr, di: dtype, strides {batch, len}. dlam (dim) fp32. dh0 (batch, dim) fp32 or NULL.
 */
typedef struct mamba_gated_bwd_ptrs {
    const void* x;
    const void* r;
    const void* i;
    const float* lam;
    const float* h0;
    const uint8_t* reset;
    const void* dy;
    const float* dlast_state;  /* or NULL */
    const float* checkpoints;  /* or NULL */
    void* dx;
    void* dr;
    void* di;
    float* dlam;
    float* dh0;                /* or NULL */
    void* workspace;           /* mamba_gated_bwd_workspace_bytes(), 256-byte aligned */
    int64_t workspace_bytes;
} mamba_gated_bwd_ptrs;

typedef struct mamba_gated_bwd_strides {
    int64_t x[2], r[2], i[2], dy[2], dx[2], dr[2], di[2];
} mamba_gated_bwd_strides;

int mamba_gated_scan_bwd(const mamba_gated_bwd_ptrs* p, const mamba_gated_shape* s, const mamba_gated_bwd_strides* st,
                         float c, mamba_scan_dtype dtype, void* stream);

/* Workspace bytes of the forward and of the backward (have_checkpoints: whether the call will be
 * given them), or a negative error code. They depend on the current device's compute-unit count. */
int64_t mamba_gated_workspace_bytes(const mamba_gated_shape* s, mamba_scan_dtype dtype);
int64_t mamba_gated_bwd_workspace_bytes(const mamba_gated_shape* s, mamba_scan_dtype dtype, int have_checkpoints);

/*
 * Layer norm over the last dimension of (rows, dim), with the residual added on the way:
 *
 *   t = x + residual, rounded to dtype (t = x without a residual); `sum` receives t
 *   y = (t - mean(t)) * rstd * weight + bias,   rstd = 1 / sqrt(mean((t - mean(t))^2) + eps)
 *
 * t is normalised as it is stored, so that the backward pass, which reads the stored t, differentiates
 * what the forward computed.
 *  - x, residual, y, sum: dtype, row strides free (>= dim for what is written). weight, bias: (dim)
 *    fp32, each may be NULL (1, 0). stats: (rows, 2) fp32 {mean, rstd} or NULL.
 *  - sum is written exactly when residual is given. y or sum may be x's or residual's own buffer
 *    with the same stride (in place), but not each other's.
 *  - eps must be finite and >= 0. With eps = 0 a constant row is 0 * inf = NaN, as the formula says. The
 *    statistics of a row with a NaN, and of a row without columns (dim = 0), are NaN.
 */
typedef struct mamba_norm_shape {
    int64_t rows, dim;
} mamba_norm_shape;

typedef struct mamba_norm_ptrs {
    const void* x;
    const void* residual;   /* or NULL */
    const float* weight;    /* or NULL */
    const float* bias;      /* or NULL */
    void* y;
    void* sum;              /* iff residual */
    float* stats;           /* (rows, 2) or NULL */
    int64_t x_stride, residual_stride, y_stride, sum_stride;
} mamba_norm_ptrs;

int mamba_layer_norm_fwd(const mamba_norm_ptrs* p, const mamba_norm_shape* s, float eps, mamba_scan_dtype dtype,
                         void* stream);

/*
 * Its gradient at t (the forward's x, or its sum) with the forward's stats. With n = (t - mean) rstd,
 * g = dy * weight:  dx = rstd (g - mean(g) - n mean(g n)) + dresidual (the gradient that reaches t
 * through the residual stream, or none);  dweight = sum_rows dy n;  dbias = sum_rows dy.
 * dx is also the gradient of the residual. dweight, dbias: (dim) fp32, each may be NULL.
 */
typedef struct mamba_norm_bwd_ptrs {
    const void* t;
    const float* weight;     /* or NULL */
    const float* stats;
    const void* dy;
    const void* dresidual;   /* or NULL */
    void* dx;
    float* dweight;          /* or NULL */
    float* dbias;            /* or NULL */
    int64_t t_stride, dy_stride, dresidual_stride, dx_stride;
    void* workspace;         /* mamba_layer_norm_bwd_workspace_bytes(), 256-byte aligned */
    int64_t workspace_bytes;
} mamba_norm_bwd_ptrs;

int mamba_layer_norm_bwd(const mamba_norm_bwd_ptrs* p, const mamba_norm_shape* s, mamba_scan_dtype dtype, void* stream);
int64_t mamba_layer_norm_bwd_workspace_bytes(const mamba_norm_shape* s);

/*
 * Token embedding: y[t, :] = scale * weight[ids[t], :], and its gradient
 * dweight[v, :] = scale * sum over the tokens with ids[t] = v of dy[t, :], in token order.
 * An id outside [0, vocab) (-1 for padding) gives a row of zeros and takes no gradient.
 *  - ids: (tokens) int64 or int32 (ids64), contiguous. weight, dweight: (vocab, dim) dtype contiguous,
 *    y, dy: (tokens, dim) dtype contiguous. Every row of dweight is written.
 *  - tokens < 2^31, vocab < 2^31.
 */
typedef struct mamba_embedding_shape {
    int64_t tokens, vocab, dim;
} mamba_embedding_shape;

int mamba_embedding_fwd(const void* ids, int ids64, const void* weight, void* y, const mamba_embedding_shape* s,
                        float scale, mamba_scan_dtype dtype, void* stream);
int mamba_embedding_bwd(const void* ids, int ids64, const void* dy, void* dweight, void* workspace,
                        int64_t workspace_bytes, const mamba_embedding_shape* s, float scale, mamba_scan_dtype dtype,
                        void* stream);
int64_t mamba_embedding_bwd_workspace_bytes(const mamba_embedding_shape* s);

/*
 * Gated feed-forward block up to its product: h = act(x w_gate^T) * (x w_up^T), act = silu or gelu in
 * its tanh form, and its gradient, which recomputes both projections:
 *   dg = dh u act'(g), du = dh act(g), each rounded to bf16 once as an operand of the products
 *   dx = dg w_gate + du w_up;  dw_gate = dg^T x;  dw_up = du^T x
 *  - x (rows, dim), w_gate, w_up (hidden, dim), h, dh (rows, hidden); all bf16, row strides free,
 *    products accumulated in fp32. dtype must be MAMBA_SCAN_BF16 (MAMBA_SCAN_ERR_UNSUPPORTED for F32).
 *  - workspace: mamba_gated_ffn_workspace_bytes() / ..._bwd_workspace_bytes(), 256-byte aligned.
 */
#define MAMBA_FFN_SILU 0
#define MAMBA_FFN_GELU_TANH 1

typedef struct mamba_ffn_shape {
    int64_t rows, dim, hidden;
} mamba_ffn_shape;

typedef struct mamba_ffn_ptrs {
    const void* x;
    const void* w_gate;
    const void* w_up;
    void* h;
    int64_t x_stride, w_gate_stride, w_up_stride, h_stride;
    void* workspace;
    int64_t workspace_bytes;
} mamba_ffn_ptrs;

typedef struct mamba_ffn_bwd_ptrs {
    const void* x;
    const void* w_gate;
    const void* w_up;
    const void* dh;
    void* dx;        /* (rows, dim) contiguous */
    void* dw_gate;   /* (hidden, dim) contiguous */
    void* dw_up;
    int64_t x_stride, w_gate_stride, w_up_stride, dh_stride;
    void* workspace;
    int64_t workspace_bytes;
} mamba_ffn_bwd_ptrs;

int mamba_gated_ffn_fwd(const mamba_ffn_ptrs* p, const mamba_ffn_shape* s, int act, mamba_scan_dtype dtype, void* stream);
int mamba_gated_ffn_bwd(const mamba_ffn_bwd_ptrs* p, const mamba_ffn_shape* s, int act, mamba_scan_dtype dtype, void* stream);
int64_t mamba_gated_ffn_workspace_bytes(const mamba_ffn_ptrs* p, const mamba_ffn_shape* s);
int64_t mamba_gated_ffn_bwd_workspace_bytes(const mamba_ffn_shape* s);

/* MAMBA_LAYERS_ABI_VERSION of the built library. */
int mamba_layers_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA_LAYERS_H */
