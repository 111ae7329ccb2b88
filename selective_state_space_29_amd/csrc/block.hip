// C-ABI entry points of the block operators: argument validation and the launch on the caller's stream. The
// contract is in include/mamba_block.h.
#include <hip/hip_runtime.h>

#include <cmath>
#include <initializer_list>
#include <stdint.h>

#include "block_launch.hpp"
#include "checks.hpp"
#include "launch.hpp"
#include "layers_common.hpp"
#include "layers_launch.hpp"

using namespace mscan;

namespace {

int64_t size_of(mamba_scan_dtype dtype) { return dtype == MAMBA_SCAN_BF16 ? 2 : 4; }

bool any_misaligned(std::initializer_list<const void*> ps, int64_t a) {
    for (const void* p : ps)
        if (misaligned(p, a)) return true;
    return false;
}

// Whether an output may lie on an input: not on it, or exactly on it row by row.
bool clash(const Bytes& out, const void* op, int64_t os, const Bytes& in, const void* ip, int64_t is, int64_t rows) {
    return meet(out, in) && !(op == ip && (os == is || rows <= 1));
}

// Zeros in fp32: gradients that are sums over nothing.
int zeros(float* p, int64_t n, hipStream_t stream) { return p && n > 0 ? launch_bwd_fill(p, nullptr, n, stream) : MAMBA_SCAN_OK; }

// ---- causal convolution ----

bool conv_bad_shape(const mamba_conv_shape& s) {
    return s.batch < 0 || s.len < 0 || s.dim < 0 || s.width < 1 || s.width > 4 || s.batch > kMaxGrid || s.len > kMaxGrid || s.dim > kMaxGrid;
}
// Runs of all sequences, one at least of each, are counted in 31 bits.
bool conv_too_large(const mamba_conv_shape& s) {
    return s.len >= (int64_t)1 << 30 || s.dim > (int64_t)1 << 22 || s.batch * (s.len > 0 ? (s.len + 7) / 8 : 1) > kMaxGrid;
}

// The layout of a (batch, len, dim) tensor: rows of channels or of steps.
struct Seq {
    int64_t rows, row;  // rows of a batch, their length
};
Seq seq_of(const mamba_conv_shape& s, int steps) { return steps ? Seq{s.dim, s.len} : Seq{s.len, s.dim}; }

bool bad_strides(const mamba_conv_shape& s, int steps, int64_t sb, int64_t sr) {
    return bad_span(s.batch, sb) || bad_span(seq_of(s, steps).rows, sr);
}
// An output whose rows meet would be written twice.
bool rows_meet(const mamba_conv_shape& s, int steps, int64_t sb, int64_t sr) {
    const Seq q = seq_of(s, steps);
    return (q.rows > 1 && sr < q.row) || (s.batch > 1 && q.rows > 0 && sb < (q.rows - 1) * sr + q.row);
}
Bytes conv_bytes(const void* p, int64_t es, const mamba_conv_shape& s, int steps, int64_t sb, int64_t sr) {
    const Seq q = seq_of(s, steps);
    return bytes_of(p, es, s.batch, sb, q.rows, sr, q.row);
}

// ---- norms ----

bool rms_bad_shape(int64_t rows, int64_t dim) { return rows < 0 || dim < 0 || rows > kMaxGrid || dim > kMaxGrid; }
constexpr int64_t kMaxGroups = 65536;

Bytes rows_bytes(const void* p, int64_t es, int64_t rows, int64_t stride, int64_t dim) { return bytes_of(p, es, 1, 0, rows, stride, dim); }

// ---- cross entropy ----

bool xent_bad_shape(const mamba_xent_shape& s) {
    constexpr int64_t most = (int64_t)1 << 30;
    return s.rows < 0 || s.dim < 0 || s.vocab < 0 || s.rows > most || s.dim > most || s.vocab > most || (s.rows > 0 && s.vocab == 0);
}
// Tiles address 256 rows of an operand with 32-bit byte offsets, and are counted in threads of a launch.
bool xent_too_large(const mamba_xent_shape& s, int64_t xs, int64_t ws) {
    constexpr int64_t most = (int64_t)1 << 21;
    return s.dim > most || (s.rows > 1 && xs > most) || (s.vocab > 1 && ws > most) ||
           (s.rows / 128 + 1) * (s.vocab / 128 + 1) > (int64_t)1 << 23;
}

}  // namespace

extern "C" {

int mamba_block_abi_version(void) { return MAMBA_BLOCK_ABI_VERSION; }

int mamba_conv_fwd(const mamba_conv_ptrs* p, const mamba_conv_shape* s, int act, mamba_scan_dtype dtype, void* stream) {
    if (!p || !s) return MAMBA_SCAN_ERR_NULL;
    if (bad_dtype(dtype)) return MAMBA_SCAN_ERR_DTYPE;
    if (conv_bad_shape(*s) || bad_strides(*s, p->x_steps, p->x_batch, p->x_row) || bad_strides(*s, p->y_steps, p->y_batch, p->y_row))
        return MAMBA_SCAN_ERR_SHAPE;
    if (act != MAMBA_CONV_NONE && act != MAMBA_CONV_SILU) return MAMBA_SCAN_ERR_ARGS;
    if (conv_too_large(*s)) return MAMBA_SCAN_ERR_UNSUPPORTED;  // before its sizes are multiplied
    const int64_t es = size_of(dtype), rows = s->batch * s->dim, state = rows * (s->width - 1) * es;
    if ((rows * s->len > 0 && (!p->x || !p->y)) || (s->dim > 0 && !p->weight)) return MAMBA_SCAN_ERR_NULL;
    if (any_misaligned({p->x, p->initial_state, p->y, p->last_state}, es) || any_misaligned({p->weight, p->bias}, 4) ||
        rows_meet(*s, p->y_steps, p->y_batch, p->y_row))
        return MAMBA_SCAN_ERR_ARGS;
    if (p->x_steps && !p->y_steps) return MAMBA_SCAN_ERR_UNSUPPORTED;
    const Bytes old = flat(p->initial_state, state);
    const Bytes ins[] = {conv_bytes(p->x, es, *s, p->x_steps, p->x_batch, p->x_row), flat(p->weight, s->dim * s->width * 4),
                         flat(p->bias, s->dim * 4), flat(p->reset, s->batch * s->len)};
    const Bytes outs[] = {conv_bytes(p->y, es, *s, p->y_steps, p->y_batch, p->y_row), flat(p->last_state, state)};
    if (any_overlap(ins, outs) || meet(old, outs[0]) || (p->last_state != p->initial_state && meet(old, outs[1])))
        return MAMBA_SCAN_ERR_ARGS;
    if (rows == 0 || (s->len == 0 && !p->last_state)) return MAMBA_SCAN_OK;
    return launch_conv_fwd(*p, *s, act, dtype == MAMBA_SCAN_BF16, static_cast<hipStream_t>(stream));
}

int64_t mamba_conv_bwd_workspace_bytes(const mamba_conv_shape* s, mamba_scan_dtype dtype, int x_steps) {
    if (!s) return MAMBA_SCAN_ERR_NULL;
    if (bad_dtype(dtype)) return MAMBA_SCAN_ERR_DTYPE;
    if (conv_bad_shape(*s)) return MAMBA_SCAN_ERR_SHAPE;
    if (conv_too_large(*s)) return MAMBA_SCAN_ERR_UNSUPPORTED;
    return s->batch * s->dim == 0 ? 0 : conv_bwd_workspace(*s, x_steps != 0);
}

int mamba_conv_bwd(const mamba_conv_bwd_ptrs* p, const mamba_conv_shape* s, int act, mamba_scan_dtype dtype, void* stream) {
    if (!p || !s) return MAMBA_SCAN_ERR_NULL;
    if (bad_dtype(dtype)) return MAMBA_SCAN_ERR_DTYPE;
    if (conv_bad_shape(*s) || bad_strides(*s, p->x_steps, p->x_batch, p->x_row) || bad_strides(*s, p->x_steps, p->dx_batch, p->dx_row) ||
        bad_strides(*s, p->dy_steps, p->dy_batch, p->dy_row))
        return MAMBA_SCAN_ERR_SHAPE;
    if (act != MAMBA_CONV_NONE && act != MAMBA_CONV_SILU) return MAMBA_SCAN_ERR_ARGS;
    if (conv_too_large(*s)) return MAMBA_SCAN_ERR_UNSUPPORTED;  // before its sizes are multiplied
    const int64_t es = size_of(dtype), rows = s->batch * s->dim, state = rows * (s->width - 1) * es;
    if ((rows * s->len > 0 && (!p->x || !p->dy || !p->dx)) || (s->dim > 0 && (!p->weight || !p->dweight))) return MAMBA_SCAN_ERR_NULL;
    if (any_misaligned({p->x, p->initial_state, p->dy, p->dlast_state, p->dx, p->dinitial_state}, es) ||
        any_misaligned({p->weight, p->bias, p->dweight, p->dbias}, 4) || rows_meet(*s, p->x_steps, p->dx_batch, p->dx_row))
        return MAMBA_SCAN_ERR_ARGS;
    if (p->x_steps && !p->dy_steps) return MAMBA_SCAN_ERR_UNSUPPORTED;
    const int rc = check_workspace(p->workspace, p->workspace_bytes, mamba_conv_bwd_workspace_bytes(s, dtype, p->x_steps));
    if (rc != MAMBA_SCAN_OK) return rc;
    const Bytes ins[] = {conv_bytes(p->x, es, *s, p->x_steps, p->x_batch, p->x_row), flat(p->weight, s->dim * s->width * 4),
                         flat(p->bias, s->dim * 4), flat(p->reset, s->batch * s->len), flat(p->initial_state, state),
                         conv_bytes(p->dy, es, *s, p->dy_steps, p->dy_batch, p->dy_row), flat(p->dlast_state, state),
                         flat(p->workspace, p->workspace_bytes)};
    const Bytes outs[] = {conv_bytes(p->dx, es, *s, p->x_steps, p->dx_batch, p->dx_row), flat(p->dweight, s->dim * s->width * 4),
                          flat(p->dbias, s->dim * 4), flat(p->dinitial_state, state)};
    if (any_overlap(ins, outs)) return MAMBA_SCAN_ERR_ARGS;
    hipStream_t hs = static_cast<hipStream_t>(stream);
    if (rows == 0) {
        const int e = zeros(p->dweight, s->dim * s->width, hs);
        return e == MAMBA_SCAN_OK ? zeros(p->dbias, s->dim, hs) : e;
    }
    return launch_conv_bwd(*p, *s, act, dtype == MAMBA_SCAN_BF16, hs);
}

// ---- block step ----

static bool step_bad_shape(const mamba_step_shape& s) {
    return s.batch < 0 || s.dim < 0 || s.batch > kMaxGrid || s.dim > kMaxGrid || s.dstate < 1 || s.dstate > 256 || s.dt_rank < 1 ||
           s.dt_rank > 512 || s.width < 2 || s.width > 4;
}
static bool step_too_large(const mamba_step_shape& s) { return s.batch * ((s.dim + 63) / 64) > (int64_t)1 << 23; }

int64_t mamba_block_step_workspace_bytes(const mamba_step_shape* s) {
    if (!s) return MAMBA_SCAN_ERR_NULL;
    if (step_bad_shape(*s)) return MAMBA_SCAN_ERR_SHAPE;
    if (step_too_large(*s)) return MAMBA_SCAN_ERR_UNSUPPORTED;
    return s->batch * s->dim == 0 ? 0 : block_step_workspace(*s);
}

int mamba_block_step(const mamba_step_ptrs* p, const mamba_step_shape* s, mamba_scan_dtype dtype, void* stream) {
    if (!p || !s) return MAMBA_SCAN_ERR_NULL;
    if (bad_dtype(dtype)) return MAMBA_SCAN_ERR_DTYPE;
    if (step_bad_shape(*s) || bad_span(s->batch, p->x_stride) || bad_span(s->batch, p->z_stride)) return MAMBA_SCAN_ERR_SHAPE;
    const int64_t es = size_of(dtype), cells = s->batch * s->dim, J = s->dt_rank + 2 * s->dstate;
    if (cells > 0 && (!p->x || !p->conv_state || !p->ssm_state || !p->conv_state_out || !p->ssm_state_out || !p->y || !p->conv_w ||
                      !p->w_x || !p->w_dt || !p->A))
        return MAMBA_SCAN_ERR_NULL;
    if (any_misaligned({p->x, p->z, p->conv_state, p->conv_state_out, p->w_x, p->w_dt}, es) ||
        any_misaligned({p->ssm_state, p->ssm_state_out, p->conv_w, p->conv_b, p->dt_bias, p->A, p->D, p->y}, 4))
        return MAMBA_SCAN_ERR_ARGS;
    if (step_too_large(*s)) return MAMBA_SCAN_ERR_UNSUPPORTED;
    const int rc = check_workspace(p->workspace, p->workspace_bytes, mamba_block_step_workspace_bytes(s));
    if (rc != MAMBA_SCAN_OK) return rc;
    const int64_t conv = cells * (s->width - 1) * es, ssm = cells * s->dstate * 4;
    const Bytes c0 = flat(p->conv_state, conv), h0 = flat(p->ssm_state, ssm);
    const Bytes ins[] = {rows_bytes(p->x, es, s->batch, p->x_stride, s->dim), rows_bytes(p->z, es, s->batch, p->z_stride, s->dim),
                         flat(p->conv_w, s->dim * s->width * 4), flat(p->conv_b, s->dim * 4), flat(p->w_x, J * s->dim * es),
                         flat(p->w_dt, s->dim * s->dt_rank * es), flat(p->dt_bias, s->dim * 4), flat(p->A, s->dim * s->dstate * 4),
                         flat(p->D, s->dim * 4), flat(p->workspace, p->workspace_bytes)};
    const Bytes outs[] = {flat(p->conv_state_out, conv), flat(p->ssm_state_out, ssm), flat(p->y, cells * 4)};
    if (any_overlap(ins, outs) || meet(outs[1], c0) || meet(outs[0], h0) || meet(outs[2], c0) || meet(outs[2], h0) ||
        (p->conv_state_out != p->conv_state && meet(outs[0], c0)) || (p->ssm_state_out != p->ssm_state && meet(outs[1], h0)))
        return MAMBA_SCAN_ERR_ARGS;
    if (cells == 0) return MAMBA_SCAN_OK;
    return launch_block_step(*p, *s, dtype == MAMBA_SCAN_BF16, static_cast<hipStream_t>(stream));
}

// ---- root-mean-square norms ----

int mamba_rms_norm_fwd(const mamba_rms_ptrs* p, const mamba_rms_shape* s, float scale, float eps, mamba_scan_dtype dtype, void* stream) {
    if (!p || !s) return MAMBA_SCAN_ERR_NULL;
    if (bad_dtype(dtype)) return MAMBA_SCAN_ERR_DTYPE;
    if (rms_bad_shape(s->rows, s->dim)) return MAMBA_SCAN_ERR_SHAPE;
    for (int64_t v : {p->x_stride, p->residual_stride, p->y_stride, p->sum_stride})
        if (bad_span(s->rows, v)) return MAMBA_SCAN_ERR_SHAPE;
    if (!(eps >= 0.0f) || std::isinf(eps) || !std::isfinite(scale)) return MAMBA_SCAN_ERR_ARGS;
    const int64_t es = size_of(dtype), cells = s->rows * s->dim;
    if (cells > 0 && (!p->x || !p->y)) return MAMBA_SCAN_ERR_NULL;
    if (cells > 0 && (p->residual != nullptr) != (p->sum != nullptr)) return MAMBA_SCAN_ERR_ARGS;
    if (any_misaligned({p->x, p->residual, p->y, p->sum}, es) || any_misaligned({p->weight, p->stats}, 4)) return MAMBA_SCAN_ERR_ARGS;
    if (s->rows > 1 && (p->y_stride < s->dim || (p->sum && p->sum_stride < s->dim))) return MAMBA_SCAN_ERR_ARGS;
    auto rows = [&](const void* q, int64_t stride) { return rows_bytes(q, es, s->rows, stride, s->dim); };
    const Bytes x = rows(p->x, p->x_stride), res = rows(p->residual, p->residual_stride);
    const Bytes ins[] = {flat(p->weight, s->dim * 4)};
    const Bytes outs[] = {rows(p->y, p->y_stride), rows(p->sum, p->sum_stride), flat(p->stats, s->rows * 4)};
    if (any_overlap(ins, outs) || meet(outs[2], x) || meet(outs[2], res) ||
        clash(outs[0], p->y, p->y_stride, x, p->x, p->x_stride, s->rows) || clash(outs[1], p->sum, p->sum_stride, x, p->x, p->x_stride, s->rows) ||
        clash(outs[0], p->y, p->y_stride, res, p->residual, p->residual_stride, s->rows) ||
        clash(outs[1], p->sum, p->sum_stride, res, p->residual, p->residual_stride, s->rows))
        return MAMBA_SCAN_ERR_ARGS;
    // rows without columns have statistics all the same: 0 / 0
    if (s->rows == 0 || (s->dim == 0 && !p->stats)) return MAMBA_SCAN_OK;
    return launch_rms_fwd(*p, *s, scale, eps, dtype == MAMBA_SCAN_BF16, static_cast<hipStream_t>(stream));
}

int64_t mamba_rms_norm_bwd_workspace_bytes(const mamba_rms_shape* s) {
    if (!s) return MAMBA_SCAN_ERR_NULL;
    if (rms_bad_shape(s->rows, s->dim)) return MAMBA_SCAN_ERR_SHAPE;
    return s->rows * s->dim == 0 ? 0 : rms_bwd_workspace(*s);
}

int mamba_rms_norm_bwd(const mamba_rms_bwd_ptrs* p, const mamba_rms_shape* s, float scale, mamba_scan_dtype dtype, void* stream) {
    if (!p || !s) return MAMBA_SCAN_ERR_NULL;
    if (bad_dtype(dtype)) return MAMBA_SCAN_ERR_DTYPE;
    if (rms_bad_shape(s->rows, s->dim)) return MAMBA_SCAN_ERR_SHAPE;
    for (int64_t v : {p->t_stride, p->dy_stride, p->dsum_stride, p->dx_stride, p->dresidual_stride})
        if (bad_span(s->rows, v)) return MAMBA_SCAN_ERR_SHAPE;
    if (!std::isfinite(scale)) return MAMBA_SCAN_ERR_ARGS;
    const int64_t es = size_of(dtype), cells = s->rows * s->dim;
    if (cells > 0 && (!p->t || !p->stats || !p->dy)) return MAMBA_SCAN_ERR_NULL;
    if (any_misaligned({p->t, p->dy, p->dsum, p->dx, p->dresidual}, es) || any_misaligned({p->weight, p->stats, p->dweight}, 4))
        return MAMBA_SCAN_ERR_ARGS;
    if (s->rows > 1 && ((p->dx && p->dx_stride < s->dim) || (p->dresidual && p->dresidual_stride < s->dim))) return MAMBA_SCAN_ERR_ARGS;
    const int rc = check_workspace(p->workspace, p->workspace_bytes, cells > 0 && p->dweight ? rms_bwd_workspace(*s) : 0);
    if (rc != MAMBA_SCAN_OK) return rc;
    auto rows = [&](const void* q, int64_t stride) { return rows_bytes(q, es, s->rows, stride, s->dim); };
    const Bytes ins[] = {rows(p->t, p->t_stride), rows(p->dy, p->dy_stride), rows(p->dsum, p->dsum_stride), flat(p->weight, s->dim * 4),
                         flat(p->stats, s->rows * 4), flat(p->workspace, p->workspace_bytes)};
    const Bytes outs[] = {rows(p->dx, p->dx_stride), rows(p->dresidual, p->dresidual_stride), flat(p->dweight, s->dim * 4)};
    if (any_overlap(ins, outs)) return MAMBA_SCAN_ERR_ARGS;
    hipStream_t hs = static_cast<hipStream_t>(stream);
    if (cells == 0) return zeros(p->dweight, s->dim, hs);
    return launch_rms_bwd(*p, *s, scale, dtype == MAMBA_SCAN_BF16, hs);
}

static bool gated_rms_bad_shape(const mamba_gated_rms_shape& s) {
    return rms_bad_shape(s.rows, s.dim) || s.groups < 1 || s.groups > kMaxGroups || s.dim % s.groups != 0;
}

int mamba_gated_rms_norm_fwd(const mamba_gated_rms_ptrs* p, const mamba_gated_rms_shape* s, int gate_first, float eps,
                             mamba_scan_dtype dtype, void* stream) {
    if (!p || !s) return MAMBA_SCAN_ERR_NULL;
    if (bad_dtype(dtype)) return MAMBA_SCAN_ERR_DTYPE;
    if (gated_rms_bad_shape(*s)) return MAMBA_SCAN_ERR_SHAPE;
    for (int64_t v : {p->x_stride, p->z_stride, p->y_stride})
        if (bad_span(s->rows, v)) return MAMBA_SCAN_ERR_SHAPE;
    if (!(eps >= 0.0f) || std::isinf(eps)) return MAMBA_SCAN_ERR_ARGS;
    const int64_t es = size_of(dtype), cells = s->rows * s->dim;
    if (cells > 0 && (!p->x || !p->z || !p->y)) return MAMBA_SCAN_ERR_NULL;
    if (any_misaligned({p->x, p->z, p->y}, es) || any_misaligned({p->weight, p->stats}, 4)) return MAMBA_SCAN_ERR_ARGS;
    if (s->rows > 1 && p->y_stride < s->dim) return MAMBA_SCAN_ERR_ARGS;
    auto rows = [&](const void* q, int64_t stride) { return rows_bytes(q, es, s->rows, stride, s->dim); };
    const Bytes x = rows(p->x, p->x_stride), z = rows(p->z, p->z_stride);
    const Bytes ins[] = {flat(p->weight, s->dim * 4)};
    const Bytes outs[] = {rows(p->y, p->y_stride), flat(p->stats, s->rows * s->groups * 4)};
    if (any_overlap(ins, outs) || meet(outs[1], x) || meet(outs[1], z) ||
        clash(outs[0], p->y, p->y_stride, x, p->x, p->x_stride, s->rows) || clash(outs[0], p->y, p->y_stride, z, p->z, p->z_stride, s->rows))
        return MAMBA_SCAN_ERR_ARGS;
    if (s->rows == 0 || (s->dim == 0 && !p->stats)) return MAMBA_SCAN_OK;
    return launch_gated_rms_fwd(*p, *s, gate_first != 0, eps, dtype == MAMBA_SCAN_BF16, static_cast<hipStream_t>(stream));
}

int64_t mamba_gated_rms_norm_bwd_workspace_bytes(const mamba_gated_rms_shape* s) {
    if (!s) return MAMBA_SCAN_ERR_NULL;
    if (gated_rms_bad_shape(*s)) return MAMBA_SCAN_ERR_SHAPE;
    return s->rows * s->dim == 0 ? 0 : gated_rms_bwd_workspace(*s);
}

int mamba_gated_rms_norm_bwd(const mamba_gated_rms_bwd_ptrs* p, const mamba_gated_rms_shape* s, int gate_first, mamba_scan_dtype dtype,
                             void* stream) {
    if (!p || !s) return MAMBA_SCAN_ERR_NULL;
    if (bad_dtype(dtype)) return MAMBA_SCAN_ERR_DTYPE;
    if (gated_rms_bad_shape(*s)) return MAMBA_SCAN_ERR_SHAPE;
    for (int64_t v : {p->x_stride, p->z_stride, p->dy_stride, p->dx_stride, p->dz_stride})
        if (bad_span(s->rows, v)) return MAMBA_SCAN_ERR_SHAPE;
    const int64_t es = size_of(dtype), cells = s->rows * s->dim;
    if (cells > 0 && (!p->x || !p->z || !p->stats || !p->dy || !p->dx || !p->dz)) return MAMBA_SCAN_ERR_NULL;
    if (any_misaligned({p->x, p->z, p->dy, p->dx, p->dz}, es) || any_misaligned({p->weight, p->stats, p->dweight}, 4))
        return MAMBA_SCAN_ERR_ARGS;
    if (s->rows > 1 && (p->dx_stride < s->dim || p->dz_stride < s->dim)) return MAMBA_SCAN_ERR_ARGS;
    const int rc = check_workspace(p->workspace, p->workspace_bytes, cells > 0 && p->dweight ? gated_rms_bwd_workspace(*s) : 0);
    if (rc != MAMBA_SCAN_OK) return rc;
    auto rows = [&](const void* q, int64_t stride) { return rows_bytes(q, es, s->rows, stride, s->dim); };
    const Bytes ins[] = {rows(p->x, p->x_stride), rows(p->z, p->z_stride), rows(p->dy, p->dy_stride), flat(p->weight, s->dim * 4),
                         flat(p->stats, s->rows * s->groups * 4), flat(p->workspace, p->workspace_bytes)};
    const Bytes outs[] = {rows(p->dx, p->dx_stride), rows(p->dz, p->dz_stride), flat(p->dweight, s->dim * 4)};
    if (any_overlap(ins, outs)) return MAMBA_SCAN_ERR_ARGS;
    hipStream_t hs = static_cast<hipStream_t>(stream);
    if (cells == 0) return zeros(p->dweight, s->dim, hs);
    return launch_gated_rms_bwd(*p, *s, gate_first != 0, dtype == MAMBA_SCAN_BF16, hs);
}

// ---- cross entropy ----

int64_t mamba_xent_workspace_bytes(const mamba_xent_ptrs* p, const mamba_xent_shape* s) {
    if (!p || !s) return MAMBA_SCAN_ERR_NULL;
    if (xent_bad_shape(*s)) return MAMBA_SCAN_ERR_SHAPE;
    if (xent_too_large(*s, p->x_stride, p->weight_stride)) return MAMBA_SCAN_ERR_UNSUPPORTED;
    return s->rows == 0 ? 0 : xent_workspace(*p, *s);
}

int mamba_xent_fwd(const mamba_xent_ptrs* p, const mamba_xent_shape* s, int target64, float scale, mamba_scan_dtype dtype, void* stream) {
    if (!p || !s) return MAMBA_SCAN_ERR_NULL;
    if (dtype != MAMBA_SCAN_BF16) return dtype == MAMBA_SCAN_F32 ? MAMBA_SCAN_ERR_UNSUPPORTED : MAMBA_SCAN_ERR_DTYPE;
    if (xent_bad_shape(*s) || bad_span(s->rows, p->x_stride) || bad_span(s->vocab, p->weight_stride)) return MAMBA_SCAN_ERR_SHAPE;
    if (!std::isfinite(scale)) return MAMBA_SCAN_ERR_ARGS;
    if (s->rows > 0 && ((s->dim > 0 && (!p->x || !p->weight)) || (!p->loss && !p->lse) || (p->loss && !p->target) || (p->total && !p->loss))) return MAMBA_SCAN_ERR_NULL;
    if (any_misaligned({p->x, p->weight}, 2) || any_misaligned({p->loss, p->lse, p->total}, 4) || misaligned(p->target, target64 ? 8 : 4))
        return MAMBA_SCAN_ERR_ARGS;
    if (xent_too_large(*s, p->x_stride, p->weight_stride)) return MAMBA_SCAN_ERR_UNSUPPORTED;
    const int rc = check_workspace(p->workspace, p->workspace_bytes, mamba_xent_workspace_bytes(p, s));
    if (rc != MAMBA_SCAN_OK) return rc;
    const Bytes ins[] = {rows_bytes(p->x, 2, s->rows, p->x_stride, s->dim), rows_bytes(p->weight, 2, s->vocab, p->weight_stride, s->dim),
                         flat(p->target, s->rows * (target64 ? 8 : 4)), flat(p->workspace, p->workspace_bytes)};
    const Bytes outs[] = {flat(p->loss, s->rows * 4), flat(p->lse, s->rows * 4), flat(p->total, 8)};
    if (any_overlap(ins, outs)) return MAMBA_SCAN_ERR_ARGS;
    if (s->rows == 0) return zeros(p->total, 2, static_cast<hipStream_t>(stream));
    return launch_xent_fwd(*p, *s, target64 != 0, scale, static_cast<hipStream_t>(stream));
}

int64_t mamba_xent_bwd_workspace_bytes(const mamba_xent_bwd_ptrs* p, const mamba_xent_shape* s) {
    if (!p || !s) return MAMBA_SCAN_ERR_NULL;
    if (xent_bad_shape(*s)) return MAMBA_SCAN_ERR_SHAPE;
    if (xent_too_large(*s, p->x_stride, p->weight_stride)) return MAMBA_SCAN_ERR_UNSUPPORTED;
    return s->rows == 0 || s->dim == 0 ? 0 : xent_bwd_workspace(*p, *s);
}

int mamba_xent_bwd(const mamba_xent_bwd_ptrs* p, const mamba_xent_shape* s, int target64, float scale, mamba_scan_dtype dtype, void* stream) {
    if (!p || !s) return MAMBA_SCAN_ERR_NULL;
    if (dtype != MAMBA_SCAN_BF16) return dtype == MAMBA_SCAN_F32 ? MAMBA_SCAN_ERR_UNSUPPORTED : MAMBA_SCAN_ERR_DTYPE;
    if (xent_bad_shape(*s) || bad_span(s->rows, p->x_stride) || bad_span(s->vocab, p->weight_stride)) return MAMBA_SCAN_ERR_SHAPE;
    if (!std::isfinite(scale) || (p->dloss_stride != 0 && p->dloss_stride != 1) || (p->dlse_stride != 0 && p->dlse_stride != 1))
        return MAMBA_SCAN_ERR_ARGS;
    if (s->rows > 0 && s->dim > 0 && (!p->x || !p->weight || !p->lse || (p->dloss && !p->target))) return MAMBA_SCAN_ERR_NULL;
    if (any_misaligned({p->x, p->weight, p->dx, p->dweight}, 2) || any_misaligned({p->lse, p->dloss, p->dlse}, 4) ||
        misaligned(p->target, target64 ? 8 : 4))
        return MAMBA_SCAN_ERR_ARGS;
    if (xent_too_large(*s, p->x_stride, p->weight_stride)) return MAMBA_SCAN_ERR_UNSUPPORTED;
    const int rc = check_workspace(p->workspace, p->workspace_bytes, mamba_xent_bwd_workspace_bytes(p, s));
    if (rc != MAMBA_SCAN_OK) return rc;
    const Bytes ins[] = {rows_bytes(p->x, 2, s->rows, p->x_stride, s->dim), rows_bytes(p->weight, 2, s->vocab, p->weight_stride, s->dim),
                         flat(p->target, s->rows * (target64 ? 8 : 4)), flat(p->lse, s->rows * 4),
                         flat(p->dloss, (p->dloss_stride ? s->rows : 1) * 4), flat(p->dlse, (p->dlse_stride ? s->rows : 1) * 4),
                         flat(p->workspace, p->workspace_bytes)};
    const Bytes outs[] = {flat(p->dx, s->rows * s->dim * 2), flat(p->dweight, s->vocab * s->dim * 2)};
    if (any_overlap(ins, outs)) return MAMBA_SCAN_ERR_ARGS;
    hipStream_t hs = static_cast<hipStream_t>(stream);
    if (s->rows == 0 || s->dim == 0) return p->dweight ? launch_ffn_zero(p->dweight, s->vocab, s->dim, s->dim, hs) : MAMBA_SCAN_OK;
    if (!p->dx && !p->dweight) return MAMBA_SCAN_OK;
    return launch_xent_bwd(*p, *s, target64 != 0, scale, hs);
}

}  // extern "C"
