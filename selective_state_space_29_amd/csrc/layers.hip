// C-ABI entry points of the layer operators: argument validation and the launch on the caller's
// stream. The contract is in include/mamba_layers.h.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cmath>
#include <stdint.h>

#include "gated.hpp"
#include "layers_common.hpp"
#include "launch.hpp"
#include "layers_launch.hpp"

using namespace mscan;

namespace mscan {

int layers_cus() {
    static std::atomic<int> cache[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
    int v = cache[dev].load(std::memory_order_relaxed);
    if (v == 0) {
        if (hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || v <= 0) return 256;
        cache[dev].store(v, std::memory_order_relaxed);
    }
    return v;
}

}  // namespace mscan

namespace {

struct Bytes {
    uintptr_t lo = 0, hi = 0;
};

// Bytes of n0 rows, `s0` elements apart, of n1 rows, `s1` apart, of n2 elements of `es` bytes.
Bytes bytes_of(const void* p, int64_t es, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2) {
    Bytes b;
    if (!p || n0 <= 0 || n1 <= 0 || n2 <= 0) return b;
    b.lo = reinterpret_cast<uintptr_t>(p);
    b.hi = b.lo + (uintptr_t)(((n0 - 1) * s0 + (n1 - 1) * s1 + n2) * es);
    return b;
}
Bytes flat(const void* p, int64_t bytes) { return bytes_of(p, 1, 1, 0, 1, 0, bytes); }

bool meet(const Bytes& a, const Bytes& b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }

template <int NI, int NO>
bool any_overlap(const Bytes (&ins)[NI], const Bytes (&outs)[NO]) {
    for (int o = 0; o < NO; ++o) {
        for (int i = 0; i < NI; ++i)
            if (meet(outs[o], ins[i])) return true;
        for (int o2 = 0; o2 < o; ++o2)
            if (meet(outs[o], outs[o2])) return true;
    }
    return false;
}

// Slices of one tensor whose rows lie side by side (dx, dr and di of a merged projection): the same
// strides, and starts at least a row's width apart within the row stride and the batch stride.
bool interleaved(const Bytes& a, const Bytes& b, const int64_t* sa, const int64_t* sb, const mamba_gated_shape& s, int64_t es) {
    const int64_t off = (int64_t)(a.lo > b.lo ? a.lo - b.lo : b.lo - a.lo) / es;
    return (s.batch <= 1 || sa[0] == sb[0]) && (s.len <= 1 || sa[1] == sb[1]) && off >= s.dim &&
           (s.len <= 1 || off + s.dim <= sa[1]) && (s.batch <= 1 || (s.len - 1) * sa[1] + off + s.dim <= sa[0]);
}

// Whether n rows `s` elements apart could not be addressed in 64 bits (or a size is negative).
bool bad_span(int64_t n, int64_t s) { return n < 0 || s < 0 || (n > 1 && s > ((int64_t)1 << 58) / n); }

bool bad_dtype(mamba_scan_dtype t) { return t != MAMBA_SCAN_F32 && t != MAMBA_SCAN_BF16; }
bool misaligned(const void* p, int64_t a) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)a != 0; }

// A workspace of at least `need` bytes, 256-byte aligned.
int check_workspace(const void* ws, int64_t have, int64_t need) {
    if (have < 0 || (have > 0 && !ws)) return MAMBA_SCAN_ERR_ARGS;
    if (need > have) return MAMBA_SCAN_ERR_WORKSPACE;
    if (need > 0 && misaligned(ws, 256)) return MAMBA_SCAN_ERR_ARGS;
    return MAMBA_SCAN_OK;
}

constexpr int64_t kMaxGrid = 0x7fffffff;

// ---- gated linear recurrence ----

bool gated_bad_shape(const mamba_gated_shape& s) {
    if (s.batch < 0 || s.len < 0 || s.dim < 0 || s.batch > kMaxGrid || s.dim > kMaxGrid) return true;
    return s.batch > 0 && s.dim > 0 && s.len > ((int64_t)1 << 48) / (s.batch * s.dim);
}

// Lanes address the rows of a chunk (256 steps at most) with 32-bit byte offsets.
bool gated_wide(const mamba_gated_shape& s, const int64_t* st, int n) {
    for (int k = 0; k < n; ++k)
        if (s.len > 1 && st[2 * k + 1] * 64 + s.dim >= ((int64_t)1 << 28)) return true;
    return s.dim >= (int64_t)1 << 28;
}

int64_t gated_nck(const mamba_gated_shape& s) { return (s.len + kGatedCk - 1) / kGatedCk; }

int64_t gated_chain_bytes(const mamba_gated_shape& s, int ways, int chunk) {
    return ways > 1 ? align256(GatedChain::words(s.batch, s.dim, (s.len + chunk - 1) / chunk) * 8) : 0;
}
int gated_fwd_chunk(bool bf16) { return 16 * gated_fwd_ts(bf16 ? 2 : 4, true); }

// Workspace of the backward: chain storage (the checkpoint pass's and then the backward's own),
// recomputed checkpoints, the chunks' sums of q.
struct GatedLayout {
    int fwd_ways, bwd_ways;
    int64_t ck, part, total;
};

GatedLayout gated_bwd_layout(const mamba_gated_shape& s, bool bf16, bool have_ck) {
    GatedLayout l;
    const int cus = layers_cus();
    l.fwd_ways = gated_fwd_ways(s, bf16, cus);
    l.bwd_ways = gated_bwd_ways(s, cus);
    const int64_t f = have_ck ? 0 : gated_chain_bytes(s, l.fwd_ways, gated_fwd_chunk(bf16)),
                  b = gated_chain_bytes(s, l.bwd_ways, kGatedCk);
    l.ck = f > b ? f : b;
    l.part = l.ck + (have_ck ? 0 : align256(s.batch * gated_nck(s) * s.dim * 4));
    l.total = l.part + align256(s.batch * gated_nck(s) * s.dim * 4);
    return l;
}

// Chunks and tickets are counted in 32 bits, the launch in workgroups.
bool gated_too_long(const mamba_gated_shape& s) {
    return s.len > (int64_t)1 << 36 || s.batch * ((s.dim + 63) / 64) + 8 > kMaxGrid / 256;
}

}  // namespace

extern "C" {

int mamba_layers_abi_version(void) { return MAMBA_LAYERS_ABI_VERSION; }

int64_t mamba_gated_workspace_bytes(const mamba_gated_shape* s, mamba_scan_dtype dtype) {
    if (!s) return MAMBA_SCAN_ERR_NULL;
    if (bad_dtype(dtype)) return MAMBA_SCAN_ERR_DTYPE;
    if (gated_bad_shape(*s)) return MAMBA_SCAN_ERR_SHAPE;
    if (s->batch * s->dim == 0 || s->len == 0) return 0;
    const bool bf16 = dtype == MAMBA_SCAN_BF16;
    return gated_chain_bytes(*s, gated_fwd_ways(*s, bf16, layers_cus()), gated_fwd_chunk(bf16));
}

int64_t mamba_gated_bwd_workspace_bytes(const mamba_gated_shape* s, mamba_scan_dtype dtype, int have_checkpoints) {
    if (!s) return MAMBA_SCAN_ERR_NULL;
    if (bad_dtype(dtype)) return MAMBA_SCAN_ERR_DTYPE;
    if (gated_bad_shape(*s)) return MAMBA_SCAN_ERR_SHAPE;
    if (s->batch * s->dim == 0 || s->len == 0) return 0;
    return gated_bwd_layout(*s, dtype == MAMBA_SCAN_BF16, have_checkpoints != 0).total;
}

int mamba_gated_scan_fwd(const mamba_gated_ptrs* p, const mamba_gated_shape* s, const mamba_gated_strides* st, float c,
                         mamba_scan_dtype dtype, void* stream) {
    if (!p || !s || !st) return MAMBA_SCAN_ERR_NULL;
    if (bad_dtype(dtype)) return MAMBA_SCAN_ERR_DTYPE;
    if (gated_bad_shape(*s)) return MAMBA_SCAN_ERR_SHAPE;
    const int64_t* sts = &st->x[0];
    for (int k = 0; k < 8; ++k)
        if (bad_span(k % 2 ? s->len : s->batch, sts[k])) return MAMBA_SCAN_ERR_SHAPE;
    if (!(c >= 0.0f) || std::isinf(c)) return MAMBA_SCAN_ERR_ARGS;
    const int64_t es = dtype == MAMBA_SCAN_BF16 ? 2 : 4;
    const int64_t rows = s->batch * s->dim, cells = rows * s->len;
    if ((cells > 0 && (!p->x || !p->r || !p->i || !p->y)) || (s->dim > 0 && !p->lam)) return MAMBA_SCAN_ERR_NULL;
    if (misaligned(p->x, es) || misaligned(p->r, es) || misaligned(p->i, es) || misaligned(p->y, es) ||
        misaligned(p->lam, 4) || misaligned(p->h0, 4) || misaligned(p->last_state, 4) || misaligned(p->checkpoints, 4))
        return MAMBA_SCAN_ERR_ARGS;
    // an output whose rows meet would be written twice
    if (s->len > 1 && st->y[1] < s->dim) return MAMBA_SCAN_ERR_ARGS;
    if (s->batch > 1 && s->len > 0 && st->y[0] < (s->len - 1) * st->y[1] + s->dim) return MAMBA_SCAN_ERR_ARGS;
    const int64_t ckn = s->batch * gated_nck(*s) * s->dim;
    auto seq = [&](const void* q, const int64_t* t) { return bytes_of(q, es, s->batch, t[0], s->len, t[1], s->dim); };
    const Bytes ins[] = {seq(p->x, st->x), seq(p->r, st->r), seq(p->i, st->i), flat(p->lam, s->dim * 4),
                         flat(p->reset, s->batch * s->len), flat(p->workspace, p->workspace_bytes)};
    const Bytes outs[] = {seq(p->y, st->y), flat(p->last_state, rows * 4), flat(p->checkpoints, ckn * 4)};
    if (any_overlap(ins, outs)) return MAMBA_SCAN_ERR_ARGS;
    const Bytes h0 = flat(p->h0, rows * 4);
    if (meet(h0, outs[0]) || meet(h0, outs[2]) || (p->last_state != p->h0 && meet(h0, outs[1]))) return MAMBA_SCAN_ERR_ARGS;
    if (rows == 0) return MAMBA_SCAN_OK;
    hipStream_t hs = static_cast<hipStream_t>(stream);

    GatedParams q{};
    q.x = p->x, q.r = p->r, q.i = p->i, q.lam = p->lam, q.h0 = p->h0, q.reset = p->reset;
    q.y = p->y, q.last = p->last_state, q.ck = p->checkpoints;
    q.batch = s->batch, q.len = s->len, q.dim = s->dim, q.nck = gated_nck(*s);
    q.sx_b = st->x[0], q.sx_t = st->x[1], q.sr_b = st->r[0], q.sr_t = st->r[1];
    q.si_b = st->i[0], q.si_t = st->i[1], q.sy_b = st->y[0], q.sy_t = st->y[1];
    q.c = c;
    if (gated_wide(*s, sts, 4) || gated_too_long(*s)) return MAMBA_SCAN_ERR_UNSUPPORTED;
    const bool bf16 = dtype == MAMBA_SCAN_BF16;
    q.ways = 1;
    if (s->len == 0)  // no step: the final state is the initial one (the short kernel's loop is empty)
        return p->last_state ? launch_gated_fwd(q, bf16, hs) : MAMBA_SCAN_OK;
    q.ways = gated_fwd_ways(*s, bf16, layers_cus());
    const int rc = check_workspace(p->workspace, p->workspace_bytes, gated_chain_bytes(*s, q.ways, gated_fwd_chunk(bf16)));
    if (rc != MAMBA_SCAN_OK) return rc;
    q.chain = static_cast<uint64_t*>(p->workspace);
    return launch_gated_fwd(q, bf16, hs);
}

int mamba_gated_scan_bwd(const mamba_gated_bwd_ptrs* p, const mamba_gated_shape* s, const mamba_gated_bwd_strides* st,
                         float c, mamba_scan_dtype dtype, void* stream) {
    if (!p || !s || !st) return MAMBA_SCAN_ERR_NULL;
    if (bad_dtype(dtype)) return MAMBA_SCAN_ERR_DTYPE;
    if (gated_bad_shape(*s)) return MAMBA_SCAN_ERR_SHAPE;
    const int64_t* sts = &st->x[0];
    for (int k = 0; k < 14; ++k)
        if (bad_span(k % 2 ? s->len : s->batch, sts[k])) return MAMBA_SCAN_ERR_SHAPE;
    if (!(c >= 0.0f) || std::isinf(c)) return MAMBA_SCAN_ERR_ARGS;
    const int64_t es = dtype == MAMBA_SCAN_BF16 ? 2 : 4;
    const int64_t rows = s->batch * s->dim, cells = rows * s->len;
    if ((cells > 0 && (!p->x || !p->r || !p->i || !p->dy || !p->dx || !p->dr || !p->di)) ||
        (s->dim > 0 && (!p->lam || !p->dlam)))
        return MAMBA_SCAN_ERR_NULL;
    for (const void* q : {p->x, p->r, p->i, p->dy, (const void*)p->dx, (const void*)p->dr, (const void*)p->di})
        if (misaligned(q, es)) return MAMBA_SCAN_ERR_ARGS;
    for (const void* q : {(const void*)p->lam, (const void*)p->h0, (const void*)p->dlast_state, (const void*)p->checkpoints,
                          (const void*)p->dlam, (const void*)p->dh0})
        if (misaligned(q, 4)) return MAMBA_SCAN_ERR_ARGS;
    for (const int64_t* o : {st->dx, st->dr, st->di}) {
        if (s->len > 1 && o[1] < s->dim) return MAMBA_SCAN_ERR_ARGS;
        if (s->batch > 1 && s->len > 0 && o[0] < (s->len - 1) * o[1] + s->dim) return MAMBA_SCAN_ERR_ARGS;
    }
    const bool have_ck = p->checkpoints != nullptr, bf16 = dtype == MAMBA_SCAN_BF16;
    const GatedLayout l = gated_bwd_layout(*s, bf16, have_ck);
    const int rc = check_workspace(p->workspace, p->workspace_bytes, cells > 0 ? l.total : 0);
    if (rc != MAMBA_SCAN_OK) return rc;
    auto seq = [&](const void* q, const int64_t* t) { return bytes_of(q, es, s->batch, t[0], s->len, t[1], s->dim); };
    const Bytes ins[] = {seq(p->x, st->x), seq(p->r, st->r), seq(p->i, st->i), seq(p->dy, st->dy), flat(p->lam, s->dim * 4),
                         flat(p->h0, rows * 4), flat(p->dlast_state, rows * 4), flat(p->reset, s->batch * s->len),
                         flat(p->checkpoints, s->batch * gated_nck(*s) * s->dim * 4),
                         flat(p->workspace, p->workspace_bytes)};
    const Bytes outs[] = {seq(p->dx, st->dx), seq(p->dr, st->dr), seq(p->di, st->di), flat(p->dlam, s->dim * 4),
                          flat(p->dh0, rows * 4)};
    const int64_t* ost[] = {st->dx, st->dr, st->di};
    for (int a = 0; a < 5; ++a) {
        for (const Bytes& in : ins)
            if (meet(outs[a], in)) return MAMBA_SCAN_ERR_ARGS;
        for (int b = 0; b < a; ++b)
            if (meet(outs[a], outs[b]) && !(a < 3 && interleaved(outs[a], outs[b], ost[a], ost[b], *s, es)))
                return MAMBA_SCAN_ERR_ARGS;
    }
    if (gated_wide(*s, sts, 7) || gated_too_long(*s)) return MAMBA_SCAN_ERR_UNSUPPORTED;
    hipStream_t hs = static_cast<hipStream_t>(stream);

    GatedBwdParams q{};
    q.x = p->x, q.r = p->r, q.i = p->i, q.lam = p->lam, q.h0 = p->h0, q.reset = p->reset;
    q.dy = p->dy, q.dlast = p->dlast_state, q.ck = p->checkpoints;
    q.dx = p->dx, q.dr = p->dr, q.di = p->di, q.dh0 = p->dh0;
    q.batch = s->batch, q.len = s->len, q.dim = s->dim, q.nck = gated_nck(*s);
    q.sx_b = st->x[0], q.sx_t = st->x[1], q.sr_b = st->r[0], q.sr_t = st->r[1], q.si_b = st->i[0], q.si_t = st->i[1];
    q.sdy_b = st->dy[0], q.sdy_t = st->dy[1], q.sdx_b = st->dx[0], q.sdx_t = st->dx[1];
    q.sdr_b = st->dr[0], q.sdr_t = st->dr[1], q.sdi_b = st->di[0], q.sdi_t = st->di[1];
    q.c = c;
    if (cells == 0) {  // sums over nothing; over no steps the initial state's gradient is the final one's
        int e = s->dim > 0 ? launch_bwd_fill(p->dlam, nullptr, s->dim, hs) : MAMBA_SCAN_OK;
        if (e == MAMBA_SCAN_OK && p->dh0 && rows > 0) e = launch_bwd_fill(p->dh0, p->dlast_state, rows, hs);
        return e;
    }
    char* ws = static_cast<char*>(p->workspace);
    if (!have_ck) {
        GatedParams f{};
        f.x = p->x, f.r = p->r, f.i = p->i, f.lam = p->lam, f.h0 = p->h0, f.reset = p->reset;
        f.ck = reinterpret_cast<float*>(ws + l.ck);
        f.batch = s->batch, f.len = s->len, f.dim = s->dim, f.nck = q.nck;
        f.sx_b = q.sx_b, f.sx_t = q.sx_t, f.sr_b = q.sr_b, f.sr_t = q.sr_t, f.si_b = q.si_b, f.si_t = q.si_t;
        f.c = c, f.ways = l.fwd_ways;
        f.chain = reinterpret_cast<uint64_t*>(ws);
        const int e = launch_gated_checkpoints(f, bf16, hs);
        if (e != MAMBA_SCAN_OK) return e;
        q.ck = f.ck;
    }
    q.chain = reinterpret_cast<uint64_t*>(ws);
    q.ways = l.bwd_ways;
    q.part = reinterpret_cast<float*>(ws + l.part);
    q.dlam = p->dlam;
    return launch_gated_bwd(q, bf16, hs);
}

// ---- layer norm ----

static bool norm_bad_shape(const mamba_norm_shape& s) {
    return s.rows < 0 || s.dim < 0 || s.rows > kMaxGrid || s.dim > kMaxGrid;
}

int mamba_layer_norm_fwd(const mamba_norm_ptrs* p, const mamba_norm_shape* s, float eps, mamba_scan_dtype dtype,
                         void* stream) {
    if (!p || !s) return MAMBA_SCAN_ERR_NULL;
    if (bad_dtype(dtype)) return MAMBA_SCAN_ERR_DTYPE;
    if (norm_bad_shape(*s)) return MAMBA_SCAN_ERR_SHAPE;
    for (int64_t v : {p->x_stride, p->residual_stride, p->y_stride, p->sum_stride})
        if (bad_span(s->rows, v)) return MAMBA_SCAN_ERR_SHAPE;
    if (!(eps >= 0.0f) || std::isinf(eps)) return MAMBA_SCAN_ERR_ARGS;
    const int64_t es = dtype == MAMBA_SCAN_BF16 ? 2 : 4, cells = s->rows * s->dim;
    if (cells > 0 && (!p->x || !p->y)) return MAMBA_SCAN_ERR_NULL;
    if (cells > 0 && (p->residual != nullptr) != (p->sum != nullptr)) return MAMBA_SCAN_ERR_ARGS;
    for (const void* q : {p->x, p->residual, (const void*)p->y, (const void*)p->sum})
        if (misaligned(q, es)) return MAMBA_SCAN_ERR_ARGS;
    if (misaligned(p->weight, 4) || misaligned(p->bias, 4) || misaligned(p->stats, 4)) return MAMBA_SCAN_ERR_ARGS;
    if (s->rows > 1 && (p->y_stride < s->dim || (p->sum && p->sum_stride < s->dim))) return MAMBA_SCAN_ERR_ARGS;
    auto rows = [&](const void* q, int64_t stride) { return bytes_of(q, es, 1, 0, s->rows, stride, s->dim); };
    const Bytes x = rows(p->x, p->x_stride), res = rows(p->residual, p->residual_stride);
    const Bytes y = rows(p->y, p->y_stride), sum = rows(p->sum, p->sum_stride), st = flat(p->stats, s->rows * 8);
    const Bytes w = flat(p->weight, s->dim * 4), b = flat(p->bias, s->dim * 4);
    // y and sum may be x's or residual's own rows: each element is read before it is written
    auto clash = [&](const Bytes& o, const void* op, int64_t os, const Bytes& in, const void* ip, int64_t is) {
        return meet(o, in) && !(op == ip && (os == is || s->rows <= 1));
    };
    if (clash(y, p->y, p->y_stride, x, p->x, p->x_stride) || clash(sum, p->sum, p->sum_stride, x, p->x, p->x_stride) ||
        clash(y, p->y, p->y_stride, res, p->residual, p->residual_stride) ||
        clash(sum, p->sum, p->sum_stride, res, p->residual, p->residual_stride))
        return MAMBA_SCAN_ERR_ARGS;
    const Bytes ins[] = {w, b}, outs[] = {y, sum, st};
    if (any_overlap(ins, outs) || meet(st, x) || meet(st, res)) return MAMBA_SCAN_ERR_ARGS;
    // rows without columns have statistics all the same: 0 / 0
    if (s->rows == 0 || (s->dim == 0 && !p->stats)) return MAMBA_SCAN_OK;
    return launch_norm_fwd(*p, *s, eps, dtype == MAMBA_SCAN_BF16, static_cast<hipStream_t>(stream));
}

int64_t mamba_layer_norm_bwd_workspace_bytes(const mamba_norm_shape* s) {
    if (!s) return MAMBA_SCAN_ERR_NULL;
    if (norm_bad_shape(*s)) return MAMBA_SCAN_ERR_SHAPE;
    return s->rows * s->dim == 0 ? 0 : norm_bwd_workspace(*s);
}

int mamba_layer_norm_bwd(const mamba_norm_bwd_ptrs* p, const mamba_norm_shape* s, mamba_scan_dtype dtype, void* stream) {
    if (!p || !s) return MAMBA_SCAN_ERR_NULL;
    if (bad_dtype(dtype)) return MAMBA_SCAN_ERR_DTYPE;
    if (norm_bad_shape(*s)) return MAMBA_SCAN_ERR_SHAPE;
    for (int64_t v : {p->t_stride, p->dy_stride, p->dresidual_stride, p->dx_stride})
        if (bad_span(s->rows, v)) return MAMBA_SCAN_ERR_SHAPE;
    const int64_t es = dtype == MAMBA_SCAN_BF16 ? 2 : 4, cells = s->rows * s->dim;
    if (cells > 0 && (!p->t || !p->stats || !p->dy || !p->dx)) return MAMBA_SCAN_ERR_NULL;
    for (const void* q : {p->t, p->dy, p->dresidual, (const void*)p->dx})
        if (misaligned(q, es)) return MAMBA_SCAN_ERR_ARGS;
    for (const void* q : {(const void*)p->weight, (const void*)p->stats, (const void*)p->dweight, (const void*)p->dbias})
        if (misaligned(q, 4)) return MAMBA_SCAN_ERR_ARGS;
    if (s->rows > 1 && p->dx_stride < s->dim) return MAMBA_SCAN_ERR_ARGS;
    const int rc = check_workspace(p->workspace, p->workspace_bytes,
                                   cells > 0 && (p->dweight || p->dbias) ? norm_bwd_workspace(*s) : 0);
    if (rc != MAMBA_SCAN_OK) return rc;
    auto rows = [&](const void* q, int64_t stride) { return bytes_of(q, es, 1, 0, s->rows, stride, s->dim); };
    const Bytes ins[] = {rows(p->t, p->t_stride), rows(p->dy, p->dy_stride), rows(p->dresidual, p->dresidual_stride),
                         flat(p->weight, s->dim * 4), flat(p->stats, s->rows * 8), flat(p->workspace, p->workspace_bytes)};
    const Bytes outs[] = {rows(p->dx, p->dx_stride), flat(p->dweight, s->dim * 4), flat(p->dbias, s->dim * 4)};
    if (any_overlap(ins, outs)) return MAMBA_SCAN_ERR_ARGS;
    hipStream_t hs = static_cast<hipStream_t>(stream);
    if (cells == 0) {
        int e = p->dweight && s->dim > 0 ? launch_bwd_fill(p->dweight, nullptr, s->dim, hs) : MAMBA_SCAN_OK;
        if (e == MAMBA_SCAN_OK && p->dbias && s->dim > 0) e = launch_bwd_fill(p->dbias, nullptr, s->dim, hs);
        return e;
    }
    return launch_norm_bwd(*p, *s, dtype == MAMBA_SCAN_BF16, hs);
}

// ---- token embedding ----

static bool embed_bad_shape(const mamba_embedding_shape& s) {
    if (s.tokens < 0 || s.vocab < 0 || s.dim < 0 || s.tokens > kMaxGrid || s.vocab > kMaxGrid || s.dim > kMaxGrid) return true;
    const int64_t most = s.tokens > s.vocab ? s.tokens : s.vocab;
    return most > 0 && s.dim > ((int64_t)1 << 46) / most;
}

static int embed_check(const void* ids, const void* in, const void* out, int64_t in_rows, int64_t out_rows,
                       const mamba_embedding_shape& s, int ids64, int64_t es, const void* ws, int64_t ws_bytes) {
    if ((s.tokens > 0 && !ids) || (in_rows * s.dim > 0 && !in) || (out_rows * s.dim > 0 && !out)) return MAMBA_SCAN_ERR_NULL;
    if (misaligned(ids, ids64 ? 8 : 4) || misaligned(in, es) || misaligned(out, es)) return MAMBA_SCAN_ERR_ARGS;
    const Bytes ins[] = {flat(ids, s.tokens * (ids64 ? 8 : 4)), flat(in, in_rows * s.dim * es), flat(ws, ws_bytes)};
    const Bytes outs[] = {flat(out, out_rows * s.dim * es)};
    return any_overlap(ins, outs) ? MAMBA_SCAN_ERR_ARGS : MAMBA_SCAN_OK;
}

int mamba_embedding_fwd(const void* ids, int ids64, const void* weight, void* y, const mamba_embedding_shape* s, float scale,
                        mamba_scan_dtype dtype, void* stream) {
    if (!s) return MAMBA_SCAN_ERR_NULL;
    if (bad_dtype(dtype)) return MAMBA_SCAN_ERR_DTYPE;
    if (embed_bad_shape(*s)) return MAMBA_SCAN_ERR_SHAPE;
    const int rc = embed_check(ids, weight, y, s->vocab, s->tokens, *s, ids64, dtype == MAMBA_SCAN_BF16 ? 2 : 4, nullptr, 0);
    if (rc != MAMBA_SCAN_OK || s->tokens * s->dim == 0) return rc;
    return launch_embedding_fwd(ids, ids64 != 0, weight, y, *s, scale, dtype == MAMBA_SCAN_BF16, static_cast<hipStream_t>(stream));
}

int64_t mamba_embedding_bwd_workspace_bytes(const mamba_embedding_shape* s) {
    if (!s) return MAMBA_SCAN_ERR_NULL;
    if (embed_bad_shape(*s)) return MAMBA_SCAN_ERR_SHAPE;
    return s->vocab * s->dim == 0 ? 0 : embedding_bwd_workspace(*s);
}

int mamba_embedding_bwd(const void* ids, int ids64, const void* dy, void* dweight, void* workspace, int64_t workspace_bytes,
                        const mamba_embedding_shape* s, float scale, mamba_scan_dtype dtype, void* stream) {
    if (!s) return MAMBA_SCAN_ERR_NULL;
    if (bad_dtype(dtype)) return MAMBA_SCAN_ERR_DTYPE;
    if (embed_bad_shape(*s)) return MAMBA_SCAN_ERR_SHAPE;
    int rc = check_workspace(workspace, workspace_bytes, mamba_embedding_bwd_workspace_bytes(s));
    if (rc != MAMBA_SCAN_OK) return rc;
    rc = embed_check(ids, dy, dweight, s->tokens, s->vocab, *s, ids64, dtype == MAMBA_SCAN_BF16 ? 2 : 4, workspace, workspace_bytes);
    if (rc != MAMBA_SCAN_OK || s->vocab * s->dim == 0) return rc;
    return launch_embedding_bwd(ids, ids64 != 0, dy, dweight, workspace, *s, scale, dtype == MAMBA_SCAN_BF16,
                                static_cast<hipStream_t>(stream));
}

// ---- gated feed-forward ----

static bool ffn_bad_shape(const mamba_ffn_shape& s) {
    constexpr int64_t most = (int64_t)1 << 30;
    return s.rows < 0 || s.dim < 0 || s.hidden < 0 || s.rows > most || s.dim > most || s.hidden > most;
}

// Tiles address 256 rows of an operand with 32-bit byte offsets.
static bool ffn_too_wide(const mamba_ffn_shape& s, int64_t xs, int64_t gs, int64_t us) {
    constexpr int64_t most = (int64_t)1 << 21;
    return s.dim > most || s.hidden > most / 2 || (s.rows > 1 && xs > most) || (s.hidden > 1 && (gs > most || us > most));
}

int64_t mamba_gated_ffn_workspace_bytes(const mamba_ffn_ptrs* p, const mamba_ffn_shape* s) {
    if (!p || !s) return MAMBA_SCAN_ERR_NULL;
    if (ffn_bad_shape(*s)) return MAMBA_SCAN_ERR_SHAPE;
    return s->rows * s->hidden == 0 || s->dim == 0 ? 0 : ffn_workspace(*p, *s);
}

int64_t mamba_gated_ffn_bwd_workspace_bytes(const mamba_ffn_shape* s) {
    if (!s) return MAMBA_SCAN_ERR_NULL;
    if (ffn_bad_shape(*s)) return MAMBA_SCAN_ERR_SHAPE;
    return s->rows == 0 || s->hidden == 0 || s->dim == 0 ? 0 : ffn_bwd_workspace(*s);
}

int mamba_gated_ffn_fwd(const mamba_ffn_ptrs* p, const mamba_ffn_shape* s, int act, mamba_scan_dtype dtype, void* stream) {
    if (!p || !s) return MAMBA_SCAN_ERR_NULL;
    if (dtype != MAMBA_SCAN_BF16) return dtype == MAMBA_SCAN_F32 ? MAMBA_SCAN_ERR_UNSUPPORTED : MAMBA_SCAN_ERR_DTYPE;
    if (ffn_bad_shape(*s)) return MAMBA_SCAN_ERR_SHAPE;
    if (bad_span(s->rows, p->x_stride) || bad_span(s->hidden, p->w_gate_stride) || bad_span(s->hidden, p->w_up_stride) ||
        bad_span(s->rows, p->h_stride))
        return MAMBA_SCAN_ERR_SHAPE;
    if (act != MAMBA_FFN_SILU && act != MAMBA_FFN_GELU_TANH) return MAMBA_SCAN_ERR_ARGS;
    if ((s->rows * s->dim > 0 && !p->x) || (s->hidden * s->dim > 0 && (!p->w_gate || !p->w_up)) ||
        (s->rows * s->hidden > 0 && !p->h))
        return MAMBA_SCAN_ERR_NULL;
    for (const void* q : {p->x, p->w_gate, p->w_up, (const void*)p->h})
        if (misaligned(q, 2)) return MAMBA_SCAN_ERR_ARGS;
    if (s->rows > 1 && p->h_stride < s->hidden) return MAMBA_SCAN_ERR_ARGS;
    if (ffn_too_wide(*s, p->x_stride, p->w_gate_stride, p->w_up_stride)) return MAMBA_SCAN_ERR_UNSUPPORTED;
    const int rc = check_workspace(p->workspace, p->workspace_bytes, mamba_gated_ffn_workspace_bytes(p, s));
    if (rc != MAMBA_SCAN_OK) return rc;
    const Bytes ins[] = {bytes_of(p->x, 2, 1, 0, s->rows, p->x_stride, s->dim),
                         bytes_of(p->w_gate, 2, 1, 0, s->hidden, p->w_gate_stride, s->dim),
                         bytes_of(p->w_up, 2, 1, 0, s->hidden, p->w_up_stride, s->dim),
                         flat(p->workspace, p->workspace_bytes)};
    const Bytes outs[] = {bytes_of(p->h, 2, 1, 0, s->rows, p->h_stride, s->hidden)};
    if (any_overlap(ins, outs)) return MAMBA_SCAN_ERR_ARGS;
    hipStream_t hs = static_cast<hipStream_t>(stream);
    if (s->rows * s->hidden == 0) return MAMBA_SCAN_OK;
    if (s->dim == 0) return launch_ffn_zero(p->h, s->rows, s->hidden, p->h_stride, hs);
    return launch_ffn_fwd(*p, *s, act, hs);
}

int mamba_gated_ffn_bwd(const mamba_ffn_bwd_ptrs* p, const mamba_ffn_shape* s, int act, mamba_scan_dtype dtype, void* stream) {
    if (!p || !s) return MAMBA_SCAN_ERR_NULL;
    if (dtype != MAMBA_SCAN_BF16) return dtype == MAMBA_SCAN_F32 ? MAMBA_SCAN_ERR_UNSUPPORTED : MAMBA_SCAN_ERR_DTYPE;
    if (ffn_bad_shape(*s)) return MAMBA_SCAN_ERR_SHAPE;
    if (bad_span(s->rows, p->x_stride) || bad_span(s->hidden, p->w_gate_stride) || bad_span(s->hidden, p->w_up_stride) ||
        bad_span(s->rows, p->dh_stride))
        return MAMBA_SCAN_ERR_SHAPE;
    if (act != MAMBA_FFN_SILU && act != MAMBA_FFN_GELU_TANH) return MAMBA_SCAN_ERR_ARGS;
    if ((s->rows * s->dim > 0 && (!p->x || !p->dx)) || (s->hidden * s->dim > 0 && (!p->w_gate || !p->w_up || !p->dw_gate || !p->dw_up)) ||
        (s->rows * s->hidden > 0 && !p->dh))
        return MAMBA_SCAN_ERR_NULL;
    for (const void* q : {p->x, p->w_gate, p->w_up, p->dh, (const void*)p->dx, (const void*)p->dw_gate, (const void*)p->dw_up})
        if (misaligned(q, 2)) return MAMBA_SCAN_ERR_ARGS;
    if (ffn_too_wide(*s, p->x_stride, p->w_gate_stride, p->w_up_stride)) return MAMBA_SCAN_ERR_UNSUPPORTED;
    const int rc = check_workspace(p->workspace, p->workspace_bytes, mamba_gated_ffn_bwd_workspace_bytes(s));
    if (rc != MAMBA_SCAN_OK) return rc;
    const Bytes ins[] = {bytes_of(p->x, 2, 1, 0, s->rows, p->x_stride, s->dim),
                         bytes_of(p->w_gate, 2, 1, 0, s->hidden, p->w_gate_stride, s->dim),
                         bytes_of(p->w_up, 2, 1, 0, s->hidden, p->w_up_stride, s->dim),
                         bytes_of(p->dh, 2, 1, 0, s->rows, p->dh_stride, s->hidden), flat(p->workspace, p->workspace_bytes)};
    const Bytes outs[] = {flat(p->dx, s->rows * s->dim * 2), flat(p->dw_gate, s->hidden * s->dim * 2),
                          flat(p->dw_up, s->hidden * s->dim * 2)};
    if (any_overlap(ins, outs)) return MAMBA_SCAN_ERR_ARGS;
    hipStream_t hs = static_cast<hipStream_t>(stream);
    if (s->rows == 0 || s->hidden == 0 || s->dim == 0) {
        int e = launch_ffn_zero(p->dx, s->rows, s->dim, s->dim, hs);
        if (e == MAMBA_SCAN_OK) e = launch_ffn_zero(p->dw_gate, s->hidden, s->dim, s->dim, hs);
        return e == MAMBA_SCAN_OK ? launch_ffn_zero(p->dw_up, s->hidden, s->dim, s->dim, hs) : e;
    }
    return launch_ffn_bwd(*p, *s, act, hs);
}

}  // extern "C"
