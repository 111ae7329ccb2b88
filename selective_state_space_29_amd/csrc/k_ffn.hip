// Gated feed-forward block up to its product (mamba_layers.h) and its gradient on gfx950, bf16.
//
//   h = act(g) u,  g = x Wg^T, u = x Wu^T          dg = dh u act'(g), du = dh act(g)
//   dx = dg Wg + du Wu;   dWg = dg^T x;   dWu = du^T x
//
// One matrix kernel, C[p][q] = sum_c X(p, c) Y(q, c), serves all products. A workgroup of 8 waves computes
// a tile of 256 x 256 (or 256 x 192; 4 waves 128 x 128): it loads 64 steps of c of both operands straight
// into LDS, a stage ahead of the one its waves multiply (v_mfma_f32_16x16x32_bf16, fp32 sums); workgroups of
// 128 x 128 that have a CU to themselves, three stages ahead (64 rows, dim 2048, hidden 8192, forward and
// backward: 102 us, 112 one stage ahead). An operand lies with c contiguous (x and the weights in the forward
// product) or with c as its rows (the weights in dx; both operands in dW); the latter is read from LDS with
// the transposing ds_read_b64_tr_b16, so no operand is ever transposed in memory. 16-byte chunks lie in LDS
// at an index XORed with their row, so that the reads of both kinds meet no bank twice; the lanes of a load
// into LDS fill consecutive places, so each lane loads the chunk whose place it fills. The rows of the MFMA
// are the q's: a lane then holds 4 consecutive q of one p, and a tile's results pass through the LDS that its
// stages no longer need, so that whole rows are stored 16 bytes a lane.
//
// The forward tile holds 128 or 64 hidden units' gate rows and the same units' up rows, so that both
// projections of a unit meet in the same lane and only h is written. The backward pass recomputes g and
// u the same way (keeping them in fp32 would move more bytes than the product takes) and rounds dg and
// du to bf16 once, as the operands of the other two products.
//
// Measured at 16384 rows, dim 768, hidden 2048 (103 GFLOP a product): forward 119 us, dg and du 150, dx 99,
// dW 113 and 12 for the join of its splits, 0.7 to 1.0 PFLOP/s; at 8192 rows, dim 4096, hidden 4096 the
// forward product reaches 1.27, where a library's plain product of 8192 x 8192 x 8192 reaches 1.4 with the
// clock at its power limit. Tiles loaded through registers took 130 us (forward) and 165 (dg and du);
// 128 x 256 with two workgroups a CU, and one wave's fragments read a half stage ahead, were slower. At
// dim 768 a tile has 12 stages, and filling the first and storing the results cost as much as 3.
//
// Operands whose rows are not 16-byte aligned or not a multiple of 8 long are first copied into padded
// rows of the workspace.
#include "layers_common.hpp"
#include "layers_launch.hpp"
#include "mat.hpp"

namespace mscan {

namespace {

template <int TP, int TQ, int WP, int WQ, int DEPTH, bool XTR, bool YTR, int EPI>
__global__ __launch_bounds__(WP * WQ * 64) __attribute__((amdgpu_waves_per_eu(DEPTH > 2 ? 1 : 2))) void ffn_mat_kernel(MatArgs m) {
    mat_tile<TP, TQ, WP, WQ, DEPTH, XTR, YTR, EPI>(m);
}

// ---- few rows ----
//
// The forward product of up to kFewRows rows: every weight is used once or a few times, so it goes from
// memory straight into the MFMA operand of the lane that loads it. A workgroup takes 16 hidden units, its
// 8 waves take stretches of 64 c in turn (128 bytes of each weight row: a lane 16 c of one unit's gate and
// up rows, in two steps of the MFMA, whose order of c is the same in both operands and otherwise free), and
// their sums meet in LDS, added in the waves' order. Loads need no alignment, so no operand is copied.
//
// Bound by the weights' bytes: 8 rows, dim 2048, hidden 8192 read 67 MB in 12.6 us, 5.3 TB/s (the tiles
// above take 24: 128 of them on 256 CUs). Up to 48 rows, as x is read again by every 16 units: with the
// call's host side, few rows against tiles, 16 rows 16.6 and 26.6 us, 32 rows 20 and 26.7, 48 rows 25.5 and
// 27.0 (dim 4096, hidden 11008: 69.5 and 67.8), 64 rows 29.6 and 27.1.
constexpr int kFewRows = 16 * 3, kFewUnits = 16, kFewWaves = 8, kFewC = 64, kFewAhead = 4;

__device__ __forceinline__ bf16x8 load_any(const uint16_t* p) {
    bf16x8 v;
    __builtin_memcpy(&v, p, 16);
    return v;
}

template <int NR>
__global__ __launch_bounds__(kFewWaves * 64) void ffn_few_kernel(MatArgs m) {
    __shared__ float sums[kFewWaves][2][NR * 256];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t f0 = (int64_t)blockIdx.x * kFewUnits;

    // rows past the last repeat it: their products are not stored, and none enters another's
    const int row = lane & 15, at = (lane >> 4) * 16;
    const int64_t f = f0 + row < m.Q ? f0 + row : m.Q - 1;
    const uint16_t* w[2] = {m.y[0] + f * m.y_stride + at, m.y[1] + f * m.up_stride + at};
    const uint16_t* x[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const int64_t pr = r * 16 + row < m.P ? r * 16 + row : m.P - 1;
        x[r] = m.x + pr * m.x_stride + at;
    }

    f32x4 acc[2][NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) acc[0][r] = acc[1][r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto add = [&](const bf16x8 (&a)[2][2], const bf16x8 (&b)[NR][2]) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int g = 0; g < 2; ++g) acc[g][r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[g][k], b[r][k], acc[g][r], 0, 0, 0);
    };

    const int64_t whole = m.C / kFewC;
    for (int64_t u = wave; u < whole; u += kFewWaves * kFewAhead) {
        bf16x8 a[kFewAhead][2][2], b[kFewAhead][NR][2];
        // all loads of a round before its first product; a stretch past the end repeats the round's first
#pragma unroll
        for (int i = 0; i < kFewAhead; ++i) {
            const int64_t c = (u + i * kFewWaves < whole ? u + i * kFewWaves : u) * kFewC;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int g = 0; g < 2; ++g) a[i][g][k] = load_any(w[g] + c + k * 8);
            }
        }
#pragma unroll
        for (int i = 0; i < kFewAhead; ++i) {
            const int64_t c = (u + i * kFewWaves < whole ? u + i * kFewWaves : u) * kFewC;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int r = 0; r < NR; ++r) b[i][r][k] = load_any(x[r] + c + k * 8);
            }
        }
#pragma unroll
        for (int i = 0; i < kFewAhead; ++i)
            if (u + i * kFewWaves < whole) add(a[i], b[i]);
    }
    if (m.C % kFewC != 0 && wave == (int)(whole % kFewWaves)) {  // the last, part stretch value by value, zeros past its end
        const int64_t c = whole * kFewC;
        const int left = (int)(m.C - c) - at;  // of this lane's 16
        auto part = [&](const uint16_t* p, int k) __attribute__((always_inline)) {
            uint16_t v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int o = k * 8 + j < left ? k * 8 + j : left - 1;  // the row's last value, before this lane's 16 if none is left
                v[j] = p[c + o];
                if (k * 8 + j >= left) v[j] = 0;
            }
            bf16x8 r;
            __builtin_memcpy(&r, v, 16);
            return r;
        };
        bf16x8 a[2][2], b[NR][2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int g = 0; g < 2; ++g) a[g][k] = part(w[g], k);
#pragma unroll
            for (int r = 0; r < NR; ++r) b[r][k] = part(x[r], k);
        }
        add(a, b);
    }

#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int r = 0; r < NR; ++r) *reinterpret_cast<f32x4*>(&sums[wave][g][r * 256 + lane * 4]) = acc[g][r];
    __syncthreads();
    for (int e = tid; e < NR * 256; e += kFewWaves * 64) {
        float g = 0.0f, u = 0.0f;
#pragma unroll
        for (int k = 0; k < kFewWaves; ++k) g += sums[k][0][e], u += sums[k][1][e];
        const int l = e / 4 % 64;
        const int64_t pr = e / 256 * 16 + (l & 15), unit = f0 + 4 * (l >> 4) + e % 4;
        if (pr < m.P && unit < m.Q) m.out[pr * m.out_stride + unit] = to_bf16(act_of(g, m.act) * u).bits;
    }
}

// Zeros: the results of products over nothing.
__global__ __launch_bounds__(256) void ffn_zero_kernel(uint16_t* p, int64_t n, int64_t cols, int64_t stride) {
    for (int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x; k < n; k += (int64_t)gridDim.x * 256)
        p[k / cols * stride + k % cols] = 0;
}

// ---- plans ----

template <bool XTR, bool YTR, int EPI>
void run_mat(MatArgs m, const Tiling& t, Launches& on) {
    m.tiles_p = t.tiles_p, m.tiles_q = t.tiles_q, m.splits = t.splits;
    const dim3 grid((unsigned)(t.tiles_p * t.tiles_q), (unsigned)t.splits);
    if (t.tp == 128) {
        if (t.alone) on(ffn_mat_kernel<128, 128, 2, 2, 4, XTR, YTR, EPI>, grid, dim3(256), m);
        else on(ffn_mat_kernel<128, 128, 2, 2, 2, XTR, YTR, EPI>, grid, dim3(256), m);
        return;
    }
    if constexpr (EPI == kEpiStore || EPI == kEpiPartial) {
        if (t.tq == 192) {
            on(ffn_mat_kernel<256, 192, 2, 4, 2, XTR, YTR, EPI>, grid, dim3(512), m);
            return;
        }
    }
    on(ffn_mat_kernel<256, 256, 2, 4, 2, XTR, YTR, EPI>, grid, dim3(512), m);
}

template <bool XTR, bool YTR>
void run_product(const MatArgs& m, const Tiling& t, Launches& on) {
    if (t.splits == 1) {
        run_mat<XTR, YTR, kEpiStore>(m, t, on);
        return;
    }
    run_mat<XTR, YTR, kEpiPartial>(m, t, on);
    MatArgs j = m;
    j.splits = t.splits;
    const dim3 grid((unsigned)(m.P < 16384 ? m.P : 16384));
    if (m.Q % 4 == 0) on(mat_join_kernel<4>, grid, dim3(256), j);
    else on(mat_join_kernel<1>, grid, dim3(256), j);
}

bool needs_copy(const mamba_ffn_shape& s, const void* x, int64_t xs, const void* wg, int64_t gs, const void* wu, int64_t us) {
    return s.dim % 8 || !row_aligned(x, xs, s.rows) || !row_aligned(wg, gs, s.hidden) || !row_aligned(wu, us, s.hidden) ||
           (s.hidden > 1 && gs != us);
}

struct Operands {
    const uint16_t *x, *wg, *wu;
    int64_t xs, ws, dim8;  // row strides; the contraction length rounded up to 8
};

int64_t copy_bytes(const mamba_ffn_shape& s) { return align256(s.rows * up(s.dim, 8) * 2) + 2 * align256(s.hidden * up(s.dim, 8) * 2); }

Operands operands(const mamba_ffn_shape& s, const void* x, int64_t xs, const void* wg, int64_t gs, const void* wu, int64_t us,
                  char* ws, Launches& on) {
    Operands o{static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(wg), static_cast<const uint16_t*>(wu), xs, gs, s.dim};
    if (!needs_copy(s, x, xs, wg, gs, wu, us)) return o;
    MatCopy c{};
    c.cols = s.dim, c.wide = up(s.dim, 8);
    uint16_t* to = reinterpret_cast<uint16_t*>(ws);
    const int64_t xb = align256(s.rows * c.wide * 2) / 2, wb = align256(s.hidden * c.wide * 2) / 2;
    c.src[0] = o.x, c.dst[0] = to, c.rows[0] = s.rows, c.stride[0] = xs;
    c.src[1] = o.wg, c.dst[1] = to + xb, c.rows[1] = s.hidden, c.stride[1] = gs;
    c.src[2] = o.wu, c.dst[2] = to + xb + wb, c.rows[2] = s.hidden, c.stride[2] = us;
    const int64_t n = s.rows > s.hidden ? s.rows : s.hidden;
    on(mat_copy_kernel, dim3((unsigned)(n < 32768 ? (n + 3) / 4 : 8192), 3), dim3(256), c);
    o.x = c.dst[0], o.wg = c.dst[1], o.wu = c.dst[2], o.xs = o.ws = o.dim8 = c.wide;
    return o;
}

MatArgs dual_mat(const mamba_ffn_shape& s, const Operands& o, int act) {
    MatArgs m{};
    m.x = o.x, m.y[0] = o.wg, m.y[1] = o.wu, m.x_stride = o.xs, m.y_stride = o.ws;
    m.P = s.rows, m.Q = s.hidden, m.C = o.dim8, m.x_cols = o.dim8;
    m.steps = steps_of(o.dim8), m.stretches = 1, m.act = act;
    return m;
}

struct BwdPlan {
    Tiling dual, dx, dw;
    int64_t fp, copy, d, part, total;  // padded hidden units; workspace offsets
};

BwdPlan bwd_plan(const mamba_ffn_shape& s) {
    BwdPlan b;
    b.fp = up(s.hidden, kTC);
    b.dual = tiling(s.rows, b.fp, true, steps_of(s.dim), false);
    b.dx = tiling(s.rows, s.dim, false, 2 * steps_of(s.hidden), true);
    b.dw = tiling(2 * b.fp, s.dim, false, steps_of(s.rows), true);
    b.copy = 0;  // room for the copies whether or not the call needs them: the size depends on the shape alone
    b.d = copy_bytes(s);
    b.part = b.d + align256(s.rows * 2 * b.fp * 2);
    const int64_t p1 = b.dx.splits > 1 ? b.dx.splits * s.rows * s.dim * 4 : 0;
    const int64_t p2 = b.dw.splits > 1 ? b.dw.splits * 2 * b.fp * s.dim * 4 : 0;
    b.total = b.part + align256(p1 > p2 ? p1 : p2);
    return b;
}

}  // namespace

int launch_ffn_zero(void* p, int64_t rows, int64_t cols, int64_t stride, hipStream_t stream) {
    const int64_t n = rows * cols;
    if (n <= 0) return MAMBA_SCAN_OK;
    const int64_t g = (n + 255) / 256;
    Launches on(stream);
    on(ffn_zero_kernel, dim3((unsigned)(g < 4096 ? g : 4096)), dim3(256), static_cast<uint16_t*>(p), n, cols, stride);
    return on.status;
}

int64_t ffn_workspace(const mamba_ffn_ptrs& p, const mamba_ffn_shape& s) {
    if (s.rows <= kFewRows) return 0;
    return needs_copy(s, p.x, p.x_stride, p.w_gate, p.w_gate_stride, p.w_up, p.w_up_stride) ? copy_bytes(s) : 0;
}

int64_t ffn_bwd_workspace(const mamba_ffn_shape& s) { return bwd_plan(s).total; }

int launch_ffn_fwd(const mamba_ffn_ptrs& p, const mamba_ffn_shape& s, int act, hipStream_t stream) {
    Launches on(stream);
    if (s.rows <= kFewRows) {
        MatArgs m{};
        m.x = static_cast<const uint16_t*>(p.x), m.x_stride = p.x_stride;
        m.y[0] = static_cast<const uint16_t*>(p.w_gate), m.y_stride = p.w_gate_stride;
        m.y[1] = static_cast<const uint16_t*>(p.w_up), m.up_stride = p.w_up_stride;
        m.P = s.rows, m.Q = s.hidden, m.C = s.dim, m.act = act;
        m.out = static_cast<uint16_t*>(p.h), m.out_stride = p.h_stride;
        const dim3 grid((unsigned)((s.hidden + kFewUnits - 1) / kFewUnits)), block(kFewWaves * 64);
        if (s.rows <= 16)
            on(ffn_few_kernel<1>, grid, block, m);
        else if (s.rows <= 32)
            on(ffn_few_kernel<2>, grid, block, m);
        else
            on(ffn_few_kernel<3>, grid, block, m);
        return on.status;
    }
    const Operands o = operands(s, p.x, p.x_stride, p.w_gate, p.w_gate_stride, p.w_up, p.w_up_stride,
                                static_cast<char*>(p.workspace), on);
    MatArgs m = dual_mat(s, o, act);
    m.out = static_cast<uint16_t*>(p.h), m.out_stride = p.h_stride;
    run_mat<false, false, kEpiDual>(m, tiling(s.rows, s.hidden, true, m.steps, false), on);
    return on.status;
}

int launch_ffn_bwd(const mamba_ffn_bwd_ptrs& p, const mamba_ffn_shape& s, int act, hipStream_t stream) {
    Launches on(stream);
    const BwdPlan b = bwd_plan(s);
    char* ws = static_cast<char*>(p.workspace);
    const Operands o = operands(s, p.x, p.x_stride, p.w_gate, p.w_gate_stride, p.w_up, p.w_up_stride, ws + b.copy, on);
    uint16_t* d = reinterpret_cast<uint16_t*>(ws + b.d);
    MatArgs m = dual_mat(s, o, act);
    m.dh = static_cast<const uint16_t*>(p.dh), m.dh_stride = p.dh_stride, m.d = d, m.seg_rows = b.fp;
    run_mat<false, false, kEpiDualBwd>(m, b.dual, on);

    MatArgs x{};  // dx[p][q] = sum over gate and up units c of d[p][c] W[c][q]
    x.x = d, x.x_stride = 2 * b.fp, x.x_cols = b.fp, x.x_seg = b.fp;
    x.y[0] = o.wg, x.y[1] = o.wu, x.y_stride = o.ws;
    x.P = s.rows, x.Q = s.dim, x.C = s.hidden;
    x.steps = steps_of(s.hidden), x.stretches = 2;
    x.out = x.out2 = static_cast<uint16_t*>(p.dx), x.out_stride = s.dim, x.seg_rows = x.seg_valid = s.rows;
    x.part = reinterpret_cast<float*>(ws + b.part);
    run_product<false, true>(x, b.dx, on);

    MatArgs w{};  // dW[f][q] = sum over tokens c of d[c][f] x[c][q]
    w.x = d, w.x_stride = 2 * b.fp;
    w.y[0] = w.y[1] = o.x, w.y_stride = o.xs;
    w.P = 2 * b.fp, w.Q = s.dim, w.C = s.rows;
    w.steps = steps_of(s.rows), w.stretches = 1;
    w.out = static_cast<uint16_t*>(p.dw_gate), w.out2 = static_cast<uint16_t*>(p.dw_up), w.out_stride = s.dim;
    w.seg_rows = b.fp, w.seg_valid = s.hidden;
    w.part = reinterpret_cast<float*>(ws + b.part);
    run_product<true, true>(w, b.dw, on);
    return on.status;
}

}  // namespace mscan
