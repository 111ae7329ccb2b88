// Cross entropy of hidden states against a large output matrix (mamba_block.h) and its gradient on gfx950, bf16.
//
//   l = scale x W^T;  lse = log sum_v exp(l_v);  loss = lse - l[target]
//   dl = (a + dlse) exp(l - lse) - a [target];   dx = scale dl W;   dW = scale dl^T x
//
// No logit is stored. Forward: the matrix kernel's tiles of 128 or 256 columns of the vocabulary end in each
// row's largest logit and sum of exponentials over their columns, and a second kernel joins a row's tiles; the tile
// that holds a row's target writes that logit, and the loss is the difference of the two logits and the sum's logarithm.
// Backward: piece by piece of the vocabulary the logits are computed
// again and end as dl (scale folded into the row's factors), rounded to bf16 as the operand of the other two
// products, whose inputs have 8 bits as well; dl of a piece is what the workspace holds. dx is summed in fp32 over
// the pieces, one after another, and rounded once behind the last.
//
// Bound by the matrix cores. 16384 x 768, vocabulary 50000: forward 1175 to 1220 us (1.03 to 1.07 PFLOP/s; the library's
// plain product of this size 1298); backward, 7 pieces: logits' gradients 194 to 206 each (0.88 to 0.93), dx 174 to 187
// (0.96 to 1.03; library 0.92 to 1.03), dW 161 to 172 (1.05 to 1.12) and its join 12.2. 64 rows: 16.7 us for the matrix's
// 77 MB (4.6 TB/s), 4.2 for the join.
//
// The rows of dl that take no part are zeros, and so are those rows in the copy of x that the backward
// multiplies with them: nothing that padding holds reaches dW.
#include "block_launch.hpp"
#include "layers_common.hpp"
#include "layers_launch.hpp"
#include "mat.hpp"
#include "rows.hpp"

namespace mscan {

namespace {

template <int TP, int TQ, int WP, int WQ, int DEPTH, bool XTR, bool YTR, int EPI>
__global__ __launch_bounds__(WP * WQ * 64) __attribute__((amdgpu_waves_per_eu(DEPTH > 2 ? 1 : 2))) void xent_mat_kernel(MatArgs m) {
    mat_tile<TP, TQ, WP, WQ, DEPTH, XTR, YTR, EPI>(m);
}

__device__ __forceinline__ int64_t target_of(const void* target, int target64, int64_t row) {
    return target64 ? static_cast<const int64_t*>(target)[row] : static_cast<const int32_t*>(target)[row];
}

// A row's tiles joined in order: 16 rows (a line of a tile's pairs) x 64 stretches of the tiles a workgroup. (Few rows
// have as many tiles as many: 64 rows x 391 tiles by 4 stretches took 9.7 us.)
constexpr int kJoinRows = 16, kJoinWays = 64;

__global__ __launch_bounds__(kJoinRows * kJoinWays) void xent_join_kernel(const float2* part, int tiles, int64_t rows, const float* at_target,
                                                                        const void* target, int target64, int64_t vocab, float* loss,
                                                                        float* lse) {
    __shared__ float2 sums[kJoinWays / 4][kJoinRows];
    const int r = threadIdx.x % kJoinRows, way = threadIdx.x / kJoinRows;
    const int64_t row = grid_block() * kJoinRows + r, at = row < rows ? row : rows - 1;  // (2^26 rows and more: 2^32 threads)
    const int per = (tiles + kJoinWays - 1) / kJoinWays, k0 = way * per, k1 = k0 + per < tiles ? k0 + per : tiles;
    float2 v = make_float2(-__builtin_inff(), 0.0f);
    for (int k = k0; k < k1; k += 4) {
        float2 p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = part[(int64_t)(k + i < k1 ? k + i : k1 - 1) * rows + at];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (k + i < k1) v = join_pair(v, p[i]);
    }
    v = join_pair(v, make_float2(__shfl_xor(v.x, 16), __shfl_xor(v.y, 16)));
    v = join_pair(v, make_float2(__shfl_xor(v.x, 32), __shfl_xor(v.y, 32)));
    if ((threadIdx.x & 63) < kJoinRows) sums[threadIdx.x >> 6][r] = v;
    __syncthreads();
    if (threadIdx.x >= kJoinRows || row >= rows) return;
#pragma unroll
    for (int k = 1; k < kJoinWays / 4; ++k) v = join_pair(v, sums[k][r]);
    const float s = hw_log2(v.y) * kLn2;
    if (lse) lse[row] = v.x + s;
    if (loss) {  // (a difference of logits, and the rest: the largest cancels whole)
        const int64_t t = target_of(target, target64, row);
        loss[row] = t >= 0 && t < vocab ? v.x - at_target[row] + s : 0.0f;
    }
}

// The sum of the rows' losses and the number of their targets: one workgroup, each thread's rows in order, then
// the lanes and waves in theirs.
__global__ __launch_bounds__(1024) void xent_total_kernel(const float* loss, const void* target, int target64, int64_t rows,
                                                          int64_t vocab, float* total) {
    __shared__ float sums[2][16];
    float s = 0.0f;
    int n = 0;  // (counts up to 2^24 are exact in fp32, more to its precision)
#pragma unroll 8
    for (int64_t r = threadIdx.x; r < rows; r += 1024) {
        const int64_t t = target_of(target, target64, r);
        s += loss[r];
        n += t >= 0 && t < vocab;
    }
    s = wave_sum(s);
    const float c = wave_sum((float)n);
    if ((threadIdx.x & 63) == 0) sums[0][threadIdx.x >> 6] = s, sums[1][threadIdx.x >> 6] = c;
    __syncthreads();
    if (threadIdx.x < 2) {
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < 16; ++k) v += sums[threadIdx.x][k];
        total[threadIdx.x] = v;
    }
}

// What the backward needs of each row, and x in padded rows, zeros where a row takes no part. A wave a row.
//
// The logits' gradients are rounded to bf16 as operands. Where every row with a target has the same factor, as in a mean
// or a sum, the factor is left out of them and multiplied with the products' sums in fp32: of a target's entry p - 1 is
// rounded instead of (p - 1) factor, and for most rows that is next to 1. (Errors of dx and dW against 64 bits, of whose
// norm their own rounding is 0.00166: up to 0.0026 with the factor in the operands, where its rounding is the same in every
// row, and 0.0017 to 0.0021 without.)
struct XentRows {
    const uint16_t* x;
    const void* target;
    const float* lse;
    const float* dloss;
    const float* dlse;
    f32x4* row;
    uint16_t* copy;
    f32x4* part;   // (parts): extremes of the factors; none where one value of dloss stands for all and there is no dlse
    float* factor;
    int64_t rows, dim, wide, vocab, sx, sloss, slse;
    int target64, parts;
    float scale;
};

// The factors of a row's target and of its softmax, from the gradients at its loss (where it has a target) and its lse.
__device__ __forceinline__ void factors_of(const XentRows& p, bool hit, float dloss, float dlse, float& a, float& f) {
    a = hit ? dloss * p.scale : 0.0f;
    f = a + dlse * p.scale;
}

// The smallest and largest of the targets' factors that are not 0, and the same of the softmax's, over a workgroup.
template <int WAVES>
__device__ __forceinline__ f32x4 extremes(f32x4 v) {
    __shared__ f32x4 all[WAVES];
    auto join = [](f32x4 p, f32x4 q) {
        return f32x4{__builtin_fminf(p[0], q[0]), __builtin_fmaxf(p[1], q[1]), __builtin_fminf(p[2], q[2]), __builtin_fmaxf(p[3], q[3])};
    };
#pragma unroll
    for (int far = 1; far < 64; far *= 2)
        v = join(v, f32x4{__shfl_xor(v[0], far), __shfl_xor(v[1], far), __shfl_xor(v[2], far), __shfl_xor(v[3], far)});
    if ((threadIdx.x & 63) == 0) all[threadIdx.x >> 6] = v;
    __syncthreads();
    v = all[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) v = join(v, all[w]);
    return v;
}

// The extremes of every parts-th stretch of rows. A thread's loads are all on their way before it uses one (16384 rows
// in one workgroup, row by row: 17 us).
constexpr int kFactorAhead = 8, kFactorRows = 1024 * kFactorAhead, kFactorParts = 256;

__global__ __launch_bounds__(1024) void xent_factor_kernel(XentRows p) {
    f32x4 v = {__builtin_inff(), 0.0f, __builtin_inff(), 0.0f};
    for (int64_t r0 = (int64_t)blockIdx.x * kFactorRows + threadIdx.x; r0 < p.rows; r0 += (int64_t)p.parts * kFactorRows) {
        int64_t t[kFactorAhead];
        float g[kFactorAhead], e[kFactorAhead];
        auto row = [&](int i) __attribute__((always_inline)) {  // (behind the last one, that one again)
            return r0 + 1024 * i < p.rows ? r0 + 1024 * i : p.rows - 1;
        };
#pragma unroll
        for (int i = 0; i < kFactorAhead; ++i) t[i] = -1, g[i] = e[i] = 0.0f;
        if (p.dloss) {
            if (p.target64) {
#pragma unroll
                for (int i = 0; i < kFactorAhead; ++i) t[i] = static_cast<const int64_t*>(p.target)[row(i)];
            } else {
#pragma unroll
                for (int i = 0; i < kFactorAhead; ++i) t[i] = static_cast<const int32_t*>(p.target)[row(i)];
            }
#pragma unroll
            for (int i = 0; i < kFactorAhead; ++i) g[i] = p.dloss[row(i) * p.sloss];
        }
        if (p.dlse) {
#pragma unroll
            for (int i = 0; i < kFactorAhead; ++i) e[i] = p.dlse[row(i) * p.slse];
        }
#pragma unroll
        for (int i = 0; i < kFactorAhead; ++i) {
            float of[2];
            factors_of(p, t[i] >= 0 && t[i] < p.vocab, g[i], e[i], of[0], of[1]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {  // a NaN or an infinity counts as one
                const float m = __builtin_fabsf(of[k]) < __builtin_inff() ? __builtin_fabsf(of[k]) : __builtin_inff();
                if (m != 0.0f) v[2 * k] = __builtin_fminf(v[2 * k], m), v[2 * k + 1] = __builtin_fmaxf(v[2 * k + 1], m);
            }
        }
    }
    v = extremes<16>(v);
    if (threadIdx.x == 0) p.part[blockIdx.x] = v;
}

__global__ __launch_bounds__(256) void xent_rows_kernel(XentRows p) {
    // the targets' common factor, or 1: where they differ, and where a softmax's factor is so far from it that the quotient
    // might leave fp32's range
    float by;
    if (p.parts == 0) {  // one value for all
        by = __builtin_fabsf(*p.dloss * p.scale);
        by = by > 0.0f && by < __builtin_inff() ? by : 1.0f;
    } else {
        static_assert(kFactorParts <= 256);
        const f32x4 v = extremes<4>((int)threadIdx.x < p.parts ? p.part[threadIdx.x] : f32x4{__builtin_inff(), 0.0f, __builtin_inff(), 0.0f});
        by = v[0] == v[1] && v[1] < __builtin_inff() && v[2] >= v[1] * 0x1p-64f && v[3] <= v[1] * 0x1p64f ? v[1] : 1.0f;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.factor = by;
    for (int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); r < p.rows; r += (int64_t)gridDim.x * 4) {
        const int64_t t = p.target ? target_of(p.target, p.target64, r) : -1;
        const bool hit = t >= 0 && t < p.vocab && p.dloss;
        float a, f;
        factors_of(p, hit, hit ? p.dloss[r * p.sloss] : 0.0f, p.dlse ? p.dlse[r * p.slse] : 0.0f, a, f);
        a /= by, f /= by;
        // 2^(l log2(e) - top) f 2^(top - lse log2(e)), top the rounded lse log2(e)
        const float top = p.lse[r] * kLog2e, rest = __builtin_fmaf(p.lse[r], kLog2e, -top);
        const float above = __builtin_fabsf(top) < __builtin_inff() ? f * hw_exp2(-rest) : f;
        if ((threadIdx.x & 63) == 0) p.row[r] = f32x4{top, above, a, __builtin_bit_cast(float, hit ? (int)t : -1)};
        const bool on = a != 0.0f || f != 0.0f;
        for (int64_t c = (int64_t)(threadIdx.x & 63) * 8; c < p.wide; c += 64 * 8) {
            const Pack<uint16_t, 8> v = load_some<uint16_t, 8>(p.x + r * p.sx + c, on ? (int)(p.dim - c) : 0);
            u32x4 w;
            __builtin_memcpy(&w, &v, 16);
            *reinterpret_cast<u32x4*>(p.copy + r * p.wide + c) = w;
        }
    }
}

template <bool XTR, bool YTR, int EPI>
void run_mat(MatArgs m, const Tiling& t, Launches& on) {
    m.tiles_p = t.tiles_p, m.tiles_q = t.tiles_q, m.splits = t.splits;
    const dim3 grid((unsigned)(t.tiles_p * t.tiles_q), (unsigned)t.splits);
    if (t.tp == 128) {
        if (t.alone) on(xent_mat_kernel<128, 128, 2, 2, 4, XTR, YTR, EPI>, grid, dim3(256), m);
        else on(xent_mat_kernel<128, 128, 2, 2, 2, XTR, YTR, EPI>, grid, dim3(256), m);
    } else if (t.tq == 192) {
        on(xent_mat_kernel<256, 192, 2, 4, 2, XTR, YTR, EPI>, grid, dim3(512), m);
    } else {
        on(xent_mat_kernel<256, 256, 2, 4, 2, XTR, YTR, EPI>, grid, dim3(512), m);
    }
}

void run_join(MatArgs m, int splits, Launches& on) {
    m.splits = splits;
    const dim3 grid((unsigned)(m.P < 16384 ? m.P : 16384));
    if (m.Q % 4 == 0) on(mat_join_kernel<4>, grid, dim3(256), m);
    else on(mat_join_kernel<1>, grid, dim3(256), m);
}

bool copies(const void* p, int64_t stride, int64_t rows, int64_t dim) { return dim % 8 != 0 || !row_aligned(p, stride, rows); }

void copy_rows(const uint16_t* src, int64_t stride, uint16_t* dst, int64_t rows, int64_t cols, Launches& on) {
    MatCopy c{};
    c.src[0] = src, c.dst[0] = dst, c.rows[0] = rows, c.stride[0] = stride, c.cols = cols, c.wide = up(cols, 8);
    on(mat_copy_kernel, dim3((unsigned)(rows < 32768 ? (rows + 3) / 4 : 8192), 1), dim3(256), c);
}

// Workspace of the forward: copies of operands whose rows are not aligned, each row's target's logit, the tiles' pairs.
struct FwdPlan {
    Tiling t;
    bool copy_x, copy_w;
    int64_t x, w, at, part, total;
};
FwdPlan fwd_plan(const mamba_xent_ptrs& p, const mamba_xent_shape& s) {
    FwdPlan f;
    f.t = tiling(s.rows, s.vocab, false, steps_of(up(s.dim, 8)), false);
    f.copy_x = copies(p.x, p.x_stride, s.rows, s.dim), f.copy_w = copies(p.weight, p.weight_stride, s.vocab, s.dim);
    f.x = 0;
    f.w = f.x + (f.copy_x ? align256(s.rows * up(s.dim, 8) * 2) : 0);
    f.at = f.w + (f.copy_w ? align256(s.vocab * up(s.dim, 8) * 2) : 0);
    f.part = f.at + align256(s.rows * 4);
    f.total = f.part + align256((int64_t)f.t.tiles_q * s.rows * 8);
    return f;
}

// Bytes of dl that a piece of the vocabulary may take, and its least width.
constexpr int64_t kPieceBytes = (int64_t)256 << 20, kPieceLeast = 1024;

struct BwdPlan {
    bool copy_w;
    int64_t width, pieces;  // columns of a piece
    Tiling tx;              // of dx, the same for every piece
    int64_t row, factor, part, x, w, d, dx, dw, total;
};

int64_t piece_of(const mamba_xent_shape& s) {
    const int64_t fit = kPieceBytes / (s.rows * 2), most = fit < 1 ? 1 : fit, n = (s.vocab + most - 1) / most;
    int64_t width = up((s.vocab + n - 1) / n, 256);
    if (width < kPieceLeast) width = kPieceLeast;
    return width < up(s.vocab, 256) ? width : up(s.vocab, 256);
}

Tiling dw_tiling(const mamba_xent_shape& s, int64_t width) { return tiling(up(width, kTC), s.dim, false, steps_of(s.rows), true); }

BwdPlan bwd_plan(const mamba_xent_bwd_ptrs& p, const mamba_xent_shape& s) {
    BwdPlan b;
    b.copy_w = copies(p.weight, p.weight_stride, s.vocab, s.dim);
    b.width = piece_of(s);
    b.pieces = (s.vocab + b.width - 1) / b.width;
    b.tx = tiling(s.rows, s.dim, false, steps_of(b.width < s.vocab ? b.width : s.vocab), true);
    int64_t dw = 0;
    for (int64_t k = 0; k < (p.dweight ? b.pieces : 0); ++k) {
        const int64_t width = s.vocab - k * b.width < b.width ? s.vocab - k * b.width : b.width;
        const int splits = dw_tiling(s, width).splits;
        if (splits > 1 && splits * up(width, kTC) > dw) dw = splits * up(width, kTC);
    }
    b.row = 0;
    b.factor = b.row + align256(s.rows * 16);
    b.part = b.factor + 256;
    b.x = b.part + kFactorParts * 16;
    b.w = b.x + align256(s.rows * up(s.dim, 8) * 2);
    b.d = b.w + (b.copy_w ? align256(s.vocab * up(s.dim, 8) * 2) : 0);
    b.dx = b.d + align256(s.rows * b.width * 2);
    b.dw = b.dx + (p.dx && (b.pieces > 1 || b.tx.splits > 1) ? align256(b.tx.splits * s.rows * s.dim * 4) : 0);
    b.total = b.dw + align256(dw * s.dim * 4);
    return b;
}

}  // namespace

int64_t xent_workspace(const mamba_xent_ptrs& p, const mamba_xent_shape& s) { return fwd_plan(p, s).total; }
int64_t xent_bwd_workspace(const mamba_xent_bwd_ptrs& p, const mamba_xent_shape& s) { return bwd_plan(p, s).total; }

int launch_xent_fwd(const mamba_xent_ptrs& p, const mamba_xent_shape& s, bool target64, float scale, hipStream_t stream) {
    Launches on(stream);
    const FwdPlan f = fwd_plan(p, s);
    char* ws = static_cast<char*>(p.workspace);
    MatArgs m{};
    m.x = static_cast<const uint16_t*>(p.x), m.x_stride = p.x_stride;
    m.y[0] = m.y[1] = static_cast<const uint16_t*>(p.weight), m.y_stride = p.weight_stride;
    const int64_t wide = up(s.dim, 8);
    if (f.copy_x) {
        uint16_t* to = reinterpret_cast<uint16_t*>(ws + f.x);
        if (s.dim > 0) copy_rows(m.x, m.x_stride, to, s.rows, s.dim, on);
        m.x = to, m.x_stride = wide;
    }
    if (f.copy_w) {
        uint16_t* to = reinterpret_cast<uint16_t*>(ws + f.w);
        if (s.dim > 0) copy_rows(m.y[0], m.y_stride, to, s.vocab, s.dim, on);
        m.y[0] = m.y[1] = to, m.y_stride = wide;
    }
    m.P = s.rows, m.Q = s.vocab, m.C = m.x_cols = wide, m.steps = steps_of(wide), m.stretches = 1;
    m.scale = scale, m.target = p.loss ? p.target : nullptr, m.target64 = target64;
    m.at_target = reinterpret_cast<float*>(ws + f.at), m.part = reinterpret_cast<float*>(ws + f.part);
    run_mat<false, false, kEpiLse>(m, f.t, on);
    on(xent_join_kernel, grid_of((s.rows + kJoinRows - 1) / kJoinRows, kJoinRows * kJoinWays), dim3(kJoinRows * kJoinWays),
       reinterpret_cast<const float2*>(m.part), f.t.tiles_q, s.rows, static_cast<const float*>(m.at_target), p.target, (int)target64, s.vocab, p.loss, p.lse);
    if (p.total) on(xent_total_kernel, dim3(1), dim3(1024), static_cast<const float*>(p.loss), p.target, (int)target64, s.rows, s.vocab, p.total);
    return on.status;
}

int launch_xent_bwd(const mamba_xent_bwd_ptrs& p, const mamba_xent_shape& s, bool target64, float scale, hipStream_t stream) {
    Launches on(stream);
    const BwdPlan b = bwd_plan(p, s);
    char* ws = static_cast<char*>(p.workspace);
    const int64_t wide = up(s.dim, 8);
    uint16_t* x = reinterpret_cast<uint16_t*>(ws + b.x);
    uint16_t* d = reinterpret_cast<uint16_t*>(ws + b.d);
    XentRows r{static_cast<const uint16_t*>(p.x), p.target, p.lse, p.dloss, p.dlse, reinterpret_cast<f32x4*>(ws + b.row), x,
               reinterpret_cast<f32x4*>(ws + b.part), reinterpret_cast<float*>(ws + b.factor), s.rows, s.dim, wide, s.vocab,
               p.x_stride, p.dloss_stride, p.dlse_stride, (int)target64, 0, scale};
    if (!p.dloss || p.dloss_stride != 0 || p.dlse) {
        const int64_t parts = (s.rows + kFactorRows - 1) / kFactorRows;
        r.parts = (int)(parts < kFactorParts ? parts : kFactorParts);
        on(xent_factor_kernel, dim3((unsigned)r.parts), dim3(1024), r);
    }
    on(xent_rows_kernel, dim3((unsigned)(s.rows < 32768 ? (s.rows + 3) / 4 : 8192)), dim3(256), r);
    const uint16_t* w = static_cast<const uint16_t*>(p.weight);
    int64_t ws_row = p.weight_stride;
    if (b.copy_w) {
        uint16_t* to = reinterpret_cast<uint16_t*>(ws + b.w);
        copy_rows(w, ws_row, to, s.vocab, s.dim, on);
        w = to, ws_row = wide;
    }
    MatArgs gx{};
    const bool one = b.pieces == 1 && b.tx.splits == 1;
    for (int64_t k = 0; k < b.pieces; ++k) {
        const int64_t v0 = k * b.width, n = s.vocab - v0 < b.width ? s.vocab - v0 : b.width;
        MatArgs m{};
        m.x = x, m.x_stride = wide, m.y[0] = m.y[1] = w + v0 * ws_row, m.y_stride = ws_row;
        m.P = s.rows, m.Q = n, m.C = m.x_cols = wide, m.steps = steps_of(wide), m.stretches = 1;
        m.scale = scale, m.row = reinterpret_cast<const float*>(ws + b.row), m.q_first = v0, m.d = d, m.seg_rows = up(n, kTC);
        run_mat<false, false, kEpiDlogits>(m, tiling(s.rows, m.seg_rows, false, m.steps, false), on);

        if (p.dx) {  // dx[p][q] = sum over the piece's columns c of d[p][c] W[c][q]
            gx = MatArgs{};
            gx.x = d, gx.x_stride = gx.x_cols = m.seg_rows, gx.y[0] = gx.y[1] = m.y[0], gx.y_stride = ws_row;
            gx.P = s.rows, gx.Q = s.dim, gx.C = n, gx.steps = steps_of(n), gx.stretches = 1;
            gx.out = gx.out2 = static_cast<uint16_t*>(p.dx), gx.out_stride = s.dim, gx.seg_rows = gx.seg_valid = s.rows;
            gx.part = reinterpret_cast<float*>(ws + b.dx), gx.add = k > 0, gx.factor = r.factor;
            if (one) run_mat<false, true, kEpiStore>(gx, b.tx, on);
            else run_mat<false, true, kEpiAdd>(gx, b.tx, on);
        }
        if (p.dweight) {  // dW[v][q] = sum over rows c of d[c][v] x[c][q]
            MatArgs g{};
            g.x = d, g.x_stride = m.seg_rows, g.y[0] = g.y[1] = x, g.y_stride = wide;
            g.P = m.seg_rows, g.Q = s.dim, g.C = s.rows, g.steps = steps_of(s.rows), g.stretches = 1;
            g.out = g.out2 = static_cast<uint16_t*>(p.dweight) + v0 * s.dim, g.out_stride = s.dim;
            g.seg_rows = m.seg_rows, g.seg_valid = n;  // an even number of columns of dl; the padding's rows are not stored
            g.part = reinterpret_cast<float*>(ws + b.dw), g.factor = r.factor;
            const Tiling t = dw_tiling(s, n);
            if (t.splits == 1) {
                run_mat<true, true, kEpiStore>(g, t, on);
            } else {
                run_mat<true, true, kEpiPartial>(g, t, on);
                run_join(g, t.splits, on);
            }
        }
    }
    if (p.dx && !one) run_join(gx, b.tx.splits, on);
    return on.status;
}

}  // namespace mscan
