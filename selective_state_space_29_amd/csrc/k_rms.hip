// Root-mean-square norms before and after a block (mamba_block.h) and their gradients, on gfx950.
//
//   residual:    t = residual + scale x (rounded),   y = t rstd weight,   rstd = 1 / sqrt(mean(t^2) + eps)
//   gate first:  v = x silu(z),  y = v rstd weight        gate last:  v = x,  y = v rstd weight silu(z)
//
// With n = v rstd and g the gradient that reaches n: dv = rstd (g - n mean(g n)), dweight = sum_rows dy n (times
// the gate where it comes last).
//
// A row (or one of its groups) is held in registers by LPR lanes, an eighth of a wave to 16 waves, NV packs of V
// values a lane, so it is read once; the next row's loads are in flight while a row is worked on. The backward keeps
// the weight's column sums in registers over a workgroup's rows and writes one row of partial sums a workgroup,
// which a second kernel adds in order.
//
// Bound by HBM. 16384 x 768 bf16 with residual 25.4 us (101 MB, 4.0 TB/s); 16384 x 1536 bf16 gated 36.3 (4.2), its
// gradient 57.6 + 4 (252 MB, 4.4); 5003 x 1001 fp32 with residual 19.8 (80 MB, 4.0), its gradient 17.2 + 3.4.
#include "block_launch.hpp"
#include "layers_common.hpp"
#include "rows.hpp"

namespace mscan {

namespace {

enum { kPlain = 0, kResidual = 1, kGateFirst = 2, kGateLast = 3 };

struct RmsArgs {
    const void* x;
    const void* other;  // residual or z
    const float* w;
    void* y;
    void* sum;
    float* stats;       // (rows, groups)
    int64_t rows, dim, groups;  // dim: of a group
    int64_t sx, so, sy, ssum;
    int64_t blocks;     // workgroups a group
    float scale, eps;
};

struct RmsBwdArgs {
    const void* v;      // t or x
    const void* dy;
    const void* other;  // dsum or z
    const float* w;
    const float* stats;
    void* dv;           // dx
    void* dother;       // dresidual or dz
    float* part;        // (blocks, groups dim)
    int64_t rows, dim, groups;
    int64_t sv, sdy, so, sdv, sdo;
    int64_t blocks;
    float scale;
};

// The value that is normalised, from x and the second input.
template <typename S, int MODE>
__device__ __forceinline__ float normed(float x, float other, float scale) {
    if constexpr (MODE == kResidual) return to_f32(from_f32<S>(__builtin_fmaf(scale, x, other)));
    if constexpr (MODE == kGateFirst) return x * silu_f(other);
    return x;
}

// Sum over the LPR lanes of a row, the same bits in each.
template <int CTRL>
__device__ __forceinline__ float lanes_add(float v) {
    return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
}
template <int LPR, int WAVES>
__device__ __forceinline__ float lanes_sum(float v, float (*lds)[2][WAVES], int slot, int wave) {
    if constexpr (LPR >= 64) {
        float s[2] = {v, 0.0f};
        row_sum<1, LPR / 64, WAVES>(s, lds, slot, wave);
        return s[0];
    } else {
        v = lanes_add<0xb1>(v);   // lanes 1 and 0, 3 and 2
        v = lanes_add<0x4e>(v);   // pairs of a quad
        v = lanes_add<0x141>(v);  // quads of 8 lanes (half row mirrored)
        if constexpr (LPR >= 16) v = lanes_add<0x140>(v);  // halves of 16 (row mirrored)
        if constexpr (LPR >= 32) v += __shfl_xor(v, 16);
        return v;
    }
}
constexpr int waves_of(int lpr) { return lpr > 64 ? lpr / 64 : 1; }

constexpr int kFwdWaves = 4;  // waves of a forward workgroup, unless a row takes more

template <typename S, int V, int NV, int LPR, int MODE>
__global__ __launch_bounds__(64 * (waves_of(LPR) > kFwdWaves ? waves_of(LPR) : kFwdWaves)) void rms_fwd_kernel(RmsArgs p) {
    constexpr int WAVES = waves_of(LPR) > kFwdWaves ? waves_of(LPR) : kFwdWaves, RPB = WAVES * 64 / LPR;
    __shared__ float lds[2][2][WAVES];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int sub = LPR < 64 ? (int)threadIdx.x / LPR : wave / waves_of(LPR), lane_row = (int)threadIdx.x - sub * LPR;
    const int64_t group = blockIdx.x % p.groups, block = blockIdx.x / p.groups, c0 = group * p.dim;
    const int64_t step = p.blocks * RPB;
    int64_t row = block * RPB + sub;
    using P = Pack<S, V>;
    P nx[NV], no[NV];
    auto fetch = [&](int64_t r) __attribute__((always_inline)) {
        const S* x = static_cast<const S*>(p.x) + r * p.sx + c0;
        const S* o = static_cast<const S*>(p.other) + r * p.so + c0;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int64_t c = (int64_t)(k * LPR + lane_row) * V;
            nx[k] = load_some<S, V>(x + c, (int)(p.dim - c));
            if constexpr (MODE != kPlain) no[k] = load_some<S, V>(o + c, (int)(p.dim - c));
        }
    };
    if (row < p.rows) fetch(row);
    float w[NV][V];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int64_t c = (int64_t)(k * LPR + lane_row) * V + j;
            w[k][j] = p.w && c < p.dim ? p.w[c0 + c] : 1.0f;
        }
    const float inv = 1.0f / (float)p.dim;
    int slot = 0;
    // every wave of the workgroup makes the same number of turns (the row sums' barriers)
    for (int64_t base = block * RPB; base < p.rows; base += step, row += step) {
        const bool on = row < p.rows;
        float t[NV][V], gate[MODE == kGateLast ? NV : 1][V];
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int64_t c = (int64_t)(k * LPR + lane_row) * V;
            P st;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float other = MODE != kPlain ? to_f32(no[k].v[j]) : 0.0f;
                const float v = on ? normed<S, MODE>(to_f32(nx[k].v[j]), other, p.scale) : 0.0f;  // 0 behind the row
                if constexpr (MODE == kResidual) st.v[j] = from_f32<S>(v);
                if constexpr (MODE == kGateLast) gate[k][j] = silu_f(other);
                t[k][j] = v;
                s = __builtin_fmaf(v, v, s);
            }
            if (MODE == kResidual && on) store_some<S, V>(static_cast<S*>(p.sum) + row * p.ssum + c0 + c, st, (int)(p.dim - c));
        }
        if (row + step < p.rows) fetch(row + step);
        s = lanes_sum<LPR, WAVES>(s, lds, slot, wave);
        slot ^= 1;
        const float rstd = __builtin_amdgcn_rsqf(__builtin_fmaf(s, inv, p.eps));
        if (on) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int64_t c = (int64_t)(k * LPR + lane_row) * V;
                P o;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float v = t[k][j] * rstd * w[k][j];
                    o.v[j] = from_f32<S>(MODE == kGateLast ? v * gate[MODE == kGateLast ? k : 0][j] : v);
                }
                store_some<S, V>(static_cast<S*>(p.y) + row * p.sy + c0 + c, o, (int)(p.dim - c));
            }
            if (p.stats && lane_row == 0) p.stats[row * p.groups + group] = rstd;
        }
    }
}

// Rows too wide for the registers of 16 waves: one workgroup a row and group, read twice.
template <typename S, int MODE>
__global__ __launch_bounds__(1024) void rms_fwd_wide_kernel(RmsArgs p) {
    __shared__ float lds[2][2][16];
    const int wave = threadIdx.x >> 6;
    const int64_t id = grid_block();
    if (id >= p.rows * p.groups) return;
    const int64_t row = id / p.groups, group = id - row * p.groups, c0 = group * p.dim;
    const S* x = static_cast<const S*>(p.x) + row * p.sx + c0;
    const S* o = static_cast<const S*>(p.other) + row * p.so + c0;
    S* y = static_cast<S*>(p.y) + row * p.sy + c0;
    auto at = [&](int64_t c) { return normed<S, MODE>(to_f32(x[c]), MODE != kPlain ? to_f32(o[c]) : 0.0f, p.scale); };
    float s[2] = {0.0f, 0.0f};
    for (int64_t c = threadIdx.x; c < p.dim; c += 1024) {
        const float v = at(c);
        s[0] = __builtin_fmaf(v, v, s[0]);
    }
    row_sum<1, 16, 16>(s, lds, 0, wave);
    const float rstd = __builtin_amdgcn_rsqf(s[0] / (float)p.dim + p.eps);
    for (int64_t c = threadIdx.x; c < p.dim; c += 1024) {
        const float v = at(c);  // before either store: y or sum may be an input's buffer
        float r = v * rstd * (p.w ? p.w[c0 + c] : 1.0f);
        if constexpr (MODE == kGateLast) r *= silu_f(to_f32(o[c]));
        if constexpr (MODE == kResidual) (static_cast<S*>(p.sum) + row * p.ssum + c0)[c] = from_f32<S>(v);
        y[c] = from_f32<S>(r);
    }
    if (p.stats && threadIdx.x == 0) p.stats[id] = rstd;
}

constexpr int kBwdWaves = 16;

// What one value contributes: n, the gradient g that reaches it, and its weight's.
template <int MODE>
struct RmsTerm {
    float n, g, dw, gate, slope;
    RmsTerm() = default;
    __device__ __forceinline__ RmsTerm(float x, float dy, float z, float w, float rstd) {
        gate = 1.0f, slope = 0.0f;
        if constexpr (MODE == kGateFirst || MODE == kGateLast) {
            const float s = hw_rcp(1.0f + hw_exp2(-z * kLog2e));
            gate = z * s;
            slope = s * __builtin_fmaf(z, 1.0f - s, 1.0f);
        }
        n = (MODE == kGateFirst ? x * gate : x) * rstd;
        const float d = MODE == kGateLast ? dy * gate : dy;
        g = d * w;
        dw = d * n;
    }
};
// The two results, from dv = rstd (g - n m): dx and dresidual, or dx and dz.
template <int MODE>
__device__ __forceinline__ void rms_out(const RmsTerm<MODE>& t, float dv, float x, float dy, float w, float scale, float& a, float& b) {
    if constexpr (MODE == kResidual) a = scale * dv, b = dv;
    else if constexpr (MODE == kGateFirst) a = dv * t.gate, b = dv * x * t.slope;
    else a = dv, b = dy * t.n * w * t.slope;
}

// MODE kResidual stands for the plain norm too (dsum may be NULL, dresidual is not written).
template <typename S, int V, int NV, int LPR, int MODE>
__global__ __launch_bounds__(64 * kBwdWaves) void rms_bwd_kernel(RmsBwdArgs p) {
    constexpr int RPB = kBwdWaves * 64 / LPR;
    constexpr bool GATED = MODE != kResidual;
    __shared__ float lds[2][2][kBwdWaves];
    __shared__ float cols[RPB > 1 ? LPR * NV * V : 1];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int sub = LPR < 64 ? (int)threadIdx.x / LPR : wave / waves_of(LPR), lane_row = (int)threadIdx.x - sub * LPR;
    const int64_t group = blockIdx.x % p.groups, block = blockIdx.x / p.groups, c0 = group * p.dim;
    const int64_t step = p.blocks * RPB;
    int64_t row = block * RPB + sub;
    using P = Pack<S, V>;
    P nv[NV], ng[NV], no[NV];
    float nrstd = 0.0f;
    const bool more = GATED || p.other;
    auto fetch = [&](int64_t r) __attribute__((always_inline)) {
        const S* v = static_cast<const S*>(p.v) + r * p.sv + c0;
        const S* g = static_cast<const S*>(p.dy) + r * p.sdy + c0;
        const S* o = static_cast<const S*>(p.other) + r * p.so + c0;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int64_t c = (int64_t)(k * LPR + lane_row) * V;
            const int n = (int)(p.dim - c);
            nv[k] = load_some<S, V>(v + c, n);
            ng[k] = load_some<S, V>(g + c, n);
            if (more) no[k] = load_some<S, V>(o + c, n);
        }
        nrstd = p.stats[r * p.groups + group];
    };
    if (row < p.rows) fetch(row);
    float w[NV][V], dw[NV][V];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int64_t c = (int64_t)(k * LPR + lane_row) * V + j;
            w[k][j] = p.w && c < p.dim ? p.w[c0 + c] : 1.0f;
            dw[k][j] = 0.0f;
        }
    const float inv = 1.0f / (float)p.dim;
    int slot = 0;
    for (int64_t base = block * RPB; base < p.rows; base += step, row += step) {
        const bool on = row < p.rows;
        P v[NV], g[NV], o[NV];
        RmsTerm<MODE> terms[NV][V];  // (gates and slopes are not computed twice: 96 us a pass at 16384 x 1536 gated, 110)
        float s = 0.0f;
        const float rstd = nrstd;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            v[k] = nv[k], g[k] = ng[k], o[k] = no[k];
            if (on) {  // (values behind the row are zeros and add nothing)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const RmsTerm<MODE> t(to_f32(v[k].v[j]), to_f32(g[k].v[j]), GATED ? to_f32(o[k].v[j]) : 0.0f, w[k][j], rstd);
                    terms[k][j] = t;
                    dw[k][j] += t.dw;
                    s = __builtin_fmaf(t.g, t.n, s);
                }
            }
        }
        if (row + step < p.rows) fetch(row + step);
        s = lanes_sum<LPR, kBwdWaves>(s, lds, slot, wave);
        slot ^= 1;
        if (on) {
            const float m = s * inv;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int64_t c = (int64_t)(k * LPR + lane_row) * V;
                P a, b;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float x = to_f32(v[k].v[j]), dy = to_f32(g[k].v[j]), z = more ? to_f32(o[k].v[j]) : 0.0f;
                    const RmsTerm<MODE>& t = terms[k][j];
                    float dv = rstd * __builtin_fmaf(-t.n, m, t.g), ra, rb;
                    if constexpr (!GATED) dv += z;
                    rms_out<MODE>(t, dv, x, dy, w[k][j], p.scale, ra, rb);
                    a.v[j] = from_f32<S>(ra), b.v[j] = from_f32<S>(rb);
                }
                if (p.dv) store_some<S, V>(static_cast<S*>(p.dv) + row * p.sdv + c0 + c, a, (int)(p.dim - c));
                if (p.dother) store_some<S, V>(static_cast<S*>(p.dother) + row * p.sdo + c0 + c, b, (int)(p.dim - c));
            }
        }
    }
    if (!p.part) return;
    float* out = p.part + block * p.dim * p.groups + c0;
    // the column sums of a wave's rows, of two lanes at a time, then of the rows that waves share, in their order
    if constexpr (LPR < 64) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int far = LPR; far < 64; far *= 2) dw[k][j] += __shfl_xor(dw[k][j], far);
    }
    if constexpr (RPB > 1) {
        constexpr int TURNS = LPR < 64 ? kBwdWaves : RPB;
        const int turn = LPR < 64 ? (int)(threadIdx.x & 63) < LPR ? wave : -1 : sub;
        for (int q = 0; q < TURNS; ++q) {
            if (turn == q) {
#pragma unroll
                for (int k = 0; k < NV; ++k)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        float* a = &cols[(k * LPR + lane_row) * V + j];
                        *a = q ? *a + dw[k][j] : dw[k][j];
                    }
            }
            __syncthreads();
        }
        for (int64_t c = threadIdx.x; c < p.dim; c += 64 * kBwdWaves) out[c] = cols[c];
    } else {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int64_t c = (int64_t)(k * LPR + lane_row) * V + j;
                if (c < p.dim) out[c] = dw[k][j];
            }
    }
}

// Wide rows: the results with the row read twice; the column sums by a kernel of their own.
template <typename S, int MODE>
__global__ __launch_bounds__(1024) void rms_bwd_wide_kernel(RmsBwdArgs p) {
    __shared__ float lds[2][2][16];
    const int wave = threadIdx.x >> 6;
    const int64_t id = grid_block();
    if (id >= p.rows * p.groups) return;
    const int64_t row = id / p.groups, group = id - row * p.groups, c0 = group * p.dim;
    const S* v = static_cast<const S*>(p.v) + row * p.sv + c0;
    const S* dy = static_cast<const S*>(p.dy) + row * p.sdy + c0;
    const S* o = p.other ? static_cast<const S*>(p.other) + row * p.so + c0 : nullptr;
    const float rstd = p.stats[id];
    float s[2] = {0.0f, 0.0f};
    for (int64_t c = threadIdx.x; c < p.dim; c += 1024) {
        const RmsTerm<MODE> t(to_f32(v[c]), to_f32(dy[c]), o ? to_f32(o[c]) : 0.0f, p.w ? p.w[c0 + c] : 1.0f, rstd);
        s[0] = __builtin_fmaf(t.g, t.n, s[0]);
    }
    row_sum<1, 16, 16>(s, lds, 0, wave);
    const float m = s[0] / (float)p.dim;
    for (int64_t c = threadIdx.x; c < p.dim; c += 1024) {
        const float x = to_f32(v[c]), d = to_f32(dy[c]), z = o ? to_f32(o[c]) : 0.0f, w = p.w ? p.w[c0 + c] : 1.0f;
        const RmsTerm<MODE> t(x, d, z, w, rstd);
        float dv = rstd * __builtin_fmaf(-t.n, m, t.g), ra, rb;
        if constexpr (MODE == kResidual) dv += z;
        rms_out<MODE>(t, dv, x, d, w, p.scale, ra, rb);
        if (p.dv) (static_cast<S*>(p.dv) + row * p.sdv + c0)[c] = from_f32<S>(ra);
        if (p.dother) (static_cast<S*>(p.dother) + row * p.sdo + c0)[c] = from_f32<S>(rb);
    }
}

template <typename S, int MODE>
__global__ __launch_bounds__(256) void rms_cols_wide_kernel(RmsBwdArgs p) {
    const int64_t wide = p.dim * p.groups, c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= wide) return;
    const int64_t group = c / p.dim, per = (p.rows + p.blocks - 1) / p.blocks, r0 = blockIdx.y * per;
    const int64_t r1 = r0 + per < p.rows ? r0 + per : p.rows;
    float s = 0.0f;
    for (int64_t r = r0; r < r1; ++r) {
        const RmsTerm<MODE> t(to_f32((static_cast<const S*>(p.v) + r * p.sv)[c]), to_f32((static_cast<const S*>(p.dy) + r * p.sdy)[c]),
                              MODE != kResidual ? to_f32((static_cast<const S*>(p.other) + r * p.so)[c]) : 0.0f, 1.0f,
                              p.stats[r * p.groups + group]);
        s += t.dw;
    }
    p.part[blockIdx.y * wide + c] = s;
}

// The workgroups' partial column sums, added in order: 32 columns x 8 stretches of the list a workgroup (of 2^29
// columns and more, more threads than a dimension of the grid counts).
__global__ __launch_bounds__(256) void rms_cols_kernel(const float* part, int blocks, int64_t wide, float* dweight) {
    __shared__ float lds[8][32];
    const int64_t c = grid_block() * 32 + (threadIdx.x & 31);
    const int g = threadIdx.x >> 5, per = (blocks + 7) / 8;
    float s = 0.0f;
    if (c < wide) s = column_sum(part, wide, c, g * per, (g + 1) * per < blocks ? (g + 1) * per : blocks);
    lds[g][threadIdx.x & 31] = s;
    __syncthreads();
    if (g == 0 && c < wide) {
#pragma unroll
        for (int q = 1; q < 8; ++q) s += lds[q][threadIdx.x & 31];
        dweight[c] = s;
    }
}

// Values of a row a lane holds, few so that many rows are in flight; 16 waves have the registers for 16 and, in
// the backward, 8 (wider rows are read twice).
constexpr int kFwdVals = 16, kBwdVals = 8;
constexpr int fwd_waves_per_cu(int wpr) { return wpr == 1 ? 16 : 32; }
constexpr int64_t kBwdBlocks = 256;  // of 16 waves; their partial column sums are written and read once more

int64_t at_least_1(int64_t n) { return n < 1 ? 1 : n; }

// Calls f(packs a lane, lanes a row) for rows of `dim` values, or `wide` where they do not fit. Packs are 16 bytes
// wherever the rows begin; rows of less than half a wave's packs share a wave (50000 x 512 bf16 in groups of 64,
// gated, forward and backward: 95 us; a wave a group 383).
template <typename S, int VALS, typename F, typename W>
auto with_layout(int64_t dim, F&& f, W&& wide) {
    constexpr int V = 16 / sizeof(S);
    auto go = [&](auto lanes) {
        constexpr int L = decltype(lanes)::value;
        return with_packs<(L < 64 ? 1 : VALS / V)>((dim + L * V - 1) / (L * V), [&](auto nv) { return f(nv, lanes); });
    };
    if (dim <= 8 * V) return go(std::integral_constant<int, 8>{});
    if (dim <= 16 * V) return go(std::integral_constant<int, 16>{});
    if (dim <= 32 * V) return go(std::integral_constant<int, 32>{});
    if (dim <= 64 * VALS) return go(std::integral_constant<int, 64>{});
    if (dim <= 256 * VALS) return go(std::integral_constant<int, 256>{});
    if (dim <= 1024 * VALS) return go(std::integral_constant<int, 1024>{});
    return wide();
}

template <typename S, int MODE>
void fwd_typed(RmsArgs q, Launches& on) {
    with_layout<S, kFwdVals>(
        q.dim,
        [&](auto nv, auto lanes) {
            constexpr int LPR = decltype(lanes)::value, WPR = waves_of(LPR), WAVES = WPR > kFwdWaves ? WPR : kFwdWaves;
            constexpr int RPB = WAVES * 64 / LPR;
            const int64_t need = (q.rows + RPB - 1) / RPB;
            const int64_t most = at_least_1((int64_t)layers_cus() * fwd_waves_per_cu(WPR) / WAVES / q.groups);
            q.blocks = need < most ? need : most;
            on(rms_fwd_kernel<S, 16 / sizeof(S), decltype(nv)::value, LPR, MODE>, dim3((unsigned)(q.blocks * q.groups)),
               dim3(64 * WAVES), q);
        },
        [&] { on(rms_fwd_wide_kernel<S, MODE>, grid_of(q.rows * q.groups, 1024), dim3(1024), q); });
}

template <typename S, int MODE>
int64_t bwd_typed(RmsBwdArgs q, Launches& on) {
    return with_layout<S, kBwdVals>(
        q.dim,
        [&](auto nv, auto lanes) {
            constexpr int LPR = decltype(lanes)::value, RPB = kBwdWaves * 64 / LPR;
            const int64_t need = (q.rows + RPB - 1) / RPB, most = at_least_1(kBwdBlocks / q.groups);
            q.blocks = need < most ? need : most;
            on(rms_bwd_kernel<S, 16 / sizeof(S), decltype(nv)::value, LPR, MODE>, dim3((unsigned)(q.blocks * q.groups)),
               dim3(64 * kBwdWaves), q);
            return q.blocks;
        },
        [&] {
            on(rms_bwd_wide_kernel<S, MODE>, grid_of(q.rows * q.groups, 1024), dim3(1024), q);
            if (!q.part) return (int64_t)0;
            q.blocks = q.rows < 64 ? q.rows : 64;
            on(rms_cols_wide_kernel<S, MODE>, dim3((unsigned)((q.dim * q.groups + 255) / 256), (unsigned)q.blocks), dim3(256), q);
            return q.blocks;
        });
}

void join(const RmsBwdArgs& q, int64_t blocks, float* dweight, Launches& on) {
    if (!dweight) return;
    const int64_t wide = q.dim * q.groups;
    on(rms_cols_kernel, grid_of((wide + 31) / 32, 256), dim3(256), static_cast<const float*>(q.part), (int)blocks, wide, dweight);
}

}  // namespace

int launch_rms_fwd(const mamba_rms_ptrs& p, const mamba_rms_shape& s, float scale, float eps, bool bf16, hipStream_t stream) {
    RmsArgs q{p.x, p.residual, p.weight, p.y, p.sum, p.stats, s.rows, s.dim, 1, p.x_stride, p.residual_stride, p.y_stride, p.sum_stride,
              1, scale, eps};
    Launches on(stream);
    if (p.residual) bf16 ? fwd_typed<bf16_t, kResidual>(q, on) : fwd_typed<float, kResidual>(q, on);
    else bf16 ? fwd_typed<bf16_t, kPlain>(q, on) : fwd_typed<float, kPlain>(q, on);
    return on.status;
}

int launch_gated_rms_fwd(const mamba_gated_rms_ptrs& p, const mamba_gated_rms_shape& s, bool gate_first, float eps, bool bf16,
                         hipStream_t stream) {
    RmsArgs q{p.x, p.z, p.weight, p.y, nullptr, p.stats, s.rows, s.dim / s.groups, s.groups, p.x_stride, p.z_stride, p.y_stride, 0,
              1, 1.0f, eps};
    Launches on(stream);
    if (gate_first) bf16 ? fwd_typed<bf16_t, kGateFirst>(q, on) : fwd_typed<float, kGateFirst>(q, on);
    else bf16 ? fwd_typed<bf16_t, kGateLast>(q, on) : fwd_typed<float, kGateLast>(q, on);
    return on.status;
}

// A row of partial sums for each workgroup, of which there are no more than rows.
int64_t parts_bytes(int64_t rows, int64_t dim) { return align256((rows < kBwdBlocks ? rows : kBwdBlocks) * dim * 4); }
int64_t rms_bwd_workspace(const mamba_rms_shape& s) { return parts_bytes(s.rows, s.dim); }
int64_t gated_rms_bwd_workspace(const mamba_gated_rms_shape& s) { return parts_bytes(s.rows, s.dim); }

int launch_rms_bwd(const mamba_rms_bwd_ptrs& p, const mamba_rms_shape& s, float scale, bool bf16, hipStream_t stream) {
    RmsBwdArgs q{p.t, p.dy, p.dsum, p.weight, p.stats, p.dx, p.dresidual, p.dweight ? static_cast<float*>(p.workspace) : nullptr,
                 s.rows, s.dim, 1, p.t_stride, p.dy_stride, p.dsum_stride, p.dx_stride, p.dresidual_stride, 1, scale};
    Launches on(stream);
    join(q, bf16 ? bwd_typed<bf16_t, kResidual>(q, on) : bwd_typed<float, kResidual>(q, on), p.dweight, on);
    return on.status;
}

int launch_gated_rms_bwd(const mamba_gated_rms_bwd_ptrs& p, const mamba_gated_rms_shape& s, bool gate_first, bool bf16,
                         hipStream_t stream) {
    RmsBwdArgs q{p.x, p.dy, p.z, p.weight, p.stats, p.dx, p.dz, p.dweight ? static_cast<float*>(p.workspace) : nullptr,
                 s.rows, s.dim / s.groups, s.groups, p.x_stride, p.dy_stride, p.z_stride, p.dx_stride, p.dz_stride, 1, 1.0f};
    Launches on(stream);
    int64_t blocks;
    if (gate_first) blocks = bf16 ? bwd_typed<bf16_t, kGateFirst>(q, on) : bwd_typed<float, kGateFirst>(q, on);
    else blocks = bf16 ? bwd_typed<bf16_t, kGateLast>(q, on) : bwd_typed<float, kGateLast>(q, on);
    join(q, blocks, p.dweight, on);
    return on.status;
}

}  // namespace mscan
