// Layer norm over the last dimension, forward and backward (mamba_layers.h), on gfx950.
//
// A row is held in registers by WPR waves (NV packs of V elements a lane), so it is read once:
// its mean, then the sums of the distances from the mean (the mean's own rounding, taken off again: a row
// far from zero loses nothing) and of their squares, then the output. Both directions are
// bound by HBM: the next row's loads are in flight while a row is worked on.
//
// Backward: with n = (t - mean) rstd and g = dy weight,
//   dx = rstd (g - mean(g) - n mean(g n)) + dresidual,   dweight = sum_rows dy n,   dbias = sum_rows dy.
// A workgroup walks its rows and keeps the two column sums in registers; it writes one row of partial
// sums, and a second kernel adds the workgroups' in order, so the result does not depend on timing.
//
// Measured: forward 16384 x 768 bf16 with residual 22 us (100 MB, 4.5 TB/s; a large copy 4.6); 16384 x 2048
// 50 forward (5.4 TB/s, partly cached), 44 + 4 backward and its column sums; 4000 x 8192 fp32 103 and 112.
#include <initializer_list>
#include <type_traits>
#include <utility>

#include "layers_common.hpp"
#include "layers_launch.hpp"

namespace mscan {

namespace {

struct NormArgs {
    const void* x;
    const void* res;
    const float* w;
    const float* b;
    void* y;
    void* sum;
    float* stats;
    int64_t rows, dim, sx, sres, sy, ssum;
    float eps;
};

struct NormBwdArgs {
    const void* t;
    const float* w;
    const float* stats;
    const void* dy;
    const void* dres;
    void* dx;
    float* part;  // (blocks, 2, dim)
    int64_t rows, dim, st, sdy, sdres, sdx;
};

// Sums of N values over the WPR waves of a row, the same bits in every thread. `slot` alternates
// between calls, so one barrier a call is enough.
template <int N, int WPR, int WAVES>
__device__ __forceinline__ void row_sum(float (&v)[2], float (*lds)[2][WAVES], int slot, int wave) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = wave_sum(v[k]);
    if constexpr (WPR > 1) {
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int k = 0; k < N; ++k) lds[slot][k][wave] = v[k];
        __syncthreads();
        const int first = wave / WPR * WPR;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            float s = 0.0f;
#pragma unroll
            for (int q = 0; q < WPR; ++q) s += lds[slot][k][first + q];
            v[k] = s;
        }
    }
}

// A variance, up from its rounding below 0; a row with a NaN keeps it (a maximum would drop it).
__device__ __forceinline__ float no_less_than_0(float v) { return v < 0.0f ? 0.0f : v; }

constexpr int kFwdWaves = 4;  // waves of a forward workgroup, unless a row takes more

template <typename S, int V, int NV, int WPR>
__global__ __launch_bounds__(64 * (WPR > kFwdWaves ? WPR : kFwdWaves)) void norm_fwd_kernel(NormArgs p) {
    constexpr int WAVES = WPR > kFwdWaves ? WPR : kFwdWaves, RPB = WAVES / WPR;
    __shared__ float lds[2][2][WAVES];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane_row = (int)threadIdx.x - wave / WPR * WPR * 64;
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t row = (int64_t)blockIdx.x * RPB + wave / WPR;
    using P = Pack<S, V>;
    P nx[NV], nr[NV];
    auto fetch = [&](int64_t r) __attribute__((always_inline)) {
        const S* x = static_cast<const S*>(p.x) + r * p.sx;
        const S* q = static_cast<const S*>(p.res) + r * p.sres;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int64_t c = (int64_t)(k * 64 * WPR + lane_row) * V;
            if (c < p.dim) {
                nx[k] = *reinterpret_cast<const P*>(x + c);
                if (p.res) nr[k] = *reinterpret_cast<const P*>(q + c);
            }
        }
    };
    if (row < p.rows) fetch(row);
    float w[NV][V], bb[NV][V];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int64_t c = (int64_t)(k * 64 * WPR + lane_row) * V + j;
            w[k][j] = p.w && c < p.dim ? p.w[c] : 1.0f;
            bb[k][j] = p.b && c < p.dim ? p.b[c] : 0.0f;
        }
    const float width = (float)p.dim, inv = 1.0f / width;
    int slot = 0;
    // every wave of the workgroup makes the same number of turns (the row sums' barriers)
    for (int64_t base = (int64_t)blockIdx.x * RPB; base < p.rows; base += step, row += step) {
        const bool on = row < p.rows;
        float t[NV][V];
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int64_t c = (int64_t)(k * 64 * WPR + lane_row) * V;
            const bool in = on && c < p.dim;
            P st;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float v = in ? to_f32(nx[k].v[j]) : 0.0f;
                if (p.res) {
                    st.v[j] = from_f32<S>(v + to_f32(nr[k].v[j]));
                    v = in ? to_f32(st.v[j]) : 0.0f;
                }
                t[k][j] = v;
                s[0] += v;
            }
            if (p.res && in) *reinterpret_cast<P*>(static_cast<S*>(p.sum) + row * p.ssum + c) = st;
        }
        if (row + step < p.rows) fetch(row + step);
        row_sum<1, WPR, WAVES>(s, lds, slot, wave);
        slot ^= 1;
        const float mean = s[0] / width;
        float q[2] = {0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const bool in = (int64_t)(k * 64 * WPR + lane_row) * V < p.dim;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float dlt = t[k][j] - mean;
                t[k][j] = dlt;
                q[0] += in ? dlt : 0.0f;
                q[1] += in ? dlt * dlt : 0.0f;
            }
        }
        row_sum<2, WPR, WAVES>(q, lds, slot, wave);
        slot ^= 1;
        const float off = q[0] * inv, var = no_less_than_0(__builtin_fmaf(-off, off, q[1] * inv));
        const float rstd = __builtin_amdgcn_rsqf(var + p.eps);
        if (on) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int64_t c = (int64_t)(k * 64 * WPR + lane_row) * V;
                P o;
#pragma unroll
                for (int j = 0; j < V; ++j) o.v[j] = from_f32<S>(__builtin_fmaf((t[k][j] - off) * rstd, w[k][j], bb[k][j]));
                if (c < p.dim) *reinterpret_cast<P*>(static_cast<S*>(p.y) + row * p.sy + c) = o;
            }
            if (p.stats && lane_row == 0) {
                p.stats[2 * row] = mean + off;
                p.stats[2 * row + 1] = rstd;
            }
        }
    }
}

// Rows too wide for the registers of 16 waves: one workgroup a row, read three times.
template <typename S>
__global__ __launch_bounds__(1024) void norm_fwd_wide_kernel(NormArgs p) {
    __shared__ float lds[2][2][16];
    const int wave = threadIdx.x >> 6;
    const int64_t row = grid_block();
    if (row >= p.rows) return;
    const S* x = static_cast<const S*>(p.x) + row * p.sx;
    const S* r = static_cast<const S*>(p.res) + row * p.sres;
    S* y = static_cast<S*>(p.y) + row * p.sy;
    S* sum = static_cast<S*>(p.sum) + row * p.ssum;
    auto at = [&](int64_t c) { return p.res ? to_f32(from_f32<S>(to_f32(x[c]) + to_f32(r[c]))) : to_f32(x[c]); };
    float s[2] = {0.0f, 0.0f};
    for (int64_t c = threadIdx.x; c < p.dim; c += 1024) s[0] += at(c);
    row_sum<1, 16, 16>(s, lds, 0, wave);
    const float mean = s[0] / (float)p.dim;
    float q[2] = {0.0f, 0.0f};
    for (int64_t c = threadIdx.x; c < p.dim; c += 1024) {
        const float d = at(c) - mean;
        q[0] += d;
        q[1] = __builtin_fmaf(d, d, q[1]);
    }
    row_sum<2, 16, 16>(q, lds, 1, wave);
    const float off = q[0] / (float)p.dim, var = no_less_than_0(__builtin_fmaf(-off, off, q[1] / (float)p.dim));
    const float rstd = __builtin_amdgcn_rsqf(var + p.eps);
    for (int64_t c = threadIdx.x; c < p.dim; c += 1024) {
        const float v = at(c);  // before either store: y or sum may be x's or residual's buffer
        const float o = __builtin_fmaf((v - mean - off) * rstd, p.w ? p.w[c] : 1.0f, p.b ? p.b[c] : 0.0f);
        if (p.res) sum[c] = from_f32<S>(v);
        y[c] = from_f32<S>(o);
    }
    if (p.stats && threadIdx.x == 0) {
        p.stats[2 * row] = mean + off;
        p.stats[2 * row + 1] = rstd;
    }
}

constexpr int kBwdWaves = 16;

template <typename S, int V, int NV, int WPR>
__global__ __launch_bounds__(64 * kBwdWaves) void norm_bwd_kernel(NormBwdArgs p) {
    constexpr int RPB = kBwdWaves / WPR;
    __shared__ float lds[2][2][kBwdWaves];
    __shared__ float cols[RPB > 1 ? 2 * 64 * WPR * NV * V : 1];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int group = wave / WPR;
    const int lane_row = (int)threadIdx.x - group * WPR * 64;
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t row = (int64_t)blockIdx.x * RPB + group;
    using P = Pack<S, V>;
    P nt[NV], ng[NV], nr[NV];
    float nmean = 0.0f, nrstd = 0.0f;
    auto fetch = [&](int64_t r) __attribute__((always_inline)) {
        const S* t = static_cast<const S*>(p.t) + r * p.st;
        const S* g = static_cast<const S*>(p.dy) + r * p.sdy;
        const S* q = static_cast<const S*>(p.dres) + r * p.sdres;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int64_t c = (int64_t)(k * 64 * WPR + lane_row) * V;
            if (c < p.dim) {
                nt[k] = *reinterpret_cast<const P*>(t + c);
                ng[k] = *reinterpret_cast<const P*>(g + c);
                if (p.dres) nr[k] = *reinterpret_cast<const P*>(q + c);
            }
        }
        nmean = p.stats[2 * r];
        nrstd = p.stats[2 * r + 1];
    };
    if (row < p.rows) fetch(row);
    float w[NV][V], dw[NV][V], db[NV][V];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int64_t c = (int64_t)(k * 64 * WPR + lane_row) * V + j;
            w[k][j] = p.w && c < p.dim ? p.w[c] : 1.0f;
            dw[k][j] = db[k][j] = 0.0f;
        }
    const float inv = 1.0f / (float)p.dim;
    int slot = 0;
    for (int64_t base = (int64_t)blockIdx.x * RPB; base < p.rows; base += step, row += step) {
        const bool on = row < p.rows;
        float n[NV][V], g[NV][V];
        P r[NV];
        float s[2] = {0.0f, 0.0f};
        const float rstd = nrstd, mean = nmean;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const bool in = on && (int64_t)(k * 64 * WPR + lane_row) * V < p.dim;
            r[k] = nr[k];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                n[k][j] = in ? (to_f32(nt[k].v[j]) - mean) * rstd : 0.0f;
                const float d = in ? to_f32(ng[k].v[j]) : 0.0f;
                dw[k][j] = __builtin_fmaf(d, n[k][j], dw[k][j]);
                db[k][j] += d;
                g[k][j] = d * w[k][j];
                s[0] += g[k][j];
                s[1] = __builtin_fmaf(g[k][j], n[k][j], s[1]);
            }
        }
        if (row + step < p.rows) fetch(row + step);
        row_sum<2, WPR, kBwdWaves>(s, lds, slot, wave);
        slot ^= 1;
        if (on) {
            const float m0 = s[0] * inv, m1 = s[1] * inv;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int64_t c = (int64_t)(k * 64 * WPR + lane_row) * V;
                P o;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float v = rstd * (g[k][j] - __builtin_fmaf(n[k][j], m1, m0));
                    if (p.dres) v += to_f32(r[k].v[j]);
                    o.v[j] = from_f32<S>(v);
                }
                if (c < p.dim) *reinterpret_cast<P*>(static_cast<S*>(p.dx) + row * p.sdx + c) = o;
            }
        }
    }
    if (!p.part) return;
    // the row groups' column sums, added in group order
    if constexpr (RPB > 1) {
        for (int q = 0; q < RPB; ++q) {
            if (group == q) {
#pragma unroll
                for (int k = 0; k < NV; ++k)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const int c = (k * 64 * WPR + lane_row) * V + j;
                        float* a = &cols[c];
                        float* b = &cols[64 * WPR * NV * V + c];
                        *a = q ? *a + dw[k][j] : dw[k][j];
                        *b = q ? *b + db[k][j] : db[k][j];
                    }
            }
            __syncthreads();
        }
        float* out = p.part + (int64_t)blockIdx.x * 2 * p.dim;
        for (int64_t c = threadIdx.x; c < p.dim; c += 64 * kBwdWaves) {
            out[c] = cols[c];
            out[p.dim + c] = cols[64 * WPR * NV * V + c];
        }
    } else {
        float* out = p.part + (int64_t)blockIdx.x * 2 * p.dim;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int64_t c = (int64_t)(k * 64 * WPR + lane_row) * V + j;
                if (c < p.dim) {
                    out[c] = dw[k][j];
                    out[p.dim + c] = db[k][j];
                }
            }
    }
}

// Wide rows: dx with the row read twice; the column sums by a kernel of their own.
template <typename S>
__global__ __launch_bounds__(1024) void norm_bwd_wide_kernel(NormBwdArgs p) {
    __shared__ float lds[2][2][16];
    const int wave = threadIdx.x >> 6;
    const int64_t row = grid_block();
    if (row >= p.rows) return;
    const S* t = static_cast<const S*>(p.t) + row * p.st;
    const S* dy = static_cast<const S*>(p.dy) + row * p.sdy;
    const S* dres = static_cast<const S*>(p.dres) + row * p.sdres;
    S* dx = static_cast<S*>(p.dx) + row * p.sdx;
    const float mean = p.stats[2 * row], rstd = p.stats[2 * row + 1];
    float s[2] = {0.0f, 0.0f};
    for (int64_t c = threadIdx.x; c < p.dim; c += 1024) {
        const float g = to_f32(dy[c]) * (p.w ? p.w[c] : 1.0f);
        s[0] += g;
        s[1] = __builtin_fmaf(g, (to_f32(t[c]) - mean) * rstd, s[1]);
    }
    row_sum<2, 16, 16>(s, lds, 0, wave);
    const float m0 = s[0] / (float)p.dim, m1 = s[1] / (float)p.dim;
    for (int64_t c = threadIdx.x; c < p.dim; c += 1024) {
        const float g = to_f32(dy[c]) * (p.w ? p.w[c] : 1.0f);
        float v = rstd * (g - __builtin_fmaf((to_f32(t[c]) - mean) * rstd, m1, m0));
        if (p.dres) v += to_f32(dres[c]);
        dx[c] = from_f32<S>(v);
    }
}

template <typename S>
__global__ __launch_bounds__(256) void norm_cols_wide_kernel(NormBwdArgs p) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= p.dim) return;
    const int64_t per = (p.rows + gridDim.y - 1) / gridDim.y, r0 = blockIdx.y * per;
    const int64_t r1 = r0 + per < p.rows ? r0 + per : p.rows;
    float a = 0.0f, b = 0.0f;
    for (int64_t r = r0; r < r1; ++r) {
        const float d = to_f32((static_cast<const S*>(p.dy) + r * p.sdy)[c]);
        const float n = (to_f32((static_cast<const S*>(p.t) + r * p.st)[c]) - p.stats[2 * r]) * p.stats[2 * r + 1];
        a = __builtin_fmaf(d, n, a);
        b += d;
    }
    float* out = p.part + (int64_t)blockIdx.y * 2 * p.dim;
    out[c] = a;
    out[p.dim + c] = b;
}

// The workgroups' partial column sums, added in order: 32 columns x 8 stretches of the list a workgroup.
__global__ __launch_bounds__(256) void norm_cols_kernel(const float* part, int blocks, int64_t dim, float* dweight,
                                                        float* dbias) {
    __shared__ float lds[8][32];
    const int64_t c = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);  // of the 2 dim columns
    const int g = threadIdx.x >> 5, per = (blocks + 7) / 8;
    float s = 0.0f;
    if (c < 2 * dim) {
        const int q1 = (g + 1) * per < blocks ? (g + 1) * per : blocks;
#pragma unroll 8
        for (int q = g * per; q < q1; ++q) s += part[(int64_t)q * 2 * dim + c];
    }
    lds[g][threadIdx.x & 31] = s;
    __syncthreads();
    if (g == 0 && c < 2 * dim) {
#pragma unroll
        for (int q = 1; q < 8; ++q) s += lds[q][threadIdx.x & 31];
        float* out = c < dim ? dweight : dbias;
        if (out) out[c < dim ? c : c - dim] = s;
    }
}

// Values of a row a lane holds. Few, so that many rows are in flight: at 16384 rows of 2048 bf16 with a
// residual the forward takes 52 us with 8 a lane (four waves a row) and 82 with 32 (one wave a row); the
// backward, which keeps two column sums and the weight beside them, 110 us forward and backward at
// 40000 x 768 with at most 8 and 155 with 16. The widest rows take what is left of 16 waves' registers.
constexpr int fwd_vals(int wpr) { return wpr == 16 ? 32 : 16; }
constexpr int bwd_vals(int wpr) { return wpr == 16 ? 16 : 8; }
constexpr int kFwdWavesPerCu = 16;  // 25.5 us at 16384 x 768; 33 with 32 (fewer rows share a wave's weights), 25.0 with 8
constexpr int64_t kBwdBlocks = 256;  // of 16 waves; their partial column sums are written and read once more

template <typename S, int V, int NV, int WPR>
void fwd_go(const NormArgs& q, Launches& on) {
    constexpr int WAVES = WPR > kFwdWaves ? WPR : kFwdWaves, RPB = WAVES / WPR;
    const int64_t need = (q.rows + RPB - 1) / RPB;
    const int64_t most = (int64_t)layers_cus() * kFwdWavesPerCu / WAVES;  // a few rows a wave: the weights are read once for them
    on(norm_fwd_kernel<S, V, NV, WPR>, dim3((unsigned)(need < most ? need : most)), dim3(64 * WAVES), q);
}

// The smallest instantiated number of packs that holds `nv` (1, 2, 3, 4, 6, 8, 12, 16, 24, 32; at most M).
template <int M, int N = 1, typename F>
auto with_packs(int64_t nv, F&& f) {
    constexpr int next = N < 4 ? N + 1 : N % 3 == 0 ? N / 3 * 4 : N / 2 * 3;
    if constexpr (next > M || N >= M) {
        return f(std::integral_constant<int, N < M ? M : N>{});
    } else {
        return nv <= N ? f(std::integral_constant<int, N>{}) : with_packs<M, next>(nv, f);
    }
}

template <typename S, int V, int WPR>
void fwd_width(const NormArgs& q, Launches& on) {
    with_packs<(fwd_vals(WPR) / V > 1 ? fwd_vals(WPR) / V : 1)>(
        (q.dim + 64 * WPR * V - 1) / (64 * WPR * V), [&](auto nv) { fwd_go<S, V, decltype(nv)::value, WPR>(q, on); });
}

template <typename S, int V>
void fwd_vec(const NormArgs& q, Launches& on) {
    if (q.dim <= 64 * fwd_vals(1)) return fwd_width<S, V, 1>(q, on);
    if (q.dim <= 256 * fwd_vals(4)) return fwd_width<S, V, 4>(q, on);
    if (q.dim <= 1024 * fwd_vals(16)) return fwd_width<S, V, 16>(q, on);
    on(norm_fwd_wide_kernel<S>, grid_of(q.rows, 1024), dim3(1024), q);
}

template <typename S, int V, int NV, int WPR>
int64_t bwd_go(const NormBwdArgs& q, Launches& on) {
    constexpr int RPB = kBwdWaves / WPR;
    const int64_t need = (q.rows + RPB - 1) / RPB, n = need < kBwdBlocks ? need : kBwdBlocks;
    on(norm_bwd_kernel<S, V, NV, WPR>, dim3((unsigned)n), dim3(64 * kBwdWaves), q);
    return n;
}

template <typename S, int V, int WPR>
int64_t bwd_width(const NormBwdArgs& q, Launches& on) {
    return with_packs<(bwd_vals(WPR) / V > 1 ? bwd_vals(WPR) / V : 1)>(
        (q.dim + 64 * WPR * V - 1) / (64 * WPR * V), [&](auto nv) { return bwd_go<S, V, decltype(nv)::value, WPR>(q, on); });
}

template <typename S, int V>
int64_t bwd_vec(const NormBwdArgs& q, Launches& on) {
    if (q.dim <= 64 * bwd_vals(1)) return bwd_width<S, V, 1>(q, on);
    if (q.dim <= 256 * bwd_vals(4)) return bwd_width<S, V, 4>(q, on);
    if (q.dim <= 1024 * bwd_vals(16)) return bwd_width<S, V, 16>(q, on);
    on(norm_bwd_wide_kernel<S>, grid_of(q.rows, 1024), dim3(1024), q);
    if (!q.part) return 0;
    const int64_t n = q.rows < 64 ? q.rows : 64;
    on(norm_cols_wide_kernel<S>, dim3((unsigned)((q.dim + 255) / 256), (unsigned)n), dim3(256), q);
    return n;
}

// The widest pack (16 bytes and down) that the width, pointers and row strides are multiples of, and that
// leaves less than half of a wave idle over the width (200000 x 100 bf16: 141 us with packs of 4, on 25
// lanes, 113 with single elements).
template <typename S, int V = 16 / sizeof(S), typename F>
auto with_pack(int64_t dim, std::initializer_list<std::pair<const void*, int64_t>> rows, F&& f) {
    if constexpr (V == 1) {
        return f(std::integral_constant<int, 1>{});
    } else {
        bool ok = dim % V == 0 && dim > 32 * V;
        for (const auto& r : rows)
            ok = ok && (!r.first || (reinterpret_cast<uintptr_t>(r.first) % (V * sizeof(S)) == 0 && r.second % V == 0));
        return ok ? f(std::integral_constant<int, V>{}) : with_pack<S, V / 2>(dim, rows, f);
    }
}

template <typename S>
void fwd_typed(const NormArgs& q, Launches& on) {
    with_pack<S>(q.dim, {{q.x, q.sx}, {q.res, q.sres}, {q.y, q.sy}, {q.sum, q.ssum}},
                 [&](auto v) { fwd_vec<S, decltype(v)::value>(q, on); });
}

template <typename S>
int64_t bwd_typed(const NormBwdArgs& q, Launches& on) {
    return with_pack<S>(q.dim, {{q.t, q.st}, {q.dy, q.sdy}, {q.dres, q.sdres}, {q.dx, q.sdx}},
                        [&](auto v) { return bwd_vec<S, decltype(v)::value>(q, on); });
}

}  // namespace

int64_t norm_bwd_workspace(const mamba_norm_shape& s) { return align256(kBwdBlocks * 2 * s.dim * 4); }

int launch_norm_fwd(const mamba_norm_ptrs& p, const mamba_norm_shape& s, float eps, bool bf16, hipStream_t stream) {
    NormArgs q{p.x, p.residual, p.weight, p.bias, p.y, p.sum, p.stats, s.rows, s.dim, p.x_stride, p.residual_stride,
               p.y_stride, p.sum_stride, eps};
    Launches on(stream);
    bf16 ? fwd_typed<bf16_t>(q, on) : fwd_typed<float>(q, on);
    return on.status;
}

int launch_norm_bwd(const mamba_norm_bwd_ptrs& p, const mamba_norm_shape& s, bool bf16, hipStream_t stream) {
    const bool sums = p.dweight || p.dbias;
    NormBwdArgs q{p.t, p.weight, p.stats, p.dy, p.dresidual, p.dx, sums ? static_cast<float*>(p.workspace) : nullptr,
                  s.rows, s.dim, p.t_stride, p.dy_stride, p.dresidual_stride, p.dx_stride};
    Launches on(stream);
    const int64_t blocks = bf16 ? bwd_typed<bf16_t>(q, on) : bwd_typed<float>(q, on);
    if (sums)
        on(norm_cols_kernel, dim3((unsigned)((2 * s.dim + 31) / 32)), dim3(256),
           static_cast<const float*>(p.workspace), (int)blocks, s.dim, p.dweight, p.dbias);
    return on.status;
}

}  // namespace mscan
