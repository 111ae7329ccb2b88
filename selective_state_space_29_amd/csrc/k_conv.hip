// Short causal convolution of each channel with its activation (mamba_block.h) and its gradient, on gfx950.
//
//   pre_t = bias + sum_{j < W} w_{W-1-j} v_{t-j},   y_t = silu(pre_t)        (tap j reaches j steps back)
//   dpre_t = dy_t silu'(pre_t);   dv_s = sum_j w_{W-1-j} dpre_{s+j};   dw_{W-1-j} = sum_t dpre_t v_{t-j}
//
// A thread computes a run of kRun steps: of one pack of channels where channels lie side by side ("rows"
// kernels), of one channel where steps do ("steps" kernels, the scan's layout). It loads what the run needs,
// the W - 1 steps before it (and, in the backward, after it) among them: they are the neighbouring runs' and
// come from the cache. A tap is dropped where a sequence begins between the value and the step: the leading
// zeros of the resets' bits up to a step are the number of steps since.
//
// Rows in, steps out (a projection's output handed to the scan): the results of 64 channels x the runs of a
// workgroup pass through LDS in 16-byte pieces whose places are XORed with the channel, so that rows are read
// and rows are written in whole lines; the backward takes dy the same way.
//
// Every kernel is bound by HBM: it reads and writes each value once. The weight's gradient is summed in
// registers over a workgroup's runs, then over its threads in order, and a second kernel adds the workgroups'.
#include <type_traits>

#include "block_launch.hpp"
#include "layers_common.hpp"
#include "rows.hpp"

namespace mscan {

namespace {

constexpr int kRun = 8;       // steps of a thread's run
constexpr int kConvThreads = 256;
constexpr int kGroup = 64;    // channels of a "rows" workgroup: lines of 128 or 256 bytes
constexpr int kMaxWidth = 4;

struct ConvArgs {
    const void* x;
    const float* w;
    const float* b;
    const void* state;
    const uint8_t* reset;
    void* y;
    void* last;
    int64_t sx_b, sx_r, sy_b, sy_r;
    int64_t batch, len, dim;
    uint32_t runs, items;  // runs of a sequence (one at least), of all sequences
    int blocks;            // workgroups a group of channels
    int silu;
};

struct ConvBwdArgs {
    const void* x;
    const float* w;
    const float* b;
    const void* state;
    const uint8_t* reset;
    const void* dy;
    const void* dlast;
    void* dx;
    void* dstate;
    float* part;  // (blocks, W + 1, dim)
    int64_t sx_b, sx_r, sg_b, sg_r, sd_b, sd_r;
    int64_t batch, len, dim;
    uint32_t runs, items;
    int blocks;
    int silu;
};

// The resets of steps t0 - 8 .. t0 + 15 as bits 0 .. 23; steps outside the sequence have none.
__device__ __forceinline__ uint32_t reset_bits(const uint8_t* row, int t0, int len) {
    uint32_t m = 0;
    if (!row) return m;
#pragma unroll
    for (int part = 0; part < 3; ++part) {
        const int s = t0 - 8 + part * 8;
        if (s < 0 || s >= len) continue;
        const Pack<uint8_t, 8> r = load_some<uint8_t, 8>(row + s, len - s);
#pragma unroll
        for (int k = 0; k < 8; ++k) m |= (r.v[k] ? 1u : 0u) << (part * 8 + k);
    }
    return m;
}

// Steps from the last reset to that of bit i, 0 at a reset; W - 1 or more where there is none near.
__device__ __forceinline__ int age_of(uint32_t bits, int i) { return __clz((int)(bits << (31 - i))); }
__device__ __forceinline__ float act_f(float pre, int silu) { return silu ? silu_f(pre) : pre; }
__device__ __forceinline__ float dact_f(float pre, int silu) {
    if (!silu) return 1.0f;
    const float s = hw_rcp(1.0f + hw_exp2(-pre * kLog2e));
    return s * __builtin_fmaf(pre, 1.0f - s, 1.0f);
}

// Row j of the state that the sequence leaves: the value of step s = len - (W - 1) + j, or the initial state's
// row s + W - 1, or zero where a reset lies after it.
template <int W>
__device__ __forceinline__ bool left_alive(const uint8_t* reset, int64_t len, int j) {
    if (!reset) return true;
    bool ok = true;
    for (int q = 1; q < W; ++q) {  // resets after s, up to the last step
        const int64_t t = len - q;
        if (t >= 0 && q < W - 1 - j && reset[t]) ok = false;
    }
    return ok;
}

// ---- channels side by side ----

template <typename S, int W, bool STEPS_OUT>
__global__ __launch_bounds__(kConvThreads) void conv_rows_fwd_kernel(ConvArgs p) {
    constexpr int V = 16 / sizeof(S), CG = kGroup / V, TG = kConvThreads / CG;
    constexpr int QPI = kRun / V, SLOTS = TG * QPI;  // 16-byte pieces of a run; of a workgroup's runs
    static_assert(SLOTS == 32 && CG <= SLOTS);
    using P = Pack<S, V>;
    __shared__ P tile[STEPS_OUT ? kGroup * SLOTS : 1];
    const int tid = threadIdx.x, cg = tid % CG, tg = tid / CG;
    const int groups = (int)((p.dim + kGroup - 1) / kGroup);
    const int group = blockIdx.x % groups;
    const int64_t c0 = (int64_t)group * kGroup + cg * V;
    const int n = (int)(p.dim - c0 < V ? p.dim - c0 : V);  // channels of this thread's pack, none if n <= 0
    const int len = (int)p.len;

    float w[V][W], b[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int k = 0; k < W; ++k) w[v][k] = v < n ? p.w[(c0 + v) * W + k] : 0.0f;
        b[v] = p.b && v < n ? p.b[c0 + v] : 0.0f;
    }
    for (uint32_t first = (blockIdx.x / groups) * TG; first < p.items; first += (uint32_t)p.blocks * TG) {
        const uint32_t item = first + tg;
        if (n > 0 && item < p.items) {
            const uint32_t bt = item / p.runs;
            const int t0 = (int)(item - bt * p.runs) * kRun;
            const S* x = static_cast<const S*>(p.x) + bt * p.sx_b + c0;
            P in[W - 1 + kRun];
#pragma unroll
            for (int i = 0; i < W - 1 + kRun; ++i) {
                const int t = t0 + i - (W - 1);
                in[i] = load_some<S, V>(x + t * p.sx_r, t >= 0 && t < len ? n : 0);
            }
            const S* state = static_cast<const S*>(p.state) + (int64_t)bt * (W - 1) * p.dim + c0;
            if (t0 == 0 && p.state) {
#pragma unroll
                for (int i = 0; i < W - 1; ++i) in[i] = load_some<S, V>(state + i * p.dim, n);
            }
            const uint8_t* reset = p.reset ? p.reset + bt * p.len : nullptr;
            const uint32_t bits = reset_bits(reset, t0, len);
            if (t0 == 0 && p.last) {
                // before anything of this thread's channels is written over: the old state is in `in`
                S* last = static_cast<S*>(p.last) + (int64_t)bt * (W - 1) * p.dim + c0;
#pragma unroll
                for (int j = 0; j < W - 1; ++j) {
                    const int s = len - (W - 1) + j;
                    P r;
                    if (s >= 0) {
                        r = load_some<S, V>(x + s * p.sx_r, n);
                    } else {
#pragma unroll
                        for (int i = 0; i < W - 1; ++i)
                            if (i == s + W - 1) r = in[i];
                    }
                    if (!left_alive<W>(reset, len, j)) r = load_some<S, V>(x, 0);
                    store_some<S, V>(last + j * p.dim, r, n);
                }
            }
            P out[kRun];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                P line[QPI];
#pragma unroll
                for (int i = 0; i < kRun; ++i) {
                    float pre = b[v];
                    const int age = age_of(bits, 8 + i);
#pragma unroll
                    for (int j = W - 1; j >= 0; --j) {
                        const float value = to_f32(in[W - 1 + i - j].v[v]);
                        pre = __builtin_fmaf(w[v][W - 1 - j], j <= age ? value : 0.0f, pre);
                    }
                    const S r = from_f32<S>(act_f(pre, p.silu));
                    if constexpr (STEPS_OUT) line[i / V].v[i % V] = r;
                    else out[i].v[v] = r;
                }
                if constexpr (STEPS_OUT) {
#pragma unroll
                    for (int h = 0; h < QPI; ++h) tile[(cg * V + v) * SLOTS + ((tg * QPI + h) ^ cg)] = line[h];
                }
            }
            if constexpr (!STEPS_OUT) {
                S* y = static_cast<S*>(p.y) + bt * p.sy_b + c0;
#pragma unroll
                for (int i = 0; i < kRun; ++i)
                    if (t0 + i < len) store_some<S, V>(y + (t0 + i) * p.sy_r, out[i], n);
            }
        }
        if constexpr (STEPS_OUT) {
            __syncthreads();
            for (int k = tid; k < kGroup * SLOTS; k += kConvThreads) {
                const int c = k / SLOTS, slot = k % SLOTS;
                const uint32_t it = first + slot / QPI;
                const int64_t ch = (int64_t)group * kGroup + c;
                if (it >= p.items || ch >= p.dim) continue;
                const uint32_t bt = it / p.runs;
                const int t = (int)(it - bt * p.runs) * kRun + slot % QPI * V;
                if (t < len)
                    store_some<S, V>(static_cast<S*>(p.y) + bt * p.sy_b + ch * p.sy_r + t, tile[c * SLOTS + (slot ^ (c / V))],
                                     len - t);
            }
            __syncthreads();
        }
    }
}

template <typename S, int W, bool STEPS_OUT>
__global__ __launch_bounds__(kConvThreads) void conv_rows_bwd_kernel(ConvBwdArgs p) {
    constexpr int V = 4, CG = kGroup / V, TG = kConvThreads / CG;
    constexpr int NX = 2 * (W - 1) + kRun, NG = W - 1 + kRun, GW = 12;  // GW: steps of dy kept for a run
    constexpr int PITCH = TG * GW + 4;                                  // of a channel's runs in LDS
    using P = Pack<S, V>;
    constexpr int TILE = STEPS_OUT ? kGroup * PITCH * (int)sizeof(S) : 16, SUMS = TG * kGroup * (W + 1) * 4;
    __shared__ __align__(16) char lds[TILE > SUMS ? TILE : SUMS];
    S* tile = reinterpret_cast<S*>(lds);
    const int tid = threadIdx.x, cg = tid % CG, tg = tid / CG;
    const int groups = (int)((p.dim + kGroup - 1) / kGroup);
    const int group = blockIdx.x % groups, block = blockIdx.x / groups;
    const int64_t c0 = (int64_t)group * kGroup + cg * V;
    const int n = (int)(p.dim - c0 < V ? p.dim - c0 : V);
    const int len = (int)p.len;

    float w[V][W], b[V], dw[V][W], db[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int k = 0; k < W; ++k) w[v][k] = v < n ? p.w[(c0 + v) * W + k] : 0.0f, dw[v][k] = 0.0f;
        b[v] = p.b && v < n ? p.b[c0 + v] : 0.0f;
        db[v] = 0.0f;
    }
    for (uint32_t first = (uint32_t)block * TG; first < p.items; first += (uint32_t)p.blocks * TG) {
        if constexpr (STEPS_OUT) {
            // dy's runs of 64 channels, with the W - 1 steps behind each
            for (int k = tid; k < kGroup * TG; k += kConvThreads) {
                const int c = k / TG, slot = k % TG;
                const uint32_t it = first + slot;
                const int64_t ch = (int64_t)group * kGroup + c;
                const bool on = it < p.items && ch < p.dim;
                const uint32_t bt = on ? it / p.runs : 0;
                const int t = on ? (int)(it - bt * p.runs) * kRun : len;
                const S* g = static_cast<const S*>(p.dy) + bt * p.sg_b + (on ? ch : 0) * p.sg_r;
                S* to = tile + c * PITCH + slot * GW;
#pragma unroll
                for (int h = 0; h < 3; ++h) {
                    const P r = load_some<S, 4>(g + t + 4 * h, len - t - 4 * h);
                    *reinterpret_cast<P*>(to + 4 * h) = r;
                }
            }
            __syncthreads();
        }
        const uint32_t item = first + tg;
        if (n > 0 && item < p.items) {
            const uint32_t bt = item / p.runs;
            const int t0 = (int)(item - bt * p.runs) * kRun;
            const S* x = static_cast<const S*>(p.x) + bt * p.sx_b + c0;
            P in[NX], g[STEPS_OUT ? 1 : NG];
#pragma unroll
            for (int i = 0; i < NX; ++i) {
                const int t = t0 + i - (W - 1);
                in[i] = load_some<S, V>(x + t * p.sx_r, t >= 0 && t < len ? n : 0);
            }
            if constexpr (!STEPS_OUT) {
                const S* dy = static_cast<const S*>(p.dy) + bt * p.sg_b + c0;
#pragma unroll
                for (int i = 0; i < NG; ++i) g[i] = load_some<S, V>(dy + (t0 + i) * p.sg_r, t0 + i < len ? n : 0);
            }
            const int64_t st = (int64_t)bt * (W - 1) * p.dim + c0;
            if (t0 == 0 && p.state) {
#pragma unroll
                for (int i = 0; i < W - 1; ++i) in[i] = load_some<S, V>(static_cast<const S*>(p.state) + st + i * p.dim, n);
            }
            const uint8_t* reset = p.reset ? p.reset + bt * p.len : nullptr;
            const uint32_t bits = reset_bits(reset, t0, len);
            // gradients of the values of steps t0 - (W - 1) .. t0 + kRun - 1; those before t0 are the initial
            // state's, in a sequence's first run
            float dv[V][W - 1 + kRun];
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int i = 0; i < W - 1 + kRun; ++i) dv[v][i] = 0.0f;
            if (p.dlast && t0 + kRun + W - 1 > len) {
#pragma unroll
                for (int i = 0; i < W - 1 + kRun; ++i) {
                    const int s = t0 + i - (W - 1), j = s - (len - (W - 1));
                    if (j < 0 || j >= W - 1 || (t0 > 0 && i < W - 1) || !left_alive<W>(reset, len, j)) continue;
                    const P r = load_some<S, V>(static_cast<const S*>(p.dlast) + st + j * p.dim, n);
#pragma unroll
                    for (int v = 0; v < V; ++v) dv[v][i] = to_f32(r.v[v]);
                }
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float line[GW];
                if constexpr (STEPS_OUT) {
                    const S* from = tile + (cg * V + v) * PITCH + tg * GW;
#pragma unroll
                    for (int h = 0; h < 3; ++h) {
                        const P r = *reinterpret_cast<const P*>(from + 4 * h);
#pragma unroll
                        for (int k = 0; k < 4; ++k) line[4 * h + k] = to_f32(r.v[k]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < NG; ++i) line[i] = to_f32(g[i].v[v]);
                }
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    const int age = age_of(bits, 8 + i);
                    float pre = b[v], seen[W];
#pragma unroll
                    for (int j = W - 1; j >= 0; --j) {
                        const float value = to_f32(in[W - 1 + i - j].v[v]);
                        seen[j] = j <= age ? value : 0.0f;
                        pre = __builtin_fmaf(w[v][W - 1 - j], seen[j], pre);
                    }
                    const float d = t0 + i < len ? line[i] * dact_f(pre, p.silu) : 0.0f;
                    if (i < kRun) {
                        db[v] += d;
#pragma unroll
                        for (int j = 0; j < W; ++j) dw[v][W - 1 - j] = __builtin_fmaf(d, seen[j], dw[v][W - 1 - j]);
                    }
#pragma unroll
                    for (int j = 0; j < W; ++j) {
                        const int to = W - 1 + i - j;
                        if (to < W - 1 + kRun) dv[v][to] = __builtin_fmaf(w[v][W - 1 - j], j <= age ? d : 0.0f, dv[v][to]);
                    }
                }
            }
            S* dx = static_cast<S*>(p.dx) + bt * p.sd_b + c0;
#pragma unroll
            for (int i = 0; i < W - 1 + kRun; ++i) {
                P r;
#pragma unroll
                for (int v = 0; v < V; ++v) r.v[v] = from_f32<S>(dv[v][i]);
                const int t = t0 + i - (W - 1);
                if (i >= W - 1) {
                    if (t < len) store_some<S, V>(dx + t * p.sd_r, r, n);
                } else if (t0 == 0 && p.dstate) {
                    store_some<S, V>(static_cast<S*>(p.dstate) + st + i * p.dim, r, n);
                }
            }
        }
        if constexpr (STEPS_OUT) __syncthreads();
    }
    // the threads' sums of a channel, in the order of their runs
    float* sums = reinterpret_cast<float*>(lds);  // (TG, W + 1, kGroup)
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int k = 0; k < W; ++k) sums[(tg * (W + 1) + k) * kGroup + cg * V + v] = dw[v][k];
        sums[(tg * (W + 1) + W) * kGroup + cg * V + v] = db[v];
    }
    __syncthreads();
    for (int k = tid; k < kGroup * (W + 1); k += kConvThreads) {
        const int64_t c = (int64_t)group * kGroup + k % kGroup;
        if (c >= p.dim) continue;
        float s = 0.0f;
#pragma unroll
        for (int q = 0; q < TG; ++q) s += sums[q * kGroup * (W + 1) + k];
        p.part[((int64_t)block * (W + 1) + k / kGroup) * p.dim + c] = s;
    }
}

// ---- steps side by side ----

// kRun + M values of a channel from step t0 - B on, zeros outside the sequence.
template <typename S, int B, int N>
__device__ __forceinline__ void load_line(const S* row, int t0, int len, float (&to)[N]) {
    static_assert(N % 4 == 0);
#pragma unroll
    for (int h = 0; h < N / 4; ++h) {
        const int t = t0 - B + 4 * h;
        const Pack<S, 4> r = load_some<S, 4>(row + t, t < 0 ? 0 : len - t);
#pragma unroll
        for (int k = 0; k < 4; ++k) to[4 * h + k] = to_f32(r.v[k]);
    }
}

template <typename S, int W>
__global__ __launch_bounds__(kConvThreads) void conv_steps_fwd_kernel(ConvArgs p, int64_t total) {
    const int64_t id = grid_block() * kConvThreads + threadIdx.x;
    if (id >= total) return;
    const int len = (int)p.len;
    // rows (batch, channel) one after another, each of `runs` runs
    const int64_t row = id / p.runs;
    const int t0 = (int)(id - row * p.runs) * kRun;
    const int64_t bt = row / p.dim, c = row - bt * p.dim;
    const S* x = static_cast<const S*>(p.x) + bt * p.sx_b + c * p.sx_r;
    float in[4 + kRun];  // steps t0 - 4 ..
    load_line<S, 4>(x, t0, len, in);
    const int64_t st = bt * (W - 1) * p.dim + c;
    if (t0 == 0 && p.state) {
#pragma unroll
        for (int i = 0; i < W - 1; ++i) in[4 - (W - 1) + i] = to_f32(static_cast<const S*>(p.state)[st + i * p.dim]);
    }
    const uint8_t* reset = p.reset ? p.reset + bt * p.len : nullptr;
    const uint32_t bits = reset_bits(reset, t0, len);
    if (t0 == 0 && p.last) {
        S* last = static_cast<S*>(p.last) + st;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int s = len - (W - 1) + j;
            float r = 0.0f;
            if (s >= 0) {
                r = to_f32(x[s]);
            } else {
#pragma unroll
                for (int i = 0; i < W - 1; ++i)
                    if (i == s + W - 1) r = in[4 - (W - 1) + i];
            }
            if (!left_alive<W>(reset, len, j)) r = 0.0f;
            last[j * p.dim] = from_f32<S>(r);
        }
    }
    float w[W];
#pragma unroll
    for (int k = 0; k < W; ++k) w[k] = p.w[c * W + k];
    const float b = p.b ? p.b[c] : 0.0f;
    Pack<S, kRun> out;
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
        const int age = age_of(bits, 8 + i);
        float pre = b;
#pragma unroll
        for (int j = W - 1; j >= 0; --j) pre = __builtin_fmaf(w[W - 1 - j], j <= age ? in[4 + i - j] : 0.0f, pre);
        out.v[i] = from_f32<S>(act_f(pre, p.silu));
    }
    store_some<S, kRun>(static_cast<S*>(p.y) + bt * p.sy_b + c * p.sy_r + t0, out, len - t0);
}

// A workgroup: one channel, every `blocks`-th stretch of its sequences' runs.
template <typename S, int W>
__global__ __launch_bounds__(kConvThreads) void conv_steps_bwd_kernel(ConvBwdArgs p) {
    const int64_t c = blockIdx.x / p.blocks;
    const int block = blockIdx.x % p.blocks;
    const int len = (int)p.len;
    float w[W], dw[W], db = 0.0f;
#pragma unroll
    for (int k = 0; k < W; ++k) w[k] = p.w[c * W + k], dw[k] = 0.0f;
    const float b = p.b ? p.b[c] : 0.0f;
    for (uint32_t item = (uint32_t)block * kConvThreads + threadIdx.x; item < p.items; item += (uint32_t)p.blocks * kConvThreads) {
        const uint32_t bt = item / p.runs;
        const int t0 = (int)(item - bt * p.runs) * kRun;
        float in[4 + kRun + 4], g[kRun + 4];
        load_line<S, 4>(static_cast<const S*>(p.x) + bt * p.sx_b + c * p.sx_r, t0, len, in);
        load_line<S, 0>(static_cast<const S*>(p.dy) + bt * p.sg_b + c * p.sg_r, t0, len, g);
        const int64_t st = (int64_t)bt * (W - 1) * p.dim + c;
        if (t0 == 0 && p.state) {
#pragma unroll
            for (int i = 0; i < W - 1; ++i) in[4 - (W - 1) + i] = to_f32(static_cast<const S*>(p.state)[st + i * p.dim]);
        }
        const uint8_t* reset = p.reset ? p.reset + bt * p.len : nullptr;
        const uint32_t bits = reset_bits(reset, t0, len);
        float dv[W - 1 + kRun];
#pragma unroll
        for (int i = 0; i < W - 1 + kRun; ++i) dv[i] = 0.0f;
        if (p.dlast && t0 + kRun + W - 1 > len) {
#pragma unroll
            for (int i = 0; i < W - 1 + kRun; ++i) {
                const int s = t0 + i - (W - 1), j = s - (len - (W - 1));
                if (j < 0 || j >= W - 1 || (t0 > 0 && i < W - 1) || !left_alive<W>(reset, len, j)) continue;
                dv[i] = to_f32(static_cast<const S*>(p.dlast)[st + j * p.dim]);
            }
        }
#pragma unroll
        for (int i = 0; i < W - 1 + kRun; ++i) {
            const int age = age_of(bits, 8 + i);
            float pre = b, seen[W];
#pragma unroll
            for (int j = W - 1; j >= 0; --j) {
                seen[j] = j <= age ? in[4 + i - j] : 0.0f;
                pre = __builtin_fmaf(w[W - 1 - j], seen[j], pre);
            }
            const float d = t0 + i < len ? g[i] * dact_f(pre, p.silu) : 0.0f;
            if (i < kRun) {
                db += d;
#pragma unroll
                for (int j = 0; j < W; ++j) dw[W - 1 - j] = __builtin_fmaf(d, seen[j], dw[W - 1 - j]);
            }
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const int to = W - 1 + i - j;
                if (to < W - 1 + kRun) dv[to] = __builtin_fmaf(w[W - 1 - j], j <= age ? d : 0.0f, dv[to]);
            }
        }
        Pack<S, kRun> out;
#pragma unroll
        for (int i = 0; i < kRun; ++i) out.v[i] = from_f32<S>(dv[W - 1 + i]);
        store_some<S, kRun>(static_cast<S*>(p.dx) + bt * p.sd_b + c * p.sd_r + t0, out, len - t0);
        if (t0 == 0 && p.dstate) {
#pragma unroll
            for (int i = 0; i < W - 1; ++i) static_cast<S*>(p.dstate)[st + i * p.dim] = from_f32<S>(dv[i]);
        }
    }
    __shared__ float sums[kConvThreads / 64][kMaxWidth + 1];
    const int wave = threadIdx.x >> 6;
#pragma unroll
    for (int k = 0; k <= W; ++k) {
        const float s = wave_sum(k < W ? dw[k < W ? k : 0] : db);
        if ((threadIdx.x & 63) == 0) sums[wave][k] = s;
    }
    __syncthreads();
    if (threadIdx.x <= W) {
        float s = 0.0f;
#pragma unroll
        for (int q = 0; q < kConvThreads / 64; ++q) s += sums[q][threadIdx.x];
        p.part[((int64_t)block * (W + 1) + threadIdx.x) * p.dim + c] = s;
    }
}

// The workgroups' partial sums, added in order.
__global__ __launch_bounds__(256) void conv_join_kernel(const float* part, int blocks, int width, int64_t dim, float* dw, float* db) {
    const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (k >= dim * (width + 1)) return;
    float s = 0.0f;
#pragma unroll 8
    for (int q = 0; q < blocks; ++q) s += part[q * dim * (width + 1) + k];
    const int64_t tap = k / dim, c = k - tap * dim;
    if (tap < width) {
        if (dw) dw[c * width + tap] = s;
    } else if (db) {
        db[c] = s;
    }
}

uint32_t runs_of(const mamba_conv_shape& s) { return s.len > 0 ? (uint32_t)((s.len + kRun - 1) / kRun) : 1; }

int64_t groups_of(const mamba_conv_shape& s) { return (s.dim + kGroup - 1) / kGroup; }

// Workgroups a group of channels (or a channel): as many as the GPU holds at a time, each to take several
// stretches of runs with the weights it has loaded.
int blocks_of(int64_t items, int64_t each, int64_t groups, int per_cu) {
    const int64_t need = (items + each - 1) / each, most = (int64_t)layers_cus() * per_cu / groups;
    const int64_t n = need < most ? need : most;
    return (int)(n < 1 ? 1 : n);
}
constexpr int kFwdPerCu = 8, kBwdPerCu = 4, kStepsBwdPerCu = 8;

int bwd_blocks(const mamba_conv_shape& s, bool x_steps) {
    const int64_t items = s.batch * runs_of(s);
    return x_steps ? blocks_of(items, kConvThreads, s.dim, kStepsBwdPerCu)
                   : blocks_of(items, kConvThreads / (kGroup / 4), groups_of(s), kBwdPerCu);
}

template <typename S, int W>
void fwd_go(ConvArgs q, bool x_steps, bool y_steps, int64_t groups, Launches& on) {
    if (x_steps) {
        const int64_t total = q.batch * q.dim * q.runs;
        on(conv_steps_fwd_kernel<S, W>, grid_of((total + kConvThreads - 1) / kConvThreads, kConvThreads), dim3(kConvThreads), q, total);
        return;
    }
    q.blocks = blocks_of(q.items, kConvThreads / (kGroup / (16 / (int)sizeof(S))), groups, kFwdPerCu);
    const dim3 grid((unsigned)(groups * q.blocks));
    if (y_steps) on(conv_rows_fwd_kernel<S, W, true>, grid, dim3(kConvThreads), q);
    else on(conv_rows_fwd_kernel<S, W, false>, grid, dim3(kConvThreads), q);
}

template <typename S, int W>
void bwd_go(const ConvBwdArgs& q, bool x_steps, bool g_steps, int64_t groups, Launches& on) {
    if (x_steps) {
        on(conv_steps_bwd_kernel<S, W>, dim3((unsigned)(q.dim * q.blocks)), dim3(kConvThreads), q);
        return;
    }
    const dim3 grid((unsigned)(groups * q.blocks));
    if (g_steps) on(conv_rows_bwd_kernel<S, W, true>, grid, dim3(kConvThreads), q);
    else on(conv_rows_bwd_kernel<S, W, false>, grid, dim3(kConvThreads), q);
}

template <typename F>
void with_width(int64_t width, F&& f) {
    if (width == 1) f(std::integral_constant<int, 1>{});
    else if (width == 2) f(std::integral_constant<int, 2>{});
    else if (width == 3) f(std::integral_constant<int, 3>{});
    else f(std::integral_constant<int, 4>{});
}

}  // namespace

int launch_conv_fwd(const mamba_conv_ptrs& p, const mamba_conv_shape& s, int act, bool bf16, hipStream_t stream) {
    ConvArgs q{p.x, p.weight, p.bias, p.initial_state, p.reset, p.y, p.last_state, p.x_batch, p.x_row, p.y_batch, p.y_row,
               s.batch, s.len, s.dim, runs_of(s), (uint32_t)(s.batch * runs_of(s)), 1, act == MAMBA_CONV_SILU};
    Launches on(stream);
    with_width(s.width, [&](auto w) {
        constexpr int W = decltype(w)::value;
        bf16 ? fwd_go<bf16_t, W>(q, p.x_steps, p.y_steps, groups_of(s), on) : fwd_go<float, W>(q, p.x_steps, p.y_steps, groups_of(s), on);
    });
    return on.status;
}

int64_t conv_bwd_workspace(const mamba_conv_shape& s, bool bf16, bool x_steps) {
    return align256((int64_t)bwd_blocks(s, x_steps) * (s.width + 1) * s.dim * 4);
}

int launch_conv_bwd(const mamba_conv_bwd_ptrs& p, const mamba_conv_shape& s, int act, bool bf16, hipStream_t stream) {
    ConvBwdArgs q{p.x, p.weight, p.bias, p.initial_state, p.reset, p.dy, p.dlast_state, p.dx, p.dinitial_state,
                  static_cast<float*>(p.workspace), p.x_batch, p.x_row, p.dy_batch, p.dy_row, p.dx_batch, p.dx_row,
                  s.batch, s.len, s.dim, runs_of(s), (uint32_t)(s.batch * runs_of(s)), bwd_blocks(s, p.x_steps),
                  act == MAMBA_CONV_SILU};
    Launches on(stream);
    with_width(s.width, [&](auto w) {
        constexpr int W = decltype(w)::value;
        bf16 ? bwd_go<bf16_t, W>(q, p.x_steps, p.dy_steps, groups_of(s), on) : bwd_go<float, W>(q, p.x_steps, p.dy_steps, groups_of(s), on);
    });
    on(conv_join_kernel, dim3((unsigned)((s.dim * (s.width + 1) + 255) / 256)), dim3(256), static_cast<const float*>(p.workspace),
       q.blocks, (int)s.width, s.dim, p.dweight, p.dbias);
    return on.status;
}

}  // namespace mscan
