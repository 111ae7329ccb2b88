// Short causal convolution of each channel with its activation (mamba_block.h) and its gradient, on gfx950.
//
//   pre_t = bias + sum_{j < W} w_{W-1-j} v_{t-j},   y_t = silu(pre_t)        (tap j reaches j steps back)
//   dpre_t = dy_t silu'(pre_t);   dv_s = sum_j w_{W-1-j} dpre_{s+j};   dw_{W-1-j} = sum_t dpre_t v_{t-j}
//
// Where channels lie side by side ("rows" kernels), a wave takes a run of 32 steps of 128 channels and walks through
// it with the last W values, and in the backward the W gradients that are not finished, in registers. Where steps do
// ("steps" kernels, the scan's layout), a thread takes a run of 8 steps of one channel. What a run needs of its
// neighbours (W - 1 steps before it and, in the backward, behind it) is loaded again, from the cache, or read from the
// next lane. A tap is dropped where a sequence begins between the value and the step: the number of steps since the
// last reset is counted along the run, or is the leading zeros of the resets' bits up to a step.
//
// Rows in, steps out (a projection's output handed to the scan): a workgroup's results pass through LDS in 16-byte
// pieces whose places are XORed with the channel, so that rows are read and rows are written in whole lines; the
// backward takes dy the same way.
//
// Bound by HBM, each value read and written once; the weight's gradient is summed in registers over a workgroup's
// runs, then over its waves in order, and a second kernel adds the workgroups'. 8 x 2048 x 1536 bf16: forward 21.8 us
// (101 MB, 4.6 TB/s, a large copy's rate), into the scan's layout 24 (4.2), gradient 39.5 + 4.8 (151 MB, 3.8; the
// vector instructions alone about 16); in the scan's layout 21 and 66 (in the latter the vector instructions take
// about 30, a third of them loading a turn and joining a workgroup's sums after four or five). 3 x 2777 x 1001 fp32 in
// the scan's layout 17 and 30. One step of 32 x 1536: 3.6.
#include <type_traits>

#include "block_launch.hpp"
#include "layers_common.hpp"
#include "rows.hpp"

namespace mscan {

namespace {

constexpr int kRun = 8;       // steps of a thread's run where steps lie side by side
constexpr int kConvThreads = 256;
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

// The resets of steps t0 - 8 .. t0 + kRun + 7 as bits from 0 on; steps outside the sequence have none.
__device__ __forceinline__ uint32_t reset_bits(const uint8_t* row, int t0, int len) {
    static_assert(kRun + 16 <= 32);
    uint32_t m = 0;
    if (!row) return m;
#pragma unroll
    for (int part = 0; part < kRun / 8 + 2; ++part) {
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
//
// A wave takes a run of steps of 64 packs of channels, so that the step, and whether a sequence begins at it, are the
// same for all its lanes: the resets around a run are one 64-bit mask, and a run without any goes without a test.
// Rows are loaded kAhead at a time, the next ones while these are worked on; a value stays in registers for the
// W - 1 steps that see it.

constexpr int kV = 2;              // channels of a lane
constexpr int kCols = 64 * kV;     // of a workgroup
constexpr int kWaves = 4;
constexpr int kRowRun = 32;        // steps of a wave's run, in the backward with the W - 1 behind it
constexpr int kAhead = 8;
enum { kAny, kFirst, kMiddle, kLast };  // turns of the backward

// A lane's kV channels of a row that begins at `row`. EVEN (an even number of channels): lanes past the last pair
// repeat it, in the same wave, so that neither loads nor stores are masked. Otherwise each channel is loaded by itself,
// the last one again where there is none, as a branch around every load costs more (8 x 2048 x 1537 bf16, forward
// and backward: 205 us with branches, 147 without; 121 with the backward's turns of whole runs).
template <typename S, bool EVEN>
struct Cols {
    static_assert(kV == 2);
    uint32_t at, at1;  // bytes from a row's start; of the second channel
    int n;             // channels that are there
    __device__ __forceinline__ Cols(int64_t c0, int64_t dim) {
        n = (int)(dim - c0 < kV ? dim - c0 : kV);
        if constexpr (EVEN) {
            at = (uint32_t)((n < kV ? dim - kV : c0) * sizeof(S)), at1 = at + sizeof(S);
        } else {
            at = (uint32_t)((n < 1 ? dim - 1 : c0) * sizeof(S)), at1 = n < 2 ? at : at + sizeof(S);
        }
    }
    __device__ __forceinline__ Pack<S, kV> load(const void* row) const {
        const char* p = static_cast<const char*>(row);
        Pack<S, kV> r;
        if constexpr (EVEN) __builtin_memcpy(&r, p + at, sizeof(r));
        else r.v[0] = *reinterpret_cast<const S*>(p + at), r.v[1] = *reinterpret_cast<const S*>(p + at1);
        return r;
    }
    __device__ __forceinline__ void store(void* row, const Pack<S, kV>& r) const {
        S* p = reinterpret_cast<S*>(static_cast<char*>(row) + at);
        if constexpr (EVEN) __builtin_memcpy(p, &r, sizeof(r));
        else store_some<S, kV>(p, r, n);
    }
};

// Bit i: whether a sequence begins at step t0 - 2 + i, of a run's steps and the two before it.
__device__ __forceinline__ uint64_t reset_mask(const uint8_t* row, int t0, int len) {
    if (!row) return 0;
    const int lane = threadIdx.x & 63, t = t0 - 2 + lane;
    return __ballot(lane < kRowRun + 2 && t >= 0 && t < len && row[t] != 0);
}

// Steps since the last reset, as a run's steps are walked through.
struct Age {
    uint64_t mask;
    int age;
    __device__ __forceinline__ explicit Age(uint64_t m) : mask(m), age(kMaxWidth) { next(), next(); }
    __device__ __forceinline__ void next() { age = mask & 1 ? 0 : age + 1, mask >>= 1; }
};

template <typename S, int W, bool STEPS_OUT, bool EVEN>
__global__ __launch_bounds__(64 * kWaves) void conv_rows_fwd_kernel(ConvArgs p) {
    constexpr int Q = 16 / sizeof(S), QPI = kRowRun / Q, SLOTS = kWaves * QPI;  // 16-byte pieces of a run's steps; of all
    using P = Pack<S, kV>;
    using Line = Pack<S, Q>;
    __shared__ Line tile[STEPS_OUT ? kCols * SLOTS : 1];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int groups = (int)((p.dim + kCols - 1) / kCols);
    const int group = blockIdx.x % groups;
    const int64_t c0 = (int64_t)group * kCols + lane * kV;
    const Cols<S, EVEN> cols(c0, p.dim);
    const int64_t cw = EVEN && c0 > p.dim - kV ? p.dim - kV : c0;  // the channels themselves
    const int len = (int)p.len;

    float w[kV][W], b[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) {
#pragma unroll
        for (int k = 0; k < W; ++k) w[v][k] = EVEN || v < cols.n ? p.w[(cw + v) * W + k] : 0.0f;
        b[v] = p.b && (EVEN || v < cols.n) ? p.b[cw + v] : 0.0f;
    }
    for (uint32_t first = (blockIdx.x / groups) * kWaves; first < p.items; first += (uint32_t)p.blocks * kWaves) {
        const uint32_t item = first + wave;
        if (item < p.items) {
            const uint32_t bt = item / p.runs;
            const int t0 = (int)(item - bt * p.runs) * kRowRun, steps = len - t0 < kRowRun ? len - t0 : kRowRun;
            const S* x = static_cast<const S*>(p.x) + bt * p.sx_b;
            S* y = static_cast<S*>(p.y) + bt * p.sy_b;
            const uint8_t* reset = p.reset ? p.reset + bt * p.len : nullptr;
            const int64_t st = (int64_t)bt * (W - 1) * p.dim;
            P next[kAhead], before[W - 1 > 0 ? W - 1 : 1]{};
            auto fetch = [&](int i0) __attribute__((always_inline)) {  // (behind the last row, that row again)
#pragma unroll
                for (int i = 0; i < kAhead; ++i) next[i] = cols.load(x + (t0 + (i0 + i < steps ? i0 + i : steps - 1)) * p.sx_r);
            };
            if (steps > 0) fetch(0);
#pragma unroll
            for (int i = 0; i < W - 1; ++i) {
                if (t0 > 0) before[i] = cols.load(x + (t0 - (W - 1) + i) * p.sx_r);
                else if (p.state) before[i] = cols.load(static_cast<const S*>(p.state) + st + i * p.dim);
            }
            const uint64_t mask = reset_mask(reset, t0, len);
            if (t0 == 0 && p.last) {
                // before anything of these channels is written over: the old state is in `before`
#pragma unroll
                for (int j = 0; j < W - 1; ++j) {
                    const int s = len - (W - 1) + j;
                    P r{};
                    if (left_alive<W>(reset, len, j)) {
                        if (s >= 0) r = cols.load(x + s * p.sx_r);
                        else
#pragma unroll
                            for (int i = 0; i < W - 1; ++i)
                                if (i == s + W - 1) r = before[i];
                    }
                    cols.store(static_cast<S*>(p.last) + st + j * p.dim, r);
                }
            }
            float seen[W][kV];  // seen[j]: the value of j steps back
#pragma unroll
            for (int j = 1; j < W; ++j)
#pragma unroll
                for (int v = 0; v < kV; ++v) seen[j - 1][v] = to_f32(before[W - 1 - j].v[v]);
            auto run = [&](auto cut) __attribute__((always_inline)) {
                Age age(mask);
                for (int i0 = 0; i0 < steps; i0 += kAhead) {
                    P now[kAhead];
#pragma unroll
                    for (int i = 0; i < kAhead; ++i) now[i] = next[i];
                    if (i0 + kAhead < steps) fetch(i0 + kAhead);
                    Line line[kV][kAhead / Q];
#pragma unroll
                    for (int i = 0; i < kAhead; ++i) {
                        P out;
                        if constexpr (decltype(cut)::value) age.next();
#pragma unroll
                        for (int v = 0; v < kV; ++v) {
#pragma unroll
                            for (int j = W - 1; j > 0; --j) seen[j][v] = !decltype(cut)::value || j <= age.age ? seen[j - 1][v] : 0.0f;
                            seen[0][v] = to_f32(now[i].v[v]);
                            float pre = b[v];
#pragma unroll
                            for (int j = W - 1; j >= 0; --j) pre = __builtin_fmaf(w[v][W - 1 - j], seen[j][v], pre);
                            out.v[v] = from_f32<S>(act_f(pre, p.silu));
                            if constexpr (STEPS_OUT) line[v][i / Q].v[i % Q] = out.v[v];
                        }
                        if constexpr (!STEPS_OUT)
                            if (i0 + i < steps) cols.store(y + (t0 + i0 + i) * p.sy_r, out);
                    }
                    if constexpr (STEPS_OUT) {
#pragma unroll
                        for (int v = 0; v < kV; ++v)
#pragma unroll
                            for (int h = 0; h < kAhead / Q; ++h)
                                tile[(lane * kV + v) * SLOTS + ((wave * QPI + i0 / Q + h) ^ (lane & (SLOTS - 1)))] = line[v][h];
                    }
                }
            };
            if (mask == 0) run(std::false_type{});
            else run(std::true_type{});
        }
        if constexpr (STEPS_OUT) {
            __syncthreads();
            for (int k = threadIdx.x; k < kCols * SLOTS; k += 64 * kWaves) {
                const int c = k / SLOTS, slot = k % SLOTS;
                const uint32_t it = first + slot / QPI;
                const int64_t ch = (int64_t)group * kCols + c;
                if (it >= p.items || ch >= p.dim) continue;
                const uint32_t bt = it / p.runs;
                const int t = (int)(it - bt * p.runs) * kRowRun + slot % QPI * Q;
                if (t < len)
                    store_some<S, Q>(static_cast<S*>(p.y) + bt * p.sy_b + ch * p.sy_r + t,
                                     tile[c * SLOTS + (slot ^ (c / kV & (SLOTS - 1)))], len - t);
            }
            __syncthreads();
        }
    }
}

// (bf16: registers for 4 workgroups a CU; left to the compiler 139 and 3: 8 x 2048 x 1536, dy as steps, 80.6 us a pass, 76.6)
template <typename S, int W, bool STEPS_OUT, bool EVEN>
__global__ __launch_bounds__(64 * kWaves, sizeof(S) == 2 ? 4 : 1) void conv_rows_bwd_kernel(ConvBwdArgs p) {
    constexpr int Q = 16 / sizeof(S), QPI = kRowRun / Q, SLOTS = kWaves * QPI, RUN = kRowRun - (W - 1);
    using P = Pack<S, kV>;
    using Line = Pack<S, Q>;
    constexpr int TILE = STEPS_OUT ? kCols * SLOTS * 16 : 16, SUMS = kWaves * kCols * (W + 1) * 4;
    __shared__ __align__(16) char lds[TILE > SUMS ? TILE : SUMS];
    Line* tile = reinterpret_cast<Line*>(lds);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int groups = (int)((p.dim + kCols - 1) / kCols);
    const int group = blockIdx.x % groups, block = blockIdx.x / groups;
    const int64_t c0 = (int64_t)group * kCols + lane * kV;
    const Cols<S, EVEN> cols(c0, p.dim);
    const int64_t cw = EVEN && c0 > p.dim - kV ? p.dim - kV : c0;
    const int pair = (int)(cw - (int64_t)group * kCols) / kV;  // of the workgroup's
    const int len = (int)p.len;

    float w[kV][W], b[kV], dw[kV][W], db[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) {
#pragma unroll
        for (int k = 0; k < W; ++k) w[v][k] = EVEN || v < cols.n ? p.w[(cw + v) * W + k] : 0.0f, dw[v][k] = 0.0f;
        b[v] = p.b && (EVEN || v < cols.n) ? p.b[cw + v] : 0.0f;
        db[v] = 0.0f;
    }
    for (uint32_t first = (uint32_t)block * kWaves; first < p.items; first += (uint32_t)p.blocks * kWaves) {
        if constexpr (STEPS_OUT) {
            // dy's runs of the workgroup's channels, each with the W - 1 steps behind it
            for (int k = threadIdx.x; k < kCols * SLOTS; k += 64 * kWaves) {
                const int c = k / SLOTS, slot = k % SLOTS;
                const uint32_t it = first + slot / QPI;
                const int64_t ch = (int64_t)group * kCols + c;
                const bool on = it < p.items && ch < p.dim;
                const uint32_t bt = on ? it / p.runs : 0;
                const int t = on ? (int)(it - bt * p.runs) * RUN + slot % QPI * Q : len;
                tile[c * SLOTS + (slot ^ (c / kV & (SLOTS - 1)))] =
                    load_some<S, Q>(static_cast<const S*>(p.dy) + bt * p.sg_b + (on ? ch : 0) * p.sg_r + t, len - t);
            }
            __syncthreads();
        }
        const uint32_t item = first + wave;
        if (item < p.items) {
            const uint32_t bt = item / p.runs;
            const int t0 = (int)(item - bt * p.runs) * RUN;
            const int most = len - t0 < RUN ? len - t0 : RUN;                      // steps of the run
            const int steps = len - t0 < kRowRun ? len - t0 : kRowRun;             // that there are with those behind it
            const S* x = static_cast<const S*>(p.x) + bt * p.sx_b;
            const S* dy = static_cast<const S*>(p.dy) + bt * p.sg_b;
            S* dx = static_cast<S*>(p.dx) + bt * p.sd_b;
            const uint8_t* reset = p.reset ? p.reset + bt * p.len : nullptr;
            const int64_t st = (int64_t)bt * (W - 1) * p.dim;
            P nx[kAhead]{}, ng[kAhead]{}, before[W - 1 > 0 ? W - 1 : 1]{};
            auto fetch = [&](int i0) __attribute__((always_inline)) {
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    const int t = t0 + (i0 + i < steps ? i0 + i : steps - 1);
                    nx[i] = cols.load(x + t * p.sx_r);
                    if constexpr (!STEPS_OUT) ng[i] = cols.load(dy + t * p.sg_r);
                }
            };
            if (steps > 0) fetch(0);
#pragma unroll
            for (int i = 0; i < W - 1; ++i) {
                if (t0 > 0) before[i] = cols.load(x + (t0 - (W - 1) + i) * p.sx_r);
                else if (p.state) before[i] = cols.load(static_cast<const S*>(p.state) + st + i * p.dim);
            }
            const uint64_t mask = reset_mask(reset, t0, len);
            float seen[W][kV], dv[W][kV];  // the value of j steps back, and its gradient as far as it has come
#pragma unroll
            for (int v = 0; v < kV; ++v) {
#pragma unroll
                for (int j = 1; j < W; ++j) seen[j - 1][v] = to_f32(before[W - 1 - j].v[v]);
#pragma unroll
                for (int j = 0; j < W; ++j) dv[j][v] = 0.0f;
            }
            // the finished gradient of step s: dx, or the initial state's in a sequence's first run
            auto emit = [&](int s, const float (&g)[kV]) __attribute__((always_inline)) {
                P r;
                float add[kV];
#pragma unroll
                for (int v = 0; v < kV; ++v) add[v] = 0.0f;
                const int j = s - (len - (W - 1));
                if (p.dlast && j >= 0 && left_alive<W>(reset, len, j)) {
                    const P l = cols.load(static_cast<const S*>(p.dlast) + st + j * p.dim);
#pragma unroll
                    for (int v = 0; v < kV; ++v) add[v] = to_f32(l.v[v]);
                }
#pragma unroll
                for (int v = 0; v < kV; ++v) r.v[v] = from_f32<S>(g[v] + add[v]);
                if (s >= 0) cols.store(dx + s * p.sd_r, r);
                else if (p.dstate) cols.store(static_cast<S*>(p.dstate) + st + (s + W - 1) * p.dim, r);
            };
            // kAhead steps from i0 on. KIND: kAny, or the first, a middle or the last turn of a run without a reset whose
            // steps, and those behind them, are all there: no test between the steps (8 x 2048 x 1537 bf16, forward and
            // backward: 147 us with the tests, 121).
            auto turn = [&](int i0, Age& age, auto cut, auto kind) __attribute__((always_inline)) {
                constexpr bool CUT = decltype(cut)::value;
                constexpr int KIND = decltype(kind)::value;
                P now[kAhead], g[kAhead];
#pragma unroll
                for (int i = 0; i < kAhead; ++i) now[i] = nx[i], g[i] = ng[i];
                if constexpr (KIND == kAny) {
                    if (i0 + kAhead < steps) fetch(i0 + kAhead);
                } else if constexpr (KIND != kLast) {
                    const S* px = x + (t0 + i0 + kAhead) * p.sx_r;
                    const S* pg = dy + (t0 + i0 + kAhead) * p.sg_r;
#pragma unroll
                    for (int i = 0; i < kAhead; ++i, px += p.sx_r, pg += p.sg_r) {
                        nx[i] = cols.load(px);
                        if constexpr (!STEPS_OUT) ng[i] = cols.load(pg);
                    }
                }
                Line line[kV][kAhead / Q];
                if constexpr (STEPS_OUT) {
#pragma unroll
                    for (int v = 0; v < kV; ++v)
#pragma unroll
                        for (int h = 0; h < kAhead / Q; ++h)
                            line[v][h] = tile[(pair * kV + v) * SLOTS + ((wave * QPI + i0 / Q + h) ^ (pair & (SLOTS - 1)))];
                }
                S* pd = dx + (t0 + i0 - (W - 1)) * p.sd_r;
#pragma unroll
                for (int i = 0; i < kAhead; ++i, pd += p.sd_r) {
                    if constexpr (CUT) age.next();
                    const bool in = KIND != kAny || i0 + i < steps;
                    const bool own = KIND == kAny ? i0 + i < most : KIND != kLast || i < kAhead - (W - 1);
#pragma unroll
                    for (int v = 0; v < kV; ++v) {
#pragma unroll
                        for (int j = W - 1; j > 0; --j) {
                            seen[j][v] = !CUT || j <= age.age ? seen[j - 1][v] : 0.0f;
                            dv[j][v] = dv[j - 1][v];
                        }
                        seen[0][v] = to_f32(now[i].v[v]);
                        dv[0][v] = 0.0f;
                        float pre = b[v];
#pragma unroll
                        for (int j = W - 1; j >= 0; --j) pre = __builtin_fmaf(w[v][W - 1 - j], seen[j][v], pre);
                        float gv;
                        if constexpr (STEPS_OUT) gv = to_f32(line[v][i / Q].v[i % Q]);
                        else gv = to_f32(g[i].v[v]);
                        const float d = in ? gv * dact_f(pre, p.silu) : 0.0f;
#pragma unroll
                        for (int j = 0; j < W; ++j)
                            dv[j][v] = __builtin_fmaf(w[v][W - 1 - j], !CUT || j <= age.age ? d : 0.0f, dv[j][v]);
                        if (own) {
                            db[v] += d;
#pragma unroll
                            for (int j = 0; j < W; ++j) dw[v][W - 1 - j] = __builtin_fmaf(d, seen[j][v], dw[v][W - 1 - j]);
                        }
                    }
                    const int s = i0 + i - (W - 1);
                    if (KIND == kAny || (KIND == kFirst && i < W - 1)) {
                        if (s < most && (s >= 0 || t0 == 0)) emit(t0 + s, dv[W - 1]);
                    } else {
                        P r;
#pragma unroll
                        for (int v = 0; v < kV; ++v) r.v[v] = from_f32<S>(dv[W - 1][v]);
                        cols.store(pd, r);
                    }
                }
            };
            Age age(mask);
            if (mask == 0 && steps == kRowRun) {
                turn(0, age, std::false_type{}, std::integral_constant<int, kFirst>{});
                for (int i0 = kAhead; i0 < kRowRun - kAhead; i0 += kAhead) turn(i0, age, std::false_type{}, std::integral_constant<int, kMiddle>{});
                turn(kRowRun - kAhead, age, std::false_type{}, std::integral_constant<int, kLast>{});
            } else {
                // (the W - 1 steps behind the last one finish the gradients that wait)
                for (int i0 = 0; i0 < most + W - 1; i0 += kAhead) turn(i0, age, std::true_type{}, std::integral_constant<int, kAny>{});
            }
        }
        if constexpr (STEPS_OUT) __syncthreads();
    }
    // the waves' sums of a channel, in their order
    float* sums = reinterpret_cast<float*>(lds);  // (kWaves, W + 1, kCols)
#pragma unroll
    for (int v = 0; v < kV; ++v) {
#pragma unroll
        for (int k = 0; k < W; ++k) sums[(wave * (W + 1) + k) * kCols + lane * kV + v] = dw[v][k];
        sums[(wave * (W + 1) + W) * kCols + lane * kV + v] = db[v];
    }
    __syncthreads();
    for (int k = threadIdx.x; k < kCols * (W + 1); k += 64 * kWaves) {
        const int64_t c = (int64_t)group * kCols + k % kCols;
        if (c >= p.dim) continue;
        float s = 0.0f;
#pragma unroll
        for (int q = 0; q < kWaves; ++q) s += sums[q * kCols * (W + 1) + k];
        p.part[((int64_t)block * (W + 1) + k / kCols) * p.dim + c] = s;
    }
}

// ---- steps side by side ----

// n / d for n below 2^31, by the product with a rounded-up 2^(31 + s) / d, s = ceil(log2 d): m = (2^(31 + s) + e) / d
// with e < d <= 2^s adds less than 1 / d to the quotient, which the floor drops.
struct Div {
    uint32_t d, m, s;
    explicit Div(int64_t by) : d((uint32_t)by), m(0), s(0) {
        while (((int64_t)1 << s) < by) ++s;
        if (s) m = (uint32_t)((((uint64_t)1 << (31 + s)) + d - 1) / d);
    }
    __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return s ? __umulhi(n, m) >> (s - 1) : n; }
};

// A whole run in one access, without a test of its own where every lane of the wave has one.
template <typename S>
__device__ __forceinline__ Pack<S, kRun> load_run(const S* p, int n, bool whole) {
    Pack<S, kRun> r;
    if (whole) __builtin_memcpy(&r, p, sizeof(r));
    else r = load_some<S, kRun>(p, n);
    return r;
}

// SMALL: fewer than 2^31 runs in all.
template <typename S, int W, bool SMALL>
__global__ __launch_bounds__(kConvThreads) void conv_steps_fwd_kernel(ConvArgs p, int64_t total, Div by_runs, Div by_dim) {
    const int64_t id = grid_block() * kConvThreads + threadIdx.x;
    if (id >= total) return;
    const int len = (int)p.len;
    // rows (batch, channel) one after another, each of `runs` runs
    const int64_t row = SMALL ? by_runs((uint32_t)id) : id / p.runs;
    const int t0 = (int)(id - row * p.runs) * kRun;
    const int64_t bt = SMALL ? by_dim((uint32_t)row) : row / p.dim, c = row - bt * p.dim;
    const S* x = static_cast<const S*>(p.x) + bt * p.sx_b + c * p.sx_r;
    const uint8_t* reset = p.reset ? p.reset + bt * p.len : nullptr;
    const bool whole = __ballot(t0 + kRun > len) == 0;
    const Pack<S, kRun> now = load_run<S>(x + t0, len - t0, whole);
    const Pack<S, 4> before = load_some<S, 4>(x + t0 - 4, t0 > 0 ? 4 : 0);
    const uint32_t bits = reset_bits(reset, t0, len);
    float w[W];
#pragma unroll
    for (int k = 0; k < W; ++k) w[k] = p.w[c * W + k];
    const float b = p.b ? p.b[c] : 0.0f;
    float in[4 + kRun];  // steps t0 - 4 ..
#pragma unroll
    for (int i = 0; i < 4; ++i) in[i] = to_f32(before.v[i]);
#pragma unroll
    for (int i = 0; i < kRun; ++i) in[4 + i] = to_f32(now.v[i]);
    const int64_t st = bt * (W - 1) * p.dim + c;
    if (t0 == 0 && p.state) {
#pragma unroll
        for (int i = 0; i < W - 1; ++i) in[4 - (W - 1) + i] = to_f32(static_cast<const S*>(p.state)[st + i * p.dim]);
    }
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
    Pack<S, kRun> out;
    auto run = [&](auto cut) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            const int age = age_of(bits, 8 + i);
            float pre = b;
#pragma unroll
            for (int j = W - 1; j >= 0; --j)
                pre = __builtin_fmaf(w[W - 1 - j], !decltype(cut)::value || j <= age ? in[4 + i - j] : 0.0f, pre);
            out.v[i] = from_f32<S>(act_f(pre, p.silu));
        }
    };
    if (__ballot(bits != 0) == 0) run(std::false_type{});
    else run(std::true_type{});
    S* y = static_cast<S*>(p.y) + bt * p.sy_b + c * p.sy_r + t0;
    if (whole) __builtin_memcpy(y, &out, sizeof(out));
    else store_some<S, kRun>(y, out, len - t0);
}

// A workgroup: one channel, every `blocks`-th stretch of its sequences' runs. A wave takes 63 runs and the one behind
// them, whose dpre the last of them needs as each needs its neighbour's: a lane reads it from the next lane instead
// of computing it again (8 x 2048 x 1536 bf16: 70 us, 90 with 11 steps computed for 8 and a load before each use).
constexpr int kOwn = 63;

template <typename S, int W>
__global__ __launch_bounds__(kConvThreads) void conv_steps_bwd_kernel(ConvBwdArgs p) {
    const int64_t c = blockIdx.x / p.blocks;
    const int block = blockIdx.x % p.blocks, lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int len = (int)p.len;
    float w[W], dw[W], db = 0.0f;
#pragma unroll
    for (int k = 0; k < W; ++k) w[k] = p.w[c * W + k], dw[k] = 0.0f;
    const float b = p.b ? p.b[c] : 0.0f;

    struct Run {
        Pack<S, 4> before;
        Pack<S, kRun> x, g;
        uint32_t bits;
    };
    // The item's batch and run, and how far both go from turn to turn.
    const uint32_t stride = (uint32_t)p.blocks * (kConvThreads / 64) * kOwn;
    const uint32_t bt_by = stride / p.runs, run_by = stride - bt_by * p.runs;
    uint32_t item = ((uint32_t)block * (kConvThreads / 64) + wave) * kOwn + lane;
    uint32_t nbt = item / p.runs, nrun = item - nbt * p.runs;
    auto fetch = [&](uint32_t it, uint32_t bt, uint32_t rn) __attribute__((always_inline)) {
        Run r;
        const bool in = it < p.items;
        if (__ballot(in) == 0) return Run{};
        if (!in) bt = 0, rn = 0;  // (reads what is there, its gradient as zeros)
        const int t0 = (int)rn * kRun;
        const bool whole = __ballot(t0 + kRun > len) == 0;
        const S* x = static_cast<const S*>(p.x) + bt * p.sx_b + c * p.sx_r + t0;
        const S* g = static_cast<const S*>(p.dy) + bt * p.sg_b + c * p.sg_r + t0;
        r.before = load_some<S, 4>(x - 4, t0 > 0 ? 4 : 0);
        r.x = load_run<S>(x, len - t0, whole);
        r.g = load_run<S>(g, len - t0, whole);
        if (!in) r.g = Pack<S, kRun>{};
        r.bits = reset_bits(p.reset ? p.reset + bt * p.len : nullptr, t0, len);
        return r;
    };
    Run next = fetch(item, nbt, nrun);
    // (a whole wave makes the same turns: lanes read their neighbours')
    for (uint32_t first = item - lane; first < p.items; first += stride, item += stride) {
        const Run now = next;
        const bool in = item < p.items, own = in && lane < kOwn;
        const uint32_t bt = in ? nbt : 0;
        const int t0 = in ? (int)nrun * kRun : len;
        nbt += bt_by, nrun += run_by;
        if (nrun >= p.runs) nrun -= p.runs, ++nbt;
        next = fetch(item + stride, nbt, nrun);
        const bool whole = __ballot(in && t0 + kRun > len) == 0;
        float v[4 + kRun];  // values of steps t0 - 4 ..
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = to_f32(now.before.v[i]);
#pragma unroll
        for (int i = 0; i < kRun; ++i) v[4 + i] = to_f32(now.x.v[i]);
        const int64_t st = (int64_t)bt * (W - 1) * p.dim + c;
        if (t0 == 0 && p.state) {
#pragma unroll
            for (int i = 0; i < W - 1; ++i) v[4 - (W - 1) + i] = to_f32(static_cast<const S*>(p.state)[st + i * p.dim]);
        }
        float dv[W - 1 + kRun];
#pragma unroll
        for (int i = 0; i < W - 1 + kRun; ++i) dv[i] = 0.0f;
        const uint8_t* reset = p.reset ? p.reset + bt * p.len : nullptr;
        if (own && p.dlast && t0 + kRun + W - 1 > len) {
#pragma unroll
            for (int i = 0; i < W - 1 + kRun; ++i) {
                const int s = t0 + i - (W - 1), j = s - (len - (W - 1));
                if (j < 0 || j >= W - 1 || (t0 > 0 && i < W - 1) || !left_alive<W>(reset, len, j)) continue;
                dv[i] = to_f32(static_cast<const S*>(p.dlast)[st + j * p.dim]);
            }
        }
        auto run = [&](auto cut, auto inside) __attribute__((always_inline)) {
            constexpr bool CUT = decltype(cut)::value, INSIDE = decltype(inside)::value;
            float d[kRun + W - 1];
#pragma unroll
            for (int i = 0; i < kRun; ++i) {
                const int age = age_of(now.bits, 8 + i);
                float pre = b, seen[W];
#pragma unroll
                for (int j = W - 1; j >= 0; --j) {
                    seen[j] = !CUT || j <= age ? v[4 + i - j] : 0.0f;
                    pre = __builtin_fmaf(w[W - 1 - j], seen[j], pre);
                }
                d[i] = INSIDE || t0 + i < len ? to_f32(now.g.v[i]) * dact_f(pre, p.silu) : 0.0f;
                db += d[i];
#pragma unroll
                for (int j = 0; j < W; ++j) dw[W - 1 - j] = __builtin_fmaf(d[i], seen[j], dw[W - 1 - j]);
            }
#pragma unroll
            for (int i = 0; i < W - 1; ++i) {
                const float behind = __shfl_down(d[i], 1);
                d[kRun + i] = t0 + kRun + i < len ? behind : 0.0f;  // behind a sequence the next lane has another
            }
#pragma unroll
            for (int i = 0; i < kRun + W - 1; ++i) {
                const int age = age_of(now.bits, 8 + i);
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    const int to = W - 1 + i - j;
                    if (to < W - 1 + kRun) dv[to] = __builtin_fmaf(w[W - 1 - j], !CUT || j <= age ? d[i] : 0.0f, dv[to]);
                }
            }
        };
        if (whole && __ballot(now.bits != 0) == 0) run(std::false_type{}, std::true_type{});
        else run(std::true_type{}, std::false_type{});
        if (!own) continue;
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
#pragma unroll
    for (int k = 0; k <= W; ++k) {
        const float s = wave_sum(lane < kOwn ? k < W ? dw[k < W ? k : 0] : db : 0.0f);
        if (lane == 0) sums[wave][k] = s;
    }
    __syncthreads();
    if (threadIdx.x <= W) {
        float s = 0.0f;
#pragma unroll
        for (int q = 0; q < kConvThreads / 64; ++q) s += sums[q][threadIdx.x];
        p.part[((int64_t)block * (W + 1) + threadIdx.x) * p.dim + c] = s;
    }
}

// The workgroups' partial sums, added in order: 32 columns x 8 stretches of the list a workgroup.
__global__ __launch_bounds__(256) void conv_join_kernel(const float* part, int blocks, int width, int64_t dim, float* dw, float* db) {
    __shared__ float lds[8][32];
    const int64_t wide = dim * (width + 1), k = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);
    const int g = threadIdx.x >> 5, per = (blocks + 7) / 8;
    float s = 0.0f;
    if (k < wide) s = column_sum(part, wide, k, g * per, (g + 1) * per < blocks ? (g + 1) * per : blocks);
    lds[g][threadIdx.x & 31] = s;
    __syncthreads();
    if (g != 0 || k >= wide) return;
#pragma unroll
    for (int q = 1; q < 8; ++q) s += lds[q][threadIdx.x & 31];
    const int64_t tap = k / dim, c = k - tap * dim;
    if (tap < width) dw[c * width + tap] = s;
    else if (db) db[c] = s;
}

int64_t groups_of(const mamba_conv_shape& s) { return (s.dim + kCols - 1) / kCols; }

// Runs of a sequence, one at least: of kRun steps where steps lie side by side, of a wave's where channels do.
uint32_t runs_of(const mamba_conv_shape& s, bool x_steps, bool bwd) {
    const int64_t run = x_steps ? kRun : bwd ? kRowRun - (s.width - 1) : kRowRun;
    return s.len > 0 ? (uint32_t)((s.len + run - 1) / run) : 1;
}

// Workgroups a group of channels (or a channel): as many as the GPU holds at a time, each to take several
// stretches of runs with the weights it has loaded.
int blocks_of(int64_t items, int64_t each, int64_t groups, int per_cu) {
    const int64_t need = (items + each - 1) / each, most = (int64_t)layers_cus() * per_cu / groups;
    const int64_t n = need < most ? need : most;
    return (int)(n < 1 ? 1 : n);
}
// (rows, gradient: 66.2 us a pass at 8 x 2048 x 1536 with 4 a CU, 67.8 with 8; steps,
// forward and gradient: 92.8 with 12, 96.7 with 32, 118 with 48)
constexpr int kFwdPerCu = 8, kBwdPerCu = 4, kStepsBwdPerCu = 12;

int bwd_blocks(const mamba_conv_shape& s, bool x_steps) {
    const int64_t items = s.batch * runs_of(s, x_steps, true);
    return x_steps ? blocks_of(items, kConvThreads / 64 * kOwn, s.dim, kStepsBwdPerCu) : blocks_of(items, kWaves, groups_of(s), kBwdPerCu);
}

template <typename S, int W>
void fwd_go(ConvArgs q, bool x_steps, bool y_steps, int64_t groups, Launches& on) {
    if (x_steps) {
        const int64_t total = q.batch * q.dim * q.runs;
        const dim3 grid = grid_of((total + kConvThreads - 1) / kConvThreads, kConvThreads);
        if (total < (int64_t)1 << 31) on(conv_steps_fwd_kernel<S, W, true>, grid, dim3(kConvThreads), q, total, Div(q.runs), Div(q.dim));
        else on(conv_steps_fwd_kernel<S, W, false>, grid, dim3(kConvThreads), q, total, Div(1), Div(1));
        return;
    }
    q.blocks = blocks_of(q.items, kWaves, groups, kFwdPerCu);
    const dim3 grid((unsigned)(groups * q.blocks));
    const dim3 block(64 * kWaves);
    if (q.dim % 2 == 0) {
        if (y_steps) on(conv_rows_fwd_kernel<S, W, true, true>, grid, block, q);
        else on(conv_rows_fwd_kernel<S, W, false, true>, grid, block, q);
    } else {
        if (y_steps) on(conv_rows_fwd_kernel<S, W, true, false>, grid, block, q);
        else on(conv_rows_fwd_kernel<S, W, false, false>, grid, block, q);
    }
}

template <typename S, int W>
void bwd_go(const ConvBwdArgs& q, bool x_steps, bool g_steps, int64_t groups, Launches& on) {
    if (x_steps) {
        on(conv_steps_bwd_kernel<S, W>, dim3((unsigned)(q.dim * q.blocks)), dim3(kConvThreads), q);
        return;
    }
    const dim3 grid((unsigned)(groups * q.blocks));
    const dim3 block(64 * kWaves);
    if (q.dim % 2 == 0) {
        if (g_steps) on(conv_rows_bwd_kernel<S, W, true, true>, grid, block, q);
        else on(conv_rows_bwd_kernel<S, W, false, true>, grid, block, q);
    } else {
        if (g_steps) on(conv_rows_bwd_kernel<S, W, true, false>, grid, block, q);
        else on(conv_rows_bwd_kernel<S, W, false, false>, grid, block, q);
    }
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
    const uint32_t runs = runs_of(s, p.x_steps, false);
    ConvArgs q{p.x, p.weight, p.bias, p.initial_state, p.reset, p.y, p.last_state, p.x_batch, p.x_row, p.y_batch, p.y_row,
               s.batch, s.len, s.dim, runs, (uint32_t)(s.batch * runs), 1, act == MAMBA_CONV_SILU};
    Launches on(stream);
    with_width(s.width, [&](auto w) {
        constexpr int W = decltype(w)::value;
        bf16 ? fwd_go<bf16_t, W>(q, p.x_steps, p.y_steps, groups_of(s), on) : fwd_go<float, W>(q, p.x_steps, p.y_steps, groups_of(s), on);
    });
    return on.status;
}

int64_t conv_bwd_workspace(const mamba_conv_shape& s, bool x_steps) {
    return align256((int64_t)bwd_blocks(s, x_steps) * (s.width + 1) * s.dim * 4);
}

int launch_conv_bwd(const mamba_conv_bwd_ptrs& p, const mamba_conv_shape& s, int act, bool bf16, hipStream_t stream) {
    const uint32_t runs = runs_of(s, p.x_steps, true);
    ConvBwdArgs q{p.x, p.weight, p.bias, p.initial_state, p.reset, p.dy, p.dlast_state, p.dx, p.dinitial_state,
                  static_cast<float*>(p.workspace), p.x_batch, p.x_row, p.dy_batch, p.dy_row, p.dx_batch, p.dx_row,
                  s.batch, s.len, s.dim, runs, (uint32_t)(s.batch * runs), bwd_blocks(s, p.x_steps),
                  act == MAMBA_CONV_SILU};
    Launches on(stream);
    with_width(s.width, [&](auto w) {
        constexpr int W = decltype(w)::value;
        bf16 ? bwd_go<bf16_t, W>(q, p.x_steps, p.dy_steps, groups_of(s), on) : bwd_go<float, W>(q, p.x_steps, p.dy_steps, groups_of(s), on);
    });
    on(conv_join_kernel, dim3((unsigned)((s.dim * (s.width + 1) + 31) / 32)), dim3(256), static_cast<const float*>(p.workspace),
       q.blocks, (int)s.width, s.dim, p.dweight, p.dbias);
    return on.status;
}

}  // namespace mscan
