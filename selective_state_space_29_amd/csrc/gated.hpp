// The gated linear recurrence (mamba_layers.h) on gfx950, forward and backward.
//
//   e_t = c log2(e) softplus(lam) sigmoid(r_t)   (= -log2 a_t)      a_t = 2^-e_t
//   h_t = a_t h_{t-1} + b_t,   b_t = m_t sigmoid(i_t) x_t,   m_t = sqrt(1 - a_t^2)
//
// One lane owns one channel and a run of TS consecutive steps. A workgroup owns CH consecutive
// channels of one batch and walks the sequence in chunks: its CH / 4 waves, of 64 / CH sub-runs each,
// hold 16 consecutive runs, so a chunk is 16 TS steps read as rows of CH contiguous channels. Each lane
// scans its run from a zero state and writes the run's pair (product of a, end state) to LDS; there the
// 16 pairs of a channel are scanned by the 16 lanes of one DPP row (every thread has one pair to scan:
// 16 CH pairs, 16 CH threads), which also carries the channel's state from chunk to chunk; each lane
// takes back the state entering its run, and one FMA a step gives the states. Every input is read once,
// so nothing but the inputs and outputs passes through HBM. (The alternative, one pass for the pairs of
// all chunks and a second for the states, reads the inputs and computes the gates twice.)
//
// Few rows: the sequence is split into segments, one workgroup each, and a pre-pass over all but the
// last writes the segments' pairs; a workgroup folds those of the segments before its own, in order.
#pragma once

#include <type_traits>

#include "layers_common.hpp"

namespace mscan {

struct GatedParams {
    const void* x;
    const void* r;
    const void* i;
    const float* lam;
    const float* h0;
    const uint8_t* reset;
    void* y;
    float* last;
    float* ck;
    float2* agg;        // (batch, nseg, dim): the segments' pairs
    int64_t batch, len, dim, nck;
    int64_t sx_b, sx_t, sr_b, sr_t, si_b, si_t, sy_b, sy_t;
    int64_t seg_len;    // steps per segment, a multiple of the chunk and of MAMBA_GATED_CHECKPOINT
    int nseg;
    float c;
};

struct GatedBwdParams {
    const void* x;
    const void* r;
    const void* i;
    const float* lam;
    const float* h0;
    const uint8_t* reset;
    const void* dy;
    const float* dlast;
    const float* ck;
    void* dx;
    void* dr;
    void* di;
    float* dh0;
    float* part;        // (batch * nseg, dim): sums of q
    float2* agg;        // (batch, nseg, dim): the segments' adjoint pairs
    int64_t batch, len, dim, nck;
    int64_t sx_b, sx_t, sr_b, sr_t, si_b, si_t, sdy_b, sdy_t, sdx_b, sdx_t, sdr_b, sdr_t, sdi_b, sdi_t;
    int64_t seg_len;
    int nseg;
    float c;
};

constexpr int kGatedCk = MAMBA_GATED_CHECKPOINT;

__device__ __forceinline__ float sigmoid_f(float v) { return hw_rcp(1.0f + hw_exp2(-v * kLog2e)); }

// 1 - a^2 = 1 - e^-v at v = 2 ln(2) e, given a. Below v = 1/4 the series
// v (1 - v/2 + v^2/6 - v^3/24 + v^4/120 - v^5/720), coefficients scaled to e (truncation below 2^-24
// relative); above, 1 - a^2 in one rounding, whose cancellation costs at most 3.6 times a's own error.
__device__ __forceinline__ float one_minus_sq(float e, float a) {
    constexpr float k = 1.3862943611198906f;  // 2 ln 2
    constexpr float c1 = k, c2 = -k * k / 2, c3 = k * k * k / 6, c4 = -k * k * k * k / 24,
                    c5 = k * k * k * k * k / 120, c6 = -k * k * k * k * k * k / 720;
    float q = __builtin_fmaf(e, c6, c5);
    q = __builtin_fmaf(e, q, c4);
    q = __builtin_fmaf(e, q, c3);
    q = __builtin_fmaf(e, q, c2);
    q = __builtin_fmaf(e, q, c1);
    const float big = __builtin_fmaf(-a, a, 1.0f);
    return e < 0.25f / k ? e * q : big;
}

// a h + b of the recurrence and of its folds. A reset's decay is exactly 0 and has to forget a state
// that is infinite or NaN too: with resets the product is the one in which 0 times anything is 0, and
// every other decay is kept above 0 (kMinDecay), so that only a reset forgets such a state.
// v_mul_legacy_f32: 0 times anything is 0
__device__ float mul_legacy(float, float) __asm("llvm.amdgcn.fmul.legacy");
constexpr float kMinDecay = 1.1754944e-38f;
template <bool RESET>
__device__ __forceinline__ float decay_fma(float a, float h, float b) {
    if constexpr (RESET) return mul_legacy(a, h) + b;
    return __builtin_fmaf(a, h, b);
}
template <bool RESET>
__device__ __forceinline__ float decay_mul(float a, float v) {
    if constexpr (RESET) return mul_legacy(a, v);
    return a * v;
}
template <bool RESET>
__device__ __forceinline__ float pair_product(float a, float b) {
    if constexpr (RESET) return a > 0.0f && b > 0.0f ? __builtin_fmaxf(a * b, kMinDecay) : 0.0f;
    return a * b;
}
// The decay of a run, 2^-e, and of a step: `on` is whether the step is a reset.
template <bool RESET>
__device__ __forceinline__ float decay_of(float e) {
    const float a = hw_exp2(-e);
    if constexpr (RESET) return e < __builtin_inff() ? __builtin_fmaxf(a, kMinDecay) : 0.0f;
    return a;
}
template <bool RESET>
__device__ __forceinline__ float decay_step(float& e, bool on) {
    if constexpr (RESET) {
        e = __builtin_fmaxf(e, on ? __builtin_inff() : 0.0f);
        return __builtin_fmaxf(hw_exp2(-e), on ? 0.0f : kMinDecay);
    }
    return hw_exp2(-e);
}

// Which (channel group, batch, segment) a workgroup works on. Workgroups go to the 8 XCDs in turn;
// groups of channels narrower than a 128-byte line are dealt so that the `share` groups of one line
// run on the same XCD, whose L2 then fetches the line once.
struct GatedPlace {
    int64_t group, b, seg;
    bool ok;
};
__device__ __forceinline__ GatedPlace gated_place(int64_t groups, int64_t batch, int nseg, int share) {
    const int64_t id = blockIdx.x, slot = id >> 3;
    const int64_t lin = ((slot / share) * 8 + (id & 7)) * share + slot % share;
    GatedPlace p;
    p.group = lin % groups;
    const int64_t rest = lin / groups;
    p.b = rest % batch;
    p.seg = rest / batch;
    p.ok = p.seg < nseg;
    return p;
}
inline int64_t gated_blocks(int64_t groups, int64_t batch, int nseg, int share) {
    const int64_t n = groups * batch * nseg, q = 8 * share;
    return (n + q - 1) / q * q;
}

// Rows of a chunk are addressed through a buffer descriptor at the wave's first row: the lane's offset
// (its sub-run's first row and its channel) in a register, the row within the run in a scalar. A lane
// without a row or channel uses an offset past the buffer, which reads 0 and drops stores, so neither
// needs a branch.
constexpr uint32_t kGatedDrop = 0xFFFFFFF0u;
template <typename P>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t gated_rsrc(P* base) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<std::remove_const_t<P>*>(base), 0, 0x7FFFFFF0, 0x00020000);
}
__device__ __forceinline__ void row_load(bf16_t& v, __amdgpu_buffer_rsrc_t r, uint32_t off, int row) {
    v.bits = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, (int)off, row, 0);
}
__device__ __forceinline__ void row_load(float& v, __amdgpu_buffer_rsrc_t r, uint32_t off, int row) {
    v = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, (int)off, row, 0));
}
__device__ __forceinline__ void row_store(bf16_t v, __amdgpu_buffer_rsrc_t r, uint32_t off, int row) {
    __builtin_amdgcn_raw_buffer_store_b16((short)v.bits, r, (int)off, row, 0);
}
__device__ __forceinline__ void row_store(float v, __amdgpu_buffer_rsrc_t r, uint32_t off, int row) {
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, (int)off, row, 0);
}

// One sequence tensor of a batch as a lane sees it.
template <typename S>
struct Seq {
    S* base;        // of the batch
    int64_t st;     // elements between steps
    uint32_t off;   // the lane's offset in the wave's rows, bytes
    __device__ __forceinline__ Seq(S* p, int64_t st_, int lane_row, int64_t d)
        : base(p), st(st_), off((uint32_t)(lane_row * (int)st_ + (int)d) * (uint32_t)sizeof(S)) {}
    __device__ __forceinline__ int row_bytes() const { return (int)st * (int)sizeof(S); }
};

template <typename S, int TS, bool FULL>
__device__ __forceinline__ void gated_rows(S (&v)[TS], const Seq<const S>& q, int64_t t_wave, int left) {
    const __amdgpu_buffer_rsrc_t r = gated_rsrc(q.base + t_wave * q.st);
#pragma unroll
    for (int k = 0; k < TS; ++k) row_load(v[k], r, FULL || k < left ? q.off : kGatedDrop, k * q.row_bytes());
}

// The reset bytes of a wave's R * TS steps as one bit each.
template <int N>
__device__ __forceinline__ uint64_t gated_reset_bits(const uint8_t* reset, int64_t t_wave, int64_t len, int lane) {
    const int64_t t = t_wave + lane;
    const bool on = lane < N && t < len && reset[t < len ? t : len - 1] != 0;
    return __ballot(on);
}

// Scans of the 16 lanes of a DPP row, one run's pair a lane (mul, add): the composition of the runs up to
// and including the lane's, in run order (UP) or from the last run down.
template <int CTRL>
__device__ __forceinline__ float dpp_from(float v, float otherwise) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, otherwise), __builtin_bit_cast(int, v),
                                                                 CTRL, 0xf, 0xf, false));
}
constexpr int kRowShl = 0x100, kRowShr = 0x110, kRowBcast = 0x150;
template <bool UP, bool RESET>
__device__ __forceinline__ void row_scan(float& a, float& h) {
    constexpr int shift = UP ? kRowShr : kRowShl;
    auto step = [&](float pa, float ph) __attribute__((always_inline)) {
        h = decay_fma<RESET>(a, ph, h);
        a = pair_product<RESET>(a, pa);
    };
    step(dpp_from<shift + 1>(a, 1.0f), dpp_from<shift + 1>(h, 0.0f));
    step(dpp_from<shift + 2>(a, 1.0f), dpp_from<shift + 2>(h, 0.0f));
    step(dpp_from<shift + 4>(a, 1.0f), dpp_from<shift + 4>(h, 0.0f));
    step(dpp_from<shift + 8>(a, 1.0f), dpp_from<shift + 8>(h, 0.0f));
}

enum { kGatedStates = 0, kGatedPairs = 1, kGatedCkOnly = 2 };  // y and states; pairs only; checkpoints only

constexpr int kRuns = 16;  // runs of a chunk: the lanes of a DPP row

// Pitch of a run's row of CH pairs in LDS: 4 more, so that the 16 runs x 4 channels a wave scans lie in
// distinct banks.
template <int CH>
constexpr int kPitch = CH + 4;

template <typename S, int CH, int TS, bool RESET, int MODE>
__global__ __launch_bounds__(CH * 16) __attribute__((amdgpu_waves_per_eu(4))) void gated_fwd_kernel(GatedParams p) {
    constexpr int R = 64 / CH, STEPS = kRuns * TS;
    static_assert(kGatedCk % TS == 0 && R * TS <= 64);
    __shared__ float2 s_pair[kRuns * kPitch<CH>];
    __shared__ float s_in[kRuns * kPitch<CH>];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ch = lane % CH, sub = lane / CH, run = wave * R + sub;
    const int s_run = lane & 15, s_ch = wave * 4 + (lane >> 4);  // the pair this thread scans
    constexpr int share = CH * (int)sizeof(S) < 128 ? 128 / (CH * (int)sizeof(S)) : 1;
    const int64_t D = p.dim, L = p.len;
    const int nseg = MODE == kGatedPairs ? p.nseg - 1 : p.nseg;
    const GatedPlace at = gated_place((D + CH - 1) / CH, p.batch, nseg, share);
    if (!at.ok) return;
    const int64_t b = at.b, seg = at.seg;
    const int64_t d_own = at.group * CH + ch, d_scan = at.group * CH + s_ch;
    const bool live = d_own < D;
    const int64_t d = live ? d_own : D - 1, ds = d_scan < D ? d_scan : D - 1;
    const int64_t t_begin = seg * p.seg_len;
    const int64_t t_end = t_begin + p.seg_len < L ? t_begin + p.seg_len : L;

    const int rows = sub * TS;
    const Seq<const S> x(static_cast<const S*>(p.x) + b * p.sx_b, p.sx_t, rows, d);
    const Seq<const S> r(static_cast<const S*>(p.r) + b * p.sr_b, p.sr_t, rows, d);
    const Seq<const S> i(static_cast<const S*>(p.i) + b * p.si_b, p.si_t, rows, d);
    const Seq<S> y(static_cast<S*>(p.y) + b * p.sy_b, p.sy_t, rows, d);
    const uint8_t* reset = RESET ? p.reset + b * L : nullptr;
    const float tl = p.c * kLog2e * softplus_f(p.lam[d]);

    float carry = 0.0f, carry_a = 1.0f;  // the scanned channel's state (and, for pairs, its decay so far)
    if (MODE != kGatedPairs) {
        carry = p.h0 ? p.h0[b * D + ds] : 0.0f;
        for (int64_t q = 0; q < seg; ++q) {
            const float2 v = p.agg[(b * p.nseg + q) * D + ds];
            carry = decay_fma<RESET>(v.x, carry, v.y);
        }
    }

    S nx[TS], nr[TS], ni[TS];
    uint64_t nbits = 0;
    auto fetch_as = [&](int64_t t0, auto full) __attribute__((always_inline)) {
        constexpr bool FULL = decltype(full)::value;
        const int64_t tw = t0 + wave * R * TS;
        const int left = (int)(t_end - tw - rows < TS ? t_end - tw - rows : TS);
        gated_rows<S, TS, FULL>(nr, r, tw, left);
        gated_rows<S, TS, FULL>(ni, i, tw, left);
        gated_rows<S, TS, FULL>(nx, x, tw, left);
        if (RESET) nbits = gated_reset_bits<R * TS>(reset, tw, L, lane);
    };
    auto fetch = [&](int64_t t0) __attribute__((always_inline)) {
        if (t0 + STEPS <= t_end) fetch_as(t0, std::true_type{});
        else fetch_as(t0, std::false_type{});
    };
    fetch(t_begin);
    auto chunk = [&](int64_t t0, auto tail) __attribute__((always_inline)) {
        constexpr bool TAIL = decltype(tail)::value;
        S cx[TS], cr[TS], ci[TS];
#pragma unroll
        for (int k = 0; k < TS; ++k) cx[k] = nx[k], cr[k] = nr[k], ci[k] = ni[k];
        const uint64_t bits = RESET ? nbits >> (sub * TS) : 0;
        if (t0 + STEPS < t_end) fetch(t0 + STEPS);
        const int64_t t_run = t0 + (int64_t)run * TS;
        const int left = (int)(t_end - t_run < TS ? t_end - t_run : TS);  // steps of this run that exist

        float a[TS], bb[TS], esum = 0.0f, h = 0.0f;
#pragma unroll
        for (int k = 0; k < TS; ++k) {
            float e = tl * sigmoid_f(to_f32(cr[k]));
            a[k] = decay_step<RESET>(e, (bits >> k) & 1);
            const float m = __builtin_amdgcn_sqrtf(one_minus_sq(e, a[k]));
            bb[k] = m * (sigmoid_f(to_f32(ci[k])) * to_f32(cx[k]));
            if constexpr (TAIL) {  // past the end the state is carried
                if (k >= left) {
                    a[k] = 1.0f;
                    bb[k] = e = 0.0f;
                }
            }
            esum += e;
            h = decay_fma<RESET>(a[k], h, bb[k]);
        }
        s_pair[run * kPitch<CH> + ch] = make_float2(decay_of<RESET>(esum), h);
        __syncthreads();
        float2 v = s_pair[s_run * kPitch<CH> + s_ch];
        row_scan<true, RESET>(v.x, v.y);
        const float after = decay_fma<RESET>(v.x, carry, v.y);
        s_in[s_run * kPitch<CH> + s_ch] = dpp_from<kRowShr + 1>(after, carry);
        carry = dpp_from<kRowBcast + 15>(after, 0.0f);
        if (MODE == kGatedPairs) carry_a = pair_product<RESET>(carry_a, dpp_from<kRowBcast + 15>(v.x, 0.0f));
        __syncthreads();
        float in = s_in[run * kPitch<CH> + ch];
        if (MODE != kGatedPairs) {
            if (p.ck && live && t_run % kGatedCk == 0 && left > 0) p.ck[(b * p.nck + t_run / kGatedCk) * D + d] = in;
        }
        if (MODE == kGatedStates) {
            const __amdgpu_buffer_rsrc_t o = gated_rsrc(y.base + (t0 + wave * R * TS) * y.st);
#pragma unroll
            for (int k = 0; k < TS; ++k) {
                in = decay_fma<RESET>(a[k], in, bb[k]);
                row_store(from_f32<S>(in), o, live && (!TAIL || k < left) ? y.off : kGatedDrop, k * y.row_bytes());
            }
        }
    };
    int64_t t0 = t_begin;
    for (; t0 + STEPS <= t_end; t0 += STEPS) chunk(t0, std::false_type{});
    if (t0 < t_end) chunk(t0, std::true_type{});
    if (s_run == 15 && d_scan < D) {
        if (MODE == kGatedPairs) p.agg[(b * p.nseg + seg) * D + ds] = make_float2(carry_a, carry);
        if (MODE == kGatedStates && p.last && seg == p.nseg - 1) p.last[b * D + ds] = carry;
    }
}

// Short calls (decode): one thread per channel of a batch, step after step.
template <typename S>
__global__ __launch_bounds__(256) void gated_step_kernel(GatedParams p) {
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (n >= p.batch * p.dim) return;
    const int64_t b = n / p.dim, d = n - b * p.dim;
    const S* x = static_cast<const S*>(p.x) + b * p.sx_b + d;
    const S* r = static_cast<const S*>(p.r) + b * p.sr_b + d;
    const S* i = static_cast<const S*>(p.i) + b * p.si_b + d;
    S* y = static_cast<S*>(p.y) + b * p.sy_b + d;
    float h = p.h0 ? p.h0[n] : 0.0f;
    const float tl = p.c * kLog2e * softplus_f(p.lam[d]);
    for (int64_t t = 0; t < p.len; ++t) {
        if (p.ck && t % kGatedCk == 0) p.ck[(b * p.nck + t / kGatedCk) * p.dim + d] = h;
        float e = tl * sigmoid_f(to_f32(r[t * p.sr_t]));
        if (p.reset && p.reset[b * p.len + t]) {
            e = __builtin_inff();
            h = 0.0f;
        }
        const float a = hw_exp2(-e);
        const float m = __builtin_amdgcn_sqrtf(one_minus_sq(e, a));
        h = __builtin_fmaf(a, h, m * (sigmoid_f(to_f32(i[t * p.si_t])) * to_f32(x[t * p.sx_t])));
        y[t * p.sy_t] = from_f32<S>(h);
    }
    if (p.last) p.last[n] = h;
}

// ---- backward ----
//
// The same decomposition, chunks of kGatedCk steps walked from the last to the first. A chunk's states
// come from its checkpoint by the forward's local scan and row scan; the adjoint mu_t = a_t g_t, with
// g_t = dy_t + mu_{t+1}, is the same recurrence from the right, mu_t = a_t mu_{t+1} + a_t dy_t, whose
// runs have the same product of a: one exchange serves both directions. Kept per step between the scans
// and the outputs: a, b, e, m sigmoid(i), b (1 - sigmoid(i)), (s / m) a sigmoid(i) x / s, dy.
// MODE kGatedPairs: the adjoint pairs of whole segments (all but the first), from r and dy alone.
template <typename S, int CH, int TS, bool RESET, int MODE>
__global__ __launch_bounds__(CH * 16) __attribute__((amdgpu_waves_per_eu(4))) void gated_bwd_kernel(GatedBwdParams p) {
    constexpr int R = 64 / CH, STEPS = kRuns * TS;
    constexpr bool FULL_MODE = MODE != kGatedPairs;
    static_assert(STEPS == kGatedCk && R * TS <= 64);
    __shared__ float2 s_pair[kRuns * kPitch<CH>];
    __shared__ float s_mu[kRuns * kPitch<CH>];
    __shared__ float2 s_in[kRuns * kPitch<CH>];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ch = lane % CH, sub = lane / CH, run = wave * R + sub;
    const int s_run = lane & 15, s_ch = wave * 4 + (lane >> 4);
    constexpr int share = CH * (int)sizeof(S) < 128 ? 128 / (CH * (int)sizeof(S)) : 1;
    const int64_t D = p.dim, L = p.len;
    const int nseg = MODE == kGatedPairs ? p.nseg - 1 : p.nseg;
    const GatedPlace at = gated_place((D + CH - 1) / CH, p.batch, nseg, share);
    if (!at.ok) return;
    const int64_t b = at.b, seg = MODE == kGatedPairs ? at.seg + 1 : at.seg;
    const int64_t d_own = at.group * CH + ch, d_scan = at.group * CH + s_ch;
    const bool live = d_own < D;
    const int64_t d = live ? d_own : D - 1, ds = d_scan < D ? d_scan : D - 1;
    const int64_t t_begin = seg * p.seg_len;
    const int64_t t_end = t_begin + p.seg_len < L ? t_begin + p.seg_len : L;

    const int rows = sub * TS;
    const Seq<const S> x(static_cast<const S*>(p.x) + b * p.sx_b, p.sx_t, rows, d);
    const Seq<const S> r(static_cast<const S*>(p.r) + b * p.sr_b, p.sr_t, rows, d);
    const Seq<const S> i(static_cast<const S*>(p.i) + b * p.si_b, p.si_t, rows, d);
    const Seq<const S> dy(static_cast<const S*>(p.dy) + b * p.sdy_b, p.sdy_t, rows, d);
    const Seq<S> dx(static_cast<S*>(p.dx) + b * p.sdx_b, p.sdx_t, rows, d);
    const Seq<S> dr(static_cast<S*>(p.dr) + b * p.sdr_b, p.sdr_t, rows, d);
    const Seq<S> di(static_cast<S*>(p.di) + b * p.sdi_b, p.sdi_t, rows, d);
    const uint8_t* reset = RESET ? p.reset + b * L : nullptr;
    const float tl = p.c * kLog2e * softplus_f(p.lam[d]);
    const float inv_tl = tl > 1e-30f ? hw_rcp(tl) : 0.0f;  // sigmoid(r) = e / tl; below, every q is 0

    float carry = 0.0f, carry_a = 1.0f;  // mu entering from the right, of the scanned channel
    if (FULL_MODE) {
        carry = p.dlast ? p.dlast[b * D + ds] : 0.0f;
        for (int64_t q = p.nseg - 1; q > seg; --q) {
            const float2 v = p.agg[(b * p.nseg + q) * D + ds];
            carry = decay_fma<RESET>(v.x, carry, v.y);
        }
    }
    float acc = 0.0f;

    S nx[TS], nr[TS], ni[TS], ng[TS];
    uint64_t nbits = 0;
    float nck = 0.0f;
    auto fetch_as = [&](int64_t t0, auto full) __attribute__((always_inline)) {
        constexpr bool FULL = decltype(full)::value;
        const int64_t tw = t0 + wave * R * TS;
        const int left = (int)(t_end - tw - rows < TS ? t_end - tw - rows : TS);
        gated_rows<S, TS, FULL>(nr, r, tw, left);
        gated_rows<S, TS, FULL>(ng, dy, tw, left);
        if (FULL_MODE) gated_rows<S, TS, FULL>(ni, i, tw, left);
        if (FULL_MODE) gated_rows<S, TS, FULL>(nx, x, tw, left);
        if (RESET) nbits = gated_reset_bits<R * TS>(reset, tw, L, lane);
        if (FULL_MODE) nck = p.ck[(b * p.nck + t0 / kGatedCk) * D + ds];
    };
    const int64_t t_last = t_begin + (t_end - t_begin - 1) / STEPS * STEPS;
    if (t_last + STEPS <= t_end) fetch_as(t_last, std::true_type{});
    else fetch_as(t_last, std::false_type{});
    auto chunk = [&](int64_t t0, auto tail) __attribute__((always_inline)) {
        constexpr bool TAIL = decltype(tail)::value;
        S cx[TS], cr[TS], ci[TS], cg[TS];
#pragma unroll
        for (int k = 0; k < TS; ++k) cx[k] = nx[k], cr[k] = nr[k], ci[k] = ni[k], cg[k] = ng[k];
        const uint64_t bits = RESET ? nbits >> (sub * TS) : 0;
        const float ck = nck;
        if (t0 > t_begin) fetch_as(t0 - STEPS, std::true_type{});
        const int64_t t_run = t0 + (int64_t)run * TS;
        const int left = (int)(t_end - t_run < TS ? t_end - t_run : TS);

        float e[TS], a[TS], bb[TS], ms[TS], bi[TS], z[TS], g[TS];
        float esum = 0.0f, hl = 0.0f, mu = 0.0f;
#pragma unroll
        for (int k = 0; k < TS; ++k) {
            const bool past = TAIL && k >= left;
            e[k] = tl * sigmoid_f(to_f32(cr[k]));
            a[k] = decay_step<RESET>(e[k], (bits >> k) & 1);
            g[k] = to_f32(cg[k]);
            if constexpr (TAIL) {  // past the end the state and the adjoint are carried
                if (past) a[k] = 1.0f, e[k] = g[k] = 0.0f;
            }
            esum += e[k];
            if constexpr (FULL_MODE) {
                const float w = one_minus_sq(e[k], a[k]);
                const float rm = w > 1.1754944e-38f ? __builtin_amdgcn_rsqf(w) : 0.0f;  // 1 / m, or 0 with m
                const float si = sigmoid_f(to_f32(ci[k]));
                const float gx = past ? 0.0f : si * to_f32(cx[k]);
                const float m = w * rm;
                ms[k] = m * si;
                bb[k] = m * gx;
                bi[k] = bb[k] * (1.0f - si);
                z[k] = gx * a[k] * rm;
                hl = decay_fma<RESET>(a[k], hl, bb[k]);
            }
        }
#pragma unroll
        for (int k = TS - 1; k >= 0; --k) mu = decay_mul<RESET>(a[k], g[k] + mu);
        s_pair[run * kPitch<CH> + ch] = make_float2(decay_of<RESET>(esum), hl);
        s_mu[run * kPitch<CH> + ch] = mu;
        __syncthreads();
        {
            float2 v = s_pair[s_run * kPitch<CH> + s_ch];
            float ra = v.x, rmu = s_mu[s_run * kPitch<CH> + s_ch];
            row_scan<false, RESET>(ra, rmu);
            const float after = decay_fma<RESET>(ra, carry, rmu);
            float2 o;
            o.y = dpp_from<kRowShl + 1>(after, carry);  // the adjoint entering the run from the right
            carry = dpp_from<kRowBcast + 0>(after, 0.0f);
            if (FULL_MODE) {
                row_scan<true, RESET>(v.x, v.y);
                o.x = dpp_from<kRowShr + 1>(decay_fma<RESET>(v.x, ck, v.y), ck);  // the state entering it
                s_in[s_run * kPitch<CH> + s_ch] = o;
            } else {
                carry_a = pair_product<RESET>(carry_a, dpp_from<kRowBcast + 0>(ra, 0.0f));
            }
        }
        __syncthreads();
        if (FULL_MODE) {
            const float2 o = s_in[run * kPitch<CH> + ch];
            float h = o.x, in = o.y;
#pragma unroll
            for (int k = 0; k < TS; ++k) {  // z becomes z - h before the step
                z[k] -= h;
                h = decay_fma<RESET>(a[k], h, bb[k]);
            }
            const int64_t tw = t0 + wave * R * TS;
            const __amdgpu_buffer_rsrc_t ox = gated_rsrc(dx.base + tw * dx.st), oi = gated_rsrc(di.base + tw * di.st),
                                         orr = gated_rsrc(dr.base + tw * dr.st);
#pragma unroll
            for (int k = TS - 1; k >= 0; --k) {
                const bool put = live && (!TAIL || k < left);
                const float gk = g[k] + in;
                in = decay_mul<RESET>(a[k], gk);
                const float ek = RESET ? __builtin_fminf(e[k], 1e30f) : e[k];
                const float q = decay_mul<RESET>(in * (ek * kLn2), z[k]);
                acc += !TAIL || k < left ? q : 0.0f;
                row_store(from_f32<S>(gk * ms[k]), ox, put ? dx.off : kGatedDrop, k * dx.row_bytes());
                row_store(from_f32<S>(gk * bi[k]), oi, put ? di.off : kGatedDrop, k * di.row_bytes());
                row_store(from_f32<S>(decay_mul<RESET>(q, __builtin_fmaf(-ek, inv_tl, 1.0f))), orr, put ? dr.off : kGatedDrop,
                          k * dr.row_bytes());
            }
        }
    };
    int64_t t0 = t_last;
    if (t0 + STEPS > t_end) {
        chunk(t0, std::true_type{});
        t0 -= STEPS;
    }
    for (; t0 >= t_begin; t0 -= STEPS) chunk(t0, std::false_type{});
    if (!FULL_MODE) {
        if (s_run == 0 && d_scan < D) p.agg[(b * p.nseg + seg) * D + ds] = make_float2(carry_a, carry);
        return;
    }
    if (p.dh0 && seg == 0 && s_run == 0 && d_scan < D) p.dh0[b * D + ds] = carry;
    // q summed over the runs, in run order
    s_mu[run * kPitch<CH> + ch] = acc;
    __syncthreads();
    if (wave == 0 && sub == 0 && live) {
        float sum = 0.0f;
        for (int q = 0; q < kRuns; ++q) sum += s_mu[q * kPitch<CH> + ch];
        p.part[(b * p.nseg + seg) * D + d] = sum;
    }
}

}  // namespace mscan
