// The gated linear recurrence (mamba_layers.h) on gfx950, forward and backward.
//
//   e_t = c log2(e) softplus(lam) sigmoid(r_t)   (= -log2 a_t)      a_t = 2^-e_t
//   h_t = a_t h_{t-1} + b_t,   b_t = m_t sigmoid(i_t) x_t,   m_t = sqrt(1 - a_t^2)
//
// One lane owns one channel and a run of TS consecutive steps. A workgroup owns CH consecutive
// channels of one batch and walks the sequence in chunks: W waves times R = 64 / CH sub-runs per wave
// hold W * R consecutive runs, so a chunk is W R TS steps read as rows of CH contiguous channels. Each
// lane scans its run from a zero state, writes the run's pair (product of a, end state) to LDS, and,
// after the chunk's one barrier, folds the pairs of the runs before its own into the state that enters
// its run; one FMA a step then gives the states. Every input is read once and the state is carried in
// registers from chunk to chunk, so nothing but the inputs and outputs passes through HBM. (The
// alternative, one pass for the pairs of all chunks and a second for the states, reads the inputs twice
// and computes the gates twice.)
//
// Few rows: the sequence is split into segments, one workgroup each, and a pre-pass over all but the
// last writes the segments' pairs; a workgroup folds those of the segments before its own, in order.
#pragma once

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
template <bool RESET>
__device__ __forceinline__ float decay_of(float e) {
    const float a = hw_exp2(-e);
    if constexpr (RESET) return e < __builtin_inff() ? __builtin_fmaxf(a, kMinDecay) : 0.0f;
    return a;
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

// Loads of TS rows of one lane's channel. FULL: every row of the wave exists; the row address is
// uniform over the wave and the lane's offset 32-bit. Otherwise rows past the end are read at the last
// one (and masked by the caller).
template <typename S, int TS, bool FULL>
__device__ __forceinline__ void gated_rows(S (&v)[TS], const S* base, int64_t st, int64_t t_wave, int lane_row,
                                           int64_t d, int64_t len) {
    if constexpr (FULL) {
        const S* row = base + t_wave * st;
        const uint32_t off = (uint32_t)(lane_row * (int)st + (int)d) * (uint32_t)sizeof(S);
#pragma unroll
        for (int k = 0; k < TS; ++k) v[k] = *reinterpret_cast<const S*>(reinterpret_cast<const char*>(row + k * st) + off);
    } else {
#pragma unroll
        for (int k = 0; k < TS; ++k) {
            const int64_t t = t_wave + lane_row + k;
            v[k] = base[(t < len ? t : len - 1) * st + d];
        }
    }
}

// Row k of a lane's run, at the same uniform row address and 32-bit offset.
template <typename S>
__device__ __forceinline__ void gated_store(S* base, int64_t st, int64_t t_wave, int lane_row, int k, int64_t d, float v) {
    const uint32_t off = (uint32_t)(lane_row * (int)st + (int)d) * (uint32_t)sizeof(S);
    *reinterpret_cast<S*>(reinterpret_cast<char*>(base + (t_wave + k) * st) + off) = from_f32<S>(v);
}

// The reset bytes of a wave's R * TS steps as one bit each.
template <int N>
__device__ __forceinline__ uint64_t gated_reset_bits(const uint8_t* reset, int64_t t_wave, int64_t len, int lane) {
    const int64_t t = t_wave + lane;
    const bool on = lane < N && t < len && reset[t < len ? t : len - 1] != 0;
    return __ballot(on);
}

enum { kGatedStates = 0, kGatedPairs = 1, kGatedCkOnly = 2 };  // y and states; pairs only; checkpoints only

template <typename S, int CH, int W, int TS, bool RESET, int MODE>
__global__ __launch_bounds__(W * 64) __attribute__((amdgpu_waves_per_eu(4))) void gated_fwd_kernel(GatedParams p) {
    constexpr int R = 64 / CH, RUNS = W * R, STEPS = RUNS * TS;
    static_assert(kGatedCk % TS == 0 && R * TS <= 64);
    __shared__ float2 s_pair[2][RUNS * CH];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ch = lane % CH, sub = lane / CH, run = wave * R + sub;
    constexpr int share = CH * (int)sizeof(S) < 128 ? 128 / (CH * (int)sizeof(S)) : 1;
    const int64_t D = p.dim, L = p.len;
    const int nseg = MODE == kGatedPairs ? p.nseg - 1 : p.nseg;
    const GatedPlace at = gated_place((D + CH - 1) / CH, p.batch, nseg, share);
    if (!at.ok) return;
    const int64_t b = at.b, seg = at.seg;
    const int64_t d_own = at.group * CH + ch;
    const bool live = d_own < D;
    const int64_t d = live ? d_own : D - 1;
    const int64_t t_begin = seg * p.seg_len;
    const int64_t t_end = t_begin + p.seg_len < L ? t_begin + p.seg_len : L;

    const S* x = static_cast<const S*>(p.x) + b * p.sx_b;
    const S* r = static_cast<const S*>(p.r) + b * p.sr_b;
    const S* i = static_cast<const S*>(p.i) + b * p.si_b;
    S* y = static_cast<S*>(p.y) + b * p.sy_b;
    const uint8_t* reset = RESET ? p.reset + b * L : nullptr;
    const float tl = p.c * kLog2e * softplus_f(p.lam[d]);

    float carry = 0.0f, carry_a = 1.0f;
    if (MODE != kGatedPairs) {
        carry = p.h0 ? p.h0[b * D + d] : 0.0f;
        for (int64_t q = 0; q < seg; ++q) {
            const float2 v = p.agg[(b * p.nseg + q) * D + d];
            carry = decay_fma<RESET>(v.x, carry, v.y);
        }
    }

    S nx[TS], nr[TS], ni[TS];
    uint64_t nbits = 0;
    auto fetch = [&](int64_t t0) __attribute__((always_inline)) {
        const int64_t tw = t0 + (int64_t)wave * R * TS;
        if (t0 + STEPS <= t_end) {
            gated_rows<S, TS, true>(nx, x, p.sx_t, tw, sub * TS, d, L);
            gated_rows<S, TS, true>(nr, r, p.sr_t, tw, sub * TS, d, L);
            gated_rows<S, TS, true>(ni, i, p.si_t, tw, sub * TS, d, L);
        } else {
            gated_rows<S, TS, false>(nx, x, p.sx_t, tw, sub * TS, d, L);
            gated_rows<S, TS, false>(nr, r, p.sr_t, tw, sub * TS, d, L);
            gated_rows<S, TS, false>(ni, i, p.si_t, tw, sub * TS, d, L);
        }
        if (RESET) nbits = gated_reset_bits<R * TS>(reset, tw, L, lane);
    };
    fetch(t_begin);
    int buf = 0;
    for (int64_t t0 = t_begin; t0 < t_end; t0 += STEPS, buf ^= 1) {
        S cx[TS], cr[TS], ci[TS];
#pragma unroll
        for (int k = 0; k < TS; ++k) cx[k] = nx[k], cr[k] = nr[k], ci[k] = ni[k];
        const uint64_t bits = RESET ? nbits >> (sub * TS) : 0;
        if (t0 + STEPS < t_end) fetch(t0 + STEPS);
        const int64_t t_run = t0 + (int64_t)run * TS;
        const int64_t left = t_end - t_run;  // steps of this run that exist, if below TS

        float a[TS], bb[TS], esum = 0.0f, h = 0.0f;
#pragma unroll
        for (int k = 0; k < TS; ++k) {
            float e = tl * sigmoid_f(to_f32(cr[k]));
            if (RESET) e = (bits >> k) & 1 ? __builtin_inff() : e;
            if (k >= left) e = 0.0f;  // past the end: the state is carried
            a[k] = decay_of<RESET>(e);
            const float m = __builtin_amdgcn_sqrtf(one_minus_sq(e, a[k]));
            const float g = sigmoid_f(to_f32(ci[k])) * to_f32(cx[k]);
            bb[k] = k >= left ? 0.0f : m * g;
            h = decay_fma<RESET>(a[k], h, bb[k]);
            esum += e;
        }
        s_pair[buf][run * CH + ch] = make_float2(decay_of<RESET>(esum), h);
        __syncthreads();
        // the state entering this run, and the chunk's end state in every lane
        float in = 0.0f;
#pragma unroll
        for (int q = 0; q < RUNS; ++q) {
            if (q == run) in = carry;
            const float2 v = s_pair[buf][q * CH + ch];
            carry = decay_fma<RESET>(v.x, carry, v.y);
            if (MODE == kGatedPairs) carry_a = pair_product<RESET>(carry_a, v.x);
        }
        if (MODE != kGatedPairs) {
            if (p.ck && live && t_run % kGatedCk == 0 && left > 0) p.ck[(b * p.nck + t_run / kGatedCk) * D + d] = in;
        }
        if (MODE == kGatedStates) {
#pragma unroll
            for (int k = 0; k < TS; ++k) {
                in = decay_fma<RESET>(a[k], in, bb[k]);
                if (live && k < left) gated_store<S>(y, p.sy_t, t0 + wave * R * TS, sub * TS, k, d, in);
            }
        }
    }
    if (wave == 0 && sub == 0 && live) {
        if (MODE == kGatedPairs) p.agg[(b * p.nseg + seg) * D + d] = make_float2(carry_a, carry);
        if (MODE == kGatedStates && p.last && seg == p.nseg - 1) p.last[b * D + d] = carry;
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
// come from its checkpoint by the forward's local scan and fold; the adjoint mu_t = a_t g_t, with
// g_t = dy_t + mu_{t+1}, is the same recurrence from the right, mu_t = a_t mu_{t+1} + a_t dy_t, whose
// runs have the same product of a: one LDS exchange and one barrier serve both directions.
// MODE kGatedPairs: the adjoint pairs of whole segments (all but the first), from r and dy alone.
template <typename S, int CH, int W, int TS, bool RESET, int MODE>
__global__ __launch_bounds__(W * 64) __attribute__((amdgpu_waves_per_eu(4))) void gated_bwd_kernel(GatedBwdParams p) {
    constexpr int R = 64 / CH, RUNS = W * R, STEPS = RUNS * TS;
    static_assert(STEPS == kGatedCk && R * TS <= 64);
    __shared__ float2 s_pair[2][RUNS * CH];
    __shared__ float s_mu[2][RUNS * CH];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ch = lane % CH, sub = lane / CH, run = wave * R + sub;
    constexpr int share = CH * (int)sizeof(S) < 128 ? 128 / (CH * (int)sizeof(S)) : 1;
    const int64_t D = p.dim, L = p.len;
    const int nseg = MODE == kGatedPairs ? p.nseg - 1 : p.nseg;
    const GatedPlace at = gated_place((D + CH - 1) / CH, p.batch, nseg, share);
    if (!at.ok) return;
    const int64_t b = at.b, seg = MODE == kGatedPairs ? at.seg + 1 : at.seg;
    const int64_t d_own = at.group * CH + ch;
    const bool live = d_own < D;
    const int64_t d = live ? d_own : D - 1;
    const int64_t t_begin = seg * p.seg_len;
    const int64_t t_end = t_begin + p.seg_len < L ? t_begin + p.seg_len : L;

    const S* x = static_cast<const S*>(p.x) + b * p.sx_b;
    const S* r = static_cast<const S*>(p.r) + b * p.sr_b;
    const S* i = static_cast<const S*>(p.i) + b * p.si_b;
    const S* dy = static_cast<const S*>(p.dy) + b * p.sdy_b;
    S* dx = static_cast<S*>(p.dx) + b * p.sdx_b;
    S* dr = static_cast<S*>(p.dr) + b * p.sdr_b;
    S* di = static_cast<S*>(p.di) + b * p.sdi_b;
    const uint8_t* reset = RESET ? p.reset + b * L : nullptr;
    const float tl = p.c * kLog2e * softplus_f(p.lam[d]);

    float carry = 0.0f, carry_a = 1.0f;  // mu entering from the right
    if (MODE != kGatedPairs) {
        carry = p.dlast ? p.dlast[b * D + d] : 0.0f;
        for (int64_t q = p.nseg - 1; q > seg; --q) {
            const float2 v = p.agg[(b * p.nseg + q) * D + d];
            carry = decay_fma<RESET>(v.x, carry, v.y);
        }
    }
    float acc = 0.0f;

    S nx[TS], nr[TS], ni[TS], ng[TS];
    uint64_t nbits = 0;
    float nck = 0.0f;
    auto fetch = [&](int64_t t0) __attribute__((always_inline)) {
        const int64_t tw = t0 + (int64_t)wave * R * TS;
        if (t0 + STEPS <= t_end) {
            if (MODE != kGatedPairs) gated_rows<S, TS, true>(nx, x, p.sx_t, tw, sub * TS, d, L);
            gated_rows<S, TS, true>(nr, r, p.sr_t, tw, sub * TS, d, L);
            if (MODE != kGatedPairs) gated_rows<S, TS, true>(ni, i, p.si_t, tw, sub * TS, d, L);
            gated_rows<S, TS, true>(ng, dy, p.sdy_t, tw, sub * TS, d, L);
        } else {
            if (MODE != kGatedPairs) gated_rows<S, TS, false>(nx, x, p.sx_t, tw, sub * TS, d, L);
            gated_rows<S, TS, false>(nr, r, p.sr_t, tw, sub * TS, d, L);
            if (MODE != kGatedPairs) gated_rows<S, TS, false>(ni, i, p.si_t, tw, sub * TS, d, L);
            gated_rows<S, TS, false>(ng, dy, p.sdy_t, tw, sub * TS, d, L);
        }
        if (RESET) nbits = gated_reset_bits<R * TS>(reset, tw, L, lane);
        if (MODE != kGatedPairs) nck = p.ck[(b * p.nck + t0 / kGatedCk) * D + d];
    };
    const int64_t t_last = t_begin + (t_end - t_begin - 1) / STEPS * STEPS;
    fetch(t_last);
    int buf = 0;
    for (int64_t t0 = t_last; t0 >= t_begin; t0 -= STEPS, buf ^= 1) {
        S cx[TS], cr[TS], ci[TS], cg[TS];
#pragma unroll
        for (int k = 0; k < TS; ++k) cx[k] = nx[k], cr[k] = nr[k], ci[k] = ni[k], cg[k] = ng[k];
        const uint64_t bits = RESET ? nbits >> (sub * TS) : 0;
        float h = nck;
        if (t0 > t_begin) fetch(t0 - STEPS);
        const int64_t t_run = t0 + (int64_t)run * TS;
        const int64_t left = t_end - t_run;

        float e[TS], a[TS], sr[TS], si[TS], bb[TS], rm[TS], g[TS];
        float esum = 0.0f, hl = 0.0f, mu = 0.0f;
#pragma unroll
        for (int k = 0; k < TS; ++k) {
            sr[k] = sigmoid_f(to_f32(cr[k]));
            e[k] = tl * sr[k];
            if (RESET) e[k] = (bits >> k) & 1 ? __builtin_inff() : e[k];
            if (k >= left) e[k] = 0.0f;
            a[k] = decay_of<RESET>(e[k]);
            esum += e[k];
            g[k] = k >= left ? 0.0f : to_f32(cg[k]);
            if (MODE != kGatedPairs) {
                const float w = one_minus_sq(e[k], a[k]);
                rm[k] = w > 1.1754944e-38f ? __builtin_amdgcn_rsqf(w) : 0.0f;  // 1 / m, or 0 with m
                si[k] = sigmoid_f(to_f32(ci[k]));
                bb[k] = k >= left ? 0.0f : w * rm[k] * (si[k] * to_f32(cx[k]));
                hl = decay_fma<RESET>(a[k], hl, bb[k]);
            }
        }
#pragma unroll
        for (int k = TS - 1; k >= 0; --k) mu = decay_mul<RESET>(a[k], g[k] + mu);
        s_pair[buf][run * CH + ch] = make_float2(decay_of<RESET>(esum), hl);
        s_mu[buf][run * CH + ch] = mu;
        __syncthreads();
        // the adjoint entering this run from the right, and the one leaving the chunk on the left
        float in = 0.0f;
#pragma unroll
        for (int q = RUNS - 1; q >= 0; --q) {
            if (q == run) in = carry;
            const float pa = s_pair[buf][q * CH + ch].x;
            carry = decay_fma<RESET>(pa, carry, s_mu[buf][q * CH + ch]);
            if (MODE == kGatedPairs) carry_a = pair_product<RESET>(carry_a, pa);
        }
        if (MODE != kGatedPairs) {
#pragma unroll
            for (int q = 0; q < RUNS - 1; ++q) {  // the state entering this run
                const float2 v = s_pair[buf][q * CH + ch];
                if (q < run) h = decay_fma<RESET>(v.x, h, v.y);
            }
            float hp[TS];
#pragma unroll
            for (int k = 0; k < TS; ++k) {
                hp[k] = h;
                h = decay_fma<RESET>(a[k], h, bb[k]);
            }
#pragma unroll
            for (int k = TS - 1; k >= 0; --k) {
                const float gk = g[k] + in;
                in = decay_mul<RESET>(a[k], gk);
                const float xf = to_f32(cx[k]);
                const float w = one_minus_sq(e[k], a[k]);
                const float vx = gk * (w * rm[k]) * si[k];
                const float s = (RESET ? __builtin_fminf(e[k], 1e30f) : e[k]) * kLn2;
                const float q = decay_mul<RESET>(in * s, si[k] * xf * a[k] * rm[k] - hp[k]);
                if (k < left) {
                    acc += q;
                    if (live) {
                        const int64_t tw = t0 + wave * R * TS;
                        gated_store<S>(dx, p.sdx_t, tw, sub * TS, k, d, vx);
                        gated_store<S>(di, p.sdi_t, tw, sub * TS, k, d, vx * xf * (1.0f - si[k]));
                        gated_store<S>(dr, p.sdr_t, tw, sub * TS, k, d, q * (1.0f - sr[k]));
                    }
                }
            }
        }
    }
    if (MODE == kGatedPairs) {
        if (wave == 0 && sub == 0 && live) p.agg[(b * p.nseg + seg) * D + d] = make_float2(carry_a, carry);
        return;
    }
    // q summed over the runs, in run order
    __syncthreads();
    s_mu[0][run * CH + ch] = acc;
    __syncthreads();
    if (wave == 0 && sub == 0 && live) {
        float sum = 0.0f;
        for (int q = 0; q < RUNS; ++q) sum += s_mu[0][q * CH + ch];
        p.part[(b * p.nseg + seg) * D + d] = sum;
        if (p.dh0 && seg == 0) p.dh0[b * D + d] = carry;
    }
}

}  // namespace mscan
