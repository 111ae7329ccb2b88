// The gated linear recurrence (mamba_layers.h) on gfx950, forward and backward.
//
//   e_t = c log2(e) softplus(lam) sigmoid(r_t)   (= -log2 a_t)      a_t = 2^-e_t
//   h_t = a_t h_{t-1} + b_t,   b_t = m_t sigmoid(i_t) x_t,   m_t = sqrt(1 - a_t^2)
//
// One lane owns one channel and a run of TS consecutive steps. A workgroup owns 64 consecutive channels
// of one batch and walks the sequence in chunks: its 16 waves hold 16 consecutive runs, so a chunk is
// 16 TS steps read as rows of 64 contiguous channels. Each lane scans its run from a zero state and
// writes the run's pair (product of a, end state) to LDS; there the 16 pairs of a channel are scanned by
// the 16 lanes of one DPP row (16 x 64 pairs, 1024 threads), which also carries the channel's state from
// chunk to chunk; each lane takes back the state entering its run, and one FMA a step gives the states.
// Every input is read once, so nothing but the inputs and outputs passes through HBM. (The alternative,
// one pass for the pairs of all chunks and a second for the states, reads the inputs and computes the
// gates twice.)
//
// Few rows: `ways` workgroups share a (batch, channel group). Each takes the next chunk by a ticket,
// scans it without its state and publishes the chunk's pair; the state entering chunk 16 k + j is that
// entering chunk 16 k, published by the one before it, carried over the published pairs of chunks 16 k ..
// 16 k + j - 1 (the lanes of a DPP row again). Every state is composed in this one order whoever works on
// the chunks, so the results do not depend on timing, and states pass from workgroup to workgroup only
// every 16 chunks. (Passing every chunk's state on to the next cost 4.7 us a chunk, a store and a load
// through memory that all XCDs see: 1855 us at 4 x 100000 x 1024 where 64 unshared workgroups take 1336.)
// Every wait ends: of the chunks not yet done, the first is the earliest ticket of the workgroup that
// holds it (tickets are taken in rising order, up to two ahead), so it is being worked on, and what it
// waits for belongs to chunks before it. (fp32 workgroups scan their next chunk, which waits for nothing,
// before they finish one.)
#pragma once

#include <type_traits>

#include "layers_common.hpp"
#include "xcd.hpp"

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
    uint64_t* chain;    // with ways > 1: GatedChain's words, zero before the launch
    int64_t batch, len, dim, nck;
    int64_t sx_b, sx_t, sr_b, sr_t, si_b, si_t, sy_b, sy_t;
    int ways;
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
    float* dlam;
    float* part;        // (batch, nck, dim): each chunk's sum of q
    uint64_t* chain;
    int64_t batch, len, dim, nck;
    int64_t sx_b, sx_t, sr_b, sr_t, si_b, si_t, sdy_b, sdy_t, sdx_b, sdx_t, sdr_b, sdr_t, sdi_b, sdi_t;
    int ways;
    float c;
};

constexpr int kGatedCk = MAMBA_GATED_CHECKPOINT;

// Steps of a run of the forward. Alone on its chain a workgroup walks 128-step chunks (8 x 2048 x 1536
// bf16, before the loop's last savings: 58 us; 64 with 256 steps, where the first chunk's load and the last
// one's stores stand alone, and 62 with 128 steps loaded two chunks ahead). Chained workgroups exchange a
// pair per chunk, and 256 steps halve that (4 x 100000 x 1024 bf16: 926 us; 1130 with 128 whose states wait
// for the next chunk, 1366 with 128 as they come; 940 since resets are selected and the series is whole);
// fp32 loads take twice the bytes and keep 128.
//
// Bound by the VALU and HBM together: an element takes 27 vector instructions and 6 transcendental ones (33
// and 6 with copies of the loaded values and without the DPP forms below). 8 x 2048 x 1536 bf16 56 us, 3.6
// TB/s with 192 of 256 compute units at work; 32 x 2000 x 2500 293 us, 4.4 TB/s; 8 x 2048 x 1536 fp32 91 us,
// 4.4 TB/s; a large copy reaches 4.6.
constexpr int gated_fwd_ts(int bytes, bool chain) { return bytes == 2 && chain ? 16 : 8; }

__device__ __forceinline__ float sigmoid_of_scaled(float s) { return hw_rcp(1.0f + hw_exp2(s)); }  // s = -log2(e) v
__device__ __forceinline__ float sigmoid_f(float v) { return sigmoid_of_scaled(-v * kLog2e); }
// Computes a value here: what was loaded for a chunk becomes what the chunk works on, without a copy, before
// the next chunk's loads take its registers.
__device__ __forceinline__ float here(float v) {
    asm volatile("" : "+v"(v));
    return v;
}

// A chunk's resets for a second loop over its steps: read again from the bits there, one scalar, where the
// compiler would keep the first loop's selections, two scalars a step.
template <bool RESET>
__device__ __forceinline__ uint32_t again(uint32_t bits) {
    if constexpr (RESET) asm volatile("" : "+s"(bits));
    return bits;
}

// 1 - a^2 = 1 - e^-v at v = 2 ln(2) e, given a. Below v = 1/4 the series
// v (1 - v/2 + v^2/6 - v^3/24 + v^4/120 - v^5/720), coefficients scaled to e (truncation below 2^-24
// relative); above, 1 - a^2 in one rounding, where cancellation costs at most 7.1 times a's own relative
// error, and its square root 3.6 times. For bf16 activations too: states, checkpoints and lam's gradient are
// fp32 there as well (three terms below v = 1/64 cost them 4 bits and saved 3 instructions of an element's
// 33: 8 x 2048 x 1536 bf16 forward 55.2 us, 56.6 so).
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

// One step, `on` being whether it is a reset (the same for the whole wave): a h + b, and a v of the adjoint.
// A reset forgets what lies before it, infinities and NaN among it, by a selection; every other step passes
// them on, a NaN of its own decay too.
template <bool RESET>
__device__ __forceinline__ float step_fma(float a, float h, float b, bool on) {
    const float v = __builtin_fmaf(a, h, b);
    return RESET && on ? b : v;
}
template <bool RESET>
__device__ __forceinline__ float step_mul(float a, float v, bool on) {
    const float w = a * v;
    return RESET && on ? 0.0f : w;
}
// A step's decay 2^-e; a reset's e is infinite.
template <bool RESET>
__device__ __forceinline__ float decay_step(float& e, bool on) {
    if constexpr (RESET) e = on ? __builtin_inff() : e;
    return hw_exp2(-e);
}
// Runs are folded as pairs (product of the decays, end state). A product of exactly 0 says that a reset lies
// in the run; every other is kept above 0 (kMinDecay). A run with a NaN decay and no reset has a NaN end state
// in either direction, so its product may be any but 0.
constexpr float kMinDecay = 1.1754944e-38f;
template <bool RESET>
__device__ __forceinline__ float decay_fma(float a, float h, float b) {
    const float v = __builtin_fmaf(a, h, b);
    return RESET && a == 0.0f ? b : v;
}
template <bool RESET>
__device__ __forceinline__ float pair_product(float a, float b) {
    if constexpr (RESET) return __builtin_fmaxf(a * b, __builtin_fminf(__builtin_fminf(a, b), kMinDecay));
    return a * b;
}
// The product of a run, 2^-(the sum of its e); bits: its resets.
template <bool RESET>
__device__ __forceinline__ float decay_of(float esum, uint32_t bits) {
    const float a = hw_exp2(-esum);
    if constexpr (RESET) return bits ? 0.0f : __builtin_fmaxf(a, kMinDecay);
    return a;
}

// A workgroup's chain (batch, channel group). The ways of the chains lie one after another, and an XCD takes one
// stretch of them: neighbouring groups, so that rows that begin inside a cache line are fetched once for two
// groups (32 x 1000 x 700 fp32, forward and backward: 300 us with neighbours on neighbouring XCDs, 248 so; no
// difference at whole lines), a chain's ways together where they fit, and every XCD the same number of
// workgroups. (Whole chains on one XCD leave XCDs idle where there are few: 1 x 100000 x 64 bf16 forward 152 us
// on one XCD, 47 on all eight; 1 x 20000 x 768 80 and 59.)
struct GatedPlace {
    int64_t chain, group, b;
    bool ok;
};
__device__ __forceinline__ GatedPlace gated_place(int64_t groups, int64_t batch, int ways) {
    const int64_t id = grid_block(), n = groups * batch * ways;
    GatedPlace p;
    p.chain = xcd_item(id, n) / ways;
    p.ok = id < n;
    p.group = p.chain % groups;
    p.b = p.chain / groups;
    return p;
}
inline int64_t gated_blocks(int64_t chains, int ways) { return chains * ways; }

// What the workgroups of a chain pass on: values beside a mark that they are there.
__device__ __forceinline__ void word_put(uint64_t* w, float v) {
    __hip_atomic_store(w, (uint64_t)1 << 32 | __float_as_uint(v), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t word_look(const uint64_t* w) {
    return __hip_atomic_load(w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
struct GatedChain {
    uint64_t* pairs;   // (batch, chunks, dim, 2)
    uint64_t* states;  // (batch, chunks / 16, dim): entering chunks 16, 32, ...
    int* tickets;      // (batch * groups)
    static __host__ __device__ int64_t state_rows(int64_t chunks) { return (chunks + 15) / 16; }
    static __host__ __device__ int64_t words(int64_t batch, int64_t dim, int64_t chunks) {
        return batch * dim * (2 * chunks + state_rows(chunks)) + (batch * ((dim + 63) / 64) + 1) / 2;
    }
    __device__ __forceinline__ GatedChain(uint64_t* w, int64_t batch, int64_t dim, int64_t chunks)
        : pairs(w), states(w + batch * dim * 2 * chunks),
          tickets(reinterpret_cast<int*>(w + batch * dim * (2 * chunks + state_rows(chunks)))) {}
};

// Rows of a chunk are addressed through a buffer descriptor at the run's first row: the lane's channel in
// a register, the row within the run in a scalar. A lane without a row or channel uses an offset past
// the buffer, which reads 0 and drops stores, so neither needs a branch.
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
    uint32_t off;   // the lane's channel, bytes
    __device__ __forceinline__ Seq(S* p, int64_t st_, int64_t d) : base(p), st(st_), off((uint32_t)d * (uint32_t)sizeof(S)) {}
    __device__ __forceinline__ int row_bytes() const { return (int)st * (int)sizeof(S); }
};

template <typename S, int TS, bool FULL>
__device__ __forceinline__ void gated_rows(S (&v)[TS], const Seq<const S>& q, int64_t t_run, int left) {
    const __amdgpu_buffer_rsrc_t r = gated_rsrc(q.base + t_run * q.st);
#pragma unroll
    for (int k = 0; k < TS; ++k) row_load(v[k], r, FULL || k < left ? q.off : kGatedDrop, k * q.row_bytes());
}

// The reset bytes of a run, a lane's own each, 0 past the run's or the sequence's end; loaded before the run's
// rows, so that no wait for them waits for the rows too, and one bit each where they are used.
template <int N>
__device__ __forceinline__ uint32_t gated_reset_byte(const uint8_t* reset, int64_t t_run, int left, int lane) {
    return __builtin_amdgcn_raw_buffer_load_b8(gated_rsrc(reset + t_run), lane < N && lane < left ? lane : (int)kGatedDrop, 0, 0);
}
__device__ __forceinline__ uint32_t gated_reset_bits(uint32_t byte) { return (uint32_t)__ballot(byte != 0); }

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
    // The same with the lane shift inside the instructions: lanes without a source keep a and add 0 to h. A
    // DPP operand is read 2 wait states after its write at the earliest, also by what follows the block.
#define MSCAN_ROW_STEP(DIR, N)                                                                    \
    "s_nop 1\n\tv_fmac_f32_dpp %1, %1, %0 " DIR ":" N " row_mask:0xf bank_mask:0xf bound_ctrl:0\n\t" \
    "v_mul_f32_dpp %0, %0, %0 " DIR ":" N " row_mask:0xf bank_mask:0xf\n\t"
#define MSCAN_ROW_STEPS(DIR) \
    MSCAN_ROW_STEP(DIR, "1") MSCAN_ROW_STEP(DIR, "2") MSCAN_ROW_STEP(DIR, "4") MSCAN_ROW_STEP(DIR, "8") "s_nop 1"
    if constexpr (!RESET) {
        if constexpr (UP) asm(MSCAN_ROW_STEPS("row_shr") : "+v"(a), "+v"(h));
        else asm(MSCAN_ROW_STEPS("row_shl") : "+v"(a), "+v"(h));
        return;
    }
#undef MSCAN_ROW_STEPS
#undef MSCAN_ROW_STEP
    step(dpp_from<shift + 1>(a, 1.0f), dpp_from<shift + 1>(h, 0.0f));
    step(dpp_from<shift + 2>(a, 1.0f), dpp_from<shift + 2>(h, 0.0f));
    step(dpp_from<shift + 4>(a, 1.0f), dpp_from<shift + 4>(h, 0.0f));
    step(dpp_from<shift + 8>(a, 1.0f), dpp_from<shift + 8>(h, 0.0f));
}

// The pair of chunk `cur` of a chain's walk, for the chunks after it.
__device__ __forceinline__ void chain_publish(const GatedChain& c, int64_t b, int64_t D, int64_t ds, bool owner, int n, int cur,
                                              float2 pair) {
    if (!owner) return;
    uint64_t* w = c.pairs + ((b * n + cur) * D + ds) * 2;
    word_put(w, pair.x);
    word_put(w + 1, pair.y);
}
// The value entering chunk `cur`, in every lane of the channel's DPP row; `first` enters chunk 0.
template <bool RESET>
__device__ __forceinline__ float chain_state(const GatedChain& c, int64_t b, int64_t D, int64_t ds, int n, int cur, int row_lane,
                                             float first) {
    const int block = cur / 16, j = cur % 16;
    float a = 1.0f, h = 0.0f, state = first;
    if (row_lane < j) {
        const uint64_t* w = c.pairs + ((b * n + block * 16 + row_lane) * D + ds) * 2;
        uint64_t va = word_look(w), vh = word_look(w + 1);
        while (!(va >> 32 && vh >> 32)) {
            __builtin_amdgcn_s_sleep(1);
            va = word_look(w), vh = word_look(w + 1);
        }
        a = __uint_as_float((uint32_t)va);
        h = __uint_as_float((uint32_t)vh);
    }
    if (block > 0) {
        const uint64_t* w = c.states + (b * GatedChain::state_rows(n) + block) * D + ds;
        uint64_t v = word_look(w);
        while (!(v >> 32)) {
            __builtin_amdgcn_s_sleep(1);
            v = word_look(w);
        }
        state = __uint_as_float((uint32_t)v);
    }
    row_scan<true, RESET>(a, h);
    return decay_fma<RESET>(dpp_from<kRowBcast + 15>(a, 1.0f), state, dpp_from<kRowBcast + 15>(h, 0.0f));
}
// The value leaving chunk `cur`, for the block of 16 chunks after it.
__device__ __forceinline__ void chain_exit(const GatedChain& c, int64_t b, int64_t D, int64_t ds, bool live, int n, int cur,
                                           float after) {
    if (cur % 16 == 15 && live && cur + 1 < n) word_put(c.states + (b * GatedChain::state_rows(n) + (cur + 1) / 16) * D + ds, after);
}

constexpr int kRuns = 16;   // runs of a chunk: the lanes of a DPP row
constexpr int kChans = 64;  // channels of a workgroup: the lanes of a wave
constexpr int kPitch = kChans + 4;  // a run's row in LDS: the 16 runs x 4 channels a wave scans lie in distinct banks

// The walk of a workgroup over the chunks of its chain, number 0 .. n - 1 in the order of the walk: all of
// them, or those it gets tickets for. The ticket after the next is asked for at the start of a chunk and
// passed on by the chunk's barriers.
template <bool CHAIN>
struct ChunkWalk {
    int* ticket;
    int (&lds)[2];
    int n, cur, next, turn = 0;
    __device__ __forceinline__ ChunkWalk(int* t, int (&l)[2], int n_) : ticket(t), lds(l), n(n_) {
        cur = draw();
        next = 1;
    }
    __device__ __forceinline__ int draw() {
        if constexpr (!CHAIN) return 0;
        __syncthreads();
        if (threadIdx.x == 0) lds[0] = atomicAdd(ticket, 1);
        __syncthreads();
        return __builtin_amdgcn_readfirstlane(lds[0]);
    }
    // The second ticket, a memory round trip after the first: the chain's other workgroups have drawn
    // their first by then, and neighbouring chunks are worked on side by side.
    __device__ __forceinline__ void second() {
        if constexpr (CHAIN) {
            next = draw();
            __syncthreads();
        }
    }
    __device__ __forceinline__ void ask() {  // before the chunk's first barrier
        if constexpr (CHAIN)
            if (threadIdx.x == 0) lds[turn] = atomicAdd(ticket, 1);
    }
    __device__ __forceinline__ void advance() {  // after it; lds[turn] is written again two chunks on
        cur = next;
        if constexpr (CHAIN) {
            next = __builtin_amdgcn_readfirstlane(lds[turn]);
            turn ^= 1;
        } else {
            ++next;
        }
    }
};

template <typename S, int TS, bool RESET, bool STATES, bool CHAIN>
__global__ __launch_bounds__(1024) void gated_fwd_kernel(GatedParams p) {
    constexpr int STEPS = kRuns * TS;
    static_assert(kGatedCk % TS == 0);
    __shared__ float2 s_pair[kRuns * kPitch];
    __shared__ float s_in[kRuns * kPitch];
    __shared__ int s_ticket[2];

    const int lane = threadIdx.x & 63;
    const int run = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int s_run = lane & 15, s_ch = run * 4 + (lane >> 4);  // the pair this thread scans
    const int64_t D = p.dim, L = p.len;
    const GatedPlace at = gated_place((D + kChans - 1) / kChans, p.batch, p.ways);
    if (!at.ok) return;
    const int64_t b = at.b;
    const int64_t d_own = at.group * kChans + lane, d_scan = at.group * kChans + s_ch;
    const bool live = d_own < D, s_live = d_scan < D;
    const int64_t d = live ? d_own : D - 1, ds = s_live ? d_scan : D - 1;

    const Seq<const S> x(static_cast<const S*>(p.x) + b * p.sx_b, p.sx_t, d);
    const Seq<const S> r(static_cast<const S*>(p.r) + b * p.sr_b, p.sr_t, d);
    const Seq<const S> i(static_cast<const S*>(p.i) + b * p.si_b, p.si_t, d);
    const Seq<S> y(static_cast<S*>(p.y) + b * p.sy_b, p.sy_t, d);
    const uint8_t* reset = RESET ? p.reset + b * L : nullptr;
    const float tl = p.c * kLog2e * softplus_f(p.lam[d]);

    float carry = p.h0 ? p.h0[b * D + ds] : 0.0f;  // the scanned channel's state entering the chunk
    const int n = (int)((L + STEPS - 1) / STEPS);
    const GatedChain chain(p.chain, p.batch, D, n);
    const float first = carry;
    ChunkWalk<CHAIN> walk(chain.tickets + at.chain, s_ticket, n);

    S nx[TS], nr[TS], ni[TS];
    uint32_t nreset = 0;
    auto fetch_as = [&](int64_t t0, auto full) __attribute__((always_inline)) {
        constexpr bool FULL = decltype(full)::value;
        const int64_t tr = t0 + run * TS;
        const int left = (int)(L - tr < TS ? L - tr : TS);
        if (RESET) nreset = gated_reset_byte<TS>(reset, tr, left, lane);
        gated_rows<S, TS, FULL>(nr, r, tr, left);
        gated_rows<S, TS, FULL>(ni, i, tr, left);
        gated_rows<S, TS, FULL>(nx, x, tr, left);
    };
    auto fetch = [&](int chunk) __attribute__((always_inline)) {
        const int64_t t0 = (int64_t)chunk * STEPS;
        if (t0 + STEPS <= L) fetch_as(t0, std::true_type{});
        else fetch_as(t0, std::false_type{});
    };
    if (walk.cur < n) fetch(walk.cur);
    walk.second();

    const int whole = (int)(L / STEPS);
    // bf16 runs of 16 steps have no registers for a second chunk's (4 x 100000 x 1024: 3500 us with it where it took 926 without)
    constexpr bool DEFER = CHAIN && sizeof(S) == 4;
    if constexpr (!DEFER) {
        auto chunk = [&](auto tail) __attribute__((always_inline)) {
            constexpr bool TAIL = decltype(tail)::value;
            const int64_t t0 = (int64_t)walk.cur * STEPS, tr = t0 + run * TS;
            float cx[TS], cr[TS], ci[TS];
#pragma unroll
            for (int k = 0; k < TS; ++k) {
                cr[k] = here(to_f32(nr[k]) * -kLog2e);
                ci[k] = here(to_f32(ni[k]) * -kLog2e);
                cx[k] = here(to_f32(nx[k]));
            }
            const uint32_t bits = RESET ? gated_reset_bits(nreset) : 0;
            walk.ask();
            if (walk.next < n) fetch(walk.next);
            const int left = (int)(L - tr < TS ? L - tr : TS);  // steps of this run that exist
            float a[TS], bb[TS], esum = 0.0f, h = 0.0f;
#pragma unroll
            for (int k = 0; k < TS; ++k) {
                float e = tl * sigmoid_of_scaled(cr[k]);
                a[k] = decay_step<RESET>(e, (bits >> k) & 1);
                const float m = __builtin_amdgcn_sqrtf(one_minus_sq(e, a[k]));
                bb[k] = m * (sigmoid_of_scaled(ci[k]) * cx[k]);
                if constexpr (TAIL) {  // past the end the state is carried
                    if (k >= left) {
                        a[k] = 1.0f;
                        bb[k] = e = 0.0f;
                    }
                }
                esum += e;
                h = step_fma<RESET>(a[k], h, bb[k], (bits >> k) & 1);
            }
            s_pair[run * kPitch + lane] = make_float2(decay_of<RESET>(esum, bits), h);
            __syncthreads();
            {
                float2 v = s_pair[s_run * kPitch + s_ch];
                row_scan<true, RESET>(v.x, v.y);
                if constexpr (CHAIN) {
                    chain_publish(chain, b, D, ds, s_live && s_run == 15, n, walk.cur, v);
                    carry = chain_state<RESET>(chain, b, D, ds, n, walk.cur, s_run, first);
                }
                const float after = decay_fma<RESET>(v.x, carry, v.y);
                if constexpr (CHAIN) chain_exit(chain, b, D, ds, s_live && s_run == 15, n, walk.cur, after);
                s_in[s_run * kPitch + s_ch] = dpp_from<kRowShr + 1>(after, carry);
                carry = dpp_from<kRowBcast + 15>(after, 0.0f);
            }
            __syncthreads();
            float in = s_in[run * kPitch + lane];
            if (p.ck && live && tr % kGatedCk == 0 && left > 0) p.ck[(b * p.nck + tr / kGatedCk) * D + d] = in;
            if (STATES) {
                const __amdgpu_buffer_rsrc_t o = gated_rsrc(y.base + tr * y.st);
                const uint32_t resets = again<RESET>(bits);
#pragma unroll
                for (int k = 0; k < TS; ++k) {
                    in = step_fma<RESET>(a[k], in, bb[k], (resets >> k) & 1);
                    row_store(from_f32<S>(in), o, live && (!TAIL || k < left) ? y.off : kGatedDrop, k * y.row_bytes());
                }
                if (p.last && walk.cur == n - 1 && s_run == 15 && s_live) p.last[b * D + ds] = carry;
            }
            walk.advance();
        };
        while (walk.cur < whole) chunk(std::false_type{});
        if (walk.cur < n) chunk(std::true_type{});
    } else {
        // A chunk's states wait until the workgroup's next chunk is scanned: its neighbours' pairs are there by
        // then, and whoever has chunks before it finishes them without waiting for this one (2 x 8000 x 1024 fp32
        // forward: 65 us, 82 without). The steps are written out again: sharing code with the loop above costs
        // that one spilled registers (4 x 100000 x 1024 bf16: 970 us where it took 926).
        int held = -1;
        uint32_t held_bits = 0;
        float a[TS], bb[TS];
        float2 pairs = make_float2(1.0f, 0.0f);
        auto resolve = [&]() __attribute__((always_inline)) {
            carry = chain_state<RESET>(chain, b, D, ds, n, held, s_run, first);
            const float after = decay_fma<RESET>(pairs.x, carry, pairs.y);
            chain_exit(chain, b, D, ds, s_live && s_run == 15, n, held, after);
            s_in[s_run * kPitch + s_ch] = dpp_from<kRowShr + 1>(after, carry);
            carry = dpp_from<kRowBcast + 15>(after, 0.0f);
        };
        auto finish = [&](auto tail) __attribute__((always_inline)) {
            constexpr bool TAIL = decltype(tail)::value;
            const int64_t tr = (int64_t)held * STEPS + run * TS;
            const int left = (int)(L - tr < TS ? L - tr : TS);
            float in = s_in[run * kPitch + lane];
            if (p.ck && live && tr % kGatedCk == 0 && left > 0) p.ck[(b * p.nck + tr / kGatedCk) * D + d] = in;
            if (STATES) {
                const __amdgpu_buffer_rsrc_t o = gated_rsrc(y.base + tr * y.st);
#pragma unroll
                for (int k = 0; k < TS; ++k) {
                    in = step_fma<RESET>(a[k], in, bb[k], (held_bits >> k) & 1);
                    row_store(from_f32<S>(in), o, live && (!TAIL || k < left) ? y.off : kGatedDrop, k * y.row_bytes());
                }
                if (p.last && held == n - 1 && s_run == 15 && s_live) p.last[b * D + ds] = carry;
            }
        };
        auto chunk = [&](auto tail) __attribute__((always_inline)) {
            constexpr bool TAIL = decltype(tail)::value;
            const int64_t tr = (int64_t)walk.cur * STEPS + run * TS;
            float cx[TS], cr[TS], ci[TS], na[TS], nb[TS];
#pragma unroll
            for (int k = 0; k < TS; ++k) {
                cr[k] = here(to_f32(nr[k]) * -kLog2e);
                ci[k] = here(to_f32(ni[k]) * -kLog2e);
                cx[k] = here(to_f32(nx[k]));
            }
            const uint32_t bits = RESET ? gated_reset_bits(nreset) : 0;
            walk.ask();
            if (walk.next < n) fetch(walk.next);
            const int left = (int)(L - tr < TS ? L - tr : TS);  // steps of this run that exist
            float esum = 0.0f, h = 0.0f;
#pragma unroll
            for (int k = 0; k < TS; ++k) {
                float e = tl * sigmoid_of_scaled(cr[k]);
                na[k] = decay_step<RESET>(e, (bits >> k) & 1);
                const float m = __builtin_amdgcn_sqrtf(one_minus_sq(e, na[k]));
                nb[k] = m * (sigmoid_of_scaled(ci[k]) * cx[k]);
                if constexpr (TAIL) {  // past the end the state is carried
                    if (k >= left) {
                        na[k] = 1.0f;
                        nb[k] = e = 0.0f;
                    }
                }
                esum += e;
                h = step_fma<RESET>(na[k], h, nb[k], (bits >> k) & 1);
            }
            s_pair[run * kPitch + lane] = make_float2(decay_of<RESET>(esum, bits), h);
            __syncthreads();
            float2 v = s_pair[s_run * kPitch + s_ch];
            row_scan<true, RESET>(v.x, v.y);
            chain_publish(chain, b, D, ds, s_live && s_run == 15, n, walk.cur, v);
            if (held >= 0) resolve();
            __syncthreads();
            if (held >= 0) finish(std::false_type{});
#pragma unroll
            for (int k = 0; k < TS; ++k) a[k] = na[k], bb[k] = nb[k];
            pairs = v;
            held_bits = bits;
            held = walk.cur;
            walk.advance();
        };
        while (walk.cur < whole) chunk(std::false_type{});
        if (walk.cur < n) chunk(std::true_type{});
        if (held < 0) return;
        __syncthreads();
        resolve();
        __syncthreads();
        if (held < whole) finish(std::false_type{});
        else finish(std::true_type{});
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
// and the outputs: a, b, e, m sigmoid(i), b (1 - sigmoid(i)), (s / m) a sigmoid(i) x / s, dy. Each
// chunk's sum of q is written by itself (added up in order afterwards), so that it does not matter which
// workgroup of a chain had which chunk. Bound by the VALU (52 plain and 6 transcendental instructions an
// element) and HBM: 8 x 2048 x 1536 bf16 98 us for 352 MB with 192 of 256 compute units at work, 3.6 TB/s.
template <typename S, int TS, bool RESET, bool CHAIN>
__global__ __launch_bounds__(1024) void gated_bwd_kernel(GatedBwdParams p) {
    constexpr int STEPS = kRuns * TS;
    static_assert(STEPS == kGatedCk);
    __shared__ float2 s_pair[kRuns * kPitch];
    __shared__ float s_mu[kRuns * kPitch];
    __shared__ float2 s_in[kRuns * kPitch];
    __shared__ float s_acc[kRuns * kPitch];
    __shared__ int s_ticket[2];

    const int lane = threadIdx.x & 63;
    const int run = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int s_run = lane & 15, s_ch = run * 4 + (lane >> 4);
    const int64_t D = p.dim, L = p.len;
    const GatedPlace at = gated_place((D + kChans - 1) / kChans, p.batch, p.ways);
    if (!at.ok) return;
    const int64_t b = at.b;
    const int64_t d_own = at.group * kChans + lane, d_scan = at.group * kChans + s_ch;
    const bool live = d_own < D, s_live = d_scan < D;
    const int64_t d = live ? d_own : D - 1, ds = s_live ? d_scan : D - 1;

    const Seq<const S> x(static_cast<const S*>(p.x) + b * p.sx_b, p.sx_t, d);
    const Seq<const S> r(static_cast<const S*>(p.r) + b * p.sr_b, p.sr_t, d);
    const Seq<const S> i(static_cast<const S*>(p.i) + b * p.si_b, p.si_t, d);
    const Seq<const S> dy(static_cast<const S*>(p.dy) + b * p.sdy_b, p.sdy_t, d);
    const Seq<S> dx(static_cast<S*>(p.dx) + b * p.sdx_b, p.sdx_t, d);
    const Seq<S> dr(static_cast<S*>(p.dr) + b * p.sdr_b, p.sdr_t, d);
    const Seq<S> di(static_cast<S*>(p.di) + b * p.sdi_b, p.sdi_t, d);
    const uint8_t* reset = RESET ? p.reset + b * L : nullptr;
    const float tl = p.c * kLog2e * softplus_f(p.lam[d]);
    // sigmoid(r) = e / tl. Below 1e-30 |q| is under 1e-14 |g sigmoid(i) x|, and its factor 1 - sigmoid(r) is left out.
    const float inv_tl = tl > 1e-30f ? hw_rcp(tl) * kLn2 : 0.0f;

    float carry = p.dlast ? p.dlast[b * D + ds] : 0.0f;  // mu entering the chunk from the right
    const int n = (int)((L + STEPS - 1) / STEPS);  // chunk n - 1 - (number of the walk)
    const GatedChain chain(p.chain, p.batch, D, n);
    const float first = carry;
    ChunkWalk<CHAIN> walk(chain.tickets + at.chain, s_ticket, n);

    S nx[TS], nr[TS], ni[TS], ng[TS];
    uint32_t nreset = 0;
    float nck = 0.0f;
    auto fetch_as = [&](int chunk, auto full) __attribute__((always_inline)) {
        constexpr bool FULL = decltype(full)::value;
        const int64_t tr = (int64_t)chunk * STEPS + run * TS;
        const int left = (int)(L - tr < TS ? L - tr : TS);
        if (RESET) nreset = gated_reset_byte<TS>(reset, tr, left, lane);
        gated_rows<S, TS, FULL>(nr, r, tr, left);
        gated_rows<S, TS, FULL>(ng, dy, tr, left);
        gated_rows<S, TS, FULL>(ni, i, tr, left);
        gated_rows<S, TS, FULL>(nx, x, tr, left);
        nck = p.ck[(b * p.nck + chunk) * D + ds];
    };
    if (walk.cur < n) {
        if (walk.cur > 0 || L % STEPS == 0) fetch_as(n - 1 - walk.cur, std::true_type{});
        else fetch_as(n - 1 - walk.cur, std::false_type{});
    }
    walk.second();
    int sums_of = -1;  // the chunk whose sums of q lie in s_acc
    auto flush = [&]() __attribute__((always_inline)) {  // after a barrier; over the runs, in a fixed order
        if (sums_of < 0) return;
        float q = s_acc[s_run * kPitch + s_ch];
        q += dpp_from<kRowShl + 8>(q, 0.0f);
        q += dpp_from<kRowShl + 4>(q, 0.0f);
        q += dpp_from<kRowShl + 2>(q, 0.0f);
        q += dpp_from<kRowShl + 1>(q, 0.0f);
        if (s_run == 0 && s_live) p.part[(b * p.nck + sums_of) * D + ds] = q;
    };
    auto chunk = [&](auto tail) __attribute__((always_inline)) {
        constexpr bool TAIL = decltype(tail)::value;
        const int which = n - 1 - walk.cur;
        const int64_t tr = (int64_t)which * STEPS + run * TS;
        // (chained, with its pointers: 44 registers spilled with it, 19 without)
        auto start = [](float v) __attribute__((always_inline)) { return CHAIN ? v : here(v); };
        float cx[TS], cr[TS], ci[TS], g[TS];
#pragma unroll
        for (int k = 0; k < TS; ++k) {
            cr[k] = start(to_f32(nr[k]) * -kLog2e);
            g[k] = start(to_f32(ng[k]));
            ci[k] = start(to_f32(ni[k]) * -kLog2e);
            cx[k] = start(to_f32(nx[k]));
        }
        const uint32_t bits = RESET ? gated_reset_bits(nreset) : 0;
        const float ck = nck;
        walk.ask();
        if (walk.next < n) fetch_as(n - 1 - walk.next, std::true_type{});  // only the walk's first chunk is cut short
        const int left = (int)(L - tr < TS ? L - tr : TS);

        float e[TS], a[TS], bb[TS], ms[TS], bi[TS], z[TS];
        float esum = 0.0f, hl = 0.0f, mu = 0.0f;
#pragma unroll
        for (int k = 0; k < TS; ++k) {
            const bool past = TAIL && k >= left;
            e[k] = tl * sigmoid_of_scaled(cr[k]);
            a[k] = decay_step<RESET>(e[k], (bits >> k) & 1);
            if constexpr (TAIL) {  // past the end the state and the adjoint are carried
                if (past) a[k] = 1.0f, e[k] = g[k] = 0.0f;
            }
            esum += e[k];
            const float w = one_minus_sq(e[k], a[k]);
            // 1 / m; where m is 0, so are e and with it all that 1 / m enters, as long as it is finite
            const float rm = __builtin_amdgcn_rsqf(__builtin_fmaxf(w, 1.1754944e-38f));
            const float si = sigmoid_of_scaled(ci[k]), v = past ? 0.0f : cx[k], rs = rm * si;
            ms[k] = w * rs;
            bb[k] = ms[k] * v;
            bi[k] = __builtin_fmaf(-bb[k], si, bb[k]);
            z[k] = a[k] * (rs * v);
            hl = step_fma<RESET>(a[k], hl, bb[k], (bits >> k) & 1);
        }
#pragma unroll
        for (int k = TS - 1; k >= 0; --k) mu = step_mul<RESET>(a[k], g[k] + mu, (bits >> k) & 1);
        s_pair[run * kPitch + lane] = make_float2(decay_of<RESET>(esum, bits), hl);
        s_mu[run * kPitch + lane] = mu;
        __syncthreads();
        {
            float2 v = s_pair[s_run * kPitch + s_ch];
            float ra = v.x, rmu = s_mu[s_run * kPitch + s_ch];
            row_scan<false, RESET>(ra, rmu);
            if constexpr (CHAIN) {
                chain_publish(chain, b, D, ds, s_live && s_run == 0, n, walk.cur, make_float2(ra, rmu));
                carry = chain_state<RESET>(chain, b, D, ds, n, walk.cur, s_run, first);
            }
            const float after = decay_fma<RESET>(ra, carry, rmu);
            if constexpr (CHAIN) chain_exit(chain, b, D, ds, s_live && s_run == 0, n, walk.cur, after);
            float2 o;
            o.y = dpp_from<kRowShl + 1>(after, carry);  // the adjoint entering the run from the right
            carry = dpp_from<kRowBcast + 0>(after, 0.0f);
            row_scan<true, RESET>(v.x, v.y);
            o.x = dpp_from<kRowShr + 1>(decay_fma<RESET>(v.x, ck, v.y), ck);  // the state entering it
            s_in[s_run * kPitch + s_ch] = o;
            flush();
        }
        __syncthreads();
        const float2 o = s_in[run * kPitch + lane];
        float in = o.y, acc = 0.0f;
        {
            float h = o.x;
            const uint32_t resets = again<RESET>(bits);
#pragma unroll
            for (int k = 0; k < TS; ++k) {  // z becomes z - h before the step
                z[k] -= h;
                h = step_fma<RESET>(a[k], h, bb[k], (resets >> k) & 1);
            }
        }
        const __amdgpu_buffer_rsrc_t ox = gated_rsrc(dx.base + tr * dx.st), oi = gated_rsrc(di.base + tr * di.st),
                                     orr = gated_rsrc(dr.base + tr * dr.st);
        const uint32_t resets = again<RESET>(bits);
#pragma unroll
        for (int k = TS - 1; k >= 0; --k) {
            const bool put = live && (!TAIL || k < left), on = (resets >> k) & 1;
            const float gk = g[k] + in;
            in = step_mul<RESET>(a[k], gk, on);
            const float q = step_mul<RESET>(in * e[k], z[k], on);  // without its factor ln 2; 0 at a reset
            acc += !TAIL || k < left ? q : 0.0f;
            row_store(from_f32<S>(gk * ms[k]), ox, put ? dx.off : kGatedDrop, k * dx.row_bytes());
            row_store(from_f32<S>(gk * bi[k]), oi, put ? di.off : kGatedDrop, k * di.row_bytes());
            row_store(from_f32<S>(step_mul<RESET>(q, __builtin_fmaf(-e[k], inv_tl, kLn2), on)), orr, put ? dr.off : kGatedDrop,
                      k * dr.row_bytes());
        }
        s_acc[run * kPitch + lane] = acc * kLn2;
        sums_of = which;
        if (p.dh0 && walk.cur == n - 1 && s_run == 0 && s_live) p.dh0[b * D + ds] = carry;
        walk.advance();
    };
    if (walk.cur == 0 && L % STEPS) chunk(std::true_type{});
    while (walk.cur < n) chunk(std::false_type{});
    __syncthreads();
    flush();
}

}  // namespace mscan
