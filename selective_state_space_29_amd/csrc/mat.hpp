// Matrix products of bf16 operands on the matrix cores (gfx950), fp32 sums: C[p][q] = sum_c X(p, c) Y(q, c) for
// one tile a workgroup, with the epilogues of the operators that use it (the gated feed-forward block, the cross
// entropy over the vocabulary), and the choice of tiles. k_ffn.hip has the reasons of the layout.
#pragma once

#include <type_traits>

#include "layers_common.hpp"

namespace mscan {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr int kTC = 64;                       // contraction steps per stage
constexpr uint32_t kDrop = 0xFFFFFFF0u;       // a byte offset past every buffer: reads 0
constexpr int kRsrcWord3 = 0x00020000;

template <int N>
using Int = std::integral_constant<int, N>;

enum { kEpiDual = 0, kEpiDualBwd = 1, kEpiStore = 2, kEpiPartial = 3, kEpiLse = 4, kEpiDlogits = 5, kEpiAdd = 6 };

struct MatArgs {
    const uint16_t* x;      // X(p, c): [p][c], or [c][p] where XTR
    const uint16_t* y[2];   // Y(q, c); dual: gate and up rows; dx: the weights of the two stretches of c
    int64_t x_stride, y_stride;
    int64_t up_stride;      // few rows: of y[1], where it may differ
    int64_t P, Q;           // extents; dual: Q hidden units
    int64_t C;              // contraction length of a stretch
    int64_t x_cols;         // X not XTR: columns of a stretch that may be read (a multiple of 8)
    int64_t x_seg;          // X not XTR: columns from one stretch to the next
    int steps;              // stages per stretch
    int stretches, splits;
    int tiles_p, tiles_q;
    // epilogues
    uint16_t* out;          // h (P, Q); dx (P, Q); dW gate
    uint16_t* out2;         // dW up
    int64_t out_stride, seg_rows, seg_valid;  // dW: rows of P up to seg_rows are gate, seg_valid of them real
    const uint16_t* dh;     // (P, Q)
    int64_t dh_stride;
    uint16_t* d;            // (P, 2 seg_rows): dg, du; dlogits: (P, seg_rows)
    int add;                // add: the partial sums are added to what is there
    float* part;            // (splits, P, Q); lse: (tiles_q, P) pairs of a row's maximum and sum of a tile
    int act;
    const float* factor;    // or NULL: what the bf16 results are multiplied with before they are rounded
    // cross entropy: logits are scale C
    float scale;
    const void* target;     // lse: (P) int64 or int32, or NULL
    int target64;
    float* at_target;       // lse: (P), the target's logit where it is one of this product's columns
    const float* row;       // dlogits: (P) of {lse log2(e) rounded, factor of 2 to what is above it, factor of the target, target's bits}
    int64_t q_first;        // dlogits: the vocabulary's column that is column 0 here
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* base, int64_t bytes) {
    const int64_t n = bytes < 0 ? 0 : bytes < 0x7FFFFFF0 ? bytes : 0x7FFFFFF0;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)n, kRsrcWord3);
}
// 16 bytes a lane straight from memory into LDS: the wave's lanes fill 1 KB of consecutive places.
__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t r, uint16_t* to, uint32_t off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)to, 16, (int)off, 0, 0, 0);
}
// Waits until at most N of the wave's loads are on their way, then for the workgroup.
template <int N>
__device__ __forceinline__ void stage_ready() {
    static_assert(N < 64);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0x0f70 | (N & 15) | (N >> 4) << 14);  // vmcnt(N)
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// act and its derivative; silu(g) = g sg(g), gelu(g) = g/2 (1 + tanh(k (g + 0.044715 g^3))), where
// (1 + tanh(z)) / 2 = sg(2z).
__device__ __forceinline__ float act_of(float g, int act) {
    const float z = act == MAMBA_FFN_SILU ? g : 1.5957691216057308f * __builtin_fmaf(0.044715f * g * g, g, g);
    return g * hw_rcp(1.0f + hw_exp2(-z * kLog2e));
}
__device__ __forceinline__ void act_grad(float g, int act, float& a, float& da) {
    const float z = act == MAMBA_FFN_SILU ? g : 1.5957691216057308f * __builtin_fmaf(0.044715f * g * g, g, g);
    const float dz = act == MAMBA_FFN_SILU ? 1.0f : 1.5957691216057308f * __builtin_fmaf(3.0f * 0.044715f * g, g, 1.0f);
    const float s = hw_rcp(1.0f + hw_exp2(-z * kLog2e));
    a = g * s;
    // far out on the negative side the polynomial overflows while s is 0: the product is 0 there
    const float slope = s * (1.0f - s);
    da = s + (slope > 0.0f ? g * dz * slope : 0.0f);
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    return (uint32_t)to_bf16(lo).bits | (uint32_t)to_bf16(hi).bits << 16;
}
// The same in one instruction (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ float half_f32(uint32_t w, int k) { return __uint_as_float(k ? w & 0xFFFF0000u : w << 16); }

// Two pairs {maximum, sum of exponentials from it} as one. A maximum drops a NaN, but the sum keeps it.
__device__ __forceinline__ float2 join_pair(float2 a, float2 b) {
    const float top = __builtin_fmaxf(a.x, b.x);
    const float fa = a.x == top ? a.y : a.y * hw_exp2((a.x - top) * kLog2e), fb = b.x == top ? b.y : b.y * hw_exp2((b.x - top) * kLog2e);
    return make_float2(top, fa + fb);
}

// Where chunk `c` (8 values) of row `row` lies in its LDS row: rows of 64 c (8 chunks, 128 bytes), of which
// 16 lanes read the same chunk of 16 rows, or of T values of a c (tr), where the 8 rows that a half wave's
// transposing read touches take 8 distinct pairs of chunks.
__device__ __forceinline__ int swz(int row, int c) { return c ^ ((row >> 1) & 7); }
template <int T>
__device__ __forceinline__ int swz_tr(int row, int c) {
    if constexpr (T % 128 != 0) return c ^ (((row >> 1 & 1) | (row >> 2 & 2)) << 1);  // odd rows lie 128 bytes further
    return c ^ (((row & 3) | ((row >> 1) & 4)) << 1);
}

template <int TP, int TQ, int WP, int WQ, int DEPTH, bool XTR, bool YTR, int EPI>
__device__ __forceinline__ void mat_tile(const MatArgs& m) {
    constexpr bool DUAL = EPI == kEpiDual || EPI == kEpiDualBwd;
    constexpr int NT = WP * WQ * 64;
    constexpr int PT = TP / WP / 16, QT = TQ / WQ / 16, QG = QT % 4 == 0 ? 4 : 3;  // QG: tiles read at a time
    constexpr int CH = kTC / 8;  // chunks of a row of c
    constexpr int XN = TP * CH / NT, YN = TQ * CH / NT;  // chunks a thread moves per stage
    static_assert(!(DUAL && (XTR || YTR)) && XN >= 1 && YN >= 1 && (!DUAL || QT % 2 == 0));
    constexpr int OQ = DUAL ? TQ / 2 : TQ, PITCH = OQ + 8;  // of the results' rows in LDS, 16 bytes apart in the banks
    constexpr int STAGES = DEPTH * (TP + TQ) * kTC, RESULTS = EPI == kEpiPartial || EPI == kEpiAdd ? 0 : TP * PITCH + (EPI == kEpiDlogits ? TP * 8 : 0);
    __shared__ __align__(16) uint16_t lds[STAGES > RESULTS ? STAGES : RESULTS];
    uint16_t(&sx)[DEPTH][TP * kTC] = *reinterpret_cast<uint16_t(*)[DEPTH][TP * kTC]>(&lds[0]);
    uint16_t(&sy)[DEPTH][TQ * kTC] = *reinterpret_cast<uint16_t(*)[DEPTH][TQ * kTC]>(&lds[DEPTH * TP * kTC]);

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wp = wave / WQ, wq = wave % WQ;

    // Workgroups go to the 8 XCDs in turn: each takes one stretch of the tile order, in which blocks of
    // 8 tiles of p follow q, so that the tiles an XCD works on at a time share operand rows in its L2.
    const int ntiles = m.tiles_p * m.tiles_q;
    int tile = blockIdx.x;
    {
        const int q8 = ntiles / 8, r8 = ntiles % 8, xcd = tile % 8, slot = tile / 8;
        tile = xcd * q8 + (xcd < r8 ? xcd : r8) + slot;
    }
    const int band = tile / (8 * m.tiles_q), in = tile % (8 * m.tiles_q);
    const int rows = m.tiles_p - band * 8 < 8 ? m.tiles_p - band * 8 : 8;
    const int64_t p0 = (int64_t)(band * 8 + in % rows) * TP;
    const int64_t q0 = (int64_t)(in / rows) * (DUAL ? TQ / 2 : TQ);

    const int total = m.steps * m.stretches;
    const int per = (total + m.splits - 1) / m.splits;
    const int s_begin = (int)blockIdx.y * per, s_end = s_begin + per < total ? s_begin + per : total;

    // Each lane's chunks of a stage: 16 bytes straight into LDS, a wave's 64 lanes to 1 KB of consecutive
    // places, so a lane picks the chunk whose place it fills.
    int xr[XN], xc[XN], yr[YN], yc[YN];
#pragma unroll
    for (int k = 0; k < XN; ++k) {
        const int l = k * NT + tid;
        xr[k] = XTR ? l / (TP / 8) : l / CH;
        xc[k] = XTR ? swz_tr<TP>(xr[k], l % (TP / 8)) : swz(xr[k], l % CH);
    }
#pragma unroll
    for (int k = 0; k < YN; ++k) {
        const int l = k * NT + tid;
        yr[k] = YTR ? l / (TQ / 8) : l / CH;
        yc[k] = YTR ? swz_tr<TQ>(yr[k], l % (TQ / 8)) : swz(yr[k], l % CH);
    }
    auto fetch = [&](int step, int buf) __attribute__((always_inline)) {
        const int seg = step >= m.steps ? 1 : 0;
        const int64_t c0 = (int64_t)(step - seg * m.steps) * kTC;
        uint16_t* tx = &sx[buf][wave * 512];
        uint16_t* ty = &sy[buf][wave * 512];
        if constexpr (XTR) {  // rows c0 + row of X, columns p
            const __amdgpu_buffer_rsrc_t r = rsrc_of(m.x + c0 * m.x_stride + p0, ((m.C - c0 - 1) * m.x_stride + m.P - p0) * 2);
#pragma unroll
            for (int k = 0; k < XN; ++k) {
                const bool ok = c0 + xr[k] < m.C && p0 + xc[k] * 8 < m.P;
                load_lds(r, tx + k * NT * 8, ok ? (uint32_t)((xr[k] * (int)m.x_stride + xc[k] * 8) * 2) : kDrop);
            }
        } else {
            const int64_t col = seg * m.x_seg + c0;
            const __amdgpu_buffer_rsrc_t r = rsrc_of(m.x + p0 * m.x_stride + col, ((m.P - p0 - 1) * m.x_stride + m.x_cols - c0) * 2);
#pragma unroll
            for (int k = 0; k < XN; ++k) {
                const bool ok = p0 + xr[k] < m.P && c0 + xc[k] * 8 < m.x_cols;
                load_lds(r, tx + k * NT * 8, ok ? (uint32_t)((xr[k] * (int)m.x_stride + xc[k] * 8) * 2) : kDrop);
            }
        }
        if constexpr (YTR) {
            const uint16_t* y = seg ? m.y[1] : m.y[0];
            const __amdgpu_buffer_rsrc_t r = rsrc_of(y + c0 * m.y_stride + q0, ((m.C - c0 - 1) * m.y_stride + m.Q - q0 + 7) * 2);
#pragma unroll
            for (int k = 0; k < YN; ++k) {
                const bool ok = c0 + yr[k] < m.C && q0 + yc[k] * 8 < m.Q;
                load_lds(r, ty + k * NT * 8, ok ? (uint32_t)((yr[k] * (int)m.y_stride + yc[k] * 8) * 2) : kDrop);
            }
        } else {
            const int64_t bytes = ((m.Q - q0 - 1) * m.y_stride + m.C - c0) * 2;
            const __amdgpu_buffer_rsrc_t r0 = rsrc_of(m.y[0] + q0 * m.y_stride + c0, bytes);
            const __amdgpu_buffer_rsrc_t r1 = rsrc_of(m.y[1] + q0 * m.y_stride + c0, bytes);
#pragma unroll
            for (int k = 0; k < YN; ++k) {
                // dual: the first half of the tile's rows are gate rows, the second the same units' up rows
                const bool up = DUAL && k >= YN / 2;
                const int row = up ? yr[k] - TQ / 2 : yr[k];
                const bool ok = q0 + row < m.Q && c0 + yc[k] * 8 < m.C;
                load_lds(up ? r1 : r0, ty + k * NT * 8, ok ? (uint32_t)((row * (int)m.y_stride + yc[k] * 8) * 2) : kDrop);
            }
        }
    };

    // tile t (16 p's or q's) of a wave: where its rows begin in the workgroup's tile
    auto p_row = [&](int t) { return wp * (TP / WP) + t * 16; };
    auto q_row = [&](int t) {
        if constexpr (DUAL) return (t < QT / 2 ? 0 : TQ / 2) + wq * (TQ / WQ / 2) + (t % (QT / 2)) * 16;
        return wq * (TQ / WQ) + t * 16;
    };
    auto frag = [&](const uint16_t* s, int row0, int kk) __attribute__((always_inline)) {
        const int row = row0 + (lane & 15);
        return *reinterpret_cast<const bf16x8*>(&s[row * kTC + swz(row, kk * 4 + (lane >> 4)) * 8]);
    };
    // Transposing reads of N tiles of 16: the lane's address of a tile in the stage's first rows, the rows of
    // half kk of the stage and the second four of a lane's eight in the offset (the places' XOR depends on the
    // lane alone). Reads and their wait in one asm block: the compiler's own form of these reads waits for
    // every load that is on its way into LDS as well, here those of the next stage.
    auto tr_at = [&](auto width, int row0) {
        constexpr int T = decltype(width)::value;
        const int i = lane & 15, n = row0 + 4 * (i & 3), c = 8 * (lane >> 4) + (i >> 2);
        return (uint32_t)(c * T + swz_tr<T>(c, n >> 3) * 8 + (n & 7)) * 2;
    };
    auto frags_tr = [&](auto width, auto count, bf16x8* to, const uint32_t* at, const uint16_t* s, auto step) __attribute__((always_inline)) {
        constexpr int T = decltype(width)::value, N = decltype(count)::value, K0 = decltype(step)::value * 32 * T * 2, K1 = K0 + 4 * T * 2;
        const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)s;
        u32x2 r[2 * N];
        if constexpr (N == 4) {
            asm volatile(
                "ds_read_b64_tr_b16 %0, %8 offset:%12\n\tds_read_b64_tr_b16 %1, %8 offset:%13\n\t"
                "ds_read_b64_tr_b16 %2, %9 offset:%12\n\tds_read_b64_tr_b16 %3, %9 offset:%13\n\t"
                "ds_read_b64_tr_b16 %4, %10 offset:%12\n\tds_read_b64_tr_b16 %5, %10 offset:%13\n\t"
                "ds_read_b64_tr_b16 %6, %11 offset:%12\n\tds_read_b64_tr_b16 %7, %11 offset:%13\n\t"
                "s_waitcnt lgkmcnt(0)"
                : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3]), "=&v"(r[4]), "=&v"(r[5]), "=&v"(r[6]), "=&v"(r[7])
                : "v"(at[0] + base), "v"(at[1] + base), "v"(at[2] + base), "v"(at[3] + base), "n"(K0), "n"(K1)
                : "memory");
        } else {
            static_assert(N == 3);
            asm volatile(
                "ds_read_b64_tr_b16 %0, %6 offset:%9\n\tds_read_b64_tr_b16 %1, %6 offset:%10\n\t"
                "ds_read_b64_tr_b16 %2, %7 offset:%9\n\tds_read_b64_tr_b16 %3, %7 offset:%10\n\t"
                "ds_read_b64_tr_b16 %4, %8 offset:%9\n\tds_read_b64_tr_b16 %5, %8 offset:%10\n\t"
                "s_waitcnt lgkmcnt(0)"
                : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3]), "=&v"(r[4]), "=&v"(r[5])
                : "v"(at[0] + base), "v"(at[1] + base), "v"(at[2] + base), "n"(K0), "n"(K1)
                : "memory");
        }
#pragma unroll
        for (int k = 0; k < N; ++k) __builtin_memcpy(&to[k], &r[2 * k], 16);
    };
    uint32_t qa[QT], pa[PT];
#pragma unroll
    for (int q = 0; q < QT; ++q) qa[q] = YTR ? tr_at(Int<TQ>{}, q_row(q)) : 0;
#pragma unroll
    for (int p = 0; p < PT; ++p) pa[p] = XTR ? tr_at(Int<TP>{}, p_row(p)) : 0;

    f32x4 acc[QT][PT];
#pragma unroll
    for (int q = 0; q < QT; ++q)
#pragma unroll
        for (int p = 0; p < PT; ++p) acc[q][p] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // what the epilogue needs of each row of the tile, a row a thread, on its way while the stages run (loaded by
    // every lane behind them, the targets cost 5 us of a tile's 26)
    f32x4 of_row = {0.0f, 0.0f, 0.0f, 0.0f};
    int64_t target = -1;
    if constexpr (EPI == kEpiLse || EPI == kEpiDlogits) {
        const int64_t pr = p0 + tid % TP < m.P ? p0 + tid % TP : m.P - 1;
        if constexpr (EPI == kEpiDlogits) of_row = *reinterpret_cast<const f32x4*>(m.row + pr * 4);
        else if (m.target) target = m.target64 ? static_cast<const int64_t*>(m.target)[pr] : static_cast<const int32_t*>(m.target)[pr];
    }

    uint32_t warm = 0;
    if (s_begin < s_end) {
        constexpr int LOADS = XN + YN;  // a stage's
#pragma unroll
        for (int d = 0; d < DEPTH - 1; ++d)
            if (s_begin + d < s_end) fetch(s_begin + d, d);
        unsigned buf = 0;
        for (int s = s_begin; s < s_end; ++s, buf = (buf + 1) % DEPTH) {
            // this stage is in LDS, and every wave is done with the one before it
            if constexpr (DEPTH == 2) {
                __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
                __syncthreads();
            } else {
                static_assert(DEPTH == 4);
                if (s + 2 < s_end) stage_ready<2 * LOADS>();
                else if (s + 1 < s_end) stage_ready<LOADS>();
                else stage_ready<0>();
            }
            if (s + DEPTH - 1 < s_end) fetch(s + DEPTH - 1, (buf + DEPTH - 1) % DEPTH);
            // one load a cache line of dh's tile: the epilogue finds it in L2 (dg and du 162 us, 168 without)
            if (EPI == kEpiDualBwd && s == s_end - 2) {
                const int64_t pr = p0 + (tid >> 1) % TP, c = q0 + (tid & 1) * 64;
                warm = m.dh[(pr < m.P ? pr : m.P - 1) * m.dh_stride + (c < m.Q ? c : m.Q - 1)];
            }
            auto half = [&](auto step) __attribute__((always_inline)) {
                constexpr int kk = decltype(step)::value;
                bf16x8 a[QT], b[PT];
                if constexpr (YTR) {
#pragma unroll
                    for (int q = 0; q < QT; q += QG) frags_tr(Int<TQ>{}, Int<QG>{}, a + q, qa + q, sy[buf], step);
                } else {
#pragma unroll
                    for (int q = 0; q < QT; ++q) a[q] = frag(sy[buf], q_row(q), kk);
                }
                if constexpr (XTR) {
#pragma unroll
                    for (int p = 0; p < PT; p += 4) frags_tr(Int<TP>{}, Int<4>{}, b + p, pa + p, sx[buf], step);
                } else {
#pragma unroll
                    for (int p = 0; p < PT; ++p) b[p] = frag(sx[buf], p_row(p), kk);
                }
#pragma unroll
                for (int q = 0; q < QT; ++q)
#pragma unroll
                    for (int p = 0; p < PT; ++p)
                        acc[q][p] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[q], b[p], acc[q][p], 0, 0, 0);
            };
            half(Int<0>{});
            half(Int<1>{});
        }
    }

    asm volatile("" ::"v"(warm));
    // A lane holds q = q0 + q_row(t) + 4 (lane / 16) .. + 3 of p = p0 + p_row(t) + lane % 16.
    const int lq = 4 * (lane >> 4), lp = lane & 15;
    if constexpr (EPI == kEpiLse) {
        // Maximum and sum of exponentials of the tile's columns, of each row: first in each of the 4 WQ lanes that hold a
        // part of the row, then over them. The maximum stays a logit and is subtracted before the exponential's factor, so
        // that the largest term is 1 and a loss at the maximum has its own digits. With an infinite maximum the
        // exponentials are taken as they are: a sum of zeros, infinity or NaN is then the row's. (Of a tile's 26 us at dim
        // 768 this takes about 3, VALU instructions, a third of them the exponentials; with the lanes joined by shuffles it
        // took 5. In base 2, with the maximum subtracted in the exponential's own product, it took 0.4 less.)
        constexpr int PARTS = 4 * WQ;
        float2(*sums)[TP] = reinterpret_cast<float2(*)[TP]>(&lds[0]);
        int* rel_of = reinterpret_cast<int*>(&sums[PARTS][0]);  // each row's target as a column of this tile, or -1
        static_assert(PARTS * TP * 8 + TP * 4 <= STAGES * 2 && NT >= TP);
        const bool whole = q0 + TQ <= m.Q;
        if (m.scale != 1.0f) {
#pragma unroll
            for (int q = 0; q < QT; ++q)
#pragma unroll
                for (int p = 0; p < PT; ++p) acc[q][p] *= m.scale;
        }
        __syncthreads();  // every wave has read its last fragments
        if (tid < TP) rel_of[tid] = target >= q0 && target < q0 + TQ && target < m.Q && p0 + tid < m.P ? (int)(target - q0) : -1;
        __syncthreads();
        int rel[PT];
#pragma unroll
        for (int p = 0; p < PT; ++p) rel[p] = rel_of[p_row(p) + lp];
#pragma unroll
        for (int p = 0; p < PT; ++p) {
            if (rel[p] >= 0) {
#pragma unroll
                for (int q = 0; q < QT; ++q)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (q_row(q) + lq + j == rel[p]) m.at_target[p0 + p_row(p) + lp] = acc[q][p][j];
            }
            if (!whole) {
#pragma unroll
                for (int q = 0; q < QT; ++q)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[q][p][j] = q0 + q_row(q) + lq + j < m.Q ? acc[q][p][j] : -__builtin_inff();
            }
            float top = acc[0][p][0];
#pragma unroll
            for (int q = 0; q < QT; ++q)
#pragma unroll
                for (int j = 0; j < 4; ++j) top = __builtin_fmaxf(top, acc[q][p][j]);
            const float base = __builtin_fabsf(top) == __builtin_inff() ? 0.0f : top;
            float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int q = 0; q < QT; ++q)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[j] += hw_exp2((acc[q][p][j] - base) * kLog2e);
            sums[wq * 4 + (lane >> 4)][p_row(p) + lp] = make_float2(top, (s[0] + s[1]) + (s[2] + s[3]));
        }
        __syncthreads();
        if (tid < TP && p0 + tid < m.P) {
            float2 r[PARTS];
            float top = -__builtin_inff(), s = 0.0f;
#pragma unroll
            for (int k = 0; k < PARTS; ++k) r[k] = sums[k][tid], top = __builtin_fmaxf(top, r[k].x);
#pragma unroll
            for (int k = 0; k < PARTS; ++k) s += r[k].x == top ? r[k].y : r[k].y * hw_exp2((r[k].x - top) * kLog2e);
            reinterpret_cast<float2*>(m.part)[q0 / TQ * m.P + p0 + tid] = make_float2(top, s);
        }
    } else if constexpr (EPI == kEpiPartial || EPI == kEpiAdd) {
#pragma unroll
        for (int p = 0; p < PT; ++p) {
            const int64_t pr = p0 + p_row(p) + lp;
            if (pr >= m.P) continue;
#pragma unroll
            for (int q = 0; q < QT; ++q) {
                const int64_t qc = q0 + q_row(q) + lq;
                if (qc >= m.Q) continue;
                float* o = m.part + ((int64_t)blockIdx.y * m.P + pr) * m.Q + qc;
                if (EPI == kEpiAdd && m.add) {
                    if (m.Q % 4 == 0) {
                        acc[q][p] += *reinterpret_cast<const f32x4*>(o);
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (qc + j < m.Q) acc[q][p][j] += o[j];
                    }
                }
                if (m.Q % 4 == 0) {
                    *reinterpret_cast<f32x4*>(o) = acc[q][p];
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (qc + j < m.Q) o[j] = acc[q][p][j];
                }
            }
        }
    } else {
        // The bf16 results pass through LDS, so that rows are moved 16 bytes a lane.
        constexpr int OC = OQ / 8;  // chunks a row
        uint16_t* stage = &lds[0];
        auto place = [&](int t, int p) { return &stage[(p_row(p) + lp) * PITCH + q_row(t) + lq]; };
        // rows of the tile to or from memory, in chunks; f(row of the tile, first column, pointer into stage)
        auto rows = [&](int64_t end, auto&& f) __attribute__((always_inline)) {
            for (int k = tid; k < TP * OC; k += NT) {
                const int r = k / OC, c = k % OC * 8;
                if (p0 + r < m.P && q0 + c < end) f(p0 + r, q0 + c, &stage[r * PITCH + c]);
            }
        };
        auto store_row = [&](uint16_t* o, int64_t col, int64_t end, const uint16_t* s) __attribute__((always_inline)) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(s);
            if (col + 8 <= end && (reinterpret_cast<uintptr_t>(o) & 15) == 0) {
                *reinterpret_cast<u32x4*>(o) = v;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (col + j < end) o[j] = (uint16_t)(v[j / 2] >> (16 * (j & 1)));
            }
        };
        __syncthreads();  // every wave has read its last fragments
        if constexpr (EPI == kEpiDualBwd) {
            // zeros in units past Q, up to the padded width that is written
            rows(m.seg_rows, [&](int64_t pr, int64_t f, uint16_t* s) {
                const uint16_t* dh = m.dh + pr * m.dh_stride + f;
                u32x4 v = {0u, 0u, 0u, 0u};
                if (f + 8 <= m.Q && (reinterpret_cast<uintptr_t>(dh) & 15) == 0) {
                    v = *reinterpret_cast<const u32x4*>(dh);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (f + j < m.Q) v[j / 2] |= (uint32_t)dh[j] << (16 * (j & 1));
                }
                *reinterpret_cast<u32x4*>(s) = v;
            });
            __syncthreads();
            // dg overwrites dh in place; du follows after the rows of dg are out
            uint2 du[QT / 2][PT];
#pragma unroll
            for (int p = 0; p < PT; ++p)
#pragma unroll
                for (int q = 0; q < QT / 2; ++q) {
                    uint16_t* s = place(q, p);
                    const uint2 w = *reinterpret_cast<const uint2*>(s);
                    const float dv[4] = {half_f32(w.x, 0), half_f32(w.x, 1), half_f32(w.y, 0), half_f32(w.y, 1)};
                    float dg[4], dd[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float a, da;
                        act_grad(acc[q][p][j], m.act, a, da);
                        dg[j] = dv[j] * acc[q + QT / 2][p][j] * da;
                        dd[j] = dv[j] * a;
                    }
                    *reinterpret_cast<uint2*>(s) = make_uint2(pack2(dg[0], dg[1]), pack2(dg[2], dg[3]));
                    du[q][p] = make_uint2(pack2(dd[0], dd[1]), pack2(dd[2], dd[3]));
                }
            auto out = [&](int64_t shift) __attribute__((always_inline)) {
                __syncthreads();
                rows(m.seg_rows, [&](int64_t pr, int64_t f, const uint16_t* s) {
                    *reinterpret_cast<u32x4*>(m.d + pr * 2 * m.seg_rows + shift + f) = *reinterpret_cast<const u32x4*>(s);
                });
            };
            out(0);
            __syncthreads();
#pragma unroll
            for (int p = 0; p < PT; ++p)
#pragma unroll
                for (int q = 0; q < QT / 2; ++q) *reinterpret_cast<uint2*>(place(q, p)) = du[q][p];
            out(m.seg_rows);
        } else {
            if constexpr (EPI == kEpiDlogits) {
                // (factor softmax - [target] factor) rounded; a row whose factors are 0 takes no part, whatever its
                // logits. Columns past Q, up to the padded width that is written, are zeros. The target is seen to
                // apart, as hardly any lane holds one (a piece of 7168 columns and 16384 rows, the target and the
                // last column tested at every value 215 us, so 204). The factor makes up for the rounding of lse log2(e), so
                // that a softmax of 1 is 1 to its last bits and leaves nothing behind when the target is taken from it.
                if (m.scale != 1.0f) {  // the forward's logits, rounded as there
#pragma unroll
                    for (int q = 0; q < QT; ++q)
#pragma unroll
                        for (int p = 0; p < PT; ++p) acc[q][p] *= m.scale;
                }
                const bool whole = q0 + TQ <= m.Q;
                static_assert(TP * 16 + TP * PITCH * 2 <= (STAGES > RESULTS ? STAGES : RESULTS) * 2);
                f32x4* rows_of = reinterpret_cast<f32x4*>(&lds[TP * PITCH]);
                if (tid < TP) rows_of[tid] = of_row;
                __syncthreads();
#pragma unroll
                for (int p = 0; p < PT; ++p) {
                    const f32x4 row = rows_of[p_row(p) + lp];
                    const bool on = row[1] != 0.0f || row[2] != 0.0f;
                    const int64_t rel = (int64_t)__float_as_int(row[3]) - m.q_first - q0;
#pragma unroll
                    for (int q = 0; q < QT; ++q)
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[q][p][j] = hw_exp2(__builtin_fmaf(acc[q][p][j], kLog2e, -row[0]));
                    // (apart from the products: an exponential's result may not be used by the next instruction)
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int q = 0; q < QT; ++q) acc[q][p] *= row[1];
                    if (rel >= 0 && rel < TQ) {
#pragma unroll
                        for (int q = 0; q < QT; ++q)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (q_row(q) + lq + j == (int)rel) acc[q][p][j] -= row[2];
                    }
                    if (!whole) {
#pragma unroll
                        for (int q = 0; q < QT; ++q)
#pragma unroll
                            for (int j = 0; j < 4; ++j) acc[q][p][j] = q0 + q_row(q) + lq + j < m.Q ? acc[q][p][j] : 0.0f;
                    }
#pragma unroll
                    for (int q = 0; q < QT; ++q) {
                        const uint32_t lo = pack_pair(acc[q][p][0], acc[q][p][1]), hi = pack_pair(acc[q][p][2], acc[q][p][3]);
                        *reinterpret_cast<uint2*>(place(q, p)) = make_uint2(on ? lo : 0u, on ? hi : 0u);
                    }
                }
                __syncthreads();
                rows(m.seg_rows, [&](int64_t pr, int64_t qc, const uint16_t* s) {
                    *reinterpret_cast<u32x4*>(m.d + pr * m.seg_rows + qc) = *reinterpret_cast<const u32x4*>(s);
                });
                return;
            }
            if constexpr (EPI == kEpiStore) {
                if (m.factor) {
                    const float by = *m.factor;
#pragma unroll
                    for (int q = 0; q < QT; ++q)
#pragma unroll
                        for (int p = 0; p < PT; ++p) acc[q][p] *= by;
                }
            }
#pragma unroll
            for (int p = 0; p < PT; ++p)
#pragma unroll
                for (int q = 0; q < (DUAL ? QT / 2 : QT); ++q) {
                    float h[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        h[j] = DUAL ? act_of(acc[q][p][j], m.act) * acc[q + (DUAL ? QT / 2 : 0)][p][j] : acc[q][p][j];
                    *reinterpret_cast<uint2*>(place(q, p)) = make_uint2(pack2(h[0], h[1]), pack2(h[2], h[3]));
                }
            __syncthreads();
            rows(m.Q, [&](int64_t pr, int64_t qc, const uint16_t* s) {
                if constexpr (DUAL) {
                    store_row(m.out + pr * m.out_stride + qc, qc, m.Q, s);
                } else {
                    const int64_t row = pr < m.seg_rows ? pr : pr - m.seg_rows;
                    if (row < m.seg_valid) store_row((pr < m.seg_rows ? m.out : m.out2) + row * m.out_stride + qc, qc, m.Q, s);
                }
            });
        }
    }
}

// The splits' partial sums of a product, added in order: V columns a lane, V = 4 where Q is a multiple of it.
template <int V>
__global__ __launch_bounds__(256) void mat_join_kernel(MatArgs m) {
    const int64_t n = m.P * m.Q, cols = m.Q / V;
    typedef float vec __attribute__((ext_vector_type(V)));
    const vec* part = reinterpret_cast<const vec*>(m.part);
    const float by = m.factor ? *m.factor : 1.0f;
    for (int64_t pr = blockIdx.x; pr < m.P; pr += gridDim.x) {
        const int64_t row = pr < m.seg_rows ? pr : pr - m.seg_rows;
        if (row >= m.seg_valid) continue;
        uint16_t* out = (pr < m.seg_rows ? m.out : m.out2) + row * m.out_stride;
        for (int64_t c = threadIdx.x; c < cols; c += 256) {
            vec s = 0.0f;
#pragma unroll 4
            for (int q = 0; q < m.splits; ++q) s += part[q * (n / V) + pr * cols + c];
            s *= by;
            if constexpr (V == 4) {
                const uint2 w = make_uint2(pack2(s[0], s[1]), pack2(s[2], s[3]));
                __builtin_memcpy(out + c * 4, &w, 8);
            } else {
                out[c] = to_bf16(s[0]).bits;
            }
        }
    }
}

// Rows copied to a padded, aligned matrix of `wide` columns, zeros past `cols`.
struct MatCopy {
    const uint16_t* src[3];
    uint16_t* dst[3];
    int64_t rows[3], stride[3], cols, wide;
};
__global__ __launch_bounds__(256) void mat_copy_kernel(MatCopy m) {
    const int which = blockIdx.y;
    if (!m.src[which]) return;
    // a wave a row
    for (int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); r < m.rows[which]; r += (int64_t)gridDim.x * 4) {
        const uint16_t* src = m.src[which] + r * m.stride[which];
        uint16_t* dst = m.dst[which] + r * m.wide;
        // 8 values a lane, the loads without a branch around them
        for (int64_t c = (int64_t)(threadIdx.x & 63) * 8; c < m.wide; c += 64 * 8) {
            uint16_t v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = src[c + j < m.cols ? c + j : m.cols - 1];
            u32x4 w;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = (uint32_t)(c + 2 * j < m.cols ? v[2 * j] : 0) | (uint32_t)(c + 2 * j + 1 < m.cols ? v[2 * j + 1] : 0) << 16;
            *reinterpret_cast<u32x4*>(dst + c) = w;
        }
    }
}

// ---- plans ----

bool row_aligned(const void* p, int64_t stride, int64_t rows) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows <= 1 || stride % 8 == 0);
}

struct Tiling {
    int tp, tq;  // 256 x 256, 256 x 192 or 128 x 128
    bool alone;  // no more workgroups than CUs
    int tiles_p, tiles_q, splits;
};

// The tile and the split of the contraction whose rounds over the GPU's CUs take least. A stage of a tile
// takes its area over the tile's rate (measured against the largest: dx of 16384 x 768 from 4096, 64 x 3
// tiles of 256 x 256 in 119 us, 64 x 4 of 256 x 192 in 102; 128 x 128 forward 138 us against 119); two
// workgroups of the smallest share a CU, where one alone takes kAlone of a pair's rounds. Splits add their
// partial sums' way through memory and the kernel that joins them. Forward and backward together, always
// 256 x 256, always 128 x 128 and this rule: 512 rows, dim 768, hidden 2048: 115, 61, 60 us; 2048 rows: 139,
// 104, 100; 8192 rows, dim 1536, hidden 4096: 814, 923, 790.
Tiling tiling(int64_t P, int64_t Q, bool dual, int steps, bool may_split) {
    const int64_t cus = layers_cus();
    auto div = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    constexpr int kTiles[3][3] = {{256, 256, 100}, {256, 192, 88}, {128, 128, 80}};
    constexpr double kStage = 2.4e-6 * 100 / (256 * 256), kAlone = 1.4, kJoinBytes = 8.0 / 5e12, kJoin = 4e-6;
    Tiling best{};
    double least = 0.0;
    for (const auto& k : kTiles) {
        if (dual && k[1] == 192) continue;
        Tiling t{k[0], k[1], false, (int)div(P, k[0]), (int)div(Q, dual ? k[1] / 2 : k[1]), 1};
        const int64_t n = (int64_t)t.tiles_p * t.tiles_q, room = k[0] == 128 ? 2 * cus : cus;
        const int most = may_split ? (int)(room / n < steps / 4 ? room / n : steps / 4) : 1;
        for (int s = 1; s == 1 || s <= most; ++s) {
            const int64_t wgs = n * s;
            double rounds = k[0] == 128 && wgs <= cus ? kAlone : (double)div(wgs, cus);
            double cost = rounds * div(steps, s) * k[0] * k[1] / k[2] * kStage;
            if (s > 1) cost += kJoin + kJoinBytes * s * (double)P * Q;
            if (best.tp == 0 || cost < least) t.splits = s, t.alone = wgs <= cus, best = t, least = cost;
        }
    }
    return best;
}

int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }
int steps_of(int64_t c) { return (int)((c + kTC - 1) / kTC); }

}  // namespace

}  // namespace mscan
