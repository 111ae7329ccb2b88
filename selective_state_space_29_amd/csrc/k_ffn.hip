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
#include <type_traits>

#include "layers_common.hpp"
#include "layers_launch.hpp"

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

enum { kEpiDual = 0, kEpiDualBwd = 1, kEpiStore = 2, kEpiPartial = 3 };

struct FfnMat {
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
    uint16_t* d;            // (P, 2 seg_rows): dg, du
    float* part;            // (splits, P, Q)
    int act;
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
__device__ __forceinline__ float half_f32(uint32_t w, int k) { return __uint_as_float(k ? w & 0xFFFF0000u : w << 16); }

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
__global__ __launch_bounds__(WP * WQ * 64) __attribute__((amdgpu_waves_per_eu(DEPTH > 2 ? 1 : 2))) void ffn_mat_kernel(FfnMat m) {
    constexpr bool DUAL = EPI == kEpiDual || EPI == kEpiDualBwd;
    constexpr int NT = WP * WQ * 64;
    constexpr int PT = TP / WP / 16, QT = TQ / WQ / 16, QG = QT % 4 == 0 ? 4 : 3;  // QG: tiles read at a time
    constexpr int CH = kTC / 8;  // chunks of a row of c
    constexpr int XN = TP * CH / NT, YN = TQ * CH / NT;  // chunks a thread moves per stage
    static_assert(!(DUAL && (XTR || YTR)) && XN >= 1 && YN >= 1 && (!DUAL || QT % 2 == 0));
    constexpr int OQ = DUAL ? TQ / 2 : TQ, PITCH = OQ + 8;  // of the results' rows in LDS, 16 bytes apart in the banks
    constexpr int STAGES = DEPTH * (TP + TQ) * kTC, RESULTS = EPI == kEpiPartial ? 0 : TP * PITCH;
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
    if constexpr (EPI == kEpiPartial) {
#pragma unroll
        for (int p = 0; p < PT; ++p) {
            const int64_t pr = p0 + p_row(p) + lp;
            if (pr >= m.P) continue;
#pragma unroll
            for (int q = 0; q < QT; ++q) {
                const int64_t qc = q0 + q_row(q) + lq;
                if (qc >= m.Q) continue;
                float* o = m.part + ((int64_t)blockIdx.y * m.P + pr) * m.Q + qc;
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
__global__ __launch_bounds__(kFewWaves * 64) void ffn_few_kernel(FfnMat m) {
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

// The splits' partial sums of a product, added in order: V columns a lane, V = 4 where Q is a multiple of it.
template <int V>
__global__ __launch_bounds__(256) void ffn_join_kernel(FfnMat m) {
    const int64_t n = m.P * m.Q, cols = m.Q / V;
    typedef float vec __attribute__((ext_vector_type(V)));
    const vec* part = reinterpret_cast<const vec*>(m.part);
    for (int64_t pr = blockIdx.x; pr < m.P; pr += gridDim.x) {
        const int64_t row = pr < m.seg_rows ? pr : pr - m.seg_rows;
        if (row >= m.seg_valid) continue;
        uint16_t* out = (pr < m.seg_rows ? m.out : m.out2) + row * m.out_stride;
        for (int64_t c = threadIdx.x; c < cols; c += 256) {
            vec s = 0.0f;
#pragma unroll 4
            for (int q = 0; q < m.splits; ++q) s += part[q * (n / V) + pr * cols + c];
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
struct FfnCopy {
    const uint16_t* src[3];
    uint16_t* dst[3];
    int64_t rows[3], stride[3], cols, wide;
};
__global__ __launch_bounds__(256) void ffn_copy_kernel(FfnCopy m) {
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

// Zeros: the results of products over nothing.
__global__ __launch_bounds__(256) void ffn_zero_kernel(uint16_t* p, int64_t n, int64_t cols, int64_t stride) {
    for (int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x; k < n; k += (int64_t)gridDim.x * 256)
        p[k / cols * stride + k % cols] = 0;
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

template <bool XTR, bool YTR, int EPI>
void run_mat(FfnMat m, const Tiling& t, Launches& on) {
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
void run_product(const FfnMat& m, const Tiling& t, Launches& on) {
    if (t.splits == 1) {
        run_mat<XTR, YTR, kEpiStore>(m, t, on);
        return;
    }
    run_mat<XTR, YTR, kEpiPartial>(m, t, on);
    FfnMat j = m;
    j.splits = t.splits;
    const dim3 grid((unsigned)(m.P < 16384 ? m.P : 16384));
    if (m.Q % 4 == 0) on(ffn_join_kernel<4>, grid, dim3(256), j);
    else on(ffn_join_kernel<1>, grid, dim3(256), j);
}

int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }
int steps_of(int64_t c) { return (int)((c + kTC - 1) / kTC); }

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
    FfnCopy c{};
    c.cols = s.dim, c.wide = up(s.dim, 8);
    uint16_t* to = reinterpret_cast<uint16_t*>(ws);
    const int64_t xb = align256(s.rows * c.wide * 2) / 2, wb = align256(s.hidden * c.wide * 2) / 2;
    c.src[0] = o.x, c.dst[0] = to, c.rows[0] = s.rows, c.stride[0] = xs;
    c.src[1] = o.wg, c.dst[1] = to + xb, c.rows[1] = s.hidden, c.stride[1] = gs;
    c.src[2] = o.wu, c.dst[2] = to + xb + wb, c.rows[2] = s.hidden, c.stride[2] = us;
    const int64_t n = s.rows > s.hidden ? s.rows : s.hidden;
    on(ffn_copy_kernel, dim3((unsigned)(n < 32768 ? (n + 3) / 4 : 8192), 3), dim3(256), c);
    o.x = c.dst[0], o.wg = c.dst[1], o.wu = c.dst[2], o.xs = o.ws = o.dim8 = c.wide;
    return o;
}

FfnMat dual_mat(const mamba_ffn_shape& s, const Operands& o, int act) {
    FfnMat m{};
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
        FfnMat m{};
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
    FfnMat m = dual_mat(s, o, act);
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
    FfnMat m = dual_mat(s, o, act);
    m.dh = static_cast<const uint16_t*>(p.dh), m.dh_stride = p.dh_stride, m.d = d, m.seg_rows = b.fp;
    run_mat<false, false, kEpiDualBwd>(m, b.dual, on);

    FfnMat x{};  // dx[p][q] = sum over gate and up units c of d[p][c] W[c][q]
    x.x = d, x.x_stride = 2 * b.fp, x.x_cols = b.fp, x.x_seg = b.fp;
    x.y[0] = o.wg, x.y[1] = o.wu, x.y_stride = o.ws;
    x.P = s.rows, x.Q = s.dim, x.C = s.hidden;
    x.steps = steps_of(s.hidden), x.stretches = 2;
    x.out = x.out2 = static_cast<uint16_t*>(p.dx), x.out_stride = s.dim, x.seg_rows = x.seg_valid = s.rows;
    x.part = reinterpret_cast<float*>(ws + b.part);
    run_product<false, true>(x, b.dx, on);

    FfnMat w{};  // dW[f][q] = sum over tokens c of d[c][f] x[c][q]
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
