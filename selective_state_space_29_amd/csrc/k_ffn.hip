// Gated feed-forward block up to its product (mamba_layers.h) and its gradient on gfx950, bf16.
//
//   h = act(g) u,  g = x Wg^T, u = x Wu^T          dg = dh u act'(g), du = dh act(g)
//   dx = dg Wg + du Wu;   dWg = dg^T x;   dWu = du^T x
//
// One matrix kernel, C[p][q] = sum_c X(p, c) Y(q, c), serves all products. A workgroup computes a TP x TQ
// tile: it moves 64 steps of c of both operands through LDS a stage ahead of the one its waves multiply
// (v_mfma_f32_16x16x32_bf16, fp32 sums). An operand lies with c contiguous (x and the weights in the
// forward product) or with c as its rows (the weights in dx; both operands in dW); the latter is read
// from LDS with the transposing ds_read_b64_tr_b16, so no operand is ever transposed in memory. 16-byte
// chunks are placed in LDS at an index XORed with their row, so that the reads of both kinds meet no bank
// twice. The rows of the MFMA are the q's: a lane then holds 4 consecutive q of one p, stored as one
// 8-byte access.
//
// The forward tile holds 64 or 128 hidden units' gate rows and the same units' up rows, so that both
// projections of a unit meet in the same lane and only h is written. The backward pass recomputes g and
// u the same way (keeping them in fp32 would move more bytes than the product takes) and rounds dg and
// du to bf16 once, as the operands of the other two products.
//
// Operands whose rows are not 16-byte aligned or not a multiple of 8 long are first copied into padded
// rows of the workspace.
#include "layers_common.hpp"
#include "layers_launch.hpp"

namespace mscan {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr int kTC = 64;                       // contraction steps per stage
constexpr uint32_t kDrop = 0xFFFFFFF0u;       // a byte offset past every buffer: reads 0
constexpr int kRsrcWord3 = 0x00020000;

enum { kEpiDual = 0, kEpiDualBwd = 1, kEpiStore = 2, kEpiPartial = 3 };

struct FfnMat {
    const uint16_t* x;      // X(p, c): [p][c], or [c][p] where XTR
    const uint16_t* y[2];   // Y(q, c); dual: gate and up rows; dx: the weights of the two stretches of c
    int64_t x_stride, y_stride;
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
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0);
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

// Where chunk `c` (8 values) of row `row` lies in its LDS row: rows of 64 c (8 chunks of 128 bytes), or of
// T values of a c (tr), where the 8 rows that a half wave's transposing read touches take 8 distinct pairs.
__device__ __forceinline__ int swz(int row, int c) { return c ^ (row & 7); }
__device__ __forceinline__ int swz_tr(int row, int c) { return c ^ (((row & 3) | ((row >> 1) & 4)) << 1); }

template <int TP, int TQ, int WP, int WQ, bool XTR, bool YTR, int EPI>
__global__ __launch_bounds__(WP * WQ * 64) void ffn_mat_kernel(FfnMat m) {
    constexpr bool DUAL = EPI == kEpiDual || EPI == kEpiDualBwd;
    constexpr int NT = WP * WQ * 64;
    constexpr int PT = TP / WP / 16, QT = TQ / WQ / 16;
    constexpr int XN = TP * 8 / NT, YN = TQ * 8 / NT;  // chunks a thread moves per stage
    static_assert(!(DUAL && (XTR || YTR)) && XN >= 1 && YN >= 1 && (!DUAL || QT % 2 == 0));
    __shared__ __align__(16) uint16_t sx[2][TP * kTC];
    __shared__ __align__(16) uint16_t sy[2][TQ * kTC];

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

    // this thread's chunks: its row and chunk in the tile, and their LDS place
    int xr[XN], xc[XN], xl[XN], yr[YN], yc[YN], yl[YN];
#pragma unroll
    for (int k = 0; k < XN; ++k) {
        const int l = k * NT + tid;
        xr[k] = XTR ? l / (TP / 8) : l / 8;
        xc[k] = XTR ? l % (TP / 8) : l % 8;
        xl[k] = XTR ? xr[k] * TP + swz_tr(xr[k], xc[k]) * 8 : xr[k] * kTC + swz(xr[k], xc[k]) * 8;
    }
#pragma unroll
    for (int k = 0; k < YN; ++k) {
        const int l = k * NT + tid;
        yr[k] = YTR ? l / (TQ / 8) : l / 8;
        yc[k] = YTR ? l % (TQ / 8) : l % 8;
        yl[k] = YTR ? yr[k] * TQ + swz_tr(yr[k], yc[k]) * 8 : yr[k] * kTC + swz(yr[k], yc[k]) * 8;
    }

    u32x4 vx[XN], vy[YN];
    auto fetch = [&](int step) __attribute__((always_inline)) {
        const int seg = step >= m.steps ? 1 : 0;
        const int64_t c0 = (int64_t)(step - seg * m.steps) * kTC;
        if constexpr (XTR) {  // rows c0 + row of X, columns p
            const __amdgpu_buffer_rsrc_t r = rsrc_of(m.x + c0 * m.x_stride + p0, ((m.C - c0 - 1) * m.x_stride + m.P - p0) * 2);
#pragma unroll
            for (int k = 0; k < XN; ++k) {
                const bool ok = c0 + xr[k] < m.C && p0 + xc[k] * 8 < m.P;
                vx[k] = load16(r, ok ? (uint32_t)((xr[k] * (int)m.x_stride + xc[k] * 8) * 2) : kDrop);
            }
        } else {
            const int64_t col = seg * m.x_seg + c0;
            const __amdgpu_buffer_rsrc_t r = rsrc_of(m.x + p0 * m.x_stride + col, ((m.P - p0 - 1) * m.x_stride + m.x_cols - c0) * 2);
#pragma unroll
            for (int k = 0; k < XN; ++k) {
                const bool ok = p0 + xr[k] < m.P && c0 + xc[k] * 8 < m.x_cols;
                vx[k] = load16(r, ok ? (uint32_t)((xr[k] * (int)m.x_stride + xc[k] * 8) * 2) : kDrop);
            }
        }
        if constexpr (YTR) {
            const uint16_t* y = seg ? m.y[1] : m.y[0];
            const __amdgpu_buffer_rsrc_t r = rsrc_of(y + c0 * m.y_stride + q0, ((m.C - c0 - 1) * m.y_stride + m.Q - q0 + 7) * 2);
#pragma unroll
            for (int k = 0; k < YN; ++k) {
                const bool ok = c0 + yr[k] < m.C && q0 + yc[k] * 8 < m.Q;
                vy[k] = load16(r, ok ? (uint32_t)((yr[k] * (int)m.y_stride + yc[k] * 8) * 2) : kDrop);
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
                vy[k] = load16(up ? r1 : r0, ok ? (uint32_t)((row * (int)m.y_stride + yc[k] * 8) * 2) : kDrop);
            }
        }
    };
    auto put = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < XN; ++k) *reinterpret_cast<u32x4*>(&sx[buf][xl[k]]) = vx[k];
#pragma unroll
        for (int k = 0; k < YN; ++k) *reinterpret_cast<u32x4*>(&sy[buf][yl[k]]) = vy[k];
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
    auto frag_tr = [&](const uint16_t* s, int T, int row0, int kk) __attribute__((always_inline)) {
        const int i = lane & 15, n = row0 + 4 * (i & 3);
        s16x4 v[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = kk * 32 + 8 * (lane >> 4) + 4 * h + (i >> 2);
            const uint16_t* a = &s[c * T + swz_tr(c, n >> 3) * 8 + (n & 7)];
            v[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)a);
        }
        bf16x8 r;
        __builtin_memcpy(&r, v, 16);
        return r;
    };

    f32x4 acc[QT][PT];
#pragma unroll
    for (int q = 0; q < QT; ++q)
#pragma unroll
        for (int p = 0; p < PT; ++p) acc[q][p] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    if (s_begin < s_end) {
        fetch(s_begin);
        put(0);
        __syncthreads();
        int buf = 0;
        for (int s = s_begin; s < s_end; ++s, buf ^= 1) {
            if (s + 1 < s_end) fetch(s + 1);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                bf16x8 a[QT], b[PT];
#pragma unroll
                for (int q = 0; q < QT; ++q) a[q] = YTR ? frag_tr(sy[buf], TQ, q_row(q), kk) : frag(sy[buf], q_row(q), kk);
#pragma unroll
                for (int p = 0; p < PT; ++p) b[p] = XTR ? frag_tr(sx[buf], TP, p_row(p), kk) : frag(sx[buf], p_row(p), kk);
#pragma unroll
                for (int q = 0; q < QT; ++q)
#pragma unroll
                    for (int p = 0; p < PT; ++p)
                        acc[q][p] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[q], b[p], acc[q][p], 0, 0, 0);
            }
            if (s + 1 < s_end) put(buf ^ 1);  // last read a stage ago, before the barrier below
            __syncthreads();
        }
    }

    // lane: q = q0 + q_row(t) + 4 (lane / 16) .. + 3 of p = p0 + p_row(t) + lane % 16
    const int lq = 4 * (lane >> 4), lp = lane & 15;
#pragma unroll
    for (int p = 0; p < PT; ++p) {
        const int64_t pr = p0 + p_row(p) + lp;
        if (pr >= m.P) continue;
        if constexpr (DUAL) {
#pragma unroll
            for (int q = 0; q < QT / 2; ++q) {
                const int64_t f = q0 + q_row(q) + lq;
                const f32x4 g = acc[q][p], u = acc[q + QT / 2][p];
                if constexpr (EPI == kEpiDual) {
                    uint16_t* o = m.out + pr * m.out_stride + f;
                    float h[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) h[j] = act_of(g[j], m.act) * u[j];
                    if (f + 3 < m.Q && (reinterpret_cast<uintptr_t>(o) & 7) == 0) {
                        *reinterpret_cast<uint2*>(o) = make_uint2(pack2(h[0], h[1]), pack2(h[2], h[3]));
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (f + j < m.Q) o[j] = to_bf16(h[j]).bits;
                    }
                } else {
                    if (f >= m.seg_rows) continue;
                    const uint16_t* dh = m.dh + pr * m.dh_stride + f;
                    float dv[4];
                    if (f + 3 < m.Q && (reinterpret_cast<uintptr_t>(dh) & 7) == 0) {
                        const uint2 w = *reinterpret_cast<const uint2*>(dh);
                        dv[0] = half_f32(w.x, 0), dv[1] = half_f32(w.x, 1), dv[2] = half_f32(w.y, 0), dv[3] = half_f32(w.y, 1);
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) dv[j] = f + j < m.Q ? half_f32(dh[j], 0) : 0.0f;
                    }
                    float dg[4], du[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float a, da;
                        act_grad(g[j], m.act, a, da);
                        dg[j] = f + j < m.Q ? dv[j] * u[j] * da : 0.0f;
                        du[j] = f + j < m.Q ? dv[j] * a : 0.0f;
                    }
                    uint16_t* o = m.d + pr * 2 * m.seg_rows + f;
                    *reinterpret_cast<uint2*>(o) = make_uint2(pack2(dg[0], dg[1]), pack2(dg[2], dg[3]));
                    *reinterpret_cast<uint2*>(o + m.seg_rows) = make_uint2(pack2(du[0], du[1]), pack2(du[2], du[3]));
                }
            }
        } else {
#pragma unroll
            for (int q = 0; q < QT; ++q) {
                const int64_t qc = q0 + q_row(q) + lq;
                if (qc >= m.Q) continue;
                const f32x4 v = acc[q][p];
                if constexpr (EPI == kEpiPartial) {
                    float* o = m.part + ((int64_t)blockIdx.y * m.P + pr) * m.Q + qc;
                    if (m.Q % 4 == 0) {
                        *reinterpret_cast<f32x4*>(o) = v;
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (qc + j < m.Q) o[j] = v[j];
                    }
                } else {
                    const int64_t row = pr < m.seg_rows ? pr : pr - m.seg_rows;
                    if (row >= m.seg_valid) continue;
                    uint16_t* o = (pr < m.seg_rows ? m.out : m.out2) + row * m.out_stride + qc;
                    if (qc + 3 < m.Q && (reinterpret_cast<uintptr_t>(o) & 7) == 0) {
                        *reinterpret_cast<uint2*>(o) = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (qc + j < m.Q) o[j] = to_bf16(v[j]).bits;
                    }
                }
            }
        }
    }
}

// The splits' partial sums of a product, added in order.
__global__ __launch_bounds__(256) void ffn_join_kernel(FfnMat m) {
    const int64_t n = m.P * m.Q;
    for (int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x; k < n; k += (int64_t)gridDim.x * 256) {
        const int64_t pr = k / m.Q, qc = k - pr * m.Q;
        const int64_t row = pr < m.seg_rows ? pr : pr - m.seg_rows;
        if (row >= m.seg_valid) continue;
        float s = 0.0f;
#pragma unroll 4
        for (int q = 0; q < m.splits; ++q) s += m.part[q * n + k];
        (pr < m.seg_rows ? m.out : m.out2)[row * m.out_stride + qc] = to_bf16(s).bits;
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
    const int64_t n = m.rows[which] * m.wide;
    for (int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x; k < n; k += (int64_t)gridDim.x * 256) {
        const int64_t r = k / m.wide, c = k - r * m.wide;
        m.dst[which][k] = c < m.cols ? m.src[which][r * m.stride[which] + c] : (uint16_t)0;
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
    int t;  // tile edge: 256 or 128
    int tiles_p, tiles_q, splits;
};

// 256-wide tiles where they fill the GPU, else 128; the contraction split where even those leave half of
// it idle and it is long.
Tiling tiling(int64_t P, int64_t Q, int64_t q_per_tile_256, int steps, bool may_split) {
    const int64_t cus = layers_cus();
    auto div = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    Tiling t{256, (int)div(P, 256), (int)div(Q, q_per_tile_256), 1};
    if ((int64_t)t.tiles_p * t.tiles_q < cus / 2 * 3 && !(may_split && steps >= 64)) {
        t.t = 128;
        t.tiles_p = (int)div(P, 128);
        t.tiles_q = (int)div(Q, q_per_tile_256 / 2);
    }
    if (may_split) {
        const int64_t n = (int64_t)t.tiles_p * t.tiles_q, room = t.t == 256 ? cus : 2 * cus;
        int64_t s = n < room ? room / n : 1;
        if (s > steps / 4) s = steps / 4;
        t.splits = s < 1 ? 1 : s > 64 ? 64 : (int)s;
    }
    return t;
}

template <bool XTR, bool YTR, int EPI>
void run_mat(FfnMat m, const Tiling& t, hipStream_t stream) {
    m.tiles_p = t.tiles_p, m.tiles_q = t.tiles_q, m.splits = t.splits;
    const dim3 grid((unsigned)(t.tiles_p * t.tiles_q), (unsigned)t.splits);
    if (t.t == 256)
        hipLaunchKernelGGL((ffn_mat_kernel<256, 256, 2, 4, XTR, YTR, EPI>), grid, dim3(512), 0, stream, m);
    else
        hipLaunchKernelGGL((ffn_mat_kernel<128, 128, 2, 2, XTR, YTR, EPI>), grid, dim3(256), 0, stream, m);
}

template <bool XTR, bool YTR>
void run_product(const FfnMat& m, const Tiling& t, hipStream_t stream) {
    if (t.splits == 1) {
        run_mat<XTR, YTR, kEpiStore>(m, t, stream);
        return;
    }
    run_mat<XTR, YTR, kEpiPartial>(m, t, stream);
    FfnMat j = m;
    j.splits = t.splits;
    const int64_t n = (m.P * m.Q + 255) / 256;
    hipLaunchKernelGGL(ffn_join_kernel, dim3((unsigned)(n < 8192 ? n : 8192)), dim3(256), 0, stream, j);
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
                  char* ws, hipStream_t stream) {
    Operands o{static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(wg), static_cast<const uint16_t*>(wu), xs, gs, s.dim};
    if (!needs_copy(s, x, xs, wg, gs, wu, us)) return o;
    FfnCopy c{};
    c.cols = s.dim, c.wide = up(s.dim, 8);
    uint16_t* to = reinterpret_cast<uint16_t*>(ws);
    const int64_t xb = align256(s.rows * c.wide * 2) / 2, wb = align256(s.hidden * c.wide * 2) / 2;
    c.src[0] = o.x, c.dst[0] = to, c.rows[0] = s.rows, c.stride[0] = xs;
    c.src[1] = o.wg, c.dst[1] = to + xb, c.rows[1] = s.hidden, c.stride[1] = gs;
    c.src[2] = o.wu, c.dst[2] = to + xb + wb, c.rows[2] = s.hidden, c.stride[2] = us;
    const int64_t n = ((s.rows > s.hidden ? s.rows : s.hidden) * c.wide + 255) / 256;
    hipLaunchKernelGGL(ffn_copy_kernel, dim3((unsigned)(n < 4096 ? n : 4096), 3), dim3(256), 0, stream, c);
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
    b.dual = tiling(s.rows, b.fp, 128, steps_of(s.dim), false);
    b.dx = tiling(s.rows, s.dim, 256, 2 * steps_of(s.hidden), true);
    b.dw = tiling(2 * b.fp, s.dim, 256, steps_of(s.rows), true);
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
    hipLaunchKernelGGL(ffn_zero_kernel, dim3((unsigned)(g < 4096 ? g : 4096)), dim3(256), 0, stream, static_cast<uint16_t*>(p), n,
                       cols, stride);
    return launch_status();
}

int64_t ffn_workspace(const mamba_ffn_ptrs& p, const mamba_ffn_shape& s) {
    return needs_copy(s, p.x, p.x_stride, p.w_gate, p.w_gate_stride, p.w_up, p.w_up_stride) ? copy_bytes(s) : 0;
}

int64_t ffn_bwd_workspace(const mamba_ffn_shape& s) { return bwd_plan(s).total; }

int launch_ffn_fwd(const mamba_ffn_ptrs& p, const mamba_ffn_shape& s, int act, hipStream_t stream) {
    const Operands o = operands(s, p.x, p.x_stride, p.w_gate, p.w_gate_stride, p.w_up, p.w_up_stride,
                                static_cast<char*>(p.workspace), stream);
    FfnMat m = dual_mat(s, o, act);
    m.out = static_cast<uint16_t*>(p.h), m.out_stride = p.h_stride;
    run_mat<false, false, kEpiDual>(m, tiling(s.rows, s.hidden, 128, m.steps, false), stream);
    return launch_status();
}

int launch_ffn_bwd(const mamba_ffn_bwd_ptrs& p, const mamba_ffn_shape& s, int act, hipStream_t stream) {
    const BwdPlan b = bwd_plan(s);
    char* ws = static_cast<char*>(p.workspace);
    const Operands o = operands(s, p.x, p.x_stride, p.w_gate, p.w_gate_stride, p.w_up, p.w_up_stride, ws + b.copy, stream);
    uint16_t* d = reinterpret_cast<uint16_t*>(ws + b.d);
    FfnMat m = dual_mat(s, o, act);
    m.dh = static_cast<const uint16_t*>(p.dh), m.dh_stride = p.dh_stride, m.d = d, m.seg_rows = b.fp;
    run_mat<false, false, kEpiDualBwd>(m, b.dual, stream);

    FfnMat x{};  // dx[p][q] = sum over gate and up units c of d[p][c] W[c][q]
    x.x = d, x.x_stride = 2 * b.fp, x.x_cols = b.fp, x.x_seg = b.fp;
    x.y[0] = o.wg, x.y[1] = o.wu, x.y_stride = o.ws;
    x.P = s.rows, x.Q = s.dim, x.C = s.hidden;
    x.steps = steps_of(s.hidden), x.stretches = 2;
    x.out = x.out2 = static_cast<uint16_t*>(p.dx), x.out_stride = s.dim, x.seg_rows = x.seg_valid = s.rows;
    x.part = reinterpret_cast<float*>(ws + b.part);
    run_product<false, true>(x, b.dx, stream);

    FfnMat w{};  // dW[f][q] = sum over tokens c of d[c][f] x[c][q]
    w.x = d, w.x_stride = 2 * b.fp;
    w.y[0] = w.y[1] = o.x, w.y_stride = o.xs;
    w.P = 2 * b.fp, w.Q = s.dim, w.C = s.rows;
    w.steps = steps_of(s.rows), w.stretches = 1;
    w.out = static_cast<uint16_t*>(p.dw_gate), w.out2 = static_cast<uint16_t*>(p.dw_up), w.out_stride = s.dim;
    w.seg_rows = b.fp, w.seg_valid = s.hidden;
    w.part = reinterpret_cast<float*>(ws + b.part);
    run_product<true, true>(w, b.dw, stream);
    return launch_status();
}

}  // namespace mscan
