// One token of each stream through a Mamba block's path from the convolution to the gate (mamba_block.h), on
// gfx950, in two launches or three.
//
//   first:   u = silu(conv_b + sum_k conv_w v_k) and the conv state's new rows; each workgroup's 64 channels'
//            share of w_x u, for up to kRows streams (its part of w_x is read once for them)
//   second:  (dt rows, B, C) = the shares added in channel order; delta = w_dt dt;  s = softplus(delta + dt_bias);
//            h' = exp(s A) h + s B u;   y = (sum_n C h' + D u) silu(z)
//
// The x projection needs every channel before any can go on, which is the boundary between the launches. All of it
// stays in fp32 from one to the other: u and the shares go through the workspace (at 64 streams of 1536 channels
// 0.9 MB beside 12.6 MB of scan state). In the second launch 4 lanes hold a channel, 4 of every 16 states each, so
// that states and A move 16 bytes a lane and the sums over states and dt rows stay within a quad; at 16 states and a
// multiple of 4 dt rows everything that does not depend on the first launch's sums is loaded before they are, otherwise
// states, A and w_dt follow them.
//
// Many streams of many channels share workgroups in the second launch, behind one that adds the shares (below).
//
// Bound by latency: at 1536 channels, 16 states and 48 dt rows bf16 one stream takes 4.2 + 3.7 us, 64 streams 5.4 +
// 6.8, of which their 15 MB need 3.3.
#include <type_traits>

#include "block_launch.hpp"
#include "layers_common.hpp"
#include "rows.hpp"

namespace mscan {

namespace {

constexpr int kCh = 64;       // channels of a workgroup, in either launch
constexpr int kRows = 8;      // streams of a workgroup of the first launch
constexpr int kThreads = 256;
constexpr int kMaxJ = 512 + 2 * 256;
constexpr int64_t kManyGroups = 512;

__host__ __device__ constexpr int up4(int n) { return (n + 3) / 4 * 4; }

struct StepArgs {
    const void* x;
    const void* z;
    const void* conv_state;
    const float* h;
    const float* conv_w;
    const float* conv_b;
    const void* w_x;
    const void* w_dt;
    const float* dt_bias;
    const float* A;
    const float* D;
    void* conv_out;
    float* h_out;
    float* y;
    float* u;      // (batch, dim)
    float* part;   // (chunks, batch, J)
    int64_t sx, sz;
    int64_t batch, dim;
    int dstate, rank, J, chunks;
};

// Sum over a quad's lanes, the same bits in each: lane pairs, then the pairs.
template <int CTRL>
__device__ __forceinline__ float quad_add(float v) {
    return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
}
__device__ __forceinline__ float quad_sum(float v) { return quad_add<0x4e>(quad_add<0xb1>(v)); }
// Over 8 lanes: the quads' sums, then the half row mirrored.
__device__ __forceinline__ float oct_sum(float v) { return quad_add<0x141>(quad_sum(v)); }

// (Loads of rows, streams and channels past the end repeat the last one: without a branch around them they are all
// on their way before the first is used.)
template <typename S, int W>
__global__ __launch_bounds__(kThreads) void step_conv_kernel(StepArgs p) {
    __shared__ __align__(16) float us[kRows][kCh];
    const int tid = threadIdx.x;
    const int chunk = blockIdx.x % p.chunks;
    const int64_t b0 = (int64_t)(blockIdx.x / p.chunks) * kRows, c0 = (int64_t)chunk * kCh;
    const int rows = (int)(p.batch - b0 < kRows ? p.batch - b0 : kRows);

    // 8 lanes a row of w_x, 8 channels each; its first rows are on their way while u is computed
    const int part = tid & 7, j0 = tid >> 3;
    const int n = (int)(p.dim - c0 < kCh ? p.dim - c0 : kCh) - part * 8;
    const S* wx = static_cast<const S*>(p.w_x) + c0 + part * 8;
    constexpr int AHEAD = 3;  // rounds of 32 rows: more than dt_rank 48 and 16 states need
    Pack<S, 8> w[AHEAD];
#pragma unroll
    for (int r = 0; r < AHEAD; ++r) w[r] = load_some<S, 8>(wx + (int64_t)(j0 + 32 * r < p.J ? j0 + 32 * r : p.J - 1) * p.dim, n);

    constexpr int PER = kRows * kCh / kThreads;  // streams of a thread
    const bool in = c0 + (tid & (kCh - 1)) < p.dim;
    const int64_t c = in ? c0 + (tid & (kCh - 1)) : p.dim - 1;
    float cw[W];
#pragma unroll
    for (int k = 0; k < W; ++k) cw[k] = p.conv_w[c * W + k];
    const float cb = p.conv_b ? p.conv_b[c] : 0.0f;
    S v[PER][W];
#pragma unroll
    for (int r = 0; r < PER; ++r) {
        const int row = r * (kThreads / kCh) + tid / kCh;
        const int64_t b = b0 + (row < rows ? row : rows - 1);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) v[r][k] = static_cast<const S*>(p.conv_state)[(b * (W - 1) + k) * p.dim + c];
        v[r][W - 1] = static_cast<const S*>(p.x)[b * p.sx + c];
    }
#pragma unroll
    for (int r = 0; r < PER; ++r) {
        const int row = r * (kThreads / kCh) + tid / kCh;
        const int64_t b = b0 + row;
        float u = cb;
#pragma unroll
        for (int k = 0; k < W; ++k) u = __builtin_fmaf(cw[k], to_f32(v[r][k]), u);
        u = silu_f(u);
        us[row][tid & (kCh - 1)] = in ? u : 0.0f;
        if (in && row < rows) {
#pragma unroll
            for (int k = 0; k < W - 1; ++k) static_cast<S*>(p.conv_out)[(b * (W - 1) + k) * p.dim + c] = v[r][k + 1];
            p.u[b * p.dim + c] = u;
        }
    }
    __syncthreads();
    float u[kRows][8];
#pragma unroll
    for (int row = 0; row < kRows; ++row)
#pragma unroll
        for (int k = 0; k < 8; ++k) u[row][k] = us[row][part * 8 + k];
    // a row's share for every stream: the 8 lanes' sums, each lane storing one stream's
    auto share = [&](const Pack<S, 8>& wr, int j) __attribute__((always_inline)) {
        float mine = 0.0f;
#pragma unroll
        for (int row = 0; row < kRows; ++row) {
            float s = 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) s = __builtin_fmaf(to_f32(wr.v[k]), u[row][k], s);
            s = oct_sum(s);
            mine = part == row ? s : mine;
        }
        if (part < rows && j < p.J) p.part[((int64_t)chunk * p.batch + b0 + part) * p.J + j] = mine;
    };
#pragma unroll
    for (int r = 0; r < AHEAD; ++r)
        if (32 * r < p.J) share(w[r], j0 + 32 * r);
    for (int j = j0 + 32 * AHEAD; j - j0 < p.J; j += 32)
        share(load_some<S, 8>(wx + (int64_t)(j < p.J ? j : p.J - 1) * p.dim, n), j);
}

// WHOLE: 16 states and a multiple of 4 dt rows, held in registers from the start.
template <typename S, bool WHOLE>
__global__ __launch_bounds__(kThreads) void step_scan_kernel(StepArgs p) {
    __shared__ __align__(16) float sums[kThreads], xd[kMaxJ];
    const int tid = threadIdx.x, q = tid & 3;
    const int64_t b = blockIdx.x / p.chunks, d0 = (int64_t)(blockIdx.x % p.chunks) * kCh;
    const bool valid = d0 + (tid >> 2) < p.dim;
    const int64_t d = valid ? d0 + (tid >> 2) : p.dim - 1;
    const int N = WHOLE ? 16 : p.dstate, R = p.rank, J = p.J;

    // the chunks' shares of row j: `ways` stretches of the chunks side by side, added in order
    const float* part = p.part + b * J;
    const int64_t next = p.batch * J;
    const int ways = J <= kThreads ? kThreads / J : 1, per = (p.chunks + ways - 1) / ways;
    auto stretch = [&](int j, int way) __attribute__((always_inline)) {
        const int k0 = way * per, k1 = k0 + per < p.chunks ? k0 + per : p.chunks;
        float s = 0.0f;
        for (int k = k0; k < k1; k += 8) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = part[(k + i < k1 ? k + i : k1 - 1) * next + j];
#pragma unroll
            for (int i = 0; i < 8; ++i) s += k + i < k1 ? v[i] : 0.0f;
        }
        return s;
    };

    // what does not wait for the projection
    const float* h = p.h + (b * p.dim + d) * N;
    const float* A = p.A + d * N;
    const S* wd = static_cast<const S*>(p.w_dt) + d * R;
    constexpr int AHEAD = 4;  // 64 dt rows
    Pack<float, 4> h0{}, a0{};
    Pack<S, 4> w[AHEAD];
    if constexpr (WHOLE) {
        __builtin_memcpy(&h0, h + q * 4, 16);
        __builtin_memcpy(&a0, A + q * 4, 16);
#pragma unroll
        for (int r = 0; r < AHEAD; ++r) __builtin_memcpy(&w[r], wd + (r * 16 + q * 4 < R ? r * 16 + q * 4 : 0), sizeof(w[r]));
    }
    const float u = p.u[b * p.dim + d];
    const float z = p.z ? to_f32(static_cast<const S*>(p.z)[b * p.sz + d]) : 0.0f;
    const float bias = p.dt_bias ? p.dt_bias[d] : 0.0f, skip = p.D ? p.D[d] : 0.0f;

    if (J <= kThreads) {
        const int way = tid / J, j = tid - way * J;
        float s = way < ways ? stretch(j, way) : 0.0f;
        sums[tid] = s;
        __syncthreads();
        if (tid < J) {
            for (int k = 1; k < ways; ++k) s += sums[k * J + tid];
            xd[tid] = s;
        }
    } else {
        for (int j = tid; j < J; j += kThreads) xd[j] = stretch(j, 0);
    }
    __syncthreads();

    float delta = 0.0f;
    auto dot = [&](const Pack<S, 4>& wr, int r) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (r + k < R) delta = __builtin_fmaf(to_f32(wr.v[k]), xd[r + k], delta);
    };
    if constexpr (WHOLE) {
#pragma unroll
        for (int r = 0; r < AHEAD; ++r) dot(w[r], r * 16 + q * 4);
    }
#pragma unroll 2
    for (int r = (WHOLE ? AHEAD * 16 : 0) + q * 4; r < R; r += 16) dot(load_some<S, 4>(wd + r, R - r), r);
    const float s = softplus_f(quad_sum(delta) + bias), su = s * u;

    float* ho = p.h_out + (b * p.dim + d) * N;
    float o = 0.0f;
    auto states = [&](const Pack<float, 4>& hv, const Pack<float, 4>& av, int n0) __attribute__((always_inline)) {
        Pack<float, 4> r{};
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (n0 + k < N) {
                r.v[k] = __builtin_fmaf(hw_exp2(s * av.v[k] * kLog2e), hv.v[k], su * xd[R + n0 + k]);
                o = __builtin_fmaf(xd[R + N + n0 + k], r.v[k], o);
            }
        if (valid) store_some<float, 4>(ho + n0, r, N - n0);
    };
    if constexpr (WHOLE) {
        states(h0, a0, q * 4);
    } else {
#pragma unroll 4
        for (int n0 = q * 4; n0 < N; n0 += 16) states(load_some<float, 4>(h + n0, N - n0), load_some<float, 4>(A + n0, N - n0), n0);
    }
    o = __builtin_fmaf(skip, u, quad_sum(o));
    if (p.z) o *= silu_f(z);
    if (valid && q == 0) p.y[b * p.dim + d] = o;
}

// ---- many streams ----
//
// The shares are added once, by a kernel of their own, and a workgroup of the scan takes kRows streams of its 64
// channels: w_dt and A are read once for them, and their states are on their way together. The sums' order is
// step_scan_kernel's, and so are the bits. At 256 streams of 4096 channels (16 states, 128 dt rows, bf16) 19 + 5 + 59
// us: 2.3 TB/s of states, bound by the latencies that 3 workgroups a CU expose one after another.

// The chunks' shares of each stream's rows, in the order of step_scan_kernel. (2^23 streams of up to 1024 sums: more
// threads than a dimension of the grid counts.)
__global__ __launch_bounds__(kThreads) void step_join_kernel(StepArgs p, float* xd) {
    const int64_t at = grid_block() * kThreads + threadIdx.x, next = p.batch * p.J;
    if (at >= next) return;
    const int ways = p.J <= kThreads ? kThreads / p.J : 1, per = (p.chunks + ways - 1) / ways;
    float sum = 0.0f;
    for (int way = 0; way < ways; ++way) {
        const int k0 = way * per, k1 = k0 + per < p.chunks ? k0 + per : p.chunks;
        float s = 0.0f;
        for (int k = k0; k < k1; k += 16) {
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = p.part[(k + i < k1 ? k + i : k1 - 1) * next + at];
#pragma unroll
            for (int i = 0; i < 16; ++i) s += k + i < k1 ? v[i] : 0.0f;
        }
        sum = way ? sum + s : s;
    }
    xd[at] = sum;
}

// LDS holds each stream's dt rows, B and C padded to multiples of 4. JM: the most that it is kept for. FULL: a
// multiple of 4 states.
template <typename S, int JM, bool FULL>
__global__ __launch_bounds__(kThreads) void step_scan_many_kernel(StepArgs p, const float* xd_all) {
    __shared__ __align__(16) float xd[kRows][JM];
    const int tid = threadIdx.x, q = tid & 3;
    const int64_t b0 = (int64_t)(blockIdx.x / p.chunks) * kRows, d0 = (int64_t)(blockIdx.x % p.chunks) * kCh;
    const int rows = (int)(p.batch - b0 < kRows ? p.batch - b0 : kRows);
    const bool valid = d0 + (tid >> 2) < p.dim;
    const int64_t d = valid ? d0 + (tid >> 2) : p.dim - 1;
    const int N = p.dstate, R = p.rank, J = p.J, at_b = up4(R), at_c = at_b + up4(N);
    const float* A = p.A + d * N;
    const S* wd = static_cast<const S*>(p.w_dt) + d * R;
    // streams past the last repeat it
    auto cell = [&](int s) __attribute__((always_inline)) { return (b0 + (s < rows ? s : rows - 1)) * p.dim + d; };
    Pack<float, 4> a, h[kRows];
    auto fetch = [&](int n0) __attribute__((always_inline)) {
        a = load_some<float, 4>(A + n0, N - n0);
#pragma unroll
        for (int s = 0; s < kRows; ++s) h[s] = load_some<float, 4>(p.h + cell(s) * N + n0, N - n0);
    };
    fetch(q * 4);
    constexpr int AHEAD = 4;  // 64 dt rows
    Pack<S, 4> w[AHEAD];
    auto fetch_w = [&](int r0) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) w[i] = load_some<S, 4>(wd + r0 + 16 * i, R - r0 - 16 * i);
    };
    fetch_w(q * 4);
    float u[kRows], z[kRows], delta[kRows];
#pragma unroll
    for (int s = 0; s < kRows; ++s) {
        u[s] = p.u[cell(s)];
        z[s] = p.z ? to_f32(static_cast<const S*>(p.z)[(b0 + (s < rows ? s : rows - 1)) * p.sz + d]) : 0.0f;
        delta[s] = 0.0f;
    }
    const float bias = p.dt_bias ? p.dt_bias[d] : 0.0f, skip = p.D ? p.D[d] : 0.0f;
    for (int j = tid; j < at_c + up4(N); j += kThreads) {
        const int k = j < at_b ? j : j < at_c ? j - at_b + R : j - at_c + R + N;
        const bool in = j < at_b ? j < R : j < at_c ? j - at_b < N : j - at_c < N;
        float v[kRows];
#pragma unroll
        for (int s = 0; s < kRows; ++s) v[s] = in ? xd_all[(b0 + (s < rows ? s : rows - 1)) * J + k] : 0.0f;
#pragma unroll
        for (int s = 0; s < kRows; ++s) xd[s][j] = v[s];
    }
    __syncthreads();

    auto four = [&](int s, int j) __attribute__((always_inline)) { return *reinterpret_cast<const Pack<float, 4>*>(&xd[s][j]); };
    for (int r0 = q * 4; r0 < R; r0 += 16 * AHEAD) {
        if (r0 >= 16 * AHEAD) fetch_w(r0);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int r = r0 + 16 * i;
            if (r >= R) continue;
#pragma unroll
            for (int s = 0; s < kRows; ++s) {
                const Pack<float, 4> x = four(s, r);
#pragma unroll
                for (int k = 0; k < 4; ++k) delta[s] = __builtin_fmaf(to_f32(w[i].v[k]), x.v[k], delta[s]);
            }
        }
    }
    float su[kRows], o[kRows];
#pragma unroll
    for (int s = 0; s < kRows; ++s) {
        delta[s] = softplus_f(quad_sum(delta[s]) + bias);
        su[s] = delta[s] * u[s];
        o[s] = 0.0f;
    }
    for (int n0 = q * 4; n0 < N; n0 += 16) {
        if (n0 >= 16) fetch(n0);
#pragma unroll
        for (int s = 0; s < kRows; ++s) {
            const Pack<float, 4> B = four(s, at_b + n0), C = four(s, at_c + n0);
            Pack<float, 4> r{};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (FULL || n0 + k < N) {
                    r.v[k] = __builtin_fmaf(hw_exp2(delta[s] * a.v[k] * kLog2e), h[s].v[k], su[s] * B.v[k]);
                    o[s] = __builtin_fmaf(C.v[k], r.v[k], o[s]);
                }
            if (valid && s < rows) store_some<float, 4>(p.h_out + cell(s) * N + n0, r, N - n0);
        }
    }
#pragma unroll
    for (int s = 0; s < kRows; ++s) {
        float v = __builtin_fmaf(skip, u[s], quad_sum(o[s]));
        if (p.z) v *= silu_f(z[s]);
        if (valid && s < rows && q == s % 4) p.y[cell(s)] = v;
    }
}

int chunks_of(const mamba_step_shape& s) { return (int)((s.dim + kCh - 1) / kCh); }

// Whether kRows streams a workgroup leave enough workgroups, and the shares that every workgroup of one stream would
// add again are many enough to pay for a launch. us a call, bf16, each stream by itself / together: 256 x 1536, J = 80
// (47 MB of shares) 24.5 / 28.1; 256 x 2048, J = 96 (100 MB) 32.3 / 35.9; J = 193 (202 MB) 146 / 128; 128 x 4096, J =
// 160 (335 MB) 62 / 42; 256 x 4096, J = 160 (671 MB) 127 / 81, with 128 states, J = 385, 608 / 436.
bool many_streams(const mamba_step_shape& s) {
    const int64_t chunks = chunks_of(s), shares = s.batch * chunks * chunks * (s.dt_rank + 2 * s.dstate) * 4;
    return (s.batch + kRows - 1) / kRows * chunks >= kManyGroups && shares >= (int64_t)128 << 20;
}

}  // namespace

int64_t block_step_workspace(const mamba_step_shape& s) {
    const int64_t sums = s.batch * (s.dt_rank + 2 * s.dstate) * 4;
    return align256(s.batch * s.dim * 4) + align256(chunks_of(s) * sums) + align256(sums);
}

int launch_block_step(const mamba_step_ptrs& p, const mamba_step_shape& s, bool bf16, hipStream_t stream) {
    char* ws = static_cast<char*>(p.workspace);
    StepArgs q{p.x, p.z, p.conv_state, p.ssm_state, p.conv_w, p.conv_b, p.w_x, p.w_dt, p.dt_bias, p.A, p.D, p.conv_state_out,
               p.ssm_state_out, p.y, reinterpret_cast<float*>(ws), reinterpret_cast<float*>(ws + align256(s.batch * s.dim * 4)),
               p.x_stride, p.z_stride, s.batch, s.dim, (int)s.dstate, (int)s.dt_rank, (int)(s.dt_rank + 2 * s.dstate), chunks_of(s)};
    Launches on(stream);
    const dim3 first((unsigned)(q.chunks * ((s.batch + kRows - 1) / kRows))), second((unsigned)(q.chunks * s.batch)), block(kThreads);
    auto go = [&](auto zero) {
        using S = decltype(zero);
        if (s.width == 2) on(step_conv_kernel<S, 2>, first, block, q);
        else if (s.width == 3) on(step_conv_kernel<S, 3>, first, block, q);
        else on(step_conv_kernel<S, 4>, first, block, q);
        if (many_streams(s)) {
            float* xd = q.part + align256((int64_t)q.chunks * s.batch * q.J * 4) / 4;
            on(step_join_kernel, grid_of((s.batch * q.J + kThreads - 1) / kThreads, kThreads), block, q, xd);
            const bool full = s.dstate % 4 == 0;
            auto scan = [&](auto most) {
                constexpr int JM = decltype(most)::value;
                if (full) on(step_scan_many_kernel<S, JM, true>, first, block, q, static_cast<const float*>(xd));
                else on(step_scan_many_kernel<S, JM, false>, first, block, q, static_cast<const float*>(xd));
            };
            up4(q.rank) + 2 * up4(q.dstate) <= 256 ? scan(std::integral_constant<int, 256>{}) : scan(std::integral_constant<int, kMaxJ>{});
        } else if (s.dstate == 16 && s.dt_rank % 4 == 0) on(step_scan_kernel<S, true>, second, block, q);
        else on(step_scan_kernel<S, false>, second, block, q);
    };
    bf16 ? go(bf16_t{}) : go(0.0f);
    return on.status;
}

}  // namespace mscan
