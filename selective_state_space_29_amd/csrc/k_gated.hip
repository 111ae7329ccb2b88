// Launchers of the gated linear recurrence.
#include "gated.hpp"
#include "layers_launch.hpp"

namespace mscan {

namespace {

constexpr int kStepMaxLen = 8;  // calls up to this length run the short kernel

// Workgroups per chain of 64 channels of a batch: as many as fill the GPU (a workgroup of 16 waves is all
// a compute unit holds) where there are fewer chains, down to one chunk for each (1 x 2000 x 2560 forward
// 29.6 us, 41.8 with four chunks for each; 2 x 3000 x 512 forward and backward 70 and 105). Short rows are
// not shared: clearing the chain and waiting costs more (1 x 500 x 700 fp32 forward and backward 46 us
// alone, 53 shared; 3 x 777 x 1000 forward 28 and 22).
constexpr int kShareLen = 640;
int ways_for(const mamba_gated_shape& s, int cus, int chunk) {
    const int64_t chains = s.batch * ((s.dim + kChans - 1) / kChans), chunks = (s.len + chunk - 1) / chunk;
    if (chains < 1 || s.len < kShareLen) return 1;
    const int64_t w = cus / chains < chunks ? cus / chains : chunks;
    return w < 1 ? 1 : (int)w;
}

// dlam[d] = sigmoid(lam) / softplus(lam) * sum of the chunks' sums of q: 16 stretches of the list a
// channel, added in order; the ratio is 1 to fp32 below lam = -20 (and both vanish far below).
__global__ __launch_bounds__(1024) void gated_dlam_kernel(const float* part, int64_t parts, const float* lam, float* dlam,
                                                          int64_t D) {
    __shared__ float lds[16][64];
    const int64_t d = grid_block() * 64 + (threadIdx.x & 63);
    const int g = threadIdx.x >> 6;
    const int64_t per = (parts + 15) / 16, q1 = (g + 1) * per < parts ? (g + 1) * per : parts;
    float s = 0.0f;
    if (d < D)
#pragma unroll 8
        for (int64_t q = g * per; q < q1; ++q) s += part[q * D + d];
    lds[g][threadIdx.x & 63] = s;
    __syncthreads();
    if (g > 0 || d >= D) return;
#pragma unroll
    for (int q = 1; q < 16; ++q) s += lds[q][threadIdx.x];
    const float v = lam[d];
    dlam[d] = v < -20.0f ? s : s * (sigmoid_f(v) * hw_rcp(softplus_f(v)));
}

__global__ __launch_bounds__(256) void gated_clear_kernel(uint4* p, int64_t n) {
    for (int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x; k < n; k += (int64_t)gridDim.x * 256) p[k] = make_uint4(0, 0, 0, 0);
}

void clear_chain(uint64_t* p, int64_t batch, int64_t dim, int64_t len, int chunk, Launches& on) {
    const int64_t n = (GatedChain::words(batch, dim, (len + chunk - 1) / chunk) + 1) / 2;  // the workspace ends on 256 bytes
    const int64_t g = (n + 511) / 512;
    on(gated_clear_kernel, dim3((unsigned)(g < 4096 ? g : 4096)), dim3(256), reinterpret_cast<uint4*>(p), n);
}

template <typename S, bool STATES>
void run_fwd(const GatedParams& q, Launches& on) {
    constexpr int TS = gated_fwd_ts(sizeof(S), false), TC = gated_fwd_ts(sizeof(S), true);
    const dim3 grid = grid_of(gated_blocks(q.batch * ((q.dim + kChans - 1) / kChans), q.ways), 1024), block(1024);
    if (q.ways > 1) {
        clear_chain(q.chain, q.batch, q.dim, q.len, kRuns * TC, on);
        if (q.reset) on(gated_fwd_kernel<S, TC, true, STATES, true>, grid, block, q);
        else on(gated_fwd_kernel<S, TC, false, STATES, true>, grid, block, q);
    } else {
        if (q.reset) on(gated_fwd_kernel<S, TS, true, STATES, false>, grid, block, q);
        else on(gated_fwd_kernel<S, TS, false, STATES, false>, grid, block, q);
    }
}

template <typename S>
void run_bwd(const GatedBwdParams& q, Launches& on) {
    const dim3 grid = grid_of(gated_blocks(q.batch * ((q.dim + kChans - 1) / kChans), q.ways), 1024), block(1024);
    if (q.ways > 1) {
        clear_chain(q.chain, q.batch, q.dim, q.len, kGatedCk, on);
        if (q.reset) on(gated_bwd_kernel<S, 8, true, true>, grid, block, q);
        else on(gated_bwd_kernel<S, 8, false, true>, grid, block, q);
    } else {
        if (q.reset) on(gated_bwd_kernel<S, 8, true, false>, grid, block, q);
        else on(gated_bwd_kernel<S, 8, false, false>, grid, block, q);
    }
    on(gated_dlam_kernel, grid_of((q.dim + 63) / 64, 1024), dim3(1024), q.part, q.batch * q.nck,
       q.lam, q.dlam, q.dim);
}

template <typename S>
void fwd_typed(const GatedParams& q, Launches& on) {
    if (q.len <= kStepMaxLen) {
        const int64_t n = q.batch * q.dim;
        on(gated_step_kernel<S>, dim3((unsigned)((n + 255) / 256)), dim3(256), q);
    } else {
        run_fwd<S, true>(q, on);
    }
}

}  // namespace

int gated_fwd_ways(const mamba_gated_shape& s, bool bf16, int cus) { return ways_for(s, cus, kRuns * gated_fwd_ts(bf16 ? 2 : 4, true)); }
int gated_bwd_ways(const mamba_gated_shape& s, int cus) { return ways_for(s, cus, kGatedCk); }

int launch_gated_fwd(const GatedParams& q, bool bf16, hipStream_t stream) {
    Launches on(stream);
    bf16 ? fwd_typed<bf16_t>(q, on) : fwd_typed<float>(q, on);
    return on.status;
}

// The checkpoints alone, for a backward that was not given them.
int launch_gated_checkpoints(const GatedParams& q, bool bf16, hipStream_t stream) {
    Launches on(stream);
    bf16 ? run_fwd<bf16_t, false>(q, on) : run_fwd<float, false>(q, on);
    return on.status;
}

int launch_gated_bwd(const GatedBwdParams& q, bool bf16, hipStream_t stream) {
    Launches on(stream);
    bf16 ? run_bwd<bf16_t>(q, on) : run_bwd<float>(q, on);
    return on.status;
}

}  // namespace mscan
