// Launchers of the gated linear recurrence.
#include "gated.hpp"
#include "layers_launch.hpp"

namespace mscan {

namespace {

constexpr int kFwdSteps = 256;  // segments are whole chunks of either forward kernel, 16 runs of 16 or 8 steps
constexpr int kStepMaxLen = 8;  // calls up to this length run the short kernel

// The widest channel group that still gives every compute unit work; segments where even the
// narrowest does not.
GatedPlan plan_for(const mamba_gated_shape& s, int cus, int chunk) {
    GatedPlan p{64, 1, 0};
    auto blocks = [&](int ch) { return s.batch * ((s.dim + ch - 1) / ch); };
    const int64_t want = cus * 3 / 4;
    for (int ch : {64, 32, 16}) {
        p.ch = ch;
        if (blocks(ch) >= want) break;
    }
    int64_t seg = (s.len + chunk - 1) / chunk * chunk;
    if (blocks(p.ch) * 2 <= cus && s.len >= 8 * chunk) {
        const int64_t n = cus / blocks(p.ch);
        const int64_t per = (s.len + n - 1) / n;
        seg = (per + chunk - 1) / chunk * chunk;
        if (seg < 4 * chunk) seg = 4 * chunk;
    }
    p.seg_len = seg > 0 ? seg : chunk;
    p.nseg = (int)((s.len + p.seg_len - 1) / p.seg_len);
    if (p.nseg < 1) p.nseg = 1;
    return p;
}

// dlam[d] = sigmoid(lam) / softplus(lam) * sum of the parts, in order; the ratio is 1 to fp32 below
// lam = -20 (and both vanish far below).
__global__ __launch_bounds__(256) void gated_dlam_kernel(const float* part, int64_t parts, const float* lam, float* dlam,
                                                         int64_t D) {
    const int64_t d = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (d >= D) return;
    float s = 0.0f;
    for (int64_t q = 0; q < parts; ++q) s += part[q * D + d];
    const float v = lam[d];
    dlam[d] = v < -20.0f ? s : s * (sigmoid_f(v) * hw_rcp(softplus_f(v)));
}

template <typename S, int CH, int MODE>
void run_fwd(const GatedParams& q, hipStream_t stream) {
    constexpr int TS = sizeof(S) == 2 ? 16 : 8;  // fp32 rows take twice the registers
    constexpr int share = CH * (int)sizeof(S) < 128 ? 128 / (CH * (int)sizeof(S)) : 1;
    const int nseg = MODE == kGatedPairs ? q.nseg - 1 : q.nseg;
    const int64_t grid = gated_blocks((q.dim + CH - 1) / CH, q.batch, nseg, share);
    if (q.reset)
        hipLaunchKernelGGL((gated_fwd_kernel<S, CH, TS, true, MODE>), dim3((unsigned)grid), dim3(CH * 16), 0, stream, q);
    else
        hipLaunchKernelGGL((gated_fwd_kernel<S, CH, TS, false, MODE>), dim3((unsigned)grid), dim3(CH * 16), 0, stream, q);
}

template <typename S, int MODE>
void pick_fwd(const GatedParams& q, int ch, hipStream_t stream) {
    if (ch == 64) run_fwd<S, 64, MODE>(q, stream);
    else if (ch == 32) run_fwd<S, 32, MODE>(q, stream);
    else run_fwd<S, 16, MODE>(q, stream);
}

template <typename S, int CH, int MODE>
void run_bwd(const GatedBwdParams& q, hipStream_t stream) {
    constexpr int TS = 8;
    constexpr int share = CH * (int)sizeof(S) < 128 ? 128 / (CH * (int)sizeof(S)) : 1;
    const int nseg = MODE == kGatedPairs ? q.nseg - 1 : q.nseg;
    const int64_t grid = gated_blocks((q.dim + CH - 1) / CH, q.batch, nseg, share);
    if (q.reset)
        hipLaunchKernelGGL((gated_bwd_kernel<S, CH, TS, true, MODE>), dim3((unsigned)grid), dim3(CH * 16), 0, stream, q);
    else
        hipLaunchKernelGGL((gated_bwd_kernel<S, CH, TS, false, MODE>), dim3((unsigned)grid), dim3(CH * 16), 0, stream, q);
}

template <typename S, int MODE>
void pick_bwd(const GatedBwdParams& q, int ch, hipStream_t stream) {
    if (ch == 64) run_bwd<S, 64, MODE>(q, stream);
    else if (ch == 32) run_bwd<S, 32, MODE>(q, stream);
    else run_bwd<S, 16, MODE>(q, stream);
}

template <typename S>
int fwd_typed(const GatedParams& q, const GatedPlan& plan, hipStream_t stream) {
    if (q.len <= kStepMaxLen) {
        const int64_t n = q.batch * q.dim;
        hipLaunchKernelGGL((gated_step_kernel<S>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream, q);
        return launch_status();
    }
    if (q.nseg > 1) pick_fwd<S, kGatedPairs>(q, plan.ch, stream);
    pick_fwd<S, kGatedStates>(q, plan.ch, stream);
    return launch_status();
}

template <typename S>
int bwd_typed(const GatedBwdParams& q, const GatedPlan& plan, float* dlam, hipStream_t stream) {
    if (q.nseg > 1) pick_bwd<S, kGatedPairs>(q, plan.ch, stream);
    pick_bwd<S, kGatedStates>(q, plan.ch, stream);
    hipLaunchKernelGGL(gated_dlam_kernel, dim3((unsigned)((q.dim + 255) / 256)), dim3(256), 0, stream, q.part,
                       q.batch * q.nseg, q.lam, dlam, q.dim);
    return launch_status();
}

}  // namespace

GatedPlan gated_plan(const mamba_gated_shape& s, int cus) { return plan_for(s, cus, kFwdSteps); }
GatedPlan gated_bwd_plan(const mamba_gated_shape& s, int cus) { return plan_for(s, cus, kGatedCk); }

int launch_gated_fwd(const GatedParams& q, const GatedPlan& plan, bool bf16, hipStream_t stream) {
    return bf16 ? fwd_typed<bf16_t>(q, plan, stream) : fwd_typed<float>(q, plan, stream);
}

// The checkpoints alone, for a backward that was not given them.
int launch_gated_checkpoints(const GatedParams& q, const GatedPlan& plan, bool bf16, hipStream_t stream) {
    if (bf16) {
        if (q.nseg > 1) pick_fwd<bf16_t, kGatedPairs>(q, plan.ch, stream);
        pick_fwd<bf16_t, kGatedCkOnly>(q, plan.ch, stream);
    } else {
        if (q.nseg > 1) pick_fwd<float, kGatedPairs>(q, plan.ch, stream);
        pick_fwd<float, kGatedCkOnly>(q, plan.ch, stream);
    }
    return launch_status();
}

int launch_gated_bwd(const GatedBwdParams& q, const GatedPlan& plan, float* dlam, bool bf16, hipStream_t stream) {
    return bf16 ? bwd_typed<bf16_t>(q, plan, dlam, stream) : bwd_typed<float>(q, plan, dlam, stream);
}

}  // namespace mscan
