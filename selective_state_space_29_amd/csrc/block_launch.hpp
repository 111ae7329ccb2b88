// Launchers of the block operators (mamba_block.h), each in a translation unit of its own; the entry points
// in block.hip validate and call these.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/mamba_block.h"

namespace mscan {

int launch_conv_fwd(const mamba_conv_ptrs& p, const mamba_conv_shape& s, int act, bool bf16, hipStream_t stream);
int launch_conv_bwd(const mamba_conv_bwd_ptrs& p, const mamba_conv_shape& s, int act, bool bf16, hipStream_t stream);
int64_t conv_bwd_workspace(const mamba_conv_shape& s, bool x_steps);

int launch_block_step(const mamba_step_ptrs& p, const mamba_step_shape& s, bool bf16, hipStream_t stream);
int64_t block_step_workspace(const mamba_step_shape& s);

int launch_rms_fwd(const mamba_rms_ptrs& p, const mamba_rms_shape& s, float scale, float eps, bool bf16, hipStream_t stream);
int launch_rms_bwd(const mamba_rms_bwd_ptrs& p, const mamba_rms_shape& s, float scale, bool bf16, hipStream_t stream);
int64_t rms_bwd_workspace(const mamba_rms_shape& s);
int launch_gated_rms_fwd(const mamba_gated_rms_ptrs& p, const mamba_gated_rms_shape& s, bool gate_first, float eps, bool bf16,
                         hipStream_t stream);
int launch_gated_rms_bwd(const mamba_gated_rms_bwd_ptrs& p, const mamba_gated_rms_shape& s, bool gate_first, bool bf16,
                         hipStream_t stream);
int64_t gated_rms_bwd_workspace(const mamba_gated_rms_shape& s);

int launch_xent_fwd(const mamba_xent_ptrs& p, const mamba_xent_shape& s, bool target64, float scale, hipStream_t stream);
int launch_xent_bwd(const mamba_xent_bwd_ptrs& p, const mamba_xent_shape& s, bool target64, float scale, hipStream_t stream);
int64_t xent_workspace(const mamba_xent_ptrs& p, const mamba_xent_shape& s);
int64_t xent_bwd_workspace(const mamba_xent_bwd_ptrs& p, const mamba_xent_shape& s);

}  // namespace mscan
