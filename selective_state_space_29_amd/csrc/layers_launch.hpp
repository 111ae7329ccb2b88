// Launchers of the layer operators, each in a translation unit of its own; the entry points in
// layers.hip validate and call these.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/mamba_layers.h"

namespace mscan {

struct GatedParams;
struct GatedBwdParams;
// workgroups per chain of 64 channels (1: no chain storage is needed)
int gated_fwd_ways(const mamba_gated_shape& s, bool bf16, int cus);
int gated_bwd_ways(const mamba_gated_shape& s, int cus);
int launch_gated_fwd(const GatedParams& q, bool bf16, hipStream_t stream);
int launch_gated_checkpoints(const GatedParams& q, bool bf16, hipStream_t stream);
int launch_gated_bwd(const GatedBwdParams& q, bool bf16, hipStream_t stream);

int launch_norm_fwd(const mamba_norm_ptrs& p, const mamba_norm_shape& s, float eps, bool bf16, hipStream_t stream);
int launch_norm_bwd(const mamba_norm_bwd_ptrs& p, const mamba_norm_shape& s, bool bf16, hipStream_t stream);
int64_t norm_bwd_workspace(const mamba_norm_shape& s);

int launch_embedding_fwd(const void* ids, bool ids64, const void* weight, void* y, const mamba_embedding_shape& s,
                         float scale, bool bf16, hipStream_t stream);
int launch_embedding_bwd(const void* ids, bool ids64, const void* dy, void* dweight, void* ws,
                         const mamba_embedding_shape& s, float scale, bool bf16, hipStream_t stream);
int64_t embedding_bwd_workspace(const mamba_embedding_shape& s);

int launch_ffn_fwd(const mamba_ffn_ptrs& p, const mamba_ffn_shape& s, int act, hipStream_t stream);
int launch_ffn_bwd(const mamba_ffn_bwd_ptrs& p, const mamba_ffn_shape& s, int act, hipStream_t stream);
int launch_ffn_zero(void* p, int64_t rows, int64_t cols, int64_t stride, hipStream_t stream);
int64_t ffn_workspace(const mamba_ffn_ptrs& p, const mamba_ffn_shape& s);
int64_t ffn_bwd_workspace(const mamba_ffn_shape& s);

}  // namespace mscan
