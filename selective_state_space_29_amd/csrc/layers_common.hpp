// Helpers shared by the layer operators (mamba_layers.h): storage types, 16-byte vectors, launch
// checks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <tuple>

#include "../../include/mamba_layers.h"
#include "common.hpp"

namespace mscan {

// fp32 to bf16, to nearest even (v_cvt_pk_bf16_f32).
__device__ __forceinline__ bf16_t to_bf16(float v) {
    const __bf16 h = (__bf16)v;
    bf16_t r;
    __builtin_memcpy(&r.bits, &h, 2);
    return r;
}

template <typename S>
__device__ __forceinline__ S from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ bf16_t from_f32<bf16_t>(float v) { return to_bf16(v); }

// V consecutive elements moved as one access where V * sizeof(S) allows it.
template <typename S, int V>
struct __align__(V * sizeof(S)) Pack {
    S v[V];
};

// Sum over the 64 lanes of a wave, the same bits in every lane: prefix sums of the 16-lane rows (DPP
// row_shr), then of the rows (row_bcast), and lane 63's total to all.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float v) {
    return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xf, false));
}
__device__ __forceinline__ float wave_sum(float v) {
    v = dpp_add<0x111, 0xf>(v);
    v = dpp_add<0x112, 0xf>(v);
    v = dpp_add<0x114, 0xf>(v);
    v = dpp_add<0x118, 0xf>(v);
    v = dpp_add<0x142, 0xa>(v);  // rows 1 and 3 take the row before's total
    v = dpp_add<0x143, 0xc>(v);  // rows 2 and 3 take the first half's
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// The launches of one call, on its stream: on(kernel, grid, block, arguments ...). The first that the runtime
// refuses is the call's status, and none follows it. (The runtime's last error is no measure: it may be that
// of another call of the thread, and belongs to that call's maker.)
struct Launches {
    hipStream_t stream;
    int status = MAMBA_SCAN_OK;
    explicit Launches(hipStream_t s) : stream(s) {}
    template <typename... P, typename... A>
    void operator()(void (*kernel)(P...), dim3 grid, dim3 block, const A&... args) {
        if (status != MAMBA_SCAN_OK) return;
        std::tuple<P...> held(args...);
        std::apply(
            [&](auto&... v) {
                void* at[] = {const_cast<void*>(static_cast<const void*>(&v))...};
                if (hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, block, at, 0, stream) != hipSuccess)
                    status = MAMBA_SCAN_ERR_LAUNCH;
            },
            held);
    }
};

inline int64_t align256(int64_t n) { return (n + 255) & ~(int64_t)255; }

// A grid of at least n workgroups. The threads of a grid's dimension are counted in 32 bits, and a launch
// past them runs what is left of the count without an error; so more workgroups than that lie over y too.
// The kernel's number of a workgroup is grid_block(); those from n on have nothing to do.
inline dim3 grid_of(int64_t n, int threads) {
    const int64_t most = (int64_t)0xFFFFFFFF / threads / 8 * 8;  // whole turns over the 8 XCDs
    return n <= most ? dim3((unsigned)n) : dim3((unsigned)most, (unsigned)((n + most - 1) / most));
}
__device__ __forceinline__ int64_t grid_block() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }
__device__ __forceinline__ int64_t grid_blocks() { return (int64_t)gridDim.y * gridDim.x; }

int layers_cus();  // compute units of the current device (layers.hip); 256 if the runtime cannot say

}  // namespace mscan
