// Private declarations of the operators beside the swap-in path
// (hs_latent_attend, hs_latent_prefill, hs_rms_norm).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "hs.h"

// The channels that share a scale of hs_rms_norm; 0: the whole row.  A group that holds the whole row is
// that, so that a kernel's group indices times the group stay below twice the widest row.
inline int hs_norm_group(int dim, int carry, int group) { return group >= dim + carry ? 0 : group; }

// hs_ops.cpp has checked the arguments; these launch.
cudaError_t hs_launch_attend(const hs_attend_t& a, cudaStream_t s);
cudaError_t hs_launch_prefill(const hs_prefill_t& a, cudaStream_t s);
cudaError_t hs_launch_norm(const hs_norm_t& a, cudaStream_t s);
size_t hs_attend_workspace_bytes(int batch, int positions, int heads, int64_t rows);
size_t hs_prefill_workspace_bytes(int64_t k_tokens, int heads);

constexpr float HS_E4M3_MAX = 448.0f;

template <typename T> struct HsType;
template <> struct HsType<__nv_bfloat16> {
    static constexpr bool is_bf16 = true;
    static __device__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __nv_bfloat16 from_float(float v) { return __float2bfloat16_rn(v); }
};
template <> struct HsType<__half> {
    static constexpr bool is_bf16 = false;
    static __device__ float to_float(__half v) { return __half2float(v); }
    static __device__ __half from_float(float v) { return __float2half_rn(v); }
};
template <> struct HsType<float> {
    static __device__ float to_float(float v) { return v; }
    static __device__ float from_float(float v) { return v; }
};

__device__ inline float hs_e4m3_to_float(uint8_t v)
{
    __nv_fp8_e4m3 x;
    x.__x = v;
    return static_cast<float>(x);
}

// Two floats rounded to T, the first in the low half.
template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b)
{
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// A launch that may set up while the kernel before it in the stream runs out; griddepcontrol.wait waits for its results.
template <typename... Params, typename... Values>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t s, Values... values)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = threads;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, values...);
}
