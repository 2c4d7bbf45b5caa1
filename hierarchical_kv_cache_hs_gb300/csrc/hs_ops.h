// Private declarations of the operators beside the swap-in path
// (hs_latent_attend, hs_latent_attend_shared, hs_latent_prefill, hs_rms_norm,
// hs_latent_write, hs_latent_read, hs_norm_rotate).
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
// after: the call's kernels may begin while the one before them in the stream runs, which has to come from the same call
// and let them; what is launched behind them with launch_after begins when that one is done.  pairs: of SMs that it may
// take (0: all).  wide: where outputs go instead of a.out, [batch][positions][heads][512], unrounded.
cudaError_t hs_launch_attend(const hs_attend_t& a, cudaStream_t s, bool after = false, int pairs = 0, float* wide = nullptr);
cudaError_t hs_launch_prefill(const hs_prefill_t& a, cudaStream_t s);
cudaError_t hs_launch_norm(const hs_norm_t& a, cudaStream_t s);
cudaError_t hs_launch_write(const hs_write_t& a, cudaStream_t s);
cudaError_t hs_launch_read(const hs_read_t& a, cudaStream_t s);
cudaError_t hs_launch_rotate(const hs_rotate_t& a, cudaStream_t s);
cudaError_t hs_launch_attend_shared(const hs_attend_t& a, const hs_prefix_t& p, cudaStream_t s);
size_t hs_attend_workspace_bytes(int batch, int positions, int heads, int64_t rows);
size_t hs_prefill_workspace_bytes(int64_t k_tokens, int heads);
size_t hs_attend_shared_workspace_bytes(int batch, int positions, int heads, int64_t rows, int64_t prefix_rows);

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
// Its blocks in clusters of `cluster` where the kernel itself says nothing of them.
template <typename... Params, typename... Values>
cudaError_t launch_after_clusters(unsigned cluster, void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t s, Values... values)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = threads;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cluster > 1) {
        at[1].id = cudaLaunchAttributeClusterDimension;
        at[1].val.clusterDim.x = cluster;
        at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, kernel, values...);
}
template <typename... Params, typename... Values>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t s, Values... values)
{
    return launch_after_clusters(1, kernel, grid, threads, smem, s, values...);
}
