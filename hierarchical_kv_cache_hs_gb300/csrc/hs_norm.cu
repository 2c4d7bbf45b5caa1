// hs_rms_norm: h = x + residual, y = h * rsqrt(mean(h^2) + eps) * weight,
// written in the input's type or as e4m3 with a scale for each group.
//
// One CTA per row.  The row's h stays in registers between the sum of squares
// and the scaling, so each input is read once and each output written once;
// the pass is bound by HBM.
#include "hs_ops.h"

namespace {

constexpr int kThreads = 256;

__device__ float block_sum(float v, float* red)
{
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.f;
    for (int i = 0; i < kThreads / 32; ++i) t += red[i];
    __syncthreads();
    return t;
}

// max that keeps a NaN
__device__ float nan_max(float a, float b) { return a != a ? a : (b != b ? b : fmaxf(a, b)); }

template <typename T, bool E4M3>
__global__ void __launch_bounds__(kThreads) hs_norm_kernel(hs_norm_t a)
{
    extern __shared__ float y[];  // [dim + carry]
    __shared__ float red[kThreads / 32];
    const int64_t row = blockIdx.x;
    const int width = a.dim + a.carry;
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* res = a.residual ? static_cast<const T*>(a.residual) + row * a.residual_stride : nullptr;
    float sum = 0.f;
    for (int i = threadIdx.x; i < width; i += kThreads) {
        float h = HsType<T>::to_float(x[i]);
        if (i < a.dim) {
            if (res) h += HsType<T>::to_float(res[i]);
            sum += h * h;
        }
        y[i] = h;
    }
    sum = block_sum(sum, red);
    const float r = rsqrtf(sum / a.dim + a.eps);
    for (int i = threadIdx.x; i < a.dim; i += kThreads) {
        const float h = y[i];
        if (res)
            static_cast<T*>(a.residual_out)[row * a.residual_out_stride + i] = HsType<T>::from_float(h);
        y[i] = h * r * HsType<T>::to_float(static_cast<const T*>(a.weight)[i]);
    }
    __syncthreads();
    if constexpr (!E4M3) {
        T* out = static_cast<T*>(a.out) + row * a.out_stride;
        for (int i = threadIdx.x; i < width; i += kThreads) out[i] = HsType<T>::from_float(y[i]);
    } else {
        uint8_t* out = static_cast<uint8_t*>(a.out) + row * a.out_stride;
        const int group = a.group ? a.group : width;
        const int groups = (width + group - 1) / group;
        for (int g = threadIdx.x >> 5; g < groups; g += kThreads / 32) {  // a warp per group
            const int end = min(width, (g + 1) * group);
            float m = 0.f;
            for (int i = g * group + (threadIdx.x & 31); i < end; i += 32) m = nan_max(m, fabsf(y[i]));
            for (int o = 16; o; o >>= 1) m = nan_max(m, __shfl_xor_sync(~0u, m, o));
            const float scale = m / HS_E4M3_MAX;
            if ((threadIdx.x & 31) == 0) a.scales[row * a.scales_stride + g] = scale;
            for (int i = g * group + (threadIdx.x & 31); i < end; i += 32)
                out[i] = __nv_cvt_float_to_fp8(scale == 0.f ? y[i] : y[i] / scale, __NV_SATFINITE, __NV_E4M3);
        }
    }
}

template <typename T>
cudaError_t launch(const hs_norm_t& a, cudaStream_t s)
{
    const size_t smem = sizeof(float) * (size_t)(a.dim + a.carry);
    auto k = a.scales ? hs_norm_kernel<T, true> : hs_norm_kernel<T, false>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)sizeof(float) * HS_MAX_NORM_DIM);
    if (e != cudaSuccess) return e;
    k<<<(unsigned)a.tokens, kThreads, smem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t hs_launch_norm(const hs_norm_t& a, cudaStream_t s)
{
    if (a.dtype == HS_TYPE_BF16) return launch<__nv_bfloat16>(a, s);
    if (a.dtype == HS_TYPE_FP16) return launch<__half>(a, s);
    return launch<float>(a, s);
}
