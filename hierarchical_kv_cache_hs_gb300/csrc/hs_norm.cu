// hs_rms_norm: h = x + residual, y = h * rsqrt(mean(h^2) + eps) * weight,
// written in the input's type or as e4m3 with a scale for each group.
//
// A row's h stays in fp32 registers between the sum of squares and the scaling, so
// each input is read once and each output written once; the pass is bound by HBM:
// 8192 x 4096 bf16 with a residual into e4m3 in groups of 128 takes 39.2 us, 6.02 TB/s
// (0.89 of a copy's rate); 65,536 cache rows (512 + 64 channels) 31 us, 3.7 TB/s, with a
// row a warp, one in flight, and a quarter of its lanes' pieces empty.
// Rows whose pieces lie on 16-byte boundaries go through hs_norm_kernel: 16-byte
// loads, a warp a row up to 128 pieces (576 16-bit channels are 72), else 8 or 16 warps.
// Any other row (odd widths, odd alignments, groups that are not a power of two of
// pieces) goes through hs_norm_any_kernel, element by element with the row in shared
// memory, bound by its instructions: 16,000 x 1021 (fp16, residual, into e4m3) takes 92 us
// where its bytes take 17.
#include "hs_ops.h"

namespace {

__device__ __forceinline__ float nan_max(float a, float b)  // keeps a NaN
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

template <typename T> struct Piece;  // 16 bytes of T as floats
template <> struct Piece<float> {
    static constexpr int n = 4;
    static __device__ void unpack(const uint4& v, float* f)
    {
        f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
    }
    static __device__ uint4 pack(const float* f)
    {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};
template <> struct Piece<__nv_bfloat16> {
    static constexpr int n = 8;
    static __device__ void unpack(const uint4& v, float* f)
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(w[i] << 16), f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    static __device__ uint4 pack(const float* f)
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&p);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <> struct Piece<__half> {
    static constexpr int n = 8;
    static __device__ void unpack(const uint4& v, float* f)
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            f[2 * i] = p.x, f[2 * i + 1] = p.y;
        }
    }
    static __device__ uint4 pack(const float* f)
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 p = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&p);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// y / scale, rounded once.  The scale's reciprocal serves its whole group: the product with it is corrected by
// its own remainder, which one fused operation gives exactly (P. Markstein, "Computation of elementary functions
// on the IBM RISC System/6000 processor", 1990).  65,536 cache rows take 31.4 us so, 8192 x 4096 with a residual
// 39.3; 41.2 and 45.3 with a division for each value; 30.9 and 39.2 with the product alone, which leaves values
// beside a border of e4m3 on its other side (5 in 10,000 of bf16 values in groups of 16).  inv 0: a scale that is
// 0 or no ordinary number.
__device__ __forceinline__ float inverse(float scale) { return scale > 1e-30f && scale < 1e30f ? 1.f / scale : 0.f; }
__device__ __forceinline__ float quotient(float y, float scale, float inv)
{
    const float q = y * inv;
    return fmaf(fmaf(-q, scale, y), inv, q);
}
__device__ __forceinline__ void quotients(float& y0, float& y1, float scale, float inv)  // of two, in paired operations
{
    asm("{\n\t.reg .b64 y, q, s, i;\n\tmov.b64 y, {%0, %1};\n\tmov.b64 s, {%2, %2};\n\tmov.b64 i, {%3, %3};\n\t"
        "mul.rn.f32x2 q, y, i;\n\tfma.rn.f32x2 y, q, s, y;\n\tfma.rn.f32x2 q, y, i, q;\n\tmov.b64 {%0, %1}, q;\n\t}"
        : "+f"(y0), "+f"(y1)
        : "f"(-scale), "f"(inv));
}
__device__ __forceinline__ float divided(float y, float scale, float inv)
{
    return inv != 0.f ? quotient(y, scale, inv) : y / (scale == 0.f ? 1.f : scale);
}

constexpr int kWarps = 8;  // of a block, where rows do not share it
// Rows element by element: up to kAnyNarrow channels a warp a row, above kAnyWide 32 warps, else 8 (fp16,
// residual, e4m3 with one scale): 22,132 x 417 40 us against 71 with 8 warps, 20,000 x 717 67 against 87, but
// 16,000 x 1021 97 against 92; 2000 x 8191 95 with 32 warps against 125 with 8, 7 x 12739 15 against 31, but
// 3000 x 5003 92 against 82.
constexpr int kAnyNarrow = 768, kAnyWide = 6144;

// NV: 16-byte pieces a thread; TEAM: warps that share a row (1: each of the block's has
// its own).
template <typename T, bool E4M3, int NV, int TEAM>
__global__ void __launch_bounds__((TEAM == 1 ? kWarps : TEAM) * 32, TEAM == 8 && NV == 2 ? 6 : TEAM == 1 && NV == 3 ? 5 : 1)
    hs_norm_kernel(const __grid_constant__ hs_norm_t a)
{
    constexpr bool WIDE = TEAM > 1;
    constexpr int P = Piece<T>::n, kTeam = TEAM * 32;
    __shared__ float red[2][TEAM];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int me = WIDE ? threadIdx.x : lane;
    const int64_t row = WIDE ? blockIdx.x : (int64_t)blockIdx.x * kWarps + warp;
    if (!WIDE && row >= a.tokens) return;
    const int normed = a.dim / P, pieces = normed + a.carry / P;
    const uint4* x = reinterpret_cast<const uint4*>(static_cast<const T*>(a.x) + row * a.x_stride);
    const uint4* res = reinterpret_cast<const uint4*>(static_cast<const T*>(a.residual) + row * a.residual_stride);
    uint4* res_out = reinterpret_cast<uint4*>(static_cast<T*>(a.residual_out) + row * a.residual_out_stride);
    const uint4* weight = static_cast<const uint4*>(a.weight);
    float h[NV][P];
    uint4 xv[NV], rv[NV], wv[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int i = v * kTeam + me;
        xv[v] = i < pieces ? x[i] : make_uint4(0, 0, 0, 0);
        if (a.residual && i < normed) rv[v] = res[i];
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int i = v * kTeam + me;
        if (NV <= 3 && i < normed) wv[v] = weight[i];
    }
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int i = v * kTeam + me;
        Piece<T>::unpack(xv[v], h[v]);
        if (i < normed) {
            if (a.residual) {
                float r[P];
                Piece<T>::unpack(rv[v], r);
#pragma unroll
                for (int k = 0; k < P; ++k) h[v][k] += r[k];
            }
#pragma unroll
            for (int k = 0; k < P; ++k) sum += h[v][k] * h[v][k];
        }
    }
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    if constexpr (WIDE) {
        if (lane == 0) red[0][warp] = sum;
        __syncthreads();  // and every input of the row has been read: outputs may overwrite it
        sum = 0.f;
#pragma unroll
        for (int w = 0; w < TEAM; ++w) sum += red[0][w];
    } else {
        __syncwarp();
    }
    const float r = rsqrtf(sum / a.dim + a.eps);
    float top = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int i = v * kTeam + me;
        if (i < normed) {
            if (a.residual) res_out[i] = Piece<T>::pack(h[v]);
            float w[P];
            Piece<T>::unpack(NV <= 3 ? wv[v] : weight[i], w);
#pragma unroll
            for (int k = 0; k < P; ++k) h[v][k] = h[v][k] * r * w[k];
        }
        if constexpr (!E4M3) {
            if (i < pieces) reinterpret_cast<uint4*>(static_cast<T*>(a.out) + row * a.out_stride)[i] = Piece<T>::pack(h[v]);
        } else if (a.group == 0) {
#pragma unroll
            for (int k = 0; k < P; ++k) top = nan_max(top, fabsf(h[v][k]));
        }
    }
    if constexpr (E4M3) {
        float* scales = a.scales + row * a.scales_stride;
        uint8_t* out = static_cast<uint8_t*>(a.out) + row * a.out_stride;
        auto store = [&](int i, float* y, float scale) {
            if (i >= pieces) return;
            const float inv = inverse(scale);
            if (inv != 0.f)
#pragma unroll
                for (int k = 0; k < P; k += 2) quotients(y[k], y[k + 1], scale, inv);
            else
#pragma unroll
                for (int k = 0; k < P; ++k) y[k] = divided(y[k], scale, 0.f);
            uint32_t q[P / 4];
#pragma unroll
            for (int k = 0; k < P / 4; ++k)
                q[k] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(y[4 * k], y[4 * k + 1]), __NV_SATFINITE, __NV_E4M3) |
                       (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(y[4 * k + 2], y[4 * k + 3]), __NV_SATFINITE, __NV_E4M3) << 16;
            if constexpr (P == 8)
                *reinterpret_cast<uint2*>(out + i * 8) = make_uint2(q[0], q[1]);
            else
                *reinterpret_cast<uint32_t*>(out + i * 4) = q[0];
        };
        if (a.group == 0) {
            for (int o = 16; o; o >>= 1) top = nan_max(top, __shfl_xor_sync(~0u, top, o));
            if constexpr (WIDE) {
                if (lane == 0) red[1][warp] = top;
                __syncthreads();
                top = red[1][0];
#pragma unroll
                for (int w = 1; w < TEAM; ++w) top = nan_max(top, red[1][w]);
            }
            const float scale = top / HS_E4M3_MAX;
            if (me == 0) scales[0] = scale;
#pragma unroll
            for (int v = 0; v < NV; ++v) store(v * kTeam + me, h[v], scale);
        } else {
            const int lanes = a.group / P;  // a power of two: a group is this many neighbouring lanes
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int i = v * kTeam + me;
                float m = 0.f;
#pragma unroll
                for (int k = 0; k < P; ++k) m = nan_max(m, fabsf(h[v][k]));
                for (int o = 1; o < lanes; o <<= 1) m = nan_max(m, __shfl_xor_sync(~0u, m, o));
                const float scale = m / HS_E4M3_MAX;
                if (i < pieces && (lane & (lanes - 1)) == 0) scales[i / lanes] = scale;
                store(i, h[v], scale);
            }
        }
    }
}

// Any width, alignment and group: the row in shared memory.  TEAM: warps that share a
// row (1: each of the block's has its own).
template <typename T, bool E4M3, int TEAM>
__global__ void __launch_bounds__((TEAM == 1 ? kWarps : TEAM) * 32) hs_norm_any_kernel(const __grid_constant__ hs_norm_t a)
{
    constexpr int kTeam = TEAM * 32;
    extern __shared__ float rows[];  // [dim + carry], a team each
    __shared__ float red[2][TEAM];
    const int lane = threadIdx.x & 31, warp = TEAM == 1 ? 0 : threadIdx.x >> 5, at = TEAM == 1 ? lane : threadIdx.x;
    const int width = a.dim + a.carry;
    const int64_t row = TEAM == 1 ? (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= a.tokens) return;
    float* y = rows + (TEAM == 1 ? (threadIdx.x >> 5) * width : 0);
    auto sync = [] {
        if (TEAM == 1)
            __syncwarp();
        else
            __syncthreads();
    };
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* res = a.residual ? static_cast<const T*>(a.residual) + row * a.residual_stride : nullptr;
    float sum = 0.f;
#pragma unroll 4
    for (int i = at; i < width; i += kTeam) {
        float h = HsType<T>::to_float(x[i]);
        if (i < a.dim) {
            if (res) h += HsType<T>::to_float(res[i]);
            sum += h * h;
        }
        y[i] = h;
    }
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    if (TEAM > 1 && lane == 0) red[0][warp] = sum;
    sync();  // and every input of the row has been read: outputs may overwrite it
    if (TEAM > 1) {
        sum = 0.f;
        for (int w = 0; w < TEAM; ++w) sum += red[0][w];
    }
    const float r = rsqrtf(sum / a.dim + a.eps);
    float m = 0.f;  // of |y|
#pragma unroll 4
    for (int i = at; i < width; i += kTeam) {
        float v = y[i];
        if (i < a.dim) {
            if (res) static_cast<T*>(a.residual_out)[row * a.residual_out_stride + i] = HsType<T>::from_float(v);
            v = v * r * HsType<T>::to_float(static_cast<const T*>(a.weight)[i]);
        }
        if constexpr (E4M3)
            y[i] = v, m = nan_max(m, fabsf(v));
        else
            static_cast<T*>(a.out)[row * a.out_stride + i] = HsType<T>::from_float(v);
    }
    if constexpr (E4M3) {
        uint8_t* out = static_cast<uint8_t*>(a.out) + row * a.out_stride;
        auto put = [&](int i, float scale, float inv) { out[i] = __nv_cvt_float_to_fp8(divided(y[i], scale, inv), __NV_SATFINITE, __NV_E4M3); };
        float* scales = a.scales + row * a.scales_stride;
        if (a.group == 0) {  // one scale
            for (int o = 16; o; o >>= 1) m = nan_max(m, __shfl_xor_sync(~0u, m, o));
            if (TEAM > 1) {
                if (lane == 0) red[1][warp] = m;
                sync();
                for (int w = 0; w < TEAM; ++w) m = nan_max(m, red[1][w]);
            }
            const float scale = m / HS_E4M3_MAX;
            if (at == 0) *scales = scale;
            const float inv = inverse(scale);
            for (int i = at; i < width; i += kTeam) put(i, scale, inv);  // each its own y
            return;
        }
        sync();
        for (int g = warp; g * a.group < width; g += TEAM) {  // a warp a group
            const int end = min(width, (g + 1) * a.group);
            m = 0.f;
            for (int i = g * a.group + lane; i < end; i += 32) m = nan_max(m, fabsf(y[i]));
            for (int o = 16; o; o >>= 1) m = nan_max(m, __shfl_xor_sync(~0u, m, o));
            const float scale = m / HS_E4M3_MAX;
            if (lane == 0) scales[g] = scale;
            const float inv = inverse(scale);
            for (int i = g * a.group + lane; i < end; i += 32) put(i, scale, inv);
        }
    }
}

template <typename T, bool E4M3, int TEAM> cudaError_t launch_any(const hs_norm_t& a, cudaStream_t s)
{
    constexpr int rows = TEAM == 1 ? kWarps : 1;
    const size_t smem = sizeof(float) * (size_t)(a.dim + a.carry) * rows;
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(hs_norm_any_kernel<T, E4M3, TEAM>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)sizeof(float) * HS_MAX_NORM_DIM);
        if (e != cudaSuccess) return e;
    }
    hs_norm_any_kernel<T, E4M3, TEAM><<<(unsigned)((a.tokens + rows - 1) / rows), (TEAM == 1 ? kWarps : TEAM) * 32, smem, s>>>(a);
    return cudaGetLastError();
}

template <typename T, bool E4M3> cudaError_t launch(const hs_norm_t& a, cudaStream_t s)
{
    constexpr int P = Piece<T>::n, el = sizeof(T);
    auto fits = [](const void* p, int64_t stride_bytes, int64_t rows, uintptr_t to) {
        return ((uintptr_t)p % to) == 0 && (rows <= 1 || stride_bytes % (int64_t)to == 0);
    };
    bool pieces16 = a.dim % P == 0 && a.carry % P == 0 && fits(a.x, a.x_stride * el, a.tokens, 16) &&
                    fits(a.weight, 0, 1, 16) && fits(a.residual, a.residual_stride * el, a.tokens, 16) &&
                    fits(a.residual_out, a.residual_out_stride * el, a.tokens, 16) &&
                    (E4M3 ? fits(a.out, a.out_stride, a.tokens, P) : fits(a.out, a.out_stride * el, a.tokens, 16));
    if (E4M3 && a.group) {
        const int lanes = a.group / P;
        pieces16 = pieces16 && a.group % P == 0 && lanes <= 32 && (lanes & (lanes - 1)) == 0;
    }
    const int pieces = (a.dim + a.carry) / P;
    if (!pieces16) {
        const int width = a.dim + a.carry;
        return width <= kAnyNarrow ? launch_any<T, E4M3, 1>(a, s) : width <= kAnyWide ? launch_any<T, E4M3, 8>(a, s) : launch_any<T, E4M3, 32>(a, s);
    } else if (pieces <= 128) {
        // A warp a row (residual, bf16): 1024 channels x 65,536 rows 81 us in 16 bits, 77 into e4m3, against 93
        // and 119 with eight warps a row; 2048 channels (256 pieces) 84 and 99 against 79 and 81.
        const unsigned grid = (unsigned)((a.tokens + kWarps - 1) / kWarps);
        if (pieces <= 32)
            hs_norm_kernel<T, E4M3, 1, 1><<<grid, kWarps * 32, 0, s>>>(a);
        else if (pieces <= 96)
            hs_norm_kernel<T, E4M3, 3, 1><<<grid, kWarps * 32, 0, s>>>(a);
        else
            hs_norm_kernel<T, E4M3, 4, 1><<<grid, kWarps * 32, 0, s>>>(a);
    } else {
        // Eight warps: 4096 channels x 16,384 rows into e4m3 74 us against 98 with 16, 8192 x 8192 78 against 93;
        // 16 warps from there: 12288 x 5461 94 against 119, 16384 x 4096 84 against 103.
        const unsigned grid = (unsigned)a.tokens;
        if (pieces <= 256)
            hs_norm_kernel<T, E4M3, 1, 8><<<grid, 256, 0, s>>>(a);
        else if (pieces <= 512)
            hs_norm_kernel<T, E4M3, 2, 8><<<grid, 256, 0, s>>>(a);
        else if (pieces <= 1024)
            hs_norm_kernel<T, E4M3, 4, 8><<<grid, 256, 0, s>>>(a);
        else if (pieces <= 2048)
            hs_norm_kernel<T, E4M3, 4, 16><<<grid, 512, 0, s>>>(a);
        else
            hs_norm_kernel<T, E4M3, 8, 16><<<grid, 512, 0, s>>>(a);
    }
    return cudaGetLastError();
}

template <typename T> cudaError_t launch(const hs_norm_t& a, cudaStream_t s)
{
    return a.scales ? launch<T, true>(a, s) : launch<T, false>(a, s);
}

}  // namespace

cudaError_t hs_launch_norm(const hs_norm_t& a, cudaStream_t s)
{
    if (a.dtype == HS_TYPE_BF16) return launch<__nv_bfloat16>(a, s);
    if (a.dtype == HS_TYPE_FP16) return launch<__half>(a, s);
    return launch<float>(a, s);
}
