// hs_latent_write: a token's cache row from its projection (norm of the latent channels,
// rotation of the rotary ones, the row's form) at its place; hs_latent_read: rows back
// as values.
//
// Both read each input once and write each output once, and are bound by memory.
// Writing: a warp a row; a lane has two 16-byte pieces of the latent channels (32 lanes x
// 2 x 8 = 512) and two of the 64 rotary channels, so every lane has the same work.
// Reading: 72 threads a row, 8 channels each (16 bytes of 16 bits).
#include "hs_pieces.h"
#include "hs_rotation.h"

namespace {

constexpr int kWarps = 8;  // rows of a block, writing

// The request of a token, and the row that it has in the request's context.  A warp's search in start: the last
// request that starts at or before the token (every lane gets it); -1: none.
struct Place {
    int request;
    int64_t row;
};
__device__ __forceinline__ int64_t clamped(int start, int64_t tokens) { return start < 0 ? 0 : start > tokens ? tokens : start; }
__device__ Place find_place(const int32_t* start, const int32_t* lengths, int batch, int64_t tokens, int64_t token)
{
    const int lane = threadIdx.x & 31;
    int first = 0, count = batch;
    for (;;) {
        const int step = (count + 31) >> 5, at = first + lane * step;
        const bool before = lane * step < count && clamped(start[at], tokens) <= token;
        const int n = __popc(__ballot_sync(~0u, before));
        if (n == 0) return {-1, 0};
        first += (n - 1) * step;
        count = min(step, count - (n - 1) * step);
        if (step == 1) break;
    }
    const int64_t end = clamped(start[first + 1], tokens);
    if (token >= end) return {-1, 0};
    return {first, (lengths ? (int64_t)lengths[first] - end : -clamped(start[first], tokens)) + token};
}

template <typename T, bool E4M3>
__global__ void __launch_bounds__(kWarps * 32) hs_write_kernel(const __grid_constant__ hs_write_t a)
{
    const int lane = threadIdx.x & 31;
    const int64_t token = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (token >= a.tokens) return;
    const T* x = static_cast<const T*>(a.x) + token * a.x_stride;
    uint4 in[2], wv[2];
#pragma unroll
    for (int v = 0; v < 2; ++v) in[v] = reinterpret_cast<const uint4*>(x)[v * 32 + lane];
    float2 r = unpack2<T>(reinterpret_cast<const uint32_t*>(x + HS_LATENT_DIM)[lane]);
    if (a.weight)
#pragma unroll
        for (int v = 0; v < 2; ++v) wv[v] = static_cast<const uint4*>(a.weight)[v * 32 + lane];
    Place place = {0, token};
    if (a.start) place = find_place(a.start, a.lengths, a.batch, a.tokens, token);
    if (place.request < 0 || place.row < 0 || place.row >= a.n_rows) return;
    uint8_t* out = static_cast<uint8_t*>(a.rows) + place.request * a.request_stride + place.row * a.row_stride;

    if (a.rotation != HS_ROTATE_NONE) {
        float2 t = hs_rotation(a.positions[token], a.inv_freq[lane]);  // of pair `lane`
        if (a.rotation == HS_ROTATE_PAIRS) {
            r = make_float2(r.x * t.x - r.y * t.y, r.x * t.y + r.y * t.x);
        } else {  // lanes 0-15 have both first channels of two pairs, lanes 16-31 their second ones
            const int pair = 2 * (lane & 15);
            const float c0 = __shfl_sync(~0u, t.x, pair), s0 = __shfl_sync(~0u, t.y, pair);
            const float c1 = __shfl_sync(~0u, t.x, pair + 1), s1 = __shfl_sync(~0u, t.y, pair + 1);
            const float ox = __shfl_xor_sync(~0u, r.x, 16), oy = __shfl_xor_sync(~0u, r.y, 16);
            r = lane < 16 ? make_float2(r.x * c0 - ox * s0, r.y * c1 - oy * s1)
                          : make_float2(ox * s0 + r.x * c0, oy * s1 + r.y * c1);
        }
    }
    float h[2][8];
#pragma unroll
    for (int v = 0; v < 2; ++v) Piece<T>::unpack(in[v], h[v]);
    if (a.weight) {
        float sum = 0.f;
#pragma unroll
        for (int v = 0; v < 2; ++v)
#pragma unroll
            for (int k = 0; k < 8; ++k) sum += h[v][k] * h[v][k];
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        const float f = rsqrtf(sum / HS_LATENT_DIM + a.eps);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            float w[8];
            Piece<T>::unpack(wv[v], w);
#pragma unroll
            for (int k = 0; k < 8; ++k) h[v][k] = h[v][k] * f * w[k];
        }
    }
    if constexpr (!E4M3) {
#pragma unroll
        for (int v = 0; v < 2; ++v) reinterpret_cast<uint4*>(out)[v * 32 + lane] = Piece<T>::pack(h[v]);
        reinterpret_cast<uint32_t*>(out + 2 * HS_LATENT_DIM)[lane] = pack2<T>(r.x, r.y);
    } else {
        float top = nan_max(fabsf(r.x), fabsf(r.y));
#pragma unroll
        for (int v = 0; v < 2; ++v)
#pragma unroll
            for (int k = 0; k < 8; ++k) top = nan_max(top, fabsf(h[v][k]));
        for (int o = 16; o; o >>= 1) top = nan_max(top, __shfl_xor_sync(~0u, top, o));
        const float scale = top / HS_E4M3_MAX, inv = inverse(scale);
        auto two = [&](float y0, float y1) -> uint32_t {
            if (inv != 0.f)
                quotients(y0, y1, scale, inv);
            else
                y0 = divided(y0, scale, 0.f), y1 = divided(y1, scale, 0.f);
            return __nv_cvt_float2_to_fp8x2(make_float2(y0, y1), __NV_SATFINITE, __NV_E4M3);
        };
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            uint32_t q[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) q[k] = two(h[v][4 * k], h[v][4 * k + 1]) | two(h[v][4 * k + 2], h[v][4 * k + 3]) << 16;
            reinterpret_cast<uint2*>(out)[v * 32 + lane] = make_uint2(q[0], q[1]);
        }
        reinterpret_cast<uint16_t*>(out + HS_LATENT_DIM)[lane] = (uint16_t)two(r.x, r.y);
        if (lane == 0) *reinterpret_cast<float*>(out + HS_ROW8_SCALE) = scale;
    }
}

constexpr int kRowThreads = HS_ROW_DIM / 8, kReadRows = 4;  // rows of a block

// R: the type of 16-bit rows, or void for 8-bit ones.
template <typename R, typename O> __global__ void __launch_bounds__(kRowThreads * kReadRows) hs_read_kernel(const __grid_constant__ hs_read_t a)
{
    __shared__ Place places[kReadRows];
    const int64_t first = (int64_t)blockIdx.x * kReadRows;
    if (a.start) {
        const int warp = threadIdx.x >> 5;
        if (warp < kReadRows && first + warp < a.tokens) {
            const Place p = find_place(a.start, a.lengths, a.batch, a.tokens, first + warp);
            if ((threadIdx.x & 31) == 0) places[warp] = p;
        }
        __syncthreads();
    }
    const int i = threadIdx.x / kRowThreads, ch = 8 * (threadIdx.x - i * kRowThreads);
    const int64_t token = first + i;
    if (token >= a.tokens) return;
    Place p;
    if (a.start) {
        p = places[i];
        if (p.request < 0) return;
    } else {
        p.request = (int)(token / a.entries);
        p.row = a.slots[p.request * a.slots_stride + token % a.entries];
    }
    float y[8] = {};
    if (p.row >= 0 && p.row < a.n_rows) {
        const uint8_t* row = static_cast<const uint8_t*>(a.rows) + p.request * a.request_stride + p.row * a.row_stride;
        if constexpr (std::is_void_v<R>) {
            const float scale = *reinterpret_cast<const float*>(row + HS_ROW8_SCALE);
            const uint2 v = *reinterpret_cast<const uint2*>(row + ch);
            const uint32_t w[2] = {v.x, v.y};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[k >> 1] >> 16 * (k & 1)), __NV_E4M3);
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
                y[2 * k] = f.x * scale, y[2 * k + 1] = f.y * scale;
            }
        } else {
            Piece<R>::unpack(*reinterpret_cast<const uint4*>(row + 2 * ch), y);
        }
    }
    uint4* out = reinterpret_cast<uint4*>(static_cast<O*>(a.out) + token * a.out_stride + ch);
    out[0] = Piece<O>::pack(y);
    if constexpr (sizeof(O) == 4) out[1] = Piece<O>::pack(y + 4);
}

template <typename R> cudaError_t launch_read(const hs_read_t& a, cudaStream_t s)
{
    const unsigned grid = (unsigned)((a.tokens + kReadRows - 1) / kReadRows);
    if (a.out_dtype == HS_TYPE_BF16)
        hs_read_kernel<R, __nv_bfloat16><<<grid, kRowThreads * kReadRows, 0, s>>>(a);
    else if (a.out_dtype == HS_TYPE_FP16)
        hs_read_kernel<R, __half><<<grid, kRowThreads * kReadRows, 0, s>>>(a);
    else
        hs_read_kernel<R, float><<<grid, kRowThreads * kReadRows, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T> cudaError_t launch_write(const hs_write_t& a, cudaStream_t s)
{
    const unsigned grid = (unsigned)((a.tokens + kWarps - 1) / kWarps);
    if (a.row_format == HS_ROWS_E4M3)
        hs_write_kernel<T, true><<<grid, kWarps * 32, 0, s>>>(a);
    else
        hs_write_kernel<T, false><<<grid, kWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t hs_launch_write(const hs_write_t& a, cudaStream_t s)
{
    return a.dtype == HS_TYPE_BF16 ? launch_write<__nv_bfloat16>(a, s) : launch_write<__half>(a, s);
}

cudaError_t hs_launch_read(const hs_read_t& a, cudaStream_t s)
{
    if (a.row_format == HS_ROWS_E4M3) return launch_read<void>(a, s);
    return a.dtype == HS_TYPE_BF16 ? launch_read<__nv_bfloat16>(a, s) : launch_read<__half>(a, s);
}
