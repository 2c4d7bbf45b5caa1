// hs_latent_write: a token's cache row from its projection (norm of the latent channels,
// rotation of the rotary ones, the row's form) at its place; hs_latent_read: rows back
// as values.
//
//   y = [c w / sqrt(mean c^2 + eps) ; R r],  R: pairs turned by position x frequency
//   16-bit rows: y rounded; 8-bit rows: s = max |y| / 448, e4m3(y / s)
//   back: the row's values, times s, rounded once to the output's type
//
// Each input is read once and each output written once (1156 + 592 bytes a token written as an 8-bit row), so the
// floor is memory's.  Inputs larger than L2, on one GB300:
//   writing 65,536 rows of 8 bits   23.6 us, 4.8 TB/s, 0.71 of a copy's rate: some 275 instructions a row, which
//                                   take 67 % of the issue slots, and what a warp does between its loads
//   reading 64 x 2048 8-bit rows by slots   37.0 us, 6.2 TB/s, 0.91 of a copy's rate: memory
//   64 rows written, 3 x 77 read    2.4 and 2.8 us: a launch and the latency of two loads in a row
//   65,536 rows into a handle's host pool   395 us of 16 bits, 191 GB/s (a copy to the host 193); 262 of 8 bits, 148
//   65,536 rows read from it        364 us of 16 bits, 208 GB/s (a copy from the host 210); 204 of 8 bits, 186
// (Times at choices further on are of the step that took them.)
#include "hs_pieces.h"
#include "hs_rotation.h"
#include "hs_tc.h"

namespace {

__device__ __forceinline__ int64_t clamped(int start, int64_t tokens) { return start < 0 ? 0 : start > tokens ? tokens : start; }

// The request that a token may belong to: a warp searches start for the last one that starts at or before it.
__device__ int find_request(const int32_t* start, int batch, int64_t tokens, int64_t token)  // every lane gets it; -1: none
{
    const int lane = threadIdx.x & 31;
    int first = 0, count = batch;
    for (;;) {
        const int step = (count + 31) >> 5;
        const bool before = lane * step < count && clamped(start[first + lane * step], tokens) <= token;
        const int n = __popc(__ballot_sync(~0u, before));
        if (n == 0) return -1;
        first += (n - 1) * step;
        count = min(step, count - (n - 1) * step);
        if (step == 1) return first;
    }
}
// Which requests tokens belong to: 32 requests' starts and lengths in a warp's lanes.  In a batch of more a search finds
// where they begin; fewer need none, which is a load's latency less.  Reading 512 contexts of 77 8-bit rows took 17.3 us
// with a search for each request of a block, and takes 13.5.
struct Span {
    int request;  // -1: the token has none
    int begin, end;
    int length;
};
struct Window {
    int first, start, length;  // this lane's: of request first + lane (start: also of `batch`)
    __device__ Window(const int32_t* starts, const int32_t* lengths, int batch, int64_t tokens, int64_t token)
    {
        first = batch < 32 ? 0 : max(find_request(starts, batch, tokens, token), 0);
        const int i = first + (int)(threadIdx.x & 31);
        start = (int)clamped(starts[min(i, batch)], tokens);  // below 2^24
        length = lengths ? lengths[min(i, batch - 1)] : 0;
    }
    // The request of a token (each lane its own) if it is among the window's but the last, else `beyond`.
    __device__ Span find(int batch, int token, bool& beyond) const
    {
        int at = 0;
#pragma unroll
        for (int step = 16; step; step >>= 1) {
            const int s = __shfl_sync(~0u, start, at + step);
            if (first + at + step < batch && s <= token) at += step;
        }
        Span f = {first + at, __shfl_sync(~0u, start, at), __shfl_sync(~0u, start, (at + 1) & 31), __shfl_sync(~0u, length, at)};
        beyond = at == 31;
        if (token < f.begin || token >= f.end) f.request = -1;
        return f;
    }
};

// ---- write -----------------------------------------------------------------------------
//
// A warp takes some tokens, one after the other, with the next one's channels on their way, and those of the one after
// to L2 (16-bit rows 27.8 -> 26.4 us, 8-bit ones without a norm 23.3 -> 21.1, with one 24.3 both).  A lane has two
// 16-byte pieces of the latent channels (32 lanes x 2 x 8 = 512) and two of the 64 rotary channels, so every lane
// has the same work; the weights and its pair's frequency stay in registers.  A block's tokens are neighbours, and its
// warps take them by turns, so that the rows that are written at one time lie side by side.  (A warp for each token
// alone, with its own loads of the weights: 34 us for the 24.3 above.)

constexpr int kWarps = 8;        // of a block
constexpr int kWriteBlocks = 3;  // an SM, at most 80 registers a thread (65,536 rows, 2 / 3 / 4 blocks: 30.3 / 27.0 / 27.6 us when it was chosen)

__device__ __forceinline__ void square2(float& s0, float& s1, float a0, float a1)  // added to the sums
{
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%0, %1};\n\tfma.rn.f32x2 y, x, x, y;\n\tmov.b64 {%0, %1}, y;\n\t}"
        : "+f"(s0), "+f"(s1)
        : "f"(a0), "f"(a1));
}
__device__ __forceinline__ float top3(float a, float b, float c)  // of magnitudes; keeps a NaN
{
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float warp_top(float v)  // likewise
{
    float d;
    asm("redux.sync.max.abs.NaN.f32 %0, %1, 0xffffffff;" : "=f"(d) : "f"(v));
    return d;
}

__device__ __forceinline__ void product2(float& a0, float& a1, float b, float rest)  // with b + rest, rounded once
{
    asm("{\n\t.reg .b64 a, b, r;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %2};\n\tmov.b64 r, {%3, %3};\n\t"
        "mul.rn.f32x2 r, a, r;\n\tfma.rn.f32x2 a, a, b, r;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "+f"(a0), "+f"(a1)
        : "f"(b), "f"(rest));
}

__device__ __noinline__ float rare_quotient(float y, float scale) { return divided(y, scale, 0.f); }

template <typename T, bool E4M3>
__global__ void __launch_bounds__(kWarps * 32, kWriteBlocks) hs_write_kernel(const __grid_constant__ hs_write_t a)
{
    const int lane = threadIdx.x & 31;
    constexpr int step = kWarps;
    const int first = (int)(a.tokens * blockIdx.x / gridDim.x) + (threadIdx.x >> 5);  // below 2^24
    const int last = (int)(a.tokens * (blockIdx.x + 1) / gridDim.x);
    if (first >= last) return;
    uint4 weight[2];
    if (a.weight)
#pragma unroll
        for (int v = 0; v < 2; ++v) weight[v] = static_cast<const uint4*>(a.weight)[v * 32 + lane];
    HsTurn freq = {0, true};
    if (a.rotation != HS_ROTATE_NONE) freq = hs_turn(a.inv_freq[lane]);
    // The tokens up to `end` belong to one request, or to none; those in [low, high) have a row, this one at `out`.
    int end = a.start ? first : last, low = first, high = last;
    uint8_t* out = static_cast<uint8_t*>(a.rows) + first * a.row_stride;

    const T* x = static_cast<const T*>(a.x) + first * a.x_stride;
    uint4 in[2];
    uint32_t rope;
    int position = 0;
    auto bring = [&](int token) {
#pragma unroll
        for (int v = 0; v < 2; ++v) in[v] = reinterpret_cast<const uint4*>(x)[v * 32 + lane];
        rope = reinterpret_cast<const uint32_t*>(x + HS_LATENT_DIM)[lane];
        if (a.rotation != HS_ROTATE_NONE) position = a.positions[token];
        x += step * a.x_stride;
        if (lane < 9 && token + 2 * step < last) tc::prefetch_l2(reinterpret_cast<const uint8_t*>(x + step * a.x_stride) + 128 * lane);
    };
    bring(first);
    for (int token = first; token < last; token += step, out += step * a.row_stride) {
        float h[2][8];
#pragma unroll
        for (int v = 0; v < 2; ++v) Piece<T>::unpack(in[v], h[v]);
        float2 r = unpack2<T>(rope);
        const int at = position;
        if (token + step < last) bring(token + step);
        if (token >= end) {
            bool beyond;
            const Span f = Window(a.start, a.lengths, a.batch, a.tokens, token).find(a.batch, token, beyond);
            low = high = end = token + 1;
            if (f.request >= 0) {
                const int64_t zero = (int64_t)f.end - f.length;  // the token whose row is 0
                end = f.end;
                low = (int)min(max(zero, (int64_t)0), a.tokens);
                high = (int)min(max(zero + a.n_rows, (int64_t)0), a.tokens);
                out = static_cast<uint8_t*>(a.rows) + f.request * a.request_stride + (token - zero) * a.row_stride;
            }
        }
        if (token < low || token >= high) continue;

        if (a.rotation != HS_ROTATE_NONE) {
            const float2 t = hs_rotation(at, freq);  // of pair `lane`
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
        float f = 1.f;
        if (a.weight) {
            float sum = 0.f, odd = 0.f;
#pragma unroll
            for (int v = 0; v < 2; ++v)
#pragma unroll
                for (int k = 0; k < 8; k += 2) square2(sum, odd, h[v][k], h[v][k + 1]);
            sum += odd;
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
            f = rsqrtf(sum / HS_LATENT_DIM + a.eps);
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                float w[8];
                Piece<T>::unpack(weight[v], w);
#pragma unroll
                for (int k = 0; k < 8; k += 2) {
                    if constexpr (!E4M3) mul2(h[v][k], h[v][k + 1], f, f);
                    mul2(h[v][k], h[v][k + 1], w[k], w[k + 1]);
                }
            }
        }
        if constexpr (!E4M3) {
#pragma unroll
            for (int v = 0; v < 2; ++v) reinterpret_cast<uint4*>(out)[v * 32 + lane] = Piece<T>::pack(h[v]);
            reinterpret_cast<uint32_t*>(out + 2 * HS_LATENT_DIM)[lane] = pack2<T>(r.x, r.y);
        } else {
            // h: x w, exact products of 16-bit values, to be multiplied by f.  The quotients by max |y| / 448 are products
            // with 448 f / max |y| (of the rotary channels 448 / max |y|) in two floats each, so that only one rounding
            // is left in them: fewer values beside a border of e4m3 fall to its other side.
            float tops[2] = {0.f, nan_max(fabsf(r.x), fabsf(r.y))};
#pragma unroll
            for (int v = 0; v < 2; ++v)
#pragma unroll
                for (int k = 0; k < 8; k += 2) tops[0] = top3(tops[0], h[v][k], h[v][k + 1]);
            tops[0] = warp_top(tops[0]), tops[1] = warp_top(tops[1]);
            const float y = tops[0] * f, top = nan_max(y, tops[1]), rest = y > tops[1] ? fmaf(tops[0], f, -y) : 0.f;
            const float scale = top / HS_E4M3_MAX, inv = 1.f / top;
            const float by = HS_E4M3_MAX * inv, by_rest = (fmaf(-by, top, HS_E4M3_MAX) - by * rest) * inv;
            const float by_f = by * f, by_f_rest = fmaf(by, f, -by_f) + by_rest * f;
            if (inverse(scale) != 0.f && by_f > 1e-30f && by_f < 1e30f) {
#pragma unroll
                for (int v = 0; v < 2; ++v)
#pragma unroll
                    for (int k = 0; k < 8; k += 2) product2(h[v][k], h[v][k + 1], by_f, by_f_rest);
                product2(r.x, r.y, by, by_rest);
            } else {  // zeros, or beyond what a reciprocal serves
#pragma unroll
                for (int v = 0; v < 2; ++v)
#pragma unroll
                    for (int k = 0; k < 8; ++k) h[v][k] = rare_quotient(h[v][k] * f, scale);
                r = make_float2(rare_quotient(r.x, scale), rare_quotient(r.y, scale));
            }
            auto two = [](float y0, float y1) -> uint32_t { return __nv_cvt_float2_to_fp8x2(make_float2(y0, y1), __NV_SATFINITE, __NV_E4M3); };
#pragma unroll
            for (int v = 0; v < 2; ++v)
                reinterpret_cast<uint2*>(out)[v * 32 + lane] = make_uint2(two(h[v][0], h[v][1]) | two(h[v][2], h[v][3]) << 16,
                                                                         two(h[v][4], h[v][5]) | two(h[v][6], h[v][7]) << 16);
            reinterpret_cast<uint16_t*>(out + HS_LATENT_DIM)[lane] = (uint16_t)two(r.x, r.y);
            // with the row's last 12 bytes: rows side by side then leave no sector half written (27.0 -> 25.1 us, 65,536 rows)
            if (lane == 0) *reinterpret_cast<float4*>(out + HS_ROW8_SCALE) = make_float4(scale, 0.f, 0.f, 0.f);
        }
    }
}

// ---- read ------------------------------------------------------------------------------
//
// 36 threads a row, 16 channels each, and kReadAhead rows of a thread on their way together: a load of 16 bytes (32 of
// 16-bit rows) and stores of 32.  One row a thread and loads and stores of 16 bytes took 63 us where this takes 37; 2, 3
// and 4 rows a thread 36.6, 36.9 and 37.5.  (Few rows are no faster with fewer a thread: a launch bounds them.)

constexpr int kReadLine = 8, kReadAhead = 3;       // rows side by side, rows of a thread
constexpr int kReadRows = kReadLine * kReadAhead;  // of a block
static_assert(kReadRows <= 32, "a warp finds the rows");

// R: the type of 16-bit rows, or void for 8-bit ones.
template <typename R, typename O>
__global__ void __launch_bounds__(kRowThreads * kReadLine) hs_read_kernel(const __grid_constant__ hs_read_t a, const bool rows32, const bool out32)
{
    __shared__ const uint8_t* places[kReadRows];  // a row's address; NULL: zeros
    __shared__ bool mine[kReadRows];              // an out row of a request
    const int64_t first = (int64_t)blockIdx.x * kReadRows;
    if (threadIdx.x < 32) {
        const int64_t token = first + threadIdx.x;
        const bool there = threadIdx.x < kReadRows && token < a.tokens;
        int request = -1;
        int64_t row = -1;
        if (a.start) {
            bool beyond;
            Span s = Window(a.start, a.lengths, a.batch, a.tokens, first).find(a.batch, there ? (int)token : 0, beyond);
            for (unsigned left = __ballot_sync(~0u, there && beyond); left; left &= left - 1) {  // behind many empty requests
                const int from = __ffs(left) - 1;
                const Span f = Window(a.start, a.lengths, a.batch, a.tokens, first + from).find(a.batch, (int)first + from, beyond);
                if ((int)threadIdx.x == from) s = f;
            }
            if (there && s.request >= 0) request = s.request, row = a.lengths ? (int64_t)s.length - s.end + token : token - s.begin;
        } else if (there) {
            request = (int)(token / a.entries);
            row = a.slots[request * a.slots_stride + token % a.entries];
        }
        if (threadIdx.x < kReadRows) {
            mine[threadIdx.x] = request >= 0;
            places[threadIdx.x] = request >= 0 && row >= 0 && row < a.n_rows
                                      ? static_cast<const uint8_t*>(a.rows) + request * a.request_stride + row * a.row_stride
                                      : nullptr;
        }
    }
    __syncthreads();
    const int line = threadIdx.x / kRowThreads, ch = 16 * (threadIdx.x - line * kRowThreads);
    uint4 v[kReadAhead][std::is_void_v<R> ? 1 : 2];
    float scale[kReadAhead];
#pragma unroll
    for (int n = 0; n < kReadAhead; ++n) {
        const uint8_t* row = places[n * kReadLine + line];
        scale[n] = 0.f;
        if constexpr (std::is_void_v<R>) {
            v[n][0] = make_uint4(0, 0, 0, 0);
            if (row) v[n][0] = *reinterpret_cast<const uint4*>(row + ch), scale[n] = *reinterpret_cast<const float*>(row + HS_ROW8_SCALE);
        } else {
            v[n][0] = v[n][1] = make_uint4(0, 0, 0, 0);
            if (row) load32(row + 2 * ch, rows32, v[n]);
        }
    }
#pragma unroll
    for (int n = 0; n < kReadAhead; ++n) {
        const int i = n * kReadLine + line;
        if (!mine[i]) continue;
        O* out = static_cast<O*>(a.out) + (first + i) * a.out_stride + ch;
        if constexpr (std::is_same_v<R, O>) {
            store32(out, out32, v[n][0], v[n][1]);
        } else {
            float y[16];
            if constexpr (std::is_void_v<R>) {
                const uint32_t e[4] = {v[n][0].x, v[n][0].y, v[n][0].z, v[n][0].w};
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(e[k >> 1] >> 16 * (k & 1)), __NV_E4M3);
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
                    y[2 * k] = f.x * scale[n], y[2 * k + 1] = f.y * scale[n];
                }
            } else {
                Piece<R>::unpack(v[n][0], y);
                Piece<R>::unpack(v[n][1], y + 8);
            }
            constexpr int P = Piece<O>::n;
#pragma unroll
            for (int k = 0; k < 16; k += 2 * P) store32(out + k, out32, Piece<O>::pack(y + k), Piece<O>::pack(y + k + P));
        }
    }
}

template <typename R, typename O> void launch_read(const hs_read_t& a, cudaStream_t s)
{
    auto fits = [](const void* p, int64_t stride) { return (uintptr_t)p % 32 == 0 && stride % 32 == 0; };
    const bool rows32 = !std::is_void_v<R> && fits(a.rows, a.row_stride | (a.batch > 1 ? a.request_stride : 0));
    const bool out32 = fits(a.out, a.tokens > 1 ? a.out_stride * (int64_t)sizeof(O) : 0);
    hs_read_kernel<R, O><<<(unsigned)((a.tokens + kReadRows - 1) / kReadRows), kRowThreads * kReadLine, 0, s>>>(a, rows32, out32);
}
template <typename R> cudaError_t launch_read(const hs_read_t& a, cudaStream_t s)
{
    if (a.out_dtype == HS_TYPE_BF16)
        launch_read<R, __nv_bfloat16>(a, s);
    else if (a.out_dtype == HS_TYPE_FP16)
        launch_read<R, __half>(a, s);
    else
        launch_read<R, float>(a, s);
    return cudaGetLastError();
}

template <typename T> cudaError_t launch_write(const hs_write_t& a, cudaStream_t s)
{
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int64_t most = (int64_t)sms * kWriteBlocks, blocks = (a.tokens + kWarps - 1) / kWarps;
    const unsigned grid = (unsigned)(blocks < most ? blocks : most);
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
