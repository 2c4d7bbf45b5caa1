// hs_norm_rotate: the norm of each head's channels and their rotation, in one pass over
// the queries and keys of a token.
//
// Bound by memory: each element is read once and written once.  A warp takes some heads
// of one token.  Its lanes form teams of 8, 16 or 32, a head each, and a lane has the
// same channels of every head that its team passes over: its weights, sines and cosines
// stay in registers.  A lane's channels come in units of 16 bytes, as two halves of 8
// that lie side by side or, for pairs whose channels are half of the rotary ones apart,
// that far apart: so a pair is always within a lane.
// Heads that are not in such units go element by element through shared memory.
#include "hs_pieces.h"
#include "hs_rotation.h"

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kWarpsEnough = 24;  // an SM

struct RotateArgs {
    hs_rotate_t a;
    int heads_warp;      // of a warp, all of one array
    int chunks[2];       // warps that share a token's queries, and its keys
    int team;            // lanes of a head
    int tokens_block, heads_block;  // of a block (element by element)
};

template <typename T> struct Half;  // 8 bytes of T as floats
template <> struct Half<float> {
    static constexpr int n = 2;
    static __device__ void unpack(const uint2& v, float* f) { f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y); }
    static __device__ uint2 pack(const float* f) { return make_uint2(__float_as_uint(f[0]), __float_as_uint(f[1])); }
};
template <typename T> struct Half16 {
    static constexpr int n = 4;
    static __device__ void unpack(const uint2& v, float* f)
    {
        const float2 a = unpack2<T>(v.x), b = unpack2<T>(v.y);
        f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
    }
    static __device__ uint2 pack(const float* f) { return make_uint2(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3])); }
};
template <> struct Half<__nv_bfloat16> : Half16<__nv_bfloat16> {};
template <> struct Half<__half> : Half16<__half> {};

// NV: units a lane, AHEAD: heads of a team on their way together.
template <typename T, int NV, int AHEAD> __global__ void __launch_bounds__(kThreads) hs_rotate_kernel(const __grid_constant__ RotateArgs g)
{
    constexpr int H = Half<T>::n, U = 2 * H;  // channels of half a unit, of a unit
    extern __shared__ float2 sines[];         // [warp][pair]
    const hs_rotate_t& a = g.a;
    const int lane = threadIdx.x & 31, all = g.chunks[0] + g.chunks[1];
    const int64_t id = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5), token = id / all;
    if (token >= a.tokens) return;
    int chunk = (int)(id - token * all);
    const int k = chunk >= g.chunks[0];  // queries or keys
    chunk -= k ? g.chunks[0] : 0;
    const int pairs = a.rope / 2, units = a.dim / U;
    const bool paired = a.rotation == HS_ROTATE_PAIRS;
    float2* turns = sines + (threadIdx.x >> 5) * pairs;
    if (pairs) {
        const int position = a.positions[token];
        for (int i = lane; i < pairs; i += 32) turns[i] = hs_rotation(position, hs_turn(a.inv_freq[i]));
        __syncwarp();
    }

    // This lane's units: where their halves lie, their weights, the sines and cosines of their pairs.
    const int at = lane & (g.team - 1), teams = 32 / g.team;
    const T* weight = static_cast<const T*>(a.weight[k]);
    int low[NV], high[NV];
    bool turned[NV], mine[NV];
    uint2 wl[NV], wh[NV];
    float2 turn[NV][H];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int u = v * g.team + at;
        mine[v] = u < units;
        int c = u * U;
        high[v] = c + H;
        const int n = c - a.rope_at;
        turned[v] = mine[v] && n >= 0 && n < a.rope;
        if (turned[v] && !paired) {  // unit i of the rotary channels: H from either half of them
            c = a.rope_at + n / 2;
            high[v] = c + pairs;
        }
        low[v] = c;
        if (weight && mine[v]) {
            wl[v] = *reinterpret_cast<const uint2*>(weight + low[v]);
            wh[v] = *reinterpret_cast<const uint2*>(weight + high[v]);
        }
#pragma unroll
        for (int i = 0; i < H; ++i) turn[v][i] = turned[v] ? turns[n / 2 + i] : make_float2(1.f, 0.f);
    }

    const int first = chunk * g.heads_warp + lane / g.team, last = min((chunk + 1) * g.heads_warp, a.heads[k]);
    const T* x = static_cast<const T*>(a.x[k]) + token * a.x_stride[k][0];
    T* out = static_cast<T*>(a.out[k]) + token * a.out_stride[k][0];
    for (int head0 = first; head0 - lane / g.team < last; head0 += AHEAD * teams) {  // the whole warp
        uint2 xl[AHEAD][NV], xh[AHEAD][NV];
#pragma unroll
        for (int m = 0; m < AHEAD; ++m) {
            const int head = head0 + m * teams;
            const T* from = x + head * a.x_stride[k][1];
#pragma unroll
            for (int v = 0; v < NV; ++v)
                if (mine[v] && head < last) {
                    xl[m][v] = *reinterpret_cast<const uint2*>(from + low[v]);
                    xh[m][v] = *reinterpret_cast<const uint2*>(from + high[v]);
                } else {
                    xl[m][v] = xh[m][v] = make_uint2(0, 0);
                }
        }
        float f[AHEAD];
        if (weight) {
#pragma unroll
            for (int m = 0; m < AHEAD; ++m) {
                f[m] = 0.f;
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    float y[U];
                    Half<T>::unpack(xl[m][v], y), Half<T>::unpack(xh[m][v], y + H);
#pragma unroll
                    for (int i = 0; i < U; ++i) f[m] += y[i] * y[i];
                }
            }
            for (int o = g.team >> 1; o; o >>= 1)
#pragma unroll
                for (int m = 0; m < AHEAD; ++m) f[m] += __shfl_xor_sync(~0u, f[m], o);
#pragma unroll
            for (int m = 0; m < AHEAD; ++m) f[m] = rsqrtf(f[m] / a.dim + a.eps);
        }
        __syncwarp();  // the heads' channels have been read: outputs may overwrite them
#pragma unroll
        for (int m = 0; m < AHEAD; ++m) {
            const int head = head0 + m * teams;
            if (head >= last) break;
            T* to = out + head * a.out_stride[k][1];
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (!mine[v]) continue;
                float y[U];
                Half<T>::unpack(xl[m][v], y), Half<T>::unpack(xh[m][v], y + H);
                if (weight) {
                    float w[U];
                    Half<T>::unpack(wl[v], w), Half<T>::unpack(wh[v], w + H);
#pragma unroll
                    for (int i = 0; i < U; ++i) y[i] = y[i] * f[m] * w[i];
                }
                auto rotate = [&](float& p, float& q, const float2& r) {
                    const float p0 = p, q0 = q;
                    p = p0 * r.x - q0 * r.y;
                    q = p0 * r.y + q0 * r.x;
                };
                if (turned[v] && paired)
#pragma unroll
                    for (int i = 0; i < H; ++i) rotate(y[2 * i], y[2 * i + 1], turn[v][i]);
                else if (turned[v])
#pragma unroll
                    for (int i = 0; i < H; ++i) rotate(y[i], y[H + i], turn[v][i]);
                *reinterpret_cast<uint2*>(to + low[v]) = Half<T>::pack(y);
                *reinterpret_cast<uint2*>(to + high[v]) = Half<T>::pack(y + H);
            }
        }
    }
}

template <typename T> struct Head {  // one of a token's heads, of either array
    const T* x;
    T* out;
    const T* weight;
};
template <typename T> __device__ __forceinline__ Head<T> head_of(const hs_rotate_t& a, int64_t token, int head)
{
    const int k = head >= a.heads[0];
    head -= k ? a.heads[0] : 0;
    return {static_cast<const T*>(a.x[k]) + token * a.x_stride[k][0] + head * a.x_stride[k][1],
            static_cast<T*>(a.out[k]) + token * a.out_stride[k][0] + head * a.out_stride[k][1],
            static_cast<const T*>(a.weight[k])};
}

// Any width, alignment and place of the rotary channels: a warp a head, its channels in shared memory.
template <typename T> __global__ void __launch_bounds__(kThreads) hs_rotate_any_kernel(const __grid_constant__ RotateArgs g)
{
    extern __shared__ float2 turns[];
    const hs_rotate_t& a = g.a;
    const int heads = a.heads[0] + a.heads[1], pairs = a.rope / 2;
    const int chunks = (heads + g.heads_block - 1) / g.heads_block;  // blocks that share a token's heads
    const int64_t first = (int64_t)(blockIdx.x / chunks) * g.tokens_block;
    const int head0 = (int)(blockIdx.x % chunks) * g.heads_block;
    const int tokens = (int)min((int64_t)g.tokens_block, a.tokens - first), some = min(g.heads_block, heads - head0);
    for (int i = threadIdx.x; i < tokens * pairs; i += kThreads) {
        const int t = i / pairs;
        turns[i] = hs_rotation(a.positions[first + t], hs_turn(a.inv_freq[i - t * pairs]));
    }
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* y = reinterpret_cast<float*>(turns + g.tokens_block * pairs) + warp * a.dim;
    for (int i = warp; i < tokens * some; i += kThreads / 32) {
        const int t = i / some;
        const Head<T> h = head_of<T>(a, first + t, head0 + i - t * some);
        float sum = 0.f, f = 1.f;
        for (int c = lane; c < a.dim; c += 32) {
            const float v = HsType<T>::to_float(h.x[c]);
            sum += v * v;
            y[c] = v;
        }
        if (h.weight) {
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
            f = rsqrtf(sum / a.dim + a.eps);
        }
        __syncwarp();  // the head's channels have been read: outputs may overwrite them
        auto normed = [&](int c) { return h.weight ? y[c] * f * HsType<T>::to_float(h.weight[c]) : y[c]; };
        for (int c = lane; c < a.dim; c += 32) {
            float v = normed(c);
            const int n = c - a.rope_at;
            if (n >= 0 && n < a.rope) {
                const bool paired = a.rotation == HS_ROTATE_PAIRS;
                const bool low = paired ? (n & 1) == 0 : n < pairs;
                const float2 r = turns[t * pairs + (paired ? n >> 1 : low ? n : n - pairs)];
                const int step = paired ? 1 : pairs;
                const float z = normed(low ? c + step : c - step);
                v = low ? v * r.x - z * r.y : z * r.y + v * r.x;
            }
            h.out[c] = HsType<T>::from_float(v);
        }
        __syncwarp();  // before the next head takes the buffer
    }
}

template <typename T> cudaError_t launch_any(RotateArgs& g, cudaStream_t s)
{
    const hs_rotate_t& a = g.a;
    const int heads = a.heads[0] + a.heads[1], items = 4 * kWarps;  // heads a block
    g.heads_block = heads < items ? heads : items;
    g.tokens_block = heads < items ? items / heads : 1;
    const int most = a.rope ? 2048 / a.rope : items;  // sines and cosines: at most 8 KB a block
    if (g.tokens_block > most) g.tokens_block = most;
    if (g.tokens_block > a.tokens) g.tokens_block = (int)a.tokens;
    const int64_t grid = (a.tokens + g.tokens_block - 1) / g.tokens_block * ((heads + g.heads_block - 1) / g.heads_block);
    const size_t smem = sizeof(float2) * g.tokens_block * (a.rope / 2) + sizeof(float) * a.dim * kWarps;
    hs_rotate_any_kernel<T><<<(unsigned)grid, kThreads, smem, s>>>(g);
    return cudaGetLastError();
}

template <typename T> cudaError_t launch(const hs_rotate_t& a, cudaStream_t s)
{
    constexpr int H = Half<T>::n;
    auto fits = [&](const void* p, const int64_t* stride, int heads) {
        return ((uintptr_t)p & 7) == 0 && (!stride || ((a.tokens <= 1 || stride[0] % H == 0) && (heads <= 1 || stride[1] % H == 0)));
    };
    bool whole = a.dim % (2 * H) == 0;
    for (int k = 0; k < 2; ++k)
        if (a.heads[k])
            whole = whole && fits(a.x[k], a.x_stride[k], a.heads[k]) && fits(a.out[k], a.out_stride[k], a.heads[k]) && fits(a.weight[k], nullptr, 0);
    RotateArgs g;
    g.a = a;
    if (a.rotation == HS_ROTATE_NONE) g.a.rope = 0;
    whole = whole && a.rope_at % (2 * H) == 0 && g.a.rope % (2 * H) == 0;
    if (!whole) return launch_any<T>(g, s);
    // the team and units a lane that leave the fewest lanes without a unit
    const int units = a.dim / (2 * H);
    int nv = 1, best = 1 << 30;
    for (int n : {1, 2, 3, 4, 8})
        for (int team = 8; team <= 32; team *= 2)
            if (n * team >= units && n * team < best) best = n * team, nv = n, g.team = team;
    const int ahead = nv == 1 ? 4 : nv <= 3 ? 2 : 1, once = ahead * (32 / g.team);  // heads of a warp at once
    // all heads of a token to a warp, whose sines and weights serve them all, but where that leaves SMs without work
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int most = a.heads[0] > a.heads[1] ? a.heads[0] : a.heads[1];
    g.heads_warp = (most + once - 1) / once * once;
    while (g.heads_warp > once && a.tokens * ((a.heads[0] + g.heads_warp - 1) / g.heads_warp) < (int64_t)sms * kWarpsEnough)
        g.heads_warp = (g.heads_warp / 2 + once - 1) / once * once;
    for (int k = 0; k < 2; ++k) g.chunks[k] = (a.heads[k] + g.heads_warp - 1) / g.heads_warp;
    const int64_t grid = (a.tokens * (g.chunks[0] + g.chunks[1]) + kWarps - 1) / kWarps;
    const size_t smem = sizeof(float2) * kWarps * (g.a.rope / 2);
    if (nv == 1)
        hs_rotate_kernel<T, 1, 4><<<(unsigned)grid, kThreads, smem, s>>>(g);
    else if (nv == 2)
        hs_rotate_kernel<T, 2, 2><<<(unsigned)grid, kThreads, smem, s>>>(g);
    else if (nv == 3)
        hs_rotate_kernel<T, 3, 2><<<(unsigned)grid, kThreads, smem, s>>>(g);
    else if (nv == 4)
        hs_rotate_kernel<T, 4, 1><<<(unsigned)grid, kThreads, smem, s>>>(g);
    else
        hs_rotate_kernel<T, 8, 1><<<(unsigned)grid, kThreads, smem, s>>>(g);
    return cudaGetLastError();
}

}  // namespace

cudaError_t hs_launch_rotate(const hs_rotate_t& a, cudaStream_t s)
{
    if (a.dtype == HS_TYPE_BF16) return launch<__nv_bfloat16>(a, s);
    if (a.dtype == HS_TYPE_FP16) return launch<__half>(a, s);
    return launch<float>(a, s);
}
