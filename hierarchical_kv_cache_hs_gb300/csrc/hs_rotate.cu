// hs_norm_rotate: the norm of each head's channels and their rotation, in one pass over
// the queries and keys of a token.
//
// Bound by memory: each element is read once and written once.  A block takes some
// tokens and some of their heads; it computes those tokens' sines and cosines once, in
// shared memory, and a team of lanes takes a head's channels in 16-byte pieces.
// Rows that are not in such pieces go element by element through shared memory.
#include "hs_pieces.h"
#include "hs_rotation.h"

namespace {

constexpr int kThreads = 256;

struct RotateArgs {
    hs_rotate_t a;
    int tokens_block, heads_block;  // of a block
    int chunks;                     // blocks that share a token's heads
    int team;                       // lanes of a head
};

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

// The tokens' sines and cosines: [token of the block][pair].
__device__ __forceinline__ void fill_turns(const RotateArgs& g, int64_t first, int tokens, float2* turns)
{
    const hs_rotate_t& a = g.a;
    const int pairs = a.rope / 2;
    if (a.rotation == HS_ROTATE_NONE) return;
    for (int i = threadIdx.x; i < tokens * pairs; i += kThreads) {
        const int t = i / pairs;
        turns[i] = hs_rotation(a.positions[first + t], a.inv_freq[i - t * pairs]);
    }
}

// NV: 16-byte pieces a lane.
template <typename T, int NV> __global__ void __launch_bounds__(kThreads) hs_rotate_kernel(const __grid_constant__ RotateArgs g)
{
    constexpr int P = Piece<T>::n;
    extern __shared__ float2 turns[];
    const hs_rotate_t& a = g.a;
    const int heads = a.heads[0] + a.heads[1];
    const int64_t first = (int64_t)(blockIdx.x / g.chunks) * g.tokens_block;
    const int head0 = (int)(blockIdx.x % g.chunks) * g.heads_block;
    const int tokens = (int)min((int64_t)g.tokens_block, a.tokens - first), some = min(g.heads_block, heads - head0);
    fill_turns(g, first, tokens, turns);
    __syncthreads();
    const int team = threadIdx.x / g.team, at = threadIdx.x - team * g.team, teams = kThreads / g.team;
    const int pieces = a.dim / P, pairs = a.rope / 2;
    const unsigned lanes = g.team == 32 ? ~0u : ((1u << g.team) - 1) << ((threadIdx.x & 31) / g.team * g.team);
    for (int i = team; i < tokens * some; i += teams) {
        const int t = i / some;
        const Head<T> h = head_of<T>(a, first + t, head0 + i - t * some);
        const float2* turn = turns + t * pairs;
        uint4 xv[NV], other[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int p = v * g.team + at;
            if (p < pieces) xv[v] = reinterpret_cast<const uint4*>(h.x)[p];
        }
        if (a.rotation == HS_ROTATE_HALVES)
#pragma unroll
            for (int v = 0; v < NV; ++v) {  // the other halves of its pairs
                const int c = (v * g.team + at) * P - a.rope_at;
                if (c >= 0 && c < a.rope) other[v] = *reinterpret_cast<const uint4*>(h.x + a.rope_at + (c < pairs ? c + pairs : c - pairs));
            }
        float y[NV][P], f = 1.f;
        float sum = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (v * g.team + at < pieces) {
                Piece<T>::unpack(xv[v], y[v]);
#pragma unroll
                for (int k = 0; k < P; ++k) sum += y[v][k] * y[v][k];
            }
        if (h.weight) {
            for (int o = g.team >> 1; o; o >>= 1) sum += __shfl_xor_sync(lanes, sum, o);
            f = rsqrtf(sum / a.dim + a.eps);
        }
        __syncwarp(lanes);  // the head's channels have been read: outputs may overwrite them
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int p = v * g.team + at, c = p * P - a.rope_at;
            if (p >= pieces) continue;
            float w[P];
            if (h.weight) {
                Piece<T>::unpack(reinterpret_cast<const uint4*>(h.weight)[p], w);
#pragma unroll
                for (int k = 0; k < P; ++k) y[v][k] = y[v][k] * f * w[k];
            }
            if (c >= 0 && c < a.rope) {
                if (a.rotation == HS_ROTATE_PAIRS) {
#pragma unroll
                    for (int k = 0; k < P; k += 2) {
                        const float2 r = turn[(c + k) / 2];
                        const float y0 = y[v][k], y1 = y[v][k + 1];
                        y[v][k] = y0 * r.x - y1 * r.y, y[v][k + 1] = y0 * r.y + y1 * r.x;
                    }
                } else {
                    const bool low = c < pairs;
                    const int pair = low ? c : c - pairs, oc = a.rope_at + (low ? c + pairs : c - pairs);
                    float z[P];
                    Piece<T>::unpack(other[v], z);
                    if (h.weight) {
                        Piece<T>::unpack(*reinterpret_cast<const uint4*>(h.weight + oc), w);
#pragma unroll
                        for (int k = 0; k < P; ++k) z[k] = z[k] * f * w[k];
                    }
#pragma unroll
                    for (int k = 0; k < P; ++k) {
                        const float2 r = turn[pair + k];
                        y[v][k] = low ? y[v][k] * r.x - z[k] * r.y : z[k] * r.y + y[v][k] * r.x;
                    }
                }
            }
            reinterpret_cast<uint4*>(h.out)[p] = Piece<T>::pack(y[v]);
        }
    }
}

// Any width, alignment and place of the rotary channels: a warp a head, its channels in shared memory.
template <typename T> __global__ void __launch_bounds__(kThreads) hs_rotate_any_kernel(const __grid_constant__ RotateArgs g)
{
    extern __shared__ float2 turns[];
    const hs_rotate_t& a = g.a;
    const int heads = a.heads[0] + a.heads[1], pairs = a.rope / 2;
    const int64_t first = (int64_t)(blockIdx.x / g.chunks) * g.tokens_block;
    const int head0 = (int)(blockIdx.x % g.chunks) * g.heads_block;
    const int tokens = (int)min((int64_t)g.tokens_block, a.tokens - first), some = min(g.heads_block, heads - head0);
    fill_turns(g, first, tokens, turns);
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

template <typename T> cudaError_t launch(const hs_rotate_t& a, cudaStream_t s)
{
    constexpr int P = Piece<T>::n;
    auto fits = [&](const void* p, const int64_t* stride, int heads) {
        return ((uintptr_t)p & 15) == 0 && (!stride || ((a.tokens <= 1 || stride[0] % P == 0) && (heads <= 1 || stride[1] % P == 0)));
    };
    bool pieces16 = a.dim % P == 0;
    for (int k = 0; k < 2; ++k)
        if (a.heads[k])
            pieces16 = pieces16 && fits(a.x[k], a.x_stride[k], a.heads[k]) && fits(a.out[k], a.out_stride[k], a.heads[k]) &&
                       fits(a.weight[k], nullptr, 0);
    if (a.rotation != HS_ROTATE_NONE)
        pieces16 = pieces16 && a.rope_at % P == 0 && (a.rotation == HS_ROTATE_PAIRS ? a.rope : a.rope / 2) % P == 0;
    RotateArgs g;
    g.a = a;
    if (a.rotation == HS_ROTATE_NONE) g.a.rope = 0;
    const int pieces = a.dim / P, heads = a.heads[0] + a.heads[1];
    int nv = 1;
    g.team = 32;
    if (pieces16) {  // the team and pieces a lane that leave the fewest lanes without a piece
        int best = 1 << 30;
        for (int n : {1, 2, 3, 4, 8})
            for (int team = 8; team <= 32; team *= 2)
                if (n * team >= pieces && n * team < best) best = n * team, nv = n, g.team = team;
    }
    const int items = 4 * kThreads / g.team;  // heads a block
    g.heads_block = heads < items ? heads : items;
    g.chunks = (heads + g.heads_block - 1) / g.heads_block;
    g.tokens_block = heads < items ? items / heads : 1;
    // sines and cosines: at most 8 KB a block
    const int most = g.a.rope ? 2048 / g.a.rope : items;
    if (g.tokens_block > most) g.tokens_block = most < 1 ? 1 : most;
    if (g.tokens_block > a.tokens) g.tokens_block = (int)a.tokens;
    const int64_t grid = (a.tokens + g.tokens_block - 1) / g.tokens_block * g.chunks;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    size_t smem = sizeof(float2) * g.tokens_block * (g.a.rope / 2);
    if (!pieces16) {
        smem += sizeof(float) * a.dim * (kThreads / 32);
        hs_rotate_any_kernel<T><<<(unsigned)grid, kThreads, smem, s>>>(g);
    } else if (nv == 1)
        hs_rotate_kernel<T, 1><<<(unsigned)grid, kThreads, smem, s>>>(g);
    else if (nv == 2)
        hs_rotate_kernel<T, 2><<<(unsigned)grid, kThreads, smem, s>>>(g);
    else if (nv == 3)
        hs_rotate_kernel<T, 3><<<(unsigned)grid, kThreads, smem, s>>>(g);
    else if (nv == 4)
        hs_rotate_kernel<T, 4><<<(unsigned)grid, kThreads, smem, s>>>(g);
    else
        hs_rotate_kernel<T, 8><<<(unsigned)grid, kThreads, smem, s>>>(g);
    return cudaGetLastError();
}

}  // namespace

cudaError_t hs_launch_rotate(const hs_rotate_t& a, cudaStream_t s)
{
    if (a.dtype == HS_TYPE_BF16) return launch<__nv_bfloat16>(a, s);
    if (a.dtype == HS_TYPE_FP16) return launch<__half>(a, s);
    return launch<float>(a, s);
}
