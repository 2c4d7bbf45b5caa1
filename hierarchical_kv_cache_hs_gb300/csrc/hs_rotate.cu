// hs_norm_rotate: the norm of each head's channels and their rotation, in one pass over
// the queries and keys of a token.
//
//   y = x w / sqrt(mean x^2 + eps);  a pair (a, b) of y becomes (a cos - b sin, a sin + b cos)
//
// Each element is read once and written once, so the floor is memory's: 8192 tokens x (32 + 8) heads of 128 bf16
// channels take 35.3 us, 4.8 TB/s, 0.70 of a copy's rate; the issue slots are 64 % taken (80 registers, 24 warps an SM),
// and what a warp does between its loads is not hidden whole.  The last 64 channels of 8192 x 32 queries of 192, in
// place: 16.6 us, 0.60.  64 x 128 heads: 3.3 us; one token: 3.2, a launch.  (Replayed from a graph, inputs larger than
// L2.  Times at choices further on are of the step that took them.)
// A ring of bulk copies through shared memory instead of loads to registers took 49 us for the 36, and values kept
// unpacked between the norm and the rotation 39 to 43: registers.
//
// A warp takes some heads of one token.  Its lanes form teams of 4 to 32, a head each, and a lane has the
// same channels of every head that its team passes over: its weights, sines and cosines
// stay in registers.  A lane's channels come in units of 16 bytes, as two halves of 8
// that lie side by side or, for pairs whose channels are half of the rotary ones apart,
// that far apart: so a pair is always within a lane.
// Heads that are not in such units go element by element through shared memory.
#include "hs_pieces.h"
#include "hs_rotation.h"
#include "hs_tc.h"

namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;  // 256 threads: 38.5 us for 36.8 (8192 tokens, 32 + 8 heads)
constexpr int kWarpsEnough = 64;  // an SM: with fewer warps in all, a token's heads are shared by several
// Up to this many heads a token go by teams of their own: 65,536 tokens x 1 head of 128 18 us against 47, x 2 heads 33
// against 81.  With more a token's warp is better filled, and its sines serve them all: 32,768 x 4 heads 30 us against
// 33, 16,384 x 8 heads 19 against 33.
constexpr int kFew = 3;

struct RotateArgs {
    hs_rotate_t a;
    float inv_dim;
    int heads_warp;      // of a warp
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

__device__ __forceinline__ float2 mul2(const float2& a, const float2& b)  // two operations in one instruction
{
    float2 d;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
// A lane's channels of a head: NV units, where their first halves lie and how far behind it the second ones, and its
// factors, weights times sines and cosines: for a rotary unit of two halves p and q (or of pairs p, q) c[0] p - c[1] q
// and c[2] p + c[3] q; else c[0] and c[1] are weights.
template <typename T, int NV> struct Lane {
    static constexpr int H = Half<T>::n, U = 2 * H;  // channels of half a unit, of a unit
    int low[NV], apart[NV], pair[NV];                // pair: the first, -1: not rotary
    bool there[NV], paired, normed;
    float c[NV][4][H];

    __device__ Lane(const hs_rotate_t& a, int team, int at) : paired(a.rotation == HS_ROTATE_PAIRS), normed(false)
    {
        const int pairs = a.rope / 2, units = a.dim / U;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int u = v * team + at, n = u * U - a.rope_at;
            there[v] = u < units;
            pair[v] = there[v] && n >= 0 && n < a.rope ? n / 2 : -1;
            const bool halves = pair[v] >= 0 && !paired;  // unit i of the rotary channels: H from either half of them
            low[v] = halves ? a.rope_at + n / 2 : u * U;
            apart[v] = halves ? pairs : H;
        }
    }
    template <typename Turn> __device__ void load_factors(const T* weight, Turn turn)  // turn(v, i): cos and sin of a pair
    {
        normed = weight != nullptr;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float w[U];
#pragma unroll
            for (int i = 0; i < U; ++i) w[i] = 1.f;
            if (weight && there[v]) {
                Half<T>::unpack(*reinterpret_cast<const uint2*>(weight + low[v]), w);
                Half<T>::unpack(*reinterpret_cast<const uint2*>(weight + low[v] + apart[v]), w + H);
            }
#pragma unroll
            for (int i = 0; i < H; ++i) {
                c[v][0][i] = w[i], c[v][1][i] = w[H + i], c[v][2][i] = c[v][3][i] = 0.f;
                if (pair[v] >= 0) {
                    const float2 r = turn(v, i);
                    const float wp = paired ? w[2 * i] : w[i], wq = paired ? w[2 * i + 1] : w[H + i];
                    c[v][0][i] = wp * r.x, c[v][1][i] = wq * r.y, c[v][2][i] = wp * r.y, c[v][3][i] = wq * r.x;
                }
            }
        }
    }
    __device__ float squares(const uint2 (&xp)[NV], const uint2 (&xq)[NV]) const
    {
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float y[U];
            Half<T>::unpack(xp[v], y), Half<T>::unpack(xq[v], y + H);
#pragma unroll
            for (int i = 0; i < U; i += 2) sum = fma2(make_float2(y[i], y[i + 1]), make_float2(y[i], y[i + 1]), sum);
        }
        return sum.x + sum.y;
    }
    __device__ void turn(int v, uint2& xp, uint2& xq, float f) const  // f: 1 / sqrt of the head's mean square
    {
        float y[U];
        Half<T>::unpack(xp, y), Half<T>::unpack(xq, y + H);
        auto two = [&](int i) { return make_float2(y[i], y[i + 1]); };
        auto put = [&](int i, const float2& d) { y[i] = d.x, y[i + 1] = d.y; };
        auto factor = [&](int n, int i) { return make_float2(c[v][n][i], c[v][n][i + 1]); };
        if (normed)
#pragma unroll
            for (int i = 0; i < U; i += 2) put(i, mul2(two(i), make_float2(f, f)));
        if (pair[v] >= 0 && paired) {
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const float p = y[2 * i], q = y[2 * i + 1];
                put(2 * i, fma2(make_float2(q, q), make_float2(-c[v][1][i], c[v][3][i]),
                                mul2(make_float2(p, p), make_float2(c[v][0][i], c[v][2][i]))));
            }
        } else if (pair[v] >= 0) {
#pragma unroll
            for (int i = 0; i < H; i += 2) {
                const float2 p = two(i), q = two(H + i), s = factor(1, i);
                put(i, fma2(make_float2(-s.x, -s.y), q, mul2(p, factor(0, i))));
                put(H + i, fma2(q, factor(3, i), mul2(p, factor(2, i))));
            }
        } else if (normed) {
#pragma unroll
            for (int i = 0; i < H; i += 2) put(i, mul2(two(i), factor(0, i))), put(H + i, mul2(two(H + i), factor(1, i)));
        }
        xp = Half<T>::pack(y), xq = Half<T>::pack(y + H);
    }
};

// NV: units a lane, AHEAD: heads of a team on their way together; of three units one, which leaves registers for a third
// more warps (8192 tokens x 32 heads of 192 37.5 us against 38.6, 4096 x 16 of 576 35.0 against 37.1).  Inputs are read past
// the caches (__ldcs: 36.8 us against 38.2).
template <typename T, int NV, int AHEAD> __global__ void __launch_bounds__(kThreads, NV == 1 ? 6 : NV == 3 ? 4 : 1) hs_rotate_kernel(const __grid_constant__ RotateArgs g)
{
    extern __shared__ float2 sines[];  // [warp][pair]
    const hs_rotate_t& a = g.a;
    const int lane = threadIdx.x & 31;
    const int64_t token = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (token >= a.tokens) return;
    const int head_first = blockIdx.y * g.heads_warp, head_last = min(head_first + g.heads_warp, a.heads[0] + a.heads[1]);
    // Wide heads leave registers for few at a time, so the others are on their way to L2 meanwhile: 44.0 -> 38.6 us for
    // 8192 tokens x 32 heads of 192, 40.6 -> 37.1 for 4096 x 16 of 576.  (Narrow ones 35.2 -> 35.5.)
    if (NV > 1 && head_last - head_first > AHEAD * (32 / g.team)) {
        const int lines = (a.dim * (int)sizeof(T) + 127) / 128;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int before = k ? a.heads[0] : 0;
            const int first = max(head_first - before, 0), last = min(head_last - before, a.heads[k]);
            const T* x = static_cast<const T*>(a.x[k]) + token * a.x_stride[k][0];
            for (int i = lane; i < (last - first) * lines; i += 32) {
                const int h = i / lines;
                tc::prefetch_l2(x + (first + h) * a.x_stride[k][1] + (i - h * lines) * (128 / (int)sizeof(T)));
            }
        }
    }
    const int pairs = a.rope / 2;
    float2* turns = sines + (threadIdx.x >> 5) * pairs;
    if (pairs) {
        const int position = a.positions[token];
        for (int i = lane; i < pairs; i += 32) turns[i] = hs_rotation(position, hs_turn(a.inv_freq[i]));
        __syncwarp();
    }
    const int teams = 32 / g.team, mine = lane / g.team;
    Lane<T, NV> l(a, g.team, lane & (g.team - 1));
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {  // queries, keys
        const int before = k ? a.heads[0] : 0;
        const int first = max(head_first - before, 0), last = min(head_last - before, a.heads[k]);
        if (first >= last) continue;
        l.load_factors(static_cast<const T*>(a.weight[k]), [&](int v, int i) { return turns[l.pair[v] + i]; });
        const int64_t x_step = a.x_stride[k][1] * teams, out_step = a.out_stride[k][1] * teams;
        const T* x = static_cast<const T*>(a.x[k]) + token * a.x_stride[k][0] + (first + mine) * a.x_stride[k][1];
        T* out = static_cast<T*>(a.out[k]) + token * a.out_stride[k][0] + (first + mine) * a.out_stride[k][1];
        for (int head0 = first + mine; head0 - mine < last; head0 += AHEAD * teams) {  // the whole warp
            uint2 xp[AHEAD][NV], xq[AHEAD][NV];
#pragma unroll
            for (int m = 0; m < AHEAD; ++m, x += x_step)
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    xp[m][v] = xq[m][v] = make_uint2(0, 0);
                    if (l.there[v] && head0 + m * teams < last) {
                        xp[m][v] = __ldcs(reinterpret_cast<const uint2*>(x + l.low[v]));
                        xq[m][v] = __ldcs(reinterpret_cast<const uint2*>(x + l.low[v] + l.apart[v]));
                    }
                }
            float f[AHEAD];
            if (l.normed) {
#pragma unroll
                for (int m = 0; m < AHEAD; ++m) f[m] = l.squares(xp[m], xq[m]);
                for (int o = g.team >> 1; o; o >>= 1)
#pragma unroll
                    for (int m = 0; m < AHEAD; ++m) f[m] += __shfl_xor_sync(~0u, f[m], o);
#pragma unroll
                for (int m = 0; m < AHEAD; ++m) f[m] = rsqrtf(f[m] * g.inv_dim + a.eps);
            }
#pragma unroll
            for (int m = 0; m < AHEAD; ++m, out += out_step) {
                if (head0 + m * teams >= last) continue;
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    if (!l.there[v]) continue;
                    l.turn(v, xp[m][v], xq[m][v], f[m]);
                    *reinterpret_cast<uint2*>(out + l.low[v]) = xp[m][v];
                    *reinterpret_cast<uint2*>(out + l.low[v] + l.apart[v]) = xq[m][v];
                }
            }
        }
    }
}

// Few heads a token: a team takes heads of one token after another, each lane with the sines of its own pairs, and the
// next head's channels on their way.  Bound by instructions, the sines' most of all (65,536 heads of 128: 0.28 of a
// copy's rate; with the library's sine and cosine 19 us instead of 18).
template <typename T, int NV> __global__ void __launch_bounds__(kThreads, NV == 1 ? 6 : 1) hs_rotate_few_kernel(const __grid_constant__ RotateArgs g)
{
    constexpr int H = Half<T>::n;
    const hs_rotate_t& a = g.a;
    const int lane = threadIdx.x & 31, teams = 32 / g.team, heads = a.heads[0] + a.heads[1];
    const uint32_t rows = (uint32_t)(a.tokens * heads), step = gridDim.x * kWarps * teams;  // below 2^28
    const uint32_t first = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * teams, mine = lane / g.team;
    Lane<T, NV> l(a, g.team, lane & (g.team - 1));
    HsTurn freq[NV][H];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < H; ++i) freq[v][i] = l.pair[v] >= 0 ? hs_turn(a.inv_freq[l.pair[v] + i]) : HsTurn{0, true};
    uint2 xp[NV], xq[NV];
    int position = 0, k = 0;
    T* out = nullptr;
    auto bring = [&](uint32_t row) {
        if (row >= rows) return;
        const uint32_t token = row / heads;
        int head = (int)(row - token * heads);
        k = head >= a.heads[0];
        head -= k ? a.heads[0] : 0;
        const T* x = static_cast<const T*>(a.x[k]) + token * a.x_stride[k][0] + head * a.x_stride[k][1];
        out = static_cast<T*>(a.out[k]) + token * a.out_stride[k][0] + head * a.out_stride[k][1];
        if (a.rotation != HS_ROTATE_NONE) position = a.positions[token];
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (l.there[v]) {
                xp[v] = __ldcs(reinterpret_cast<const uint2*>(x + l.low[v]));
                xq[v] = __ldcs(reinterpret_cast<const uint2*>(x + l.low[v] + l.apart[v]));
            }
    };
#pragma unroll
    for (int v = 0; v < NV; ++v) xp[v] = xq[v] = make_uint2(0, 0);
    bring(first + mine);
    for (uint32_t row0 = first; row0 < rows; row0 += step) {  // the whole warp
        uint2 p[NV], q[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) p[v] = xp[v], q[v] = xq[v];
        const int at = position, array = k;
        T* to = out;
        bring(row0 + step + mine);
        l.load_factors(static_cast<const T*>(a.weight[array]), [&](int v, int i) { return hs_rotation(at, freq[v][i]); });
        float f = l.squares(p, q);
        for (int o = g.team >> 1; o; o >>= 1) f += __shfl_xor_sync(~0u, f, o);
        f = rsqrtf(f * g.inv_dim + a.eps);
        if (row0 + mine < rows)
#pragma unroll
            for (int v = 0; v < NV; ++v)
                if (l.there[v]) {
                    l.turn(v, p[v], q[v], f);
                    *reinterpret_cast<uint2*>(to + l.low[v]) = p[v];
                    *reinterpret_cast<uint2*>(to + l.low[v] + l.apart[v]) = q[v];
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
    const int64_t first = (int64_t)blockIdx.x * g.tokens_block;
    const int head0 = blockIdx.y * g.heads_block;
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
    const dim3 grid((unsigned)((a.tokens + g.tokens_block - 1) / g.tokens_block), (heads + g.heads_block - 1) / g.heads_block);
    const size_t smem = sizeof(float2) * g.tokens_block * (a.rope / 2) + sizeof(float) * a.dim * kWarps;
    hs_rotate_any_kernel<T><<<grid, kThreads, smem, s>>>(g);
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
    // The team and units a lane that leave the fewest lanes without a unit; teams of 4 for heads of up to 4 units (8192
    // tokens x 68 heads of 32: 21.1 us against 29.4 with 8) and for few heads (32,768 x 2 of 96: 13.6 against 17.4), but
    // not with several units a lane for many (8192 x 36 of 96: 40.0 against 34.1; of 80 40.0 against 33.1).
    const int units = a.dim / (2 * H);
    int nv = 1, best = 1 << 30;
    for (int n : {1, 2, 3, 4, 8})  // 8 of 32-bit types: 1024 channels of 16 bits are 128 units, 4 a lane
        for (int team = 4; team <= 32; team *= 2)
            if (n * team >= units && n * team < best && (team > 4 || n == 1 || a.heads[0] + a.heads[1] <= kFew)) best = n * team, nv = n, g.team = team;
    const int ahead = nv == 1 ? 4 : nv == 2 ? 2 : 1, once = ahead * (32 / g.team);  // heads of a warp at once
    // all heads of a token to a warp, whose sines and weights serve them all, but where that leaves SMs without work
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int heads = a.heads[0] + a.heads[1];
    g.inv_dim = 1.f / a.dim;
    if (heads <= kFew && nv <= 3) {
        const int64_t teams = (a.tokens * heads + 32 / g.team - 1) / (32 / g.team), most = (int64_t)sms * (nv == 1 ? 6 : 3);
        const unsigned blocks = (unsigned)((teams + kWarps - 1) / kWarps < most ? (teams + kWarps - 1) / kWarps : most);
        if (nv == 1)
            hs_rotate_few_kernel<T, 1><<<blocks, kThreads, 0, s>>>(g);
        else if (nv == 2)
            hs_rotate_few_kernel<T, 2><<<blocks, kThreads, 0, s>>>(g);
        else
            hs_rotate_few_kernel<T, 3><<<blocks, kThreads, 0, s>>>(g);
        return cudaGetLastError();
    }
    g.heads_warp = (heads + once - 1) / once * once;
    while (g.heads_warp > once && a.tokens * ((heads + g.heads_warp - 1) / g.heads_warp) < (int64_t)sms * kWarpsEnough)
        g.heads_warp = (g.heads_warp / 2 + once - 1) / once * once;
    // a block takes the same heads of several tokens
    const dim3 grid((unsigned)((a.tokens + kWarps - 1) / kWarps), (heads + g.heads_warp - 1) / g.heads_warp);
    const size_t smem = sizeof(float2) * kWarps * (g.a.rope / 2);
    if (nv == 1)
        hs_rotate_kernel<T, 1, 4><<<grid, kThreads, smem, s>>>(g);
    else if (nv == 2)
        hs_rotate_kernel<T, 2, 2><<<grid, kThreads, smem, s>>>(g);
    else if (nv == 3)
        hs_rotate_kernel<T, 3, 1><<<grid, kThreads, smem, s>>>(g);
    else if (nv == 4)
        hs_rotate_kernel<T, 4, 1><<<grid, kThreads, smem, s>>>(g);
    else if constexpr (sizeof(T) == 4)
        hs_rotate_kernel<T, 8, 1><<<grid, kThreads, smem, s>>>(g);
    return cudaGetLastError();
}

}  // namespace

cudaError_t hs_launch_rotate(const hs_rotate_t& a, cudaStream_t s)
{
    if (a.dtype == HS_TYPE_BF16) return launch<__nv_bfloat16>(a, s);
    if (a.dtype == HS_TYPE_FP16) return launch<__half>(a, s);
    return launch<float>(a, s);
}
