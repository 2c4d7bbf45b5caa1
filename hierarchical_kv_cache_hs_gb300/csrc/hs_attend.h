// What the two kernels of hs_latent_attend share: how the work is cut, which rows a
// tile holds, and how 8-bit rows become operands.
#pragma once

#include <type_traits>

#include "hs_ops.h"
#include "hs_tc.h"

namespace hs_attn {

using tc::wait;

constexpr int kTile = 64;  // rows a tile

// A unit is a request, a position and a block of heads; its rows come in tiles, one at
// least.  The tiles of all units form one line, which the workers (an SM, or a pair of
// SMs) cut into equal pieces (flat), or whole units go to each.  A unit's own time (its
// queries, its sums' way out) counts as `cost` tiles before its first one, but for the
// line's first unit: every piece has that once.  A cut inside it is a cut at the unit's
// start, so a worker may get no piece; the one before a piece that starts inside a unit
// always has one.
struct Args {
    hs_attend_t a;
    int head_blocks;
    int flat;
    int units;         // at most HS_MAX_BATCH x HS_MAX_POSITIONS x HS_MAX_HEADS / 128, below 2^31
    int unit_tiles;    // tiles of a unit; with lengths, the most that one has
    int workers;
    int cost;
    int64_t share;     // slots: tiles (and cost) a worker, and how many workers have one more
    int extra;
    int unit_share, unit_extra;  // units a worker, likewise

    // Fill in the cut: whole units, or pieces where those are `join` tiles' time shorter.
    void cut(int most, int64_t rows, int join, int unit_cost)
    {
        cost = unit_cost;
        unit_tiles = rows <= kTile ? 1 : (int)((rows + kTile - 1) / kTile);
        const int64_t total = (int64_t)units * unit_tiles;
        workers = (int)(total < most ? total : most);
        flat = (int64_t)((units + workers - 1) / workers) * unit_tiles > (total + workers - 1) / workers + join;
        if (!flat && workers > units) workers = units;
        const int64_t line = (int64_t)units * (unit_tiles + cost) - cost;
        share = line / workers;
        extra = (int)(line % workers);
        unit_share = units / workers;
        unit_extra = units % workers;
    }
};

struct Start {  // where a worker's piece of the line begins (unit -1: it has none)
    int unit, tile;
};
struct Piece {
    long long count;  // its tiles
    int unit, tile;
};

__device__ __forceinline__ int request_tiles(const hs_attend_t& a, long long b)
{
    long long n = a.entries;
    if (!a.slots) {
        n = a.lengths[b];
        n = n < 0 ? 0 : n > a.n_rows ? a.n_rows : n;
    }
    return n <= kTile ? 1 : (int)((n + kTile - 1) / kTile);
}

// Worker i's piece (one warp; every lane gets it).
__device__ __forceinline__ Piece find_piece(const Args& g, int i)
{
    const hs_attend_t& a = g.a;
    const int lane = threadIdx.x & 31;
    const int upr = a.positions * g.head_blocks;  // units a request
    Piece p;
    if (!g.flat) {
        p.unit = g.unit_share * i + min(i, g.unit_extra);
        p.tile = 0;
        const int n = g.unit_share + (i < g.unit_extra);
        p.count = (long long)n * g.unit_tiles;
        if (!a.slots) {
            const int end = p.unit + n;
            p.count = 0;
            for (int b = p.unit / upr + lane; b < a.batch && b * upr < end; b += 32)
                p.count += (long long)(min(b * upr + upr, end) - max(b * upr, p.unit)) * request_tiles(a, b);
            for (int o = 16; o; o >>= 1) p.count += __shfl_xor_sync(~0u, p.count, o);
        }
        return p;
    }
    if (a.slots) {
        const int per = g.unit_tiles + g.cost;
        auto place = [&](int x, int& unit, int& tile) {
            const long long at = g.cost + g.share * x + min(x, g.extra);
            unit = at < 0x7fffffff ? (int)((unsigned)at / (unsigned)per) : (int)(at / per);
            tile = max(0, (int)(at - (long long)unit * per) - g.cost);
        };
        int unit, tile;
        place(i, p.unit, p.tile);
        place(i + 1, unit, tile);
        p.count = (long long)(unit - p.unit) * g.unit_tiles + tile - p.tile;
        return p;
    }
    long long total = 0;
    for (int b = lane; b < a.batch; b += 32) total += (long long)request_tiles(a, b) * upr;
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(~0u, total, o);
    const long long n = total < g.workers ? total : g.workers;
    p.unit = p.tile = 0;
    p.count = 0;
    if (i >= n) return p;
    const long long line = total + (long long)g.cost * (g.units - 1);
    const long long lo = g.cost + line * i / n, hi = g.cost + line * (i + 1) / n;
    long long before = 0, from = 0, to = total;  // tiles before lo, before hi
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
        const int b = b0 + lane;
        const long long tiles = b < a.batch ? request_tiles(a, b) : 0, per = tiles + g.cost;
        const long long own = b < a.batch ? per * upr : 0;
        long long incl = own;
        for (int o = 1; o < 32; o <<= 1) {
            const long long up = __shfl_up_sync(~0u, incl, o);
            if (lane >= o) incl += up;
        }
        const long long at = before + incl - own;  // where request b begins
        const unsigned at_lo = __ballot_sync(~0u, lo >= at && lo < at + own);
        const unsigned at_hi = __ballot_sync(~0u, hi >= at && hi < at + own);
        if (at_lo | at_hi) {
            auto place = [&](long long x, int& unit, int& tile) {  // and the tiles before it
                const int u = (int)((x - at) / per);
                unit = b * upr + u;
                tile = max(0, (int)(x - at - u * per) - g.cost);
                return at - (long long)g.cost * upr * b + u * tiles + tile;
            };
            int unit = 0, tile = 0;
            long long tiles_before = 0;
            if (at_lo) {
                const int src = __ffs(at_lo) - 1;
                if (lane == src) tiles_before = place(lo, unit, tile);
                p.unit = __shfl_sync(~0u, unit, src);
                p.tile = __shfl_sync(~0u, tile, src);
                from = __shfl_sync(~0u, tiles_before, src);
            }
            if (at_hi) {
                const int src = __ffs(at_hi) - 1;
                if (lane == src) tiles_before = place(hi, unit, tile);
                to = __shfl_sync(~0u, tiles_before, src);
                break;
            }
        }
        before += __shfl_sync(~0u, incl, 31);
    }
    p.count = to - from;
    return p;
}

// The units, or parts of units, of a piece, in order.
struct Walk {
    const Args& g;
    long long left;
    int unit, tile;
    // the current one: tiles [t0, t1) of `tiles`
    long long b;
    int p, hb, t0, t1, tiles;
    long long rows;  // entries, or allowed rows

    __device__ Walk(const Args& args, const Piece& x) : g(args), left(x.count), unit(x.unit), tile(x.tile) {}

    __device__ bool next()
    {
        if (left <= 0) return false;
        const hs_attend_t& a = g.a;
        const int pos = unit / g.head_blocks, request = pos / a.positions;
        b = request;
        p = pos - request * a.positions;
        hb = unit - pos * g.head_blocks;
        tiles = request_tiles(a, b);
        rows = a.entries;
        if (!a.slots) {
            rows = a.lengths[b];
            rows = rows > a.n_rows ? a.n_rows : rows;
            rows = rows - a.positions + 1 + p;
            rows = rows < 0 ? 0 : rows;
        }
        t0 = tile;
        t1 = (long long)(tiles - t0) <= left ? tiles : t0 + (int)left;
        left -= t1 - t0;
        ++unit;
        tile = 0;
        return true;
    }
};

// The row at a place of a tile: entry i of the list, or the i-th row.
struct Lookup {
    const hs_attend_t& a;
    const int32_t* slots;
    long long n;
    __device__ Lookup(const hs_attend_t& args, const Walk& w)
        : a(args), slots(args.slots ? args.slots + w.b * args.slots_stride[0] + w.p * args.slots_stride[1] : nullptr), n(w.rows)
    {
    }
    // The list's entry, unchecked: looked at an iteration later, so that no warp waits for it here.
    __device__ int raw(int tile, int at) const
    {
        const long long i = (long long)tile * kTile + at;
        return i >= n ? -1 : slots ? slots[i] : (int)i;
    }
    __device__ int row(int raw) const { return raw >= 0 && raw < a.n_rows ? raw : -1; }  // or -1
};

// Lines of 16 8-bit rows (row of lane l < 16: at) to L2, eight lanes a row.  (A bulk
// prefetch a row took about 2,000 clocks a tile to issue.)
__device__ __forceinline__ void prefetch_rows(const uint8_t* rows, int64_t row_stride, int at)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int n = 0; n < 16; n += 4) {
        const int r = __shfl_sync(~0u, at, n + (lane >> 3));
        if (r < 0) continue;
        const uint8_t* row = rows + r * row_stride;
        const int c = (lane & 7) * 128;
        if (c < HS_ROW8_BYTES) tc::prefetch_l2(row + c);
        if ((lane & 7) == 0) tc::prefetch_l2(row + HS_ROW8_BYTES - 1);
    }
}

// Four e4m3 values as two pairs of fp16, which holds each of them (and NaN).
__device__ __forceinline__ void widen(uint32_t v, uint32_t& lo, uint32_t& hi)
{
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(v));
}
// 16 e4m3 values as two 16-byte pieces of fp16 at dst + c0 and dst + c1.
__device__ __forceinline__ void store_wide(const uint4& v, uint32_t dst, int c0, int c1)
{
    uint32_t e[8];
    widen(v.x, e[0], e[1]);
    widen(v.y, e[2], e[3]);
    widen(v.z, e[4], e[5]);
    widen(v.w, e[6], e[7]);
    tc::st_shared16(dst + c0, e[0], e[1], e[2], e[3]);
    tc::st_shared16(dst + c1, e[4], e[5], e[6], e[7]);
}

// With 8-bit rows the products are in fp16; a bf16 query is scaled by a power of two that
// takes its largest magnitude `top` to [2^13, 2^14), so that what is 2^-28 of it or more
// stays exact.  The power, at most 126 (a top below 2^-113 then stays lower, and every bf16
// from 2^-133 up exact); infinities stay as they are.
__device__ __forceinline__ int power_up(float top)
{
    const int ex = (int)(__float_as_uint(top) >> 23);
    return ex == 255 ? 0 : min(140 - ex, 126);
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
__device__ __forceinline__ float largest_bf16(const uint4& v)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[k] << 16)), fabsf(__uint_as_float(w[k] & 0xffff0000u))));
    return top;
}
__device__ __forceinline__ uint4 bf16_to_half(const uint4& v, float f)
{
    auto two = [&](uint32_t w) { return pack2<__half>(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xffff0000u) * f); };
    return make_uint4(two(v.x), two(v.y), two(v.z), two(v.w));
}

// A row of 8 bits moves the running reference by its score and the log2 of its scale, so that
// weights times scales stay in fp16's range.  Scales below 2^-100, 0 among them, count as that:
// beside rows that score far below, such a row's weight then stays at 2^108 or less.
constexpr float kLeastLogScale = -100.f;

// The x-th unit that several workers worked on, found at the first start of a piece inside
// it: workers first..last have its pieces (false: there is no such unit).  The whole block
// calls it, at least 256 threads for up to 256 workers.
__device__ __forceinline__ bool find_cut(const Start* start, int workers, int x, int& unit, int& first, int& last)
{
    __shared__ int counts[8], at, cut_unit;
    const int t = threadIdx.x;
    if (t == 0) at = 0;
    int mine = -1;
    bool inside = false, cut = false;
    if (t > 0 && t < workers) {
        mine = start[t].unit;
        inside = mine >= 0 && start[t].tile > 0;
        cut = inside && !(start[t - 1].unit == mine && start[t - 1].tile > 0);
    }
    const unsigned m = __ballot_sync(~0u, cut);
    if (t < 256 && (t & 31) == 0) counts[t >> 5] = __popc(m);
    __syncthreads();
    if (cut) {
        int before = __popc(m & ((1u << (t & 31)) - 1));
        for (int w = 0; w < t >> 5; ++w) before += counts[w];
        if (before == x) at = t, cut_unit = mine;
    }
    __syncthreads();
    if (at == 0) return false;
    unit = cut_unit;
    first = at - 1;
    last = first + __syncthreads_count(inside && mine == unit);
    return true;
}

// The kernels: a pair of SMs for up to 128 heads; and one SM for up to 32 heads and 8-bit
// rows, whose conversion, done twice by a pair, bounds them there (256 requests x 2048
// rows: 102 against 204 us with 16 heads, 128 against 206 with 32; a form for 48 heads took
// 262 where the pair takes 209, one for 16-bit rows 154 where it takes 140 with 16).
constexpr int kNarrowHeads = 32;
cudaError_t launch_pair(const hs_attend_t& a, int sms, cudaStream_t s);
cudaError_t launch_narrow(const hs_attend_t& a, int sms, cudaStream_t s);
size_t pair_workspace(int64_t units, int64_t tiles);
size_t narrow_workspace(int64_t units, int64_t tiles, int heads);

}  // namespace hs_attn
