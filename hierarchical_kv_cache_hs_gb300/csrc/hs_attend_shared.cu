// hs_latent_attend_shared: absorbed latent attention of a batch over a prefix that all its
// requests share, joined with their own rows' part (hs_latent_attend).
//
// All queries of the batch (request, position, head) form one line; a unit is 128 of them
// and the prefix's rows are the same for every unit, so this is one dense product: S = Q K^T,
// O = softmax(S) K[:, :512].  A pair of SMs (a cluster of two CTAs) takes a unit, 64 queries
// in each CTA, and walks the rows in tiles of 128: tcgen05 products of the pair (M = 128)
// accumulate S (64 columns a CTA) and the whole of O (256 columns) in tensor memory, which
// also holds 6 of the queries' 9 blocks of 64 channels (192 columns).  The copy engine
// brings rows by a tensor map: of each tile a CTA gets its 64 rows whole (its half of
// Q K^T's B operand, in three groups of three blocks) and all 128 rows' half of the latent
// channels (its half of the second product's B operand, in four groups of two blocks); both
// kinds go through rings, so that copies run about a tile ahead.
//
// Bound by the tensor cores: a tile takes 2,370 clocks where its products alone need 2,210 (8-bit rows 2,600, their
// softmax multiplies scales): 64 requests x 128 heads x 32,768 rows take 314 us in a burst, 1.86 PFLOP/s, and 340 to
// 375 under the power cap, with the own rows' part and the join.  Tiles of 128 rows, since a product of 128 x 64 x 16
// takes 26 clocks where one of 128 x 128 x 16 takes 33 (its A operand is read once for twice the columns); one buffer
// of S is enough, since O(t) stands between S(t+1) and S(t+2).
//
// Few tiles are bound by what surrounds them: the queries' way in (3 us), a pair's sums' way out (3 us), the join.
// The own rows' part, whose tiles follow one another in latency, then runs beside this kernel on SMs of its own
// (pairs_beside), and a prefix is widened meanwhile.
//
// Warps of a CTA: 0-3 queries, softmax and outputs, 4 brings keys, 5 values, 6 issues the
// products (in the pair's first CTA), in the order S(t+1), O(t), so that a tile's softmax
// has the time of both.
//
// A prefix of 8-bit rows is widened to fp16 in the workspace first (exactly; the row scales
// multiply scores and weights): each row is read by every unit, so it is widened once
// instead of once a unit.  So is one with lengths: there a row that some requests do not
// see may hold anything, and weights of 0 times values that are not finite would be NaN;
// such a row becomes zeros with a NaN in its rotary channels, which only keys have.
#include <cuda.h>

#include <atomic>

#include "hs_attend.h"
#include "hs_pieces.h"

namespace hs_attn {
namespace {

constexpr int kThreads = 7 * 32;
constexpr int kRows = 128;  // rows a tile

constexpr int kQTmem = 6;
constexpr int kBlock = 64 * 128;                   // bytes of 64 rows x 64 channels
constexpr int kKGroup = 3 * kBlock, kVGroup = 2 * kBlock;
constexpr int kKStages = 4, kVStages = 5;
constexpr int kOffK = (9 - kQTmem) * kBlock;       // the queries' other blocks lie before
constexpr int kOffV = kOffK + kKStages * kKGroup;
constexpr int kOffP = kOffV + kVStages * kVGroup;  // [64 keys' block][64 queries][128 B]
constexpr int kOffAux = kOffP + 2 * kBlock;

struct Aux {
    uint64_t kfull[kKStages], kfree[kKStages], vfull[kVStages], vfree[kVStages], qready, sfull, sread, pready, pvdone, spare;
    uint64_t scales_full[2], scales_free[2];
    uint32_t tmem;
    int dead;
    Piece piece;
    int8_t q_up[64];  // power of two on a bf16 query held in fp16
    float red[2][128];
    alignas(16) float scales[2][2][kRows];  // of 8-bit rows, and their logarithms, by the tile's parity
};
constexpr int kSmem = kOffAux + (int)sizeof(Aux);
static_assert(kSmem <= 232448, "shared memory");

// What a pair leaves of a unit: its queries' sums, unscaled.
struct Sums {
    float o[128][512];
    float ref[128], sum[128];
};

constexpr uint32_t kColO = 0, kColS = 256, kColQ = 320;  // tensor memory columns

struct SharedArgs : Cut {
    hs_attend_t a;              // queries and outputs
    const int32_t* prefix_lengths;
    int64_t prefix_rows;
    int64_t queries;            // below 2^31
    const float* scales;        // of 8-bit rows
    const float* log_scales;    // base 2, not below kLeastLogScale
    const float* own_lse;       // NULL: no own rows
    const float* own_out;       // their part, [queries][512]
    Sums* parts;                // two a pair, then one a unit with all_join
    bool all_join;              // units leave through the join, whole ones too
    Start* starts;              // with lengths: where each pair's piece starts
    int* error;
};

__device__ __forceinline__ int64_t seen_rows(const SharedArgs& g, int64_t request)  // of the prefix
{
    if (!g.prefix_lengths) return g.prefix_rows;
    const int64_t n = g.prefix_lengths[request];
    return n < 0 ? 0 : n > g.prefix_rows ? g.prefix_rows : n;
}
__device__ __forceinline__ int request_of(const SharedArgs& g, int64_t query)
{
    return (int)((unsigned)query / ((unsigned)g.a.positions * (unsigned)g.a.heads));
}
// Where a query's vector begins in an array of these strides.
__device__ __forceinline__ int64_t offset_of(const SharedArgs& g, int64_t query, const int64_t* stride)
{
    const unsigned pos = (unsigned)query / (unsigned)g.a.heads, b = pos / (unsigned)g.a.positions;
    return b * stride[0] + (pos - b * g.a.positions) * stride[1] + ((unsigned)query - pos * g.a.heads) * stride[2];
}

// Tiles of a unit: up to the last row that one of its queries sees, one at least.
__host__ __device__ __forceinline__ int tiles_to(long long rows) { return rows <= kRows ? 1 : (int)((rows + kRows - 1) / kRows); }
__device__ __forceinline__ int tiles_of(const SharedArgs& g, int unit)
{
    const int64_t q0 = (int64_t)unit * 128;
    const int last = request_of(g, min(q0 + 128, g.queries) - 1);
    long long most = 0;
    for (int b = request_of(g, q0); b <= last; ++b) most = max(most, (long long)seen_rows(g, b));
    return tiles_to(most);
}

// Pair i's piece of a line whose units have tiles of their own, with lengths: the line's equal parts, as line_piece's
// (a whole warp calls it).
__device__ Piece ragged_piece(const SharedArgs& g, int i)
{
    const int lane = threadIdx.x & 31;
    long long tiles = 0;
    for (int u = lane; u < g.units; u += 32) tiles += tiles_of(g, u);
    for (int o = 16; o; o >>= 1) tiles += __shfl_xor_sync(~0u, tiles, o);
    const long long n = tiles < g.workers ? tiles : g.workers, line = tiles + (long long)g.cost * (g.units - 1);
    if (i >= n) return {0, 0, 0};
    const long long places[2] = {g.cost + line * i / n, g.cost + line * (i + 1) / n};  // of this piece and the next
    long long passed = 0, before[2] = {0, tiles};  // tiles before each
    Piece p = {0, 0, 0};
    for (int u0 = 0; u0 < g.units && passed <= places[1]; u0 += 32) {
        const int u = u0 + lane, t = u < g.units ? tiles_of(g, u) : 0;
        const long long mine = t ? t + g.cost : 0;
        long long incl = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const long long up = __shfl_up_sync(~0u, incl, o);
            if (lane >= o) incl += up;
        }
        const long long at = passed + incl - mine;  // where this unit begins
        for (int k = 0; k < 2; ++k) {
            const unsigned here = __ballot_sync(~0u, places[k] >= at && places[k] < at + mine);
            if (!here) continue;
            const int src = __ffs(here) - 1, tile = max(0, (int)(places[k] - at) - g.cost);
            before[k] = __shfl_sync(~0u, at - (long long)g.cost * u + tile, src);
            if (k == 0) p.unit = u0 + src, p.tile = __shfl_sync(~0u, tile, src);
        }
        passed += __shfl_sync(~0u, incl, 31);
    }
    p.count = before[1] - before[0];
    return p;
}

struct Stretch {  // the units, or parts of units, of a piece (a whole warp walks it)
    const SharedArgs& g;
    long long left;
    int unit, tile;
    int at, t0, t1;  // the current unit and its tiles
    bool whole;
    __device__ Stretch(const SharedArgs& args, const Piece& x) : g(args), left(x.count), unit(x.unit), tile(x.tile) {}
    __device__ bool next()
    {
        if (left <= 0) return false;
        int tiles = g.unit_tiles;
        if (g.prefix_lengths) {  // tiles_of, by the warp
            const int64_t q0 = (int64_t)unit * 128;
            const int last = request_of(g, min(q0 + 128, g.queries) - 1);
            long long most = 0;
            for (int b = request_of(g, q0) + (threadIdx.x & 31); b <= last; b += 32) most = max(most, (long long)seen_rows(g, b));
            for (int o = 16; o; o >>= 1) most = max(most, __shfl_xor_sync(~0u, most, o));
            tiles = tiles_to(most);
        }
        at = unit;
        t0 = tile;
        t1 = (long long)(tiles - t0) <= left ? tiles : t0 + (int)left;
        whole = t0 == 0 && t1 == tiles;
        left -= t1 - t0;
        ++unit;
        tile = 0;
        return true;
    }
};

// One block of 64 rows x 64 channels by the tensor map; its bytes count on the barrier of the pair's first CTA.
__device__ __forceinline__ void tile_load(uint32_t dst, const CUtensorMap* map, int channel, int row, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
                 "l"(map), "r"(channel), "r"(row), "r"(bar)
                 : "memory");
}

// Keys (and 8-bit rows' scales) or values of a piece's tiles (a warp; its first lane starts the copies).
template <bool KEYS, bool SCALES> __device__ void bring(const SharedArgs& g, const CUtensorMap* map, uint32_t sbase, Aux* x, uint32_t rank)
{
    constexpr int kStages = KEYS ? kKStages : kVStages, kBlocks = KEYS ? 3 : 2, kBytes = kBlocks * kBlock;
    uint64_t* full = KEYS ? x->kfull : x->vfull;
    uint64_t* free = KEYS ? x->kfree : x->vfree;
    int stage = 0;
    uint32_t phase = 1;  // the first round waits for nothing
    asm volatile("bar.sync 2, 192;" ::: "memory");  // the first queries' loads have been sent
    long long j = 0;  // tiles so far
    Stretch w(g, x->piece);
    while (w.next())
        for (int t = w.t0; t < w.t1; ++t, ++j) {
            if (SCALES && (threadIdx.x & 31) == 0) {
                const int s = j & 1;
                wait(tc::smem_addr(&x->scales_free[s]), (uint32_t)(j >> 1 & 1) ^ 1, &x->dead, g.error);
                if (!*(volatile int*)&x->dead) {
                    const uint32_t bar = tc::smem_addr(&x->scales_full[s]);
                    tc::mbar_expect(bar, 2 * kRows * sizeof(float));
                    tc::bulk_load(tc::smem_addr(x->scales[s][0]), g.scales + (int64_t)t * kRows, kRows * sizeof(float), bar);
                    tc::bulk_load(tc::smem_addr(x->scales[s][1]), g.log_scales + (int64_t)t * kRows, kRows * sizeof(float), bar);
                }
            }
#pragma unroll 1
            for (int n = 0; n < (KEYS ? 3 : 4); ++n) {
                if ((threadIdx.x & 31) == 0) {
                    wait(tc::smem_addr(&free[stage]), phase, &x->dead, g.error);
                    if (!*(volatile int*)&x->dead) {
                        const uint32_t bar = tc::smem_addr(&full[stage]), bar0 = tc::map_to_rank(bar, 0);
                        if (rank == 0) tc::mbar_expect(bar, 2 * kBytes);
                        const uint32_t dst = sbase + (KEYS ? kOffK : kOffV) + stage * kBytes;
                        const int channel = 64 * (KEYS ? 3 * n : 4 * (int)rank + 2 * (n & 1));
                        const int row = t * kRows + 64 * (KEYS ? (int)rank : n >> 1);
#pragma unroll
                        for (int c = 0; c < kBlocks; ++c) tile_load(dst + c * kBlock, map, channel + 64 * c, row, bar0);
                    }
                }
                __syncwarp();
                if (++stage == kStages) stage = 0, phase ^= 1;
            }
        }
}

// After a wait that gave up: what was issued must be complete before tensor memory is freed.
__device__ void drain(Aux* x)
{
    if (!*(volatile int*)&x->dead) return;
    if (tc::elect_one()) tc::commit<2>(tc::smem_addr(&x->spare));
    __syncwarp();
    tc::mbar_wait(tc::smem_addr(&x->spare), 0);
}

template <typename T> __device__ void multiply(const SharedArgs& g, uint32_t sbase, Aux* x)
{
    constexpr uint32_t id_s = tc::inst_desc(HsType<T>::is_bf16, 128, kRows, false, false);
    constexpr uint32_t id_o = tc::inst_desc(HsType<T>::is_bf16, 128, 256, false, true);
    const uint32_t tmem = __shfl_sync(~0u, x->tmem, 0);
    const uint64_t q_desc = tc::smem_desc(sbase, 16, 1024), k_base = tc::smem_desc(sbase + kOffK, 16, 1024);
    const uint64_t p_desc = tc::smem_desc(sbase + kOffP, 16, 1024), v_base = tc::smem_desc(sbase + kOffV, kBlock, 1024);
    int ks = 0, vs = 0;
    uint32_t kphase = 0, vphase = 0;
    long long j = 0;  // tiles so far
    int pieces = 0;
    auto values = [&](long long i, bool first) {  // O of tile i
        wait(tc::smem_addr(&x->pready), i & 1, &x->dead, g.error);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int keys = n >> 1, half = n & 1;
            wait(tc::smem_addr(&x->vfull[vs]), vphase, &x->dead, g.error);
            __syncwarp();
            tc::fence_after();
            const uint64_t v_desc = v_base + vs * (kVGroup >> 4);
            if (tc::elect_one()) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    tc::mma_ss<2>(tmem + kColO + 128 * half, p_desc + ((keys * kBlock + k * 32) >> 4), v_desc + ((k * 2048) >> 4), id_o,
                                  !(first && keys == 0 && k == 0));
                tc::commit<2>(tc::smem_addr(&x->vfree[vs]));
                if (n == 3) tc::commit<2>(tc::smem_addr(&x->pvdone));
            }
            __syncwarp();
            if (++vs == kVStages) vs = 0, vphase ^= 1;
        }
    };
    Stretch w(g, x->piece);
    while (w.next()) {
        wait(tc::smem_addr(&x->qready), pieces++ & 1, &x->dead, g.error);
        for (int t = w.t0; t < w.t1; ++t, ++j) {
            if (j >= 1) wait(tc::smem_addr(&x->sread), (j - 1) & 1, &x->dead, g.error);  // S has been read
#pragma unroll
            for (int n = 0; n < 3; ++n) {
                wait(tc::smem_addr(&x->kfull[ks]), kphase, &x->dead, g.error);
                __syncwarp();
                tc::fence_after();
                const uint64_t k_desc = k_base + ks * (kKGroup >> 4);
                if (tc::elect_one()) {
#pragma unroll
                    for (int i = 0; i < 3; ++i)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int c = 3 * n + i;
                            const uint64_t b = k_desc + ((i * kBlock + k * 32) >> 4);
                            if (c < kQTmem)
                                tc::mma_ts<2>(tmem + kColS, tmem + kColQ + 32 * c + 8 * k, b, id_s, (c | k) != 0);
                            else
                                tc::mma_ss<2>(tmem + kColS, q_desc + (((c - kQTmem) * kBlock + k * 32) >> 4), b, id_s, true);
                        }
                    tc::commit<2>(tc::smem_addr(&x->kfree[ks]));
                    if (n == 2) tc::commit<2>(tc::smem_addr(&x->sfull));
                }
                __syncwarp();
                if (++ks == kKStages) ks = 0, kphase ^= 1;
            }
            if (t > w.t0) values(j - 1, t - 1 == w.t0);
        }
        values(j - 1, w.t1 - 1 == w.t0);
    }
    drain(x);
}

// A CTA's 64 queries to tensor and shared memory, by the four softmax warps: eight lanes read 128 bytes of a query
// together, all of a thread's 36 pieces in flight; two blocks at a time then pass through P's buffer to tensor memory
// (a pair's product of 128 rows computes half of its columns in lanes 64-127, which read their own copy of A).
template <typename T, bool E4M3>
__device__ void bring_queries(const SharedArgs& g, uint32_t sbase, uint32_t tmem, Aux* x, int64_t first, bool begin, uint32_t qready)
{
    const int t = threadIdx.x, ch = t & 7;
    uint4 v[4][9];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        const int64_t query = first + 16 * n + (t >> 3);
        const bool ok = query < g.queries;
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const T*>(g.a.q) + (ok ? offset_of(g, query, g.a.q_stride) : 0)) + ch;
#pragma unroll
        for (int c = 0; c < 9; ++c) v[n][c] = ok ? q[8 * c] : make_uint4(0, 0, 0, 0);
    }
    if (begin) asm volatile("bar.arrive 2, 192;" ::: "memory");  // the first rows' copies come behind these loads
    if constexpr (E4M3 && HsType<T>::is_bf16)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            float top = 0.f;
#pragma unroll
            for (int c = 0; c < 9; ++c) top = fmaxf(top, largest_bf16(v[n][c]));
            for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
            const int up = power_up(top);
            if (ch == 0) x->q_up[16 * n + (t >> 3)] = (int8_t)up;
#pragma unroll
            for (int c = 0; c < 9; ++c) v[n][c] = bf16_to_half(v[n][c], power_of_two(up));
        }
    auto store = [&](uint32_t block, const uint4& w, int row) {
        tc::st_shared16(block + row * 128 + ((ch ^ (row & 7)) << 4), w.x, w.y, w.z, w.w);
    };
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int c = kQTmem; c < 9; ++c) store(sbase + (c - kQTmem) * kBlock, v[n][c], 16 * n + (t >> 3));
    const int row = t & 63;
#pragma unroll
    for (int c = 0; c < kQTmem; c += 2) {
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) store(sbase + kOffP + k * kBlock, v[n][c + k], 16 * n + (t >> 3));
        asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint32_t r[32];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint4 w = tc::ld_shared16(sbase + kOffP + k * kBlock + row * 128 + ((i ^ (row & 7)) << 4));
                r[4 * i] = w.x, r[4 * i + 1] = w.y, r[4 * i + 2] = w.z, r[4 * i + 3] = w.w;
            }
            tc::tmem_st32(tmem + kColQ + 32 * (c + k), r);
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
    }
    tc::tmem_wait_st();
    tc::fence_async_shared();
    tc::fence_before();
    __syncwarp();
    if ((t & 31) == 0) tc::mbar_arrive_cluster(qready);
}

// The two parts of a query, the prefix's (sum at reference ref, in powers of two) and the own rows' (lse): the
// factors on the prefix's unscaled sums and on the own rows' output, and the whole's lse.
struct Mix {
    float prefix, own, lse;
};
__device__ __forceinline__ Mix mix(float ref, float sum, float own_lse)
{
    const bool some = sum > 0.f || sum != sum, mine = own_lse != -INFINITY;
    if (!some && !mine) return {0.f, 0.f, -INFINITY};
    const float l = own_lse * 1.4426950408889634f;
    const float top = !mine ? ref : !some ? l : fmaxf(ref, l);
    const float a = some ? tc::exp2_approx(ref - top) : 0.f, b = mine ? tc::exp2_approx(l - top) : 0.f;
    const float total = (some ? sum * a : 0.f) + b, inv = 1.f / total;
    return {a * inv, b * inv, (top + log2f(total)) * 0.6931471805599453f};
}

template <typename T, bool E4M3> __device__ void soften(const SharedArgs& g, uint32_t sbase, Aux* x, uint32_t rank, int pair)
{
    const hs_attend_t& a = g.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = threadIdx.x & 63, half = threadIdx.x >> 6;
    const uint32_t tmem = x->tmem + ((uint32_t)warp << 21);  // this warp's 32 lanes
    const uint32_t sread = tc::map_to_rank(tc::smem_addr(&x->sread), 0), pready = tc::map_to_rank(tc::smem_addr(&x->pready), 0),
                   qready = tc::map_to_rank(tc::smem_addr(&x->qready), 0);
    const float c0 = a.scale * 1.4426950408889634f;
    long long j = 0;
    bool begin = true;
    Stretch w(g, x->piece);
    while (w.next()) {
        const int64_t query = (int64_t)w.at * 128 + rank * 64 + row;
        float ref = 0.f, sum = 0.f;
        bring_queries<T, E4M3>(g, sbase, tmem, x, (int64_t)w.at * 128 + rank * 64, begin, qready);
        begin = false;
        const int64_t next = (int64_t)w.unit * 128 + rank * 64 + (threadIdx.x >> 1);
        if (w.left > 0 && next < g.queries) {  // the next unit's queries on their way to L2 (150 x 128 heads, 300 rows: 71.6 -> 69.4 us)
            const T* q = static_cast<const T*>(a.q) + offset_of(g, next, a.q_stride) + (threadIdx.x & 1) * 320;
#pragma unroll
            for (int i = 0; i < 5; ++i)
                if ((threadIdx.x & 1) * 320 + 64 * i < HS_ROW_DIM) tc::prefetch_l2(q + 64 * i);
        }
        const float c = E4M3 && HsType<T>::is_bf16 ? power_of_two(-x->q_up[row]) * c0 : c0;
        const int64_t limit = query < g.queries ? seen_rows(g, request_of(g, query)) : 0;
        bool seen = false;  // a row that counts has been met: ref is a maximum
        for (int t = w.t0; t < w.t1; ++t, ++j) {
            const int64_t key0 = (int64_t)t * kRows + 64 * half;
            const int live = (int)min(max(limit - key0, (int64_t)0), (int64_t)64);  // keys of these 64 that count
            const int s = j & 1;
            float wt[E4M3 ? 64 : 1];
            if constexpr (E4M3) {
                wait(tc::smem_addr(&x->scales_full[s]), j >> 1 & 1, &x->dead, g.error);
#pragma unroll
                for (int i = 0; i < 64; i += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(&x->scales[s][0][64 * half + i]);
                    wt[i] = f.x, wt[i + 1] = f.y, wt[i + 2] = f.z, wt[i + 3] = f.w;
                }
            }
            wait(tc::smem_addr(&x->sfull), j & 1, &x->dead, g.error);
            tc::fence_after();
            uint32_t r[2][32];
            tc::tmem_ld32(tmem + kColS, r[0]);
            tc::tmem_ld32(tmem + kColS + 32, r[1]);
            tc::tmem_wait_ld(r[0]);
            tc::tmem_wait_ld(r[1]);
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_cluster(sread);  // the next tile's scores may come
            float v[64], top = -INFINITY;
#pragma unroll
            for (int i = 0; i < 64; i += 2) {
                v[i] = __uint_as_float(r[i >> 5][i & 31]), v[i + 1] = __uint_as_float(r[i >> 5][(i & 31) + 1]);
                mul2(v[i], v[i + 1], c, c);
                if constexpr (E4M3) mul2(v[i], v[i + 1], wt[i], wt[i + 1]);
            }
            if (live < 64)
#pragma unroll
                for (int i = 0; i < 64; ++i)
                    if (i >= live) v[i] = -INFINITY;
            if constexpr (E4M3) {
#pragma unroll
                for (int i = 0; i < 64; i += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(&x->scales[s][1][64 * half + i]);
                    float lw[4] = {f.x, f.y, f.z, f.w};
                    tc::add2(lw[0], lw[1], v[i], v[i + 1]);
                    tc::add2(lw[2], lw[3], v[i + 2], v[i + 3]);
                    top = tc::max3(tc::max3(top, lw[0], lw[1]), lw[2], lw[3]);
                }
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(tc::smem_addr(&x->scales_free[s]));
            } else {
#pragma unroll
                for (int i = 0; i < 64; i += 2) top = tc::max3(top, v[i], v[i + 1]);
            }
            x->red[s][threadIdx.x] = top;
            asm volatile("bar.sync 1, 128;" ::: "memory");
            top = fmaxf(top, x->red[s][threadIdx.x ^ 64]);
            float keep = 1.f;
            if (top > -INFINITY && (!seen || top > ref + 8.f)) {
                keep = tc::exp2_approx(fminf(ref - top, 126.f));
                sum *= keep;
                ref = top;
            }
            const bool scale_o = seen && keep != 1.f;
            seen = seen || top > -INFINITY;
            uint32_t e[32];
            float sums[2] = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                float p0 = v[2 * i], p1 = v[2 * i + 1];
                tc::add2(p0, p1, -ref, -ref);
                p0 = tc::exp2_approx(p0), p1 = tc::exp2_approx(p1);
                tc::add2(sums[0], sums[1], p0, p1);
                if constexpr (E4M3) mul2(p0, p1, wt[2 * i], wt[2 * i + 1]);
                e[i] = pack2<std::conditional_t<E4M3, __half, T>>(p0, p1);
            }
            sum += sums[0] + sums[1];
            // P's buffer and O are free once the last tile's product is done
            if (j >= 1) wait(tc::smem_addr(&x->pvdone), (j - 1) & 1, &x->dead, g.error);
            if (__any_sync(~0u, scale_o)) {
                if (!scale_o) keep = 1.f;
                tc::fence_after();
#pragma unroll 1
                for (int n = 0; n < 256; n += 32) {
                    tc::tmem_ld32(tmem + kColO + n, r[0]);
                    tc::tmem_wait_ld(r[0]);
#pragma unroll
                    for (int i = 0; i < 32; ++i) r[0][i] = __float_as_uint(__uint_as_float(r[0][i]) * keep);
                    tc::tmem_st32(tmem + kColO + n, r[0]);
                }
                tc::tmem_wait_st();
            }
            const uint32_t dst = sbase + kOffP + half * kBlock + row * 128;
#pragma unroll
            for (int n = 0; n < 8; ++n) tc::st_shared16(dst + ((n ^ (row & 7)) << 4), e[4 * n], e[4 * n + 1], e[4 * n + 2], e[4 * n + 3]);
            tc::fence_async_shared();
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_cluster(pready);
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
        x->red[0][threadIdx.x] = sum;
        asm volatile("bar.sync 1, 128;" ::: "memory");
        sum += x->red[0][threadIdx.x ^ 64];
        asm volatile("bar.sync 1, 128;" ::: "memory");
        wait(tc::smem_addr(&x->pvdone), (j - 1) & 1, &x->dead, g.error);
        tc::fence_after();
        // The piece's end: O and the sums leave, through shared memory, so that eight lanes write 128 bytes of a query
        // together: 32 channels of each half at a time, [half][query][128 B], in P's buffer and the queries' by turns.
        const int64_t query0 = (int64_t)w.at * 128 + rank * 64;
        const int row0 = threadIdx.x >> 3, ch = threadIdx.x & 7;  // this thread takes each sixteenth of the buffer's rows
        auto leave = [&](auto&& put) {
#pragma unroll 2
            for (int n = 0; n < 256; n += 32) {
                const uint32_t buffer = sbase + (n & 32 ? 0 : kOffP);
                uint32_t r[32];
                __syncwarp();
                tc::tmem_ld32(tmem + kColO + n, r);
                tc::tmem_wait_ld(r);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    tc::st_shared16(buffer + threadIdx.x * 128 + ((i ^ (row & 7)) << 4), r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
                asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int at = 16 * i + row0;
                    put(i, 256 * (i >> 2) + n + 4 * ch, tc::ld_shared16(buffer + at * 128 + ((ch ^ (at & 7)) << 4)));
                }
            }
        };
        if (g.all_join || !w.whole) {
            Sums* part = g.parts + (w.whole ? 2 * kMaxPairs + w.at : 2 * pair + (w.t0 == 0));
            leave([&](int i, int c, const uint4& v) {
                const int at = 16 * (i & 3) + row0;
                if (query0 + at < g.queries) *reinterpret_cast<uint4*>(&part->o[rank * 64 + at][c]) = v;
            });
            if (half == 0) part->ref[rank * 64 + row] = ref, part->sum[rank * 64 + row] = sum;
        } else {  // joined with the own rows' part: the call's outputs
            asm volatile("griddepcontrol.wait;" ::: "memory");
            const bool there = query < g.queries;
            const Mix m = mix(ref, sum, there && g.own_lse ? g.own_lse[query] : -INFINITY);
            if (half == 0) x->red[0][row] = m.prefix, x->red[1][row] = m.own;
            if (there && a.lse && half == 0) a.lse[query] = m.lse;
            asm volatile("bar.sync 1, 128;" ::: "memory");
            T* out[4];  // this thread's rows, and their factors
            float2 f[4];
            bool some[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = 16 * i + row0;
                some[i] = query0 + at < g.queries;
                out[i] = static_cast<T*>(a.out) + (some[i] ? offset_of(g, query0 + at, a.out_stride) : 0);
                f[i] = make_float2(x->red[0][at], x->red[1][at]);
            }
            const float* own = g.own_out + (query0 + row0) * HS_LATENT_DIM;
            float4 old[8];
            auto bring = [&](int n) {  // a step ahead
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    old[i] = some[i & 3] && f[i & 3].y != 0.f && n < 256
                                 ? *reinterpret_cast<const float4*>(own + 16 * (i & 3) * HS_LATENT_DIM + 256 * (i >> 2) + n + 4 * ch)
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
            };
            bring(0);
            leave([&](int i, int c, const uint4& v) {
                const float2 e = f[i & 3];
                auto joined = [&](uint32_t o, float own) { return (e.x != 0.f ? __uint_as_float(o) * e.x : 0.f) + (e.y != 0.f ? own * e.y : 0.f); };
                if (some[i & 3])
                    *reinterpret_cast<uint2*>(out[i & 3] + c) = make_uint2(pack2<T>(joined(v.x, old[i].x), joined(v.y, old[i].y)), pack2<T>(joined(v.z, old[i].z), joined(v.w, old[i].w)));
                if (i == 7) bring(c - 256 - 4 * ch + 32);
            });
        }
        tc::fence_before();
        asm volatile("bar.sync 1, 128;" ::: "memory");  // the buffers have been read
    }
}

template <typename T, bool E4M3>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    hs_attend_shared_kernel(const __grid_constant__ SharedArgs g, const __grid_constant__ CUtensorMap map)
{
    using Operand = std::conditional_t<E4M3, __half, T>;
    extern __shared__ __align__(1024) uint8_t base[];  // the swizzled blocks need 1024
    const uint32_t sbase = tc::smem_addr(base);
    Aux* x = reinterpret_cast<Aux*>(base + kOffAux);
    const uint32_t rank = tc::cluster_rank();
    const int pair = blockIdx.x >> 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join may queue up behind this grid
    if (warp == 0) tc::tmem_alloc<2>(tc::smem_addr(&x->tmem), 512);
    if (warp == 5 && g.prefix_lengths) {
        const Piece p = ragged_piece(g, pair);
        if (lane == 0) x->piece = p;
        if (lane == 0 && rank == 0) g.starts[pair] = {p.count > 0 ? p.unit : -1, p.tile};
    }
    if (warp == 6 && lane == 0) {
        if (!g.prefix_lengths) x->piece = g.flat ? line_piece(g, pair) : whole_piece(g, pair);
        x->dead = 0;
        for (int i = 0; i < kKStages; ++i) tc::mbar_init(tc::smem_addr(&x->kfull[i]), 1), tc::mbar_init(tc::smem_addr(&x->kfree[i]), 1);
        for (int i = 0; i < kVStages; ++i) tc::mbar_init(tc::smem_addr(&x->vfull[i]), 1), tc::mbar_init(tc::smem_addr(&x->vfree[i]), 1);
        for (int i = 0; i < 2; ++i) tc::mbar_init(tc::smem_addr(&x->scales_full[i]), 1), tc::mbar_init(tc::smem_addr(&x->scales_free[i]), 4);
        tc::mbar_init(tc::smem_addr(&x->qready), 8);
        tc::mbar_init(tc::smem_addr(&x->sfull), 1);
        tc::mbar_init(tc::smem_addr(&x->sread), 8);
        tc::mbar_init(tc::smem_addr(&x->pready), 8);
        tc::mbar_init(tc::smem_addr(&x->pvdone), 1);
        tc::mbar_init(tc::smem_addr(&x->spare), 1);
        tc::mbar_init_fence();
    }
    tc::fence_before();
    __syncwarp();
    __syncthreads();
    tc::cluster_sync();
    tc::fence_after();

    if (x->piece.count > 0) {
        if (warp < 4)
            soften<T, E4M3>(g, sbase, x, rank, pair);
        else if (warp == 4)
            bring<true, E4M3>(g, &map, sbase, x, rank);
        else if (warp == 5)
            bring<false, false>(g, &map, sbase, x, rank);
        else if (rank == 0)
            multiply<Operand>(g, sbase, x);
        if (*(volatile int*)&x->dead) {  // copies may be in flight, and count on the first CTA's barriers: half a millisecond
            const long long t0 = clock64();
            while (clock64() - t0 < 1000000) {}
        }
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    tc::cluster_sync_relaxed();  // no CTA leaves while the other may signal it
    tc::fence_after();
    if (warp == 0) tc::tmem_free<2>(x->tmem, 512);
    asm volatile("griddepcontrol.wait;" ::: "memory");  // so that the join comes after the own rows' part, too
}

// Where pair i's piece of the line begins, and the pair whose piece holds a place.
__device__ __forceinline__ long long piece_begin(const Cut& g, int i) { return g.cost + g.share * i + min(i, g.extra); }
__device__ __forceinline__ int piece_at(const Cut& g, long long at)
{
    at -= g.cost;
    const long long longer = (g.share + 1) * g.extra;
    const bool in = at < longer;
    const long long from = in ? at : at - longer, by = g.share + in;
    return (in ? 0 : g.extra) + (from < 0x7fffffff && by < 0x7fffffff ? (int)((unsigned)from / (unsigned)by) : (int)(from / by));
}

// Join the pieces of units with one another and with the own rows' part: blocks y take unit y (all_join) or, where
// whole units have left by themselves, the unit that pair y + 1 begins inside, if it is the first to do so (with lengths,
// the y-th such unit).  Each query's 128 channels are one or several warps', which share its pieces; one pass, and the
// order of the sums is fixed.
template <int N> struct Joined {  // of 4 N channels
    float top, sum;
    float4 acc[N];
    __device__ void add(float ref, float l, const float4 (&o)[N])
    {
        // without a branch, so that the loads of several pieces are in flight; a sum of 0: no row counted
        const float up = l == 0.f ? top : fmaxf(top, ref), base = up == -INFINITY ? 0.f : up;
        const float keep = tc::exp2_approx(top - base), w = l == 0.f ? 0.f : tc::exp2_approx(ref - base);
        top = up;
        sum = sum * keep + w * l;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            acc[k].x = acc[k].x * keep + (l == 0.f ? 0.f : w * o[k].x);
            acc[k].y = acc[k].y * keep + (l == 0.f ? 0.f : w * o[k].y);
            acc[k].z = acc[k].z * keep + (l == 0.f ? 0.f : w * o[k].z);
            acc[k].w = acc[k].w * keep + (l == 0.f ? 0.f : w * o[k].w);
        }
    }
};
// N: of 128 channels, a warp's.
template <typename T, int WARPS, int N> __global__ void __launch_bounds__(256) hs_attend_shared_join_kernel(const __grid_constant__ SharedArgs g)
{
    __shared__ Joined<N> others[WARPS > 1 ? 8 : 1][32];
    const hs_attend_t& a = g.a;
    int unit = blockIdx.y, first = 0, last = 0;
    if (g.prefix_lengths && g.all_join) {
        // The pairs that have the unit: the last whose piece starts at its start or before, to the last that starts
        // inside it or before.
        asm volatile("griddepcontrol.wait;" ::: "memory");
        for (int i0 = 0; i0 < g.workers; i0 += 32) {
            const int i = i0 + (threadIdx.x & 31);
            const Start s = i < g.workers ? g.starts[i] : Start{-1, 0};
            const unsigned before = __ballot_sync(~0u, s.unit >= 0 && (s.unit < unit || (s.unit == unit && s.tile == 0)));
            const unsigned inside = __ballot_sync(~0u, s.unit >= 0 && s.unit <= unit);
            if (before) first = i0 + 31 - __clz(before);
            if (inside) last = i0 + 31 - __clz(inside);
        }
    } else if (g.prefix_lengths) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (!find_cut(g.starts, g.workers, blockIdx.y, unit, first, last)) return;
    } else if (g.flat) {
        const int per = g.unit_tiles + g.cost;
        const long long here = piece_begin(g, blockIdx.y + 1);
        if (!g.all_join) unit = here < 0x7fffffff ? (int)((unsigned)here / (unsigned)per) : (int)(here / per);
        const long long begin = (long long)unit * per + g.cost;  // the unit's first tile
        first = piece_at(g, begin), last = piece_at(g, begin + g.unit_tiles - 1);
        if (!g.all_join && (here <= begin || first != (int)blockIdx.y)) {
            asm volatile("griddepcontrol.wait;" ::: "memory");  // what follows this grid follows the pairs' too
            return;
        }
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp % WARPS;
    const int id = blockIdx.x * (8 / WARPS) + warp / WARPS, row = id / (4 / N), ch = 128 * N * (id % (4 / N)) + 4 * lane;
    const int64_t query = (int64_t)unit * 128 + row;
    if (query >= g.queries) return;  // all warps of the query
    T* out = static_cast<T*>(a.out) + offset_of(g, query, a.out_stride) + ch;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float own_lse = -INFINITY;
    float4 old[N];
#pragma unroll
    for (int k = 0; k < N; ++k) old[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (g.own_lse && part == 0) {
        own_lse = g.own_lse[query];
#pragma unroll
        for (int k = 0; k < N; ++k) old[k] = *reinterpret_cast<const float4*>(g.own_out + query * HS_LATENT_DIM + ch + 128 * k);
    }
    Joined<N> j;
    j.top = -INFINITY, j.sum = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k) j.acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kAtOnce = WARPS > 1 ? 8 : 4;  // 75 pieces 31.2 us against 33.1 with 4 (1 request x 16
                                               // heads, 65,536 rows); units of 6 pieces 48 against 47
#pragma unroll kAtOnce
    for (int n = first + part; n <= last; n += WARPS) {
        const Sums& p = g.parts[first == last ? 2 * kMaxPairs + unit : 2 * n + (n == first)];
        float4 o[N];
#pragma unroll
        for (int k = 0; k < N; ++k) o[k] = *reinterpret_cast<const float4*>(&p.o[row][ch + 128 * k]);
        j.add(p.ref[row], p.sum[row], o);
    }
    if constexpr (WARPS > 1) {
        if (part) others[warp][lane] = j;
        asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / WARPS), "r"(32 * WARPS) : "memory");
        if (part) return;
#pragma unroll
        for (int w = 1; w < WARPS; ++w) j.add(others[warp + w][lane].top, others[warp + w][lane].sum, others[warp + w][lane].acc);
    }
    const Mix m = mix(j.top, j.sum, own_lse);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        auto joined = [&](float sum, float own) { return (j.sum == 0.f ? 0.f : sum * m.prefix) + (m.own != 0.f ? own * m.own : 0.f); };
        *reinterpret_cast<uint2*>(out + 128 * k) = make_uint2(pack2<T>(joined(j.acc[k].x, old[k].x), joined(j.acc[k].y, old[k].y)),
                                                             pack2<T>(joined(j.acc[k].z, old[k].z), joined(j.acc[k].w, old[k].w)));
    }
    if (a.lse && ch == 0) a.lse[query] = m.lse;
}

// The prefix's rows as 16-bit operands.  8-bit values become fp16 beside their scales (and base-2 logarithms; those of
// the last tile's absent rows too).  A row with a value that is not finite becomes zeros with NaN in a rotary channel.
// Laid out as hs_latent_read's kernel: 36 threads a row, three rows of a thread on their way together (65,536 8-bit rows
// 18.5 us, the 113 MB at 6.1 TB/s; a warp a row took 1 us more).
constexpr int kWidenLine = 8, kWidenAhead = 3, kWidenRows = kWidenLine * kWidenAhead;

template <typename T, bool E4M3>
__global__ void __launch_bounds__(kRowThreads * kWidenLine)
    hs_prefix_kernel(const uint8_t* rows, int64_t row_stride, int64_t n, int64_t padded, uint8_t* wide, float* scales, float* log_scales,
                     const bool rows32, const bool wide32)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the own rows' part needs nothing from here
    __shared__ int bad[kWidenRows];
    const int line = threadIdx.x / kRowThreads, ch = 16 * (threadIdx.x - line * kRowThreads);
    const int64_t first = (int64_t)blockIdx.x * kWidenRows + line;
    if (threadIdx.x < kWidenRows) bad[threadIdx.x] = 0;
    uint4 v[kWidenAhead][2];
    float scale[kWidenAhead];
#pragma unroll
    for (int m = 0; m < kWidenAhead; ++m) {
        const int64_t i = first + m * kWidenLine;
        const uint8_t* row = rows + i * row_stride;
        v[m][0] = v[m][1] = make_uint4(0, 0, 0, 0);
        scale[m] = 1.f;
        if (i >= n) continue;
        if constexpr (E4M3)
            v[m][1] = *reinterpret_cast<const uint4*>(row + ch), scale[m] = *reinterpret_cast<const float*>(row + HS_ROW8_SCALE);
        else
            load32(row + 2 * ch, rows32, v[m]);
    }
    __syncthreads();  // the marks are clear
#pragma unroll
    for (int m = 0; m < kWidenAhead; ++m) {
        if constexpr (E4M3) {
            const uint4 e = v[m][1];
            widen(e.x, v[m][0].x, v[m][0].y), widen(e.y, v[m][0].z, v[m][0].w);
            widen(e.z, v[m][1].x, v[m][1].y), widen(e.w, v[m][1].z, v[m][1].w);
        }
        constexpr uint32_t kAll = HsType<T>::is_bf16 ? 0x7f80u : 0x7c00u;  // the exponent of what is not finite
        bool some = E4M3 && !(fabsf(scale[m]) < INFINITY);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t w[4] = {v[m][k].x, v[m][k].y, v[m][k].z, v[m][k].w};
#pragma unroll
            for (int q = 0; q < 4; ++q) some = some || (w[q] & kAll) == kAll || (w[q] >> 16 & kAll) == kAll;
        }
        if (some) bad[m * kWidenLine + line] = 1;
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < kWidenAhead; ++m) {
        const int64_t i = first + m * kWidenLine;
        const bool none = bad[m * kWidenLine + line] != 0;
        if (none) v[m][0] = make_uint4(0, 0, 0, 0), v[m][1] = make_uint4(0, ch == HS_ROW_DIM - 16 ? 0x7fffu : 0u, 0, 0);
        if (i < n) store32(wide + i * (2 * HS_ROW_DIM) + 2 * ch, wide32, v[m][0], v[m][1]);
        if (E4M3 && ch == 0 && i < padded) {
            const bool plain = i >= n || none;
            scales[i] = plain ? 1.f : scale[m];
            log_scales[i] = plain ? 0.f : fmaxf(log2f(fabsf(scale[m])), kLeastLogScale);
        }
    }
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                   const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
std::atomic<EncodeTiledFn> g_encode{nullptr};

// A map of rows [n][576] of 16 bits, in blocks of 64 x 64; rows behind the last are zeros.
cudaError_t map_rows(CUtensorMap* map, const void* rows, int64_t n, int64_t stride)
{
    EncodeTiledFn fn = g_encode.load();
    if (!fn) {  // found through the runtime, so that the library does not link the driver library itself
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q);
        if (e != cudaSuccess) return e;
        if (q != cudaDriverEntryPointSuccess || !p) return cudaErrorSymbolNotFound;
        fn = reinterpret_cast<EncodeTiledFn>(p);
        g_encode.store(fn);
    }
    const cuuint64_t dims[2] = {HS_ROW_DIM, (cuuint64_t)n}, strides[1] = {(cuuint64_t)(n > 1 ? stride : 2 * HS_ROW_DIM)};
    const cuuint32_t box[2] = {64, 64}, step[2] = {1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(rows), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

int64_t padded_rows(int64_t n) { return (n + kRows - 1) / kRows * kRows; }

// Up to this many units leave through the join: it has many blocks for the work that then is left when the own rows'
// part is done, where a pair of SMs takes 6 us for a unit.  More have not the place (0.26 MB a unit), and not the need:
// 200 units 191 us so, and 196 through the join (4096 rows); 300 434 and 442 (8192 rows).  As they wait for the own rows'
// part, that then comes first: beside it, 200 units of 100 rows took 131 us, and take 79.
constexpr int64_t kJoinUnits = 2 * kMaxPairs;

// Workspace: hs_latent_attend's for the own rows (its error word is the call's), then their lse and outputs (in 32 bits:
// they are rounded once, in the join; twice, outputs of mostly own rows were off by 0.0027, once by 0.0021, in bf16), the partial results,
// where the pairs' pieces start, the prefix's rows in 16 bits, scales and their logarithms.  More requests never need
// less, so that a workspace for a loop's largest batch serves its smaller ones: units above kJoinUnits have its sums, too.
struct Layout {
    size_t lse, own, parts, starts, rows, scales, logs, end;
    Layout(int batch, int positions, int heads, int64_t own_rows, int64_t prefix_rows)
    {
        auto after = [](size_t at, size_t bytes) { return (at + bytes + 255) / 256 * 256; };
        lse = after(0, hs_attend_workspace_bytes(batch, positions, heads, own_rows));
        own = after(lse, sizeof(float) * batch * positions * (size_t)heads);
        parts = after(own, own_rows > 0 ? sizeof(float) * HS_LATENT_DIM * batch * positions * (size_t)heads : 0);
        const int64_t units = ((int64_t)batch * positions * heads + 127) / 128;
        starts = after(parts, sizeof(Sums) * (2 * kMaxPairs + (units < kJoinUnits ? units : kJoinUnits)));
        rows = after(starts, sizeof(Start) * kMaxPairs);
        scales = after(rows, 2 * HS_ROW_DIM * (size_t)prefix_rows);
        logs = after(scales, sizeof(float) * padded_rows(prefix_rows));
        end = after(logs, sizeof(float) * padded_rows(prefix_rows));
    }
};

template <typename T, bool E4M3> cudaError_t launch(const SharedArgs& g, const CUtensorMap& map, cudaStream_t s)
{
    cudaError_t e = cudaFuncSetAttribute(hs_attend_shared_kernel<T, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (g.own_lse)  // may begin while the own rows' part runs out, and reads it at its units' ends
        e = launch_after(hs_attend_shared_kernel<T, E4M3>, dim3(2 * g.workers), kThreads, kSmem, s, g, map);
    else
        hs_attend_shared_kernel<T, E4M3><<<2 * g.workers, kThreads, kSmem, s>>>(g, map), e = cudaGetLastError();
    if (e != cudaSuccess || (!g.all_join && (!g.flat || g.workers <= 1))) return e;
    // Eight warps share the pieces where a unit has many: 1 unit of 76 pieces 58 us against 89 (8 requests x 16 heads,
    // 65,536 rows); of 10 to 20 pieces 40 and 70 against 43 and 74 with a warp (16 requests x 3 x 32 heads, 4096 rows;
    // 64 x 32 heads, 16,384 rows), where two warps share them.  A warp takes 256 channels where there are enough warps:
    // 80 units 65 us against 71, 100 units 61 against 66; but 8 units 51.5 against 50.
    const int blocks = g.all_join ? g.units : g.workers - 1;
    if (g.workers >= 16 * g.units) return launch_after(hs_attend_shared_join_kernel<T, 8, 1>, dim3(512, blocks), 256, 0, s, g);
    if (g.units < 16) return launch_after(hs_attend_shared_join_kernel<T, 1, 1>, dim3(64, blocks), 256, 0, s, g);
    return launch_after(hs_attend_shared_join_kernel<T, 1, 2>, dim3(32, blocks), 256, 0, s, g);
}

// The prefix's rows in the workspace, in 16 bits.
cudaError_t widen_prefix(SharedArgs& g, const hs_prefix_t& p, uint8_t* ws, const Layout& at, cudaStream_t s)
{
    const int64_t padded = padded_rows(p.n_rows);
    const uint8_t* from = static_cast<const uint8_t*>(p.rows);
    uint8_t* wide = ws + at.rows;
    float* scales = reinterpret_cast<float*>(ws + at.scales);
    float* logs = reinterpret_cast<float*>(ws + at.logs);
    const bool rows32 = ((uintptr_t)from | (p.n_rows > 1 ? (uintptr_t)p.row_stride : 0)) % 32 == 0, wide32 = (uintptr_t)wide % 32 == 0;
    auto run = [&](auto kernel) {
        const unsigned grid = (unsigned)((padded + kWidenRows - 1) / kWidenRows);
        kernel<<<grid, kRowThreads * kWidenLine, 0, s>>>(from, p.row_stride, p.n_rows, padded, wide, scales, logs, rows32, wide32);
    };
    if (g.a.row_format == HS_ROWS_E4M3)
        run(hs_prefix_kernel<__half, true>);
    else if (g.a.dtype == HS_TYPE_BF16)
        run(hs_prefix_kernel<__nv_bfloat16, false>);
    else
        run(hs_prefix_kernel<__half, false>);
    g.scales = scales;
    g.log_scales = logs;
    return cudaGetLastError();
}

}  // namespace
}  // namespace hs_attn

size_t hs_attend_shared_workspace_bytes(int batch, int positions, int heads, int64_t rows, int64_t prefix_rows)
{
    return hs_attn::Layout(batch, positions, heads, rows, prefix_rows).end;
}

cudaError_t hs_launch_attend_shared(const hs_attend_t& a, const hs_prefix_t& p, cudaStream_t s)
{
    using namespace hs_attn;
    if (p.n_rows == 0) return hs_launch_attend(a, s);
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const Layout at(a.batch, a.positions, a.heads, a.slots ? a.entries : a.n_rows, p.n_rows);
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    SharedArgs g = {};
    g.a = a;
    g.prefix_lengths = p.lengths;
    g.prefix_rows = p.n_rows;
    g.queries = (int64_t)a.batch * a.positions * a.heads;
    g.parts = reinterpret_cast<Sums*>(ws + at.parts);
    g.starts = reinterpret_cast<Start*>(ws + at.starts);
    g.all_join = g.queries <= 128 * kJoinUnits;
    g.error = reinterpret_cast<int*>(ws);
    CUtensorMap map;
    const bool e4m3 = a.row_format == HS_ROWS_E4M3, widened = e4m3 || p.lengths;
    if (widened) {
        e = widen_prefix(g, p, ws, at, s);
        if (e == cudaSuccess) e = map_rows(&map, ws + at.rows, p.n_rows, 2 * HS_ROW_DIM);
    } else {
        e = map_rows(&map, p.rows, p.n_rows, p.row_stride);
    }
    if (e != cudaSuccess) return e;
    g.units = (int)((g.queries + 127) / 128);
    const int all = sms / 2 < kMaxPairs ? (sms > 1 ? sms / 2 : 1) : kMaxPairs;
    const bool own_rows = a.n_rows > 0 && (!a.slots || a.entries > 0);
    const bool beside = own_rows && g.all_join;  // units that leave by themselves wait for their own rows' part
    const int own_pairs = beside ? pairs_beside(a, p.lengths, g.units, tiles_to(p.n_rows), all) : all, pairs = own_pairs < all ? all - own_pairs : all;
    // The own rows' part comes directly before the prefix's kernel, which begins on the SMs that it leaves.
    if (own_rows) {
        hs_attend_t own = a;
        own.lse = reinterpret_cast<float*>(ws + at.lse);
        g.own_lse = own.lse;
        g.own_out = reinterpret_cast<float*>(ws + at.own);
        e = hs_launch_attend(own, s, widened, own_pairs, reinterpret_cast<float*>(ws + at.own));
        if (e != cudaSuccess) return e;
    }
    g.cut(pairs, p.n_rows, 5, kSharedUnitCost, kRows);
    if (g.flat) {
        // Each pair's partial results go out and come back, 1.2 us for ten pairs where a tile takes 1.4: few tiles take
        // fewer pairs.
        auto time = [&](int64_t n) { return ((int64_t)g.units * (g.unit_tiles + kSharedUnitCost) + n - 1) / n * 1400 + n * 120; };
        int best = pairs;
        for (int n = pairs - 1; n > 0 && n > g.units; --n)
            if (time(n) < time(best)) best = n;
        g.cut(best, p.n_rows, 5, kSharedUnitCost, kRows);
    }
    if (p.lengths && !g.flat) {  // the device cuts the line
        const int64_t tiles = (int64_t)g.units * g.unit_tiles;
        g.workers = (int)(tiles < pairs ? tiles : pairs);
        g.flat = 1;
    }
    if (a.dtype == HS_TYPE_BF16) return e4m3 ? launch<__nv_bfloat16, true>(g, map, s) : launch<__nv_bfloat16, false>(g, map, s);
    return e4m3 ? launch<__half, true>(g, map, s) : launch<__half, false>(g, map, s);
}
