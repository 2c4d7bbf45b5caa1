// hs_latent_attend: absorbed latent attention over listed or leading rows.
//
// For one request and position, S = Q K^T and O = softmax(S) K[:, :512], with
// the same 576-channel rows as keys and values of up to 128 heads.  A pair of
// SMs (a cluster of two CTAs) takes up to 128 heads, 64 in each CTA, and walks
// the rows in tiles of 64; tcgen05 products of the pair (cta_group::2, M = 128)
// accumulate S (two buffers) and the whole of O (64 heads x 512 channels, 256
// columns a CTA) in tensor memory.  Each CTA brings half the tile's rows whole
// (its half of Q K^T's B operand) and all 64 rows' half of the latent channels
// (its half of the second product's B operand, read along the channels).
//
// Warps of a CTA: 0-3 softmax, 4-7 bring the keys (two warps take the even tiles,
// two the odd ones), 8-11 the values and the queries, 12 and 13 issue the products
// (in the pair's first CTA).  A rescale of O is rare: the running reference moves
// only when a maximum exceeds it by more than 2^8.
//
// Bound by the chain of a tile's steps (rows, scores, softmax, values; 26 clocks a
// 128 x 64 x 16 product of the pair): 64 requests x 2048 rows x 128 heads take 43 us, 0.59
// of a copy's rate in bytes and 0.45 of a product's in operations, on 64 of 76 pairs.  128
// heads a pair, since rows are the traffic: each row's latent half comes twice from L2,
// once from HBM.  8-bit rows are bound by their widening, which both CTAs do: 64 requests x
// 2048 x 128 heads take 67 us, 131072 rows x 128 heads 69, 55 of them 27 tiles in a row on
// each pair and the rest the join.
//
// Work split: the tiles of all units (a unit: request, position, 128 heads) form
// one line that is cut into equal pieces, one a pair; units cut in two leave
// their sums in the workspace and a second kernel joins them.
#include "hs_attend.h"

namespace hs_attn {
namespace {

constexpr int kThreads = 14 * 32;
// Tiles' time that a unit's queries, first scores and output take.  Without it pieces of several short
// units end last: contexts of 32768, 1, 20001 and 777 rows 43 -> 34 us, 24 ragged ones of up to 16,384
// rows 56 -> 35, 90 requests x 2048 rows x 128 heads 91 -> 86 (4: 35, 38, 87; 12: 34, 35, 83, but 8-bit
// rows of 24 ragged contexts 43 -> 45).
constexpr int kUnitCost = 7;
constexpr int kMaxPairs = 76;     // pairs of SMs

// Shared memory of a CTA.
constexpr int kQTmem = 6;                        // of Q's 9 blocks of 64 channels, those in tensor memory; the others here:
constexpr int kQBytes = (9 - kQTmem) * 64 * 128; // [64 heads][128 B] each
constexpr int kKStages = 3;
constexpr int kMeta = 8;
constexpr int kKBytes = 9 * 32 * 128;            // 9 blocks, [32 rows][128 B]
constexpr int kVBytes = 4 * 64 * 128;            // 4 blocks, [64 rows][128 B]
constexpr int kPBytes = 64 * 128;                // [64 heads][64 rows]
constexpr int kOffK = kQBytes;
constexpr int kOffV = kOffK + kKStages * kKBytes;  // (a piece's queries on their way to tensor memory pass here)
constexpr int kOffP = kOffV + 2 * kVBytes;
constexpr int kOffAux = kOffP + 2 * kPBytes;

struct Aux {
    uint64_t kfull[kKStages], kfree[kKStages], vfull[2], qhere, lifted, qfull, sfull[2], sread[2], pready[2], pvdone[2], spare[2];
    uint32_t tmem;
    int dead;
    Piece piece;
    // Per tile, kMeta deep: a tile's keys may arrive while the softmax four tiles back still reads these.
    uint16_t valid[kMeta][2][2];  // [half][warp]: one bit a row
    alignas(16) float scale[kMeta][kTile];
    __half log_scale[kMeta][kTile];  // only moves the reference: its rounding cancels
    int8_t q_up[2][64];          // power of two on a bf16 query held in fp16, by the parity of the piece
    float red[2][128];
};
constexpr int kSmem = kOffAux + (int)sizeof(Aux);
static_assert(kSmem <= 232448, "shared memory");

// Tensor memory columns.
constexpr uint32_t kColO = 0, kColS = 256, kColQ = 320;

// Workspace: an error word, where each pair's piece starts, and two partial results a pair.
struct Partial {
    float o[2][256][128];  // [CTA][column][lane]
    float ref[2][128], sum[2][128];
};
constexpr size_t kOffStart = 256;
constexpr size_t kOffPartial = kOffStart + sizeof(Start) * (kMaxPairs + 4);

// ---- the warps' parts ------------------------------------------------------------

// Keys: this CTA's 32 rows of each tile, whole.  Two warps take the even tiles and two
// the odd ones, 16 rows a warp; they also say which of the tile's 64 rows count.
template <typename T, bool E4M3>
__device__ void bring_keys(const Args& g, uint32_t sbase, Aux* x, uint32_t rank, int* error)
{
    const hs_attend_t& a = g.a;
    const int lane = threadIdx.x & 31, wg = (threadIdx.x >> 5) - 4;
    const int turn = wg >> 1, w = wg & 1;
    // lanes 0-15 look up the rows to bring, the others 16 of the other CTA's
    const int mine = (lane < 16 ? 32 * (int)rank : 32 * (1 - (int)rank)) + 16 * w + (lane & 15);
    long long j = 0;  // tiles so far
    Walk walk(g, x->piece);
    while (walk.next()) {
        const uint8_t* rows = static_cast<const uint8_t*>(a.rows) + walk.b * a.request_stride;
        const Lookup lookup(a, walk);
        int t = walk.t0;
        if ((j & 1) != turn) ++t;  // these warps' first tile of the piece
        // Rows of these warps' next three tiles, each looked up an iteration before it is used.  8-bit rows of
        // the third go to L2 ahead (3 to 6% faster; with 16-bit rows, 1 to 4% slower).
        int next = lookup.row(lookup.raw(t, mine)), after = lookup.row(lookup.raw(t + 2, mine));
        int ahead = lookup.raw(t + 4, mine);
        if constexpr (E4M3) prefetch_rows(rows, a.row_stride, after);
        for (; t < walk.t1; t += 2) {
            const long long jt = j + t - walk.t0;
            const int row = next;
            next = after;
            after = lookup.row(ahead);
            if constexpr (E4M3)
                if (t + 4 < walk.t1) prefetch_rows(rows, a.row_stride, after);
            ahead = lookup.raw(t + 6, mine);
            const int m = (int)(jt % kMeta), stage = (int)(jt % kKStages);
            const uint32_t reuse = (uint32_t)(jt / kKStages - 1) & 1;
            const uint32_t k_smem = sbase + kOffK + stage * kKBytes;
            const unsigned ok_bits = __ballot_sync(~0u, row >= 0);
            if constexpr (!E4M3) {
                if (jt >= kKStages) wait(tc::smem_addr(&x->kfree[stage]), reuse, &x->dead, error);
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const int tok = n * 4 + (lane >> 3), ch = lane & 7;  // 16-byte piece of a block
                    const int r = __shfl_sync(~0u, row, tok);
                    // absent rows are zeros (nothing is read; q is only an address that exists)
                    const uint8_t* src = (r < 0 ? static_cast<const uint8_t*>(a.q) : rows + r * a.row_stride) + ch * 16;
                    const uint32_t dst = k_smem + (16 * w + tok) * 128 + ((ch ^ (tok & 7)) << 4);
#pragma unroll
                    for (int c = 0; c < 9; ++c) tc::cp_async16(dst + c * 4096, src + c * 128, r >= 0);
                }
            } else {
                float sc = row >= 0 ? *reinterpret_cast<const float*>(rows + row * a.row_stride + HS_ROW8_SCALE) : 1.f;
                const int ch = lane & 3;  // 16 channels of a block
                uint4 v[2][9];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const int r = __shfl_sync(~0u, row, n * 8 + (lane >> 2));
#pragma unroll
                    for (int c = 0; c < 9; ++c)
                        v[n][c] = r >= 0 ? *reinterpret_cast<const uint4*>(rows + r * a.row_stride + c * 64 + ch * 16)
                                         : make_uint4(0, 0, 0, 0);
                }
                if (jt >= kKStages) wait(tc::smem_addr(&x->kfree[stage]), reuse, &x->dead, error);
                x->scale[m][mine] = sc;
                x->log_scale[m][mine] = __float2half(fmaxf(log2f(fabsf(sc)), kLeastLogScale));
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const int tok = n * 8 + (lane >> 2), r0 = tok & 7;
                    const uint32_t dst = k_smem + (16 * w + tok) * 128;
#pragma unroll
                    for (int c = 0; c < 9; ++c)
                        store_wide(v[n][c], dst + c * 4096, ((2 * ch) ^ r0) << 4, ((2 * ch + 1) ^ r0) << 4);
                }
            }
            if (lane == 0) {
                x->valid[m][rank][w] = (uint16_t)(ok_bits & 0xffff);
                x->valid[m][1 - rank][w] = (uint16_t)(ok_bits >> 16);
            }
            tc::cp_async_commit();
            tc::cp_async_wait<0>();
            tc::fence_async_shared();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_cluster(tc::map_to_rank(tc::smem_addr(&x->kfull[stage]), 0));
        }
        j += walk.t1 - walk.t0;
    }
}

// Values: the latent channels of this CTA's half, of a tile's 64 rows.  Two warps
// a stage, 32 rows each.  All four warps bring a piece's queries first.
template <typename T, bool E4M3>
__device__ void bring_values(const Args& g, uint32_t sbase, Aux* x, uint32_t rank, int* error)
{
    const hs_attend_t& a = g.a;
    const int lane = threadIdx.x & 31, wg = (threadIdx.x >> 5) - 8;
    const int stage = wg >> 1, w = wg & 1;
    const uint32_t full = tc::map_to_rank(tc::smem_addr(&x->vfull[stage]), 0);
    const uint32_t v_smem = sbase + kOffV + stage * kVBytes;
    const int mine = 32 * w + lane;
    const int block0 = 4 * (int)rank;  // the first of this CTA's blocks of 64 channels
    long long j = 0;
    Walk walk(g, x->piece);
    for (int pieces = 0; walk.next(); ++pieces) {
        const uint8_t* rows = static_cast<const uint8_t*>(a.rows) + walk.b * a.request_stride;
        const Lookup lookup(a, walk);
        int t = walk.t0;
        if ((j & 1) != stage) ++t;
        int next = lookup.raw(t, mine);
        // The last piece's products are done.  (A parity tells two phases apart, so the tile before the
        // last one is waited for first.)
        if (j >= 2) wait(tc::smem_addr(&x->pvdone[j & 1]), ((j - 2) >> 1) & 1, &x->dead, error);
        if (j >= 1) wait(tc::smem_addr(&x->pvdone[(j - 1) & 1]), ((j - 1) >> 1) & 1, &x->dead, error);
        const T* q = static_cast<const T*>(a.q) + walk.b * a.q_stride[0] + walk.p * a.q_stride[1];
#pragma unroll 1
        for (int n = 0; n < 4; ++n) {
            const int r = 16 * wg + n * 4 + (lane >> 3);
            const int head = walk.hb * 128 + (int)rank * 64 + r;
            const bool ok = head < a.heads;
            const uint8_t* src = reinterpret_cast<const uint8_t*>(q + (ok ? head : 0) * a.q_stride[2]) + (lane & 7) * 16;
            const uint32_t dst = r * 128 + (((lane & 7) ^ (r & 7)) << 4);
            auto block = [&](int c) { return dst + sbase + (c < kQTmem ? kOffV + c * 8192 : (c - kQTmem) * 8192); };
            if constexpr (E4M3 && HsType<T>::is_bf16) {
                uint4 v[9];
                float top = 0.f;
#pragma unroll
                for (int c = 0; c < 9; ++c) {
                    v[c] = ok ? *reinterpret_cast<const uint4*>(src + c * 128) : make_uint4(0, 0, 0, 0);
                    top = fmaxf(top, largest_bf16(v[c]));
                }
                for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
                const int up = power_up(top);
                if ((lane & 7) == 0) x->q_up[pieces & 1][r] = (int8_t)up;
#pragma unroll
                for (int c = 0; c < 9; ++c) {
                    const uint4 e = bf16_to_half(v[c], power_of_two(up));
                    tc::st_shared16(block(c), e.x, e.y, e.z, e.w);
                }
            } else {
#pragma unroll
                for (int c = 0; c < 9; ++c) tc::cp_async16(block(c), src + c * 128, ok);
            }
        }
        tc::cp_async_commit();
        tc::cp_async_wait<0>();
        tc::fence_async_shared();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tc::smem_addr(&x->qhere));
        wait(tc::smem_addr(&x->lifted), pieces & 1, &x->dead, error);
        for (; t < walk.t1; t += 2) {
            const long long jt = j + t - walk.t0;
            const int row = lookup.row(next);
            next = lookup.raw(t + 2, mine);
            if constexpr (!E4M3) {
                if (jt >= 2) wait(tc::smem_addr(&x->pvdone[stage]), ((jt - 2) >> 1) & 1, &x->dead, error);
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                    const int tok = n * 4 + (lane >> 3), ch = lane & 7;
                    const int r = __shfl_sync(~0u, row, tok);
                    const uint8_t* src = (r < 0 ? static_cast<const uint8_t*>(a.q) : rows + r * a.row_stride) + ch * 16 + block0 * 128;
                    const uint32_t dst = v_smem + (32 * w + tok) * 128 + ((ch ^ (tok & 7)) << 4);
#pragma unroll
                    for (int c = 0; c < 4; ++c) tc::cp_async16(dst + c * 8192, src + c * 128, r >= 0);
                }
            } else {
                const int ch = lane & 3;
                uint4 v[4][4];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const int r = __shfl_sync(~0u, row, n * 8 + (lane >> 2));
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        v[n][c] = r >= 0 ? *reinterpret_cast<const uint4*>(rows + r * a.row_stride + (block0 + c) * 64 + ch * 16)
                                         : make_uint4(0, 0, 0, 0);
                }
                if (jt >= 2) wait(tc::smem_addr(&x->pvdone[stage]), ((jt - 2) >> 1) & 1, &x->dead, error);
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const int tok = n * 8 + (lane >> 2), r0 = tok & 7;
                    const uint32_t dst = v_smem + (32 * w + tok) * 128;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        store_wide(v[n][c], dst + c * 8192, ((2 * ch) ^ r0) << 4, ((2 * ch + 1) ^ r0) << 4);
                }
            }
            tc::cp_async_commit();
            tc::cp_async_wait<0>();
            tc::fence_async_shared();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_cluster(full);
        }
        j += walk.t1 - walk.t0;
    }
}

// Q K^T of one tile into buffer S, and P V into O (the warp's elected lane).
template <typename T, int S>
__device__ __forceinline__ void issue_qk(uint32_t sbase, uint32_t tmem, uint64_t k_desc, uint64_t& kfree, Aux* x)
{
    constexpr uint32_t id = tc::inst_desc(HsType<T>::is_bf16, 128, kTile, false, false);
    const uint64_t q_desc = tc::smem_desc(sbase, 16, 1024);
    if (tc::elect_one()) {
#pragma unroll
        for (int c = 0; c < kQTmem; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                tc::mma_ts<2>(tmem + kColS + 32 * S, tmem + kColQ + 32 * c + 8 * k, k_desc + ((c * 4096 + k * 32) >> 4), id,
                              (c | k) != 0);
#pragma unroll
        for (int c = kQTmem; c < 9; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                tc::mma_ss<2>(tmem + kColS + 32 * S, q_desc + (((c - kQTmem) * 8192 + k * 32) >> 4),
                              k_desc + ((c * 4096 + k * 32) >> 4), id, true);
        tc::commit<2>(tc::smem_addr(&x->sfull[S]));
        tc::commit<2>(tc::smem_addr(&kfree));
    }
    __syncwarp();
}
template <typename T, int S> __device__ __forceinline__ void issue_pv(uint32_t sbase, uint32_t tmem, Aux* x, bool first)
{
    constexpr uint32_t id = tc::inst_desc(HsType<T>::is_bf16, 128, 256, false, true);
    const uint64_t p_desc = tc::smem_desc(sbase + kOffP + S * kPBytes, 16, 1024);
    const uint64_t v_desc = tc::smem_desc(sbase + kOffV + S * kVBytes, 8192, 1024);
    if (tc::elect_one()) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                tc::mma_ss<2>(tmem + kColO + 128 * h, p_desc + ((k * 32) >> 4), v_desc + ((h * 16384 + k * 2048) >> 4), id,
                              !(first && k == 0));
        tc::commit<2>(tc::smem_addr(&x->pvdone[S]));
    }
    __syncwarp();
}

// After a wait that gave up: what was issued must be complete before tensor memory is freed.
__device__ void drain(Aux* x, int which)
{
    if (!*(volatile int*)&x->dead) return;
    if (tc::elect_one()) tc::commit<2>(tc::smem_addr(&x->spare[which]));
    __syncwarp();
    tc::mbar_wait(tc::smem_addr(&x->spare[which]), 0);
}

// The products are issued by two warps of the pair's first CTA, one for Q K^T and
// one for P V: a warp does not get past products it has issued until they have
// nearly run, and would bring the other product late.
template <typename T> __device__ void multiply_qk(const Args& g, uint32_t sbase, Aux* x, int* error)
{
    const uint32_t tmem = __shfl_sync(~0u, x->tmem, 0);
    const uint64_t k_base = tc::smem_desc(sbase + kOffK, 16, 1024);
    long long j = 0;
    int pieces = 0, stage = 0;
    uint32_t phase = 0;
    Walk walk(g, x->piece);
    while (walk.next()) {
        wait(tc::smem_addr(&x->qfull), pieces++ & 1, &x->dead, error);
        for (int t = walk.t0; t < walk.t1; ++t, ++j) {
            const int s = (int)(j & 1);
            // S's buffer has been read
            if (j >= 2) wait(tc::smem_addr(&x->sread[s]), ((j - 2) >> 1) & 1, &x->dead, error);
            wait(tc::smem_addr(&x->kfull[stage]), phase, &x->dead, error);
            __syncwarp();
            tc::fence_after();
            const uint64_t k_desc = k_base + stage * (kKBytes >> 4);
            if (s)
                issue_qk<T, 1>(sbase, tmem, k_desc, x->kfree[stage], x);
            else
                issue_qk<T, 0>(sbase, tmem, k_desc, x->kfree[stage], x);
            if (++stage == kKStages) stage = 0, phase ^= 1;
        }
    }
    drain(x, 0);
}
template <typename T> __device__ void multiply_pv(const Args& g, uint32_t sbase, Aux* x, int* error)
{
    const uint32_t tmem = __shfl_sync(~0u, x->tmem, 0);
    long long j = 0;
    Walk walk(g, x->piece);
    while (walk.next()) {
        for (int t = walk.t0; t < walk.t1; ++t, ++j) {
            const int s = (int)(j & 1);
            wait(tc::smem_addr(&x->vfull[s]), (j >> 1) & 1, &x->dead, error);
            wait(tc::smem_addr(&x->pready[s]), (j >> 1) & 1, &x->dead, error);
            __syncwarp();
            tc::fence_after();
            if (s)
                issue_pv<T, 1>(sbase, tmem, x, t == walk.t0);
            else
                issue_pv<T, 0>(sbase, tmem, x, t == walk.t0);
        }
    }
    drain(x, 1);
}

// Copy 6 of Q's 9 blocks of channels to tensor memory: products that read A there leave
// shared memory, whose bandwidth bounds a tile, to the others.  A pair's product of
// 128 rows computes half of its columns in lanes 64-127, which read their own copy of A.
__device__ __forceinline__ void lift_queries(uint32_t sbase, uint32_t tmem, uint32_t qfull, uint32_t lifted)
{
    const int row = threadIdx.x & 63;
#pragma unroll
    for (int c = 0; c < kQTmem; ++c) {
        uint32_t r[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint4 v = tc::ld_shared16(sbase + kOffV + c * 8192 + row * 128 + ((i ^ (row & 7)) << 4));
            r[4 * i] = v.x, r[4 * i + 1] = v.y, r[4 * i + 2] = v.z, r[4 * i + 3] = v.w;
        }
        tc::tmem_st32(tmem + kColQ + 32 * c, r);
    }
    tc::tmem_wait_st();
    tc::fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
        tc::mbar_arrive_cluster(qfull);
        tc::mbar_arrive(lifted);
    }
}

// Softmax of 64 heads: thread (head, half) takes 32 of a tile's 64 rows.
template <typename T, bool E4M3>
__device__ void soften(const Args& g, uint32_t sbase, Aux* x, uint32_t rank, int pair, uint8_t* ws, int* error)
{
    const hs_attend_t& a = g.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = threadIdx.x & 63, half = threadIdx.x >> 6;
    const uint32_t tmem = x->tmem + ((uint32_t)warp << 21);  // this warp's 32 lanes
    float c = a.scale * 1.4426950408889634f;
    long long j = 0;
    Walk walk(g, x->piece);
    const uint32_t sread[2] = {tc::map_to_rank(tc::smem_addr(&x->sread[0]), 0),
                               tc::map_to_rank(tc::smem_addr(&x->sread[1]), 0)};
    const uint32_t pready[2] = {tc::map_to_rank(tc::smem_addr(&x->pready[0]), 0),
                                tc::map_to_rank(tc::smem_addr(&x->pready[1]), 0)};
    const uint32_t qfull = tc::map_to_rank(tc::smem_addr(&x->qfull), 0);
    for (int pieces = 0; walk.next(); ++pieces) {
        wait(tc::smem_addr(&x->qhere), pieces & 1, &x->dead, error);
        lift_queries(sbase, tmem, qfull, tc::smem_addr(&x->lifted));
        float ref = 0.f, sum = 0.f;
        bool seen = false;  // a row that counts has been met: ref is a maximum
        for (int t = walk.t0; t < walk.t1; ++t, ++j) {
            const int s = j & 1;
            wait(tc::smem_addr(&x->sfull[s]), (j >> 1) & 1, &x->dead, error);
            tc::fence_after();
            uint32_t r[32];
            tc::tmem_ld32(tmem + kColS + 32 * s, r);
            tc::tmem_wait_ld(r);
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_cluster(sread[s]);  // the tile after next may come
            if constexpr (E4M3 && HsType<T>::is_bf16)
                if (t == walk.t0)
                    c = power_of_two(-x->q_up[pieces & 1][row]) * (a.scale * 1.4426950408889634f);
            const uint32_t valid = reinterpret_cast<const uint32_t*>(x->valid[j % kMeta])[half];
            const float* wt = x->scale[j % kMeta] + 32 * half;
            const __half* lw = x->log_scale[j % kMeta] + 32 * half;
            float v[32], top = -INFINITY;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                v[i] = __uint_as_float(r[i]) * c;
                if constexpr (E4M3) v[i] *= wt[i];
            }
            if (valid != ~0u)
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (!(valid >> i & 1)) v[i] = -INFINITY;
#pragma unroll
            for (int i = 0; i < 32; ++i) top = fmaxf(top, E4M3 ? v[i] + __half2float(lw[i]) : v[i]);
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
            // the buffer of P is free once the product two tiles ago is done
            if (j >= 2) wait(tc::smem_addr(&x->pvdone[s]), ((j - 2) >> 1) & 1, &x->dead, error);
            if (__any_sync(~0u, scale_o)) {
                if (!scale_o) keep = 1.f;
                wait(tc::smem_addr(&x->pvdone[1 - s]), ((j - 1) >> 1) & 1, &x->dead, error);
                tc::fence_after();
#pragma unroll 1
                for (int n = 0; n < 256; n += 32) {
                    tc::tmem_ld32(tmem + kColO + n, r);
                    tc::tmem_wait_ld(r);
#pragma unroll
                    for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * keep);
                    tc::tmem_st32(tmem + kColO + n, r);
                }
                tc::tmem_wait_st();
            }
            const uint32_t dst = sbase + kOffP + s * kPBytes + row * 128;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                uint32_t e[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k = n * 8 + 2 * i;
                    float p0 = tc::exp2_approx(v[k] - ref), p1 = tc::exp2_approx(v[k + 1] - ref);
                    sum += p0 + p1;
                    if constexpr (E4M3) {
                        p0 *= wt[k];
                        p1 *= wt[k + 1];
                    }
                    e[i] = pack2<std::conditional_t<E4M3, __half, T>>(p0, p1);
                }
                tc::st_shared16(dst + (((half * 4 + n) ^ (row & 7)) << 4), e[0], e[1], e[2], e[3]);
            }
            tc::fence_async_shared();
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_cluster(pready[s]);
        }
        // The piece's end: O and the sums leave.
        asm volatile("bar.sync 1, 128;" ::: "memory");
        x->red[0][threadIdx.x] = sum;
        asm volatile("bar.sync 1, 128;" ::: "memory");
        sum += x->red[0][threadIdx.x ^ 64];
        asm volatile("bar.sync 1, 128;" ::: "memory");
        wait(tc::smem_addr(&x->pvdone[(j - 1) & 1]), ((j - 1) >> 1) & 1, &x->dead, error);
        tc::fence_after();
        const int head = walk.hb * 128 + (int)rank * 64 + row;
        const bool whole = walk.t0 == 0 && walk.t1 == walk.tiles;
        Partial* part = reinterpret_cast<Partial*>(ws + kOffPartial) + 2 * pair + (walk.t0 == 0 ? 1 : 0);
        const bool some = sum > 0.f || sum != sum;
        const float inv = some ? 1.f / sum : 0.f;
        if (whole) {
            // Through the buffers of P, so that eight lanes write 128 bytes of a head together: 64 channels
            // of each half at a time, [half][head][128 B].
            T* out = static_cast<T*>(a.out) + walk.b * a.out_stride[0] + walk.p * a.out_stride[1];
            const uint32_t mine = sbase + kOffP + threadIdx.x * 128;
#pragma unroll 1
            for (int n = 0; n < 256; n += 64) {
                uint32_t r[32];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    __syncwarp();
                    tc::tmem_ld32(tmem + kColO + n + 32 * q, r);
                    tc::tmem_wait_ld(r);
                    auto f = [&](int k) { return some ? __uint_as_float(r[k]) * inv : 0.f; };
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        tc::st_shared16(mine + (((4 * q + i) ^ (row & 7)) << 4), pack2<T>(f(8 * i), f(8 * i + 1)),
                                        pack2<T>(f(8 * i + 2), f(8 * i + 3)), pack2<T>(f(8 * i + 4), f(8 * i + 5)),
                                        pack2<T>(f(8 * i + 6), f(8 * i + 7)));
                }
                asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int at = 16 * i + (threadIdx.x >> 3), ch = threadIdx.x & 7;  // of 128 rows of the buffer
                    const int h = walk.hb * 128 + (int)rank * 64 + (at & 63);
                    const uint4 v = tc::ld_shared16(sbase + kOffP + at * 128 + ((ch ^ (at & 7)) << 4));
                    if (h < a.heads)
                        *reinterpret_cast<uint4*>(out + (int64_t)h * a.out_stride[2] + 256 * (at >> 6) + n + 8 * ch) = v;
                }
                asm volatile("bar.sync 1, 128;" ::: "memory");
            }
        } else {
#pragma unroll 1
            for (int n = 0; n < 256; n += 32) {
                uint32_t r[32];
                __syncwarp();
                tc::tmem_ld32(tmem + kColO + n, r);
                tc::tmem_wait_ld(r);
                if (head < a.heads)
#pragma unroll
                    for (int i = 0; i < 32; ++i) part->o[rank][n + i][threadIdx.x] = __uint_as_float(r[i]);
            }
        }
        if (head < a.heads) {
            if (!whole) {
                part->ref[rank][threadIdx.x] = ref;
                part->sum[rank][threadIdx.x] = sum;
            } else if (a.lse && half == 0) {
                a.lse[(walk.b * a.positions + walk.p) * a.heads + head] =
                    some ? (ref + log2f(sum)) * 0.6931471805599453f : -INFINITY;
            }
        }
        tc::fence_before();
    }
}

template <typename T, bool E4M3>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) hs_attend_kernel(const __grid_constant__ Args g)
{
    using Operand = std::conditional_t<E4M3, __half, T>;
    extern __shared__ __align__(1024) uint8_t base[];  // the swizzled tiles need 1024
    const uint32_t sbase = tc::smem_addr(base);
    Aux* x = reinterpret_cast<Aux*>(base + kOffAux);
    const hs_attend_t& a = g.a;
    const uint32_t rank = tc::cluster_rank();
    const int pair = blockIdx.x >> 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    int* error = reinterpret_cast<int*>(ws);

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join may queue up behind this grid
    if (warp == 0) tc::tmem_alloc<2>(tc::smem_addr(&x->tmem), 512);
    if (warp == 12) {
        const Piece p = find_piece(g, pair);
        if (lane == 0) {
            x->piece = p;
            x->dead = 0;
            if (rank == 0) reinterpret_cast<Start*>(ws + kOffStart)[pair] = {p.count > 0 ? p.unit : -1, p.tile};
            for (int i = 0; i < 2; ++i) {
                tc::mbar_init(tc::smem_addr(&x->vfull[i]), 4);
                tc::mbar_init(tc::smem_addr(&x->sfull[i]), 1);
                tc::mbar_init(tc::smem_addr(&x->sread[i]), 8);
                tc::mbar_init(tc::smem_addr(&x->pready[i]), 8);
                tc::mbar_init(tc::smem_addr(&x->pvdone[i]), 1);
                tc::mbar_init(tc::smem_addr(&x->spare[i]), 1);
            }
            for (int i = 0; i < kKStages; ++i) {
                tc::mbar_init(tc::smem_addr(&x->kfull[i]), 4);
                tc::mbar_init(tc::smem_addr(&x->kfree[i]), 1);
            }
            tc::mbar_init(tc::smem_addr(&x->qhere), 4);
            tc::mbar_init(tc::smem_addr(&x->lifted), 4);
            tc::mbar_init(tc::smem_addr(&x->qfull), 8);
            tc::mbar_init_fence();
        }
    }
    tc::fence_before();
    __syncwarp();
    __syncthreads();
    tc::cluster_sync();
    tc::fence_after();

    if (x->piece.count > 0) {
        if (warp < 4)
            soften<T, E4M3>(g, sbase, x, rank, pair, ws, error);
        else if (warp < 8)
            bring_keys<T, E4M3>(g, sbase, x, rank, error);
        else if (warp < 12)
            bring_values<T, E4M3>(g, sbase, x, rank, error);
        else if (rank == 0 && warp == 12)
            multiply_qk<Operand>(g, sbase, x, error);
        else if (rank == 0)
            multiply_pv<Operand>(g, sbase, x, error);
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    tc::cluster_sync_relaxed();  // no CTA leaves while the other may signal it
    tc::fence_after();
    if (warp == 0) tc::tmem_free<2>(x->tmem, 512);
}

// Join the pieces of the units that several pairs worked on: block x takes the
// x-th such unit (found at the first start of a piece inside it), one CTA's half
// of its heads.  Four groups of 128 threads, one a lane: with SPLIT they take every
// fourth piece of COLS columns, else every piece of COLS columns each; in one pass,
// and the order of the sums is fixed.
template <typename T, int COLS, bool SPLIT>
__global__ void __launch_bounds__(512) hs_attend_join_kernel(const __grid_constant__ Args g, int pairs)
{
    constexpr int kGroups = SPLIT ? 4 : 1;  // that share pieces
    __shared__ float tops[4][128], sums[4][128], cols[SPLIT ? 3 : 1][COLS][128];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const hs_attend_t& a = g.a;
    const uint8_t* ws = static_cast<const uint8_t*>(a.workspace);
    const Partial* parts = reinterpret_cast<const Partial*>(ws + kOffPartial);
    int unit, first, last;
    if (!find_cut(reinterpret_cast<const Start*>(ws + kOffStart), pairs, blockIdx.x, unit, first, last)) return;
    const int t = threadIdx.x;
    const int rank = blockIdx.y, c0 = SPLIT ? COLS * blockIdx.z : COLS * (4 * blockIdx.z + (t >> 7));
    const int lane = t & 127, group = SPLIT ? t >> 7 : 0, row = lane & 63, half = lane >> 6;
    const int pos = unit / g.head_blocks, hb = unit - pos * g.head_blocks;
    const long long b = pos / a.positions;
    const int p = pos - (int)b * a.positions;
    const int head = hb * 128 + rank * 64 + row;
    if (hb * 128 + rank * 64 >= a.heads) return;
    const bool live = head < a.heads;
    float acc[COLS] = {}, sum = 0.f, top = -INFINITY;
    if (live)
#pragma unroll(COLS == 4 ? 8 : 2)
        for (int n = first + group; n <= last; n += kGroups) {
            const Partial& q = parts[2 * n + (n == first)];
            const float ref = q.ref[rank][lane], l = q.sum[rank][lane];
            float o[COLS];
#pragma unroll
            for (int k = 0; k < COLS; ++k) o[k] = q.o[rank][c0 + k][lane];
            // without a branch, so that the loads of several pieces are in flight; a sum of 0: no row counted
            const float up = l == 0.f ? top : fmaxf(top, ref), base = up == -INFINITY ? 0.f : up;
            const float keep = tc::exp2_approx(top - base), w = l == 0.f ? 0.f : tc::exp2_approx(ref - base);
            top = up;
            sum = sum * keep + w * l;
#pragma unroll
            for (int k = 0; k < COLS; ++k) acc[k] = acc[k] * keep + (l == 0.f ? 0.f : w * o[k]);
        }
    if (SPLIT) {
        tops[group][lane] = top;
        sums[group][lane] = sum;
        if (group)
#pragma unroll
            for (int k = 0; k < COLS; ++k) cols[group - 1][k][lane] = acc[k];
        __syncthreads();
    }
    if (group || !live) return;
    if (SPLIT) {
        top = fmaxf(fmaxf(tops[0][lane], tops[1][lane]), fmaxf(tops[2][lane], tops[3][lane]));
        const float base = top == -INFINITY ? 0.f : top;
        float w = tc::exp2_approx(tops[0][lane] - base);
        sum *= w;
#pragma unroll
        for (int k = 0; k < COLS; ++k) acc[k] *= w;
        for (int n = 1; n < 4; ++n) {
            w = tc::exp2_approx(tops[n][lane] - base);
            sum += w * sums[n][lane];
#pragma unroll
            for (int k = 0; k < COLS; ++k) acc[k] += w * cols[n - 1][k][lane];
        }
    }
    const bool some = sum > 0.f || sum != sum;
    const float inv = some ? 1.f / sum : 0.f;
    T* out = static_cast<T*>(a.out) + b * a.out_stride[0] + p * a.out_stride[1] + (int64_t)head * a.out_stride[2] +
             256 * half + c0;
#pragma unroll
    for (int k = 0; k < COLS; k += 4)
        *reinterpret_cast<uint2*>(out + k) =
            make_uint2(pack2<T>(acc[k] * inv, acc[k + 1] * inv), pack2<T>(acc[k + 2] * inv, acc[k + 3] * inv));
    if (a.lse && half == 0 && c0 == 0)
        a.lse[(b * a.positions + p) * a.heads + head] = some ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

template <typename T, bool E4M3> cudaError_t launch(const Args& g, cudaStream_t s)
{
    cudaError_t e = cudaFuncSetAttribute(hs_attend_kernel<T, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    hs_attend_kernel<T, E4M3><<<2 * g.workers, kThreads, kSmem, s>>>(g);
    e = cudaGetLastError();
    if (e != cudaSuccess || !g.flat || g.workers <= 1) return e;
    // At most `cut` units are cut.  A block's time is latency, so many units, of few pieces each, take few
    // blocks: requests of 2048 listed rows x 128 heads 75 against 86 us with 90 of them, 38 against 43 with
    // 32, 30 against 32 with 16 (64 heads: 36 and 36 with 32, 28 against 26 with 16).  Of contexts one may
    // hold most pieces, so they split them (24 ragged ones 45 against 49).  Few units take narrower columns:
    // 4 ragged contexts (128 heads) 31 against 38, 8 of them 29 against 37 (8 equal ones 37 against 33); but
    // 8 requests of 2048 listed rows 27 against 23, hence their lower limit.
    const int cut = g.units < g.workers - 1 ? g.units : g.workers - 1, halves = g.a.heads > 64 ? 2 : 1;
    if (g.a.slots && cut * halves >= 32)
        return launch_after(hs_attend_join_kernel<T, 16, false>, dim3(cut, halves, 256 / 64), 512, 0, s, g, g.workers);
    if (cut * halves <= (g.a.slots ? 8 : 16))
        return launch_after(hs_attend_join_kernel<T, 4, true>, dim3(cut, halves, 256 / 4), 512, 0, s, g, g.workers);
    return launch_after(hs_attend_join_kernel<T, 16, true>, dim3(cut, halves, 256 / 16), 512, 0, s, g, g.workers);
}

}  // namespace

size_t pair_workspace(int64_t units, int64_t tiles)
{
    return kOffPartial + sizeof(Partial) * 2 * (size_t)(units * tiles < kMaxPairs ? units * tiles : kMaxPairs);
}

cudaError_t launch_pair(const hs_attend_t& a, int sms, cudaStream_t s)
{
    Args g;
    g.a = a;
    g.head_blocks = (a.heads + 127) / 128;
    g.units = a.batch * a.positions * g.head_blocks;
    // Pieces also write and join up to two partial results a pair: about 10 us, 10 tiles' time.
    g.cut(sms / 2 < kMaxPairs ? (sms > 1 ? sms / 2 : 1) : kMaxPairs, a.slots ? a.entries : a.n_rows, 10, kUnitCost);
    const bool e4m3 = a.row_format == HS_ROWS_E4M3;
    if (a.dtype == HS_TYPE_BF16)
        return e4m3 ? launch<__nv_bfloat16, true>(g, s) : launch<__nv_bfloat16, false>(g, s);
    return e4m3 ? launch<__half, true>(g, s) : launch<__half, false>(g, s);
}

}  // namespace hs_attn

size_t hs_attend_workspace_bytes(int batch, int positions, int heads, int64_t rows)
{
    const int64_t tiles = rows <= hs_attn::kTile ? 1 : (rows + hs_attn::kTile - 1) / hs_attn::kTile;
    const int64_t units = (int64_t)batch * positions;
    const size_t pair = hs_attn::pair_workspace(units * ((heads + 127) / 128), tiles);
    if (heads > hs_attn::kNarrowHeads) return pair;
    const size_t narrow = hs_attn::narrow_workspace(units, tiles, heads);  // either, by the rows' form
    return narrow > pair ? narrow : pair;
}

cudaError_t hs_launch_attend(const hs_attend_t& a, cudaStream_t s)
{
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    return a.row_format == HS_ROWS_E4M3 && a.heads <= hs_attn::kNarrowHeads ? hs_attn::launch_narrow(a, sms, s)
                                                                            : hs_attn::launch_pair(a, sms, s);
}
