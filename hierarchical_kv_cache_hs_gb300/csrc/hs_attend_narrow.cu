// hs_latent_attend over 8-bit rows for up to 32 heads: one SM takes all heads of a request
// and position.
//
// The products are turned around, so that rows and channels, not heads, fill the tensor
// core's 128 (or 64) rows: S^T = K Q^T for a tile of 64 rows (M = 64, N = heads), and
// O^T += V^T P^T (M = 128 channels four times, N = heads), where V^T is the key tile read
// along its channels.  A row is widened to fp16 and brought to shared memory once, and
// read twice.  Bound by the chain of a stage (rows, widening, scores, softmax, values) with
// two stages of widened rows; a third (72 KB) does not fit, one of rows as they come (36 KB)
// would with 16 heads and was not tried.  256 requests x 2048 rows x 16 heads take 102 us,
// 3.2 TB/s (0.47 of a copy's rate), 93 of them here and the rest the join; 32 heads 128.
//
// Warps: 0-3 softmax, 4-11 bring the rows (four a stage) and the queries, 12 and 13 issue
// the products.  The running reference of a head moves only when a maximum exceeds it by
// more than 2^8.  Work is cut as in the kernel for more heads.
#include "hs_attend.h"

namespace hs_attn {
namespace {

constexpr int kThreads = 14 * 32;
// Tiles' time that a unit's queries, first scores and output take: 24 ragged contexts of up to 16,384
// rows 47 -> 35 us, 200 requests x 1000 rows x 32 heads 76 -> 72, 256 x 2048 x 16 102 (7: 34, 73, 105).
constexpr int kUnitCost = 3;
constexpr int kMaxCtas = 152;
constexpr int kStageBytes = 9 * 64 * 128;  // 9 blocks of 64 channels, [64 rows][128 B]
constexpr int kBlock = 64 * 128;

// NH: heads, padded to the products' N.
template <int NH> struct Layout {
    static constexpr int off_q = 2 * kStageBytes;              // 9 blocks, [NH][128 B]
    static constexpr int off_p = off_q + 9 * NH * 128;         // two buffers, [NH][128 B] each
    static constexpr int off_aux = off_p + 2 * NH * 128;
    // Tensor memory: sums of the four groups of 128 channels, then two buffers of scores.
    static constexpr uint32_t col_s = 4 * NH;
    static constexpr uint32_t cols = NH == 32 ? 256 : 128;
};

template <int NH> struct Aux {
    uint64_t full[2], qfull, qfree, sfull[2], pready[2], pvdone[2], spare[2];
    uint32_t tmem;
    int dead;
    Piece piece;
    uint16_t valid[4][4];          // by tile, four deep; one bit a row
    alignas(8) float scale[4][kTile];
    // Power of two on a bf16 query held in fp16, by the piece, three deep: piece n + 3's is written once the
    // products with keys of piece n + 2 are done.  The last of those waits for the softmax's arrival two tiles
    // earlier, which follows its read of piece n's power even where a piece has one tile (two deep, it need not).
    int8_t q_up[3][NH];
    float top[2][4][NH];           // maxima by warp, by the parity of the tile
    float red[4][NH];              // by warp: sums, and factors on O
    float inv[NH];                 // of the sums at a piece's end
};
template <int NH> constexpr int smem_bytes() { return Layout<NH>::off_aux + (int)sizeof(Aux<NH>); }
static_assert(smem_bytes<32>() <= 232448, "shared memory");

template <int NH> struct Partial {
    float o[4][NH][128];  // [channels / 128][head][channel]
    float ref[NH], sum[NH];
};
constexpr size_t kOffStart = 256;
constexpr size_t kOffPartial = kOffStart + sizeof(Start) * kMaxCtas;

// Rows of a tile, four warps of 16 rows each; and the queries, eight warps a head at a time.
template <typename T, int NH> __device__ void bring(const Args& g, uint32_t sbase, Aux<NH>* x, int* error)
{
    const hs_attend_t& a = g.a;
    const int lane = threadIdx.x & 31, wg = (threadIdx.x >> 5) - 4;
    const int stage = wg >> 2, w = wg & 3;
    const uint32_t k_smem = sbase + stage * kStageBytes, full = tc::smem_addr(&x->full[stage]);
    const int mine = 16 * w + (lane & 15);
    long long j = 0;
    Walk walk(g, x->piece);
    for (int pieces = 0; walk.next(); ++pieces) {
        const uint8_t* rows = static_cast<const uint8_t*>(a.rows) + walk.b * a.request_stride;
        const Lookup lookup(a, walk);
        int t = walk.t0;
        if ((j & 1) != stage) ++t;  // this stage's first tile of the piece
        int next = lookup.raw(t, mine);  // looked at an iteration later
        // Q, once the last piece's products with keys are done.
        if (pieces) wait(tc::smem_addr(&x->qfree), (pieces - 1) & 1, &x->dead, error);
        const T* q = static_cast<const T*>(a.q) + walk.b * a.q_stride[0] + walk.p * a.q_stride[1];
        for (int h = wg; h < NH; h += 8) {
            const bool ok = h < a.heads;
            const uint4* src = reinterpret_cast<const uint4*>(q + (ok ? h : 0) * a.q_stride[2]);
            const uint32_t dst = sbase + Layout<NH>::off_q + h * 128;
            uint4 v[3];
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                const int c = 32 * i + lane;  // of 72 pieces
                v[i] = ok && c < 72 ? src[c] : make_uint4(0, 0, 0, 0);
                if constexpr (HsType<T>::is_bf16) top = fmaxf(top, largest_bf16(v[i]));
            }
            if constexpr (HsType<T>::is_bf16) {
                for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
                const int up = power_up(top);
                if (lane == 0) x->q_up[pieces % 3][h] = (int8_t)up;
#pragma unroll
                for (int i = 0; i < 3; ++i) v[i] = bf16_to_half(v[i], power_of_two(up));
            }
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                const int c = 32 * i + lane;
                if (c < 72) tc::st_shared16(dst + (c >> 3) * NH * 128 + (((c & 7) ^ (h & 7)) << 4), v[i].x, v[i].y, v[i].z, v[i].w);
            }
        }
        tc::fence_async_shared();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tc::smem_addr(&x->qfull));
        for (; t < walk.t1; t += 2) {
            const long long jt = j + t - walk.t0;
            const int row = lookup.row(next);
            next = lookup.raw(t + 2, mine);
            const int m = (int)(jt & 3);
            const unsigned ok_bits = __ballot_sync(~0u, row >= 0);
            const float sc = row >= 0 ? *reinterpret_cast<const float*>(rows + row * a.row_stride + HS_ROW8_SCALE) : 1.f;
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
            if (jt >= 2) wait(tc::smem_addr(&x->pvdone[stage]), ((jt - 2) >> 1) & 1, &x->dead, error);
            if (lane < 16) x->scale[m][mine] = sc;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int tok = n * 8 + (lane >> 2), r0 = tok & 7;
                const uint32_t dst = k_smem + (16 * w + tok) * 128;
#pragma unroll
                for (int c = 0; c < 9; ++c)
                    store_wide(v[n][c], dst + c * kBlock, ((2 * ch) ^ r0) << 4, ((2 * ch + 1) ^ r0) << 4);
            }
            if (lane == 0) x->valid[m][w] = (uint16_t)ok_bits;
            tc::fence_async_shared();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(full);
        }
        j += walk.t1 - walk.t0;
    }
}

template <int NH> __device__ void drain(Aux<NH>* x, int which)
{
    if (!*(volatile int*)&x->dead) return;  // after a wait that gave up: what was issued must be complete
    if (tc::elect_one()) tc::commit<1>(tc::smem_addr(&x->spare[which]));
    __syncwarp();
    tc::mbar_wait(tc::smem_addr(&x->spare[which]), 0);
}

// S^T = K Q^T, issued by one warp.
template <int NH> __device__ void multiply_qk(const Args& g, uint32_t sbase, Aux<NH>* x, int* error)
{
    constexpr uint32_t id = tc::inst_desc(false, 64, NH, false, false);
    const uint32_t tmem = __shfl_sync(~0u, x->tmem, 0) + Layout<NH>::col_s;
    const uint64_t k_base = tc::smem_desc(sbase, 16, 1024), q_desc = tc::smem_desc(sbase + Layout<NH>::off_q, 16, 1024);
    long long j = 0;
    int pieces = 0;
    Walk walk(g, x->piece);
    while (walk.next()) {
        wait(tc::smem_addr(&x->qfull), pieces++ & 1, &x->dead, error);
        for (int t = walk.t0; t < walk.t1; ++t, ++j) {
            const int s = (int)(j & 1);
            // S's buffer has been read
            if (j >= 2) wait(tc::smem_addr(&x->pready[s]), ((j - 2) >> 1) & 1, &x->dead, error);
            wait(tc::smem_addr(&x->full[s]), (j >> 1) & 1, &x->dead, error);
            __syncwarp();
            tc::fence_after();
            const uint64_t k_desc = k_base + s * (kStageBytes >> 4);
            if (tc::elect_one()) {
#pragma unroll
                for (int c = 0; c < 9; ++c)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc::mma_ss<1>(tmem + NH * s, k_desc + ((c * kBlock + k * 32) >> 4), q_desc + ((c * NH * 128 + k * 32) >> 4), id,
                                      (c | k) != 0);
                tc::commit<1>(tc::smem_addr(&x->sfull[s]));
                if (t + 1 == walk.t1) tc::commit<1>(tc::smem_addr(&x->qfree));
            }
            __syncwarp();
        }
    }
    drain(x, 0);
}

// O^T += V^T P^T, issued by another.
template <int NH> __device__ void multiply_pv(const Args& g, uint32_t sbase, Aux<NH>* x, int* error)
{
    constexpr uint32_t id = tc::inst_desc(false, 128, NH, true, false);
    const uint32_t tmem = __shfl_sync(~0u, x->tmem, 0);
    const uint64_t v_base = tc::smem_desc(sbase, kBlock, 1024), p_base = tc::smem_desc(sbase + Layout<NH>::off_p, 16, 1024);
    long long j = 0;
    Walk walk(g, x->piece);
    while (walk.next()) {
        for (int t = walk.t0; t < walk.t1; ++t, ++j) {
            const int s = (int)(j & 1);
            wait(tc::smem_addr(&x->pready[s]), (j >> 1) & 1, &x->dead, error);
            __syncwarp();
            tc::fence_after();
            const uint64_t v_desc = v_base + s * (kStageBytes >> 4);
            const uint64_t p_desc = p_base + s * (NH * 128 >> 4);
            const bool first = t == walk.t0;
            if (tc::elect_one()) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc::mma_ss<1>(tmem + NH * i, v_desc + ((2 * i * kBlock + k * 2048) >> 4), p_desc + ((k * 32) >> 4), id,
                                      !(first && k == 0));
                tc::commit<1>(tc::smem_addr(&x->pvdone[s]));
            }
            __syncwarp();
        }
    }
    drain(x, 1);
}

// NH columns of scores of this warp's 16 rows: thread (r, c) = (lane / 4, lane % 4) gets rows r and r + 8 of
// columns 8 g + 2 c and 8 g + 2 c + 1, as v[4 g + 2 (row half) + column parity].
template <int NH> __device__ __forceinline__ void load_scores(uint32_t addr, uint32_t (&v)[NH / 2])
{
    if constexpr (NH == 16)
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                     : "r"(addr));
    else
        asm volatile(
            "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
            "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
            : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
              "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
            : "r"(addr));
    // the registers pass through the wait, so that nothing reads them before
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < NH / 2; ++i) asm volatile("" : "+r"(v[i]));
}

template <int N> __device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&r)[N])
{
    if constexpr (N == 16)
        tc::tmem_ld16(addr, r);
    else
        tc::tmem_ld32(addr, r);
    tc::tmem_wait_ld(r);
}
template <int N> __device__ __forceinline__ void tmem_store(uint32_t addr, const uint32_t (&r)[N])
{
    if constexpr (N == 16)
        tc::tmem_st16(addr, r);
    else
        tc::tmem_st32(addr, r);
}

template <typename T, int NH> __device__ void soften(const Args& g, uint32_t sbase, Aux<NH>* x, uint8_t* ws, int* error)
{
    constexpr int NG = NH / 8, N = NH;
    const hs_attend_t& a = g.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r0 = lane >> 2, c0 = 2 * (lane & 3);
    const uint32_t lanes = (uint32_t)warp << 21;
    const uint32_t tmem = x->tmem + lanes;
    long long j = 0;
    Walk walk(g, x->piece);
    for (int pieces = 0; walk.next(); ++pieces) {
        float c[2 * NG], ref[2 * NG], sum[2 * NG];  // of this thread's columns (heads)
        unsigned seen = 0;                          // columns whose reference is a maximum
#pragma unroll
        for (int i = 0; i < 2 * NG; ++i) c[i] = a.scale * 1.4426950408889634f, ref[i] = 0.f, sum[i] = 0.f;
        for (int t = walk.t0; t < walk.t1; ++t, ++j) {
            const int s = (int)(j & 1), m = (int)(j & 3);
            wait(tc::smem_addr(&x->sfull[s]), (j >> 1) & 1, &x->dead, error);
            tc::fence_after();
            if constexpr (HsType<T>::is_bf16)
                if (t == walk.t0)
#pragma unroll
                    for (int i = 0; i < 2 * NG; ++i)
                        c[i] *= power_of_two(-x->q_up[pieces % 3][8 * (i >> 1) + c0 + (i & 1)]);
            uint32_t r[NH / 2];
            load_scores<NH>(tmem + Layout<NH>::col_s + NH * s, r);
            const unsigned valid = x->valid[m][warp];
            const bool ok0 = valid >> r0 & 1, ok1 = valid >> (r0 + 8) & 1;
            const float w0 = x->scale[m][16 * warp + r0], w1 = x->scale[m][16 * warp + r0 + 8];
            // only move the reference
            const float lw0 = fmaxf(tc::log2_approx(fabsf(w0)), kLeastLogScale), lw1 = fmaxf(tc::log2_approx(fabsf(w1)), kLeastLogScale);
            float v[NH / 2], top[2 * NG];
#pragma unroll
            for (int i = 0; i < 2 * NG; ++i) {  // column i: registers 4 (i / 2) + i % 2 and + 2
                const int k = 4 * (i >> 1) + (i & 1);
                v[k] = ok0 ? __uint_as_float(r[k]) * c[i] * w0 : -INFINITY;
                v[k + 2] = ok1 ? __uint_as_float(r[k + 2]) * c[i] * w1 : -INFINITY;
                top[i] = fmaxf(v[k] + lw0, v[k + 2] + lw1);
            }
#pragma unroll
            for (int o = 4; o < 32; o <<= 1)
#pragma unroll
                for (int i = 0; i < 2 * NG; ++i) top[i] = fmaxf(top[i], __shfl_xor_sync(~0u, top[i], o));
            if (lane < 4)
#pragma unroll
                for (int i = 0; i < NG; ++i) *reinterpret_cast<float2*>(&x->top[s][warp][8 * i + c0]) = make_float2(top[2 * i], top[2 * i + 1]);
            asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                float2 q = *reinterpret_cast<float2*>(&x->top[s][0][8 * i + c0]);
#pragma unroll
                for (int k = 1; k < 4; ++k) {
                    const float2 n = *reinterpret_cast<float2*>(&x->top[s][k][8 * i + c0]);
                    q.x = fmaxf(q.x, n.x), q.y = fmaxf(q.y, n.y);
                }
                top[2 * i] = q.x, top[2 * i + 1] = q.y;
            }
            // every warp sees the same maxima, so they agree on what follows
            float keep[2 * NG];
            bool scale_o = false;
#pragma unroll
            for (int i = 0; i < 2 * NG; ++i) {
                keep[i] = 1.f;
                const bool had = seen >> i & 1;
                if (top[i] > -INFINITY && (!had || top[i] > ref[i] + 8.f)) {
                    keep[i] = tc::exp2_approx(fminf(ref[i] - top[i], 126.f));
                    sum[i] *= keep[i];
                    ref[i] = top[i];
                    if (!had) {
                        seen |= 1u << i;
                        keep[i] = 1.f;  // O of this head holds nothing yet
                    }
                    scale_o = scale_o || had;
                }
            }
            // The buffer of P is free once the product that read it last is done.
            if (j >= 2) wait(tc::smem_addr(&x->pvdone[s]), ((j - 2) >> 1) & 1, &x->dead, error);
            if (__any_sync(~0u, scale_o) && t > walk.t0) {
                wait(tc::smem_addr(&x->pvdone[1 - s]), ((j - 1) >> 1) & 1, &x->dead, error);
                tc::fence_after();
                if (lane < 4)
#pragma unroll
                    for (int i = 0; i < NG; ++i)
                        *reinterpret_cast<float2*>(&x->red[warp][8 * i + c0]) = make_float2(keep[2 * i], keep[2 * i + 1]);
                __syncwarp();
#pragma unroll 1
                for (int n = 0; n < 4 * NH; n += N) {
                    uint32_t o[N];
                    tmem_load(tmem + n, o);
#pragma unroll
                    for (int i = 0; i < N; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * x->red[warp][i]);
                    tmem_store(tmem + n, o);
                }
                tc::tmem_wait_st();
                __syncwarp();
            }
            // P^T: row (head), 64 of the tile's rows along it
            const uint32_t p_smem = sbase + Layout<NH>::off_p + s * NH * 128;
#pragma unroll
            for (int i = 0; i < 2 * NG; ++i) {
                const int k = 4 * (i >> 1) + (i & 1), head = 8 * (i >> 1) + c0 + (i & 1);
                const float p0 = tc::exp2_approx(v[k] - ref[i]), p1 = tc::exp2_approx(v[k + 2] - ref[i]);
                sum[i] += p0 + p1;
                const uint32_t both = pack2<__half>(p0 * w0, p1 * w1);
                const uint32_t dst = p_smem + head * 128 + 2 * r0;
                const uint32_t sw = (uint32_t)head & 7;
                asm volatile("st.shared.b16 [%0], %1;" ::"r"(dst + (((2 * warp) ^ sw) << 4)), "h"((uint16_t)(both & 0xffff)) : "memory");
                asm volatile("st.shared.b16 [%0], %1;" ::"r"(dst + (((2 * warp + 1) ^ sw) << 4)), "h"((uint16_t)(both >> 16)) : "memory");
            }
            tc::fence_async_shared();
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(tc::smem_addr(&x->pready[s]));
        }
        // The piece's end: the sums over all rows of a head, then O^T leaves, a channel a thread.
#pragma unroll
        for (int o = 4; o < 32; o <<= 1)
#pragma unroll
            for (int i = 0; i < 2 * NG; ++i) sum[i] += __shfl_xor_sync(~0u, sum[i], o);
        if (lane < 4)
#pragma unroll
            for (int i = 0; i < NG; ++i) *reinterpret_cast<float2*>(&x->red[warp][8 * i + c0]) = make_float2(sum[2 * i], sum[2 * i + 1]);
        asm volatile("bar.sync 1, 128;" ::: "memory");
        const bool whole = walk.t0 == 0 && walk.t1 == walk.tiles;
        Partial<NH>* part = reinterpret_cast<Partial<NH>*>(ws + kOffPartial) + 2 * blockIdx.x + (walk.t0 == 0 ? 1 : 0);
        const long long unit = walk.b * a.positions + walk.p;
        if (warp == 0 && lane < 4)
#pragma unroll
            for (int i = 0; i < 2 * NG; ++i) {
                const int head = 8 * (i >> 1) + c0 + (i & 1);
                const float l = x->red[0][head] + x->red[1][head] + x->red[2][head] + x->red[3][head];
                x->inv[head] = l > 0.f || l != l ? 1.f / l : 0.f;
                if (!whole)
                    part->ref[head] = ref[i], part->sum[head] = l;
                else if (a.lse && head < a.heads)
                    a.lse[unit * a.heads + head] = l > 0.f || l != l ? (ref[i] + log2f(l)) * 0.6931471805599453f : -INFINITY;
            }
        wait(tc::smem_addr(&x->pvdone[(j - 1) & 1]), ((j - 1) >> 1) & 1, &x->dead, error);
        tc::fence_after();
        asm volatile("bar.sync 1, 128;" ::: "memory");
        T* out = static_cast<T*>(a.out) + walk.b * a.out_stride[0] + walk.p * a.out_stride[1] + 32 * warp + lane;
#pragma unroll 1
        for (int n = 0; n < 4 * NH; n += N) {
            uint32_t o[N];
            __syncwarp();
            tmem_load(tmem + n, o);
            const int i = n / NH;
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const int head = k;
                if (head >= a.heads) continue;
                if (whole) {
                    const float f = x->inv[head];  // 0: no row counted
                    out[head * a.out_stride[2] + 128 * i] = HsType<T>::from_float(f == 0.f ? 0.f : __uint_as_float(o[k]) * f);
                } else {
                    part->o[i][head][32 * warp + lane] = __uint_as_float(o[k]);
                }
            }
        }
        tc::fence_before();
        asm volatile("bar.sync 1, 128;" ::: "memory");  // red and inv are free again
    }
}

template <typename T, int NH>
__global__ void __launch_bounds__(kThreads, 1) hs_attend_narrow_kernel(const __grid_constant__ Args g)
{
    extern __shared__ __align__(1024) uint8_t base[];  // the swizzled tiles need 1024
    const uint32_t sbase = tc::smem_addr(base);
    Aux<NH>* x = reinterpret_cast<Aux<NH>*>(base + Layout<NH>::off_aux);
    const hs_attend_t& a = g.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    int* error = reinterpret_cast<int*>(ws);

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join may queue up behind this grid
    if (warp == 0) tc::tmem_alloc<1>(tc::smem_addr(&x->tmem), Layout<NH>::cols);
    if (warp == 12) {
        const Piece p = find_piece(g, blockIdx.x);
        if (lane == 0) {
            x->piece = p;
            x->dead = 0;
            reinterpret_cast<Start*>(ws + kOffStart)[blockIdx.x] = {p.count > 0 ? p.unit : -1, p.tile};
            for (int i = 0; i < 2; ++i) {
                tc::mbar_init(tc::smem_addr(&x->full[i]), 4);
                tc::mbar_init(tc::smem_addr(&x->sfull[i]), 1);
                tc::mbar_init(tc::smem_addr(&x->pready[i]), 4);
                tc::mbar_init(tc::smem_addr(&x->pvdone[i]), 1);
                tc::mbar_init(tc::smem_addr(&x->spare[i]), 1);
            }
            tc::mbar_init(tc::smem_addr(&x->qfull), 8);
            tc::mbar_init(tc::smem_addr(&x->qfree), 1);
            tc::mbar_init_fence();
        }
    }
    tc::fence_before();
    __syncwarp();
    __syncthreads();
    tc::fence_after();

    if (x->piece.count > 0) {
        if (warp < 4)
            soften<T, NH>(g, sbase, x, ws, error);
        else if (warp < 12)
            bring<T, NH>(g, sbase, x, error);
        else if (warp == 12)
            multiply_qk<NH>(g, sbase, x, error);
        else
            multiply_pv<NH>(g, sbase, x, error);
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 0) tc::tmem_free<1>(x->tmem, Layout<NH>::cols);
}

// Join the pieces of the units that several SMs worked on: block (x, y) takes the x-th such
// unit and four heads, a channel a thread.  The order of the sums is fixed.
constexpr int kJoinHeads = 4;
template <typename T, int NH>
__global__ void __launch_bounds__(512) hs_attend_narrow_join_kernel(const __grid_constant__ Args g, int ctas)
{
    __shared__ float weight[kMaxCtas][kJoinHeads], total[kJoinHeads], reference[kJoinHeads];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const hs_attend_t& a = g.a;
    const uint8_t* ws = static_cast<const uint8_t*>(a.workspace);
    const Partial<NH>* parts = reinterpret_cast<const Partial<NH>*>(ws + kOffPartial);
    int unit, first, last;
    if (!find_cut(reinterpret_cast<const Start*>(ws + kOffStart), ctas, blockIdx.x, unit, first, last)) return;
    const int t = threadIdx.x, h0 = kJoinHeads * blockIdx.y, n = last - first + 1;
    auto part = [&](int i) -> const Partial<NH>& { return parts[2 * (first + i) + (i == 0)]; };
    // Weights of the pieces: a warp a head.
    if (t < 32 * kJoinHeads) {
        const int k = t >> 5, lane = t & 31;
        float top = -INFINITY, sum = 0.f;
        for (int i = lane; i < n; i += 32)
            if (part(i).sum[h0 + k] != 0.f) top = fmaxf(top, part(i).ref[h0 + k]);
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
        for (int i = lane; i < n; i += 32) {
            const float l = part(i).sum[h0 + k];  // 0: no row counted
            const float w = l == 0.f ? 0.f : tc::exp2_approx(part(i).ref[h0 + k] - top);
            weight[i][k] = w;
            sum += w * l;
        }
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        if (lane == 0) total[k] = sum, reference[k] = top;
    }
    __syncthreads();
    float acc[kJoinHeads] = {};
#pragma unroll 4
    for (int i = 0; i < n; ++i)
#pragma unroll
        for (int k = 0; k < kJoinHeads; ++k) {
            const float w = weight[i][k], o = part(i).o[t >> 7][h0 + k][t & 127];
            acc[k] += w == 0.f ? 0.f : w * o;
        }
    const long long b = unit / a.positions;
    const int p = unit - (int)b * a.positions;
    T* out = static_cast<T*>(a.out) + b * a.out_stride[0] + p * a.out_stride[1] + t;
#pragma unroll
    for (int k = 0; k < kJoinHeads; ++k) {
        if (h0 + k >= a.heads) continue;
        const float l = total[k];
        const bool some = l > 0.f || l != l;
        out[(h0 + k) * a.out_stride[2]] = HsType<T>::from_float(some ? acc[k] / l : 0.f);
        if (a.lse && t == 0) a.lse[(int64_t)unit * a.heads + h0 + k] = some ? (reference[k] + log2f(l)) * 0.6931471805599453f : -INFINITY;
    }
}

template <typename T, int NH> cudaError_t launch(const Args& g, cudaStream_t s)
{
    cudaError_t e = cudaFuncSetAttribute(hs_attend_narrow_kernel<T, NH>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<NH>());
    if (e != cudaSuccess) return e;
    hs_attend_narrow_kernel<T, NH><<<g.workers, kThreads, smem_bytes<NH>(), s>>>(g);
    e = cudaGetLastError();
    if (e != cudaSuccess || !g.flat || g.workers <= 1) return e;
    const int cut = g.units < g.workers - 1 ? g.units : g.workers - 1;  // at most this many units are cut
    return launch_after(hs_attend_narrow_join_kernel<T, NH>, dim3(cut, (g.a.heads + kJoinHeads - 1) / kJoinHeads), 512, 0, s, g, g.workers);
}

}  // namespace

size_t narrow_workspace(int64_t units, int64_t tiles, int heads)
{
    const size_t part = heads <= 16 ? sizeof(Partial<16>) : sizeof(Partial<32>);
    return kOffPartial + part * 2 * (size_t)(units * tiles < kMaxCtas ? units * tiles : kMaxCtas);
}

cudaError_t launch_narrow(const hs_attend_t& a, int sms, cudaStream_t s)
{
    Args g;
    g.a = a;
    g.head_blocks = 1;
    g.units = a.batch * a.positions;
    // Pieces also write and join up to two partial results an SM: about 8 us, 6 tiles' time.
    g.cut(sms < kMaxCtas ? sms : kMaxCtas, a.slots ? a.entries : a.n_rows, 6, kUnitCost);
    if (a.dtype == HS_TYPE_BF16) return a.heads <= 16 ? launch<__nv_bfloat16, 16>(g, s) : launch<__nv_bfloat16, 32>(g, s);
    return a.heads <= 16 ? launch<__half, 16>(g, s) : launch<__half, 32>(g, s);
}

}  // namespace hs_attn
