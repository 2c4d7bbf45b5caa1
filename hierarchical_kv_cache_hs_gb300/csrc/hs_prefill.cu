// hs_latent_prefill: expanded latent attention of ragged prompts, causal.
//
// Three launches.
// (1) Expansion: keys and values of every head, [k; v] = [w_uk; w_uv] latent, a
//     product of k_tokens x 256 heads x 512.  A pair of SMs (cta_group::2, M = N =
//     256) keeps 256 tokens' latents in shared memory and runs through heads; the
//     weights' half that each CTA brings serves both.
// (2) Attention: a pair of SMs takes 512 queries of a head as two tiles of 256 that
//     take turns: while one tile's scores are softened, the other's products run.
//     The scores (then the weights, in place) and the sums of both tiles fill tensor
//     memory; keys (192 channels) and values pass through shared memory in blocks of
//     128 tokens, which the expansion has written as they lie there; each CTA holds
//     half of a block.
// (3) Join: the blocks of all units (head, 512 queries) form one line that is cut
//     into equal pieces, one a pair; units cut in two or more are joined.
//
// 8192 tokens x 32 heads (bf16) take 562 us, 1,345 TFLOP/s (0.70 of a product's rate):
// (1) 52, bound by what it writes and L2; (2) 471, bound by the softmax of a tile where it
// outlasts the other tile's products.  512 tokens after 15,872 cached 8-bit rows x 16
// heads (fp16): 135, of them 60 and 72, the second's start within the first's end.
//
// Keys, values and softmax weights are rounded to the call's type before their products,
// as the tensor core takes them: bf16 results are 0.0026 to 0.0028 off 64 bits (relative,
// in norm) where one rounding at the end gives 0.0017; sums and statistics are fp32.
// Values and weights in fp16 for bf16 calls would come closer, but bf16 values reach past
// fp16's range: each token would need a power of two of its own, on each weight, in the
// softmax, which is the bound.
#include "hs_ops.h"
#include "hs_tc.h"

namespace {

using tc::wait;

constexpr int kMaxPairs = 76;

// Workspace: an error word, where each pair's piece starts, two partial results a
// pair; then, for blocks of 128 tokens (counted over all requests, the tail padded to
// 256 tokens with zeros), the tiles that the attention copies to shared memory as
// they are, rows of 128 bytes with the 128-byte swizzle:
//   keys    [head][block][2 x 64 tokens][2 x 64 channels][64 tokens]
//   values  [head][block][2 x 64 channels][128 tokens]
//   rotary  [block][128 tokens]
struct Start {
    int b, h, qt, kb;
};
struct Partial {
    float o[4][128][128];  // [128 queries][channel][query]
    float ref[4][128], sum[4][128];
};
constexpr size_t kOffStart = 256;
constexpr size_t kOffPartial = kOffStart + sizeof(Start) * (kMaxPairs + 4);
constexpr size_t kOffKeys = kOffPartial + sizeof(Partial) * 2 * kMaxPairs;

constexpr int kBlock = 32768;  // keys, or values, of a block and head
constexpr int kRope = 16384;   // rotary channels of a block

struct Args {
    hs_prefill_t a;
    uint8_t* keys;
    uint8_t* values;
    uint8_t* rope;
    int64_t blocks;
    int flat;  // 1: equal pieces of the line of blocks; 0: whole units
};

// A NaN or an infinity among two values of T.
template <typename T> __device__ __forceinline__ bool not_finite(uint32_t v)
{
    const uint32_t m = HsType<T>::is_bf16 ? 0x7f80u : 0x7c00u;
    return (v & m) == m || (v >> 16 & m) == m;
}
// Two e4m3 values as T (exact).
template <typename T> __device__ __forceinline__ uint32_t widen2(uint32_t v)
{
    uint32_t h;
    asm("{\n\t.reg .b16 a;\n\tcvt.u16.u32 a, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(h) : "r"(v));
    if constexpr (!HsType<T>::is_bf16) return h;
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return pack2<T>(f.x, f.y);
}

// ---- (1) expansion -----------------------------------------------------------------

constexpr int kEStages = 4;
constexpr int kEBring = 2 * kEStages;          // warps that bring weights, two a stage
constexpr int kEThreads = (5 + kEBring) * 32;  // warps 0-3 write, then those, the last issues the products
constexpr int kEOffB = 8 * 16384;  // latents: 8 blocks of 64 channels, [128 tokens][128 B]
constexpr int kEOffOut = kEOffB + kEStages * 16384;  // two pieces on their way out, 64 channels of 128 tokens each
constexpr int kEOffAux = kEOffOut + 2 * 16384;
struct EAux {
    uint64_t afull, bfull[kEStages], bfree[kEStages], dfull[2], dfree[2], spare;
    uint32_t tmem;
    int dead;
};
constexpr int kESmem = kEOffAux + (int)sizeof(EAux);

template <typename T, bool E4M3>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kEThreads, 1) hs_expand_kernel(const __grid_constant__ Args g)
{
    extern __shared__ __align__(1024) uint8_t base[];
    const uint32_t sbase = tc::smem_addr(base);
    EAux* x = reinterpret_cast<EAux*>(base + kEOffAux);
    const hs_prefill_t& a = g.a;
    const uint32_t rank = tc::cluster_rank();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int* error = static_cast<int*>(a.workspace);
    // This pair's piece of the line of jobs (256 tokens, head).
    const int64_t jobs = (a.k_tokens + 255) / 256 * a.heads;
    const int64_t pairs = gridDim.x >> 1, pair = blockIdx.x >> 1;
    const int64_t lo = jobs * pair / pairs, hi = jobs * (pair + 1) / pairs;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == 0) tc::tmem_alloc<2>(tc::smem_addr(&x->tmem), 512);
    if (threadIdx.x == 0) {
        x->dead = 0;
        tc::mbar_init(tc::smem_addr(&x->afull), 2 * kEBring);
        for (int i = 0; i < kEStages; ++i) {
            tc::mbar_init(tc::smem_addr(&x->bfull[i]), 4);
            tc::mbar_init(tc::smem_addr(&x->bfree[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(tc::smem_addr(&x->dfull[i]), 1);
            tc::mbar_init(tc::smem_addr(&x->dfree[i]), 8);
        }
        tc::mbar_init(tc::smem_addr(&x->spare), 1);
        tc::mbar_init_fence();
    }
    tc::fence_before();
    __syncthreads();
    tc::cluster_sync();
    tc::fence_after();

    if (warp < 4) {
        // A token a thread: values first (a value that is not finite becomes 0 and its key NaN: a weight
        // of 0 must hide it from the queries that do not see it, and the others must get NaN).
        const uint32_t tmem = x->tmem + ((uint32_t)warp << 21);
        const uint32_t dfree[2] = {tc::map_to_rank(tc::smem_addr(&x->dfree[0]), 0),
                                   tc::map_to_rank(tc::smem_addr(&x->dfree[1]), 0)};
        for (int64_t job = lo; job < hi; ++job) {
            const int n = (int)(job - lo), d = n & 1;
            const int64_t mt = job / a.heads, h = job - mt * a.heads;
            const int64_t token = mt * 256 + 128 * (int)rank + threadIdx.x;
            const bool live = token < a.k_tokens;
            float scale = 1.f;
            if (E4M3 && live)
                scale = *reinterpret_cast<const float*>(static_cast<const uint8_t*>(a.rows) + token * a.row_stride + HS_ROW8_SCALE);
            wait(tc::smem_addr(&x->dfull[d]), (n >> 1) & 1, &x->dead, error);
            tc::fence_after();
            bool bad = false;
            const int64_t tile = h * g.blocks + mt * 2 + rank;
            const int tok = threadIdx.x;
#pragma unroll 1
            for (int piece = 0; piece < 4; ++piece) {  // 64 channels: values, then keys
                const bool keys = piece >= 2;
                const int cb = piece & 1;
                const uint32_t buf = sbase + kEOffOut + cb * 16384;
                uint32_t r[2][32];
                tc::tmem_ld32(tmem + 256 * d + (keys ? 0 : 128) + 64 * cb, r[0]);
                tc::tmem_ld32(tmem + 256 * d + (keys ? 0 : 128) + 64 * cb + 32, r[1]);
                // the piece that was in this buffer has been read
                if (threadIdx.x == 0) tc::bulk_wait_read<1>();
                asm volatile("bar.sync 3, 128;" ::: "memory");
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t e[16];
                    tc::tmem_wait_ld(r[half]);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float p = __uint_as_float(r[half][2 * i]), q = __uint_as_float(r[half][2 * i + 1]);
                        if (E4M3) p *= scale, q *= scale;
                        e[i] = pack2<T>(p, q);
                        if (!keys && not_finite<T>(e[i])) bad = true, e[i] = 0;
                    }
                    if (keys && bad) e[0] = ~0u;
                    // keys lie as two tiles of 64 tokens, values as one of 128: the same bytes
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        tc::st_shared16(buf + tok * 128 + (((half * 4 + i) ^ (tok & 7)) << 4), e[4 * i], e[4 * i + 1], e[4 * i + 2],
                                        e[4 * i + 3]);
                }
                tc::fence_async_shared();
                asm volatile("bar.sync 3, 128;" ::: "memory");
                if (threadIdx.x == 0) {
                    if (keys) {
                        uint8_t* dst = g.keys + tile * kBlock + cb * 8192;
                        tc::bulk_store(dst, buf, 8192);
                        tc::bulk_store(dst + 16384, buf + 8192, 8192);
                    } else {
                        tc::bulk_store(g.values + tile * kBlock + cb * 16384, buf, 16384);
                    }
                    tc::bulk_commit();
                }
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_cluster(dfree[d]);
        }
        if (threadIdx.x == 0) tc::bulk_wait_all();
    } else if (warp < 4 + kEBring) {
        const int me = warp - 4, s = me >> 1, half = me & 1;
        const uint32_t bfull = tc::map_to_rank(tc::smem_addr(&x->bfull[s]), 0);
        const uint32_t afull = tc::map_to_rank(tc::smem_addr(&x->afull), 0);
        const uint8_t* w = static_cast<const uint8_t*>(rank ? a.w_uv : a.w_uk);
        const int ch = lane & 7;
        int fills = 0;  // of this warp's stage
        int64_t at = -1;
        for (int64_t job = lo; job < hi; ++job) {
            const int64_t mt = job / a.heads, h = job - mt * a.heads;
            if (mt != at) {
                // The earlier tokens' products are done: each stage's last one is (each of these warps waits
                // for its own stage).
                if (fills) wait(tc::smem_addr(&x->bfree[s]), (fills - 1) & 1, &x->dead, error);
                asm volatile("bar.sync 2, %0;" ::"n"(32 * kEBring) : "memory");
                at = mt;
                for (int i = me; i < 32; i += kEBring) {  // a quarter of a block of channels each
                    const int kb = i >> 2;
#pragma unroll
                    for (int n = 0; n < 8; ++n) {
                        const int r = (i & 3) * 32 + n * 4 + (lane >> 3);
                        const int64_t token = mt * 256 + 128 * (int)rank + r;
                        const bool live = token < a.k_tokens;
                        const uint8_t* src = static_cast<const uint8_t*>(a.rows) + (live ? token : 0) * a.row_stride;
                        const uint32_t dst = sbase + kb * 16384 + r * 128 + ((ch ^ (r & 7)) << 4);
                        if constexpr (!E4M3) {
                            tc::cp_async16(dst, src + kb * 128 + ch * 16, live);
                        } else {
                            const uint2 v = live ? *reinterpret_cast<const uint2*>(src + kb * 64 + ch * 8) : make_uint2(0, 0);
                            tc::st_shared16(dst, widen2<T>(v.x & 0xffff), widen2<T>(v.x >> 16), widen2<T>(v.y & 0xffff),
                                            widen2<T>(v.y >> 16));
                        }
                    }
                }
                if (h == 0) {  // the rotary channels' tile (of 8-bit rows: scaled, and rounded to T)
                    for (int i = 32 * me + lane; i < 128 * 8; i += 32 * kEBring) {
                        const int tok = i >> 3;
                        const int64_t token = mt * 256 + 128 * (int)rank + tok;
                        const uint8_t* src = static_cast<const uint8_t*>(a.rows) + token * a.row_stride;
                        uint4 e = make_uint4(0, 0, 0, 0);
                        if (token < a.k_tokens) {
                            if constexpr (!E4M3) {
                                e = *reinterpret_cast<const uint4*>(src + (HS_LATENT_DIM + (i & 7) * 8) * 2);
                            } else {
                                const float f = *reinterpret_cast<const float*>(src + HS_ROW8_SCALE);
                                const uint2 v = *reinterpret_cast<const uint2*>(src + HS_LATENT_DIM + (i & 7) * 8);
                                auto two = [&](uint32_t w) { return pack2<T>(hs_e4m3_to_float(w & 0xff) * f, hs_e4m3_to_float(w >> 8 & 0xff) * f); };
                                e = make_uint4(two(v.x), two(v.x >> 16), two(v.y), two(v.y >> 16));
                            }
                        }
                        *reinterpret_cast<uint4*>(g.rope + (mt * 2 + rank) * kRope + tok * 128 + (((i & 7) ^ (tok & 7)) << 4)) = e;
                    }
                }
                tc::cp_async_commit();
                tc::cp_async_wait<0>();
                tc::fence_async_shared();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive_cluster(afull);
            }
            // the piece's n-th block of channels goes to stage n % kEStages
            for (int kb = 0; kb < 8; ++kb) {
                if ((8 * (job - lo) + kb) % kEStages != s) continue;
                if (fills) wait(tc::smem_addr(&x->bfree[s]), (fills - 1) & 1, &x->dead, error);
                ++fills;
                const int r0 = 64 * half + (lane >> 3);
                const uint8_t* src = w + ((h * HS_HEAD_DIM + r0) * HS_LATENT_DIM + kb * 64 + ch * 8) * 2;
                const uint32_t dst = sbase + kEOffB + s * 16384 + r0 * 128;
#pragma unroll
                for (int n = 0; n < 16; ++n)
                    tc::cp_async16(dst + n * 512 + ((ch ^ ((n * 4 + r0) & 7)) << 4), src + (int64_t)n * 4 * HS_LATENT_DIM * 2, true);
                tc::cp_async_commit();
                tc::cp_async_wait<0>();
                tc::fence_async_shared();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive_cluster(bfull);
            }
        }
    } else if (rank == 0) {
        const uint32_t tmem = __shfl_sync(~0u, x->tmem, 0);
        constexpr uint32_t id = tc::inst_desc(HsType<T>::is_bf16, 256, 256, false, false);
        int64_t at = -1;
        int tiles = 0, stage = 0;
        uint32_t phase = 0;
        const uint64_t a_desc = tc::smem_desc(sbase, 16, 1024), b_desc = tc::smem_desc(sbase + kEOffB, 16, 1024);
        for (int64_t job = lo; job < hi; ++job) {
            const int n = (int)(job - lo), d = n & 1;
            const int64_t mt = job / a.heads;
            if (mt != at) wait(tc::smem_addr(&x->afull), tiles++ & 1, &x->dead, error);
            at = mt;
            if (n >= 2) wait(tc::smem_addr(&x->dfree[d]), ((n - 2) >> 1) & 1, &x->dead, error);
#pragma unroll 1
            for (int kb = 0; kb < 8; ++kb) {
                wait(tc::smem_addr(&x->bfull[stage]), phase, &x->dead, error);
                __syncwarp();
                tc::fence_after();
                const uint64_t ad = a_desc + kb * 1024, bd = b_desc + stage * 1024;
                if (tc::elect_one()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) tc::mma_ss<2>(tmem + 256 * d, ad + 2 * k, bd + 2 * k, id, (kb | k) != 0);
                    tc::commit<2>(tc::smem_addr(&x->bfree[stage]));
                    if (kb == 7) tc::commit<2>(tc::smem_addr(&x->dfull[d]));
                }
                __syncwarp();
                if (++stage == kEStages) stage = 0, phase ^= 1;
            }
        }
        if (*(volatile int*)&x->dead) {  // what was issued must be complete before tensor memory is freed
            if (tc::elect_one()) tc::commit<2>(tc::smem_addr(&x->spare));
            __syncwarp();
            tc::mbar_wait(tc::smem_addr(&x->spare), 0);
        }
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    tc::cluster_sync();
    tc::fence_after();
    if (warp == 0) tc::tmem_free<2>(x->tmem, 512);
}

// ---- (2) attention -----------------------------------------------------------------

constexpr int kThreads = 12 * 32;  // warps 0-7 softmax (four a tile), 8-9 queries, 10 keys and values, 11 products
constexpr int kStages = 3;
constexpr int kQTile = 3 * 16384;                 // 3 blocks of 64 channels, [128 queries][128 B]
constexpr int kOffK = 2 * kQTile;
constexpr int kKStage = kBlock / 2 + kRope / 2;   // 64 tokens: 3 blocks of 64 channels, [64][128 B]
constexpr int kOffV = kOffK + kStages * kKStage;
constexpr int kVStage = kBlock / 2;               // 64 channels of 128 tokens
constexpr int kOffAux = kOffV + kStages * kVStage;
struct Aux {
    // kfull, vfull: this CTA's half; kpeer, vpeer (first CTA): the other's
    uint64_t qfull, qfree, kfull[kStages], kpeer[kStages], kfree[kStages], vfull[kStages], vpeer[kStages], vfree[kStages];
    uint64_t sfull[2], pfull[2][2], odone[2], spare;  // pfull: weights of a block's first and second 64 keys
    uint32_t tmem;
    int dead;
    Start start, stop;  // this pair's piece of the line
    int any;
};
constexpr int kSmem = kOffAux + (int)sizeof(Aux);
static_assert(kSmem <= 232448, "shared memory");

// Tensor memory of tile s: scores (then weights) at 256 s, sums at 256 s + 128.

// Stage and phase of the block after this one.
struct Ring {
    int s = 0;
    uint32_t phase = 0;
    __device__ void step()
    {
        if (++s == kStages) s = 0, phase ^= 1;
    }
};

// Blocks' time that a unit's queries, first scores and output take: by it pieces of many
// short units and pieces of few long ones end together (8192 tokens, 32 heads: 575 us
// without it, 564 with 3, 565 with 2, 564 with 4, 590 with 6).
constexpr int kUnitCost = 3;

struct Request {
    long long q0, k0;
    int n, m;  // queries, rows
    __device__ Request(const hs_prefill_t& a, int b)
    {
        auto clamp = [](long long v, long long most) { return v < 0 ? 0 : v > most ? most : v; };
        q0 = clamp(a.q_start[b], a.q_tokens);
        k0 = clamp(a.k_start[b], a.k_tokens);
        const long long q1 = clamp(a.q_start[b + 1], a.q_tokens), k1 = clamp(a.k_start[b + 1], a.k_tokens);
        n = q1 > q0 ? (int)(q1 - q0) : 0;
        m = k1 > k0 ? (int)(k1 - k0) : 0;
    }
    __device__ int q_tiles() const { return (n + 511) / 512; }
    // Key blocks, from the one that holds the request's first row, that queries below `end` see.
    __device__ int blocks_to(int end) const
    {
        const long long keys = (long long)(end < n ? end : n) + m - n;  // the last of them sees this many
        return keys <= 0 ? 0 : (int)(((k0 & 127) + keys + 127) / 128);
    }
    __device__ int blocks(int qt) const { return max(1, blocks_to(512 * qt + 512)); }
    // What the line is cut by: blocks, and kUnitCost of them for a unit's own time; or units.
    __device__ long long size_of_head(bool flat) const
    {
        if (!flat) return q_tiles();
        long long t = 0;
        for (int i = 0; i < q_tiles(); ++i) t += blocks(i) + kUnitCost;
        return t;
    }
};

// The units, or parts of units, of a pair's piece, in order.
struct Walk {
    const hs_prefill_t& a;
    const Start stop;
    int b, h, qt, kb;
    bool done;
    Request r;
    // the current one
    int head, tile, t0, t1, blocks;
    __device__ Walk(const Args& g, const Aux* x)
        : a(g.a), stop(x->stop), b(x->start.b), h(x->start.h), qt(x->start.qt), kb(x->start.kb), done(false), r(g.a, x->start.b)
    {
    }
    __device__ bool next()
    {
        if (done) return false;
        while (qt >= r.q_tiles()) {
            qt = 0;
            if (r.n == 0 || ++h >= a.heads) {
                h = 0;
                if (++b >= a.batch) return false;
                r = Request(a, b);
            }
        }
        head = h;
        tile = qt;
        blocks = r.blocks(qt);
        t0 = kb;
        t1 = blocks;
        if (b == stop.b && h == stop.h && qt == stop.qt) {
            if (t0 >= stop.kb) return false;
            t1 = stop.kb;
            done = true;
        }
        kb = 0;
        ++qt;
        return true;
    }
    // Blocks that tile s of the piece works on: [t0, end(s)).
    __device__ int end(int s) const
    {
        if (512 * tile + 256 * s >= r.n) return t0;
        const int e = r.blocks_to(512 * tile + 256 * s + 256);
        return e < t0 ? t0 : e < t1 ? e : t1;
    }
};

// Queries of a piece: this CTA's 128 of a tile a warp.
template <typename T> __device__ void bring_queries(const Args& g, uint32_t sbase, Aux* x, uint32_t rank, int* error)
{
    const hs_prefill_t& a = g.a;
    const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - 8, ch = lane & 7;
    const uint32_t qfull = tc::map_to_rank(tc::smem_addr(&x->qfull), 0);
    Walk walk(g, x);
    for (int pieces = 0; walk.next(); ++pieces) {
        // Q's readers, the last piece's products with keys, are done.
        if (pieces) wait(tc::smem_addr(&x->qfree), (pieces - 1) & 1, &x->dead, error);
        const T* q = static_cast<const T*>(a.q) + walk.head * a.q_stride[1];
        const int q0 = 512 * walk.tile + 256 * w + 128 * (int)rank;
#pragma unroll 8
        for (int n = 0; n < 32; ++n) {
            const int r = n * 4 + (lane >> 3), at = q0 + r;
            const bool live = at < walk.r.n;
            const uint8_t* src = reinterpret_cast<const uint8_t*>(q + (walk.r.q0 + (live ? at : 0)) * a.q_stride[0]) + ch * 16;
            const uint32_t dst = sbase + w * kQTile + r * 128 + ((ch ^ (r & 7)) << 4);
#pragma unroll
            for (int c = 0; c < 3; ++c) tc::cp_async16(dst + c * 16384, src + c * 128, live);
        }
        tc::cp_async_commit();
        tc::cp_async_wait<0>();
        tc::fence_async_shared();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_cluster(qfull);
    }
}

// Keys and values: this CTA's half of whole tiles, by one thread.
__device__ void bring_tiles(const Args& g, uint32_t sbase, Aux* x, uint32_t rank, int* error)
{
    long long j = 0;
    Ring ring, last;
    Walk walk(g, x);
    while (walk.next()) {
        const int64_t block0 = walk.r.k0 / 128;
        for (int t = walk.t0; t < walk.t1; ++t, ++j) {
            // a block past the rows (a piece without any key) is any block that exists
            const int64_t block = block0 + t < g.blocks ? block0 + t : 0, tile = walk.head * g.blocks + block;
            const int s = ring.s;
            const uint32_t kbar = tc::smem_addr(&x->kfull[s]), vbar = tc::smem_addr(&x->vfull[s]);
            const uint32_t kdst = sbase + kOffK + s * kKStage, vdst = sbase + kOffV + s * kVStage;
            if (j >= kStages) wait(tc::smem_addr(&x->kfree[s]), ring.phase ^ 1, &x->dead, error);
            if (g.blocks == 0) {  // no rows at all
                tc::mbar_arrive(kbar);
            } else {
                tc::mbar_expect(kbar, kKStage);
                tc::bulk_load(kdst, g.keys + tile * kBlock + rank * (kBlock / 2), kBlock / 2, kbar);
                tc::bulk_load(kdst + kBlock / 2, g.rope + block * kRope + rank * (kRope / 2), kRope / 2, kbar);
            }
            if (j >= kStages) wait(tc::smem_addr(&x->vfree[s]), ring.phase ^ 1, &x->dead, error);
            if (g.blocks == 0) {
                tc::mbar_arrive(vbar);
            } else {
                tc::mbar_expect(vbar, kVStage);
                tc::bulk_load(vdst, g.values + tile * kBlock + rank * kVStage, kVStage, vbar);
            }
            last = ring;
            ring.step();
        }
    }
    // What is in flight has landed before the CTA ends; after a wait that gave up nothing else sees to it.
    if (j >= 1 && *(volatile int*)&x->dead)
        for (int s = 0; s < kStages && s < j; ++s) {
            const uint32_t phase = s <= last.s ? last.phase : last.phase ^ 1;
            tc::mbar_wait(tc::smem_addr(&x->kfull[s]), phase);
            tc::mbar_wait(tc::smem_addr(&x->vfull[s]), phase);
        }
}

// The second CTA tells the first that its half of a block has come.
__device__ void forward(const Args& g, Aux* x, int* error)
{
    Ring ring;
    Walk walk(g, x);
    while (walk.next())
        for (int t = walk.t0; t < walk.t1; ++t, ring.step()) {
            wait(tc::smem_addr(&x->kfull[ring.s]), ring.phase, &x->dead, error);
            tc::mbar_arrive_cluster(tc::map_to_rank(tc::smem_addr(&x->kpeer[ring.s]), 0));
            wait(tc::smem_addr(&x->vfull[ring.s]), ring.phase, &x->dead, error);
            tc::mbar_arrive_cluster(tc::map_to_rank(tc::smem_addr(&x->vpeer[ring.s]), 0));
        }
}

// Q K^T of tile S with the keys at k_desc, and P V of tile S with the values at v_desc.
template <typename T, int S> __device__ __forceinline__ void issue_qk(uint32_t sbase, uint32_t tmem, uint64_t k_desc, Aux* x)
{
    constexpr uint32_t id = tc::inst_desc(HsType<T>::is_bf16, 256, 128, false, false);
    const uint64_t q_desc = tc::smem_desc(sbase + S * kQTile, 16, 1024);
    if (tc::elect_one()) {
#pragma unroll
        for (int c = 0; c < 3; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                tc::mma_ss<2>(tmem + 256 * S, q_desc + ((c * 16384 + k * 32) >> 4), k_desc + ((c * 8192 + k * 32) >> 4), id,
                              (c | k) != 0);
        tc::commit<2>(tc::smem_addr(&x->sfull[S]));
    }
    __syncwarp();
}
template <typename T, int S, int HALF> __device__ __forceinline__ void issue_pv(uint32_t tmem, uint64_t v_desc, Aux* x, bool first)
{
    constexpr uint32_t id = tc::inst_desc(HsType<T>::is_bf16, 256, 128, false, true);
    if (tc::elect_one()) {
#pragma unroll
        for (int k = 4 * HALF; k < 4 * HALF + 4; ++k)
            tc::mma_ts<2>(tmem + 256 * S + 128, tmem + 256 * S + 8 * k, v_desc + ((k * 2048) >> 4), id, !(first && k == 0));
        if (HALF) tc::commit<2>(tc::smem_addr(&x->odone[S]));
    }
    __syncwarp();
}

// The products, issued by one warp of the first CTA in the order in which the tiles
// take turns: P V of a block, then Q K^T of the next one, of tile 0 and then of tile
// 1.  (Issued by a warp a tile, the two tiles' products ran interleaved, both tiles'
// scores came at the same time, and the tensor core idled through both softmaxes.)
template <typename T> __device__ void multiply(const Args& g, uint32_t sbase, Aux* x, int* error)
{
    const uint32_t tmem = __shfl_sync(~0u, x->tmem, 0);
    const uint64_t k_base = tc::smem_desc(sbase + kOffK, 16, 1024), v_base = tc::smem_desc(sbase + kOffV, 16384, 1024);
    int pieces = 0;
    uint32_t phase[2] = {0, 0};  // of pfull
    Ring now, next;              // the block of P V, and of Q K^T
    Walk walk(g, x);
    auto release = [](uint64_t& bar) {  // in both CTAs, when all products so far are complete
        if (tc::elect_one()) tc::commit<2>(tc::smem_addr(&bar));
        __syncwarp();
    };
    auto keys_come = [&]() {
        wait(tc::smem_addr(&x->kfull[next.s]), next.phase, &x->dead, error);
        wait(tc::smem_addr(&x->kpeer[next.s]), next.phase, &x->dead, error);
        __syncwarp();
        tc::fence_after();
    };
    while (walk.next()) {
        const int end[2] = {walk.end(0), walk.end(1)};
        wait(tc::smem_addr(&x->qfull), pieces++ & 1, &x->dead, error);
        keys_come();
        uint64_t k_desc = k_base + next.s * (kKStage >> 4);
        if (walk.t0 < end[0]) issue_qk<T, 0>(sbase, tmem, k_desc, x);
        if (walk.t0 < end[1]) issue_qk<T, 1>(sbase, tmem, k_desc, x);
        release(x->kfree[next.s]);
        if (walk.t1 - walk.t0 == 1) release(x->qfree);
        next.step();
        for (int t = walk.t0; t < walk.t1; ++t) {
            const bool more = t + 1 < walk.t1;
            wait(tc::smem_addr(&x->vfull[now.s]), now.phase, &x->dead, error);
            wait(tc::smem_addr(&x->vpeer[now.s]), now.phase, &x->dead, error);
            const uint64_t v_desc = v_base + now.s * (kVStage >> 4);
            k_desc = k_base + next.s * (kKStage >> 4);
#pragma unroll
            for (int tile = 0; tile < 2; ++tile) {
                if (t < end[tile]) {
                    wait(tc::smem_addr(&x->pfull[tile][0]), phase[tile], &x->dead, error);
                    __syncwarp();
                    tc::fence_after();
                    if (tile == 0)
                        issue_pv<T, 0, 0>(tmem, v_desc, x, t == walk.t0);
                    else
                        issue_pv<T, 1, 0>(tmem, v_desc, x, t == walk.t0);
                    wait(tc::smem_addr(&x->pfull[tile][1]), phase[tile], &x->dead, error);
                    phase[tile] ^= 1;
                    __syncwarp();
                    tc::fence_after();
                    if (tile == 0)
                        issue_pv<T, 0, 1>(tmem, v_desc, x, false);
                    else
                        issue_pv<T, 1, 1>(tmem, v_desc, x, false);
                }
                if (tile == 1) release(x->vfree[now.s]);
                if (tile == 0 && more) keys_come();
                if (t + 1 < end[tile]) {
                    if (tile == 0)
                        issue_qk<T, 0>(sbase, tmem, k_desc, x);
                    else
                        issue_qk<T, 1>(sbase, tmem, k_desc, x);
                }
            }
            now.step();
            if (more) {
                release(x->kfree[next.s]);
                if (t + 2 == walk.t1) release(x->qfree);
                next.step();
            }
        }
    }
    if (*(volatile int*)&x->dead) {  // what was issued must be complete before tensor memory is freed
        release(x->spare);
        tc::mbar_wait(tc::smem_addr(&x->spare), 0);
    }
}

// Softmax of one tile: a query a thread.
template <typename T> __device__ void soften(const Args& g, Aux* x, uint32_t rank, uint8_t* ws, int* error)
{
    const hs_prefill_t& a = g.a;
    const int lane = threadIdx.x & 31, tile = threadIdx.x >> 7, row = threadIdx.x & 127;
    const uint32_t tmem = x->tmem + 256 * tile + ((uint32_t)((threadIdx.x >> 5) & 3) << 21);
    const bool flip = a.scale < 0.f;  // scores are negated then, so that the scale is not negative
    const float c = fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1e-37f);  // not 0: a masked score stays -inf
    const uint32_t pfull[2] = {tc::map_to_rank(tc::smem_addr(&x->pfull[tile][0]), 0),
                               tc::map_to_rank(tc::smem_addr(&x->pfull[tile][1]), 0)};
    long long mine = 0;
    Walk walk(g, x);
    while (walk.next()) {
        const int end = walk.end(tile);
        const int at = 512 * walk.tile + 256 * tile + 128 * (int)rank + row;
        const int skip = (int)(walk.r.k0 & 127);                       // the first block's tokens of other requests
        const int keys = min(at + 1 + walk.r.m - walk.r.n, walk.r.m);  // the keys this query sees
        float ref = 0.f, sum = 0.f;
        bool seen = false;
        for (int t = walk.t0; t < end; ++t, ++mine) {
            wait(tc::smem_addr(&x->sfull[tile]), mine & 1, &x->dead, error);
            tc::fence_after();
            const int some = keys + skip - 128 * t;  // this block's keys are [lead, some)
            const int lead = t == 0 ? skip : 0;
            uint32_t v[4][32];  // the scores
#pragma unroll
            for (int n = 0; n < 4; ++n) tc::tmem_ld32(tmem + 32 * n, v[n]);
            float tops[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                tc::tmem_wait_ld(v[n]);
                if (flip)
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[n][i] ^= 0x80000000u;
                if (some < 32 * n + 32 || lead > 32 * n)
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (32 * n + i >= some || 32 * n + i < lead) v[n][i] = 0xff800000u;
                tops[n] = fmaxf(__uint_as_float(v[n][0]), __uint_as_float(v[n][1]));
#pragma unroll
                for (int i = 2; i < 32; i += 2)
                    tops[n] = tc::max3(tops[n], __uint_as_float(v[n][i]), __uint_as_float(v[n][i + 1]));
            }
            float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
            top *= c;
            float keep = 1.f;
            if (top > -INFINITY && (!seen || top > ref + 8.f)) {
                keep = tc::exp2_approx(fminf(ref - top, 126.f));
                sum *= keep;
                ref = top;
            }
            const bool scale_o = seen && keep != 1.f;
            seen = seen || top > -INFINITY;
            if (__any_sync(~0u, scale_o)) {
                if (!scale_o) keep = 1.f;
                if (t > walk.t0) {
                    wait(tc::smem_addr(&x->odone[tile]), (mine - 1) & 1, &x->dead, error);
                    tc::fence_after();
                }
#pragma unroll 1
                for (int n = 0; n < 128; n += 16) {
                    uint32_t r[16];
                    tc::tmem_ld16(tmem + 128 + n, r);
                    tc::tmem_wait_ld(r);
#pragma unroll
                    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * keep);
                    tc::tmem_st16(tmem + 128 + n, r);
                }
                tc::tmem_wait_st();
            }
            float sums[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                uint32_t e[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float p0, p1;
                    tc::fma2(p0, p1, __uint_as_float(v[n][2 * i]), __uint_as_float(v[n][2 * i + 1]), c, -ref);
                    p0 = tc::exp2_approx(p0);
                    p1 = tc::exp2_approx(p1);
                    tc::add2(sums[2 * (i & 1)], sums[2 * (i & 1) + 1], p0, p1);
                    e[i] = pack2<T>(p0, p1);
                }
                tc::tmem_st16(tmem + 16 * n, e);
                if (n & 1) {  // the product may begin with the first half
                    tc::tmem_wait_st();
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive_cluster(pfull[n >> 1]);
                }
            }
            sum += (sums[0] + sums[1]) + (sums[2] + sums[3]);
        }
        // The piece's end.
        const bool worked = end > walk.t0;
        if (worked) {
            wait(tc::smem_addr(&x->odone[tile]), (mine - 1) & 1, &x->dead, error);
            tc::fence_after();
        }
        const bool live = at < walk.r.n;
        const bool whole = walk.t0 == 0 && walk.t1 == walk.blocks;
        Partial* part = reinterpret_cast<Partial*>(ws + kOffPartial) + 2 * (blockIdx.x >> 1) + (walk.t0 == 0 ? 1 : 0);
        const int quarter = 2 * tile + (int)rank;
        const bool some = worked && (sum > 0.f || sum != sum);
        const float inv = some ? 1.f / sum : 0.f;
        T* out = static_cast<T*>(a.out) + (walk.r.q0 + at) * a.out_stride[0] + walk.head * a.out_stride[1];
#pragma unroll 1
        for (int n = 0; n < 128; n += 32) {
            uint32_t r[32];
            __syncwarp();
            tc::tmem_ld32(tmem + 128 + n, r);
            tc::tmem_wait_ld(r);
            if (!live) {
                // a thread without a query has nothing to write
            } else if (whole) {
#pragma unroll
                for (int i = 0; i < 32; i += 8) {
                    auto f = [&](int k) { return some ? __uint_as_float(r[i + k]) * inv : 0.f; };
                    *reinterpret_cast<uint4*>(out + n + i) = make_uint4(pack2<T>(f(0), f(1)), pack2<T>(f(2), f(3)),
                                                                        pack2<T>(f(4), f(5)), pack2<T>(f(6), f(7)));
                }
            } else if (worked) {
#pragma unroll
                for (int i = 0; i < 32; ++i) part->o[quarter][n + i][row] = __uint_as_float(r[i]);
            }
        }
        if (live) {
            if (!whole) {
                part->ref[quarter][row] = ref;
                part->sum[quarter][row] = worked ? sum : 0.f;
            } else if (a.lse) {
                a.lse[(walk.r.q0 + at) * a.heads + walk.head] = some ? (ref + log2f(sum)) * 0.6931471805599453f : -INFINITY;
            }
        }
        tc::fence_before();
    }
}

template <typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) hs_prefill_kernel(const __grid_constant__ Args g)
{
    extern __shared__ __align__(1024) uint8_t base[];
    const uint32_t sbase = tc::smem_addr(base);
    Aux* x = reinterpret_cast<Aux*>(base + kOffAux);
    const hs_prefill_t& a = g.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = tc::cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    int* error = reinterpret_cast<int*>(ws);

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == 0) tc::tmem_alloc<2>(tc::smem_addr(&x->tmem), 512);
    if (warp == 11) {
        // This pair's piece of the line: from where its share begins to where the next one's does.
        long long total = 0;
        for (int b = lane; b < a.batch; b += 32) total += Request(a, b).size_of_head(g.flat) * a.heads;
        for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(~0u, total, o);
        const long long share = total / pairs;
        const int extra = (int)(total - share * pairs);
        const long long lo = share * pair + min(pair, extra), hi = lo + share + (pair < extra);
        Start lo_at = {a.batch, 0, 0, 0}, hi_at = lo_at;
        long long before = 0;
        for (int b0 = 0; b0 < a.batch && before <= hi; b0 += 32) {
            const int b = b0 + lane;
            const long long per = b < a.batch ? Request(a, b).size_of_head(g.flat) : 0;
            long long incl = per * a.heads;
            for (int o = 1; o < 32; o <<= 1) {
                const long long up = __shfl_up_sync(~0u, incl, o);
                if (lane >= o) incl += up;
            }
            const long long at = before + incl - per * a.heads;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const long long pos = k ? hi : lo;
                const bool here = pos >= at && pos < at + per * a.heads;
                const unsigned who = __ballot_sync(~0u, here);
                if (!who) continue;
                Start st = {b, 0, 0, 0};
                if (here) {
                    const Request r(a, b);
                    long long off = pos - at;
                    st.h = (int)(off / per);
                    off -= st.h * per;
                    if (g.flat) {
                        for (; off >= r.blocks(st.qt) + kUnitCost; ++st.qt) off -= r.blocks(st.qt) + kUnitCost;
                        st.kb = off > kUnitCost ? (int)off - kUnitCost : 0;
                    } else {
                        st.qt = (int)off;
                    }
                }
                const int src = __ffs(who) - 1;
                st.b = __shfl_sync(~0u, st.b, src);
                st.h = __shfl_sync(~0u, st.h, src);
                st.qt = __shfl_sync(~0u, st.qt, src);
                st.kb = __shfl_sync(~0u, st.kb, src);
                (k ? hi_at : lo_at) = st;
            }
            before += __shfl_sync(~0u, incl, 31);
        }
        if (lane == 0) {
            const bool any = lo_at.b < a.batch &&
                             !(lo_at.b == hi_at.b && lo_at.h == hi_at.h && lo_at.qt == hi_at.qt && lo_at.kb == hi_at.kb);
            x->any = any;
            x->start = lo_at;
            x->stop = hi_at;
            x->dead = 0;
            if (rank == 0) reinterpret_cast<Start*>(ws + kOffStart)[pair] = any ? lo_at : Start{-1, 0, 0, 0};
            tc::mbar_init(tc::smem_addr(&x->qfull), 4);
            tc::mbar_init(tc::smem_addr(&x->qfree), 1);
            for (int k = 0; k < kStages; ++k) {
                tc::mbar_init(tc::smem_addr(&x->kfull[k]), 1);
                tc::mbar_init(tc::smem_addr(&x->kpeer[k]), 1);
                tc::mbar_init(tc::smem_addr(&x->kfree[k]), 1);
                tc::mbar_init(tc::smem_addr(&x->vfull[k]), 1);
                tc::mbar_init(tc::smem_addr(&x->vpeer[k]), 1);
                tc::mbar_init(tc::smem_addr(&x->vfree[k]), 1);
            }
            for (int k = 0; k < 2; ++k) {
                tc::mbar_init(tc::smem_addr(&x->sfull[k]), 1);
                tc::mbar_init(tc::smem_addr(&x->pfull[k][0]), 8);
                tc::mbar_init(tc::smem_addr(&x->pfull[k][1]), 8);
                tc::mbar_init(tc::smem_addr(&x->odone[k]), 1);
            }
            tc::mbar_init(tc::smem_addr(&x->spare), 1);
            tc::mbar_init_fence();
        }
    }
    tc::fence_before();
    __syncwarp();
    __syncthreads();
    tc::cluster_sync();
    tc::fence_after();
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the expansion's keys and values

    if (x->any) {
        if (warp < 8)
            soften<T>(g, x, rank, ws, error);
        else if (warp < 10)
            bring_queries<T>(g, sbase, x, rank, error);
        else if (warp == 11 && rank == 0)
            multiply<T>(g, sbase, x, error);
        else if (warp == 11 && lane == 0)
            forward(g, x, error);
        else if (warp == 10 && lane == 0)
            bring_tiles(g, sbase, x, rank, error);
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    tc::cluster_sync();
    tc::fence_after();
    if (warp == 0) tc::tmem_free<2>(x->tmem, 512);
}

// ---- (3) join ------------------------------------------------------------------------

// Block x takes the x-th unit that several pairs worked on (found at the first start
// of a piece inside it) and 128 of its queries, a thread of each group of 128 a query.
// SPLIT: 16 channels a block, four groups that take every fourth piece; else each group
// takes channels of its own and every piece.  The order of the sums is fixed.
constexpr int kJoinCols = 16;  // channels a thread
template <typename T, bool SPLIT>
__global__ void __launch_bounds__(512) hs_prefill_join_kernel(const __grid_constant__ Args g, int pairs)
{
    constexpr int kGroups = SPLIT ? 4 : 1;  // that share pieces
    __shared__ float tops[4][128], sums[4][128], cols[SPLIT ? 3 : 1][kJoinCols][128];
    __shared__ int counts[8], first_cut;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const hs_prefill_t& a = g.a;
    const uint8_t* ws = static_cast<const uint8_t*>(a.workspace);
    const Partial* parts = reinterpret_cast<const Partial*>(ws + kOffPartial);
    const Start* start = reinterpret_cast<const Start*>(ws + kOffStart);
    const int t = threadIdx.x;
    if (t == 0) first_cut = 0;
    auto same = [](const Start& p, const Start& q) { return p.b == q.b && p.h == q.h && p.qt == q.qt; };
    Start mine = {-1, 0, 0, 0};
    bool inside = false, cut = false;
    if (t > 0 && t < pairs) {
        mine = start[t];
        const Start prev = start[t - 1];
        inside = mine.b >= 0 && mine.kb > 0;
        cut = inside && !(same(mine, prev) && prev.kb > 0);
    }
    const unsigned ballot = __ballot_sync(~0u, cut);
    if (t < 256 && (t & 31) == 0) counts[t >> 5] = __popc(ballot);
    __syncthreads();
    if (cut) {
        int before = __popc(ballot & ((1u << (t & 31)) - 1));
        for (int w = 0; w < t >> 5; ++w) before += counts[w];
        if (before == (int)blockIdx.x) first_cut = t;
    }
    __syncthreads();
    if (first_cut == 0) return;
    const Start unit = start[first_cut];
    const int first = first_cut - 1, last = first + __syncthreads_count(inside && same(mine, unit));
    const Request r(a, unit.b);
    const int row = t & 127, group = SPLIT ? t >> 7 : 0;
    const int quarter = blockIdx.y, c0 = SPLIT ? kJoinCols * blockIdx.z : kJoinCols * (4 * blockIdx.z + (t >> 7));
    const int at = 512 * unit.qt + 128 * quarter + row;
    if (512 * unit.qt + 128 * quarter >= r.n) return;
    const bool live = at < r.n;
    float acc[kJoinCols] = {}, sum = 0.f, top = -INFINITY;
    if (live)
#pragma unroll 2
        for (int n = first + group; n <= last; n += kGroups) {
            const Partial& q = parts[2 * n + (n == first)];
            const float ref = q.ref[quarter][row], l = q.sum[quarter][row];
            // without a branch, so that the loads of several pieces are in flight; a sum of 0: no key counted
            float o[kJoinCols];
#pragma unroll
            for (int k = 0; k < kJoinCols; ++k) o[k] = q.o[quarter][c0 + k][row];
            const float up = l == 0.f ? top : fmaxf(top, ref), base = up == -INFINITY ? 0.f : up;
            const float keep = tc::exp2_approx(top - base), w = l == 0.f ? 0.f : tc::exp2_approx(ref - base);
            top = up;
            sum = sum * keep + w * l;
#pragma unroll
            for (int k = 0; k < kJoinCols; ++k) acc[k] = acc[k] * keep + (l == 0.f ? 0.f : w * o[k]);
        }
    if (SPLIT) {
        tops[group][row] = top;
        sums[group][row] = sum;
        if (group)
#pragma unroll
            for (int k = 0; k < kJoinCols; ++k) cols[group - 1][k][row] = acc[k];
        __syncthreads();
    }
    if (group || !live) return;
    if (SPLIT) {
        top = fmaxf(fmaxf(tops[0][row], tops[1][row]), fmaxf(tops[2][row], tops[3][row]));
        const float ref = top == -INFINITY ? 0.f : top;
        float w = tc::exp2_approx(tops[0][row] - ref);
        sum *= w;
#pragma unroll
        for (int k = 0; k < kJoinCols; ++k) acc[k] *= w;
        for (int n = 1; n < 4; ++n) {
            w = tc::exp2_approx(tops[n][row] - ref);
            sum += w * sums[n][row];
#pragma unroll
            for (int k = 0; k < kJoinCols; ++k) acc[k] += w * cols[n - 1][k][row];
        }
    }
    const bool some = sum > 0.f || sum != sum;
    const float inv = some ? 1.f / sum : 0.f;
    T* out = static_cast<T*>(a.out) + (r.q0 + at) * a.out_stride[0] + unit.h * a.out_stride[1] + c0;
#pragma unroll
    for (int k = 0; k < kJoinCols; k += 8)
        *reinterpret_cast<uint4*>(out + k) = make_uint4(pack2<T>(acc[k] * inv, acc[k + 1] * inv), pack2<T>(acc[k + 2] * inv, acc[k + 3] * inv),
                                                        pack2<T>(acc[k + 4] * inv, acc[k + 5] * inv), pack2<T>(acc[k + 6] * inv, acc[k + 7] * inv));
    if (a.lse && c0 == 0)
        a.lse[(r.q0 + at) * a.heads + unit.h] = some ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

template <typename T, bool E4M3> cudaError_t launch(const Args& g, int pairs, cudaStream_t s)
{
    const hs_prefill_t& a = g.a;
    cudaError_t e = cudaFuncSetAttribute(hs_expand_kernel<T, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, kESmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(hs_prefill_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (a.k_tokens > 0) {
        const int64_t jobs = (a.k_tokens + 255) / 256 * a.heads;
        hs_expand_kernel<T, E4M3><<<2 * (int)(jobs < pairs ? jobs : pairs), kEThreads, kESmem, s>>>(g);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    // Behind the expansion, whose start means that all earlier work is done, it may set up early.
    if (a.k_tokens > 0) {
        e = launch_after(hs_prefill_kernel<T>, dim3(2 * pairs), kThreads, kSmem, s, g);
    } else {
        hs_prefill_kernel<T><<<2 * pairs, kThreads, kSmem, s>>>(g);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) return e;
    if (pairs < 2 || !g.flat) return cudaSuccess;
    const int64_t units = (a.q_tokens / 512 + a.batch) * a.heads;  // at most
    const unsigned cut = (unsigned)(units < pairs - 1 ? units : pairs - 1);
    // A block's time is latency, so many units (of few pieces each) take few blocks: 557 against 567 us
    // for 8192 tokens with 32 heads; 512 queries over 16,384 rows 127 against 135 us with 16 heads (at most
    // 32 units are cut), 83 and 83 with 8, but 69 against 66 with 4 and 83 against 75 with one.
    if (cut >= 16) return launch_after(hs_prefill_join_kernel<T, false>, dim3(cut, 4, HS_HEAD_DIM / (4 * kJoinCols)), 512, 0, s, g, pairs);
    return launch_after(hs_prefill_join_kernel<T, true>, dim3(cut, 4, HS_HEAD_DIM / kJoinCols), 512, 0, s, g, pairs);
}

}  // namespace

size_t hs_prefill_workspace_bytes(int64_t k_tokens, int heads)
{
    const size_t blocks = (size_t)((k_tokens + 255) / 256) * 2;
    return kOffKeys + blocks * ((size_t)heads * 2 * kBlock + kRope);
}

cudaError_t hs_launch_prefill(const hs_prefill_t& a, cudaStream_t s)
{
    int dev = 0, sms = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (err != cudaSuccess) return err;
    const int pairs = sms / 2 > kMaxPairs ? kMaxPairs : sms < 2 ? 1 : sms / 2;
    const bool e = a.row_format == HS_ROWS_E4M3;
    Args g;
    g.a = a;
    g.blocks = (a.k_tokens + 255) / 256 * 2;
    // Pieces where whole units (a pair's are consecutive ones) would take longer by more than the join, which
    // takes about 9 blocks' time, were all tokens one request's; a unit of 512 queries earlier sees 4 blocks fewer.
    // 4, 16 and 64 heads, whole units against pieces: 768 tokens 29 and 31, 29 and 35, 54 and 62 us; 1024 tokens
    // 35 and 32, 37 and 39, 62 and 71; 2048 tokens 49 and 38, 57 and 59, 134 and 136.
    const int64_t tiles = a.q_tokens > 512 ? (a.q_tokens + 511) / 512 : 1, units = (tiles + a.batch - 1) * a.heads;
    const int64_t longest = ((a.q_tokens > a.k_tokens ? a.q_tokens : a.k_tokens) + 127) / 128 + kUnitCost;
    auto last = [&](int64_t n) { return n * longest - 2 * n * (n - 1); };  // a head's last n units
    const int64_t each = (units + pairs - 1) / pairs;
    g.flat = each / tiles * last(tiles) + last(each % tiles) > units * last(tiles) / (tiles * pairs) + 9;
    g.keys = static_cast<uint8_t*>(a.workspace) + kOffKeys;
    g.values = g.keys + (size_t)g.blocks * a.heads * kBlock;
    g.rope = g.values + (size_t)g.blocks * a.heads * kBlock;
    if (a.dtype == HS_TYPE_BF16)
        return e ? launch<__nv_bfloat16, true>(g, pairs, s) : launch<__nv_bfloat16, false>(g, pairs, s);
    return e ? launch<__half, true>(g, pairs, s) : launch<__half, false>(g, pairs, s);
}
