// hs_latent_prefill: expanded latent attention of ragged prompts.
//
// Two launches.  The first expands the rows: keys and values of every head
// (k_j = w_uk latent_j, v_j = w_uv latent_j) into the workspace.  The second
// is the attention: a warp per (query, head) that walks its request's keys.
#include "hs_ops.h"

namespace {

constexpr int kWarps = 8;
constexpr int kTokens = 8;  // rows a CTA of the expansion takes

// Workspace: keys [k_tokens][heads][128], then values [k_tokens][heads][128].
template <typename T, bool E4M3>
__global__ void __launch_bounds__(2 * HS_HEAD_DIM) hs_expand_kernel(hs_prefill_t a)
{
    __shared__ float lat[kTokens][HS_LATENT_DIM];
    const int64_t t0 = (int64_t)blockIdx.x * kTokens;
    const int head = blockIdx.y;
    for (int i = threadIdx.x; i < kTokens * HS_LATENT_DIM; i += blockDim.x) {
        const int t = i / HS_LATENT_DIM, c = i % HS_LATENT_DIM;
        float v = 0.f;
        if (t0 + t < a.k_tokens) {
            const uint8_t* row = static_cast<const uint8_t*>(a.rows) + (t0 + t) * a.row_stride;
            v = E4M3 ? hs_e4m3_to_float(row[c]) * *reinterpret_cast<const float*>(row + HS_ROW8_SCALE)
                     : HsType<T>::to_float(reinterpret_cast<const T*>(row)[c]);
        }
        lat[t][c] = v;
    }
    __syncthreads();
    const int d = threadIdx.x % HS_HEAD_DIM;
    const bool value = threadIdx.x >= HS_HEAD_DIM;
    const T* w = static_cast<const T*>(value ? a.w_uv : a.w_uk) + ((int64_t)head * HS_HEAD_DIM + d) * HS_LATENT_DIM;
    float acc[kTokens] = {};
    for (int c = 0; c < HS_LATENT_DIM; ++c) {
        const float wv = HsType<T>::to_float(w[c]);
        for (int t = 0; t < kTokens; ++t) acc[t] += wv * lat[t][c];
    }
    T* dst = static_cast<T*>(a.workspace) + (value ? a.k_tokens * a.heads * HS_HEAD_DIM : 0);
    for (int t = 0; t < kTokens; ++t)
        if (t0 + t < a.k_tokens)
            dst[((t0 + t) * a.heads + head) * HS_HEAD_DIM + d] = HsType<T>::from_float(acc[t]);
}

template <typename T, bool E4M3>
__global__ void __launch_bounds__(kWarps * 32) hs_prefill_kernel(hs_prefill_t a)
{
    const int lane = threadIdx.x & 31;
    const int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int head = blockIdx.y;
    int r = 0;  // the request of query i: the last with q_start[r] <= i
    int64_t q0 = 0, q1 = 0;
    for (; r < a.batch; ++r) {
        q0 = a.q_start[r];
        q1 = a.q_start[r + 1];
        if (i >= q0 && i < q1) break;
    }
    if (r == a.batch || i >= a.q_tokens) return;
    int64_t k0 = a.k_start[r], k1 = a.k_start[r + 1];
    k0 = k0 < 0 ? 0 : k0;
    k1 = k1 > a.k_tokens ? a.k_tokens : k1;
    q1 = q1 > a.q_tokens ? a.q_tokens : q1;
    const int64_t n = (i - q0) + (k1 - k0) - (q1 - q0) + 1;
    const T* q = static_cast<const T*>(a.q) + i * a.q_stride[0] + head * a.q_stride[1];
    float qr[6], acc[4] = {};
    for (int j = 0; j < 6; ++j) qr[j] = HsType<T>::to_float(q[lane + 32 * j]);
    float m = -INFINITY, l = 0.f;
    for (int64_t t = k0; t < k0 + n; ++t) {
        const T* k = static_cast<const T*>(a.workspace) + (t * a.heads + head) * HS_HEAD_DIM;
        const T* v = k + a.k_tokens * a.heads * HS_HEAD_DIM;
        const uint8_t* row = static_cast<const uint8_t*>(a.rows) + t * a.row_stride;
        float s = 0.f, w = 1.f;
        if (E4M3) w = *reinterpret_cast<const float*>(row + HS_ROW8_SCALE);
        for (int j = 0; j < 4; ++j) s += qr[j] * HsType<T>::to_float(k[lane + 32 * j]);
        for (int j = 0; j < 2; ++j) {
            const int c = HS_LATENT_DIM + lane + 32 * j;
            s += qr[4 + j] * (E4M3 ? hs_e4m3_to_float(row[c]) * w
                                   : HsType<T>::to_float(reinterpret_cast<const T*>(row)[c]));
        }
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
        s *= a.scale;
        const float top = fmaxf(m, s);
        const float keep = m == -INFINITY ? 0.f : __expf(m - top);
        const float p = __expf(s - top);
        l = l * keep + p;
        for (int j = 0; j < 4; ++j) acc[j] = acc[j] * keep + p * HsType<T>::to_float(v[lane + 32 * j]);
        m = top;
    }
    T* out = static_cast<T*>(a.out) + i * a.out_stride[0] + head * a.out_stride[1];
    for (int j = 0; j < 4; ++j) out[lane + 32 * j] = HsType<T>::from_float(n > 0 ? acc[j] / l : 0.f);
    if (a.lse && lane == 0) a.lse[i * a.heads + head] = n > 0 ? m + __logf(l) : -INFINITY;
}

template <typename T, bool E4M3>
cudaError_t launch(const hs_prefill_t& a, cudaStream_t s)
{
    if (a.k_tokens > 0) {
        const dim3 grid((unsigned)((a.k_tokens + kTokens - 1) / kTokens), a.heads);
        hs_expand_kernel<T, E4M3><<<grid, 2 * HS_HEAD_DIM, 0, s>>>(a);
    }
    const dim3 grid((unsigned)((a.q_tokens + kWarps - 1) / kWarps), a.heads);
    hs_prefill_kernel<T, E4M3><<<grid, kWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t hs_prefill_workspace_bytes(int64_t k_tokens, int heads)
{
    return 256 + (size_t)k_tokens * heads * 2 * HS_HEAD_DIM * 2;
}

cudaError_t hs_launch_prefill(const hs_prefill_t& a, cudaStream_t s)
{
    const bool e = a.row_format == HS_ROWS_E4M3;
    if (a.dtype == HS_TYPE_BF16)
        return e ? launch<__nv_bfloat16, true>(a, s) : launch<__nv_bfloat16, false>(a, s);
    return e ? launch<__half, true>(a, s) : launch<__half, false>(a, s);
}
