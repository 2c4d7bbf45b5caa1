// hs_latent_attend: absorbed latent attention over listed or leading rows.
//
// One warp per (request, position, head); it keeps the query (18 channels a
// lane), the running maximum and sum and the 16 output channels of each lane
// in registers, and walks the rows once.
#include "hs_ops.h"

namespace {

constexpr int kWarps = 8;

template <typename T, bool E4M3>
__global__ void __launch_bounds__(kWarps * 32) hs_attend_kernel(hs_attend_t a)
{
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (unit >= (int64_t)a.batch * a.positions * a.heads) return;
    const int head = (int)(unit % a.heads);
    const int pos = (int)(unit / a.heads % a.positions);
    const int64_t b = unit / a.heads / a.positions;
    const T* q = static_cast<const T*>(a.q) + b * a.q_stride[0] + pos * a.q_stride[1] + head * a.q_stride[2];
    const uint8_t* rows = static_cast<const uint8_t*>(a.rows) + b * a.request_stride;
    float qr[18], acc[16];
    for (int i = 0; i < 18; ++i) qr[i] = HsType<T>::to_float(q[lane + 32 * i]);
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
    float m = -INFINITY, l = 0.f;
    const int32_t* slots = a.slots ? a.slots + b * a.slots_stride[0] + pos * a.slots_stride[1] : nullptr;
    int64_t n = a.entries;
    if (!slots) {
        int64_t len = a.lengths[b];
        len = len < 0 ? 0 : len > a.n_rows ? a.n_rows : len;
        n = len - a.positions + 1 + pos;
    }
    for (int64_t i = 0; i < n; ++i) {
        const int64_t slot = slots ? slots[i] : i;
        if (slot < 0 || slot >= a.n_rows) continue;
        const uint8_t* row = rows + slot * a.row_stride;
        float v[18], s = 0.f;
        for (int j = 0; j < 18; ++j) {
            v[j] = E4M3 ? hs_e4m3_to_float(row[lane + 32 * j])
                        : HsType<T>::to_float(reinterpret_cast<const T*>(row)[lane + 32 * j]);
            s += qr[j] * v[j];
        }
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
        float w = 1.f;
        if (E4M3) w = *reinterpret_cast<const float*>(row + HS_ROW8_SCALE);
        s *= a.scale * w;
        const float top = fmaxf(m, s);
        const float keep = m == -INFINITY ? 0.f : __expf(m - top);
        const float p = __expf(s - top);
        l = l * keep + p;
        for (int j = 0; j < 16; ++j) acc[j] = acc[j] * keep + p * w * v[j];
        m = top;
    }
    T* out = static_cast<T*>(a.out) + b * a.out_stride[0] + pos * a.out_stride[1] + head * a.out_stride[2];
    for (int j = 0; j < 16; ++j) out[lane + 32 * j] = HsType<T>::from_float(l > 0.f || l != l ? acc[j] / l : 0.f);
    if (a.lse && lane == 0) a.lse[unit] = l > 0.f || l != l ? m + __logf(l) : -INFINITY;
}

template <typename T>
cudaError_t launch(const hs_attend_t& a, cudaStream_t s)
{
    const int64_t units = (int64_t)a.batch * a.positions * a.heads;
    auto k = a.row_format == HS_ROWS_E4M3 ? hs_attend_kernel<T, true> : hs_attend_kernel<T, false>;
    k<<<(unsigned)((units + kWarps - 1) / kWarps), kWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t hs_attend_workspace_bytes(int, int, int, int64_t) { return 256; }

cudaError_t hs_launch_attend(const hs_attend_t& a, cudaStream_t s)
{
    return a.dtype == HS_TYPE_BF16 ? launch<__nv_bfloat16>(a, s) : launch<__half>(a, s);
}
