// Host side of the operators beside the swap-in path: the argument checks of
// hs_latent_attend, hs_latent_prefill and hs_rms_norm.  Every check is made
// before any CUDA call, and nothing is enqueued when one fails.
#include <cmath>

#include "hs_ops.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// A stride in elements of a 16-bit array whose rows are read in 16-byte pieces.
// Only strides that are used (more than one entry along the axis) must fit.
bool stride_ok(int64_t stride, int64_t count) { return count <= 1 || (stride >= 0 && stride % 8 == 0); }

// The same of an output: two of its rows must not lie on one another.
bool out_stride_ok(int64_t stride, int64_t count, int channels) { return stride_ok(stride, count) && (count <= 1 || stride >= channels); }

bool is_16bit(int dtype) { return dtype == HS_TYPE_BF16 || dtype == HS_TYPE_FP16; }

int row_bytes(int format)
{
    return format == HS_ROWS_16BIT ? 2 * HS_ROW_DIM : format == HS_ROWS_E4M3 ? HS_ROW8_BYTES : 0;
}

int result(cudaError_t e)
{
    if (e == cudaSuccess) return HS_OK;
    cudaGetLastError();
    return HS_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t hs_latent_attend_workspace(int batch, int positions, int heads, int64_t rows)
{
    if (batch <= 0 || positions <= 0 || heads <= 0 || rows < 0 || rows > INT32_MAX ||
        batch > HS_MAX_BATCH || positions > HS_MAX_POSITIONS || heads > HS_MAX_HEADS)
        return 0;
    return hs_attend_workspace_bytes(batch, positions, heads, rows);
}

int hs_latent_attend(const hs_attend_t* args, hs_stream_t stream)
{
    if (!args) return HS_ERR_ARG;
    const hs_attend_t& a = *args;
    if (!is_16bit(a.dtype) || !row_bytes(a.row_format)) return HS_ERR_ARG;
    if (a.batch <= 0 || a.positions <= 0 || a.heads <= 0 || a.entries < 0 || a.n_rows < 0)
        return HS_ERR_ARG;
    if (!a.q || !a.out || (!a.rows && a.n_rows > 0)) return HS_ERR_ARG;
    if ((a.slots != nullptr) == (a.lengths != nullptr)) return HS_ERR_ARG;
    if (!std::isfinite(a.scale)) return HS_ERR_ARG;
    if (a.batch > HS_MAX_BATCH || a.positions > HS_MAX_POSITIONS || a.heads > HS_MAX_HEADS ||
        a.n_rows > INT32_MAX)
        return HS_ERR_LIMIT;
    if (!aligned(a.q, 16) || !aligned(a.out, 16) || !aligned(a.rows, 16) || !aligned(a.slots, 4) ||
        !aligned(a.lengths, 4) || !aligned(a.lse, 4) || !aligned(a.workspace, 16))
        return HS_ERR_ARG;
    const int64_t n[3] = {a.batch, a.positions, a.heads};
    for (int i = 0; i < 3; ++i)
        if (!stride_ok(a.q_stride[i], n[i]) || !out_stride_ok(a.out_stride[i], n[i], HS_LATENT_DIM)) return HS_ERR_ARG;
    if (a.n_rows > 1 && (a.row_stride < row_bytes(a.row_format) || a.row_stride % 16)) return HS_ERR_ARG;
    if (a.batch > 1 && (a.request_stride < 0 || a.request_stride % 16)) return HS_ERR_ARG;
    if (a.slots && ((a.batch > 1 && a.slots_stride[0] < 0) || (a.positions > 1 && a.slots_stride[1] < 0)))
        return HS_ERR_ARG;
    const size_t need = hs_attend_workspace_bytes(a.batch, a.positions, a.heads,
                                                  a.slots ? a.entries : a.n_rows);
    if (a.workspace_bytes < need || (need > 0 && !a.workspace)) return HS_ERR_ARG;
    return result(hs_launch_attend(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t hs_latent_prefill_workspace(int64_t k_tokens, int heads)
{
    if (k_tokens < 0 || heads <= 0 || k_tokens > HS_MAX_TOKENS || heads > HS_MAX_HEADS) return 0;
    return hs_prefill_workspace_bytes(k_tokens, heads);
}

int hs_latent_prefill(const hs_prefill_t* args, hs_stream_t stream)
{
    if (!args) return HS_ERR_ARG;
    const hs_prefill_t& a = *args;
    if (!is_16bit(a.dtype) || !row_bytes(a.row_format)) return HS_ERR_ARG;
    if (a.batch <= 0 || a.heads <= 0 || a.q_tokens < 0 || a.k_tokens < 0) return HS_ERR_ARG;
    if (!a.q_start || !a.k_start || !a.w_uk || !a.w_uv) return HS_ERR_ARG;
    if (a.q_tokens > 0 && (!a.q || !a.out)) return HS_ERR_ARG;
    if (!a.rows && a.k_tokens > 0) return HS_ERR_ARG;
    if (!std::isfinite(a.scale)) return HS_ERR_ARG;
    if (a.batch > HS_MAX_BATCH || a.heads > HS_MAX_HEADS || a.q_tokens > HS_MAX_TOKENS ||
        a.k_tokens > HS_MAX_TOKENS)
        return HS_ERR_LIMIT;
    if (!aligned(a.q, 16) || !aligned(a.out, 16) || !aligned(a.rows, 16) || !aligned(a.w_uk, 16) ||
        !aligned(a.w_uv, 16) || !aligned(a.q_start, 4) || !aligned(a.k_start, 4) ||
        !aligned(a.lse, 4) || !aligned(a.workspace, 16))
        return HS_ERR_ARG;
    const int64_t n[2] = {a.q_tokens, a.heads};
    for (int i = 0; i < 2; ++i)
        if (!stride_ok(a.q_stride[i], n[i]) || !out_stride_ok(a.out_stride[i], n[i], HS_HEAD_DIM)) return HS_ERR_ARG;
    if (a.k_tokens > 1 && (a.row_stride < row_bytes(a.row_format) || a.row_stride % 16)) return HS_ERR_ARG;
    const size_t need = hs_prefill_workspace_bytes(a.k_tokens, a.heads);
    if (a.workspace_bytes < need || (need > 0 && !a.workspace)) return HS_ERR_ARG;
    if (a.q_tokens == 0) return HS_OK;
    return result(hs_launch_prefill(a, reinterpret_cast<cudaStream_t>(stream)));
}

int hs_rms_norm(const hs_norm_t* args, hs_stream_t stream)
{
    if (!args) return HS_ERR_ARG;
    const hs_norm_t& a = *args;
    if (!is_16bit(a.dtype) && a.dtype != HS_TYPE_FP32) return HS_ERR_ARG;
    if (a.dim <= 0 || a.carry < 0 || a.group < 0 || a.tokens < 0) return HS_ERR_ARG;
    if (!a.weight || (a.tokens > 0 && (!a.x || !a.out))) return HS_ERR_ARG;
    if (a.tokens > 0 && (a.residual != nullptr) != (a.residual_out != nullptr)) return HS_ERR_ARG;
    if (a.group > 0 && !a.scales && a.tokens > 0) return HS_ERR_ARG;
    if (!(a.eps >= 0.0f) || !std::isfinite(a.eps)) return HS_ERR_ARG;
    if (a.dim > HS_MAX_NORM_DIM || a.carry > HS_MAX_NORM_DIM - a.dim || a.tokens > HS_MAX_TOKENS)
        return HS_ERR_LIMIT;
    const uintptr_t el = a.dtype == HS_TYPE_FP32 ? 4 : 2;
    if (!aligned(a.x, el) || !aligned(a.residual, el) || !aligned(a.residual_out, el) ||
        !aligned(a.weight, el) || (!a.scales && !aligned(a.out, el)) || !aligned(a.scales, 4))
        return HS_ERR_ARG;
    const int64_t width = (int64_t)a.dim + a.carry;
    const int64_t groups = a.group ? (width + a.group - 1) / a.group : 1;
    if (a.tokens > 1 && (a.x_stride < 0 || a.out_stride < width ||
                         (a.residual && (a.residual_stride < 0 || a.residual_out_stride < a.dim)) ||
                         (a.scales && a.scales_stride < groups)))
        return HS_ERR_ARG;
    if (a.tokens == 0) return HS_OK;
    hs_norm_t b = a;
    b.group = hs_norm_group(a.dim, a.carry, a.group);
    return result(hs_launch_norm(b, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
