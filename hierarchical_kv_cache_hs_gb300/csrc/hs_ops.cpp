// Host side of the operators beside the swap-in path: the argument checks of
// hs_latent_attend, hs_latent_attend_shared, hs_latent_prefill, hs_rms_norm,
// hs_latent_write, hs_latent_read and hs_norm_rotate.  Every check is made before any
// CUDA call, and nothing is enqueued when one fails.
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

// The arguments of hs_latent_attend but for its workspace.
int check_attend(const hs_attend_t& a)
{
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
    return HS_OK;
}

// A row array that is read or written in 16-byte pieces.
int check_rows(const void* rows, int64_t n_rows, int64_t row_stride, int64_t request_stride, int format, int batch)
{
    if (n_rows < 0 || (!rows && n_rows > 0) || !aligned(rows, 16)) return HS_ERR_ARG;
    if (n_rows > 1 && (row_stride < row_bytes(format) || row_stride % 16)) return HS_ERR_ARG;
    if (batch > 1 && (request_stride < 0 || request_stride % 16)) return HS_ERR_ARG;
    return n_rows > INT32_MAX ? HS_ERR_LIMIT : HS_OK;
}

// An output of [n0][n1] rows of `channels` (strides in the same unit): one axis inside the other, and no two rows on one another.
bool apart(const int64_t* stride, int64_t n0, int64_t n1, int channels)
{
    if (n0 <= 1 || n1 <= 1) return (n0 <= 1 || stride[0] >= channels) && (n1 <= 1 || stride[1] >= channels);
    const bool first_inside = stride[0] < stride[1];
    const int64_t in = stride[first_inside ? 0 : 1], out = stride[first_inside ? 1 : 0], n = first_inside ? n0 : n1;
    return in >= channels && out >= channels && (out - channels) / (n - 1) >= in;
}

int check_rotation(int rotation, int rope, const int32_t* positions, const float* inv_freq)
{
    if (rotation < HS_ROTATE_NONE || rotation > HS_ROTATE_HALVES) return HS_ERR_ARG;
    if (rotation != HS_ROTATE_NONE && (rope <= 0 || rope % 2 || !positions || !inv_freq)) return HS_ERR_ARG;
    return aligned(positions, 4) && aligned(inv_freq, 4) ? HS_OK : HS_ERR_ARG;
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
    if (const int rc = check_attend(a)) return rc;
    const size_t need = hs_attend_workspace_bytes(a.batch, a.positions, a.heads,
                                                  a.slots ? a.entries : a.n_rows);
    if (a.workspace_bytes < need || (need > 0 && !a.workspace)) return HS_ERR_ARG;
    return result(hs_launch_attend(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t hs_latent_attend_shared_workspace(int batch, int positions, int heads, int64_t rows, int64_t prefix_rows, int row_format)
{
    if (!hs_latent_attend_workspace(batch, positions, heads, rows) || (int64_t)batch * positions * heads > INT32_MAX ||
        prefix_rows < 0 || prefix_rows > INT32_MAX || !row_bytes(row_format))
        return 0;
    return hs_attend_shared_workspace_bytes(batch, positions, heads, rows, prefix_rows);
}

int hs_latent_attend_shared(const hs_attend_t* args, const hs_prefix_t* prefix, hs_stream_t stream)
{
    if (!args || !prefix) return HS_ERR_ARG;
    const hs_attend_t& a = *args;
    const hs_prefix_t& p = *prefix;
    if (const int rc = check_attend(a)) return rc;
    if (p.n_rows < 0 || (!p.rows && p.n_rows > 0)) return HS_ERR_ARG;
    if (p.n_rows > INT32_MAX || (int64_t)a.batch * a.positions * a.heads > INT32_MAX || (p.n_rows > 1 && p.row_stride >= (int64_t)1 << 40))
        return HS_ERR_LIMIT;
    if (!aligned(p.rows, 16) || !aligned(p.lengths, 4)) return HS_ERR_ARG;
    if (p.n_rows > 1 && (p.row_stride < row_bytes(a.row_format) || p.row_stride % 16)) return HS_ERR_ARG;
    const size_t need = hs_attend_shared_workspace_bytes(a.batch, a.positions, a.heads, a.slots ? a.entries : a.n_rows, p.n_rows);
    if (a.workspace_bytes < need || !a.workspace) return HS_ERR_ARG;
    return result(hs_launch_attend_shared(a, p, reinterpret_cast<cudaStream_t>(stream)));
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

int hs_latent_write(const hs_write_t* args, hs_stream_t stream)
{
    if (!args) return HS_ERR_ARG;
    const hs_write_t& a = *args;
    if (!is_16bit(a.dtype) || !row_bytes(a.row_format)) return HS_ERR_ARG;
    if (a.tokens < 0 || (a.start && (a.batch <= 0 || !a.lengths))) return HS_ERR_ARG;
    if (a.tokens > HS_MAX_TOKENS || (a.start && a.batch > HS_MAX_BATCH)) return HS_ERR_LIMIT;
    if (a.tokens == 0) return HS_OK;
    if (!a.x || !aligned(a.x, 16) || !aligned(a.weight, 16) || !aligned(a.start, 4) || !aligned(a.lengths, 4)) return HS_ERR_ARG;
    if (!stride_ok(a.x_stride, a.tokens)) return HS_ERR_ARG;
    if (!(a.eps >= 0.0f) || !std::isfinite(a.eps)) return HS_ERR_ARG;
    if (const int rc = check_rotation(a.rotation, HS_ROPE_DIM, a.positions, a.inv_freq)) return rc;
    const int batch = a.start ? a.batch : 1;
    if (const int rc = check_rows(a.rows, a.n_rows, a.row_stride, a.request_stride, a.row_format, batch)) return rc;
    if (!a.start && a.n_rows < a.tokens) return HS_ERR_ARG;
    // rows of two requests on one another would be written twice
    const int64_t strides[2] = {a.request_stride, a.row_stride};
    if (a.n_rows > 0 && !apart(strides, batch, a.n_rows, row_bytes(a.row_format))) return HS_ERR_ARG;
    return result(hs_launch_write(a, reinterpret_cast<cudaStream_t>(stream)));
}

int hs_latent_read(const hs_read_t* args, hs_stream_t stream)
{
    if (!args) return HS_ERR_ARG;
    const hs_read_t& a = *args;
    if (!is_16bit(a.dtype) || !row_bytes(a.row_format) || (!is_16bit(a.out_dtype) && a.out_dtype != HS_TYPE_FP32)) return HS_ERR_ARG;
    if ((a.slots != nullptr) == (a.start != nullptr) || a.batch <= 0 || a.tokens < 0) return HS_ERR_ARG;
    if (a.slots && (a.entries < 0 || a.tokens != (int64_t)a.batch * a.entries)) return HS_ERR_ARG;
    if (a.tokens > HS_MAX_TOKENS || a.batch > HS_MAX_BATCH) return HS_ERR_LIMIT;
    if (a.tokens == 0) return HS_OK;
    if (!a.out || !aligned(a.out, 16) || !aligned(a.slots, 4) || !aligned(a.start, 4) || !aligned(a.lengths, 4)) return HS_ERR_ARG;
    if (a.slots && a.batch > 1 && a.slots_stride < 0) return HS_ERR_ARG;
    const int pieces = a.out_dtype == HS_TYPE_FP32 ? 4 : 8;  // of 16 bytes
    if (a.tokens > 1 && (a.out_stride < HS_ROW_DIM || a.out_stride % pieces)) return HS_ERR_ARG;
    if (const int rc = check_rows(a.rows, a.n_rows, a.row_stride, a.request_stride, a.row_format, a.batch)) return rc;
    return result(hs_launch_read(a, reinterpret_cast<cudaStream_t>(stream)));
}

int hs_norm_rotate(const hs_rotate_t* args, hs_stream_t stream)
{
    if (!args) return HS_ERR_ARG;
    const hs_rotate_t& a = *args;
    if (!is_16bit(a.dtype) && a.dtype != HS_TYPE_FP32) return HS_ERR_ARG;
    if (a.dim <= 0 || a.tokens < 0 || a.heads[0] <= 0 || a.heads[1] < 0) return HS_ERR_ARG;
    if (a.rope < 0 || a.rope_at < 0 || (a.rotation == HS_ROTATE_NONE && a.rope)) return HS_ERR_ARG;
    if (!(a.eps >= 0.0f) || !std::isfinite(a.eps)) return HS_ERR_ARG;
    if (a.dim > HS_MAX_HEAD_CHANNELS || a.heads[0] > HS_MAX_HEADS || a.heads[1] > HS_MAX_HEADS || a.tokens > HS_MAX_TOKENS)
        return HS_ERR_LIMIT;
    if (a.rope > a.dim || a.rope_at > a.dim - a.rope) return HS_ERR_ARG;
    if (a.tokens == 0) return HS_OK;  // arrays of no tokens have no address, the keys' neither
    if ((a.x[1] != nullptr) != (a.heads[1] > 0)) return HS_ERR_ARG;
    if (const int rc = check_rotation(a.rotation, a.rope, a.positions, a.inv_freq)) return rc;
    const uintptr_t el = a.dtype == HS_TYPE_FP32 ? 4 : 2;
    for (int k = 0; k < 2; ++k) {
        if (!a.heads[k]) continue;
        if (!a.x[k] || !a.out[k] || !aligned(a.x[k], el) || !aligned(a.out[k], el) || !aligned(a.weight[k], el)) return HS_ERR_ARG;
        if ((a.tokens > 1 && a.x_stride[k][0] < 0) || (a.heads[k] > 1 && a.x_stride[k][1] < 0)) return HS_ERR_ARG;
        if (!apart(a.out_stride[k], a.tokens, a.heads[k], a.dim)) return HS_ERR_ARG;
    }
    return result(hs_launch_rotate(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
