// C-ABI entry points of the context operators: argument checks and argument
// packing.  The kernels are in attention_fwd.hip,
// attention_bwd.hip and norm.hip.
#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <cstring>

#include "context.h"

namespace sn {
namespace {

bool aligned_for(const void *p, int dtype) {
    return (reinterpret_cast<uintptr_t>(p) & (dtype == SN_F32 ? 3 : 1)) == 0;
}

sn_status check_ctx_ws(const void *ws, size_t ws_bytes, size_t need) {
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255) != 0 || ws_bytes < need) return SN_ERR_WORKSPACE;
    return SN_OK;
}

sn_status check_attn_sizes(const sn_cross_attention *op) {
    if (!op || op->n_segments < 1 || op->n_q < 0 || op->n_k < 0) return SN_ERR_INVALID;
    if (op->max_q < 0 || op->max_q > op->n_q || op->max_k < 0 || op->max_k > op->n_k) return SN_ERR_INVALID;
    // the longest segment bounds the sum of all
    if ((int64_t)op->max_q * op->n_segments < op->n_q || (int64_t)op->max_k * op->n_segments < op->n_k)
        return SN_ERR_INVALID;
    if (op->n_heads < 1 || op->n_kv_heads < 1 || op->n_heads % op->n_kv_heads != 0) return SN_ERR_INVALID;
    if (op->n_heads > 65535) return SN_ERR_INVALID;
    if (op->head_dim < 1 || op->head_dim > SN_MAX_HEAD_DIM) return SN_ERR_INVALID;
    if (op->dtype != SN_F32 && op->dtype != SN_BF16) return SN_ERR_INVALID;
    // rows are counted with their heads in 32-bit block and row indices
    if ((int64_t)op->n_q * op->n_heads > INT32_MAX || (int64_t)op->n_k * op->n_kv_heads > INT32_MAX)
        return SN_ERR_INVALID;
    if (op->bias && (op->n_buckets < 1 || op->n_buckets > SN_MAX_BUCKETS)) return SN_ERR_INVALID;
    // the launches hold the longest segment's tiles for every segment
    if (!attn_forward_fits(*op) || !attn_backward_fits(*op)) return SN_ERR_INVALID;
    return SN_OK;
}

sn_status check_attn(const sn_cross_attention *op) {
    SN_TRY(check_attn_sizes(op));
    if (!op->q_ptr || !op->k_ptr || !std::isfinite(op->scale)) return SN_ERR_INVALID;
    if ((op->n_q > 0 && !op->q) || (op->n_k > 0 && (!op->k || !op->v))) return SN_ERR_INVALID;
    if (!aligned_for(op->q, op->dtype) || !aligned_for(op->k, op->dtype) || !aligned_for(op->v, op->dtype))
        return SN_ERR_INVALID;
    if (op->bias && op->n_buckets > 1) {
        if (!op->thresholds) return SN_ERR_INVALID;
        for (int i = 1; i < op->n_buckets - 1; ++i)
            if (op->thresholds[i] < op->thresholds[i - 1]) return SN_ERR_INVALID;
        if ((int64_t)op->thresholds[op->n_buckets - 2] - op->thresholds[0] > SN_MAX_BUCKET_SPAN) return SN_ERR_INVALID;
    }
    return SN_OK;
}

size_t attn_workspace(const sn_cross_attention &op) {
    return std::max(attn_forward_workspace(op), attn_backward_workspace(op));
}

// Whether a tensor's rows can be read 16 bytes at a time, and 64 of them
// from one base with 31-bit byte offsets.
bool rows_fast(const sn_cross_attention &op, const void *p, int64_t stride, int64_t head_stride) {
    const int64_t per = op.dtype == SN_F32 ? 4 : 8;
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride % per == 0 && head_stride % per == 0 &&
           op.head_dim % 8 == 0 && stride >= 0 && stride < (1ll << 24) / (op.dtype == SN_F32 ? 4 : 2);
}

// Whether a contiguous output's rows can be written four elements at a time.
bool rows_of_four(const sn_cross_attention &op, const void *p, int dtype) {
    return op.head_dim % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & (dtype == SN_F32 ? 15 : 7)) == 0;
}

AttnArgs attn_args(const sn_cross_attention &op, void *ws) {
    AttnArgs a{};
    a.B = op.n_segments;
    a.n_q = op.n_q; a.n_k = op.n_k;
    a.max_q = op.max_q; a.max_k = op.max_k;
    a.q_ptr = op.q_ptr; a.k_ptr = op.k_ptr;
    a.H = op.n_heads; a.Hkv = op.n_kv_heads; a.G = op.n_heads / op.n_kv_heads; a.D = op.head_dim;
    a.scale = op.scale;
    a.q = op.q; a.k = op.k; a.v = op.v;
    a.qs = op.q_stride; a.qh = op.q_head_stride;
    a.ks = op.k_stride; a.kh = op.k_head_stride;
    a.vs = op.v_stride; a.vh = op.v_head_stride;
    a.keep = op.keep;
    a.bias = op.bias;
    a.nb = op.bias ? op.n_buckets : 0;
    a.q_pos = op.q_pos; a.k_pos = op.k_pos;
    a.status = reinterpret_cast<int *>(ws);
    for (int i = 0; i < SN_MAX_BUCKETS; ++i) a.thr[i] = i + 1 < a.nb ? op.thresholds[i] : INT32_MAX;
    if (a.nb > 1) {   // from one below the first threshold (if there is one below) to the last
        a.lut_base = a.thr[0] == INT32_MIN ? INT32_MIN : a.thr[0] - 1;
        a.lut_n = (int)((int64_t)a.thr[a.nb - 2] - a.lut_base + 1);
    } else {
        a.lut_n = a.nb;
    }
    a.lut_run = std::abs((int64_t)a.lut_base) < (1 << 30);
    a.fast = rows_fast(op, op.q, op.q_stride, op.q_head_stride) && rows_fast(op, op.k, op.k_stride, op.k_head_stride) &&
             rows_fast(op, op.v, op.v_stride, op.v_head_stride);
    return a;
}

sn_status check_norm_sizes(const sn_group_norm *op) {
    if (!op || op->n_segments < 1 || op->n_rows < 0) return SN_ERR_INVALID;
    if (op->max_rows < 0 || op->max_rows > op->n_rows || (int64_t)op->max_rows * op->n_segments < op->n_rows)
        return SN_ERR_INVALID;
    if (op->n_channels < 1 || op->n_channels > 65536 || op->n_groups < 1 || op->n_channels % op->n_groups != 0)
        return SN_ERR_INVALID;
    if (op->dtype != SN_F32 && op->dtype != SN_BF16) return SN_ERR_INVALID;
    if (op->activation < SN_ACT_NONE || op->activation > SN_ACT_SILU) return SN_ERR_INVALID;
    return SN_OK;
}

sn_status check_norm(const sn_group_norm *op) {
    SN_TRY(check_norm_sizes(op));
    if (!op->row_ptr || !(op->eps > 0.0f) || !std::isfinite(op->eps)) return SN_ERR_INVALID;
    if ((op->n_rows > 0 && !op->x) || !aligned_for(op->x, op->dtype)) return SN_ERR_INVALID;
    return SN_OK;
}

sn_status attn_forward_checked(const sn_cross_attention *op, void *o, float *rows, float *lse, void *ws, size_t ws_bytes,
                               void *stream) {
    SN_TRY(check_attn(op));
    SN_TRY(check_ctx_ws(ws, ws_bytes, attn_workspace(*op)));
    if (op->n_q == 0) return SN_OK;
    if (!o || !aligned_for(o, op->dtype)) return SN_ERR_INVALID;
    AttnArgs a = attn_args(*op, ws);
    a.out4 = rows_of_four(*op, o, op->dtype) && rows_of_four(*op, rows, SN_F32);
    return attn_forward(a, op->dtype, o, rows, lse, static_cast<char *>(ws), reinterpret_cast<hipStream_t>(stream));
}

NormArgs norm_args(const sn_group_norm &op, void *ws) {
    NormArgs a{};
    a.B = op.n_segments; a.n_rows = op.n_rows; a.max_rows = op.max_rows;
    a.C = op.n_channels; a.groups = op.n_groups; a.width = op.n_channels / op.n_groups;
    a.act = op.activation; a.eps = op.eps;
    a.ptr = op.row_ptr; a.x = op.x; a.xs = op.x_stride;
    a.gamma = op.gamma; a.beta = op.beta;
    a.status = reinterpret_cast<int *>(ws);
    return a;
}

}  // namespace
}  // namespace sn

using namespace sn;

extern "C" {

sn_status sn_relative_thresholds(int32_t n_buckets, int32_t max_distance, int32_t *thresholds) {
    if (n_buckets < 4 || n_buckets > SN_MAX_BUCKETS || (n_buckets & 1) || !thresholds) return SN_ERR_INVALID;
    const int half = n_buckets / 2, near = half / 2, wide = half - near;
    if (max_distance <= near || max_distance > SN_MAX_BUCKET_SPAN / 2) return SN_ERR_INVALID;
    for (int j = 1; j < half; ++j) {   // smallest distance of bucket j of a half
        int first = j;
        if (j >= near)   // near (max/near)^((j - near)/wide), up to the next whole number
            first = (int)std::ceil(near * std::pow((double)max_distance / near, (double)(j - near) / wide) - 1e-9);
        thresholds[half - 1 - j] = 1 - first;   // -rel >= first  <=>  rel < 1 - first
        thresholds[half - 1 + j] = 1 + first;   // rel - 1 >= first
    }
    thresholds[half - 1] = 1;
    return SN_OK;
}

size_t sn_cross_attention_workspace_bytes(const sn_cross_attention *op) {
    return check_attn_sizes(op) == SN_OK ? attn_workspace(*op) : 0;
}

sn_status sn_cross_attention_forward(const sn_cross_attention *op, void *o, float *lse, void *ws, size_t ws_bytes,
                                     void *stream) {
    return attn_forward_checked(op, o, nullptr, lse, ws, ws_bytes, stream);
}

sn_status sn_cross_attention_forward_train(const sn_cross_attention *op, void *o, float *rows, float *lse, void *ws,
                                           size_t ws_bytes, void *stream) {
    SN_TRY(check_attn(op));
    if (op->n_q > 0 && (!lse || (op->dtype == SN_BF16 && !rows) || !aligned_for(rows, SN_F32))) return SN_ERR_INVALID;
    return attn_forward_checked(op, o, rows, lse, ws, ws_bytes, stream);
}

sn_status sn_cross_attention_backward(const sn_cross_attention *op, const float *rows, const float *lse, const void *d_o,
                                      int64_t d_o_stride, int64_t d_o_head_stride, void *dq, void *dk, void *dv,
                                      float *dbias, void *ws, size_t ws_bytes, void *stream) {
    SN_TRY(check_attn(op));
    SN_TRY(check_ctx_ws(ws, ws_bytes, attn_workspace(*op)));
    if (op->n_q > 0 && (!rows || !lse || !d_o || !dq)) return SN_ERR_INVALID;
    if (op->n_k > 0 && (!dk || !dv)) return SN_ERR_INVALID;
    if (op->bias && !dbias) return SN_ERR_INVALID;
    if (!aligned_for(rows, SN_F32) || !aligned_for(d_o, op->dtype) || !aligned_for(dq, op->dtype) ||
        !aligned_for(dk, op->dtype) || !aligned_for(dv, op->dtype))
        return SN_ERR_INVALID;
    AttnArgs a = attn_args(*op, ws);
    a.d_o = d_o;
    a.gs = d_o_stride;
    a.gh = d_o_head_stride;
    a.out4 = rows_of_four(*op, dq, op->dtype) && rows_of_four(*op, dk, op->dtype) && rows_of_four(*op, dv, op->dtype);
    a.fast = a.fast && rows_fast(*op, d_o, d_o_stride, d_o_head_stride) && (reinterpret_cast<uintptr_t>(rows) & 15) == 0;
    return attn_backward(a, op->dtype, rows, lse, dq, dk, dv, op->bias ? dbias : nullptr, static_cast<char *>(ws),
                         reinterpret_cast<hipStream_t>(stream));
}

size_t sn_group_norm_workspace_bytes(const sn_group_norm *op) {
    return check_norm_sizes(op) == SN_OK && norm_fits(*op) ? norm_workspace(*op) : 0;
}

sn_status sn_group_norm_forward(const sn_group_norm *op, void *y, float *mean, float *rstd, void *ws, size_t ws_bytes,
                                void *stream) {
    SN_TRY(check_norm(op));
    SN_TRY(check_ctx_ws(ws, ws_bytes, norm_workspace(*op)));
    if (op->n_rows > 0 && (!y || !aligned_for(y, op->dtype))) return SN_ERR_INVALID;
    return norm_forward(norm_args(*op, ws), op->dtype, y, mean, rstd, static_cast<char *>(ws),
                        reinterpret_cast<hipStream_t>(stream));
}

sn_status sn_group_norm_backward(const sn_group_norm *op, const float *mean, const float *rstd, const void *dy,
                                 int64_t dy_stride, void *dx, float *dgamma, float *dbeta, void *ws, size_t ws_bytes,
                                 void *stream) {
    SN_TRY(check_norm(op));
    SN_TRY(check_ctx_ws(ws, ws_bytes, norm_workspace(*op)));
    if (!mean || !rstd) return SN_ERR_INVALID;
    if (op->n_rows > 0 && (!dy || !dx || !aligned_for(dy, op->dtype) || !aligned_for(dx, op->dtype)))
        return SN_ERR_INVALID;
    NormArgs a = norm_args(*op, ws);
    a.dy = dy;
    a.dys = dy_stride;
    return norm_backward(a, op->dtype, mean, rstd, dx, dgamma, dbeta, static_cast<char *>(ws),
                         reinterpret_cast<hipStream_t>(stream));
}

}  // extern "C"
