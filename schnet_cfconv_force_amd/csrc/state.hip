// C-ABI entry points of the rotation of heads and of the state cache:
// argument checks and argument packing.  The kernels are in rotary.hip,
// cache.hip and cache_attend.hip.
#include <cfloat>
#include <cmath>

#include "state.h"

namespace sn {
namespace {

bool aligned_for(const void *p, int dtype) {
    return (reinterpret_cast<uintptr_t>(p) & (dtype == SN_F32 ? 3 : 1)) == 0;
}

sn_status check_ws(const void *ws, size_t ws_bytes, size_t need) {
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255) != 0 || ws_bytes < need) return SN_ERR_WORKSPACE;
    return SN_OK;
}

// --------------------------------------------------------------- rotation of heads

sn_status check_rotary_sizes(const sn_head_rotary *op) {
    if (!op || op->n_rows < 0 || op->n_heads < 1 || op->n_kv_heads < 0) return SN_ERR_INVALID;
    if (op->n_heads > 65535 || op->n_kv_heads > 65535) return SN_ERR_INVALID;
    if (op->head_dim < 1 || op->head_dim > SN_MAX_HEAD_DIM) return SN_ERR_INVALID;
    if (op->dtype != SN_F32 && op->dtype != SN_BF16) return SN_ERR_INVALID;
    if ((op->norm & ~1) != 0 || (op->interleaved & ~1) != 0) return SN_ERR_INVALID;
    if (op->n_pairs < 0 || op->n_pairs > op->head_dim / 2) return SN_ERR_INVALID;
    if (op->n_pairs > 0 && (op->n_axes < 1 || op->n_axes > SN_MAX_AXES)) return SN_ERR_INVALID;
    return rotary_fits(*op) ? SN_OK : SN_ERR_INVALID;
}

sn_status check_rotary(const sn_head_rotary *op) {
    SN_TRY(check_rotary_sizes(op));
    // a normal number: the reciprocal root of a smaller one is none
    if (op->norm && !(op->eps >= FLT_MIN && std::isfinite(op->eps))) return SN_ERR_INVALID;
    if (!op->norm && (op->q_weight || op->k_weight)) return SN_ERR_INVALID;
    if (op->n_pairs > 0) {
        if (!op->freqs || !op->axes || (op->n_rows > 0 && !op->positions) || !aligned_for(op->positions, SN_F32))
            return SN_ERR_INVALID;
        for (int j = 0; j < op->n_pairs; ++j)
            if (!(std::fabs(op->freqs[j]) < kMaxFrequency) || op->axes[j] < 0 || op->axes[j] >= op->n_axes) return SN_ERR_INVALID;
    }
    if (op->n_rows > 0 && (!op->q || (op->n_kv_heads > 0 && !op->k))) return SN_ERR_INVALID;
    if (!aligned_for(op->q, op->dtype) || !aligned_for(op->k, op->dtype) || !aligned_for(op->q_weight, SN_F32) ||
        !aligned_for(op->k_weight, SN_F32))
        return SN_ERR_INVALID;
    return SN_OK;
}

RotaryArgs rotary_args(const sn_head_rotary &op, void *q_out, void *k_out) {
    RotaryArgs a{};
    a.n_rows = op.n_rows; a.D = op.head_dim; a.P = op.n_pairs; a.interleaved = op.interleaved;
    a.H = op.n_heads; a.Hkv = op.n_kv_heads;
    a.eps = op.eps;
    a.positions = op.positions;
    a.t[0].x = op.q; a.t[0].xs = op.q_stride; a.t[0].xh = op.q_head_stride; a.t[0].w = op.q_weight; a.t[0].out = q_out;
    a.t[1].x = op.k; a.t[1].xs = op.k_stride; a.t[1].xh = op.k_head_stride; a.t[1].w = op.k_weight; a.t[1].out = k_out;
    for (int j = 0; j < op.n_pairs; ++j) {
        a.turns[j] = op.freqs[j] / (2.0 * M_PI);
        a.axes[j] = (uint8_t)op.axes[j];
    }
    return a;
}

// --------------------------------------------------------------- state cache

sn_status check_cache_sizes(const sn_cache *op) {
    if (!op || op->n_pages < 1 || op->n_kv_heads < 1 || op->n_kv_heads > 65535) return SN_ERR_INVALID;
    if (op->page_size < 16 || op->page_size > 1024 || (op->page_size & (op->page_size - 1))) return SN_ERR_INVALID;
    if (op->head_dim < 1 || op->head_dim > SN_MAX_HEAD_DIM) return SN_ERR_INVALID;
    if (op->dtype != SN_F32 && op->dtype != SN_BF16) return SN_ERR_INVALID;
    if (op->codes < SN_CODES_NONE || op->codes > SN_CODES_E4M3) return SN_ERR_INVALID;
    if (op->n_sequences < 1 || op->n_sequences > 65535 || op->n_rows < 0 || op->max_rows < 0 || op->max_rows > op->n_rows) return SN_ERR_INVALID;
    if ((int64_t)op->max_rows * op->n_sequences < op->n_rows) return SN_ERR_INVALID;
    // positions, with a tile behind the last, and rows with their heads are counted in 32 bits
    if (op->max_pages < 1 || (int64_t)op->max_pages * op->page_size > (1 << 30)) return SN_ERR_INVALID;
    return (int64_t)op->n_rows * op->n_kv_heads <= INT32_MAX ? SN_OK : SN_ERR_INVALID;
}

// What an attention needs besides; whether its launch holds the rows is attend_fits.
sn_status check_attend(const sn_cache *op) {
    if (op->n_heads < 1 || op->n_heads > 65535 || op->n_heads % op->n_kv_heads != 0) return SN_ERR_INVALID;
    if ((op->causal & ~1) != 0 || op->window < 0 || (op->window > 0 && !op->causal)) return SN_ERR_INVALID;
    return SN_OK;
}

sn_status check_cache(const sn_cache *op) {
    SN_TRY(check_cache_sizes(op));
    if (!op->k || !op->v || !op->row_ptr || !op->table || !op->lengths) return SN_ERR_INVALID;
    if ((reinterpret_cast<uintptr_t>(op->k) | reinterpret_cast<uintptr_t>(op->v)) & 15) return SN_ERR_INVALID;
    if (op->codes != SN_CODES_NONE &&
        (!op->k_scale || !op->v_scale ||
         ((reinterpret_cast<uintptr_t>(op->k_scale) | reinterpret_cast<uintptr_t>(op->v_scale)) & 15)))
        return SN_ERR_INVALID;
    return SN_OK;
}

CacheArgs cache_args(const sn_cache &op, void *ws) {
    CacheArgs a{};
    a.n_pages = op.n_pages; a.page = op.page_size; a.page_shift = __builtin_ctz(op.page_size);
    a.Hkv = op.n_kv_heads; a.D = op.head_dim; a.Dp = SN_CACHE_ROW(op.head_dim);
    a.k = op.k; a.v = op.v; a.k_scale = op.k_scale; a.v_scale = op.v_scale;
    a.B = op.n_sequences; a.n_rows = op.n_rows; a.max_rows = op.max_rows; a.max_pages = op.max_pages;
    a.row_ptr = op.row_ptr; a.table = op.table; a.lengths = op.lengths;
    a.status = reinterpret_cast<int *>(ws);
    a.H = op.n_heads; a.G = op.n_heads / op.n_kv_heads;
    a.scale = op.scale; a.causal = op.causal; a.window = op.window;
    a.q = op.q; a.qs = op.q_stride; a.qh = op.q_head_stride;
    const int64_t per = op.dtype == SN_F32 ? 4 : 8;
    a.q_vec = (reinterpret_cast<uintptr_t>(op.q) & 15) == 0 && a.qs % per == 0 && a.qh % per == 0 && a.D % 8 == 0;
    return a;
}

}  // namespace
}  // namespace sn

using namespace sn;

extern "C" {

sn_status sn_rotary_frequencies(int32_t n_axes, const int32_t *sections, double base, int32_t shared, double *freqs,
                                int32_t *axes) {
    if (n_axes < 1 || n_axes > SN_MAX_AXES || !sections || !freqs || !axes) return SN_ERR_INVALID;
    if (!(base > 0.0) || !std::isfinite(base)) return SN_ERR_INVALID;
    int64_t n = 0;
    for (int a = 0; a < n_axes; ++a) {
        if (sections[a] < 1) return SN_ERR_INVALID;
        n += sections[a];
    }
    if (n > kMaxPairs) return SN_ERR_INVALID;
    auto frequency = [&](int a, int i, int j) {
        return shared ? std::pow(base, -(double)j / (double)n) : std::pow(base, -(double)i / sections[a]);
    };
    int j = 0;
    for (int a = 0; a < n_axes; ++a)        // a base far below 1 gives a rising ladder
        for (int i = 0; i < sections[a]; ++i, ++j)
            if (!(frequency(a, i, j) < kMaxFrequency)) return SN_ERR_INVALID;
    j = 0;
    for (int a = 0; a < n_axes; ++a)
        for (int i = 0; i < sections[a]; ++i, ++j) {
            axes[j] = a;
            freqs[j] = frequency(a, i, j);
        }
    return SN_OK;
}

size_t sn_head_rotary_workspace_bytes(const sn_head_rotary *op) {
    return check_rotary_sizes(op) == SN_OK ? rotary_workspace(*op) : 0;
}

sn_status sn_head_rotary_forward(const sn_head_rotary *op, void *q_out, void *k_out, void *ws, size_t ws_bytes,
                                 void *stream) {
    SN_TRY(check_rotary(op));
    SN_TRY(check_ws(ws, ws_bytes, rotary_workspace(*op)));
    if (op->n_rows == 0) return SN_OK;
    if (!q_out || (op->n_kv_heads > 0 && !k_out) || !aligned_for(q_out, op->dtype) || !aligned_for(k_out, op->dtype))
        return SN_ERR_INVALID;
    return rotary_forward(rotary_args(*op, q_out, k_out), op->dtype, op->norm, reinterpret_cast<hipStream_t>(stream));
}

sn_status sn_head_rotary_backward(const sn_head_rotary *op, const void *d_q, int64_t d_q_stride, int64_t d_q_head_stride,
                                  const void *d_k, int64_t d_k_stride, int64_t d_k_head_stride, void *dq, void *dk,
                                  float *dq_weight, float *dk_weight, void *ws, size_t ws_bytes, void *stream) {
    SN_TRY(check_rotary(op));
    SN_TRY(check_ws(ws, ws_bytes, rotary_workspace(*op)));
    if (op->n_rows > 0 && (!d_q || !dq || (op->n_kv_heads > 0 && (!d_k || !dk)))) return SN_ERR_INVALID;
    if (!op->norm && (dq_weight || dk_weight)) return SN_ERR_INVALID;
    if (!aligned_for(d_q, op->dtype) || !aligned_for(d_k, op->dtype) || !aligned_for(dq, op->dtype) ||
        !aligned_for(dk, op->dtype) || !aligned_for(dq_weight, SN_F32) || !aligned_for(dk_weight, SN_F32))
        return SN_ERR_INVALID;
    RotaryArgs a = rotary_args(*op, dq, dk);
    a.t[0].dy = d_q; a.t[0].gs = d_q_stride; a.t[0].gh = d_q_head_stride;
    a.t[1].dy = d_k; a.t[1].gs = d_k_stride; a.t[1].gh = d_k_head_stride;
    return rotary_backward(a, op->dtype, op->norm, dq_weight, dk_weight, static_cast<char *>(ws),
                           reinterpret_cast<hipStream_t>(stream));
}

size_t sn_cache_workspace_bytes(const sn_cache *op) {
    if (check_cache_sizes(op) != SN_OK || check_attend(op) != SN_OK) return 0;
    return attend_fits(*op) ? attend_workspace(*op) : kWsBase;
}

sn_status sn_cache_write(const sn_cache *op, const void *k, int64_t k_stride, int64_t k_head_stride, const void *v,
                         int64_t v_stride, int64_t v_head_stride, void *ws, size_t ws_bytes, void *stream) {
    SN_TRY(check_cache(op));
    SN_TRY(check_ws(ws, ws_bytes, kWsBase));
    if (op->n_rows == 0) return SN_OK;
    if (!k || !v || !aligned_for(k, op->dtype) || !aligned_for(v, op->dtype)) return SN_ERR_INVALID;
    return cache_write(cache_args(*op, ws), op->dtype, op->codes, k, k_stride, k_head_stride, v, v_stride, v_head_stride,
                       reinterpret_cast<hipStream_t>(stream));
}

sn_status sn_cache_read(const sn_cache *op, void *k_out, void *v_out, void *ws, size_t ws_bytes, void *stream) {
    SN_TRY(check_cache(op));
    SN_TRY(check_ws(ws, ws_bytes, kWsBase));
    if (op->n_rows == 0) return SN_OK;
    if (!k_out || !v_out || !aligned_for(k_out, op->dtype) || !aligned_for(v_out, op->dtype)) return SN_ERR_INVALID;
    return cache_read(cache_args(*op, ws), op->dtype, op->codes, k_out, v_out, reinterpret_cast<hipStream_t>(stream));
}

sn_status sn_cache_attend(const sn_cache *op, void *o, float *lse, void *ws, size_t ws_bytes, void *stream) {
    SN_TRY(check_cache(op));
    SN_TRY(check_attend(op));
    if (!attend_fits(*op) || !std::isfinite(op->scale)) return SN_ERR_INVALID;
    SN_TRY(check_ws(ws, ws_bytes, attend_workspace(*op)));
    if (op->n_rows == 0) return SN_OK;
    if (!op->q || !o || !aligned_for(op->q, op->dtype) || !aligned_for(o, op->dtype) || !aligned_for(lse, SN_F32))
        return SN_ERR_INVALID;
    return cache_attend(cache_args(*op, ws), op->dtype, op->codes, o, lse, static_cast<char *>(ws),
                        reinterpret_cast<hipStream_t>(stream));
}

}  // extern "C"
