// Shared declarations of the context operators (cross attention with a
// relative position bias; group norm with an activation).
#pragma once

#include <hip/hip_bf16.h>

#include "sn_internal.h"

namespace sn {

// --------------------------------------------------------------- element types

typedef __bf16 bf16;

__device__ inline float to_f32(float v) { return v; }
__device__ inline float to_f32(bf16 v) { return (float)v; }

// --------------------------------------------------------------- grids

// A launch counts its threads in 32 bits.
inline bool grid_fits(int64_t blocks, int threads) { return blocks * threads <= UINT32_MAX; }

// --------------------------------------------------------------- ragged rows

// Rows of segment b: start and length, or length 0 where the pointer array
// contradicts the sizes that the host was given (flagged in the status word).
__device__ inline void segment_rows(const int32_t *ptr, int b, int n_segments, int n_rows, int max_rows, int *status,
                                    int &start, int &len) {
    // b is the same in the whole block: scalar reads, straight into scalar registers
    const auto p = (const __attribute__((address_space(4))) int32_t *)(uintptr_t)ptr;
    const int s = p[b], e = p[b + 1];
    start = s;
    len = e - s;
    if (s < 0 || e < s || e > n_rows || e - s > max_rows || (b == 0 && s != 0) ||
        (b == n_segments - 1 && e != n_rows)) {
        len = 0;
        start = 0;
        if (threadIdx.x == 0) flag_status(status, SN_ERR_INVALID);
    }
}

// --------------------------------------------------------------- attention

struct AttnArgs {
    int B, n_q, n_k, max_q, max_k;
    const int32_t *q_ptr, *k_ptr;
    int H, Hkv, G, D;
    float scale;
    const void *q, *k, *v, *d_o;
    int64_t qs, qh, ks, kh, vs, vh, gs, gh;   // row and head strides (g: d_o)
    const uint8_t *keep;
    const float *bias;
    int nb;                                   // buckets (0: no bias)
    const int32_t *q_pos, *k_pos;
    int *status;
    // derived
    int fast;                                 // every tensor's rows suit 16-byte reads at 31-bit offsets in a tile
    int out4;                                 // every output's rows suit stores of four elements
    int Gs, subs;                             // heads of a row block's subgroup, subgroups of a key/value head
    int row_tiles, splits;                    // row tiles of the longest segment, key splits
    int lut_base, lut_n;                      // first offset and length of the position table
    int lut_run;                              // its offsets stay clear of the type's ends
    int32_t thr[SN_MAX_BUCKETS];              // padded with the largest value
};

// Whether a call of these sizes has grids that fit, with some pointers and
// thresholds; the launches check their own.
bool attn_forward_fits(const sn_cross_attention &op);
bool attn_backward_fits(const sn_cross_attention &op);
size_t attn_forward_workspace(const sn_cross_attention &op);
size_t attn_backward_workspace(const sn_cross_attention &op);
sn_status attn_forward(AttnArgs a, int dtype, void *o, float *rows, float *lse, char *ws, hipStream_t s);
sn_status attn_backward(AttnArgs a, int dtype, const float *o, const float *lse, void *dq, void *dk, void *dv,
                        float *dbias, char *ws, hipStream_t s);

// --------------------------------------------------------------- group norm

struct NormArgs {
    int B, n_rows, max_rows, C, groups, width, act;
    float eps;
    const int32_t *ptr;
    const void *x, *dy;
    int64_t xs, dys;
    const float *gamma, *beta;
    int *status;
};

bool norm_fits(const sn_group_norm &op);
size_t norm_workspace(const sn_group_norm &op);
sn_status norm_forward(const NormArgs &a, int dtype, void *y, float *mean, float *rstd, char *ws, hipStream_t s);
sn_status norm_backward(const NormArgs &a, int dtype, const float *mean, const float *rstd, void *dx, float *dgamma,
                        float *dbeta, char *ws, hipStream_t s);

}  // namespace sn
