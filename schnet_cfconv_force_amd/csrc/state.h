// Shared declarations of the rotation of heads and of the state cache.
#pragma once

#include "context.h"

namespace sn {

typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Stores of N values that go past the caches, or not.  (The empty statements
// keep the compiler from merging the two kinds into one without the hint.)
template <int N, typename V>
__device__ inline void store_past(const V *v, V *p, bool past) {
    if (past) {
        asm volatile("");
#pragma unroll
        for (int i = 0; i < N; ++i) __builtin_nontemporal_store(v[i], p + i);
        asm volatile("");
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = v[i];
    }
}

// --------------------------------------------------------------- rotation of heads

constexpr int kMaxPairs = SN_MAX_HEAD_DIM / 2;
constexpr double kMaxFrequency = 0x1p52;    // from here on fp64 holds no angle of any position

struct RotaryTensor {
    const void *x, *dy;             // rows; gradients of the turned rows (backward)
    int64_t xs, xh, gs, gh;         // row and head strides
    const float *w;
    void *out;                      // turned rows, or the rows' gradients
};

struct RotaryArgs {
    int n_rows, D, P, interleaved;
    int H, Hkv;
    float eps;
    const int32_t *positions;
    RotaryTensor t[2];              // q, k
    double turns[kMaxPairs];        // full turns a position
    uint8_t axes[kMaxPairs];
};

size_t rotary_workspace(const sn_head_rotary &op);
bool rotary_fits(const sn_head_rotary &op);
sn_status rotary_forward(const RotaryArgs &a, int dtype, bool norm, hipStream_t s);
sn_status rotary_backward(const RotaryArgs &a, int dtype, bool norm, float *dq_weight, float *dk_weight, char *ws,
                          hipStream_t s);

// --------------------------------------------------------------- state cache

struct CacheArgs {
    int n_pages, page, page_shift;
    int Hkv, D, Dp;                 // Dp: elements of a row in a page
    void *k, *v;
    float *k_scale, *v_scale;
    int B, n_rows, max_rows, max_pages;
    const int32_t *row_ptr, *table, *lengths;
    int *status;
    int H, G;
    float scale;
    int causal, window;
    const void *q;
    int64_t qs, qh;
    int q_vec;                      // q's rows suit 16-byte reads
};

// Rows of sequence b in the call (r0, n) and its length, or n = 0 where the
// device arrays contradict the sizes: every row has a place of its own.
__device__ inline void sequence_rows(const CacheArgs &a, int b, int &r0, int &n, int &length) {
    segment_rows(a.row_ptr, b, a.B, a.n_rows, a.max_rows, a.status, r0, n);
    const auto lengths = (const __attribute__((address_space(4))) int32_t *)(uintptr_t)a.lengths;
    length = lengths[b];
    if (length < 0 || length > (int64_t)a.max_pages * a.page || length < n) {
        if (n > 0 && threadIdx.x == 0) flag_status(a.status, SN_ERR_INVALID);
        n = 0;
        length = 0;
    }
}

bool attend_fits(const sn_cache &op);
size_t attend_workspace(const sn_cache &op);
sn_status cache_write(const CacheArgs &a, int dtype, int codes, const void *k, int64_t ks, int64_t kh, const void *v,
                      int64_t vs, int64_t vh, hipStream_t s);
sn_status cache_read(const CacheArgs &a, int dtype, int codes, void *k, void *v, hipStream_t s);
sn_status cache_attend(const CacheArgs &a, int dtype, int codes, void *o, float *lse, char *ws, hipStream_t s);

// --------------------------------------------------------------- codes

__device__ inline float e4m3_value(uint8_t c) { return __builtin_amdgcn_cvt_f32_fp8((int)c, 0); }

// Eight codes of a row from its values x inv.  int8: adding 1.5 2^23 leaves the
// nearest whole number (ties to even) in the lowest bits; the product is
// rounded before, by itself.
template <int CODES>
__device__ inline uint2 encode8(const float (&x)[8], float inv) {
#pragma clang fp contract(off)
    uint2 r;
    if constexpr (CODES == SN_CODES_E4M3) {
        int lo = 0, hi = 0;
        lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * inv, x[1] * inv, lo, false);
        lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[2] * inv, x[3] * inv, lo, true);
        hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[4] * inv, x[5] * inv, hi, false);
        hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[6] * inv, x[7] * inv, hi, true);
        r.x = (uint32_t)lo;
        r.y = (uint32_t)hi;
    } else {
        uint32_t c[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float y = x[j] * inv;
            c[j] = __float_as_uint(y + 12582912.0f);
        }
        // byte 0 of each: pairs, then both pairs
        const uint32_t p0 = __builtin_amdgcn_perm(c[1], c[0], 0x0c0c0400u), p1 = __builtin_amdgcn_perm(c[3], c[2], 0x04000c0cu);
        const uint32_t p2 = __builtin_amdgcn_perm(c[5], c[4], 0x0c0c0400u), p3 = __builtin_amdgcn_perm(c[7], c[6], 0x04000c0cu);
        r.x = p0 | p1;
        r.y = p2 | p3;
    }
    return r;
}
template <int CODES>
__device__ inline void decode8(uint2 r, float (&x)[8]) {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const int c = (int)(w ? r.y : r.x);
        if constexpr (CODES == SN_CODES_E4M3) {
            x[4 * w] = __builtin_amdgcn_cvt_f32_fp8(c, 0);
            x[4 * w + 1] = __builtin_amdgcn_cvt_f32_fp8(c, 1);
            x[4 * w + 2] = __builtin_amdgcn_cvt_f32_fp8(c, 2);
            x[4 * w + 3] = __builtin_amdgcn_cvt_f32_fp8(c, 3);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) x[4 * w + j] = (float)(int8_t)(c >> (8 * j));
        }
    }
}

}  // namespace sn
