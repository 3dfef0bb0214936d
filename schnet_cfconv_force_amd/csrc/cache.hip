// Rows of keys and values to their places in the pages, and back.
//
// A group of lanes holds a row of a head, a lane eight of its elements; the
// largest magnitude is joined over the group, so a row is read once and its
// codes and its scale are written once.
#include <algorithm>

#include "state.h"

namespace sn {
namespace {

constexpr int kThreads = 256;

struct CacheRowsIO {
    const void *x[2];          // k, v given
    int64_t xs[2], xh[2];
    void *out[2];              // k, v read back
    int vec;                   // rows given or returned suit 16-byte accesses
};

// Lanes of a row: a power of two that holds Dp / 8.
inline int lanes_of(int Dp) {
    int n = 2;
    while (n * 8 < Dp) n *= 2;
    return n;
}

template <typename T>
__device__ inline void load_row8(const T *p, int d, int D, bool vec, float (&x)[8]) {
    if (vec && d < D) {
        typedef T vec_t __attribute__((ext_vector_type(16 / sizeof(T))));
#pragma unroll
        for (int i = 0; i < 8; i += 16 / sizeof(T)) {
            const vec_t v = *reinterpret_cast<const vec_t *>(p + d + i);
#pragma unroll
            for (int j = 0; j < (int)(16 / sizeof(T)); ++j) x[i + j] = to_f32(v[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = d + j < D ? to_f32(p[d + j]) : 0.0f;
    }
}
template <typename T>
__device__ inline void store_row8(T *p, int d, int D, bool vec, const float (&x)[8]) {
    if (vec && d < D) {
        typedef T vec_t __attribute__((ext_vector_type(16 / sizeof(T))));
#pragma unroll
        for (int i = 0; i < 8; i += 16 / sizeof(T)) {
            vec_t v;
#pragma unroll
            for (int j = 0; j < (int)(16 / sizeof(T)); ++j) v[j] = (T)x[i + j];
            *reinterpret_cast<vec_t *>(p + d + i) = v;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (d + j < D) p[d + j] = (T)x[j];
    }
}

template <typename T, int CODES>
__global__ __launch_bounds__(kThreads) void cache_write_kernel(CacheArgs a, CacheRowsIO io, int lanes, int chunk_rows) {
    int r0, n, length;
    sequence_rows(a, blockIdx.y, true, r0, n, length);
    const int first = blockIdx.x * chunk_rows, rows = min(chunk_rows, n - first);
    const int lane = threadIdx.x % lanes, d = lane * 8;
    for (int i = threadIdx.x / lanes; i < rows * 2 * a.Hkv; i += kThreads / lanes) {
        const int h = i % a.Hkv, n_ = i / a.Hkv & 1, row = first + i / a.Hkv / 2;
        const T *src = static_cast<const T *>(io.x[n_]) + (r0 + row) * io.xs[n_] + h * io.xh[n_];
        float x[8];
        load_row8(src, d, a.D, io.vec, x);
        const int at = length - n + row, page = page_of(a, blockIdx.y, at);
        const int64_t place = (((int64_t)max(page, 0) * a.Hkv + h) << a.page_shift) + (at & (a.page - 1));
        if constexpr (CODES == SN_CODES_NONE) {
            if (page >= 0 && d < a.Dp) store_row8(static_cast<T *>(n_ ? a.v : a.k) + place * a.Dp, d, a.Dp, true, x);
        } else {
            // magnitudes compared as bits: a NaN is above an infinity is above all else
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(x[j]) & 0x7fffffffu);
            for (int o = lanes >> 1; o > 0; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
            constexpr float kTop = CODES == SN_CODES_INT8 ? 127.0f : 448.0f;
            const float amax = __uint_as_float(top);
            const bool bad = top >= 0x7f800000u, live = !bad && amax >= 0x1p-100f;
            const float scale = bad ? __uint_as_float(0x7fc00000u) : live ? amax / kTop : 0.0f;
            uint2 codes = {0, 0};
            if (live) codes = encode8<CODES>(x, kTop / amax);
            if (page >= 0 && d < a.Dp) {
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(n_ ? a.v : a.k) + place * a.Dp + d) = codes;
                if (lane == 0) (n_ ? a.v_scale : a.k_scale)[place] = scale;
            }
        }
    }
}

template <typename T, int CODES>
__global__ __launch_bounds__(kThreads) void cache_read_kernel(CacheArgs a, CacheRowsIO io, int lanes, int chunk_rows) {
    int r0, n, length;
    sequence_rows(a, blockIdx.y, true, r0, n, length);
    const int first = blockIdx.x * chunk_rows, rows = min(chunk_rows, n - first);
    const int lane = threadIdx.x % lanes, d = lane * 8;
    for (int i = threadIdx.x / lanes; i < rows * 2 * a.Hkv; i += kThreads / lanes) {
        const int h = i % a.Hkv, n_ = i / a.Hkv & 1, row = first + i / a.Hkv / 2;
        const int at = length - n + row, page = page_of(a, blockIdx.y, at);
        const int64_t place = (((int64_t)max(page, 0) * a.Hkv + h) << a.page_shift) + (at & (a.page - 1));
        float x[8] = {};
        if (page >= 0 && d < a.Dp) {
            if constexpr (CODES == SN_CODES_NONE) {
                load_row8(static_cast<const T *>(n_ ? a.v : a.k) + place * a.Dp, d, a.Dp, true, x);
            } else {
                decode8<CODES>(*reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(n_ ? a.v : a.k) + place * a.Dp + d), x);
                const float scale = (n_ ? a.v_scale : a.k_scale)[place];
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] *= scale;
            }
        }
        T *dst = static_cast<T *>(io.out[n_]) + ((int64_t)(r0 + row) * a.Hkv + h) * a.D;
        store_row8(dst, d, a.D, io.vec, x);
    }
}

// Rows of a block: about four rounds of its groups.
int chunk_of(const CacheArgs &a, int lanes) { return std::max(1, 4 * (kThreads / lanes) / (2 * a.Hkv)); }

template <typename T, int CODES>
sn_status launch(const CacheArgs &a, const CacheRowsIO &io, bool write, hipStream_t s) {
    const int lanes = lanes_of(a.Dp), rows = chunk_of(a, lanes);
    const dim3 grid((a.max_rows + rows - 1) / rows, a.B);
    ProfScope prof(write ? K_CACHE_WRITE : K_CACHE_READ, s);
    if (write)
        cache_write_kernel<T, CODES><<<grid, kThreads, 0, s>>>(a, io, lanes, rows);
    else
        cache_read_kernel<T, CODES><<<grid, kThreads, 0, s>>>(a, io, lanes, rows);
    return launch_status();
}
template <typename T>
sn_status launch(const CacheArgs &a, int codes, const CacheRowsIO &io, bool write, hipStream_t s) {
    if (codes == SN_CODES_INT8) return launch<T, SN_CODES_INT8>(a, io, write, s);
    if (codes == SN_CODES_E4M3) return launch<T, SN_CODES_E4M3>(a, io, write, s);
    return launch<T, SN_CODES_NONE>(a, io, write, s);
}

bool rows_vec(const CacheArgs &a, int dtype, const void *p, int64_t s, int64_t h) {
    const int64_t per = dtype == SN_F32 ? 4 : 8;
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && s % per == 0 && h % per == 0 && a.D % 8 == 0;
}

}  // namespace

bool cache_fits(const sn_cache &op) {
    // one row a block at the least
    return op.n_sequences <= 65535 && grid_fits((int64_t)op.max_rows * op.n_sequences, kThreads);
}

sn_status cache_write(const CacheArgs &a, int dtype, int codes, const void *k, int64_t ks, int64_t kh, const void *v,
                      int64_t vs, int64_t vh, hipStream_t s) {
    CacheRowsIO io{{k, v}, {ks, vs}, {kh, vh}, {}, rows_vec(a, dtype, k, ks, kh) && rows_vec(a, dtype, v, vs, vh)};
    return dtype == SN_F32 ? launch<float>(a, codes, io, true, s) : launch<bf16>(a, codes, io, true, s);
}

sn_status cache_read(const CacheArgs &a, int dtype, int codes, void *k, void *v, hipStream_t s) {
    CacheRowsIO io{{}, {}, {}, {k, v}, rows_vec(a, dtype, k, 0, 0) && rows_vec(a, dtype, v, 0, 0)};
    return dtype == SN_F32 ? launch<float>(a, codes, io, false, s) : launch<bf16>(a, codes, io, false, s);
}

}  // namespace sn
