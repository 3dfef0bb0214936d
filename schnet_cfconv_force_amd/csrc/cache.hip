// Rows of keys and values to their places in the pages, and back.
//
// A group of lanes holds a row of a head, a lane eight of its elements; the
// largest magnitude is joined over the group, so a row is read once and its
// codes and its scale are written once.  What it costs is those bytes: 48 x
// <= 4096 rows of 8 x 128, bf16 to int8, 790 MB a pass: written at 5.0 TB/s (the
// vector units nine tenths busy with the codes), read back at 5.1.
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

// Rows beyond this are in no cache when they are read: they are stored past it
// (48 x <= 4096 rows of 8 x 128, bf16, 500 MB: written and read back 405 us ->
// 385; 8 x <= 2000, 42 MB: 35 -> 41).
constexpr int64_t kPast = 128 << 20;

// A launch has a place for the longest sequence's rows in every sequence.  Beyond
// this many blocks, most of them empty, a block takes several chunks in turn.
constexpr int kBlocks = 1 << 22;

// How rows are cut (host).  An item is a row of a head, of k or of v; a block
// takes chunk_rows rows' items in order, its groups one each in turn.
struct CacheCut {
    int lane_bits;              // a group has 2^lane_bits lanes
    int chunk_rows;
    uint32_t next_chunk;        // rows from a block's chunk to its next (a length is at most 2^30)
    int step_row, step_head;    // from one item of a group to the next (heads of k, then of v)
    bool past;                  // rows are stored past the caches
};

// A group's items in turn.
struct Item {
    int row, head;
    __device__ inline void next(const CacheCut &c, int heads) {
        row += c.step_row;
        head += c.step_head;
        if (head >= heads) {
            head -= heads;
            ++row;
        }
    }
};

// Items of a group on their way at once, and of a block's groups: 48 x <= 4096
// rows of 8 x 128, bf16 to int8 and back, 158 + 156 us; with two 167 + 166, with
// eight 169 + 165; in blocks of eight items a group 163 + 167, of 32 182 + 191.
constexpr int kItems = 4;

// Eight elements of a row as they lie in memory, zero from D on.
template <typename T>
struct Raw {
    typedef uint32_t quad __attribute__((ext_vector_type(4)));
    quad r[sizeof(T) / 2];
    __device__ inline void load(const T *p, int d, int D, bool vec, bool has) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) r[i] = quad{0, 0, 0, 0};
        if (!has || d >= D) return;
        if (vec) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i) r[i] = *reinterpret_cast<const quad *>(p + d + i * 16 / sizeof(T));
        } else {
            T x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = d + j < D ? p[d + j] : (T)0.0f;
            __builtin_memcpy(r, x, sizeof(x));
        }
    }
    __device__ inline void get(float (&x)[8]) const {
        T y[8];
        __builtin_memcpy(y, r, sizeof(y));
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = to_f32(y[j]);
    }
    __device__ inline void set(const float (&x)[8]) {
        T y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = (T)x[j];
        __builtin_memcpy(r, y, sizeof(y));
    }
    __device__ inline void store(T *p, int d, int D, bool vec, bool past) const {
        if (d >= D) return;
        if (vec) {
            store_past<sizeof(T) / 2>(r, reinterpret_cast<quad *>(p + d), past);
        } else {
            T y[8];
            __builtin_memcpy(y, r, sizeof(y));
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (d + j < D) p[d + j] = y[j];
        }
    }
};

// Largest of the group's values, in every lane of it (at most sixteen lanes).
template <int CTRL>
__device__ inline uint32_t dpp_max(uint32_t v) {
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xf, 0xf, true));
}
__device__ inline uint32_t group_max(uint32_t v, int bits) {
    v = dpp_max<0xb1>(v);                   // quad_perm 1 0 3 2
    if (bits > 1) v = dpp_max<0x4e>(v);     // quad_perm 2 3 0 1
    if (bits > 2) v = dpp_max<0x141>(v);    // row_half_mirror
    if (bits > 3) v = dpp_max<0x140>(v);    // row_mirror
    return v;
}

template <typename T, int CODES>
__global__ __launch_bounds__(kThreads) void cache_write_kernel(CacheArgs a, CacheRowsIO io, CacheCut c) {
    int r0, n, length;
    sequence_rows(a, blockIdx.y, r0, n, length);
    const int heads = 2 * a.Hkv;
    const int lane = threadIdx.x & ((1 << c.lane_bits) - 1), d = lane * 8, group = threadIdx.x >> c.lane_bits;
    const int32_t *table = a.table + (int64_t)blockIdx.y * a.max_pages;
    for (uint32_t chunk = blockIdx.x * c.chunk_rows; chunk < (uint32_t)n; chunk += c.next_chunk) {
        const int first = (int)chunk, rows = min(c.chunk_rows, n - first);
        Item at{group / heads, group % heads};
        while (at.row < rows) {
            Item item[kItems];
            Raw<T> raw[kItems];
            int page[kItems];
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                item[i] = at;
                at.next(c, heads);
                const bool has = item[i].row < rows, is_v = item[i].head >= a.Hkv;
                const int h = item[i].head - (is_v ? a.Hkv : 0), row = first + item[i].row;
                raw[i].load(static_cast<const T *>(io.x[is_v]) + (r0 + row) * io.xs[is_v] + h * io.xh[is_v], d, a.D, io.vec, has);
                page[i] = has ? table[(length - n + row) >> a.page_shift] : 0;
            }
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                const bool is_v = item[i].head >= a.Hkv;
                const int h = item[i].head - (is_v ? a.Hkv : 0), pos = length - n + first + item[i].row;
                if (item[i].row >= rows) break;
                const bool ok = (uint32_t)page[i] < (uint32_t)a.n_pages;
                if (!ok && lane == 0) flag_status(a.status, SN_ERR_INVALID);
                const int64_t place = (((int64_t)page[i] * a.Hkv + h) << a.page_shift) + (pos & (a.page - 1));
                if constexpr (CODES == SN_CODES_NONE) {
                    if (ok) raw[i].store(static_cast<T *>(is_v ? a.v : a.k) + place * a.Dp, d, a.Dp, true, c.past);
                } else {
                    float x[8];
                    raw[i].get(x);
                    // magnitudes compared as bits: a NaN is above an infinity is above all else
                    uint32_t top = 0;
#pragma unroll
                    for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(x[j]) & 0x7fffffffu);
                    top = group_max(top, c.lane_bits);
                    constexpr float kTop = CODES == SN_CODES_INT8 ? 127.0f : 448.0f;
                    const float amax = __uint_as_float(top);
                    const bool bad = top >= 0x7f800000u, live = !bad && amax >= 0x1p-100f;
                    const float scale = bad ? __uint_as_float(0x7fc00000u) : live ? amax / kTop : 0.0f;
                    uint2 codes = {0, 0};
                    if (live) codes = encode8<CODES>(x, kTop / amax);
                    if (ok && d < a.Dp) {
                        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(is_v ? a.v : a.k) + place * a.Dp + d) = codes;
                        if (lane == 0) (is_v ? a.v_scale : a.k_scale)[place] = scale;
                    }
                }
            }
        }
    }
}

template <typename T, int CODES>
__global__ __launch_bounds__(kThreads) void cache_read_kernel(CacheArgs a, CacheRowsIO io, CacheCut c) {
    int r0, n, length;
    sequence_rows(a, blockIdx.y, r0, n, length);
    const int heads = 2 * a.Hkv;
    const int lane = threadIdx.x & ((1 << c.lane_bits) - 1), d = lane * 8, group = threadIdx.x >> c.lane_bits;
    const int32_t *table = a.table + (int64_t)blockIdx.y * a.max_pages;
    for (uint32_t chunk = blockIdx.x * c.chunk_rows; chunk < (uint32_t)n; chunk += c.next_chunk) {
        const int first = (int)chunk, rows = min(c.chunk_rows, n - first);
        Item at{group / heads, group % heads};
        while (at.row < rows) {
            Item item[kItems];
            int page[kItems];
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                item[i] = at;
                at.next(c, heads);
                page[i] = item[i].row < rows ? table[(length - n + first + item[i].row) >> a.page_shift] : -1;
            }
            Raw<T> raw[kItems];
            uint2 codes[kItems];
            float scale[kItems];
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                const bool is_v = item[i].head >= a.Hkv, ok = (uint32_t)page[i] < (uint32_t)a.n_pages;
                const int h = item[i].head - (is_v ? a.Hkv : 0), pos = length - n + first + item[i].row;
                const int64_t place = (((int64_t)(ok ? page[i] : 0) * a.Hkv + h) << a.page_shift) + (pos & (a.page - 1));
                if (!ok && item[i].row < rows && lane == 0) flag_status(a.status, SN_ERR_INVALID);
                if constexpr (CODES == SN_CODES_NONE) {
                    raw[i].load(static_cast<const T *>(is_v ? a.v : a.k) + place * a.Dp, d, a.Dp, true, ok);
                } else {
                    codes[i] = uint2{0, 0};
                    scale[i] = 0.0f;
                    if (ok && d < a.Dp) {
                        codes[i] = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(is_v ? a.v : a.k) + place * a.Dp + d);
                        scale[i] = (is_v ? a.v_scale : a.k_scale)[place];
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                if (item[i].row >= rows) break;
                const bool is_v = item[i].head >= a.Hkv;
                const int h = item[i].head - (is_v ? a.Hkv : 0);
                if constexpr (CODES != SN_CODES_NONE) {
                    float x[8];
                    decode8<CODES>(codes[i], x);
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] *= scale[i];
                    raw[i].set(x);
                }
                raw[i].store(static_cast<T *>(io.out[is_v]) + ((int64_t)(r0 + first + item[i].row) * a.Hkv + h) * a.D, d, a.D, io.vec, c.past);
            }
        }
    }
}

template <typename T, int CODES>
sn_status launch(const CacheArgs &a, const CacheRowsIO &io, bool write, hipStream_t s) {
    CacheCut c;
    c.lane_bits = 1;
    while (8 << c.lane_bits < a.Dp) ++c.lane_bits;
    const int groups = kThreads >> c.lane_bits, heads = 2 * a.Hkv;
    c.step_row = groups / heads;
    c.step_head = groups % heads;
    c.chunk_rows = std::max(1, kItems * groups / heads);
    c.past = (int64_t)a.n_rows * heads * a.D * (int64_t)sizeof(T) > kPast;
    const int chunks = (int)(((int64_t)a.max_rows + c.chunk_rows - 1) / c.chunk_rows);
    const dim3 grid(std::min(chunks, kBlocks / a.B), a.B);
    c.next_chunk = grid.x * (uint32_t)c.chunk_rows;
    ProfScope prof(write ? K_CACHE_WRITE : K_CACHE_READ, s);
    if (write)
        cache_write_kernel<T, CODES><<<grid, kThreads, 0, s>>>(a, io, c);
    else
        cache_read_kernel<T, CODES><<<grid, kThreads, 0, s>>>(a, io, c);
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
