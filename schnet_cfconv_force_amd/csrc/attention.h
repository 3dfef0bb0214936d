// Tiles, products and position buckets shared by the attention kernels.
//
// Every product runs on v_mfma_f32_32x32x16_bf16.  bf16 rows enter as they
// are (one plane); an fp32 row is held as three bf16 planes, x = x0 + x1 + x2
// (8 + 8 + 8 bits: the residuals are exact, so the sum is x to 2^-24), and a
// product of two of them is the six plane products of weight 2^-16 or more.
// Six bf16 products cost 6/16 of one fp32 matrix instruction of that size.
//
// Layout of one 32x32x16 product (64 lanes): A fragment of lane l = row l%32,
// k = 8(l/32) + j; B fragment = column l%32, k = 8(l/32) + j; accumulator of
// lane l = column l%32, rows 8(r/4) + 4(l/32) + r%4.  The sums over k may run
// in any order if both operands agree on it: a finished 32x32 score tile
// (its rows the next product's k) is used as the B operand as it lies in the
// registers, with slot j of half h standing for k = 8(j/4) + 4h + j%4, and
// frag_cols() reads the A operand in that order.
#pragma once

#include "context.h"

namespace sn {

typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short short4v __attribute__((ext_vector_type(4)));
typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef float floatx2 __attribute__((ext_vector_type(2)));

__device__ inline floatx16 zero16() {
    return floatx16{0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kAttnThreads = 256;   // four wavefronts
constexpr int kLutMax = 2048;       // entries of a position table (SN_MAX_BUCKET_SPAN + 2)

template <int NP>
struct RowOf { using T = float; };
template <>
struct RowOf<1> { using T = bf16; };

// Eight consecutive elements of a row as NP planes.
template <int NP>
struct Frag { bf16x8 p[NP]; };

template <int NP>
__device__ inline Frag<NP> split8f(const float (&x)[8]) {
    Frag<NP> f;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        float r[2] = {x[j], x[j + 1]};
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            const bf16x2 h = __builtin_convertvector((floatx2{r[0], r[1]}), bf16x2);
            f.p[n][j] = h[0];
            f.p[n][j + 1] = h[1];
            r[0] -= (float)h[0];
            r[1] -= (float)h[1];
        }
    }
    return f;
}

// SWAPPED: the order of mma(b, a), so that a product and its transpose agree.
template <int NP, bool SWAPPED = false>
__device__ inline floatx16 mma(const Frag<NP> &a, const Frag<NP> &b, floatx16 c) {
    if constexpr (NP == 3 && SWAPPED) {
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[0], b.p[2], c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[1], b.p[1], c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[2], b.p[0], c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[0], b.p[1], c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[1], b.p[0], c, 0, 0, 0);
    } else if constexpr (NP == 3) {   // the small terms first
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[2], b.p[0], c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[1], b.p[1], c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[0], b.p[2], c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[1], b.p[0], c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[0], b.p[1], c, 0, 0, 0);
    }
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[0], b.p[0], c, 0, 0, 0);
}

// Ends a chain of products whose sums vector instructions read next: the
// hardware does not hold such a read back until the last product is through
// (12 wait states for eight passes), and where a branch lies between, the
// compiler (ROCm 7.2) was seen to count the waits along its longer side only,
// so that the last registers were read early.  Here they pass through this
// block, in the chain's own straight line.
__device__ inline void settle(floatx16 &x) { asm volatile("s_nop 7\n\ts_nop 3" : "+v"(x)); }

// --------------------------------------------------------------- tiles in LDS

// A tile row holds DP elements in chunks of eight (16 bytes); chunk c of row
// r lies at position c ^ swizzle(r).  Sixteen rows read at one chunk, and
// four rows from a multiple of four read over four chunks, each touch every
// bank once.
template <int DP>
__device__ inline int swizzle(int row) {
    if constexpr (DP == 128) return ((row & 3) << 2) | ((row >> 2) & 3);
    if constexpr (DP == 64) return ((row & 2) << 1) | ((row >> 2) & 3);
    return (row >> 2) & 3;
}
template <int DP>
__device__ inline int tile_at(int row, int chunk) {
    return row * DP + ((chunk ^ swizzle<DP>(row)) << 3);
}

// LDS addresses are byte offsets: a tile's (uniform, a multiple of 256) plus a
// lane's.
typedef __attribute__((address_space(3))) char *lds_ptr;
__device__ inline uint32_t lds_offset(const void *p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char *)(const char *)p;
}

// A lane's places in a tile.  The swizzle leaves the chunk's upper bits to
// the fragment's index alone, so an index is one exclusive-or away, and rows
// 16 further are a constant.
template <int DP>
struct TileLane {
    uint32_t rows, cols, cols8;
    __device__ inline TileLane(int lane) {
        rows = 2 * tile_at<DP>(lane & 31, lane >> 5);
        const int i = lane & 15, row = 4 * (lane >> 5) + (i >> 2), d = (lane & 16) + 4 * (i & 3);
        cols = 2 * (tile_at<DP>(row, d >> 3) + (d & 7));
        cols8 = 2 * (tile_at<DP>(row + 8, d >> 3) + (d & 7));
    }
    // Rows row0 .. row0 + 31 of the tile (row0 a multiple of 32), elements
    // 16 s + 8 (l/32) ..: an A operand whose rows are tile rows.
    __device__ inline bf16x8 frag_rows(uint32_t tile, int row0, int s) const {
        const uint32_t at = (rows + tile) ^ (s << 5);
        return *(__attribute__((address_space(3))) const bf16x8 *)(lds_ptr)(uintptr_t)(at + row0 * 2 * DP);
    }
    // Elements 32 e .. 32 e + 31 as rows, tile rows row0 .. row0 + 15 (a
    // multiple of 16) as k in the order of a score tile's registers: the
    // transposing LDS read hands lane i of sixteen the column i of the 4 x 16
    // block that the sixteen lanes address.
    __device__ inline bf16x8 frag_cols(uint32_t tile, int row0, int e) const {
        typedef __attribute__((address_space(3))) short4v *lds4;
        const uint32_t a0 = ((cols + tile) ^ (e << 6)) + row0 * 2 * DP, a1 = ((cols8 + tile) ^ (e << 6)) + row0 * 2 * DP;
        const bf16x4 a = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(uintptr_t)a0));
        const bf16x4 b = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(uintptr_t)a1));
        return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    }
};
// The same with NP planes, `plane` bytes apart.
template <int NP, int DP>
__device__ inline Frag<NP> frag_rows(const TileLane<DP> &l, uint32_t tile, uint32_t plane, int row0, int s) {
    Frag<NP> f;
#pragma unroll
    for (int n = 0; n < NP; ++n) f.p[n] = l.frag_rows(tile + n * plane, row0, s);
    return f;
}
template <int NP, int DP>
__device__ inline Frag<NP> frag_cols(const TileLane<DP> &l, uint32_t tile, uint32_t plane, int row0, int e) {
    Frag<NP> f;
#pragma unroll
    for (int n = 0; n < NP; ++n) f.p[n] = l.frag_cols(tile + n * plane, row0, e);
    return f;
}
// One plane: the column fragments of a 32-row tile on their way ahead of
// their use, [16 rows][element block].
template <int DP>
struct ColsAhead {
    bf16x8 f[2][DP / 32];
    __device__ inline void load(const TileLane<DP> &l, uint32_t tile, int row0) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < DP / 32; ++e) f[u][e] = l.frag_cols(tile, row0 + 16 * u, e);
    }
};
// A B over all of a row's elements, A the tile's rows row0 .. row0 + 31.  One
// plane: begin() sends for every operand, and what is computed until finish()
// covers their way.
template <int NP, int DP>
struct RowsProduct {
    bf16x8 f[NP == 1 ? DP / 16 : 1];
    __device__ inline void begin(const TileLane<DP> &l, uint32_t tile, int row0) {
        if constexpr (NP == 1)
#pragma unroll
            for (int s = 0; s < DP / 16; ++s) f[s] = l.frag_rows(tile, row0, s);
    }
    template <bool SWAPPED = false>
    __device__ inline floatx16 finish(const TileLane<DP> &l, uint32_t tile, uint32_t plane, int row0,
                                      const Frag<NP> (&b)[DP / 16]) const {
        floatx16 x = zero16();
#pragma unroll
        for (int s = 0; s < DP / 16; ++s) {
            if constexpr (NP == 1)
                x = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[s], b[s].p[0], x, 0, 0, 0);
            else
                x = mma<NP, SWAPPED>(frag_rows<NP, DP>(l, tile, plane, row0, s), b[s], x);
        }
        return x;
    }
};

// Eight elements at `p` (elements d .. d + 7 of a row of D; zero beyond D),
// as loaded.  vec: the row and its strides are 16-byte aligned and D is a
// multiple of eight.
template <int NP>
struct Raw8 {
    float4 v[NP == 1 ? 1 : 2];
};
template <int NP>
__device__ inline Raw8<NP> raw_zero() {
    Raw8<NP> r;
    r.v[0] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if constexpr (NP == 3) r.v[1] = r.v[0];
    return r;
}
template <int NP>
__device__ inline Raw8<NP> load8(const typename RowOf<NP>::T *p, int d, int D, bool vec) {
    Raw8<NP> r = raw_zero<NP>();
    if (d >= D) return r;
    if (vec) {
        r.v[0] = *reinterpret_cast<const float4 *>(p);
        if constexpr (NP == 3) r.v[1] = *reinterpret_cast<const float4 *>(p + 4);
    } else if constexpr (NP == 1) {
        bf16x8 t;
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = d + j < D ? p[j] : (bf16)0.0f;
        r.v[0] = __builtin_bit_cast(float4, t);
    } else {
        float t[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = d + j < D ? p[j] : 0.0f;
        r.v[0] = make_float4(t[0], t[1], t[2], t[3]);
        r.v[1] = make_float4(t[4], t[5], t[6], t[7]);
    }
    return r;
}
template <int NP>
__device__ inline Frag<NP> to_frag(const Raw8<NP> &r) {
    if constexpr (NP == 1) {
        Frag<1> f;
        f.p[0] = __builtin_bit_cast(bf16x8, r.v[0]);
        return f;
    } else {
        const float x[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
        return split8f<NP>(x);
    }
}

// One tile of R rows on its way from global memory to LDS, by NT threads:
// load() issues the reads into registers, store() splits and writes them, so
// nothing waits for memory between the two.
//
// FAST: 16-byte aligned rows within 2^31 bytes of the tile's first.  They
// are read through a buffer descriptor that ends with the tile's last valid
// row: what lies beyond, and elements from D on (sent out of range), come
// back as zeros without a branch or a 64-bit address per read.
template <int NP, int DP, int R, int NT, bool FAST>
struct TileMove {
    using T = typename RowOf<NP>::T;
    static constexpr int CH = DP / 8, IT = (R * CH + NT - 1) / NT;
    static constexpr bool kExact = IT * NT == R * CH;
    Raw8<NP> raw[IT];
    uint32_t off, step;
    const T *next;      // first row of the tile that load() takes
    int left;           // rows from there on
    int full;           // bytes of a full tile
    int64_t stride;
    __device__ inline void init(int64_t row_stride, int D, int tid) {
        stride = row_stride;
        if constexpr (FAST) {
            const int c = tid % CH;
            off = (kExact || tid < R * CH) && 8 * c < D ? (uint32_t)((tid / CH) * stride + 8 * c) * sizeof(T) : 0x80000000u;
            step = (uint32_t)(NT / CH * stride) * sizeof(T);
            full = (int)(((R - 1) * stride + D) * sizeof(T));
        }
    }
    __device__ inline void seek(const T *base, int rows) {
        next = base;
        left = rows;
    }
    // the tile's rows at `next`, those from `left` on zero; goes on by `rows`
    __device__ inline void load(int D, int tid, int rows = R) {
        if constexpr (FAST) {
            const int bytes = left >= R ? full : left > 0 ? (int)(((left - 1) * stride + D) * sizeof(T)) : 0;
            const __amdgpu_buffer_rsrc_t rsrc =
                __builtin_amdgcn_make_buffer_rsrc(const_cast<T *>(next), 0, bytes, 0x00020000);
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                const uint32_t at = off + it * step;
                raw[it].v[0] = __builtin_bit_cast(float4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, at, 0, 0));
                if constexpr (NP == 3)
                    raw[it].v[1] = __builtin_bit_cast(float4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, at + 16, 0, 0));
            }
        } else {
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                const int c = tid + it * NT, row = c / CH, d = (c % CH) * 8;
                raw[it] = raw_zero<NP>();
                if (row < left && row < R) raw[it] = load8<NP>(next + row * stride + d, d, D, false);
            }
        }
        next += rows * stride;
        left -= rows;
    }
    // partial: rows whose bit in `kept` is clear become zero
    __device__ inline void store(bf16 *tile, int tid, bool partial, uint64_t kept) {
        if (partial)
#pragma unroll
            for (int it = 0; it < IT; ++it)
                if (!((kept >> ((tid + it * NT) / CH & 63)) & 1)) raw[it] = raw_zero<NP>();
#pragma unroll
        for (int it = 0; it < IT; ++it) {
            const int c = tid + it * NT;
            if (!kExact && c >= R * CH) continue;
            const Frag<NP> f = to_frag<NP>(raw[it]);
            const int at = tile_at<DP>(c / CH, c % CH);
#pragma unroll
            for (int n = 0; n < NP; ++n) *reinterpret_cast<bf16x8 *>(tile + n * R * DP + at) = f.p[n];
        }
    }
};

// --------------------------------------------------------------- wavefront sums

// Smallest value over the 64 lanes, in every lane (DPP row shifts and row
// broadcasts: no LDS traffic).
__device__ inline int wave_min(int v) {
    v = min(v, __builtin_amdgcn_update_dpp(v, v, 0x111, 0xf, 0xf, false));
    v = min(v, __builtin_amdgcn_update_dpp(v, v, 0x112, 0xf, 0xf, false));
    v = min(v, __builtin_amdgcn_update_dpp(v, v, 0x114, 0xf, 0xf, false));
    v = min(v, __builtin_amdgcn_update_dpp(v, v, 0x118, 0xf, 0xf, false));
    v = min(v, __builtin_amdgcn_update_dpp(v, v, 0x142, 0xf, 0xf, false));
    v = min(v, __builtin_amdgcn_update_dpp(v, v, 0x143, 0xf, 0xf, false));
    return __builtin_amdgcn_readlane(v, 63);
}
__device__ inline int wave_max(int v) { return ~wave_min(~v); }

// Orders a wavefront's own exchange through LDS: what its lanes wrote before
// is what they read after.  The hardware keeps the order of one wavefront's
// LDS operations; the barrier (no instruction) keeps the compiler from
// sending some lanes ahead of others past it, which a fence alone does not.
__device__ inline void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Sum and maximum of a lane's value and that of its other half (lane ^ 32):
// the swap instruction leaves the lower half's value in one register of every
// lane and the upper half's in the other.
__device__ inline float half_sum(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ inline float half_max(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// A value that is the same in every lane, in scalar registers.
__device__ inline int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// --------------------------------------------------------------- positions

// thr is padded with the type's largest value, so 32 are read at a
// time.
__device__ inline int bucket_of(const AttnArgs &a, int rel) {
    int n = 0;
    for (int t = 0; t < a.nb - 1; t += 32)
#pragma unroll
        for (int j = 0; j < 32; ++j) n += rel >= a.thr[t + j];
    return min(n, a.nb - 1);
}
// Entry of the position table for one offset: the table holds every offset
// from below the first threshold to the last one, its ends stand for all
// beyond.
__device__ inline int lut_index(const AttnArgs &a, int rel) {
    return min(max(rel, a.lut_base), a.lut_base + (a.lut_n - 1)) - a.lut_base;
}
__device__ inline int offset_of(int k_pos, int q_pos) { return __builtin_elementwise_sub_sat(k_pos, q_pos); }
// In LDS a table has kLutPad more entries at each end, copies of its ends.
// Where one side's positions run without gaps, up to 64 consecutive offsets
// are then consecutive entries from run_index() on, wherever they lie, and
// an element's entry is a constant away.
constexpr int kLutPad = 64;
__device__ inline int lut_stride(const AttnArgs &a) { return a.lut_n + 2 * kLutPad; }
__device__ inline int run_index(const AttnArgs &a, int first_rel) {
    return min(max(first_rel, a.lut_base - kLutPad), a.lut_base + a.lut_n) - (a.lut_base - kLutPad);
}

// --------------------------------------------------------------- rows of a block

// The queries of a segment and the heads of a subgroup (gs heads of one
// key/value head) form one list of rows, r = query gs + head: a query's
// heads read the same keys, so few queries still fill a tile.
struct RowBlock {
    int b, hk, sub, split, tile;   // segment, key/value head, subgroup, key split, row tile
    int q0, nq, k0, nk;            // the segment's rows
    int h0, gs;                    // first head, heads of the subgroup
};

// The block's place in the batch; false where there is nothing to do.
// Row tiles are the fastest index and xcd_block() keeps neighbours on one
// XCD, so the tiles that read the same keys share an L2.
__device__ inline bool locate(const AttnArgs &a, RowBlock &w) {
    const int n = a.B * a.Hkv * a.subs * a.splits * a.row_tiles;
    int i = xcd_block(n);
    if (i < 0) return false;
    w.tile = i % a.row_tiles; i /= a.row_tiles;
    w.split = i % a.splits; i /= a.splits;
    w.sub = i % a.subs; i /= a.subs;
    w.hk = i % a.Hkv;
    w.b = i / a.Hkv;
    w.h0 = w.hk * a.G + w.sub * a.Gs;
    w.gs = min(a.Gs, a.G - w.sub * a.Gs);
    segment_rows(a.q_ptr, w.b, a.B, a.n_q, a.max_q, a.status, w.q0, w.nq);
    segment_rows(a.k_ptr, w.b, a.B, a.n_k, a.max_k, a.status, w.k0, w.nk);
    // in scalar registers: the tiles' buffer descriptors are made of them
    w.q0 = uniform(w.q0); w.nq = uniform(w.nq);
    w.k0 = uniform(w.k0); w.nk = uniform(w.nk);
    return true;
}

// A bias in log2 units; from -2^20 down it removes the key.  Scores that far
// down have lost their digits beside it, and with every key of a row there the
// log-sum could not hold what the backward pass's p is made of.
__device__ inline float bias_log2(float b) {
    const float x = b * kLog2e;
    return x <= -1048576.0f ? -INFINITY : x;
}

// Position table of the subgroup's heads, in log2 units.
__device__ inline void fill_lut(const AttnArgs &a, const RowBlock &w, float *lut) {
    for (int e = threadIdx.x; e < lut_stride(a); e += blockDim.x) {
        const int bk = bucket_of(a, a.lut_base + min(max(e - kLutPad, 0), a.lut_n - 1));
        for (int g = 0; g < w.gs; ++g) lut[g * lut_stride(a) + e] = bias_log2(a.bias[(int64_t)(w.h0 + g) * a.nb + bk]);
    }
}

// The kept keys of a tile, by every wavefront (lane = key), and their
// positions, which one wavefront leaves in LDS for all.
template <int KT>
struct KeyInfo {
    int4 head;      // smallest and largest of the kept keys, whether all run (first, first + 1, ...), the first
    int pos[KT];
};
template <int KT>
struct KeyLoad {
    int pos, key0, n;
    uint8_t kept;
    __device__ inline void load(const AttnArgs &a, const RowBlock &w, int first_key, bool positions, int lane) {
        key0 = first_key;
        n = min(w.nk - key0, KT);
        const int j = key0 + lane;
        kept = 0;
        pos = j;
        if (positions && a.k_pos && lane < n) pos = a.k_pos[w.k0 + j];
        if (a.keep && lane < n) kept = a.keep[w.k0 + j];
    }
    __device__ inline uint64_t mask(const AttnArgs &a) const {
        return a.keep ? __ballot(kept != 0) : n >= 64 ? ~0ull : (1ull << n) - 1;
    }
    __device__ inline void store(KeyInfo<KT> &k, uint64_t mask, int lane) const {
        const int first = uniform(pos);
        const bool run = !__any(lane < n && (pos != first + lane || abs(pos) >= 1 << 30));
        // (an empty mask: the tile is passed over)
        int lo = first + __ffsll((unsigned long long)mask) - 1, hi = first + 63 - __clzll((long long)mask);
        if (!run) {
            const bool ok = (mask >> lane) & 1;
            lo = wave_min(ok ? pos : 0x7fffffff);
            hi = wave_max(ok ? pos : (int)0x80000000);
        }
        if (lane < KT) k.pos[lane] = pos;
        if (lane == 0) k.head = make_int4(lo, hi, run, first);
    }
};

// Where one side's positions lie, in scalar registers.
struct PosRange {
    int lo, hi, run, first;
};
__device__ inline PosRange uniform_range(int4 v) { return {uniform(v.x), uniform(v.y), uniform(v.z), uniform(v.w)}; }
template <int KT>
__device__ inline bool is_partial(uint64_t mask) { return mask != (KT == 64 ? ~0ull : 0xffffffffull); }

}  // namespace sn
