// Attention of a sequence's newest rows over its pages.
//
//   s_j = scale q.k_j, p_j = exp(s_j - m), o = sum p_j v_j / sum p_j
//
// A unit is a sequence, a key/value head and a tile of 16 NR rows: the rows
// r = t G + g of the sequence's t-th new row and the g-th of the G heads that
// share the keys.  Few rows read many keys, so the bytes of K and V are what
// it costs; they go from memory straight into the registers that the matrix
// instructions read, and nothing of them passes through LDS.
//
// One 16-key block lies in one page (pages hold a multiple of 16), so its base
// is scalar.  Scores are formed transposed, S^T = K Q^T (16x16 products): a
// lane (n = l%16, g = l/16) reads dims of key n and receives row n's scores of
// keys 4g .. 4g+3.  These are the k slots of lane (n, g) in O^T = V^T P^T, so
// the weights stay where they are; for V the lane reads DP/16 neighbouring
// dims of keys 4g .. 4g+3 (a wavefront four whole rows at a time), and the
// pairs of keys that the 16-bit operand wants are one byte permutation each.
//
// Every wavefront walks its own tiles with its own running maximum and sum
// and joins the others' at the end of the piece.  The tiles of all units form
// one line that is cut evenly over the blocks, wherever sequences end; a unit
// that is cut leaves partial rows (fp32), which a second launch joins.
#include <algorithm>
#include <type_traits>

#include "state.h"

namespace sn {
namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float floatx2 __attribute__((ext_vector_type(2)));

// How rows lie in the pages: in their own type, or as codes beside rows of T.
template <typename T_, int CODES_, int DP_, int NR_>
struct Form {
    using T = T_;
    static constexpr int CODES = CODES_, DP = DP_, NR = NR_;
    static constexpr bool F32 = std::is_same<T, float>::value && CODES == SN_CODES_NONE;   // products in fp32
    static constexpr int ES = CODES != SN_CODES_NONE ? 1 : (int)sizeof(T);
    static constexpr int QP = std::is_same<T, float>::value ? 3 : 1;    // bf16 planes of q, exact to 2^-24
    // bf16 planes of the weights: 16 bits beside bf16 rows, 24 beside fp32 ones
    static constexpr int PP = std::is_same<T, float>::value ? 3 : 2;
    // 16-key blocks of a tile: about 8 KB of keys a wavefront where registers allow
    static constexpr int NB = F32 ? (DP == 128 ? 1 : 2) : DP == 128 ? 2 : 4;
    static constexpr int TILE = 16 * NB;
    static constexpr int W = DP / 16;       // dims that a lane reads of a value row
    // registers of a key block and of a value row
    static constexpr int KREGS = F32 ? DP / 4 : ES == 2 ? DP / 8 : DP / 16;
    static constexpr int VREGS = (W * ES + 3) / 4;
};

struct AttendCut {
    int row_tiles;      // of the sequence with the most rows
    int units;          // of a sequence: key/value heads x row tiles
    int blocks;         // that share the line of tiles; 0: every unit is one block's
    int least;          // tiles of a block at the least
};

// A row's statistics in a partial result: maximum (of scores in powers of
// two) and sum.
struct Partials {
    float *o;           // [2 blocks][16 NR][DP], divided by the sum
    float2 *ml;         // [2 blocks][16 NR]
};

// --------------------------------------------------------------- sequences

// What a unit needs of its sequence.
struct Sequence {
    int r0, n, length;      // the call's rows, all rows
    int begin;              // first position that any row sees, down to a multiple of 16
    int tiles;              // tiles of a unit (0: nothing to write)
};
template <class F>
__device__ inline Sequence sequence_of(const CacheArgs &a, int b) {
    Sequence s;
    const int start = a.row_ptr[b], end = a.row_ptr[b + 1];
    s.length = a.lengths[b];
    s.r0 = start;
    s.n = end - start;
    if (start < 0 || end < start || end > a.n_rows || end - start > a.max_rows || (b == 0 && start != 0) ||
        (b == a.B - 1 && end != a.n_rows) ||
        (s.n > 0 && (s.length < 0 || s.length > (int64_t)a.max_pages * a.page || (a.causal && s.length < s.n)))) {
        flag_status(a.status, SN_ERR_INVALID);
        s.n = 0;
    }
    s.begin = a.window > 0 ? max(0, s.length - s.n + 1 - a.window) & ~15 : 0;
    // a row that sees nothing is written too: one tile at the least
    s.tiles = s.n > 0 ? max(1, (s.length - s.begin + F::TILE - 1) / F::TILE) : 0;
    return s;
}
__device__ inline Sequence uniform_sequence(Sequence s) {
    s.r0 = __builtin_amdgcn_readfirstlane(s.r0);
    s.n = __builtin_amdgcn_readfirstlane(s.n);
    s.length = __builtin_amdgcn_readfirstlane(s.length);
    s.begin = __builtin_amdgcn_readfirstlane(s.begin);
    s.tiles = __builtin_amdgcn_readfirstlane(s.tiles);
    return s;
}

// The line of all units' tiles: sequence by sequence, in each unit by unit.
struct Line {
    int64_t total;
    int b;              // the sequence asked for
    int64_t first;      // its first tile in the line
};
// by_tile: the sequence that holds tile `at`; else the first tile of sequence
// `at`.  shared: 8 words of LDS.
template <class F, class At>
__device__ inline Line line_of(const CacheArgs &a, int units, At at_of, bool by_tile, int64_t *shared) {
    Line r{0, 0, 0};
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int64_t at = 0;
    for (int pass = a.B > kThreads ? 0 : 1; pass < 2; ++pass) {     // many sequences: the total first
        int64_t base = 0;
        for (int b0 = 0; b0 < a.B; b0 += kThreads) {
            const int b = b0 + threadIdx.x;
            const int64_t own = b < a.B ? (int64_t)sequence_of<F>(a, b).tiles * units : 0;
            int64_t sum = own;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int64_t below = __shfl_up(sum, o);
                if (lane >= o) sum += below;
            }
            if (lane == 63) shared[wave] = sum;
            __syncthreads();
            int64_t before = base;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                if (w < wave) before += shared[w];
                base += shared[w];
            }
            if (pass == 1) {
                if (a.B <= kThreads) at = at_of(base);
                const int64_t first = before + sum - own;
                if (b < a.B && (by_tile ? at >= first && at < first + own : at == b)) {
                    shared[kWaves] = b;
                    shared[kWaves + 1] = first;
                }
            }
            __syncthreads();
        }
        r.total = base;
        at = at_of(base);
    }
    r.b = __builtin_amdgcn_readfirstlane((int)shared[kWaves]);
    r.first = shared[kWaves + 1];
    return r;
}
// Blocks that share a line of `total` tiles, and the first tile of block i.
__device__ inline int sharers(const AttendCut &c, int64_t total) {
    return (int)min((int64_t)c.blocks, max((int64_t)1, total / c.least));
}
__device__ inline int64_t share(int64_t total, int i, int n) { return total * i / n; }

// --------------------------------------------------------------- products

// Sum and maximum over the four lanes that hold a row.
template <class Op>
__device__ inline float row_join(float v, Op op) {
    auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = op(__uint_as_float(r[0]), __uint_as_float(r[1]));
    r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return op(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ inline float row_max(float v) { return row_join(v, [](float x, float y) { return fmaxf(x, y); }); }
__device__ inline float row_sum(float v) { return row_join(v, [](float x, float y) { return x + y; }); }

// Ends a chain of products whose sums vector instructions read next, in the
// chain's own straight line: where a branch lies between, the compiler was
// seen to count the wait states of its longer side only.
__device__ inline void settle(floatx4 &x) { asm volatile("s_nop 7\n\ts_nop 3" : "+v"(x)); }
template <int N>
__device__ inline void settle(floatx4 (&x)[N]) {
    settle(x[0]);
#pragma unroll
    for (int i = 1; i < N; ++i) asm volatile("" : "+v"(x[i]));
}

__device__ inline bf16x8 pairs8(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __builtin_bit_cast(bf16x8, (u32x4{a, b, c, d}));
}

// Two codes (bytes 2h, 2h + 1) as bf16, which holds either kind exactly.
template <int CODES>
__device__ inline uint32_t codes_to_bf16(uint32_t c, int h) {
    if constexpr (CODES == SN_CODES_E4M3) {
        return h ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)c, 1.0f, true))
                 : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)c, 1.0f, false));
    } else {
        const float x = (float)(int8_t)(c >> (16 * h)), y = (float)(int8_t)(c >> (16 * h + 8));
        return __builtin_amdgcn_perm(__float_as_uint(y), __float_as_uint(x), 0x07060302u);
    }
}

// --------------------------------------------------------------- tiles

template <class F>
struct Tile {
    uint32_t k[F::NB][F::KREGS];
    uint32_t v[F::NB][4][F::VREGS];
    floatx4 ks[F::CODES ? F::NB : 1], vs[F::CODES ? F::NB : 1];
    // dims that a row does not have are not loaded: they stay zero
    __device__ inline Tile() {
#pragma unroll
        for (int b = 0; b < F::NB; ++b) {
#pragma unroll
            for (int c = 0; c < F::KREGS; ++c) k[b][c] = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < F::VREGS; ++c) v[b][i][c] = 0;
        }
    }
};

template <int N>
__device__ inline void load_regs(uint32_t (&r)[N], int at, const char *p) {
    if constexpr (N >= 4) {
        const u32x4 v = *reinterpret_cast<const u32x4 *>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) r[at + i] = v[i];
    } else if constexpr (N == 2) {
        const u32x2 v = *reinterpret_cast<const u32x2 *>(p);
        r[at] = v[0];
        r[at + 1] = v[1];
    } else {
        r[at] = *reinterpret_cast<const uint32_t *>(p);
    }
}

// A lane's places in a 16-key block, and what is the same for a whole unit.
template <class F>
struct Walk {
    const CacheArgs &a;
    const __attribute__((address_space(4))) int32_t *table;     // the sequence's pages
    int hk, key0, end;      // key/value head; first key of tile 0 (a multiple of 16), end of the keys
    uint32_t ko, vo, row;   // byte offsets: the key row's dims, the value rows' dims, a row
    bool kd[4], vd;         // whether the row has the dims
    int g;

    __device__ inline Walk(const CacheArgs &a_) : a(a_) {
        const int lane = threadIdx.x & 63, n = lane & 15;
        g = lane >> 4;
        row = a.Dp * F::ES;
        const int kd0 = F::F32 ? 4 * g : F::ES == 2 || F::DP == 32 ? 8 * g : 16 * g;      // first dim of a load
        ko = n * row + kd0 * F::ES;
        vo = 4 * g * row + n * F::W * F::ES;
        vd = n * F::W < a.Dp;
        const int step = F::F32 ? 16 : F::ES == 2 ? 32 : 64;
#pragma unroll
        for (int c = 0; c < 4; ++c) kd[c] = c * step + kd0 < a.Dp;
    }
    __device__ inline int key_of(int tile, int b) const { return key0 + tile * F::TILE + 16 * b; }
    // Pages of a tile's blocks; blocks behind the last key stand for the last one.
    __device__ inline void pages(int tile, int (&pg)[F::NB]) const {
#pragma unroll
        for (int b = 0; b < F::NB; ++b) pg[b] = table[min(key_of(tile, b), (end - 1) & ~15) >> a.page_shift];
    }
    // Place of a block's first key, in rows of the pages.
    __device__ inline int64_t place(int tile, int b, const int (&pg)[F::NB]) const {
        const int key = min(key_of(tile, b), (end - 1) & ~15);
        const int page = (uint32_t)pg[b] < (uint32_t)a.n_pages ? pg[b] : 0;
        return (((int64_t)page * a.Hkv + hk) << a.page_shift) + (key & (a.page - 1));
    }
    __device__ inline void load_keys(int tile, const int (&pg)[F::NB], Tile<F> &t) const {
#pragma unroll
        for (int b = 0; b < F::NB; ++b) {
            const int64_t at = place(tile, b, pg);
            const char *p = static_cast<const char *>(a.k) + at * row + ko;
            if constexpr (F::KREGS == 2) {
                if (kd[0]) load_regs<2>(t.k[b], 0, p);
            } else {
#pragma unroll
                for (int c = 0; c < F::KREGS; c += 4)       // 64 bytes of a row between two loads
                    if (c / 4 < 4 ? kd[c / 4 & 3] : c / 4 * 16 + 4 * g < a.Dp) load_regs<F::KREGS>(t.k[b], c, p + c / 4 * 64);
            }
            if constexpr (F::CODES != SN_CODES_NONE) t.ks[b] = *reinterpret_cast<const floatx4 *>(a.k_scale + at + 4 * g);
        }
    }
    __device__ inline void load_values(int tile, const int (&pg)[F::NB], Tile<F> &t) const {
#pragma unroll
        for (int b = 0; b < F::NB; ++b) {
            const int64_t at = place(tile, b, pg);
            const char *p = static_cast<const char *>(a.v) + at * row + vo;
            if (vd)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (F::W * F::ES == 2) {
                        t.v[b][i][0] = *reinterpret_cast<const uint16_t *>(p + i * row);
                    } else {
#pragma unroll
                        for (int c = 0; c < F::VREGS; c += 4) load_regs<F::VREGS>(t.v[b][i], c, p + i * row + 4 * c);
                    }
                }
            if constexpr (F::CODES != SN_CODES_NONE) t.vs[b] = *reinterpret_cast<const floatx4 *>(a.v_scale + at + 4 * g);
        }
    }
};

// A unit's rows of queries in a lane: row n of each 16, the dims that its
// lane's keys have.
template <class F>
struct Queries {
    bf16x8 f[F::F32 ? 1 : F::NR][F::F32 ? 1 : F::DP / 32][F::F32 ? 1 : F::QP];
    float x[F::F32 ? F::NR : 1][F::F32 ? F::DP / 4 : 1];

    __device__ inline void load(const CacheArgs &a, const Sequence &s, int hk, int tile) {
        using T = typename F::T;
        const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
#pragma unroll
        for (int nr = 0; nr < F::NR; ++nr) {
            const int r = (tile * F::NR + nr) * 16 + n, t = r / a.G, h = hk * a.G + r % a.G;
            const bool live = t < s.n;
            const T *q = static_cast<const T *>(a.q) + (live ? (s.r0 + t) * a.qs + h * a.qh : 0);
            if constexpr (F::F32) {
#pragma unroll
                for (int i = 0; i < F::DP / 4; ++i) {
                    const int d = i / 4 * 16 + 4 * g + i % 4;
                    x[nr][i] = live && d < a.D ? q[d] : 0.0f;
                }
            } else {
#pragma unroll
                for (int c = 0; c < F::DP / 32; ++c) {
                    // dims of product c: of 8-bit rows a lane reads 16, two products' worth
                    const int d0 = F::ES == 2 || F::DP == 32 ? 32 * c + 8 * g : c / 2 * 64 + 16 * g + c % 2 * 8;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float y = live && d0 + e < a.D ? to_f32(q[d0 + e]) : 0.0f;
#pragma unroll
                        for (int p = 0; p < F::QP; ++p) {
                            f[nr][c][p][e] = (bf16)y;
                            y -= (float)f[nr][c][p][e];
                        }
                    }
                }
            }
        }
    }
};

// Running state of a wavefront: per row the maximum (powers of two), a lane's
// part of the sum, and the rows.
template <class F>
struct State {
    float m[F::NR], l[F::NR];
    floatx4 acc[F::NR][F::W];
    int first[F::NR], last[F::NR];      // positions that row n sees: [first, last)
};

template <class F>
__device__ inline bf16x8 key_operand(const Tile<F> &t, int b, int c) {
    const uint32_t(&k)[F::KREGS] = t.k[b];
    if constexpr (F::CODES == SN_CODES_NONE) {
        return pairs8(k[4 * c], k[4 * c + 1], k[4 * c + 2], k[4 * c + 3]);
    } else {
        const uint32_t x = k[2 * c], y = k[2 * c + 1];
        return pairs8(codes_to_bf16<F::CODES>(x, 0), codes_to_bf16<F::CODES>(x, 1), codes_to_bf16<F::CODES>(y, 0),
                      codes_to_bf16<F::CODES>(y, 1));
    }
}

// Values of blocks b and b + 1 with two dims' pairs of keys: operands of dims
// 2h and 2h + 1 of the lane's W.
template <class F>
__device__ inline void value_operands(const Tile<F> &t, int b, int h, bf16x8 &x, bf16x8 &y) {
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {       // keys 2i and 2i + 1 of the lane's eight
        const uint32_t(&r0)[F::VREGS] = t.v[b + i / 2][2 * (i & 1)];
        const uint32_t(&r1)[F::VREGS] = t.v[b + i / 2][2 * (i & 1) + 1];
        uint32_t p, q;
        if constexpr (F::CODES == SN_CODES_NONE) {
            p = r0[h];
            q = r1[h];
        } else {
            p = codes_to_bf16<F::CODES>(r0[h / 2], h % 2);
            q = codes_to_bf16<F::CODES>(r1[h / 2], h % 2);
        }
        lo[i] = __builtin_amdgcn_perm(q, p, 0x05040100u);
        hi[i] = __builtin_amdgcn_perm(q, p, 0x07060302u);
    }
    x = pairs8(lo[0], lo[1], lo[2], lo[3]);
    y = pairs8(hi[0], hi[1], hi[2], hi[3]);
}

// One tile: scores, the running maximum and sum, and the weighted values; the
// next tile's keys are sent for when the scores are formed, its values when
// they are added, so a wavefront holds one tile and waits for it while the
// others compute.
template <class F>
__device__ inline void take(const Walk<F> &w, Tile<F> &t, int tile, const int (&pg)[F::NB], int next, const int (&next_pg)[F::NB],
                            const Queries<F> &q, State<F> &st, float scale2, int all_first, int all_last) {
    constexpr int NB = F::NB, NR = F::NR;
    const int g = w.g, key = w.key_of(tile, 0);
    int there[NB];      // keys of the block
    bool absent = false;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const bool ok = (uint32_t)pg[b] < (uint32_t)w.a.n_pages;
        there[b] = min(max(w.end - w.key_of(tile, b), 0), 16);
        if (!ok && there[b] > 0) {
            if (threadIdx.x % 64 == 0) flag_status(w.a.status, SN_ERR_INVALID);
            there[b] = 0;
        }
        absent |= there[b] < 16;
    }
    floatx4 s[NR][NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) s[nr][b] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
        if constexpr (F::F32) {
#pragma unroll
            for (int i = 0; i < F::DP / 4; ++i)
#pragma unroll
                for (int nr = 0; nr < NR; ++nr)
                    s[nr][b] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(t.k[b][i]), q.x[nr][i], s[nr][b], 0, 0, 0);
        } else {
#pragma unroll
            for (int c = 0; c < F::DP / 32; ++c) {
                const bf16x8 k = key_operand<F>(t, b, c);
#pragma unroll
                for (int p = F::QP - 1; p >= 0; --p)
#pragma unroll
                    for (int nr = 0; nr < NR; ++nr)
                        s[nr][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, q.f[nr][c][p], s[nr][b], 0, 0, 0);
            }
        }
    }
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) settle(s[nr]);
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                s[nr][b][r] *= scale2;
                if constexpr (F::CODES != SN_CODES_NONE) s[nr][b][r] *= t.ks[b][r];
            }
    if (next >= 0) w.load_keys(next, next_pg, t);
    if (absent || key < all_first || key + F::TILE > all_last) {
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int at = 4 * g + r, pos = key + 16 * b + at;
                    if (at >= there[b] || pos < st.first[nr] || pos >= st.last[nr]) s[nr][b][r] = -INFINITY;
                }
    }
    if (absent) {       // whatever lies in absent rows must not meet a weight of zero
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (4 * g + i >= there[b])
#pragma unroll
                    for (int c = 0; c < F::VREGS; ++c) t.v[b][i][c] = 0;
    }
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
        float top = s[nr][0][0];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r) top = fmaxf(top, s[nr][b][r]);
        top = fmaxf(st.m[nr], row_max(top));
        settle(st.acc[nr]);
        if (__ballot(top != st.m[nr]) != 0) {
            const float keep = top == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(st.m[nr] - top);
            st.l[nr] *= keep;
#pragma unroll
            for (int j = 0; j < F::W; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) st.acc[nr][j][r] *= keep;
            st.m[nr] = top;
        }
        const float base = top == -INFINITY ? 0.0f : top;
        float sum = 0.0f;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float p = __builtin_amdgcn_exp2f(s[nr][b][r] - base);
                sum += p;
                s[nr][b][r] = p;
                if constexpr (F::CODES != SN_CODES_NONE) s[nr][b][r] = p == 0.0f ? 0.0f : p * t.vs[b][r];
            }
        st.l[nr] += sum;
    }
    if constexpr (F::F32) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < F::W; ++j)
#pragma unroll
                    for (int nr = 0; nr < NR; ++nr)
                        st.acc[nr][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(t.v[b][i][j]), s[nr][b][i],
                                                                             st.acc[nr][j], 0, 0, 0);
    } else {
#pragma unroll
        for (int b = 0; b < NB; b += 2) {
            bf16x8 p[NR][F::PP];
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    floatx2 x = {s[nr][b + e / 4][e % 4], s[nr][b + e / 4][e % 4 + 1]};
#pragma unroll
                    for (int n = 0; n < F::PP; ++n) {
                        const bf16x2 y = __builtin_convertvector(x, bf16x2);
                        p[nr][n][e] = y[0];
                        p[nr][n][e + 1] = y[1];
                        x[0] -= (float)y[0];
                        x[1] -= (float)y[1];
                    }
                }
#pragma unroll
            for (int h = 0; h < F::W / 2; ++h) {
                bf16x8 x, y;
                value_operands<F>(t, b, h, x, y);
#pragma unroll
                for (int n = F::PP - 1; n >= 0; --n)
#pragma unroll
                    for (int nr = 0; nr < NR; ++nr) {
                        st.acc[nr][2 * h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, p[nr][n], st.acc[nr][2 * h], 0, 0, 0);
                        st.acc[nr][2 * h + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(y, p[nr][n], st.acc[nr][2 * h + 1], 0, 0, 0);
                    }
            }
        }
    }
    if (next >= 0) w.load_values(next, next_pg, t);
}

// --------------------------------------------------------------- rows apart

// A row by the definition in fp32, of keys [first, last): for rows whose sums
// are not finite.  A masked key's value, infinite or not, is not touched; a
// weight that underflows still lets an infinity through.  The block's threads
// score a key each, then take a dim each.
template <class F>
__device__ inline float row_value(const CacheArgs &a, const void *base, const float *scales, int64_t place, int d) {
    using T = typename F::T;
    if constexpr (F::CODES == SN_CODES_NONE) {
        return to_f32(static_cast<const T *>(base)[place * a.Dp + d]);
    } else {
        const uint8_t c = static_cast<const uint8_t *>(base)[place * a.Dp + d];
        return (F::CODES == SN_CODES_INT8 ? (float)(int8_t)c : e4m3_value(c)) * scales[place];
    }
}
__device__ inline float block_join(float v, bool sum, float *buf) {
    v = sum ? row_sum(v) : row_max(v);
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) {
        const float other = __shfl_xor(v, o);
        v = sum ? v + other : fmaxf(v, other);
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
    __syncthreads();
    v = buf[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v = sum ? v + buf[w] : fmaxf(v, buf[w]);
    return v;
}
// buf: kThreads + kWaves words of LDS.  Returns dim threadIdx.x.
template <class F>
__device__ inline float plain_row(const CacheArgs &a, int b, int hk, int64_t q_at, int first, int last, float scale2, float *buf,
                                  float &m, float &l) {
    using T = typename F::T;
    float *weights = buf + kWaves;
    auto place_of = [&](int j) {
        const int page = a.table[(int64_t)b * a.max_pages + (j >> a.page_shift)];
        return (uint32_t)page < (uint32_t)a.n_pages ? (((int64_t)page * a.Hkv + hk) << a.page_shift) + (j & (a.page - 1))
                                                    : (int64_t)-1;
    };
    auto score = [&](int j, int64_t place) {
        float s = 0.0f;
        for (int d = 0; d < a.D; ++d)
            s += to_f32(static_cast<const T *>(a.q)[q_at + d]) * row_value<F>(a, a.k, a.k_scale, place, d);
        return s * scale2;
    };
    float top = -INFINITY, nan = 0.0f;
    for (int j = first + threadIdx.x; j < last; j += kThreads) {
        const int64_t place = place_of(j);
        if (place < 0) continue;
        const float s = score(j, place);
        top = fmaxf(top, s);
        if (s != s) nan = s;
    }
    m = block_join(top, false, buf);
    nan = block_join(nan, true, buf);
    const float base = m == -INFINITY ? 0.0f : m;
    float sum = 0.0f, o = 0.0f;
    for (int pass = 0; pass < 2; ++pass) {      // the sum, then weights that are at most one
        for (int j0 = first; j0 < last; j0 += kThreads) {
            const int j = j0 + threadIdx.x;
            float e = -1.0f;
            if (j < last) {
                const int64_t place = place_of(j);
                if (place >= 0) e = __builtin_amdgcn_exp2f(score(j, place) - base);
            }
            if (pass == 0) {
                if (e != -1.0f) sum += e;
                continue;
            }
            __syncthreads();
            weights[threadIdx.x] = e;
            __syncthreads();
            if ((int)threadIdx.x < a.D)
                for (int i = 0; i < min(kThreads, last - j0); ++i) {
                    if (weights[i] == -1.0f) continue;
                    const float v = row_value<F>(a, a.v, a.v_scale, place_of(j0 + i), threadIdx.x), p = weights[i] / l;
                    o += v * (fabsf(v) < INFINITY ? p : fmaxf(p, 1e-38f));
                }
        }
        if (pass == 0) l = block_join(sum, true, buf) + nan;
    }
    return o + nan;
}

// --------------------------------------------------------------- a piece of a unit

template <class F>
struct Exchange {
    float ml[kWaves][16 * F::NR][2];
    float rows[kWaves][16 * F::NR][F::DP + 4];
    float stats[16 * F::NR][2];
    int odd[16 * F::NR], any;
    float plain[kThreads + kWaves];
};

// Keys of tiles [t0, t1) of a unit.  slot < 0: the whole unit, its rows are
// finished; else a partial result.
template <class F>
__device__ inline void piece(const CacheArgs &a, const AttendCut &c, int b, const Sequence &s, int unit, int t0, int t1, int slot,
                             const Partials &parts, typename F::T *o, float *lse, Exchange<F> &x) {
    // the same in the whole block, in scalar registers
    b = __builtin_amdgcn_readfirstlane(b);
    unit = __builtin_amdgcn_readfirstlane(unit);
    t0 = __builtin_amdgcn_readfirstlane(t0);
    t1 = __builtin_amdgcn_readfirstlane(t1);
    slot = __builtin_amdgcn_readfirstlane(slot);
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int hk = unit / c.row_tiles, tile = unit % c.row_tiles, rows = min(s.n * a.G - tile * 16 * F::NR, 16 * F::NR);
    if (rows <= 0) return;      // fewer rows than the sequence with the most
    const float scale2 = a.scale * kLog2e;
    Walk<F> w(a);
    w.table = (const __attribute__((address_space(4))) int32_t *)(uintptr_t)(a.table + (int64_t)b * a.max_pages);
    w.hk = hk;
    w.key0 = s.begin + t0 * F::TILE;
    w.end = min(s.begin + t1 * F::TILE, s.length);
    // positions that a row t sees
    auto last_of = [&](int t) { return a.causal ? s.length - s.n + t + 1 : s.length; };
    auto first_of = [&](int t) { return a.window > 0 ? max(0, last_of(t) - a.window) : 0; };
    State<F> st;
#pragma unroll
    for (int nr = 0; nr < F::NR; ++nr) {
        const int t = min((tile * F::NR + nr) * 16 + n, s.n * a.G - 1) / a.G;
        st.first[nr] = first_of(t);
        st.last[nr] = last_of(t);
        st.m[nr] = -INFINITY;
        st.l[nr] = 0.0f;
#pragma unroll
        for (int j = 0; j < F::W; ++j) st.acc[nr][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    const int all_first = first_of((tile * 16 * F::NR + rows - 1) / a.G), all_last = last_of(tile * 16 * F::NR / a.G);
    const int tiles = w.end > w.key0 ? (w.end - w.key0 + F::TILE - 1) / F::TILE : 0;
    if (wave < tiles) {
        Queries<F> q;
        Tile<F> tile_regs;
        int pg[F::NB], next_pg[F::NB];
        w.pages(wave, pg);
        w.load_keys(wave, pg, tile_regs);
        w.load_values(wave, pg, tile_regs);
        q.load(a, s, hk, tile);
        w.pages(min(wave + kWaves, tiles - 1), next_pg);
        for (int i = wave; i < tiles; i += kWaves) {
            const int next = i + kWaves;
            int after[F::NB];       // pages are asked for two tiles ahead
            w.pages(min(next + kWaves, tiles - 1), after);
            take<F>(w, tile_regs, i, pg, next < tiles ? next : -1, next_pg, q, st, scale2, all_first, all_last);
#pragma unroll
            for (int b = 0; b < F::NB; ++b) {
                pg[b] = next_pg[b];
                next_pg[b] = after[b];
            }
        }
    }
    // the wavefronts' rows on one maximum, then their sum
    __syncthreads();
#pragma unroll
    for (int nr = 0; nr < F::NR; ++nr) {
        const float l = row_sum(st.l[nr]);
        if (g == 0) {
            x.ml[wave][nr * 16 + n][0] = st.m[nr];
            x.ml[wave][nr * 16 + n][1] = l;
        }
        if (threadIdx.x < 16) x.odd[nr * 16 + n] = 0;
    }
    if (threadIdx.x == 0) x.any = 0;
    __syncthreads();
#pragma unroll
    for (int nr = 0; nr < F::NR; ++nr) {
        const int r = nr * 16 + n;
        float top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int v = 0; v < kWaves; ++v) top = fmaxf(top, x.ml[v][r][0]);
        const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
        for (int v = 0; v < kWaves; ++v) sum += x.ml[v][r][1] * __builtin_amdgcn_exp2f(x.ml[v][r][0] - base);
        const float keep = __builtin_amdgcn_exp2f(st.m[nr] - base) / (sum == 0.0f ? 1.0f : sum);
        settle(st.acc[nr]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < F::W; ++j) x.rows[wave][r][(4 * g + i) * F::W + j] = st.acc[nr][j][i] * keep;
        if (wave == 0 && g == 0) {
            x.stats[r][0] = top;
            x.stats[r][1] = sum;
        }
    }
    __syncthreads();
    auto put = [&](int r, int d, float v) {
        if (slot >= 0) {
            parts.o[((int64_t)slot * 16 * F::NR + r) * F::DP + d] = v;
        } else {
            const int row = tile * 16 * F::NR + r, t = row / a.G, h = hk * a.G + row % a.G;
            o[((int64_t)(s.r0 + t) * a.H + h) * a.D + d] = (typename F::T)v;
        }
    };
    auto put_stats = [&](int r, float m, float l) {
        if (slot >= 0) {
            parts.ml[(int64_t)slot * 16 * F::NR + r] = make_float2(m, l);
        } else if (lse) {
            const int row = tile * 16 * F::NR + r, t = row / a.G, h = hk * a.G + row % a.G;
            lse[(int64_t)(s.r0 + t) * a.H + h] = m == -INFINITY ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
        }
    };
    for (int i = threadIdx.x; i < rows * F::DP; i += kThreads) {
        const int r = i / F::DP, d = i % F::DP;
        float v = 0.0f;
#pragma unroll
        for (int u = 0; u < kWaves; ++u) v += x.rows[u][r][d];
        if (!(fabsf(v) < INFINITY) && d < a.D) {
            x.odd[r] = 1;
            x.any = 1;
        }
        if (d < a.D) put(r, d, v);
    }
    if ((int)threadIdx.x < rows) put_stats(threadIdx.x, x.stats[threadIdx.x][0], x.stats[threadIdx.x][1]);
    __syncthreads();
    if (!x.any) return;
    for (int r = 0; r < rows; ++r) {
        if (!x.odd[r]) continue;
        const int row = tile * 16 * F::NR + r, t = row / a.G, h = hk * a.G + row % a.G;
        float m, l;
        const float v = plain_row<F>(a, b, hk, (s.r0 + t) * a.qs + h * a.qh, max(first_of(t), w.key0), min(last_of(t), w.end),
                                     scale2, x.plain, m, l);
        if ((int)threadIdx.x < a.D) put(r, threadIdx.x, v);
        if (threadIdx.x == 0) put_stats(r, m, l);
        __syncthreads();
    }
}

template <class F>
__global__ __launch_bounds__(kThreads, 2) void attend_kernel(CacheArgs a, AttendCut c, Partials parts, typename F::T *o, float *lse) {
    __shared__ Exchange<F> x;
    __shared__ int64_t words[kWaves + 2];
    if (c.blocks == 0) {        // a unit a block
        const int id = xcd_block(a.B * c.units);
        if (id < 0) return;
        const int b = id / c.units;
        const Sequence s = uniform_sequence(sequence_of<F>(a, b));
        if (s.tiles > 0) piece<F>(a, c, b, s, id % c.units, 0, s.tiles, -1, parts, o, lse, x);
        return;
    }
    const int id = xcd_block(c.blocks);
    if (id < 0) return;
    int n = 1;
    const Line line = line_of<F>(a, c.units, [&](int64_t total) {
        n = sharers(c, total);
        return id < n ? share(total, id, n) : (int64_t)-1; }, true, words);
    if (id >= n || line.total == 0) return;
    int64_t at = share(line.total, id, n);
    const int64_t end = share(line.total, id + 1, n);
    int64_t first = line.first;
    for (int b = line.b; at < end; ++b) {
        const Sequence s = uniform_sequence(sequence_of<F>(a, b));
        if (s.tiles == 0) continue;
        while (at < end && at < first + (int64_t)s.tiles * c.units) {
            const int unit = (int)((at - first) / s.tiles);
            const int64_t u0 = first + (int64_t)unit * s.tiles, u1 = u0 + s.tiles, stop = min(u1, end);
            // the block's first piece may begin inside a unit; else, if it is not whole, its last ends inside
            const int slot = at == u0 && stop == u1 ? -1 : at == u0 ? 2 * id + 1 : 2 * id;
            piece<F>(a, c, b, s, unit, (int)(at - u0), (int)(stop - u0), slot, parts, o, lse, x);
            at = stop;
        }
        first += (int64_t)s.tiles * c.units;
    }
}

// Units that were cut: their rows' partial results on one maximum, in order.
template <class F>
__global__ __launch_bounds__(kThreads) void attend_join_kernel(CacheArgs a, AttendCut c, Partials parts, typename F::T *o, float *lse) {
    __shared__ int64_t words[kWaves + 2];
    const int b = blockIdx.x / c.units, unit = blockIdx.x % c.units;
    const Line line = line_of<F>(a, c.units, [&](int64_t) { return (int64_t)b; }, false, words);
    const Sequence s = uniform_sequence(sequence_of<F>(a, b));
    if (s.tiles == 0) return;
    const int n = sharers(c, line.total);
    const int64_t u0 = line.first + (int64_t)unit * s.tiles, u1 = u0 + s.tiles;
    // the block of tile t is the last one whose share begins at or before it
    auto block_of = [&](int64_t t) { return (int)(((t + 1) * n - 1) / line.total); };
    const int i0 = block_of(u0), i1 = block_of(u1 - 1);
    if (i0 == i1) return;
    const int hk = unit / c.row_tiles, tile = unit % c.row_tiles, rows = min(s.n * a.G - tile * 16 * F::NR, 16 * F::NR);
    auto slot_of = [&](int i) { return share(line.total, i, n) <= u0 ? 2 * i + 1 : 2 * i; };
    for (int i = threadIdx.x; i < rows * F::DP; i += kThreads) {
        const int r = i / F::DP, d = i % F::DP;
        const int row = tile * 16 * F::NR + r, t = row / a.G, h = hk * a.G + row % a.G;
        float top = -INFINITY, sum = 0.0f, v = 0.0f;
        for (int k = i0; k <= i1; ++k) top = fmaxf(top, parts.ml[(int64_t)slot_of(k) * 16 * F::NR + r].x);
        const float base = top == -INFINITY ? 0.0f : top;
        for (int k = i0; k <= i1; ++k) {
            const int64_t at = (int64_t)slot_of(k) * 16 * F::NR + r;
            const float2 ml = parts.ml[at];
            if (ml.y == 0.0f) continue;
            const float e = ml.y * __builtin_amdgcn_exp2f(ml.x - base), x = parts.o[at * F::DP + d];
            sum += e;
            v += x * (fabsf(x) < INFINITY ? e : fmaxf(e, 1e-38f));
        }
        if (d < a.D) o[((int64_t)(s.r0 + t) * a.H + h) * a.D + d] = (typename F::T)(sum == 0.0f ? 0.0f : v / sum);
        if (lse && d == 0)
            lse[(int64_t)(s.r0 + t) * a.H + h] = top == -INFINITY ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * kLn2;
    }
}

// --------------------------------------------------------------- launches

constexpr int kSharers = 512;       // two blocks on each CU

inline int rows_per_tile(int rows) { return rows > 16 ? 2 : 1; }

AttendCut cut_of(int B, int Hkv, int64_t rows, int64_t capacity, int tile_keys) {
    AttendCut c;
    const int per = 16 * rows_per_tile((int)std::min<int64_t>(rows, 64));
    c.row_tiles = (int)std::max<int64_t>(1, (rows + per - 1) / per);
    c.units = Hkv * c.row_tiles;
    c.least = kWaves;
    c.blocks = kSharers;
    const int64_t tiles = (capacity + tile_keys - 1) / tile_keys + 1;
    if ((int64_t)B * c.units >= 16 * kSharers || tiles <= 4 * kWaves) c.blocks = 0;
    return c;
}

// A cut for sizes alone; the launch makes its own with the form's tile.
AttendCut cut_of(const sn_cache &op) {
    return cut_of(op.n_sequences, op.n_kv_heads, (int64_t)op.max_rows * (op.n_heads / op.n_kv_heads), INT32_MAX, 16);
}

inline int padded(int D) { return D <= 32 ? 32 : D <= 64 ? 64 : 128; }

template <class F>
sn_status launch(const CacheArgs &a, void *o, float *lse, char *ws, hipStream_t s) {
    using T = typename F::T;
    const AttendCut c = cut_of(a.B, a.Hkv, (int64_t)a.max_rows * a.G, (int64_t)a.max_pages * a.page, F::TILE);
    Partials parts;
    parts.ml = reinterpret_cast<float2 *>(ws + kWsBase);
    parts.o = reinterpret_cast<float *>(ws + kWsBase + sizeof(float2) * 2 * kSharers * 16 * F::NR);
    ProfScope prof(K_CACHE_ATTEND, s);
    const int grid = xcd_grid(c.blocks ? c.blocks : a.B * c.units);
    attend_kernel<F><<<grid, kThreads, 0, s>>>(a, c, parts, static_cast<T *>(o), lse);
    SN_TRY(launch_status());
    if (c.blocks) attend_join_kernel<F><<<a.B * c.units, kThreads, 0, s>>>(a, c, parts, static_cast<T *>(o), lse);
    return launch_status();
}
template <typename T, int CODES, int DP>
sn_status launch(const CacheArgs &a, void *o, float *lse, char *ws, hipStream_t s) {
    return rows_per_tile(std::min<int64_t>((int64_t)a.max_rows * a.G, 64)) == 2 ? launch<Form<T, CODES, DP, 2>>(a, o, lse, ws, s)
                                                                      : launch<Form<T, CODES, DP, 1>>(a, o, lse, ws, s);
}
template <typename T, int CODES>
sn_status launch(const CacheArgs &a, void *o, float *lse, char *ws, hipStream_t s) {
    if (a.Dp <= 32) return launch<T, CODES, 32>(a, o, lse, ws, s);
    if (a.Dp <= 64) return launch<T, CODES, 64>(a, o, lse, ws, s);
    return launch<T, CODES, 128>(a, o, lse, ws, s);
}
template <typename T>
sn_status launch(const CacheArgs &a, int codes, void *o, float *lse, char *ws, hipStream_t s) {
    if (codes == SN_CODES_INT8) return launch<T, SN_CODES_INT8>(a, o, lse, ws, s);
    if (codes == SN_CODES_E4M3) return launch<T, SN_CODES_E4M3>(a, o, lse, ws, s);
    return launch<T, SN_CODES_NONE>(a, o, lse, ws, s);
}

}  // namespace

// Units are blocks of their own, or of the join.
bool attend_fits(const sn_cache &op) {
    return grid_fits((int64_t)op.n_sequences * cut_of(op).units + kXcds, kThreads);
}

size_t attend_workspace(const sn_cache &op) {
    const size_t rows = (size_t)2 * kSharers * 16 * rows_per_tile((int)std::min<int64_t>((int64_t)op.max_rows * (op.n_heads / op.n_kv_heads), 64));
    return kWsBase + rows * (sizeof(float2) + padded(op.head_dim) * sizeof(float));
}

sn_status cache_attend(const CacheArgs &a, int dtype, int codes, void *o, float *lse, char *ws, hipStream_t s) {
    return dtype == SN_F32 ? launch<float>(a, codes, o, lse, ws, s) : launch<bf16>(a, codes, o, lse, ws, s);
}

}  // namespace sn
