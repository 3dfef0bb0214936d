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
// that is cut leaves partial rows (fp32), which a second launch joins.  (Every
// sequence has as many units as the one with the most rows: those without rows
// end at once, but their tiles are on the line.  8 x 20000 keys, 32/8 heads of
// 128, bf16: 112 us for single rows, 272 where one sequence has 32.)
//
// Measured (one new row a sequence): 32 x <= 20000 keys, 32/8 heads of 128, bf16,
// 1.65 GB: 262 us, 6.3 TB/s, where a copy reaches 5.2; the same in e4m3, 0.85 GB:
// 154 us, 5.5 TB/s.  Short histories are bound by a chain of dependent reads
// (lengths, pages, keys) and by the rounds a wavefront takes: 271 keys, 4 x 32
// fp32: 6.7 us; 64 x <= 1076 keys, 8 x 16 int8 beside fp32 rows: 15 us, half of it
// vector instructions.
#include <algorithm>
#include <type_traits>

#include "state.h"

namespace sn {
namespace {

constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float floatx2 __attribute__((ext_vector_type(2)));

// How rows lie in the pages: in their own type, or as codes beside rows of T.
template <typename T_, int CODES_, int DP_, int NR_, bool PAST_ = false>
struct Form {
    using T = T_;
    static constexpr int CODES = CODES_, DP = DP_, NR = NR_;
    static constexpr bool F32 = std::is_same<T, float>::value && CODES == SN_CODES_NONE;   // products in fp32
    static constexpr int ES = CODES != SN_CODES_NONE ? 1 : (int)sizeof(T);
    static constexpr int QP = std::is_same<T, float>::value ? 3 : 1;    // bf16 planes of q, exact to 2^-24
    static constexpr int PP = 3;        // of the weights, which keep their 24 bits
    // 16-key blocks of a tile: about 8 KB of keys a wavefront where registers allow
    static constexpr int NB = F32 ? (DP == 128 ? 1 : DP == 16 ? 4 : 2) : DP == 128 || (ES == 1 && DP == 32) ? 2 : 4;
    static constexpr int TILE = 16 * NB;
    static constexpr int W = DP / 16;       // dims that a lane reads of a value row
    // registers of a key block and of a value row
    static constexpr int KREGS = F32 ? DP / 4 : ES == 2 ? DP / 8 : DP / 16;
    static constexpr int VREGS = (W * ES + 3) / 4;
    static constexpr int AUX = PAST_ ? 2 : 0;       // of a load: 2 goes past the caches
    // blocks that a CU holds: short rows of one tile fit 128 registers
    static constexpr int BLOCKS = DP <= 32 && NR == 1 ? 2 : 1;
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
    int2 *cuts;         // [sequence][unit]: first and last block that share the unit
    float2 *ml;         // [2 blocks][16 NR]
    float *o;           // [2 blocks][16 NR][DP], divided by the sum
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
    s.begin = s.n > 0 && a.window > 0 ? max(0, s.length - s.n + 1 - a.window) & ~15 : 0;
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

// The line of all units' tiles, sequence by sequence, in each unit by unit,
// cut into n shares that differ by one tile at most.  (The host keeps a line
// below 2^31 tiles.)
struct Line {
    int total, part;        // tiles; tiles of the smaller shares
    int n, more;            // shares; the first `more` have one tile more
    __device__ inline Line(const AttendCut &c, int total_) : total(total_) {
        n = min(c.blocks, max(1, total / c.least));
        part = total / n;
        more = total - part * n;
    }
    __device__ inline int begin(int i) const { return part * i + min(i, more); }
    __device__ inline int share_of(int tile) const {
        const int wide = (part + 1) * more;
        return tile < wide ? tile / (part + 1) : more + (tile - wide) / part;
    }
};

// The sequence in which block `id`'s share begins, that sequence's first tile
// in the line and the line's length.  Every wavefront finds them by itself, a
// lane for a sequence.
struct Start {
    int total, first, b;
    Sequence s;
};
template <class F>
__device__ inline Start start_of(const CacheArgs &a, const AttendCut &c, int id) {
    const int lane = threadIdx.x & 63;
    Start r{0, 0, -1, {}};
    int at = -1;
    for (int pass = a.B > 64 ? 0 : 1; pass < 2; ++pass) {       // many sequences: the total first
        int base = 0;
        for (int b0 = 0; b0 < a.B; b0 += 64) {
            Sequence s;
            s.tiles = 0;
            if (b0 + lane < a.B) s = sequence_of<F>(a, b0 + lane);
            const int own = s.tiles * c.units;
            int sum = own;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int below = __shfl_up(sum, o);
                if (lane >= o) sum += below;
            }
            const int first = base + sum - own;
            base += __builtin_amdgcn_readlane(sum, 63);
            if (pass == 0) continue;
            if (a.B <= 64) {
                const Line line(c, base);
                at = id < line.n ? line.begin(id) : -1;
            }
            const uint64_t here = __ballot(at >= first && at < first + own);
            if (here != 0) {
                const int l = __builtin_ctzll(here);
                r.b = b0 + l;
                r.first = __builtin_amdgcn_readlane(first, l);
                r.s.r0 = __builtin_amdgcn_readlane(s.r0, l);
                r.s.n = __builtin_amdgcn_readlane(s.n, l);
                r.s.length = __builtin_amdgcn_readlane(s.length, l);
                r.s.begin = __builtin_amdgcn_readlane(s.begin, l);
                r.s.tiles = __builtin_amdgcn_readlane(s.tiles, l);
            }
        }
        r.total = base;
        if (pass == 0) {
            const Line line(c, base);
            at = id < line.n ? line.begin(id) : -1;
        }
    }
    return r;
}

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
};

// Blocks are read through buffer descriptors: the base is scalar, a lane's
// offset a constant of the walk, and dims that a row does not have are asked
// for out of range, which gives zeros without a branch.
constexpr uint32_t kNowhere = 0x80000000u;
__device__ inline __amdgpu_buffer_rsrc_t block_at(const void *p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, 0x7fffffff, 0x00020000);
}
template <int BYTES, int AUX>
__device__ inline void load_bytes(uint32_t *r, __amdgpu_buffer_rsrc_t block, uint32_t lane, int offset) {
    if constexpr (BYTES == 2) {
        r[0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(block, lane, offset, AUX);
    } else if constexpr (BYTES == 4) {
        r[0] = __builtin_amdgcn_raw_buffer_load_b32(block, lane, offset, AUX);
    } else if constexpr (BYTES == 8) {
        const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(block, lane, offset, AUX));
        r[0] = v[0];
        r[1] = v[1];
    } else {
        const u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(block, lane, offset, AUX));
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = v[i];
        if constexpr (BYTES == 32) load_bytes<16, AUX>(r + 4, block, lane + 16, offset);
    }
}

// A lane's places in a 16-key block, and what is the same for a whole unit.
template <class F>
struct Walk {
    const CacheArgs &a;
    const __attribute__((address_space(4))) int32_t *table;     // the sequence's pages
    int hk, key0;           // key/value head; first key of tile 0 (a multiple of 16)
    int from, end;          // keys that some row of the unit sees
    int row;                // bytes of a row
    static constexpr int KBYTES = F::KREGS == 2 ? 8 : 16, KLOADS = F::KREGS * 4 / KBYTES;
    uint32_t ko[KLOADS], vo;    // a lane's offsets in a block: its key row's dims, its value row's dims
    int g;

    __device__ inline Walk(const CacheArgs &a_) : a(a_) {
        const int lane = threadIdx.x & 63, n = lane & 15;
        g = lane >> 4;
        row = a.Dp * F::ES;
        constexpr int per = KBYTES / F::ES;                     // dims of a load; four lanes have a row's next 4 per
#pragma unroll
        for (int c = 0; c < KLOADS; ++c) {
            const int d = 4 * per * c + per * g;
            ko[c] = d < a.Dp ? n * row + d * F::ES : kNowhere;
        }
        vo = n * F::W < a.Dp ? 4 * g * row + n * F::W * F::ES : kNowhere;
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
            const __amdgpu_buffer_rsrc_t block = block_at(static_cast<const char *>(a.k) + at * row);
#pragma unroll
            for (int c = 0; c < KLOADS; ++c) load_bytes<KBYTES, F::AUX>(&t.k[b][c * KBYTES / 4], block, ko[c], 0);
            if constexpr (F::CODES != SN_CODES_NONE)
                t.ks[b] = __builtin_bit_cast(floatx4, __builtin_amdgcn_raw_buffer_load_b128(block_at(a.k_scale + at), 16 * g, 0, 0));
        }
    }
    __device__ inline void load_values(int tile, const int (&pg)[F::NB], Tile<F> &t) const {
#pragma unroll
        for (int b = 0; b < F::NB; ++b) {
            const int64_t at = place(tile, b, pg);
            const __amdgpu_buffer_rsrc_t block = block_at(static_cast<const char *>(a.v) + at * row);
#pragma unroll
            for (int i = 0; i < 4; ++i) load_bytes<F::W * F::ES, F::AUX>(t.v[b][i], block, vo, i * row);
            if constexpr (F::CODES != SN_CODES_NONE)
                t.vs[b] = __builtin_bit_cast(floatx4, __builtin_amdgcn_raw_buffer_load_b128(block_at(a.v_scale + at), 16 * g, 0, 0));
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
                for (int i = 0; i < F::DP / 4; i += 4) {
                    const int d = i / 4 * 16 + 4 * g;
                    floatx4 y = {0.0f, 0.0f, 0.0f, 0.0f};
                    if (a.q_vec) {
                        if (live && d < a.D) y = *reinterpret_cast<const floatx4 *>(q + d);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (live && d + e < a.D) y[e] = q[d + e];
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[nr][i + e] = y[e];
                }
            } else {
#pragma unroll
                for (int c = 0; c < F::DP / 32; ++c) {
                    // dims of product c: of 8-bit rows a lane reads 16, two products' worth
                    const int d0 = F::ES == 2 || F::DP == 32 ? 32 * c + 8 * g : c / 2 * 64 + 16 * g + c % 2 * 8;
                    T raw[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) raw[e] = (T)0.0f;
                    if (a.q_vec) {
                        typedef T vec_t __attribute__((ext_vector_type(16 / sizeof(T))));
                        if (live && d0 < a.D)
#pragma unroll
                            for (int e = 0; e < 8; e += 16 / sizeof(T)) {
                                const vec_t y = *reinterpret_cast<const vec_t *>(q + d0 + e);
#pragma unroll
                                for (int i = 0; i < (int)(16 / sizeof(T)); ++i) raw[e + i] = y[i];
                            }
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (live && d0 + e < a.D) raw[e] = q[d0 + e];
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float y = to_f32(raw[e]);
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
    int from[NB], there[NB];    // the block's keys that are there: [from, there)
    bool absent = false;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const bool ok = (uint32_t)pg[b] < (uint32_t)w.a.n_pages;
        there[b] = min(max(w.end - w.key_of(tile, b), 0), 16);
        from[b] = max(w.from - w.key_of(tile, b), 0);
        if (!ok && there[b] > 0) {
            if (threadIdx.x % 64 == 0) flag_status(w.a.status, SN_ERR_INVALID);
            there[b] = 0;
        }
        absent |= there[b] < 16 || from[b] > 0;
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
                    if (at >= there[b] || pos < st.first[nr] || pos >= st.last[nr]) {
                        s[nr][b][r] = -INFINITY;
                        // its scale may be anything; with one tile of rows it is this row's alone
                        if constexpr (F::CODES != SN_CODES_NONE && NR == 1) t.vs[b][r] = 0.0f;
                    }
                }
    }
    if (absent) {       // whatever lies in absent rows must not meet a weight of zero
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (4 * g + i >= there[b] || 4 * g + i < from[b])
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
                // a seen key's scale counts whatever its weight
                if constexpr (F::CODES != SN_CODES_NONE)
                    s[nr][b][r] = NR > 1 && s[nr][b][r] == -INFINITY ? 0.0f : p * t.vs[b][r];
                else
                    s[nr][b][r] = p;
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
    if (m == INFINITY && nan == 0.0f) l = 1.0f;     // an infinite score: its log-sum is infinite, its row is not a number
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
    // positions that a row t sees, and those that some row of the unit does
    auto last_of = [&](int t) { return a.causal ? s.length - s.n + t + 1 : s.length; };
    auto first_of = [&](int t) { return a.window > 0 ? max(0, last_of(t) - a.window) : 0; };
    const int t_first = tile * 16 * F::NR / a.G, t_last = (tile * 16 * F::NR + rows - 1) / a.G;
    w.key0 = s.begin + t0 * F::TILE;
    w.from = first_of(t_first);
    w.end = min(s.begin + t1 * F::TILE, last_of(t_last));
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
    const int all_first = first_of(t_last), all_last = last_of(t_first);
    const int tiles = w.end > w.key0 ? (w.end - w.key0 + F::TILE - 1) / F::TILE : 0;
    const int mine = max(w.from - w.key0, 0) / F::TILE + wave;      // the wavefront's first tile
    if (mine < tiles) {
        Queries<F> q;
        Tile<F> tile_regs;
        int pg[F::NB], next_pg[F::NB];
        w.pages(mine, pg);
        q.load(a, s, hk, tile);
        w.load_keys(mine, pg, tile_regs);
        w.load_values(mine, pg, tile_regs);
        w.pages(min(mine + kWaves, tiles - 1), next_pg);
        for (int i = mine; i < tiles; i += kWaves) {
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
            lse[(int64_t)(s.r0 + t) * a.H + h] = (m + __builtin_amdgcn_logf(l)) * kLn2;      // no key: -inf and the log of 0
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
        if (d < a.D || slot >= 0) put(r, d, v);
    }
    if ((int)threadIdx.x < rows) {
        const int r = threadIdx.x, t = (tile * 16 * F::NR + r) / a.G;
        put_stats(r, x.stats[r][0], x.stats[r][1]);
        // keys to see and no score above -inf
        if (x.stats[r][0] == -INFINITY && max(first_of(t), w.key0) < min(last_of(t), w.end)) {
            x.odd[r] = 1;
            x.any = 1;
        }
    }
    __syncthreads();
    if (!x.any) return;
    for (int r = 0; r < rows; ++r) {
        if (!x.odd[r]) continue;
        const int row = tile * 16 * F::NR + r, t = row / a.G, h = hk * a.G + row % a.G;
        float m, l;
        float v = plain_row<F>(a, b, hk, (s.r0 + t) * a.qs + h * a.qh, max(first_of(t), w.key0), min(last_of(t), w.end),
                               scale2, x.plain, m, l);
        // every score of the piece is -inf: no weight beside other pieces; the join knows the row by its sum if there are none
        if (slot >= 0 && m == -INFINITY && l == 0.0f && v != v) {
            v = 0.0f;
            l = 1.0f;
        }
        if ((int)threadIdx.x < a.D) put(r, threadIdx.x, v);
        if (threadIdx.x == 0) put_stats(r, m, l);
        __syncthreads();
    }
}

template <class F>
__global__ __launch_bounds__(kThreads, 2 * F::BLOCKS) void attend_kernel(CacheArgs a, AttendCut c, Partials parts, typename F::T *o, float *lse) {
    __shared__ Exchange<F> x;
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
    const Start start = start_of<F>(a, c, id);
    if (start.b < 0) return;        // fewer shares than blocks, or no tiles
    const Line line(c, start.total);
    int at = line.begin(id), first = start.first, b = start.b;
    const int end = line.begin(id + 1);
    Sequence s = start.s;
    while (true) {
        while (s.tiles > 0 && at < end && at < first + s.tiles * c.units) {
            const int unit = (at - first) / s.tiles, u0 = first + unit * s.tiles, u1 = u0 + s.tiles, stop = min(u1, end);
            // the block's first piece may begin inside a unit; else, if it is not whole, its last ends inside
            const int slot = at == u0 && stop == u1 ? -1 : at == u0 ? 2 * id + 1 : 2 * id;
            if (at == u0 && threadIdx.x == 0)
                parts.cuts[(int64_t)b * c.units + unit] = make_int2(id, stop == u1 ? id : line.share_of(u1 - 1));
            piece<F>(a, c, b, s, unit, at - u0, stop - u0, slot, parts, o, lse, x);
            at = stop;
        }
        first += s.tiles * c.units;
        if (at >= end || ++b >= a.B) return;
        s = uniform_sequence(sequence_of<F>(a, b));
    }
}

// Units that were cut: their rows' partial results on one maximum, in order.
constexpr int kJoinThreads = 256, kJoinWeights = 4096;
template <class F>
__global__ __launch_bounds__(kJoinThreads) void attend_join_kernel(CacheArgs a, AttendCut c, Partials parts, typename F::T *o, float *lse) {
    constexpr int R = 16 * F::NR;
    __shared__ float weights[kJoinWeights], sums[R][2];
    __shared__ alignas(16) float held[kJoinThreads * 4];
    const int b = blockIdx.x / c.units, unit = blockIdx.x % c.units;
    const int2 cut = parts.cuts[blockIdx.x];
    const Sequence s = uniform_sequence(sequence_of<F>(a, b));
    if (s.tiles == 0) return;       // no block wrote here
    const int hk = unit / c.row_tiles, tile = unit % c.row_tiles, rows = min(s.n * a.G - tile * R, R), n = cut.y - cut.x + 1;
    if (n <= 1 || rows <= 0) return;
    // the first piece is its block's last one, the others are their blocks' first
    auto slot_of = [&](int k) { return k == 0 ? 2 * cut.x + 1 : 2 * (cut.x + k); };
    auto at_of = [&](int k, int r) { return (int64_t)slot_of(k) * R + r; };
    // a row's maximum and sum: the sixteen lanes of a group
    for (int r = threadIdx.x / 16; r < rows; r += kJoinThreads / 16) {
        float top = -INFINITY, sum = 0.0f;
        for (int k = threadIdx.x % 16; k < n; k += 16) top = fmaxf(top, parts.ml[at_of(k, r)].x);
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
        const float base = top == -INFINITY ? 0.0f : top;
        for (int k = threadIdx.x % 16; k < n; k += 16) {
            const float2 ml = parts.ml[at_of(k, r)];
            sum += ml.y * (ml.x == top ? 1.0f : __builtin_amdgcn_exp2f(ml.x - base));      // infinite ones too
        }
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) sum += __shfl_xor(sum, o);
        if (threadIdx.x % 16 == 0) {
            sums[r][0] = top;
            sums[r][1] = sum;
        }
    }
    // four elements a thread; where the rows are few, several threads share
    // them and take every parts-th piece
    const int quads = rows * (F::DP / 4), parallel = max(1, kJoinThreads / quads), part = threadIdx.x / quads;
    const int chunk = kJoinWeights / R;
    for (int q0 = 0; q0 < quads; q0 += kJoinThreads) {
        const int quad = q0 + (parallel > 1 ? (int)threadIdx.x % quads : (int)threadIdx.x), r = quad * 4 / F::DP;
        const bool has = quad < quads && part < parallel;
        floatx4 v = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int k0 = 0; k0 < n; k0 += chunk) {
            __syncthreads();
            const int m = min(chunk, n - k0);
            for (int i = threadIdx.x; i < m * R; i += kJoinThreads) {
                if (i % R >= rows) continue;
                const float2 ml = parts.ml[at_of(k0 + i / R, i % R)];
                const float top = sums[i % R][0], sum = sums[i % R][1];
                const float e = ml.x == top ? 1.0f : __builtin_amdgcn_exp2f(ml.x - (top == -INFINITY ? 0.0f : top));
                weights[i] = ml.y * e / (sum == 0.0f ? 1.0f : sum);
            }
            __syncthreads();
            if (!has) continue;
            const floatx4 before = v;
#pragma unroll 8
            for (int k = part; k < m; k += parallel)
                v += weights[k * R + r] * *reinterpret_cast<const floatx4 *>(parts.o + at_of(k0 + k, 0) * F::DP + quad * 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (fabsf(v[e]) < INFINITY) continue;
                // a weight that underflows still lets an infinity through
                v[e] = before[e];
                for (int k = part; k < m; k += parallel) {
                    const float w = weights[k * R + r], x = parts.o[at_of(k0 + k, 0) * F::DP + quad * 4 + e];
                    v[e] += x * (fabsf(x) < INFINITY ? w : fmaxf(w, 1e-38f));
                }
            }
        }
        if (parallel > 1) {
            __syncthreads();
            if (has) *reinterpret_cast<floatx4 *>(&held[threadIdx.x * 4]) = v;
            __syncthreads();
            if (part == 0)
                for (int p = 1; p < parallel; ++p) v += *reinterpret_cast<const floatx4 *>(&held[(p * quads + threadIdx.x) * 4]);
        }
        if (!has || part > 0) continue;
        const int row = tile * R + r, t = row / a.G, h = hk * a.G + row % a.G;
        if (sums[r][0] == -INFINITY && sums[r][1] > 0.0f) v = floatx4{NAN, NAN, NAN, NAN};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int d = quad * 4 % F::DP + e;
            if (d < a.D) o[((int64_t)(s.r0 + t) * a.H + h) * a.D + d] = (typename F::T)v[e];
        }
        if (lse && quad * 4 % F::DP == 0)
            lse[(int64_t)(s.r0 + t) * a.H + h] = (sums[r][0] + __builtin_amdgcn_logf(sums[r][1])) * kLn2;
    }
}

// --------------------------------------------------------------- launches

constexpr int kCus = 256;

inline int padded(int D) { return D <= 32 ? 32 : D <= 64 ? 64 : 128; }
inline int64_t rows_of(int max_rows, int G) { return (int64_t)max_rows * G; }

// Tiles of 16 rows for which a block reads the keys once.  Two halve what is
// read, but their blocks are half as many and take a CU alone: 64 x 8 rows of
// 32/8 heads over 1000 keys, bf16, 64: 45 us with one, 35 with two; 128: 67 and
// 55, e4m3 56 and 43; 8 x 16 rows over 500 keys, 128: 11.5 and 16.  Heads of 32
// gain nothing (19 and 20), and fp32 rows of 128 do not fit the registers twice
// (114 and 132, 8-bit rows 55 and 63).
inline int tiles_of_block(int dtype, int DP, int64_t sequences, int Hkv, int64_t rows) {
    if (rows <= 16 || DP == 32 || (DP == 128 && dtype == SN_F32)) return 1;
    return sequences * Hkv * ((rows + 15) / 16) >= 2 * kCus ? 2 : 1;
}

AttendCut cut_of(int Hkv, int64_t rows, int nr) {
    AttendCut c{};
    c.row_tiles = (int)std::max<int64_t>(1, (rows + 16 * nr - 1) / (16 * nr));
    c.units = Hkv * c.row_tiles;
    c.least = kWaves;
    return c;
}

// Keys that a row may see, and the bytes of all sequences' keys and values:
// sequences are taken to be a little over half of what the table holds.
inline int64_t span_of(const CacheArgs &a) {
    const int64_t all = (int64_t)a.max_pages * a.page;
    return a.window > 0 ? std::min(all, (int64_t)a.window + a.max_rows + 15) : all;
}
inline double bytes_of(const CacheArgs &a, int es) { return 0.6 * a.B * (double)span_of(a) * a.Hkv * 2 * a.Dp * es; }

// Whether units are cut.  A block takes about 2 us for a round (a tile of each
// wavefront; 1.5 us with short rows).  Few units: cut where the rounds that a unit
// takes one after the other are 11 us longer than the bytes (the join, its launch
// and the shorter pieces cost 4 to 6, and what is left has to be gained; 1 x 4000
// keys, 32/8 x 128 bf16: 40 us whole, 19 cut; 1 x 1000: 14.9 and 14.8; 8 x 4000:
// 43 and 33; 16 x 2000: 27 and 32).  Units on every CU: cut where the longest
// ones would keep some CUs alone (32 x <= 20000: 331 and 262; 64 x <= 12000: 385
// and 304; 64 x 1000: 46 and 50).  Many units even out by themselves.  The host
// knows what the table holds, not the lengths: short ones in a table with room
// are cut where that does not pay (271 keys, 4 x 32 fp32: 6.7 and 10.4).
template <class F>
bool worth_cutting(const CacheArgs &a, const AttendCut &c) {
    const double units = (double)a.B * c.units, places = kCus * F::BLOCKS;
    const int64_t tiles = (span_of(a) + F::TILE - 1) / F::TILE + 1;
    const double rounds = (double)tiles / kWaves;
    const double streaming = bytes_of(a, F::ES) * c.row_tiles / 5.2e6;  // us at 5.2 TB/s
    if (units * tiles > INT32_MAX) return false;                        // a line of tiles is counted in 32 bits
    return units < places ? (F::BLOCKS == 2 ? 1.5 : 2.0) * rounds > 11.0 + streaming || streaming > 80.0 : units < 4 * places && streaming > 80.0;
}

inline size_t cuts_bytes(const AttendCut &c, int B) { return align256(sizeof(int2) * (size_t)B * c.units); }

template <class F>
sn_status launch(const CacheArgs &a, void *o, float *lse, char *ws, hipStream_t s) {
    using T = typename F::T;
    AttendCut c = cut_of(a.Hkv, rows_of(a.max_rows, a.G), F::NR);
    if (worth_cutting<F>(a, c)) c.blocks = kCus * F::BLOCKS;
    Partials parts;
    parts.cuts = reinterpret_cast<int2 *>(ws + kWsBase);
    parts.ml = reinterpret_cast<float2 *>(ws + kWsBase + cuts_bytes(c, a.B));
    parts.o = reinterpret_cast<float *>(parts.ml + 2 * kCus * F::BLOCKS * 16 * F::NR);
    ProfScope prof(K_CACHE_ATTEND, s);
    const int grid = xcd_grid(c.blocks ? c.blocks : a.B * c.units);
    attend_kernel<F><<<grid, kThreads, 0, s>>>(a, c, parts, static_cast<T *>(o), lse);
    SN_TRY(launch_status());
    if (c.blocks) attend_join_kernel<F><<<a.B * c.units, kJoinThreads, 0, s>>>(a, c, parts, static_cast<T *>(o), lse);
    return launch_status();
}
// Whether the rows are read past the caches: they are read once, and are more
// than the caches hold (32 x <= 20000 keys, 32/8 x 128 bf16, 1.6 GB: 295 us and
// 262 past them; 64 x <= 12000, 4 x 32 fp32, 480 MB: 98 and 88; 32 x 4000, 520 MB:
// 94 and 83; 16 x 4000, 260 MB: 46 and 67).  8-bit rows gain where units are cut
// (32 x <= 20000, 875 MB: 166 and 157) and little elsewhere (64 x 4000: 104 and 98).
// By the table, too: 16 x 4000 in one for 8000 takes 67, in one for 32000 (cut) 52.
template <class F>
bool reads_past(const CacheArgs &a) {
    const AttendCut c = cut_of(a.Hkv, rows_of(a.max_rows, a.G), 1);
    return c.row_tiles == 1 && bytes_of(a, F::ES) > 3e8 && (F::CODES == SN_CODES_NONE || worth_cutting<F>(a, c));
}

template <typename T, int CODES, int DP>
sn_status launch(const CacheArgs &a, void *o, float *lse, char *ws, hipStream_t s) {
    constexpr int dtype = std::is_same<T, float>::value ? SN_F32 : SN_BF16;
    if constexpr (CODES == SN_CODES_NONE || DP == 128)
        if (reads_past<Form<T, CODES, DP, 1>>(a)) return launch<Form<T, CODES, DP, 1, true>>(a, o, lse, ws, s);
    if constexpr (DP == 64 || (DP == 128 && dtype == SN_BF16))
        if (tiles_of_block(dtype, DP, a.B, a.Hkv, rows_of(a.max_rows, a.G)) == 2) return launch<Form<T, CODES, DP, 2>>(a, o, lse, ws, s);
    return launch<Form<T, CODES, DP, 1>>(a, o, lse, ws, s);
}
template <typename T, int CODES>
sn_status launch(const CacheArgs &a, void *o, float *lse, char *ws, hipStream_t s) {
    // fp32 products take heads of 16 as they are, bf16 ones 32 dims at a time
    if constexpr (std::is_same<T, float>::value && CODES == SN_CODES_NONE)
        if (a.Dp <= 16) return launch<T, CODES, 16>(a, o, lse, ws, s);
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

// Rows with their heads are counted in 32 bits; units are blocks of their own, or of the join.
bool attend_fits(const sn_cache &op) {
    if ((int64_t)op.n_rows * op.n_heads > INT32_MAX) return false;
    const AttendCut c = cut_of(op.n_kv_heads, rows_of(op.max_rows, op.n_heads / op.n_kv_heads), 1);
    return grid_fits((int64_t)op.n_sequences * c.units + kXcds, kThreads);
}

size_t attend_workspace(const sn_cache &op) {
    const int64_t rows = rows_of(op.max_rows, op.n_heads / op.n_kv_heads);
    const int DP = padded(op.head_dim), nr = tiles_of_block(op.dtype, DP, op.n_sequences, op.n_kv_heads, rows);
    const size_t held = (size_t)2 * kCus * (DP == 32 ? 2 : 1) * 16 * nr;
    return kWsBase + cuts_bytes(cut_of(op.n_kv_heads, rows, nr), op.n_sequences) + held * (sizeof(float2) + DP * sizeof(float));
}

sn_status cache_attend(const CacheArgs &a, int dtype, int codes, void *o, float *lse, char *ws, hipStream_t s) {
    return dtype == SN_F32 ? launch<float>(a, codes, o, lse, ws, s) : launch<bf16>(a, codes, o, lse, ws, s);
}

}  // namespace sn
