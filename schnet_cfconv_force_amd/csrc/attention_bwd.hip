// Cross attention with a learned relative position bias, backward.
//
//   p_ij = exp(s_ij - lse_i), dP = dO v^T, delta_i = sum_j p_ij dP_ij, dS = p (dP - delta)
//   dq = scale dS k, dk = scale dS^T q, dv = p^T dO, dbias = sums of dS over a bucket
//
// Two passes that recompute the scores, one over the keys for a block of
// rows (dq, the bias sums, delta) and one over the rows for a block of keys
// (dk, dv): seven products instead of five, but every sum has one owner and
// one order, so there are no atomics and the bits repeat.  Shared heads are
// further rows of the second pass and sum there.
//
// delta starts as dO_i.o_i of the unrounded o.  What that and the forward's
// roundings leave is exactly what the row's dS fails to sum to zero by:
// e_i = sum_j dS_ij, as sum_j p_ij = 1.  The second pass takes delta + e; the
// bias sums, which are fp32 whatever the rows are, are taken there.  For that
// both passes round alike: the scores' products in one order, the exponents as
// s scale + (bias - lse), whichever way a tile's bias is read, and
// sums over many rows are joined pairwise (fp32, 1272 rows of 16 keys: dbias
// 2.0e-6 of its norm off without the two, 2.9e-7 with them).  A segment's only
// kept key has p = 1 whatever its score: its dS is zero, not what rounding
// leaves.  The first pass counts the kept keys for the second.
#include <algorithm>

#include "attention.h"

namespace sn {
namespace {

// p and dS are carried times 2^12 and the factor is taken out of the
// finished sums: exp flushes what is below 2^-126 to zero, which moves the
// smallest p that counts to 2^-138 (a key that no row attends to has
// gradients of that size, and they are still right).  The factor is part of
// exp's argument, whose rounding is the largest error of an fp32 p: 12 is
// about what p = 1/length needs to leave it near zero (2^24 doubled the error
// of the gradients).
constexpr float kLift = 12.0f;
constexpr float kUnlift = 1.0f / 4096.0f;

struct BwdArgs {
    const float *o;     // before its rounding
    const float *lse;
    void *dq, *dk, *dv;
    float2 *row;        // [n_q H] {lse log2e - 12 (+inf: no key), delta}
    float *part_bias;   // [Hkv][B key_tiles splits][G nb]
    float *part_kv;     // [split][n_k Hkv][2][D] (splits > 1)
    int *kept;          // [B] kept keys (with a mask, of the segments that have rows)
};

// Keys of a tile in LDS, of which 32 at a time are computed: 64 halve the
// barriers where two such tiles leave LDS for two blocks on a CU (2 x 2048 x
// 2048, heads of 64: 302 -> 288 us for the training step).
template <int NP, int DP>
constexpr int kDqTile = NP * DP <= 96 ? 64 : 32;

// Pairwise: sums over thousands of rows that cancel keep their digits.
__device__ inline float tree_sum(const floatx16 &x) {
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = x[i] + x[i + 8];
#pragma unroll
    for (int n = 4; n > 0; n /= 2)
#pragma unroll
        for (int i = 0; i < n; ++i) s[i] += s[i + n];
    return s[0];
}

// four: the row is aligned for four elements and D a multiple of them.
template <typename T>
__device__ inline void write4(T *row, int d, int D, bool four, floatx4 v) {
    if (four) {
        if (d >= D) return;
        if constexpr (sizeof(T) == 2)
            *reinterpret_cast<bf16x4 *>(row + d) = __builtin_convertvector(v, bf16x4);
        else
            *reinterpret_cast<floatx4 *>(row + d) = v;
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (d + i < D) row[d + i] = (T)v[i];
}

// dq and the rows' delta: a wavefront owns 32 rows, the block's four share the
// key tiles, as in the forward kernel for many rows.  S^T and dP^T put a row's
// scores in one lane, so L and delta are one register each, and dS^T is the
// next product's operand as it lies.  Bound by latency: product, exponential
// and product follow each other, and two wavefronts on a SIMD do not cover it.
// Two segments of up to 2048 x 2048, 16 heads of 64, bf16: 99 us, 335 TFLOP/s;
// a wavefront waits a third of its time, the vector units are 31 % busy, the
// matrix units 14 %.  64 of up to 269 x 271, 4 heads of 32, fp32: 35 us, 44 % of
// it waiting (the start is as long as the tiles).  <1, 128> spills 26 registers.
template <int NP, int DP, bool FAST>
__global__ __launch_bounds__(kAttnThreads, NP == 1 || DP == 32 ? 2 : 1) void attn_dq_kernel(AttnArgs a, BwdArgs g) {
    using T = typename RowOf<NP>::T;
    constexpr int kDqKeys = kDqTile<NP, DP>, kTile = NP * kDqKeys * DP;
    __shared__ __align__(256) bf16 tiles[2][2][kTile];   // [buffer][K, V]
    __shared__ KeyInfo<kDqKeys> info[2];
    extern __shared__ float lut[];   // [head of the subgroup][lut_stride]
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), half = lane >> 5;
    RowBlock w;
    if (!locate(a, w)) return;
    if (w.tile * 128 >= w.nq * w.gs) return;

    const T *K = (const T *)a.k + w.k0 * a.ks + w.hk * a.kh, *V = (const T *)a.v + w.k0 * a.vs + w.hk * a.vh;
    const int n_tiles = (w.nk + kDqKeys - 1) / kDqKeys;
    TileMove<NP, DP, kDqKeys, kAttnThreads, FAST> mk, mv;
    KeyLoad<kDqKeys> kl;
    mk.init(a.ks, a.D, tid);
    mv.init(a.vs, a.D, tid);
    mk.seek(K, w.nk);
    mv.seek(V, w.nk);
    auto load = [&](int t) {
        mk.load(a.D, tid);
        mv.load(a.D, tid);
        kl.load(a, w, t * kDqKeys, a.nb && wave == 0, lane);
    };
    auto store = [&](int buf) {
        const uint64_t mask = kl.mask(a);
        mk.store(tiles[buf][0], tid, a.keep && is_partial<kDqKeys>(mask), mask);
        mv.store(tiles[buf][1], tid, a.keep && is_partial<kDqKeys>(mask), mask);
        if (a.nb && wave == 0) kl.store(info[buf], mask, lane);
        return mask;
    };

    // the first tile, the rows and the bias are on their way together
    const int r = w.tile * 128 + wave * 32 + (lane & 31), qi = r / w.gs, hg = r % w.gs;
    const int row = qi < w.nq ? w.q0 + qi : -1;
    const int64_t at = (int64_t)row * a.H + w.h0 + hg;
    const bool active = __any(row >= 0);
    const float c = fabsf(a.scale) * kLog2e;
    Raw8<NP> rq[DP / 16], rg[DP / 16];
    Raw8<3> ro[DP / 16];
    if (n_tiles > 0) load(0);
#pragma unroll
    for (int s = 0; s < DP / 16; ++s) {
        rq[s] = rg[s] = raw_zero<NP>();
        ro[s] = raw_zero<3>();
    }
    int pos = 0;
    float lse = -INFINITY;
    if (row >= 0) {
        const T *pq = (const T *)a.q + row * a.qs + (w.h0 + hg) * a.qh;
        const T *pg = (const T *)a.d_o + row * a.gs + (w.h0 + hg) * a.gh;
        const float *po = g.o + at * a.D;
#pragma unroll
        for (int s = 0; s < DP / 16; ++s) {
            const int d = 16 * s + 8 * half;
            rq[s] = load8<NP>(pq + d, d, a.D, FAST);
            rg[s] = load8<NP>(pg + d, d, a.D, FAST);
            ro[s] = load8<3>(po + d, d, a.D, FAST);
        }
        pos = a.q_pos ? a.q_pos[row] : qi;
        lse = g.lse[at];
    }
    if (a.nb) fill_lut(a, w, lut);
    Frag<NP> q[DP / 16], dO[DP / 16];
    float delta = 0.0f;
#pragma unroll
    for (int s = 0; s < DP / 16; ++s) {
        q[s] = to_frag<NP>(rq[s]);
        dO[s] = to_frag<NP>(rg[s]);
        if (a.scale < 0.0f)
#pragma unroll
            for (int n = 0; n < NP; ++n) q[s].p[n] = -q[s].p[n];
        const float y[8] = {ro[s].v[0].x, ro[s].v[0].y, ro[s].v[0].z, ro[s].v[0].w,
                            ro[s].v[1].x, ro[s].v[1].y, ro[s].v[1].z, ro[s].v[1].w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float x = 0.0f;
#pragma unroll
            for (int n = NP - 1; n >= 0; --n) x += (float)dO[s].p[n][j];
            delta = fmaf(x, y[j], delta);
        }
    }
    delta = half_sum(delta);
    const float L = lse == -INFINITY ? INFINITY : fmaf(lse, kLog2e, -kLift);
    const int pos_lo = wave_min(row >= 0 ? pos : 0x7fffffff), pos_hi = wave_max(row >= 0 ? pos : (int)0x80000000);

    floatx16 dq[DP / 32];
#pragma unroll
    for (int e = 0; e < DP / 32; ++e) dq[e] = zero16();
    float row_ds = 0.0f;    // sum of the row's dS (this half's keys)
    int n_kept = 0;
    const TileLane<DP> tl(lane);
    const uint32_t lds0 = lds_offset(tiles);
    constexpr uint32_t kPlane = kDqKeys * DP * sizeof(bf16), kBytes = NP * kPlane;
    uint64_t mask = 0;
    if (n_tiles > 0) mask = store(0);
    if (n_tiles > 1) load(1);
    __syncthreads();
    for (int t = 0; t < n_tiles; ++t) {   // tile t is in LDS, t + 1 in registers or on its way there
        const int buf = t & 1;
        const uint32_t kt = lds0 + 2 * buf * kBytes, vt = kt + kBytes;
        const KeyInfo<kDqKeys> &ki = info[buf];
        n_kept += __popcll(mask);
        if (active && mask) {
            float less = -L;
            const float *mine = lut + hg * lut_stride(a);
            PosRange keys{};
            bool table = false, undecided = a.nb;   // the tile's bias is looked up once, by the first half that has a key
#pragma unroll
            for (int sub = 0; sub < kDqKeys / 32; ++sub) {
                const uint32_t sub_mask = (uint32_t)(mask >> (32 * sub));
                if (kDqKeys > 32 && !sub_mask) continue;
                int4 range;
                if (undecided) range = ki.head;
                RowsProduct<NP, DP> rs, rd;
                rs.begin(tl, kt, 32 * sub);
                rd.begin(tl, vt, 32 * sub);
                if (undecided) {
                    undecided = false;
                    keys = uniform_range(range);
                    const int first = lut_index(a, offset_of(keys.lo, pos_hi)), last = lut_index(a, offset_of(keys.hi, pos_lo));
                    table = first != last;
                    if (!table) less += mine[kLutPad + first];
                }
                __builtin_amdgcn_sched_barrier(0);
                floatx16 s = rs.finish(tl, kt, kPlane, 32 * sub, q), dp = rd.finish(tl, vt, kPlane, 32 * sub, dO);
                ColsAhead<DP> kf;
                if constexpr (NP == 1) {
                    kf.load(tl, kt, 32 * sub);
                    __builtin_amdgcn_sched_barrier(0);
                }
                settle(s);
                settle(dp);
                if (table) {
                    if (a.lut_run && keys.run) {
                        const float *at = mine + run_index(a, offset_of(keys.first, pos)) + 4 * half + 32 * sub;
#pragma unroll
                        for (int i = 0; i < 16; ++i) s[i] = fmaf(s[i], c, at[8 * (i / 4) + i % 4] + less);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int e = lut_index(a, offset_of(ki.pos[32 * sub + 8 * (i / 4) + 4 * half + i % 4], pos));
                            s[i] = fmaf(s[i], c, mine[kLutPad + e] + less);
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) s[i] = fmaf(s[i], c, less);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) s[i] = __builtin_amdgcn_exp2f(s[i]) * (dp[i] - delta);
                if (sub_mask != 0xffffffffu) {
                    const uint32_t kept = sub_mask >> (4 * half);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (!((kept >> (8 * (i / 4) + i % 4)) & 1)) s[i] = 0.0f;
                }
                row_ds += tree_sum(s);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float x[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = s[8 * u + j];
                    // bf16 rows: dS is rounded to 8 bits here, at most 2^-8 of
                    // each term, as rounding dq: 2.4e-3 of its norm off, 1.7e-3
                    // of it its own rounding
                    const Frag<NP> ds = split8f<NP>(x);
#pragma unroll
                    for (int e = 0; e < DP / 32; ++e) {
                        if constexpr (NP == 1)
                            dq[e] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf.f[u][e], ds.p[0], dq[e], 0, 0, 0);
                        else
                            dq[e] = mma<NP>(frag_cols<NP, DP>(tl, kt, kPlane, 32 * sub + 16 * u, e), ds, dq[e]);
                    }
                }
            }
        }
        if (t + 1 < n_tiles) mask = store(buf ^ 1);
        if (t + 2 < n_tiles) load(t + 2);
        __syncthreads();
    }
    // the row's sum of dS in units of p (sum_j p_ij is 2^12 by construction)
    const float err = half_sum(row_ds) * kUnlift;
    if (a.keep && w.tile == 0 && w.sub == 0 && w.hk == 0 && tid == 0) g.kept[w.b] = n_kept;
    if (row >= 0) {
        T *out = (T *)g.dq + at * a.D;
        const float f = n_kept == 1 ? 0.0f : a.scale * kUnlift;
#pragma unroll
        for (int e = 0; e < DP / 32; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                write4<T>(out, 32 * e + 8 * i + 4 * half, a.D, a.out4,
                          floatx4{dq[e][4 * i], dq[e][4 * i + 1], dq[e][4 * i + 2], dq[e][4 * i + 3]} * f);
        if (half == 0) g.row[at] = make_float2(L, delta + err);
    }
}

// dbias[h][b]: the key blocks' sums, in their order.  One block per 64 of a
// key/value head's (head, bucket) pairs; its wavefronts take every sixteenth
// (4 us for 320 sums of 4 x 32 pairs: a launch and the reads' latency).
__global__ __launch_bounds__(1024) void attn_dbias_kernel(AttnArgs a, const float *part, float *dbias) {
    __shared__ double red[16][64];
    const int cols = a.G * a.nb, hk = blockIdx.y, n = a.B * a.row_tiles * a.splits;
    const int i = blockIdx.x * 64 + (threadIdx.x & 63), wave = threadIdx.x >> 6;
    double s = 0.0;
    if (i < cols)
#pragma unroll 4
        for (int k = wave; k < n; k += 16) s += part[((int64_t)hk * n + k) * cols + i];
    red[wave][threadIdx.x & 63] = s;
    __syncthreads();
    if (wave != 0 || i >= cols) return;
    for (int k = 1; k < 16; ++k) s += red[k][threadIdx.x];
    dbias[(int64_t)hk * cols + i] = (float)(s * kUnlift);
}

// What the rows of a tile need beside q and dO.
struct RowInfo {
    int4 head;                   // smallest and largest position, whether all run (first, first + 1, ...), the first
    float less[32], delta[32];   // -L
    int pos[32];
};

// The bias sums of a tile whose offsets span several buckets.  LDS float
// atomics take about 150 clocks each (16 per tile and wavefront doubled the
// kernel), so where the positions on both sides run without gaps, the tile's
// dS goes through LDS in a skewed layout instead: a lane reads one diagonal
// (one offset), sums it and adds it to its entry of a table of offsets.
// Other positions add to columns of their own [bucket][column], the halves
// of a wavefront in turn.  Both are one order; the buckets are summed when
// the head is done.
constexpr int kRunLut = 512;                    // longest position table that takes the diagonals
constexpr int kSkewRow = 17, kSkewRows = 62;    // [key + 15][row of 16], zeros around the 32 keys
constexpr int kRunPad = 64;                     // offsets beyond the table that a tile can reach
struct BiasLds {
    int lut, sums, skew, run, total;            // in floats
};
__host__ __device__ inline BiasLds bias_lds(int lut_n, int nb) {
    BiasLds l;
    l.lut = 0;                                  // {bias log2e, bucket} of one head
    l.sums = 2 * (lut_n + 2 * kLutPad);         // [wavefront][bucket][32]
    l.skew = l.sums + 4 * 32 * nb;              // [wavefront][kSkewRows][kSkewRow]
    l.run = l.skew + (lut_n <= kRunLut ? 4 * kSkewRows * kSkewRow : 0);   // [wavefront][lut_n + 2 kRunPad]
    l.total = l.run + (lut_n <= kRunLut ? 4 * (lut_n + 2 * kRunPad) : 0);
    return l;
}

// dk, dv and the bias sums: a wavefront owns 32 keys, the block's four share
// the tiles of 32 rows of every head that reads these keys.  S and dP put a
// key's column in one lane; p and dS are the operands of dv and dk as they
// lie.  Bound by latency, with two wavefronts on a SIMD at most and a barrier
// every 32 rows (tiles of 64 rows spilled).  Two segments of up to 2048 x 2048,
// 16 heads of 64, bf16: 137 us, 323 TFLOP/s; a wavefront waits 42 % of its
// time, the vector units are 21 % busy, the matrix units 12 % (without a bias
// the backward pass takes 170 us instead of 205 on segments of equal length);
// 64 segments of up to 269 x 271, 4 heads of 32, fp32: 47 us, 52 % waiting.
// Heads of 128 do not fit the registers: <3, 128> spills 85, <1, 64> three.
template <int NP, int DP>
constexpr int dkv_buffers() { return NP == 3 && DP == 128 ? 1 : 2; }   // 160 KB of LDS

template <int NP, int DP, bool FAST>
__global__ __launch_bounds__(kAttnThreads, DP == 32 || (NP == 1 && DP < 128) ? 2 : 1) void attn_dkv_kernel(AttnArgs a, BwdArgs g) {
    using T = typename RowOf<NP>::T;
    constexpr int kRows = 32, kTile = NP * kRows * DP;
    constexpr int kBuf = dkv_buffers<NP, DP>();
    __shared__ __align__(256) bf16 tiles[kBuf][2][kTile];   // [buffer][q, dO]
    __shared__ RowInfo info[kBuf];
    extern __shared__ __align__(16) float bias_mem[];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), half = lane >> 5;
    const BiasLds bl = bias_lds(a.lut_n, a.nb);
    float2 *lut = reinterpret_cast<float2 *>(bias_mem);
    float *sums = bias_mem + bl.sums;
    float *mine = sums + wave * a.nb * 32 + (lane & 31);   // the lane's column
    const int run_n = a.lut_n + 2 * kRunPad;
    float *skew = bias_mem + bl.skew + wave * kSkewRows * kSkewRow, *run = bias_mem + bl.run + wave * run_n;
    const bool small_lut = a.nb && a.lut_n <= kRunLut;
    const int n_blocks = a.B * a.Hkv * a.splits * a.row_tiles;
    int i0 = xcd_block(n_blocks);
    if (i0 < 0) return;
    const int key_tile = i0 % a.row_tiles; i0 /= a.row_tiles;
    const int split = i0 % a.splits; i0 /= a.splits;
    const int hk = i0 % a.Hkv, b = i0 / a.Hkv;
    int q0, nq, k0, nk;
    segment_rows(a.q_ptr, b, a.B, a.n_q, a.max_q, a.status, q0, nq);
    segment_rows(a.k_ptr, b, a.B, a.n_k, a.max_k, a.status, k0, nk);
    q0 = uniform(q0); nq = uniform(nq);
    k0 = uniform(k0); nk = uniform(nk);
    float *part = a.nb ? g.part_bias + (((int64_t)hk * a.B + b) * a.row_tiles * a.splits + key_tile * a.splits + split) * a.G * a.nb
                       : nullptr;
    if (key_tile * 128 >= nk) {
        for (int i = tid; a.nb && i < a.G * a.nb; i += kAttnThreads) part[i] = 0.0f;
        return;
    }
    const bool lone = (a.keep && nq > 0 ? g.kept[b] : nk) == 1;   // one kept key in the segment
    // the rows of all heads that share these keys, head by head
    const int per_head = (nq + kRows - 1) / kRows, n_tiles = per_head * a.G, per = (n_tiles + a.splits - 1) / a.splits;
    const int t0 = split * per, t1 = min(n_tiles, t0 + per);
    TileMove<NP, DP, kRows, kAttnThreads, FAST> mq, mg;
    mq.init(a.qs, a.D, tid);
    mg.init(a.gs, a.D, tid);
    // the tile that is loaded next: its head (of the G) and first row
    int next_head = t0 < t1 ? t0 / per_head : 0, next_row = t0 < t1 ? t0 % per_head * kRows : 0;
    auto seek = [&]() {   // (past the last head: never loaded)
        const int h = hk * a.G + next_head;
        mq.seek((const T *)a.q + (q0 + next_row) * a.qs + h * a.qh, nq - next_row);
        mg.seek((const T *)a.d_o + (q0 + next_row) * a.gs + h * a.gh, nq - next_row);
    };
    seek();
    float2 ri;
    int ri_pos, ri_n;
    auto load = [&]() {
        const int h = hk * a.G + next_head, r0 = next_row;
        mq.load(a.D, tid);
        mg.load(a.D, tid);
        if (wave == 0) {
            ri_n = min(nq - r0, kRows);
            ri = make_float2(INFINITY, 0.0f);
            ri_pos = r0 + lane;
            if (lane < ri_n) {
                ri = g.row[(int64_t)(q0 + r0 + lane) * a.H + h];
                if (a.q_pos) ri_pos = a.q_pos[q0 + r0 + lane];
            }
        }
        next_row += kRows;
        if (next_row >= nq) {
            next_row = 0;
            ++next_head;
            seek();
        }
    };

    // the first tile, the keys and the bias are on their way together
    const int j = key_tile * 128 + wave * 32 + (lane & 31);
    const bool have = j < nk;
    Raw8<NP> rk[DP / 16], rv[DP / 16];
    if (t0 < t1) load();
#pragma unroll
    for (int s = 0; s < DP / 16; ++s) rk[s] = rv[s] = raw_zero<NP>();
    uint8_t keep = have;
    int pos = j;
    if (have) {
        const T *pk = (const T *)a.k + (int64_t)(k0 + j) * a.ks + hk * a.kh;
        const T *pv = (const T *)a.v + (int64_t)(k0 + j) * a.vs + hk * a.vh;
#pragma unroll
        for (int s = 0; s < DP / 16; ++s) {
            const int d = 16 * s + 8 * half;
            rk[s] = load8<NP>(pk + d, d, a.D, FAST);
            rv[s] = load8<NP>(pv + d, d, a.D, FAST);
        }
        if (a.keep) keep = a.keep[k0 + j];
        if (a.k_pos) pos = a.k_pos[k0 + j];
    }
    if (a.nb)
        for (int e = tid; e < lut_stride(a); e += kAttnThreads)
            lut[e].y = __int_as_float(bucket_of(a, a.lut_base + min(max(e - kLutPad, 0), a.lut_n - 1)));
    if (small_lut)
        for (int i = lane; i < kSkewRows * kSkewRow; i += 64) skew[i] = 0.0f;
    const bool kept = keep != 0, active = __any(kept);
    Frag<NP> k[DP / 16], v[DP / 16];
#pragma unroll
    for (int s = 0; s < DP / 16; ++s) {
        k[s] = to_frag<NP>(kept ? rk[s] : raw_zero<NP>());
        v[s] = to_frag<NP>(kept ? rv[s] : raw_zero<NP>());
        if (a.scale < 0.0f)
#pragma unroll
            for (int n = 0; n < NP; ++n) k[s].p[n] = -k[s].p[n];
    }
    const float c = fabsf(a.scale) * kLog2e;
    const float kept_add = kept ? 0.0f : -INFINITY;   // an absent key's column of p, and with it of dS, is zero
    const int pos_lo = wave_min(kept ? pos : 0x7fffffff), pos_hi = wave_max(kept ? pos : (int)0x80000000);

    // kept keys whose positions run: the first key's position
    const int key_base = pos - (lane & 31), key0 = wave_min(kept ? key_base : 0x7fffffff);
    const bool key_run = small_lut && !__any(kept && (key_base != key0 || abs(pos) >= 1 << 30));

    auto store = [&](int buf) {
        mq.store(tiles[buf][0], tid, false, 0);
        mg.store(tiles[buf][1], tid, false, 0);
        if (wave == 0) {
            const int first = uniform(ri_pos);
            const bool run = !__any(lane < ri_n && (ri_pos != first + lane || abs(ri_pos) >= 1 << 30));
            int lo = first, hi = first + ri_n - 1;
            if (!run) {
                lo = wave_min(lane < ri_n ? ri_pos : 0x7fffffff);
                hi = wave_max(lane < ri_n ? ri_pos : (int)0x80000000);
            }
            if (lane < kRows) {
                info[buf].less[lane] = -ri.x;
                info[buf].delta[lane] = ri.y;
                info[buf].pos[lane] = ri_pos;
            }
            if (lane == 0) info[buf].head = make_int4(lo, hi, run, first);
        }
    };
    const TileLane<DP> tl(lane);
    const uint32_t lds0 = lds_offset(tiles);
    constexpr uint32_t kPlane = kRows * DP * sizeof(bf16), kBytes = NP * kPlane;
    floatx16 dk[DP / 32], dv[DP / 32];
#pragma unroll
    for (int e = 0; e < DP / 32; ++e) dk[e] = dv[e] = zero16();
    float run_ds = 0.0f;        // of the tiles since the bucket last changed
    int run_bucket = -1, head = -1;
    auto add_column = [&](int bk, float x) {
        if (half == 0) atomicAdd(mine + bk * 32, x);
        wave_sync();
        if (half == 1) atomicAdd(mine + bk * 32, x);
        wave_sync();
    };
    auto flush = [&]() {
        if (run_bucket >= 0) add_column(run_bucket, run_ds);
        run_ds = 0.0f;
        run_bucket = -1;
    };
    // the head's sums are complete: the wavefronts' tables of offsets become
    // one, then four threads per bucket add its columns and its offsets, in
    // one order
    auto finish_head = [&]() {
        flush();
        __syncthreads();
        float *all = bias_mem + bl.run;
        if (small_lut)
            for (int e = tid; e < run_n; e += kAttnThreads)
                all[e] = (all[e] + all[run_n + e]) + (all[2 * run_n + e] + all[3 * run_n + e]);
        __syncthreads();
        const int bk = tid >> 2, q = tid & 3;
        if (bk < a.nb) {
            float s = 0.0f;
#pragma unroll 8
            for (int k = 0; k < 32; ++k) s += sums[(q * a.nb + bk) * 32 + (k + bk) % 32];
            if (small_lut) {
                const int from = bk == 0 ? 0 : (int)((int64_t)a.thr[bk - 1] - a.lut_base) + kRunPad;
                const int to = bk == a.nb - 1 ? run_n : (int)((int64_t)a.thr[bk] - a.lut_base) + kRunPad;
#pragma unroll 4
                for (int e = from + q; e < to; e += 4) s += all[e];
            }
            s += __shfl_xor(s, 1, 64);
            s += __shfl_xor(s, 2, 64);
            if (q == 0) part[head * a.nb + bk] = lone ? 0.0f : s;
        }
        __syncthreads();
    };
    if (a.nb)   // heads that this split does not reach
        for (int i = tid; i < a.G * a.nb; i += kAttnThreads)
            if (t0 >= t1 || i / a.nb < t0 / per_head || i / a.nb > (t1 - 1) / per_head) part[i] = 0.0f;
    int tile_head = 0, loaded_head = next_row == 0 ? next_head - 1 : next_head;   // of the tiles in LDS and in registers
    if (t0 < t1) store(0);
    tile_head = loaded_head;
    if (t0 + 1 < t1) {
        loaded_head = next_head;
        load();
    }
    __syncthreads();
    for (int t = t0; t < t1; ++t) {   // tile t is in LDS, t + 1 in registers or on its way there
        const int buf = kBuf == 2 ? (t - t0) & 1 : 0;
        if (a.nb && tile_head != head) {   // every wavefront is past the last use of the table (barrier below)
            if (head >= 0) finish_head();
            head = tile_head;
            for (int e = tid; e < lut_stride(a); e += kAttnThreads)
                lut[e].x = bias_log2(a.bias[(int64_t)(hk * a.G + head) * a.nb + __float_as_int(lut[e].y)]);
            for (int i = tid; i < 4 * a.nb * 32; i += kAttnThreads) sums[i] = 0.0f;
            if (small_lut)
                for (int i = tid; i < 4 * run_n; i += kAttnThreads) bias_mem[bl.run + i] = 0.0f;
            __syncthreads();
        }
        const uint32_t qt = lds0 + 2 * buf * kBytes, gt = qt + kBytes;
        const RowInfo &ri_t = info[buf];
        if (active) {
            int4 range;
            if (a.nb) range = ri_t.head;
            RowsProduct<NP, DP> rs, rd;
            rs.begin(tl, qt, 0);
            rd.begin(tl, gt, 0);
            float less[16], delta[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                less[i] = ri_t.less[8 * (i / 4) + 4 * half + i % 4] + kept_add;
                delta[i] = ri_t.delta[8 * (i / 4) + 4 * half + i % 4];
            }
            float add = 0.0f;
            PosRange rows{};
            int bucket = -1;
            bool table = false;
            if (a.nb) {
                rows = uniform_range(range);
                const int first = lut_index(a, offset_of(pos_lo, rows.hi)), last = lut_index(a, offset_of(pos_hi, rows.lo));
                table = first != last;
                if (!table) {
                    const float2 e = lut[kLutPad + first];
                    add = e.x;
                    bucket = uniform(__float_as_int(e.y));
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            floatx16 s = rs.template finish<true>(tl, qt, kPlane, 0, k), dp = rd.template finish<true>(tl, gt, kPlane, 0, v);
            ColsAhead<DP> qf, gf;
            if constexpr (NP == 1) {
                gf.load(tl, gt, 0);
                qf.load(tl, qt, 0);
                __builtin_amdgcn_sched_barrier(0);
            }
            settle(s);
            settle(dp);
            if (table) {
                if (a.lut_run && rows.run) {   // later rows, smaller offsets
                    const float2 *at = lut + run_index(a, offset_of(pos, rows.first + 31)) + 3 - 4 * half;
#pragma unroll
                    for (int i = 0; i < 16; ++i) s[i] = fmaf(s[i], c, at[28 - 8 * (i / 4) - i % 4].x + less[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        s[i] = fmaf(s[i], c, lut[kLutPad + lut_index(a, offset_of(pos, ri_t.pos[8 * (i / 4) + 4 * half + i % 4]))].x + less[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) s[i] = fmaf(s[i], c, add + less[i]);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float p = __builtin_amdgcn_exp2f(s[i]);
                s[i] = p;
                dp[i] = p * (dp[i] - delta[i]);
            }
            if (a.nb) {
                if (!table) {
                    if (bucket != run_bucket) flush();
                    run_bucket = bucket;
                    run_ds += tree_sum(dp);
                } else if (key_run && rows.run) {
                    const int first = rows.first;
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            skew[((lane & 31) + 15) * kSkewRow + 8 * (i / 4) + 4 * half + i % 4] =
                                dp[8 * u + i];
                        wave_sync();
                        float x = 0.0f;   // offset key - row = lane - 15
                        if (lane < 47) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) x += skew[lane * kSkewRow + i * (kSkewRow + 1)];
                            run[key0 - (first + 16 * u) + (lane - 15) - a.lut_base + kRunPad] += x;
                        }
                        wave_sync();
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int e = lut_index(a, offset_of(pos, ri_t.pos[8 * (i / 4) + 4 * half + i % 4]));
                        add_column(__float_as_int(lut[kLutPad + e].y), dp[i]);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float x[8], y[8];
#pragma unroll
                for (int jj = 0; jj < 8; ++jj) {
                    x[jj] = s[8 * u + jj];
                    y[jj] = dp[8 * u + jj];
                }
                // bf16 rows: 8 bits here too.  dk and dv are 2.3e-3 of their
                // norms off, 1.7e-3 of it their own rounding; 16 bits are two
                // products and six instructions a score more
                const Frag<NP> p = split8f<NP>(x), ds = split8f<NP>(y);
#pragma unroll
                for (int e = 0; e < DP / 32; ++e) {
                    if constexpr (NP == 1) {
                        dv[e] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(gf.f[u][e], p.p[0], dv[e], 0, 0, 0);
                        dk[e] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(qf.f[u][e], ds.p[0], dk[e], 0, 0, 0);
                    } else {
                        dv[e] = mma<NP>(frag_cols<NP, DP>(tl, gt, kPlane, 16 * u, e), p, dv[e]);
                        dk[e] = mma<NP>(frag_cols<NP, DP>(tl, qt, kPlane, 16 * u, e), ds, dk[e]);
                    }
                }
            }
        }
        if constexpr (kBuf == 1) __syncthreads();
        if (t + 1 < t1) {
            store(kBuf == 2 ? buf ^ 1 : 0);
            tile_head = loaded_head;
        }
        if (t + 2 < t1) {
            loaded_head = next_head;
            load();
        }
        __syncthreads();
    }
    if (a.nb && head >= 0) finish_head();
    if (!have) return;
    const int64_t at = (int64_t)(k0 + j) * a.Hkv + hk;
    const float fk = lone ? 0.0f : a.scale * kUnlift;
#pragma unroll
    for (int e = 0; e < DP / 32; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int d = 32 * e + 8 * i + 4 * half;
            floatx4 xk, xv;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                xk[n] = kept ? dk[e][4 * i + n] * fk : 0.0f;   // zero whatever the rows hold
                xv[n] = kept ? dv[e][4 * i + n] * kUnlift : 0.0f;
            }
            if (a.splits > 1) {
                float *p = g.part_kv + (((int64_t)split * a.n_k * a.Hkv + at) * 2) * a.D;
                write4<float>(p, d, a.D, a.D % 4 == 0, xk);
                write4<float>(p + a.D, d, a.D, a.D % 4 == 0, xv);
            } else {
                write4<T>((T *)g.dk + at * a.D, d, a.D, a.out4, xk);
                write4<T>((T *)g.dv + at * a.D, d, a.D, a.out4, xv);
            }
        }
}

// dk, dv: the sums of the row splits, in their order (5.5 us for 24 segments
// of up to 517 keys, 2 heads of 40: a launch and a read).
template <typename T>
__global__ __launch_bounds__(256) void attn_dkv_join_kernel(AttnArgs a, BwdArgs g) {
    const int64_t n = (int64_t)a.n_k * a.Hkv * 2 * a.D, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    float s = 0.0f;
    for (int k = 0; k < a.splits; ++k) s += g.part_kv[k * n + i];
    const int64_t at = i / (2 * a.D);
    const int d = (int)(i % (2 * a.D));
    T *out = d < a.D ? (T *)g.dk + at * a.D + d : (T *)g.dv + at * a.D + (d - a.D);
    *out = (T)s;
}

// The rows of the dk, dv pass are split up to two blocks for every CU, as long
// as each has eight tiles of them: 4096 rows on 64 keys of 2 heads take 683 us
// unsplit and 58 us split; 24 x 701 x 517, 6 heads of 40 on 2: 178 against 143
// us, and 158 us with twice as many.
struct BwdPlan {
    int Gs, subs, row_tiles;    // rows of the dq pass
    int key_tiles, splits;      // keys of the dk, dv pass, splits of its rows
};

BwdPlan bwd_plan(int B, int Hkv, int G, int max_q, int max_k, int lut_n) {
    BwdPlan p;
    p.Gs = std::max(1, std::min({8, G, kLutMax / std::max(1, lut_n)}));
    p.subs = (G + p.Gs - 1) / p.Gs;
    p.row_tiles = (int)std::max<int64_t>(1, ((int64_t)max_q * p.Gs + 127) / 128);
    p.key_tiles = std::max(1, (max_k + 127) / 128);
    const int64_t blocks = (int64_t)B * Hkv * p.key_tiles, tiles = (int64_t)G * ((max_q + 31) / 32);   // of 32 rows
    p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(512 / blocks, tiles / 8));
    return p;
}

bool fits(const BwdPlan &p, int B, int Hkv) {
    return grid_fits((int64_t)B * Hkv * p.subs * p.row_tiles + kXcds, kAttnThreads) &&
           grid_fits((int64_t)B * Hkv * p.splits * p.key_tiles + kXcds, kAttnThreads);
}

struct BwdLayout {
    size_t row, bias, kv, kept, total;
};
BwdLayout bwd_layout(const BwdPlan &p, int B, int Hkv, int H, int64_t n_q, int64_t n_k, int D, int nb) {
    BwdLayout L;
    size_t o = kWsBase;
    auto take = [&](size_t bytes) { size_t r = o; o = align256(o + bytes); return r; };
    L.row = take(n_q * H * sizeof(float2));
    L.bias = take((size_t)H * B * p.key_tiles * p.splits * nb * sizeof(float));
    L.kv = take(p.splits > 1 ? (size_t)p.splits * n_k * Hkv * 2 * D * sizeof(float) : 0);
    L.kept = take(B * sizeof(int));
    L.total = o;
    return L;
}

template <int NP, int DP, bool FAST>
sn_status launch(const AttnArgs &a0, const BwdArgs &g, const BwdPlan &p, hipStream_t s) {
    using T = typename RowOf<NP>::T;
    AttnArgs a = a0;
    a.Gs = p.Gs; a.subs = p.subs;
    if (a.n_q) {
        a.row_tiles = p.row_tiles;
        a.splits = 1;
        attn_dq_kernel<NP, DP, FAST><<<xcd_grid(a.B * a.Hkv * a.subs * a.row_tiles), kAttnThreads,
                                       a.nb ? (size_t)a.Gs * (a.lut_n + 2 * kLutPad) * sizeof(float) : 0, s>>>(a, g);
        SN_TRY(launch_status());
    }
    if (a.n_k) {
        a.row_tiles = p.key_tiles;
        a.splits = p.splits;
        attn_dkv_kernel<NP, DP, FAST><<<xcd_grid(a.B * a.Hkv * a.splits * a.row_tiles), kAttnThreads,
                                        a.nb ? bias_lds(a.lut_n, a.nb).total * sizeof(float) : 0, s>>>(a, g);
        SN_TRY(launch_status());
        if (a.splits > 1) {
            const int64_t n = (int64_t)a.n_k * a.Hkv * 2 * a.D;
            attn_dkv_join_kernel<T><<<(int)((n + 255) / 256), 256, 0, s>>>(a, g);
            SN_TRY(launch_status());
        }
    }
    return SN_OK;
}

template <int NP, bool FAST>
sn_status launch_dim(const AttnArgs &a, const BwdArgs &g, const BwdPlan &p, hipStream_t s) {
    if (a.D <= 32) return launch<NP, 32, FAST>(a, g, p, s);
    if (a.D <= 64) return launch<NP, 64, FAST>(a, g, p, s);
    return launch<NP, 128, FAST>(a, g, p, s);
}

__global__ void fill_zero_kernel(float *x, int n) {
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i < n) x[i] = 0.0f;
}

}  // namespace

// The thresholds, which are not read here, decide how many heads share a
// table (1 to 8): the plan of each.
static BwdPlan plan_of(const sn_cross_attention &op, int heads) {
    return bwd_plan(op.n_segments, op.n_kv_heads, op.n_heads / op.n_kv_heads, op.max_q, op.max_k, kLutMax / heads);
}

bool attn_backward_fits(const sn_cross_attention &op) {
    for (int heads = 1; heads <= 8; ++heads)
        if (fits(plan_of(op, heads), op.n_segments, op.n_kv_heads)) return true;
    return false;
}

size_t attn_backward_workspace(const sn_cross_attention &op) {
    size_t need = kWsBase;
    for (int heads = 1; heads <= 8; ++heads) {
        const BwdPlan p = plan_of(op, heads);
        need = std::max(need, bwd_layout(p, op.n_segments, op.n_kv_heads, op.n_heads, op.n_q, op.n_k, op.head_dim,
                                         SN_MAX_BUCKETS).total);
    }
    return need;
}

sn_status attn_backward(AttnArgs a, int dtype, const float *o, const float *lse, void *dq, void *dk, void *dv,
                        float *dbias, char *ws, hipStream_t s) {
    ProfScope prof(K_ATTN_BWD, s);
    const BwdPlan p = bwd_plan(a.B, a.Hkv, a.G, a.max_q, a.max_k, a.lut_n);
    if (!fits(p, a.B, a.Hkv)) return SN_ERR_INVALID;
    const BwdLayout L = bwd_layout(p, a.B, a.Hkv, a.H, a.n_q, a.n_k, a.D, a.nb);
    BwdArgs g{o, lse, dq, dk, dv, reinterpret_cast<float2 *>(ws + L.row), reinterpret_cast<float *>(ws + L.bias),
              reinterpret_cast<float *>(ws + L.kv), reinterpret_cast<int *>(ws + L.kept)};
    if (a.fast)
        SN_TRY((dtype == SN_F32 ? launch_dim<3, true>(a, g, p, s) : launch_dim<1, true>(a, g, p, s)));
    else
        SN_TRY((dtype == SN_F32 ? launch_dim<3, false>(a, g, p, s) : launch_dim<1, false>(a, g, p, s)));
    if (!dbias) return SN_OK;
    if (a.n_k) {
        a.row_tiles = p.key_tiles; a.splits = p.splits;
        attn_dbias_kernel<<<dim3((a.G * a.nb + 63) / 64, a.Hkv), 1024, 0, s>>>(a, g.part_bias, dbias);
    } else {
        fill_zero_kernel<<<(a.H * a.nb + 255) / 256, 256, 0, s>>>(dbias, a.H * a.nb);
    }
    return launch_status();
}

}  // namespace sn
