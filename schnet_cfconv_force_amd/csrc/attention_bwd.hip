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
// delta starts as dO_i.o_i from the rounded o.  What that (and the forward's
// 16-bit p) leaves is exactly what the row's dS fails to sum to zero by:
// e_i = sum_j dS_ij.  The bias sums are corrected by it, dbias -= e_i times
// the row's sum of p over the bucket, and the second pass takes delta + e.
#include <algorithm>

#include "attention.h"

namespace sn {
namespace {

// p and dS are carried times 2^24 and the factor is taken out of the
// finished sums: exp flushes what is below 2^-126 to zero, which moves the
// smallest p that counts to 2^-150 (a key that no row attends to has
// gradients of that size, and they are still right).
constexpr float kLift = 24.0f;
constexpr float kUnlift = 1.0f / 16777216.0f;

struct BwdArgs {
    const void *o;
    const float *lse;
    void *dq, *dk, *dv;
    float2 *row;        // [n_q H] {lse log2e - 24 (+inf: no key), delta}
    float *part_bias;   // [Hkv subs][B row_tiles][Gs nb]
    float *part_kv;     // [split][n_k Hkv][2][D] (splits > 1)
};

// LDS of the dq kernel: tiles, then the position table {bias log2e, bucket},
// then the bias sums {dS, p} [wavefront][bucket][row].
constexpr int kDqKeys = 32;
template <int NP, int DP>
constexpr int dq_buffers() { return NP == 3 && DP == 128 ? 1 : 2; }   // 160 KB of LDS
template <int NP, int DP>
constexpr size_t dq_tile_bytes() { return size_t(dq_buffers<NP, DP>()) * 2 * NP * kDqKeys * DP * sizeof(bf16); }

template <typename T>
__device__ inline void write4(T *row, int d, int D, floatx4 v) {
    if (D % 4 == 0) {
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

template <int NP, int DP>
__global__ __launch_bounds__(kAttnThreads, NP == 1 ? 2 : 1) void attn_dq_kernel(AttnArgs a, BwdArgs g) {
    using T = typename RowOf<NP>::T;
    constexpr int kBuf = dq_buffers<NP, DP>(), kTile = NP * kDqKeys * DP;
    extern __shared__ __align__(16) char lds_bytes[];
    bf16 *tiles = reinterpret_cast<bf16 *>(lds_bytes);   // [buffer][K, V]
    float2 *lut = reinterpret_cast<float2 *>(lds_bytes + dq_tile_bytes<NP, DP>());
    float *sums = reinterpret_cast<float *>(lut + a.Gs * a.lut_n);
    __shared__ KeyInfo<kDqKeys> info[2];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, half = lane >> 5;
    RowBlock w;
    if (!locate(a, w)) return;
    float *part = a.nb ? g.part_bias + ((int64_t)(w.hk * a.subs + w.sub) * a.B * a.row_tiles +
                                        (w.b * a.row_tiles + w.tile)) * (a.Gs * a.nb)
                       : nullptr;
    if (w.tile * 128 >= w.nq * w.gs) {
        for (int i = tid; a.nb && i < a.Gs * a.nb; i += kAttnThreads) part[i] = 0.0f;
        return;
    }
    if (a.nb) {
        for (int e = tid; e < a.lut_n; e += kAttnThreads) {
            const int bk = bucket_of(a, a.lut_base + e);
            for (int h = 0; h < w.gs; ++h)
                lut[h * a.lut_n + e] = make_float2(a.bias[(int64_t)(w.h0 + h) * a.nb + bk] * kLog2e, __int_as_float(bk));
        }
        for (int i = tid; i < 4 * a.nb * 64; i += kAttnThreads) sums[i] = 0.0f;
    }
    // the lane's column of its wavefront's sums: {dS, p} of bucket b at mine + 64 b
    float *mine = sums + wave * a.nb * 64 + (lane & 31) * 2;

    const int r = w.tile * 128 + wave * 32 + (lane & 31), qi = r / w.gs, hg = r % w.gs;
    const int row = qi < w.nq ? w.q0 + qi : -1;
    const int64_t at = (int64_t)row * a.H + w.h0 + hg;
    const bool active = __any(row >= 0);
    const float c = fabsf(a.scale) * kLog2e;
    Frag<NP> q[DP / 16], dO[DP / 16];
    float delta = 0.0f, L = INFINITY;
#pragma unroll
    for (int s = 0; s < DP / 16; ++s) {
        const int d = 16 * s + 8 * half;
        Raw8<NP> rq = raw_zero<NP>(), rg = rq, ro = rq;
        if (row >= 0) {
            rq = load8<NP>((const T *)a.q + row * a.qs + (w.h0 + hg) * a.qh + d, d, a.D, a.vec & 1);
            rg = load8<NP>((const T *)a.d_o + row * a.gs + (w.h0 + hg) * a.gh + d, d, a.D, a.vec & 8);
            ro = load8<NP>((const T *)g.o + at * a.D + d, d, a.D, a.vec & 16);
        }
        q[s] = to_frag<NP>(rq);
        dO[s] = to_frag<NP>(rg);
        if (a.scale < 0.0f)
#pragma unroll
            for (int n = 0; n < NP; ++n) q[s].p[n] = -q[s].p[n];
        const Frag<NP> fo = to_frag<NP>(ro);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float x = 0.0f, y = 0.0f;
#pragma unroll
            for (int n = NP - 1; n >= 0; --n) {
                x += (float)dO[s].p[n][j];
                y += (float)fo.p[n][j];
            }
            delta = fmaf(x, y, delta);
        }
    }
    delta += half_swap(delta);
    int pos = 0;
    if (row >= 0) {
        pos = a.q_pos ? a.q_pos[row] : qi;
        const float lse = g.lse[at];
        L = lse == -INFINITY ? INFINITY : lse * kLog2e - kLift;
    }
    const int pos_lo = wave_min(row >= 0 ? pos : 0x7fffffff), pos_hi = wave_max(row >= 0 ? pos : (int)0x80000000);

    const T *K = (const T *)a.k + w.k0 * a.ks + w.hk * a.kh, *V = (const T *)a.v + w.k0 * a.vs + w.hk * a.vh;
    const uint8_t *keep = a.keep ? a.keep + w.k0 : nullptr;
    const int n_tiles = (w.nk + kDqKeys - 1) / kDqKeys;
    TileMove<NP, DP, kDqKeys, kAttnThreads> mk, mv;
    KeyLoad kl;
    auto load = [&](int t) {
        mk.load(K, a.ks, t * kDqKeys, w.nk, a.D, a.vec & 2, tid, keep);
        mv.load(V, a.vs, t * kDqKeys, w.nk, a.D, a.vec & 4, tid, keep);
        if (wave == 0) kl.load(a, w, t * kDqKeys, kDqKeys, lane);
    };
    auto store = [&](int buf) {
        mk.store(tiles + 2 * buf * kTile, tid);
        mv.store(tiles + (2 * buf + 1) * kTile, tid);
        if (wave == 0) kl.store(info[buf], lane);
    };
    floatx16 dq[DP / 32];
#pragma unroll
    for (int e = 0; e < DP / 32; ++e)
#pragma unroll
        for (int i = 0; i < 16; ++i) dq[e][i] = 0.0f;
    float row_ds = 0.0f;                        // sum of the row's dS (this half's keys)
    float run_ds = 0.0f, run_p = 0.0f;          // of the tiles since the bucket last changed
    int run_bucket = -1;
    auto flush = [&]() {
        // the halves of a row add in turn: one order
        if (half == 0) { atomicAdd(mine + 64 * run_bucket, run_ds); atomicAdd(mine + 64 * run_bucket + 1, run_p); }
        __builtin_amdgcn_wave_barrier();
        if (half == 1) { atomicAdd(mine + 64 * run_bucket, run_ds); atomicAdd(mine + 64 * run_bucket + 1, run_p); }
        __builtin_amdgcn_wave_barrier();
        run_ds = run_p = 0.0f;
    };
    if (n_tiles > 0) {
        load(0);
        store(0);
    }
    __syncthreads();
    for (int t = 0; t < n_tiles; ++t) {
        const int buf = kBuf == 2 ? t & 1 : 0;
        if (t + 1 < n_tiles) load(t + 1);
        const bf16 *kt = tiles + 2 * buf * kTile, *vt = kt + kTile;
        const KeyInfo<kDqKeys> &ki = info[buf];
        const uint32_t mask = (uint32_t)uniform64(ki.mask);
        if (active && mask) {
            floatx16 s, dp;
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = dp[i] = 0.0f;
#pragma unroll
            for (int k = 0; k < DP / 16; ++k) s = mma<NP>(frag_rows<NP, DP>(kt, kDqKeys * DP, 0, k, lane), q[k], s);
#pragma unroll
            for (int k = 0; k < DP / 16; ++k) dp = mma<NP>(frag_rows<NP, DP>(vt, kDqKeys * DP, 0, k, lane), dO[k], dp);
            settle(s);
            settle(dp);
            float add = 0.0f;
            int bucket = -1;
            bool table = false;
            if (a.nb) {
                const int lo = __builtin_amdgcn_readfirstlane(ki.lo), hi = __builtin_amdgcn_readfirstlane(ki.hi);
                const int first = lut_index(a, offset_of(lo, pos_hi)), last = lut_index(a, offset_of(hi, pos_lo));
                const float2 entry = lut[hg * a.lut_n + first];
                add = entry.x;
                bucket = __builtin_amdgcn_readfirstlane(__float_as_int(entry.y));
                table = first != last;
            }
            const uint32_t keys = mask >> (4 * half);
            if (!table) {
                float sum_ds = 0.0f, sum_p = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float p = __builtin_amdgcn_exp2f(fmaf(s[i], c, add) - L);
                    if (mask != 0xffffffffu && !((keys >> (8 * (i / 4) + i % 4)) & 1)) p = 0.0f;
                    const float ds = p * (dp[i] - delta);
                    s[i] = ds;
                    sum_ds += ds;
                    sum_p += p;
                }
                row_ds += sum_ds;
                if (a.nb) {
                    if (bucket != run_bucket) {
                        if (run_bucket >= 0) flush();
                        run_bucket = bucket;
                    }
                    run_ds += sum_ds;
                    run_p += sum_p;
                }
            } else {
                int bk[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int e = lut_index(a, offset_of(ki.pos[8 * (i / 4) + 4 * half + i % 4], pos));
                    const float2 entry = lut[hg * a.lut_n + e];
                    bk[i] = __float_as_int(entry.y);
                    float p = __builtin_amdgcn_exp2f(fmaf(s[i], c, entry.x) - L);
                    if (!((keys >> (8 * (i / 4) + i % 4)) & 1)) p = 0.0f;
                    const float ds = p * (dp[i] - delta);
                    s[i] = ds;
                    dp[i] = p;
                    row_ds += ds;
                }
#pragma unroll
                for (int turn = 0; turn < 2; ++turn) {
                    if (half == turn)
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            atomicAdd(mine + 64 * bk[i], s[i]);
                            atomicAdd(mine + 64 * bk[i] + 1, dp[i]);
                        }
                    __builtin_amdgcn_wave_barrier();
                }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = s[8 * u + j];
                // bf16 rows: dS is rounded to 8 bits here, as p is in the
                // forward pass: at most 2^-8 of each term, as rounding dq
                const Frag<NP> ds = split8f<NP>(x);
#pragma unroll
                for (int e = 0; e < DP / 32; ++e)
                    dq[e] = mma<NP>(frag_cols<NP, DP>(kt, kDqKeys * DP, 16 * u, e, lane), ds, dq[e]);
            }
        }
        if constexpr (kBuf == 1) __syncthreads();
        if (t + 1 < n_tiles) store(kBuf == 2 ? buf ^ 1 : 0);
        __syncthreads();
    }
    // the row's sum of dS in units of p (sum_j p_ij is 2^24 by construction)
    const float err = (row_ds + half_swap(row_ds)) * kUnlift;
    if (row >= 0) {
        T *out = (T *)g.dq + at * a.D;
#pragma unroll
        for (int e = 0; e < DP / 32; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                write4<T>(out, 32 * e + 8 * i + 4 * half, a.D,
                          floatx4{dq[e][4 * i], dq[e][4 * i + 1], dq[e][4 * i + 2], dq[e][4 * i + 3]} *
                              (a.scale * kUnlift));
        if (half == 0) g.row[at] = make_float2(L, delta + err);
    }
    if (!a.nb) return;
    if (run_bucket >= 0) flush();
    // err per row, then every (head, bucket) sums its rows in order
    __syncthreads();
    float *errs = reinterpret_cast<float *>(tiles);
    if (half == 0) errs[wave * 32 + lane] = row >= 0 ? err : 0.0f;
    __syncthreads();
    for (int i = tid; i < a.Gs * a.nb; i += kAttnThreads) {
        const int h = i / a.nb, b = i % a.nb;
        float sum = 0.0f;
        for (int k = 0; k < 128; ++k) {
            if ((w.tile * 128 + k) % w.gs != h) continue;
            const float *x = sums + ((k >> 5) * a.nb + b) * 64 + (k & 31) * 2;
            sum += x[0] - errs[k] * x[1];
        }
        part[i] = sum;
    }
}

// dbias[h][b]: the row blocks' sums, in their order.  One block per subgroup
// and 64 of its (head, bucket) pairs; four wavefronts take every fourth.
__global__ __launch_bounds__(256) void attn_dbias_kernel(AttnArgs a, const float *part, float *dbias) {
    __shared__ double red[4][64];
    const int cols = a.Gs * a.nb, group = blockIdx.y, hk = group / a.subs, sub = group % a.subs;
    const int i = blockIdx.x * 64 + (threadIdx.x & 63), wave = threadIdx.x >> 6, n = a.B * a.row_tiles;
    double s = 0.0;
    if (i < cols)
        for (int k = wave; k < n; k += 4) s += part[((int64_t)group * n + k) * cols + i];
    red[wave][threadIdx.x & 63] = s;
    __syncthreads();
    if (wave != 0 || i >= cols) return;
    const int h = i / a.nb;
    if (sub * a.Gs + h >= a.G) return;
    s = (red[0][threadIdx.x] + red[1][threadIdx.x]) + (red[2][threadIdx.x] + red[3][threadIdx.x]);
    dbias[(int64_t)(hk * a.G + sub * a.Gs + h) * a.nb + i % a.nb] = (float)(s * kUnlift);
}

// What the rows of a tile need beside q and dO.
struct RowInfo {
    float L[32], delta[32];
    int pos[32];
    int lo, hi;
};

template <int NP, int DP>
__global__ __launch_bounds__(kAttnThreads, NP == 1 && DP < 128 ? 2 : 1) void attn_dkv_kernel(AttnArgs a, BwdArgs g) {
    using T = typename RowOf<NP>::T;
    constexpr int kRows = 32, kTile = NP * kRows * DP;
    __shared__ __align__(16) bf16 tiles[2][2][kTile];   // [buffer][q, dO]
    __shared__ RowInfo info[2];
    __shared__ float lut[kLutMax];
    __shared__ uint8_t lut_bucket[kLutMax];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, half = lane >> 5;
    const int n_blocks = a.B * a.Hkv * a.splits * a.row_tiles;
    int i0 = xcd_block(n_blocks);
    if (i0 < 0) return;
    const int key_tile = i0 % a.row_tiles; i0 /= a.row_tiles;
    const int split = i0 % a.splits; i0 /= a.splits;
    const int hk = i0 % a.Hkv, b = i0 / a.Hkv;
    int q0, nq, k0, nk;
    segment_rows(a.q_ptr, b, a.B, a.n_q, a.max_q, a.status, q0, nq);
    segment_rows(a.k_ptr, b, a.B, a.n_k, a.max_k, a.status, k0, nk);
    if (key_tile * 128 >= nk) return;
    const int j = key_tile * 128 + wave * 32 + (lane & 31);
    const bool have = j < nk, kept = have && (!a.keep || a.keep[k0 + j]);
    const bool active = __any(kept);
    if (a.nb)
        for (int e = tid; e < a.lut_n; e += kAttnThreads) lut_bucket[e] = (uint8_t)bucket_of(a, a.lut_base + e);
    Frag<NP> k[DP / 16], v[DP / 16];
#pragma unroll
    for (int s = 0; s < DP / 16; ++s) {
        const int d = 16 * s + 8 * half;
        Raw8<NP> rk = raw_zero<NP>(), rv = rk;
        if (kept) {
            rk = load8<NP>((const T *)a.k + (int64_t)(k0 + j) * a.ks + hk * a.kh + d, d, a.D, a.vec & 2);
            rv = load8<NP>((const T *)a.v + (int64_t)(k0 + j) * a.vs + hk * a.vh + d, d, a.D, a.vec & 4);
        }
        k[s] = to_frag<NP>(rk);
        v[s] = to_frag<NP>(rv);
        if (a.scale < 0.0f)
#pragma unroll
            for (int n = 0; n < NP; ++n) k[s].p[n] = -k[s].p[n];
    }
    const float c = fabsf(a.scale) * kLog2e;
    const int pos = kept ? (a.k_pos ? a.k_pos[k0 + j] : j) : 0;
    const int pos_lo = wave_min(kept ? pos : 0x7fffffff), pos_hi = wave_max(kept ? pos : (int)0x80000000);

    // the rows of all heads that share these keys, head by head
    const int per_head = (nq + kRows - 1) / kRows, n_tiles = per_head * a.G, per = (n_tiles + a.splits - 1) / a.splits;
    const int t0 = split * per, t1 = min(n_tiles, t0 + per);
    TileMove<NP, DP, kRows, kAttnThreads> mq, mg;
    float2 ri;
    int ri_pos;
    auto load = [&](int t) {
        const int h = hk * a.G + t / per_head, r0 = t % per_head * kRows;
        mq.load((const T *)a.q + q0 * a.qs + h * a.qh, a.qs, r0, nq, a.D, a.vec & 1, tid, nullptr);
        mg.load((const T *)a.d_o + q0 * a.gs + h * a.gh, a.gs, r0, nq, a.D, a.vec & 8, tid, nullptr);
        if (tid < kRows) {
            const int row = r0 + tid;
            ri = make_float2(INFINITY, 0.0f);
            ri_pos = row;
            if (row < nq) {
                ri = g.row[(int64_t)(q0 + row) * a.H + h];
                if (a.q_pos) ri_pos = a.q_pos[q0 + row];
            }
        }
    };
    auto store = [&](int t, int buf) {
        mq.store(tiles[buf][0], tid);
        mg.store(tiles[buf][1], tid);
        if (wave == 0) {
            const bool in = lane < kRows && t % per_head * kRows + lane < nq;
            const int lo = wave_min(in ? ri_pos : 0x7fffffff), hi = wave_max(in ? ri_pos : (int)0x80000000);
            if (lane < kRows) {
                info[buf].L[lane] = ri.x;
                info[buf].delta[lane] = ri.y;
                info[buf].pos[lane] = ri_pos;
            }
            if (lane == 0) {
                info[buf].lo = lo;
                info[buf].hi = hi;
            }
        }
    };
    floatx16 dk[DP / 32], dv[DP / 32];
#pragma unroll
    for (int e = 0; e < DP / 32; ++e)
#pragma unroll
        for (int i = 0; i < 16; ++i) dk[e][i] = dv[e][i] = 0.0f;
    int head = -1;
    if (t0 < t1) {
        load(t0);
        store(t0, 0);
    }
    __syncthreads();
    for (int t = t0; t < t1; ++t) {
        const int buf = (t - t0) & 1;
        if (t + 1 < t1) load(t + 1);
        if (a.nb && t / per_head != head) {   // every wavefront is past the last use of the table (barrier below)
            head = t / per_head;
            for (int e = tid; e < a.lut_n; e += kAttnThreads)
                lut[e] = a.bias[(int64_t)(hk * a.G + head) * a.nb + lut_bucket[e]] * kLog2e;
            __syncthreads();
        }
        const bf16 *qt = tiles[buf][0], *gt = tiles[buf][1];
        const RowInfo &ri_t = info[buf];
        if (active) {
            floatx16 s, dp;
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = dp[i] = 0.0f;
#pragma unroll
            for (int e = 0; e < DP / 16; ++e) s = mma<NP>(frag_rows<NP, DP>(qt, kRows * DP, 0, e, lane), k[e], s);
#pragma unroll
            for (int e = 0; e < DP / 16; ++e) dp = mma<NP>(frag_rows<NP, DP>(gt, kRows * DP, 0, e, lane), v[e], dp);
            settle(s);
            settle(dp);
            float add = 0.0f;
            bool table = false;
            if (a.nb) {
                const int lo = __builtin_amdgcn_readfirstlane(ri_t.lo), hi = __builtin_amdgcn_readfirstlane(ri_t.hi);
                const int first = lut_index(a, offset_of(pos_lo, hi)), last = lut_index(a, offset_of(pos_hi, lo));
                add = lut[first];
                table = first != last;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int row = 8 * (i / 4) + 4 * half + i % 4;
                float x = add;
                if (table) x = lut[lut_index(a, offset_of(pos, ri_t.pos[row]))];
                const float p = __builtin_amdgcn_exp2f(fmaf(s[i], c, x) - ri_t.L[row]);
                s[i] = p;
                dp[i] = p * (dp[i] - ri_t.delta[row]);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float x[8], y[8];
#pragma unroll
                for (int jj = 0; jj < 8; ++jj) {
                    x[jj] = s[8 * u + jj];
                    y[jj] = dp[8 * u + jj];
                }
                const Frag<NP> p = split8f<NP>(x), ds = split8f<NP>(y);
#pragma unroll
                for (int e = 0; e < DP / 32; ++e) {
                    dv[e] = mma<NP>(frag_cols<NP, DP>(gt, kRows * DP, 16 * u, e, lane), p, dv[e]);
                    dk[e] = mma<NP>(frag_cols<NP, DP>(qt, kRows * DP, 16 * u, e, lane), ds, dk[e]);
                }
            }
        }
        if (t + 1 < t1) store(t + 1, buf ^ 1);
        __syncthreads();
    }
    if (!have) return;
    const int64_t at = (int64_t)(k0 + j) * a.Hkv + hk;
    const float fk = kept ? a.scale * kUnlift : 0.0f, fv = kept ? kUnlift : 0.0f;
#pragma unroll
    for (int e = 0; e < DP / 32; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int d = 32 * e + 8 * i + 4 * half;
            floatx4 xk, xv;
#pragma unroll
            for (int n = 0; n < 4; ++n) {   // an absent key's column holds anything
                xk[n] = kept ? dk[e][4 * i + n] * fk : 0.0f;
                xv[n] = kept ? dv[e][4 * i + n] * fv : 0.0f;
            }
            if (a.splits > 1) {
                float *p = g.part_kv + (((int64_t)split * a.n_k * a.Hkv + at) * 2) * a.D;
                write4<float>(p, d, a.D, xk);
                write4<float>(p + a.D, d, a.D, xv);
            } else {
                write4<T>((T *)g.dk + at * a.D, d, a.D, xk);
                write4<T>((T *)g.dv + at * a.D, d, a.D, xv);
            }
        }
}

// dk, dv: the sums of the row splits, in their order.
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
    const int64_t blocks = (int64_t)B * Hkv * p.key_tiles, tiles = (int64_t)G * ((max_q + 31) / 32);
    p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(512 / blocks, tiles / 8));
    return p;
}

struct BwdLayout {
    size_t row, bias, kv, total;
};
BwdLayout bwd_layout(const BwdPlan &p, int B, int Hkv, int H, int64_t n_q, int64_t n_k, int D, int nb) {
    BwdLayout L;
    size_t o = kWsBase;
    auto take = [&](size_t bytes) { size_t r = o; o = align256(o + bytes); return r; };
    L.row = take(n_q * H * sizeof(float2));
    L.bias = take((size_t)Hkv * p.subs * B * p.row_tiles * p.Gs * nb * sizeof(float));
    L.kv = take(p.splits > 1 ? (size_t)p.splits * n_k * Hkv * 2 * D * sizeof(float) : 0);
    L.total = o;
    return L;
}

template <int NP, int DP>
sn_status launch(const AttnArgs &a0, const BwdArgs &g, const BwdPlan &p, hipStream_t s) {
    using T = typename RowOf<NP>::T;
    AttnArgs a = a0;
    a.Gs = p.Gs; a.subs = p.subs;
    if (a.n_q) {
        a.row_tiles = p.row_tiles;
        a.splits = 1;
        const size_t lds = dq_tile_bytes<NP, DP>() + (a.nb ? (size_t)a.Gs * a.lut_n * sizeof(float2) + 4 * a.nb * 256 : 0);
        attn_dq_kernel<NP, DP><<<xcd_grid(a.B * a.Hkv * a.subs * a.row_tiles), kAttnThreads, lds, s>>>(a, g);
        SN_TRY(launch_status());
    }
    if (a.n_k) {
        a.row_tiles = p.key_tiles;
        a.splits = p.splits;
        attn_dkv_kernel<NP, DP><<<xcd_grid(a.B * a.Hkv * a.splits * a.row_tiles), kAttnThreads, 0, s>>>(a, g);
        SN_TRY(launch_status());
        if (a.splits > 1) {
            const int64_t n = (int64_t)a.n_k * a.Hkv * 2 * a.D;
            attn_dkv_join_kernel<T><<<(int)((n + 255) / 256), 256, 0, s>>>(a, g);
            SN_TRY(launch_status());
        }
    }
    return SN_OK;
}

template <int NP>
sn_status launch_dim(const AttnArgs &a, const BwdArgs &g, const BwdPlan &p, hipStream_t s) {
    if (a.D <= 32) return launch<NP, 32>(a, g, p, s);
    if (a.D <= 64) return launch<NP, 64>(a, g, p, s);
    return launch<NP, 128>(a, g, p, s);
}

__global__ void fill_zero_kernel(float *x, int n) {
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i < n) x[i] = 0.0f;
}

}  // namespace

size_t attn_backward_workspace(const sn_cross_attention &op) {
    // the thresholds, which are not read here, decide how many heads share a table
    size_t need = kWsBase;
    for (int heads = 1; heads <= 8; ++heads) {
        const BwdPlan p = bwd_plan(op.n_segments, op.n_kv_heads, op.n_heads / op.n_kv_heads, op.max_q, op.max_k,
                                   kLutMax / heads);
        need = std::max(need, bwd_layout(p, op.n_segments, op.n_kv_heads, op.n_heads, op.n_q, op.n_k, op.head_dim,
                                         SN_MAX_BUCKETS).total);
    }
    return need;
}

sn_status attn_backward(AttnArgs a, int dtype, const void *o, const float *lse, void *dq, void *dk, void *dv,
                        float *dbias, char *ws, hipStream_t s) {
    ProfScope prof(K_ATTN_BWD, s);
    const BwdPlan p = bwd_plan(a.B, a.Hkv, a.G, a.max_q, a.max_k, a.lut_n);
    const BwdLayout L = bwd_layout(p, a.B, a.Hkv, a.H, a.n_q, a.n_k, a.D, a.nb);
    if (a.D % 8 == 0 && (reinterpret_cast<uintptr_t>(o) & 15) == 0) a.vec |= 16;
    BwdArgs g{o, lse, dq, dk, dv, reinterpret_cast<float2 *>(ws + L.row), reinterpret_cast<float *>(ws + L.bias),
              reinterpret_cast<float *>(ws + L.kv)};
    SN_TRY(dtype == SN_F32 ? launch_dim<3>(a, g, p, s) : launch_dim<1>(a, g, p, s));
    if (!dbias) return SN_OK;
    if (a.n_q) {
        a.Gs = p.Gs; a.subs = p.subs; a.row_tiles = p.row_tiles;
        attn_dbias_kernel<<<dim3((a.Gs * a.nb + 63) / 64, a.Hkv * a.subs), 256, 0, s>>>(a, g.part_bias, dbias);
    } else {
        fill_zero_kernel<<<(a.H * a.nb + 255) / 256, 256, 0, s>>>(dbias, a.H * a.nb);
    }
    return launch_status();
}

}  // namespace sn
