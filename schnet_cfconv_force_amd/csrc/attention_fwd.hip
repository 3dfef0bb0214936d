// Cross attention with a learned relative position bias, forward.
//
//   s_ij = scale q_i.k_j + bias[bucket(k_pos_j - q_pos_i)],  o_i = sum_j softmax_j(s_ij) v_j
//
// One pass over the keys with the running maximum m, sum l and unnormalised
// row O: a tile's p = 2^(s log2e - m) joins as O += p v, l += sum p, and when
// m rises by more than 8 both are scaled by 2^(m_old - m_new) (a smaller
// rise is left in p, which stays below 2^8).
//
// A wavefront owns 32 rows.  It computes S^T = K Q^T, so a lane holds one
// row's scores: the maximum and sum are register operations and one exchange
// with the lane's other half, m and l are one register each, and the score
// tile is the B operand of O^T += V^T P^T as it lies.
#include <algorithm>

#include "attention.h"

namespace sn {
namespace {

struct FwdOut {
    void *o;
    float *rows;        // o before its rounding, for the backward pass (bf16; or null)
    float *lse;
    float *part_o;      // [split][n_q H][D] unnormalised rows (splits > 1)
    float2 *part_ml;    // [split][n_q H] their maximum (log2) and sum
};

// What a wavefront keeps of its 32 rows (a lane: row lane % 32).
template <int NP, int DP, bool FAST>
struct RowState {
    static constexpr int PP = NP == 1 ? 2 : NP;   // planes of p; see the product with v
    Frag<NP> q[DP / 16];
    floatx16 o[DP / 32];
    float m, l;
    int row, g, pos;        // query row (-1: none), head of the subgroup, position
    int pos_lo, pos_hi;     // of the wavefront's rows
    float c;                // |scale| log2e; the sign of the scale is in q

    // begin() issues the loads of the rows, finish() uses them.
    __device__ inline void begin(const AttnArgs &a, const RowBlock &w, int r0, int lane, Raw8<NP> (&raw)[DP / 16]) {
        using T = typename RowOf<NP>::T;
        const int r = r0 + (lane & 31), qi = r / w.gs;
        g = r % w.gs;
        row = qi < w.nq ? w.q0 + qi : -1;
        pos = qi;
#pragma unroll
        for (int s = 0; s < DP / 16; ++s) {
            const int d = 16 * s + 8 * (lane >> 5);
            raw[s] = raw_zero<NP>();
            if (row >= 0)
                raw[s] = load8<NP>((const T *)a.q + row * a.qs + (w.h0 + g) * a.qh + d, d, a.D, FAST);
        }
        if (row >= 0 && a.q_pos) pos = a.q_pos[row];
    }
    __device__ inline void finish(const AttnArgs &a, const Raw8<NP> (&raw)[DP / 16]) {
        c = fabsf(a.scale) * kLog2e;
#pragma unroll
        for (int s = 0; s < DP / 16; ++s) {
            q[s] = to_frag<NP>(raw[s]);
            if (a.scale < 0.0f)
#pragma unroll
                for (int n = 0; n < NP; ++n) q[s].p[n] = -q[s].p[n];
        }
        pos_lo = wave_min(row >= 0 ? pos : 0x7fffffff);
        pos_hi = wave_max(row >= 0 ? pos : (int)0x80000000);
        m = -INFINITY;
        l = 0.0f;
#pragma unroll
        for (int e = 0; e < DP / 32; ++e) o[e] = zero16();
    }

    // One tile of KT keys (KT / 32 score tiles) at the LDS offsets kt, vt.
    // mask: the kept keys; ki: their positions (used with a bias).
    template <int KT>
    __device__ inline void step(const AttnArgs &a, const TileLane<DP> &tl, uint32_t kt, uint32_t vt, uint64_t mask,
                                const KeyInfo<KT> &ki, const float *lut, int lane) {
        constexpr int NS = KT / 32;
        constexpr uint32_t kPlane = KT * DP * sizeof(bf16);
        const int half = lane >> 5;
        int4 head;
        if (a.nb) head = ki.head;
        RowsProduct<NP, DP> rp[NS];
#pragma unroll
        for (int u = 0; u < NS; ++u) rp[u].begin(tl, kt, 32 * u);
        // x = s c + add, in log2 units: one bias for a tile whose offsets all
        // fall in one bucket, else c is folded in below, element by element
        float mul = c, add = 0.0f;
        const float *mine = lut + g * lut_stride(a);
        PosRange keys{};
        bool table = false;
        if (a.nb) {
            keys = uniform_range(head);
            const int first = lut_index(a, offset_of(keys.lo, pos_hi)), last = lut_index(a, offset_of(keys.hi, pos_lo));
            table = first != last;
            if (!table) add = mine[kLutPad + first];
        }
        __builtin_amdgcn_sched_barrier(0);
        floatx16 s[NS];
#pragma unroll
        for (int u = 0; u < NS; ++u) s[u] = rp[u].finish(tl, kt, kPlane, 32 * u, q);
        // one plane: the values are on their way during the softmax
        ColsAhead<DP> vf[NS];
        if constexpr (NP == 1) {
#pragma unroll
            for (int u = 0; u < NS; ++u) vf[u].load(tl, vt, 32 * u);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int u = 0; u < NS; ++u) settle(s[u]);
        if (table) {
            mul = 1.0f;
            if (a.lut_run && keys.run) {
                const float *at = mine + run_index(a, offset_of(keys.first, pos)) + 4 * half;
#pragma unroll
                for (int u = 0; u < NS; ++u)
#pragma unroll
                    for (int i = 0; i < 16; ++i) s[u][i] = fmaf(s[u][i], c, at[32 * u + 8 * (i / 4) + i % 4]);
            } else {
#pragma unroll
                for (int u = 0; u < NS; ++u)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int at = lut_index(a, offset_of(ki.pos[32 * u + 8 * (i / 4) + 4 * half + i % 4], pos));
                        s[u][i] = fmaf(s[u][i], c, mine[kLutPad + at]);
                    }
            }
        }
        if (is_partial<KT>(mask)) {
            const uint64_t mine = mask >> (4 * half);
#pragma unroll
            for (int u = 0; u < NS; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (!((mine >> (32 * u + 8 * (i / 4) + i % 4)) & 1)) s[u][i] = -INFINITY;
        }
        float mx = s[0][0];
#pragma unroll
        for (int u = 0; u < NS; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[u][i]);
        mx = half_max(mx);
        mx = mx == -INFINITY ? mx : fmaf(mx, mul, add);   // no key, whatever the scale
        if (__any(mx > m + 8.0f)) {
            const float mn = fmaxf(m, mx);
            const float f = mn == m ? 1.0f : __builtin_amdgcn_exp2f(m - mn);   // both -inf: nothing to scale
            m = mn;
            l *= f;
#pragma unroll
            for (int e = 0; e < DP / 32; ++e) o[e] *= f;
        }
        // p = 2^(x - m); a row without a key so far: 2^-inf = 0.  An absent
        // key must stay at -inf: a zero multiplier would make it NaN
        const float less = add - (m == -INFINITY ? 0.0f : m);
        mul = mul == 0.0f ? 1e-38f : mul;
#pragma unroll
        for (int u = 0; u < NS; ++u) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[u][i] = __builtin_amdgcn_exp2f(fmaf(s[u][i], mul, less));
                l += s[u][i];
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                float x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = s[u][8 * t + j];
                // bf16 rows: p keeps 16 bits.  8 would cost O as much as its
                // own rounding (2.3e-3 of its norm off instead of 1.7e-3), and
                // an error of O is one of the backward pass's delta, which dq
                // has no other sum to correct by (rows of few keys: dq 2.4
                // times as far off as its rounding, 1.4 with 16)
                const Frag<PP> p = split8f<PP>(x);
#pragma unroll
                for (int e = 0; e < DP / 32; ++e) {
                    if constexpr (NP == 1) {
                        o[e] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[u].f[t][e], p.p[1], o[e], 0, 0, 0);
                        o[e] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[u].f[t][e], p.p[0], o[e], 0, 0, 0);
                    } else
                        o[e] = mma<NP>(frag_cols<NP, DP>(tl, vt, kPlane, 32 * u + 16 * t, e), p, o[e]);
                }
            }
        }
    }
};

// One finished row: O / l, or the partial row of a key split.
template <int NP>
__device__ inline void write_row4(const AttnArgs &a, const FwdOut &out, int split, int64_t at, int d, floatx4 v,
                                  float inv) {
    using T = typename RowOf<NP>::T;
    if (a.splits > 1) {
        float *p = out.part_o + ((int64_t)split * a.n_q * a.H + at) * a.D;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (d + i < a.D) p[d + i] = v[i];
        return;
    }
    T *o = (T *)out.o + at * a.D;
    v *= inv;
    float *rows = NP == 1 && out.rows ? out.rows + at * a.D : nullptr;
    if (a.out4) {
        if (d >= a.D) return;
        if (rows) *reinterpret_cast<floatx4 *>(rows + d) = v;
        if constexpr (NP == 1)
            *reinterpret_cast<bf16x4 *>(o + d) = __builtin_convertvector(v, bf16x4);
        else
            *reinterpret_cast<floatx4 *>(o + d) = v;
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (d + i < a.D) {
            o[d + i] = (T)v[i];
            if (rows) rows[d + i] = v[i];
        }
}

// Of a row's maximum (log2) and sum; no key: -inf, and the row is zeros.  A sum
// that is not a number stays one.
__device__ inline float log_sum(float m, float l) {
    return l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.69314718055994531f;
}
__device__ inline float inverse(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }

__device__ inline void write_stats(const AttnArgs &a, const FwdOut &out, int split, int64_t at, float m, float l) {
    if (a.splits > 1)
        out.part_ml[(int64_t)split * a.n_q * a.H + at] = make_float2(m, l);
    else if (out.lse)
        out.lse[at] = log_sum(m, l);
}

// One row and head by the definition in fp32, by one wavefront: where the
// products cannot give it.  They are sums over bf16 parts (of p, and of fp32
// rows), and the parts of an infinity or of what bf16 rounds to one are no sum;
// a large value may overflow beside p > 1.  Lanes take a key each for the
// scores and the running maximum and sum, then an element each for the row.
// q0, k0, nk: the segment's rows; row: the query's.
template <int NP>
__device__ inline void plain_row(const AttnArgs &a, const FwdOut &out, int row, int h, int q0, int k0, int nk, int lane) {
    using T = typename RowOf<NP>::T;
    const int hk = h / a.G;
    const T *q = (const T *)a.q + row * a.qs + h * a.qh;
    const T *K = (const T *)a.k + k0 * a.ks + hk * a.kh, *V = (const T *)a.v + k0 * a.vs + hk * a.vh;
    const int pos = a.q_pos ? a.q_pos[row] : row - q0;
    auto kept = [&](int j) { return j < nk && (!a.keep || a.keep[k0 + j]); };
    auto score = [&](int j) {   // in log2 units
        float dot = 0.0f;
#pragma unroll 1
        for (int d = 0; d < a.D; ++d) dot = fmaf(to_f32(q[d]), to_f32(K[(int64_t)j * a.ks + d]), dot);
        const float x = dot * (a.scale * kLog2e);
        if (!a.nb) return x;
        return x + bias_log2(a.bias[(int64_t)h * a.nb + bucket_of(a, offset_of(a.k_pos ? a.k_pos[k0 + j] : j, pos))]);
    };
    float m = -INFINITY, l = 0.0f;
#pragma unroll 1
    for (int j = lane; j < nk; j += 64) {
        const float x = kept(j) ? score(j) : -INFINITY;
        if (x == -INFINITY) continue;
        const float mn = fmaxf(m, x);   // (a score that is no number: the sum is none)
        l = (m == -INFINITY ? l : l * __builtin_amdgcn_exp2f(m - mn)) + __builtin_amdgcn_exp2f(x - mn);
        m = mn;
    }
    float top = m;
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    l = l == 0.0f ? 0.0f : l * __builtin_amdgcn_exp2f(m - top);
    for (int o = 32; o > 0; o >>= 1) l += __shfl_xor(l, o, 64);
    const float inv = inverse(l);
    float acc[2] = {0.0f, 0.0f};
#pragma unroll 1
    for (int j0 = 0; j0 < nk && l != 0.0f; j0 += 64) {
        const bool have = kept(j0 + lane);
        const float p = have ? __builtin_amdgcn_exp2f(score(j0 + lane) - top) * inv : 0.0f;
        uint64_t left = __ballot(have);
        while (left) {
            const int t = __ffsll((unsigned long long)left) - 1;
            left &= left - 1;
            const float pt = __shfl(p, t, 64);
            for (int u = 0; u < 2; ++u)
                if (lane + 64 * u < a.D) acc[u] = fmaf(pt, to_f32(V[(int64_t)(j0 + t) * a.vs + lane + 64 * u]), acc[u]);
        }
    }
    const int64_t at = (int64_t)row * a.H + h;
    for (int u = 0; u < 2; ++u) {
        const int d = lane + 64 * u;
        if (d >= a.D) continue;
        ((T *)out.o)[at * a.D + d] = (T)acc[u];
        if (NP == 1 && out.rows) out.rows[at * a.D + d] = acc[u];
    }
    if (lane == 0 && out.lse) out.lse[at] = log_sum(top, l);
}
// The kernel's first argument, read anew: what only the path above uses is not
// kept in scalar registers through the kernel.
__device__ inline const AttnArgs &args_anew() {
    auto p = (uint64_t)(const void *)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *(const AttnArgs *)p;
}
// Whether a sum is none of the ordinary ones, so that its row goes there.
__device__ inline bool beyond(float x) { return !(fabsf(x) <= 0x1p120f); }
template <int DP>
__device__ inline bool beyond(const floatx16 (&o)[DP / 32], float l) {
    bool b = beyond(l);
#pragma unroll
    for (int e = 0; e < DP / 32; ++e)
#pragma unroll
        for (int i = 0; i < 16; ++i) b |= beyond(o[e][i]);
    return b;
}

// Keys of a tile: 64 halve the barriers and the running sums' exchanges, 32
// where 64 would not leave registers for two blocks on a CU (2 x 2048 x 2048,
// 16 heads of 64, bf16: 79 us against 97 with 32; 15668 x 1000, 8 heads of
// 16, fp32: 103 against 111).
template <int NP, int DP>
constexpr int kRowKeys = DP == 32 || (NP == 1 && DP == 64) ? 64 : 32;

// Many rows: each wavefront owns 32 of the block's 128 rows and all of them
// read the same key tiles, staged in LDS while the tile before is computed:
// a tile is read from memory once for 128 rows and split into planes once.
// Two blocks on a CU let one wavefront's products run beside the other's
// softmax.  What bounds it is the softmax in series with the products: a score
// takes a dozen vector instructions and an exponential.  Measured: 2 x 4096 x
// 4096, 16 heads of 128 on 4, bf16: 470 us, 585 TFLOP/s of the 1220 that a
// large library product reaches (416 us with p in 8 bits); the vector units
// are 53 % busy, the matrix units 35 %, and a wavefront waits 28 % of its time.
// fp32, six products for one: 64 segments of up to 269 x 271, 4 heads of 32:
// 26 us, 40 TFLOP/s, half of a wavefront's time in waits (start and five tiles).
template <int NP, int DP, int KT, bool FAST>
__global__ __launch_bounds__(kAttnThreads, DP == 32 ? 3 : NP == 1 ? 2 : 1) void attn_rows_kernel(AttnArgs a, FwdOut out) {
    using T = typename RowOf<NP>::T;
    constexpr int kTile = NP * KT * DP;
    __shared__ __align__(256) bf16 tiles[2][2][kTile];   // [buffer][K, V]
    __shared__ KeyInfo<KT> info[2];
    extern __shared__ float lut[];   // [head of the subgroup][lut_stride]
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    RowBlock w;
    if (!locate(a, w)) return;
    if (w.tile * 128 >= w.nq * w.gs) return;
    const T *K = (const T *)a.k + w.k0 * a.ks + w.hk * a.kh, *V = (const T *)a.v + w.k0 * a.vs + w.hk * a.vh;
    const int n_tiles = (w.nk + KT - 1) / KT, per = (n_tiles + a.splits - 1) / a.splits;
    const int t0 = w.split * per, t1 = min(n_tiles, t0 + per);

    const TileLane<DP> tl(lane);
    const uint32_t lds0 = lds_offset(tiles);
    constexpr uint32_t kBytes = kTile * sizeof(bf16);
    TileMove<NP, DP, KT, kAttnThreads, FAST> mk, mv;
    KeyLoad<KT> kl;
    mk.init(a.ks, a.D, tid);
    mv.init(a.vs, a.D, tid);
    mk.seek(K + t0 * KT * a.ks, w.nk - t0 * KT);
    mv.seek(V + t0 * KT * a.vs, w.nk - t0 * KT);
    auto load = [&](int t) {
        mk.load(a.D, tid);
        mv.load(a.D, tid);
        kl.load(a, w, t * KT, a.nb && wave == 0, lane);
    };
    auto store = [&](int buf) {
        const uint64_t mask = kl.mask(a);
        mk.store(tiles[buf][0], tid, a.keep && is_partial<KT>(mask), mask);
        mv.store(tiles[buf][1], tid, a.keep && is_partial<KT>(mask), mask);
        if (a.nb && wave == 0) kl.store(info[buf], mask, lane);
        return mask;
    };
    // the first tile, the rows and the bias are on their way together
    uint64_t mask = 0;
    RowState<NP, DP, FAST> st;
    Raw8<NP> raw[DP / 16];
    if (t0 < t1) load(t0);
    st.begin(a, w, w.tile * 128 + wave * 32, lane, raw);
    if (a.nb) fill_lut(a, w, lut);
    if (t0 < t1) mask = store(0);
    if (t0 + 1 < t1) load(t0 + 1);
    st.finish(a, raw);
    const bool active = __any(st.row >= 0);
    __syncthreads();
    for (int t = t0; t < t1; ++t) {   // tile t is in LDS, t + 1 in registers or on its way there
        const int buf = (t - t0) & 1;
        if (active && mask)
            st.template step<KT>(a, tl, lds0 + 2 * buf * kBytes, lds0 + (2 * buf + 1) * kBytes, mask, info[buf], lut, lane);
        if (t + 1 < t1) mask = store(buf ^ 1);
        if (t + 2 < t1) load(t + 2);
        __syncthreads();
    }
    const float l = half_sum(st.l), inv = inverse(l);
    uint64_t odd = a.splits > 1 ? 0 : __ballot(st.row >= 0 && beyond<DP>(st.o, l));   // (joined first otherwise)
    odd = (odd | odd >> 32) & 0xffffffffull;
    if (st.row >= 0 && !((odd >> (lane & 31)) & 1)) {
        const int64_t at = (int64_t)st.row * a.H + w.h0 + st.g;
#pragma unroll
        for (int e = 0; e < DP / 32; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                write_row4<NP>(a, out, w.split, at, 32 * e + 8 * i + 4 * (lane >> 5),
                               floatx4{st.o[e][4 * i], st.o[e][4 * i + 1], st.o[e][4 * i + 2], st.o[e][4 * i + 3]}, inv);
        if (lane < 32) write_stats(a, out, w.split, at, st.m, l);
    }
    while (odd) {
        const int r = w.tile * 128 + wave * 32 + __ffsll((unsigned long long)odd) - 1;
        odd &= odd - 1;
        plain_row<NP>(args_anew(), out, w.q0 + r / w.gs, w.h0 + r % w.gs, w.q0, w.k0, w.nk, lane);
    }
}

// Few rows (at most 32 of a key/value head's subgroup): every wavefront
// holds all of them and takes every NW-th tile of 32 keys, with tiles of its
// own in LDS, so no wavefront waits for another until the rows are joined at
// the end.  The keys and values are read once, and that is what bounds it:
// 32 sequences of up to 16384 keys, 8 heads of 128, bf16: 293 us, 4.85 TB/s
// beside a large copy's 5.06 (1422 MB read, 1421 needed).  One row over 269 keys: 10 us, a launch and one
// chain of dependent loads, products and exchanges.
template <int NP, int DP, int NW, bool FAST>
__global__ __launch_bounds__(64 * NW) void attn_few_kernel(AttnArgs a, FwdOut out) {
    using T = typename RowOf<NP>::T;
    constexpr int kTile = NP * 32 * DP;
    constexpr int kJoin = NW * DP * 33 * 2;   // the wavefronts' O^T in fp32, as bf16 elements
    constexpr int kLds = 2 * NW * kTile > kJoin ? 2 * NW * kTile : kJoin;
    __shared__ __align__(256) bf16 lds[kLds];
    __shared__ KeyInfo<32> info[NW];
    extern __shared__ float lut[];   // [head of the subgroup][lut_stride]
    __shared__ float wave_m[NW][32], wave_l[NW][32];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    RowBlock w;
    if (!locate(a, w)) return;
    if (w.tile * 32 >= w.nq * w.gs) return;
    const T *K = (const T *)a.k + w.k0 * a.ks + w.hk * a.kh, *V = (const T *)a.v + w.k0 * a.vs + w.hk * a.vh;
    const int n_tiles = (w.nk + 31) / 32, per = (n_tiles + a.splits - 1) / a.splits;
    const int t0 = w.split * per, t1 = min(n_tiles, t0 + per);
    bf16 *kt = lds + 2 * wave * kTile, *vt = kt + kTile;

    TileMove<NP, DP, 32, 64, FAST> mk, mv;
    KeyLoad<32> kl;
    mk.init(a.ks, a.D, lane);
    mv.init(a.vs, a.D, lane);
    int t = t0 + wave;
    mk.seek(K + t * 32 * a.ks, w.nk - t * 32);
    mv.seek(V + t * 32 * a.vs, w.nk - t * 32);
    auto load = [&](int t) {
        mk.load(a.D, lane, 32 * NW);
        mv.load(a.D, lane, 32 * NW);
        kl.load(a, w, t * 32, a.nb, lane);
    };
    if (t < t1) load(t);
    RowState<NP, DP, FAST> st;
    Raw8<NP> raw[DP / 16];
    st.begin(a, w, w.tile * 32, lane, raw);
    if (a.nb) fill_lut(a, w, lut);
    st.finish(a, raw);
    const TileLane<DP> tl(lane);
    const uint32_t lds_k = uniform((int)lds_offset(kt)), lds_v = lds_k + kTile * sizeof(bf16);
    __syncthreads();
    for (; t < t1; t += NW) {
        const uint64_t mask = kl.mask(a);
        mk.store(kt, lane, a.keep && is_partial<32>(mask), mask);
        mv.store(vt, lane, a.keep && is_partial<32>(mask), mask);
        if (a.nb) kl.store(info[wave], mask, lane);
        wave_sync();
        if (t + NW < t1) load(t + NW);
        if (mask) st.template step<32>(a, tl, lds_k, lds_v, mask, info[wave], lut, lane);
        wave_sync();
    }
    // join the wavefronts' rows, in their order
    const float lw = half_sum(st.l);
    const uint64_t far = __ballot(beyond<DP>(st.o, lw));
    if (lane < 32) {
        wave_m[wave][lane] = st.m;
        wave_l[wave][lane] = ((far | far >> 32) >> lane) & 1 ? NAN : lw;   // (and so of all of the row)
    }
    __syncthreads();
    float m = -INFINITY, l = 0.0f;
    for (int v = 0; v < NW; ++v) m = fmaxf(m, wave_m[v][lane & 31]);
    for (int v = 0; v < NW; ++v)
        if (wave_l[v][lane & 31] != 0.0f)
            l += wave_l[v][lane & 31] * __builtin_amdgcn_exp2f(wave_m[v][lane & 31] - m);
    const int n = min(32, w.nq * w.gs - w.tile * 32);
    const uint32_t odd = a.splits > 1 ? 0 : (uint32_t)__ballot(lane < n && beyond(l));   // (split rows: joined first)
    const float f = st.m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(st.m - m);
    float *rows = reinterpret_cast<float *>(lds);   // [wavefront][DP][33]
#pragma unroll
    for (int e = 0; e < DP / 32; ++e)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            rows[(wave * DP + 32 * e + 8 * (i / 4) + 4 * (lane >> 5) + i % 4) * 33 + (lane & 31)] = st.o[e][i] * f;
    __syncthreads();
    if (tid < 32 && st.row >= 0 && !((odd >> lane) & 1)) write_stats(a, out, w.split, (int64_t)st.row * a.H + w.h0 + st.g, m, l);
    if (wave == 0 && lane < 32) wave_l[0][lane] = inverse(l);
    __syncthreads();
    for (int i = tid; i < n * (DP / 4); i += 64 * NW) {
        const int r = i / (DP / 4), d = (i % (DP / 4)) * 4, rr = w.tile * 32 + r;
        if ((odd >> r) & 1) continue;
        const int64_t at = (int64_t)(w.q0 + rr / w.gs) * a.H + w.h0 + rr % w.gs;
        floatx4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < NW; ++v)
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] += rows[(v * DP + d + j) * 33 + r];
        write_row4<NP>(a, out, w.split, at, d, x, wave_l[0][r]);
    }
    for (int r = wave; r < 32 && odd; r += NW)
        if ((odd >> r) & 1) {
            const int rr = w.tile * 32 + r;
            plain_row<NP>(args_anew(), out, w.q0 + rr / w.gs, w.h0 + rr % w.gs, w.q0, w.k0, w.nk, lane);
        }
}

// Join the key splits of a row: one wavefront per row and head (9 us for 1024
// rows of 128 in 4 splits: a launch and two dependent loads).
template <int NP>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, FwdOut out) {
    using T = typename RowOf<NP>::T;
    const int64_t rows = (int64_t)a.n_q * a.H, at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (at >= rows) return;
    float m = -INFINITY, l = 0.0f;
    for (int k = 0; k < a.splits; ++k) m = fmaxf(m, out.part_ml[k * rows + at].x);
    float acc[2] = {0.0f, 0.0f};
    for (int k = 0; k < a.splits; ++k) {
        const float2 p = out.part_ml[k * rows + at];
        if (p.y == 0.0f) continue;   // no key in this split
        const float f = __builtin_amdgcn_exp2f(p.x - m);
        l = fmaf(p.y, f, l);
        for (int u = 0; u < 2; ++u)
            if (lane + 64 * u < a.D) acc[u] = fmaf(out.part_o[(k * rows + at) * a.D + lane + 64 * u], f, acc[u]);
    }
    if (__any(beyond(l) || beyond(acc[0]) || beyond(acc[1]))) {
        const int row = uniform((int)(at / a.H));
        int q0 = 0, nq = 0, k0 = 0, nk = 0;
        for (int b = 0; b < a.B && !(row >= q0 && row < q0 + nq); ++b) {   // its segment
            segment_rows(a.q_ptr, b, a.B, a.n_q, a.max_q, a.status, q0, nq);
            segment_rows(a.k_ptr, b, a.B, a.n_k, a.max_k, a.status, k0, nk);
        }
        if (row >= q0 && row < q0 + nq) plain_row<NP>(args_anew(), out, row, (int)(at % a.H), q0, k0, nk, lane);
        return;
    }
    const float inv = inverse(l);
    for (int u = 0; u < 2; ++u) {
        const int d = lane + 64 * u;
        if (d >= a.D) continue;
        ((T *)out.o)[at * a.D + d] = (T)(acc[u] * inv);
        if (NP == 1 && out.rows) out.rows[at * a.D + d] = acc[u] * inv;
    }
    if (lane == 0 && out.lse) out.lse[at] = log_sum(m, l);
}

// How the rows are cut: few rows or many, row tiles, key splits.
//
// Few: where a key/value head's rows fill one wavefront at most, each of the
// others would only repeat or idle (64 segments of 32 x 271, fp32, heads of
// 32: 12.7 us against 19.0 with the kernel for many; 16 of 32 x 2048, bf16,
// heads of 64: 26 against 30).  Two wavefronts' rows go to the other (64 x
// 271: 19.5 against 21.9; 64 of 64 x 600, 8 heads, bf16: 32 against 44 for
// heads of 64, 45 against 73 for 128), also where few blocks of bf16 rows
// would gain from this one (32 of 64 x 1024, 8 heads of 128: 59 against 49).
//
// Splits: as many as give every CU a block (few) or two (many), as long as
// each has 1024 or 256 keys to pay for its start and the join.  One row over
// 16384 keys of 8 heads: 179 us unsplit, 53 us from 512 keys, 42 us from
// 1024, 43 us from 2048, where 4 x 4096 is 36 instead of 28 us; one block for
// every CU instead of four: 16 x 4096, bf16, heads of 64, 40 -> 35 us.  Many,
// 40 x 4096 of 8 heads: 94 us unsplit, 29.3 with two blocks, 29.6 with four.
struct FwdPlan {
    bool few;
    int Gs, subs, row_tiles, splits;
};

FwdPlan fwd_plan(int B, int Hkv, int G, int max_q, int max_k, int lut_n) {
    FwdPlan p;
    p.Gs = std::max(1, std::min({8, G, kLutMax / std::max(1, lut_n)}));
    p.subs = (G + p.Gs - 1) / p.Gs;
    p.few = (int64_t)max_q * p.Gs <= 32;
    p.row_tiles = std::max<int64_t>(1, ((int64_t)max_q * p.Gs + (p.few ? 31 : 127)) / (p.few ? 32 : 128));
    const int64_t blocks = (int64_t)B * Hkv * p.subs * p.row_tiles;
    const int64_t want = p.few ? 256 : 512, least = p.few ? 1024 : 256;
    p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(want / blocks, max_k / least));
    return p;
}

// Wavefronts of a few-rows block: 160 KB of LDS hold their tiles.
constexpr int few_waves(int np, int dp) { return np * dp <= 96 ? 8 : np * dp <= 192 ? 4 : 2; }

bool fits(const FwdPlan &p, int B, int Hkv, int waves) {
    return grid_fits((int64_t)B * Hkv * p.subs * p.splits * p.row_tiles + kXcds, p.few ? 64 * waves : kAttnThreads);
}

template <int NP, int DP, bool FAST>
sn_status launch(const AttnArgs &a, const FwdOut &out, const FwdPlan &p, hipStream_t s) {
    if (!fits(p, a.B, a.Hkv, few_waves(NP, DP))) return SN_ERR_INVALID;
    const int grid = xcd_grid(a.B * a.Hkv * a.subs * a.splits * a.row_tiles);
    constexpr int NW = few_waves(NP, DP);
    const size_t lut = a.nb ? (size_t)a.Gs * (a.lut_n + 2 * kLutPad) * sizeof(float) : 0;
    if (p.few)
        attn_few_kernel<NP, DP, NW, FAST><<<grid, 64 * NW, lut, s>>>(a, out);
    else
        attn_rows_kernel<NP, DP, kRowKeys<NP, DP>, FAST><<<grid, kAttnThreads, lut, s>>>(a, out);
    SN_TRY(launch_status());
    if (a.splits > 1) {
        attn_join_kernel<NP><<<(int)(((int64_t)a.n_q * a.H + 3) / 4), 256, 0, s>>>(a, out);
        SN_TRY(launch_status());
    }
    return SN_OK;
}

template <int NP, bool FAST>
sn_status launch_dim(const AttnArgs &a, const FwdOut &out, const FwdPlan &p, hipStream_t s) {
    if (a.D <= 32) return launch<NP, 32, FAST>(a, out, p, s);
    if (a.D <= 64) return launch<NP, 64, FAST>(a, out, p, s);
    return launch<NP, 128, FAST>(a, out, p, s);
}

}  // namespace

// The thresholds, which are not read here, decide how many heads share a
// table (1 to 8): the plan of each.
static FwdPlan plan_of(const sn_cross_attention &op, int heads) {
    return fwd_plan(op.n_segments, op.n_kv_heads, op.n_heads / op.n_kv_heads, op.max_q, op.max_k, kLutMax / heads);
}

bool attn_forward_fits(const sn_cross_attention &op) {
    const int dp = op.head_dim <= 32 ? 32 : op.head_dim <= 64 ? 64 : 128;
    for (int heads = 1; heads <= 8; ++heads)
        if (fits(plan_of(op, heads), op.n_segments, op.n_kv_heads, few_waves(op.dtype == SN_F32 ? 3 : 1, dp))) return true;
    return false;
}

size_t attn_forward_workspace(const sn_cross_attention &op) {
    size_t splits = 1;
    for (int heads = 1; heads <= 8; ++heads) splits = std::max<size_t>(splits, plan_of(op, heads).splits);
    if (splits == 1) return kWsBase;
    const size_t rows = (size_t)op.n_q * op.n_heads;
    return kWsBase + align256(rows * splits * sizeof(float2)) + align256(rows * splits * op.head_dim * sizeof(float));
}

sn_status attn_forward(AttnArgs a, int dtype, void *o, float *rows, float *lse, char *ws, hipStream_t s) {
    ProfScope prof(K_ATTN_FWD, s);
    const FwdPlan p = fwd_plan(a.B, a.Hkv, a.G, a.max_q, a.max_k, a.lut_n);
    a.Gs = p.Gs; a.subs = p.subs; a.row_tiles = p.row_tiles; a.splits = p.splits;
    const size_t n = (size_t)a.n_q * a.H;
    FwdOut out{o, dtype == SN_BF16 ? rows : nullptr, lse, nullptr, nullptr};
    if (p.splits > 1) {
        out.part_ml = reinterpret_cast<float2 *>(ws + kWsBase);
        out.part_o = reinterpret_cast<float *>(ws + kWsBase + align256(n * p.splits * sizeof(float2)));
    }
    if (dtype == SN_F32) return a.fast ? launch_dim<3, true>(a, out, p, s) : launch_dim<3, false>(a, out, p, s);
    return a.fast ? launch_dim<1, true>(a, out, p, s) : launch_dim<1, false>(a, out, p, s);
}

}  // namespace sn
