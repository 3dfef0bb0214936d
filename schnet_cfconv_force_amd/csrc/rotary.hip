// Norm of each head and rotation of its pairs by positions, forward and
// backward.
//
//   xh = x rstd, rstd = 1 / sqrt(mean x^2 + eps), z = w xh
//   pair (a, b) turns by t = position frequency:
//     y_a = z_a cos t - z_b sin t,  y_b = z_b cos t + z_a sin t
//   g = dy turned back, dw = sum g xh, h = g w, dx = rstd (h - xh mean(h xh))
//
// What it costs is one read and one write of the rows (32768 rows of 32 + 8 heads
// of 128, bf16, 671 MB: 133 us, 5.1 TB/s, a copy's rate).  A group of lanes owns a
// head, a lane V of its pairs: its elements are two vectors of V (a's and b's,
// or adjacent pairs), so a pair never leaves the lane.  A block's groups take
// the heads of its rows in memory's order (lanes that walk the heads of a row of
// their own spread a wavefront over eight rows: 153 us).  The block forms the
// sines and cosines of its rows once, for all heads, in LDS.  Where pairs do not
// come in fours a lane takes single elements, at 2 to 4 TB/s (runs_of).
#include <algorithm>

#include "state.h"

namespace sn {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPartials = 1024;   // blocks of a backward pass, and with them partial weight gradients
constexpr int kHeads = 4;               // of a group, on their way at once
// Blocks that a pass makes before a block takes more rows than one.  Forward and
// backward replayed from a graph (called, the host adds to the shorter ones): 7001
// rows of 6 + 2 heads of 40, bf16, 17.4 us with 512, 21.9 with 1024, 48 with 4096,
// 17.5 with 256; 17216 rows of 4 + 4 heads of 32, fp32, 26.0, 24.0, 35 and 26.0.
constexpr int kBlocks = 512;
// Outputs beyond this stay in no cache until they are read: they are stored past
// it (32768 rows of 32 + 8 heads of 128, bf16: 143 us -> 135; 16384, a step: 181
// -> 149; 17216 rows of 4 + 4 heads of 32, fp32, 18 MB: 9.9 -> 9.1; with smaller
// ones, which the next kernel finds in the cache, there is nothing to gain).
constexpr int64_t kStream = 16 << 20;

// How rows and heads are cut (host).  A block takes `rows` rows at a time; their
// heads, in memory's order, go to its groups one each in turn.
struct RotaryCut {
    int units;      // lanes of a group that have pairs
    int lane_bits;  // a group has 2^lane_bits lanes
    int width;      // pairs of a row in the block's table of angles
    int rows;
    int step_row[2], step_head[2];      // of q and of k: from one head of a group to its next
    int blocks[2];  // of q and of k (grid y)
    float inv_D;
    bool stream;    // stores go past the caches
    bool single;    // one block of q and one of k (backward): no sums are left to join
};

template <typename T, int V>
struct VecOf { typedef T type __attribute__((ext_vector_type(V))); };

// A lane's two runs of elements.
struct Place {
    int a, b;       // first elements
    int pair;       // the first pair
    int turned;     // pairs that turn, the lane's first: of adjacent ones some, else all or none
    bool has_a, has_b;
};
template <int V, bool IL>
__device__ inline Place place_of(int u, int units, int D, int P) {
    Place p;
    p.pair = u * V;
    p.turned = max(0, min(P - p.pair, V));
    if (IL) {
        p.a = 2 * V * u;
        p.b = p.a + V;
    } else if (p.turned) {
        p.a = u * V;
        p.b = P + u * V;
    } else {                    // what does not turn, in order
        p.a = 2 * V * u;
        p.b = p.a + V;
    }
    p.has_a = u < units && p.a < D;
    p.has_b = u < units && p.b < D;
    return p;
}

// A run as it lies in memory, zero where the row does not have it.
template <typename T, int V>
struct Run {
    typename VecOf<T, V>::type v;
    __device__ inline void load(const T *p, bool has) {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = (T)0.0f;
        if (!has) return;
        if constexpr (V == 1)
            v[0] = p[0];
        else
            v = *reinterpret_cast<const typename VecOf<T, V>::type *>(p);
    }
    __device__ inline void get(float *x) const {
#pragma unroll
        for (int e = 0; e < V; ++e) x[e] = to_f32(v[e]);
    }
};
template <typename T, int V>
__device__ inline void store_run(T *p, bool has, const float *x, bool stream) {
    if (!has) return;
    if constexpr (V == 1) {
        p[0] = (T)x[0];
    } else {
        typename VecOf<T, V>::type v;
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = (T)x[e];
        store_past<1>(&v, reinterpret_cast<typename VecOf<T, V>::type *>(p), stream);
    }
}

// Sum over a group of lanes, a power of two, in every lane: neighbours and
// pairs within four, mirrors of eight and sixteen, then the swaps of rows.
template <int CTRL>
__device__ inline float dpp_sum(float v) {
    const int x = __float_as_int(v);
    return v + __int_as_float(__builtin_amdgcn_update_dpp(x, x, CTRL, 0xf, 0xf, true));
}
__device__ inline float group_sum(float v, int lanes) {
    if (lanes > 1) v = dpp_sum<0xb1>(v);        // quad_perm 1 0 3 2
    if (lanes > 2) v = dpp_sum<0x4e>(v);        // quad_perm 2 3 0 1
    if (lanes > 4) v = dpp_sum<0x141>(v);       // row_half_mirror
    if (lanes > 8) v = dpp_sum<0x140>(v);       // row_mirror
    if (lanes > 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    if (lanes > 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    return v;
}

// Sines and cosines of a block's rows, in LDS: once for all heads.  Angles in
// full turns are reduced in fp64; what is left is at most half a turn, in fp32 with
// its rounding as a small second turn.  Pairs that do not turn have an angle of zero.
constexpr int kTable = 1024;
__device__ inline void fill_table(const RotaryArgs &a, const RotaryCut &k, int row0, int rows, float2 *table) {
    for (int i = threadIdx.x; i < rows * k.width; i += kThreads) {
        const int r = i / k.width, j = i - r * k.width;
        float2 cs = make_float2(1.0f, 0.0f);
        if (j < a.P) {
            const double turn = (double)a.positions[(int64_t)a.axes[j] * a.n_rows + row0 + r] * a.turns[j], part = turn - rint(turn);
            const float near = (float)part, rest = (float)(2.0 * M_PI) * (float)(part - (double)near);
            float sine, cosine;
            sincospif(2.0f * near, &sine, &cosine);
            cs = make_float2(fmaf(-sine, rest, cosine), fmaf(cosine, rest, sine));
        }
        table[i] = cs;
    }
}
template <int V>
__device__ inline void take_angles(const float2 *table, float (&c)[V], float (&s)[V]) {
    if constexpr (V == 1) {
        c[0] = table[0].x;
        s[0] = table[0].y;
    } else {
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            const float4 x = *reinterpret_cast<const float4 *>(table + e);
            c[e] = x.x;
            s[e] = x.y;
            c[e + 1] = x.z;
            s[e + 1] = x.w;
        }
    }
}

// What does not turn is left alone: an infinity times a sine of zero would reach its neighbour.
template <int V, bool IL>
__device__ inline void turn(float (&x)[2 * V], const Place &p, const float (&c)[V], const float (&s)[V], float sign) {
    if (p.turned == 0) return;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        float &a = x[IL ? 2 * e : e], &b = x[IL ? 2 * e + 1 : V + e];
        const float ta = a * c[e] - sign * b * s[e], tb = b * c[e] + sign * a * s[e];
        a = !IL || e < p.turned ? ta : a;
        b = !IL || e < p.turned ? tb : b;
    }
}

template <int V>
__device__ inline void load_weights(const float *weights, const Place &p, float (&w)[2 * V]) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
        w[e] = weights && p.has_a ? weights[p.a + e] : 1.0f;
        w[V + e] = weights && p.has_b ? weights[p.b + e] : 1.0f;
    }
}

// A group's heads in turn.
struct Head {
    int row, head;      // row of the block's
    __device__ inline void next(const RotaryCut &k, int n, int heads) {
        row += k.step_row[n];
        head += k.step_head[n];
        if (head >= heads) {
            head -= heads;
            ++row;
        }
    }
};

// N heads of a group are on their way at once.
template <typename T, int V, bool IL, bool NORM, int N>
__global__ __launch_bounds__(kThreads) void rotary_forward_kernel(RotaryArgs a, RotaryCut k) {
    __shared__ alignas(16) float2 table[kTable];
    const int n = blockIdx.y;
    if ((int)blockIdx.x >= k.blocks[n]) return;
    const RotaryTensor &t = a.t[n];
    const int heads = n ? a.Hkv : a.H, lanes = 1 << k.lane_bits, u = threadIdx.x & (lanes - 1);
    const int row0 = blockIdx.x * k.rows, rows = min(k.rows, a.n_rows - row0);
    const Place p = place_of<V, IL>(u, k.units, a.D, a.P);
    const int group = threadIdx.x >> k.lane_bits;
    Head at{group / heads, group % heads};
    float w[2 * V];
    bool filled = false;
    while (true) {
        Head h[N];
        Run<T, V> ra[N], rb[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            h[i] = at;
            at.next(k, n, heads);
            const bool has = h[i].row < rows;
            const T *from = static_cast<const T *>(t.x) + (row0 + h[i].row) * t.xs + h[i].head * t.xh;
            ra[i].load(from + p.a, p.has_a && has);
            rb[i].load(from + p.b, p.has_b && has);
        }
        if (!filled) {      // the first heads are on their way meanwhile
            if (NORM) load_weights<V>(t.w, p, w);
            fill_table(a, k, row0, rows, table);
            __syncthreads();
            filled = true;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (h[i].row >= rows) return;
            float v[2 * V], c[V], s[V];
            ra[i].get(v);
            rb[i].get(v + V);
            take_angles<V>(table + h[i].row * k.width + min(p.pair, k.width - V), c, s);
            if (NORM) {
                float sq = 0.0f;
#pragma unroll
                for (int e = 0; e < 2 * V; ++e) sq += v[e] * v[e];
                const float r = __builtin_amdgcn_rsqf(group_sum(sq, lanes) * k.inv_D + a.eps);
#pragma unroll
                for (int e = 0; e < 2 * V; ++e) v[e] *= r * w[e];
            }
            turn<V, IL>(v, p, c, s, 1.0f);
            T *to = static_cast<T *>(t.out) + ((int64_t)(row0 + h[i].row) * heads + h[i].head) * a.D;
            store_run<T, V>(to + p.a, p.has_a, v, k.stream);
            store_run<T, V>(to + p.b, p.has_b, v + V, k.stream);
        }
    }
}

// Runs of rows in turn by blocks; a block leaves the weight gradients of its
// rows in partials[q, k][block][D], the only one in their place.
template <typename T, int V, bool IL, bool NORM, int N>
__global__ __launch_bounds__(kThreads) void rotary_backward_kernel(RotaryArgs a, RotaryCut k, float *partials, float *dq_weight,
                                                                   float *dk_weight) {
    __shared__ alignas(16) float2 table[kTable];
    __shared__ float sums[NORM ? kThreads * 2 * V : 1];
    const int n = blockIdx.y;
    if ((int)blockIdx.x >= k.blocks[n]) return;
    const RotaryTensor &t = a.t[n];
    const int heads = n ? a.Hkv : a.H, lanes = 1 << k.lane_bits, u = threadIdx.x & (lanes - 1), groups = kThreads >> k.lane_bits;
    const Place p = place_of<V, IL>(u, k.units, a.D, a.P);
    const int group = threadIdx.x >> k.lane_bits;
    float dw[2 * V] = {}, w[2 * V];
    if (NORM) load_weights<V>(t.w, p, w);
    for (int64_t row0 = (int64_t)blockIdx.x * k.rows; row0 < a.n_rows; row0 += (int64_t)k.blocks[n] * k.rows) {
        const int rows = (int)min((int64_t)k.rows, a.n_rows - row0);
        Head at{group / heads, group % heads};
        bool filled = false;
        while (at.row < rows || !filled) {
            Head h[N];
            Run<T, V> xa[N], xb[N], ga[N], gb[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                h[i] = at;
                at.next(k, n, heads);
                const bool has = h[i].row < rows;
                const T *from = static_cast<const T *>(t.dy) + (row0 + h[i].row) * t.gs + h[i].head * t.gh;
                ga[i].load(from + p.a, p.has_a && has);
                gb[i].load(from + p.b, p.has_b && has);
                if (NORM) {
                    const T *x = static_cast<const T *>(t.x) + (row0 + h[i].row) * t.xs + h[i].head * t.xh;
                    xa[i].load(x + p.a, p.has_a && has);
                    xb[i].load(x + p.b, p.has_b && has);
                }
            }
            if (!filled) {
                __syncthreads();        // the rows before are done with the table
                fill_table(a, k, (int)row0, rows, table);
                __syncthreads();
                filled = true;
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (h[i].row >= rows) break;
                float g[2 * V], c[V], s[V];
                ga[i].get(g);
                gb[i].get(g + V);
                take_angles<V>(table + h[i].row * k.width + min(p.pair, k.width - V), c, s);
                turn<V, IL>(g, p, c, s, -1.0f);
                if (NORM) {
                    float v[2 * V];
                    xa[i].get(v);
                    xb[i].get(v + V);
                    float sq = 0.0f, dot = 0.0f;
#pragma unroll
                    for (int e = 0; e < 2 * V; ++e) {
                        sq += v[e] * v[e];
                        dot += g[e] * w[e] * v[e];
                    }
                    const float r = __builtin_amdgcn_rsqf(group_sum(sq, lanes) * k.inv_D + a.eps);
                    const float m = group_sum(dot, lanes) * k.inv_D * r * r;
#pragma unroll
                    for (int e = 0; e < 2 * V; ++e) {
                        dw[e] += g[e] * (v[e] * r);
                        g[e] = r * (g[e] * w[e] - v[e] * m);
                    }
                }
                T *to = static_cast<T *>(t.out) + ((row0 + h[i].row) * heads + h[i].head) * a.D;
                store_run<T, V>(to + p.a, p.has_a, g, k.stream);
                store_run<T, V>(to + p.b, p.has_b, g + V, k.stream);
            }
        }
    }
    if (!NORM || !(n ? dk_weight : dq_weight)) return;
    // the only block has the whole sums
    float *out = k.single ? (n ? dk_weight : dq_weight) : partials + ((int64_t)n * kMaxPartials + blockIdx.x) * a.D;
#pragma unroll
    for (int e = 0; e < 2 * V; ++e) sums[e * kThreads + threadIdx.x] = dw[e];
    __syncthreads();
    // element e of lane u, of all groups
    for (int i = threadIdx.x; i < k.units * 2 * V; i += kThreads) {
        const int lane = i % k.units, e = i / k.units;
        const float *of = sums + e * kThreads + lane;
        double part[4] = {};        // up to 256 groups' sums: one after the other in fp32 they lost some digits
        for (int g = 0; g < groups; g += 4)
#pragma unroll
            for (int j = 0; j < 4; ++j) part[j] += of[(g + j) << k.lane_bits];
        const float sum = (float)((part[0] + part[1]) + (part[2] + part[3]));
        const Place p = place_of<V, IL>(lane, k.units, a.D, a.P);
        const int d = e < V ? p.a + e : p.b + e - V;
        if (d < a.D) out[d] = sum;
    }
}

// dw[d] of q and of k = the sum of the blocks' partials, in one order, in fp64.
__global__ __launch_bounds__(kThreads) void rotary_weights_kernel(const float *partials, RotaryCut k, int D, float *dq_weight,
                                                                  float *dk_weight) {
    __shared__ double sums[kThreads];
    const int n = blockIdx.y, d = blockIdx.x;
    float *out = n ? dk_weight : dq_weight;
    if (!out) return;
    double sum = 0.0;
    for (int b = threadIdx.x; b < k.blocks[n]; b += kThreads) sum += partials[((int64_t)n * kMaxPartials + b) * D + d];
    sums[threadIdx.x] = sum;
    for (int o = kThreads / 2; o > 0; o >>= 1) {
        __syncthreads();
        if (threadIdx.x < o) sums[threadIdx.x] += sums[threadIdx.x + o];
    }
    if (threadIdx.x == 0) out[d] = (float)sums[0];
}

// A lane's vector length: as long as every run of V elements lies whole in
// one aligned place of every tensor, else 1 (32768 rows of 32 + 8 heads of 128,
// bf16, 64 pairs in halves 132 us, 37 pairs 212, a step 322 and 559; of 80, 10
// pairs in halves 205, adjacent 110; 8 + 8 heads of 20, fp32, 84 MB: 24).
template <typename T>
bool runs_of(const RotaryArgs &a, int V, bool backward) {
    if (a.D % (2 * V) != 0 || (!a.interleaved && a.P % V != 0)) return false;
    auto fits = [&](const void *p, int64_t s, int64_t h) {
        return (reinterpret_cast<uintptr_t>(p) & (V * sizeof(T) - 1)) == 0 && s % V == 0 && h % V == 0;
    };
    for (int n = 0; n < (a.Hkv ? 2 : 1); ++n) {
        const RotaryTensor &t = a.t[n];
        if (!fits(t.x, t.xs, t.xh) || !fits(t.out, 0, 0)) return false;
        if (backward && !fits(t.dy, t.gs, t.gh)) return false;
    }
    return true;
}

RotaryCut cut_of(const RotaryArgs &a, int V, int size, bool backward) {
    RotaryCut k;
    k.units = (a.D + 2 * V - 1) / (2 * V);
    k.lane_bits = 0;
    while (1 << k.lane_bits < k.units) ++k.lane_bits;
    k.width = k.units * V;
    k.inv_D = 1.0f / (float)a.D;
    k.stream = (int64_t)a.n_rows * (a.H + a.Hkv) * a.D * size > kStream;
    const int groups = kThreads >> k.lane_bits;
    // four heads a group, and rows for kBlocks blocks
    k.rows = std::min(std::max(1, kHeads * groups / a.H), kTable / k.width);
    k.rows = std::max(1, std::min(k.rows, a.n_rows / kBlocks));
    // Four heads a group are one block's: a launch that joins the weights' sums costs
    // more than more blocks give (forward and backward of 4 + 4 heads of 32, fp32,
    // with the join and without: 1 row 23.6 and 21.4 us, 64 rows 23.5 and 20.8;
    // replayed from a graph 9.9 and 7.5, 10.6 and 11.1: no longer than that). Keys
    // there must be, for the join also writes the zeros of a weight without heads.
    k.single = backward && a.n_rows > 0 && a.Hkv > 0 && a.n_rows <= kTable / k.width &&
               (int64_t)a.n_rows * std::max(a.H, a.Hkv) <= kHeads * groups;
    if (k.single) k.rows = a.n_rows;
    for (int n = 0; n < 2; ++n) {
        const int heads = n ? a.Hkv : a.H;
        k.step_row[n] = heads ? groups / heads : 0;
        k.step_head[n] = heads ? groups % heads : 0;
        const int blocks = heads ? (a.n_rows + k.rows - 1) / k.rows : 0;
        k.blocks[n] = backward ? std::min(blocks, kMaxPartials) : blocks;
    }
    return k;
}

template <typename T, int V, bool IL, bool NORM>
sn_status launch(const RotaryArgs &a, float *partials, bool backward, float *dqw, float *dkw, hipStream_t s) {
    const RotaryCut k = cut_of(a, V, (int)sizeof(T), backward);
    ProfScope prof(backward ? K_ROTARY_BWD : K_ROTARY_FWD, s);
    const dim3 grid(std::max(k.blocks[0], k.blocks[1]), a.Hkv ? 2 : 1);
    // several heads of a group on their way where it has them
    const bool many = (int64_t)k.rows * std::max(a.H, a.Hkv) > (kThreads >> k.lane_bits);
    if (grid.x > 0) {       // no rows: the weights' zeros alone
        if (!backward) {
            if (many)
                rotary_forward_kernel<T, V, IL, NORM, kHeads><<<grid, kThreads, 0, s>>>(a, k);
            else
                rotary_forward_kernel<T, V, IL, NORM, 1><<<grid, kThreads, 0, s>>>(a, k);
            return launch_status();
        }
        if (many)
            rotary_backward_kernel<T, V, IL, NORM, 2><<<grid, kThreads, 0, s>>>(a, k, partials, dqw, dkw);
        else
            rotary_backward_kernel<T, V, IL, NORM, 1><<<grid, kThreads, 0, s>>>(a, k, partials, dqw, dkw);
        SN_TRY(launch_status());
    }
    if (NORM && !k.single && (dqw || dkw)) rotary_weights_kernel<<<dim3(a.D, 2), kThreads, 0, s>>>(partials, k, a.D, dqw, dkw);
    return launch_status();
}

template <typename T, int V>
sn_status launch(const RotaryArgs &a, bool norm, float *partials, bool backward, float *dqw, float *dkw, hipStream_t s) {
    if (a.interleaved)
        return norm ? launch<T, V, true, true>(a, partials, backward, dqw, dkw, s)
                    : launch<T, V, true, false>(a, partials, backward, dqw, dkw, s);
    return norm ? launch<T, V, false, true>(a, partials, backward, dqw, dkw, s)
                : launch<T, V, false, false>(a, partials, backward, dqw, dkw, s);
}

sn_status launch(const RotaryArgs &a, int dtype, bool norm, float *partials, bool backward, float *dqw, float *dkw,
                 hipStream_t s) {
    if (dtype == SN_F32) {
        if (runs_of<float>(a, 4, backward)) return launch<float, 4>(a, norm, partials, backward, dqw, dkw, s);
        return launch<float, 1>(a, norm, partials, backward, dqw, dkw, s);
    }
    if (runs_of<bf16>(a, 8, backward)) return launch<bf16, 8>(a, norm, partials, backward, dqw, dkw, s);
    if (runs_of<bf16>(a, 4, backward)) return launch<bf16, 4>(a, norm, partials, backward, dqw, dkw, s);
    return launch<bf16, 1>(a, norm, partials, backward, dqw, dkw, s);
}

}  // namespace

size_t rotary_workspace(const sn_head_rotary &op) {
    return kWsBase + (size_t)kMaxPartials * 2 * op.head_dim * sizeof(float);
}

// A forward pass has at most a block for every row.
bool rotary_fits(const sn_head_rotary &op) { return grid_fits(op.n_rows, kThreads); }

sn_status rotary_forward(const RotaryArgs &a, int dtype, bool norm, hipStream_t s) {
    return launch(a, dtype, norm, nullptr, false, nullptr, nullptr, s);
}

sn_status rotary_backward(const RotaryArgs &a, int dtype, bool norm, float *dq_weight, float *dk_weight, char *ws,
                          hipStream_t s) {
    return launch(a, dtype, norm, reinterpret_cast<float *>(ws + kWsBase), true, dq_weight, dk_weight, s);
}

}  // namespace sn
