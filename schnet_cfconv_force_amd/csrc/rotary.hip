// Norm of each head and rotation of its pairs by positions, forward and
// backward.
//
//   xh = x rstd, rstd = 1 / sqrt(mean x^2 + eps), z = w xh
//   pair (a, b) turns by t = position frequency:
//     y_a = z_a cos t - z_b sin t,  y_b = z_b cos t + z_a sin t
//   g = dy turned back, dw = sum g xh, h = g w, dx = rstd (h - xh mean(h xh))
//
// A group of lanes owns a row's pairs, a lane V of them: its elements are two
// vectors of V (a's and b's, or adjacent pairs), so a pair never leaves the
// lane, and the sines and cosines are formed once for all heads of the row
// that the lane walks.
#include <algorithm>

#include "state.h"

namespace sn {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPartials = 1024;   // blocks of a backward pass, and with them partial weight gradients
// Lanes that a pass keeps busy before a lane takes two heads or more: 17216 rows
// of 4 + 4 heads of 32, fp32, a step: 26.6 us with 65536, 28.5 with twice as
// many, 30.4 with four times; 4096 rows of 32 + 8 heads of 128, bf16: 21.0, 20.0
// and 25.0; with half as many 25.7 there.
constexpr int64_t kFill = 65536;
// Outputs beyond this stay in no cache until they are read: they are stored past
// it (32768 rows of 32 + 8 heads of 128, bf16: 159 us -> 144; 17216 rows of
// 4 + 4 heads of 32, fp32, 18 MB: 9.3 -> 8.3; bf16, 9 MB: 9.4 -> 10.3).
constexpr int64_t kStream = 16 << 20;

// How rows and heads are cut (host).
struct RotaryCut {
    int units;      // lanes of a group that have pairs
    int lanes;      // lanes of a group, a power of two
    int lane_bits;
    // of q and of k, each with blocks of its own (grid y)
    int slices[2];  // groups that share a row, each with a run of its heads
    int heads[2];   // heads of a slice
    int blocks[2];
    float inv_D;
    bool stream;    // stores go past the caches
};

template <typename T, int V>
struct VecOf { typedef T type __attribute__((ext_vector_type(V))); };

// A lane's two runs of elements.
struct Place {
    int a, b;       // first elements
    int pair;       // the first pair
    bool turned, has_a, has_b;
};
template <int V, bool IL>
__device__ inline Place place_of(int u, int units, int D, int P) {
    Place p;
    p.pair = u * V;
    p.turned = p.pair < P;      // of adjacent pairs the first: each is asked for on its own
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

// The pairs' frequencies and axes in LDS: lanes that index the arguments one by
// one would wait for them again and again.
struct Pairs {
    double turns[kMaxPairs];
    int axes[kMaxPairs];
    __device__ inline void load(const RotaryArgs &a) {
        if ((int)threadIdx.x < a.P) {
            turns[threadIdx.x] = a.turns[threadIdx.x];
            axes[threadIdx.x] = a.axes[threadIdx.x];
        }
        __syncthreads();
    }
};

// Angles in full turns are reduced in fp64; what is left is at most half a turn.
template <int V>
__device__ inline void angles(const RotaryArgs &a, const Pairs &pairs, int row, const Place &p, float (&c)[V], float (&s)[V]) {
    int at[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const int j = p.pair + e;
        at[e] = j < a.P ? a.positions[(int64_t)pairs.axes[j] * a.n_rows + row] : 0;
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const int j = p.pair + e;
        const double turn = j < a.P ? (double)at[e] * pairs.turns[j] : 0.0;
        sincospif(2.0f * (float)(turn - rint(turn)), &s[e], &c[e]);
    }
}

template <int V, bool IL>
__device__ inline void turn(float (&x)[2 * V], const float (&c)[V], const float (&s)[V], float sign) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
        float &a = x[IL ? 2 * e : e], &b = x[IL ? 2 * e + 1 : V + e];
        const float ta = a * c[e] - sign * b * s[e], tb = b * c[e] + sign * a * s[e];
        a = ta;
        b = tb;
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

// A group's row and run of heads.
struct Part {
    int row, h0, h1;
    bool live;
};
__device__ inline Part part_of(const RotaryArgs &a, const RotaryCut &k, int n, uint32_t group) {
    Part r;
    const uint32_t row = group / (uint32_t)k.slices[n];
    r.live = row < (uint32_t)a.n_rows;
    r.row = r.live ? (int)row : 0;
    r.h0 = (int)(group - row * k.slices[n]) * k.heads[n];
    r.h1 = r.live ? min(r.h0 + k.heads[n], n ? a.Hkv : a.H) : r.h0;
    return r;
}

// N heads are on their way at once.
template <typename T, int V, bool IL, bool NORM, int N>
__global__ __launch_bounds__(kThreads) void rotary_forward_kernel(RotaryArgs a, RotaryCut k) {
    __shared__ Pairs pairs;
    const int n = blockIdx.y;
    if ((int)blockIdx.x >= k.blocks[n]) return;
    pairs.load(a);
    const RotaryTensor &t = a.t[n];
    const Part part = part_of(a, k, n, (blockIdx.x * (uint32_t)kThreads + threadIdx.x) >> k.lane_bits);
    Place p = place_of<V, IL>(threadIdx.x & (k.lanes - 1), k.units, a.D, a.P);
    p.has_a &= part.live;
    p.has_b &= part.live;
    const T *x = static_cast<const T *>(t.x) + part.row * t.xs;
    T *y = static_cast<T *>(t.out) + (int64_t)part.row * (n ? a.Hkv : a.H) * a.D;
    float c[V], s[V], w[2 * V];
    for (int hb = part.h0; hb < part.h1; hb += N) {
        Run<T, V> ra[N], rb[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const T *from = x + (hb + i) * t.xh;
            ra[i].load(from + p.a, p.has_a && hb + i < part.h1);
            rb[i].load(from + p.b, p.has_b && hb + i < part.h1);
        }
        if (hb == part.h0) {        // the first heads are on their way meanwhile
            if (NORM) load_weights<V>(t.w, p, w);
            angles<V>(a, pairs, part.row, p, c, s);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float v[2 * V];
            ra[i].get(v);
            rb[i].get(v + V);
            if (NORM) {
                float sq = 0.0f;
#pragma unroll
                for (int e = 0; e < 2 * V; ++e) sq += v[e] * v[e];
                const float r = __builtin_amdgcn_rsqf(group_sum(sq, k.lanes) * k.inv_D + a.eps);
#pragma unroll
                for (int e = 0; e < 2 * V; ++e) v[e] *= r * w[e];
            }
            turn<V, IL>(v, c, s, 1.0f);
            T *to = y + (int64_t)(hb + i) * a.D;
            store_run<T, V>(to + p.a, p.has_a && hb + i < part.h1, v, k.stream);
            store_run<T, V>(to + p.b, p.has_b && hb + i < part.h1, v + V, k.stream);
        }
    }
}

// Rows in turn by groups; a block leaves the weight gradients of its rows in
// partials[q, k][block][D].
template <typename T, int V, bool IL, bool NORM, int N>
__global__ __launch_bounds__(kThreads) void rotary_backward_kernel(RotaryArgs a, RotaryCut k, float *partials) {
    __shared__ Pairs pairs;
    __shared__ float sums[kThreads * 2 * V];
    const int n = blockIdx.y;
    if ((int)blockIdx.x >= k.blocks[n]) return;
    pairs.load(a);
    const RotaryTensor &t = a.t[n];
    const int groups = kThreads >> k.lane_bits;
    const Place p0 = place_of<V, IL>(threadIdx.x & (k.lanes - 1), k.units, a.D, a.P);
    float dw[2 * V] = {}, w[2 * V];
    if (NORM) load_weights<V>(t.w, p0, w);
    const uint32_t all = (uint32_t)a.n_rows * k.slices[n];
    for (uint32_t g0 = blockIdx.x * groups; g0 < all; g0 += k.blocks[n] * groups) {
        const Part part = part_of(a, k, n, g0 + (threadIdx.x >> k.lane_bits));
        Place p = p0;
        p.has_a &= part.live;
        p.has_b &= part.live;
        const T *x = static_cast<const T *>(t.x) + part.row * t.xs, *dy = static_cast<const T *>(t.dy) + part.row * t.gs;
        T *dx = static_cast<T *>(t.out) + (int64_t)part.row * (n ? a.Hkv : a.H) * a.D;
        float c[V], s[V];
        for (int hb = part.h0; hb < part.h1; hb += N) {
            Run<T, V> xa[N], xb[N], ga[N], gb[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const bool has = hb + i < part.h1;
                const T *from = dy + (hb + i) * t.gh;
                ga[i].load(from + p.a, p.has_a && has);
                gb[i].load(from + p.b, p.has_b && has);
                if (NORM) {
                    const T *rows = x + (hb + i) * t.xh;
                    xa[i].load(rows + p.a, p.has_a && has);
                    xb[i].load(rows + p.b, p.has_b && has);
                }
            }
            if (hb == part.h0) angles<V>(a, pairs, part.row, p, c, s);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float g[2 * V];
                ga[i].get(g);
                gb[i].get(g + V);
                turn<V, IL>(g, c, s, -1.0f);
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
                    const float r = __builtin_amdgcn_rsqf(group_sum(sq, k.lanes) * k.inv_D + a.eps);
                    const float m = group_sum(dot, k.lanes) * k.inv_D * r * r;
#pragma unroll
                    for (int e = 0; e < 2 * V; ++e) {
                        dw[e] += g[e] * (v[e] * r);
                        g[e] = r * (g[e] * w[e] - v[e] * m);
                    }
                }
                T *to = dx + (int64_t)(hb + i) * a.D;
                store_run<T, V>(to + p.a, p.has_a && hb + i < part.h1, g, k.stream);
                store_run<T, V>(to + p.b, p.has_b && hb + i < part.h1, g + V, k.stream);
            }
        }
    }
    if (!NORM || !partials) return;
#pragma unroll
    for (int e = 0; e < 2 * V; ++e) sums[e * kThreads + threadIdx.x] = dw[e];
    __syncthreads();
    float *out = partials + ((int64_t)n * kMaxPartials + blockIdx.x) * a.D;
    // element e of lane u, of all groups
    for (int i = threadIdx.x; i < k.units * 2 * V; i += kThreads) {
        const int lane = i % k.units, e = i / k.units;
        float sum = 0.0f;
        for (int g = 0; g < groups; ++g) sum += sums[e * kThreads + g * k.lanes + lane];
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
    double sum = 0.0;
    for (int b = threadIdx.x; b < k.blocks[n]; b += kThreads) sum += partials[((int64_t)n * kMaxPartials + b) * D + d];
    sums[threadIdx.x] = sum;
    for (int o = kThreads / 2; o > 0; o >>= 1) {
        __syncthreads();
        if (threadIdx.x < o) sums[threadIdx.x] += sums[threadIdx.x + o];
    }
    if (threadIdx.x == 0 && out) out[d] = (float)sums[0];
}

// A lane's vector length: as long as every run of V elements lies whole in
// one aligned place of every tensor, else 1.
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
    k.lanes = 1;
    while (k.lanes < k.units) k.lanes *= 2;
    k.lane_bits = __builtin_ctz(k.lanes);
    k.inv_D = 1.0f / (float)a.D;
    k.stream = (int64_t)a.n_rows * (a.H + a.Hkv) * a.D * size > kStream;
    const int64_t per = kThreads / k.lanes;
    for (int n = 0; n < 2; ++n) {
        const int heads = n ? a.Hkv : a.H;
        int run = std::max(heads, 1);
        // a head a group while that leaves SIMDs without a wavefront or two
        while (run > 1 && (int64_t)a.n_rows * ((heads + run - 1) / run) * k.lanes < kFill) run = (run + 1) / 2;
        k.heads[n] = run;
        k.slices[n] = std::max(1, (heads + run - 1) / run);
        const int64_t blocks = heads ? ((int64_t)a.n_rows * k.slices[n] + per - 1) / per : 0;
        k.blocks[n] = (int)(backward ? std::min<int64_t>(blocks, kMaxPartials) : blocks);
    }
    return k;
}

template <typename T, int V, bool IL, bool NORM>
sn_status launch(const RotaryArgs &a, float *partials, bool backward, float *dqw, float *dkw, hipStream_t s) {
    const RotaryCut k = cut_of(a, V, (int)sizeof(T), backward);
    ProfScope prof(backward ? K_ROTARY_BWD : K_ROTARY_FWD, s);
    const dim3 grid(std::max(k.blocks[0], k.blocks[1]), a.Hkv ? 2 : 1);
    const bool many = std::max(k.heads[0], k.heads[1]) > 1;
    if (grid.x > 0) {       // no rows: the weights' zeros alone
        if (!backward) {
            if (many)
                rotary_forward_kernel<T, V, IL, NORM, 4><<<grid, kThreads, 0, s>>>(a, k);
            else
                rotary_forward_kernel<T, V, IL, NORM, 1><<<grid, kThreads, 0, s>>>(a, k);
            return launch_status();
        }
        if (many)
            rotary_backward_kernel<T, V, IL, NORM, 2><<<grid, kThreads, 0, s>>>(a, k, partials);
        else
            rotary_backward_kernel<T, V, IL, NORM, 1><<<grid, kThreads, 0, s>>>(a, k, partials);
        SN_TRY(launch_status());
    }
    if (NORM && (dqw || dkw)) rotary_weights_kernel<<<dim3(a.D, 2), kThreads, 0, s>>>(partials, k, a.D, dqw, dkw);
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

// A forward pass has at most a group of 64 lanes for every head of every row.
bool rotary_fits(const sn_head_rotary &op) {
    return grid_fits((int64_t)op.n_rows * (op.n_heads + op.n_kv_heads) + 4, 64);
}

sn_status rotary_forward(const RotaryArgs &a, int dtype, bool norm, hipStream_t s) {
    return launch(a, dtype, norm, nullptr, false, nullptr, nullptr, s);
}

sn_status rotary_backward(const RotaryArgs &a, int dtype, bool norm, float *dq_weight, float *dk_weight, char *ws,
                          hipStream_t s) {
    return launch(a, dtype, norm, reinterpret_cast<float *>(ws + kWsBase), true, dq_weight, dk_weight, s);
}

}  // namespace sn
