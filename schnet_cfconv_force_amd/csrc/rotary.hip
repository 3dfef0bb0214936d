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

// How rows and heads are cut (host).
struct RotaryCut {
    int units;      // lanes of a group that have pairs
    int lanes;      // lanes of a group, a power of two
    int slices;     // groups that share a row, each with a run of its heads
    int heads;      // heads of a slice
    int blocks;
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

template <typename T, int V>
__device__ inline void load_run(const T *p, bool has, float *x) {
    if constexpr (V == 1) {
        x[0] = has ? to_f32(p[0]) : 0.0f;
    } else {
        typename VecOf<T, V>::type v;
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = (T)0.0f;
        if (has) v = *reinterpret_cast<const typename VecOf<T, V>::type *>(p);
#pragma unroll
        for (int e = 0; e < V; ++e) x[e] = to_f32(v[e]);
    }
}
template <typename T, int V>
__device__ inline void store_run(T *p, bool has, const float *x) {
    if (!has) return;
    if constexpr (V == 1) {
        p[0] = (T)x[0];
    } else {
        typename VecOf<T, V>::type v;
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = (T)x[e];
        *reinterpret_cast<typename VecOf<T, V>::type *>(p) = v;
    }
}

__device__ inline float group_sum(float v, int lanes) {
    for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// Angles in full turns are reduced in fp64; what is left is at most half a turn.
template <int V, bool IL>
__device__ inline void angles(const RotaryArgs &a, int row, const Place &p, float (&c)[V], float (&s)[V]) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
        c[e] = 1.0f;
        s[e] = 0.0f;
        const int j = p.pair + e;
        if (j < a.P) {
            const double turn = (double)a.positions[(int64_t)a.axes[j] * a.n_rows + row] * a.turns[j];
            sincospif(2.0f * (float)(turn - rint(turn)), &s[e], &c[e]);
        }
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

template <typename T, int V, bool IL, bool NORM>
__global__ __launch_bounds__(kThreads) void rotary_forward_kernel(RotaryArgs a, RotaryCut k) {
    const int64_t group = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / k.lanes;
    const int u = threadIdx.x % k.lanes;
    const int64_t row64 = group / k.slices;
    const bool live = row64 < a.n_rows;
    const int row = live ? (int)row64 : 0, slice = (int)(group % k.slices);
    Place p = place_of<V, IL>(u, k.units, a.D, a.P);
    p.has_a &= live;
    p.has_b &= live;
    float c[V], s[V];
    angles<V, IL>(a, row, p, c, s);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const RotaryTensor &t = a.t[n];
        const int first = n ? a.H : 0, heads = n ? a.Hkv : a.H;
        const int h0 = max(slice * k.heads - first, 0), h1 = min((slice + 1) * k.heads - first, heads);
        if (h0 >= h1) continue;
        float w[2 * V];
        if (NORM) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                w[e] = t.w && p.has_a ? t.w[p.a + e] : 1.0f;
                w[V + e] = t.w && p.has_b ? t.w[p.b + e] : 1.0f;
            }
        }
        const T *x = static_cast<const T *>(t.x) + row * t.xs;
        T *y = static_cast<T *>(t.out) + (int64_t)row * heads * a.D;
        for (int h = h0; h < h1; ++h) {
            float v[2 * V];
            load_run<T, V>(x + h * t.xh + p.a, p.has_a, v);
            load_run<T, V>(x + h * t.xh + p.b, p.has_b, v + V);
            if (NORM) {
                float sq = 0.0f;
#pragma unroll
                for (int e = 0; e < 2 * V; ++e) sq += v[e] * v[e];
                const float r = 1.0f / sqrtf(group_sum(sq, k.lanes) / (float)a.D + a.eps);
#pragma unroll
                for (int e = 0; e < 2 * V; ++e) v[e] *= r * w[e];
            }
            turn<V, IL>(v, c, s, 1.0f);
            store_run<T, V>(y + (int64_t)h * a.D + p.a, p.has_a, v);
            store_run<T, V>(y + (int64_t)h * a.D + p.b, p.has_b, v + V);
        }
    }
}

// Rows in turn by groups; a block leaves the weight gradients of its rows in
// partials[block][q, k][D].
template <typename T, int V, bool IL, bool NORM>
__global__ __launch_bounds__(kThreads) void rotary_backward_kernel(RotaryArgs a, RotaryCut k, float *partials) {
    __shared__ float sums[kThreads * 2 * V];
    const int u = threadIdx.x % k.lanes, groups = kThreads / k.lanes;
    const Place p0 = place_of<V, IL>(u, k.units, a.D, a.P);
    float dw[2][2 * V] = {};
    const int64_t all = (int64_t)a.n_rows * k.slices;
    for (int64_t g0 = (int64_t)blockIdx.x * groups; g0 < all; g0 += (int64_t)gridDim.x * groups) {
        const int64_t group = g0 + threadIdx.x / k.lanes;
        const bool live = group < all;
        const int row = live ? (int)(group / k.slices) : 0, slice = live ? (int)(group % k.slices) : 0;
        Place p = p0;
        p.has_a &= live;
        p.has_b &= live;
        float c[V], s[V];
        angles<V, IL>(a, row, p, c, s);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const RotaryTensor &t = a.t[n];
            const int first = n ? a.H : 0, heads = n ? a.Hkv : a.H;
            const int h0 = max(slice * k.heads - first, 0), h1 = min((slice + 1) * k.heads - first, heads);
            if (h0 >= h1) continue;
            float w[2 * V];
            if (NORM) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    w[e] = t.w && p.has_a ? t.w[p.a + e] : 1.0f;
                    w[V + e] = t.w && p.has_b ? t.w[p.b + e] : 1.0f;
                }
            }
            const T *x = static_cast<const T *>(t.x) + row * t.xs, *dy = static_cast<const T *>(t.dy) + row * t.gs;
            T *dx = static_cast<T *>(t.out) + (int64_t)row * heads * a.D;
            for (int h = h0; h < h1; ++h) {
                float g[2 * V];
                load_run<T, V>(dy + h * t.gh + p.a, p.has_a, g);
                load_run<T, V>(dy + h * t.gh + p.b, p.has_b, g + V);
                turn<V, IL>(g, c, s, -1.0f);
                if (NORM) {
                    float v[2 * V];
                    load_run<T, V>(x + h * t.xh + p.a, p.has_a, v);
                    load_run<T, V>(x + h * t.xh + p.b, p.has_b, v + V);
                    float sq = 0.0f, dot = 0.0f;
#pragma unroll
                    for (int e = 0; e < 2 * V; ++e) {
                        sq += v[e] * v[e];
                        dot += g[e] * w[e] * v[e];
                    }
                    const float r = 1.0f / sqrtf(group_sum(sq, k.lanes) / (float)a.D + a.eps);
                    const float m = group_sum(dot, k.lanes) / (float)a.D * r * r;
#pragma unroll
                    for (int e = 0; e < 2 * V; ++e) {
                        if (p.has_a) dw[n][e] += g[e] * (v[e] * r);
                        g[e] = r * (g[e] * w[e] - v[e] * m);
                    }
                }
                store_run<T, V>(dx + (int64_t)h * a.D + p.a, p.has_a, g);
                store_run<T, V>(dx + (int64_t)h * a.D + p.b, p.has_b, g + V);
            }
        }
    }
    if (!NORM || !partials) return;
    for (int n = 0; n < 2; ++n) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 2 * V; ++e) sums[e * kThreads + threadIdx.x] = dw[n][e];
        __syncthreads();
        float *out = partials + ((int64_t)blockIdx.x * 2 + n) * a.D;
        // lane u of the first groups joins element e of all groups
        for (int i = threadIdx.x; i < k.units * 2 * V; i += kThreads) {
            const int lane = i % k.units, e = i / k.units;
            float sum = 0.0f;
            for (int g = 0; g < groups; ++g) sum += sums[e * kThreads + g * k.lanes + lane];
            const Place p = place_of<V, IL>(lane, k.units, a.D, a.P);
            const int d = e < V ? p.a + e : p.b + e - V;
            if (d < a.D) out[d] = sum;
        }
    }
}

// dw[n][d] = the sum of the blocks' partials, in one order, in fp64.
__global__ __launch_bounds__(kThreads) void rotary_weights_kernel(const float *partials, int blocks, int D, float *dq_weight,
                                                                  float *dk_weight) {
    __shared__ double sums[kThreads];
    float *out = blockIdx.y ? dk_weight : dq_weight;
    const int d = blockIdx.x;
    double sum = 0.0;
    for (int b = threadIdx.x; b < blocks; b += kThreads) sum += partials[((int64_t)b * 2 + blockIdx.y) * D + d];
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

RotaryCut cut_of(const RotaryArgs &a, int V, bool backward) {
    RotaryCut k;
    k.units = (a.D + 2 * V - 1) / (2 * V);
    k.lanes = 1;
    while (k.lanes < k.units) k.lanes *= 2;
    const int heads = a.H + a.Hkv;
    k.heads = heads;
    // every head a group of its own while that leaves CUs without a wavefront
    while (k.heads > 1 && (int64_t)a.n_rows * ((heads + k.heads - 1) / k.heads) * k.lanes < 256 * 8 * 64) k.heads = (k.heads + 1) / 2;
    k.slices = (heads + k.heads - 1) / k.heads;
    const int64_t groups = (int64_t)a.n_rows * k.slices, per = kThreads / k.lanes;
    const int64_t blocks = (groups + per - 1) / per;
    k.blocks = (int)(backward ? std::min<int64_t>(blocks, kMaxPartials) : blocks);
    return k;
}

template <typename T, int V, bool IL, bool NORM>
sn_status launch(const RotaryArgs &a, float *partials, bool backward, float *dqw, float *dkw, hipStream_t s) {
    const RotaryCut k = cut_of(a, V, backward);
    ProfScope prof(backward ? K_ROTARY_BWD : K_ROTARY_FWD, s);
    if (!backward) {
        rotary_forward_kernel<T, V, IL, NORM><<<k.blocks, kThreads, 0, s>>>(a, k);
        return launch_status();
    }
    if (k.blocks > 0) rotary_backward_kernel<T, V, IL, NORM><<<k.blocks, kThreads, 0, s>>>(a, k, partials);   // no rows: the weights' zeros alone
    SN_TRY(launch_status());
    if (NORM && (dqw || dkw)) rotary_weights_kernel<<<dim3(a.D, 2), kThreads, 0, s>>>(partials, k.blocks, a.D, dqw, dkw);
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
