// Group norm with an activation over the rows of each segment, channels
// last, forward and backward.
//
//   xh = (x - mean) rstd, z = gamma xh + beta, y = act(z)
//   dz = dy act'(z), dbeta = sum dz, dgamma = sum dz xh,
//   dx = rstd (dz gamma - mean(dz gamma) - xh mean(dz gamma xh))
//
// A block owns a slab: some rows of a segment times a run of channels (whole
// groups, or a piece of one that is wider than the block).  A thread owns one
// vector of channels of the slab and every RP-th row, so per-channel
// quantities are registers.  Where the longest segment's slab fits a block's
// registers, one launch does everything and x (and dy) is read once.  Longer
// segments are cut into chunks of rows: one launch leaves each chunk's
// statistics, the next joins them and reads the rows again.
//
// The mean is subtracted before squaring (in the chunk by its own mean, in
// the join by n_c (mean_c - mean)^2), so a large common offset costs no
// digits of the variance.  All sums are fp32 in a block and fp64 in a join,
// each in one order.
#include <algorithm>
#include <type_traits>

#include "context.h"

namespace sn {
namespace {

constexpr int kThreads = 512;
constexpr int kMaxGroups = kThreads / 32;   // groups of a slab: 32 lanes join each

template <int ACT>
__device__ inline float act_fwd(float z) {
    if constexpr (ACT == SN_ACT_SSP) return ssp(z);
    if constexpr (ACT == SN_ACT_SILU) return z * sigm(z);
    return z;
}
template <int ACT>
__device__ inline float act_grad(float z) {
    if constexpr (ACT == SN_ACT_SSP) return sigm(z);
    if constexpr (ACT == SN_ACT_SILU) {
        const float s = sigm(z);
        return s * (1.0f + z * (1.0f - s));
    }
    return 1.0f;
}

// V consecutive elements of a row, as they lie in memory.
template <typename T, int V>
struct Vec {
    typedef T type __attribute__((ext_vector_type(V)));
    type v;
};
template <typename T>
struct Vec<T, 1> {
    struct type {
        T x;
        __device__ inline T &operator[](int) { return x; }
        __device__ inline T operator[](int) const { return x; }
    };
    type v;
};
template <typename T, int V>
__device__ inline Vec<T, V> load_vec(const T *p) {
    Vec<T, V> r;
    r.v = *reinterpret_cast<const typename Vec<T, V>::type *>(p);
    return r;
}
template <typename T, int V>
__device__ inline void store_vec(T *p, const float (&x)[V]) {
    typename Vec<T, V>::type t;
#pragma unroll
    for (int j = 0; j < V; ++j) t[j] = (T)x[j];
    *reinterpret_cast<typename Vec<T, V>::type *>(p) = t;
}

// How rows and channels are cut (host).
struct NormCut {
    int V;          // channels of a vector
    int gs;         // groups of a slab (1 where a slab is a piece of a group)
    int piece;      // channels of a piece; 0: slabs hold whole groups
    int slabs;      // slabs of a row
    int chunks;     // chunks of the longest segment
    int chunk_rows;
    int it;         // vectors that a thread holds of a chunk
    bool fused;     // one launch: a thread holds all its vectors of a segment
};

// A block's slab.
struct Slab {
    int b, slab, chunk;
    int r0, n;          // the segment's rows
    int first, rows;    // the chunk's rows, relative to r0
    int c0, cs;         // first channel, channels
    int g0, gs;         // first group, groups
    int piece, pieces;  // piece of the group
    int cv, rp;         // vectors of a slab row, rows per pass
    int col, row;       // this thread's vector (-1: none) and first row
    int group;          // its group within the slab
    int wv;             // vectors of one of the slab's groups
};

__device__ inline bool locate(const NormArgs &a, const NormCut &k, int block, Slab &s) {
    // a segment's rows in order, all their slabs before the next rows: what lies
    // beyond a short segment is spread over the dies (8 segments of up to 16384
    // rows of 512 in bf16: forward 74 -> 67 us against slab by slab)
    s.slab = block % k.slabs;
    s.chunk = block / k.slabs % k.chunks;
    s.b = block / k.chunks / k.slabs;
    segment_rows(a.ptr, s.b, a.B, a.n_rows, a.max_rows, a.status, s.r0, s.n);
    s.first = s.chunk * k.chunk_rows;
    s.rows = min(k.chunk_rows, s.n - s.first);
    if (k.piece) {
        s.pieces = k.slabs / a.groups;
        s.piece = s.slab % s.pieces;
        s.g0 = s.slab / s.pieces;
        s.gs = 1;
        s.c0 = s.g0 * a.width + s.piece * k.piece;
        s.cs = min(k.piece, a.width - s.piece * k.piece);
    } else {
        s.pieces = 1;
        s.piece = 0;
        s.g0 = s.slab * k.gs;
        s.gs = min(k.gs, a.groups - s.g0);
        s.c0 = s.g0 * a.width;
        s.cs = s.gs * a.width;
    }
    s.cv = s.cs / k.V;
    s.rp = kThreads / s.cv;
    s.wv = s.cv / s.gs;
    const int t = threadIdx.x;
    s.row = t / s.cv;
    s.col = s.row < s.rp ? t % s.cv : -1;
    s.group = s.col < 0 ? 0 : s.col / s.wv;
    return s.rows > 0;
}

template <typename F>
__device__ inline F half_wave_sum(F v) {
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor(v, o, 32);
    return v;
}

// Sum of v over the threads of each group, returned to all of them.  Where
// the vectors of a row and of a group are powers of two, a group's lanes
// differ from the others' in whole bits of the lane index: those of a
// wavefront add by exchanges, the wavefronts through buf [wavefront][group]
// (zeroed before).  Otherwise 32 lanes add a group's threads in strides.
constexpr int kWaves = kThreads / 64;
struct SumLds {
    float wave[2][kWaves][kMaxGroups], all[kThreads], out[kMaxGroups];
};
__device__ inline void clear_sums(SumLds &l) {
    if (threadIdx.x < 2 * kWaves * kMaxGroups) (&l.wave[0][0][0])[threadIdx.x] = 0.0f;
    __syncthreads();
}
__device__ inline bool in_bits(const Slab &s) { return (s.cv & (s.cv - 1)) == 0 && (s.wv & (s.wv - 1)) == 0; }
__device__ inline float group_sum(const Slab &s, float v, SumLds &l, int turn) {
    if (in_bits(s)) {
        int mine = 0;   // lane bits that are summed over
#pragma unroll
        for (int o = 1; o < 64; o <<= 1)
            if (o < s.wv || o >= s.cv) {
                v += __shfl_xor(v, o, 64);
                mine |= o;
            }
        if ((threadIdx.x & 63 & mine) == 0 && s.col >= 0) l.wave[turn][threadIdx.x >> 6][s.group] = v;
        __syncthreads();
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) sum += l.wave[turn][w][s.group];
        return sum;
    }
    __syncthreads();
    l.all[threadIdx.x] = v;
    __syncthreads();
    const int g = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float sum = 0.0f;
    if (g < s.gs)
        for (int i = lane; i < s.rp * s.wv; i += 32) sum += l.all[i / s.wv * s.cv + g * s.wv + i % s.wv];
    sum = half_wave_sum(sum);
    if (g < s.gs && lane == 0) l.out[g] = sum;
    __syncthreads();
    return l.out[s.group];
}

template <int V>
__device__ inline void load_affine(const NormArgs &a, const Slab &s, float (&ga)[V], float (&be)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
        ga[j] = 1.0f;
        be[j] = 0.0f;
        if (s.col >= 0) {
            const int c = s.c0 + s.col * V + j;
            if (a.gamma) ga[j] = a.gamma[c];
            if (a.beta) be[j] = a.beta[c];
        }
    }
}

// The chunk's mean and sum of squared differences from it, of the thread's
// group, from the vectors held in registers.
template <typename T, int V, int IT>
__device__ inline float2 chunk_stats(const Slab &s, const Vec<T, V> (&x)[IT], SumLds &lds) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < IT; ++i)
        if (s.col >= 0 && s.row + i * s.rp < s.rows)
#pragma unroll
            for (int j = 0; j < V; ++j) sum += to_f32(x[i].v[j]);
    const float mu = group_sum(s, sum, lds, 0) / ((float)s.rows * (s.wv * V));
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < IT; ++i)
        if (s.col >= 0 && s.row + i * s.rp < s.rows)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = to_f32(x[i].v[j]) - mu;
                sum = fmaf(d, d, sum);
            }
    return make_float2(mu, group_sum(s, sum, lds, 1));
}

template <typename T, int V, int IT>
__device__ inline void load_rows(const NormCut &k, const Slab &s, const T *base, int64_t stride, Vec<T, V> (&x)[IT]) {
    const T *p = base + (int64_t)(s.r0 + s.first) * stride + s.c0 + s.col * V;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
#pragma unroll
        for (int j = 0; j < V; ++j) x[i].v[j] = (T)0.0f;
        const int r = s.row + i * s.rp;
        if (s.col >= 0 && r < s.rows) x[i] = load_vec<T, V>(p + r * stride);
    }
}

template <typename T, int V, int ACT>
__device__ inline void write_y(const Vec<T, V> &x, float mu, float r, const float (&ga)[V],
                               const float (&be)[V], T *p) {
    float y[V];
#pragma unroll
    for (int j = 0; j < V; ++j) y[j] = act_fwd<ACT>(fmaf((to_f32(x.v[j]) - mu) * r, ga[j], be[j]));
    store_vec<T, V>(p, y);
}

// ------------------------------------------------------------------ forward

// The whole segment in registers: statistics and output in one pass, x read
// once.  269 rows of 128 in fp32: 6.4 us, a launch and two sums over a block;
// 64 segments of up to as many: 7 us for 8.4 MB, one wave of 256 blocks whose
// loads, sums and stores follow each other.
template <typename T, int V, int IT, int ACT>
__global__ __launch_bounds__(kThreads) void norm_fwd_kernel(NormArgs a, NormCut k, T *y, float *mean, float *rstd) {
    __shared__ SumLds lds;
    Slab s;
    const bool any = locate(a, k, blockIdx.x, s);
    if (!any) {   // an empty segment
        if (threadIdx.x < s.gs) {
            if (mean) mean[s.b * a.groups + s.g0 + threadIdx.x] = 0.0f;
            if (rstd) rstd[s.b * a.groups + s.g0 + threadIdx.x] = 1.0f / sqrtf(a.eps);
        }
        return;
    }
    Vec<T, V> x[IT];
    load_rows<T, V, IT>(k, s, (const T *)a.x, a.xs, x);
    float ga[V], be[V];
    load_affine<V>(a, s, ga, be);
    clear_sums(lds);
    const float2 st = chunk_stats<T, V, IT>(s, x, lds);
    if (s.col < 0) return;
    const float m = st.x, r = 1.0f / sqrtf(st.y / ((float)s.rows * a.width) + a.eps);
    if (s.row == 0 && s.col % s.wv == 0) {
        const int at = s.b * a.groups + s.g0 + s.group;
        if (mean) mean[at] = m;
        if (rstd) rstd[at] = r;
    }
    T *p = y + (int64_t)s.r0 * a.C + s.c0 + s.col * V;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int row = s.row + i * s.rp;
        if (row < s.rows) write_y<T, V, ACT>(x[i], m, r, ga, be, p + (int64_t)row * a.C);
    }
}

// Memory bound: 8 segments of 16384 rows of 512 in bf16, 134 MB, take 77 us with
// the launch that follows, 5.2 TB/s; of ragged ones (101 MB a tensor) the blocks
// are one wave on the card, whose start and end cost a sixth: 24 us, 4.2 TB/s.
// part [b][group][chunk pieces + piece]: the chunk's {mean, sum of squared
// differences} of each group
template <typename T, int V, int IT>
__global__ __launch_bounds__(kThreads) void norm_stats_kernel(NormArgs a, NormCut k, float2 *part) {
    __shared__ SumLds lds;
    Slab s;
    if (!locate(a, k, blockIdx.x, s)) return;
    Vec<T, V> x[IT];
    load_rows<T, V, IT>(k, s, (const T *)a.x, a.xs, x);
    clear_sums(lds);
    const float2 st = chunk_stats<T, V, IT>(s, x, lds);
    if (s.row == 0 && s.col >= 0 && s.col % s.wv == 0)
        part[((int64_t)s.b * a.groups + s.g0 + s.group) * k.chunks * s.pieces + s.chunk * s.pieces + s.piece] = st;
}

// Joins the chunks' statistics (each block for itself: a launch less) and
// writes this chunk's rows; the same ragged segments in 42 us, 4.8 TB/s.
template <typename T, int V, int ACT>
__global__ __launch_bounds__(kThreads) void norm_apply_kernel(NormArgs a, NormCut k, const float2 *part, T *y,
                                                              float *mean, float *rstd) {
    __shared__ float mu[kMaxGroups], rs[kMaxGroups];
    Slab s;
    const bool any = locate(a, k, gridDim.x - 1 - blockIdx.x, s);   // the rows read last are the likeliest in a cache
    if (!any && s.chunk > 0) return;
    float ga[V], be[V];
    load_affine<V>(a, s, ga, be);
    const int g = threadIdx.x >> 5, l = threadIdx.x & 31;
    if (g < s.gs) {
        // every chunk but the last has the same rows, every piece but the last the same channels
        const int chunks = (s.n + k.chunk_rows - 1) / k.chunk_rows, n = chunks * s.pieces;
        const int last_rows = s.n - (chunks - 1) * k.chunk_rows;
        const int width = k.piece ? k.piece : a.width, last_width = a.width - (s.pieces - 1) * width;
        auto count = [&](int i) {
            const int c = s.pieces == 1 ? i : i / s.pieces, p = s.pieces == 1 ? 0 : i % s.pieces;
            return (double)(c == chunks - 1 ? last_rows : k.chunk_rows) * (p == s.pieces - 1 ? last_width : width);
        };
        const float2 *p = part + ((int64_t)s.b * a.groups + s.g0 + g) * k.chunks * s.pieces;
        const double cnt = (double)s.n * a.width;
        double sum = 0.0;
#pragma unroll 8
        for (int i = l; i < n; i += 32) sum += count(i) * p[i].x;
        const double m = s.n ? half_wave_sum(sum) / cnt : 0.0;
        sum = 0.0;
#pragma unroll 8
        for (int i = l; i < n; i += 32) {
            const double d = p[i].x - m;
            sum += p[i].y + count(i) * d * d;
        }
        const double var = s.n ? half_wave_sum(sum) / cnt : 0.0;
        if (l == 0) {
            mu[g] = (float)m;
            rs[g] = 1.0f / sqrtf((float)var + a.eps);
            if (s.chunk == 0 && s.piece == 0) {
                if (mean) mean[s.b * a.groups + s.g0 + g] = mu[g];
                if (rstd) rstd[s.b * a.groups + s.g0 + g] = rs[g];
            }
        }
    }
    __syncthreads();
    if (s.col < 0 || !any) return;
    const float m = mu[s.group], r = rs[s.group];
    const int64_t base = s.r0 + s.first;
    const T *px = (const T *)a.x + base * a.xs + s.c0 + s.col * V;
    T *py = y + base * a.C + s.c0 + s.col * V;
#pragma unroll 4
    for (int row = s.row; row < s.rows; row += s.rp)
        write_y<T, V, ACT>(load_vec<T, V>(px + row * a.xs), m, r, ga, be, py + (int64_t)row * a.C);
}

// ------------------------------------------------------------------ backward

// dz and xh of one vector.
template <typename T, int V, int ACT>
__device__ inline void dz_xh(const Vec<T, V> &x, const Vec<T, V> &dy, float mu, float r,
                             const float (&ga)[V], const float (&be)[V], float (&dz)[V], float (&xh)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
        xh[j] = (to_f32(x.v[j]) - mu) * r;
        dz[j] = to_f32(dy.v[j]) * act_grad<ACT>(fmaf(xh[j], ga[j], be[j]));
    }
}
template <typename T, int V, int ACT>
__device__ inline void write_dx(const Vec<T, V> &x, const Vec<T, V> &dy, float mu, float r, float m1,
                                float m2, const float (&ga)[V], const float (&be)[V], T *p) {
    // dz gamma rounded as it is in the mean: a group of one element gives 0
#pragma clang fp contract(off)
    float dz[V], xh[V];
    dz_xh<T, V, ACT>(x, dy, mu, r, ga, be, dz, xh);
#pragma unroll
    for (int j = 0; j < V; ++j) dz[j] = r * (dz[j] * ga[j] - m1 - xh[j] * m2);
    store_vec<T, V>(p, dz);
}

// Sums over the block's rows of every channel's two values, out [2][cs].
// Rows of one wavefront (a row's vectors a power of two below 64) add by
// exchanges; what remains goes to buf [2][rows][cs], kThreads / cs threads per
// channel add the rows in strides, then one thread the rest.
template <int V>
struct ChannelLds {
    float buf[2 * kThreads * V];
    float join[2 * kThreads];
    float out[2 * kThreads * V];
};
template <int V>
__device__ inline void channel_sums(const Slab &s, float (&sx)[V], float (&sz)[V], ChannelLds<V> &l) {
    const int t = threadIdx.x;
    int rows = s.rp, row = s.row;
    bool writes = s.col >= 0;
    if ((s.cv & (s.cv - 1)) == 0 && s.cv < 64) {
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1)
            if (o >= s.cv)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    sx[j] += __shfl_xor(sx[j], o, 64);
                    sz[j] += __shfl_xor(sz[j], o, 64);
                }
        rows = kWaves;
        row = t >> 6;
        writes = (t & 63) < s.cv;
    }
    if (writes)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            l.buf[row * s.cs + s.col * V + j] = sx[j];
            l.buf[(rows + row) * s.cs + s.col * V + j] = sz[j];
        }
    __syncthreads();
    const int parts = max(1, min(kThreads / s.cs, rows / 4));
    for (int i = t; i < parts * s.cs; i += kThreads) {
        const int c = i % s.cs, q = i / s.cs;
        float x = 0.0f, z = 0.0f;
        for (int r = q; r < rows; r += parts) {
            x += l.buf[r * s.cs + c];
            z += l.buf[(rows + r) * s.cs + c];
        }
        if (parts == 1) {
            l.out[c] = x;
            l.out[s.cs + c] = z;
        } else {
            l.join[q * s.cs + c] = x;
            l.join[(parts + q) * s.cs + c] = z;
        }
    }
    __syncthreads();
    if (parts > 1) {
        for (int c = t; c < s.cs; c += kThreads) {
            float x = 0.0f, z = 0.0f;
            for (int q = 0; q < parts; ++q) {
                x += l.join[q * s.cs + c];
                z += l.join[(parts + q) * s.cs + c];
            }
            l.out[c] = x;
            l.out[s.cs + c] = z;
        }
        __syncthreads();
    }
}

// The whole segment in registers, x and dy read once.  seg [b][2][C]: its sums
// of dz xh and dz.  64 segments of up to 269 rows of 128 in fp32: 8.5 us for 12.6
// MB, as the forward launch.
template <typename T, int V, int IT, int ACT>
__global__ __launch_bounds__(kThreads) void norm_bwd_kernel(NormArgs a, NormCut k, const float *mean,
                                                            const float *rstd, T *dx, float *seg) {
    __shared__ ChannelLds<V> lds;
    __shared__ float gm[2][kMaxGroups];
    Slab s;
    const bool any = locate(a, k, blockIdx.x, s);
    if (!any) {
        for (int c = threadIdx.x; c < s.cs; c += kThreads) {
            seg[(int64_t)s.b * 2 * a.C + s.c0 + c] = 0.0f;
            seg[((int64_t)s.b * 2 + 1) * a.C + s.c0 + c] = 0.0f;
        }
        return;
    }
    Vec<T, V> x[IT], dy[IT];
    load_rows<T, V, IT>(k, s, (const T *)a.x, a.xs, x);
    load_rows<T, V, IT>(k, s, (const T *)a.dy, a.dys, dy);
    float ga[V], be[V], sx[V], sz[V];
    load_affine<V>(a, s, ga, be);
    const float mu = mean[s.b * a.groups + s.g0 + s.group], r = rstd[s.b * a.groups + s.g0 + s.group];
#pragma unroll
    for (int j = 0; j < V; ++j) sx[j] = sz[j] = 0.0f;
#pragma unroll
    for (int i = 0; i < IT; ++i)
        if (s.row + i * s.rp < s.rows) {
            float dz[V], xh[V];
            dz_xh<T, V, ACT>(x[i], dy[i], mu, r, ga, be, dz, xh);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                sx[j] = fmaf(dz[j], xh[j], sx[j]);
                sz[j] += dz[j];
            }
        }
    channel_sums<V>(s, sx, sz, lds);
    for (int c = threadIdx.x; c < s.cs; c += kThreads) {
        seg[(int64_t)s.b * 2 * a.C + s.c0 + c] = lds.out[c];
        seg[((int64_t)s.b * 2 + 1) * a.C + s.c0 + c] = lds.out[s.cs + c];
    }
    const int g = threadIdx.x >> 5, l = threadIdx.x & 31;
    if (g < s.gs) {
        float m1 = 0.0f, m2 = 0.0f;
        for (int c = g * a.width + l; c < (g + 1) * a.width; c += 32) {
            const float w = a.gamma ? a.gamma[s.c0 + c] : 1.0f;
            m2 = fmaf(w, lds.out[c], m2);
            m1 = fmaf(w, lds.out[s.cs + c], m1);
        }
        m1 = half_wave_sum(m1);
        m2 = half_wave_sum(m2);
        if (l == 0) {
            const float cnt = (float)s.rows * a.width;
            gm[0][g] = m1 / cnt;
            gm[1][g] = m2 / cnt;
        }
    }
    __syncthreads();
    if (s.col < 0) return;
    T *p = dx + (int64_t)s.r0 * a.C + s.c0 + s.col * V;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int row = s.row + i * s.rp;
        if (row < s.rows)
            write_dx<T, V, ACT>(x[i], dy[i], mu, r, gm[0][s.group], gm[1][s.group], ga, be, p + (int64_t)row * a.C);
    }
}

// part [b][chunk][2][C]: the chunk's sums of dz xh and dz.  8 segments of
// 16384 rows of 512 in bf16: 127 us with the two launches that follow, 5.3
// TB/s; ragged ones (101 MB a tensor) in 58 us, 3.5 TB/s, two streams beside
// the activation's slope (an exponential and a reciprocal an element).
template <typename T, int V, int ACT>
__global__ __launch_bounds__(kThreads) void norm_bwd_sums_kernel(NormArgs a, NormCut k, const float *mean,
                                                                 const float *rstd, float *part) {
    __shared__ ChannelLds<V> lds;
    Slab s;
    if (!locate(a, k, blockIdx.x, s)) return;
    float ga[V], be[V], sx[V], sz[V];
    load_affine<V>(a, s, ga, be);
#pragma unroll
    for (int j = 0; j < V; ++j) sx[j] = sz[j] = 0.0f;
    const float mu = mean[s.b * a.groups + s.g0 + s.group], r = rstd[s.b * a.groups + s.g0 + s.group];
    if (s.col >= 0) {
        const int64_t base = s.r0 + s.first;
        const T *px = (const T *)a.x + base * a.xs + s.c0 + s.col * V;
        const T *pg = (const T *)a.dy + base * a.dys + s.c0 + s.col * V;
#pragma unroll 4
        for (int row = s.row; row < s.rows; row += s.rp) {
            float dz[V], xh[V];
            dz_xh<T, V, ACT>(load_vec<T, V>(px + row * a.xs), load_vec<T, V>(pg + row * a.dys), mu, r, ga, be, dz, xh);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                sx[j] = fmaf(dz[j], xh[j], sx[j]);
                sz[j] += dz[j];
            }
        }
    }
    channel_sums<V>(s, sx, sz, lds);
    float *p = part + ((int64_t)s.b * k.chunks + s.chunk) * 2 * a.C + s.c0;
    for (int c = threadIdx.x; c < s.cs; c += kThreads) {
        p[c] = lds.out[c];
        p[a.C + c] = lds.out[s.cs + c];
    }
}

// Joins the chunks of a segment, one block per segment and group: seg
// [b][2][C] and the group's means of dz gamma and dz gamma xh (5 us).
__global__ __launch_bounds__(256) void norm_bwd_join_kernel(NormArgs a, NormCut k, const float *part, float *seg,
                                                            float2 *gmean) {
    __shared__ double red[2][256];
    const int b = blockIdx.x / a.groups, g = blockIdx.x % a.groups, t = threadIdx.x;
    int r0, n;
    segment_rows(a.ptr, b, a.B, a.n_rows, a.max_rows, a.status, r0, n);
    const int chunks = (n + k.chunk_rows - 1) / k.chunk_rows;
    // 256 / w threads share a channel's chunks; wider groups go in rounds
    const int w = min(a.width, 256), share = 256 / w;
    double m1 = 0.0, m2 = 0.0;
    for (int c0 = 0; c0 < a.width; c0 += w) {
        const int c = c0 + t % w, q = t / w;
        double x = 0.0, z = 0.0;
        if (c < a.width && q < share)
            for (int i = q; i < chunks; i += share) {
                const float *p = part + ((int64_t)b * k.chunks + i) * 2 * a.C + g * a.width + c;
                x += p[0];
                z += p[a.C];
            }
        __syncthreads();
        red[0][t] = x;
        red[1][t] = z;
        __syncthreads();
        if (t < w && c < a.width) {
            for (int i = 1; i < share; ++i) {
                x += red[0][i * w + t];
                z += red[1][i * w + t];
            }
            seg[(int64_t)b * 2 * a.C + g * a.width + c] = (float)x;
            seg[((int64_t)b * 2 + 1) * a.C + g * a.width + c] = (float)z;
            const double ga = a.gamma ? a.gamma[g * a.width + c] : 1.0f;
            m2 += ga * x;
            m1 += ga * z;
        }
    }
    __syncthreads();
    red[0][t] = m1;
    red[1][t] = m2;
    __syncthreads();
    for (int o = 128; o > 0; o >>= 1) {
        if (t < o) {
            red[0][t] += red[0][t + o];
            red[1][t] += red[1][t + o];
        }
        __syncthreads();
    }
    const double cnt = n ? (double)n * a.width : 1.0;
    if (t == 0) gmean[blockIdx.x] = make_float2((float)(red[0][0] / cnt), (float)(red[1][0] / cnt));
}

// dgamma and dbeta of 64 channels: the segments' sums, in their order.
__device__ inline void param_sums(int block, const NormArgs &a, const float *seg, float *dgamma, float *dbeta,
                                  double (*red)[64]) {
    const int t = threadIdx.x, c = block * 64 + (t & 63), q = t >> 6;
    double x = 0.0, z = 0.0;
    if (c < a.C)
        for (int b = q; b < a.B; b += kThreads / 64) {
            x += seg[(int64_t)b * 2 * a.C + c];
            z += seg[((int64_t)b * 2 + 1) * a.C + c];
        }
    red[2 * q][t & 63] = x;
    red[2 * q + 1][t & 63] = z;
    __syncthreads();
    if (q != 0 || c >= a.C) return;
    for (int i = 1; i < kThreads / 64; ++i) {
        x += red[2 * i][t];
        z += red[2 * i + 1][t];
    }
    if (dgamma) dgamma[c] = (float)x;
    if (dbeta) dbeta[c] = (float)z;
}

__global__ __launch_bounds__(kThreads) void norm_param_kernel(NormArgs a, const float *seg, float *dgamma,
                                                              float *dbeta) {
    __shared__ double red[kThreads / 32][64];
    param_sums(blockIdx.x, a, seg, dgamma, dbeta, red);
}

// dx of a chunk's rows (the same ragged segments: 67
// us, 4.5 TB/s); the first `params` blocks sum dgamma and dbeta
// instead (one launch less).
template <typename T, int V, int ACT>
__global__ __launch_bounds__(kThreads) void norm_bwd_apply_kernel(NormArgs a, NormCut k, const float *mean,
                                                                  const float *rstd, const float2 *gmean, T *dx,
                                                                  const float *seg, float *dgamma, float *dbeta,
                                                                  int params) {
    __shared__ double red[kThreads / 32][64];
    if ((int)blockIdx.x < params) {
        param_sums(blockIdx.x, a, seg, dgamma, dbeta, red);
        return;
    }
    Slab s;
    if (!locate(a, k, gridDim.x - 1 - blockIdx.x, s) || s.col < 0) return;
    float ga[V], be[V];
    load_affine<V>(a, s, ga, be);
    const int at = s.b * a.groups + s.g0 + s.group;
    const float mu = mean[at], r = rstd[at];
    const float2 m = gmean[at];
    const int64_t base = s.r0 + s.first;
    const T *px = (const T *)a.x + base * a.xs + s.c0 + s.col * V;
    const T *pg = (const T *)a.dy + base * a.dys + s.c0 + s.col * V;
    T *pd = dx + base * a.C + s.c0 + s.col * V;
#pragma unroll 4
    for (int row = s.row; row < s.rows; row += s.rp)
        write_dx<T, V, ACT>(load_vec<T, V>(px + row * a.xs), load_vec<T, V>(pg + row * a.dys), mu, r, m.x, m.y, ga, be,
                       pd + (int64_t)row * a.C);
}

// ------------------------------------------------------------------ launches

// Vectors that a thread of a fused launch can hold.  The launch takes the
// smallest of 4, 8 and 16 that the longest segment needs: more registers are
// fewer blocks on a CU (256 segments of 269 rows of 128 in fp32: 17 and 37 us
// forward and backward with 8, 22 and 48 us with 16).  Backward holds x and
// dy, so that 16 of both lose to a second read (64 segments of 1500 rows: 55
// us against 50); forward 16 still win (28 us against 32).
constexpr int kHold = 16, kHoldBwd = 8;
constexpr int kHoldStats = 8;    // of a chunk
// Vectors that a thread of the backward pass adds one after the other: its fp32
// sums lose up to half a unit of the sum so far with each, and chunks are
// joined in fp64.
constexpr int kSerial = 64;
// One block for every CU, and two in the backward pass, whose chunks are
// cheap: 15668 rows of 128 as one segment take 16 and 21 us forward and
// backward; with a quarter of the chunks 18 and 23 (8 segments of 16384 rows
// of 512 in bf16: backward 130 -> 276 us), with four times as many 29 and 26.
constexpr int kWantBlocks = 256;

// V: the widest vector that divides a group and suits every tensor.
// backward: its chunks need not fit the registers, and a longer one spares
// joins of a channel's sums.
NormCut norm_cut(int B, int max_rows, int C, int groups, int es, int V, bool backward) {
    NormCut k{};
    const int width = C / groups;
    k.V = V;
    const int wv = width / V;
    auto whole = [&](int bytes) {   // groups of a slab of about that many bytes a row
        const int want = std::max(1, (bytes + width * es - 1) / (width * es));
        return std::max(1, std::min({want, kMaxGroups, groups, kThreads / std::max(1, wv)}));
    };
    auto rows_held = [&](int gs, int it) { return kThreads / (gs * wv) * it; };
    if (wv <= kThreads) {
        // one launch: full 128-byte lines where the segment still fits and
        // they make a block for every CU (64 segments of 700 rows of 128 in
        // bf16: 19 us forward without the narrower slabs, 15 us with them;
        // 64 of 269 rows in fp32 13 us in two launches, 10 us in one)
        for (int bytes = 128; bytes >= 16; bytes /= 2) {
            const int gs = whole(bytes);
            if (rows_held(gs, backward ? kHoldBwd : kHold) < max_rows) continue;
            if (bytes > 32 && gs > 1 && (int64_t)B * ((groups + gs - 1) / gs) < 256) continue;
            k.gs = gs;
            k.slabs = (groups + gs - 1) / gs;
            k.chunks = 1;
            k.chunk_rows = std::max(1, max_rows);
            k.it = rows_held(gs, 4) >= max_rows ? 4 : rows_held(gs, 8) >= max_rows ? 8 : kHold;
            k.fused = true;
            return k;
        }
        k.gs = whole(128);
        k.slabs = (groups + k.gs - 1) / k.gs;
    } else {
        k.gs = 1;
        k.piece = kThreads * V;
        k.slabs = groups * ((width + k.piece - 1) / k.piece);
    }
    const int cv = k.piece ? kThreads : k.gs * wv, rp = kThreads / cv;
    const int64_t blocks = (int64_t)B * k.slabs;
    const int most = rp * (backward ? kSerial : kHoldStats), least = (max_rows + most - 1) / most;
    const int want_blocks = backward ? 2 * kWantBlocks : kWantBlocks;
    const int want = (int)std::min<int64_t>((max_rows + rp - 1) / rp, (want_blocks + blocks - 1) / blocks);
    k.chunks = std::max(1, std::max(least, want));
    k.chunk_rows = (std::max(1, max_rows) + k.chunks - 1) / k.chunks;
    k.chunk_rows = (k.chunk_rows + rp - 1) / rp * rp;
    k.chunks = std::max(1, (max_rows + k.chunk_rows - 1) / k.chunk_rows);
    k.it = kHoldStats;
    return k;
}

// The widest vector for a tensor's rows.
int vector_of(int V, const void *p, int64_t stride, int es) {
    while (V > 1 && (reinterpret_cast<uintptr_t>(p) % (V * es) != 0 || stride % V != 0)) V /= 2;
    return V;
}

struct NormLayout {
    size_t seg, gmean, part, total;
};
NormLayout norm_layout(const NormCut &k, int64_t B, int64_t C, int64_t groups) {
    NormLayout L;
    size_t o = kWsBase;
    auto take = [&](size_t bytes) { size_t r = o; o = align256(o + bytes); return r; };
    L.seg = take(B * 2 * C * sizeof(float));
    L.gmean = take(B * groups * sizeof(float2));
    const int64_t pieces = k.piece ? k.slabs / groups : 1;
    L.part = take(k.fused ? 0
                          : std::max(B * groups * k.chunks * pieces * (int64_t)sizeof(float2),
                                     B * k.chunks * 2 * C * (int64_t)sizeof(float)));
    L.total = o;
    return L;
}

bool fits(const NormCut &k, int B, int C, int groups) {
    return grid_fits((int64_t)B * k.slabs * k.chunks + (C + 63) / 64, kThreads) &&
           (k.fused || grid_fits((int64_t)B * groups, 256));
}

template <typename T, int V, int ACT>
sn_status forward_v(const NormArgs &a, void *y, float *mean, float *rstd, char *ws, hipStream_t s) {
    const NormCut k = norm_cut(a.B, a.max_rows, a.C, a.groups, sizeof(T), V, false);
    if (!fits(k, a.B, a.C, a.groups)) return SN_ERR_INVALID;
    const NormLayout L = norm_layout(k, a.B, a.C, a.groups);
    const int grid = a.B * k.slabs * k.chunks;
    if (k.fused) {
        if (k.it == 4)
            norm_fwd_kernel<T, V, 4, ACT><<<grid, kThreads, 0, s>>>(a, k, (T *)y, mean, rstd);
        else if (k.it == 8)
            norm_fwd_kernel<T, V, 8, ACT><<<grid, kThreads, 0, s>>>(a, k, (T *)y, mean, rstd);
        else
            norm_fwd_kernel<T, V, kHold, ACT><<<grid, kThreads, 0, s>>>(a, k, (T *)y, mean, rstd);
        return launch_status();
    }
    float2 *part = reinterpret_cast<float2 *>(ws + L.part);
    norm_stats_kernel<T, V, kHoldStats><<<grid, kThreads, 0, s>>>(a, k, part);
    SN_TRY(launch_status());
    norm_apply_kernel<T, V, ACT><<<grid, kThreads, 0, s>>>(a, k, part, (T *)y, mean, rstd);
    return launch_status();
}

template <typename T, int V, int ACT>
sn_status backward_v(const NormArgs &a, const float *mean, const float *rstd, void *dx, float *dgamma, float *dbeta,
                     char *ws, hipStream_t s) {
    const NormCut k = norm_cut(a.B, a.max_rows, a.C, a.groups, sizeof(T), V, true);
    if (!fits(k, a.B, a.C, a.groups)) return SN_ERR_INVALID;
    const NormLayout L = norm_layout(k, a.B, a.C, a.groups);
    const int grid = a.B * k.slabs * k.chunks, params = dgamma || dbeta ? (a.C + 63) / 64 : 0;
    float *seg = reinterpret_cast<float *>(ws + L.seg), *part = reinterpret_cast<float *>(ws + L.part);
    float2 *gmean = reinterpret_cast<float2 *>(ws + L.gmean);
    if (k.fused) {
        if (k.it == 4)
            norm_bwd_kernel<T, V, 4, ACT><<<grid, kThreads, 0, s>>>(a, k, mean, rstd, (T *)dx, seg);
        else
            norm_bwd_kernel<T, V, kHoldBwd, ACT><<<grid, kThreads, 0, s>>>(a, k, mean, rstd, (T *)dx, seg);
        SN_TRY(launch_status());
        if (params) norm_param_kernel<<<params, kThreads, 0, s>>>(a, seg, dgamma, dbeta);
        return launch_status();
    }
    norm_bwd_sums_kernel<T, V, ACT><<<grid, kThreads, 0, s>>>(a, k, mean, rstd, part);
    SN_TRY(launch_status());
    norm_bwd_join_kernel<<<a.B * a.groups, 256, 0, s>>>(a, k, part, seg, gmean);
    SN_TRY(launch_status());
    norm_bwd_apply_kernel<T, V, ACT><<<grid + params, kThreads, 0, s>>>(a, k, mean, rstd, gmean, (T *)dx, seg, dgamma,
                                                                  dbeta, params);
    return launch_status();
}

template <typename T>
int widest(const NormArgs &a, const void *out, bool backward) {
    int V = 16 / sizeof(T);
    while (V > 1 && a.width % V != 0) V /= 2;
    V = vector_of(V, a.x, a.xs, sizeof(T));
    V = vector_of(V, out, a.C, sizeof(T));
    if (backward) V = vector_of(V, a.dy, a.dys, sizeof(T));
    return V;
}

// Calls f with the vector and the activation as constants.
template <int V, typename F>
sn_status with_act(int act, F f) {
    using std::integral_constant;
    return act == SN_ACT_SSP    ? f(integral_constant<int, V>(), integral_constant<int, SN_ACT_SSP>())
           : act == SN_ACT_SILU ? f(integral_constant<int, V>(), integral_constant<int, SN_ACT_SILU>())
                                : f(integral_constant<int, V>(), integral_constant<int, SN_ACT_NONE>());
}
template <typename T, typename F>
sn_status with_vector(int V, int act, F f) {
    if constexpr (sizeof(T) == 2)
        if (V == 8) return with_act<8>(act, f);
    return V == 4 ? with_act<4>(act, f) : V == 2 ? with_act<2>(act, f) : with_act<1>(act, f);
}

template <typename T>
sn_status forward_t(const NormArgs &a, void *y, float *mean, float *rstd, char *ws, hipStream_t s) {
    return with_vector<T>(widest<T>(a, y, false), a.act, [&](auto V, auto ACT) {
        return forward_v<T, V.value, ACT.value>(a, y, mean, rstd, ws, s);
    });
}
template <typename T>
sn_status backward_t(const NormArgs &a, const float *mean, const float *rstd, void *dx, float *dgamma, float *dbeta,
                     char *ws, hipStream_t s) {
    return with_vector<T>(widest<T>(a, dx, true), a.act, [&](auto V, auto ACT) {
        return backward_v<T, V.value, ACT.value>(a, mean, rstd, dx, dgamma, dbeta, ws, s);
    });
}

}  // namespace

// Calls f with the two passes' cuts for each vector (which one is taken
// depends on the tensors).
template <typename F>
static void each_cut(const sn_group_norm &op, F f) {
    const int es = op.dtype == SN_F32 ? 4 : 2, width = op.n_channels / op.n_groups;
    auto cut = [&](int V, bool backward) {
        return norm_cut(op.n_segments, op.max_rows, op.n_channels, op.n_groups, es, V, backward);
    };
    for (int V = 16 / es; V >= 1; V /= 2)
        if (width % V == 0) f(cut(V, false), cut(V, true));
}

bool norm_fits(const sn_group_norm &op) {
    bool some = false;
    each_cut(op, [&](const NormCut &fwd, const NormCut &bwd) {
        some = some || (fits(fwd, op.n_segments, op.n_channels, op.n_groups) &&
                        fits(bwd, op.n_segments, op.n_channels, op.n_groups));
    });
    return some;
}

size_t norm_workspace(const sn_group_norm &op) {
    size_t need = kWsBase;
    each_cut(op, [&](const NormCut &fwd, const NormCut &bwd) {
        for (const NormCut &k : {fwd, bwd})
            need = std::max(need, norm_layout(k, op.n_segments, op.n_channels, op.n_groups).total);
    });
    return need;
}

sn_status norm_forward(const NormArgs &a, int dtype, void *y, float *mean, float *rstd, char *ws, hipStream_t s) {
    ProfScope prof(K_NORM_FWD, s);
    return dtype == SN_F32 ? forward_t<float>(a, y, mean, rstd, ws, s) : forward_t<bf16>(a, y, mean, rstd, ws, s);
}

sn_status norm_backward(const NormArgs &a, int dtype, const float *mean, const float *rstd, void *dx, float *dgamma,
                        float *dbeta, char *ws, hipStream_t s) {
    ProfScope prof(K_NORM_BWD, s);
    return dtype == SN_F32 ? backward_t<float>(a, mean, rstd, dx, dgamma, dbeta, ws, s)
                           : backward_t<bf16>(a, mean, rstd, dx, dgamma, dbeta, ws, s);
}

}  // namespace sn
