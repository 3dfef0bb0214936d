// Cross attention with a learned relative position bias, forward and
// backward, one wavefront per row.
//
//   s_ij = scale q_i.k_j + bias[bucket(k_pos_j - q_pos_i)],  p = softmax_j s
//   o = p v;  dP = dO v^T, delta_i = dO_i.o_i, dS = p (dP - delta)
//   dq = scale dS k, dk = scale dS^T q, dv = p^T dO, dbias = sums of dS
#include "context.h"

namespace sn {
namespace {

constexpr int kBiasBlocks = 64;   // partial sums of the bias gradient per head

// The backward pass carries p and dS times 2^24 and takes the factor out of
// the finished sums: exp flushes what is below 2^-126 to zero, which moves
// the smallest p that counts to 2^-150 (a key that no row attends to has
// gradients of that size, and they are still right).
constexpr float kLiftLn = 16.635532333438686f;   // 24 ln 2
constexpr float kUnlift = 1.0f / 16777216.0f;

__device__ inline int bucket_of(const AttnArgs &a, int rel) {
    int n = 0;
    for (int t = 0; t + 1 < a.nb; ++t) n += rel >= a.thr[t];
    return n;
}

__device__ inline float wave_max(float v) {
    for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
    return v;
}
__device__ inline float wave_sum(float v) {
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}

__device__ inline int find_segment(const AttnArgs &a, const int32_t *ptr, int row) {
    int lo = 0, hi = a.B;   // the last b with ptr[b] <= row
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (ptr[mid] <= row) lo = mid; else hi = mid;
    }
    return lo;
}

template <typename T>
__device__ inline float dot(const float *x, const T *y, int D) {
    float s = 0.0f;
    for (int d = 0; d < D; ++d) s = fmaf(x[d], to_f32(y[d]), s);
    return s;
}

// score of the lane's key for the row in LDS
template <typename T>
__device__ inline float score(const AttnArgs &a, const float *q, const T *k, int h, int qp, int kpos) {
    float s = dot(q, k, a.D) * a.scale;
    if (a.nb) s += a.bias[(int64_t)h * a.nb + bucket_of(a, __builtin_elementwise_sub_sat(kpos, qp))];
    return s;
}

template <typename T>
__global__ __launch_bounds__(64) void fwd_kernel(AttnArgs a, T *o, float *o_acc, float *lse) {
    __shared__ float q[128], p[64];
    const int row = blockIdx.x / a.H, h = blockIdx.x % a.H, lane = threadIdx.x;
    const int b = find_segment(a, a.q_ptr, row);
    int q0, nq, k0, nk;
    segment_rows(a.q_ptr, b, a.B, a.n_q, a.max_q, a.status, q0, nq);
    segment_rows(a.k_ptr, b, a.B, a.n_k, a.max_k, a.status, k0, nk);
    if (row < q0 || row >= q0 + nq) return;
    const T *qr = (const T *)a.q + row * a.qs + h * a.qh;
    for (int d = lane; d < 128; d += 64) q[d] = d < a.D ? to_f32(qr[d]) : 0.0f;
    __syncthreads();
    const T *K = (const T *)a.k + k0 * a.ks + (h / a.G) * a.kh, *V = (const T *)a.v + k0 * a.vs + (h / a.G) * a.vh;
    const int qp = a.q_pos ? a.q_pos[row] : row - q0;
    float m = -INFINITY, l = 0.0f, acc[2] = {0.0f, 0.0f};
    for (int j0 = 0; j0 < nk; j0 += 64) {
        const int j = j0 + lane;
        float s = -INFINITY;
        if (j < nk && (!a.keep || a.keep[k0 + j]))
            s = score(a, q, K + j * a.ks, h, qp, a.k_pos ? a.k_pos[k0 + j] : j);
        const float mt = wave_max(s);
        if (mt == -INFINITY) continue;
        const float mn = fmaxf(m, mt), c = fast_exp(m - mn);
        const float e = s == -INFINITY ? 0.0f : fast_exp(s - mn);
        l = l * c + wave_sum(e);
        m = mn;
        p[lane] = e;
        __syncthreads();
        acc[0] *= c;
        acc[1] *= c;
        for (int t = 0; t < 64 && j0 + t < nk; ++t) {
            const float w = p[t];
            if (w == 0.0f) continue;
            for (int u = 0; u < 2; ++u)
                if (lane + 64 * u < a.D) acc[u] = fmaf(w, to_f32(V[(j0 + t) * a.vs + lane + 64 * u]), acc[u]);
        }
        __syncthreads();
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    const int64_t at = (int64_t)row * a.H + h;
    for (int u = 0; u < 2; ++u) {
        const int d = lane + 64 * u;
        if (d >= a.D) continue;
        o[at * a.D + d] = from_f32<T>(acc[u] * inv);
        if (o_acc) o_acc[at * a.D + d] = acc[u] * inv;
    }
    if (lse && lane == 0) lse[at] = l > 0.0f ? m + fast_log(l) : -INFINITY;
}

// grid: H x kBiasBlocks; block y takes every kBiasBlocks-th row
template <typename T>
__global__ __launch_bounds__(64) void dq_kernel(AttnArgs a, const float *o_acc, const float *lse, T *dq, float *part) {
    __shared__ float q[128], g[128], ds[64], sums[SN_MAX_BUCKETS];
    __shared__ int bk[64];
    const int h = blockIdx.x, lane = threadIdx.x;
    sums[lane] = 0.0f;
    for (int row = blockIdx.y; row < a.n_q; row += kBiasBlocks) {
        const int b = find_segment(a, a.q_ptr, row);
        int q0, nq, k0, nk;
        segment_rows(a.q_ptr, b, a.B, a.n_q, a.max_q, a.status, q0, nq);
        segment_rows(a.k_ptr, b, a.B, a.n_k, a.max_k, a.status, k0, nk);
        if (row < q0 || row >= q0 + nq) continue;
        const T *qr = (const T *)a.q + row * a.qs + h * a.qh, *gr = (const T *)a.d_o + row * a.gs + h * a.gh;
        const int64_t at = (int64_t)row * a.H + h;
        float delta = 0.0f;
        __syncthreads();
        for (int d = lane; d < 128; d += 64) {
            q[d] = d < a.D ? to_f32(qr[d]) : 0.0f;
            g[d] = d < a.D ? to_f32(gr[d]) : 0.0f;
            if (d < a.D) delta = fmaf(g[d], o_acc[at * a.D + d], delta);
        }
        delta = wave_sum(delta);
        const float L = lse[at];
        const int qp = a.q_pos ? a.q_pos[row] : row - q0;
        const T *K = (const T *)a.k + k0 * a.ks + (h / a.G) * a.kh, *V = (const T *)a.v + k0 * a.vs + (h / a.G) * a.vh;
        float acc[2] = {0.0f, 0.0f};
        for (int j0 = 0; j0 < nk; j0 += 64) {
            const int j = j0 + lane;
            __syncthreads();
            ds[lane] = 0.0f;
            bk[lane] = -1;
            if (j < nk && (!a.keep || a.keep[k0 + j])) {
                const int kp = a.k_pos ? a.k_pos[k0 + j] : j;
                const float p = fast_exp(score(a, q, K + j * a.ks, h, qp, kp) - L + kLiftLn);
                ds[lane] = p * (dot(g, V + j * a.vs, a.D) - delta);
                bk[lane] = a.nb ? bucket_of(a, __builtin_elementwise_sub_sat(kp, qp)) : 0;
            }
            __syncthreads();
            for (int t = 0; t < 64; ++t) {
                if (bk[t] < 0) continue;
                if (bk[t] == lane) sums[lane] += ds[t];
                for (int u = 0; u < 2; ++u)
                    if (lane + 64 * u < a.D) acc[u] = fmaf(ds[t], to_f32(K[(j0 + t) * a.ks + lane + 64 * u]), acc[u]);
            }
        }
        for (int u = 0; u < 2; ++u)
            if (lane + 64 * u < a.D) dq[at * a.D + lane + 64 * u] = from_f32<T>(acc[u] * (a.scale * kUnlift));
    }
    if (part && lane < a.nb) part[((int64_t)blockIdx.y * a.H + h) * a.nb + lane] = sums[lane];
}

__global__ __launch_bounds__(64) void dbias_kernel(int n, const float *part, float *dbias) {
    const int i = blockIdx.x * 64 + threadIdx.x;
    if (i >= n) return;
    double s = 0.0;
    for (int k = 0; k < kBiasBlocks; ++k) s += part[(int64_t)k * n + i];
    dbias[i] = (float)(s * kUnlift);
}

template <typename T>
__global__ __launch_bounds__(64) void dkv_kernel(AttnArgs a, const float *o_acc, const float *lse, T *dk, T *dv) {
    __shared__ float k[128], v[128], ps[64], ds[64];
    const int key = blockIdx.x / a.Hkv, hk = blockIdx.x % a.Hkv, lane = threadIdx.x;
    const int b = find_segment(a, a.k_ptr, key);
    int q0, nq, k0, nk;
    segment_rows(a.q_ptr, b, a.B, a.n_q, a.max_q, a.status, q0, nq);
    segment_rows(a.k_ptr, b, a.B, a.n_k, a.max_k, a.status, k0, nk);
    if (key < k0 || key >= k0 + nk) return;
    const bool kept = !a.keep || a.keep[key];
    const T *kr = (const T *)a.k + key * a.ks + hk * a.kh, *vr = (const T *)a.v + key * a.vs + hk * a.vh;
    for (int d = lane; d < 128; d += 64) {
        k[d] = d < a.D ? to_f32(kr[d]) : 0.0f;
        v[d] = d < a.D ? to_f32(vr[d]) : 0.0f;
    }
    const int kp = a.k_pos ? a.k_pos[key] : key - k0;
    float ak[2] = {0.0f, 0.0f}, av[2] = {0.0f, 0.0f};
    const int n = kept ? nq * a.G : 0;   // the rows of every head that shares this key
    for (int r0 = 0; r0 < n; r0 += 64) {
        __syncthreads();
        ps[lane] = ds[lane] = 0.0f;
        if (r0 + lane < n) {
            const int row = q0 + (r0 + lane) / a.G, h = hk * a.G + (r0 + lane) % a.G;
            const T *qr = (const T *)a.q + row * a.qs + h * a.qh, *gr = (const T *)a.d_o + row * a.gs + h * a.gh;
            const int64_t at = (int64_t)row * a.H + h;
            const float p = fast_exp(score(a, k, qr, h, a.q_pos ? a.q_pos[row] : row - q0, kp) - lse[at] + kLiftLn);
            float delta = 0.0f;
            for (int d = 0; d < a.D; ++d) delta = fmaf(to_f32(gr[d]), o_acc[at * a.D + d], delta);
            ps[lane] = p;
            ds[lane] = p * (dot(v, gr, a.D) - delta);
        }
        __syncthreads();
        for (int t = 0; t < 64 && r0 + t < n; ++t) {
            const int row = q0 + (r0 + t) / a.G, h = hk * a.G + (r0 + t) % a.G;
            for (int u = 0; u < 2; ++u) {
                const int d = lane + 64 * u;
                if (d >= a.D) continue;
                ak[u] = fmaf(ds[t], to_f32(((const T *)a.q)[row * a.qs + h * a.qh + d]), ak[u]);
                av[u] = fmaf(ps[t], to_f32(((const T *)a.d_o)[row * a.gs + h * a.gh + d]), av[u]);
            }
        }
    }
    const int64_t at = ((int64_t)key * a.Hkv + hk) * a.D;
    for (int u = 0; u < 2; ++u) {
        const int d = lane + 64 * u;
        if (d >= a.D) continue;
        dk[at + d] = from_f32<T>(ak[u] * (a.scale * kUnlift));
        dv[at + d] = from_f32<T>(av[u] * kUnlift);
    }
}

template <typename T>
sn_status forward_t(const AttnArgs &a, void *o, float *o_acc, float *lse, hipStream_t s) {
    ProfScope prof(K_ATTN_FWD, s);
    fwd_kernel<T><<<a.n_q * a.H, 64, 0, s>>>(a, (T *)o, o_acc, lse);
    return launch_status();
}

template <typename T>
sn_status backward_t(const AttnArgs &a, const float *o_acc, const float *lse, void *dq, void *dk, void *dv,
                     float *dbias, char *ws, hipStream_t s) {
    ProfScope prof(K_ATTN_BWD, s);
    float *part = dbias ? reinterpret_cast<float *>(ws + kWsBase) : nullptr;
    dq_kernel<T><<<dim3(a.H, kBiasBlocks), 64, 0, s>>>(a, o_acc, lse, (T *)dq, part);
    SN_TRY(launch_status());
    if (a.n_k) {
        dkv_kernel<T><<<a.n_k * a.Hkv, 64, 0, s>>>(a, o_acc, lse, (T *)dk, (T *)dv);
        SN_TRY(launch_status());
    }
    if (dbias) {
        const int n = a.H * a.nb;
        dbias_kernel<<<(n + 63) / 64, 64, 0, s>>>(n, part, dbias);
        SN_TRY(launch_status());
    }
    return SN_OK;
}

}  // namespace

size_t attn_workspace(const sn_cross_attention &op) {
    return kWsBase + (size_t)kBiasBlocks * op.n_heads * SN_MAX_BUCKETS * sizeof(float);
}

sn_status attn_forward(const AttnArgs &a, int dtype, void *o, float *o_acc, float *lse, char *ws, hipStream_t s) {
    return dtype == SN_F32 ? forward_t<float>(a, o, o_acc, lse, s) : forward_t<bf16>(a, o, o_acc, lse, s);
}

sn_status attn_backward(const AttnArgs &a, int dtype, const float *o_acc, const float *lse, void *dq, void *dk,
                        void *dv, float *dbias, char *ws, hipStream_t s) {
    return dtype == SN_F32 ? backward_t<float>(a, o_acc, lse, dq, dk, dv, dbias, ws, s)
                           : backward_t<bf16>(a, o_acc, lse, dq, dk, dv, dbias, ws, s);
}

}  // namespace sn
