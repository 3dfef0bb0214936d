// Attention of a sequence's newest rows over its pages.
#include <algorithm>

#include "state.h"

namespace sn {
namespace {

constexpr int kThreads = 256;

__device__ inline float block_max(float v, float *buf) {
    __syncthreads();
    buf[threadIdx.x] = v;
    for (int o = kThreads / 2; o > 0; o >>= 1) {
        __syncthreads();
        if (threadIdx.x < o) buf[threadIdx.x] = fmaxf(buf[threadIdx.x], buf[threadIdx.x + o]);
    }
    __syncthreads();
    return buf[0];
}
__device__ inline float block_sum(float v, float *buf) {
    __syncthreads();
    buf[threadIdx.x] = v;
    for (int o = kThreads / 2; o > 0; o >>= 1) {
        __syncthreads();
        if (threadIdx.x < o) buf[threadIdx.x] += buf[threadIdx.x + o];
    }
    __syncthreads();
    return buf[0];
}

// A row of a head in fp32, eight elements from d on, without its scale.
template <typename T, int CODES>
__device__ inline void page_row8(const void *base, int64_t at, float (&x)[8]) {
    if constexpr (CODES == SN_CODES_NONE) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = to_f32(static_cast<const T *>(base)[at + j]);
    } else {
        decode8<CODES>(*reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(base) + at), x);
    }
}

// One block for each row and head: a thread scores a key of 256, then takes
// eight elements of some keys' values.
template <typename T, int CODES>
__global__ __launch_bounds__(kThreads) void attend_plain_kernel(CacheArgs a, T *o, float *lse) {
    __shared__ float q[SN_MAX_HEAD_DIM], p[kThreads], buf[kThreads], sums[kThreads][8];
    const int h = blockIdx.x % a.H, t = blockIdx.x / a.H, hk = h / a.G;
    int r0, n, length;
    sequence_rows(a, blockIdx.y, a.causal, r0, n, length);
    if (t >= n) return;
    const int row = r0 + t;
    for (int d = threadIdx.x; d < SN_MAX_HEAD_DIM; d += kThreads)
        q[d] = d < a.D ? to_f32(static_cast<const T *>(a.q)[row * a.qs + h * a.qh + d]) : 0.0f;
    const int end = a.causal ? length - n + t + 1 : length;
    const int begin = a.window > 0 ? max(0, end - a.window) : 0;
    const int chunks = a.Dp / 8, chunk = threadIdx.x % chunks, part = threadIdx.x / chunks, parts = kThreads / chunks;
    float acc[8] = {}, m = -INFINITY, l = 0.0f;
    for (int j0 = begin; j0 < end; j0 += kThreads) {
        __syncthreads();
        const int j = j0 + threadIdx.x;
        float s = -INFINITY, vs = 0.0f;
        if (j < end) {
            const int page = page_of(a, blockIdx.y, j);
            if (page >= 0) {
                const int64_t place = (((int64_t)page * a.Hkv + hk) << a.page_shift) + (j & (a.page - 1));
                float dot = 0.0f;
                for (int d = 0; d < a.Dp; d += 8) {
                    float x[8];
                    page_row8<T, CODES>(a.k, place * a.Dp + d, x);
#pragma unroll
                    for (int e = 0; e < 8; ++e) dot += d + e < a.D ? q[d + e] * x[e] : 0.0f;
                }
                s = dot * a.scale;
                vs = 1.0f;
                if (CODES != SN_CODES_NONE) {
                    s *= a.k_scale[place];
                    vs = a.v_scale[place];
                }
            }
        }
        const float top = fmaxf(m, block_max(s, buf));
        const float base = top == -INFINITY ? 0.0f : top;
        const float e = s == -INFINITY ? 0.0f : expf(s - base), keep = m == -INFINITY ? 0.0f : expf(m - base);
        l = l * keep + block_sum(e, buf);
        m = top;
        p[threadIdx.x] = e == 0.0f ? 0.0f : e * vs;
        __syncthreads();    // every thread has the sum before its place is used again
        buf[threadIdx.x] = s;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] *= keep;
        if (part < parts)
            for (int i = part; i < min(kThreads, end - j0); i += parts) {
                if (buf[i] == -INFINITY) continue;
                const int page = page_of(a, blockIdx.y, j0 + i);
                const int64_t place = (((int64_t)page * a.Hkv + hk) << a.page_shift) + ((j0 + i) & (a.page - 1));
                float x[8];
                page_row8<T, CODES>(a.v, place * a.Dp + chunk * 8, x);
#pragma unroll
                for (int i8 = 0; i8 < 8; ++i8) acc[i8] += p[i] * x[i8];
            }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[threadIdx.x][i] = part < parts ? acc[i] : 0.0f;
    __syncthreads();
    for (int d = threadIdx.x; d < a.D; d += kThreads) {
        float x = 0.0f;
        for (int i = 0; i < parts; ++i) x += sums[i * chunks + d / 8][d % 8];
        o[((int64_t)row * a.H + h) * a.D + d] = (T)(m == -INFINITY ? 0.0f : x / l);
    }
    if (lse && threadIdx.x == 0) lse[(int64_t)row * a.H + h] = m == -INFINITY ? -INFINITY : m + logf(l);
}

template <typename T, int CODES>
sn_status launch(const CacheArgs &a, void *o, float *lse, hipStream_t s) {
    ProfScope prof(K_CACHE_ATTEND, s);
    attend_plain_kernel<T, CODES><<<dim3(a.max_rows * a.H, a.B), kThreads, 0, s>>>(a, static_cast<T *>(o), lse);
    return launch_status();
}
template <typename T>
sn_status launch(const CacheArgs &a, int codes, void *o, float *lse, hipStream_t s) {
    if (codes == SN_CODES_INT8) return launch<T, SN_CODES_INT8>(a, o, lse, s);
    if (codes == SN_CODES_E4M3) return launch<T, SN_CODES_E4M3>(a, o, lse, s);
    return launch<T, SN_CODES_NONE>(a, o, lse, s);
}

}  // namespace

bool attend_fits(const sn_cache &op) { return grid_fits((int64_t)op.max_rows * op.n_heads * op.n_sequences, kThreads); }

size_t attend_workspace(const sn_cache &) { return kWsBase; }

sn_status cache_attend(const CacheArgs &a, int dtype, int codes, void *o, float *lse, char *, hipStream_t s) {
    return dtype == SN_F32 ? launch<float>(a, codes, o, lse, s) : launch<bf16>(a, codes, o, lse, s);
}

}  // namespace sn
