// Group norm with an activation over the rows of each segment, channels
// last, forward and backward: one block per segment and group.
//
//   xh = (x - mean) rstd, z = gamma xh + beta, y = act(z)
//   dz = dy act'(z), dbeta = sum dz, dgamma = sum dz xh,
//   dx = rstd (dz gamma - mean(dz gamma) - xh mean(dz gamma xh))
#include "context.h"

namespace sn {
namespace {

constexpr int kThreads = 256;

__device__ inline float act_fwd(float z, int act) {
    if (act == SN_ACT_SSP) return ssp(z);
    if (act == SN_ACT_SILU) return z * sigm(z);
    return z;
}
__device__ inline float act_grad(float z, int act) {
    if (act == SN_ACT_SSP) return sigm(z);
    if (act == SN_ACT_SILU) {
        const float s = sigm(z);
        return s * (1.0f + z * (1.0f - s));
    }
    return 1.0f;
}

__device__ inline float block_sum(float v, float *red) {
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.0f;
    for (int w = 0; w < kThreads / 64; ++w) s += red[w];
    return s;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void fwd_kernel(NormArgs a, T *y, float *mean, float *rstd) {
    __shared__ float red[kThreads / 64];
    const int b = blockIdx.x / a.groups, g = blockIdx.x % a.groups;
    int r0, n;
    segment_rows(a.ptr, b, a.B, a.n_rows, a.max_rows, a.status, r0, n);
    const T *x = (const T *)a.x + r0 * a.xs + g * a.width;
    const int64_t cnt = (int64_t)n * a.width;
    float s = 0.0f;
    for (int64_t i = threadIdx.x; i < cnt; i += kThreads) s += to_f32(x[i / a.width * a.xs + i % a.width]);
    const float mu = cnt ? block_sum(s, red) / (float)cnt : 0.0f;
    s = 0.0f;
    for (int64_t i = threadIdx.x; i < cnt; i += kThreads) {
        const float d = to_f32(x[i / a.width * a.xs + i % a.width]) - mu;
        s = fmaf(d, d, s);
    }
    const float var = cnt ? block_sum(s, red) / (float)cnt : 0.0f;
    const float r = 1.0f / sqrtf(var + a.eps);
    for (int64_t i = threadIdx.x; i < cnt; i += kThreads) {
        const int c = g * a.width + (int)(i % a.width);
        const float xh = (to_f32(x[i / a.width * a.xs + i % a.width]) - mu) * r;
        const float z = fmaf(xh, a.gamma ? a.gamma[c] : 1.0f, a.beta ? a.beta[c] : 0.0f);
        y[(r0 + i / a.width) * a.C + c] = from_f32<T>(act_fwd(z, a.act));
    }
    if (threadIdx.x == 0) {
        if (mean) mean[blockIdx.x] = mu;
        if (rstd) rstd[blockIdx.x] = r;
    }
}

// part [B][2][C]: the sums over the segment's rows of dz xh and dz
template <typename T>
__global__ __launch_bounds__(kThreads) void bwd_kernel(NormArgs a, const float *mean, const float *rstd, T *dx,
                                                       float *part) {
    __shared__ float red[kThreads / 64];
    const int b = blockIdx.x / a.groups, g = blockIdx.x % a.groups;
    int r0, n;
    segment_rows(a.ptr, b, a.B, a.n_rows, a.max_rows, a.status, r0, n);
    const float mu = mean[blockIdx.x], r = rstd[blockIdx.x];
    const T *x = (const T *)a.x, *dy = (const T *)a.dy;
    float m1 = 0.0f, m2 = 0.0f;
    for (int c = g * a.width; c < (g + 1) * a.width; ++c) {
        const float ga = a.gamma ? a.gamma[c] : 1.0f, be = a.beta ? a.beta[c] : 0.0f;
        float sx = 0.0f, sz = 0.0f;
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const float xh = (to_f32(x[(int64_t)(r0 + i) * a.xs + c]) - mu) * r;
            const float dz = to_f32(dy[(int64_t)(r0 + i) * a.dys + c]) * act_grad(fmaf(xh, ga, be), a.act);
            sx = fmaf(dz, xh, sx);
            sz += dz;
        }
        sx = block_sum(sx, red);
        sz = block_sum(sz, red);
        if (threadIdx.x == 0) {
            part[((int64_t)b * 2) * a.C + c] = sx;
            part[((int64_t)b * 2 + 1) * a.C + c] = sz;
        }
        m1 = fmaf(sz, ga, m1);
        m2 = fmaf(sx, ga, m2);
    }
    const float inv = n ? 1.0f / ((float)n * a.width) : 0.0f;
    m1 *= inv;
    m2 *= inv;
    for (int64_t i = threadIdx.x; i < (int64_t)n * a.width; i += kThreads) {
        const int c = g * a.width + (int)(i % a.width);
        const int64_t row = r0 + i / a.width;
        const float ga = a.gamma ? a.gamma[c] : 1.0f, be = a.beta ? a.beta[c] : 0.0f;
        const float xh = (to_f32(x[row * a.xs + c]) - mu) * r;
        const float dz = to_f32(dy[row * a.dys + c]) * act_grad(fmaf(xh, ga, be), a.act);
        dx[row * a.C + c] = from_f32<T>(r * (dz * ga - m1 - xh * m2));
    }
}

__global__ __launch_bounds__(64) void param_kernel(int B, int C, const float *part, float *dgamma, float *dbeta) {
    const int c = blockIdx.x * 64 + threadIdx.x;
    if (c >= C) return;
    double sx = 0.0, sz = 0.0;
    for (int b = 0; b < B; ++b) {
        sx += part[((int64_t)b * 2) * C + c];
        sz += part[((int64_t)b * 2 + 1) * C + c];
    }
    if (dgamma) dgamma[c] = (float)sx;
    if (dbeta) dbeta[c] = (float)sz;
}

template <typename T>
sn_status backward_t(const NormArgs &a, const float *mean, const float *rstd, void *dx, float *dgamma, float *dbeta,
                     char *ws, hipStream_t s) {
    ProfScope prof(K_NORM_BWD, s);
    float *part = reinterpret_cast<float *>(ws + kWsBase);
    bwd_kernel<T><<<a.B * a.groups, kThreads, 0, s>>>(a, mean, rstd, (T *)dx, part);
    SN_TRY(launch_status());
    if (dgamma || dbeta) {
        param_kernel<<<(a.C + 63) / 64, 64, 0, s>>>(a.B, a.C, part, dgamma, dbeta);
        SN_TRY(launch_status());
    }
    return SN_OK;
}

}  // namespace

size_t norm_workspace(const sn_group_norm &op) {
    return kWsBase + (size_t)op.n_segments * 2 * op.n_channels * sizeof(float);
}

sn_status norm_forward(const NormArgs &a, int dtype, void *y, float *mean, float *rstd, char *ws, hipStream_t s) {
    ProfScope prof(K_NORM_FWD, s);
    if (dtype == SN_F32)
        fwd_kernel<float><<<a.B * a.groups, kThreads, 0, s>>>(a, (float *)y, mean, rstd);
    else
        fwd_kernel<bf16><<<a.B * a.groups, kThreads, 0, s>>>(a, (bf16 *)y, mean, rstd);
    return launch_status();
}

sn_status norm_backward(const NormArgs &a, int dtype, const float *mean, const float *rstd, void *dx, float *dgamma,
                        float *dbeta, char *ws, hipStream_t s) {
    return dtype == SN_F32 ? backward_t<float>(a, mean, rstd, dx, dgamma, dbeta, ws, s)
                           : backward_t<bf16>(a, mean, rstd, dx, dgamma, dbeta, ws, s);
}

}  // namespace sn
