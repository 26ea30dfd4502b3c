// Gated linear recurrence h_t = exp(log_alpha_t) h_{t-1} + x_t, its backward
// pass and its single-token step. One thread per (sequence, channel) walks the
// tokens in order.
#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {

namespace {

// Token range of sequence n: the dense batch's [n T, (n + 1) T), or the packed
// offsets clamped into [0, T] (a decreasing pair is an empty sequence).
__device__ __forceinline__ void token_range(const int* cu, int n, int T, long long& begin, int& len) {
    if (!cu) {
        begin = (long long)n * T;
        len = T;
        return;
    }
    const int b = min(max(cu[n], 0), T), e = min(max(cu[n + 1], 0), T);
    begin = b;
    len = max(e - b, 0);
}

template <typename T>
__global__ void recurrence_fwd_kernel(const T* log_alpha, const T* x, const float* h0, T* h, float* h_T,
                                      const int* cu, int N, int TT, int D) {
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= (long long)N * D) return;
    const int n = (int)(i / D), c = (int)(i % D);
    long long begin;
    int len;
    token_range(cu, n, TT, begin, len);
    float s = h0 ? h0[i] : 0.f;
    for (int t = 0; t < len; ++t) {
        const long long j = (begin + t) * D + c;
        s = fmaf(expf(to_f32(log_alpha[j])), s, to_f32(x[j]));
        h[j] = from_f32<T>(s);
    }
    if (h_T) h_T[i] = s;
}

template <typename T>
__global__ void recurrence_bwd_kernel(const T* log_alpha, const T* h, const float* h0, const T* dh, const float* dh_T,
                                      T* dx, T* dla, float* dh0, const int* cu, int N, int TT, int D) {
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= (long long)N * D) return;
    const int n = (int)(i / D), c = (int)(i % D);
    long long begin;
    int len;
    token_range(cu, n, TT, begin, len);
    float s = dh_T ? dh_T[i] : 0.f;
    for (int t = len - 1; t >= 0; --t) {
        const long long j = (begin + t) * D + c;
        s += to_f32(dh[j]);
        dx[j] = from_f32<T>(s);
        s *= expf(to_f32(log_alpha[j]));
        const float before = t > 0 ? to_f32(h[j - D]) : (h0 ? h0[i] : 0.f);
        dla[j] = from_f32<T>(s * before);
    }
    if (dh0) dh0[i] = s;
}

template <typename T>
__global__ void recurrence_step_kernel(const T* log_alpha, const T* x, const float* h_in, float* h_out, T* y,
                                       long long cells) {
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= cells) return;
    const float s = fmaf(expf(to_f32(log_alpha[i])), h_in[i], to_f32(x[i]));
    h_out[i] = s;
    y[i] = from_f32<T>(s);
}

constexpr int kThreads = 128;
unsigned blocks_for(long long cells) { return (unsigned)((cells + kThreads - 1) / kThreads); }

}  // namespace

cudaError_t launch_recurrence_fwd(const RecurrenceArgs& a, cudaStream_t stream) {
    auto go = [&](auto t) {
        using T = decltype(t);
        recurrence_fwd_kernel<T><<<blocks_for((long long)a.N * a.D), kThreads, 0, stream>>>(
            (const T*)a.log_alpha, (const T*)a.x, a.state0, (T*)a.out, a.state_end, a.cu_seqlens, a.N, a.T, a.D);
        return cudaGetLastError();
    };
    return a.bf16 ? go(__nv_bfloat16()) : go(float());
}

cudaError_t launch_recurrence_bwd(const RecurrenceArgs& a, cudaStream_t stream) {
    auto go = [&](auto t) {
        using T = decltype(t);
        recurrence_bwd_kernel<T><<<blocks_for((long long)a.N * a.D), kThreads, 0, stream>>>(
            (const T*)a.log_alpha, (const T*)a.h_fwd, a.h0, (const T*)a.x, a.state0, (T*)a.out, (T*)a.out_la,
            a.state_end, a.cu_seqlens, a.N, a.T, a.D);
        return cudaGetLastError();
    };
    return a.bf16 ? go(__nv_bfloat16()) : go(float());
}

cudaError_t launch_recurrence_step(const void* la, const void* x, const float* h_in, float* h_out, void* y,
                                   long long cells, int bf16, cudaStream_t stream) {
    auto go = [&](auto t) {
        using T = decltype(t);
        recurrence_step_kernel<T><<<blocks_for(cells), kThreads, 0, stream>>>((const T*)la, (const T*)x, h_in, h_out,
                                                                               (T*)y, cells);
        return cudaGetLastError();
    };
    return bf16 ? go(__nv_bfloat16()) : go(float());
}

}  // namespace kda
