// Queries and keys of a layer: norm per head and rotation by position in one
// pass, and the backward pass. One warp per (token, head).
//
//     y = R (w x r),  r = (m + eps)^-1/2,  m = share * sum x^2
// (share = 1 for the L2 norm, 1/d for the RMS norm.) With u = R^T dy, n = x r:
//     dw = sum u n,   dx = r (w u - share * n * sum(w u n)).
#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {

namespace {

struct Side {
    const void *x, *w, *dy;
    void* y;
    float* dw;
    long long stride_t, stride_h;
    int H;
    float scale;
};

__device__ __forceinline__ long long position_of(const QkArgs& a, long long t) {
    const long long p = a.pos_bytes == 8 ? ((const long long*)a.positions)[t] : (long long)((const int*)a.positions)[t];
    return min(max(p, 0ll), (long long)a.max_pos - 1);
}

// Partner channel, and this channel's cosine and signed sine: y_c = x_c cos + x_partner sin.
__device__ __forceinline__ int turn(const QkArgs& a, long long pos, int c, float& cs, float& sn) {
    const int half = a.rot / 2;
    cs = 1.f;
    sn = 0.f;
    if (c >= a.rot) return c;
    const int i = a.interleaved ? c / 2 : c % half;
    const bool first = a.interleaved ? c % 2 == 0 : c < half;
    cs = a.cos[pos * half + i];
    sn = a.sin[pos * half + i];
    if (first) sn = -sn;
    return a.interleaved ? (c ^ 1) : (first ? c + half : c - half);
}

__device__ __forceinline__ float rnorm(const float* x, int d, float share, float eps) {
    float top = 0.f, ss = 0.f;
    const int lane = threadIdx.x & 31;
    for (int c = lane; c < d; c += 32) top = fmaxf(top, fabsf(x[c]));
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    const float down = top > 1e15f ? 0x1p-80f : 1.f;
    for (int c = lane; c < d; c += 32) ss = fmaf(x[c] * down, x[c] * down, ss);
    ss = warp_sum(ss);
    return down * rsqrtf(fmaf(ss, share, eps * down * down));
}

template <typename T>
__global__ void qk_fwd_kernel(QkArgs a) {
    __shared__ float sx[4][256];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, H = a.Hq + a.Hk;
    const long long row = (long long)blockIdx.x * 4 + warp;
    if (row >= (long long)a.n * H) return;
    const long long t = row / H;
    int h = (int)(row % H);
    const bool is_q = h < a.Hq;
    if (!is_q) h -= a.Hq;
    const T* x = is_q ? (const T*)a.q + t * a.q_stride_t + h * a.q_stride_h
                      : (const T*)a.k + t * a.k_stride_t + h * a.k_stride_h;
    T* y = is_q ? (T*)a.q_out + (t * a.Hq + h) * a.d : (T*)a.k_out + (t * a.Hk + h) * a.d;
    const T* w = (const T*)(is_q ? a.q_weight : a.k_weight);
    float* s = sx[warp];
    for (int c = lane; c < a.d; c += 32) s[c] = to_f32(x[c]);
    __syncwarp();
    const float r = rnorm(s, a.d, a.norm ? 1.f / a.d : 1.f, a.eps);
    __syncwarp();
    for (int c = lane; c < a.d; c += 32) s[c] = s[c] * r * (w ? to_f32(w[c]) : 1.f);
    __syncwarp();
    const long long pos = a.positions ? position_of(a, t) : 0;
    for (int c = lane; c < a.d; c += 32) {
        float cs, sn;
        const int p = turn(a, pos, c, cs, sn);
        y[c] = from_f32<T>((s[c] * cs + s[p] * sn) * (is_q ? a.q_scale : 1.f));
    }
}

// One CTA walks rows (token, head) of one side with a stride; dw partials per CTA.
template <typename T>
__global__ void qk_bwd_kernel(QkArgs a, float* part) {
    __shared__ float su[4][256], sn_[4][256], sw[4][256];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool is_q = blockIdx.y == 0;
    const int H = is_q ? a.Hq : a.Hk;
    const T* w = (const T*)(is_q ? a.q_weight : a.k_weight);
    float* u = su[warp];
    float* n = sn_[warp];
    float* dw = sw[warp];
    const float share = a.norm ? 1.f / a.d : 1.f;
    for (int c = lane; c < a.d; c += 32) dw[c] = 0.f;
    for (long long row = (long long)blockIdx.x * 4 + warp; row < (long long)a.n * H; row += (long long)gridDim.x * 4) {
        const long long t = row / H;
        const int h = (int)(row % H);
        const T* x = is_q ? (const T*)a.q + t * a.q_stride_t + h * a.q_stride_h
                          : (const T*)a.k + t * a.k_stride_t + h * a.k_stride_h;
        const T* dy = (const T*)(is_q ? a.d_q_out : a.d_k_out) + row * a.d;
        T* dx = (T*)(is_q ? a.q_out : a.k_out) + row * a.d;
        const long long pos = a.positions ? position_of(a, t) : 0;
        __syncwarp();
        for (int c = lane; c < a.d; c += 32) {
            n[c] = to_f32(x[c]);
            float cs, sn;
            const int p = turn(a, pos, c, cs, sn);
            u[c] = (to_f32(dy[c]) * cs - to_f32(dy[p]) * sn) * (is_q ? a.q_scale : 1.f);
        }
        __syncwarp();
        const float r = rnorm(n, a.d, share, a.eps);
        __syncwarp();
        float dot = 0.f;
        for (int c = lane; c < a.d; c += 32) {
            n[c] *= r;
            dw[c] = fmaf(u[c], n[c], dw[c]);
            u[c] *= w ? to_f32(w[c]) : 1.f;
            dot = fmaf(u[c], n[c], dot);
        }
        dot = warp_sum(dot) * share;
        for (int c = lane; c < a.d; c += 32) dx[c] = from_f32<T>(r * (u[c] - n[c] * dot));
    }
    __syncthreads();
    if (!part) return;
    for (int c = threadIdx.x; c < a.d; c += blockDim.x)
        part[((size_t)blockIdx.y * gridDim.x + blockIdx.x) * a.d + c] = (sw[0][c] + sw[1][c]) + (sw[2][c] + sw[3][c]);
}

__global__ void qk_dw_kernel(const float* part, float* dwq, float* dwk, int blocks, int d) {
    float* dw = blockIdx.x == 0 ? dwq : dwk;
    if (!dw) return;
    for (int c = threadIdx.x; c < d; c += blockDim.x) {
        double s = 0;
        for (int b = 0; b < blocks; ++b) s += part[((size_t)blockIdx.x * blocks + b) * d + c];
        dw[c] = (float)s;
    }
}

constexpr int kBwdBlocks = 592;

}  // namespace

size_t qk_norm_rope_bwd_workspace_bytes(int n, int Hq, int Hk, int d) {
    (void)n; (void)Hq; (void)Hk;
    return (size_t)2 * kBwdBlocks * d * sizeof(float);
}

cudaError_t launch_qk_norm_rope(const QkArgs& a, cudaStream_t stream) {
    const unsigned blocks = (unsigned)(((long long)a.n * (a.Hq + a.Hk) + 3) / 4);
    if (a.bf16) qk_fwd_kernel<__nv_bfloat16><<<blocks, 128, 0, stream>>>(a);
    else qk_fwd_kernel<float><<<blocks, 128, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_qk_norm_rope_bwd(const QkArgs& a, cudaStream_t stream) {
    float* part = a.d_q_weight || a.d_k_weight ? (float*)a.workspace : nullptr;
    const dim3 grid(kBwdBlocks, 2);
    if (a.bf16) qk_bwd_kernel<__nv_bfloat16><<<grid, 128, 0, stream>>>(a, part);
    else qk_bwd_kernel<float><<<grid, 128, 0, stream>>>(a, part);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess || !part) return err;
    qk_dw_kernel<<<2, 256, 0, stream>>>(part, a.d_q_weight, a.d_k_weight, kBwdBlocks, a.d);
    return cudaGetLastError();
}

}  // namespace kda
