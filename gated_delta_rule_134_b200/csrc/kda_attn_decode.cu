// Attention of one new token per sequence over a paged key-value cache. One
// CTA per (sequence, query head); each warp walks every fourth position with a
// running maximum and sum, and the warps are joined at the end.
#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {

namespace {

template <typename T, int D>
__global__ void attn_decode_kernel(AttnDecodeArgs a) {
    constexpr int W = 4, E = D / 32;
    __shared__ float so[W][D], sm[W], sl[W];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n = blockIdx.x / a.Hq, h = blockIdx.x % a.Hq, hk = h / (a.Hq / a.Hk);
    const int held = a.seq_lens[n], cap = a.max_pages * a.page_size;
    const bool put = a.k_new && held >= 0;
    // positions [first, last) are candidates; the new one, `held`, is the last of them
    const long long total = held < 0 ? 0 : (long long)held + (put ? 1 : 0);  // a length near 2^31 must not wrap
    const int last = (int)min(total, (long long)cap);
    const int first = a.window ? (int)min(max(0ll, total - a.window), (long long)last) : 0;
    const int* table = a.page_table + (size_t)n * a.max_pages;
    const T* q = (const T*)a.q + ((size_t)n * a.Hq + h) * D;
    float qv[E], acc[E], m = -INFINITY, l = 0.f;
    for (int e = 0; e < E; ++e) {
        qv[e] = to_f32(q[lane * E + e]) * a.scale;
        acc[e] = 0.f;
    }
    for (int p = first + warp; p < last; p += W) {
        const int page = table[p / a.page_size];
        if (page < 0 || page >= a.n_pages) continue;
        const size_t at = (((size_t)page * a.Hk + hk) * a.page_size + p % a.page_size) * D;
        const T *kp = (const T*)a.k_cache + at, *vp = (const T*)a.v_cache + at;
        if (put && p == held) {
            kp = (const T*)a.k_new + ((size_t)n * a.Hk + hk) * D;
            vp = (const T*)a.v_new + ((size_t)n * a.Hk + hk) * D;
            if (h % (a.Hq / a.Hk) == 0)
                for (int e = 0; e < E; ++e) {
                    ((T*)a.k_cache)[at + lane * E + e] = kp[lane * E + e];
                    ((T*)a.v_cache)[at + lane * E + e] = vp[lane * E + e];
                }
        }
        float s = 0.f;
        for (int e = 0; e < E; ++e) s = fmaf(qv[e], to_f32(kp[lane * E + e]), s);
        s = warp_sum(s);
        if (s == -INFINITY) continue;
        const float top = fmaxf(m, s), keep = expf(m - top), p_ = expf(s - top);
        l = l * keep + p_;
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * keep + p_ * to_f32(vp[lane * E + e]);
        m = top;
    }
    for (int e = 0; e < E; ++e) so[warp][lane * E + e] = acc[e];
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
    __syncthreads();
    float top = -INFINITY, sum = 0.f;
    for (int w = 0; w < W; ++w)
        if (sl[w] != 0.f) top = fmaxf(top, sm[w]);
    for (int w = 0; w < W; ++w)
        if (sl[w] != 0.f) sum += sl[w] * expf(sm[w] - top);
    for (int c = threadIdx.x; c < D; c += blockDim.x) {
        float o = 0.f;
        for (int w = 0; w < W; ++w)
            if (sl[w] != 0.f) o += so[w][c] * expf(sm[w] - top);
        ((T*)a.o)[((size_t)n * a.Hq + h) * D + c] = from_f32<T>(sum == 0.f ? 0.f : o / sum);
    }
    if (a.lse && threadIdx.x == 0) a.lse[(size_t)n * a.Hq + h] = sum == 0.f ? -INFINITY : top + logf(sum);
}

}  // namespace

size_t attn_decode_workspace_bytes(int N, int Hq, int Hk, int d) {
    (void)N; (void)Hq; (void)Hk; (void)d;
    return 0;
}

cudaError_t launch_attn_decode(const AttnDecodeArgs& a, cudaStream_t stream) {
    const unsigned blocks = (unsigned)a.N * a.Hq;
    if (a.bf16) {
        if (a.d == 64) attn_decode_kernel<__nv_bfloat16, 64><<<blocks, 128, 0, stream>>>(a);
        else attn_decode_kernel<__nv_bfloat16, 128><<<blocks, 128, 0, stream>>>(a);
    } else {
        if (a.d == 64) attn_decode_kernel<float, 64><<<blocks, 128, 0, stream>>>(a);
        else attn_decode_kernel<float, 128><<<blocks, 128, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace kda
