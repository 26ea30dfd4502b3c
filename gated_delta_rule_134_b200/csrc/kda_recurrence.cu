// Gated linear recurrence h_t = exp(log_alpha_t) h_{t-1} + x_t, its backward
// pass and its single-token step.
//
// Both directions are one affine scan per channel: a span of tokens maps the
// state that enters it to A s + H, and spans compose,
//     (A2, H2) after (A1, H1) = (A2 A1, A2 H1 + H2).
// Forward, a token is (a_t, x_t). Backward, with c the gradient of the state
// that a token hands on, a token is (a_t, a_t dh_t), walked from the last to the
// first: dx_t = dh_t + c, c <- a_t dx_t, dlog_alpha_t = c h_{t-1}.
//
// What bounds it: HBM, 3 (backward 5) elements of the tensors per token and
// channel, each read or written once. One cluster of CTAs owns a (sequence,
// slice of 128 bytes of channels) and walks the tokens; each pass of the walk is
// a tile of tokens per CTA, held in registers: a thread has R consecutive tokens
// of 16 bytes of channels, composes them, the four token groups of a warp are
// composed by shuffles, the warps through shared memory, the CTAs of the cluster
// through distributed shared memory (one cluster barrier a tile), and the thread
// then runs its tokens again from the state that enters them. The next tile's
// loads are in flight meanwhile. The sequential depth is T / (tokens of a
// cluster's tile); clusters of more than one CTA are taken where sequences times
// channel slices do not fill the GPU. Nothing waits on a flag, and the order of
// every product and sum is fixed by the sizes alone.
#include "kda_common.cuh"
#include "kda_internal.h"

#include <cooperative_groups.h>

namespace kda {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kGroups = kThreads / 8;  // token groups of a CTA (8 threads across the channels)
constexpr int kMaxCluster = 8;

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

// 16 bytes of one token's channels: 8 bf16 or 4 floats.
template <typename T> struct Pack {
    static constexpr int V = 16 / sizeof(T);
    uint32_t w[4];
    __device__ __forceinline__ float get(int i) const {
        if constexpr (V == 4) return __uint_as_float(w[i]);
        else return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
    __device__ __forceinline__ void clear() { w[0] = w[1] = w[2] = w[3] = 0u; }
};

template <typename T> __device__ __forceinline__ float decay(float log_alpha);
template <> __device__ __forceinline__ float decay<float>(float x) { return expf(x); }
// two units in the last place of 32 bits off at most for |x| < 1: far below a bf16 input's own step
template <> __device__ __forceinline__ float decay<__nv_bfloat16>(float x) { return __expf(x); }

// Channel i of this thread, within the slice: neighbours where 16-byte rows allow
// wide accesses; else eight apart, so that the eight threads of a token group
// read neighbouring elements.
template <typename T, bool ALIGNED> __device__ __forceinline__ int channel_of(int col, int i) {
    return ALIGNED ? col * Pack<T>::V + i : col + 8 * i;
}

template <typename T, bool ALIGNED>
__device__ __forceinline__ Pack<T> load_row(const T* row, int c0, int col, int D, bool on) {
    constexpr int V = Pack<T>::V;
    Pack<T> p;
    p.clear();
    if (!on) return p;
    if constexpr (ALIGNED) {
        if (c0 + col * V < D) {
            const uint4 v = __ldcs(reinterpret_cast<const uint4*>(row + c0 + col * V));
            p.w[0] = v.x; p.w[1] = v.y; p.w[2] = v.z; p.w[3] = v.w;
        }
    } else if constexpr (V == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = c0 + channel_of<T, false>(col, i);
            if (c < D) p.w[i] = __float_as_uint(__ldcs(reinterpret_cast<const float*>(row) + c));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = c0 + channel_of<T, false>(col, i);
            if (c < D) p.w[i >> 1] |= (uint32_t)__ldcs(reinterpret_cast<const unsigned short*>(row) + c) << (i & 1 ? 16 : 0);
        }
    }
    return p;
}

template <typename T, bool ALIGNED>
__device__ __forceinline__ void store_row(T* row, int c0, int col, int D, const float (&x)[Pack<T>::V]) {
    constexpr int V = Pack<T>::V;
    if constexpr (ALIGNED) {
        if (c0 + col * V >= D) return;
        uint4 v;
        if constexpr (V == 4) {
            v = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&b);
            }
            v = make_uint4(w[0], w[1], w[2], w[3]);
        }
        __stcs(reinterpret_cast<uint4*>(row + c0 + col * V), v);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = c0 + channel_of<T, false>(col, i);
            if (c < D) row[c] = from_f32<T>(x[i]);
        }
    }
}

// R: tokens of a thread. CLUSTER: the cluster has more than one CTA.
template <typename T, bool ALIGNED, bool BWD, int R, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, 2) recurrence_scan_kernel(RecurrenceArgs a, int slices) {
    constexpr int V = Pack<T>::V, CT = 8 * V, TILE = kGroups * R;
    __shared__ float2 s_warp[kWarps][CT];                               // a warp's span, then what enters it from the CTA's start
    __shared__ float2 s_cta[CLUSTER ? 2 : 1][CLUSTER ? kMaxCluster : 1][CT];  // the CTAs' spans, by parity of the tile
    __shared__ float s_in[CT];                                          // the state that enters this CTA's tile
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, col = lane & 7, group = tid >> 3;
    int rank = 0, size = 1;
    long long id = blockIdx.x;
    if constexpr (CLUSTER) {
        const cg::cluster_group cl = cg::this_cluster();
        rank = (int)cl.block_rank();
        size = (int)cl.num_blocks();
        id /= size;
    }
    const int n = (int)(id / slices), c0 = (int)(id % slices) * CT, D = a.D;
    long long begin;
    int len;
    token_range(a.cu_seqlens, n, a.T, begin, len);
    const T *la = (const T*)a.log_alpha + begin * D, *x = (const T*)a.x + begin * D;
    const T* hf = BWD ? (const T*)a.h_fwd + begin * D : nullptr;
    T* out = (T*)a.out + begin * D;
    T* out_la = BWD ? (T*)a.out_la + begin * D : nullptr;

    // Threads tid < CT keep the state of channel c0 + tid between tiles.
    const bool keeps = tid < CT && c0 + tid < D;
    float state = keeps && a.state0 ? a.state0[(long long)n * D + c0 + tid] : 0.f;
    if constexpr (CLUSTER) cg::this_cluster().sync();  // every CTA has started, and has read its state

    // token of this thread's step i in tile `tile`, in walking order; -1: past the end
    auto token = [&](int tile, int i) {
        const unsigned at = (unsigned)(tile * size + rank) * TILE + group * R + i;  // below len + 8 TILE: no wrap
        return at < (unsigned)len ? (BWD ? len - 1 - (int)at : (int)at) : -1;
    };
    Pack<T> pl[R], px[R], ph[BWD ? R : 1];
    auto fetch = [&](int tile) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int t = token(tile, i);
            const long long row = (long long)max(t, 0) * D;
            pl[i] = load_row<T, ALIGNED>(la + row, c0, col, D, t >= 0);
            px[i] = load_row<T, ALIGNED>(x + row, c0, col, D, t >= 0);
            if constexpr (BWD) ph[i] = load_row<T, ALIGNED>(hf + row - (t > 0 ? D : 0), c0, col, D, t > 0);
        }
    };
    const long long step = (long long)size * TILE;
    const int tiles = (int)((len + step - 1) / step);
    if (tiles > 0) fetch(0);
    for (int tile = 0; tile < tiles; ++tile) {
        Pack<T> cl[R], cx[R], ch[BWD ? R : 1];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            cl[i] = pl[i];
            cx[i] = px[i];
            if constexpr (BWD) ch[i] = ph[i];
        }
        if (tile + 1 < tiles) fetch(tile + 1);
        // this thread's tokens as one span
        float A[V], H[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            A[e] = 1.f;
            H[e] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float d = decay<T>(cl[i].get(e)), v = cx[i].get(e);
                A[e] *= d;
                H[e] = BWD ? d * (H[e] + v) : fmaf(d, H[e], v);
            }
        // composed over the warp's token groups (lanes 8 apart); E: what lies before this group in the warp
        float EA[V], EH[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float pa = __shfl_up_sync(~0u, A[e], 8), pk = __shfl_up_sync(~0u, H[e], 8);
            if (lane >= 8) {
                H[e] = fmaf(A[e], pk, H[e]);
                A[e] *= pa;
            }
            pa = __shfl_up_sync(~0u, A[e], 16);
            pk = __shfl_up_sync(~0u, H[e], 16);
            if (lane >= 16) {
                H[e] = fmaf(A[e], pk, H[e]);
                A[e] *= pa;
            }
            EA[e] = __shfl_up_sync(~0u, A[e], 8);
            EH[e] = __shfl_up_sync(~0u, H[e], 8);
            if (lane < 8) {
                EA[e] = 1.f;
                EH[e] = 0.f;
            }
            if (lane >= 24) s_warp[warp][channel_of<T, ALIGNED>(col, e)] = make_float2(A[e], H[e]);
        }
        __syncthreads();
        if (tid < CT) {
            float2 w[kWarps];
#pragma unroll
            for (int k = 0; k < kWarps; ++k) w[k] = s_warp[k][tid];
            float2 all = make_float2(1.f, 0.f);
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                s_warp[k][tid] = all;
                all = make_float2(all.x * w[k].x, fmaf(w[k].x, all.y, w[k].y));
            }
            if constexpr (CLUSTER) {
                const cg::cluster_group cl_ = cg::this_cluster();
                for (int r = 0; r < size; ++r)
                    *cl_.map_shared_rank(&s_cta[tile & 1][rank][tid], r) = all;
            } else {
                s_in[tid] = state;
                state = fmaf(all.x, state, all.y);
            }
        }
        if constexpr (CLUSTER) {
            cg::this_cluster().sync();
            if (tid < CT) {
                for (int r = 0; r < size; ++r) {
                    if (r == rank) s_in[tid] = state;
                    const float2 w = s_cta[tile & 1][r][tid];
                    state = fmaf(w.x, state, w.y);
                }
            }
        }
        __syncthreads();
        // the tokens again, from the state that enters them
        float s[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const int c = channel_of<T, ALIGNED>(col, e);
            const float2 w = s_warp[warp][c];
            s[e] = fmaf(EA[e], fmaf(w.x, s_in[c], w.y), EH[e]);
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int t = token(tile, i);
            float y[V], z[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float d = decay<T>(cl[i].get(e)), v = cx[i].get(e);
                if constexpr (BWD) {
                    y[e] = s[e] + v;
                    s[e] = d * y[e];
                    float before = ch[i].get(e);
                    if (t == 0) {
                        const int c = c0 + channel_of<T, ALIGNED>(col, e);
                        before = a.h0 && c < D ? a.h0[(long long)n * D + c] : 0.f;
                    }
                    z[e] = s[e] * before;
                } else {
                    y[e] = s[e] = fmaf(d, s[e], v);
                }
            }
            if (t >= 0) {
                store_row<T, ALIGNED>(out + (long long)t * D, c0, col, D, y);
                if constexpr (BWD) store_row<T, ALIGNED>(out_la + (long long)t * D, c0, col, D, z);
            }
        }
        __syncwarp();
    }
    if (keeps && rank == 0 && a.state_end) a.state_end[(long long)n * D + c0 + tid] = state;
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

template <typename T, bool ALIGNED, bool BWD>
cudaError_t launch_scan(const RecurrenceArgs& a, cudaStream_t stream) {
    constexpr int R = BWD ? 2 : 4;
    const int slices = (a.D + 8 * Pack<T>::V - 1) / (8 * Pack<T>::V);
    const long long rows = (long long)a.N * slices;
    // CTAs of a cluster: as many as fill two CTAs on each SM, no more than the tokens give tiles to
    const long long tokens = a.cu_seqlens ? (a.T + a.N - 1) / a.N : a.T;
    int size = 1;
    while (size < kMaxCluster && rows * size * 2 <= 2 * 148 && (long long)size * kGroups * R < tokens) size *= 2;
    if (size == 1) {
        recurrence_scan_kernel<T, ALIGNED, BWD, R, false><<<(unsigned)rows, kThreads, 0, stream>>>(a, slices);
        return cudaGetLastError();
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * size));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = size;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, recurrence_scan_kernel<T, ALIGNED, BWD, R, true>, a, slices);
}

template <bool BWD> cudaError_t launch_scan_any(const RecurrenceArgs& a, cudaStream_t stream) {
    const bool aligned = a.D % (a.bf16 ? 8 : 4) == 0;  // then every row begins on 16 bytes
    if (a.bf16)
        return aligned ? launch_scan<__nv_bfloat16, true, BWD>(a, stream) : launch_scan<__nv_bfloat16, false, BWD>(a, stream);
    return aligned ? launch_scan<float, true, BWD>(a, stream) : launch_scan<float, false, BWD>(a, stream);
}

}  // namespace

cudaError_t launch_recurrence_fwd(const RecurrenceArgs& a, cudaStream_t stream) { return launch_scan_any<false>(a, stream); }
cudaError_t launch_recurrence_bwd(const RecurrenceArgs& a, cudaStream_t stream) { return launch_scan_any<true>(a, stream); }

cudaError_t launch_recurrence_step(const void* la, const void* x, const float* h_in, float* h_out, void* y,
                                   long long cells, int bf16, cudaStream_t stream) {
    auto go = [&](auto t) {
        using T = decltype(t);
        recurrence_step_kernel<T><<<(unsigned)((cells + 127) / 128), 128, 0, stream>>>((const T*)la, (const T*)x, h_in, h_out,
                                                                                      (T*)y, cells);
        return cudaGetLastError();
    };
    return bf16 ? go(__nv_bfloat16()) : go(float());
}

}  // namespace kda
