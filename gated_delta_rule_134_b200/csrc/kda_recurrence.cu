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
// slice of 128 bytes of channels) and walks the tokens, a tile of tokens per CTA
// at a time. A thread has R consecutive tokens of 16 bytes of channels; it copies
// them into shared memory two tiles ahead (it alone reads them back, so no
// barrier is due) and then
//   1. composes its tokens into one span (A, H) and leaves it in shared memory;
//   2. as (channel, part) composes the spans of one part of the CTA's token
//      groups, then the parts' spans, and leaves the CTA's to the cluster;
//   3. walks the CTAs and parts before its own, which gives the state that enters
//      each of its groups, and leaves these in shared memory;
//   4. runs its tokens again from the state that enters them and writes them.
// The sequential depth is T / (tokens of a cluster's tile). Nothing waits on a
// flag, and the order of every product and sum is fixed by the sizes alone.
#include "kda_async.cuh"
#include "kda_common.cuh"
#include "kda_internal.h"

#include <cooperative_groups.h>

namespace kda {

namespace {

namespace cg = cooperative_groups;

constexpr int kTokens = 4;  // of a thread
constexpr int kMaxCluster = 16;  // above 8 a device may refuse a cluster size: B200 takes 16

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
    static __device__ __forceinline__ Pack of(const uint4& v) {
        Pack p;
        p.w[0] = v.x; p.w[1] = v.y; p.w[2] = v.z; p.w[3] = v.w;
        return p;
    }
};

// e^x. For bf16 inputs 2^(x log2 e), off by 2^-22 for |x| < 1: far below the input's own step.
template <typename T> __device__ __forceinline__ float decay(float x);
template <> __device__ __forceinline__ float decay<float>(float x) { return expf(x); }
template <> __device__ __forceinline__ float decay<__nv_bfloat16>(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
    return y;
}

// ALIGN: what every row's first byte is a multiple of, 16, 4 or (bf16 alone) 2. It sets a thread's channels within the
// slice: 16 bytes at once; else 4-byte words eight apart, so that the eight threads of a token group touch neighbouring
// words.
template <typename T, int ALIGN> __device__ __forceinline__ int channel_of(int col, int e) {
    constexpr int V = Pack<T>::V, P = 4 / sizeof(T);  // elements of a word
    return ALIGN == 16 ? col * V + e : (col + 8 * (e / P)) * P + e % P;
}

__device__ __forceinline__ void cp_async4(void* dst, const void* src, bool on) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src), "r"(on ? 4 : 0)
                 : "memory");
}

// One row's channels of this thread; zeros where `on` is false or past the last channel.
template <typename T, int ALIGN>
__device__ __forceinline__ Pack<T> read_row(const T* row, int c0, int col, int D, bool on) {
    constexpr int P = 4 / sizeof(T);
    Pack<T> r;
    r.w[0] = r.w[1] = r.w[2] = r.w[3] = 0u;
    if constexpr (ALIGN == 16) {
        const int c = c0 + col * Pack<T>::V;
        if (on && c < D) r = Pack<T>::of(__ldcs(reinterpret_cast<const uint4*>(row + c)));
    } else if constexpr (ALIGN == 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = c0 + (col + 8 * j) * P;
            if (on && c < D) r.w[j] = __ldcs(reinterpret_cast<const unsigned*>(row + c));
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = c0 + channel_of<T, ALIGN>(col, e);
            if (on && c < D) r.w[e >> 1] |= (uint32_t)__ldcs(reinterpret_cast<const unsigned short*>(row) + c) << (e & 1 ? 16 : 0);
        }
    }
    return r;
}

// Stage `slot` ([token of the tile][32 words], then one more word a token) gets this warp's 4 R tokens of one tensor,
// without waiting. `first`: the row of the CTA's first token; `step`: from a token to the next (D or -D); `left`: the
// number of tokens there are. With 16-byte rows every thread copies what it will read; else a warp copies one token's 32
// words at a time, because copies that touch four rows at once are bound by the load unit (the readers then need
// __syncwarp). Words are swizzled by token group, so that the four groups of a warp read different banks. Rows that
// begin in the middle of a word (ALIGN 2, every other row) are copied from that word on, 33 words, and shifted by the
// reader; a word that reaches past the tensor's end `stop` is read by halves.
template <typename T, int ALIGN, int R, int THREADS>
__device__ __forceinline__ void copy_tile(uint32_t* slot, const T* first, int step, int left, int c0, int D, const T* stop) {
    constexpr int P = 4 / sizeof(T);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = lane & 7;
    if constexpr (ALIGN == 16) {
        const int k0 = (threadIdx.x >> 3) * R, c = c0 + col * Pack<T>::V;
#pragma unroll
        for (int i = 0; i < R; ++i)
            cp_async16(reinterpret_cast<uint4*>(slot) + i * THREADS + threadIdx.x, first + (long long)(k0 + i) * step + c,
                       k0 + i < left && c < D);
        return;
    }
    const int k0 = warp * 4 * R;
    uint32_t* to = slot + k0 * 32;
    left -= k0;
    if constexpr (ALIGN == 4) {
        const int c = c0 + lane * P;
        if (c >= D) left = 0;
        const T* row = first + (long long)k0 * step + c;
#pragma unroll
        for (int k = 0; k < 4 * R; ++k, row += step) cp_async4(to + k * 32 + (lane ^ (8 * (k / R))), row, k < left);
    } else {
        const int n = min(D - c0, 64);
        const char* at = reinterpret_cast<const char*>(first + (long long)k0 * step + c0);
        // the word that holds the tensor's last element may lie in this warp's rows
        const char* last = step > 0 ? at + 2ll * step * (min(left, 4 * R) - 1) : at;
        const bool ends = left > 0 && last + 4 * 33 > reinterpret_cast<const char*>(stop);
        const int left0 = 2 * lane < n ? left : 0, left1 = 2 * lane - 1 < n ? left : 0;  // rows that need this lane's word
        {
            const char* mine = at + 2ll * step * lane;  // lane k: the 33rd word of row k
            if (lane < 4 * R && (reinterpret_cast<uintptr_t>(mine) & 2)) {
                const char* w = mine - 2 + 128;
                const bool on = lane < left && n == 64;
                uint32_t* dst = slot + THREADS / 8 * R * 32 + k0 + lane;
                if (on && w + 4 > reinterpret_cast<const char*>(stop)) *dst = *reinterpret_cast<const unsigned short*>(w);
                else cp_async4(dst, w, on);
            }
        }
        if (!ends) {
#pragma unroll
            for (int k = 0; k < 4 * R; ++k, at += 2ll * step) {
                const uintptr_t w = reinterpret_cast<uintptr_t>(at);
                cp_async4(to + k * 32 + (lane ^ (8 * (k / R))), reinterpret_cast<const char*>(w & ~(uintptr_t)2) + 4 * lane,
                          k < (w & 2 ? left1 : left0));
            }
        } else {
#pragma unroll 1
            for (int k = 0; k < 4 * R; ++k, at += 2ll * step) {
                const uintptr_t w = reinterpret_cast<uintptr_t>(at);
                const char* from = reinterpret_cast<const char*>(w & ~(uintptr_t)2) + 4 * lane;
                const bool on = k < (w & 2 ? left1 : left0);
                uint32_t* dst = to + k * 32 + (lane ^ (8 * (k / R)));
                if (on && from + 4 > reinterpret_cast<const char*>(stop)) *dst = *reinterpret_cast<const unsigned short*>(from);
                else cp_async4(dst, from, on);
            }
        }
    }
}
// This thread's channels of its token i; `odd`: the row begins in the middle of a word.
template <typename T, int ALIGN, int R, int THREADS> __device__ __forceinline__ Pack<T> slot_of(const uint32_t* slot, int i, bool odd) {
    if constexpr (ALIGN == 16) return Pack<T>::of(reinterpret_cast<const uint4*>(slot)[i * THREADS + threadIdx.x]);
    const int col = threadIdx.x & 7, group = threadIdx.x >> 3, turn = 8 * (group & 3);
    const uint32_t* at = slot + (group * R + i) * 32;
    Pack<T> r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int k = col + 8 * j;
        r.w[j] = at[k ^ turn];
        if constexpr (ALIGN == 2) {
            if (odd) r.w[j] = __funnelshift_r(r.w[j], k == 31 ? slot[THREADS / 8 * R * 32 + group * R + i] : at[(k + 1) ^ turn], 16);
        }
    }
    return r;
}

template <typename T, int ALIGN>
__device__ __forceinline__ void store_row(T* row, int c0, int col, int D, const float (&x)[Pack<T>::V]) {
    constexpr int V = Pack<T>::V, P = 4 / sizeof(T);
    if constexpr (ALIGN == 2) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const int c = c0 + channel_of<T, ALIGN>(col, e);
            if (c < D) row[c] = from_f32<T>(x[e]);
        }
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (V == 4) {
                w[i] = __float_as_uint(x[i]);
            } else {
                const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&b);
            }
        }
        if constexpr (ALIGN == 16) {
            if (c0 + col * V < D) __stcs(reinterpret_cast<uint4*>(row + c0 + col * V), make_uint4(w[0], w[1], w[2], w[3]));
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = c0 + (col + 8 * j) * P;
                if (c < D) *reinterpret_cast<uint32_t*>(row + c) = w[j];
            }
        }
    }
}

// Shared memory: the ring of stages, the spans of the token groups, the states that enter them, and the spans of the
// parts of all CTAs of the cluster, by parity of the tile.
template <typename T, int R, int THREADS> struct ScanSmem {
    static constexpr int kGroups = THREADS / 8;             // token groups of a CTA (8 threads across the channels)
    static constexpr int CT = 8 * Pack<T>::V;              // channels of a slice
    static constexpr int kParts = THREADS / CT, kPer = kGroups / kParts;
    static constexpr int kSlot = R * THREADS * 16 + kGroups * R * 4;  // one tensor's tile, and a word more a token
    static constexpr int kStage = 2 * kSlot, kStages = 2;
    static constexpr int kSpans = kGroups * CT * (int)sizeof(float2), kStates = kGroups * CT * (int)sizeof(float);
    static constexpr int kBytes = kStages * kStage + kSpans + kStates + (kParts + 2) * CT * (int)sizeof(float2);
};

// A cluster barrier that publishes this thread's writes to its own CTA's shared memory, and them alone: the full
// release would wait for the tile's stores to global memory, 1.5 us.
__device__ __forceinline__ void cluster_exchange() {
    asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
}

// R: tokens of a thread. CLUSTER: the cluster has more than one CTA.
template <typename T, int ALIGN, bool BWD, int R, int THREADS, bool CLUSTER>
__global__ void __launch_bounds__(THREADS, 512 / THREADS) recurrence_scan_kernel(RecurrenceArgs a, int slices) {
    using Sm = ScanSmem<T, R, THREADS>;
    constexpr int V = Pack<T>::V, CT = Sm::CT, TILE = Sm::kGroups * R, PARTS = Sm::kParts, PER = Sm::kPer, S = Sm::kStages;
    extern __shared__ __align__(16) unsigned char smem[];
    uint32_t* ring = reinterpret_cast<uint32_t*>(smem);
    float4* spans = reinterpret_cast<float4*>(smem + S * Sm::kStage);                  // [group][pair of V/2][col]: A, H, A, H
    float* states = reinterpret_cast<float*>(smem + S * Sm::kStage + Sm::kSpans);      // [group][quad of V/4][col][4]
    float2* parts = reinterpret_cast<float2*>(smem + S * Sm::kStage + Sm::kSpans + Sm::kStates);  // [part][channel]
    float2* whole_of = parts + PARTS * CT;  // [parity][channel]: the CTA's span, read by the cluster
    const int tid = threadIdx.x, col = tid & 7, group = tid >> 3;
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

    // As (channel, part): channel p in the order of `spans`, that is element e = 2 pair + half of thread column pcol. Every
    // part keeps the channel's state, by the same operations.
    const int p = tid % CT, part = tid / CT, pair = p / 16, pcol = p % 16 / 2, half = p % 2;
    const int pc = c0 + channel_of<T, ALIGN>(pcol, 2 * pair + half);
    float state = pc < D && a.state0 ? a.state0[(long long)n * D + pc] : 0.f;
    if constexpr (CLUSTER) cg::this_cluster().sync();  // every CTA has started, and has read its state

    // token k of this CTA's tile `tile`, in walking order; -1: past the end
    auto token = [&](int tile, int k) {
        const unsigned at = (unsigned)(tile * size + rank) * TILE + k;  // below len + 16 TILE: no wrap
        return at < (unsigned)len ? (BWD ? len - 1 - (int)at : (int)at) : -1;
    };
    constexpr int kSlot = Sm::kSlot / 4;
    // the end of the tensors, for ALIGN 2
    const long long cells = (a.cu_seqlens ? 1ll : (long long)a.N) * a.T * D;
    const T *la_stop = (const T*)a.log_alpha + cells, *x_stop = (const T*)a.x + cells;
    auto fetch = [&](int tile) {
        uint32_t* to = ring + (tile & 1) * 2 * kSlot;
        const long long at = (long long)(tile * size + rank) * TILE;
        const int left = (int)min(max(len - at, 0ll), (long long)TILE);
        const long long row = (BWD ? len - 1 - at : at) * D;
        copy_tile<T, ALIGN, R, THREADS>(to, la + row, BWD ? -D : D, left, c0, D, la_stop);
        copy_tile<T, ALIGN, R, THREADS>(to + kSlot, x + row, BWD ? -D : D, left, c0, D, x_stop);
    };
    const long long step = (long long)size * TILE;
    const int tiles = (int)((len + step - 1) / step);
    for (int k = 0; k < S; ++k) {
        if (k < tiles) fetch(k);
        cp_async_commit();
    }
    for (int tile = 0; tile < tiles; ++tile) {
        // 1. this thread's tokens as one span
        cp_async_wait<S - 1>();
        if constexpr (ALIGN != 16) __syncwarp();
        F2 d[R][V / 2], A[V / 2], H[V / 2];
        Pack<T> px[R], ph[BWD ? R : 1];
        if constexpr (BWD) {  // h_{t-1}: read now, used at the tile's end
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int t = token(tile, group * R + i);
                ph[i] = read_row<T, ALIGN>(hf + (long long)max(t - 1, 0) * D, c0, col, D, t > 0);
            }
        }
        {
            const uint32_t* from = ring + (tile & 1) * 2 * kSlot;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                // D is odd and the tensors begin on 16 bytes: every other row begins in the middle of a word
                // (those past the end, which hold zeros, counted on: the copy goes by the same rows)
                const unsigned at = (unsigned)(tile * size + rank) * TILE + group * R + i;
                const bool odd = ALIGN == 2 && (((unsigned)begin + (BWD ? len - 1 - at : at)) & 1);
                const Pack<T> pl = slot_of<T, ALIGN, R, THREADS>(from, i, odd);
                px[i] = slot_of<T, ALIGN, R, THREADS>(from + kSlot, i, odd);
#pragma unroll
                for (int e = 0; e < V / 2; ++e) {
                    d[i][e] = f2(decay<T>(pl.get(2 * e)), decay<T>(pl.get(2 * e + 1)));
                    const F2 v = f2(px[i].get(2 * e), px[i].get(2 * e + 1));
                    if (i == 0) {
                        A[e] = d[i][e];
                        H[e] = BWD ? f2_mul(d[i][e], v) : v;
                    } else {
                        A[e] = f2_mul(A[e], d[i][e]);
                        H[e] = BWD ? f2_mul(d[i][e], f2_add(H[e], v)) : f2_fma(d[i][e], H[e], v);
                    }
                }
            }
        }
        if constexpr (ALIGN != 16) __syncwarp();
        if (tile + S < tiles) fetch(tile + S);
        cp_async_commit();
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
            const float2 A_ = f2_parts(A[e]), H_ = f2_parts(H[e]);
            spans[(group * (V / 2) + e) * 8 + col] = make_float4(A_.x, H_.x, A_.y, H_.y);
        }
        __syncthreads();
        // 2. as (channel, part): the part's span, the CTA's
        float2 w[PER];
#pragma unroll
        for (int k = 0; k < PER; ++k)
            w[k] = reinterpret_cast<const float2*>(spans)[((part * PER + k) * (V / 2) + pair) * 16 + pcol * 2 + half];
        float2 all = w[0];
#pragma unroll
        for (int k = 1; k < PER; ++k) all = make_float2(all.x * w[k].x, fmaf(w[k].x, all.y, w[k].y));
        parts[part * CT + p] = all;
        __syncthreads();
        float2 before = make_float2(1.f, 0.f), whole = before;  // of the CTA's parts: those before this one, all
#pragma unroll
        for (int k = 0; k < PARTS; ++k) {
            const float2 u = parts[k * CT + p];
            if (k == part) before = whole;
            whole = make_float2(whole.x * u.x, fmaf(u.x, whole.y, u.y));
        }
        // 3. the state that enters this part's groups; the state after the cluster's tile
        float s = state;
        if constexpr (CLUSTER) {
            float2* mine = whole_of + (tile & 1) * CT + p;
            if (part == 0) *mine = whole;
            cluster_exchange();
            for (int r0 = 0; r0 < size; r0 += 8) {
                float2 u[8];
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (r0 + r < size) u[r] = *cg::this_cluster().map_shared_rank(mine, r0 + r);
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (r0 + r < size) {
                        if (r0 + r == rank) s = state;
                        state = fmaf(u[r].x, state, u[r].y);
                    }
            }
        } else {
            state = fmaf(whole.x, state, whole.y);
        }
        s = fmaf(before.x, s, before.y);
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            states[(((part * PER + k) * (V / 4) + pair / 2) * 8 + pcol) * 4 + (pair & 1) * 2 + half] = s;
            s = fmaf(w[k].x, s, w[k].y);
        }
        __syncthreads();
        // 4. the tokens again, from the state that enters them
        F2 cur[V / 2];
#pragma unroll
        for (int q = 0; q < V / 4; ++q) {
            const float4 v = reinterpret_cast<const float4*>(states)[(group * (V / 4) + q) * 8 + col];
            cur[2 * q] = f2(v.x, v.y);
            cur[2 * q + 1] = f2(v.z, v.w);
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int t = token(tile, group * R + i);
            float y[V], z[V];
#pragma unroll
            for (int e = 0; e < V / 2; ++e) {
                const F2 v = f2(px[i].get(2 * e), px[i].get(2 * e + 1));
                F2 o;
                if constexpr (BWD) {
                    o = f2_add(cur[e], v);
                    cur[e] = f2_mul(d[i][e], o);
                    float b0 = ph[i].get(2 * e), b1 = ph[i].get(2 * e + 1);
                    if (t == 0) {
                        const int e0 = c0 + channel_of<T, ALIGN>(col, 2 * e), e1 = c0 + channel_of<T, ALIGN>(col, 2 * e + 1);
                        b0 = a.h0 && e0 < D ? a.h0[(long long)n * D + e0] : 0.f;
                        b1 = a.h0 && e1 < D ? a.h0[(long long)n * D + e1] : 0.f;
                    }
                    const float2 zz = f2_parts(f2_mul(cur[e], f2(b0, b1)));
                    z[2 * e] = zz.x;
                    z[2 * e + 1] = zz.y;
                } else {
                    o = cur[e] = f2_fma(d[i][e], cur[e], v);
                }
                const float2 yy = f2_parts(o);
                y[2 * e] = yy.x;
                y[2 * e + 1] = yy.y;
            }
            if (t >= 0) {
                store_row<T, ALIGN>(out + (long long)t * D, c0, col, D, y);
                if constexpr (BWD) store_row<T, ALIGN>(out_la + (long long)t * D, c0, col, D, z);
            }
        }
    }
    cp_async_wait<0>();
    if constexpr (CLUSTER) cg::this_cluster().sync();  // no CTA ends while another reads its shared memory
    if (part == 0 && rank == 0 && pc < D && a.state_end) a.state_end[(long long)n * D + pc] = state;
}

// One token: four cells a thread, 16 bytes of state (the tensors are contiguous, so their rows do not matter).
template <typename T>
__global__ void __launch_bounds__(256) recurrence_step_kernel(const T* log_alpha, const T* x, const float* h_in, float* h_out, T* y,
                                                              long long cells) {
    const long long i = ((long long)blockIdx.x * blockDim.x + threadIdx.x) * 4;
    if (i + 4 <= cells) {
        float la[4], v[4];
        if constexpr (sizeof(T) == 4) {
            const float4 l4 = *reinterpret_cast<const float4*>(log_alpha + i), x4 = *reinterpret_cast<const float4*>(x + i);
            la[0] = l4.x; la[1] = l4.y; la[2] = l4.z; la[3] = l4.w;
            v[0] = x4.x; v[1] = x4.y; v[2] = x4.z; v[3] = x4.w;
        } else {
            const uint2 l2 = *reinterpret_cast<const uint2*>(log_alpha + i), x2 = *reinterpret_cast<const uint2*>(x + i);
            const uint32_t l[2] = {l2.x, l2.y}, w[2] = {x2.x, x2.y};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                la[e] = __uint_as_float(e & 1 ? l[e >> 1] & 0xffff0000u : l[e >> 1] << 16);
                v[e] = __uint_as_float(e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
            }
        }
        const float4 h = *reinterpret_cast<const float4*>(h_in + i);
        const float4 s = make_float4(fmaf(expf(la[0]), h.x, v[0]), fmaf(expf(la[1]), h.y, v[1]), fmaf(expf(la[2]), h.z, v[2]),
                                     fmaf(expf(la[3]), h.w, v[3]));
        *reinterpret_cast<float4*>(h_out + i) = s;
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<float4*>(y + i) = s;
        } else {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(s.x, s.y), hi = __floats2bfloat162_rn(s.z, s.w);
            *reinterpret_cast<uint2*>(y + i) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
        }
        return;
    }
    for (long long k = i; k < cells; ++k) {
        const float s = fmaf(expf(to_f32(log_alpha[k])), h_in[k], to_f32(x[k]));
        h_out[k] = s;
        y[k] = from_f32<T>(s);
    }
}

template <typename T, int ALIGN, bool BWD, int THREADS, bool CLUSTER>
cudaError_t launch_scan_as(const RecurrenceArgs& a, int slices, int size, cudaStream_t stream) {
    using Sm = ScanSmem<T, kTokens, THREADS>;
    auto kernel = recurrence_scan_kernel<T, ALIGN, BWD, kTokens, THREADS, CLUSTER>;
    static std::atomic<unsigned long long> raised{0};
    cudaError_t err = size > 8 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) : cudaSuccess;
    if (err == cudaSuccess) err = allow_smem(kernel, Sm::kBytes, raised);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)a.N * slices * size));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = Sm::kBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = size;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = CLUSTER ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a, slices);
}

template <typename T, int ALIGN, bool BWD>
cudaError_t launch_scan(const RecurrenceArgs& a, cudaStream_t stream) {
    constexpr int CT = 8 * Pack<T>::V;
    const int slices = (a.D + CT - 1) / CT;
    const long long rows = (long long)a.N * slices;
    const long long tokens = a.cu_seqlens ? (a.T + a.N - 1) / a.N : a.T;
    // CTAs of a cluster: one from 75 rows on (128 rows, T 8192 backward: 127 us, with two 131; 96 rows, T 4096: 36 and
    // 44); below, as many as fill two CTAs on each SM, so that one computes while the other exchanges (64 rows, T 4096:
    // 24 us with four, 31 with two, 40 with one), no more than the tokens give tiles to; sixteen only where all clusters
    // of them fit at once (T 16384: six rows 27 us, with eight 34; eight rows 37 and 34).
    int size = 1;
    while (rows < 75 && size < (rows <= 6 ? kMaxCluster : 8) && rows * size * 2 <= 2 * 148 &&
           (long long)size * (256 / 8) * kTokens < tokens)
        size *= 2;
    if (size > 1) return launch_scan_as<T, ALIGN, BWD, 256, true>(a, slices, size, stream);
    // One CTA of 512 threads on an SM takes tiles of twice the tokens, and its SM's share of the bandwidth with fewer
    // barriers: 256 rows, T 8192 132 us (two CTAs of 256 threads: 150); 96 rows, T 4096 backward 51 (65). It pays where
    // the rows fill their rounds of 148 (192 rows: 67 us against 57) and there are tokens enough (T 200: 7.4 against 5.8).
    const long long rounds = (rows + 147) / 148;
    if (tokens >= 512 && (rounds == 1 || rows * 5 >= rounds * 148 * 4)) return launch_scan_as<T, ALIGN, BWD, 512, false>(a, slices, 1, stream);
    return launch_scan_as<T, ALIGN, BWD, 256, false>(a, slices, 1, stream);
}

template <bool BWD> cudaError_t launch_scan_any(const RecurrenceArgs& a, cudaStream_t stream) {
    const long long row = (long long)a.D * (a.bf16 ? 2 : 4);  // bytes of a row: the first begins on 16
    if (a.bf16) {
        if (row % 16 == 0) return launch_scan<__nv_bfloat16, 16, BWD>(a, stream);
        return row % 4 == 0 ? launch_scan<__nv_bfloat16, 4, BWD>(a, stream) : launch_scan<__nv_bfloat16, 2, BWD>(a, stream);
    }
    return row % 16 == 0 ? launch_scan<float, 16, BWD>(a, stream) : launch_scan<float, 4, BWD>(a, stream);
}

}  // namespace

cudaError_t launch_recurrence_fwd(const RecurrenceArgs& a, cudaStream_t stream) { return launch_scan_any<false>(a, stream); }
cudaError_t launch_recurrence_bwd(const RecurrenceArgs& a, cudaStream_t stream) { return launch_scan_any<true>(a, stream); }

cudaError_t launch_recurrence_step(const void* la, const void* x, const float* h_in, float* h_out, void* y,
                                   long long cells, int bf16, cudaStream_t stream) {
    auto go = [&](auto t) {
        using T = decltype(t);
        // 64 threads a block for few cells, so that they meet all SMs
        const int threads = cells < 148ll * 1024 ? 64 : 256;
        const long long blocks = (cells + threads * 4 - 1) / (threads * 4);
        recurrence_step_kernel<T><<<(unsigned)blocks, threads, 0, stream>>>((const T*)la, (const T*)x, h_in, h_out, (T*)y, cells);
        return cudaGetLastError();
    };
    return bf16 ? go(__nv_bfloat16()) : go(float());
}

}  // namespace kda
