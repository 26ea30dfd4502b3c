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
// channel, each read or written once. A row is a (sequence, slice of 128 bytes of
// channels); one CTA walks its tokens, a tile at a time. A thread has kTokens
// consecutive tokens of 16 bytes of channels; it copies them into shared memory
// two tiles ahead (with 16-byte rows it alone reads them back, so no barrier is
// due) and then
//   1. composes its tokens into one span (A, H) and leaves it in shared memory;
//   2. as (channel, part) composes the spans of one part of the CTA's token
//      groups, then the parts' spans;
//   3. walks the parts before its own, which gives the state that enters each of
//      its groups, and leaves these in shared memory;
//   4. runs its tokens again from the state that enters them and writes them.
// B4 T8192 D4096 bf16 takes 134-139 us, by the B200 (0.90-0.93 of the measured copy
// bandwidth), the backward pass of B2 114-117 us (0.89-0.91). Where rows are few, a
// cluster of CTAs shares one (recurrence_cluster_kernel). The order of every product and sum is
// fixed by the sizes alone.
#include "kda_async.cuh"
#include "kda_common.cuh"
#include "kda_internal.h"
#include "kda_sm100.cuh"

#include <cooperative_groups.h>

namespace kda {

namespace {

namespace cg = cooperative_groups;

constexpr int kTokens = 4;  // of a thread
constexpr int kMaxCluster = 16;  // above 8 a device may refuse a cluster size: B200 takes 16

// Set where a wait gave up.
__device__ unsigned g_recurrence_late;

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

// e^x. For bf16 inputs 2^(x log2 e) by one instruction. All of them tried, it is as near as expf for |x| < 1 (both 1.9 times
// 2^-24 off at most, 1.4 for |x| < 2^-8: slow decays over long sequences lose nothing); beyond that the roundings of log2 e
// and of the product count, at most 2 |x| 2^-24 of a decay that is small then. With expf the forward pass of B4 T8192 D4096
// takes 148 us, so 134.
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

// At most `bytes` of the 16 at `src`, zeros for the rest.
__device__ __forceinline__ void cp_async16_some(void* dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src), "r"(bytes)
                 : "memory");
}

// One row's channels of this thread as row_of returns them; zeros where `on` is false or past the last channel. Loading
// and shifting are apart, so that the loads can be under way. Rows that are even in 2-byte elements alone are read by the
// words that lie on 4 bytes: where the row begins within such a word, the thread has the second half of what it needs
// from the next lane, the last lane's very last from a load of its own. (By 2-byte loads and stores the backward pass of
// T16384 D1001 bf16 takes 251 us, so 149; the forward pass 94 and 84.)
template <typename T, int ALIGN> struct RowWords {
    Pack<T> p;
    uint32_t last;
};
template <typename T, int ALIGN>
__device__ __forceinline__ RowWords<T, ALIGN> read_row(const T* row, int c0, int col, int D, bool on) {
    constexpr int P = 4 / sizeof(T);
    RowWords<T, ALIGN> r;
    r.p.w[0] = r.p.w[1] = r.p.w[2] = r.p.w[3] = r.last = 0u;
    if constexpr (ALIGN == 16) {
        const int c = c0 + col * Pack<T>::V;
        if (on && c < D) r.p = Pack<T>::of(__ldcs(reinterpret_cast<const uint4*>(row + c)));
    } else if constexpr (ALIGN == 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = c0 + (col + 8 * j) * P;
            if (on && c < D) r.p.w[j] = __ldcs(reinterpret_cast<const unsigned*>(row + c));
        }
    } else {
        // the tensor begins on 4 bytes: a row that does not has an element before it
        const int odd = (int)(reinterpret_cast<uintptr_t>(row) >> 1 & 1);
        const unsigned short* half = reinterpret_cast<const unsigned short*>(row);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = c0 + (col + 8 * j) * P - odd;
            if (on && c + 1 < D) r.p.w[j] = __ldcs(reinterpret_cast<const unsigned*>(half + c));
            else if (on && c < D) r.p.w[j] = __ldcs(half + c);
        }
        if (on && odd && col == 7 && c0 + 63 < D) r.last = __ldcs(half + c0 + 63);
    }
    return r;
}
// Called by all lanes.
template <typename T, int ALIGN> __device__ __forceinline__ Pack<T> row_of(const RowWords<T, ALIGN>& r, const T* row, int col) {
    if constexpr (ALIGN != 2) return r.p;
    const int shift = (int)(reinterpret_cast<uintptr_t>(row) & 2) * 8;
    Pack<T> p;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t give = col == 0 ? (j < 3 ? r.p.w[(j + 1) & 3] : 0u) : r.p.w[j];
        uint32_t next = __shfl_sync(0xffffffffu, give, (col + 1) & 7, 8);
        if (j == 3 && col == 7) next = r.last;
        p.w[j] = __funnelshift_r(r.p.w[j], next, shift);
    }
    return p;
}

// The bytes of one tensor's tile in shared memory. With 16-byte rows: [token of a thread][thread], 16 bytes each. Else
// every token has the nine 16-byte pieces that its 128 bytes may touch; the token groups lie 32 bytes further apart, so
// that the four of a warp read different banks.
constexpr int kRowPieces = 9;
template <int ALIGN, int R> constexpr int group_bytes() { return ALIGN == 16 ? R * 8 * 16 : R * kRowPieces * 16 + 32; }

// Copies this warp's 4 R tokens of one tensor into its tile, without waiting. `first`: the row of the CTA's first token;
// `step`: from a token to the next (D or -D); `left`: the number of tokens there are; tokens past them become zeros. With
// 16-byte rows every thread copies what it will read; else the lanes share the pieces of all rows, begin each row at the
// 16 bytes that hold its first element, and stop at the tensor's end (the readers then need __syncwarp).
template <typename T, int ALIGN, int R, int THREADS>
__device__ __forceinline__ void copy_tile(unsigned char* slot, const T* first, int step, int left, int c0, int D, const T* stop) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if constexpr (ALIGN == 16) {
        const int k0 = (threadIdx.x >> 3) * R, c = c0 + (lane & 7) * Pack<T>::V;
#pragma unroll
        for (int i = 0; i < R; ++i)
            cp_async16(slot + (i * THREADS + threadIdx.x) * 16, first + (long long)(k0 + i) * step + c, k0 + i < left && c < D);
    } else {
        const int bytes = min(D - c0, (int)(128 / sizeof(T))) * (int)sizeof(T);
        auto copy = [&](int k, int piece) {  // k: token of the CTA's tile
            const uintptr_t row = reinterpret_cast<uintptr_t>(first + (long long)k * step + c0);
            const uintptr_t from = (row & ~(uintptr_t)15) + piece * 16;
            int n = k < left && piece * 16 < (int)(row & 15) + bytes ? 16 : 0;
            if (n && from + 16 > reinterpret_cast<uintptr_t>(stop)) n = (int)(reinterpret_cast<uintptr_t>(stop) - from);
            cp_async16_some(slot + (k / R) * group_bytes<ALIGN, R>() + (k % R * kRowPieces + piece) * 16, reinterpret_cast<const void*>(from), n);
        };
        // a token group's eight lanes take the first eight pieces of its rows, then the warp's lanes a ninth piece each
#pragma unroll
        for (int i = 0; i < R; ++i) copy((threadIdx.x >> 3) * R + i, lane & 7);
        static_assert(4 * R <= 32);
        if (lane < 4 * R) copy(warp * 4 * R + lane, 8);
    }
}
// This thread's channels of its token i; `off`: the row's first byte modulo 16.
template <typename T, int ALIGN, int R, int THREADS> __device__ __forceinline__ Pack<T> slot_of(const unsigned char* slot, int i, int off) {
    if constexpr (ALIGN == 16) return Pack<T>::of(reinterpret_cast<const uint4*>(slot)[i * THREADS + threadIdx.x]);
    const int col = threadIdx.x & 7, group = threadIdx.x >> 3;
    const uint32_t* at = reinterpret_cast<const uint32_t*>(slot + group * group_bytes<ALIGN, R>() + i * kRowPieces * 16) + (off >> 2) + col;
    Pack<T> r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        r.w[j] = at[8 * j];
        if constexpr (ALIGN == 2) r.w[j] = __funnelshift_r(r.w[j], at[8 * j + 1], off & 2 ? 16 : 0);
    }
    return r;
}

// Writes this thread's channels of a row, where `on`. Called by all lanes.
template <typename T, int ALIGN>
__device__ __forceinline__ void store_row(T* row, int c0, int col, int D, bool on, const float (&x)[Pack<T>::V]) {
    constexpr int V = Pack<T>::V, P = 4 / sizeof(T);
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
        if (on && c0 + col * V < D) __stcs(reinterpret_cast<uint4*>(row + c0 + col * V), make_uint4(w[0], w[1], w[2], w[3]));
    } else if constexpr (ALIGN == 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = c0 + (col + 8 * j) * P;
            if (on && c < D) *reinterpret_cast<uint32_t*>(row + c) = w[j];
        }
    } else {
        const int odd = (int)(reinterpret_cast<uintptr_t>(row) >> 1 & 1);
        unsigned short* half = reinterpret_cast<unsigned short*>(row);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t give = col == 7 ? (j > 0 ? w[(j + 3) & 3] : 0u) : w[j];
            const uint32_t before = __shfl_sync(0xffffffffu, give, (col + 7) & 7, 8);
            const uint32_t v = odd ? __funnelshift_l(before, w[j], 16) : w[j];
            const int c = c0 + (col + 8 * j) * P - odd;
            if (!on || c >= D) continue;
            if (c < c0) half[c0] = (unsigned short)(v >> 16);  // the word's first half is another slice's or row's
            else if (c + 1 < D) *reinterpret_cast<uint32_t*>(half + c) = v;
            else half[c] = (unsigned short)v;
        }
        if (on && odd && col == 7 && c0 + 63 < D) half[c0 + 63] = (unsigned short)(w[3] >> 16);
    }
}

// Sizes, and shared memory: the ring of STAGES stages, the spans of the token groups, the states that enter them
// (STATES copies), the spans of the CTA's parts, and the CTA's span by parity of the tile.
template <typename T, int ALIGN, int R, int THREADS, int STAGES, int STATES> struct ScanSmem {
    static constexpr int V = Pack<T>::V, CT = 8 * V;        // channels of a thread, of a slice
    static constexpr int kGroups = THREADS / 8;            // token groups of a CTA (8 threads across the channels)
    static constexpr int kTile = kGroups * R;              // tokens
    static constexpr int kParts = THREADS / CT, kPer = kGroups / kParts;
    static constexpr int kSlot = kGroups * group_bytes<ALIGN, R>();  // one tensor's tile
    static constexpr int kStage = 2 * kSlot;
    static constexpr int kSpans = kGroups * CT * (int)sizeof(float2), kStates = kGroups * CT * (int)sizeof(float);
    static constexpr int kBytes = STAGES * kStage + kSpans + STATES * kStates + kParts * CT * (int)sizeof(float2);

    unsigned char* ring;
    float4* spans;      // [group][pair of V/2][col]: A, H, A, H
    float* states;      // [copy][group][quad of V/4][col][4]
    float2* parts;      // [part][channel]
    float2* whole;      // what follows
    __device__ __forceinline__ explicit ScanSmem(unsigned char* smem) {
        ring = smem;
        spans = reinterpret_cast<float4*>(smem + STAGES * kStage);
        states = reinterpret_cast<float*>(smem + STAGES * kStage + kSpans);
        parts = reinterpret_cast<float2*>(smem + STAGES * kStage + kSpans + STATES * kStates);
        whole = parts + kParts * CT;
    }
    __device__ __forceinline__ unsigned char* stage(int k) const { return ring + k * kStage; }
};

// What a thread knows of its sequence and slice, and the steps that both scan kernels take.
template <typename T, int ALIGN, bool BWD, int R, int THREADS, typename Sm>
struct Walk {
    static constexpr int V = Sm::V, CT = Sm::CT, PER = Sm::kPer, PARTS = Sm::kParts;
    const RecurrenceArgs& a;
    int rank, size, n, c0, D, len, col, group;
    long long begin;
    const T *la, *x, *hf, *la_stop, *x_stop;
    T *out, *out_la;
    // As (channel, part): channel p in the order of the spans, that is element e = 2 pair + half of thread column pcol.
    int p, part, pair, pcol, half, pc;

    __device__ __forceinline__ Walk(const RecurrenceArgs& a_, int n_, long long id, int slices, int rank_, int size_)
        : a(a_), rank(rank_), size(size_), n(n_) {
        const int tid = threadIdx.x;
        c0 = (int)(id % slices) * CT;
        D = a.D;
        token_range(a.cu_seqlens, n, a.T, begin, len);
        la = (const T*)a.log_alpha + begin * D;
        x = (const T*)a.x + begin * D;
        hf = BWD ? (const T*)a.h_fwd + begin * D : nullptr;
        out = (T*)a.out + begin * D;
        out_la = BWD ? (T*)a.out_la + begin * D : nullptr;
        const long long cells = (a.cu_seqlens ? 1ll : (long long)a.N) * a.T * D;  // the end of the tensors
        la_stop = (const T*)a.log_alpha + cells;
        x_stop = (const T*)a.x + cells;
        col = tid & 7;
        group = tid >> 3;
        p = tid % CT;
        part = tid / CT;
        pair = p / 16;
        pcol = p % 16 / 2;
        half = p % 2;
        pc = c0 + channel_of<T, ALIGN>(pcol, 2 * pair + half);
    }
    __device__ __forceinline__ int tiles() const {
        const long long step = (long long)size * Sm::kTile;
        return (int)((len + step - 1) / step);
    }
    __device__ __forceinline__ float first_state() const { return pc < D && a.state0 ? a.state0[(long long)n * D + pc] : 0.f; }
    __device__ __forceinline__ void last_state(float s) const {
        if (part == 0 && rank == 0 && pc < D && a.state_end) a.state_end[(long long)n * D + pc] = s;
    }
    // number, in walking order, of token k of this CTA's tile `tile`: below len + 16 tiles, so no wrap
    __device__ __forceinline__ unsigned number(int tile, int k) const { return (unsigned)(tile * size + rank) * Sm::kTile + k; }
    // the token itself; -1: past the end
    __device__ __forceinline__ int token(int tile, int i) const {
        const unsigned at = number(tile, group * R + i);
        return at < (unsigned)len ? (BWD ? len - 1 - (int)at : (int)at) : -1;
    }
    __device__ __forceinline__ void fetch(unsigned char* to, int tile) const {
        const long long at = number(tile, 0);
        const int left = (int)min(max(len - at, 0ll), (long long)Sm::kTile);
        const long long row = (BWD ? len - 1 - at : at) * D;
        copy_tile<T, ALIGN, R, THREADS>(to, la + row, BWD ? -D : D, left, c0, D, la_stop);
        copy_tile<T, ALIGN, R, THREADS>(to + Sm::kSlot, x + row, BWD ? -D : D, left, c0, D, x_stop);
    }
    // Token i of a fetched tile.
    __device__ __forceinline__ void read(const unsigned char* from, int tile, int i, Pack<T>& pl, Pack<T>& px) const {
        // the tensors and the slices begin on 16 bytes, so both rows begin alike (past the end are zeros, wherever read)
        const int off = ALIGN == 16 ? 0 : (int)(((unsigned)begin + (unsigned)token(tile, i)) * (unsigned)D * (unsigned)sizeof(T) & 15u);
        pl = slot_of<T, ALIGN, R, THREADS>(from, i, off);
        px = slot_of<T, ALIGN, R, THREADS>(from + Sm::kSlot, i, off);
    }
    __device__ __forceinline__ const T* before(int t) const { return hf + (long long)max(t - 1, 0) * D; }
    // h_{t-1} of the thread's tokens (zeros for the first token, whose is h0)
    __device__ __forceinline__ void read_before(int tile, RowWords<T, ALIGN> (&ph)[R]) const {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int t = token(tile, i);
            ph[i] = read_row<T, ALIGN>(before(t), c0, col, D, t > 0);
        }
    }
    __device__ __forceinline__ static void decays(const Pack<T>& pl, F2 (&d)[V / 2]) {
#pragma unroll
        for (int e = 0; e < V / 2; ++e) d[e] = f2(decay<T>(pl.get(2 * e)), decay<T>(pl.get(2 * e + 1)));
    }
    // (A, H) <- the token after (A, H)
    __device__ __forceinline__ static void compose(bool first, const F2 (&d)[V / 2], const Pack<T>& px, F2 (&A)[V / 2], F2 (&H)[V / 2]) {
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
            const F2 v = f2(px.get(2 * e), px.get(2 * e + 1));
            A[e] = first ? d[e] : f2_mul(A[e], d[e]);
            if (BWD) H[e] = f2_mul(d[e], first ? v : f2_add(H[e], v));
            else H[e] = first ? v : f2_fma(d[e], H[e], v);
        }
    }
    __device__ __forceinline__ void put_span(const Sm& sm, const F2 (&A)[V / 2], const F2 (&H)[V / 2]) const {
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
            const float2 A_ = f2_parts(A[e]), H_ = f2_parts(H[e]);
            sm.spans[(group * (V / 2) + e) * 8 + col] = make_float4(A_.x, H_.x, A_.y, H_.y);
        }
    }
    // The spans of this part's groups; the part's span goes to sm.parts.
    __device__ __forceinline__ void part_span(const Sm& sm, float2 (&w)[PER]) const {
#pragma unroll
        for (int k = 0; k < PER; ++k)
            w[k] = reinterpret_cast<const float2*>(sm.spans)[((part * PER + k) * (V / 2) + pair) * 16 + pcol * 2 + half];
        float2 all = w[0];
#pragma unroll
        for (int k = 1; k < PER; ++k) all = make_float2(all.x * w[k].x, fmaf(w[k].x, all.y, w[k].y));
        sm.parts[part * CT + p] = all;
    }
    // Of the CTA's parts: those before this one, all.
    __device__ __forceinline__ void whole_span(const Sm& sm, float2& before, float2& whole) const {
        before = whole = make_float2(1.f, 0.f);
#pragma unroll
        for (int k = 0; k < PARTS; ++k) {
            const float2 u = sm.parts[k * CT + p];
            if (k == part) before = whole;
            whole = make_float2(whole.x * u.x, fmaf(u.x, whole.y, u.y));
        }
    }
    // The states that enter this part's groups, from the one that enters the part.
    __device__ __forceinline__ void put_states(float* states, float s, const float2 (&w)[PER]) const {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            states[(((part * PER + k) * (V / 4) + pair / 2) * 8 + pcol) * 4 + (pair & 1) * 2 + half] = s;
            s = fmaf(w[k].x, s, w[k].y);
        }
    }
    __device__ __forceinline__ void own_state(const float* states, F2 (&cur)[V / 2]) const {
#pragma unroll
        for (int q = 0; q < V / 4; ++q) {
            const float4 v = reinterpret_cast<const float4*>(states)[(group * (V / 4) + q) * 8 + col];
            cur[2 * q] = f2(v.x, v.y);
            cur[2 * q + 1] = f2(v.z, v.w);
        }
    }
    // Token i from the state that enters it: writes its outputs, moves the state on.
    __device__ __forceinline__ void run_token(int tile, int i, const F2 (&d)[V / 2], const Pack<T>& px, const RowWords<T, ALIGN>& words,
                                              F2 (&cur)[V / 2]) const {
        const int t = token(tile, i);
        Pack<T> ph;
        if constexpr (BWD) ph = row_of<T, ALIGN>(words, before(t), col);
        float y[V], z[V];
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
            const F2 v = f2(px.get(2 * e), px.get(2 * e + 1));
            F2 o;
            if constexpr (BWD) {
                o = f2_add(cur[e], v);
                cur[e] = f2_mul(d[e], o);
                float b0 = ph.get(2 * e), b1 = ph.get(2 * e + 1);
                if (t == 0) {
                    const int e0 = c0 + channel_of<T, ALIGN>(col, 2 * e), e1 = c0 + channel_of<T, ALIGN>(col, 2 * e + 1);
                    b0 = a.h0 && e0 < D ? a.h0[(long long)n * D + e0] : 0.f;
                    b1 = a.h0 && e1 < D ? a.h0[(long long)n * D + e1] : 0.f;
                }
                const float2 zz = f2_parts(f2_mul(cur[e], f2(b0, b1)));
                z[2 * e] = zz.x;
                z[2 * e + 1] = zz.y;
            } else {
                o = cur[e] = f2_fma(d[e], cur[e], v);
            }
            const float2 yy = f2_parts(o);
            y[2 * e] = yy.x;
            y[2 * e + 1] = yy.y;
        }
        store_row<T, ALIGN>(out + (long long)t * D, c0, col, D, t >= 0, y);
        if constexpr (BWD) store_row<T, ALIGN>(out_la + (long long)t * D, c0, col, D, t >= 0, z);
    }
};

// The k-th longest of N <= THREADS packed sequences: CTAs are given out in this order, so that no long sequence begins
// when the others are done (nine sequences of 0 to 3400 tokens, D 2048: 46.7 us in the order they lie, 40.8 so). Every CTA
// counts for itself, N steps: many short sequences lose more than they gain (256 of 64 tokens, D 4096: 329 us, the same
// tokens as a dense batch 137).
template <int THREADS> __device__ __forceinline__ int longest(const RecurrenceArgs& a, int k, int* scratch) {
    const int i = threadIdx.x;
    long long begin;
    int len = -1;
    if (i < a.N) {
        token_range(a.cu_seqlens, i, a.T, begin, len);
        scratch[i] = len;
    }
    __syncthreads();
    int before = 0;
    for (int j = 0; j < a.N; ++j) before += scratch[j] > len || (scratch[j] == len && j < i);
    if (i < a.N && before == k) scratch[THREADS] = i;
    __syncthreads();
    const int n = scratch[THREADS];
    __syncthreads();
    return n;
}

// One CTA a row. R: tokens of a thread.
template <typename T, int ALIGN, bool BWD, int R, int THREADS>
__global__ void __launch_bounds__(THREADS, 512 / THREADS) recurrence_scan_kernel(RecurrenceArgs a, int slices) {
    constexpr int S = 2;
    using Sm = ScanSmem<T, ALIGN, R, THREADS, S, 1>;
    constexpr int V = Sm::V;
    extern __shared__ __align__(16) unsigned char smem[];
    const Sm sm(smem);
    int n = blockIdx.x / slices;
    if (a.cu_seqlens && a.N > 1 && a.N <= THREADS) n = longest<THREADS>(a, n, reinterpret_cast<int*>(sm.spans));
    const Walk<T, ALIGN, BWD, R, THREADS, Sm> walk(a, n, blockIdx.x, slices, 0, 1);
    float state = walk.first_state();  // every part keeps its channel's, by the same operations
    const int tiles = walk.tiles();
    for (int k = 0; k < S; ++k) {
        if (k < tiles) walk.fetch(sm.stage(k), k);
        cp_async_commit();
    }
    for (int tile = 0; tile < tiles; ++tile) {
        // 1. this thread's tokens as one span
        cp_async_wait<S - 1>();
        if constexpr (ALIGN != 16) __syncwarp();
        F2 d[R][V / 2], A[V / 2], H[V / 2];
        Pack<T> px[R];
        RowWords<T, ALIGN> ph[R];
        if constexpr (BWD) walk.read_before(tile, ph);  // used at the tile's end
#pragma unroll
        for (int i = 0; i < R; ++i) {
            Pack<T> pl;
            walk.read(sm.stage(tile & 1), tile, i, pl, px[i]);
            walk.decays(pl, d[i]);
            walk.compose(i == 0, d[i], px[i], A, H);
        }
        if constexpr (ALIGN != 16) __syncwarp();
        if (tile + S < tiles) walk.fetch(sm.stage(tile & 1), tile + S);
        cp_async_commit();
        walk.put_span(sm, A, H);
        __syncthreads();
        // 2. as (channel, part): the part's span, the CTA's
        float2 w[Sm::kPer], before, whole;
        walk.part_span(sm, w);
        __syncthreads();
        walk.whole_span(sm, before, whole);
        // 3. the state that enters this part's groups; the state after the tile
        walk.put_states(sm.states, fmaf(before.x, state, before.y), w);
        state = fmaf(whole.x, state, whole.y);
        __syncthreads();
        // 4. the tokens again, from the state that enters them
        F2 cur[V / 2];
        walk.own_state(sm.states, cur);
#pragma unroll
        for (int i = 0; i < R; ++i) walk.run_token(tile, i, d[i], px[i], ph[i], cur);
    }
    cp_async_wait<0>();
    walk.last_state(state);
}

// A 64-bit store into the shared memory of CTA `rank` of the cluster, counted there by the mbarrier at the same place as
// `bar` here. It needs no fence: a cluster barrier with its release would wait for the stores to global memory, 1 us.
__device__ __forceinline__ void push(const void* to, uint64_t* bar, int rank, float2 x) {
    uint32_t at, b;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(sm100::smem_u32(to)), "r"(rank));
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(sm100::smem_u32(bar)), "r"(rank));
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(at),
                 "r"(__float_as_uint(x.x)), "r"(__float_as_uint(x.y)), "r"(b)
                 : "memory");
}

// A cluster of CTAs a row, where rows are few: what counts is the time of one round of tiles. So the rounds overlap: the
// spans of tile k + 1 are composed and handed to the cluster before tile k is run, and the exchange of tile k has tile
// k - 1's run to finish in. The spans are pushed into every CTA's inbox and counted by its mbarrier; a wait that is not
// met in a.wait_cycles sets g_recurrence_late, and the kernel ends without waiting, pushing or arming a barrier again (the
// others' next waits then give up too). An inbox slot is written again two tiles later, when its owner has sent the tile
// between, which it does after having read the slot and armed its barrier again.
template <typename T, int ALIGN, bool BWD, int R, int THREADS, int S>
__global__ void __launch_bounds__(THREADS, 1) recurrence_cluster_kernel(RecurrenceArgs a, int slices) {
    using Sm = ScanSmem<T, ALIGN, R, THREADS, S, 2>;
    constexpr int V = Sm::V, CT = Sm::CT;
    extern __shared__ __align__(16) unsigned char smem[];
    const Sm sm(smem);
    const cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), size = (int)cluster.num_blocks();
    const Walk<T, ALIGN, BWD, R, THREADS, Sm> walk(a, blockIdx.x / size / slices, blockIdx.x / size, slices, rank, size);
    float state = walk.first_state();
    float2* inbox = sm.whole;  // [parity][rank][channel]: the CTAs' spans
    uint64_t* bar = reinterpret_cast<uint64_t*>(inbox + 2 * kMaxCluster * CT);  // [parity]: they have arrived
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) sm100::mbar_init(bar + i, 1);
        sm100::fence_mbar_init();
        for (int i = 0; i < 2; ++i) sm100::mbar_arrive_expect_tx(bar + i, size * CT * 8);
    }
    cluster.sync();  // every CTA has started, has read its state and set up its barriers
    const int tiles = walk.tiles();
#pragma unroll 1
    for (int k = 0; k < S - 1; ++k) {
        if (k < tiles) walk.fetch(sm.stage(k), k);
        cp_async_commit();
    }
    float2 w[Sm::kPer], before = make_float2(1.f, 0.f);
    bool late = false;  // a wait gave up
    // decays and inputs of the tile that is run, and of the one after it
    F2 d[R][V / 2], d1[R][V / 2];
    Pack<T> px[R], px1[R];
    // the thread's span of a tile that has arrived
    auto span = [&](int tile, F2 (&A)[V / 2], F2 (&H)[V / 2]) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            Pack<T> pl;
            walk.read(sm.stage(tile % S), tile, i, pl, px1[i]);
            walk.decays(pl, d1[i]);
            walk.compose(i == 0, d1[i], px1[i], A, H);
        }
    };
    // from the spans in shared memory to the CTA's span, handed to the cluster
    auto publish = [&](int tile) {
        walk.part_span(sm, w);
        __syncthreads();
        float2 whole;
        walk.whole_span(sm, before, whole);
        if (late || (a.test_withhold && rank == 0)) return;
        for (int r = walk.part; r < size; r += Sm::kParts) push(inbox + ((tile & 1) * kMaxCluster + rank) * CT + walk.p, bar + (tile & 1), r, whole);
    };
    if (tiles > 0) {
        cp_async_wait<S - 2>();
        if constexpr (ALIGN != 16) __syncwarp();
        F2 A[V / 2], H[V / 2];
        span(0, A, H);
        walk.put_span(sm, A, H);
        __syncthreads();
        publish(0);
    }
#pragma unroll 1
    for (int tile = 0; tile < tiles; ++tile) {
        const bool more = tile + 1 < tiles;
        if constexpr (ALIGN != 16) __syncwarp();  // the stage that is filled next was read by the whole warp
        if (tile + S - 1 < tiles) walk.fetch(sm.stage((tile + S - 1) % S), tile + S - 1);
        cp_async_commit();
#pragma unroll
        for (int i = 0; i < R; ++i) {
            px[i] = px1[i];
#pragma unroll
            for (int e = 0; e < V / 2; ++e) d[i][e] = d1[i][e];
        }
        RowWords<T, ALIGN> ph[R];
        if constexpr (BWD) walk.read_before(tile, ph);
        F2 A[V / 2], H[V / 2];
        if (more) {
            cp_async_wait<S - 2>();
            if constexpr (ALIGN != 16) __syncwarp();
            span(tile + 1, A, H);
        }
        // the state that enters this CTA's tile; the state after the cluster's
        if (!late) late = !sm100::mbar_wait_bounded(bar + (tile & 1), (tile >> 1) & 1, a.wait_cycles);
        const float2* theirs = inbox + (tile & 1) * kMaxCluster * CT + walk.p;
        float s = state;
        for (int r = 0; r < size; ++r) {
            const float2 u = theirs[r * CT];
            if (r == rank) s = state;
            state = fmaf(u.x, state, u.y);
        }
        // of tile + 2. Only after a phase that was completed: a barrier must get no arrival more than a phase takes.
        if (threadIdx.x == 0 && !late) sm100::mbar_arrive_expect_tx(bar + (tile & 1), size * CT * 8);
        float* states = sm.states + (tile & 1) * (Sm::kStates / 4);
        walk.put_states(states, fmaf(before.x, s, before.y), w);
        if (more) walk.put_span(sm, A, H);
        __syncthreads();
        if (more) publish(tile + 1);
        F2 cur[V / 2];
        walk.own_state(states, cur);
#pragma unroll
        for (int i = 0; i < R; ++i) walk.run_token(tile, i, d[i], px[i], ph[i], cur);
    }
    cp_async_wait<0>();
    if (late) {
        g_recurrence_late = 1;
        // what others have pushed lands in microseconds: not in the shared memory of a CTA that has ended
        for (const long long t0 = clock64(); clock64() - t0 < (1ll << 17);) {}
    }
    cluster.sync();  // no CTA ends while another may still write to its shared memory
    walk.last_state(state);
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

template <typename T, int ALIGN, bool BWD, int THREADS>
cudaError_t launch_rows(const RecurrenceArgs& a, int slices, cudaStream_t stream) {
    using Sm = ScanSmem<T, ALIGN, kTokens, THREADS, 2, 1>;
    auto kernel = recurrence_scan_kernel<T, ALIGN, BWD, kTokens, THREADS>;
    static std::atomic<unsigned long long> raised{0};
    const cudaError_t err = allow_smem(kernel, Sm::kBytes, raised);
    if (err != cudaSuccess) return err;
    kernel<<<(unsigned)((long long)a.N * slices), THREADS, Sm::kBytes, stream>>>(a, slices);
    return cudaGetLastError();
}

// A thread's tokens in a cluster. Eight of a float row fill as many registers as four of a bf16 one and halve the rounds:
// T16384 D1000 39 us, with four 44. Not so where a thread has the backward pass's h beside them (82 and 67); for unaligned
// rows eight leave no room for a third stage, and six take 63 us where four take 59.
template <typename T, int ALIGN, bool BWD> constexpr int cluster_tokens() { return sizeof(T) == 4 && ALIGN == 16 && !BWD ? 8 : 4; }

template <typename T, int ALIGN, bool BWD>
cudaError_t launch_clusters(const RecurrenceArgs& a, int slices, int size, cudaStream_t stream) {
    constexpr int THREADS = 256, R = cluster_tokens<T, ALIGN, BWD>(), S = R == 4 ? 4 : 3;
    using Sm = ScanSmem<T, ALIGN, R, THREADS, S, 2>;
    constexpr int kBytes = Sm::kBytes + 2 * kMaxCluster * Sm::CT * (int)sizeof(float2) + 16;
    auto kernel = recurrence_cluster_kernel<T, ALIGN, BWD, R, THREADS, S>;
    static std::atomic<unsigned long long> raised{0};
    cudaError_t err = size > 8 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) : cudaSuccess;
    if (err == cudaSuccess) err = allow_smem(kernel, kBytes, raised);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)a.N * slices * size));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = kBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = size;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, slices);
}

template <typename T, int ALIGN, bool BWD>
cudaError_t launch_scan(const RecurrenceArgs& a, cudaStream_t stream) {
    constexpr int CT = 8 * Pack<T>::V;
    const int slices = (a.D + CT - 1) / CT;
    const long long rows = (long long)a.N * slices;
    const long long tokens = tokens_of(a);
    // CTAs of a cluster. From 75 rows on one: the rows alone fill the SMs (128 rows, T 8192 backward: 127 us, with two
    // 131). Below, about as many as fit on the GPU at once, one an SM, where a cluster takes SMs of one GPC (one B200 says
    // that it holds 7 of sixteen, 15 of eight, 33 of four; it depends on which SMs a GPU has): six clusters of sixteen
    // (four rows, T 65536: 52 us, with eight 98), fourteen of eight (twelve rows, T 32768: 53 us, with sixteen 57),
    // thirty-four of four (32 rows, T 16384: 52 us, with two 89), else two; 15 and 16 rows take clusters of sixteen in
    // three rounds (T 32768: 82 us, with four 97). No more than the tokens give tiles to.
    const int most = rows <= 6 ? 16 : rows <= 14 ? 8 : rows <= 16 ? 16 : rows <= 34 ? 4 : rows < 75 ? 2 : 1;
    int size = 1;
    while (size < most && (long long)size * (256 / 8) * cluster_tokens<T, ALIGN, BWD>() < tokens) size *= 2;
    if (a.test_withhold && size == 1) return cudaErrorInvalidValue;
    if (size > 1) return launch_clusters<T, ALIGN, BWD>(a, slices, size, stream);
    // One CTA of 512 threads on an SM takes tiles of twice the tokens, and its SM's share of the bandwidth with fewer
    // barriers: 256 rows, T 8192 132 us (two CTAs of 256 threads: 150); 96 rows, T 4096 backward 51 (65). It pays where
    // the rows fill their rounds of 148 (192 rows: 67 us against 57) and there are tokens enough (T 200: 7.4 against 5.8).
    const long long rounds = (rows + 147) / 148;
    if (tokens >= 512 && (rounds == 1 || rows * 5 >= rounds * 148 * 4)) return launch_rows<T, ALIGN, BWD, 512>(a, slices, stream);
    return launch_rows<T, ALIGN, BWD, 256>(a, slices, stream);
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

cudaError_t recurrence_late(unsigned* flag) {
    cudaError_t err = cudaMemcpyFromSymbol(flag, g_recurrence_late, sizeof(*flag));
    const unsigned zero = 0;
    if (err == cudaSuccess && *flag) err = cudaMemcpyToSymbol(g_recurrence_late, &zero, sizeof(zero));
    return err;
}

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
