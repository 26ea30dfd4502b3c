// Queries and keys of a layer: norm per head and rotation by position in one
// pass, and the backward pass.
//
//     y = R (w x r),  r = (share * sum x^2 + eps)^-1/2      (share: 1 for L2, 1/d for RMS)
// With u = R^T dy, n = x r:
//     dw = sum u n,   dx = r (w u - share * n * sum(w u n)).
//
// What bounds it: HBM, 2 (backward 3) elements of the tensors per channel. A
// head is read once by a group of LANES lanes, 8 channels (16 or 32 bytes) a
// lane, and stays in registers: the sums are shuffles within the group, and the
// rotation's partner channel is either in the same lane (interleaved pairs) or,
// unnormalised, in the lane rot/16 away (halves). A group takes up to `chunk`
// heads of one token, so that the token's row of the tables, with the weight
// multiplied in, is read once for them all. 32768 tokens x 64 heads of 128, bf16:
// 158 us (1.05 of the measured copy bandwidth); backward of 8192 x 40: 49-51 us
// (0.77-0.80, bound by its instructions and by the second kernel that sums the weights).
#include <algorithm>
#include <type_traits>

#include "kda_async.cuh"
#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {

namespace {

constexpr int kThreads = 256;
constexpr long long kBwdCtas = 296;  // of the backward pass: two on each of 148 SMs
enum { kNoTurn = 0, kHalves = 1, kPairs = 2 };

// One side (queries or keys) of a call.
struct Side {
    const void *x, *w, *dy;
    void* y;
    long long stride_t, stride_h;
    int H;
    float scale;
};

__device__ __forceinline__ Side side_of(const QkArgs& a, bool is_q) {
    return is_q ? Side{a.q, a.q_weight, a.d_q_out, a.q_out, a.q_stride_t, a.q_stride_h, a.Hq, a.q_scale}
                : Side{a.k, a.k_weight, a.d_k_out, a.k_out, a.k_stride_t, a.k_stride_h, a.Hk, 1.f};
}

// 8 channels as they lie in memory.
template <typename T> struct Raw {
    static constexpr int W = 8 * sizeof(T) / 4;
    uint32_t w[W];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < W; i += 4) {
            const uint4 v = reinterpret_cast<const uint4*>(p)[i / 4];
            w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
        }
    }
    __device__ __forceinline__ void load_pieces(const uint4* p, int apart) {
#pragma unroll
        for (int i = 0; i < W; i += 4) {
            const uint4 v = p[i / 4 * apart];
            w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0u;
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (W == 8) return __uint_as_float(w[i]);
        else return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
    // By a power of two: exact but for what falls below the type's smallest numbers.
    __device__ __forceinline__ void scale(float f) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if constexpr (W == 8) {
                w[i] = __float_as_uint(get(i) * f);
            } else {
                const __nv_bfloat162 b = __floats2bfloat162_rn(get(2 * i) * f, get(2 * i + 1) * f);
                w[i] = *reinterpret_cast<const uint32_t*>(&b);
            }
        }
    }
    __device__ __forceinline__ F2 pair(int i) const { return f2(get(2 * i), get(2 * i + 1)); }
};

__device__ __forceinline__ void store8(float* p, const float (&y)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(y[0], y[1], y[2], y[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(y[4], y[5], y[6], y[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&y)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <int LANES> __device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
    return x;
}

// Two sums at once.
template <int LANES> __device__ __forceinline__ F2 group_sum2(F2 x) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
        const float2 p = f2_parts(x);
        x = f2_add(x, f2(__shfl_xor_sync(~0u, p.x, o), __shfl_xor_sync(~0u, p.y, o)));
    }
    return x;
}

// r of a head from its sum of squares. Where that leaves 32 bits the head is
// rescaled by 2^-80 first, and eps by 2^-160 (a large one still counts beside it).
__device__ __forceinline__ float small_eps(float eps) { return eps * 0x1p-80f * 0x1p-80f; }
template <typename T, int LANES>
__device__ __forceinline__ float rnorm(const Raw<T>& x, float ss, float share, float eps) {
    float r = rsqrtf(fmaf(ss, share, eps));
    const bool out = !(ss < 1e37f);
    if (__any_sync(~0u, out)) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(x.get(e) * 0x1p-80f, x.get(e) * 0x1p-80f, s);
        s = group_sum<LANES>(s);
        if (out) r = 0x1p-80f * rsqrtf(fmaf(s, share, small_eps(eps)));
    }
    return r;
}

__device__ __forceinline__ long long position_of(const QkArgs& a, long long t) {
    const long long p = a.pos_bytes == 8 ? ((const long long*)a.positions)[t] : (long long)((const int*)a.positions)[t];
    return min(max(p, 0ll), (long long)a.max_pos - 1);
}

// This lane's cosines and sines, the sines signed as in y_c = x_c cos + x_partner sin
// (1 and 0 for channels that are not rotated). Returns the lane that holds the partners.
template <int MODE>
__device__ __forceinline__ int turn_of(const QkArgs& a, long long pos, int c, int lane, float (&cs)[8], float (&sn)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        cs[e] = 1.f;
        sn[e] = 0.f;
    }
    if (MODE == kNoTurn || c >= a.rot) return lane;
    const int half = a.rot / 2;
    const size_t row = (size_t)pos * half;
    if (MODE == kHalves) {
        const bool first = c < half;
        const int i = first ? c : c - half;
        const float4 *pc = reinterpret_cast<const float4*>(a.cos + row + i), *ps = reinterpret_cast<const float4*>(a.sin + row + i);
        const float4 c0 = __ldg(pc), c1 = __ldg(pc + 1), s0 = __ldg(ps), s1 = __ldg(ps + 1);
        cs[0] = c0.x; cs[1] = c0.y; cs[2] = c0.z; cs[3] = c0.w; cs[4] = c1.x; cs[5] = c1.y; cs[6] = c1.z; cs[7] = c1.w;
        sn[0] = s0.x; sn[1] = s0.y; sn[2] = s0.z; sn[3] = s0.w; sn[4] = s1.x; sn[5] = s1.y; sn[6] = s1.z; sn[7] = s1.w;
        if (first) {
#pragma unroll
            for (int e = 0; e < 8; ++e) sn[e] = -sn[e];
        }
        return first ? lane + half / 8 : lane - half / 8;
    }
    const float4 c0 = __ldg(reinterpret_cast<const float4*>(a.cos + row + c / 2)), s0 = __ldg(reinterpret_cast<const float4*>(a.sin + row + c / 2));
    const float cc[4] = {c0.x, c0.y, c0.z, c0.w}, ss[4] = {s0.x, s0.y, s0.z, s0.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        cs[e] = cc[e / 2];
        sn[e] = e % 2 ? ss[e / 2] : -ss[e / 2];
    }
    return lane;
}

// The partner channels of x, unnormalised.
template <typename T, int MODE> __device__ __forceinline__ Raw<T> partners(const Raw<T>& x, int from) {
    Raw<T> p = x;
    if constexpr (MODE == kHalves) {
#pragma unroll
        for (int i = 0; i < Raw<T>::W; ++i) p.w[i] = __shfl_sync(~0u, x.w[i], from);
    } else if constexpr (MODE == kPairs) {
        if constexpr (Raw<T>::W == 8) {
#pragma unroll
            for (int i = 0; i < 8; ++i) p.w[i] = x.w[i ^ 1];
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) p.w[i] = __funnelshift_l(x.w[i], x.w[i], 16);
        }
    }
    return p;
}

template <typename T, int LANES, int MODE>
__global__ void __launch_bounds__(kThreads) qk_fwd_kernel(QkArgs a, int chunk, int q_chunks, int chunks) {
    constexpr int GROUPS = kThreads / LANES, AHEAD = 4;
    const int lane = threadIdx.x & 31, c = (threadIdx.x % LANES) * 8;
    const long long item = (long long)blockIdx.x * GROUPS + threadIdx.x / LANES;
    const long long t = item / chunks;
    const int part = (int)(item % chunks);
    const bool live = t < a.n, is_q = part < q_chunks, mine = live && c < a.d;
    const Side s = side_of(a, is_q);
    const int h0 = (is_q ? part : part - q_chunks) * chunk, heads = live ? min(chunk, s.H - h0) : 0;
    const T* x = (const T*)s.x + (live ? t * s.stride_t + h0 * s.stride_h : 0) + c;
    T* y = (T*)s.y + (live ? (t * s.H + h0) * a.d : 0) + c;
    Raw<T> v[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
        v[i].clear();
        if (mine && i < heads) v[i].load(x + i * s.stride_h);
    }
    float cw[8], sw[8];  // cosine and signed sine, times the weight of the channel they meet and the side's scale
    int from = lane;
    if (mine) from = turn_of<MODE>(a, MODE == kNoTurn ? 0 : position_of(a, t), c, lane, cw, sw);
    else {
#pragma unroll
        for (int e = 0; e < 8; ++e) cw[e] = sw[e] = 0.f;
    }
    // A warp may hold groups of both sides, of which one alone has a weight: the exchange is outside of any condition.
    Raw<T> w;
    w.clear();
    if (mine && s.w) w.load((const T*)s.w + c);
    const Raw<T> wp = partners<T, MODE>(w, from);
    if (s.w) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            cw[e] *= w.get(e);
            sw[e] *= wp.get(e);
        }
    }
    if (s.scale != 1.f) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            cw[e] *= s.scale;
            sw[e] *= s.scale;
        }
    }
    const float share = a.norm ? 1.f / a.d : 1.f;
    // every lane of a warp runs as many rounds as its longest group: the shuffles take all of them
    const int rounds = __reduce_max_sync(~0u, heads);
    for (int h = 0; h < rounds; h += AHEAD) {
        Raw<T> u[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            u[i] = v[i];
            if (mine && h + AHEAD + i < heads) v[i].load(x + (h + AHEAD + i) * s.stride_h);
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (h + i >= rounds) break;
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(u[i].get(e), u[i].get(e), ss);
            ss = group_sum<LANES>(ss);
            const float r = rnorm<T, LANES>(u[i], ss, share, a.eps);
            const Raw<T> p = partners<T, MODE>(u[i], from);
            float out[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float z = u[i].get(e) * r * cw[e];
                out[e] = MODE == kNoTurn ? z : fmaf(p.get(e) * r, sw[e], z);
            }
            if (mine && h + i < heads) store8(y + (long long)(h + i) * a.d, out);
        }
    }
}

// CTAs below q_ctas walk the queries, the others the keys. A side's heads are cut into `parts` of `chunk` (the last may
// hold fewer); a group keeps to one part and walks the tokens with a stride. Loads run AHEAD heads before the
// arithmetic, across the tokens. `part_sums` gets each CTA's sum of the weight's gradient. The arithmetic is on
// pairs of channels (one instruction for two products), without which the kernel would be bound by its instructions.
template <typename T> struct BwdPlan {
    static constexpr int kRowBytes = 8 * sizeof(T);                 // a thread's channels of one head
    static constexpr int kStages = sizeof(T) == 2 ? 6 : 4;           // heads in flight (bf16: with 8 or 12 it is 2 to 4 % slower)
    static constexpr int kSmem = kStages * 2 * kRowBytes * kThreads;  // 48 or 64 KB
};

template <typename T, int LANES, int MODE>
__global__ void __launch_bounds__(kThreads, 2) qk_bwd_kernel(QkArgs a, int q_chunk, int k_chunk, int q_ctas, float* part_sums) {
    using Plan = BwdPlan<T>;
    constexpr int GROUPS = kThreads / LANES, S = Plan::kStages, W = Plan::kRowBytes / 16;
    extern __shared__ __align__(16) uint4 ring[];  // [stage][x, dy][16-byte piece][thread]: read by the thread that filled it
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // qk_dw_kernel: waits for this grid's end
    const int lane = threadIdx.x & 31, c = (threadIdx.x % LANES) * 8;
    const bool is_q = (int)blockIdx.x < q_ctas;
    const Side s = side_of(a, is_q);
    const int cta = is_q ? blockIdx.x : blockIdx.x - q_ctas, ctas = is_q ? q_ctas : gridDim.x - q_ctas;
    const int chunk = is_q ? q_chunk : k_chunk, parts = (s.H + chunk - 1) / chunk;
    const int group = cta * GROUPS + threadIdx.x / LANES;
    const int stride = max(ctas * GROUPS / parts, 1);  // tokens that are worked on at once
    const int part = group % parts, t0 = group / parts, h0 = part * chunk;
    const bool on = c < a.d && t0 < stride;
    const int heads = on ? min(chunk, s.H - h0) : 0;
    const int rounds = (int)(((long long)a.n + stride - 1) / stride);  // the same for all groups: the shuffles take whole warps
    const float share = a.norm ? 1.f / a.d : 1.f;

    // the loading side: head lh of token lt
    long long lt = t0;
    int lh = 0;
    const T* x = (const T*)s.x + (on ? lt * s.stride_t + h0 * s.stride_h : 0) + c;
    const T* dy = (const T*)s.dy + (on ? (lt * s.H + h0) * a.d : 0) + c;
    const long long next_x = stride * s.stride_t - chunk * s.stride_h, next_dy = ((long long)stride * s.H - chunk) * a.d;
    auto load = [&](int stage) {  // heads past the end become zeros
        const bool fill = lh < heads && lt < a.n;  // a copy of zeros does not touch its source
        uint4* to = ring + stage * 2 * W * kThreads + threadIdx.x;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            cp_async16(to + i * kThreads, x + i * 16 / sizeof(T), fill);
            cp_async16(to + (W + i) * kThreads, dy + i * 16 / sizeof(T), fill);
        }
        cp_async_commit();
        x += s.stride_h;
        dy += a.d;
        if (++lh == chunk) {
            lh = 0;
            lt += stride;
            x += next_x;
            dy += next_dy;
        }
    };
#pragma unroll 1
    for (int i = 0; i < S - 1; ++i) load(i);
    F2 w[4], dw[4];
    {
        Raw<T> raw;
        raw.clear();
        if (s.w && on) raw.load((const T*)s.w + c);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w[e] = s.w ? raw.pair(e) : f2(1.f, 1.f);
            dw[e] = f2(0.f, 0.f);
        }
    }
    auto ahead = [&](long long at) { return MODE != kNoTurn && on && at < a.n ? position_of(a, at) : 0; };
    long long t = t0, pos = ahead(t0);
    T* dx = (T*)s.y + (on ? (t * s.H + h0) * a.d : 0) + c;
    const long long next_dx = ((long long)stride * s.H - chunk) * a.d;
    int stage = 0, into = S - 1;
#pragma unroll 1
    for (int round = 0; round < rounds; ++round, t += stride, dx += next_dx) {
        const int mine = t < a.n ? heads : 0;  // heads of this token
        float cc[8], ss[8];
        int from = lane;
        if (mine) from = turn_of<MODE>(a, pos, c, lane, cc, ss);
        else {
#pragma unroll
            for (int e = 0; e < 8; ++e) cc[e] = ss[e] = 0.f;
        }
        pos = ahead(t + stride);
        F2 cs[4], sn[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            cs[e] = f2(cc[2 * e] * s.scale, cc[2 * e + 1] * s.scale);
            sn[e] = f2(-ss[2 * e] * s.scale, -ss[2 * e + 1] * s.scale);  // R^T: the sine with the other sign
        }
#pragma unroll 1
        for (int h = 0; h < chunk; ++h, dx += a.d) {
            cp_async_wait<S - 2>();
            Raw<T> ux, uy;
            ux.load_pieces(ring + stage * 2 * W * kThreads + threadIdx.x, kThreads);
            uy.load_pieces(ring + (stage * 2 + 1) * W * kThreads + threadIdx.x, kThreads);
            load(into);
            into = stage;
            stage = stage + 1 == S ? 0 : stage + 1;
            const Raw<T> p = partners<T, MODE>(uy, from);
            F2 u[4], uw[4], sum = f2(0.f, 0.f), dot = f2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                u[e] = f2_mul(uy.pair(e), cs[e]);
                if (MODE != kNoTurn) u[e] = f2_fma(p.pair(e), sn[e], u[e]);
                uw[e] = f2_mul(u[e], w[e]);
                sum = f2_fma(ux.pair(e), ux.pair(e), sum);
                dot = f2_fma(uw[e], ux.pair(e), dot);  // of x: of n it is r times that
            }
            const float2 sums = f2_parts(sum), dots = f2_parts(dot);
            F2 both = group_sum2<LANES>(f2(sums.x + sums.y, dots.x + dots.y));
            float2 all = f2_parts(both);
            float r = rsqrtf(fmaf(all.x, share, a.eps)), r_out = r;
            const bool out = !(all.x < 1e37f);
            if (__any_sync(~0u, out)) {  // squares that leave 32 bits: the same from 2^-80 x, exact in T
                Raw<T> small = ux;
                small.scale(0x1p-80f);
                sum = dot = f2(0.f, 0.f);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    sum = f2_fma(small.pair(e), small.pair(e), sum);
                    dot = f2_fma(uw[e], small.pair(e), dot);
                }
                const float2 s2 = f2_parts(sum), d2 = f2_parts(dot);
                const float2 again = f2_parts(group_sum2<LANES>(f2(s2.x + s2.y, d2.x + d2.y)));
                if (out) {
                    ux = small;
                    all.y = again.y;
                    r = rsqrtf(fmaf(again.x, share, small_eps(a.eps)));
                    r_out = 0x1p-80f * r;
                }
            }
            const float m = -share * r * all.y;
            const F2 r2 = f2(r, r), m2 = f2(m, m), ro = f2(r_out, r_out);
            float o[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {  // heads past the end are zeros: they add none to dw
                const F2 n = f2_mul(ux.pair(e), r2);
                dw[e] = f2_fma(u[e], n, dw[e]);
                const float2 y = f2_parts(f2_mul(ro, f2_fma(n, m2, uw[e])));
                o[2 * e] = y.x;
                o[2 * e + 1] = y.y;
            }
            if (h < mine) store8(dx, o);
        }
    }
    cp_async_wait<0>();
    if (!part_sums) return;
    __shared__ float s_dw[kThreads / 32][LANES * 8];
    // groups of the warp, then warps, then (qk_dw_kernel) CTAs
    float all[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 y = f2_parts(dw[e]);
        all[2 * e] = y.x;
        all[2 * e + 1] = y.y;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int o = LANES; o < 32; o <<= 1) all[e] += __shfl_xor_sync(~0u, all[e], o);
    if (lane < LANES) {
#pragma unroll
        for (int e = 0; e < 8; ++e) s_dw[threadIdx.x / 32][c + e] = all[e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.d; i += kThreads) {
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < kThreads / 32; ++k) sum += s_dw[k][i];
        part_sums[(size_t)blockIdx.x * a.d + i] = sum;
    }
}

// Sums the CTAs' parts, in a fixed order: block (side, 32 channels), 32 rows of threads.
__global__ void __launch_bounds__(1024) qk_dw_kernel(const float* part, float* dwq, float* dwk, int q_ctas, int ctas, int d) {
    __shared__ float s[32][33];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float* dw = blockIdx.x == 0 ? dwq : dwk;
    if (!dw) return;
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.y * 32 + x;
    const int b = blockIdx.x == 0 ? 0 : q_ctas, e = blockIdx.x == 0 ? q_ctas : ctas;
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < (int)(kBwdCtas + 31) / 32; ++k) {  // all loads at once
        const int i = b + y + 32 * k;
        sum += c < d && i < e ? part[(size_t)i * d + c] : 0.f;
    }
    s[y][x] = sum;
    __syncthreads();
    sum = warp_sum(s[x][y]);  // channel y of the block
    if (x == 0 && blockIdx.y * 32 + y < d) dw[blockIdx.y * 32 + y] = sum;
}


template <typename F> cudaError_t with_lanes(int d, F f) {
    if (d <= 8) return f(std::integral_constant<int, 1>());
    if (d <= 16) return f(std::integral_constant<int, 2>());
    if (d <= 32) return f(std::integral_constant<int, 4>());
    if (d <= 64) return f(std::integral_constant<int, 8>());
    if (d <= 128) return f(std::integral_constant<int, 16>());
    return f(std::integral_constant<int, 32>());
}
template <typename F> cudaError_t with_mode(const QkArgs& a, F f) {
    if (!a.positions) return f(std::integral_constant<int, kNoTurn>());
    return a.interleaved ? f(std::integral_constant<int, kPairs>()) : f(std::integral_constant<int, kHalves>());
}

}  // namespace

size_t qk_norm_rope_bwd_workspace_bytes(int n, int Hq, int Hk, int d) {
    (void)n; (void)Hq; (void)Hk;
    return (size_t)kBwdCtas * d * sizeof(float);
}

cudaError_t launch_qk_norm_rope(const QkArgs& a, cudaStream_t stream) {
    return with_lanes(a.d, [&](auto lanes) {
        return with_mode(a, [&](auto mode) {
            constexpr int L = decltype(lanes)::value, M = decltype(mode)::value, GROUPS = kThreads / L;
            // heads of a group: 8 where that still gives every SM 32 warps, fewer for few tokens
            int chunk = 8;
            auto items = [&] { return (long long)a.n * ((a.Hq + chunk - 1) / chunk + (a.Hk + chunk - 1) / chunk); };
            while (chunk > 1 && items() * L < 148ll * 1024) chunk /= 2;
            const int q_chunks = (a.Hq + chunk - 1) / chunk, chunks = q_chunks + (a.Hk + chunk - 1) / chunk;
            const unsigned blocks = (unsigned)((items() + GROUPS - 1) / GROUPS);
            if (a.bf16) qk_fwd_kernel<__nv_bfloat16, L, M><<<blocks, kThreads, 0, stream>>>(a, chunk, q_chunks, chunks);
            else qk_fwd_kernel<float, L, M><<<blocks, kThreads, 0, stream>>>(a, chunk, q_chunks, chunks);
            return cudaGetLastError();
        });
    });
}

cudaError_t launch_qk_norm_rope_bwd(const QkArgs& a, cudaStream_t stream) {
    float* part = a.d_q_weight || a.d_k_weight ? (float*)a.workspace : nullptr;
    int q_ctas = 0, ctas = 0;
    const cudaError_t err = with_lanes(a.d, [&](auto lanes) {
        return with_mode(a, [&](auto mode) {
            constexpr int L = decltype(lanes)::value, M = decltype(mode)::value, GROUPS = kThreads / L;
            // Heads of a group: up to 8, in equal parts; fewer where there are few tokens, more where there are so many
            // heads that their parts would outnumber the groups.
            int most = std::max(8, (a.Hq + a.Hk + 63) / 64);
            auto parts_of = [&](int H) { return (H + most - 1) / most; };
            auto parts = [&] { return (long long)parts_of(a.Hq) + parts_of(a.Hk); };
            while (most > 1 && a.n * parts() * L < 148ll * 512 && 2 * parts() + 2 <= 148 * GROUPS) most /= 2;
            auto chunk_of = [&](int H) { return H ? (H + parts_of(H) - 1) / parts_of(H) : 1; };
            // CTAs of each side in the ratio of its work: groups for every part at least, for every part of a token at most
            auto fewest = [&](int H) { return ((long long)parts_of(H) + GROUPS - 1) / GROUPS; };
            auto useful = [&](int H) { return ((long long)a.n * parts_of(H) + GROUPS - 1) / GROUPS; };
            const long long q_work = (long long)parts_of(a.Hq) * chunk_of(a.Hq), work = q_work + (long long)parts_of(a.Hk) * chunk_of(a.Hk);
            if (a.n == 0 || work == 0) return cudaSuccess;
            const long long q = std::min(std::max(kBwdCtas * q_work / work, fewest(a.Hq)), kBwdCtas - fewest(a.Hk));
            q_ctas = (int)std::min(q, useful(a.Hq));
            const int k_ctas = (int)std::min(kBwdCtas - q_ctas, useful(a.Hk));
            ctas = q_ctas + k_ctas;
            static std::atomic<unsigned long long> raised[2];  // of this size and mode: float, bf16
            auto go = [&](auto kernel, int smem) {
                const cudaError_t e = allow_smem(kernel, smem, raised[a.bf16]);
                if (e != cudaSuccess) return e;
                kernel<<<ctas, kThreads, smem, stream>>>(a, chunk_of(a.Hq), chunk_of(a.Hk), q_ctas, part);
                return cudaGetLastError();
            };
            if (a.bf16) return go(qk_bwd_kernel<__nv_bfloat16, L, M>, BwdPlan<__nv_bfloat16>::kSmem);
            return go(qk_bwd_kernel<float, L, M>, BwdPlan<float>::kSmem);
        });
    });
    if (err != cudaSuccess || !part) return err;
    // launched while the first kernel runs; it waits for its end there
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2, (a.d + 31) / 32);
    cfg.blockDim = dim3(1024);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, qk_dw_kernel, (const float*)part, a.d_q_weight, a.d_k_weight, q_ctas, ctas, a.d);
}

}  // namespace kda
