// Attention of one new token per sequence over a paged key-value cache.
//
//     o = sum_p e^{s_p - m} v_p / sum_p e^{s_p - m},   s_p = scale q.k_p,  m = max_p s_p
//
// with the running maximum and sum of a softmax that is read once: every key
// and value row is loaded once and meets all query heads that share it.
//
// What bounds it: HBM. A context position costs 2 d elements of cache per
// key-value head and 4 d flop per query head, so the products run on warp MMAs
// (16 query heads x 16 positions; fewer heads leave rows empty, which costs
// nothing while the loads set the pace).
//
// Split: the positions of all (sequence, key-value head, block of 16 query
// heads) are cut into tiles of 16, and the list of all tiles is cut into equal
// contiguous ranges, one per warp ("worker"), whatever the lengths are: a
// batch of one long and many short contexts loads every SM alike. Workers find
// their range from seq_lens on the device. A worker that holds all tiles of a
// pair writes its output; else it leaves (m, l, O) in the workspace, where it
// has two places: 0 for a range that continues a pair, 1 for one that begins a
// pair and does not end it. attn_join_kernel joins the pieces in order. A warp
// works for itself (no block barrier in the loop): it copies 16 rows of K and V
// a stage with 16-byte cp.async, several stages ahead, across the ends of pairs.
#include "kda_common.cuh"
#include "kda_internal.h"
#include "kda_sm100.cuh"

namespace kda {

namespace {

constexpr int kTile = 16;                          // positions of a tile
constexpr int kHeads = 16;                         // query heads of a block (rows of the MMA)
constexpr int kWarps = 4;                          // workers of a CTA
constexpr int kCtas = 296;                         // two on each of 148 SMs
constexpr int kWorkers = kCtas * kWarps;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// The attended positions [first, last) of a row, and its number of tiles.
struct Row {
    int held, first, last, tiles;
};

__device__ __forceinline__ Row row_of(const AttnDecodeArgs& a, int n) {
    Row r;
    r.held = a.seq_lens[n];
    const bool put = a.k_new != nullptr && r.held >= 0;
    const long long total = r.held < 0 ? 0 : (long long)r.held + (put ? 1 : 0);  // a length near 2^31 must not wrap
    r.last = (int)min(total, (long long)a.max_pages * a.page_size);
    r.first = a.window ? (int)min(max(0ll, total - a.window), (long long)r.last) : 0;
    r.tiles = (r.last - r.first + kTile - 1) / kTile;
    return r;
}

// Workspace: per (worker, place) the pieces' O [heads][D], then their (m, l)
// [heads], then per pair the worker that begins it and its number of pieces.
struct Pieces {
    float* o;
    float2* ml;
    int2* pair;
    int rows;
};

__host__ __device__ __forceinline__ Pieces pieces_of(void* ws, int G, int D) {
    Pieces p;
    p.rows = G < kHeads ? G : kHeads;
    p.o = (float*)ws;
    p.ml = (float2*)(p.o + (size_t)2 * kWorkers * p.rows * D);
    p.pair = (int2*)(p.ml + (size_t)2 * kWorkers * p.rows);
    return p;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

template <int D> struct Bf16Stage {
    static constexpr int kRowBytes = D * 2, kBytes = 2 * kTile * kRowBytes;  // K then V
    static constexpr int kStages = 24576 / kBytes;                          // 24 KB a warp: 3 (D = 128) or 6
};

template <int D>
constexpr int attn_smem_bytes() {
    return kWarps * Bf16Stage<D>::kStages * (Bf16Stage<D>::kBytes + 16);
}

// HALF: at most 8 query heads, so rows 8..15 of the MMA are empty.
template <int D, bool HALF>
__global__ void __launch_bounds__(kWarps * 32, 2) attn_split_kernel(AttnDecodeArgs a) {
    using St = Bf16Stage<D>;
    using T = __nv_bfloat16;
    constexpr int S = St::kStages, RB = St::kRowBytes, CH = RB / 16;  // 16-byte chunks of a row
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ long long s_part[kWarps], s_rem[kWarps];
    __shared__ int s_row[kWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = a.Hq / a.Hk, blocks = (G + kHeads - 1) / kHeads, P = a.Hk * blocks;
    const Pieces ws = pieces_of(a.workspace, G, D);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // Tiles of all rows before thread tid's rows, and of all rows.
    const int per = (a.N + kWarps * 32 - 1) / (kWarps * 32), row0 = min(tid * per, a.N), row1 = min(row0 + per, a.N);
    long long mine = 0;
    for (int n = row0; n < row1; ++n) mine += row_of(a, n).tiles;
    mine *= P;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(~0u, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) s_part[warp] = incl;
    __syncthreads();
    long long total = 0, before = incl - mine;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_part[w];
        total += s_part[w];
    }
    const long long W = max(1ll, (total + kWorkers - 1) / kWorkers);  // tiles of a worker
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        long long u = (long long)(blockIdx.x * kWarps + w) * W;
        if (u >= before && u < before + mine) {
            u -= before;
            int n = row0;
            for (long long tiles; u >= (tiles = (long long)row_of(a, n).tiles * P); ++n) u -= tiles;
            s_row[w] = n;
            s_rem[w] = u;
        }
    }
    // rows without any attended position
    for (int n = blockIdx.x; n < a.N; n += gridDim.x) {
        if (row_of(a, n).tiles) continue;
        uint4* o = (uint4*)((T*)a.o + (size_t)n * a.Hq * D);
        for (int i = tid; i < a.Hq * CH; i += kWarps * 32) o[i] = make_uint4(0, 0, 0, 0);
        for (int i = tid; i < a.Hq; i += kWarps * 32)
            if (a.lse) a.lse[(size_t)n * a.Hq + i] = -INFINITY;
        for (int i = tid; i < P; i += kWarps * 32) ws.pair[(size_t)n * P + i] = make_int2(0, 0);
    }
    __syncthreads();

    const int worker = blockIdx.x * kWarps + warp;
    if ((long long)worker * W >= total) return;
    const int count = (int)min(W, total - (long long)worker * W);
    unsigned char* ring = smem + (size_t)warp * S * St::kBytes;
    int4* metas = reinterpret_cast<int4*>(smem + (size_t)kWarps * S * St::kBytes) + warp * S;
    const uint32_t ring_u32 = sm100::smem_u32(ring);

    // ---- the loading side: tile t of pair p of row n, `left` tiles to go
    int n = s_row[warp], left = count;
    Row row = row_of(a, n);
    int p = (int)(s_rem[warp] / row.tiles), t = (int)(s_rem[warp] % row.tiles);
    bool began = t == 0;     // this worker holds the pair's first tile
    bool fresh = true;       // the next tile begins a range of one pair
    int page = -1;           // of position first + 16 t + lane (lanes 0..15)
    auto look_up = [&]() {
        const int pos = row.first + t * kTile + (lane & 15);
        page = pos < row.last ? a.page_table[(size_t)n * a.max_pages + pos / a.page_size] : -1;
    };
    look_up();
    auto issue = [&](int stage) {
        if (left > 0) {
            const int hk = p / blocks, hb = p % blocks;
            const int pos = row.first + t * kTile + (lane & 15);
            const bool valid = page >= 0 && page < a.n_pages;
            const bool fresh_token = valid && a.k_new && pos == row.held;
            const long long at = valid ? (((long long)page * a.Hk + hk) * a.page_size + pos % a.page_size) * D : -1;
            const unsigned mask = __ballot_sync(~0u, valid && lane < 16), news = __ballot_sync(~0u, fresh_token && lane < 16);
            const int new_row = news ? __ffs(news) - 1 : -1;
            const uint32_t dst = ring_u32 + stage * St::kBytes;
            const size_t new_at = ((size_t)n * a.Hk + hk) * D;
            const int c = lane % CH;
#pragma unroll
            for (int i = 0; i < kTile * CH / 32; ++i) {
                const int r = i * (32 / CH) + lane / CH;
                const long long src = __shfl_sync(~0u, at, r);
                const bool is_new = r == new_row, on = src >= 0;
                const T* kp = is_new ? (const T*)a.k_new + new_at : (const T*)a.k_cache + (on ? src : 0);
                const T* vp = is_new ? (const T*)a.v_new + new_at : (const T*)a.v_cache + (on ? src : 0);
                const uint32_t to = dst + r * RB + ((c ^ (r & 7)) << 4);
                cp_async16(to, kp + c * 8, on);
                cp_async16(to + kTile * RB, vp + c * 8, on);
            }
            if (news && hb == 0) {  // put the new token's key and value where the table says
                const long long to = __shfl_sync(~0u, at, new_row);
                for (int i = lane; i < 2 * CH; i += 32) {
                    const bool v = i >= CH;
                    const int e = (v ? i - CH : i) * 8;
                    *reinterpret_cast<uint4*>((T*)(v ? a.v_cache : a.k_cache) + to + e) =
                        *reinterpret_cast<const uint4*>((const T*)(v ? a.v_new : a.k_new) + new_at + e);
                }
            }
            const bool pair_ends = t + 1 == row.tiles, range_ends = pair_ends || left == 1;
            if (lane == 0) {
                const int place = began ? (pair_ends ? 2 : 1) : 0;  // 2: the whole pair
                metas[stage] = make_int4(n, p, mask | (fresh ? 1u << 16 : 0) | (range_ends ? 1u << 17 : 0) | place << 18, 0);
                if (t == 0)
                    ws.pair[(size_t)n * P + p] =
                        make_int2(worker, row.tiles <= left ? 1 : 1 + (int)((row.tiles - left + W - 1) / W));
            }
            --left;
            fresh = range_ends;
            if (!pair_ends) {
                ++t;
            } else if (left > 0) {
                t = 0;
                began = true;
                if (++p == P) {
                    p = 0;
                    do row = row_of(a, ++n);
                    while (row.tiles == 0);  // tiles are left, so a row with some follows
                }
            }
            if (left > 0) look_up();
        }
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < S - 1; ++s) issue(s);

    // ---- the computing side
    const float scale2 = a.scale * kLog2e;
    const int g = lane >> 2, c2 = (lane & 3) * 2;
    uint32_t qf[D / 16][4];
    float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    // ldmatrix rows of this lane: for K (positions x channels) and, transposed, for V
    const int mat = lane >> 3, r8 = lane & 7;
    const uint32_t k_row = (r8 + (mat >> 1) * 8) * RB, v_row = (r8 + (mat & 1) * 8) * RB;
    int stage = 0, into = S - 1;
    for (int step = 0; step < count; ++step) {
        cp_async_wait<S - 2>();
        __syncwarp();
        issue(into);
        into = into + 1 == S ? 0 : into + 1;
        const int4 meta = metas[stage];
        const uint32_t kt = ring_u32 + stage * St::kBytes, vt = kt + kTile * RB;
        const int hk = meta.y / blocks, hb = meta.y % blocks, heads = min(kHeads, G - hb * kHeads);
        const size_t out_row = (size_t)meta.x * a.Hq + (size_t)hk * G + hb * kHeads;  // of head 0
        if (meta.z & (1 << 16)) {
            const T* q = (const T*)a.q + out_row * D;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                const int at = ks * 16 + c2;
                qf[ks][0] = g < heads ? *reinterpret_cast<const uint32_t*>(q + g * D + at) : 0u;
                qf[ks][2] = g < heads ? *reinterpret_cast<const uint32_t*>(q + g * D + at + 8) : 0u;
                qf[ks][1] = !HALF && g + 8 < heads ? *reinterpret_cast<const uint32_t*>(q + (g + 8) * D + at) : 0u;
                qf[ks][3] = !HALF && g + 8 < heads ? *reinterpret_cast<const uint32_t*>(q + (g + 8) * D + at + 8) : 0u;
            }
#pragma unroll
            for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
            m[0] = m[1] = -INFINITY;
            l[0] = l[1] = 0.f;
        }
        float s[2][4] = {};
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            uint32_t b[4];
            ldsm4(b, kt + k_row + (((2 * ks + (mat & 1)) ^ r8) << 4));
            mma_bf16(s[0], qf[ks], b[0], b[1]);
            mma_bf16(s[1], qf[ks], b[2], b[3]);
        }
        // scores in log2 units; positions that are not attended: -infinity
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s[j][e] = (meta.z >> (j * 8 + c2 + (e & 1))) & 1 ? s[j][e] * scale2 : -INFINITY;
        float keep[2] = {1.f, 1.f};
#pragma unroll
        for (int h = 0; h < (HALF ? 1 : 2); ++h) {
            float top = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
            top = fmaxf(fmaxf(top, __shfl_xor_sync(~0u, top, 2)), m[h]);
            const float base = top == -INFINITY ? 0.f : top;  // nothing attended so far: weights of 0
            keep[h] = exp2_fast(m[h] - base);
            m[h] = top;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                s[j][2 * h] = exp2_fast(s[j][2 * h] - base);
                s[j][2 * h + 1] = exp2_fast(s[j][2 * h + 1] - base);
                sum += s[j][2 * h] + s[j][2 * h + 1];
            }
            l[h] = fmaf(l[h], keep[h], sum);
        }
        if (__any_sync(~0u, keep[0] != 1.f || keep[1] != 1.f)) {
#pragma unroll
            for (int j = 0; j < D / 8; ++j) {
                o[j][0] *= keep[0];
                o[j][1] *= keep[0];
                if (!HALF) {
                    o[j][2] *= keep[1];
                    o[j][3] *= keep[1];
                }
            }
        }
        // the weights as the left operand (bf16, at most half a step off each; l sums them unrounded)
        const uint32_t pf[4] = {pack_bf16(s[0][0], s[0][1]), HALF ? 0u : pack_bf16(s[0][2], s[0][3]),
                                pack_bf16(s[1][0], s[1][1]), HALF ? 0u : pack_bf16(s[1][2], s[1][3])};
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            uint32_t b[4];
            ldsm4_trans(b, vt + v_row + (((2 * j + (mat >> 1)) ^ r8) << 4));
            mma_bf16(o[2 * j], pf, b[0], b[1]);
            mma_bf16(o[2 * j + 1], pf, b[2], b[3]);
        }
        if (meta.z & (1 << 17)) {
            const int place = meta.z >> 18;
#pragma unroll
            for (int h = 0; h < (HALF ? 1 : 2); ++h) {
                float sum = l[h];
                sum += __shfl_xor_sync(~0u, sum, 1);
                sum += __shfl_xor_sync(~0u, sum, 2);
                const int head = g + 8 * h;
                if (head >= heads) continue;
                if (place == 2) {
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;
                    uint32_t* to = reinterpret_cast<uint32_t*>((T*)a.o + (out_row + head) * D + c2);
#pragma unroll
                    for (int j = 0; j < D / 8; ++j) to[j * 4] = pack_bf16(o[j][2 * h] * inv, o[j][2 * h + 1] * inv);
                    if (a.lse && (lane & 3) == 0)
                        a.lse[out_row + head] = sum == 0.f ? -INFINITY : fmaf(m[h], kLn2, logf(sum));
                } else {
                    const size_t at = (size_t)(2 * worker + place) * ws.rows + head;
                    float* to = ws.o + at * D + c2;
#pragma unroll
                    for (int j = 0; j < D / 8; ++j)
                        *reinterpret_cast<float2*>(to + j * 8) = make_float2(o[j][2 * h], o[j][2 * h + 1]);
                    if ((lane & 3) == 0) ws.ml[at] = make_float2(m[h], sum);
                }
            }
        }
        stage = stage + 1 == S ? 0 : stage + 1;
    }
    cp_async_wait<0>();
}

// Joins the pieces of every pair that lies in several workers, in their order:
// piece 0 in place 1 of the worker that begins the pair, the others in place 0
// of the workers after it. blockIdx.x: a run of `chunk` pairs; blockIdx.y: heads.
constexpr int kJoinWarps = 8;

template <typename T, int D>
__global__ void __launch_bounds__(kJoinWarps * 32) attn_join_kernel(AttnDecodeArgs a, int pairs, int chunk) {
    constexpr int E = D / 32;
    __shared__ float so[kJoinWarps][D], sl[kJoinWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = a.Hq / a.Hk, blocks = (G + kHeads - 1) / kHeads, P = a.Hk * blocks;
    const Pieces ws = pieces_of(a.workspace, G, D);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ int2 found[kJoinWarps * 32];
    const int begin = blockIdx.x * chunk, end = min(begin + chunk, pairs);
    for (int i = begin, from = begin; i < end; ++i) {
        if (i == from) {  // the next 256 pairs; most of them lie in one worker
            const int2 mine = i + (int)threadIdx.x < end ? ws.pair[i + threadIdx.x] : make_int2(0, 0);
            found[threadIdx.x] = mine;
            from += kJoinWarps * 32;
            const bool some = __syncthreads_or(mine.y > 1);
            if (!some) {
                i = from - 1;
                continue;
            }
        }
        const int2 pair = found[(i - begin) % (kJoinWarps * 32)];
        if (i + 1 == from) __syncthreads();  // all have read it before the next 256 replace it
        if (pair.y < 2) continue;
        const int n = i / P, p = i % P, hk = p / blocks, hb = p % blocks, heads = min(kHeads, G - hb * kHeads);
        for (int h = blockIdx.y; h < heads; h += gridDim.y) {
            auto slot = [&](int k) { return (size_t)(2 * (pair.x + k) + (k == 0 ? 1 : 0)) * ws.rows + h; };
            float top = -INFINITY;
            for (int k = lane; k < pair.y; k += 32) top = fmaxf(top, ws.ml[slot(k)].x);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
            const float base = top == -INFINITY ? 0.f : top;
            float acc[E] = {}, l = 0.f;
#pragma unroll 4
            for (int k = warp; k < pair.y; k += kJoinWarps) {
                const size_t at = slot(k);
                const float2 ml = ws.ml[at];
                const float f = exp2_fast(ml.x - base);
                l = fmaf(ml.y, f, l);
                const float* from = ws.o + at * D + lane * E;
                if constexpr (E == 4) {
                    const float4 x = *reinterpret_cast<const float4*>(from);
                    acc[0] = fmaf(x.x, f, acc[0]); acc[1] = fmaf(x.y, f, acc[1]);
                    acc[2] = fmaf(x.z, f, acc[2]); acc[3] = fmaf(x.w, f, acc[3]);
                } else {
                    const float2 x = *reinterpret_cast<const float2*>(from);
                    acc[0] = fmaf(x.x, f, acc[0]); acc[1] = fmaf(x.y, f, acc[1]);
                }
            }
#pragma unroll
            for (int e = 0; e < E; ++e) so[warp][lane * E + e] = acc[e];
            if (lane == 0) sl[warp] = l;
            __syncthreads();
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < kJoinWarps; ++w) sum += sl[w];
            const size_t out = (size_t)n * a.Hq + (size_t)hk * G + hb * kHeads + h;
            for (int c = threadIdx.x; c < D; c += kJoinWarps * 32) {
                float x = 0.f;
#pragma unroll
                for (int w = 0; w < kJoinWarps; ++w) x += so[w][c];
                ((T*)a.o)[out * D + c] = from_f32<T>(sum == 0.f ? 0.f : x / sum);
            }
            if (a.lse && threadIdx.x == 0) a.lse[out] = sum == 0.f ? -INFINITY : fmaf(top, kLn2, logf(sum));
            __syncthreads();
        }
    }
}

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
    const int G = Hq / Hk, blocks = (G + kHeads - 1) / kHeads;
    const Pieces p = pieces_of(nullptr, G, d);
    return (size_t)((char*)(p.pair + (size_t)N * Hk * blocks) - (char*)nullptr);
}

template <int D>
static cudaError_t launch_attn_bf16(const AttnDecodeArgs& a, cudaStream_t stream) {
    const int G = a.Hq / a.Hk, pairs = a.N * a.Hk * ((G + kHeads - 1) / kHeads);
    auto split = G <= 8 ? attn_split_kernel<D, true> : attn_split_kernel<D, false>;
    constexpr int smem = attn_smem_bytes<D>();
    cudaError_t err = cudaFuncSetAttribute(split, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
    split<<<kCtas, kWarps * 32, smem, stream>>>(a);
    if ((err = cudaGetLastError()) != cudaSuccess) return err;
    // The join starts while the split kernel runs (programmatic dependent launch) and waits for its end there.
    const int chunk = (pairs + kWorkers - 1) / kWorkers;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((pairs + chunk - 1) / chunk, pairs < 148 ? (G < kHeads ? G : kHeads) : 1);
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_join_kernel<__nv_bfloat16, D>, a, pairs, chunk);
}

cudaError_t launch_attn_decode(const AttnDecodeArgs& a, cudaStream_t stream) {
    if (a.bf16) return a.d == 64 ? launch_attn_bf16<64>(a, stream) : launch_attn_bf16<128>(a, stream);
    const unsigned blocks = (unsigned)a.N * a.Hq;
    if (a.d == 64) attn_decode_kernel<float, 64><<<blocks, 128, 0, stream>>>(a);
    else attn_decode_kernel<float, 128><<<blocks, 128, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace kda
