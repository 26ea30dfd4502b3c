// Attention of one new token per sequence over a paged key-value cache.
//
//     o = sum_p e^{s_p - m} v_p / sum_p e^{s_p - m},   s_p = scale q.k_p,  m = max_p s_p
//
// with the running maximum and sum of a softmax that is read once: every key
// and value row is loaded once and meets all query heads that share it.
//
// What bounds it: HBM. A context position costs 2 d elements of cache per
// key-value head and 4 d flop per query head, so the products run on warp MMAs
// (16 positions x 8 or 16 query heads; fewer heads leave columns empty, which
// costs nothing while the loads set the pace). 64 rows of 256 to 16384 positions,
// 8 key-value heads, d 128, bf16: 170-172 us, 0.93-0.94 of the measured copy
// bandwidth, the tensor pipe 13 % busy.
//
// Split: the positions of all (sequence, key-value head, block of 16 query
// heads) are cut into tiles of 16, and the list of all tiles is cut into equal
// contiguous ranges, one per warp ("worker"), whatever the lengths are: a
// batch of one long and many short contexts loads every SM alike in this kernel.
// (To begin and to end a pair costs as much as some tiles, so each pair counts
// kBegin more.) The join's warps go by the number of pairs, so one very long
// context among many has its many pieces joined by one warp a head (131072
// positions and 63 rows of 256: 124 us, 0.75 of the copy bandwidth).
// Workers find their range from seq_lens on the device. A worker that holds all
// tiles of a pair writes its output; else it leaves (m, l, O) in the workspace,
// where it has two places: 0 for a range that continues a pair, 1 for one that begins a
// pair and does not end it. attn_join_kernel joins the pieces in order. A warp
// works for itself (no block barrier in the loop): it copies 16 rows of K and V
// a stage with 16-byte cp.async, several stages ahead, across the ends of pairs.
#include "kda_async.cuh"
#include "kda_common.cuh"
#include "kda_internal.h"
#include "kda_sm100.cuh"

namespace kda {

namespace {

constexpr int kTile = 16;   // positions of a tile
constexpr int kHeads = 16;  // query heads of a block
constexpr int kBegin = 3;   // what a pair costs beside its tiles, in tiles (256 rows of 0 to 300: with 1 24.9 us, 3 21.4, 6 23.6)
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Stages of a worker's ring, workers of a CTA and CTAs of an SM: 190 to 220 KB
// of cache rows an SM, by as many warps as the registers allow.
template <typename T, int D> struct Plan;
template <> struct Plan<__nv_bfloat16, 128> { static constexpr int kStages = 3, kWarps = 4, kCtasPerSm = 2; };
template <> struct Plan<__nv_bfloat16, 64> { static constexpr int kStages = 4, kWarps = 4, kCtasPerSm = 3; };
template <> struct Plan<float, 128> { static constexpr int kStages = 2, kWarps = 7, kCtasPerSm = 1; };
template <> struct Plan<float, 64> { static constexpr int kStages = 2, kWarps = 6, kCtasPerSm = 2; };

template <typename T, int D> struct Geometry : Plan<T, D> {
    static constexpr int kRowBytes = D * (int)sizeof(T), kChunks = kRowBytes / 16;
    static constexpr int kStageBytes = 2 * kTile * kRowBytes;  // K then V
    using Plan<T, D>::kWarps;
    static constexpr int kCtas = 148 * Plan<T, D>::kCtasPerSm, kWorkers = kCtas * kWarps;
    static constexpr int kSmem = kWarps * Plan<T, D>::kStages * (kStageBytes + 16);
};

int workers_of(int bf16, int d) {
    if (bf16) return d == 64 ? Geometry<__nv_bfloat16, 64>::kWorkers : Geometry<__nv_bfloat16, 128>::kWorkers;
    return d == 64 ? Geometry<float, 64>::kWorkers : Geometry<float, 128>::kWorkers;
}

// The attended positions [first, last) of a row, and its number of tiles.
struct Row {
    int held, first, last, tiles;
};

__device__ __forceinline__ Row row_from(const AttnDecodeArgs& a, int held) {
    Row r;
    r.held = held;
    const bool put = a.k_new != nullptr && held >= 0;
    const long long total = held < 0 ? 0 : (long long)held + (put ? 1 : 0);  // a length near 2^31 must not wrap
    r.last = (int)min(total, (long long)a.max_pages * a.page_size);
    r.first = a.window ? (int)min(max(0ll, total - a.window), (long long)r.last) : 0;
    r.tiles = (r.last - r.first + kTile - 1) / kTile;
    return r;
}
__device__ __forceinline__ Row row_of(const AttnDecodeArgs& a, int n) { return row_from(a, a.seq_lens[n]); }
// A pair of this row in the list of all work: kBegin units, then its tiles.
__device__ __forceinline__ int units_of(const Row& r) { return r.tiles ? r.tiles + kBegin : 0; }

// Workspace: per (worker, place) the pieces' O [heads][D], then their (m, l)
// [heads], then per pair the worker that begins it and its number of pieces.
struct Pieces {
    float* o;
    float2* ml;
    int2* pair;
    int rows;
};

__host__ __device__ __forceinline__ Pieces pieces_of(void* ws, int workers, int G, int D) {
    Pieces p;
    p.rows = G < kHeads ? G : kHeads;
    p.o = (float*)ws;
    p.ml = (float2*)(p.o + (size_t)2 * workers * p.rows * D);
    p.pair = (int2*)(p.ml + (size_t)2 * workers * p.rows);
    return p;
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

// Two weights as two bf16 parts each, hi and lo = x - hi rounded, together off by 2^-16 x at most. hi is x cut to bf16 from
// just below, so that lo is above 0 too (in bf16, for x above 2^-110): an infinite value keeps its sign.
__device__ __forceinline__ void split_bf16(float x0, float x1, uint32_t& hi, uint32_t& lo) {
    const uint32_t h0 = __float_as_uint(x0 * (1.f - 0x1p-23f)), h1 = __float_as_uint(x1 * (1.f - 0x1p-23f));
    hi = __byte_perm(h0, h1, 0x7632);
    lo = pack_bf16(x0 - __uint_as_float(h0 & 0xffff0000u), x1 - __uint_as_float(h1 & 0xffff0000u));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x = hi + lo: hi is x rounded to tf32's 11 significant bits, lo the rest. The MMA ignores lo's bits past its own 11,
// 2^-22 |x| at most. An infinity goes into lo alone: products with the other operand's hi then have its sign, and there
// is no infinity times a part that happens to be zero.
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
    hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    if (!(fabsf(x) < INFINITY)) hi = 0u;
    lo = __float_as_uint(x - __uint_as_float(hi));
}
__device__ __forceinline__ float lds_f32(uint32_t at) {
    float x;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(at) : "memory");
    return x;
}

// What the loading side tells the computing side about a stage's tile.
struct Tile {
    int out_row;    // n Hq + first query head of the block
    int heads;      // of the block
    unsigned bits;  // attended positions (0..15), kFresh, kEnds, place (2: a whole pair)
};
constexpr unsigned kFresh = 1u << 16, kEnds = 1u << 17;
constexpr int kPlaceShift = 18;

// The loading side of a worker: walks the tiles of its range and fills the ring.
template <typename T, int D>
struct Feed {
    using Geo = Geometry<T, D>;
    const AttnDecodeArgs& a;
    int2* pair_out;
    uint32_t ring;
    int4* metas;
    int worker, lane, G, blocks;
    long long W;
    // tile t of pair (hk, hb) of row n, `left` units to go (0: the range is done)
    int n, hk, hb, t, left, issued;
    Row row;
    int next_held;       // of row n + 1, loaded ahead
    bool began, fresh;   // this worker holds the pair's first tile; the next tile begins a range of one pair
    int page_at, off;    // lanes 0..15 (16..31 alike): the position's entry in the table, and its row in the page
    int from, pages, pages2;  // lane i holds the table's entries from + i and from + 32 + i

    __device__ __forceinline__ int entry(int i) const {
        return i < a.max_pages ? a.page_table[(size_t)n * a.max_pages + i] : -1;
    }
    __device__ __forceinline__ void place_tile() {
        const int pos = row.first + t * kTile + (lane & 15);
        page_at = pos / a.page_size;
        off = pos - page_at * a.page_size;
    }
    __device__ __forceinline__ void fetch_pages(bool anew) {
        const int p0 = __shfl_sync(~0u, page_at, 0);
        if (anew || p0 < from || p0 >= from + 64) {
            from = p0 & ~31;
            pages = entry(from + lane);
            pages2 = entry(from + 32 + lane);
        } else if (p0 >= from + 32) {
            from += 32;
            pages = pages2;
            pages2 = entry(from + 32 + lane);
        }
    }
    // `count` units from unit `rem` of row n_
    __device__ __forceinline__ void begin(int n_, long long rem, int count) {
        left = count;
        issued = 0;
        n = n_;
        row = row_of(a, n);
        next_held = n + 1 < a.N ? a.seq_lens[n + 1] : -1;
        const int p = (int)(rem / units_of(row)), v = (int)(rem % units_of(row)) - kBegin;
        t = max(v, 0);
        left = max(left + min(v, 0), 0);
        hk = p / blocks;
        hb = p % blocks;
        began = t == 0;
        fresh = true;
        place_tile();
        fetch_pages(true);
    }
    __device__ __forceinline__ void advance() {
        const bool pair_ends = t + 1 == row.tiles;
        --left;
        fresh = pair_ends;
        if (left == 0) return;
        if (!pair_ends) {
            ++t;
            if (a.page_size >= kTile) {
                off += kTile;
                if (off >= a.page_size) {
                    off -= a.page_size;
                    ++page_at;
                }
            } else {
                place_tile();
            }
            fetch_pages(false);
            return;
        }
        if ((left = max(left - kBegin, 0)) == 0) return;
        t = 0;
        began = true;
        bool anew = false;
        if (++hb == blocks) {
            hb = 0;
            if (++hk == a.Hk) {
                hk = 0;
                anew = true;
                do {  // tiles are left, so a row with some follows
                    ++n;
                    row = row_from(a, next_held);
                    next_held = n + 1 < a.N ? a.seq_lens[n + 1] : -1;
                } while (row.tiles == 0);
            }
        }
        place_tile();
        fetch_pages(anew);
    }
    // Copies the next tile into `stage` (nothing once the range is done); always commits one group.
    __device__ __forceinline__ void issue(int stage) {
        if (left > 0) {
            constexpr int CH = Geo::kChunks, RB = Geo::kRowBytes, RowsAt = 32 / (CH < 32 ? CH : 32);
            const int in = page_at - from;
            const int lo = __shfl_sync(~0u, pages, in & 31), hi = __shfl_sync(~0u, pages2, in & 31);
            const int page = in < 32 ? lo : hi, pos = row.first + t * kTile + (lane & 15);
            const bool valid = pos < row.last && (unsigned)page < (unsigned)a.n_pages;
            // row of the cache; the cache holds fewer than 2^31 of them
            const int at = valid ? (page * a.Hk + hk) * a.page_size + off : -1;
            const unsigned mask = __ballot_sync(~0u, valid) & 0xffffu;
            const bool pair_ends = t + 1 == row.tiles, put = a.k_new && pair_ends && row.held < row.last;
            const int new_row = put ? row.held - row.first - t * kTile : 0;  // the pair's last position
            const int c = lane % CH, r0 = lane / CH;
            const unsigned char *kb = (const unsigned char*)a.k_cache + c * 16, *vb = (const unsigned char*)a.v_cache + c * 16;
            const uint32_t dst = ring + stage * Geo::kStageBytes + r0 * RB;
            if (!(put && (mask >> new_row & 1))) {
#pragma unroll
                for (int i = 0; i < kTile / RowsAt; ++i) {
                    const int r = i * RowsAt + r0, src = __shfl_sync(~0u, at, r);
                    const size_t o = (size_t)(src < 0 ? 0 : src) * RB;
                    const uint32_t to = dst + i * RowsAt * RB + ((c ^ (r & 7)) << 4);
                    cp_async16(to, kb + o, src >= 0);
                    cp_async16(to + kTile * RB, vb + o, src >= 0);
                }
            } else {
                // The tile with the new token: its row comes from the arguments, and goes into the cache.
                const size_t new_at = ((size_t)n * a.Hk + hk) * RB + c * 16;
                const unsigned char *kn = (const unsigned char*)a.k_new + new_at, *vn = (const unsigned char*)a.v_new + new_at;
#pragma unroll 1
                for (int i = 0; i < kTile / RowsAt; ++i) {
                    const int r = i * RowsAt + r0, src = __shfl_sync(~0u, at, r);
                    const size_t o = (size_t)(src < 0 ? 0 : src) * RB;
                    const uint32_t to = dst + i * RowsAt * RB + ((c ^ (r & 7)) << 4);
                    const bool is_new = r == new_row;
                    cp_async16(to, is_new ? kn : kb + o, src >= 0);
                    cp_async16(to + kTile * RB, is_new ? vn : vb + o, src >= 0);
                    if (is_new && hb == 0) {
                        *reinterpret_cast<uint4*>((unsigned char*)a.k_cache + o + c * 16) = *reinterpret_cast<const uint4*>(kn);
                        *reinterpret_cast<uint4*>((unsigned char*)a.v_cache + o + c * 16) = *reinterpret_cast<const uint4*>(vn);
                    }
                }
            }
            const bool range_ends = pair_ends || left == 1;
            if (fresh) {  // the queries are read when the tile is worked on: have them in L2 by then
                const int head0 = hk * G + hb * kHeads, lines = min(kHeads, G - hb * kHeads) * RB / 128;
                if (lane < lines)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"((const char*)a.q + ((size_t)n * a.Hq + head0) * RB + lane * 128));
            }
            ++issued;
            if (lane == 0) {
                const int place = began ? (pair_ends ? 2 : 1) : 0;
                const int head0 = hk * G + hb * kHeads;
                metas[stage] = make_int4(n * a.Hq + head0, min(kHeads, G - hb * kHeads),
                                         (int)(mask | (fresh ? kFresh : 0) | (range_ends ? kEnds : 0) | (unsigned)place << kPlaceShift), 0);
                if (t == 0)
                    pair_out[((size_t)n * a.Hk + hk) * blocks + hb] =
                        make_int2(worker, row.tiles <= left ? 1 : 1 + (int)((row.tiles - left + W - 1) / W));
            }
            advance();
        }
        cp_async_commit();
    }
};

// What the split kernels share before their loops: the range of this warp. False: it has none.
// Rows without any attended position get their zeros here.
template <typename T, int D>
__device__ __forceinline__ bool find_range(const AttnDecodeArgs& a, const Pieces& ws, long long& W, int& count, int& row, long long& rem) {
    constexpr int kWorkers = Geometry<T, D>::kWorkers, CH = Geometry<T, D>::kChunks, kWarps = Geometry<T, D>::kWarps;
    __shared__ long long s_part[kWarps], s_rem[kWarps];
    __shared__ int s_row[kWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = a.Hq / a.Hk, P = a.Hk * ((G + kHeads - 1) / kHeads);
    // Units of all rows before thread tid's rows, and of all rows.
    const int per = (a.N + kWarps * 32 - 1) / (kWarps * 32), row0 = min(tid * per, a.N), row1 = min(row0 + per, a.N);
    long long mine = 0;
    for (int n = row0; n < row1; ++n) mine += units_of(row_of(a, n));
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
    W = total <= kWorkers ? 1 : (total + kWorkers - 1) / kWorkers;  // units of a worker
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        long long u = (long long)(blockIdx.x * kWarps + w) * W;
        if (u >= before && u < before + mine) {
            u -= before;
            int n = row0;
            for (long long units; u >= (units = (long long)units_of(row_of(a, n)) * P); ++n) u -= units;
            s_row[w] = n;
            s_rem[w] = u;
        }
    }
    for (int n = blockIdx.x; n < a.N; n += gridDim.x) {
        if (row_of(a, n).tiles) continue;
        uint4* o = (uint4*)((T*)a.o + (size_t)n * a.Hq * D);
        for (int i = tid; i < a.Hq * CH; i += kWarps * 32) o[i] = make_uint4(0, 0, 0, 0);
        for (int i = tid; i < a.Hq; i += kWarps * 32)
            if (a.lse) a.lse[(size_t)n * a.Hq + i] = -INFINITY;
        for (int i = tid; i < P; i += kWarps * 32) ws.pair[(size_t)n * P + i] = make_int2(0, 0);
    }
    __syncthreads();
    const long long begin = (long long)(blockIdx.x * kWarps + warp) * W;
    if (begin >= total) return false;
    count = (int)min(W, total - begin);
    row = s_row[warp];
    rem = s_rem[warp];
    return true;
}

// The positions are the rows of the MMAs, the query heads their columns (NT
// blocks of 8), so that few heads waste little:
//     S^T [16 x 8 NT] = K Q^T,  O^T [D x 8 NT] += V^T P^T.
// bf16 operands go in as they are, the weights in two parts of bf16 with a
// product each: one part alone, 2^-9 off a weight, costs as much accuracy again
// as the rounding of the output, and saves little (64 rows of 256 to 16384
// positions 170.7 us, with both 171.7; 256 rows of 0 to 300 21.8 and 22.5; 32
// heads to a key-value head of 64, 64 rows of 2048, 31.5 and 34.3). 32-bit
// operands are split into two tf32 parts each, and three products taken (the fourth,
// lo * lo, is below 2^-22 of the whole), which keeps 32-bit accuracy. The split
// is integer rounding and a subtraction: with the conversion instruction in its
// place 64 rows of 1000 positions took 169 us, with these 95 (and 99 since every
// tile's products are added outside the MMA).
// The weights' maximum is a reference that moves only when a score passes it by
// more than 2^8: until then weights reach 2^8, far from any overflow in 32
// bits, and neither a reduction over the warp nor a rescaling is due.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(Plan<T, D>::kWarps * 32, Plan<T, D>::kCtasPerSm) attn_split_kernel(AttnDecodeArgs a) {
    using Geo = Geometry<T, D>;
    constexpr bool BF = sizeof(T) == 2;
    constexpr int S = Geo::kStages, RB = Geo::kRowBytes, kWarps = Geo::kWarps;
    constexpr int KS = BF ? D / 16 : D / 8;  // steps of the K Q^T product
    constexpr bool SPLIT_Q = !BF && NT == 1;  // both tf32 parts of the queries kept (16 heads: split anew each time)
    constexpr float kSlackLog2 = 8.f;
    extern __shared__ __align__(128) unsigned char smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = a.Hq / a.Hk;
    const Pieces ws = pieces_of(a.workspace, Geo::kWorkers, G, D);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    long long W, rem;
    int count, row;
    if (!find_range<T, D>(a, ws, W, count, row, rem)) return;
    const int worker = blockIdx.x * kWarps + warp;
    const uint32_t ring = sm100::smem_u32(smem) + warp * S * Geo::kStageBytes;
    int4* metas = reinterpret_cast<int4*>(smem + (size_t)kWarps * S * Geo::kStageBytes) + warp * S;
    Feed<T, D> feed{a, ws.pair, ring, metas, worker, lane, G, (G + kHeads - 1) / kHeads, W};
    feed.begin(row, rem, count);
#pragma unroll 1
    for (int s = 0; s < S - 1; ++s) feed.issue(s);

    const float scale2 = a.scale * kLog2e;
    const int g = lane >> 2, c = lane & 3, c2 = c * 2, mat = lane >> 3, r8 = lane & 7;
    const uint32_t k_at = (r8 + (mat & 1) * 8) * RB, v_at = (r8 + (mat >> 1) * 8) * RB;
    uint32_t qf[KS][NT][2], ql[SPLIT_Q ? KS : 1][NT][2];
    float o[D / 16][NT][4], m[NT][2], l[NT][2];
    int stage = 0, into = S - 1;
#pragma unroll 1
    for (int step = 0; step < feed.issued; ++step) {
        cp_async_wait<S - 2>();
        __syncwarp();
        feed.issue(into);
        into = into + 1 == S ? 0 : into + 1;
        const int4 meta = metas[stage];
        const unsigned bits = (unsigned)meta.z;
        const int heads = meta.y;
        const uint32_t kt = ring + stage * Geo::kStageBytes, vt = kt + kTile * RB;
        stage = stage + 1 == S ? 0 : stage + 1;
        if (bits & kFresh) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const bool on = g + 8 * j < heads;
                const T* qh = (const T*)a.q + (size_t)(meta.x + (on ? g + 8 * j : 0)) * D;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    if constexpr (BF) {
                        qf[ks][j][0] = on ? *reinterpret_cast<const uint32_t*>(qh + ks * 16 + c2) : 0u;
                        qf[ks][j][1] = on ? *reinterpret_cast<const uint32_t*>(qh + ks * 16 + c2 + 8) : 0u;
                    } else {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float x = on ? qh[ks * 8 + c + 4 * e] : 0.f;
                            if constexpr (SPLIT_Q) split_tf32(x, qf[ks][j][e], ql[ks][j][e]);
                            else qf[ks][j][e] = __float_as_uint(x);
                        }
                    }
                }
                m[j][0] = m[j][1] = -INFINITY;
                l[j][0] = l[j][1] = 0.f;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.f;
            }
        }
        float s[NT][4] = {}, s2[NT][4] = {};  // two sums: half the chain of dependent products
        if constexpr (BF) {
#pragma unroll
            for (int ks = 0; ks < KS; ks += 2) {
                uint32_t kf[2][4];
                ldsm4(kf[0], kt + k_at + (((2 * ks + (mat >> 1)) ^ r8) << 4));
                ldsm4(kf[1], kt + k_at + (((2 * ks + 2 + (mat >> 1)) ^ r8) << 4));
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    mma_bf16(s[j], kf[0], qf[ks][j][0], qf[ks][j][1]);
                    mma_bf16(s2[j], kf[1], qf[ks + 1][j][0], qf[ks + 1][j][1]);
                }
            }
        } else {
            // an 8 x 8 matrix of 16-bit elements is one of 8 rows x 4 32-bit ones: lane 4 r + x gets element x of row r
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                uint32_t x[4], hi[4], lo[4];
                ldsm4(x, kt + k_at + (((2 * ks + (mat >> 1)) ^ r8) << 4));
#pragma unroll
                for (int e = 0; e < 4; ++e) split_tf32(__uint_as_float(x[e]), hi[e], lo[e]);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    uint32_t bh[2], bl[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if constexpr (SPLIT_Q) {
                            bh[e] = qf[ks][j][e];
                            bl[e] = ql[ks][j][e];
                        } else {
                            split_tf32(__uint_as_float(qf[ks][j][e]), bh[e], bl[e]);
                        }
                    }
                    mma_tf32(s2[j], lo, bh[0], bh[1]);
                    mma_tf32(s2[j], hi, bl[0], bl[1]);
                    mma_tf32(s[j], hi, bh[0], bh[1]);
                }
            }
        }
        // scores in log2 units: elements 0, 1 are position g of heads c2, c2 + 1 (+ 8 j), elements 2, 3 position g + 8
        const bool on_lo = bits >> g & 1, on_hi = bits >> (g + 8) & 1;
        bool past = false;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                s[j][e] = on_lo ? (s[j][e] + s2[j][e]) * scale2 : -INFINITY;
                s[j][e + 2] = on_hi ? (s[j][e + 2] + s2[j][e + 2]) * scale2 : -INFINITY;
                past |= fmaxf(s[j][e], s[j][e + 2]) > m[j][e] + kSlackLog2;
            }
        if (__any_sync(~0u, past)) {  // move the references to the maxima, for all heads of the warp
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float top = fmaxf(s[j][e], s[j][e + 2]);
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, x));
                    top = fmaxf(top, m[j][e]);
                    const float keep = m[j][e] == top ? 1.f : exp2_fast(m[j][e] - top);
                    m[j][e] = top;
                    l[j][e] *= keep;
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        o[i][j][e] *= keep;
                        o[i][j][e + 2] *= keep;
                    }
                }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float base = m[j][e] == -INFINITY ? 0.f : m[j][e];  // nothing attended so far: weights of 0
                s[j][e] = exp2_fast(s[j][e] - base);
                s[j][e + 2] = exp2_fast(s[j][e + 2] - base);
                l[j][e] += s[j][e] + s[j][e + 2];
            }
        if constexpr (BF) {
            uint32_t ph[NT][2], pl[NT][2];  // the weights' two parts as the right operand
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    uint32_t hi, lo;
                    split_bf16(s[j][2 * b], s[j][2 * b + 1], hi, lo);
                    ph[j][b] = transpose8x8(hi);
                    pl[j][b] = transpose8x8(lo);
                }
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                uint32_t vf[4];
                ldsm4_trans(vf, vt + v_at + (((2 * i + (mat & 1)) ^ r8) << 4));
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    mma_bf16(o[i][j], vf, pl[j][0], pl[j][1]);
                    mma_bf16(o[i][j], vf, ph[j][0], ph[j][1]);
                }
            }
        } else {
            // Inner index x of the right operand stands for position 2 x (x < 4) or 2 (x - 4) + 1 of 8: lane 4 h + c holds
            // head h's weights of positions 2 c and 2 c + 1. The same order in the left operand makes its loads free of
            // bank conflicts: rows 0, 2, 4, 6 (and 1, 3, 5, 7) of the swizzled tile lie in different banks.
            uint32_t ph[2][NT][2], pl[2][NT][2];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int src = (c2 + e) * 4 + (g >> 1);
                        const float x0 = __shfl_sync(~0u, s[j][2 * b], src), x1 = __shfl_sync(~0u, s[j][2 * b + 1], src);
                        split_tf32(g & 1 ? x1 : x0, ph[b][j][e], pl[b][j][e]);
                    }
            const uint32_t v0 = vt + c2 * RB + (((g >> 2) ^ c2) << 4) + (g & 3) * 4;              // channel g of position 2 c
            const uint32_t v1 = vt + (c2 + 1) * RB + (((g >> 2) ^ (c2 + 1)) << 4) + (g & 3) * 4;  // of 2 c + 1
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                // A tile's products by themselves, then added here: the MMA rounds its sums towards zero, which over a
                // hundred tiles would be off by 2^-16.
                float add[NT][4] = {};
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)  // elements 0, 1: channels 16 i + g, + 8 of position 2 c; 2, 3: of 2 c + 1
                        split_tf32(lds_f32(((e >> 1 ? v1 : v0) ^ ((i & 1) * 64 + (e & 1) * 32)) + b * 8 * RB + (i >> 1) * 128), hi[e], lo[e]);
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        mma_tf32(add[j], lo, ph[b][j][0], ph[b][j][1]);
                        mma_tf32(add[j], hi, pl[b][j][0], pl[b][j][1]);
                        mma_tf32(add[j], hi, ph[b][j][0], ph[b][j][1]);
                    }
                }
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][j][e] += add[j][e];
            }
        }
        if (bits & kEnds) {
            const int place = (int)(bits >> kPlaceShift);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float sum[2], inv[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    sum[e] = l[j][e];
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) sum[e] += __shfl_xor_sync(~0u, sum[e], x);
                    inv[e] = sum[e] == 0.f ? 0.f : 1.f / sum[e];
                }
                const int head = c2 + 8 * j;  // of element 0; element 1: the next
                if (place == 2) {
                    if constexpr (BF) {
                        T* to = (T*)a.o + (size_t)(meta.x + g + 8 * j) * D + c2;
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {  // transposed: lane 4 h + x holds channels 2 x, 2 x + 1 of head h
                            const uint32_t lo = transpose8x8(pack_bf16(o[i][j][0] * inv[0], o[i][j][1] * inv[1]));
                            const uint32_t hi = transpose8x8(pack_bf16(o[i][j][2] * inv[0], o[i][j][3] * inv[1]));
                            if (g + 8 * j < heads) {
                                *reinterpret_cast<uint32_t*>(to + i * 16) = lo;
                                *reinterpret_cast<uint32_t*>(to + i * 16 + 8) = hi;
                            }
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            if (head + e >= heads) continue;
                            float* to = (float*)a.o + (size_t)(meta.x + head + e) * D + g;
#pragma unroll
                            for (int i = 0; i < D / 16; ++i) {
                                to[i * 16] = o[i][j][e] * inv[e];
                                to[i * 16 + 8] = o[i][j][e + 2] * inv[e];
                            }
                        }
                    }
                    if (a.lse && g < 2 && head + g < heads) {
                        const float all = g ? sum[1] : sum[0], ref = g ? m[j][1] : m[j][0];
                        a.lse[meta.x + head + g] = all == 0.f ? -INFINITY : fmaf(ref, kLn2, logf(all));
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (head + e >= heads) continue;
                        const size_t at = (size_t)(2 * worker + place) * ws.rows + head + e;
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            ws.o[at * D + i * 16 + g] = o[i][j][e];
                            ws.o[at * D + i * 16 + 8 + g] = o[i][j][e + 2];
                        }
                        if (g == 0) ws.ml[at] = make_float2(m[j][e], sum[e]);
                    }
                }
            }
        }
    }
    cp_async_wait<0>();
}

// Joins the pieces of every (pair, query head) that lies in several workers, in
// their order: piece 0 in place 1 of the worker that begins the pair, the others
// in place 0 of the workers after it. WARPS warps share the pieces: 32 or 8
// where there are few pairs, so many pieces of each (one pair of 1184 pieces: 36
// us a call with 8, 22 with 32), 1 where there are many. A warp loads up to four
// pieces at once, maxima and sums with them, so that the chain of dependent
// loads is two long.
constexpr int kJoinWarps = 8;  // of a block, where a warp works alone

template <typename T, int D, int WARPS>
__global__ void __launch_bounds__((WARPS == 1 ? kJoinWarps : WARPS) * 32) attn_join_kernel(AttnDecodeArgs a, int items) {
    constexpr int E = D / 32, B = 4;
    __shared__ float so[WARPS == 1 ? 1 : WARPS][D];
    __shared__ float2 sml[WARPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = a.Hq / a.Hk, blocks = (G + kHeads - 1) / kHeads, P = a.Hk * blocks;
    const Pieces ws = pieces_of(a.workspace, Geometry<T, D>::kWorkers, G, D);
    const int item = WARPS == 1 ? blockIdx.x * kJoinWarps + warp : blockIdx.x;
    if (item >= items) return;
    const int i = item / ws.rows, h = item % ws.rows;
    const int n = i / P, p = i % P, hk = p / blocks, hb = p % blocks;
    if (h >= G - hb * kHeads) return;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int2 pair = ws.pair[i];
    if (pair.y < 2) return;
    auto slot = [&](int k) { return (size_t)(2 * (pair.x + k) + (k == 0 ? 1 : 0)) * ws.rows + h; };
    float acc[E] = {}, sum = 0.f, ref = -INFINITY;
    for (int k = WARPS == 1 ? 0 : warp; k < pair.y; k += WARPS * B) {
        float2 ml[B];
        float x[B][E];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const bool on = k + b * WARPS < pair.y;
            const size_t at = slot(on ? k + b * WARPS : k);
            ml[b] = on ? ws.ml[at] : make_float2(-INFINITY, 0.f);
            const float* from = ws.o + at * D + lane * E;
            if constexpr (E == 4) {
                const float4 v = *reinterpret_cast<const float4*>(from);
                x[b][0] = v.x; x[b][1] = v.y; x[b][2] = v.z; x[b][3] = v.w;
            } else {
                const float2 v = *reinterpret_cast<const float2*>(from);
                x[b][0] = v.x; x[b][1] = v.y;
            }
        }
        float top = ref;
#pragma unroll
        for (int b = 0; b < B; ++b) top = fmaxf(top, ml[b].x);
        const float keep = ref == top ? 1.f : exp2_fast(ref - top);
        ref = top;
        sum *= keep;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] *= keep;
#pragma unroll
        for (int b = 0; b < B; ++b) {
            // Nothing attended in this piece, or no such piece. The maximum would not tell: it passes over NaN scores, and
            // stays -inf where a piece has no others. Their sum is NaN, and goes on.
            if (ml[b].y == 0.f) continue;
            const float f = exp2_fast(ml[b].x - top);
            sum = fmaf(ml[b].y, f, sum);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(x[b][e], f, acc[e]);
        }
    }
    const size_t out = (size_t)n * a.Hq + (size_t)hk * G + hb * kHeads + h;
    if constexpr (WARPS == 1) {
#pragma unroll
        for (int e = 0; e < E; ++e) ((T*)a.o)[out * D + lane * E + e] = from_f32<T>(sum == 0.f ? 0.f : acc[e] / sum);
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) so[warp][lane * E + e] = acc[e];
        if (lane == 0) sml[warp] = make_float2(ref, sum);
        __syncthreads();
        ref = -INFINITY;
        sum = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) ref = fmaxf(ref, sml[w].x);
        auto factor = [&](int w) { return sml[w].y == 0.f ? 0.f : exp2_fast(sml[w].x - ref); };
#pragma unroll
        for (int w = 0; w < WARPS; ++w) sum = fmaf(sml[w].y, factor(w), sum);
        for (int c = threadIdx.x; c < D; c += WARPS * 32) {
            float x = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) x = fmaf(so[w][c], factor(w), x);
            ((T*)a.o)[out * D + c] = from_f32<T>(sum == 0.f ? 0.f : x / sum);
        }
    }
    if (a.lse && (WARPS == 1 ? lane : (int)threadIdx.x) == 0)
        a.lse[out] = sum == 0.f ? -INFINITY : fmaf(ref, kLn2, logf(sum));
}

}  // namespace

size_t attn_decode_workspace_bytes(int N, int Hq, int Hk, int d) {
    const int G = Hq / Hk, blocks = (G + kHeads - 1) / kHeads;
    const int bf = workers_of(1, d), f = workers_of(0, d);
    const Pieces p = pieces_of(nullptr, bf > f ? bf : f, G, d);
    return (size_t)((char*)(p.pair + (size_t)N * Hk * blocks) - (char*)nullptr);
}

template <typename T, int D, int NT>
static cudaError_t launch_attn(const AttnDecodeArgs& a, cudaStream_t stream) {
    using Geo = Geometry<T, D>;
    auto split = attn_split_kernel<T, D, NT>;
    const int G = a.Hq / a.Hk, pairs = a.N * a.Hk * ((G + kHeads - 1) / kHeads);
    static std::atomic<unsigned long long> raised{0};
    cudaError_t err = allow_smem(split, Geo::kSmem, raised);
    if (err != cudaSuccess) return err;
    split<<<Geo::kCtas, Geo::kWarps * 32, Geo::kSmem, stream>>>(a);
    if ((err = cudaGetLastError()) != cudaSuccess) return err;
    // The join is launched while the split kernel runs (programmatic dependent launch) and waits for its end.
    const int warps = pairs < 16 ? 32 : pairs < 148 ? 8 : 1;
    const int items = pairs * (G < kHeads ? G : kHeads);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(warps > 1 ? items : (items + kJoinWarps - 1) / kJoinWarps);
    cfg.blockDim = dim3(32 * (warps > 1 ? warps : kJoinWarps));
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, warps == 32 ? attn_join_kernel<T, D, 32> : warps == 8 ? attn_join_kernel<T, D, 8> : attn_join_kernel<T, D, 1>, a, items);
}

template <typename T, int D>
static cudaError_t launch_attn_heads(const AttnDecodeArgs& a, cudaStream_t stream) {
    return a.Hq / a.Hk <= 8 ? launch_attn<T, D, 1>(a, stream) : launch_attn<T, D, 2>(a, stream);
}

cudaError_t launch_attn_decode(const AttnDecodeArgs& a, cudaStream_t stream) {
    if (a.bf16)
        return a.d == 64 ? launch_attn_heads<__nv_bfloat16, 64>(a, stream) : launch_attn_heads<__nv_bfloat16, 128>(a, stream);
    return a.d == 64 ? launch_attn_heads<float, 64>(a, stream) : launch_attn_heads<float, 128>(a, stream);
}

}  // namespace kda
