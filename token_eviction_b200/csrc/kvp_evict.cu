// Eviction from a paged cache by accumulated attention weight, in place.
//
// A head's rows are ranked by their weights' bits, which order as the weights do (all are
// non-negative or count as zero); T, the key of the last row that stays, is found by its bits from
// the top, and the rows that change places are listed in row order: the evicted places below
// t - w and the kept rows at or past it. Those are copied (keys, values, weight), then the window.
// Nothing else moves: a head that gives up e of its rows copies at most e + w.
//
// evict_select (up to 16 K rows a CTA): one CTA, or a cluster of 8, per head, each thread holding the
// keys of kPer consecutive rows in registers. Eight bits of T a round, by a histogram in shared
// memory that one warp scans; a cluster's CTAs write theirs into one another's shared memory (a round of
// a cluster takes 1.4 us, half of it the cluster's barrier). It ends as soon as all keys that share T's bits
// stay. One scan of packed counts then gives every thread its places in the lists. A head with few
// rows to copy is finished here; one that gives up few rows (a decode's step: one) has them picked
// one by one instead, by every warp the lightest of its own rows and then by one warp of all of
// those. (512 heads that give up one row of 2049: 7.2 us, 11.5 by rounds; rounds are as fast from
// about 10 rows on.)
// (Two bits a round by counting keys against three candidates, with no atomics: 28 us where this
// takes 17 for 512 heads of 2064 rows.)
// evict_select_long: longer rows, keys in shared memory or read again each round, four bits a round by
// packed counters.
// evict_move: copies the listed rows of the other heads. Only rows in [t - w, t) are both a source and
// a place to write to: the kept rows there are the first of the list, and the block that copies
// them copies the window after them.
#include <cooperative_groups.h>

#include <algorithm>

#include "kvp_cache.cuh"
#include "kvp_ptx.cuh"

namespace cg = cooperative_groups;

namespace kvp {
namespace {

constexpr int kMaxThreads = 1024, kMaxWarps = kMaxThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kSliceCap = 48 * 1024;     // keys a CTA of evict_select_long holds in shared memory
constexpr int kClusters = 15;             // clusters of 8 CTAs with an SM each that run at once
constexpr int kManyThreads = 384;         // most threads of the CTAs that share an SM with others
constexpr int kPerMost = 16;             // keys a thread of evict_select holds
constexpr int kMoveThreads = 256, kMoveCtas = 3;   // of evict_move: threads, CTAs an SM
constexpr int kMoveLoads = 8;            // 16-byte loads a lane of evict_move has in flight,
constexpr int kOwnLoads = 4;             // and of evict_select, where it copies rows itself:
constexpr int kOwn = 384;                // past t - w up to as many, where there are heads enough to fill the card
                                         // (512 heads of 2176 rows to 2048: 25 us, 34 by evict_move)
constexpr int kLight = 8;                // rows given up up to which evict_select picks them one by one, and
constexpr int kFew = 64;                 // rows past t - w up to which evict_select copies them itself (one CTA a head)

struct EvictArgs {
    CacheView c;
    const float* acc;
    float* acc_out;
    uint4* k_pages;
    uint4* v_pages;
    const int32_t* budgets;   // NULL: B
    int32_t* lens_out;
    int32_t* src;             // NULL: not wanted
    int B, s, w;
    // workspace
    int4* info;               // [heads]: n, t, rows listed, 1 + those below t (0: nothing left to copy)
    int32_t* from;            // [heads][B]: listed rows, ascending
    int32_t* to;              // [heads][B]: the places they move to, ascending
    uint8_t* stays;           // [heads][stays_stride]: a bit a row below t - w that keeps its place (clusters of evict_select)
    size_t stays_stride;
    int row_chunks;           // d / 8
    bool many;                // heads enough to fill the card
    int slice;                // evict_select_long: keys that shared memory holds per CTA; 0: read again each round
};

__device__ __forceinline__ uint32_t key_of(float weight) {
    const int bits = __float_as_int(weight);
    return bits > 0 && bits <= 0x7F800000 ? (uint32_t)bits : 0u;   // negative, zero and NaN: 0
}

struct Counts {               // of a warp's or a CTA's rows
    int gt_low, eq_low, gt_high, eq_high;
};

struct SelectShared {
    uint32_t warp_digits[2][kMaxWarps][8];       // 16 counters of 16 bits
    int digits[2][kMaxCluster][16];              // every CTA's sums
    Counts warp_counts[kMaxWarps];
    Counts cta_counts[kMaxCluster];
};

template <int C>
__device__ __forceinline__ void sync_all() {
    if (C > 1) cg::this_cluster().sync();
    else __syncthreads();
}

template <int C>
__global__ void __launch_bounds__(kMaxThreads, 1) evict_select_long(const EvictArgs a) {
    extern __shared__ __align__(16) uint32_t keys[];
    __shared__ SelectShared sh;
    ptx::grid_dependency_wait();
    const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 31, warp = tid >> 5, warps = threads >> 5;
    const int head = blockIdx.x / C, rank = blockIdx.x % C;
    const int n = a.c.len(head);
    const int least = max(a.s + a.w, 1);
    const int t = a.budgets ? min(max(a.budgets[head], least), a.B) : a.B;
    const int w = a.w, s = a.s;
    const int32_t* table = a.c.table + (size_t)head * a.c.max_pages;
    const bool full = n > t;
    int32_t* src = a.src ? a.src + (size_t)head * a.B : nullptr;

    // this CTA's slice of the rows [0, n)
    const int per = ((n + C - 1) / C + 15) / 16 * 16;
    const int lo = min(n, rank * per), hi = min(n, lo + per);
    const int stay = full ? t - w : n;           // rows below keep their places, or are replaced later
    const bool in_smem = a.slice > 0;
    const bool copy = a.acc_out != a.acc;
    if (copy || (full && in_smem)) {
        for (int j = lo + 4 * tid; j < hi; j += 4 * threads) {   // four rows lie in one page
            const int page = table[j >> a.c.page_shift];
            const bool there = page >= 0 && page < a.c.num_pages;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            const size_t row = ((size_t)max(page, 0) << a.c.page_shift) + (j & ((1 << a.c.page_shift) - 1));
            if (there) x = *(const float4*)(a.acc + row);
            if (in_smem && full && KVP_CHECK(j - lo + 4 <= a.slice, 709, head, j))
                *(uint4*)(keys + (j - lo)) = make_uint4(key_of(x.x), key_of(x.y), key_of(x.z), key_of(x.w));
            if (there && copy) {
                if (j + 4 <= stay) {
                    *(float4*)(a.acc_out + row) = x;
                } else {
                    if (j < stay) a.acc_out[row] = x.x;
                    if (j + 1 < stay) a.acc_out[row + 1] = x.y;
                    if (j + 2 < stay) a.acc_out[row + 2] = x.z;
                }
            }
        }
    }
    if (src) {
        const int last = full ? t : n;           // rows past the new length
        for (int i = last + rank * threads + tid; i < a.B; i += C * threads) src[i] = -1;
        if (!full)
            for (int i = rank * threads + tid; i < n; i += C * threads) src[i] = i;
    }
    if (!full) {
        if (rank == 0 && tid == 0) {
            a.info[head] = make_int4(n, t, 0, 0);
            a.lens_out[head] = n;                // (a CTA that reads lens after this clamps to the same n)
        }
        return;                                  // the same in every CTA of the cluster
    }
    auto key_at = [&](int j) -> uint32_t {
        if (in_smem) return keys[j - lo];
        const long long row = a.c.row(head, j);
        return row < 0 ? 0u : key_of(a.acc[row]);
    };
    const int c0 = max(lo, s), c1 = min(hi, n - w);   // candidates of this CTA
    sync_all<C>();                                    // keys staged; every CTA of the cluster runs

    // ---- the key of the last row that stays
    uint32_t prefix = 0, mask = 0;
    int krem = t - s - w;
    bool all = false;                                 // all rows that match the prefix stay
    int buf = 0;
    for (int shift = 28; shift >= 0 && krem > 0 && !all; shift -= 4, buf ^= 1) {
        uint32_t even[4] = {}, odd[4] = {};           // 16-bit pairs of counters (0,2) and (1,3) of four digits
        for (int j0 = c0; j0 < c1; j0 += 255 * threads) {      // byte counters hold 255
            uint32_t byte[4] = {};
            for (int j = j0 + tid; j < min(c1, j0 + 255 * threads); j += threads) {
                const uint32_t u = key_at(j);
                if ((u & mask) == prefix) {
                    const uint32_t dg = (u >> shift) & 15u, one = 1u << (8 * (dg & 3));
#pragma unroll
                    for (int q = 0; q < 4; ++q) byte[q] += (dg >> 2) == q ? one : 0u;
                }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                even[q] += byte[q] & 0x00FF00FFu;
                odd[q] += (byte[q] >> 8) & 0x00FF00FFu;
            }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            even[q] = __reduce_add_sync(0xffffffffu, even[q]);
            odd[q] = __reduce_add_sync(0xffffffffu, odd[q]);
        }
        if (lane == 0) {
            *(uint4*)&sh.warp_digits[buf][warp][0] = make_uint4(even[0], odd[0], even[1], odd[1]);
            *(uint4*)&sh.warp_digits[buf][warp][4] = make_uint4(even[2], odd[2], even[3], odd[3]);
        }
        __syncthreads();
        // digit d lies in word (d / 4) * 2 + (d & 1), upper half if d & 2
        if (tid < 16 * C) {
            const int dg = tid & 15, word = (dg >> 2) * 2 + (dg & 1), up = (dg & 2) * 8;
            int sum = 0;
            for (int x = 0; x < warps; ++x) sum += (sh.warp_digits[buf][x][word] >> up) & 0xFFFFu;
            if (C > 1) *cg::this_cluster().map_shared_rank(&sh.digits[buf][rank][dg], tid >> 4) = sum;
            else sh.digits[buf][0][dg] = sum;
        }
        sync_all<C>();
        int mine = 0;                                 // lane x < 16: rows of digit 15 - x
        if (lane < 16) {
#pragma unroll
            for (int x = 0; x < C; ++x) mine += sh.digits[buf][x][15 - lane];
        }
        int inc = mine;
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        const unsigned at = __ballot_sync(0xffffffffu, lane < 16 && inc - mine < krem && krem <= inc);
        const int x = __ffs(at) - 1;                  // there is one: the candidates are more than krem
        prefix |= (uint32_t)(15 - x) << shift;
        mask |= 15u << shift;
        krem -= __shfl_sync(0xffffffffu, inc - mine, x);
        all = krem == __shfl_sync(0xffffffffu, mine, x);
    }
    if (t - s - w == 0) prefix = mask = 0xFFFFFFFFu;  // no candidate stays: no key is as large
    const int need_eq = t - s - w == 0 ? 0 : krem;    // rows equal to the prefix that stay, lowest first

    // ---- list what changes places: a warp takes a contiguous stretch of the CTA's candidates
    const int split = t - w;
    const int span = c1 - c0;
    const int per_warp = span > 0 ? ((span + warps - 1) / warps + 31) / 32 * 32 : 0;
    const int w0 = min(c1, c0 + warp * per_warp), w1 = min(c1, w0 + per_warp);
    Counts mine = {};
    for (int j0 = w0; j0 < w1; j0 += 32) {
        const int j = j0 + lane;
        const uint32_t u = j < w1 ? key_at(j) & mask : 0u;
        const unsigned gt = __ballot_sync(0xffffffffu, j < w1 && u > prefix);
        const unsigned eq = __ballot_sync(0xffffffffu, j < w1 && u == prefix);
        const unsigned low = __ballot_sync(0xffffffffu, j < split);
        mine.gt_low += __popc(gt & low);
        mine.eq_low += __popc(eq & low);
        mine.gt_high += __popc(gt & ~low);
        mine.eq_high += __popc(eq & ~low);
    }
    if (lane == 0) sh.warp_counts[warp] = mine;
    __syncthreads();
    if (warp == 0) {
        Counts m = lane < warps ? sh.warp_counts[lane] : Counts{};
        m.gt_low = __reduce_add_sync(0xffffffffu, m.gt_low);
        m.eq_low = __reduce_add_sync(0xffffffffu, m.eq_low);
        m.gt_high = __reduce_add_sync(0xffffffffu, m.gt_high);
        m.eq_high = __reduce_add_sync(0xffffffffu, m.eq_high);
        if (C > 1) {
            if (lane < C) *cg::this_cluster().map_shared_rank(&sh.cta_counts[rank], lane) = m;
        } else if (lane == 0) {
            sh.cta_counts[0] = m;
        }
    }
    sync_all<C>();
    // rows before this warp's stretch: equal ones, kept ones below split and past it
    int eq = 0, kept_low = 0, kept_high = 0, listed = 0;
    auto add = [&](const Counts& m) {
        const int left = max(0, need_eq - eq), el = min(m.eq_low, left), eh = min(m.eq_high, left - el);
        kept_low += m.gt_low + el;
        kept_high += m.gt_high + eh;
        eq += m.eq_low + m.eq_high;
    };
    for (int x = 0; x < rank; ++x) add(sh.cta_counts[x]);
    for (int x = 0; x < warp; ++x) add(sh.warp_counts[x]);
    {
        const int e0 = eq, l0 = kept_low, h0 = kept_high;
        if (rank == 0 && warp == 0) {                 // all of them: what is listed
            for (int x = 0; x < C; ++x) add(sh.cta_counts[x]);
            listed = kept_high;
            eq = e0;
            kept_low = l0;
            kept_high = h0;
            if (lane == 0) a.lens_out[head] = t;      // every CTA has read lens
        }
    }
    int32_t* from = a.from + (size_t)head * a.B;
    int32_t* to = a.to + (size_t)head * a.B;
    const unsigned below = (1u << lane) - 1u;
    for (int j0 = w0; j0 < w1; j0 += 32) {
        const int j = j0 + lane;
        const bool in = j < w1;
        const uint32_t u = in ? key_at(j) & mask : 0u;
        const unsigned eqm = __ballot_sync(0xffffffffu, in && u == prefix);
        const bool kept = in && (u > prefix || (u == prefix && eq + __popc(eqm & below) < need_eq));
        const unsigned keptm = __ballot_sync(0xffffffffu, kept);
        const unsigned lowm = __ballot_sync(0xffffffffu, j < split);
        if (in && j < split) {
            if (kept) {
                if (src) src[j] = j;
            } else {
                // evicted places before j: candidates below it less those kept
                const int at = (j - s) - (kept_low + __popc(keptm & lowm & below));
                if (KVP_CHECK(at >= 0 && at < a.B, 701, head, at)) to[at] = j;
            }
        } else if (kept) {
            const int at = kept_high + __popc(keptm & ~lowm & below);
            if (KVP_CHECK(at < a.B, 702, head, at)) from[at] = j;
        }
        kept_low += __popc(keptm & lowm);
        kept_high += __popc(keptm & ~lowm);
        eq += __popc(eqm);
    }
    if (src)
        for (int i = rank * threads + tid; i < s; i += C * threads) src[i] = i;
    // listed rows below t, for evict_move: the first of the list
    cg::this_cluster().sync();                        // the lists are there
    if (rank == 0 && warp == 0) {
        int early = 0;
        for (int i = lane; i - lane < min(listed, w); i += 32)
            early += __popc(__ballot_sync(0xffffffffu, i < min(listed, w) && from[i] < t));
        if (lane == 0) a.info[head] = make_int4(n, t, listed, 1 + early);
    }
}

// Copies rows pair(i) = (source, place) of a head, i in [first, last), `chunk` (up to 32) at a time by
// each warp: a lane looks up one row's pages and copies its weight; then the warp copies the
// rows, kLoads loads in flight. kBarrier: all rows of a round (kLoads loads a warp) are read by
// every thread of the block before any is written.
template <int D, int kLoads, bool kBarrier, typename PairOf>
__device__ __forceinline__ void move_rows(const EvictArgs& a, int head, int first, int last, int stride, int chunk,
                                          int warp, PairOf pair) {
    constexpr int kPieces = D / 8, kLanes = 2 * kPieces, kAtOnce = 32 / kLanes;   // rows a load instruction covers
    constexpr int kBatch = kLoads * kAtOnce;
    const int lane = threadIdx.x & 31, piece = lane % kPieces, sub = lane / kLanes;
    uint4* pool = (lane / kPieces) & 1 ? a.v_pages : a.k_pages;
    for (int round = first; round < last; round += stride) {
        const int base = round + warp * chunk, here = min(chunk, last - base);   // rows of this warp (may be < 1)
        long long from = -1, to = -1;
        float weight = 0.f;
        if (lane < here) {
            const int2 p = pair(base + lane);
            if (KVP_CHECK(p.x >= 0 && p.x < a.c.cap() && p.y >= 0 && p.y < min(a.B, a.c.cap()), 703, p.x, p.y)) {
                from = a.c.row(head, p.x);
                to = a.c.row(head, p.y);
                if (a.src) a.src[(size_t)head * a.B + p.y] = p.x;
            }
            if (from < 0) to = -1;
            if (to >= 0) weight = a.acc[from];
        }
        if (!kBarrier && to >= 0) a.acc_out[to] = weight;
        for (int i0 = 0; i0 < (kBarrier ? kBatch : here); i0 += kBatch) {
            uint4 x[kLoads];
            long long at[kLoads];
#pragma unroll
            for (int r = 0; r < kLoads; ++r) {
                const int i = i0 + r * kAtOnce + sub;
                const long long f = __shfl_sync(0xffffffffu, from, i & 31);
                at[r] = __shfl_sync(0xffffffffu, to, i & 31);
                if (i >= here) at[r] = -1;
                if (at[r] >= 0) x[r] = pool[f * kPieces + piece];
            }
            if (kBarrier) __syncthreads();
#pragma unroll
            for (int r = 0; r < kLoads; ++r)
                if (at[r] >= 0) pool[at[r] * kPieces + piece] = x[r];
            if (kBarrier && to >= 0) a.acc_out[to] = weight;
        }
        if (kBarrier) __syncthreads();
    }
}
// Rows that a warp's kLoads loads cover.
template <int D>
__host__ __device__ constexpr int batch_rows(int loads) {
    return loads * (32 / (D / 4));
}

// parts + 1 blocks per head: the first copies the listed rows below t, then the window; the others
// share the rest of the list, and (fill) first write what evict_select left of src and acc_out: rows
// that keep their places, and -1 past the new length.
template <int D>
__global__ void __launch_bounds__(kMoveThreads, kMoveCtas) evict_move(const EvictArgs a, int parts, int chunk, bool fill) {
    constexpr int kWarps = kMoveThreads / 32, kBatch = batch_rows<D>(kMoveLoads);
    ptx::grid_dependency_wait();
    const int head = blockIdx.x / (parts + 1), part = blockIdx.x % (parts + 1), warp = threadIdx.x >> 5;
    const int4 info = a.info[head];
    const int n = info.x, t = info.y, listed = info.z, early = info.w - 1, w = a.w, round = chunk * kWarps;
    if (fill && part > 0) {
        const bool full = n > t, copy = a.acc_out != a.acc;
        const int last = full ? t : n, split = full ? t - w : n;
        int32_t* src = a.src ? a.src + (size_t)head * a.B : nullptr;
        const int first = ((part - 1) * kMoveThreads + threadIdx.x) * 4, step = parts * kMoveThreads * 4;
        for (int j = first; j < split && (src || copy); j += step) {   // four rows: they lie in one page
            const int here = min(4, split - j);
            const uint32_t bits = full ? a.stays[(size_t)head * a.stays_stride + j / 8] >> (j & 4) : 15u;
            const long long row = copy ? a.c.row(head, j) : -1;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (row >= 0) x = *(const float4*)(a.acc + row);
            const float v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i >= here || !(bits >> i & 1)) continue;
                if (src) src[j + i] = j + i;
                if (row >= 0) a.acc_out[row + i] = v[i];
            }
        }
        if (src)
            for (int j = last + (part - 1) * kMoveThreads + threadIdx.x; j < a.B; j += parts * kMoveThreads) src[j] = -1;
    }
    if (early < 0) return;
    const int32_t* from = a.from + (size_t)head * a.B;
    const int32_t* to = a.to + (size_t)head * a.B;
    auto pair = [&](int i) { return make_int2(from[i], to[i]); };
    if (part == 0) {
        move_rows<D, kMoveLoads, false>(a, head, 0, early, kWarps * kBatch, kBatch, warp, pair);
        __syncthreads();
        move_rows<D, kMoveLoads, true>(a, head, 0, w, kWarps * kBatch, kBatch, warp,
                                       [&](int i) { return make_int2(n - w + i, t - w + i); });
    } else {
        move_rows<D, kMoveLoads, false>(a, head, early + (part - 1) * round, listed, parts * round, chunk, warp, pair);
    }
}

// The listed rows, then the window, by one CTA.
template <int D>
__device__ __forceinline__ void own_moves(const EvictArgs& a, int head, int n, int t, int listed, const int* from, const int* to) {
    constexpr int kBatch = batch_rows<D>(kOwnLoads);
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5, w = a.w;
    move_rows<D, kOwnLoads, false>(a, head, 0, listed, warps * kBatch, kBatch, warp,
                                   [&](int i) { return make_int2(from[i], to[i]); });
    __syncthreads();
    move_rows<D, kOwnLoads, true>(a, head, 0, w, warps * kBatch, kBatch, warp,
                                  [&](int i) { return make_int2(n - w + i, t - w + i); });
}

constexpr int kBins = 256;

template <int C>
struct PickShared {
    union {
        __align__(16) uint32_t hist[4][kBins];       // of this CTA's keys, a digit a round; or
        uint2 light[C == 1 ? kMaxWarps : 1][kLight]; // a warp's lightest rows, in the order they go: key, row
    };
    __align__(16) uint32_t all[2][C > 1 ? C : 1][kBins];   // every CTA's, of the cluster
    unsigned long long warp_scan[kMaxWarps];         // packed counts: a warp's, then those before it
    unsigned long long cta_scan[C];                  // every CTA's
    uint32_t T;                                      // what warp 0 found in the last round
    int above;
    bool exact;
    int listed;
    int from[C == 1 ? kOwn : 1], to[C == 1 ? kOwn : 1];   // listed rows, where they are copied here;
    long long to_row[kFew];                          // where the places lie in the pool;
    long long row[kFew];                             // rows [t - w, n): where they lie (-1: no page),
    float weight[kFew];                              // and their weights
};

// Counts of a run of rows, 16 bits each: kept by their key (gt) or equal to T (eq), below split (low)
// and not.
__device__ __forceinline__ unsigned long long pack4(int gt_low, int eq_low, int gt_high, int eq_high) {
    return (unsigned long long)gt_low | (unsigned long long)eq_low << 16 | (unsigned long long)gt_high << 32 |
           (unsigned long long)eq_high << 48;
}

__device__ __forceinline__ unsigned long long warp_inclusive(unsigned long long x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// A warp lists its rows: put(i, j) for each of them, j ascending, i from this thread's `at` on for its own.
// bits: of rows [j0, j0 + kPer). 32 rows at a time, so that a warp's entries lie side by side (a
// thread that writes its own rows' touches a sector each: 8 heads of 131072 rows: 65 us, 61.5 so).
template <int kPer, typename Put>
__device__ __forceinline__ void list_rows(uint32_t bits, int at, int j0, Put put) {
    constexpr int kShare = 32 / kPer;                // threads that have 32 rows
    if (!__any_sync(0xffffffffu, bits)) return;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < kShare; o <<= 1) bits |= __shfl_down_sync(0xffffffffu, bits, o) << (o * kPer);
    j0 = __shfl_sync(0xffffffffu, j0, 0) + lane;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
        const uint32_t word = __shfl_sync(0xffffffffu, bits, q * kShare);
        const int first = __shfl_sync(0xffffffffu, at, q * kShare);
        if (word >> lane & 1) put(first + __popc(word & ((1u << lane) - 1)), j0 + 32 * q);
    }
}

template <int C, int kPer, int kThreads = kMaxThreads, int kCtas = 1>
__global__ void __launch_bounds__(kThreads, kCtas) evict_select(const EvictArgs a) {
    extern __shared__ __align__(16) uint32_t keys[];   // (C = 1) rows [t - w, n), where they are few
    __shared__ PickShared<C> sh;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 31, warp = tid >> 5, warps = threads >> 5;
    const int head = blockIdx.x / C, rank = blockIdx.x % C;
    const int n = a.c.len(head);
    const int t = a.budgets ? min(max(a.budgets[head], max(a.s + a.w, 1)), a.B) : a.B;
    const int w = a.w, s = a.s;
    const bool full = n > t;
    if (C > 1) ptx::cluster_arrive();                     // this thread has read lens
    const int split = full ? t - w : n;              // rows below keep their places, or are replaced
    int32_t* src = a.src ? a.src + (size_t)head * a.B : nullptr;
    const bool fill = C == 1;                        // (a cluster leaves it to evict_move)
    // With few rows past t - w, all that can move are fetched while the rest is worked out.
    const bool here = C == 1 && full && n - split <= kFew;

    // ---- rows [j0, j0 + kPer) are this thread's. A key is the weight's bits plus one; 0: no candidate.
    const int j0 = (rank * threads + tid) * kPer;
    uint32_t key[kPer];
    if (full || fill) {
        const int32_t* table = a.c.table + (size_t)head * a.c.max_pages;
        float4 x[kPer / 4];
        long long row[kPer / 4];
#pragma unroll
        for (int q = 0; q < kPer / 4; ++q) {
            const int j = j0 + 4 * q;                // four rows lie in one page
            const int page = j < n ? table[j >> a.c.page_shift] : -1;
            row[q] = page < 0 || page >= a.c.num_pages
                         ? -1 : ((long long)page << a.c.page_shift) + (j & ((1 << a.c.page_shift) - 1));
        }
        // of the rows that may move, this warp's: r = warp + warps * lane
        const int r_mine = warp + warps * lane;
        const long long r_row = here && r_mine < n - split ? a.c.row(head, split + r_mine) : -1;
#pragma unroll
        for (int q = 0; q < kPer / 4; ++q) x[q] = row[q] >= 0 ? *(const float4*)(a.acc + row[q]) : make_float4(0.f, 0.f, 0.f, 0.f);
        if (here) {
            const int chunks = a.row_chunks;         // 16-byte chunks of a row of keys (then as many of values)
            if (r_mine < n - split) {
                sh.row[r_mine] = r_row;
                if (r_row >= 0)
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(ptx::smem_u32(&sh.weight[r_mine])), "l"(a.acc + r_row) : "memory");
            }
            const uint4* pool = (lane < chunks ? a.k_pages : a.v_pages) + (lane & (chunks - 1));
            for (int r = warp, i = 0; r < n - split; r += warps, ++i) {
                const long long from = __shfl_sync(0xffffffffu, r_row, i);
                if (from >= 0 && lane < 2 * chunks)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                     ptx::smem_u32((uint4*)keys + r * 2 * chunks + lane)), "l"(pool + from * chunks) : "memory");
            }
        }
#pragma unroll
        for (int q = 0; q < kPer / 4; ++q) {
            const float v[4] = {x[q].x, x[q].y, x[q].z, x[q].w};
            const int j = j0 + 4 * q;
#pragma unroll
            for (int i = 0; i < 4; ++i) key[4 * q + i] = key_of(v[i]) + 1;
            if (fill && row[q] >= 0 && a.acc_out != a.acc) {
                if (j + 4 <= split) {
                    *(float4*)(a.acc_out + row[q]) = x[q];
                } else {
#pragma unroll
                    for (int i = 0; i < 3; ++i)
                        if (j + i < split) a.acc_out[row[q] + i] = v[i];
                }
            }
        }
    }
    if (fill && src) {
        // rows that stay (those that move write theirs later), and what lies past the new length
        const int last = full ? t : n;
        for (int i = tid; i < a.B; i += threads) {
            if (i < split) src[i] = i;
            else if (i >= last) src[i] = -1;
        }
    }
    if (!full) {
        if (C > 1) ptx::cluster_wait();
        if (rank == 0 && tid == 0) {
            a.info[head] = make_int4(n, t, 0, 0);
            a.lens_out[head] = n;
        }
        return;                                      // the same in every CTA of the cluster
    }
    // a bit a row: candidates, and rows below split
    constexpr uint32_t kAllRows = (1u << kPer) - 1;
    auto first_bits = [&](int last) { return last <= j0 ? 0u : last - j0 >= kPer ? kAllRows : (1u << (last - j0)) - 1; };
    const uint32_t cand = first_bits(n - w) & ~first_bits(s), low = first_bits(split);
    if (cand != kAllRows) {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (!(cand >> i & 1)) key[i] = 0;
    }
    int32_t* from = a.from + (size_t)head * a.B;
    int32_t* to = a.to + (size_t)head * a.B;
    int listed = 0;
    const bool own = here || (C == 1 && a.many && n - split <= kOwn);   // this CTA copies the rows
    if (here && n - t <= kLight) {
        // ---- the n - t rows that go, one by one: the smallest key, of equal ones the highest row
        const int gone = n - t;
        uint32_t least = 0xFFFFFFFFu;                // this thread's smallest key, and its highest row that has it
        int which = 0;
        auto look = [&]() {
            least = 0xFFFFFFFFu;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (key[i] != 0 && key[i] <= least) least = key[i], which = i;
        };
        look();
        for (int i = 0; i < gone; ++i) {
            const uint32_t m = __reduce_min_sync(0xffffffffu, least);
            const int owner = 31 - __clz(__ballot_sync(0xffffffffu, least == m));
            if (lane == owner) {
                sh.light[warp][i] = make_uint2(m, (uint32_t)(j0 + which));
#pragma unroll
                for (int x = 0; x < kPer; ++x)
                    if (x == which) key[x] = 0;
                look();
            }
        }
        __syncthreads();
        if (warp == 0) {
            int taken = 0;                           // lane x: of warp x's rows
            uint2 next = lane < warps ? sh.light[lane][0] : make_uint2(0xFFFFFFFFu, 0u);
            uint32_t mine = 0xFFFFFFFFu;             // lane i: the i-th row that goes
            for (int i = 0; i < gone; ++i) {
                const uint32_t m = __reduce_min_sync(0xffffffffu, next.x);
                const int owner = 31 - __clz(__ballot_sync(0xffffffffu, next.x == m));   // a higher warp has higher rows
                const uint32_t row = __shfl_sync(0xffffffffu, next.y, owner);
                if (lane == i) mine = row;
                if (lane == owner) next = ++taken < gone ? sh.light[lane][taken] : make_uint2(0xFFFFFFFFu, 0u);
            }
            // [split, split + gone) are the candidates past split: those that stay take the places below it
            const bool is_low = lane < gone && (int)mine < split;
            const unsigned lows = __ballot_sync(0xffffffffu, is_low);
            const uint32_t high_bit = lane < gone && !is_low ? 1u << (mine - split) : 0u;
            const uint32_t stay_high = ((1u << gone) - 1) & ~__reduce_or_sync(0xffffffffu, high_bit);
            int place = 0;                           // evicted places below this one
            for (int x = 0; x < gone; ++x) {
                const uint32_t other = __shfl_sync(0xffffffffu, mine, x);
                place += (lows >> x & 1) && other < mine;
            }
            if (is_low && KVP_CHECK(place < kFew, 705, head, place)) {
                sh.to[place] = (int)mine;
                sh.to_row[place] = a.c.row(head, (int)mine);
            }
            if (stay_high >> lane & 1) sh.from[__popc(stay_high & ((1u << lane) - 1))] = split + lane;
            if (lane == 0) {
                sh.listed = __popc(lows);
                a.info[head] = make_int4(n, t, __popc(lows), 0);
                a.lens_out[head] = t;
            }
        }
        __syncthreads();
        listed = sh.listed;
    } else {
        for (int i = tid; i < 4 * kBins; i += threads) (&sh.hist[0][0])[i] = 0;
        if (C > 1) ptx::cluster_wait();                       // every CTA of the cluster runs and has read lens
        __syncthreads();

        // ---- T: the largest value that at least kk keys reach
        const int kk = t - s - w;                        // candidates that stay; there are more than kk
        uint32_t T = kk > 0 ? 0u : 0xFFFFFFFFu;
        int above = 0;                                   // keys known to lie above those that T's bits leave open
        bool exact = kk == 0;                            // just kk keys reach T
#pragma unroll
        for (int round = 0; round < 4; ++round) {
            if (exact) break;
            const int bits = round < 3 ? 8 : 7, shift = round < 3 ? 23 - 8 * round : 0;
            uint32_t* hist = sh.hist[round];
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                // the bits above this digit are T's, and it is a candidate
                if (key[i] != 0 && (round == 0 || (key[i] ^ T) >> (shift + bits) == 0))
                    atomicAdd(&hist[key[i] >> shift & ((1u << bits) - 1)], 1u);
            }
            __syncthreads();
            if (C > 1) {                                 // every CTA gets every CTA's counts
                for (int i = tid; i < C * kBins / 4; i += threads) {
                    uint4* to = (uint4*)sh.all[round & 1][rank] + i % (kBins / 4);
                    *cg::this_cluster().map_shared_rank(to, i / (kBins / 4)) = ((const uint4*)hist)[i % (kBins / 4)];
                }
                sync_all<C>();
            }
            if (warp == 0) {
                // lane x: digits 255 - 8 x down to 248 - 8 x
                int bin[8] = {};
#pragma unroll
                for (int x = 0; x < C; ++x) {
                    const uint4* from = (const uint4*)((C > 1 ? sh.all[round & 1][x] : hist) + kBins - 8 - 8 * lane);
                    const uint4 lo = from[0], hi = from[1];
                    bin[0] += hi.w, bin[1] += hi.z, bin[2] += hi.y, bin[3] += hi.x;
                    bin[4] += lo.w, bin[5] += lo.z, bin[6] += lo.y, bin[7] += lo.x;
                }
                int inc = ((bin[0] + bin[1]) + (bin[2] + bin[3])) + ((bin[4] + bin[5]) + (bin[6] + bin[7]));
                const int sum = inc;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += y;
                }
                const int want = kk - above;             // the want-th key from the top is T
                if (inc - sum < want && want <= inc) {   // one lane: there are more than kk keys
                    int before = inc - sum, digit = 255 - 8 * lane, count = 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        count = bin[i];
                        if (before + count >= want) break;
                        before += count;
                        --digit;
                    }
                    sh.T = T | (uint32_t)digit << shift;
                    sh.above = above + before;
                    sh.exact = before + count == want;
                }
            }
            __syncthreads();
            T = sh.T;
            above = sh.above;
            exact = sh.exact;
            // (warp 0 writes them again only after the next round's barrier)
        }
        // rows whose key is T that stay, lowest first; none is needed where just kk keys reach T
        const int need_eq = exact ? 0 : kk - above;
        const uint32_t over = exact ? T - 1 : T;     // (T > 0 where just kk reach it: all candidates, which are more, reach 0)
        uint32_t gt = 0, eqm = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) gt |= key[i] > over ? 1u << i : 0u;
        if (!exact) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) eqm |= key[i] == T ? 1u << i : 0u;
        }

        // ---- places in the lists: counts before this thread's rows
        const unsigned long long mine = pack4(__popc(gt & low), __popc(eqm & low), __popc(gt & ~low), __popc(eqm & ~low));
        unsigned long long before = warp_inclusive(mine) - mine;
        if (lane == 31) sh.warp_scan[warp] = before + mine;
        __syncthreads();
        if (warp == 0) {
            const unsigned long long v = lane < warps ? sh.warp_scan[lane] : 0ull, inc = warp_inclusive(v);
            if (lane < warps) sh.warp_scan[lane] = inc - v;
            const unsigned long long all = __shfl_sync(0xffffffffu, inc, 31);
            if (C > 1) {
                if (lane < C) *cg::this_cluster().map_shared_rank(&sh.cta_scan[rank], lane) = all;
            } else if (lane == 0) {
                sh.cta_scan[0] = all;
            }
        }
        sync_all<C>();
        before += sh.warp_scan[warp];
        // 16 bits hold a CTA's counts, not a cluster's
        int b_gt_low = (int)(before & 0xFFFF), b_eq_low = (int)(before >> 16 & 0xFFFF), b_gt_high = (int)(before >> 32 & 0xFFFF),
            b_eq_high = (int)(before >> 48), all_eq_low = 0, all_gt_high = 0, all_eq_high = 0;
#pragma unroll
        for (int x = 0; x < C; ++x) {
            const unsigned long long v = sh.cta_scan[x];
            const int gl = (int)(v & 0xFFFF), el = (int)(v >> 16 & 0xFFFF), gh = (int)(v >> 32 & 0xFFFF), eh = (int)(v >> 48);
            if (x < rank) b_gt_low += gl, b_eq_low += el, b_gt_high += gh, b_eq_high += eh;
            all_eq_low += el;
            all_gt_high += gh;
            all_eq_high += eh;
        }
        // equal rows stay from the lowest on, and the low ones come first
        listed = all_gt_high + min(all_eq_low + all_eq_high, need_eq) - min(all_eq_low, need_eq);
        const int eq = b_eq_low + b_eq_high, room = max(0, need_eq - eq);    // equal rows before; of this thread's, that stay
        const int kept_low = b_gt_low + min(b_eq_low, need_eq);
        const int kept_high = b_gt_high + min(eq, need_eq) - min(b_eq_low, need_eq);
        while (__popc(eqm) > room) eqm &= ~(1u << (31 - __clz(eqm)));         // drops the highest
        const uint32_t kept = gt | eqm;
        // evicted places: candidates before this thread's rows less those kept
        int at = max(0, min(j0, n - w) - s) - kept_low;
        uint32_t out_low = cand & low & ~kept, in_high = kept & ~low;
        const int early = kept_high + __popc(in_high & first_bits(t));       // listed rows below t, if row t is this thread's
        if (own) {
            for (; out_low; out_low &= out_low - 1, ++at) {
                const int j = j0 + __ffs(out_low) - 1;
                if (!KVP_CHECK(at >= 0 && at < (here ? kFew : kOwn), 706, head, at)) break;
                sh.to[at] = j;
                if (here) sh.to_row[at] = a.c.row(head, j);
            }
            at = kept_high;
            for (; in_high; in_high &= in_high - 1, ++at)
                if (KVP_CHECK(at >= 0 && at < kOwn, 707, head, at)) sh.from[at] = j0 + __ffs(in_high) - 1;
        } else {
            list_rows<kPer>(out_low, at, j0, [&](int i, int j) { if (KVP_CHECK(i >= 0 && i < a.B, 701, head, i)) to[i] = j; });
            list_rows<kPer>(in_high, kept_high, j0, [&](int i, int j) { if (KVP_CHECK(i >= 0 && i < a.B, 702, head, i)) from[i] = j; });
        }
        if (!fill) {
            // evict_move fills in src and acc_out of the rows that stay: a bit each
            const uint32_t stays = low & (kept | first_bits(s));
            if (j0 < split && KVP_CHECK((size_t)j0 / 8 + kPer / 8 <= a.stays_stride, 708, head, j0)) {
                if (kPer == 16) ((uint16_t*)a.stays)[((size_t)head * a.stays_stride + j0 / 8) / 2] = (uint16_t)stays;
                else a.stays[(size_t)head * a.stays_stride + j0 / 8] = (uint8_t)stays;
            }
        }
        if (j0 <= t && t < j0 + kPer)                    // row t is this thread's
            a.info[head] = make_int4(n, t, listed, own ? 0 : 1 + early);
        if (rank == 0 && tid == 0) a.lens_out[head] = t;
        // (the cluster's CTAs write into one another's shared memory only before the last sync_all)
    }
    if (here) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
        // a warp a row: the listed ones, then the window; all that is read is in shared memory
        const int chunks = a.row_chunks;
        uint4* pool = (lane < chunks ? a.k_pages : a.v_pages) + (lane & (chunks - 1));
        for (int i = warp; i < listed + w; i += warps) {
            const bool is_listed = i < listed;
            const int r = is_listed ? sh.from[i] - split : n - w - split + i - listed;     // source
            const int place = is_listed ? sh.to[i] : split + i - listed;
            if (!KVP_CHECK(r >= 0 && r < kFew && listed <= kFew && place >= 0 && place < t, 704, r, place)) continue;
            const long long to_row = is_listed ? sh.to_row[i] : sh.row[i - listed];
            if (src && lane == 0) src[place] = split + r;
            if (sh.row[r] < 0 || to_row < 0) continue;
            if (lane < 2 * chunks) pool[to_row * chunks] = ((const uint4*)keys)[r * 2 * chunks + lane];
            if (lane == 0) a.acc_out[to_row] = sh.weight[r];
        }
    } else if (own) {
        __syncthreads();
        if (a.row_chunks == 16) own_moves<128>(a, head, n, t, listed, sh.from, sh.to);
        else own_moves<64>(a, head, n, t, listed, sh.from, sh.to);
    }
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// `kernel` with clusters of C CTAs, one per head.
cudaError_t launch_heads(void (*kernel)(const EvictArgs), const EvictArgs& a, int C, int threads, size_t smem,
                         cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.c.heads * C));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = C > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

// Bytes of a head's bits, a multiple of two (evict_select writes 16 of them at a time).
static size_t stays_stride(const kvp_cache_shape& s) { return (size_t)s.max_pages * s.page_size / 8; }

size_t evict_workspace_bytes(const kvp_cache_shape& s, const kvp_evict& e) {
    const size_t heads = (size_t)s.batch * s.hkv;
    return align256(heads * sizeof(int4)) + 2 * align256(heads * e.budget * sizeof(int32_t)) +
           align256(heads * stays_stride(s));
}

cudaError_t launch_evict(const kvp_cache_shape& s, const kvp_evict& e, const int32_t* budgets,
                         uint16_t* k_pages, uint16_t* v_pages, const float* acc, float* acc_out,
                         const int32_t* table, const int32_t* lens, int32_t* lens_out, int32_t* src,
                         void* workspace, cudaStream_t st) {
    const int heads = s.batch * s.hkv, cap = s.max_pages * s.page_size;
    char* ws = (char*)workspace;
    EvictArgs a;
    a.c = cache_view(s, table, lens);
    a.acc = acc;
    a.acc_out = acc_out;
    a.k_pages = (uint4*)k_pages;
    a.v_pages = (uint4*)v_pages;
    a.budgets = budgets;
    a.lens_out = lens_out;
    a.src = src;
    a.B = e.budget;
    a.s = e.sinks;
    a.w = e.window;
    a.info = (int4*)ws;
    a.from = (int32_t*)(ws + align256((size_t)heads * sizeof(int4)));
    a.to = (int32_t*)(ws + align256((size_t)heads * sizeof(int4)) + align256((size_t)heads * e.budget * 4));
    a.stays = (uint8_t*)(ws + align256((size_t)heads * sizeof(int4)) + 2 * align256((size_t)heads * e.budget * 4));
    a.stays_stride = stays_stride(s);
    a.slice = 0;
    a.row_chunks = s.head_dim / 8;
    a.many = heads >= num_sms();
    // CTAs per head: 8 where rows are many and heads few. (8 heads of 16384 rows: 15.0 us, 17.8 by a CTA each; 32: 37.3,
    // 37.9; 72 of 12000: 39.0, 31.1; 32 of 8192: 28.9, 27.4; 8 of 8192: 13.5, 13.8.)
    const int sms = num_sms();
    const int C = cap > 8192 && (heads * 4 < sms || cap > kMaxThreads * kPerMost) ? 8 : 1;
    const int slice = (cap + C - 1) / C;
    cudaError_t err;
    bool fill = false;
    if (slice <= kMaxThreads * kPerMost) {
        // 8 keys a thread, or 16 where the threads that takes would keep other CTAs off their SM: a
        // cluster's more than run at once (64 heads of 30000 rows: 65 us with 8, 59 with 16; 24 of 24000: 44.9, 46.4),
        // a CTA's more than kManyThreads. 256 threads at least: they copy rows too.
        const int with8 = std::max(256, (slice + 255) / 256 * 32);
        const bool fit8 = C == 1 ? with8 <= kManyThreads : with8 <= 256 || heads <= kMaxThreads / with8 * kClusters;
        const int per = fit8 ? 8 : kPerMost;
        const int threads = std::max(256, (slice + per * 32 - 1) / (per * 32) * 32);
        if (C == 8) {
            err = launch_heads(per == 8 ? evict_select<8, 8> : evict_select<8, kPerMost>, a, C, threads, 0, st);
            fill = true;
        } else {
            err = launch_heads(per == 8 ? evict_select<1, 8, kManyThreads, 3> : evict_select<1, kPerMost>, a, C, threads, (size_t)kFew * s.head_dim * 4, st);
        }
    } else {
        a.slice = (slice + 15) / 16 * 16 <= kSliceCap ? (slice + 15) / 16 * 16 : 0;
        err = allow_dynamic_smem((const void*)evict_select_long<8>, (size_t)a.slice * 4);
        if (err == cudaSuccess) err = launch_heads(evict_select_long<8>, a, 8, kMaxThreads, (size_t)a.slice * 4, st);
    }
    if (err != cudaSuccess) return err;
    // rows that can change places per head; blocks enough to fill the card with them
    // evict_select copies them all where a head can have but few
    if (C == 1 && !budgets && cap - e.budget + e.window <= (a.many ? kOwn : kFew)) return cudaSuccess;
    const int most = std::min(e.budget, std::max(0, cap - e.budget));
    // rows a warp takes at a time: 32, fewer where that would leave warps without any
    const int warps = sms * kMoveCtas * (kMoveThreads / 32), batch = s.head_dim == 128 ? batch_rows<128>(kMoveLoads) : batch_rows<64>(kMoveLoads);
    const int chunk = (int)std::min<long long>(32, std::max<long long>(batch, (long long)heads * most / warps / batch * batch));
    const int round = chunk * (kMoveThreads / 32);
    const int filled = fill ? std::min(e.budget, cap) : 0;
    const int want = std::max((most + round - 1) / round, (filled + kMoveThreads * 4 - 1) / (kMoveThreads * 4));
    // one wave of blocks for few heads; for many, whose share of a wave would be a block or less, four
    const int wave = sms * kMoveCtas;
    const int parts = std::max(1, std::min(want, heads * 4 <= wave ? wave / heads - 1 : (4 * wave + heads - 1) / heads));
    return s.head_dim == 128 ? launch_dependent(evict_move<128>, heads * (parts + 1), kMoveThreads, 0, st, a, parts, chunk, fill)
                             : launch_dependent(evict_move<64>, heads * (parts + 1), kMoveThreads, 0, st, a, parts, chunk, fill);
}

#ifdef KVP_CHECKS
KVP_DEFINE_CHECK_READER(take_check_evict)
#endif

}  // namespace kvp
