// Eviction from a paged cache by accumulated attention weight, in place.
//
// evict_select: a cluster of C CTAs per head. Each CTA holds the keys of a slice of the head's
// rows in shared memory: a weight's bits, which order as the weights do (all are non-negative
// or count as zero). A radix select, four bits a round from the top, finds the key T of the
// last row that stays: every thread counts its keys' digits in 16 packed byte counters, warps
// add them by redux, CTAs exchange 16 sums each, and every warp of every CTA finds the same
// digit, so a round costs one block barrier and (C > 1) one cluster barrier; no atomics, whatever
// the distribution. It stops early once all keys that share the prefix stay. The rows that
// change places are then listed, in row order, by counts exchanged once: the evicted places below
// t - w and the kept rows at or past it.
// evict_move: copies the listed rows (keys, values, weight), then the window. Only rows in
// [t - w, t) are both a source and a place to write to: the kept rows there are the first of
// the list, and the block that copies them copies the window after them.
#include <cooperative_groups.h>

#include <algorithm>

#include "kvp_cache.cuh"
#include "kvp_ptx.cuh"

namespace cg = cooperative_groups;

namespace kvp {
namespace {

constexpr int kMaxThreads = 1024, kMaxWarps = kMaxThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kSliceCap = 48 * 1024;     // keys a CTA holds in shared memory
constexpr int kMoveThreads = 256, kMoveRows = 4;

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
    int4* info;               // [heads]: n, t, rows listed, -
    int32_t* from;            // [heads][B]: listed rows, ascending
    int32_t* to;              // [heads][B]: the places they move to, ascending
    int slice;                // keys that shared memory holds per CTA; 0: keys are read from acc again and again
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
__global__ void __launch_bounds__(kMaxThreads, 1) evict_select(const EvictArgs a) {
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
            if (in_smem && full)
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
            if (lane == 0) {
                a.info[head] = make_int4(n, t, listed, 0);
                a.lens_out[head] = t;                 // every CTA has read lens
            }
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
    if (C > 1) cg::this_cluster().sync();             // shared memory outlives its readers
}

// Rows `from` -> `to` of a head, kMoveRows at a time per group of lanes; all rows of a round are
// read before any is written (by every thread of the block when kBarrier).
template <int D, bool kBarrier, typename Pair>
__device__ __forceinline__ void move_rows(const EvictArgs& a, int head, int first, int last, int stride, Pair pair) {
    constexpr int kPieces = D / 8, kLanes = 2 * kPieces, kGroups = kMoveThreads / kLanes;
    const int lane = threadIdx.x % kLanes, piece = lane % kPieces, group = threadIdx.x / kLanes;
    uint4* pool = lane >= kPieces ? a.v_pages : a.k_pages;
    for (int base = first; base < last; base += stride) {
        uint4 x[kMoveRows];
        float wt[kMoveRows];
        long long dst[kMoveRows];
#pragma unroll
        for (int r = 0; r < kMoveRows; ++r) {
            dst[r] = -1;
            const int i = base + r * kGroups + group;
            if (i >= last) continue;
            const int2 p = pair(i);
            const long long from = a.c.row(head, p.x), to = a.c.row(head, p.y);
            if (a.src && lane == 0) a.src[(size_t)head * a.B + p.y] = p.x;
            if (from < 0 || to < 0) continue;
            dst[r] = to;
            x[r] = pool[from * kPieces + piece];
            if (lane == 0) wt[r] = a.acc[from];
        }
        if (kBarrier) __syncthreads();
#pragma unroll
        for (int r = 0; r < kMoveRows; ++r) {
            if (dst[r] < 0) continue;
            if (!KVP_CHECK(dst[r] < ((long long)a.c.num_pages << a.c.page_shift), 703, head, base)) continue;
            pool[dst[r] * kPieces + piece] = x[r];
            if (lane == 0) a.acc_out[dst[r]] = wt[r];
        }
        if (kBarrier) __syncthreads();
    }
}

// parts blocks per head: the listed rows that lie past t are dealt over all of them; block 0 first
// copies those below t, then the window.
template <int D>
__global__ void __launch_bounds__(kMoveThreads) evict_move(const EvictArgs a, int parts) {
    constexpr int kRound = kMoveThreads / (D / 4) * kMoveRows;
    ptx::grid_dependency_wait();
    const int head = blockIdx.x / parts, part = blockIdx.x % parts;
    const int4 info = a.info[head];
    const int n = info.x, t = info.y, listed = info.z, w = a.w;
    if (n <= t) return;
    const int32_t* from = a.from + (size_t)head * a.B;
    const int32_t* to = a.to + (size_t)head * a.B;
    auto pair = [&](int i) { return make_int2(from[i], to[i]); };
    // listed rows in [t - w, t): the first of the list
    int early = 0;
    for (int i = 0; i < min(listed, w); i += kMoveThreads)
        early += __syncthreads_count(i + (int)threadIdx.x < min(listed, w) && from[i + threadIdx.x] < t);
    if (part == 0) {
        move_rows<D, false>(a, head, 0, early, kRound, pair);
        __syncthreads();
        move_rows<D, true>(a, head, 0, w, kRound, [&](int i) { return make_int2(n - w + i, t - w + i); });
    }
    move_rows<D, false>(a, head, early + part * kRound, listed, parts * kRound, pair);
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

template <int C>
cudaError_t launch_select_c(const EvictArgs& a, int threads, size_t smem, cudaStream_t st) {
    const cudaError_t e = allow_dynamic_smem((const void*)evict_select<C>, smem);
    if (e != cudaSuccess) return e;
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
    return cudaLaunchKernelEx(&cfg, evict_select<C>, a);
}

}  // namespace

size_t evict_workspace_bytes(const kvp_cache_shape& s, const kvp_evict& e) {
    const size_t heads = (size_t)s.batch * s.hkv;
    return align256(heads * sizeof(int4)) + 2 * align256(heads * e.budget * sizeof(int32_t));
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
    // CTAs per head: 8 where the heads alone would leave most SMs idle and rows are many
    const int sms = num_sms();
    const int C = (long long)cap > 4096 && (heads * 2 < sms || cap > kSliceCap) ? 8 : 1;
    const int slice = ((cap + C - 1) / C + 15) / 16 * 16;
    a.slice = slice <= kSliceCap ? slice : 0;
    const size_t smem = (size_t)a.slice * 4;
    int threads = 128;
    while (threads < kMaxThreads && threads * 8 < slice) threads *= 2;
    cudaError_t err = C == 8 ? launch_select_c<8>(a, threads, smem, st) : launch_select_c<1>(a, threads, smem, st);
    if (err != cudaSuccess) return err;
    // rows that can change places per head, and blocks enough to fill the card with them
    const int round = kMoveThreads / (s.head_dim / 4) * kMoveRows;
    const int most = std::min(e.budget, std::max(0, cap - e.budget));
    const int parts = std::max(1, std::min((most + round - 1) / round, (sms * 6 + heads - 1) / heads));
    return s.head_dim == 128 ? launch_dependent(evict_move<128>, heads * parts, kMoveThreads, 0, st, a, parts)
                             : launch_dependent(evict_move<64>, heads * parts, kMoveThreads, 0, st, a, parts);
}

#ifdef KVP_CHECKS
KVP_DEFINE_CHECK_READER(take_check_evict)
#endif

}  // namespace kvp
