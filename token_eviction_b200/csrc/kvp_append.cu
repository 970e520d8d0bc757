// Appending rows to a paged cache: row i of a head's new rows becomes its row len + i.
//
// A bit copy, bound by HBM when rows are many and by the launch when there is one per head.
// A warp takes kRows rows at a time; the 2 d * 2 bytes of a row's key and value are 32 (d = 128)
// or 16 (d = 64) pieces of 16 bytes, one a lane, so every load and store covers whole rows, and
// the loads of all kRows rows are issued before the first store.
#include <algorithm>

#include "kvp_cache.cuh"
#include "kvp_ptx.cuh"

namespace kvp {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 4;      // rows in flight per group of lanes

struct AppendArgs {
    CacheView c;
    const uint4* k_new;
    const uint4* v_new;
    const int32_t* counts;   // NULL: n rows per head
    const float* weight;
    uint4* k_pages;
    uint4* v_pages;
    float* acc;
    int32_t* lens_out;       // NULL: left to append_lens
    int hkv, n;
    long long rows;          // b * hkv * n
};

// Row r of the flattened new rows: its head and its place among that head's new rows (head = -1:
// past the sequence's counts).
__device__ __forceinline__ void place_of(const AppendArgs& a, long long r, int& head, int& i) {
    if (a.counts == nullptr) {
        head = (int)(r / a.n);
        i = (int)(r - (long long)head * a.n);
        return;
    }
    const long long per = (long long)a.hkv * a.n;
    const int seq = (int)(r / per);
    long long left = r - seq * per;
    head = -1;
    for (int h = 0; h < a.hkv; ++h) {
        const int cnt = max(0, a.counts[(size_t)seq * a.hkv + h]);
        if (left < cnt) {
            head = seq * a.hkv + h;
            i = (int)left;
            return;
        }
        left -= cnt;
    }
}

// Rows that head `head` appends: its count, cut where the sequence's rows end.
__device__ __forceinline__ int rows_of(const int32_t* counts, int hkv, int n, int head) {
    if (counts == nullptr) return n;
    const int seq = head / hkv;
    long long left = (long long)hkv * n;
    int cnt = 0;
    for (int h = seq * hkv; h <= head; ++h) {
        cnt = (int)min((long long)max(0, counts[h]), left);
        left -= cnt;
    }
    return cnt;
}

template <int D>
__global__ void __launch_bounds__(kThreads) append_rows(const AppendArgs a) {
    constexpr int kPieces = D / 8;                 // 16-byte pieces of a key
    constexpr int kLanes = 2 * kPieces;            // lanes that carry one row
    ptx::grid_dependency_wait();
    const int lane = threadIdx.x % kLanes, piece = lane % kPieces;
    const bool is_v = lane >= kPieces;
    const uint4* from = is_v ? a.v_new : a.k_new;
    uint4* to = is_v ? a.v_pages : a.k_pages;
    const long long groups = (long long)gridDim.x * (kThreads / kLanes);
    const long long g0 = (long long)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
    for (long long base = g0 * kRows; base < a.rows; base += groups * kRows) {
        uint4 piece_of[kRows];
        long long dst[kRows];
#pragma unroll
        for (int t = 0; t < kRows; ++t) {
            dst[t] = -1;
            const long long r = base + t;
            if (r >= a.rows) continue;
            piece_of[t] = from[r * kPieces + piece];
            int head, i = 0;
            place_of(a, r, head, i);
            if (head < 0) continue;
            const long long j = (long long)a.c.len(head) + i;
            if (j < a.c.cap()) dst[t] = a.c.row(head, (int)j);
        }
#pragma unroll
        for (int t = 0; t < kRows; ++t) {
            if (dst[t] < 0) continue;
            if (!KVP_CHECK(dst[t] < ((long long)a.c.num_pages << a.c.page_shift), 501, (int)base, t)) continue;
            to[dst[t] * kPieces + piece] = piece_of[t];
            if (lane == 0 && a.acc) a.acc[dst[t]] = a.weight ? a.weight[base + t] : 0.f;
        }
    }
    if (a.lens_out) {
        for (int h = blockIdx.x * kThreads + threadIdx.x; h < a.c.heads; h += gridDim.x * kThreads)
            a.lens_out[h] = (int)min((long long)a.c.len(h) + rows_of(a.counts, a.hkv, a.n, h), (long long)a.c.cap());
    }
}

// lens in place: after every reader of the old lengths (append_rows) has finished.
__global__ void __launch_bounds__(kThreads) append_lens(const int32_t* counts, int32_t* lens, int heads, int hkv,
                                                        int n, int cap) {
    ptx::grid_dependency_wait();
    for (int h = blockIdx.x * kThreads + threadIdx.x; h < heads; h += gridDim.x * kThreads) {
        const int len = min(max(lens[h], 0), cap);
        lens[h] = (int)min((long long)len + rows_of(counts, hkv, n, h), (long long)cap);
    }
}

}  // namespace

cudaError_t launch_append(const kvp_cache_shape& s, const uint16_t* k_new, const uint16_t* v_new, int n,
                          const int32_t* counts, const float* weight, uint16_t* k_pages, uint16_t* v_pages,
                          float* acc, const int32_t* table, const int32_t* lens, int32_t* lens_out,
                          cudaStream_t st) {
    const bool in_place = lens_out == lens;
    AppendArgs a;
    a.c = cache_view(s, table, lens);
    a.k_new = (const uint4*)k_new;
    a.v_new = (const uint4*)v_new;
    a.counts = counts;
    a.weight = weight;
    a.k_pages = (uint4*)k_pages;
    a.v_pages = (uint4*)v_pages;
    a.acc = acc;
    a.lens_out = in_place ? nullptr : lens_out;
    a.hkv = s.hkv;
    a.n = n;
    a.rows = (long long)a.c.heads * n;
    const int per_cta = kThreads / (s.head_dim / 4) * kRows;
    const long long want = std::max<long long>(1, (a.rows + per_cta - 1) / per_cta);
    const int grid = (int)std::min<long long>(want, (long long)num_sms() * 8);
    cudaError_t e = s.head_dim == 128 ? launch_dependent(append_rows<128>, grid, kThreads, 0, st, a)
                                      : launch_dependent(append_rows<64>, grid, kThreads, 0, st, a);
    if (e != cudaSuccess || !in_place) return e;
    const int lgrid = std::min((a.c.heads + kThreads - 1) / kThreads, num_sms());
    return launch_dependent(append_lens, lgrid, kThreads, 0, st, counts, lens_out, a.c.heads, s.hkv, n, a.c.cap());
}

#ifdef KVP_CHECKS
KVP_DEFINE_CHECK_READER(take_check_append)
#endif

}  // namespace kvp
