// Appending rows to a paged cache: row i of a head's new rows becomes its row len + i.
//
// A bit copy, bound by HBM when rows are many and by the launch and three dependent reads (length,
// page, then the store) when there is one per head. A row's key and value are 32 (d = 128) or 16
// (d = 64) pieces of 16 bytes; a warp takes kLoads loads of them, all issued before anything is
// looked up, while a lane a row finds where the row goes and writes its weight.
#include <algorithm>

#include "kvp_cache.cuh"
#include "kvp_ptx.cuh"

namespace kvp {
namespace {

constexpr int kThreads = 128;
constexpr int kLoads = 8;     // 16-byte loads a lane has in flight

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

// Row r of the flattened new rows (a lane a row; all lanes of the warp take part, r < 0: none): its head
// (-1: past the sequence's counts, or none) and its place among that head's new rows.
__device__ __forceinline__ void place_of(const AppendArgs& a, long long r, int& head, int& i) {
    if (a.counts == nullptr) {
        head = r < 0 ? -1 : (int)(r / a.n);
        i = (int)(r - (long long)head * a.n);
        return;
    }
    const long long per = (long long)a.hkv * a.n;
    const int lane = threadIdx.x & 31, seq = r < 0 ? -1 : (int)(r / per);
    const long long left = r - seq * per;
    head = -1;
    i = 0;
    // the warp's rows lie in a few sequences: for each, prefix sums of its heads' counts, 32 at a time
    for (unsigned todo = __ballot_sync(0xffffffffu, seq >= 0); todo;) {
        const int s = __shfl_sync(0xffffffffu, seq, __ffs(todo) - 1);
        long long base = 0;                           // rows of the heads before
        for (int h0 = 0; h0 < a.hkv; h0 += 32) {
            long long end = h0 + lane < a.hkv ? max(0, a.counts[(size_t)s * a.hkv + h0 + lane]) : 0;
            const long long cnt = end;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, end, o);
                if (lane >= o) end += y;
            }
            end += base;
            const int heads = min(32, a.hkv - h0);
            for (int x = 0; x < heads; ++x) {
                const long long e = __shfl_sync(0xffffffffu, end, x), b = e - __shfl_sync(0xffffffffu, cnt, x);
                if (seq == s && left >= b && left < e) {
                    head = s * a.hkv + h0 + x;
                    i = (int)(left - b);
                }
            }
            base = __shfl_sync(0xffffffffu, end, 31);
        }
        todo &= ~__ballot_sync(0xffffffffu, seq == s);
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

// Rows that a warp's kLoads loads cover.
template <int D>
__host__ __device__ constexpr int batch_rows() {
    return kLoads * (32 / (D / 4));
}

template <int D>
__global__ void __launch_bounds__(kThreads) append_rows(const AppendArgs a) {
    constexpr int kPieces = D / 8, kLanes = 2 * kPieces, kAtOnce = 32 / kLanes, kBatch = batch_rows<D>();
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const int lane = threadIdx.x & 31, piece = lane % kPieces, sub = lane / kLanes;
    const bool is_v = (lane / kPieces) & 1;
    const uint4* from = (is_v ? a.v_new : a.k_new) + piece;
    uint4* to = (is_v ? a.v_pages : a.k_pages) + piece;
    const long long warps = (long long)gridDim.x * (kThreads / 32);
    const long long w0 = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    for (long long base = w0 * kBatch; base < a.rows; base += warps * kBatch) {
        const int here = (int)min((long long)kBatch, a.rows - base);
        uint4 x[kLoads];
#pragma unroll
        for (int l = 0; l < kLoads; ++l)
            if (l * kAtOnce + sub < here) x[l] = from[(base + l * kAtOnce + sub) * kPieces];
        int head, i;
        place_of(a, lane < here ? base + lane : -1, head, i);
        long long dst = -1;
        if (head >= 0 && KVP_CHECK(head < a.c.heads && i >= 0, 501, head, i)) {
            const long long j = (long long)a.c.len(head) + i;
            if (j < a.c.cap()) dst = a.c.row(head, (int)j);
            if (dst >= 0 && a.acc) a.acc[dst] = a.weight ? a.weight[base + lane] : 0.f;
        }
#pragma unroll
        for (int l = 0; l < kLoads; ++l) {
            const long long d = __shfl_sync(0xffffffffu, dst, (l * kAtOnce + sub) & 31);
            if (l * kAtOnce + sub < here && d >= 0) to[d * kPieces] = x[l];
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
    const int per_cta = (s.head_dim == 128 ? batch_rows<128>() : batch_rows<64>()) * (kThreads / 32);
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
