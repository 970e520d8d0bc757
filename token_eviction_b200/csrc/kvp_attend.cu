// Attention of one new token over a paged cache, split over the cache's rows and joined:
//   t_gj = q_g . k_j / sqrt(d), out_g = sum_j 2^(t_gj log2 e - lse2_g) v_j, acc_j += sum_g p_gj.
//
// Bound: every cached row is read once, 4 d bytes of key and value for 4 G d flops: G flops a
// byte, far below what the card can multiply while it reads (G <= 16 needs under 110 TFLOP/s at
// the measured 6.56 TB/s). So the matrix products are warp-level mma.sync m16n8k16, whose
// operands go from the ring in shared memory to registers with no barrier between warps, and
// the kernel is built around bytes in flight.
//
// attend_split: the units (a head's rows against up to 8, or 16, of its query heads) laid end to
// end are one run of tiles of 64 rows, cut evenly over two CTAs per SM (but long runs leave their last
// eighth to short ones, and very short runs are made fewer: Cutting).
// Each of a CTA's four warps streams its 16 rows of every tile through a ring of its own
// (cp.async, 16-byte pieces, swizzled for ldmatrix), keeps the running maximum and sum of a
// softmax, and never waits for another warp until the unit ends. There the four warps' parts
// are joined in shared memory; a unit that lies within one CTA is finished, others leave a part
// (unnormalised output, maximum, sum) in the workspace.
// attend_join: joins the parts of the units that were cut (a CTA has two at most), in the order of
// the rows. attend_join_few: the same where units are few and have very many parts.
// attend_short (few heads with short caches, as an eviction leaves them): a cluster of 8 CTAs a head,
// one launch. A warp has up to four groups of 16 rows, of which its ring holds four, three (d = 128) or
// two (d = 128, G > 8) at a time; the CTAs' parts are joined through distributed shared memory and the
// logits never leave the SM.
// The weights that acc gains need the final sum, so the logits go through the workspace (4 G bytes
// a row against 4 d of the row itself) and are read back, mostly from L2, by the CTA that finished
// the unit, or by attend_join for units that were cut (attend_weigh, where units are few or a head's several).
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "kvp_cache.cuh"
#include "kvp_ptx.cuh"

namespace cg = cooperative_groups;

namespace kvp {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kGroup = 16;                        // rows a warp takes at a time
constexpr int kTile = kWarps * kGroup;            // rows a CTA takes at a time
constexpr int kCtasPerSm = 2;
constexpr int kResident = kPlanGrid * kCtasPerSm;
constexpr int kMaxGrid = 2 * kResident;           // the workspace holds parts for as many CTAs
constexpr int kLongRun = 32;                      // tiles of a run from which runs of unequal speed are balanced
constexpr int kShortRun = 6;                      // and tiles of the short runs that do it, at least
constexpr int kMinRun = 4, kManyParts = 128;      // tiles of a run, at least, where a unit would have more parts
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;
constexpr int kJoinPieces = 2;                    // blocks of attend_join that weigh one share, at most
constexpr int kFewUnits = 4;                      // units up to which a cluster joins each query head,
constexpr int kFewSteps = 6;                      // and steps of adding up their sums from which it does so with acc too
constexpr int kCluster = 8;                       // its CTAs, and those of attend_short for a head,
constexpr int kShortWarps = 8, kShortThreads = kShortWarps * 32;
constexpr int kShortRows = 512;                   // rows each may have,
constexpr int kShortCtas = 120;                   // and CTAs in all: 15 clusters of 8 SMs find room on 148
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLowest = -3.4028234663852886e38f;  // of a maximum over nothing: finite, so that
                                                    // differences of maxima are never inf - inf

// Where a CTA's run begins: its unit, the tile within it.
struct Start {
    int unit, tile;
};

// A CTA's share of a unit that other CTAs share too: tiles [tile, tile + count) of the unit. Its
// n parts are those of CTAs c0 .. c0 + n - 1: c0's last unit if `later`, the first of the others.
struct Cut {
    int unit, tile, count, head;       // unit = -1: no such share
    int c0, n, later, len;

    __device__ __forceinline__ size_t slot(int i) const { return 2 * (size_t)(c0 + i) + (i == 0 && later ? 1 : 0); }
};

struct AttendArgs {
    CacheView c;
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    uint16_t* out;
    float* lse;          // NULL: not wanted
    float* acc;          // NULL: not wanted
    int resident;        // CTAs of attend_split that run at once; the grid may have more
    int many;            // CTAs from which their runs are not cut below kMinRun tiles
    int G, ng, gq;       // query heads per head; units per head; query heads per unit (the last: fewer)
    float scale2;        // log2 e / sqrt(d)
    // workspace
    Cut* cuts;           // [2 grid]: what each CTA's first and last unit had of it, where they were cut
    Cut* firsts;         // [units]: a cut unit's first share (unit = -1: not cut); NULL where units are not few
    float2* stats;       // [2 grid][gq]: a part's maximum and sum, log2 domain
    float* parts;        // [2 grid][gq][d]: a part's unnormalised output
    float* lse2;         // [heads * G], where attend_weigh adds the weights (acc, and more than one unit a head or firsts)
    float* logits;       // [heads * G][cap]: q . k; NULL without acc
};

__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) / kTile; }

// T tiles cut into contiguous runs, a CTA each. The first `first` CTAs are resident together; SMs
// that lie nearer to the memory finish up to an eighth earlier than the rest, so of long runs the
// last eighth of the tiles is left to `more` CTAs with short ones, which the hardware starts where
// a CTA has ended. (24 caches of 0 to 16383 rows, GQA-7: 86 us, 87 without; 64 of 8192: 361, 377.)
// Where attend_join would have to join more than `many` parts of very few tiles, which takes longer than
// their rows, fewer CTAs take part. (2 heads of 30000 rows, G 4, acc: 14.2 us, 15.2 without.)
struct Cutting {
    long long T, B;          // tiles; those of the first CTAs
    int first, more;

    __device__ __forceinline__ Cutting(long long tiles, int resident, int grid, int many) {
        T = B = tiles;
        first = (int)min(T, (long long)resident);
        if (first > many && T < (long long)kMinRun * first) first = (int)((T + kMinRun - 1) / kMinRun);
        more = 0;
        if (grid > resident && T >= (long long)kLongRun * resident) {
            more = (int)min((long long)(grid - resident), T / 8 / kShortRun);
            B = T - T / 8;
        }
    }
    __device__ __forceinline__ int ctas() const { return first + more; }
    __device__ __forceinline__ long long begin(int c) const {
        if (c >= ctas()) return T;
        return c <= first ? scaled(c, B, first) : B + scaled(c - first, T - B, more);
    }
    __device__ __forceinline__ int owner(long long t) const {   // the CTA whose run holds tile t
        if (t < B) return (int)scaled_up(t + 1, first, B) - 1;
        return first + (int)scaled_up(t - B + 1, more, T - B) - 1;
    }

private:
    // floor and ceil of x y / z; in 32 bits where no product passes them
    __device__ __forceinline__ long long scaled(long long x, long long y, long long z) const {
        return T < (1 << 22) ? (long long)((uint32_t)x * (uint32_t)y / (uint32_t)z) : x * y / z;
    }
    __device__ __forceinline__ long long scaled_up(long long x, long long y, long long z) const {
        return T < (1 << 22) ? (long long)(((uint32_t)x * (uint32_t)y + (uint32_t)z - 1) / (uint32_t)z) : (x * y + z - 1) / z;
    }
    static_assert((1ll << 22) * kResident + (1 << 22) < (1ll << 32), "a run's bounds in 32 bits");
};

// ---- types
template <typename T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
    static constexpr float kBias = 0.f;      // added to a weight's exponent before rounding
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        uint32_t r;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    static __device__ __forceinline__ float2 unpack(uint32_t p) {
        return make_float2(__uint_as_float(p << 16), __uint_as_float(p & 0xFFFF0000u));
    }
    static __device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    }
};
template <>
struct Pair<__half> {
    // Weights lie in [0, 1] and fp16 has no normal number below 2^-14: they are kept 2^14
    // larger (so is their sum), which puts full precision down to 2^-28 of the largest.
    static constexpr float kBias = 14.f;
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        uint32_t r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    static __device__ __forceinline__ float2 unpack(uint32_t p) {
        return __half22float2(*reinterpret_cast<__half2*>(&p));
    }
    static __device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    }
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr)
                 : "memory");
}
// 16 bytes global -> shared.
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy)
                 : "memory");
}
// The same, or 16 zero bytes (src is not read).
__device__ __forceinline__ void cp16_or_zero(uint32_t dst, const void* src, bool read) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(read ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// acc += the weights of rows [j0, j1) of `head` (j0 a multiple of 4), from their logits: one thread
// four rows at a time. lse2[g] = +inf where query head g has no weights to give.
template <int kStride>
__device__ __forceinline__ void add_weights(const AttendArgs& a, int head, int j0, int j1, int tid, const float* lse2) {
    const int cap = a.c.cap();
    for (int j = j0 + tid * 4; j < j1; j += kStride * 4) {
        if (!KVP_CHECK(head >= 0 && head < a.c.heads && j >= 0 && j + 3 < cap, 601, head, j)) continue;
        const long long row = a.c.row(head, j);              // four rows lie in one page
        if (row < 0) continue;
        const float* lp = a.logits + (size_t)head * a.G * cap + j;
        float* ap = a.acc + row;
        float4 x = *(const float4*)ap;                       // (the page's next rows past the last one)
        float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll 4
        for (int g = 0; g < a.G; ++g) {
            const float4 t = *(const float4*)(lp + (size_t)g * cap);
            const float l = lse2[g];
            s0 += ptx::ex2(fmaf(t.x, a.scale2, -l));
            s1 += ptx::ex2(fmaf(t.y, a.scale2, -l));
            s2 += ptx::ex2(fmaf(t.z, a.scale2, -l));
            s3 += ptx::ex2(fmaf(t.w, a.scale2, -l));
        }
        x.x += s0;
        x.y += s1;
        x.z += s2;
        x.w += s3;
        if (j + 4 <= j1) {
            *(float4*)ap = x;
        } else {
            ap[0] = x.x;
            if (j + 1 < j1) ap[1] = x.y;
            if (j + 2 < j1) ap[2] = x.z;
        }
    }
}

// Where tile `want` of the run lies: every thread of the CTA sums a stretch of heads' tiles, and
// the one whose stretch holds `want` walks it. Sets *at (shared) and returns the total.
__device__ __forceinline__ Cutting find_start(const CacheView& c, int ng, int resident, int many, long long* warp_sums,
                                              Start* at) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (c.heads + kThreads - 1) / kThreads;
    const int h0 = min(c.heads, tid * per), h1 = min(c.heads, h0 + per);
    long long sum = 0;
    for (int h = h0; h < h1; ++h) sum += (long long)tiles_of(c.len(h)) * ng;
    long long inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    long long before = 0, T = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += warp_sums[w];
        T += warp_sums[w];
    }
    const Cutting cutting(T, resident, gridDim.x, many);
    long long from = before + inc - sum;
    const long long want = (int)blockIdx.x < cutting.ctas() ? cutting.begin(blockIdx.x) : -1;
    if (want >= from && want < from + sum) {
        for (int h = h0; h < h1; ++h) {
            const int nt = tiles_of(c.len(h));
            const long long n = (long long)nt * ng;
            if (want < from + n) {
                const int i = (int)(want - from);
                at->unit = h * ng + i / nt;
                at->tile = i % nt;
                break;
            }
            from += n;
        }
    }
    __syncthreads();
    return cutting;
}

// A warp's walk over the units that have tiles, from a given one on. A register of each lane
// holds one of 32 heads' lengths, so that a stretch of empty heads costs one load for 32.
struct Walk {
    int head, sub, tile, nt, len;   // unit = head * ng + sub
    int base, lane_len;

    __device__ __forceinline__ void load(const CacheView& c) {
        const int h = base + (threadIdx.x & 31);
        lane_len = h < c.heads ? c.len(h) : 0;
    }
    // `loaded`: lane_len holds the first 32 heads' lengths
    __device__ __forceinline__ void begin(const CacheView& c, int ng, const Start& s, bool loaded) {
        head = s.unit / ng;
        sub = s.unit - head * ng;
        tile = s.tile;
        base = head & ~31;
        if (!loaded) load(c);
        len = __shfl_sync(0xffffffffu, lane_len, head & 31);
        nt = tiles_of(len);
    }
    // The next tile; the caller knows that there is one.
    __device__ __forceinline__ void next(const CacheView& c, int ng) {
        if (++tile < nt) return;
        tile = 0;
        if (++sub < ng) return;
        sub = 0;
        ++head;
        while (head < c.heads) {
            if ((head & ~31) != base) {
                base = head & ~31;
                load(c);
            }
            const unsigned live = __ballot_sync(0xffffffffu, lane_len > 0) >> (head & 31);
            if (live) {
                head += __ffs(live) - 1;
                break;
            }
            head = base + 32;
        }
        len = __shfl_sync(0xffffffffu, lane_len, head & 31);
        nt = tiles_of(len);
    }
};

// Of up to 32 heads every warp finds its CTA's run by itself, a length a lane, with no barrier and no
// second read of the lengths.
__device__ __forceinline__ Cutting find_start_32(const CacheView& c, int ng, int resident, int many, Start* at, int* lane_len) {
    const int lane = threadIdx.x & 31;
    *lane_len = lane < c.heads ? c.len(lane) : 0;
    const int nt = tiles_of(*lane_len), n = nt * ng;          // (at most 2^19 tiles each)
    int inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    const Cutting cutting(__shfl_sync(0xffffffffu, inc, 31), resident, gridDim.x, many);
    const int want = (int)cutting.begin(min((int)blockIdx.x, cutting.ctas()));
    const unsigned past = __ballot_sync(0xffffffffu, inc > want);
    const int head = past ? __ffs(past) - 1 : 0;
    const int i = want - __shfl_sync(0xffffffffu, inc - n, head), head_tiles = max(1, __shfl_sync(0xffffffffu, nt, head));
    at->unit = head * ng + i / head_tiles;
    at->tile = i % head_tiles;
    return cutting;
}

// What a warp notes about a group when it issues its loads and reads when it consumes it.
struct __align__(16) Meta {
    int head, sub;       // the unit
    int row0;            // the group's first row within the head
    int valid_flags;     // rows of it that are there (0: nothing was loaded), and flags
};
// kFirst, kLast: of the unit, within this CTA's run; kWhole: the run has all of the unit
constexpr int kFirst = 32, kLast = 64, kWhole = 128, kValid = 31;

// How 16 rows of keys or values lie in shared memory, and how a warp fetches and reads them. A row's
// 16-byte chunks are stored xor (row & 7), so that eight rows' same chunk lies in eight bank groups.
template <int D>
struct Group16 {
    static constexpr int kRowBytes = D * 2;
    static constexpr int kChunks = D / 8;                       // 16-byte chunks of a row
    static constexpr int kHalf = kGroup * kRowBytes;            // a group's keys (then its values)
    static constexpr int kStage = 2 * kHalf;
    static constexpr int kRowsAt = 32 / kChunks;                // rows that one load of the warp covers

    const uint8_t *k, *v, *k_lane, *v_lane;
    uint32_t dst_lane;       // offset of this lane's first chunk in a stage
    uint64_t policy;

    __device__ __forceinline__ Group16(const AttendArgs& a) {
        const int lane = threadIdx.x & 31, chunk = lane % kChunks, lrow = lane / kChunks;   // lrow < kRowsAt <= 4
        k = (const uint8_t*)a.k;
        v = (const uint8_t*)a.v;
        k_lane = k + lrow * kRowBytes + chunk * 16;
        v_lane = v + lrow * kRowBytes + chunk * 16;
        dst_lane = lrow * kRowBytes + ((chunk ^ lrow) << 4);
        policy = ptx::policy_evict_first();   // rows are read once; what L2 holds better is the logits
    }
    // Rows [row, row + valid) of the pool into the stage at `stage`, zeros behind them.
    __device__ __forceinline__ void fetch(uint32_t stage, size_t row, int valid) const {
        const size_t off = row * kRowBytes;
        const uint32_t dst = stage + dst_lane;
        if (valid == kGroup) {
            const uint8_t *ks = k_lane + off, *vs = v_lane + off;
#pragma unroll
            for (int i = 0; i < kGroup / kRowsAt; ++i) {
                const int r = i * kRowsAt;                 // lrow | r: they share no bits
                cp16((dst ^ ((r & 7) << 4)) + r * kRowBytes, ks + r * kRowBytes, policy);
            }
#pragma unroll
            for (int i = 0; i < kGroup / kRowsAt; ++i) {
                const int r = i * kRowsAt;
                cp16((dst ^ ((r & 7) << 4)) + r * kRowBytes + kHalf, vs + r * kRowBytes, policy);
            }
        } else if (valid > 0) {
            const int lrow = (threadIdx.x & 31) / kChunks;
#pragma unroll 1
            for (int r = 0; r < kGroup; r += kRowsAt) {
                const bool in = lrow + r < valid;
                const size_t from = in ? off + (size_t)r * kRowBytes : 0;
                const uint32_t to = (dst ^ ((r & 7) << 4)) + r * kRowBytes;
                cp16_or_zero(to, (in ? k_lane : k) + from, in);
                cp16_or_zero(to + kHalf, (in ? v_lane : v) + from, in);
            }
        }
    }
};

// A warp's running softmax over groups of 16 rows, for up to 16 query heads (kWide), one row each of
// the MMA's 16; or for up to 8, whose weights fill rows 0-7 and the remainders left by rounding
// them to T rows 8-15: the product with V then carries about twice T's precision, for free, since
// the MMA has 16 rows anyway. Of 9 to 16 query heads the weights alone fill the rows and the
// remainders would take a second product; they are left out, which adds half a step of T to each
// weight (4000 random rows: the result's error is 2.0e-3 of its norm in bf16, 1.7e-3 with remainders;
// 2.5e-4 in fp16, 2.1e-4). Maximum, sum and logits are fp32 in both.
template <typename T, int D, bool kWide>
struct Running {
    static constexpr int kNt = D / 8;         // 8-column tiles of the output
    static constexpr int kR = kWide ? 2 : 1;  // rows of the MMA that are query heads: gid, gid + 8
    static constexpr int kQ = 8 * kR;
    float o[kNt][4];
    float m_run[2], l_run[2];                 // running maximum (log2 units) and sum
    uint32_t qf[D / 16][2 * kR];

    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int i = 0; i < kNt; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        m_run[0] = m_run[1] = kLowest;
        l_run[0] = l_run[1] = 0.f;
    }
    // q: the unit's first query head, of nq
    __device__ __forceinline__ void read_q(const uint16_t* q, int nq) {
        const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
        const uint32_t* qp = (const uint32_t*)q;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            const int at32 = ks * 8 + tig;              // pairs of columns
            qf[ks][0] = gid < nq ? qp[gid * (D / 2) + at32] : 0u;
            qf[ks][1] = gid < nq ? qp[gid * (D / 2) + at32 + 4] : 0u;
            if (kWide) {
                qf[ks][kR] = gid + 8 < nq ? qp[(gid + 8) * (D / 2) + at32] : 0u;
                qf[ks][2 * kR - 1] = gid + 8 < nq ? qp[(gid + 8) * (D / 2) + at32 + 4] : 0u;
            }
        }
    }
    // The group in the stage at `stage`, `valid` > 0 rows of it. put(r, row, x, y): products q . k of
    // query head gid + 8 r with rows `row` and row + 1.
    template <typename Put>
    __device__ __forceinline__ void take(uint32_t stage, int valid, float scale2, Put put) {
        constexpr int kRowBytes = Group16<D>::kRowBytes;
        const int lane = threadIdx.x & 31, tig = lane & 3;
        // a lane's address for ldmatrix: chunk c of its row lies 16 c bytes on, by xor
        const int k_row = (lane & 7) + ((lane >> 4) & 1) * 8, v_row = (lane & 7) + ((lane >> 3) & 1) * 8;
        const uint32_t sk = stage + k_row * kRowBytes + ((((lane >> 3) & 1) ^ (k_row & 7)) << 4);
        const uint32_t sv = stage + Group16<D>::kHalf + v_row * kRowBytes + ((((lane >> 4) & 1) ^ (v_row & 7)) << 4);
        // logits of 16 rows: two tiles of 8 rows, two chains each
        float c[2][2][4] = {};
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            uint32_t b0, b1, b2, b3;
            ldsm4(sk ^ (ks << 5), b0, b1, b2, b3);
            const uint32_t a1 = kWide ? qf[ks][kR] : 0u, a3 = kWide ? qf[ks][2 * kR - 1] : 0u;
            Pair<T>::mma(c[ks & 1][0], qf[ks][0], a1, qf[ks][1], a3, b0, b1);
            Pair<T>::mma(c[ks & 1][1], qf[ks][0], a1, qf[ks][1], a3, b2, b3);
        }
        float t[2][2 * kR];                   // [8-row tile][query head gid: 2 cached rows, gid + 8: 2]
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 2 * kR; ++i) t[n][i] = c[0][n][i] + c[1][n][i];
        if (valid < kGroup) {
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 0; i < 2 * kR; ++i)
                    if (n * 8 + 2 * tig + (i & 1) >= valid) t[n][i] = -INFINITY;
        }
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            put(r, 2 * tig, t[0][2 * r], t[0][2 * r + 1]);
            put(r, 2 * tig + 8, t[1][2 * r], t[1][2 * r + 1]);
        }
        uint32_t pa[4];                       // the weights as the A operand of P V
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            float mx = fmaxf(fmaxf(t[0][2 * r], t[0][2 * r + 1]), fmaxf(t[1][2 * r], t[1][2 * r + 1]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * scale2;
            if (__any_sync(0xffffffffu, mx > m_run[r])) {
                const float m_new = fmaxf(m_run[r], mx), f = ptx::ex2(m_run[r] - m_new);
                l_run[r] *= f;
#pragma unroll
                for (int i = 0; i < kNt; ++i) {
                    o[i][2 * r] *= f;
                    o[i][2 * r + 1] *= f;
                    if (!kWide) {             // rows 8-15 are the same query heads' remainders
                        o[i][2] *= f;
                        o[i][3] *= f;
                    }
                }
                m_run[r] = m_new;
            }
            const float off = Pair<T>::kBias - m_run[r];
            const float p0 = ptx::ex2(fmaf(t[0][2 * r], scale2, off)), p1 = ptx::ex2(fmaf(t[0][2 * r + 1], scale2, off));
            const float p2 = ptx::ex2(fmaf(t[1][2 * r], scale2, off)), p3 = ptx::ex2(fmaf(t[1][2 * r + 1], scale2, off));
            l_run[r] += (p0 + p1) + (p2 + p3);
            pa[r] = Pair<T>::pack(p0, p1);
            pa[r + 2] = Pair<T>::pack(p2, p3);
            if (!kWide) {
                const float2 h0 = Pair<T>::unpack(pa[0]), h1 = Pair<T>::unpack(pa[2]);
                pa[1] = Pair<T>::pack(p0 - h0.x, p1 - h0.y);
                pa[3] = Pair<T>::pack(p2 - h1.x, p3 - h1.y);
            }
        }
#pragma unroll
        for (int i = 0; i < kNt; i += 2) {
            uint32_t b0, b1, b2, b3;
            ldsm4t(sv ^ (i << 4), b0, b1, b2, b3);
            Pair<T>::mma(o[i], pa[0], pa[1], pa[2], pa[3], b0, b1);
            Pair<T>::mma(o[i + 1], pa[0], pa[1], pa[2], pa[3], b2, b3);
        }
    }
    // This warp's part: unnormalised output [kQ][D] (columns xor part_swizzle(row)), maximum and sum [kQ].
    __device__ __forceinline__ void put_part(float* part, float2* stat) const {
        const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            float l = l_run[r];
            l += __shfl_xor_sync(0xffffffffu, l, 1);
            l += __shfl_xor_sync(0xffffffffu, l, 2);
            const int row = gid + 8 * r;
            if (tig == 0) stat[row] = make_float2(m_run[r], l);
#pragma unroll
            for (int i = 0; i < kNt; ++i) {
                const float x = kWide ? o[i][2 * r] : o[i][0] + o[i][2];
                const float y = kWide ? o[i][2 * r + 1] : o[i][1] + o[i][3];
                *(float2*)(part + row * D + ((i * 8 + 2 * tig) ^ part_swizzle(row))) = make_float2(x, y);
            }
        }
    }
    static __device__ __forceinline__ int part_swizzle(int row) { return (row & 3) << 3; }
};

// A warp adds up kParts parts of one query head: columns [lane D / 32, ...) of it in val; the maximum
// and the sum returned. part(x): its output; stat(x): its maximum and sum.
template <int D, int kParts, typename PartOf, typename StatOf>
__device__ __forceinline__ float2 add_parts(float (&val)[D / 32], PartOf part, StatOf stat) {
    float2 st[kParts];
    float top = kLowest, l = 0.f;
#pragma unroll
    for (int x = 0; x < kParts; ++x) {
        st[x] = stat(x);
        top = fmaxf(top, st[x].x);
    }
#pragma unroll
    for (int c = 0; c < D / 32; ++c) val[c] = 0.f;
#pragma unroll
    for (int x = 0; x < kParts; ++x) {
        const float f = ptx::ex2(st[x].x - top);
        const float* from = part(x);
        l += f * st[x].y;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) val[c] += f * from[c];
    }
    return make_float2(top, l);
}

// A finished query head: its output (a lane D / 32 columns) and, by lane 0, its log-sum-exp. Returns
// log2 of the sum, +inf where there is none.
template <typename T, int D>
__device__ __forceinline__ float put_output(const AttendArgs& a, size_t query, const float (&val)[D / 32], float2 st) {
    const int lane = threadIdx.x & 31;
    const float inv = st.y == 0.f ? 0.f : 1.f / st.y;               // a NaN sum stays one
#pragma unroll
    for (int c = 0; c < D / 32; c += 2)
        ((uint32_t*)a.out)[(query * D + lane * (D / 32) + c) / 2] = Pair<T>::pack(val[c] * inv, val[c + 1] * inv);
    // the sum and the output are 2^kBias larger
    const float lse2 = st.x - Pair<T>::kBias + log2f(st.y);         // -inf where the sum is 0
    if (lane == 0 && a.lse) a.lse[query] = lse2 * kLn2;
    if (lane == 0 && a.lse2) a.lse2[query] = lse2;
    return st.y == 0.f ? INFINITY : lse2;
}

constexpr uint32_t kRingAlign = 256;      // rows of 256 bytes: a chunk's bits of an address are free for xor

template <typename T, int D, bool kWide, int kStages>
struct Split {
    static constexpr int kStage = Group16<D>::kStage;
    static constexpr size_t kSmem = (size_t)kWarps * kStages * kStage + kRingAlign;
    static_assert(Running<T, D, kWide>::kQ * D * 4 <= kStage, "a warp's part is joined in the stage it has consumed");
};

template <typename T, int D, bool kWide, int kStages>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) attend_split(const AttendArgs a) {
    constexpr int kStage = Group16<D>::kStage, kQ = Running<T, D, kWide>::kQ;
    extern __shared__ __align__(16) uint8_t raw[];
    uint8_t* const ring = raw + (-ptx::smem_u32(raw) & (kRingAlign - 1));
    __shared__ long long warp_sums[kWarps];
    __shared__ Start sh_at;
    __shared__ Meta meta[kWarps][kStages];
    __shared__ float2 sh_stat[kWarps][kQ];
    __shared__ float sh_lse2[kQ];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gid = lane >> 2;
    const int grid = gridDim.x, cta = blockIdx.x;

    ptx::grid_dependency_wait();
    Start at;
    Walk w;
    const bool few = a.c.heads <= 32;
    const Cutting cutting = few ? find_start_32(a.c, a.ng, a.resident, a.many, &at, &w.lane_len)
                                : find_start(a.c, a.ng, a.resident, a.many, warp_sums, &sh_at);
    if (!few) at = sh_at;
    ptx::launch_dependents();
    // heads without rows
    for (int h = cta; h < a.c.heads; h += grid) {
        if (a.c.len(h) > 0) continue;
        for (int e = tid; e < a.G * D; e += kThreads) ((T*)a.out)[(size_t)h * a.G * D + e] = T(0.f);
        if (a.lse && tid < a.G) a.lse[(size_t)h * a.G + tid] = -INFINITY;
        if (a.firsts && tid < a.ng) a.firsts[h * a.ng + tid].unit = -1;
    }
    if (tid < 2) a.cuts[2 * cta + tid].unit = -1;
    if (cta >= cutting.ctas()) return;
    const long long r0 = cutting.begin(cta);
    const int steps = (int)(cutting.begin(cta + 1) - r0);

    // ---- the issuing side: the walk is one tile ahead of its loads, so that its page is at hand
    w.begin(a.c, a.ng, at, few);
    const uint32_t my_ring = ptx::smem_u32(ring) + warp * kStages * kStage;
    // pages of the walk's unit, a lane each: of this warp's groups in tiles [page_base, page_base + 32)
    int page_base = 0, pages = -1;
    auto load_pages = [&]() {
        page_base = w.tile;
        const int row0 = (page_base + lane) * kTile + warp * kGroup;
        pages = -1;
        if (row0 < w.len && KVP_CHECK(w.head >= 0 && w.head < a.c.heads && row0 >= 0, 603, w.head, row0)) {
            const int p = a.c.table[(size_t)w.head * a.c.max_pages + (row0 >> a.c.page_shift)];
            if (p < a.c.num_pages) pages = p;
        }
    };
    load_pages();
    int issued = 0, fill = 0;                // groups issued; the stage the next one goes to
    bool fresh = true;                       // the walk's tile is the run's first of its unit
    bool begins = w.tile == 0;               // and the unit's first
    const Group16<D> group(a);
    const int page_mask = (1 << a.c.page_shift) - 1;
    auto issue = [&]() {
        if (issued < steps) {
            const int row0 = w.tile * kTile + warp * kGroup;
            const int page = __shfl_sync(0xffffffffu, pages, w.tile - page_base);
            const int valid = page < 0 ? 0 : min(kGroup, w.len - row0);   // (-1 too past the head's rows)
            const bool ends = w.tile == w.nt - 1;
            if (lane == 0) {
                Meta m;
                m.head = w.head;
                m.sub = w.sub;
                m.row0 = row0;
                m.valid_flags = valid | (fresh ? kFirst : 0) | (ends || issued == steps - 1 ? kLast : 0) |
                                (ends && begins ? kWhole : 0);
                meta[warp][fill] = m;
            }
            group.fetch(my_ring + fill * kStage, ((size_t)page << a.c.page_shift) + (row0 & page_mask), valid);
            fill = fill == kStages - 1 ? 0 : fill + 1;
            ++issued;
            if (issued < steps) {
                const int head = w.head, sub = w.sub;
                w.next(a.c, a.ng);
                fresh = w.head != head || w.sub != sub;
                if (fresh) begins = true;
                if (fresh || w.tile - page_base >= 32) load_pages();
            }
        }
        cp_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue();

    // ---- the consuming side
    Running<T, D, kWide> run;
    {                                         // the first unit's query heads, while its rows are on their way
        const int first_head = at.unit / a.ng, first_g = (at.unit - first_head * a.ng) * a.gq;
        run.read_q(a.q + ((size_t)first_head * a.G + first_g) * D, min(a.gq, a.G - first_g));
    }
    int segment = 0, seg_step = 0;            // units begun before this one; the step that began it
    int head = 0, g0 = 0, nq = 0;             // the unit's head, first query head and how many
    float* lp = nullptr;                      // logits of query head gid of the unit
    const size_t lp_row = (size_t)a.c.cap();

    int stage = 0;
    for (int step = 0; step < steps; ++step) {
        cp_wait<kStages - 2>();
        __syncwarp();
        const Meta m = meta[warp][stage];
        issue();                              // into the stage consumed one step ago
        const int valid = m.valid_flags & kValid;
        if (m.valid_flags & kFirst) {
            seg_step = step;
            head = m.head;
            g0 = m.sub * a.gq;
            nq = min(a.gq, a.G - g0);
            run.reset();
            if (step > 0) run.read_q(a.q + ((size_t)head * a.G + g0) * D, nq);
            lp = a.logits + ((size_t)head * a.G + g0 + gid) * lp_row;
        }
        if (valid > 0) {
            run.take(my_ring + stage * kStage, valid, a.scale2, [&](int r, int row, float x, float y) {
                if (a.logits && gid + 8 * r < nq && KVP_CHECK(m.row0 + row + 1 < a.c.cap(), 604, head, m.row0 + row))
                    *(float2*)(lp + r * 8 * lp_row + m.row0 + row) = make_float2(x, y);
            });
        }
        if (m.valid_flags & kLast) {
            // ---- join the four warps' parts, each in the stage it has just consumed
            __syncwarp();
            run.put_part((float*)(ring + (size_t)(warp * kStages + stage) * kStage), sh_stat[warp]);
            __syncthreads();
            const int slot = 2 * cta + (segment ? 1 : 0);
            const bool whole = m.valid_flags & kWhole;
            // a warp every kWarps-th query head, a lane kCols columns
            constexpr int kCols = D / 32;
            for (int row = warp; row < nq; row += kWarps) {
                float val[kCols];
                const int col = (lane * kCols) ^ run.part_swizzle(row);
                const float2 st = add_parts<D, kWarps>(
                    val, [&](int x) { return (const float*)(ring + (size_t)(x * kStages + stage) * kStage) + row * D + col; },
                    [&](int x) { return sh_stat[x][row]; });
                if (whole) {
                    const float lse2 = put_output<T, D>(a, (size_t)head * a.G + g0 + row, val, st);
                    if (lane == 0) sh_lse2[row] = lse2;
                } else if (KVP_CHECK(slot < 2 * kMaxGrid && segment < 2, 605, slot, step)) {
                    float* to = a.parts + ((size_t)slot * a.gq + row) * D + lane * kCols;
#pragma unroll
                    for (int c = 0; c < kCols; ++c) to[c] = val[c];
                    if (lane == 0) a.stats[(size_t)slot * a.gq + row] = make_float2(st.x - Pair<T>::kBias, st.y);
                }
            }
            __syncthreads();
            if (!whole && tid == 0) {
                Cut x;
                const int tile = m.row0 / kTile - (step - seg_step);   // the share's first
                x.unit = head * a.ng + m.sub;
                x.head = head;
                x.tile = tile;
                x.count = step - seg_step + 1;
                x.len = a.c.len(head);
                const long long first = r0 + seg_step - tile;          // the unit's first tile of all
                x.c0 = cutting.owner(first);
                x.n = cutting.owner(first + tiles_of(x.len) - 1) - x.c0 + 1;
                x.later = cutting.begin(x.c0) < first;
                if (KVP_CHECK(x.c0 >= 0 && x.n > 0 && x.c0 + x.n <= cutting.ctas() && tile >= 0, 606, x.c0, x.n)) a.cuts[slot] = x;
                if (a.firsts && tile == 0 && KVP_CHECK(x.unit < kFewUnits, 607, x.unit, tile)) a.firsts[x.unit] = x;
            }
            if (whole && a.firsts && tid == 0) a.firsts[head * a.ng + m.sub].unit = -1;
            if (whole && a.logits && !a.lse2)
                add_weights<kThreads>(a, head, 0, a.c.len(head), tid, sh_lse2);
            segment = 1;
        }
        stage = stage == kStages - 1 ? 0 : stage + 1;
    }
}

// (kStages: as many groups of a warp as fit in flight beside the logits; a warp has 4 at most.)
template <typename T, int D, bool kWide, int kStages>
struct Short {
    static constexpr int kQ = Running<T, D, kWide>::kQ;
    static constexpr int kStage = Group16<D>::kStage;
    static constexpr int kLogitRow = kShortRows + 8;            // floats of a query head's logits: eight
                                                                // query heads' pairs in distinct banks
    static constexpr size_t kRing = (size_t)kShortWarps * kStages * kStage;
    static constexpr size_t kSmem = kRing + (size_t)kQ * kLogitRow * sizeof(float) + kRingAlign;
    static_assert(kQ * D * 4 <= kStage, "a warp's part is joined in a stage");
    static_assert(kShortRows / kGroup <= 4 * kShortWarps, "a warp has at most 4 groups");
};

template <typename T, int D, bool kWide, int kStages>
__global__ void __launch_bounds__(kShortThreads, 1) attend_short(const AttendArgs a) {
    using S = Short<T, D, kWide, kStages>;
    constexpr int kStage = S::kStage, kQ = S::kQ, kCols = D / 32;
    extern __shared__ __align__(16) uint8_t raw[];
    uint8_t* const ring = raw + (-ptx::smem_u32(raw) & (kRingAlign - 1));
    float* const logits = (float*)(ring + S::kRing);            // [kQ][kLogitRow]
    __shared__ float2 warp_stat[kShortWarps][kQ], cta_stat[kQ];
    __shared__ __align__(16) float cta_part[kQ][D];
    __shared__ float sh_lse2[kQ];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gid = lane >> 2;
    const int head = blockIdx.x / kCluster, rank = blockIdx.x % kCluster, nq = a.G;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    Running<T, D, kWide> run;
    run.reset();
    run.read_q(a.q + (size_t)head * a.G * D, nq);
    const int len = a.c.len(head);
    if (len == 0) {                                             // the same in every CTA of the cluster
        if (rank == 0) {
            for (int e = tid; e < nq * D; e += kShortThreads) ((T*)a.out)[(size_t)head * nq * D + e] = T(0.f);
            if (a.lse && tid < nq) a.lse[(size_t)head * nq + tid] = -INFINITY;
        }
        return;
    }
    // groups [first, last) of the head's are this CTA's; this warp's i-th is first + warp + kShortWarps i
    const int groups = (len + kGroup - 1) / kGroup, per = (groups + kCluster - 1) / kCluster;
    const int first = min(groups, rank * per), last = min(groups, first + per);
    const int mine = max(0, (last - first - warp + kShortWarps - 1) / kShortWarps);
    const int page_mask = (1 << a.c.page_shift) - 1;
    int pages = -1;                                             // lane i: of this warp's i-th group
    if (lane < mine) {
        const int p = a.c.table[(size_t)head * a.c.max_pages + ((first + warp + kShortWarps * lane) * kGroup >> a.c.page_shift)];
        if (p < a.c.num_pages) pages = p;
    }
    const Group16<D> group(a);
    const uint32_t my_ring = ptx::smem_u32(ring) + warp * kStages * kStage;
    auto valid_of = [&](int i) {
        return __shfl_sync(0xffffffffu, pages, i) < 0 ? 0 : min(kGroup, len - (first + warp + kShortWarps * i) * kGroup);
    };
    auto fetch = [&](int i) {
        if (i < mine) {
            const int valid = valid_of(i), row0 = (first + warp + kShortWarps * i) * kGroup;
            const int page = __shfl_sync(0xffffffffu, pages, i);
            group.fetch(my_ring + i % kStages * kStage, ((size_t)max(page, 0) << a.c.page_shift) + (row0 & page_mask), valid);
        }
        cp_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages; ++i) fetch(i);
    // what this thread's four rows have drawn so far
    const int row_first = first * kGroup, row_last = min(len, last * kGroup), j = row_first + tid * 4;
    long long acc_row = -1;
    float4 drawn = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.acc && j < row_last) {
        acc_row = a.c.row(head, j);                             // four rows lie in one page
        if (acc_row >= 0) drawn = *(const float4*)(a.acc + acc_row);
    }
    for (int i = 0; i < mine; ++i) {
        cp_wait<kStages - 1>();
        __syncwarp();
        const int valid = valid_of(i);
        if (valid > 0) {
            float* to = logits + gid * S::kLogitRow + (warp + kShortWarps * i) * kGroup;
            run.take(my_ring + i % kStages * kStage, valid, a.scale2, [&](int r, int row, float x, float y) {
                if (a.acc && KVP_CHECK(gid + 8 * r < kQ && (warp + kShortWarps * i) * kGroup + row + 1 < S::kLogitRow, 608, head, i))
                    *(float2*)(to + r * 8 * S::kLogitRow + row) = make_float2(x, y);
            });
        }
        __syncwarp();                                           // the stage has been read
        fetch(i + kStages);
    }
    // ---- join the warps' parts, then the CTAs'
    run.put_part((float*)(ring + (size_t)warp * kStages * kStage), warp_stat[warp]);
    __syncthreads();
    for (int row = warp; row < nq; row += kShortWarps) {
        float val[kCols];
        const int col = (lane * kCols) ^ run.part_swizzle(row);
        const float2 st = add_parts<D, kShortWarps>(
            val, [&](int x) { return (const float*)(ring + (size_t)x * kStages * kStage) + row * D + col; },
            [&](int x) { return warp_stat[x][row]; });
#pragma unroll
        for (int c = 0; c < kCols; ++c) cta_part[row][lane * kCols + c] = val[c];
        if (lane == 0) cta_stat[row] = st;
    }
    ptx::cluster_arrive();
    ptx::cluster_wait();
    cg::cluster_group cluster = cg::this_cluster();
    for (int row = warp; row < nq; row += kShortWarps) {
        float val[kCols];
        auto stat = [&](int x) { return *cluster.map_shared_rank(&cta_stat[row], x); };
        if (row % kCluster == rank) {                           // its output is this CTA's to write
            const float2 st = add_parts<D, kCluster>(
                val, [&](int x) { return (const float*)cluster.map_shared_rank(&cta_part[row][lane * kCols], x); }, stat);
            const float lse2 = put_output<T, D>(a, (size_t)head * nq + row, val, st);
            if (lane == 0) sh_lse2[row] = lse2;
        } else if (a.acc) {
            float2 st = lane < kCluster ? stat(lane) : make_float2(kLowest, 0.f);
            float top = st.x;
#pragma unroll
            for (int o = kCluster / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            float l = st.y * ptx::ex2(st.x - top);
#pragma unroll
            for (int o = kCluster / 2; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            if (lane == 0) sh_lse2[row] = l == 0.f ? INFINITY : top - Pair<T>::kBias + log2f(l);
        }
    }
    ptx::cluster_arrive();                                      // this thread has read the others' shared memory
    __syncthreads();
    if (acc_row >= 0 && KVP_CHECK(tid * 4 + 3 < S::kLogitRow, 602, head, j)) {
        for (int g = 0; g < nq; ++g) {
            const float4 t = *(const float4*)(logits + g * S::kLogitRow + tid * 4);
            const float l = sh_lse2[g];
            drawn.x += ptx::ex2(fmaf(t.x, a.scale2, -l));
            drawn.y += ptx::ex2(fmaf(t.y, a.scale2, -l));
            drawn.z += ptx::ex2(fmaf(t.z, a.scale2, -l));
            drawn.w += ptx::ex2(fmaf(t.w, a.scale2, -l));
        }
        float* to = a.acc + acc_row;
        if (j + 4 <= row_last) {
            *(float4*)to = drawn;
        } else {
            to[0] = drawn.x;
            if (j + 1 < row_last) to[1] = drawn.y;
            if (j + 2 < row_last) to[2] = drawn.z;
        }
    }
    ptx::cluster_wait();                                        // its shared memory outlives its readers
}

// A warp's sum over the parts of a unit for query head `row`: log2 of it, and (mine) the maximum
// of part `lane`.
__device__ __forceinline__ float joined_lse2(const AttendArgs& a, const Cut& p, int row, float& mine) {
    const int lane = threadIdx.x & 31;
    float2 st = lane < p.n ? a.stats[p.slot(lane) * a.gq + row] : make_float2(kLowest, 0.f);
    mine = st.x;
    float top = st.x, l = st.y;
    for (int i = lane + 32; i < p.n; i += 32) {
        st = a.stats[p.slot(i) * a.gq + row];
        const float m = fmaxf(top, st.x);
        l = l * ptx::ex2(top - m) + st.y * ptx::ex2(st.x - m);
        top = m;
    }
    float m = top;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    l *= ptx::ex2(top - m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    return m + log2f(l);
}

// Two kinds of blocks, none with more than one short chain of reads. The first, `pieces` for every
// share of a cut unit (with acc; one for the short runs' shares), add its rows' weights. Then `rows`
// blocks for every CTA of attend_split, one a query head, join the outputs of the units whose first
// share it had.
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads, 6) attend_join(const AttendArgs a, int weighers, int pieces, int rows) {
    __shared__ float sh_lse2[16];
    ptx::grid_dependency_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int longs = 2 * a.resident * pieces;
    if ((int)blockIdx.x < weighers) {
        const bool is_long = (int)blockIdx.x < longs;
        if (!is_long) pieces = 1;
        const Cut p = a.cuts[is_long ? blockIdx.x / pieces : 2 * a.resident + blockIdx.x - longs];
        const int piece = is_long ? blockIdx.x % pieces : 0;
        constexpr int kRound = kJoinThreads * 4;
        const int last = min(p.len, (p.tile + p.count) * kTile), first = p.tile * kTile + piece * kRound;
        if (p.unit < 0 || first >= last) return;
        for (int row = warp; row < a.G; row += kJoinWarps) {
            float mine;
            const float x = joined_lse2(a, p, row, mine);
            if (lane == 0) sh_lse2[row] = x == -INFINITY ? INFINITY : x;
        }
        __syncthreads();
        for (int j = first; j < last; j += pieces * kRound)
            add_weights<kJoinThreads>(a, p.head, j, min(last, j + kRound), tid, sh_lse2);
        return;
    }
    // a warp every kJoinWarps-th part, kAhead of them read before their sum is known; a lane kCols columns
    constexpr int kCols = D / 32, kAhead = 32 / kJoinWarps;
    using Piece = typename std::conditional<kCols == 4, float4, float2>::type;
    __shared__ float sh_val[kJoinWarps][D];
    const int cta = (blockIdx.x - weighers) / rows, row = (blockIdx.x - weighers) % rows;
    for (int s = 0; s < 2; ++s) {
        const Cut p = a.cuts[2 * cta + s];
        if (p.unit < 0 || p.tile != 0) continue;
        const int g0 = (p.unit - p.head * a.ng) * a.gq;
        if (g0 + row >= a.G) continue;
        Piece y[kAhead];
        auto read = [&](int base) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int part = base + i * kJoinWarps + warp;
                if (part < p.n && KVP_CHECK(p.slot(part) < 2 * kMaxGrid, 609, p.c0, part))
                    y[i] = ((const Piece*)(a.parts + (p.slot(part) * a.gq + row) * D))[lane];
            }
        };
        read(0);
        float mine;
        const float lse2 = joined_lse2(a, p, row, mine);
        const size_t query = (size_t)p.head * a.G + g0 + row;
        float val[kCols] = {};
        for (int base = 0; base < p.n; base += 32) {
            if (base > 0) {
                read(base);
                mine = base + lane < p.n ? a.stats[p.slot(base + lane) * a.gq + row].x : kLowest;
            }
            const float f = lse2 == -INFINITY ? 0.f : ptx::ex2(mine - lse2);  // of part base + lane
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int part = i * kJoinWarps + warp;
                const float fi = __shfl_sync(0xffffffffu, f, part);
                if (base + part >= p.n) continue;
#pragma unroll
                for (int c = 0; c < kCols; ++c) val[c] += fi * ((const float*)&y[i])[c];
            }
        }
#pragma unroll
        for (int c = 0; c < kCols; ++c) sh_val[warp][lane * kCols + c] = val[c];
        __syncthreads();
        if (tid < D) {
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < kJoinWarps; ++w) sum += sh_val[w][tid];
            ((T*)a.out)[query * D + tid] = T(sum);
        }
        if (tid == 0) {
            if (a.lse) a.lse[query] = lse2 * kLn2;
            if (a.lse2) a.lse2[query] = lse2;
        }
        __syncthreads();
    }
}

// The outputs of few units, whose parts are many: a cluster a query head, an eighth of its parts a CTA. (attend_weigh
// then adds the weights.) One head of 131072 rows: G 8 18.2 us, 28.5 by attend_join; G 16 19.5, 37.4; with acc 22.3
// and 25.0, 28.1 and 39.8 by attend_join, whose every weighing block adds up the parts' sums again.
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads, 2) attend_join_few(const AttendArgs a, int rows) {
    constexpr int kAhead = 5, kCols = D / 32;
    using Piece = typename std::conditional<kCols == 4, float4, float2>::type;
    __shared__ __align__(16) float warp_part[kJoinWarps][D], cta_part[D];
    __shared__ float2 warp_stat[kJoinWarps], cta_stat;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, join = blockIdx.x / kCluster, rank = blockIdx.x % kCluster;
    const Cut p = a.firsts[join / rows];
    const int row = join % rows, g0 = p.unit < 0 ? 0 : (p.unit - p.head * a.ng) * a.gq;
    if (p.unit < 0 || g0 + row >= a.G) return;                  // the whole cluster
    float top = kLowest, l = 0.f, val[kCols] = {};
    const int last = p.n * (rank + 1) / kCluster;
    for (int base = p.n * rank / kCluster + warp; base < last; base += kAhead * kJoinWarps) {
        float2 st[kAhead];
        Piece y[kAhead];
        float m = top;
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
            const int part = base + x * kJoinWarps;
            st[x] = make_float2(kLowest, 0.f);
            y[x] = Piece{};
            if (part >= last || !KVP_CHECK(p.slot(part) < 2 * kMaxGrid, 610, p.c0, part)) continue;
            const size_t at = p.slot(part) * a.gq + row;
            st[x] = a.stats[at];
            y[x] = ((const Piece*)(a.parts + at * D))[lane];
        }
#pragma unroll
        for (int x = 0; x < kAhead; ++x) m = fmaxf(m, st[x].x);
        const float f = ptx::ex2(top - m);
        l *= f;
#pragma unroll
        for (int c = 0; c < kCols; ++c) val[c] *= f;
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
            const float fx = ptx::ex2(st[x].x - m);
            l += fx * st[x].y;
#pragma unroll
            for (int c = 0; c < kCols; ++c) val[c] += fx * ((const float*)&y[x])[c];
        }
        top = m;
    }
#pragma unroll
    for (int c = 0; c < kCols; ++c) warp_part[warp][lane * kCols + c] = val[c];
    if (lane == 0) warp_stat[warp] = make_float2(top, l);
    __syncthreads();
    if (warp == 0) {
        const float2 st = add_parts<D, kJoinWarps>(
            val, [&](int x) { return warp_part[x] + lane * kCols; }, [&](int x) { return warp_stat[x]; });
#pragma unroll
        for (int c = 0; c < kCols; ++c) cta_part[lane * kCols + c] = val[c];
        if (lane == 0) cta_stat = st;
    }
    ptx::cluster_arrive();
    ptx::cluster_wait();
    if (rank == 0 && warp == 0) {
        cg::cluster_group cluster = cg::this_cluster();
        float2 st = add_parts<D, kCluster>(
            val, [&](int x) { return (const float*)cluster.map_shared_rank(&cta_part[lane * kCols], x); },
            [&](int x) { return *cluster.map_shared_rank(&cta_stat, x); });
        st.x += Pair<T>::kBias;                                 // (taken off the parts' maxima)
        put_output<T, D>(a, (size_t)p.head * a.G + g0 + row, val, st);
    }
    __syncwarp();
    ptx::cluster_arrive();                                      // its shared memory outlives its readers
    ptx::cluster_wait();
}

// acc += the weights, where units are few or a head's query heads are several (G > 16): `per` blocks a head,
// once all of its sums are known.
__global__ void __launch_bounds__(kJoinThreads) attend_weigh(const AttendArgs a, int per) {
    __shared__ float sh_lse2[kMaxCacheGroup];
    ptx::grid_dependency_wait();
    const int head = blockIdx.x / per, len = a.c.len(head);
    if (len == 0) return;
    for (int g = threadIdx.x; g < a.G; g += kJoinThreads) {
        const float x = a.lse2[(size_t)head * a.G + g];
        sh_lse2[g] = x == -INFINITY ? INFINITY : x;
    }
    __syncthreads();
    const int cap = a.c.cap();
    for (int j = blockIdx.x % per * kJoinThreads + threadIdx.x; j < len; j += per * kJoinThreads) {
        const long long row = a.c.row(head, j);
        if (row < 0) continue;
        const float* lp = a.logits + (size_t)head * a.G * cap + j;
        const float drawn = a.acc[row];
        float sum = 0.f;
#pragma unroll 8
        for (int g = 0; g < a.G; ++g) sum += ptx::ex2(fmaf(lp[(size_t)g * cap], a.scale2, -sh_lse2[g]));
        a.acc[row] = drawn + sum;
    }
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

struct Layout {
    int ng, gq;
    size_t cuts, firsts, stats, parts, lse2, logits, bytes;
};

// bytes = 0: more tiles than the kernels count in 32 bits.
Layout layout_of(const kvp_cache_shape& s, bool accumulate) {
    Layout l = {};
    const int G = s.hq / s.hkv, d = s.head_dim;
    const long long heads = (long long)s.batch * s.hkv, cap = (long long)s.max_pages * s.page_size;
    l.gq = G <= 8 ? 8 : 16;
    l.ng = (G + l.gq - 1) / l.gq;
    if (heads * l.ng * ((cap + kTile - 1) / kTile) > INT32_MAX) return l;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += align256(bytes);
        return here;
    };
    l.cuts = take((size_t)2 * kMaxGrid * sizeof(Cut));
    l.firsts = take(kFewUnits * sizeof(Cut));
    l.stats = take((size_t)2 * kMaxGrid * l.gq * sizeof(float2));
    l.parts = take((size_t)2 * kMaxGrid * l.gq * d * sizeof(float));
    if (accumulate) {
        if (l.ng > 1 || heads <= kFewUnits) l.lse2 = take((size_t)heads * G * sizeof(float));
        l.logits = take((size_t)heads * G * cap * sizeof(float));
    }
    l.bytes = at;
    return l;
}

template <typename T, int D, bool kWide, int kStages>
cudaError_t launch_split(const AttendArgs& a, int grid, cudaStream_t st) {
    auto kernel = attend_split<T, D, kWide, kStages>;
    constexpr size_t smem = Split<T, D, kWide, kStages>::kSmem;
    const cudaError_t e = allow_dynamic_smem((const void*)kernel, smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, grid, kThreads, smem, st, a);
}

// launch_dependent, in clusters of kCluster CTAs.
template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kernel)(KArgs...), int grid, int block, size_t smem, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kCluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, KArgs(args)...);
}

template <typename T, int D, bool kWide, int kStages>
cudaError_t launch_short(const AttendArgs& a, cudaStream_t st) {
    auto kernel = attend_short<T, D, kWide, kStages>;
    constexpr size_t smem = Short<T, D, kWide, kStages>::kSmem;
    const cudaError_t e = allow_dynamic_smem((const void*)kernel, smem);
    if (e != cudaSuccess) return e;
    return launch_clusters(kernel, a.c.heads * kCluster, kShortThreads, smem, st, a);
}

// Tiles, at most.
long long most_tiles(const AttendArgs& a) { return (long long)a.c.heads * a.ng * ((a.c.cap() + kTile - 1) / kTile); }

// As many CTAs of attend_split as are resident at once, but no more than there can be tiles.
int resident_ctas(const AttendArgs& a) {
    return (int)std::min<long long>(most_tiles(a), std::min(num_sms(), kPlanGrid) * kCtasPerSm);
}

// Whether attend_join_few joins the units. With acc attend_weigh has to follow it (3 us), which pays where every weighing
// block of attend_join would add up sums for longer: a warp ceil(G / 8) query heads, a lane every 32nd of a
// unit's parts. (G 16, 296 parts, 20 steps: 39.8 us, 25.0 so; G 12, 94 parts, 6: 15.2, 13.6; G 4, 148 parts, 5: 13.4, 15.6.)
bool joins_few(const AttendArgs& a) {
    const int units = a.c.heads * a.ng;
    if (units > kFewUnits) return false;
    return !a.acc || a.ng > 1 || (a.G + kJoinWarps - 1) / kJoinWarps * ((a.resident / units + 31) / 32) >= kFewSteps;
}

template <typename T, int D>
cudaError_t launch_all(const AttendArgs& a, cudaStream_t st) {
    constexpr int kStages = D == 128 ? 3 : 6;
    // One launch where heads are so few that their clusters run at once, and no table holds more rows
    // than a cluster takes. (8 heads of 2111 rows: 6.6 us, 9.3 by
    // attend_split and attend_join; 2 heads of 512: 3.9, 6.7.)
    if (a.ng == 1 && a.c.heads * kCluster <= std::min(kShortCtas, num_sms()) && a.c.cap() <= kCluster * kShortRows) {
        if (a.gq == 16) return launch_short<T, D, true, D == 128 ? 2 : 4>(a, st);
        return launch_short<T, D, false, D == 128 ? 3 : 4>(a, st);
    }
    // as many CTAs with short runs again where runs can be long
    const long long most = most_tiles(a);
    const int more = most >= (long long)kLongRun * a.resident ? a.resident : 0;
    cudaError_t e = a.gq == 16 ? launch_split<T, D, true, kStages>(a, a.resident + more, st)
                               : launch_split<T, D, false, kStages>(a, a.resident + more, st);
    if (e != cudaSuccess) return e;
    const long long share = (most + a.resident - 1) / a.resident * kTile;       // rows of a share, at most
    const int pieces = (int)std::min<long long>(kJoinPieces, (share + kJoinThreads * 4 - 1) / (kJoinThreads * 4));
    const int weighers = a.logits && !a.lse2 ? 2 * (a.resident * pieces + more) : 0, rows = std::min(a.G, a.gq);
    e = a.firsts ? launch_clusters(attend_join_few<T, D>, a.c.heads * a.ng * rows * kCluster, kJoinThreads, 0, st, a, rows)
                 : launch_dependent(attend_join<T, D>, weighers + (a.resident + more) * rows, kJoinThreads, 0, st, a,
                                    weighers, pieces, rows);
    if (e != cudaSuccess || !a.lse2) return e;
    const int per = std::max(1, std::min(num_sms() * 8 / a.c.heads, (a.c.cap() + kJoinThreads - 1) / kJoinThreads));
    return launch_dependent(attend_weigh, a.c.heads * per, kJoinThreads, 0, st, a, per);
}

}  // namespace

size_t attend_workspace_bytes(const kvp_cache_shape& s, bool accumulate) { return layout_of(s, accumulate).bytes; }

cudaError_t launch_attend(const kvp_cache_shape& s, const uint16_t* q, const uint16_t* k_pages,
                          const uint16_t* v_pages, const int32_t* table, const int32_t* lens, uint16_t* out,
                          float* lse, float* acc, void* workspace, cudaStream_t st) {
    const Layout l = layout_of(s, acc != nullptr);
    char* ws = (char*)workspace;
    AttendArgs a;
    a.c = cache_view(s, table, lens);
    a.q = q;
    a.k = k_pages;
    a.v = v_pages;
    a.out = out;
    a.lse = lse;
    a.acc = acc;
    a.G = s.hq / s.hkv;
    a.ng = l.ng;
    a.gq = l.gq;
    a.scale2 = (float)(1.4426950408889634 / sqrt((double)s.head_dim));
    a.cuts = (Cut*)(ws + l.cuts);
    a.stats = (float2*)(ws + l.stats);
    a.parts = (float*)(ws + l.parts);
    a.resident = resident_ctas(a);
    a.firsts = joins_few(a) ? (Cut*)(ws + l.firsts) : nullptr;
    a.many = a.firsts ? INT_MAX : (int)std::min<long long>(INT_MAX, (long long)kManyParts * a.c.heads * a.ng);
    a.lse2 = acc && (l.ng > 1 || a.firsts) ? (float*)(ws + l.lse2) : nullptr;
    a.logits = acc ? (float*)(ws + l.logits) : nullptr;
    if (s.dtype == KVP_BF16)
        return s.head_dim == 128 ? launch_all<__nv_bfloat16, 128>(a, st)
                                 : launch_all<__nv_bfloat16, 64>(a, st);
    return s.head_dim == 128 ? launch_all<__half, 128>(a, st) : launch_all<__half, 64>(a, st);
}

#ifdef KVP_CHECKS
KVP_DEFINE_CHECK_READER(take_check_attend)
#endif

}  // namespace kvp
