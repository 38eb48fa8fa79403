// The paged cache's bookkeeping and its uncompressed form: block tables and slot maps from request lengths,
// storing new keys and values (with per-page channel bounds), page selection and paged decode attention.
//
// A page holds 16 tokens.  Head page e = page * H_kv + h is the 16 rows of kv head h in a page; row t % 16 of
// head page e is row e * 16 + t % 16 of a pool, the row a slot names (the paged layout of tq_attend_args).
#pragma once

#include <climits>

#include "tq_device.cuh"

namespace tq {
namespace dev {

constexpr int kPage = 16;

// ------------------------------------------------------------------------------------------ planning

struct PlanParams {
    const int32_t* new_lens;
    const int32_t* seq_lens;
    int32_t* table;
    int32_t* ring;
    const int32_t* state;              // {index of the first free page in the ring, free pages}
    int64_t* slots;
    int32_t* row_start;
    int32_t* start_pos;
    int32_t* seq_lens_out;
    int32_t* state_out;
    int batch, width, num_pages, heads;
    int64_t max_tokens;
};

constexpr int kPlanThreads = 1024;
constexpr int kSlotTile = 256;         // tokens whose slots one CTA of plan_slots_kernel writes

// Inclusive scan of two values over the block (every thread takes part); `total` receives the block's sums.
__device__ __forceinline__ void block_scan2(int64_t& a, int64_t& b, int64_t (&total)[2], int64_t (*warp_sums)[2]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t ta = __shfl_up_sync(0xffffffffu, a, o), tb = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) { a += ta; b += tb; }
    }
    __syncthreads();                                     // warp_sums may still be read from the scan before
    if (lane == 31) { warp_sums[warp][0] = a; warp_sums[warp][1] = b; }
    __syncthreads();
    if (warp == 0) {
        int64_t sa = lane < nwarps ? warp_sums[lane][0] : 0, sb = lane < nwarps ? warp_sums[lane][1] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t ta = __shfl_up_sync(0xffffffffu, sa, o), tb = __shfl_up_sync(0xffffffffu, sb, o);
            if (lane >= o) { sa += ta; sb += tb; }
        }
        if (lane < nwarps) { warp_sums[lane][0] = sa; warp_sums[lane][1] = sb; }
    }
    __syncthreads();
    if (warp > 0) { a += warp_sums[warp - 1][0]; b += warp_sums[warp - 1][1]; }
    total[0] = warp_sums[nwarps - 1][0];
    total[1] = warp_sums[nwarps - 1][1];
}

// The slot of kv head 0 of input row `token`, or -1: rows of refused or finished requests, rows past the last
// request's, and tokens whose table entry names no page.
__device__ __forceinline__ int64_t plan_slot(const PlanParams& p, int64_t token) {
    int lo = 0, hi = p.batch;                            // the first request whose rows end after `token`
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (p.row_start[mid + 1] <= token) lo = mid + 1; else hi = mid;
    }
    if (lo == p.batch) return -1;
    const int start = p.start_pos[lo];
    if (start < 0) return -1;
    const int64_t pos = start + (token - p.row_start[lo]);
    const int page = p.table[static_cast<int64_t>(lo) * p.width + pos / kPage];
    if (page < 0 || page >= p.num_pages) return -1;
    return static_cast<int64_t>(page) * p.heads * kPage + pos % kPage;
}

// Slots of `n` tokens from `token0` on: one search per token, then the tokens' H_kv slots with coalesced stores.
__device__ __forceinline__ void write_slots(const PlanParams& p, int64_t token0, int n, int64_t* base) {
    for (int i = threadIdx.x; i < n; i += blockDim.x) base[i] = plan_slot(p, token0 + i);
    __syncthreads();
    int64_t* dst = p.slots + token0 * p.heads;
    for (int i = threadIdx.x; i < n * p.heads; i += blockDim.x) {
        const int t = i / p.heads, h = i - t * p.heads;
        dst[i] = base[t] < 0 ? -1 : base[t] + h * kPage;
    }
}

// One CTA: lengths, admission, table rows and the free ring.  Admission is a prefix rule (a request that needs
// pages gets them when the running sum of needs up to it is within the free count), so two scans decide it for
// every request at once.  Pages are taken from the ring's start and given back at its end, so what this call reads
// and what it writes never overlap.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanParams p, bool with_slots) {
    __shared__ int64_t s_warp[32][2];
    __shared__ int64_t s_base[kPlanThreads];
    __shared__ int s_old[kPlanThreads], s_need[kPlanThreads], s_from[kPlanThreads], s_gone[kPlanThreads],
        s_to[kPlanThreads];
    __shared__ int s_taken;
    // the slot grid (a programmatic dependent) may be scheduled; it waits for this grid's completion
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x;
    const int cap = p.num_pages;
    int head = p.state[0], count = p.state[1];
    head = (head < 0 || head >= cap) ? 0 : head;
    count = count < 0 ? 0 : (count > cap ? cap : count);
    const int64_t most = static_cast<int64_t>(p.width) * kPage;
    if (tid == 0) {
        s_taken = 0;
        p.row_start[0] = 0;
    }
    int64_t rows_before = 0, gone_before = 0, need_before = 0, total[2];
    for (int b0 = 0; b0 < p.batch; b0 += kPlanThreads) {
        const int b = b0 + tid;
        const bool active = b < p.batch;
        const int want = active ? p.new_lens[b] : 0;
        int64_t len = active ? p.seq_lens[b] : 0;
        len = len < 0 ? 0 : (len > most ? most : len);
        const int64_t req = want > 0 ? want : 0;
        const int64_t old_pages = (len + kPage - 1) / kPage;
        const int64_t gone = want < 0 ? old_pages : 0;
        int64_t end = req, gone_end = gone;
        block_scan2(end, gone_end, total, s_warp);
        end += rows_before;
        gone_end += gone_before;
        rows_before += total[0];
        gone_before += total[1];
        const bool fits = active && want >= 0 && len + req <= most && end <= p.max_tokens;
        const int64_t need = fits ? (len + req + kPage - 1) / kPage - old_pages : 0;
        int64_t upto = need, unused = 0;
        block_scan2(upto, unused, total, s_warp);
        upto += need_before;
        need_before += total[0];
        const bool ok = fits && (need == 0 || upto <= count);
        if (ok && need > 0) atomicMax(&s_taken, static_cast<int>(upto));
        if (active) {
            p.row_start[b + 1] = end > INT_MAX ? INT_MAX : static_cast<int>(end);
            p.start_pos[b] = ok ? static_cast<int>(len) : -1;
            p.seq_lens_out[b] = want < 0 ? 0 : static_cast<int>(len + (ok ? req : 0));
        }
        const int64_t to = gone_end - gone;
        s_old[tid] = static_cast<int>(old_pages);
        s_need[tid] = ok ? static_cast<int>(need) : 0;
        s_from[tid] = ok ? static_cast<int>(upto - need) : 0;
        s_gone[tid] = static_cast<int>(gone);
        s_to[tid] = to > cap ? cap : static_cast<int>(to);
        __syncthreads();
        // table rows and the ring: the block's threads in equal groups, a request per group
        const int n = p.batch - b0 < kPlanThreads ? p.batch - b0 : kPlanThreads;
        int per = kPlanThreads;
        while (per > 32 && per * n > kPlanThreads) per >>= 1;
        const int lane = tid & (per - 1);
        for (int i = tid / per; i < n; i += kPlanThreads / per) {
            int32_t* row = p.table + static_cast<int64_t>(b0 + i) * p.width;
            const int need_i = s_need[i], gone_i = s_gone[i];
            int32_t* fresh = row + s_old[i];
            const int from = head + s_from[i];           // below 2 cap: from + j - head < count <= cap
#pragma unroll 4
            for (int j = lane; j < need_i; j += per) {
                const int at = from + j;
                fresh[j] = p.ring[at >= cap ? at - cap : at];
            }
            const int64_t to_i = static_cast<int64_t>(count) + s_to[i];
            for (int j = lane; j < gone_i && to_i + j < cap; j += per) {
                const int at = static_cast<int>(to_i + j) - (cap - head);
                p.ring[at < 0 ? at + cap : at] = row[j];
            }
        }
        __syncthreads();
    }
    if (tid == 0) {
        const int taken = s_taken;
        const int64_t room = cap - count;
        const int back = static_cast<int>(gone_before < room ? gone_before : room);
        const int next = head + taken;
        p.state_out[0] = next >= cap ? next - cap : next;
        p.state_out[1] = count - taken + back;
    }
    if (with_slots) {
        for (int64_t t0 = 0; t0 < p.max_tokens; t0 += kPlanThreads) {
            const int n = static_cast<int>(p.max_tokens - t0 < kPlanThreads ? p.max_tokens - t0 : kPlanThreads);
            write_slots(p, t0, n, s_base);
            __syncthreads();
        }
    }
}

// Slots of larger calls: one CTA per kSlotTile input rows, after plan_kernel.
__global__ void __launch_bounds__(kSlotTile) plan_slots_kernel(const PlanParams p) {
    __shared__ int64_t s_base[kSlotTile];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kSlotTile;
    const int n = static_cast<int>(p.max_tokens - t0 < kSlotTile ? p.max_tokens - t0 : kSlotTile);
    write_slots(p, t0, n, s_base);
}

// ------------------------------------------------------------------------------- appending to pages

template <typename T> struct Pair;                       // two 16-bit values and their minimum / maximum
template <> struct Pair<__half> {
    using type = __half2;
    static __device__ __forceinline__ float2 floats(uint32_t u) { return __half22float2(*reinterpret_cast<__half2*>(&u)); }
};
template <> struct Pair<__nv_bfloat16> {
    using type = __nv_bfloat162;
    static __device__ __forceinline__ float2 floats(uint32_t u) {
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }
};

template <typename T>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    using P = typename Pair<T>::type;
    const P r = __hmin2(*reinterpret_cast<P*>(&a), *reinterpret_cast<P*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
template <typename T>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    using P = typename Pair<T>::type;
    const P r = __hmax2(*reinterpret_cast<P*>(&a), *reinterpret_cast<P*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}

template <int W> struct Words;                           // W 32-bit words moved by one load or store
template <> struct Words<1> { using type = uint32_t; };
template <> struct Words<2> { using type = uint2; };
template <> struct Words<4> { using type = uint4; };

struct AppendParams {
    const void* k;                     // [n][H_kv][d] rows: token stride and head stride in elements
    const void* v;
    int64_t k_token, k_head, v_token, v_head;
    const int64_t* slots;              // [n][H_kv]
    int64_t n;
    int64_t rows;                      // pool rows: num_pages * H_kv * 16
    void* k_pool;                      // nullable
    void* v_pool;                      // nullable
    void* bounds;                      // nullable: [num_pages][H_kv][2][d]
    int heads, tile;                   // tokens whose page runs one warp looks after (1 .. 16)
};

constexpr int kAppendWarps = 8;

// One warp owns the page runs (consecutive input tokens of one kv head in one page) that start in its tile of
// tokens, and follows the last one past the tile's end.  A run's rows are read once: stored to the pool and folded
// into the page's channel bounds, which no other warp touches, so nothing is atomic and the result does not depend
// on the order of warps.  A lane holds d / 32 channels of a row.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kAppendWarps) append_kernel(const AppendParams p) {
    constexpr int W = D / 64;                            // words per lane and row
    constexpr int kBatch = 8;                            // rows in flight
    using Vec = typename Words<W>::type;
    const int lane = threadIdx.x & 31;
    const int64_t gw = static_cast<int64_t>(blockIdx.x) * kAppendWarps + (threadIdx.x >> 5);
    const int h = static_cast<int>(gw % p.heads);
    const int64_t t0 = gw / p.heads * p.tile;
    if (t0 >= p.n) return;
    const T* k = static_cast<const T*>(p.k) + h * p.k_head + lane * 2 * W;
    const T* v = static_cast<const T*>(p.v) + h * p.v_head + lane * 2 * W;
    T* k_pool = static_cast<T*>(p.k_pool);
    T* v_pool = static_cast<T*>(p.v_pool);
    auto slot_of = [&](int64_t t) -> int64_t {           // the slot of token t, -1 where the row is not stored
        const int64_t s = (t >= 0 && t < p.n) ? p.slots[t * p.heads + h] : -1;
        return s < p.rows ? s : -1;
    };
    // lane l looks at token t0 - 1 + l
    const int64_t slot = slot_of(t0 - 1 + lane);
    const int64_t page = slot < 0 ? -1 : slot / kPage;
    const int64_t prev = __shfl_up_sync(0xffffffffu, page, 1);
    unsigned starts = __ballot_sync(0xffffffffu, page >= 0 && page != prev) & ((2u << p.tile) - 2u);
    while (starts) {
        int at = __ffs(starts) - 1;
        starts &= starts - 1;
        const int64_t run = __shfl_sync(0xffffffffu, page, at);
        int64_t token = t0 - 1 + at, ws = slot;          // the run's next token; slots of the window it lies in
        unsigned same = __ballot_sync(0xffffffffu, page == run) >> at;
        bool fresh = false;                              // the page's first token is new: its old bounds do not count
        alignas(16) uint32_t lo[W], hi[W];
        bool any = false;
        while (true) {
            const int len = ~same ? __ffs(~same) - 1 : 32;
            const unsigned mask = (len >= 32 ? 0xffffffffu : ((1u << len) - 1u)) << at;
            fresh |= (__ballot_sync(0xffffffffu, ws % kPage == 0) & mask) != 0;
            for (int j0 = 0; j0 < len; j0 += kBatch) {
                Vec kr[kBatch], vr[kBatch];
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    if (j0 + u < len) {
                        kr[u] = *reinterpret_cast<const Vec*>(k + (token + j0 + u) * p.k_token);
                        if (v_pool) vr[u] = *reinterpret_cast<const Vec*>(v + (token + j0 + u) * p.v_token);
                    }
                }
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int64_t s = __shfl_sync(0xffffffffu, ws, (at + j0 + u) & 31);
                    if (j0 + u < len) {
                        if (k_pool) *reinterpret_cast<Vec*>(k_pool + s * D + lane * 2 * W) = kr[u];
                        if (v_pool) *reinterpret_cast<Vec*>(v_pool + s * D + lane * 2 * W) = vr[u];
                        const uint32_t* w = reinterpret_cast<const uint32_t*>(&kr[u]);
#pragma unroll
                        for (int i = 0; i < W; ++i) {
                            lo[i] = any ? min2<T>(lo[i], w[i]) : w[i];
                            hi[i] = any ? max2<T>(hi[i], w[i]) : w[i];
                        }
                        any = true;
                    }
                }
            }
            if (at + len < 32) break;
            // the run reaches the window's end: look at the next 32 tokens
            token += len;
            at = 0;
            ws = slot_of(token + lane);
            same = __ballot_sync(0xffffffffu, ws >= 0 && ws / kPage == run);
            if (!(same & 1u)) break;
        }
        if (p.bounds) {
            T* b = static_cast<T*>(p.bounds) + run * 2 * D + lane * 2 * W;
            if (!fresh) {
                const Vec ol = *reinterpret_cast<const Vec*>(b), oh = *reinterpret_cast<const Vec*>(b + D);
                const uint32_t *pl = reinterpret_cast<const uint32_t*>(&ol), *ph = reinterpret_cast<const uint32_t*>(&oh);
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    lo[i] = min2<T>(lo[i], pl[i]);
                    hi[i] = max2<T>(hi[i], ph[i]);
                }
            }
            *reinterpret_cast<Vec*>(b) = *reinterpret_cast<Vec*>(lo);
            *reinterpret_cast<Vec*>(b + D) = *reinterpret_cast<Vec*>(hi);
        }
    }
}

// ------------------------------------------------------------------------------------- page selection

struct SelectParams {
    const void* q;                     // [B] rows of H_q heads: q_stride elements from one sequence to the next
    int64_t q_stride;
    const void* bounds;                // [num_pages][H_kv][2][d]
    const int32_t* table;              // [B][width]
    const int32_t* seq_lens;           // [B]
    int32_t* pages;                    // [B][H_kv][budget]
    int32_t* lens;                     // [B][H_kv]
    int heads, group, width, num_pages, budget, keep_first, keep_last;
    int share_cap;                     // pages one CTA can hold
};

constexpr int kSelThreads = 256;
constexpr int kSelUnroll = 4;          // pages a lane group scores at a time

// shared memory of select_kernel: keys and page ids of the CTA's pages, then the query's positive and negative parts
inline __host__ __device__ size_t select_smem(int share_cap, int group, int d) {
    return static_cast<size_t>(share_cap) * 8 + static_cast<size_t>(group) * d * 8;
}

__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t v;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(v));
    return v;
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t v;
    asm("mov.u32 %0, %%cluster_ctaid.x;" : "=r"(v));
    return v;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A 32-bit word of the same shared-memory variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_load(const void* p, uint32_t rank) {
    uint32_t a, v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

// Scores and the `budget` best pages of one (sequence, kv head), by one cluster of CTAs that share its pages out in
// order.
//
// The score of a page is max over the group's query heads of U_g = sum_c max(q_gc lo_c, q_gc hi_c), which is at least
// q_g . k for every key in the page.  With lo <= hi the larger product is (q > 0 ? q hi : q lo), computed as two
// fused multiply-adds of max(q, 0) with hi and min(q, 0) with lo: one of the products is a zero, and products of
// 16-bit values are exact in fp32, so each step is a plain rounded addition.  The order of additions is part of the
// operator (a lane's 8 channels as an even and an odd chain, then lanes i and i + half), so that the choice of pages
// can be reproduced bit for bit.
//
// The choice itself is a radix selection over order-preserving keys, 8 bits a pass: every CTA counts its keys, the
// cluster's counts are added up through distributed shared memory, and every CTA finds the same threshold.  Ties at
// the threshold go to the lowest page index.
template <typename T, int D>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectParams p) {
    constexpr int LP = D / 8;                            // lanes per page
    constexpr int GW = 32 / LP;                          // lane groups per warp
    constexpr int U = kSelUnroll;
    static_assert(U == 4, "the reduction below spreads four pages over the lanes of a group");
    extern __shared__ __align__(16) uint8_t smem[];
    float* qp = reinterpret_cast<float*>(smem);          // [G][2][LP][4]: max(q, 0)
    float* qn = qp + p.group * D;                        // the same of min(q, 0)
    uint32_t* keys = reinterpret_cast<uint32_t*>(qn + p.group * D);
    int32_t* ids = reinterpret_cast<int32_t*>(keys + p.share_cap);
    __shared__ uint32_t s_hist[4][256];
    __shared__ uint32_t s_pick[2];
    __shared__ uint32_t s_warp[kSelThreads / 32 + 1];
    __shared__ uint32_t s_count[2];

    const uint32_t cs = cluster_size(), rank = cluster_rank();
    const int row = blockIdx.x / cs;
    const int b = row / p.heads, h = row - b * p.heads;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t most = static_cast<int64_t>(p.width) * kPage;
    int64_t len = p.seq_lens[b];
    len = len < 0 ? 0 : (len > most ? most : len);
    const int nb = static_cast<int>((len + kPage - 1) / kPage);
    const int32_t* table = p.table + static_cast<int64_t>(b) * p.width;
    int32_t* out = p.pages + static_cast<int64_t>(row) * p.budget;
    if (rank == 0 && tid == 0)
        p.lens[row] = static_cast<int>(nb <= p.budget ? len : len - static_cast<int64_t>(nb - p.budget) * kPage);
    if (nb <= p.budget) {                                // every page is kept
        for (int j = rank * kSelThreads + tid; j < p.budget; j += cs * kSelThreads) {
            const int id = j < nb ? table[j] : -1;
            out[j] = (id < 0 || id >= p.num_pages) ? -1 : id * p.heads + h;
        }
        return;
    }
    const int share = (nb + cs - 1) / cs;
    const int p0 = rank * share;
    const int cnt = nb - p0 < 0 ? 0 : (nb - p0 < share ? nb - p0 : share);
    // ---- the query and the page ids
    const T* q = static_cast<const T*>(p.q) + b * p.q_stride + static_cast<int64_t>(h) * p.group * D;
    for (int i = tid; i < p.group * D; i += kSelThreads) {
        const float x = static_cast<float>(q[i]);
        const int g = i / D, c = i % D;
        const int at = g * D + (c % 8 / 4) * (D / 2) + c / 8 * 4 + c % 4;
        qp[at] = fmaxf(x, 0.f);
        qn[at] = fminf(x, 0.f);
    }
    for (int j = tid; j < cnt; j += kSelThreads) ids[j] = table[p0 + j];
    for (int i = tid; i < 4 * 256; i += kSelThreads) s_hist[i / 256][i % 256] = 0;
    __syncthreads();
    // ---- scores
    const int l = lane % LP;
    const bool hi_half = (l & (LP / 2)) != 0, hi_quarter = (l & (LP / 4)) != 0;
    const float4* qp4 = reinterpret_cast<const float4*>(qp) + l;
    const float4* qn4 = reinterpret_cast<const float4*>(qn) + l;
    const T* bounds = static_cast<const T*>(p.bounds) + static_cast<int64_t>(h) * 2 * D + l * 8;
    const int64_t page_stride = static_cast<int64_t>(p.heads) * 2 * D;
    constexpr int kStep = (kSelThreads / 32) * GW * U;
    for (int base = (warp * GW + lane / LP) * U; base - (lane / LP) * U < cnt; base += kStep) {
        float2 lo[U][4], hi[U][4];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int id = base + u < cnt ? ids[base + u] : -1;
            uint4 a = make_uint4(0u, 0u, 0u, 0u), c = a;
            if (id >= 0 && id < p.num_pages) {
                const T* src = bounds + id * page_stride;
                a = __ldg(reinterpret_cast<const uint4*>(src));
                c = __ldg(reinterpret_cast<const uint4*>(src + D));
            }
            const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, cw[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                lo[u][i] = Pair<T>::floats(aw[i]);
                hi[u][i] = Pair<T>::floats(cw[i]);
            }
        }
        float best = -INFINITY;
        for (int g = 0; g < p.group; ++g) {
            const float4 p0v = qp4[g * (D / 4)], p1v = qp4[g * (D / 4) + LP];
            const float4 n0v = qn4[g * (D / 4)], n1v = qn4[g * (D / 4) + LP];
            const float2 pq[4] = {{p0v.x, p0v.y}, {p0v.z, p0v.w}, {p1v.x, p1v.y}, {p1v.z, p1v.w}};
            const float2 nq[4] = {{n0v.x, n0v.y}, {n0v.z, n0v.w}, {n1v.x, n1v.y}, {n1v.z, n1v.w}};
            float v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float2 acc = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc = __ffma2_rn(pq[i], hi[u][i], acc);
                    acc = __ffma2_rn(nq[i], lo[u][i], acc);
                }
                v[u] = acc.x + acc.y;
            }
            // lanes i and i + LP/2 add up: the upper half goes on with pages 2, 3, the lower with 0, 1; then quarters
            const float k0 = hi_half ? v[2] : v[0], k1 = hi_half ? v[3] : v[1];
            const float g0 = hi_half ? v[0] : v[2], g1 = hi_half ? v[1] : v[3];
            const float w0 = k0 + __shfl_xor_sync(0xffffffffu, g0, LP / 2);
            const float w1 = k1 + __shfl_xor_sync(0xffffffffu, g1, LP / 2);
            float s = (hi_quarter ? w1 : w0) + __shfl_xor_sync(0xffffffffu, hi_quarter ? w0 : w1, LP / 4);
#pragma unroll
            for (int o = LP / 8; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            // a NaN sum must not hide behind another head's number
            best = (s > best || s != s) ? s : best;
        }
        const int j = base + (hi_half ? 2 : 0) + (hi_quarter ? 1 : 0);
        if ((l & (LP / 4 - 1)) == 0 && j < cnt) {
            const int at = p0 + j, id = ids[j];
            uint32_t bits = __float_as_uint(best + 0.f);             // -0 counts as 0
            bits = (bits >> 31) ? ~bits : bits | 0x80000000u;
            if (best != best || id < 0 || id >= p.num_pages) bits = 0u;
            if (at < p.keep_first || at >= nb - p.keep_last) bits = 0xffffffffu;
            keys[j] = bits;
        }
    }
    __syncthreads();
    // ---- the budget-th largest key of the cluster
    uint32_t prefix = 0, mask = 0, need = static_cast<uint32_t>(p.budget);
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
        for (int j = tid; j < cnt; j += kSelThreads)
            if ((keys[j] & mask) == prefix) atomicAdd(&s_hist[pass][(keys[j] >> shift) & 255u], 1u);
        cluster_sync();
        // thread t takes bin 255 - t, so that an inclusive scan counts the keys from the largest bin down
        uint32_t c = 0;
        for (uint32_t r = 0; r < cs; ++r) c += cluster_load(&s_hist[pass][255 - tid], r);
        uint32_t incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t t = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += t;
        }
        if (lane == 31) s_warp[warp] = incl;
        __syncthreads();
        for (int w = 0; w < warp; ++w) incl += s_warp[w];
        if (incl >= need && incl - c < need) {
            s_pick[0] = 255u - tid;
            s_pick[1] = incl - c;
        }
        __syncthreads();
        prefix |= s_pick[0] << shift;
        mask |= 255u << shift;
        need -= s_pick[1];
        __syncthreads();
    }
    // keys above `prefix` are in, and the first `need` of those equal to it
    uint32_t mine = 0;                                   // above: low half, equal: high half
    for (int j = tid; j < cnt; j += kSelThreads) mine += (keys[j] > prefix ? 1u : 0u) + (keys[j] == prefix ? 0x10000u : 0u);
#pragma unroll
    for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) s_warp[warp] = mine;
    __syncthreads();
    if (tid == 0) {
        uint32_t a = 0;
        for (int w = 0; w < kSelThreads / 32; ++w) a += s_warp[w];
        s_count[0] = a & 0xffffu;
        s_count[1] = a >> 16;
    }
    cluster_sync();
    uint32_t above = 0, equal = 0;                       // in the CTAs before this one
    for (uint32_t r = 0; r < rank; ++r) {
        above += cluster_load(&s_count[0], r);
        equal += cluster_load(&s_count[1], r);
    }
    for (int j0 = 0; j0 < cnt; j0 += kSelThreads) {
        const int j = j0 + tid;
        const uint32_t key = j < cnt ? keys[j] : 0u;
        const bool gt = j < cnt && key > prefix, eq = j < cnt && key == prefix;
        const unsigned mg = __ballot_sync(0xffffffffu, gt), me = __ballot_sync(0xffffffffu, eq);
        if (lane == 0) s_warp[warp] = __popc(mg) | (__popc(me) << 16);
        __syncthreads();
        uint32_t before = 0, all = 0;
        for (int w = 0; w < kSelThreads / 32; ++w) {
            before += w < warp ? s_warp[w] : 0u;
            all += s_warp[w];
        }
        const uint32_t g_at = above + (before & 0xffffu) + __popc(mg & ((1u << lane) - 1u));
        const uint32_t e_at = equal + (before >> 16) + __popc(me & ((1u << lane) - 1u));
        if (gt || (eq && e_at < need)) {
            const int id = ids[j];
            out[g_at + (e_at < need ? e_at : need)] = (id < 0 || id >= p.num_pages) ? -1 : id * p.heads + h;
        }
        above += all & 0xffffu;
        equal += all >> 16;
        __syncthreads();
    }
    cluster_sync();                                      // a neighbour may still read this CTA's counts
}

// -------------------------------------------------------------------- attention over uncompressed pages

struct AttendPagesParams {
    const void* q;                     // [B] rows of H_q heads: q_stride elements from one sequence to the next
    const void* k_pool;
    const void* v_pool;
    const int32_t* table;              // [units][width]: page ids, or head page ids of a selection
    const int32_t* lens;               // [units]
    float* out;                        // [B][H_q][d]
    float* partials;                   // [CTAs][2][16 + 8 d]
    struct AttendPagesMeta* meta;      // [CTAs]
    int64_t q_stride, k_page, v_page;  // elements; *_page: from one page to the next
    int units, mult;                   // table rows, and kv heads that share a table row (1 for selections)
    int width, num_ids, heads, group;
    int min_pages;                     // pages a CTA takes at least
    float scale_log2;
};

// What the join needs of the CTA that starts inside a row: the row and its range on the flattened page axis.
struct AttendPagesMeta {
    int64_t row_begin, row_end, share;
    int row, pad;
};

template <int D>
struct PagesCfg {
    static constexpr int kWarps = 4;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kPageBytes = kPage * D * 2;                 // one page of keys (or values) of a kv head
    static constexpr int kStages = (D == 64) ? 6 : 3;                // pages of keys and values in flight per warp
    static constexpr int kCtasPerSm = (D == 256) ? 1 : 2;
    static constexpr int kRing = kWarps * kStages * 2 * kPageBytes;
    static constexpr int kHeadStride = D + 4;                        // spreads the accumulator rows over the banks
    static constexpr int kComb = 16 + 8 * kHeadStride;               // floats per warp: m[8], l[8], O[8][D + 4]
    static constexpr int kSmem = kRing + kWarps * kComb * 4;
    static constexpr int kPart = 16 + 8 * D;                         // floats per partial: m[8], l[8], O[8][D]
};

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                 uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A pair of fp32 weights as a sum of 16-bit pairs: two fp16 terms keep 22 bits, three bf16 terms 24.
template <typename T> struct Weights;
template <> struct Weights<__half> {
    static constexpr int kTerms = 2;
    static __device__ __forceinline__ void split(float x, float y, uint32_t (&t)[kTerms]) {
        const __half2 h = __floats2half2_rn(x, y);
        const float2 f = __half22float2(h);
        const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
        t[0] = *reinterpret_cast<const uint32_t*>(&h);
        t[1] = *reinterpret_cast<const uint32_t*>(&l);
    }
};
template <> struct Weights<__nv_bfloat16> {
    static constexpr int kTerms = 3;
    static __device__ __forceinline__ void split(float x, float y, uint32_t (&t)[kTerms]) {
#pragma unroll
        for (int i = 0; i < kTerms; ++i) {               // the upper 16 bits; the rest is exact
            const uint32_t ux = __float_as_uint(x), uy = __float_as_uint(y);
            t[i] = __byte_perm(ux, uy, 0x7632);
            x -= __uint_as_float(ux & 0xffff0000u);
            y -= __uint_as_float(uy & 0xffff0000u);
        }
    }
};

// A place on the flattened page axis: units in order, the kv heads of a unit in order, then pages.
struct PageCursor {
    int unit, m, pg, pages;            // pages: of this unit
};

__device__ __forceinline__ int64_t unit_len(const AttendPagesParams& p, int u) {
    const int64_t most = static_cast<int64_t>(p.width) * kPage;
    const int64_t t = p.lens[u];
    return t < 0 ? 0 : (t > most ? most : t);
}
__device__ __forceinline__ int unit_pages(const AttendPagesParams& p, int u) {
    return static_cast<int>((unit_len(p, u) + kPage - 1) / kPage);
}

// Moves on by n pages; past the last page the cursor stays behind the last unit.
__device__ __forceinline__ void advance(const AttendPagesParams& p, PageCursor& c, int n) {
    c.pg += n;
    while (c.pg >= c.pages) {
        c.pg -= c.pages;
        if (++c.m == p.mult) {
            c.m = 0;
            do {
                if (++c.unit >= p.units) { c.pages = INT_MAX; return; }
                c.pages = unit_pages(p, c.unit);
            } while (c.pages == 0);
        }
    }
}

// Attention of one new token over a paged cache.  softmax(scale q k^T) v needs every key and value once and a few
// operations per byte, so the kernel is bound by how fast pages can be read, and the grid is laid out for that alone:
// all pages of the call, in the order (table row, kv head, page), are cut into equal shares, one per resident CTA,
// whatever the lengths of the sequences are.  A share covers parts of one or several rows (a row: one sequence and
// kv head with its query heads); a row that lies inside one share is finished there, and attend_pages_join_kernel
// joins the others.  The running maximum and sum (fp32) make the split exact up to rounding.
//
// Warp w of a CTA takes pages w, w + 4, ... of the share and keeps kStages of them in flight in its own ring of
// shared memory with 16-byte cp.async copies, so no warp waits for another until a row ends.  16-byte chunk c of a
// page's row r sits at chunk c ^ (r % 8): the copies and both ldmatrix reads are then free of bank conflicts.
//   scores  S[head][token]  = q (A, 8 of 16 rows used) x k (B)
//   values  O^T[col][head] += v^T (A) x p (B): the scores' fragment layout is that of p, nothing moves between lanes
// p is 2^(s - m + 12) split into 16-bit terms (see Weights), so that rounding it costs no accuracy; with 8 heads or
// fewer per row the tensor work is a small part of the time either way.
template <typename T, int D>
__global__ void __launch_bounds__(PagesCfg<D>::kThreads, PagesCfg<D>::kCtasPerSm)
    attend_pages_kernel(const AttendPagesParams p) {
    using C = PagesCfg<D>;
    constexpr int S = C::kStages;
    constexpr int KS = D / 16;                           // k-steps of the scores, and 16-column tiles of the values
    constexpr float kPExp = 12.f;                        // weights carry 2^12 so that small ones keep their fp16 bits
    constexpr float kSlack = 3.f;                        // a logit may pass the running maximum by this before it moves
    extern __shared__ __align__(16) uint8_t smem[];
    float* comb = reinterpret_cast<float*>(smem + C::kRing);
    int64_t* s_setup = reinterpret_cast<int64_t*>(comb); // used before the first row ends only
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gid = lane >> 2, tig = lane & 3;
    const int G = p.group;

    // ---- this CTA's share
    int64_t sum = 0;
    for (int u = tid; u < p.units; u += C::kThreads) sum += unit_pages(p, u);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s_setup[warp] = sum;
    // rows without a token are nobody's page: their zeros are written here
    for (int u = blockIdx.x; u < p.units; u += gridDim.x) {
        if (unit_pages(p, u) == 0) {
            float* o = p.out + static_cast<int64_t>(u) * p.mult * G * D;
            for (int i = tid; i < p.mult * G * D; i += C::kThreads) o[i] = 0.f;
        }
    }
    __syncthreads();
    const int64_t total = (s_setup[0] + s_setup[1] + s_setup[2] + s_setup[3]) * p.mult;
    int64_t share = (total + gridDim.x - 1) / gridDim.x;
    if (share < p.min_pages) share = p.min_pages;
    const int64_t x0 = blockIdx.x * share;
    const int64_t x1 = x0 + share < total ? x0 + share : total;
    if (x0 >= total) {
        if (tid == 0) p.meta[blockIdx.x].row = -1;
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        return;
    }
    int64_t carry = 0;                                   // pages of the units before this tile of units
    for (int u0 = 0; u0 < p.units; u0 += C::kThreads) {
        const int n = u0 + tid < p.units ? unit_pages(p, u0 + tid) : 0;
        int64_t incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t t = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += t;
        }
        __syncthreads();                                 // the sums above, and the tile before, have been read
        if (lane == 31) s_setup[warp] = incl;
        __syncthreads();
        int64_t all = 0;
#pragma unroll
        for (int w = 0; w < C::kWarps; ++w) {
            if (w < warp) incl += s_setup[w];
            all += s_setup[w];
        }
        const int64_t begin = (carry + incl - n) * p.mult, end = (carry + incl) * p.mult;
        if (x0 >= begin && x0 < end) {
            s_setup[4] = u0 + tid;
            s_setup[5] = x0 - begin;
            s_setup[6] = n;
        }
        carry += all;
        if (carry * p.mult > x0) break;
    }
    __syncthreads();
    PageCursor seg;
    seg.unit = static_cast<int>(s_setup[4]);
    seg.pages = static_cast<int>(s_setup[6]);
    seg.m = static_cast<int>(s_setup[5] / seg.pages);
    seg.pg = static_cast<int>(s_setup[5] % seg.pages);
    __syncthreads();                                     // the rows' results may overwrite the set-up words
    if (tid == 0) {
        AttendPagesMeta m;
        m.row_begin = x0 - seg.pg;
        m.row_end = m.row_begin + seg.pages;
        m.share = share;
        m.row = seg.unit * p.mult + seg.m;
        m.pad = 0;
        p.meta[blockIdx.x] = m;
    }

    // ---- the copy ring
    const T* k_pool = static_cast<const T*>(p.k_pool);
    const T* v_pool = static_cast<const T*>(p.v_pool);
    const uint32_t ring = smem_u32(smem) + warp * S * 2 * C::kPageBytes;
    constexpr int CR = D / 8;                            // chunks per row
    constexpr int kCopies = kPage * CR / 32;             // 16-byte copies per lane, page and tensor
    PageCursor ld = seg;
    int64_t xl = x0 + warp;                              // the next page to be copied
    if (warp) advance(p, ld, warp);
    auto page_id = [&]() -> int {
        return xl < x1 ? __ldg(p.table + static_cast<int64_t>(ld.unit) * p.width + ld.pg) : -1;
    };
    unsigned good = 0;                                   // bit s: stage s holds a page (its id named one)
    auto issue = [&](int s, int id, int m) {
        good &= ~(1u << s);
        if (id >= 0 && id < p.num_ids) {
            good |= 1u << s;
            const T* ks = k_pool + id * p.k_page + m * (kPage * D) + lane * 8;
            const T* vs = v_pool + id * p.v_page + m * (kPage * D) + lane * 8;
            const uint32_t dst = ring + s * 2 * C::kPageBytes;
#pragma unroll
            for (int j = 0; j < kCopies; ++j) {
                const int n = j * 32 + lane, r = n / CR, c = n % CR;
                const uint32_t off = r * (2 * D) + (((c & ~7) | ((c ^ r) & 7)) << 4);
                cp_async16(dst + off, ks + j * 256);
            }
#pragma unroll
            for (int j = 0; j < kCopies; ++j) {
                const int n = j * 32 + lane, r = n / CR, c = n % CR;
                const uint32_t off = r * (2 * D) + (((c & ~7) | ((c ^ r) & 7)) << 4);
                cp_async16(dst + C::kPageBytes + off, vs + j * 256);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int next_id, next_m;
    {
        int id[S], m[S];
#pragma unroll
        for (int s = 0; s < S; ++s) {
            id[s] = page_id();
            m[s] = ld.m;
            xl += C::kWarps;
            if (xl < x1) advance(p, ld, C::kWarps);
        }
#pragma unroll
        for (int s = 0; s < S; ++s) issue(s, id[s], m[s]);
        next_id = page_id();
        next_m = ld.m;
    }

    // ---- rows
    int stage = 0;
    int64_t xw = x0 + warp;                              // this warp's next page
    int64_t xs = x0;
    const int mrow = (lane & 7) + ((lane >> 4) << 3);    // ldmatrix: matrices 0, 1 are rows 0-7, matrices 2, 3 rows 8-15
    const int mchunk = ((lane >> 3) & 1) ^ (lane & 7);   // and matrices 1, 3 the odd 16-byte chunk
    while (xs < x1) {
        const int64_t len = unit_len(p, seg.unit);
        const int64_t xe = xs + (seg.pages - seg.pg) < x1 ? xs + (seg.pages - seg.pg) : x1;
        const int64_t row = static_cast<int64_t>(seg.unit) * p.mult + seg.m;
        const int64_t row_begin = xs - seg.pg, row_end = row_begin + seg.pages;
        uint32_t qa[KS][2];
        {
            const int64_t b = row / p.heads;
            const int h = static_cast<int>(row - b * p.heads);
            const T* q = static_cast<const T*>(p.q) + b * p.q_stride + (static_cast<int64_t>(h) * G + gid) * D + 2 * tig;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                qa[ks][0] = gid < G ? __ldg(reinterpret_cast<const uint32_t*>(q + 16 * ks)) : 0u;
                qa[ks][1] = gid < G ? __ldg(reinterpret_cast<const uint32_t*>(q + 16 * ks + 8)) : 0u;
            }
        }
        float o[KS][4];
#pragma unroll
        for (int i = 0; i < KS; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        float m_run = -INFINITY, m_thr = -INFINITY, m_off = 0.f, l_run = 0.f;
        for (; xw < xe; xw += C::kWarps) {
            asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
            __syncwarp();
            const int64_t left = len - (xw - row_begin) * kPage;
            const int valid = left < kPage ? static_cast<int>(left) : kPage;
            if (good >> stage & 1u) {
                const uint32_t kb = ring + stage * 2 * C::kPageBytes + mrow * (2 * D);
                float sc[2][2][4] = {};
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    uint32_t f[4];
                    ldmatrix_x4(f, kb + ((mchunk ^ (2 * ks & 7)) << 4) + 128 * (ks / 4));
                    mma16816<T>(sc[ks & 1][0], qa[ks][0], 0u, qa[ks][1], 0u, f[0], f[1]);
                    mma16816<T>(sc[ks & 1][1], qa[ks][0], 0u, qa[ks][1], 0u, f[2], f[3]);
                }
                // head gid, tokens 2 tig, 2 tig + 1, 2 tig + 8, 2 tig + 9
                float lg[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) lg[e] = (sc[0][e >> 1][e & 1] + sc[1][e >> 1][e & 1]) * p.scale_log2;
                uint32_t vm0 = 0xffffffffu, vm1 = 0xffffffffu;   // which values of the tokens count
                if (valid < kPage) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (2 * tig + (e & 1) + 8 * (e >> 1) >= valid) lg[e] = -INFINITY;
                    vm0 = (2 * tig < valid ? 0xffffu : 0u) | (2 * tig + 1 < valid ? 0xffff0000u : 0u);
                    vm1 = (2 * tig + 8 < valid ? 0xffffu : 0u) | (2 * tig + 9 < valid ? 0xffff0000u : 0u);
                }
                const float lm = fmaxf(fmaxf(lg[0], lg[1]), fmaxf(lg[2], lg[3]));
                if (__any_sync(0xffffffffu, lm > m_thr)) {
                    float mq = fmaxf(lm, __shfl_xor_sync(0xffffffffu, lm, 1));
                    mq = fmaxf(mq, __shfl_xor_sync(0xffffffffu, mq, 2));
                    float corr = 1.f;
                    if (mq > m_thr) {
                        corr = exp2_approx(m_run - mq);          // 0 while m_run is -inf
                        m_run = mq;
                        m_thr = mq + kSlack;
                        m_off = mq - kPExp;
                        l_run *= corr;
                    }
                    // accumulator columns are heads 2 tig and 2 tig + 1
                    const float ca = __shfl_sync(0xffffffffu, corr, 8 * tig);
                    const float cb = __shfl_sync(0xffffffffu, corr, 8 * tig + 4);
#pragma unroll
                    for (int i = 0; i < KS; ++i) {
                        o[i][0] *= ca; o[i][1] *= cb; o[i][2] *= ca; o[i][3] *= cb;
                    }
                }
                float pr[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) pr[e] = exp2_approx(lg[e] - m_off);
                l_run += (pr[0] + pr[1]) + (pr[2] + pr[3]);
                constexpr int NT = Weights<T>::kTerms;
                uint32_t w0[NT], w1[NT];
                Weights<T>::split(pr[0], pr[1], w0);
                Weights<T>::split(pr[2], pr[3], w1);
                const uint32_t vb = kb + C::kPageBytes;
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    uint32_t f[4];
                    ldmatrix_x4_trans(f, vb + ((mchunk ^ (2 * i & 7)) << 4) + 128 * (i / 4));
                    if (valid < kPage) {                         // what lies behind the last token may be anything
                        f[0] &= vm0; f[1] &= vm0; f[2] &= vm1; f[3] &= vm1;
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t) mma16816<T>(o[i], f[0], f[1], f[2], f[3], w0[t], w1[t]);
                }
            }
            __syncwarp();                                        // every lane is done with the stage
            issue(stage, next_id, next_m);
            xl += C::kWarps;
            if (xl < x1) advance(p, ld, C::kWarps);
            next_id = page_id();
            next_m = ld.m;
            stage = stage + 1 == S ? 0 : stage + 1;
        }
        // ---- the warps' parts of this row
        l_run += __shfl_xor_sync(0xffffffffu, l_run, 1);
        l_run += __shfl_xor_sync(0xffffffffu, l_run, 2);
        float* mine = comb + warp * C::kComb;
        if (tig == 0) {
            mine[gid] = m_run;
            mine[8 + gid] = l_run;
        }
#pragma unroll
        for (int i = 0; i < KS; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                mine[16 + (2 * tig + (e & 1)) * C::kHeadStride + 16 * i + gid + 8 * (e >> 1)] = o[i][e];
        }
        __syncthreads();
        const bool whole = row_begin >= x0 && row_end <= x1;
        // a share has at most two rows that it does not finish: one that began before it, one that goes on behind it
        float* part = p.partials + (static_cast<int64_t>(blockIdx.x) * 2 + (xs == x0 ? 0 : 1)) * C::kPart;
        for (int i = tid; i < G * D; i += C::kThreads) {
            const int g = i / D, col = i % D;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < C::kWarps; ++w) M = fmaxf(M, comb[w * C::kComb + g]);
            const float Mu = M == -INFINITY ? 0.f : M;
            float L = 0.f, O = 0.f;
#pragma unroll
            for (int w = 0; w < C::kWarps; ++w) {
                const float f = exp2_approx(comb[w * C::kComb + g] - Mu);
                L = fmaf(comb[w * C::kComb + 8 + g], f, L);
                O = fmaf(comb[w * C::kComb + 16 + g * C::kHeadStride + col], f, O);
            }
            if (whole) {
                p.out[(row * G + g) * D + col] = L > 0.f ? O / L : 0.f;
            } else {
                part[16 + g * D + col] = O;
                if (col == 0) {
                    part[g] = M;
                    part[8 + g] = L;
                }
            }
        }
        __syncthreads();                                         // the next row's parts go to the same place
        advance(p, seg, seg.pages - seg.pg);
        xs = xe;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Joins the rows that lie in several shares: CTA (i, g) takes head g of the row that crosses from share i - 1 into
// share i, if that is the row's first crossing.  out = sum O 2^(m - M) / sum l 2^(m - M).
constexpr int kJoinThreads = 512;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) attend_pages_join_kernel(const AttendPagesParams p) {
    constexpr int kPart = PagesCfg<D>::kPart;
    constexpr int kSlices = kJoinThreads / D;
    constexpr int kBatch = 8;                            // parts a thread reads at a time
    __shared__ float s_o[kSlices][D];
    __shared__ float s_ml[kSlices][2];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t i = blockIdx.x + 1;
    const int g = blockIdx.y, tid = threadIdx.x, col = tid % D, slice = tid / D;
    const AttendPagesMeta m = p.meta[i];
    if (m.row < 0 || m.row_begin >= i * m.share || m.row_begin < (i - 1) * m.share) return;
    const int first = static_cast<int>(i - 1), last = static_cast<int>((m.row_end - 1) / m.share);
    // the row is the first share's second part unless that share begins with it
    const int slot = m.row_begin == (i - 1) * m.share ? 0 : 1;
    float M = -INFINITY, L = 0.f, O = 0.f;
    for (int k0 = first + slice; k0 <= last; k0 += kSlices * kBatch) {
        float mv[kBatch], lv[kBatch], ov[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int k = k0 + u * kSlices;
            const float* ps = p.partials + (static_cast<int64_t>(k <= last ? k : first) * 2 +
                                            ((k == first || k > last) ? slot : 0)) * kPart;
            mv[u] = k <= last ? __ldcg(ps + g) : -INFINITY;
            lv[u] = __ldcg(ps + 8 + g);
            ov[u] = __ldcg(ps + 16 + g * D + col);
        }
        float Mn = M;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) Mn = fmaxf(Mn, mv[u]);
        const float Mu = Mn == -INFINITY ? 0.f : Mn;
        const float c = exp2_approx(M - Mu);
        L *= c;
        O *= c;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const float f = exp2_approx(mv[u] - Mu);
            L = fmaf(lv[u], f, L);
            O = fmaf(ov[u], f, O);
        }
        M = Mn;
    }
    s_o[slice][col] = O;
    if (col == 0) {
        s_ml[slice][0] = M;
        s_ml[slice][1] = L;
    }
    __syncthreads();
    if (slice == 0) {
        float Mt = s_ml[0][0];
#pragma unroll
        for (int k = 1; k < kSlices; ++k) Mt = fmaxf(Mt, s_ml[k][0]);
        const float Mu = Mt == -INFINITY ? 0.f : Mt;
        float Lt = 0.f, Ot = 0.f;
#pragma unroll
        for (int k = 0; k < kSlices; ++k) {
            const float f = exp2_approx(s_ml[k][0] - Mu);
            Lt = fmaf(s_ml[k][1], f, Lt);
            Ot = fmaf(s_o[k][col], f, Ot);
        }
        p.out[(static_cast<int64_t>(m.row) * p.group + g) * D + col] = Lt > 0.f ? Ot / Lt : 0.f;
    }
}

}  // namespace dev
}  // namespace tq
