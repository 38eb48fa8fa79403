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

// Every kernel here is launched as a programmatic dependent of what precedes it in the stream.  It begins by waiting
// until all of that is complete and visible, and lets the kernel behind it be scheduled early (which waits in turn), so
// that a step's launches do not each add their latency.
__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void release_stream() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void begin_dependent() {
    wait_for_stream();
    release_stream();
}

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

constexpr int kPlanThreads = 1024;      // requests a CTA of plan_kernel plans at a time, at most
constexpr int kSlotTile = 256;         // tokens whose slots one CTA of plan_slots_kernel writes
constexpr int kSlotBatch = 2048;       // row starts it keeps in shared memory

// Inclusive scan of two values over the block (every thread takes part); `total` receives the block's sums.
template <int NT>
__device__ __forceinline__ void block_scan2(int64_t& a, int64_t& b, int64_t (&total)[2], int64_t (*warp_sums)[2]) {
    constexpr int NW = NT / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t ta = __shfl_up_sync(0xffffffffu, a, o), tb = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) { a += ta; b += tb; }
    }
    __syncthreads();                                     // warp_sums may still be read from the scan before
    if (lane == 31) { warp_sums[warp][0] = a; warp_sums[warp][1] = b; }
    __syncthreads();
    // every warp adds up the warps before it
    int64_t sa = lane < NW ? warp_sums[lane][0] : 0, sb = lane < NW ? warp_sums[lane][1] : 0;
    int64_t ba = lane < warp ? sa : 0, bb = lane < warp ? sb : 0;
#pragma unroll
    for (int o = (NW > 16 ? 16 : NW / 2); o; o >>= 1) {
        sa += __shfl_xor_sync(0xffffffffu, sa, o);
        sb += __shfl_xor_sync(0xffffffffu, sb, o);
        ba += __shfl_xor_sync(0xffffffffu, ba, o);
        bb += __shfl_xor_sync(0xffffffffu, bb, o);
    }
    a += __shfl_sync(0xffffffffu, ba, 0);
    b += __shfl_sync(0xffffffffu, bb, 0);
    total[0] = __shfl_sync(0xffffffffu, sa, 0);
    total[1] = __shfl_sync(0xffffffffu, sb, 0);
}

// The slot of kv head 0 of a page's row, -1 if the id names no page.
__device__ __forceinline__ int64_t page_slot(const PlanParams& p, int page, int64_t pos) {
    return (page < 0 || page >= p.num_pages) ? -1 : static_cast<int64_t>(page) * p.heads * kPage + pos % kPage;
}

// One CTA: lengths, admission, table rows and the free ring; with_slots: the slots too.  Admission is a prefix rule (a
// request that needs pages gets them when the running sum of needs up to it is within the free count), so two scans
// decide it for every request at once.  Pages are taken from the ring's start and given back at its end, so what this
// call reads and what it writes never overlap, and a request's slots follow from its table row as it was and from its
// part of the ring, without waiting for the table.
template <int NT>
__global__ void __launch_bounds__(NT) plan_kernel(const PlanParams p, bool with_slots) {
    __shared__ int64_t s_warp[NT / 32][2];
    __shared__ int s_len[NT], s_need[NT], s_from[NT], s_gone[NT], s_to[NT], s_req[NT];
    __shared__ int64_t s_row[NT];
    __shared__ int s_taken;
    begin_dependent();
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
    for (int b0 = 0; b0 < p.batch; b0 += NT) {
        const int b = b0 + tid;
        const bool active = b < p.batch;
        const int want = active ? p.new_lens[b] : 0;
        int64_t len = active ? p.seq_lens[b] : 0;
        len = len < 0 ? 0 : (len > most ? most : len);
        const int64_t req = want > 0 ? want : 0;
        const int64_t old_pages = (len + kPage - 1) / kPage;
        const int64_t gone = want < 0 ? old_pages : 0;
        int64_t end = req, gone_end = gone;
        block_scan2<NT>(end, gone_end, total, s_warp);
        end += rows_before;
        gone_end += gone_before;
        rows_before += total[0];
        gone_before += total[1];
        const bool fits = active && want >= 0 && len + req <= most && end <= p.max_tokens;
        const int64_t need = fits ? (len + req + kPage - 1) / kPage - old_pages : 0;
        int64_t upto = need, unused = 0;
        block_scan2<NT>(upto, unused, total, s_warp);
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
        s_len[tid] = ok ? static_cast<int>(len) : ~static_cast<int>(old_pages);     // refused: the pages it has
        s_need[tid] = ok ? static_cast<int>(need) : 0;
        s_from[tid] = ok ? static_cast<int>(upto - need) : 0;
        s_gone[tid] = static_cast<int>(gone);
        s_to[tid] = to > cap ? cap : static_cast<int>(to);
        s_req[tid] = static_cast<int>(req);
        s_row[tid] = end - req;
        __syncthreads();
        // table rows, ring and slots: the block's threads in equal groups, a request per group
        const int n = p.batch - b0 < NT ? p.batch - b0 : NT;
        int per = NT;
        while (per > 1 && per * n > NT) per >>= 1;
        const int lane = tid & (per - 1);
        for (int i = tid / per; i < n; i += NT / per) {
            int32_t* row = p.table + static_cast<int64_t>(b0 + i) * p.width;
            const int need_i = s_need[i], gone_i = s_gone[i], len_i = s_len[i];
            const int old = len_i < 0 ? ~len_i : (len_i + kPage - 1) / kPage;
            const int from = head + s_from[i];           // below 2 cap: from + j - head < count <= cap
            auto fresh = [&](int j) { return p.ring[from + j >= cap ? from + j - cap : from + j]; };
#pragma unroll 4
            for (int j = lane; j < need_i; j += per) row[old + j] = fresh(j);
            const int64_t to_i = static_cast<int64_t>(count) + s_to[i];
            for (int j = lane; j < gone_i && to_i + j < cap; j += per) {
                const int at = static_cast<int>(to_i + j) - (cap - head);
                p.ring[at < 0 ? at + cap : at] = row[j];
            }
            if (with_slots) {
                // rows past max_tokens belong to requests that were refused
                const int64_t left = p.max_tokens - s_row[i];
                const int rows = static_cast<int>(left < 0 ? 0 : (s_req[i] < left ? s_req[i] : left));
                int64_t* dst = p.slots + s_row[i] * p.heads;
                for (int e = lane; e < rows * p.heads; e += per) {
                    const int t = e / p.heads;
                    int64_t slot = -1;
                    if (len_i >= 0) {
                        const int64_t pos = static_cast<int64_t>(len_i) + t;
                        const int pg = static_cast<int>(pos / kPage);
                        slot = page_slot(p, pg < old ? row[pg] : fresh(pg - old), pos);
                    }
                    dst[e] = slot < 0 ? -1 : slot + (e - t * p.heads) * kPage;
                }
            }
        }
        __syncthreads();
    }
    if (with_slots) {                                    // input rows behind the last request's
        for (int64_t e = rows_before * p.heads + tid; e < p.max_tokens * p.heads; e += NT) p.slots[e] = -1;
    }
    if (tid == 0) {
        const int taken = s_taken;
        const int64_t room = cap - count;
        const int back = static_cast<int>(gone_before < room ? gone_before : room);
        const int next = head + taken;
        p.state_out[0] = next >= cap ? next - cap : next;
        p.state_out[1] = count - taken + back;
    }
}

// Slots of larger calls, after plan_kernel: one CTA per kSlotTile input rows, one search per token for its request
// (in shared memory up to kSlotBatch requests), then the tokens' H_kv slots with coalesced stores.
__global__ void __launch_bounds__(kSlotTile) plan_slots_kernel(const PlanParams p) {
    __shared__ int64_t s_base[kSlotTile];
    __shared__ int s_ends[kSlotBatch];
    begin_dependent();
    const int tid = threadIdx.x;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kSlotTile;
    const int n = static_cast<int>(p.max_tokens - t0 < kSlotTile ? p.max_tokens - t0 : kSlotTile);
    const int* ends = p.row_start + 1;
    if (p.batch <= kSlotBatch) {
        for (int i = tid; i < p.batch; i += kSlotTile) s_ends[i] = ends[i];
        __syncthreads();
        ends = s_ends;
    }
    int64_t base = -1;
    if (tid < n) {
        const int64_t token = t0 + tid;
        int lo = 0, hi = p.batch;                        // the first request whose rows end after `token`
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (ends[mid] <= token) lo = mid + 1; else hi = mid;
        }
        if (lo < p.batch) {
            const int start = p.start_pos[lo];
            const int64_t pos = start + (token - (lo ? ends[lo - 1] : 0));
            if (start >= 0) base = page_slot(p, p.table[static_cast<int64_t>(lo) * p.width + pos / kPage], pos);
        }
    }
    s_base[tid] = base;
    __syncthreads();
    int64_t* dst = p.slots + t0 * p.heads;
    for (int i = tid; i < n * p.heads; i += kSlotTile) {
        const int t = i / p.heads, h = i - t * p.heads;
        dst[i] = s_base[t] < 0 ? -1 : s_base[t] + h * kPage;
    }
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
template <int W> union Words32 {
    typename Words<W>::type vec;
    uint32_t w[W];
};

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
// on the order of warps.  A lane holds d / 32 channels of a row.  VALUES: there is a value pool.
template <typename T, int D, bool VALUES>
__global__ void __launch_bounds__(32 * kAppendWarps, D == 256 && VALUES ? 2 : 3) append_kernel(const AppendParams p) {
    constexpr int W = D / 64;                            // words per lane and row
    constexpr int kBatch = 8;                            // rows in flight
    using Vec = typename Words<W>::type;
    const int lane = threadIdx.x & 31;
    begin_dependent();
    const int64_t gw = static_cast<int64_t>(blockIdx.x) * kAppendWarps + (threadIdx.x >> 5);
    const int h = static_cast<int>(gw % p.heads);
    const int64_t t0 = gw / p.heads * p.tile;
    if (t0 >= p.n) return;
    const T* k = static_cast<const T*>(p.k) + h * p.k_head + lane * 2 * W;
    const T* v = static_cast<const T*>(p.v) + h * p.v_head + lane * 2 * W;
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
        bool first = true;
        T* k_pool = static_cast<T*>(p.k_pool) + run * (kPage * D) + lane * 2 * W;
        T* v_pool = static_cast<T*>(p.v_pool) + run * (kPage * D) + lane * 2 * W;
        Words32<W> lo, hi, old_lo, old_hi;
        while (true) {
            const int len = ~same ? __ffs(~same) - 1 : 32;
            const unsigned mask = (len >= 32 ? 0xffffffffu : ((1u << len) - 1u)) << at;
            fresh |= (__ballot_sync(0xffffffffu, ws >= 0 && ws % kPage == 0) & mask) != 0;
            for (int j0 = 0; j0 < len; j0 += kBatch) {
                Words32<W> kr[kBatch], vr[VALUES ? kBatch : 1];
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    if (j0 + u < len) {
                        kr[u].vec = *reinterpret_cast<const Vec*>(k + (token + j0 + u) * p.k_token);
                        if constexpr (VALUES) vr[u].vec = *reinterpret_cast<const Vec*>(v + (token + j0 + u) * p.v_token);
                    }
                }
                if (first) {                             // the old bounds come with the first rows
                    if (p.bounds && !fresh) {
                        const T* b = static_cast<const T*>(p.bounds) + run * 2 * D + lane * 2 * W;
                        old_lo.vec = *reinterpret_cast<const Vec*>(b);
                        old_hi.vec = *reinterpret_cast<const Vec*>(b + D);
                    } else {
                        old_lo = kr[0];
                        old_hi = kr[0];
                    }
                    lo = kr[0];
                    hi = kr[0];
                    first = false;
                }
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    // the run's rows lie in one page: a slot is the page's first plus 0 .. 15
                    const int s = __shfl_sync(0xffffffffu, static_cast<int>(ws) & (kPage - 1), (at + j0 + u) & 31) * D;
                    if (j0 + u < len) {
                        if (p.k_pool) *reinterpret_cast<Vec*>(k_pool + s) = kr[u].vec;
                        if constexpr (VALUES) *reinterpret_cast<Vec*>(v_pool + s) = vr[u].vec;
#pragma unroll
                        for (int i = 0; i < W; ++i) {
                            lo.w[i] = min2<T>(lo.w[i], kr[u].w[i]);
                            hi.w[i] = max2<T>(hi.w[i], kr[u].w[i]);
                        }
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
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    lo.w[i] = min2<T>(lo.w[i], old_lo.w[i]);
                    hi.w[i] = max2<T>(hi.w[i], old_hi.w[i]);
                }
            }
            *reinterpret_cast<Vec*>(b) = lo.vec;
            *reinterpret_cast<Vec*>(b + D) = hi.vec;
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
    int tile;                          // pages a CTA of score_kernel scores
    int room;                          // pages whose keys (and, unless SCORED, ids) select_kernel's shared memory holds
    uint32_t* keys;                    // [B][H_kv][width]: keys of score_kernel (select_kernel's SCORED form)
};

constexpr int kScoreThreads = 256;     // threads that score pages together: a CTA of score_kernel, or of select_kernel
constexpr int kScoreTile = 256;        // pages a CTA of score_kernel scores, at most
constexpr int kSortThreads = 1024;     // threads of select_kernel's SCORED form

inline __host__ __device__ size_t query_smem(int group, int d) { return static_cast<size_t>(group) * d * 8; }

// The query's heads of one kv head as max(q, 0) and min(q, 0) in shared memory, [G][2][d / 8][4]: lane l of a group
// finds its channels 8 l .. 8 l + 7 in two 16-byte words without bank conflicts.
template <typename T, int D>
__device__ __forceinline__ void load_query(const SelectParams& p, int b, int h, float* qp, float* qn) {
    const T* q = static_cast<const T*>(p.q) + b * p.q_stride + static_cast<int64_t>(h) * p.group * D;
    for (int i = threadIdx.x; i < p.group * D; i += kScoreThreads) {
        const float x = static_cast<float>(q[i]);
        const int g = i / D, c = i % D;
        const int at = g * D + (c % 8 / 4) * (D / 2) + c / 8 * 4 + c % 4;
        qp[at] = fmaxf(x, 0.f);
        qn[at] = fminf(x, 0.f);
    }
}

// One round of scoring: keys (order-preserving bits of the scores) of pages base .. base + U - 1 for each lane group of
// d / 8 lanes, of the cnt pages from p0 on of a row of nb pages.  lo16, hi16: this lane's 8 channels of the bounds.
//
// The score of a page is max over the group's query heads of U_g = sum_c max(q_gc lo_c, q_gc hi_c), which is at least
// q_g . k for every key in the page.  With lo <= hi the larger product is (q > 0 ? q hi : q lo), computed as two
// fused multiply-adds of max(q, 0) with hi and min(q, 0) with lo: one of the products is a zero, and products of
// 16-bit values are exact in fp32, so each step is a plain rounded addition.  The order of additions is part of the
// operator (a lane's 8 channels as an even and an odd chain, then lanes i and i + half), so that the choice of pages
// can be reproduced bit for bit; it also rules out the tensor cores, whose order is not defined.
template <typename T, int D, int U>
__device__ __forceinline__ void score_round(const SelectParams& p, const float4* qp4, const float4* qn4, const uint4 (&lo16)[U],
                                            const uint4 (&hi16)[U], int nb, int p0, int cnt, int base, const int32_t* ids,
                                            uint32_t* keys) {
    constexpr int LP = D / 8;                            // lanes per page
    static_assert(U == 2 || U == 4, "the reduction below spreads two or four pages over the lanes of a group");
    constexpr int kHeads = U == 4 ? 2 : 1;               // heads in flight: one's products run under the other's shuffles
    const int l = threadIdx.x % LP;
    const bool upper = (l & (LP / 2)) != 0, odd = (l & (LP / 4)) != 0;
    float2 lo[U][4], hi[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t aw[4] = {lo16[u].x, lo16[u].y, lo16[u].z, lo16[u].w};
        const uint32_t cw[4] = {hi16[u].x, hi16[u].y, hi16[u].z, hi16[u].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[u][i] = Pair<T>::floats(aw[i]);
            hi[u][i] = Pair<T>::floats(cw[i]);
        }
    }
    float best = -INFINITY;
#pragma unroll kHeads
    for (int g = 0; g < p.group; ++g) {
        const float4 p0v = qp4[g * (D / 4)], p1v = qp4[g * (D / 4) + LP];
        const float4 n0v = qn4[g * (D / 4)], n1v = qn4[g * (D / 4) + LP];
        const float2 pq[4] = {{p0v.x, p0v.y}, {p0v.z, p0v.w}, {p1v.x, p1v.y}, {p1v.z, p1v.w}};
        const float2 nq[4] = {{n0v.x, n0v.y}, {n0v.z, n0v.w}, {n1v.x, n1v.y}, {n1v.z, n1v.w}};
        float v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float2 acc = __fmul2_rn(pq[0], hi[u][0]);
            acc = __ffma2_rn(nq[0], lo[u][0], acc);
#pragma unroll
            for (int i = 1; i < 4; ++i) {
                acc = __ffma2_rn(pq[i], hi[u][i], acc);
                acc = __ffma2_rn(nq[i], lo[u][i], acc);
            }
            v[u] = acc.x + acc.y;
        }
        // lanes i and i + LP/2 add up, the upper half going on with one half of the pages and the lower with the
        // other; then quarters
        float s;
        if constexpr (U == 4) {
            const float k0 = upper ? v[2] : v[0], k1 = upper ? v[3] : v[1];
            const float g0 = upper ? v[0] : v[2], g1 = upper ? v[1] : v[3];
            const float w0 = k0 + __shfl_xor_sync(0xffffffffu, g0, LP / 2);
            const float w1 = k1 + __shfl_xor_sync(0xffffffffu, g1, LP / 2);
            s = (odd ? w1 : w0) + __shfl_xor_sync(0xffffffffu, odd ? w0 : w1, LP / 4);
        } else {
            s = (upper ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, upper ? v[0] : v[1], LP / 2);
            s += __shfl_xor_sync(0xffffffffu, s, LP / 4);
        }
#pragma unroll
        for (int o = LP / 8; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        // a sum that is not a number does not hide behind another head's
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(best) : "f"(s));
    }
    const int j = base + (U == 4 ? (upper ? 2 : 0) + (odd ? 1 : 0) : (upper ? 1 : 0));
    if ((l & (LP / U - 1)) == 0 && j < cnt) {
        const int at = p0 + j, id = ids[j];
        uint32_t bits = __float_as_uint(best + 0.f);                 // -0 counts as 0
        bits = (bits >> 31) ? ~bits : bits | 0x80000000u;
        if (best != best || id < 0 || id >= p.num_pages) bits = 0u;
        if (at < p.keep_first || at >= nb - p.keep_last) bits = 0xffffffffu;
        keys[j] = bits;
    }
}

__device__ __forceinline__ int64_t select_len(const SelectParams& p, int b) {
    const int64_t most = static_cast<int64_t>(p.width) * kPage, len = p.seq_lens[b];
    return len < 0 ? 0 : (len > most ? most : len);
}

// Keys of a call with few rows, where a CTA per row would leave most of the GPU idle: a CTA per row and kScoreTile
// pages.  Four pages per lane group share each read of the query from shared memory.  With the registers that takes
// there are 16 warps on an SM, too few to hide the loads, so each lane's next bounds are copied (cp.async) to a slot
// that only it reads while it works on the ones before.
template <int D>
constexpr int score_smem(int group) { return static_cast<int>(query_smem(group, D)) + 2 * 4 * 2 * 16 * kScoreThreads; }

template <typename T, int D>
__global__ void __launch_bounds__(kScoreThreads, 2) score_kernel(const SelectParams p) {
    constexpr int U = 4, LP = D / 8, GW = 32 / LP;
    constexpr int kRound = (kScoreThreads / 32) * GW * U;            // pages per round of the block
    extern __shared__ __align__(16) uint8_t smem[];
    float* qp = reinterpret_cast<float*>(smem);
    float* qn = qp + p.group * D;
    uint4* slots = reinterpret_cast<uint4*>(qn + p.group * D) + threadIdx.x;   // [2][U][lo, hi][threads]
    __shared__ int32_t s_ids[kScoreTile];
    static_assert(kScoreTile == kScoreThreads, "a thread per page id");
    begin_dependent();
    const int tiles = (p.width + p.tile - 1) / p.tile;
    const int row = blockIdx.x / tiles, b = row / p.heads, h = row - b * p.heads;
    const int64_t len = select_len(p, b);
    const int p0 = (blockIdx.x - row * tiles) * p.tile;
    load_query<T, D>(p, b, h, qp, qn);
    if (p0 + threadIdx.x < p.width) s_ids[threadIdx.x] = p.table[static_cast<int64_t>(b) * p.width + p0 + threadIdx.x];
    const int nb = static_cast<int>((len + kPage - 1) / kPage);
    if (p0 >= nb || nb <= p.budget) return;
    const int cnt = nb - p0 < p.tile ? nb - p0 : p.tile;
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LP;
    const float4* qp4 = reinterpret_cast<const float4*>(qp) + l;
    const float4* qn4 = reinterpret_cast<const float4*>(qn) + l;
    const T* bounds = static_cast<const T*>(p.bounds) + static_cast<int64_t>(h) * 2 * D + l * 8;
    const int64_t page_stride = static_cast<int64_t>(p.heads) * 2 * D;
    const int w0 = warp * GW * U;                        // the warp's first page of a round
    auto fetch = [&](int round) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = round * kRound + w0 + lane / LP * U + u;
            const int id = j < cnt ? s_ids[j] : -1;
            if (id >= 0 && id < p.num_pages) {           // else the slot's old contents are scored and not used
                const T* src = bounds + id * page_stride;
                const uint32_t dst = smem_u32(slots + (round & 1) * U * 2 * kScoreThreads + u * 2 * kScoreThreads);
                cp_async16(dst, src);
                cp_async16(dst + 16 * kScoreThreads, src + D);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    fetch(0);
    uint32_t* keys = p.keys + static_cast<int64_t>(row) * p.width + p0;
    for (int round = 0; round * kRound + w0 < cnt; ++round) {
        fetch(round + 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        uint4 lo[U], hi[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            lo[u] = slots[((round & 1) * U + u) * 2 * kScoreThreads];
            hi[u] = slots[((round & 1) * U + u) * 2 * kScoreThreads + kScoreThreads];
        }
        score_round<T, D, U>(p, qp4, qn4, lo, hi, nb, p0, cnt, round * kRound + w0 + lane / LP * U, s_ids, keys);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// The `budget` best pages of one (sequence, kv head), by one CTA.  SCORED: score_kernel has computed the keys; else the
// CTA computes its row's keys first, several CTAs to an SM so that one
// row's selection runs under another's loads.
//
// The choice is a radix selection: the keys' range is cut into 256 bins, the bin that holds the budget-th largest
// key is found and cut again, until it goes in whole or holds one value, whose ties go to the lowest page index.  The
// range starts at the smallest and largest score, not at the key's top bits, which all scores tend to share: two
// passes usually do, and few keys fall into one bin at a time.  Pages kept in any case do not take part.
template <typename T, int D, bool SCORED>
__global__ void __launch_bounds__(SCORED ? kSortThreads : kScoreThreads, SCORED ? 1 : 4) select_kernel(const SelectParams p) {
    constexpr int NT = SCORED ? kSortThreads : kScoreThreads;
    constexpr int NW = NT / 32;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ uint32_t s_hist[2][256];
    __shared__ uint32_t s_pick[3];
    __shared__ uint32_t s_warp[NW], s_warp2[NW];
    begin_dependent();
    const int row = blockIdx.x;
    const int b = row / p.heads, h = row - b * p.heads;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int32_t* table = p.table + static_cast<int64_t>(b) * p.width;
    const int64_t len = select_len(p, b);
    float* qp = reinterpret_cast<float*>(smem);
    float* qn = qp + p.group * D;
    uint32_t* room = reinterpret_cast<uint32_t*>(SCORED ? qp : qn + p.group * D);
    int32_t* ids = reinterpret_cast<int32_t*>(room + p.room);
    if constexpr (!SCORED) {                             // read while the length is on its way
        load_query<T, D>(p, b, h, qp, qn);
        for (int j = tid; j < p.width; j += NT) ids[j] = table[j];
    }
    if (tid < 256) s_hist[0][tid] = s_hist[1][tid] = 0;
    const int nb = static_cast<int>((len + kPage - 1) / kPage);
    int32_t* out = p.pages + static_cast<int64_t>(row) * p.budget;
    if (tid == 0) p.lens[row] = static_cast<int>(nb <= p.budget ? len : len - static_cast<int64_t>(nb - p.budget) * kPage);
    if (nb <= p.budget) {                                // every page is kept
        for (int j = tid; j < p.budget; j += NT) {
            const int id = j < nb ? table[j] : -1;
            out[j] = (id < 0 || id >= p.num_pages) ? -1 : id * p.heads + h;
        }
        return;
    }
    // Thread t looks after pages j0 .. j1 - 1.  Up to kHeld of them stay in registers; the keys of longer rows are read
    // again in every pass (from shared memory, or from L2 if they do not fit there).
    constexpr int kHeld = 8;
    const int chunk = (nb + NT - 1) / NT;
    const int j0 = tid * chunk < nb ? tid * chunk : nb, j1 = j0 + chunk < nb ? j0 + chunk : nb;
    const bool held = chunk <= kHeld;
    const uint32_t* keys = room;
    uint32_t key[kHeld];
    int id[kHeld];
    if constexpr (SCORED) {
        const uint32_t* src = p.keys + static_cast<int64_t>(row) * p.width;
        if (held || nb > p.room) {
            keys = src;
        } else {
#pragma unroll 4
            for (int j = tid; j < nb; j += NT) room[j] = __ldcg(src + j);
        }
    } else {
        __syncthreads();
        constexpr int U = 2, LP = D / 8, GW = 32 / LP;
        const int l = lane % LP;
        const T* bounds = static_cast<const T*>(p.bounds) + static_cast<int64_t>(h) * 2 * D + l * 8;
        const int64_t page_stride = static_cast<int64_t>(p.heads) * 2 * D;
        for (int w0 = warp * GW * U; w0 < nb; w0 += NW * GW * U) {
            const int base = w0 + lane / LP * U;
            uint4 lo[U], hi[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int id = base + u < nb ? ids[base + u] : -1;
                lo[u] = hi[u] = make_uint4(0u, 0u, 0u, 0u);
                if (id >= 0 && id < p.num_pages) {
                    lo[u] = __ldg(reinterpret_cast<const uint4*>(bounds + id * page_stride));
                    hi[u] = __ldg(reinterpret_cast<const uint4*>(bounds + id * page_stride + D));
                }
            }
            score_round<T, D, U>(p, reinterpret_cast<const float4*>(qp) + l, reinterpret_cast<const float4*>(qn) + l, lo, hi, nb,
                                 0, nb, base, ids, room);
        }
    }
    __syncthreads();
    if (held) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            key[i] = j0 + i < j1 ? (SCORED ? __ldcg(keys + j0 + i) : keys[j0 + i]) : 0u;
            id[i] = j0 + i < j1 ? (SCORED ? table[j0 + i] : ids[j0 + i]) : -1;
        }
    }
    auto each = [&](auto f) {                            // f(page, its key, its id if it is held) for the thread's pages
        if (held) {
#pragma unroll
            for (int i = 0; i < kHeld; ++i)
                if (j0 + i < j1) f(j0 + i, key[i], id[i]);
        } else {
            for (int j = j0; j < j1; ++j) f(j, keys[j], 0);
        }
    };
    // ---- the range of the keys that compete: pages c0 .. c1 - 1
    const int c0 = p.keep_first, c1 = nb - p.keep_last < j1 ? nb - p.keep_last : j1;
    uint32_t least = 0xffffffffu, most = 0u;
    each([&](int j, uint32_t k, int) {
        if (j >= c0 && j < c1) {
            least = min(least, k);
            most = max(most, k);
        }
    });
    least = __reduce_min_sync(0xffffffffu, least);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) {
        s_warp[warp] = least;
        s_warp2[warp] = most;
    }
    __syncthreads();
    least = __reduce_min_sync(0xffffffffu, lane < NW ? s_warp[lane] : 0xffffffffu);
    most = __reduce_max_sync(0xffffffffu, lane < NW ? s_warp2[lane] : 0u);
    // ---- the threshold: of the keys from `bound` to `bound` + 2^bits - 1, the `need` largest are in; all above are
    uint32_t need = static_cast<uint32_t>(p.budget - p.keep_first - p.keep_last);
    int bits = 32 - __clz(static_cast<int>(most - least));
    bool whole = need == 0;                              // everything from `bound` on is in
    uint32_t bound = need == 0 ? 0xffffffffu : least;    // (need 0: nothing but the pages kept in any case)
    for (int pass = 0; !whole; ++pass) {
        const int shift = bits > 8 ? bits - 8 : 0;
        const uint32_t width = bits == 32 ? 0xffffffffu : (1u << bits) - 1u;
        uint32_t* hist = s_hist[pass & 1];
        each([&](int j, uint32_t k, int) {
            if (j >= c0 && j < c1 && k - bound <= width) atomicAdd(&hist[(k - bound) >> shift], 1u);
        });
        __syncthreads();
        // thread t takes bin 255 - t, so that an inclusive scan counts the keys from the largest bin down
        uint32_t c = 0, incl = 0;
        if (tid < 256) {
            incl = c = hist[255 - tid];
            s_hist[(pass & 1) ^ 1][tid] = 0;             // for the next pass
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t t = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += t;
            }
            if (lane == 31) s_warp[warp] = incl;
        }
        __syncthreads();
        if (tid < 256) {
#pragma unroll
            for (int w = 0; w < 8; ++w) incl += w < warp ? s_warp[w] : 0u;
            if (incl >= need && incl - c < need) {       // one thread
                s_pick[0] = 255u - tid;
                s_pick[1] = incl - c;
                s_pick[2] = incl;
            }
        }
        __syncthreads();
        bound += s_pick[0] << shift;
        whole = s_pick[2] == need;
        need -= s_pick[1];
        bits = shift;
        if (shift == 0) break;
    }
    // ---- the list: keys from `from` on, and the first `need` of those equal to `bound`
    const uint32_t from = whole ? bound : bound + 1;     // bound < 2^32 - 1: that key is of pages kept in any case
    if (whole) need = 0;
    uint32_t n_in = 0, n_tie = 0;
    each([&](int, uint32_t k, int) {
        n_in += k >= from ? 1u : 0u;
        n_tie += k < from && k == bound ? 1u : 0u;
    });
    uint32_t in_before = n_in, ties_before = n_tie;      // in the threads before this one
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t a = __shfl_up_sync(0xffffffffu, in_before, o), t = __shfl_up_sync(0xffffffffu, ties_before, o);
        if (lane >= o) {
            in_before += a;
            ties_before += t;
        }
    }
    __syncthreads();                                     // the sums before have been read
    if (lane == 31) {
        s_warp[warp] = in_before;
        s_warp2[warp] = ties_before;
    }
    __syncthreads();
    in_before += __reduce_add_sync(0xffffffffu, lane < warp ? s_warp[lane] : 0u) - n_in;
    ties_before += __reduce_add_sync(0xffffffffu, lane < warp ? s_warp2[lane] : 0u) - n_tie;
    each([&](int j, uint32_t k, int page) {
        const bool in = k >= from, tie = !in && k == bound;
        if (in || (tie && ties_before < need)) {
            const int e = held ? page : (SCORED ? table[j] : ids[j]);
            out[in_before + (ties_before < need ? ties_before : need)] = (e < 0 || e >= p.num_pages) ? -1 : e * p.heads + h;
        }
        in_before += in ? 1u : 0u;
        ties_before += tie ? 1u : 0u;
    });
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
    struct AttendPagesMeta* meta;      // [CTAs], or [rows] if the join goes by rows
    int64_t q_stride, k_page, v_page;  // elements; *_page: from one page to the next
    int units, mult;                   // table rows, and kv heads that share a table row (1 for selections)
    int width, num_ids, heads, group;
    int min_share;                     // what a CTA takes at least
    bool direct;                       // one CTA per row: nothing is cut, nothing joined
    int rows_join;                     // rows (units * mult) if the join goes by rows, else 0
    int join_heads;                    // heads that one CTA of the join takes
    float scale_log2;
};

// What the join needs, of the row that a share starts in or, going by rows, of each row: the shares its pages lie in.
struct AttendPagesMeta {
    int row;                           // -1: nothing to join
    int first, last;
    int pad;
};

template <int D>
struct PagesCfg {
    static constexpr int kWarps = 4;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kPageBytes = kPage * D * 2;                 // one page of keys (or values) of a kv head
    // Pages of keys and values in flight per warp, 96 to 128 KB per SM.  More only lengthens the queues at the memory,
    // which SMs leave at different speeds while the shares are equal: 4, 3 and 3 pages at d = 64, 128 and 256 take
    // 50.6, 89.6 and 94.4 us where 2 take 48.0, 85.4 and 92.1 (64 ragged sequences, 131072 tokens, 64 selected pages).
    static constexpr int kStages = 2;
    static constexpr int kCtasPerSm = (D == 64) ? 3 : (D == 128) ? 2 : 1;
    static constexpr int kRing = kWarps * kStages * 2 * kPageBytes;
    // what a row costs besides its pages (its query, the joining of the warps' parts), in pages; a multiple of kWarps
    static constexpr int kRowCost = 8;
    static constexpr int kHeadStride = D + 4;                        // spreads the accumulator rows over the banks
    // floats per warp: m[8], l[8], O[G][D + 4].  What a group of fewer than 8 heads leaves free lets the join's CTAs
    // become resident before the last share is done.
    static constexpr __host__ __device__ int comb(int group) { return 16 + group * kHeadStride; }
    static constexpr int smem(int group) { return kRing + kWarps * comb(group) * 4; }
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

// A place on the flattened axis: units in order, the kv heads of a unit in order, and for each of these rows
// kRowCost places for the row itself, then its pages.  Units without a page take no place.  The host refuses tables
// whose axis could reach 2^31.
struct PageCursor {
    int x;                             // of page pg of row (unit, m)
    int unit, m, pg, pages;            // pages: of this unit
};

__device__ __forceinline__ int unit_len(const AttendPagesParams& p, int u) {
    const int t = p.lens[u], most = p.width * kPage;     // width < 2^27
    return t < 0 ? 0 : (t > most ? most : t);
}
__device__ __forceinline__ int unit_pages(const AttendPagesParams& p, int u) { return (unit_len(p, u) + kPage - 1) / kPage; }

// Moves on by n pages; past the last page the cursor stays behind the last unit.
template <int ROW_COST>
__device__ __forceinline__ void advance(const AttendPagesParams& p, PageCursor& c, int n) {
    c.pg += n;
    c.x += n;
    while (c.pg >= c.pages) {
        c.pg -= c.pages;
        c.x += ROW_COST;
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
// all pages of the call, in the order (table row, kv head, page), are cut into shares of equal cost, one per resident
// CTA, whatever the lengths of the sequences are.  A share covers parts of one or several rows (a row: one sequence
// and kv head with its query heads, whose own cost counts as kRowCost pages); a row that lies inside one share is
// finished there, and attend_pages_join_kernel joins the others.  Calls with short table rows take a CTA per row and
// need no join.  The running maximum and sum (fp32) make the split exact up to rounding.
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
    int* s_setup = reinterpret_cast<int*>(comb);         // used before the first row ends only
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gid = lane >> 2, tig = lane & 3;
    const int G = p.group;

    wait_for_stream();
    // ---- this CTA's share
    int x0 = 0, x1, share = INT_MAX;
    PageCursor seg;                                      // the first page at or behind x0
    auto write_zeros = [&]() {                           // rows without a token are nobody's page
        for (int u = blockIdx.x; u < p.units; u += gridDim.x) {
            if (unit_pages(p, u) == 0) {
                float* o = p.out + static_cast<int64_t>(u) * p.mult * G * D;
                for (int i = tid; i < p.mult * G * D; i += C::kThreads) o[i] = 0.f;
                if (p.rows_join)
                    for (int i = tid; i < p.mult; i += C::kThreads) p.meta[u * p.mult + i].row = -1;
            }
        }
    };
    if (p.direct) {
        seg.x = seg.pg = 0;
        seg.unit = blockIdx.x / p.mult;
        seg.m = blockIdx.x - seg.unit * p.mult;
        seg.pages = x1 = unit_pages(p, seg.unit);
        if (x1 == 0) {
            for (int i = tid; i < G * D; i += C::kThreads) p.out[static_cast<int64_t>(blockIdx.x) * G * D + i] = 0.f;
            return;
        }
    } else {
        // thread t looks at units t * per .. t * per + per - 1
        auto unit_cost = [&](int u) -> int {                 // of each of the unit's rows
            const int n = unit_pages(p, u);
            return n ? n + C::kRowCost : 0;
        };
        const int per = (p.units + C::kThreads - 1) / C::kThreads;
        const int u0 = tid * per, u1 = u0 + per < p.units ? u0 + per : p.units;
        int own = 0;
    #pragma unroll 4
        for (int u = u0; u < u1; ++u) own += unit_cost(u);
        int incl = own;
    #pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += t;
        }
        if (lane == 31) s_setup[warp] = incl;
        __syncthreads();
        int total = 0;
    #pragma unroll
        for (int w = 0; w < C::kWarps; ++w) {
            if (w < warp) incl += s_setup[w];
            total += s_setup[w];
        }
        total *= p.mult;
        share = (total + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
        if (share < p.min_share) share = p.min_share;
        // past the last share x0 may pass 2^31: unsigned
        const unsigned start = blockIdx.x * static_cast<unsigned>(share);
        if (start >= static_cast<unsigned>(total)) {
            if (!p.rows_join && tid == 0) p.meta[blockIdx.x].row = -1;
            write_zeros();
            return;
        }
        x0 = static_cast<int>(start);
        x1 = total - x0 < share ? total : x0 + share;
        {
            int begin = (incl - own) * p.mult;
            if (x0 >= begin && x0 < incl * p.mult) {         // one thread: its units are read again
                for (int u = u0; u < u1; ++u) {
                    const int cost = unit_cost(u), end = begin + cost * p.mult;
                    if (x0 < end) {
                        s_setup[C::kWarps] = u;
                        s_setup[C::kWarps + 1] = x0 - begin;
                        s_setup[C::kWarps + 2] = cost;
                        break;
                    }
                    begin = end;
                }
            }
        }
        __syncthreads();
        {
            const int off = s_setup[C::kWarps + 1], cost = s_setup[C::kWarps + 2];
            seg.unit = s_setup[C::kWarps];
            seg.pages = cost - C::kRowCost;
            seg.m = off / cost;
            const int in_row = off - seg.m * cost;
            seg.pg = in_row < C::kRowCost ? 0 : in_row - C::kRowCost;
            seg.x = x0 - in_row + C::kRowCost + seg.pg;
        }
        __syncthreads();                                     // the rows' results may overwrite the set-up words
    }

    // ---- the copy ring
    const T* k_pool = static_cast<const T*>(p.k_pool);
    const T* v_pool = static_cast<const T*>(p.v_pool);
    const uint32_t ring = smem_u32(smem) + warp * S * 2 * C::kPageBytes;
    constexpr int CR = D / 8;                            // chunks per row
    constexpr int kCopies = kPage * CR / 32;             // 16-byte copies per lane, page and tensor
    // warp w takes the pages whose place is w modulo kWarps
    auto first_of = [&](int x) { return (warp - x) & (C::kWarps - 1); };
    PageCursor ld = seg;                                 // the next page to be copied
    if (first_of(seg.x)) advance<C::kRowCost>(p, ld, first_of(seg.x));
    auto page_id = [&]() -> int {
        return ld.x < x1 ? __ldg(p.table + static_cast<int64_t>(ld.unit) * p.width + ld.pg) : -1;
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
            if (ld.x < x1) advance<C::kRowCost>(p, ld, C::kWarps);
        }
#pragma unroll
        for (int s = 0; s < S; ++s) issue(s, id[s], m[s]);
        next_id = page_id();
        next_m = ld.m;
    }
    // while the first pages are on their way
    if (!p.direct) write_zeros();
    if (!p.direct && !p.rows_join && tid == 0) {
        // the row that crosses into this share, if this is its first crossing
        const int row_begin = seg.x - seg.pg, first = row_begin / share;
        AttendPagesMeta m;
        m.row = row_begin < x0 && first == static_cast<int>(blockIdx.x) - 1 ? seg.unit * p.mult + seg.m : -1;
        m.first = first;
        m.last = (row_begin + seg.pages - 1) / share;
        m.pad = 0;
        p.meta[blockIdx.x] = m;
    }

    // ---- rows
    int stage = 0;
    const int mrow = (lane & 7) + ((lane >> 4) << 3);    // ldmatrix: matrices 0, 1 are rows 0-7, matrices 2, 3 rows 8-15
    const int mchunk = ((lane >> 3) & 1) ^ (lane & 7);   // and matrices 1, 3 the odd 16-byte chunk
    while (seg.x < x1) {
        const int len = unit_len(p, seg.unit);
        const int row = seg.unit * p.mult + seg.m;
        const int row_begin = seg.x - seg.pg, row_end = row_begin + seg.pages;
        const int xe = row_end < x1 ? row_end : x1;
        uint32_t qa[KS][2];
        {
            const int b = row / p.heads, h = row - b * p.heads;
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
        for (int x = seg.x + first_of(seg.x); x < xe; x += C::kWarps) {
            asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
            __syncwarp();
            const int left = len - (x - row_begin) * kPage;
            const int valid = left < kPage ? left : kPage;
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
            if (ld.x < x1) advance<C::kRowCost>(p, ld, C::kWarps);
            next_id = page_id();
            next_m = ld.m;
            stage = stage + 1 == S ? 0 : stage + 1;
        }
        // ---- the warps' parts of this row
        l_run += __shfl_xor_sync(0xffffffffu, l_run, 1);
        l_run += __shfl_xor_sync(0xffffffffu, l_run, 2);
        const int kComb = C::comb(G);
        float* mine = comb + warp * kComb;
        if (tig == 0) {
            mine[gid] = m_run;
            mine[8 + gid] = l_run;
        }
#pragma unroll
        for (int i = 0; i < KS; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (2 * tig + (e & 1) < G)
                    mine[16 + (2 * tig + (e & 1)) * C::kHeadStride + 16 * i + gid + 8 * (e >> 1)] = o[i][e];
        }
        __syncthreads();
        const bool whole = row_begin >= x0 && row_end <= x1;
        // a share has at most two rows that it does not finish: one that began before it, one that goes on behind it
        float* part = p.partials + (static_cast<int64_t>(blockIdx.x) * 2 + (row_begin < x0 ? 0 : 1)) * C::kPart;
        if (p.rows_join && tid == 0 && row_begin >= x0) {        // the row begins here
            AttendPagesMeta m;
            m.row = whole ? -1 : row;
            m.first = blockIdx.x;
            m.last = (row_end - 1) / share;
            m.pad = 0;
            p.meta[row] = m;
        }
        for (int i = tid; i < G * D; i += C::kThreads) {
            const int g = i / D, col = i % D;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < C::kWarps; ++w) M = fmaxf(M, comb[w * kComb + g]);
            const float Mu = M == -INFINITY ? 0.f : M;
            float L = 0.f, O = 0.f;
#pragma unroll
            for (int w = 0; w < C::kWarps; ++w) {
                const float f = exp2_approx(comb[w * kComb + g] - Mu);
                L = fmaf(comb[w * kComb + 8 + g], f, L);
                O = fmaf(comb[w * kComb + 16 + g * C::kHeadStride + col], f, O);
            }
            if (whole) {
                p.out[(static_cast<int64_t>(row) * G + g) * D + col] = L > 0.f ? O / L : 0.f;
            } else {
                part[16 + g * D + col] = O;
                if (col == 0) {
                    part[g] = M;
                    part[8 + g] = L;
                }
            }
        }
        __syncthreads();                                         // the next row's parts go to the same place
        advance<C::kRowCost>(p, seg, seg.pages - seg.pg);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    // only now: CTAs of the kernel behind this one that wait on an SM keep others of this grid's size from fitting when
    // calls follow one another (64 ragged sequences at d = 64: 59.9 us with the release at the start, 50.6 us here)
    release_stream();
}

// Joins the rows that lie in several shares.  out = sum O 2^(m - M) / sum l 2^(m - M).  With no more rows than shares
// CTA x takes row x, else the row that crosses from share x into share x + 1 if that is the row's first crossing; CTA y
// takes heads y * join_heads ... A thread has four columns of a head; slices of the block take every so-manieth part
// and are added up at the end.
constexpr int kJoinThreads = 256;      // at most

template <int D>
__global__ void __launch_bounds__(kJoinThreads, 4) attend_pages_join_kernel(const AttendPagesParams p) {
    constexpr int kPart = PagesCfg<D>::kPart;
    constexpr int kBatch = 8;                            // parts a thread reads at a time
    __shared__ float4 s_o[kJoinThreads];
    __shared__ float2 s_ml[kJoinThreads];
    wait_for_stream();
    const AttendPagesMeta m = p.meta[p.rows_join ? blockIdx.x : blockIdx.x + 1];
    if (m.row < 0) return;
    const int g0 = blockIdx.y * p.join_heads;
    const int heads = p.group - g0 < p.join_heads ? p.group - g0 : p.join_heads;
    const int items = heads * (D / 4), slices = blockDim.x / items;
    const int tid = threadIdx.x, slice = tid / items, item = tid - slice * items;
    const int g = g0 + item / (D / 4), c = item % (D / 4) * 4;
    const int first = m.first, last = m.last;
    float M = -INFINITY, L = 0.f;
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = slice < slices ? first + slice : last + 1; k0 <= last; k0 += slices * kBatch) {
        float mv[kBatch], lv[kBatch];
        float4 ov[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            // the row is the second unfinished one of the share it begins in, and the first of the others
            const int k = k0 + u * slices <= last ? k0 + u * slices : k0;
            const float* ps = p.partials + (static_cast<int64_t>(k) * 2 + (k == first ? 1 : 0)) * kPart;
            mv[u] = k0 + u * slices <= last ? __ldcg(ps + g) : -INFINITY;
            lv[u] = __ldcg(ps + 8 + g);
            ov[u] = __ldcg(reinterpret_cast<const float4*>(ps + 16 + g * D + c));
        }
        float Mn = M;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) Mn = fmaxf(Mn, mv[u]);
        const float Mu = Mn == -INFINITY ? 0.f : Mn;
        float f = exp2_approx(M - Mu);
        L *= f;
        O.x *= f; O.y *= f; O.z *= f; O.w *= f;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            f = exp2_approx(mv[u] - Mu);                 // 0 for what is read twice
            L = fmaf(lv[u], f, L);
            O.x = fmaf(ov[u].x, f, O.x);
            O.y = fmaf(ov[u].y, f, O.y);
            O.z = fmaf(ov[u].z, f, O.z);
            O.w = fmaf(ov[u].w, f, O.w);
        }
        M = Mn;
    }
    s_o[tid] = O;
    s_ml[tid] = make_float2(M, L);
    __syncthreads();
    if (slice == 0) {
        for (int k = 1; k < slices; ++k) M = fmaxf(M, s_ml[k * items + item].x);
        const float Mu = M == -INFINITY ? 0.f : M;
        L = 0.f;
        O = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < slices; ++k) {
            const float2 ml = s_ml[k * items + item];
            const float4 o = s_o[k * items + item];
            const float f = exp2_approx(ml.x - Mu);
            L = fmaf(ml.y, f, L);
            O.x = fmaf(o.x, f, O.x);
            O.y = fmaf(o.y, f, O.y);
            O.z = fmaf(o.z, f, O.z);
            O.w = fmaf(o.w, f, O.w);
        }
        const float r = L > 0.f ? 1.f / L : 0.f;
        O.x *= r; O.y *= r; O.z *= r; O.w *= r;
        *reinterpret_cast<float4*>(p.out + (static_cast<int64_t>(m.row) * p.group + g) * D + c) = O;
    }
}

}  // namespace dev
}  // namespace tq
