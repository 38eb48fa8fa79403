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
// that a step's launches do not each add their latency.  What it reads may be written while it is already resident, so it
// loads nothing through the non-coherent path, which is for data that is read-only as long as the grid lives.
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
    int tile;                          // tokens of a CTA of plan_slots_ahead_kernel
    bool apart;                        // its first CTA does what plan_beside_kernel does otherwise
};

constexpr int kPlanThreads = 1024;      // requests a CTA of plan_kernel plans at a time, at most
constexpr int kSlotTile = 256;         // threads of the slots' kernels, and tokens they take at a time
constexpr int kSlotTiles = 2;          // times that, at most, for a CTA of plan_slots_ahead_kernel
constexpr int kSlotBatch = 2048;       // row starts it keeps in shared memory
constexpr int kCopies = 8;             // page ids a thread of plan_kernel moves at a time

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

// Admission is a prefix rule (a request that needs pages gets them when the running sum of needs up to it is within the
// free count), so two scans decide it for every request at once.  Pages are taken from the ring's start and given back at
// its end, so what a call reads of table and ring and what it writes there never overlap, and a request's slots follow
// from its table row as it was and from its part of the ring, without waiting for the table.
struct FreeRing {
    int head, count;
    __device__ explicit FreeRing(const PlanParams& p) : head(p.state[0]), count(p.state[1]) {
        head = (head < 0 || head >= p.num_pages) ? 0 : head;
        count = count < 0 ? 0 : (count > p.num_pages ? p.num_pages : count);
    }
    // the j-th page of those that are taken (j < count <= num_pages)
    __device__ __forceinline__ int page(const PlanParams& p, int j) const {
        return p.ring[head + j >= p.num_pages ? head + j - p.num_pages : head + j];
    }
};

struct PlannedRequest {
    bool active, finished, ok;
    int64_t len, req, old_pages, end;                    // end: of its input rows
    int64_t need, upto;                                  // pages it takes, and the needs up to and including it
    int64_t gone, gone_end;                              // pages it gives back, and those up to and including it
};

struct PlanSums { int64_t rows = 0, gone = 0, need = 0; };           // of the requests before

// Request b0 + threadIdx.x, by the whole block.
template <int NT>
__device__ __forceinline__ PlannedRequest plan_request(const PlanParams& p, int b0, int count, PlanSums& before,
                                                       int64_t (*warp_sums)[2]) {
    const int64_t most = static_cast<int64_t>(p.width) * kPage;
    const int b = b0 + threadIdx.x;
    PlannedRequest r;
    r.active = b < p.batch;
    const int want = r.active ? p.new_lens[b] : 0;
    const int64_t len = r.active ? p.seq_lens[b] : 0;
    r.finished = want < 0;
    r.len = len < 0 ? 0 : (len > most ? most : len);
    r.req = want > 0 ? want : 0;
    r.old_pages = (r.len + kPage - 1) / kPage;
    r.gone = r.finished ? r.old_pages : 0;
    r.end = r.req;
    r.gone_end = r.gone;
    int64_t total[2];
    block_scan2<NT>(r.end, r.gone_end, total, warp_sums);
    r.end += before.rows;
    r.gone_end += before.gone;
    before.rows += total[0];
    before.gone += total[1];
    const bool fits = r.active && !r.finished && r.len + r.req <= most && r.end <= p.max_tokens;
    r.need = fits ? (r.len + r.req + kPage - 1) / kPage - r.old_pages : 0;
    int64_t unused = 0;
    r.upto = r.need;
    block_scan2<NT>(r.upto, unused, total, warp_sums);
    r.upto += before.need;
    before.need += total[0];
    r.ok = fits && (r.need == 0 || r.upto <= count);
    return r;
}

// The first of n requests whose rows (or pages) end after `token`.
__device__ __forceinline__ int request_of(const int* ends, int n, int64_t token) {
    int lo = 0;
    while (lo < n) {
        const int mid = (lo + n) >> 1;
        if (ends[mid] <= token) lo = mid + 1; else n = mid;
    }
    return lo;
}

__device__ __forceinline__ int plan_len(const PlannedRequest& r) {   // after the step
    return r.finished ? 0 : static_cast<int>(r.len + (r.ok ? r.req : 0));
}
__device__ __forceinline__ void write_rows(const PlanParams& p, int b, const PlannedRequest& r) {
    p.row_start[b + 1] = r.end > INT_MAX ? INT_MAX : static_cast<int>(r.end);
    p.start_pos[b] = r.ok ? static_cast<int>(r.len) : -1;
}
__device__ __forceinline__ void write_state(const PlanParams& p, const FreeRing& ring, int taken, int64_t gone) {
    const int room = p.num_pages - ring.count, next = ring.head + taken;
    p.state_out[0] = next >= p.num_pages ? next - p.num_pages : next;
    p.state_out[1] = ring.count - taken + static_cast<int>(gone < room ? gone : room);
}

// One CTA: lengths, admission, the free ring and table rows; SLOTS: the slots too.
template <int NT, bool SLOTS>
__global__ void __launch_bounds__(NT) plan_kernel(const PlanParams p) {
    __shared__ int64_t s_warp[NT / 32][2];
    __shared__ int s_len[NT], s_need[NT], s_from[NT], s_gone[NT], s_to[NT], s_req[NT];
    __shared__ int64_t s_row[NT];
    __shared__ int s_taken;
    begin_dependent();
    const int tid = threadIdx.x;
    const int cap = p.num_pages;
    const FreeRing ring(p);
    const int head = ring.head, count = ring.count;
    if (tid == 0) {
        s_taken = 0;
        p.row_start[0] = 0;
    }
    PlanSums sums;
    for (int b0 = 0; b0 < p.batch; b0 += NT) {
        const PlannedRequest r = plan_request<NT>(p, b0, count, sums, s_warp);
        if (r.ok && r.need > 0) atomicMax(&s_taken, static_cast<int>(r.upto));
        if (r.active) {
            write_rows(p, b0 + tid, r);
            p.seq_lens_out[b0 + tid] = plan_len(r);
        }
        const int64_t to = r.gone_end - r.gone;
        s_len[tid] = r.ok ? static_cast<int>(r.len) : ~static_cast<int>(r.old_pages);     // refused: the pages it has
        s_need[tid] = r.ok ? static_cast<int>(r.need) : 0;
        s_from[tid] = r.ok ? static_cast<int>(r.upto - r.need) : 0;
        s_gone[tid] = static_cast<int>(r.gone);
        s_to[tid] = to > cap ? cap : static_cast<int>(to);
        s_req[tid] = static_cast<int>(r.req);
        s_row[tid] = r.end - r.req;
        __syncthreads();
        // table rows, ring and slots: the block's threads in equal groups, a request per group
        const int n = p.batch - b0 < NT ? p.batch - b0 : NT;
        int per = NT;
        while (per > 1 && per * n > NT) per >>= 1;
        const int lane = tid & (per - 1);
        for (int i = tid / per; i < n; i += NT / per) {
            int32_t* row = p.table + static_cast<int64_t>(b0 + i) * p.width;
            const int need_i = s_need[i], gone_i = s_gone[i], len_i = s_len[i], from = s_from[i];
            const int old = len_i < 0 ? ~len_i : (len_i + kPage - 1) / kPage;
            // kCopies reads before the first write: nothing else tells the compiler that they do not overlap
            for (int j0 = lane; j0 < need_i; j0 += per * kCopies) {
                int id[kCopies];
#pragma unroll
                for (int u = 0; u < kCopies; ++u) id[u] = j0 + u * per < need_i ? ring.page(p, from + j0 + u * per) : 0;
#pragma unroll
                for (int u = 0; u < kCopies; ++u)
                    if (j0 + u * per < need_i) row[old + j0 + u * per] = id[u];
            }
            const int64_t to_i = static_cast<int64_t>(count) + s_to[i];
            const int back = gone_i < cap - to_i ? gone_i : static_cast<int>(cap - to_i);
            for (int j0 = lane; j0 < back; j0 += per * kCopies) {
                int id[kCopies];
#pragma unroll
                for (int u = 0; u < kCopies; ++u) id[u] = j0 + u * per < back ? row[j0 + u * per] : 0;
#pragma unroll
                for (int u = 0; u < kCopies; ++u) {
                    const int at = static_cast<int>(to_i + j0 + u * per) - (cap - head);
                    if (j0 + u * per < back) p.ring[at < 0 ? at + cap : at] = id[u];
                }
            }
            if constexpr (SLOTS) {
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
                        slot = page_slot(p, pg < old ? row[pg] : ring.page(p, from + pg - old), pos);
                    }
                    dst[e] = slot < 0 ? -1 : slot + (e - t * p.heads) * kPage;
                }
            }
        }
        __syncthreads();
    }
    if constexpr (SLOTS) {                    // input rows behind the last request's
        for (int64_t e = sums.rows * p.heads + tid; e < p.max_tokens * p.heads; e += NT) p.slots[e] = -1;
    }
    if (tid == 0) write_state(p, ring, s_taken, sums.gone);
}

// The slots of a CTA's n tokens from the first slot of each, with coalesced stores.
__device__ __forceinline__ void write_slots(const PlanParams& p, int64_t t0, int n, const int64_t* base) {
    int64_t* dst = p.slots + t0 * p.heads;
    const int t_step = kSlotTile / p.heads, h_step = kSlotTile - t_step * p.heads;
    int t = threadIdx.x / p.heads, h = threadIdx.x - t * p.heads;
    for (int i = threadIdx.x; i < n * p.heads; i += kSlotTile) {
        dst[i] = base[t] < 0 ? -1 : base[t] + h * kPage;
        t += t_step;
        h += h_step;
        if (h >= p.heads) {
            h -= p.heads;
            ++t;
        }
    }
}

// What plan_slots_ahead_kernel leaves of a call, by one CTA.  BESIDE: as a kernel of its own, which is launched behind that
// grid but runs beside it: that grid has waited for all before it, nothing that it writes is read here, and what it reads
// is overwritten when it is done.
template <bool BESIDE>
__device__ __forceinline__ void plan_rest(const PlanParams& p, int64_t (*s_warp)[2], int* s_gone) {
    __shared__ int s_taken;
    const int tid = threadIdx.x;
    const int cap = p.num_pages;
    const FreeRing ring(p);
    if (tid == 0) {
        s_taken = 0;
        p.row_start[0] = 0;
    }
    PlanSums sums;
    const PlannedRequest r = plan_request<kSlotTile>(p, 0, ring.count, sums, s_warp);
    if (r.ok && r.need > 0) atomicMax(&s_taken, static_cast<int>(r.upto));
    if (r.active) write_rows(p, tid, r);
    s_gone[tid] = r.gone_end > cap ? cap : static_cast<int>(r.gone_end);
    __syncthreads();
    // the pages given back, one after the other
    const int back = sums.gone < cap - ring.count ? static_cast<int>(sums.gone) : cap - ring.count;
    for (int j0 = tid; j0 < back; j0 += kSlotTile * kCopies) {
        int id[kCopies];
#pragma unroll
        for (int u = 0; u < kCopies; ++u) {
            const int j = j0 + u * kSlotTile;
            if (j < back) {
                const int b = request_of(s_gone, p.batch, j);
                id[u] = p.table[static_cast<int64_t>(b) * p.width + j - (b ? s_gone[b - 1] : 0)];
            }
        }
#pragma unroll
        for (int u = 0; u < kCopies; ++u) {
            const int j = j0 + u * kSlotTile, at = ring.count + j - (cap - ring.head);
            if (j < back) p.ring[at < 0 ? at + cap : at] = id[u];
        }
    }
    if constexpr (BESIDE) wait_for_stream();
    if (r.active) p.seq_lens_out[tid] = plan_len(r);
    if (tid == 0) write_state(p, ring, s_taken, sums.gone);
}

__global__ void __launch_bounds__(kSlotTile) plan_beside_kernel(const PlanParams p) {
    __shared__ int64_t s_warp[kSlotTile / 32][2];
    __shared__ int s_gone[kSlotTile];
    release_stream();
    plan_rest<true>(p, s_warp, s_gone);
}

// Slots and table rows of larger calls of up to kSlotTile requests, before the rest of the plan: a CTA per p.tile
// input rows that plans the whole batch for itself, which costs less than waiting for another kernel's plan (8 heads, 64
// requests of 64 tokens: 3.3 us, 8.1 with the slots behind the plan; 116736 tokens: 5.0 and 10.3, with one or four times
// kSlotTile rows to a CTA 5.4 and 5.8).  A new page is entered in its table row with its first token.
// If no output lies over an input (p.apart), the rest of the plan is the first CTA's (116736 tokens: 4.4 us).
__global__ void __launch_bounds__(kSlotTile) plan_slots_ahead_kernel(const PlanParams p) {
    __shared__ int64_t s_warp[kSlotTile / 32][2];
    __shared__ int64_t s_base[kSlotTile * kSlotTiles];
    __shared__ int s_ends[kSlotTile], s_len[kSlotTile], s_from[kSlotTile];
    begin_dependent();
    const int tid = threadIdx.x;
    if (p.apart && blockIdx.x == 0) {
        plan_rest<false>(p, s_warp, s_ends);
        return;
    }
    const int64_t t0 = static_cast<int64_t>(blockIdx.x - (p.apart ? 1 : 0)) * p.tile;
    const int n = static_cast<int>(p.max_tokens - t0 < p.tile ? p.max_tokens - t0 : p.tile);
    const FreeRing ring(p);
    PlanSums sums;
    const PlannedRequest r = plan_request<kSlotTile>(p, 0, ring.count, sums, s_warp);
    s_ends[tid] = r.end > INT_MAX ? INT_MAX : static_cast<int>(r.end);
    s_len[tid] = r.ok ? static_cast<int>(r.len) : -1;
    s_from[tid] = r.ok ? static_cast<int>(r.upto - r.need) : 0;
    __syncthreads();
    int at[kSlotTiles], id[kSlotTiles];           // all reads before the first write
    int64_t pos[kSlotTiles];
#pragma unroll
    for (int u = 0; u < kSlotTiles; ++u) {
        const int64_t token = t0 + u * kSlotTile + tid;
        id[u] = -1;
        pos[u] = 1;
        if (u * kSlotTile + tid < n) {
            const int b = request_of(s_ends, p.batch, token);
            const int len = b < p.batch ? s_len[b] : -1;
            if (len >= 0) {
                pos[u] = len + (token - (b ? s_ends[b - 1] : 0));
                const int pg = static_cast<int>(pos[u] / kPage), old = (len + kPage - 1) / kPage;
                at[u] = b;
                id[u] = pg < old ? p.table[static_cast<int64_t>(b) * p.width + pg] : ring.page(p, s_from[b] + pg - old);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < kSlotTiles; ++u) {
        if (pos[u] % kPage == 0) p.table[static_cast<int64_t>(at[u]) * p.width + pos[u] / kPage] = id[u];   // a new page
        s_base[u * kSlotTile + tid] = page_slot(p, id[u], pos[u]);
    }
    __syncthreads();
    write_slots(p, t0, n, s_base);
}

// The same for larger batches, after plan_kernel and by its results: one search per token for its request (in shared
// memory up to kSlotBatch requests).
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
        const int b = request_of(ends, p.batch, token);
        if (b < p.batch) {
            const int start = p.start_pos[b];
            const int64_t pos = start + (token - (b ? ends[b - 1] : 0));
            if (start >= 0) base = page_slot(p, p.table[static_cast<int64_t>(b) * p.width + pos / kPage], pos);
        }
    }
    s_base[tid] = base;
    __syncthreads();
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

constexpr int kAppendWarps = 4;

// One warp owns the page runs (consecutive input tokens of one kv head in one page) that start in its tile of
// tokens, and follows the last one past the tile's end.  A run's rows are read once: stored to the pool and folded
// into the page's channel bounds, which no other warp touches, so nothing is atomic and the result does not depend
// on the order of warps.  A lane holds d / 32 channels of a row.  VALUES: there is a value pool.
template <typename T, int D, bool VALUES>
__global__ void __launch_bounds__(32 * kAppendWarps, D == 256 && VALUES ? 4 : 6) append_kernel(const AppendParams p) {
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
    if (p.tile == kPage) {                               // rows that are nearly sure to be read, while the slots come
        constexpr int kLines = D / 64;                   // of 128 bytes, per row
        for (int x = lane; x < kPage * kLines; x += 32) {
            const int64_t t = t0 + x / kLines;
            if (t < p.n) {
                const int64_t at = x % kLines * 64 - lane * 2 * W;
                asm volatile("prefetch.global.L2 [%0];" ::"l"(k + t * p.k_token + at));
                if constexpr (VALUES) asm volatile("prefetch.global.L2 [%0];" ::"l"(v + t * p.v_token + at));
            }
        }
    }
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
    int room;                          // pages whose keys and ids select_kernel's shared memory holds
    int parts;                         // CTAs per row in select_kernel's SCORED form (a power of two, at most 8)
    uint32_t* keys;                    // [B][H_kv][key_stride]: keys of score_kernel (select_kernel's SCORED form)
    float* sizes;                      // [B][H_kv][tiles]: see score_pages
};

constexpr int kScoreThreads = 256;     // threads that score pages together: a CTA of score_kernel, or of select_kernel
constexpr int kScoreTile = 256;        // pages a CTA of score_kernel scores, at most
constexpr int kSortThreads = 512;      // threads of select_kernel's SCORED form

// Keys of a row, in the workspace or in shared memory, are followed by others up to a multiple of kKeyGroup: a warp reads
// four per lane at a time.
constexpr int kKeyGroup = 128;
inline __host__ __device__ int64_t key_stride(int width) {
    return (static_cast<int64_t>(width) + kKeyGroup - 1) / kKeyGroup * kKeyGroup;
}

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


__device__ __forceinline__ float max_nan(float a, float b) {         // not a number if one of the two is none
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Order-preserving bits of a score; -0 counts as 0, and what is not a number ranks below everything.
__device__ __forceinline__ uint32_t score_key(float s) {
    const uint32_t bits = __float_as_uint(s + 0.f);
    return s != s ? 0u : ((bits >> 31) ? ~bits : bits | 0x80000000u);
}
__device__ __forceinline__ float key_score(uint32_t key) {
    return __uint_as_float((key >> 31) ? key ^ 0x80000000u : ~key);
}

__device__ __forceinline__ int64_t select_len(const SelectParams& p, int b) {
    const int64_t most = static_cast<int64_t>(p.width) * kPage, len = p.seq_lens[b];
    return len < 0 ? 0 : (len > most ? most : len);
}

// The score of a page is max over the group's query heads of U_g = sum_c max(q_gc lo_c, q_gc hi_c), which is at least
// q_g . k for every key in the page.  With lo <= hi the larger product is (q > 0 ? q hi : q lo), so U_g is the product
// of max(q, 0) with hi plus that of min(q, 0) with lo.  Products of 16-bit values are exact in fp32, and the order in
// which they are added up is part of the operator, so that the choice of pages can be reproduced bit for bit.
// With an infinite bound that sum of two products can be 0 times infinity where U_g is a number; pages that come out as not a
// number get their scores from the definition.
//
// The tensor cores add in an order of their own, but nothing else is fast enough to keep up with the memory: on the
// FMA pipe with that order 8192 pages x 8 kv heads x 8 query heads take 13 us, here 4.5.  So every score is first
// computed on the tensor cores, together with its size sum |q| |bound| from the same operands, and the selection asks
// for the scores in the defined order only where they could change its outcome (see select_kernel).

// How far a score from the tensor cores may be from the one in the defined order, as a part of the largest size in the
// row.  In that order a product takes part in at most 10 rounded additions: 10 2^-24.  The tensor cores make d / 8
// steps in four chains of d / 32; a step adds 16 products to a sum, each cut off behind 24 bits of the largest: below
// 17 d / 32 2^-23 of the chains' sizes, which add up to the row's.  Three more additions join the chains.
template <int D>
constexpr float kScoreError = (17.f * D / 32.f + 7.f) / 8388608.f;

// The key of page `id` by its score in the defined order, by a whole warp: each 8 channels as an even and an odd chain,
// the two added, then the upper half of the sums onto the lower.  q: the group's heads.
template <typename T, int D>
__device__ __forceinline__ uint32_t exact_key(const SelectParams& p, int h, int id, const uint4* q) {
    constexpr int LP = D / 8;                            // lanes with channels; the others repeat theirs
    const int l = (threadIdx.x & 31) % LP;
    const T* page = static_cast<const T*>(p.bounds) + (static_cast<int64_t>(id) * p.heads + h) * 2 * D;
    const uint4 lw = *reinterpret_cast<const uint4*>(page + 8 * l), hw = *reinterpret_cast<const uint4*>(page + D + 8 * l);
    const uint32_t lo[4] = {lw.x, lw.y, lw.z, lw.w}, hi[4] = {hw.x, hw.y, hw.z, hw.w};
    float best = -INFINITY;
#pragma unroll 4
    for (int g = 0; g < p.group; ++g) {
        const uint4 qw = q[g * LP + l];
        const uint32_t x[4] = {qw.x, qw.y, qw.z, qw.w};
        float even = 0.f, odd = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = Pair<T>::floats(x[i]), a = Pair<T>::floats(lo[i]), c = Pair<T>::floats(hi[i]);
            const float qe = f.x == f.x ? f.x : 0.f, qo = f.y == f.y ? f.y : 0.f;
            even += max_nan(qe * a.x, qe * c.x);
            odd += max_nan(qo * a.y, qo * c.y);
        }
        float s = even + odd;
#pragma unroll
        for (int o = LP / 2; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        best = max_nan(best, s);
    }
    return score_key(best);
}

// Keys of the cnt pages from p0 on of a row of nb pages by the whole block, and the largest size among them (returned
// to every thread of the warp that saw it).  ids: the pages' ids.  A warp takes 16 pages as the rows of its MMAs; head g
// (or the last one) is column g.  The order of channels inside an MMA is free, so a lane's share of a row is 16-byte
// words straight from memory: channels 32 c + 8 tig .. + 7 of rows gid and gid + 8 are the operands of two steps.
template <typename T, int D>
__device__ __forceinline__ float score_pages(const SelectParams& p, int b, int h, int nb, int p0, int cnt, const int32_t* ids,
                                             uint32_t* keys) {
    using P = typename Pair<T>::type;
    constexpr int NC = D / 32;                           // 16-byte words of a row per lane
    constexpr int kBatch = NC < 4 ? NC : 4;              // of these, in flight at a time (for each of two rows, lo and hi)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
    uint4 query[NC];                                     // of head gid
    {
        const T* q = static_cast<const T*>(p.q) + b * p.q_stride +
                     (static_cast<int64_t>(h) * p.group + (gid < p.group ? gid : p.group - 1)) * D + 8 * tig;
#pragma unroll
        for (int c = 0; c < NC; ++c) query[c] = *reinterpret_cast<const uint4*>(q + 32 * c);
    }
    const T* bounds = static_cast<const T*>(p.bounds) + static_cast<int64_t>(h) * 2 * D + 8 * tig;
    const int64_t page_stride = static_cast<int64_t>(p.heads) * 2 * D;
    float size = 0.f;
    for (int j0 = warp * 16; j0 < cnt; j0 += kScoreThreads / 2) {
        const T* src[2];
        bool there[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int j = j0 + gid + 8 * r, id = j < cnt ? ids[j] : -1;
            there[r] = id >= 0 && id < p.num_pages;
            src[r] = bounds + (there[r] ? id : 0) * page_stride;
        }
        float s[4][4] = {}, a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c0 = 0; c0 < NC; c0 += kBatch) {
            uint4 lo[kBatch][2], hi[kBatch][2];
#pragma unroll
            for (int c = 0; c < kBatch; ++c) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    lo[c][r] = hi[c][r] = make_uint4(0u, 0u, 0u, 0u);
                    if (there[r]) {
                        lo[c][r] = *reinterpret_cast<const uint4*>(src[r] + 32 * (c0 + c));
                        hi[c][r] = *reinterpret_cast<const uint4*>(src[r] + 32 * (c0 + c) + D);
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < kBatch; ++c) {
                const uint4 w = query[c0 + c];           // its two parts take no registers between the pages
                const uint32_t qp[4] = {max2<T>(w.x, 0u), max2<T>(w.y, 0u), max2<T>(w.z, 0u), max2<T>(w.w, 0u)};
                const uint32_t qn[4] = {min2<T>(w.x, 0u), min2<T>(w.y, 0u), min2<T>(w.z, 0u), min2<T>(w.w, 0u)};
                const uint4 &l0 = lo[c][0], &l1 = lo[c][1], &h0 = hi[c][0], &h1 = hi[c][1];
                mma16816<T>(s[0], h0.x, h1.x, h0.y, h1.y, qp[0], qp[1]);
                mma16816<T>(s[1], h0.z, h1.z, h0.w, h1.w, qp[2], qp[3]);
                mma16816<T>(s[2], l0.x, l1.x, l0.y, l1.y, qn[0], qn[1]);
                mma16816<T>(s[3], l0.z, l1.z, l0.w, l1.w, qn[2], qn[3]);
                constexpr uint32_t kAbs = 0x7fff7fffu, kMinus = 0x80008000u;          // |hi| max(q, 0) - |lo| min(q, 0)
                mma16816<T>(a, h0.x & kAbs, h1.x & kAbs, h0.y & kAbs, h1.y & kAbs, qp[0], qp[1]);
                mma16816<T>(a, h0.z & kAbs, h1.z & kAbs, h0.w & kAbs, h1.w & kAbs, qp[2], qp[3]);
                mma16816<T>(a, l0.x | kMinus, l1.x | kMinus, l0.y | kMinus, l1.y | kMinus, qn[0], qn[1]);
                mma16816<T>(a, l0.z | kMinus, l1.z | kMinus, l0.w | kMinus, l1.w | kMinus, qn[2], qn[3]);
            }
        }
        // rows gid and gid + 8: the maximum over the heads, columns 2 tig and 2 tig + 1 of this and the quad's lanes
#pragma unroll
        for (int e = 0; e < 4; ++e) s[0][e] = (s[0][e] + s[1][e]) + (s[2][e] + s[3][e]);
        float best[2] = {max_nan(s[0][0], s[0][1]), max_nan(s[0][2], s[0][3])};
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            best[0] = max_nan(best[0], __shfl_xor_sync(0xffffffffu, best[0], o));
            best[1] = max_nan(best[1], __shfl_xor_sync(0xffffffffu, best[1], o));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) size = a[e] > size && a[e] <= 3.402823466e38f ? a[e] : size;   // finite ones
        const int j = j0 + gid + 8 * tig;
        if (tig < 2 && j < cnt) {
            uint32_t key = (tig ? there[1] : there[0]) ? score_key(tig ? best[1] : best[0]) : 0u;
            const int at = p0 + j;
            if (at < p.keep_first || at >= nb - p.keep_last) key = 0xffffffffu;
            keys[j] = key;
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) size = fmaxf(size, __shfl_xor_sync(0xffffffffu, size, o));
    return size;
}

// The keys of a row's nb pages whose scores came out as not a number, from the definition, by NT threads.  table: the row's page ids.
// Rarely called, and apart, so that it takes no registers elsewhere.
template <typename T, int D, int NT>
__device__ __noinline__ void score_by_definition(const void* bounds, const uint4* q, const int32_t* table, int heads, int group, int num_pages,
                                                 int h, int nb, uint32_t* keys) {
    SelectParams p;
    p.bounds = bounds;
    p.heads = heads;
    p.group = group;
#pragma unroll 1
    for (int j = threadIdx.x >> 5; j < nb; j += NT / 32) {
        if (keys[j] != 0u) continue;                     // a number, or kept in any case
        const int id = table[j];
        const uint32_t key = id < 0 || id >= num_pages ? 0u : exact_key<T, D>(p, h, id, q);
        __syncwarp();
        if ((threadIdx.x & 31) == 0) keys[j] = key;
    }
    __syncthreads();
}

// Keys of a call with few rows, where a CTA per row would leave most of the GPU idle: a CTA per row and p.tile pages.
template <typename T, int D>
__global__ void __launch_bounds__(kScoreThreads, 2) score_kernel(const SelectParams p) {
    __shared__ int32_t s_ids[kScoreTile];
    __shared__ float s_size[kScoreThreads / 32];
    static_assert(kScoreTile == kScoreThreads, "a thread per page id");
    begin_dependent();
    const int tiles = (p.width + p.tile - 1) / p.tile;
    const int row = blockIdx.x / tiles, b = row / p.heads, h = row - b * p.heads, tile = blockIdx.x - row * tiles;
    const int64_t len = select_len(p, b);
    const int p0 = tile * p.tile;
    if (threadIdx.x < p.tile && p0 + threadIdx.x < p.width)
        s_ids[threadIdx.x] = p.table[static_cast<int64_t>(b) * p.width + p0 + threadIdx.x];
    const int nb = static_cast<int>((len + kPage - 1) / kPage);
    if (p0 >= nb || nb <= p.budget) return;
    const int cnt = nb - p0 < p.tile ? nb - p0 : p.tile;
    __syncthreads();
    const float size = score_pages<T, D>(p, b, h, nb, p0, cnt, s_ids, p.keys + row * key_stride(p.width) + p0);
    if ((threadIdx.x & 31) == 0) s_size[threadIdx.x >> 5] = size;
    __syncthreads();
    if (threadIdx.x == 0) {
        float m = 0.f;
        for (int w = 0; w < kScoreThreads / 32; ++w) m = fmaxf(m, s_size[w]);
        p.sizes[static_cast<int64_t>(row) * tiles + tile] = m;
    }
}

// The `budget` best pages of one (sequence, kv head), by one CTA.  SCORED: score_kernel has computed the keys; else the
// CTA computes its row's keys first, several CTAs to an SM so that one row's selection runs under another's loads.
//
// The choice is a radix selection: the keys' range is cut into 1024 bins and the bin that holds the budget-th largest
// key is found.  The range starts at the smallest and largest score, not at the key's top bits, which all scores tend to
// share.  Pages kept in any case do not take part.
//
// The keys are the tensor cores' scores.  With e the largest error these may have (kScoreError of the row's largest
// size), a page more than 2 e above the bin is in by its score in the defined order too, and one more than 2 e below it
// is out.  The others are put in a list, get their scores in the defined order and are ranked against each other, ties
// by page index.  If the list cannot hold them all, these scores take the place of the keys, and the range is cut until
// a bin goes in whole or holds one value.
//
// The work of one row is bound by the instructions of one SM, a few per key, so keys are read four at a time, what does
// not compete has a key of its own (no tests of the page's index), and nothing is done per page that is left out.  With
// few rows several CTAs make a row's choice, each for itself, and write out a part of it (8 rows of 8192 pages: 16.9 us
// with one, 15.9 with 4, 15.8 with 8, 16.1 with 16).  Without SCORED two CTAs of an SM have the registers that the loads
// want at d = 128 and 256 (512 rows of 200 pages: 20.8 and 31.1 us; three CTAs 24.6 and 39.4), four at d = 64 (10.9; three 13.9).
template <typename T, int D, bool SCORED>
__global__ void __launch_bounds__(SCORED ? kSortThreads : kScoreThreads, SCORED ? 1 : (D == 64 ? 4 : 2))
    select_kernel(const SelectParams p) {
    constexpr int NT = SCORED ? kSortThreads : kScoreThreads;
    constexpr int NW = NT / 32;
    constexpr int kList = 256, kBins = 1024, kBinBits = 10, kOwn = kBins / NT;    // bins of a thread
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) uint32_t s_hist[kBins];
    __shared__ uint32_t s_pick[3];
    __shared__ uint32_t s_warp[NW], s_warp2[NW], s_warp3[NW];
    __shared__ float s_size[NW];
    __shared__ uint32_t s_key[kList];
    __shared__ int s_page[kList];
    __shared__ int s_listed[2];                          // entries of the list; those above the bin
    __shared__ uint4 s_q[8 * D / 8];                     // the group's heads
    begin_dependent();
    const int row = blockIdx.x;
    const int b = row / p.heads, h = row - b * p.heads;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int32_t* table = p.table + static_cast<int64_t>(b) * p.width;
    const int64_t len = select_len(p, b);
    uint32_t* keys = reinterpret_cast<uint32_t*>(smem);
    int32_t* ids = reinterpret_cast<int32_t*>(keys + p.room);
    // what does not depend on the length is read while that is on its way
    const int tiles = SCORED ? (p.width + p.tile - 1) / p.tile : 0;
    float size = 0.f;
    if constexpr (SCORED) {
        const uint32_t* src = p.keys + row * key_stride(p.width);
#pragma unroll 4
        for (int j = tid * 4; j < p.room; j += NT * 4)   // what lies behind the last key is overwritten below
            *reinterpret_cast<uint4*>(keys + j) = __ldcg(reinterpret_cast<const uint4*>(src + j));
        if (tid < tiles) size = __ldcg(p.sizes + static_cast<int64_t>(row) * tiles + tid);
    }
    const int known = p.width < p.room ? p.width : p.room;           // page ids in shared memory
#pragma unroll 4
    for (int j = tid; j < known; j += NT) {
        if constexpr (SCORED)                            // not needed before the list is complete
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(ids + j)), "l"(table + j) : "memory");
        else
            ids[j] = table[j];
    }
    const T* q = static_cast<const T*>(p.q) + b * p.q_stride + static_cast<int64_t>(h) * p.group * D;
    for (int i = tid; i < p.group * D / 8; i += NT) s_q[i] = reinterpret_cast<const uint4*>(q)[i];
    for (int i = tid; i < kBins; i += NT) s_hist[i] = 0;
    if (tid < 2) s_listed[tid] = 0;
    const int nb = static_cast<int>((len + kPage - 1) / kPage);
    int32_t* out = p.pages + static_cast<int64_t>(row) * p.budget;
    auto head_page = [&](int id) { return (id < 0 || id >= p.num_pages) ? -1 : id * p.heads + h; };
    const int part = SCORED ? blockIdx.y : 0;
    if (tid == 0 && part == 0) p.lens[row] = static_cast<int>(nb <= p.budget ? len : len - static_cast<int64_t>(nb - p.budget) * kPage);
    if (nb <= p.budget) {                                // every page is kept
        if constexpr (SCORED) asm volatile("cp.async.wait_all;" ::: "memory");       // no copy outlives its CTA
        if (part == 0)
            for (int j = tid; j < p.budget; j += NT) out[j] = head_page(j < nb ? table[j] : -1);
        return;
    }
    const int padded = static_cast<int>(key_stride(nb));
    auto id_of = [&](int j) { return SCORED && j >= known ? table[j] : ids[j]; };
    if constexpr (SCORED) {
        __syncthreads();
        // the passes over a very long sequence read the L2 cache
        if (padded > p.room) keys = p.keys + row * key_stride(p.width);
        const int used = (nb + p.tile - 1) / p.tile;     // tiles with a page
        if (tid >= used) size = 0.f;
        for (int i = tid + NT; i < used; i += NT) size = fmaxf(size, __ldcg(p.sizes + static_cast<int64_t>(row) * tiles + i));
        for (int o = 16; o; o >>= 1) size = fmaxf(size, __shfl_xor_sync(0xffffffffu, size, o));
    } else {
        __syncthreads();
        size = score_pages<T, D>(p, b, h, nb, 0, nb, ids, keys);
    }
    constexpr uint32_t kKept = 0xffffffffu;              // the key of pages that do not compete, and of none
    if (nb + tid < padded) keys[nb + tid] = kKept;       // padded - nb < kKeyGroup <= NT
    if (lane == 0) s_size[warp] = size;
    __syncthreads();
    // Warp w looks after pages j0 .. j1 - 1, four to a lane.
    const int chunk = (padded / kKeyGroup + NW - 1) / NW * kKeyGroup;
    const int j0 = warp * chunk + lane * 4, j1 = (warp + 1) * chunk < padded ? (warp + 1) * chunk : padded;
    auto each = [&](auto f) {                            // f(a key)
#pragma unroll 1
        for (int j = j0; j < j1; j += kKeyGroup) {
            const uint4 k = *reinterpret_cast<const uint4*>(keys + j);
            f(k.x); f(k.y); f(k.z); f(k.w);
        }
    };
    const uint32_t wanted = static_cast<uint32_t>(p.budget - p.keep_first - p.keep_last);   // of those that compete
    uint32_t from = 0xffffffffu, bound = 0xffffffffu, need = 0;      // in: keys from `from` on, and `need` equal to `bound`
    // The range of the block's keys, and whether one of them is no number; from each thread the smallest and largest of its own.
    auto block_range = [&](uint32_t& least, uint32_t& most) {
        uint32_t low = __reduce_min_sync(0xffffffffu, least), high = __reduce_max_sync(0xffffffffu, most);
        uint32_t best = __reduce_min_sync(0xffffffffu, most);
        __syncthreads();                                 // the sums before have been read
        if (lane == 0) {
            s_warp[warp] = low;
            s_warp2[warp] = high;
            s_warp3[warp] = best;
        }
        __syncthreads();
        least = __reduce_min_sync(0xffffffffu, lane < NW ? s_warp[lane] : 0xffffffffu);
        most = __reduce_max_sync(0xffffffffu, lane < NW ? s_warp2[lane] : 0u);
        best = __reduce_min_sync(0xffffffffu, lane < NW ? s_warp3[lane] : 0xffffffffu);
        const bool none = least == 0u;
        // every thread has a key from the smallest of the threads' largest ones on: if no more are wanted, it ends there
        if (best > 0u && need <= NT) least = best - 1u;
        --most;
        return none;
    };
    if (wanted > 0) {
        need = wanted;
        float error = s_size[lane < NW ? lane : 0];
        for (int o = 16; o; o >>= 1) error = fmaxf(error, __shfl_xor_sync(0xffffffffu, error, o));
        error *= 2.f * kScoreError<D>;
        int bits = 32;
        bool exact = false, defined = false;             // defined: no score that is a number by the definition counts as none
        for (bool again = true; again;) {
            if (bits == 32) {
                // the range of the keys that compete
                uint32_t least = 0xffffffffu, most = 0u;
                each([&](uint32_t k) {
                    least = min(least, k);
                    most = max(most, k + 1u);            // kKept: 0
                });
                if (block_range(least, most) && !defined && !exact) {
                    defined = true;
                    score_by_definition<T, D, NT>(p.bounds, s_q, table, p.heads, p.group, p.num_pages, h, nb, keys);
                    continue;
                }
                bound = least;
                bits = 32 - __clz(static_cast<int>(most - least));
            }
            // count the keys from `bound` to `bound` + 2^bits - 1 in kBins bins and find the bin of the need-th largest
            const int shift = bits > kBinBits ? bits - kBinBits : 0;
            const uint32_t width = min(bits == 32 ? 0xffffffffu : (1u << bits) - 1u, kKept - 1u - bound);
            each([&](uint32_t k) {
                if (k - bound <= width) atomicAdd(&s_hist[(k - bound) >> shift], 1u);
            });
            __syncthreads();
            // from the largest bin down: thread t takes kOwn bins from kBins - 1 - kOwn t on
            const int top_bin = kBins - 1 - kOwn * tid;
            uint32_t c[kOwn], incl = 0;
#pragma unroll
            for (int i = 0; i < kOwn; ++i) {
                c[i] = s_hist[top_bin - i];
                s_hist[top_bin - i] = 0;                 // for the next pass
                incl += c[i];
            }
            const uint32_t own = incl;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t t = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += t;
            }
            if (lane == 31) s_warp[warp] = incl;
            __syncthreads();
            uint32_t before = incl - own + __reduce_add_sync(0xffffffffu, lane < warp ? s_warp[lane] : 0u);
#pragma unroll
            for (int i = 0; i < kOwn; ++i) {
                if (before < need && before + c[i] >= need) {        // one bin
                    s_pick[0] = top_bin - i;
                    s_pick[1] = before;
                    s_pick[2] = before + c[i];
                }
                before += c[i];
            }
            __syncthreads();
            if (exact) {
                bound += s_pick[0] << shift;
                const bool whole = s_pick[2] == need;    // everything from `bound` on is in
                need = whole ? 0u : need - s_pick[1];
                bits = shift;
                again = !whole && bits > 0;
                from = whole ? bound : bound + 1;        // bound < 2^32 - 1: that key is of pages kept in any case
                __syncthreads();                         // s_pick has been read
                continue;
            }
            // the list: this bin's keys and those within the error of it
            const uint32_t bottom = bound + (s_pick[0] << shift), top = bottom + ((1u << shift) - 1u);
            const uint32_t low = min(bottom, score_key(__fsub_rd(key_score(bottom), error)));
            const uint32_t high = max(top, score_key(__fadd_ru(key_score(top), error)));
#pragma unroll 1
            for (int j = j0; j < j1; j += kKeyGroup) {
                const uint4 k4 = *reinterpret_cast<const uint4*>(keys + j);
                const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w}, span = high - low;
                unsigned some = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) some |= k[i] - low <= span ? 1u << i : 0u;
                if (some) {
#pragma unroll 1
                    for (; some; some &= some - 1) {
                        const int i = __ffs(some) - 1, at = atomicAdd(&s_listed[0], 1);
                        const uint32_t key = keys[j + i];
                        if (key > top) atomicAdd(&s_listed[1], 1);
                        if (at < kList) {
                            s_key[at] = key;
                            s_page[at] = j + i;
                        }
                    }
                }
            }
            if constexpr (SCORED) asm volatile("cp.async.wait_all;" ::: "memory");
            __syncthreads();
            const int n = s_listed[0];
            // entries of the list that are in
            const int want = static_cast<int>(need) - (static_cast<int>(s_pick[1]) - s_listed[1]);
            if (error == 0.f) {                          // without a size all scores are 0: nothing to compute
                exact = true;
                bits = 32;
                continue;
            }
            if (n > kList) {
#pragma unroll 1
                for (int j = j0 - lane * 4 + lane; j < j1; j += 32) {
                    const uint32_t k = keys[j];
                    uint32_t now = k == kKept ? k : (k > high ? kKept - 1u : 0u);
#pragma unroll 1
                    for (unsigned rest = __ballot_sync(0xffffffffu, k != 0u && k >= low && k <= high); rest; rest &= rest - 1) {
                        const int src = __ffs(rest) - 1;
                        const uint32_t k2 = exact_key<T, D>(p, h, id_of(j - lane + src), s_q);
                        if (lane == src) now = k2;
                    }
                    keys[j] = now;
                }
                __syncthreads();
                exact = true;
                bits = 32;
                continue;
            }
            if (want > 0 && want < n) {
#pragma unroll 1
                for (int x = warp; x < n; x += NW) {     // what is not a number (key 0) is so in any order
                    const uint32_t k = s_key[x] ? exact_key<T, D>(p, h, id_of(s_page[x]), s_q) : 0u;
                    __syncwarp();
                    if (lane == 0) s_key[x] = k;
                }
                __syncthreads();
            }
            for (int e = warp; e < n; e += NW) {         // a warp per entry: how many go before it
                const uint32_t mine = s_key[e];
                const int page = s_page[e];
                int rank = 0;
                for (int x = lane; x < n; x += 32) rank += (s_key[x] > mine || (s_key[x] == mine && s_page[x] < page)) ? 1 : 0;
                rank = __reduce_add_sync(0xffffffffu, rank);
                if (lane == 0) keys[page] = rank < want ? kKept : 0u;
            }
            __syncthreads();
            from = high + 1;                             // high < 2^32 - 1
            need = 0;
            again = false;
        }
    }
    // ---- the pages that are in, in ascending order
    uint32_t n_in = 0, n_tie = 0;
    each([&](uint32_t k) {
        n_in += k >= from ? 1u : 0u;
        n_tie += k < from && k == bound ? 1u : 0u;
    });
    n_in = __reduce_add_sync(0xffffffffu, n_in);
    n_tie = __reduce_add_sync(0xffffffffu, n_tie);
    if constexpr (SCORED) asm volatile("cp.async.wait_all;" ::: "memory");   // if there was no list
    __syncthreads();                                     // the sums before have been read
    if (lane == 0) {
        s_warp[warp] = n_in;
        s_warp2[warp] = n_tie;
    }
    __syncthreads();
    // the part's warps take equal runs of key groups, which begin in the chunk of warp `in_chunk` of the sums above
    const int parts = SCORED ? p.parts : 1, groups = chunk / kKeyGroup, run = (groups + parts - 1) / parts;
    const int part_end = (part + 1) * (NW / parts) * groups, g0 = part * (NW / parts) * groups + warp * run;
    const int g1 = g0 + run < part_end ? g0 + run : part_end;
    const int in_chunk = g0 < part_end ? g0 / groups : 0;            // warps behind the part's last run have none
    uint32_t in_before = __reduce_add_sync(0xffffffffu, lane < in_chunk ? s_warp[lane] : 0u);
    uint32_t ties_before = __reduce_add_sync(0xffffffffu, lane < in_chunk ? s_warp2[lane] : 0u);
    const unsigned lower = (1u << lane) - 1u;            // the lanes before
#pragma unroll 1
    for (int g = g0 < part_end ? in_chunk * groups : g1; g < g1 && g * kKeyGroup < padded; ++g) {
        const int j = g * kKeyGroup + lane * 4;
        const uint4 k4 = *reinterpret_cast<const uint4*>(keys + j);
        const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
        uint32_t i_at = in_before, t_at = ties_before;   // of the lane's first page
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned in = __ballot_sync(0xffffffffu, k[i] >= from);
            i_at += __popc(in & lower);
            in_before += __popc(in);
        }
        if (need) {                                      // else no key is a tie
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const unsigned tie = __ballot_sync(0xffffffffu, k[i] < from && k[i] == bound);
                t_at += __popc(tie & lower);
                ties_before += __popc(tie);
            }
        }
        if (g < g0) continue;
        uint4 id4;                                       // ids of keys behind the last page are not used
        if (!SCORED || j + 3 < p.room) {
            id4 = *reinterpret_cast<const uint4*>(ids + j);
        } else {
            id4.x = j < nb ? table[j] : 0;
            id4.y = j + 1 < nb ? table[j + 1] : 0;
            id4.z = j + 2 < nb ? table[j + 2] : 0;
            id4.w = j + 3 < nb ? table[j + 3] : 0;
        }
        const uint32_t id[4] = {id4.x, id4.y, id4.z, id4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool is_in = k[i] >= from, is_tie = !is_in && k[i] == bound && t_at < need;
            if ((is_in || is_tie) && j + i < nb) out[i_at + (t_at < need ? t_at : need)] = head_page(static_cast<int>(id[i]));
            i_at += is_in ? 1u : 0u;
            t_at += is_tie ? 1u : 0u;
        }
    }
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

// WIDE: calls of a few short rows, a CTA each, which have an SM for themselves.  A warp needs 0.6 us for a page then, not
// for its bytes but for its chain of instructions, so there are twice as many warps (8 rows of 13 pages at d = 128: 4.2 us,
// with four warps 5.0; of 32 pages 6.3 and 7.3).
template <int D, bool WIDE = false>
struct PagesCfg {
    static constexpr int kWarps = WIDE ? 8 : 4;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kPageBytes = kPage * D * 2;                 // one page of keys (or values) of a kv head
    // Pages of keys and values in flight per warp, 96 to 128 KB per SM.  More only lengthens the queues at the memory,
    // which SMs leave at different speeds while the shares are equal: 4, 3 and 3 pages at d = 64, 128 and 256 take
    // 50.6, 89.6 and 94.4 us where 2 take 48.0, 85.4 and 92.1 (64 ragged sequences, 131072 tokens, 64 selected pages).
    static constexpr int kStages = 2;
    static constexpr int kCtasPerSm = WIDE ? 1 : (D == 64) ? 3 : (D == 128) ? 2 : 1;
    static constexpr int kRing = kWarps * kStages * 2 * kPageBytes;
    // what a row costs besides its pages (its query, the joining of the warps' parts), in pages; a multiple of kWarps
    static constexpr int kRowCost = 8;
    static constexpr int kHeadStride = D + 4;                        // spreads the accumulator rows over the banks
    // floats per warp: m[8], l[8], O[G][D + 4].  What a group of fewer than 8 heads leaves free lets the join's CTAs
    // become resident before the last share is done.
    static constexpr __host__ __device__ int comb(int group) { return 16 + group * kHeadStride; }
    // d = 256 has no registers left for the query's fragments: each warp keeps its copy in shared memory
    static constexpr bool kQueryInSmem = D == 256;
    static constexpr int kQueryBytes = kQueryInSmem ? D / 16 * 32 * 8 : 0;
    static constexpr int smem(int group) { return kRing + kWarps * (comb(group) * 4 + kQueryBytes); }
    static constexpr int kPart = 16 + 8 * D;                         // floats per partial: m[8], l[8], O[8][D]
};

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
// operations per byte, so a large call is bound by how fast pages can be read, and the grid is laid out for that alone:
// all pages of the call, in the order (table row, kv head, page), are cut into shares of equal cost, one per resident
// CTA, whatever the lengths of the sequences are.  A share covers parts of one or several rows (a row: one sequence
// and kv head with its query heads, whose own cost counts as kRowCost pages); a row that lies inside one share is
// finished there, and attend_pages_join_kernel joins the others.  Calls with short table rows take a CTA per row and
// need no join.  The running maximum and sum (fp32) make the split exact up to rounding.
//
// Warp w of a CTA takes pages w, w + kWarps, ... of the share and keeps kStages of them in flight in its own ring of
// shared memory with 16-byte cp.async copies, so no warp waits for another until a row ends.  16-byte chunk c of a
// page's row r sits at chunk c ^ (r % 8): the copies and both ldmatrix reads are then free of bank conflicts.
//   scores  S[head][token]  = q (A, 8 of 16 rows used) x k (B)
//   values  O^T[col][head] += v^T (A) x p (B): the scores' fragment layout is that of p, nothing moves between lanes
// p is 2^(s - m + 12) split into 16-bit terms (see Weights), so that rounding it costs no accuracy; with 8 heads or
// fewer per row the tensor work is a small part of the time either way.
template <typename T, int D, bool WIDE>
__global__ void __launch_bounds__(PagesCfg<D, WIDE>::kThreads, PagesCfg<D, WIDE>::kCtasPerSm)
    attend_pages_kernel(const AttendPagesParams p) {
    using C = PagesCfg<D, WIDE>;
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
    const bool direct = WIDE || p.direct;
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
    if (direct) {
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
        return ld.x < x1 ? p.table[static_cast<int64_t>(ld.unit) * p.width + ld.pg] : -1;
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
    if (!direct) write_zeros();
    if (!direct && !p.rows_join && tid == 0) {
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
        uint32_t qa[C::kQueryInSmem ? 1 : KS][2];
        uint2* const qs = reinterpret_cast<uint2*>(comb + C::kWarps * C::comb(G)) + warp * (KS * 32) + lane;
        {
            const int b = row / p.heads, h = row - b * p.heads;
            const T* q = static_cast<const T*>(p.q) + b * p.q_stride + (static_cast<int64_t>(h) * G + gid) * D + 2 * tig;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const uint32_t a = gid < G ? *reinterpret_cast<const uint32_t*>(q + 16 * ks) : 0u;
                const uint32_t c = gid < G ? *reinterpret_cast<const uint32_t*>(q + 16 * ks + 8) : 0u;
                if constexpr (C::kQueryInSmem) {
                    qs[ks * 32] = make_uint2(a, c);      // read back by this lane only
                } else {
                    qa[ks][0] = a;
                    qa[ks][1] = c;
                }
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
                    uint2 a;
                    if constexpr (C::kQueryInSmem) a = qs[ks * 32]; else a = make_uint2(qa[ks][0], qa[ks][1]);
                    mma16816<T>(sc[ks & 1][0], a.x, 0u, a.y, 0u, f[0], f[1]);
                    mma16816<T>(sc[ks & 1][1], a.x, 0u, a.y, 0u, f[2], f[3]);
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
                    // the page's part by itself: the tensor cores cut sums off where fp32 additions round
                    float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int t = NT - 1; t >= 0; --t) mma16816<T>(part, f[0], f[1], f[2], f[3], w0[t], w1[t]);
                    o[i][0] += part[0]; o[i][1] += part[1]; o[i][2] += part[2]; o[i][3] += part[3];
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
                p.out[(static_cast<int64_t>(row) * G + g) * D + col] = L == 0.f ? 0.f : O / L;
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
    // only now: CTAs of the kernel behind this one that wait on an SM can keep others of this grid's size from fitting when
    // calls follow one another (64 ragged sequences at d = 64: 48.3 us, with the release at the start 48.8)
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
        const float r = L == 0.f ? 0.f : 1.f / L;   // not a number stays so
        O.x *= r; O.y *= r; O.z *= r; O.w *= r;
        *reinterpret_cast<float4*>(p.out + (static_cast<int64_t>(m.row) * p.group + g) * D + c) = O;
    }
}

}  // namespace dev
}  // namespace tq
