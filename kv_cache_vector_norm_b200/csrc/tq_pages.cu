// libtq: the paged-cache entry points of include/tq.h (planning, append, selection, attention over uncompressed
// pages).  Host-side validation and launches; the kernels are in tq_pages_kernels.cuh.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>

#include "tq_internal.h"
#include "tq_pages_kernels.cuh"

using namespace tq;
using namespace tq::dev;

namespace {

#define TQ_CUDA(call, what)                                                                        \
    do {                                                                                           \
        cudaError_t e_ = (call);                                                                   \
        if (e_ != cudaSuccess) return fail(TQ_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e_));    \
    } while (0)

#define TQ_NEED(cond, status, ...)                                                                 \
    do {                                                                                           \
        if (!(cond)) return fail(status, __VA_ARGS__);                                             \
    } while (0)

// Whether n values at a and at b share no byte.
bool apart(const int32_t* a, const int32_t* b, int64_t n) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x + 4 * n <= y || y + 4 * n <= x;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A limit on the pages of a pool and on a table's width: page indices, slots of a page and sums of two of them stay
// within 32 bits.
constexpr int kMaxPages = 1 << 30;

int device_sms() {
    static std::atomic<int> cache[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 148;
    int v = cache[dev & 63].load();
    if (v == 0) {
        if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v < 1) v = 148;
        cache[dev & 63].store(v);
    }
    return v;
}

// Function attributes are set once per device and kernel.
template <auto Kernel>
cudaError_t prepare_kernel(int smem) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load() & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) done.fetch_or(bit);
    return e;
}

// Launch a kernel as a programmatic dependent of the work before it (see begin_dependent).
template <typename P, typename... Rest>
cudaError_t launch(void (*kernel)(P, Rest...), unsigned grid_x, unsigned grid_y, int threads, size_t smem, cudaStream_t st,
                   const P& p, Rest... rest) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid_x, grid_y);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, rest...);
}

tq_status check_heads(const char* fn, int batch, int hq, int hkv) {
    TQ_NEED(batch >= 1 && hq >= 1 && hkv >= 1, TQ_ERR_INVALID_ARG, "%s: batch, num_q_heads, num_kv_heads must be >= 1", fn);
    TQ_NEED(hq % hkv == 0, TQ_ERR_INVALID_ARG, "%s: num_q_heads=%d is not a multiple of num_kv_heads=%d", fn, hq, hkv);
    TQ_NEED(hq / hkv <= 8, TQ_ERR_UNSUPPORTED, "%s: GQA group %d > 8", fn, hq / hkv);
    TQ_NEED(static_cast<int64_t>(batch) * hkv <= (1 << 26), TQ_ERR_UNSUPPORTED, "%s: more than 2^26 (sequence, kv head) rows", fn);
    return TQ_OK;
}

tq_status check_d_dtype(const char* fn, int d, int dtype) {
    TQ_NEED(d == 64 || d == 128 || d == 256, TQ_ERR_UNSUPPORTED, "%s: head_dim=%d (supported: 64, 128, 256)", fn, d);
    TQ_NEED(dtype == TQ_F16 || dtype == TQ_BF16, TQ_ERR_UNSUPPORTED, "%s: dtype=%d (supported: TQ_F16, TQ_BF16)", fn, dtype);
    return TQ_OK;
}

tq_status check_pool(const char* fn, int num_pages, int heads) {
    TQ_NEED(num_pages >= 1 && num_pages <= kMaxPages && static_cast<int64_t>(num_pages) * heads <= kMaxPages,
            TQ_ERR_INVALID_ARG, "%s: num_pages=%d with %d kv heads (1 .. 2^30 head pages)", fn, num_pages, heads);
    return TQ_OK;
}

#define TQ_DISPATCH_TD(dtype, d, fn, ...)                                                          \
    switch ((d) * 4 + (dtype)) {                                                                   \
        case 64 * 4 + TQ_F16: return fn<__half, 64>(__VA_ARGS__);                                  \
        case 128 * 4 + TQ_F16: return fn<__half, 128>(__VA_ARGS__);                                \
        case 256 * 4 + TQ_F16: return fn<__half, 256>(__VA_ARGS__);                                \
        case 64 * 4 + TQ_BF16: return fn<__nv_bfloat16, 64>(__VA_ARGS__);                          \
        case 128 * 4 + TQ_BF16: return fn<__nv_bfloat16, 128>(__VA_ARGS__);                        \
        default: return fn<__nv_bfloat16, 256>(__VA_ARGS__);                                       \
    }

}  // namespace

// ------------------------------------------------------------------------------------------ planning

extern "C" tq_status tq_plan_pages(const tq_plan_args* a, void* stream) {
    clear_error();
    const char* fn = "tq_plan_pages";
    TQ_NEED(a, TQ_ERR_INVALID_ARG, "%s: args is NULL", fn);
    TQ_NEED(a->batch >= 1 && a->batch <= (1 << 24), TQ_ERR_INVALID_ARG, "%s: batch=%d outside 1 .. 2^24", fn, a->batch);
    TQ_NEED(a->num_kv_heads >= 1 && a->num_kv_heads <= 1024, TQ_ERR_INVALID_ARG, "%s: num_kv_heads=%d outside 1 .. 1024", fn, a->num_kv_heads);
    TQ_NEED(a->max_blocks >= 1 && a->max_blocks <= (1 << 26), TQ_ERR_INVALID_ARG, "%s: max_blocks=%d outside 1 .. 2^26", fn, a->max_blocks);
    tq_status s = check_pool(fn, a->num_pages, a->num_kv_heads);
    if (s != TQ_OK) return s;
    TQ_NEED(a->max_tokens >= 0 && a->max_tokens < (1ll << 31), TQ_ERR_INVALID_ARG, "%s: max_tokens=%lld outside 0 .. 2^31 - 1", fn,
            static_cast<long long>(a->max_tokens));
    TQ_NEED(a->new_lens && a->seq_lens && a->block_table && a->free_pages && a->free_state && a->row_start && a->start_pos &&
                a->seq_lens_out && a->free_state_out && (a->slots || a->max_tokens == 0),
            TQ_ERR_INVALID_ARG, "%s: NULL pointer in args", fn);
    TQ_NEED(aligned(a->new_lens, 4) && aligned(a->seq_lens, 4) && aligned(a->block_table, 4) && aligned(a->free_pages, 4) &&
                aligned(a->free_state, 4) && aligned(a->row_start, 4) && aligned(a->start_pos, 4) &&
                aligned(a->seq_lens_out, 4) && aligned(a->free_state_out, 4) && aligned(a->slots, 8),
            TQ_ERR_INVALID_ARG, "%s: misaligned pointer in args", fn);
    PlanParams p;
    p.new_lens = a->new_lens;
    p.seq_lens = a->seq_lens;
    p.table = a->block_table;
    p.ring = a->free_pages;
    p.state = a->free_state;
    p.slots = a->slots;
    p.row_start = a->row_start;
    p.start_pos = a->start_pos;
    p.seq_lens_out = a->seq_lens_out;
    p.state_out = a->free_state_out;
    p.batch = a->batch;
    p.width = a->max_blocks;
    p.num_pages = a->num_pages;
    p.heads = a->num_kv_heads;
    p.max_tokens = a->max_tokens;
    p.tile = kSlotTile;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // Up to 256 requests the slots' grid plans for itself, and its first CTA does the rest if no output lies over an input
    // (8 heads, 64 requests of one token: 2.5 us, of 64 tokens 2.8).
    // Else the rest takes a second kernel, so a decode step's few slots are written by one planning CTA: with 8 heads 64
    // requests of one token take 3.5 us in one kernel (and 2 us less on the host) and 3.0 in two, 256 take 5.3 and 3.5.  Past
    // 256 requests the slots come behind the plan: 512 take 7.5 us in one kernel and 8.4 in two, 1024 take 11.8 and 8.6.
    // Up to 256 requests one CTA of 256 threads scans faster than one of 1024 (64 requests: 3.5 us, 5.7).
    const bool few = a->batch <= kSlotTile;
    p.apart = few && apart(a->seq_lens, a->seq_lens_out, a->batch) && apart(a->free_state, a->free_state_out, 2);
    const int64_t tiles = (a->max_tokens + kSlotTile - 1) / kSlotTile, each = (tiles + device_sms() - 1) / device_sms();
    if (!p.apart && a->max_tokens * a->num_kv_heads <= (few ? 1024 : 4096)) {
        TQ_CUDA(few ? launch(plan_kernel<kSlotTile, true>, 1, 1, kSlotTile, 0, st, p)
                    : launch(plan_kernel<kPlanThreads, true>, 1, 1, kPlanThreads, 0, st, p),
                "tq_plan_pages: launch");
    } else if (few) {
        p.tile = kSlotTile * static_cast<int>(each < 1 ? 1 : (each < kSlotTiles ? each : kSlotTiles));
        TQ_CUDA(launch(plan_slots_ahead_kernel, static_cast<unsigned>((a->max_tokens + p.tile - 1) / p.tile + (p.apart ? 1 : 0)), 1,
                       kSlotTile, 0, st, p),
                "tq_plan_pages: slot launch");
        if (!p.apart) TQ_CUDA(launch(plan_beside_kernel, 1, 1, kSlotTile, 0, st, p), "tq_plan_pages: launch");
    } else {
        TQ_CUDA(launch(plan_kernel<kPlanThreads, false>, 1, 1, kPlanThreads, 0, st, p), "tq_plan_pages: launch");
        TQ_CUDA(launch(plan_slots_kernel, static_cast<unsigned>(tiles), 1, kSlotTile, 0, st, p), "tq_plan_pages: slot launch");
    }
    return TQ_OK;
}

// -------------------------------------------------------------------------------------------- append

namespace {

template <typename T, int D>
tq_status launch_append(const AppendParams& p, cudaStream_t st) {
    const int64_t warps = (p.n + p.tile - 1) / p.tile * p.heads;
    const unsigned grid = static_cast<unsigned>((warps + kAppendWarps - 1) / kAppendWarps);
    TQ_CUDA(launch(p.v_pool ? append_kernel<T, D, true> : append_kernel<T, D, false>, grid, 1, 32 * kAppendWarps, 0, st, p),
            "tq_append_pages: launch");
    return TQ_OK;
}

}  // namespace

extern "C" tq_status tq_append_pages(const tq_append_args* a, void* stream) {
    clear_error();
    const char* fn = "tq_append_pages";
    TQ_NEED(a, TQ_ERR_INVALID_ARG, "%s: args is NULL", fn);
    tq_status s = check_d_dtype(fn, a->head_dim, a->dtype);
    if (s != TQ_OK) return s;
    TQ_NEED(a->num_kv_heads >= 1 && a->num_kv_heads <= 1024, TQ_ERR_INVALID_ARG, "%s: num_kv_heads=%d outside 1 .. 1024", fn, a->num_kv_heads);
    if ((s = check_pool(fn, a->num_pages, a->num_kv_heads)) != TQ_OK) return s;
    TQ_NEED(a->num_tokens >= 0 && a->num_tokens < (1ll << 31), TQ_ERR_INVALID_ARG, "%s: num_tokens=%lld outside 0 .. 2^31 - 1", fn,
            static_cast<long long>(a->num_tokens));
    TQ_NEED(a->k_pool || a->v_pool || a->bounds, TQ_ERR_INVALID_ARG, "%s: k_pool, v_pool and bounds are all NULL", fn);
    if (a->num_tokens == 0) return TQ_OK;
    TQ_NEED(a->k && a->slots, TQ_ERR_INVALID_ARG, "%s: k and slots must be non-NULL", fn);
    TQ_NEED(!a->v_pool || a->v, TQ_ERR_INVALID_ARG, "%s: v_pool without v", fn);
    TQ_NEED(aligned(a->k, 16) && aligned(a->v, 16) && aligned(a->k_pool, 16) && aligned(a->v_pool, 16) && aligned(a->bounds, 16) &&
                aligned(a->slots, 8),
            TQ_ERR_INVALID_ARG, "%s: k, v, k_pool, v_pool and bounds must be 16-byte aligned", fn);
    TQ_NEED(a->k_token_stride % 8 == 0 && a->k_head_stride % 8 == 0 && a->k_token_stride >= 0 && a->k_head_stride >= 0,
            TQ_ERR_INVALID_ARG, "%s: k strides must be non-negative multiples of 8", fn);
    TQ_NEED(!a->v_pool || (a->v_token_stride % 8 == 0 && a->v_head_stride % 8 == 0 && a->v_token_stride >= 0 && a->v_head_stride >= 0),
            TQ_ERR_INVALID_ARG, "%s: v strides must be non-negative multiples of 8", fn);
    AppendParams p;
    p.k = a->k;
    p.v = a->v;
    p.k_token = a->k_token_stride;
    p.k_head = a->k_head_stride;
    p.v_token = a->v_token_stride;
    p.v_head = a->v_head_stride;
    p.slots = a->slots;
    p.n = a->num_tokens;
    p.rows = static_cast<int64_t>(a->num_pages) * a->num_kv_heads * kPage;
    p.k_pool = a->k_pool;
    p.v_pool = a->v_pool;
    p.bounds = a->bounds;
    p.heads = a->num_kv_heads;
    // Whether tokens fill pages together or lie in pages of their own is not known here.  A warp per token suits the
    // few tokens of a decode step (64 tokens in a page each, 8 heads of d = 128: 2.1 us; 16 tokens per warp: 14.2), 16
    // tokens per warp a prefill (8192 in a row: 14.0 us; one per warp: 27.7); 4 in between (1024 tokens in a page each
    // 6.2 us, in a row 4.7; one per warp 5.6 and 5.3, 16 per warp 13.6 and 3.3).
    const int64_t rows = a->num_tokens * a->num_kv_heads;
    p.tile = rows <= 2048 ? 1 : (rows <= 16384 ? 4 : 16);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    TQ_DISPATCH_TD(a->dtype, a->head_dim, launch_append, p, st);
}

// -------------------------------------------------------------------------------------------- select

namespace {

constexpr int kSelSmem = 200 << 10;
constexpr int kSortRoom = 24576;       // pages that select_kernel's SCORED form keeps in shared memory

struct SelectPlan {
    bool scored;                       // the keys are computed by a grid of their own, through the workspace
    int tile;                          // pages a CTA of that grid takes
    int room;                          // pages whose keys select_kernel keeps in shared memory
    int parts;                         // its CTAs per row in the SCORED form
    size_t workspace_bytes;
};

tq_status plan_select(const char* fn, const tq_select_args* a, SelectPlan* plan) {
    TQ_NEED(a, TQ_ERR_INVALID_ARG, "%s: args is NULL", fn);
    tq_status s = check_heads(fn, a->batch, a->num_q_heads, a->num_kv_heads);
    if (s != TQ_OK) return s;
    if ((s = check_d_dtype(fn, a->head_dim, a->dtype)) != TQ_OK) return s;
    if ((s = check_pool(fn, a->num_pages, a->num_kv_heads)) != TQ_OK) return s;
    TQ_NEED(a->max_blocks >= 1 && a->max_blocks <= (1 << 26), TQ_ERR_INVALID_ARG, "%s: max_blocks=%d outside 1 .. 2^26", fn, a->max_blocks);
    TQ_NEED(a->budget >= 1 && a->keep_first >= 0 && a->keep_last >= 1 && a->keep_first <= a->budget &&
                a->keep_last <= a->budget - a->keep_first,
            TQ_ERR_INVALID_ARG, "%s: budget=%d must hold keep_first=%d (>= 0) and keep_last=%d (>= 1) pages", fn, a->budget,
            a->keep_first, a->keep_last);
    const int64_t rows = static_cast<int64_t>(a->batch) * a->num_kv_heads;
    const int width = a->max_blocks;
    // With fewer rows than SMs the scores take a grid over all pages; with many rows, or with few pages, a second
    // kernel costs more than it brings, unless a row's keys and page ids do not fit one CTA's shared memory.  Measured
    // with two kernels and with one, d = 128: 8 rows of 300 pages 7.7 and 7.8 us, of 600 8.2 and 10.4, 128 rows of 300
    // pages 12.3 and 8.6, of 600 17.4 and 16.0, 512 rows of 600 pages 53.7 and 38.1, of 200 33.5 and 20.8.  (So with about as
    // many rows as SMs one kernel would be as good up to some 700 pages; the rule is from before its loads had the registers.)
    const bool fits = key_stride(width) * 8 <= kSelSmem;
    plan->scored = !fits || (rows < device_sms() && width > 384);
    plan->room = plan->scored && key_stride(width) > kSortRoom ? kSortRoom : static_cast<int>(key_stride(width));
    // several CTAs of select_kernel can make a row's choice only if they do not share its keys
    plan->parts = 1;
    while (plan->scored && plan->room == key_stride(width) && plan->parts < 8 && rows * plan->parts * 2 <= device_sms()) plan->parts *= 2;
    // two scoring CTAs to an SM with equal work, unless that leaves them little
    int64_t tile = (rows * width + 2 * device_sms() - 1) / (2 * device_sms());
    tile = (tile + 15) / 16 * 16;
    plan->tile = static_cast<int>(tile < 64 ? 64 : (tile > kScoreTile ? kScoreTile : tile));
    TQ_NEED(rows * ((width + plan->tile - 1) / plan->tile) < (1ll << 31), TQ_ERR_UNSUPPORTED,
            "%s: too many (sequence, kv head) rows for max_blocks=%d", fn, width);
    plan->workspace_bytes =
        plan->scored ? static_cast<size_t>(rows) * (static_cast<size_t>(key_stride(width)) + (width + plan->tile - 1) / plan->tile) * 4 : 0;
    return TQ_OK;
}

template <typename T, int D>
tq_status launch_select(const SelectParams& p, int64_t rows, bool scored, cudaStream_t st) {
    const unsigned grid = static_cast<unsigned>(rows);
    if (!scored) {
        constexpr auto kern = select_kernel<T, D, false>;
        TQ_CUDA((prepare_kernel<kern>(kSelSmem)), "tq_select_pages: cudaFuncSetAttribute");
        TQ_CUDA(launch(kern, grid, 1, kScoreThreads, static_cast<size_t>(p.room) * 8, st, p), "tq_select_pages: launch");
        return TQ_OK;
    }
    constexpr auto kern = select_kernel<T, D, true>;
    TQ_CUDA((prepare_kernel<kern>(kSortRoom * 8)), "tq_select_pages: cudaFuncSetAttribute");
    const unsigned tiles = (p.width + p.tile - 1) / p.tile;
    TQ_CUDA(launch(score_kernel<T, D>, grid * tiles, 1, kScoreThreads, 0, st, p), "tq_select_pages: score launch");
    TQ_CUDA(launch(kern, grid, p.parts, kSortThreads, static_cast<size_t>(p.room) * 8, st, p), "tq_select_pages: launch");
    return TQ_OK;
}

}  // namespace

extern "C" tq_status tq_select_pages_workspace_bytes(const tq_select_args* a, size_t* bytes) {
    clear_error();
    TQ_NEED(bytes, TQ_ERR_INVALID_ARG, "tq_select_pages_workspace_bytes: bytes is NULL");
    *bytes = 0;
    SelectPlan plan;
    tq_status s = plan_select("tq_select_pages_workspace_bytes", a, &plan);
    if (s != TQ_OK) return s;
    *bytes = plan.workspace_bytes;
    return TQ_OK;
}

extern "C" tq_status tq_select_pages(const tq_select_args* a, void* stream) {
    clear_error();
    const char* fn = "tq_select_pages";
    SelectPlan plan;
    tq_status s = plan_select(fn, a, &plan);
    if (s != TQ_OK) return s;
    TQ_NEED(a->q && a->bounds && a->block_table && a->seq_lens && a->pages && a->lens, TQ_ERR_INVALID_ARG, "%s: NULL pointer in args", fn);
    TQ_NEED(plan.workspace_bytes == 0 || (a->workspace && a->workspace_bytes >= plan.workspace_bytes), TQ_ERR_INVALID_ARG,
            "%s: workspace of %zu bytes required (got %zu)", fn, plan.workspace_bytes, a->workspace ? a->workspace_bytes : static_cast<size_t>(0));
    TQ_NEED(aligned(a->q, 16) && aligned(a->bounds, 16), TQ_ERR_INVALID_ARG, "%s: q and bounds must be 16-byte aligned", fn);
    TQ_NEED(a->q_stride % 8 == 0 && a->q_stride >= 0, TQ_ERR_INVALID_ARG, "%s: q_stride must be a non-negative multiple of 8", fn);
    TQ_NEED(aligned(a->block_table, 4) && aligned(a->seq_lens, 4) && aligned(a->pages, 4) && aligned(a->lens, 4) && aligned(a->workspace, 16),
            TQ_ERR_INVALID_ARG, "%s: misaligned pointer in args", fn);
    SelectParams p;
    p.q = a->q;
    p.q_stride = a->q_stride;
    p.bounds = a->bounds;
    p.table = a->block_table;
    p.seq_lens = a->seq_lens;
    p.pages = a->pages;
    p.lens = a->lens;
    p.heads = a->num_kv_heads;
    p.group = a->num_q_heads / a->num_kv_heads;
    p.width = a->max_blocks;
    p.num_pages = a->num_pages;
    p.budget = a->budget;
    p.keep_first = a->keep_first;
    p.keep_last = a->keep_last;
    p.tile = plan.tile;
    p.room = plan.room;
    p.parts = plan.parts;
    const int64_t rows = static_cast<int64_t>(a->batch) * a->num_kv_heads;
    p.keys = static_cast<uint32_t*>(a->workspace);
    p.sizes = plan.scored ? reinterpret_cast<float*>(p.keys + rows * key_stride(p.width)) : nullptr;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    TQ_DISPATCH_TD(a->dtype, a->head_dim, launch_select, p, rows, plan.scored, st);
}

// -------------------------------------------------------------------------------------------- attend

namespace {

// A share is at least a row's own cost and a page for each warp.
template <int D>
constexpr int min_share() { return PagesCfg<D>::kRowCost + PagesCfg<D>::kWarps; }

// Short table rows are not split: a second launch takes longer than a CTA needs for them.  A CTA of four warps takes rows
// of up to 32 pages (d = 128, not split and split: 512 rows of 32 pages 26.5 and 29.5 us; d = 64, 512 rows of 64 30.9 and
// 28.1); one of eight, in calls that leave every row an SM, up to 48 (8 rows of 48 pages: d = 128 7.8 and 7.6, d = 64 5.7 and
// 6.9; of 64, d = 128: 9.4 and 7.6), or 64 if a split brings less than two SMs to a row (128 rows of 64: 10.1 and 12.8).
// At d = 256 eight warps' pages do not fit.
int direct_pages(int d, int64_t rows) {
    const int sms = device_sms();
    return d == 256 || rows > sms ? 32 : (2 * rows > sms ? 64 : 48);
}

struct PagesPlan {
    bool direct, wide;
    int ctas, rows_join;
    size_t meta_bytes, workspace_bytes;
};

tq_status plan_attend_pages(const char* fn, const tq_attend_pages_args* a, PagesPlan* plan) {
    TQ_NEED(a, TQ_ERR_INVALID_ARG, "%s: args is NULL", fn);
    tq_status s = check_heads(fn, a->batch, a->num_q_heads, a->num_kv_heads);
    if (s != TQ_OK) return s;
    if ((s = check_d_dtype(fn, a->head_dim, a->dtype)) != TQ_OK) return s;
    if ((s = check_pool(fn, a->num_pages, a->num_kv_heads)) != TQ_OK) return s;
    TQ_NEED(a->max_blocks >= 1 && a->max_blocks <= (1 << 26), TQ_ERR_INVALID_ARG, "%s: max_blocks=%d outside 1 .. 2^26", fn, a->max_blocks);
    TQ_NEED(a->selected == 0 || a->selected == 1, TQ_ERR_INVALID_ARG, "%s: selected=%d (0 or 1)", fn, a->selected);
    const int d = a->head_dim;
    const int row_cost = d == 64 ? PagesCfg<64>::kRowCost : d == 128 ? PagesCfg<128>::kRowCost : PagesCfg<256>::kRowCost;
    const int per_sm = d == 64 ? PagesCfg<64>::kCtasPerSm : d == 128 ? PagesCfg<128>::kCtasPerSm : PagesCfg<256>::kCtasPerSm;
    const int least = d == 64 ? min_share<64>() : d == 128 ? min_share<128>() : min_share<256>();
    const int64_t cost = static_cast<int64_t>(a->batch) * a->num_kv_heads * (a->max_blocks + row_cost);   // at most
    const int64_t slots = static_cast<int64_t>(device_sms()) * per_sm;
    const int64_t want = (cost + least - 1) / least;
    TQ_NEED(cost < (1ll << 31), TQ_ERR_UNSUPPORTED, "%s: batch=%d with %d kv heads and max_blocks=%d holds 2^31 pages or more", fn,
            a->batch, a->num_kv_heads, a->max_blocks);
    const int rows = a->batch * a->num_kv_heads;
    plan->direct = a->max_blocks <= direct_pages(d, rows);
    plan->wide = plan->direct && d != 256 && rows <= device_sms();
    const int shares = static_cast<int>(want < slots ? want : slots);
    plan->ctas = plan->direct ? rows : shares;
    // the join goes by rows if there are no more of them than shares
    plan->rows_join = !plan->direct && rows <= shares ? rows : 0;
    // past 32 pages a workspace is asked for whether or not this call is split, so that whether a caller has to provide one
    // depends on max_blocks alone
    plan->meta_bytes = a->max_blocks <= 32 ? 0 : static_cast<size_t>(shares) * sizeof(AttendPagesMeta);
    plan->workspace_bytes = a->max_blocks <= 32 ? 0 : plan->meta_bytes + static_cast<size_t>(shares) * 2 * (16 + 8 * d) * 4;
    return TQ_OK;
}

template <typename T, int D, bool WIDE>
cudaError_t launch_attend_main(const AttendPagesParams& p, int ctas, cudaStream_t st) {
    using C = PagesCfg<D, WIDE>;
    constexpr auto kern = attend_pages_kernel<T, D, WIDE>;
    const cudaError_t e = prepare_kernel<kern>(C::smem(8));
    return e != cudaSuccess ? e : launch(kern, ctas, 1, C::kThreads, C::smem(p.group), st, p);
}

template <typename T, int D>
tq_status launch_attend_pages(AttendPagesParams& p, int ctas, bool wide, cudaStream_t st) {
    p.min_share = min_share<D>();
    if constexpr (D != 256) {
        if (wide) TQ_CUDA((launch_attend_main<T, D, true>(p, ctas, st)), "tq_attend_pages: launch");
    }
    if (!wide) TQ_CUDA((launch_attend_main<T, D, false>(p, ctas, st)), "tq_attend_pages: launch");
    if (!p.direct && ctas > 1)
        TQ_CUDA(launch(attend_pages_join_kernel<D>, p.rows_join ? p.rows_join : ctas - 1, (p.group + p.join_heads - 1) / p.join_heads,
                       p.rows_join ? kJoinThreads : p.join_heads * D /* four slices */, 0, st, p),
                "tq_attend_pages: join launch");
    return TQ_OK;
}

}  // namespace

extern "C" tq_status tq_attend_pages_workspace_bytes(const tq_attend_pages_args* a, size_t* bytes) {
    clear_error();
    TQ_NEED(bytes, TQ_ERR_INVALID_ARG, "tq_attend_pages_workspace_bytes: bytes is NULL");
    *bytes = 0;
    PagesPlan plan;
    tq_status s = plan_attend_pages("tq_attend_pages_workspace_bytes", a, &plan);
    if (s != TQ_OK) return s;
    *bytes = plan.workspace_bytes;
    return TQ_OK;
}

extern "C" tq_status tq_attend_pages(const tq_attend_pages_args* a, void* stream) {
    clear_error();
    const char* fn = "tq_attend_pages";
    PagesPlan plan;
    tq_status s = plan_attend_pages(fn, a, &plan);
    if (s != TQ_OK) return s;
    TQ_NEED(a->q && a->k_pool && a->v_pool && a->block_table && a->seq_lens && a->out, TQ_ERR_INVALID_ARG, "%s: NULL pointer in args", fn);
    TQ_NEED(plan.workspace_bytes == 0 || (a->workspace && a->workspace_bytes >= plan.workspace_bytes), TQ_ERR_INVALID_ARG,
            "%s: workspace of %zu bytes required (got %zu)", fn, plan.workspace_bytes, a->workspace ? a->workspace_bytes : static_cast<size_t>(0));
    TQ_NEED(aligned(a->q, 16) && aligned(a->k_pool, 16) && aligned(a->v_pool, 16) && aligned(a->out, 16) && aligned(a->workspace, 16),
            TQ_ERR_INVALID_ARG, "%s: q, k_pool, v_pool, out and workspace must be 16-byte aligned", fn);
    TQ_NEED(aligned(a->block_table, 4) && aligned(a->seq_lens, 4), TQ_ERR_INVALID_ARG, "%s: block_table and seq_lens must be 4-byte aligned", fn);
    TQ_NEED(a->q_stride % 8 == 0 && a->q_stride >= 0, TQ_ERR_INVALID_ARG, "%s: q_stride must be a non-negative multiple of 8", fn);
    const int64_t dense = static_cast<int64_t>(a->num_kv_heads) * kPage * a->head_dim;
    TQ_NEED(a->k_page_stride % 8 == 0 && a->v_page_stride % 8 == 0 && a->k_page_stride >= dense && a->v_page_stride >= dense,
            TQ_ERR_INVALID_ARG, "%s: page strides must be multiples of 8 and at least num_kv_heads * 16 * head_dim", fn);
    TQ_NEED(!a->selected || (a->k_page_stride == dense && a->v_page_stride == dense), TQ_ERR_INVALID_ARG,
            "%s: selected pages need contiguous pools", fn);
    AttendPagesParams p;
    p.q = a->q;
    p.k_pool = a->k_pool;
    p.v_pool = a->v_pool;
    p.table = a->block_table;
    p.lens = a->seq_lens;
    p.out = a->out;
    p.meta = static_cast<AttendPagesMeta*>(a->workspace);
    p.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(a->workspace) + plan.meta_bytes);
    p.q_stride = a->q_stride;
    p.heads = a->num_kv_heads;
    p.group = a->num_q_heads / a->num_kv_heads;
    p.width = a->max_blocks;
    const float scale = (a->scale == 0.f) ? 1.0f / std::sqrt(static_cast<float>(a->head_dim)) : a->scale;
    p.scale_log2 = scale * 1.4426950408889634f;
    if (a->selected) {                 // a table row per (sequence, kv head) of head pages
        p.units = a->batch * a->num_kv_heads;
        p.mult = 1;
        p.num_ids = a->num_pages * a->num_kv_heads;
        p.k_page = p.v_page = static_cast<int64_t>(kPage) * a->head_dim;
    } else {                           // a table row per sequence, shared by its kv heads
        p.units = a->batch;
        p.mult = a->num_kv_heads;
        p.num_ids = a->num_pages;
        p.k_page = a->k_page_stride;
        p.v_page = a->v_page_stride;
    }
    p.direct = plan.direct;
    p.rows_join = plan.rows_join;
    // rows in many shares are joined by a CTA per head (or per few, so that the CTAs are resident together), those in
    // the few shares that many rows have by a CTA for 64 threads' worth of heads
    p.join_heads = 256 / a->head_dim;
    if (plan.rows_join) {
        p.join_heads = 1;
        while (p.join_heads < p.group && p.rows_join * ((p.group + p.join_heads - 1) / p.join_heads) > device_sms()) ++p.join_heads;
    }
    if (p.join_heads > p.group) p.join_heads = p.group;
    if (p.join_heads * a->head_dim / 4 > kJoinThreads) p.join_heads = kJoinThreads * 4 / a->head_dim;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    TQ_DISPATCH_TD(a->dtype, a->head_dim, launch_attend_pages, p, plan.ctas, plan.wide, st);
}
