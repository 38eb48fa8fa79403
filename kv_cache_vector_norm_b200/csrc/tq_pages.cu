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
cudaError_t prepare_kernel(int smem, bool wide_clusters) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load() & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && wide_clusters) e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) done.fetch_or(bit);
    return e;
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
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // a decode step's few slots are written by the planning CTA itself, a prefill's by a grid of their own
    const bool one = a->max_tokens <= 1024;
    plan_kernel<<<1, kPlanThreads, 0, st>>>(p, one);
    TQ_CUDA(cudaGetLastError(), "tq_plan_pages: launch");
    if (!one) {
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>((a->max_tokens + kSlotTile - 1) / kSlotTile));
        cfg.blockDim = dim3(kSlotTile);
        cfg.stream = st;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        TQ_CUDA(cudaLaunchKernelEx(&cfg, plan_slots_kernel, p), "tq_plan_pages: slot launch");
    }
    return TQ_OK;
}

// -------------------------------------------------------------------------------------------- append

namespace {

template <typename T, int D>
tq_status launch_append(const AppendParams& p, cudaStream_t st) {
    const int64_t warps = (p.n + p.tile - 1) / p.tile * p.heads;
    append_kernel<T, D><<<static_cast<unsigned>((warps + kAppendWarps - 1) / kAppendWarps), 32 * kAppendWarps, 0, st>>>(p);
    TQ_CUDA(cudaGetLastError(), "tq_append_pages: launch");
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
    // a decode step's tokens lie in pages of their own: one warp each; a prefill's fill whole pages
    p.tile = a->num_tokens * a->num_kv_heads <= 16384 ? 1 : 16;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    TQ_DISPATCH_TD(a->dtype, a->head_dim, launch_append, p, st);
}

// -------------------------------------------------------------------------------------------- select

namespace {

constexpr int kSelSmem = 200 << 10;
constexpr int kMaxCluster = 16;

template <typename T, int D>
tq_status launch_select(SelectParams& p, int batch, cudaStream_t st) {
    constexpr auto kern = select_kernel<T, D>;
    TQ_CUDA((prepare_kernel<kern>(kSelSmem, true)), "tq_select_pages: cudaFuncSetAttribute");
    const int64_t rows = static_cast<int64_t>(batch) * p.heads;
    const int cap = static_cast<int>((kSelSmem - select_smem(0, p.group, D)) / 8);
    // enough CTAs per row to cover the SMs, but at least 64 pages each, and as many as its pages need to fit
    int cs = 1;
    while (cs < kMaxCluster && (rows * cs < device_sms() && p.width / (2 * cs) >= 64)) cs *= 2;
    while (cs < kMaxCluster && (p.width + cs - 1) / cs > cap) cs *= 2;
    p.share_cap = (p.width + cs - 1) / cs;
    TQ_NEED(p.share_cap <= cap && p.share_cap < 65536, TQ_ERR_UNSUPPORTED, "tq_select_pages: max_blocks=%d (at most %d)", p.width,
            kMaxCluster * cap);
    TQ_NEED(rows * cs < (1ll << 31), TQ_ERR_UNSUPPORTED, "tq_select_pages: too many rows");
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cs;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(rows * cs));
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = select_smem(p.share_cap, p.group, D);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    TQ_CUDA(cudaLaunchKernelEx(&cfg, kern, p), "tq_select_pages: launch");
    return TQ_OK;
}

}  // namespace

extern "C" tq_status tq_select_pages(const tq_select_args* a, void* stream) {
    clear_error();
    const char* fn = "tq_select_pages";
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
    TQ_NEED(a->q && a->bounds && a->block_table && a->seq_lens && a->pages && a->lens, TQ_ERR_INVALID_ARG, "%s: NULL pointer in args", fn);
    TQ_NEED(aligned(a->q, 16) && aligned(a->bounds, 16), TQ_ERR_INVALID_ARG, "%s: q and bounds must be 16-byte aligned", fn);
    TQ_NEED(a->q_stride % 8 == 0 && a->q_stride >= 0, TQ_ERR_INVALID_ARG, "%s: q_stride must be a non-negative multiple of 8", fn);
    TQ_NEED(aligned(a->block_table, 4) && aligned(a->seq_lens, 4) && aligned(a->pages, 4) && aligned(a->lens, 4), TQ_ERR_INVALID_ARG,
            "%s: misaligned pointer in args", fn);
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
    p.share_cap = 0;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    TQ_DISPATCH_TD(a->dtype, a->head_dim, launch_select, p, a->batch, st);
}

// -------------------------------------------------------------------------------------------- attend

namespace {

constexpr int kMinPages = 4;           // pages a CTA takes at least: one per warp

struct PagesPlan {
    int ctas;
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
    const int64_t pages = static_cast<int64_t>(a->batch) * a->num_kv_heads * a->max_blocks;   // at most
    const int64_t slots = static_cast<int64_t>(device_sms()) * (a->head_dim == 256 ? PagesCfg<256>::kCtasPerSm : PagesCfg<128>::kCtasPerSm);
    const int64_t want = (pages + kMinPages - 1) / kMinPages;
    plan->ctas = static_cast<int>(want < slots ? want : slots);
    plan->meta_bytes = static_cast<size_t>(plan->ctas) * sizeof(AttendPagesMeta);
    plan->workspace_bytes = plan->meta_bytes + static_cast<size_t>(plan->ctas) * 2 * (16 + 8 * a->head_dim) * 4;
    return TQ_OK;
}

template <typename T, int D>
tq_status launch_attend_pages(const AttendPagesParams& p, int ctas, cudaStream_t st) {
    using C = PagesCfg<D>;
    constexpr auto kern = attend_pages_kernel<T, D>;
    TQ_CUDA((prepare_kernel<kern>(C::kSmem, false)), "tq_attend_pages: cudaFuncSetAttribute");
    kern<<<ctas, C::kThreads, C::kSmem, st>>>(p);
    TQ_CUDA(cudaGetLastError(), "tq_attend_pages: launch");
    if (ctas > 1) {
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(ctas - 1, p.group);
        cfg.blockDim = dim3(kJoinThreads);
        cfg.stream = st;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        TQ_CUDA(cudaLaunchKernelEx(&cfg, attend_pages_join_kernel<D>, p), "tq_attend_pages: join launch");
    }
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
    TQ_NEED(a->workspace && a->workspace_bytes >= plan.workspace_bytes, TQ_ERR_INVALID_ARG,
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
    p.min_pages = kMinPages;
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
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    TQ_DISPATCH_TD(a->dtype, a->head_dim, launch_attend_pages, p, plan.ctas, st);
}
