// C ABI of the paged 8-bit cache (declared in include/iskv.h): argument checks,
// the choice of kernel, launches.  Nothing is allocated or kept here.
#include <nvtx3/nvToolsExt.h>

#include <cfloat>
#include <cmath>
#include <cstdlib>

#include "q8_common.cuh"

using namespace iskv;

namespace {

struct TraceRange {
    explicit TraceRange(const char* name) { nvtxRangePushA(name); }
    ~TraceRange() { nvtxRangePop(); }
};

// True for memory that kernels on device `dev` may use directly.
bool on_device(const void* p, int dev) {
    cudaPointerAttributes at;
    if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    if (at.type == cudaMemoryTypeManaged) return true;
    return at.type == cudaMemoryTypeDevice && at.device == dev;
}

bool all_on_device(const void* const* ptrs, int n) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    for (int i = 0; i < n; ++i)
        if (ptrs[i] && !on_device(ptrs[i], dev)) return false;
    return true;
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

int check_store(const iskv_q8_pages* s) {
    if (!s || s->pages < 1 || s->kv_heads < 1 || (int64_t)s->pages * ISKV_PAGE > INT32_MAX ||
        (int64_t)s->pages * s->kv_heads > INT32_MAX)
        return ISKV_ERR_INVALID_ARG;
    if (s->code != ISKV_CODE_INT8 && s->code != ISKV_CODE_E4M3) return ISKV_ERR_INVALID_ARG;
    if (s->head_dim != kHeadDim || s->page != ISKV_PAGE || s->kv_heads > 65535) return ISKV_ERR_UNSUPPORTED;
    if (!s->k || !s->v || !s->k_scale || !s->v_scale) return ISKV_ERR_INVALID_ARG;
    if (!aligned(s->k, 16) || !aligned(s->v, 16) || !aligned(s->k_scale, 4) || !aligned(s->v_scale, 4))
        return ISKV_ERR_INVALID_ARG;
    return ISKV_OK;
}

int elem_bytes(int dtype) { return dtype == ISKV_BF16 ? 2 : 4; }

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) {
        cudaGetLastError();
        return 148;
    }
    return n;
}

// Clock cycles a pipeline wait of the attention kernels may take before the call
// gives up with DEVICE_TIMEOUT; tests shorten it through the environment to make
// waits run out on purpose (ISKV_TEST_PIPELINE_WAIT_CYCLES, read at the first call).
long long wait_cycles() {
    static const long long w = [] {
        const char* e = std::getenv("ISKV_TEST_PIPELINE_WAIT_CYCLES");
        const long long n = e ? std::atoll(e) : 0;
        return n > 0 ? n : tc::kWaitCycles;
    }();
    return w;
}

// Row tiles of the split kernel in eights of rows.  Several tiles of a request
// read the same keys from L2, and one tile's code is the faster: two pay only for
// long fp32 prompts (6 requests of 9000 tokens, 3 heads a group: 2 KV heads: 48 rows
// 48 us either way, 192 rows 142 against 103; 8 KV heads: 148 against 122 and 528
// against 339).
int row_tiles8(int g, int max_new, int dtype) { return dtype == ISKV_F32 && (int64_t)max_new * g > 64 ? 2 : 1; }

// Whether the split kernel gives whole (request, head, tile) items to its CTAs,
// so that no second launch has to join parts: where requests are very short, or
// short and many.  (8 KV heads, requests as long as the table; one launch
// against two, when the rule was chosen: 1 request of 64 tokens 8.9 us against 11.2,
// of 512 14.8 against 11.9; 64 requests of 512 26.6 against 28.5, ragged ones of up
// to 1024 36 against 34; with the rule now 8.8, 12.1, 28.3 and 34.4.)
bool whole_items(int width, int batch, int kv_heads, int ctas) {
    return width <= 2 || (width <= 8 && (int64_t)batch * kv_heads >= 2 * (int64_t)ctas);
}

int64_t rows_floats(int ctas, int tiles8, int dtype) {
    return (int64_t)ctas * q8::rows_parts(tiles8, dtype == ISKV_F32) * 8 * tiles8 * (kHeadDim + 2);
}

int64_t prompt_floats(int ctas) { return (int64_t)ctas * 2 * q8::kPromptRows * (kHeadDim + 2); }

// Query rows per KV head up to which the split kernel takes a request: the
// tcgen05 kernel turns every code into an operand whatever the rows, the split
// kernel goes over the codes once per 8 rows (8 KV heads, 4 heads a group,
// 16K tokens: 32 rows 38 us against 40, 64 rows 57 against 41; 32 requests of 8K
// tokens: 234 against 277 and 406 against 278).
constexpr int64_t kPromptMinRows = 32;

bool is_prompt(int g, int max_new, int dtype) { return dtype == ISKV_BF16 && (int64_t)max_new * g > kPromptMinRows; }

}  // namespace

extern "C" {

int iskv_page_plan(const iskv_page_plan_args* a, void* stream) {
    TraceRange trace_("iskv_page_plan");
    if (!a || a->batch < 0 || a->width < 1 || a->pages < 1 || a->tokens < 0 ||
        (int64_t)a->pages * ISKV_PAGE > INT32_MAX || (int64_t)a->width * ISKV_PAGE > INT32_MAX)
        return ISKV_ERR_INVALID_ARG;
    if (a->batch > q8::kMaxBatch) return ISKV_ERR_UNSUPPORTED;
    if (!a->free_pages || !a->n_free || !a->cu || !a->n_free_out || !a->status) return ISKV_ERR_INVALID_ARG;
    if (a->batch > 0 && (!a->lens || !a->add || !a->table || !a->lens_out)) return ISKV_ERR_INVALID_ARG;
    if (a->tokens > 0 && !a->slots) return ISKV_ERR_INVALID_ARG;
    const void* ptrs[] = {a->lens, a->add, a->table, a->free_pages, a->n_free, a->lens_out, a->cu, a->slots,
                          a->n_free_out, a->status};
    for (const void* p : ptrs)
        if (!aligned(p, 4)) return ISKV_ERR_INVALID_ARG;
    if (!all_on_device(ptrs, 10)) return ISKV_ERR_INVALID_ARG;
    return q8::launch_page_plan(*a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? ISKV_OK : ISKV_ERR_CUDA;
}

int iskv_q8_append(const iskv_q8_pages* store, const void* k, const void* v, int dtype, int64_t k_stride,
                   int64_t v_stride, int64_t n, const int32_t* slots, int32_t* status, void* stream) {
    TraceRange trace_("iskv_q8_append");
    const int rc = check_store(store);
    if (rc != ISKV_OK) return rc;
    if (n < 0 || n > INT32_MAX || (dtype != ISKV_F32 && dtype != ISKV_BF16)) return ISKV_ERR_INVALID_ARG;
    if (n == 0) return ISKV_OK;
    const int64_t per16 = 16 / elem_bytes(dtype), row = (int64_t)store->kv_heads * kHeadDim;
    if (!k || !v || !slots || !aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4) || !aligned(status, 4))
        return ISKV_ERR_INVALID_ARG;
    for (int64_t st : {k_stride, v_stride})
        if (n > 1 && (st % per16 != 0 || st < row)) return ISKV_ERR_INVALID_ARG;   // (a single row has no next one)
    const void* ptrs[] = {store->k, store->v, store->k_scale, store->v_scale, k, v, slots, status};
    if (!all_on_device(ptrs, 8)) return ISKV_ERR_INVALID_ARG;
    q8::AppendArgs a{};
    a.x[0] = k;
    a.x[1] = v;
    a.stride[0] = k_stride;
    a.stride[1] = v_stride;
    a.store[0] = store->k;
    a.store[1] = store->v;
    a.scale[0] = store->k_scale;
    a.scale[1] = store->v_scale;
    a.slots = slots;
    a.status = status;
    a.n = n;
    a.pages = store->pages;
    a.kv_heads = store->kv_heads;
    // one token per CTA while that gives up to 16 CTAs per SM, then more
    const int64_t ctas = n * store->kv_heads * 2, want = (int64_t)16 * sm_count();
    a.window = 1;
    while (a.window < ISKV_PAGE && ctas / a.window > want) a.window *= 2;
    return q8::launch_q8_append(a, store->code, dtype, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? ISKV_OK : ISKV_ERR_CUDA;
}

int64_t iskv_q8_workspace(int32_t q_heads, int32_t kv_heads, int64_t tokens, int32_t max_new, int32_t dtype) {
    if (q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0 || q_heads / kv_heads > kMaxGroup || tokens < 0 ||
        max_new < 1 || (dtype != ISKV_F32 && dtype != ISKV_BF16))
        return -1;
    const int ctas = sm_count();
    const int g = q_heads / kv_heads;
    if (is_prompt(g, max_new, dtype)) return prompt_floats(ctas) * 4 + (int64_t)ctas * q8::kMetaBytes;
    return rows_floats(ctas, row_tiles8(g, max_new, dtype), dtype) * 4 + (int64_t)ctas * q8::kMetaBytes;
}

int iskv_q8_attention(const iskv_q8_pages* store, const iskv_q8_attention_args* a, void* stream) {
    TraceRange trace_("iskv_q8_attention");
    const int rc = check_store(store);
    if (rc != ISKV_OK) return rc;
    if (!a || a->batch < 0 || a->width < 1 || a->q_heads < 1 || a->q_heads % store->kv_heads != 0 || a->tokens < 0 ||
        a->tokens > INT32_MAX || a->max_new < 1 || a->window < 0 || (int64_t)a->width * ISKV_PAGE > INT32_MAX ||
        (a->dtype != ISKV_F32 && a->dtype != ISKV_BF16))
        return ISKV_ERR_INVALID_ARG;
    if (!(a->scale > 0.f) || !(a->scale < INFINITY) || !(a->cap >= 0.f) || !(a->cap < INFINITY)) return ISKV_ERR_INVALID_ARG;
    const int g = a->q_heads / store->kv_heads;
    if (g > kMaxGroup || a->batch > q8::kMaxBatch) return ISKV_ERR_UNSUPPORTED;
    if (a->batch == 0 || a->tokens == 0) return ISKV_OK;
    if (!a->q || !a->out || !a->table || !a->lens || !a->cu || !a->workspace) return ISKV_ERR_INVALID_ARG;
    if (!aligned(a->q, 16) || !aligned(a->out, 16) || !aligned(a->workspace, 16) || !aligned(a->table, 4) ||
        !aligned(a->lens, 4) || !aligned(a->cu, 4) || !aligned(a->prefix, 4) || !aligned(a->slopes, 4) || !aligned(a->status, 4))
        return ISKV_ERR_INVALID_ARG;
    if (a->tokens > 1 &&
        (a->q_stride % (16 / elem_bytes(a->dtype)) != 0 || a->q_stride < (int64_t)a->q_heads * kHeadDim))
        return ISKV_ERR_INVALID_ARG;
    const int64_t row = (int64_t)a->q_heads * kHeadDim, es = elem_bytes(a->dtype);
    if (overlap(a->q, ((a->tokens - 1) * a->q_stride + row) * es, a->out, a->tokens * row * es)) return ISKV_ERR_INVALID_ARG;
    const void* ptrs[] = {store->k, store->v, store->k_scale, store->v_scale, a->q, a->out, a->table, a->lens, a->cu,
                          a->prefix, a->slopes, a->workspace, a->status};
    if (!all_on_device(ptrs, 13)) return ISKV_ERR_INVALID_ARG;
    if (a->workspace_bytes < iskv_q8_workspace(a->q_heads, store->kv_heads, a->tokens, a->max_new, a->dtype))
        return ISKV_ERR_CAPACITY;
    q8::AttnArgs p{};
    p.q = a->q;
    p.out = a->out;
    p.k = static_cast<const uint8_t*>(store->k);
    p.v = static_cast<const uint8_t*>(store->v);
    p.k_scale = store->k_scale;
    p.v_scale = store->v_scale;
    p.table = a->table;
    p.lens = a->lens;
    p.cu = a->cu;
    p.prefix = a->prefix;
    p.slopes = a->slopes;
    p.tokens = a->tokens;
    p.q_stride = a->q_stride;
    p.batch = a->batch;
    p.width = a->width;
    p.pages = store->pages;
    p.kv_heads = store->kv_heads;
    p.g = g;
    p.window = a->window;
    p.scale = a->scale;
    p.cap = a->cap;
    p.cap_inv = a->cap > 0.f ? std::fmin(1.f / a->cap, FLT_MAX) : 0.f;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int tiles8 = row_tiles8(g, a->max_new, a->dtype);
    const bool prompt = is_prompt(g, a->max_new, a->dtype);
    p.tq = (prompt ? q8::kPromptRows / 2 : 8 * tiles8) / g;
    p.ctas = sm_count();
    const int64_t parts = (int64_t)p.ctas * (prompt ? 2 * q8::kPromptRows : q8::rows_parts(tiles8, a->dtype == ISKV_F32) * 8 * tiles8);
    p.part = static_cast<float*>(a->workspace);
    p.ml = p.part + parts * kHeadDim;
    p.meta = reinterpret_cast<int*>(p.ml + parts * 2);
    p.status = a->status;
    p.wait_cycles = wait_cycles();
    p.patient = p.wait_cycles >= tc::kWaitCycles;
    p.whole = whole_items(a->width, a->batch, store->kv_heads, p.ctas);
    if (prompt)
        return q8::launch_q8_prompt(p, store->code, s) == cudaSuccess ? ISKV_OK : ISKV_ERR_CUDA;
    return q8::launch_q8_rows(p, store->code, a->dtype == ISKV_F32, tiles8, s) == cudaSuccess ? ISKV_OK : ISKV_ERR_CUDA;
}

}  // extern "C"
