// Shared pieces of the paged 8-bit cache (iskv_page_plan, iskv_q8_append,
// iskv_q8_attention): launch descriptors, code conversions, small scans.
#pragma once

#include <atomic>

#include "iskv_internal.cuh"
#include "tc_util.cuh"

namespace iskv {
namespace q8 {

constexpr int kPage = ISKV_PAGE;      // tokens per page
constexpr int kMaxBatch = 8192;       // requests per call
constexpr int kStepTokens = 32;       // tokens a warp of the split kernel takes at a time
constexpr float kMinAmax = 5.421010862427522e-20f;   // 2^-64: below it a block counts as zeros
constexpr float kLog2e = 1.4426950408889634f;
// Softmax weights are kept times 2^kWeightShift, so that their 16-bit form
// stays clear of fp16's subnormal range down to 2^-28 of the largest one.
constexpr float kWeightShift = 14.f;

// Raises a kernel's dynamic shared memory limit once per device instead of at
// every launch (launch latency is most of a small call).
struct SmemOnce {
    std::atomic<uint64_t> done{0};
    template <typename F>
    cudaError_t set(F* kernel, size_t bytes) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
        if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
        return e;
    }
};

// Launches a kernel that may come up while the one before it in the stream ends.
// It calls after_previous() before it touches memory, which waits for that
// kernel's end and its writes.  (What it reads may be written until then, so none
// of it is read-only for the kernel's whole life, as __ldg would ask.)  Kernels but the joins call let_next() at once, so
// that what follows them need not wait for its own launch. (A grid that is up
// while a join's many blocks run slows them by more than its launch.) A page plan and eight layers of
// append and attention, 1000 keys a request: batch 1 119 -> 113 us as a graph,
// batch 64 394 -> 364 us launched one by one (387 -> 386 as a graph).
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, int cluster, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 0 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
__device__ __forceinline__ void let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

struct AppendArgs {
    const void* x[2];          // k, v
    int64_t stride[2];         // elements from token to token
    void* store[2];
    float* scale[2];
    const int32_t* slots;
    int32_t* status;
    int64_t n;
    int pages, kv_heads;
    int window;                // tokens whose runs one CTA looks after
};

struct AttnArgs {
    const void* q;
    void* out;
    const uint8_t* k;
    const uint8_t* v;
    const float* k_scale;
    const float* v_scale;
    const int32_t* table;
    const int32_t* lens;
    const int32_t* cu;
    const int32_t* prefix;
    const float* slopes;
    int64_t tokens, q_stride;
    int batch, width, pages, kv_heads, g;
    int window;
    float scale, cap, cap_inv;
    int tq;                    // query tokens per row tile
    int ctas;                  // CTAs
    int whole;                 // split kernel: a CTA takes whole items, none is joined across CTAs
    float* part;               // partial results of warps and CTAs
    float* ml;                 // their running maxima and sums
    int* status;               // sticky, or nullptr
    int* meta;                 // per CTA: what it leaves to be joined
    long long wait_cycles;     // clock cycles that a wait may take
    int patient;               // whether a try of a long wait may sleep (0: waits that must run out do)
};

// One try of a wait for the phase of a barrier.
__device__ __forceinline__ bool try_phase(const AttnArgs& p, uint64_t* bar, uint32_t parity) {
    if (p.patient) return tc::mbar_try_wait(bar, parity);
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(tc::smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// ---------------------------------------------------------------------------
// Codes to fp16, two at a time, exactly.
// ---------------------------------------------------------------------------
template <int CODE>
struct Codes;

template <>
struct Codes<ISKV_CODE_INT8> {
    // 1024 + (c + 128) is an fp16 whose low byte is c with its top bit
    // flipped; subtracting 1152 leaves c.
    static __device__ __forceinline__ uint32_t bias(uint32_t x) { return x ^ 0x80808080u; }
    static __device__ __forceinline__ uint32_t sub(uint32_t x) {
        const __half2 k = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
        const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&x), k);
        return *reinterpret_cast<const uint32_t*>(&r);
    }
    static __device__ __forceinline__ uint32_t lo(uint32_t biased) {
        return sub(__byte_perm(biased, 0x64646464u, 0x4140));
    }
    static __device__ __forceinline__ uint32_t hi(uint32_t biased) {
        return sub(__byte_perm(biased, 0x64646464u, 0x4342));
    }
};

template <>
struct Codes<ISKV_CODE_E4M3> {
    static __device__ __forceinline__ uint32_t bias(uint32_t x) { return x; }
    static __device__ __forceinline__ uint32_t cvt(uint16_t x) {
        uint32_t r;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(x));
        return r;
    }
    static __device__ __forceinline__ uint32_t lo(uint32_t x) { return cvt((uint16_t)(x & 0xffffu)); }
    static __device__ __forceinline__ uint32_t hi(uint32_t x) { return cvt((uint16_t)(x >> 16)); }
};

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float lg2(float x) {
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// cap * tanh(x / cap), off by at most 2^-20 of x; inv: 1 / cap (host: finite).
// Below half the cap it is x times a polynomial in (x / cap)^2 (minimax of the
// relative error, 2^-26; 2^-23 with its roundings), which is exact for caps far
// above x; from there on cap (1 - 2 / (1 + e^(2t))), whose error of a few 2^-23 of
// the cap is one of 2^-21 of tanh there, and whose limits are exact (e^(2t)
// reaches 0 and infinity).
constexpr float kCapLow = 0.5f;
__device__ __forceinline__ float capped_low(float x, float inv) {
    const float t = x * inv, u = t * t;
    float y = fmaf(0.01724136434495449f, u, -0.05304544046521187f);
    y = fmaf(y, u, 0.13325878977775574f);
    y = fmaf(y, u, -0.333331435918808f);
    return x * fmaf(y, u, 1.f);
}
__device__ __forceinline__ float capped(float x, float cap, float inv) {
    const float t = x * inv;
    float y = capped_low(x, inv);
    if (!(fabsf(t) < kCapLow)) y = cap * (1.f - __fdividef(2.f, 1.f + ex2(2.f * kLog2e * t)));
    return y;
}

// ---------------------------------------------------------------------------
// What a request's queries see, in steps of `kStep` tokens.
// ---------------------------------------------------------------------------
template <int kStep>
struct Seen {
    int first, n, len;      // first query row, queries, stored tokens
    int pre;                // prefix tokens (0 .. len)
    int a, lo;              // steps 0 .. a-1 and from lo on hold what is seen
    int steps;              // number of them
    __device__ __forceinline__ int step_of(int i) const { return i < a ? i : i - a + lo; }
};

template <int kStep>
__device__ __forceinline__ Seen<kStep> seen_of(const AttnArgs& p, int b) {
    Seen<kStep> r;
    const int c0 = p.cu[b];
    const int64_t c1 = p.cu[b + 1];
    const int64_t top = c1 < p.tokens ? c1 : p.tokens;
    r.first = c0 < 0 ? 0 : c0;
    r.n = top > r.first ? (int)(top - r.first) : 0;
    int64_t len = p.lens[b];
    const int64_t room = (int64_t)p.width * kPage;
    len = len < 0 ? 0 : (len > room ? room : len);
    r.len = (int)len;
    r.pre = 0;
    if (p.prefix) {
        const int f = p.prefix[b];
        r.pre = f < 0 ? 0 : (f > r.len ? r.len : f);
    }
    r.a = 0;
    r.lo = 0;
    if (p.window > 0) {
        int64_t w0 = (int64_t)r.len - r.n - p.window + 1;   // first key the first query sees
        if (w0 < 0) w0 = 0;
        r.lo = (int)(w0 / kStep);
        r.a = (r.pre + kStep - 1) / kStep;
        if (r.a > r.lo) r.a = r.lo;
    }
    const int end = (r.len + kStep - 1) / kStep;
    r.steps = r.a + (end > r.lo ? end - r.lo : 0);
    if (r.n == 0) r.steps = 0;
    else if (r.steps == 0) r.steps = 1;   // nothing stored: one empty step, so that zeros are written
    return r;
}

cudaError_t launch_page_plan(const iskv_page_plan_args& a, cudaStream_t s);
cudaError_t launch_q8_append(const AppendArgs& a, int code, int dtype, cudaStream_t s);
cudaError_t launch_q8_prompt(const AttnArgs& a, int code, cudaStream_t s);
cudaError_t launch_q8_rows(const AttnArgs& a, int code, bool f32, int tiles8, cudaStream_t s);

// Warps per CTA of the split kernel for row tiles of 8 * tiles8 rows; its
// workspace holds two partials of every warp and two of the CTA.
constexpr int rows_warps(int tiles8, bool f32) { return tiles8 == 1 && !f32 ? 12 : 8; }
constexpr int rows_parts(int tiles8, bool f32) { return 2 * rows_warps(tiles8, f32) + 2; }

constexpr int kPromptRows = 256;   // query rows that the prompt kernel takes together
constexpr int kMetaBytes = 32;     // per CTA, either kernel

}  // namespace q8
}  // namespace iskv
