// iskv_q8_append: new K and V rows as 8-bit codes with one scale per page and
// KV head.
//
// A run is the rows of one call that land in one page.  A CTA looks after a
// window of tokens for one head, of K or of V: its threads compare each slot
// with the one before, which finds all runs that start in the window and their
// lengths at once, and then takes them one by one.  The rows of a run (at most
// 64 x 128) stay in registers, in their own type, between the pass that finds
// the largest value and the pass that codes them, so each element is read once
// and its code written once.  Only where a run continues a page and needs a
// larger scale are the page's earlier codes read and coded again.
//
// int8 codes are rint(x / s).  The quotient is taken as a product with 1 / s,
// which is off by less than 2^-15 for |x / s| <= 127: only where that could
// move it across a half is the division done.  e4m3 scales are powers of two,
// and the product is the quotient.
//
// Bound by DRAM for prompts (3 bytes per bf16 element: 16K tokens of 8 heads in
// 18 us in a graph, 5.6 TB/s, 20 one by one) and by launch and load latency for single tokens (64 of them
// in 4.4 us).  Finding the runs by one comparison per thread instead of a loop
// over the window, and the quotients by products, were 100 -> 26 us of the 16K
// tokens; magnitudes compared as integers 26 -> 18.
#include "q8_common.cuh"

namespace iskv {
namespace q8 {

namespace {

constexpr int kThreads = 128;
constexpr int kPasses = kPage * kHeadDim / (kThreads * 8);   // 8: 8 elements per thread and pass

// 8 elements as they are stored.
template <typename T> struct Raw;
template <>
struct Raw<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = *reinterpret_cast<const float4*>(p);
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    // the largest magnitude's fp32 bits: they order like the values, with
    // infinity and NaN above all numbers
    __device__ __forceinline__ uint32_t top() const {
        const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
        return m;
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
};
template <>
struct Raw<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ uint32_t top() const {
        const uint32_t k = 0x7fff7fffu;
        const uint32_t m = __vmaxu2(__vmaxu2(a.x & k, a.y & k), __vmaxu2(a.z & k, a.w & k));
        return max(m & 0xffff0000u, m << 16);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};

// The scale that covers values up to `top`.
template <int CODE>
__device__ __forceinline__ float scale_of(float top) {
    if (!(top >= kMinAmax)) return 0.f;
    if (CODE == ISKV_CODE_INT8) return __fmul_rn(top, 1.f / 127.f);
    // 448 = 1.75 * 2^8: top = m 2^x with m in [1, 2) needs 2^(x - 8), or the
    // next power where m > 1.75
    const uint32_t u = __float_as_uint(top);
    const int e = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float((uint32_t)e << 23);
}

// Codes of 8 quotients x / s, s > 0, with inv = 1 / s.
constexpr float kMagic = 12582912.f;   // 1.5 * 2^23: adding it rounds to a whole number, half to even
template <int CODE>
__device__ __forceinline__ uint2 code8(float (&v)[8], float s, float inv) {
    if constexpr (CODE == ISKV_CODE_INT8) {
        float y[8], near = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = __fmul_rn(v[e], inv);
            y[e] = __fadd_rn(x, kMagic);
            near = fmaxf(near, fabsf(__fsub_rn(x, __fsub_rn(y[e], kMagic))));
        }
        if (near > 0.4999f) {   // some product may be on the wrong side of a half
#pragma unroll 1
            for (int e = 0; e < 8; ++e) {
                const float x = __fdiv_rn(v[0], s);
                const float z = __fadd_rn(fminf(fmaxf(x, -127.f), 127.f), kMagic);
#pragma unroll
                for (int k = 0; k < 7; ++k) { v[k] = v[k + 1]; y[k] = y[k + 1]; }
                y[7] = z;
            }
        }
        uint32_t b[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) b[e] = __float_as_uint(y[e]);
        return make_uint2(__byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410),
                          __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410));
    }
    else {
        uint16_t c[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c[e]) : "f"(__fmul_rn(v[2 * e + 1], inv)), "f"(__fmul_rn(v[2 * e], inv)));
        return make_uint2(c[0] | ((uint32_t)c[1] << 16), c[2] | ((uint32_t)c[3] << 16));
    }
}

// Values f c of 4 codes as codes again (0 <= f <= 1).
template <int CODE>
__device__ __forceinline__ uint32_t recode4(const float (&u)[4], float f) {
    float x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = __fmul_rn(u[e], f);
    if (CODE == ISKV_CODE_INT8) {
        uint32_t b[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) b[e] = __float_as_uint(__fadd_rn(x[e], kMagic));
        return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    }
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x[1]), "f"(x[0]));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x[3]), "f"(x[2]));
    return lo | ((uint32_t)hi << 16);
}

template <int CODE>
__device__ __forceinline__ void decode4(uint32_t x, float (&v)[4]) {
    const uint32_t b = Codes<CODE>::bias(x);
    const uint32_t l = Codes<CODE>::lo(b), h = Codes<CODE>::hi(b);
    const float2 fl = __half22float2(*reinterpret_cast<const __half2*>(&l));
    const float2 fh = __half22float2(*reinterpret_cast<const __half2*>(&h));
    v[0] = fl.x; v[1] = fl.y; v[2] = fh.x; v[3] = fh.y;
}

template <int CODE, typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 8 : 5) q8_append_kernel(const AppendArgs p) {
    let_next();
    after_previous();
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int head = blockIdx.y, which = blockIdx.z;
    const T* x = static_cast<const T*>(which ? p.x[1] : p.x[0]);
    const int64_t stride = which ? p.stride[1] : p.stride[0];
    uint8_t* store = static_cast<uint8_t*>(which ? p.store[1] : p.store[0]);
    float* scale = which ? p.scale[1] : p.scale[0];
    const int64_t t0 = (int64_t)blockIdx.x * p.window;
    const int64_t n_slots = (int64_t)p.pages * kPage;
    __shared__ float s_top[kThreads / 32];
    __shared__ uint32_t s_break[kThreads / 32];   // tokens t0 + 0 .. 127: it does not go on where the one before ended
    __shared__ uint32_t s_start[2];               // tokens of the window where a run starts
    __shared__ int s_slot[kPage];

    {
        const int64_t i = t0 + t;
        const bool in = i < p.n;
        const int64_t slot = in ? p.slots[i] : -1;
        const int64_t before = in && i > 0 ? p.slots[i - 1] : -1;
        const bool good = slot >= 0 && slot < n_slots;
        if (in && t < p.window && !good && slot != -1 && p.status) atomicMin(p.status, ISKV_ERR_INVALID_ARG);
        const uint32_t m = __ballot_sync(0xffffffffu, !good || slot % kPage == 0 || before != slot - 1);
        const uint32_t g = __ballot_sync(0xffffffffu, good && t < p.window);
        if (lane == 0) {
            s_break[warp] = m;
            if (warp < 2) s_start[warp] = m & g;
        }
        if (t < kPage) s_slot[t] = (int)slot;
    }
    __syncthreads();
#pragma unroll 1
    for (uint64_t todo = s_start[0] | (uint64_t)s_start[1] << 32; todo != 0; todo &= todo - 1) {   // uniform over the CTA
        const int j = __ffsll((long long)todo) - 1;
        const int64_t i = t0 + j, slot = s_slot[j];
        const int row0 = (int)(slot % kPage);
        // rows of the run: up to the next break (within 64 tokens, as the page ends)
        int n;
        {
            const int a = j + 1;
            uint32_t m = a < 128 ? s_break[a >> 5] >> (a & 31) : 1u;
            n = a;
            if (m == 0u) {
                int w = (a >> 5) + 1;
                while (w < kThreads / 32 && s_break[w] == 0u) ++w;
                n = w < kThreads / 32 ? 32 * w + __ffs(s_break[w]) - 1 : 128;
            } else {
                n = a + __ffs(m) - 1;
            }
            n = min(n - j, kPage - row0);
        }

        // 16 threads per row, 8 rows per pass
        const int col = (t & 15) * 8;
        Raw<T> v[kPasses];
#pragma unroll
        for (int s = 0; s < kPasses; ++s) {
            const int r = s * (kThreads / 16) + (t >> 4);
            if (r < n) v[s].load(x + (i + r) * stride + head * kHeadDim + col);
            else v[s].zero();
        }
        uint32_t bits = 0;
#pragma unroll
        for (int s = 0; s < kPasses; ++s) bits = max(bits, v[s].top());
        if (bits >= 0x7f800000u) {   // infinities and NaN are stored as zeros and do not count
            if (p.status) atomicMin(p.status, ISKV_ERR_RANGE);
            float m = 0.f;
#pragma unroll 1
            for (int s = 0; s < kPasses; ++s) {
                const int r = s * (kThreads / 16) + (t >> 4);
                if (r >= n) continue;
                Raw<T> w;
                w.load(x + (i + r) * stride + head * kHeadDim + col);
                float u[8];
                w.get(u);
#pragma unroll
                for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(u[e]) < INFINITY ? fabsf(u[e]) : 0.f);
            }
            bits = __float_as_uint(m) | 0x80000000u;   // (finite: the top bit marks the thread)
        }
        const bool dirty = bits >> 31;
        const uint32_t most = __reduce_max_sync(0xffffffffu, bits & 0x7fffffffu);
        if (lane == 0) s_top[warp] = __uint_as_float(most);
        const int64_t block = (slot / kPage) * p.kv_heads + head;
        const float before = row0 > 0 ? scale[block] : 0.f;
        __syncthreads();   // every thread has read the old scale
        float top = s_top[0];
#pragma unroll
        for (int w = 1; w < kThreads / 32; ++w) top = fmaxf(top, s_top[w]);
        const float now = fmaxf(before, scale_of<CODE>(top));
        uint8_t* base = store + block * (kPage * kHeadDim);
        if (t == 0) scale[block] = now;
        // the page's earlier rows, where their scale has grown
        if (row0 > 0 && now > before) {
            const float f = __fdiv_rn(before, now);
            for (int r = t >> 4; r < row0; r += kThreads / 16) {
                uint2* at = reinterpret_cast<uint2*>(base + r * kHeadDim + col);
                uint2 c = *at;
                float u[4];
                decode4<CODE>(c.x, u);
                c.x = recode4<CODE>(u, f);
                decode4<CODE>(c.y, u);
                c.y = recode4<CODE>(u, f);
                *at = c;
            }
        }
        const float inv = now > 0.f ? __fdiv_rn(1.f, now) : 0.f;
#pragma unroll
        for (int s = 0; s < kPasses; ++s) {
            const int r = s * (kThreads / 16) + (t >> 4);
            if (r >= n) continue;
            uint2 c = make_uint2(0u, 0u);
            if (now > 0.f) {
                float u[8];
                v[s].get(u);
                if (dirty) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) u[e] = fabsf(u[e]) < INFINITY ? u[e] : 0.f;
                }
                c = code8<CODE>(u, now, inv);
            }
            *reinterpret_cast<uint2*>(base + (row0 + r) * kHeadDim + col) = c;
        }
        __syncthreads();   // s_top is free again
    }
}

}  // namespace

cudaError_t launch_q8_append(const AppendArgs& a, int code, int dtype, cudaStream_t s) {
    if (a.n == 0) return cudaSuccess;
    const dim3 grid((unsigned)((a.n + a.window - 1) / a.window), a.kv_heads, 2);
    if (code == ISKV_CODE_INT8) {
        if (dtype == ISKV_F32) return launch_early(q8_append_kernel<ISKV_CODE_INT8, float>, grid, kThreads, 0, s, 0, a);
        else return launch_early(q8_append_kernel<ISKV_CODE_INT8, __nv_bfloat16>, grid, kThreads, 0, s, 0, a);
    } else {
        if (dtype == ISKV_F32) return launch_early(q8_append_kernel<ISKV_CODE_E4M3, float>, grid, kThreads, 0, s, 0, a);
        else return launch_early(q8_append_kernel<ISKV_CODE_E4M3, __nv_bfloat16>, grid, kThreads, 0, s, 0, a);
    }
}

}  // namespace q8
}  // namespace iskv
