// iskv_q8_append: new K and V rows as 8-bit codes with one scale per page and
// KV head.
//
// A run is the rows of one call that land in one page; the thread that sees a
// slot which does not follow on from the one before it has found a run's
// start.  One CTA takes one run of one head, of K or of V: the rows (at most
// 64 x 128) are held in registers between the pass that finds the largest
// value and the pass that codes them, so each element is read once and its
// code written once.  Only where a run continues a page and needs a larger
// scale are the page's earlier codes read and coded again.
//
// Bound by DRAM for prompts (3 bytes per bf16 element) and by launch and load
// latency for single tokens.
#include "q8_common.cuh"

namespace iskv {
namespace q8 {

namespace {

constexpr int kThreads = 128;
constexpr int kPasses = kPage * kHeadDim / (kThreads * 8);   // 8: 8 elements per thread and pass

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&v)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

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

// x / s as a code; s > 0.  For e4m3 s is a power of two and the quotient exact.
template <int CODE>
__device__ __forceinline__ uint32_t code4(float a, float b, float c, float d) {
    if (CODE == ISKV_CODE_INT8) {
        // rounded half to even; |x| / s <= 127 up to the rounding of s
        const int ia = __float2int_rn(fminf(fmaxf(a, -127.f), 127.f)), ib = __float2int_rn(fminf(fmaxf(b, -127.f), 127.f));
        const int ic = __float2int_rn(fminf(fmaxf(c, -127.f), 127.f)), id = __float2int_rn(fminf(fmaxf(d, -127.f), 127.f));
        return (ia & 255) | ((ib & 255) << 8) | ((ic & 255) << 16) | ((uint32_t)id << 24);
    }
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
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
__global__ void __launch_bounds__(kThreads) q8_append_kernel(const AppendArgs p) {
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int head = blockIdx.y, which = blockIdx.z;
    const T* x = static_cast<const T*>(which ? p.x[1] : p.x[0]);
    const int64_t stride = which ? p.stride[1] : p.stride[0];
    uint8_t* store = static_cast<uint8_t*>(which ? p.store[1] : p.store[0]);
    float* scale = which ? p.scale[1] : p.scale[0];
    const int64_t t0 = (int64_t)blockIdx.x * p.window;
    const int64_t t1 = t0 + p.window < p.n ? t0 + p.window : p.n;
    const int64_t n_slots = (int64_t)p.pages * kPage;
    __shared__ float s_top[kThreads / 32];
    __shared__ int s_run[2];

    for (int64_t i = t0; i < t1; ++i) {   // uniform over the CTA
        const int64_t slot = p.slots[i];
        if (slot < 0 || slot >= n_slots) {
            if (slot != -1 && t == 0 && p.status) atomicMin(p.status, ISKV_ERR_INVALID_ARG);
            continue;
        }
        const int row0 = (int)(slot % kPage);
        if (i > 0 && row0 != 0 && p.slots[i - 1] == slot - 1) continue;   // inside a run
        // rows of the run: how far the slots go on one by one inside the page
        if (warp < 2) {
            const bool on = t < kPage - row0 && i + t < p.n && p.slots[i + t] == slot + t;
            const uint32_t m = __ballot_sync(0xffffffffu, on);
            if (lane == 0) s_run[warp] = m == 0xffffffffu ? 32 : __ffs(~m) - 1;
        }
        __syncthreads();
        const int n = s_run[0] < 32 ? s_run[0] : 32 + s_run[1];

        // 16 threads per row, 8 rows per pass
        const int col = (t & 15) * 8;
        float v[kPasses][8];
        float top = 0.f;
        bool bad = false;
#pragma unroll
        for (int s = 0; s < kPasses; ++s) {
            const int r = s * (kThreads / 16) + (t >> 4);
            if (r < n) {
                load8<T>(x + (i + r) * stride + head * kHeadDim + col, v[s]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[s][e] = 0.f;
            }
        }
#pragma unroll
        for (int s = 0; s < kPasses; ++s)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float m = fabsf(v[s][e]);
                if (!(m < INFINITY)) {   // infinities and NaN are stored as zeros
                    bad = true;
                    v[s][e] = 0.f;
                } else {
                    top = fmaxf(top, m);
                }
            }
        if (bad && p.status) atomicMin(p.status, ISKV_ERR_RANGE);
        top = warp_max(top);
        if (lane == 0) s_top[warp] = top;
        const int64_t block = (slot / kPage) * p.kv_heads + head;
        const float before = row0 > 0 ? scale[block] : 0.f;
        __syncthreads();   // every thread has read the old scale
        top = s_top[0];
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
                c.x = code4<CODE>(__fmul_rn(u[0], f), __fmul_rn(u[1], f), __fmul_rn(u[2], f), __fmul_rn(u[3], f));
                decode4<CODE>(c.y, u);
                c.y = code4<CODE>(__fmul_rn(u[0], f), __fmul_rn(u[1], f), __fmul_rn(u[2], f), __fmul_rn(u[3], f));
                *at = c;
            }
        }
#pragma unroll
        for (int s = 0; s < kPasses; ++s) {
            const int r = s * (kThreads / 16) + (t >> 4);
            if (r >= n) continue;
            uint2 c = make_uint2(0u, 0u);
            if (now > 0.f) {
                float u[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] = __fdiv_rn(v[s][e], now);
                c.x = code4<CODE>(u[0], u[1], u[2], u[3]);
                c.y = code4<CODE>(u[4], u[5], u[6], u[7]);
            }
            *reinterpret_cast<uint2*>(base + (row0 + r) * kHeadDim + col) = c;
        }
        __syncthreads();   // s_run and s_top are free again
    }
}

}  // namespace

cudaError_t launch_q8_append(const AppendArgs& a, int code, int dtype, cudaStream_t s) {
    if (a.n == 0) return cudaSuccess;
    const dim3 grid((unsigned)((a.n + a.window - 1) / a.window), a.kv_heads, 2);
    if (code == ISKV_CODE_INT8) {
        if (dtype == ISKV_F32) q8_append_kernel<ISKV_CODE_INT8, float><<<grid, kThreads, 0, s>>>(a);
        else q8_append_kernel<ISKV_CODE_INT8, __nv_bfloat16><<<grid, kThreads, 0, s>>>(a);
    } else {
        if (dtype == ISKV_F32) q8_append_kernel<ISKV_CODE_E4M3, float><<<grid, kThreads, 0, s>>>(a);
        else q8_append_kernel<ISKV_CODE_E4M3, __nv_bfloat16><<<grid, kThreads, 0, s>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace q8
}  // namespace iskv
