// iskv_q8_attention for few query rows per KV head: single tokens, drafts to
// verify, fp32 queries.  Split along the keys over the whole GPU.
//
// Mathematics.  Keys and values are codes times one scale per page and head,
// so the scale leaves the dot products: with c the codes,
//     score = (scale s_k) (q . c_k),   out = sum w s_v c_v / sum w.
// One exponential carries the value scale too: with
//     w = 2^(score log2 e + log2 s_v - M),  M the running maximum,
// the numerator is sum w c_v and the denominator sum w / s_v, whose factor
// 1 / s_v is one number per page.  (A page of scale 0 counts in the denominator
// alone.  It takes the scale of the first other page that the row sees; a row that
// has seen none counts in scale 1 and changes over then.  So its weights neither
// raise M above those of small values, whose fp16 weights would lose bits, nor
// vanish beside large ones.)  Codes are exact in fp16.  Queries are
// multiplied by a power of two per row (their largest element then lies in
// [2^14, 2^15)) and are exact in fp16 down to 2^-38 of it for bf16 input; fp32
// queries, and the weights that go with them, take two fp16 parts (22 bits).
// For bf16 queries the weights are rounded to fp16 (2^-12 relative, an eighth
// of the output's own rounding); sums and maxima stay in fp32.
//
// Layout.  The products are taken transposed: S^T = K Q^T and O^T = V^T P^T,
// so that the keys fill the 16 rows of m16n8k16 and the few query rows its 8
// columns (half the instructions of the other order when there are at most 8
// rows), and a lane ends up with 16 consecutive output elements of its two
// rows.  P^T turns from accumulator to operand layout by movmatrix.  The order
// of the 128 elements inside a dot product is free, so a lane takes 32
// consecutive codes of a key row (two 16-byte loads) instead of the
// instruction's interleaved pairs.  Tensor cores carry it by mma.sync here: at
// 8 columns the kernel needs about a tenth of their rate, and waits for memory.
//
// Work.  Requests, heads, row tiles and 32-token steps are numbered through;
// every CTA finds its equal share of the steps from the lengths itself (one
// pass over the requests, no plan on the host) and every warp its share of
// that, so lengths may differ freely.  A warp runs its own pipeline of tensor
// copies (a stage is 4 KB of K and 4 KB of V, swizzled as the fragment loads
// want them; one lane issues both) and never waits for another warp until its
// share is done.  What one warp finishes alone is written at once; what several
// warps share is joined in the CTA, what several CTAs share by a second small
// kernel.
//
// What bounds it: DRAM for long caches (8 KV heads, 32 query heads, int8: 8 x 32K
// tokens 98 us on one GPU and 105 on another, 84 and 78 % of the measured copy rate;
// 96 ragged requests of up to 16K tokens, e4m3, capped, 304 and 326 us, 88 and 82 %;
// fp32 queries, with twice the products, 8 x 32K tokens 126 us, 65 %), for short ones the latency of
// about six dependent memory accesses, two launches and the first fetch of the
// code (1 request of 1K tokens 12 us, of 64 tokens 9 us with one launch).
#include <cuda.h>

#include "q8_common.cuh"
#include "q8_split.h"
#include "tc_util.cuh"

namespace iskv {
namespace q8 {

namespace {

// Warps and pipeline stages per warp.  The loop is bound by the latency of its
// own instructions, so the light variant takes 12 warps of 168 registers with
// two stages each (measured against 8 warps with three: 96 ragged requests of up
// to 16K tokens 353 -> 317 us, 8 x 32K tokens 117 -> 116 us); two row tiles or
// fp32 parts need more registers and take 8.
template <int NT, bool F32>
struct Shape {
    static constexpr int kWarps = rows_warps(NT, F32);
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kStages = kWarps > 8 ? 2 : 3;
};
constexpr int kStoreBytes = kStepTokens * kHeadDim;      // K or V of one step: 4 KB
constexpr int kStageBytes = 2 * kStoreBytes;

using Req = Seen<kStepTokens>;

__device__ __forceinline__ int tiles_of(const AttnArgs& p, int n) { return (n + p.tq - 1) / p.tq; }

// A box of the tensor map: 32 rows of 128 codes from row `row` of (page, head) `block` on.
__device__ __forceinline__ void copy_step(uint32_t dst, const CUtensorMap* map, int row, int block, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(0), "r"(row), "r"(block), "r"(tc::smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack(uint32_t x) {
    return __half22float2(*reinterpret_cast<const __half2*>(&x));
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

// A place in the numbered-through steps.  (No divisions on the way: straight-line
// code is fetched from L2 by every SM at every launch, and a call of this kernel
// is as long as its code is.)
struct Cursor {
    int b, h, tile, step;
    int tiles;
    Req r;
    __device__ __forceinline__ void load(const AttnArgs& p) {
        r = seen_of<kStepTokens>(p, b);
        tiles = tiles_of(p, r.n);
    }
    // to the next step; the caller knows that there is one
    __device__ __forceinline__ void next(const AttnArgs& p) {
        if (++step < r.steps) return;
        step = 0;
        if (++tile < tiles) return;
        tile = 0;
        if (++h < p.kv_heads) return;
        h = 0;
#pragma unroll 1
        do {
            ++b;
            load(p);
        } while (r.steps == 0);
    }
};

// What the CTA knows of each of its warps' two partials.
struct Part {
    int64_t id;       // request << 32 | item, -1: none
    int begins, ends; // whether it holds the item's first / last step
};

// A request's items (KV head, row tile) and the steps of each.
__device__ __forceinline__ int2 shape_of(const AttnArgs& p, int b) {
    const Req r = seen_of<kStepTokens>(p, b);
    return make_int2(tiles_of(p, r.n) * p.kv_heads, r.steps);
}

template <bool F32, int N>
__device__ __forceinline__ void store_out(const AttnArgs& p, int64_t at, const float (&v)[N]) {
    if (F32) {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at);
#pragma unroll
        for (int i = 0; i < N / 4; ++i) o[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
        uint2* o = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + at);
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const __nv_bfloat162 a = __floats2bfloat162_rn(v[4 * i], v[4 * i + 1]);
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[4 * i + 2], v[4 * i + 3]);
            o[i] = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
        }
    }
}

// One row's sum over partials i = first, first + step, ... < n (at(i): the i-th
// partial's row in the workspace), relative to the largest of their maxima: the
// lane's four columns in o, the denominator in l.
template <typename At>
__device__ __forceinline__ void sum_parts(const AttnArgs& p, int first, int step, int n, At at, int lane, float& M, float& l, float (&o)[4]) {
    M = -INFINITY;
    l = 0.f;
    o[0] = o[1] = o[2] = o[3] = 0.f;
#pragma unroll 1
    for (int i0 = first; i0 < n; i0 += 32 * step) {   // 32 partials at a time, their maxima in the lanes
        const int i = i0 + lane * step;
        const float2 ml = i < n ? *reinterpret_cast<const float2*>(p.ml + at(i) * 2) : make_float2(-INFINITY, 0.f);
        const float now = fmaxf(M, warp_max(ml.x));
        const float base = now == -INFINITY ? 0.f : now;
        const float f = ex2(ml.x - base), g = ex2(M - base);
        l = l * g + warp_sum(f * ml.y);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] *= g;
        M = now;
        const int m = min(32, (n - i0 + step - 1) / step);
#pragma unroll 4
        for (int k = 0; k < m; ++k) {
            const float4 v = *reinterpret_cast<const float4*>(p.part + at(i0 + k * step) * kHeadDim + 4 * lane);
            const float w = __shfl_sync(0xffffffffu, f, k);
            o[0] += w * v.x;
            o[1] += w * v.y;
            o[2] += w * v.z;
            o[3] += w * v.w;
        }
    }
}

// The joined row: to its place in out, or to partial row `to` (>= 0).
template <bool F32>
__device__ __forceinline__ void put_row(const AttnArgs& p, int64_t out_at, int64_t to, float M, float l, float (&o)[4], int lane) {
    if (to < 0) {
        const float inv = l > 0.f ? __fdividef(1.f, l) : (l == 0.f ? 0.f : l);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] *= inv;
        store_out<F32, 4>(p, out_at + 4 * lane, o);
    } else {
        *reinterpret_cast<float4*>(p.part + to * kHeadDim + 4 * lane) = make_float4(o[0], o[1], o[2], o[3]);
        if (lane == 0) *reinterpret_cast<float2*>(p.ml + to * 2) = make_float2(M, l);
    }
}

// Row `row` of (request, item): its place in out; false where it has none.
__device__ __forceinline__ bool place_of(const AttnArgs& p, int b, int item, int row, int64_t* at) {
    const Req r = seen_of<kStepTokens>(p, b);
    const int tiles = tiles_of(p, r.n), h = item / tiles, tile = item - h * tiles;
    const int k = row / p.g, token = tile * p.tq + k, head = h * p.g + row - k * p.g;
    *at = ((int64_t)(r.first + token) * p.kv_heads * p.g + head) * kHeadDim;
    return k < p.tq && token < r.n;
}

// Meta words per CTA: [0] whether its partial 0 ends an item; [1] CTAs that
// follow with the rest of the item that its partial 1 begins (0: none); [2]
// that item's request, [3] its item.
constexpr int kMeta = 4;

template <int CODE, int NT, bool F32, bool MOD>
__global__ void __launch_bounds__(Shape<NT, F32>::kThreads, 1) q8_rows_kernel(const __grid_constant__ AttnArgs p, const __grid_constant__ CUtensorMap map_k,
                                                                               const __grid_constant__ CUtensorMap map_v) {
    constexpr int kWarps = Shape<NT, F32>::kWarps, kThreads = Shape<NT, F32>::kThreads, kStages = Shape<NT, F32>::kStages;
    constexpr int kPartsPerCta = 2 * kWarps + 2;
    extern __shared__ uint8_t dyn[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~(uintptr_t)1023);
    __shared__ int64_t s_scan[2][kWarps], s_off[kWarps], s_bound[2];
    __shared__ int s_b[kWarps];
    __shared__ Part s_part[kWarps][2];
    __shared__ int s_list[2 * kWarps], s_first[2 * kWarps + 1], s_groups;
    __shared__ int s_page[kWarps][kStages];
    __shared__ uint64_t s_full[kWarps][kStages];
    constexpr int R = 8 * NT, PARTS = F32 ? 2 : 1;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int r = lane >> 2, q = lane & 3;
    const int cta = blockIdx.x;
    let_next();
    if (t == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_k));
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_v));
    }
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < kStages; ++i) tc::mbar_init(&s_full[warp][i], 1);
        tc::fence_mbar_init();
    }
    after_previous();

    // ---- this CTA's and this warp's share of the steps --------------------
    const int chunk = (p.batch + kThreads - 1) / kThreads;
    const int b0 = min(p.batch, t * chunk), b1 = min(p.batch, b0 + chunk);
    int64_t mine = 0, items = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
        const int2 n = shape_of(p, b);
        items += n.x;
        mine += (int64_t)n.x * n.y;
    }
    int64_t incl = mine, incl_items = items;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, incl, o), v = __shfl_up_sync(0xffffffffu, incl_items, o);
        if (lane >= o) {
            incl += u;
            incl_items += v;
        }
    }
    if (lane == 31) {
        s_scan[0][warp] = incl;
        s_scan[1][warp] = incl_items;
    }
    if (t < kWarps) s_part[t][0].id = s_part[t][1].id = -1;
    __syncthreads();
    int64_t total = 0, ex = incl - mine, all_items = 0, ex_items = incl_items - items;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) {
            ex += s_scan[0][w];
            ex_items += s_scan[1][w];
        }
        total += s_scan[0][w];
        all_items += s_scan[1][w];
    }
    int64_t u0, u1;
    if (p.whole) {   // whole items: nothing is left to be joined
        const int64_t per_cta = (all_items + gridDim.x - 1) / gridDim.x;
        if (t < 2) s_bound[t] = total;
        __syncthreads();
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
            const int64_t want = (cta + k) * per_cta;
            if (want >= ex_items && want < ex_items + items) {
                int64_t at_item = ex_items, at = ex;
                int b = b0;
#pragma unroll 1
                for (;; ++b) {
                    const int2 n = shape_of(p, b);
                    if (want < at_item + n.x) {
                        at += (want - at_item) * n.y;
                        break;
                    }
                    at_item += n.x;
                    at += (int64_t)n.x * n.y;
                }
                s_bound[k] = at;
            }
        }
        __syncthreads();
        u0 = s_bound[0];
        u1 = s_bound[1];
    } else {
        const int64_t per_cta = (total + gridDim.x - 1) / gridDim.x;
        u0 = cta * per_cta;
        u1 = min(total, u0 + per_cta);
    }
    if (u0 >= u1) {   // uniform over the CTA
        if (t < kMeta) p.meta[cta * kMeta + t] = 0;
        return;
    }
    const int64_t per_warp = (u1 - u0 + kWarps - 1) / kWarps;
    if (mine > 0) {
#pragma unroll 1
        for (int w = 0; w < kWarps; ++w) {
            const int64_t u = u0 + w * per_warp;
            if (u < u1 && u >= ex && u < ex + mine) {
                int64_t off = u - ex;
                int b = b0;
#pragma unroll 1
                for (;; ++b) {
                    const int2 n = shape_of(p, b);
                    if (off < (int64_t)n.x * n.y) break;
                    off -= (int64_t)n.x * n.y;
                }
                s_b[w] = b;
                s_off[w] = off;
            }
        }
    }
    __syncthreads();

    const int64_t w0 = u0 + warp * per_warp;
    const int64_t n_steps = min(u1, w0 + per_warp) - w0;   // steps of this warp (may be <= 0)
    uint8_t* ring = smem + warp * (kStages * kStageBytes);
    const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
    const int my_parts = (cta * kPartsPerCta) + 2 * warp;
    // rows of this lane inside a row tile, as (token, head of the group): of its
    // query row r and of its result rows 2q, 2q + 1 (8 more per tile of 8)
    int q_k[NT], q_g[NT], o_k[NT][2], o_g[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        q_k[n] = (n * 8 + r) / p.g;
        q_g[n] = n * 8 + r - q_k[n] * p.g;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int src = 8 * q + 4 * c;
            o_k[n][c] = __shfl_sync(0xffffffffu, q_k[n], src);
            o_g[n][c] = __shfl_sync(0xffffffffu, q_g[n], src);
        }
    }

    int gave_up = 0;
    if (n_steps > 0) {
        Cursor in, at;
        at.b = s_b[warp];
        at.load(p);
        {
            const StepPlace s = place_of_step(s_off[warp], at.tiles, at.r.steps);
            at.h = s.h;
            at.tile = s.tile;
            at.step = s.step;
        }
        in = at;
        int left = (int)min(n_steps, (int64_t)INT32_MAX), to_issue = left;

        uint32_t qf[PARTS][NT][8][2];          // queries as B fragments
        float rowf[NT][2];                     // score factor of rows 2q, 2q + 1 of each tile of 8
        int pos[NT][2], see_from[NT][2];       // the causal span (see_from, pos]
        float slope[NT][2];
        float M[NT][2], l[NT][2], o[NT][8][4];
        float lz[NT][2];                       // log2 of the scale for pages of scale 0; infinity: none yet
        int pmin = 0, pmax = 0, first_step = 0;
        bool fresh = true, settled = false;    // settled: every row has its lz

        auto page_of = [&](const Cursor& c) {
            const int tok = c.r.step_of(c.step) * kStepTokens;
            return tok < c.r.len ? p.table[(int64_t)c.b * p.width + tok / kPage] : -1;
        };
        int page = page_of(in), fill = 0, stage = 0;
        uint32_t phase = 0;   // a bit per stage
        bool failed = false;
        // kStages - 1 steps are on their way before the first is used
#pragma unroll 1
        for (int ahead = 1 - kStages; left > 0; ++ahead) {
            if (to_issue > 0) {
                const int tok = in.r.step_of(in.step) * kStepTokens;
                const bool ok = page >= 0 && page < p.pages;
                if (lane == 0) {
                    s_page[warp][fill] = ok ? page : -1;
                    uint64_t* bar = &s_full[warp][fill];
                    const uint32_t dst = ring_at + fill * kStageBytes;
                    tc::mbar_arrive_expect_tx(bar, ok ? kStageBytes : 0);
                    if (ok) {
                        const int block = page * p.kv_heads + in.h;
                        copy_step(dst, &map_k, tok % kPage, block, bar);
                        copy_step(dst + kStoreBytes, &map_v, tok % kPage, block, bar);
                    }
                }
                fill = fill + 1 == kStages ? 0 : fill + 1;
                if (--to_issue > 0) {
                    in.next(p);
                    page = page_of(in);
                }
            }
            if (ahead < 0) continue;

            if (fresh) {   // an item begins: its queries
                fresh = false;
                settled = false;
                first_step = at.step;
                pmin = at.r.len - at.r.n + at.tile * p.tq;
                pmax = min(at.r.len - 1, pmin + p.tq - 1);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float x[32];
                    const int token = at.tile * p.tq + q_k[n];
                    const bool on = q_k[n] < p.tq && token < at.r.n;
                    const int64_t src = (int64_t)(at.r.first + token) * p.q_stride + (at.h * p.g + q_g[n]) * kHeadDim + 32 * q;
                    if (F32) {
                        const float4* f4 = reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + src);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 v = on ? f4[i] : make_float4(0.f, 0.f, 0.f, 0.f);
                            x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
                        }
                    } else {
                        const uint4* u4 = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + src);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint4 v = on ? u4[i] : make_uint4(0u, 0u, 0u, 0u);
                            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                x[8 * i + 2 * k] = __uint_as_float(w[k] << 16);
                                x[8 * i + 2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
                            }
                        }
                    }
                    float top = 0.f;
#pragma unroll
                    for (int i = 0; i < 32; ++i) top = fmaxf(top, fabsf(x[i]));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    // 2^up brings the row's largest element into [2^14, 2^15)
                    int up = 14 - ((int)(__float_as_uint(top) >> 23) - 127);
                    up = max(-126, min(126, up));
                    const float f = __uint_as_float((uint32_t)(up + 127) << 23);
                    const float down = __uint_as_float((uint32_t)(127 - up) << 23) * (p.scale * (MOD ? 1.f : kLog2e));
#pragma unroll
                    for (int s = 0; s < 8; ++s) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float a = x[4 * s + 2 * i] * f, b = x[4 * s + 2 * i + 1] * f;
                            qf[0][n][s][i] = pack(a, b);
                            if (F32) {
                                const float2 hi = unpack(qf[0][n][s][i]);
                                qf[PARTS - 1][n][s][i] = pack(a - hi.x, b - hi.y);
                            }
                        }
                    }
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        rowf[n][c] = __shfl_sync(0xffffffffu, down, 8 * q + 4 * c);
                        const int tk = at.tile * p.tq + o_k[n][c];
                        pos[n][c] = at.r.len - at.r.n + min(tk, at.r.n - 1);
                        slope[n][c] = MOD && p.slopes && o_k[n][c] < p.tq ? p.slopes[at.h * p.g + o_g[n][c]] * kLog2e : 0.f;
                        see_from[n][c] = p.window > 0 ? max(-1, pos[n][c] - p.window) : -1;
                        M[n][c] = -INFINITY;
                        l[n][c] = 0.f;
                        lz[n][c] = INFINITY;
                    }
#pragma unroll
                    for (int m = 0; m < 8; ++m)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[n][m][i] = 0.f;
                }
            }

            __syncwarp();
            if (!p.patient || !tc::mbar_try_wait(&s_full[warp][stage], (phase >> stage) & 1)) {
                const long long deadline = clock64() + p.wait_cycles;
                while (!failed && !try_phase(p, &s_full[warp][stage], (phase >> stage) & 1)) failed = clock64() > deadline;
            }
            if (__any_sync(0xffffffffu, failed)) {   // out is left incomplete
                failed = true;
                gave_up = 1;
                if (lane == 0 && p.status) atomicMin(p.status, ISKV_ERR_DEVICE_TIMEOUT);
                break;
            }
            phase ^= 1u << stage;
            const int this_page = s_page[warp][stage];
            const int tok = at.r.step_of(at.step) * kStepTokens;
            const int stop = this_page < 0 ? 0 : at.r.len;      // stored tokens end here
            if (tok + kStepTokens > stop) {
                // what stands behind the last token (codes of an earlier owner, which
                // may be NaN) becomes zeros; hidden keys need no such care
#pragma unroll 1
                for (int e = lane; e < kStoreBytes / 16; e += 32)
                    if (tok + (e >> 3) >= stop)
                        *reinterpret_cast<uint4*>(ring + stage * kStageBytes + kStoreBytes + e * 16) = make_uint4(0u, 0u, 0u, 0u);
                tc::fence_async_smem();   // before the next copy into this stage
                __syncwarp();
            }
            const int64_t block = (int64_t)max(this_page, 0) * p.kv_heads + at.h;
            // (a page that is not there has no scales: those of page 0 may be anything)
            const float sk = this_page < 0 ? 0.f : p.k_scale[block], sv = this_page < 0 ? 0.f : p.v_scale[block];
            const uint32_t kb = ring_at + stage * kStageBytes, vb = kb + kStoreBytes;
            stage = stage + 1 == kStages ? 0 : stage + 1;

            // ---- S^T = K Q^T: two tiles of 16 tokens ----------------------
            float sc[NT][2][4];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                uint32_t c0[8], c1[8];   // codes 32q .. 32q + 31 of tokens 16m + r and 16m + r + 8
                const int ra = 16 * m + r;
                {
                    const uint32_t ka = kb + ra * kHeadDim, kc = ka + 8 * kHeadDim;
                    const uint4 a = lds128(ka + (((2 * q) ^ (ra & 7)) << 4)), b = lds128(ka + (((2 * q + 1) ^ (ra & 7)) << 4));
                    const uint4 c = lds128(kc + (((2 * q) ^ (ra & 7)) << 4)), d = lds128(kc + (((2 * q + 1) ^ (ra & 7)) << 4));
                    c0[0] = a.x; c0[1] = a.y; c0[2] = a.z; c0[3] = a.w;
                    c0[4] = b.x; c0[5] = b.y; c0[6] = b.z; c0[7] = b.w;
                    c1[0] = c.x; c1[1] = c.y; c1[2] = c.z; c1[3] = c.w;
                    c1[4] = d.x; c1[5] = d.y; c1[6] = d.z; c1[7] = d.w;
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[n][m][e] = 0.f;
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                    const uint32_t x0 = Codes<CODE>::bias(c0[s]), x1 = Codes<CODE>::bias(c1[s]);
                    const uint32_t a[4] = {Codes<CODE>::lo(x0), Codes<CODE>::lo(x1), Codes<CODE>::hi(x0), Codes<CODE>::hi(x1)};
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int z = 0; z < PARTS; ++z) mma16816(sc[n][m], a, qf[z][n][s][0], qf[z][n][s][1]);
                }
            }

            // ---- weights ---------------------------------------------------
            const bool valued = sv > 0.f;
            const float lsv = valued ? lg2(sv) : 0.f, isv = __fdividef(1.f, sv);
            const bool whole = tok + kStepTokens <= stop &&
                               ((tok + kStepTokens - 1 <= pmin && (p.window == 0 || tok > pmax - p.window)) ||
                                tok + kStepTokens <= at.r.pre);
            uint32_t pf[PARTS][NT][2][2];   // P^T as B fragments: [16-token half][8 tokens]
            bool unsettled = false;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float top[2] = {-INFINITY, -INFINITY}, is[2] = {isv, isv};
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int c = e & 1, key = tok + 16 * m + r + 8 * (e >> 1);
                        float x = sc[n][m][e] * (rowf[n][c] * sk);
                        if (MOD) {
                            if (p.cap > 0.f) x = capped(x, p.cap, p.cap_inv);
                            x *= kLog2e;
                            x -= slope[n][c] * fabsf((float)(pos[n][c] - key));
                        }
                        x += lsv;
                        if (!whole) {
                            const bool on = key < stop && ((key <= pos[n][c] && key > see_from[n][c]) || key < at.r.pre);
                            x = on ? x : -INFINITY;
                        }
                        sc[n][m][e] = x;
                        top[c] = fmaxf(top[c], x);
                    }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    top[c] = fmaxf(top[c], __shfl_xor_sync(0xffffffffu, top[c], 4));
                    top[c] = fmaxf(top[c], __shfl_xor_sync(0xffffffffu, top[c], 8));
                    top[c] = fmaxf(top[c], __shfl_xor_sync(0xffffffffu, top[c], 16));
                }
                if (!(valued && settled)) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        if (!valued) {
                            const float ls = lz[n][c] < INFINITY ? lz[n][c] : 0.f;
                            is[c] = ex2(-ls);
                            top[c] += ls;
#pragma unroll
                            for (int m = 0; m < 2; ++m)
#pragma unroll
                                for (int e = c; e < 4; e += 2) sc[n][m][e] += ls;
                        } else if (top[c] > -INFINITY && lz[n][c] == INFINITY) {   // what came before counted in scale 1
                            M[n][c] += lsv;
                            l[n][c] *= isv;
                            lz[n][c] = lsv;
                        }
                    }
                    unsettled |= fmaxf(lz[n][0], lz[n][1]) == INFINITY;
                    if (n == NT - 1) settled = settled || __all_sync(0xffffffffu, !unsettled);
                }
                const bool grew = top[0] > M[n][0] || top[1] > M[n][1];
                if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float now = fmaxf(M[n][c], top[c]);
                        const float f = now == -INFINITY ? 1.f : ex2(M[n][c] - now);
                        M[n][c] = now;
                        l[n][c] *= f;
#pragma unroll
                        for (int m = 0; m < 8; ++m) {
                            o[n][m][c] *= f;
                            o[n][m][c + 2] *= f;
                        }
                    }
                }
                float sum[2] = {0.f, 0.f};
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float base = (M[n][c] == -INFINITY ? 0.f : M[n][c]) - kWeightShift;
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int e = c; e < 4; e += 2) {
                            sc[n][m][e] = ex2(sc[n][m][e] - base);
                            sum[c] += sc[n][m][e];
                        }
                    l[n][c] += sum[c] * is[c];
                }
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int i2 = 0; i2 < 2; ++i2) {
                        const float a = sc[n][m][2 * i2], b = sc[n][m][2 * i2 + 1];
                        const uint32_t hi = pack(a, b);
                        pf[0][n][m][i2] = transpose8(valued ? hi : 0u);   // (what scale 0 multiplies is nothing, whatever the codes)
                        if (F32) {
                            const float2 f = unpack(hi);
                            pf[PARTS - 1][n][m][i2] = transpose8(valued ? pack(a - f.x, b - f.y) : 0u);
                        }
                    }
            }

            // ---- O^T += V^T P^T: two halves of 16 tokens -------------------
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                uint4 v[4];   // codes 16r .. 16r + 15 of tokens 2q, 2q + 1, 2q + 8, 2q + 9
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int row = 16 * m + 2 * q + (k & 1) + 8 * (k >> 1);
                    v[k] = lds128(vb + row * kHeadDim + ((r ^ (row & 7)) << 4));
                }
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const uint32_t t0 = w == 0 ? v[0].x : w == 1 ? v[0].y : w == 2 ? v[0].z : v[0].w;
                    const uint32_t t1 = w == 0 ? v[1].x : w == 1 ? v[1].y : w == 2 ? v[1].z : v[1].w;
                    const uint32_t t2 = w == 0 ? v[2].x : w == 1 ? v[2].y : w == 2 ? v[2].z : v[2].w;
                    const uint32_t t3 = w == 0 ? v[3].x : w == 1 ? v[3].y : w == 2 ? v[3].z : v[3].w;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint32_t sel = half ? 0x7362 : 0x5140;   // the two tokens' codes side by side
                        const uint32_t x = Codes<CODE>::bias(__byte_perm(t0, t1, sel));
                        const uint32_t y = Codes<CODE>::bias(__byte_perm(t2, t3, sel));
                        const uint32_t a[4] = {Codes<CODE>::lo(x), Codes<CODE>::hi(x), Codes<CODE>::lo(y), Codes<CODE>::hi(y)};
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int z = 0; z < PARTS; ++z) mma16816(o[n][2 * w + half], a, pf[z][n][m][0], pf[z][n][m][1]);
                    }
                }
            }
            __syncwarp();   // the stage may be filled again

            // ---- end of an item, or of this warp's share -------------------
            --left;
            const bool last = at.step + 1 == at.r.steps;
            if (last || left == 0) {
                const bool whole_item = last && first_step == 0;
                const int slot = first_step != 0 ? 0 : 1;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float den = l[n][c];
                        den += __shfl_xor_sync(0xffffffffu, den, 4);
                        den += __shfl_xor_sync(0xffffffffu, den, 8);
                        den += __shfl_xor_sync(0xffffffffu, den, 16);
                        const int token = at.tile * p.tq + o_k[n][c], head = at.h * p.g + o_g[n][c];
                        if (o_k[n][c] >= p.tq || token >= at.r.n) continue;
                        float v[16];
#pragma unroll
                        for (int m = 0; m < 8; ++m) {
                            v[2 * m] = o[n][m][c];
                            v[2 * m + 1] = o[n][m][c + 2];
                        }
                        if (whole_item) {
                            const float inv = den > 0.f ? __fdividef(1.f, den) : (den == 0.f ? 0.f : den);
#pragma unroll
                            for (int k = 0; k < 16; ++k) v[k] *= inv;
                            store_out<F32, 16>(p, ((int64_t)(at.r.first + token) * p.kv_heads * p.g + head) * kHeadDim + 16 * r, v);
                        } else {
                            const int64_t k = (int64_t)(my_parts + slot) * R + n * 8 + 2 * q + c;
                            float4* to = reinterpret_cast<float4*>(p.part + k * kHeadDim + 16 * r);
#pragma unroll
                            for (int m = 0; m < 4; ++m)
                                to[m] = make_float4(v[4 * m], v[4 * m + 1], v[4 * m + 2], v[4 * m + 3]);
                            if (r == 0) *reinterpret_cast<float2*>(p.ml + k * 2) = make_float2(M[n][c], den);
                        }
                    }
                if (!whole_item && lane == 0)
                    s_part[warp][slot] = Part{((int64_t)at.b << 32) | (uint32_t)(at.h * at.tiles + at.tile), first_step == 0, last};
                fresh = true;
            }
            if (left > 0) at.next(p);
        }
    }

    if (__syncthreads_or(gave_up)) {
        // copies may be on their way to warps that have given up: they land within
        // microseconds; the CTA ends long after
        const long long until = clock64() + 20000000;
        while (clock64() < until) __nanosleep(1000);
    }

    // ---- items that several warps of this CTA share ------------------------
    // A group is the parts of one item, which follow each other; (group, row)
    // pairs are dealt to the warps.
    if (t < kMeta) p.meta[cta * kMeta + t] = 0;
    if (warp == 0) {
        const int64_t id = lane < 2 * kWarps ? s_part[lane >> 1][lane & 1].id : -1;
        const uint32_t there = __ballot_sync(0xffffffffu, id >= 0);
        const uint32_t below = there & ((1u << lane) - 1u);
        const int64_t before = __shfl_sync(0xffffffffu, id, below ? 31 - __clz(below) : 0);
        const bool head = id >= 0 && (below == 0 || before != id);
        const uint32_t heads = __ballot_sync(0xffffffffu, head);
        if (id >= 0) s_list[__popc(below)] = lane;
        if (head) s_first[__popc(heads & ((1u << lane) - 1u))] = __popc(below);
        if (lane == 0) {
            s_groups = __popc(heads);
            s_first[__popc(heads)] = __popc(there);
        }
    }
    __syncthreads();
#pragma unroll 1
    for (int e = warp; e < s_groups * R; e += kWarps) {
        const int grp = e / R, row = e % R, first = s_first[grp], n = s_first[grp + 1] - first;
        const Part a = s_part[s_list[first] >> 1][s_list[first] & 1];
        const int ends = s_part[s_list[first + n - 1] >> 1][s_list[first + n - 1] & 1].ends;
        const int b = (int)(a.id >> 32), item = (int)(uint32_t)a.id;
        const bool final = a.begins && ends;
        if (row == 0 && lane == 0 && !final) {
            int* m = p.meta + cta * kMeta;
            if (!a.begins) {
                m[0] = ends;
            } else {
                m[1] = 1;
                m[2] = b;
                m[3] = item;
            }
        }
        int64_t out_at;
        if (!place_of(p, b, item, row, &out_at)) continue;
        float M, l, o[4];
        const int64_t base = (int64_t)cta * kPartsPerCta * R + row;
        sum_parts(p, 0, 1, n, [&](int k) { return base + s_list[first + k] * R; }, lane, M, l, o);
        put_row<F32>(p, out_at, final ? -1 : base + (2 * kWarps + (a.begins ? 1 : 0)) * R, M, l, o, lane);
    }
}

// Items that several CTAs share: CTA c joins a row of the one that its partial
// 1 begins with the partials 0 of the CTAs after it, up to the one that ends it.
// Each warp sums some of the partials.
template <int NT, bool F32>
__global__ void __launch_bounds__(256) q8_join_kernel(const __grid_constant__ AttnArgs p) {
    constexpr int R = 8 * NT, kWarps = Shape<NT, F32>::kWarps, kPartsPerCta = 2 * kWarps + 2;
    const int cta = blockIdx.x, row = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __shared__ float s_ml[8][2], s_o[8][kHeadDim];
    // (no let_next(): eight layers of 64 requests 359 us without, 362 with it)
    after_previous();
    const int4 m = *reinterpret_cast<const int4*>(p.meta + cta * kMeta);
    if (m.y == 0) return;
    int64_t out_at;
    if (!place_of(p, m.z, m.w, row, &out_at)) return;
    int n = 1;   // partials: how many CTAs follow
#pragma unroll 1
    for (int c0 = cta + 1; c0 < p.ctas; c0 += 32) {
        const uint32_t hit = __ballot_sync(0xffffffffu, c0 + lane < p.ctas && p.meta[(c0 + lane) * kMeta] != 0);
        n += hit ? __ffs(hit) : 32;
        if (hit) break;
    }
    n = min(n, p.ctas - cta);
    float M, l, o[4];
    sum_parts(p, warp, 8, n,
              [&](int k) { return (int64_t)((cta + k) * kPartsPerCta + 2 * kWarps + (k == 0 ? 1 : 0)) * R + row; }, lane, M, l, o);
    if (lane == 0) {
        s_ml[warp][0] = M;
        s_ml[warp][1] = l;
    }
    *reinterpret_cast<float4*>(&s_o[warp][4 * lane]) = make_float4(o[0], o[1], o[2], o[3]);
    __syncthreads();
    if (warp > 0) return;
    float top = M;
#pragma unroll
    for (int w = 1; w < 8; ++w) top = fmaxf(top, s_ml[w][0]);
    const float base = top == -INFINITY ? 0.f : top;
    l = 0.f;
    o[0] = o[1] = o[2] = o[3] = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        const float f = ex2(s_ml[w][0] - base);
        const float4 v = *reinterpret_cast<const float4*>(&s_o[w][4 * lane]);
        l += f * s_ml[w][1];
        o[0] += f * v.x;
        o[1] += f * v.y;
        o[2] += f * v.z;
        o[3] += f * v.w;
    }
    put_row<F32>(p, out_at, -1, top, l, o, lane);
}

// The codes of one store as [pages * kv_heads][64][128] bytes, copied 32 rows at
// a time with the 128-byte swizzle (chunk c of row t stands at c ^ (t & 7)).
bool tensor_map(const AttnArgs& a, const uint8_t* codes, CUtensorMap* map) {
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static Encode encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<Encode>(f);
    }();
    if (!encode) return false;
    const cuuint64_t dims[3] = {kHeadDim, kPage, (cuuint64_t)a.pages * a.kv_heads};
    const cuuint64_t strides[2] = {kHeadDim, kPage * kHeadDim};
    const cuuint32_t box[3] = {kHeadDim, kStepTokens, 1}, step[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(codes), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int CODE, int NT, bool F32, bool MOD>
cudaError_t run(const AttnArgs& a, cudaStream_t s) {
    using S = Shape<NT, F32>;
    constexpr int kSmemBytes = S::kWarps * S::kStages * kStageBytes + 1024;
    static SmemOnce once;
    cudaError_t e = once.set(q8_rows_kernel<CODE, NT, F32, MOD>, kSmemBytes);
    if (e != cudaSuccess) return e;
    CUtensorMap map_k, map_v;
    if (!tensor_map(a, a.k, &map_k) || !tensor_map(a, a.v, &map_v)) return cudaErrorInvalidValue;
    e = launch_early(q8_rows_kernel<CODE, NT, F32, MOD>, dim3(a.ctas), S::kThreads, kSmemBytes, s, 0, a, map_k, map_v);
    if (e != cudaSuccess || a.whole) return e;
    return launch_early(q8_join_kernel<NT, F32>, dim3(a.ctas, 8 * NT), 256, 0, s, 0, a);
}

template <int CODE>
cudaError_t by_type(const AttnArgs& a, bool f32, int tiles8, cudaStream_t s) {
    const bool mod = a.cap > 0.f || a.slopes != nullptr;
    if (!f32) return mod ? run<CODE, 1, false, true>(a, s) : run<CODE, 1, false, false>(a, s);
    if (tiles8 == 1) return mod ? run<CODE, 1, true, true>(a, s) : run<CODE, 1, true, false>(a, s);
    return mod ? run<CODE, 2, true, true>(a, s) : run<CODE, 2, true, false>(a, s);
}

}  // namespace

cudaError_t launch_q8_rows(const AttnArgs& a, int code, bool f32, int tiles8, cudaStream_t s) {
    return code == ISKV_CODE_INT8 ? by_type<ISKV_CODE_INT8>(a, f32, tiles8, s)
                                  : by_type<ISKV_CODE_E4M3>(a, f32, tiles8, s);
}

}  // namespace q8
}  // namespace iskv
