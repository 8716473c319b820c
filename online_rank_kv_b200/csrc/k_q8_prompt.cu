// iskv_q8_attention for prompts: many query rows per KV head, on tcgen05.
//
// Mathematics: as in the split kernel (k_q8_rows.cu) -- codes are exact in
// fp16, the key scale multiplies scores, and one exponential
//     w = 2^(score log2 e + log2 s_v - M)
// gives the numerator sum w c_v and the denominator sum w / s_v.  M is raised
// only when a row's maximum has grown by more than 2^8 (weights then stay below
// 2^15 with the shift of 2^7 that keeps them off fp16's subnormals), so the
// accumulator in tensor memory is rescaled a few times per row, not per tile.
//
// One CTA per SM holds two tiles of 128 query rows (query tokens x the heads
// that share a KV head) against key tiles of 128 tokens:
//   warps 0-3, 4-7  softmax of tile 0 and of tile 1, one thread per row: scores
//                   from TMEM, weights as fp16 back over them, and the rare
//                   rescaling; also load, scale and store their own Q rows
//   warps 8-11      turn the codes of K and V tiles into fp16 operands (global
//                   memory -> registers one tile ahead -> swizzled shared memory)
//   warp 12         one thread issues every MMA: S_i = Q_i K^T, O_i += P_i V
// While one tile's softmax runs, the other tile's two products do.  TMEM: S_0,
// S_1 (fp32, the fp16 weights over their first half), O_0, O_1, 128 columns
// each.  K and V tiles have two buffers each.
//
// Work: (KV head, pair of query tiles, key tile) are numbered through and every
// CTA takes an equal contiguous range, so that causal triangles, ragged batches
// and short chunks on long caches all fill the GPU; a pair that crosses CTAs is
// joined from its partial sums by a second kernel.
//
// Bounds per key tile and pair (148 SMs at 1.85 GHz): 2048 cycles of MMA, 2048
// cycles of exponentials (16 per SM and clock), about 1500 issue slots per
// scheduler.
#include "q8_common.cuh"
#include "tc_util.cuh"

namespace iskv {
namespace q8 {

namespace {

constexpr int kM = 128;                    // query rows per tile
constexpr int kN = 128;                    // keys per tile
constexpr int kTileBytes = kN * kHeadDim * 2;   // one fp16 operand tile: 32 KB
constexpr int kHalf = kTileBytes / 2;      // 64 of its 128 columns: rows of 128 bytes
constexpr int kSoftmaxWarps = 8, kCodeWarps = 4;
constexpr int kThreads = 32 * (kSoftmaxWarps + kCodeWarps + 1);
constexpr float kShift = 7.f;
constexpr float kRaise = 8.f;

struct Shared {
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
    uint64_t q_full, s_full[2], p_full[2], pv_done[2], drain;
    uint32_t tmem;
    int failed;
    int64_t scan[16];
    int64_t start_off;
    int start_b, start_pair;
};
// dynamic shared memory: 1024-byte aligned [K 2 tiles][V 2 tiles][Q 2 tiles]
constexpr int kSmemBytes = 6 * kTileBytes + 1024;

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,"
        "%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,"
        "%29,%30,%31,%32};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}

// Shared-memory operand with 128-byte rows, 128-byte swizzle (the 16-byte chunk
// c of row t stands at chunk c ^ (t & 7)).  K-major (Q, K): sbo = 1024 between
// groups of 8 rows.  MN-major (V, whose rows are the reduction index): sbo =
// 1024 between groups of 8 rows, lbo = kHalf between 64-column halves.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)((lbo >> 4) & 0x3FFFu) << 16 |
           (uint64_t)((sbo >> 4) & 0x3FFFu) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// Waits are bounded: the limit is about a second, a pipeline step microseconds.
__device__ __forceinline__ bool wait_for(Shared& sh, uint64_t* bar, uint32_t parity) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    const long long deadline = clock64() + tc::kWaitCycles;
    while (!tc::mbar_try_wait(bar, parity)) {
        if (*(volatile int*)&sh.failed) return false;
        if (clock64() > deadline) {
            sh.failed = 1;
            return false;
        }
    }
    return true;
}

// The key tiles that a pair of query tiles sees.
struct Span {
    int p0;            // position of the pair's first query
    int a, lo, tiles;
    __device__ __forceinline__ int tile_of(int i) const { return i < a ? i : i - a + lo; }
};
__device__ __forceinline__ Span span_of(const AttnArgs& p, const Seen<kN>& r, int pair) {
    Span s;
    const int t0 = pair * 2 * p.tq;
    s.p0 = r.len - r.n + t0;
    const int p1 = min(r.len - 1, s.p0 + 2 * p.tq - 1);
    const int pre = (r.pre + kN - 1) / kN;
    const int hi = p1 < 0 ? 0 : p1 / kN + 1;
    int64_t w0 = p.window > 0 ? (int64_t)s.p0 - p.window + 1 : 0;
    s.lo = w0 > 0 ? (int)(w0 / kN) : 0;
    if (pre >= s.lo) {
        s.a = 0;
        s.lo = 0;
        s.tiles = max(pre, hi);
    } else {
        s.a = pre;
        s.tiles = pre + max(0, hi - s.lo);
    }
    if (s.tiles == 0) s.tiles = 1;   // nothing to see: one hidden tile, so that zeros are written
    return s;
}

__device__ __forceinline__ int pairs_of(const AttnArgs& p, int b) {
    const int64_t c0 = p.cu[b] < 0 ? 0 : p.cu[b];
    const int64_t c1 = p.cu[b + 1] < p.tokens ? p.cu[b + 1] : p.tokens;
    return c1 > c0 ? (int)((c1 - c0 + 2 * p.tq - 1) / (2 * p.tq)) : 0;
}

// A CTA's run through (head, request, pair, tile).
struct Walk {
    int h, b, pair, pairs;
    int t0, t1;             // key tiles of the present piece: [t0, t1) of span.tiles
    int64_t left;           // tiles still to do, this piece's included
    Seen<kN> r;
    Span span;
    __device__ __forceinline__ void cut() {
        t1 = (int)(left < span.tiles - t0 ? t0 + left : span.tiles);
    }
    __device__ __forceinline__ void start(const AttnArgs& p, int h_, int b_, int pair_, int tile, int64_t n) {
        h = h_;
        b = b_;
        pair = pair_;
        left = n;
        r = seen_of<kN>(p, b);
        pairs = pairs_of(p, b);
        span = span_of(p, r, pair);
        t0 = tile;
        cut();
    }
    __device__ __forceinline__ bool next(const AttnArgs& p) {
        left -= t1 - t0;
        if (left <= 0) return false;
        if (++pair == pairs) {
            pair = 0;
            do {
                if (++b == p.batch) {
                    b = 0;
                    ++h;
                }
                pairs = pairs_of(p, b);
            } while (pairs == 0);
            r = seen_of<kN>(p, b);
        }
        span = span_of(p, r, pair);
        t0 = 0;
        cut();
        return true;
    }
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == span.tiles; }
};

// bits lo .. hi-1 of 32 (clipped)
__device__ __forceinline__ uint32_t bits(int lo, int hi) {
    lo = max(lo, 0);
    hi = min(hi, 32);
    if (hi <= lo) return 0u;
    return (0xffffffffu >> (32 - (hi - lo))) << lo;
}

// Meta words per CTA, as in the split kernel: [0] its partial 0 ends an item;
// [1] its partial 1 begins one; [2] request, [3] KV head, [4] pair.
constexpr int kMeta = 8;

template <int CODE, bool MOD>
__global__ void __launch_bounds__(kThreads, 1) q8_prompt_kernel(const AttnArgs p) {
    extern __shared__ uint8_t dyn[];
    __shared__ Shared sh;
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~(uintptr_t)1023);
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int cta = blockIdx.x;

    // ---- this CTA's range -------------------------------------------------
    // pairs of query tiles up to each request, then tiles up to each pair
    int* s_pairs = reinterpret_cast<int*>(base);   // [batch + 1], before the tiles use it
    {
        const int chunk = (p.batch + kThreads - 1) / kThreads;
        const int b0 = min(p.batch, t * chunk), b1 = min(p.batch, b0 + chunk);
        int64_t mine = 0;
        for (int b = b0; b < b1; ++b) mine += pairs_of(p, b);
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        if (lane == 31) sh.scan[warp] = incl;
        __syncthreads();
        int64_t ex = incl - mine, all = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) ex += sh.scan[w];
            all += sh.scan[w];
        }
        for (int b = b0; b < b1; ++b) {
            s_pairs[b] = (int)ex;
            ex += pairs_of(p, b);
        }
        if (t == 0) s_pairs[p.batch] = (int)all;
        __syncthreads();
    }
    const int n_pairs = s_pairs[p.batch];
    auto request_of = [&](int pair) {
        int lo = 0, hi = p.batch;
        while (hi - lo > 1) {
            const int m = (lo + hi) >> 1;
            if (s_pairs[m] <= pair) lo = m;
            else hi = m;
        }
        return lo;
    };
    int64_t total = 0, left = 0;
    int start_h = 0;
    {
        const int chunk = (n_pairs + kThreads - 1) / kThreads;
        const int q0 = min(n_pairs, t * chunk), q1 = min(n_pairs, q0 + chunk);
        int64_t mine = 0;
        int b = q0 < q1 ? request_of(q0) : 0;
        const int first_b = b;
        for (int i = q0; i < q1; ++i) {
            while (i >= s_pairs[b + 1]) ++b;
            mine += span_of(p, seen_of<kN>(p, b), i - s_pairs[b]).tiles;
        }
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        __syncthreads();
        if (lane == 31) sh.scan[warp] = incl;
        __syncthreads();
        int64_t ex = incl - mine, per_head = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) ex += sh.scan[w];
            per_head += sh.scan[w];
        }
        total = per_head * p.kv_heads;
        const int64_t per_cta = (total + gridDim.x - 1) / gridDim.x;
        const int64_t u0 = cta * per_cta, u1 = min(total, u0 + per_cta);
        left = u1 - u0;
        if (left > 0) {
            start_h = (int)(u0 / per_head);
            int64_t off = u0 % per_head;
            if (off >= ex && off < ex + mine) {
                off -= ex;
                int i = q0;
                b = first_b;
                for (;; ++i) {
                    while (i >= s_pairs[b + 1]) ++b;
                    const int n = span_of(p, seen_of<kN>(p, b), i - s_pairs[b]).tiles;
                    if (off < n) break;
                    off -= n;
                }
                sh.start_b = b;
                sh.start_pair = i - s_pairs[b];
                sh.start_off = off;
            }
        }
    }
    if (t < kMeta) p.meta[cta * kMeta + t] = 0;
    if (left <= 0) return;   // uniform over the CTA

    // ---- barriers and tensor memory ---------------------------------------
    if (t == 0) {
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&sh.k_full[i], 32 * kCodeWarps);
            tc::mbar_init(&sh.v_full[i], 32 * kCodeWarps);
            tc::mbar_init(&sh.k_empty[i], 1);
            tc::mbar_init(&sh.v_empty[i], 1);
            tc::mbar_init(&sh.s_full[i], 1);
            tc::mbar_init(&sh.p_full[i], kM);
            tc::mbar_init(&sh.pv_done[i], 1);
        }
        tc::mbar_init(&sh.q_full, 2 * kM);
        tc::mbar_init(&sh.drain, 1);
        sh.failed = 0;
        tc::fence_mbar_init();
    }
    if (warp == kSoftmaxWarps + kCodeWarps) {
        tc::tmem_alloc(&sh.tmem, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = sh.tmem;
    uint8_t* sK = base;
    uint8_t* sV = base + 2 * kTileBytes;
    uint8_t* sQ = base + 4 * kTileBytes;

    Walk w;
    w.start(p, start_h, sh.start_b, sh.start_pair, (int)sh.start_off, left);

    if (warp < kSoftmaxWarps) {
        // =================== softmax: one thread per row ====================
        const int i = warp >> 2, row = t & (kM - 1);
        const uint32_t quad = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + i * kN + quad, tO = tmem + 2 * kN + i * kHeadDim + quad;
        uint8_t* q_row = sQ + i * kTileBytes + row * 128;
        int n = 0;          // key tiles done
        bool ok = true;
        do {
            // ---- this row's query ----
            const int k = row / p.g;
            const int token = w.pair * 2 * p.tq + i * p.tq + k;
            const int head = w.h * p.g + row % p.g;
            const bool on = k < p.tq && token < w.r.n;
            float rowf;
            {
                const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                                  (int64_t)(w.r.first + (on ? token : 0)) * p.q_stride +
                                                                  head * kHeadDim);
                uint4 x[16];
                float top = 0.f;
#pragma unroll
                for (int c = 0; c < 16; ++c) x[c] = on ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    const uint32_t v[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(v[e] << 16)), fabsf(__uint_as_float(v[e] & 0xffff0000u))));
                }
                int up = 14 - ((int)(__float_as_uint(top) >> 23) - 127);
                up = max(-126, min(126, up));
                const float f = __uint_as_float((uint32_t)(up + 127) << 23);
                rowf = __uint_as_float((uint32_t)(127 - up) << 23) * (p.scale * (MOD ? 1.f : kLog2e));
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    const uint32_t v[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
                    uint32_t o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const __half2 hh = __floats2half2_rn(__uint_as_float(v[e] << 16) * f,
                                                             __uint_as_float(v[e] & 0xffff0000u) * f);
                        o[e] = *reinterpret_cast<const uint32_t*>(&hh);
                    }
                    *reinterpret_cast<uint4*>(q_row + (c >> 3) * kHalf + (((c & 7) ^ (row & 7)) << 4)) =
                        make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
            tc::fence_async_smem();
            tc::mbar_arrive(&sh.q_full);

            const int pos = w.r.len - w.r.n + min(token, w.r.n - 1);
            const int see_from = p.window > 0 ? max(-1, pos - p.window) : -1;   // sees (see_from, pos] and the prefix
            const float slope = MOD && p.slopes && on ? p.slopes[head] * kLog2e : 0.f;
            // the span of positions of this warp's rows
            const int wp_min = __reduce_min_sync(0xffffffffu, pos), wp_max = __reduce_max_sync(0xffffffffu, pos);
            float M = -INFINITY, l = 0.f;

            // page numbers two tiles ahead, scales one tile ahead
            auto page_at = [&](int ti, int half) {
                if (ti >= w.t1) return -1;
                const int tok = w.span.tile_of(ti) * kN + half * kPage;
                return tok < w.r.len ? __ldg(p.table + (int64_t)w.b * p.width + tok / kPage) : -1;
            };
            auto valid = [&](int page) { return page >= 0 && page < p.pages; };
            int pg[2] = {page_at(w.t0, 0), page_at(w.t0, 1)};
            float sk[2], sv[2];
            bool there[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                there[e] = valid(pg[e]);
                const int64_t at = (int64_t)(there[e] ? pg[e] : 0) * p.kv_heads + w.h;
                sk[e] = there[e] ? __ldg(p.k_scale + at) : 0.f;
                sv[e] = there[e] ? __ldg(p.v_scale + at) : 1.f;
                pg[e] = page_at(w.t0 + 1, e);
            }
            for (int ti = w.t0; ti < w.t1; ++ti, ++n) {
                float a[2], lsv[2], isv[2];
                bool use[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    a[e] = rowf * sk[e];
                    const float s = sv[e] > 0.f ? sv[e] : 1.f;
                    lsv[e] = lg2(s);
                    isv[e] = __fdividef(1.f, s);
                    use[e] = there[e];
                    there[e] = valid(pg[e]);
                    const int64_t at = (int64_t)(there[e] ? pg[e] : 0) * p.kv_heads + w.h;
                    sk[e] = there[e] ? __ldg(p.k_scale + at) : 0.f;
                    sv[e] = there[e] ? __ldg(p.v_scale + at) : 1.f;
                    pg[e] = page_at(ti + 2, e);
                }
                const int key0 = w.span.tile_of(ti) * kN;
                const bool clear = use[0] && use[1] && key0 + kN <= w.r.len &&
                                   ((key0 + kN - 1 <= wp_min && (p.window == 0 || key0 > wp_max - p.window)) ||
                                    key0 + kN <= w.r.pre);
                uint32_t mask[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
                if (!clear) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int k0 = key0 + 32 * c;
                        mask[c] = (bits(see_from + 1 - k0, pos + 1 - k0) | bits(0, w.r.pre - k0)) & bits(0, w.r.len - k0);
                        if (!use[c >> 1]) mask[c] = 0u;
                    }
                }
                ok = ok && wait_for(sh, &sh.s_full[i], n & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc::tc_fence_after();

                // ---- the row's maximum ----
                float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t s[32];
                    tmem_ld32(tS + 32 * c, s);
                    tc::tmem_wait_ld();
                    if (MOD) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            float x = __uint_as_float(s[e]) * a[c >> 1];
                            if (p.cap > 0.f) x = p.cap * tanh_abs(__fdividef(x, p.cap));
                            x = x * kLog2e - slope * fabsf((float)(pos - (key0 + 32 * c + e)));
                            s[e] = __float_as_uint(x);
                        }
                        tmem_st32(tS + 32 * c, s);
                    }
                    float m = -INFINITY;
                    if (clear) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) m = fmaxf(m, __uint_as_float(s[e]));
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) m = fmaxf(m, (mask[c] >> e) & 1u ? __uint_as_float(s[e]) : -INFINITY);
                    }
                    top[c >> 1] = fmaxf(top[c >> 1], m);
                }
                if (MOD) {
                    tc::tmem_wait_st();
                    a[0] = a[1] = 1.f;
                }
                float now = -INFINITY;
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (top[e] > -INFINITY) now = fmaxf(now, fmaf(top[e], a[e], lsv[e]));
                const bool raise = now > M + kRaise || (M == -INFINITY && now > -INFINITY);
                if (__any_sync(0xffffffffu, raise)) {
                    const float f = raise && M > -INFINITY ? ex2(M - now) : 1.f;
                    if (raise) M = now;
                    l *= f;
                    if (ti > w.t0) {   // the accumulator holds earlier tiles
                        ok = wait_for(sh, &sh.pv_done[i], (n - 1) & 1);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        tc::tc_fence_after();
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            uint32_t o[32];
                            tmem_ld32(tO + 32 * c, o);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st32(tO + 32 * c, o);
                        }
                    }
                }
                // ---- weights ----
                // One fused multiply-add per weight: x - M with x unrounded, M and
                // M - log2 s_v rounded, off by 2^-24 |M| between pages.  Beyond
                // |M| = 2^10 (and for hidden keys) x is rounded like M was, so that
                // the row's largest key gives exactly x - M = 0.
                const float Mb = M == -INFINITY ? 0.f : M;
                const bool plain = clear && __all_sync(0xffffffffu, fabsf(Mb) < 1024.f);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t s[32], o[16];
                    tmem_ld32(tS + 32 * c, s);
                    tc::tmem_wait_ld();
                    const float aa = a[c >> 1], ls = lsv[c >> 1], bb = ls + (kShift - Mb);
                    float sum = 0.f;
                    if (plain) {
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const float x = ex2(fmaf(__uint_as_float(s[e]), aa, bb));
                            const float y = ex2(fmaf(__uint_as_float(s[e + 1]), aa, bb));
                            sum += x + y;
                            const __half2 hh = __floats2half2_rn(x, y);
                            o[e >> 1] = *reinterpret_cast<const uint32_t*>(&hh);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float x = ex2((fmaf(__uint_as_float(s[e]), aa, ls) - Mb) + kShift);
                            float y = ex2((fmaf(__uint_as_float(s[e + 1]), aa, ls) - Mb) + kShift);
                            x = (mask[c] >> e) & 1u ? x : 0.f;
                            y = (mask[c] >> (e + 1)) & 1u ? y : 0.f;
                            sum += x + y;
                            const __half2 hh = __floats2half2_rn(x, y);
                            o[e >> 1] = *reinterpret_cast<const uint32_t*>(&hh);
                        }
                    }
                    l += sum * isv[c >> 1];
                    tc::tmem_st16(tS + 16 * c, o);
                }
                tc::tmem_wait_st();
                tc::tc_fence_before();
                tc::mbar_arrive(&sh.p_full[i]);
            }
            if (!ok) break;

            // ---- end of the piece ----
            ok = wait_for(sh, &sh.pv_done[i], (n - 1) & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc::tc_fence_after();
            const bool whole = w.whole();
            const int slot = cta * 2 + (w.t0 == 0 ? 1 : 0);
            const int64_t at = (int64_t)slot * (2 * kM) + i * kM + row;
            const float inv = l > 0.f ? __fdiv_rn(1.f, l) : (l == 0.f ? 0.f : l);
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) +
                                 ((int64_t)(w.r.first + token) * p.kv_heads * p.g + head) * kHeadDim;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t o[32];
                __syncwarp();
                tmem_ld32(tO + 32 * c, o);
                tc::tmem_wait_ld();
                if (!on) {
                } else if (whole) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        uint32_t v[4];
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(o[e + 2 * z]) * inv,
                                                                            __uint_as_float(o[e + 2 * z + 1]) * inv);
                            v[z] = *reinterpret_cast<const uint32_t*>(&b2);
                        }
                        *reinterpret_cast<uint4*>(out + 32 * c + e) = make_uint4(v[0], v[1], v[2], v[3]);
                    }
                } else {
                    float4* to = reinterpret_cast<float4*>(p.part + at * kHeadDim + 32 * c);
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        to[e / 4] = make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]),
                                                __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
                }
            }
            if (!whole) {
                if (on) *reinterpret_cast<float2*>(p.ml + at * 2) = make_float2(M, l);
                if (t == 0) {
                    int* m = p.meta + cta * kMeta;
                    if (w.t0 > 0) {
                        m[0] = w.t1 == w.span.tiles;
                    } else {
                        m[1] = 1;
                        m[2] = w.b;
                        m[3] = w.h;
                        m[4] = w.pair;
                    }
                }
            }
            tc::tc_fence_before();
        } while (w.next(p));
    } else if (warp < kSoftmaxWarps + kCodeWarps) {
        // =================== codes to operand tiles =========================
        // Per pass a warp takes 4 rows of 128 codes, 8 lanes a row.  A lane's 16
        // codes become chunks 2c and 2c + 1 of one 64-column half; lanes of the
        // second half store theirs in the other order, which keeps the 8 lanes
        // of a row on different banks.
        const int u = t - 32 * kSoftmaxWarps;
        const int c = u & 7, row0 = u >> 3;           // 16 rows per pass, 8 passes
        const int first = c >> 2;                     // which of its two chunks goes first
        int n = 0;
        uint4 ck[8], cv[8];
        auto load = [&](int ti) {
            const int tok0 = w.span.tile_of(ti) * kN;
            int pages[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int tok = tok0 + e * kPage;
                pages[e] = tok < w.r.len ? __ldg(p.table + (int64_t)w.b * p.width + tok / kPage) : -1;
            }
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                const int rr = s * 16 + row0;
                const int page = pages[s >> 2];
                const bool on = page >= 0 && page < p.pages && tok0 + rr < w.r.len;
                const int64_t at = ((int64_t)page * p.kv_heads + w.h) * (kPage * kHeadDim) + (rr & (kPage - 1)) * kHeadDim + c * 16;
                ck[s] = on ? __ldg(reinterpret_cast<const uint4*>(p.k + at)) : make_uint4(0u, 0u, 0u, 0u);
                cv[s] = on ? __ldg(reinterpret_cast<const uint4*>(p.v + at)) : make_uint4(0u, 0u, 0u, 0u);
            }
        };
        auto put = [&](uint8_t* tile, const uint4 (&x)[8]) {
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                const int rr = s * 16 + row0;
                uint8_t* to = tile + (c >> 2) * kHalf + rr * 128;
                const uint32_t v[4] = {Codes<CODE>::bias(x[s].x), Codes<CODE>::bias(x[s].y), Codes<CODE>::bias(x[s].z),
                                       Codes<CODE>::bias(x[s].w)};
                const uint4 lo = make_uint4(Codes<CODE>::lo(v[0]), Codes<CODE>::hi(v[0]), Codes<CODE>::lo(v[1]), Codes<CODE>::hi(v[1]));
                const uint4 hi = make_uint4(Codes<CODE>::lo(v[2]), Codes<CODE>::hi(v[2]), Codes<CODE>::lo(v[3]), Codes<CODE>::hi(v[3]));
                const int c0 = 2 * (c & 3);
                *reinterpret_cast<uint4*>(to + (((c0 + first) ^ (rr & 7)) << 4)) = first ? hi : lo;
                *reinterpret_cast<uint4*>(to + (((c0 + 1 - first) ^ (rr & 7)) << 4)) = first ? lo : hi;
            }
        };
        bool ok = true;
        load(w.t0);
        int ti = w.t0;
        for (;;) {
            const int st = n & 1;
            const uint32_t free_par = ((n >> 1) & 1) ^ 1;
            ok = wait_for(sh, &sh.k_empty[st], free_par);
            if (!ok) break;
            put(sK + st * kTileBytes, ck);
            tc::fence_async_smem();
            tc::mbar_arrive(&sh.k_full[st]);
            ok = wait_for(sh, &sh.v_empty[st], free_par);
            if (!ok) break;
            put(sV + st * kTileBytes, cv);
            tc::fence_async_smem();
            tc::mbar_arrive(&sh.v_full[st]);
            ++n;
            if (++ti == w.t1) {
                if (!w.next(p)) break;
                ti = w.t0;
            }
            load(ti);
        }
    } else if (lane == 0) {
        // =================== MMA ============================================
        const uint32_t idS = tc::idesc_f32acc(0, kM, kN, 0, 0), idO = tc::idesc_f32acc(0, kM, kHeadDim, 0, 1);
        const uint32_t aK = tc::smem_u32(sK), aV = tc::smem_u32(sV), aQ = tc::smem_u32(sQ);
        auto scores = [&](int i, int st) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t o = (k >> 2) * kHalf + (k & 3) * 32;
                tc::mma_f16_ss(tmem + i * kN, desc_sw128(aQ + i * kTileBytes + o, 16, 1024),
                               desc_sw128(aK + st * kTileBytes + o, 16, 1024), idS, k > 0);
            }
            tc::mma_commit(&sh.s_full[i]);
        };
        auto values = [&](int i, int st, bool more) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                tc::mma_f16_ts(tmem + 2 * kN + i * kHeadDim, tmem + i * kN + k * 8,
                               desc_sw128(aV + st * kTileBytes + k * 2048, kHalf, 1024), idO, more || k > 0);
            tc::mma_commit(&sh.pv_done[i]);
        };
        int n = 0, piece = 0;
        bool ok = true;
        do {
            ok = wait_for(sh, &sh.q_full, piece & 1) && wait_for(sh, &sh.k_full[n & 1], (n >> 1) & 1);
            if (!ok) break;
            tc::tc_fence_after();
            scores(0, n & 1);
            scores(1, n & 1);
            tc::mma_commit(&sh.k_empty[n & 1]);
            for (int ti = w.t0; ti < w.t1 && ok; ++ti, ++n) {
                const bool more = ti + 1 < w.t1;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (i == 0) ok = wait_for(sh, &sh.v_full[n & 1], (n >> 1) & 1);
                    ok = ok && wait_for(sh, &sh.p_full[i], n & 1);
                    if (!ok) break;
                    tc::tc_fence_after();
                    values(i, n & 1, ti > w.t0);
                    if (i == 1) tc::mma_commit(&sh.v_empty[n & 1]);
                    if (more) {
                        if (i == 0) ok = wait_for(sh, &sh.k_full[(n + 1) & 1], ((n + 1) >> 1) & 1);
                        if (!ok) break;
                        tc::tc_fence_after();
                        scores(i, (n + 1) & 1);
                        if (i == 1) tc::mma_commit(&sh.k_empty[(n + 1) & 1]);
                    }
                }
            }
            ++piece;
        } while (ok && w.next(p));
        // every MMA has ended before tensor memory is given back
        tc::mma_commit(&sh.drain);
        const long long deadline = clock64() + tc::kWaitCycles;
        tc::mbar_wait(&sh.drain, 0, deadline);
    }
    __syncwarp();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == kSoftmaxWarps + kCodeWarps) tc::tmem_dealloc(tmem, 512);
    if (t == 0 && sh.failed && p.status) atomicMin(p.status, ISKV_ERR_DEVICE_TIMEOUT);
}

// Pairs that several CTAs share: CTA c's partial 1 begins one, the partials 0
// of the CTAs after it go on, up to the one that ends it.
__global__ void __launch_bounds__(256) q8_prompt_join_kernel(const AttnArgs p) {
    const int cta = blockIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int* m = p.meta + cta * kMeta;
    if (m[1] == 0) return;
    int n = 0;
    while (cta + 1 + n < p.ctas) {
        ++n;
        if (p.meta[(cta + n) * kMeta] != 0) break;
    }
    const Seen<kN> r = seen_of<kN>(p, m[2]);
    const int lane = threadIdx.x & 31;
    const int rows = 2 * kM / gridDim.y;
    for (int k = threadIdx.x >> 5; k < rows; k += 8) {
        const int row = blockIdx.y * rows + k;
        const int q = (row & (kM - 1)) / p.g;
        const int token = m[4] * 2 * p.tq + (row / kM) * p.tq + q;
        if (q >= p.tq || token >= r.n) continue;
        const int head = m[3] * p.g + (row & (kM - 1)) % p.g;
        auto at = [&](int i) { return (int64_t)((cta + i) * 2 + (i == 0 ? 1 : 0)) * (2 * kM) + row; };
        float M = -INFINITY;
        for (int i = 0; i <= n; ++i) M = fmaxf(M, p.ml[at(i) * 2]);
        const float base = M == -INFINITY ? 0.f : M;
        float l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int i = 0; i <= n; ++i) {
            const float2 ml = *reinterpret_cast<const float2*>(p.ml + at(i) * 2);
            const float4 v = *reinterpret_cast<const float4*>(p.part + at(i) * kHeadDim + 4 * lane);
            const float f = ex2(ml.x - base);
            l += f * ml.y;
            o[0] += f * v.x;
            o[1] += f * v.y;
            o[2] += f * v.z;
            o[3] += f * v.w;
        }
        const float inv = l > 0.f ? __fdiv_rn(1.f, l) : (l == 0.f ? 0.f : l);
        const __nv_bfloat162 x = __floats2bfloat162_rn(o[0] * inv, o[1] * inv), y = __floats2bfloat162_rn(o[2] * inv, o[3] * inv);
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) +
                                  ((int64_t)(r.first + token) * p.kv_heads * p.g + head) * kHeadDim + 4 * lane) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
    }
}

template <int CODE, bool MOD>
cudaError_t run(const AttnArgs& a, cudaStream_t s) {
    static SmemOnce once;
    cudaError_t e = once.set(q8_prompt_kernel<CODE, MOD>, kSmemBytes);
    if (e != cudaSuccess) return e;
    q8_prompt_kernel<CODE, MOD><<<a.ctas, kThreads, kSmemBytes, s>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.ctas, 8);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, q8_prompt_join_kernel, a);
}

}  // namespace

cudaError_t launch_q8_prompt(const AttnArgs& a, int code, cudaStream_t s) {
    const bool mod = a.cap > 0.f || a.slopes != nullptr;
    if (code == ISKV_CODE_INT8) return mod ? run<ISKV_CODE_INT8, true>(a, s) : run<ISKV_CODE_INT8, false>(a, s);
    return mod ? run<ISKV_CODE_E4M3, true>(a, s) : run<ISKV_CODE_E4M3, false>(a, s);
}

}  // namespace q8
}  // namespace iskv
