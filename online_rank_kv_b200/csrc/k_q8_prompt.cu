// iskv_q8_attention for prompts: many query rows per KV head, on tcgen05.
//
// Mathematics: as in the split kernel (k_q8_rows.cu) -- codes are exact in
// fp16, the key scale multiplies scores, and one exponential
//     w = 2^(score log2 e + log2 s_v - M)
// gives the numerator sum w c_v and the denominator sum w / s_v.  M is raised
// only when a row's maximum has grown past it by more than 2^15, where weights
// would leave fp16, so the accumulator in tensor memory is rescaled once or
// twice per row, not per page.  (The largest weight is at least 1; at fp16's
// smallest steps the others are off by 2^-25 of it.)  Pages of scale 0 as there.
//
// One CTA per SM holds two tiles of 128 query rows (query tokens x the heads
// that share a KV head) and goes through the keys in steps of one page:
//   warps 0-3, 4-7  softmax of tile 0 and of tile 1, one thread per row: scores
//                   from TMEM, weights as fp16 back over them, and the rare
//                   rescaling; also load, scale and store their own Q rows
//   warps 8-11      turn codes (shared memory) into fp16 operand tiles
//   warps 12, 14    issue the MMAs of tile 0 and of tile 1: S_i = Q_i K^T,
//                   O_i += P_i V
//   warp 13         walks the CTA's work, looks up pages and scales 32 steps at
//                   a time and tells the others about each step through a ring
//                   of eight descriptions
//   warp 15         copies the steps' codes in (8 KB per operand by the bulk copy
//                   engine)
// Each tile has two score buffers of 64 columns: a tile's softmax works on one
// page's scores while the MMAs of the page before (its values, then the scores
// of the page after next, into the buffer that it frees) run, so neither waits
// for the other's latency.  TMEM: S_0, S_1 (fp32, two buffers of 64 columns
// each, the fp16 weights over a buffer's first half), O_0, O_1, 128 columns
// each.  K and V operand tiles have four buffers each, codes two.
//
// Work: (KV head, pair of query tiles, page) are numbered through and every
// CTA takes an equal contiguous range, so that causal triangles, ragged batches
// and short chunks on long caches all fill the GPU; a pair that crosses CTAs is
// joined from its partial sums by a second kernel.
//
// What bounds it: a page and pair of tiles is 1024 cycles of MMA at the nominal
// rate, about 1400 as issued here (64-column score products wait for Q in shared
// memory), and 1024 cycles of exponentials (16 per SM and clock) less the quarter
// on the FMA pipe.  It takes about 2000: the two tiles' chains -- weights handed
// over, their values' product, the scores after next, softmax -- do not overlap
// fully.  Whatever lengthens the way from scores to weights shows at once: the
// sums taken behind the hand-over instead of before it were 683 -> 574 us of an
// 8192-token prompt (32 query, 8 KV heads).  That prompt takes 557 us in a graph of
// four, 987 TFLOP/s, 60 % of the measured matrix rate, and 610 us in long runs, 55 %,
// at the power limit.  A cap takes the prompt to 1115 us, a distance bias to 1010:
// more arithmetic on the softmax warps, whose chain is the bound.  Tried and
// slower: 128-column scores in one buffer (726 against 659), no maximum but a check
// of the sums (645 against 558).
#include "q8_common.cuh"
#include "tc_util.cuh"

namespace iskv {
namespace q8 {

namespace {

constexpr int kM = 128;                    // query rows per tile
constexpr int kN = kPage;                  // keys per step
// fp16 operand tiles stand as two halves of 64 columns, rows of 128 bytes
constexpr int kHalf = kN * 128, kTileBytes = 2 * kHalf;     // K, V: 16 KB
constexpr int kQHalf = kM * 128, kQBytes = 2 * kQHalf;      // Q: 32 KB
constexpr int kBuffers = 4;                // K and V operand tiles
constexpr int kSoftmaxWarps = 8, kCodeWarps = 4;
// Registers per thread, by warpgroup: 2 x 176 + 80 + 80 = 4 x 128, what the
// launch has.
constexpr int kThreads = 32 * (kSoftmaxWarps + kCodeWarps + 4);
constexpr int kSoftmaxRegs = 176, kCodeRegs = 80, kOtherRegs = 80;
constexpr int kMmaWarp = kSoftmaxWarps + kCodeWarps, kWalkWarp = kMmaWarp + 1, kCopyWarp = kMmaWarp + 3;
// How far (in powers of two) a row's maximum may pass M before M is raised: the
// weights then reach 2^15.
constexpr float kRaise = 15.f;
// Of 4 pairs of exponentials, those taken on the FMA pipe (8192-token prompt:
// none 590 us, one of eight 568, one of four 558, two 607).
constexpr int kPolyOf4 = 1;
// What the start and the end of a pair cost, in steps, where work is split
// (8192-token prompt: 4 571 us, 6 553, 8 558, 12 570).
constexpr int kPieceSteps = 6;

// One step, as the walking warp describes it.
struct Step {
    int end, key0;          // end: of the work, nothing else holds then
    int left;               // steps of the piece that follow
    int page;               // -1: there is none
    float sk, lsv, isv;     // key scale, log2 of the value scale, its inverse (0: a page of scale 0)
    int len, pre, n, first; // the request: tokens, prefix, queries, first query row
    int token0, h;          // the pair's first query, KV head
    int slot;               // partial slot, -1: the piece is the whole pair
};
constexpr int kSteps = 8;

struct Shared {
    Step step[kSteps];
    uint64_t info_full[kSteps], info_empty[kSteps];
    uint64_t c_full[2][2], c_empty[2][2];                 // codes of K, of V
    uint64_t full[2][kBuffers], empty[2][kBuffers];       // operand tiles of K, of V
    uint64_t q_full[2], s_full[2][2], p_full[2][2], drain[2];
    // Even and odd steps apart: a softmax may be a step ahead of its values'
    // product, and a parity tells only neighbouring phases apart.
    uint64_t pv_done[2][2];
    uint32_t tmem;
    int failed;
    int64_t scan[16];
    int64_t start_off;
    int start_b, start_pair;
};
constexpr int kCodeBytes = kN * kHeadDim;   // K or V codes of a step: 8 KB
// dynamic shared memory: 1024-byte aligned [K tiles][V tiles][Q 2 tiles][K codes 2][V codes 2]
constexpr int kSmemBytes = 2 * kBuffers * kTileBytes + 2 * kQBytes + 4 * kCodeBytes + 1024;

template <int N>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

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
// Waits for this thread's TMEM loads.  The registers that they fill pass through
// the wait, so that no use of them can be moved in front of it.
__device__ __forceinline__ void tmem_wait(uint32_t (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]),
                   "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]),
                   "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_wait(uint32_t (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
                 :
                 : "memory");
}

// Two fp32 operations per instruction.
__device__ __forceinline__ uint64_t pair(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint32_t x, uint32_t y, uint64_t a, uint64_t b) {
    uint64_t r;
    asm("{\n\t.reg .b64 t;\n\tmov.b64 t, {%1, %2};\n\tfma.rn.f32x2 %0, t, %3, %4;\n\t}" : "=l"(r) : "r"(x), "r"(y), "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// Sums of weights: what is below 2^-126 counts as nothing (ex2_poly's hidden keys).
__device__ __forceinline__ uint64_t sum2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.ftz.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float2 split(uint64_t a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
    return r;
}
// The largest of three, NaN if any is.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// 2^x of two numbers on the FMA pipe: x = n + f with |f| <= 1/2, a polynomial for
// 2^f (minimax of the relative error, 2.7e-6; the weight is rounded to 2^-11
// behind it), n added to its exponent.  x is at most kRaise; from -126 down
// (hidden keys: -inf) the result is just below 2^-126, which fp16 drops and sum2
// takes as nothing.
__device__ __forceinline__ float2 ex2_poly(uint64_t x2) {
    const float2 x = split(x2);
    const uint64_t magic = pair(12582912.f, 12582912.f), minus = pair(-12582912.f, -12582912.f), one = pair(-1.f, -1.f);
    const uint64_t c = pair(fmaxf(x.x, -126.f), fmaxf(x.y, -126.f));
    const uint64_t r = add2(c, magic), n = add2(r, minus);
    const uint64_t f = fma2(n, one, c);
    uint64_t y = fma2(pair(0.009570102207362652f, 0.009570102207362652f), f, pair(0.05591785907745361f, 0.05591785907745361f));
    y = fma2(y, f, pair(0.240247443318367f, 0.240247443318367f));
    y = fma2(y, f, pair(0.6931217908859253f, 0.6931217908859253f));
    y = fma2(y, f, pair(0.9999992847442627f, 0.9999992847442627f));
    const float2 ry = split(r), yy = split(y);
    return make_float2(__uint_as_float(__float_as_uint(yy.x) + (__float_as_uint(ry.x) << 23)),
                       __uint_as_float(__float_as_uint(yy.y) + (__float_as_uint(ry.y) << 23)));
}

// 32 bytes to global memory: one store where the address allows it.
__device__ __forceinline__ void store32(void* to, const uint32_t (&v)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                     "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(to)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4*>(to)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
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
__device__ __forceinline__ bool wait_longer(const AttnArgs& p, Shared& sh, uint64_t* bar, uint32_t parity) {
    const long long deadline = clock64() + p.wait_cycles;
    while (!try_phase(p, bar, parity)) {
        if (*(volatile int*)&sh.failed) return false;
        if (clock64() > deadline) {
            sh.failed = 1;
            return false;
        }
    }
    return true;
}
// A lane's wait, and a warp's.  When one has given up, the warp's lanes leave their
// role together: lanes apart would miss each other at the next warp or CTA barrier.
__device__ __forceinline__ bool lane_wait(const AttnArgs& p, Shared& sh, uint64_t* bar, uint32_t parity) {
    return tc::mbar_try_wait(bar, parity) || wait_longer(p, sh, bar, parity);
}
__device__ __forceinline__ bool wait_for(const AttnArgs& p, Shared& sh, uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, lane_wait(p, sh, bar, parity));
}

// The steps that a pair of query tiles sees.
struct Span {
    int p0;            // position of the pair's first query
    int a, lo, steps;
    __device__ __forceinline__ int step_of(int i) const { return i < a ? i : i - a + lo; }
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
        s.steps = max(pre, hi);
    } else {
        s.a = pre;
        s.steps = pre + max(0, hi - s.lo);
    }
    if (s.steps == 0) s.steps = 1;   // nothing to see: one hidden step, so that zeros are written
    return s;
}

__device__ __forceinline__ int pairs_of(const AttnArgs& p, int b) {
    const int64_t c0 = p.cu[b] < 0 ? 0 : p.cu[b];
    const int64_t c1 = p.cu[b + 1] < p.tokens ? p.cu[b + 1] : p.tokens;
    return c1 > c0 ? (int)((c1 - c0 + 2 * p.tq - 1) / (2 * p.tq)) : 0;
}

// A CTA's run through (head, request, pair, step).  A pair costs its steps and
// kPieceSteps, which stand in front of them.
struct Walk {
    int h, b, pair, pairs;
    int t0, t1;             // the present piece: steps [t0, t1) of span.steps
    int64_t left;           // cost still to spend, this piece's included
    Seen<kN> r;
    Span span;
    // the piece from cost offset `off` of the pair on; false: no step of it is this CTA's
    __device__ __forceinline__ bool cut(int64_t off) {
        const int64_t end = off + left - kPieceSteps;
        t0 = off > kPieceSteps ? (int)(off - kPieceSteps) : 0;
        t1 = (int)(end < span.steps ? end : span.steps);
        left -= span.steps + kPieceSteps - off;
        return t1 > t0;
    }
    __device__ __forceinline__ bool start(const AttnArgs& p, int h_, int b_, int pair_, int64_t off, int64_t n) {
        h = h_;
        b = b_;
        pair = pair_;
        left = n;
        r = seen_of<kN>(p, b);
        pairs = pairs_of(p, b);
        span = span_of(p, r, pair);
        return cut(off);
    }
    __device__ __forceinline__ bool next(const AttnArgs& p) {
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
        return cut(0);
    }
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

// =================== softmax: one thread per row ============================
template <bool MOD>
__device__ __forceinline__ void softmax_role(const AttnArgs& p, Shared& sh, uint8_t* sQ, uint32_t tmem, int warp, int lane) {
    const int i = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t quad = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + i * 2 * kN + quad, tO = tmem + 4 * kN + i * kHeadDim + quad;
    const int k = row / p.g, hg = row % p.g;
    const int c16 = lane & 15, up16 = lane >> 4;
    uint8_t* const q_rows = sQ + i * kQBytes + (warp & 3) * 32 * 128;   // the warp's rows, both halves

    int token = 0, head = 0;
    bool on = false;
    uint4 x[16];   // the warp's queries: two rows per load, 16 lanes a row
    auto load = [&](const Step& st) {
        token = st.token0 + i * p.tq + k;
        head = st.h * p.g + hg;
        on = k < p.tq && token < st.n;
        const __nv_bfloat16* q0 = static_cast<const __nv_bfloat16*>(p.q) + (int64_t)st.first * p.q_stride + c16 * 8;
        const int64_t own = on ? (int64_t)token * p.q_stride + head * kHeadDim : -1;
#pragma unroll
        for (int z = 0; z < 16; ++z) {
            const int64_t src = __shfl_sync(0xffffffffu, own, 2 * z + up16);
            x[z] = src >= 0 ? *reinterpret_cast<const uint4*>(q0 + src) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    {
        const bool ok = wait_for(p, sh, &sh.info_full[0], 0);
        if (!ok || sh.step[0].end) return;
        load(sh.step[0]);
    }

    // of the piece before: running maximum and sum, its place
    float M = -INFINITY, l = 0.f;
    int64_t place = -1;
    int slot = -1;
    bool more = true;
    const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0, wide_part = (reinterpret_cast<uintptr_t>(p.part) & 31) == 0;
    for (int n = 0;;) {   // pieces
        // ---- queries (stored even where there are none any more: nothing reads them) ----
        float rowf = 0.f;
#pragma unroll
        for (int z = 0; z < 16; ++z) {
            const int r32 = 2 * z + up16;
            const uint32_t v[4] = {x[z].x, x[z].y, x[z].z, x[z].w};
            // bf16 magnitudes order like their bits: the row's largest exponent
            uint32_t top = __vmaxu2(__vmaxu2(v[0] & 0x7fff7fffu, v[1] & 0x7fff7fffu),
                                    __vmaxu2(v[2] & 0x7fff7fffu, v[3] & 0x7fff7fffu));
            top = max(top >> 16, top & 0xffffu);
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            // 2^up brings the row's largest element into [2^14, 2^15)
            const int up = max(-126, min(126, 14 - ((int)(top >> 7) - 127)));
            const float f = __uint_as_float((uint32_t)(up + 127) << 23);
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const __half2 hh = __floats2half2_rn(__uint_as_float(v[e] << 16) * f, __uint_as_float(v[e] & 0xffff0000u) * f);
                o[e] = *reinterpret_cast<const uint32_t*>(&hh);
            }
            *reinterpret_cast<uint4*>(q_rows + (c16 >> 3) * kQHalf + r32 * 128 + (((c16 & 7) ^ (r32 & 7)) << 4)) =
                make_uint4(o[0], o[1], o[2], o[3]);
            // the row's own thread keeps 2^-up
            const int mine = __shfl_sync(0xffffffffu, up, (lane & 1) << 4);
            if ((lane >> 1) == z)
                rowf = __uint_as_float((uint32_t)(127 - mine) << 23) * (p.scale * (MOD ? 1.f : kLog2e));
        }
        if (more) {
            tc::fence_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&sh.q_full[i]);
        }
        // ---- results of the piece before, while the next one's scores start ----
        if (n > 0) {
            const float inv = l > 0.f ? __fdiv_rn(1.f, l) : (l == 0.f ? 0.f : l);
            const int64_t at = (int64_t)slot * (2 * kM) + i * kM + row;
            __nv_bfloat16* const out = static_cast<__nv_bfloat16*>(p.out) + place;
            float* const part = p.part + at * kHeadDim;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t o[32];
                __syncwarp();
                tmem_ld32(tO + 32 * c, o);
                tmem_wait(o);
                if (place < 0) {
                } else if (slot < 0) {
#pragma unroll
                    for (int e = 0; e < 32; e += 16) {
                        uint32_t v[8];
#pragma unroll
                        for (int z = 0; z < 8; ++z) {
                            const __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(o[e + 2 * z]) * inv,
                                                                            __uint_as_float(o[e + 2 * z + 1]) * inv);
                            v[z] = *reinterpret_cast<const uint32_t*>(&b2);
                        }
                        store32(out + 32 * c + e, v, wide);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        const uint32_t v[8] = {o[e], o[e + 1], o[e + 2], o[e + 3], o[e + 4], o[e + 5], o[e + 6], o[e + 7]};
                        store32(part + 32 * c + e, v, wide_part);
                    }
                }
            }
            if (slot >= 0 && place >= 0) *reinterpret_cast<float2*>(p.ml + at * 2) = make_float2(M, l);
            tc::tc_fence_before();
            __syncwarp();
            if (!more) return;
        }

        const int n_q = sh.step[n % kSteps].n, len = sh.step[n % kSteps].len, pre = sh.step[n % kSteps].pre;
        const int pos = len - n_q + min(token, n_q - 1);
        const int see_from = p.window > 0 ? max(-1, pos - p.window) : -1;   // sees (see_from, pos] and the prefix
        const float slope = MOD && p.slopes && on ? p.slopes[head] * kLog2e : 0.f;
        const int wp_min = __reduce_min_sync(0xffffffffu, pos), wp_max = __reduce_max_sync(0xffffffffu, pos);
        M = -INFINITY;
        l = 0.f;
        bool huge = false;   // some row of the warp has |M| >= 2^10
        // log2 of the scale that pages of scale 0 take: that of the first other page
        // which the row sees (infinity: none yet, they count in scale 1)
        float lz = INFINITY;
        bool settled = false;

        for (bool first = true;; first = false) {   // steps
            const Step& st = sh.step[n % kSteps];
            bool ok = wait_for(p, sh, &sh.info_full[n % kSteps], (n / kSteps) & 1);
            if (!ok) return;
            const uint32_t tSn = tS + (n & 1) * kN;
            const int key0 = st.key0;
            const bool there = st.page >= 0;
            const bool clear = there && key0 + kN <= len &&
                               ((key0 + kN - 1 <= wp_min && (p.window == 0 || key0 > wp_max - p.window)) || key0 + kN <= pre);
            // the smallest normal number in place of zero keeps hidden scores at -inf
            float a = fmaxf(rowf * st.sk, 1.17549435e-38f);
            float lsv = st.lsv, isv = st.isv;
            const int left = st.left;
            const bool valued = isv > 0.f;
            __syncwarp();
            // (a piece's first step is given back behind its scores: the MMA warp
            // has read it then)
            if (left != 0 && !first && lane == 0) tc::mbar_arrive(&sh.info_empty[n % kSteps]);
            ok = wait_for(p, sh, &sh.s_full[i][n & 1], (n >> 1) & 1);
            if (!ok) return;
            if (left != 0 && first && lane == 0) tc::mbar_arrive(&sh.info_empty[n % kSteps]);
            tc::tc_fence_after();
            uint32_t s[kN];
            tmem_ld32(tSn, *reinterpret_cast<uint32_t(*)[32]>(s));
            tmem_ld32(tSn + 32, *reinterpret_cast<uint32_t(*)[32]>(s + 32));
            tmem_wait(*reinterpret_cast<uint32_t(*)[32]>(s));
            tmem_wait(*reinterpret_cast<uint32_t(*)[32]>(s + 32));
            if (MOD) {
                // (each choice once for all keys: made key by key they cost more than the work)
                if (p.cap > 0.f) {
                    float far = 0.f;
#pragma unroll
                    for (int e = 0; e < kN; ++e) far = fmaxf(far, fabsf(__uint_as_float(s[e])));
                    if (__all_sync(0xffffffffu, far * a * p.cap_inv < kCapLow)) {
#pragma unroll
                        for (int e = 0; e < kN; ++e) s[e] = __float_as_uint(capped_low(__uint_as_float(s[e]) * a, p.cap_inv));
                    } else {
#pragma unroll
                        for (int e = 0; e < kN; ++e) s[e] = __float_as_uint(capped(__uint_as_float(s[e]) * a, p.cap, p.cap_inv));
                    }
                    a = 1.f;
                }
                a *= kLog2e;
                if (p.slopes) {
                    const float d0 = (float)(pos - key0);
#pragma unroll
                    for (int e = 0; e < kN; ++e) s[e] = __float_as_uint(__uint_as_float(s[e]) * a - slope * fabsf(d0 - (float)e));
                    a = 1.f;
                }
            }
            if (!clear) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int k0 = key0 + 32 * c;
                    uint32_t m = (bits(see_from + 1 - k0, pos + 1 - k0) | bits(0, pre - k0)) & bits(0, len - k0);
                    if (!there) m = 0u;
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (!((m >> e) & 1u)) s[32 * c + e] = 0xff800000u;   // -inf
                }
            }
            // ---- the row's maximum ----
            float top;
            {
                float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < kN; e += 2)
                    m[(e >> 1) & 3] = max3(m[(e >> 1) & 3], __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
                top = max3(m[0], m[1], max3(m[2], m[3], m[3]));
            }
            if (!(valued && settled)) {
                if (!valued) {
                    lsv = lz < INFINITY ? lz : 0.f;
                    isv = ex2(-lsv);
                } else {
                    if (top > -INFINITY && lz == INFINITY) {   // what came before counted in scale 1
                        M += lsv;
                        l *= isv;
                        lz = lsv;
                    }
                    settled = __all_sync(0xffffffffu, lz < INFINITY);
                    huge = __any_sync(0xffffffffu, M > -INFINITY && fabsf(M) >= 1024.f);
                }
            }
            const float now = fmaf(top, a, lsv);
            const bool raise = now > M + kRaise || (M == -INFINITY && now > -INFINITY);
            if (__any_sync(0xffffffffu, raise)) {
                const float f = raise && M > -INFINITY ? ex2(M - now) : 1.f;
                if (raise) M = now;
                huge = __any_sync(0xffffffffu, M > -INFINITY && fabsf(M) >= 1024.f);
                l *= f;
                if (!first) {   // the accumulator holds earlier steps
                    ok = wait_for(p, sh, &sh.pv_done[i][(n - 1) & 1], ((n - 1) >> 1) & 1);
                    if (!ok) return;
                    tc::tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < 8; ++c) {
                        uint32_t o[16];
                        tc::tmem_ld16(tO + 16 * c, o);
                        tmem_wait(o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tc::tmem_st16(tO + 16 * c, o);
                    }
                }
            }
            // ---- weights ----
            // One fused multiply-add per weight: x - M with x unrounded, M and
            // M - log2 s_v rounded, off by 2^-24 |M| between pages.  From
            // |M| = 2^10 on, x is rounded like M was first, so that the row's
            // largest key gives exactly x - M = 0.
            const float Mb = M == -INFINITY ? 0.f : M;
            float b = lsv - Mb;
            if (huge) {
#pragma unroll
                for (int e = 0; e < kN; ++e) s[e] = __float_as_uint(fmaf(__uint_as_float(s[e]), a, lsv) - Mb);
                a = 1.f;
                b = 0.f;
            }
            const uint64_t aa = pair(a, a), bb = pair(b, b);
            uint64_t sum0 = 0, sum1 = 0;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t o[16];
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const uint64_t x2 = fma2(s[32 * c + e], s[32 * c + e + 1], aa, bb);
                    float2 y;
                    if (((e >> 1) & 3) < kPolyOf4) {
                        y = ex2_poly(x2);
                    } else {
                        y = split(x2);
                        y.x = ex2(y.x);
                        y.y = ex2(y.y);
                    }
                    if (e & 2) sum1 = sum2(sum1, pair(y.x, y.y));
                    else sum0 = sum2(sum0, pair(y.x, y.y));
                    const __half2 hh = __floats2half2_rn(y.x, y.y);
                    o[e >> 1] = *reinterpret_cast<const uint32_t*>(&hh);
                }
                tc::tmem_st16(tSn + 16 * c, o);
            }
            tc::tmem_wait_st();
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&sh.p_full[i][n & 1]);
            const float2 s2 = split(sum2(sum0, sum1));   // (nobody waits for these)
            // (a score that is NaN or +infinity, of a query that is not finite, makes the
            // row NaN; ex2_poly would pass over it)
            l = top < INFINITY ? l + (s2.x + s2.y) * isv : __int_as_float(0x7fffffff);
            if (left == 0) break;
            ++n;
        }

        // ---- end of the piece: the next one's queries, and the last values ----
        {
            const Step& st = sh.step[n % kSteps];
            slot = st.slot;
            place = on ? ((int64_t)(st.first + token) * p.kv_heads * p.g + head) * kHeadDim : -1;
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&sh.info_empty[n % kSteps]);
        }
        const int last = n++;
        bool ok = wait_for(p, sh, &sh.info_full[n % kSteps], (n / kSteps) & 1);
        if (!ok) return;
        more = !sh.step[n % kSteps].end;
        if (more) load(sh.step[n % kSteps]);
        ok = wait_for(p, sh, &sh.pv_done[i][last & 1], (last >> 1) & 1);
        if (!ok) return;
        tc::tc_fence_after();
    }
}

// =================== codes to operand tiles =================================
// Per pass 8 threads take 128 codes, 16 each, which become two neighbouring
// 16-byte chunks of one 64-column half.  The 4 threads of the second half take
// the neighbouring row: its swizzle differs in the lowest bit, so the 8 stores
// go to different banks.
template <int CODE>
__device__ __forceinline__ void code_tile(uint8_t* tile, const uint8_t* codes, int u, int rows) {
    const int c = u & 7, row0 = (u >> 3) ^ (c >> 2), c0 = 2 * (c & 3);
    uint4 x[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) x[s] = *reinterpret_cast<const uint4*>(codes + (s * 16 + row0) * kHeadDim + c * 16);
    if (rows < kN) {   // behind the last token, or a page that is not there
#pragma unroll
        for (int s = 0; s < 4; ++s)
            if (s * 16 + row0 >= rows) x[s] = make_uint4(0u, 0u, 0u, 0u);
    }
    uint8_t* const to = tile + (c >> 2) * kHalf + row0 * 128;
    uint8_t* const to0 = to + ((c0 ^ (row0 & 7)) << 4);
    uint8_t* const to1 = to + (((c0 + 1) ^ (row0 & 7)) << 4);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const uint32_t v[4] = {Codes<CODE>::bias(x[s].x), Codes<CODE>::bias(x[s].y), Codes<CODE>::bias(x[s].z),
                               Codes<CODE>::bias(x[s].w)};
        *reinterpret_cast<uint4*>(to0 + s * 2048) =
            make_uint4(Codes<CODE>::lo(v[0]), Codes<CODE>::hi(v[0]), Codes<CODE>::lo(v[1]), Codes<CODE>::hi(v[1]));
        *reinterpret_cast<uint4*>(to1 + s * 2048) =
            make_uint4(Codes<CODE>::lo(v[2]), Codes<CODE>::hi(v[2]), Codes<CODE>::lo(v[3]), Codes<CODE>::hi(v[3]));
    }
}

template <int CODE>
__device__ __forceinline__ void code_role(const AttnArgs& p, Shared& sh, uint8_t* sK, const uint8_t* sKc, int u, int lane) {
    for (int n = 0;; ++n) {
        const Step& st = sh.step[n % kSteps];
        bool ok = lane_wait(p, sh, &sh.info_full[n % kSteps], (n / kSteps) & 1);
        const int rows = st.page >= 0 ? st.len - st.key0 : 0;
        const bool valued = st.isv > 0.f;   // (what scale 0 multiplies is nothing, whatever the codes)
        if (!__all_sync(0xffffffffu, ok && !st.end)) return;
        if (lane == 0) tc::mbar_arrive(&sh.info_empty[n % kSteps]);
        const int bf = n % kBuffers;
#pragma unroll 1
        for (int v = 0; v < 2; ++v) {   // K, then V
            ok = lane_wait(p, sh, &sh.c_full[v][n & 1], (n >> 1) & 1) &&
                 lane_wait(p, sh, &sh.empty[v][bf], ((n / kBuffers) & 1) ^ 1);
            if (ok) code_tile<CODE>(sK + (kBuffers * v + bf) * kTileBytes, sKc + (2 * v + (n & 1)) * kCodeBytes, u, v == 0 || valued ? rows : 0);
            tc::fence_async_smem();
            if (!__all_sync(0xffffffffu, ok)) return;
            if (lane == 0) {
                tc::mbar_arrive(&sh.full[v][bf]);
                tc::mbar_arrive(&sh.c_empty[v][n & 1]);
            }
        }
    }
}

// =================== MMA ====================================================
// The whole warp runs this and one lane issues: the descriptors then stay in
// uniform registers (a branch for one lane around it all costs 100 cycles per
// MMA beside the other warps, against the 64 that the MMA itself takes).
__device__ __forceinline__ bool elect() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// Tile i's MMAs.  A step's description is read where a piece begins only, without
// an arrival of its own: the softmax warps of both tiles give a piece's first step
// back behind its scores, which either MMA warp issues after this read.
__device__ __forceinline__ void mma_role(const AttnArgs& p, Shared& sh, uint32_t aK, uint32_t aQ, uint32_t tmem, int i) {
    constexpr uint32_t idS = tc::idesc_f32acc(0, kM, kN, 0, 0), idO = tc::idesc_f32acc(0, kM, kHeadDim, 0, 1);
    const uint64_t dK = desc_sw128(aK, 16, 1024), dQ = desc_sw128(aQ + i * kQBytes, 16, 1024);
    const uint64_t dV = desc_sw128(aK + kBuffers * kTileBytes, kHalf, 1024);
    const uint32_t tS = tmem + 2 * i * kN, tO = tmem + 4 * kN + i * kHeadDim;
    const bool leader = elect();   // one lane for all: a commit covers its own thread's MMAs
    auto waited = [&](uint64_t* bar, uint32_t parity) { return wait_for(p, sh, bar, parity); };
    // scores of step n (descriptors step in units of 16 bytes); false: a wait gave up
    auto scores = [&](int n) {
        const int bf = n % kBuffers;
        if (!waited(&sh.full[0][bf], (n / kBuffers) & 1)) return false;
        tc::tc_fence_after();
        const uint64_t b = dK + bf * (kTileBytes >> 4);
        if (leader) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                tc::mma_f16_ss(tS + (n & 1) * kN, dQ + (((k >> 2) * kQHalf + (k & 3) * 32) >> 4),
                               b + (((k >> 2) * kHalf + (k & 3) * 32) >> 4), idS, k > 0);
            tc::mma_commit(&sh.s_full[i][n & 1]);
            tc::mma_commit(&sh.empty[0][bf]);
        }
        __syncwarp();
        return true;
    };
    bool ok = true;
    for (int n = 0, piece = 0; ok; ++piece) {
        ok = waited(&sh.info_full[n % kSteps], (n / kSteps) & 1);
        if (!ok || uniform(sh.step[n % kSteps].end)) break;
        int ahead = 0;                     // steps of the piece whose scores are on their way
        const int steps = uniform(sh.step[n % kSteps].left) + 1;
        ok = waited(&sh.q_full[i], piece & 1);
        // the scores run two steps ahead of the values
#pragma unroll 1
        for (int z = -2; z < steps && ok; ++z) {
            if (z >= 0) {
                const int m = n + z, bf = m % kBuffers;
                ok = waited(&sh.full[1][bf], (m / kBuffers) & 1) && waited(&sh.p_full[i][m & 1], (m >> 1) & 1);
                if (!ok) break;
                tc::tc_fence_after();
                const uint64_t b = dV + bf * (kTileBytes >> 4);
                const uint32_t more = z > 0 ? 1u : 0u;
                if (leader) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc::mma_f16_ts(tO, tS + (m & 1) * kN + k * 8, b + k * (2048 >> 4), idO, k > 0 ? 1u : more);
                    tc::mma_commit(&sh.pv_done[i][m & 1]);
                    tc::mma_commit(&sh.empty[1][bf]);
                }
                __syncwarp();
            }
            if (ahead < steps) ok = scores(n + ahead++);
        }
        n += steps;
    }
    // every MMA has ended before tensor memory is given back
    if (leader) tc::mma_commit(&sh.drain[i]);
    __syncwarp();
    tc::mbar_wait(&sh.drain[i], 0, clock64() + tc::kWaitCycles);
}

// =================== the walk ===============================================
__device__ __forceinline__ void walk_role(const AttnArgs& p, Shared& sh, int start_h, int64_t left, int lane) {
    Walk w;
    bool more = w.start(p, start_h, sh.start_b, sh.start_pair, sh.start_off, left);
    if (!more) more = w.next(p);
    int n = 0;
    bool ok = true;
    while (ok && more) {
        const bool begins = w.t0 == 0, ends = w.t1 == w.span.steps;
        const int slot = begins && ends ? -1 : (int)blockIdx.x * 2 + (begins ? 1 : 0);
        if (lane == 0 && slot >= 0) {
            int* m = p.meta + blockIdx.x * kMeta;
            if (!begins) {
                m[0] = ends;
            } else {
                m[1] = 1;
                m[2] = w.b;
                m[3] = w.h;
                m[4] = w.pair;
            }
        }
        // its queries are on their way to L2 while the piece before is worked on
        for (int row = lane; row < 2 * kM; row += 32) {
            const int rr = row & (kM - 1), k = rr / p.g, token = w.pair * 2 * p.tq + (row / kM) * p.tq + k;
            if (k < p.tq && token < w.r.n) {
                const __nv_bfloat16* at = static_cast<const __nv_bfloat16*>(p.q) + (int64_t)(w.r.first + token) * p.q_stride +
                                          (w.h * p.g + rr % p.g) * kHeadDim;
                asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
                asm volatile("prefetch.global.L2 [%0];" ::"l"(at + 64));
            }
        }
        int page = -1;
        float sk = 0.f, lsv = 0.f, isv = 1.f;
        for (int i = w.t0; i < w.t1; ++i, ++n) {
            const int in = (i - w.t0) & 31;
            if (in == 0) {   // pages and scales of 32 steps, one per lane
                const int j = i + lane;
                const int tok = w.span.step_of(j) * kN;
                page = j < w.t1 && tok < w.r.len ? p.table[(int64_t)w.b * p.width + tok / kPage] : -1;
                if (page >= p.pages) page = -1;
                const int64_t at = (int64_t)max(page, 0) * p.kv_heads + w.h;
                sk = page >= 0 ? p.k_scale[at] : 0.f;
                const float sv = page >= 0 ? p.v_scale[at] : 0.f;
                lsv = lg2(sv);
                isv = sv > 0.f ? __fdividef(1.f, sv) : 0.f;
            }
            ok = wait_for(p, sh, &sh.info_empty[n % kSteps], ((n / kSteps) & 1) ^ 1);
            if (!ok) break;
            if (lane == in) {
                Step& st = sh.step[n % kSteps];
                st.end = 0;
                st.key0 = w.span.step_of(i) * kN;
                st.left = w.t1 - 1 - i;
                st.page = page;
                st.sk = sk;
                st.lsv = lsv;
                st.isv = isv;
                st.len = w.r.len;
                st.pre = w.r.pre;
                st.n = w.r.n;
                st.first = w.r.first;
                st.token0 = w.pair * 2 * p.tq;
                st.h = w.h;
                st.slot = slot;
                tc::mbar_arrive(&sh.info_full[n % kSteps]);
            }
            __syncwarp();
        }
        if (ok) more = w.next(p);
    }
    if (ok) {
        ok = wait_for(p, sh, &sh.info_empty[n % kSteps], ((n / kSteps) & 1) ^ 1);
        if (ok && lane == 0) {
            sh.step[n % kSteps].end = 1;
            tc::mbar_arrive(&sh.info_full[n % kSteps]);
        }
    }
}

// =================== copies of codes ========================================
__device__ __forceinline__ void copy_role(const AttnArgs& p, Shared& sh, uint8_t* sKc, int lane) {
    bool ok = true;
    for (int n = 0;; ++n) {
        ok = wait_for(p, sh, &sh.info_full[n % kSteps], (n / kSteps) & 1);
        if (!ok || sh.step[n % kSteps].end) break;
        const int page = sh.step[n % kSteps].page;
        const int64_t at = ((int64_t)max(page, 0) * p.kv_heads + sh.step[n % kSteps].h) * kCodeBytes;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sh.info_empty[n % kSteps]);
#pragma unroll 1
        for (int v = 0; v < 2 && ok; ++v) {   // K, then V
            ok = wait_for(p, sh, &sh.c_empty[v][n & 1], ((n >> 1) & 1) ^ 1);
            if (ok && lane == 0) {
                uint64_t* bar = &sh.c_full[v][n & 1];
                tc::mbar_arrive_expect_tx(bar, page >= 0 ? kCodeBytes : 0);
                if (page >= 0) tc::bulk_g2s(sKc + (2 * v + (n & 1)) * kCodeBytes, (v ? p.v : p.k) + at, kCodeBytes, bar);
            }
            __syncwarp();
        }
        if (!ok) break;
    }
}

template <int CODE, bool MOD>
__global__ void __launch_bounds__(kThreads, 1) q8_prompt_kernel(const AttnArgs p) {
    extern __shared__ uint8_t dyn[];
    __shared__ Shared sh;
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~(uintptr_t)1023);
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int cta = blockIdx.x;
    let_next();
    after_previous();

    // ---- this CTA's range -------------------------------------------------
    // pairs of query tiles up to each request, then cost up to each pair
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
            mine += span_of(p, seen_of<kN>(p, b), i - s_pairs[b]).steps + kPieceSteps;
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
                    const int n = span_of(p, seen_of<kN>(p, b), i - s_pairs[b]).steps + kPieceSteps;
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
        for (int i = 0; i < kSteps; ++i) {
            tc::mbar_init(&sh.info_full[i], 1);
            tc::mbar_init(&sh.info_empty[i], kSoftmaxWarps + kCodeWarps + 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&sh.q_full[i], kSoftmaxWarps / 2);
            tc::mbar_init(&sh.drain[i], 1);
            for (int z = 0; z < kBuffers; ++z) {
                tc::mbar_init(&sh.full[i][z], kCodeWarps);
                tc::mbar_init(&sh.empty[i][z], 2);
            }
            for (int z = 0; z < 2; ++z) {
                tc::mbar_init(&sh.c_full[i][z], 1);
                tc::mbar_init(&sh.c_empty[i][z], kCodeWarps);
                tc::mbar_init(&sh.s_full[i][z], 1);
                tc::mbar_init(&sh.pv_done[i][z], 1);
                tc::mbar_init(&sh.p_full[i][z], kSoftmaxWarps / 2);
            }
        }
        sh.failed = 0;
        tc::fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tc::tmem_alloc(&sh.tmem, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = sh.tmem;
    uint8_t* sK = base;                                   // K tiles, then V tiles
    uint8_t* sQ = base + 2 * kBuffers * kTileBytes;
    uint8_t* sKc = sQ + 2 * kQBytes;                      // K codes, then V codes

    if (warp < kSoftmaxWarps) {
        more_registers<kSoftmaxRegs>();
        softmax_role<MOD>(p, sh, sQ, tmem, warp, lane);
    } else if (warp < kSoftmaxWarps + kCodeWarps) {
        fewer_registers<kCodeRegs>();
        code_role<CODE>(p, sh, sK, sKc, t - 32 * kSoftmaxWarps, lane);
    } else {
        fewer_registers<kOtherRegs>();
        if (warp == kMmaWarp || warp == kMmaWarp + 2) {
            mma_role(p, sh, uniform(tc::smem_u32(sK)), uniform(tc::smem_u32(sQ)), uniform(tmem), uniform(warp - kMmaWarp) >> 1);
        } else if (warp == kWalkWarp) {
            walk_role(p, sh, start_h, left, lane);
        } else if (warp == kCopyWarp) {
            copy_role(p, sh, sKc, lane);
        }
    }
    __syncwarp();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (sh.failed) {
        // copies may be on their way to readers that have given up: they land
        // within microseconds; the CTA ends long after
        if (t == 0 && p.status) atomicMin(p.status, ISKV_ERR_DEVICE_TIMEOUT);
        const long long until = clock64() + 20000000;
        while (clock64() < until) __nanosleep(1000);
        __syncthreads();
    }
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 512);
}

// Pairs that several CTAs share: CTA c's partial 1 begins one, the partials 0
// of the CTAs after it go on, up to the one that ends it.  A warp joins a row at
// a time, its partials' maxima in the lanes.
__global__ void __launch_bounds__(256) q8_prompt_join_kernel(const AttnArgs p) {
    const int cta = blockIdx.x, lane = threadIdx.x & 31;
    // (no let_next(): 558 us with it, 555 without for one prompt of 8192 tokens,
    // 1285 against 1254 for 8 layers of 512 new ones behind up to 20K)
    after_previous();
    const int* m = p.meta + cta * kMeta;
    if (m[1] == 0) return;
    const int b = m[2], h = m[3], pair = m[4];
    int n = 1;   // partials
#pragma unroll 1
    for (int c0 = cta + 1; c0 < p.ctas; c0 += 32) {
        const uint32_t hit = __ballot_sync(0xffffffffu, c0 + lane < p.ctas && p.meta[(c0 + lane) * kMeta] != 0);
        n += hit ? __ffs(hit) : 32;
        if (hit) break;
    }
    n = min(n, p.ctas - cta);
    const Seen<kN> r = seen_of<kN>(p, b);
    const int rows = 2 * kM / gridDim.y;
#pragma unroll 1
    for (int k = threadIdx.x >> 5; k < rows; k += 8) {
        const int row = blockIdx.y * rows + k, in = row & (kM - 1), q = in / p.g;
        const int token = pair * 2 * p.tq + (row / kM) * p.tq + q, head = h * p.g + in - q * p.g;
        if (q >= p.tq || token >= r.n) continue;
        auto at = [&](int i) { return (int64_t)((cta + i) * 2 + (i == 0 ? 1 : 0)) * (2 * kM) + row; };
        float M = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int i0 = 0; i0 < n; i0 += 32) {
            const float2 ml = i0 + lane < n ? *reinterpret_cast<const float2*>(p.ml + at(i0 + lane) * 2) : make_float2(-INFINITY, 0.f);
            const float now = fmaxf(M, warp_max(ml.x)), base = now == -INFINITY ? 0.f : now;
            const float f = ex2(ml.x - base), g = ex2(M - base);
            l = l * g + warp_sum(f * ml.y);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] *= g;
            M = now;
            const int c = min(32, n - i0);
#pragma unroll 4
            for (int i = 0; i < c; ++i) {
                const float4 v = *reinterpret_cast<const float4*>(p.part + at(i0 + i) * kHeadDim + 4 * lane);
                const float w = __shfl_sync(0xffffffffu, f, i);
                o[0] += w * v.x;
                o[1] += w * v.y;
                o[2] += w * v.z;
                o[3] += w * v.w;
            }
        }
        const float inv = l > 0.f ? __fdividef(1.f, l) : (l == 0.f ? 0.f : l);
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
    e = launch_early(q8_prompt_kernel<CODE, MOD>, dim3(a.ctas), kThreads, kSmemBytes, s, 0, a);
    if (e != cudaSuccess) return e;
    return launch_early(q8_prompt_join_kernel, dim3(a.ctas, 16), 256, 0, s, 0, a);
}

}  // namespace

cudaError_t launch_q8_prompt(const AttnArgs& a, int code, cudaStream_t s) {
    const bool mod = a.cap > 0.f || a.slopes != nullptr;
    if (code == ISKV_CODE_INT8) return mod ? run<ISKV_CODE_INT8, true>(a, s) : run<ISKV_CODE_INT8, false>(a, s);
    return mod ? run<ISKV_CODE_E4M3, true>(a, s) : run<ISKV_CODE_E4M3, false>(a, s);
}

}  // namespace q8
}  // namespace iskv
