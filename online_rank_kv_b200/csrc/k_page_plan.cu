// iskv_page_plan: one step of the page tables, from request lengths.
//
// Three running sums over the requests carry the whole step: added tokens
// (cu), new blocks (which page of the stack each takes) and pages given back
// (where on the stack each goes).  Everything else follows from them: the
// j-th new block takes stack entry top - 1 - j, the k-th page given back is
// stack entry n_free + k, and a token's slot from its request's row.
//
// Bound by latency: a decode step moves a few kilobytes (64 requests 5.7 us, 1500
// requests with 30K new tokens 11 us).  So it is one launch
// of one cluster (1 to 8 CTAs, by the number of slots to write), in which
// every CTA sums over all requests by itself; nothing is exchanged but one
// cluster barrier, which ends the reads of lens and n_free before lens_out and
// n_free_out, which may be the same memory, are written.  No CTA reads what
// another one writes in the same step: a page that a new block takes is read
// from below n_free, or from the table row of the ended request that gives it
// back, and slots of new blocks find their page the same way instead of
// through the table.
#include <cooperative_groups.h>

#include "q8_common.cuh"

namespace cg = cooperative_groups;

namespace iskv {
namespace q8 {

namespace {

constexpr int kThreads = 1024;

// index of the last entry <= x in the ascending array v[0..n] (v[0] = 0 <= x < v[n])
__device__ __forceinline__ int last_at_most(const int* v, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (v[m] <= x) lo = m;
        else hi = m;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads) page_plan_kernel(const iskv_page_plan_args a) {
    extern __shared__ int sh[];
    let_next();
    after_previous();
    __shared__ long long warp_sum[3][32], s_total[3];
    const int B = a.batch;
    int* s_len = sh;                  // [B]
    int* s_cu = s_len + B;            // [B + 1]
    int* s_need = s_cu + B + 1;       // [B + 1]
    int* s_back = s_need + B + 1;     // [B + 1]
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int chunk = (B + kThreads - 1) / kThreads;
    const int b0 = min(B, t * chunk), b1 = min(B, b0 + chunk);
    const long long room = (long long)a.width * kPage;
    const long long n_free = *a.n_free;

    // this thread's requests
    long long sum[3] = {0, 0, 0};
    int bad_arg = n_free < 0 || n_free > a.pages, bad_cap = 0;
    for (int b = b0; b < b1; ++b) {
        const long long len = a.lens[b], add = a.add[b];
        s_len[b] = (int)len;
        if (len < 0 || len > room || add < -1) {
            bad_arg = 1;
            continue;
        }
        const long long had = (len + kPage - 1) / kPage;
        if (add < 0) {
            sum[2] += had;
        } else {
            if (len + add > room) bad_cap = 1;
            sum[0] += add;
            sum[1] += (len + add + kPage - 1) / kPage - had;
        }
    }
    // exclusive sums over the threads
    long long ex[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        long long v = sum[i];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        ex[i] = v - sum[i];
        if (lane == 31) warp_sum[i][warp] = v;
    }
    __syncthreads();
    if (warp < 3) {
        long long v = warp_sum[warp][lane];
        const long long own = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        warp_sum[warp][lane] = v - own;
        if (lane == 31) s_total[warp] = v;
    }
    bad_arg = __syncthreads_or(bad_arg);
    bad_cap = __syncthreads_or(bad_cap);
    long long total[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        ex[i] += warp_sum[i][warp];
        total[i] = s_total[i];
    }
    const long long top = n_free + total[2];
    if (!bad_arg && top > a.pages) bad_arg = 1;
    if (total[0] > a.tokens || total[1] > top) bad_cap = 1;
    const bool refused = bad_arg || bad_cap;

    if (!refused) {
        for (int b = b0; b < b1; ++b) {
            const int len = s_len[b], add = a.add[b];
            const int had = (len + kPage - 1) / kPage;
            s_cu[b] = (int)ex[0];
            s_need[b] = (int)ex[1];
            s_back[b] = (int)ex[2];
            if (add < 0) {
                ex[2] += had;
            } else {
                ex[0] += add;
                ex[1] += (len + add + kPage - 1) / kPage - had;
            }
        }
        if (t == 0) {
            s_cu[B] = (int)total[0];
            s_need[B] = (int)total[1];
            s_back[B] = (int)total[2];
        }
    }
    __syncthreads();
    cg::this_cluster().sync();   // every CTA has read lens and n_free

    const int gt = blockIdx.x * kThreads + t, step = gridDim.x * kThreads;
    const uint32_t n_slots = (uint32_t)a.tokens;   // (up to 2^31 - 1: steps past it stay within 32 bits without a sign)
    if (gt == 0) {
        *a.status = bad_arg ? ISKV_ERR_INVALID_ARG : bad_cap ? ISKV_ERR_CAPACITY : ISKV_OK;
        *a.n_free_out = (int)(refused ? n_free : top - total[1]);
    }
    if (refused) {
        for (int b = gt; b < B; b += step) a.lens_out[b] = s_len[b];
        for (int b = gt; b <= B; b += step) a.cu[b] = 0;
        for (uint32_t i = gt; i < n_slots; i += step) a.slots[i] = -1;
        return;
    }
    const int nf = (int)n_free, n1 = (int)top;
    const int added = (int)total[0], fresh = (int)total[1], back = (int)total[2];
    // the k-th page given back, and the page of the j-th new block
    auto page_back = [&](int k) {
        const int b = last_at_most(s_back, B, k);
        return a.table[(int64_t)b * a.width + (k - s_back[b])];
    };
    auto page_new = [&](int j) {
        const int i = n1 - 1 - j;
        return i < nf ? a.free_pages[i] : page_back(i - nf);
    };
    for (int b = gt; b < B; b += step) {
        const bool ended = s_back[b + 1] > s_back[b];   // (an ended request without pages held nothing)
        a.lens_out[b] = ended ? 0 : s_len[b] + (s_cu[b + 1] - s_cu[b]);
    }
    for (int b = gt; b <= B; b += step) a.cu[b] = s_cu[b];
    // where there are many slots, a thread's four follow each other: one search,
    // and mostly one page
    const int per = a.tokens <= step ? 1 : 4;
    for (uint32_t i0 = per * gt; i0 < n_slots; i0 += per * step) {
        int b = i0 < (uint32_t)added ? last_at_most(s_cu, B, (int)i0) : B, of = -1, base = -1;
#pragma unroll 1
        for (int e = 0; e < per; ++e) {
            if (i0 + e >= n_slots) break;
            const int i = (int)(i0 + e);
            int slot = -1;
            if (i < added) {
                while (i >= s_cu[b + 1]) {
                    ++b;
                    of = -1;
                }
                const int pos = s_len[b] + (i - s_cu[b]), block = pos / kPage;
                if (block != of) {
                    of = block;
                    const int had = (s_len[b] + kPage - 1) / kPage;
                    const int page = block < had ? a.table[(int64_t)b * a.width + block] : page_new(s_need[b] + block - had);
                    base = page >= 0 && page < a.pages ? page * kPage : -1;
                }
                slot = base < 0 ? -1 : base + pos % kPage;
            }
            a.slots[i] = slot;
        }
    }
    for (int j = gt; j < fresh; j += step) {
        const int b = last_at_most(s_need, B, j);
        const int had = (s_len[b] + kPage - 1) / kPage;
        a.table[(int64_t)b * a.width + had + (j - s_need[b])] = page_new(j);
    }
    for (int k = gt; k < back; k += step) a.free_pages[nf + k] = page_back(k);
}

}  // namespace

cudaError_t launch_page_plan(const iskv_page_plan_args& a, cudaStream_t s) {
    const size_t smem = ((size_t)4 * a.batch + 3) * sizeof(int);
    static SmemOnce once;
    const cudaError_t e = once.set(page_plan_kernel, ((size_t)4 * kMaxBatch + 3) * sizeof(int));
    if (e != cudaSuccess) return e;
    // four slots per thread, up to what a portable cluster holds
    int ctas = 1;
    while (ctas < 8 && (int64_t)ctas * 4 * kThreads < a.tokens) ctas *= 2;
    return launch_early(page_plan_kernel, dim3(ctas), kThreads, smem, s, ctas, a);
}

}  // namespace q8
}  // namespace iskv
