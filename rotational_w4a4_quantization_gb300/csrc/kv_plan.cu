// kv_plan.cu -- block tables and slots of the paged cache from the requests' lengths (sm_103a).
//
// Request b has c_b tokens in the cache and gets n_b more; a page holds P tokens:
//   kept_b = ceil(c_b / P), need_b = ceil((c_b + n_b) / P)   (as far as its table row reaches)
//   pages  free[head + sum_{a<b} (need_a - kept_a) + i] become entries kept_b + i of its row;
//   token j of its n_b is at place c_b + j, in row sum_{a<b} n_a + j of the step.
//
// All of it follows from two running sums over the requests.  One launch, whose blocks wait for
// nobody: each scans the requests by itself (1024 of them are 8 KB from L2 and one block
// reduction), then takes its share of the tokens and of the table's rows.  A token's request
// is found by bisection over the block's per-thread sums and a walk of at most `per` requests.
//
// Bound by latency: the launch, lengths from L2, a scan, the page's number, a store.  In a graph on
// the same inputs (after a flush of L2): 64 requests of one token 4.0 us (5.6); 509 prompts of up to
// 768 tokens, 214,213 rows, 6.1 us (6.9).  Each block goes over all requests, so it is not for very many:
// 512 of one token 4.2 us, 4096 9.4, 16384 64, 65536 500.
#include "rq.h"
#include "rq_internal.h"

namespace rq {
namespace {

constexpr int kPThreads = 512;

struct PlanParams {
    const int32_t *contexts, *news, *base, *free_pages, *head;
    int32_t *table, *offsets, *head_out;
    int64_t *slots, *positions;
    int64_t width, free_count, total;
    int seqs, log_page;
};

struct PlanSeq {
    int64_t ctx, n;
    int64_t kept, need;         // pages before and after the step, within the table's row
};

__device__ __forceinline__ PlanSeq plan_seq(const PlanParams &p, int b) {
    PlanSeq s;
    s.ctx = max(0, p.contexts[b]);
    s.n = max(0, p.news[b]);
    const int64_t up = (int64_t(1) << p.log_page) - 1;
    s.kept = min((s.ctx + up) >> p.log_page, p.width);
    s.need = min((s.ctx + s.n + up) >> p.log_page, p.width);
    return s;
}

// Page number `i` steps into the free list, -1 where it has none.
__device__ __forceinline__ int32_t plan_page(const PlanParams &p, int64_t i) {
    return i >= 0 && i < p.free_count ? p.free_pages[i] : -1;
}

__global__ void __launch_bounds__(kPThreads) kv_plan_kernel(const __grid_constant__ PlanParams p) {
    __shared__ int64_t tokens[kPThreads + 1], pages[kPThreads + 1];    // before each thread's requests
    __shared__ int64_t warp_sum[2][kPThreads / 32];
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int per = (p.seqs + kPThreads - 1) / kPThreads;
    const int first = min(p.seqs, t * per), last = min(p.seqs, (t + 1) * per);
    const int64_t head = p.head ? (int64_t)*p.head : 0;

    int64_t n = 0, need = 0;
    for (int b = first; b < last; ++b) {
        const PlanSeq s = plan_seq(p, b);
        n += s.n;
        need += s.need - s.kept;
    }
    int64_t incl_n = n, incl_need = need;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, incl_n, o), y = __shfl_up_sync(0xffffffffu, incl_need, o);
        if (lane >= o) {
            incl_n += x;
            incl_need += y;
        }
    }
    if (lane == 31) {
        warp_sum[0][warp] = incl_n;
        warp_sum[1][warp] = incl_need;
    }
    __syncthreads();
    for (int w = 0; w < warp; ++w) {
        incl_n += warp_sum[0][w];
        incl_need += warp_sum[1][w];
    }
    tokens[t] = incl_n - n;
    pages[t] = incl_need - need;
    if (t == kPThreads - 1) {
        tokens[kPThreads] = incl_n;
        pages[kPThreads] = incl_need;
    }
    __syncthreads();

    if (blockIdx.x == 0) {
        int64_t at = tokens[t];
        for (int b = first; b < last; ++b) {
            p.offsets[b] = (int32_t)min(at, (int64_t)0x7fffffff);
            at += max(0, p.news[b]);
        }
        if (t == 0) {
            p.offsets[p.seqs] = (int32_t)min(tokens[kPThreads], (int64_t)0x7fffffff);
            *p.head_out = (int32_t)min(head + pages[kPThreads], (int64_t)0x7fffffff);
        }
    }

    // rows of the table, a warp each: new pages behind the kept ones, -1 behind those
    constexpr int kWarps = kPThreads / 32;
    for (int64_t b = (int64_t)blockIdx.x * kWarps + warp; b < p.seqs; b += (int64_t)gridDim.x * kWarps) {
        int64_t at = head + pages[b / per];
        for (int a = (int)(b / per) * per; a < b; ++a) {
            const PlanSeq s = plan_seq(p, a);
            at += s.need - s.kept;
        }
        const PlanSeq s = plan_seq(p, (int)b);
        for (int64_t j = s.kept + lane; j < p.width; j += 32)
            p.table[b * p.width + j] = j < s.need ? plan_page(p, at + j - s.kept) : -1;
    }

    for (int64_t row = (int64_t)blockIdx.x * kPThreads + t; row < p.total; row += (int64_t)gridDim.x * kPThreads) {
        int64_t slot = -1, position = 0;
        if (row < tokens[kPThreads]) {
            int lo = 0, hi = kPThreads;              // the last stretch that begins at or before row
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (tokens[mid] <= row) lo = mid;
                else hi = mid;
            }
            int64_t at = tokens[lo], page = head + pages[lo];
            int b = lo * per;
            PlanSeq s = plan_seq(p, b);
            while (row >= at + s.n) {
                at += s.n;
                page += s.need - s.kept;
                s = plan_seq(p, ++b);
            }
            const int64_t place = s.ctx + row - at, j = place >> p.log_page;
            // kept entries are nobody's to write
            const int32_t number = j >= p.width ? -1 : j < s.kept ? p.table[b * p.width + j] : plan_page(p, page + j - s.kept);
            if (number >= 0) slot = ((int64_t)number << p.log_page) + (place & ((int64_t(1) << p.log_page) - 1));
            position = place + (p.base ? p.base[b] : 0);
        }
        p.slots[row] = slot;
        p.positions[row] = position;
    }
}

}  // namespace

cudaError_t launch_kv_plan(const PlanCall &c, cudaStream_t stream) {
    PlanParams p{};
    p.contexts = c.contexts;
    p.news = c.news;
    p.base = c.base;
    p.free_pages = c.free_pages;
    p.head = c.head;
    p.table = c.table;
    p.offsets = c.offsets;
    p.head_out = c.head_out;
    p.slots = c.slots;
    p.positions = c.positions;
    p.width = c.width;
    p.free_count = c.free_count;
    p.total = c.total;
    p.seqs = (int)c.seqs;
    while ((int64_t(1) << p.log_page) < c.page_size) ++p.log_page;
    const int64_t rows = (c.total + kPThreads - 1) / kPThreads, tables = (c.seqs + kPThreads / 32 - 1) / (kPThreads / 32);
    int64_t blocks = rows > tables ? rows : tables;
    const int64_t most = 2 * (int64_t)device_sm_count();
    if (blocks > most) blocks = most;
    if (blocks < 1) blocks = 1;
    kv_plan_kernel<<<(unsigned)blocks, kPThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace rq
