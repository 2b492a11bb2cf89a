// Block tables, slots and query ranges of one serving step, from the requests' lengths.
//
// Request b needs need_b = ceil((c + n) / ps) - ceil(c / ps) pages.  Two exclusive prefix sums over the
// batch give everything: the demand of the usable requests before b (pages, tokens) decides whether b
// is served, and the pages and tokens of the served ones before it place its share of the free stack
// and its packed tokens.  Each new page holds at least one new token, in its row 0, so the thread of
// that token writes the page's block-table entry.
#include "kernels.h"

namespace pa {

namespace {

constexpr int kStepThreads = 1024;

struct Pair {
    long long a, b;
};

// Exclusive prefix sum of one pair per thread over the block; total in every thread.
__device__ __forceinline__ Pair block_scan(Pair v, Pair *warp_sums, Pair &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Pair inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long xa = __shfl_up_sync(0xffffffffu, inc.a, o), xb = __shfl_up_sync(0xffffffffu, inc.b, o);
        if (lane >= o) {
            inc.a += xa;
            inc.b += xb;
        }
    }
    __syncthreads();  // warp_sums may still be read from an earlier scan
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    Pair before{0, 0};
    total = {0, 0};
    for (int w = 0; w < kStepThreads / 32; ++w) {
        const Pair s = warp_sums[w];
        if (w < warp) {
            before.a += s.a;
            before.b += s.b;
        }
        total.a += s.a;
        total.b += s.b;
    }
    return {before.a + inc.a - v.a, before.b + inc.b - v.b};
}

}  // namespace

__global__ void __launch_bounds__(kStepThreads, 1) paged_attn_step_tables_kernel(const StepTablesParams p) {
    extern __shared__ int32_t sm[];
    int32_t *s_cached = sm;           // [B]
    int32_t *s_first = sm + p.B;      // [B] pages taken by the served requests before b
    int32_t *s_start = sm + 2 * p.B;  // [B + 1]
    __shared__ Pair warp_sums[kStepThreads / 32];
    const int ps = 1 << p.ps_shift;
    const int tid = threadIdx.x;
    const int per = (p.B + kStepThreads - 1) / kStepThreads;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    bool refused = false, bad_page = false;
    const int count_in = *p.free_count;
    const int F = min(max(count_in, 0), p.free_cap);
    if (tid == 0 && F != count_in) refused = true;

    // demand of the usable requests
    auto demand = [&](int c, int n) -> Pair {
        if (c < 0 || n < 0) return {0, -1};
        const long long have = ((long long)c + ps - 1) >> p.ps_shift;
        const long long want = ((long long)c + n + ps - 1) >> p.ps_shift;
        if (want > p.W) return {0, -1};
        return {want - have, n};
    };
    Pair sum{0, 0}, total;
    for (int b = b0; b < b1; ++b) {
        const int c = p.cached_lens[b];
        s_cached[b] = c;
        const Pair d = demand(c, p.new_lens[b]);
        if (d.b >= 0) {
            sum.a += d.a;
            sum.b += d.b;
        }
    }
    Pair run = block_scan(sum, warp_sums, total);
    // the served requests (s_first[b] = -1 marks the others until the second scan)
    sum = {0, 0};
    for (int b = b0; b < b1; ++b) {
        const int n = p.new_lens[b];
        const Pair d = demand(s_cached[b], n);
        bool served = false;
        if (d.b >= 0) {
            run.a += d.a;
            run.b += d.b;
            served = (d.a == 0 || run.a <= F) && run.b <= p.T;
        }
        s_first[b] = served ? 0 : -1;
        if (served) {
            sum.a += d.a;
            sum.b += d.b;
        } else if (n != 0 || s_cached[b] < 0) {
            refused = true;
        }
    }
    run = block_scan(sum, warp_sums, total);
    for (int b = b0; b < b1; ++b) {
        const int c = s_cached[b];
        const bool served = s_first[b] == 0;
        const Pair d = demand(c, p.new_lens[b]);
        s_first[b] = (int)run.a;
        s_start[b] = (int)run.b;
        p.q_start[b] = (int)run.b;
        p.q_offset[b] = c;
        p.seq_lens[b] = served ? c + (int)d.b : c;
        if (served) {
            run.a += d.a;
            run.b += d.b;
        }
    }
    const int n_tok = (int)total.b;
    if (tid == 0) {
        s_start[p.B] = n_tok;
        p.q_start[p.B] = n_tok;
        *p.free_left = F - (int)total.a;
    }
    __syncthreads();

    for (int t = tid; t < p.T; t += kStepThreads) {
        if (t >= n_tok) {
            p.slots[t] = -1;
            continue;
        }
        int lo = 0, hi = p.B;  // s_start[lo] <= t < s_start[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_start[mid] <= t)
                lo = mid;
            else
                hi = mid;
        }
        const int c = s_cached[lo];
        const int pos = c + (t - s_start[lo]);
        const int page = pos >> p.ps_shift, have = (int)(((long long)c + ps - 1) >> p.ps_shift);
        int32_t *entry = p.block_table + (long long)lo * p.W + page;
        int id;
        if (page >= have) {
            id = p.free_pages[F - 1 - (s_first[lo] + page - have)];
            if ((pos & (ps - 1)) == 0) *entry = id;
        } else {
            id = *entry;
        }
        const bool ok = id >= 0 && id < p.num_pages;
        bad_page |= !ok;
        p.slots[t] = ok ? (id << p.ps_shift) + (pos & (ps - 1)) : -1;
    }
    if (refused) atomicOr(p.err, (unsigned int)PA_ERRBIT_REFUSED);
    if (bad_page) atomicOr(p.err, (unsigned int)PA_ERRBIT_PAGE_RANGE);
}

cudaError_t launch_step_tables(const StepTablesParams &p, cudaStream_t stream) {
    const size_t smem = ((size_t)3 * p.B + 1) * sizeof(int32_t);
    static SmemLimit limit;
    const cudaError_t e = limit.raise((const void *)paged_attn_step_tables_kernel,
                                      ((size_t)3 * PA_STEP_MAX_BATCH + 1) * sizeof(int32_t));
    if (e != cudaSuccess) return e;
    paged_attn_step_tables_kernel<<<1, kStepThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace pa
