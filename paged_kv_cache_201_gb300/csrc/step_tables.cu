// Block tables, slots and query ranges of one serving step, from the requests' lengths.
//
// Request b needs need_b = ceil((c + n) / ps) - ceil(c / ps) pages.  Two exclusive prefix sums over the
// batch give everything: the demand of the usable requests before b (pages, tokens) decides whether b
// is served, and the pages and tokens of the served ones before it place its share of the free stack
// and its packed tokens.  Each new page holds at least one new token, in its row 0, so the thread of
// that token writes the page's block-table entry.
//
// One cluster of CTAs, each of which computes both sums over the whole batch for itself (a few integers
// a request) and then writes its share of the tokens: no workspace and no second launch.  A cluster
// barrier separates every CTA's reads of the lengths from the first CTA's writes, so that the outputs
// may be the inputs' own arrays.  The step is a chain of a few trips to memory; what is read and written
// (0.3 MB for 1024 requests and 65536 tokens) would take 0.04 us at the copy rate; measured, that step takes
// 8.0 us, and one of 16 requests with a token each 2.4.
#include "kernels.h"

namespace pa {

namespace {

struct Pair {
    long long a, b;  // pages, tokens
};

// Exclusive prefix sum of one pair per thread over the block; total in every thread.
template <int THREADS>
__device__ __forceinline__ Pair block_scan(Pair v, Pair *warp_sums, Pair &total) {
    constexpr int WARPS = THREADS / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Pair inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long xa = __shfl_up_sync(0xffffffffu, inc.a, o);
        const long long xb = __shfl_up_sync(0xffffffffu, inc.b, o);
        if (lane >= o) {
            inc.a += xa;
            inc.b += xb;
        }
    }
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    // every warp sums the warps before it, one to a lane
    Pair w = lane < WARPS ? warp_sums[lane] : Pair{0, 0}, run = w;
#pragma unroll
    for (int o = 1; o < WARPS; o <<= 1) {
        const long long xa = __shfl_up_sync(0xffffffffu, run.a, o);
        const long long xb = __shfl_up_sync(0xffffffffu, run.b, o);
        if (lane >= o) {
            run.a += xa;
            run.b += xb;
        }
    }
    total.a = __shfl_sync(0xffffffffu, run.a, WARPS - 1);
    total.b = __shfl_sync(0xffffffffu, run.b, WARPS - 1);
    const long long before_a = __shfl_sync(0xffffffffu, run.a - w.a, warp);
    const long long before_b = __shfl_sync(0xffffffffu, run.b - w.b, warp);
    return {before_a + inc.a - v.a, before_b + inc.b - v.b};
}

}  // namespace

// PER: requests of a thread at most; CLUSTER: more than one CTA.
template <int THREADS, int PER, bool CLUSTER>
__global__ void __launch_bounds__(THREADS, 1) paged_attn_step_tables_kernel(const StepTablesParams p) {
    extern __shared__ int32_t sm[];
    int32_t *s_cached = sm;           // [B]
    int32_t *s_first = sm + p.B;      // [B] pages taken by the served requests before b
    int32_t *s_start = sm + 2 * p.B;  // [B + 1]
    __shared__ Pair warp_sums[2][THREADS / 32];
    constexpr int NT = CLUSTER ? 4 : 1;
    const int ps = 1 << p.ps_shift;
    const int tid = threadIdx.x, rank = CLUSTER ? blockIdx.x : 0;
    const int per = (p.B + THREADS - 1) / THREADS;
    const int b0 = min(tid * per, p.B), mine = min(per, p.B - b0);
    bool refused = false, bad_page = false;
    const int count_in = *p.free_count;
    const int F = min(max(count_in, 0), p.free_cap);
    if (tid == 0 && F != count_in) refused = true;

    // demand of the usable requests; n = -1: not usable
    int c[PER] = {}, n[PER] = {};
    auto pages_of = [&](int i) {
        return (((long long)c[i] + n[i] + ps - 1) >> p.ps_shift) - (((long long)c[i] + ps - 1) >> p.ps_shift);
    };
    Pair sum{0, 0}, total;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        c[i] = i < mine ? __ldcg(p.cached_lens + b0 + i) : 0;
        n[i] = i < mine ? __ldcg(p.new_lens + b0 + i) : 0;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (c[i] < 0 || n[i] < 0 || (((long long)c[i] + n[i] + ps - 1) >> p.ps_shift) > p.W) {
            refused |= n[i] != 0 || c[i] < 0;
            n[i] = -1;
            continue;
        }
        sum.a += pages_of(i);
        sum.b += n[i];
    }
    Pair run = block_scan<THREADS>(sum, warp_sums[0], total);
    // the served requests; the others ask for nothing
    sum = {0, 0};
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (n[i] < 0) continue;
        const long long d = pages_of(i);
        run.a += d;
        run.b += n[i];
        if ((d != 0 && run.a > F) || run.b > p.T) {
            refused |= n[i] != 0;
            n[i] = -1;
            continue;
        }
        sum.a += d;
        sum.b += n[i];
    }
    run = block_scan<THREADS>(sum, warp_sums[1], total);
    if (CLUSTER)  // every CTA has read the lengths and the count
        asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (i >= mine) continue;
        const int b = b0 + i;
        s_cached[b] = c[i];
        s_first[b] = (int)run.a;
        s_start[b] = (int)run.b;
        if (rank == 0) {
            p.q_start[b] = (int)run.b;
            p.q_offset[b] = c[i];
            p.seq_lens[b] = c[i] + max(n[i], 0);
        }
        if (n[i] > 0) {
            run.a += pages_of(i);
            run.b += n[i];
        }
    }
    const int n_tok = (int)total.b;
    if (tid == 0) {
        s_start[p.B] = n_tok;
        if (rank == 0) {
            p.q_start[p.B] = n_tok;
            *p.free_left = F - (int)total.a;
        }
    }
    __syncthreads();

    // NT consecutive tokens a thread: one search, and their page ids in one trip
    const long long step = (long long)(CLUSTER ? gridDim.x : 1) * THREADS * NT;
    for (long long t0 = (long long)(rank * THREADS + tid) * NT; t0 < p.T; t0 += step) {
        int lo = 0, hi = p.B;  // s_start[lo] <= t0 < s_start[hi], if t0 has a request
        if (t0 < n_tok) {
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_start[mid] <= t0)
                    lo = mid;
                else
                    hi = mid;
            }
        }
        int id[NT], row[NT];
        int32_t *fresh[NT];  // the block-table entry that the token writes
#pragma unroll
        for (int k = 0; k < NT; ++k) {
            const int t = (int)t0 + k;
            row[k] = -1;
            fresh[k] = nullptr;
            if (t0 + k >= n_tok) continue;
            while (s_start[lo + 1] <= t) ++lo;
            const int cached = s_cached[lo];
            const int pos = cached + (t - s_start[lo]);
            const int page = pos >> p.ps_shift, have = (int)(((long long)cached + ps - 1) >> p.ps_shift);
            int32_t *entry = p.block_table + (long long)lo * p.W + page;
            row[k] = pos & (ps - 1);
            if (page >= have) {
                id[k] = __ldg(p.free_pages + (F - 1 - (s_first[lo] + page - have)));
                if (row[k] == 0) fresh[k] = entry;
            } else {
                id[k] = *entry;
            }
        }
#pragma unroll
        for (int k = 0; k < NT; ++k) {
            if (t0 + k >= p.T) continue;
            if (fresh[k]) *fresh[k] = id[k];
            const bool ok = row[k] >= 0 && id[k] >= 0 && id[k] < p.num_pages;
            bad_page |= row[k] >= 0 && !ok;
            p.slots[t0 + k] = ok ? (id[k] << p.ps_shift) + row[k] : -1;
        }
    }
    if (refused && rank == 0) atomicOr(p.err, (unsigned int)PA_ERRBIT_REFUSED);
    if (bad_page) atomicOr(p.err, (unsigned int)PA_ERRBIT_PAGE_RANGE);
}

template <int THREADS, int PER, bool CLUSTER>
static cudaError_t launch_step(const StepTablesParams &p, int ctas, cudaStream_t stream) {
    auto kern = paged_attn_step_tables_kernel<THREADS, PER, CLUSTER>;
    static SmemLimit limit;
    const cudaError_t e = limit.raise((const void *)kern, ((size_t)3 * THREADS * PER + 1) * sizeof(int32_t));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = ((size_t)3 * p.B + 1) * sizeof(int32_t);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = ctas;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = CLUSTER ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

cudaError_t launch_step_tables(const StepTablesParams &p, cudaStream_t stream) {
    // A CTA for up to 1024 tokens, a cluster of up to eight for more.
    int ctas = 1;
    while (ctas < 8 && ctas * 1024 < p.T) ctas *= 2;
    if (p.B <= 256 && ctas == 1) return launch_step<256, 1, false>(p, 1, stream);
    if (p.B <= 1024) return ctas == 1 ? launch_step<1024, 1, false>(p, 1, stream) : launch_step<1024, 1, true>(p, ctas, stream);
    return launch_step<1024, PA_STEP_MAX_BATCH / 1024, true>(p, ctas, stream);
}

}  // namespace pa
