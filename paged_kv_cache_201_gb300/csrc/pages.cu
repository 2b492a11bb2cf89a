// Pages shared, given back and moved together: the bookkeeping of a paged cache on the device.
//
// Each call is one launch of one cluster of CTAs, which takes its steps between cluster barriers; what a step
// needs from another CTA's shared memory (counts of a scan) it reads there, so no call needs a workspace or a second
// launch.  What the requests come to (prefix sums of at most PA_STEP_MAX_BATCH small numbers) every CTA works out for
// itself; the listed pages, one after the other over the rows, are shared out in runs, one a warp.
//
// Sums of page counts do not depend on the order of their atomics.  Where an order shows (the stack of free pages), it is
// fixed: a page that several rows give back belongs to the smallest place that lists it, found with an atomic
// minimum in page_shares itself.  A page's count runs from its owners - 1 down; below 0 the page is free, and
// the places' numbers, INT_MIN + e with e < 2^30, lie below every count that is reached.
//
// What bounds them is the chain of dependent trips to memory and of barriers, not bytes.  A prompt of 63 pages forked to
// 4 rows, copied and freed takes 10.6 us, 192 rows of some 190 pages 25; 8 rows of some 90 freed 7.5, 1024 rows of some 180 pages
// 35 (the random reads of page_shares from 16 multiprocessors); a compaction's plan 12 for 2048 pages, 20 for 32768.  The 1024
// rows took 122 with places searched for again in every pass and atomics on every page, 45 with a round's places in registers,
// 16 CTAs instead of 8 and none for pages that nobody shares, 35 with fewer barriers and no wait for the last stores.  The 8 rows
// took 4 us more while every warp went through all sixteen turns of a round.
#include <limits.h>

#include "kv4.cuh"
#include "sparse_common.cuh"

namespace pa {

namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kMaxCtas = 8, kWideCtas = 16;
constexpr int kUsed = 1, kFree = 2;  // marks of a page
constexpr int kPer = PA_STEP_MAX_BATCH / kThreads;  // requests of a thread at most

struct Pair {
    int a, b;
};

// Exclusive prefix sums over the block, one pair a thread; the totals in every thread.
__device__ __forceinline__ Pair block_scan(Pair v, Pair *warp_sums, Pair &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Pair inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int xa = __shfl_up_sync(0xffffffffu, inc.a, o), xb = __shfl_up_sync(0xffffffffu, inc.b, o);
        if (lane >= o) inc.a += xa, inc.b += xb;
    }
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    Pair w = warp_sums[lane], run = w;  // every warp sums the warps before it
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int xa = __shfl_up_sync(0xffffffffu, run.a, o), xb = __shfl_up_sync(0xffffffffu, run.b, o);
        if (lane >= o) run.a += xa, run.b += xb;
    }
    total.a = __shfl_sync(0xffffffffu, run.a, 31);
    total.b = __shfl_sync(0xffffffffu, run.b, 31);
    const int before_a = __shfl_sync(0xffffffffu, run.a - w.a, warp);
    const int before_b = __shfl_sync(0xffffffffu, run.b - w.b, warp);
    __syncthreads();  // warp_sums may be written again
    return {before_a + inc.a - v.a, before_b + inc.b - v.b};
}

// All threads of the cluster; what they wrote before, everybody sees after.  One CTA needs no more than its own barrier.
__device__ __forceinline__ void sync_all(int ctas) {
    if (ctas == 1)
        __syncthreads();
    else
        cluster_barrier();
}

// The sums over the cluster's warps before this one, from a pair a warp, and over all of them.  warp_sums: [kWarps]; *s_cta
// is the CTA's sum, which its peers read until the next barrier of all.
__device__ __forceinline__ Pair cluster_scan(Pair mine, Pair *warp_sums, Pair *s_cta, int ctas, int rank, Pair &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) warp_sums[warp] = mine;
    __syncthreads();
    const Pair w = warp_sums[lane];  // every warp sums the warps before it
    const bool first = lane < warp;
    Pair before{__reduce_add_sync(0xffffffffu, first ? w.a : 0), __reduce_add_sync(0xffffffffu, first ? w.b : 0)};
    total = {__reduce_add_sync(0xffffffffu, w.a), __reduce_add_sync(0xffffffffu, w.b)};
    if (ctas == 1) return before;
    if (threadIdx.x == 0) *s_cta = total;
    cluster_barrier();
    Pair v{0, 0};  // CTA `lane`'s
    if (lane < ctas)
        asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];"
                     : "=r"(v.a), "=r"(v.b)
                     : "r"(peer_addr(smem_u32(s_cta), lane))
                     : "memory");
    total = {__reduce_add_sync(0xffffffffu, v.a), __reduce_add_sync(0xffffffffu, v.b)};
    if (lane >= rank) v = {0, 0};
    before.a += __reduce_add_sync(0xffffffffu, v.a);
    before.b += __reduce_add_sync(0xffffffffu, v.b);
    return before;
}

// Pages of a row of this length; lengths past the row's width are cut.
__device__ __forceinline__ int pages_of(const PagesParams &p, int len, bool &clipped) {
    const long long most = (long long)p.W << p.ps_shift;
    if (len > most) {
        clipped = true;
        len = (int)most;
    }
    return (max(len, 0) + (1 << p.ps_shift) - 1) >> p.ps_shift;
}

// Places e = 0 .. total - 1 of the lists, place e the (e - s_start[i])-th of list i with s_start[i] <= e < s_start[i + 1].
// The list of place e, none before lo: mostly lo or the next.
__device__ __forceinline__ int list_of(const int *s_start, int n, int e, int lo) {
    if (lo + 1 >= n || s_start[lo + 1] > e) return lo;
    if (++lo + 1 >= n || s_start[lo + 1] > e) return lo;
    int hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_start[mid] <= e)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// A warp's run of the places, PT at a time to a lane: load(k, i, j) for all of them, then use(k, live) for all.
template <int PT, typename L, typename U>
__device__ __forceinline__ void for_places(const int *s_start, int n, int total, int warp_all, int warps_all, L load, U use) {
    const int run = ((total + warps_all - 1) / warps_all + 31) & ~31;
    const int e0 = (int)min((long long)warp_all * run, (long long)total), e1 = (int)min((long long)e0 + run, (long long)total);
    int lo = 0;
    for (int first = e0; first < e1; first += 32 * PT) {
#pragma unroll
        for (int k = 0; k < PT; ++k) {
            if (first + 32 * k >= e1) break;
            const int e = first + 32 * k + (threadIdx.x & 31);
            if (e < e1) {
                lo = list_of(s_start, n, e, lo);
                load(k, lo, e - s_start[lo]);
            }
        }
#pragma unroll
        for (int k = 0; k < PT; ++k) {
            if (first + 32 * k >= e1) break;
            use(k, first + 32 * k + (int)(threadIdx.x & 31) < e1);
        }
    }
}

}  // namespace

// PER: requests of a thread at most.
template <int PER>
__global__ void __launch_bounds__(kThreads, 1) paged_attn_fork_kernel(const PagesParams p) {
    wait_for_stream();
    extern __shared__ int sm[];
    int *s_start = sm, *s_row = sm + p.n + 1;  // [n + 1] first places, [n] parent's row
    int *s_named = s_row + p.n;                // [B] the first request that names a child
    int *s_child = s_named;                    // [n] the child's row, once that is known
    __shared__ Pair warp_sums[kWarps];
    const int tid = threadIdx.x, ctas = gridDim.x, rank = blockIdx.x;
    const int per = (p.n + kThreads - 1) / kThreads;
    const int i0 = min(tid * per, p.n), mine = min(per, p.n - i0);
    const int ps_mask = (1 << p.ps_shift) - 1;
    bool refused = false, clipped = false, bad_page = false;
    const int count_in = *p.free_count;
    const int F = min(max(count_in, 0), p.free_cap);
    refused |= F != count_in;

    for (int b = tid; b < p.B; b += kThreads) s_named[b] = INT_MAX;
    __syncthreads();
    int par[PER], chi[PER], len[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        par[k] = k < mine ? __ldg(p.rows + i0 + k) : -1;
        chi[k] = k < mine ? __ldg(p.children + i0 + k) : -1;
        len[k] = k < mine && p.prefix_lens ? __ldg(p.prefix_lens + i0 + k) : INT_MAX;
        if (par[k] != -1 && chi[k] >= 0 && chi[k] < p.B) atomicMin(s_named + chi[k], i0 + k);
    }
    __syncthreads();
    // usable requests: len the shared length; others: -1
    Pair sum{0, 0}, total;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const bool asked = par[k] != -1;
        bool ok = asked && par[k] >= 0 && par[k] < p.B && chi[k] >= 0 && chi[k] < p.B && par[k] != chi[k] && len[k] >= 0;
        ok = ok && s_named[chi[k]] == i0 + k && __ldcg(p.seq_lens + chi[k]) == 0;
        if (ok) {
            const int have = max(__ldcg(p.seq_lens + par[k]), 0);
            const long long most = (long long)p.W << p.ps_shift;
            clipped |= have > most;
            len[k] = (int)min((long long)min(len[k], have), most);
        } else {
            refused |= asked;
            len[k] = -1;
        }
        sum.a += ok && (len[k] & ps_mask) != 0;
    }
    Pair run = block_scan(sum, warp_sums, total);  // pages that the usable requests before need
    sum = {0, 0};
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        if (len[k] < 0) continue;
        const int need = (len[k] & ps_mask) != 0;
        run.a += need;
        if (need && run.a > F) {
            refused = true;
            len[k] = -1;
            continue;
        }
        sum.a += need;
        sum.b += len[k] >> p.ps_shift;
    }
    run = block_scan(sum, warp_sums, total);  // of the served ones: pages taken, full pages
    sync_all(ctas);                        // every CTA has read the lengths and the count
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        if (k >= mine) continue;
        const int i = i0 + k;
        const bool served = len[k] >= 0, need = served && (len[k] & ps_mask) != 0;
        s_start[i] = run.b;
        s_row[i] = par[k];
        s_child[i] = chi[k];
        if (rank == 0) {
            int from = -1, to = -1;
            if (need) {
                const int j = len[k] >> p.ps_shift;
                from = __ldg(p.block_table + (long long)par[k] * p.W + j);
                to = __ldg(p.free_pages + (F - 1 - run.a));
                p.block_table[(long long)chi[k] * p.W + j] = to;
                if (from < 0 || from >= p.num_pages || to < 0 || to >= p.num_pages) {
                    bad_page = true;
                    from = to = -1;
                }
            }
            p.copies[2 * i] = from;
            p.copies[2 * i + 1] = to;
        }
        if (served) {
            run.a += need;
            run.b += len[k] >> p.ps_shift;
        }
    }
    if (tid == 0) s_start[p.n] = total.b;
    if (rank == 0) {
        if (tid == 0) *p.free_left = F - total.a;
        if (p.lens_out != p.seq_lens)
            for (int b = tid; b < p.B; b += kThreads) p.lens_out[b] = p.seq_lens[b];
    }
    __syncthreads();
    if (rank == 0) {
#pragma unroll
        for (int k = 0; k < PER; ++k)
            if (k < mine && len[k] >= 0) p.lens_out[chi[k]] = len[k];
    }
    // the full pages' entries; no row that is read here is written (a child's length was 0)
    constexpr int PT = 8;
    int id[PT];
    int32_t *to[PT];
    for_places<PT>(
        s_start, p.n, total.b, rank * kWarps + (tid >> 5), ctas * kWarps,
        [&](int k, int i, int j) {
            id[k] = __ldg(p.block_table + (long long)s_row[i] * p.W + j);
            to[k] = p.block_table + (long long)s_child[i] * p.W + j;
        },
        [&](int k, bool live) {
            if (!live) return;
            *to[k] = id[k];
            if (id[k] >= 0 && id[k] < p.num_pages)
                atomicAdd(p.shares + id[k], 1);
            else
                bad_page = true;
        });
    if (refused) atomicOr(p.err, (unsigned int)PA_ERRBIT_REFUSED);
    if (clipped) atomicOr(p.err, (unsigned int)PA_ERRBIT_SEQ_CLIPPED);
    if (bad_page) atomicOr(p.err, (unsigned int)PA_ERRBIT_PAGE_RANGE);
}

template <int PER>
__global__ void __launch_bounds__(kThreads, 1) paged_attn_free_kernel(const PagesParams p) {
    wait_for_stream();
    extern __shared__ int sm[];
    int *s_start = sm, *s_row = sm + p.n + 1;  // [n + 1] first places, [n] rows
    int *s_named = s_row + p.n;                // [B] the first request that names a row
    __shared__ Pair warp_sums[kWarps];
    __shared__ __align__(8) Pair s_cta;
    __shared__ int s_any;  // rounds (from 1) whose pages somebody shares
    const int tid = threadIdx.x, lane = tid & 31, ctas = gridDim.x, rank = blockIdx.x;
    const int warp_all = rank * kWarps + (tid >> 5), warps_all = ctas * kWarps;
    // No CTA stores into a peer's s_any before that peer runs and has cleared it: the wait stands before the rounds.
    if (tid == 0) s_any = 0;
    if (ctas > 1) asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    const int per = (p.n + kThreads - 1) / kThreads;
    const int i0 = min(tid * per, p.n), mine = min(per, p.n - i0);
    bool refused = false, clipped = false, bad_page = false;
    const int count_in = *p.free_count;
    const int F = min(max(count_in, 0), p.free_cap);
    refused |= F != count_in;

    for (int b = tid; b < p.B; b += kThreads) s_named[b] = INT_MAX;
    __syncthreads();
    int row[PER], pages[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        row[k] = k < mine ? __ldg(p.rows + i0 + k) : -1;
        if (row[k] != -1 && (row[k] < 0 || row[k] >= p.B)) {
            refused = true;
            row[k] = -1;
        }
        if (row[k] >= 0) atomicMin(s_named + row[k], i0 + k);
    }
    __syncthreads();
    Pair sum{0, 0}, total;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        if (row[k] >= 0 && s_named[row[k]] != i0 + k) row[k] = -1;  // named before
        pages[k] = row[k] >= 0 ? pages_of(p, __ldcg(p.seq_lens + row[k]), clipped) : 0;
        sum.a += pages[k];
    }
    Pair run = block_scan(sum, warp_sums, total);
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        if (k >= mine) continue;
        s_start[i0 + k] = run.a;
        s_row[i0 + k] = row[k];
        run.a += pages[k];
    }
    if (tid == 0) s_start[p.n] = total.a;
    __syncthreads();
    if (ctas > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    if (rank == 0 && p.lens_out != p.seq_lens)  // the rows' zeros follow behind a barrier
        for (int b = tid; b < p.B; b += kThreads) p.lens_out[b] = p.seq_lens[b];
    // Rounds of at most PT places a lane, the last places first, as the rows end one after the other: a page is pushed in
    // the round that takes its last owner.  A page that nobody shares needs no count.
    constexpr int PT = 16;
    const int round = warps_all * 32 * PT;
    long long top = F;  // the stack's
    for (int r = (total.a - 1) / round; r >= 0 && total.a > 0; --r) {
        const int first = r * round, size = min(round, total.a - first);
        const int run = ((size + warps_all - 1) / warps_all + 31) & ~31;  // of a warp, at most 32 PT
        const int e0 = first + min(warp_all * run, size) + lane, e1 = first + min(warp_all * run + run, size);
        const int turns = run / 32;  // of a lane: all loops end there (few places would pay for sixteen otherwise)
        int id[PT], before[PT];
        int lo = 0;
#pragma unroll
        for (int k = 0; k < PT; ++k) {
            if (k >= turns) break;
            const int e = e0 + 32 * k;
            id[k] = -1;
            if (e >= e1) continue;
            lo = list_of(s_start, p.n, e, lo);
            id[k] = __ldg(p.block_table + (long long)s_row[lo] * p.W + e - s_start[lo]);
        }
#pragma unroll
        for (int k = 0; k < PT; ++k) {  // only now: the loads above are on their way together
            if (k >= turns) break;
            if (id[k] < 0 || id[k] >= p.num_pages) {
                bad_page |= e0 + 32 * k < e1;
                id[k] = -1;
            }
        }
        unsigned push = 0, shared = 0;  // bits of this lane's places
#pragma unroll
        for (int k = 0; k < PT; ++k) {
            if (k >= turns) break;
            before[k] = id[k] >= 0 ? __ldcg(p.shares + id[k]) : 0;
        }
#pragma unroll
        for (int k = 0; k < PT; ++k) {
            if (k >= turns) break;
            if (id[k] >= 0) (before[k] == 0 ? push : shared) |= 1u << k;
        }
        const int number = r + 1;
        if (__any_sync(0xffffffffu, shared) && lane < ctas)
            asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(peer_addr(smem_u32(&s_any), lane)), "r"(number) : "memory");
        sync_all(ctas);  // every count is read as it was, and the lengths
        if (*(volatile int *)&s_any == number) {
#pragma unroll
            for (int k = 0; k < PT; ++k) {
                if (k >= turns) break;
                if (shared >> k & 1) atomicSub(p.shares + id[k], 1);
            }
            sync_all(ctas);
            // the first place of every page that is free now
#pragma unroll
            for (int k = 0; k < PT; ++k) {
                if (k >= turns) break;
                if (shared >> k & 1) before[k] = __ldcg(p.shares + id[k]);
            }
#pragma unroll
            for (int k = 0; k < PT; ++k) {
                if (k >= turns) break;
                if ((shared >> k & 1) && before[k] >= 0) shared &= ~(1u << k);
                if (shared >> k & 1) atomicMin(p.shares + id[k], INT_MIN + e0 + 32 * k);
            }
            sync_all(ctas);
#pragma unroll
            for (int k = 0; k < PT; ++k) {
                if (k >= turns) break;
                if (shared >> k & 1) before[k] = __ldcg(p.shares + id[k]);
            }
        }
        Pair n_mine{0, 0}, pushed;
#pragma unroll
        for (int k = 0; k < PT; ++k) {
            if (k >= turns) break;
            if ((shared >> k & 1) && before[k] == INT_MIN + e0 + 32 * k) push |= 1u << k;
        }
        n_mine.a = __reduce_add_sync(0xffffffffu, __popc(push));
        int at = cluster_scan(n_mine, warp_sums, &s_cta, ctas, rank, pushed).a;
        top += pushed.a;
#pragma unroll
        for (int k = 0; k < PT; ++k) {
            if (k >= turns) break;
            const unsigned all = __ballot_sync(0xffffffffu, push >> k & 1);
            if (push >> k & 1) {
                const long long to = top - 1 - (at + __popc(all & ((1u << lane) - 1)));
                if (shared >> k & 1) p.shares[id[k]] = 0;
                if (to < p.free_cap)
                    p.free_pages[to] = id[k];
                else
                    refused = true;
            }
            at += __popc(all);
        }
        if (r > 0)
            sync_all(ctas);  // the counts of the next round are this one's
        else if (ctas > 1)  // s_cta has been read; what was written needs no wait (1024 rows freed 36.9 -> 35.0 us)
            asm volatile("barrier.cluster.arrive.relaxed;\n\tbarrier.cluster.wait;" ::: "memory");
    }
    if (total.a == 0) sync_all(ctas);  // every CTA has read the lengths and the count
    if (rank == 0) {
#pragma unroll
        for (int k = 0; k < PER; ++k)
            if (row[k] >= 0) p.lens_out[row[k]] = 0;
        if (tid == 0) *p.free_left = (int)min(top, (long long)p.free_cap);
    }
    if (refused) atomicOr(p.err, (unsigned int)PA_ERRBIT_REFUSED);
    if (clipped) atomicOr(p.err, (unsigned int)PA_ERRBIT_SEQ_CLIPPED);
    if (bad_page) atomicOr(p.err, (unsigned int)PA_ERRBIT_PAGE_RANGE);
}

// The used pages to the pool's start.  With U(x) the used pages at or above x and F(x) the free ones below, the first x
// with F(x) >= U(x) has F(x) = U(x) (one of the two moves by one from page to page): below it every free page takes one
// of the used pages above, and what lies at or above it and was used or free is free.  Marks stand in page_map until its
// values do.
template <int PER>
__global__ void __launch_bounds__(kThreads, 1) paged_attn_compact_kernel(const PagesParams p) {
    wait_for_stream();
    extern __shared__ int sm[];
    int *s_start = sm;  // [B + 1]
    __shared__ Pair warp_sums[kWarps];
    __shared__ __align__(8) Pair s_cta;
    __shared__ int s_border[2];
    const int tid = threadIdx.x, lane = tid & 31, ctas = gridDim.x, rank = blockIdx.x;
    const int warp_all = rank * kWarps + (tid >> 5), warps_all = ctas * kWarps;
    const long long all = (long long)ctas * kThreads, tid_all = (long long)rank * kThreads + tid;
    const int P = (int)p.num_pages;
    bool refused = false, clipped = false, bad_page = false;
    const int count_in = *p.free_count;
    const int F = min(max(count_in, 0), p.free_cap);
    refused |= F != count_in;
    auto in_pool = [&](int id) { return id >= 0 && id < P; };

    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, p.B), mine = min(per, p.B - b0);
    int pages[PER];
    Pair sum{0, 0}, total;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        pages[k] = k < mine ? pages_of(p, __ldg(p.seq_lens + b0 + k), clipped) : 0;
        sum.a += pages[k];
    }
    Pair run = block_scan(sum, warp_sums, total);
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        if (k >= mine) continue;
        s_start[b0 + k] = run.a;
        run.a += pages[k];
    }
    if (tid == 0) {
        s_start[p.B] = total.a;
        s_border[0] = s_border[1] = 0;
    }
    for (long long x = tid_all; x < P; x += all) __stcg(p.page_map + x, 0);
    sync_all(ctas);
    constexpr int PT = 4;
    for (long long x0 = tid_all; x0 < F; x0 += all * PT) {
        int id[PT];
#pragma unroll
        for (int k = 0; k < PT; ++k) id[k] = x0 + k * all < F ? __ldg(p.free_pages + x0 + k * all) : 0x7fffffff;
#pragma unroll
        for (int k = 0; k < PT; ++k) {
            if (x0 + k * all >= F) continue;
            if (in_pool(id[k]))
                refused |= (atomicOr(p.page_map + id[k], kFree) & kFree) != 0;
            else
                bad_page = true;
        }
    }
    int ids[PT];
    int32_t *entry[PT];
    for_places<PT>(
        s_start, p.B, total.a, warp_all, warps_all,
        [&](int k, int i, int j) { ids[k] = __ldcg(p.block_table + (long long)i * p.W + j); },
        [&](int k, bool live) {
            if (!live) return;
            if (in_pool(ids[k]))
                atomicOr(p.page_map + ids[k], kUsed);
            else
                bad_page = true;
        });
    sync_all(ctas);
    // every warp's run of pages: its used (a) and free (b) ones, and those of the runs before
    const int seg = (int)(((long long)P + warps_all - 1) / warps_all + 31) & ~31;
    const int x0 = (int)min((long long)warp_all * seg, (long long)P), x1 = (int)min((long long)x0 + seg, (long long)P);
    auto marks = [&](int x, unsigned &used, unsigned &idle) {
        const int m = x + lane < x1 ? __ldcg(p.page_map + x + lane) : 0;
        refused |= m == (kUsed | kFree);
        used = __ballot_sync(0xffffffffu, m & kUsed);
        idle = __ballot_sync(0xffffffffu, m == kFree);
    };
    Pair n_mine{0, 0};
#pragma unroll 4
    for (int x = x0; x < x1; x += 32) {
        unsigned used, idle;
        marks(x, used, idle);
        n_mine.a += __popc(used);
        n_mine.b += __popc(idle);
    }
    const Pair before = cluster_scan(n_mine, warp_sums, &s_cta, ctas, rank, total);
    // the border: in the run where F(x) reaches U(x), which one warp of the cluster finds out for all
    if (before.b < total.a - before.a && before.b + n_mine.b >= total.a - before.a - n_mine.a) {
        int u = total.a - before.a, f = before.b, border = x0;
        for (int x = x0; x < x1 && f < u; x += 32) {
            unsigned used, idle;
            marks(x, used, idle);
            const unsigned upto = 2u << lane;  // 0 for lane 31: all
            const bool there = f + __popc(idle & (upto - 1)) >= u - __popc(used & (upto - 1));
            const unsigned first = __ballot_sync(0xffffffffu, there);
            if (first) {
                border = x + __ffs(first);
                f += __popc(idle & ((2u << (__ffs(first) - 1)) - 1));
                break;
            }
            f += __popc(idle);
            u -= __popc(used);
        }
        if (lane < ctas) {
            asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(peer_addr(smem_u32(s_border), lane)), "r"(border) : "memory");
            asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(peer_addr(smem_u32(s_border + 1), lane)), "r"(f) : "memory");
        }
    }
    sync_all(ctas);
    const int border = s_border[0], n_moves = s_border[1];
    // below the border U(0) - n_moves pages are used; at and above it as many are left free as there were
    int u = before.a, f = before.b;
#pragma unroll 4
    for (int x = x0; x < x1; x += 32) {
        unsigned used, idle;
        marks(x, used, idle);
        const unsigned below = (1u << lane) - 1;
        const int id = x + lane, ku = u + __popc(used & below), kf = f + __popc(idle & below);
        const bool is_used = used >> lane & 1, is_idle = idle >> lane & 1;
        if (id < border) {
            if (is_idle) p.moves[2 * kf + 1] = id;
        } else if (is_used || is_idle) {
            if (is_used) p.moves[2 * (ku - (total.a - n_moves))] = id;
            p.free_pages[total.b - 1 - (ku - (total.a - n_moves) + kf - n_moves)] = id;
        }
        // a page that moves: which move it is, until its new id is known
        if (id < x1) __stcg(p.page_map + id, is_used && id >= border ? ~(ku - (total.a - n_moves)) : id);
        u += __popc(used);
        f += __popc(idle);
    }
    if (rank == 0 && tid == 0) {
        *p.n_moves = n_moves;
        *p.free_left = total.b;
    }
    sync_all(ctas);
    for (long long k = tid_all; k < n_moves; k += all) {
        const int from = __ldcg(p.moves + 2 * k), to = __ldcg(p.moves + 2 * k + 1);
        __stcg(p.page_map + from, to);
        p.shares[to] = p.shares[from];
        p.shares[from] = 0;
    }
    // beside it the tables, which find either the new id or the move
    for_places<PT>(
        s_start, p.B, s_start[p.B], warp_all, warps_all,
        [&](int k, int i, int j) {
            ids[k] = __ldcg(p.block_table + (long long)i * p.W + j);
            entry[k] = p.block_table + (long long)i * p.W + j;
        },
        [&](int k, bool live) {
            if (!live || !in_pool(ids[k])) return;
            int now = __ldcg(p.page_map + ids[k]);
            if (now < 0) now = __ldcg(p.moves + 2ll * ~now + 1);
            if (now != ids[k]) *entry[k] = now;
        });
    if (refused) atomicOr(p.err, (unsigned int)PA_ERRBIT_REFUSED);
    if (clipped) atomicOr(p.err, (unsigned int)PA_ERRBIT_SEQ_CLIPPED);
    if (bad_page) atomicOr(p.err, (unsigned int)PA_ERRBIT_PAGE_RANGE);
}

namespace {

// A cluster for `work` pages at most, which the tables' width makes of rows: one CTA up to `alone` (its barrier is its own), from
// there four and more, `per` pages each.  Two are never better than one or four: 32 rows of up to 126 pages freed 10.4 us by
// one, 12.4 by two, 10.5 by four; 64 of up to 251 14.5 by one, 12.4 by sixteen; a compaction of 2048 pages with its copies 25.6
// by one, 27.6 by two, of 6000 39.0 by one, 37.7 by four.
struct ClusterLimit {
    SmemLimit smem, wide;
};
template <typename K>
cudaError_t launch_cluster(K kern, ClusterLimit &limit, size_t smem, size_t smem_max, long long work, long long alone, long long per,
                           int most, const PagesParams &p, cudaStream_t stream) {
    cudaError_t e = limit.smem.raise((const void *)kern, smem_max);
    int ctas = work <= alone ? 1 : 4;
    while (ctas > 1 && ctas < most && ctas * per < work) ctas *= 2;
    if (e == cudaSuccess && ctas > 8) e = limit.wide.allow_wide_clusters((const void *)kern);
    if (e != cudaSuccess) return e;
    return launch_behind(kern, dim3(ctas), kThreads, smem, ctas, stream, p);
}

size_t lists_smem(long long n, long long B) { return (size_t)(2 * n + 1 + (n > B ? n : B)) * sizeof(int); }

}  // namespace

template <int PER>
static cudaError_t launch_fork_n(const PagesParams &p, cudaStream_t stream) {
    static ClusterLimit limit;
    return launch_cluster(paged_attn_fork_kernel<PER>, limit, lists_smem(p.n, p.B),
                          lists_smem((long long)kThreads * PER, PA_STEP_MAX_BATCH), (long long)p.n * p.W, 2048, 1024, kWideCtas, p,
                          stream);
}
cudaError_t launch_fork(const PagesParams &p, cudaStream_t stream) {
    return p.n <= kThreads ? launch_fork_n<1>(p, stream) : launch_fork_n<kPer>(p, stream);
}

template <int PER>
static cudaError_t launch_free_n(const PagesParams &p, cudaStream_t stream) {
    static ClusterLimit limit;
    return launch_cluster(paged_attn_free_kernel<PER>, limit, lists_smem(p.n, p.B),
                          lists_smem((long long)kThreads * PER, PA_STEP_MAX_BATCH), (long long)p.n * p.W, 2048, 1024, kWideCtas, p,
                          stream);
}
cudaError_t launch_free(const PagesParams &p, cudaStream_t stream) {
    return p.n <= kThreads ? launch_free_n<1>(p, stream) : launch_free_n<kPer>(p, stream);
}

template <int PER>
static cudaError_t launch_compact_n(const PagesParams &p, cudaStream_t stream) {
    static ClusterLimit limit;
    const long long entries = (long long)p.B * p.W;
    return launch_cluster(paged_attn_compact_kernel<PER>, limit, (size_t)(p.B + 1) * sizeof(int),
                          ((size_t)kThreads * PER + 1) * sizeof(int), entries > p.num_pages ? entries : p.num_pages, 4096, 2048,
                          kMaxCtas, p, stream);
}
cudaError_t launch_compact(const PagesParams &p, cudaStream_t stream) {
    return p.B <= kThreads ? launch_compact_n<1>(p, stream) : launch_compact_n<kPer>(p, stream);
}

}  // namespace pa
