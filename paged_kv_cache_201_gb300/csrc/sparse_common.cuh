// Device helpers of the calls over selected pages: which sequence a query token belongs to and how far
// it sees.
#pragma once

#include "kernels.h"

namespace pa {

// x[i] = rint((x[i] / a) * 127) for |x[i]| <= a, 0 < a < inf, in float32 steps rounded to nearest even;
// inv = 127 / a.  x inv and the two-step value are each within 127 * 2^-23 < 2e-5 of the exact quotient,
// so they round to the same integer unless x inv lies within 1e-3 of a border: only then (one value in
// 500; and where inv overflows) are the divisions carried out.
template <int N>
__device__ __forceinline__ void quantise8(float (&x)[N], float a, float inv) {
    float r[N];
    bool clear = true;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float y = x[i] * inv;
        r[i] = rintf(y);
        clear = clear && fabsf(y - r[i]) <= 0.499f;
    }
    if (!clear) {
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] = rintf(__fmul_rn(__fdiv_rn(x[i], a), 127.f));
    }
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = r[i];
}

__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// The shared-memory address of CTA `rank` of the cluster that corresponds to the local one.
__device__ __forceinline__ uint32_t peer_addr(uint32_t local, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
    return r;
}

__device__ __forceinline__ float4 peer_load4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ float peer_load(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// Two launches of a call: the second, over the short sequences, may start beside the first's last CTAs (its
// inputs are older than both launches, its rows are others) and ends behind it, its last CTA waiting for the
// first launch; what follows on the stream follows both.
__device__ __forceinline__ void let_second_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
struct BehindFirst {
    const bool waits;
    __device__ __forceinline__ explicit BehindFirst(const SparseParams &sp)
        : waits(sp.group_min && blockIdx.x == gridDim.x - 1) {}
    __device__ __forceinline__ ~BehindFirst() {
        if (waits) asm volatile("griddepcontrol.wait;" ::: "memory");
    }
};
// The launch attributes of such kernels: a cluster of S CTAs, and for a second launch the early start.
inline int second_launch_attrs(cudaLaunchAttribute (&attr)[2], int S, bool second) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = S;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    return second ? 2 : 1;
}

// Each entry of a packed batch's q_start is looked at by one thread of the grid, whoever's rows it holds: a
// search from a row may pass a malformed sequence by.  The loads are on their way while the kernel finds its
// own sequence; report() follows.
struct RangeCheck {
    long long b, n_tok;
    int q0 = 0, q1 = 0;
    __device__ __forceinline__ RangeCheck(const SparseParams &sp)
        : b((long long)blockIdx.x * blockDim.x + threadIdx.x), n_tok(sp.n_tok) {
        load(sp.f);
    }
    __device__ __forceinline__ void load(const FwdParams &p) {
        if (!p.q_start || b >= p.B) return;
        q0 = __ldg(p.q_start + b);
        q1 = __ldg(p.q_start + b + 1);
    }
    __device__ __forceinline__ void report(const FwdParams &p) {
        while (p.q_start && b < p.B) {
            if (q0 < 0 || q1 < q0 || q1 > n_tok) atomicOr(p.err, (unsigned int)PA_ERRBIT_QSTART);
            b += (long long)gridDim.x * blockDim.x;
            load(p);
        }
    }
};

struct TokenRow {
    int b;      // sequence; -1: the row belongs to none (padding, or a malformed q_start)
    int reach;  // keys the token may see
};

// Query token t.  In a packed batch, the sequence is the largest b with q_start[b] <= t; a decode
// batch has one token a sequence, so b = t is tried before the binary search.  One thread's view:
// every caller of a block gets the same answer.
__device__ __forceinline__ TokenRow token_row(const FwdParams &p, long long t, long long n_tok, bool report) {
    int b, n, i, L;
    if (!p.q_start) {
        b = (int)(t / p.Sq);
        n = p.Sq;
        i = (int)(t - (long long)b * p.Sq);
        L = __ldg(p.seq_lens + b);
    } else {
        int lo = 0, hi = p.B;  // q_start[lo] <= t < q_start[hi] for a well-formed batch
        int q0 = 0, q1 = 0;
        L = 0;
        if (t < p.B) {  // one trip to memory for a decode batch
            q0 = __ldg(p.q_start + t);
            q1 = __ldg(p.q_start + t + 1);
            L = __ldg(p.seq_lens + t);
            if (q0 <= t) {
                lo = (int)t;
                if (q1 > t) hi = lo + 1;
            }
        }
        if (hi - lo > 1) {
            do {
                const int mid = (lo + hi) >> 1;
                if (__ldg(p.q_start + mid) <= t)
                    lo = mid;
                else
                    hi = mid;
            } while (hi - lo > 1);
            q0 = __ldg(p.q_start + lo);
            q1 = __ldg(p.q_start + lo + 1);
            L = __ldg(p.seq_lens + lo);
        } else if (lo != t) {
            q0 = __ldg(p.q_start);  // one sequence, and t past it
            q1 = __ldg(p.q_start + 1);
            L = __ldg(p.seq_lens);
        }
        if (q0 < 0 || q1 < q0 || q1 > n_tok || t < q0 || t >= q1) return {-1, 0};
        b = lo;
        n = q1 - q0;
        i = (int)(t - q0);
    }
    L = max(L, 0);
    if (L > p.W * p.ps) {  // never read past the sequence's block-table row
        if (report) atomicOr(p.err, (unsigned int)PA_ERRBIT_SEQ_CLIPPED);
        L = p.W * p.ps;
    }
    return {b, row_key_limit(p, b, L, i, n)};
}

// Where a call has launched the tcgen05 kernel for the long runs of a packed batch, the other kernel's units may
// be the tokens that a short sequence can have, `most` = group_min - 1 of each of the B sequences in blocks of
// TT (by_seq; fewer than the rows of q where the batch is mostly long runs).  The rows of block `unit`: first
// and count, 0 where the sequence is another's or shorter.
__device__ __forceinline__ int short_rows(const SparseParams &sp, long long unit, int TT, long long &first) {
    const FwdParams &p = sp.f;
    const int most = sp.group_min - 1, blocks = (most + TT - 1) / TT;
    const int b = (int)(unit / blocks), i = (int)(unit - (long long)b * blocks) * TT;
    if (b >= p.B) return 0;
    const int q0 = __ldg(p.q_start + b), n = __ldg(p.q_start + b + 1) - q0;
    first = (long long)q0 + i;
    if (q0 < 0 || n < 0 || (long long)q0 + n > sp.n_tok) return 0;
    return n > most ? 0 : max(0, min(TT, n - i));
}
inline long long short_blocks(const SparseParams &sp, int TT) {
    return (long long)sp.f.B * ((sp.group_min - 1 + TT - 1) / TT);
}

}  // namespace pa
