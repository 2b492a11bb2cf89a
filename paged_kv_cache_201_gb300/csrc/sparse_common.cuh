// Device helpers of the calls over selected pages: which sequence a query token belongs to and how far
// it sees.
#pragma once

#include "kernels.h"

namespace pa {

struct TokenRow {
    int b;      // sequence; -1: the row belongs to none (padding, or a malformed q_start)
    int reach;  // keys the token may see
};

// Query token t.  In a packed batch, the sequence is the largest b with q_start[b] <= t; a decode
// batch has one token a sequence, so b = t is tried before the binary search.  One thread's view:
// every caller of a block gets the same answer.
__device__ __forceinline__ TokenRow token_row(const FwdParams &p, long long t, long long n_tok, bool report) {
    int b, n, i;
    if (!p.q_start) {
        b = (int)(t / p.Sq);
        n = p.Sq;
        i = (int)(t - (long long)b * p.Sq);
    } else {
        int lo = 0, hi = p.B;  // q_start[lo] <= t < q_start[hi] for a well-formed batch
        if (t < p.B && __ldg(p.q_start + t) <= t) {
            lo = (int)t;
            if (__ldg(p.q_start + t + 1) > t) hi = lo + 1;
        }
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (__ldg(p.q_start + mid) <= t)
                lo = mid;
            else
                hi = mid;
        }
        const int q0 = __ldg(p.q_start + lo), q1 = __ldg(p.q_start + lo + 1);
        if (q0 < 0 || q1 < q0 || q1 > n_tok) {
            if (report) atomicOr(p.err, (unsigned int)PA_ERRBIT_QSTART);
            return {-1, 0};
        }
        if (t < q0 || t >= q1) return {-1, 0};
        b = lo;
        n = q1 - q0;
        i = (int)(t - q0);
    }
    int L = max(__ldg(p.seq_lens + b), 0);
    if (L > p.W * p.ps) {  // never read past the sequence's block-table row
        if (report) atomicOr(p.err, (unsigned int)PA_ERRBIT_SEQ_CLIPPED);
        L = p.W * p.ps;
    }
    return {b, row_key_limit(p, b, L, i, n)};
}

}  // namespace pa
