// What the page-selection kernels share: reading queries, and taking the pages of largest score of a row of
// scores in shared memory.
#pragma once

#include <float.h>

#include "sparse_common.cuh"

namespace pa {

// Order-preserving map of a float to an unsigned number, and back (no NaN comes here).
__device__ __forceinline__ unsigned ordered(float x) {
    const unsigned u = __float_as_uint(x);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float value_of(unsigned k) { return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu)); }

// Which of a row's scores are taken: those above `cut`, and of those at it the first `ties` pages; or,
// if `whole`, all that are at least `cut`.
struct Threshold {
    float cut;
    bool whole;
    __device__ __forceinline__ bool above(float x) const { return whole ? x >= cut : x > cut; }
    __device__ __forceinline__ bool at(float x) const { return !whole && x == cut; }
};

// The want-th largest of a row's scores, by narrowing a bracket: `reach_lo` >= want scores reach lo,
// `reach_hi` reach hi, fewer than want exceed it, and both are scores of the row.  count(c): how many are
// >= c, in every thread.  Two of three steps interpolate between the counts, which takes some five steps
// where the scores are spread smoothly; the third halves the values, and after 24 steps the numbers between
// are halved (infinite scores, or a few very large ones).  It ends as soon as exactly `want` scores reach a
// candidate.
template <typename Count>
__device__ __forceinline__ Threshold find_threshold(float lo, float hi, int reach_lo, int reach_hi, int want,
                                                    Count count) {
    if (reach_hi >= want) return {hi, reach_hi == want};  // ties at the top, or exactly so many
    unsigned kl = ordered(lo), kh = ordered(hi);  // want or more reach kl, fewer reach kh
    float cl = (float)reach_lo, ch = (float)reach_hi;
#pragma unroll 1
    for (int step = 0; kh - kl > 1; ++step) {
        unsigned k = kl + (kh - kl) / 2;
        if (step < 24) {
            const float vl = value_of(kl), vh = value_of(kh);
            const float part = step % 3 == 2 ? 0.5f : __fdividef(cl - (float)want, cl - ch);
            const float mid = vl + part * (vh - vl);
            if (fabsf(mid) <= FLT_MAX) k = min(max(ordered(mid), kl + 1), kh - 1);
        }
        const float c = value_of(k);
        const int n = count(c);
        if (n == want) return {c, true};
        if (n > want) {
            kl = k;
            cl = (float)n;
        } else {
            kh = k;
            ch = (float)n;
        }
    }
    return {value_of(kl), false};
}

// Elements i .. i + 15 of q (16-byte aligned), whose type is a value here: only the quantisation reads it.
__device__ __forceinline__ void q_load16(const void *q, int dtype, long long i, float (&v)[16]) {
    if (dtype == PA_F32) {
        const float4 *src = reinterpret_cast<const float4 *>(static_cast<const float *>(q) + i);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4 x = __ldg(src + k);
            v[4 * k] = x.x, v[4 * k + 1] = x.y, v[4 * k + 2] = x.z, v[4 * k + 3] = x.w;
        }
        return;
    }
    const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const unsigned short *>(q) + i);
    const uint4 x = __ldg(src), y = __ldg(src + 1);
    const uint32_t u[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float2 f = dtype == PA_BF16 ? MmaOp<__nv_bfloat16>::unpack(u[k]) : MmaOp<__half>::unpack(u[k]);
        v[2 * k] = f.x, v[2 * k + 1] = f.y;
    }
}

// Score j of a row of n; past the row a NaN, which no comparison takes.
__device__ __forceinline__ float score_at(const float *row, int n, int j) {
    return j < n ? row[j] : __uint_as_float(0x7fffffffu);
}

__device__ __forceinline__ float warp_min(float x) { return value_of(__reduce_min_sync(0xffffffffu, ordered(x))); }
__device__ __forceinline__ float warp_max(float x) { return value_of(__reduce_max_sync(0xffffffffu, ordered(x))); }

// Writes the pages of 32 NK scores k (score i * 32 + lane of a run) that are taken: those above the
// threshold and, while there are `ties` of them left in the row, those at it.  gt / eq: scores above / at it
// before the run, moved on.
template <int NK>
__device__ __forceinline__ void write_pages(const float (&k)[NK], Threshold thr, int ties, int &gt, int &eq, int base,
                                            int32_t *out, int lane) {
    const unsigned below = (1u << lane) - 1;
    if (thr.whole) {
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            const bool up = k[i] >= thr.cut;
            const unsigned ups = __ballot_sync(0xffffffffu, up);
            if (up) out[gt + __popc(ups & below)] = base + i * 32 + lane;
            gt += __popc(ups);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < NK; ++i) {
        const bool up = k[i] > thr.cut, at = k[i] == thr.cut;
        const unsigned ups = __ballot_sync(0xffffffffu, up), ats = __ballot_sync(0xffffffffu, at);
        const int e = eq + __popc(ats & below);
        if (up || (at && e < ties)) out[gt + __popc(ups & below) + min(e, ties)] = base + i * 32 + lane;
        gt += __popc(ups);
        eq += __popc(ats);
    }
}

// A token's selection by one warp, its scores in registers (n <= 32 NK).
template <int NK>
__device__ __forceinline__ void warp_select(const float *row, int n, int want, int base, int32_t *out, int lane) {
    float k[NK], lo = INFINITY, hi = -INFINITY;
#pragma unroll
    for (int i = 0; i < NK; ++i) {
        k[i] = score_at(row, n, i * 32 + lane);
        lo = fminf(lo, k[i]);  // fminf and fmaxf return the number where one of the two is NaN
        hi = fmaxf(hi, k[i]);
    }
    lo = warp_min(lo);
    hi = warp_max(hi);
    auto count = [&](float c) {
        int s = 0;
#pragma unroll
        for (int i = 0; i < NK; ++i) s += k[i] >= c;
        return (int)__reduce_add_sync(0xffffffffu, s);
    };
    const Threshold thr = find_threshold(lo, hi, n, count(hi), want, count);
    int up = 0;
    if (!thr.whole) {
#pragma unroll
        for (int i = 0; i < NK; ++i) up += k[i] > thr.cut;
        up = __reduce_add_sync(0xffffffffu, up);
    }
    int gt = 0, eq = 0;
    write_pages<NK>(k, thr, want - up, gt, eq, base, out, lane);
}

// The same for a row of any length, its scores read from shared memory in every pass.
__device__ __forceinline__ void warp_select_long(const float *row, int n, int want, int base, int32_t *out, int lane) {
    float lo = INFINITY, hi = -INFINITY;
#pragma unroll 8
    for (int j = lane; j < n; j += 32) {
        lo = fminf(lo, row[j]);
        hi = fmaxf(hi, row[j]);
    }
    lo = warp_min(lo);
    hi = warp_max(hi);
    auto count = [&](float c) {
        int s = 0;
#pragma unroll 8
        for (int j = lane; j < n; j += 32) s += row[j] >= c;
        return (int)__reduce_add_sync(0xffffffffu, s);
    };
    const Threshold thr = find_threshold(lo, hi, n, count(hi), want, count);
    int up = 0;
    if (!thr.whole) {
#pragma unroll 8
        for (int j = lane; j < n; j += 32) up += row[j] > thr.cut;
        up = __reduce_add_sync(0xffffffffu, up);
    }
    int gt = 0, eq = 0;
    for (int j = 0; j < n; j += 128) {
        float k[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) k[i] = score_at(row, n, j + i * 32 + lane);
        write_pages<4>(k, thr, want - up, gt, eq, base + j, out, lane);
    }
}

}  // namespace pa
