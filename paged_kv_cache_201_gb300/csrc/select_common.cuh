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

// The want-th largest of a row's scores, by bisection from a bracket: at least `want` scores reach lo,
// fewer exceed hi, and both are scores of the row.  count(c): how many are >= c, in every thread.  The
// values are bisected first; what is not found in 14 steps is found by bisection of the numbers between
// (infinite scores).  It ends as soon as exactly `want` scores reach a candidate.
template <typename Count>
__device__ __forceinline__ Threshold find_threshold(float lo, float hi, int want, Count count) {
    unsigned kl = ordered(lo), kh = ordered(hi) + 1;  // want or more reach kl, fewer reach kh
    for (int step = 0; kh - kl > 1; ++step) {
        unsigned k = kl + (kh - kl) / 2;
        if (step < 14) {
            const float mid = 0.5f * value_of(kl) + 0.5f * value_of(kh - 1);
            if (fabsf(mid) <= FLT_MAX) k = min(max(ordered(mid), kl + 1), kh - 1);
        }
        const float c = value_of(k);
        const int n = count(c);
        if (n == want) return {c, true};
        if (n > want)
            kl = k;
        else
            kh = k;
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

// A row's scores sorted into equal parts of [lo, hi]; not decreasing in x, so the parts above the one that
// holds the threshold are taken whole and only that part is searched further.
struct Bins {
    float lo, per;
    int last;
    __device__ __forceinline__ Bins(float lo_, float hi, int n) : lo(lo_), per((float)n / (hi - lo_)), last(n - 1) {}
    __device__ __forceinline__ bool usable() const { return per > 0.f && per <= FLT_MAX; }  // a finite, wide range
    __device__ __forceinline__ int of(float x) const { return min((int)((x - lo) * per), last); }
};

// The part that holds the want-th largest score, counted from the top by one warp: lane l holds the counts
// of parts PL l .. PL l + PL - 1.  Returns its index, and how many scores lie in higher parts and in it.
template <int PL>
__device__ __forceinline__ int find_bin(const int (&c)[PL], int want, int lane, int &above, int &in) {
    int mine = 0;
#pragma unroll
    for (int i = 0; i < PL; ++i) mine += c[i];
    int from = mine;  // scores in this lane's parts and all higher lanes'
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_down_sync(0xffffffffu, from, o);
        if (lane + o < 32) from += x;
    }
    const int owner = 31 - __clz((int)__ballot_sync(0xffffffffu, from >= want));  // the highest such lane
    int up = from - mine, bin = 0, n = 0;
    bool found = false;
#pragma unroll
    for (int i = PL - 1; i >= 0; --i) {
        if (!found) {
            bin = i;
            n = c[i];
            if (up + n >= want)
                found = true;
            else
                up += n;
        }
    }
    above = __shfl_sync(0xffffffffu, up, owner);
    in = __shfl_sync(0xffffffffu, n, owner);
    return owner * PL + __shfl_sync(0xffffffffu, bin, owner);
}

constexpr int kBinsPerLane = 4, kBins = 32 * kBinsPerLane;  // of one warp; a CTA's warps have four times as many

// Writes the pages of 32 NK scores k (score i * 32 + lane of a run) that are taken: those above the
// threshold and, while there are `ties` of them left in the row, those at it.  gt / eq: scores above / at it
// before the run, moved on.
template <int NK>
__device__ __forceinline__ void write_pages(const float (&k)[NK], Threshold thr, int ties, int &gt, int &eq, int base,
                                            int32_t *out, int lane) {
    const unsigned below = (1u << lane) - 1;
#pragma unroll
    for (int i = 0; i < NK; ++i) {
        const bool up = thr.above(k[i]), at = thr.at(k[i]);
        const unsigned ups = __ballot_sync(0xffffffffu, up);
        const unsigned ats = thr.whole ? 0u : __ballot_sync(0xffffffffu, at);
        const int e = eq + __popc(ats & below);
        if (up || (at && e < ties)) out[gt + __popc(ups & below) + min(e, ties)] = base + i * 32 + lane;
        gt += __popc(ups);
        eq += __popc(ats);
    }
}

// A token's selection by one warp, its scores in registers (n <= 32 NK); hist: kBins counters of the warp.
template <int NK>
__device__ __forceinline__ void warp_select(const float *row, int n, int want, int base, int32_t *out, int *hist,
                                            int lane) {
    float k[NK], lo = INFINITY, hi = -INFINITY;
    *reinterpret_cast<int4 *>(hist + lane * 4) = make_int4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < NK; ++i) {
        k[i] = score_at(row, n, i * 32 + lane);
        lo = fminf(lo, k[i]);  // fminf and fmaxf return the number where one of the two is NaN
        hi = fmaxf(hi, k[i]);
    }
    lo = warp_min(lo);
    hi = warp_max(hi);
    const Bins bins(lo, hi, kBins);
    bool done = false;
    Threshold thr{lo, false};
    if (bins.usable()) {
#pragma unroll
        for (int i = 0; i < NK; ++i)
            if (i * 32 + lane < n) atomicAdd(hist + bins.of(k[i]), 1);
        __syncwarp();
        const int4 h = *reinterpret_cast<const int4 *>(hist + lane * 4);
        const int c[4] = {h.x, h.y, h.z, h.w};
        int above, in;
        const int bin = find_bin<4>(c, want, lane, above, in);
        lo = INFINITY;
        hi = -INFINITY;
#pragma unroll
        for (int i = 0; i < NK; ++i)
            if (i * 32 + lane < n && bins.of(k[i]) == bin) {
                lo = fminf(lo, k[i]);
                hi = fmaxf(hi, k[i]);
            }
        lo = warp_min(lo);
        hi = warp_max(hi);
        done = above + in == want;
        if (done) thr = {lo, true};
        __syncwarp();  // before the counters are cleared for another row
    }
    if (!done)
        thr = find_threshold(lo, hi, want, [&](float c) {
            int s = 0;
#pragma unroll
            for (int i = 0; i < NK; ++i) s += k[i] >= c;
            return (int)__reduce_add_sync(0xffffffffu, s);
        });
    int up = 0;
    if (!thr.whole) {
#pragma unroll
        for (int i = 0; i < NK; ++i) up += thr.above(k[i]);
        up = __reduce_add_sync(0xffffffffu, up);
    }
    int gt = 0, eq = 0;
    write_pages<NK>(k, thr, want - up, gt, eq, base, out, lane);
}

// The same for a row of any length, its scores read from shared memory in every pass.
__device__ __forceinline__ void warp_select_long(const float *row, int n, int want, int base, int32_t *out, int *hist,
                                                 int lane) {
    float lo = INFINITY, hi = -INFINITY;
    *reinterpret_cast<int4 *>(hist + lane * 4) = make_int4(0, 0, 0, 0);
#pragma unroll 8
    for (int j = lane; j < n; j += 32) {
        lo = fminf(lo, row[j]);
        hi = fmaxf(hi, row[j]);
    }
    lo = warp_min(lo);
    hi = warp_max(hi);
    const Bins bins(lo, hi, kBins);
    bool done = false;
    Threshold thr{lo, false};
    if (bins.usable()) {
#pragma unroll 8
        for (int j = lane; j < n; j += 32) atomicAdd(hist + bins.of(row[j]), 1);
        __syncwarp();
        const int4 h = *reinterpret_cast<const int4 *>(hist + lane * 4);
        const int c[4] = {h.x, h.y, h.z, h.w};
        int above, in;
        const int bin = find_bin<4>(c, want, lane, above, in);
        lo = INFINITY;
        hi = -INFINITY;
#pragma unroll 8
        for (int j = lane; j < n; j += 32)
            if (bins.of(row[j]) == bin) {
                lo = fminf(lo, row[j]);
                hi = fmaxf(hi, row[j]);
            }
        lo = warp_min(lo);
        hi = warp_max(hi);
        done = above + in == want;
        if (done) thr = {lo, true};
        __syncwarp();  // before the counters are cleared for another row
    }
    if (!done)
        thr = find_threshold(lo, hi, want, [&](float c) {
            int s = 0;
#pragma unroll 8
            for (int j = lane; j < n; j += 32) s += row[j] >= c;
            return (int)__reduce_add_sync(0xffffffffu, s);
        });
    int up = 0;
    if (!thr.whole) {
#pragma unroll 8
        for (int j = lane; j < n; j += 32) up += thr.above(row[j]);
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
