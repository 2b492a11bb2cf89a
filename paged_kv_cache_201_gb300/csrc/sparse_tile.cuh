// What the kernels over runs of tokens share: a tile of consecutive query tokens of one sequence, the
// mask of the tokens that list a page, and the ascending list of the pages that any of them lists.
#pragma once

#include "sparse_common.cuh"

namespace pa {

constexpr int kTileMaxTokens = 32;  // bits of a page's token mask

struct TokenTile {
    int b;           // sequence
    int n_seq, i0;   // its query tokens, the first of them in the tile
    int nt;          // tokens of the tile
    long long tok0;  // row of q of token i0
    int L;           // keys of the sequence
};

// Sequence b's tiles of TPC tokens are blocks [first(b), first(b + 1)) of a packed batch, first(b) =
// floor(q_start[b] / TPC) + b: at least as many as it has, the rest exit.
__device__ __forceinline__ long long first_tile(const FwdParams &p, int b, int TPC) {
    return (long long)__ldg(p.q_start + b) / TPC + b;
}
inline long long count_tiles(const SparseParams &sp, int TPC) {
    const FwdParams &p = sp.f;
    return p.q_start ? sp.n_tok / TPC + p.B : (long long)p.B * ((p.Sq + TPC - 1) / TPC);
}

// Tile `tile`; false where it is nobody's, or a sequence's of fewer than group_min tokens.
__device__ __forceinline__ bool token_tile(const SparseParams &sp, long long tile, int TPC, TokenTile &x) {
    const FwdParams &p = sp.f;
    if (!p.q_start) {
        const int tiles = (p.Sq + TPC - 1) / TPC;
        x.b = (int)(tile / tiles);
        x.n_seq = p.Sq;
        x.i0 = (int)(tile - (long long)x.b * tiles) * TPC;
        x.tok0 = (long long)x.b * p.Sq + x.i0;
    } else {
        int lo = 0, hi = p.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (first_tile(p, mid, TPC) <= tile)
                lo = mid;
            else
                hi = mid;
        }
        x.b = lo;
        const int q0 = __ldg(p.q_start + lo), q1 = __ldg(p.q_start + lo + 1);
        if (q0 < 0 || q1 < q0 || q1 > sp.n_tok) return false;
        x.n_seq = q1 - q0;
        const long long j = tile - first_tile(p, lo, TPC);
        if (x.n_seq < sp.group_min || j < 0 || j * TPC >= x.n_seq) return false;
        x.i0 = (int)j * TPC;
        x.tok0 = (long long)q0 + x.i0;
    }
    x.nt = min(TPC, x.n_seq - x.i0);
    x.L = max(__ldg(p.seq_lens + x.b), 0);
    if (x.L > p.W * p.ps) {
        if (threadIdx.x == 0) atomicOr(p.err, (unsigned int)PA_ERRBIT_SEQ_CLIPPED);
        x.L = p.W * p.ps;
    }
    return true;
}

// The pages of a listed tile, by all WARPS warps of the CTA.  s_mask [np] (zeroed before; behind a barrier)
// becomes the tokens that list each page, put(i, j) receives the i-th listed page; s_count [WARPS].  Returns
// the number of listed pages, or -1 if a token names a page twice.  Ends with a barrier.
template <int WARPS, typename Put>
__device__ __forceinline__ int list_pages(const SparseParams &sp, const TokenTile &x, int kvh, int ps_shift, int np,
                                          const int *s_reach, uint32_t *s_mask, int *s_count, Put put) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ps = 1 << ps_shift;
    bool twice = false;
    for (int tok = warp; tok < x.nt; tok += WARPS) {
        const int32_t *list = sp.sel + ((x.tok0 + tok) * sp.f.Hkv + kvh) * sp.K;
        const int np_tok = (s_reach[tok] + ps - 1) >> ps_shift;
#pragma unroll 4
        for (int e = lane; e < sp.K; e += 32) {
            const int j = __ldg(list + e);
            if (j >= 0 && j < np_tok) twice |= (atomicOr(s_mask + j, 1u << tok) >> tok) & 1u;
        }
    }
    if (__syncthreads_or(twice)) return -1;
    // each warp a run of pages; counts first, then places
    const int run = ((np + WARPS - 1) / WARPS + 31) / 32 * 32, j0 = min(warp * run, np), j1 = min(j0 + run, np);
    int n = 0;
    for (int j = j0 + lane; j - lane < j1; j += 32) n += __popc(__ballot_sync(0xffffffffu, j < j1 && s_mask[j] != 0u));
    if (lane == 0) s_count[warp] = n;
    __syncthreads();
    int at = 0, all = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) at += s_count[w];
        all += s_count[w];
    }
    for (int j = j0 + lane; j - lane < j1; j += 32) {
        const unsigned on = __ballot_sync(0xffffffffu, j < j1 && s_mask[j] != 0u);
        if (j < j1 && s_mask[j] != 0u) put(at + __popc(on & ((1u << lane) - 1)), j);
        at += __popc(on);
    }
    __syncthreads();
    return all;
}

}  // namespace pa
