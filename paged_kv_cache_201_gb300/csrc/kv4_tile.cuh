// What the kernels over a 4-bit cache share: their parameters, which tokens a tile holds, and the limits of a weight.
#pragma once

#include "kv4.cuh"
#include "sparse_common.cuh"

namespace pa {

namespace {

// A weight is 2^(score - ref): ref lies kRefBelow below the largest score when it is moved, which it is once a score lies
// kRefMost above it.
constexpr float kRefBelow = 11.f, kRefMost = 15.f;
constexpr float kLeastFactor = 0x1p-100f;  // a scale of 0 leaves this: kNegInf times it is still no NaN, and any sum times it 0
constexpr float kNoRef = -3e38f;  // before the first key; finite, so that kNegInf - ref is no NaN

struct Kv4Params {
    SparseParams s;
    int S;         // CTAs that share a unit's keys: a cluster, or with part_out a grid's
    float *part_out, *part_state;  // [S, rows of q x heads, D] and [S, rows, 2] (reference, sum) for the second launch
    int TT, HT;    // tokens of a unit; head tiles of a kv head
    int min_tokens;  // tcgen05 kernel, packed batches: of sequences of so many tokens or more
    int seq_tiles; // tiles of every sequence: a uniform batch, or the short runs of a packed one (0: by rows of q)
    int longest_first;  // the mma kernel's sequences by length
};

// What the f16 pair hi lacks of the two weights, as an f16 pair: the differences are exact, and taken from the halves as they
// stand, without a conversion of each.
__device__ __forceinline__ uint32_t remainder(uint32_t hi, float w0, float w1) {
    float x, y;
    asm("{\n\t.reg .b16 p, q;\n\tmov.b32 {p, q}, %2;\n\tsub.f32.f16 %0, p, %3;\n\tsub.f32.f16 %1, q, %4;\n\t}"
        : "=f"(x), "=f"(y)
        : "r"(hi), "f"(w0), "f"(w1));
    return MmaOp<__half>::pack(-x, -y);
}

// A unit's tokens: cnt of sequence b from its token i on; q0 the sequence's first row of q, n its tokens, len its keys.
struct Tile {
    int b, n, i, cnt, len;
    long long q0;
};

// Packed batches: sequence b's tiles are q_start[b] / TT + b and on, which leaves room for all of them; with one
// token a tile they are its rows.  One trip to memory for a batch of up to 32 sequences or of single tokens.
__device__ __forceinline__ Tile find_tile(const Kv4Params &p, int tile, int lane) {
    const FwdParams &f = p.s.f;
    Tile u{0, 0, 0, 0, 0, 0};
    int q0, q1;
    if (p.seq_tiles) {
        u.b = tile / p.seq_tiles;
        u.i = (tile - u.b * p.seq_tiles) * p.TT;
        u.len = __ldg(f.seq_lens + u.b);
        if (!f.q_start) {
            u.n = f.Sq;
            u.q0 = (long long)u.b * f.Sq;
            u.cnt = min(p.TT, u.n - u.i);
            return u;
        }
        q0 = __ldg(f.q_start + u.b);
        q1 = __ldg(f.q_start + u.b + 1);
    } else {
        auto key = [&](int b, int q) { return p.TT == 1 ? q : max(q, 0) / p.TT + b; };
        if (f.B <= 32) {  // a sequence a lane
            const bool mine = lane < f.B;
            const int a = mine ? __ldg(f.q_start + lane) : 0, e = mine ? __ldg(f.q_start + lane + 1) : 0;
            const int len = mine ? __ldg(f.seq_lens + lane) : 0;
            const unsigned below = __ballot_sync(0xffffffffu, mine && key(lane, a) <= tile);
            u.b = below ? 31 - __clz(below) : 0;
            q0 = __shfl_sync(0xffffffffu, a, u.b);
            q1 = __shfl_sync(0xffffffffu, e, u.b);
            u.len = __shfl_sync(0xffffffffu, len, u.b);
        } else {
            const int guess = min(p.TT == 1 ? tile : tile - tile / (p.TT + 1), f.B - 1);  // a token a sequence
            q0 = __ldg(f.q_start + guess);
            q1 = __ldg(f.q_start + guess + 1);
            u.b = guess;
            u.len = __ldg(f.seq_lens + guess);
            if (key(guess, q0) > tile || key(guess + 1, q1) <= tile) {
                int lo = 0, hi = f.B;  // key(lo) <= tile < key(hi)
                while (hi - lo > 1) {  // 31 borders a trip
                    const int step = (hi - lo + 31) / 32;
                    const int b = lo + (lane + 1) * step;
                    const bool below = b < hi && key(b, __ldg(f.q_start + b)) <= tile;
                    const int k = __popc(__ballot_sync(0xffffffffu, below));
                    hi = min(hi, lo + (k + 1) * step);
                    lo += k * step;
                }
                u.b = lo;
                q0 = __ldg(f.q_start + lo);
                q1 = __ldg(f.q_start + lo + 1);
                u.len = __ldg(f.seq_lens + lo);
            }
        }
        u.i = (tile - key(u.b, q0)) * p.TT;
    }
    if (q0 < 0 || q1 < q0 || q1 > p.s.n_tok) return u;
    u.q0 = q0;
    u.n = q1 - q0;
    if (u.i < 0 || u.n < p.min_tokens || (p.s.group_min && u.n >= p.s.group_min)) return u;  // malformed, or the other kernel's
    u.cnt = min(p.TT, u.n - u.i);
    return u;
}

}  // namespace

}  // namespace pa
