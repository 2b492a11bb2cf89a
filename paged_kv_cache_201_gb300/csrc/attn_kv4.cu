// Attention over a 4-bit cache for bf16 / f16 queries: single tokens and short runs, and whatever the tcgen05 kernel
// does not take.
//
// A unit is up to 8 NR query rows (tokens x the heads of a kv head) of one sequence.  A cluster of CTAs shares its
// keys in blocks of 16, every warp of it a run of them, with a ring of its own: nothing is shared and nobody waits for
// another warp until the states are merged.  Products are transposed, S^T = K Q^T and O^T = V^T P^T, so that keys and
// head dimension fill the MMA's 16-row side and a group of up to eight heads its 8-wide side.
//
//   * A step is two blocks.  The block of a (page, kv head), codes and scales of K and V, is contiguous; 16 rows of a larger
//     page land as a page of 16 rows does.
//   * Codes become f16 operands in registers, (u - 8) x scale / 8 or / 128, without rounding (kv4.cuh): a logic
//     operation and a fused multiply-add for two elements, and a shift for eight.  The shares come back in the queries, in the
//     score's factor, when the states are written and in the final division.
//   * K: a lane's 16 (D = 128) bytes are consecutive elements of its key; a register pairs elements d and d + 4, and
//     so do the query operands.  V: O^T's operand pairs two keys of one element.  A byte permutation of two keys'
//     words pairs their halves before the codes are taken apart, so V needs no transposition.
//   * Softmax statistics are float32.  A weight is 2^(score - ref), ref at least 11 below the largest score so far
//     when it was last moved and never more than 15 below any: weights stay below 2^15, ref (and with it every sum)
//     moves rarely, and in f16 nothing above 2^-36 of the row's largest weight is lost.
//   * A weight is an f16 high part plus its remainder, within 2^-22 of it: where the values cancel, a high part alone (2^-11)
//     left bf16 outputs up to 44 times as far off as their own rounding and the float32 sums do.  Units of up to four rows (single tokens of G <= 4) have the
//     remainders' products in columns that nobody else uses: 256 sequences take 164 us, with two products 183, with the
//     high parts alone 159.
//   * The rows of S^T are keys r ^ (r >> 1 & 1): with the four keys of a V load in different rows modulo
//     two, their shared-memory loads have half the bank conflicts, and K's none.
//
// Any byte stands for a finite number, so what lies behind a sequence's last key needs no cleaning: its weight is 0.
//
// What bounds it is instructions: 336 a block of 16 keys of 128 and warp, 138 of them on the integer pipe and 132 on the
// one of multiplications, issued in 67 % of cycles by four warps a scheduler, which wait for those pipes (ncu); memory
// keeps nobody waiting.  256 sequences of 0.4 to 1 times 4096 tokens (8 kv heads of 128, G = 4, bf16) take 164 us, 5.2 TB/s
// or 78 % of the copy rate; one of 131072 tokens, as 19 CTAs a kv head, 39 us, 58 %.
#include <limits.h>

#include "kv4.cuh"
#include "kv4_tile.cuh"
#include "mma_common.cuh"

namespace pa {

using namespace mmac;

namespace {

constexpr int kBlockKeys = 16, kStepKeys = 32;
// Which sequence (or row of a batch of single tokens) the CTAs of place `place` take, so that the longest start first and
// the last to start are short: up to 256 of them by eight classes of length.  Every place has one and every one a place.
__device__ __forceinline__ int longest_first(const FwdParams &f, int place, int lane) {
    constexpr int N = 8;
    int len[N], least = INT_MAX, most = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int b = 32 * k + lane;
        len[k] = b < f.B ? max(__ldg(f.seq_lens + b), 0) : -1;
    }
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (len[k] >= 0) least = min(least, len[k]), most = max(most, len[k]);
    least = __reduce_min_sync(0xffffffffu, least);
    most = __reduce_max_sync(0xffffffffu, most);
    const float scale = 8.f / ((float)(most - least) + 1.f);
    int of[N];  // class, the longest's 0
    uint32_t count = 0;  // of this lane's, four bits a class
#pragma unroll
    for (int k = 0; k < N; ++k) {
        of[k] = len[k] < 0 ? 8 : min((int)((float)(most - len[k]) * scale), 7);
        if (len[k] >= 0) count += 1u << (4 * of[k]);
    }
    uint32_t all[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) all[i] = __reduce_add_sync(0xffffffffu, count >> (4 * i) & 0x000F000Fu);
    int c = 0, left = place;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int n = all[i & 3] >> (i < 4 ? 0 : 16) & 0xffff;
        if (c == i && left >= n) {
            left -= n;
            ++c;
        }
    }
    int found = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const unsigned in = __ballot_sync(0xffffffffu, of[k] == c);
        const bool me = of[k] == c && __popc(in & ((1u << lane) - 1)) == left;
        const unsigned who = __ballot_sync(0xffffffffu, me);
        if (who) found = 32 * k + __ffs(who) - 1;
        left -= __popc(in);
    }
    return found;
}

// A unit: up to R rows r = token x heads + head of tile u and kv head kvh.
struct Unit {
    Tile u;
    int kvh, h0, heads, rows;
    int L, k_hi;  // keys of the sequence; those that the unit's last token, which reaches furthest, sees
    __device__ __forceinline__ Unit(const Kv4Params &p, int R, int index, int lane, int ps_shift, bool report) {
        const FwdParams &f = p.s.f;
        h0 = index % p.HT * R;
        index /= p.HT;
        kvh = index % f.Hkv;
        index /= f.Hkv;
        if (p.longest_first) {  // see make_plan
            const int tiles = max(p.seq_tiles, 1), place = index / tiles;
            index = longest_first(f, place, lane) * tiles + (index - place * tiles);
        }
        u = find_tile(p, index, lane);
        heads = min(R, f.G - h0);
        rows = L = k_hi = 0;
        if (u.cnt <= 0) return;
        rows = u.cnt * heads;
        L = max(u.len, 0);
        if (L > f.W << ps_shift) {  // never read past the sequence's block-table row
            if (report) atomicOr(f.err, (unsigned int)PA_ERRBIT_SEQ_CLIPPED);
            L = f.W << ps_shift;
        }
        k_hi = limit(f, u.cnt - 1);
    }
    __device__ __forceinline__ int limit(const FwdParams &f, int token) const {
        return row_key_limit(f, u.b, L, u.i + token, u.n);
    }
    __device__ __forceinline__ long long row(const FwdParams &f, int r) const {
        return (u.q0 + u.i + r / heads) * f.Hq + kvh * f.G + h0 + r % heads;
    }
};

__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)) : "memory");
}

// A warp's ring: blocks [b0, b1) of 16 keys (b0 even), two a step, into NST slots of its own, filled in order.  The copies
// are 16 bytes a lane and the warp waits for its own by count: a bulk copy's barrier, its byte count and its uniform
// operands cost 44 instructions a block.  PAGE16: pages of 16 rows, whose blocks are contiguous; a step's rows of a larger
// page land as two of those.
template <int D, int NST, bool PAGE16>
struct Ring {
    static constexpr int kBlock = kBlockKeys * D / 8 * 9;  // bytes of a block: as a page of 16 rows
    static constexpr int kStep = 2 * kBlock;
    static constexpr int kCodes = kBlockKeys * D / 2, kScales = kBlockKeys * D / kv4::kGroup;
    static constexpr int kPages = PAGE16 ? 2 : 1;  // of a step
    const FwdParams &p;
    const int32_t *table;        // this sequence's row
    const uint8_t *from;         // page 0's block of this kv head, at this lane's codes
    uint32_t stride;             // bytes from page to page
    uint32_t smem, slot_at;      // this lane's codes in slot 0 and in the next one to fill
    int v_codes, scales;         // larger pages: from there to the V codes, to this lane's scales
    int blk, b1, ps_shift, lane;
    int id[kPages];              // pages of the next step to fill

    __device__ __forceinline__ Ring(const FwdParams &f, int b, int kvh, int shift, int block0, int block1, uint32_t smem_,
                                    int lane_)
        : p(f), table(f.block_table + (long long)b * f.W), blk(block0), b1(block1), ps_shift(shift), lane(lane_) {
        const int ps = 1 << shift, size = kv4::block_bytes(ps, D);
        stride = (uint32_t)f.Hkv * (uint32_t)size;
        from = static_cast<const uint8_t *>(f.k_cache) + (long long)kvh * size + lane * 16;
        smem = slot_at = smem_ + lane * 16;
        v_codes = ps * (D / 2);
        constexpr int kLanes = kScales / 16;  // of a side's scales
        scales = ps * D + (lane < kLanes ? 0 : (ps - kBlockKeys) * (D / kv4::kGroup));
        look_up();
    }
    __device__ __forceinline__ void look_up() {
        if (PAGE16) {
#pragma unroll
            for (int hb = 0; hb < kPages; ++hb) id[hb] = blk + hb < b1 ? __ldg(table + blk + hb) : 0;
        } else {
            id[0] = blk < b1 ? __ldg(table + (blk >> (ps_shift - 4))) : 0;
        }
    }
    // A page outside the pool is not followed: its rows become zeros.
    __device__ __forceinline__ void no_page(uint32_t to) {
        if (lane == 0) atomicOr(p.err, (unsigned int)PA_ERRBIT_PAGE_RANGE);
        for (int i = lane * 16; i < kBlock; i += 512)
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(to - lane * 16 + i), "r"(0) : "memory");
    }
    // A block's copies, from a page's start (of this lane's codes) and, in a larger page, its row.
    __device__ __forceinline__ void copy_block(uint32_t to, const uint8_t *page, int row) {
        const bool my_scales = lane < 2 * kScales / 16;
        if (PAGE16) {
#pragma unroll
            for (int i = 0; i < 2 * kCodes; i += 512) copy16(to + i, page + i);
            if (my_scales) copy16(to + 2 * kCodes, page + 2 * kCodes);
        } else {
            const uint8_t *k = page + row * (D / 2), *v = k + v_codes;
#pragma unroll
            for (int i = 0; i < kCodes; i += 512) {
                copy16(to + i, k + i);
                copy16(to + kCodes + i, v + i);
            }
            if (my_scales) copy16(to + 2 * kCodes, page + scales + row * (D / kv4::kGroup));
        }
    }
    __device__ __forceinline__ const uint8_t *page_at(int at) const { return from + (unsigned long long)(uint32_t)at * stride; }
    // Starts the copies of the next step into its slot, which nobody reads any more.
    __device__ __forceinline__ void fill() {
        const uint32_t last = max((uint32_t)id[0], (uint32_t)id[kPages - 1]);
        const int row = (blk << 4) & ((1 << ps_shift) - 1);
        if (blk + 1 < b1 && last < (uint32_t)p.num_pages) {  // two blocks, their pages in the pool
            copy_block(slot_at, page_at(id[0]), row);
            copy_block(slot_at + kBlock, page_at(id[kPages - 1]), row + kBlockKeys);
        } else {
#pragma unroll 1
            for (int hb = 0; hb < 2 && blk + hb < b1; ++hb) {
                const int at = hb ? id[kPages - 1] : id[0];
                if ((uint32_t)at < (uint32_t)p.num_pages)
                    copy_block(slot_at + hb * kBlock, page_at(at), row + hb * kBlockKeys);
                else
                    no_page(slot_at + hb * kBlock);
            }
        }
        blk += 2;
        look_up();
        slot_at = slot_at == smem + (NST - 1) * kStep ? smem : slot_at + kStep;
    }
};

template <int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[N]) {
    if constexpr (N == 1) {
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(addr) : "memory");
    } else if constexpr (N == 2) {
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr) : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                         : "r"(addr + 4 * i)
                         : "memory");
    }
}
// N (1, 2 or 4) consecutive bytes, the first lowest.
template <int N>
__device__ __forceinline__ uint32_t lds_bytes(uint32_t addr) {
    uint32_t v;
    if constexpr (N == 1)
        asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    else if constexpr (N == 2)
        asm volatile("ld.shared.u16 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    else
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// A query row's D / 4 elements of this lane as f16 operand pairs, pair 4 w + k = elements 8 w + k and 8 w + k + 4.
// Returns the factor of their products.  negate: as -q.
template <typename T, int D>
__device__ __forceinline__ float load_q(const T *row, bool valid, bool negate, int tq, uint32_t (&w)[D / 8]) {
    const uint4 *src = reinterpret_cast<const uint4 *>(row + tq * (D / 4));
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        const uint4 x = valid ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
        w[4 * i] = __byte_perm(x.x, x.z, 0x5410);
        w[4 * i + 1] = __byte_perm(x.x, x.z, 0x7632);
        w[4 * i + 2] = __byte_perm(x.y, x.w, 0x5410);
        w[4 * i + 3] = __byte_perm(x.y, x.w, 0x7632);
    }
    if (negate)
#pragma unroll
        for (int i = 0; i < D / 8; ++i) w[i] ^= 0x80008000u;
    float am = kv4::largest_of<T>(w);
    am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
    am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
    return kv4::scale_query<T>(w, am);
}

template <typename T>
__device__ __forceinline__ void store4(T *o, float4 v) {
    uint2 w = make_uint2(MmaOp<T>::pack(v.x, v.y), MmaOp<T>::pack(v.z, v.w));
    *reinterpret_cast<uint2 *>(o) = w;
}

// Elements c .. c + 3 of a row whose sums are o (of values / 8) and sum, with reference M.
template <typename T, int D>
__device__ __forceinline__ void store_row(const FwdParams &f, long long row, int c, float4 o, float M, float sum) {
    const float inv = sum != 0.f ? 8.f / sum : 0.f;  // a NaN stays one
    store4<T>(static_cast<T *>(f.out) + row * D + c, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    if (c == 0 && f.lse) f.lse[row] = sum != 0.f ? M * kLn2 + logf(sum) : kNegInf;
}

// Shared memory of the merge: rows [warps][R][D + 4], references and sums [warps][R], then the CTA's own [R] each.
__host__ __device__ constexpr size_t merge_bytes(int D, int R, int warps) {
    return ((size_t)warps * R * (D + 4) + (2 * warps + 2) * R) * 4;
}
__host__ __device__ constexpr int ring_slots(int D) { return D == 64 ? 4 : D == 128 ? 3 : 2; }

// HALF: the unit has four rows at most, and columns c and c + 4 of the products are row c: the same scores twice, then the
// weights' high parts in the first four columns and the remainders in the others, in one product.
template <typename T, int D, int NR, int NW, int MINB, bool PAGE16, bool HALF>
__global__ void __launch_bounds__(NW * 32, MINB) paged_attn_kv4_kernel(const Kv4Params p, int ps_shift) {
    static_assert(!HALF || NR == 1, "four rows are one tile of eight columns");
    constexpr int kParts = HALF ? 1 : 2;  // products of V and the weights
    using Op = MmaOp<__half>;
    constexpr int R = 8 * NR, NST = ring_slots(D), kThreads = NW * 32;
    constexpr int MT = D / 16;  // 16-wide head-dim tiles of O^T
    constexpr int KW = D / 32;  // words of a lane's part of a K row: D / 4 elements
    constexpr int VW = D / 64;  // words of a lane's part of a V row: D / 8 elements
    constexpr int KS = D / 64;  // K scales of a lane's part
    constexpr int VS = D == 256 ? 2 : 1;
    using RingT = Ring<D, NST, PAGE16>;
    extern __shared__ __align__(128) uint8_t smem[];
    const FwdParams &f = p.s.f;
    if (!p.s.group_min) wait_for_stream();  // else beside the tcgen05 kernel, which came behind the stream's others
    RangeCheck ranges(p.s);
    BehindFirst behind(p.s);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)(blockIdx.x % p.S);
    const Unit un(p, R, (int)(blockIdx.x / p.S), lane, ps_shift, threadIdx.x == 0);
    ranges.report(f);
    if (un.rows == 0) return;
    const int rows = un.rows, k_hi = un.k_hi;
    auto row_index = [&](int r) { return un.row(f, r); };
    if (k_hi <= 0) {
        if (rank == 0) {
            for (int i = threadIdx.x; i < rows * (D / 4); i += kThreads)
                store4<T>(static_cast<T *>(f.out) + row_index(i / (D / 4)) * D + i % (D / 4) * 4, make_float4(0.f, 0.f, 0.f, 0.f));
            if (f.lse && threadIdx.x < rows) f.lse[row_index(threadIdx.x)] = kNegInf;
        }
        return;
    }
    // this warp's run of the blocks
    const int blocks = (k_hi - 1) / kBlockKeys + 1;
    const int share = 2 * ((blocks + 2 * p.S * NW - 1) / (2 * p.S * NW));
    const int b0 = min((rank * NW + warp) * share, blocks), b1 = min(b0 + share, blocks);
    const int steps = (b1 - b0 + 1) / 2;

    const uint32_t ring_smem = smem_u32(smem) + warp * NST * RingT::kStep;
    RingT ring(f, un.u.b, un.kvh, ps_shift, b0, b1, ring_smem, lane);
#pragma unroll 1
    for (int st = 0; st < NST; ++st) {
        if (st < steps) ring.fill();
        asm volatile("cp.async.commit_group;" ::: "memory");
    }

    const int g = lane >> 2, tq = lane & 3;
    const int kg = g ^ ((g >> 1) & 1);  // this lane's K rows of a block: keys kg and kg + 8
    const int va = (2 * tq) ^ (tq & 1), vb = (2 * tq + 1) ^ (tq & 1);  // V keys va, vb, va + 8, vb + 8
    uint32_t qb[NR][D / 8];
    float srow[NR][2];
    int lim[NR][2];  // keys of the rows of this lane's score columns; rows past the unit's: all
    int all_below = b1 * kBlockKeys;
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
        const int r = HALF ? g & 3 : nr * 8 + g;
        const bool valid = r < rows;
        const T *q = static_cast<const T *>(f.q) + (valid ? q_row_offset(f, row_index(r)) : 0);
        const float factor = load_q<T, D>(q, valid, f.scale_log2 < 0.f, tq, qb[nr]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int rc = HALF ? (2 * tq + e) & 3 : nr * 8 + 2 * tq + e;
            srow[nr][e] = fmaxf(fabsf(f.scale_log2) * __shfl_sync(0xffffffffu, factor, 4 * (2 * tq + e)), kLeastFactor);
            lim[nr][e] = min(rc < rows ? un.limit(f, rc / un.heads) : INT_MAX, b1 * kBlockKeys);
            all_below = min(all_below, lim[nr][e]);
        }
    }
    all_below = __reduce_min_sync(0xffffffffu, all_below);  // keys that every row sees
    float ref[NR][2], l[NR][2], acc[NR][MT][4];
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
        ref[nr][0] = ref[nr][1] = kNoRef;
        l[nr][0] = l[nr][1] = 0.f;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) acc[nr][mt][0] = acc[nr][mt][1] = acc[nr][mt][2] = acc[nr][mt][3] = 0.f;
    }
    // offsets of this lane's parts within a block
    constexpr kv4::Layout at{kBlockKeys, D};
    const uint32_t k_off = at.codes(0, kg) + tq * (D / 8), ks_off = at.scales(0, kg) + tq * KS;
    const uint32_t va_off = at.codes(1, va) + g * (D / 16), vb_off = at.codes(1, vb) + g * (D / 16);
    const uint32_t vs_col = at.scales(1, 0) + (D == 64 ? g >> 1 : g * VS);
    int slot = 0;
#pragma unroll 1
    for (int t = 0; t < steps; ++t) {
        const uint32_t base = ring_smem + slot * RingT::kStep;
        const int j0 = (b0 + 2 * t) * kBlockKeys;
        asm volatile("cp.async.wait_group %0;" ::"n"(NST - 1) : "memory");  // a step is a group
        __syncwarp();
        // ---- S^T = K Q^T, the two blocks' products in turn
        float sc[2][NR][4];
        uint32_t ksb[2][2];
#pragma unroll
        for (int hb = 0; hb < 2; ++hb) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                ksb[hb][i] = lds_bytes<KS>(base + hb * RingT::kBlock + ks_off + i * 8 * (D / 16));
            }
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) sc[hb][nr][0] = sc[hb][nr][1] = sc[hb][nr][2] = sc[hb][nr][3] = 0.f;
        }
#pragma unroll
        for (int w = 0; w < KW; ++w)
#pragma unroll
            for (int hb = 0; hb < 2; ++hb) {
                uint32_t h[2][4];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    // the scale of word w: byte w / 2 of the lane's; of two at a time (256 sequences 164 -> 159 us)
                    const kv4::ScalePair two = kv4::scale_pair(__byte_perm(ksb[hb][i], 0, w < 4 ? 0x4140 : 0x4342));
                    // (word by word: a whole row's at once leaves too few registers, 3 us of 192 then)
                    uint32_t code[1];
                    lds_words<1>(base + hb * RingT::kBlock + k_off + i * 8 * (D / 2) + 4 * w, code);
                    if (w / 2 % 2 == 0)
                        kv4::unpack8<0>(code[0], two, h[i]);
                    else
                        kv4::unpack8<1>(code[0], two, h[i]);
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t a[4] = {h[0][2 * k], h[1][2 * k], h[0][2 * k + 1], h[1][2 * k + 1]};
#pragma unroll
                    for (int nr = 0; nr < NR; ++nr)
                        Op::run(sc[hb][nr], a, qb[nr][4 * w + 2 * k], qb[nr][4 * w + 2 * k + 1]);
                }
            }
        // ---- weights; a score more than kRefMost above its reference moves it
        float mx[NR][2];
        bool over = false;
        if (j0 > all_below - kStepKeys) {
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                        for (int kh = 0; kh < 2; ++kh)
                            if (hb * kBlockKeys + kg + 8 * kh >= lim[nr][e] - j0) sc[hb][nr][2 * kh + e] = kNegInf;
        }
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                mx[nr][e] = fmaxf(fmaxf(sc[0][nr][e], sc[0][nr][2 + e]), fmaxf(sc[1][nr][e], sc[1][nr][2 + e])) * srow[nr][e];
                over |= mx[nr][e] > ref[nr][e] + kRefMost;
            }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) {
                float al[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float m = mx[nr][e];
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                    const float next = fmaxf(ref[nr][e], m - kRefBelow);
                    al[e] = fast_exp2(ref[nr][e] - next);
                    ref[nr][e] = next;
                    l[nr][e] *= al[e];
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[nr][mt][i] *= al[i & 1];
            }
        }
        uint32_t pb[2][NR][kParts][2];  // [block][row tile][high part / remainder][keys 0-7 / 8-15]
#pragma unroll
        for (int hb = 0; hb < 2; ++hb)
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) {
                float w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = fast_exp2(fmaf(sc[hb][nr][i], srow[nr][i & 1], -ref[nr][i & 1]));
                l[nr][0] += w[0] + w[2];
                l[nr][1] += w[1] + w[3];
#pragma unroll
                for (int kh = 0; kh < 2; ++kh) {
                    const uint32_t hi = Op::pack(w[2 * kh], w[2 * kh + 1]);
                    const uint32_t lo = remainder(hi, w[2 * kh], w[2 * kh + 1]);
                    if constexpr (HALF) {
                        pb[hb][nr][0][kh] = movmatrix_trans(tq < 2 ? hi : lo);
                    } else {
                        pb[hb][nr][0][kh] = movmatrix_trans(hi);
                        pb[hb][nr][1][kh] = movmatrix_trans(lo);
                    }
                }
            }
        // ---- O^T += V^T P^T
#pragma unroll
        for (int hb = 0; hb < 2; ++hb) {
            const uint32_t blk = base + hb * RingT::kBlock;
            uint32_t vw[4][VW];
            kv4::ScalePair vs[2][VS];  // of the keys (va, vb) and (va + 8, vb + 8)
#pragma unroll
            for (int kh = 0; kh < 2; ++kh) {
                lds_words<VW>(blk + va_off + kh * 8 * (D / 2), vw[2 * kh]);
                lds_words<VW>(blk + vb_off + kh * 8 * (D / 2), vw[2 * kh + 1]);
                const uint32_t a = lds_bytes<VS>(blk + vs_col + (va + 8 * kh) * (D / 16));
                const uint32_t b = lds_bytes<VS>(blk + vs_col + (vb + 8 * kh) * (D / 16));
#pragma unroll
                for (int i = 0; i < VS; ++i)
                    vs[kh][i] = kv4::scale_pair(__byte_perm(a, b, 0x3430 + i * 0x0101));
            }
            if (hb == 1) {  // the step is in registers
                __syncwarp();
                if (t + NST < steps) ring.fill();
                asm volatile("cp.async.commit_group;" ::: "memory");
            }
#pragma unroll
            for (int w = 0; w < VW; ++w)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t h[2][4];
#pragma unroll
                    for (int kh = 0; kh < 2; ++kh)
                        kv4::unpack8(__byte_perm(vw[2 * kh][w], vw[2 * kh + 1][w], half ? 0x7632 : 0x5410),
                                     vs[kh][w * VS / VW], h[kh]);
#pragma unroll
                    for (int part = 0; part < kParts; ++part)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t a[4] = {h[0][2 * k], h[0][2 * k + 1], h[1][2 * k], h[1][2 * k + 1]};
#pragma unroll
                            for (int nr = 0; nr < NR; ++nr)
                                Op::run(acc[nr][4 * w + 2 * half + k], a, pb[hb][nr][part][0], pb[hb][nr][part][1]);
                        }
                }
        }
        slot = slot + 1 == NST ? 0 : slot + 1;
    }
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[nr][e] += __shfl_xor_sync(0xffffffffu, l[nr][e], 4);
            l[nr][e] += __shfl_xor_sync(0xffffffffu, l[nr][e], 8);
            l[nr][e] += __shfl_xor_sync(0xffffffffu, l[nr][e], 16);
        }
    if constexpr (HALF) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[0][mt][i] += __shfl_xor_sync(0xffffffffu, acc[0][mt][i], 2);
    }
    // ---- the warps' states: tile mt's rows g and g + 8 are elements g D / 8 + 2 mt and the next
    float *sm = reinterpret_cast<float *>(smem);
    constexpr int STRIDE = D + 4;
    float *s_m = sm + NW * R * STRIDE, *s_l = s_m + NW * R, *s_cta = s_l + NW * R;  // s_cta: [R] references, [R] sums
    __syncthreads();  // no warp reads its ring any more
    float *wa = sm + warp * R * STRIDE;
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
        if (HALF && tq >= 2) break;  // rows 0 .. 3
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                *reinterpret_cast<float2 *>(wa + (nr * 8 + 2 * tq + e) * STRIDE + g * (D / 8) + 2 * mt) =
                    make_float2(kv4::kEvenShare * acc[nr][mt][e], acc[nr][mt][2 + e]);
        if (g == 0) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                s_m[warp * R + nr * 8 + 2 * tq + e] = ref[nr][e];
                s_l[warp * R + nr * 8 + 2 * tq + e] = l[nr][e];
            }
        }
    }
    __syncthreads();
    auto store = [&](int r, int c, float4 o, float M, float sum) { store_row<T, D>(f, row_index(r), c, o, M, sum); };
    for (int i = threadIdx.x; i < rows * (D / 4); i += kThreads) {
        const int r = i / (D / 4), c = i % (D / 4) * 4;
        float M = kNoRef, sum = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) M = fmaxf(M, s_m[w * R + r]);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float k = fast_exp2(s_m[w * R + r] - M);
            const float4 v = *reinterpret_cast<const float4 *>(sm + (w * R + r) * STRIDE + c);
            sum += k * s_l[w * R + r];
            o.x += k * v.x, o.y += k * v.y, o.z += k * v.z, o.w += k * v.w;
        }
        if (p.part_out) {
            const long long at_row = rank * p.s.n_tok * f.Hq + row_index(r);
            *reinterpret_cast<float4 *>(p.part_out + at_row * D + c) = o;
            if (c == 0) *reinterpret_cast<float2 *>(p.part_state + 2 * at_row) = make_float2(M, sum);
        } else if (p.S == 1) {
            store(r, c, o, M, sum);
        } else {  // the row's slot of warp 0 is this thread's alone
            *reinterpret_cast<float4 *>(sm + r * STRIDE + c) = o;
            if (c == 0) {
                s_cta[r] = M;
                s_cta[R + r] = sum;
            }
        }
    }
    if (p.S == 1 || p.part_out) return;
    // ---- the CTAs' states: each stores its share of the rows' elements
    cluster_barrier();
    for (int i = rank * kThreads + threadIdx.x; i < rows * (D / 4); i += p.S * kThreads) {
        const int r = i / (D / 4), c = i % (D / 4) * 4;
        const uint32_t at_m = smem_u32(s_cta + r), at_l = smem_u32(s_cta + R + r), at_o = smem_u32(sm + r * STRIDE + c);
        float M = kNoRef, sum = 0.f;
        for (int x = 0; x < p.S; ++x) M = fmaxf(M, peer_load(peer_addr(at_m, x)));
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int x = 0; x < p.S; ++x) {
            const float k = fast_exp2(peer_load(peer_addr(at_m, x)) - M);
            const float4 v = peer_load4(peer_addr(at_o, x));
            sum += k * peer_load(peer_addr(at_l, x));
            o.x += k * v.x, o.y += k * v.y, o.z += k * v.z, o.w += k * v.w;
        }
        store(r, c, o, M, sum);
    }
    cluster_barrier();  // the peers have read this CTA's memory
}

// The second launch where a grid's CTAs shared the keys: one row of a unit a CTA, its parts dealt out to the warps.
template <typename T, int D>
__global__ void __launch_bounds__(128) paged_attn_kv4_join_kernel(const Kv4Params p, int R, int ps_shift) {
    const FwdParams &f = p.s.f;
    constexpr int C = D / 4, TG = 128 / C;  // threads of a row, parts at once
    __shared__ float4 s_o[TG][C];
    __shared__ float s_l[TG];
    const int c = threadIdx.x % C, tg = threadIdx.x / C, r = blockIdx.x % R;
    const Unit un(p, R, (int)(blockIdx.x / R), threadIdx.x & 31, ps_shift, false);
    wait_for_stream();
    if (r >= un.rows || un.k_hi <= 0) return;
    const long long row = un.row(f, r), rows = p.s.n_tok * f.Hq;
    const float2 *state = reinterpret_cast<const float2 *>(p.part_state) + row;
    float M = kNoRef, sum = 0.f;
    for (int x = threadIdx.x & 31; x < p.S; x += 32) M = fmaxf(M, __ldcg(state + x * rows).x);
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, i));
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int U = 8;  // parts of a thread on their way together
    for (int x0 = tg; x0 < p.S; x0 += U * TG) {
        float2 st[U];
        float4 v[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int x = min(x0 + i * TG, p.S - 1);
            st[i] = __ldcg(state + x * rows);
            v[i] = __ldcg(reinterpret_cast<const float4 *>(p.part_out + (x * rows + row) * D) + c);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const float k = x0 + i * TG < p.S ? fast_exp2(st[i].x - M) : 0.f;
            sum += k * st[i].y;
            o.x += k * v[i].x, o.y += k * v[i].y, o.z += k * v[i].z, o.w += k * v[i].w;
        }
    }
    s_o[tg][c] = o;
    if (c == 0) s_l[tg] = sum;
    __syncthreads();
    if (tg != 0) return;
#pragma unroll
    for (int x = 1; x < TG; ++x) {
        const float4 v = s_o[x][c];
        sum += s_l[x];
        o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
    }
    store_row<T, D>(f, row, c * 4, o, M, sum);
}

// How a call is cut: units of 8 NR rows, the keys of each shared by S CTAs of `warps` warps.
struct Plan {
    int nr, warps, HT, TT, seq_tiles;
    long long units;
    int S;
    bool grid;  // S of the grid's CTAs, joined by a second launch; else a cluster
    bool longest_first;
    bool half;  // units of four rows at most
};
Plan make_plan(const SparseParams &sp, int sms, long long ws_bytes) {
    const FwdParams &f = sp.f;
    Plan a{};
    // rows of an average sequence (a uniform batch: of every one)
    const double rows = (f.q_start ? (double)sp.n_tok / f.B : (double)f.Sq) * f.G;
    a.nr = f.D == 256 || rows <= 8 || (f.G > 16 && f.G <= 24) ? 1 : 2;
    const int R = 8 * a.nr, full = f.D == 256 ? 8 : a.nr == 2 ? 12 : 16;  // warps that fill a multiprocessor
    const int ctas = f.D == 256 ? 2 : a.nr == 2 ? 3 : 4;                  // CTAs that do otherwise
    a.HT = (f.G + R - 1) / R;
    a.TT = f.q_start && sp.n_tok <= f.B ? 1 : f.G < R ? R / f.G : 1;
    a.half = a.nr == 1 && f.G * (f.q_start ? a.TT : a.TT < f.Sq ? a.TT : f.Sq) <= 4;
    long long tiles;
    if (!f.q_start || sp.by_seq) {
        a.seq_tiles = ((f.q_start ? sp.group_min - 1 : f.Sq) + a.TT - 1) / a.TT;
        tiles = (long long)f.B * a.seq_tiles;
    } else {
        tiles = a.TT == 1 ? sp.n_tok : sp.n_tok / a.TT + f.B;
    }
    a.units = tiles * f.Hkv * a.HT;
    a.S = 1;
    if (a.units == 0) return a;
    // Few units: their keys go to several CTAs, as long as a warp keeps two steps of the longest sequence.  While every CTA
    // can have a multiprocessor of its own it takes all of it (half as large ones of a cluster would be packed onto half
    // of the multiprocessors).  Clusters of two or four: 15 of eight and 7 of sixteen fit at once, which leaves too many
    // multiprocessors idle; with a workspace any number of the grid's CTAs, and a second launch.
    const long long keys = (long long)f.W * f.ps;
    a.warps = full;
    while (a.S < 4 && a.units * 2 * a.S <= sms && keys >= 4ll * kStepKeys * full * a.S) a.S *= 2;
    long long n = sms / a.units;
    const long long most = keys / (2ll * kStepKeys * full), part = sp.n_tok * f.Hq * (f.D + 2) * 4;
    n = n < most ? n : most;
    if (!sp.group_min && n > a.S && ws_bytes / part >= n && a.units * R <= 0x7fffffffLL) {
        // 1024 keys take a multiprocessor some 4 us at head_dim 128, the second launch takes 3
        const double one = 4.0 * keys / 1024 * f.D / 128;
        if (one / n + 3 < one / a.S) {
            a.S = (int)n;
            a.grid = true;
        }
    }
    if (a.units * a.S <= sms) return a;
    a.warps = full / ctas;
    while (a.S < 4 && a.units * a.S * 2 <= (long long)sms * ctas && keys >= 4ll * kStepKeys * a.warps * a.S) a.S *= 2;
    // More than one wave of CTAs: the longest sequences first, lest one starts when the others end.  Sequences of 0.4 to 1
    // times the table's 4096 columns, 8 kv heads: 256 of them 178 -> 170 us, 152 114 -> 101, 110 99 -> 89.  Finding the
    // sequence costs a CTA half a microsecond: with 1024 columns 100 sequences 29.5 -> 27.2, but 256 59.7 -> 61.2 (2048
    // columns: 96.8 -> 95.1).  Past 256 sequences, more lengths than a warp holds eight to a lane, the order is the caller's: 300
    // take 194 us mixed and 176 with the longest first in the table, 512 319 and 300.
    const long long wave = (long long)sms * ctas, n_ctas = a.units * a.S;
    a.longest_first = n_ctas > wave && f.B > 1 && f.B <= 256 && (keys >= 2048 || (keys >= 1024 && n_ctas <= 2 * wave)) &&
                      (a.seq_tiles > 0 || (a.TT == 1 && sp.n_tok == f.B));
    return a;
}

template <typename T, int D, int NR, int NW, int MINB, bool HALF>
cudaError_t launch_kv4(Kv4Params p, const Plan &a, cudaStream_t stream) {
    constexpr int R = 8 * NR;
    constexpr size_t ring = (size_t)NW * ring_slots(D) * 2 * kv4::block_bytes(kBlockKeys, D);
    constexpr size_t smem = ring > merge_bytes(D, R, NW) ? ring : merge_bytes(D, R, NW);
    const FwdParams &f = p.s.f;
    if (a.units * a.S > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    p.S = a.S;
    p.HT = a.HT;
    p.TT = a.TT;
    p.seq_tiles = a.seq_tiles;
    p.longest_first = a.longest_first;
    if (a.grid) {
        p.part_out = static_cast<float *>(p.s.ws);
        p.part_state = p.part_out + a.S * p.s.n_tok * f.Hq * D;
    }
    const bool page16 = f.ps == kBlockKeys;
    const int ps_shift = f.ps == 16 ? 4 : f.ps == 32 ? 5 : 6;
    auto kern = page16 ? paged_attn_kv4_kernel<T, D, NR, NW, MINB, true, HALF> : paged_attn_kv4_kernel<T, D, NR, NW, MINB, false, HALF>;
    static SmemLimit limits[2];
    cudaError_t e = limits[page16].raise((const void *)kern, smem);
    if (e != cudaSuccess) return e;
    e = launch_behind(kern, dim3((unsigned)(a.units * a.S)), NW * 32, smem, a.grid ? 1 : a.S, stream, p, ps_shift);
    if (e != cudaSuccess || !a.grid) return e;
    return launch_behind(paged_attn_kv4_join_kernel<T, D>, dim3((unsigned)(a.units * R)), 128, 0, 1, stream, p, R, ps_shift);
}

template <typename T, int D, bool HALF>
cudaError_t launch_kv4_rows8(const Kv4Params &p, const Plan &a, cudaStream_t stream) {
    if constexpr (D == 256)
        return a.warps == 8 ? launch_kv4<T, D, 1, 8, 1, HALF>(p, a, stream) : launch_kv4<T, D, 1, 4, 2, HALF>(p, a, stream);
    else
        return a.warps == 16 ? launch_kv4<T, D, 1, 16, 1, HALF>(p, a, stream) : launch_kv4<T, D, 1, 4, 4, HALF>(p, a, stream);
}

template <typename T, int D>
cudaError_t launch_kv4_d(const Kv4Params &p, const Plan &a, cudaStream_t stream) {
    if constexpr (D != 256)
        if (a.nr == 2)
            return a.warps == 12 ? launch_kv4<T, D, 2, 12, 1, false>(p, a, stream) : launch_kv4<T, D, 2, 4, 3, false>(p, a, stream);
    return a.half ? launch_kv4_rows8<T, D, true>(p, a, stream) : launch_kv4_rows8<T, D, false>(p, a, stream);
}

template <typename T>
cudaError_t launch_kv4_t(const Kv4Params &p, const Plan &a, cudaStream_t stream) {
    if (p.s.f.D == 64) return launch_kv4_d<T, 64>(p, a, stream);
    if (p.s.f.D == 128) return launch_kv4_d<T, 128>(p, a, stream);
    return launch_kv4_d<T, 256>(p, a, stream);
}

}  // namespace

long long kv4_workspace_bytes(const SparseParams &sp, int sms) {
    const Plan a = make_plan(sp, sms, LLONG_MAX);
    return a.grid ? a.S * sp.n_tok * sp.f.Hq * (sp.f.D + 2) * 4 : 0;
}

cudaError_t launch_kv4_mma(const SparseParams &sp, int dtype, int sms, cudaStream_t stream) {
    Kv4Params p{};
    p.s = sp;
    const Plan a = make_plan(sp, sms, sp.ws ? sp.ws_bytes : 0);
    if (a.units == 0) return cudaSuccess;
    if (dtype == PA_BF16) return launch_kv4_t<__nv_bfloat16>(p, a, stream);
    return launch_kv4_t<__half>(p, a, stream);
}

}  // namespace pa
