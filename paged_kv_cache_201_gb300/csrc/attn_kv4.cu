// Attention over a 4-bit cache for bf16 / f16 queries: single tokens and short runs, and whatever the tcgen05 kernel
// does not take.
//
// A unit is up to 8 NR query rows (tokens x the heads of a kv head) of one sequence; a cluster of CTAs shares its
// keys, and each CTA's four consumer warps share the CTA's: warp w takes keys [16 w, 16 w + 16) of every 64-key
// stage.  Products are transposed, S^T = K Q^T and O^T = V^T P^T, so that keys and head dimension fill the MMA's
// 16-row side and a group of up to eight heads its 8-wide side.
//
//   * A (page, kv head) block, codes and scales of K and V, is contiguous: one untiled bulk copy a page.
//   * Codes become f16 operands in registers, (u - 8) x scale / 8, without rounding (kv4.cuh): a shift, a logic
//     operation and a fused multiply-add for two elements.  The eighth comes back in the score's factor and in
//     the final division.
//   * K: a lane's 16 (D = 128) bytes are consecutive elements of its key; a register pairs elements d and d + 4, and
//     so do the query operands.  V: O^T's operand pairs two keys of one element.  A byte permutation of two keys'
//     words pairs their halves before the codes are taken apart, so V needs no transposition.
//   * Softmax statistics are float32.  A weight is 2^(score - ref), ref at least 11 below the largest score so far
//     when it was last moved and never more than 15 below any: weights stay below 2^15, ref (and with it every sum)
//     moves rarely, and as an f16 high part and remainder a weight is held to 2^-24, 2^-31 of the row's largest or
//     less.
//   * The rows of S^T are physical keys r ^ (r >> 1 & 1): with the four keys of a V load in different rows modulo
//     two, their shared-memory loads have half the bank conflicts, and K's none.
//
// Any byte stands for a finite number, so what lies behind a sequence's last key needs no cleaning: its weight is 0.
#include <type_traits>

#include "kv4.cuh"
#include "mma_common.cuh"
#include "sparse_common.cuh"

namespace pa {

using namespace mmac;

namespace {

constexpr int kStageKeys = 64;
constexpr float kRefBelow = 11.f, kRefMost = 15.f;

struct Kv4Params {
    SparseParams s;
    int S;         // CTAs of a cluster
    int TT, HT;    // tokens of a unit; head tiles of a kv head
    int seq_tiles; // tiles of every sequence: a uniform batch, or the short runs of a packed one (0: by rows of q)
};

// A unit's tokens: cnt of sequence b from its token i on; q0 the sequence's first row of q, n its tokens.
struct Tile {
    int b, n, i, cnt;
    long long q0;
};

// Packed batches: sequence b's tiles are q_start[b] / TT + b and on, which leaves room for all of them; with one
// token a tile they are its rows.
__device__ __forceinline__ Tile find_tile(const Kv4Params &p, int tile, int lane) {
    const FwdParams &f = p.s.f;
    Tile u{0, 0, 0, 0, 0};
    if (p.seq_tiles) {
        u.b = tile / p.seq_tiles;
        u.i = (tile - u.b * p.seq_tiles) * p.TT;
        if (!f.q_start) {
            u.n = f.Sq;
            u.q0 = (long long)u.b * f.Sq;
            u.cnt = min(p.TT, u.n - u.i);
            return u;
        }
    }
    auto key = [&](int b, int q) { return p.TT == 1 ? q : max(q, 0) / p.TT + b; };
    if (!p.seq_tiles) {
        int lo = 0, hi = f.B;  // key(lo) <= tile < key(hi)
        const int guess = min(p.TT == 1 ? tile : tile - tile / (p.TT + 1), f.B - 1);  // a token a sequence
        if (key(guess, __ldg(f.q_start + guess)) <= tile) {
            lo = guess;
            if (key(guess + 1, __ldg(f.q_start + guess + 1)) > tile) hi = lo + 1;
        } else {
            hi = max(guess, 1);
        }
        while (hi - lo > 1) {  // 31 borders a trip
            const int step = (hi - lo + 31) / 32;
            const int b = lo + (lane + 1) * step;
            const bool below = b < hi && key(b, __ldg(f.q_start + b)) <= tile;
            const int k = __popc(__ballot_sync(0xffffffffu, below));
            hi = min(hi, lo + (k + 1) * step);
            lo += k * step;
        }
        u.b = lo;
    }
    const int q0 = __ldg(f.q_start + u.b), q1 = __ldg(f.q_start + u.b + 1);
    if (q0 < 0 || q1 < q0 || q1 > p.s.n_tok) return u;
    u.q0 = q0;
    u.n = q1 - q0;
    if (!p.seq_tiles) u.i = (tile - key(u.b, q0)) * p.TT;
    if (u.i < 0 || (p.s.group_min && u.n >= p.s.group_min)) return u;  // malformed, or the other kernel's
    u.cnt = min(p.TT, u.n - u.i);
    return u;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
                 : "memory");
}

// Pages [pg0, pg_end) of row bt_row, kStageKeys keys a stage.  An id outside the pool is not followed: its block
// becomes zeros.
template <int NSTAGE>
__device__ __forceinline__ void produce(const FwdParams &p, const int32_t *bt_row, int kvh, int pg0, int pg_end,
                                        int n_tiles, int ps_shift, int block, uint32_t sbase, uint32_t bar_full,
                                        uint32_t bar_empty, int lane) {
    const int pps = kStageKeys >> ps_shift;
    const uint32_t stage_bytes = (uint32_t)(pps * block);
    const uint8_t *pool = static_cast<const uint8_t *>(p.k_cache);
    int batch = pg0;
    int id_cur = batch + lane < pg_end ? __ldg(bt_row + batch + lane) : 0;
    int id_next = batch + 32 + lane < pg_end ? __ldg(bt_row + batch + 32 + lane) : 0;
    bool bad = false;
    int issued = 0;
    for (int t = 0; t < n_tiles; ++t) {
        const int st = t % NSTAGE;
        if (t >= NSTAGE) {
            const bool ok = mbar_wait(bar_empty + 8 * st, ((t / NSTAGE) - 1) & 1, p.err);
            bad = __any_sync(0xffffffffu, !ok);
            if (bad) break;
        }
        const int first = pg0 + t * pps;
        if (first >= batch + 32) {
            batch += 32;
            id_cur = id_next;
            const int nx = batch + 32 + lane;
            id_next = nx < pg_end ? __ldg(bt_row + nx) : 0;
        }
        const int id = __shfl_sync(0xffffffffu, id_cur, (first + lane - batch) & 31);
        const bool mine = lane < min(pps, pg_end - first);
        const bool in_pool = id >= 0 && (long long)id < p.num_pages;
        const uint32_t dst = sbase + (uint32_t)st * stage_bytes + (uint32_t)(lane * block);
        const unsigned good = __ballot_sync(0xffffffffu, mine && in_pool);
        if (mine && !in_pool) {
            atomicOr(p.err, (unsigned int)PA_ERRBIT_PAGE_RANGE);
            for (int i = 0; i < block; i += 16)
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(dst + i), "r"(0) : "memory");
            fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(bar_full + 8 * st, (uint32_t)(__popc(good) * block));
        __syncwarp();
        if (mine && in_pool)
            bulk_load(dst, pool + ((long long)id * p.Hkv + kvh) * block, (uint32_t)block, bar_full + 8 * st);
        issued = t + 1;
    }
    // every copy must have landed before the CTA may exit
    for (int t = max(0, issued - NSTAGE); t < issued; ++t) mbar_wait(bar_full + 8 * (t % NSTAGE), (t / NSTAGE) & 1, p.err);
}

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
// bf16 rows are multiplied by a power of two that brings them into f16; inv is its inverse.
template <typename T, int D>
__device__ __forceinline__ void load_q(const T *row, bool valid, int tq, uint32_t (&w)[D / 8], float &inv) {
    const uint4 *src = reinterpret_cast<const uint4 *>(row + tq * (D / 4));
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        const uint4 x = valid ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
        w[4 * i] = __byte_perm(x.x, x.z, 0x5410);
        w[4 * i + 1] = __byte_perm(x.x, x.z, 0x7632);
        w[4 * i + 2] = __byte_perm(x.y, x.w, 0x5410);
        w[4 * i + 3] = __byte_perm(x.y, x.w, 0x7632);
    }
    inv = 1.f;
    if (std::is_same<T, __nv_bfloat16>::value) {
        float am = 0.f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
            am = fmaxf(am, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xffff0000u))));
        am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
        am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
        const float sc = f16_row_scale(am, inv);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) w[i] = bf16x2_to_f16x2_scaled(w[i], sc);
    }
}

template <typename T>
__device__ __forceinline__ void store4(T *o, float4 v) {
    uint2 w = make_uint2(MmaOp<T>::pack(v.x, v.y), MmaOp<T>::pack(v.z, v.w));
    *reinterpret_cast<uint2 *>(o) = w;
}

// Shared memory of the merge: rows [4 warps][R][D + 4], maxima and sums [4][R], then the CTA's own [R] each.
__host__ __device__ constexpr size_t merge_bytes(int D, int R) { return ((size_t)4 * R * (D + 4) + 10 * R) * 4; }

}  // namespace

template <typename T, int D, int NR, int NSTAGE, int MINB>
__global__ void __launch_bounds__(kMmaThreads, MINB) paged_attn_kv4_kernel(const Kv4Params p, int ps_shift) {
    using Op = MmaOp<__half>;
    constexpr int R = 8 * NR;
    constexpr int MT = D / 16;    // 16-wide head-dim tiles of O^T
    constexpr int KW = D / 32;    // words of a lane's part of a K row: D / 4 elements
    constexpr int VW = D / 64;    // words of a lane's part of a V row: D / 8 elements
    constexpr int KS = D / 64;    // K scales of a lane's part
    constexpr int VS = D == 256 ? 2 : 1;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t bars[2 * NSTAGE];
    const FwdParams &f = p.s.f;
    RangeCheck ranges(p.s);
    BehindFirst behind(p.s);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)(blockIdx.x % p.S);
    int unit = (int)(blockIdx.x / p.S);
    const int ht = unit % p.HT;
    unit /= p.HT;
    const int kvh = unit % f.Hkv;
    const Tile u = find_tile(p, unit / f.Hkv, lane);
    ranges.report(f);
    if (u.cnt <= 0) return;

    const int ps = 1 << ps_shift;
    const int block = kv4::block_bytes(ps, D);
    int L = max(__ldg(f.seq_lens + u.b), 0);
    if (L > f.W * ps) {  // never read past the sequence's block-table row
        if (threadIdx.x == 0) atomicOr(f.err, (unsigned int)PA_ERRBIT_SEQ_CLIPPED);
        L = f.W * ps;
    }
    // unit rows r = token x heads + head; the last token reaches furthest
    const int h0 = ht * R, heads = min(R, f.G - h0);
    const int rows = u.cnt * heads;
    auto row_index = [&](int r) { return (u.q0 + u.i + r / heads) * f.Hq + kvh * f.G + h0 + r % heads; };
    const int k_hi = row_key_limit(f, u.b, L, u.i + u.cnt - 1, u.n);
    if (k_hi <= 0) {
        if (rank == 0) {
            for (int i = threadIdx.x; i < rows * (D / 4); i += kMmaThreads)
                store4<T>(static_cast<T *>(f.out) + row_index(i / (D / 4)) * D + i % (D / 4) * 4, make_float4(0.f, 0.f, 0.f, 0.f));
            if (f.lse && threadIdx.x < rows) f.lse[row_index(threadIdx.x)] = kNegInf;
        }
        return;
    }
    // this CTA's share of the stages
    const int stages = (k_hi + kStageKeys - 1) / kStageKeys;
    const int share = (stages + p.S - 1) / p.S;
    const int s0 = min(rank * share, stages);
    const int n_tiles = min(share, stages - s0);
    const int k_lo = s0 * kStageKeys;

    const uint32_t sbase = smem_u32(smem);
    const uint32_t stage_bytes = (uint32_t)((kStageKeys >> ps_shift) * block);
    const uint32_t bar_full = smem_u32(&bars[0]), bar_empty = smem_u32(&bars[NSTAGE]);
    if (threadIdx.x == 0) {
        for (int st = 0; st < NSTAGE; ++st) {
            mbar_init(bar_full + 8 * st, 1);
            mbar_init(bar_empty + 8 * st, kMmaConsumerWarps);
        }
        fence_barrier_init();
    }
    __syncthreads();

    bool bad = false;
    float *sm = reinterpret_cast<float *>(smem);
    constexpr int STRIDE = D + 4;
    float *s_m = sm + 4 * R * STRIDE, *s_l = s_m + 4 * R, *s_cta = s_l + 4 * R;  // s_cta: [R] references, [R] sums
    if (warp == kMmaConsumerWarps) {
        const int pg_end = (min(k_hi, k_lo + n_tiles * kStageKeys) + ps - 1) >> ps_shift;
        produce<NSTAGE>(f, f.block_table + (long long)u.b * f.W, kvh, k_lo >> ps_shift, pg_end, n_tiles, ps_shift, block,
                        sbase, bar_full, bar_empty, lane);
    } else {
        const int g = lane >> 2, tq = lane & 3;
        const int kw0 = warp * 16;
        const int kg = g ^ ((g >> 1) & 1);  // this lane's K rows: keys kg and kg + 8
        const int va = (2 * tq) ^ (tq & 1), vb = (2 * tq + 1) ^ (tq & 1);  // V keys va, vb, va + 8, vb + 8
        uint32_t qb[NR][D / 8];
        float srow[NR][2];
        int lim[NR][2];
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            const int r = nr * 8 + g;
            const bool valid = r < rows;
            const T *q = static_cast<const T *>(f.q) + (valid ? q_row_offset(f, row_index(r)) : 0);
            float inv;
            load_q<T, D>(q, valid, tq, qb[nr], inv);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int rc = nr * 8 + 2 * tq + e;
                srow[nr][e] = 8.f * f.scale_log2 * __shfl_sync(0xffffffffu, inv, 4 * (2 * tq + e));
                lim[nr][e] = rc < rows ? row_key_limit(f, u.b, L, u.i + rc / heads, u.n) : 0;
            }
        }
        float ref[NR][2], l[NR][2], acc[NR][MT][4];
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            ref[nr][0] = ref[nr][1] = kNegInf;
            l[nr][0] = l[nr][1] = 0.f;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) acc[nr][mt][0] = acc[nr][mt][1] = acc[nr][mt][2] = acc[nr][mt][3] = 0.f;
        }
        // offsets of this lane's parts within a stage
        const uint32_t blk = (uint32_t)((kw0 >> ps_shift) * block);
        const int r0 = kw0 & (ps - 1);
        const kv4::Layout at{ps, D};
        const uint32_t k_off = blk + at.codes(0, r0 + kg) + tq * (D / 8);
        const uint32_t ks_off = blk + at.scales(0, r0 + kg) + tq * KS;
        const uint32_t v_off = blk + at.codes(1, r0) + g * (D / 16);
        const uint32_t vs_off = blk + at.scales(1, r0) + (D == 64 ? g >> 1 : g * VS);

        for (int t = 0; t < n_tiles; ++t) {
            const int st = t % NSTAGE;
            const uint32_t base = sbase + (uint32_t)st * stage_bytes;
            const int j0 = k_lo + t * kStageKeys + kw0 + kg;  // the position of this lane's first K row
            const bool active = k_lo + t * kStageKeys + kw0 < k_hi;  // warp-uniform
            {
                const bool ok = mbar_wait(bar_full + 8 * st, (t / NSTAGE) & 1, f.err);
                if (__any_sync(0xffffffffu, !ok)) {
                    bad = true;
                    break;
                }
            }
            uint32_t kw[2][KW], vw[4][VW], ksb[2], vsb[4];
            if (active) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    lds_words<KW>(base + k_off + i * 8 * (D / 2), kw[i]);
                    ksb[i] = lds_bytes<KS>(base + ks_off + i * 8 * (D / 16));
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = (i & 1 ? vb : va) + (i & 2 ? 8 : 0);
                    lds_words<VW>(base + v_off + key * (D / 2), vw[i]);
                    vsb[i] = lds_bytes<VS>(base + vs_off + key * (D / 16));
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_empty + 8 * st);  // the stage is in registers
            if (!active) continue;

            // ---- S^T = K Q^T
            float sc[NR][4];
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) sc[nr][0] = sc[nr][1] = sc[nr][2] = sc[nr][3] = 0.f;
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                uint32_t h[2][4];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    // the scale of word w: byte w / 2 of the lane's, in both halves
                    uint32_t s, c;
                    kv4::scale_pair(__byte_perm(ksb[i], 0, 0x4040 + (w / 2) * 0x0101), s, c);
                    kv4::unpack8(kw[i][w], s, c, h[i]);
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t a[4] = {h[0][2 * k], h[1][2 * k], h[0][2 * k + 1], h[1][2 * k + 1]};
#pragma unroll
                    for (int nr = 0; nr < NR; ++nr) Op::run(sc[nr], a, qb[nr][4 * w + 2 * k], qb[nr][4 * w + 2 * k + 1]);
                }
            }
            // ---- weights; a score more than kRefMost above its reference moves it
            uint32_t pb[NR][2][2];  // [row tile][high part / remainder][keys 0-7 / 8-15]
            bool over = false;
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    sc[nr][e] = j0 < lim[nr][e] ? sc[nr][e] * srow[nr][e] : kNegInf;
                    sc[nr][2 + e] = j0 + 8 < lim[nr][e] ? sc[nr][2 + e] * srow[nr][e] : kNegInf;
                    over |= fmaxf(sc[nr][e], sc[nr][2 + e]) > ref[nr][e] + kRefMost;
                }
            if (__any_sync(0xffffffffu, over)) {
#pragma unroll
                for (int nr = 0; nr < NR; ++nr) {
                    float al[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = fmaxf(sc[nr][e], sc[nr][2 + e]);
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                        const float next = fmaxf(ref[nr][e], mx - kRefBelow);
                        al[e] = next == kNegInf ? 1.f : fast_exp2(ref[nr][e] - next);  // a row without a key so far
                        ref[nr][e] = next;
                        l[nr][e] *= al[e];
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[nr][mt][i] *= al[i & 1];
                }
            }
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) {
                float w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float r = ref[nr][i & 1];
                    w[i] = fast_exp2(sc[nr][i] - (r == kNegInf ? 0.f : r));
                }
                l[nr][0] += w[0] + w[2];
                l[nr][1] += w[1] + w[3];
#pragma unroll
                for (int kh = 0; kh < 2; ++kh) {
                    const uint32_t hi = Op::pack(w[2 * kh], w[2 * kh + 1]);
                    const float2 x = Op::unpack(hi);
                    pb[nr][0][kh] = movmatrix_trans(hi);
                    pb[nr][1][kh] = movmatrix_trans(Op::pack(w[2 * kh] - x.x, w[2 * kh + 1] - x.y));
                }
            }
            // ---- O^T += V^T P^T
            uint32_t vs[2][VS], vc[2][VS];  // of the keys (va, vb) and (va + 8, vb + 8)
#pragma unroll
            for (int kh = 0; kh < 2; ++kh)
#pragma unroll
                for (int i = 0; i < VS; ++i)
                    kv4::scale_pair(__byte_perm(vsb[2 * kh], vsb[2 * kh + 1], 0x3430 + i * 0x0101), vs[kh][i], vc[kh][i]);
#pragma unroll
            for (int w = 0; w < VW; ++w)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t h[2][4];
#pragma unroll
                    for (int kh = 0; kh < 2; ++kh)
                        kv4::unpack8(__byte_perm(vw[2 * kh][w], vw[2 * kh + 1][w], half ? 0x7632 : 0x5410),
                                     vs[kh][w * VS / VW], vc[kh][w * VS / VW], h[kh]);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int mt = 4 * w + 2 * half + k;
                        const uint32_t a[4] = {h[0][2 * k], h[0][2 * k + 1], h[1][2 * k], h[1][2 * k + 1]};
#pragma unroll
                        for (int nr = 0; nr < NR; ++nr) {
                            Op::run(acc[nr][mt], a, pb[nr][0][0], pb[nr][0][1]);
                            Op::run(acc[nr][mt], a, pb[nr][1][0], pb[nr][1][1]);
                        }
                    }
                }
        }
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[nr][e] += __shfl_xor_sync(0xffffffffu, l[nr][e], 4);
                l[nr][e] += __shfl_xor_sync(0xffffffffu, l[nr][e], 8);
                l[nr][e] += __shfl_xor_sync(0xffffffffu, l[nr][e], 16);
            }
        // ---- the warps' states: tile mt's rows g and g + 8 are elements g D / 8 + 2 mt and the next
        named_bar_sync(1, kMmaConsumerWarps * 32);  // no warp reads the ring any more
        float *wa = sm + warp * R * STRIDE;
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    *reinterpret_cast<float2 *>(wa + (nr * 8 + 2 * tq + e) * STRIDE + g * (D / 8) + 2 * mt) =
                        make_float2(acc[nr][mt][e], acc[nr][mt][2 + e]);
            if (g == 0) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    s_m[warp * R + nr * 8 + 2 * tq + e] = ref[nr][e];
                    s_l[warp * R + nr * 8 + 2 * tq + e] = bad ? __uint_as_float(0x7fc00000u) : l[nr][e];
                }
            }
        }
        named_bar_sync(1, kMmaConsumerWarps * 32);
        for (int i = threadIdx.x; i < rows * (D / 4); i += kMmaConsumerWarps * 32) {
            const int r = i / (D / 4), c = i % (D / 4) * 4;
            float M = kNegInf;
#pragma unroll
            for (int w = 0; w < 4; ++w) M = fmaxf(M, s_m[w * R + r]);
            float sum = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float k = M == kNegInf ? 0.f : exp2f(s_m[w * R + r] - M);
                const float4 v = *reinterpret_cast<const float4 *>(sm + (w * R + r) * STRIDE + c);
                sum += k * s_l[w * R + r];
                o.x += k * v.x, o.y += k * v.y, o.z += k * v.z, o.w += k * v.w;
            }
            if (p.S == 1) {
                const float inv = sum != 0.f ? 8.f / sum : 0.f;  // a NaN stays one
                const long long ri = row_index(r);
                store4<T>(static_cast<T *>(f.out) + ri * D + c, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
                if (c == 0 && f.lse) f.lse[ri] = sum != 0.f ? M * kLn2 + logf(sum) : kNegInf;
            } else {  // the row's slot of warp 0 is this thread's alone
                *reinterpret_cast<float4 *>(sm + r * STRIDE + c) = o;
                if (c == 0) {
                    s_cta[r] = M;
                    s_cta[R + r] = sum;
                }
            }
        }
    }
    if (p.S == 1) return;
    // ---- the CTAs' states: each stores its share of the rows' elements
    cluster_barrier();
    for (int i = rank * kMmaThreads + threadIdx.x; i < rows * (D / 4); i += p.S * kMmaThreads) {
        const int r = i / (D / 4), c = i % (D / 4) * 4;
        const uint32_t at_m = smem_u32(s_cta + r), at_l = smem_u32(s_cta + R + r), at_o = smem_u32(sm + r * STRIDE + c);
        float M = kNegInf;
        for (int x = 0; x < p.S; ++x) M = fmaxf(M, peer_load(peer_addr(at_m, x)));
        float sum = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int x = 0; x < p.S; ++x) {
            const float k = M == kNegInf ? 0.f : exp2f(peer_load(peer_addr(at_m, x)) - M);
            const float4 v = peer_load4(peer_addr(at_o, x));
            sum += k * peer_load(peer_addr(at_l, x));
            o.x += k * v.x, o.y += k * v.y, o.z += k * v.z, o.w += k * v.w;
        }
        const float inv = sum != 0.f ? 8.f / sum : 0.f;  // a NaN stays one
        const long long ri = row_index(r);
        store4<T>(static_cast<T *>(f.out) + ri * D + c, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
        if (c == 0 && f.lse) f.lse[ri] = sum != 0.f ? M * kLn2 + logf(sum) : kNegInf;
    }
    cluster_barrier();  // the peers have read this CTA's memory
}

template <typename T, int D, int NR>
static cudaError_t launch_kv4(Kv4Params p, int sms, cudaStream_t stream) {
    constexpr int R = 8 * NR;
    constexpr int NSTAGE = D == 64 ? 8 : 4;
    constexpr int MINB = D == 256 ? 1 : NR == 1 ? 3 : 2;
    constexpr size_t ring = (size_t)NSTAGE * kStageKeys * D / 8 * 9;
    constexpr size_t smem = ring > merge_bytes(D, R) ? ring : merge_bytes(D, R);
    const FwdParams &f = p.s.f;
    p.HT = (f.G + R - 1) / R;
    p.TT = f.q_start && p.s.n_tok <= f.B ? 1 : f.G < R ? R / f.G : 1;
    long long tiles;
    if (!f.q_start) {
        p.seq_tiles = (f.Sq + p.TT - 1) / p.TT;
        tiles = (long long)f.B * p.seq_tiles;
    } else if (p.s.by_seq) {
        p.seq_tiles = (p.s.group_min - 1 + p.TT - 1) / p.TT;
        tiles = (long long)f.B * p.seq_tiles;
    } else {
        p.seq_tiles = 0;
        tiles = p.TT == 1 ? p.s.n_tok : p.s.n_tok / p.TT + f.B;
    }
    const long long units = tiles * f.Hkv * p.HT;
    int S = 1;
    while (S < 8 && units * S * 2 <= (long long)sms * MINB && (long long)f.W * f.ps >= 256ll * S) S *= 2;
    p.S = S;
    if (units == 0) return cudaSuccess;
    if (units * S > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    auto kern = paged_attn_kv4_kernel<T, D, NR, NSTAGE, MINB>;
    static SmemLimit limit;
    const cudaError_t e = limit.raise((const void *)kern, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(units * S));
    cfg.blockDim = dim3(kMmaThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    cfg.attrs = attr;
    cfg.numAttrs = second_launch_attrs(attr, S, p.s.group_min != 0);
    int sh = 0;
    while ((1 << sh) < f.ps) ++sh;
    return cudaLaunchKernelEx(&cfg, kern, p, sh);
}

template <typename T, int D>
static cudaError_t launch_kv4_d(const Kv4Params &p, int sms, cudaStream_t stream) {
    const FwdParams &f = p.s.f;
    // rows of an average sequence (a uniform batch: of every one)
    const double rows = (f.q_start ? (double)p.s.n_tok / f.B : (double)f.Sq) * f.G;
    if constexpr (D != 256) {
        if (rows > 8 && !(f.G > 16 && f.G <= 24)) return launch_kv4<T, D, 2>(p, sms, stream);
    }
    return launch_kv4<T, D, 1>(p, sms, stream);
}

template <typename T>
static cudaError_t launch_kv4_t(const Kv4Params &p, int sms, cudaStream_t stream) {
    if (p.s.f.D == 64) return launch_kv4_d<T, 64>(p, sms, stream);
    if (p.s.f.D == 128) return launch_kv4_d<T, 128>(p, sms, stream);
    return launch_kv4_d<T, 256>(p, sms, stream);
}

cudaError_t launch_kv4_mma(const SparseParams &sp, int dtype, int sms, cudaStream_t stream) {
    Kv4Params p{};
    p.s = sp;
    if (dtype == PA_BF16) return launch_kv4_t<__nv_bfloat16>(p, sms, stream);
    return launch_kv4_t<__half>(p, sms, stream);
}

}  // namespace pa
