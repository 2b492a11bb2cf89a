// Attention over listed pages for runs of query tokens of one sequence, on the 5th-generation tensor cores
// (bf16 / f16, head_dim 64 or 128, up to 128 query heads to a kv head, scale > 0).
//
// A CTA takes up to 128 rows (TPC = min(32, 128 / G) consecutive tokens x the G heads of a kv head) and walks
// the union of the tokens' page lists, each page once, in 128-key tiles of 128 / page_size listed pages:
//   warp 0      loads the Q tile, then K pages by TMA into a two-slot ring; warp 2 the V pages
//   warp 1      issues tcgen05.mma: S = Q K^T into one of two S buffers of tensor memory (128 float32
//               columns), then O += P V with P read from tensor memory; P V of a tile is issued behind
//               Q K^T of the next one
//   warp 3      clears the V rows of the last tile that hold no key of the sequence (any bits)
//   warps 4-11  softmax, two threads to a row, 64 columns each: a 16-key block counts for a row if the row's
//               token lists its page (one bit), so its offset in exp2(s c + off) is the negated maximum or
//               -inf: the mask costs no instruction for a key.  A block that no token of the warp's rows
//               lists is passed by, its P 0.  O is rescaled in tensor memory only when the
//               maximum has grown by a few powers of two (struct Scaling).  P is written over S as 16-bit
//               pairs, high part and remainder (two products): 2^-16 of itself for bf16, 2^-22 for f16 down to
//               its quantum.  At the end they scale the rows by their sums and store them.
// A masked key's weight is 0, but 0 times an infinity or a NaN in V is a NaN.  Such values are rare, so no
// product is guarded: a CTA whose result is not finite, and one whose lists name a page twice (it counts
// twice), does its tokens again on CUDA cores, where a key that is not seen is not multiplied.
// The products run over all rows of every listed page, whoever lists it: at random lists (64 of some 400
// pages a token, 32 tokens, G = 4) six times what the lists ask for, at 1.15 us a tile (head_dim 128).  936
// such tokens of 8 kv heads take 145 us in either type; read token by token their lists move 3.9 GB through L2,
// 451 us.  Lists that overlap more cost less here.
// What bounds it: the softmax's chain (131 us in f16, 124 in bf16, without loads and products), before the
// products (110 alone) and the pages' way from L2 (890 MB, 99 alone).  With f16 weights of one part, 11 bits,
// f16 took 127 us, 5 % further from the exact result.  Sixty-four tokens a CTA, two tiles of rows over the
// same pages, halve the loads, but leave a thread a whole row: 131 us then.
#include <float.h>

#include <type_traits>

#include "sparse_simt.cuh"
#include "sparse_tile.cuh"
#include "tc05.cuh"

namespace pa {

namespace {

constexpr int kSt5Threads = 384, kSt5Warps = kSt5Threads / 32;
// Registers once the roles part: 128 x 64 + 256 x 208 are fewer than the launch's 384 x 168.
constexpr uint32_t kSt5LoadRegs = 64, kSt5SoftmaxRegs = 208;
constexpr int kSt5Half = 128 * 128;    // bytes of one 64-column half of a 128-row tile
constexpr uint32_t kSt5ColO = 256;

// A row's weights are p = exp2(s c - m), m its maximum less kTop, and O is rescaled only when the maximum has
// grown by more than kGrow powers of two: the largest p lies in [2^kTop, 2^(kTop + kGrow)].  bf16 has float32's
// exponents.  f16 has a quantum of 2^-24 and ends at 2^16, so there the weights are moved up: those down to
// 2^-24 of a row's largest keep 11 bits in the pair, and none loses more than 2^-35 of the largest.  A smaller
// kGrow would move them further up, but 936 tokens that take 145 us with 5 (and with 8) take 155 with 3.
template <typename T>
struct Scaling {
    static constexpr float kTop = 0.f, kGrow = 8.f;
};
template <>
struct Scaling<__half> {
    static constexpr float kTop = 10.f, kGrow = 5.f;
};

enum { S_QF = 0, S_KF = 1, S_KE = 3, S_VF = 5, S_VE = 7, S_PF = 9, S_COUNT = 11 };

// One listed page of the union: its logical index and the tokens that list it.
struct Listed {
    int j;
    uint32_t tokens;
};

// Two float32 operations an instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// P for 32 keys of one row, two 16-key blocks with their own offsets: p = exp2(s c + off[block]); the sums of
// the p go to l, the 32 columns at taddr receive [16 of high parts | 16 of remainders], 16-bit pairs.  any:
// whether a row of the warp has the block listed; its P is 0 if not.
template <typename T>
__device__ __forceinline__ void block_exp(const uint32_t (&u)[32], float c, const float (&off)[2], const bool (&any)[2],
                                          float2 &l, uint32_t taddr) {
    uint32_t hi[16], lo[16];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        if (any[b]) {
#pragma unroll
            for (int i = 8 * b; i < 8 * b + 8; ++i) {
                const float2 x = fma2(make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1])),
                                      make_float2(c, c), make_float2(off[b], off[b]));
                const float p0 = fast_exp2(x.x), p1 = fast_exp2(x.y);
                l = add2(l, make_float2(p0, p1));
                if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                    // the high parts truncated to their top 16 bits; p - high is then exact in float32 and below
                    // 2^-7 p, and its bf16 rounding leaves P within 2^-16 of p
                    hi[i] = __byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x7632);
                    lo[i] = MmaOp<T>::pack(p0 - __uint_as_float(__float_as_uint(p0) & 0xffff0000u),
                                           p1 - __uint_as_float(__float_as_uint(p1) & 0xffff0000u));
                } else {
                    // rounded to nearest, the remainder exact before its own rounding: within 2^-22 of p, or 2^-25
                    hi[i] = MmaOp<T>::pack(p0, p1);
                    const float2 h = MmaOp<T>::unpack(hi[i]);
                    lo[i] = MmaOp<T>::pack(p0 - h.x, p1 - h.y);
                }
            }
        } else {
#pragma unroll
            for (int i = 8 * b; i < 8 * b + 8; ++i) hi[i] = lo[i] = 0u;
        }
    }
    tc05::st_16cols(taddr, hi);
    tc05::st_16cols(taddr + 16u, lo);
}

}  // namespace

template <typename T, int D>
__global__ void __launch_bounds__(kSt5Threads, 1)
    paged_attn_sparse_tc05_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                                  const __grid_constant__ CUtensorMap tmV, const SparseParams sp, int ps_shift,
                                  int TPC, uint32_t idesc_qk, uint32_t idesc_pv) {
    constexpr int NH = D / 64, kTile = NH * kSt5Half;  // a tile of Q, K or V: NH 64-column halves
    const FwdParams &p = sp.f;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[S_COUNT];
    __shared__ uint32_t s_tmem;
    __shared__ float s_xmax[2][2][128];  // [tile parity][column half][row] partial maxima
    __shared__ float s_lsum[2][128];     // [column half][row] partial sums
    __shared__ int s_reach[kTileMaxTokens], s_count[kSt5Warps], s_redo;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ps = 1 << ps_shift;
    const int kvh = blockIdx.x % p.Hkv;
    TokenTile x;
    let_second_start();
    RangeCheck ranges(sp);
    const bool here = token_tile(sp, blockIdx.x / p.Hkv, TPC, x);
    ranges.report(p);
    if (!here) return;
    if (tid < x.nt) s_reach[tid] = row_key_limit(p, x.b, x.L, x.i0 + tid, x.n_seq);
    const int reach_max = row_key_limit(p, x.b, x.L, x.i0 + x.nt - 1, x.n_seq);  // grows with the token
    const int reach_min = row_key_limit(p, x.b, x.L, x.i0, x.n_seq);
    const int np = (reach_max + ps - 1) >> ps_shift;

    // shared memory: Q | K x2 | V x2 (128-row tiles of swizzled 64-column halves), list, masks
    const uint32_t raw = smem_u32(smem_raw), sbase = (raw + 1023u) & ~1023u;
    const uint32_t sQ = sbase;
    auto sK = [&](int s) { return sbase + (uint32_t)kTile * (1u + (uint32_t)s); };
    auto sV = [&](int s) { return sbase + (uint32_t)kTile * (3u + (uint32_t)s); };
    Listed *s_list = reinterpret_cast<Listed *>(smem_raw + (sbase - raw) + 5 * kTile);  // [W]
    uint32_t *s_mask = reinterpret_cast<uint32_t *>(s_list + p.W);                         // [W]
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    if (tid == 0) {
        mbar_init(bar(S_QF), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(S_KF + i), 1);
            mbar_init(bar(S_KE + i), 1);
            mbar_init(bar(S_VF + i), 1);
            mbar_init(bar(S_VE + i), 1);
            mbar_init(bar(S_PF + i), 8 + 1);
        }
        fence_barrier_init();
    }
    for (int j = tid; j < np; j += kSt5Threads) s_mask[j] = 0u;
    if (warp == 1) {
        tc05::tmem_alloc(smem_u32(&s_tmem), 512);
        tc05::tmem_relinquish();
    }
    tc05::fence_before_sync();
    __syncthreads();
    tc05::fence_after_sync();
    const uint32_t tmem = s_tmem;
    int n_list = list_pages<kSt5Warps>(sp, x, kvh, ps_shift, np, s_reach, s_mask, s_count,
                                       [&](int i, int j) { s_list[i] = {j, s_mask[j]}; });
    if (tid == 0) s_redo = n_list < 0 ? 1 : 0;
    n_list = max(n_list, 0);
    __syncthreads();
    const int ppt = 128 >> ps_shift;  // listed pages of a tile
    const int n_tiles = (n_list + ppt - 1) / ppt;

    if (warp < 4) {
        tc05::setmaxnreg_dec<kSt5LoadRegs>();
        bool bad = false;
        if (warp == 0 || warp == 2) {
            // ---------------------------------------------------------------- TMA: Q and K, or V
            const bool kq = warp == 0;
            const CUtensorMap *tm = kq ? &tmK : &tmV;
            const int b_full = kq ? S_KF : S_VF, b_empty = kq ? S_KE : S_VE;
            if (lane == 0) {
                tma_prefetch_desc(tm);
                if (kq && n_tiles > 0) {
                    tma_prefetch_desc(&tmQ);
                    mbar_arrive_expect_tx(bar(S_QF), (uint32_t)(NH * TPC * p.G * 128));
#pragma unroll
                    for (int h = 0; h < NH; ++h)
                        tma_load_4d(sQ + (uint32_t)h * kSt5Half, &tmQ, bar(S_QF), 0, h, kvh * p.G, (int)x.tok0);
                }
            }
            const uint32_t box = (uint32_t)ps * 128u;
            const int32_t *bt = p.block_table + (long long)x.b * p.W;
            auto entry = [&](int e) {  // first token of the entry's page, -ps for an id outside the pool
                const int id = e < n_list ? __ldg(bt + s_list[e].j) : 0;
                if (id < 0 || id >= p.num_pages) {
                    atomicOr(p.err, (unsigned int)PA_ERRBIT_PAGE_RANGE);
                    return -ps;  // wholly out of the tensor: the box reads as zeros
                }
                return id << ps_shift;
            };
            int batch = 0, cur = entry(lane), nxt = entry(32 + lane), issued = 0;
            for (int t = 0; t < n_tiles; ++t) {
                const int slot = t & 1, first = t * ppt;
                if (first >= batch + 32) {
                    batch += 32;
                    cur = nxt;
                    nxt = entry(batch + 32 + lane);
                }
                const int tok = __shfl_sync(0xffffffffu, cur, (first + lane / NH - batch) & 31);
                const int nvalid = min(ppt, n_list - first);
                if (t >= 2) {
                    const bool ok = mbar_wait(bar(b_empty + slot), ((t >> 1) - 1) & 1, p.err);
                    bad = __any_sync(0xffffffffu, !ok);
                    if (bad) break;
                }
                if (lane == 0) mbar_arrive_expect_tx(bar(b_full + slot), (uint32_t)nvalid * (uint32_t)NH * box);
                __syncwarp();
                if (lane / NH < nvalid)
                    tma_load_4d((kq ? sK(slot) : sV(slot)) + (uint32_t)(lane % NH * kSt5Half) + (uint32_t)(lane / NH) * box, tm,
                                bar(b_full + slot), 0, tok, lane % NH, kvh);
                issued = t + 1;
            }
            // no copy may outlive the CTA
            for (int t = max(0, issued - 2); t < issued; ++t) mbar_wait(bar(b_full + (t & 1)), (t >> 1) & 1, p.err);
            if (kq && n_tiles > 0) mbar_wait(bar(S_QF), 0, p.err);
        } else if (warp == 1) {
            // ---------------------------------------------------------------- products
            // The whole warp runs this, its values the same in every lane as the compiler can see, and one lane issues:
            // the operands then live in uniform registers (with one lane's own, an instruction took 60 cycles).
            auto same = [](auto v) { return __shfl_sync(0xffffffffu, v, 0); };
            const int nt = same(n_tiles);
            const uint32_t tm = same(tmem);
            if (nt > 0) {
                const bool leader = tc05::elect_one();
                const uint32_t dhi = tc05::smem_desc_sw128_hi(1024);
                const uint32_t dq = tc05::smem_desc_sw128_lo(sQ, 16);
                const uint32_t dk0 = tc05::smem_desc_sw128_lo(sK(0), 16), dk1 = tc05::smem_desc_sw128_lo(sK(1), 16);
                const uint32_t dv0 = tc05::smem_desc_sw128_lo(sV(0), (uint32_t)kSt5Half);
                const uint32_t dv1 = tc05::smem_desc_sw128_lo(sV(1), (uint32_t)kSt5Half);
                bad = !mbar_wait(bar(S_QF), 0, p.err);
                // Q K^T of tile t, then P V of the tile before
                for (int t = 0; t <= nt; ++t) {
                    if (t < nt) {
                        const int slot = t & 1;
                        bad = bad || !mbar_wait(bar(S_KF + slot), (t >> 1) & 1, p.err);
                        if (__any_sync(0xffffffffu, bad)) break;
                        tc05::fence_after_sync();
                        const uint32_t d = tm + (slot ? 128u : 0u), dk = slot ? dk1 : dk0;
                        if (leader) {
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                // columns 16 kk .. + 15: 64-column half kk / 4, 32-byte slice kk % 4 of its rows
                                const uint32_t off = ((uint32_t)(kk >> 2) * kSt5Half + (uint32_t)(kk & 3) * 32u) >> 4;
                                tc05::mma_ss_lh(d, dq + off, dhi, dk + off, dhi, idesc_qk, kk > 0 ? 1u : 0u);
                            }
                            tc05::commit(bar(S_KE + slot));  // K slot free, S holds the scores
                        }
                    }
                    if (t > 0) {
                        const int slot = (t - 1) & 1;
                        bad = !mbar_wait(bar(S_PF + slot), ((t - 1) >> 1) & 1, p.err);  // P there, V cleared
                        if (__any_sync(0xffffffffu, bad)) break;
                        tc05::fence_after_sync();
                        const uint32_t pcol = tm + (slot ? 128u : 0u), dv = slot ? dv1 : dv0;
                        if (leader) {
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk) {
                                // keys 16 kk .. + 15: half kk & 1 of 32-key chunk kk / 2, high parts at + 0,
                                // remainders at + 16
                                const uint32_t vlo = dv + (uint32_t)kk * (2048u >> 4);
                                const uint32_t pa = pcol + 32u * (uint32_t)(kk >> 1) + 8u * (uint32_t)(kk & 1);
                                tc05::mma_ts_lh(tm + kSt5ColO, pa, vlo, dhi, idesc_pv, (t > 1 || kk > 0) ? 1u : 0u);
                                tc05::mma_ts_lh(tm + kSt5ColO, pa + 16u, vlo, dhi, idesc_pv, 1u);
                            }
                            tc05::commit(bar(S_VE + slot));  // V slot free, O holds this tile's product
                        }
                    }
                }
            }
            __syncwarp();
        } else {
            // ---------------------------------------------------------------- V rows without a key
            for (int t = 0; t < n_tiles; ++t) {
                const int slot = t & 1;
                if (!bad) bad = __any_sync(0xffffffffu, !mbar_wait(bar(S_VF + slot), (t >> 1) & 1, p.err));
                if (!bad && t == n_tiles - 1) {
                    // only the list's last page can reach past the last token's keys
                    const int in_tile = n_list - 1 - t * ppt;
                    const int z0 = in_tile * ps + min(ps, reach_max - (s_list[n_list - 1].j << ps_shift));
                    for (int i = lane; i < (128 - z0) * 8 * NH; i += 32) {
                        const int c = i >> 3;  // 128-byte row half
                        const uint32_t a = sV(slot) + (uint32_t)(c % NH) * kSt5Half + (uint32_t)(z0 + c / NH) * 128u +
                                           16u * (uint32_t)(i & 7);
                        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(a), "r"(0u) : "memory");
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(S_PF + slot));
            }
        }
    } else {
        // -------------------------------------------------------------------- softmax and output
        tc05::setmaxnreg_inc<kSt5SoftmaxRegs>();
        const int hh = (warp >> 2) - 1;  // keys 64 hh .. + 63 of a tile
        const int r = (warp & 3) * 32 + lane;
        const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
        const int tk = r / p.G;
        const bool row_valid = tk < x.nt;  // at most TPC tokens, TPC G <= 128
        const int lim = row_valid ? s_reach[tk] : 0;
        const uint32_t bit = row_valid ? 1u << tk : 0u;
        // those of the warp's rows
        const int w0 = (warp & 3) * 32 / p.G, w1 = min((warp & 3) * 32 + 31, TPC * p.G - 1) / p.G;
        const uint32_t warp_bits = w1 < w0 ? 0u : (w1 >= 31 ? 0xffffffffu : (2u << w1) - 1u) & ~((1u << w0) - 1u);
        const float c2 = p.scale_log2;
        bool bad = false;
        float m_used = kNegInf;
        float2 l2 = make_float2(0.f, 0.f);  // sums of even and odd keys
        // the pages of a tile's four 16-key blocks, one tile ahead
        Listed page[4];
        auto look_up = [&](int t) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = t * ppt + ((64 * hh + 16 * i) >> ps_shift);
                page[i] = e < n_list ? s_list[e] : Listed{-1, 0u};
            }
        };
        look_up(0);
        for (int t = 0; t < n_tiles; ++t) {
            const int st = t & 1;
            // this row's four 16-key blocks: listed by its token, by any of the warp's
            bool on[4], any[4];
            int nv[4];  // keys of the block that the token sees
            int end = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int pos = (page[i].j << ps_shift) + ((64 * hh + 16 * i) & (ps - 1));
                on[i] = page[i].tokens & bit;
                any[i] = page[i].tokens & warp_bits;
                nv[i] = on[i] ? lim - pos : 0;
                end = max(end, page[i].j >= 0 ? pos + 16 : 0x7fffffff);
            }
            if (!bad) bad = !mbar_wait(bar(S_KE + st), (t >> 1) & 1, p.err);
            __syncwarp();
            tc05::fence_after_sync();
            const uint32_t sbuf = tmem + lane_addr + (st ? 128u : 0u) + 64u * (uint32_t)hh;
            uint32_t ua[32], ub[32];
            float mx = kNegInf;
            tc05::ld_32cols(sbuf, ua);
            tc05::ld_32cols(sbuf + 32u, ub);
            tc05::wait_ld();
            {
                if (end > reach_min) {  // some key is past some token's reach, or was never loaded
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        if (j >= nv[0]) ua[j] = 0xff800000u;
                        if (j >= nv[1]) ua[16 + j] = 0xff800000u;
                        if (j >= nv[2]) ub[j] = 0xff800000u;
                        if (j >= nv[3]) ub[16 + j] = 0xff800000u;
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (!any[i]) continue;
                    const uint32_t(&u)[32] = i < 2 ? ua : ub;
                    float a = __uint_as_float(u[(i & 1) * 16]), b = __uint_as_float(u[(i & 1) * 16 + 1]);
#pragma unroll
                    for (int j = 2; j < 16; j += 2) {
                        a = fmaxf(a, __uint_as_float(u[(i & 1) * 16 + j]));
                        b = fmaxf(b, __uint_as_float(u[(i & 1) * 16 + j + 1]));
                    }
                    if (on[i]) mx = fmaxf(mx, fmaxf(a, b));
                }
            }
            s_xmax[st][hh][r] = mx;
            look_up(t + 1);
            named_bar_sync(1, 256);
            mx = fmaxf(mx, s_xmax[st][hh ^ 1][r]);
            const float m_new = fmaxf(m_used, mx * c2 - Scaling<T>::kTop);
            const bool need = m_new > m_used + Scaling<T>::kGrow;  // also when m_used is -inf and m_new is not
            if (__any_sync(0xffffffffu, need || bad) && !(bad = __any_sync(0xffffffffu, bad))) {
                const float alpha = need ? exp2f(m_used - m_new) : 1.f;
                if (need) {
                    l2.x *= alpha;
                    l2.y *= alpha;
                    m_used = m_new;
                }
                if (t > 0) {
                    bad = __any_sync(0xffffffffu, !mbar_wait(bar(S_VE + ((t - 1) & 1)), ((t - 1) >> 1) & 1, p.err));
                    if (!bad) {
                        tc05::fence_after_sync();
#pragma unroll 1
                        for (int c = NH * hh; c < NH * hh + NH; ++c) {
                            uint32_t o[32];
                            tc05::ld_32cols(tmem + lane_addr + kSt5ColO + 32u * c, o);
                            tc05::wait_ld();
#pragma unroll
                            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
                            tc05::st_32cols(tmem + lane_addr + kSt5ColO + 32u * c, o);
                        }
                    }
                }
            }
            if (!bad) {
                const float nmu = m_used == kNegInf ? 0.f : -m_used;  // -inf - (-inf) guard
                const float oa[2] = {on[0] ? nmu : kNegInf, on[1] ? nmu : kNegInf};
                const float ob[2] = {on[2] ? nmu : kNegInf, on[3] ? nmu : kNegInf};
                const bool na[2] = {any[0], any[1]}, nb[2] = {any[2], any[3]};
                block_exp<T>(ua, c2, oa, na, l2, sbuf);
                block_exp<T>(ub, c2, ob, nb, l2, sbuf + 32u);
                tc05::wait_st();
            }
            tc05::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(S_PF + st));
        }
        // the row's sum, then its half of the columns
        s_lsum[hh][r] = l2.x + l2.y;
        named_bar_sync(1, 256);
        const float l = s_lsum[0][r] + s_lsum[1][r];
        if (!bad && n_tiles > 0)
            bad = __any_sync(0xffffffffu, !mbar_wait(bar(S_VE + ((n_tiles - 1) & 1)), ((n_tiles - 1) >> 1) & 1, p.err));
        tc05::fence_after_sync();
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const long long row = (x.tok0 + tk) * p.Hq + (long long)kvh * p.G + (r - tk * p.G);
        bool finite = l <= FLT_MAX;
        if (!bad) {
#pragma unroll 1
            for (int c = NH * hh; c < NH * hh + NH; ++c) {
                uint32_t o[32];
                if (n_tiles > 0) {
                    tc05::ld_32cols(tmem + lane_addr + kSt5ColO + 32u * c, o);
                    tc05::wait_ld();
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = 0u;
                }
#pragma unroll
                for (int j = 0; j < 32; ++j) finite = finite && fabsf(__uint_as_float(o[j])) <= FLT_MAX;
                if (row_valid) {
                    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<T *>(p.out) + row * D + 32 * c);
                    auto pk = [&](int i) {
                        return MmaOp<T>::pack(__uint_as_float(o[i]) * inv, __uint_as_float(o[i + 1]) * inv);
                    };
#pragma unroll
                    for (int j = 0; j < 4; ++j) dst[j] = make_uint4(pk(8 * j), pk(8 * j + 2), pk(8 * j + 4), pk(8 * j + 6));
                }
            }
            if (row_valid && hh == 0 && p.lse) p.lse[row] = l == 0.f ? kNegInf : m_used * kLn2 + logf(l);
            if (__any_sync(0xffffffffu, row_valid && !finite) && lane == 0) atomicOr(&s_redo, 1);
        } else if (lane == 0) {
            atomicOr(&s_redo, 2);  // timed out: the ring may still be written
        }
        named_bar_sync(1, 256);
        if (*(volatile int *)&s_redo == 1) {
            // ---------------------------------------------------------------- again, on CUDA cores
            float *scratch = reinterpret_cast<float *>(smem_raw + (sbase - raw));
            static_assert(simt_scratch<D, 4, 8>() * 4 <= 5 * kTile, "the scratch must fit in the tiles");
            for (int tok = 0; tok < x.nt; ++tok) {
                const TokenRow tr{x.b, s_reach[tok]};
                for (int hc = 0; hc * 4 < p.G; ++hc) {
                    simt_token<T, D, 4, 8, 1, false>(sp, tr, x.tok0 + tok, kvh, hc, scratch, tid - 128, 0, 1,
                                             [] { named_bar_sync(1, 256); });
                    named_bar_sync(1, 256);  // before the scratch is used again
                }
            }
        }
    }
    tc05::fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc05::fence_after_sync();
        tc05::tmem_dealloc(tmem, 512);
    }
}

template <typename T, int D>
static cudaError_t launch_st5(const SparseParams &sp, const CUtensorMap &tmq, const CUtensorMap &tmk,
                              const CUtensorMap &tmv, cudaStream_t stream) {
    const FwdParams &p = sp.f;
    auto kern = paged_attn_sparse_tc05_kernel<T, D>;
    const size_t tiles_bytes = 5 * (D / 64) * kSt5Half + 1024;
    static SmemLimit limit;
    cudaError_t e = limit.raise((const void *)kern, tiles_bytes + (size_t)kSparseTc05MaxPages * 12);
    if (e != cudaSuccess) return e;
    // The softmax warps' register increase is served from what the launch holds: a build that gave the
    // kernel fewer registers a thread would leave them waiting, so it is refused.
    static std::atomic<int> launch_regs{0};
    int regs = launch_regs.load(std::memory_order_relaxed);
    if (!regs) {
        cudaFuncAttributes fa;
        if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
        regs = fa.numRegs;
        launch_regs.store(regs, std::memory_order_relaxed);
    }
    if (regs * kSt5Threads < 128 * (int)kSt5LoadRegs + 256 * (int)kSt5SoftmaxRegs) return cudaErrorInvalidConfiguration;
    int ps_shift = 0;
    while ((1 << ps_shift) < p.ps) ++ps_shift;
    const int TPC = sparse_tile_tokens(p.G);
    const long long units = count_tiles(sp, TPC) * p.Hkv;
    if (units > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const bool bf = std::is_same<T, __nv_bfloat16>::value;
    kern<<<(unsigned)units, kSt5Threads, tiles_bytes + (size_t)p.W * 12, stream>>>(
        tmq, tmk, tmv, sp, ps_shift, TPC, tc05::idesc_f16(bf, false, 128, 128), tc05::idesc_f16(bf, true, 128, D));
    return cudaGetLastError();
}

int sparse_tile_tokens(int G) { return G > 128 ? 0 : 128 / G < kTileMaxTokens ? 128 / G : kTileMaxTokens; }

cudaError_t launch_sparse_tc05(const SparseParams &sp, int dtype, const CUtensorMap &tmq, const CUtensorMap &tmk,
                               const CUtensorMap &tmv, cudaStream_t stream) {
    if (dtype == PA_BF16)
        return sp.f.D == 64 ? launch_st5<__nv_bfloat16, 64>(sp, tmq, tmk, tmv, stream)
                            : launch_st5<__nv_bfloat16, 128>(sp, tmq, tmk, tmv, stream);
    return sp.f.D == 64 ? launch_st5<__half, 64>(sp, tmq, tmk, tmv, stream)
                        : launch_st5<__half, 128>(sp, tmq, tmk, tmv, stream);
}

}  // namespace pa
