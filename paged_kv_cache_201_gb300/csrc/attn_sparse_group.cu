// Attention over listed pages for runs of query tokens of one sequence (prompt chunks), bf16 / f16.
//
// Token by token, a chunk's lists are read once for each token: 936 tokens of 8 kv heads over 64 pages of 16
// (f16) move 3.9 GB through L2 at 8.7 TB/s, 451 us, although the lists of neighbouring tokens overlap.
// Here a CTA takes kGroupWarps x (16 / G) consecutive tokens of one kv head and walks the union of their
// lists, each page once:
//   * the lists become one token mask a logical page in shared memory, and its non-empty entries a page
//     list in ascending order;
//   * a producer warp streams the listed pages by TMA, as in the token kernel, into a ring of 64-key stages;
//   * each of the eight consumer warps owns 16 rows (16 / G tokens x G heads) and its own softmax state, and
//     skips the 16-key blocks that none of its tokens lists.  Rows of tokens that do not list a page, and
//     keys past a token's reach, get score -inf.
// A masked key's weight is 0, but 0 times an infinity or a NaN in V is a NaN.  Such values are rare, so no
// product is guarded: a CTA whose result is not finite, and one whose lists name a page twice (it counts
// twice), does its tokens again on CUDA cores, where a key that is not seen is not multiplied.
// P enters the second product as a 16-bit high part plus its remainder for bf16; f16 weights (2^-12 of
// themselves, below the output's own rounding) go in alone.
#include <float.h>

#include "mma_common.cuh"
#include "sparse_simt.cuh"
#include "sparse_tile.cuh"

namespace pa {

using namespace mmac;

namespace {

template <typename T>
struct IsBf16 {
    static constexpr bool value = false;
};
template <>
struct IsBf16<__nv_bfloat16> {
    static constexpr bool value = true;
};

constexpr int kGroupWarps = 8;
constexpr int kGroupAllWarps = kGroupWarps + 4;  // the producer's warpgroup: one warp of it works
constexpr int kGroupThreads = kGroupAllWarps * 32;
// Registers of a thread once the two kinds part: 8 warps x 232 + 4 x 24 are fewer than the launch's
// 12 x 168 (a scheduler holds three warps, which caps the launch there).
constexpr int kGroupConsumerRegs = 232, kGroupProducerRegs = 24;

}  // namespace

template <typename T, int D, int NSTAGE>
__global__ void __launch_bounds__(kGroupThreads, 1)
    paged_attn_sparse_group_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                                   const SparseParams sp, int ps_shift, int TPW) {
    using Op = MmaOp<T>;
    constexpr bool kSplitP = IsBf16<T>::value;
    constexpr int kStage = Geo<D>::kStageBytes;
    constexpr int kChunks = Geo<D>::kChunks;
    const FwdParams &p = sp.f;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[3 * NSTAGE];
    __shared__ int s_reach[kTileMaxTokens];
    __shared__ int s_count[kGroupAllWarps];
    __shared__ int s_redo;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ps = 1 << ps_shift;
    const int kvh = blockIdx.x % p.Hkv;
    const long long tile = blockIdx.x / p.Hkv;
    const int TPC = kGroupWarps * TPW;

    TokenTile x;
    if (!token_tile(sp, tile, TPC, x)) return;
    const int b = x.b, nt = x.nt, n_seq = x.n_seq, i0 = x.i0, L = x.L;
    const long long tok0 = x.tok0;
    if (tid < nt) s_reach[tid] = row_key_limit(p, b, L, i0 + tid, n_seq);
    const int reach_max = p.causal ? row_key_limit(p, b, L, i0 + nt - 1, n_seq) : L;  // grows with the token
    const int np = (reach_max + ps - 1) >> ps_shift;

    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    uint32_t *s_mask = reinterpret_cast<uint32_t *>(smem_raw + (sbase - raw) + NSTAGE * 2 * kStage);  // [W] tokens of a page
    int *s_list = reinterpret_cast<int *>(s_mask + p.W);                                              // [W]
    const uint32_t bar_fk = smem_u32(&bars[0]), bar_fv = smem_u32(&bars[NSTAGE]), bar_em = smem_u32(&bars[2 * NSTAGE]);
    if (tid == 0) {
        for (int i = 0; i < NSTAGE; ++i) {
            mbar_init(bar_fk + 8 * i, 1);
            mbar_init(bar_fv + 8 * i, 1);
            mbar_init(bar_em + 8 * i, kGroupWarps);
        }
        fence_barrier_init();
    }
    for (int j = tid; j < np; j += kGroupThreads) s_mask[j] = 0u;
    __syncthreads();

    int n_list = list_pages<kGroupAllWarps>(sp, x, kvh, ps_shift, np, s_reach, s_mask, s_count,
                                            [&](int i, int j) { s_list[i] = j; });
    if (tid == 0) s_redo = n_list < 0 ? 1 : 0;
    n_list = max(n_list, 0);
    __syncthreads();

    const int pps = kMmaTileKeys >> ps_shift;
    const int n_tiles = (n_list + pps - 1) / pps;
    bool bad = false;
    if (warp >= kGroupWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kGroupProducerRegs));
        if (warp != kGroupWarps) return;
        // ---------------------------------------------------------------- producer
        if (lane == 0) {
            tma_prefetch_desc(&tmK);
            tma_prefetch_desc(&tmV);
        }
        const uint32_t box_bytes = (uint32_t)(Geo<D>::NH * ps * 128);
        const int32_t *bt = p.block_table + (long long)b * p.W;
        auto entry = [&](int e) {  // first token of the entry's page, -ps for an id outside the pool
            const int id = e < n_list ? __ldg(bt + s_list[e]) : 0;
            if (id < 0 || id >= p.num_pages) {
                atomicOr(p.err, (unsigned int)PA_ERRBIT_PAGE_RANGE);
                return -ps;  // wholly out of the tensor: the box reads as zeros
            }
            return id << ps_shift;
        };
        int batch = 0, cur = entry(lane), nxt = entry(32 + lane);
        int issued = 0;
        for (int t = 0; t < n_tiles; ++t) {
            const int st = t % NSTAGE;
            if (t >= NSTAGE) {
                const bool ok = mbar_wait(bar_em + 8 * st, ((t / NSTAGE) - 1) & 1, p.err);
                bad = __any_sync(0xffffffffu, !ok);
                if (bad) break;
            }
            const int first = t * pps;
            if (first >= batch + 32) {
                batch += 32;
                cur = nxt;
                nxt = entry(batch + 32 + lane);
            }
            const int tok = __shfl_sync(0xffffffffu, cur, (first - batch + lane) & 31);
            const int nvalid = min(pps, n_list - first);
            if (lane == 0) {
                mbar_arrive_expect_tx(bar_fk + 8 * st, (uint32_t)nvalid * box_bytes);
                mbar_arrive_expect_tx(bar_fv + 8 * st, (uint32_t)nvalid * box_bytes);
            }
            __syncwarp();
            if (lane < nvalid) {
                const uint32_t dst = sbase + (uint32_t)(st * 2 * kStage) + (uint32_t)lane * box_bytes;
                tma_load_4d(dst, &tmK, bar_fk + 8 * st, 0, tok, 0, kvh);
                tma_load_4d(dst + kStage, &tmV, bar_fv + 8 * st, 0, tok, 0, kvh);
            }
            issued = t + 1;
        }
        // every copy must have landed before the ring is reused or the CTA exits
        for (int t = max(0, issued - NSTAGE); t < issued; ++t) {
            mbar_wait(bar_fk + 8 * (t % NSTAGE), (t / NSTAGE) & 1, p.err);
            mbar_wait(bar_fv + 8 * (t % NSTAGE), (t / NSTAGE) & 1, p.err);
        }
        return;
    }
    {
        // ---------------------------------------------------------------- consumers (no tile if `redo`)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kGroupConsumerRegs));
        const int g = lane >> 2, tq = lane & 3;
        const int G = p.G;
        // rows g and g + 8: token and head within the warp's TPW tokens
        const int ta = warp * TPW + g / G, tb = warp * TPW + (g + 8) / G;
        const bool va = g < TPW * G && ta < nt, vb = g + 8 < TPW * G && tb < nt;
        const long long rowa = (tok0 + ta) * p.Hq + (long long)kvh * G + g % G;
        const long long rowb = (tok0 + tb) * p.Hq + (long long)kvh * G + (g + 8) % G;
        const int lim_a = va ? s_reach[ta] : 0, lim_b = vb ? s_reach[tb] : 0;
        const uint32_t bit_a = va ? 1u << ta : 0u, bit_b = vb ? 1u << tb : 0u;
        const uint32_t warp_bits = (TPW == 32 ? 0xffffffffu : ((1u << TPW) - 1)) << (warp * TPW);
        const T *qa = static_cast<const T *>(p.q) + (va ? q_row_offset(p, rowa) : 0);
        const T *qb = static_cast<const T *>(p.q) + (vb ? q_row_offset(p, rowb) : 0);
        uint32_t qf[D / 16][4];
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const int c0 = kk * 16 + 2 * tq;
            qf[kk][0] = va ? __ldg(reinterpret_cast<const uint32_t *>(qa + c0)) : 0u;
            qf[kk][1] = vb ? __ldg(reinterpret_cast<const uint32_t *>(qb + c0)) : 0u;
            qf[kk][2] = va ? __ldg(reinterpret_cast<const uint32_t *>(qa + c0 + 8)) : 0u;
            qf[kk][3] = vb ? __ldg(reinterpret_cast<const uint32_t *>(qb + c0 + 8)) : 0u;
        }
        float m_a = kNegInf, m_b = kNegInf, l_a = 0.f, l_b = 0.f;
        float acc[D / 8][4];
#pragma unroll
        for (int n = 0; n < D / 8; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
        const int mi = lane >> 3, rr = lane & 7;
        // Shared-memory offsets of the operand loads within a block's rows: 16-byte chunk c of row r lies at
        // (c % 8) ^ (r % 8) of its 128-byte half row, and r % 8 is the lane's rr in every block.
        uint32_t xk[4], xv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            xk[i] = (uint32_t)(((2 * i + (mi & 1)) ^ rr) << 4);
            xv[i] = (uint32_t)(((2 * i + (mi >> 1)) ^ rr) << 4);
        }
        const int rk = rr + ((mi >> 1) << 3), rv = rr + ((mi & 1) << 3);  // the lane's row in a block
        const uint32_t half = (uint32_t)(ps << 7);                        // bytes of a page's half rows
        // every row of the warp sees keys below lim_min
        const int lim_min = (int)__reduce_min_sync(0xffffffffu, (unsigned)min(va ? lim_a : 0x7fffffff, vb ? lim_b : 0x7fffffff));

        for (int t = 0; t < n_tiles; ++t) {
            const int st = t % NSTAGE;
            const uint32_t par = (uint32_t)(t / NSTAGE) & 1;
            const uint32_t kbuf = sbase + (uint32_t)(st * 2 * kStage), vbuf = kbuf + kStage;
            // the stage's four 16-key blocks, one to a lane: logical position, and the tokens that list it
            const int e = t * pps + ((lane & 3) * 16 >> ps_shift);
            const int j = e < n_list ? s_list[e] : 0;
            uint32_t mask = e < n_list ? s_mask[j] : 0u;
            const int pos = (j << ps_shift) + ((lane & 3) * 16 & (ps - 1));
            if (pos >= reach_max) mask = 0u;
            unsigned act = __ballot_sync(0xffffffffu, lane < 4 && (mask & warp_bits));
            if (!bad) bad = __any_sync(0xffffffffu, !mbar_wait(bar_fk + 8 * st, par, p.err));
            if (!bad) bad = __any_sync(0xffffffffu, !mbar_wait(bar_fv + 8 * st, par, p.err));
            if (bad) act = 0;
            while (act) {
                // two blocks at a time (an odd last one beside itself, listed by no row)
                int c[2], ps_c[2];
                uint32_t mask_c[2];
                c[0] = __ffs((int)act) - 1;
                act &= act - 1;
                const bool two = act != 0;
                c[1] = two ? __ffs((int)act) - 1 : c[0];
                act &= act - 1;
                uint32_t row0[2];  // byte offset of the block's first row in a stage buffer
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    mask_c[i] = __shfl_sync(0xffffffffu, mask, c[i]);
                    ps_c[i] = __shfl_sync(0xffffffffu, pos, c[i]);
                    const int k0 = c[i] * 16, page = k0 >> ps_shift;
                    row0[i] = (uint32_t)(((page * Geo<D>::NH << ps_shift) + (k0 & (ps - 1))) << 7);
                }
                if (!two) mask_c[1] = 0u;
                float sc[2][2][4];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int n = 0; n < 2; ++n) sc[i][n][0] = sc[i][n][1] = sc[i][n][2] = sc[i][n][3] = 0.f;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t b0, b1, b2, b3;
                        ldmatrix_x4(kbuf + row0[i] + (rk << 7) + (kk >> 2) * half + xk[kk & 3], b0, b1, b2, b3);
                        Op::run(sc[i][0], qf[kk], b0, b1);
                        Op::run(sc[i][1], qf[kk], b2, b3);
                    }
                float mx_a = kNegInf, mx_b = kNegInf;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bool on_a = mask_c[i] & bit_a, on_b = mask_c[i] & bit_b;
                    if (ps_c[i] + 16 <= lim_min) {  // no key of the block is past a row's reach
                        const float off_a = on_a ? 0.f : kNegInf, off_b = on_b ? 0.f : kNegInf;
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            sc[i][n][0] = fmaf(sc[i][n][0], p.scale_log2, off_a);
                            sc[i][n][1] = fmaf(sc[i][n][1], p.scale_log2, off_a);
                            sc[i][n][2] = fmaf(sc[i][n][2], p.scale_log2, off_b);
                            sc[i][n][3] = fmaf(sc[i][n][3], p.scale_log2, off_b);
                        }
                    } else {
                        const int na = on_a ? lim_a - ps_c[i] : 0, nb = on_b ? lim_b - ps_c[i] : 0;
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            const int k0 = n * 8 + 2 * tq;
                            sc[i][n][0] = k0 < na ? sc[i][n][0] * p.scale_log2 : kNegInf;
                            sc[i][n][1] = k0 + 1 < na ? sc[i][n][1] * p.scale_log2 : kNegInf;
                            sc[i][n][2] = k0 < nb ? sc[i][n][2] * p.scale_log2 : kNegInf;
                            sc[i][n][3] = k0 + 1 < nb ? sc[i][n][3] * p.scale_log2 : kNegInf;
                        }
                    }
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        mx_a = fmaxf(mx_a, fmaxf(sc[i][n][0], sc[i][n][1]));
                        mx_b = fmaxf(mx_b, fmaxf(sc[i][n][2], sc[i][n][3]));
                    }
                }
                mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, 1));
                mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, 1));
                mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, 2));
                mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, 2));
                const float mn_a = fmaxf(m_a, mx_a), mn_b = fmaxf(m_b, mx_b);
                // -inf - (-inf) guard: a row whose scores are all -inf uses 0 as its offset
                const float mu_a = mn_a == kNegInf ? 0.f : mn_a, mu_b = mn_b == kNegInf ? 0.f : mn_b;
                if (__any_sync(0xffffffffu, mn_a != m_a || mn_b != m_b)) {
                    const float al_a = fast_exp2(m_a - mu_a), al_b = fast_exp2(m_b - mu_b);
                    l_a *= al_a;
                    l_b *= al_b;
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        acc[n][0] *= al_a;
                        acc[n][1] *= al_a;
                        acc[n][2] *= al_b;
                        acc[n][3] *= al_b;
                    }
                    m_a = mn_a;
                    m_b = mn_b;
                }
                uint32_t ph[2][4], pl[2][4];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const float p0 = fast_exp2(sc[i][n][0] - mu_a), p1 = fast_exp2(sc[i][n][1] - mu_a);
                        const float p2 = fast_exp2(sc[i][n][2] - mu_b), p3 = fast_exp2(sc[i][n][3] - mu_b);
                        l_a += p0 + p1;
                        l_b += p2 + p3;
                        ph[i][2 * n] = Op::pack(p0, p1);
                        ph[i][2 * n + 1] = Op::pack(p2, p3);
                        if (kSplitP) {
                            const float2 ha = Op::unpack(ph[i][2 * n]), hb = Op::unpack(ph[i][2 * n + 1]);
                            pl[i][2 * n] = Op::pack(p0 - ha.x, p1 - ha.y);
                            pl[i][2 * n + 1] = Op::pack(p2 - hb.x, p3 - hb.y);
                        }
                    }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int cnt = reach_max - ps_c[i];
                    if (cnt < 16) {
                        // keys past every token's reach hold any bits: every warp that reads them zeroes them
                        for (int idx = lane; idx < 16 * kChunks; idx += 32) {
                            const int key = idx / kChunks;
                            if (key >= cnt)
                                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                                                 kv_chunk_addr<D>(vbuf, c[i] * 16 + key, idx % kChunks, ps_shift)),
                                             "r"(0u)
                                             : "memory");
                        }
                        fence_proxy_async_smem();  // before the slot is written by TMA again
                        __syncwarp();
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)  // one block after the other: every sum rests between its products
#pragma unroll
                    for (int jj = 0; jj < D / 16; ++jj) {
                        uint32_t b0, b1, b2, b3;
                        ldmatrix_x4_trans(vbuf + row0[i] + (rv << 7) + (jj >> 2) * half + xv[jj & 3], b0, b1, b2, b3);
                        Op::run(acc[2 * jj], ph[i], b0, b1);
                        Op::run(acc[2 * jj + 1], ph[i], b2, b3);
                        if (kSplitP) {
                            Op::run(acc[2 * jj], pl[i], b0, b1);
                            Op::run(acc[2 * jj + 1], pl[i], b2, b3);
                        }
                    }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_em + 8 * st);
        }
        l_a += __shfl_xor_sync(0xffffffffu, l_a, 1);
        l_a += __shfl_xor_sync(0xffffffffu, l_a, 2);
        l_b += __shfl_xor_sync(0xffffffffu, l_b, 1);
        l_b += __shfl_xor_sync(0xffffffffu, l_b, 2);
        const float inv_a = l_a == 0.f ? 0.f : 1.f / l_a, inv_b = l_b == 0.f ? 0.f : 1.f / l_b;
        bool finite = (!va || l_a <= FLT_MAX) && (!vb || l_b <= FLT_MAX);
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
            finite = finite && (!va || (fabsf(acc[n][0]) <= FLT_MAX && fabsf(acc[n][1]) <= FLT_MAX)) &&
                     (!vb || (fabsf(acc[n][2]) <= FLT_MAX && fabsf(acc[n][3]) <= FLT_MAX));
            const int col = n * 8 + 2 * tq;
            if (va && !bad)
                *reinterpret_cast<uint32_t *>(static_cast<T *>(p.out) + rowa * D + col) = Op::pack(acc[n][0] * inv_a, acc[n][1] * inv_a);
            if (vb && !bad)
                *reinterpret_cast<uint32_t *>(static_cast<T *>(p.out) + rowb * D + col) = Op::pack(acc[n][2] * inv_b, acc[n][3] * inv_b);
        }
        if (p.lse && tq == 0 && !bad) {
            if (va) p.lse[rowa] = l_a == 0.f ? kNegInf : m_a * kLn2 + logf(l_a);
            if (vb) p.lse[rowb] = l_b == 0.f ? kNegInf : m_b * kLn2 + logf(l_b);
        }
        if (__any_sync(0xffffffffu, !finite && !bad) && lane == 0) s_redo = 1;
        if (__any_sync(0xffffffffu, bad) && lane == 0) s_redo = 2;  // timed out: the ring may still be written
    }
    named_bar_sync(1, kGroupWarps * 32);
    if (*(volatile int *)&s_redo != 1) return;
    // ---------------------------------------------------------------- again, on CUDA cores
    float *scratch = reinterpret_cast<float *>(smem_raw + (sbase - raw));
    static_assert(simt_scratch<D, 4, kGroupWarps>() * 4 <= NSTAGE * 2 * kStage, "the scratch must fit in the ring");
    for (int tok = 0; tok < nt; ++tok) {
        const TokenRow tr{b, s_reach[tok]};
        for (int hc = 0; hc * 4 < p.G; ++hc) {
            simt_token<T, D, 4, kGroupWarps>(sp, tr, tok0 + tok, kvh, hc, scratch, tid,
                                             [] { named_bar_sync(1, kGroupWarps * 32); });
            named_bar_sync(1, kGroupWarps * 32);  // before the scratch is used again
        }
    }
}

template <typename T, int D, int NSTAGE>
static cudaError_t launch_group_t(const SparseParams &sp, const CUtensorMap &tmk, const CUtensorMap &tmv,
                                  cudaStream_t stream) {
    const FwdParams &p = sp.f;
    auto kern = paged_attn_sparse_group_kernel<T, D, NSTAGE>;
    const size_t ring = mma_smem_bytes(D, NSTAGE);
    static SmemLimit limit;
    const cudaError_t e = limit.raise((const void *)kern, ring + (size_t)kSparseGroupMaxPages * 8);
    if (e != cudaSuccess) return e;
    int ps_shift = 0;
    while ((1 << ps_shift) < p.ps) ++ps_shift;
    const int TPW = sparse_group_tokens(p.G) / kGroupWarps, TPC = kGroupWarps * TPW;
    const long long units = count_tiles(sp, TPC) * p.Hkv;
    if (units > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    kern<<<(unsigned)units, kGroupThreads, ring + (size_t)p.W * 8, stream>>>(tmk, tmv, sp, ps_shift, TPW);
    return cudaGetLastError();
}

cudaError_t launch_sparse_group(const SparseParams &sp, int dtype, const CUtensorMap &tmk, const CUtensorMap &tmv,
                                cudaStream_t stream) {
    if (dtype == PA_BF16)
        return sp.f.D == 64 ? launch_group_t<__nv_bfloat16, 64, 4>(sp, tmk, tmv, stream)
                            : launch_group_t<__nv_bfloat16, 128, 4>(sp, tmk, tmv, stream);
    return sp.f.D == 64 ? launch_group_t<__half, 64, 4>(sp, tmk, tmv, stream)
                        : launch_group_t<__half, 128, 4>(sp, tmk, tmv, stream);
}

// Tokens of a CTA: eight warps of 16 / G tokens, at most 32 in all; 0 where the kernel does not apply.
int sparse_group_tokens(int G) {
    if (G < 1 || G > 16) return 0;
    const int per_warp = 16 / G;
    return kGroupWarps * (per_warp < kTileMaxTokens / kGroupWarps ? per_warp : kTileMaxTokens / kGroupWarps);
}

}  // namespace pa
