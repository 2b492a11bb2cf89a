// Attention over listed pages on tensor cores (bf16 / f16).
//
// One cluster of S CTAs = one (query token, kv head, tile of 16 query heads); CTA s of it takes the
// s-th part of the token's page list.
//   * warp 4 (producer) turns list entries into page ids 32 at a time (one per lane) and issues one TMA
//     box per page and pool (page_size tokens x one kv head x head_dim, 128-byte swizzled) into a ring of
//     64-key stages.  An entry that lists nothing issues no box and adds no bytes to the stage's barrier.
//   * warps 0-3 each own 16 keys of a stage, all in one page since page_size >= 16, so a key's mask is one
//     count for each warp and stage: min(16, reach - first key).  S = Q K^T and O += P V are
//     mma.m16n8k16 with float32 accumulators; P enters as a 16-bit high part plus its remainder, which
//     keeps the weights to 2^-17 in bf16, to 2^-22 in f16.  f16 has a quantum of 2^-24, so there P is moved up
//     by 2^15 (the largest weight is 1, the largest f16 below 2^16): none loses more than 2^-40 of the largest.
//     Online softmax in the log2 domain, one pass over K and V.
//   * the 4 S warp states are merged once at the end: each CTA leaves its four in shared memory and the
//     cluster's CTAs share out the output columns, S lanes to four of them, each lane reading one CTA's
//     states over distributed shared memory.  No workspace, no second launch, and a fixed order of sums.
// A decode step is bound by HBM: its lists differ between kv heads, so nothing is read twice.  256
// sequences, 8 kv heads of 128, 64 pages of 16 tokens each (1.08 GB): 174 us, 6.2 TB/s, 91 % of the
// copy rate.  One sequence of 131072 tokens, 128 of its 32-token pages: 11.6 us (2.5 at the copy rate), latency:
// list, table, pages, products and the cluster's merge follow one another.
#include <type_traits>

#include "mma_common.cuh"
#include "sparse_common.cuh"

namespace pa {

using namespace mmac;

namespace {

constexpr int kNW = kMmaConsumerWarps;

template <typename T>
constexpr float kWeightUp = std::is_same<T, __half>::value ? 32768.f : 1.f;

template <int D>
struct Merge {  // a CTA's states: acc [4][16][D + 4], m [4][16], l [4][16]
    static constexpr int kRow = D + 4;
    static constexpr int kAcc = kNW * 16 * kRow;
    static constexpr int kBytes = (kAcc + 2 * kNW * 16) * 4;
};

}  // namespace

template <typename T, int D, int NSTAGE>
__global__ void __launch_bounds__(kMmaThreads, D == 256 ? 1 : 2)
    paged_attn_sparse_mma_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                                 const SparseParams sp, int ps_shift, int S, int row_tiles) {
    using Op = MmaOp<T>;
    constexpr int kStage = Geo<D>::kStageBytes;
    constexpr int kChunks = Geo<D>::kChunks;
    const FwdParams &p = sp.f;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[3 * NSTAGE];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ps = 1 << ps_shift;
    const int s = blockIdx.x % S;
    int unit = blockIdx.x / S;
    const int kvh = unit % p.Hkv;
    unit /= p.Hkv;
    const int rt = unit % row_tiles;
    long long t_row = unit / row_tiles;
    const BehindFirst order(sp);
    if (sp.by_seq && short_rows(sp, t_row, 1, t_row) == 0) return;  // the whole cluster: it has one token
    const int pps = kMmaTileKeys >> ps_shift;  // list entries of a stage
    // this CTA's entries [e0, e1): whole stages
    const int per = ((sp.K + S - 1) / S + pps - 1) / pps * pps;
    const int e0 = min((long long)s * per, (long long)sp.K), e1 = min(e0 + per, sp.K);
    const int n_tiles = (e1 - e0 + pps - 1) / pps;
    const int32_t *list = sp.sel + (t_row * p.Hkv + kvh) * sp.K;
    // the producer's first entries are on their way while the row's sequence is looked up
    auto listed = [&](int e) { return e < e1 ? __ldg(list + e) : -1; };
    int j_cur = -1, j_nxt = -1;
    if (warp == kNW) {
        if (lane == 0) {
            tma_prefetch_desc(&tmK);
            tma_prefetch_desc(&tmV);
        }
        j_cur = listed(e0 + lane);
        j_nxt = listed(e0 + 32 + lane);
    }
    RangeCheck ranges(sp);
    const TokenRow tr = token_row(p, t_row, sp.n_tok, threadIdx.x == 0);
    if (!sp.group_min) ranges.report(p);  // else the tcgen05 kernel has
    if (tr.b < 0) return;
    if (sp.group_min && __ldg(p.q_start + tr.b + 1) - __ldg(p.q_start + tr.b) >= sp.group_min) return;

    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    const uint32_t bar_fk = smem_u32(&bars[0]), bar_fv = smem_u32(&bars[NSTAGE]), bar_em = smem_u32(&bars[2 * NSTAGE]);
    if (threadIdx.x == 0) {
        for (int i = 0; i < NSTAGE; ++i) {
            mbar_init(bar_fk + 8 * i, 1);
            mbar_init(bar_fv + 8 * i, 1);
            mbar_init(bar_em + 8 * i, kNW);
        }
        fence_barrier_init();
    }
    __syncthreads();

    const int np = (tr.reach + ps - 1) >> ps_shift;

    const int g = lane >> 2, tq = lane & 3;
    const int ra = rt * 16 + g, rb = ra + 8;  // query heads of the group
    float m_a = kNegInf, m_b = kNegInf, l_a = 0.f, l_b = 0.f;
    float acc[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
    bool bad = false;

    if (warp == kNW) {
        // ---------------------------------------------------------------- producer
        const uint32_t box_bytes = (uint32_t)(Geo<D>::NH * ps * 128);
        const int32_t *bt = p.block_table + (long long)tr.b * p.W;
        // first token of a listed page, -ps for an id outside the pool, -1 for an entry that lists nothing
        auto entry = [&](int j) {
            if (j < 0 || j >= np) return -1;
            const int id = __ldg(bt + j);
            if (id < 0 || id >= p.num_pages) {
                atomicOr(p.err, (unsigned int)PA_ERRBIT_PAGE_RANGE);
                return -ps;  // wholly out of the tensor: the box reads as zeros
            }
            return id << ps_shift;
        };
        int batch = e0;
        int cur = entry(j_cur), nxt = entry(j_nxt);
        int issued = 0;
        for (int t = 0; t < n_tiles; ++t) {
            const int st = t % NSTAGE;
            if (t >= NSTAGE) {
                const bool ok = mbar_wait(bar_em + 8 * st, ((t / NSTAGE) - 1) & 1, p.err);
                bad = __any_sync(0xffffffffu, !ok);
                if (bad) break;
            }
            const int first = e0 + t * pps;
            if (first >= batch + 32) {
                batch += 32;
                cur = nxt;
                nxt = entry(listed(batch + 32 + lane));
            }
            const int tok = __shfl_sync(0xffffffffu, cur, (first - batch + lane) & 31);
            const bool on = lane < pps && tok != -1;
            const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, on)) * box_bytes;
            if (lane == 0) {
                mbar_arrive_expect_tx(bar_fk + 8 * st, bytes);
                mbar_arrive_expect_tx(bar_fv + 8 * st, bytes);
            }
            __syncwarp();
            if (on) {
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
    } else {
        // ---------------------------------------------------------------- consumers
        const bool va = ra < p.G, vb = rb < p.G;
        const long long row0 = t_row * p.Hq + (long long)kvh * p.G;
        const T *qa = static_cast<const T *>(p.q) + q_row_offset(p, row0 + (va ? ra : 0));
        const T *qb = static_cast<const T *>(p.q) + q_row_offset(p, row0 + (vb ? rb : 0));
        uint32_t qf[D / 16][4];
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const int c0 = kk * 16 + 2 * tq;
            qf[kk][0] = va ? __ldg(reinterpret_cast<const uint32_t *>(qa + c0)) : 0u;
            qf[kk][1] = vb ? __ldg(reinterpret_cast<const uint32_t *>(qb + c0)) : 0u;
            qf[kk][2] = va ? __ldg(reinterpret_cast<const uint32_t *>(qa + c0 + 8)) : 0u;
            qf[kk][3] = vb ? __ldg(reinterpret_cast<const uint32_t *>(qb + c0 + 8)) : 0u;
        }
        const int kw0 = warp * 16;                 // this warp's first key in a stage
        const int my_e = e0 + (kw0 >> ps_shift);   // its list entry in stage 0
        const int in_page = kw0 & (ps - 1);
        int j_next = my_e < e1 ? __ldg(list + my_e) : -1;
        const int mi = lane >> 3, rr = lane & 7;
        for (int t = 0; t < n_tiles; ++t) {
            const int st = t % NSTAGE;
            const uint32_t par = (uint32_t)(t / NSTAGE) & 1;
            const uint32_t kbuf = sbase + (uint32_t)(st * 2 * kStage), vbuf = kbuf + kStage;
            const int j = j_next;
            const int e_next = my_e + (t + 1) * pps;
            j_next = e_next < e1 ? __ldg(list + e_next) : -1;
            // keys of this warp in the stage that the token may see
            const int cnt = (j >= 0 && j < np) ? min(16, tr.reach - (j << ps_shift) - in_page) : 0;
            if (!bad) bad = __any_sync(0xffffffffu, !mbar_wait(bar_fk + 8 * st, par, p.err));
            const bool active = !bad && cnt > 0;
            uint32_t ph[2][2], pl[2][2];
            if (active) {
                float sc[2][4] = {};
                const int key = kw0 + rr + ((mi >> 1) << 3);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    uint32_t b0, b1, b2, b3;
                    ldmatrix_x4(kv_chunk_addr<D>(kbuf, key, 2 * kk + (mi & 1), ps_shift), b0, b1, b2, b3);
                    Op::run(sc[0], qf[kk], b0, b1);
                    Op::run(sc[1], qf[kk], b2, b3);
                }
                float mx_a = kNegInf, mx_b = kNegInf;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const int k0 = n * 8 + 2 * tq;
                    sc[n][0] = k0 < cnt ? sc[n][0] * p.scale_log2 : kNegInf;
                    sc[n][1] = k0 + 1 < cnt ? sc[n][1] * p.scale_log2 : kNegInf;
                    sc[n][2] = k0 < cnt ? sc[n][2] * p.scale_log2 : kNegInf;
                    sc[n][3] = k0 + 1 < cnt ? sc[n][3] * p.scale_log2 : kNegInf;
                    mx_a = fmaxf(mx_a, fmaxf(sc[n][0], sc[n][1]));
                    mx_b = fmaxf(mx_b, fmaxf(sc[n][2], sc[n][3]));
                }
                mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, 1));
                mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, 2));
                mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, 1));
                mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, 2));
                const float mn_a = fmaxf(m_a, mx_a), mn_b = fmaxf(m_b, mx_b);
                // -inf - (-inf) guard: a row whose scores are all -inf uses 0 as its offset
                const float mu_a = mn_a == kNegInf ? 0.f : mn_a, mu_b = mn_b == kNegInf ? 0.f : mn_b;
                const float al_a = exp2f(m_a - mu_a), al_b = exp2f(m_b - mu_b);
                m_a = mn_a;
                m_b = mn_b;
                float rs_a = 0.f, rs_b = 0.f;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    float p0 = exp2f(sc[n][0] - mu_a), p1 = exp2f(sc[n][1] - mu_a);
                    float p2 = exp2f(sc[n][2] - mu_b), p3 = exp2f(sc[n][3] - mu_b);
                    rs_a += p0 + p1;
                    rs_b += p2 + p3;
                    p0 *= kWeightUp<T>, p1 *= kWeightUp<T>, p2 *= kWeightUp<T>, p3 *= kWeightUp<T>;
                    ph[n][0] = Op::pack(p0, p1);
                    ph[n][1] = Op::pack(p2, p3);
                    const float2 ha = Op::unpack(ph[n][0]), hb = Op::unpack(ph[n][1]);
                    pl[n][0] = Op::pack(p0 - ha.x, p1 - ha.y);
                    pl[n][1] = Op::pack(p2 - hb.x, p3 - hb.y);
                }
                l_a = l_a * al_a + rs_a;
                l_b = l_b * al_b + rs_b;
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    acc[n][0] *= al_a;
                    acc[n][1] *= al_a;
                    acc[n][2] *= al_b;
                    acc[n][3] *= al_b;
                }
            }
            if (!bad) bad = __any_sync(0xffffffffu, !mbar_wait(bar_fv + 8 * st, par, p.err));
            if (active && !bad) {
                if (cnt < 16) {
                    // keys the token may not see hold any bits: their weight is 0, but 0 * NaN is NaN
                    for (int idx = lane; idx < 16 * kChunks; idx += 32) {
                        const int key = idx / kChunks;
                        if (key >= cnt)
                            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                                             kv_chunk_addr<D>(vbuf, kw0 + key, idx % kChunks, ps_shift)),
                                         "r"(0u)
                                         : "memory");
                    }
                    fence_proxy_async_smem();  // before the slot is written by TMA again
                    __syncwarp();
                }
                const uint32_t ah[4] = {ph[0][0], ph[0][1], ph[1][0], ph[1][1]};
                const uint32_t al[4] = {pl[0][0], pl[0][1], pl[1][0], pl[1][1]};
                const int key = kw0 + rr + ((mi & 1) << 3);
#pragma unroll
                for (int jj = 0; jj < D / 16; ++jj) {
                    uint32_t b0, b1, b2, b3;
                    ldmatrix_x4_trans(kv_chunk_addr<D>(vbuf, key, 2 * jj + (mi >> 1), ps_shift), b0, b1, b2, b3);
                    Op::run(acc[2 * jj], ah, b0, b1);
                    Op::run(acc[2 * jj + 1], ah, b2, b3);
                    Op::run(acc[2 * jj], al, b0, b1);
                    Op::run(acc[2 * jj + 1], al, b2, b3);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_em + 8 * st);
        }
        l_a += __shfl_xor_sync(0xffffffffu, l_a, 1);
        l_a += __shfl_xor_sync(0xffffffffu, l_a, 2);
        l_b += __shfl_xor_sync(0xffffffffu, l_b, 1);
        l_b += __shfl_xor_sync(0xffffffffu, l_b, 2);
    }

    // ------------------------------------------------------------------ merge the cluster's 4 S states
    constexpr int kRow = Merge<D>::kRow;
    float *sm = reinterpret_cast<float *>(smem_raw + (sbase - raw));
    float *s_m = sm + Merge<D>::kAcc, *s_l = s_m + kNW * 16;
    __syncthreads();  // the ring is drained: every copy has landed and been read
    if (warp < kNW) {
        float *wa = sm + warp * 16 * kRow;
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
            const int col = n * 8 + 2 * tq;
            *reinterpret_cast<float2 *>(wa + g * kRow + col) = make_float2(acc[n][0], acc[n][1]);
            *reinterpret_cast<float2 *>(wa + (g + 8) * kRow + col) = make_float2(acc[n][2], acc[n][3]);
        }
        if (tq == 0) {
            s_m[warp * 16 + g] = m_a;
            s_m[warp * 16 + g + 8] = m_b;
            s_l[warp * 16 + g] = l_a;
            s_l[warp * 16 + g + 8] = l_b;
        }
    }
    if (S > 1)
        cluster_barrier();
    else
        __syncthreads();
    const int rows = min(16, p.G - rt * 16);
    const long long row0 = t_row * p.Hq + (long long)kvh * p.G + rt * 16;
    const uint32_t m_addr = sbase + Merge<D>::kAcc * 4, l_addr = m_addr + kNW * 16 * 4;
    // Four columns of a row to S lanes, each the states of one CTA: every load of a lane is on its way before
    // the first is needed, and the lanes' sums are added in a fixed order.
    const int items = rows * (D / 4);
    for (int i0 = (s * kMmaThreads + warp * 32) / S; i0 < items; i0 += kMmaThreads) {
        const int idx = i0 + lane / S, cta = lane % S;
        const int r = idx < items ? idx / (D / 4) : 0, c = idx % (D / 4) * 4;
        float m[kNW], l[kNW];
        float4 v[kNW];
#pragma unroll
        for (int w = 0; w < kNW; ++w) {
            m[w] = peer_load(peer_addr(m_addr + (w * 16 + r) * 4, cta));
            l[w] = peer_load(peer_addr(l_addr + (w * 16 + r) * 4, cta));
            v[w] = peer_load4(peer_addr(sbase + ((w * 16 + r) * kRow + c) * 4, cta));
        }
        float M = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
        for (int o = 1; o < S; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        const float mu = M == kNegInf ? 0.f : M;
        float L = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kNW; ++w) {
            const float x = exp2f(m[w] - mu);
            L = fmaf(x, l[w], L);
            o.x = fmaf(x, v[w].x, o.x);
            o.y = fmaf(x, v[w].y, o.y);
            o.z = fmaf(x, v[w].z, o.z);
            o.w = fmaf(x, v[w].w, o.w);
        }
        for (int k = 1; k < S; k <<= 1) {
            L += __shfl_xor_sync(0xffffffffu, L, k);
            o.x += __shfl_xor_sync(0xffffffffu, o.x, k);
            o.y += __shfl_xor_sync(0xffffffffu, o.y, k);
            o.z += __shfl_xor_sync(0xffffffffu, o.z, k);
            o.w += __shfl_xor_sync(0xffffffffu, o.w, k);
        }
        if (cta != 0 || idx >= items) continue;
        // a row without a key: 0 and -inf (a NaN sum stays a NaN)
        const float inv = L == 0.f ? 0.f : 1.f / (L * kWeightUp<T>);
        uint2 packed;
        packed.x = Op::pack(o.x * inv, o.y * inv);
        packed.y = Op::pack(o.z * inv, o.w * inv);
        *reinterpret_cast<uint2 *>(static_cast<T *>(p.out) + (row0 + r) * D + c) = packed;
        if (c == 0 && p.lse) p.lse[row0 + r] = L == 0.f ? kNegInf : M * kLn2 + logf(L);
    }
    if (S > 1) cluster_barrier();  // peers may still be reading this CTA's states
}

template <typename T, int D, int NSTAGE>
static cudaError_t launch_sparse_mma_t(const SparseParams &sp, int sms, const CUtensorMap &tmk,
                                       const CUtensorMap &tmv, cudaStream_t stream) {
    const FwdParams &p = sp.f;
    auto kern = paged_attn_sparse_mma_kernel<T, D, NSTAGE>;
    const size_t smem = mma_smem_bytes(D, NSTAGE);
    static_assert(Merge<D>::kBytes <= NSTAGE * 2 * Geo<D>::kStageBytes, "the merge must fit in the ring");
    static SmemLimit limit;
    const cudaError_t e = limit.raise((const void *)kern, smem);
    if (e != cudaSuccess) return e;
    int ps_shift = 0;
    while ((1 << ps_shift) < p.ps) ++ps_shift;
    const int row_tiles = (p.G + 15) / 16;
    const long long units = (sp.by_seq ? short_blocks(sp, 1) : sp.n_tok) * p.Hkv * row_tiles;
    // Split a list over a cluster while its CTAs do not yet fill two per multiprocessor and each keeps
    // two stages of its own.
    const long long stages = ((long long)sp.K * p.ps + kMmaTileKeys - 1) / kMmaTileKeys;
    int S = 1;
    while (S < 8 && units * S * 2 <= 2ll * sms && stages >= 4ll * S) S *= 2;
    if (units * S > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(units * S));
    cfg.blockDim = dim3(kMmaThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2]{};
    cfg.numAttrs = second_launch_attrs(attr, S, sp.group_min > 0);
    cfg.attrs = attr;
    return cudaLaunchKernelEx(&cfg, kern, tmk, tmv, sp, ps_shift, S, row_tiles);
}

template <typename T>
static cudaError_t launch_sparse_mma_dt(const SparseParams &sp, int sms, const CUtensorMap &tmk,
                                        const CUtensorMap &tmv, cudaStream_t stream) {
    if (sp.f.D == 64) return launch_sparse_mma_t<T, 64, 4>(sp, sms, tmk, tmv, stream);
    if (sp.f.D == 128) return launch_sparse_mma_t<T, 128, 3>(sp, sms, tmk, tmv, stream);
    return launch_sparse_mma_t<T, 256, 3>(sp, sms, tmk, tmv, stream);
}

cudaError_t launch_sparse_mma(const SparseParams &sp, int dtype, int sms, const CUtensorMap &tmk,
                              const CUtensorMap &tmv, cudaStream_t stream) {
    if (dtype == PA_BF16) return launch_sparse_mma_dt<__nv_bfloat16>(sp, sms, tmk, tmv, stream);
    return launch_sparse_mma_dt<__half>(sp, sms, tmk, tmv, stream);
}

}  // namespace pa
