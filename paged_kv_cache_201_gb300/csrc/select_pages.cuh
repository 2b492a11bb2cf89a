// The pages a query token attends to, by an 8-bit score of each page's key envelope.
//
// With qi the group's queries in 8 bits and lo / hi the page's corners, s = max_h sum_d max(qi lo, qi hi)
// = max_h (min(qi, 0) . lo + max(qi, 0) . hi): an integer dot product of length 2 D, below 2^24, then one
// float32 product with the page's scale.  The score, and so the selection, is the same bits in any order
// of evaluation.
//
// The dot products run on the f16 tensor cores (m16n8k16, float32 accumulators), exactly: pages are the
// 16 rows, query heads the columns, and k runs over a page's 2 D envelope bytes.  GB300's 8-bit integer
// products reach 150 TOP/s, its f16 ones 600 (both measured with mma.sync).  A stored byte e becomes the
// f16 number (e + 128) 2^-24, a subnormal whose bits are the byte itself: one XOR and two byte permutes
// for four elements.  A product's sum is then (sum_d q e + 128 sum_d q) 2^-24 with an integer below
// 2^23 in the bracket, and the second term is known for each head.  k may run in any order, so each lane
// takes the 16 consecutive bytes that one wide load gives it.
//
// One cluster of S CTAs = one kv head and TT consecutive query tokens (1 in a decode batch; up to 32 / G
// in prompt chunks, whose tokens read the same envelopes).  Its pages are shared out to the CTAs; their
// scores meet in the first CTA's shared memory, which finds each token's threshold by narrowing a bracket and
// writes the pages above it in order.  Where there are
// enough rows to fill the GPU with single warps, a warp takes a row by itself (WPU = 1): its latencies
// (lengths, table, envelopes, threshold search) then overlap with other rows' instead of holding three idle
// warps at barriers.
//
// 256 sequences of some 3000 tokens, 8 kv heads (98 MB of envelopes): 29.3 us, 3.3 TB/s, half the copy rate.
// A row's chain (table, envelopes, some six counting steps, writing) is as long as its bytes' way from
// DRAM, and warps of one wave go through it together.  Four warps a row took 36 us.  L2 prefetches of the
// next rows' envelopes (both kinds of instruction) made it slower, 40 to 45 us.  Two sequences of up to
// 131072 tokens in 32-token pages, 4 kv heads: 15.8 us, a chain of latencies (clusters of eight CTAs, then one CTA's threshold search).
#pragma once

#include "select_common.cuh"

namespace pa {

namespace {

constexpr int kSelWarps = 4;
template <int WPU>
constexpr int kSelCtaWarps = WPU > kSelWarps ? WPU : kSelWarps;  // of a CTA whose rows take WPU warps each
constexpr int kRowWarps = 1;           // of a row, where rows fill the GPU
constexpr int kSelMaxTokens = 32;      // of one CTA
constexpr int kWarpSelectPages = 1024;  // longest row a warp of its own selects from
constexpr float kTwo24 = 16777216.f;
constexpr float kNoHead = -1e30f;      // score of a column without a head

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint2 b) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y));
}

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

constexpr int kBins = 512;

struct SelectPlan {
    int TT;    // query tokens of a CTA
    int Gp;    // columns of a token: G rounded up to a power of two (G <= 8), or all of them
    int gs;    // its logarithm (TT > 1)
    int S;     // CTAs of a cluster
    int Wk;    // score stride of a token in shared memory
    int dtype; // of q
};

}  // namespace

template <int D, int NT, int WPU>
__global__ void __launch_bounds__(kSelCtaWarps<WPU> * 32, 16 / kSelCtaWarps<WPU>)
    paged_attn_select_kernel(const SparseParams sp, const SelectPlan plan) {
    constexpr int KS = 2 * D / 16;  // k steps of a page's envelope
    constexpr int NC = 2 * D / 64;  // 16-byte loads of a lane and page
    constexpr int COLS = 8 * NT;
    const FwdParams &p = sp.f;
    constexpr int UNITS = kSelCtaWarps<WPU> / WPU;  // of a CTA
    extern __shared__ __align__(16) uint8_t sm_raw[];
    __shared__ __align__(8) float s_sub_[UNITS][COLS];  // -128 2^-24 sum_d q of a column, or kNoHead
    __shared__ int s_seq_[UNITS][kSelMaxTokens], s_reach_[UNITS][kSelMaxTokens];
    __shared__ unsigned s_amax_[UNITS][kSelMaxTokens];  // bits of the largest |q| of each token's group
    __shared__ int s_red[2][WPU][2];
    __shared__ __align__(16) int s_hist[kBins];
    const int lane = threadIdx.x & 31, wi = threadIdx.x >> 5;
    const int warp = wi % WPU, tid = warp * 32 + lane;  // within the unit
    constexpr int kThreads = WPU * 32;
    const int me = wi / WPU;
    const int g = lane >> 2, tq = lane & 3;
    static_assert(WPU == 1 || UNITS == 1, "a unit is a warp or the CTA");
    auto sync = [] {
        if (WPU == 1)
            __syncwarp();
        else
            __syncthreads();
    };
    const size_t unit_bytes = (size_t)KS * NT * 32 * sizeof(uint2) + (size_t)plan.TT * plan.Wk * 4;
    uint2 *s_b = reinterpret_cast<uint2 *>(sm_raw + me * unit_bytes);    // [KS][NT][32] query fragments
    float *s_key = reinterpret_cast<float *>(s_b + KS * NT * 32);  // [TT][Wk]
    float *s_sub = s_sub_[me];
    int *s_seq = s_seq_[me], *s_reach = s_reach_[me];
    unsigned *s_amax = s_amax_[me];
    const int S = plan.S, rank = blockIdx.x % S;
    const long long unit = (long long)(blockIdx.x / S) * UNITS + me;
    const int h = (int)(unit % p.Hkv);
    long long t0 = unit / p.Hkv * plan.TT;
    const BehindFirst order(sp);
    RangeCheck ranges(sp);
    if (!sp.by_seq && t0 >= sp.n_tok) {  // a warp of its own without a row
        if (!sp.group_min) ranges.report(p);
        return;
    }
    int nt_tok = 0;
    if (sp.by_seq) {
        nt_tok = short_rows(sp, unit / p.Hkv, plan.TT, t0);
        if (nt_tok == 0) return;  // the whole cluster: it has these tokens
    } else {
        nt_tok = (int)min((long long)plan.TT, sp.n_tok - t0);
    }
    // a peer's shared memory may be written only once it runs
    if (S > 1) asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    if (tid < nt_tok) {
        const TokenRow tr = token_row(p, t0 + tid, sp.n_tok, true);
        // a long run of tokens is the tcgen05 kernel's
        const bool other = tr.b >= 0 && sp.group_min && __ldg(p.q_start + tr.b + 1) - __ldg(p.q_start + tr.b) >= sp.group_min;
        s_seq[tid] = other ? -1 : tr.b;
        s_reach[tid] = tr.reach;
    }
    if (!sp.group_min) ranges.report(p);  // else the tcgen05 kernel has
    if (S > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    sync();

    for (int i0 = 0, i1 = 0; i0 < nt_tok; i0 = i1) {  // tokens [i0, i1) of one sequence
        const int b = s_seq[i0];
        int np_max = 0;
        for (i1 = i0; i1 < nt_tok && s_seq[i1] == b; ++i1) np_max = max(np_max, (s_reach[i1] + p.ps - 1) / p.ps);
        if (b < 0) continue;
        const int m0 = sp.sink, m1 = np_max - sp.local;  // pages that may need a score
        const int want = sp.K - sp.sink - sp.local;
        const bool scored = np_max > sp.K && want > 0;
        const int32_t *bt = p.block_table + (long long)b * p.W;
        // this CTA's tiles of 16 pages
        const int tiles = scored ? (m1 - m0 + 15) / 16 : 0, per = (tiles + S - 1) / S;
        const int tile0 = min(rank * per, tiles), tile1 = min(tile0 + per, tiles);

        // A lane's two pages of a tile.  A page that is not there (past the row, or an id outside the
        // pool) reads page 0; its score is dropped or set to 0 below.
        const uint4 *src[2];  // envelope bytes, from this lane's first 16 on
        const float *src_scale[2];
        bool in_pool[2];
        int id_next[2];
        uint4 raw[2][NC];
        auto load_ids = [&](int tile) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int j = m0 + tile * 16 + g + r * 8;
                id_next[r] = tile < tile1 && j < m1 ? __ldg(bt + j) : 0;
            }
        };
        auto point = [&] {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                in_pool[r] = id_next[r] >= 0 && id_next[r] < p.num_pages;
                if (!in_pool[r]) atomicOr(p.err, (unsigned int)PA_ERRBIT_PAGE_RANGE);
                const long long at = (long long)(in_pool[r] ? id_next[r] : 0) * p.Hkv + h;
                src[r] = reinterpret_cast<const uint4 *>(sp.env + at * 2 * D) + tq;
                src_scale[r] = sp.env_scale + at;
            }
        };
        float scale[2];
        if (tile0 + warp < tile1) {
            load_ids(tile0 + warp);
            point();
            load_ids(tile0 + warp + WPU);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                scale[r] = __ldg(src_scale[r]);
#pragma unroll
                for (int c = 0; c < NC; ++c) raw[r][c] = __ldg(src[r] + c * 4);
            }
        }

        const int passes = plan.Gp > COLS ? (p.G + COLS - 1) / COLS : 1;
        // Queries to 8 bits.  Lane (g, tq) holds column g's elements 64 c + 16 tq .. + 15, which are its
        // slots in the fragments of k steps 4 c .. 4 c + 3 (lo corners) and KS / 2 further (hi corners).
        const bool one_token = plan.TT == 1 || passes > 1;
        if (scored) {
            for (int i = tid; i < plan.TT; i += kThreads) s_amax[i] = 0u;
            sync();
            const int groups = one_token ? (p.G + 7) / 8 : NT;
            for (int n = warp; n < groups; n += WPU) {
                const int col = n * 8 + g;
                const int tok = i0 + (one_token ? 0 : col >> plan.gs), hd = one_token ? col : col & (plan.Gp - 1);
                unsigned a = 0;  // magnitudes order as their bits, infinities and NaNs on top
                if (hd < p.G && tok < i1) {
                    const long long q0 = q_row_offset(p, (t0 + tok) * p.Hq + (long long)h * p.G + hd) + tq * 16;
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        float x[16];
                        q_load16(p.q, plan.dtype, q0 + c * 64, x);
#pragma unroll
                        for (int e = 0; e < 16; ++e) a = max(a, __float_as_uint(x[e]) & 0x7fffffffu);
                    }
                }
                a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
                a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
                if (tq == 0 && a != 0) atomicMax(&s_amax[tok], a);
            }
        }
        for (int pass = 0; scored && pass < passes; ++pass) {
            sync();  // s_amax is there; s_b of the last pass has been read
            const int heads = passes > 1 ? min(COLS, p.G - pass * COLS) : p.G;
#pragma unroll
            for (int n = warp; n < NT; n += WPU) {
                const int col = n * 8 + g;
                const int tok = i0 + (one_token ? 0 : col >> plan.gs), hd = one_token ? col : col & (plan.Gp - 1);
                const bool there = hd < heads && tok < i1;
                // a non-finite query scores 0 everywhere
                const unsigned bits = there ? s_amax[tok] : 0u;
                const float a = bits < 0x7f800000u ? __uint_as_float(bits) : 0.f, inv = 127.f / a;
                const long long q0 =
                    q_row_offset(p, there ? (t0 + tok) * p.Hq + (long long)h * p.G + pass * COLS + hd : 0) + tq * 16;
                float sum = 0.f;
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    float x[16] = {};
                    if (a > 0.f) {
                        q_load16(p.q, plan.dtype, q0 + c * 64, x);
                        quantise8<16>(x, a, inv);
#pragma unroll
                        for (int e = 0; e < 16; ++e) sum += x[e];
                    }
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const __half2 zero = __float2half2_rn(0.f);
                        const __half2 u = __floats2half2_rn(x[4 * w], x[4 * w + 1]);
                        const __half2 v = __floats2half2_rn(x[4 * w + 2], x[4 * w + 3]);
                        auto put = [&](int k, const __half2 &y, const __half2 &z) {
                            s_b[(k * NT + n) * 32 + lane] = make_uint2(*reinterpret_cast<const uint32_t *>(&y),
                                                                      *reinterpret_cast<const uint32_t *>(&z));
                        };
                        put(c * 4 + w, __hmin2(u, zero), __hmin2(v, zero));
                        put(c * 4 + w + KS / 2, __hmax2(u, zero), __hmax2(v, zero));
                    }
                }
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);  // whole numbers: exact
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                if (tq == 0) s_sub[col] = there ? -128.f / kTwo24 * sum : kNoHead;
            }
            sync();
            // In a block of tokens a lane writes the scores of columns 8 n + 2 tq (the first of a token's,
            // else none): token i0 + tok0 + n tok_step, while n tok_step < tok_left.
            const int tok0 = one_token ? 0 : (2 * tq) >> plan.gs, tok_step = one_token ? 0 : 8 >> plan.gs;
            const int tok_left = one_token || ((2 * tq) & (plan.Gp - 1)) ? 0 : i1 - i0 - tok0;
            const int row_step = tok_step * plan.Wk;
            float *s_mine = s_key + tok0 * plan.Wk + g;
            for (int tile = tile0 + warp; tile < tile1; tile += WPU) {
                const int j0 = m0 + tile * 16 + g;
                float cur_scale[2];
                bool marked[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    cur_scale[r] = in_pool[r] ? scale[r] : 0.f;
                    marked[r] = !(cur_scale[r] < INFINITY);  // a NaN is no bound either
                }
                // Each 16 bytes make room for the next tile's once they are converted, so those are on
                // their way while this tile is scored.  After the last tile the first is read again,
                // for the next pass.
                const bool last = tile + WPU >= tile1, more = !last || pass + 1 < passes;
                if (last && more) load_ids(tile0 + warp);
                if (more) {
                    point();
                    load_ids((last ? tile0 + warp : tile + WPU) + WPU);
#pragma unroll
                    for (int r = 0; r < 2; ++r) scale[r] = __ldg(src_scale[r]);
                }
                // with one column tile, two sets of sums halve the chain of dependent products
                constexpr int SETS = NT == 1 ? 2 : 1;
                float acc[NT][4], odd[4] = {};
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float2 init = *reinterpret_cast<const float2 *>(s_sub + n * 8 + 2 * tq);
                    acc[n][0] = acc[n][2] = init.x;
                    acc[n][1] = acc[n][3] = init.y;
                }
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const uint32_t wa[4] = {raw[0][c].x, raw[0][c].y, raw[0][c].z, raw[0][c].w};
                    const uint32_t wb[4] = {raw[1][c].x, raw[1][c].y, raw[1][c].z, raw[1][c].w};
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t xa = wa[w] ^ 0x80808080u, xb = wb[w] ^ 0x80808080u;
                        const uint32_t a[4] = {__byte_perm(xa, 0, 0x4140), __byte_perm(xb, 0, 0x4140),
                                               __byte_perm(xa, 0, 0x4342), __byte_perm(xb, 0, 0x4342)};
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            mma_f16(SETS == 2 && (w & 1) ? odd : acc[n], a, s_b[((c * 4 + w) * NT + n) * 32 + lane]);
                    }
                    if (more) {
                        raw[0][c] = __ldg(src[0] + c * 4);
                        raw[1][c] = __ldg(src[1] + c * 4);
                    }
                }
                if (SETS == 2)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[0][e] += odd[e];  // whole numbers: exact
                // scores of (page g / g + 8, columns 2 tq, 2 tq + 1) in units of 2^24, largest over a
                // token's heads
                auto score_of = [&](float s, int r) {
                    return marked[r] ? INFINITY : __fmul_rn(s * kTwo24, cur_scale[r]);
                };
                if (one_token) {
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float best = fmaxf(acc[0][2 * r], acc[0][2 * r + 1]);
#pragma unroll
                        for (int n = 1; n < NT; ++n) best = fmaxf(best, fmaxf(acc[n][2 * r], acc[n][2 * r + 1]));
                        best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 1));
                        best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 2));
                        const int j = j0 + r * 8;
                        if (tq == 0 && j < m1) {
                            // the scale is not negative: the largest score is that of the largest sum
                            float x = score_of(best, r);
                            if (pass > 0) x = fmaxf(x, s_key[j - m0]);
                            s_key[j - m0] = x;
                        }
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            float x = acc[n][2 * r];
                            const float y = acc[n][2 * r + 1];
                            const bool store = j0 + r * 8 < m1 && n * tok_step < tok_left;
                            float *dst = s_mine + n * row_step + tile * 16 + r * 8;
                            if (plan.gs == 0) {
                                if (store) {
                                    dst[0] = score_of(x, r);
                                    if (n * tok_step + 1 < tok_left) dst[plan.Wk] = score_of(y, r);
                                }
                                continue;
                            }
                            x = fmaxf(x, y);
                            if (plan.gs >= 2) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                            if (plan.gs >= 3) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                            if (store) dst[0] = score_of(x, r);
                        }
                    }
                }
            }
        }

        if (S > 1) {
            // this CTA's scores into the first one's shared memory
            if (scored && rank != 0) {
                sync();
                const int a = tile0 * 16, e = min(tile1 * 16, m1 - m0);
                for (int i = 0; i < i1 - i0; ++i)
                    for (int j = a + tid; j < e; j += kThreads) {
                        uint32_t dst;
                        asm("mapa.shared::cluster.u32 %0, %1, %2;"
                            : "=r"(dst)
                            : "r"(smem_u32(s_key + i * plan.Wk + j)), "r"(0));
                        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(dst), "r"(__float_as_uint(s_key[i * plan.Wk + j])) : "memory");
                    }
            }
            asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
        } else {
            sync();
        }
        if (rank == 0) {
            // token i's scored pages are the first n_i: np_i - local - sink
            for (int i = i0 + warp; i < i1; i += WPU) {
                const int np = (s_reach[i] + p.ps - 1) / p.ps;
                int32_t *out = sp.sel_out + ((t0 + i) * p.Hkv + h) * sp.K;
                if (np <= sp.K) {
                    for (int j = lane; j < sp.K; j += 32) out[j] = j < np ? j : -1;
                    continue;
                }
                for (int j = lane; j < sp.sink; j += 32) out[j] = j;
                for (int j = lane; j < sp.local; j += 32) out[sp.K - sp.local + j] = np - sp.local + j;
                const int n = np - sp.local - sp.sink;
                const float *row = s_key + (i - i0) * plan.Wk;
                if (want == 0 || n > kWarpSelectPages) continue;
                if (n <= 256)
                    warp_select<8>(row, n, want, sp.sink, out + sp.sink, lane);
                else if (n <= 512)
                    warp_select<16>(row, n, want, sp.sink, out + sp.sink, lane);
                else
                    warp_select<kWarpSelectPages / 32>(row, n, want, sp.sink, out + sp.sink, lane);
            }
            // longer rows: the CTA counts and writes them together
            for (int i = i0; UNITS == 1 && i < i1 && want > 0; ++i) {
                const int np = (s_reach[i] + p.ps - 1) / p.ps, n = np - sp.local - sp.sink;
                if (np <= sp.K || n <= kWarpSelectPages) continue;
                const float *row = s_key + (i - i0) * plan.Wk;
                for (int j = tid; j < kBins; j += kThreads) s_hist[j] = 0;
                int turn = 0;  // two sets of partial results: one barrier an exchange
                auto exchange = [&](int x, int y) {
                    if (lane == 0) s_red[turn][warp][0] = x, s_red[turn][warp][1] = y;
                    sync();
                    turn ^= 1;
                };
                auto range = [&](float &lo, float &hi) {
                    exchange(__float_as_int(warp_min(lo)), __float_as_int(warp_max(hi)));
#pragma unroll
                    for (int w = 0; w < WPU; ++w) {
                        lo = fminf(lo, __int_as_float(s_red[turn ^ 1][w][0]));
                        hi = fmaxf(hi, __int_as_float(s_red[turn ^ 1][w][1]));
                    }
                };
                auto total = [&](int s) {
                    exchange(__reduce_add_sync(0xffffffffu, s), 0);
                    s = 0;
#pragma unroll
                    for (int w = 0; w < WPU; ++w) s += s_red[turn ^ 1][w][0];
                    return s;
                };
                float lo = INFINITY, hi = -INFINITY;
#pragma unroll 4
                for (int j = tid; j < n; j += kThreads) {
                    lo = fminf(lo, row[j]);
                    hi = fmaxf(hi, row[j]);
                }
                range(lo, hi);
                const Bins bins(lo, hi, kBins);
                bool done = false;
                int reach_lo = n;  // scores that reach lo
                Threshold thr{lo, false};
                if (bins.usable()) {
#pragma unroll 4
                    for (int j = tid; j < n; j += kThreads) atomicAdd(s_hist + bins.of(row[j]), 1);
                    sync();
                    int c[kBins / 32], above, in;
#pragma unroll
                    for (int k = 0; k < kBins / 32; k += 4) {
                        const int4 x = *reinterpret_cast<const int4 *>(s_hist + lane * (kBins / 32) + k);
                        c[k] = x.x, c[k + 1] = x.y, c[k + 2] = x.z, c[k + 3] = x.w;
                    }
                    const int bin = find_bin<kBins / 32>(c, want, lane, above, in);
                    lo = INFINITY;
                    hi = -INFINITY;
#pragma unroll 4
                    for (int j = tid; j < n; j += kThreads)
                        if (bins.of(row[j]) == bin) {
                            lo = fminf(lo, row[j]);
                            hi = fmaxf(hi, row[j]);
                        }
                    range(lo, hi);
                    reach_lo = above + in;
                    done = reach_lo == want;
                    if (done) thr = {lo, true};
                }
                if (!done) {
                    auto count = [&](float c) {
                        int s = 0;
#pragma unroll 4
                        for (int j = tid; j < n; j += kThreads) s += row[j] >= c;
                        return total(s);
                    };
                    thr = find_threshold(lo, hi, reach_lo, count(hi), want, count);
                }
                // each warp a run of scores, after counting the runs before it
                const int run = (n + WPU * 128 - 1) / (WPU * 128) * 128, a = min(warp * run, n), e = min(a + run, n);
                int gt = 0, eq = 0;
#pragma unroll 4
                for (int j = a + lane; j < e; j += 32) {
                    gt += thr.above(row[j]);
                    eq += thr.at(row[j]);
                }
                exchange(__reduce_add_sync(0xffffffffu, gt), __reduce_add_sync(0xffffffffu, eq));
                int all = 0;
                gt = eq = 0;
#pragma unroll
                for (int w = 0; w < WPU; ++w) {
                    if (w < warp) gt += s_red[turn ^ 1][w][0], eq += s_red[turn ^ 1][w][1];
                    all += s_red[turn ^ 1][w][0];
                }
                int32_t *out = sp.sel_out + ((t0 + i) * p.Hkv + h) * sp.K + sp.sink;
                for (int j = a; j < e; j += 128) {
                    float k[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) k[x] = score_at(row, e, j + x * 32 + lane);
                    write_pages<4>(k, thr, want - all, gt, eq, sp.sink + j, out, lane);
                }
                sync();  // the counters are used again by the next row
            }
        }
        if (i1 < nt_tok) {  // the next sequence's scores go to the same place
            if (S > 1)
                asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
            else
                sync();
        }
    }
}

template <int D, int NT, int WPU>
static cudaError_t launch_select_t(const SparseParams &sp, const SelectPlan &plan, cudaStream_t stream) {
    auto kern = paged_attn_select_kernel<D, NT, WPU>;
    const size_t frag = (size_t)(2 * D / 16) * NT * 32 * sizeof(uint2);
    static SmemLimit limit;
    constexpr int UNITS = kSelCtaWarps<WPU> / WPU;
    const size_t most = UNITS > 1 ? UNITS * (frag + kWarpSelectPages * 4) : frag + (size_t)PA_SELECT_MAX_PAGES * 4;
    const cudaError_t e = limit.raise((const void *)kern, most);
    if (e != cudaSuccess) return e;
    const long long rows = (sp.by_seq ? short_blocks(sp, plan.TT) : (sp.n_tok + plan.TT - 1) / plan.TT) * sp.f.Hkv;
    const long long units = (rows + UNITS - 1) / UNITS;  // clusters
    if (units * plan.S > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(units * plan.S));
    cfg.blockDim = dim3(kSelCtaWarps<WPU> * 32);
    cfg.dynamicSmemBytes = UNITS * (frag + (size_t)plan.TT * plan.Wk * 4);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2]{};
    cfg.numAttrs = second_launch_attrs(attr, plan.S, sp.group_min > 0);
    cfg.attrs = attr;
    return cudaLaunchKernelEx(&cfg, kern, sp, plan);
}

template <int D>
cudaError_t launch_select_d(const SparseParams &sp, int dtype, int sms, cudaStream_t stream) {
    const FwdParams &p = sp.f;
    SelectPlan plan{};
    plan.dtype = dtype;
    plan.Wk = (p.W + 3) / 4 * 4;
    int NT;
    if (p.G > 8) {  // one token's heads fill the columns
        NT = p.G <= 16 ? 2 : 4;
        plan.Gp = p.G;
        plan.TT = 1;
    } else {
        plan.Gp = 1;
        while (plan.Gp < p.G) plan.Gp *= 2, ++plan.gs;
        // Prompt chunks: as many tokens a CTA as fill 32, 16 or 8 columns while their scores take at most
        // 64 KB and there is a CTA for every multiprocessor, for 8 columns every other one (96 tokens of 8
        // heads, G = 1: 22 us, single tokens 33; 64 tokens, 64 CTAs: no better than single ones, 20); a batch
        // of mostly single tokens takes one.
        NT = 4;
        plan.TT = 32 / plan.Gp;
        auto fits = [&] {
            return (long long)plan.TT * plan.Wk * 4 <= 65536 &&
                   (sp.n_tok + plan.TT - 1) / plan.TT * p.Hkv * (NT == 1 ? 2 : 1) >= sms;
        };
        while (NT > 1 && !fits()) {
            NT /= 2;
            plan.TT /= 2;
        }
        if (!fits() || sp.n_tok < 4ll * p.B) {
            NT = 1;
            plan.TT = 1;
        }
    }
    const long long rows = (sp.by_seq ? short_blocks(sp, plan.TT) : (sp.n_tok + plan.TT - 1) / plan.TT) * p.Hkv;
    plan.S = 1;
    // A warp to a row once that gives every multiprocessor eight warps.
    if (plan.TT == 1 && NT <= 2 && p.W <= kWarpSelectPages && rows >= 8ll * sms)
        return NT == 1 ? launch_select_t<D, 1, kRowWarps>(sp, plan, stream) : launch_select_t<D, 2, kRowWarps>(sp, plan, stream);
    // Few rows: a cluster shares their pages, each CTA at least two tiles for each of its warps.
    while (plan.S < 8 && rows * plan.S * 2 <= 2ll * sms && p.W >= plan.S * 2 * 2 * kSelWarps * 16) plan.S *= 2;
    // Long rows, up to four CTAs a multiprocessor: twice the warps (152 rows of up to 3900 pages, head_dim 128: 42
    // -> 31 us, 320 rows of 2500: 51 -> 49; 800 rows of 1500: 64 -> 67).
    if (rows * plan.S <= 4ll * sms && p.W > 1024) {
        if (NT == 1) return launch_select_t<D, 1, 8>(sp, plan, stream);
        if (NT == 2) return launch_select_t<D, 2, 8>(sp, plan, stream);
        return launch_select_t<D, 4, 8>(sp, plan, stream);
    }
    if (NT == 1) return launch_select_t<D, 1, kSelWarps>(sp, plan, stream);
    if (NT == 2) return launch_select_t<D, 2, kSelWarps>(sp, plan, stream);
    return launch_select_t<D, 4, kSelWarps>(sp, plan, stream);
}

}  // namespace pa
