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
// scores, as ordered 32-bit keys, meet in the first CTA's shared memory, which finds each token's
// threshold key by bisection over the key bits and writes the pages above it in order.
#include <float.h>

#include "sparse_common.cuh"

namespace pa {

namespace {

constexpr int kSelWarps = 4;
constexpr int kSelThreads = kSelWarps * 32;
constexpr int kSelMaxTokens = 32;      // of one CTA
constexpr float kTwo24 = 16777216.f;
constexpr float kNoHead = 1e30f;       // subtracted from the column of a head that is not there

// Order-preserving map of a float to an unsigned key (no NaN comes here).
__device__ __forceinline__ unsigned ordered(float x) {
    const unsigned u = __float_as_uint(x + 0.f);  // -0 becomes +0
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint2 b) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y));
}

// The want-th largest of n keys (0 < want < n) as (threshold, pages at the threshold to take): keys
// above the threshold are taken whole.  count(c): how many keys are >= c, in every thread.  lo / hi: the
// smallest and largest key.  Ends as soon as exactly `want` keys reach a candidate.
template <typename Count>
__device__ __forceinline__ unsigned threshold_key(unsigned lo, unsigned hi, int want, Count count) {
    // bits above the first one in which lo and hi differ are common to all keys
    const int top = lo == hi ? -1 : 31 - __clz((int)(lo ^ hi));
    unsigned thr = top == 31 ? 0u : top < 0 ? lo : (lo >> (top + 1)) << (top + 1);
    for (int bit = top; bit >= 0; --bit) {
        const unsigned cand = thr | (1u << bit);
        const int c = count(cand);
        if (c >= want) {
            thr = cand;
            if (c == want) break;
        }
    }
    return thr;
}

// Elements i .. i + 3 of q, whose type is a value here: only the quantisation reads it.
__device__ __forceinline__ void q_load4(const void *q, int dtype, long long i, float (&v)[4]) {
    if (dtype == PA_F32) {
        const float4 x = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(q) + i));
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
        return;
    }
    const uint2 u = __ldg(reinterpret_cast<const uint2 *>(static_cast<const unsigned short *>(q) + i));
    const float2 x = dtype == PA_BF16 ? MmaOp<__nv_bfloat16>::unpack(u.x) : MmaOp<__half>::unpack(u.x);
    const float2 y = dtype == PA_BF16 ? MmaOp<__nv_bfloat16>::unpack(u.y) : MmaOp<__half>::unpack(u.y);
    v[0] = x.x, v[1] = x.y, v[2] = y.x, v[3] = y.y;
}

struct SelectPlan {
    int TT;    // query tokens of a CTA
    int Gp;    // columns of a token: G rounded up to a power of two (G <= 8), or all of them
    int S;     // CTAs of a cluster
    int Wk;    // key stride of a token in shared memory
    int dtype; // of q
};

// One warp writes a token's pages: `thr` as threshold_key gives it.
__device__ __forceinline__ void write_selected(const unsigned *keys, int n, int want, unsigned thr, int base,
                                               int32_t *out, int lane) {
    int above = 0;
    for (int j = lane; j < n; j += 32) above += keys[j] > thr;
    above = __reduce_add_sync(0xffffffffu, above);
    int ties = want - above, done = 0;  // the first `ties` pages at the threshold are taken
    const unsigned below = (1u << lane) - 1;
    for (int j0 = 0; j0 < n && done < want; j0 += 32) {
        const int j = j0 + lane;
        const unsigned key = j < n ? keys[j] : 0u;
        const bool eq = j < n && key == thr;
        const unsigned eqs = __ballot_sync(0xffffffffu, eq);
        const bool take = (j < n && key > thr) || (eq && __popc(eqs & below) < ties);
        const unsigned taken = __ballot_sync(0xffffffffu, take);
        if (take) out[done + __popc(taken & below)] = base + j;
        done += __popc(taken);
        ties -= min(ties, __popc(eqs));
    }
}

// A token's selection by one warp, its keys in registers (n <= 32 NK).
template <int NK>
__device__ __forceinline__ void warp_select(const unsigned *keys, int n, int want, int base, int32_t *out, int lane) {
    unsigned k[NK], lo = 0xffffffffu, hi = 0;
#pragma unroll
    for (int i = 0; i < NK; ++i) {
        const int j = i * 32 + lane;
        k[i] = j < n ? keys[j] : 0u;  // 0 is below every key
        if (j < n) lo = min(lo, k[i]);
        hi = max(hi, k[i]);
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    const unsigned thr = threshold_key(lo, hi, want, [&](unsigned c) {
        int s = 0;
#pragma unroll
        for (int i = 0; i < NK; ++i) s += k[i] >= c;
        return (int)__reduce_add_sync(0xffffffffu, s);
    });
    write_selected(keys, n, want, thr, base, out, lane);
}

}  // namespace

template <int D, int NT>
__global__ void __launch_bounds__(kSelThreads)
    paged_attn_select_kernel(const SparseParams sp, const SelectPlan plan) {
    constexpr int KS = 2 * D / 16;  // k steps of a page's envelope
    constexpr int NC = 2 * D / 64;  // 16-byte loads of a lane and page
    constexpr int COLS = 8 * NT;
    const FwdParams &p = sp.f;
    extern __shared__ __align__(16) uint8_t sm_raw[];
    uint2 *s_b = reinterpret_cast<uint2 *>(sm_raw);                         // [KS][NT][32] query fragments
    unsigned *s_key = reinterpret_cast<unsigned *>(s_b + KS * NT * 32);     // [TT][Wk]
    __shared__ float s_sub[COLS];                  // 128 sum_d q of a column, or kNoHead
    __shared__ int s_seq[kSelMaxTokens], s_reach[kSelMaxTokens];
    __shared__ unsigned s_red[kSelWarps][2];
    __shared__ unsigned s_amax[kSelMaxTokens];  // bits of the largest |q| of each token's group
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, tq = lane & 3;
    const int S = plan.S, rank = blockIdx.x % S;
    const int unit = blockIdx.x / S;
    const int h = unit % p.Hkv;
    const long long t0 = (long long)(unit / p.Hkv) * plan.TT;
    const int nt_tok = (int)min((long long)plan.TT, sp.n_tok - t0);
    // a peer's shared memory may be written only once it runs
    if (S > 1) asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    if (tid < nt_tok) {
        const TokenRow tr = token_row(p, t0 + tid, sp.n_tok, true);
        s_seq[tid] = tr.b;
        s_reach[tid] = tr.reach;
    }
    if (S > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    __syncthreads();

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

        // A lane's two pages of a tile: id (-1: outside the pool, -2: none), envelope bytes and scale.
        int id[2];
        uint4 raw[2][NC];
        float scale[2];
        auto load_ids = [&](int tile, int (&x)[2]) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int j = m0 + tile * 16 + g + r * 8;
                x[r] = tile < tile1 && j < m1 ? max(__ldg(bt + j), -1) : -2;
            }
        };
        auto load_pages = [&](const int (&x)[2], uint4 (&v)[2][NC], float (&sc)[2]) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const bool ok = x[r] >= 0 && x[r] < p.num_pages;
                if (!ok && x[r] != -2) atomicOr(p.err, (unsigned int)PA_ERRBIT_PAGE_RANGE);
                const long long at = (long long)(ok ? x[r] : 0) * p.Hkv + h;
                const uint4 *src = reinterpret_cast<const uint4 *>(sp.env + at * 2 * D) + tq;
#pragma unroll
                for (int c = 0; c < NC; ++c) v[r][c] = ok ? __ldg(src + c * 4) : make_uint4(0u, 0u, 0u, 0u);
                sc[r] = ok ? __ldg(sp.env_scale + at) : 0.f;
            }
        };
        int id_next[2];
        load_ids(tile0 + warp, id);
        load_ids(tile0 + warp + kSelWarps, id_next);
        load_pages(id, raw, scale);

        const int passes = plan.Gp > COLS ? (p.G + COLS - 1) / COLS : 1;
        constexpr int NQ = (D / 4 + 31) / 32;  // 4-element groups of a head a lane takes
        if (scored) {
            if (tid < kSelMaxTokens) s_amax[tid] = 0u;
            __syncthreads();
            // heads to the warps, `per_tok` of them to a token
            const int per_tok = passes > 1 || plan.TT == 1 ? p.G : plan.Gp, cols = per_tok * (i1 - i0);
#pragma unroll 2
            for (int w = warp; w < cols; w += kSelWarps) {
                const int tok = i0 + w / per_tok, hd = w % per_tok;
                if (hd >= p.G) continue;
                const long long q0 = q_row_offset(p, (t0 + tok) * p.Hq + (long long)h * p.G + hd);
                unsigned a = 0;  // magnitudes order as their bits, infinities and NaNs on top
#pragma unroll
                for (int i = 0; i < NQ; ++i) {
                    const int d = (i * 32 + lane) * 4;
                    if (D % 128 == 0 || d < D) {
                        float x[4];
                        q_load4(p.q, plan.dtype, q0 + d, x);
#pragma unroll
                        for (int e = 0; e < 4; ++e) a = max(a, __float_as_uint(x[e]) & 0x7fffffffu);
                    }
                }
                a = __reduce_max_sync(0xffffffffu, a);
                if (lane == 0) atomicMax(&s_amax[tok], a);
            }
        }
        for (int pass = 0; scored && pass < passes; ++pass) {
            __syncthreads();  // s_amax is there; s_b of the last pass has been read
            // Query columns in 8 bits: each group of four elements d .. d + 3 is one lane's slot in the
            // fragments of k step ks (lo corners) and ks + KS / 2 (hi corners).
            const int heads = passes > 1 ? min(COLS, p.G - pass * COLS) : p.G;
#pragma unroll 2
            for (int w = warp; w < COLS; w += kSelWarps) {
                const int tok = i0 + (passes > 1 || plan.TT == 1 ? 0 : w / plan.Gp);
                const int hd = passes > 1 || plan.TT == 1 ? w : w % plan.Gp;
                const bool there = hd < heads && tok < i1;
                // a non-finite query scores 0 everywhere
                const unsigned bits = there ? s_amax[tok] : 0u;
                const float a = bits < 0x7f800000u ? __uint_as_float(bits) : 0.f;
                const long long q0 =
                    q_row_offset(p, there ? (t0 + tok) * p.Hq + (long long)h * p.G + pass * COLS + hd : 0);
                int sum = 0;
#pragma unroll
                for (int i = 0; i < NQ; ++i) {
                    const int m = (i * 32 + lane) * 4;
                    if (D % 128 != 0 && m >= D) continue;
                    float x[4] = {0.f, 0.f, 0.f, 0.f};
                    if (a > 0.f) q_load4(p.q, plan.dtype, q0 + m, x);
                    __half lo[4], hi[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float y = a > 0.f ? rintf(__fmul_rn(__fdiv_rn(x[e], a), 127.f)) : 0.f;
                        sum += (int)y;
                        lo[e] = __float2half_rn(fminf(y, 0.f));
                        hi[e] = __float2half_rn(fmaxf(y, 0.f));
                    }
                    // byte m = 64 c + 16 tq + 4 w + e of the envelope is element e of lane tq in k step 4 c + w
                    const int ks = (m >> 6) * 4 + ((m & 15) >> 2), l = (w & 7) * 4 + ((m & 63) >> 4);
                    auto put = [&](int k, const __half (&v)[4]) {
                        const __half2 x2 = __halves2half2(v[0], v[1]), y2 = __halves2half2(v[2], v[3]);
                        s_b[(k * NT + (w >> 3)) * 32 + l] = make_uint2(*reinterpret_cast<const uint32_t *>(&x2),
                                                                      *reinterpret_cast<const uint32_t *>(&y2));
                    };
                    put(ks, lo);
                    put(ks + KS / 2, hi);
                }
                sum = __reduce_add_sync(0xffffffffu, sum);
                if (lane == 0) s_sub[w] = there ? 128.f * (float)sum : kNoHead;
            }
            __syncthreads();
            for (int tile = tile0 + warp; tile < tile1; tile += kSelWarps) {
                // the next tile's pages are on their way while this one is scored
                uint4 cur[2][NC];
                float cur_scale[2];
                const int j0 = m0 + tile * 16 + g;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    cur_scale[r] = scale[r];
#pragma unroll
                    for (int c = 0; c < NC; ++c) cur[r][c] = raw[r][c];
                }
                const bool last = tile + kSelWarps >= tile1;
                if (!last || pass + 1 < passes) {
                    if (last) {  // the next pass begins again
                        load_ids(tile0 + warp, id);
                        load_ids(tile0 + warp + kSelWarps, id_next);
                    } else {
                        id[0] = id_next[0], id[1] = id_next[1];
                        load_ids(tile + 2 * kSelWarps, id_next);
                    }
                    load_pages(id, raw, scale);
                }
                float acc[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const uint32_t wa[4] = {cur[0][c].x, cur[0][c].y, cur[0][c].z, cur[0][c].w};
                    const uint32_t wb[4] = {cur[1][c].x, cur[1][c].y, cur[1][c].z, cur[1][c].w};
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t xa = wa[w] ^ 0x80808080u, xb = wb[w] ^ 0x80808080u;
                        const uint32_t a[4] = {__byte_perm(xa, 0, 0x4140), __byte_perm(xb, 0, 0x4140),
                                               __byte_perm(xa, 0, 0x4342), __byte_perm(xb, 0, 0x4342)};
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma_f16(acc[n], a, s_b[((c * 4 + w) * NT + n) * 32 + lane]);
                    }
                }
                // whole scores of (page g / g + 8, columns 2 tq, 2 tq + 1), largest over a token's heads
                auto key_of = [&](float s, int r) {
                    return ordered(cur_scale[r] == INFINITY ? INFINITY : __fmul_rn(s, cur_scale[r]));
                };
                if (plan.TT == 1 || passes > 1) {
                    float best[2] = {-2e30f, -2e30f};
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            best[e >> 1] = fmaxf(best[e >> 1], acc[n][e] * kTwo24 - s_sub[n * 8 + 2 * tq + (e & 1)]);
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 1));
                        best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 2));
                        const int j = j0 + r * 8;
                        if (tq == 0 && j < m1) {
                            // the scale is not negative: the largest key is the key of the largest score
                            unsigned key = key_of(best[r], r);
                            if (pass > 0) key = max(key, s_key[j - m0]);
                            s_key[j - m0] = key;
                        }
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            float x = acc[n][2 * r] * kTwo24 - s_sub[n * 8 + 2 * tq];
                            float y = acc[n][2 * r + 1] * kTwo24 - s_sub[n * 8 + 2 * tq + 1];
                            const int j = j0 + r * 8;
                            if (plan.Gp == 1) {
                                const int tok = n * 8 + 2 * tq;
                                if (j < m1) {
                                    if (i0 + tok < i1) s_key[tok * plan.Wk + j - m0] = key_of(x, r);
                                    if (i0 + tok + 1 < i1) s_key[(tok + 1) * plan.Wk + j - m0] = key_of(y, r);
                                }
                                continue;
                            }
                            x = fmaxf(x, y);
                            if (plan.Gp >= 4) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                            if (plan.Gp >= 8) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                            const int col = n * 8 + 2 * tq, tok = col / plan.Gp;
                            if (col % plan.Gp == 0 && i0 + tok < i1 && j < m1) s_key[tok * plan.Wk + j - m0] = key_of(x, r);
                        }
                    }
                }
            }
        }

        if (S > 1) {
            // this CTA's keys into the first one's shared memory
            if (scored && rank != 0) {
                __syncthreads();
                const int a = tile0 * 16, e = min(tile1 * 16, m1 - m0);
                for (int i = 0; i < i1 - i0; ++i)
                    for (int j = a + tid; j < e; j += kSelThreads) {
                        uint32_t dst;
                        asm("mapa.shared::cluster.u32 %0, %1, %2;"
                            : "=r"(dst)
                            : "r"(smem_u32(s_key + i * plan.Wk + j)), "r"(0));
                        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(dst), "r"(s_key[i * plan.Wk + j]) : "memory");
                    }
            }
            asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
        } else {
            __syncthreads();
        }
        if (rank == 0) {
            // token i's scored pages are the first n_i: np_i - local - sink
            for (int i = i0 + warp; i < i1; i += kSelWarps) {
                const int np = (s_reach[i] + p.ps - 1) / p.ps;
                int32_t *out = sp.sel_out + ((t0 + i) * p.Hkv + h) * sp.K;
                if (np <= sp.K) {
                    for (int j = lane; j < sp.K; j += 32) out[j] = j < np ? j : -1;
                    continue;
                }
                for (int j = lane; j < sp.sink; j += 32) out[j] = j;
                for (int j = lane; j < sp.local; j += 32) out[sp.K - sp.local + j] = np - sp.local + j;
                const int n = np - sp.local - sp.sink;
                const unsigned *keys = s_key + (i - i0) * plan.Wk;
                if (want == 0 || n > 1024) continue;
                if (n <= 256)
                    warp_select<8>(keys, n, want, sp.sink, out + sp.sink, lane);
                else if (n <= 512)
                    warp_select<16>(keys, n, want, sp.sink, out + sp.sink, lane);
                else
                    warp_select<32>(keys, n, want, sp.sink, out + sp.sink, lane);
            }
            // longer rows: the whole CTA counts, one warp writes
            for (int i = i0; i < i1 && want > 0; ++i) {
                const int np = (s_reach[i] + p.ps - 1) / p.ps, n = np - sp.local - sp.sink;
                if (np <= sp.K || n <= 1024) continue;
                const unsigned *keys = s_key + (i - i0) * plan.Wk;
                unsigned lo = 0xffffffffu, hi = 0;
                for (int j = tid; j < n; j += kSelThreads) {
                    lo = min(lo, keys[j]);
                    hi = max(hi, keys[j]);
                }
                lo = __reduce_min_sync(0xffffffffu, lo);
                hi = __reduce_max_sync(0xffffffffu, hi);
                if (lane == 0) s_red[warp][0] = lo, s_red[warp][1] = hi;
                __syncthreads();
#pragma unroll
                for (int w = 0; w < kSelWarps; ++w) {
                    lo = min(lo, s_red[w][0]);
                    hi = max(hi, s_red[w][1]);
                }
                __syncthreads();
                const unsigned thr = threshold_key(lo, hi, want, [&](unsigned c) {
                    int s = 0;
                    for (int j = tid; j < n; j += kSelThreads) s += keys[j] >= c;
                    s = __reduce_add_sync(0xffffffffu, s);
                    if (lane == 0) s_red[warp][0] = s;
                    __syncthreads();
                    s = 0;
#pragma unroll
                    for (int w = 0; w < kSelWarps; ++w) s += s_red[w][0];
                    __syncthreads();
                    return s;
                });
                int32_t *out = sp.sel_out + ((t0 + i) * p.Hkv + h) * sp.K;
                if (warp == 0) write_selected(keys, n, want, thr, sp.sink, out + sp.sink, lane);
            }
        }
        if (i1 < nt_tok) {  // the next sequence's keys go to the same place
            if (S > 1)
                asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
            else
                __syncthreads();
        }
    }
}

template <int D, int NT>
static cudaError_t launch_select_t(const SparseParams &sp, const SelectPlan &plan, cudaStream_t stream) {
    auto kern = paged_attn_select_kernel<D, NT>;
    const size_t frag = (size_t)(2 * D / 16) * NT * 32 * sizeof(uint2);
    static SmemLimit limit;
    const cudaError_t e = limit.raise((const void *)kern, frag + (size_t)PA_SELECT_MAX_PAGES * 4);
    if (e != cudaSuccess) return e;
    const long long units = (sp.n_tok + plan.TT - 1) / plan.TT * sp.f.Hkv;
    if (units * plan.S > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(units * plan.S));
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = frag + (size_t)plan.TT * plan.Wk * 4;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = plan.S;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, sp, plan);
}

template <int D>
static cudaError_t launch_select_d(const SparseParams &sp, int dtype, int sms, cudaStream_t stream) {
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
        while (plan.Gp < p.G) plan.Gp *= 2;
        // Prompt chunks: as many tokens a CTA as fill 32, 16 or 8 columns while their keys take at most
        // 64 KB and there is a CTA for every multiprocessor; a batch of mostly single tokens takes one.
        NT = 4;
        plan.TT = 32 / plan.Gp;
        auto fits = [&] {
            return (long long)plan.TT * plan.Wk * 4 <= 65536 && (sp.n_tok + plan.TT - 1) / plan.TT * p.Hkv >= sms;
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
    // Few rows: a cluster shares their pages, each CTA at least two tiles for each of its warps.
    const long long units = (sp.n_tok + plan.TT - 1) / plan.TT * p.Hkv;
    plan.S = 1;
    while (plan.S < 8 && units * plan.S * 2 <= 2ll * sms && p.W >= plan.S * 2 * 2 * kSelWarps * 16) plan.S *= 2;
    if (NT == 1) return launch_select_t<D, 1>(sp, plan, stream);
    if (NT == 2) return launch_select_t<D, 2>(sp, plan, stream);
    return launch_select_t<D, 4>(sp, plan, stream);
}

cudaError_t launch_select_pages(const SparseParams &sp, int dtype, int sms, cudaStream_t stream) {
    if (sp.f.D == 64) return launch_select_d<64>(sp, dtype, sms, stream);
    if (sp.f.D == 128) return launch_select_d<128>(sp, dtype, sms, stream);
    return launch_select_d<256>(sp, dtype, sms, stream);
}

}  // namespace pa
