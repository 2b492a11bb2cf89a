// The pages that runs of query tokens attend to, scored on the 5th-generation tensor cores (head_dim 64 or
// 128, up to 32 query heads to a kv head).
//
// The score is that of select_pages.cuh: s = max_h (min(qi, 0) . lo + max(qi, 0) . hi) over integers of 8 bits, here
// f16 numbers (exact), summed in float32 (exact, below 2^23), then one product with the page's scale.
// A CTA takes TT consecutive tokens of a sequence and one kv head.  Its queries are quantised once into the B
// operand (TT x Gp columns, Gp the heads rounded up to a power of two, head 0 repeated in the gap; 2 D deep);
// the pages go through in tiles of 128 rows: 16 bytes a thread from global memory, converted (XOR, two byte
// permutes and two half2 subtractions for four bytes) into the A operand, 2 D / 16 tcgen05.mma issued by
// one thread into one of two tensor-memory buffers, and while they run the tile before is read out: a
// thread holds one page and 32 columns, takes each token's maximum and stores the score.  Then each warp
// takes the pages of two tokens.
//
// 936 tokens of 8 kv heads over some 400 pages take 44.9 us in two waves of CTAs, the kernel of
// select_pages.cuh 58; 3.3 us is the products' floor.  Half of a CTA's time is the selection, bound by
// instructions (a warp counts a row's 400 scores six times), a quarter the set-up (queries to 8 bits).
#include <type_traits>

#include "select_common.cuh"
#include "sparse_tile.cuh"
#include "tc05.cuh"

namespace pa {

namespace {

constexpr int kSelTcThreads = 512, kSelTcWarps = 16;
constexpr int kSelTcHalf = 128 * 128;  // bytes of 64 f16 columns of 128 rows

// Byte offset of 16-byte chunk c (8 f16 of a 64-column half) of a row in the 128-byte swizzle.
__device__ __forceinline__ uint32_t chunk_at(int row, int c) { return (uint32_t)(row * 128 + ((c ^ (row & 7)) << 4)); }

__device__ __forceinline__ void store16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// Four bytes as two pairs of f16 numbers: 0x64uu is 1024 + uu, and uu = byte + 128.
__device__ __forceinline__ void widen(uint32_t w, uint32_t &lo, uint32_t &hi) {
    const uint32_t x = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(x, 0x64646464u, 0x4140), b = __byte_perm(x, 0x64646464u, 0x4342);
    const __half2 off = __float2half2_rn(1152.f);
    const __half2 u = __hsub2(*reinterpret_cast<const __half2 *>(&a), off);
    const __half2 v = __hsub2(*reinterpret_cast<const __half2 *>(&b), off);
    lo = *reinterpret_cast<const uint32_t *>(&u);
    hi = *reinterpret_cast<const uint32_t *>(&v);
}

}  // namespace

template <int D, int GS>
__global__ void __launch_bounds__(kSelTcThreads, 1)
    paged_attn_select_tc05_kernel(const SparseParams sp, int dtype, int TT, int Wk) {
    constexpr int KH = 2 * D / 64;          // 64-column halves of the operands' depth
    constexpr int Gp = 1 << GS;
    constexpr int PIECES = 2 * D / 16;      // 16-byte pieces of a page's envelope
    constexpr int PER = 128 * PIECES / kSelTcThreads;  // of a thread and tile
    const FwdParams &p = sp.f;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[2];
    __shared__ uint32_t s_tmem;
    __shared__ int s_reach[kTileMaxTokens];
    __shared__ unsigned s_amax[kTileMaxTokens];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.x % p.Hkv;
    TokenTile x;
    let_second_start();
    RangeCheck ranges(sp);
    const bool here = token_tile(sp, blockIdx.x / p.Hkv, TT, x);
    ranges.report(p);
    if (!here) return;
    const int N = (TT * Gp + 15) / 16 * 16;  // columns; those past the tokens' are never read out
    if (tid < x.nt) s_reach[tid] = row_key_limit(p, x.b, x.L, x.i0 + tid, x.n_seq);
    if (tid < kTileMaxTokens) s_amax[tid] = 0u;
    const int reach_max = row_key_limit(p, x.b, x.L, x.i0 + x.nt - 1, x.n_seq);  // grows with the token
    const int np_max = (reach_max + p.ps - 1) / p.ps;
    const int m0 = sp.sink, m1 = np_max - sp.local, want = sp.K - sp.sink - sp.local;
    const int tiles = np_max > sp.K && want > 0 ? (m1 - m0 + 127) / 128 : 0;

    // shared memory: A [KH][128 rows] | B [KH][N rows] | scores [TT][Wk]
    const uint32_t raw = smem_u32(smem_raw), sA = (raw + 1023u) & ~1023u, sB = sA + KH * kSelTcHalf;
    const uint32_t b_half = (uint32_t)N * 128u;
    float *s_score = reinterpret_cast<float *>(smem_raw + (sA - raw) + KH * kSelTcHalf + KH * N * 128);
    const uint32_t bar0 = smem_u32(&bars[0]);
    if (tid == 0) {
        mbar_init(bar0, 1);
        mbar_init(bar0 + 8, 1);
        fence_barrier_init();
    }
    if (warp == 0) {
        tc05::tmem_alloc(smem_u32(&s_tmem), 256);
        tc05::tmem_relinquish();
    }

    // ---------------------------------------------------------------- pages on their way
    const int32_t *bt = p.block_table + (long long)x.b * p.W;
    uint4 page[PER];
    int ids[PER];
    float scale_next = 0.f;
    // piece k of this thread: page row and 16 bytes of its envelope
    auto row_of = [&](int k) { return (tid + k * kSelTcThreads) / PIECES; };
    const int piece = tid % PIECES;  // the same for every k
    auto load_ids = [&](int tile) {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int j = m0 + tile * 128 + row_of(k);
            ids[k] = tile < tiles && j < m1 ? __ldg(bt + j) : 0;
        }
    };
    auto load_pages = [&] {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const bool ok = ids[k] >= 0 && ids[k] < p.num_pages;
            if (!ok) atomicOr(p.err, (unsigned int)PA_ERRBIT_PAGE_RANGE);
            page[k] = __ldg(reinterpret_cast<const uint4 *>(sp.env + ((long long)(ok ? ids[k] : 0) * p.Hkv + h) * 2 * D) + piece);
        }
    };
    // the scale of the page that this thread reads out of tile `tile`: 0 outside the pool
    const int out_row = (warp & 3) * 32 + lane;
    auto load_scale = [&](int tile) {
        const int j = m0 + tile * 128 + out_row;
        const int id = tile < tiles && j < m1 ? __ldg(bt + j) : -1;
        return id >= 0 && id < p.num_pages ? __ldg(sp.env_scale + (long long)id * p.Hkv + h) : 0.f;
    };
    if (tiles > 0) {
        load_ids(0);
        load_pages();
        load_ids(1);
        scale_next = load_scale(0);
    }

    // ---------------------------------------------------------------- queries to 8 bits: B
    tc05::fence_before_sync();
    __syncthreads();
    tc05::fence_after_sync();
    const uint32_t tmem = s_tmem;
    if (tiles > 0) {
        constexpr int QP = D / 16;  // 16-element pieces of a head
        constexpr int MOST = (128 * QP + kSelTcThreads - 1) / kSelTcThreads;
        float q[MOST][16];
#pragma unroll
        for (int k = 0; k < MOST; ++k) {
            const int idx = tid + k * kSelTcThreads, col = idx / QP, d = idx % QP * 16, tok = col >> GS;
            const int head = (col & (Gp - 1)) < p.G ? col & (Gp - 1) : 0;
            unsigned a = 0;  // magnitudes order as their bits, infinities and NaNs on top
            if (col < N && tok < x.nt) {
                q_load16(p.q, dtype, q_row_offset(p, (x.tok0 + tok) * p.Hq + (long long)h * p.G + head) + d, q[k]);
#pragma unroll
                for (int e = 0; e < 16; ++e) a = max(a, __float_as_uint(q[k][e]) & 0x7fffffffu);
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) q[k][e] = 0.f;
            }
#pragma unroll
            for (int o = 1; o < QP; o <<= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
            if (col < N && d == 0 && a != 0) atomicMax(&s_amax[tok], a);
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < MOST; ++k) {
            const int idx = tid + k * kSelTcThreads, col = idx / QP, d = idx % QP * 16;
            if (col >= N) continue;
            // a non-finite query scores 0 everywhere
            const unsigned bits = s_amax[col >> GS];
            const float a = bits < 0x7f800000u ? __uint_as_float(bits) : 0.f;
            if (a > 0.f) {
                quantise8<16>(q[k], a, 127.f / a);
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) q[k][e] = 0.f;
            }
            uint32_t lo[8], hi[8];
            const __half2 zero = __float2half2_rn(0.f);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const __half2 v = __floats2half2_rn(q[k][2 * e], q[k][2 * e + 1]);
                const __half2 l = __hmin2(v, zero), u = __hmax2(v, zero);
                lo[e] = *reinterpret_cast<const uint32_t *>(&l);
                hi[e] = *reinterpret_cast<const uint32_t *>(&u);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int m = d + 8 * c;  // depth: lo corners at m, hi corners at D + m
                const uint32_t at = sB + (uint32_t)(m >> 6) * b_half + chunk_at(col, m >> 3 & 7);
                store16(at, lo[4 * c], lo[4 * c + 1], lo[4 * c + 2], lo[4 * c + 3]);
                store16(at + (uint32_t)(KH / 2) * b_half, hi[4 * c], hi[4 * c + 1], hi[4 * c + 2], hi[4 * c + 3]);
            }
        }
    }

    // ---------------------------------------------------------------- tiles of 128 pages
    const uint32_t idesc = tc05::idesc_f16(false, false, 128, N);
    bool bad = false;
    float scale = 0.f;
    const int group = warp >> 2;  // of 32 columns
    // Read tile t out of tensor memory: this thread's page, 32 columns.
    auto read_out = [&](int t) {
        if (group * 32 >= TT * Gp || bad) return;
        uint32_t u[32];
        tc05::ld_32cols(tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)((t & 1) * 128 + group * 32), u);
        tc05::wait_ld();
        const int j = t * 128 + out_row;  // score index
        if (m0 + j >= m1) return;
        float *dst = s_score + (group * (32 >> GS)) * Wk + j;
#pragma unroll
        for (int tok = 0; tok < (32 >> GS); ++tok) {
            float s = __uint_as_float(u[tok << GS]);
#pragma unroll
            for (int e = 1; e < Gp; ++e) s = fmaxf(s, __uint_as_float(u[(tok << GS) + e]));
            if (group * (32 >> GS) + tok < x.nt) dst[tok * Wk] = scale < INFINITY ? __fmul_rn(s, scale) : INFINITY;
        }
    };
    for (int t = 0; t < tiles; ++t) {
        // A is free once the products of tile t - 1 are done, which its read-out waits for too
        if (t > 0 && !bad) bad = !mbar_wait(bar0 + 8 * ((t - 1) & 1), ((t - 1) >> 1) & 1, p.err);
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int r = row_of(k), c = piece * 2;  // chunks c, c + 1 of the row
            const uint32_t w[4] = {page[k].x, page[k].y, page[k].z, page[k].w};
            uint32_t f[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) widen(w[i], f[2 * i], f[2 * i + 1]);
            const uint32_t half = sA + (uint32_t)(c >> 3) * kSelTcHalf;
            store16(half + chunk_at(r, c & 7), f[0], f[1], f[2], f[3]);
            store16(half + chunk_at(r, (c & 7) + 1), f[4], f[5], f[6], f[7]);
        }
        const float scale_now = scale_next;
        if (t + 1 < tiles) {
            load_pages();
            load_ids(t + 2);
            scale_next = load_scale(t + 1);
        }
        fence_proxy_async_smem();
        tc05::fence_before_sync();
        bad = __syncthreads_or(bad);  // A (and B) written, tile t - 2 read out
        if (warp == 0 && !bad) {
            // the values the same in every lane as the compiler can see: operands in uniform registers
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0) + (uint32_t)((t & 1) * 128);
            tc05::fence_after_sync();
            const uint32_t dhi = tc05::smem_desc_sw128_hi(1024);
            const uint32_t da = tc05::smem_desc_sw128_lo(sA, 16), db = tc05::smem_desc_sw128_lo(sB, 16);
            if (tc05::elect_one()) {
#pragma unroll
                for (int kk = 0; kk < KH * 4; ++kk) {
                    const uint32_t oa = ((uint32_t)(kk >> 2) * kSelTcHalf + (uint32_t)(kk & 3) * 32u) >> 4;
                    const uint32_t ob = ((uint32_t)(kk >> 2) * b_half + (uint32_t)(kk & 3) * 32u) >> 4;
                    tc05::mma_ss_lh(tm, da + oa, dhi, db + ob, dhi, idesc, kk > 0 ? 1u : 0u);
                }
                tc05::commit(bar0 + 8 * (t & 1));
            }
            __syncwarp();
        }
        tc05::fence_after_sync();
        if (t > 0) read_out(t - 1);
        scale = scale_now;
    }
    if (tiles > 0) {
        if (!bad) bad = !mbar_wait(bar0 + 8 * ((tiles - 1) & 1), ((tiles - 1) >> 1) & 1, p.err);
        tc05::fence_after_sync();
        read_out(tiles - 1);
    }
    tc05::fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        tc05::fence_after_sync();
        tc05::tmem_dealloc(tmem, 256);
    }

    // ---------------------------------------------------------------- each token's pages
    for (int i = warp; i < x.nt; i += kSelTcWarps) {
        const int np = (s_reach[i] + p.ps - 1) / p.ps;
        int32_t *out = sp.sel_out + ((x.tok0 + i) * p.Hkv + h) * sp.K;
        if (np <= sp.K) {
            for (int j = lane; j < sp.K; j += 32) out[j] = j < np ? j : -1;
            continue;
        }
        for (int j = lane; j < sp.sink; j += 32) out[j] = j;
        for (int j = lane; j < sp.local; j += 32) out[sp.K - sp.local + j] = np - sp.local + j;
        const int n = np - sp.local - sp.sink;
        if (want == 0) continue;
        const float *row = s_score + i * Wk;
        if (n <= 256)
            warp_select<8>(row, n, want, sp.sink, out + sp.sink, lane);
        else if (n <= 512)
            warp_select<16>(row, n, want, sp.sink, out + sp.sink, lane);
        else
            warp_select_long(row, n, want, sp.sink, out + sp.sink, lane);
    }
}

template <int D, int GS>
static cudaError_t launch_select_tc05_t(const SparseParams &sp, int dtype, int TT, cudaStream_t stream) {
    auto kern = paged_attn_select_tc05_kernel<D, GS>;
    static SmemLimit limit;
    const cudaError_t e = limit.raise((const void *)kern, kSelectTc05MaxSmem);
    if (e != cudaSuccess) return e;
    const int Wk = (sp.f.W + 3) / 4 * 4;
    const long long units = count_tiles(sp, TT) * sp.f.Hkv;
    if (units > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    kern<<<(unsigned)units, kSelTcThreads, select_tc05_smem(D, ((TT << GS) + 15) / 16 * 16, TT, sp.f.W), stream>>>(sp, dtype, TT, Wk);
    return cudaGetLastError();
}

size_t select_tc05_smem(int D, int N, int TT, int W) {
    return (size_t)(2 * D / 64) * (kSelTcHalf + N * 128) + (size_t)TT * ((W + 3) / 4 * 4) * 4 + 1024;
}

// Tokens of a CTA: as many as fill 128, 64, 32 or 16 columns, at most 32, with their scores in shared memory; 0
// where the kernel does not apply.
int select_tile_tokens(int D, int G, int W) {
    if ((D != 64 && D != 128) || G > 32) return 0;
    int Gp = 1;
    while (Gp < G) Gp *= 2;
    for (int N = 128; N >= 16; N /= 2) {
        const int TT = N / Gp < kTileMaxTokens ? N / Gp : kTileMaxTokens;
        if (TT * Gp >= 16 && select_tc05_smem(D, TT * Gp, TT, W) <= kSelectTc05MaxSmem) return TT;
    }
    return 0;
}

cudaError_t launch_select_tc05(const SparseParams &sp, int dtype, int sms, cudaStream_t stream) {
    int GS = 0;
    while ((1 << GS) < sp.f.G) ++GS;
    // One CTA an SM, and its time grows with its tokens: the tile that makes whole waves of them (936 tokens
    // of 8 kv heads: 25 tokens in two waves instead of 32 in 1.6).
    const int most = select_tile_tokens(sp.f.D, sp.f.G, sp.f.W);
    int TT = most;
    long long best = 0;
    for (int t = most; 2 * t > most; --t) {
        const long long tiles = sp.f.q_start ? (sp.n_tok + t - 1) / t : (long long)sp.f.B * ((sp.f.Sq + t - 1) / t);
        const long long cost = (tiles * sp.f.Hkv + sms - 1) / sms * (t + 8);  // the set-up weighs as 8 tokens
        if (!best || cost < best) best = cost, TT = t;
    }
    auto pick = [&](auto d) {
        constexpr int D = decltype(d)::value;
        switch (GS) {
            case 0: return launch_select_tc05_t<D, 0>(sp, dtype, TT, stream);
            case 1: return launch_select_tc05_t<D, 1>(sp, dtype, TT, stream);
            case 2: return launch_select_tc05_t<D, 2>(sp, dtype, TT, stream);
            case 3: return launch_select_tc05_t<D, 3>(sp, dtype, TT, stream);
            case 4: return launch_select_tc05_t<D, 4>(sp, dtype, TT, stream);
            default: return launch_select_tc05_t<D, 5>(sp, dtype, TT, stream);
        }
    };
    return sp.f.D == 64 ? pick(std::integral_constant<int, 64>{}) : pick(std::integral_constant<int, 128>{});
}

}  // namespace pa
