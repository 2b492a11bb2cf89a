// Attention over a 4-bit cache for runs of query tokens, on the 5th-generation tensor cores (bf16 / f16 queries,
// head_dim 64 or 128, up to 128 query heads to a kv head).
//
// A CTA takes two tiles of up to 128 rows (TT = 128 / G tokens x the G heads of a kv head, each) of one sequence over
// 128-key tiles of its cache, which it turns into f16 once for both:
//   warp 0       issues tcgen05.mma: S = Q K^T of a tile of rows into 128 columns of tensor memory, then O += P V with P
//                read from there.  The two tiles of rows take turns, one's products under the other's softmax.
//   warps 4-7    read codes and scales into registers a tile ahead and write K and V, (u - 8) scale / 8 or / 128 without
//                rounding (kv4.cuh), as swizzled f16 tiles, two slots each.  A register pairs elements d and d + 4 of eight, so
//                eight elements land in the order 0 4 1 5 2 6 3 7; Q is written in the same one, and the output's
//                columns are put back when they are stored.
//   warps 8-15   softmax, a thread a row, warps 8-11 the first tile's: weights as in attn_kv4.cu, P over S as f16 pairs of
//                high parts and remainders, O rescaled in tensor memory when a reference moves.
// Q is read, moved into f16's range row by row and written swizzled by all warps at the start.  Any byte of the cache is
// a finite number, so keys past a row's limit are only left out of its weights.
//
// Two tiles of rows over 128 keys are 16.8 MFLOP and 8.4 more for the remainders, 2.0 us of a multiprocessor at the GPU's measured
// bf16 rate; they take 2.3.  Chunks of 512 and 419 tokens over 8192 and 5720 keys (8 kv heads of 128, G = 4, bf16) are 120
// CTAs of up to 64 such steps, one wave on 152 multiprocessors: 154 us, the tensor pipe active in two thirds of a working one's cycles.  Two of 512 over 8192 keys take 169, the mma.sync kernel
// 714.  With the high parts alone the first take 126, and where the values cancel the outputs are up to 6 times as far
// off as their rounding and the float32 sums leave them.  Measured no faster, then against 121: codes turned by seven warps instead of four (129), S read twice instead of
// held in registers (139), page ids looked up a tile earlier (147), P handed over in halves (149), K and V in halves of 64
// keys (172).
#include <limits.h>

#include "kv4_tile.cuh"
#include "mma_common.cuh"
#include "tc05.cuh"

namespace pa {

namespace {

constexpr int kThreads = 512;
// Registers once the roles part: 128 x 40 + 128 x 96 + 256 x 184 are fewer than the launch's 512 x 128.
constexpr uint32_t kIssueRegs = 40, kCodeRegs = 96, kSoftmaxRegs = 184;
constexpr int kHalf = 128 * 128;  // bytes of a 64-column half of a 128-row tile
constexpr uint32_t kColO = 256;

enum { B_KF = 0, B_KE = 2, B_VF = 4, B_VE = 6, B_SF = 8, B_PF = 10, B_PD = 12, B_COUNT = 14 };

// Two float32 operations an instruction.
__device__ __forceinline__ float2 fma2f(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2f(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// Shared address of 16-byte chunk c (of 8) of row r of a swizzled half.
__device__ __forceinline__ uint32_t chunk_at(uint32_t half, int r, int c) {
    return half + (uint32_t)(r * 128) + (uint32_t)((c ^ (r & 7)) << 4);
}
__device__ __forceinline__ void sts16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// The codes of one side (0 K, 1 V) of a 128-key tile that a thread of the code warps turns into f16: for each of its
// D / 32 turns 16 bytes, 32 elements of one key, and their two scales.
template <int D>
struct Codes {
    static constexpr int kTurns = D / 32, kChunks = D / 32, kRows = 32 / kChunks;  // rows of a warp's turn
    uint4 code[kTurns];
    uint32_t scale[kTurns];
    __device__ __forceinline__ static int first_row(int turn, int w) { return (turn * 4 + w) * kRows; }
    __device__ __forceinline__ static int row(int turn, int w, int lane) {
        return first_row(turn, w) + (lane & 7) + (lane / (8 * kChunks)) * 8;
    }
    __device__ __forceinline__ static int chunk(int lane) { return (lane >> 3) % kChunks; }
    // pool: page 0's block of this kv head; id: the turn's page, -1: none
    __device__ __forceinline__ void load(const uint8_t *pool, uint32_t stride, const int (&id)[kTurns], int side, int ps, int w,
                                         int lane) {
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
            code[i] = make_uint4(0u, 0u, 0u, 0u);
            scale[i] = 0u;
            if (id[i] < 0) continue;
            const uint8_t *block = pool + (unsigned long long)(uint32_t)id[i] * stride;
            const kv4::Layout at{ps, D};
            const int r = row(i, w, lane) & (ps - 1), c = chunk(lane);
            code[i] = __ldg(reinterpret_cast<const uint4 *>(block + at.codes(side, r)) + c);
            scale[i] = __ldg(reinterpret_cast<const uint16_t *>(block + at.scales(side, r)) + c);
        }
    }
    __device__ __forceinline__ void store(uint32_t tile, int w, int lane) const {
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
            const int r = row(i, w, lane), c = chunk(lane);
            const uint32_t half = tile + (uint32_t)(c >> 1) * kHalf;
            const uint32_t word[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t h[4];
                kv4::unpack8(word[k], kv4::scale_pair(__byte_perm(scale[i], 0, 0x4040 + (k / 2) * 0x0101)), h);
                sts16(chunk_at(half, r, (c & 1) * 4 + k), h[0], h[1], h[2], h[3]);
            }
        }
    }
};

}  // namespace

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attn_kv4_tc05_kernel(const Kv4Params p, int ps_shift, uint32_t idesc_qk, uint32_t idesc_pv) {
    using Op = MmaOp<__half>;
    constexpr int NH = D / 64, kTile = NH * kHalf;  // bytes of a tile of Q, K or V
    const FwdParams &f = p.s.f;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[B_COUNT];
    __shared__ uint32_t s_tmem;
    __shared__ float s_factor[256];
    __shared__ long long s_row[256];  // a thread's row of out, -1: none (kept here, not in the softmax warps' registers)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ps = 1 << ps_shift;
    const int part = blockIdx.x % p.S, unit = blockIdx.x / p.S, kvh = unit % f.Hkv;
    let_second_start();
    RangeCheck ranges(p.s);
    const Tile u = find_tile(p, unit / f.Hkv, lane);
    ranges.report(f);
    if (u.cnt <= 0) return;
    int L = max(u.len, 0);
    if (L > f.W << ps_shift) {  // never read past the sequence's block-table row
        if (tid == 0) atomicOr(f.err, (unsigned int)PA_ERRBIT_SEQ_CLIPPED);
        L = f.W << ps_shift;
    }
    const int k_hi = row_key_limit(f, u.b, L, u.i + u.cnt - 1, u.n);  // the last token reaches furthest
    // this CTA's share of the 128-key tiles
    const int all_tiles = k_hi > 0 ? ((k_hi - 1) >> 7) + 1 : 0, share = (all_tiles + p.S - 1) / p.S;
    const int tile0 = min(part * share, all_tiles), n_tiles = min(share, all_tiles - tile0);
    const int half_tokens = p.TT / 2;  // tokens of a tile of rows

    // shared memory: Q x2 | K x2 | V x2
    const uint32_t raw = smem_u32(smem_raw), sbase = (raw + 1023u) & ~1023u;
    auto sQ = [&](int i) { return sbase + (uint32_t)(kTile * i); };
    auto sK = [&](int i) { return sbase + (uint32_t)(kTile * (2 + i)); };
    auto sV = [&](int i) { return sbase + (uint32_t)(kTile * (4 + i)); };
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(B_KF + i), 4);
            mbar_init(bar(B_KE + i), 1);
            mbar_init(bar(B_VF + i), 4);
            mbar_init(bar(B_VE + i), 1);
            mbar_init(bar(B_SF + i), 1);
            mbar_init(bar(B_PF + i), 4);
            mbar_init(bar(B_PD + i), 1);
        }
        fence_barrier_init();
    }
    if (warp == 0) {
        tc05::tmem_alloc(smem_u32(&s_tmem), 512);
        tc05::tmem_relinquish();
    }
    // ---- Q: 16 bytes a thread, D / 8 threads a row; a row's largest magnitude brings it into f16
    {
        constexpr int C = D / 8;
        const int c = tid % C;
#pragma unroll 1
        for (int r = tid / C; r < 256; r += kThreads / C) {
            const int tile = r >> 7, tk = tile * half_tokens + (r & 127) / f.G, h = (r & 127) % f.G;
            const bool valid = (r & 127) < half_tokens * f.G && tk < u.cnt;
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (valid)
                x = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(f.q) +
                                                          q_row_offset(f, (u.q0 + u.i + tk) * f.Hq + kvh * f.G + h)) + c);
            uint32_t w[4] = {__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632), __byte_perm(x.y, x.w, 0x5410),
                             __byte_perm(x.y, x.w, 0x7632)};
            if (f.scale_log2 < 0.f)  // as -q: the factor is positive
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] ^= 0x80008000u;
            float am = kv4::largest_of<T>(w);
#pragma unroll
            for (int o = 1; o < C; o <<= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
            const float factor = kv4::scale_query<T>(w, am);
            sts16(chunk_at(sQ(tile) + (uint32_t)(c >> 3) * kHalf, r & 127, c & 7), w[0], w[1], w[2], w[3]);
            if (c == 0) s_factor[r] = fmaxf(fabsf(f.scale_log2) * factor, kLeastFactor);
        }
        fence_proxy_async_smem();
    }
    tc05::fence_before_sync();
    __syncthreads();
    tc05::fence_after_sync();
    const uint32_t tmem = s_tmem;

    if (warp < 4) {
        tc05::setmaxnreg_dec<kIssueRegs>();
        if (warp == 0 && n_tiles > 0) {
            // The whole warp runs this, its values the same in every lane as the compiler can see, and one lane issues: the
            // operands then live in uniform registers.
            auto same = [](auto v) { return __shfl_sync(0xffffffffu, v, 0); };
            const int nt = same(n_tiles);
            const uint32_t tm = same(tmem);
            const bool leader = tc05::elect_one();
            const uint32_t dhi = tc05::smem_desc_sw128_hi(1024);
            const uint32_t dq0 = tc05::smem_desc_sw128_lo(sQ(0), 16), dq1 = tc05::smem_desc_sw128_lo(sQ(1), 16);
            const uint32_t dk0 = tc05::smem_desc_sw128_lo(sK(0), 16), dk1 = tc05::smem_desc_sw128_lo(sK(1), 16);
            const uint32_t dv0 = tc05::smem_desc_sw128_lo(sV(0), (uint32_t)kHalf), dv1 = tc05::smem_desc_sw128_lo(sV(1), (uint32_t)kHalf);
            auto qk = [&](int tile, int t) {
                const uint32_t d = tm + 128u * (uint32_t)tile, dq = tile ? dq1 : dq0, dk = t & 1 ? dk1 : dk0;
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        // columns 16 kk .. + 15: 64-column half kk / 4, 32-byte slice kk % 4 of its rows
                        const uint32_t off = ((uint32_t)(kk >> 2) * kHalf + (uint32_t)(kk & 3) * 32u) >> 4;
                        tc05::mma_ss_lh(d, dq + off, dhi, dk + off, dhi, idesc_qk, kk > 0 ? 1u : 0u);
                    }
                    if (tile == 1) tc05::commit(bar(B_KE + (t & 1)));
                    tc05::commit(bar(B_SF + tile));
                }
            };
            auto pv = [&](int tile, int t) {
                const uint32_t pcol = tm + 128u * (uint32_t)tile, o = tm + kColO + (uint32_t)(D * tile), dv = t & 1 ? dv1 : dv0;
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {  // keys 16 kk .. + 15
                        const uint32_t vlo = dv + (uint32_t)kk * (2048u >> 4);
                        const uint32_t pa = pcol + 32u * (uint32_t)(kk >> 1) + 8u * (uint32_t)(kk & 1);
                        tc05::mma_ts_lh(o, pa, vlo, dhi, idesc_pv, (t > 0 || kk > 0) ? 1u : 0u);
                        tc05::mma_ts_lh(o, pa + 16u, vlo, dhi, idesc_pv, 1u);  // the remainders
                    }
                    if (tile == 1) tc05::commit(bar(B_VE + (t & 1)));
                    tc05::commit(bar(B_PD + tile));  // the last one is waited for before the CTA ends
                }
            };
            // whether a wait ran out (the same in every lane, as the compiler can see: the loop's counters stay uniform)
            auto gone = [&](int b, int phase) {
                const bool ok = mbar_wait(bar(b), (uint32_t)phase & 1u, f.err);
                tc05::fence_after_sync();
                return __any_sync(0xffffffffu, !ok);
            };
            if (!gone(B_KF, 0)) {
                qk(0, 0);
                qk(1, 0);
                for (int t = 0; t < nt; ++t) {
                    if (gone(B_VF + (t & 1), t >> 1)) break;
                    if (gone(B_PF + 0, t)) break;
                    pv(0, t);
                    if (t + 1 < nt) {
                        if (gone(B_KF + ((t + 1) & 1), (t + 1) >> 1)) break;
                        qk(0, t + 1);  // over S, and the P that the products before have read by then
                    }
                    if (gone(B_PF + 1, t)) break;
                    pv(1, t);
                    if (t + 1 < nt) qk(1, t + 1);
                }
            }
        }
        __syncwarp();
    } else if (warp < 8) {
        tc05::setmaxnreg_dec<kCodeRegs>();
        const int w = warp - 4;
        using C = Codes<D>;
        const uint8_t *pool = static_cast<const uint8_t *>(f.k_cache) + (long long)kvh * kv4::block_bytes(ps, D);
        const uint32_t stride = (uint32_t)f.Hkv * (uint32_t)kv4::block_bytes(ps, D);
        const int32_t *row = f.block_table + (long long)u.b * f.W;
        const uint32_t np = k_hi > 0 ? (uint32_t)((k_hi - 1) >> ps_shift) + 1 : 0;
        // page of a tile's turn; tiles behind the last may begin past 2^31 keys
        auto page = [&](int t, int i) { return ((uint32_t)(tile0 + t) * 128u + (uint32_t)C::first_row(i, w)) >> ps_shift; };
        auto look_up = [&](int t, int (&id)[C::kTurns]) {
#pragma unroll
            for (int i = 0; i < C::kTurns; ++i) id[i] = page(t, i) < np ? __ldg(row + page(t, i)) : -1;
        };
        auto check = [&](int t, int (&id)[C::kTurns]) {  // ids outside the pool read as zeros
#pragma unroll
            for (int i = 0; i < C::kTurns; ++i)
                if ((uint32_t)id[i] >= (uint32_t)f.num_pages) {
                    if (lane == 0 && page(t, i) < np)
                        atomicOr(f.err, (unsigned int)PA_ERRBIT_PAGE_RANGE);
                    id[i] = -1;
                }
        };
        C k, v;
        int now[C::kTurns], next[C::kTurns];
        look_up(0, now);
        check(0, now);
        k.load(pool, stride, now, 0, ps, w, lane);
        v.load(pool, stride, now, 1, ps, w, lane);
        look_up(1, next);
        bool bad = false;
#pragma unroll 1
        for (int t = 0; t < n_tiles && !bad; ++t) {
            const int slot = t & 1;
            check(t + 1, next);
            auto side = [&](C &x, int s, int empty, int full, uint32_t tile) {
                if (t >= 2) bad = bad || __any_sync(0xffffffffu, !mbar_wait(bar(empty + slot), ((t >> 1) - 1) & 1, f.err));
                if (bad) return;
                x.store(tile, w, lane);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(full + slot));
                if (t + 1 < n_tiles) x.load(pool, stride, next, s, ps, w, lane);
            };
            side(k, 0, B_KE, B_KF, sK(slot));
            side(v, 1, B_VE, B_VF, sV(slot));
            look_up(t + 2, next);
        }
    } else {
        tc05::setmaxnreg_inc<kSoftmaxRegs>();
        const int tile = (warp - 8) >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t sbuf = tmem + lane_addr + 128u * (uint32_t)tile, obuf = tmem + lane_addr + kColO + (uint32_t)(D * tile);
        const int tk = tile * half_tokens + r / f.G;
        const bool valid = r < half_tokens * f.G && tk < u.cnt;
        const int lim = valid ? row_key_limit(f, u.b, L, u.i + tk, u.n) : INT_MAX;
        s_row[tile * 128 + r] = valid ? (u.q0 + u.i + tk) * f.Hq + kvh * f.G + r % f.G : -1;
        const int all_below = __reduce_min_sync(0xffffffffu, lim);  // keys that every row of the warp sees
        const float factor = s_factor[tile * 128 + r];
        float ref = kNoRef;
        float2 l2 = make_float2(0.f, 0.f);  // sums of even and odd keys
        bool bad = false;
#pragma unroll 1
        for (int t = 0; t < n_tiles && !bad; ++t) {
            bad = __any_sync(0xffffffffu, !mbar_wait(bar(B_SF + tile), (uint32_t)t & 1u, f.err));
            if (bad) break;
            tc05::fence_after_sync();
            uint32_t s[4][32];
#pragma unroll
            for (int i = 0; i < 4; ++i) tc05::ld_32cols(sbuf + 32u * i, s[i]);
            tc05::wait_ld();
            const int j0 = (tile0 + t) * 128;
            if (j0 > all_below - 128) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (32 * i + j >= lim - j0) s[i][j] = 0xff800000u;
            }
            float m[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                m[i] = fmaxf(__uint_as_float(s[i][0]), __uint_as_float(s[i][1]));
#pragma unroll
                for (int j = 2; j < 32; j += 2) m[i] = fmaxf(fmaxf(m[i], __uint_as_float(s[i][j])), __uint_as_float(s[i][j + 1]));
            }
            const float mx = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * factor;
            const bool over = mx > ref + kRefMost;
            if (__any_sync(0xffffffffu, over)) {
                const float to = over ? mx - kRefBelow : ref;
                const float alpha = fast_exp2(ref - to);
                ref = to;
                l2.x *= alpha;
                l2.y *= alpha;
                if (t > 0) {
                    bad = __any_sync(0xffffffffu, !mbar_wait(bar(B_PD + tile), (uint32_t)(t - 1) & 1u, f.err));
                    if (bad) break;
                    tc05::fence_after_sync();
#pragma unroll 1
                    for (int c = 0; c < D / 16; ++c) {
                        uint32_t o[16];
                        tc05::ld_16cols(obuf + 16u * c, o);
                        tc05::wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
                        tc05::st_16cols(obuf + 16u * c, o);
                    }
                }
            }
            const float2 fac = make_float2(factor, factor), off = make_float2(-ref, -ref);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float2 x = fma2f(make_float2(__uint_as_float(s[i][2 * j]), __uint_as_float(s[i][2 * j + 1])), fac, off);
                    const float w0 = fast_exp2(x.x), w1 = fast_exp2(x.y);
                    l2 = add2f(l2, make_float2(w0, w1));
                    hi[j] = Op::pack(w0, w1);
                    lo[j] = remainder(hi[j], w0, w1);
                }
                tc05::st_16cols(sbuf + 32u * i, hi);
                tc05::st_16cols(sbuf + 32u * i + 16u, lo);
            }
            tc05::wait_st();
            tc05::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_PF + tile));
        }
        // ---- the row
        if (n_tiles > 0 && !bad)
            bad = __any_sync(0xffffffffu, !mbar_wait(bar(B_PD + tile), (uint32_t)(n_tiles - 1) & 1u, f.err));
        tc05::fence_after_sync();
        const float l = l2.x + l2.y, inv = l != 0.f ? 8.f / l : 0.f;  // a NaN stays one
        if (!bad) {
            const long long row = *(volatile long long *)&s_row[tile * 128 + r];
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                if (n_tiles > 0) {
                    tc05::ld_32cols(obuf + 32u * c, o);
                    tc05::wait_ld();
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = 0u;
                }
                // columns 0 1 2 .. 7 hold elements 0 4 1 5 2 6 3 7
                auto e = [&](int i, int x) {
                    return (x & 1 ? 1.f : kv4::kEvenShare) * __uint_as_float(o[8 * i + (x < 4 ? 2 * x : 2 * x - 7)]);
                };
                if (row >= 0 && p.part_out) {
                    float4 *dst = reinterpret_cast<float4 *>(p.part_out + (part * p.s.n_tok * f.Hq + row) * D + 32 * c);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        dst[2 * i] = make_float4(e(i, 0), e(i, 1), e(i, 2), e(i, 3));
                        dst[2 * i + 1] = make_float4(e(i, 4), e(i, 5), e(i, 6), e(i, 7));
                    }
                } else if (row >= 0) {
                    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<T *>(f.out) + row * D + 32 * c);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        auto pk = [&](int x) { return MmaOp<T>::pack(e(i, x) * inv, e(i, x + 1) * inv); };
                        dst[i] = make_uint4(pk(0), pk(2), pk(4), pk(6));
                    }
                }
            }
            if (row >= 0 && p.part_out)
                *reinterpret_cast<float2 *>(p.part_state + 2 * (part * p.s.n_tok * f.Hq + row)) = make_float2(ref, l);
            else if (row >= 0 && f.lse)
                f.lse[row] = l != 0.f ? ref * kLn2 + logf(l) : kNegInf;
        }
    }
    tc05::fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        tc05::fence_after_sync();
        tc05::tmem_dealloc(tmem, 512);
    }
}

// The parts of rows whose keys several CTAs shared, a warp a row.
template <typename T, int D>
__global__ void __launch_bounds__(256) paged_attn_kv4_join_runs_kernel(const Kv4Params p) {
    const FwdParams &f = p.s.f;
    const int lane = threadIdx.x & 31, unit = blockIdx.x / 32, kvh = unit % f.Hkv;
    const Tile u = find_tile(p, unit / f.Hkv, lane);
    const int tr = (blockIdx.x % 32) * 8 + (threadIdx.x >> 5), r = tr & 127, half_tokens = p.TT / 2;
    const int tk = (tr >> 7) * half_tokens + r / f.G;
    if (r >= half_tokens * f.G || tk >= u.cnt) return;
    const long long row = (u.q0 + u.i + tk) * f.Hq + kvh * f.G + r % f.G, rows = p.s.n_tok * f.Hq;
    const float2 *state = reinterpret_cast<const float2 *>(p.part_state) + row;
    float M = kNoRef, sum = 0.f;
    for (int x = 0; x < p.S; ++x) M = fmaxf(M, __ldcg(state + x * rows).x);
    constexpr int C = D / 4;  // lanes with elements
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int x = 0; x < p.S; ++x) {
        const float2 st = __ldcg(state + x * rows);
        const float k = fast_exp2(st.x - M);
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(p.part_out + (x * rows + row) * D) + lane % C);
        sum += k * st.y;
        o.x += k * v.x, o.y += k * v.y, o.z += k * v.z, o.w += k * v.w;
    }
    const float inv = sum != 0.f ? 8.f / sum : 0.f;  // a NaN stays one
    if (lane < C)
        *reinterpret_cast<uint2 *>(static_cast<T *>(f.out) + row * D + 4 * lane) =
            make_uint2(MmaOp<T>::pack(o.x * inv, o.y * inv), MmaOp<T>::pack(o.z * inv, o.w * inv));
    if (lane == 0 && f.lse) f.lse[row] = sum != 0.f ? M * kLn2 + logf(sum) : kNegInf;
}

template <typename T, int D>
static cudaError_t launch_tc(const Kv4Params &p, long long units, cudaStream_t stream) {
    auto kern = paged_attn_kv4_tc05_kernel<T, D>;
    constexpr size_t smem = 6 * (D / 64) * kHalf + 1024;
    static SmemLimit limit;
    cudaError_t e = limit.raise((const void *)kern, smem);
    if (e != cudaSuccess) return e;
    // The softmax warps' register increase is served from what the launch holds: a build that gave the kernel fewer
    // registers a thread would leave them waiting, so it is refused.
    static std::atomic<int> launch_regs{0};
    int regs = launch_regs.load(std::memory_order_relaxed);
    if (!regs) {
        cudaFuncAttributes fa;
        if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
        regs = fa.numRegs;
        launch_regs.store(regs, std::memory_order_relaxed);
    }
    if (regs * kThreads < 128 * (int)(kIssueRegs + kCodeRegs) + 256 * (int)kSoftmaxRegs) return cudaErrorInvalidConfiguration;
    const FwdParams &f = p.s.f;
    kern<<<(unsigned)(units * p.S), kThreads, smem, stream>>>(p, f.ps == 16 ? 4 : f.ps == 32 ? 5 : 6,
                                                              tc05::idesc_f16(false, false, 128, 128),
                                                              tc05::idesc_f16(false, true, 128, D));
    return cudaGetLastError();
}

// What the launches of a call have in common; units: tiles x kv heads.
static Kv4Params runs_params(const SparseParams &sp, int S, long long &units) {
    const FwdParams &f = sp.f;
    Kv4Params p{};
    p.s = sp;
    p.s.group_min = 0;
    p.min_tokens = sp.group_min;
    p.TT = kv4_tile_tokens(f.D, f.G);
    p.seq_tiles = f.q_start ? 0 : (f.Sq + p.TT - 1) / p.TT;
    p.S = S;
    if (S > 1) {
        p.part_out = static_cast<float *>(sp.ws);
        p.part_state = p.part_out + S * sp.n_tok * f.Hq * f.D;
    }
    units = (f.q_start ? sp.n_tok / p.TT + f.B : (long long)f.B * p.seq_tiles) * f.Hkv;
    return p;
}

int kv4_tile_tokens(int D, int G) { return D == 256 || G > 128 ? 0 : 2 * (128 / G); }

cudaError_t launch_kv4_tc05(const SparseParams &sp, int dtype, int S, cudaStream_t stream) {
    long long units;
    const Kv4Params p = runs_params(sp, S, units);
    if (units == 0) return cudaSuccess;
    if (units * S > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (dtype == PA_BF16)
        return sp.f.D == 64 ? launch_tc<__nv_bfloat16, 64>(p, units, stream) : launch_tc<__nv_bfloat16, 128>(p, units, stream);
    return sp.f.D == 64 ? launch_tc<__half, 64>(p, units, stream) : launch_tc<__half, 128>(p, units, stream);
}

cudaError_t launch_kv4_join_runs(const SparseParams &sp, int dtype, int S, cudaStream_t stream) {
    long long units;
    const Kv4Params p = runs_params(sp, S, units);
    if (units == 0) return cudaSuccess;
    if (units * 32 > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    auto kern = dtype == PA_BF16
                    ? sp.f.D == 64 ? paged_attn_kv4_join_runs_kernel<__nv_bfloat16, 64> : paged_attn_kv4_join_runs_kernel<__nv_bfloat16, 128>
                    : sp.f.D == 64 ? paged_attn_kv4_join_runs_kernel<__half, 64> : paged_attn_kv4_join_runs_kernel<__half, 128>;
    kern<<<(unsigned)(units * 32), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace pa
