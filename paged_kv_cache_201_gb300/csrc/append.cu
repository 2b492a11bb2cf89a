// New tokens' K and V rows into their slots, and the envelopes of the pages they land in.
//
// One launch of two kinds of CTAs.  The copying ones move rows, a warp for one kv head of TPW tokens.  The
// others, placed first in the grid, take the envelopes: a warp finds the tokens that close a page (none of
// the next 64 tokens lies in it) and takes the smallest and largest key elements of the page's rows
// 0 .. r, from k_new where this call writes them (told by the slots of the 63 tokens before) and from the
// cache where an earlier one did; it waits for no copy.  Minima and maxima are exact whatever their
// order, so an envelope is the same bits whether a page is filled at once or token by token.
// Kept apart, the long chain of an envelope (slots, rows, reduction, division) overlaps the copies; where
// few pages close, as in a prompt, the CTA's warps share a page's rows.  6656 prompt tokens of 8 heads of
// 128 (f16, 64-token pages) take 14.1 us, 58 % of the copy rate; with the closing warps among the copying
// ones they took 21, and the copies alone take 10.7.  A decode step of 256 tokens takes 5.4 us, a chain
// of three trips to memory.
#include <float.h>

#include "sparse_common.cuh"

namespace pa {

namespace {

// Eight 16-bit or four 32-bit elements of a 16-byte chunk.
template <typename T>
__device__ __forceinline__ void unpack16(uint4 u, float (&v)[16 / sizeof(T)]) {
    if constexpr (sizeof(T) == 4) {
        v[0] = __uint_as_float(u.x), v[1] = __uint_as_float(u.y);
        v[2] = __uint_as_float(u.z), v[3] = __uint_as_float(u.w);
    } else {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = MmaOp<T>::unpack(w[i]);
            v[2 * i] = f.x, v[2 * i + 1] = f.y;
        }
    }
}

constexpr int kOld = 255;  // a row that an earlier call wrote

// How a warp reads rows of one kv head, 16 bytes a lane.
template <typename T, int D>
struct Rows {
    static constexpr int E = 16 / (int)sizeof(T);  // elements of a chunk
    static constexpr int CH = D / E;               // chunks of a row
    static constexpr int LPR = CH < 32 ? CH : 32;  // lanes of a row
    static constexpr int CPL = CH / LPR;           // chunks of a lane
    static constexpr int RPI = 32 / LPR;           // rows a warp reads at once
    static constexpr int U = 8 / CPL;              // such reads on their way together
};

// A page that gets its last new token of the call: rows 0 .. row; row r is token t - from[r]'s, or the
// cache's where from[r] is kOld.
struct Closing {
    int t, page, row;  // row < 0: none
    uint8_t from[64];
};

// The smallest and largest elements of rows [r1, r2) of a closing page, by one warp: lane l of each group
// of LPR lanes ends up with chunks l, l + LPR of both.  Returns whether an element is not finite.
template <typename T, int D>
__device__ __forceinline__ bool row_bounds(const AppendParams &p, const Closing &cl, int h, int r1, int r2,
                                           float (&lo)[Rows<T, D>::CPL][Rows<T, D>::E],
                                           float (&hi)[Rows<T, D>::CPL][Rows<T, D>::E], int lane) {
    using R = Rows<T, D>;
    const int c0 = lane % R::LPR, r0 = lane / R::LPR;
    const long long row_elems = (long long)p.Hkv * D;
    const T *fresh = static_cast<const T *>(p.k_new) + h * D + cl.t * p.k_stride;
    const T *page = static_cast<const T *>(p.k_cache) + ((long long)cl.page << p.ps_shift) * row_elems + h * D;
#pragma unroll
    for (int i = 0; i < R::CPL; ++i)
#pragma unroll
        for (int e = 0; e < R::E; ++e) lo[i][e] = INFINITY, hi[i][e] = -INFINITY;
    bool odd = false;
    for (int r3 = r1; r3 < r2; r3 += R::RPI * R::U) {
        uint4 u[R::U][R::CPL];
#pragma unroll
        for (int k = 0; k < R::U; ++k) {
            const int r = min(r3 + k * R::RPI + r0, r2 - 1);  // past the last row, that row again
            const int back = cl.from[r];
            const T *src = back != kOld ? fresh - back * p.k_stride : page + r * row_elems;
#pragma unroll
            for (int i = 0; i < R::CPL; ++i) u[k][i] = reinterpret_cast<const uint4 *>(src)[c0 + i * R::LPR];
        }
#pragma unroll
        for (int k = 0; k < R::U; ++k)
#pragma unroll
            for (int i = 0; i < R::CPL; ++i) {
                float x[R::E];
                unpack16<T>(u[k][i], x);
#pragma unroll
                for (int e = 0; e < R::E; ++e) {
                    odd |= !(fabsf(x[e]) <= FLT_MAX);
                    lo[i][e] = fminf(lo[i][e], x[e]);
                    hi[i][e] = fmaxf(hi[i][e], x[e]);
                }
            }
    }
#pragma unroll
    for (int i = 0; i < R::CPL; ++i)
#pragma unroll
        for (int e = 0; e < R::E; ++e)
#pragma unroll
            for (int o = R::LPR; o < 32; o <<= 1) {
                lo[i][e] = fminf(lo[i][e], __shfl_xor_sync(0xffffffffu, lo[i][e], o));
                hi[i][e] = fmaxf(hi[i][e], __shfl_xor_sync(0xffffffffu, hi[i][e], o));
            }
    return __any_sync(0xffffffffu, odd);
}

// A closing page's envelope by one warp.
template <typename T, int D>
__device__ __forceinline__ void warp_envelope(const AppendParams &p, const Closing &cl, bool twice, int h, int lane) {
    using R = Rows<T, D>;
    float lo[R::CPL][R::E], hi[R::CPL][R::E];
    const bool odd = row_bounds<T, D>(p, cl, h, 0, cl.row + 1, lo, hi, lane) || twice;
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < R::CPL; ++i)
#pragma unroll
        for (int e = 0; e < R::E; ++e) a = fmaxf(a, fmaxf(fabsf(lo[i][e]), fabsf(hi[i][e])));
    a = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(a)));  // not negative: ordered as bits
    const long long unit = (long long)cl.page * p.Hkv + h;
    if (lane == 0) p.env_scale[unit] = odd ? INFINITY : __fdiv_rn(a, 127.f);
    if (lane >= R::LPR) return;
    const float inv = 127.f / a;
#pragma unroll
    for (int i = 0; i < R::CPL; ++i)
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            float(&x)[R::E] = side ? hi[i] : lo[i];
            if (!odd && a > 0.f)
                quantise8<R::E>(x, a, inv);
            else
#pragma unroll
                for (int e = 0; e < R::E; ++e) x[e] = 0.f;
            uint32_t w[R::E / 4];
#pragma unroll
            for (int e = 0; e < R::E; e += 4)
                w[e / 4] = ((int)x[e] & 0xff) | ((int)x[e + 1] & 0xff) << 8 | ((int)x[e + 2] & 0xff) << 16 |
                           (unsigned)(int)x[e + 3] << 24;
            int8_t *dst = p.env + (unit * 2 + side) * D + (lane + i * R::LPR) * R::E;
            if constexpr (R::E == 8)
                *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
            else
                *reinterpret_cast<uint32_t *>(dst) = w[0];
        }
}

constexpr int kAppendThreads = 128, kAppendWarps = 4;

// The envelopes of one or two closing pages by a CTA: SPLIT warps share a page's rows.  s_part:
// [kAppendWarps][2][D] partial bounds, s_max: [kAppendWarps / SPLIT] zeros.
template <typename T, int D, int SPLIT>
__device__ __forceinline__ void cta_envelope(const AppendParams &p, const Closing &cl, bool twice, int h,
                                             float *s_part, unsigned *s_max, int warp, int lane) {
    using R = Rows<T, D>;
    constexpr int EPT = D / (SPLIT * 32) > 0 ? D / (SPLIT * 32) : 1;  // elements of a thread in the second half
    const int part = warp % SPLIT, n = cl.row + 1, share = (n + SPLIT - 1) / SPLIT;
    const int r1 = min(part * share, n), r2 = min(r1 + share, n);
    float lo[R::CPL][R::E], hi[R::CPL][R::E];
    const bool odd = row_bounds<T, D>(p, cl, h, r1, r2, lo, hi, lane) || twice;
    if (lane < R::LPR) {
#pragma unroll
        for (int i = 0; i < R::CPL; ++i)
#pragma unroll
            for (int e = 0; e < R::E; ++e) {
                s_part[2 * warp * D + (lane + i * R::LPR) * R::E + e] = lo[i][e];
                s_part[(2 * warp + 1) * D + (lane + i * R::LPR) * R::E + e] = hi[i][e];
            }
    }
    unsigned *top = s_max + warp / SPLIT;  // bits of the largest |element|; a NaN where one is not finite
    if (odd && lane == 0) atomicMax(top, 0x7fffffffu);
    __syncthreads();
    const float *first = s_part + 2 * (warp - part) * D;
    const int d0 = part * 32 + lane;
    float x[2][EPT];
    unsigned a = 0;
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
        const int d = d0 + i * SPLIT * 32;
        x[0][i] = INFINITY, x[1][i] = -INFINITY;
        if (d >= D) continue;
#pragma unroll
        for (int w = 0; w < SPLIT; ++w) {
            x[0][i] = fminf(x[0][i], first[2 * w * D + d]);
            x[1][i] = fmaxf(x[1][i], first[(2 * w + 1) * D + d]);
        }
        a = max(a, __float_as_uint(fmaxf(fabsf(x[0][i]), fabsf(x[1][i]))));
    }
    a = __reduce_max_sync(0xffffffffu, a);
    if (lane == 0) atomicMax(top, a);
    __syncthreads();
    a = *top;
    const float big = __uint_as_float(a);
    const long long unit = (long long)cl.page * p.Hkv + h;
    if (part == 0 && lane == 0) p.env_scale[unit] = a >= 0x7f800000u ? INFINITY : __fdiv_rn(big, 127.f);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        if (a < 0x7f800000u && a > 0)
            quantise8<EPT>(x[side], big, 127.f / big);
        else
#pragma unroll
            for (int i = 0; i < EPT; ++i) x[side][i] = 0.f;
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            const int d = d0 + i * SPLIT * 32;
            if (d < D) p.env[(unit * 2 + side) * D + d] = (int8_t)(int)x[side][i];
        }
    }
}

}  // namespace

// TPW: tokens of a copying warp; ET: tokens of an envelope CTA.
template <typename T, int D, int TPW, int ET>
__global__ void __launch_bounds__(kAppendThreads) paged_attn_append_kernel(const AppendParams p, int env_ctas) {
    constexpr int CH = D * (int)sizeof(T) / 16;  // 16-byte chunks of a row
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    if ((int)blockIdx.x < env_ctas) {
        const int t0 = (int)(blockIdx.x / p.Hkv) * ET, h = blockIdx.x % p.Hkv;
        __shared__ int s_slot[ET + 128];  // of tokens t0 - 64 ..
        for (int i = threadIdx.x; i < ET + 128; i += kAppendThreads) {
            const int t = t0 - 64 + i;
            s_slot[i] = t >= 0 && t < p.T ? p.slots[t] : -1;
        }
        __shared__ Closing s_close[kAppendWarps];
        __shared__ unsigned s_max[2];
        __shared__ bool s_closes[ET];
        __shared__ __align__(16) float s_part[kAppendWarps * 2 * D];
        Closing &cl = s_close[warp];
        if (threadIdx.x < 2) s_max[threadIdx.x] = 0u;
        __syncthreads();
        auto here = [&](int slot, int page) { return slot >= 0 && slot >> p.ps_shift == page; };
#pragma unroll
        for (int k = warp; k < ET; k += kAppendWarps) {
            const int mine = s_slot[64 + k], page = mine >> p.ps_shift;
            const bool later = here(s_slot[65 + k + lane], page) || (k + 97 + lane < ET + 128 && here(s_slot[k + 97 + lane], page));
            const bool any = __any_sync(0xffffffffu, later);
            if (lane == 0) s_closes[k] = mine >= 0 && mine < p.num_slots && !any;
        }
        __syncthreads();
        const unsigned closes = __ballot_sync(0xffffffffu, lane < ET && s_closes[lane < ET ? lane : 0]);
        const int n = __popc(closes);
        // the c-th closing token's page: its rows' sources.  Returns whether two tokens name a row: either may end up
        // in the cache, so the page has no bound, as one with a non-finite key.
        auto look_up = [&](int c) {
            const int k = (int)__fns(closes, 0, c + 1), page = s_slot[64 + k] >> p.ps_shift;
            cl.from[lane] = cl.from[lane + 32] = kOld;
            __syncwarp();
            int row = 0, tokens = 0;
            unsigned long long rows = 0;
#pragma unroll
            for (int back = lane; back < 64; back += 32) {
                const int x = s_slot[64 + k - back];
                const bool on = here(x, page);
                tokens += __popc(__ballot_sync(0xffffffffu, on));
                if (on) {
                    const int r = x & ((1 << p.ps_shift) - 1);
                    cl.from[r] = (uint8_t)back;
                    rows |= 1ull << r;
                    row = max(row, r);
                }
            }
            row = __reduce_max_sync(0xffffffffu, row);
            const int named = __popc(__reduce_or_sync(0xffffffffu, (unsigned)rows)) +
                              __popc(__reduce_or_sync(0xffffffffu, (unsigned)(rows >> 32)));
            if (lane == 0) {
                cl.t = t0 + k;
                cl.page = page;
                cl.row = row;
            }
            __syncwarp();
            return named != tokens;
        };
        if (n == 1) {  // as in a prompt
            const bool twice = look_up(0);
            cta_envelope<T, D, 4>(p, cl, twice, h, s_part, s_max, warp, lane);
        } else if (n == 2) {
            const bool twice = look_up(warp / 2);
            cta_envelope<T, D, 2>(p, cl, twice, h, s_part, s_max, warp, lane);
        } else {
#pragma unroll 1
            for (int c = warp; c < n; c += kAppendWarps) {
                const bool twice = look_up(c);
                warp_envelope<T, D>(p, cl, twice, h, lane);
                __syncwarp();  // before cl is written for another page
            }
        }
        return;
    }

    constexpr int N = (2 * CH + 31) / 32;  // chunks of a token's two rows, per lane
    const long long unit = (long long)(blockIdx.x - env_ctas) * kAppendWarps + warp;
    const long long group = unit / p.Hkv;
    const int h = (int)(unit - group * p.Hkv);
    if (group * TPW >= p.T) return;
    const int t0 = (int)group * TPW;
    const int mine = lane < TPW && t0 + lane < p.T ? p.slots[t0 + lane] : -1;
    if (mine != -1 && (mine < 0 || mine >= p.num_slots)) atomicOr(p.err, (unsigned int)PA_ERRBIT_PAGE_RANGE);
    const long long row_elems = (long long)p.Hkv * D;
    int slot[TPW];
    uint4 v[TPW][N];
#pragma unroll
    for (int k = 0; k < TPW; ++k) {
        slot[k] = __shfl_sync(0xffffffffu, mine, k);
        if (slot[k] < 0 || slot[k] >= p.num_slots) {
            slot[k] = -1;
            continue;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = i * 32 + lane;
            const T *src = c < CH ? static_cast<const T *>(p.k_new) + (t0 + k) * p.k_stride
                                  : static_cast<const T *>(p.v_new) + (t0 + k) * p.v_stride;
            if (c < 2 * CH) v[k][i] = __ldg(reinterpret_cast<const uint4 *>(src + h * D) + (c < CH ? c : c - CH));
        }
    }
#pragma unroll
    for (int k = 0; k < TPW; ++k) {
        if (slot[k] < 0) continue;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = i * 32 + lane;
            T *dst = static_cast<T *>(c < CH ? p.k_cache : p.v_cache) + slot[k] * row_elems + h * D;
            if (c < 2 * CH) reinterpret_cast<uint4 *>(dst)[c < CH ? c : c - CH] = v[k][i];
        }
    }
}

template <typename T, int D, int TPW, int ET>
static cudaError_t launch_append_k(const AppendParams &p, cudaStream_t stream) {
    const long long env = p.env ? ((long long)p.T + ET - 1) / ET * p.Hkv : 0;
    const long long units = ((long long)p.T + TPW - 1) / TPW * p.Hkv;
    const long long blocks = env + (units + kAppendWarps - 1) / kAppendWarps;
    if (blocks == 0) return cudaSuccess;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    paged_attn_append_kernel<T, D, TPW, ET><<<(unsigned)blocks, kAppendThreads, 0, stream>>>(p, (int)env);
    return cudaGetLastError();
}

template <typename T, int D>
static cudaError_t launch_append_d(const AppendParams &p, cudaStream_t stream) {
    // Prompts (warps for every multiprocessor many times over): several tokens a warp and few closing
    // pages among them (14.1 us as above; 27.7 with one token a warp); single tokens: a warp each, most of
    // them closing a page (1024 of 8 heads 11.3 us, 20.9 the other way).  The rule cannot tell a very large batch of
    // single tokens from a prompt: 2048 take 28.9 us with the first plan, 21.1 with the second, 4096 take 47 and 46.
    if ((long long)p.T * p.Hkv >= 16384) return launch_append_k<T, D, 4, 32>(p, stream);
    return launch_append_k<T, D, 1, 4>(p, stream);
}

template <typename T>
static cudaError_t launch_append_t(const AppendParams &p, int D, cudaStream_t stream) {
    if (D == 64) return launch_append_d<T, 64>(p, stream);
    if (D == 128) return launch_append_d<T, 128>(p, stream);
    return launch_append_d<T, 256>(p, stream);
}

cudaError_t launch_append(const AppendParams &p, int dtype, int D, cudaStream_t stream) {
    if (dtype == PA_F32) return launch_append_t<float>(p, D, stream);
    if (dtype == PA_BF16) return launch_append_t<__nv_bfloat16>(p, D, stream);
    return launch_append_t<__half>(p, D, stream);
}

}  // namespace pa
