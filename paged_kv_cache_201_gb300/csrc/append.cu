// New tokens' K and V rows into their slots, and the envelopes of the pages they land in.
//
// One warp per kv head and TPW consecutive tokens copies their rows.  The warp that holds the last new
// token of a page also takes the page's smallest and largest key elements over rows 0 .. r: minima and
// maxima are exact whatever their order, so an envelope is the same bits whether a page is filled at
// once or token by token.  Rows of this call's run come from k_new (their stores by other warps may still
// be under way), older rows from the cache; for a prompt they are in L2, just read by the neighbours.
// A decode step is a chain of three trips to memory (slots, rows, stores).
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

// The envelope of the page that token t (slot `slot`) closes, by one warp; run: tokens t - run + 1 .. t
// lie in the page's rows up to slot's.
template <typename T, int D>
__device__ __forceinline__ void page_envelope(const AppendParams &p, int t, int h, int slot, int run, int lane) {
    constexpr int E = 16 / (int)sizeof(T);       // elements of a chunk
    constexpr int CH = D / E;                    // chunks of a row
    constexpr int LPR = CH < 32 ? CH : 32;       // lanes of a row
    constexpr int CPL = CH / LPR;                // chunks of a lane
    constexpr int RPI = 32 / LPR;                // rows a warp reads at once
    constexpr int U = 8 / CPL;                   // such reads on their way together
    const int ps = 1 << p.ps_shift, row = slot & (ps - 1);
    const int c0 = lane % LPR, r0 = lane / LPR;
    const long long row_elems = (long long)p.Hkv * D;
    const T *fresh = static_cast<const T *>(p.k_new) + h * D + t * p.k_stride;
    const T *page = static_cast<const T *>(p.k_cache) + (slot - row) * row_elems + h * D;
    float lo[CPL][E], hi[CPL][E];
#pragma unroll
    for (int i = 0; i < CPL; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) lo[i][e] = INFINITY, hi[i][e] = -INFINITY;
    bool odd = false;  // an infinity or a NaN among the keys
    for (int r1 = 0; r1 <= row; r1 += RPI * U) {
        uint4 u[U][CPL];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int r = min(r1 + k * RPI + r0, row);  // past the last row, that row again
            const T *src = row - r < run ? fresh - (row - r) * p.k_stride : page + r * row_elems;
#pragma unroll
            for (int i = 0; i < CPL; ++i) u[k][i] = reinterpret_cast<const uint4 *>(src)[c0 + i * LPR];
        }
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
            for (int i = 0; i < CPL; ++i) {
                float x[E];
                unpack16<T>(u[k][i], x);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    odd |= !(fabsf(x[e]) <= FLT_MAX);
                    lo[i][e] = fminf(lo[i][e], x[e]);
                    hi[i][e] = fmaxf(hi[i][e], x[e]);
                }
            }
    }
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < CPL; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) {
#pragma unroll
            for (int o = LPR; o < 32; o <<= 1) {
                lo[i][e] = fminf(lo[i][e], __shfl_xor_sync(0xffffffffu, lo[i][e], o));
                hi[i][e] = fmaxf(hi[i][e], __shfl_xor_sync(0xffffffffu, hi[i][e], o));
            }
            a = fmaxf(a, fmaxf(fabsf(lo[i][e]), fabsf(hi[i][e])));
        }
    a = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(a)));  // not negative: ordered as bits
    odd = __any_sync(0xffffffffu, odd);
    const long long unit = (long long)(slot >> p.ps_shift) * p.Hkv + h;
    if (lane == 0) p.env_scale[unit] = odd ? INFINITY : __fdiv_rn(a, 127.f);
    if (r0 != 0) return;
    const float inv = 127.f / a;
#pragma unroll
    for (int i = 0; i < CPL; ++i)
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            float(&x)[E] = side ? hi[i] : lo[i];
            if (!odd && a > 0.f)
                quantise8<E>(x, a, inv);
            else
#pragma unroll
                for (int e = 0; e < E; ++e) x[e] = 0.f;
            uint32_t w[E / 4];
#pragma unroll
            for (int e = 0; e < E; e += 4)
                w[e / 4] = ((int)x[e] & 0xff) | ((int)x[e + 1] & 0xff) << 8 | ((int)x[e + 2] & 0xff) << 16 |
                           (unsigned)(int)x[e + 3] << 24;
            int8_t *dst = p.env + (unit * 2 + side) * D + (c0 + i * LPR) * E;
            if constexpr (E == 8)
                *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
            else
                *reinterpret_cast<uint32_t *>(dst) = w[0];
        }
}

}  // namespace

template <typename T, int D, int TPW>
__global__ void __launch_bounds__(256) paged_attn_append_kernel(const AppendParams p) {
    constexpr int CH = D * (int)sizeof(T) / 16;  // 16-byte chunks of a row
    constexpr int N = (2 * CH + 31) / 32;        // of a token's two rows, per lane
    const long long unit = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const long long group = unit / p.Hkv;
    const int h = (int)(unit - group * p.Hkv);
    if (group * TPW >= p.T) return;
    const int t0 = (int)group * TPW;
    // slots t0 - 64 .. t0 + TPW, one trip: lane l holds t0 + TPW - 1 - l, t0 + TPW - 33 - l, ...
    const int tl = min(t0 + TPW, p.T) - 1;  // the warp's last token
    const int s_next = tl + 1 < p.T ? p.slots[tl + 1] : -1;
    int s[3];
#pragma unroll
    for (int i = 0; i < 3; ++i)
        s[i] = tl - i * 32 - lane >= 0 && (i == 0 || p.env) ? p.slots[tl - i * 32 - lane] : -1;

    int slot[TPW];
    uint4 v[TPW][N];
    const long long row_elems = (long long)p.Hkv * D;
#pragma unroll
    for (int k = 0; k < TPW; ++k) {  // token tl - k
        slot[k] = __shfl_sync(0xffffffffu, s[0], k);
        const bool on = tl - k >= t0 && slot[k] >= 0 && slot[k] < p.num_slots;
        if (!on) {
            if (tl - k >= t0 && slot[k] != -1 && lane == 0) atomicOr(p.err, (unsigned int)PA_ERRBIT_PAGE_RANGE);
            slot[k] = -1;
            continue;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = i * 32 + lane;
            const T *src = c < CH ? static_cast<const T *>(p.k_new) + (tl - k) * p.k_stride
                                  : static_cast<const T *>(p.v_new) + (tl - k) * p.v_stride;
            if (c < 2 * CH) v[k][i] = reinterpret_cast<const uint4 *>(src + h * D)[c < CH ? c : c - CH];
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
    if (!p.env) return;
    const int ps = 1 << p.ps_shift;
#pragma unroll 1
    for (int k = 0; k < TPW; ++k) {
        const int t = tl - k;
        const int mine = __shfl_sync(0xffffffffu, s[0], k), next = k == 0 ? s_next : __shfl_sync(0xffffffffu, s[0], k - 1);
        if (t < t0 || mine < 0 || mine >= p.num_slots) continue;
        const int row = mine & (ps - 1);
        if (row != ps - 1 && next == mine + 1) continue;  // a later token closes the page
        // token tl - l lies in the page's run if its slot is l - k rows before token t's
        unsigned long long in = 0;  // bit j: token t - j
#pragma unroll
        for (int i = 2; i >= 0; --i) {
            const int j = i * 32 + lane - k;
            const unsigned b = __ballot_sync(0xffffffffu, j >= 0 && j <= row && s[i] == mine - j);
            in |= i * 32 - k >= 0 ? (i * 32 - k < 64 ? (unsigned long long)b << (i * 32 - k) : 0ull) : (unsigned long long)(b >> k);
        }
        const int run = ~in ? __ffsll((long long)~in) - 1 : 64;
        page_envelope<T, D>(p, t, h, mine, run, lane);
    }
}

template <typename T, int D>
static cudaError_t launch_append_d(const AppendParams &p, cudaStream_t stream) {
    // Several tokens a warp once there are warps for every multiprocessor many times over.
    const bool many = (long long)p.T * p.Hkv >= 16384;
    const long long blocks = ((long long)(many ? (p.T + 3) / 4 : p.T) * p.Hkv + 7) / 8;
    if (blocks == 0) return cudaSuccess;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (many)
        paged_attn_append_kernel<T, D, 4><<<(unsigned)blocks, 256, 0, stream>>>(p);
    else
        paged_attn_append_kernel<T, D, 1><<<(unsigned)blocks, 256, 0, stream>>>(p);
    return cudaGetLastError();
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
