// New tokens' K and V rows into their slots, and the envelopes of the pages they land in.
//
// One warp per (token, kv head) copies its two rows.  The warp of the last new token of a page also
// takes the page's smallest and largest key elements over rows 0 .. r: minima and maxima are exact
// whatever their order, so an envelope is the same bits whether a page is filled at once or token by
// token.  Rows of this call's run come from k_new (their stores by other warps may still be under
// way), older rows from the cache.
#include <float.h>

#include "sparse_common.cuh"

namespace pa {

namespace {

template <typename T>
__device__ __forceinline__ void load4(const T *src, float (&v)[4]) {
    if constexpr (sizeof(T) == 4) {
        const float4 x = *reinterpret_cast<const float4 *>(src);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
        const uint2 x = *reinterpret_cast<const uint2 *>(src);
        const float2 a = MmaOp<T>::unpack(x.x), b = MmaOp<T>::unpack(x.y);
        v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
    }
}

}  // namespace

template <typename T, int D>
__global__ void __launch_bounds__(256) paged_attn_append_kernel(const AppendParams p) {
    constexpr int kRowChunks = D * (int)sizeof(T) / 16;  // 16-byte chunks of a row
    constexpr int kQuads = D / 4;                        // 4-element groups of a row
    constexpr int NQ = (kQuads + 31) / 32;               // per lane
    const long long unit = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (unit >= (long long)p.T * p.Hkv) return;
    const int t = (int)(unit / p.Hkv), h = (int)(unit - (long long)t * p.Hkv);
    const int slot = p.slots[t];
    if (slot < 0 || slot >= p.num_slots) {
        if (slot != -1 && lane == 0) atomicOr(p.err, (unsigned int)PA_ERRBIT_PAGE_RANGE);
        return;
    }
    const T *kn = static_cast<const T *>(p.k_new) + h * D;
    const T *vn = static_cast<const T *>(p.v_new) + h * D;
    const uint4 *ks = reinterpret_cast<const uint4 *>(kn + t * p.k_stride);
    const uint4 *vs = reinterpret_cast<const uint4 *>(vn + t * p.v_stride);
    const long long row_elems = (long long)p.Hkv * D;
    uint4 *kd = reinterpret_cast<uint4 *>(static_cast<T *>(p.k_cache) + slot * row_elems + h * D);
    uint4 *vd = reinterpret_cast<uint4 *>(static_cast<T *>(p.v_cache) + slot * row_elems + h * D);
#pragma unroll
    for (int c = lane; c < kRowChunks; c += 32) {
        kd[c] = ks[c];
        vd[c] = vs[c];
    }
    if (!p.env) return;

    const int ps = 1 << p.ps_shift;
    const int row = slot & (ps - 1);
    if (row != ps - 1 && t + 1 < p.T && p.slots[t + 1] == slot + 1) return;  // a later token closes the page
    // rows [row - run, row] are this call's tokens t - run .. t
    unsigned long long mine = 0;
    for (int j0 = 0; j0 < ps; j0 += 32) {
        const int j = j0 + lane;  // row row - j by token t - j
        const bool ok = j <= row && j <= t && p.slots[t - j] == slot - j;
        mine |= (unsigned long long)__ballot_sync(0xffffffffu, ok) << j0;
    }
    const int run = ~mine ? __ffsll((long long)~mine) - 1 : 64;  // tokens of the run, t itself included
    float lo[NQ][4], hi[NQ][4];
#pragma unroll
    for (int i = 0; i < NQ; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) lo[i][e] = INFINITY, hi[i][e] = -INFINITY;
    bool odd = false;  // an infinity or a NaN among the keys
    const T *page = static_cast<const T *>(p.k_cache) + (slot - row) * row_elems + h * D;
    for (int r = 0; r <= row; ++r) {
        const T *src = row - r < run ? kn + (t - (row - r)) * p.k_stride : page + r * row_elems;
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            const int g = lane + i * 32;
            if (kQuads % 32 == 0 || g < kQuads) {
                float x[4];
                load4(src + g * 4, x);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    odd |= !(fabsf(x[e]) <= FLT_MAX);
                    lo[i][e] = fminf(lo[i][e], x[e]);
                    hi[i][e] = fmaxf(hi[i][e], x[e]);
                }
            }
        }
    }
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < NQ; ++i)
        if (kQuads % 32 == 0 || lane + i * 32 < kQuads)
#pragma unroll
            for (int e = 0; e < 4; ++e) a = fmaxf(a, fmaxf(fabsf(lo[i][e]), fabsf(hi[i][e])));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    odd = __any_sync(0xffffffffu, odd);
    const long long unit_out = (long long)(slot >> p.ps_shift) * p.Hkv + h;
    char4 *env = reinterpret_cast<char4 *>(p.env + unit_out * 2 * D);
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        const int g = lane + i * 32;
        if (kQuads % 32 != 0 && g >= kQuads) continue;
        char4 cl = make_char4(0, 0, 0, 0), ch = cl;
        if (!odd && a > 0.f) {
            const float inv = 127.f / a;
            quantise8<4>(lo[i], a, inv);
            quantise8<4>(hi[i], a, inv);
            cl = make_char4((int)lo[i][0], (int)lo[i][1], (int)lo[i][2], (int)lo[i][3]);
            ch = make_char4((int)hi[i][0], (int)hi[i][1], (int)hi[i][2], (int)hi[i][3]);
        }
        env[g] = cl;
        env[kQuads + g] = ch;
    }
    if (lane == 0) p.env_scale[unit_out] = odd ? INFINITY : __fdiv_rn(a, 127.f);
}

template <typename T>
static cudaError_t launch_append_t(const AppendParams &p, int D, cudaStream_t stream) {
    const long long blocks = ((long long)p.T * p.Hkv + 7) / 8;
    if (blocks == 0) return cudaSuccess;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (D == 64)
        paged_attn_append_kernel<T, 64><<<(unsigned)blocks, 256, 0, stream>>>(p);
    else if (D == 128)
        paged_attn_append_kernel<T, 128><<<(unsigned)blocks, 256, 0, stream>>>(p);
    else
        paged_attn_append_kernel<T, 256><<<(unsigned)blocks, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_append(const AppendParams &p, int dtype, int D, cudaStream_t stream) {
    if (dtype == PA_F32) return launch_append_t<float>(p, D, stream);
    if (dtype == PA_BF16) return launch_append_t<__nv_bfloat16>(p, D, stream);
    return launch_append_t<__half>(p, D, stream);
}

}  // namespace pa
