// The pages a query token attends to, by an 8-bit score of each page's key envelope.
//
// With qi the group's queries in 8 bits and lo / hi the page's corners, s = max_h sum_d max(qi lo, qi hi)
// = max_h (min(qi, 0) . lo + max(qi, 0) . hi): an integer dot product of length 2 D, below 2^24, then one
// float32 product with the page's scale.  The score, and so the selection, is the same bits in any order
// of evaluation.  One CTA per (token, kv head): the scores of its candidate pages as ordered 32-bit keys
// in shared memory, then the threshold key by 32 bisections over the bits.
#include <float.h>

#include "sparse_common.cuh"

namespace pa {

namespace {

constexpr int kSelThreads = 128;
constexpr int kSelHeads = 64;  // heads of a group scored at a time

// Order-preserving map of a float to an unsigned key (no NaN comes here).
__device__ __forceinline__ unsigned ordered(float x) {
    const unsigned u = __float_as_uint(x + 0.f);  // -0 becomes +0
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

}  // namespace

template <typename T>
__global__ void __launch_bounds__(kSelThreads) paged_attn_select_kernel(const SparseParams sp) {
    const FwdParams &p = sp.f;
    extern __shared__ unsigned s_key[];  // [candidates between the forced pages]
    __shared__ __align__(16) int8_t s_q[kSelHeads * 256];
    __shared__ float s_red[kSelThreads / 32];
    __shared__ int s_cnt[kSelThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = blockIdx.x % p.Hkv;
    const long long t = blockIdx.x / p.Hkv;
    const TokenRow tr = token_row(p, t, sp.n_tok, tid == 0);
    if (tr.b < 0) return;
    const int np = (tr.reach + p.ps - 1) / p.ps;
    int32_t *out = sp.sel_out + (t * p.Hkv + h) * sp.K;
    if (np <= sp.K) {
        for (int j = tid; j < sp.K; j += kSelThreads) out[j] = j < np ? j : -1;
        return;
    }
    const int m0 = sp.sink, m1 = np - sp.local, n = m1 - m0;  // scored pages; n > want
    const int want = sp.K - sp.sink - sp.local;
    for (int j = tid; j < sp.sink; j += kSelThreads) out[j] = j;
    for (int j = tid; j < sp.local; j += kSelThreads) out[sp.K - sp.local + j] = m1 + j;
    if (want == 0) return;

    // the group's queries in 8 bits
    const int ne = p.G * p.D;
    const T *q = static_cast<const T *>(p.q) + q_row_offset(p, t * p.Hq + (long long)h * p.G);
    float a = 0.f;
    bool odd = false;
    for (int i = tid; i < ne; i += kSelThreads) {
        const float x = fabsf(to_float(q[i]));
        odd |= !(x <= FLT_MAX);
        a = fmaxf(a, x);
    }
    for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    if (lane == 0) s_red[warp] = a;
    odd = __syncthreads_or(odd);
    a = s_red[0];
    for (int w = 1; w < kSelThreads / 32; ++w) a = fmaxf(a, s_red[w]);

    const int32_t *bt = p.block_table + (long long)tr.b * p.W;
    for (int g0 = 0; g0 < p.G; g0 += kSelHeads) {  // heads whose queries fit the buffer
        const int gn = min(kSelHeads, p.G - g0);
        __syncthreads();
        for (int i = tid; i < gn * p.D; i += kSelThreads) {
            const float x = to_float(q[g0 * p.D + i]);
            s_q[i] = (odd || a == 0.f) ? 0 : (signed char)(int)rintf(__fmul_rn(__fdiv_rn(x, a), 127.f));
        }
        __syncthreads();
        for (int j = tid; j < n; j += kSelThreads) {
            const int id = bt[m0 + j];
            unsigned key;
            if (id < 0 || id >= p.num_pages) {
                if (g0 == 0) atomicOr(p.err, (unsigned int)PA_ERRBIT_PAGE_RANGE);
                key = ordered(0.f);
            } else {
                const long long unit = (long long)id * p.Hkv + h;
                const int *lo = reinterpret_cast<const int *>(sp.env + unit * 2 * p.D);
                const int *hi = lo + p.D / 4;
                int best = -0x7fffffff;
                for (int g = 0; g < gn; ++g) {
                    const int *qg = reinterpret_cast<const int *>(s_q + g * p.D);
                    int s = 0;
                    for (int d = 0; d < p.D / 4; ++d) {
                        const int x = qg[d];
                        s = __dp4a((int)__vmins4(x, 0), lo[d], s);
                        s = __dp4a((int)__vmaxs4(x, 0), hi[d], s);
                    }
                    best = max(best, s);
                }
                const float scale = sp.env_scale[unit];
                key = ordered(scale == INFINITY ? INFINITY : __fmul_rn((float)best, scale));
            }
            s_key[j] = g0 == 0 ? key : max(s_key[j], key);  // the scale is not negative: max of keys = key of max
        }
    }
    __syncthreads();
    // the want-th largest key: the largest value that at least `want` keys reach
    unsigned thr = 0;
    for (int bit = 31; bit >= 0; --bit) {
        const unsigned cand = thr | (1u << bit);
        int c = 0;
        for (int j = tid; j < n; j += kSelThreads) c += s_key[j] >= cand;
        c = __reduce_add_sync(0xffffffffu, c);
        if (lane == 0) s_cnt[warp] = c;
        __syncthreads();
        c = 0;
        for (int w = 0; w < kSelThreads / 32; ++w) c += s_cnt[w];
        __syncthreads();
        if (c >= want) thr = cand;
    }
    if (warp != 0) return;
    int above = 0;
    for (int j = lane; j < n; j += 32) above += s_key[j] > thr;
    above = __reduce_add_sync(0xffffffffu, above);
    int ties = want - above, done = 0;  // the first `ties` pages at the threshold are taken
    for (int j0 = 0; j0 < n; j0 += 32) {
        const int j = j0 + lane;
        const unsigned key = j < n ? s_key[j] : 0u;
        const unsigned gt = __ballot_sync(0xffffffffu, j < n && key > thr);
        const unsigned eq = __ballot_sync(0xffffffffu, j < n && key == thr);
        const unsigned below = (1u << lane) - 1;
        const bool take = (gt >> lane & 1) || ((eq >> lane & 1) && __popc(eq & below) < ties);
        const unsigned taken = __ballot_sync(0xffffffffu, take);
        if (take) out[sp.sink + done + __popc(taken & below)] = m0 + j;
        done += __popc(taken);
        ties -= min(ties, __popc(eq));
    }
}

cudaError_t launch_select_pages(const SparseParams &p, int dtype, cudaStream_t stream) {
    const long long units = p.n_tok * p.f.Hkv;
    if (units == 0) return cudaSuccess;
    if (units > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    auto kern = dtype == PA_F32 ? paged_attn_select_kernel<float>
                                : dtype == PA_BF16 ? paged_attn_select_kernel<__nv_bfloat16> : paged_attn_select_kernel<__half>;
    const size_t smem = (size_t)p.f.W * 4;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)units, kSelThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace pa
