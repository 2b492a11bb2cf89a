// Attention of one query token and a chunk of its heads over its listed pages, on CUDA cores.
//
// A warp's four 8-lane groups each take every (4 NW)-th key of a listed page and run their own online
// softmax (log2 domain, one pass over K and V); the 4 NW states are merged once at the end.  The mask is
// a count: a listed page j gives its first min(page_size, reach - j page_size) keys, and a key that is not
// seen is not multiplied with anything.
#pragma once

#include "sparse_common.cuh"

namespace pa {

template <typename T, int N>
__device__ __forceinline__ void load_row(const T *src, float (&v)[N]) {
    // lane l of an 8-lane group holds elements i * 32 + l * 4 .. + 3
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            const float4 x = __ldg(reinterpret_cast<const float4 *>(src + i * 32));
            v[4 * i] = x.x, v[4 * i + 1] = x.y, v[4 * i + 2] = x.z, v[4 * i + 3] = x.w;
        } else {
            const uint2 x = __ldg(reinterpret_cast<const uint2 *>(src + i * 32));
            const float2 a = MmaOp<T>::unpack(x.x), b = MmaOp<T>::unpack(x.y);
            v[4 * i] = a.x, v[4 * i + 1] = a.y, v[4 * i + 2] = b.x, v[4 * i + 3] = b.y;
        }
    }
}

// Floats of shared memory that simt_token takes.
template <int D, int HG, int NW>
constexpr int simt_scratch() { return NW * HG * (D + 2); }

// Token t (reach and sequence in tr), kv head kvh, query heads hc HG .. + HG - 1 of the group; called by NW
// warps of a CTA, tid 0 .. 32 NW - 1 among them, with `sync` a barrier over them.  PAGES: listed pages whose
// keys are loaded together.  CLUSTER: CTA s of a cluster of S takes the s-th part of the list, and they
// share out the merge; `sync` is a barrier over the cluster, passed once more by the caller at the end.
template <typename T, int D, int HG, int NW, int PAGES, bool CLUSTER, typename Sync>
__device__ __forceinline__ void simt_token(const SparseParams &sp, const TokenRow tr, long long t, int kvh, int hc,
                                           float *scratch, int tid, int s, int S, Sync sync) {
    constexpr int N = D / 8;
    const FwdParams &p = sp.f;
    const int lane = tid & 31, warp = tid >> 5;
    const int l8 = lane & 7, stream = warp * 4 + (lane >> 3);
    const int g0 = hc * HG, gn = min(HG, p.G - g0);
    const long long row0 = t * p.Hq + (long long)kvh * p.G + g0;

    float q[HG][N], acc[HG][N], m[HG], l[HG];
#pragma unroll
    for (int g = 0; g < HG; ++g) {
        load_row(static_cast<const T *>(p.q) + q_row_offset(p, row0 + min(g, gn - 1)) + l8 * 4, q[g]);
        m[g] = kNegInf;
        l[g] = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) acc[g][i] = 0.f;
    }
    const int32_t *list = sp.sel + (t * p.Hkv + kvh) * sp.K;
    const int32_t *bt = p.block_table + (long long)tr.b * p.W;
    const int np = (tr.reach + p.ps - 1) / p.ps;
    const long long row_elems = (long long)p.Hkv * D;
    const int part = CLUSTER ? (sp.K + S - 1) / S : sp.K;
    const int e_first = CLUSTER ? min(s * part, sp.K) : 0, e_last = CLUSTER ? min(e_first + part, sp.K) : sp.K;
    for (int e0 = e_first; e0 < e_last; e0 += 32) {
        // 32 entries' pages in two trips, a lane each
        int my_j = e0 + lane < e_last ? __ldg(list + e0 + lane) : -1, my_id = 0;
        if (my_j >= np) my_j = -1;
        if (my_j >= 0) my_id = __ldg(bt + my_j);
        const bool out_of_pool = my_j >= 0 && (my_id < 0 || my_id >= p.num_pages);
        if (out_of_pool && warp == 0) atomicOr(p.err, (unsigned int)PA_ERRBIT_PAGE_RANGE);
        unsigned live = __ballot_sync(0xffffffffu, my_j >= 0);
        while (live) {
            int nv[PAGES], id[PAGES];  // keys of a page that the token sees
            bool on[PAGES];
#pragma unroll
            for (int u = 0; u < PAGES; ++u) {
                const int src = live ? __ffs((int)live) - 1 : 0;
                const int j = __shfl_sync(0xffffffffu, my_j, src);
                id[u] = __shfl_sync(0xffffffffu, my_id, src);
                on[u] = id[u] >= 0 && id[u] < p.num_pages;
                nv[u] = live ? min(p.ps, tr.reach - j * p.ps) : 0;
                live &= live - 1;
            }
            int most = nv[0];
#pragma unroll
            for (int u = 1; u < PAGES; ++u) most = max(most, nv[u]);
            for (int k0 = 0; k0 < most; k0 += NW * 4) {
                const int key = k0 + stream;
                float kk[PAGES][N], vv[PAGES][N];
#pragma unroll
                for (int u = 0; u < PAGES; ++u) {
                    const long long off = ((long long)id[u] * p.ps + key) * row_elems + (long long)kvh * D + l8 * 4;
                    if (key < nv[u] && on[u]) {
                        load_row(static_cast<const T *>(p.k_cache) + off, kk[u]);
                        load_row(static_cast<const T *>(p.v_cache) + off, vv[u]);
                    } else {
#pragma unroll
                        for (int i = 0; i < N; ++i) kk[u][i] = vv[u][i] = 0.f;
                    }
                }
#pragma unroll
                for (int u = 0; u < PAGES; ++u)
#pragma unroll
                    for (int g = 0; g < HG; ++g) {
                        float s = 0.f;
#pragma unroll
                        for (int i = 0; i < N; ++i) s = fmaf(q[g][i], kk[u][i], s);
                        s += __shfl_xor_sync(0xffffffffu, s, 1);
                        s += __shfl_xor_sync(0xffffffffu, s, 2);
                        s += __shfl_xor_sync(0xffffffffu, s, 4);
                        s = key < nv[u] ? s * p.scale_log2 : kNegInf;
                        const float mn = fmaxf(m[g], s);
                        const float mu = mn == kNegInf ? 0.f : mn;
                        const float al = exp2f(m[g] - mu), w = exp2f(s - mu);
                        m[g] = mn;
                        l[g] = l[g] * al + w;
#pragma unroll
                        for (int i = 0; i < N; ++i) acc[g][i] = fmaf(w, vv[u][i], acc[g][i] * al);
                    }
            }
        }
    }
    // merge the 4 NW states (of each CTA of a cluster): across the warp's groups by shuffles, across the warps in
    // shared memory
    float *s_acc = scratch, *s_m = s_acc + NW * HG * D, *s_l = s_m + NW * HG;  // [NW][HG][D], [NW][HG] twice
#pragma unroll
    for (int g = 0; g < HG; ++g) {
#pragma unroll
        for (int o = 8; o <= 16; o <<= 1) {
            const float mo = __shfl_xor_sync(0xffffffffu, m[g], o), lo = __shfl_xor_sync(0xffffffffu, l[g], o);
            const float mn = fmaxf(m[g], mo), mu = mn == kNegInf ? 0.f : mn;
            const float a = exp2f(m[g] - mu), b = exp2f(mo - mu);
            m[g] = mn;
            l[g] = l[g] * a + lo * b;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float x = __shfl_xor_sync(0xffffffffu, acc[g][i], o);
                acc[g][i] = acc[g][i] * a + x * b;
            }
        }
        if (lane < 8) {
#pragma unroll
            for (int i = 0; i < N; ++i) s_acc[(warp * HG + g) * D + (i >> 2) * 32 + l8 * 4 + (i & 3)] = acc[g][i];
            if (lane == 0) s_m[warp * HG + g] = m[g], s_l[warp * HG + g] = l[g];
        }
    }
    sync();
    auto state = [&](const float *x, int cta) { return CLUSTER ? peer_load(peer_addr(smem_u32(x), cta)) : *x; };
    const int ctas = CLUSTER ? S : 1;
    for (int idx = (CLUSTER ? s * NW * 32 : 0) + tid; idx < gn * D; idx += ctas * NW * 32) {
        const int g = idx / D, d = idx % D;
        float M = kNegInf, L = 0.f, o = 0.f;
#pragma unroll 4
        for (int cta = 0; cta < ctas; ++cta)
#pragma unroll
            for (int w = 0; w < NW; ++w) M = fmaxf(M, state(s_m + w * HG + g, cta));
        const float mu = M == kNegInf ? 0.f : M;
#pragma unroll 4
        for (int cta = 0; cta < ctas; ++cta)
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float x = exp2f(state(s_m + w * HG + g, cta) - mu);
                L = fmaf(x, state(s_l + w * HG + g, cta), L);
                o = fmaf(x, state(s_acc + (w * HG + g) * D + d, cta), o);
            }
        // a row without a key: 0 and -inf (a NaN sum stays a NaN)
        static_cast<T *>(p.out)[(row0 + g) * D + d] = from_float<T>(L == 0.f ? 0.f : o / L);
        if (d == 0 && p.lse) p.lse[row0 + g] = L == 0.f ? kNegInf : M * kLn2 + logf(L);
    }
}

}  // namespace pa
