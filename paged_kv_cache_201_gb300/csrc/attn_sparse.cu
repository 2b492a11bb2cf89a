// Attention over listed pages on CUDA cores: the kernel for f32.  One CTA, or a cluster with a part of the
// list each, per (query token, kv head, chunk of HG query heads); see sparse_simt.cuh.  Five sequences of
// three tokens, lists of nine 16-token pages, head_dim 64: 6.7 us, the latency of a list's pages.  256 sequences, 8 kv heads of 128, G = 4,
// lists of 64 16-token pages (2.15 GB): 494 us, 64 % of the copy rate, bound by the products' instructions
// and by 255 registers (two CTAs an SM; three, 168 registers, take 602).  Two pages loaded together, entries
// looked up 32 at a time: 560 us with one after the other (head_dim 256: 343 -> 262).
#include "sparse_simt.cuh"

namespace pa {

constexpr int kSparseWarps = 4;

template <typename T, int D, int HG, bool CLUSTER>
__global__ void __launch_bounds__(kSparseWarps * 32) paged_attn_sparse_simt_kernel(const SparseParams sp, int S) {
    __shared__ float scratch[simt_scratch<D, HG, kSparseWarps>()];
    const FwdParams &p = sp.f;
    const int chunks = (p.G + HG - 1) / HG;
    int unit = blockIdx.x;
    const int s = CLUSTER ? unit % S : 0;
    if (CLUSTER) unit /= S;
    const int hc = unit % chunks;
    unit /= chunks;
    const int kvh = unit % p.Hkv;
    const long long t = unit / p.Hkv;
    RangeCheck ranges(sp);
    const TokenRow tr = token_row(p, t, sp.n_tok, threadIdx.x == 0);
    ranges.report(p);
    if (tr.b < 0) return;  // the whole cluster: it has one token
    auto sync = [] {
        if (CLUSTER)
            cluster_barrier();
        else
            __syncthreads();
    };
    simt_token<T, D, HG, kSparseWarps, 2, CLUSTER>(sp, tr, t, kvh, hc, scratch, threadIdx.x, s, S, sync);
    if (CLUSTER) sync();  // peers may still be reading this CTA's states
}

template <typename T, int D, int HG>
static cudaError_t launch_sparse_simt_t(const SparseParams &sp, int sms, cudaStream_t stream) {
    const FwdParams &p = sp.f;
    const long long units = sp.n_tok * p.Hkv * ((p.G + HG - 1) / HG);
    if (units == 0) return cudaSuccess;
    // Few rows: a list split over a cluster while its CTAs do not fill two per multiprocessor and each keeps
    // eight pages (8 rows of 128 pages, head_dim 128: 12.7 us, 55 on a CTA each).
    int S = 1;
    while (S < 8 && units * S * 2 <= 2ll * sms && sp.K >= 16 * S) S *= 2;
    if (units * S > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(units * S));
    cfg.blockDim = dim3(kSparseWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2]{};
    cfg.numAttrs = second_launch_attrs(attr, S, false);
    cfg.attrs = attr;
    return S > 1 ? cudaLaunchKernelEx(&cfg, paged_attn_sparse_simt_kernel<T, D, HG, true>, sp, S)
                 : cudaLaunchKernelEx(&cfg, paged_attn_sparse_simt_kernel<T, D, HG, false>, sp, S);
}

cudaError_t launch_sparse_simt(const SparseParams &sp, int sms, cudaStream_t stream) {
    if (sp.f.D == 64) return launch_sparse_simt_t<float, 64, 4>(sp, sms, stream);
    if (sp.f.D == 128) return launch_sparse_simt_t<float, 128, 4>(sp, sms, stream);
    return launch_sparse_simt_t<float, 256, 2>(sp, sms, stream);
}

}  // namespace pa
