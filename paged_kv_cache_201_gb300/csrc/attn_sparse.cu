// Attention over listed pages on CUDA cores: the kernel for f32.  One CTA per (query token, kv head, chunk
// of HG query heads); see sparse_simt.cuh.  Five sequences of three tokens, lists of nine 16-token pages,
// head_dim 64: 6.7 us, the latency of one list's pages after another.  256 sequences, 8 kv heads of 128, G = 4,
// lists of 64 16-token pages (2.15 GB): 494 us, 64 % of the copy rate, bound by the products' instructions
// and by 255 registers (two CTAs an SM; three, 168 registers, take 602).  Two pages loaded together, entries
// looked up 32 at a time: 560 us with one after the other (head_dim 256: 343 -> 262).
#include "sparse_simt.cuh"

namespace pa {

constexpr int kSparseWarps = 4;

template <typename T, int D, int HG>
__global__ void __launch_bounds__(kSparseWarps * 32) paged_attn_sparse_simt_kernel(const SparseParams sp) {
    __shared__ float scratch[simt_scratch<D, HG, kSparseWarps>()];
    const FwdParams &p = sp.f;
    const int chunks = (p.G + HG - 1) / HG;
    int unit = blockIdx.x;
    const int hc = unit % chunks;
    unit /= chunks;
    const int kvh = unit % p.Hkv;
    const long long t = unit / p.Hkv;
    RangeCheck ranges(sp);
    const TokenRow tr = token_row(p, t, sp.n_tok, threadIdx.x == 0);
    ranges.report(p);
    if (tr.b < 0) return;
    simt_token<T, D, HG, kSparseWarps, 2>(sp, tr, t, kvh, hc, scratch, threadIdx.x, [] { __syncthreads(); });
}

template <typename T>
static cudaError_t launch_sparse_simt_t(const SparseParams &sp, cudaStream_t stream) {
    const FwdParams &p = sp.f;
    const int hg = p.D == 256 ? 2 : 4;
    const long long units = sp.n_tok * p.Hkv * ((p.G + hg - 1) / hg);
    if (units == 0) return cudaSuccess;
    if (units > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (p.D == 64)
        paged_attn_sparse_simt_kernel<T, 64, 4><<<(unsigned)units, kSparseWarps * 32, 0, stream>>>(sp);
    else if (p.D == 128)
        paged_attn_sparse_simt_kernel<T, 128, 4><<<(unsigned)units, kSparseWarps * 32, 0, stream>>>(sp);
    else
        paged_attn_sparse_simt_kernel<T, 256, 2><<<(unsigned)units, kSparseWarps * 32, 0, stream>>>(sp);
    return cudaGetLastError();
}

cudaError_t launch_sparse_simt(const SparseParams &sp, cudaStream_t stream) {
    return launch_sparse_simt_t<float>(sp, stream);
}

}  // namespace pa
