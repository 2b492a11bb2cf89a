// The selection where a block-table row is no longer than top_k: every page that a token reaches is selected,
// so nothing is scored and the lists are only written.
//
// A warp looks up TPW consecutive tokens, a lane each (their searches in q_start overlap), then writes their
// lists, the kv heads' one behind another.  12000 prompt tokens of 5 heads, top_k = 5 (1.2 MB) take 4.4 us, the
// latency of the look-up; the scoring kernels took 78.
#include "sparse_common.cuh"

namespace pa {

constexpr int kSelectAllWarps = 4;

__global__ void __launch_bounds__(kSelectAllWarps * 32) paged_attn_select_all_kernel(const SparseParams sp, int TPW) {
    const FwdParams &p = sp.f;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long t0 = ((long long)blockIdx.x * kSelectAllWarps + warp) * TPW;
    RangeCheck ranges(sp);
    int np = -1;  // pages of this lane's token; -1: a row of no sequence
    if (lane < TPW && t0 + lane < sp.n_tok) {
        const TokenRow tr = token_row(p, t0 + lane, sp.n_tok, true);
        if (tr.b >= 0) np = (tr.reach + p.ps - 1) / p.ps;
    }
    ranges.report(p);
    const long long per_token = (long long)p.Hkv * sp.K;
    const int first = lane % sp.K, step = 32 % sp.K;
    for (int i = 0; i < TPW; ++i) {
        const int n = __shfl_sync(0xffffffffu, np, i);
        if (n < 0) continue;
        int32_t *out = sp.sel_out + (t0 + i) * per_token;
        int j = first;
        for (long long e = lane; e < per_token; e += 32) {
            out[e] = j < n ? j : -1;
            j += step;
            if (j >= sp.K) j -= sp.K;
        }
    }
}

cudaError_t launch_select_all(const SparseParams &sp, int sms, cudaStream_t stream) {
    int TPW = 32;
    while (TPW > 1 && sp.n_tok < 8ll * sms * TPW) TPW /= 2;  // eight warps a multiprocessor
    const long long blocks = (sp.n_tok + (long long)TPW * kSelectAllWarps - 1) / ((long long)TPW * kSelectAllWarps);
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    paged_attn_select_all_kernel<<<(unsigned)blocks, kSelectAllWarps * 32, 0, stream>>>(sp, TPW);
    return cudaGetLastError();
}

}  // namespace pa
