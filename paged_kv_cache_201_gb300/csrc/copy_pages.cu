// Page contents from page to page in several pools.
//
// A CTA moves chunks of kChunk bytes; the chunks of a pair's page in every pool stand in one row, so that a few pairs
// already occupy every multiprocessor.  The number of pairs may be on the device: the grid is sized for all and walks.
// 8192 moves of 64 KB (1.07 GB read and written) take 165 us, 6.5 TB/s or 97 % of the copy rate; four pages of 18 KB in two
// pools 3.4 us, a launch and two trips to memory.
#include "kernels.h"
#include "kv4.cuh"

namespace pa {

namespace {

constexpr int kThreads = 256;
constexpr int kU = 4;                                // 16-byte loads of a thread on their way together
constexpr long long kChunk = 16ll * kThreads * kU;   // bytes of a CTA's turn

template <typename V>
__device__ __forceinline__ void copy_chunk(const uint8_t *src, uint8_t *dst, long long bytes) {
    const V *s = reinterpret_cast<const V *>(src);
    V *d = reinterpret_cast<V *>(dst);
    const int n = (int)(bytes / (long long)sizeof(V));
    for (int i = threadIdx.x; i < n; i += kThreads * kU) {
        V v[kU];
#pragma unroll
        for (int k = 0; k < kU; ++k)
            if (i + k * kThreads < n) v[k] = __ldcs(s + i + k * kThreads);
#pragma unroll
        for (int k = 0; k < kU; ++k)
            if (i + k * kThreads < n) d[i + k * kThreads] = v[k];
    }
}

}  // namespace

__global__ void __launch_bounds__(kThreads) paged_attn_copy_pages_kernel(const __grid_constant__ CopyPagesParams p,
                                                                         int chunks) {
    wait_for_stream();
    const int pairs = p.n_pairs ? min(max(__ldg(p.n_pairs), 0), p.max_pairs) : p.max_pairs;
    const long long units = (long long)pairs * chunks;
    for (long long unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int k = (int)(unit / chunks);
        int c = (int)(unit - (long long)k * chunks);
        const int from = __ldg(p.pairs + 2ll * k), to = __ldg(p.pairs + 2ll * k + 1);
        if (from == -1 || to == -1) continue;
        if (from < 0 || from >= p.num_pages || to < 0 || to >= p.num_pages) {
            if (threadIdx.x == 0) atomicOr(p.err, (unsigned int)PA_ERRBIT_PAGE_RANGE);
            continue;
        }
        int i = 0;
        for (;;) {
            const int here = (int)((p.bytes[i] + kChunk - 1) / kChunk);
            if (c < here) break;
            c -= here;
            ++i;
        }
        const long long size = p.bytes[i], at = c * kChunk, left = min(kChunk, size - at);
        const uint8_t *src = p.pool[i] + from * size + at;
        uint8_t *dst = p.pool[i] + to * size + at;
        if (((size | (long long)reinterpret_cast<uintptr_t>(p.pool[i])) & 15) == 0)
            copy_chunk<uint4>(src, dst, left);
        else
            copy_chunk<uint32_t>(src, dst, left);
    }
}

cudaError_t launch_copy_pages(const CopyPagesParams &p, int sms, cudaStream_t stream) {
    long long chunks = 0;
    for (int i = 0; i < p.n_pools; ++i) chunks += (p.bytes[i] + kChunk - 1) / kChunk;
    if (chunks == 0 || p.max_pairs == 0) return cudaSuccess;
    if (chunks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const long long units = chunks * p.max_pairs, most = 8ll * sms;
    return launch_behind(paged_attn_copy_pages_kernel, dim3((unsigned)(units < most ? units : most)), kThreads, 0, 1, stream, p,
                         (int)chunks);
}

}  // namespace pa
