// Host-side launchers of the paged-attention kernels (internal to the library).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "common.cuh"

namespace pa {

// Tensor-core kernel modes.
enum { MODE_DECODE = 0, MODE_PREFILL = 1, MODE_SPLITS = 2 };

constexpr int kMmaTileKeys = 64;      // keys per pipeline stage
constexpr int kMmaConsumerWarps = 4;  // warps doing QK / softmax / PV
constexpr int kMmaThreads = (kMmaConsumerWarps + 1) * 32;
constexpr int kDecodeRows = 16;       // query rows of one decode CTA (one m16 tile)
constexpr int kPrefillRows = 64;      // query rows of one prefill CTA (4 warps x 16)
// MODE_SPLITS: decode whose splits are short.  A CTA takes kMmaConsumerWarps consecutive splits
// of one (sequence, kv head) and each consumer warp owns one of them; every split is at most
// kGroupSplitPages pages, so a group's page ids fit one warp-wide load.
constexpr int kGroupSplitPages = 32 / kMmaConsumerWarps;
// Stages of one group at most: four splits of kGroupSplitPages pages of up to 64 tokens, 64-key
// stages.  Each has its own full barriers (waited once, at phase 0): the warps consume the ring's
// slots out of step with one another, so a per-slot parity could be two phases behind.
constexpr int kGroupMaxStages = kMmaConsumerWarps * kGroupSplitPages;

// Dynamic shared memory of the tensor-core kernel for a pipeline depth.
size_t mma_smem_bytes(int head_dim, int stages);

cudaError_t launch_mma(const FwdParams &p, int mode, int dtype, const CUtensorMap &tmk, const CUtensorMap &tmv,
                       cudaStream_t stream);
// Variable-length batch (p.q_start set, p.B sequences, total_q packed query tokens).
cudaError_t launch_mma_varlen(const FwdParams &p, long long total_q, int dtype, const CUtensorMap &tmk,
                              const CUtensorMap &tmv, cudaStream_t stream);
// 8-bit pools (kv_dtype PA_FP8_E4M3 or PA_INT8) with per-(page, kv head) scales in p.k_scale /
// p.v_scale; bf16/f16 queries.
cudaError_t launch_mma_kvq(const FwdParams &p, int mode, int dtype, int kv_dtype, const CUtensorMap &tmk,
                           const CUtensorMap &tmv, cudaStream_t stream);
// tcgen05 prefill: bf16/f16, head_dim 128, (Hq/Hkv) dividing 128.
size_t tc05_smem_bytes();
cudaError_t launch_tc05(const FwdParams &p, int dtype, const CUtensorMap &tmq, const CUtensorMap &tmk,
                        const CUtensorMap &tmv, const CUtensorMap &tmo, cudaStream_t stream);
// Variable-length batch (p.q_start, total_q packed tokens, at most kTc05VarlenMaxBatch sequences):
// the sequences of at least 64 query rows, on at most max_ctas SMs (0: every SM).
constexpr int kTc05VarlenMaxBatch = 1024;
cudaError_t launch_tc05_varlen(const FwdParams &p, long long total_q, int dtype, const CUtensorMap &tmq,
                               const CUtensorMap &tmk, const CUtensorMap &tmv, const CUtensorMap &tmo,
                               int max_ctas, cudaStream_t stream);
cudaError_t launch_simt(const FwdParams &p, int dtype, cudaStream_t stream);
// One query row per (sequence, kv head), bf16/f16, head_dim 64/128: CUDA cores over the TMA ring.
cudaError_t launch_simt_decode(const FwdParams &p, int dtype, const CUtensorMap &tmk, const CUtensorMap &tmv,
                               cudaStream_t stream);
// head_dim 256, bf16/f16: transposed products, 8-row units.
cudaError_t launch_mma_t(const FwdParams &p, int dtype, const CUtensorMap &tmk, const CUtensorMap &tmv,
                         cudaStream_t stream);
cudaError_t launch_combine(const float *part_out, const float *part_lse, int S, long long rows, int D,
                           int out_dtype, void *out, float *lse, cudaStream_t stream);
cudaError_t launch_plan(const int32_t *seq_lens, int B, int ps, int S, int32_t *plan, cudaStream_t stream);
cudaError_t launch_wait_probe(unsigned int *err, unsigned long long limit_ns, cudaStream_t stream);
cudaError_t launch_gather(const void *cache, const int32_t *block_table, const int32_t *seq_lens, int B, int W,
                          int ps, int Hkv, int D, int esize, long long num_pages, int out_tokens, void *out,
                          unsigned int *err, cudaStream_t stream);

// ---------------------------------------------------------------- serving step over selected pages
// Raise a kernel's dynamic shared memory limit to `bytes` once per device: the attribute is a driver
// call of its own, and these launches take a few microseconds in all.  `done` belongs to the kernel.
struct SmemLimit {
    std::atomic<uint64_t> done[2];
    cudaError_t raise(const void *kern, size_t bytes) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const bool known = dev >= 0 && dev < 128;
        const uint64_t bit = 1ull << (dev & 63);
        if (known && (done[dev >> 6].load(std::memory_order_acquire) & bit)) return cudaSuccess;
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (e == cudaSuccess && known) done[dev >> 6].fetch_or(bit, std::memory_order_release);
        return e;
    }
};

struct StepTablesParams {
    const int32_t *cached_lens, *new_lens, *free_pages, *free_count;
    int32_t *block_table, *seq_lens, *q_offset, *q_start, *slots, *free_left;
    unsigned int *err;
    long long num_pages;
    int free_cap, B, T, ps_shift, W;
};
cudaError_t launch_step_tables(const StepTablesParams &p, cudaStream_t stream);

struct AppendParams {
    const void *k_new, *v_new;
    const int32_t *slots;
    void *k_cache, *v_cache;
    int8_t *env;       // [num_pages, Hkv, 2, D] or null
    float *env_scale;  // [num_pages, Hkv]
    unsigned int *err;
    long long k_stride, v_stride;  // elements between tokens
    long long num_slots;           // num_pages * ps
    int T, Hkv, ps_shift;
};
cudaError_t launch_append(const AppendParams &p, int dtype, int D, cudaStream_t stream);

// The pages a query token attends to.  f.Sq is the uniform batch's query count; with f.q_start the
// tokens are packed and n_tok is the row count of q.
struct SparseParams {
    FwdParams f;
    const int8_t *env;  // selection only
    const float *env_scale;
    int32_t *sel_out;
    const int32_t *sel;  // attention only: [n_tok, Hkv, K]
    long long n_tok;
    int K, sink, local;
    int group_min;  // packed batches: sequences of so many tokens are the tcgen05 kernel's (0: none)
    int by_seq;     // the other kernel's units are group_min - 1 tokens of every sequence, not the rows of q
};
// Runs of tokens of a sequence, scored with tcgen05: head_dim 64 / 128, G <= 32.  select_tile_tokens: tokens of
// one CTA (0: not for this shape or table width).
constexpr size_t kSelectTc05MaxSmem = 224 * 1024;
size_t select_tc05_smem(int D, int N, int TT, int W);
int select_tile_tokens(int D, int G, int W);
cudaError_t launch_select_all(const SparseParams &p, int sms, cudaStream_t stream);  // rows of at most top_k pages
cudaError_t launch_select_tc05(const SparseParams &p, int dtype, int sms, cudaStream_t stream);
cudaError_t launch_select_pages_64(const SparseParams &p, int dtype, int sms, cudaStream_t stream);
cudaError_t launch_select_pages_128(const SparseParams &p, int dtype, int sms, cudaStream_t stream);
cudaError_t launch_select_pages_256(const SparseParams &p, int dtype, int sms, cudaStream_t stream);
inline cudaError_t launch_select_pages(const SparseParams &p, int dtype, int sms, cudaStream_t stream) {
    return (p.f.D == 64 ? launch_select_pages_64 : p.f.D == 128 ? launch_select_pages_128 : launch_select_pages_256)(
        p, dtype, sms, stream);
}
// bf16/f16: tensor cores, a list's pages split over a cluster when there are few rows (sms: SM count)
cudaError_t launch_sparse_mma(const SparseParams &p, int dtype, int sms, const CUtensorMap &tmk,
                              const CUtensorMap &tmv, cudaStream_t stream);
// bf16/f16, head_dim 64/128, G <= 128, scale > 0: runs of a sequence's tokens that share page loads, on
// tcgen05; at most kSparseTc05MaxPages pages a sequence.  sparse_tile_tokens: tokens of one CTA (0: not for
// this G).
constexpr int kSparseTc05MaxPages = 4608;
int sparse_tile_tokens(int G);
cudaError_t launch_sparse_tc05(const SparseParams &p, int dtype, const CUtensorMap &tmq, const CUtensorMap &tmk,
                               const CUtensorMap &tmv, cudaStream_t stream);
// f32: CUDA cores, a list split over a cluster when there are few rows
cudaError_t launch_sparse_simt(const SparseParams &p, int sms, cudaStream_t stream);

}  // namespace pa
