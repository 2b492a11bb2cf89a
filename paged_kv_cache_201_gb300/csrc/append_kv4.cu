// New tokens' K and V rows into a 4-bit pool, and rows of slots read back as the values they stand for.
//
// A thread takes eight elements, 16 (or in float32 32) bytes; two neighbours share a scale, so the only exchange is
// one shuffle of their largest magnitudes.  Both calls move bytes: the codes are exact whole-number decisions, made
// with a product and a comparison an element (see quantise), which hide behind the loads.
#include <float.h>

#include "kernels.h"
#include "kv4.cuh"

namespace pa {

namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ void load8(const T *src, float (&x)[8]) {
    if constexpr (sizeof(T) == 4) {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(src)), b = __ldg(reinterpret_cast<const float4 *>(src) + 1);
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
        const uint4 u = __ldg(reinterpret_cast<const uint4 *>(src));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = MmaOp<T>::unpack(w[i]);
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        }
    }
}

// clamp(rint(x / s), -7, 7) + 8 of eight elements, one to four bits.  The quotient's rounding cannot move it across
// a border (see scale_byte: a border times s has at most eight significant bits).
__device__ __forceinline__ uint32_t quantise(const float (&x)[8], float s) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float c = fminf(fmaxf(rintf(__fdiv_rn(x[i], s)), -7.f), 7.f);
        w |= (uint32_t)((int)c + 8) << (4 * i);
    }
    return w;
}

}  // namespace

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) paged_attn_append_kv4_kernel(const Kv4RowsParams p) {
    constexpr int C = D / 8;  // threads of a row
    const long long unit = (long long)blockIdx.x * kThreads + threadIdx.x;
    const int c = (int)(unit % C);
    const long long row = unit / C;  // (token, side, kv head)
    const int h = (int)(row % p.Hkv);
    const long long ts = row / p.Hkv;
    const int side = (int)(ts & 1), t = (int)(ts >> 1);
    const bool live = ts < 2ll * p.T;
    const int slot = live ? __ldg(p.slots + t) : -1;
    const bool ok = slot >= 0 && slot < p.num_slots;
    if (slot != -1 && !ok && c == 0) atomicOr(p.err, (unsigned int)PA_ERRBIT_PAGE_RANGE);
    float x[8];
    float a = 0.f;
    bool odd = false;
    if (ok) {
        const T *src = static_cast<const T *>(side ? p.v : p.k) + t * (side ? p.v_stride : p.k_stride) + h * D + c * 8;
        load8<T>(src, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            odd |= !(fabsf(x[i]) <= FLT_MAX);
            x[i] = x[i] == x[i] ? x[i] : 0.f;
            a = fmaxf(a, fabsf(x[i]));
        }
    }
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
    if (odd) atomicOr(p.err, (unsigned int)PA_ERRBIT_NONFINITE);
    if (!ok) return;
    const uint32_t byte = kv4::scale_byte(a);
    const kv4::Layout at{1 << p.ps_shift, D};
    const int r = slot & (at.ps - 1);
    uint8_t *block = p.pool + ((long long)(slot >> p.ps_shift) * p.Hkv + h) * kv4::block_bytes(at.ps, D);
    *reinterpret_cast<uint32_t *>(block + at.codes(side, r) + 4 * c) =
        byte ? quantise(x, kv4::scale_value(byte)) : 0x88888888u;
    if ((c & 1) == 0) block[at.scales(side, r) + c / 2] = (uint8_t)byte;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) paged_attn_gather_kv4_kernel(const Kv4RowsParams p) {
    constexpr int C = D / 8;
    const long long unit = (long long)blockIdx.x * kThreads + threadIdx.x;
    const int c = (int)(unit % C);
    const long long row = unit / C;
    const int h = (int)(row % p.Hkv);
    const long long ts = row / p.Hkv;
    if (ts >= 2ll * p.T) return;
    const int side = (int)(ts & 1), t = (int)(ts >> 1);
    const int slot = __ldg(p.slots + t);
    const bool ok = slot >= 0 && slot < p.num_slots;
    if (slot != -1 && !ok && c == 0) atomicOr(p.err, (unsigned int)PA_ERRBIT_PAGE_RANGE);
    float x[8] = {};
    if (ok) {
        const kv4::Layout at{1 << p.ps_shift, D};
        const int r = slot & (at.ps - 1);
        const uint8_t *block = p.pool + ((long long)(slot >> p.ps_shift) * p.Hkv + h) * kv4::block_bytes(at.ps, D);
        const uint32_t w = *reinterpret_cast<const uint32_t *>(block + at.codes(side, r) + 4 * c);
        const float s = kv4::scale_value(block[at.scales(side, r) + c / 2]);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (float)((int)(w >> (4 * i) & 15u) - 8) * s;
    }
    T *dst = static_cast<T *>(side ? p.v_out : p.k_out) + ((long long)t * p.Hkv + h) * D + c * 8;
    if constexpr (sizeof(T) == 4) {
        reinterpret_cast<float4 *>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4 *>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        *reinterpret_cast<uint4 *>(dst) = make_uint4(MmaOp<T>::pack(x[0], x[1]), MmaOp<T>::pack(x[2], x[3]),
                                                     MmaOp<T>::pack(x[4], x[5]), MmaOp<T>::pack(x[6], x[7]));
    }
}

template <typename T, int D>
static cudaError_t launch_rows(const Kv4RowsParams &p, cudaStream_t stream) {
    const long long units = 2ll * p.T * p.Hkv * (D / 8);
    const long long blocks = (units + kThreads - 1) / kThreads;
    if (blocks == 0) return cudaSuccess;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (p.k_out)
        paged_attn_gather_kv4_kernel<T, D><<<(unsigned)blocks, kThreads, 0, stream>>>(p);
    else
        paged_attn_append_kv4_kernel<T, D><<<(unsigned)blocks, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename T>
static cudaError_t launch_rows_t(const Kv4RowsParams &p, int D, cudaStream_t stream) {
    if (D == 64) return launch_rows<T, 64>(p, stream);
    if (D == 128) return launch_rows<T, 128>(p, stream);
    return launch_rows<T, 256>(p, stream);
}

cudaError_t launch_kv4_rows(const Kv4RowsParams &p, int dtype, int D, cudaStream_t stream) {
    if (dtype == PA_F32) return launch_rows_t<float>(p, D, stream);
    if (dtype == PA_BF16) return launch_rows_t<__nv_bfloat16>(p, D, stream);
    return launch_rows_t<__half>(p, D, stream);
}

}  // namespace pa
