// New tokens' K and V rows into a 4-bit pool, and rows of slots read back as the values they stand for.
//
// A thread of the first takes the 16 elements of a scale, so nothing is exchanged; one of the second eight.  Both move
// bytes.  What could hold the first up is arithmetic: with a division, a comparison for NaN and a look for infinities
// an element, 6994 prompt tokens of 8 heads of 128 (f16) took 21 us; with some 7 operations an element they take 11, 48 % of
// the copy rate (37 MB).  Reading them back takes 9.6; 261 single tokens 3.5 and 3.4, a chain of two trips to memory.
#include <float.h>

#include <type_traits>

#include "kernels.h"
#include "kv4.cuh"

namespace pa {

namespace {

constexpr int kThreads = 256;

// 16 elements as they are stored.
template <typename T>
struct Raw {
    static constexpr int N = (int)sizeof(T);  // 16-byte parts
    uint4 part[N];
    __device__ __forceinline__ void load(const T *src) {
#pragma unroll
        for (int i = 0; i < N; ++i) part[i] = __ldg(reinterpret_cast<const uint4 *>(src) + i);
    }
    __device__ __forceinline__ uint32_t word(int i) const {
        const uint4 &u = part[i / 4];
        return i % 4 == 0 ? u.x : i % 4 == 1 ? u.y : i % 4 == 2 ? u.z : u.w;
    }
    __device__ __forceinline__ void values(float (&x)[16]) const {
#pragma unroll
        for (int i = 0; i < 4 * N; ++i) {
            if constexpr (sizeof(T) == 4) {
                x[i] = __uint_as_float(word(i));
            } else {
                const float2 f = MmaOp<T>::unpack(word(i));
                x[2 * i] = f.x, x[2 * i + 1] = f.y;
            }
        }
    }
    // The largest magnitude as the type's bits, which are ordered as the magnitudes are; infinities and NaN above all.
    __device__ __forceinline__ uint32_t top() const {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4 * N; ++i) {
            if constexpr (sizeof(T) == 4)
                m = max(m, word(i) & 0x7fffffffu);
            else
                m = __vmaxu2(m, word(i) & 0x7fff7fffu);
        }
        if constexpr (sizeof(T) == 4)
            return m;
        else
            return max(m & 0xffffu, m >> 16);
    }
    __device__ __forceinline__ static float magnitude(uint32_t top) {
        if constexpr (sizeof(T) == 4)
            return __uint_as_float(top);
        else
            return MmaOp<T>::unpack(top).x;
    }
    static constexpr uint32_t kInfinity = sizeof(T) == 4 ? 0x7f800000u : std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
};

// clamp(rint(x / s), -7, 7) + 8 of eight elements, one to four bits.  CLAMP: quotients may be past 7.5 (they are not
// where the scale is neither the largest nor a subnormal number).
template <bool CLAMP>
__device__ __forceinline__ uint32_t quantise(const float *x, kv4::Reciprocal s) {
    constexpr float kMagic = 12582912.f + 8.f;  // 1.5 x 2^23: the sum's last bits are the integer
    uint32_t z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float q = kv4::divide(x[i], s);
        if (CLAMP) q = fminf(fmaxf(q, -7.f), 7.f);
        z[i] = __float_as_uint(q + kMagic);
    }
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = (z[2 * i + 1] << 4 & 0xf0u) | (z[2 * i] & 0x0fu);
    return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
}

}  // namespace

// A block: one kv head's K or V rows of U x kThreads / (D / 16) tokens.
template <typename T, int D, int U>
__global__ void __launch_bounds__(kThreads) paged_attn_append_kv4_kernel(const Kv4RowsParams p) {
    wait_for_stream();
    constexpr int C = D / kv4::kGroup, TPB = kThreads / C;  // threads of a row, rows at once
    const int c = threadIdx.x % C, side = blockIdx.y & 1, h = blockIdx.y >> 1;
    const long long t0 = (long long)blockIdx.x * (TPB * U) + threadIdx.x / C;
    const T *src = static_cast<const T *>(side ? p.v : p.k) + h * D + c * kv4::kGroup;
    const long long stride = side ? p.v_stride : p.k_stride;
    const kv4::Layout at{1 << p.ps_shift, D};
    int slot[U];
    Raw<T> raw[U];
#pragma unroll
    for (int k = 0; k < U; ++k) slot[k] = t0 + k * TPB < p.T ? __ldg(p.slots + t0 + k * TPB) : -1;
#pragma unroll
    for (int k = 0; k < U; ++k) {
        if (slot[k] < 0 || slot[k] >= p.num_slots) {
            if (slot[k] != -1 && c == 0) atomicOr(p.err, (unsigned int)PA_ERRBIT_PAGE_RANGE);
            slot[k] = -1;
        } else {
            raw[k].load(src + (t0 + k * TPB) * stride);
        }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
        if (slot[k] < 0) continue;
        float x[16];
        raw[k].values(x);
        const uint32_t top = raw[k].top();
        float a = Raw<T>::magnitude(top);
        if (top >= Raw<T>::kInfinity) {  // infinities count as the largest value, NaN as 0
            atomicOr(p.err, (unsigned int)PA_ERRBIT_NONFINITE);
            a = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                x[i] = x[i] == x[i] ? fminf(fmaxf(x[i], -FLT_MAX), FLT_MAX) : 0.f;
                a = fmaxf(a, fabsf(x[i]));
            }
        }
        const uint32_t byte = kv4::scale_byte(a);
        const int r = slot[k] & (at.ps - 1);
        uint8_t *block = p.pool + ((long long)(slot[k] >> p.ps_shift) * p.Hkv + h) * kv4::block_bytes(at.ps, D);
        uint2 code = make_uint2(0x88888888u, 0x88888888u);
        if (byte) {
            const kv4::Reciprocal s = kv4::reciprocal(kv4::scale_value(byte));
            if (byte >= 8 && byte < kv4::kMaxScaleByte)
                code = make_uint2(quantise<false>(x, s), quantise<false>(x + 8, s));
            else
                code = make_uint2(quantise<true>(x, s), quantise<true>(x + 8, s));
        }
        *reinterpret_cast<uint2 *>(block + at.codes(side, r) + 8 * c) = code;
        block[at.scales(side, r) + c] = (uint8_t)byte;
    }
}

template <typename T, int D, int U>
__global__ void __launch_bounds__(kThreads) paged_attn_gather_kv4_kernel(const Kv4RowsParams p) {
    wait_for_stream();
    constexpr int C = D / 8, TPB = kThreads / C;
    const int c = threadIdx.x % C, side = blockIdx.y & 1, h = blockIdx.y >> 1;
    const long long t0 = (long long)blockIdx.x * (TPB * U) + threadIdx.x / C;
    const kv4::Layout at{1 << p.ps_shift, D};
    int slot[U];
    uint32_t w[U];
    float s[U];
#pragma unroll
    for (int k = 0; k < U; ++k) slot[k] = t0 + k * TPB < p.T ? __ldg(p.slots + t0 + k * TPB) : -1;
#pragma unroll
    for (int k = 0; k < U; ++k) {
        w[k] = 0x88888888u;
        s[k] = 0.f;
        if (slot[k] < 0 || slot[k] >= p.num_slots) {
            if (slot[k] != -1 && c == 0) atomicOr(p.err, (unsigned int)PA_ERRBIT_PAGE_RANGE);
            continue;
        }
        const int r = slot[k] & (at.ps - 1);
        const uint8_t *block = p.pool + ((long long)(slot[k] >> p.ps_shift) * p.Hkv + h) * kv4::block_bytes(at.ps, D);
        w[k] = *reinterpret_cast<const uint32_t *>(block + at.codes(side, r) + 4 * c);
        s[k] = kv4::scale_value(block[at.scales(side, r) + c / 2]);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
        if (t0 + k * TPB >= p.T) continue;
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (float)((int)(w[k] >> (4 * i) & 15u) - 8) * s[k];
        T *dst = static_cast<T *>(side ? p.v_out : p.k_out) + ((t0 + k * TPB) * p.Hkv + h) * D + c * 8;
        if constexpr (sizeof(T) == 4) {
            reinterpret_cast<float4 *>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
            reinterpret_cast<float4 *>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
        } else {
            *reinterpret_cast<uint4 *>(dst) = make_uint4(MmaOp<T>::pack(x[0], x[1]), MmaOp<T>::pack(x[2], x[3]),
                                                         MmaOp<T>::pack(x[4], x[5]), MmaOp<T>::pack(x[6], x[7]));
        }
    }
}

template <typename T, int D, int U>
static cudaError_t launch_rows_u(const Kv4RowsParams &p, cudaStream_t stream) {
    const int rows = kThreads / (p.k_out ? D / 8 : D / kv4::kGroup) * U;
    const dim3 grid((unsigned)(((long long)p.T + rows - 1) / rows), (unsigned)(2 * p.Hkv));
    return launch_behind(p.k_out ? paged_attn_gather_kv4_kernel<T, D, U> : paged_attn_append_kv4_kernel<T, D, U>, grid, kThreads, 0,
                         1, stream, p);
}

template <typename T, int D>
static cudaError_t launch_rows(const Kv4RowsParams &p, cudaStream_t stream) {
    // Rows for every multiprocessor many times over: several loads of a thread on their way together.
    if ((long long)p.T * p.Hkv * (D / 8) >= (1 << 19)) return launch_rows_u<T, D, 4>(p, stream);
    return launch_rows_u<T, D, 1>(p, stream);
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
