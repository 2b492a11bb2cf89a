// The 4-bit cache: how a pool's bytes stand for K and V elements.
//
// The block of a (page, kv head) is contiguous: the K codes of its page_size rows (D / 2 bytes a row: element 2i
// in the low half of byte i, 2i + 1 in the high one), the V codes, the K scales (D / 16 bytes a row) and the V
// scales.  A code u in 0 .. 15 stands for u - 8, a scale byte for a number of five exponent and three mantissa
// bits without a sign: shifted left by 7 its bits are the f16 number's; bytes past kMaxScaleByte count as it, so
// that any byte is finite.  The element is (u - 8) x scale: at most four significant bits by four, an exact f16
// and bf16 number.
#pragma once

#include "mma_common.cuh"

namespace pa {

// See launch_behind: everything that the stream's earlier kernels wrote is there, and they have read what they read.
__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

namespace kv4 {

constexpr int kGroup = 16;                 // elements that share a scale
constexpr uint32_t kMaxScaleByte = 0xDE;   // 7168: nine times the largest scale is still an f16 number (see unpack8)
constexpr float kMaxScale = 7168.f;

__host__ __device__ constexpr int block_bytes(int ps, int D) { return ps * D / 8 * 9; }

// Where a row's parts stand in a block.
struct Layout {
    int ps, D;
    __host__ __device__ constexpr int codes(int side, int row) const { return (side * ps + row) * (D / 2); }
    __host__ __device__ constexpr int scales(int side, int row) const { return ps * D + (side * ps + row) * (D / kGroup); }
};

__device__ __forceinline__ float scale_value(uint32_t byte) {
    return __half2float(__ushort_as_half((unsigned short)(min(byte, kMaxScaleByte) << 7)));
}

// x / d rounded to nearest even, or beside it by less than 2^-45 of the quotient before its one rounding: hi is 1 / d
// in float32 and lo what that lacks.  Where the exact quotient is a border between two results (a number of at most five
// significant bits), so is this; where it lies beside one, it is more than half a unit in the last place off it (x
// is a unit off d times the border, which has at most nine significant bits, and d < 8 in the units of its exponent), and
// stays on its side.
struct Reciprocal {
    float hi, lo;
};
__device__ __forceinline__ float divide(float x, Reciprocal d) { return fmaf(x, d.hi, __fmul_rn(x, d.lo)); }
__device__ __forceinline__ Reciprocal reciprocal(float d) {
    const float hi = __frcp_rn(d);
    return {hi, __fmul_rn(fmaf(-hi, d, 1.f), hi)};
}

// The scale byte of 16 elements whose largest magnitude is a (not a NaN): a / 7 rounded to nearest even.
__device__ __forceinline__ uint32_t scale_byte(float a) {
    constexpr Reciprocal seventh{1.f / 7.f, (float)(1.0 / 7.0 - (double)(1.f / 7.f))};
    const float t = fminf(divide(fminf(a, 8.f * kMaxScale), seventh), kMaxScale);
    if (t < 0x1p-14f) return (uint32_t)__float2int_rn(t * 0x1p17f);  // multiples of 2^-17
    const uint32_t u = __float_as_uint(t);
    return min(((u + 0x7FFFFu + ((u >> 20) & 1u)) >> 20) - (112u << 3), kMaxScaleByte);
}

// Eight codes of a word -> four f16 pairs, pair k = codes k and k + 4: the odd ones as (u - 8) x scale / 8, the even ones,
// which lie four bits lower, as (u - 8) x scale / 128.  To put a few bits below the leading one of 1024 is the usual way to make
// small integers f16 numbers; the shares and constants are this format's.  A code put below the leading bits of an f16 number reads
// 1024 + 16 u or 1024 + u, and with s = scale / 128, c = -9 scale and d = -8.0625 scale
//   (1024 + 16 u) s + c = (u - 8) scale / 8,   (1024 + u) s + d = (u - 8) scale / 128
// in one rounding, which has nothing to round (an f16 number's last bit is 2^-24 at least, the smallest scale's
// 2^-17; c and d are a scale's four significant bits times 9 and 129).  The missing 16 of the even elements is put into the
// queries and into the output's columns; bringing the even codes up to the odd ones' place takes two shifts a word
// (256 sequences 170 us instead of 164).
// HALF 0, 1: that half of b and c for both halves of a, which the instruction chooses by itself (as a statement of its own the
// choice takes a move: 162 us instead of 159).  kPair: each its own.
constexpr int kPair = -1;
template <int HALF>
__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    if constexpr (HALF == kPair)
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    else if constexpr (HALF == 0)
        asm("{\n\t.reg .b16 p, q, r, t;\n\t.reg .b32 x, y;\n\tmov.b32 {p, q}, %2;\n\tmov.b32 {r, t}, %3;\n\t"
            "mov.b32 x, {p, p};\n\tmov.b32 y, {r, r};\n\tfma.rn.f16x2 %0, %1, x, y;\n\t}"
            : "=r"(d) : "r"(a), "r"(b), "r"(c));
    else
        asm("{\n\t.reg .b16 p, q, r, t;\n\t.reg .b32 x, y;\n\tmov.b32 {p, q}, %2;\n\tmov.b32 {r, t}, %3;\n\t"
            "mov.b32 x, {q, q};\n\tmov.b32 y, {t, t};\n\tfma.rn.f16x2 %0, %1, x, y;\n\t}"
            : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// (a & mask) | 0x64006400, as the one operation that it is (written in C the decode kernel executed 494 instructions a block
// of 16 keys instead of 431).
__device__ __forceinline__ uint32_t code_in_f16(uint32_t a, uint32_t mask) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(mask), "r"(0x64006400u));
    return d;
}
constexpr float kEvenShare = 16.f;  // what an even element lacks beside an odd one
struct ScalePair {  // of two scales, one for each half of a pair
    uint32_t s, c, d;
};
template <int HALF = kPair>
__device__ __forceinline__ void unpack8(uint32_t w, ScalePair x, uint32_t (&h)[4]) {
    const uint32_t v = w >> 8;
    h[0] = fma2<HALF>(code_in_f16(w, 0x000F000Fu), x.s, x.d);
    h[1] = fma2<HALF>(code_in_f16(w, 0x00F000F0u), x.s, x.c);
    h[2] = fma2<HALF>(code_in_f16(v, 0x000F000Fu), x.s, x.d);
    h[3] = fma2<HALF>(code_in_f16(v, 0x00F000F0u), x.s, x.c);
}
// From two scale bytes, one in the low byte of each half of x.
__device__ __forceinline__ ScalePair scale_pair(uint32_t x) {
    uint32_t f;
    asm("min.f16x2 %0, %1, %2;" : "=r"(f) : "r"(x << 7), "r"(0x6F006F00u));  // 7168; a NaN's bits give it too
    return {mul2(f, 0x20002000u), mul2(f, 0xC880C880u), mul2(f, 0xC808C808u)};  // 2^-7, -9, -8.0625
}

// A row of queries in f16: by a power of two into its range, elements that meet odd ones a sixteenth of that.  w: pairs, the
// even elements' first; largest: the row's largest magnitude.  The result, with the factors of the keys' elements, is
// to be multiplied by the value returned.
template <typename T, int N>
__device__ __forceinline__ float scale_query(uint32_t (&w)[N], float largest) {
    float inv;
    const float even = mmac::f16_row_scale(largest, inv), odd = even / kEvenShare;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float2 x = MmaOp<T>::unpack(w[i]);
        const float f = i & 1 ? odd : even;
        w[i] = MmaOp<__half>::pack(x.x * f, x.y * f);
    }
    return 8.f * kEvenShare * inv;
}
template <typename T, int N>
__device__ __forceinline__ float largest_of(const uint32_t (&w)[N]) {
    float am = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float2 x = MmaOp<T>::unpack(w[i]);
        am = fmaxf(am, fmaxf(fabsf(x.x), fabsf(x.y)));
    }
    return am;
}

}  // namespace kv4
}  // namespace pa
