// opq_fp8_format.cuh — the 8-bit block format: e4m3 codes (4 exponent bits, 3 mantissa bits,
// largest value 448) with one fp32 scale per block of up to 128 values.
//
//   m     = max(largest finite |x| of the block, 2^-64)
//   scale = fl32(m / 448)
//   code  = the e4m3 number nearest 448 x / m, ties to even;  +-inf -> +-448, NaN -> NaN
//   value = fl32(code * scale), rounded once more to the output's 16-bit type
//
// The code is exact for bf16 and fp16 inputs, with one multiplication and one mask per value. The
// encoder multiplies by (448 / m) (1 + 2^-21), formed in fp32, so that the fp32 product is the real
// quotient 448 x / m times 1 + e with 0 < e < 2^-20, and clears the product's four lowest bits.
//   - A quotient halfway between two codes has at most 5 significant bits; its product is above it
//     by less than the 2^-19 that the mask removes, so the mask returns it exactly and the
//     conversion sees the tie.
//   - Any other quotient differs from every midpoint by at least 2^-16 of its size (448 x has at
//     most 14 bits, m 11, a midpoint 5), which neither e nor the mask can bridge.
// Infinities stay infinite and saturate to 448, NaN stays NaN. (Dividing, or correcting the product
// by a residual, gives the same codes at two to four times the arithmetic.)
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace opqfp8 {

constexpr int kBlock = 128;                       // values that share a scale along the row
constexpr float kFloor = 5.421010862427522e-20f;  // 2^-64

enum { DT_BF16 = 0, DT_FP16 = 1 };

// Per-block constants of m. Each takes a division, some ten instructions or more, so where lanes
// hold several blocks each block's are formed by one lane and handed around.
__device__ __forceinline__ float floored(float amax) { return fmaxf(amax, kFloor); }
__device__ __forceinline__ float block_scale(float m) { return m / 448.0f; }
__device__ __forceinline__ float block_mul(float m) { return (448.0f / m) * 1.000000476837158203125f; }   // 1 + 2^-21

// Two fp32 operands per instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

// Two fp32 values to e4m3, nearest even, magnitudes above 448 to 448, NaN kept: x in bits 0..7.
__device__ __forceinline__ uint32_t cvt_e4m3x2(float2 v) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(v.y), "f"(v.x));
    return d;
}

// Two e4m3 values (bits 0..7 and 8..15) to fp32, exact (through fp16, whose range and precision
// contain e4m3's).
__device__ __forceinline__ float2 decode_e4m3x2(uint16_t c) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

template <int DT>
__device__ __forceinline__ float2 unpack16(uint32_t w) {
    if (DT == DT_BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
template <int DT>
__device__ __forceinline__ uint32_t pack16(float2 v) {
    uint32_t d;
    if (DT == DT_BF16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(v.y), "f"(v.x));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(v.y), "f"(v.x));
    return d;
}
// One fp32 value rounded to the 16-bit type.
template <int DT>
__device__ __forceinline__ uint16_t pack16_1(float v) {
    return (uint16_t)pack16<DT>(make_float2(v, 0.0f));
}
template <int DT>
__device__ __forceinline__ float unpack16_1(uint16_t v) {
    return DT == DT_BF16 ? __uint_as_float((uint32_t)v << 16) : __half2float(__ushort_as_half(v));
}

// Magnitudes order as integers; bits at or above kInfBits say that an infinity or a NaN is among
// the values.
template <int DT>
constexpr uint32_t kInfBits = DT == DT_BF16 ? 0x7F80u : 0x7C00u;

// Per half: the larger magnitude (NaN if there is one) with some sign, one instruction.
template <int DT>
__device__ __forceinline__ uint32_t absmax2(uint32_t a, uint32_t b) {
    uint32_t d;
    if (DT == DT_BF16)
        asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else
        asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// of eight values: two candidates, in the halves
template <int DT>
__device__ __forceinline__ uint32_t absmax8(const uint4 &v) {
    return absmax2<DT>(absmax2<DT>(v.x, v.y), absmax2<DT>(v.z, v.w));
}
// the larger of a word's halves, without its sign
template <int DT>
__device__ __forceinline__ uint32_t absmax_bits(uint32_t w) {
    return absmax2<DT>(w, w >> 16) & 0x7FFFu;
}
// The same over the finite values only (the rare block that holds an infinity or a NaN).
template <int DT>
__device__ __forceinline__ uint32_t absmax8_finite(const uint4 &v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
        if (lo < kInfBits<DT>) best = max(best, lo);
        if (hi < kInfBits<DT>) best = max(best, hi);
    }
    return best;
}
template <int DT>
__device__ __forceinline__ float bits_to_float(uint32_t b) {
    return unpack16_1<DT>((uint16_t)b);
}

// Eight values to eight codes; mul = block_mul(m).
template <int DT>
__device__ __forceinline__ uint2 encode8(const uint4 &v, float mul) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 q = mul2(unpack16<DT>(w[i]), make_float2(mul, mul));
        q.x = __uint_as_float(__float_as_uint(q.x) & 0xFFFFFFF0u);
        q.y = __uint_as_float(__float_as_uint(q.y) & 0xFFFFFFF0u);
        c[i] = cvt_e4m3x2(q);
    }
    return make_uint2(__byte_perm(c[0], c[1], 0x5410u), __byte_perm(c[2], c[3], 0x5410u));
}

// Largest magnitudes of U blocks, each held by LANES neighbouring lanes (eight values a lane):
// two blocks' maxima travel in one word. A block with an infinity or a NaN takes its finite values'.
template <int DT, int LANES, int U>
__device__ __forceinline__ void block_maxima(const uint4 (&v)[U], uint32_t (&mx)[U]) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < U; i += 2) {
        const uint32_t a = absmax8<DT>(v[i]), b = absmax8<DT>(v[i + 1 < U ? i + 1 : i]);
        uint32_t w = absmax2<DT>(__byte_perm(a, b, 0x5410u), __byte_perm(a, b, 0x7632u));   // a's, b's
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) w = absmax2<DT>(w, __shfl_xor_sync(0xFFFFFFFFu, w, o));
        mx[i] = w & 0x7FFFu;
        if (i + 1 < U) mx[i + 1] = (w >> 16) & 0x7FFFu;
        top = absmax2<DT>(top, w);
    }
    if (__any_sync(0xFFFFFFFFu, absmax_bits<DT>(top) >= kInfBits<DT>)) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            uint32_t f = absmax8_finite<DT>(v[i]);
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1) f = max(f, __shfl_xor_sync(0xFFFFFFFFu, f, o));
            mx[i] = f;
        }
    }
}

// n / d and n % d for n < 2^31 by a multiplication (d is fixed per launch).
struct FastDiv {
    uint32_t d, mul, shift;
    __host__ static FastDiv make(uint32_t d) {
        FastDiv f{};
        f.d = d;
        uint32_t s = 0;
        while (((uint64_t)1 << s) < d) ++s;
        f.mul = (uint32_t)((((uint64_t)1 << (31 + s)) + d - 1) / d);   // d = 1: 2^31
        f.shift = 31 + s;
        return f;
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const { return (uint32_t)(((uint64_t)n * mul) >> shift); }
};

}  // namespace opqfp8
