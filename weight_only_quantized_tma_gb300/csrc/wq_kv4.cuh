// wq_kv4.cuh -- device helpers for the 4-bit key / value cache (include/wq.h,
// wq_kv4_layout): 16-bit arithmetic in the cache's type, the unpack of code words and
// addressing inside a page block.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sm103_ptx.cuh"
#include "wq_internal.h"

namespace wq {

// Two values of the cache's type in a register.
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if (BF16) return ptx::f32x2_to_bf16x2(lo, hi);
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
    if (BF16) return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
// a * b + c on both halves, one rounding each (subnormals kept).
template <bool BF16>
__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    if (BF16)
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    else
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
template <bool BF16>
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
    uint32_t r;
    if (BF16)
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Smaller / larger of both halves; a NaN in either operand gives NaN.
template <bool BF16>
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    if (BF16)
        asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <bool BF16>
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    if (BF16)
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Codes to numbers.  A code OR-ed into the low mantissa bits of a constant gives
// base + q (fp16: 1024 + q at bits 0-3, 64 + q at bits 4-7; bf16: 128 + q at bits
// 0-3); subtracting the base is exact, and one fma gives RN(lo + q * s).
template <bool BF16>
struct Codes {
    static constexpr uint32_t kMagic = BF16 ? 0x43004300u : 0x64006400u;
    // codes in bits 0-3 and 16-19 of x
    static __device__ __forceinline__ uint32_t low(uint32_t x) {
        return sub2<BF16>(ptx::lop3_and_or(x, 0x000F000Fu, kMagic), kMagic);
    }
    // codes in bits 4-7 and 20-23
    static __device__ __forceinline__ uint32_t high(uint32_t x) {
        if (BF16) return low(x >> 4);
        return sub2<false>(ptx::lop3_and_or(x, 0x00F000F0u, 0x54005400u), 0x54005400u);
    }
};

// Eight codes of one word to the values of d = 0..7 in order, as four pairs.
// s2, lo2: the group's s and lo in both halves.
template <bool BF16>
__device__ __forceinline__ uint4 word_values(uint32_t w, uint32_t s2, uint32_t lo2) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t b = (w >> (8 * i)) & 0xFFu;
        o[i] = fma2<BF16>(Codes<BF16>::low(b | (b << 12)), s2, lo2);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Sums of bf16 values may pass what fp32 holds, so the attention kernels add them up in units of
// kSumUnit: that leaves 2^30 for the number of tokens and for a running maximum that lags behind,
// and rounds values below 2^-96 to 2^-104.
template <bool BF16>
constexpr float kSumUnit = BF16 ? 1073741824.0f : 1.0f;   // 2^30
// a pair (s, lo) in these units
template <bool BF16>
__device__ __forceinline__ uint32_t summand(uint32_t pair) {
    if (BF16) asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(pair) : "r"(0x30803080u));
    return pair;
}

// Codes to operands of the attention kernels: RN(lo + q s) for every s and lo, the value that the
// cache stands for (word_values gives the same).  Eight codes take 13 operations in fp16, 15 in
// bf16.
template <bool BF16>
struct Operand {
    uint32_t s, lo;
    Operand() = default;
    // s and lo of the low and of the high half, in the cache's type
    __device__ __forceinline__ Operand(uint32_t s2, uint32_t lo2) : s(s2), lo(lo2) {}
    // one pair (s, lo) for both halves
    static __device__ __forceinline__ Operand both(uint32_t pair) {
        return Operand(__byte_perm(pair, 0, 0x1010), __byte_perm(pair, 0, 0x3232));
    }
    // codes in bits 0-3 and 16-19 of x; in bits 4-7 and 20-23
    __device__ __forceinline__ uint32_t low(uint32_t x) const { return fma2<BF16>(Codes<BF16>::low(x), s, lo); }
    __device__ __forceinline__ uint32_t high(uint32_t x) const { return fma2<BF16>(Codes<BF16>::high(x), s, lo); }
};

// The same in bf16 with 9 operations for 8 codes, in units of 1 / kUp and for most pairs.  A number
// with exponent field 0 or 1 is its 8 low bits times 2^-133, so a code that is merely masked out is
// q 2^-133 (bits 0-3) or q 2^-129 (bits 4-7), and one fma with s 2^53 or s 2^49 and lo 2^-80 gives
// (lo + q s) 2^-80: no magic number, no subtraction, no shift for the upper code.  Steps s from
// 2^75 on overflow; what is no multiple of 2^-53 is rounded to one, by 2^-53 at most.  Where s and
// lo are zero or 2^-46 at least there is nothing to round.
struct ShortOperand {
    static constexpr float kUp = 1.2089258196146292e24f;   // 2^80
    uint32_t s_low, s_high, lo;
    ShortOperand() = default;
    __device__ __forceinline__ ShortOperand(uint32_t s2, uint32_t lo2) {
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(s_low) : "r"(s2), "r"(0x5A005A00u));
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(s_high) : "r"(s2), "r"(0x58005800u));
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(lo2), "r"(0x17801780u));
    }
    static __device__ __forceinline__ ShortOperand both(uint32_t pair) {
        return ShortOperand(__byte_perm(pair, 0, 0x1010), __byte_perm(pair, 0, 0x3232));
    }
    __device__ __forceinline__ uint32_t low(uint32_t x) const { return fma2<true>(x & 0x000F000Fu, s_low, lo); }
    __device__ __forceinline__ uint32_t high(uint32_t x) const { return fma2<true>(x & 0x00F000F0u, s_high, lo); }
    // Whether a pair is none of those that are taken exactly.
    static __device__ __forceinline__ bool refuses(uint32_t pair) {
        const uint32_t s = pair & 0x7FFFu, l = pair >> 16 & 0x7FFFu;
        constexpr uint32_t least = (127 - 46) << 7, past = (127 + 75) << 7;
        return (s != 0 && (s < least || s >= past)) || (l != 0 && (l < least || l >= past));
    }
};

// Two fp32 values in a 64-bit register: one instruction for both.
__device__ __forceinline__ uint64_t f2(float x, float y) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
    return d;
}
__device__ __forceinline__ float2 un2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma_f2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add_f2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Offsets inside a page block.
__device__ __forceinline__ int kv4_codes_at(const Kv4View& c, int which, int place) {
    return (which * c.P + place) * (c.D >> 1);
}
__device__ __forceinline__ int kv4_pairs_at(const Kv4View& c, int which, int place) {
    return c.P * c.D + (which * c.P + place) * ((c.D >> c.g_shift) * 4);
}

}  // namespace wq
