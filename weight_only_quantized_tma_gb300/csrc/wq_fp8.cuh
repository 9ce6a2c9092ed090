// wq_fp8.cuh -- device helpers for 8-bit (e4m3) activations with a scale for each token and
// block of 128 values (include/wq.h, "8-bit activations").
#pragma once

#include "wq_kv4.cuh"

namespace wq {

__device__ __forceinline__ float about_reciprocal(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Larger of both; a NaN in either gives NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Four fp32 to four e4m3 codes (a in the lowest byte), nearest even, at most +-448.
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
        "mov.b32 %0, {l, h};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

// The scale of a block whose largest magnitude is `most`, and its values' codes.  An infinity or a NaN in the block gives
// a NaN for the scale and codes of 0: the block's values are NaN.
// Both divisions are Markstein's method: a product with the reciprocal, corrected once by its exact residual.  most / 448
// is rounded exactly (where the residual would leave the normal range the scale is the least one).  A value's quotient by
// the scale decides its code as the exactly rounded fp32 quotient does, ties included: the reciprocal, a Newton step
// behind the special function unit's, is rounded exactly (compared for every mantissa), and both quotients lie on the
// same side of every middle between two codes (compared for every mantissa of a scale with the values around what rounds
// to a middle, the only ones that could differ).  Of scales between 2^-96 and 2^-93, whose residuals lose bits below
// fp32's range, eight with one value each come out on the other side.  (The product alone puts one code in 2000 of bf16
// values there.  Without the correction 8192 x 11008 fp16 values take 40.3 us instead of 40.8; a branch that brings low
// scales into range costs 41.8.)
struct BlockScale {
    float scale, div, inv;       // inv: minus the reciprocal of div
    uint32_t keep;               // 0: codes of 0
    __device__ __forceinline__ explicit BlockScale(float most) {
        const bool finite = most <= 3.402823466e38f;
        const float q = most * (1.0f / 448.0f);
        div = fmaxf(fmaf(fmaf(-448.0f, q, most), 1.0f / 448.0f, q), 0x1p-96f);     // (not finite: the least)
        const float r = about_reciprocal(div);
        inv = -fmaf(r, fmaf(-div, r, 1.0f), r);
        scale = finite ? div : __int_as_float(0x7FC00000);
        keep = finite ? 0xFFFFFFFFu : 0u;
    }
    // A quotient: residuals have the signs that keep a zero's.
    __device__ __forceinline__ float over(float y) const {
        const float q = y * -inv;
        return fmaf(fmaf(div, q, -y), inv, q);
    }
    // Minus two quotients (packed numbers have no sign to turn on the way).
    __device__ __forceinline__ float2 minus(uint64_t y) const {
        const uint64_t by = f2(inv, inv), n = mul_f2(y, by);
        return un2(fma_f2(fma_f2(f2(div, div), n, y), by, n));
    }
    // Codes of four values, the first in the lowest byte: packed where every instruction counts (8192 x 11008 fp16 values
    // 40.9 us, 43.6 one by one), one by one where registers do (gated 4096 x 11008 x 4096 289 us, packed 293).
    __device__ __forceinline__ uint32_t codes(uint64_t a, uint64_t b) const {
        const float2 m = minus(a), n = minus(b);
        return (to_e4m3x4(m.x, m.y, n.x, n.y) ^ 0x80808080u) & keep;
    }
    __device__ __forceinline__ uint32_t codes(float a, float b, float c, float d) const {
        return to_e4m3x4(over(a), over(b), over(c), over(d)) & keep;
    }
    __device__ __forceinline__ uint8_t code(float y) const { return (uint8_t)(to_e4m3x4(over(y), 0.f, 0.f, 0.f) & keep); }
};

// The largest magnitude of a warp's values in every lane; a NaN among them gives NaN.
__device__ __forceinline__ float warp_most(float v) {
    float r;
    asm volatile("redux.sync.max.abs.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// g / (1 + exp(-g)): -0 where exp overflows to infinity, NaN at minus infinity (0 times it).  The exponential and the
// reciprocal are the special function unit's own: the exponential's argument is off by 2^-24 of itself, the exponential by
// as much as that is, which at -88 is 2^-18 of the result and nothing beside a rounding to 16 or 8 bits.  Their results
// below the normal range are zeros, so the reciprocal is taken of a quarter of 1 + exp(-g), which ends at 2^126.  (In
// packed pairs: 293.9 us for gated 4096 x 11008 x 4096, 291.5 so.)
__device__ __forceinline__ float silu(float g) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
    return g * 0.25f * about_reciprocal(fmaf(e, 0.25f, 0.25f));
}

}  // namespace wq
