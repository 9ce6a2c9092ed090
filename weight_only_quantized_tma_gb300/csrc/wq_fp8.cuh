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

// The scale of a block whose largest magnitude is `most`, and what its values are multiplied with.  An
// infinity or a NaN in the block gives a NaN for the scale (and codes of 0): the block's values are NaN.
// most / 448 is rounded exactly: the product with 1 / 448 and one correction by its exact residual (Markstein's method;
// where the residual would leave the normal range the scale is the least one).  A value's product with the reciprocal
// is within 2^-22 of its quotient, so that only one that close to the middle between two codes can become the other
// of them.
struct BlockScale {
    float scale, inv;
    __device__ __forceinline__ explicit BlockScale(float most) {
        const bool finite = most <= 3.402823466e38f;
        const float q = most * (1.0f / 448.0f);
        scale = finite ? fmaxf(fmaf(fmaf(-448.0f, q, most), 1.0f / 448.0f, q), 0x1p-96f) : __int_as_float(0x7FC00000);
        inv = finite ? about_reciprocal(scale) : 0.0f;
    }
};

// The largest magnitude of a warp's values in every lane; a NaN among them gives NaN.
__device__ __forceinline__ float warp_most(float v) {
    float r;
    asm volatile("redux.sync.max.abs.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// g / (1 + exp(-g)): -0 far below (exp overflows to infinity), NaN at minus infinity (0 times it).  The exponential and
// the reciprocal are the special function unit's own, whose results below the normal range are zeros.
__device__ __forceinline__ float silu(float g) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
    return g * about_reciprocal(1.0f + e);
}

}  // namespace wq
