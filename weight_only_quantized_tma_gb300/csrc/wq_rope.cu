// wq_rope.cu -- norms of queries and keys for each head and their rotation by position
// (include/wq.h: wq_qk_norm_rope).
//
//   y = x * rsqrt(mean(x^2) + eps) * w,   (a, b) -> (a cos - b sin, b cos + a sin)
//
// A row (one head of one token) is D / 8 lanes.  A lane holds two chunks of 4 values: for
// the rotated part chunk j and chunk j + rot / 8, which are each other's partners in the
// half-split form, so no value moves between lanes; the sum of squares is the only
// exchange (xor shuffles).
#include "wq_kv4.cuh"

namespace wq {
namespace {

template <bool BF16>
__device__ __forceinline__ void load4(const uint16_t* p, float (&x)[4]) {
    const uint2 r = *reinterpret_cast<const uint2*>(p);
    const float2 a = unpack2<BF16>(r.x), b = unpack2<BF16>(r.y);
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
}

template <bool BF16, int LPR>
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(const RopeParams p) {
    const int lane = threadIdx.x % LPR;
    const int64_t row = (int64_t)blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
    const int heads = p.Hq + p.Hkv;
    const int64_t t = row / heads;
    const int h = (int)(row - t * heads);
    bool active = t < p.T && lane * 8 < p.D;
    int64_t pos = 0;
    if (t < p.T) {
        pos = p.positions[t];
        if (pos < 0 || pos >= p.max_pos) {
            if (lane == 0) atomicOr(p.status, DEVICE_INDEX);
            active = false;
        }
    }
    const bool is_q = h < p.Hq;
    const int64_t in_at = is_q ? t * p.q_stride + (int64_t)h * p.D : t * p.k_stride + (int64_t)(h - p.Hq) * p.D;
    const int64_t out_at =
        is_q ? t * p.q_out_stride + (int64_t)h * p.D : t * p.k_out_stride + (int64_t)(h - p.Hq) * p.D;
    const uint16_t* src = static_cast<const uint16_t*>(is_q ? p.q : p.k) + in_at;
    uint16_t* dst = static_cast<uint16_t*>(is_q ? p.q_out : p.k_out) + out_at;
    const uint16_t* w = static_cast<const uint16_t*>(is_q ? p.q_weight : p.k_weight);
    // the two chunks (in values)
    const int pairs = p.rot >> 3;               // lanes with rotated chunks
    const bool turns = lane < pairs;
    const int ca = turns ? 4 * lane : p.rot + 8 * (lane - pairs);
    const int cb = turns ? ca + (p.rot >> 1) : ca + 4;
    float a[4] = {0.f, 0.f, 0.f, 0.f}, b[4] = {0.f, 0.f, 0.f, 0.f};
    if (active) {
        load4<BF16>(src + ca, a);
        load4<BF16>(src + cb, b);
    }
    // every lane takes part in the exchange: rows with and without a weight share warps
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) sum += a[i] * a[i] + b[i] * b[i];
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (w != nullptr && active) {
        const float r = rsqrtf(sum / (float)p.D + p.eps);
        float wa[4], wb[4];
        load4<BF16>(w + ca, wa);
        load4<BF16>(w + cb, wb);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = a[i] * r * wa[i];
            b[i] = b[i] * r * wb[i];
        }
    }
    if (!active) return;
    if (turns) {
        const float* cs = p.cos_sin + pos * p.rot;
        const float* sn = cs + (p.rot >> 1);
        if (p.interleaved) {
            const float2 c0 = *reinterpret_cast<const float2*>(cs + ca / 2), c1 = *reinterpret_cast<const float2*>(cs + cb / 2);
            const float2 s0 = *reinterpret_cast<const float2*>(sn + ca / 2), s1 = *reinterpret_cast<const float2*>(sn + cb / 2);
            const float x0 = a[0], x1 = a[2], y0 = b[0], y1 = b[2];
            a[0] = x0 * c0.x - a[1] * s0.x, a[1] = a[1] * c0.x + x0 * s0.x;
            a[2] = x1 * c0.y - a[3] * s0.y, a[3] = a[3] * c0.y + x1 * s0.y;
            b[0] = y0 * c1.x - b[1] * s1.x, b[1] = b[1] * c1.x + y0 * s1.x;
            b[2] = y1 * c1.y - b[3] * s1.y, b[3] = b[3] * c1.y + y1 * s1.y;
        } else {
            const float4 c = *reinterpret_cast<const float4*>(cs + ca), s = *reinterpret_cast<const float4*>(sn + ca);
            const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = a[i];
                a[i] = x * cc[i] - b[i] * ss[i];
                b[i] = b[i] * cc[i] + x * ss[i];
            }
        }
    }
    *reinterpret_cast<uint2*>(dst + ca) = make_uint2(pack2<BF16>(a[0], a[1]), pack2<BF16>(a[2], a[3]));
    *reinterpret_cast<uint2*>(dst + cb) = make_uint2(pack2<BF16>(b[0], b[1]), pack2<BF16>(b[2], b[3]));
}

template <bool BF16>
cudaError_t launch(const RopeParams& p, cudaStream_t st) {
    const int64_t rows = p.T * (p.Hq + p.Hkv);
    auto grid = [&](int lpr) { return (unsigned)((rows * lpr + 255) / 256); };
    if (p.D <= 64)
        qk_norm_rope_kernel<BF16, 8><<<grid(8), 256, 0, st>>>(p);
    else if (p.D <= 128)
        qk_norm_rope_kernel<BF16, 16><<<grid(16), 256, 0, st>>>(p);
    else
        qk_norm_rope_kernel<BF16, 32><<<grid(32), 256, 0, st>>>(p);
    return cudaPeekAtLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeParams& p, bool bf16, int sms, cudaStream_t st) {
    (void)sms;
    return bf16 ? launch<true>(p, st) : launch<false>(p, st);
}

}  // namespace wq
