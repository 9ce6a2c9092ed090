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

// One group of LPR lanes takes `per` query heads or `per` key heads of one token, U at a time:
// the U rows' loads are all issued before the first is used, and the token's angles, the
// weight and the addresses are worked out once for all of them (8192 tokens of 64 heads of 128:
// 73.7 us with one row for each group, now 48.1 us, 273 MB at 5.7 TB/s; warps wait for memory
// half of the time, issue slots 64% full).
template <bool BF16, int LPR, int U>
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(const RopeParams p) {
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int lane = threadIdx.x % LPR;
    const uint32_t group = blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
    const uint32_t tok = fastdiv(group, p.div_groups);
    const int gi = (int)(group - tok * p.div_groups.d);
    const int64_t t = tok;
    const bool is_q = gi < p.q_groups;
    const int h_begin = (is_q ? gi : gi - p.q_groups) * p.per;
    const int heads = min(p.per, (is_q ? p.Hq : p.Hkv) - h_begin);
    bool active = t < p.T && lane * 8 < p.D;
    int64_t pos = 0;
    if (t < p.T) {
        pos = p.positions[t];
        if (pos < 0 || pos >= p.max_pos) {
            if (lane == 0) atomicOr(p.status, DEVICE_INDEX);
            active = false;
        }
    }
    const uint16_t* src = (is_q ? static_cast<const uint16_t*>(p.q) + t * p.q_stride
                                : static_cast<const uint16_t*>(p.k) + t * p.k_stride) + h_begin * p.D;
    uint16_t* dst = (is_q ? static_cast<uint16_t*>(p.q_out) + t * p.q_out_stride
                          : static_cast<uint16_t*>(p.k_out) + t * p.k_out_stride) + h_begin * p.D;
    const uint16_t* w = static_cast<const uint16_t*>(is_q ? p.q_weight : p.k_weight);
    // the two chunks (in values)
    const int pairs = p.rot >> 3;               // lanes with rotated chunks
    const bool turns = active && lane < pairs;
    const int ca = lane < pairs ? 4 * lane : p.rot + 8 * (lane - pairs);
    const int cb = lane < pairs ? ca + (p.rot >> 1) : ca + 4;
    // cosines and sines of the chunks' pairs: (a[i], b[i]), or neighbours in a and in b
    float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
    if (turns) {
        const float* cs = p.cos_sin + pos * p.rot;
        const float* sn = cs + (p.rot >> 1);
        if (p.interleaved) {
            const float2 c0 = *reinterpret_cast<const float2*>(cs + ca / 2), c1 = *reinterpret_cast<const float2*>(cs + cb / 2);
            const float2 s0 = *reinterpret_cast<const float2*>(sn + ca / 2), s1 = *reinterpret_cast<const float2*>(sn + cb / 2);
            c[0] = c0.x, c[1] = c0.y, c[2] = c1.x, c[3] = c1.y;
            s[0] = s0.x, s[1] = s0.y, s[2] = s1.x, s[3] = s1.y;
        } else {
            const float4 cv = *reinterpret_cast<const float4*>(cs + ca), sv = *reinterpret_cast<const float4*>(sn + ca);
            c[0] = cv.x, c[1] = cv.y, c[2] = cv.z, c[3] = cv.w;
            s[0] = sv.x, s[1] = sv.y, s[2] = sv.z, s[3] = sv.w;
        }
    }
    const float inv_d = 1.0f / (float)p.D;
    float wa[4] = {1.f, 1.f, 1.f, 1.f}, wb[4] = {1.f, 1.f, 1.f, 1.f};
    if (w != nullptr && active) {
        load4<BF16>(w + ca, wa);
        load4<BF16>(w + cb, wb);
    }
    for (int h0 = 0; h0 < p.per; h0 += U) {   // the same count for every lane
        uint2 ra[U], rb[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            ra[u] = rb[u] = make_uint2(0u, 0u);
            if (active && h0 + u < heads) {
                ra[u] = *reinterpret_cast<const uint2*>(src + (h0 + u) * p.D + ca);
                rb[u] = *reinterpret_cast<const uint2*>(src + (h0 + u) * p.D + cb);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float a[4], b[4];
            const float2 a0 = unpack2<BF16>(ra[u].x), a1 = unpack2<BF16>(ra[u].y);
            const float2 b0 = unpack2<BF16>(rb[u].x), b1 = unpack2<BF16>(rb[u].y);
            a[0] = a0.x, a[1] = a0.y, a[2] = a1.x, a[3] = a1.y;
            b[0] = b0.x, b[1] = b0.y, b[2] = b1.x, b[3] = b1.y;
            // every lane takes part in the exchange: rows with and without a weight share warps
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) sum += a[i] * a[i] + b[i] * b[i];
#pragma unroll
            for (int off = LPR / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            if (!active || h0 + u >= heads) continue;
            if (w != nullptr) {
                const float r = rsqrtf(sum * inv_d + p.eps);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[i] = a[i] * r * wa[i];
                    b[i] = b[i] * r * wb[i];
                }
            }
            if (turns) {
                if (p.interleaved) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float x = a[2 * i], y = b[2 * i];
                        a[2 * i] = x * c[i] - a[2 * i + 1] * s[i];
                        a[2 * i + 1] = a[2 * i + 1] * c[i] + x * s[i];
                        b[2 * i] = y * c[2 + i] - b[2 * i + 1] * s[2 + i];
                        b[2 * i + 1] = b[2 * i + 1] * c[2 + i] + y * s[2 + i];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float x = a[i];
                        a[i] = x * c[i] - b[i] * s[i];
                        b[i] = b[i] * c[i] + x * s[i];
                    }
                }
            }
            uint16_t* out = dst + (h0 + u) * p.D;
            *reinterpret_cast<uint2*>(out + ca) = make_uint2(pack2<BF16>(a[0], a[1]), pack2<BF16>(a[2], a[3]));
            *reinterpret_cast<uint2*>(out + cb) = make_uint2(pack2<BF16>(b[0], b[1]), pack2<BF16>(b[2], b[3]));
        }
    }
}

template <bool BF16, int LPR, int U>
cudaError_t launch_u(RopeParams p, int per, cudaStream_t st) {
    p.per = per;
    p.q_groups = (p.Hq + per - 1) / per;
    const uint32_t groups = (uint32_t)(p.q_groups + (p.Hkv + per - 1) / per);
    const int64_t all = p.T * groups;
    p.div_groups = make_fastdiv(groups, (uint32_t)(all + 256));
    return launch_pdl(qk_norm_rope_kernel<BF16, LPR, U>, (unsigned)((all * LPR + 255) / 256), 256, 0, st, p);
}

template <bool BF16, int LPR>
cudaError_t launch(const RopeParams& p, int sms, cudaStream_t st) {
    // As many heads for each group as leave two full blocks for each SM: 16 read the angles and
    // the weight least often, 1 spreads a decode step's few rows widest.  (8192 tokens of 32
    // query and 32 key heads of 128, rows in flight x heads: 2 x 16 48.1 us, 2 x 8 49.9, 2 x 32
    // 53.0, 2 x 4 54.3, 4 x 16 57.1, 4 x 8 57.8, 1 x 16 59.5, 2 x 2 66.1.)
    const int64_t want = (int64_t)sms * 2 * (256 / LPR);
    for (int per = 16; per >= 4; per /= 2)
        if (p.T * ((p.Hq + per - 1) / per + (p.Hkv + per - 1) / per) >= want) return launch_u<BF16, LPR, 2>(p, per, st);
    return launch_u<BF16, LPR, 1>(p, 1, st);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeParams& p, bool bf16, int sms, cudaStream_t st) {
    if (p.D <= 64) return bf16 ? launch<true, 8>(p, sms, st) : launch<false, 8>(p, sms, st);
    if (p.D <= 128) return bf16 ? launch<true, 16>(p, sms, st) : launch<false, 16>(p, sms, st);
    return bf16 ? launch<true, 32>(p, sms, st) : launch<false, 32>(p, sms, st);
}

}  // namespace wq
