// wq_attn_simple.cu -- attention over the 4-bit cache, the plain way: one warp for each
// query row walks its visible tokens with a running maximum and sum, fp32 throughout.
#include "wq_kv4.cuh"

namespace wq {
namespace {

template <bool BF16, int D>
__global__ void __launch_bounds__(128) attn_simple_kernel(const AttnParams p) {
    constexpr int E = D / 32;   // values of d per lane
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int64_t t = row / p.Hq;
    const int h = (int)(row - t * p.Hq);
    if (t >= p.T) return;
    int64_t seq = -1;
    int i = 0, n = 1;
    if (p.cu_q == nullptr) {
        seq = t;
    } else {
        for (int64_t b0 = 0; b0 < p.B && seq < 0; b0 += 32) {
            const int64_t b = b0 + lane;
            const bool mine = b < p.B && p.cu_q[b] <= t && t < p.cu_q[b + 1];
            const uint32_t m = __ballot_sync(0xffffffffu, mine);
            if (m) seq = b0 + __ffs(m) - 1;
        }
        if (seq < 0) return;
        i = (int)t - p.cu_q[seq];
        n = p.cu_q[seq + 1] - p.cu_q[seq];
    }
    int64_t L = p.lens[seq];
    if (L > p.table_stride * p.c.P) {
        L = p.table_stride * p.c.P;
        if (lane == 0) atomicOr(p.status, DEVICE_INDEX);
    }
    const int64_t pos = L - n + i;
    const int64_t end = p.causal ? (pos + 1 < L ? pos + 1 : L) : L;
    const int64_t begin = p.window > 0 && pos + 1 > p.window ? pos + 1 - p.window : 0;
    const uint16_t* q = static_cast<const uint16_t*>(p.q) + t * p.q_stride + (int64_t)h * D + lane * E;
    float x[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; e += 2) {
        const float2 f = unpack2<BF16>(*reinterpret_cast<const uint32_t*>(q + e));
        x[e] = f.x, x[e + 1] = f.y;
        o[e] = o[e + 1] = 0.f;
    }
    const int kh = h / p.group;
    for (int64_t j = begin; j < end; ++j) {
        int64_t page = p.table[seq * p.table_stride + (j >> p.c.p_shift)];
        if (page < 0 || page >= p.c.num_pages) {
            if (lane == 0) atomicOr(p.status, DEVICE_INDEX);
            page = 0;
        }
        const int place = (int)(j & (p.c.P - 1));
        const uint8_t* block = p.c.pages + page * p.c.page_bytes + (int64_t)kh * p.c.block_bytes;
        float kv[2][E];
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const uint8_t* codes = block + kv4_codes_at(p.c, which, place) + lane * E / 2;
            const uint32_t pair = *reinterpret_cast<const uint32_t*>(block + kv4_pairs_at(p.c, which, place) +
                                                                     ((lane * E) >> p.c.g_shift) * 4);
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const uint32_t b = codes[e / 2];
                const float2 f = unpack2<BF16>(fma2<BF16>(Codes<BF16>::low(b | (b << 12)), __byte_perm(pair, 0, 0x1010),
                                                          __byte_perm(pair, 0, 0x3232)));
                kv[which][e] = f.x, kv[which][e + 1] = f.y;
            }
        }
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s += x[e] * kv[0][e];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= p.scale;
        const float m1 = fmaxf(m, s), safe = m1 == -INFINITY ? 0.f : m1;
        const float w = __expf(m - safe), e1 = __expf(s - safe);
        l = l * w + e1;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * w + e1 * kv[1][e];
        m = m1;
    }
    uint16_t* out = static_cast<uint16_t*>(p.out) + t * p.out_stride + (int64_t)h * D + lane * E;
    const bool empty = begin >= end;
#pragma unroll
    for (int e = 0; e < E; e += 2)
        *reinterpret_cast<uint32_t*>(out + e) = empty ? 0u : pack2<BF16>(o[e] / l, o[e + 1] / l);
    if (p.lse != nullptr && lane == 0) p.lse[t * p.Hq + h] = empty ? -INFINITY : m + logf(l);
}

}  // namespace

cudaError_t launch_attn_kv4_simple(const AttnParams& p, bool bf16, int sms, cudaStream_t st) {
    (void)sms;
    const unsigned grid = (unsigned)((p.T * p.Hq + 3) / 4);
    if (p.c.D == 128)
        bf16 ? attn_simple_kernel<true, 128><<<grid, 128, 0, st>>>(p) : attn_simple_kernel<false, 128><<<grid, 128, 0, st>>>(p);
    else
        bf16 ? attn_simple_kernel<true, 64><<<grid, 128, 0, st>>>(p) : attn_simple_kernel<false, 64><<<grid, 128, 0, st>>>(p);
    return cudaPeekAtLastError();
}

}  // namespace wq
