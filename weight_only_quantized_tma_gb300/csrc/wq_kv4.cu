// wq_kv4.cu -- quantising keys and values into the paged 4-bit cache, and reading the
// cache back (include/wq.h: wq_kv4_write, wq_kv4_read).
#include "wq_kv4.cuh"

namespace wq {
namespace {

// The nearest integer to d / s (half to even) for d >= 0, s > 0: q0 = rint(d * (1 / s))
// is within one of it, the residual d - q0 s is exact in fp32 (q0 s has 15 significant
// bits, the difference is below s on a grid of 2^-21 s or coarser), and comparing it with
// s / 2 decides exactly.
__device__ __forceinline__ int nearest_code(float d, float s, float inv) {
    float q = rintf(d * inv);
    const float e = fmaf(-q, s, d);
    const float ae = fabsf(e), h = 0.5f * s;
    if (ae > h)
        q += copysignf(1.0f, e);
    else if (ae == h) {
        const float q1 = q + copysignf(1.0f, e);
        if (((int)q1 & 1) == 0) q = q1;
    }
    const int i = (int)q;
    return i < 0 ? 0 : (i > 15 ? 15 : i);
}

// One lane takes 8 values of a row (16 bytes in, one word of codes out); the G / 8 lanes
// of a group find its least and greatest value with xor shuffles.
template <bool BF16, int D>
__global__ void __launch_bounds__(256) kv4_write_kernel(const Kv4RowsParams p) {
    constexpr int LPR = D / 8;
    const int lane_in_row = threadIdx.x % LPR;
    const int64_t rows = p.T * p.c.heads * 2;
    const int64_t row = (int64_t)blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
    const int which = (int)(row & 1);
    const int64_t th = row >> 1;
    const int64_t t = th / p.c.heads;
    const int h = (int)(th - t * p.c.heads);
    int64_t slot = -1;
    if (row < rows) {
        slot = p.slots[t];
        if (slot >= p.c.num_pages << p.c.p_shift) {
            if (lane_in_row == 0) atomicOr(p.status, DEVICE_INDEX);
            slot = -1;
        }
    }
    uint4 raw = make_uint4(0u, 0u, 0u, 0u);
    if (slot >= 0) {
        const uint16_t* src = static_cast<const uint16_t*>(which ? p.v : p.k) +
                              t * (which ? p.v_stride : p.k_stride) + (int64_t)h * D + lane_in_row * 8;
        raw = __ldcs(reinterpret_cast<const uint4*>(src));
    }
    uint32_t mn = min2_nan<BF16>(min2_nan<BF16>(raw.x, raw.y), min2_nan<BF16>(raw.z, raw.w));
    uint32_t mx = max2_nan<BF16>(max2_nan<BF16>(raw.x, raw.y), max2_nan<BF16>(raw.z, raw.w));
    for (int off = p.c.G / 16; off > 0; off >>= 1) {
        mn = min2_nan<BF16>(mn, __shfl_xor_sync(0xffffffffu, mn, off));
        mx = max2_nan<BF16>(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    }
    mn = min2_nan<BF16>(mn, __byte_perm(mn, 0, 0x1032));
    mx = max2_nan<BF16>(mx, __byte_perm(mx, 0, 0x1032));
    if (slot < 0) return;
    float lo = unpack2<BF16>(mn).x;
    const float range = unpack2<BF16>(mx).x - lo;
    uint32_t pair = (pack2<BF16>(__fdiv_rn(range, 15.0f), 0.0f) & 0xFFFFu) | (mn << 16);
    float s = unpack2<BF16>(pair).x;
    // a rounded-up step must not carry the last code past the type's range
    const float last = unpack2<BF16>(pack2<BF16>(fmaf(15.0f, s, lo), 0.0f)).x;
    if (last == __int_as_float(0x7f800000) && s < last) s = unpack2<BF16>(--pair).x;
    uint32_t word = 0;
    if (!(s < __int_as_float(0x7f800000))) {          // an infinity, a NaN or an overflow: NaN throughout
        pair = BF16 ? 0x7FC07FC0u : 0x7E007E00u;
    } else if (s > 0.0f) {
        float up = 1.0f;
        if (s < 1e-30f) up = 1.2089258196146292e24f;  // 2^80: keeps 1 / s and the residual in range
        const float su = s * up, inv = __frcp_rn(su);
        const uint32_t words[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2<BF16>(words[i]);
            word |= (uint32_t)nearest_code((f.x - lo) * up, su, inv) << (8 * i);
            word |= (uint32_t)nearest_code((f.y - lo) * up, su, inv) << (8 * i + 4);
        }
    }
    const int64_t page = slot >> p.c.p_shift;
    const int place = (int)(slot & (p.c.P - 1));
    uint8_t* block = p.c.pages + page * p.c.page_bytes + (int64_t)h * p.c.block_bytes;
    *reinterpret_cast<uint32_t*>(block + kv4_codes_at(p.c, which, place) + lane_in_row * 4) = word;
    if (((lane_in_row * 8) & (p.c.G - 1)) == 0)
        *reinterpret_cast<uint32_t*>(block + kv4_pairs_at(p.c, which, place) + ((lane_in_row * 8) >> p.c.g_shift) * 4) =
            pair;
}

// The inverse: one lane turns a word of codes into 8 values (16 bytes out).
template <bool BF16, int D>
__global__ void __launch_bounds__(256) kv4_read_kernel(const Kv4RowsParams p) {
    constexpr int LPR = D / 8;
    const int lane_in_row = threadIdx.x % LPR;
    const int64_t rows = p.T * p.c.heads * 2;
    const int64_t row = (int64_t)blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
    if (row >= rows) return;
    const int which = (int)(row & 1);
    const int64_t th = row >> 1;
    const int64_t t = th / p.c.heads;
    const int h = (int)(th - t * p.c.heads);
    const int64_t slot = p.slots[t];
    uint4 o = make_uint4(0u, 0u, 0u, 0u);
    if (slot >= p.c.num_pages << p.c.p_shift) {
        if (lane_in_row == 0) atomicOr(p.status, DEVICE_INDEX);
    } else if (slot >= 0) {
        const int64_t page = slot >> p.c.p_shift;
        const int place = (int)(slot & (p.c.P - 1));
        const uint8_t* block = p.c.pages + page * p.c.page_bytes + (int64_t)h * p.c.block_bytes;
        const uint32_t w = *reinterpret_cast<const uint32_t*>(block + kv4_codes_at(p.c, which, place) + lane_in_row * 4);
        const uint32_t pair = *reinterpret_cast<const uint32_t*>(block + kv4_pairs_at(p.c, which, place) +
                                                                 ((lane_in_row * 8) >> p.c.g_shift) * 4);
        o = word_values<BF16>(w, __byte_perm(pair, 0, 0x1010), __byte_perm(pair, 0, 0x3232));
    }
    uint16_t* dst = static_cast<uint16_t*>(const_cast<void*>(which ? p.v : p.k)) +
                    t * (which ? p.v_stride : p.k_stride) + (int64_t)h * D + lane_in_row * 8;
    __stcs(reinterpret_cast<uint4*>(dst), o);
}

}  // namespace

cudaError_t launch_kv4_write(const Kv4RowsParams& p, bool bf16, int sms, cudaStream_t st) {
    (void)sms;
    const int64_t per = 256 / (p.c.D / 8), rows = p.T * p.c.heads * 2;
    const unsigned grid = (unsigned)((rows + per - 1) / per);
    if (p.c.D == 128)
        bf16 ? kv4_write_kernel<true, 128><<<grid, 256, 0, st>>>(p) : kv4_write_kernel<false, 128><<<grid, 256, 0, st>>>(p);
    else
        bf16 ? kv4_write_kernel<true, 64><<<grid, 256, 0, st>>>(p) : kv4_write_kernel<false, 64><<<grid, 256, 0, st>>>(p);
    return cudaPeekAtLastError();
}

cudaError_t launch_kv4_read(const Kv4RowsParams& p, bool bf16, int sms, cudaStream_t st) {
    (void)sms;
    const int64_t per = 256 / (p.c.D / 8), rows = p.T * p.c.heads * 2;
    const unsigned grid = (unsigned)((rows + per - 1) / per);
    if (p.c.D == 128)
        bf16 ? kv4_read_kernel<true, 128><<<grid, 256, 0, st>>>(p) : kv4_read_kernel<false, 128><<<grid, 256, 0, st>>>(p);
    else
        bf16 ? kv4_read_kernel<true, 64><<<grid, 256, 0, st>>>(p) : kv4_read_kernel<false, 64><<<grid, 256, 0, st>>>(p);
    return cudaPeekAtLastError();
}

}  // namespace wq
