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

// RN(x / 15) in fp32: the product with 1 / 15 and one correction by its exact residual
// (Markstein's method).
// (Results below the normal range, whose residual is not exact, are divided.)
__device__ __forceinline__ float fifteenth(float x) {
    if (x < 1e-30f) return __fdiv_rn(x, 15.0f);
    const float q = x * (1.0f / 15.0f);
    return fmaf(fmaf(-15.0f, q, x), 1.0f / 15.0f, q);
}
__device__ __forceinline__ float about_reciprocal(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// A group of D / 8 lanes takes one token and HP of its heads, keys and values: 2 HP rows,
// whose loads are all issued before the first is used.
struct GroupPlace {
    int64_t t, slot;        // slot < 0: none
    int h0, heads;          // first head; how many there are
    uint8_t* block;         // the slot's page block of head h0
    int place;
};
template <int D, int HP>
__device__ __forceinline__ GroupPlace group_place(const Kv4RowsParams& p, int lane) {
    const uint32_t g = blockIdx.x * (256 / (D / 8)) + threadIdx.x / (D / 8), t = fastdiv(g, p.div_groups);
    GroupPlace r;
    r.t = t;
    r.h0 = (int)(g - t * p.div_groups.d) * HP;
    r.heads = min(HP, p.c.heads - r.h0);
    r.slot = -1;
    r.block = nullptr;
    r.place = 0;
    if (r.t >= p.T) return r;
    r.slot = p.slots[t];
    if (r.slot >= p.c.num_pages << p.c.p_shift) {
        if (lane == 0) atomicOr(p.status, DEVICE_INDEX);
        r.slot = -1;
    }
    r.place = (int)(r.slot & (p.c.P - 1));
    r.block = p.c.pages + (r.slot >> p.c.p_shift) * p.c.page_bytes + (int64_t)r.h0 * p.c.block_bytes;
    return r;
}

// One lane takes 8 values of a row (16 bytes in, one word of codes out); the G / 8 lanes
// of a quantisation group find its least and greatest value with xor shuffles.  Two codes
// cost four packed operations: the difference, a multiply-add whose rounding gives the
// integer, that integer and its exact residual; only where the largest residual reaches
// half a step (ties, and the products that rounded the wrong way) is the exact search above
// run.  Bound by instructions (16384 tokens of 32 heads of 128, 344 MB: 118 us with an address
// and unpacked arithmetic for each row, now 87 us, the issue slots 78% full).  The least and the
// greatest value have shuffles of their own; one packed (least, -greatest) would halve them.
template <bool BF16, int D, int G, int HP>
__global__ void __launch_bounds__(256) kv4_write_kernel(const Kv4RowsParams p) {
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int lane = threadIdx.x % (D / 8);
    const GroupPlace at = group_place<D, HP>(p, lane);
    uint4 raw[HP][2];
    {
        const uint16_t* k = static_cast<const uint16_t*>(p.k) + at.t * p.k_stride + at.h0 * D + lane * 8;
        const uint16_t* v = static_cast<const uint16_t*>(p.v) + at.t * p.v_stride + at.h0 * D + lane * 8;
#pragma unroll
        for (int u = 0; u < HP; ++u) {
            raw[u][0] = raw[u][1] = make_uint4(0u, 0u, 0u, 0u);
            if (at.slot >= 0 && u < at.heads) {
                raw[u][0] = __ldcs(reinterpret_cast<const uint4*>(k + u * D));
                raw[u][1] = __ldcs(reinterpret_cast<const uint4*>(v + u * D));
            }
        }
    }
    const int pair_at = lane * 8 / G * 4;
    const bool first = lane * 8 % G == 0;
#pragma unroll
    for (int u = 0; u < HP; ++u)
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const uint32_t words[4] = {raw[u][which].x, raw[u][which].y, raw[u][which].z, raw[u][which].w};
            uint32_t mn = min2_nan<BF16>(min2_nan<BF16>(words[0], words[1]), min2_nan<BF16>(words[2], words[3]));
            uint32_t mx = max2_nan<BF16>(max2_nan<BF16>(words[0], words[1]), max2_nan<BF16>(words[2], words[3]));
#pragma unroll
            for (int off = G / 16; off > 0; off >>= 1) {
                mn = min2_nan<BF16>(mn, __shfl_xor_sync(0xffffffffu, mn, off));
                mx = max2_nan<BF16>(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            }
            mn = min2_nan<BF16>(mn, __byte_perm(mn, 0, 0x1032));
            mx = max2_nan<BF16>(mx, __byte_perm(mx, 0, 0x1032));
            if (at.slot < 0 || u >= at.heads) continue;
            const float lo = unpack2<BF16>(mn).x;
            const float range = unpack2<BF16>(mx).x - lo;
            uint32_t pair = (pack2<BF16>(fifteenth(range), 0.0f) & 0xFFFFu) | (mn << 16);
            float s = unpack2<BF16>(pair).x;
            // a rounded-up step must not carry the last code past the type's range
            const float last = unpack2<BF16>(pack2<BF16>(fmaf(15.0f, s, lo), 0.0f)).x;
            if (last == __int_as_float(0x7f800000) && s < last) s = unpack2<BF16>(--pair).x;
            uint32_t word = 0;
            if (!(s < __int_as_float(0x7f800000))) {          // an infinity, a NaN or an overflow: NaN throughout
                pair = BF16 ? 0x7FC07FC0u : 0x7E007E00u;
            } else if (s > 0.0f) {
                const float inv = about_reciprocal(s);
                const uint64_t lo2 = f2(-lo, -lo), inv2 = f2(inv, inv), s2 = f2(-s, -s);
                const uint64_t big = f2(12582912.0f, 12582912.0f), small = f2(-12582912.0f, -12582912.0f);   // 1.5 * 2^23
                float2 q[4];
                float worst = 0.f, worst1 = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = unpack2<BF16>(words[i]);
                    const uint64_t d = add_f2(f2(f.x, f.y), lo2);
                    const uint64_t n = add_f2(fma_f2(d, inv2, big), small);    // rounded to an integer
                    const float2 e = un2(fma_f2(n, s2, d));
                    q[i] = un2(n);
                    worst = fmaxf(worst, fabsf(e.x));
                    worst1 = fmaxf(worst1, fabsf(e.y));
                }
                // (steps below 1e-30 and codes past 15, which only subnormal steps have, take
                // the search too)
                if (fmaxf(worst, worst1) < 0.5f * s && s >= 1e-30f && range <= 15.4f * s) {
                    // four codes as one integer below 2^16, in the low bits of 2^23 + it
                    const float a = fmaf(fmaf(fmaf(q[1].y, 16.f, q[1].x), 16.f, q[0].y), 16.f, q[0].x + 8388608.f);
                    const float b = fmaf(fmaf(fmaf(q[3].y, 16.f, q[3].x), 16.f, q[2].y), 16.f, q[2].x + 8388608.f);
                    word = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x5410);
                } else {
                    const float up = s < 1e-30f ? 1.2089258196146292e24f : 1.0f;   // 2^80: keeps 1 / s and the residual in range
                    const float su = s * up, iu = __frcp_rn(su);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 f = unpack2<BF16>(words[i]);
                        word |= (uint32_t)nearest_code((f.x - lo) * up, su, iu) << (8 * i);
                        word |= (uint32_t)nearest_code((f.y - lo) * up, su, iu) << (8 * i + 4);
                    }
                }
            }
            uint8_t* block = at.block + u * p.c.block_bytes;
            *reinterpret_cast<uint32_t*>(block + kv4_codes_at(p.c, which, at.place) + lane * 4) = word;
            if (first) *reinterpret_cast<uint32_t*>(block + kv4_pairs_at(p.c, which, at.place) + pair_at) = pair;
        }
}

// The inverse: one lane turns a word of codes into 8 values (16 bytes out).  Bound by memory:
// 50001 tokens of 8 heads of 128, 269 MB, in 42 us (6.4 TB/s).
template <bool BF16, int D, int HP>
__global__ void __launch_bounds__(256) kv4_read_kernel(const Kv4RowsParams p) {
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int lane = threadIdx.x % (D / 8);
    const GroupPlace at = group_place<D, HP>(p, lane);
    if (at.t >= p.T) return;
    const int pair_at = ((lane * 8) >> p.c.g_shift) * 4;
    uint32_t w[HP][2], pair[HP][2];
#pragma unroll
    for (int u = 0; u < HP; ++u)
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            w[u][which] = pair[u][which] = 0u;
            if (at.slot >= 0 && u < at.heads) {
                const uint8_t* block = at.block + u * p.c.block_bytes;
                w[u][which] = *reinterpret_cast<const uint32_t*>(block + kv4_codes_at(p.c, which, at.place) + lane * 4);
                pair[u][which] = *reinterpret_cast<const uint32_t*>(block + kv4_pairs_at(p.c, which, at.place) + pair_at);
            }
        }
    uint16_t* k = static_cast<uint16_t*>(const_cast<void*>(p.k)) + at.t * p.k_stride + at.h0 * D + lane * 8;
    uint16_t* v = static_cast<uint16_t*>(const_cast<void*>(p.v)) + at.t * p.v_stride + at.h0 * D + lane * 8;
#pragma unroll
    for (int u = 0; u < HP; ++u)
#pragma unroll
        for (int which = 0; which < 2; ++which)
            if (u < at.heads)
                __stcs(reinterpret_cast<uint4*>((which ? v : k) + u * D),
                       word_values<BF16>(w[u][which], __byte_perm(pair[u][which], 0, 0x1010),
                                         __byte_perm(pair[u][which], 0, 0x3232)));
}

template <bool BF16, int D, int HP>
cudaError_t rows_launch(Kv4RowsParams p, bool write, cudaStream_t st) {
    const uint32_t groups = (uint32_t)((p.c.heads + HP - 1) / HP);
    const int64_t all = p.T * groups, per = 256 / (D / 8);
    p.div_groups = make_fastdiv(groups, (uint32_t)(all + 256));
    const unsigned grid = (unsigned)((all + per - 1) / per);
    if (!write) return launch_pdl(kv4_read_kernel<BF16, D, HP>, grid, 256, 0, st, p);
    if (p.c.G == 32) return launch_pdl(kv4_write_kernel<BF16, D, 32, HP>, grid, 256, 0, st, p);
    if (p.c.G == 64) return launch_pdl(kv4_write_kernel<BF16, D, 64, HP>, grid, 256, 0, st, p);
    return launch_pdl(kv4_write_kernel<BF16, D, D == 128 ? 128 : 64, HP>, grid, 256, 0, st, p);
}

template <int HP>
cudaError_t rows_launch_hp(const Kv4RowsParams& p, bool bf16, bool write, cudaStream_t st) {
    if (p.c.D == 128) return bf16 ? rows_launch<true, 128, HP>(p, write, st) : rows_launch<false, 128, HP>(p, write, st);
    return bf16 ? rows_launch<true, 64, HP>(p, write, st) : rows_launch<false, 64, HP>(p, write, st);
}

// Two heads for each group of lanes where that still leaves two blocks for each SM.
cudaError_t rows_any(const Kv4RowsParams& p, bool bf16, bool write, int sms, cudaStream_t st) {
    return p.T * ((p.c.heads + 1) / 2) * (p.c.D / 8) >= (int64_t)sms * 2 * 256 ? rows_launch_hp<2>(p, bf16, write, st)
                                                                               : rows_launch_hp<1>(p, bf16, write, st);
}

}  // namespace

cudaError_t launch_kv4_write(const Kv4RowsParams& p, bool bf16, int sms, cudaStream_t st) {
    return rows_any(p, bf16, true, sms, st);
}

cudaError_t launch_kv4_read(const Kv4RowsParams& p, bool bf16, int sms, cudaStream_t st) {
    return rows_any(p, bf16, false, sms, st);
}

}  // namespace wq
