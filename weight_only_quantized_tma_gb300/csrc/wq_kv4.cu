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

// Where a row (one token's keys or values of one head) comes from and goes to.
struct RowPlace {
    int which, h;
    int64_t t, slot;    // slot < 0: none
};
__device__ __forceinline__ RowPlace row_place(const Kv4RowsParams& p, uint32_t row, bool report) {
    RowPlace r;
    r.which = (int)(row & 1u);
    const uint32_t th = row >> 1, t = fastdiv(th, p.div_heads);
    r.t = t;
    r.h = (int)(th - t * p.div_heads.d);
    r.slot = -1;
    if (r.t < p.T) {
        r.slot = p.slots[t];
        if (r.slot >= p.c.num_pages << p.c.p_shift) {
            if (report) atomicOr(p.status, DEVICE_INDEX);
            r.slot = -1;
        }
    }
    return r;
}
__device__ __forceinline__ uint8_t* row_block(const Kv4RowsParams& p, const RowPlace& r, int& place) {
    place = (int)(r.slot & (p.c.P - 1));
    return p.c.pages + (r.slot >> p.c.p_shift) * p.c.page_bytes + (int64_t)r.h * p.c.block_bytes;
}

// One lane takes 8 values of a row (16 bytes in, one word of codes out); the G / 8 lanes
// of a group find its least and greatest value with xor shuffles.  A group of lanes takes
// U rows whose loads are all issued first.  A code costs five operations: the difference,
// a multiply-add whose rounding gives the integer, that integer, its exact residual and
// the largest residual so far; only where that reaches half a step (ties, and the products
// that rounded the wrong way) is the exact search above run.
template <bool BF16, int D, int U>
__global__ void __launch_bounds__(256) kv4_write_kernel(const Kv4RowsParams p) {
    constexpr int LPR = D / 8;
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int lane_in_row = threadIdx.x % LPR;
    const uint32_t row0 = (blockIdx.x * (256 / LPR) + threadIdx.x / LPR) * U;
    RowPlace at[U];
    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        at[u] = row_place(p, row0 + u, lane_in_row == 0);
        raw[u] = make_uint4(0u, 0u, 0u, 0u);
        if (at[u].slot >= 0) {
            const uint16_t* src = static_cast<const uint16_t*>(at[u].which ? p.v : p.k) +
                                  at[u].t * (at[u].which ? p.v_stride : p.k_stride) + (int64_t)at[u].h * D + lane_in_row * 8;
            raw[u] = __ldcs(reinterpret_cast<const uint4*>(src));
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        uint32_t mn = min2_nan<BF16>(min2_nan<BF16>(raw[u].x, raw[u].y), min2_nan<BF16>(raw[u].z, raw[u].w));
        uint32_t mx = max2_nan<BF16>(max2_nan<BF16>(raw[u].x, raw[u].y), max2_nan<BF16>(raw[u].z, raw[u].w));
        for (int off = p.c.G / 16; off > 0; off >>= 1) {
            mn = min2_nan<BF16>(mn, __shfl_xor_sync(0xffffffffu, mn, off));
            mx = max2_nan<BF16>(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        }
        mn = min2_nan<BF16>(mn, __byte_perm(mn, 0, 0x1032));
        mx = max2_nan<BF16>(mx, __byte_perm(mx, 0, 0x1032));
        if (at[u].slot < 0) continue;
        const float lo = unpack2<BF16>(mn).x;
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
            const uint32_t words[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
            const float inv = __frcp_rn(s), half = 0.5f * s;
            float q[8], worst = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = unpack2<BF16>(words[i]);
                const float d0 = f.x - lo, d1 = f.y - lo;
                q[2 * i] = fmaf(d0, inv, 12582912.0f) - 12582912.0f;       // 1.5 * 2^23: rounds to an integer
                q[2 * i + 1] = fmaf(d1, inv, 12582912.0f) - 12582912.0f;
                worst = fmaxf(worst, fmaxf(fabsf(fmaf(-q[2 * i], s, d0)), fabsf(fmaf(-q[2 * i + 1], s, d1))));
            }
            // (a NaN fails the test; steps below 1e-30 and codes past 15, which only
            // subnormal steps have, take the search too)
            if (worst < half && s >= 1e-30f && range <= 15.4f * s) {
                const float a = fmaf(fmaf(fmaf(q[3], 16.f, q[2]), 16.f, q[1]), 16.f, q[0]);
                const float b = fmaf(fmaf(fmaf(q[7], 16.f, q[6]), 16.f, q[5]), 16.f, q[4]);
                word = (uint32_t)(int)a | ((uint32_t)(int)b << 16);
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
        int place;
        uint8_t* block = row_block(p, at[u], place);
        *reinterpret_cast<uint32_t*>(block + kv4_codes_at(p.c, at[u].which, place) + lane_in_row * 4) = word;
        if (((lane_in_row * 8) & (p.c.G - 1)) == 0)
            *reinterpret_cast<uint32_t*>(block + kv4_pairs_at(p.c, at[u].which, place) +
                                         ((lane_in_row * 8) >> p.c.g_shift) * 4) = pair;
    }
}

// The inverse: one lane turns a word of codes into 8 values (16 bytes out).
template <bool BF16, int D, int U>
__global__ void __launch_bounds__(256) kv4_read_kernel(const Kv4RowsParams p) {
    constexpr int LPR = D / 8;
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int lane_in_row = threadIdx.x % LPR;
    const uint32_t row0 = (blockIdx.x * (256 / LPR) + threadIdx.x / LPR) * U;
    RowPlace at[U];
    uint32_t w[U], pair[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        at[u] = row_place(p, row0 + u, lane_in_row == 0);
        w[u] = pair[u] = 0u;
        if (at[u].slot >= 0) {
            int place;
            const uint8_t* block = row_block(p, at[u], place);
            w[u] = *reinterpret_cast<const uint32_t*>(block + kv4_codes_at(p.c, at[u].which, place) + lane_in_row * 4);
            pair[u] = *reinterpret_cast<const uint32_t*>(block + kv4_pairs_at(p.c, at[u].which, place) +
                                                         ((lane_in_row * 8) >> p.c.g_shift) * 4);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (at[u].t >= p.T) continue;
        uint16_t* dst = static_cast<uint16_t*>(const_cast<void*>(at[u].which ? p.v : p.k)) +
                        at[u].t * (at[u].which ? p.v_stride : p.k_stride) + (int64_t)at[u].h * D + lane_in_row * 8;
        __stcs(reinterpret_cast<uint4*>(dst),
               word_values<BF16>(w[u], __byte_perm(pair[u], 0, 0x1010), __byte_perm(pair[u], 0, 0x3232)));
    }
}

template <bool BF16, int D, int U>
cudaError_t rows_launch(const Kv4RowsParams& p, bool write, cudaStream_t st) {
    const int64_t per = 256 / (D / 8) * U, rows = p.T * p.c.heads * 2;
    const unsigned grid = (unsigned)((rows + per - 1) / per);
    return write ? launch_pdl(kv4_write_kernel<BF16, D, U>, grid, 256, 0, st, p)
                 : launch_pdl(kv4_read_kernel<BF16, D, U>, grid, 256, 0, st, p);
}

template <int U>
cudaError_t rows_launch_u(const Kv4RowsParams& p, bool bf16, bool write, cudaStream_t st) {
    if (p.c.D == 128) return bf16 ? rows_launch<true, 128, U>(p, write, st) : rows_launch<false, 128, U>(p, write, st);
    return bf16 ? rows_launch<true, 64, U>(p, write, st) : rows_launch<false, 64, U>(p, write, st);
}

// Four rows for each group of lanes where that still leaves two blocks for each SM.
cudaError_t rows_any(const Kv4RowsParams& p, bool bf16, bool write, int sms, cudaStream_t st) {
    const int64_t rows = p.T * p.c.heads * 2;
    return rows * (p.c.D / 8) >= (int64_t)sms * 2 * 256 * 4 ? rows_launch_u<4>(p, bf16, write, st)
                                                            : rows_launch_u<1>(p, bf16, write, st);
}

}  // namespace

cudaError_t launch_kv4_write(const Kv4RowsParams& p, bool bf16, int sms, cudaStream_t st) {
    return rows_any(p, bf16, true, sms, st);
}

cudaError_t launch_kv4_read(const Kv4RowsParams& p, bool bf16, int sms, cudaStream_t st) {
    return rows_any(p, bf16, false, sms, st);
}

}  // namespace wq
