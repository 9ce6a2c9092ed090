// wq_norm.cu -- root-mean-square norm of rows with the residual's addition, its output in 16 bits or in
// 8 bits with scales, and the quantiser of 16-bit rows (include/wq.h: wq_add_rms_norm,
// wq_add_rms_norm_fp8, wq_quantize_fp8).
//
//   s = x + residual,   y = s * rsqrt(mean(s^2) + eps) * w
//
// in fp32, from the sum before it is rounded: one rounding of y and one of s.
#include "wq_fp8.cuh"

namespace wq {
namespace {

// Eight 16-bit values as four pairs of fp32 (one instruction then works on two), and back.
template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& r, uint64_t (&x)[4]) {
    const float2 a = unpack2<BF16>(r.x), b = unpack2<BF16>(r.y), c = unpack2<BF16>(r.z), d = unpack2<BF16>(r.w);
    x[0] = f2(a.x, a.y), x[1] = f2(b.x, b.y), x[2] = f2(c.x, c.y), x[3] = f2(d.x, d.y);
}
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const uint64_t (&x)[4]) {
    const float2 a = un2(x[0]), b = un2(x[1]), c = un2(x[2]), d = un2(x[3]);
    return make_uint4(pack2<BF16>(a.x, a.y), pack2<BF16>(b.x, b.y), pack2<BF16>(c.x, c.y), pack2<BF16>(d.x, d.y));
}

// 16 bytes that are used once: they take no place in L1 from the weight, which every row of an SM reads.
__device__ __forceinline__ uint4 load_once(const uint16_t* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

// The largest magnitude of 8 values of each of 16 neighbouring lanes (a block of 128).
__device__ __forceinline__ float block_most(const uint64_t (&y)[4]) {
    const float2 a = un2(y[0]), b = un2(y[1]), c = un2(y[2]), d = un2(y[3]);
    float m = max_nan(fabsf(a.x), fabsf(a.y), fabsf(b.x));
    m = max_nan(m, fabsf(b.y), fabsf(c.x));
    m = max_nan(m, fabsf(c.y), fabsf(d.x));
    m = max_nan(m, fabsf(d.y));
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
    return m;
}
__device__ __forceinline__ uint2 codes8(const uint64_t (&y)[4], const BlockScale& q) {
    return make_uint2(q.codes(y[0], y[1]), q.codes(y[2], y[3]));
}

// A row's total, the same in each of its threads; `part` is the block's, one for each turn.
__device__ __forceinline__ float row_total(float v, float* part) {
    const int warps = (int)(blockDim.x >> 5);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    float all = 0.f;
#pragma unroll
    for (int w = 0; w < 16; w += 4) {      // (four in one load: 8192 x 4096 to 8 bits 44.7 -> 43.8 us)
        if (w >= warps) break;
        const float4 q = *reinterpret_cast<const float4*>(part + w);
        all += q.x, all += w + 1 < warps ? q.y : 0.f, all += w + 2 < warps ? q.z : 0.f, all += w + 3 < warps ? q.w : 0.f;
    }
    return all;
}

// Eight values of row t from `at` on, times inv and the weight, to the output.
template <bool BF16, bool QUANT>
__device__ __forceinline__ void finish_values(const NormParams& p, int64_t t, int at, uint64_t (&v)[4], float inv) {
    const bool in = t < p.T && at < p.H;
    uint64_t w[4];
    unpack8<BF16>(at < p.H ? __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.weight) + at)) : make_uint4(0, 0, 0, 0), w);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = mul_f2(mul_f2(v[i], f2(inv, inv)), w[i]);
    if (QUANT) {
        // lanes past the row hold zeros (0 * inv * 0, where inv may be infinite: not those)
        if (at >= p.H) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = 0;
        }
        const BlockScale q(block_most(v));
        if (in) {
            *reinterpret_cast<uint2*>(p.codes + t * p.H + at) = codes8(v, q);
            if ((threadIdx.x & 15) == 0) p.scales[(int64_t)(at >> 7) * p.T + t] = q.scale;
        }
    } else if (in) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + t * p.out_stride + at) = pack8<BF16>(v);
    }
}

// Where a row's sum of squares, or the mean with eps, has left fp32's range (a row of numbers around 2^64 and above, or
// all of them tiny without an eps that outweighs them) the squares are taken of f s; as the root may be below 2^-126 or
// past 2^128 itself, the values are multiplied with g first.
struct Range {
    bool large;
    float f, g;
    __device__ __forceinline__ explicit Range(bool l) : large(l), f(l ? 0x1p-72f : 0x1p80f), g(l ? 0x1p-32f : 0x1p32f) {}
    __device__ __forceinline__ float square(uint64_t (&v)[4]) const {
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 u = un2(mul_f2(v[i], f2(f, f)));
            sq += u.x * u.x + u.y * u.y;
            v[i] = mul_f2(v[i], f2(g, g));
        }
        return sq;
    }
    // of g s, from the total of squares
    __device__ __forceinline__ float inverse(float sq, float inv_h, float eps) const {
        return rsqrtf(sq * inv_h + eps * f * f) * (large ? 0x1p-40f : 0x1p48f);
    }
};

// Such a row without a residual, from memory once more: no register of the usual way is held for it.
template <bool BF16, int C, bool QUANT>
__device__ __noinline__ void norm_again(const NormParams& p, int64_t t, bool large, float* part) {
    const Range range(large);
    const int first = 8 * (int)threadIdx.x, step = 8 * (int)blockDim.x;
    auto load = [&](int at, uint64_t (&v)[4]) {
        const uint16_t* x = static_cast<const uint16_t*>(p.x) + t * p.x_stride + at;
        unpack8<BF16>(t < p.T && at < p.H ? *reinterpret_cast<const uint4*>(x) : make_uint4(0, 0, 0, 0), v);
        return range.square(v);
    };
    float sq = 0.f;
#pragma unroll 1
    for (int at = first; at < C * step; at += step) {
        uint64_t v[4];
        sq += load(at, v);
    }
    const float inv = range.inverse(row_total(sq, part), p.inv_h, p.eps);
#pragma unroll 1
    for (int at = first; at < C * step; at += step) {
        uint64_t v[4];
        load(at, v);
        finish_values<BF16, QUANT>(p, t, at, v, inv);
    }
}

// One row for each group of `blockDim.x` threads (blockDim.y rows in a block; more than one only where a
// row is one warp).  Thread i holds values 8 (i + c blockDim.x) .. + 7 of chunk c < C, so 16 neighbouring
// lanes hold one block of 128.  Bound by memory from some 100 rows on, as far as rows are on their way: hence the
// bounds on registers, which keep 1000 to 2000 threads on an SM (512 for rows past 16384 values with a residual; 4000 x
// 11008 to 8 bits 41 -> 34 us), and the weight read late.  8192 x 4096 with a residual: 42.1 us (6.4 TB/s), to 8 bits
// 43.6 (5.4 TB/s; issue slots 72 % full).  The mean is the sum times 1 / H, a rounding more than a division.  Tried:
// blocks that stay, rows arriving by bulk copies (43 to 46 us), the next row loaded into registers early (43 to 44).
template <bool BF16, int C, bool ADD, bool QUANT>
__global__ void __launch_bounds__(512, C == 8 ? (ADD ? 1 : 2) : C == 4 ? (ADD ? 2 : 3) : C == 2 ? (ADD ? 3 : 4) : 4) norm_kernel(const __grid_constant__ NormParams p) {
    __shared__ __align__(16) float part[2][16];
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool row = t < p.T;
    const uint16_t* x = static_cast<const uint16_t*>(p.x) + t * p.x_stride;
    const uint16_t* r = static_cast<const uint16_t*>(p.residual) + t * p.r_stride;
    // With a residual the fp32 sums are kept for the output, without one the 16-bit row is (half the registers, so
    // more rows are on their way in an SM).
    uint64_t s[C][4];
    uint4 xr[C], rr[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int at = 8 * (int)(threadIdx.x + c * blockDim.x);
        const bool in = row && at < p.H;
        xr[c] = in ? load_once(x + at) : make_uint4(0, 0, 0, 0);
        if (ADD) rr[c] = in ? load_once(r + at) : make_uint4(0, 0, 0, 0);
    }
    uint64_t squares = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int at = 8 * (int)(threadIdx.x + c * blockDim.x);
        unpack8<BF16>(xr[c], s[c]);
        if (ADD) {
            uint64_t b[4];
            unpack8<BF16>(rr[c], b);
#pragma unroll
            for (int i = 0; i < 4; ++i) s[c][i] = add_f2(s[c][i], b[i]);
            if (row && at < p.H)
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.sum) + t * p.sum_stride + at) = pack8<BF16>(s[c]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) squares = fma_f2(s[c][i], s[c][i], squares);
    }
    const float sum = row_total(un2(squares).x + un2(squares).y, part[0]), mean = sum * p.inv_h + p.eps;
    float inv = rsqrtf(mean);
    const bool large = !(mean <= 3.402823466e38f);
    if (large || (sum < 0x1p-90f && p.eps < 0x1p-80f)) {      // (the row's threads agree on it)
        if (!ADD) return norm_again<BF16, C, QUANT>(p, t, large, part[1]);
        const Range range(large);
        float sq = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c) sq += range.square(s[c]);
        inv = range.inverse(row_total(sq, part[1]), p.inv_h, p.eps);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (!ADD) unpack8<BF16>(xr[c], s[c]);
        finish_values<BF16, QUANT>(p, t, 8 * (int)(threadIdx.x + c * blockDim.x), s[c], inv);
    }
}

// Threads of a row, 8 C values each.
int threads_of(int H, int C) { return (H + 256 * C - 1) / (256 * C) * 32; }

template <bool BF16, int C, bool ADD, bool QUANT>
cudaError_t launch_row_each(const NormParams& p, cudaStream_t st) {
    const int threads = threads_of(p.H, C), rows = threads == 32 ? 4 : 1;
    return launch_pdl(norm_kernel<BF16, C, ADD, QUANT>, (unsigned)((p.T + rows - 1) / rows), dim3(threads, rows), 0, st, p);
}

template <bool BF16, bool ADD, bool QUANT>
cudaError_t launch_norm(const NormParams& p, cudaStream_t st) {
    if (p.H <= 4096) return launch_row_each<BF16, 1, ADD, QUANT>(p, st);
    if (p.H <= 8192) return launch_row_each<BF16, 2, ADD, QUANT>(p, st);
    if (p.H <= 16384) return launch_row_each<BF16, 4, ADD, QUANT>(p, st);
    return launch_row_each<BF16, 8, ADD, QUANT>(p, st);   // up to 512 threads: H <= 32768
}

template <bool BF16>
cudaError_t launch_norm_t(const NormParams& p, cudaStream_t st) {
    if (p.codes != nullptr)
        return p.residual != nullptr ? launch_norm<BF16, true, true>(p, st) : launch_norm<BF16, false, true>(p, st);
    return p.residual != nullptr ? launch_norm<BF16, true, false>(p, st) : launch_norm<BF16, false, false>(p, st);
}

// 16 tokens for each block of 256 threads: 16 lanes take one token's block of 128, U of them in turn whose
// loads are all issued first.  The scales of 16 tokens are neighbours.
template <bool BF16, int U>
__global__ void __launch_bounds__(256, 6) quantize_kernel(const NormParams p) {
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int lane = threadIdx.x & 15;
    const uint32_t tg = fastdiv(blockIdx.x, p.div_blocks);
    const int kb0 = (int)(blockIdx.x - tg * p.div_blocks.d) * U;
    const int64_t t = (int64_t)tg * 16 + (threadIdx.x >> 4);
    const bool row = t < p.T;
    const uint16_t* x = static_cast<const uint16_t*>(p.x) + t * p.x_stride;
    uint4 xr[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int at = (kb0 + u) * 128 + 8 * lane;
        xr[u] = row && at < p.H ? *reinterpret_cast<const uint4*>(x + at) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int at = (kb0 + u) * 128 + 8 * lane;
        uint64_t y[4];
        unpack8<BF16>(xr[u], y);
        const BlockScale q(block_most(y));
        if (row && at < p.H) {
            *reinterpret_cast<uint2*>(p.codes + t * p.H + at) = codes8(y, q);
            if (lane == 0) p.scales[(int64_t)(kb0 + u) * p.T + t] = q.scale;
        }
    }
}

template <bool BF16, int U>
cudaError_t launch_quantize_u(NormParams p, cudaStream_t st) {
    const int64_t across = ((p.H + 127) / 128 + U - 1) / U, all = (p.T + 15) / 16 * across;
    if (all >= (1LL << 31)) return cudaErrorInvalidValue;
    p.div_blocks = make_fastdiv((uint32_t)across, (uint32_t)all);
    return launch_pdl(quantize_kernel<BF16, U>, (unsigned)all, 256, 0, st, p);
}

}  // namespace

cudaError_t launch_add_rms_norm(const NormParams& p, bool bf16, cudaStream_t st) {
    return bf16 ? launch_norm_t<true>(p, st) : launch_norm_t<false>(p, st);
}

cudaError_t launch_quantize_fp8(const NormParams& p, bool bf16, int sms, cudaStream_t st) {
    const bool many = (p.T + 15) / 16 * ((p.H + 127) / 128) >= 16LL * sms;
    if (many) return bf16 ? launch_quantize_u<true, 4>(p, st) : launch_quantize_u<false, 4>(p, st);
    return bf16 ? launch_quantize_u<true, 1>(p, st) : launch_quantize_u<false, 1>(p, st);
}

}  // namespace wq
