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

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& r, float (&x)[8]) {
    const float2 a = unpack2<BF16>(r.x), b = unpack2<BF16>(r.y), c = unpack2<BF16>(r.z), d = unpack2<BF16>(r.w);
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y, x[4] = c.x, x[5] = c.y, x[6] = d.x, x[7] = d.y;
}
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3]), pack2<BF16>(x[4], x[5]), pack2<BF16>(x[6], x[7]));
}

// The largest magnitude of 8 values of each of 16 neighbouring lanes (a block of 128).
__device__ __forceinline__ float block_most(const float (&y)[8]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_nan(m, fabsf(y[i]));
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
    return m;
}
__device__ __forceinline__ uint2 codes8(const float (&y)[8], float inv) {
    if (inv == 0.f) return make_uint2(0u, 0u);   // (a NaN times 0 would be one)
    return make_uint2(to_e4m3x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                      to_e4m3x4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
}

// rsqrt(mean + eps) from a sum of squares; `again(f)` gives the sum of (f s)^2 where the plain one has
// left fp32's range (a row of numbers around 2^64 and above, or all of them tiny without an eps that
// outweighs them).
template <typename Again>
__device__ __forceinline__ float inverse_rms(float sum, float inv_h, float eps, Again again) {
    if (!(sum <= 3.402823466e38f)) return rsqrtf(again(0x1p-72f) * inv_h + eps * 0x1p-144f) * 0x1p-72f;
    if (sum < 0x1p-90f && eps < 0x1p-80f) return rsqrtf(again(0x1p80f) * inv_h + eps * 0x1p80f * 0x1p80f) * 0x1p80f;
    return rsqrtf(sum * inv_h + eps);
}

// One row for each group of `blockDim.x` threads (blockDim.y rows in a block; more than one only where a
// row is one warp).  Thread i holds values 8 (i + c blockDim.x) .. + 7 of chunk c < C, so 16 neighbouring
// lanes hold one block of 128.
template <bool BF16, int C, bool ADD, bool QUANT>
__global__ void __launch_bounds__(1024) norm_kernel(const NormParams p) {
    __shared__ float part[2][32];
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int lane = threadIdx.x & 31, warps = (int)(blockDim.x >> 5);
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool row = t < p.T;
    const uint16_t* x = static_cast<const uint16_t*>(p.x) + t * p.x_stride;
    const uint16_t* r = static_cast<const uint16_t*>(p.residual) + t * p.r_stride;
    float s[C][8];
    uint4 xr[C], rr[C], wr[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int at = 8 * (int)(threadIdx.x + c * blockDim.x);
        const bool in = row && at < p.H;
        xr[c] = in ? *reinterpret_cast<const uint4*>(x + at) : make_uint4(0, 0, 0, 0);
        if (ADD) rr[c] = in ? *reinterpret_cast<const uint4*>(r + at) : make_uint4(0, 0, 0, 0);
        wr[c] = at < p.H ? __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.weight) + at)) : make_uint4(0, 0, 0, 0);
    }
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        unpack8<BF16>(xr[c], s[c]);
        if (ADD) {
            float b[8];
            unpack8<BF16>(rr[c], b);
#pragma unroll
            for (int i = 0; i < 8; ++i) s[c][i] += b[i];
            const int at = 8 * (int)(threadIdx.x + c * blockDim.x);
            if (row && at < p.H)
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.sum) + t * p.sum_stride + at) = pack8<BF16>(s[c]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += s[c][i] * s[c][i];
    }
    // the row's total, the same in each of its threads
    auto total = [&](float v, int turn) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
        if (warps == 1) return v;
        if (lane == 0) part[turn][threadIdx.x >> 5] = v;
        __syncthreads();
        float all = 0.f;
        for (int w = 0; w < warps; ++w) all += part[turn][w];
        return all;
    };
    const float inv = inverse_rms(total(sum, 0), p.inv_h, p.eps, [&](float f) {
        float v = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) v += (f * s[c][i]) * (f * s[c][i]);
        return total(v, 1);   // (the row's threads agree on whether they come here)
    });
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int at = 8 * (int)(threadIdx.x + c * blockDim.x);
        float w[8];
        unpack8<BF16>(wr[c], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[c][i] = s[c][i] * inv * w[i];
        if (QUANT) {
            // lanes past the row hold zeros (0 * inv * 0, where inv may be infinite: not those)
            if (at >= p.H) {
#pragma unroll
                for (int i = 0; i < 8; ++i) s[c][i] = 0.f;
            }
            const BlockScale q(block_most(s[c]));
            if (row && at < p.H) {
                *reinterpret_cast<uint2*>(p.codes + t * p.H + at) = codes8(s[c], q.inv);
                if ((lane & 15) == 0) p.scales[(int64_t)(at >> 7) * p.T + t] = q.scale;
            }
        } else if (row && at < p.H) {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + t * p.out_stride + at) = pack8<BF16>(s[c]);
        }
    }
}

template <bool BF16, int C>
cudaError_t launch_c(const NormParams& p, int threads, cudaStream_t st) {
    const int rows = threads == 32 ? 4 : 1;
    const unsigned grid = (unsigned)((p.T + rows - 1) / rows);
    const dim3 block(threads, rows);
    if (p.codes != nullptr)
        return p.residual != nullptr ? launch_pdl(norm_kernel<BF16, C, true, true>, grid, block, 0, st, p)
                                     : launch_pdl(norm_kernel<BF16, C, false, true>, grid, block, 0, st, p);
    return p.residual != nullptr ? launch_pdl(norm_kernel<BF16, C, true, false>, grid, block, 0, st, p)
                                 : launch_pdl(norm_kernel<BF16, C, false, false>, grid, block, 0, st, p);
}

template <bool BF16>
cudaError_t launch_norm_t(const NormParams& p, cudaStream_t st) {
    auto threads = [&](int c) { return (int)((p.H + 256 * c - 1) / (256 * c)) * 32; };
    if (threads(1) <= 512) return launch_c<BF16, 1>(p, threads(1), st);
    if (threads(2) <= 512) return launch_c<BF16, 2>(p, threads(2), st);
    return launch_c<BF16, 4>(p, threads(4), st);   // up to 1024 threads: H <= 32768
}

// 16 tokens for each block of 256 threads: 16 lanes take one token's block of 128, U of them in turn whose
// loads are all issued first.  The scales of 16 tokens are neighbours.
template <bool BF16, int U>
__global__ void __launch_bounds__(256) quantize_kernel(const NormParams p) {
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
        float y[8];
        unpack8<BF16>(xr[u], y);
        const BlockScale q(block_most(y));
        if (row && at < p.H) {
            *reinterpret_cast<uint2*>(p.codes + t * p.H + at) = codes8(y, q.inv);
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
