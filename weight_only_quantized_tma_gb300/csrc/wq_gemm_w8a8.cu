// wq_gemm_w8a8.cu -- products of 8-bit activations and 8-bit weights (include/wq.h: wq_gemm_w8a8_fp8,
// wq_gemm_w8a8_fp8_gated).
//
//   out[m, n] = sum_kb  a_scale[kb, m] w_scale[n / 128, kb]  sum_{k in kb} a[m, k] w[n, k]
//
// Plain kernel: 32 tokens x 128 weight rows for each block of 256 threads, products and sums in fp32.
#include "wq_fp8.cuh"

namespace wq {
namespace {

__device__ __forceinline__ float from_e4m3(uint8_t v) {
    const uint32_t h = ptx::e4m3x2_to_f16x2(v);
    return __half2float(__ushort_as_half((unsigned short)(h & 0xFFFFu)));
}

template <bool GATED>
__global__ void __launch_bounds__(256) w8a8_plain_kernel(const W8A8Params p) {
    constexpr int P = GATED ? 2 : 1;
    __shared__ float as[32][33], ws[P][128][33];
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int64_t m0 = (int64_t)blockIdx.y * 32;
    const int nb = blockIdx.x, tx = threadIdx.x & 31, ty = threadIdx.x >> 5;   // rows tx + 32 j, tokens ty * 4 + i
    const int64_t n0 = (int64_t)nb * 128;
    const int64_t nblocks = (p.N + 127) / 128;
    float acc[P][4][4] = {};
    for (int kb = 0; kb < p.kblocks; ++kb) {
        float part[P][4][4] = {};
        for (int k0 = kb * 128; k0 < kb * 128 + 128 && k0 < p.K; k0 += 32) {
            __syncthreads();
            for (int e = threadIdx.x; e < 32 * 32; e += 256) {
                const int64_t m = m0 + e / 32;
                const int k = k0 + e % 32;
                as[e / 32][e % 32] = m < p.M && k < p.K ? from_e4m3(p.a[m * p.K + k]) : 0.f;
            }
            for (int h = 0; h < P; ++h)
                for (int e = threadIdx.x; e < 128 * 32; e += 256) {
                    const int64_t n = n0 + e / 32;
                    const int k = k0 + e % 32;
                    ws[h][e / 32][e % 32] = n < p.N && k < p.K ? from_e4m3(p.w[(h * p.N + n) * p.K + k]) : 0.f;
                }
            __syncthreads();
            for (int k = 0; k < 32; ++k)
#pragma unroll
                for (int h = 0; h < P; ++h)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) part[h][i][j] += as[ty * 4 + i][k] * ws[h][tx + 32 * j][k];
        }
#pragma unroll
        for (int h = 0; h < P; ++h) {
            const float sw = p.w_scale[(h * nblocks + nb) * p.kblocks + kb];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t m = m0 + ty * 4 + i;
                const float s = m < p.M ? sw * p.a_scale[(int64_t)kb * p.M + m] : 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[h][i][j] += s * part[h][i][j];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + ty * 4 + i;
        float v[4], top = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t n = n0 + tx + 32 * j;
            v[j] = acc[0][i][j];
            if (GATED) v[j] = v[j] / (1.f + __expf(-v[j])) * acc[P - 1][i][j];
            if (!GATED && p.bias != nullptr && n < p.N) v[j] += p.out_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.bias)[n]) : __half2float(static_cast<const __half*>(p.bias)[n]);
            if (n < p.N) top = max_nan(top, fabsf(v[j]));
            if (p.out != nullptr && m < p.M && n < p.N) {
                if (p.out_bf16) static_cast<__nv_bfloat16*>(p.out)[m * p.N + n] = __float2bfloat16_rn(v[j]);
                else static_cast<__half*>(p.out)[m * p.N + n] = __float2half_rn(v[j]);
            }
        }
        if (GATED && p.codes != nullptr) {
            for (int off = 16; off > 0; off >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, off));
            const BlockScale q(top);
            if (m < p.M) {
                for (int j = 0; j < 4; ++j)
                    if (n0 + tx + 32 * j < p.N) p.codes[m * p.N + n0 + tx + 32 * j] = q.inv == 0.f ? 0 : (uint8_t)to_e4m3x4(v[j] * q.inv, 0.f, 0.f, 0.f);
                if (tx == 0) p.scales[(int64_t)nb * p.M + m] = q.scale;
            }
        }
    }
}

}  // namespace

cudaError_t launch_w8a8(const W8A8Params& p, int sms, cudaStream_t st) {
    (void)sms;
    const dim3 grid((unsigned)((p.N + 127) / 128), (unsigned)((p.M + 31) / 32));
    if (p.gated) w8a8_plain_kernel<true><<<grid, 256, 0, st>>>(p);
    else w8a8_plain_kernel<false><<<grid, 256, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace wq
