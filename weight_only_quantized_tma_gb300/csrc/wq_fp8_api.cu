// wq_fp8_api.cu -- C entry points around 8-bit projections (include/wq.h): norm with the residual's
// addition, quantiser, products of 8-bit activations and weights.  Argument validation and launches;
// host code only.
#include <cmath>
#include <cuda_runtime.h>
#include <cstdint>

#include "../../include/wq.h"
#include "wq_internal.h"

using namespace wq;

namespace {

constexpr int64_t kMaxTokens = (1LL << 31) - 1;
constexpr int64_t kMaxStride = 1LL << 40;
constexpr int64_t kMaxWidth = 32768;      // of a normed row: 512 threads x 64 values

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
wq_status finish_launch(cudaError_t e) { return e == cudaSuccess ? WQ_OK : WQ_ERR_CUDA; }
bool type_ok(int dtype) { return dtype == WQ_F16 || dtype == WQ_BF16; }
bool stride_ok(int64_t stride, int64_t row) { return stride >= row && stride <= kMaxStride && stride % 8 == 0; }

wq_status norm_call(const void* x, int64_t x_stride, const void* residual, int64_t r_stride, wq_dtype dtype, int64_t T,
                    int64_t H, const void* weight, float eps, void* sum, int64_t sum_stride, void* out,
                    int64_t out_stride, uint8_t* codes, float* scales, bool quant, wq_stream_t stream) {
    const int64_t step = quant ? 16 : 8;
    if (T < 0 || T > kMaxTokens || H < step || H > kMaxWidth || H % step != 0 || !(eps >= 0.0f) || std::isinf(eps))
        return WQ_ERR_SHAPE;
    if (!type_ok(dtype)) return WQ_ERR_DTYPE;
    if (T == 0) return WQ_OK;
    if (!x || !weight || (residual && !sum) || (quant ? !codes || !scales : !out)) return WQ_ERR_NULL;
    if (!stride_ok(x_stride, H) || (residual && (!stride_ok(r_stride, H) || !stride_ok(sum_stride, H))) ||
        (!quant && !stride_ok(out_stride, H)))
        return WQ_ERR_SHAPE;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(sum, 16) || !aligned(out, 16) ||
        !aligned(codes, 16) || !aligned(scales, 4))
        return WQ_ERR_MISALIGNED;
    if (residual && !quant && sum == out) return WQ_ERR_SHAPE;      // (each would be the other's)
    DeviceState d{};
    const wq_status st = (wq_status)current_device_state(&d);
    if (st != WQ_OK) return st;
    NormParams p{};
    p.x = x;
    p.x_stride = x_stride;
    p.residual = residual;
    p.r_stride = r_stride;
    p.sum = sum;
    p.sum_stride = sum_stride;
    p.weight = weight;
    p.out = out;
    p.out_stride = out_stride;
    p.codes = codes;
    p.scales = scales;
    p.T = T;
    p.H = (int)H;
    p.eps = eps;
    p.inv_h = 1.0f / (float)H;
    return finish_launch(launch_add_rms_norm(p, dtype == WQ_BF16, (cudaStream_t)stream));
}

wq_status product_call(const uint8_t* a, const float* a_scale, const uint8_t* w, const float* w_scale, const void* bias,
                       int64_t M, int64_t N, int64_t K, wq_dtype dtype, void* out, uint8_t* codes, float* scales,
                       bool gated, wq_stream_t stream) {
    const int64_t step = gated ? 16 : 8;
    // (weight rows and k are coordinates of 32-bit tensor maps)
    if (M < 0 || M > kMaxTokens || N < step || N % step != 0 || N > (1LL << 29) || K < 16 || K % 16 != 0 ||
        K > (1LL << 30) || N * K >= (1LL << 40) || (M + 255) / 256 * ((N + 127) / 128) >= (1LL << 30))
        return WQ_ERR_SHAPE;
    if ((out || !gated) && !type_ok(dtype)) return WQ_ERR_DTYPE;
    if (M == 0) return WQ_OK;
    if (!a || !a_scale || !w || !w_scale) return WQ_ERR_NULL;
    if (gated ? (out ? codes || scales : !codes || !scales) : !out) return WQ_ERR_NULL;
    if (!aligned(a, 16) || !aligned(w, 16) || !aligned(a_scale, 4) || !aligned(w_scale, 4) || !aligned(bias, 2) ||
        !aligned(out, 16) || !aligned(codes, 16) || !aligned(scales, 4))
        return WQ_ERR_MISALIGNED;
    DeviceState d{};
    const wq_status st = (wq_status)current_device_state(&d);
    if (st != WQ_OK) return st;
    W8A8Params p{};
    p.a = a;
    p.a_scale = a_scale;
    p.w = w;
    p.w_scale = w_scale;
    p.bias = bias;
    p.out = out;
    p.codes = codes;
    p.scales = scales;
    p.M = M;
    p.N = N;
    p.K = (int)K;
    p.kblocks = (int)((K + 127) / 128);
    p.gated = gated;
    p.out_bf16 = out && dtype == WQ_BF16;
    p.status = d.status;
    p.timeout_ns = d.timeout_ns;
    return finish_launch(launch_w8a8(p, d.sms, (cudaStream_t)stream));
}

}  // namespace

extern "C" {

wq_status wq_add_rms_norm(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                          wq_dtype dtype, int64_t T, int64_t H, const void* weight, float eps, void* sum,
                          int64_t sum_stride, void* out, int64_t out_stride, wq_stream_t stream) {
    return norm_call(x, x_stride, residual, residual_stride, dtype, T, H, weight, eps, sum, sum_stride, out, out_stride,
                     nullptr, nullptr, false, stream);
}

wq_status wq_add_rms_norm_fp8(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                              wq_dtype dtype, int64_t T, int64_t H, const void* weight, float eps, void* sum,
                              int64_t sum_stride, uint8_t* codes, float* scales, wq_stream_t stream) {
    return norm_call(x, x_stride, residual, residual_stride, dtype, T, H, weight, eps, sum, sum_stride, nullptr, 0, codes,
                     scales, true, stream);
}

wq_status wq_quantize_fp8(const void* x, int64_t x_stride, wq_dtype dtype, int64_t T, int64_t K, uint8_t* codes,
                          float* scales, wq_stream_t stream) {
    if (T < 0 || T > kMaxTokens || K < 16 || K % 16 != 0 || K > (1LL << 30)) return WQ_ERR_SHAPE;
    if (!type_ok(dtype)) return WQ_ERR_DTYPE;
    if (T == 0) return WQ_OK;
    if (!x || !codes || !scales) return WQ_ERR_NULL;
    // (blocks of 16 tokens x 128 values are counted in 31 bits)
    if (!stride_ok(x_stride, K) || (T + 15) / 16 * ((K + 127) / 128) >= kMaxTokens) return WQ_ERR_SHAPE;
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return WQ_ERR_MISALIGNED;
    DeviceState d{};
    const wq_status st = (wq_status)current_device_state(&d);
    if (st != WQ_OK) return st;
    NormParams p{};
    p.x = x;
    p.x_stride = x_stride;
    p.codes = codes;
    p.scales = scales;
    p.T = T;
    p.H = (int)K;
    return finish_launch(launch_quantize_fp8(p, dtype == WQ_BF16, d.sms, (cudaStream_t)stream));
}

wq_status wq_gemm_w8a8_fp8(const uint8_t* a, const float* a_scale, const uint8_t* w, const float* w_scale,
                           const void* bias, int64_t M, int64_t N, int64_t K, wq_dtype dtype, void* out,
                           wq_stream_t stream) {
    return product_call(a, a_scale, w, w_scale, bias, M, N, K, dtype, out, nullptr, nullptr, false, stream);
}

wq_status wq_gemm_w8a8_fp8_gated(const uint8_t* a, const float* a_scale, const uint8_t* w, const float* w_scale,
                                 int64_t M, int64_t F, int64_t K, wq_dtype dtype, void* out, uint8_t* codes,
                                 float* scales, wq_stream_t stream) {
    return product_call(a, a_scale, w, w_scale, nullptr, M, F, K, dtype, out, codes, scales, true, stream);
}

}  // extern "C"
