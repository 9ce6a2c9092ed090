// wq_attn_api.cu -- C entry points between the projections of an attention layer
// (include/wq.h): norm + rotation, the 4-bit cache, attention over it.  Argument
// validation and launches; host code only.
#include <algorithm>
#include <cmath>
#include <cuda_runtime.h>
#include <cstdint>

#include "../../include/wq.h"
#include "wq_internal.h"

using namespace wq;

namespace {

constexpr int64_t kMaxTokens = (1LL << 31) - 1;
constexpr int64_t kMaxStride = 1LL << 40;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
wq_status finish_launch(cudaError_t e) { return e == cudaSuccess ? WQ_OK : WQ_ERR_CUDA; }
int log2i(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

wq_status check_layout(const wq_kv4_layout* l, uint8_t* pages, Kv4View* v) {
    if (!l) return WQ_ERR_NULL;
    if (l->kv_heads < 1 || l->kv_heads > 65535 || l->num_pages < 0 || l->num_pages > kMaxTokens) return WQ_ERR_SHAPE;
    if (l->head_dim != 64 && l->head_dim != 128) return WQ_ERR_SHAPE;
    if (l->page_size != 16 && l->page_size != 32 && l->page_size != 64 && l->page_size != 128) return WQ_ERR_SHAPE;
    if ((l->group != 32 && l->group != 64 && l->group != 128) || l->group > l->head_dim) return WQ_ERR_GROUP;
    if (l->dtype != WQ_F16 && l->dtype != WQ_BF16) return WQ_ERR_DTYPE;
    v->pages = pages;
    v->num_pages = l->num_pages;
    v->heads = l->kv_heads;
    v->D = l->head_dim;
    v->G = l->group;
    v->P = l->page_size;
    v->p_shift = log2i(l->page_size);
    v->g_shift = log2i(l->group);
    v->block_bytes = v->P * (v->D + 8 * (v->D / v->G));
    v->page_bytes = (int64_t)v->block_bytes * v->heads;
    return WQ_OK;
}

bool stride_ok(int64_t stride, int64_t row, int64_t step) {
    return stride >= row && stride <= kMaxStride && stride % step == 0;
}

// The few-row kernel's tiles hold 8 to 24 rows, the many-row kernel's 256.  Where the first
// would unpack the codes twice the second is as fast or faster once sequences are long.  Few / many
// rows, us, 8 key heads in bf16 (fp16 within 3 us of it), cold:
//   rows                             24       32       40       64      128
//   24 sequences of 4096, D = 64    53/80    88/80    88/82   119/84   223/90
//   24 sequences of 4096, D = 128   88/131  143/133  145/137  201/141  375/154
//   8 sequences of 1000, D = 64     20/27    27/31    27/31    31/33    41/41
//   8 sequences of 1000, D = 128    37/39    41/37    41/41    47/45    68/61
// (lengths are on the device, so the rule is on rows alone).
bool many_rows(int64_t rows) { return rows > 24; }

size_t attn_ws(const Kv4View& c, bool bf16, int64_t rows, int sms) {
    return many_rows(rows) ? attn_kv4_prompt_ws(c, sms) : attn_kv4_decode_ws(c, bf16, rows, sms);
}

wq_status rows_call(const void* k, int64_t k_stride, const void* v, int64_t v_stride, const int64_t* slots, int64_t T,
                    const wq_kv4_layout* layout, uint8_t* pages, wq_stream_t stream, bool write) {
    Kv4RowsParams p{};
    wq_status st = check_layout(layout, pages, &p.c);
    if (st != WQ_OK) return st;
    if (T < 0 || T > kMaxTokens) return WQ_ERR_SHAPE;
    if (T == 0) return WQ_OK;
    if (!k || !v || !slots || (!pages && p.c.num_pages > 0)) return WQ_ERR_NULL;
    const int64_t row = (int64_t)p.c.heads * p.c.D;
    if (!stride_ok(k_stride, row, 8) || !stride_ok(v_stride, row, 8) || T * p.c.heads >= kMaxTokens - 4096)
        return WQ_ERR_SHAPE;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(pages, 16) || !aligned(slots, 8)) return WQ_ERR_MISALIGNED;
    DeviceState d{};
    if ((st = (wq_status)current_device_state(&d)) != WQ_OK) return st;
    p.k = k;
    p.v = v;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.slots = slots;
    p.T = T;
    p.status = d.status;
    const bool bf16 = layout->dtype == WQ_BF16;
    return finish_launch(write ? launch_kv4_write(p, bf16, d.sms, (cudaStream_t)stream)
                               : launch_kv4_read(p, bf16, d.sms, (cudaStream_t)stream));
}

}  // namespace

extern "C" {

wq_status wq_qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, wq_dtype dtype, int64_t T,
                          int32_t Hq, int32_t Hkv, int32_t D, const void* q_weight, const void* k_weight, float eps,
                          const int64_t* positions, const float* cos_sin, int64_t max_pos, int32_t rot,
                          int32_t interleaved, void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                          wq_stream_t stream) {
    if (T < 0 || T > kMaxTokens || Hq < 1 || Hkv < 1 || Hq > 65535 || Hkv > 65535 || D < 8 || D > 256 || D % 8 != 0)
        return WQ_ERR_SHAPE;
    if (rot < 8 || rot > D || rot % 8 != 0 || max_pos < 0 || !(eps >= 0.0f) || std::isinf(eps)) return WQ_ERR_SHAPE;
    if (dtype != WQ_F16 && dtype != WQ_BF16) return WQ_ERR_DTYPE;
    if (T == 0) return WQ_OK;
    if (!q || !k || !positions || !cos_sin || !q_out || !k_out) return WQ_ERR_NULL;
    const int64_t rq = (int64_t)Hq * D, rk = (int64_t)Hkv * D;
    if (!stride_ok(q_stride, rq, 4) || !stride_ok(k_stride, rk, 4) || !stride_ok(q_out_stride, rq, 4) ||
        !stride_ok(k_out_stride, rk, 4) || T * (Hq + Hkv) >= kMaxTokens - 4096)
        return WQ_ERR_SHAPE;
    if (!aligned(q, 8) || !aligned(k, 8) || !aligned(q_out, 8) || !aligned(k_out, 8) || !aligned(q_weight, 8) ||
        !aligned(k_weight, 8) || !aligned(positions, 8) || !aligned(cos_sin, 16))
        return WQ_ERR_MISALIGNED;
    DeviceState d{};
    const wq_status st = (wq_status)current_device_state(&d);
    if (st != WQ_OK) return st;
    RopeParams p{};
    p.q = q;
    p.k = k;
    p.q_out = q_out;
    p.k_out = k_out;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.q_out_stride = q_out_stride;
    p.k_out_stride = k_out_stride;
    p.q_weight = q_weight;
    p.k_weight = k_weight;
    p.positions = positions;
    p.cos_sin = cos_sin;
    p.T = T;
    p.max_pos = max_pos;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.D = D;
    p.rot = rot;
    p.interleaved = interleaved != 0;
    p.eps = eps;
    p.status = d.status;
    return finish_launch(launch_qk_norm_rope(p, dtype == WQ_BF16, d.sms, (cudaStream_t)stream));
}

wq_status wq_kv4_page_bytes(const wq_kv4_layout* layout, size_t* bytes) {
    Kv4View v{};
    const wq_status st = check_layout(layout, nullptr, &v);
    if (st != WQ_OK) return st;
    if (!bytes) return WQ_ERR_NULL;
    *bytes = (size_t)v.page_bytes;
    return WQ_OK;
}

wq_status wq_kv4_write(const void* k, int64_t k_stride, const void* v, int64_t v_stride, const int64_t* slots,
                       int64_t T, const wq_kv4_layout* layout, uint8_t* pages, wq_stream_t stream) {
    return rows_call(k, k_stride, v, v_stride, slots, T, layout, pages, stream, true);
}

wq_status wq_kv4_read(const uint8_t* pages, const wq_kv4_layout* layout, const int64_t* slots, int64_t T, void* k,
                      int64_t k_stride, void* v, int64_t v_stride, wq_stream_t stream) {
    return rows_call(k, k_stride, v, v_stride, slots, T, layout, const_cast<uint8_t*>(pages), stream, false);
}

wq_status wq_attn_kv4_workspace_bytes(const wq_kv4_layout* layout, int32_t q_heads, int64_t max_q, size_t* bytes) {
    Kv4View v{};
    wq_status st = check_layout(layout, nullptr, &v);
    if (st != WQ_OK) return st;
    if (!bytes) return WQ_ERR_NULL;
    if (q_heads < 1 || q_heads > 65535 || q_heads % v.heads != 0 || max_q < 1) return WQ_ERR_SHAPE;
    DeviceState d{};
    if ((st = (wq_status)current_device_state(&d)) != WQ_OK) return st;
    *bytes = attn_ws(v, layout->dtype == WQ_BF16, std::min(max_q, kMaxTokens) * (q_heads / v.heads), d.sms);
    return WQ_OK;
}

wq_status wq_attn_kv4(const void* q, int64_t q_stride, int32_t q_heads, const int32_t* cu_q, int64_t B, int64_t T,
                      int64_t max_q, const uint8_t* pages, const wq_kv4_layout* layout, const int32_t* block_table,
                      int64_t table_stride, const int32_t* kv_lens, float scale, int32_t causal, int32_t window,
                      void* out, int64_t out_stride, float* lse, void* ws, size_t ws_bytes, wq_stream_t stream) {
    AttnParams p{};
    wq_status st = check_layout(layout, const_cast<uint8_t*>(pages), &p.c);
    if (st != WQ_OK) return st;
    if (q_heads < 1 || q_heads > 65535 || q_heads % p.c.heads != 0) return WQ_ERR_SHAPE;
    if (B < 0 || B > kMaxTokens || T < 0 || T > kMaxTokens || max_q < 1 || table_stride < 0 ||
        table_stride > kMaxTokens || window < 0 || (window > 0 && !causal) || !(std::fabs(scale) <= 0x1p127f))
        return WQ_ERR_SHAPE;
    if (!cu_q && T != B) return WQ_ERR_SHAPE;
    if (T * (q_heads / p.c.heads) >= kMaxTokens - 4096) return WQ_ERR_SHAPE;
    if (T == 0 || B == 0) return WQ_OK;
    if (!q || !out || !kv_lens || (!block_table && table_stride > 0) || (!pages && p.c.num_pages > 0)) return WQ_ERR_NULL;
    const int64_t row = (int64_t)q_heads * p.c.D;
    if (!stride_ok(q_stride, row, 8) || !stride_ok(out_stride, row, 8)) return WQ_ERR_SHAPE;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(pages, 16) || !aligned(cu_q, 4) || !aligned(block_table, 4) ||
        !aligned(kv_lens, 4) || !aligned(lse, 4) || !aligned(ws, 16))
        return WQ_ERR_MISALIGNED;
    DeviceState d{};
    if ((st = (wq_status)current_device_state(&d)) != WQ_OK) return st;
    p.q = q;
    p.out = out;
    p.lse = lse;
    p.q_stride = q_stride;
    p.out_stride = out_stride;
    p.cu_q = cu_q;
    p.table = block_table;
    p.lens = kv_lens;
    // without pages no token is cached: every length is cut to 0
    p.table_stride = p.c.num_pages > 0 ? table_stride : 0;
    p.most = (int)std::min(p.table_stride << p.c.p_shift, kMaxTokens - 4096);
    p.B = B;
    p.T = T;
    p.Hq = q_heads;
    p.group = q_heads / p.c.heads;
    p.div_group = make_fastdiv((uint32_t)p.group, (uint32_t)kMaxTokens);
    p.causal = causal != 0;
    p.window = window;
    p.scale = scale;
    p.status = d.status;
    p.timeout_ns = d.timeout_ns;
    const bool bf16 = layout->dtype == WQ_BF16;
    const int64_t rows = std::min(max_q, kMaxTokens) * p.group;
    if (!ws || ws_bytes < attn_ws(p.c, bf16, rows, d.sms)) return WQ_ERR_WORKSPACE;
    p.ws_count = static_cast<uint32_t*>(ws);
    p.ws_part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kAttnCounterBytes);
    if (many_rows(rows)) return finish_launch(launch_attn_kv4_prompt(p, bf16, d.sms, (cudaStream_t)stream));
    return finish_launch(launch_attn_kv4_decode(p, bf16, rows, d.sms, (cudaStream_t)stream));
}

}  // extern "C"
