// wq_attn_prompt.cu -- instantiations of the many-row attention kernel over the 4-bit cache.
#include "wq_attn_prompt.cuh"

namespace wq {
namespace {

template <bool BF16, int D>
cudaError_t launch(const AttnParams& p, int sms, cudaStream_t st) {
    using C = PromptCfg<D>;
    const int stage = (kPromptTN * (D + 8 * (D / p.c.G)) + 127) / 128 * 128;
    constexpr int most = 1024 + C::OFF_RAW + C::RAW_STAGES * kPromptTN * (D + 8 * (D / 32));
    static_assert(most <= 227 * 1024, "shared memory");
    cudaError_t e = cudaFuncSetAttribute(attn_prompt_kernel<BF16, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
    return launch_pdl(attn_prompt_kernel<BF16, D>, (unsigned)sms, kPromptThreads, 1024 + C::OFF_RAW + C::RAW_STAGES * stage, st,
                      p, stage);
}

}  // namespace

cudaError_t launch_attn_kv4_prompt(const AttnParams& p, bool bf16, int sms, cudaStream_t st) {
    if (bf16) return p.c.D == 128 ? launch<true, 128>(p, sms, st) : launch<true, 64>(p, sms, st);
    return p.c.D == 128 ? launch<false, 128>(p, sms, st) : launch<false, 64>(p, sms, st);
}
size_t attn_kv4_prompt_ws(const Kv4View& c, int sms) {
    return kAttnCounterBytes + (size_t)sms * 2 * attn_slot_floats(kPromptRows, c.D) * 4;
}

}  // namespace wq
