// wq_attn_decode.cu -- instantiations of the few-row attention kernel over the 4-bit cache.
#include <atomic>
#include <type_traits>

#include "wq_attn_decode.cuh"

namespace wq {
namespace {

constexpr int kMaxDevices = 64;

template <bool BF16, int D, int NT>
struct Launcher {
    using C = DecodeCfg<D, NT>;
    static int stage_bytes(const Kv4View& c) { return (kDecodeTN * (D + 8 * (D / c.G)) + 127) / 128 * 128; }
    static int smem(const Kv4View& c) { return C::OFF_RING + kDecodeStages * stage_bytes(c); }
    static int blocks_per_sm(const Kv4View& c) {
        // resident blocks for each group size; asked (and the kernel's shared memory allowed) once for
        // each instantiation and device
        static std::atomic<int> known[kMaxDevices][3];
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
        std::atomic<int>& k = known[dev][c.g_shift - 5];
        int n = k.load(std::memory_order_relaxed);
        if (n == 0) {
            const int bytes = smem(c);
            if (cudaFuncSetAttribute(attn_decode_kernel<BF16, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     C::OFF_RING + kDecodeStages * ((kDecodeTN * (D + 8 * (D / 32)) + 127) / 128 * 128)) !=
                    cudaSuccess ||
                cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, attn_decode_kernel<BF16, D, NT>, 160, bytes) !=
                    cudaSuccess ||
                n < 1)
                return 0;
            k.store(n, std::memory_order_relaxed);
        }
        return n;
    }
    static cudaError_t launch(const AttnParams& p, int sms, cudaStream_t st) {
        const int per = blocks_per_sm(p.c);
        if (per == 0) return cudaErrorInvalidConfiguration;
        return launch_pdl(attn_decode_kernel<BF16, D, NT>, (unsigned)(sms * per), 160, smem(p.c), st, p, stage_bytes(p.c));
    }
    static size_t ws_bytes(const Kv4View& c, int sms) {
        return kAttnCounterBytes + (size_t)sms * blocks_per_sm(c) * 2 * attn_slot_floats(C::R, D) * 4;
    }
};

template <typename F>
auto pick(const Kv4View& c, bool bf16, int64_t rows, F f) {
    auto nt = [&](auto b, auto d) {
        constexpr bool B = decltype(b)::value;
        constexpr int DD = decltype(d)::value;
        // as few row tiles as can be (each unpacks the codes anew), of equal height
        const int64_t eights = (rows + 7) / 8, tiles = (eights + kDecodeMaxNT - 1) / kDecodeMaxNT;
        const int64_t n = (eights + tiles - 1) / tiles;
        if (n <= 1) return f(Launcher<B, DD, 1>{});
        if (n == 2) return f(Launcher<B, DD, 2>{});
        return f(Launcher<B, DD, 3>{});
    };
    using I64 = std::integral_constant<int, 64>;
    using I128 = std::integral_constant<int, 128>;
    if (bf16) return c.D == 128 ? nt(std::true_type{}, I128{}) : nt(std::true_type{}, I64{});
    return c.D == 128 ? nt(std::false_type{}, I128{}) : nt(std::false_type{}, I64{});
}

}  // namespace

cudaError_t launch_attn_kv4_decode(const AttnParams& p, bool bf16, int64_t rows, int sms, cudaStream_t st) {
    return pick(p.c, bf16, rows, [&](auto l) { return decltype(l)::launch(p, sms, st); });
}
size_t attn_kv4_decode_ws(const Kv4View& c, bool bf16, int64_t rows, int sms) {
    return pick(c, bf16, rows, [&](auto l) { return decltype(l)::ws_bytes(c, sms); });
}

}  // namespace wq
