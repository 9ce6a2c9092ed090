// wq_gemm_w8a8.cu -- products of 8-bit activations and 8-bit weights (include/wq.h: wq_gemm_w8a8_fp8,
// wq_gemm_w8a8_fp8_gated): which kernel, its tensor maps, its launch.
#include <algorithm>
#include <mutex>

#include "wq_w8a8_mid.cuh"
#include "wq_w8a8_narrow.cuh"
#include "wq_w8a8_wide.cuh"

namespace wq {
namespace {

constexpr int kMaxDevices = 64;
constexpr int kMaxSplits = 8;

// One instantiation of the kernels with one tile for each cluster of `splits` blocks: its attributes, and how many
// clusters of S blocks the device holds at once (asked once for each device).  TM tokens x 128 weight rows (of each
// half) a tile, BOX_W weight rows a copy.
template <typename C, void (*KERNEL)(W8A8Params), int TM, int CTAS, int BOX_W>
struct Split {
    static constexpr auto kernel = KERNEL;
    struct Device {
        std::once_flag once;
        cudaError_t err = cudaSuccess;
        int clusters[kMaxSplits + 1] = {};
    };
    static const Device* device(int sms) {
        static Device devices[kMaxDevices];
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
        Device& d = devices[dev];
        std::call_once(d.once, [&]() {
            d.err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
            if (d.err == cudaSuccess) d.err = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
            // The query counts one block of a kernel with tensor memory for each SM; CTAS are resident (304 blocks of
            // CTAS = 2 ran at once on 152 SMs, in clusters of two as well, 296 in clusters of four), and what the query
            // leaves over in each part of the GPU then holds clusters too.
            d.clusters[1] = CTAS * sms;
            for (int S = 2; S <= C::SMAX && d.err == cudaSuccess; ++S) {
                cudaLaunchConfig_t cfg = {};
                cudaLaunchAttribute attr = {};
                fill(cfg, &attr, (unsigned)S, S, nullptr);
                int n = 0;
                if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) (void)cudaGetLastError(), n = 0;
                if (CTAS > 1) n = CTAS * n + std::max(0, sms - n * S) / S;
                d.clusters[S] = n - (n + 31) / 32;   // (fewer are placed at once than the query reports)
            }
        });
        return d.err == cudaSuccess ? &d : nullptr;
    }
    static void fill(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, unsigned grid, int S, cudaStream_t st) {
        cfg.gridDim = dim3(grid);
        cfg.blockDim = dim3(C::NTHREADS);
        cfg.dynamicSmemBytes = C::SMEM;
        cfg.stream = st;
        attr->id = cudaLaunchAttributeClusterDimension;
        attr->val.clusterDim.x = (unsigned)S;
        attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    // Slices of K that end soonest, and when, in 10 ns: the rounds of clusters times (`block` for each block of K and `ends`
    // to start and end), and 1 us for the exchange.  0 slices: the device cannot be asked.
    struct Plan {
        int splits;
        int64_t cost;
    };
    static Plan plan(const W8A8Params& p, int sms, int block, int ends) {
        const Device* d = device(sms);
        Plan best{0, 0};
        if (!d) return best;
        const int64_t tiles = (p.M + TM - 1) / TM * ((p.N + 127) / 128);
        for (int s = 1; s <= C::SMAX && (s == 1 || p.kblocks >= 2 * s); ++s) {
            if (d->clusters[s] < 1) continue;
            const int64_t rounds = (tiles + d->clusters[s] - 1) / d->clusters[s];
            const int64_t cost = rounds * ((p.kblocks + s - 1) / s * block + ends) + (s > 1 ? 100 : 0);
            if (s == 1 || cost < best.cost) best = Plan{s, cost};
        }
        return best;
    }
    static cudaError_t launch(W8A8Params p, int S, cudaStream_t st) {
        if (S < 1) return cudaErrorInvalidDevice;
        const int64_t tiles_m = (p.M + TM - 1) / TM, tiles_n = (p.N + 127) / 128, tiles = tiles_m * tiles_n;
        if (tiles * kMaxSplits >= (1LL << 31)) return cudaErrorInvalidValue;
        p.tiles_m = (int)tiles_m;
        p.tiles_n = (int)tiles_n;
        p.splits = S;
        p.box_m = (int)std::min<int64_t>(TM, p.M);
        const uint64_t a_dims[2] = {(uint64_t)p.K, (uint64_t)p.M}, a_strides[1] = {(uint64_t)p.K};
        const uint64_t w_dims[3] = {(uint64_t)p.K, (uint64_t)p.N, (uint64_t)C::H};
        const uint64_t w_strides[2] = {(uint64_t)p.K, (uint64_t)p.K * p.N};
        const uint32_t a_box[2] = {128, (uint32_t)p.box_m}, w_box[3] = {128, BOX_W, 1};
        if (!encode_tensor_map(&p.tmap_a, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.a, 2, a_dims, a_strides, a_box,
                               CU_TENSOR_MAP_SWIZZLE_128B) ||
            !encode_tensor_map(&p.tmap_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.w, 3, w_dims, w_strides, w_box,
                               CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[2] = {};
        fill(cfg, &attr[1], (unsigned)(tiles * S), S, st);
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = S > 1 ? 2 : 1;
        return cudaLaunchKernelEx(&cfg, kernel, p);
    }
};

template <typename C>
using Narrow = Split<C, w8a8_narrow_kernel<C>, C::BN, C::CTAS, 128>;
template <bool GATED>
using Mid = Split<MidCfg<GATED>, w8a8_mid_kernel<MidCfg<GATED>>, 128, 1, 64>;

// Pairs of blocks over tiles of 256 tokens x 256 weight rows.
template <bool GATED>
struct Wide {
    using C = WideCfg<GATED>;
    static constexpr auto kernel = w8a8_wide_kernel<C>;
    struct Device {
        std::once_flag once;
        cudaError_t err = cudaSuccess;
        int pairs = 0;       // held at once
    };
    static const Device* device() {
        static Device devices[kMaxDevices];
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
        Device& d = devices[dev];
        std::call_once(d.once, [&]() {
            d.err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute attr = {};
            fill(cfg, &attr, 2, nullptr);
            if (d.err == cudaSuccess) d.err = cudaOccupancyMaxActiveClusters(&d.pairs, kernel, &cfg);
        });
        return d.err == cudaSuccess && d.pairs > 0 ? &d : nullptr;
    }
    static void fill(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, unsigned grid, cudaStream_t st) {
        cfg.gridDim = dim3(grid);
        cfg.blockDim = dim3(C::NTHREADS);
        cfg.dynamicSmemBytes = C::SMEM;
        cfg.stream = st;
        attr->id = cudaLaunchAttributeClusterDimension;
        attr->val.clusterDim.x = 2;
        attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    // When its rounds of tiles have ended, in 10 ns: `block` for each block of K, 2 us for each tile, 3 for the kernel.
    static int64_t cost(const W8A8Params& p, int block) {
        const Device* d = device();
        if (!d) return INT64_MAX;
        const int64_t tiles = (p.M + 255) / 256 * ((p.N + C::TILE_N - 1) / C::TILE_N);
        return (tiles + d->pairs - 1) / d->pairs * ((int64_t)p.kblocks * block + 200) + 300;
    }
    static cudaError_t launch(W8A8Params p, cudaStream_t st) {
        const Device* d = device();
        if (!d) return cudaErrorInvalidDevice;
        const int64_t tiles_m = (p.M + 255) / 256, tiles_n = (p.N + C::TILE_N - 1) / C::TILE_N;
        if (tiles_m * tiles_n >= (1LL << 30) || tiles_n >= (1LL << 27)) return cudaErrorInvalidValue;
        p.tiles_m = (int)tiles_m;
        p.tiles_n = (int)tiles_n;
        p.div_group = make_fastdiv((uint32_t)(C::GROUP * tiles_n), (uint32_t)(tiles_m * tiles_n));
        const uint64_t a_dims[2] = {(uint64_t)p.K, (uint64_t)p.M}, a_strides[1] = {(uint64_t)p.K};
        const uint64_t w_dims[3] = {(uint64_t)p.K, (uint64_t)p.N, (uint64_t)C::H};
        const uint64_t w_strides[2] = {(uint64_t)p.K, (uint64_t)p.K * p.N};
        const uint32_t a_box[2] = {128, 128}, w_box[3] = {128, 64, 1};
        const bool codes = p.out == nullptr;
        const uint64_t o_dims[2] = {(uint64_t)p.N, (uint64_t)p.M}, o_strides[1] = {(uint64_t)p.N * (codes ? 1 : 2)};
        const uint32_t o_box[2] = {64, 32};
        if (!encode_tensor_map(&p.tmap_a, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.a, 2, a_dims, a_strides, a_box,
                               CU_TENSOR_MAP_SWIZZLE_128B) ||
            !encode_tensor_map(&p.tmap_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.w, 3, w_dims, w_strides, w_box,
                               CU_TENSOR_MAP_SWIZZLE_128B) ||
            !encode_tensor_map(&p.tmap_out, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16,
                               codes ? (const void*)p.codes : p.out, 2, o_dims, o_strides, o_box,
                               codes ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[2] = {};
        fill(cfg, &attr[1], 2 * (unsigned)std::min<int64_t>(tiles_m * tiles_n, d->pairs), st);
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        return cudaLaunchKernelEx(&cfg, kernel, p);
    }
};

// Up to 32 tokens weight rows are the tensor cores' M dimension: nothing of a tile is unused but what 16 or 32 exceed
// the tokens by, and two blocks are resident on each SM.  From there on tokens are, in tiles of a block's own or of a
// pair's, whichever ends first.  What a block of K takes is measured (10 ns): 33 in a tile of a block's own (62 gated),
// 42 (44) in a pair's, which is four times as large (gated twice).  Both measured, in us:
//   tokens x rows x K           own   pair      tokens x rows x K, gated    own   pair
//   333 x 4096 x 4096          14.3   18.9      64 x 11008 x 4096          22.7   34.5
//   512 x 4096 x 4096          14.9   19.1      250 x 4096 x 4096          22.7   19.0
//   768 x 4096 x 4096          35.9   19.2      250 x 11008 x 4096         46.8   35.3
//   333 x 12288 x 4096         29.6   33.6      777 x 6928 x 2560          53.5   34.9
//   512 x 12288 x 4096         43.7   34.1
// (Weight rows as M in tiles of 64 or 128 tokens took longer than tokens as M from 33 tokens on, by an eighth to a third.)
template <bool GATED>
cudaError_t launch_many(const W8A8Params& p, int sms, cudaStream_t st) {
    const typename Mid<GATED>::Plan own = Mid<GATED>::plan(p, sms, GATED ? 62 : 33, 400);
    if (Wide<GATED>::cost(p, GATED ? 44 : 42) < own.cost) return Wide<GATED>::launch(p, st);
    return Mid<GATED>::launch(p, own.splits, st);
}
template <typename K>
cudaError_t launch_few(const W8A8Params& p, int sms, cudaStream_t st) {
    return K::launch(p, K::plan(p, sms, 50, 200).splits, st);
}

}  // namespace

cudaError_t launch_w8a8(const W8A8Params& p, int sms, cudaStream_t st) {
    if (p.M > 32) return p.gated ? launch_many<true>(p, sms, st) : launch_many<false>(p, sms, st);
    if (p.gated) {
        if (p.M <= 16) return launch_few<Narrow<NarrowCfg<16, true, 3, 8, 2, true>>>(p, sms, st);
        return launch_few<Narrow<NarrowCfg<32, true, 3, 8, 2, true>>>(p, sms, st);
    }
    if (p.M <= 16) return launch_few<Narrow<NarrowCfg<16, false, 4, 8, 2, false>>>(p, sms, st);
    return launch_few<Narrow<NarrowCfg<32, false, 5, 8, 2, true>>>(p, sms, st);
}

}  // namespace wq
