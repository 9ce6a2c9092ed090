// wq_w8a8_wide.cuh -- product of e4m3 activations and e4m3 weights for many tokens: tokens are the tensor
// cores' M dimension, so a thread's row has one activation scale and its 128 columns one weight scale.
//
//   acc[m][n] += (a_scale[kb][m] w_scale[n / 128][kb]) * D_kb[m][n]
//
// A pair of blocks (cluster of two, cta_group::2) computes 256 tokens x 256 weight rows: each holds its 128
// tokens and the copies of half of the weight rows, D_kb of 128 k is one accumulation of four products in one
// of two buffers of tensor memory (256 columns each, all 512), and while the tensor cores fill one, eight warps
// read the other, scale it and add it in registers (128 columns for each thread of two warpgroups).  GATED: the
// 256 rows are 64 of the gate, the same 64 of up, the next 64 of the gate, of up, so a thread holds gate and up
// of the same 64 numbers, and the pair's tile is one block of 128 of the output.
#pragma once

#include "wq_common.cuh"
#include "wq_fp8.cuh"

namespace wq {

template <bool GATED_>
struct WideCfg {
    static constexpr bool GATED = GATED_;
    static constexpr int H = GATED ? 2 : 1;
    static constexpr int NTHREADS = 384;        // warp 0 copies, 1 and 3 products, 2 tensor memory and scales, 4-11 sums
    static constexpr int STAGES = GATED ? 5 : 4;
    static constexpr int STAGE = 2 * 128 * 128;             // 128 tokens, 128 weight rows
    static constexpr int OUT_WARP = GATED ? 4096 : 8192;    // a warp's part of the output: 32 rows of 128 or 256 bytes
    static constexpr int OFF_OUT = STAGES * STAGE;
    static constexpr int MOST = 2048;           // codes take half of a warp's part; largest magnitudes [2 tiles][32] behind
    // Scales of a block of K: 128 tokens', two of the weights.  They are part of the stage of the block before (its
    // products wait for them too; the first block's are with its own), so that sums that can be read find the next
    // block's scales without a wait of their own, and read them while they wait for its products: beside tensor cores
    // that read shared memory a wait takes about 100 cycles, a read hardly less (8192 x 4096 x 11008: 363 us with a
    // barrier of their own, 356 us with loads from memory two blocks ahead, 274 us in the stage; 8192 x 2048 x 11008
    // gated: 272 us read behind the wait, 265 us before it).  A slot is filled again SCN - 1 blocks on, when the
    // products of STAGES blocks before that have ended, for which the sums two blocks earlier had to be read, which
    // is at least the block whose scales these were.
    static constexpr int SCN = 8;
    static constexpr int SC_SLOT = 130 * 4 + 8;
    static constexpr int OFF_SC = OFF_OUT + 8 * OUT_WARP;
    static constexpr int OFF_BAR = OFF_SC + SCN * SC_SLOT;
    static constexpr int NBAR = 2 * STAGES + 4 + 4 + 2;         // full, empty, acc full / empty (2), pairs of warps (4), final
    static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;
    static constexpr int SMEM = OFF_MISC + 16 + 1024;
    static constexpr int TILE_N = GATED ? 128 : 256;            // columns of the output
    static constexpr int GROUP = 8;             // token tiles that the walk keeps together
    // Columns of the sums that a load reads: 32 leave fewer waits for loads (8192 x 12288 x 4096: 304 -> 302 us), but
    // the gated kernel, with two factors, then spills inside the loop (8192 x 2048 x 11008, gated: 271 -> 348 us).
    static constexpr int LOAD = GATED ? 16 : 32;
    // registers: 168 x 384 at launch = 72 x 128 + 216 x 256
    static constexpr int REGS_ISSUE = 72, REGS_SUM = 216;
    static_assert(SCN >= STAGES + 3 && (SCN & (SCN - 1)) == 0 && OFF_BAR % 8 == 0, "scales");
    static_assert(SMEM <= 232448, "shared memory");
};

template <typename C>
__global__ void __launch_bounds__(C::NTHREADS, 1) w8a8_wide_kernel(const __grid_constant__ W8A8Params p) {
    constexpr int STAGES = C::STAGES, H = C::H, SCN = C::SCN, LOAD = C::LOAD;
    constexpr bool GATED = C::GATED;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = ptx::smem_u32(smem);
    const uint32_t bar0 = sbase + C::OFF_BAR;
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (STAGES + s); };
    auto acc_full = [&](int b) { return bar0 + 8u * (2 * STAGES + b); };
    auto acc_empty = [&](int b) { return bar0 + 8u * (2 * STAGES + 2 + b); };
    auto pair_bar = [&](int q) { return bar0 + 8u * (2 * STAGES + 4 + q); };
    const uint32_t final_bar = bar0 + 8u * (2 * STAGES + 8);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)ptx::cluster_ctarank();     // 0 issues the products of both

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            // its own copies, its scales, and the other block's of both, passed on
            ptx::mbar_init(full(s), rank == 0 ? 34 : 33);
            ptx::mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) ptx::mbar_init(acc_full(b), 1), ptx::mbar_init(acc_empty(b), 16);
        for (int q = 0; q < 4; ++q) ptx::mbar_init(pair_bar(q), 2);
        ptx::mbar_init(final_bar, 1), ptx::mbar_init(final_bar + 8u, 1);
        *abort_flag = 0u;
        ptx::fence_barrier_init();
        ptx::fence_proxy_async_smem();
        ptx::prefetch_tmap(&p.tmap_a);
        ptx::prefetch_tmap(&p.tmap_w);
        ptx::prefetch_tmap(&p.tmap_out);
    }
    if (warp == 2) {
        ptx::tmem_alloc<2>(sbase + C::OFF_MISC, 512);
        ptx::tmem_relinquish<2>();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();      // both blocks' barriers are initialised
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();

    const int n_tiles = p.tiles_m * p.tiles_n, first = (int)(blockIdx.x >> 1), step = (int)(gridDim.x >> 1);
    // GROUP token tiles at a time, theirs fastest: the tiles in flight are about as many of one kind as of the
    // other, so that they read few panels and write neighbouring columns
    auto tile_at = [&](int t, int& mt, int& nt) {
        const int q = (int)fastdiv((uint32_t)t, p.div_group), r = t - q * (int)p.div_group.d;
        const int high = min(C::GROUP, p.tiles_m - q * C::GROUP);
        nt = r / high;
        mt = q * C::GROUP + r - nt * high;
    };
    const int64_t wblocks = (p.N + 127) >> 7;
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity, uint32_t code) {
        if (ok) ok = bounded_wait<true>(bar, parity, abort_flag, p.status, code, p.timeout_ns);
        return ok;
    };
    auto wait_all = [&](uint32_t bar, uint32_t parity, uint32_t code) {      // a warp's lanes together
        return ok = warp_wait<true>(ok, bar, parity, abort_flag, p.status, code, p.timeout_ns);
    };

    if (warp < 4) {
        ptx::regs_dec<C::REGS_ISSUE>();
        if (warp == 0 && lane == 0) {
            // -------------------------------------------------------- copies
            const uint64_t pol = ptx::policy_evict_last();
            int s = 0;
            uint32_t ph = 0;
            long long issued = 0;
            for (int t = first; t < n_tiles && ok; t += step) {
                int mt, nt;
                tile_at(t, mt, nt);
                for (int kb = 0; kb < p.kblocks && wait(empty(s), ph ^ 1u, DEVICE_TIMEOUT_PRODUCER); ++kb) {
                    const uint32_t dst = sbase + s * C::STAGE;
                    ptx::mbar_arrive_expect_tx(full(s), C::STAGE);
                    ptx::tma_load_2d(dst, &p.tmap_a, kb * 128, mt * 256 + rank * 128, full(s), pol);
#pragma unroll
                    for (int i = 0; i < 2; ++i)    // 64 rows of the gate and of up, or 128 rows
                        ptx::tma_load_3d(dst + 16384 + i * 8192, &p.tmap_w, kb * 128,
                                         nt * C::TILE_N + (GATED ? 64 * rank : 128 * rank + 64 * i), GATED ? i : 0, full(s), pol);
                    ++issued;
                    if (++s == STAGES) s = 0, ph ^= 1u;
                }
            }
            // every stage released: the commits that arrive here have all landed
            for (int j = 0; j < STAGES && wait(empty(s), ph ^ 1u, DEVICE_TIMEOUT_PRODUCER); ++j)
                if (++s == STAGES) s = 0, ph ^= 1u;
            if (!ok)
                for (long long j = issued > STAGES ? issued - STAGES : 0; j < issued; ++j)
                    if (!drain_wait(full((int)(j % STAGES)), (uint32_t)(j / STAGES) & 1u, p.timeout_ns))
                        atomicOr(p.status, DEVICE_TIMEOUT_DRAIN);
        } else if (warp == 2) {
            // -------------------------------------------------------- scales
            // (a warp of their own: in the warp of the copies they made it the slowest, 267 -> 259 us for 8192 x 4096 x 11008)
            int t = first, kb = 0, s = 0, c = 0;
            uint32_t ph = 0;
            int rows = 0;
            const float *sa = p.a_scale, *sw = p.w_scale;
            auto copy = [&]() {       // the next block's, if there is one
                if (t >= n_tiles) return;
                if (kb == 0) {
                    int mt, nt;
                    tile_at(t, mt, nt);
                    const int64_t m0 = (int64_t)mt * 256 + rank * 128;
                    rows = (int)max((int64_t)0, min((int64_t)128, p.M - m0));
                    sa = p.a_scale + (rows > 0 ? m0 : 0);
                    // lanes 0 and 1: the tile's two blocks of weight rows, or the gate's and up's
                    const int64_t wb = GATED ? (lane & 1) * wblocks + nt : min((int64_t)2 * nt + (lane & 1), wblocks - 1);
                    sw = p.w_scale + wb * p.kblocks;
                }
                const uint32_t sc = sbase + C::OFF_SC + c * C::SC_SLOT;
#pragma unroll
                for (int r = lane; r < 128; r += 32) ptx::cp_async4(sc + 4 * r, sa + (r < rows ? r : 0), r < rows);
                if (lane < 2) ptx::cp_async4(sc + 4 * (128 + lane), sw + kb, true);
                sa += p.M;
                if (++kb == p.kblocks) kb = 0, t += step;
                if (++c == SCN) c = 0;
            };
            const long long all = (long long)((n_tiles - first + step - 1) / step) * p.kblocks;
            for (long long i = 0; i < all; ++i) {
                if (!wait_all(empty(s), ph ^ 1u, DEVICE_TIMEOUT_PRODUCER)) break;
                if (i == 0) copy();       // the first block's own
                copy();
                ptx::cp_async_arrive(full(s));
                if (++s == STAGES) s = 0, ph ^= 1u;
            }
            ptx::cp_async_wait_all();
        } else if (warp == 1 && lane == 0 && rank == 1) {
            // -------------------------------------------------------- the landing of this block's copies, passed on
            const uint32_t to = ptx::mapa_shared(full(0), 0);
            int s = 0;
            uint32_t ph = 0;
            for (int t = first; t < n_tiles && ok; t += step)
                for (int kb = 0; kb < p.kblocks && wait(full(s), ph, DEVICE_TIMEOUT_MMA); ++kb) {
                    ptx::mbar_arrive_cluster(to + 8u * s);
                    if (++s == STAGES) s = 0, ph ^= 1u;
                }
        } else if ((warp == 1 || warp == 3) && lane == 0 && rank == 0) {
            // -------------------------------------------------------- products
            // Two warps issue in turn, each for one buffer of sums: a block's waits, commits and loop (some 250 cycles)
            // then lie beside the other warp's products, which the tensor cores only take as fast as they work.
            constexpr uint32_t idesc = ptx::make_idesc_e4m3(256, 256);
            const uint32_t b = warp >> 1;
            const long long all = (long long)((n_tiles - first + step - 1) / step) * p.kblocks;
            int s = (int)b;
            uint32_t ph = 0, use = 0;      // use: how often this buffer has been used
            for (long long n = b; n < all; n += 2, ++use) {
                if (!wait(full(s), ph, DEVICE_TIMEOUT_MMA) || !wait(acc_empty(b), (use & 1u) ^ 1u, DEVICE_TIMEOUT_MMA)) break;
                ptx::tc_fence_after();
                const uint32_t a_lo = ptx::sdesc_lo(sbase + s * C::STAGE), b_lo = a_lo + (16384 >> 4);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    ptx::mma_f8_ss<2>(tmem + b * 256, a_lo + 2 * k, ptx::kSdescHi, b_lo + 2 * k, ptx::kSdescHi, idesc, k > 0);
                ptx::mma_commit_pair(acc_full(b));
                ptx::mma_commit_pair(empty(s));
                if ((s += 2) >= STAGES) s -= STAGES, ph ^= 1u;
            }
            // the last arrivals of the other block land before this one may end
            if (use > 0) wait(acc_empty(b), (use - 1) & 1u, DEVICE_TIMEOUT_MMA);
            if (!ok) {
                ptx::mma_commit<2>(final_bar + 8u * b);
                if (!drain_wait(final_bar + 8u * b, 0, p.timeout_ns)) atomicOr(p.status, DEVICE_TIMEOUT_DRAIN);
            }
        }
        __syncwarp();
    } else {
        ptx::regs_inc<C::REGS_SUM>();
        // ------------------------------------------------------------ sums
        const int g = (warp - 4) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t base = tmem + ((uint32_t)(quarter * 32) << 16) + g * 128;
        const uint32_t acc_empty0 = ptx::mapa_shared(acc_empty(0), 0);
        uint8_t* out_s = smem + C::OFF_OUT + (warp - 4) * C::OUT_WARP;
        uint32_t n = 0, turn = 0;
        wait_all(acc_full(0), 0, DEVICE_TIMEOUT_TRANSFORM);      // the first scales have landed
        for (int t = first; t < n_tiles && ok; t += step, ++turn) {
            // Pairs of neighbouring columns, as the packed products take them: as single numbers ten of them were spilled
            // (8192 x 4096 x 11008, with the wider loads: 259 -> 255 us, 8192 x 2048 x 11008 gated: 270 -> 267 us).
            uint64_t sum[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) sum[i] = 0;
            for (int kb = 0; kb < p.kblocks; ++kb, ++n) {
                const uint32_t b = n & 1u;
                const volatile float* sc = reinterpret_cast<const volatile float*>(smem + C::OFF_SC + n % SCN * C::SC_SLOT);
                uint64_t s[H];
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const float f = sc[row] * sc[128 + (GATED ? h : g)];
                    s[h] = f2(f, f);
                }
                if (!wait_all(acc_full(b), n >> 1 & 1u, DEVICE_TIMEOUT_TRANSFORM)) break;
                ptx::tc_fence_after();
                uint32_t v[2][LOAD];
                ptx::tmem_ld(base + b * 256, v[0]);
#pragma unroll
                for (int c = 0; c < 128 / LOAD; ++c) {
                    ptx::tmem_wait_ld_of(v[c & 1]);
                    if (c < 128 / LOAD - 1) {
                        ptx::tmem_ld(base + b * 256 + LOAD * (c + 1), v[(c + 1) & 1]);
                    } else {
                        ptx::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive_cluster(acc_empty0 + 8u * b);
                    }
#pragma unroll
                    for (int j = 0; j < LOAD; j += 2) {
                        const int col = LOAD * c + j;
                        sum[col / 2] = fma_f2(f2(__uint_as_float(v[c & 1][j]), __uint_as_float(v[c & 1][j + 1])),
                                              s[GATED ? col >> 6 : 0], sum[col / 2]);
                    }
                }
            }
            if (!ok) break;
            float acc[128];
#pragma unroll
            for (int i = 0; i < 64; ++i) {
                const float2 r = un2(sum[i]);
                acc[2 * i] = r.x, acc[2 * i + 1] = r.y;
            }
            // ---- output: through this warp's part of shared memory, 32 rows copied out by one thread
            if (lane == 0) ptx::bulk_wait_group_read0();     // the last copy has read it
            __syncwarp();
            int mt, nt;
            tile_at(t, mt, nt);
            const int64_t m = (int64_t)mt * 256 + rank * 128 + row;
            const int64_t n0 = (int64_t)nt * C::TILE_N + g * (128 / H);
            const bool any = n0 < p.N && m - lane < p.M;      // the warp has something to store
            if constexpr (GATED) {
#pragma unroll
                for (int i = 0; i < 64; ++i) acc[i] = silu(acc[i]) * acc[64 + i];
            } else if (p.bias != nullptr && n0 < p.N) {
#pragma unroll
                for (int i = 0; i < 128; ++i)
                    if (n0 + i < p.N)
                        acc[i] += p.out_bf16 ? load_16bit<true>(p.bias, (size_t)(n0 + i)) : load_16bit<false>(p.bias, (size_t)(n0 + i));
            }
            if (!GATED || p.out != nullptr) {
                // rows of 128 bytes (64 columns), in the order of the 128-byte swizzle
#pragma unroll
                for (int c = 0; c < 128 / H; c += 8) {
                    const uint4 o = p.out_bf16 ? make_uint4(pack2<true>(acc[c], acc[c + 1]), pack2<true>(acc[c + 2], acc[c + 3]),
                                                            pack2<true>(acc[c + 4], acc[c + 5]), pack2<true>(acc[c + 6], acc[c + 7]))
                                               : make_uint4(pack2<false>(acc[c], acc[c + 1]), pack2<false>(acc[c + 2], acc[c + 3]),
                                                            pack2<false>(acc[c + 4], acc[c + 5]), pack2<false>(acc[c + 6], acc[c + 7]));
                    *reinterpret_cast<uint4*>(out_s + (c >> 6) * 4096 + swz(lane * 128 + (c & 63) * 2, 7)) = o;
                }
            } else {
                // the block's largest: this thread's 64 and those of the same row in the other warpgroup
                float most = 0.f;
#pragma unroll
                for (int i = 0; i < 64; i += 2) most = max_nan(most, fabsf(acc[i]), fabsf(acc[i + 1]));     // (past N: products of zeros)
                const int at = C::MOST + (int)(turn & 1u) * 128 + 4 * lane;
                *reinterpret_cast<float*>(out_s + at) = most;
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(pair_bar(quarter));
                if (!wait_all(pair_bar(quarter), turn & 1u, DEVICE_TIMEOUT_EPILOGUE)) break;
                const BlockScale q(max_nan(most, *reinterpret_cast<const float*>(smem + C::OFF_OUT + ((warp - 4) ^ 4) * C::OUT_WARP + at)));
                if (g == 0 && m < p.M) p.scales[(int64_t)nt * p.M + m] = q.scale;
                // rows of 64 bytes, in the order of the 64-byte swizzle (plain rows share banks: 289 -> 284 us for 4096 x
                // 11008 x 4096)
#pragma unroll
                for (int c = 0; c < 64; c += 16) {
                    uint32_t o[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float* a = acc + c + 4 * j;
                        o[j] = q.codes(a[0], a[1], a[2], a[3]);
                    }
                    *reinterpret_cast<uint4*>(out_s + lane * 64 + (c ^ ((lane >> 1 & 3) << 4))) = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && any) {
                const int y = (int)(m - lane);
                ptx::tma_store_2d(&p.tmap_out, ptx::smem_u32(out_s), (int)n0, y);
                if (!GATED && n0 + 64 < p.N) ptx::tma_store_2d(&p.tmap_out, ptx::smem_u32(out_s) + 4096, (int)n0 + 64, y);
                ptx::bulk_commit_group();
            }
        }
        if (lane == 0) ptx::bulk_wait_group0();
        __syncwarp();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();      // neither block leaves, or frees tensor memory, while the other may need it
    ptx::tc_fence_after();
    if (warp == 2) ptx::tmem_dealloc<2>(tmem, 512);
}

}  // namespace wq
