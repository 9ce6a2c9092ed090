// wq_w8a8_narrow.cuh -- product of e4m3 activations and e4m3 weights for few tokens: weight rows are the
// tensor cores' M dimension, tokens the N dimension.
//
//   acc[n][m] += (a_scale[kb][m] w_scale[n / 128][kb]) * D_kb[n][m],   D_kb = the tensor cores' sum over block kb
//
// D_kb of 128 k is one accumulation in tensor memory (four products of 32 k); the scales differ from block to
// block and are any fp32 number, so each block's sum is read back, scaled and added in registers, from one of
// two buffers while the tensor cores fill the other.  A tile is 128 weight rows, one block of scales, so a
// row's factor is its token's scale times one number.  GATED: 128 rows of the gate and the 128 rows of up with
// the same numbers, each with its own accumulator: silu(gate) * up then needs no exchange between threads, and
// the 128 rows are the output's block.
//
// Few tokens are bound by reading the weights: `splits` blocks of threads, one cluster, share a tile's k, so that
// the grid fills the GPU.  Each then sends its sums to the owners of the columns (tokens in groups of four) by
// st.async; an owner adds the slices in order and finishes its tokens for all 128 rows.
#pragma once

#include "wq_common.cuh"
#include "wq_fp8.cuh"

namespace wq {

template <int BN_, bool GATED_, int STAGES_, int SMAX_, int CTAS_>
struct NarrowCfg {
    static constexpr int BN = BN_, STAGES = STAGES_, SMAX = SMAX_, CTAS = CTAS_;
    static constexpr bool GATED = GATED_;
    static constexpr int H = GATED ? 2 : 1;
    static constexpr int NTHREADS = 224;                    // warps 0-3 sums, 4 copies, 5 products, 6 scales
    static constexpr int W_TILE = 128 * 128;
    static constexpr int STAGE = H * W_TILE + BN * 128;     // weight tiles, then the tokens' rows
    static constexpr int SCN = 8;                           // slots of scales: BN tokens', then the weights'
    static constexpr int SC_SLOT = (BN + 4) * 4;
    static constexpr int OFF_SC = STAGES * STAGE;
    static constexpr int OFF_INBOX = OFF_SC + SCN * SC_SLOT;
    static constexpr int INBOX = SMAX > 1 ? (BN / 4 + SMAX - 1) * 128 * 16 * H : 0;
    static constexpr int OFF_MOST = OFF_INBOX + INBOX;      // largest magnitudes [4 warps][BN]
    static constexpr int OFF_BAR = OFF_MOST + (GATED ? 4 * BN * 4 : 0);
    // barriers: full, empty (stages), acc full, acc empty (2), scales full, empty, inbox, final; then TMEM address, abort
    static constexpr int NBAR = 2 * STAGES + 4 + 2 * SCN + 2;
    static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;
    static constexpr int SMEM = OFF_MISC + 16 + 1024;
    static constexpr int TMEM_COLS = 2 * H * BN < 32 ? 32 : 2 * H * BN;
    static_assert(STAGE % 1024 == 0 && OFF_INBOX % 16 == 0 && OFF_BAR % 8 == 0, "alignment");
    static_assert(TMEM_COLS * CTAS <= 512 && SMEM <= (CTAS == 1 ? 232448 : 115712), "resident blocks");
};

template <typename C>
__global__ void __launch_bounds__(C::NTHREADS, C::CTAS) w8a8_narrow_kernel(const __grid_constant__ W8A8Params p) {
    constexpr int BN = C::BN, H = C::H, STAGES = C::STAGES, SCN = C::SCN;
    constexpr bool GATED = C::GATED;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = ptx::smem_u32(smem);
    const uint32_t bar0 = sbase + C::OFF_BAR;
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (STAGES + s); };
    auto acc_full = [&](int b) { return bar0 + 8u * (2 * STAGES + b); };
    auto acc_empty = [&](int b) { return bar0 + 8u * (2 * STAGES + 2 + b); };
    auto sc_full = [&](int s) { return bar0 + 8u * (2 * STAGES + 4 + s); };
    auto sc_empty = [&](int s) { return bar0 + 8u * (2 * STAGES + 4 + SCN + s); };
    const uint32_t inbox_bar = bar0 + 8u * (2 * STAGES + 4 + 2 * SCN), final_bar = inbox_bar + 8u;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const int S = p.splits;
    const int rank = S > 1 ? (int)ptx::cluster_ctarank() : 0;
    const int tile = (int)blockIdx.x / S;
    const int nt = tile / p.tiles_m, mt = tile - nt * p.tiles_m;      // a weight tile's token tiles are neighbours
    const int64_t m0 = (int64_t)mt * BN;
    const int cols = (int)min((int64_t)BN, p.M - m0);
    const int kb0 = (int)((int64_t)p.kblocks * rank / S), n_kb = (int)((int64_t)p.kblocks * (rank + 1) / S) - kb0;
    // columns in groups of four: this block finishes groups [g0, g0 + own)
    const int groups = (cols + 3) / 4, per = S > 1 ? (groups + S - 1) / S : BN / 4;
    const int g0 = S > 1 ? rank * per : 0, own = max(0, min(per, groups - g0));

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) ptx::mbar_init(full(s), 1), ptx::mbar_init(empty(s), 1);
        for (int b = 0; b < 2; ++b) ptx::mbar_init(acc_full(b), 1), ptx::mbar_init(acc_empty(b), 4);
        for (int s = 0; s < SCN; ++s) ptx::mbar_init(sc_full(s), 32), ptx::mbar_init(sc_empty(s), 4);
        ptx::mbar_init(inbox_bar, 1);
        ptx::mbar_init(final_bar, 1);
        *abort_flag = 0u;
        ptx::fence_barrier_init();
        if (S > 1 && own > 0) ptx::mbar_arrive_expect_tx(inbox_bar, (uint32_t)(S * H * 128 * own * 16));
        ptx::fence_proxy_async_smem();
        ptx::prefetch_tmap(&p.tmap_w);
        ptx::prefetch_tmap(&p.tmap_a);
    }
    if (warp == 5) {
        ptx::tmem_alloc<1>(sbase + C::OFF_MISC, C::TMEM_COLS);
        ptx::tmem_relinquish<1>();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (S > 1) ptx::cluster_arrive_relaxed();
    const uint32_t tmem = *tmem_slot;
    // every input may come from the kernel before this one
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();

    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity, uint32_t code) {
        if (ok) ok = bounded_wait(bar, parity, abort_flag, p.status, code, p.timeout_ns);
        return ok;
    };
    float acc[H * BN];
#pragma unroll
    for (int i = 0; i < H * BN; ++i) acc[i] = 0.f;

    if (warp == 4) {
        // ------------------------------------------------------------ copies
        if (lane == 0) {
            const uint64_t pol_w = p.tiles_m == 1 ? ptx::policy_evict_first() : ptx::policy_evict_last();
            const uint64_t pol_a = ptx::policy_evict_last();
            const uint32_t bytes = (uint32_t)(H * C::W_TILE + p.box_m * 128);
            int i = 0, s = 0;
            uint32_t ph = 0;
            for (; i < n_kb && wait(empty(s), ph ^ 1u, DEVICE_TIMEOUT_PRODUCER); ++i) {
                const uint32_t dst = sbase + s * C::STAGE;
                ptx::mbar_arrive_expect_tx(full(s), bytes);
#pragma unroll
                for (int h = 0; h < H; ++h)
                    ptx::tma_load_3d(dst + h * C::W_TILE, &p.tmap_w, (kb0 + i) * 128, nt * 128, h, full(s), pol_w);
                ptx::tma_load_2d(dst + H * C::W_TILE, &p.tmap_a, (kb0 + i) * 128, (int)m0, full(s), pol_a);
                if (++s == STAGES) s = 0, ph ^= 1u;
            }
            // every stage released: the commits that arrive here have all landed
            for (int j = 0; j < STAGES && wait(empty(s), ph ^ 1u, DEVICE_TIMEOUT_PRODUCER); ++j)
                if (++s == STAGES) s = 0, ph ^= 1u;
            if (!ok)   // copies in flight land before the block ends
                for (int j = max(0, i - STAGES); j < i; ++j)
                    if (!drain_wait(full(j % STAGES), (uint32_t)(j / STAGES) & 1u, p.timeout_ns))
                        atomicOr(p.status, DEVICE_TIMEOUT_DRAIN);
        }
        __syncwarp();
    } else if (warp == 5) {
        // ------------------------------------------------------------ products
        if (lane == 0) {
            constexpr uint32_t idesc = ptx::make_idesc_e4m3(128, BN);
            int s = 0;
            uint32_t ph = 0;
            for (int i = 0; i < n_kb; ++i) {
                const int b = i & 1;
                if (!wait(acc_empty(b), ((uint32_t)(i >> 1) & 1u) ^ 1u, DEVICE_TIMEOUT_MMA) ||
                    !wait(full(s), ph, DEVICE_TIMEOUT_MMA))
                    break;
                ptx::tc_fence_after();
                const uint32_t w_lo = ptx::sdesc_lo(sbase + s * C::STAGE);
                const uint32_t t_lo = ptx::sdesc_lo(sbase + s * C::STAGE + H * C::W_TILE);
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int h = 0; h < H; ++h)
                        ptx::mma_f8_ss<1>(tmem + (b * H + h) * BN, w_lo + h * (C::W_TILE >> 4) + 2 * k, ptx::kSdescHi,
                                          t_lo + 2 * k, ptx::kSdescHi, idesc, k > 0);
                ptx::mma_commit<1>(acc_full(b));
                ptx::mma_commit<1>(empty(s));
                if (++s == STAGES) s = 0, ph ^= 1u;
            }
            if (!ok) {
                ptx::mma_commit<1>(final_bar);
                if (!drain_wait(final_bar, 0, p.timeout_ns)) atomicOr(p.status, DEVICE_TIMEOUT_DRAIN);
            }
        }
        __syncwarp();
    } else if (warp == 6) {
        // ------------------------------------------------------------ scales
        const int64_t wblocks = ((p.N + 127) >> 7) * p.kblocks;
        const float* sw = p.w_scale + (int64_t)nt * p.kblocks + kb0 + (lane < H ? lane * wblocks : 0);
        const float* sa = p.a_scale + (int64_t)kb0 * p.M + m0;
        for (int i = 0; i < n_kb; ++i) {
            const int s = i % SCN;
            if (!__all_sync(0xffffffffu, wait(sc_empty(s), ((uint32_t)(i / SCN) & 1u) ^ 1u, DEVICE_TIMEOUT_PRODUCER))) break;
            const uint32_t dst = sbase + C::OFF_SC + s * C::SC_SLOT;
#pragma unroll
            for (int c = lane; c < BN; c += 32) ptx::cp_async4(dst + 4 * c, sa + (c < cols ? c : 0), c < cols);
            if (lane < H) ptx::cp_async4(dst + 4 * (BN + lane), sw + i, true);
            ptx::cp_async_arrive(sc_full(s));
            sa += p.M;
        }
        ptx::cp_async_wait_all();
    } else {
        // ------------------------------------------------------------ sums
        constexpr int CH = BN * H >= 32 ? 32 : 16, NC = BN * H / CH;
        const uint32_t base = tmem + ((uint32_t)(warp * 32) << 16);
        for (int i = 0; i < n_kb; ++i) {
            const int b = i & 1, s = i % SCN;
            wait(sc_full(s), (uint32_t)(i / SCN) & 1u, DEVICE_TIMEOUT_TRANSFORM);
            if (!__all_sync(0xffffffffu, wait(acc_full(b), (uint32_t)(i >> 1) & 1u, DEVICE_TIMEOUT_TRANSFORM))) break;
            ptx::tc_fence_after();
            const float* sc = reinterpret_cast<const float*>(smem + C::OFF_SC + s * C::SC_SLOT);
            uint64_t sw[H];
#pragma unroll
            for (int h = 0; h < H; ++h) sw[h] = f2(sc[BN + h], sc[BN + h]);
            uint32_t v[2][CH];
            auto load = [&](int c) {
                if constexpr (CH == 32) ptx::tmem_ld32(base + b * H * BN + c * CH, v[c & 1]);
                else ptx::tmem_ld16(base + b * H * BN + c * CH, v[c & 1]);
            };
            load(0);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                ptx::tmem_wait_ld_of(v[c & 1]);
                if (c + 1 < NC) {
                    load(c + 1);
                } else {
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(acc_empty(b));
                }
#pragma unroll
                for (int j = 0; j < CH; j += 4) {
                    const int col = c * CH + j, h = col / BN;
                    const float4 t = *reinterpret_cast<const float4*>(sc + col % BN);
                    const uint64_t s01 = mul_f2(f2(t.x, t.y), sw[h]), s23 = mul_f2(f2(t.z, t.w), sw[h]);
                    const uint32_t* d = v[c & 1] + j;
                    const float2 r01 = un2(fma_f2(f2(__uint_as_float(d[0]), __uint_as_float(d[1])), s01, f2(acc[col], acc[col + 1])));
                    const float2 r23 = un2(fma_f2(f2(__uint_as_float(d[2]), __uint_as_float(d[3])), s23, f2(acc[col + 2], acc[col + 3])));
                    acc[col] = r01.x, acc[col + 1] = r01.y, acc[col + 2] = r23.x, acc[col + 3] = r23.y;
                }
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(sc_empty(s));
        }
    }
    // From here on every thread runs the same sequence (no early exit before the barriers).
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 5) ptx::tmem_dealloc<1>(tmem, C::TMEM_COLS);
    if (S > 1) ptx::cluster_wait();   // every block of the cluster has initialised its barriers
    if (warp >= 4) return;
    ok = *abort_flag == 0u;
    const int row = threadIdx.x;      // of the tile
    if (C::SMAX > 1 && S > 1) {
        if (ok) {
#pragma unroll
            for (int j = 0; j < BN / 4; ++j) {
                if (j < groups) {
                    const int owner = j / per;
                    const uint32_t bar = ptx::mapa_shared(inbox_bar, (uint32_t)owner);
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        const uint32_t at = sbase + C::OFF_INBOX + (uint32_t)(((rank * H + h) * 128 + row) * per + j - owner * per) * 16u;
                        const float* a = acc + h * BN + 4 * j;
                        ptx::st_async_v4f32(ptx::mapa_shared(at, (uint32_t)owner), a[0], a[1], a[2], a[3], bar);
                    }
                }
            }
        }
        if (own == 0) return;
        ok = ok && bounded_wait<true>(inbox_bar, 0u, abort_flag, p.status, DEVICE_TIMEOUT_EPILOGUE, p.timeout_ns);
#pragma unroll
        for (int j = 0; j < BN / 4; ++j) {
            if (j < own && ok) {
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int q = 0; q < S; ++q) {
                        const float4 u = *reinterpret_cast<const float4*>(
                            smem + C::OFF_INBOX + (((q * H + h) * 128 + row) * per + j) * 16);
                        t.x += u.x, t.y += u.y, t.z += u.z, t.w += u.w;
                    }
                    float* a = acc + h * BN + 4 * j;
                    a[0] = t.x, a[1] = t.y, a[2] = t.z, a[3] = t.w;
                }
            }
        }
    }
    // ---- the tokens m_first .. of this block, all rows of the tile
    const int64_t m_first = m0 + 4 * g0;
    const int mine = (int)min((int64_t)(4 * own), p.M - m_first);
    const int64_t n = (int64_t)nt * 128 + row;
    if (GATED) {
#pragma unroll
        for (int c = 0; c < BN; ++c) acc[c] = silu(acc[c]) * acc[(H - 1) * BN + c];
    }
    if (p.out != nullptr) {
        if (ok && n < p.N) {
            const float bias = !GATED && p.bias != nullptr
                                   ? (p.out_bf16 ? load_16bit<true>(p.bias, (size_t)n) : load_16bit<false>(p.bias, (size_t)n))
                                   : 0.f;
            uint16_t* out = static_cast<uint16_t*>(p.out) + m_first * p.N + n;
#pragma unroll
            for (int c = 0; c < BN; ++c)
                if (c < mine) out[c * p.N] = p.out_bf16 ? to_16bit<true>(acc[c] + bias) : to_16bit<false>(acc[c] + bias);
        }
        return;
    }
    if constexpr (GATED) {
        float* most = reinterpret_cast<float*>(smem + C::OFF_MOST);
#pragma unroll
        for (int c = 0; c < BN; ++c) {
            if (c < mine) {
                const float m = warp_most(n < p.N ? acc[c] : 0.f);
                if (lane == 0) most[warp * BN + c] = m;
            }
        }
        ptx::named_barrier_sync(1, 128);
        // codes [token][row] through the (free) stages, so that a token's 128 leave together
        uint8_t* stage = smem;
#pragma unroll
        for (int c = 0; c < BN; ++c) {
            if (c < mine) {
                const BlockScale q(max_nan(max_nan(most[c], most[BN + c]), max_nan(most[2 * BN + c], most[3 * BN + c])));
                stage[c * 128 + row] = q.inv == 0.f ? 0 : (uint8_t)to_e4m3x4(acc[c] * q.inv, 0.f, 0.f, 0.f);
                if (row == 0 && ok) p.scales[(int64_t)nt * p.M + m_first + c] = q.scale;
            }
        }
        ptx::named_barrier_sync(1, 128);
        for (int e = row; e < mine * 8 && ok; e += 128) {
            const int64_t at = (int64_t)nt * 128 + 16 * (e & 7);
            if (at < p.N)
                *reinterpret_cast<uint4*>(p.codes + (m_first + (e >> 3)) * p.N + at) = *reinterpret_cast<const uint4*>(stage + 16 * e);
        }
    }
}

}  // namespace wq
