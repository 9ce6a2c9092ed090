// wq_w8a8_narrow.cuh -- product of e4m3 activations and e4m3 weights for up to 32 tokens, which are one tile: weight rows
// are the tensor cores' M dimension, tokens the N dimension.
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
// the grid fills the GPU.  Each then lays its sums out in shared memory and sends each owner of columns (tokens in
// groups of four) its part in one copy; an owner adds the slices in order and finishes its tokens for all 128 rows.
// (16-byte stores that each count on the owner's barrier took longer than the products.)
#pragma once

#include "wq_common.cuh"
#include "wq_fp8.cuh"

namespace wq {

// ALIAS: the slices' sums arrive in the stages' memory as well, behind one more cluster barrier.
template <int BN_, bool GATED_, int STAGES_, int SMAX_, int CTAS_, bool ALIAS_>
struct NarrowCfg {
    static constexpr int BN = BN_, STAGES = STAGES_, SMAX = SMAX_, CTAS = CTAS_;
    static constexpr bool GATED = GATED_, ALIAS = ALIAS_;
    static constexpr int H = GATED ? 2 : 1;
    static constexpr int NTHREADS = 256;                    // warps 0-3 sums, 4 copies, 5 and 6 products, 7 scales
    static constexpr int W_TILE = 128 * 128;
    static constexpr int STAGE = H * W_TILE + BN * 128;     // weight tiles, then the tokens' rows
    // Scales of a block of K: BN tokens', then the weights'.  They are part of the block's stage (its products wait
    // for them too).  A slot is filled again SCN blocks on, when the products of STAGES blocks before that have ended,
    // for which the sums two blocks earlier had to be released, and those of the block before that were finished with:
    // nobody reads it any more.
    static constexpr int SCN = 8;
    static constexpr int SC_SLOT = (BN + 4) * 4;
    static constexpr int OFF_SC = STAGES * STAGE;
    static constexpr int INBOX = (BN / 4 + SMAX - 1) * 128 * 16 * H;
    static constexpr int OUTBOX = BN / 4 * 128 * 16 * H;      // in the stages
    static constexpr int OFF_INBOX = ALIAS ? OUTBOX : OFF_SC + SCN * SC_SLOT;
    static constexpr int OFF_MOST = OFF_SC + SCN * SC_SLOT + (ALIAS ? 0 : INBOX);      // largest magnitudes [4 warps][BN]
    static constexpr int OFF_BAR = OFF_MOST + (GATED ? 4 * BN * 4 : 0);
    // barriers: full, empty (stages), acc full, acc empty (2), inbox, final; then TMEM address, abort
    static constexpr int NBAR = 2 * STAGES + 4 + 3;
    static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;
    static constexpr int SMEM = OFF_MISC + 16 + 1024;
    static constexpr int TMEM_COLS = 2 * H * BN < 32 ? 32 : 2 * H * BN;
    static_assert(SCN >= STAGES + 3 && OUTBOX + (ALIAS ? INBOX : 0) <= STAGES * STAGE, "scales, inbox");
    static_assert(STAGE % 1024 == 0 && OFF_INBOX % 16 == 0 && OFF_BAR % 8 == 0, "alignment");
    static_assert(TMEM_COLS * CTAS <= 512 && CTAS * (SMEM + 1024) <= 233472, "resident blocks");
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
    const uint32_t inbox_bar = bar0 + 8u * (2 * STAGES + 4), final_bar = inbox_bar + 8u;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    volatile uint32_t* lost = tmem_slot + 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const int S = p.splits;
    const int rank = S > 1 ? (int)ptx::cluster_ctarank() : 0;
    const int nt = (int)blockIdx.x / S, cols = (int)p.M;
    const int kb0 = (int)((int64_t)p.kblocks * rank / S), n_kb = (int)((int64_t)p.kblocks * (rank + 1) / S) - kb0;
    // columns in groups of four: this block finishes groups [g0, g0 + own)
    const int groups = (cols + 3) / 4, per = S > 1 ? (groups + S - 1) / S : BN / 4;
    const int g0 = S > 1 ? rank * per : 0, own = max(0, min(per, groups - g0));

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) ptx::mbar_init(full(s), 33), ptx::mbar_init(empty(s), 1);
        for (int b = 0; b < 2; ++b) ptx::mbar_init(acc_full(b), 1), ptx::mbar_init(acc_empty(b), 4);
        ptx::mbar_init(inbox_bar, 1);
        ptx::mbar_init(final_bar, 1), ptx::mbar_init(final_bar + 8u, 1);
        *abort_flag = 0u;
        *lost = 0u;
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
    // every input may come from the kernel before this one; the first weights are on their way to L2 meanwhile
    if (warp == 4 && lane < min(n_kb, STAGES)) {
#pragma unroll
        for (int h = 0; h < H; ++h) ptx::tma_prefetch_3d(&p.tmap_w, (kb0 + lane) * 128, nt * 128, h);
    }
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();

    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity, uint32_t code) {
        if (ok) ok = bounded_wait(bar, parity, abort_flag, p.status, code, p.timeout_ns);
        return ok;
    };
    auto wait_all = [&](uint32_t bar, uint32_t parity, uint32_t code) {      // a warp's lanes together
        return ok = warp_wait(ok, bar, parity, abort_flag, p.status, code, p.timeout_ns);
    };
    float acc[H * BN];
#pragma unroll
    for (int i = 0; i < H * BN; ++i) acc[i] = 0.f;

    if (warp == 4) {
        // ------------------------------------------------------------ copies
        if (lane == 0) {
            const uint64_t pol_w = ptx::policy_evict_first();
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
                ptx::tma_load_2d(dst + H * C::W_TILE, &p.tmap_a, (kb0 + i) * 128, 0, full(s), pol_a);
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
    } else if (warp == 7) {
        // ------------------------------------------------------------ scales
        const int64_t wblocks = ((p.N + 127) >> 7) * p.kblocks;
        const float* sw = p.w_scale + (int64_t)nt * p.kblocks + kb0 + (lane < H ? lane * wblocks : 0);
        const float* sa = p.a_scale + (int64_t)kb0 * p.M;
        int s = 0;
        uint32_t ph = 0;
        for (int i = 0; i < n_kb && wait_all(empty(s), ph ^ 1u, DEVICE_TIMEOUT_PRODUCER); ++i) {
            const uint32_t sc = sbase + C::OFF_SC + i % SCN * C::SC_SLOT;
#pragma unroll
            for (int c = lane; c < BN; c += 32) ptx::cp_async4(sc + 4 * c, sa + (c < cols ? c : 0), c < cols);
            if (lane < H) ptx::cp_async4(sc + 4 * (BN + lane), sw + i, true);
            ptx::cp_async_arrive(full(s));
            sa += p.M;
            if (++s == STAGES) s = 0, ph ^= 1u;
        }
        ptx::cp_async_wait_all();
    } else if (warp >= 5) {
        // ------------------------------------------------------------ products
        if (lane == 0) {
            // Two warps issue in turn, each for one buffer of sums: a block's waits, commits and loop (some 250 cycles)
            // then lie beside the other warp's products, which the tensor cores only take as fast as they work.
            constexpr uint32_t idesc = ptx::make_idesc_e4m3(128, BN);
            const int b = warp - 5;
            int s = b;
            uint32_t ph = 0;
            for (int i = b; i < n_kb; i += 2) {
                if (!wait(acc_empty(b), ((uint32_t)(i >> 1) & 1u) ^ 1u, DEVICE_TIMEOUT_MMA) || !wait(full(s), ph, DEVICE_TIMEOUT_MMA))
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
                if ((s += 2) >= STAGES) s -= STAGES, ph ^= 1u;
            }
            if (!ok) {
                ptx::mma_commit<1>(final_bar + 8u * b);
                if (!drain_wait(final_bar + 8u * b, 0, p.timeout_ns)) atomicOr(p.status, DEVICE_TIMEOUT_DRAIN);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ sums
        constexpr int CH = BN * H == 16 ? 16 : 32, NC = BN * H / CH;
        const uint32_t base = tmem + ((uint32_t)(warp * 32) << 16);
        for (int i = 0; i < n_kb; ++i) {
            const int b = i & 1;
            if (!wait_all(acc_full(b), (uint32_t)(i >> 1) & 1u, DEVICE_TIMEOUT_TRANSFORM)) break;
            ptx::tc_fence_after();
            uint32_t v[2][CH];
            auto load = [&](int c) { ptx::tmem_ld(base + b * H * BN + c * CH, v[c & 1]); };
            const float* sc = reinterpret_cast<const float*>(smem + C::OFF_SC + i % SCN * C::SC_SLOT);
            uint64_t sw[H];
#pragma unroll
            for (int h = 0; h < H; ++h) sw[h] = f2(sc[BN + h], sc[BN + h]);
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
        }
    }
    // From here on every thread runs the same sequence (no early exit before the barriers).
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 5) ptx::tmem_dealloc<1>(tmem, C::TMEM_COLS);
    if (S > 1) ptx::cluster_wait();   // every block of the cluster has initialised its barriers
    if (C::ALIAS && S > 1) ptx::cluster_sync();   // and has read its stages
    if (warp >= 4) {
        if (S > 1) ptx::cluster_arrive_relaxed(), ptx::cluster_wait();   // (the barrier behind the exchange)
        return;
    }
    ok = __all_sync(0xffffffffu, *abort_flag == 0u);
    const int row = threadIdx.x;      // of the tile
    // From here on sums lie in shared memory, [part][half][group of columns][row], and are worked on in small loops:
    // code that runs once is bound by its own fetching (unrolled over 128 columns in registers it took four times as long
    // as the loop over 32 blocks of K).
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int j = 0; j < BN / 4; ++j)
            *reinterpret_cast<float4*>(smem + ((h * (BN / 4) + j) * 128 + row) * 16) =
                make_float4(acc[h * BN + 4 * j], acc[h * BN + 4 * j + 1], acc[h * BN + 4 * j + 2], acc[h * BN + 4 * j + 3]);
    if (S > 1) {
        // each owner's groups of columns are one piece for each half
        ptx::fence_proxy_async_smem();
        ptx::named_barrier_sync(1, 128);
        if (ok && threadIdx.x < S) {
            const int owner = threadIdx.x, theirs = min(per, groups - owner * per);
            const uint32_t bar = ptx::mapa_shared(inbox_bar, (uint32_t)owner);
            if (theirs > 0)
#pragma unroll
                for (int h = 0; h < H; ++h)
                    ptx::bulk_send(ptx::mapa_shared(sbase + C::OFF_INBOX + (uint32_t)((rank * H + h) * per * 2048), (uint32_t)owner),
                                   sbase + (uint32_t)((h * (BN / 4) + owner * per) * 2048), (uint32_t)(theirs * 2048), bar);
        }
        __syncwarp();
        if (own > 0) ok = warp_wait<true>(ok, inbox_bar, 0u, abort_flag, p.status, DEVICE_TIMEOUT_EPILOGUE, p.timeout_ns);
        if (!ok) tell_lost(sbase + C::OFF_MISC + 8u, S);
        // Nobody leaves before all have what was sent to them: what they sent has then been read.
        ptx::cluster_arrive_relaxed();
    }
    // ---- the tokens m_first .. of this block, all rows of the tile
    const int64_t m_first = 4 * g0, n = (int64_t)nt * 128 + row;
    const int mine = (int)min((int64_t)(4 * own), p.M - m_first);
    uint8_t* parts = smem + (S > 1 ? C::OFF_INBOX : 0) + row * 16;
    float* most = reinterpret_cast<float*>(smem + C::OFF_MOST);
    const bool codes = GATED && p.out == nullptr;
    const float bias = !GATED && p.bias != nullptr && n < p.N
                           ? (p.out_bf16 ? load_16bit<true>(p.bias, (size_t)n) : load_16bit<false>(p.bias, (size_t)n))
                           : 0.f;
#pragma unroll 1
    for (int j = 0; j < own && ok; ++j) {
        float4 t[H];
#pragma unroll
        for (int h = 0; h < H; ++h) t[h] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
        for (int q = 0; q < S; ++q)
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const float4 u = *reinterpret_cast<const float4*>(parts + ((q * H + h) * per + j) * 2048);
                t[h].x += u.x, t[h].y += u.y, t[h].z += u.z, t[h].w += u.w;
            }
        float v[4] = {t[0].x, t[0].y, t[0].z, t[0].w};
        if constexpr (GATED) {
            v[0] = silu(v[0]) * t[1].x, v[1] = silu(v[1]) * t[1].y, v[2] = silu(v[2]) * t[1].z, v[3] = silu(v[3]) * t[1].w;
        }
        if (codes) {
            *reinterpret_cast<float4*>(parts + j * 2048) = make_float4(v[0], v[1], v[2], v[3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float m = warp_most(n < p.N ? v[e] : 0.f);
                if (lane == 0) most[warp * BN + 4 * j + e] = m;
            }
        } else if (n < p.N) {
            uint16_t* out = static_cast<uint16_t*>(p.out) + (m_first + 4 * j) * p.N + n;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (4 * j + e < mine)
                    out[e * p.N] = p.out_bf16 ? to_16bit<true>(v[e] + bias) : to_16bit<false>(v[e] + bias);
        }
    }
    if (codes) {
        ptx::named_barrier_sync(1, 128);
        ok = __all_sync(0xffffffffu, ok && *abort_flag == 0u);     // (another warp may not have its largest magnitudes)
#pragma unroll 1
        for (int j = 0; j < own && ok; ++j) {
            const float4 t = *reinterpret_cast<const float4*>(parts + j * 2048);
            const float v[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int c = 4 * j + e;
                if (c < mine) {
                    const BlockScale q(max_nan(max_nan(most[c], most[BN + c]), max_nan(most[2 * BN + c], most[3 * BN + c])));
                    if (n < p.N)
                        p.codes[(m_first + c) * p.N + n] = q.code(v[e]);
                    if (row == 0) p.scales[(int64_t)nt * p.M + m_first + c] = q.scale;
                }
            }
        }
    }
    if (S > 1) {
        __syncwarp();
        ptx::cluster_wait();
        land_lost(lost, own > 0, inbox_bar, p.timeout_ns);
    }
}

}  // namespace wq
