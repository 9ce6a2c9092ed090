// wq_w8a8_mid.cuh -- product of e4m3 activations and e4m3 weights for some tokens (a draft batch, a short prompt):
// tokens are the tensor cores' M dimension as in wq_w8a8_wide.cuh, but a tile is one block of threads' own:
// 128 tokens x 128 weight rows (GATED: 128 of the gate and the same 128 of up), and `splits` blocks, one cluster,
// may share its k.  The sums then go through shared memory: a warp finishes a token's 128 columns, so that stores
// are whole lines and the largest of a block of 128 needs no exchange.
#pragma once

#include "wq_common.cuh"
#include "wq_fp8.cuh"

namespace wq {

template <bool GATED_>
struct MidCfg {
    static constexpr bool GATED = GATED_;
    static constexpr int H = GATED ? 2 : 1;
    static constexpr int NTHREADS = 384;                    // warp 0 copies, 1 and 3 products, 2 tensor memory and scales, 4-11 sums
    static constexpr int SMAX = GATED ? 1 : 8;              // (both halves' sums of two slices do not fit)
    static constexpr int N = 128 * H;                       // weight rows of a tile
    static constexpr int CT = N / 2;                        // columns of a thread
    static constexpr int STAGE = 128 * 128 + N * 128;
    static constexpr int STAGES = GATED ? 4 : 6;
    static constexpr int SCN = 8;                           // slots of scales, as in wq_w8a8_wide.cuh
    static constexpr int SC_SLOT = 130 * 4 + 8;
    static constexpr int OFF_SC = STAGES * STAGE;
    // sums in shared memory, over the stages: [group of four columns][row], an odd number of rows apart
    static constexpr int NG = N / 4, PITCH = 129;
    static constexpr int OUTBOX = NG * PITCH * 16;
    static constexpr int INBOX = SMAX > 1 ? NG * (128 + 2 * SMAX) * 16 : 0;
    static constexpr int OFF_BAR = OFF_SC + SCN * SC_SLOT;
    static constexpr int NBAR = 2 * STAGES + 4 + 3;         // full, empty, acc full / empty (2), inbox, final
    static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;
    static constexpr int SMEM = OFF_MISC + 16 + 1024;
    static constexpr int TMEM_COLS = 2 * N;
    static constexpr int REGS_ISSUE = 72, REGS_SUM = 216;   // 168 x 384 at launch = 72 x 128 + 216 x 256
    static_assert(SMEM <= 232448 && OUTBOX + INBOX <= STAGES * STAGE, "shared memory");
    static_assert(SCN >= STAGES + 2 && OFF_BAR % 8 == 0, "scales");
};

template <typename C>
__global__ void __launch_bounds__(C::NTHREADS, 1) w8a8_mid_kernel(const __grid_constant__ W8A8Params p) {
    constexpr int STAGES = C::STAGES, H = C::H, SCN = C::SCN, CT = C::CT, NG = C::NG;
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
    const int tile = (int)blockIdx.x / S;
    const int nt = tile / p.tiles_m, mt = tile - nt * p.tiles_m;      // a weight tile's token tiles are neighbours
    const int64_t m0 = (int64_t)mt * 128;
    const int rows = (int)min((int64_t)128, p.M - m0);
    const int kb0 = (int)((int64_t)p.kblocks * rank / S), n_kb = (int)((int64_t)p.kblocks * (rank + 1) / S) - kb0;
    // this block finishes rows [r0, r0 + own) of the tile
    const int per = (rows + S - 1) / S, r0 = rank * per, own = max(0, min(per, rows - r0));

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) ptx::mbar_init(full(s), 33), ptx::mbar_init(empty(s), 1);
        for (int b = 0; b < 2; ++b) ptx::mbar_init(acc_full(b), 1), ptx::mbar_init(acc_empty(b), 8);
        ptx::mbar_init(inbox_bar, 1);
        ptx::mbar_init(final_bar, 1), ptx::mbar_init(final_bar + 8u, 1);
        *abort_flag = 0u;
        *lost = 0u;
        ptx::fence_barrier_init();
        if (S > 1 && own > 0) ptx::mbar_arrive_expect_tx(inbox_bar, (uint32_t)(S * NG * own * 16));
        ptx::fence_proxy_async_smem();
        ptx::prefetch_tmap(&p.tmap_w);
        ptx::prefetch_tmap(&p.tmap_a);
    }
    if (warp == 2) {
        ptx::tmem_alloc<1>(sbase + C::OFF_MISC, C::TMEM_COLS);
        ptx::tmem_relinquish<1>();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (S > 1) ptx::cluster_arrive_relaxed();
    const uint32_t tmem = *tmem_slot;
    // the 64 weight rows of part i of a tile: rows of the tile in turn, or of the gate and of up in turn
    auto w_row = [&](int i) { return nt * 128 + 64 * (GATED ? i >> 1 : i); };
    auto w_half = [&](int i) { return GATED ? i & 1 : 0; };
    // every input may come from the kernel before this one; the first weights are on their way to L2 meanwhile
    if (warp == 0 && lane < min(n_kb, STAGES)) {
#pragma unroll
        for (int i = 0; i < C::N / 64; ++i) ptx::tma_prefetch_3d(&p.tmap_w, (kb0 + lane) * 128, w_row(i), w_half(i));
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

    if (warp < 4) {
        ptx::regs_dec<C::REGS_ISSUE>();
        if (warp == 0 && lane == 0) {
            // -------------------------------------------------------- copies
            const uint64_t pol_w = p.tiles_m == 1 ? ptx::policy_evict_first() : ptx::policy_evict_last();
            const uint64_t pol_a = ptx::policy_evict_last();
            const uint32_t bytes = (uint32_t)(C::N * 128 + p.box_m * 128);
            int i = 0, s = 0;
            uint32_t ph = 0;
            for (; i < n_kb && wait(empty(s), ph ^ 1u, DEVICE_TIMEOUT_PRODUCER); ++i) {
                const uint32_t dst = sbase + s * C::STAGE;
                ptx::mbar_arrive_expect_tx(full(s), bytes);
#pragma unroll
                for (int j = 0; j < C::N / 64; ++j)
                    ptx::tma_load_3d(dst + 16384 + j * 8192, &p.tmap_w, (kb0 + i) * 128, w_row(j), w_half(j), full(s), pol_w);
                ptx::tma_load_2d(dst, &p.tmap_a, (kb0 + i) * 128, (int)m0, full(s), pol_a);
                if (++s == STAGES) s = 0, ph ^= 1u;
            }
            // every stage released: the commits that arrive here have all landed
            for (int j = 0; j < STAGES && wait(empty(s), ph ^ 1u, DEVICE_TIMEOUT_PRODUCER); ++j)
                if (++s == STAGES) s = 0, ph ^= 1u;
            if (!ok)   // copies in flight land before the block ends
                for (int j = max(0, i - STAGES); j < i; ++j)
                    if (!drain_wait(full(j % STAGES), (uint32_t)(j / STAGES) & 1u, p.timeout_ns))
                        atomicOr(p.status, DEVICE_TIMEOUT_DRAIN);
        } else if (warp == 2) {
            // -------------------------------------------------------- scales
            const int64_t wblocks = ((p.N + 127) >> 7) * p.kblocks;
            const float* sw = p.w_scale + (int64_t)nt * p.kblocks + kb0 + (lane < H ? lane * wblocks : 0);
            const float* sa = p.a_scale + (int64_t)kb0 * p.M + m0;
            int s = 0;
            uint32_t ph = 0;
            for (int i = 0; i < n_kb && wait_all(empty(s), ph ^ 1u, DEVICE_TIMEOUT_PRODUCER); ++i) {
                const uint32_t sc = sbase + C::OFF_SC + i % SCN * C::SC_SLOT;
#pragma unroll
                for (int r = lane; r < 128; r += 32) ptx::cp_async4(sc + 4 * r, sa + (r < rows ? r : 0), r < rows);
                if (lane < H) ptx::cp_async4(sc + 4 * (128 + lane), sw + i, true);
                ptx::cp_async_arrive(full(s));
                sa += p.M;
                if (++s == STAGES) s = 0, ph ^= 1u;
            }
            ptx::cp_async_wait_all();
        } else if ((warp == 1 || warp == 3) && lane == 0) {
            // -------------------------------------------------------- products
            // Two warps issue in turn, each for one buffer of sums: a block's waits, commits and loop (some 250 cycles)
            // then lie beside the other warp's products, which the tensor cores only take as fast as they work.
            constexpr uint32_t idesc = ptx::make_idesc_e4m3(128, C::N);
            const int b = warp >> 1;
            int s = b;
            uint32_t ph = 0;
            for (int i = b; i < n_kb; i += 2) {
                if (!wait(full(s), ph, DEVICE_TIMEOUT_MMA) || !wait(acc_empty(b), ((uint32_t)(i >> 1) & 1u) ^ 1u, DEVICE_TIMEOUT_MMA))
                    break;
                ptx::tc_fence_after();
                const uint32_t a_lo = ptx::sdesc_lo(sbase + s * C::STAGE), b_lo = a_lo + (16384 >> 4);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    ptx::mma_f8_ss<1>(tmem + b * C::N, a_lo + 2 * k, ptx::kSdescHi, b_lo + 2 * k, ptx::kSdescHi, idesc, k > 0);
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
        ptx::regs_inc<C::REGS_SUM>();
        // ------------------------------------------------------------ sums
        const int g = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t base = tmem + ((uint32_t)((warp & 3) * 32) << 16) + g * CT;
        float acc[CT];
#pragma unroll
        for (int i = 0; i < CT; ++i) acc[i] = 0.f;
        for (int i = 0; i < n_kb; ++i) {
            const int b = i & 1;
            if (!wait_all(acc_full(b), (uint32_t)(i >> 1) & 1u, DEVICE_TIMEOUT_TRANSFORM)) break;
            ptx::tc_fence_after();
            uint32_t v[2][16];
            ptx::tmem_ld16(base + b * C::N, v[0]);
            const float* sc = reinterpret_cast<const float*>(smem + C::OFF_SC + i % SCN * C::SC_SLOT);
            uint64_t s[H];
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const float f = sc[row] * sc[128 + h];
                s[h] = f2(f, f);
            }
#pragma unroll
            for (int c = 0; c < CT / 16; ++c) {
                ptx::tmem_wait_ld_of(v[c & 1]);
                if (c + 1 < CT / 16) {
                    ptx::tmem_ld16(base + b * C::N + 16 * (c + 1), v[(c + 1) & 1]);
                } else {
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(acc_empty(b));
                }
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    const int col = 16 * c + j;
                    const float2 r = un2(fma_f2(f2(__uint_as_float(v[c & 1][j]), __uint_as_float(v[c & 1][j + 1])),
                                                s[GATED ? c >> 2 : 0], f2(acc[col], acc[col + 1])));
                    acc[col] = r.x, acc[col + 1] = r.y;
                }
            }
        }
        // The last products have been read, so the stages are free: sums go there.  GATED: gate first, then up.
        __syncwarp();
#pragma unroll
        for (int j = 0; j < CT / 4; ++j) {
            const int group = GATED ? (j >> 4) * 32 + 16 * g + (j & 15) : 16 * g + j;
            *reinterpret_cast<float4*>(smem + (group * C::PITCH + row) * 16) =
                make_float4(acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]);
        }
        ptx::fence_proxy_async_smem();
    }
    // From here on every thread runs the same sequence (no early exit before the barriers).
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 2) ptx::tmem_dealloc<1>(tmem, C::TMEM_COLS);
    if (S > 1) {
        ptx::cluster_wait();      // every block of the cluster has initialised its barriers,
        ptx::cluster_sync();      // and has read its stages
    }
    if (warp < 4) {               // (these warps have given registers away)
        if (S > 1) ptx::cluster_arrive_relaxed(), ptx::cluster_wait();   // the barrier behind the exchange
        return;
    }
    ok = __all_sync(0xffffffffu, *abort_flag == 0u);
    if (S > 1) {
        const int in_pitch = per | 1;
        if (ok)
            for (int e = threadIdx.x - 128; e < NG * S; e += 256) {
                const int group = e % NG, owner = e / NG, theirs = min(per, rows - owner * per);
                if (theirs > 0)
                    ptx::bulk_send(ptx::mapa_shared(sbase + C::OUTBOX + (uint32_t)((rank * NG + group) * in_pitch * 16), (uint32_t)owner),
                                   sbase + (uint32_t)((group * C::PITCH + owner * per) * 16), (uint32_t)(theirs * 16),
                                   ptx::mapa_shared(inbox_bar, (uint32_t)owner));
            }
        __syncwarp();
        if (own > 0) ok = warp_wait<true>(ok, inbox_bar, 0u, abort_flag, p.status, DEVICE_TIMEOUT_EPILOGUE, p.timeout_ns);
        if (!ok) tell_lost(sbase + C::OFF_MISC + 8u, S);
        // Nobody leaves before all have what was sent to them: what they sent has then been read.
        ptx::cluster_arrive_relaxed();
    }
    // ---- a warp for each token: 4 columns for each lane
    const uint8_t* parts = smem + (S > 1 ? C::OUTBOX : 0);
    const int pitch = S > 1 ? per | 1 : C::PITCH;
    const int64_t n = (int64_t)nt * 128 + 4 * lane;
    float bias[4] = {0.f, 0.f, 0.f, 0.f};
    if (!GATED && p.bias != nullptr && n < p.N)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            bias[e] = p.out_bf16 ? load_16bit<true>(p.bias, (size_t)(n + e)) : load_16bit<false>(p.bias, (size_t)(n + e));
#pragma unroll 1
    for (int r = warp - 4; r < own && ok; r += 8) {
        float4 t[H];
#pragma unroll
        for (int h = 0; h < H; ++h) t[h] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
        for (int q = 0; q < S; ++q)
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const float4 u = *reinterpret_cast<const float4*>(parts + ((q * NG + h * 32 + lane) * pitch + r) * 16);
                t[h].x += u.x, t[h].y += u.y, t[h].z += u.z, t[h].w += u.w;
            }
        float v[4] = {t[0].x + bias[0], t[0].y + bias[1], t[0].z + bias[2], t[0].w + bias[3]};
        if constexpr (GATED) {
            v[0] = silu(v[0]) * t[1].x, v[1] = silu(v[1]) * t[1].y, v[2] = silu(v[2]) * t[1].z, v[3] = silu(v[3]) * t[1].w;
        }
        const int64_t m = m0 + r0 + r;
        if (!GATED || p.out != nullptr) {
            if (n < p.N)
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + m * p.N + n) =
                    p.out_bf16 ? make_uint2(pack2<true>(v[0], v[1]), pack2<true>(v[2], v[3]))
                               : make_uint2(pack2<false>(v[0], v[1]), pack2<false>(v[2], v[3]));
        } else {
            // (columns past N are products of zeros)
            const BlockScale q(warp_most(max_nan(max_nan(fabsf(v[0]), fabsf(v[1])), max_nan(fabsf(v[2]), fabsf(v[3])))));
            if (n < p.N)
                *reinterpret_cast<uint32_t*>(p.codes + m * p.N + n) = q.codes(v[0], v[1], v[2], v[3]);
            if (lane == 0) p.scales[(int64_t)nt * p.M + m] = q.scale;
        }
    }
    if (S > 1) {
        __syncwarp();
        ptx::cluster_wait();
        land_lost(lost, own > 0, inbox_bar, p.timeout_ns);
    }
}

}  // namespace wq
