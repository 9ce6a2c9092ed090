// wq_attn_prompt.cuh -- attention of many query rows (prompts and long drafts) over the
// 4-bit cache on the tcgen05 tensor cores.
//
//   S = Q K^T,  P = exp2(scale' S - m),  O += P V,  out = O / sum P
//
// An item is 256 rows (query tokens x heads of a group, so a key head's codes are unpacked
// once for all of them) as two 128-row tiles; cached tokens come in tiles of 64.  Bound by
// the tensor cores and by the softmax between the products (a quarter of the exponentials'
// unit and half of the issue slots).  What keeps them busy: each row tile has two S buffers,
// so its softmax finds the next S ready when it has signalled the last P (with one, product,
// softmax and product followed one another); four slots each of unpacked keys and values;
// and as little as possible between two products.
//   warps 0-3 / 4-7   softmax of row tile 0 / 1, a thread for each row: S from tensor memory,
//                     P back over it.  It runs under the row's maximum so far, and is
//                     repeated under a new one (O rescaled) only where a sum shows that a
//                     score passed that maximum by more than 2^8; at the end O -> out;
//   warps 8-11, 12-15 unpack keys / values: two threads for each token, codes -> RN(lo + q s)
//                     into swizzled shared-memory tiles;
//   warps 16, 17      issue the MMAs of row tile 0 / 1 (PV, then the S after next): the queue
//                     before the tensor core is short, so while one warp waits the other's
//                     products run;
//   warp 18           copies page blocks into a three-stage ring with bulk copies (warp 19
//                     only fills the warpgroup, which hands its registers on).
// Both operand tiles have the same image [D / 64][64 tokens][128 B]: K is read K-major, V
// MN-major, so V is never transposed.  Eight codes of a word land in the order 0 4 1 5 2 6
// 3 7 that the unpack gives; Q is stored in the same order and O is read back through it.
//
// Measured: 4096 queries over 16384 tokens, 32 query and 8 key heads of 128, bf16: 822 us, 1170
// TFLOP/s, the tensor pipe 64% busy.  (Products of 64 columns from shared memory take 48 cycles
// in place of 32, 128 bytes of operands a cycle: 1261 cycles for 64 tokens and 256 rows.)
#pragma once

#include "wq_attn_sched.cuh"
#include "wq_common.cuh"

namespace wq {

constexpr int kPromptTN = 64;
constexpr int kPromptRows = 256;
constexpr int kPromptThreads = 640;
// Registers of a thread by role; a block is launched with 96 for each, and the five
// warpgroups' shares add up to no more than the same 480.
constexpr int kRegsSoftmax = 144, kRegsUnpack = 72, kRegsIssue = 48;
static_assert(2 * kRegsSoftmax + 2 * kRegsUnpack + kRegsIssue <= 5 * 96, "register split");

template <int D>
struct PromptCfg {
    static constexpr int Q_TILE = 128 * D * 2;             // 128 rows of D
    static constexpr int Q_HALF = 128 * 128;               // its part of 64 columns
    static constexpr int KV_TILE = 64 * D * 2;             // 64 tokens of D
    static constexpr int KV_HALF = 64 * 128;
    static constexpr int SLOTS = 4;                        // of keys, and of values
    static constexpr int RAW_STAGES = 3;
    static constexpr int OFF_Q = 0;                        // two row tiles
    static constexpr int OFF_K = OFF_Q + 2 * Q_TILE;
    static constexpr int OFF_V = OFF_K + SLOTS * KV_TILE;
    static constexpr int OFF_BAR = OFF_V + SLOTS * KV_TILE;
    static constexpr int NBARS = 2 * RAW_STAGES + 4 * SLOTS + 17;
    static constexpr int OFF_MISC = OFF_BAR + NBARS * 8;
    static constexpr int OFF_RAW = (OFF_MISC + 16 + 127) / 128 * 128;
    static constexpr int MERGE_ROWS = 32;                  // merge weights live in the Q tiles
    // tensor memory columns
    static constexpr int S_COL = 0, O_COL = 256;           // S_i at 128 i + 64 buffer, O_i at 256 + 128 i; P over S
};

template <bool BF16, int D>
__global__ void __launch_bounds__(kPromptThreads, 1) attn_prompt_kernel(const AttnParams p, const int stage_bytes) {
    using C = PromptCfg<D>;
    constexpr int R = kPromptRows, TN = kPromptTN, KS = D / 16, RS = C::RAW_STAGES, NS = C::SLOTS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = ptx::smem_u32(smem);
    const uint32_t bar0 = sbase + C::OFF_BAR;
    auto raw_full = [&](int i) { return bar0 + 8u * i; };
    auto raw_empty = [&](int i) { return bar0 + 8u * (RS + i); };
    // which: 0 keys, 1 values
    auto kv_full = [&](int which, int i) { return bar0 + 8u * (2 * RS + 2 * NS * which + i); };
    auto kv_empty = [&](int which, int i) { return bar0 + 8u * (2 * RS + 2 * NS * which + NS + i); };
    const uint32_t bar1 = bar0 + 8u * (2 * RS + 4 * NS);
    auto q_full = [&](int i) { return bar1 + 8u * i; };
    auto o_empty = [&](int i) { return bar1 + 8u * (2 + i); };
    // of row tile i and S buffer h
    auto s_full = [&](int i, int h) { return bar1 + 8u * (4 + 2 * i + h); };
    auto p_full = [&](int i, int h) { return bar1 + 8u * (8 + 2 * i + h); };
    // The PV of a tile in buffer h has ended.  One barrier for each buffer: the softmax runs
    // a PV ahead, and on one barrier for all it would take the phase before for the one it
    // waits for (a wait tells phases apart by parity alone).
    auto o_done = [&](int i, int h) { return bar1 + 8u * (12 + 2 * i + h); };
    const uint32_t final_bar = bar1 + 8u * 16;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    volatile int* last_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 8);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < RS; ++i) ptx::mbar_init(raw_full(i), 1), ptx::mbar_init(raw_empty(i), 8);
        for (int i = 0; i < 2 * NS; ++i)
            ptx::mbar_init(kv_full(i / NS, i % NS), 4), ptx::mbar_init(kv_empty(i / NS, i % NS), 2);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(q_full(i), 4);
            ptx::mbar_init(o_empty(i), 4);
            for (int h = 0; h < 2; ++h) {
                ptx::mbar_init(s_full(i, h), 1);
                ptx::mbar_init(p_full(i, h), 4);
                ptx::mbar_init(o_done(i, h), 1);
            }
        }
        ptx::mbar_init(final_bar, 2);
        *abort_flag = 0u;
        ptx::fence_barrier_init();
        ptx::fence_proxy_async_smem();
    }
    if (warp == 16) {
        ptx::tmem_alloc<1>(sbase + C::OFF_MISC, 512);
        ptx::tmem_relinquish<1>();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = 0;   // all 512 columns are allocated: they start at column 0
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();

    Walk w{};
    const Runs runs = walk_begin<R, TN>(p, blockIdx.x, gridDim.x, w);
    const int pair_row = 4 * (D >> p.c.g_shift);
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity, uint32_t code) {
        if (ok) ok = bounded_wait(bar, parity, abort_flag, p.status, code, p.timeout_ns);
        return ok;
    };
    auto item_rows = [&]() { return min(R, w.s.n * p.group - w.rt * R); };
    auto tile_begin = [&]() { return w.v.t0 + (int)(w.u - w.item0); };
    auto tile_end = [&]() { return w.v.t0 + (int)(min(w.item0 + w.units, w.u1) - w.item0); };

    if (warp >= 16) {
    ptx::regs_dec<kRegsIssue>();
    if (warp == 18) {
        // ------------------------------------------------------------ producer
        const uint64_t pol = ptx::policy_evict_last();
        const int vp = min(p.c.P, TN);                          // tokens of a page inside a tile
        const int vblock = vp * (D + 2 * pair_row);
        const bool parted = p.c.P > TN;                         // half of a page of 128: four pieces
        int s = 0;
        uint32_t ph = 0, issued = 0;
        for (; w.u < w.u1 && ok; walk_next<R, TN>(p, w)) {
            if (w.u == w.item0 && lane == 0 && p.lens[w.b] > p.most)
                atomicOr(p.status, DEVICE_INDEX);
            const int te = tile_end();
            for (int t = tile_begin(); t < te; ++t) {
                const int tok = t * TN;
                // the tile's pages that hold a token to be seen: [skip, pages)
                const int pages = min((w.v.hi - tok + vp - 1) / vp, TN / vp);
                const int skip = max(w.v.lo - tok, 0) / vp;
                const bool mine = parted ? (lane < 4 && pages > 0) : (lane >= skip && lane < pages);
                const int64_t page = mine ? safe_page(p, w.b, (tok >> p.c.p_shift) + (parted ? 0 : lane)) : 0;
                ok = __all_sync(0xffffffffu, wait(raw_empty(s), ph ^ 1u, DEVICE_TIMEOUT_PRODUCER));
                if (!ok) break;
                if (lane == 0) {
                    if (pages > skip)
                        ptx::mbar_arrive_expect_tx(raw_full(s), (uint32_t)((pages - skip) * vblock));
                    else
                        ptx::mbar_arrive(raw_full(s));
                }
                __syncwarp();
                const uint32_t dst = sbase + C::OFF_RAW + s * stage_bytes;
                const uint8_t* block = p.c.pages + page * p.c.page_bytes + (int64_t)w.head * p.c.block_bytes;
                if (mine && !parted) ptx::bulk_load(dst + lane * vblock, block, vblock, raw_full(s), pol);
                if (mine && parted) {
                    const int place = tok & (p.c.P - 1), which = lane & 1;
                    if (lane < 2)
                        ptx::bulk_load(dst + which * vp * (D / 2), block + kv4_codes_at(p.c, which, place), vp * (D / 2),
                                       raw_full(s), pol);
                    else
                        ptx::bulk_load(dst + vp * D + which * vp * pair_row, block + kv4_pairs_at(p.c, which, place),
                                       vp * pair_row, raw_full(s), pol);
                }
                issued |= 1u << s;
                if (++s == RS) s = 0, ph ^= 1u;
            }
        }
        // copies in flight land before the block may end: whoever waits for them may have given up
        for (int i = 0; i < RS; ++i)
            if (issued >> i & 1u) drain_wait(raw_full(i), i < s ? ph : ph ^ 1u, p.timeout_ns);
    } else if (warp < 18) {
        // ------------------------------------------------------------ MMA issuers
        // One lane for each row tile, and as few instructions between products as can be: a
        // product of 128 x 128 x 16 takes 64 cycles, a branch in one lane about 30 and a commit
        // about 50, so the steady loop tests its three barriers together, with one branch.  The products of a tile are unrolled with constant
        // offsets, and the whole of tensor memory is ours, so its addresses are constants.
        const int i = warp - 16;
        if (lane == 0) {
            constexpr uint32_t id_s = ptx::make_idesc_f16(BF16, 128, TN);
            constexpr uint32_t id_o = ptx::make_idesc_f16(BF16, 128, D) | ptx::kIdescBTransposed;
            const uint32_t q_lo = ptx::sdesc_lo(sbase + C::OFF_Q + i * C::Q_TILE);
            const uint32_t k_lo = ptx::sdesc_lo(sbase + C::OFF_K), v_lo = ptx::sdesc_lo_mn(sbase + C::OFF_V, C::KV_HALF);
            const uint32_t s_tm = C::S_COL + 128 * i, o_tm = C::O_COL + 128 * i;
            const uint32_t b_q = q_full(i), b_s = s_full(i, 0), b_p = p_full(i, 0), b_od = o_done(i, 0), b_oe = o_empty(i);
            const uint32_t b_kf = kv_full(0, 0), b_ke = kv_empty(0, 0), b_vf = kv_full(1, 0), b_ve = kv_empty(1, 0);
            uint32_t nk = 0, nv = 0;        // tiles of keys and of values so far: slot n % 4, lap n / 4
            uint32_t ns = 0, np = 0;        // S and P of this row tile so far: buffer n % 2
            uint32_t q_ph = 0, o_ph = 1;
            auto ready = [&](uint32_t bar, uint32_t parity) {
                if (!ptx::mbar_try_wait(bar, parity)) wait(bar, parity, DEVICE_TIMEOUT_MMA);
            };
            auto qk = [&]() {               // S = Q K^T of the next tile
                const uint32_t slot = nk & (NS - 1), h = ns & 1u;
                ready(b_kf + 8 * slot, nk / NS & 1u);
                if (!ok) return;
                ptx::tc_fence_after();
                const uint32_t b = k_lo + slot * (C::KV_TILE >> 4), d = s_tm + TN * h;
#pragma unroll
                for (int k = 0; k < KS; ++k)
                    ptx::mma_f16_ss(d, q_lo + (k >> 2) * (C::Q_HALF >> 4) + (k & 3) * 2, ptx::kSdescHi,
                                    b + (k >> 2) * (C::KV_HALF >> 4) + (k & 3) * 2, ptx::kSdescHi, id_s, k > 0);
                ptx::mma_commit(b_s + 8 * h);
                ptx::mma_commit(b_ke + 8 * slot);
                ++nk, ++ns;
            };
            for (; w.u < w.u1 && ok; walk_next<R, TN>(p, w)) {
                const int tiles = tile_end() - tile_begin();
                if (i == 1 && item_rows() <= 128) {
                    // no rows in this tile: only hand the slots on
                    for (int t = 0; t < tiles && ok; ++t) {
                        ready(b_kf + 8 * (nk & (NS - 1)), nk / NS & 1u);
                        ptx::mbar_arrive(b_ke + 8 * (nk & (NS - 1)));
                        ready(b_vf + 8 * (nv & (NS - 1)), nv / NS & 1u);
                        ptx::mbar_arrive(b_ve + 8 * (nv & (NS - 1)));
                        ++nk, ++nv;
                    }
                    continue;
                }
                ready(b_q, q_ph);
                q_ph ^= 1u;
                if (ok) qk();
                if (ok && tiles > 1) qk();
                ready(b_oe, o_ph);
                o_ph ^= 1u;
                int t = 0;
                for (; t + 2 < tiles; ++t) {
                    // steady: PV of this tile, then S of the tile after next into the same buffer
                    const uint32_t vs = nv & (NS - 1), ks = nk & (NS - 1), h = np & 1u;
                    const uint32_t bar_v = b_vf + 8 * vs, bar_k = b_kf + 8 * ks, bar_p = b_p + 8 * h;
                    const uint32_t par_v = nv / NS & 1u, par_k = nk / NS & 1u, par_p = np >> 1 & 1u;
                    const bool all = ptx::mbar_test_wait(bar_v, par_v) & ptx::mbar_test_wait(bar_k, par_k) &
                                     ptx::mbar_test_wait(bar_p, par_p);
                    if (!all) {
                        wait(bar_v, par_v, DEVICE_TIMEOUT_MMA);
                        wait(bar_p, par_p, DEVICE_TIMEOUT_MMA);
                        if (!wait(bar_k, par_k, DEVICE_TIMEOUT_MMA)) break;
                    }
                    ptx::tc_fence_after();
                    const uint32_t d = s_tm + TN * h, bv = v_lo + vs * (C::KV_TILE >> 4), bk = k_lo + ks * (C::KV_TILE >> 4);
#pragma unroll
                    for (int k = 0; k < TN / 16; ++k)
                        ptx::mma_f16_ts(o_tm, d + 8 * k, bv + k * (2048 >> 4), ptx::kSdescHi, id_o, k > 0 || t > 0);
                    ptx::mma_commit(b_od + 8 * h);
                    ptx::mma_commit(b_ve + 8 * vs);
#pragma unroll
                    for (int k = 0; k < KS; ++k)
                        ptx::mma_f16_ss(d, q_lo + (k >> 2) * (C::Q_HALF >> 4) + (k & 3) * 2, ptx::kSdescHi,
                                        bk + (k >> 2) * (C::KV_HALF >> 4) + (k & 3) * 2, ptx::kSdescHi, id_s, k > 0);
                    ptx::mma_commit(b_s + 8 * h);
                    ptx::mma_commit(b_ke + 8 * ks);
                    ++nv, ++np, ++nk, ++ns;
                }
                for (; t < tiles && ok; ++t) {   // the last two
                    const uint32_t slot = nv & (NS - 1), h = np & 1u;
                    ready(b_vf + 8 * slot, nv / NS & 1u);
                    ready(b_p + 8 * h, np >> 1 & 1u);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    const uint32_t b = v_lo + slot * (C::KV_TILE >> 4), a = s_tm + TN * h;
#pragma unroll
                    for (int k = 0; k < TN / 16; ++k)
                        ptx::mma_f16_ts(o_tm, a + 8 * k, b + k * (2048 >> 4), ptx::kSdescHi, id_o, k > 0 || t > 0);
                    ptx::mma_commit(b_od + 8 * h);
                    ptx::mma_commit(b_ve + 8 * slot);
                    ++nv, ++np;
                }
            }
            // the MMAs in flight end before tensor memory is freed: whoever waits for them may have given up
            ptx::mma_commit(final_bar);
            drain_wait(final_bar, 0u, p.timeout_ns);
        }
        __syncwarp();
    }
    } else if (warp >= 8) {
        ptx::regs_dec<kRegsUnpack>();
        // ------------------------------------------------------------ unpack
        const int which = (warp - 8) >> 2;         // keys, values
        const int tt = (threadIdx.x & 127) >> 1;   // the token of the tile
        const int side = threadIdx.x & 1;          // which half of its d
        const int vp = min(p.c.P, TN), place = tt & (vp - 1);
        const int block_at = tt / vp * (vp * (D + 2 * pair_row));
        const int codes_at = block_at + (which * vp + place) * (D / 2) + side * (D / 4);
        const int vpairs_at = block_at + vp * D + (vp + place) * pair_row;
        const int pairs_at = vpairs_at - (1 - which) * vp * pair_row;
        const uint32_t off_kv = which ? C::OFF_V : C::OFF_K;
        int s = 0;
        uint32_t ph = 0, n = 0;                    // n: tiles so far, slot n % 4
        for (; w.u < w.u1; walk_next<R, TN>(p, w)) {
            const int rows = item_rows(), te = tile_end();
            const int pos0 = w.s.L - w.s.n + row_token(p, w.rt * R);
            const int pos1 = w.s.L - w.s.n + row_token(p, w.rt * R + rows - 1);
            const int all_hi = p.causal ? min(w.s.L, pos0 + 1) : w.s.L;
            const int all_lo = first_seen(p, pos1);
            for (int t = tile_begin(); t < te; ++t, ++n) {
                const int tok = t * TN;
                const uint32_t slot = n & (NS - 1);
                ok = __all_sync(0xffffffffu, wait(raw_full(s), ph, DEVICE_TIMEOUT_TRANSFORM));
                ok = __all_sync(0xffffffffu, wait(kv_empty(which, slot), (n / NS & 1u) ^ 1u, DEVICE_TIMEOUT_TRANSFORM));
                if (ok) {
                    const uint8_t* st = smem + C::OFF_RAW + s * stage_bytes;
                    uint8_t* dst = smem + off_kv + slot * C::KV_TILE + tt * 128;
                    bool clear = false, spoil = false;
                    if (tok < all_lo || tok + TN > all_hi) {
                        // 0 * NaN must not reach rows that do not see a token: values
                        // nobody sees are cleared, and a NaN among a seen token's
                        // values moves to its key, where each row's mask applies
                        uint32_t z = 0;
                        for (int j = 0; j < pair_row; j += 4)
                            z = fma2<BF16>(*reinterpret_cast<const uint32_t*>(st + vpairs_at + j), 0u, z);
                        spoil = (z & 0x7FFF7FFFu) != 0;
                        clear = which == 1 && (spoil || tok + tt < w.v.lo || tok + tt >= w.v.hi);
                        spoil = which == 0 && spoil;
                    }
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        // 32 codes; the order spreads a quarter warp's reads and writes over the banks
                        const int part = D == 128 ? c ^ (tt >> 1 & 1) ^ side : 0;
                        const uint4 cw = *reinterpret_cast<const uint4*>(st + codes_at + part * 16);
                        const int d0 = side * (D / 2) + part * 32;
                        uint32_t pair = *reinterpret_cast<const uint32_t*>(st + pairs_at + (d0 >> p.c.g_shift) * 4);
                        if (clear) pair = 0u;
                        if (spoil) pair = BF16 ? 0x7FC07FC0u : 0x7E007E00u;
                        if (which) pair = summand<BF16>(pair);
                        const Operand<BF16> op = Operand<BF16>::both(pair);
                        const uint32_t words[4] = {cw.x, cw.y, cw.z, cw.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t x = words[j], y = x >> 8;
                            const int chunk = (d0 >> 3) + j;
                            *reinterpret_cast<uint4*>(dst + (chunk >> 3) * C::KV_HALF + (((chunk & 7) ^ (tt & 7)) << 4)) =
                                make_uint4(op.low(x), op.high(x), op.low(y), op.high(y));
                        }
                    }
                    ptx::fence_proxy_async_smem();
                }
                __syncwarp();
                if (ok && lane == 0) {
                    ptx::mbar_arrive(kv_full(which, slot));
                    ptx::mbar_arrive(raw_empty(s));
                }
                if (++s == RS) s = 0, ph ^= 1u;
            }
        }
    } else {
        ptx::regs_inc<kRegsSoftmax>();
        // ------------------------------------------------------------ softmax
        const int i = warp >> 2;                     // row tile
        const int r1 = threadIdx.x & 127;            // row of the tile
        const int r = threadIdx.x;                   // row of the item
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const uint32_t s_tm = tmem + lanes + C::S_COL + 128 * i, o_tm = tmem + lanes + C::O_COL + 128 * i;
        // a negative scale moves its sign to Q, and a zero one goes to Q altogether, so that a masked
        // -inf stays -inf
        const float sl2 = p.scale == 0.f ? 1.f : fabsf(p.scale) * 1.4426950408889634f;
        const uint32_t flip = p.scale < 0.f ? 0x80008000u : 0u;
        const uint64_t sl = f2(sl2, sl2);
        uint32_t n = 0;                              // tiles of this row tile so far: S buffer n % 2
        for (; w.u < w.u1; walk_next<R, TN>(p, w)) {
            const int rows = item_rows();
            const bool idle = 128 * i >= rows;       // no rows in this tile
            const int row = w.rt * R + min(r, rows - 1);
            const int qt = row_token(p, row);
            const int64_t tq = w.s.q0 + qt;
            const int head = w.head * p.group + row - qt * p.group;
            const int pos = w.s.L - w.s.n + qt;
            const int hi = p.causal ? min(w.s.L, pos + 1) : w.s.L;
            const int lo = first_seen(p, pos);
            if (!idle) {
                const uint16_t* src = static_cast<const uint16_t*>(p.q) + tq * p.q_stride + (int64_t)head * D;
                uint8_t* dst = smem + C::OFF_Q + i * C::Q_TILE + r1 * 128;
#pragma unroll 4
                for (int ch = 0; ch < D / 8; ++ch) {
                    uint4 v = *reinterpret_cast<const uint4*>(src + ch * 8);
                    if (r >= rows) v = make_uint4(0u, 0u, 0u, 0u);
                    v.x ^= flip, v.y ^= flip, v.z ^= flip, v.w ^= flip;
                    if (p.scale == 0.f)
                        v = make_uint4(fma2<BF16>(v.x, 0u, 0u), fma2<BF16>(v.y, 0u, 0u), fma2<BF16>(v.z, 0u, 0u),
                                       fma2<BF16>(v.w, 0u, 0u));
                    *reinterpret_cast<uint4*>(dst + (ch >> 3) * C::Q_HALF + (((ch & 7) ^ (r1 & 7)) << 4)) =
                        make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                                   __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(q_full(i));
            }
            const int tb = tile_begin(), te = tile_end();
            float m = -INFINITY, l = 0.f;
            if (!idle) {
#pragma unroll 1
                for (int t = tb; t < te; ++t, ++n) {
                    const uint32_t s_now = s_tm + TN * (n & 1u);
                    if (ok) ok = __all_sync(0xffffffffu, wait(s_full(i, n & 1u), n >> 1 & 1u, DEVICE_TIMEOUT_EPILOGUE));
                    if (!ok) break;
                    ptx::tc_fence_after();
                    uint32_t v[64];
                    ptx::tmem_ld64(s_now, v);
                    const int h = hi - t * TN, b = lo - t * TN;      // this row sees columns [b, h)
                    const bool masked = __any_sync(0xffffffffu, b > 0 || h < TN);
                    ptx::tmem_wait_ld();
                    if (masked) {
                        // the few tiles on a mask's edge: bit k of `see` is column k
                        const uint64_t below = h >= 64 ? ~0ull : h <= 0 ? 0ull : (1ull << h) - 1;
                        const uint64_t from = b <= 0 ? ~0ull : b >= 64 ? 0ull : ~((1ull << b) - 1);
                        const uint32_t see[2] = {(uint32_t)(below & from), (uint32_t)((below & from) >> 32)};
#pragma unroll
                        for (int k = 0; k < 64; ++k)
                            if (!(see[k >> 5] >> (k & 31) & 1u)) v[k] = 0xFF800000u;
                    }
                    // Under the maximum so far a sum below 2^14 shows that no probability
                    // passed 2^14, which both types hold; else the tile is done again under
                    // the new maximum.  Rows that have seen nothing have none yet.
                    float sum;
#pragma unroll 1
                    for (bool again = __any_sync(0xffffffffu, m == -INFINITY);;) {
                        if (again) {
                            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                            for (int k = 0; k < 64; k += 8)
#pragma unroll
                                for (int c = 0; c < 4; ++c)
                                    mx[c] = max3(mx[c], __uint_as_float(v[k + 2 * c]), __uint_as_float(v[k + 2 * c + 1]));
                            const float top = sl2 * max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
                            const bool grow = top > m + 8.f;
                            const float m1 = grow ? top : m, f = grow ? part_weight(m, m1) : 1.f;
                            m = m1;
                            l *= f;
                            if (t > tb && __any_sync(0xffffffffu, grow)) {
                                // O is scaled between products: the last one has to have ended
                                ok = __all_sync(0xffffffffu, wait(o_done(i, (n - 1) & 1u), (n - 1) >> 1 & 1u, DEVICE_TIMEOUT_EPILOGUE));
                                if (!ok) break;
                                ptx::tc_fence_after();
#pragma unroll 1
                                for (int c = 0; c < D; c += 16) {
                                    uint32_t x[16];
                                    ptx::tmem_ld16(o_tm + c, x);
                                    ptx::tmem_wait_ld();
#pragma unroll
                                    for (int k = 0; k < 16; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * f);
                                    ptx::tmem_st16(o_tm + c, x);
                                }
                            }
                        }
                        const float mm = m == -INFINITY ? 0.f : m;
                        const uint64_t nm = f2(-mm, -mm);
                        uint64_t la = 0, lb = 0;
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            uint32_t o[16];
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                const int at = 32 * c + 2 * k;
                                float2 e = un2(fma_f2(f2(__uint_as_float(v[at]), __uint_as_float(v[at + 1])), sl, nm));
                                e.x = ex2(e.x), e.y = ex2(e.y);
                                if (k & 1)
                                    lb = add_f2(lb, f2(e.x, e.y));
                                else
                                    la = add_f2(la, f2(e.x, e.y));
                                o[k] = pack2<BF16>(e.x, e.y);
                            }
                            ptx::tmem_st16(s_now + 16 * c, o);   // S is in registers: P may cover it before the check
                        }
                        const float2 ls = un2(add_f2(la, lb));
                        sum = ls.x + ls.y;
                        if (again || !__any_sync(0xffffffffu, !(sum < 16384.f))) break;
                        again = true;
                        ptx::tmem_wait_st();   // the second P is stored over the first
                    }
                    if (!ok) break;
                    l += sum;
                    ptx::tmem_wait_st();
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(p_full(i, n & 1u));
                }
                if (ok) ok = __all_sync(0xffffffffu, wait(o_done(i, (n - 1) & 1u), (n - 1) >> 1 & 1u, DEVICE_TIMEOUT_EPILOGUE));
                ptx::tc_fence_after();
            }
            // ---- the item's result, or this block's part of it
            const bool whole = w.u == w.item0 && w.item0 + w.units <= w.u1;
            const int b_first = whole ? 0 : run_of(runs, w.item0);
            const int parts = whole ? 1 : run_of(runs, w.item0 + w.units - 1) - b_first + 1;
            float* part = p.ws_part + (size_t)(2 * blockIdx.x + (w.u == w.item0 ? 1 : 0)) * attn_slot_floats(R, D);
            if (!idle && ok) {
                const float inv = l == 0.f ? 0.f : kSumUnit<BF16> / l;
                uint16_t* out = static_cast<uint16_t*>(p.out) + tq * p.out_stride + (int64_t)head * D;
                float* po = part + (size_t)r * D;
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                    uint32_t v[16];
                    ptx::tmem_ld16(o_tm + c, v);
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        // columns hold d = 0 4 1 5 2 6 3 7 of each eight
                        float d[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) d[(k >> 1) + 4 * (k & 1)] = __uint_as_float(v[8 * j + k]);
                        if (r < rows) {
                            if (whole) {
                                *reinterpret_cast<uint4*>(out + c + 8 * j) =
                                    make_uint4(pack2<BF16>(d[0] * inv, d[1] * inv), pack2<BF16>(d[2] * inv, d[3] * inv),
                                               pack2<BF16>(d[4] * inv, d[5] * inv), pack2<BF16>(d[6] * inv, d[7] * inv));
                            } else {
                                float4* dst = reinterpret_cast<float4*>(po + c + 8 * j);
                                __stcg(dst, make_float4(d[0], d[1], d[2], d[3]));
                                __stcg(dst + 1, make_float4(d[4], d[5], d[6], d[7]));
                            }
                        }
                    }
                }
                if (r < rows) {
                    if (!whole)
                        __stcg(reinterpret_cast<float2*>(part + R * D) + r, make_float2(m, l));
                    else if (p.lse != nullptr)
                        p.lse[tq * p.Hq + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
                }
            }
            if (!idle) {
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(o_empty(i));
            }
            if (!whole) {
                ptx::named_barrier_sync(1, 256);
                if (threadIdx.x == 0) {
                    int last = 0;
                    if (ok) {
                        last = arrive_ticket(p.ws_count + b_first) + 1 == (uint32_t)parts;
                        if (last) p.ws_count[b_first] = 0u;
                    }
                    *last_flag = last;
                }
                ptx::named_barrier_sync(1, 256);
                if (*last_flag) {
                    merge_parts<BF16, D, R, C::MERGE_ROWS, 256>(p, w, b_first, parts,
                                                                reinterpret_cast<float*>(smem + C::OFF_Q), threadIdx.x, 1);
                }
            }
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 16) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc<1>(*tmem_slot, 512);
    }
}

}  // namespace wq
