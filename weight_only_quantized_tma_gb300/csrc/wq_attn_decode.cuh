// wq_attn_decode.cuh -- attention of few query rows over the 4-bit cache.
//
//   S^T = K Q^T,  P = exp2(scale' S - m),  O^T += V^T P^T,  out = O / sum P
//
// Bound by the bytes of the cache (D + 8 D / G for each token and key head), so the
// kernel streams them once, with the fewest instructions for each code:
//   * cached tokens are the M dimension of the mma.sync m16n8k16 tiles (16 tokens x 8 query
//     rows), so the 8 rows of a group of heads fill a tile that single tokens leave empty
//     the other way round, and a lane's K operand is consecutive codes of one token;
//   * the order of d inside a product is free: lane c of a quad takes codes c D / 4 ..
//     (c + 1) D / 4 of its token, all in one group (G >= 32 >= D / 4), so one pair (s, lo)
//     serves it; Q is loaded in the same order.  V^T: lane g takes codes g D / 8 .. of four
//     tokens; two tokens' words are merged with byte permutes, since a pair of the V^T
//     operand is two tokens of one d;
//   * code -> number is a mask and one fma in bf16 (ShortOperand, wq_kv4.cuh), a magic number,
//     an exact subtraction and one fma in fp16: RN(lo + q s), the value that the cache stands
//     for, in every kernel.  An item whose pairs or queries are too large or too small for
//     ShortOperand is done again, straight from the cache, with the longer form (64 sequences
//     with values of some 2^-60 or 2^80 take three to four times as long);
//   * the running maximum moves only when a score passes it by more than 2^8, so most
//     tiles pay one vote in place of a reduction.
// Warps 0-3 each take 32 of the 128 tokens of a tile (with 8 rows as two products side by
// side) with their own maximum, sum and O, and meet once for each item; warp 4 copies page
// blocks into a ring with bulk copies.
//
// Measured: 64 sequences of 300 to 16384 tokens, 32 query and 8 key heads of 128, bf16: 147 us
// for 582 MB (4.0 TB/s).  What bounds it is the latency between a warp's instructions (issue
// slots 58% full), not a unit: in an earlier form of 148 us copies alone took 100 and arithmetic
// alone 138.
#pragma once

#include <type_traits>

#include "wq_attn_sched.cuh"
#include "wq_common.cuh"

namespace wq {

constexpr int kDecodeTN = 128;     // tokens of a tile
constexpr int kDecodeStages = 3;
constexpr int kDecodeBlocks = 2;   // 16-token blocks of a warp in a tile
constexpr int kDecodeMaxNT = 3;    // most groups of 8 rows in a row tile

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

template <int D, int NT>
struct DecodeCfg {
    static constexpr int R = 8 * NT;
    static constexpr int KS = D / 16;              // k steps of Q K^T = m tiles of V^T
    static constexpr bool Q_SMEM = NT > 1;         // Q operands: registers, or shared memory
    static constexpr int REGS = KS * NT * 4 + 4 * NT;                     // a lane's O, m and l
    static constexpr int OFF_EX = 0;                                      // two warps' results
    static constexpr int EX_BYTES = 2 * REGS * 32 * 4;
    static constexpr int OFF_Q = OFF_EX + EX_BYTES;
    static constexpr int Q_BYTES = Q_SMEM ? KS * NT * 32 * 8 : 0;
    static constexpr int OFF_W = OFF_Q + Q_BYTES;                         // merge weights
    static constexpr int W_BYTES = R * 33 * 4;
    static constexpr int OFF_BAR = (OFF_W + W_BYTES + 15) / 16 * 16;
    static constexpr int OFF_MISC = OFF_BAR + 2 * kDecodeStages * 8;
    static constexpr int OFF_RING = (OFF_MISC + 16 + 127) / 128 * 128;
    static constexpr int SIDE = NT == 1 ? 2 : 1;     // blocks side by side: more hide latencies, but need registers
    static constexpr int MIN_BLOCKS = NT == 1 ? 3 : 2;
};

// The token of row r (0..15) of a 16-token tile: neighbours differ in parity (K rows of a
// quad pair fall on both halves of the banks) and so do a quad's rows 0, 2, 4, 6 (V).
__device__ __forceinline__ int token_of_row(int r) { return r ^ ((r >> 1) & 1); }

// Q operands of 8 rows of an item, in the order of the codes.  Returns whether one is so large that
// the rounding of ShortOperand could move its scores: values are off by 2^-53 at most, D <= 128 of
// them times 2^33 / scale by 2^-13.
template <bool BF16, int D>
__device__ __forceinline__ bool load_q(const AttnParams& p, const Walk& w, int R, int nt, uint32_t (&q)[D / 16][2]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    constexpr int WK = D / 32;
    const int rows = min(R, w.s.n * p.group - w.rt * R);
    const int r = nt * 8 + g;
    uint32_t raw[D / 8];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) raw[i] = 0u;
    if (r < rows) {
        const int row = w.rt * R + r, qt = row_token(p, row);
        const uint16_t* src = static_cast<const uint16_t*>(p.q) + (int64_t)(w.s.q0 + qt) * p.q_stride +
                              (w.head * p.group + row - qt * p.group) * D + c * (D / 4);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const uint4 v = *reinterpret_cast<const uint4*>(src + 8 * i);
            raw[4 * i] = v.x, raw[4 * i + 1] = v.y, raw[4 * i + 2] = v.z, raw[4 * i + 3] = v.w;
        }
    }
#pragma unroll
    for (int j = 0; j < WK; ++j) {   // values 8j .. 8j + 7: pairs (0,4) (1,5) (2,6) (3,7)
        q[2 * j][0] = __byte_perm(raw[4 * j], raw[4 * j + 2], 0x5410);
        q[2 * j][1] = __byte_perm(raw[4 * j], raw[4 * j + 2], 0x7632);
        q[2 * j + 1][0] = __byte_perm(raw[4 * j + 1], raw[4 * j + 3], 0x5410);
        q[2 * j + 1][1] = __byte_perm(raw[4 * j + 1], raw[4 * j + 3], 0x7632);
    }
    uint32_t most = 0;
    if constexpr (BF16)
#pragma unroll
        for (int i = 0; i < D / 8; ++i) most = __vmaxu2(most, raw[i] & 0x7FFF7FFFu);
    const float2 m2 = unpack2<true>(most);
    return __any_sync(0xffffffffu, !(fmaxf(m2.x, m2.y) * fabsf(p.scale) <= 8.589934592e9f));
}

// Where a compute warp is in the ring.
struct RingPlace {
    int s;
    uint32_t ph;
    bool ok;
};
// What a warp has met that tells whether ShortOperand was exact.
struct Seen {
    uint32_t k_step;   // the largest s_low of a key: infinite where it overflowed
    uint32_t v_any;    // bits that a lane's value pairs have set
};

// A compute warp's part of an item, token tiles [tb, te): sums o, maxima m and sums of
// probabilities l, with operands of type Op (ShortOperand: o in units of 1 / kUp, else of
// kSumUnit), out of the ring or straight from the cache.
template <bool BF16, int D, int NT, typename Op, bool RING>
__device__ __forceinline__ void decode_tiles(const AttnParams& p, const Walk& w, int tb, int te, uint8_t* smem,
                                             int stage_bytes, const uint32_t (&qr)[DecodeCfg<D, NT>::Q_SMEM ? 1 : D / 16][2],
                                             RingPlace& r, float (&o)[D / 16][NT][4], float (&m)[NT][2],
                                             float (&l)[NT][2], Seen& seen) {
    using C = DecodeCfg<D, NT>;
    constexpr int R = C::R, KS = C::KS, TN = kDecodeTN, ST = kDecodeStages, NB = C::SIDE;
    constexpr int WK = D / 32;        // words of codes of a lane and token: K
    constexpr int WV = D / 64;        // V
    constexpr bool SHORT = std::is_same_v<Op, ShortOperand>;
    const uint32_t sbase = ptx::smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    auto full_bar = [&](int s) { return sbase + C::OFF_BAR + 8u * s; };
    auto empty_bar = [&](int s) { return sbase + C::OFF_BAR + 8u * (ST + s); };
    volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC);
    const uint2* qs = reinterpret_cast<const uint2*>(smem + C::OFF_Q);
    const float to_log2 = p.scale * 1.4426950408889634f * (SHORT ? ShortOperand::kUp : 1.0f);
    const int pair_row = 4 * (D >> p.c.g_shift);                // bytes of a token's pairs
    // this warp's blocks of 16 tokens inside a tile (a page holds a multiple of 16): codes
    // and pairs of keys; those of values follow at fixed distances
    uint32_t all_codes[kDecodeBlocks], all_pairs[kDecodeBlocks];
#pragma unroll
    for (int n = 0; n < kDecodeBlocks; ++n) {
        const int at = 16 * (kDecodeBlocks * warp + n), in_page = at & (p.c.P - 1);
        const uint32_t page_at = (uint32_t)((at >> p.c.p_shift) * p.c.block_bytes);
        all_codes[n] = page_at + in_page * (D / 2);
        all_pairs[n] = page_at + p.c.P * D + in_page * pair_row;
    }
    const uint32_t v_codes_off = p.c.P * (D / 2), v_pairs_off = p.c.P * pair_row;
    const int row_k[2] = {token_of_row(g), token_of_row(g) + 8};
    const int row_v[4] = {token_of_row(2 * c), token_of_row(2 * c + 1), token_of_row(2 * c) + 8,
                          token_of_row(2 * c + 1) + 8};
    const int k_group = ((c * (D / 4)) >> p.c.g_shift) * 4, v_group = ((g * (D / 8)) >> p.c.g_shift) * 4;

    const int rows = min(R, w.s.n * p.group - w.rt * R);
    // tokens that each of this lane's rows sees: [lo, hi)
    int lo[NT][2], hi[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int pos = w.s.L - w.s.n + row_token(p, w.rt * R + nt * 8 + 2 * c + i);
            hi[nt][i] = p.causal ? min(w.s.L, pos + 1) : w.s.L;
            lo[nt][i] = first_seen(p, pos);
        }
    // tokens that every row sees
    const int pos0 = w.s.L - w.s.n + row_token(p, w.rt * R);
    const int pos1 = w.s.L - w.s.n + row_token(p, w.rt * R + rows - 1);
    const int all_hi = p.causal ? min(w.s.L, pos0 + 1) : w.s.L;
    const int all_lo = first_seen(p, pos1);

#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[k][nt][i] = 0.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) m[nt][0] = m[nt][1] = -INFINITY, l[nt][0] = l[nt][1] = 0.f;

    for (int t = tb; t < te; ++t) {
        if constexpr (RING)
            if (r.ok) r.ok = __all_sync(0xffffffffu, bounded_wait(full_bar(r.s), r.ph, abort_flag, p.status,
                                                                  DEVICE_TIMEOUT_TRANSFORM, p.timeout_ns));
#pragma unroll 1
        for (int part = 0; part < kDecodeBlocks / NB; ++part) {
        const int tok = t * TN + 16 * (kDecodeBlocks * warp + part * NB);
        if (r.ok && tok < w.v.hi && tok + 16 * NB > w.v.lo) {
            const uint8_t *k_codes[NB], *k_pairs[NB];
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                if constexpr (RING) {
                    const uint8_t* st = smem + C::OFF_RING + r.s * stage_bytes;
                    k_codes[n] = st + (NB == 1 && part ? all_codes[kDecodeBlocks - 1] : all_codes[n]);
                    k_pairs[n] = st + (NB == 1 && part ? all_pairs[kDecodeBlocks - 1] : all_pairs[n]);
                } else {
                    // (a block that nobody sees: the nearest that somebody does)
                    const int at = max(min(tok + 16 * n, (w.v.hi - 1) & ~15), w.v.lo & ~15), in_page = at & (p.c.P - 1);
                    const uint8_t* block = p.c.pages + safe_page(p, w.b, at >> p.c.p_shift) * p.c.page_bytes +
                                           (int64_t)w.head * p.c.block_bytes;
                    k_codes[n] = block + in_page * (D / 2);
                    k_pairs[n] = block + p.c.P * D + in_page * pair_row;
                }
            }
            const bool masked = tok < all_lo || tok + 16 * NB > all_hi;
            // ---- S^T: 16 tokens x R rows for each block
            uint32_t kw[NB][2][WK], kp[NB][2];
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint8_t* src = k_codes[n] + row_k[i] * (D / 2) + c * (D / 8);
                    if constexpr (WK == 4) {
                        const uint4 v = *reinterpret_cast<const uint4*>(src);
                        kw[n][i][0] = v.x, kw[n][i][1] = v.y, kw[n][i][2] = v.z, kw[n][i][3] = v.w;
                    } else {
                        const uint2 v = *reinterpret_cast<const uint2*>(src);
                        kw[n][i][0] = v.x, kw[n][i][1] = v.y;
                    }
                    kp[n][i] = *reinterpret_cast<const uint32_t*>(k_pairs[n] + row_k[i] * pair_row + k_group);
                }
            if (masked) {
                // What a row does not see must not reach it as 0 * NaN: values that
                // nobody sees are cleared below, and a NaN among a seen token's values
                // moves to its key, where the mask of each row applies.
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t z = 0;
                        for (int j = 0; j < pair_row; j += 4)
                            z = fma2<BF16>(*reinterpret_cast<const uint32_t*>(k_pairs[n] + v_pairs_off +
                                                                              row_k[i] * pair_row + j), 0u, z);
                        if (z & 0x7FFF7FFFu) kp[n][i] = BF16 ? 0x7FC07FC0u : 0x7E007E00u;
                        const int tt = tok + 16 * n + row_k[i];
                        if (tt < w.v.lo || tt >= w.v.hi) kp[n][i] = 0u;
                    }
            }
            float sc[NB][NT][4];
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) sc[n][nt][0] = sc[n][nt][1] = sc[n][nt][2] = sc[n][nt][3] = 0.f;
            {
                Op k0[NB], k1[NB];
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    k0[n] = Op::both(kp[n][0]);
                    k1[n] = Op::both(kp[n][1]);
                    if constexpr (SHORT) seen.k_step = max(seen.k_step, max(k0[n].s_low, k1[n].s_low));
                }
#pragma unroll
                for (int j = 0; j < WK; ++j) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
#pragma unroll
                        for (int n = 0; n < NB; ++n) {
                            const uint32_t x0 = h ? kw[n][0][j] >> 8 : kw[n][0][j], x1 = h ? kw[n][1][j] >> 8 : kw[n][1][j];
                            const uint32_t a[4] = {k0[n].low(x0), k1[n].low(x1), k0[n].high(x0), k1[n].high(x1)};
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                if constexpr (C::Q_SMEM) {
                                    const uint2 q = qs[((2 * j + h) * NT + nt) * 32 + lane];
                                    mma16816<BF16>(sc[n][nt], a, q.x, q.y);
                                } else {
                                    mma16816<BF16>(sc[n][nt], a, qr[2 * j + h][0], qr[2 * j + h][1]);
                                }
                            }
                        }
                    }
                }
            }
            // ---- probabilities (scores in units of log2)
            bool grow = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float top = -INFINITY;
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        float x0 = sc[n][nt][i] * to_log2, x1 = sc[n][nt][2 + i] * to_log2;
                        if (masked) {
                            const int t0 = tok + 16 * n + row_k[0], t1 = tok + 16 * n + row_k[1];
                            if (t0 < lo[nt][i] || t0 >= hi[nt][i]) x0 = -INFINITY;
                            if (t1 < lo[nt][i] || t1 >= hi[nt][i]) x1 = -INFINITY;
                        }
                        sc[n][nt][i] = x0, sc[n][nt][2 + i] = x1;
                        top = fmaxf(top, fmaxf(x0, x1));
                    }
                    grow |= top > m[nt][i] + 8.f;
                }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float f[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float x = fmaxf(sc[0][nt][i], sc[0][nt][2 + i]);
#pragma unroll
                        for (int n = 1; n < NB; ++n) x = fmaxf(x, fmaxf(sc[n][nt][i], sc[n][nt][2 + i]));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                        x = fmaxf(x, m[nt][i]);
                        f[i] = part_weight(m[nt][i], x);
                        m[nt][i] = x;
                        l[nt][i] *= f[i];
                    }
#pragma unroll
                    for (int k = 0; k < KS; ++k)
                        o[k][nt][0] *= f[0], o[k][nt][2] *= f[0], o[k][nt][1] *= f[1], o[k][nt][3] *= f[1];
                }
            }
            uint32_t pb[NB][NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float m0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0], m1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    const float p0 = ex2(sc[n][nt][0] - m0), p1 = ex2(sc[n][nt][1] - m1), p2 = ex2(sc[n][nt][2] - m0),
                                p3 = ex2(sc[n][nt][3] - m1);
                    l[nt][0] += p0 + p2;
                    l[nt][1] += p1 + p3;
                    pb[n][nt][0] = transpose8x8(pack2<BF16>(p0, p1));
                    pb[n][nt][1] = transpose8x8(pack2<BF16>(p2, p3));
                }
            }
            // ---- O^T += V^T P^T
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                uint32_t vw[4][WV], vpair[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint8_t* src = k_codes[n] + v_codes_off + row_v[i] * (D / 2) + g * (D / 16);
                    if constexpr (WV == 2) {
                        const uint2 v = *reinterpret_cast<const uint2*>(src);
                        vw[i][0] = v.x, vw[i][1] = v.y;
                    } else {
                        vw[i][0] = *reinterpret_cast<const uint32_t*>(src);
                    }
                    vpair[i] = *reinterpret_cast<const uint32_t*>(k_pairs[n] + v_pairs_off + row_v[i] * pair_row + v_group);
                }
                if (masked) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int tt = tok + 16 * n + row_v[i];
                        if (tt < w.v.lo || tt >= w.v.hi || (fma2<BF16>(vpair[i], 0u, 0u) & 0x7FFF7FFFu)) vpair[i] = 0u;
                    }
                }
                if constexpr (SHORT) seen.v_any |= vpair[0] | vpair[1] | vpair[2] | vpair[3];
                if constexpr (!SHORT)
#pragma unroll
                    for (int i = 0; i < 4; ++i) vpair[i] = summand<BF16>(vpair[i]);
                const Op vab(__byte_perm(vpair[0], vpair[1], 0x5410), __byte_perm(vpair[0], vpair[1], 0x7632));
                const Op vcd(__byte_perm(vpair[2], vpair[3], 0x5410), __byte_perm(vpair[2], vpair[3], 0x7632));
#pragma unroll
                for (int j = 0; j < WV; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t sel = 0x4400u + 0x1111u * i;
                        const uint32_t xab = __byte_perm(vw[0][j], vw[1][j], sel), xcd = __byte_perm(vw[2][j], vw[3][j], sel);
                        const uint32_t a[4] = {vab.low(xab), vab.high(xab), vcd.low(xcd), vcd.high(xcd)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma16816<BF16>(o[4 * j + i][nt], a, pb[n][nt][0], pb[n][nt][1]);
                    }
            }
        }
        }
        if constexpr (RING) {
            __syncwarp();
            if (r.ok && lane == 0) ptx::mbar_arrive(empty_bar(r.s));
            if (++r.s == ST) r.s = 0, r.ph ^= 1u;
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], 4);
            l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], 8);
            l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], 16);
        }
}

// Whether ShortOperand rounds one of the values that a compute warp has worked with: looks at the
// pairs in the cache again, a lane for each of 32 tokens and 16 tiles' loads at a time.
template <int D>
__device__ __forceinline__ bool decode_rounded(const AttnParams& p, const Walk w, int tb, int te) {
    constexpr int N = 16;
    const int pair_row = 4 * (D >> p.c.g_shift), first = 32 * (threadIdx.x >> 5) + (threadIdx.x & 31);
    bool found = false;
    for (int t = tb; t < te; t += N) {
        const uint8_t* pairs[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int tt = (t + j) * kDecodeTN + first;
            pairs[j] = nullptr;
            if (t + j < te && tt >= w.v.lo && tt < w.v.hi) {
                const int64_t page = p.table[(int64_t)w.b * p.table_stride + (tt >> p.c.p_shift)];
                pairs[j] = p.c.pages + (page >= 0 && page < p.c.num_pages ? page : 0) * p.c.page_bytes +
                           (int64_t)w.head * p.c.block_bytes + p.c.P * D + (tt & (p.c.P - 1)) * pair_row;
            }
        }
        for (int x = 0; x < pair_row; x += 4) {
            uint32_t k[N], v[N];
#pragma unroll
            for (int j = 0; j < N; ++j) {
                k[j] = pairs[j] ? *reinterpret_cast<const uint32_t*>(pairs[j] + x) : 0u;
                v[j] = pairs[j] ? *reinterpret_cast<const uint32_t*>(pairs[j] + p.c.P * pair_row + x) : 0u;
            }
#pragma unroll
            for (int j = 0; j < N; ++j) found |= ShortOperand::refuses(k[j]) || ShortOperand::refuses(v[j]);
        }
    }
    return __any_sync(0xffffffffu, found);
}

// The same once more for every s and lo, from the cache itself, where it is needed: o, m and l are in
// `back`, and the new ones go there.  A call with everything in memory, so that the kernel's registers
// stay with the quick form (147 us for the 64 sequences; inlined some 10 us more, with o, m and l held
// across the call 15, with Operand for every item 20, without looking for what is not exact 5 less).
template <int D, int NT>
__device__ __noinline__ void decode_again(const AttnParams& p, const Walk w, int tb, int te, uint8_t* smem, float* back,
                                          bool sure) {
    if (!sure && !decode_rounded<D>(p, w, tb, te)) return;
    constexpr int KS = D / 16;
    float o[KS][NT][4], m[NT][2], l[NT][2];
    uint32_t qr[DecodeCfg<D, NT>::Q_SMEM ? 1 : KS][2];
    if constexpr (!DecodeCfg<D, NT>::Q_SMEM) load_q<true, D>(p, w, 8 * NT, 0, qr);
    RingPlace r{0, 0u, true};
    Seen seen{};
    decode_tiles<true, D, NT, Operand<true>, false>(p, w, tb, te, smem, 0, qr, r, o, m, l, seen);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) back[(k * NT + nt) * 4 + i] = o[k][nt][i];
#pragma unroll
        for (int i = 0; i < 2; ++i) back[KS * NT * 4 + nt * 4 + i] = m[nt][i], back[KS * NT * 4 + nt * 4 + 2 + i] = l[nt][i];
    }
}

template <bool BF16, int D, int NT>
__global__ void __launch_bounds__(160, (DecodeCfg<D, NT>::MIN_BLOCKS)) attn_decode_kernel(
    const __grid_constant__ AttnParams p, const int stage_bytes) {
    using C = DecodeCfg<D, NT>;
    constexpr int R = C::R, KS = C::KS, TN = kDecodeTN, ST = kDecodeStages;
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t sbase = ptx::smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto full_bar = [&](int s) { return sbase + C::OFF_BAR + 8u * s; };
    auto empty_bar = [&](int s) { return sbase + C::OFF_BAR + 8u * (ST + s); };
    volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC);
    volatile int* last_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            ptx::mbar_init(full_bar(s), 1);
            ptx::mbar_init(empty_bar(s), 4);
        }
        *abort_flag = 0u;
        ptx::fence_barrier_init();
        ptx::fence_proxy_async_smem();
    }
    __syncthreads();
    // every input may come from the kernel before
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();

    Walk w;
    const Runs runs = walk_begin<R, TN>(p, blockIdx.x, gridDim.x, w);

    if (warp == 4) {
        // ------------------------------------------------------------ producer
        const uint64_t pol = ptx::policy_evict_first();
        int s = 0;
        uint32_t ph = 0;
        bool ok = true;
        uint32_t issued = 0;
        for (; w.u < w.u1 && ok; walk_next<R, TN>(p, w)) {
            if (w.u == w.item0 && lane == 0 && p.lens[w.b] > p.most)
                atomicOr(p.status, DEVICE_INDEX);
            const int tb = w.v.t0 + (int)(w.u - w.item0), te = w.v.t0 + (int)(min(w.item0 + w.units, w.u1) - w.item0);
            for (int t = tb; t < te && ok; ++t) {
                const int tok = t * TN;
                // the tile's pages that hold a token to be seen: [skip, pages)
                const int pages = min((w.v.hi - tok + p.c.P - 1) >> p.c.p_shift, TN >> p.c.p_shift);
                const int skip = max(w.v.lo - tok, 0) >> p.c.p_shift;
                const bool mine = lane >= skip && lane < pages;
                const int64_t page = mine ? safe_page(p, w.b, (tok >> p.c.p_shift) + lane) : 0;
                ok = bounded_wait(empty_bar(s), ph ^ 1u, abort_flag, p.status, DEVICE_TIMEOUT_PRODUCER, p.timeout_ns);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane == 0) {
                    if (pages > skip)
                        ptx::mbar_arrive_expect_tx(full_bar(s), (uint32_t)((pages - skip) * p.c.block_bytes));
                    else
                        ptx::mbar_arrive(full_bar(s));
                }
                __syncwarp();
                if (mine)
                    ptx::bulk_load(sbase + C::OFF_RING + s * stage_bytes + lane * p.c.block_bytes,
                                   p.c.pages + page * p.c.page_bytes + (int64_t)w.head * p.c.block_bytes,
                                   p.c.block_bytes, full_bar(s), pol);
                issued |= 1u << s;
                if (++s == ST) s = 0, ph ^= 1u;
            }
        }
        // The copies in flight land before the block may end: whoever waits for them may have given up,
        // this warp or another.  A stage passed in this lap was filled with parity ph, the others in the
        // lap before.
        for (int i = 0; i < ST; ++i)
            if (issued >> i & 1u) drain_wait(full_bar(i), i < s ? ph : ph ^ 1u, p.timeout_ns);
        return;
    }

    // ---------------------------------------------------------------- compute warps
    const int g = lane >> 2, c = lane & 3;
    float* ex = reinterpret_cast<float*>(smem + C::OFF_EX);
    uint2* qs = reinterpret_cast<uint2*>(smem + C::OFF_Q);
    volatile uint8_t* q_large = smem + C::OFF_MISC + 8;
    RingPlace ring{0, 0u, true};
    uint32_t qr[C::Q_SMEM ? 1 : KS][2];

    for (; w.u < w.u1; walk_next<R, TN>(p, w)) {
        const int rows = min(R, w.s.n * p.group - w.rt * R);
        // ---- Q operands of the item, in the order of the codes
        bool doubt = false;   // that ShortOperand is exact
        if constexpr (C::Q_SMEM) {
            ptx::named_barrier_sync(1, 128);
            for (int nt = warp; nt < NT; nt += 4) {
                uint32_t q[KS][2];
                const bool large = load_q<BF16, D>(p, w, R, nt, q);
                if (lane == 0) q_large[nt] = large;
#pragma unroll
                for (int k = 0; k < KS; ++k) qs[(k * NT + nt) * 32 + lane] = make_uint2(q[k][0], q[k][1]);
            }
            ptx::named_barrier_sync(1, 128);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) doubt |= q_large[nt] != 0;
        } else {
            doubt = load_q<BF16, D>(p, w, R, 0, qr);
        }
        float o[KS][NT][4], m[NT][2], l[NT][2];
        const int tb = w.v.t0 + (int)(w.u - w.item0), te = w.v.t0 + (int)(min(w.item0 + w.units, w.u1) - w.item0);
        Seen seen{0u, 0u};
        decode_tiles<BF16, D, NT, std::conditional_t<BF16, ShortOperand, Operand<false>>, true>(
            p, w, tb, te, smem, stage_bytes, qr, ring, o, m, l, seen);
        const bool ok = ring.ok;
        if constexpr (BF16) {
            // Where that was not exact, once more.  An overflow shows in the keys' largest step or makes a
            // sum infinite or NaN.  Values that were rounded, by 2^-53 at most, matter to large queries
            // and to results below 2^-30; what is 0 because all of a lane's values are is none of these,
            // and for the rest (a sum of many values is exactly 0 now and then) the pairs tell.  With
            // scales above 2^25 scores themselves may leave fp32's range in these units.
            bool again = seen.k_step >= 0x7F800000u || fabsf(p.scale) > 33554432.f;
            seen.v_any |= __shfl_xor_sync(0xffffffffu, seen.v_any, 1);
            seen.v_any |= __shfl_xor_sync(0xffffffffu, seen.v_any, 2);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float least = INFINITY, sum = l[nt][i];
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        least = fminf(least, fminf(fabsf(o[k][nt][i]), fabsf(o[k][nt][2 + i])));
                        sum += fabsf(o[k][nt][i]) + fabsf(o[k][nt][2 + i]);
                    }
                    again |= !(sum < INFINITY);
                    if (nt * 8 + 2 * c + i < rows && (seen.v_any & 0x7FFF7FFFu))
                        doubt |= least < l[nt][i] * 7.703719777548943e-34f;   // 2^-110
                }
            again = __any_sync(0xffffffffu, again);
            constexpr float unit = ShortOperand::kUp / kSumUnit<true>;
            if (__builtin_expect(ok && (again || __any_sync(0xffffffffu, doubt)), 0)) {
                float back[C::REGS];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int k = 0; k < KS; ++k)
#pragma unroll
                        for (int i = 0; i < 4; ++i) back[(k * NT + nt) * 4 + i] = o[k][nt][i] * unit;
#pragma unroll
                    for (int i = 0; i < 2; ++i) back[KS * NT * 4 + nt * 4 + i] = m[nt][i], back[KS * NT * 4 + nt * 4 + 2 + i] = l[nt][i];
                }
                decode_again<D, NT>(p, w, tb, te, smem, back, again);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int k = 0; k < KS; ++k)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[k][nt][i] = back[(k * NT + nt) * 4 + i];
#pragma unroll
                    for (int i = 0; i < 2; ++i) m[nt][i] = back[KS * NT * 4 + nt * 4 + i], l[nt][i] = back[KS * NT * 4 + nt * 4 + 2 + i];
                }
            } else {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < KS; ++k)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[k][nt][i] *= unit;
            }
        }

        // ---- the four warps' results, pairwise
        auto put = [&](int slot) {
            float* e = ex + slot * C::REGS * 32 + lane;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int i = 0; i < 4; ++i) e[((k * NT + nt) * 4 + i) * 32] = o[k][nt][i];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    e[(KS * NT * 4 + nt * 4 + i) * 32] = m[nt][i];
                    e[(KS * NT * 4 + nt * 4 + 2 + i) * 32] = l[nt][i];
                }
            }
        };
        auto add = [&](int slot) {
            const float* e = ex + slot * C::REGS * 32 + lane;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float f[2], h[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float m2 = e[(KS * NT * 4 + nt * 4 + i) * 32], l2 = e[(KS * NT * 4 + nt * 4 + 2 + i) * 32];
                    const float M = fmaxf(m[nt][i], m2);
                    f[i] = part_weight(m[nt][i], M), h[i] = part_weight(m2, M);
                    m[nt][i] = M;
                    l[nt][i] = l[nt][i] * f[i] + l2 * h[i];
                }
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        o[k][nt][i] = o[k][nt][i] * f[i & 1] + e[((k * NT + nt) * 4 + i) * 32] * h[i & 1];
            }
        };
        ptx::named_barrier_sync(1, 128);   // the slots are free
        if (warp >= 2) put(warp - 2);
        ptx::named_barrier_sync(1, 128);
        if (warp < 2) add(warp);
        if (warp == 1) put(1);
        ptx::named_barrier_sync(1, 128);
        const bool whole = w.u == w.item0 && w.item0 + w.units <= w.u1;
        const int b_first = whole ? 0 : run_of(runs, w.item0);
        const int parts = whole ? 1 : run_of(runs, w.item0 + w.units - 1) - b_first + 1;
        if (warp == 0) {
            add(1);
            if (whole && ok) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int r = nt * 8 + 2 * c + i;
                        if (r >= rows) continue;
                        const int row = w.rt * R + r, qt = row_token(p, row);
                        const int64_t t = w.s.q0 + qt;
                        const int head = w.head * p.group + row - qt * p.group;
                        const float inv = l[nt][i] == 0.f ? 0.f : kSumUnit<BF16> / l[nt][i];
                        uint16_t* out = static_cast<uint16_t*>(p.out) + t * p.out_stride + (int64_t)head * D + g * (D / 8);
#pragma unroll
                        for (int k = 0; k < KS; k += 4)
                            *reinterpret_cast<uint4*>(out + 2 * k) = make_uint4(
                                pack2<BF16>(o[k][nt][i] * inv, o[k][nt][2 + i] * inv),
                                pack2<BF16>(o[k + 1][nt][i] * inv, o[k + 1][nt][2 + i] * inv),
                                pack2<BF16>(o[k + 2][nt][i] * inv, o[k + 2][nt][2 + i] * inv),
                                pack2<BF16>(o[k + 3][nt][i] * inv, o[k + 3][nt][2 + i] * inv));
                        if (p.lse != nullptr && g == 0)
                            p.lse[t * p.Hq + head] =
                                l[nt][i] == 0.f ? -INFINITY : (m[nt][i] + log2f(l[nt][i])) * 0.6931471805599453f;
                    }
            } else if (ok) {
                float* slot = p.ws_part + (size_t)(2 * blockIdx.x + (w.u == w.item0 ? 1 : 0)) * attn_slot_floats(R, D);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int r = nt * 8 + 2 * c + i;
                        if (r >= rows) continue;
#pragma unroll
                        for (int k = 0; k < KS; k += 2)
                            __stcg(reinterpret_cast<float4*>(slot + r * D + g * (D / 8) + 2 * k),
                                   make_float4(o[k][nt][i], o[k][nt][2 + i], o[k + 1][nt][i], o[k + 1][nt][2 + i]));
                        if (g == 0)
                            __stcg(reinterpret_cast<float2*>(slot + R * D) + r, make_float2(m[nt][i], l[nt][i]));
                    }
                __syncwarp();
                if (lane == 0) {
                    const int last = arrive_ticket(p.ws_count + b_first) + 1 == (uint32_t)parts;
                    if (last) p.ws_count[b_first] = 0u;
                    *last_flag = last;
                }
            } else if (lane == 0) {
                *last_flag = 0;
            }
        }
        if (!whole) {
            ptx::named_barrier_sync(1, 128);
            if (*last_flag) {
                merge_parts<BF16, D, R, R, 128>(p, w, b_first, parts, reinterpret_cast<float*>(smem + C::OFF_W),
                                             threadIdx.x, 1);
            }
        }
    }
}

}  // namespace wq
