// wq_attn_sched.cuh -- how the attention kernels share out their work.
//
// An item is one row tile (R consecutive rows; a row is a query token and one of the
// heads that share a key head) of one key head of one sequence; it walks the tiles of TN
// cached tokens that its rows can see.  The tiles of all items, laid end to end (sequence,
// row tile, key head, tile), are cut into equal runs, one for each block, so that unequal
// lengths leave no block with more work than another; an item that spans blocks leaves a
// partial result from each, and the last block to finish adds them in the order of the
// tiles, so results do not depend on timing.  Lengths live on the device: every block
// finds its own run with a scan over the sequences.
#pragma once

#include "wq_kv4.cuh"

namespace wq {

// 64-bit tile numbers almost always fit 32 bits, where a division is several times shorter.
__device__ __forceinline__ int64_t div_short(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
    return a / b;
}

struct SeqInfo {
    int q0;      // first query row of q
    int n;       // new tokens
    int L;       // cached tokens
    int tiles;   // row tiles
};

template <int R>
__device__ __forceinline__ SeqInfo seq_info(const AttnParams& p, int b) {
    SeqInfo s;
    if (p.cu_q == nullptr) {
        s.q0 = b;
        s.n = 1;
    } else {
        const int a = min(max(p.cu_q[b], 0), (int)p.T), e = min(max(p.cu_q[b + 1], 0), (int)p.T);
        s.q0 = a;
        s.n = max(e - a, 0);
    }
    s.L = min(max(p.lens[b], 0), p.most);
    s.tiles = (int)(((uint32_t)(s.n * p.group) + R - 1) / R);
    return s;
}

// The query token of a row; its head follows from the rest.
__device__ __forceinline__ int row_token(const AttnParams& p, int row) {
    return (int)fastdiv((uint32_t)row, p.div_group);
}

// The first token that a query at this position sees.  Queries before the first token see none: all of
// them count as position -1, so that no window makes the difference wrap.
__device__ __forceinline__ int first_seen(const AttnParams& p, int pos) {
    return p.window > 0 ? max(pos, -1) + 1 - p.window : 0;
}

struct Span {
    int lo, hi;      // tokens that some row of the tile sees: [lo, hi)
    int t0, t1;      // token tiles, at least one
};

template <int R, int TN>
__device__ __forceinline__ Span row_tile_span(const AttnParams& p, const SeqInfo& s, int rt) {
    const int rows = s.n * p.group;
    const int first = row_token(p, rt * R), last = row_token(p, min((rt + 1) * R, rows) - 1);
    Span v;
    v.hi = p.causal ? max(0, min(s.L, s.L - s.n + last + 1)) : s.L;
    v.lo = max(0, first_seen(p, s.L - s.n + first));
    if (v.lo >= v.hi) v.lo = v.hi = 0;
    v.t0 = v.lo / TN;
    v.t1 = max((v.hi + TN - 1) / TN, v.t0 + 1);   // an empty tile still writes its rows
    return v;
}

template <int R, int TN>
__device__ __forceinline__ int64_t seq_units(const AttnParams& p, int b) {
    if (b >= p.B) return 0;
    const SeqInfo s = seq_info<R>(p, b);
    int64_t u = 0;
    for (int rt = 0; rt < s.tiles; ++rt) {
        const Span v = row_tile_span<R, TN>(p, s, rt);
        u += v.t1 - v.t0;
    }
    return u * p.c.heads;
}

// The walk over a block's run [u, u1): the current item and the part of it that is ours.
struct Walk {
    int64_t u, u1;         // global tile numbers
    int64_t item0;         // of the item's first tile
    int b, rt, head;
    SeqInfo s;
    Span v;
    int units;             // of the item
};

// Run i of `used` runs of `total` tiles begins at tile run_begin: the first total % used
// runs are one tile longer.
struct Runs {
    int64_t len, longer;   // tiles of a short run, number of long runs
};
__device__ __forceinline__ Runs make_runs(int64_t total, int used) {
    const int64_t len = div_short(total, used);
    return Runs{len, total - len * used};
}
__device__ __forceinline__ int64_t run_begin(const Runs& r, int i) { return r.len * i + min((int64_t)i, r.longer); }
// The run that holds tile u.
__device__ __forceinline__ int run_of(const Runs& r, int64_t u) {
    const int64_t edge = (r.len + 1) * r.longer;
    return (int)(u < edge ? div_short(u, r.len + 1) : r.longer + div_short(u - edge, r.len));
}

// Sum and inclusive prefix over a warp; 32-bit shuffles where no lane holds much.
__device__ __forceinline__ int64_t warp_sum(int64_t x) {
    if (__all_sync(0xffffffffu, x < (1 << 26))) return (int64_t)__reduce_add_sync(0xffffffffu, (uint32_t)x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}
__device__ __forceinline__ int64_t warp_prefix(int64_t x) {
    const int lane = threadIdx.x & 31;
    if (__all_sync(0xffffffffu, x < (1 << 26))) {
        int y = (int)x;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, y, off);
            if (lane >= off) y += v;
        }
        return y;
    }
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += v;
    }
    return x;
}

// Executed by a full warp.  How the tiles are cut into runs, and this block's walk.
template <int R, int TN>
__device__ __forceinline__ Runs walk_begin(const AttnParams& p, int block, int blocks, Walk& w) {
    const int lane = threadIdx.x & 31;
    int64_t total = 0, mine = 0;
    for (int64_t b0 = 0; b0 < p.B; b0 += 32) {
        mine = seq_units<R, TN>(p, (int)(b0 + lane));
        total += warp_sum(mine);
    }
    const int used = (int)min((int64_t)blocks, total);
    w.u = w.u1 = 0;
    if (block >= used) return Runs{0, 0};
    const Runs runs = make_runs(total, used);
    w.u = run_begin(runs, block);
    w.u1 = run_begin(runs, block + 1);
    int64_t base = 0;
    for (int64_t b0 = 0; b0 < p.B; b0 += 32) {
        if (p.B > 32) mine = seq_units<R, TN>(p, (int)(b0 + lane));
        const int64_t upto = warp_prefix(mine);
        const uint32_t m = __ballot_sync(0xffffffffu, base + upto > w.u);
        if (m) {
            const int l = __ffs(m) - 1;
            w.b = (int)b0 + l;
            w.item0 = base + __shfl_sync(0xffffffffu, upto - mine, l);
            break;
        }
        base += __shfl_sync(0xffffffffu, upto, 31);
    }
    // inside the sequence: row tile, then head
    w.s = seq_info<R>(p, w.b);
    for (w.rt = 0;; ++w.rt) {
        w.v = row_tile_span<R, TN>(p, w.s, w.rt);
        w.units = w.v.t1 - w.v.t0;
        const int64_t all = (int64_t)w.units * p.c.heads;
        if (w.item0 + all > w.u) break;
        w.item0 += all;
    }
    w.head = (int)div_short(w.u - w.item0, w.units);
    w.item0 += (int64_t)w.head * w.units;
    return runs;
}

// Past the current item's part; the next item if any of the run is left.
template <int R, int TN>
__device__ __forceinline__ void walk_next(const AttnParams& p, Walk& w) {
    w.item0 += w.units;
    w.u = w.item0;
    if (w.u >= w.u1) return;
    if (++w.head < p.c.heads) return;
    w.head = 0;
    if (++w.rt >= w.s.tiles) {
        w.rt = 0;
        do {
            w.s = seq_info<R>(p, ++w.b);
        } while (w.s.tiles == 0);
    }
    w.v = row_tile_span<R, TN>(p, w.s, w.rt);
    w.units = w.v.t1 - w.v.t0;
}

__device__ __forceinline__ int64_t safe_page(const AttnParams& p, int b, int entry) {
    const int64_t page = p.table[(int64_t)b * p.table_stride + entry];
    if (page >= 0 && page < p.c.num_pages) return page;
    atomicOr(p.status, DEVICE_INDEX);
    return 0;
}

// Workspace: arrival counters, one for each block, then two partial results for each
// block (the item it continues, the item it leaves unfinished): R rows of D sums in units of
// kSumUnit, then R pairs (maximum, sum of probabilities).
__host__ __device__ constexpr size_t attn_slot_floats(int R, int D) { return (size_t)R * (D + 2); }

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// Arrival on an item's counter: what this thread has written, or seen written through a
// barrier, is visible to whoever arrives later.
__device__ __forceinline__ uint32_t arrive_ticket(uint32_t* count) {
    uint32_t before;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(count) : "memory");
    return before;
}
// weight of a part with maximum m under the common maximum M (log2 domain)
__device__ __forceinline__ float part_weight(float m, float M) { return m == -INFINITY ? 0.0f : ex2(m - M); }

// Adds the partial results of an item, in the order of its tiles, and writes out and lse.
// Executed by NTHR threads (warps 0 .. NTHR / 32 - 1) of the last block to arrive, RB rows
// of the item's R at a time.  weights: shared, RB * 33 floats.
template <bool BF16, int D, int R, int RB, int NTHR>
__device__ __forceinline__ void merge_parts(const AttnParams& p, const Walk& w, int first_block, int parts,
                                            float* weights, int tid, uint32_t barrier) {
    constexpr int CH = D / 4;                       // float4 chunks of a row
    constexpr int PER = (RB * CH + NTHR - 1) / NTHR;
    constexpr int NW = NTHR / 32, RW = (RB + NW - 1) / NW;
    const int all = min(R, w.s.n * p.group - w.rt * R);
    const int warp = tid >> 5, lane = tid & 31;
    // the first part is what its block left unfinished, the others what theirs continued
    auto slot = [&](int j) {
        return p.ws_part + (size_t)(2 * (first_block + j) + (j == 0 ? 1 : 0)) * attn_slot_floats(R, D);
    };
    for (int r0 = 0; r0 < all; r0 += RB) {
        const int rows = min(RB, all - r0);
        float4 acc[PER];
        float lsum[RW], mrun[RW];
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < RW; ++k) lsum[k] = 0.f, mrun[k] = -INFINITY;
        for (int j0 = 0; j0 < parts; j0 += 32) {
            const int cnt = min(32, parts - j0);
#pragma unroll
            for (int k = 0; k < RW; ++k) {
                const int r = warp + k * NW;
                float2 ml = make_float2(-INFINITY, 0.f);
                if (lane < cnt && r < rows)
                    ml = __ldcg(reinterpret_cast<const float2*>(slot(j0 + lane) + R * D) + r0 + r);
                float M = fmaxf(ml.x, mrun[k]);
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
                const float f = part_weight(mrun[k], M), wt = part_weight(ml.x, M);
                float l = wt * ml.y;
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
                lsum[k] = lsum[k] * f + l;
                mrun[k] = M;
                if (r < RB) {
                    weights[r * 33 + lane] = wt;
                    if (lane == 0) weights[r * 33 + 32] = f;
                }
            }
            ptx::named_barrier_sync(barrier, NTHR);
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int idx = tid + i * NTHR, r = idx / CH, ch = idx % CH;
                if (r >= rows) continue;
                const float f = weights[r * 33 + 32];
                acc[i].x *= f, acc[i].y *= f, acc[i].z *= f, acc[i].w *= f;
#pragma unroll 8
                for (int j = 0; j < cnt; ++j) {
                    const float4 v = __ldcg(reinterpret_cast<const float4*>(slot(j0 + j)) + (r0 + r) * CH + ch);
                    const float wt = weights[r * 33 + j];
                    if (wt != 0.f) {   // a part that saw nothing holds nothing
                        acc[i].x += wt * v.x, acc[i].y += wt * v.y, acc[i].z += wt * v.z, acc[i].w += wt * v.w;
                    }
                }
            }
            ptx::named_barrier_sync(barrier, NTHR);
        }
#pragma unroll
        for (int k = 0; k < RW; ++k) {
            const int r = warp + k * NW;
            if (lane == 0 && r < rows) {
                weights[r * 33] = lsum[k];
                if (p.lse != nullptr) {
                    const int row = w.rt * R + r0 + r, qt = row_token(p, row);
                    p.lse[(int64_t)(w.s.q0 + qt) * p.Hq + w.head * p.group + row - qt * p.group] =
                        lsum[k] == 0.f ? -INFINITY : (mrun[k] + log2f(lsum[k])) * 0.6931471805599453f;
                }
            }
        }
        ptx::named_barrier_sync(barrier, NTHR);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int idx = tid + i * NTHR, r = idx / CH, ch = idx % CH;
            if (r >= rows) continue;
            const float l = weights[r * 33], inv = l == 0.f ? 0.f : kSumUnit<BF16> / l;
            const int row = w.rt * R + r0 + r, qt = row_token(p, row);
            uint16_t* out = static_cast<uint16_t*>(p.out) + (int64_t)(w.s.q0 + qt) * p.out_stride +
                            (w.head * p.group + row - qt * p.group) * D + ch * 4;
            *reinterpret_cast<uint2*>(out) = make_uint2(pack2<BF16>(acc[i].x * inv, acc[i].y * inv),
                                                        pack2<BF16>(acc[i].z * inv, acc[i].w * inv));
        }
        ptx::named_barrier_sync(barrier, NTHR);   // the weights may be written again
    }
}

}  // namespace wq
