// fa_chunk.cuh -- what the kernels over a paged cache share (attention of new tokens, key
// weights): a sequence's new tokens and keys, the split of the work over the CTAs, and the joining
// of partial rows.
//
// Rows. A key head serves G query heads, so the G * n (new token, query head) pairs of a sequence
// and key head are the rows that read the same K and V. Rows go in tiles of T = R / G whole tokens
// (at most R rows; row r is token r / G of the tile, head r % G of the group), so that a tile's Q is
// one box in memory; a work item is (sequence, key head, row tile), and its steps are the key tiles
// of BN keys that its last token sees (at least one, so that rows that see nothing are written
// too).
//
// Split. The steps of all items, in the order (sequence, key head, row tile, key tile), are cut
// into runs of equal cost, one per CTA, whatever items they fall into: a serving batch of one long
// and many short sequences then keeps every SM busy to the end, and a single sequence's keys are read
// by all of them. An item that falls into several runs leaves an unnormalised O with (m, l) for
// each piece in the workspace; chunk_combine_kernel joins the pieces in the order of the keys
// (fixed, so the same call gives the same bits). A CTA has at most two such pieces: the end of an
// item begun by an earlier CTA (slot 2 c) and the beginning of one that a later CTA finishes
// (slot 2 c + 1). Pieces lie column by column, [slot][D][R]: the writers hold a row per thread, so
// a store of one column is a run of consecutive floats.
#pragma once
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "fa_internal.h"
#include "fa_ptx.cuh"
#include "fa_sync.cuh"

namespace fa {

struct ChunkSeq {
    int q0, n, kv;  // first token row, new tokens, keys in the cache
};

// Sequence b; offsets and lengths outside the tensors or the table are cut to them.
__device__ __forceinline__ ChunkSeq chunk_seq(const ChunkParams &p, int b) {
    ChunkSeq s;
    const int c0 = __ldg(p.cu_seqlens + b), c1 = __ldg(p.cu_seqlens + b + 1), kv = __ldg(p.kv_lens + b);
    s.q0 = min(max(c0, 0), p.total);
    s.n = max(min(c1, p.total) - s.q0, 0);
    s.kv = min(max(kv, 0), p.capacity);
    return s;
}

// Reports offsets or lengths of sequence b that chunk_seq had to cut.
__device__ __forceinline__ void chunk_check(const ChunkParams &p, int b) {
    const int c0 = __ldg(p.cu_seqlens + b), c1 = __ldg(p.cu_seqlens + b + 1), kv = __ldg(p.kv_lens + b);
    if (c0 < 0 || c1 < c0 || c1 > p.total || kv < 0 || kv > p.capacity) record_error(FA_ERR_INDEX, 712);
}

// Keys that new token i sees: all of them, or (causal) those up to its own.
template <bool CAUSAL>
__device__ __forceinline__ int token_keys(const ChunkSeq &s, int i) {
    return CAUSAL ? max(0, s.kv - s.n + i + 1) : s.kv;
}

// Keys that the last of the tokens before `end` sees, and the steps of the tile that ends there.
template <bool CAUSAL>
__device__ __forceinline__ int tile_keys(const ChunkSeq &s, int end) {
    return token_keys<CAUSAL>(s, min(end, s.n) - 1);
}
template <int BN, bool CAUSAL>
__device__ __forceinline__ int tile_steps(const ChunkSeq &s, int end) {
    return max(1, (tile_keys<CAUSAL>(s, end) + BN - 1) / BN);
}
// log2 of the cost of a step of the tile of T tokens that begins at token i: a step that fills two
// MMA tiles (TILES = 2, T / 2 tokens each) costs twice as much as one that fills one.
template <int TILES>
__device__ __forceinline__ int step_shift(const ChunkSeq &s, int T, int i) {
    return (TILES == 2 && s.n - i > (T >> 1)) ? 1 : 0;
}

// a / b for a, b >= 0 (b > 0), in 32 bits where they fit (they nearly always do, and a 64-bit
// division is a long subroutine).
__device__ __forceinline__ int64_t div_up_or_down(int64_t a, int64_t b, bool up) {
    if (up) a += b - 1;
    if ((a | b) >> 32 == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// Where a CTA's run begins: the item in which cost `lo` falls, which begins at cost `pos`; an item costs
// ITEM (loading Q, the epilogue), then its steps. The run takes the steps that begin in [lo, hi); `per` is
// hi - lo of a whole run. (Without ITEM, CTAs whose runs hold several short items ended 35 % later
// than those with one: 9 sequences of up to 333 tokens over 2777.)
struct ChunkStart {
    int b, h, t;
    int64_t pos, lo, hi, per;
};

// Cost of an item: its tile begins at token i.
template <int TILES, int BN, int ITEM, bool CAUSAL>
__device__ __forceinline__ int64_t item_cost(const ChunkSeq &s, int T, int i) {
    return ITEM + (static_cast<int64_t>(tile_steps<BN, CAUSAL>(s, i + T)) << step_shift<TILES>(s, T, i));
}
// Cost of one key head of a sequence.
template <int TILES, int BN, int ITEM, bool CAUSAL>
__device__ __forceinline__ int64_t head_cost(const ChunkSeq &s, int T) {
    int64_t sum = 0;
    for (int i = 0; i < s.n; i += T) sum += item_cost<TILES, BN, ITEM, CAUSAL>(s, T, i);
    return sum;
}

__device__ __forceinline__ int64_t warp_sum64(int64_t v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ int64_t warp_scan64(int64_t v, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
    }
    return v;
}

// One warp finds CTA cta's run (out: shared memory, written by one lane). A few sequences (long prompts: many
// tiles each) are gone through one by one, a lane per tile; many (a serving batch) with four consecutive
// sequences per lane, so that up to 128 cost one round of loads. (A lane per sequence took 2 us more
// for one sequence of 32 tiles.)
template <int TILES, int BN, int ITEM, bool CAUSAL>
__device__ __forceinline__ void chunk_locate(const ChunkParams &p, int cta, int ctas, ChunkStart *out) {
    constexpr int PER = 4, FEW = 8;
    const int lane = threadIdx.x & 31, T = p.tile_tokens;
    const bool few = p.num_seqs <= FEW;
    int64_t cost[PER], total = 0, mine = 0;
    ChunkSeq own = chunk_seq(p, min(lane, p.num_seqs - 1));  // few: sequence `lane`
    auto seq_of = [&](int b) {
        return ChunkSeq{__shfl_sync(0xffffffffu, own.q0, b), __shfl_sync(0xffffffffu, own.n, b), __shfl_sync(0xffffffffu, own.kv, b)};
    };
    auto costs = [&](int base) {
        mine = 0;
        ChunkSeq s[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) s[i] = chunk_seq(p, min(base + lane * PER + i, p.num_seqs - 1));
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (base + lane * PER + i >= p.num_seqs) s[i].n = 0;
            cost[i] = head_cost<TILES, BN, ITEM, CAUSAL>(s[i], T) * p.Hkv;
            mine += cost[i];
        }
    };
    if (few) {  // mine: cost of a key head of sequence `lane`
        for (int b = 0; b < p.num_seqs; ++b) {
            const ChunkSeq s = seq_of(b);
            int64_t sum = 0;
            for (int i = lane * T; i < s.n; i += 32 * T) sum += item_cost<TILES, BN, ITEM, CAUSAL>(s, T, i);
            sum = warp_sum64(sum);
            total += sum * p.Hkv;
            if (lane == b) mine = sum;
        }
    } else {
        for (int base = 0; base < p.num_seqs; base += 32 * PER) {
            costs(base);
            total += warp_sum64(mine);
        }
    }
    if (cta == 0)
        for (int b = lane; b < p.num_seqs; b += 32) chunk_check(p, b);
    int64_t per = div_up_or_down(total, ctas, true);
    if (per < p.min_cost) per = p.min_cost;
    const int64_t start = per * cta, end = min(start + per, total);
    if (start >= total) {
        if (lane == 0) *out = ChunkStart{0, 0, 0, 0, 0, 0, per};
        return;
    }
    int64_t before = 0;
    if (few) {
        for (int b = 0; b < p.num_seqs; ++b) {
            const int64_t one = __shfl_sync(0xffffffffu, mine, b);
            if (start >= before + one * p.Hkv) {
                before += one * p.Hkv;
                continue;
            }
            const ChunkSeq s = seq_of(b);
            const int64_t h = div_up_or_down(start - before, one, false);
            int64_t pos = before + h * one;
            for (int t0 = 0; t0 * static_cast<int64_t>(T) < s.n; t0 += 32) {
                const int i = (t0 + lane) * T;
                const int64_t c = i < s.n ? item_cost<TILES, BN, ITEM, CAUSAL>(s, T, i) : 0;
                const int64_t incl = warp_scan64(c, lane), at = pos + incl - c;
                if (start >= at && start < at + c) *out = ChunkStart{b, static_cast<int>(h), t0 + lane, at, start, end, per};
                pos += __shfl_sync(0xffffffffu, incl, 31);
                if (start < pos) break;
            }
            break;
        }
        return;
    }
    for (int base = 0; base < p.num_seqs; base += 32 * PER) {
        if (p.num_seqs > 32 * PER) costs(base);
        const int64_t incl = warp_scan64(mine, lane);
        int64_t at = before + incl - mine;  // cost before this lane's sequences
        if (start >= at && start < at + mine) {
            int b = base + lane * PER;
            int64_t mine_b = cost[0];
#pragma unroll
            for (int i = 1; i < PER; ++i)
                if (start >= at + mine_b) {
                    at += mine_b;
                    mine_b = cost[i];
                    b = base + lane * PER + i;
                }
            const ChunkSeq s = chunk_seq(p, b);
            const int64_t one = div_up_or_down(mine_b, p.Hkv, false);
            const int64_t h = div_up_or_down(start - at, one, false);
            int64_t pos = at + h * one;
            int t = 0;
            for (int i = 0;; i += T, ++t) {
                const int64_t n = item_cost<TILES, BN, ITEM, CAUSAL>(s, T, i);
                if (start < pos + n) break;
                pos += n;
            }
            *out = ChunkStart{b, static_cast<int>(h), t, pos, start, end, per};
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
}

// A role's walk over its CTA's run: item after item, each the key tiles [j0, j1) of one row tile
// (tokens [i0, i0 + tokens) of the sequence).
template <int TILES, int BN, int ITEM, bool CAUSAL>
struct ChunkWalk {
    ChunkSeq s;
    int b, h, i0, j0, j1, steps, keys, tokens, shift;
    int64_t pos;
    const ChunkStart *run;  // in shared memory
    // false when the CTA has no work
    __device__ __forceinline__ bool begin(const ChunkParams &p, const ChunkStart *st) {
        run = st;
        if (st->lo >= st->hi) return false;
        b = st->b;
        h = st->h;
        i0 = st->t * p.tile_tokens;
        pos = st->pos;
        s = chunk_seq(p, b);
        set(p);
        if (j0 >= steps) return next(p);  // lo falls behind the start of the item's last step
        return j1 > j0;
    }
    __device__ __forceinline__ void set(const ChunkParams &p) {
        keys = tile_keys<CAUSAL>(s, i0 + p.tile_tokens);
        steps = max(1, (keys + BN - 1) / BN);
        tokens = min(p.tile_tokens, s.n - i0);
        shift = step_shift<TILES>(s, p.tile_tokens, i0);
        const int64_t round = (1 << shift) - 1;
        j0 = static_cast<int>(max(int64_t(0), run->lo - pos - ITEM + round) >> shift);
        j1 = static_cast<int>(min(static_cast<int64_t>(steps), max(int64_t(0), run->hi - pos - ITEM + round) >> shift));
    }
    // moves to the next item; false at the end of the run
    __device__ __forceinline__ bool next(const ChunkParams &p) {
        pos += ITEM + (static_cast<int64_t>(steps) << shift);
        if (pos >= run->hi) return false;
        i0 += p.tile_tokens;
        if (i0 >= s.n) {
            i0 = 0;
            if (++h == p.Hkv) {
                h = 0;
                do {
                    if (++b >= p.num_seqs) return false;
                    s = chunk_seq(p, b);
                } while (s.n == 0);
            }
        }
        set(p);
        return j1 > j0;  // (the run may end before the item's first step)
    }
    __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == steps; }
    // workspace slot of a piece that is not whole
    __device__ __forceinline__ int slot() const { return 2 * blockIdx.x + (j0 == 0 ? 1 : 0); }
    // The item begun here, for the joining: its pieces run up to the CTA in whose run its last step
    // begins (a run is at least as long as a step, so none between is empty).
    __device__ __forceinline__ ChunkDesc desc(const ChunkParams &p) const {
        const int64_t last = pos + ITEM + (static_cast<int64_t>(steps - 1) << shift);
        return ChunkDesc{static_cast<int>(div_up_or_down(last, run->per, false)) - static_cast<int>(blockIdx.x) + 1, s.q0 + i0,
                         tokens, h * p.G};
    }
};

// Cache row of key position pos (below the sequence's length) of sequence b. An entry outside the
// pool reads page 0 instead and sets `bad`.
__device__ __forceinline__ int chunk_page_row(const ChunkParams &p, int b, int pos, bool &bad) {
    int pg = __ldg(p.block_table + static_cast<int64_t>(b) * p.max_blocks + (pos >> p.page_shift));
    if (pg < 0 || pg >= p.num_pages) {
        bad = true;
        pg = 0;
    }
    return (pg << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
}

// A producer warp's walk over the key tiles of its CTA's run, one tile ahead in the block table: lane i holds
// the cache row of the tile's position i << piece_log (2^piece_log rows, which lie in one page). The table's entries of the
// next tile are asked for before the current one's copies are issued; looked up when they were needed,
// they cost half a microsecond a part, more than a small tile's arithmetic.
template <typename Walk, int BN>
struct ChunkTiles {
    Walk w;
    int h, valid, row, piece_log;  // the current tile: key head, its keys, this lane's cache row
    int j, ahead;
    bool more, bad;
    __device__ __forceinline__ ChunkTiles(const ChunkParams &p, const ChunkStart *run, int log) : piece_log(log), bad(false) {
        more = w.begin(p, run);
        j = more ? w.j0 : 0;
        look(p);
    }
    __device__ __forceinline__ void look(const ChunkParams &p) {
        const int in = (threadIdx.x & 31) << piece_log, pos = j * BN + in;
        ahead = more && in < BN && pos < w.keys ? __ldg(p.block_table + static_cast<int64_t>(w.b) * p.max_blocks + (pos >> p.page_shift)) : 0;
    }
    // takes the next tile; false at the end of the run
    __device__ __forceinline__ bool take(const ChunkParams &p) {
        if (!more) return false;
        h = w.h;
        valid = min(BN, w.keys - j * BN);
        int pg = ahead;
        if (pg < 0 || pg >= p.num_pages) {
            bad = true;
            pg = 0;
        }
        row = (pg << p.page_shift) + ((j * BN + ((threadIdx.x & 31) << piece_log)) & ((1 << p.page_shift) - 1));
        if (++j >= w.j1) {
            more = w.next(p);
            j = more ? w.j0 : 0;
        }
        look(p);
        return true;
    }
};

// How a lane takes part in the copies of a tile's part: NB column blocks of ROWS rows in boxes of 2^log rows,
// one box per lane (there are never more than 16); lanes past the part's boxes copy nothing. All of it is
// the same for every tile, so a part costs the issuing warp a shuffle and the copy (with the divisions in
// the loop it took half a microsecond a part, and tiles of D = 64 waited for it).
template <int NB, int ROWS, int SW>
struct BoxLane {
    int log, box, blk, dst, from;  // rows of a box, this lane's box and block, its bytes' place, row's lane
    __device__ __forceinline__ BoxLane(int page_shift, int piece_log, int r0 = 0) {
        static_assert((ROWS & (ROWS - 1)) == 0 && (ROWS / 16) * NB <= 32, "a lane per box");
        const int lane = threadIdx.x & 31;
        log = min(page_shift, ROWS == 128 ? 7 : 6);
        static_assert(ROWS == 128 || ROWS == 64, "rows of a part");
        box = lane / NB;
        blk = lane % NB;
        dst = (blk * ROWS + (box << log)) * SW;
        from = ((r0 + (box << log)) >> piece_log) & 31;
    }
    __device__ __forceinline__ int boxes(int have) const { return (min(max(have, 0), ROWS) + (1 << log) - 1) >> log; }
    __device__ __forceinline__ uint32_t bytes(int n) const { return static_cast<uint32_t>(n << log) * (NB * SW); }
};

__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Joins the pieces of the item that CTA blockIdx.x began and did not finish: m = max of the pieces', l
// and O summed with each piece scaled by 2^(m_i - m), the maximum running as in the attention itself; NaN in a
// piece's l or O stays NaN. A lane
// takes four neighbouring rows (one 16-byte load of a column), a warp LR * 4 rows and CL columns at a load;
// the loads of several pieces are issued together, before anything is known of the pieces (what the joining
// takes is latency: one load after another, it took 6 us for four pieces of 16 rows and 20 us for two of
// 256). Launched with programmatic dependence: it waits on the device for the attention kernel's
// end, so its launch costs no gap.
template <int D, bool BF16, int R>
struct CombineCfg {
    static constexpr int LR = R / 4 < 32 ? R / 4 : 32, CL = 32 / LR;  // lanes for rows, columns of a load
    static constexpr int LOADS = CL == 1 ? 8 : 2, COLS = CL * LOADS;  // of a warp
    static constexpr int AHEAD = CL == 1 ? 2 : 4;                     // pieces in flight
    static constexpr int UNITS = (R / (4 * LR)) * (D / COLS);         // warps' work of a whole tile
    static_assert(D % COLS == 0, "columns of a warp");
};
template <int D, bool BF16, int R>
__global__ void __launch_bounds__(256) chunk_combine_kernel(const ChunkParams p) {
    using C = CombineCfg<D, BF16, R>;
    constexpr int CL = C::CL, LOADS = C::LOADS;
    const int lane = threadIdx.x & 31, lr = lane % C::LR, cl = lane / C::LR;
    const int unit = blockIdx.y * 8 + (threadIdx.x >> 5);
    const int c0 = (unit % (D / C::COLS)) * C::COLS + cl, r0 = (unit / (D / C::COLS)) * (4 * C::LR) + lr * 4;
    pdl_wait();
    const ChunkDesc d = p.desc[blockIdx.x];
    if (d.pieces < 2 || unit >= C::UNITS) return;
    auto slot = [&](int k) { return static_cast<int64_t>(k == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + k)); };
    auto stats = [&](int k, float *m, float *l) {  // of rows r0 .. r0 + 3
        const float4 *q = reinterpret_cast<const float4 *>(p.part_ml + slot(k) * R + r0);
        const float4 a = q[0], b = q[1];
        m[0] = a.x; l[0] = a.y; m[1] = a.z; l[1] = a.w;
        m[2] = b.x; l[2] = b.y; m[3] = b.z; l[3] = b.w;
    };
    float m[4], l[4] = {0.f, 0.f, 0.f, 0.f}, acc[LOADS][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = -INFINITY;
#pragma unroll
    for (int c = 0; c < LOADS; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[c][i] = 0.f;
#pragma unroll 1
    for (int k = 0; k < d.pieces; k += C::AHEAD) {
        float4 v[C::AHEAD][LOADS];
        float pm[C::AHEAD][4], pl[C::AHEAD][4];
#pragma unroll
        for (int q = 0; q < C::AHEAD; ++q) {
            const int kq = min(k + q, d.pieces - 1);
            stats(kq, pm[q], pl[q]);
            const float *o = p.part_o + (slot(kq) * D + c0) * R + r0;
#pragma unroll
            for (int c = 0; c < LOADS; ++c) v[q][c] = *reinterpret_cast<const float4 *>(o + c * CL * R);
        }
#pragma unroll
        for (int q = 0; q < C::AHEAD; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // a piece in which the row saw nothing (l = 0), or that was read twice, adds nothing. (Its m does not
                // say so: the maximum passes over NaN, and a piece of NaN scores alone has m = -inf beside l = NaN.)
                if (k + q >= d.pieces || pl[q][i] == 0.f) continue;
                const float to = fmaxf(m[i], pm[q][i]);
                const float a0 = ex2_approx(m[i] - to), a1 = ex2_approx(pm[q][i] - to);  // (2^-inf = 0 at the first)
                m[i] = to;
                l[i] = fmaf(l[i], a0, pl[q][i] * a1);
#pragma unroll
                for (int c = 0; c < LOADS; ++c)
                    acc[c][i] = fmaf(acc[c][i], a0, a1 * (i == 0 ? v[q][c].x : (i == 1 ? v[q][c].y : (i == 2 ? v[q][c].z : v[q][c].w))));
            }
    }
    // row r of the tile: token and head (rows past the last token of an MMA tile are nobody's)
    const int half = R / p.mma_tiles, T = p.tile_tokens / p.mma_tiles;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = r0 + i, sub = r / half, rr = r - sub * half, ti = rr / p.G, tk = sub * T + ti;
        if (ti >= T || tk >= d.tokens) continue;
        const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
        const int64_t tok = d.token + tk;
        const int head = d.head + rr - ti * p.G;
        uint16_t *out = static_cast<uint16_t *>(p.out) + (tok * p.Hq + head) * D + c0;
        if constexpr (CL == 1) {
#pragma unroll
            for (int c = 0; c < LOADS; c += 4) {
                uint32_t x[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float lo = acc[c + 2 * q][i] * inv, hi = acc[c + 2 * q + 1][i] * inv;
                    x[q] = BF16 ? pack2_bf16(lo, hi) : pack2_f16(lo, hi);
                }
                *reinterpret_cast<uint2 *>(out + c) = make_uint2(x[0], x[1]);
            }
        } else {
#pragma unroll
            for (int c = 0; c < LOADS; ++c) {
                const uint32_t x = BF16 ? pack2_bf16(acc[c][i] * inv, 0.f) : pack2_f16(acc[c][i] * inv, 0.f);
                out[c * CL] = static_cast<uint16_t>(x);
            }
        }
        if (p.lse && c0 == 0)
            p.lse[static_cast<int64_t>(head) * p.total + tok] = l[i] == 0.f ? -INFINITY : m[i] * 0.6931471805599453f + logf(l[i]);
    }
}

template <int D, bool BF16, int R>
static cudaError_t launch_combine(const ChunkParams &p, int ctas, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, (CombineCfg<D, BF16, R>::UNITS + 7) / 8, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, chunk_combine_kernel<D, BF16, R>, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace fa
