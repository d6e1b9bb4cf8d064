// fa_chunk.cuh -- what the kernels over a paged cache share (attention of new tokens, key
// weights): a sequence's new tokens and keys, the split of the work over the CTAs, and the joining
// of partial rows.
//
// Rows. A key head serves G query heads, so the G * n (new token, query head) pairs of a sequence
// and key head are the rows that read the same K and V: row r is token r / G, head r % G of the
// group. Rows go in tiles of R; a work item is (sequence, key head, row tile), and its steps are
// the key tiles of BN keys that its last row sees (at least one, so that rows that see nothing
// are written too).
//
// Split. The steps of all items, in the order (sequence, key head, row tile, key tile), are cut
// into runs of equal cost, one per CTA, whatever items they fall into: a serving batch of one long and
// many short sequences then keeps every SM busy to the end, and a single sequence's keys are read
// by all of them. An item that falls into several runs leaves an unnormalised O with (m, l) for
// each piece in the workspace; chunk_combine_kernel joins the pieces in the order of the keys
// (fixed, so the same call gives the same bits). A CTA has at most two such pieces: the end of an
// item begun by an earlier CTA (slot 2 c) and the beginning of one that a later CTA finishes
// (slot 2 c + 1).
#pragma once
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "fa_internal.h"
#include "fa_ptx.cuh"
#include "fa_sync.cuh"

namespace fa {

struct ChunkSeq {
    int q0, n, rows, kv;  // first token row, new tokens, n * G, keys in the cache
};

// Sequence b; offsets and lengths outside the tensors or the table are cut to them.
__device__ __forceinline__ ChunkSeq chunk_seq(const ChunkParams &p, int b) {
    ChunkSeq s;
    const int c0 = __ldg(p.cu_seqlens + b), c1 = __ldg(p.cu_seqlens + b + 1), kv = __ldg(p.kv_lens + b);
    s.q0 = min(max(c0, 0), p.total);
    s.n = max(min(c1, p.total) - s.q0, 0);
    s.rows = s.n * p.G;
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

// Keys that the last row of tile t sees, and the tile's steps.
template <int R, bool CAUSAL>
__device__ __forceinline__ int tile_keys(const ChunkParams &p, const ChunkSeq &s, int t) {
    return token_keys<CAUSAL>(s, (min((t + 1) * R, s.rows) - 1) / p.G);
}
template <int R, int BN, bool CAUSAL>
__device__ __forceinline__ int tile_steps(const ChunkParams &p, const ChunkSeq &s, int t) {
    return max(1, (tile_keys<R, CAUSAL>(p, s, t) + BN - 1) / BN);
}
// Cost of a step of tile t: 2 where the tile fills more than one 128-row MMA tile, else 1.
template <int R>
__device__ __forceinline__ int tile_weight(const ChunkSeq &s, int t) {
    return (R > 128 && s.rows - t * R > 128) ? 2 : 1;
}

// Where a CTA's run begins: the item in which cost `lo` falls, whose own steps begin at cost `pos`.
// The run takes the steps that begin in [lo, hi); `per` is hi - lo of a whole run.
struct ChunkStart {
    int b, h, t;
    int64_t pos, lo, hi, per;
};

// Cost of one key head of a sequence.
template <int R, int BN, bool CAUSAL>
__device__ __forceinline__ int64_t head_cost(const ChunkParams &p, const ChunkSeq &s) {
    const int tiles = (s.rows + R - 1) / R;
    int64_t sum = 0;
    for (int t = 0; t < tiles; ++t) sum += tile_steps<R, BN, CAUSAL>(p, s, t) * tile_weight<R>(s, t);
    return sum;
}

__device__ __forceinline__ int64_t warp_sum64(int64_t v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// One warp finds CTA cta's run (out: shared memory, written by one lane). Each lane takes four
// consecutive sequences at a time, so up to 128 sequences cost one round of loads.
template <int R, int BN, bool CAUSAL>
__device__ __forceinline__ void chunk_locate(const ChunkParams &p, int cta, int ctas, ChunkStart *out) {
    constexpr int PER = 4;
    const int lane = threadIdx.x & 31;
    int64_t cost[PER], total = 0, mine = 0;
    auto costs = [&](int base) {
        mine = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int b = base + lane * PER + i;
            cost[i] = b < p.num_seqs ? head_cost<R, BN, CAUSAL>(p, chunk_seq(p, b)) * p.Hkv : 0;
            mine += cost[i];
        }
    };
    for (int base = 0; base < p.num_seqs; base += 32 * PER) {
        costs(base);
        total += warp_sum64(mine);
    }
    if (cta == 0)
        for (int b = lane; b < p.num_seqs; b += 32) chunk_check(p, b);
    int64_t per = (total + ctas - 1) / ctas;
    if (per < p.min_steps) per = p.min_steps;
    const int64_t start = per * cta;
    if (start >= total) {
        if (lane == 0) *out = ChunkStart{0, 0, 0, 0, 0, 0, per};
        return;
    }
    int64_t before = 0;
    for (int base = 0; base < p.num_seqs; base += 32 * PER) {
        if (p.num_seqs > 32 * PER) costs(base);
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        int64_t at = before + incl - mine;  // steps before this lane's sequences
        if (start >= at && start < at + mine) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                if (start >= at && start < at + cost[i]) {
                    const int b = base + lane * PER + i;
                    const ChunkSeq s = chunk_seq(p, b);
                    const int64_t one = cost[i] / p.Hkv;
                    const int h = static_cast<int>((start - at) / one);
                    int64_t pos = at + h * one;
                    int t = 0;
                    for (;; ++t) {
                        const int64_t n = static_cast<int64_t>(tile_steps<R, BN, CAUSAL>(p, s, t)) * tile_weight<R>(s, t);
                        if (start < pos + n) break;
                        pos += n;
                    }
                    *out = ChunkStart{b, h, t, pos, start, min(start + per, total), per};
                }
                at += cost[i];
            }
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
}

// A role's walk over its CTA's run: item after item, each the key tiles [j0, j1) of one row tile.
template <int R, int BN, bool CAUSAL>
struct ChunkWalk {
    ChunkSeq s;
    int b, h, t, j0, j1, steps, keys, tiles, rows, weight;  // rows: valid rows of the tile
    int64_t pos, lo, hi;
    // false when the CTA has no work
    __device__ __forceinline__ bool begin(const ChunkParams &p, const ChunkStart &st) {
        lo = st.lo;
        hi = st.hi;
        if (lo >= hi) return false;
        b = st.b;
        h = st.h;
        t = st.t;
        pos = st.pos;
        s = chunk_seq(p, b);
        tiles = (s.rows + R - 1) / R;
        set(p);
        return j0 < steps || next(p);  // lo may fall behind the start of the item's last step
    }
    __device__ __forceinline__ void set(const ChunkParams &p) {
        keys = tile_keys<R, CAUSAL>(p, s, t);
        steps = max(1, (keys + BN - 1) / BN);
        rows = min(R, s.rows - t * R);
        weight = tile_weight<R>(s, t);
        j0 = static_cast<int>(max(int64_t(0), lo - pos + weight - 1) / weight);
        j1 = static_cast<int>(min(static_cast<int64_t>(steps), (hi - pos + weight - 1) / weight));
    }
    // moves to the next item; false at the end of the run
    __device__ __forceinline__ bool next(const ChunkParams &p) {
        pos += static_cast<int64_t>(steps) * weight;
        if (pos >= hi) return false;
        if (++t == tiles) {
            t = 0;
            if (++h == p.Hkv) {
                h = 0;
                do {
                    if (++b >= p.num_seqs) return false;
                    s = chunk_seq(p, b);
                } while (s.rows == 0);
                tiles = (s.rows + R - 1) / R;
            }
        }
        set(p);
        return true;
    }
    __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == steps; }
    // workspace slot of a piece that is not whole
    __device__ __forceinline__ int slot() const { return 2 * blockIdx.x + (j0 == 0 ? 1 : 0); }
    // pieces of the item begun here: runs up to the one in which its last step begins (a run is
    // at least as long as a step, so none between is empty)
    __device__ __forceinline__ int pieces(int64_t per) const {
        return static_cast<int>((pos + static_cast<int64_t>(steps - 1) * weight) / per) - static_cast<int>(blockIdx.x) + 1;
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

__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Joins the pieces of the item that CTA blockIdx.x began and did not finish, rows
// [blockIdx.y * 8, +8) of the tile, a row per warp: m = max of the pieces', l and O summed with
// each piece scaled by 2^(m_i - m). Launched with programmatic dependence: it waits on the device
// for the attention kernel's end, so its launch costs no gap.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) chunk_combine_kernel(const ChunkParams p, int R) {
    pdl_wait();
    const int4 d = p.desc[blockIdx.x];  // sequence, key head, row tile, pieces
    if (d.w < 2) return;
    const int r = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const ChunkSeq s = chunk_seq(p, d.x);
    const int row = d.z * R + r;
    if (r >= R || row >= s.rows) return;
    auto slot = [&](int i) { return static_cast<int64_t>(i == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + i)) * R + r; };
    float m = -INFINITY;
    for (int i = lane; i < d.w; i += 32) m = fmaxf(m, p.part_ml[slot(i)].x);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    constexpr int CPL = D / 32;  // columns a lane
    float acc[CPL], l = 0.f;
#pragma unroll
    for (int k = 0; k < CPL; ++k) acc[k] = 0.f;
    if (m != -INFINITY) {
#pragma unroll 4
        for (int i = 0; i < d.w; ++i) {
            const float2 ml = p.part_ml[slot(i)];
            const float a = ex2_approx(ml.x - m);  // a piece that saw nothing: 2^-inf = 0
            l = fmaf(ml.y, a, l);
            const float *o = p.part_o + slot(i) * D;
            if constexpr (CPL == 1) {
                acc[0] = fmaf(o[lane], a, acc[0]);
            } else {
#pragma unroll
                for (int k = 0; k < CPL / 2; ++k) {
                    const float2 v = *reinterpret_cast<const float2 *>(o + k * 64 + 2 * lane);
                    acc[2 * k] = fmaf(v.x, a, acc[2 * k]);
                    acc[2 * k + 1] = fmaf(v.y, a, acc[2 * k + 1]);
                }
            }
        }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const int64_t tok = s.q0 + row / p.G;
    const int head = d.y * p.G + row % p.G;
    uint16_t *out = static_cast<uint16_t *>(p.out) + (tok * p.Hq + head) * D;
    if constexpr (CPL == 1) {
        const uint32_t u = BF16 ? pack2_bf16(acc[0] * inv, 0.f) : pack2_f16(acc[0] * inv, 0.f);
        out[lane] = static_cast<uint16_t>(u);
    } else {
#pragma unroll
        for (int k = 0; k < CPL / 2; ++k) {
            const float x = acc[2 * k] * inv, y = acc[2 * k + 1] * inv;
            *reinterpret_cast<uint32_t *>(out + k * 64 + 2 * lane) = BF16 ? pack2_bf16(x, y) : pack2_f16(x, y);
        }
    }
    if (p.lse && lane == 0)
        p.lse[static_cast<int64_t>(head) * p.total + tok] = l > 0.f ? m * 0.6931471805599453f + logf(l) : -INFINITY;
}

template <int D, bool BF16>
static cudaError_t launch_combine(const ChunkParams &p, int R, int ctas, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, (R + 7) / 8, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, chunk_combine_kernel<D, BF16>, p, R);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace fa
