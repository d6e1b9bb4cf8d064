// fa_chunk_tile.cu -- attention of new tokens over a paged cache where a key head has many rows
// (fa_fwd_paged_chunk; prompt chunks): tiles of 128 rows on the tensor core.
//
// Rows are (new token, query head of the group), so a tile of a call with shared key heads holds
// 128 / G tokens (whole ones: G = 6 fills 126 rows) and every K/V tile that is loaded serves all of
// them. A CTA walks its run of steps
// (fa_chunk.cuh), each one 128-key tile against two 128-row tiles A and B (one at D = 256, where two
// O accumulators do not fit in TMEM), with the roles of the dense forward:
//   warps 0-3, 4-7  softmax of tile A, B: a thread per row; running maximum and sum in registers, P
//                   16-bit into TMEM (over S, or into columns of its own at D <= 64 so that the next
//                   S can be computed meanwhile), O rescaled in TMEM when the maximum grew by 2^8.
//   warp 8          K/V tiles by TMA, a box per page piece, the lanes issuing side by side.
//   warp 9          tcgen05.mma: S_t = Q_t K^T, O_t += P_t V, A and B in turn, so that the tensor core
//                   works on one while the softmax of the other runs. (An item of one row tile: A and B are
//                   its even and odd key tiles.) Before an item's last PV it clears
//                   the rows of V past the last key.
//   warp 10         D <= 64: issues the PVs (warp 9 then the QKs only).
//   warp 11         Q tiles by TMA, each once the last item's QKs have read its buffer.
// Rows of a tile past the sequence's last are computed on whatever lies there and not stored; a
// softmax warp without a row skips the exponentials. An item that the split cuts leaves O, m and l in the workspace.
//
// Bound, as the dense forward, by softmax and MMAs waiting for one another (both pipes 54 % busy); measured with
// the joining: 2048 tokens over 8192 keys (32 heads on 8, D = 128) 220 to 240 us in short runs, 1.0 to 1.09 PFLOP/s (fa_fwd on a
// problem of the same products 1.16), 254 us, 0.95 PFLOP/s, over seconds, when the power cap lowers the clock; first scores
// after 6, joining 14. 9 sequences of up to 333 tokens over 2777 (D = 64) 51 us: first scores after 5, CTAs that end up to 5
// apart, joining 9. P in 16 bits makes the error of out against 64 bits 1.4 times that of the output's rounding alone (bf16 2.3e-3
// beside 1.7e-3).
#include "fa_chunk.cuh"
#include "fa_fwd_kernel.cuh"

namespace fa {

namespace {

// Shared-memory map, TMEM columns and register split: those of the dense forward (Cfg); the barrier
// area holds this kernel's barriers and the run's start.
template <int D>
struct TileCfg : Cfg<D> {
    using B = Cfg<D>;
    static constexpr int R = B::BM * B::MAXQ;
    static constexpr int ITEM = 2;  // an item's cost besides its steps (about 2 us; a step of one tile takes 1)
    static constexpr int BARS = 2 + 2 + 2 * B::NS + 2 + 2 + 2 + 2 + 1 + 2;
    static constexpr int OFF_START = B::OFF_BAR + BARS * 8;
    static constexpr int OFF_TMEM = OFF_START + static_cast<int>(sizeof(ChunkStart));
    static_assert(BARS * 8 + sizeof(ChunkStart) + 8 <= 512, "barrier area");
    static constexpr int OFF_ML = B::USED;  // (m, l) of the odd key tiles' rows (128)
    static constexpr int OFF_WALK = OFF_ML + 1024;  // the softmax warps' walks
    static constexpr int END = OFF_WALK + B::NUM_SOFTMAX_WARPS * 64 + 1024;
    static constexpr int SMEM = END > B::SMEM_BYTES ? END : B::SMEM_BYTES;
    static_assert(OFF_TMEM + 8 <= OFF_ML && SMEM <= 227 * 1024, "shared memory");
};

template <int D, bool BF16, bool CAUSAL>
__global__ void __launch_bounds__(TileCfg<D>::NUM_THREADS, 1)
chunk_tile_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const ChunkParams p) {
    using C = TileCfg<D>;
    using Walk = ChunkWalk<C::MAXQ, C::BN, C::ITEM, CAUSAL>;
    constexpr int BM = C::BM, BN = C::BN, SW = C::SW, NS = C::NS, U = C::UNITS;
    constexpr bool SINGLE = C::MAXQ == 1, DEC = C::DECOUPLED;
    constexpr int CPB = SW / 16;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sQ = smem + C::OFF_Q, *sKV = smem + C::OFF_KV;
    uint64_t *q_full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *q_free = q_full + 2, *kv_full = q_free + 2, *kv_empty = kv_full + NS, *s_full = kv_empty + NS;
    uint64_t *p_full = s_full + 2, *pv_done = p_full + 2, *s_free = pv_done + 2, *drain = s_free + 2;
    uint64_t *x_full = drain + 1, *x_free = x_full + 1;  // split keys: B's results are there, are read
    float2 *sML = reinterpret_cast<float2 *>(smem + C::OFF_ML);
    ChunkStart *start = reinterpret_cast<ChunkStart *>(smem + C::OFF_START);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_TMEM);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_TMEM + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint64_t lim = p.timeout_ns;
    constexpr int W_TMA = C::WARP_TMA, W_MMA = C::WARP_MMA, W_PV = C::WARP_MMA + 1, W_Q = C::WARP_MMA + 2;

    pdl_launch_dependents();
    if (threadIdx.x == 32 * W_TMA) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(&q_full[t], 1);
            mbar_init(&q_free[t], 1);
            mbar_init(&s_full[t], 1);
            mbar_init(&p_full[t], 128);
            mbar_init(&pv_done[t], 1);
            mbar_init(&s_free[t], 4);
        }
        for (int s = 0; s < NS; ++s) {
            mbar_init(&kv_full[s], 1);
            mbar_init(&kv_empty[s], 1);
        }
        mbar_init(drain, DEC ? 2 : 1);
        mbar_init(x_full, 128);
        mbar_init(x_free, 128);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    if (warp == W_MMA) {
        tmem_alloc(tmem_slot, C::TMEM_COLS);
        tmem_relinquish();
    }
    if (warp == 0) chunk_locate<C::MAXQ, BN, C::ITEM, CAUSAL>(p, blockIdx.x, gridDim.x, start);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const int TT = p.tile_tokens / C::MAXQ;  // tokens of an MMA tile

    if (warp >= C::NUM_SOFTMAX_WARPS) {
        if constexpr (C::SPLIT_REGS) regs_dec<C::regs_low(false)>();
        Walk w;
        if (warp == W_TMA) {
            // ------------------------------------------------------------ K/V producer
            bool ok = true;
            int u = 0;  // ring parts issued
            const uint64_t pol = l2_policy_evict_last();
            constexpr int VR = C::VROWS_PER_UNIT, KB = C::KBLK_PER_UNIT;
            const int log = min(p.page_shift, VR == 64 ? 6 : 7);
            ChunkTiles<Walk, BN> tiles(p, start, log);
            const BoxLane<KB, BN, SW> bk(p.page_shift, log);      // a part of K_j: KB column blocks of all rows
            const BoxLane<C::NBLK, VR, SW> bv(p.page_shift, log);  // a part of V_j: VR rows of all blocks
            auto begin = [&](int stage, uint32_t bytes) {
                if (u >= NS && !__all_sync(0xffffffffu, wait_bounded(&kv_empty[stage], ((u / NS) - 1) & 1, abort_flag, lim, 750)))
                    return false;
                if (lane == 0) mbar_arrive_expect_tx(&kv_full[stage], bytes);
                __syncwarp();
                return true;
            };
            while (ok && tiles.take(p)) {
                const int nk = bk.boxes(tiles.valid), row_k = __shfl_sync(0xffffffffu, tiles.row, bk.from);
#pragma unroll
                for (int sub = 0; sub < U; ++sub, ++u) {
                    const int stage = u % NS;
                    if (!(ok = ok && begin(stage, bk.bytes(nk)))) break;
                    if (bk.box < nk)
                        tma_load_3d(sKV + stage * C::UNIT_BYTES + bk.dst, &tm_k, &kv_full[stage], (sub * KB + bk.blk) * C::SWE,
                                    tiles.h, row_k, pol);
                }
#pragma unroll
                for (int sub = 0; sub < U; ++sub, ++u) {
                    const int stage = u % NS, nv = bv.boxes(tiles.valid - sub * VR);
                    const int row_v = __shfl_sync(0xffffffffu, tiles.row, (bv.from + ((sub * VR) >> log)) & 31);
                    if (!(ok = ok && begin(stage, bv.bytes(nv)))) break;
                    if (bv.box < nv)
                        tma_load_3d(sKV + stage * C::UNIT_BYTES + bv.dst, &tm_v, &kv_full[stage], bv.blk * C::SWE, tiles.h, row_v, pol);
                }
            }
            if (__any_sync(0xffffffffu, tiles.bad) && lane == 0) record_error(FA_ERR_INDEX, 751);
            if (*abort_flag) {  // the copies in flight land before the shared memory goes away
                for (int v = max(0, u - NS); v < u; ++v) {
                    const uint64_t t0 = global_timer_ns();
                    while (!mbar_try_wait(&kv_full[v % NS], (v / NS) & 1) && global_timer_ns() - t0 < lim) {
                    }
                }
            }
        } else if (warp == W_MMA || (DEC && warp == W_PV)) {
            // ------------------------------------------------------------ MMA issuer(s)
            bool ok = true;
            int u0 = 0, nq[2] = {0, 0};
            int ga = 0, gb = 0;  // running key steps of tiles A, B
            auto wait = [&](uint64_t *bar, uint32_t ph, int where) {
                if (ok) ok = __all_sync(0xffffffffu, wait_bounded(bar, ph, abort_flag, lim, where));
                return ok;
            };
            // S_t = Q_qt K_jj^T, the tile's step ts; `first`: the first tile to use this K, `last`: the last
            auto qk = [&](int t, int qt, int jj, int ts, bool first, bool last, bool item_end) {
                const int gs = (t ? gb : ga) + ts, buf = SINGLE ? (gs & 1) : t;
                if (jj == 0 && !wait(&q_full[qt], nq[qt] & 1, 760 + qt)) return;
                if (DEC && gs > 0 && !wait(&s_free[t], (gs - 1) & 1, 762 + t)) return;
                tc_fence_after_sync();
                constexpr uint32_t idesc = idesc_f16(BM, BN, BF16, false), dhi = smem_desc_hi(8 * SW, C::LAYOUT);
                const uint32_t q_lo = smem_desc_lo(smem_u32(sQ + qt * C::Q_BYTES), 16);
                constexpr int UK = D / 16 / U;
#pragma unroll
                for (int un = 0; un < U; ++un) {
                    const int part = u0 + 2 * jj * U + un, stage = part % NS;
                    if (first) {
                        if (!wait(&kv_full[stage], (part / NS) & 1, 764)) return;
                        tc_fence_after_sync();
                    }
                    const uint32_t k_lo = smem_desc_lo(smem_u32(sKV + stage * C::UNIT_BYTES), 16);
#pragma unroll
                    for (int kk = 0; kk < UK; ++kk) {
                        const int k = un * UK + kk;
                        const uint32_t blk = (k * 32) / SW, off = (k * 32) % SW, lb = blk - un * C::KBLK_PER_UNIT;
                        umma_ss_elect(tmem + buf * BN, q_lo + ((blk * BM * SW + off) >> 4), k_lo + ((lb * BN * SW + off) >> 4), dhi,
                                      idesc, k > 0 ? 1u : 0u);
                    }
                    if (un + 1 == U) umma_commit_elect(&s_full[buf]);
                    if (last) umma_commit_elect(&kv_empty[stage]);
                }
                if (item_end) umma_commit_elect(&q_free[qt]);
            };
            // O_t += P_t V_jj; valid < BN: V_jj's rows from `valid` on are past the last key and are
            // cleared first (what the page or the ring holds there may be NaN, and 0 NaN = NaN)
            auto pv = [&](int t, int jj, int ts, bool first, bool last, int valid) {
                const int gs = (t ? gb : ga) + ts, buf = SINGLE ? (gs & 1) : t;
                const int part0 = u0 + (2 * jj + 1) * U;
                if (first) {
#pragma unroll
                    for (int un = 0; un < U; ++un) {
                        const int part = part0 + un, stage = part % NS;
                        if (!wait(&kv_full[stage], (part / NS) & 1, 768)) return;
                        if (valid >= BN) continue;
                        const uint32_t dst = smem_u32(sKV + stage * C::UNIT_BYTES);
                        const int r0 = max(0, valid - un * C::VROWS_PER_UNIT);
                        constexpr int CPR = D / 8;  // whole swizzled rows: the order of their chunks does not matter
                        for (int i = lane; i < (C::VROWS_PER_UNIT - r0) * CPR; i += 32) {
                            const int r = r0 + i / CPR, ch = i % CPR;
                            st_shared_v4(dst + (ch / CPB) * C::VROWS_PER_UNIT * SW + r * SW + (ch % CPB) * 16, 0u, 0u, 0u, 0u);
                        }
                    }
                    if (valid < BN) {
                        fence_proxy_async_smem();  // the zeros, before the tensor core reads them
                        __syncwarp();
                    }
                }
                if (!wait(&p_full[buf], (SINGLE ? (gs >> 1) : gs) & 1, 766 + t)) return;
                tc_fence_after_sync();
                constexpr uint32_t idesc = idesc_f16(BM, D, BF16, true), dhi = smem_desc_hi(8 * SW, C::LAYOUT);
                const uint32_t a = tmem + (DEC ? C::P_COL + 64 * t : buf * BN), o = tmem + C::O_COL + t * D;
                constexpr int UV = BN / 16 / U;
#pragma unroll
                for (int un = 0; un < U; ++un) {
                    const int stage = (part0 + un) % NS;
                    const uint32_t v_lo = smem_desc_lo(smem_u32(sKV + stage * C::UNIT_BYTES), C::VROWS_PER_UNIT * SW);
#pragma unroll
                    for (int kk = 0; kk < UV; ++kk) {
                        const int k = un * UV + kk;
                        umma_ts_elect(o, a + k * 8, v_lo + ((kk * 16 * SW) >> 4), dhi, idesc, (ts > 0 || k > 0) ? 1u : 0u);
                    }
                    if (un + 1 == U) umma_commit_elect(&pv_done[t]);
                    if (last) umma_commit_elect(&kv_empty[stage]);
                }
            };
            const bool do_qk = !DEC || warp == W_MMA, do_pv = !DEC || warp == W_PV;
            for (bool more = w.begin(p, start); more && ok; more = w.next(p)) {
                const int n = w.j1 - w.j0;
                const bool two = !SINGLE && w.tokens > TT;
                const int end = w.keys - w.j0 * BN;  // keys of the segment (its last tile may reach past them)
                auto valid = [&](int jj) { return max(0, end - jj * BN); };
                if (SINGLE) {
                    for (int i = 0; ok && i < 2 * n; ++i) {
                        bool is_v;
                        int j;
                        decode_step(i, n, is_v, j);
                        if (is_v) pv(0, j, j, true, true, valid(j));
                        else qk(0, 0, j, j, true, true, j == n - 1);
                    }
                    ga += n;
                } else {
                    // Steps of A and B in turn, the QKs two ahead of the PVs. Two row tiles: A and B of key tile o / 2;
                    // one: key tile o, the even ones through A, the odd ones through B. (One loop for both: each
                    // copy of an issue is a hundred instructions, and more of them than the instruction cache
                    // holds beside the softmax made short items 12 % slower.)
                    const int N = two ? 2 * n : n;
#pragma unroll 1
                    for (int o = -2; ok && o < N; ++o) {
                        if (do_pv && o >= 0) {
                            const int t = o & 1, j = two ? o >> 1 : o;
                            pv(t, j, o >> 1, !two || t == 0, !two || t == 1, valid(j));
                        }
                        if (do_qk && ok && o + 2 < N) {
                            const int t = o & 1, j = two ? (o + 2) >> 1 : o + 2;
                            qk(t, two ? t : 0, j, (o + 2) >> 1, !two || t == 0, !two || t == 1, j == n - 1);
                        }
                    }
                    ga += (N + 1) >> 1;
                    gb += N >> 1;
                    if (two) nq[1]++;
                }
                u0 += 2 * U * n;
                nq[0]++;
            }
            umma_commit_elect(drain);
            const uint64_t t0 = global_timer_ns();
            while (!mbar_try_wait(drain, 0) && global_timer_ns() - t0 < lim) {
            }
        } else if (warp == W_Q) {
            // ------------------------------------------------------------ Q tiles
            // One box per column block: the G heads of TT tokens, rows token-major. Rows past them are
            // never written: they hold whatever was there, and nobody reads their results.
            if (lane == 0) {
                bool ok = true;
                int nq[2] = {0, 0};
                const uint64_t pol = l2_policy_evict_first();
                for (bool more = w.begin(p, start); more && ok; more = w.next(p)) {
                    const bool two = !SINGLE && w.tokens > TT;
                    for (int t = 0; t < (two ? 2 : 1); ++t) {
                        if (nq[t] > 0 && !wait_bounded(&q_free[t], (nq[t] - 1) & 1, abort_flag, lim, 770 + t)) {
                            ok = false;
                            break;
                        }
                        mbar_arrive_expect_tx(&q_full[t], TT * p.G * D * 2);
#pragma unroll
                        for (int blk = 0; blk < C::NBLK; ++blk)
                            tma_load_4d(sQ + t * C::Q_BYTES + blk * BM * SW, &tm_q, &q_full[t], blk * C::SWE, 0, w.h,
                                        w.s.q0 + w.i0 + t * TT, pol);
                        nq[t]++;
                    }
                }
                if (*abort_flag) {  // the copies in flight land before the shared memory goes away
                    for (int t = 0; t < 2; ++t) {
                        const uint64_t t0 = global_timer_ns();
                        while (nq[t] > 0 && !mbar_try_wait(&q_full[t], (nq[t] - 1) & 1) && global_timer_ns() - t0 < lim) {
                        }
                    }
                }
            }
        }
    } else {
        // ------------------------------------------------------------ softmax + epilogue
        if constexpr (C::SPLIT_REGS) regs_inc<C::regs_high(false)>();
        const int t = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t o_addr = tmem + lane_base + C::O_COL + t * D;
        const float sc = p.scale_log2;
        bool ok = true;
        int gbase = 0, splits = 0;  // steps of this tile; items with split keys
        bool owe = false;           // B: the last such item's results may not have been read yet
        // The walk waits in shared memory while an item's steps run: these warps are at their register limit
        // there (kept in registers it spills into the loop: 192 -> 223 us at D = 64, 2048 tokens over 8192).
        static_assert(sizeof(Walk) <= 64, "a walk's place");
        Walk *const parked = reinterpret_cast<Walk *>(smem + C::OFF_WALK + warp * 64);
        if (threadIdx.x == 0) p.desc[blockIdx.x] = ChunkDesc{0, 0, 0, 0};
        Walk w;
#pragma unroll 1
        for (bool more = w.begin(p, start); more; more = w.next(p)) {
            if (threadIdx.x == 0 && w.j0 == 0 && w.j1 < w.steps) p.desc[blockIdx.x] = w.desc(p);
            // With one row tile in the item A and B share it, A taking the segment's even key tiles and B the odd
            // ones, each with its own (m, l) and O (one tile alone would wait for itself at every step: 1.4 us
            // a step against 1.7 for two); A joins them at the end.
            bool busy;        // this warp has a row
            int n, hi, stride;  // this warpgroup's steps; keys this row sees, counted from its first key tile
            {
                const bool split = !SINGLE && w.tokens <= TT;
                n = split ? (w.j1 - w.j0 + 1 - t) >> 1 : w.j1 - w.j0;
                if (n == 0) continue;
                const int first = split ? 0 : t * TT;              // the tile's first token
                const int rows = min(w.tokens - first, TT) * p.G;  // of this MMA tile
                busy = quarter * 32 < rows;
                stride = split ? 2 * BN : BN;
                hi = (r < rows ? token_keys<CAUSAL>(w.s, w.i0 + first + r / p.G) : w.keys) - (w.j0 + (split ? t : 0)) * BN;
                __syncwarp();
                if (lane == 0) *parked = w;
                __syncwarp();
            }
            if (owe) {  // O_B is written again from this item's first PV on
                owe = false;
                if (ok) ok = __all_sync(0xffffffffu, wait_bounded(x_free, (splits - 1) & 1, abort_flag, lim, 790));
            }
            float m = -INFINITY, l = 0.f;
#pragma unroll 1
            for (int jj = 0; ok && jj < n; ++jj, hi -= stride) {
                const int gs = gbase + jj, buf = SINGLE ? (gs & 1) : t;
                const uint32_t ph = (SINGLE ? (gs >> 1) : gs) & 1;
                if (!__all_sync(0xffffffffu, wait_bounded(&s_full[buf], ph, abort_flag, lim, 780 + t))) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                if (!busy) {
                    if (DEC && lane == 0) mbar_arrive(&s_free[t]);
                    if ((SINGLE || DEC) && jj > 0 &&
                        !__all_sync(0xffffffffu, wait_bounded(&pv_done[t], (gs - 1) & 1, abort_flag, lim, 782))) {
                        ok = false;
                        break;
                    }
                    mbar_arrive(&p_full[buf]);
                    continue;
                }
                uint32_t sr[BN];
#pragma unroll
                for (int cc = 0; cc < BN / 32; ++cc) tmem_ld32(tmem + lane_base + buf * BN + cc * 32, sr + cc * 32);
                tmem_ld_wait();
                tmem_reg_fence<BN>(sr);
                if (DEC) {
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s_free[t]);
                }
                if (__any_sync(0xffffffffu, hi < BN)) {
#pragma unroll
                    for (int i = 0; i < BN; ++i)
                        if (i >= hi) sr[i] = __float_as_uint(-INFINITY);
                }
                const float m_cand = row_max<BN>(sr) * sc;
                const bool grow = m_cand > m + 8.0f;
                float alpha = 1.f;
                if (grow) {
                    alpha = ex2_approx(m - m_cand);
                    m = m_cand;
                }
                const bool warp_grow = __any_sync(0xffffffffu, grow);
                const float neg_m = (m == -INFINITY) ? 0.f : -m;
                auto rescale = [&]() {  // O holds the earlier tiles' sum: to the new running maximum
                    const uint64_t a2 = f2(alpha, alpha);
#pragma unroll 1
                    for (int cc = 0; cc < D / 32; ++cc) {
                        uint32_t o[32];
                        tmem_ld32(o_addr + cc * 32, o);
                        tmem_ld_wait();
                        tmem_reg_fence<32>(o);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float x, y;
                            f2_split(fmul2(f2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), a2), x, y);
                            o[2 * i] = __float_as_uint(x);
                            o[2 * i + 1] = __float_as_uint(y);
                        }
                        tmem_st32(o_addr + cc * 32, o);
                    }
                };
                if constexpr (DEC) {
                    uint32_t pk[BN / 2];
                    const float rs = softmax_row_to_regs<BN, BF16>(sr, sc, neg_m, pk);
                    l = fmaf(l, alpha, rs);
                    if (jj > 0) {  // P's columns and O are free once the last PV is done
                        if (!__all_sync(0xffffffffu, wait_bounded(&pv_done[t], (gs - 1) & 1, abort_flag, lim, 784))) {
                            ok = false;
                            break;
                        }
                        tc_fence_after_sync();
                        if (warp_grow) rescale();
                    }
#pragma unroll
                    for (int cc = 0; cc < BN / 64; ++cc) tmem_st32(tmem + lane_base + C::P_COL + 64 * t + cc * 32, pk + cc * 32);
                    tmem_st_wait();
                } else {
                    const float rs = softmax_chunk_store<BN, BF16>(sr, sc, neg_m, tmem + lane_base + buf * BN);
                    l = fmaf(l, alpha, rs);
                    tmem_st_wait();
                    if (jj > 0) {
                        // two tiles: PV_t(j - 1) was issued before QK_t(j), so s_full has shown it done
                        if (SINGLE &&
                            !__all_sync(0xffffffffu, wait_bounded(&pv_done[t], (gs - 1) & 1, abort_flag, lim, 786))) {
                            ok = false;
                            break;
                        }
                        if (warp_grow) {
                            tc_fence_after_sync();
                            rescale();
                            tmem_st_wait();
                        }
                    }
                }
                tc_fence_before_sync();
                mbar_arrive(&p_full[buf]);
            }
            if (ok) ok = __all_sync(0xffffffffu, wait_bounded(&pv_done[t], (gbase + n - 1) & 1, abort_flag, lim, 788 + t));
            gbase += n;
            w = *parked;
            const bool split = !SINGLE && w.tokens <= TT, joins = split && w.j1 - w.j0 > 1;
            const int first = split ? 0 : t * TT;
            const bool row_ok = r < min(w.tokens - first, TT) * p.G;
            float scale_a = 1.f, scale_b = 0.f;
            if (joins) {
                ++splits;
                if (t == 1) {  // B: (m, l) to A, which reads O_B out of TMEM
                    if (!ok) continue;
                    sML[r] = make_float2(m, l);
                    tc_fence_before_sync();
                    mbar_arrive(x_full);
                    owe = true;
                    continue;
                }
                if (ok) ok = __all_sync(0xffffffffu, wait_bounded(x_full, (splits - 1) & 1, abort_flag, lim, 792));
                if (ok) {
                    const float2 b = sML[r];
                    const float to = fmaxf(m, b.x);
                    scale_a = m == -INFINITY ? 0.f : ex2_approx(m - to);
                    scale_b = b.x == -INFINITY ? 0.f : ex2_approx(b.x - to);
                    m = to;
                    l = l * scale_a + b.y * scale_b;
                }
            }
            if (!ok) continue;
            tc_fence_after_sync();
            if (!busy) {
                if (joins) mbar_arrive(x_free);
                continue;
            }
            const bool whole = w.whole();
            const int ti = r / p.G;
            const int64_t tok = w.s.q0 + w.i0 + first + ti;
            const int head = w.h * p.G + r - ti * p.G;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            uint16_t *out = static_cast<uint16_t *>(p.out) + (tok * p.Hq + head) * D;
            const int64_t slot = w.slot();
            const int pr = split ? r : t * BM + r;              // row of the item's tile
            float *po = p.part_o + slot * D * C::R + pr;        // column by column
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
                uint32_t o[32];
                tmem_ld32(o_addr + c0, o);
                tmem_ld_wait();
                tmem_reg_fence<32>(o);
                if (joins) {
                    uint32_t x[32];
                    tmem_ld32(o_addr + D + c0, x);  // O_B
                    tmem_ld_wait();
                    tmem_reg_fence<32>(x);
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        o[k] = __float_as_uint(fmaf(__uint_as_float(o[k]), scale_a, __uint_as_float(x[k]) * scale_b));
                }
                if (!whole) {
#pragma unroll
                    for (int v = 0; v < 32; ++v) po[(c0 + v) * C::R] = __uint_as_float(o[v]);
                } else if (row_ok) {
                    uint32_t x[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        x[k] = pack2<BF16>(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv);
                    if (p.out_align32) {
                        st_global_v8(out + c0, x);
                        st_global_v8(out + c0 + 16, x + 8);
                    } else {
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            *reinterpret_cast<uint4 *>(out + c0 + v * 8) = make_uint4(x[4 * v], x[4 * v + 1], x[4 * v + 2], x[4 * v + 3]);
                    }
                }
                __syncwarp();
            }
            if (joins) {
                tc_fence_before_sync();
                mbar_arrive(x_free);
            }
            if (!whole)
                p.part_ml[slot * C::R + pr] = make_float2(m, l);
            else if (row_ok && p.lse)
                p.lse[static_cast<int64_t>(head) * p.total + tok] = l == 0.f ? -INFINITY : m * 0.6931471805599453f + logf(l);
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == W_MMA) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

template <int D, bool BF16, bool CAUSAL>
cudaError_t launch(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const ChunkParams &p, int ctas,
                   cudaStream_t st) {
    using C = TileCfg<D>;
    auto kern = chunk_tile_kernel<D, BF16, CAUSAL>;
    static uint64_t attr_set_mask = 0;  // per device; setting it twice is harmless
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (!(__atomic_load_n(&attr_set_mask, __ATOMIC_ACQUIRE) & bit)) {
        if (C::SPLIT_REGS) {
            // the register split draws on the registers the CTA launches with
            cudaFuncAttributes fa_attr;
            e = cudaFuncGetAttributes(&fa_attr, kern);
            if (e != cudaSuccess) return e;
            if (fa_attr.numRegs * C::NUM_THREADS < 128 * C::regs_low(false) + 256 * C::regs_high(false))
                return cudaErrorInvalidConfiguration;
        }
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        __atomic_fetch_or(&attr_set_mask, bit, __ATOMIC_RELEASE);
    }
    kern<<<ctas, C::NUM_THREADS, C::SMEM, st>>>(tq, tk, tv, p);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_combine<D, BF16, C::R>(p, ctas, st);
}

template <int D>
cudaError_t launch_d(bool bf16, bool causal, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                     const ChunkParams &p, int ctas, cudaStream_t st) {
    if (bf16) return causal ? launch<D, true, true>(tq, tk, tv, p, ctas, st) : launch<D, true, false>(tq, tk, tv, p, ctas, st);
    return causal ? launch<D, false, true>(tq, tk, tv, p, ctas, st) : launch<D, false, false>(tq, tk, tv, p, ctas, st);
}

}  // namespace

cudaError_t launch_chunk_tile(int D, bool bf16, bool causal, const CUtensorMap &tq, const CUtensorMap &tk,
                              const CUtensorMap &tv, const ChunkParams &p, int ctas, cudaStream_t st) {
    switch (D) {
        case 32: return launch_d<32>(bf16, causal, tq, tk, tv, p, ctas, st);
        case 64: return launch_d<64>(bf16, causal, tq, tk, tv, p, ctas, st);
        case 128: return launch_d<128>(bf16, causal, tq, tk, tv, p, ctas, st);
        case 256: return launch_d<256>(bf16, causal, tq, tk, tv, p, ctas, st);
        default: return cudaErrorInvalidValue;
    }
}

int chunk_tile_rows(int D) { return D == 256 ? 128 : 256; }
int chunk_tile_k_box(int, int page_size) { return page_size < 128 ? page_size : 128; }
int chunk_tile_v_box(int D, int page_size) {
    const int rows = D == 256 ? 64 : 128;
    return page_size < rows ? page_size : rows;
}

cudaError_t chunk_tile_error_addrs(int **code, int **where) { return device_error_addrs(code, where); }

}  // namespace fa
