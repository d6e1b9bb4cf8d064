// fa_key_weights_tile.cu -- the attention weight that each cached key received, for calls with many
// rows a key head (fa_paged_key_weights; prompt chunks), on the tensor core.
//
// S^T = K Q^T with the keys as the MMA's 128 rows and the rows of a tile (128 / G new tokens, G heads
// each) as its columns: a TMEM lane is a key, so the sum over rows is an addition in the registers of
// the key's thread, over all the row tiles that see it. What bounds it is the exponentials: one per
// (row, key) at 16 per clock and SM, 1024 clocks per 128 x 128 tile against 64 D / 16 for the MMAs.
// An item is KT = 2 neighbouring key tiles A and B (one at D = 256) of one (sequence, key head), whose K
// stays in shared memory while the row tiles pass:
//   warps 0-7, 8-15  tile A, B: S^T from TMEM, weights 2^(s c - lse), the key's sum; four warps a
//                    half of the columns, 32 in registers at a time (with four a tile, all columns at
//                    once, two warps a scheduler did not cover one another's waits: 2 x 777 tokens over
//                    13332 keys, 16 heads on 4, D = 64: 108 us, now 85)
//   and then one     K by TMA (page pieces), two buffers (one at D = 256)
//   each for         the MMAs, two S^T buffers per tile
//                    Q tiles by TMA through a ring
//                    the row tiles' -lse (log2 units) into the ring's stages
// The steps (row tiles of items) are cut into runs of equal cost, one per CTA, as in fa_chunk.cuh; an
// item that a cut falls into leaves partial sums in the workspace, which key_weights_join_kernel adds up
// in the order of the rows: no atomics, the same call gives the same bits.
// Measured: 2 x 777 tokens over 3333 keys (16 heads on 4, D = 64) 33 us: the run is found after 2.5, the first
// scores are there after 5, the CTAs end at 26 on average and at 30, joining takes 3. 2048 tokens over 8192 keys
// (32 heads on 8, D = 128) 183 us, 2.6 exponentials per ns of 4.5; CTAs end at 163 on average, the last at 182.
#include "fa_chunk.cuh"
#include "fa_fwd_kernel.cuh"

namespace fa {

namespace {

template <int D>
struct KtCfg {
    static constexpr int KT = D == 256 ? 1 : 2, KB = D == 256 ? 1 : 2;  // key tiles of an item, K buffers
    static constexpr int BN = 128, KEYS = KT * BN;
    static constexpr int SW = (2 * D >= 128) ? 128 : 2 * D, SWE = SW / 2, NBLK = D / SWE;
    static constexpr uint32_t LAYOUT = (SW == 128) ? kLayoutSw128 : kLayoutSw64;
    static constexpr int TILE = BN * D * 2;         // bytes of a K or Q tile
    static constexpr int K_BYTES = KT * TILE;
    static constexpr int NQ = D >= 128 ? 2 : 4;
    static constexpr int OFF_Q = KB * K_BYTES;
    static constexpr int OFF_L = OFF_Q + NQ * TILE;  // NQ x 128 floats
    static constexpr int OFF_SUM = OFF_L + NQ * BN * 4;  // 2 x KEYS floats: the second column half's sums
    // Items by turns: how many keys the item's rows of NaN lse see. The -lse are at most NQ steps, so as many items, ahead.
    static constexpr int LIMITS = 8, OFF_NAN = OFF_SUM + 2 * KEYS * 4;
    static constexpr int OFF_BAR = OFF_NAN + LIMITS * 4;
    static_assert(NQ < LIMITS, "limits of items that are still worked on");
    static constexpr int BARS = 2 * KB + 3 * NQ + 4 * KT + 1;
    static constexpr int OFF_START = OFF_BAR + BARS * 8;
    static constexpr int OFF_TMEM = OFF_START + static_cast<int>(sizeof(ChunkStart));
    static constexpr int USED = OFF_TMEM + 8 + 1024;
    static constexpr int SMEM = USED > 120 * 1024 ? USED : 120 * 1024;  // one CTA (and its TMEM) per SM
    static constexpr int COLS = BN / 2;             // columns of a tile that a warp takes
    static constexpr int NUM_S_WARPS = 8 * KT;
    static constexpr int THREADS = 32 * (NUM_S_WARPS + 4);
    static constexpr uint32_t TMEM_COLS = KT * 256;
    static_assert(USED <= 227 * 1024, "shared memory");
};

// A walk over (sequence, key head, KEYS keys), each with the row tiles [t0, t1) of this run.
template <int KT, bool CAUSAL>
struct KeyTileWalk {
    static constexpr int KEYS = KT * 128;
    ChunkSeq s;
    int b, h, j, first, steps, t0, t1, shift;  // first: row tile that first sees the item's keys
    int64_t pos, lo, hi;
    __device__ static __forceinline__ int first_tile(const ChunkSeq &s, int T, int j) {
        return CAUSAL ? max(0, j * KEYS - (s.kv - s.n)) / T : 0;  // token i sees key k when i >= k - (kv - n)
    }
    __device__ static __forceinline__ int step_log(const ChunkSeq &s, int j) {
        return (KT == 2 && s.kv - j * KEYS > 128) ? 1 : 0;
    }
    __device__ static __forceinline__ int64_t item_cost(const ChunkSeq &s, int T, int tiles, int j) {
        return static_cast<int64_t>(tiles - first_tile(s, T, j)) << step_log(s, j);
    }
    __device__ static int64_t head_cost(const ChunkSeq &s, int T) {
        if (s.n == 0) return 0;
        const int tiles = (s.n + T - 1) / T;
        int j = alike(s);
        int64_t sum = static_cast<int64_t>(j) * (tiles * KT);
        for (; j * KEYS < s.kv; ++j) sum += item_cost(s, T, tiles, j);
        return sum;
    }
    // The first so many items cost the same: every row tile sees them, and they have KT key tiles.
    __device__ static __forceinline__ int alike(const ChunkSeq &s) {
        const int full = (s.kv - 1) / KEYS;  // (all but the last)
        return !CAUSAL ? full : (s.kv >= s.n ? min(full, (s.kv - s.n) / KEYS + 1) : 0);
    }
    // As chunk_locate: a few sequences one by one, a lane per item; many with four per lane. (A lane a sequence took
    // 6 us for two of 52 items.)
    __device__ static void locate(const ChunkParams &p, int cta, int ctas, ChunkStart *out) {
        constexpr int PER = 4, FEW = 8;
        const int lane = threadIdx.x & 31, T = p.tile_tokens;
        const bool few = p.num_seqs <= FEW;
        int64_t cost[PER], total = 0, mine = 0;
        const ChunkSeq own = chunk_seq(p, min(lane, p.num_seqs - 1));  // few: sequence `lane`
        auto seq_of = [&](int b) {
            return ChunkSeq{__shfl_sync(0xffffffffu, own.q0, b), __shfl_sync(0xffffffffu, own.n, b),
                            __shfl_sync(0xffffffffu, own.kv, b)};
        };
        auto costs = [&](int base) {
            mine = 0;
            ChunkSeq q[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i) q[i] = chunk_seq(p, min(base + lane * PER + i, p.num_seqs - 1));
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                if (base + lane * PER + i >= p.num_seqs) q[i].n = 0;
                cost[i] = head_cost(q[i], T) * p.Hkv;
                mine += cost[i];
            }
        };
        if (few) {  // mine: cost of a key head of sequence `lane`
            for (int b = 0; b < p.num_seqs; ++b) {
                const ChunkSeq s = seq_of(b);
                const int tiles = (s.n + T - 1) / T;
                int64_t sum = 0;
                if (s.n > 0)
                    for (int j = lane; j * KEYS < s.kv; j += 32) sum += item_cost(s, T, tiles, j);
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
        if (per < KT) per = KT;  // at least a step
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
                const int tiles = (s.n + T - 1) / T;
                const int64_t h = div_up_or_down(start - before, one, false);
                int64_t pos = before + h * one;
                for (int j0 = 0; j0 * KEYS < s.kv; j0 += 32) {
                    const int j = j0 + lane;
                    const int64_t c = j * KEYS < s.kv ? item_cost(s, T, tiles, j) : 0;
                    const int64_t incl = warp_scan64(c, lane), at = pos + incl - c;
                    if (start >= at && start < at + c) *out = ChunkStart{b, static_cast<int>(h), j, at, start, end, per};
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
            int64_t at = before + incl - mine;
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
                const int tiles = (s.n + T - 1) / T;
                const int64_t one = div_up_or_down(mine_b, p.Hkv, false);
                const int64_t h = div_up_or_down(start - at, one, false);
                int64_t pos = at + h * one;
                int j = static_cast<int>(min(static_cast<int64_t>(alike(s)), div_up_or_down(start - pos, tiles * KT, false)));
                pos += static_cast<int64_t>(j) * (tiles * KT);
                for (;; ++j) {
                    const int64_t n = item_cost(s, T, tiles, j);
                    if (start < pos + n) break;
                    pos += n;
                }
                *out = ChunkStart{b, static_cast<int>(h), j, pos, start, end, per};
            }
            before += __shfl_sync(0xffffffffu, incl, 31);
        }
    }
    __device__ __forceinline__ bool begin(const ChunkParams &p, const ChunkStart &st) {
        lo = st.lo;
        hi = st.hi;
        if (lo >= hi) return false;
        b = st.b;
        h = st.h;
        j = st.t;
        pos = st.pos;
        s = chunk_seq(p, b);
        set(p);
        return t0 < first + steps || next(p);
    }
    __device__ __forceinline__ void set(const ChunkParams &p) {
        const int tiles = (s.n + p.tile_tokens - 1) / p.tile_tokens;
        first = first_tile(s, p.tile_tokens, j);
        steps = tiles - first;
        shift = step_log(s, j);
        const int64_t round = (1 << shift) - 1;
        t0 = first + static_cast<int>(max(int64_t(0), lo - pos + round) >> shift);
        t1 = first + static_cast<int>(min(static_cast<int64_t>(steps), (hi - pos + round) >> shift));
    }
    __device__ __forceinline__ bool next(const ChunkParams &p) {
        pos += static_cast<int64_t>(steps) << shift;
        if (pos >= hi) return false;
        if (++j * KEYS >= s.kv) {
            j = 0;
            if (++h == p.Hkv) {
                h = 0;
                do {
                    if (++b >= p.num_seqs) return false;
                    s = chunk_seq(p, b);
                } while (s.n == 0 || s.kv == 0);
            }
        }
        set(p);
        return true;
    }
    __device__ __forceinline__ bool whole() const { return t0 == first && t1 == first + steps; }
    __device__ __forceinline__ int slot() const { return 2 * blockIdx.x + (t0 == first ? 1 : 0); }
    __device__ __forceinline__ ChunkDesc desc(int64_t per) const {
        const int64_t last = pos + (static_cast<int64_t>(steps - 1) << shift);
        return ChunkDesc{static_cast<int>(div_up_or_down(last, per, false)) - static_cast<int>(blockIdx.x) + 1, b, h, j};
    }
};

template <int D, bool BF16, bool CAUSAL>
__global__ void __launch_bounds__(KtCfg<D>::THREADS, 1)
key_weights_tile_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k, const ChunkParams p) {
    using C = KtCfg<D>;
    using Walk = KeyTileWalk<C::KT, CAUSAL>;
    constexpr int BN = C::BN, SW = C::SW, NQ = C::NQ, KT = C::KT, KB = C::KB, COLS = C::COLS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *sL = reinterpret_cast<float *>(smem + C::OFF_L);
    int *sNan = reinterpret_cast<int *>(smem + C::OFF_NAN);
    uint64_t *k_full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR), *k_empty = k_full + KB;
    uint64_t *q_full = k_empty + KB, *q_empty = q_full + NQ, *l_full = q_empty + NQ;
    uint64_t *s_full = l_full + NQ, *s_free = s_full + 2 * KT, *drain = s_free + 2 * KT;  // [tile][buffer]
    ChunkStart *start = reinterpret_cast<ChunkStart *>(smem + C::OFF_START);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_TMEM);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_TMEM + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint64_t lim = p.timeout_ns;
    constexpr int W_K = C::NUM_S_WARPS, W_MMA = W_K + 1, W_Q = W_K + 2, W_L = W_K + 3;
    const int T = p.tile_tokens;

    pdl_launch_dependents();
    if (threadIdx.x == 32 * W_K) {
        for (int i = 0; i < KB; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < NQ; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1 + C::NUM_S_WARPS);  // the MMAs' commit, the warps that read -lse
            mbar_init(&l_full[i], 1);
        }
        for (int i = 0; i < 2 * KT; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_free[i], 8);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
    }
    if (warp == W_MMA) {
        tmem_alloc(tmem_slot, C::TMEM_COLS);
        tmem_relinquish();
    }
    if (warp == 0) Walk::locate(p, blockIdx.x, gridDim.x, start);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    Walk w;

    if (warp == W_K) {
        // ------------------------------------------------------------ K: the item's key tiles
        bool bad = false, ok = true;
        int it = 0;
        const int box = min(1 << p.page_shift, BN);
        const uint64_t pol = l2_policy_evict_first();
        for (bool more = w.begin(p, *start); more && ok; more = w.next(p), ++it) {
            const int buf = it % KB;
            if (it >= KB && !__all_sync(0xffffffffu, wait_bounded(&k_empty[buf], ((it / KB) - 1) & 1, abort_flag, lim, 790))) {
                ok = false;
                break;
            }
            const int valid = min(C::KEYS, w.s.kv - w.j * C::KEYS), boxes = (valid + box - 1) / box;
            if (lane == 0) mbar_arrive_expect_tx(&k_full[buf], boxes * box * D * 2);
            __syncwarp();
            for (int i = lane; i < boxes * C::NBLK; i += 32) {
                const int bx = i / C::NBLK, blk = i % C::NBLK, r = bx * box;
                const int row = chunk_page_row(p, w.b, w.j * C::KEYS + r, bad);
                tma_load_3d(smem + buf * C::K_BYTES + (r / BN) * C::TILE + (blk * BN + r % BN) * SW, &tm_k, &k_full[buf],
                            blk * C::SWE, w.h, row, pol);
            }
        }
        if (__any_sync(0xffffffffu, bad) && lane == 0) record_error(FA_ERR_INDEX, 791);
        if (*abort_flag) {  // the copies in flight land before the shared memory goes away
            for (int v = max(0, it - KB); v < it; ++v) {
                const uint64_t t0 = global_timer_ns();
                while (!mbar_try_wait(&k_full[v % KB], (v / KB) & 1) && global_timer_ns() - t0 < lim) {
                }
            }
        }
    } else if (warp == W_Q) {
        // ------------------------------------------------------------ Q tiles
        if (lane == 0) {
            bool ok = true;
            int u = 0;
            const uint64_t pol = l2_policy_evict_last();
            for (bool more = w.begin(p, *start); more && ok; more = w.next(p)) {
                for (int t = w.t0; t < w.t1; ++t, ++u) {
                    const int st = u % NQ;
                    if (u >= NQ && !wait_bounded(&q_empty[st], ((u / NQ) - 1) & 1, abort_flag, lim, 792)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&q_full[st], T * p.G * D * 2);
#pragma unroll
                    for (int blk = 0; blk < C::NBLK; ++blk)
                        tma_load_4d(smem + C::OFF_Q + st * C::TILE + blk * BN * SW, &tm_q, &q_full[st], blk * C::SWE, 0, w.h,
                                    w.s.q0 + t * T, pol);
                }
            }
            if (*abort_flag) {
                for (int v = max(0, u - NQ); v < u; ++v) {
                    const uint64_t t0 = global_timer_ns();
                    while (!mbar_try_wait(&q_full[v % NQ], (v / NQ) & 1) && global_timer_ns() - t0 < lim) {
                    }
                }
            }
        }
    } else if (warp == W_L) {
        // ------------------------------------------------------------ -lse of the rows, log2 units
        bool ok = true;
        int u = 0, it = 0;
        for (bool more = w.begin(p, *start); more && ok; more = w.next(p), ++it) {
            int nan = 0;  // a row whose lse is NaN: keys [0, nan) are seen by one
            for (int t = w.t0; t < w.t1; ++t, ++u) {
                const int st = u % NQ;
                float x[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int c = lane + 32 * k, ti = c / p.G, i = t * T + ti;
                    x[k] = -INFINITY;  // no row: no weight
                    if (ti < T && i < w.s.n) {
                        const float v = __ldg(p.lse_in + static_cast<int64_t>(w.h * p.G + c - ti * p.G) * p.total + w.s.q0 + i);
                        // A row that saw nothing gives no weight either. Nor does one whose lse is NaN in the sums: with NaN in
                        // them its masked keys would be NaN too (-inf + NaN); those that it sees become so at the end.
                        if (v > -INFINITY) x[k] = v * -1.4426950408889634f;
                        if (v != v) nan = max(nan, token_keys<CAUSAL>(w.s, i));
                    }
                }
                if (u >= NQ && !__all_sync(0xffffffffu, wait_bounded(&q_empty[st], ((u / NQ) - 1) & 1, abort_flag, lim, 793))) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) sL[st * BN + lane + 32 * k] = x[k];
                nan = __reduce_max_sync(0xffffffffu, nan);
                if (lane == 0) sNan[it % C::LIMITS] = nan;
                __syncwarp();
                if (lane == 0) mbar_arrive(&l_full[st]);
            }
        }
    } else if (warp == W_MMA) {
        // ------------------------------------------------------------ S^T = K Q^T
        bool ok = true;
        int u = 0, it = 0;
        int uses[2] = {0, 0};  // steps of tiles A, B
        auto wait = [&](uint64_t *bar, uint32_t ph, int where) {
            if (ok) ok = __all_sync(0xffffffffu, wait_bounded(bar, ph, abort_flag, lim, where));
            return ok;
        };
        constexpr uint32_t idesc = idesc_f16(128, BN, BF16, false), dhi = smem_desc_hi(8 * SW, C::LAYOUT);
        for (bool more = w.begin(p, *start); more && ok; more = w.next(p), ++it) {
            const int kbuf = it % KB;
            const bool two = w.shift == 1;
            if (!wait(&k_full[kbuf], (it / KB) & 1, 794)) break;
            for (int t = w.t0; ok && t < w.t1; ++t, ++u) {
                const int st = u % NQ;
                if (!wait(&q_full[st], (u / NQ) & 1, 795)) break;
                const uint32_t q_lo = smem_desc_lo(smem_u32(smem + C::OFF_Q + st * C::TILE), 16);
#pragma unroll
                for (int a = 0; a < KT; ++a) {
                    if (a == 1 && !two) continue;
                    const int n = uses[a]++, buf = n & 1;
                    if (n >= 2 && !wait(&s_free[a * 2 + buf], ((n >> 1) - 1) & 1, 796)) break;
                    tc_fence_after_sync();
                    const uint32_t k_lo = smem_desc_lo(smem_u32(smem + kbuf * C::K_BYTES + a * C::TILE), 16);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t off = ((k * 32) / SW) * BN * SW + (k * 32) % SW;
                        umma_ss_elect(tmem + (a * 2 + buf) * BN, k_lo + (off >> 4), q_lo + (off >> 4), dhi, idesc, k > 0 ? 1u : 0u);
                    }
                    umma_commit_elect(&s_full[a * 2 + buf]);
                }
                if (ok) umma_commit_elect(&q_empty[st]);
            }
            if (ok) umma_commit_elect(&k_empty[kbuf]);
        }
        umma_commit_elect(drain);
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait(drain, 0) && global_timer_ns() - t0 < lim) {
        }
    } else {
        // ------------------------------------------------------------ weights and their sums
        const int a = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3, in = a * BN + quarter * 32 + lane;
        const uint32_t at_tmem = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + a * 2 * BN + half * COLS;
        float *sums = reinterpret_cast<float *>(smem + C::OFF_SUM);
        const uint64_t c2 = f2(p.scale_log2, p.scale_log2);
        bool ok = true;
        int u = 0, uses = 0, it = 0;
        ChunkDesc desc{0, 0, 0, 0};
#pragma unroll 1
        for (bool more = w.begin(p, *start); more; more = w.next(p), ++it) {
            if (w.t0 == w.first && w.t1 < w.first + w.steps) desc = w.desc(start->per);
            const bool mine = a == 0 || w.shift == 1;
            const int key = w.j * C::KEYS + in;
            const bool busy = mine && key - lane < w.s.kv;  // this warp has a key
            float *at = p.weights + (static_cast<int64_t>(w.b) * p.Hkv + w.h) * p.width + key;
            const bool whole = w.whole();
            const float was = half == 0 && whole && busy && key < w.s.kv ? *at : 0.f;
            // tokens from `sees` on see this key
            const int sees = CAUSAL ? max(0, key - (w.s.kv - w.s.n)) : 0;
            uint64_t acc[4] = {f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll 1
            for (int t = w.t0; ok && t < w.t1; ++t, ++u) {
                const int st = u % NQ;
                const int buf = uses & 1;
                if (mine) {
                    if (!__all_sync(0xffffffffu, wait_bounded(&s_full[a * 2 + buf], (uses >> 1) & 1, abort_flag, lim, 797))) {
                        ok = false;
                        break;
                    }
                    ++uses;
                    tc_fence_after_sync();
                }
                // (every warp: an idle one that did not wait would release the stage rounds ahead)
                if (!__all_sync(0xffffffffu, wait_bounded(&l_full[st], (u / NQ) & 1, abort_flag, lim, 798))) {
                    ok = false;
                    break;
                }
                if (busy) {
                    // columns [lo, hi) are rows that see the key
                    const int lo = (sees - t * T) * p.G - half * COLS, hi = min(T, w.s.n - t * T) * p.G - half * COLS;
                    const bool masked = __any_sync(0xffffffffu, lo > 0) || hi < COLS;
#pragma unroll
                    for (int c = 0; c < COLS; c += 32) {  // 32 columns in registers at a time
                        uint32_t sr[32];
                        tmem_ld32(at_tmem + buf * BN + c, sr);
                        tmem_ld_wait();
                        tmem_reg_fence<32>(sr);
                        if (masked) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (c + i < lo || c + i >= hi) sr[i] = __float_as_uint(-INFINITY);
                        }
                        const float4 *nl = reinterpret_cast<const float4 *>(sL + st * BN + half * COLS + c);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 l = nl[i];
                            float x0, x1, x2, x3;
                            f2_split(ffma2(f2(__uint_as_float(sr[4 * i]), __uint_as_float(sr[4 * i + 1])), c2, f2(l.x, l.y)), x0, x1);
                            f2_split(ffma2(f2(__uint_as_float(sr[4 * i + 2]), __uint_as_float(sr[4 * i + 3])), c2, f2(l.z, l.w)), x2, x3);
                            acc[(2 * i) & 3] = fadd2(acc[(2 * i) & 3], f2(ex2_approx(x0), ex2_approx(x1)));
                            acc[(2 * i + 1) & 3] = fadd2(acc[(2 * i + 1) & 3], f2(ex2_approx(x2), ex2_approx(x3)));
                        }
                    }
                    tc_fence_before_sync();
                }
                __syncwarp();
                if (mine && lane == 0) mbar_arrive(&s_free[a * 2 + buf]);
                if (lane == 0) mbar_arrive(&q_empty[st]);
            }
            float lo, hi;
            f2_split(fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3])), lo, hi);
            // the halves' sums, the items by turns (every warp takes every item, whatever became of its waits)
            float *other = sums + (it & 1) * C::KEYS + in;
            if (half == 1) *other = lo + hi;
            asm volatile("bar.sync %0, 256;" ::"r"(1 + a) : "memory");
            if (half == 1 || !ok || !busy) continue;
            const float sum = key < sNan[it % C::LIMITS] ? NAN : (lo + hi) + *other;
            if (!whole)
                p.part_o[static_cast<int64_t>(w.slot()) * C::KEYS + in] = sum;
            else if (key < w.s.kv)
                *at = was + sum;
        }
        if (threadIdx.x == 0) p.desc[blockIdx.x] = desc;
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == W_MMA) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// Adds up the pieces of the item that CTA blockIdx.x began and did not finish, in order.
template <int KEYS>
__global__ void __launch_bounds__(KEYS) key_weights_join_kernel(const ChunkParams p) {
    pdl_wait();
    const ChunkDesc d = p.desc[blockIdx.x];  // pieces, sequence, key head, item of KEYS keys
    if (d.pieces < 2) return;
    const int b = d.token, h = d.tokens, key = d.head * KEYS + threadIdx.x;
    if (key >= chunk_seq(p, b).kv) return;
    float sum = 0.f;
    for (int k = 0; k < d.pieces; ++k)
        sum += p.part_o[static_cast<int64_t>(k == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + k)) * KEYS + threadIdx.x];
    p.weights[(static_cast<int64_t>(b) * p.Hkv + h) * p.width + key] += sum;
}

template <int D, bool BF16, bool CAUSAL>
cudaError_t launch(const CUtensorMap &tq, const CUtensorMap &tk, const ChunkParams &p, int ctas, cudaStream_t st) {
    using C = KtCfg<D>;
    auto kern = key_weights_tile_kernel<D, BF16, CAUSAL>;
    static uint64_t attr_set_mask = 0;  // per device; setting it twice is harmless
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (!(__atomic_load_n(&attr_set_mask, __ATOMIC_ACQUIRE) & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        __atomic_fetch_or(&attr_set_mask, bit, __ATOMIC_RELEASE);
    }
    kern<<<ctas, C::THREADS, C::SMEM, st>>>(tq, tk, p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, 1, 1);
    cfg.blockDim = dim3(C::KEYS, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, key_weights_join_kernel<C::KEYS>, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int D>
cudaError_t launch_d(bool bf16, bool causal, const CUtensorMap &tq, const CUtensorMap &tk, const ChunkParams &p, int ctas,
                     cudaStream_t st) {
    if (bf16) return causal ? launch<D, true, true>(tq, tk, p, ctas, st) : launch<D, true, false>(tq, tk, p, ctas, st);
    return causal ? launch<D, false, true>(tq, tk, p, ctas, st) : launch<D, false, false>(tq, tk, p, ctas, st);
}

}  // namespace

cudaError_t launch_key_weights_tile(int D, bool bf16, bool causal, const CUtensorMap &tq, const CUtensorMap &tk,
                                    const ChunkParams &p, int ctas, cudaStream_t st) {
    switch (D) {
        case 32: return launch_d<32>(bf16, causal, tq, tk, p, ctas, st);
        case 64: return launch_d<64>(bf16, causal, tq, tk, p, ctas, st);
        case 128: return launch_d<128>(bf16, causal, tq, tk, p, ctas, st);
        case 256: return launch_d<256>(bf16, causal, tq, tk, p, ctas, st);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t key_weights_tile_error_addrs(int **code, int **where) { return device_error_addrs(code, where); }

}  // namespace fa
