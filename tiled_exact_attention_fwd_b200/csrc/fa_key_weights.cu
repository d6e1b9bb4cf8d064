// fa_key_weights.cu -- the attention weight that each cached key received from a call's new tokens
// (fa_paged_key_weights): weights[b, h, j] += sum over the rows of key head h that see key j of
// exp(scale q.k_j - lse).
//
// The scores are formed again from q and K with the LSE that the attention returned, so only K is
// read (half of the cache). A work item is a tile of BN keys of one (sequence, key head); its CTA
// goes over every row tile that sees it, so a key's sum is formed in one place, in a fixed
// order, and added to the buffer by a plain load and store. Items go to the CTAs in equal runs of
// row tiles. S is computed transposed, S^T = K Q^T: a thread then holds scores of its own keys, and
// the sum over rows is an addition in its registers. Bound by reading K once: 64 single tokens over up to 8192
// keys (32 heads on 8, D = 128) 110 to 117 us for 693 MB, 5.9 to 6.3 TB/s; what is left is the start (finding the run; its costs
// are summed in closed form over the key tiles that all rows see: 3 us less than one by one).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa.h"
#include "fa_chunk.cuh"
#include "fa_internal.h"
#include "fa_mma.cuh"
#include "fa_ptx.cuh"
#include "fa_sync.cuh"

namespace fa {

namespace {

// First row tile that sees key tile j.
template <int R, int BN, bool CAUSAL>
__device__ __forceinline__ int first_tile(const ChunkParams &p, const ChunkSeq &s, int j) {
    if (!CAUSAL) return 0;
    return max(0, j * BN - (s.kv - s.n)) * p.G / R;  // token i sees key j * BN when i >= j * BN - (kv - n)
}

struct KeyStart {
    int b, h, j;
    int64_t left;
};

// A walk over key tiles: (sequence, key head, key tile), each with the row tiles [t0, tiles).
template <int R, int BN, bool CAUSAL>
struct KeyWalk {
    ChunkSeq s;
    int b, h, j, jn, t0, tiles;
    int64_t left;  // row tiles of the run that are left
    __device__ static int64_t head_cost(const ChunkParams &p, const ChunkSeq &s) {
        if (s.n == 0) return 0;
        const int tiles = (s.n * p.G + R - 1) / R, jn = (s.kv + BN - 1) / BN, same = seen_by_all(s, jn);
        int64_t sum = static_cast<int64_t>(tiles) * same;
        for (int j = same; j < jn; ++j) sum += tiles - first_tile<R, BN, CAUSAL>(p, s, j);
        return sum;
    }
    // Key tiles that every row tile sees: the first so many of the sequence's jn.
    __device__ static __forceinline__ int seen_by_all(const ChunkSeq &s, int jn) {
        return !CAUSAL ? jn : (s.kv >= s.n ? min(jn, (s.kv - s.n) / BN + 1) : 0);
    }
    __device__ __forceinline__ void seq(const ChunkParams &p) {
        s = chunk_seq(p, b);
        jn = (s.kv + BN - 1) / BN;
        tiles = (s.n * p.G + R - 1) / R;
    }
    // one warp: where run `cta` begins (st->j: key tile); a run takes the items that begin in it
    __device__ static void locate(const ChunkParams &p, int cta, int ctas, KeyStart *st) {
        constexpr int PER = 4;
        const int lane = threadIdx.x & 31;
        int64_t cost[PER], total = 0, mine = 0;
        auto costs = [&](int base) {
            mine = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int b = base + lane * PER + i;
                cost[i] = b < p.num_seqs ? head_cost(p, chunk_seq(p, b)) * p.Hkv : 0;
                mine += cost[i];
            }
        };
        for (int base = 0; base < p.num_seqs; base += 32 * PER) {
            costs(base);
            total += warp_sum64(mine);
        }
        if (cta == 0)
            for (int b = lane; b < p.num_seqs; b += 32) chunk_check(p, b);
        const int64_t per = div_up_or_down(total, ctas, true), start = per * cta;
        if (lane == 0) *st = KeyStart{0, 0, 0, 0};
        __syncwarp();
        if (start >= total) return;
        int64_t before = 0;
        for (int base = 0; base < p.num_seqs; base += 32 * PER) {
            if (p.num_seqs > 32 * PER) costs(base);
            int64_t incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            int64_t at = before + incl - mine;
            if (start >= at && start < at + mine) {
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    if (start >= at && start < at + cost[i]) {
                        const int b = base + lane * PER + i;
                        const ChunkSeq s = chunk_seq(p, b);
                        const int tiles = (s.n * p.G + R - 1) / R;
                        int64_t rem = start - at;
                        const int64_t one = div_up_or_down(cost[i], p.Hkv, false);
                        int h = static_cast<int>(div_up_or_down(rem, one, false));
                        rem -= h * one;
                        // the first item whose own start lies at or after `start`
                        int j = static_cast<int>(min(static_cast<int64_t>(seen_by_all(s, (s.kv + BN - 1) / BN)),
                                                     div_up_or_down(rem, tiles, true)));
                        int64_t sum = static_cast<int64_t>(j) * tiles;
                        while (sum < rem) {
                            sum += tiles - first_tile<R, BN, CAUSAL>(p, s, j);
                            ++j;
                        }
                        const int64_t skipped = sum - rem;  // steps of the run that belong to an item begun before it
                        const int64_t left = min(per, total - start) - skipped;
                        *st = KeyStart{b, h, j, left};
                    }
                    at += cost[i];
                }
            }
            before += __shfl_sync(0xffffffffu, incl, 31);
        }
    }
    __device__ __forceinline__ bool begin(const ChunkParams &p, const KeyStart &st) {
        left = st.left;
        if (left <= 0) return false;
        b = st.b;
        h = st.h;
        j = st.j;
        seq(p);
        return settle(p);
    }
    // j may be one past the head's last tile: on to the next head or sequence
    __device__ __forceinline__ bool settle(const ChunkParams &p) {
        while (j >= jn || s.n == 0) {
            j = 0;
            if (s.n == 0 || jn == 0 || ++h == p.Hkv) {
                h = 0;
                if (++b >= p.num_seqs) return false;
                seq(p);
            }
        }
        t0 = first_tile<R, BN, CAUSAL>(p, s, j);
        return true;
    }
    __device__ __forceinline__ bool next(const ChunkParams &p) {
        left -= tiles - t0;
        if (left <= 0) return false;
        ++j;
        return settle(p);
    }
};

constexpr int kKeyBox = 128;  // cache rows of a TMA box, at most (fa_key_weights_tile.cu's too)

template <int D>
struct KeyCfg {
    static constexpr int R = 16;                   // rows a step
    // consumer warps (at D <= 64 four did not keep up with the memory: 95 us, eight 68, for 64 single tokens
    // over 8192), keys of each
    static constexpr int NW = D <= 64 ? 8 : 4, KPW = 32;
    static constexpr int BN = NW * KPW;
    static constexpr int SW = (2 * D >= 128) ? 128 : 2 * D;
    static constexpr int SWE = SW / 2, NBLK = D / SWE;
    static constexpr int STAGE = BN * D * 2;
    static constexpr int NS = STAGE >= 65536 ? 3 : (STAGE >= 32768 ? 6 : 8);
    static constexpr int OFF_BAR = NS * STAGE;
    static constexpr int OFF_START = OFF_BAR + 2 * NS * 8;
    static constexpr int OFF_ABORT = OFF_START + static_cast<int>(sizeof(KeyStart));
    static constexpr int SMEM = OFF_ABORT + 16 + 1024;
    static constexpr int THREADS = 32 * (NW + 1);
};

template <int D, bool BF16, bool CAUSAL>
__global__ void __launch_bounds__(KeyCfg<D>::THREADS, 1)
key_weights_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const ChunkParams p) {
    using C = KeyCfg<D>;
    constexpr int R = C::R, BN = C::BN, KPW = C::KPW, SW = C::SW, NS = C::NS;
    using Walk = KeyWalk<R, BN, CAUSAL>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR), *empty = full + NS;
    KeyStart *start = reinterpret_cast<KeyStart *>(smem + C::OFF_START);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_ABORT);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == C::NW * 32) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], C::NW);
        }
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_k);
    }
    if (warp == 0) Walk::locate(p, blockIdx.x, gridDim.x, start);
    __syncthreads();
    const KeyStart st = *start;
    if (warp == C::NW) {
        Walk w;
        bool bad = false;
        int u = 0;
        const uint64_t pol = l2_policy_evict_first();
        const int box = min(1 << p.page_shift, kKeyBox);
        for (bool more = w.begin(p, st); more; more = w.next(p), ++u) {
            const int stage = u % NS;
            if (u >= NS && !__all_sync(0xffffffffu, wait_bounded(&empty[stage], ((u / NS) - 1) & 1, abort_flag, p.timeout_ns, 730)))
                break;
            const int boxes = (min(BN, w.s.kv - w.j * BN) + box - 1) / box;
            if (lane == 0) mbar_arrive_expect_tx(&full[stage], boxes * box * D * 2);
            __syncwarp();
            uint8_t *dst = smem + stage * C::STAGE;
            for (int i = lane; i < boxes * C::NBLK; i += 32) {
                const int bx = i / C::NBLK, blk = i % C::NBLK;
                const int row = chunk_page_row(p, w.b, w.j * BN + bx * box, bad);
                tma_load_3d(dst + blk * BN * SW + bx * box * SW, &tm_k, &full[stage], blk * C::SWE, w.h, row, pol);
            }
        }
        if (__any_sync(0xffffffffu, bad) && lane == 0) record_error(FA_ERR_INDEX, 731);
        if (*abort_flag) {
            for (int v = max(0, u - NS); v < u; ++v) {
                const uint64_t t0 = global_timer_ns();
                while (!mbar_try_wait(&full[v % NS], (v / NS) & 1) && global_timer_ns() - t0 < p.timeout_ns) {
                }
            }
        }
    } else {
        const int g = lane >> 2, t4 = lane & 3, mi = lane >> 3, lr = lane & 7;
        const uint32_t base = smem_u32(smem);
        auto swz = [](int r, int cc) { return (cc ^ (SW == 128 ? (r & 7) : ((r >> 1) & 3))) << 4; };
        constexpr int CPB = SW / 16;
        Walk w;
        int u = 0;
        int hb = -1, hh = -1, ht = -1;       // whose Q rows are held
        uint32_t qf[2][D / 16][2];           // rows 0-7 and 8-15 of the tile as B fragments
        float ls[2][2];                      // lse in log2 units of rows 8 i + 2 t4, + 1 (inf: row absent)
        int lim[2][2];                       // keys each of them sees
        for (bool more = w.begin(p, st); more; more = w.next(p), ++u) {
            const int stage = u % NS;
            const int k0 = w.j * BN + warp * KPW;  // this warp's first key
            float *wp = p.weights + (static_cast<int64_t>(w.b) * p.Hkv + w.h) * p.width + k0;
            float was[2][2], sum[2][2];            // keys 16 i + g, + 8
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int key = i * 16 + k * 8 + g;
                    was[i][k] = (t4 == 0 && k0 + key < w.s.kv) ? wp[key] : 0.f;
                    sum[i][k] = 0.f;
                }
            if (!__all_sync(0xffffffffu, wait_bounded(&full[stage], (u / NS) & 1, abort_flag, p.timeout_ns, 732))) break;
            const uint32_t sk = base + stage * C::STAGE;
            for (int t = w.t0; t < w.tiles; ++t) {
                if (w.b != hb || w.h != hh || t != ht) {
                    hb = w.b;
                    hh = w.h;
                    ht = t;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int pr = t * R + i * 8 + g;
                        const bool there = pr < w.s.n * p.G;
                        const int64_t tok = w.s.q0 + (there ? pr / p.G : 0);
                        const uint32_t *q = reinterpret_cast<const uint32_t *>(
                            static_cast<const uint16_t *>(p.q) + (tok * p.Hq + w.h * p.G + (there ? pr % p.G : 0)) * D);
#pragma unroll
                        for (int k = 0; k < D / 16; ++k) {
                            qf[i][k][0] = there ? __ldg(q + k * 8 + t4) : 0u;
                            qf[i][k][1] = there ? __ldg(q + k * 8 + 4 + t4) : 0u;
                        }
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int r = t * R + i * 8 + 2 * t4 + k;
                            lim[i][k] = 0;
                            ls[i][k] = 0.f;
                            if (r < w.s.n * p.G) {
                                const float x = p.lse_in[static_cast<int64_t>(w.h * p.G + r % p.G) * p.total + w.s.q0 + r / p.G];
                                // a row that saw nothing above -inf gives no weight: 2^(s - inf)
                                ls[i][k] = x == -INFINITY ? INFINITY : x * 1.4426950408889634f;
                                lim[i][k] = token_keys<CAUSAL>(w.s, r / p.G);
                            }
                        }
                    }
                }
                float s[2][2][4];
#pragma unroll
                for (int i = 0; i < 16; ++i) (&s[0][0][0])[i] = 0.f;
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int r = warp * KPW + i * 16 + (mi & 1) * 8 + lr, ch = 2 * k + (mi >> 1);
                        uint32_t f[4];
                        ldmatrix_x4(f, sk + (ch / CPB) * BN * SW + r * SW + swz(r, ch % CPB));
                        mma_16816<BF16>(s[i][0], f, qf[0][k][0], qf[0][k][1]);
                        mma_16816<BF16>(s[i][1], f, qf[1][k][0], qf[1][k][1]);
                    }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int key = k0 + i * 16 + (k >> 1) * 8 + g;
                            const float x = ex2_approx(fmaf(s[i][n][k], p.scale_log2, -ls[n][k & 1]));
                            if (key < lim[n][k & 1]) sum[i][k >> 1] += x;
                        }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[stage]);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float x = sum[i][k];
                    x += __shfl_xor_sync(0xffffffffu, x, 1);
                    x += __shfl_xor_sync(0xffffffffu, x, 2);
                    const int key = i * 16 + k * 8 + g;
                    if (t4 == 0 && k0 + key < w.s.kv) wp[key] = was[i][k] + x;
                }
        }
    }
    __syncthreads();
}

template <int D, bool BF16, bool CAUSAL>
cudaError_t launch(const CUtensorMap &tk, const ChunkParams &p, int ctas, cudaStream_t st) {
    using C = KeyCfg<D>;
    auto kern = key_weights_rows_kernel<D, BF16, CAUSAL>;
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
    kern<<<ctas, C::THREADS, C::SMEM, st>>>(tk, p);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(bool bf16, bool causal, const CUtensorMap &tk, const ChunkParams &p, int ctas, cudaStream_t st) {
    if (bf16) return causal ? launch<D, true, true>(tk, p, ctas, st) : launch<D, true, false>(tk, p, ctas, st);
    return causal ? launch<D, false, true>(tk, p, ctas, st) : launch<D, false, false>(tk, p, ctas, st);
}

}  // namespace

cudaError_t launch_key_weights(int D, bool bf16, bool causal, const CUtensorMap &tk, const ChunkParams &p, int ctas,
                               cudaStream_t st) {
    switch (D) {
        case 32: return launch_d<32>(bf16, causal, tk, p, ctas, st);
        case 64: return launch_d<64>(bf16, causal, tk, p, ctas, st);
        case 128: return launch_d<128>(bf16, causal, tk, p, ctas, st);
        case 256: return launch_d<256>(bf16, causal, tk, p, ctas, st);
        default: return cudaErrorInvalidValue;
    }
}

int key_weights_box(int page_size) { return page_size < kKeyBox ? page_size : kKeyBox; }

cudaError_t key_weights_error_addrs(int **code, int **where) { return device_error_addrs(code, where); }

}  // namespace fa
