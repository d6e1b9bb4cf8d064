// fa_chunk_rows.cu -- attention of new tokens over a paged cache where a key head has few rows
// (fa_fwd_paged_chunk; single tokens above all): tiles of 16 rows, bounded by reading K and V.
//
// A row reads every key of its sequence and does 4 D operations with 4 D bytes of K and V that
// its group shares, so with up to 16 rows the time is that of the bytes; what the kernel needs is
// loads in flight and an SM that never waits for arithmetic. One CTA per SM walks an equal run of
// the steps of all items (fa_chunk.cuh):
//   last warp    producer: brings K and V tiles of BN keys through an NS-stage ring by TMA, a box
//                per page piece, the lanes issuing a tile's boxes side by side.
//   consumers    (4 warps, 8 at D <= 64) each takes 16 keys of every tile by itself: S = Q K^T and O += P V with
//                mma.sync m16n8k16 (16 rows fill the tile; a 128-row tcgen05 tile would compute 8 to
//                128 times the rows there are, and its softmax would run one row per thread), its
//                own running (m, l) and its own O in registers, so that warps meet only at the
//                end of an item, where they are joined through shared memory.
// The running maximum is in log2 units and moves only when it grows by more than 2^8 (the final
// 1/l cancels it exactly); P is rounded to the input type for the second product, the sums l take
// the unrounded values; all statistics and O are 32-bit.
// Rows of V past the last key (a page's tail) are cleared in shared memory before they meet P = 0:
// a NaN left in a page does not reach the output.
//
// Measured: 64 single tokens over up to 8192 keys (32 heads on 8, D = 128) 207 us for 1344 MB, 6.5 TB/s, a copy's
// rate; the same at D = 64 122, at D = 32 77; 4 over up to 1000 keys 16 us (14.5 from a graph), of which the bytes would take 3:
// the rest is latency (the first scores after 4, the last items done after 10, joining 3).
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

template <int D>
struct RowsCfg {
    static constexpr int R = 16;
    static constexpr int NW = D <= 64 ? 8 : 4;       // consumer warps
    static constexpr int KPW = 16;                   // keys a warp takes of a tile
    static constexpr int BN = NW * KPW;
    static constexpr int SW = (2 * D >= 128) ? 128 : 2 * D;
    static constexpr int SWE = SW / 2;
    static constexpr int NBLK = D / SWE;
    static constexpr int TILE = BN * D * 2;          // bytes of a K (or V) tile
    static constexpr int STAGE = 2 * TILE;
    // 128 KB on the way (192 at D = 256, whose stages are 64 KB): with more, the memory's rate falls (64 single
    // tokens over 8192, D = 128: 192 KB 216 us, 160 KB 208, 128 KB 207).
    static constexpr int NS = STAGE >= 65536 ? 3 : (STAGE >= 32768 ? 4 : 8);
    static constexpr int DH = D < 128 ? D : 128;     // columns of O joined at a time
    static constexpr int OROW = DH + 4;              // floats; keeps the 8 rows of a store apart in the banks
    static constexpr int OFF_O = NS * STAGE;
    static constexpr int OFF_ML = OFF_O + NW * R * OROW * 4;
    static constexpr int OFF_BAR = OFF_ML + NW * R * 8;
    static constexpr int OFF_START = OFF_BAR + 2 * NS * 8;
    static constexpr int OFF_ABORT = OFF_START + static_cast<int>(sizeof(ChunkStart));
    static constexpr int SMEM = OFF_ABORT + 16 + 1024;
    static constexpr int THREADS = 32 * (NW + 1);
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

template <int THREADS>
__device__ __forceinline__ void consumers_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

template <int D, bool BF16, bool CAUSAL>
__global__ void __launch_bounds__(RowsCfg<D>::THREADS, 1)
chunk_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const ChunkParams p) {
    using C = RowsCfg<D>;
    constexpr int R = C::R, BN = C::BN, KPW = C::KPW, SW = C::SW, NS = C::NS;
    using Walk = ChunkWalk<1, BN, 0, CAUSAL>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *sO = reinterpret_cast<float *>(smem + C::OFF_O);
    float2 *sML = reinterpret_cast<float2 *>(smem + C::OFF_ML);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR), *empty = full + NS;
    ChunkStart *start = reinterpret_cast<ChunkStart *>(smem + C::OFF_START);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_ABORT);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    pdl_launch_dependents();
    if (threadIdx.x == C::NW * 32) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], C::NW);
        }
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    if (warp == 0) chunk_locate<1, BN, 0, CAUSAL>(p, blockIdx.x, gridDim.x, start);
    __syncthreads();

    if (warp == C::NW) {
        // ------------------------------------------------------------ producer
        int u = 0;  // stages filled
        const uint64_t pol = l2_policy_evict_first();
        const int log = min(p.page_shift, BN == 64 ? 6 : 7);
        ChunkTiles<Walk, BN> tiles(p, start, log);
        const BoxLane<C::NBLK, BN, SW> bl(p.page_shift, log);
        while (tiles.take(p)) {
            const int stage = u % NS, n = bl.boxes(tiles.valid), row = __shfl_sync(0xffffffffu, tiles.row, bl.from);
            if (u >= NS && !__all_sync(0xffffffffu, wait_bounded(&empty[stage], ((u / NS) - 1) & 1, abort_flag, p.timeout_ns, 710)))
                break;
            if (lane == 0) mbar_arrive_expect_tx(&full[stage], 2 * bl.bytes(n));
            __syncwarp();
            if (bl.box < n) {
                uint8_t *dst = smem + stage * C::STAGE + bl.dst;
                tma_load_3d(dst, &tm_k, &full[stage], bl.blk * C::SWE, tiles.h, row, pol);
                tma_load_3d(dst + C::TILE, &tm_v, &full[stage], bl.blk * C::SWE, tiles.h, row, pol);
            }
            ++u;
        }
        if (__any_sync(0xffffffffu, tiles.bad) && lane == 0) record_error(FA_ERR_INDEX, 711);
        if (*abort_flag) {  // the copies in flight land before the shared memory goes away
            for (int v = max(0, u - NS); v < u; ++v) {
                const uint64_t t0 = global_timer_ns();
                while (!mbar_try_wait(&full[v % NS], (v / NS) & 1) && global_timer_ns() - t0 < p.timeout_ns) {
                }
            }
        }
    } else {
        // ------------------------------------------------------------ consumers
        const int g = lane >> 2, t4 = lane & 3;
        const int mi = lane >> 3, lr = lane & 7;  // ldmatrix: matrix and row this lane addresses
        const uint32_t base = smem_u32(smem);
        auto swz = [](int r, int cc) { return (cc ^ (SW == 128 ? (r & 7) : ((r >> 1) & 3))) << 4; };
        constexpr int CPB = SW / 16;
        bool ok = true;
        int u = 0;
        ChunkDesc desc{0, 0, 0, 0};
        Walk w;
        for (bool more = w.begin(p, start); more; more = w.next(p)) {
            // Q rows g and g + 8 of the tile as A fragments
            uint32_t qf[D / 16][4];
            const uint32_t *q0 = nullptr, *q1 = nullptr;
            int lim0 = w.keys, lim1 = w.keys;  // keys each row sees (rows past the last: any)
            {
                const int rows = w.tokens * p.G;
                auto row = [&](int r, int &lim) -> const uint32_t * {
                    if (r >= rows) return nullptr;
                    const int i = w.i0 + r / p.G;
                    lim = token_keys<CAUSAL>(w.s, i);
                    return reinterpret_cast<const uint32_t *>(
                        static_cast<const uint16_t *>(p.q) + (static_cast<int64_t>(w.s.q0 + i) * p.Hq + w.h * p.G + r % p.G) * D);
                };
                q0 = row(g, lim0);
                q1 = row(g + 8, lim1);
            }
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                qf[k][0] = q0 ? __ldg(q0 + k * 8 + t4) : 0u;
                qf[k][1] = q1 ? __ldg(q1 + k * 8 + t4) : 0u;
                qf[k][2] = q0 ? __ldg(q0 + k * 8 + 4 + t4) : 0u;
                qf[k][3] = q1 ? __ldg(q1 + k * 8 + 4 + t4) : 0u;
            }
            const int all_see = CAUSAL ? token_keys<CAUSAL>(w.s, w.i0) : w.keys;  // keys that every row sees
            float o[D / 8][4];
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[i][k] = 0.f;
            float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
            for (int j = w.j0; j < w.j1; ++j, ++u) {
                const int stage = u % NS;
                if (ok) ok = __all_sync(0xffffffffu, wait_bounded(&full[stage], (u / NS) & 1, abort_flag, p.timeout_ns, 720));
                const int k0 = j * BN + warp * KPW;  // this warp's first key
                const int mine = min(KPW, w.keys - k0);
                if (ok && mine > 0) {
                    const uint32_t sk = base + stage * C::STAGE, sv = sk + C::TILE;
                    const int kr = warp * KPW;
                    if (mine < KPW) {
                        // V rows past the last key hold whatever the page or the ring held
                        constexpr int CH = D / 8;
                        for (int i = lane; i < (KPW - mine) * CH; i += 32) {
                            const int r = kr + mine + i / CH, ch = i % CH;
                            st_shared_v4(sv + (ch / CPB) * BN * SW + r * SW + swz(r, ch % CPB), 0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();  // before a later copy into the same rows
                        __syncwarp();
                    }
                    float s[KPW / 8][4];
#pragma unroll
                    for (int i = 0; i < KPW / 8; ++i)
#pragma unroll
                        for (int k = 0; k < 4; ++k) s[i][k] = 0.f;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
#pragma unroll
                        for (int i = 0; i < KPW / 16; ++i) {
                            const int r = kr + i * 16 + (mi >> 1) * 8 + lr, ch = 2 * k + (mi & 1);
                            uint32_t f[4];
                            ldmatrix_x4(f, sk + (ch / CPB) * BN * SW + r * SW + swz(r, ch % CPB));
                            mma_16816<BF16>(s[2 * i], qf[k], f[0], f[1]);
                            mma_16816<BF16>(s[2 * i + 1], qf[k], f[2], f[3]);
                        }
                    }
                    if (k0 + KPW > all_see || mine < KPW) {
#pragma unroll
                        for (int i = 0; i < KPW / 8; ++i)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (k0 + i * 8 + 2 * t4 + (k & 1) >= (k < 2 ? lim0 : lim1)) s[i][k] = -INFINITY;
                    }
                    float x0 = fmaxf(s[0][0], s[0][1]), x1 = fmaxf(s[0][2], s[0][3]);
#pragma unroll
                    for (int i = 1; i < KPW / 8; ++i) {
                        x0 = fmax3(x0, s[i][0], s[i][1]);
                        x1 = fmax3(x1, s[i][2], s[i][3]);
                    }
                    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
                    x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
                    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2)) * p.scale_log2;
                    x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2)) * p.scale_log2;
                    const bool grow0 = x0 > m0 + 8.f, grow1 = x1 > m1 + 8.f;
                    if (__any_sync(0xffffffffu, grow0 || grow1)) {
                        float a0 = 1.f, a1 = 1.f;
                        if (grow0) { a0 = ex2_approx(m0 - x0); m0 = x0; }
                        if (grow1) { a1 = ex2_approx(m1 - x1); m1 = x1; }
                        l0 *= a0;
                        l1 *= a1;
#pragma unroll
                        for (int i = 0; i < D / 8; ++i) {
                            o[i][0] *= a0; o[i][1] *= a0;
                            o[i][2] *= a1; o[i][3] *= a1;
                        }
                    }
                    const float n0 = m0 == -INFINITY ? 0.f : -m0, n1 = m1 == -INFINITY ? 0.f : -m1;
#pragma unroll
                    for (int i = 0; i < KPW / 8; ++i) {
                        s[i][0] = ex2_approx(fmaf(s[i][0], p.scale_log2, n0));
                        s[i][1] = ex2_approx(fmaf(s[i][1], p.scale_log2, n0));
                        s[i][2] = ex2_approx(fmaf(s[i][2], p.scale_log2, n1));
                        s[i][3] = ex2_approx(fmaf(s[i][3], p.scale_log2, n1));
                        l0 += s[i][0] + s[i][1];
                        l1 += s[i][2] + s[i][3];
                    }
#pragma unroll
                    for (int i = 0; i < KPW / 16; ++i) {
                        uint32_t a[4];
                        a[0] = pack16<BF16>(s[2 * i][0], s[2 * i][1]);
                        a[1] = pack16<BF16>(s[2 * i][2], s[2 * i][3]);
                        a[2] = pack16<BF16>(s[2 * i + 1][0], s[2 * i + 1][1]);
                        a[3] = pack16<BF16>(s[2 * i + 1][2], s[2 * i + 1][3]);
                        const int r = kr + i * 16 + (mi & 1) * 8 + lr;
#pragma unroll
                        for (int nd = 0; nd < D / 16; ++nd) {
                            const int ch = 2 * nd + (mi >> 1);
                            uint32_t f[4];
                            ldmatrix_x4_trans(f, sv + (ch / CPB) * BN * SW + r * SW + swz(r, ch % CPB));
                            mma_16816<BF16>(o[2 * nd], a, f[0], f[1]);
                            mma_16816<BF16>(o[2 * nd + 1], a, f[2], f[3]);
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[stage]);
            }
            // ---- join the warps' rows
            l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
            l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
            l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
            l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
            if (t4 == 0) {
                sML[warp * R + g] = make_float2(m0, l0);
                sML[warp * R + g + 8] = make_float2(m1, l1);
            }
            const bool whole = w.whole();
            const int rows = w.tokens * p.G;
            constexpr int TPR = 2 * C::NW;                             // threads a row
            const int row = threadIdx.x / TPR, col8 = threadIdx.x % TPR;
#pragma unroll
            for (int half = 0; half < D / C::DH; ++half) {
                constexpr int NT = C::DH / 8;
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const float *oi = o[half * NT + i];
                    if (g < rows)
                        *reinterpret_cast<float2 *>(sO + (warp * R + g) * C::OROW + i * 8 + 2 * t4) = make_float2(oi[0], oi[1]);
                    if (g + 8 < rows)
                        *reinterpret_cast<float2 *>(sO + (warp * R + g + 8) * C::OROW + i * 8 + 2 * t4) = make_float2(oi[2], oi[3]);
                }
                consumers_sync<32 * C::NW>();
                if (row < rows) {
                    float m = -INFINITY, l = 0.f, a[C::NW];
#pragma unroll
                    for (int v = 0; v < C::NW; ++v) m = fmaxf(m, sML[v * R + row].x);
#pragma unroll
                    for (int v = 0; v < C::NW; ++v) {
                        const float2 ml = sML[v * R + row];
                        a[v] = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - m);
                        l = fmaf(ml.y, a[v], l);
                    }
                    const int64_t tok = w.s.q0 + w.i0 + row / p.G;
                    const int head = w.h * p.G + row % p.G;
                    const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
                    uint16_t *out = static_cast<uint16_t *>(p.out) + (tok * p.Hq + head) * D + half * C::DH;
                    const int64_t slot = w.slot();
                    float *po = p.part_o + (slot * D + half * C::DH) * R + row;
#pragma unroll
                    for (int c = 0; c < (C::DH + 4 * TPR - 1) / (4 * TPR); ++c) {
                        const int col = c * (4 * TPR) + col8 * 4;
                        if (col >= C::DH) break;
                        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int v = 0; v < C::NW; ++v) {
                            const float4 y = *reinterpret_cast<const float4 *>(sO + (v * R + row) * C::OROW + col);
                            x.x = fmaf(y.x, a[v], x.x);
                            x.y = fmaf(y.y, a[v], x.y);
                            x.z = fmaf(y.z, a[v], x.z);
                            x.w = fmaf(y.w, a[v], x.w);
                        }
                        if (whole) {
                            *reinterpret_cast<uint2 *>(out + col) =
                                make_uint2(pack16<BF16>(x.x * inv, x.y * inv), pack16<BF16>(x.z * inv, x.w * inv));
                        } else {
                            po[col * R] = x.x;
                            po[(col + 1) * R] = x.y;
                            po[(col + 2) * R] = x.z;
                            po[(col + 3) * R] = x.w;
                        }
                    }
                    if (half == 0 && col8 == 0) {
                        if (!whole)
                            p.part_ml[slot * R + row] = make_float2(m, l);
                        else if (p.lse)
                            p.lse[static_cast<int64_t>(head) * p.total + tok] =
                                l == 0.f ? -INFINITY : m * 0.6931471805599453f + logf(l);
                    }
                }
                consumers_sync<32 * C::NW>();
            }
            if (w.j0 == 0 && w.j1 < w.steps) desc = w.desc(p);
        }
        if (threadIdx.x == 0) p.desc[blockIdx.x] = desc;
    }
    __syncthreads();
}

template <int D, bool BF16, bool CAUSAL>
cudaError_t launch(const CUtensorMap &tk, const CUtensorMap &tv, const ChunkParams &p, int ctas, cudaStream_t st) {
    using C = RowsCfg<D>;
    auto kern = chunk_rows_kernel<D, BF16, CAUSAL>;
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
    kern<<<ctas, C::THREADS, C::SMEM, st>>>(tk, tv, p);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_combine<D, BF16, C::R>(p, ctas, st);
}

template <int D>
cudaError_t launch_d(bool bf16, bool causal, const CUtensorMap &tk, const CUtensorMap &tv, const ChunkParams &p, int ctas,
                     cudaStream_t st) {
    if (bf16) return causal ? launch<D, true, true>(tk, tv, p, ctas, st) : launch<D, true, false>(tk, tv, p, ctas, st);
    return causal ? launch<D, false, true>(tk, tv, p, ctas, st) : launch<D, false, false>(tk, tv, p, ctas, st);
}

}  // namespace

cudaError_t launch_chunk_rows(int D, bool bf16, bool causal, const CUtensorMap &tk, const CUtensorMap &tv,
                              const ChunkParams &p, int ctas, cudaStream_t st) {
    switch (D) {
        case 32: return launch_d<32>(bf16, causal, tk, tv, p, ctas, st);
        case 64: return launch_d<64>(bf16, causal, tk, tv, p, ctas, st);
        case 128: return launch_d<128>(bf16, causal, tk, tv, p, ctas, st);
        case 256: return launch_d<256>(bf16, causal, tk, tv, p, ctas, st);
        default: return cudaErrorInvalidValue;
    }
}

int chunk_rows_tile() { return 16; }
int chunk_rows_box(int D, int page_size) {
    const int bn = D <= 64 ? 128 : 64;
    return page_size < bn ? page_size : bn;
}

cudaError_t chunk_rows_error_addrs(int **code, int **where) { return device_error_addrs(code, where); }

}  // namespace fa
