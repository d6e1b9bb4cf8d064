// fa_evict.cu -- eviction from a paged cache by accumulated attention weight (fa_paged_evict):
// which keys of each (sequence, key head) stay, and closing up their rows in place.
//
// Select. Of n > budget keys the last `recent` stay, and of the others the budget - recent of
// most weight, the lowest slot first where weights are equal. One CTA per (sequence, key head): the
// weight of rank k is found by a radix select over the order-preserving image of the float (11, 11 and 10
// bits, histograms in shared memory: with the exponent's last bits in the first digit few threads meet in a
// bin), then one pass in slot order writes the kept slots, with block-wide prefix sums over "kept" and
// "equal to the threshold". Everything is counted in integers: the result does not depend on
// the order of the threads.
//
// Move. Row j of the closed-up cache is row kept[j] >= j of the old one, so rows move towards the
// front only, and a CTA that walks j upwards in chunks may read a chunk ahead: what it writes, [j,
// j + CHUNK), no later chunk reads. Loads of a chunk are separated from its stores by a barrier.
// Columns are independent: a CTA takes SLICE bytes of one head's K or V rows, so that B * Hkv *
// (4 D / SLICE) CTAs share the bytes. Bound by reading and writing the rows that move (rows
// that stay in place are skipped).
//
// Measured: 16 sequences of up to 8192 keys, 8 heads of 128, cut to 2048: 71 us, of which the selection 15 and the
// moving 50 (273 MB: 5.5 TB/s); 3 of 777 to 300: 14 us, both kernels' latency. One sequence of 32768 keys to 4096 47 us,
// of 131072 to 16384 194: the selection is then one CTA for each of 8 heads, and past 16384 keys it reads the weights again
// in each pass. (Four passes of 8 bits in the
// selection, no overlap of the two kernels: 74 us.)
#include <cuda_runtime.h>
#include <stdint.h>

#include "fa.h"
#include "fa_internal.h"
#include "fa_sync.cuh"

namespace fa {

namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelItems = 4;   // consecutive slots per thread
constexpr int kHistCopies = 2, kBins = 2048;
constexpr int kSelHeld = 16;   // images held in a thread's registers over the passes (the rest is read again)

// Order-preserving image: a > b as floats <=> image(a) > image(b); -0 equals 0, NaN is above +inf.
__device__ __forceinline__ uint32_t weight_image(float w) {
    if (w != w) return 0xffffffffu;
    const uint32_t u = __float_as_uint(w + 0.0f);  // -0 + 0 = 0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Block-wide exclusive prefix sum of a packed pair of counts; `total` receives the block's sum.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *warp_sums, uint32_t &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    uint32_t w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += x;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    const uint32_t before = warp == 0 ? 0u : __shfl_sync(0xffffffffu, w, warp - 1);
    __syncthreads();
    return before + incl - v;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p) {
    __shared__ __align__(8) uint32_t hist[kHistCopies][kBins];
    __shared__ uint32_t warp_sums[32];
    __shared__ uint32_t s_digit, s_rank;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the moving CTAs may wait beside these
    const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
    const int64_t bh = static_cast<int64_t>(b) * p.Hkv + h;
    const float *w = p.weights + bh * p.width;
    float *nw = p.new_weights + bh * p.width;
    int32_t *kept = p.kept + bh * p.budget;
    const int raw = p.kv_lens[b];
    const int n = min(max(raw, 0), p.capacity);
    if (raw != n && h == 0 && tid == 0) record_error(FA_ERR_INDEX, 740);
    const int m = min(n, p.budget);
    if (h == 0 && tid == 0) p.new_lens[b] = m;
    if (n <= p.budget) {
        for (int i = tid; i < p.width; i += kSelThreads) nw[i] = i < n ? w[i] : 0.f;
        for (int i = tid; i < p.budget; i += kSelThreads) kept[i] = i < n ? i : -1;
        return;
    }
    const int old = n - min(n, p.recent);  // slots that compete
    const int k = p.budget - (n - old);    // of which this many stay
    uint32_t threshold = 0xffffffffu;      // stay: image above it, and `ties` of those equal to it
    uint32_t ties = 0;
    if (k > 0) {
        uint32_t prefix = 0, rank = k;  // the rank-th largest among those that match the prefix
        uint32_t held[kSelHeld];
#pragma unroll
        for (int q = 0; q < kSelHeld; ++q) {
            const int i = q * kSelThreads + tid;
            held[q] = i < old ? weight_image(w[i]) : 0u;
        }
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), above = pass == 1 ? 21 : 10;  // 11, 11, 10 bits
            const uint32_t digits = pass == 2 ? 1023u : 2047u;
            for (int i = tid; i < kHistCopies * kBins; i += kSelThreads) (&hist[0][0])[i] = 0;
            __syncthreads();
            uint32_t *mine = hist[(tid >> 5) % kHistCopies];
            auto count = [&](uint32_t x) {
                if (pass == 0 || (x >> above) == (prefix >> above)) atomicAdd(&mine[(x >> shift) & digits], 1u);
            };
#pragma unroll
            for (int q = 0; q < kSelHeld; ++q)
                if (q * kSelThreads + tid < old) count(held[q]);
            for (int i = kSelHeld * kSelThreads + tid; i < old; i += kSelThreads) count(weight_image(w[i]));
            __syncthreads();
            // thread t takes digits 2 (1023 - t) + 1 and 2 (1023 - t): ranks from the largest digit down
            uint32_t c[2] = {0, 0};
#pragma unroll
            for (int q = 0; q < kHistCopies; ++q) {
                const uint2 v = *reinterpret_cast<const uint2 *>(&hist[q][2 * (kSelThreads - 1 - tid)]);
                c[0] += v.y;
                c[1] += v.x;
            }
            uint32_t total;
            const uint32_t before = block_scan(c[0] + c[1], warp_sums, total);
            if (before < rank && rank <= before + c[0] + c[1]) {
                const bool first = rank <= before + c[0];
                s_digit = 2 * (kSelThreads - 1 - tid) + (first ? 1 : 0);
                s_rank = rank - before - (first ? 0 : c[0]);
            }
            __syncthreads();
            prefix |= s_digit << shift;
            rank = s_rank;
        }
        threshold = prefix;
        ties = rank;
    }
    // kept slots in order; packed counts: kept outright (low half), equal to the threshold (high)
    uint32_t base = 0, equal = 0;
    for (int i0 = 0; i0 < n; i0 += kSelThreads * kSelItems) {
        uint32_t flag[kSelItems], c = 0;
        float x[kSelItems];
#pragma unroll
        for (int q = 0; q < kSelItems; ++q) {
            const int i = i0 + tid * kSelItems + q;
            flag[q] = 0;
            x[q] = 0.f;
            if (i < n) {
                x[q] = w[i];
                const uint32_t im = weight_image(x[q]);
                if (i >= old || (k > 0 && im > threshold)) flag[q] = 1u;
                else if (k > 0 && im == threshold) flag[q] = 1u << 16;
            }
            c += flag[q];
        }
        uint32_t total;
        const uint32_t at = block_scan(c, warp_sums, total);
        uint32_t out = base + (at & 0xffffu), eq = equal + (at >> 16);
        // of the equal ones before this slot, those that stay count too
        uint32_t pos = out + min(eq, ties);
#pragma unroll
        for (int q = 0; q < kSelItems; ++q) {
            const int i = i0 + tid * kSelItems + q;
            bool stay = flag[q] == 1u;
            if (flag[q] == 1u << 16) {
                stay = eq < ties;
                ++eq;
            }
            if (stay) {
                kept[pos] = i;
                nw[pos] = x[q];
                ++pos;
            }
        }
        base += total & 0xffffu;
        equal += total >> 16;
    }
    for (int i = m + tid; i < p.width; i += kSelThreads) nw[i] = 0.f;
}

constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 4;

// One head's K (first half of blockIdx.x's slices) or V rows, SLICE bytes of each. In the iteration of
// chunk c the loads of chunk c + 1 are issued and the places of chunk c + 2 looked up before chunk c is
// stored.
template <int SLICE>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p, int slices) {
    constexpr int LPR = SLICE / 16;               // lanes a row
    constexpr int RPT = kMoveThreads / LPR;       // rows of one load of the CTA
    constexpr int U = kMoveUnroll, CHUNK = RPT * U;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int b = blockIdx.z, h = blockIdx.y;
    const int n = min(max(p.kv_lens[b], 0), p.capacity);
    if (n <= p.budget) return;
    const int half = slices / 2;
    const bool is_v = static_cast<int>(blockIdx.x) >= half;
    const int slice = blockIdx.x - (is_v ? half : 0);
    const int64_t row_bytes = static_cast<int64_t>(p.Hkv) * p.D * 2;
    uint8_t *pool = static_cast<uint8_t *>(is_v ? p.v_cache : p.k_cache) + static_cast<int64_t>(h) * p.D * 2 + slice * SLICE +
                    (threadIdx.x % LPR) * 16;
    const int32_t *kept = p.kept + (static_cast<int64_t>(b) * p.Hkv + h) * p.budget;
    const int32_t *bt = p.block_table + static_cast<int64_t>(b) * p.max_blocks;
    const int r = threadIdx.x / LPR, mask = (1 << p.page_shift) - 1;
    bool bad = false;
    // rows of the pool that chunk j0 moves (to: -1 where nothing moves)
    auto places = [&](int j0, int *from, int *to) {
        int src[U];
#pragma unroll
        for (int q = 0; q < U; ++q) {
            const int j = j0 + q * RPT + r;
            src[q] = j < p.budget ? __ldcg(kept + j) : j;
        }
#pragma unroll
        for (int q = 0; q < U; ++q) {
            const int j = j0 + q * RPT + r;
            from[q] = to[q] = -1;
            if (src[q] != j) {
                const int pf = __ldg(bt + (src[q] >> p.page_shift)), pt = __ldg(bt + (j >> p.page_shift));
                if (pf < 0 || pf >= p.num_pages || pt < 0 || pt >= p.num_pages) {
                    bad = true;
                } else {
                    from[q] = (pf << p.page_shift) + (src[q] & mask);
                    to[q] = (pt << p.page_shift) + (j & mask);
                }
            }
        }
    };
    int from[U], to[U], nfrom[U], nto[U];
    uint4 v[U], nv[U];
    auto fetch = [&](const int *at, uint4 *x) {
#pragma unroll
        for (int q = 0; q < U; ++q)
            if (at[q] >= 0)
                asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(x[q].x), "=r"(x[q].y), "=r"(x[q].z), "=r"(x[q].w)
                             : "l"(pool + at[q] * row_bytes)
                             : "memory");
    };
    places(0, from, to);
    fetch(from, v);
    places(CHUNK, nfrom, nto);
    for (int j0 = 0; j0 < p.budget; j0 += CHUNK) {
        int ffrom[U], fto[U];
        fetch(nfrom, nv);
        places(j0 + 2 * CHUNK, ffrom, fto);
        __syncthreads();  // chunk j0 is read (by all) before any of it is written
#pragma unroll
        for (int q = 0; q < U; ++q)
            if (to[q] >= 0) *reinterpret_cast<uint4 *>(pool + to[q] * row_bytes) = v[q];
#pragma unroll
        for (int q = 0; q < U; ++q) {
            v[q] = nv[q];
            to[q] = nto[q];
            nfrom[q] = ffrom[q];
            nto[q] = fto[q];
        }
    }
    if (bad) record_error(FA_ERR_INDEX, 741);
}

template <int SLICE>
cudaError_t launch_move(const EvictParams &p, cudaStream_t st) {
    const int slices = 2 * p.D * 2 / SLICE;
    cudaLaunchConfig_t cfg = {};  // waits on the device for the kept slots
    cfg.gridDim = dim3(slices, p.Hkv, p.batch);
    cfg.blockDim = dim3(kMoveThreads, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, evict_move_kernel<SLICE>, p, slices);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, cudaStream_t st) {
    evict_select_kernel<<<dim3(p.Hkv, p.batch), kSelThreads, 0, st>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // Wider slices are kinder to the memory, narrower ones make more CTAs. 8192 keys cut to 2048, 8 heads of 128, slices of
    // 32 / 64 / 128 / 256 bytes (us), the rule's the best of them or within 6 %:
    //   sequences  2: 25 / 27 / 34 / 51     4: 31 / 33 / 40 / 58      8: 49 / 43 / 53 / 68      12: 68 / 64 / 64 / 91
    //             16: 86 / 74 / 71 / 92    24: 131 / 114 / 119 / 115  32: 167 / 142 / 136 / 129  64: 330 / 270 / 264 / 251
    const int64_t bytes = static_cast<int64_t>(p.batch) * p.Hkv * p.D * 4;  // of all heads' K and V rows
    if (bytes >= 1024 * 256 && p.D >= 128) return launch_move<256>(p, st);
    if (bytes >= 512 * 128 && p.D >= 64) return launch_move<128>(p, st);
    if (bytes >= 256 * 64) return launch_move<64>(p, st);
    return launch_move<32>(p, st);
}

cudaError_t evict_error_addrs(int **code, int **where) { return device_error_addrs(code, where); }

}  // namespace fa
