// fa_evict.cu -- eviction from a paged cache by accumulated attention weight (fa_paged_evict):
// which keys of each (sequence, key head) stay, and closing up their rows in place.
//
// Select. Of n > budget keys the last `recent` stay, and of the others the budget - recent of
// most weight, the lowest slot first where weights are equal. One CTA per (sequence, key head): the
// weight of rank k is found by a radix select over the order-preserving image of the float (four
// passes of 8 bits, histograms in shared memory, one copy per warp group against contention),
// then one pass in slot order writes the kept slots, with block-wide prefix sums over "kept" and
// "equal to the threshold". Everything is counted in integers: the result does not depend on
// the order of the threads.
//
// Move. Row j of the closed-up cache is row kept[j] >= j of the old one, so rows move towards the
// front only, and a CTA that walks j upwards in chunks may read a chunk ahead: what it writes, [j,
// j + CHUNK), no later chunk reads. Loads of a chunk are separated from its stores by a barrier.
// Columns are independent: a CTA takes SLICE bytes of one head's K or V rows, so that B * Hkv *
// (4 D / SLICE) CTAs share the bytes. Bound by reading and writing the rows that move (rows
// that stay in place are skipped).
#include <cuda_runtime.h>
#include <stdint.h>

#include "fa.h"
#include "fa_internal.h"
#include "fa_sync.cuh"

namespace fa {

namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelItems = 4;   // consecutive slots per thread
constexpr int kHistCopies = 8;
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
    __shared__ uint32_t hist[kHistCopies][256];
    __shared__ uint32_t warp_sums[32];
    __shared__ uint32_t s_digit, s_rank;
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
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < kHistCopies * 256; i += kSelThreads) (&hist[0][0])[i] = 0;
            __syncthreads();
            uint32_t *mine = hist[(tid >> 5) % kHistCopies];
            auto count = [&](uint32_t x, bool valid) {
                if (shift == 24) {
                    // the top byte (sign and exponent) takes few values: one addition per value and warp
                    const uint32_t d = valid ? x >> 24 : 256u;
                    const uint32_t peers = __match_any_sync(0xffffffffu, d);
                    if (valid && (threadIdx.x & 31) == __ffs(peers) - 1) atomicAdd(&mine[d], __popc(peers));
                } else if (valid && (x >> (shift + 8)) == (prefix >> (shift + 8))) {
                    atomicAdd(&mine[(x >> shift) & 255], 1u);
                }
            };
#pragma unroll
            for (int q = 0; q < kSelHeld; ++q)
                if (q * kSelThreads < old) count(held[q], q * kSelThreads + tid < old);
            for (int i0 = kSelHeld * kSelThreads; i0 < old; i0 += kSelThreads)
                count(i0 + tid < old ? weight_image(w[i0 + tid]) : 0u, i0 + tid < old);
            __syncthreads();
            if (tid < 256) {  // thread d takes digit 255 - d: ranks from the largest digit down
                uint32_t c = 0;
#pragma unroll
                for (int q = 0; q < kHistCopies; ++q) c += hist[q][255 - tid];
                uint32_t incl = c;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
                    if ((tid & 31) >= o) incl += x;
                }
                if ((tid & 31) == 31) warp_sums[tid >> 5] = incl;
                asm volatile("bar.sync 1, 256;" ::: "memory");
                for (int i = 0; i < (tid >> 5); ++i) incl += warp_sums[i];
                if (incl - c < rank && rank <= incl) {
                    s_digit = 255 - tid;
                    s_rank = rank - (incl - c);
                }
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
            src[q] = j < p.budget ? __ldg(kept + j) : j;
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
    const int which = p.slice ? p.slice : 64;
    if (which >= 256 && p.D >= 128) return launch_move<256>(p, st);
    if (which >= 128 && p.D >= 64) return launch_move<128>(p, st);
    return launch_move<64>(p, st);
}

cudaError_t evict_error_addrs(int **code, int **where) { return device_error_addrs(code, where); }

}  // namespace fa
