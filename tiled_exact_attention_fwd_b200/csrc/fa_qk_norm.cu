// fa_qk_norm.cu -- RMS norm of queries and keys for each head and the position rotation, in one
// pass over the data (fa_qk_norm_rope), the same with k and v written into the pages of a cache
// (fa_qk_norm_rope_paged), and the gradients (fa_qk_norm_rope_bwd).
//
// Mathematics, for one head row x of D values, weights w, and the token's angles (c, s):
//   r = 1 / sqrt(mean(x^2) + eps),  n = w x r,  y = R n,
//   R turns the pairs (a, b) of the first `rot` values: (a c - b s, b c + a s); a pair is (i,
//   i + rot/2), or (2i, 2i + 1) when interleaved. (r is the row's, so it is multiplied in last.)
// Backward: g = R^T dy (the angles turned back), u = w g, t = sum(u x),
//   dx = r u - x r^3 t / D,  dw = sum over tokens and heads of g x r.
//
// Everything is bytes: each row is read once and written once (backward: x and dy read, dx
// written). A lane takes two 16-byte chunks of a row, chosen so that both halves of each pair are
// its own (Turn): no exchange but the row's sum, log2(D / 16) shuffles, and all arithmetic in pairs of
// floats (with a chunk a lane, and the partners' values by shuffles, the instructions took as long as the
// bytes). Two CTAs an SM walk over the tokens, each warp with the rows of two batches in flight while it
// works on one. All arithmetic is 32-bit; an output is rounded once. The weight gradients are summed in
// registers, then over the CTA's warps in shared memory, then over the CTAs by a second launch in a
// fixed order (no atomics: the same inputs give the same bits).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "fa.h"
#include "fa_internal.h"
#include "fa_ptx.cuh"
#include "fa_seq.cuh"
#include "fa_sync.cuh"

namespace fa {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Eight 16-bit values as four pairs of floats, and back (one rounding).
template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4 &v, uint64_t *f) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (BF16) {
            f[i] = f2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
        } else {
            const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
            f[i] = f2(t.x, t.y);
        }
    }
}
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const uint64_t *f) {
    uint4 v;
    uint32_t *u = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        f2_split(f[i], lo, hi);
        u[i] = BF16 ? pack2_bf16(lo, hi) : pack2_f16(lo, hi);
    }
    return v;
}

// Eight weights from element e on (ones where there are none).
template <bool BF16>
__device__ __forceinline__ void load_weights(const void *w, int w32, int e, uint64_t *f) {
    if (!w) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = f2(1.f, 1.f);
    } else if (w32) {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(w) + e);
        const float4 a = __ldg(p), b = __ldg(p + 1);
        f[0] = f2(a.x, a.y);
        f[1] = f2(a.z, a.w);
        f[2] = f2(b.x, b.y);
        f[3] = f2(b.z, b.w);
    } else {
        unpack8<BF16>(__ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(w) + e)), f);
    }
}

// A lane's part of a row: the 8-value chunks that begin at elements A and B, chosen so that both halves of
// every pair lie in one lane: of the turned part, chunk i and chunk i + rot/16; of the rest, neighbours.
template <int D, bool INTER>
struct Turn {
    static constexpr int LPR = D / 16;  // lanes per row
    int A, B;
    bool turned;
    // Half pairs: cosine and sine of A's elements (and B's) in pairs. Neighbouring pairs: cosine and sine of A's
    // four pairs, then B's.
    uint64_t c[4], s[4];
    __device__ __forceinline__ Turn(int lane, int rot) {
        const int l = lane % LPR, half = rot / 16;
        turned = l < half;
        A = turned ? l * 8 : rot + (l - half) * 16;
        B = turned ? A + rot / 2 : A + 8;
    }
    __device__ __forceinline__ void load(const float *row, int rot) {
        if (!turned) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                c[i] = f2(1.f, 1.f);
                s[i] = f2(0.f, 0.f);
            }
            return;
        }
        const float4 *pc = reinterpret_cast<const float4 *>(row + (INTER ? A / 2 : A));
        const float4 *qc = INTER ? reinterpret_cast<const float4 *>(row + B / 2) : pc + 1;
        const float4 a = __ldg(pc), b = __ldg(qc), u = __ldg(pc + rot / 8), v = __ldg(qc + rot / 8);
        c[0] = f2(a.x, a.y);
        c[1] = f2(a.z, a.w);
        c[2] = f2(b.x, b.y);
        c[3] = f2(b.z, b.w);
        s[0] = f2(u.x, u.y);
        s[1] = f2(u.z, u.w);
        s[2] = f2(v.x, v.y);
        s[3] = f2(v.z, v.w);
    }
    // (xa, xb) turned by the angles, in place
    __device__ __forceinline__ void apply(uint64_t *xa, uint64_t *xb) const {
        if (INTER) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // pair i of each chunk: (a c - b s, b c + a s)
                float c0, c1, s0, s1, p, q;
                f2_split(c[i >> 1], c0, c1);
                f2_split(s[i >> 1], s0, s1);
                const float ca = (i & 1) ? c1 : c0, sa = (i & 1) ? s1 : s0;
                f2_split(c[2 + (i >> 1)], c0, c1);
                f2_split(s[2 + (i >> 1)], s0, s1);
                const float cb = (i & 1) ? c1 : c0, sb = (i & 1) ? s1 : s0;
                f2_split(xa[i], p, q);
                xa[i] = f2(fmaf(p, ca, -(q * sa)), fmaf(q, ca, p * sa));
                f2_split(xb[i], p, q);
                xb[i] = f2(fmaf(p, cb, -(q * sb)), fmaf(q, cb, p * sb));
            }
        } else {
            const uint64_t minus = f2(-1.f, -1.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint64_t sn = fmul2(s[i], minus), a = xa[i];
                xa[i] = ffma2(a, c[i], fmul2(xb[i], sn));
                xb[i] = ffma2(xb[i], c[i], fmul2(a, s[i]));
            }
        }
    }
};

// The backward holds more per value (weights, their gradients, angles), so there a lane takes one chunk of a
// row, elements [e, e + 8), and the other halves of half pairs come from the lane `src`.
template <int D, bool INTER>
struct TurnBack {
    static constexpr int LPR = D / 8;
    int e, src;
    bool turned, upper;
    uint64_t c[4], s[4];  // g_i = c_i dy_i + s_i dy_p, p the other half of the pair
    __device__ __forceinline__ TurnBack(int lane, int rot) {
        const int l = lane % LPR, half = rot / 16;
        e = l * 8;
        turned = e < rot;
        upper = !INTER && turned && l >= half;
        src = (INTER || !turned) ? lane : (upper ? lane - half : lane + half);
    }
    __device__ __forceinline__ void load(const float *row, int rot) {
        if (!turned) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                c[i] = f2(1.f, 1.f);
                s[i] = f2(0.f, 0.f);
            }
        } else if (INTER) {
            const float4 a = __ldg(reinterpret_cast<const float4 *>(row + e / 2));
            const float4 b = __ldg(reinterpret_cast<const float4 *>(row + rot / 2 + e / 2));
            c[0] = f2(a.x, a.x);
            c[1] = f2(a.y, a.y);
            c[2] = f2(a.z, a.z);
            c[3] = f2(a.w, a.w);
            s[0] = f2(b.x, -b.x);
            s[1] = f2(b.y, -b.y);
            s[2] = f2(b.z, -b.z);
            s[3] = f2(b.w, -b.w);
        } else {
            const float4 *pc = reinterpret_cast<const float4 *>(row + (upper ? e - rot / 2 : e));
            const float4 a = __ldg(pc), b = __ldg(pc + 1), u = __ldg(pc + rot / 8), v = __ldg(pc + rot / 8 + 1);
            const uint64_t sg = upper ? f2(-1.f, -1.f) : f2(1.f, 1.f);
            c[0] = f2(a.x, a.y);
            c[1] = f2(a.z, a.w);
            c[2] = f2(b.x, b.y);
            c[3] = f2(b.z, b.w);
            s[0] = fmul2(f2(u.x, u.y), sg);
            s[1] = fmul2(f2(u.z, u.w), sg);
            s[2] = fmul2(f2(v.x, v.y), sg);
            s[3] = fmul2(f2(v.z, v.w), sg);
        }
    }
};

// Sums of two values over a row's lanes: the first exchange leaves each lane with one of the two, so the
// pair costs log2(LPR) + 1 shuffles.
template <int LPR>
__device__ __forceinline__ void row_sum2(float &a, float &b) {
    const bool odd = threadIdx.x & 1;
    float v = odd ? b : a;
    v += __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
#pragma unroll
    for (int o = LPR / 2; o >= 2; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const float w = __shfl_xor_sync(0xffffffffu, v, 1);
    a = odd ? w : v;
    b = odd ? v : w;
}

// Sum over a row's lanes of both halves of two pair accumulators.
template <int LPR>
__device__ __forceinline__ float row_sum(uint64_t a, uint64_t b) {
    float lo, hi;
    f2_split(fadd2(a, b), lo, hi);
    float v = lo + hi;
#pragma unroll
    for (int o = LPR / 2; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A token's row of the angle table; a position outside it sets `bad` (reported at the kernel's end: a
// call here would hold back the loads around it) and row 0 is read instead (that output is wrong, but
// nothing outside the table is read).
__device__ __forceinline__ const float *angle_row(const QkNormParams &p, int64_t pos, bool &bad) {
    if (pos < 0 || pos >= p.max_pos) {
        bad = true;
        pos = 0;
    }
    return p.cos_sin + pos * p.rot;
}

// The kinds of rows (q, k, paged: v) have CTAs of their own: CTA blockIdx.x is number `cta` of `ctas` of
// its kind.
struct Share {
    int kind, cta, ctas;
    __device__ __forceinline__ explicit Share(const QkNormParams &p) {
        const int x = blockIdx.x;
        kind = x < p.ctas_q ? 0 : (x < p.ctas_q + p.ctas_k ? 1 : 2);
        cta = x - (kind == 0 ? 0 : (kind == 1 ? p.ctas_q : p.ctas_q + p.ctas_k));
        ctas = kind == 0 ? p.ctas_q : (kind == 1 ? p.ctas_k : static_cast<int>(gridDim.x) - p.ctas_q - p.ctas_k);
    }
};

// A warp's walk over the rows of its kind: batches of `batch` heads of a token, an equal run of neighbouring ones
// for each warp (so that the tokens need not divide by the warps, and a run's batches share their token's
// angles).
struct Walk {
    int64_t tok, left, last;
    int heads, batch, hb;
    __device__ __forceinline__ Walk(const QkNormParams &p, const Share &sh, int batch_) : last(p.n - 1), batch(batch_) {
        heads = sh.kind == 0 ? p.Hq : p.Hk;
        const int per = (heads + batch - 1) / batch;
        const int64_t total = p.n * per, warps = static_cast<int64_t>(sh.ctas) * kWarps;
        const int64_t w = static_cast<int64_t>(sh.cta) * kWarps + (threadIdx.x >> 5);
        const int64_t whole = total / warps, rest = total - whole * warps, first = whole * w + (w < rest ? w : rest);
        left = whole + (w < rest ? 1 : 0);
        tok = first / per;
        hb = static_cast<int>(first - tok * per) * batch;
    }
    __device__ __forceinline__ bool more() const { return left > 0; }
    // to the next batch; true where it begins a token
    __device__ __forceinline__ bool next() {
        --left;
        hb += batch;
        if (hb < heads) return false;
        hb = 0;
        ++tok;
        return true;
    }
    // the token after this one (this one where there is none)
    __device__ __forceinline__ int64_t next_token() const { return tok < last ? tok + 1 : last; }
};

// Measured at 8192 tokens of 64 heads of 128 (forward / backward, us): two rows a lane, two CTAs an SM and
// three slots 51 / 72 to 76, as the inputs lie in memory (as fast as a plain copy of the forward's bytes, 51); four slots 53 / 71; two slots 53 / 91; four rows in the
// backward 71.6. Three CTAs, whose registers spill, 54.5 / 105; the next rows in registers instead of a ring 60.5 / 86.
// Runs of neighbouring batches for each warp, against whole tokens by turns (timed in turn): 32 heads beside 8 of 128 39 / 55
// against 42 / 59, beside 2 of 64 23 / 35 against 86 / 92 (there the CTAs were shared out by heads, and a token of few heads
// costs a warp as much as one of many); 32 beside 32, where the tokens divide by the warps, 51 / 72 against 50 / 76. Appending
// 4 x 2048 tokens of 32 + 2 x 8 heads of 128: 49 us for 201 MB, 4.1 TB/s; 64 single tokens 6, the host time of the call.
constexpr int kRows = 2;   // rows a lane takes at a time
constexpr int kPerSm = 2;  // CTAs an SM
constexpr int kSlots = 3;  // batches in the ring, one of them being worked on

// Rows on their way: each thread copies its own chunks into its own places of a ring of kSlots batches in
// shared memory (cp.async) and reads them back itself, so nothing has to be synchronised, and what is in
// flight does not take registers. V: 16-byte chunks a thread takes of a batch.
template <int V>
struct Ring {
    static constexpr int BYTES = kSlots * V * kThreads * 16;
    uint32_t base;
    int in, out;
    __device__ __forceinline__ explicit Ring(const uint8_t *smem) : base(smem_u32(smem) + threadIdx.x * 16), in(0), out(0) {}
    __device__ __forceinline__ void put(int v, const uint16_t *src, bool there) const {
        cp_async_16_zfill(base + (in * V + v) * kThreads * 16, src, there ? 16u : 0u);
    }
    __device__ __forceinline__ void filled() {  // (also where nothing was put: batches are counted)
        asm volatile("cp.async.commit_group;" ::: "memory");
        in = in + 1 == kSlots ? 0 : in + 1;
    }
    __device__ __forceinline__ void wait() const { asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 2) : "memory"); }
    __device__ __forceinline__ uint4 get(int v) const { return ld_shared_v4(base + (out * V + v) * kThreads * 16); }
    __device__ __forceinline__ void next() { out = out + 1 == kSlots ? 0 : out + 1; }
};

// PAGED: k and v rows go to the token's slot in the pages.
template <int D, bool BF16, bool INTER, bool PAGED>
__global__ void __launch_bounds__(kThreads, kPerSm) qk_norm_fwd_kernel(const QkNormParams p) {
    constexpr int LPR = D / 16, RPI = 32 / LPR, U = kRows, BATCH = RPI * U;  // lanes a row, rows of a load
    extern __shared__ __align__(16) uint8_t smem[];
    const int lane = threadIdx.x & 31, row_in = lane / LPR;
    const Share sh(p);
    const int kind = sh.kind;
    const uint16_t *x0 = static_cast<const uint16_t *>(kind == 0 ? p.q : (kind == 1 ? p.k : p.v));
    const int64_t xs = kind == 0 ? p.q_stride : (kind == 1 ? p.k_stride : p.v_stride);
    bool bad = false, lost = false;
    Walk w(p, sh, BATCH);
    if (!w.more()) return;
    // where token w.tok's row of heads goes (PAGED: null where it has no place), and its position
    auto place = [&](int64_t &pos) -> uint16_t * {
        if constexpr (!PAGED) {
            return static_cast<uint16_t *>(kind == 0 ? p.q_out : p.k_out) + w.tok * (kind == 0 ? p.q_out_stride : p.k_out_stride);
        } else {
            // rows of no sequence stay as they are, and what their positions hold does not matter (a batch of a fixed
            // size leaves old or negative ones there)
            const bool in = w.tok >= p.cu_seqlens[0] && w.tok < p.cu_seqlens[p.num_seqs];
            const int b = in ? warp_seq_of_token(p.cu_seqlens, p.num_seqs, static_cast<int>(w.tok), lane) : -1;
            if (b < 0 || b >= p.num_seqs) {  // (or offsets that do not rise)
                pos = 0;
                return nullptr;
            }
            const int64_t slot = static_cast<int64_t>(p.kv_lens[b]) - p.cu_seqlens[b + 1] + w.tok;
            if (!p.positions) pos = slot;
            if (kind == 0) return static_cast<uint16_t *>(p.q_out) + w.tok * p.q_out_stride;
            int pg = -1;
            if (slot >= 0 && slot < (static_cast<int64_t>(p.max_blocks) << p.page_shift))
                pg = p.block_table[static_cast<int64_t>(b) * p.max_blocks + (slot >> p.page_shift)];
            if (pg < 0 || pg >= p.num_pages) {  // no place for this token: reported, nothing written
                lost = true;
                return nullptr;
            }
            const int64_t row = (static_cast<int64_t>(pg) << p.page_shift) + (slot & ((1 << p.page_shift) - 1));
            return static_cast<uint16_t *>(kind == 1 ? p.k_out : p.v_out) + row * p.Hk * D;
        }
    };
    Turn<D, INTER> turn(lane, p.rot);
    Ring<2 * U> ring(smem);
    Walk wl = w;  // of the loads
    auto fetch = [&]() {
        if (wl.more()) {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int h = wl.hb + i * RPI + row_in;
                const bool there = h < wl.heads;
                const uint16_t *x = x0 + wl.tok * xs + (there ? h * D : 0);
                ring.put(2 * i, x + turn.A, there);
                ring.put(2 * i + 1, x + turn.B, there);
            }
            wl.next();
        }
        ring.filled();
    };
#pragma unroll
    for (int k = 0; k < kSlots - 1; ++k) fetch();
    uint64_t wa[4], wb[4];
    if (kind < 2) {
        load_weights<BF16>(kind == 0 ? p.wq : p.wk, p.w32, turn.A, wa);
        load_weights<BF16>(kind == 0 ? p.wq : p.wk, p.w32, turn.B, wb);
    }
    int64_t pos = p.positions && kind < 2 ? p.positions[w.tok] : 0;
    uint16_t *dst = place(pos);
    if (kind < 2) turn.load(angle_row(p, pos, bad), p.rot);
    int64_t pos_next = p.positions && kind < 2 ? p.positions[w.next_token()] : 0;
    while (true) {
        ring.wait();
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int h = w.hb + i * RPI + row_in;
            uint16_t *out = dst + h * D;
            const bool store = dst && h < w.heads;
            const uint4 va = ring.get(2 * i), vb = ring.get(2 * i + 1);
            if (PAGED && kind == 2) {  // values: a copy
                if (store) {
                    *reinterpret_cast<uint4 *>(out + turn.A) = va;
                    *reinterpret_cast<uint4 *>(out + turn.B) = vb;
                }
                continue;
            }
            uint64_t xa[4], xb[4], ssa = f2(0.f, 0.f), ssb = ssa;
            unpack8<BF16>(va, xa);
            unpack8<BF16>(vb, xb);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                ssa = ffma2(xa[k], xa[k], ssa);
                ssb = ffma2(xb[k], xb[k], ssb);
                xa[k] = fmul2(xa[k], wa[k]);
                xb[k] = fmul2(xb[k], wb[k]);
            }
            const float r = rsqrtf(row_sum<LPR>(ssa, ssb) * (1.0f / D) + p.eps);
            const uint64_t r2 = f2(r, r);
            turn.apply(xa, xb);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                xa[k] = fmul2(xa[k], r2);
                xb[k] = fmul2(xb[k], r2);
            }
            if (store) {
                *reinterpret_cast<uint4 *>(out + turn.A) = pack8<BF16>(xa);
                *reinterpret_cast<uint4 *>(out + turn.B) = pack8<BF16>(xb);
            }
        }
        ring.next();
        fetch();  // into the slot of the batch before
        const bool turned_to = w.next();
        if (!w.more()) break;
        if (turned_to) {
            pos = pos_next;
            dst = place(pos);
            if (kind < 2) {
                turn.load(angle_row(p, pos, bad), p.rot);
                if (p.positions) pos_next = p.positions[w.next_token()];
            }
        }
    }
    cp_async_wait_all();
    if (bad && lane == 0) record_error(FA_ERR_INDEX, 700);
    if (lost && lane == 0) record_error(FA_ERR_INDEX, 701);
}

// Backward: the same walk over x and dy, adding g x r of each row to eight weight-gradient sums a lane.
template <int D, bool BF16, bool INTER>
__global__ void __launch_bounds__(kThreads, kPerSm) qk_norm_bwd_kernel(const QkNormParams p) {
    constexpr int LPR = D / 8, RPI = 32 / LPR, U = kRows, BATCH = RPI * U;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float part[kWarps][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row_in = lane / LPR;
    const Share sh(p);
    const int kind = sh.kind;
    TurnBack<D, INTER> turn(lane, p.rot);
    const uint16_t *x0 = static_cast<const uint16_t *>(kind == 0 ? p.q : p.k) + turn.e;
    const uint16_t *dy0 = static_cast<const uint16_t *>(kind == 0 ? p.dq_out : p.dk_out) + turn.e;
    uint16_t *dx0 = static_cast<uint16_t *>(kind == 0 ? p.q_out : p.k_out) + turn.e;
    const int64_t xs = kind == 0 ? p.q_stride : p.k_stride, dys = kind == 0 ? p.dq_out_stride : p.dk_out_stride;
    const int64_t dxs = kind == 0 ? p.q_out_stride : p.k_out_stride;
    bool bad = false;
    Walk w(p, sh, BATCH), wl = w;  // wl: of the loads
    Ring<2 * U> ring(smem);
    auto fetch = [&]() {
        if (wl.more()) {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int h = wl.hb + i * RPI + row_in;
                const bool there = h < wl.heads;
                const int at = there ? h * D : 0;
                ring.put(2 * i, x0 + wl.tok * xs + at, there);
                ring.put(2 * i + 1, dy0 + wl.tok * dys + at, there);
            }
            wl.next();
        }
        ring.filled();
    };
#pragma unroll
    for (int k = 0; k < kSlots - 1; ++k) fetch();
    uint64_t wt[4], dw[4];
    load_weights<BF16>(kind == 0 ? p.wq : p.wk, p.w32, turn.e, wt);
#pragma unroll
    for (int k = 0; k < 4; ++k) dw[k] = f2(0.f, 0.f);
    int64_t pos_next = 0;
    if (w.more()) {
        turn.load(angle_row(p, p.positions[w.tok], bad), p.rot);
        pos_next = p.positions[w.next_token()];
    }
    while (w.more()) {
        ring.wait();
        uint16_t *const dst = dx0 + w.tok * dxs;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int h = w.hb + i * RPI + row_in;
            const bool there = h < w.heads;
            const uint4 vx = ring.get(2 * i), vy = ring.get(2 * i + 1);
            uint64_t x[4], g[4], o[4];
            unpack8<BF16>(vx, x);
            unpack8<BF16>(vy, g);
            if (INTER) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float lo, hi;
                    f2_split(g[k], lo, hi);
                    o[k] = f2(hi, lo);
                }
            } else {
                uint4 other;
                other.x = __shfl_sync(0xffffffffu, vy.x, turn.src);
                other.y = __shfl_sync(0xffffffffu, vy.y, turn.src);
                other.z = __shfl_sync(0xffffffffu, vy.z, turn.src);
                other.w = __shfl_sync(0xffffffffu, vy.w, turn.src);
                unpack8<BF16>(other, o);
            }
            uint64_t ss2 = f2(0.f, 0.f), t2 = ss2;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                g[k] = ffma2(g[k], turn.c[k], fmul2(o[k], turn.s[k]));  // g = R^T dy
                o[k] = fmul2(g[k], wt[k]);                              // u
                ss2 = ffma2(x[k], x[k], ss2);
                t2 = ffma2(o[k], x[k], t2);
            }
            float ss, t, hi;
            f2_split(ss2, ss, hi);
            ss += hi;
            f2_split(t2, t, hi);
            t += hi;
            row_sum2<LPR>(ss, t);
            const float r = rsqrtf(ss * (1.0f / D) + p.eps);
            const float q = -r * r * t * (1.0f / D);
            const uint64_t r2 = f2(r, r), q2 = f2(q, q), rw = there ? r2 : f2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                dw[k] = ffma2(g[k], fmul2(x[k], rw), dw[k]);
                o[k] = fmul2(ffma2(x[k], q2, o[k]), r2);  // r (u - x r^2 t / D)
            }
            if (there) *reinterpret_cast<uint4 *>(dst + h * D) = pack8<BF16>(o);
        }
        ring.next();
        fetch();  // into the slot of the batch before
        if (w.next() && w.more()) {
            turn.load(angle_row(p, pos_next, bad), p.rot);
            pos_next = p.positions[w.next_token()];
        }
    }
    cp_async_wait_all();
    if (bad && lane == 0) record_error(FA_ERR_INDEX, 700);
    if (!p.partials) return;
    // the rows of a warp, then the CTA's warps, in a fixed order
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float x[2];
        f2_split(dw[k], x[0], x[1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int o = LPR; o < 32; o <<= 1) x[i] += __shfl_xor_sync(0xffffffffu, x[i], o);
            if (row_in == 0) part[warp][turn.e + 2 * k + i] = x[i];
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < D; e += kThreads) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) sum += part[i][e];
        p.partials[static_cast<int64_t>(blockIdx.x) * D + e] = sum;
    }
}

// The weights' gradients: blockIdx.y 0 sums the partials of the q CTAs, 1 those of the k CTAs; 32 columns
// a block, 32 slices of the CTAs a column.
__global__ void __launch_bounds__(1024) qk_norm_dw_kernel(const QkNormParams p, int D) {
    __shared__ float s[32][33];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
    const int c0 = blockIdx.y == 0 ? 0 : p.ctas_q, c1 = c0 + (blockIdx.y == 0 ? p.ctas_q : p.ctas_k);
    float sum = 0.f;
#pragma unroll 4
    for (int c = c0 + slice; c < c1; c += 32) sum += p.partials[static_cast<int64_t>(c) * D + col];
    s[slice][lane] = sum;
    __syncthreads();
    if (slice == 0) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) sum += s[i][lane];
        float *out = blockIdx.y == 0 ? p.dwq : p.dwk;
        if (out) out[col] = sum;
    }
}

// Launches a kernel with the ring's dynamic shared memory (the opt-in above 48 KB is a per-device function
// attribute, set at the kernel's first launch on a device; setting it twice is harmless).
template <auto Kernel>
cudaError_t launch_ring(int bytes, int grid, const QkNormParams &p, cudaStream_t st) {
    static uint64_t attr_set_mask = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (!(__atomic_load_n(&attr_set_mask, __ATOMIC_ACQUIRE) & bit)) {
        e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        __atomic_fetch_or(&attr_set_mask, bit, __ATOMIC_RELEASE);
    }
    Kernel<<<grid, kThreads, bytes, st>>>(p);
    return cudaGetLastError();
}

template <int D, bool BF16, bool INTER>
cudaError_t launch_d(bool backward, QkNormParams p, cudaStream_t st) {
    const int batch = 32 / (backward ? D / 8 : D / 16) * kRows;  // heads a warp works on at a time
    const bool paged = p.cu_seqlens != nullptr;
    // kPerSm CTAs an SM, shared out by the kinds' rows as they are worked on (whole batches), no more than there are
    // batches for.
    const int64_t most = kQkNormCtas;
    auto batches = [&](int heads) { return static_cast<int64_t>((heads + batch - 1) / batch); };
    const int64_t all = batches(p.Hq) + batches(p.Hk) * (paged ? 2 : 1);
    auto share = [&](int heads) {
        const int64_t need = (p.n * batches(heads) + kWarps - 1) / kWarps, mine = most * batches(heads) / all;
        return static_cast<int>(std::min(need, std::max<int64_t>(mine, 1)));
    };
    p.ctas_q = share(p.Hq);
    p.ctas_k = share(p.Hk);
    const int grid = p.ctas_q + p.ctas_k + (paged ? p.ctas_k : 0);
    if (backward) {
        cudaError_t e = launch_ring<qk_norm_bwd_kernel<D, BF16, INTER>>(Ring<2 * kRows>::BYTES, grid, p, st);
        if (e != cudaSuccess || !p.partials) return e;
        cudaLaunchConfig_t cfg = {};  // waits on the device for the kernel above
        cfg.gridDim = dim3(D / 32, 2, 1);
        cfg.blockDim = dim3(1024, 1, 1);
        cfg.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, qk_norm_dw_kernel, p, D);
        return e != cudaSuccess ? e : cudaGetLastError();
    }
    constexpr int bytes = Ring<2 * kRows>::BYTES;
    return paged ? launch_ring<qk_norm_fwd_kernel<D, BF16, INTER, true>>(bytes, grid, p, st)
                 : launch_ring<qk_norm_fwd_kernel<D, BF16, INTER, false>>(bytes, grid, p, st);
}

template <int D>
cudaError_t launch_t(bool backward, bool bf16, bool inter, const QkNormParams &p, cudaStream_t st) {
    if (bf16) return inter ? launch_d<D, true, true>(backward, p, st) : launch_d<D, true, false>(backward, p, st);
    return inter ? launch_d<D, false, true>(backward, p, st) : launch_d<D, false, false>(backward, p, st);
}

}  // namespace

cudaError_t launch_qk_norm(int D, bool bf16, bool interleaved, bool backward, const QkNormParams &p, cudaStream_t st) {
    switch (D) {
        case 32: return launch_t<32>(backward, bf16, interleaved, p, st);
        case 64: return launch_t<64>(backward, bf16, interleaved, p, st);
        case 128: return launch_t<128>(backward, bf16, interleaved, p, st);
        case 256: return launch_t<256>(backward, bf16, interleaved, p, st);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t qk_norm_error_addrs(int **code, int **where) { return device_error_addrs(code, where); }

}  // namespace fa
