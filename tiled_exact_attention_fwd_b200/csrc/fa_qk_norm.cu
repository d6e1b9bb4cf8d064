// fa_qk_norm.cu -- RMS norm of queries and keys for each head and the position rotation, in one
// pass over the data (fa_qk_norm_rope), the same with k and v written into the pages of a cache
// (fa_qk_norm_rope_paged), and the gradients (fa_qk_norm_rope_bwd).
//
// Mathematics, for one head row x of D values, weights w, and the token's angles (c, s):
//   r = 1 / sqrt(mean(x^2) + eps),  n = w * x * r,  y = R n,
//   R turns the pairs (a, b) of the first `rot` values: (a c - b s, b c + a s); a pair is (i,
//   i + rot/2), or (2i, 2i + 1) when interleaved. With a_i = w_i c_i and b_i = -+ w_p s_i (p the
//   other half of the pair) the row is y_i = r (x_i a_i + x_p b_i): the weights and angles are
//   multiplied together once per token and stay in registers for its heads.
// Backward: g = R^T dy (the angles turned back), u = w g, t = sum(u x),
//   dx = r u - x r^3 t / D,  dw = sum over tokens and heads of g x r.
//
// Everything is bytes: each row is read once and written once (backward: x and dy read, dx
// written), a 16-byte vector per lane, a row on D / 8 neighbouring lanes, so a row's sums are
// log2(D / 8) shuffles. Two CTAs an SM walk over the tokens, each warp with the next rows in flight
// while it works on the current ones. All arithmetic is 32-bit; an output is
// rounded once. The weight gradients are summed in registers, then over the CTA's warps in
// shared memory, then over the CTAs by a second launch in a fixed order (no atomics: the same
// inputs give the same bits).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "fa.h"
#include "fa_internal.h"
#include "fa_ptx.cuh"
#include "fa_seq.cuh"
#include "fa_sync.cuh"

namespace fa {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4 &v, float *f) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (BF16) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        } else {
            const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
            f[2 * i] = t.x;
            f[2 * i + 1] = t.y;
        }
    }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float *f) {
    uint4 v;
    uint32_t *u = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = BF16 ? pack2_bf16(f[2 * i], f[2 * i + 1]) : pack2_f16(f[2 * i], f[2 * i + 1]);
    return v;
}

__device__ __forceinline__ uint4 shfl4(const uint4 &v, int src) {
    uint4 o;
    o.x = __shfl_sync(0xffffffffu, v.x, src);
    o.y = __shfl_sync(0xffffffffu, v.y, src);
    o.z = __shfl_sync(0xffffffffu, v.z, src);
    o.w = __shfl_sync(0xffffffffu, v.w, src);
    return o;
}

// Eight weights from element e on (ones where there are none).
template <bool BF16>
__device__ __forceinline__ void load_weights(const void *w, int w32, int e, float *f) {
    if (!w) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = 1.f;
    } else if (w32) {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(w) + e);
        const float4 a = __ldg(p), b = __ldg(p + 1);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
        unpack8<BF16>(__ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(w) + e)), f);
    }
}

// How this lane's eight values (elements [e, e + 8) of a row) are turned.
template <int D, bool INTER>
struct Turn {
    static constexpr int LPR = D / 8;  // lanes per row
    int src;                           // lane that holds the other halves of the pairs (itself when in-lane or not turned)
    int pe;                            // first element of that lane
    bool turned, upper;                // any element turned; elements are second halves (INTER: neither)
    __device__ __forceinline__ Turn(int lane, int rot) {
        const int sub = lane % LPR, e = sub * 8, hl = rot / 16;  // half of the turned part in lanes
        turned = e < rot;
        upper = !INTER && turned && e >= rot / 2;
        src = (INTER || !turned) ? lane : (upper ? lane - hl : lane + hl);
        pe = (INTER || !turned) ? e : (upper ? e - rot / 2 : e + rot / 2);
    }
    // cos and signed sin of each element: y_i = c_i x_i + s_i x_p (sign -1: turned back)
    __device__ __forceinline__ void angles(const float *row, int rot, int lane, float sign, float *c, float *s) const {
        const int e = (lane % LPR) * 8;
        if (!turned) {
#pragma unroll
            for (int i = 0; i < 8; ++i) { c[i] = 1.f; s[i] = 0.f; }
            return;
        }
        if (INTER) {
            const float4 a = __ldg(reinterpret_cast<const float4 *>(row + e / 2));
            const float4 b = __ldg(reinterpret_cast<const float4 *>(row + rot / 2 + e / 2));
            const float ca[4] = {a.x, a.y, a.z, a.w}, sa[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                c[2 * i] = c[2 * i + 1] = ca[i];
                s[2 * i] = -sign * sa[i];
                s[2 * i + 1] = sign * sa[i];
            }
        } else {
            const int k = upper ? e - rot / 2 : e;
            const float4 *pc = reinterpret_cast<const float4 *>(row + k);
            const float4 *ps = reinterpret_cast<const float4 *>(row + rot / 2 + k);
            const float4 a = __ldg(pc), b = __ldg(pc + 1), u = __ldg(ps), v = __ldg(ps + 1);
            const float sg = upper ? sign : -sign;
            c[0] = a.x; c[1] = a.y; c[2] = a.z; c[3] = a.w; c[4] = b.x; c[5] = b.y; c[6] = b.z; c[7] = b.w;
            s[0] = sg * u.x; s[1] = sg * u.y; s[2] = sg * u.z; s[3] = sg * u.w;
            s[4] = sg * v.x; s[5] = sg * v.y; s[6] = sg * v.z; s[7] = sg * v.w;
        }
    }
};

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
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

// Rows are read once: not kept in L1. (Not the read-only path: the output may be the input.)
__device__ __forceinline__ uint4 ld_row(const uint16_t *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
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

// A warp's walk over the work units of its kind: a unit is one token and up to p.heads_per_warp
// consecutive heads, worked on in batches of BATCH heads. The next batch is asked for before the current
// one is worked on, a unit's angles a batch before it begins, and its position a unit before that, so
// that the loads that depend on one another are never waited for in a row.
struct Walk {
    int64_t unit, units, step, tok, ahead;  // ahead: position of the unit after the current one
    int per_token, heads, hb, h1;
    __device__ __forceinline__ Walk(const QkNormParams &p, const Share &sh) {
        per_token = sh.kind == 0 ? p.q_units : p.k_units;
        heads = sh.kind == 0 ? p.Hq : p.Hk;
        units = p.n * per_token;
        step = static_cast<int64_t>(sh.ctas) * kWarps;
        unit = static_cast<int64_t>(sh.cta) * kWarps + (threadIdx.x >> 5);
        ahead = p.positions && unit < units ? p.positions[unit / per_token] : 0;
    }
    // takes unit `unit`; its position
    __device__ __forceinline__ int64_t enter(const QkNormParams &p) {
        tok = unit / per_token;
        hb = static_cast<int>(unit - tok * per_token) * p.heads_per_warp;
        h1 = min(heads, hb + p.heads_per_warp);
        const int64_t pos = ahead;
        if (p.positions && unit + step < units) ahead = p.positions[(unit + step) / per_token];
        return pos;
    }
};

constexpr int kFwdRows = 4, kBwdRows = 2;  // rows a lane takes at a time

// PAGED: k and v rows go to the token's slot in the pages.
template <int D, bool BF16, bool INTER, bool PAGED>
__global__ void __launch_bounds__(kThreads, 2) qk_norm_fwd_kernel(const QkNormParams p) {
    constexpr int LPR = D / 8, RPI = 32 / LPR, U = kFwdRows, BATCH = RPI * U;  // lanes a row, rows of a load
    const int lane = threadIdx.x & 31, sub = lane % LPR, row_in = lane / LPR;
    const Share sh(p);
    const int kind = sh.kind;
    const uint16_t *x0 = static_cast<const uint16_t *>(kind == 0 ? p.q : (kind == 1 ? p.k : p.v)) + sub * 8;
    const int64_t xs = kind == 0 ? p.q_stride : (kind == 1 ? p.k_stride : p.v_stride);
    bool bad = false, lost = false;
    Walk w(p, sh);
    // where token w.tok's row of heads goes (PAGED: null where it has no place), and its position
    auto place = [&](int64_t &pos) -> uint16_t * {
        if constexpr (!PAGED) {
            return static_cast<uint16_t *>(kind == 0 ? p.q_out : p.k_out) +
                   w.tok * (kind == 0 ? p.q_out_stride : p.k_out_stride) + sub * 8;
        } else {
            // rows of no sequence stay as they are
            if (w.tok < p.cu_seqlens[0] || w.tok >= p.cu_seqlens[p.num_seqs]) return nullptr;
            const int b = warp_seq_of_token(p.cu_seqlens, p.num_seqs, static_cast<int>(w.tok), lane);
            if (b < 0 || b >= p.num_seqs) return nullptr;  // offsets that do not rise
            const int64_t slot = static_cast<int64_t>(p.kv_lens[b]) - p.cu_seqlens[b + 1] + w.tok;
            if (!p.positions) pos = slot;
            if (kind == 0) return static_cast<uint16_t *>(p.q_out) + w.tok * p.q_out_stride + sub * 8;
            int pg = -1;
            if (slot >= 0 && slot < (static_cast<int64_t>(p.max_blocks) << p.page_shift))
                pg = p.block_table[static_cast<int64_t>(b) * p.max_blocks + (slot >> p.page_shift)];
            if (pg < 0 || pg >= p.num_pages) {  // no place for this token: reported, nothing written
                lost = true;
                return nullptr;
            }
            const int64_t row = (static_cast<int64_t>(pg) << p.page_shift) + (slot & ((1 << p.page_shift) - 1));
            return static_cast<uint16_t *>(kind == 1 ? p.k_out : p.v_out) + row * p.Hk * D + sub * 8;
        }
    };
    auto load = [&](uint4 *v) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int h = w.hb + i * RPI + row_in;
            v[i] = h < w.h1 ? ld_row(x0 + w.tok * xs + h * D) : make_uint4(0, 0, 0, 0);
        }
    };
    const Turn<D, INTER> turn(lane, p.rot);
    const void *wt = kind == 0 ? p.wq : p.wk;
    float wi[8], wp[8];
    if (kind < 2) {
        load_weights<BF16>(wt, p.w32, sub * 8, wi);
        load_weights<BF16>(wt, p.w32, turn.pe, wp);
    }
    uint4 v[U];
    float c[8], s[8], a[8], b[8];  // angles of the unit to come; y_i = r (x_i a_i + x_p b_i)
    bool more = w.unit < w.units, fresh = true;
    uint16_t *y = nullptr;
    if (more) {
        int64_t pos = w.enter(p);
        load(v);
        y = place(pos);
        if (kind < 2) turn.angles(angle_row(p, pos, bad), p.rot, lane, 1.f, c, s);
    }
#pragma unroll 1
    while (more) {
        if (fresh && kind < 2) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                a[i] = wi[i] * c[i];
                b[i] = wp[INTER ? (i ^ 1) : i] * s[i];
            }
        }
        const int hb = w.hb, h1 = w.h1;
        uint16_t *const dst = y;
        uint4 nv[U];
        w.hb += BATCH;
        fresh = w.hb >= w.h1;
        if (fresh) {
            w.unit += w.step;
            more = w.unit < w.units;
            if (more) {
                int64_t pos = w.enter(p);
                load(nv);
                y = place(pos);
                if (kind < 2) turn.angles(angle_row(p, pos, bad), p.rot, lane, 1.f, c, s);
            }
        } else {
            load(nv);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int h = hb + i * RPI + row_in;
            if (PAGED && kind == 2) {  // values: a copy
                if (dst && h < h1) *reinterpret_cast<uint4 *>(dst + h * D) = v[i];
                continue;
            }
            float xi[8], xp[8], out[8];
            unpack8<BF16>(v[i], xi);
            if (INTER) {
#pragma unroll
                for (int k = 0; k < 8; ++k) xp[k] = xi[k ^ 1];
            } else {
                unpack8<BF16>(shfl4(v[i], turn.src), xp);
            }
            float ss = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) ss = fmaf(xi[k], xi[k], ss);
            const float r = rsqrtf(row_sum<LPR>(ss) * (1.0f / D) + p.eps);
#pragma unroll
            for (int k = 0; k < 8; ++k) out[k] = r * fmaf(xi[k], a[k], xp[k] * b[k]);
            if (dst && h < h1) *reinterpret_cast<uint4 *>(dst + h * D) = pack8<BF16>(out);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) v[i] = nv[i];
    }
    if (bad && lane == 0) record_error(FA_ERR_INDEX, 700);
    if (lost && lane == 0) record_error(FA_ERR_INDEX, 701);
}

// Backward: the same walk over x and dy, adding g x r of each row to eight weight-gradient sums a lane.
template <int D, bool BF16, bool INTER>
__global__ void __launch_bounds__(kThreads, 2) qk_norm_bwd_kernel(const QkNormParams p) {
    constexpr int LPR = D / 8, RPI = 32 / LPR, U = kBwdRows, BATCH = RPI * U;
    __shared__ float part[kWarps][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % LPR, row_in = lane / LPR;
    const Turn<D, INTER> turn(lane, p.rot);
    const Share sh(p);
    const int kind = sh.kind;
    const uint16_t *x0 = static_cast<const uint16_t *>(kind == 0 ? p.q : p.k) + sub * 8;
    const uint16_t *dy0 = static_cast<const uint16_t *>(kind == 0 ? p.dq_out : p.dk_out) + sub * 8;
    uint16_t *dx0 = static_cast<uint16_t *>(kind == 0 ? p.q_out : p.k_out) + sub * 8;
    const int64_t xs = kind == 0 ? p.q_stride : p.k_stride, dys = kind == 0 ? p.dq_out_stride : p.dk_out_stride;
    const int64_t dxs = kind == 0 ? p.q_out_stride : p.k_out_stride;
    bool bad = false;
    Walk w(p, sh);
    float wi[8], dw[8];
    load_weights<BF16>(kind == 0 ? p.wq : p.wk, p.w32, sub * 8, wi);
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[k] = 0.f;
    auto load = [&](uint4 *ox, uint4 *oy) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int h = w.hb + i * RPI + row_in;
            ox[i] = h < w.h1 ? ld_row(x0 + w.tok * xs + h * D) : make_uint4(0, 0, 0, 0);
            oy[i] = h < w.h1 ? ld_row(dy0 + w.tok * dys + h * D) : make_uint4(0, 0, 0, 0);
        }
    };
    uint4 vx[U], vy[U];
    float c[8], s[8], nc[8], ns[8];
    bool more = w.unit < w.units, fresh = true;
    if (more) {
        const int64_t pos = w.enter(p);
        load(vx, vy);
        turn.angles(angle_row(p, pos, bad), p.rot, lane, -1.f, nc, ns);
    }
#pragma unroll 1
    while (more) {
        if (fresh) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                c[i] = nc[i];
                s[i] = ns[i];
            }
        }
        const int hb = w.hb, h1 = w.h1;
        uint16_t *const dx = dx0 + w.tok * dxs;
        uint4 nx[U], ny[U];
        w.hb += BATCH;
        fresh = w.hb >= w.h1;
        if (fresh) {
            w.unit += w.step;
            more = w.unit < w.units;
            if (more) {
                const int64_t pos = w.enter(p);
                load(nx, ny);
                turn.angles(angle_row(p, pos, bad), p.rot, lane, -1.f, nc, ns);
            }
        } else {
            load(nx, ny);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int h = hb + i * RPI + row_in;
            float xi[8], yi[8], yp[8], u[8];
            unpack8<BF16>(vx[i], xi);
            unpack8<BF16>(vy[i], yi);
            if (INTER) {
#pragma unroll
                for (int k = 0; k < 8; ++k) yp[k] = yi[k ^ 1];
            } else {
                unpack8<BF16>(shfl4(vy[i], turn.src), yp);
            }
            float ss = 0.f, t = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                u[k] = fmaf(yi[k], c[k], yp[k] * s[k]);  // g = R^T dy
                ss = fmaf(xi[k], xi[k], ss);
                t = fmaf(u[k] * wi[k], xi[k], t);
            }
            ss = row_sum<LPR>(ss);
            t = row_sum<LPR>(t);
            const float r = rsqrtf(ss * (1.0f / D) + p.eps);
            const float q = r * r * t * (1.0f / D);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (h < h1) dw[k] = fmaf(u[k], xi[k] * r, dw[k]);
                u[k] = r * (u[k] * wi[k] - xi[k] * q);
            }
            if (h < h1) *reinterpret_cast<uint4 *>(dx + h * D) = pack8<BF16>(u);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            vx[i] = nx[i];
            vy[i] = ny[i];
        }
    }
    if (bad && lane == 0) record_error(FA_ERR_INDEX, 700);
    if (!p.partials) return;
    // the rows of a warp, then the CTA's warps, in a fixed order
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int o = LPR; o < 32; o <<= 1) dw[k] += __shfl_xor_sync(0xffffffffu, dw[k], o);
    if (row_in == 0)
#pragma unroll
        for (int k = 0; k < 8; ++k) part[warp][sub * 8 + k] = dw[k];
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

template <int D, bool BF16, bool INTER>
cudaError_t launch_d(bool backward, QkNormParams p, cudaStream_t st) {
    constexpr int RPI = 32 / (D / 8);
    const int batch = RPI * (backward ? kBwdRows : kFwdRows);  // heads a warp works on at a time
    const bool paged = p.cu_seqlens != nullptr;
    // Two CTAs an SM, shared out by the kinds' heads. A unit is one batch while that leaves CTAs idle, else
    // up to four batches of a token, which share its angles.
    const int most = kQkNormCtas;
    auto units = [&](int heads, int per) { return static_cast<int64_t>((heads + per - 1) / per); };
    const int heads = p.Hq + p.Hk * (paged ? 2 : 1);
    p.heads_per_warp = batch;
    if (p.n * (units(p.Hq, batch) + units(p.Hk, batch) * (paged ? 2 : 1)) > static_cast<int64_t>(most) * kWarps * 4)
        p.heads_per_warp = 4 * batch;
    p.q_units = static_cast<int>(units(p.Hq, p.heads_per_warp));
    p.k_units = static_cast<int>(units(p.Hk, p.heads_per_warp));
    auto share = [&](int of_heads, int per_token) {
        const int64_t need = (p.n * per_token + kWarps - 1) / kWarps;
        int64_t mine = static_cast<int64_t>(most) * of_heads / heads;
        if (mine < 1) mine = 1;
        return static_cast<int>(need < mine ? need : mine);
    };
    p.ctas_q = share(p.Hq, p.q_units);
    p.ctas_k = share(p.Hk, p.k_units);
    const int grid = p.ctas_q + p.ctas_k + (paged ? p.ctas_k : 0);
    if (backward) {
        qk_norm_bwd_kernel<D, BF16, INTER><<<grid, kThreads, 0, st>>>(p);
        cudaError_t e = cudaGetLastError();
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
    if (paged)
        qk_norm_fwd_kernel<D, BF16, INTER, true><<<grid, kThreads, 0, st>>>(p);
    else
        qk_norm_fwd_kernel<D, BF16, INTER, false><<<grid, kThreads, 0, st>>>(p);
    return cudaGetLastError();
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
