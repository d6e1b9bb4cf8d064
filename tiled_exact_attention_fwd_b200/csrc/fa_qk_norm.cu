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
// log2(D / 8) shuffles. A warp takes one token and a chunk of consecutive heads, UNROLL rows a
// lane at a time so that several loads are in flight. All arithmetic is 32-bit; an output is
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

// A token's row of the angle table; a position outside it is reported and row 0 read instead
// (that output is wrong, but nothing outside the table is read).
__device__ __forceinline__ const float *angle_row(const QkNormParams &p, int64_t pos, int lane) {
    if (pos < 0 || pos >= p.max_pos) {
        if (lane == 0) record_error(FA_ERR_INDEX, 700);
        pos = 0;
    }
    return p.cos_sin + pos * p.rot;
}

// Work unit: one token and up to p.heads_per_warp consecutive heads of q, of k, or (paged) of v.
// PAGED: k and v rows go to the token's slot in the pages.
template <int D, bool BF16, bool INTER, bool PAGED, int UNROLL>
__global__ void __launch_bounds__(kThreads) qk_norm_fwd_kernel(const QkNormParams p) {
    constexpr int LPR = D / 8, RPI = 32 / LPR;  // lanes a row, rows an iteration
    const int lane = threadIdx.x & 31, sub = lane % LPR, row_in = lane / LPR;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int64_t tok = unit / p.units_per_token;
    if (tok >= p.n) return;
    int u = static_cast<int>(unit - tok * p.units_per_token);
    const int kind = u < p.q_units ? 0 : (u < p.q_units + p.k_units ? 1 : 2);
    u -= kind == 0 ? 0 : (kind == 1 ? p.q_units : p.q_units + p.k_units);
    const int heads = kind == 0 ? p.Hq : p.Hk;
    const int h0 = u * p.heads_per_warp, h1 = min(heads, h0 + p.heads_per_warp);

    const uint16_t *x = static_cast<const uint16_t *>(kind == 0 ? p.q : (kind == 1 ? p.k : p.v)) +
                        tok * (kind == 0 ? p.q_stride : (kind == 1 ? p.k_stride : p.v_stride));
    uint16_t *y = nullptr;
    int64_t pos = 0;
    if (PAGED) {
        const int total = p.cu_seqlens[p.num_seqs];
        if (tok < p.cu_seqlens[0] || tok >= total) return;  // rows of no sequence stay as they are
        const int b = warp_seq_of_token(p.cu_seqlens, p.num_seqs, static_cast<int>(tok), lane);
        const int64_t slot = static_cast<int64_t>(p.kv_lens[b]) - p.cu_seqlens[b + 1] + tok;
        pos = p.positions ? p.positions[tok] : slot;
        if (kind == 0) {
            y = static_cast<uint16_t *>(p.q_out) + tok * p.q_out_stride;
        } else {
            int pg = -1;
            if (slot >= 0 && slot < (static_cast<int64_t>(p.max_blocks) << p.page_shift))
                pg = p.block_table[static_cast<int64_t>(b) * p.max_blocks + (slot >> p.page_shift)];
            if (pg < 0 || pg >= p.num_pages) {  // no place for this token: reported, nothing written
                if (lane == 0) record_error(FA_ERR_INDEX, 701);
                return;
            }
            const int64_t row = (static_cast<int64_t>(pg) << p.page_shift) + (slot & ((1 << p.page_shift) - 1));
            y = static_cast<uint16_t *>(kind == 1 ? p.k_out : p.v_out) + row * p.Hk * D;
        }
    } else {
        pos = p.positions[tok];
        y = static_cast<uint16_t *>(kind == 0 ? p.q_out : p.k_out) + tok * (kind == 0 ? p.q_out_stride : p.k_out_stride);
    }

    if (PAGED && kind == 2) {  // values: a copy
        for (int h = h0 + row_in; h < h1; h += RPI * UNROLL) {
            uint4 v[UNROLL];
#pragma unroll
            for (int i = 0; i < UNROLL; ++i)
                if (h + i * RPI < h1) v[i] = *reinterpret_cast<const uint4 *>(x + (h + i * RPI) * D + sub * 8);
#pragma unroll
            for (int i = 0; i < UNROLL; ++i)
                if (h + i * RPI < h1) *reinterpret_cast<uint4 *>(y + (h + i * RPI) * D + sub * 8) = v[i];
        }
        return;
    }

    const Turn<D, INTER> turn(lane, p.rot);
    float a[8], b[8];  // y_i = r (x_i a_i + x_p b_i)
    {
        const void *w = kind == 0 ? p.wq : p.wk;
        float c[8], s[8], wi[8], wp[8];
        turn.angles(angle_row(p, pos, lane), p.rot, lane, 1.f, c, s);
        load_weights<BF16>(w, p.w32, sub * 8, wi);
        load_weights<BF16>(w, p.w32, turn.pe, wp);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            a[i] = wi[i] * c[i];
            b[i] = wp[INTER ? (i ^ 1) : i] * s[i];
        }
    }
    for (int hb = h0; hb < h1; hb += RPI * UNROLL) {
        uint4 v[UNROLL];
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) {
            const int h = hb + i * RPI + row_in;
            v[i] = h < h1 ? *reinterpret_cast<const uint4 *>(x + h * D + sub * 8) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) {
            const int h = hb + i * RPI + row_in;
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
            const float r = 1.0f / sqrtf(row_sum<LPR>(ss) * (1.0f / D) + p.eps);
#pragma unroll
            for (int k = 0; k < 8; ++k) out[k] = r * fmaf(xi[k], a[k], xp[k] * b[k]);
            if (h < h1) *reinterpret_cast<uint4 *>(y + h * D + sub * 8) = pack8<BF16>(out);
        }
    }
}

// Backward: a fixed grid of p.grid CTAs, each warp walking units gridDim.x * kWarps apart, first
// those of q, then those of k, adding g x r of its rows to eight weight-gradient sums a lane.
template <int D, bool BF16, bool INTER, int UNROLL>
__global__ void __launch_bounds__(kThreads) qk_norm_bwd_kernel(const QkNormParams p) {
    constexpr int LPR = D / 8, RPI = 32 / LPR;
    __shared__ float part[kWarps][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % LPR, row_in = lane / LPR;
    const Turn<D, INTER> turn(lane, p.rot);
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
    for (int kind = 0; kind < 2; ++kind) {
        const int heads = kind == 0 ? p.Hq : p.Hk, per_token = kind == 0 ? p.q_units : p.k_units;
        const void *w = kind == 0 ? p.wq : p.wk;
        float wi[8], dw[8];
        load_weights<BF16>(w, p.w32, sub * 8, wi);
#pragma unroll
        for (int k = 0; k < 8; ++k) dw[k] = 0.f;
        for (int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + warp; unit < p.n * per_token; unit += step) {
            const int64_t tok = unit / per_token;
            const int h0 = static_cast<int>(unit - tok * per_token) * p.heads_per_warp;
            const int h1 = min(heads, h0 + p.heads_per_warp);
            const uint16_t *x = static_cast<const uint16_t *>(kind == 0 ? p.q : p.k) + tok * (kind == 0 ? p.q_stride : p.k_stride);
            const uint16_t *dy = static_cast<const uint16_t *>(kind == 0 ? p.dq_out : p.dk_out) +
                                 tok * (kind == 0 ? p.dq_out_stride : p.dk_out_stride);
            uint16_t *dx = static_cast<uint16_t *>(kind == 0 ? p.q_out : p.k_out) +
                           tok * (kind == 0 ? p.q_out_stride : p.k_out_stride);
            float c[8], s[8];
            turn.angles(angle_row(p, p.positions[tok], lane), p.rot, lane, -1.f, c, s);
            for (int hb = h0; hb < h1; hb += RPI * UNROLL) {
                uint4 vx[UNROLL], vy[UNROLL];
#pragma unroll
                for (int i = 0; i < UNROLL; ++i) {
                    const int h = hb + i * RPI + row_in;
                    vx[i] = h < h1 ? *reinterpret_cast<const uint4 *>(x + h * D + sub * 8) : make_uint4(0, 0, 0, 0);
                    vy[i] = h < h1 ? *reinterpret_cast<const uint4 *>(dy + h * D + sub * 8) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < UNROLL; ++i) {
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
                    const float r = 1.0f / sqrtf(ss * (1.0f / D) + p.eps);
                    const float q = r * r * t * (1.0f / D);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        if (h < h1) dw[k] = fmaf(u[k], xi[k] * r, dw[k]);
                        u[k] = r * (u[k] * wi[k] - xi[k] * q);
                    }
                    if (h < h1) *reinterpret_cast<uint4 *>(dx + h * D + sub * 8) = pack8<BF16>(u);
                }
            }
        }
        if (!p.partials) continue;
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
            p.partials[(static_cast<int64_t>(blockIdx.x) * 2 + kind) * D + e] = sum;
        }
        __syncthreads();
    }
}

// dw[kind][e] = sum over the CTAs' partials: 32 columns a block, 8 CTA slices a column.
__global__ void __launch_bounds__(kThreads) qk_norm_dw_kernel(const float *partials, int ctas, int D, float *dwq, float *dwk) {
    __shared__ float s[kWarps][32];
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;  // of 2 * D
    float sum = 0.f;
    for (int c = slice; c < ctas; c += kWarps) sum += partials[static_cast<int64_t>(c) * 2 * D + col];
    s[slice][lane] = sum;
    __syncthreads();
    if (slice == 0) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) sum += s[i][lane];
        float *out = col < D ? dwq : dwk;
        if (out) out[col < D ? col : col - D] = sum;
    }
}

template <int D, bool BF16, bool INTER>
cudaError_t launch_d(bool backward, QkNormParams p, cudaStream_t st) {
    constexpr int RPI = 32 / (D / 8);
    // 4 rows a lane in flight forward, 2 (of x and dy each) backward
    p.heads_per_warp = RPI * (backward ? 2 : 4);
    p.q_units = (p.Hq + p.heads_per_warp - 1) / p.heads_per_warp;
    p.k_units = (p.Hk + p.heads_per_warp - 1) / p.heads_per_warp;
    if (backward) {
        const int64_t most = (p.n * (p.q_units > p.k_units ? p.q_units : p.k_units) + kWarps - 1) / kWarps;
        const int grid = static_cast<int>(most < kQkNormBwdCtas ? most : kQkNormBwdCtas);
        qk_norm_bwd_kernel<D, BF16, INTER, 2><<<grid, kThreads, 0, st>>>(p);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess || !p.partials) return e;
        qk_norm_dw_kernel<<<2 * D / 32, kThreads, 0, st>>>(p.partials, grid, D, p.dwq, p.dwk);
        return cudaGetLastError();
    }
    const bool paged = p.cu_seqlens != nullptr;
    p.units_per_token = p.q_units + p.k_units * (paged ? 2 : 1);
    const int64_t grid = (p.n * p.units_per_token + kWarps - 1) / kWarps;
    if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
    if (paged)
        qk_norm_fwd_kernel<D, BF16, INTER, true, 4><<<static_cast<unsigned>(grid), kThreads, 0, st>>>(p);
    else
        qk_norm_fwd_kernel<D, BF16, INTER, false, 4><<<static_cast<unsigned>(grid), kThreads, 0, st>>>(p);
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
