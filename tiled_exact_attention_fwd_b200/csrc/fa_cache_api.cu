// fa_cache_api.cu -- the C ABI of the operators around a paged cache: argument validation, tensor
// maps and dispatch of the query/key norm with rotation, attention of new tokens over the pages,
// key weights and eviction. As in fa_api.cu nothing here allocates or synchronises.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <initializer_list>
#include <numeric>

#include "fa.h"
#include "fa_internal.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int log2_of(int v) {
    int s = 0;
    while ((1 << s) < v) ++s;
    return s;
}

// Page geometry: a power of two of at least 16 rows, pools below 2^31 rows.
bool pages_ok(int max_blocks, int page_size, int num_pages) {
    if (max_blocks <= 0 || num_pages <= 0) return false;
    if (page_size < 16 || page_size > (1 << 20) || (page_size & (page_size - 1)) != 0) return false;
    return static_cast<int64_t>(num_pages) * page_size <= INT32_MAX;
}

// Keys that a table row can name: positions, and those of the tile behind them, stay below 2^31.
int capacity_of(int max_blocks, int page_size) {
    const int64_t c = static_cast<int64_t>(max_blocks) * page_size;
    return c > fa::kMaxSeqKeys ? fa::kMaxSeqKeys : static_cast<int>(c);
}

bool overlap(const void *a, int64_t na, const void *b, int64_t nb) {
    const char *x = static_cast<const char *>(a), *y = static_cast<const char *>(b);
    return x < y + nb && y < x + na;
}

// Whether a result shares memory with an operand or with another result (buffers that are not given share none).
// Pools are left out: which of their pages a call touches is known to its table alone, and pages may lie among other
// things.
struct Buffer {
    const void *p;
    int64_t bytes;
};
bool clash(std::initializer_list<Buffer> results, std::initializer_list<Buffer> operands) {
    for (const Buffer *r = results.begin(); r != results.end(); ++r) {
        if (!r->p) continue;
        for (const Buffer &o : operands)
            if (o.p && overlap(r->p, r->bytes, o.p, o.bytes)) return true;
        for (const Buffer *o = results.begin(); o != r; ++o)
            if (o->p && overlap(r->p, r->bytes, o->p, o->bytes)) return true;
    }
    return false;
}

// n rows of `width` bytes, `stride` bytes apart (n = 1: a buffer).
struct RowSet {
    const void *p;
    int64_t n, stride, width;
};
RowSet one(const void *p, int64_t bytes) { return {p, 1, bytes, bytes}; }
// Whether a row of a and one of b share memory. Rows of one stride may lie between one another (views of a
// fused projection): they are compared by their places within the stride, which is exact. So are different strides,
// within their greatest common divisor, which takes some that interleave for rows that meet.
bool rows_meet(const RowSet &a, const RowSet &b) {
    if (!a.p || !b.p || !overlap(a.p, (a.n - 1) * a.stride + a.width, b.p, (b.n - 1) * b.stride + b.width)) return false;
    if (a.n == 1 && b.n == 1) return true;
    const int64_t g = a.n == 1 ? b.stride : (b.n == 1 ? a.stride : std::gcd(a.stride, b.stride));
    int64_t d = (static_cast<const char *>(b.p) - static_cast<const char *>(a.p)) % g;
    if (d < 0) d += g;
    return d < a.width || d + b.width > g;
}
bool same_rows(const RowSet &a, const RowSet &b) {
    return a.p == b.p && a.width == b.width && (a.stride == b.stride || a.n == 1);
}
// Whether a result of a norm meets an operand or another result; it may be one of its own operands `in` itself.
struct NormResult {
    RowSet rows;
    RowSet in[2];
};
bool norm_clash(std::initializer_list<NormResult> results, std::initializer_list<RowSet> operands) {
    for (const NormResult *r = results.begin(); r != results.end(); ++r) {
        auto itself = [&](const RowSet &o) {
            for (const RowSet &in : r->in)
                if (in.p && same_rows(in, o) && same_rows(r->rows, o)) return true;
            return false;
        };
        for (const RowSet &o : operands)
            if (rows_meet(r->rows, o) && !itself(o)) return true;
        for (const NormResult *o = results.begin(); o != r; ++o)
            if (rows_meet(r->rows, o->rows)) return true;
    }
    return false;
}

// Up to 128 query heads share a key head (a token's rows lie in one MMA tile).
bool heads_ok(int Hq, int Hkv) { return Hq > 0 && Hkv > 0 && Hq % Hkv == 0 && Hq / Hkv <= 128; }

// Checks shared by the three norm entry points.
fa_status norm_check(const void *q, const void *k, const float *cos_sin, int64_t max_pos, int rot, int64_t n, int Hq, int Hk,
                     int D, float eps, fa_dtype dtype) {
    if (dtype != FA_FP16 && dtype != FA_BF16) return FA_ERR_DTYPE;
    if (!fa::host_head_dim_ok(D)) return FA_ERR_HEADDIM;
    if (n < 0 || n > INT32_MAX || Hq <= 0 || Hk <= 0 || Hq > 65536 || Hk > 65536) return FA_ERR_SHAPE;
    if (rot < 16 || rot > D || rot % 16 != 0 || max_pos <= 0 || !(eps >= 0.f) || isinf(eps)) return FA_ERR_SHAPE;
    if (n == 0) return FA_OK;
    if (!q || !k || !cos_sin) return FA_ERR_NULL;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(cos_sin, 16)) return FA_ERR_ALIGN;
    return FA_OK;
}

bool stride_ok(int64_t stride, int H, int D) { return stride >= static_cast<int64_t>(H) * D && stride % 8 == 0; }

fa_status done(cudaError_t e) { return e == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

size_t round256(size_t v) { return (v + 255) & ~size_t(255); }

// Whether a call whose sequences have up to max_q_len new tokens runs in tiles of 16 rows.
bool few_rows(int G, int max_q_len) {
    return G <= fa::chunk_rows_tile() && static_cast<int64_t>(max_q_len) * G <= fa::chunk_rows_tile();
}

// Rows of a work item's tile.
int chunk_tile(int G, int D, int max_q_len) {
    return few_rows(G, max_q_len) ? fa::chunk_rows_tile() : fa::chunk_tile_rows(D);
}

// Whether K and V pools that a call writes would have a page in common whatever the table says, or parts of pages. Pools
// that lie a number of whole pages apart may interleave (K and V pages by turns).
bool pools_meet(const void *k, const void *v, int num_pages, int page_size, int Hkv, int D) {
    const int64_t page = static_cast<int64_t>(page_size) * Hkv * D * 2, pool = num_pages * page;
    return overlap(k, pool, v, pool) && (k == v || (static_cast<const char *>(v) - static_cast<const char *>(k)) % page != 0);
}
int64_t table_bytes(int num_seqs, int max_blocks) { return static_cast<int64_t>(num_seqs) * max_blocks * 4; }

size_t chunk_bytes(int R, int D, size_t *ml, size_t *o) {
    const size_t slots = 2 * static_cast<size_t>(fa::kChunkMaxCtas) * R;
    *ml = round256(fa::kChunkMaxCtas * sizeof(fa::ChunkDesc));
    *o = *ml + round256(slots * sizeof(float2));
    return *o + slots * D * sizeof(float);
}

// Checks and parameters shared by the attention of new tokens and the key weights.
fa_status chunk_params(fa::ChunkParams &p, const void *q, const int32_t *block_table, int max_blocks, int page_size,
                       int num_pages, const int32_t *cu_seqlens, const int32_t *kv_lens, int num_seqs, int total, int Hq,
                       int Hkv, int D, float scale) {
    if (!aligned(q, 16) || !aligned(block_table, 4) || !aligned(cu_seqlens, 4) || !aligned(kv_lens, 4)) return FA_ERR_ALIGN;
    p = fa::ChunkParams{};
    p.q = q;
    p.cu_seqlens = cu_seqlens;
    p.kv_lens = kv_lens;
    p.block_table = block_table;
    p.num_seqs = num_seqs;
    p.total = total;
    p.max_blocks = max_blocks;
    p.page_shift = log2_of(page_size);
    p.num_pages = num_pages;
    p.capacity = capacity_of(max_blocks, page_size);
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.G = Hq / Hkv;
    if (!(scale > 0.f)) scale = 1.0f / sqrtf(static_cast<float>(D));
    p.scale_log2 = scale * 1.4426950408889634f;
    p.timeout_ns = fa::host_wait_limit_ns();
    return FA_OK;
}

fa_status chunk_check(int max_blocks, int page_size, int num_pages, int num_seqs, int total, int max_q_len, int Hq, int Hkv,
                      int D, fa_dtype dtype) {
    if (dtype != FA_FP16 && dtype != FA_BF16) return FA_ERR_DTYPE;
    if (!fa::host_head_dim_ok(D)) return FA_ERR_HEADDIM;
    if (!heads_ok(Hq, Hkv) || Hq > 65536 || num_seqs < 0 || total < 0 || max_q_len < 0) return FA_ERR_SHAPE;
    if (static_cast<int64_t>(total) * (Hq / Hkv) > INT32_MAX / 2) return FA_ERR_SHAPE;
    return pages_ok(max_blocks, page_size, num_pages) ? FA_OK : FA_ERR_SHAPE;
}

int chunk_ctas() {
    const int sms = fa::host_sm_count();
    return sms > fa::kChunkMaxCtas ? fa::kChunkMaxCtas : sms;
}

}  // namespace

extern "C" {

fa_status fa_qk_norm_rope(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *q_weight,
                          const void *k_weight, int weight_fp32, const float *cos_sin, int64_t max_pos, int rot_dim,
                          const int64_t *positions, void *q_out, int64_t q_out_stride, void *k_out, int64_t k_out_stride,
                          int64_t n, int Hq, int Hkv, int D, float eps, int interleaved, fa_dtype dtype, void *stream) {
    const fa_status st = norm_check(q, k, cos_sin, max_pos, rot_dim, n, Hq, Hkv, D, eps, dtype);
    if (st != FA_OK || n == 0) return st;
    if (!positions || !q_out || !k_out) return FA_ERR_NULL;
    if (!stride_ok(q_stride, Hq, D) || !stride_ok(k_stride, Hkv, D) || !stride_ok(q_out_stride, Hq, D) ||
        !stride_ok(k_out_stride, Hkv, D))
        return FA_ERR_ALIGN;
    if (!aligned(q_out, 16) || !aligned(k_out, 16) || !aligned(q_weight, 16) || !aligned(k_weight, 16) ||
        !aligned(positions, 8))
        return FA_ERR_ALIGN;
    const int64_t wq = Hq * int64_t(D) * 2, wk = Hkv * int64_t(D) * 2, weight = D * (weight_fp32 ? 4 : 2);
    const RowSet rq{q, n, q_stride * 2, wq}, rk{k, n, k_stride * 2, wk}, none{};
    if (norm_clash({{{q_out, n, q_out_stride * 2, wq}, {rq, none}}, {{k_out, n, k_out_stride * 2, wk}, {rk, none}}},
                   {rq, rk, one(q_weight, weight), one(k_weight, weight), one(positions, n * 8)}))
        return FA_ERR_SHAPE;
    fa::QkNormParams p{};
    p.q = q; p.k = k;
    p.q_stride = q_stride; p.k_stride = k_stride;
    p.wq = q_weight; p.wk = k_weight; p.w32 = weight_fp32 != 0;
    p.cos_sin = cos_sin; p.max_pos = max_pos; p.rot = rot_dim; p.positions = positions;
    p.q_out = q_out; p.k_out = k_out;
    p.q_out_stride = q_out_stride; p.k_out_stride = k_out_stride;
    p.n = n; p.Hq = Hq; p.Hk = Hkv; p.eps = eps;
    return done(fa::launch_qk_norm(D, dtype == FA_BF16, interleaved != 0, false, p, static_cast<cudaStream_t>(stream)));
}

fa_status fa_qk_norm_rope_paged(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                                int64_t v_stride, const void *q_weight, const void *k_weight, int weight_fp32,
                                const float *cos_sin, int64_t max_pos, int rot_dim, const int64_t *positions, void *q_out,
                                int64_t q_out_stride, void *k_cache, void *v_cache, const int32_t *block_table,
                                int max_blocks_per_seq, int page_size, int num_pages, const int32_t *cu_seqlens,
                                const int32_t *kv_lens, int num_seqs, int64_t n, int Hq, int Hkv, int D, float eps,
                                int interleaved, fa_dtype dtype, void *stream) {
    const fa_status st = norm_check(q, k, cos_sin, max_pos, rot_dim, n, Hq, Hkv, D, eps, dtype);
    if (st != FA_OK) return st;
    if (num_seqs < 0 || !pages_ok(max_blocks_per_seq, page_size, num_pages)) return FA_ERR_SHAPE;
    if (n == 0 || num_seqs == 0) return FA_OK;
    if (!v || !q_out || !k_cache || !v_cache || !block_table || !cu_seqlens || !kv_lens) return FA_ERR_NULL;
    if (!stride_ok(q_stride, Hq, D) || !stride_ok(k_stride, Hkv, D) || !stride_ok(v_stride, Hkv, D) ||
        !stride_ok(q_out_stride, Hq, D))
        return FA_ERR_ALIGN;
    if (!aligned(v, 16) || !aligned(q_out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(q_weight, 16) ||
        !aligned(k_weight, 16) || !aligned(positions, 8) || !aligned(block_table, 4) || !aligned(cu_seqlens, 4) ||
        !aligned(kv_lens, 4))
        return FA_ERR_ALIGN;
    const int64_t wq = Hq * int64_t(D) * 2, wk = Hkv * int64_t(D) * 2, weight = D * (weight_fp32 ? 4 : 2);
    const RowSet rq{q, n, q_stride * 2, wq}, none{};
    if (pools_meet(k_cache, v_cache, num_pages, page_size, Hkv, D) ||
        norm_clash({{{q_out, n, q_out_stride * 2, wq}, {rq, none}}},
                   {rq, {k, n, k_stride * 2, wk}, {v, n, v_stride * 2, wk}, one(q_weight, weight), one(k_weight, weight),
                    one(positions, n * 8), one(block_table, table_bytes(num_seqs, max_blocks_per_seq)),
                    one(cu_seqlens, (num_seqs + int64_t(1)) * 4), one(kv_lens, num_seqs * int64_t(4))}))
        return FA_ERR_SHAPE;
    fa::QkNormParams p{};
    p.q = q; p.k = k; p.v = v;
    p.q_stride = q_stride; p.k_stride = k_stride; p.v_stride = v_stride;
    p.wq = q_weight; p.wk = k_weight; p.w32 = weight_fp32 != 0;
    p.cos_sin = cos_sin; p.max_pos = max_pos; p.rot = rot_dim; p.positions = positions;
    p.q_out = q_out; p.k_out = k_cache; p.v_out = v_cache;
    p.q_out_stride = q_out_stride;
    p.n = n; p.Hq = Hq; p.Hk = Hkv; p.eps = eps;
    p.cu_seqlens = cu_seqlens; p.kv_lens = kv_lens; p.block_table = block_table;
    p.num_seqs = num_seqs; p.max_blocks = max_blocks_per_seq; p.page_shift = log2_of(page_size); p.num_pages = num_pages;
    return done(fa::launch_qk_norm(D, dtype == FA_BF16, interleaved != 0, false, p, static_cast<cudaStream_t>(stream)));
}

int64_t fa_qk_norm_rope_bwd_workspace(int D) {
    return fa::host_head_dim_ok(D) ? static_cast<int64_t>(fa::kQkNormCtas + 1) * D * sizeof(float) : 0;
}

fa_status fa_qk_norm_rope_bwd(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *q_weight,
                              const void *k_weight, int weight_fp32, const float *cos_sin, int64_t max_pos, int rot_dim,
                              const int64_t *positions, const void *dq_out, int64_t dq_out_stride, const void *dk_out,
                              int64_t dk_out_stride, void *dq, int64_t dq_stride, void *dk, int64_t dk_stride,
                              float *dq_weight, float *dk_weight, void *workspace, int64_t workspace_bytes, int64_t n, int Hq,
                              int Hkv, int D, float eps, int interleaved, fa_dtype dtype, void *stream) {
    const fa_status st = norm_check(q, k, cos_sin, max_pos, rot_dim, n, Hq, Hkv, D, eps, dtype);
    if (st != FA_OK) return st;
    const bool weights = dq_weight || dk_weight;
    if (!aligned(dq_weight, 4) || !aligned(dk_weight, 4)) return FA_ERR_ALIGN;
    if (n == 0) {  // no rows: the weights' gradients are zero
        cudaError_t e = cudaSuccess;
        if (dq_weight) e = cudaMemsetAsync(dq_weight, 0, D * sizeof(float), static_cast<cudaStream_t>(stream));
        if (e == cudaSuccess && dk_weight) e = cudaMemsetAsync(dk_weight, 0, D * sizeof(float), static_cast<cudaStream_t>(stream));
        return done(e);
    }
    if (!positions || !dq_out || !dk_out || !dq || !dk || (weights && !workspace)) return FA_ERR_NULL;
    if (weights && workspace_bytes < fa_qk_norm_rope_bwd_workspace(D)) return FA_ERR_SHAPE;
    if (!stride_ok(q_stride, Hq, D) || !stride_ok(k_stride, Hkv, D) || !stride_ok(dq_out_stride, Hq, D) ||
        !stride_ok(dk_out_stride, Hkv, D) || !stride_ok(dq_stride, Hq, D) || !stride_ok(dk_stride, Hkv, D))
        return FA_ERR_ALIGN;
    if (!aligned(dq_out, 16) || !aligned(dk_out, 16) || !aligned(dq, 16) || !aligned(dk, 16) || !aligned(q_weight, 16) ||
        !aligned(k_weight, 16) || !aligned(positions, 8) || !aligned(workspace, 16))
        return FA_ERR_ALIGN;
    const int64_t wq = Hq * int64_t(D) * 2, wk = Hkv * int64_t(D) * 2, weight = D * (weight_fp32 ? 4 : 2);
    const RowSet rq{q, n, q_stride * 2, wq}, rk{k, n, k_stride * 2, wk}, gq{dq_out, n, dq_out_stride * 2, wq},
        gk{dk_out, n, dk_out_stride * 2, wk}, none{};
    if (norm_clash({{{dq, n, dq_stride * 2, wq}, {gq, rq}}, {{dk, n, dk_stride * 2, wk}, {gk, rk}}, {one(dq_weight, D * 4), {none, none}},
                    {one(dk_weight, D * 4), {none, none}}, {one(weights ? workspace : nullptr, fa_qk_norm_rope_bwd_workspace(D)), {none, none}}},
                   {rq, rk, gq, gk, one(q_weight, weight), one(k_weight, weight), one(positions, n * 8)}))
        return FA_ERR_SHAPE;
    fa::QkNormParams p{};
    p.q = q; p.k = k;
    p.q_stride = q_stride; p.k_stride = k_stride;
    p.wq = q_weight; p.wk = k_weight; p.w32 = weight_fp32 != 0;
    p.cos_sin = cos_sin; p.max_pos = max_pos; p.rot = rot_dim; p.positions = positions;
    p.dq_out = dq_out; p.dk_out = dk_out;
    p.dq_out_stride = dq_out_stride; p.dk_out_stride = dk_out_stride;
    p.q_out = dq; p.k_out = dk;
    p.q_out_stride = dq_stride; p.k_out_stride = dk_stride;
    p.partials = weights ? static_cast<float *>(workspace) : nullptr;
    p.dwq = dq_weight; p.dwk = dk_weight;
    p.n = n; p.Hq = Hq; p.Hk = Hkv; p.eps = eps;
    return done(fa::launch_qk_norm(D, dtype == FA_BF16, interleaved != 0, true, p, static_cast<cudaStream_t>(stream)));
}

int64_t fa_fwd_paged_chunk_workspace(int Hq, int Hkv, int D, int max_q_len) {
    if (!heads_ok(Hq, Hkv) || !fa::host_head_dim_ok(D) || max_q_len < 0) return 0;
    size_t ml, o;
    return static_cast<int64_t>(chunk_bytes(chunk_tile(Hq / Hkv, D, max_q_len), D, &ml, &o));
}

fa_status fa_fwd_paged_chunk(const void *q, const void *k_cache, const void *v_cache, const int32_t *block_table,
                             int max_blocks_per_seq, int page_size, int num_pages, const int32_t *cu_seqlens,
                             const int32_t *kv_lens, int num_seqs, int total, int max_q_len, void *out, float *lse,
                             void *workspace, int64_t workspace_bytes, int Hq, int Hkv, int D, float scale, int causal,
                             fa_dtype dtype, void *stream) {
    fa_status st = chunk_check(max_blocks_per_seq, page_size, num_pages, num_seqs, total, max_q_len, Hq, Hkv, D, dtype);
    if (st != FA_OK) return st;
    if (total == 0 || num_seqs == 0) return FA_OK;
    if (!q || !k_cache || !v_cache || !block_table || !cu_seqlens || !kv_lens || !out || !workspace) return FA_ERR_NULL;
    if (workspace_bytes < fa_fwd_paged_chunk_workspace(Hq, Hkv, D, max_q_len)) return FA_ERR_SHAPE;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(workspace, 256))
        return FA_ERR_ALIGN;
    fa::ChunkParams p;
    st = chunk_params(p, q, block_table, max_blocks_per_seq, page_size, num_pages, cu_seqlens, kv_lens, num_seqs, total, Hq,
                      Hkv, D, scale);
    if (st != FA_OK) return st;
    const int64_t rows_q = static_cast<int64_t>(total) * Hq;
    if (clash({{out, rows_q * D * 2}, {lse, rows_q * 4}, {workspace, fa_fwd_paged_chunk_workspace(Hq, Hkv, D, max_q_len)}},
              {{q, rows_q * D * 2}, {block_table, table_bytes(num_seqs, max_blocks_per_seq)},
               {cu_seqlens, (num_seqs + int64_t(1)) * 4}, {kv_lens, num_seqs * int64_t(4)}}))
        return FA_ERR_SHAPE;
    p.out = out;
    p.lse = lse;
    const int R = chunk_tile(p.G, D, max_q_len);
    size_t ml, o;
    chunk_bytes(R, D, &ml, &o);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.desc = reinterpret_cast<fa::ChunkDesc *>(ws);
    p.part_ml = reinterpret_cast<float2 *>(ws + ml);
    p.part_o = reinterpret_cast<float *>(ws + o);
    const int ctas = chunk_ctas();
    if (ctas <= 0) return FA_ERR_CUDA;
    const bool bf16 = dtype == FA_BF16;
    const bool few = few_rows(p.G, max_q_len);
    const int inner = fa::fwd_box_inner_elems(D);
    const int k_box = few ? fa::chunk_rows_box(D, page_size) : fa::chunk_tile_k_box(D, page_size);
    const int v_box = few ? fa::chunk_rows_box(D, page_size) : fa::chunk_tile_v_box(D, page_size);
    p.mma_tiles = few ? 1 : R / 128;
    p.tile_tokens = p.mma_tiles * ((few ? R : 128) / p.G);
    p.min_cost = p.mma_tiles;  // at least the cost of a step
    p.out_align32 = aligned(out, 32);
    CUtensorMap tk, tv;
    const int64_t rows = static_cast<int64_t>(num_pages) * page_size;
    if (!fa::host_encode_pool_map(&tk, k_cache, bf16, D, Hkv, rows, inner, k_box) ||
        !fa::host_encode_pool_map(&tv, v_cache, bf16, D, Hkv, rows, inner, v_box))
        return FA_ERR_CUDA;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (few) return done(fa::launch_chunk_rows(D, bf16, causal != 0, tk, tv, p, ctas, cs));
    CUtensorMap tq;
    if (!fa::host_encode_group_map(&tq, q, bf16, D, p.G, Hkv, total, inner, 128 / p.G)) return FA_ERR_CUDA;
    return done(fa::launch_chunk_tile(D, bf16, causal != 0, tq, tk, tv, p, ctas, cs));
}

int64_t fa_paged_key_weights_workspace(int Hq, int Hkv, int D, int max_q_len) {
    if (!heads_ok(Hq, Hkv) || !fa::host_head_dim_ok(D) || max_q_len < 0 || few_rows(Hq / Hkv, max_q_len)) return 0;
    return static_cast<int64_t>(round256(fa::kChunkMaxCtas * sizeof(fa::ChunkDesc)) +
                                2 * fa::kChunkMaxCtas * fa::kKeyWeightsPiece * sizeof(float));
}

fa_status fa_paged_key_weights(const void *q, const void *k_cache, const int32_t *block_table, int max_blocks_per_seq,
                               int page_size, int num_pages, const int32_t *cu_seqlens, const int32_t *kv_lens, int num_seqs,
                               int total, int max_q_len, const float *lse, float *weights, int64_t width, void *workspace,
                               int64_t workspace_bytes, int Hq, int Hkv, int D, float scale, int causal, fa_dtype dtype,
                               void *stream) {
    fa_status st = chunk_check(max_blocks_per_seq, page_size, num_pages, num_seqs, total, max_q_len, Hq, Hkv, D, dtype);
    if (st != FA_OK) return st;
    if (width < static_cast<int64_t>(max_blocks_per_seq) * page_size) return FA_ERR_SHAPE;
    if (total == 0 || num_seqs == 0) return FA_OK;
    const bool few = few_rows(Hq / Hkv, max_q_len);
    if (!q || !k_cache || !block_table || !cu_seqlens || !kv_lens || !lse || !weights || (!few && !workspace)) return FA_ERR_NULL;
    if (!few && workspace_bytes < fa_paged_key_weights_workspace(Hq, Hkv, D, max_q_len)) return FA_ERR_SHAPE;
    if (!aligned(k_cache, 16) || !aligned(lse, 4) || !aligned(weights, 4) || (!few && !aligned(workspace, 256)))
        return FA_ERR_ALIGN;
    fa::ChunkParams p;
    st = chunk_params(p, q, block_table, max_blocks_per_seq, page_size, num_pages, cu_seqlens, kv_lens, num_seqs, total, Hq,
                      Hkv, D, scale);
    if (st != FA_OK) return st;
    const int64_t rows_q = static_cast<int64_t>(total) * Hq;
    if (clash({{weights, static_cast<int64_t>(num_seqs) * Hkv * width * 4},
               {few ? nullptr : workspace, fa_paged_key_weights_workspace(Hq, Hkv, D, max_q_len)}},
              {{q, rows_q * D * 2}, {lse, rows_q * 4}, {block_table, table_bytes(num_seqs, max_blocks_per_seq)},
               {cu_seqlens, (num_seqs + int64_t(1)) * 4}, {kv_lens, num_seqs * int64_t(4)}}))
        return FA_ERR_SHAPE;
    p.lse_in = lse;
    p.weights = weights;
    p.width = width;
    const int ctas = chunk_ctas();
    if (ctas <= 0) return FA_ERR_CUDA;
    const bool bf16 = dtype == FA_BF16;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const int inner = fa::fwd_box_inner_elems(D);
    CUtensorMap tk, tq;
    if (!fa::host_encode_pool_map(&tk, k_cache, bf16, D, Hkv, static_cast<int64_t>(num_pages) * page_size, inner,
                             fa::key_weights_box(page_size)))
        return FA_ERR_CUDA;
    if (few) return done(fa::launch_key_weights(D, bf16, causal != 0, tk, p, ctas, cs));
    p.tile_tokens = 128 / p.G;
    p.mma_tiles = 1;
    p.desc = static_cast<fa::ChunkDesc *>(workspace);
    p.part_o = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + round256(fa::kChunkMaxCtas * sizeof(fa::ChunkDesc)));
    if (!fa::host_encode_group_map(&tq, q, bf16, D, p.G, Hkv, total, inner, p.tile_tokens)) return FA_ERR_CUDA;
    return done(fa::launch_key_weights_tile(D, bf16, causal != 0, tq, tk, p, ctas, cs));
}

fa_status fa_paged_evict(void *k_cache, void *v_cache, const int32_t *block_table, int max_blocks_per_seq, int page_size,
                         int num_pages, const int32_t *kv_lens, const float *weights, int64_t width, int budget, int recent,
                         int32_t *kept, int32_t *new_lens, float *new_weights, int B, int Hkv, int D, fa_dtype dtype,
                         void *stream) {
    if (dtype != FA_FP16 && dtype != FA_BF16) return FA_ERR_DTYPE;
    if (!fa::host_head_dim_ok(D)) return FA_ERR_HEADDIM;
    if (B < 0 || B > 65535 || Hkv <= 0 || Hkv > 65535 || budget <= 0 || recent < 0 || recent > budget) return FA_ERR_SHAPE;
    if (!pages_ok(max_blocks_per_seq, page_size, num_pages)) return FA_ERR_SHAPE;
    if (width < static_cast<int64_t>(max_blocks_per_seq) * page_size || width > fa::kMaxSeqKeys || budget > width) return FA_ERR_SHAPE;
    if (B == 0) return FA_OK;
    if (!k_cache || !v_cache || !block_table || !kv_lens || !weights || !kept || !new_lens || !new_weights) return FA_ERR_NULL;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(block_table, 4) || !aligned(kv_lens, 4) ||
        !aligned(weights, 4) || !aligned(kept, 4) || !aligned(new_lens, 4) || !aligned(new_weights, 4))
        return FA_ERR_ALIGN;
    // the inputs are read again while the results are written, and K and V rows move side by side
    const int64_t heads = static_cast<int64_t>(B) * Hkv, w_bytes = heads * width * 4, lens = B * int64_t(4);
    if (pools_meet(k_cache, v_cache, num_pages, page_size, Hkv, D) ||
        clash({{kept, heads * budget * 4}, {new_lens, lens}, {new_weights, w_bytes}},
              {{weights, w_bytes}, {kv_lens, lens}, {block_table, table_bytes(B, max_blocks_per_seq)}}))
        return FA_ERR_SHAPE;
    fa::EvictParams p{};
    p.k_cache = k_cache; p.v_cache = v_cache;
    p.block_table = block_table; p.kv_lens = kv_lens;
    p.batch = B; p.max_blocks = max_blocks_per_seq; p.page_shift = log2_of(page_size); p.num_pages = num_pages;
    p.capacity = capacity_of(max_blocks_per_seq, page_size);
    p.Hkv = Hkv; p.D = D;
    p.weights = weights; p.width = width; p.budget = budget; p.recent = recent;
    p.kept = kept; p.new_lens = new_lens; p.new_weights = new_weights;
    return done(fa::launch_evict(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
