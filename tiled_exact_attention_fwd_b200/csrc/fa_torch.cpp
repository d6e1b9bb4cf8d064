// fa_torch.cpp -- the Python binding's marshalling for the operators around a paged cache: checks of
// the tensors, allocation of results and workspaces, the call into the C ABI of include/fa.h. These
// calls run several times per generated token, where the same steps taken in Python (10 to 28 us a
// call) would cost more than the kernels (4 to 12 us). Nothing is computed here.
//
// Each function returns the C call's status first; the Python side raises FAError for one that is not 0.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <algorithm>

#include "fa.h"

namespace {

using at::Tensor;
using Maybe = std::optional<Tensor>;

fa_dtype dtype_code(const Tensor &t) {
    if (t.scalar_type() == at::kHalf) return FA_FP16;
    TORCH_CHECK_TYPE(t.scalar_type() == at::kBFloat16, "unsupported dtype ", t.scalar_type(), "; expected float16 or bfloat16");
    return FA_BF16;
}

void *ptr(const Maybe &t) { return t ? t->data_ptr() : nullptr; }

// A contiguous tensor of one dtype on the operands' device.
void plain(const char *name, const Tensor &t, at::ScalarType dtype, const at::Device &dev) {
    TORCH_CHECK_VALUE(t.scalar_type() == dtype, name, " must be ", dtype, ", got ", t.scalar_type());
    TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
    TORCH_CHECK_VALUE(t.device() == dev, name, " must be on ", dev, ", is on ", t.device());
}

// Token rows of a (..., H, D) tensor, and the elements from one to the next: the heads of a token are
// contiguous, the tokens lie at one stride.
struct Rows {
    int64_t n, stride, H, D;
    void *data;
};
Rows rows(const char *name, const Tensor &t) {
    TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a CUDA tensor");
    const auto size = t.sizes(), step = t.strides();
    const int64_t dim = t.dim();
    TORCH_CHECK_VALUE(dim >= 3, name, " must be (..., heads, head dim)");
    Rows r{1, 0, size[dim - 2], size[dim - 1], t.data_ptr()};
    TORCH_CHECK_VALUE((r.D <= 1 || step[dim - 1] == 1) && (r.H <= 1 || step[dim - 2] == r.D), "the heads of a token of ", name,
                      " must be contiguous");
    r.stride = r.H * r.D;
    if (t.numel() == 0) {
        r.n = 0;
        return r;
    }
    for (int64_t i = dim - 3; i >= 0; --i) {
        if (size[i] == 1) continue;
        if (r.n == 1)
            r.stride = step[i];
        else
            TORCH_CHECK_VALUE(step[i] == r.stride * r.n, "the tokens of ", name, " must lie at one stride");
        r.n *= size[i];
    }
    return r;
}

// The same of a caller-given tensor that has to be like another.
Rows rows_like(const char *name, const Tensor &t, const Tensor &like) {
    TORCH_CHECK_VALUE(t.sizes() == like.sizes() && t.scalar_type() == like.scalar_type() && t.device() == like.device(), name,
                      " must be ", like.scalar_type(), " ", like.sizes(), " on ", like.device(), ", got ", t.scalar_type(), " ",
                      t.sizes(), " on ", t.device());
    return rows(name, t);
}

Tensor fresh_like(const Tensor &t) { return at::empty(t.sizes(), t.options()); }
Tensor fresh(at::IntArrayRef size, at::ScalarType dtype, const Tensor &on) { return at::empty(size, on.options().dtype(dtype)); }

void *stream_of(const at::Device &dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

// What the norm entry points share.
struct Norm {
    Rows q, k;
    fa_dtype dtype;
    void *wq, *wk;
    int w32;
    const float *cos_sin;
    int64_t rows;
    int rot;
    const int64_t *positions;
};
Norm norm_args(const Tensor &q, const Tensor &k, const Maybe &q_weight, const Maybe &k_weight, const Tensor &cos_sin,
               const Maybe &positions) {
    Norm a{};
    a.q = rows("q", q);
    a.k = rows("k", k);
    a.dtype = dtype_code(q);
    const auto lead = q.sizes().slice(0, q.dim() - 2);
    const at::Device dev = q.device();
    TORCH_CHECK_VALUE(k.dim() == q.dim() && k.sizes().slice(0, k.dim() - 2) == lead && a.k.D == a.q.D &&
                          k.scalar_type() == q.scalar_type() && k.device() == dev,
                      "q and k must share their leading shape, head dim, dtype and device");
    const Maybe *weights[2] = {&q_weight, &k_weight};
    for (int i = 0; i < 2; ++i) {
        const Maybe &w = *weights[i];
        if (!w) continue;
        const bool is32 = w->scalar_type() == at::kFloat;
        plain(i ? "k_weight" : "q_weight", *w, is32 ? at::kFloat : q.scalar_type(), dev);
        TORCH_CHECK_VALUE(w->dim() == 1 && w->size(0) == a.q.D, "the weights must be (", a.q.D, ",), got ", w->sizes());
        TORCH_CHECK_VALUE(i == 0 || !q_weight || is32 == (a.w32 != 0), "q_weight and k_weight must share one dtype");
        a.w32 = is32;
    }
    a.wq = ptr(q_weight);
    a.wk = ptr(k_weight);
    plain("cos_sin", cos_sin, at::kFloat, dev);
    TORCH_CHECK_VALUE(cos_sin.dim() == 2, "cos_sin must be (positions, rot_dim)");
    a.cos_sin = static_cast<const float *>(cos_sin.data_ptr());
    a.rows = cos_sin.size(0);
    a.rot = static_cast<int>(cos_sin.size(1));
    if (positions) {
        plain("positions", *positions, at::kLong, dev);
        TORCH_CHECK_VALUE(positions->sizes() == lead, "positions must be of q's leading shape");
        a.positions = static_cast<const int64_t *>(positions->data_ptr());
    }
    return a;
}

std::tuple<int, Tensor, Tensor> qk_norm_rope(const Tensor &q, const Tensor &k, const Maybe &q_weight, const Maybe &k_weight,
                                             const Tensor &cos_sin, const Tensor &positions, double eps, bool interleaved,
                                             const Maybe &q_out, const Maybe &k_out) {
    const Norm a = norm_args(q, k, q_weight, k_weight, cos_sin, positions);
    const c10::cuda::OptionalCUDAGuard guard(q.device());
    const Tensor yq = q_out ? *q_out : fresh_like(q), yk = k_out ? *k_out : fresh_like(k);
    const Rows rq = rows_like("q_out", yq, q), rk = rows_like("k_out", yk, k);
    const int st = fa_qk_norm_rope(a.q.data, a.q.stride, a.k.data, a.k.stride, a.wq, a.wk, a.w32, a.cos_sin, a.rows, a.rot,
                                   a.positions, rq.data, rq.stride, rk.data, rk.stride, a.q.n, a.q.H, a.k.H, a.q.D,
                                   static_cast<float>(eps), interleaved, a.dtype, stream_of(q.device()));
    return {st, yq, yk};
}

std::tuple<int, Tensor, Tensor, Maybe, Maybe> qk_norm_rope_bwd(const Tensor &q, const Tensor &k, const Maybe &q_weight,
                                                               const Maybe &k_weight, const Tensor &cos_sin,
                                                               const Tensor &positions, const Tensor &dq_out,
                                                               const Tensor &dk_out, double eps, bool interleaved) {
    const Norm a = norm_args(q, k, q_weight, k_weight, cos_sin, positions);
    const Rows gq = rows_like("dq_out", dq_out, q), gk = rows_like("dk_out", dk_out, k);
    const c10::cuda::OptionalCUDAGuard guard(q.device());
    const Tensor dq = fresh_like(q), dk = fresh_like(k);
    Maybe dwq, dwk, ws;
    if (q_weight) dwq = fresh({a.q.D}, at::kFloat, q);
    if (k_weight) dwk = fresh({a.q.D}, at::kFloat, q);
    const int64_t size = dwq || dwk ? fa_qk_norm_rope_bwd_workspace(static_cast<int>(a.q.D)) : 0;
    if (size) ws = fresh({size}, at::kByte, q);
    const int st = fa_qk_norm_rope_bwd(a.q.data, a.q.stride, a.k.data, a.k.stride, a.wq, a.wk, a.w32, a.cos_sin, a.rows, a.rot,
                                       a.positions, gq.data, gq.stride, gk.data, gk.stride, dq.data_ptr(), a.q.H * a.q.D,
                                       dk.data_ptr(), a.k.H * a.k.D, static_cast<float *>(ptr(dwq)),
                                       static_cast<float *>(ptr(dwk)), ptr(ws), size, a.q.n, a.q.H, a.k.H, a.q.D,
                                       static_cast<float>(eps), interleaved, a.dtype, stream_of(q.device()));
    return {st, dq, dk, dwq, dwk};
}

// Page pools and their table.
struct Pages {
    const int32_t *table, *kv_lens;
    int max_blocks, page_size, num_pages, num;
    int64_t Hkv, D;
};
Pages page_args(const Tensor &k_cache, const Tensor *v_cache, const Tensor &block_table, const Tensor &kv_lens) {
    TORCH_CHECK_VALUE(k_cache.is_cuda() && k_cache.is_contiguous(), "k_cache must be a contiguous CUDA tensor");
    TORCH_CHECK_VALUE(k_cache.dim() == 4, "k_cache must be (num_pages, page_size, Hkv, D)");
    const at::Device dev = k_cache.device();
    if (v_cache) {
        plain("v_cache", *v_cache, k_cache.scalar_type(), dev);
        TORCH_CHECK_VALUE(v_cache->sizes() == k_cache.sizes(), "k_cache and v_cache must share one shape");
    }
    plain("kv_lens", kv_lens, at::kInt, dev);
    plain("block_table", block_table, at::kInt, dev);
    TORCH_CHECK_VALUE(kv_lens.dim() == 1 && block_table.dim() == 2 && block_table.size(0) == kv_lens.size(0),
                      "kv_lens must be (sequences,) and block_table (sequences, max_blocks_per_seq)");
    TORCH_CHECK_VALUE(k_cache.size(0) <= INT32_MAX && k_cache.size(1) <= INT32_MAX && block_table.size(1) <= INT32_MAX &&
                          kv_lens.size(0) <= INT32_MAX, "page pools are too large");
    return {static_cast<const int32_t *>(block_table.data_ptr()), static_cast<const int32_t *>(kv_lens.data_ptr()),
            static_cast<int>(block_table.size(1)), static_cast<int>(k_cache.size(1)), static_cast<int>(k_cache.size(0)),
            static_cast<int>(kv_lens.size(0)), k_cache.size(2), k_cache.size(3)};
}

// Packed new tokens over pools.
const int32_t *packed_args(const Tensor &q, const Tensor &k_cache, const Tensor &cu_seqlens, const Pages &g) {
    plain("cu_seqlens", cu_seqlens, at::kInt, k_cache.device());
    TORCH_CHECK_VALUE(cu_seqlens.dim() == 1 && cu_seqlens.size(0) == g.num + 1, "cu_seqlens must hold one more entry than kv_lens");
    TORCH_CHECK_VALUE(q.dim() == 3 && q.size(2) == g.D && q.scalar_type() == k_cache.scalar_type() && q.device() == k_cache.device(),
                      "q must be (total, Hq, D) with the caches' head dim, dtype and device");
    TORCH_CHECK_VALUE(q.size(0) <= INT32_MAX, "too many tokens");
    return static_cast<const int32_t *>(cu_seqlens.data_ptr());
}

std::tuple<int, Tensor> qk_norm_rope_paged(const Tensor &q, const Tensor &k, const Tensor &v, const Maybe &q_weight,
                                           const Maybe &k_weight, const Tensor &cos_sin, const Maybe &positions,
                                           const Tensor &k_cache, const Tensor &v_cache, const Tensor &block_table,
                                           const Tensor &cu_seqlens, const Tensor &kv_lens, double eps, bool interleaved,
                                           const Maybe &q_out) {
    const Norm a = norm_args(q, k, q_weight, k_weight, cos_sin, positions);
    const Pages g = page_args(k_cache, &v_cache, block_table, kv_lens);
    const int32_t *cu = packed_args(q, k_cache, cu_seqlens, g);
    TORCH_CHECK_VALUE(a.k.H == g.Hkv, "k and v must be (total, Hkv, D) like the caches' rows");
    const Rows rv = rows_like("v", v, k);
    const c10::cuda::OptionalCUDAGuard guard(q.device());
    const Tensor y = q_out ? *q_out : fresh_like(q);
    const Rows rq = rows_like("q_out", y, q);
    const int st = fa_qk_norm_rope_paged(a.q.data, a.q.stride, a.k.data, a.k.stride, rv.data, rv.stride, a.wq, a.wk, a.w32,
                                         a.cos_sin, a.rows, a.rot, a.positions, rq.data, rq.stride, k_cache.data_ptr(),
                                         v_cache.data_ptr(), g.table, g.max_blocks, g.page_size, g.num_pages, cu, g.kv_lens,
                                         g.num, a.q.n, a.q.H, a.k.H, a.q.D, static_cast<float>(eps), interleaved, a.dtype,
                                         stream_of(q.device()));
    return {st, y};
}

std::tuple<int, Tensor, Maybe> fwd_paged_chunk(const Tensor &q, const Tensor &k_cache, const Tensor &v_cache,
                                               const Tensor &block_table, const Tensor &cu_seqlens, const Tensor &kv_lens,
                                               int max_q_len, const Maybe &out, const Maybe &lse, double scale, bool causal,
                                               bool return_lse, const Maybe &workspace) {
    const Pages g = page_args(k_cache, &v_cache, block_table, kv_lens);
    const int32_t *cu = packed_args(q, k_cache, cu_seqlens, g);
    TORCH_CHECK_VALUE(q.is_contiguous(), "q must be contiguous");
    const at::Device dev = q.device();
    const int64_t total = q.size(0), Hq = q.size(1);
    const fa_dtype dtype = dtype_code(q);
    const c10::cuda::OptionalCUDAGuard guard(dev);
    const Tensor o = out ? *out : fresh_like(q);
    if (out) {
        plain("out", o, q.scalar_type(), dev);
        TORCH_CHECK_VALUE(o.sizes() == q.sizes(), "out must be ", q.sizes(), ", got ", o.sizes());
    }
    Maybe l = lse;
    if (l) {
        plain("lse", *l, at::kFloat, dev);
        TORCH_CHECK_VALUE(l->dim() == 2 && l->size(0) == Hq && l->size(1) == total, "lse must be (Hq, total)");
    } else if (return_lse) {
        l = fresh({Hq, total}, at::kFloat, q);
    }
    Tensor ws;
    int64_t size = 0;
    if (workspace) {
        ws = *workspace;
        TORCH_CHECK_VALUE(ws.is_contiguous() && ws.device() == dev, "workspace must be contiguous and on ", dev);
        size = ws.numel() * ws.element_size();
    } else {
        size = fa_fwd_paged_chunk_workspace(Hq, g.Hkv, g.D, max_q_len);
        ws = fresh({size}, at::kByte, q);
    }
    const int st = fa_fwd_paged_chunk(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), g.table, g.max_blocks, g.page_size,
                                      g.num_pages, cu, g.kv_lens, g.num, total, max_q_len, o.data_ptr(),
                                      static_cast<float *>(ptr(l)), ws.data_ptr(), size, Hq, g.Hkv, g.D,
                                      static_cast<float>(scale), causal, dtype, stream_of(dev));
    return {st, o, l};
}

const Tensor &weights_arg(const Tensor &weights, const Pages &g, const at::Device &dev) {
    plain("weights", weights, at::kFloat, dev);
    TORCH_CHECK_VALUE(weights.dim() == 3 && weights.size(0) == g.num && weights.size(1) == g.Hkv,
                      "weights must be (sequences, Hkv, width)");
    return weights;
}

int paged_key_weights(const Tensor &q, const Tensor &k_cache, const Tensor &block_table, const Tensor &cu_seqlens,
                      const Tensor &kv_lens, int max_q_len, const Tensor &lse, const Tensor &weights, double scale, bool causal,
                      const Maybe &workspace) {
    const Pages g = page_args(k_cache, nullptr, block_table, kv_lens);
    const int32_t *cu = packed_args(q, k_cache, cu_seqlens, g);
    TORCH_CHECK_VALUE(q.is_contiguous(), "q must be contiguous");
    const at::Device dev = q.device();
    const int64_t total = q.size(0), Hq = q.size(1);
    plain("lse", lse, at::kFloat, dev);
    TORCH_CHECK_VALUE(lse.dim() == 2 && lse.size(0) == Hq && lse.size(1) == total, "lse must be (Hq, total)");
    weights_arg(weights, g, dev);
    const fa_dtype dtype = dtype_code(q);
    const c10::cuda::OptionalCUDAGuard guard(dev);
    Maybe ws = workspace;
    int64_t size = 0;
    if (ws) {
        TORCH_CHECK_VALUE(ws->is_contiguous() && ws->device() == dev, "workspace must be contiguous and on ", dev);
        size = ws->numel() * ws->element_size();
    } else {
        size = fa_paged_key_weights_workspace(Hq, g.Hkv, g.D, max_q_len);
        if (size) ws = fresh({size}, at::kByte, q);
    }
    return fa_paged_key_weights(q.data_ptr(), k_cache.data_ptr(), g.table, g.max_blocks, g.page_size, g.num_pages, cu, g.kv_lens,
                                g.num, total, max_q_len, static_cast<const float *>(lse.data_ptr()),
                                static_cast<float *>(weights.data_ptr()), weights.size(2), ptr(ws), size, Hq, g.Hkv, g.D,
                                static_cast<float>(scale), causal, dtype, stream_of(dev));
}

std::tuple<int, Tensor, Tensor, Tensor> paged_evict(const Tensor &k_cache, const Tensor &v_cache, const Tensor &block_table,
                                                    const Tensor &kv_lens, const Tensor &weights, int budget, int recent) {
    const Pages g = page_args(k_cache, &v_cache, block_table, kv_lens);
    const at::Device dev = k_cache.device();
    weights_arg(weights, g, dev);
    const fa_dtype dtype = dtype_code(k_cache);
    const c10::cuda::OptionalCUDAGuard guard(dev);
    // (a budget that the call below refuses allocates no more than one that it takes)
    const int64_t held = std::clamp<int64_t>(budget, 0, weights.size(2));
    const Tensor kept = fresh({g.num, g.Hkv, held}, at::kInt, kv_lens);
    const Tensor new_lens = fresh_like(kv_lens), new_weights = fresh_like(weights);
    const int st = fa_paged_evict(k_cache.data_ptr(), v_cache.data_ptr(), g.table, g.max_blocks, g.page_size, g.num_pages,
                                  g.kv_lens, static_cast<const float *>(weights.data_ptr()), weights.size(2), budget, recent,
                                  static_cast<int32_t *>(kept.data_ptr()), static_cast<int32_t *>(new_lens.data_ptr()),
                                  static_cast<float *>(new_weights.data_ptr()), g.num, g.Hkv, g.D, dtype, stream_of(dev));
    return {st, kept, new_lens, new_weights};
}

}  // namespace

PYBIND11_MODULE(_fa_torch, m) {
    m.def("qk_norm_rope", &qk_norm_rope);
    m.def("qk_norm_rope_bwd", &qk_norm_rope_bwd);
    m.def("qk_norm_rope_paged", &qk_norm_rope_paged);
    m.def("fwd_paged_chunk", &fwd_paged_chunk);
    m.def("paged_key_weights", &paged_key_weights);
    m.def("paged_evict", &paged_evict);
}
