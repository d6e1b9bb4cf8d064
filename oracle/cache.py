"""Float64 definitions of the operators around a paged cache (test infrastructure, plain torch on the
CPU, loops over sequences and heads): norm of queries and keys with the position rotation and its
gradients, the append, attention of new tokens over the pages, key weights, eviction.

Where a test needs an error bound, a function also returns the size of the terms that were summed."""
from __future__ import annotations

import math

import torch


def _f(x):
    return x.detach().cpu().double()


def rotate(x, cos_sin, positions, interleaved, back=False):
    """x (n, H, D) float64, the pairs of its first cos_sin.shape[1] values turned by their token's angles."""
    rot = cos_sin.shape[1]
    cs = _f(cos_sin)[positions.cpu()]
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:] * (-1 if back else 1)
    y = x.clone()
    first = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    second = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    a, b = x[..., first], x[..., second]
    y[..., first] = a * c - b * s
    y[..., second] = b * c + a * s
    return y


def norm_rope(x, w, cos_sin, positions, eps, interleaved):
    """-> (y, size of y's terms), both (n, H, D)."""
    x = _f(x)
    n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if w is not None:
        n = n * _f(w)
    size = rotate(n.abs(), cos_sin.abs(), positions, interleaved, back=False)
    # |a| |c| + |b| |s| in both halves: turn the absolute values both ways and take the larger
    size = torch.maximum(size, rotate(n.abs(), cos_sin.abs(), positions, interleaved, back=True))
    return rotate(n, cos_sin, positions, interleaved), size


def norm_rope_bwd(x, w, cos_sin, positions, dy, eps, interleaved):
    """-> (dx, dw, size of dx's terms, size of dw's terms)."""
    x, dy = _f(x), _f(dy)
    D = x.shape[-1]
    w = torch.ones(D, dtype=torch.float64) if w is None else _f(w)
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    g = rotate(dy, cos_sin, positions, interleaved, back=True)
    ga = torch.maximum(rotate(dy.abs(), cos_sin.abs(), positions, interleaved, back=True),
                       rotate(dy.abs(), cos_sin.abs(), positions, interleaved))
    u = g * w
    dx = r * u - x * r ** 3 * (u * x).sum(-1, keepdim=True) / D
    size = r * ga * w.abs() + x.abs() * r ** 3 * (ga * w.abs() * x.abs()).sum(-1, keepdim=True) / D
    return dx, (g * x * r).sum((0, 1)), size, (ga * x.abs() * r).sum((0, 1))


def token_rows(cache, block_table, b, n):
    """Keys 0 .. n - 1 of sequence b out of a pool: (n, Hkv, D) float64."""
    page = cache.shape[1]
    rows = [cache[int(block_table[b, i // page]), i % page] for i in range(n)]
    return torch.stack(rows).detach().cpu().double() if rows else torch.zeros((0,) + tuple(cache.shape[2:]), dtype=torch.float64)


def chunk_attention(q, k_cache, v_cache, block_table, cu_seqlens, kv_lens, scale=None, causal=True):
    """-> out (total, Hq, D), lse (Hq, total), size of out's terms, size of the scores' terms (Hq, total);
    rows of no sequence are NaN."""
    q, k_cache, v_cache, block_table = (t.detach().cpu() for t in (q, k_cache, v_cache, block_table))
    total, Hq, D = q.shape
    Hkv = k_cache.shape[2]
    G = Hq // Hkv
    scale = 1 / math.sqrt(D) if scale is None else scale
    out = torch.full((total, Hq, D), math.nan, dtype=torch.float64)
    size = out.clone()
    lse = torch.full((Hq, total), math.nan, dtype=torch.float64)
    ssize = lse.clone()
    cu, kv = cu_seqlens.tolist(), kv_lens.tolist()
    for b in range(len(kv)):
        n = cu[b + 1] - cu[b]
        k, v = token_rows(k_cache, block_table, b, kv[b]), token_rows(v_cache, block_table, b, kv[b])
        for h in range(Hq):
            for i in range(n):
                see = max(0, kv[b] - n + i + 1) if causal else kv[b]
                x, r = q[cu[b] + i, h].double(), cu[b] + i
                if see == 0:
                    out[r, h], size[r, h], lse[h, r], ssize[h, r] = 0, 0, -math.inf, 0
                    continue
                z = k[:see, h // G] @ x * scale
                lse[h, r] = torch.logsumexp(z, 0)
                p = torch.softmax(z, 0)
                out[r, h] = p @ v[:see, h // G]
                size[r, h] = p @ v[:see, h // G].abs()
                ssize[h, r] = (k[:see, h // G].abs() @ x.abs()).max() * scale
    return out, lse, size, ssize


def key_weights(q, k_cache, block_table, cu_seqlens, kv_lens, lse, width, scale=None, causal=True):
    """-> what the call adds to the weights, (B, Hkv, width), and the largest score term."""
    q, k_cache, block_table, lse = (t.detach().cpu() for t in (q, k_cache, block_table, lse))
    total, Hq, D = q.shape
    Hkv = k_cache.shape[2]
    G = Hq // Hkv
    scale = 1 / math.sqrt(D) if scale is None else scale
    cu, kv = cu_seqlens.tolist(), kv_lens.tolist()
    add = torch.zeros(len(kv), Hkv, width, dtype=torch.float64)
    most = 0.0
    for b in range(len(kv)):
        n = cu[b + 1] - cu[b]
        k = token_rows(k_cache, block_table, b, kv[b])
        for h in range(Hq):
            for i in range(n):
                see = max(0, kv[b] - n + i + 1) if causal else kv[b]
                r = cu[b] + i
                if see == 0 or lse[h, r] == -math.inf:
                    continue
                x = q[r, h].double()
                add[b, h // G, :see] += torch.exp(k[:see, h // G] @ x * scale - lse[h, r].double())
                most = max(most, float((k[:see, h // G].abs() @ x.abs()).max() * scale))
    return add, most


def evict(weights, kv_lens, budget, recent):
    """-> kept (B, Hkv, budget) int32, new lengths, new weights: by sorting (weight, slot) pairs."""
    weights = weights.detach().cpu()
    B, H, width = weights.shape
    kept = torch.full((B, H, budget), -1, dtype=torch.int32)
    out = torch.zeros_like(weights)
    lens = []
    for b, n in enumerate(kv_lens.tolist()):
        m = min(n, budget)
        lens.append(m)
        for h in range(H):
            if n <= budget:
                stay = list(range(n))
            else:
                old = n - min(n, recent)
                key = lambda i: (-math.inf if math.isnan(weights[b, h, i]) else -float(weights[b, h, i]),  # noqa: E731
                                 0 if math.isnan(weights[b, h, i]) else 1, i)
                stay = sorted(sorted(range(old), key=key)[:m - (n - old)] + list(range(old, n)))
            kept[b, h, :m] = torch.tensor(stay, dtype=torch.int32)
            out[b, h, :m] = weights[b, h, stay]
    return kept, torch.tensor(lens, dtype=torch.int32), out


def move_rows(cache, block_table, kept, kv_lens, budget):
    """The pool after eviction: row kept[b, h, j] of each head at slot j (a copy, on the CPU)."""
    old, new = cache.detach().cpu(), cache.detach().cpu().clone()
    page = cache.shape[1]
    for b, n in enumerate(kv_lens.tolist()):
        for h in range(cache.shape[2]):
            for j in range(min(n, budget)):
                i = int(kept[b, h, j])
                new[int(block_table[b, j // page]), j % page, h] = old[int(block_table[b, i // page]), i % page, h]
    return new
