"""The serving-cache operators and the query/key norm with rotation, as measured cases.

`listed()` names the cases, `draw()` gives more of the same ranges, `prepare()` makes a case's
inputs on the GPU, `run()` makes one pass (in plain torch, or through the library where `own` is
set), `work()` counts what a pass cannot do without and `exact()` computes it in 64 bits.

Operators:
  norm_rope      RMS norm of queries and keys for each head, then the position rotation; the cases
                 with op "append" are its form where a cache is kept: q out, k and v into their pages
  norm_rope_bwd  its gradients: of q, k and the two norm weights
  chunk          attention of each sequence's new tokens over its paged cache
  key_weights    attention weight that each cached key received, added up
  evict          keep the keys of most weight and the latest ones, close up the pages
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # training step's forward at 8192 tokens of 32 heads of 128, every head with its own keys
        dict(name="norm_rope 8192x32x128", op="norm_rope", tokens=8192, hq=32, hkv=32, d=128, rot=128, interleaved=False,
             fused=False, dtype="bf16"),
        # its backward
        dict(name="norm_rope_bwd 8192x32x128", op="norm_rope_bwd", tokens=8192, hq=32, hkv=32, d=128, rot=128,
             interleaved=False, fused=False, dtype="bf16"),
        # backward of an odd batch read out of one fused projection, partly rotated, neighbouring pairs
        dict(name="norm_rope_bwd 1733x12x64", op="norm_rope_bwd", tokens=1733, hq=12, hkv=4, d=64, rot=32,
             interleaved=True, fused=True, dtype="fp16"),
        # one serving step of 64 sequences: a token each, straight into the pages (launch latency)
        dict(name="append 64x1", op="append", batch=64, new=1, ragged=False, length=500, hq=32, hkv=8, d=128, rot=128,
             interleaved=False, page=64, dtype="bf16"),
        # single tokens of a few short sequences (latency)
        dict(name="chunk 4x1 over 1000", op="chunk", batch=4, new=1, length=1000, ragged=True, hq=16, hkv=16, d=128,
             page=16, causal=True, dtype="bf16"),
        # a serving step: single tokens of 64 sequences up to 8192 long, four queries to a key head
        dict(name="chunk 64x1 over 8192", op="chunk", batch=64, new=1, length=8192, ragged=True, hq=32, hkv=8, d=128,
             page=64, causal=True, dtype="bf16"),
        # a long prompt in chunks: the last 2048 tokens of 8192
        dict(name="chunk 1x2048 over 8192", op="chunk", batch=1, new=2048, length=8192, ragged=False, hq=32, hkv=8,
             d=128, page=128, causal=True, dtype="bf16"),
        # odd chunks of nine sequences, no shared heads, small pages
        dict(name="chunk 9x333 over 2777", op="chunk", batch=9, new=333, length=2777, ragged=True, hq=12, hkv=12, d=64,
             page=16, causal=True, dtype="fp16"),
        # the serving step's weights, key by key
        dict(name="key_weights 64x1 over 8192", op="key_weights", batch=64, new=1, length=8192, ragged=True, hq=32,
             hkv=8, d=128, page=64, causal=True, dtype="bf16"),
        # a prompt chunk's weights
        dict(name="key_weights 2x777 over 3333", op="key_weights", batch=2, new=777, length=3333, ragged=True, hq=16,
             hkv=4, d=64, page=32, causal=True, dtype="fp16"),
        # sixteen long sequences cut down to 2048 keys a head
        dict(name="evict 16x8192 to 2048", op="evict", batch=16, length=8192, ragged=True, hkv=8, d=128, page=64,
             budget=2048, recent=256, dtype="bf16"),
        # three short ones, small pages (latency)
        dict(name="evict 3x777 to 300", op="evict", batch=3, length=777, ragged=True, hkv=12, d=64, page=16,
             budget=300, recent=32, dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_bwd", "append", "chunk", "chunk", "chunk", "key_weights", "evict"])
    d = rng.choice([32, 64, 64, 128, 128, 128, 256])
    hkv = rng.choice([1, 2, 3, 4, 8, 12, 16])
    group = rng.choice([1, 1, 2, 3, 4, 5, 8])
    dtype = rng.choice(["fp16", "bf16"])
    c = dict(op=op, hkv=hkv, d=d, dtype=dtype)
    rot = rng.choice([r for r in (16, 32, 64, 128, 256) if r <= d] + [d, d])
    if op in ("norm_rope", "norm_rope_bwd"):
        c.update(tokens=_log(rng, 1, max(2, 8192 * 64 * 128 // (d * hkv * (group + 1)) // 2)), hq=hkv * group, rot=rot,
                 interleaved=rng.random() < 0.5, fused=rng.random() < 0.5)
        c["tokens"] = min(c["tokens"], 8192)
        return c
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "evict":
        batch = _log(rng, 1, 16)
        length = _log(rng, 40, 8192)
        budget = max(2, int(length * rng.uniform(0.1, 0.9)))
        c.update(batch=batch, length=length, ragged=rng.random() < 0.7, page=page, budget=budget,
                 recent=rng.randint(0, budget), hkv=min(hkv, 8))
        return c
    batch = _log(rng, 1, 64)
    new = rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 17, 1024)])
    # scores, and keys and values, stay below those of the largest listed cases
    new = max(1, min(new, int(3e8 / (batch * hkv * group)) // 1024))
    most = min(8192, int(4e8 / (d * hkv * batch)), int(3e8 / (batch * new * hkv * group)))
    length = max(new, _log(rng, 1, max(2, most)))
    c.update(batch=batch, new=new, length=length, ragged=rng.random() < 0.7, hq=hkv * group, page=page)
    if op == "append":
        c.update(length=min(length, new + 300), rot=rot, interleaved=rng.random() < 0.5)
    else:
        c.update(causal=rng.random() < 0.8)
    return c


def _spread(most, least, n, ragged, turn):
    """n lengths up to `most`, the first the longest: all the same, or spread over three quarters."""
    return [max(least, int(round(most * (1 - (0.75 * ((i * turn) % 1.0) if ragged else 0.0))))) for i in range(n)]


def _lengths(c):
    new = _spread(c["new"], 1, c["batch"], c["ragged"], 0.7548776662)
    kv = _spread(c["length"], 1, c["batch"], c["ragged"], 0.6180339887)
    return new, [max(k, n) for k, n in zip(kv, new)]


# ----------------------------------------------------------------------------- inputs
def _randn(g, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(scale).to(dtype)


def _angles(g, rows, rot):
    inv = 10000.0 ** (-torch.arange(0, rot // 2, device="cuda", dtype=torch.float64) * 2 / rot)
    a = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def _pages(g, c, lengths, more=0):
    page = c["page"]
    need = [-(-n // page) for n in lengths]
    cols = max(need) + more
    total = sum(need) + 3
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    start = torch.tensor([sum(need[:i]) for i in range(len(need))], device="cuda")[:, None]
    col = torch.arange(cols, device="cuda")[None, :]
    there = col < torch.tensor(need, device="cuda")[:, None]
    table = torch.where(there, order[(start + col).clamp(max=total - 1)], torch.full((), -1, device="cuda", dtype=torch.int32))
    return total, table.contiguous()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt, d, hkv = DTYPES[c["dtype"]], c["d"], c["hkv"]
    s = dict(case=c, op=c["op"])
    i32 = lambda v: torch.tensor(v, device="cuda", dtype=torch.int32)  # noqa: E731
    if c["op"] in ("norm_rope", "norm_rope_bwd"):
        n, hq = c["tokens"], c["hq"]
        if c["fused"]:
            qkv = _randn(g, (n, hq + 2 * hkv, d), dt, 2.0)
            s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hkv]
        else:
            s["q"], s["k"] = _randn(g, (n, hq, d), dt, 2.0), _randn(g, (n, hkv, d), dt, 2.0)
        s["wq"] = (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt)
        s["wk"] = (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt)
        s["table"] = _angles(g, 8192, c["rot"])
        s["positions"] = torch.randint(0, 8192, (n,), generator=g, device="cuda")
        if c["op"] == "norm_rope_bwd":
            s["dq_out"], s["dk_out"] = _randn(g, (n, hq, d), dt), _randn(g, (n, hkv, d), dt)
        return s
    if c["op"] == "evict":
        kv = _spread(c["length"], 1, c["batch"], c["ragged"], 0.6180339887)
        total, s["block_table"] = _pages(g, c, kv)
        s["width"] = s["block_table"].shape[1] * c["page"]
        s["kv_lens"], s["longest"] = i32(kv), max(kv)
        s["weights"] = torch.exp(1.5 * torch.randn(c["batch"], hkv, s["width"], generator=g, device="cuda"))
        s["k_cache"] = _randn(g, (total, c["page"], hkv, d), dt)
        s["v_cache"] = _randn(g, (total, c["page"], hkv, d), dt)
        return s
    new, kv = _lengths(c)
    hq = c["hq"]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    total, s["block_table"] = _pages(g, c, kv, 1)
    s["cu_seqlens"], s["kv_lens"], s["most_new"], s["longest"] = i32(cu), i32(kv), max(new), max(kv)
    s["k_cache"] = _randn(g, (total, c["page"], hkv, d), dt)
    s["v_cache"] = _randn(g, (total, c["page"], hkv, d), dt)
    s["q"] = _randn(g, (cu[-1], hq, d), dt)
    if c["op"] == "append":
        s["k"], s["v"] = _randn(g, (cu[-1], hkv, d), dt, 2.0), _randn(g, (cu[-1], hkv, d), dt)
        s["wq"] = (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt)
        s["wk"] = (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt)
        s["table"] = _angles(g, 8192, c["rot"])
        s["positions"] = torch.randint(0, 8192, (cu[-1],), generator=g, device="cuda")
    if c["op"] == "key_weights":
        s["lse"] = _plain_chunk(s)[1]
        s["weights"] = torch.rand(c["batch"], hkv, s["block_table"].shape[1] * c["page"], generator=g, device="cuda")
    return s


# ----------------------------------------------------------------------------- plain forms
def _rotate(x, table, positions, rot, interleaved, back=False):
    """x (n, heads, d): the first `rot` values turned by each token's angles (back: the other way)."""
    cs = table[positions][:, None, :]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    sin = -sin if back else sin
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rot:]], -1)


EPS = 1e-6


def _plain_norm_rope(x, w, s):
    x32 = x.float()
    x32 = x32 * torch.rsqrt(x32.square().mean(-1, keepdim=True) + EPS) * w.float()
    return _rotate(x32, s["table"], s["positions"], s["case"]["rot"], s["case"]["interleaved"]).to(x.dtype)


def _plain_norm_rope_bwd(x, w, dy, s):
    x32 = x.float()
    r = torch.rsqrt(x32.square().mean(-1, keepdim=True) + EPS)
    g = _rotate(dy.float(), s["table"], s["positions"], s["case"]["rot"], s["case"]["interleaved"], back=True)
    xhat = x32 * r
    gw = g * w.float()
    dx = r * (gw - xhat * (gw * xhat).mean(-1, keepdim=True))
    return dx.to(x.dtype), (g * xhat).sum((0, 1))


def _rows_of_keys(s, longest):
    j = torch.arange(longest, device="cuda")
    page = s["case"]["page"]
    return (s["block_table"].long().clamp(min=0)[:, j // page] * page + j % page)  # (batch, longest)


def _plain_append(s):
    q = _plain_norm_rope(s["q"], s["wq"], s)
    k = _plain_norm_rope(s["k"], s["wk"], s)
    n = q.shape[0]
    r = torch.arange(n, device="cuda")
    cu = s["cu_seqlens"].long()
    b = torch.searchsorted(cu, r, right=True) - 1
    slot = s["kv_lens"].long()[b] - cu[b + 1] + r
    page = s["case"]["page"]
    row = s["block_table"].long()[b, slot // page] * page + slot % page
    s["k_cache"].flatten(0, 1).index_copy_(0, row, k)
    s["v_cache"].flatten(0, 1).index_copy_(0, row, s["v"])
    return q, s["k_cache"], s["v_cache"]


def _plain_scores(s):
    """scores (batch, hkv, rows, longest) with -inf where a row sees nothing, the rows being
    (new token, head of the group), and each packed token's place in them."""
    c = s["case"]
    hkv, d, group = c["hkv"], c["d"], c["hq"] // c["hkv"]
    cu, kv = s["cu_seqlens"].long(), s["kv_lens"].long()
    i = torch.arange(s["most_new"], device="cuda")
    j = torch.arange(s["longest"], device="cuda")
    tok = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[tok].unflatten(2, (hkv, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    rows = _rows_of_keys(s, s["longest"])
    k = s["k_cache"].flatten(0, 1)[rows].float().permute(0, 2, 3, 1)
    scores = torch.matmul(q, k) / math.sqrt(d)
    n = (cu[1:] - cu[:-1])[:, None]
    last = (kv[:, None] - n + i + 1) if c["causal"] else kv[:, None].expand(-1, s["most_new"])
    last = torch.where(i < n, last, torch.zeros_like(last))
    seen = (j < last[..., None]).repeat_interleave(group, 1)[:, None]
    return scores.masked_fill_(~seen, float("-inf")), rows


def _packed(x, s):
    """(batch, hkv, rows, w) back to (tokens, hq, w)."""
    cu = s["cu_seqlens"].long()
    r = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(cu, r, right=True) - 1
    x = x.unflatten(2, (s["most_new"], -1)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    return x[b, r - cu[b]]


def _plain_chunk(s):
    scores, rows = _plain_scores(s)
    m = scores.amax(-1, keepdim=True)
    m0 = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = scores.sub_(m0).exp_()
    total = p.sum(-1, keepdim=True)
    v = s["v_cache"].flatten(0, 1)[rows].float().permute(0, 2, 1, 3)
    out = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = m0 + total.log()
    return _packed(out, s).to(s["q"].dtype), _packed(lse, s)[..., 0].t().contiguous()


def _plain_key_weights(s):
    scores, _ = _plain_scores(s)
    hkv, group = s["case"]["hkv"], s["case"]["hq"] // s["case"]["hkv"]
    cu = s["cu_seqlens"].long()
    tok = (cu[:-1, None] + torch.arange(s["most_new"], device="cuda")).clamp(max=s["q"].shape[0] - 1)
    lse = s["lse"].t()[tok].unflatten(2, (hkv, group)).permute(0, 2, 1, 3).flatten(2, 3)[..., None]
    p = torch.where(torch.isinf(lse), torch.zeros_like(scores), scores.sub_(lse).exp_())
    s["weights"][..., :s["longest"]] += p.sum(2)
    return s["weights"]


def _plain_evict(s):
    c = s["case"]
    page, budget, recent, width = c["page"], c["budget"], c["recent"], s["width"]
    kv = s["kv_lens"].long()[:, None, None]
    j = torch.arange(width, device="cuda")
    late = (j >= kv - recent) & (j < kv)
    key = torch.where(late, torch.full((), float("inf"), device="cuda"), s["weights"])
    key = torch.where(j < kv, key, torch.full((), -1.0, device="cuda"))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :budget]
    order = torch.where(torch.arange(order.shape[-1], device="cuda") < kv, order, torch.full_like(order, width))
    kept = order.sort(-1).values
    new = torch.minimum(s["kv_lens"], torch.full_like(s["kv_lens"], budget))
    live = kept < width
    src = torch.where(live, kept, torch.zeros_like(kept))
    weights = torch.zeros_like(s["weights"])
    weights[..., :kept.shape[-1]] = torch.where(live, s["weights"].gather(-1, src), torch.zeros_like(weights[..., :1]))
    bt = s["block_table"].long().clamp(min=0)
    b = torch.arange(c["batch"], device="cuda")[:, None, None]
    h = torch.arange(c["hkv"], device="cuda")[None, :, None]
    to = torch.arange(kept.shape[-1], device="cuda").expand_as(kept)
    to = torch.where(live, to, torch.zeros_like(to))  # a slot that is not kept copies slot 0's key on itself
    first = torch.where(live, src, kept[..., :1].expand_as(src))
    from_row, to_row = bt[b, first // page] * page + first % page, bt[b, to // page] * page + to % page
    kf, vf = s["k_cache"].flatten(0, 1), s["v_cache"].flatten(0, 1)
    k, v = kf[from_row, h], vf[from_row, h]
    kf[to_row, h] = k
    vf[to_row, h] = v
    kept = torch.where(live, kept, torch.full_like(kept, -1)).int()
    return torch.nn.functional.pad(kept, (0, budget - kept.shape[-1]), value=-1), new, weights, s["k_cache"], s["v_cache"]


def run(state):
    s, op = state, state["op"]
    c = s["case"]
    if own:
        import tiled_exact_attention_fwd_b200 as fa
        if op == "norm_rope":
            return fa.fa_qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["table"], s["positions"], eps=EPS,
                                      interleaved=c["interleaved"])
        if op == "norm_rope_bwd":
            return fa.fa_qk_norm_rope_bwd(s["q"], s["k"], s["wq"], s["wk"], s["table"], s["positions"], s["dq_out"],
                                          s["dk_out"], eps=EPS, interleaved=c["interleaved"])
        if op == "append":
            q = fa.fa_qk_norm_rope_paged(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["table"], s["positions"],
                                         s["k_cache"], s["v_cache"], s["block_table"], s["cu_seqlens"], s["kv_lens"],
                                         eps=EPS, interleaved=c["interleaved"])
            return q, s["k_cache"], s["v_cache"]
        if op == "chunk":
            return fa.fa_fwd_paged_chunk(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["cu_seqlens"],
                                         s["kv_lens"], s["most_new"], causal=c["causal"])
        if op == "key_weights":
            return fa.fa_paged_key_weights(s["q"], s["k_cache"], s["block_table"], s["cu_seqlens"], s["kv_lens"],
                                           s["most_new"], s["lse"], s["weights"], causal=c["causal"])
        kept, new, weights = fa.fa_paged_evict(s["k_cache"], s["v_cache"], s["block_table"], s["kv_lens"], s["weights"],
                                               c["budget"], c["recent"])
        return kept, new, weights, s["k_cache"], s["v_cache"]
    if op == "norm_rope":
        return _plain_norm_rope(s["q"], s["wq"], s), _plain_norm_rope(s["k"], s["wk"], s)
    if op == "norm_rope_bwd":
        dq, dwq = _plain_norm_rope_bwd(s["q"], s["wq"], s["dq_out"], s)
        dk, dwk = _plain_norm_rope_bwd(s["k"], s["wk"], s["dk_out"], s)
        return dq, dk, dwq, dwk
    if op == "append":
        return _plain_append(s)
    if op == "chunk":
        return _plain_chunk(s)
    if op == "key_weights":
        return _plain_key_weights(s)
    return _plain_evict(s)


# ----------------------------------------------------------------------------- work
def work(case):
    c, d, hkv = case, case["d"], case["hkv"]
    row = 2 * d  # bytes of one head of one token
    if c["op"] in ("norm_rope", "norm_rope_bwd"):
        n, heads = c["tokens"], c["hq"] + hkv
        moved = 2 if c["op"] == "norm_rope" else 3
        per = 5 if c["op"] == "norm_rope" else 14
        return {"bytes": n * (heads * row * moved + 4 * c["rot"] + 8) + 4 * row, "flops": per * n * heads * d}
    if c["op"] == "evict":
        kv = _spread(c["length"], 1, c["batch"], c["ragged"], 0.6180339887)
        # what has to move: of the keys that stay, those that change places (all but the share
        # that chance leaves in place), read and written once; the weights read and written
        moved = sum(c["budget"] for n in kv if n > c["budget"])
        return {"bytes": hkv * (moved * 2 * 2 * row + sum(4 * n + 8 * min(n, c["budget"]) for n in kv)), "flops": hkv * sum(kv)}
    new, kv = _lengths(c)
    tokens, hq = sum(new), c["hq"]
    if c["op"] == "append":
        return {"bytes": tokens * ((hq + 2 * hkv) * row * 2 + 4 * c["rot"] + 8), "flops": 5 * tokens * (hq + hkv) * d}
    pairs = sum(n * k - (n * (n - 1) // 2 if c["causal"] else 0) for n, k in zip(new, kv))
    if c["op"] == "chunk":
        return {"bytes": tokens * hq * (2 * row + 4) + sum(kv) * hkv * 2 * row, "flops": 4 * pairs * hq * d}
    return {"bytes": tokens * hq * (row + 4) + sum(kv) * hkv * (row + 8), "flops": 2 * pairs * hq * d}


# ----------------------------------------------------------------------------- in 64 bits
def _exact_turn(x, s, sign):
    """Each pair (a, b) as the complex number a + ib times e^(i sign angle), in 64 bits."""
    rot, n = s["case"]["rot"], x.shape[0]
    half = rot // 2
    cs = s["table"][s["positions"]].double()
    turn = torch.complex(cs[:, :half], sign * cs[:, half:]).reshape(n, 1, half)
    head = x[..., :rot]
    if s["case"]["interleaved"]:
        z = torch.view_as_complex(head.reshape(n, -1, half, 2).contiguous()) * turn
        y = torch.view_as_real(z).reshape(n, -1, rot)
    else:
        z = torch.complex(head[..., :half].contiguous(), head[..., half:].contiguous()) * turn
        y = torch.cat((z.real, z.imag), 2)
    return torch.cat((y, x[..., rot:]), 2)


def _exact_norm(x, w, s):
    x = x.double()
    y = x / (x.pow(2).sum(2, keepdim=True) / x.shape[2] + EPS).sqrt() * w.double()
    return _exact_turn(y, s, 1.0)


def _exact_norm_bwd(x, w, dy, s):
    x, w = x.double(), w.double()
    d = x.shape[2]
    g = _exact_turn(dy.double(), s, -1.0)
    root = (x.pow(2).sum(2, keepdim=True) / d + EPS).sqrt()
    # d/dx_i of sum_j g_j w_j x_j / root: g_i w_i / root - x_i sum_j g_j w_j x_j / (d root^3)
    dx = g * w / root - x * (g * w * x).sum(2, keepdim=True) / (d * root.pow(3))
    return dx, (g * x / root).reshape(-1, d).sum(0)


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    d, hkv = c["d"], c["hkv"]
    if op == "norm_rope":
        return _exact_norm(s["q"], s["wq"], s), _exact_norm(s["k"], s["wk"], s)
    if op == "norm_rope_bwd":
        dq, dwq = _exact_norm_bwd(s["q"], s["wq"], s["dq_out"], s)
        dk, dwk = _exact_norm_bwd(s["k"], s["wk"], s["dk_out"], s)
        return dq, dk, dwq, dwk
    page, kv = c["page"], s["kv_lens"].tolist()
    bt = s["block_table"].long()
    if op == "evict":
        w, kc, vc = s["weights"].double(), s["k_cache"].double(), s["v_cache"].double()
        kept = torch.full((c["batch"], hkv, c["budget"]), -1, dtype=torch.int32, device="cuda")
        out_w = torch.zeros_like(w)
        for b, n in enumerate(kv):
            m = min(n, c["budget"])
            rows = (bt[b, :-(-n // page), None] * page + torch.arange(page, device="cuda")).flatten()[:n]
            for h in range(hkv):
                old = n - min(n, c["recent"])
                best = torch.sort(-w[b, h, :old], stable=True).indices[:m - (n - old)]
                stay = torch.cat([best, torch.arange(old, n, device="cuda")]).sort().values
                kept[b, h, :m] = stay.int()
                out_w[b, h, :m] = w[b, h, stay]
                for pool in (kc, vc):
                    flat = pool.flatten(0, 1)
                    flat[rows[:m], h] = flat[rows[stay], h].clone()
        return kept, s["kv_lens"].clamp(max=c["budget"]), out_w, kc, vc
    new = (s["cu_seqlens"][1:] - s["cu_seqlens"][:-1]).tolist()
    cu = s["cu_seqlens"].tolist()
    if op == "append":
        q, k = _exact_norm(s["q"], s["wq"], s), _exact_norm(s["k"], s["wk"], s)
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        for b, n in enumerate(new):
            slots = torch.arange(kv[b] - n, kv[b], device="cuda")
            rows = bt[b, slots // page]
            kc[rows, slots % page] = k[cu[b]:cu[b + 1]]
            vc[rows, slots % page] = s["v"][cu[b]:cu[b + 1]].double()
        return q, kc, vc
    group = c["hq"] // hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros((c["hq"], s["q"].shape[0]), dtype=torch.float64, device="cuda")
    weights = s["weights"].double() if op == "key_weights" else None
    for b, n in enumerate(new):
        at = slice(cu[b], cu[b + 1])
        pages = bt[b, :-(-kv[b] // page)]
        k = s["k_cache"][pages].flatten(0, 1)[:kv[b]].double()
        v = s["v_cache"][pages].flatten(0, 1)[:kv[b]].double()
        seen = torch.ones(n, kv[b], dtype=torch.bool, device="cuda")
        if c["causal"]:
            seen = torch.tril(seen, diagonal=kv[b] - n)
        for h in range(c["hq"]):
            z = s["q"][at, h].double() @ k[:, h // group].t() * d ** -0.5
            z = torch.where(seen, z, torch.full((), -math.inf, dtype=z.dtype, device="cuda"))
            if op == "key_weights":
                weights[b, h // group, :kv[b]] += torch.exp(z - s["lse"][h, at, None].double()).sum(0)
            else:
                lse[h, at] = torch.logsumexp(z, 1)
                out[at, h] = torch.softmax(z, 1) @ v[:, h // group]
    return weights if op == "key_weights" else (out, lse)
