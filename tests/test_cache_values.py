"""The operators around a paged cache on values that the draws of test_cache_ops.py do not hold, against
the same definitions in 64 bits and with its tolerances: NaN and infinities in what a row sees, scores that grow
along the keys, other scales; results in place; calls beside one another."""
import math

import pytest
import torch

import fa_inputs
from oracle import cache as oc
from test_cache_ops import CHUNK, DT, U, angles, chunk_inputs, half_step, norm_inputs, on, pools, round_tol, same, score_tol, within


def check(dev, q, kc, vc, bt, cu, lens, max_q, dt, causal=True, scale=None):
    """Attention and key weights against their definitions (test_cache_ops.py derives the tolerances)."""
    import tiled_exact_attention_fwd_b200 as fa
    args = [t.to(dev) for t in (q, kc, vc, bt, cu, lens)]
    out, lse = fa.fa_fwd_paged_chunk(*args, max_q, causal=causal, scale=scale)
    ref, rl, size, ssize = oc.chunk_attention(q, kc, vc, bt, cu, lens, causal=causal, scale=scale)
    e = score_tol(ssize)
    w = torch.zeros(len(lens), kc.shape[2], bt.shape[1] * kc.shape[1], device=dev)
    fa.fa_paged_key_weights(args[0], args[1], *args[3:], max_q, lse, w, causal=causal, scale=scale)
    add, most = oc.key_weights(q, kc, bt, cu, lens, lse.cpu(), w.shape[2], causal=causal, scale=scale)
    assert fa.fa_device_status()[0] == 0
    within(out, ref, half_step(dt) * ref.abs() + (half_step(dt) + 2 * e.t()[..., None]) * size + 2.0 ** -25, "out")
    within(lse, rl, e + 2.0 ** -23 * rl.abs(), "lse")
    # A row's weight below fp32's smallest normal number, 2^-126 = 1.18e-38, counts as 0 (2.4e-40 of a sum of 6.0e-38 goes
    # so): a sum loses at most that much for each of its rows, which no tolerance relative to the sum covers.
    flushed = max_q * (q.shape[1] // kc.shape[2]) * 2.0 ** -126
    within(w, add, (2.0 ** -19 * (most + 1) + 1024 * U) * add + flushed, "weights")
    return out, lse, w


# Sequences, new tokens of each, keys of each. One sequence: each step (64 or 128 keys) is a run of its own, so every
# item is cut at every step. Many: runs of several items, most of them whole.
LAYOUTS = {"cut": (1, 900), "whole": (100, 150)}


@pytest.mark.gpu
@pytest.mark.parametrize("few", [True, False])
@pytest.mark.parametrize("layout", ["cut", "whole"])
@pytest.mark.parametrize("D", [32, 64, 128, 256])
def test_key_weights_of_rows_without_a_finite_lse(cuda_device, D, layout, few):
    """A row whose lse is NaN makes the weights of the keys that it sees NaN, and of no other key; one whose lse is -inf
    gives nothing, but NaN where its score is (a NaN query: all keys that it sees)."""
    import tiled_exact_attention_fwd_b200 as fa
    count, kv = LAYOUTS[layout]
    n = 1 if few else 20
    dtype = "bf16" if D > 64 else "fp16"
    q, kc, vc, bt, cu, lens = chunk_inputs([n] * count, [kv] * count, 6, 3, D, 16, dtype, 7 + D, behind=0)
    _, lse, _, _ = oc.chunk_attention(q, kc, vc, bt, cu, lens)
    lse = lse.float()
    lse[1, n // 3::n] = math.nan
    lse[0, n // 2::n] = lse[3, n // 2::n] = lse[5, n // 4::n] = -math.inf
    q[n // 4::n, 5] = math.nan
    w = torch.zeros(count, 3, bt.shape[1] * 16, device=cuda_device)
    fa.fa_paged_key_weights(*(t.to(cuda_device) for t in (q, kc, bt, cu, lens)), n, lse.to(cuda_device), w)
    add, most = oc.key_weights(q, kc, bt, cu, lens, lse, w.shape[2])
    add[:, 2, :kv - n + n // 4 + 1] = math.nan
    nan = torch.isnan(add)
    seen = kv - n + n // 3 + 1  # keys of the row whose lse is NaN
    assert bool(nan[:, 0, :seen].all()) and not bool(nan[:, 0, seen:].any()) and not bool(nan[:, 1].any())
    within(w, add, (2.0 ** -19 * (most + 1) + 1024 * U) * add, "weights")
    assert fa.fa_device_status()[0] == 0


@pytest.mark.gpu
@pytest.mark.parametrize("few", [True, False])
@pytest.mark.parametrize("layout", ["cut", "whole"])
@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("where", ["query", "keys", "last key"])
def test_nan_stays_nan(cuda_device, where, D, layout, few):
    """NaN in one row of each sequence, in a run of keys of one key head (a whole step of the split), or in the
    last key of one key head: NaN in every row that sees it and in the weights of the keys that such a row
    sees, whether the split cuts its item or not, and in nothing else."""
    count, kv = LAYOUTS[layout]
    n = 1 if few else 20
    dtype = "bf16" if D > 64 else "fp16"
    q, kc, vc, bt, cu, lens = chunk_inputs([n] * count, [kv] * count, 4, 2, D, 16, dtype, 3 + D, behind=0)
    if where == "query":
        q[n // 2::n, 1] = math.nan
    else:
        first, end = {"keys": (128, 256) if layout == "cut" else (64, 128), "last key": (kv - 1, kv)}[where]
        for b in range(count):
            for i in range(first, end):
                kc[bt[b, i // 16], i % 16, 1] = math.nan
    out, lse, w = check(cuda_device, q, kc, vc, bt, cu, lens, n, DT[dtype])
    rows = torch.isnan(lse.t()).cpu()  # (token, head)
    want = torch.zeros_like(rows)
    if where == "query":
        want[n // 2::n, 1] = True
    elif where == "keys":
        want[:, 2:] = True
    else:
        want[n - 1::n, 2:] = True
    assert torch.equal(rows, want) and torch.equal(torch.isnan(out).all(-1).cpu(), want) and torch.equal(torch.isnan(out).any(-1).cpu(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("few", [True, False])
@pytest.mark.parametrize("layout", ["cut", "whole"])
@pytest.mark.parametrize("D", [64, 128])
def test_infinite_scores(cuda_device, D, layout, few):
    """One infinite value in a key: its score is +inf for some rows (NaN, as a softmax over it is) and -inf for the
    others, for which the key is as if it were not there."""
    import tiled_exact_attention_fwd_b200 as fa
    dev, dt = cuda_device, torch.bfloat16
    count, kv = LAYOUTS[layout]
    n, at = 1 if few else 20, 70
    q, kc, vc, bt, cu, lens = chunk_inputs([n] * count, [kv] * count, 4, 2, D, 16, "bf16", 5 + D, behind=0)
    for b in range(count):
        kc[bt[b, at // 16], at % 16, :, 0] = math.inf
    args = [t.to(dev) for t in (q, kc, vc, bt, cu, lens)]
    out, lse = fa.fa_fwd_paged_chunk(*args, n)
    ref, rl, size, _ = oc.chunk_attention(q, kc, vc, bt, cu, lens)
    _, _, _, ssize = oc.chunk_attention(q, torch.where(kc.isinf(), torch.zeros_like(kc), kc), vc, bt, cu, lens)
    up = (q[..., 0] > 0)  # (token, head): score +inf
    assert bool((q[..., 0] != 0).all()) and bool((~up).any())  # (4 rows may all be of one sign)
    assert torch.equal(torch.isnan(out).all(-1).cpu(), up) and torch.equal(torch.isnan(lse.t()).cpu(), up)
    e = score_tol(ssize)
    tol = half_step(dt) * ref.abs() + (half_step(dt) + 2 * e.t()[..., None]) * size
    within(out.cpu()[~up], ref[~up], tol[~up], "out")
    within(lse.t().cpu()[~up], rl.t()[~up], (e + 2.0 ** -23 * rl.abs()).t()[~up], "lse")
    w = torch.zeros(count, 2, bt.shape[1] * 16, device=dev)
    fa.fa_paged_key_weights(args[0], args[1], *args[3:], n, lse, w)
    add, most = oc.key_weights(q, torch.where(kc.isinf(), torch.zeros_like(kc), kc), bt, cu, lens, lse.cpu(), w.shape[2])
    add[..., at] = torch.where(torch.isnan(add[..., at]), add[..., at], torch.zeros(()).double())
    within(w, add, (2.0 ** -19 * (most + 1) + 1024 * U) * add, "weights")
    assert fa.fa_device_status()[0] == 0


@pytest.mark.gpu
@pytest.mark.parametrize("new", [[1, 1], [20, 3]])
def test_infinite_values(cuda_device, new):
    """An infinite value in a column of V that every row sees: that column is infinite, the others as they are."""
    q, kc, vc, bt, cu, lens = chunk_inputs(new, [300, 40], 4, 2, 64, 16, "bf16", 8, behind=0)
    for b in range(2):
        vc[bt[b, 0], 5, 1, 7] = math.inf
    out, _, _ = check(cuda_device, q, kc, vc, bt, cu, lens, max(new), torch.bfloat16)
    assert bool((out[:, 2:, 7] == math.inf).all()) and int(torch.isinf(out).sum()) == 2 * sum(new)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hk,D,behind", [(4, 2, 64, 3), (3, 1, 256, 40), (32, 8, 128, 700)])
def test_append_with_rows_of_no_sequence(cuda_device, hq, hk, D, behind):
    """Rows behind the last sequence may hold any position: nothing of theirs is written or reported; a token of a
    sequence whose position is outside the table still is."""
    import tiled_exact_attention_fwd_b200 as fa
    dev, new, kv, page = cuda_device, [3, 0, 1, 5], [20, 7, 1, 64], 16
    total = sum(new)
    q, k, v, wq, wk, cs, pos = norm_inputs(total + behind, hq, hk, D, D, torch.bfloat16, torch.bfloat16, True, 9)
    pos[total:] = torch.tensor([-1, 1 << 40, 97, -(1 << 62)]).repeat(behind)[:behind]
    _, _, bt = pools(kv, page, hk, D, torch.bfloat16, 6)
    kc, vc = (torch.full((sum(-(-n // page) for n in kv) + 2, page, hk, D), 3.0, dtype=torch.bfloat16, device=dev) for _ in range(2))
    cu = fa_inputs.cu_seqlens_from_lengths(new)
    lens = torch.tensor(kv, dtype=torch.int32)
    for bad in (False, True):
        if bad:
            pos[total - 1] = 97
        out = torch.full((total + behind, hq, D), 7.0, dtype=torch.bfloat16, device=dev)
        fa.fa_qk_norm_rope_paged(on(dev, q), on(dev, k), on(dev, v), wq.to(dev), wk.to(dev), cs.to(dev), pos.to(dev), kc, vc,
                                 bt.to(dev), cu.to(dev), lens.to(dev), q_out=out)
        assert fa.fa_device_status()[0] == (-8 if bad else 0)
        live = total - int(bad)
        ref, size = oc.norm_rope(q[:live], wq, cs, pos[:live], 1e-6, False)
        within(out[:live], ref, round_tol(ref, size, torch.bfloat16, 32), "q")
        assert bool((out[total:] == 7.0).all())
        for pool in (kc, vc):
            assert int((pool != 3.0).any(-1).any(-1).sum()) == total  # the tokens' rows, and no others


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,hq,hk,D,rot,dtype,inter", [
    (1, 2, 1, 32, 32, "bf16", False), (37, 5, 2, 64, 48, "fp16", True), (700, 16, 4, 128, 128, "bf16", False),
    (2100, 3, 3, 256, 64, "bf16", True)])
def test_norm_results_in_place_and_between_one_another(cuda_device, tokens, hq, hk, D, rot, dtype, inter):
    """Results as columns of one buffer, gradients over what they are formed from, through the C entries: the bits of dense
    results, and nothing between them touched."""
    import tiled_exact_attention_fwd_b200 as fa
    dev, dt, lib = cuda_device, DT[dtype], fa.lib()
    q, k, v, wq, wk, cs, pos = norm_inputs(tokens, hq, hk, D, rot, dt, dt, True, 13)
    wq, wk, cs, pos = (t.to(dev) for t in (wq, wk, cs, pos))
    cols = hq + 2 * hk

    def fused(a, b):  # views like norm_inputs' fused ones, the last columns 9
        x = torch.full((tokens, cols, D), 9.0, dtype=dt, device=dev)
        x[:, :hq], x[:, hq:hq + hk] = a, b
        return x, x[:, :hq], x[:, hq:hq + hk]

    _, fq, fk = fused(q.to(dev), k.to(dev))
    gq, gk = fa_inputs.normal((tokens, hq, D), dt, 91).to(dev), fa_inputs.normal((tokens, hk, D), dt, 92).to(dev)
    yq, yk = fa.fa_qk_norm_rope(fq, fk, wq, wk, cs, pos, eps=1e-5, interleaved=inter)
    buf, oq, ok = fused(torch.zeros_like(gq), torch.zeros_like(gk))
    fa.fa_qk_norm_rope(fq, fk, wq, wk, cs, pos, eps=1e-5, interleaved=inter, q_out=oq, k_out=ok)
    assert torch.equal(oq, yq) and torch.equal(ok, yk) and bool((buf[:, hq + hk:] == 9).all())
    want = fa.fa_qk_norm_rope_bwd(fq, fk, wq, wk, cs, pos, gq, gk, eps=1e-5, interleaved=inter)
    ws = torch.empty(lib.fa_qk_norm_rope_bwd_workspace(D), dtype=torch.uint8, device=dev)

    def call(xq, xk, dyq, dyk, dq, dk):
        dw = torch.full((2, D), float("nan"), device=dev)
        st = lib.fa_qk_norm_rope_bwd(
            xq.data_ptr(), xq.stride(0), xk.data_ptr(), xk.stride(0), wq.data_ptr(), wk.data_ptr(), 0, cs.data_ptr(), cs.shape[0],
            rot, pos.data_ptr(), dyq.data_ptr(), dyq.stride(0), dyk.data_ptr(), dyk.stride(0), dq.data_ptr(), dq.stride(0),
            dk.data_ptr(), dk.stride(0), dw[0].data_ptr(), dw[1].data_ptr(), ws.data_ptr(), ws.numel(), tokens, hq, hk, D, 1e-5,
            int(inter), int(dtype == "bf16"), torch.cuda.current_stream().cuda_stream)
        assert st == 0
        for got, ref in zip((dq, dk, dw[0], dw[1]), want):
            assert torch.equal(got, ref)

    buf, oq, ok = fused(torch.zeros_like(gq), torch.zeros_like(gk))
    call(fq, fk, gq, gk, oq, ok)  # columns of a buffer
    assert bool((buf[:, hq + hk:] == 9).all())
    buf, oq, ok = fused(gq, gk)
    call(fq, fk, oq, ok, oq, ok)  # over the gradients that come in
    assert bool((buf[:, hq + hk:] == 9).all())
    buf, oq, ok = fused(q.to(dev), k.to(dev))
    call(oq, ok, gq, gk, oq, ok)  # over q and k
    assert bool((buf[:, hq + hk:] == 9).all())
    assert fa.fa_device_status()[0] == 0


@pytest.mark.gpu
@pytest.mark.parametrize("budget,recent", [(2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (65, 0), (0, 0), (-1, 0), (-2 ** 31, 0), (4, 5), (4, -1)])
def test_evict_refuses_its_numbers_before_it_allocates(cuda_device, budget, recent):
    """(8 * 8 heads of 2^31 kept slots would be 550 GB.)"""
    import tiled_exact_attention_fwd_b200 as fa
    dev = cuda_device
    kc, vc = (torch.zeros(32, 16, 8, 32, dtype=torch.bfloat16, device=dev) for _ in range(2))
    bt = torch.arange(32, dtype=torch.int32, device=dev).view(8, 4)
    lens = torch.full((8,), 20, dtype=torch.int32, device=dev)
    with pytest.raises(fa.FAError) as e:
        fa.fa_paged_evict(kc, vc, bt, lens, torch.zeros(8, 8, 64, device=dev), budget, recent)
    assert e.value.status == -2


# Rows of a step kernel: single tokens; two row tiles of an item (one at D = 256); one, whose key tiles two warpgroups share.
GROWING = {"few": (1, 4, 2), "two tiles": (130, 2, 2), "one tile": (20, 8, 2)}


def growing_inputs(kind, D, count=64, kv=1000):
    """Sequences over one another's pages whose key j is larger by 2.2 for every 128 keys before it: the largest score of a
    window of 128 keys then grows by about the 8 (in log2 units) from which on the running maximum moves."""
    n, hq, hk = GROWING[kind]
    q, kc, vc, bt, _, _ = chunk_inputs([n] * count, [kv], hq, hk, D, 16, "bf16", 19 + D, behind=0)
    for j in range(kv):
        kc[bt[0, j // 16], j % 16] *= 1 + 2.2 * (j // 128)
    cu = fa_inputs.cu_seqlens_from_lengths([n] * count)
    return q, kc, vc, bt.expand(count, -1).contiguous(), cu, torch.tensor([kv - 3 * b for b in range(count)], dtype=torch.int32), n


@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("kind", list(GROWING))
def test_growing_inputs_grow(kind, D):
    """In every window but the first, some rows' largest score is more than 8 over all that came before, and some rows' is
    not: such a row moves its maximum there wherever the split began its run. And a run holds several steps: there are
    more than 4 times as many (of up to 128 keys) as SMs."""
    n, hq, hk = GROWING[kind]
    q, kc, _, bt, _, lens, _ = growing_inputs(kind, D)
    k = oc.token_rows(kc, bt, 0, 1000)
    z = torch.einsum("thd,khd->thk", q.double(), k.repeat_interleave(hq // hk, 1)) * math.log2(math.e) / math.sqrt(D)
    z = torch.nn.functional.pad(z[..., :int(lens[-1]) - n], (0, -(int(lens[-1]) - n) % 128), value=-math.inf)  # keys that all rows see
    most = z.view(*z.shape[:2], -1, 128).amax(-1)
    moves = most[..., 1:] > most.cummax(-1).values[..., :-1] + 8
    share = moves.double().mean((0, 1))[:5]  # of the rows, in each whole window
    assert bool((share > 0.05).all()) and bool((share < 0.95).all())
    if kind != "few":  # 32 rows of a warp: some move, some do not
        warps = moves[..., :5].reshape(-1, 5)[:moves.shape[0] * hq // 32 * 32].view(-1, 32, 5)
        assert bool((warps.any(1) & ~warps.all(1)).double().mean() > 0.5)
    assert len(lens) * hk * (int(lens[-1]) // 128) > 4 * 148


@pytest.mark.gpu
@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("kind", list(GROWING))
def test_growing_scores(cuda_device, kind, D):
    """O and the sums rescaled while the steps run."""
    *args, n = growing_inputs(kind, D)
    check(cuda_device, *args, n, torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.3, 1.0])
@pytest.mark.parametrize("case", [CHUNK[i] for i in (0, 2, 4, 7, 8, 9, 11, 12, 15, 18)])
def test_scale(cuda_device, case, scale):
    new, kv, hq, hk, D, page, dtype, causal = case
    inputs = chunk_inputs(new, kv, hq, hk, D, page, dtype, 27 + sum(kv), behind=0)
    check(cuda_device, *inputs, max(new), DT[dtype], causal=causal, scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,hq,hk,D", [(3000, 8, 2, 128), (40, 4, 4, 64)])
def test_gradients_replayed_while_eager_calls_run(cuda_device, tokens, hq, hk, D):
    """A captured backward replayed on one stream while eager ones run on two others, many of them in flight."""
    import tiled_exact_attention_fwd_b200 as fa
    q, k, v, wq, wk, cs, pos = (None if t is None else on(cuda_device, t) for t in
                                norm_inputs(tokens, hq, hk, D, D, torch.bfloat16, torch.bfloat16, True, 3))
    grads = [(torch.randn_like(q), torch.randn_like(k)) for _ in range(3)]
    wants = [fa.fa_qk_norm_rope_bwd(q, k, wq, wk, cs, pos, *g) for g in grads]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fa.fa_qk_norm_rope_bwd(q, k, wq, wk, cs, pos, *grads[0])
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    eager, kept = [], []
    for _ in range(25):
        with torch.cuda.stream(streams[0]):
            graph.replay()
            kept.append([t.clone() for t in got])
        for i in (1, 2):
            with torch.cuda.stream(streams[i]):
                eager.append((i, fa.fa_qk_norm_rope_bwd(q, k, wq, wk, cs, pos, *grads[i])))
    torch.cuda.synchronize()
    assert all(same(t, wants[0]) for t in kept) and all(same(t, wants[i]) for i, t in eager)


@pytest.mark.gpu
@pytest.mark.parametrize("few", [True, False])
def test_replayed_over_other_lengths(cuda_device, few):
    """A captured step (append, attention, weights, eviction) replayed after the lengths, the offsets and the table have been
    changed in place, with sequences that left the batch: the bits of eager calls, rows of no sequence as they were."""
    import tiled_exact_attention_fwd_b200 as fa
    dev, B, cols, page, hq, hk, D = cuda_device, 6, 40, 16, 8, 2, 64
    total = 6 if few else 200
    g = fa_inputs.generator(3)
    x = [fa_inputs.normal((total, h, D), torch.bfloat16, 40 + h).to(dev) for h in (hq, hk, hk)]
    pools0 = [torch.randn(B * cols, page, hk, D, generator=g).bfloat16().to(dev) for _ in range(2)]
    kc, vc = (t.clone() for t in pools0)
    bt = torch.arange(B * cols, dtype=torch.int32, device=dev).view(B, cols).contiguous()
    cu, lens = torch.zeros(B + 1, dtype=torch.int32, device=dev), torch.zeros(B, dtype=torch.int32, device=dev)
    cs, q, out = angles(cols * page, D).to(dev), torch.empty_like(x[0]), torch.empty_like(x[0])
    lse, w = torch.empty(hq, total, device=dev), torch.empty(B, hk, cols * page, device=dev)

    def reset():
        kc.copy_(pools0[0]), vc.copy_(pools0[1]), w.zero_()
        for t in (q, out, lse):
            t.fill_(7.0)

    def step():
        fa.fa_qk_norm_rope_paged(*x, None, None, cs, None, kc, vc, bt, cu, lens, q_out=q)
        fa.fa_fwd_paged_chunk(q, kc, vc, bt, cu, lens, 1 if few else 150, out=out, lse=lse)
        fa.fa_paged_key_weights(q, kc, bt, cu, lens, 1 if few else 150, lse, w)
        return fa.fa_paged_evict(kc, vc, bt, lens, w, 300, 40)

    new = [[1, 1, 1, 1, 1, 1], [1, 0, 1, 1, 0, 0], [0] * 6] if few else [[50, 1, 0, 149, 0, 0], [150, 0, 1, 1, 20, 3], [0, 0, 0, 0, 0, 7]]
    kv = [[100, 640, 1, 320, 17, 400], [640, 5, 555, 2, 0, 301], [640] * 6] if few else [[600, 1, 30, 640, 0, 9], [150, 640, 400, 2, 90, 33], [640] * 6]

    def lay(i):
        cu.copy_(fa_inputs.cu_seqlens_from_lengths(new[i])), lens.copy_(torch.tensor(kv[i], dtype=torch.int32))
        bt.copy_(torch.randperm(B * cols, generator=fa_inputs.generator(i)).view(B, cols).int())
        reset()

    lay(0)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        results = step()
    for i in (1, 2, 0):
        lay(i)
        want = [t.clone() for t in (*step(), q, out, lse, w, kc, vc)]
        reset()
        graph.replay()
        assert same(want, [*results, q, out, lse, w, kc, vc])
        live = sum(new[i])
        assert all(bool((t[live:] == 7.0).all()) for t in (q, out, lse.t()))
    assert fa.fa_device_status()[0] == 0


@pytest.mark.gpu
@pytest.mark.parametrize("wtype", [torch.float32, torch.bfloat16])
def test_weights_of_one_of_the_two(cuda_device, wtype):
    import tiled_exact_attention_fwd_b200 as fa
    dev, dt = cuda_device, torch.bfloat16
    q, k, v, wq, wk, cs, pos = norm_inputs(50, 4, 2, 64, 64, dt, wtype, False, 3)
    gq, gk = fa_inputs.normal(q.shape, dt, 1), fa_inputs.normal(k.shape, dt, 2)
    for a, b in ((wq, None), (None, wk)):
        args = [on(dev, t) for t in (q, k, a, b, cs, pos)]
        for got, x, w in zip(fa.fa_qk_norm_rope(*args), (q, k), (a, b)):
            ref, size = oc.norm_rope(x, w, cs, pos, 1e-6, False)
            within(got, ref, round_tol(ref, size, dt, 32), "norm_rope")
        got = fa.fa_qk_norm_rope_bwd(*args, gq.to(dev), gk.to(dev), stream=0)  # (stream 0: the default one)
        for x, w, dy, dx, dw in ((q, a, gq, got[0], got[2]), (k, b, gk, got[1], got[3])):
            rx, rw, sx, sw = oc.norm_rope_bwd(x, w, cs, pos, dy, 1e-6, False)
            within(dx, rx, round_tol(rx, sx, dt, 64), "dx")
            assert (dw is None) == (w is None)
            if w is not None:
                within(dw, rw, 97 * U * sw, "dw")
    assert fa.fa_device_status()[0] == 0


@pytest.mark.gpu
@pytest.mark.parametrize("new", [1, 20])
def test_longest_cache(cuda_device, new):
    """2^31 - 2^20 keys, all pages one page of 2^20: the attention of that page, 2047 times its sum; each key's
    weight a 2047th. (The new tokens see all keys, so every position up to the last counts.)"""
    import tiled_exact_attention_fwd_b200 as fa
    dev, page, pages, D = cuda_device, 1 << 20, 2047, 32
    kc, vc = (fa_inputs.normal((1, page, 1, D), torch.bfloat16, s).to(dev) for s in (1, 2))
    vc += 1
    q = fa_inputs.normal((new, 2, D), torch.bfloat16, 3).to(dev)
    bt = torch.zeros(1, pages, dtype=torch.int32, device=dev)
    cu, lens = torch.tensor([0, new], dtype=torch.int32, device=dev), torch.tensor([page * pages], dtype=torch.int32, device=dev)
    out, lse = fa.fa_fwd_paged_chunk(q, kc, vc, bt, cu, lens, new, causal=False)
    z = torch.einsum("thd,kd->thk", q.double(), kc[0, :, 0].double()) / math.sqrt(D)
    rl, p = torch.logsumexp(z, -1), torch.softmax(z, -1)
    v = vc[0, :, 0].double()
    ref, size = p @ v, p @ v.abs()
    # A CTA's run is 2^31 / 148 keys, 113 thousand steps of 128; each adds up to 8 times (16 keys an MMA) to a sum of 32 bits,
    # and an MMA may cut what does not fit instead of rounding it: 2^-23 each at most
    long = 2 ** 31 / 128 / 148 * 8 * 2 * U
    e = 2.0 ** -20 * (z.abs().amax() + 1) * 8
    within(out, ref.cpu(), (half_step(torch.bfloat16) * (ref.abs() + size) + (2 * e + 2 * long) * size).cpu(), "out")
    within(lse, (rl + math.log(pages)).t().cpu(), (e + long + 2.0 ** -20).cpu().expand(2, new), "lse")
    w = torch.zeros(1, 1, page * pages, device=dev)
    fa.fa_paged_key_weights(q, kc, bt, cu, lens, new, lse, w, causal=False)
    each = (p.sum((0, 1)) / pages)  # of a page's keys
    for i in (0, 1, 1023, 2045, 2046):
        got = w[0, 0, i * page:(i + 1) * page].double()
        assert bool(((got - each).abs() <= each * (2 * e + 2 * long)).all())
    assert bool((w != 0).all()) and fa.fa_device_status()[0] == 0


@pytest.mark.gpu
@pytest.mark.parametrize("new", [[1, 1, 1], [30, 1, 7]])
def test_pools_of_one_buffer(cuda_device, new):
    """K and V pages by turns in one buffer, the two pools a page apart: the bits of pools of their own."""
    import tiled_exact_attention_fwd_b200 as fa
    dev, page, hq, hk, D, kv = cuda_device, 16, 4, 2, 64, [100, 40, 33]
    total = sum(new)
    x = [fa_inputs.normal((total, h, D), torch.bfloat16, 40 + h).to(dev) for h in (hq, hk, hk)]
    both = torch.randn(24, 2, page, hk, D, generator=fa_inputs.generator(1)).bfloat16().to(dev)
    bt = torch.randperm(24, generator=fa_inputs.generator(2)).view(3, 8).int().to(dev)
    cu, lens = fa_inputs.cu_seqlens_from_lengths(new).to(dev), torch.tensor(kv, dtype=torch.int32, device=dev)
    cs, pages = angles(128, D).to(dev), both.flatten(0, 1)
    seen = []
    for kc, vc, table in ((both[:, 0].contiguous(), both[:, 1].contiguous(), bt), (pages[:-1], pages[1:], 2 * bt)):
        w = torch.zeros(3, hk, 8 * page, device=dev)
        q = fa.fa_qk_norm_rope_paged(*x, None, None, cs, None, kc, vc, table, cu, lens)
        out, lse = fa.fa_fwd_paged_chunk(q, kc, vc, table, cu, lens, max(new))
        fa.fa_paged_key_weights(q, kc, table, cu, lens, max(new), lse, w)
        res = fa.fa_paged_evict(kc, vc, table, lens, w, 30, 5)
        pools = (kc, vc) if kc.shape[0] == 24 else (both[:, 0], both[:, 1])
        seen.append([t.clone() for t in (q, out, lse, w, *res, *pools)])
    assert same(*seen) and fa.fa_device_status()[0] == 0
