"""The operators around a paged cache against their definitions in 64 bits (oracle/cache.py): norm of
queries and keys with the position rotation and its gradients, the append, attention of new tokens,
key weights, eviction, and a run of them together.

Tolerances. An output of type t is rounded once: eps_t / 2 of its value (plus half of fp16's smallest
step). Before that everything is fp32: a norm's row takes about 20 roundings of 2^-24 on its terms
(sum of squares by lanes and shuffles, square root, reciprocal, two products, a sum), so 32 * 2^-24 of
the terms' size; gradients twice that. Attention rounds each weight of the second product once
(eps_t / 2 of sum p |v|), and a score's error moves its weight by as much: fp32 sums of D products are
taken to 2^-20 of the terms' size (the exponent's own rounding, 2^-24 of at most 2^4 scores, and the
approximate exp2, 2^-22, are inside it), once for the weight and once for the sum."""
import math

import pytest
import torch

import fa_inputs
from oracle import cache as oc

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24


def half_step(t):
    return torch.finfo(t).eps / 2


def within(got, ref, tol, what):
    got = got.detach().cpu().double()
    same = (got == ref) | (torch.isnan(got) & torch.isnan(ref))  # infinities and NaN where the definition has them
    bad = ~same & ~((got - ref).abs() <= tol)
    if bad.any():
        i = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: {float(got[i])} for "
                             f"{float(ref[i])}, {float((got - ref).abs()[i]):.3e} over {float(tol.expand_as(ref)[i]):.3e}")


def round_tol(ref, size, dtype, units):
    return half_step(dtype) * ref.abs() + units * U * size + (2.0 ** -25 if dtype == torch.float16 else 0.0)


def angles(rows, rot, seed=0):
    inv = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)
    a = torch.arange(rows, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def weights_of(D, dtype, seed):
    return (1 + 0.3 * torch.randn(D, generator=fa_inputs.generator(seed))).to(dtype)


# --------------------------------------------------------------------------- the definitions themselves
@pytest.mark.parametrize("interleaved", [False, True])
def test_definition_of_the_norm_gradient_is_the_derivative(interleaved):
    x = fa_inputs.normal((3, 2, 32), torch.float64, 1)
    w = weights_of(32, torch.float64, 2)
    dy = fa_inputs.normal((3, 2, 32), torch.float64, 3)
    cs, pos = angles(50, 16), torch.tensor([0, 7, 49])
    dx, dw, _, _ = oc.norm_rope_bwd(x, w, cs, pos, dy, 1e-6, interleaved)
    f = lambda x, w: float((oc.norm_rope(x, w, cs, pos, 1e-6, interleaved)[0] * dy).sum())  # noqa: E731
    h = 1e-6
    for i in [(0, 0, 0), (1, 1, 5), (2, 0, 31), (2, 1, 16)]:
        e = torch.zeros_like(x)
        e[i] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - float(dx[i])) < 1e-7 * max(1, abs(float(dx[i])))
    for i in (0, 9, 31):
        e = torch.zeros_like(w)
        e[i] = h
        assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - float(dw[i])) < 1e-7 * max(1, abs(float(dw[i])))


def test_definition_of_chunk_attention_is_dense_attention():
    import oracle
    q, k, v = fa_inputs.dense_qkv(1, 40, 2, 32, torch.float16, seed=3)
    kc, vc, bt = fa_inputs.paged_kv(k, v, 16, seed=4)
    O, L = oracle.attention_dense(q, k, v, causal=True)
    out, lse, _, _ = oc.chunk_attention(q[0, 25:], kc, vc, bt, torch.tensor([0, 15]), torch.tensor([40]))
    assert (out - torch.from_numpy(O[0, 25:])).abs().max() < 1e-12
    assert (lse - torch.from_numpy(L[0, :, 25:])).abs().max() < 1e-12


def test_definition_of_key_weights_sums_to_the_rows():
    q, k, v = fa_inputs.dense_qkv(1, 33, 2, 32, torch.float32, seed=5)
    kc, vc, bt = fa_inputs.paged_kv(k[:, :, :1].contiguous(), v[:, :, :1].contiguous(), 16, seed=6)
    cu, kv = torch.tensor([0, 9]), torch.tensor([33])
    _, lse, _, _ = oc.chunk_attention(q[0, :9], kc, vc, bt, cu, kv)
    add, _ = oc.key_weights(q[0, :9], kc, bt, cu, kv, lse, 48)
    assert abs(float(add.sum()) - 18) < 1e-10 and float(add[..., 33:].abs().sum()) == 0


def test_definition_of_eviction():
    w = torch.tensor([[[5.0, 1, 5, 0, 2, 2, 9, 9]]])
    kept, lens, nw = oc.evict(w, torch.tensor([7]), 4, 2)
    assert kept.tolist() == [[[0, 2, 5, 6]]] and lens.tolist() == [4] and nw.tolist() == [[[5, 5, 2, 9, 0, 0, 0, 0]]]


# --------------------------------------------------------------------------- refusals (no GPU needed)
class TestRefusals:
    @pytest.fixture(scope="class")
    def lib(self):
        from tiled_exact_attention_fwd_b200 import build
        build.build()
        import tiled_exact_attention_fwd_b200 as fa
        return fa.lib()

    # 16-byte aligned addresses that are never read: every call below is refused on the host
    P = 4096

    def norm(self, lib, **kw):
        a = dict(q=self.P, qs=256, k=self.P, ks=128, wq=None, wk=None, w32=0, cs=self.P, rows=64, rot=64, pos=self.P,
                 qo=self.P, qos=256, ko=self.P, kos=128, n=4, hq=4, hk=2, d=64, eps=1e-6, inter=0, dt=1)
        a.update(kw)
        return lib.fa_qk_norm_rope(*a.values(), None)

    @pytest.mark.parametrize("change,status", [
        (dict(dt=2), -3), (dict(d=96), -4), (dict(n=-1), -2), (dict(hq=0), -2), (dict(hk=-3), -2), (dict(rot=0), -2),
        (dict(rot=24), -2), (dict(rot=128), -2), (dict(rows=0), -2), (dict(eps=-1.0), -2), (dict(eps=math.nan), -2),
        (dict(eps=math.inf), -2), (dict(q=None), -1), (dict(cs=None), -1), (dict(pos=None), -1), (dict(qo=None), -1),
        (dict(q=4104), -5), (dict(ko=4097), -5), (dict(pos=4100), -5), (dict(wq=4104), -5), (dict(qs=248), -5),
        (dict(kos=132), -5), (dict(n=0), 0)])
    def test_norm(self, lib, change, status):
        assert self.norm(lib, **change) == status

    def bwd(self, lib, **kw):
        a = dict(q=self.P, qs=256, k=self.P, ks=128, wq=None, wk=None, w32=0, cs=self.P, rows=64, rot=64, pos=self.P,
                 dqo=self.P, dqos=256, dko=self.P, dkos=128, dq=self.P, dqs=256, dk=self.P, dks=128, dwq=self.P, dwk=self.P,
                 ws=self.P, wsb=1 << 30, n=4, hq=4, hk=2, d=64, eps=1e-6, inter=0, dt=1)
        a.update(kw)
        return lib.fa_qk_norm_rope_bwd(*a.values(), None)

    @pytest.mark.parametrize("change,status", [
        (dict(dt=2), -3), (dict(d=48), -4), (dict(rot=8), -2), (dict(dqo=None), -1), (dict(dk=None), -1),
        (dict(ws=None), -1), (dict(wsb=100), -2), (dict(dqs=4), -5), (dict(dkos=129), -5), (dict(dwq=4097), -5),
        (dict(ws=4100), -5), (dict(n=0, dwq=None, dwk=None), 0)])
    def test_bwd(self, lib, change, status):
        assert self.bwd(lib, **change) == status

    def paged(self, lib, **kw):
        a = dict(q=self.P, qs=256, k=self.P, ks=128, v=self.P, vs=128, wq=None, wk=None, w32=0, cs=self.P, rows=64, rot=64,
                 pos=None, qo=self.P, qos=256, kc=self.P, vc=self.P, bt=self.P, mb=4, page=16, pages=9, cu=self.P, kv=self.P,
                 num=2, n=4, hq=4, hk=2, d=64, eps=1e-6, inter=0, dt=1)
        a.update(kw)
        return lib.fa_qk_norm_rope_paged(*a.values(), None)

    @pytest.mark.parametrize("change,status", [
        (dict(page=8), -2), (dict(page=48), -2), (dict(page=1 << 21), -2), (dict(pages=0), -2), (dict(mb=0), -2),
        (dict(pages=1 << 28), -2), (dict(num=-1), -2), (dict(v=None), -1), (dict(bt=None), -1), (dict(cu=None), -1),
        (dict(kv=None), -1), (dict(kc=4104), -5), (dict(bt=4098), -5), (dict(vs=64), -5), (dict(num=0), 0), (dict(n=0), 0)])
    def test_paged(self, lib, change, status):
        assert self.paged(lib, **change) == status

    def chunk(self, lib, **kw):
        a = dict(q=self.P, kc=self.P, vc=self.P, bt=self.P, mb=4, page=16, pages=9, cu=self.P, kv=self.P, num=2, total=4,
                 mq=2, out=self.P, lse=self.P, ws=self.P, wsb=1 << 40, hq=4, hk=2, d=64, scale=0.0, causal=1, dt=0)
        a.update(kw)
        return lib.fa_fwd_paged_chunk(*a.values(), None)

    @pytest.mark.parametrize("change,status", [
        (dict(dt=5), -3), (dict(d=80), -4), (dict(hq=5), -2), (dict(hk=0), -2), (dict(num=-1), -2), (dict(total=-1), -2),
        (dict(mq=-1), -2), (dict(total=1 << 30), -2), (dict(page=24), -2), (dict(q=None), -1), (dict(vc=None), -1),
        (dict(out=None), -1), (dict(ws=None), -1), (dict(wsb=1000), -2), (dict(ws=4096 + 16), -5), (dict(q=4100), -5),
        (dict(lse=4097), -5), (dict(kv=4097), -5), (dict(total=0), 0), (dict(num=0), 0)])
    def test_chunk(self, lib, change, status):
        assert self.chunk(lib, **change) == status

    def test_chunk_workspace(self, lib):
        assert lib.fa_fwd_paged_chunk_workspace(4, 2, 64, 1) > 0
        for bad in [(5, 2, 64, 1), (129, 1, 64, 1), (4, 0, 64, 1), (4, 2, 65, 1), (4, 2, 64, -1)]:
            assert lib.fa_fwd_paged_chunk_workspace(*bad) == 0 and lib.fa_paged_key_weights_workspace(*bad) == 0

    def keys(self, lib, **kw):
        a = dict(q=self.P, kc=self.P, bt=self.P, mb=4, page=16, pages=9, cu=self.P, kv=self.P, num=2, total=4, mq=2,
                 lse=self.P, w=self.P, width=64, ws=self.P, wsb=1 << 30, hq=4, hk=2, d=64, scale=0.0, causal=1, dt=0)
        a.update(kw)
        return lib.fa_paged_key_weights(*a.values(), None)

    @pytest.mark.parametrize("change,status", [
        (dict(dt=5), -3), (dict(d=80), -4), (dict(hq=3), -2), (dict(width=63), -2), (dict(lse=None), -1), (dict(w=None), -1),
        (dict(w=4097), -5), (dict(kc=4100), -5), (dict(mq=9, ws=None), -1), (dict(mq=9, wsb=1000), -2),
        (dict(mq=9, ws=4096 + 16), -5), (dict(total=0), 0)])
    def test_key_weights(self, lib, change, status):
        assert self.keys(lib, **change) == status

    def evict(self, lib, **kw):
        a = dict(kc=self.P, vc=self.P, bt=self.P, mb=4, page=16, pages=9, kv=self.P, w=self.P, width=64, budget=8, recent=2,
                 kept=self.P, nl=2 * self.P, nw=2 * self.P, b=2, hk=2, d=64, dt=0)
        a.update(kw)
        return lib.fa_paged_evict(*a.values(), None)

    @pytest.mark.parametrize("change,status", [
        (dict(dt=2), -3), (dict(d=16), -4), (dict(budget=0), -2), (dict(budget=65), -2), (dict(recent=9), -2),
        (dict(recent=-1), -2), (dict(width=60), -2), (dict(hk=0), -2), (dict(b=-1), -2), (dict(kept=None), -1),
        (dict(vc=None), -1), (dict(kc=4104), -5), (dict(nw=4096), -2), (dict(nl=4096), -2), (dict(nl=8194), -5),
        (dict(b=0), 0)])
    def test_evict(self, lib, change, status):
        assert self.evict(lib, **change) == status

    # the inputs at 1 << 20 (weights: 2 * 2 * 64 * 4 = 1024 bytes) and 1 << 21 (lengths: 8 bytes)
    @pytest.mark.parametrize("change", [
        dict(nw=(1 << 20) + 1020), dict(nw=(1 << 20) - 1020), dict(kept=(1 << 20) + 512), dict(kept=(1 << 20) - 124),
        dict(nl=(1 << 20) + 4), dict(nl=(1 << 21) + 4), dict(kept=(1 << 21) - 4), dict(nw=(1 << 21) - 1000),
        dict(width=(1 << 31) - 1, mb=1 << 26)])
    def test_evict_overlaps(self, lib, change):
        a = dict(w=1 << 20, kv=1 << 21, kept=1 << 22, nl=1 << 23, nw=1 << 24)
        a.update(change)
        assert self.evict(lib, **a) == -2


# --------------------------------------------------------------------------- norm and rotation
def norm_inputs(tokens, hq, hk, D, rot, dtype, wtype, fused, seed):
    if fused:
        x = fa_inputs.normal((tokens, hq + 2 * hk, D), dtype, seed)
        q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    else:
        q, k, v = (fa_inputs.normal((tokens, h, D), dtype, seed + i) for i, h in enumerate((hq, hk, hk)))
    wq = None if wtype is None else weights_of(D, wtype, seed + 5)
    wk = None if wtype is None else weights_of(D, wtype, seed + 6)
    pos = torch.randint(0, 97, (tokens,), generator=fa_inputs.generator(seed + 7))
    return q, k, v, wq, wk, angles(97, rot), pos


def on(dev, t):
    if t is None:
        return None
    if t.is_contiguous():
        return t.to(dev)
    base = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device=dev)
    base.copy_(t)
    return base


NORM = [  # tokens, hq, hk, D, rot, dtype, weights, interleaved, fused
    (1, 1, 1, 32, 32, "bf16", "same", False, False),
    (5, 3, 1, 32, 16, "fp16", "fp32", True, True),
    (7, 8, 8, 64, 64, "bf16", None, False, True),
    (33, 5, 5, 64, 32, "fp16", "same", False, False),
    (19, 4, 2, 64, 48, "bf16", "fp32", True, False),
    (61, 9, 3, 128, 128, "bf16", "same", False, True),
    (17, 16, 2, 128, 128, "fp16", "same", True, False),
    (40, 7, 7, 128, 16, "fp16", None, False, False),
    (13, 6, 3, 256, 256, "bf16", "fp32", False, False),
    (9, 2, 1, 256, 64, "fp16", "same", True, True),
    (700, 12, 4, 64, 64, "bf16", "same", False, False),
    # more batches than warps, a part of a batch at the end of each token
    (6001, 5, 1, 32, 32, "bf16", "same", False, False),
    (1501, 17, 3, 128, 64, "fp16", "fp32", True, True),
    (2100, 1, 9, 256, 256, "bf16", "same", False, False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,hq,hk,D,rot,dtype,wtype,inter,fused", NORM)
def test_norm_rope(cuda_device, tokens, hq, hk, D, rot, dtype, wtype, inter, fused):
    import tiled_exact_attention_fwd_b200 as fa
    dt = DT[dtype]
    wt = {"same": dt, "fp32": torch.float32, None: None}[wtype]
    q, k, v, wq, wk, cs, pos = norm_inputs(tokens, hq, hk, D, rot, dt, wt, fused, 11 + tokens)
    if tokens > 3:
        q[1], k[2] = 0, 0  # rows of zeros: 0 / sqrt(eps)
    dq, dk = on(cuda_device, q), on(cuda_device, k)
    args = [on(cuda_device, t) for t in (wq, wk, cs, pos)]
    yq, yk = fa.fa_qk_norm_rope(dq, dk, *args, eps=1e-5, interleaved=inter)
    for got, x, w in ((yq, q, wq), (yk, k, wk)):
        ref, size = oc.norm_rope(x, w, cs, pos, 1e-5, inter)
        within(got, ref, round_tol(ref, size, dt, 32), "norm_rope")
    # in place, and as (batch, length, heads, D)
    fa.fa_qk_norm_rope(dq, dk, *args, eps=1e-5, interleaved=inter, q_out=dq, k_out=dk)
    assert torch.equal(dq, yq) and torch.equal(dk, yk)
    assert fa.fa_device_status()[0] == 0


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,hq,hk,D,rot,dtype,wtype,inter,fused", NORM)
def test_norm_rope_bwd(cuda_device, tokens, hq, hk, D, rot, dtype, wtype, inter, fused):
    import tiled_exact_attention_fwd_b200 as fa
    dt = DT[dtype]
    wt = {"same": dt, "fp32": torch.float32, None: None}[wtype]
    q, k, v, wq, wk, cs, pos = norm_inputs(tokens, hq, hk, D, rot, dt, wt, fused, 31 + tokens)
    gq, gk = fa_inputs.normal((tokens, hq, D), dt, 91), fa_inputs.normal((tokens, hk, D), dt, 92)
    dev = [on(cuda_device, t) for t in (q, k, wq, wk, cs, pos, gq, gk)]
    got = fa.fa_qk_norm_rope_bwd(*dev, eps=1e-5, interleaved=inter)
    for x, w, g, dx, dw in ((q, wq, gq, got[0], got[2]), (k, wk, gk, got[1], got[3])):
        rx, rw, sx, sw = oc.norm_rope_bwd(x, w, cs, pos, g, 1e-5, inter)
        within(dx, rx, round_tol(rx, sx, dt, 64), "dx")
        if w is None:
            assert dw is None
        else:  # each sum takes at most tokens * heads / 256 + 30 roundings one after another, of partial sums
            assert dw.dtype == torch.float32
            within(dw, rw, (96 + tokens * max(hq, hk) / 256) * U * sw, "dw")
    again = fa.fa_qk_norm_rope_bwd(*dev, eps=1e-5, interleaved=inter)
    for a, b in zip(got, again):
        assert a is None or torch.equal(a, b)
    assert fa.fa_device_status()[0] == 0


@pytest.mark.gpu
def test_norm_rope_shapes_and_errors(cuda_device):
    import tiled_exact_attention_fwd_b200 as fa
    dev = cuda_device
    q, k, v, wq, wk, cs, pos = norm_inputs(12, 4, 2, 64, 64, torch.bfloat16, torch.bfloat16, False, 3)
    q, k, wq, wk, cs, pos = (t.to(dev) for t in (q, k, wq, wk, cs, pos))
    a = fa.fa_qk_norm_rope(q, k, wq, wk, cs, pos)
    b = fa.fa_qk_norm_rope(q.view(3, 4, 4, 64), k.view(3, 4, 2, 64), wq, wk, cs, pos.view(3, 4))
    assert b[0].shape == (3, 4, 4, 64) and torch.equal(a[0], b[0].view_as(a[0])) and torch.equal(a[1], b[1].view_as(a[1]))
    e = fa.fa_qk_norm_rope(q[:0], k[:0], wq, wk, cs, pos[:0])
    assert e[0].shape == (0, 4, 64)
    g = fa.fa_qk_norm_rope_bwd(q[:0], k[:0], wq, wk, cs, pos[:0], q[:0], k[:0])
    assert float(g[2].abs().sum() + g[3].abs().sum()) == 0
    # a position outside the table: reported, the other tokens as they are
    bad = pos.clone()
    bad[3], bad[5] = 97, -1
    c = fa.fa_qk_norm_rope(q, k, wq, wk, cs, bad)
    assert fa.fa_device_status()[0] == -8
    ok = [i for i in range(12) if i not in (3, 5)]
    assert torch.equal(c[0][ok], a[0][ok])
    with pytest.raises(ValueError):
        fa.fa_qk_norm_rope(q, k, wq[:32], wk, cs, pos)
    with pytest.raises(ValueError):
        fa.fa_qk_norm_rope(q, k, wq, wk.float(), cs, pos)
    with pytest.raises(ValueError):
        fa.fa_qk_norm_rope(q, k, wq, wk, cs.half(), pos)
    with pytest.raises(ValueError):
        fa.fa_qk_norm_rope(q, k, wq, wk, cs, pos.int())
    with pytest.raises(ValueError):
        fa.fa_qk_norm_rope(q.transpose(0, 1), k.transpose(0, 1), wq, wk, cs, pos)
    with pytest.raises(ValueError):
        fa.fa_qk_norm_rope(q, k, wq, wk, cs, pos, q_out=q[:6])
    with pytest.raises(fa.FAError):
        fa.fa_qk_norm_rope(q, k, wq, wk, cs[:, :24].contiguous(), pos)


# --------------------------------------------------------------------------- a paged cache
def pools(lengths, page, hk, D, dtype, seed, fill=float("nan")):
    """Pages in a random order with `fill` in every row that holds no key; the table's unused entries
    are out of range on purpose (never read)."""
    g = fa_inputs.generator(seed)
    need = [-(-n // page) for n in lengths]
    total = sum(need) + 2
    order = torch.randperm(total, generator=g).to(torch.int32)
    table = torch.full((len(lengths), max(need + [1]) + 1), 1 << 30, dtype=torch.int32)
    kc = torch.full((total, page, hk, D), fill, dtype=dtype)
    vc = kc.clone()
    at = 0
    for b, n in enumerate(lengths):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        for i in range(n):
            kc[table[b, i // page], i % page] = torch.randn(hk, D, generator=g).to(dtype)
            vc[table[b, i // page], i % page] = torch.randn(hk, D, generator=g).to(dtype)
    return kc, vc, table


@pytest.mark.gpu
@pytest.mark.parametrize("new,kv,hq,hk,D,rot,page,dtype,inter,slots", [
    ([1], [1], 1, 1, 32, 32, 16, "bf16", False, True),
    ([1, 1, 1], [17, 16, 40], 8, 2, 128, 128, 16, "bf16", False, False),
    ([5, 0, 33, 1], [5, 9, 70, 64], 6, 3, 64, 32, 32, "fp16", True, True),
    ([20, 3], [20, 90], 4, 4, 256, 256, 64, "bf16", False, False),
])
def test_append(cuda_device, new, kv, hq, hk, D, rot, page, dtype, inter, slots):
    import tiled_exact_attention_fwd_b200 as fa
    dt = DT[dtype]
    total = sum(new)
    behind = 3  # rows of no sequence
    q, k, v, wq, wk, cs, pos = norm_inputs(total + behind, hq, hk, D, rot, dt, dt, True, 5)
    kc, vc, bt = pools(kv, page, hk, D, dt, 6)
    bt_ok = torch.where(bt < kc.shape[0], bt, torch.zeros_like(bt))
    cu = fa_inputs.cu_seqlens_from_lengths(new)
    lens = torch.tensor(kv, dtype=torch.int32)
    slot = torch.cat([torch.arange(m - n, m) for n, m in zip(new, kv)] + [torch.zeros(behind, dtype=torch.int64)])
    if slots:
        pos = slot
    want_k, want_v = kc.clone(), vc.clone()
    tol_k = torch.zeros(kc.shape, dtype=torch.float64)
    ref, size = oc.norm_rope(k, wk, cs, pos, 1e-6, inter)
    ref_k = want_k.double()
    r = 0
    for b, n in enumerate(new):
        for i in range(n):
            s = kv[b] - n + i
            ref_k[bt_ok[b, s // page], s % page] = ref[r]
            tol_k[bt_ok[b, s // page], s % page] = round_tol(ref[r], size[r], dt, 32)
            want_v[bt_ok[b, s // page], s % page] = v[r]
            r += 1
    dev = cuda_device
    dkc, dvc = kc.to(dev), vc.to(dev)
    out = torch.full((total + behind, hq, D), 7.0, dtype=dt, device=dev)
    got = fa.fa_qk_norm_rope_paged(on(dev, q), on(dev, k), on(dev, v), wq.to(dev), wk.to(dev), cs.to(dev),
                                   None if slots else pos.to(dev), dkc, dvc, bt.to(dev), cu.to(dev), lens.to(dev),
                                   interleaved=inter, q_out=out)
    assert got is out
    rq, sq = oc.norm_rope(q, wq, cs, pos, 1e-6, inter)
    within(out[:total], rq[:total], round_tol(rq, sq, dt, 32)[:total], "q")
    assert bool((out[total:] == 7.0).all())
    within(dkc, ref_k, tol_k, "k pages")
    assert torch.equal(dvc.cpu().view(torch.int16), want_v.view(torch.int16))
    assert fa.fa_device_status()[0] == 0


@pytest.mark.gpu
def test_append_without_a_place(cuda_device):
    """Slots before the cache, past the table and in pages outside the pool: reported, nothing written."""
    import tiled_exact_attention_fwd_b200 as fa
    dev = cuda_device
    q, k, v, wq, wk, cs, pos = norm_inputs(6, 2, 1, 64, 64, torch.bfloat16, torch.bfloat16, False, 3)
    kc = torch.zeros(4, 16, 1, 64, dtype=torch.bfloat16, device=dev)
    vc = torch.zeros_like(kc)
    bt = torch.tensor([[0, 1], [2, 9], [3, -1]], dtype=torch.int32, device=dev)
    cu = torch.tensor([0, 2, 4, 6], dtype=torch.int32, device=dev)
    for lens, rows in (([1, 33, 17], {(0, 0), (3, 15)}), ([40, 18, 34], set()), ([2, 16, 16], {(0, 0), (0, 1), (2, 14), (2, 15), (3, 14), (3, 15)})):
        kc.zero_(), vc.zero_()
        fa.fa_qk_norm_rope_paged(q.to(dev), k.to(dev), v.to(dev), None, None, cs.to(dev), pos.to(dev), kc, vc, bt, cu,
                                 torch.tensor(lens, dtype=torch.int32, device=dev))
        st = fa.fa_device_status()[0]
        assert st == (0 if len(rows) == 6 else -8)
        for pool in (kc, vc):
            assert {(int(a), int(b)) for a, b in pool.abs().sum((2, 3)).nonzero()} == rows


CHUNK = [  # new tokens, keys, hq, hk, D, page, dtype, causal
    ([1], [1], 1, 1, 32, 16, "bf16", True),
    ([1], [300], 4, 4, 64, 16, "fp16", True),
    ([1, 1, 1, 1], [1, 127, 128, 129], 8, 2, 128, 16, "bf16", True),
    ([1] * 7, [63, 64, 65, 1, 700, 2, 333], 6, 2, 128, 64, "fp16", True),
    ([1, 1], [500, 31], 16, 1, 256, 32, "bf16", True),
    ([2, 3, 1], [40, 200, 90], 8, 2, 64, 32, "bf16", True),
    ([1, 5, 0, 17], [0, 3, 50, 200], 4, 2, 128, 16, "bf16", True),  # no keys, fewer keys than tokens, no tokens
    ([3, 2], [130, 0], 10, 2, 64, 128, "fp16", False),
    ([50], [50], 3, 3, 32, 16, "bf16", True),
    ([130, 7], [131, 400], 5, 1, 64, 64, "bf16", True),
    ([33, 128, 65], [512, 128, 100], 4, 1, 128, 128, "bf16", True),
    ([70, 1, 20], [70, 260, 300], 6, 2, 128, 16, "fp16", False),
    ([40, 150], [333, 150], 2, 1, 256, 256, "bf16", True),
    ([64], [200], 7, 1, 256, 16, "fp16", False),
    ([260, 3], [261, 700], 2, 2, 128, 32, "bf16", True),
    # one row tile, its key tiles split between two warpgroups: 1, 2, 3, many of them, an odd and an even count
    ([20, 9, 31, 25, 18], [100, 256, 300, 1300, 129], 4, 1, 128, 64, "bf16", True),
    ([20, 1, 1, 40, 1], [640, 770, 128, 900, 1], 6, 3, 64, 16, "fp16", True),
    ([33, 70, 18], [1025, 130, 20], 2, 2, 32, 32, "bf16", False),
    ([17], [2100], 5, 1, 64, 128, "bf16", True),
    ([300, 20, 129, 1], [600, 520, 257, 900], 2, 1, 128, 16, "bf16", True),  # two tiles and one by turns
]


def chunk_inputs(new, kv, hq, hk, D, page, dtype, seed, behind=2):
    dt = DT[dtype]
    q = fa_inputs.normal((sum(new) + behind, hq, D), dt, seed)
    kc, vc, bt = pools(kv, page, hk, D, dt, seed + 1)
    return q, kc, vc, bt, fa_inputs.cu_seqlens_from_lengths(new), torch.tensor(kv, dtype=torch.int32)


def score_tol(ssize):
    return 2.0 ** -20 * (ssize + 1)


@pytest.mark.gpu
@pytest.mark.parametrize("new,kv,hq,hk,D,page,dtype,causal", CHUNK)
def test_chunk(cuda_device, new, kv, hq, hk, D, page, dtype, causal):
    import tiled_exact_attention_fwd_b200 as fa
    dev, dt = cuda_device, DT[dtype]
    q, kc, vc, bt, cu, lens = chunk_inputs(new, kv, hq, hk, D, page, dtype, 17 + sum(kv))
    total = sum(new)
    out = torch.full(q.shape, 5.0, dtype=dt, device=dev)
    lse = torch.full((hq, q.shape[0]), 5.0, device=dev)
    args = [t.to(dev) for t in (q, kc, vc, bt, cu, lens)]
    fa.fa_fwd_paged_chunk(*args, max(new), out=out, lse=lse, causal=causal)
    assert fa.fa_device_status()[0] == 0
    ref, rl, size, ssize = oc.chunk_attention(q, kc, vc, bt, cu, lens, causal=causal)
    assert bool((out[total:] == 5.0).all()) and bool((lse[:, total:] == 5.0).all())  # rows of no sequence
    ref, rl, size, ssize = ref[:total], rl[:, :total], size[:total], ssize[:, :total]
    e = score_tol(ssize)
    tol = half_step(dt) * ref.abs() + (half_step(dt) + 2 * e.t()[..., None]) * size
    within(out[:total], ref, tol + (2.0 ** -25 if dt == torch.float16 else 0), "out")
    within(lse[:, :total], rl, e + 2.0 ** -23 * rl.abs(), "lse")
    o2, l2 = fa.fa_fwd_paged_chunk(*args, max(new), causal=causal)
    assert torch.equal(o2[:total], out[:total]) and torch.equal(l2[:, :total], lse[:, :total])
    o3, none = fa.fa_fwd_paged_chunk(*args, max(new), causal=causal, return_lse=False)
    assert none is None and torch.equal(o3[:total], out[:total])


@pytest.mark.gpu
@pytest.mark.parametrize("new,kv,hq,hk,D,page,dtype,causal", CHUNK)
def test_key_weights(cuda_device, new, kv, hq, hk, D, page, dtype, causal):
    import tiled_exact_attention_fwd_b200 as fa
    dev = cuda_device
    q, kc, vc, bt, cu, lens = chunk_inputs(new, kv, hq, hk, D, page, dtype, 23 + sum(kv))
    width = bt.shape[1] * page + 5
    _, rl, _, _ = oc.chunk_attention(q, kc, vc, bt, cu, lens, causal=causal)
    lse = rl.float()
    before = torch.rand(len(kv), hk, width, generator=fa_inputs.generator(9))
    w = before.to(dev)
    args = [t.to(dev) for t in (q, kc, bt, cu, lens)]
    got = fa.fa_paged_key_weights(*args, max(new), lse.to(dev), w, causal=causal)
    assert got is w and fa.fa_device_status()[0] == 0
    add, most = oc.key_weights(q, kc, bt, cu, lens, lse, width, causal=causal)
    ref = before.double() + add
    # each weight by its score's error (and the LSE's product with log2 e, 2^-24 of up to 2^5), the sum of
    # up to 2^10 rows in a fixed order and the addition to the buffer
    rel = 2 * 2.0 ** -20 * (most + 1) + 1024 * U
    within(w, ref, rel * add + U * ref, "weights")
    assert torch.equal(w.cpu()[add == 0], before[add == 0])


@pytest.mark.gpu
@pytest.mark.parametrize("lengths,hk,D,page,budget,recent,dtype", [
    ([1], 1, 32, 16, 1, 0, "bf16"),
    ([5, 40, 0, 16], 2, 64, 16, 16, 4, "fp16"),
    ([300, 17, 299], 3, 128, 16, 100, 0, "bf16"),
    ([700, 650], 1, 256, 64, 257, 256, "fp16"),
    ([512, 1030], 2, 128, 32, 512, 512, "bf16"),
    ([5000], 2, 32, 256, 4099, 100, "bf16"),
])
@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
def test_evict(cuda_device, lengths, hk, D, page, budget, recent, dtype, kind):
    import tiled_exact_attention_fwd_b200 as fa
    dev = cuda_device
    kc, vc, bt = pools(lengths, page, hk, D, DT[dtype], 3, fill=2.0)
    width = bt.shape[1] * page
    g = fa_inputs.generator(5)
    w = torch.exp(2 * torch.randn(len(lengths), hk, width, generator=g))
    if kind == "ties":
        w = torch.randint(0, 3, w.shape, generator=g).float()
    if kind == "odd":  # zeros of both signs, infinities, NaN, negative and tiny values
        odd = torch.tensor([0.0, -0.0, math.inf, math.nan, -1.0, 1e-42, -math.inf, 3.4e38])
        w = torch.where(torch.rand(w.shape, generator=g) < 0.5, odd[torch.randint(0, 8, w.shape, generator=g)], w)
    budget = min(budget, width)
    recent = min(recent, budget)
    lens = torch.tensor(lengths, dtype=torch.int32)
    kept, new, nw = oc.evict(w, lens, budget, recent)
    want_k, want_v = (oc.move_rows(c, bt, kept, lens, budget) for c in (kc, vc))
    dkc, dvc, dw = kc.to(dev), vc.to(dev), w.to(dev)
    got = fa.fa_paged_evict(dkc, dvc, bt.to(dev), lens.to(dev), dw, budget, recent)
    assert fa.fa_device_status()[0] == 0
    assert torch.equal(got[0].cpu(), kept) and torch.equal(got[1].cpu(), new)
    assert torch.equal(got[2].cpu().nan_to_num(7.5e37), nw.nan_to_num(7.5e37))
    # rows of the kept slots; what lies behind them in a sequence's pages is left as it was
    assert torch.equal(dkc.cpu(), want_k) and torch.equal(dvc.cpu(), want_v)
    assert torch.equal(dw.cpu().nan_to_num(7.5e37), w.nan_to_num(7.5e37))


@pytest.mark.gpu
def test_bad_tables_and_lengths_are_reported(cuda_device):
    import tiled_exact_attention_fwd_b200 as fa
    dev = cuda_device
    q, kc, vc, bt, cu, lens = chunk_inputs([1, 1, 4], [40, 33, 60], 4, 2, 64, 16, "bf16", 8, behind=0)
    args = [t.to(dev) for t in (q, kc, vc, bt, cu, lens)]
    good, lse = fa.fa_fwd_paged_chunk(*args, 4)
    bad = bt.clone()
    bad[1, 1] = kc.shape[0]
    out, _ = fa.fa_fwd_paged_chunk(args[0], args[1], args[2], bad.to(dev), *args[4:], 4)
    assert fa.fa_device_status()[0] == -8
    assert torch.equal(out[0], good[0]) and torch.equal(out[2:], good[2:])
    bad[1, 1] = -7
    w = torch.zeros(3, 2, bt.shape[1] * 16, device=dev)
    fa.fa_paged_key_weights(args[0], args[1], bad.to(dev), *args[4:], 4, lse, w)
    assert fa.fa_device_status()[0] == -8
    full = torch.where(bt < kc.shape[0], bt, torch.zeros_like(bt)).to(dev)
    for kv in ([40, -5, 60], [40, 33, 100000]):  # cut to 0 and to the table
        lens2 = torch.tensor(kv, dtype=torch.int32, device=dev)
        out, _ = fa.fa_fwd_paged_chunk(args[0], args[1], args[2], full, args[4], lens2, 4)
        assert fa.fa_device_status()[0] == -8
        assert torch.equal(out[0], good[0])
        fa.fa_paged_key_weights(args[0], args[1], full, args[4], lens2, 4, lse, w)
        assert fa.fa_device_status()[0] == -8
    for c in ([0, 1, 2, 600], [0, 1, 2, -3], [-4, 1, 2, 6]):
        fa.fa_fwd_paged_chunk(*args[:4], torch.tensor(c, dtype=torch.int32, device=dev), args[5], 4)
        assert fa.fa_device_status()[0] == -8
    evict_bt = full.clone()
    evict_bt[0, 1] = 10 ** 6
    before = args[1].clone()
    fa.fa_paged_evict(args[1], args[2], evict_bt, args[5], torch.rand_like(w), 20, 0)
    assert fa.fa_device_status()[0] == -8
    args[1].copy_(before)
    kept, new, _ = fa.fa_paged_evict(args[1], args[2], full, torch.tensor([40, -1, 10 ** 8], dtype=torch.int32, device=dev),
                                     torch.rand_like(w), 20, 0)
    assert fa.fa_device_status()[0] == -8 and new.tolist() == [20, 0, 20]


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hk,D,dtype", [(8, 2, 64, "bf16"), (4, 4, 128, "fp16")])
def test_a_cache_s_life(cuda_device, hq, hk, D, dtype):
    """Prompts in chunks, then single tokens, weights added up, eviction, and on: each step checked against
    the definitions applied to the cache as it is then."""
    import tiled_exact_attention_fwd_b200 as fa
    dev, dt, page, budget, recent = cuda_device, DT[dtype], 16, 40, 8
    B, g = 3, fa_inputs.generator(77)
    cols = 6
    kc = torch.full((B * cols + 1, page, hk, D), float("nan"), dtype=dt, device=dev)
    vc = kc.clone()
    bt = torch.randperm(B * cols, generator=g).view(B, cols).to(torch.int32).to(dev)
    wq, wk, cs = weights_of(D, dt, 1).to(dev), weights_of(D, dt, 2).to(dev), angles(300, D).to(dev)
    weights = torch.zeros(B, hk, cols * page, device=dev)
    lens, seen = [0] * B, [0] * B
    for step, new in enumerate([[20, 1, 33], [1, 30, 17], [1, 1, 1], [25, 1, 1], [1, 1, 1]]):
        total = sum(new)
        x = [torch.randn(total, h, D, generator=g).to(dt).to(dev) for h in (hq, hk, hk)]
        pos = torch.cat([torch.arange(s, s + n) for s, n in zip(seen, new)]).to(dev)
        lens = [a + n for a, n in zip(lens, new)]
        seen = [a + n for a, n in zip(seen, new)]
        cu, kv = fa_inputs.cu_seqlens_from_lengths(new).to(dev), torch.tensor(lens, dtype=torch.int32, device=dev)
        q = fa.fa_qk_norm_rope_paged(*x, wq, wk, cs, pos, kc, vc, bt, cu, kv)
        ref, size = oc.norm_rope(x[0], wq, cs, pos, 1e-6, False)
        within(q, ref, round_tol(ref, size, dt, 32), "q")
        out, lse = fa.fa_fwd_paged_chunk(q, kc, vc, bt, cu, kv, max(new))
        ref, rl, size, ssize = oc.chunk_attention(q, kc, vc, bt, cu, kv)
        e = score_tol(ssize)
        within(out, ref, half_step(dt) * ref.abs() + (half_step(dt) + 2 * e.t()[..., None]) * size + 2.0 ** -25, "out")
        before = weights.cpu().double()
        fa.fa_paged_key_weights(q, kc, bt, cu, kv, max(new), lse, weights)
        add, most = oc.key_weights(q, kc, bt, cu, kv, lse, weights.shape[2])
        within(weights, before + add, (2.0 ** -19 * (most + 1) + 1024 * U) * add + U * (before + add), "weights")
        kept, nl, nw = oc.evict(weights, kv, budget, recent)
        want = [oc.move_rows(c, bt, kept, kv, budget) for c in (kc, vc)]
        got, kv, weights = fa.fa_paged_evict(kc, vc, bt, kv, weights, budget, recent)
        assert torch.equal(got.cpu(), kept) and torch.equal(weights.cpu(), nw) and kv.tolist() == nl.tolist()
        for c, w in zip((kc, vc), want):
            assert torch.equal(c.cpu().view(torch.int16), w.view(torch.int16))
        lens = kv.tolist()
    assert fa.fa_device_status()[0] == 0


# --------------------------------------------------------------------------- batches, streams, graphs
def check_chunk_and_weights(dev, new, kv, hq, hk, D, page, dtype, seed, max_q=None):
    import tiled_exact_attention_fwd_b200 as fa
    dt, max_q = DT[dtype], max(new) if max_q is None else max_q
    q, kc, vc, bt, cu, lens = chunk_inputs(new, kv, hq, hk, D, page, dtype, seed, behind=0)
    args = [t.to(dev) for t in (q, kc, vc, bt, cu, lens)]
    out, lse = fa.fa_fwd_paged_chunk(*args, max_q)
    ref, rl, size, ssize = oc.chunk_attention(q, kc, vc, bt, cu, lens)
    e = score_tol(ssize)
    within(out, ref, half_step(dt) * ref.abs() + (half_step(dt) + 2 * e.t()[..., None]) * size + 2.0 ** -25, "out")
    within(lse, rl, e + 2.0 ** -23 * rl.abs(), "lse")
    w = torch.zeros(len(kv), hk, bt.shape[1] * page, device=dev)
    fa.fa_paged_key_weights(args[0], args[1], *args[3:], max_q, lse, w)
    add, most = oc.key_weights(q, kc, bt, cu, lens, lse.cpu(), w.shape[2])
    within(w, add, (2.0 ** -19 * (most + 1) + 1024 * U) * add, "weights")
    assert fa.fa_device_status()[0] == 0


@pytest.mark.gpu
@pytest.mark.parametrize("count", [8, 9, 33, 128, 129, 300])
@pytest.mark.parametrize("few", [True, False])
def test_many_sequences(cuda_device, count, few):
    """The split's ways over a batch: one by one, in one round of loads, in several."""
    g = fa_inputs.generator(count)
    new = torch.randint(0, 3, (count,), generator=g) if few else torch.tensor([0, 1, 40, 90])[torch.randint(0, 4, (count,), generator=g)]
    new[-1] = 1 if few else 40
    kv = (new + torch.randint(0, 150, (count,), generator=g)).tolist()
    check_chunk_and_weights(cuda_device, new.tolist(), kv, 6, 2, 64, 16, "bf16", 41 + count)


@pytest.mark.gpu
@pytest.mark.parametrize("new,kv,max_q", [([20, 1, 7], [90, 300, 7], 1), ([1, 2, 1], [400, 33, 17], 4000)])
def test_max_q_len_does_not_change_the_result(cuda_device, new, kv, max_q):
    check_chunk_and_weights(cuda_device, new, kv, 8, 2, 128, 16, "bf16", 5, max_q)


@pytest.mark.gpu
@pytest.mark.parametrize("few", [True, False])
@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 512, 1024])
def test_every_page_size(cuda_device, page, D, few):
    new, kv = ([1, 2, 1], [5, 700, 257]) if few else ([30, 1, 17], [35, 700, 257])
    check_chunk_and_weights(cuda_device, new, kv, 4, 2, D, page, "bf16", 7)


@pytest.mark.gpu
@pytest.mark.parametrize("D,hq,hk", [(64, 128, 1), (32, 20, 1), (128, 34, 2), (256, 96, 3)])
def test_many_heads_a_key_head(cuda_device, D, hq, hk):
    check_chunk_and_weights(cuda_device, [1, 3, 0, 9], [200, 3, 50, 300], hq, hk, D, 32, "fp16", 51)


@pytest.mark.gpu
@pytest.mark.parametrize("new", [[1, 1, 1], [30, 1, 2]])
def test_outputs_of_any_allowed_alignment(cuda_device, new):
    """out 16 but not 32 bytes from a boundary, lse 4; the caller's workspace full of NaN, or too small."""
    import tiled_exact_attention_fwd_b200 as fa
    dev = cuda_device
    q, kc, vc, bt, cu, lens = chunk_inputs(new, [700, 40, 129], 4, 2, 64, 16, "bf16", 61, behind=0)
    args = [t.to(dev) for t in (q, kc, vc, bt, cu, lens)]
    want, wl = fa.fa_fwd_paged_chunk(*args, max(new))
    out = torch.empty(q.numel() + 8, dtype=q.dtype, device=dev)[8:].view(q.shape)
    lse = torch.empty(wl.numel() + 1, device=dev)[1:].view(wl.shape)
    size = fa.fa_fwd_paged_chunk_workspace(4, 2, 64, max(new))
    ws = torch.full((size // 4,), float("nan"), device=dev)
    fa.fa_fwd_paged_chunk(*args, max(new), out=out, lse=lse, workspace=ws)
    assert torch.equal(out, want) and torch.equal(lse, wl)
    with pytest.raises(fa.FAError):
        fa.fa_fwd_paged_chunk(*args, max(new), workspace=ws[:-1])
    with pytest.raises(fa.FAError):
        fa.fa_fwd_paged_chunk(*args, max(new), workspace=ws.view(torch.uint8)[16:])
    for bad in (dict(out=out.half()), dict(out=out[:1]), dict(lse=lse[:1]), dict(lse=lse.t().contiguous()), dict(workspace=ws.cpu())):
        with pytest.raises(ValueError):
            fa.fa_fwd_paged_chunk(*args, max(new), **bad)
    with pytest.raises(ValueError):
        fa.fa_fwd_paged_chunk(args[0].transpose(0, 1), *args[1:], max(new))
    with pytest.raises(ValueError):
        fa.fa_fwd_paged_chunk(*args[:5], args[5].long(), max(new))
    with pytest.raises(ValueError):
        fa.fa_fwd_paged_chunk(*args[:4], args[4][:-1], args[5], max(new))
    with pytest.raises(ValueError):
        fa.fa_paged_key_weights(args[0], args[1], *args[3:], max(new), wl, torch.zeros(3, 2, 8, device=dev).double())
    with pytest.raises(fa.FAError):
        fa.fa_paged_key_weights(args[0], args[1], *args[3:], max(new), wl, torch.zeros(3, 2, 8, device=dev))
    with pytest.raises(ValueError):
        fa.fa_paged_evict(args[1], args[2], args[3], args[5], torch.zeros(3, 1, 4096, device=dev), 4, 0)


class Step:
    """One step of a serving loop on buffers of its own: append, attention, weights, eviction."""

    def __init__(self, dev, new, kv, hq, hk, D, seed):
        self.new, self.max_q = new, max(new)
        total, page = sum(new), 16
        _, kc, vc, bt, cu, lens = chunk_inputs(new, kv, hq, hk, D, page, "bf16", seed, behind=0)
        self.pools = [torch.nan_to_num(t, 1.0).to(dev) for t in (kc, vc)]
        self.kc, self.vc = (t.clone() for t in self.pools)
        self.bt, self.cu, self.lens = bt.to(dev), cu.to(dev), lens.to(dev)
        self.x = [fa_inputs.normal((total, h, D), torch.bfloat16, seed + i).to(dev) for i, h in enumerate((hq, hk, hk))]
        self.wq, self.cs = weights_of(D, torch.bfloat16, seed).to(dev), angles(4096, D).to(dev)
        self.pos = torch.arange(total, device=dev)
        self.w = torch.zeros(len(kv), hk, bt.shape[1] * page, device=dev)

    def reset(self):
        self.kc.copy_(self.pools[0]), self.vc.copy_(self.pools[1]), self.w.zero_()

    def run(self, stream=None):
        import tiled_exact_attention_fwd_b200 as fa
        q = fa.fa_qk_norm_rope_paged(*self.x, self.wq, self.wq, self.cs, self.pos, self.kc, self.vc, self.bt, self.cu,
                                     self.lens, stream=stream)
        out, lse = fa.fa_fwd_paged_chunk(q, self.kc, self.vc, self.bt, self.cu, self.lens, self.max_q, stream=stream)
        fa.fa_paged_key_weights(q, self.kc, self.bt, self.cu, self.lens, self.max_q, lse, self.w, stream=stream)
        return [q, out, lse, *fa.fa_paged_evict(self.kc, self.vc, self.bt, self.lens, self.w, 100, 20, stream=stream)]

    def state(self, results):
        return [t.clone() for t in (*results, self.kc, self.vc, self.w)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


STEPS = [([1] * 5, [700, 3, 130, 999, 64], 8, 2, 128), ([40, 1, 0, 150], [300, 500, 20, 151], 4, 2, 64)]


@pytest.mark.gpu
def test_captured_and_replayed(cuda_device):
    """Steps captured into graphs of their own give, replayed in any order and at the same time on two
    streams, with the inputs changed in place, the bits of eager calls."""
    steps = [Step(cuda_device, *s, seed=71 + i) for i, s in enumerate(STEPS)]
    for s in steps:  # first calls outside a capture
        s.run()
    graphs, results = [], []
    for s in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            results.append(s.run())
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for turn in range(6):
        for s in steps:
            s.x[0].copy_(torch.randn(s.x[0].shape, generator=fa_inputs.generator(turn)))
            s.reset()
        wants = []
        for s in steps:
            wants.append(s.state(s.run()))
            s.reset()
        torch.cuda.synchronize()
        for i in (0, 1) if turn % 2 else (1, 0):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for s, r, want in zip(steps, results, wants):
            assert same(s.state(r), want)


@pytest.mark.gpu
@pytest.mark.parametrize("as_int", [False, True])
def test_other_streams_and_two_calls_at_once(cuda_device, as_int):
    steps = [Step(cuda_device, *s, seed=81 + i) for i, s in enumerate(STEPS)]
    wants = []
    for s in steps:
        wants.append(s.state(s.run()))
        s.reset()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        results = [s.run(stream=st.cuda_stream if as_int else st) for s, st in zip(steps, streams)]
        torch.cuda.synchronize()
        for s, r, want in zip(steps, results, wants):
            assert same(s.state(r), want)
            s.reset()
        torch.cuda.synchronize()


@pytest.mark.gpu
def test_gradients_captured_beside_an_eager_graph(cuda_device):
    """The backward captured while eager work on the same tensors goes on."""
    import tiled_exact_attention_fwd_b200 as fa
    q, k, v, wq, wk, cs, pos = (None if t is None else on(cuda_device, t) for t in
                                norm_inputs(300, 4, 2, 64, 64, torch.bfloat16, torch.bfloat16, True, 3))
    gq, gk = torch.randn_like(q), torch.randn_like(k)
    want = fa.fa_qk_norm_rope_bwd(q, k, wq, wk, cs, pos, gq, gk)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = fa.fa_qk_norm_rope_bwd(q, k, wq, wk, cs, pos, gq, gk)
        y = fa.fa_qk_norm_rope(q, k, wq, wk, cs, pos)
    for _ in range(3):
        for t in got + y:
            t.fill_(float("nan"))
        g.replay()
        again = fa.fa_qk_norm_rope_bwd(q, k, wq, wk, cs, pos, gq, gk)
        assert same(got, want) and same(again, want)
        assert same(y, fa.fa_qk_norm_rope(q, k, wq, wk, cs, pos))


# --------------------------------------------------------------------------- long caches
@pytest.mark.gpu
@pytest.mark.parametrize("length,budget,recent", [(40000, 17000, 100), (33000, 33000 // 16 * 16, 0), (20000, 1, 1), (16385, 16384, 0)])
def test_evict_from_long_caches(cuda_device, length, budget, recent):
    """More keys than the selection holds in registers."""
    import tiled_exact_attention_fwd_b200 as fa
    dev, page, hk, D = cuda_device, 64, 2, 32
    g = fa_inputs.generator(length)
    cols = -(-length // page)
    bt = torch.randperm(cols, generator=g).to(torch.int32)[None]
    kc, vc = (torch.randn(cols, page, hk, D, generator=g).bfloat16() for _ in range(2))
    w = torch.randint(0, 500, (1, hk, cols * page), generator=g).float()
    lens = torch.tensor([length], dtype=torch.int32)
    kept, new, nw = oc.evict(w, lens, budget, recent)
    want = [oc.move_rows(c, bt, kept, lens, budget) for c in (kc, vc)]
    dk, dv = kc.to(dev), vc.to(dev)
    got = fa.fa_paged_evict(dk, dv, bt.to(dev), lens.to(dev), w.to(dev), budget, recent)
    assert torch.equal(got[0].cpu(), kept) and torch.equal(got[1].cpu(), new) and torch.equal(got[2].cpu(), nw)
    assert torch.equal(dk.cpu(), want[0]) and torch.equal(dv.cpu(), want[1])


@pytest.mark.gpu
def test_offsets_past_32_bits(cuda_device):
    """Pools of 2^31 elements and a few pages more (4.3 GB each): a step whose keys lie in the first and the last pages gives what
    the same keys give in a small pool."""
    import tiled_exact_attention_fwd_b200 as fa
    dev, page, hq, hk, D = cuda_device, 256, 8, 8, 128
    pages = 2 ** 31 // (page * hk * D) + 4
    assert (pages - 4) * page * hk * D >= 2 ** 31
    lens = torch.tensor([700, 500], dtype=torch.int32, device=dev)
    small = torch.arange(5, dtype=torch.int32, device=dev)
    big = torch.tensor([pages - 1, 0, pages - 3, pages - 2, pages - 4], dtype=torch.int32, device=dev)
    cut = lambda t: torch.stack([t[:3], torch.cat([t[3:], t[:1]])])  # noqa: E731  (the last entry is never read)
    for new in ([1, 1], [100, 40]):
        total = sum(new)
        x = [fa_inputs.normal((total, h, D), torch.bfloat16, i).to(dev) for i, h in enumerate((hq, hk, hk))]
        cu, cs = fa_inputs.cu_seqlens_from_lengths(new).to(dev), angles(1000, D).to(dev)
        seen = []
        for n, order in ((5, small), (pages, big)):
            kc, vc = (torch.empty(n, page, hk, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
            for i, c in enumerate((kc, vc)):
                c[order.long()] = fa_inputs.normal((5, page, hk, D), torch.bfloat16, 90 + i).to(dev)
            w = torch.zeros(2, hk, 3 * page, device=dev)
            q = fa.fa_qk_norm_rope_paged(*x, None, None, cs, None, kc, vc, cut(order), cu, lens)
            out, lse = fa.fa_fwd_paged_chunk(q, kc, vc, cut(order), cu, lens, max(new))
            fa.fa_paged_key_weights(q, kc, cut(order), cu, lens, max(new), lse, w)
            res = fa.fa_paged_evict(kc, vc, cut(order), lens, w, 300, 50)
            seen.append([q, out, lse, w, *res, kc[order.long()], vc[order.long()]])
            assert fa.fa_device_status()[0] == 0
            del kc, vc
        assert same(*seen)
