"""Calls of the operators around a paged cache whose results overlap what they read or one another: refused on
the host. No GPU is needed: no address here is ever read."""
import pytest

MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from tiled_exact_attention_fwd_b200 import build
    build.build()
    import tiled_exact_attention_fwd_b200 as fa
    return fa.lib()


class TestChunk:
    """q and out: 4 * 4 * 64 * 2 = 2048 bytes, lse 64, table 32, cu_seqlens 12, kv_lens 8."""

    def call(self, lib, **kw):
        a = dict(q=MB, kc=2 * MB, vc=3 * MB, bt=4 * MB, mb=4, page=16, pages=9, cu=5 * MB, kv=6 * MB, num=2, total=4, mq=2,
                 out=7 * MB, lse=8 * MB, ws=16 * MB, wsb=1 << 40, hq=4, hk=2, d=64, scale=0.0, causal=1, dt=0)
        a.update(kw)
        return lib.fa_fwd_paged_chunk(*a.values(), None)

    @pytest.mark.parametrize("change", [
        dict(out=MB), dict(out=MB + 2032), dict(out=MB - 2032), dict(out=4 * MB - 2032),
        dict(out=4 * MB + 16), dict(out=5 * MB), dict(out=6 * MB), dict(lse=MB), dict(lse=4 * MB + 28),
        dict(lse=5 * MB + 8), dict(lse=6 * MB - 60), dict(lse=7 * MB + 2044), dict(lse=7 * MB - 60), dict(out=16 * MB), dict(lse=16 * MB + 4),
        dict(ws=7 * MB), dict(ws=MB), dict(ws=MB // 2, mq=9, q=MB)])
    def test_overlaps(self, lib, change):
        assert self.call(lib, **change) == -2


class TestKeyWeights:
    """weights: 2 * 2 * 64 * 4 = 1024 bytes."""

    def call(self, lib, **kw):
        a = dict(q=MB, kc=2 * MB, bt=4 * MB, mb=4, page=16, pages=9, cu=5 * MB, kv=6 * MB, num=2, total=4, mq=2, lse=7 * MB,
                 w=8 * MB, width=64, ws=16 * MB, wsb=1 << 30, hq=4, hk=2, d=64, scale=0.0, causal=1, dt=0)
        a.update(kw)
        return lib.fa_paged_key_weights(*a.values(), None)

    @pytest.mark.parametrize("change", [
        dict(w=MB), dict(w=MB - 1020), dict(w=MB + 2044), dict(w=4 * MB + 28), dict(w=5 * MB + 8), dict(w=6 * MB - 1020),
        dict(w=7 * MB + 60), dict(w=7 * MB - 1020), dict(ws=8 * MB, mq=9), dict(ws=7 * MB, mq=9), dict(ws=MB, mq=9)])
    def test_overlaps(self, lib, change):
        assert self.call(lib, **change) == -2


class TestEvict:
    """weights and new weights: 2 * 2 * 64 * 4 = 1024 bytes, kept 128, lengths 8, table 32, pools 9 * 4096."""

    def call(self, lib, **kw):
        a = dict(kc=MB, vc=2 * MB, bt=3 * MB, mb=4, page=16, pages=9, kv=4 * MB, w=5 * MB, width=64, budget=8, recent=2,
                 kept=6 * MB, nl=7 * MB, nw=8 * MB, b=2, hk=2, d=64, dt=0)
        a.update(kw)
        return lib.fa_paged_evict(*a.values(), None)

    @pytest.mark.parametrize("change", [
        dict(nl=6 * MB), dict(nl=6 * MB + 124), dict(nw=6 * MB - 1020), dict(kept=8 * MB + 1020), dict(nl=8 * MB + 512), dict(nw=7 * MB + 4),
        dict(vc=MB), dict(vc=MB + 36848), dict(kc=2 * MB + 16), dict(vc=MB + 4096 + 16), dict(vc=MB - 2048),
        dict(kept=3 * MB + 28), dict(nw=3 * MB)])
    def test_overlaps(self, lib, change):
        assert self.call(lib, **change) == -2


class TestNorm:
    """4 tokens; q rows of 4 * 64 * 2 = 512 bytes, k rows of 256; views of a fused buffer: rows of 1024 bytes."""

    def call(self, lib, **kw):
        a = dict(q=MB, qs=256, k=2 * MB, ks=128, wq=9 * MB, wk=10 * MB, w32=0, cs=3 * MB, rows=64, rot=64, pos=4 * MB, qo=5 * MB,
                 qos=256, ko=6 * MB, kos=128, n=4, hq=4, hk=2, d=64, eps=1e-6, inter=0, dt=1)
        a.update(kw)
        return lib.fa_qk_norm_rope(*a.values(), None)

    @pytest.mark.parametrize("change", [
        dict(qo=2 * MB), dict(ko=MB), dict(qo=MB + 16), dict(qo=MB - 2032), dict(qo=MB, qos=264), dict(qo=6 * MB), dict(ko=5 * MB + 2032),
        dict(qo=4 * MB), dict(ko=4 * MB + 16), dict(qo=9 * MB), dict(ko=10 * MB + 112), dict(w32=1, ko=10 * MB + 240),
        # one fused buffer: q in its bytes 0-511 of a row, k in 512-767
        dict(qs=512, k=MB + 512, ks=512, qo=MB + 16, qos=512), dict(qs=512, k=MB + 512, ks=512, qo=MB, qos=512, ko=MB + 768 - 16, kos=512, n=3, q=MB + 1024),
        dict(qs=512, k=MB + 512, ks=512, qo=MB + 512, qos=512), dict(qs=512, k=MB + 512, ks=512, ko=MB + 256, kos=512),
        dict(qs=512, k=MB + 512, ks=512, qo=MB, qos=256), dict(n=1, qo=MB + 496), dict(n=1, ko=MB + 256)])
    def test_forward(self, lib, change):
        assert self.call(lib, **change) == -2

    def paged(self, lib, **kw):
        a = dict(q=MB, qs=256, k=2 * MB, ks=128, v=7 * MB, vs=128, wq=None, wk=None, w32=0, cs=3 * MB, rows=64, rot=64, pos=None,
                 qo=5 * MB, qos=256, kc=16 * MB, vc=17 * MB, bt=8 * MB, mb=4, page=16, pages=9, cu=9 * MB, kv=10 * MB, num=2, n=4,
                 hq=4, hk=2, d=64, eps=1e-6, inter=0, dt=1)
        a.update(kw)
        return lib.fa_qk_norm_rope_paged(*a.values(), None)

    @pytest.mark.parametrize("change", [
        dict(vc=16 * MB), dict(vc=16 * MB + 36848), dict(vc=16 * MB - 4096 - 16), dict(qo=2 * MB), dict(qo=7 * MB), dict(qo=7 * MB - 2032),
        dict(qo=8 * MB), dict(qo=9 * MB), dict(qo=10 * MB), dict(qo=MB + 512), dict(qo=MB, qos=264), dict(pos=5 * MB)])
    def test_paged(self, lib, change):
        assert self.paged(lib, **change) == -2

    def bwd(self, lib, **kw):
        a = dict(q=MB, qs=256, k=2 * MB, ks=128, wq=9 * MB, wk=10 * MB, w32=0, cs=3 * MB, rows=64, rot=64, pos=4 * MB, dqo=5 * MB,
                 dqos=256, dko=6 * MB, dkos=128, dq=7 * MB, dqs=256, dk=8 * MB, dks=128, dwq=11 * MB, dwk=12 * MB, ws=16 * MB,
                 wsb=1 << 30, n=4, hq=4, hk=2, d=64, eps=1e-6, inter=0, dt=1)
        a.update(kw)
        return lib.fa_qk_norm_rope_bwd(*a.values(), None)

    @pytest.mark.parametrize("change", [
        dict(dq=6 * MB), dict(dk=5 * MB), dict(dq=5 * MB + 16), dict(dq=5 * MB, dqs=264), dict(dq=2 * MB), dict(dk=MB), dict(dk=7 * MB),
        dict(dwq=7 * MB), dict(dwk=11 * MB + 252), dict(dwq=9 * MB), dict(ws=11 * MB), dict(ws=7 * MB), dict(dk=4 * MB),
        dict(q=5 * MB, dq=5 * MB + 32)])
    def test_backward(self, lib, change):
        assert self.bwd(lib, **change) == -2


@pytest.mark.parametrize("built", [True, False])
def test_binding_that_does_not_load(lib, monkeypatch, tmp_path, built):
    """A compiled binding that is there but does not load (built against another torch) is not called missing."""
    import sys

    import tiled_exact_attention_fwd_b200 as fa
    monkeypatch.setattr(fa, "_ext", None)
    monkeypatch.delattr(fa, "_fa_torch", raising=False)
    monkeypatch.setitem(sys.modules, fa.__name__ + "._fa_torch", None)  # its import raises ImportError
    if built:
        (tmp_path / "_fa_torch.so").touch()
    monkeypatch.setattr(fa, "_HERE", str(tmp_path))
    with pytest.raises(RuntimeError, match="does not load.*--force" if built else "is not built"):
        fa._binding()
