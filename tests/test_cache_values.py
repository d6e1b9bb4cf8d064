"""The operators around a paged cache on values that the draws of test_cache_ops.py do not hold, against
the same definitions in 64 bits and with its tolerances: NaN and infinities in what a row sees."""
import math

import pytest
import torch

import fa_inputs
from oracle import cache as oc
from test_cache_ops import DT, U, chunk_inputs, within


# Sequences, new tokens of each, keys of each. One sequence: each step (64 or 128 keys) is a run of its own, so every
# item is cut at every step. Many: runs of several items, most of them whole.
LAYOUTS = {"cut": (1, 900), "whole": (100, 150)}


@pytest.mark.gpu
@pytest.mark.parametrize("few", [True, False])
@pytest.mark.parametrize("layout", ["cut", "whole"])
@pytest.mark.parametrize("D", [32, 64, 128, 256])
def test_key_weights_of_rows_without_a_finite_lse(cuda_device, D, layout, few):
    """A row whose lse is NaN makes the weights of the keys that it sees NaN, and of no other key; a row whose lse is
    -inf gives nothing, whatever its query holds."""
    import tiled_exact_attention_fwd_b200 as fa
    count, kv = LAYOUTS[layout]
    n = 1 if few else 20
    dtype = "bf16" if D > 64 else "fp16"
    q, kc, vc, bt, cu, lens = chunk_inputs([n] * count, [kv] * count, 4, 2, D, 16, dtype, 7 + D, behind=0)
    _, lse, _, _ = oc.chunk_attention(q, kc, vc, bt, cu, lens)
    lse = lse.float()
    lse[1, n // 3::n] = math.nan
    lse[0, n // 2::n] = lse[3, n // 2::n] = -math.inf
    q[n // 2::n, 0], q[n // 2::n, 3] = math.nan, math.inf
    w = torch.zeros(count, 2, bt.shape[1] * 16, device=cuda_device)
    fa.fa_paged_key_weights(*(t.to(cuda_device) for t in (q, kc, bt, cu, lens)), n, lse.to(cuda_device), w)
    add, most = oc.key_weights(q, kc, bt, cu, lens, lse, w.shape[2])
    seen = kv - n + n // 3 + 1  # keys of the row with NaN
    nan = torch.isnan(add)
    assert bool(nan[:, 0, :seen].all()) and not bool(nan[:, 0, seen:].any()) and not bool(nan[:, 1].any())
    within(w, add, (2.0 ** -19 * (most + 1) + 1024 * U) * add, "weights")
    assert fa.fa_device_status()[0] == 0
