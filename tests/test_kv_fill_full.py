"""Cache fill up to the last slot."""

import pytest
import torch

from contextual_sparsity_decode_gb300 import binding as dv
from dvtest import TORCH, f64, within_ulp_product

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d_h", [64, 128])
def test_every_slot_of_a_full_cache_is_filled(dtype, d_h):
    """pos = n_max: the repair reads and writes positions before pos only, so a
    cache that is full can be filled; one position more is refused."""
    B, d, h, n_max = 2, 192, 2, 144
    W = (torch.randn(h, 3, d_h, d, generator=torch.Generator().manual_seed(3)) / 8).to(TORCH[dtype]).cuda()
    kv, ref = (dv.KV.empty(B, h, n, d_h, d, TORCH[dtype], "cuda") for n in (n_max, n_max + 16))
    X = torch.randn(B, n_max, d, generator=torch.Generator().manual_seed(4)).to(TORCH[dtype]).cuda()
    kv.X.copy_(X)
    ref.X[:, :n_max] = X
    idx = torch.arange(h, dtype=torch.int32, device="cuda").repeat(B, 1)
    cnt = torch.full((B,), h, dtype=torch.int32, device="cuda")
    pos = torch.tensor([n_max, n_max - 5], dtype=torch.int32, device="cuda")
    ws = dv.workspace(dv.dv_sparse_attn_workspace_size(B, d, h, d_h, h, n_max + 16))
    for c in (kv, ref):
        dv.dv_kv_repair(c, W, pos, idx, cnt, ws)
        assert dv.dv_check(ws) == (0, 0)
    assert kv.valid[0].all() and kv.valid[1, :, :n_max - 5].all() and not kv.valid[1, :, n_max - 5:].any()
    assert torch.equal(kv.K, ref.K[:, :, :n_max]) and torch.equal(kv.V, ref.V[:, :, :n_max])
    assert within_ulp_product(f64(kv.K)[0, 1], f64(X)[0], f64(W)[1, 1], dtype)
    pos.fill_(n_max + 1)
    kv.valid.zero_()
    dv.dv_kv_repair(kv, W, pos, idx, cnt, ws)
    assert dv.dv_check(ws) == (9, n_max + 1)
    assert not kv.valid.any()
