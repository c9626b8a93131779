"""Passes of the decoder over 4-bit layers, block by block against 64 bits: every position
of a dense prompt (a captured pass over all neurons, launches overlapped) and every call of
a tree's pass.  Tolerances as in test_stack_q4.py."""

import numpy as np
import pytest
import torch

from synth import Workload

from test_q4 import EPS, mlp_reference
from test_stack_q4 import check_mlp, decoder

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,B,group,mixed", [("f16", 1, 64, False), ("bf16", 1, 128, True), ("f32", 1, 64, False),
                                                 ("f16", 2, 128, False), ("bf16", 5, 64, True)])
def test_every_position_of_a_prompt(dtype, B, group, mixed):
    w = Workload("q4p", 44, d=256, h=4, d_h=64, N=512, r=64, dtype=dtype, layers=3, n_prompt=8, neuron_pct=30, head_pct=50)
    dec = decoder(w, B, group, mixed)
    E = torch.randn(B, 5, w.d, generator=torch.Generator().manual_seed(2)).cuda()
    seen = []

    def position(t):
        dec.check()
        assert all(c.tolist() == [w.N] * B for c in dec.neur_cnt)
        assert torch.equal(dec.r_in0, E[:, t])
        check_mlp(dec)
        seen.append(t)

    dec.prefill_dense(E, 5, on_position=position)
    assert seen == list(range(5)) and dec.k_neurons == w.k_neurons


@pytest.mark.parametrize("dtype,B,T,mixed", [("f16", 1, 1, False), ("bf16", 1, 2, True), ("f16", 1, 40, False), ("f16", 2, 17, False),
                                             ("f32", 1, 5, False), ("bf16", 3, 4, True)])
def test_every_call_of_a_trees_pass(dtype, B, T, mixed):
    """Nodes go through the MLP 32 at a time: the last call of a tree may hold one or two."""
    w = Workload("q4v", 45, d=256, h=4, d_h=64, N=512, r=64, dtype=dtype, layers=2, n_prompt=8, neuron_pct=30, head_pct=100)
    dec = decoder(w, B, 64, mixed)
    E = torch.randn(B, T, w.d, generator=torch.Generator().manual_seed(3)).cuda()
    mlp, calls = dec._mlp, []

    def seen(l, y, idx, cnt, out, *ws):
        before = out.clone()
        mlp(l, y, idx, cnt, out, *ws)
        calls.append((l, y.clone(), idx.clone(), cnt.clone(), before, out.clone()))

    dec._mlp = seen
    streams = dec.verify_tree(E)
    dec.check()
    assert [c[1].shape[0] for c in calls] == [min(32, B * T - i) for i in range(0, B * T, 32)] * w.layers
    for l, y, idx, cnt, before, after in calls:
        W = dec.layers[l]
        if "W1q" not in W:
            continue
        ref, tol = mlp_reference(y, W["W1q"], W["W2q"], idx.cpu(), cnt.cpu())
        mid, out = before.double().cpu().numpy(), after.double().cpu().numpy()
        assert np.abs(ref).max() > 0
        assert np.all(np.abs(out - mid - ref) <= tol + 2 * EPS * np.maximum(np.abs(out), np.abs(mid)))
    last = torch.cat([c[5] for c in calls if c[0] == w.layers - 1])
    assert torch.equal(streams.view(B * T, w.d), last)
