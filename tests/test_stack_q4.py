"""The decoder with its MLP in 4 bits and tokens drawn through a 4-bit head: every
block on its own inputs against 64 bits, eager and captured.

Tolerances: the MLP's as in test_q4.py, and the residual stream's own rounding
(2^-24 of the larger of its two values); logits as the products of
test_q4.py; tokens are equal for the logits that the head gave."""

import math

import numpy as np
import pytest
import torch

from contextual_sparsity_decode_gb300 import binding as dv
from contextual_sparsity_decode_gb300.stack import SparseDecoder, quantize_mlp
from synth import Workload, embeddings, layer_weights, residual_input

from test_q4 import EPS, matvec_bound, mlp_reference, opened
from test_sample import reference

pytestmark = pytest.mark.gpu


def decoder(w, B, group, mixed=False, n_max=64):
    layers = [layer_weights(w, l, device="cuda") for l in range(w.layers)]
    small = quantize_mlp(layers, group)
    if mixed:
        small[0] = layers[0]
    dec = SparseDecoder(small, B, n_max, w.k_heads, w.k_neurons, 1 / math.sqrt(w.d_h), trace=True)
    dec.prefill([torch.stack([embeddings(w, w.n_prompt, f"X{l}/{b}", device="cuda") for b in range(B)])
                 for l in range(w.layers)], w.n_prompt)
    dec.r_stream.copy_(residual_input(w, B, "r0", device="cuda"))
    return dec


def check_mlp(dec):
    for l, W in enumerate(dec.layers):
        if "W1q" not in W:
            continue
        ref, tol = mlp_reference(dec.y_m[l], W["W1q"], W["W2q"], dec.neur_idx[l].cpu(), dec.neur_cnt[l].cpu())
        mid, out = dec.r_mid[l].double().cpu().numpy(), dec.r_out[l].double().cpu().numpy()
        assert np.abs(ref).max() > 0
        # (the sum into the stream: its own rounding)
        assert np.all(np.abs(out - mid - ref) <= tol + 2 * EPS * np.maximum(np.abs(out), np.abs(mid)))


def check_sample(dec, u, T=None, k=None, p=None, least=None):
    y = dec.y_head.double().cpu().numpy()
    H = opened(dec.head.q, dec.head.scale, dec.d, dec.head.group)
    got = dec.logits.double().cpu().numpy()
    assert np.all(np.abs(got - y @ H.T) <= matvec_bound(dec.d, H, y))
    pick = lambda t, b, other: other if t is None else float(t[b])  # noqa: E731
    for b in range(dec.B):
        token, prob, _ = reference(got[b], float(u[b]), pick(T, b, 1.0), int(pick(k, b, 0)), pick(p, b, 1.0), pick(least, b, 0.0))
        assert int(dec.token[b]) == token
        assert abs(float(dec.prob[b]) - prob) <= prob * (2.0 ** -24 + 2.0 ** -30 + got.shape[1] * 2.0 ** -40)


@pytest.mark.parametrize("dtype,B,group,mixed", [("f16", 1, 128, False), ("bf16", 1, 64, False), ("f16", 2, 64, True),
                                                 ("bf16", 5, 128, False), ("f32", 1, 128, True)])
def test_steps_and_tokens(dtype, B, group, mixed):
    w = Workload("q4", 41, d=256, h=4, d_h=64, N=1024, r=64, dtype=dtype, layers=3, n_prompt=9, neuron_pct=20, head_pct=50)
    dec = decoder(w, B, group, mixed)
    V = 1003
    head = dv.Q4.of((torch.randn(V, w.d, generator=torch.Generator().manual_seed(4)) * 0.3).to(dec.dtype).cuda(), group)
    dec.set_head(head)
    g = torch.Generator().manual_seed(B)
    u = torch.rand(B, generator=g).cuda()
    T, p = torch.full((B,), 0.8, device="cuda"), torch.full((B,), 0.9, device="cuda")
    k = torch.full((B,), 40, dtype=torch.int32, device="cuda")
    dec.step_ops()
    dec.sample(u, T, k, p)
    dec.check()
    check_mlp(dec)
    check_sample(dec, u, T, k, p)
    eager = dec.token.clone(), dec.prob.clone()
    # the same step and draw as one graph, then with other numbers
    dec2 = decoder(w, B, group, mixed)
    dec2.set_head(head)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            dec2.step_ops()
            dec2.sample(u, T, k, p)
            dv.dv_positions_advance(dec2.pos, 0, dec2.n_max)
    torch.cuda.current_stream().wait_stream(s)
    graph.replay()
    if B == 1:   # (2+ rows: the attention adds its partial sums in any order)
        assert torch.equal(dec2.token, eager[0]) and torch.equal(dec2.prob, eager[1])
    for _ in range(3):
        u.copy_(torch.rand(B, generator=g))
        graph.replay()
        dec2.check()
        check_mlp(dec2)
        check_sample(dec2, u, T, k, p)


def test_prompt_and_drafted_trees_run_in_4_bits():
    w = Workload("q4t", 42, d=256, h=4, d_h=64, N=512, r=64, dtype="f16", layers=2, n_prompt=8, neuron_pct=30, head_pct=100)
    dec = decoder(w, 1, 64)
    E = (torch.randn(1, 3, w.d, generator=torch.Generator().manual_seed(1))).cuda()
    dec.prefill_dense(E, 3)
    check_mlp_dense = dec.r_out[1].clone()
    assert torch.isfinite(check_mlp_dense).all()
    tree = dec.verify_tree(E)
    dec.check()
    # a node's stream is the one that a decode step leaves with the tree's heads: here all of them
    one = decoder(w, 1, 64)
    one.prefill_dense(E, 3)
    one.r_stream.copy_(E[:, 0])
    one.step_ops()
    one.check()
    d = (one.r_stream - tree[:, 0]).norm() / one.r_stream.norm()
    assert d <= 2e-3   # q and the attention's result in f16: 2^-11 each, and their way through two layers


def test_heads_and_layers_of_other_shapes_are_refused():
    w = Workload("q4r", 43, d=256, h=4, d_h=64, N=512, r=64, dtype="f16", layers=2, n_prompt=4)
    dec = decoder(w, 1, 64)
    with pytest.raises(ValueError):
        dec.sample(torch.zeros(1, device="cuda"))
    for bad in (dv.Q4.empty(10, 128, torch.float16), dv.Q4.empty(10, 256, torch.bfloat16),
                dv.Q4.empty(10, 256, torch.float16, device="cpu")):
        with pytest.raises(ValueError):
            dec.set_head(bad)
    layers = quantize_mlp([layer_weights(w, 0, device="cuda")], 64)
    layers[0]["W2q"] = dv.Q4.empty(512, 128, torch.float16)
    with pytest.raises(ValueError):
        SparseDecoder(layers, 1, 32, w.k_heads, w.k_neurons, 0.1)
