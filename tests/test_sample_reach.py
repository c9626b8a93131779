"""Rows in which fewer than top_k tokens weigh anything, with a nucleus after it: the
histogram of the top k is not reached and the nucleus takes the cluster's bins over."""

import numpy as np
import pytest
import torch

from contextual_sparsity_decode_gb300 import binding as dv

from test_sample import normal, param, reference, uniforms

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,B,V,T,half", [
    ("bf16", 5, 91937, 0.3, True), ("f16", 60, 40000, 0.3, False), ("f32", 1, 500000, 0.2, False), ("bf16", 3, 128001, 0.1, False),
    ("f32", 200, 9000, 0.5, True), ("f16", 16, 524288, 0.02, False), ("bf16", 1, 1000, 0.05, True)])
def test_fewer_than_top_k_within_reach(dt, B, V, T, half):
    x = normal(B, V, dt, 7) * 10
    if half:
        x[:, ::2] = float("-inf")
    logits, u = x.cuda(), param(uniforms(B, 3))
    ks = [(50, 300, 5000, V - 1)[b % 4] for b in range(B)]
    args = dict(temperature=param([T] * B), top_k=param(ks, torch.int32), top_p=param([(0.95, 0.5, 0.999)[b % 3] for b in range(B)]))
    ws = dv.workspace(256)
    token, prob = torch.full((B,), -7, dtype=torch.int32, device="cuda"), torch.zeros(B, device="cuda")
    dv.dv_sample(logits, u, token, ws, prob=prob, **args)
    assert dv.dv_check(ws) == (0, 0)
    x64 = logits.double().cpu().numpy()
    within = [int((x64[b] > x64[b].max() - 28 * T).sum()) for b in range(B)]
    assert any(n < min(k, V - 1) for n, k in zip(within, ks))
    for b in range(0, B, max(1, B // 8)):
        t, p, _ = reference(x64[b], float(u[b]), float(args["temperature"][b]), ks[b], float(args["top_p"][b]))
        assert int(token[b]) == t and abs(float(prob[b]) - p) <= 1e-6 * p
    for _ in range(30):
        again = torch.full_like(token, -7)
        dv.dv_sample(logits, u, again, ws, **args)
        assert torch.equal(again, token)
