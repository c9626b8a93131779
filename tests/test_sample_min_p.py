"""min_p on either side of a token's weight, down to the smallest that count.

A token's weight w (1 being the best one's) is held to 2^-29 of itself and 2^-40, so a
min_p further below it than that keeps the token, and one further above drops it.
u = 1 draws the last kept token: the probe stands last, so it is drawn if and only if it is kept."""

import numpy as np
import pytest
import torch

from contextual_sparsity_decode_gb300 import binding as dv

from test_sample import param, run

pytestmark = pytest.mark.gpu

INF = np.float32(np.inf)


def thresholds(w):
    """The float32 nearest to w that have to keep it and to drop it (None: no
    positive one keeps it)."""
    off = w * 2.0 ** -29 + 2.0 ** -40
    keep = np.float32(w - off)
    while float(keep) >= w - off:
        keep = np.nextafter(keep, -INF)
    drop = np.float32(w + off)
    while float(drop) <= w + off:
        drop = np.nextafter(drop, INF)
    return (keep if keep > 0 else None), drop


@pytest.mark.parametrize("kw", [dict(), dict(top_k=5), dict(top_k=900)])
@pytest.mark.parametrize("V,T", [(2, 1.0), (1000, 0.7), (40000, 1.9)])
def test_min_p_beside_known_weights(V, T, kw):
    """Weights from 2^-0.3 to 2^-39.9: the best token first, -inf, the probe last."""
    T = float(np.float32(T))
    steps = np.concatenate([np.linspace(0.3, 12, 30), np.linspace(12.4, 36, 40), np.linspace(36.1, 39.9, 40)])
    rows = torch.full((len(steps), V), float("-inf"))
    rows[:, 0] = 7.25
    rows[:, V - 1] = 7.25 - torch.from_numpy(steps * np.log(2.0) * T)
    w = np.exp((rows[:, V - 1].double() - 7.25).numpy() / T)   # (a difference that 64 bits hold)
    keep, drop = zip(*(thresholds(float(x)) for x in w))
    n = len(steps)
    args = {k: param([v] * n, torch.int32) for k, v in kw.items()}
    logits, u, temp = rows.cuda(), param([1.0] * n), param([T] * n)
    token, _, status = run(logits, u, temperature=temp, min_p=param([0.0 if k is None else float(k) for k in keep]), **args)
    assert status == (0, 0)
    for i in range(n):
        if keep[i] is not None:
            assert int(token[i]) == V - 1, (steps[i], keep[i], w[i])
    token, prob, status = run(logits, u, temperature=temp, min_p=param([float(x) for x in drop]), **args)
    assert status == (0, 0) and token.tolist() == [0] * n and torch.equal(prob.cpu(), torch.ones(n))


@pytest.mark.parametrize("p", [0.5, 0.99])
def test_min_p_after_a_nucleus(p):
    """256 equal best tokens and a probe behind them that the nucleus keeps: p is taken of
    the mass with it, min_p decides."""
    V, T = 257, 1.0
    for d in (-0.5, -2.0, -3.0):
        w = float(np.exp(np.float64(np.float32(d))))
        keep, drop = thresholds(w)
        row = torch.zeros(2, V)
        row[:, V - 1] = d
        # everything but less than the probe's weight: the nucleus ends with the probe
        top_p = float(np.float32((256 + w / 2) / (256 + w)))
        token, _, status = run(row.cuda(), param([1.0, 1.0]), temperature=param([T, T]), min_p=param([float(keep), float(drop)]),
                               top_p=param([top_p, top_p]))
        assert status == (0, 0) and token.tolist() == [V - 1, V - 2]
        # a nucleus that ends among the equal ones leaves nothing for min_p to decide
        token, _, status = run(row.cuda(), param([1.0, 1.0]), temperature=param([T, T]), min_p=param([float(keep), float(drop)]),
                               top_p=param([p * 0.9, p * 0.9]))
        assert status == (0, 0) and int(token[0]) == int(token[1]) < V - 2
