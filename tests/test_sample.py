"""dv_sample against its definition in 64 bits, row by row.

Tokens are equal.  (The kernel's weights are within 2^-30 of themselves or 2^-40,
so a drawn u is on the other side of a border with a probability of about V times
the error of a sum, below 1e-5 for every row here; borders are tested where all
sums are exact.)  Probabilities: the chosen token's weight is taken in 64 bits and
the sum of the others is within 2^-30 + V 2^-40 of its size, then one rounding to
fp32: 2^-24 + 2^-30 + V 2^-40 relative."""

import numpy as np
import pytest
import torch

from contextual_sparsity_decode_gb300 import binding as dv

from dvtest import TORCH


COLD, HOT = float(np.float32(1e-30)), float(np.float32(1e30))   # temperatures within, or 0


def reference(x, u, T=1.0, k=0, p=1.0, least=0.0):
    """(token, probability, kept) of one row of float64 logits."""
    if not np.any(x > -np.inf) or np.any(np.isnan(x) | (x == np.inf)) or not (T == 0 or COLD <= T <= HOT) or np.isnan(u + p + least):
        return -1, 0.0, 0
    order = np.argsort(-x, kind="stable")
    if T == 0:
        return int(order[0]), 1.0, 1
    w = np.exp((x - x[order[0]]) / T)
    if k > 0:
        order = order[:k]
    if p < 1:
        upto = np.cumsum(w[order])
        before = upto - w[order]
        n = int(np.searchsorted(-(before < max(p, 0) * upto[-1]).astype(int), 0))   # the first that is not
        order = order[:max(n, 1)]
    kept = np.sort(order[w[order] >= min(least, 1.0)])
    upto = np.cumsum(w[kept])
    i = min(int(np.searchsorted(upto, max(u, 0) * upto[-1], side="right")), len(kept) - 1)
    while w[kept[i]] == 0:
        i -= 1
    return int(kept[i]), w[kept[i]] / upto[-1], len(kept)


def run(logits, u, ws=None, **kw):
    B, V = logits.shape
    ws = ws if ws is not None else dv.workspace(dv.dv_sample_workspace_size(B, V))
    token = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    prob = torch.full((B,), -7.0, device="cuda")
    dv.dv_sample(logits, u, token, ws, prob=prob, **kw)
    return token, prob, dv.dv_check(ws)


def param(v, dtype=torch.float32):
    return None if v is None else torch.tensor(v, dtype=dtype).cuda()


def check(logits, u, T=None, k=None, p=None, least=None):
    """Every row against the definition; the parameters are lists or None."""
    B, V = logits.shape
    token, prob, status = run(logits, param(u), temperature=param(T), top_k=param(k, torch.int32), top_p=param(p),
                              min_p=param(least))
    x = logits.double().cpu().numpy()
    f32 = lambda v, b, other: other if v is None else float(np.float32(v[b]))  # noqa: E731
    bad = None
    for b in range(B):
        t, q, _ = reference(x[b], f32(u, b, 0), f32(T, b, 1.0), k[b] if k is not None else 0, f32(p, b, 1.0),
                            f32(least, b, 0.0))
        assert int(token[b]) == t, (b, int(token[b]), t)
        assert abs(float(prob[b]) - q) <= q * (2.0 ** -24 + 2.0 ** -30 + V * 2.0 ** -40), (b, float(prob[b]), q)
        if t < 0 and bad is None:
            bad = b
    if bad is None:
        assert status == (0, 0)
    else:
        assert status[0] == 1
    return token


def normal(B, V, dt, seed, std=3.0):
    return (torch.randn(B, V, generator=torch.Generator().manual_seed(seed)) * std).to(TORCH[dt])


def uniforms(B, seed):
    return torch.rand(B, generator=torch.Generator().manual_seed(900 + seed)).tolist()


SIZES = [(3, 1), (4, 2), (5, 7), (9, 33), (8, 300), (6, 1000), (5, 4097), (3, 8191), (4, 32000), (3, 50257), (2, 128001)]
FILTERS = [
    dict(), dict(k=1), dict(k=5), dict(k=50), dict(k=257), dict(k=1000), dict(p=0.9), dict(p=0.5), dict(p=0.01),
    dict(p=0.999), dict(least=0.05), dict(least=1.0), dict(k=40, p=0.9), dict(k=700, p=0.8), dict(k=700, p=0.95, least=0.01),
    dict(k=20, least=0.1), dict(p=0.95, least=0.02), dict(k=20, p=0.7, least=0.3), dict(p=0.0), dict(k=3, p=0.0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,V", SIZES)
def test_draws_of_normal_logits(dt, B, V):
    for n, f in enumerate(FILTERS):
        logits = normal(B, V, dt, 17 * V + n)
        if V > 40:
            logits[:, 3:V:29] = float("-inf")
        T = [[0.7, 1.0, 1.3, 0.25][(b + n) % 4] for b in range(B)]
        T = None if n % 5 == 4 else T
        many = {key: [v] * B for key, v in f.items()}
        check(logits.cuda(), uniforms(B, n + V), T, many.get("k"), many.get("p"), many.get("least"))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("V", [262144, 524288])
def test_the_largest_vocabularies(dt, V):
    logits = normal(4, V, dt, V).cuda()
    for n, f in enumerate(({}, dict(k=50), dict(k=3000, p=0.9), dict(p=0.95), dict(least=0.001))):
        many = {key: [v] * 4 for key, v in f.items()}
        check(logits, uniforms(4, n), [0.8, 1.0, 0.0, 1.5], many.get("k"), many.get("p"), many.get("least"))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [64, 5000, 40000])
def test_shapes_of_distributions(dt, V):
    """Flat rows, a few distinct values, a steep row, a row far from zero, one
    finite token, values beside each other, every filter passing among equals."""
    B = 10
    g = torch.Generator().manual_seed(V)
    x = torch.zeros(B, V)
    x[1] = torch.randint(0, 4, (V,), generator=g).float()
    x[2] = -torch.arange(V).float() * 0.5
    x[3] = torch.randn(V, generator=g) * 0.1 - 300
    x[4], x[4, V // 2] = float("-inf"), 2.0
    x[5] = 1.0 + torch.randint(0, 3, (V,), generator=g) * 2.0 ** -10
    x[6] = torch.randn(V, generator=g).sign() * 20
    x[7] = torch.randn(V, generator=g) * 2
    x[7] = torch.where(x[7] > 0, 0.0, -0.0)
    x[8, :V // 3] = -60000.0
    x[9] = torch.linspace(-30, 0, V)
    logits = x.to(TORCH[dt]).cuda()
    for n, f in enumerate(FILTERS):
        many = {key: [v] * B for key, v in f.items()}
        for T in (None, [0.05] * B, [40.0] * B):
            check(logits, uniforms(B, n), T, many.get("k"), many.get("p"), many.get("least"))


@pytest.mark.gpu
@pytest.mark.parametrize("V", [8, 256, 4096, 65536])
def test_borders_where_all_sums_are_exact(V):
    """Equal logits: every weight is one, u = i / V is exactly token i, and
    exact shares keep exact numbers of tokens."""
    u = [i / V for i in (0, 1, 2, V // 2 - 1, V // 2, V - 1)] + [float(np.nextafter(np.float32(1), np.float32(0)))]
    logits = torch.full((len(u), V), -2.5).cuda()
    token, _, _ = run(logits, param(u))
    assert token.tolist() == [0, 1, 2, V // 2 - 1, V // 2, V - 1, V - 1]
    n = len(u)
    # half of the mass: the first half of the tokens; u = i / (V / 2)
    token, prob, _ = run(logits, param([2 * v for v in u[:3]] + u[3:]), top_p=param([0.5] * n))
    assert token.tolist()[:3] == [0, 1, 2] and token.max() == V // 2 - 1
    assert torch.equal(prob.cpu(), torch.full((n,), 2.0 / V))
    token, prob, _ = run(logits, param([1.0] * n), top_k=param([V // 4] * n, torch.int32), top_p=param([0.5] * n))
    assert token.tolist() == [V // 8 - 1] * n and torch.equal(prob.cpu(), torch.full((n,), 8.0 / V))
    # just above half of it keeps one more
    token, _, _ = run(logits, param([1.0] * n), top_p=param([float(np.nextafter(np.float32(0.5), np.float32(1)))] * n))
    assert token.tolist() == [V // 2] * n
    # min_p of exactly the best's probability keeps what is equal to it
    token, _, _ = run(logits, param(u), min_p=param([1.0] * n))
    assert token.tolist() == [0, 1, 2, V // 2 - 1, V // 2, V - 1, V - 1]


@pytest.mark.gpu
def test_numbers_outside_count_as_the_nearest_inside():
    logits = normal(6, 500, "f32", 3).cuda()
    kw = dict(temperature=param([0.9] * 6))
    inside = run(logits, param([0.0, 0.0, float(np.nextafter(np.float32(1), np.float32(0)))] * 2), **kw)[0]
    assert torch.equal(run(logits, param([-1.0, -0.0, 1.0, float("-inf"), -3e38, float("inf")]), **kw)[0], inside)
    # filters beyond their range
    u = param(uniforms(6, 1))
    plain = run(logits, u)[0]
    assert torch.equal(run(logits, u, top_k=param([0, -1, 500, 501, 2 ** 31 - 1, -2 ** 31], torch.int32))[0], plain)
    assert torch.equal(run(logits, u, top_p=param([1.0, 1.5, 3e38, float("inf"), 1.0, 2.0]))[0], plain)
    assert torch.equal(run(logits, u, min_p=param([0.0, -1.0, -0.0, float("-inf"), -3e38, 0.0]))[0], plain)
    best = logits.argmax(dim=1).int()
    assert torch.equal(run(logits, u, top_p=param([0.0, -1.0, float("-inf"), 1e-30, -0.0, 1e-9]))[0], best)
    assert torch.equal(run(logits, u, min_p=param([1.0, 1.5, float("inf"), 3e38, 2.0, 1.0]))[0], best)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_extreme_temperatures_and_logits(dt):
    big = float(torch.finfo(TORCH[dt]).max)
    V = 700
    x = torch.randn(8, V, generator=torch.Generator().manual_seed(8))
    x[0], x[0, 400] = -big, big
    x[1] = -big
    x[2] = x[2] * big / 16
    x[3] = x[3] * float(torch.finfo(TORCH[dt]).tiny)
    x[4, ::2] = -big
    x[5, 5] = x[5, 600] = 30.0
    logits = x.to(TORCH[dt]).cuda()
    for T in (1e-30, 1e-6, 1.0, 1e6, 1e30, 3e38):
        for f in (dict(), dict(k=30), dict(k=300), dict(p=0.6), dict(k=400, p=0.3), dict(least=0.5)):
            many = {key: [v] * 8 for key, v in f.items()}
            check(logits, uniforms(8, 2), [T] * 8, many.get("k"), many.get("p"), many.get("least"))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_greedy_rows_take_the_first_of_the_best(dt):
    logits = normal(6, 9001, dt, 5)
    logits[0, 77] = logits[0, 8999] = 50.0
    logits[1, 9000] = logits[1, 4500] = 40.0
    logits[2] = 0
    logits[3, 1:] = float("-inf")
    u = uniforms(6, 4)
    token = check(logits.cuda(), u, [0.0] * 6, [50] * 6, [0.5] * 6)
    assert token.tolist()[:4] == [77, 4500, 0, 0]
    # greedy and drawn rows in one batch
    check(logits.cuda(), u, [0.0, 1.0] * 3)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [50, 20000])
def test_rows_without_a_distribution_are_reported_and_leave_the_others(V):
    logits = normal(9, V, "f32", 1)
    logits[1, 7] = float("nan")
    logits[2, V - 1] = float("inf")
    logits[3] = float("-inf")
    logits[8, 0] = float("nan")
    T = [1.0, 1.0, 1.0, 1.0, -1.0, float("nan"), float("inf"), 0.5, 0.0]
    token = check(logits.cuda(), uniforms(9, 1), T)
    assert token.tolist()[1:7] == [-1] * 6 and token[8] == -1 and token[0] >= 0 and token[7] >= 0
    good = normal(3, V, "f32", 2).cuda()
    nan = float("nan")
    for kw in (dict(top_p=param([0.5, nan, 0.5])), dict(min_p=param([0.1, nan, 0.1]))):
        t, q, status = run(good, param([0.3, 0.3, 0.3]), **kw)
        assert t[1] == -1 and q[1] == 0 and t[0] >= 0 and t[2] >= 0 and status == (1, 1)
    t, _, status = run(good, param([0.3, 0.3, nan]))
    assert t[2] == -1 and t[0] >= 0 and status == (1, 2)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_rows_at_any_address(dt):
    """Rows apart by odd strides, from every offset to a 16-byte boundary; what lies
    between them is not read."""
    for V in (1, 2, 9, 1001, 33333):
        for off in range(0, 9, 1 if V < 1000 else 3):
            buf = torch.full((5, V + off + 3), float("nan"), dtype=TORCH[dt])
            buf[:, off:off + V] = normal(5, V, dt, V + off)
            rows = buf.cuda()[:, off:off + V]
            assert rows.stride(0) == V + off + 3
            check(rows, uniforms(5, off), [0.9] * 5, [60] * 5, [0.9] * 5)
            check(rows, uniforms(5, off), [0.9] * 5)
            check(rows, uniforms(5, off), [0.0] * 5)


@pytest.mark.gpu
def test_a_row_gets_the_same_token_in_any_batch():
    """Splits of a row over CTAs follow the batch; sums do not depend on them."""
    V = 60000
    logits = normal(300, V, "bf16", 9).cuda()
    u = param(uniforms(300, 9))
    for f in (dict(), dict(top_p=0.95), dict(top_k=600), dict(top_k=30, top_p=0.8)):
        kw = {key: param([v] * 300, torch.int32 if key == "top_k" else torch.float32) for key, v in f.items()}
        token, prob, _ = run(logits, u, **kw)
        for n in (1, 2, 7, 40, 150):
            t, q, _ = run(logits[:n], u[:n].contiguous(), **{key: v[:n].contiguous() for key, v in kw.items()})
            assert torch.equal(t, token[:n]) and torch.equal(q, prob[:n])
        t, q, _ = run(logits, u, **kw)
        assert torch.equal(t, token) and torch.equal(q, prob)


@pytest.mark.gpu
def test_frequencies_follow_the_probabilities():
    """Evenly spaced numbers: every token is drawn as often as its share says, to
    one draw at either end."""
    V, n = 12, 4096
    x = torch.linspace(0, 3, V)
    logits = x.repeat(n, 1).cuda()
    u = ((torch.arange(n) + 0.5) / n).cuda()
    token = run(logits, u)[0].long().cpu()
    share = torch.softmax(x.double(), 0) * n
    assert ((torch.bincount(token, minlength=V).double() - share).abs() <= 1).all()
    assert bool((token[1:] >= token[:-1]).all())
