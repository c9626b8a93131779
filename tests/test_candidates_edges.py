"""Operators for several candidates per sequence at sizes that take their less
common branches, against the same references in 64 bits.

Relative error of a row's sum of exponentials, and so the error of its
log-sum-exp, whatever the row (half-steps of 2^-24): the terms, and the scalings
of a warp's, a block's and a part's sum are exponentials of 2^-22 each, 4 x 4; a
thread's sum is scaled by one when the maximum rises by 1, at most 16 times
before what it held is below the new maximum's term alone (e^-16 2^22 < 1), 5 with
its product's rounding: 16 x 5; arguments, up to 22 in all (lower terms do not
count), are rounded three times, 3 x 22; a tile's 16 terms take five additions,
the running sum stays within 2, a part's 256 sums take eight: 15.  Together 177
half-steps; a score is rounded once more."""

import math

import numpy as np
import pytest
import torch

from contextual_sparsity_decode_gb300 import binding as dv
from test_candidates import DT, Case, _beam_ref, _cache, _compact_ref, _copy, _gen, _i32, _same
from test_guards import Guarded

pytestmark = pytest.mark.gpu

TIMEOUT = 6
LSE_TOL = 177 * 2.0 ** -24


def _select(logits, cum, K, done=None, end=0):
    S, W, V = logits.shape
    ws = dv.workspace(dv.dv_beam_select_workspace_size(S, W, V, K))
    score = torch.full((S, K), float("nan"), device="cuda")
    token, beam = (torch.full((S, K), -1, dtype=torch.int32, device="cuda") for _ in range(2))
    dv.dv_beam_select(logits, cum, score, token, beam, ws, done=done, end_token=end)
    assert dv.dv_check(ws) == (0, 0)
    return score, token, beam


def _beam_check(logits, cum, K, done=None, end=0):
    """Tokens and beams exactly, scores within LSE_TOL and their rounding."""
    rs, rt, rb = _beam_ref(logits, cum, K, None if done is None else done.cpu().numpy(), end)
    score, token, beam = _select(logits, cum, K, done, end)
    assert np.array_equal(token.cpu().numpy(), rt) and np.array_equal(beam.cpu().numpy(), rb)
    got = score.double().cpu().numpy()
    fine = np.isfinite(rs)
    assert np.array_equal(fine, np.isfinite(got)) and (got[~fine] == -np.inf).all()
    assert (np.abs(got[fine] - rs[fine]) <= 2.0 ** -24 * np.abs(rs[fine]) + LSE_TOL).all()


def test_beam_sums_do_not_lose_bits_with_the_vocabulary():
    """304 rows of 2^22 tokens, one part each: 0 for the first 4096, then one
    value -u for the rest, another for every row.  A running fp32 sum rounds the
    same way at every step (up to 1e-5 in all).

    Tolerance of a score: its own rounding, 2^-24 relative, and the
    log-sum-exp's relative error: an exponential, 2^-22 (two units in the last
    place), its argument, |u| <= 0.6, below 2^-24; a tile's 16 terms, five
    additions; the running sum, kept to 2 x 2^-24; a part's 256 sums, eight
    additions: 4 + 1 + 5 + 2 + 8 = 20 half-steps of 2^-24."""
    S, W, V, K = 38, 8, 1 << 22, 8
    u = torch.arange(1, S * W + 1, device="cuda").float().div(512).view(S, W)       # exact in f16
    logits = (-u)[:, :, None].expand(S, W, V).to(torch.float16).contiguous()
    logits[:, :, :4096] = 0
    score, token, beam = _select(logits, torch.zeros(S, W, device="cuda"), K)
    lse = (4096 + (V - 4096) * torch.exp(-u.double())).log()                        # descends with u
    assert (beam == W - 1).all() and torch.equal(token, torch.arange(K, device="cuda").int().expand(S, K))
    want = -lse[:, -1:]
    err = (score.double() - want).abs() - (2.0 ** -24 * want.abs() + 20 * 2.0 ** -24)
    assert err.max() <= 0, err.max()
    # every row, as the only beam of its sequence
    score, _, _ = _select(logits.view(S * W, 1, V), torch.zeros(S * W, 1, device="cuda"), 1)
    want = -lse.view(-1, 1)
    err = (score.double() - want).abs() - (2.0 ** -24 * want.abs() + 20 * 2.0 ** -24)
    assert err.max() <= 0, err.max()


def test_beam_sums_of_rows_that_rise():
    """The maximum grows with every tile, a little or by much, and the sum has
    to follow: logits a v / V for a = 0.01 ... 40."""
    rows, V = 304, 1 << 18
    a = torch.logspace(-2, math.log10(40), rows, device="cuda")
    x = (a[:, None] * (torch.arange(V, device="cuda") / V)[None]).view(rows, 1, V).contiguous()
    score, token, _ = _select(x, torch.zeros(rows, 1, device="cuda"), 1)
    lse = torch.logsumexp(x.double(), 2)
    top, at = x.max(2)
    want = top.double() - lse
    tol = 2.0 ** -24 * want.abs() + LSE_TOL
    assert ((score.double() - want).abs() <= tol).all()
    assert (x.gather(2, token.long()[:, :, None])[..., 0] == top).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_a_beam_s_tokens_are_in_the_order_of_their_logits(dt):
    """Logits so small that their scores are equal in double precision: whatever
    K is, a beam's tokens come by logit, and equal ones by index."""
    x = torch.zeros(1, 2, 40, device="cuda")
    x[0, :, 0], x[0, :, 7], x[0, :, 30] = 1e-20, 2e-20, 3e-20
    x[0, :, 1] = -1e-20
    order = [30, 7, 0, 2, 3, 4]
    for K in range(1, 7):
        score, token, beam = _select(x.to(DT[dt]), torch.tensor([[0.0, -1.0]], device="cuda"), K)
        assert token[0].tolist() == order[:K] and beam[0].tolist() == [0] * K
    many = torch.zeros(1, 32, 100, device="cuda")      # ... and where the candidates do not fit a list
    many[0, :, 0], many[0, :, 7] = 1e-20, 2e-20
    cum = torch.zeros(1, 32, device="cuda")
    _, token, beam = _select(many.to(DT[dt]), cum, 64)
    assert token[0].tolist() == [7, 0] + [v for v in range(64) if v not in (0, 7)] and (beam == 0).all()


@pytest.mark.parametrize("start", [16, 17, 2 ** 31 - 1])
def test_reorder_reports_errors_behind_the_last_position(start):
    """Nothing to move (the beams share everything): a parent that is none is
    reported all the same, and nothing changes."""
    kvs = _cache(2, 3, 2, 16, 64, "f16", 5)
    want = _copy(kvs)
    layers, ws = dv.KVLayers(kvs), dv.workspace(256)
    dv.dv_kv_reorder(layers, _i32([16, 16, 16]), _i32([[1, 3, 0]]), ws, start=_i32([start]))
    assert dv.dv_check(ws) == (5, 3)
    dv.dv_kv_reorder(layers, _i32([16, 17, 16]), _i32([[1, 1, 2]]), ws, start=_i32([start]))
    assert dv.dv_check(ws) == (9, 17)
    dv.dv_kv_reorder(layers, _i32([16, 16, 16]), _i32([[1, 2, 0]]), ws, start=_i32([start]))
    assert dv.dv_check(ws) == (0, 0)
    _same(kvs, want)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_beam_rows_off_a_boundary_over_many_tiles(dt):
    """Rows that begin off a 16-byte boundary, the first and the last at the very
    ends of their memory, and long enough that every stage of the ring is used
    again after tokens were stored to it one by one."""
    S, V, K = 304, 65537, 5
    big = torch.randn(S * V + 1, generator=_gen(71), device="cuda").to(DT[dt])
    _beam_check(big[1:].view(S, 1, V), -torch.rand(S, 1, generator=_gen(72), device="cuda"), K)


@pytest.mark.tc
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("d_h", [64, 128])
def test_tree_attention_waits_give_up(dt, d_h):
    """With a limit of a nanosecond the copies' producer gives up at a ring that
    the products have not freed (a CTA has several dozen tiles), and every other
    role behind it.  The call reports it, writes nothing outside its outputs,
    and the next one is right, bit for bit."""
    c = Case(dt, d_h, [4000] * 4, 64, 32, seed=41, n_max=4064)
    c.call()
    assert dv.dv_check(c.ws) == (0, 0)
    want = c.out.clone()
    out, ws = Guarded(tuple(c.out.shape), DT[dt]), Guarded((c.ws.numel(),), torch.uint8)
    c.out, c.ws = out.t, ws.t
    statuses = []
    prev = dv.dv_set_wait_limit_ns(1)
    try:
        for _ in range(3):
            c.call()
            statuses.append(dv.dv_check(c.ws)[0])
    finally:
        dv.dv_set_wait_limit_ns(prev)
    assert TIMEOUT in statuses and set(statuses) <= {0, TIMEOUT}, statuses
    c.out.zero_()
    c.call()
    assert dv.dv_check(c.ws) == (0, 0)
    assert torch.equal(c.out, want) and out.intact() and ws.intact()


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_beam_scan_waits_give_up(dt):
    """The same of the beam selection's scan: the logits are out of the L2 cache,
    and its first copy is still on its way."""
    big = torch.empty(1 << 29, dtype=torch.uint8, device="cuda")
    S, W, V, K = 6, 8, 60001, 16
    logits = torch.randn(S, W, V, generator=_gen(61), device="cuda").to(DT[dt])
    cum = -torch.rand(S, W, generator=_gen(62), device="cuda")
    ws = Guarded((dv.dv_beam_select_workspace_size(S, W, V, K),), torch.uint8)
    score = Guarded((S, K), torch.float32)
    token, beam = Guarded((S, K), torch.int32), Guarded((S, K), torch.int32)
    call = lambda: dv.dv_beam_select(logits, cum, score.t, token.t, beam.t, ws.t)  # noqa: E731
    call()
    assert dv.dv_check(ws.t) == (0, 0)
    want = [x.t.clone() for x in (score, token, beam)]
    statuses = []
    prev = dv.dv_set_wait_limit_ns(1)
    try:
        for _ in range(3):
            big.fill_(1)
            torch.cuda.synchronize()
            call()
            statuses.append(dv.dv_check(ws.t)[0])
    finally:
        dv.dv_set_wait_limit_ns(prev)
    assert TIMEOUT in statuses and set(statuses) <= {0, TIMEOUT}, statuses
    call()
    assert dv.dv_check(ws.t) == (0, 0)
    assert all(torch.equal(x.t, w) and x.intact() for x, w in zip((score, token, beam), want)) and ws.intact()


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [100, 9001])
def test_beam_more_equal_candidates_than_a_list_holds(dt, V):
    """32 beams of equal logits, 64 wanted: more than 1024 candidates reach the
    last place."""
    x = torch.zeros(2, 32, V, device="cuda", dtype=DT[dt])
    cum = torch.zeros(2, 32, device="cuda")
    cum[1, 5:] = -0.5
    _beam_check(x, cum, 64)
    x[:, ::3, V // 2] = 1.0
    done = torch.zeros(2, 32, dtype=torch.uint8, device="cuda")
    done[:, 1::4] = 1
    _beam_check(x, cum, 64, done, V // 3)


@pytest.mark.parametrize("dt,S,W,V,K", [("f16", 1, 2, 300001, 16), ("f32", 1, 1, 1000003, 64), ("bf16", 2, 2, 262145, 5),
                                        ("bf16", 1, 1, 4194304, 33)])
def test_beam_rows_of_many_parts(dt, S, W, V, K):
    """More parts a row than a warp has lanes."""
    g = _gen(V)
    x = (3 * torch.randn(S, W, V, generator=g, device="cuda")).to(DT[dt])
    cum = -torch.rand(S, W, generator=g, device="cuda")
    _beam_check(x, cum, K)
    x[..., :] = (torch.arange(V, device="cuda") // 50000).float().to(DT[dt])       # runs over several parts
    _beam_check(x, cum, K)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("K", [1, 7, 64])
def test_beam_lists_cut_back_inside_a_part(dt, K):
    """80 rows of 50003 tokens (parts of several tiles) that fill the lists of
    groups: ascending, descending, in runs, ties of a few values, the best in the
    hands of a few threads."""
    S, V = 80, 50003
    v = torch.arange(V, device="cuda")
    g = _gen(K)
    rows = torch.stack([
        v / V, -v / V, (v // 700 % 5).float(), (v // 4096).float(), (v % 4096 // 16).float(),
        torch.randint(0, 3, (V,), generator=g, device="cuda").float(),
        torch.where((v // 8) % 256 < 9, 4.0 + torch.randn(V, generator=g, device="cuda"), torch.full((V,), -4.0, device="cuda")),
        torch.where(v % 4096 > 2000, v / V, torch.full((V,), -float("inf"), device="cuda")),
    ])
    x = rows[torch.arange(S, device="cuda") % len(rows)][:, None].to(DT[dt]).contiguous()
    _beam_check(x, -torch.rand(S, 1, generator=g, device="cuda"), K)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B", [32, 33, 64, 70])
def test_tree_attention_of_many_sequences(dt, B):
    """Around and above the 32 sequences that a warp plans at once."""
    Case(dt, 64, [(29 * b) % 190 for b in range(B)], 4, 2, nodes=[(b * 7 + 1) % 5 for b in range(B)], mask="tree", seed=B).check()


@pytest.mark.parametrize("dt", ["f32", "f16"])
def test_tree_attention_of_the_largest_batch(dt):
    B = 512
    Case(dt, 64, [(b * 37) % 90 for b in range(B)], 2, 1, nodes=[(b * 5 + 1) % 3 for b in range(B)], mask=None, seed=3,
         heads=[[0] if b % 11 else [] for b in range(B)]).check()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_compact_of_long_lists(dt):
    """Lists of more entries than a warp reads at once, kept in place and from
    further back; lists that stop ascending where one read ends."""
    B, cap, n_max = 6, 70, 160
    up = list(range(0, 140, 2))
    lists = [list(range(64)), up[:33], up, list(range(3, 67)), up[:32] + [62] + up[33:40], up[:31] + [58, 70]]
    pos = [5, 0, 20, 90, 4, 6]
    kvs = _cache(2, B, 2, n_max, 64, dt, 77)
    want = _copy(kvs)
    idx = torch.zeros(B, cap, dtype=torch.int32)
    for b, x in enumerate(lists):
        idx[b, :len(x)] = torch.tensor(x, dtype=torch.int32)
    for b in range(4):
        _compact_ref(want, b, pos[b], lists[b])
    layers, ws, p = dv.KVLayers(kvs), dv.workspace(256), _i32(pos)
    dv.dv_kv_compact(layers, p, idx.cuda(), _i32([len(x) for x in lists]), ws, new_pos=p)
    assert dv.dv_check(ws)[0] == 5
    _same(kvs, want)
    assert p.tolist() == [a + len(x) for a, x in zip(pos[:4], lists)] + pos[4:]
