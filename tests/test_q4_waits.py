"""Waits of the 4-bit products on the tensor cores and of sampling that have to give
up: with a limit of a nanosecond, and inputs that are not in the L2 cache, a
wait whose first tries fail is the last.  A try lasts about as long as one copy alone takes, so that
sizes are such that copies or products queue, and a call is repeated until it reports a wait, 20 times at
most.  It writes nothing outside its outputs and workspace, and the next call is right bit for
bit.  (The limit is a host setting; every wait ends.)"""

import pytest
import torch

from contextual_sparsity_decode_gb300 import binding as dv

from dvtest import TORCH
from test_guards import Guarded, _ws
from test_q4 import lists, matrix, vectors
from test_sample import param, uniforms

pytestmark = pytest.mark.gpu
TIMEOUT = 6


def gives_up(call, outputs, ws, codes):
    """`call` with the shortest limit reports a wait of the kernels whose waits have these
    numbers; the call after it repeats the one before it."""
    big = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    call()
    assert dv.dv_check(ws.t) == (0, 0)
    want = [o.t.clone() for o in outputs]
    found = []
    prev = dv.dv_set_wait_limit_ns(1)
    try:
        while len(found) < 20 and TIMEOUT not in (status for status, _ in found):
            big.fill_(1)
            torch.cuda.synchronize()
            call()
            found.append(dv.dv_check(ws.t))
    finally:
        dv.dv_set_wait_limit_ns(prev)
    late = [info for status, info in found if status == TIMEOUT]
    assert late and all(info in codes for info in late), found
    assert all(status in (0, TIMEOUT) for status, _ in found), found
    for o in outputs:
        o.t.zero_()
    call()
    assert dv.dv_check(ws.t) == (0, 0)
    assert all(torch.equal(o.t, w) and o.intact() for o, w in zip(outputs, want)) and ws.intact()


@pytest.mark.tc
@pytest.mark.parametrize("dt,B,N,d,group", [("bf16", 8, 40000, 1024, 64), ("f16", 32, 25600, 2048, 128), ("f32", 9, 30000, 1024, 64),
                                            ("f16", 16, 9000, 5120, 64)])
def test_products_of_many_rows(dt, B, N, d, group):
    W, y = matrix(N, d, dt, group), vectors(B, d, dt)
    out, ws = Guarded((B, N), torch.float32), _ws(dv.dv_q4_matvec_workspace_size(B, d, N))
    gives_up(lambda: dv.dv_q4_matvec(y, W, out.t, ws.t), [out], ws, range(71, 77))


@pytest.mark.tc
@pytest.mark.parametrize("dt,B,N,d,k,group", [("f16", 9, 30000, 4096, 4000, 128), ("bf16", 20, 30000, 2056, 4000, 64)])
def test_both_products_of_the_mlp(dt, B, N, d, k, group):
    W1, W2, y = matrix(N, d, dt, group, 1), matrix(N, d, dt, group, 2), vectors(B, d, dt)
    idx, cnt = (t.cuda() for t in lists(B, N, k))
    out, ws = Guarded((B, d), torch.float32), _ws(dv.dv_q4_sparse_mlp_workspace_size(B, d, N, k))
    gives_up(lambda: dv.dv_q4_sparse_mlp(y, W1, W2, idx, cnt, out.t, ws.t), [out], ws, [*range(71, 77), *range(81, 87)])


@pytest.mark.tc
@pytest.mark.parametrize("dt,B,N,d,k,group", [("bf16", 8, 12000, 2048, 6000, 64), ("f16", 16, 7000, 4096, 3000, 128),
                                              ("f32", 32, 5000, 1024, 3000, 64)])
def test_the_second_product(dt, B, N, d, k, group):
    """(Few rows: the first one has no waits.  The codes of W2 are read from the host's
    memory: from the GPU's they come within the first try.)"""
    W1, W2, y = matrix(N, d, dt, group, 1), matrix(N, d, dt, group, 2), vectors(B, d, dt)
    idx, cnt = (t.cuda() for t in lists(B, N, k))
    far = W2.q.cpu().pin_memory()
    W2.c = dv.dv_q4(far.data_ptr(), W2.scale.data_ptr(), group)
    out, ws = Guarded((B, d), torch.float32), _ws(dv.dv_q4_sparse_mlp_workspace_size(B, d, N, k))
    gives_up(lambda: dv.dv_q4_sparse_mlp(y, W1, W2, idx, cnt, out.t, ws.t), [out], ws, range(81, 87))


@pytest.mark.parametrize("dt,B,V", [("f32", 60, 500000), ("bf16", 200, 60000), ("f16", 100, 524288)])
@pytest.mark.parametrize("kw", [dict(), dict(top_k=40), dict(top_p=0.9)])
def test_the_samplers_copies(dt, B, V, kw):
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = (torch.randn(B, V, device="cuda", generator=g) * 3).to(TORCH[dt])   # more than 20 MB
    u = param(uniforms(B, 2))
    args = {k: param([v] * B, torch.int32 if k == "top_k" else torch.float32) for k, v in kw.items()}
    token, prob, ws = Guarded((B,), torch.int32), Guarded((B,), torch.float32), _ws(dv.dv_sample_workspace_size(B, V))
    gives_up(lambda: dv.dv_sample(logits, u, token.t, ws.t, prob=prob.t, **args), [token, prob], ws, [61])


def test_a_limit_of_a_millisecond_is_not_met_by_a_call_in_order():
    """(The shortest with tries before the timer is read.)"""
    B, N, d = 8, 40000, 1024
    W, y = matrix(N, d, "bf16", 64), vectors(B, d, "bf16")
    ws = dv.workspace(dv.dv_q4_matvec_workspace_size(B, d, N))
    out, again = torch.zeros(B, N, device="cuda"), torch.zeros(B, N, device="cuda")
    dv.dv_q4_matvec(y, W, out, ws)
    prev = dv.dv_set_wait_limit_ns(1_000_000)
    try:
        dv.dv_q4_matvec(y, W, again, ws)
    finally:
        dv.dv_set_wait_limit_ns(prev)
    assert dv.dv_check(ws) == (0, 0) and torch.equal(out, again)
