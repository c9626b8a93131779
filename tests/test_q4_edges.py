"""4-bit matrices and sampling at their edges: guard regions around what is
written, waits that give up, captured and replayed calls, other streams, launch
overlap, long lists and long rows.  Tolerances as in test_q4.py and test_sample.py."""

import numpy as np
import pytest
import torch

from contextual_sparsity_decode_gb300 import binding as dv

from dvtest import TORCH
from test_guards import Guarded, _ws
from test_q4 import EPS, lists, matrix, matvec_bound, mlp_reference, opened, vectors
from test_sample import normal, param, reference, uniforms

pytestmark = pytest.mark.gpu
TIMEOUT = 6


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B", [1, 2, 3, 9, 20, 32])
def test_nothing_is_written_outside(dt, B):
    N, d, k, group = 333, 456, 77, 64
    W1, W2, y = matrix(N, d, dt, group, 1), matrix(N, d, dt, 128, 2), vectors(B, d, dt)
    parts = [Guarded((B, N), torch.float32), _ws(dv.dv_q4_matvec_workspace_size(B, d, N)), Guarded((B, d), torch.float32),
             _ws(dv.dv_q4_sparse_mlp_workspace_size(B, d, N, k)), Guarded((B,), torch.int32), Guarded((B,), torch.float32),
             _ws(dv.dv_sample_workspace_size(B, N)), Guarded((N, 256), torch.uint8), Guarded((N, 8), TORCH[dt]),
             Guarded((N, d), TORCH[dt])]
    head, ws_h, out, ws_m, token, prob, ws_s, q, scale, values = (p.t for p in parts)
    dv.dv_q4_matvec(y, W1, head, ws_h)
    idx, cnt = lists(B, N, k)
    dv.dv_q4_sparse_mlp(y, W1, W2, idx.cuda(), cnt.cuda(), out, ws_m)
    for kw in (dict(), dict(top_k=param([20] * B, torch.int32)), dict(top_k=param([300] * B, torch.int32)),
               dict(top_p=param([0.9] * B)), dict(temperature=param([0.0] * B))):
        dv.dv_sample(head, param(uniforms(B, 1)), token, ws_s, prob=prob, **kw)
    W = (torch.randn(N, d, generator=torch.Generator().manual_seed(1)) * 0.1).to(TORCH[dt]).cuda()
    dv.dv_q4_quantize(W, dv.Q4(q, scale, d, 64), values=values)
    torch.cuda.synchronize()
    assert all(p.intact() for p in parts)
    for ws in (ws_h, ws_m, ws_s):
        assert dv.dv_check(ws) == (0, 0)


def test_nothing_is_written_outside_large():
    for B, N, d, k in ((1, 3000, 2048, 2500), (8, 2000, 1024, 400)):
        W1, W2, y = matrix(N, d, "f16", 128, 1), matrix(N, d, "f16", 64, 2), vectors(B, d, "f16")
        parts = [Guarded((B, N), torch.float32), _ws(dv.dv_q4_matvec_workspace_size(B, d, N)), Guarded((B, d), torch.float32),
                 _ws(dv.dv_q4_sparse_mlp_workspace_size(B, d, N, k))]
        dv.dv_q4_matvec(y, W1, parts[0].t, parts[1].t)
        idx, cnt = lists(B, N, k)
        dv.dv_q4_sparse_mlp(y, W1, W2, idx.cuda(), cnt.cuda(), parts[2].t, parts[3].t)
        torch.cuda.synchronize()
        assert all(p.intact() for p in parts)


@pytest.fixture
def shortest_wait():
    prev = dv.dv_set_wait_limit_ns(1)
    try:
        yield
    finally:
        dv.dv_set_wait_limit_ns(prev)


# A wait is first tried once, for as long as the hardware lets a try last, and the limit is
# looked at only if that try fails: at a limit of a nanosecond a call either gives up and says
# so, or has had all it waited for, and then it must be right.


def _gave_up(ws):
    status = dv.dv_check(ws)[0]
    assert status in (0, TIMEOUT)
    return status == TIMEOUT


@pytest.mark.parametrize("B,N,d", [(8, 40000, 1024), (32, 128 * 200, 2048)])
def test_the_tensor_core_products_waits_give_up(B, N, d, shortest_wait):
    W, y = matrix(N, d, "bf16", 64), vectors(B, d, "bf16")
    ws = dv.workspace(dv.dv_q4_matvec_workspace_size(B, d, N))
    out = torch.zeros(B, N, device="cuda")
    dv.dv_q4_matvec(y, W, out, ws)
    gave_up = _gave_up(ws)
    dv.dv_set_wait_limit_ns(0)
    first, second = torch.zeros(B, N, device="cuda"), torch.zeros(B, N, device="cuda")
    dv.dv_q4_matvec(y, W, first, ws)
    dv.dv_q4_matvec(y, W, second, dv.workspace(dv.dv_q4_matvec_workspace_size(B, d, N)))
    assert dv.dv_check(ws) == (0, 0) and torch.equal(first, second)
    assert gave_up or torch.equal(out, first)
    rows = torch.arange(0, N, 997)
    part = dv.Q4(W.q[rows.cuda()].contiguous(), W.scale[rows.cuda()].contiguous(), d, 64)
    W64, y64 = opened(part.q, part.scale, d, 64), y.double().cpu().numpy()
    assert np.all(np.abs(first.double().cpu().numpy()[:, rows] - y64 @ W64.T) <= matvec_bound(d, W64, y64))


def test_the_batched_mlp_after_a_wait_that_gave_up(shortest_wait):
    B, N, d, k = 9, 30000, 1024, 4000
    W1, W2, y = matrix(N, d, "f16", 128, 1), matrix(N, d, "f16", 128, 2), vectors(B, d, "f16")
    idx, cnt = (t.cuda() for t in lists(B, N, k))
    ws = dv.workspace(dv.dv_q4_sparse_mlp_workspace_size(B, d, N, k))
    out = torch.zeros(B, d, device="cuda")
    dv.dv_q4_sparse_mlp(y, W1, W2, idx, cnt, out, ws)
    gave_up = _gave_up(ws)
    dv.dv_set_wait_limit_ns(0)
    again, fresh = torch.zeros(B, d, device="cuda"), torch.zeros(B, d, device="cuda")
    dv.dv_q4_sparse_mlp(y, W1, W2, idx, cnt, again, ws)
    dv.dv_q4_sparse_mlp(y, W1, W2, idx, cnt, fresh, dv.workspace(dv.dv_q4_sparse_mlp_workspace_size(B, d, N, k)))
    assert dv.dv_check(ws) == (0, 0) and torch.equal(again, fresh)
    assert gave_up or torch.equal(out, fresh)


@pytest.mark.parametrize("B", [1, 200])
def test_the_samplers_waits_give_up(B, shortest_wait):
    V = 500000 if B == 1 else 60000
    logits, u = normal(B, V, "f32", 3).cuda(), param(uniforms(B, 2))
    ws = dv.workspace(256)
    token, prob = torch.full((B,), 5, dtype=torch.int32, device="cuda"), torch.ones(B, device="cuda")
    dv.dv_sample(logits, u, token, ws, prob=prob)
    gave_up = _gave_up(ws)
    late = token == -1
    assert bool(late.any()) == gave_up and bool((prob[late] == 0).all())
    early = token.clone()
    dv.dv_set_wait_limit_ns(0)
    dv.dv_sample(logits, u, token, ws, prob=prob)
    assert dv.dv_check(ws) == (0, 0)
    assert torch.equal(token[~late], early[~late])
    x = logits.double().cpu().numpy()
    for b in range(0, B, 23):
        assert int(token[b]) == reference(x[b], float(u[b]))[0]


@pytest.mark.parametrize("B,dt", [(1, "f16"), (2, "bf16"), (6, "f16"), (4, "f32"), (20, "bf16")])
def test_captured_calls_take_new_inputs(B, dt):
    N, d, k = 700, 512, 90
    W1, W2, y = matrix(N, d, dt, 64, 1), matrix(N, d, dt, 128, 2), vectors(B, d, dt)
    idx, cnt = (t.cuda() for t in lists(B, N, k))
    u = param(uniforms(B, 0))
    ws = [dv.workspace(n) for n in (dv.dv_q4_matvec_workspace_size(B, d, N), dv.dv_q4_sparse_mlp_workspace_size(B, d, N, k), 256)]
    head, out, token = torch.zeros(B, N, device="cuda"), torch.zeros(B, d, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    p = param([0.9] * B)

    def calls(head, out, token, ws):
        dv.dv_q4_sparse_mlp(y, W1, W2, idx, cnt, out, ws[1])
        dv.dv_q4_matvec(y, W1, head, ws[0])
        dv.dv_sample(head, u, token, ws[2], top_p=p)

    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            calls(head, out, token, ws)
    torch.cuda.current_stream().wait_stream(s)
    for n in range(3):
        y.copy_(vectors(B, d, dt, n + 1))
        idx.copy_(lists(B, N, k, seed=n + 1)[0])
        u.copy_(param(uniforms(B, n + 1)))
        graph.replay()
        want = torch.zeros_like(head), torch.zeros_like(out), torch.zeros_like(token)
        calls(*want, [dv.workspace(w.numel()) for w in ws])
        assert torch.equal(head, want[0]) and torch.equal(out, want[1]) and torch.equal(token, want[2])


def test_two_streams_with_their_own_workspaces():
    B, N, d, k = 4, 3000, 1024, 500
    W1, W2 = matrix(N, d, "f16", 128, 1), matrix(N, d, "f16", 128, 2)
    work = []
    for n in range(2):
        y = vectors(B if n else 1, d, "f16", n)
        b = y.shape[0]
        idx, cnt = (t.cuda() for t in lists(b, N, k, seed=n))
        out, head = torch.zeros(b, d, device="cuda"), torch.zeros(b, N, device="cuda")
        ws = dv.workspace(dv.dv_q4_sparse_mlp_workspace_size(b, d, N, k)), dv.workspace(dv.dv_q4_matvec_workspace_size(b, d, N))
        work.append((y, idx, cnt, out, head, ws, torch.cuda.Stream()))

    def calls(y, idx, cnt, out, head, ws, stream):
        dv.dv_q4_sparse_mlp(y, W1, W2, idx, cnt, out, ws[0], stream=stream)
        dv.dv_q4_matvec(y, W1, head, ws[1], stream=stream)

    want = []
    for w in work:
        calls(*w[:-1], None)
        torch.cuda.synchronize()
        want.append((w[3].clone(), w[4].clone()))
        w[3].zero_(), w[4].zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for w in work:
            calls(*w)
    torch.cuda.synchronize()
    for w, (out, head) in zip(work, want):
        assert torch.equal(w[3], out) and torch.equal(w[4], head)


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_launch_overlap_changes_nothing(dt):
    """Layer norm, sparse MLP, layer norm, ... at level 1, as a decoder orders them."""
    N, d, k, layers = 600, 512, 200, 6
    W = [(matrix(N, d, dt, 128, 2 * l), matrix(N, d, dt, 64, 2 * l + 1)) for l in range(layers)]
    idx = [tuple(t.cuda() for t in lists(1, N, k, seed=l)) for l in range(layers)]
    x0 = torch.randn(1, d, generator=torch.Generator().manual_seed(1)).cuda()
    ws = dv.workspace(dv.dv_q4_sparse_mlp_workspace_size(1, d, N, k))
    got = []
    for level in (0, 1, 1):
        prev = dv.dv_set_launch_overlap(level)
        try:
            x = x0.clone()
            ys = [torch.zeros(1, d, dtype=TORCH[dt], device="cuda") for _ in range(layers)]
            for l in range(layers):
                dv.dv_layernorm(x, ys[l])
                dv.dv_q4_sparse_mlp(ys[l], *W[l], *idx[l], x, ws, accumulate=True)
        finally:
            dv.dv_set_launch_overlap(prev)
        got.append(x.clone())
    assert dv.dv_check(ws) == (0, 0)
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


def gpu_opened(W, rows):
    """Weights of some rows in 64 bits, on the GPU."""
    t = torch.arange(W.d, device="cuda")
    bit = 4 * (t % 8 // 2) + 16 * (t % 2)
    byte = t // 128 * 64 + 4 * (2 * (t % 64 // 8) + t % 128 // 64) + bit // 8
    return (((W.q[rows][:, byte] >> (bit % 8).to(torch.uint8)) & 15).double() - 8) * W.scale[rows][:, t // W.group].double()


@pytest.mark.parametrize("B,N,d,k,group", [(1, 12000, 16384, 12000, 64), (1, 300, 32768, 150, 64), (2, 100, 32768, 60, 128),
                                           (3, 64, 32768, 40, 64), (2, 65536, 64, 65536, 64), (32, 65536, 64, 3000, 128)])
def test_long_lists_and_long_rows(B, N, d, k, group):
    dt = "bf16"
    W1, W2, y = matrix(N, d, dt, group, 1), matrix(N, d, dt, group, 2), vectors(B, d, dt)
    idx, cnt = lists(B, N, k)
    ws = dv.workspace(dv.dv_q4_sparse_mlp_workspace_size(B, d, N, k))
    out = torch.zeros(B, d, device="cuda")
    dv.dv_q4_sparse_mlp(y, W1, W2, idx.cuda(), cnt.cuda(), out, ws)
    assert dv.dv_check(ws) == (0, 0)
    blocks, union = (d + 127) // 128, min(N, B * k)
    for b in range(B):
        ref, tol = torch.zeros(d, dtype=torch.float64, device="cuda"), torch.zeros(d, dtype=torch.float64, device="cuda")
        for n in range(0, k, 1000):
            rows = idx[b, n:n + 1000].long().cuda()
            A, C, x = gpu_opened(W1, rows), gpu_opened(W2, rows), y[b].double()
            a = torch.relu(A @ x)
            off = (160 + 4 * blocks) * EPS * (A.abs() @ x.abs())
            ref += a @ C
            tol += off @ C.abs() + (3 * 17 * (union // 16 + 1) + 32) * EPS * ((a + off) @ C.abs())
        assert bool(((out[b].double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("B,d,dt", [(1, 32768, "f32"), (2, 32768, "bf16"), (32, 32768, "f16"), (5, 32768, "f32"), (1, 8, "f16"),
                                    (3, 64, "bf16"), (3, 56, "bf16")])
def test_matvec_of_the_longest_and_shortest_rows(B, d, dt):
    N = 40
    W, y = matrix(N, d, dt, 128), vectors(B, d, dt)
    out = torch.zeros(B, N, device="cuda")
    dv.dv_q4_matvec(y, W, out, dv.workspace(dv.dv_q4_matvec_workspace_size(B, d, N)))
    W64, y64 = opened(W.q, W.scale, d, 128), y.double().cpu().numpy()
    assert np.all(np.abs(out.double().cpu().numpy() - y64 @ W64.T) <= matvec_bound(d, W64, y64))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_vectors_of_very_different_elements(dt):
    """Outliers, tiny vectors and tiny parts of vectors (a group's unit follows its
    largest element: the error is of that, per element)."""
    N, d = 60, 1024
    W = matrix(N, d, dt, 128)
    W64 = opened(W.q, W.scale, d, 128)
    y = torch.randn(6, d, generator=torch.Generator().manual_seed(2))
    y[0, 7] = 3000.0
    y[1] *= 2.0 ** -12
    y[2, ::3] *= 2.0 ** -10
    y[3, 128:] = 0
    y[4] = 0
    y[5] *= torch.linspace(-8, 4, d).exp2()
    y = y.to(TORCH[dt]).cuda()
    for b in range(6):
        one = y[b:b + 1].contiguous()
        out = torch.zeros(1, N, device="cuda")
        dv.dv_q4_matvec(one, W, out, dv.workspace(dv.dv_q4_matvec_workspace_size(1, d, N)))
        x = one.double().cpu().numpy()
        # 2^-31 of the group's largest magnitude for each element
        top = np.abs(x).reshape(1, -1, 128).max(axis=2).repeat(128, axis=1)
        slack = 2.0 ** -31 * top @ np.abs(W64).T
        assert np.all(np.abs(out.double().cpu().numpy() - x @ W64.T) <= matvec_bound(d, W64, x) + slack)


@pytest.mark.parametrize("B", [1, 2, 5])
def test_units_at_the_ends_of_the_range(B):
    """Large scales with small vectors and the other way round: products that fit."""
    N, d = 24, 256
    for up in (2.0 ** 118, 2.0 ** -118):
        W = matrix(N, d, "f32", 128)
        W.scale.mul_(up)
        y = (torch.randn(B, d, generator=torch.Generator().manual_seed(1)) / up).cuda()
        out = torch.zeros(B, N, device="cuda")
        dv.dv_q4_matvec(y, W, out, dv.workspace(dv.dv_q4_matvec_workspace_size(B, d, N)))
        W64, y64 = opened(W.q, W.scale, d, 128), y.double().cpu().numpy()
        assert np.all(np.abs(out.double().cpu().numpy() - y64 @ W64.T) <= matvec_bound(d, W64, y64))


@pytest.mark.parametrize("B,dt", [(1, "f16"), (2, "bf16"), (4, "f32"), (7, "f16"), (20, "bf16")])
def test_lists_in_any_order(B, dt):
    """The same rows in descending order and shuffled: entries of a list are a set."""
    N, d, k = 400, 384, 90
    W1, W2, y = matrix(N, d, dt, 64, 1), matrix(N, d, dt, 128, 2), vectors(B, d, dt)
    idx, cnt = lists(B, N, k)
    ref, tol = mlp_reference(y, W1, W2, idx, cnt)
    for order in (torch.arange(k).flip(0), torch.randperm(k, generator=torch.Generator().manual_seed(5))):
        out = torch.zeros(B, d, device="cuda")
        dv.dv_q4_sparse_mlp(y, W1, W2, idx[:, order].contiguous().cuda(), cnt.cuda(), out,
                            dv.workspace(dv.dv_q4_sparse_mlp_workspace_size(B, d, N, k)))
        assert np.all(np.abs(out.double().cpu().numpy() - ref) <= tol)


@pytest.mark.parametrize("B,dt", [(3, "f16"), (8, "bf16"), (20, "f16"), (4, "f32"), (2, "f16")])
def test_one_vectors_nan_is_its_own(B, dt):
    """A NaN in one vector, and a row with a NaN scale that only another
    vector's list names, leave the others' results as they were."""
    N, d, k = 300, 256, 40
    W1, W2, y = matrix(N, d, dt, 128, 1), matrix(N, d, dt, 64, 2), vectors(B, d, dt)
    y[1, 5] = float("nan")
    idx, cnt = lists(B, N, k)
    row = int(idx[1, 0])
    idx[0] = torch.tensor([j for j in range(N) if j != row][:k])
    if B > 2:
        idx[2:] = idx[0]
    W2.scale[row] = float("nan")
    ws = dv.workspace(dv.dv_q4_sparse_mlp_workspace_size(B, d, N, k))
    out, head = torch.zeros(B, d, device="cuda"), torch.zeros(B, N, device="cuda")
    dv.dv_q4_sparse_mlp(y, W1, W2, idx.cuda(), cnt.cuda(), out, ws)
    dv.dv_q4_matvec(y, W1, head, dv.workspace(dv.dv_q4_matvec_workspace_size(B, d, N)))
    others = [b for b in range(B) if b != 1]
    assert bool(torch.isnan(head[1]).all()) and bool(torch.isnan(out[1]).all())
    W64, y64 = opened(W1.q, W1.scale, d, 128), y[others].double().cpu().numpy()
    assert np.all(np.abs(head[others].double().cpu().numpy() - y64 @ W64.T) <= matvec_bound(d, W64, y64))
    W2.scale[row] = 1.0   # (no list of the others names it)
    ref, tol = mlp_reference(y[others], W1, W2, idx[others], cnt[others])
    assert np.all(np.abs(out[others].double().cpu().numpy() - ref) <= tol)


# ---- three and more vectors with many rows (tensor cores), in 64 bits on the GPU


def opened_on_gpu(W):
    return torch.cat([gpu_opened(W, torch.arange(n, min(W.N, n + 4096), device="cuda")) for n in range(0, W.N, 4096)])


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("B,N,d,group", [
    (2, 8300, 20000, 64), (3, 8300, 64, 64), (3, 8300, 72, 128), (8, 8321, 512, 64), (5, 9000, 520, 128), (8, 19456, 1000, 128), (7, 19457, 136, 64),
    (9, 5200, 1096, 64), (16, 5200, 128, 128), (16, 12345, 2056, 64), (17, 3700, 200, 64), (32, 3700, 1544, 128),
    (32, 9999, 640, 64), (31, 39000, 328, 128), (20, 4000, 5000, 64)])
def test_matvec_of_many_rows(dt, B, N, d, group):
    W, y = matrix(N, d, dt, group, 1), vectors(B, d, dt)
    ws = dv.workspace(dv.dv_q4_matvec_workspace_size(B, d, N))
    out = torch.full((B, N), float("nan"), device="cuda")
    dv.dv_q4_matvec(y, W, out, ws)
    W64, y64, blocks = opened_on_gpu(W), y.double(), (d + 127) // 128
    ref = y64 @ W64.T
    # (a cut tile's parts are added in fp32, one rounding each: fewer than the blocks)
    tol = (160 + 5 * blocks) * EPS * (y64.abs() @ W64.abs().T) + 1e-38
    assert bool(((out.double() - ref).abs() <= tol).all())
    again, more = torch.empty(B, N, device="cuda"), torch.ones(B, N, device="cuda")
    dv.dv_q4_matvec(y, W, again, ws)
    assert torch.equal(out, again)
    dv.dv_q4_matvec(y, W, more, ws, accumulate=True)
    assert torch.equal(more, out + 1)
    assert dv.dv_check(ws) == (0, 0)


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("B,N,d,k,groups", [(3, 20000, 328, 4200, (64, 128)), (8, 30000, 1024, 1600, (128, 64)), (16, 20000, 136, 500, (64, 64)),
                                            (32, 16000, 520, 200, (128, 128)), (25, 9000, 64, 9000, (64, 128))])
def test_mlp_of_many_rows(dt, B, N, d, k, groups):
    W1, W2, y = matrix(N, d, dt, groups[0], 1), matrix(N, d, dt, groups[1], 2), vectors(B, d, dt)
    idx, cnt = lists(B, N, k, counts=[0, k + 5] + [k - 3 * (b % 7) for b in range(B - 2)])
    idx[2, 3] = N                                   # outside: skipped
    ws = dv.workspace(dv.dv_q4_sparse_mlp_workspace_size(B, d, N, k))
    out = torch.zeros(B, d, device="cuda")
    dv.dv_q4_sparse_mlp(y, W1, W2, idx.cuda(), cnt.cuda(), out, ws)
    status, _ = dv.dv_check(ws)
    assert status != 0
    A, C = opened_on_gpu(W1), opened_on_gpu(W2)
    blocks, union = (d + 127) // 128, min(N, B * k)
    for b in range(B):
        rows = idx[b, :min(int(cnt[b]), k)].long()
        rows = rows[rows < N].cuda()
        x = y[b].double()
        a = torch.relu(A[rows] @ x)
        off = (160 + 4 * blocks) * EPS * (A[rows].abs() @ x.abs())
        tol = off @ C[rows].abs() + (3 * 17 * (union // 16 + 1) + 32) * EPS * ((a + off) @ C[rows].abs()) + 1e-38
        assert bool(((out[b].double() - a @ C[rows]).abs() <= tol).all())
    assert bool((out[0] == 0).all())


def test_one_vectors_nan_is_its_own_with_many_rows():
    B, N, d = 12, 9001, 384
    W, y = matrix(N, d, "bf16", 64), vectors(B, d, "bf16")
    W.scale[4321] = float("nan")
    y[5, 100] = float("inf")
    out = torch.zeros(B, N, device="cuda")
    dv.dv_q4_matvec(y, W, out, dv.workspace(dv.dv_q4_matvec_workspace_size(B, d, N)))
    finite = torch.isfinite(out)
    finite[5], finite[:, 4321] = True, True
    assert bool(finite.all()) and bool(torch.isnan(out[:, 4321]).all()) and not bool(torch.isfinite(out[5]).any())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("counts", [(0, 0, 0, 0), (0, 1, 0, 0), (3, -5, 60, 0), (0, 0, 0, 4400)])
def test_short_lists_under_a_large_bound(dt, counts):
    """Lists that leave most CTAs of a grid sized for their bound without rows."""
    B, N, d, k = 4, 20000, 264, 4400
    W1, W2, y = matrix(N, d, dt, 64, 1), matrix(N, d, dt, 128, 2), vectors(B, d, dt)
    idx, cnt = lists(B, N, k, counts=list(counts))
    start = torch.randn(B, d, generator=torch.Generator().manual_seed(3)).cuda()
    ws = dv.workspace(dv.dv_q4_sparse_mlp_workspace_size(B, d, N, k))
    out, more = torch.full((B, d), float("nan"), device="cuda"), start.clone()
    dv.dv_q4_sparse_mlp(y, W1, W2, idx.cuda(), cnt.cuda(), out, ws)
    dv.dv_q4_sparse_mlp(y, W1, W2, idx.cuda(), cnt.cuda(), more, ws, accumulate=True)
    ref, tol = mlp_reference(y, W1, W2, idx, cnt.clamp(min=0))
    assert np.all(np.abs(out.double().cpu().numpy() - ref) <= tol)
    assert torch.equal(more, start + out)
    assert dv.dv_check(ws) == (0, 0)
