"""Matrices in 4 bits against plain forms in 64 bits: quantisation, products
with every row, the sparse MLP over listed rows.

Tolerances.  A code less 8 times a 16-bit factor, or a 16-bit piece of a 32-bit
one, is exact in fp32, and the pieces add up to the factor, so only sums round.
An m16n8k16 product adds 17 numbers and may drop what is below 2^-24 of the
largest of each: 17 x 2^-24 of the sum of magnitudes.  A group of 128 is a chain
of 8 of them; then come one product with the scale and one sum per group (at most
two groups a block), and 24 sums over warps and pieces, 2^-24 each:
(136 + 4 blocks + 24) 2^-24 sum |w y|.  A product of 128 elements at once on the
tensor cores' accumulators is the same chain of 8.  The integer products of one
and two vectors are exact; their fixed point is off by 2^-31 of the largest of a
group for each element, 2^-31 128 of the group's largest magnitude times its
largest weight at most, which the normal vectors here stay far below 136 2^-24 of the
sum with, and a conversion, a product and a sum a group are 4 2^-24 a block.  The second product of the MLP is a chain
of three products for each 16 rows a warp meets (all of them, at most), one
rounding of a_j s each, and sums over 8 warps, 8 CTAs and 3 pieces, on top of what
its activations are off by."""

import numpy as np
import pytest
import torch

from contextual_sparsity_decode_gb300 import binding as dv

from dvtest import TORCH

EPS = 2.0 ** -24


def opened(q, scale, d, group):
    """Weights [N][d] in 64 bits, element by element from the layout."""
    q, s = q.cpu().numpy().astype(np.int64), scale.double().cpu().numpy()
    t = np.arange(d)
    k = 2 * (t % 64 // 8) + t % 128 // 64          # word of the block
    bit = 4 * (t % 8 // 2) + 16 * (t % 2)
    code = (q[:, t // 128 * 64 + 4 * k + bit // 8] >> (bit % 8)) & 15
    return (code - 8) * s[:, t // group]


def plain_quantized(W, group):
    """Codes less 8 and scales in 64 bits."""
    x, (N, d) = W.double().cpu(), W.shape
    code, scale = torch.zeros(N, d, dtype=torch.float64), torch.zeros(N, -(-d // group), dtype=torch.float64)
    for i in range(scale.shape[1]):
        g = x[:, i * group:(i + 1) * group]
        scale[:, i] = (g.abs().amax(1) / 7).to(W.dtype).double()
        s = scale[:, i:i + 1]
        code[:, i * group:(i + 1) * group] = torch.where(s > 0, torch.round(g / s).clamp(-8, 7), 0.0)
    return code, scale


def matrix(N, d, dt, group, seed=0, device="cuda"):
    g = torch.Generator().manual_seed(1000 * seed + N + d)
    q = torch.randint(0, 256, (N, (d + 127) // 128 * 64), dtype=torch.uint8, generator=g)
    s = (torch.rand(N, -(-d // group), generator=g) * 0.01 + 0.001).to(TORCH[dt])
    return dv.Q4(q.to(device), s.to(device), d, group)


def vectors(B, d, dt, seed=0):
    g = torch.Generator().manual_seed(77 + seed)
    return torch.randn(B, d, generator=g).to(TORCH[dt]).cuda()


# --------------------------------------------------------------------- quantisation

@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N,d,group", [(1, 8, 64), (3, 64, 64), (5, 72, 64), (4, 128, 128), (7, 136, 128), (33, 1000, 64),
                                       (130, 2048, 128), (9, 5120, 128)])
def test_codes_scales_and_values_are_the_formulas(dt, N, d, group):
    W = (torch.randn(N, d, generator=torch.Generator().manual_seed(d)) * 0.02).to(TORCH[dt])
    W[0, :8] = 0
    if N > 2:
        W[1] = 0                                   # a row of nothing: scales 0, codes 8
        # quotients on the border between two codes, and just beside it
        W[2, :8] = torch.tensor([7.0, 0.5, 1.5, -2.5, 6.5, -6.5, -7.0, 3.5]).to(W.dtype)
        if d >= 16:
            W[2, 8:16] = torch.nextafter(W[2, :8].float(), torch.zeros(8)).to(W.dtype)
    Q = dv.Q4.empty(N, d, W.dtype, group)
    values = torch.full((N, d), 9.0, dtype=W.dtype, device="cuda")
    dv.dv_q4_quantize(W.cuda(), Q, values=values)
    code, scale = plain_quantized(W, group)
    assert torch.equal(Q.scale.double().cpu(), scale)
    assert np.array_equal(opened(Q.q, torch.ones_like(Q.scale), d, group), code.numpy())
    want = (code * scale.repeat_interleave(group, 1)[:, :d]).to(W.dtype)
    assert torch.equal(values.cpu() + 0.0, want + 0.0)
    # blocks end in codes 8
    full = dv.Q4(Q.q, torch.ones(N, -(-(Q.q.shape[1] * 2) // group), dtype=W.dtype, device="cuda"), Q.q.shape[1] * 2, group)
    assert not opened(full.q, full.scale, full.d, group)[:, d:].any()
    again = dv.Q4.of(W.cuda(), group)
    assert torch.equal(again.q, Q.q) and torch.equal(again.scale, Q.scale)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_tiny_huge_and_unclean_groups(dt):
    big = float(torch.finfo(TORCH[dt]).max)
    tiny = float(torch.finfo(TORCH[dt]).smallest_normal) * 2.0 ** -8 if dt != "f32" else 1e-37
    W = torch.zeros(6, 256)
    W[0, :] = torch.linspace(-1, 1, 256) * big
    W[1, :] = torch.linspace(-1, 1, 256) * tiny
    W[2, 5], W[2, 130:] = float("nan"), 1.0
    W[3, 200], W[3, :128] = float("-inf"), 0.5
    W[4, 7] = -1.0
    W[5, :] = torch.randn(256, generator=torch.Generator().manual_seed(3))
    W = W.to(TORCH[dt])
    Q = dv.Q4.empty(6, 256, W.dtype, 128)
    values = torch.zeros_like(W, device="cuda")
    dv.dv_q4_quantize(W.cuda(), Q, values=values)
    clean = W.clone()
    clean[2, :128] = 0
    clean[3, 128:] = 0
    code, scale = plain_quantized(clean, 128)
    scale[2, 0] = scale[3, 1] = float("nan")
    assert torch.equal(torch.isnan(Q.scale.cpu()), torch.isnan(scale))
    assert torch.equal(torch.nan_to_num(Q.scale.double().cpu(), posinf=9e99), torch.nan_to_num(scale, posinf=9e99))
    assert np.array_equal(opened(Q.q, torch.ones_like(Q.scale), 256, 128), code.numpy())
    v = values.cpu()
    assert torch.isnan(v[2, :128]).all() and torch.isnan(v[3, 128:]).all()
    assert torch.isfinite(v[2, 128:]).all() and torch.isfinite(v[3, :128]).all()


# --------------------------------------------------------------------- products with every row

def matvec_bound(d, W, y):
    blocks = (d + 127) // 128
    return (160 + 4 * blocks) * EPS * (np.abs(y) @ np.abs(W).T) + 1e-38


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,N,d,group", [
    (1, 1, 8, 64), (1, 15, 64, 64), (1, 16, 128, 128), (1, 17, 136, 128), (2, 33, 1000, 64), (3, 128, 2048, 128),
    (5, 130, 1024, 64), (8, 257, 776, 128), (9, 64, 512, 64), (11, 31, 264, 128), (16, 200, 640, 64),
    (17, 48, 384, 128), (32, 513, 1280, 64), (31, 16, 5120, 128), (1, 5000, 5120, 128), (1, 40, 16384, 64),
])
def test_matvec(dt, B, N, d, group):
    W, y = matrix(N, d, dt, group), vectors(B, d, dt)
    W64, y64 = opened(W.q, W.scale, d, group), y.double().cpu().numpy()
    ws = dv.workspace(dv.dv_q4_matvec_workspace_size(B, d, N))
    out = torch.full((B, N), float("nan"), device="cuda")
    dv.dv_q4_matvec(y, W, out, ws)
    got, bound = out.double().cpu().numpy(), matvec_bound(d, W64, y64)
    assert np.all(np.abs(got - y64 @ W64.T) <= bound)
    # added to what is there, and again the same
    base = torch.randn(B, N, generator=torch.Generator().manual_seed(5)).cuda()
    more = base.clone()
    dv.dv_q4_matvec(y, W, more, ws, accumulate=True)
    assert torch.equal(more, base + out)
    # every row is its own: one vector at a time gives the same to rounding
    if B > 1:
        one = torch.zeros(1, N, device="cuda")
        dv.dv_q4_matvec(y[B - 1:].contiguous(), W, one, ws)
        assert np.all(np.abs(one[0].double().cpu().numpy() - got[B - 1]) <= 2 * bound[B - 1])


@pytest.mark.gpu
def test_matvec_of_unclean_vectors_and_rows_stays_in_its_rows():
    for dt in ("f16", "bf16", "f32"):
        B, N, d = 4, 40, 256
        W, y = matrix(N, d, dt, 128), vectors(B, d, dt)
        W.scale[7, 1] = float("nan")
        y[2, 9] = float("inf")
        y[3, 200] = float("nan")
        out = torch.zeros(B, N, device="cuda")
        dv.dv_q4_matvec(y, W, out, dv.workspace(dv.dv_q4_matvec_workspace_size(B, d, N)))
        bad = ~torch.isfinite(out.cpu())
        want = torch.zeros(B, N, dtype=torch.bool)
        want[:, 7] = True
        want[2:] = True
        assert torch.equal(bad, want), dt


@pytest.mark.gpu
def test_matvec_largest_32_bit_values():
    """Pieces of the largest values stay finite."""
    d = 128
    W = dv.Q4(torch.full((16, 64), 0x99, dtype=torch.uint8, device="cuda"),
              torch.full((16, 1), 2.0 ** -8, device="cuda"), d, 128)      # every weight 2^-8
    y = torch.zeros(1, d, device="cuda")
    y[0, 3] = torch.finfo(torch.float32).max
    out = torch.zeros(1, 16, device="cuda")
    dv.dv_q4_matvec(y, W, out, dv.workspace(dv.dv_q4_matvec_workspace_size(1, d, 16)))
    assert torch.equal(out.cpu(), torch.full((1, 16), torch.finfo(torch.float32).max / 256))


# --------------------------------------------------------------------- sparse MLP

def lists(B, N, k, seed=0, counts=None):
    g = torch.Generator().manual_seed(seed + 11)
    idx = torch.stack([torch.randperm(N, generator=g)[:k].sort().values for _ in range(B)]).int()
    cnt = torch.tensor(counts if counts is not None else [k] * B, dtype=torch.int32)
    return idx, cnt


def mlp_reference(y, W1, W2, idx, cnt):
    """out, and how far the kernels may be off it."""
    y64 = y.double().cpu().numpy()
    A, C = opened(W1.q, W1.scale, W1.d, W1.group), opened(W2.q, W2.scale, W2.d, W2.group)
    B, d = y64.shape
    out, tol = np.zeros((B, d)), np.zeros((B, d))
    for b in range(B):
        S = sorted({int(j) for j in idx[b][:min(int(cnt[b]), idx.shape[1])] if 0 <= j < W1.N})
        if not S:
            continue
        a = np.maximum(A[S] @ y64[b], 0)
        off = matvec_bound(d, A[S], y64[b])
        out[b] = a @ C[S]
        union = min(W1.N, idx.numel())
        chain = 3 * 17 * (union // 16 + 1) + 32
        tol[b] = off @ np.abs(C[S]) + chain * EPS * ((a + off) @ np.abs(C[S])) + 1e-38
    return out, tol


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,N,d,k,g1,g2", [
    (1, 16, 8, 1, 64, 64), (1, 100, 64, 17, 64, 128), (1, 300, 136, 300, 128, 64), (1, 512, 1000, 40, 64, 64),
    (1, 2048, 2048, 410, 128, 128), (2, 300, 264, 33, 128, 64), (3, 256, 128, 7, 64, 64), (4, 512, 640, 64, 128, 128),
    (8, 400, 776, 50, 64, 128), (9, 200, 256, 20, 128, 64), (16, 1000, 512, 90, 64, 64), (32, 700, 392, 40, 128, 128),
    (17, 260, 1280, 260, 64, 64), (1, 9000, 256, 9000, 128, 128), (12, 4000, 128, 900, 128, 64),
])
def test_sparse_mlp(dt, B, N, d, k, g1, g2):
    W1, W2, y = matrix(N, d, dt, g1, 1), matrix(N, d, dt, g2, 2), vectors(B, d, dt)
    idx, cnt = lists(B, N, k, counts=[max(0, k - 3 * b) for b in range(B)])
    ws = dv.workspace(dv.dv_q4_sparse_mlp_workspace_size(B, d, N, k))
    out = torch.full((B, d), float("nan"), device="cuda")
    dv.dv_q4_sparse_mlp(y, W1, W2, idx.cuda(), cnt.cuda(), out, ws)
    assert dv.dv_check(ws) == (0, 0)
    ref, tol = mlp_reference(y, W1, W2, idx, cnt)
    assert np.all(np.abs(out.double().cpu().numpy() - ref) <= tol)
    base = torch.randn(B, d, generator=torch.Generator().manual_seed(5)).cuda()
    more = base.clone()
    dv.dv_q4_sparse_mlp(y, W1, W2, idx.cuda(), cnt.cuda(), more, ws, accumulate=True)
    assert torch.equal(more, base + out)
    assert dv.dv_check(ws) == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("B", [1, 3])
def test_sparse_mlp_lists_with_nothing_strangers_and_repeats(B):
    N, d, k = 200, 256, 24
    W1, W2, y = matrix(N, d, "f16", 128, 1), matrix(N, d, "f16", 64, 2), vectors(B, d, "f16")
    ws = dv.workspace(dv.dv_q4_sparse_mlp_workspace_size(B, d, N, k))
    idx, cnt = lists(B, N, k)

    def run(idx, cnt, accumulate=False, start=float("nan")):
        out = torch.full((B, d), start, device="cuda")
        dv.dv_q4_sparse_mlp(y, W1, W2, idx.cuda(), cnt.cuda(), out, ws, accumulate=accumulate)
        return out

    none = torch.zeros(B, dtype=torch.int32)
    assert not run(idx, none).any() and bool((run(idx, none, True, 3.0) == 3.0).all())
    assert not run(idx, none - 5).any()
    assert dv.dv_check(ws) == (0, 0)
    # an entry outside is skipped and reported
    strange = idx.clone()
    strange[B - 1, 5] = N
    ref, tol = mlp_reference(y, W1, W2, strange, cnt)
    assert np.all(np.abs(run(strange, cnt).double().cpu().numpy() - ref) <= tol)
    assert dv.dv_check(ws) == (5, N)
    # twice in a list: once
    twice = idx.clone()
    twice[0, 7] = twice[0, 6]
    ref, tol = mlp_reference(y, W1, W2, twice, cnt)
    assert np.all(np.abs(run(twice, cnt).double().cpu().numpy() - ref) <= tol)
    assert dv.dv_check(ws) == (0, 0)
    # a count above cap is cut off and reported
    long = cnt.clone()
    long[B - 1] = k + 9
    assert torch.equal(run(idx, long), run(idx, cnt))
    assert dv.dv_check(ws) == (8, k + 9)


@pytest.mark.gpu
def test_sparse_mlp_rows_keep_to_their_own_lists():
    """A row of W2 that holds a NaN reaches the sequences that list it, and an
    idle neuron's reaches none."""
    B, N, d, k = 2, 64, 128, 8
    W1, W2, y = matrix(N, d, "bf16", 128, 1), matrix(N, d, "bf16", 128, 2), vectors(B, d, "bf16")
    A = opened(W1.q, W1.scale, d, 128) @ y.double().cpu().numpy().T      # [N][B]
    live = int(np.argmax(A[:, 0]))
    idle = int(np.argmin(A[:, 1]))
    assert A[live, 0] > 0 > A[idle, 1] and live != idle
    W2.scale[live] = float("nan")
    W2.scale[idle] = float("nan")
    rest = [j for j in range(N) if j not in (live, idle)]
    idx = torch.tensor([sorted(rest[:k - 1] + [live]), sorted(rest[k:2 * k - 1] + [idle])], dtype=torch.int32)
    cnt = torch.full((B,), k, dtype=torch.int32)
    ws = dv.workspace(dv.dv_q4_sparse_mlp_workspace_size(B, d, N, k))
    out = torch.zeros(B, d, device="cuda")
    dv.dv_q4_sparse_mlp(y, W1, W2, idx.cuda(), cnt.cuda(), out, ws)
    assert torch.isnan(out[0]).all() and torch.isfinite(out[1]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_codes_beside_every_border(dt):
    """Values at and next to (k + 1/2) s for scales of all kinds: the nearer code,
    the even one in the middle."""
    t, n = TORCH[dt], 64
    scales = torch.tensor([1.0, 0.75, 3.3, 1e-3, 7e-4, 0.0199, 5e-6, 123.0, 1 / 3, 0.0625] +
                          ([1e-30, 3e-32, 1e-38, 2e-41] if dt != "f16" else [6e-8, 3e-6]))
    W = torch.zeros(len(scales), n, dtype=t)
    for i, s in enumerate(scales):
        top = (7 * s).to(t)
        s = float((top.double() / 7).to(t))
        v = torch.tensor([(k + 0.5) * s for k in range(-7, 7)], dtype=torch.float64).to(t)
        up, down = torch.full_like(v, float("inf")), torch.full_like(v, float("-inf"))
        near = torch.cat([v, torch.nextafter(v, up), torch.nextafter(v, down)])
        W[i, 0], W[i, 1:1 + len(near)] = top, near
        W[i] = torch.where(W[i].abs() > top, top, W[i])
    Q = dv.Q4.of(W.cuda(), 64)
    code, scale = plain_quantized(W, 64)
    assert torch.equal(Q.scale.double().cpu(), scale)
    assert np.array_equal(opened(Q.q, torch.ones_like(Q.scale), n, 64), code.numpy())
