"""4-bit products whose sums are whole numbers that every kernel holds exactly, so
that results are equal to the last bit and one row, element, share or part too few or
too many changes them.

Matrices hold scales of 1, 2 and 1/2; vectors hold whole numbers of at most 3.
Sums stay below 2^20 in steps of 1/4 (asserted on the reference), fixed point
is exact (numbers of two bits below the largest), and every piece but the first of a
32-bit factor is 0.  In the MLP a vector has one element that is not 0, and the
listed rows' weights there are positive: every listed row has a positive activation, and
without it some output is another."""

import pytest
import torch

from contextual_sparsity_decode_gb300 import binding as dv

from dvtest import TORCH
from test_q4_edges import gpu_opened

pytestmark = pytest.mark.gpu


def whole_matrix(N, d, dt, group, seed, powers=(1.0, 2.0, 0.5)):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + N + d)
    q = torch.randint(0, 256, (N, (d + 127) // 128 * 64), dtype=torch.uint8, device="cuda", generator=g)
    at = torch.randint(0, len(powers), (N, -(-d // group)), device="cuda", generator=g)
    return dv.Q4(q, torch.tensor(powers, device="cuda")[at].to(TORCH[dt]), d, group)


def set_codes(W, rows, t, codes):
    """Element t of some rows."""
    e, block = t % 8, t // 128
    bit = 4 * (e // 2) + 16 * (e % 2)
    byte = block * 64 + 4 * (2 * (t % 64 // 8) + t % 128 // 64) + bit // 8
    old = W.q[rows, byte]
    W.q[rows, byte] = (old & (0x0F if bit % 8 else 0xF0)) | (codes << (bit % 8)).to(torch.uint8)


def exact_total(x):
    assert float(x.abs().max()) < 2.0 ** 20 and bool((x * 4 == (x * 4).round()).all())
    return x.float()


MATVEC = [(1, 1, 8, 64), (1, 4097, 1000, 64), (1, 1217, 5120, 128), (2, 2433, 776, 64), (2, 40, 16392, 128), (3, 100, 200, 64),
          (3, 9001, 328, 128), (8, 19457, 1032, 64), (8, 5000, 2048, 128), (9, 16, 5120, 64), (16, 8200, 640, 128),
          (17, 3649, 4104, 64), (32, 24321, 136, 128), (32, 300, 392, 64), (30, 8000, 1544, 128)]


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("B,N,d,group", MATVEC)
def test_products_with_every_row(dt, B, N, d, group):
    W = whole_matrix(N, d, dt, group, 1)
    y = torch.randint(-3, 4, (B, d), generator=torch.Generator().manual_seed(B + d)).to(TORCH[dt]).cuda()
    want = torch.cat([y.double() @ gpu_opened(W, torch.arange(n, min(N, n + 4096), device="cuda")).T for n in range(0, N, 4096)], dim=1)
    want = exact_total(want)
    ws = dv.workspace(dv.dv_q4_matvec_workspace_size(B, d, N))
    out = torch.full((B, N), float("nan"), device="cuda")
    dv.dv_q4_matvec(y, W, out, ws)
    assert torch.equal(out, want)
    dv.dv_q4_matvec(y, W, out, ws, accumulate=True)
    assert torch.equal(out, 2 * want) and dv.dv_check(ws) == (0, 0)


# lengths of a list beside multiples of a step of four rows, of 64 and 128 rows, of the shares of 152
# CTAs (of four and of 64 rows each), and of what is staged at a time
LENGTHS = [1, 2, 3, 4, 5, 63, 65, 66, 67, 129, 607, 609, 611, 1217, 2431, 2434, 4867, 9727, 9729, 9731]
ROWS = [(136, 64, 128), (520, 128, 64)]


def check_mlp(dt, B, N, d, g1, g2, n, seed=0, cap=None):
    """A list of n rows (B = 1), or B lists whose union has n."""
    W1, W2 = whole_matrix(N, d, dt, g1, 2 + seed, powers=(1.0,)), whole_matrix(N, d, dt, g2, 3 + seed)
    g = torch.Generator().manual_seed(n + 31 * B + seed)
    rows = torch.randperm(N, generator=g)[:n].sort().values
    member = torch.rand(B, n, generator=g) < (1.0 if B == 1 else 0.4)
    member[torch.randint(0, B, (n,), generator=g), torch.arange(n)] = True    # every row in one list at least
    cnt = member.sum(dim=1).int()
    cap = max(int(cnt.max()), 1) if cap is None else cap
    idx = torch.full((B, cap), N - 1, dtype=torch.int32)                      # (behind a list: not read as entries)
    y = torch.zeros(B, d)
    at = torch.randperm(d, generator=g)[:B]
    for b in range(B):
        idx[b, :cnt[b]] = rows[member[b]].int()
        y[b, at[b]] = float(1 + b % 3)
        set_codes(W1, rows.cuda(), int(at[b]), torch.randint(9, 12, (n,), generator=g).cuda())
    y = y.to(TORCH[dt]).cuda()
    want = torch.zeros(B, d, dtype=torch.float64, device="cuda")
    step = max(1, 30_000_000 // d)
    for i in range(0, n, step):
        r = rows[i:i + step].cuda()
        a = y.double() @ gpu_opened(W1, r).T
        assert float(a.min()) >= 1
        want += (a * member[:, i:i + step].cuda()) @ gpu_opened(W2, r)
    want = exact_total(want)
    ws = dv.workspace(dv.dv_q4_sparse_mlp_workspace_size(B, d, N, cap))
    out = torch.full((B, d), float("nan"), device="cuda")
    dv.dv_q4_sparse_mlp(y, W1, W2, idx.cuda(), cnt.cuda(), out, ws)
    assert torch.equal(out, want), (n, int((out != want).sum()))
    dv.dv_q4_sparse_mlp(y, W1, W2, idx.cuda(), cnt.cuda(), out, ws, accumulate=True)
    assert torch.equal(out, 2 * want) and dv.dv_check(ws) == (0, 0)


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("d,g1,g2", ROWS)
@pytest.mark.parametrize("B", [1, 2, 3, 8, 11, 20, 32])
def test_lists_of_all_lengths(dt, B, d, g1, g2):
    for n in LENGTHS:
        check_mlp(dt, B, 10007, d, g1, g2, n)


@pytest.mark.parametrize("dt,B,N,d,group,n", [
    ("bf16", 1, 65536, 64, 64, 65533), ("f16", 1, 65536, 64, 128, 65536), ("bf16", 2, 65536, 64, 64, 65536), ("f32", 1, 40001, 72, 64, 40001),
    ("bf16", 1, 12000, 16384, 64, 11999), ("f16", 1, 6100, 8200, 128, 6083), ("f32", 2, 3000, 16384, 64, 2999),
    ("bf16", 32, 65536, 64, 128, 65535), ("f16", 25, 9000, 64, 64, 8999), ("f32", 12, 30000, 264, 128, 29999),
    ("bf16", 3, 20000, 2056, 64, 19999), ("f16", 16, 16050, 1032, 64, 16049), ("bf16", 4, 3000, 32768, 128, 2999)])
def test_long_lists(dt, B, N, d, group, n):
    check_mlp(dt, B, N, d, group, group, n)


@pytest.mark.parametrize("B", [1, 2, 5, 32])
def test_short_lists_under_a_large_bound(B):
    """Grids sized for the bound: most CTAs have nothing."""
    for n in (1, 65, 700):
        check_mlp("bf16", B, 20000, 264, 64, 128, n, cap=20000)
