"""Tree attention, compaction, beam selection and beam reordering on the GPU
against plain implementations in 64 bits.

Tolerance of the attention, element by element:
    step/2 |o| + 2 e A,      A = sum_j p_j |V_j| / sum_j p_j,
where step/2 = 2^-11 (f16), 2^-8 (bf16), 2^-24 (f32) is the output's rounding
and e bounds the relative error of a weight p_j:
    e = |scale| (d_h + 8) 2^-23 max_j sum_i |q_i K_ji|   fp32 sum of d_h products
      + n 2^-24 + 2^-20                                  sums of n weights and the exponentials
      + 2^-16                                            weights as two 16-bit halves (bf16; f16: less)
An error of e in the weights moves numerator and denominator by at most e A
each, hence 2 e A.  Elements below the storage type's smallest normal number
are off by at most half its smallest step (2^-25 for f16).
"""

import numpy as np
import pytest
import torch

from contextual_sparsity_decode_gb300 import binding as dv
from test_guards import Guarded

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ tree attention

def random_tree(T, g):
    m = torch.zeros(T, T, dtype=torch.bool)
    for t in range(T):
        p = int(torch.randint(-1, t, (1,), generator=g)) if t else -1
        if p >= 0:
            m[t] = m[p]
        m[t, t] = True
    return m


class Case:
    def __init__(self, dt, d_h, ns, T, h, g=1, nodes=None, mask="tree", heads=None, n_max=None, seed=1, std=1.0,
                 fill=0.0):
        gen, cpu = _gen(seed), torch.Generator().manual_seed(seed)
        B = len(ns)
        self.dt, self.T, self.h, self.g, self.ns, self.scale = dt, T, h, g, ns, d_h ** -0.5
        n_max = n_max or max(16, (max(ns) + T + 15) // 16 * 16)
        self.q = torch.randn(B, T, h * g, d_h, generator=gen, device="cuda").mul_(std).to(DT[dt])
        K, V = (torch.full((B, h, n_max, d_h), fill, dtype=DT[dt], device="cuda") for _ in range(2))
        self.nodes_list = nodes or [T] * B
        for b in range(B):
            n = ns[b] + self.nodes_list[b]
            for t in (K, V):
                t[b, :, :n] = torch.randn(h, n, d_h, generator=gen, device="cuda").to(DT[dt])
        self.kv = dv.KV(K, V, None, None)
        self.pos = _i32(ns)
        self.nodes = _i32(nodes) if nodes else None
        self.mask = None
        if isinstance(mask, torch.Tensor):
            self.mask = mask.cuda()
        elif mask == "tree":
            self.mask = torch.stack([random_tree(T, cpu) for _ in range(B)]).cuda()
        elif mask == "shared":
            self.mask = random_tree(T, cpu).to(torch.uint8).cuda() * 7
        self.heads = heads
        self.head_idx = self.head_count = None
        if heads is not None:
            cap = max(1, max(len(x) for x in heads))
            idx = torch.full((B, cap), -5, dtype=torch.int32)
            for b, x in enumerate(heads):
                idx[b, :len(x)] = torch.tensor(x, dtype=torch.int32)
            self.head_idx, self.head_count = idx.cuda(), _i32([len(x) for x in heads])
        self.out = torch.full_like(self.q, float("nan"))
        self.ws = dv.workspace(dv.dv_tree_attn_workspace_size(B, T, h, g, d_h))

    def call(self, stream=None):
        dv.dv_tree_attn(self.q, self.kv, self.pos, self.scale, self.out, self.ws, mask=self.mask, nodes=self.nodes,
                        head_idx=self.head_idx, head_count=self.head_count, stream=stream)

    def visible(self, b):
        T, nd = self.T, self.nodes_list[b]
        m = torch.tril(torch.ones(T, T)) if self.mask is None else self.mask[b] if self.mask.dim() == 3 else self.mask
        m = (m.cpu() != 0).cuda()[:nd, :nd]
        return torch.cat([torch.ones(nd, self.ns[b], dtype=torch.bool, device="cuda"), m], 1)

    def reference(self):
        """(out, tolerance) in float64."""
        ref = torch.zeros(self.q.shape, dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(ref)
        d_h = self.q.shape[3]
        for b in range(self.q.shape[0]):
            nd = self.nodes_list[b]
            vis = self.visible(b)
            n = vis.shape[1]
            for i in range(self.h) if self.heads is None else self.heads[b]:
                k, v = self.kv.K[b, i, :n].double(), self.kv.V[b, i, :n].double()
                for e in range(self.g):
                    x = i * self.g + e
                    q = self.q[b, :nd, x].double()
                    s = torch.where(vis, q @ k.T * self.scale, torch.tensor(-np.inf, device="cuda", dtype=torch.float64))
                    top = s.amax(1, keepdim=True)
                    p = torch.exp(s - torch.where(torch.isinf(top), torch.zeros_like(top), top))
                    l = p.sum(1, keepdim=True)
                    p = p / torch.where(l > 0, l, torch.ones_like(l))
                    vz = torch.where(vis.any(0)[:, None], v, torch.zeros_like(v))   # rows that nobody sees
                    ref[b, :nd, x] = p @ vz
                    size = torch.where(vis, q.abs() @ k.abs().T, torch.zeros_like(s)).amax(1, keepdim=True)
                    err = (abs(self.scale) * (d_h + 8) * 2.0 ** -23 * size + n * 2.0 ** -24 + 2.0 ** -20
                           + (0 if self.dt == "f32" else 2.0 ** -16))
                    tol[b, :nd, x] = 2 * err * (p @ vz.abs())
        return ref, tol + HALF[self.dt] * ref.abs() + (2.0 ** -25 if self.dt == "f16" else 0)

    def check(self):
        self.call()
        assert dv.dv_check(self.ws) == (0, 0)
        ref, tol = self.reference()
        got = self.out.double()
        assert torch.isfinite(got).all()
        over = (got - ref).abs() - tol
        assert over.max() <= 0, f"worst {over.max():.3g} at {np.unravel_index(int(over.argmax()), over.shape)}"
        first = self.out.clone()
        self.out.fill_(float("nan"))
        self.call()                                   # the workspace is reusable, results repeat bit for bit
        assert dv.dv_check(self.ws) == (0, 0)
        assert torch.equal(first, self.out)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d_h", [64, 128])
@pytest.mark.parametrize("ns,T,h,g,mask", [
    ([0], 1, 1, 1, None),                       # one key
    ([1], 1, 3, 1, None),
    ([63, 64, 65], 1, 2, 1, "tree"),            # the edge of a tile, single tokens
    ([0, 5, 127, 128], 7, 3, 1, "tree"),
    ([100], 64, 2, 1, "shared"),
    ([31, 200], 65, 2, 1, None),                # the tree itself crosses a tile
    ([3000], 5, 2, 1, "tree"),                  # one unit over many CTAs
    ([500, 20], 30, 2, 5, "tree"),              # 150 rows: two row blocks
    ([129, 7], 3, 2, 3, "shared"),
    ([700], 33, 1, 4, None),                    # 132 rows
])
def test_tree_attention(dt, d_h, ns, T, h, g, mask):
    Case(dt, d_h, ns, T, h, g=g, mask=mask, seed=len(ns) * 100 + T).check()


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_tree_attention_many_units(dt):
    """More units than CTAs: shares start and end inside units."""
    Case(dt, 64, [(37 * b) % 300 for b in range(23)], 9, 11, mask="tree", seed=5).check()


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d_h", [64, 128])
def test_tree_attention_lists_and_partial_trees(dt, d_h):
    """Heads outside the list, an empty list, trees that are not full, an
    empty tree: all rows of out are written, the others with zeros."""
    c = Case(dt, d_h, [70, 0, 129, 12], 6, 5, nodes=[6, 3, 0, 1], heads=[[0, 3], [1, 2, 4], [0, 1], []], seed=9)
    c.check()
    assert (c.out[2] == 0).all() and (c.out[3] == 0).all() and (c.out[0, :, 1] == 0).all()


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_rows_that_see_nothing_are_zero(dt):
    """No committed position and an empty mask row (row 1), or a mask of
    zeros altogether."""
    m = torch.zeros(4, 4, dtype=torch.bool)
    m[0, 0] = m[2, 1] = m[3, 0] = m[3, 3] = True
    c = Case(dt, 64, [0], 4, 2, mask=m)
    c.check()
    assert (c.out[0, 1] == 0).all()
    # a single visible key has weight one
    assert torch.equal(c.out[0, 2], c.kv.V[0, :, 1])
    z = Case(dt, 128, [0, 40], 3, 2, mask=torch.zeros(3, 3, dtype=torch.uint8))
    z.check()
    assert (z.out[0] == 0).all()


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d_h", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_a_row_does_not_see_does_not_reach_it(dt, d_h, bad):
    """Positions behind the tree and nodes that a row does not see may hold
    anything; a row that sees such a node gets what the formula gives."""
    T = 6
    m = torch.eye(T, dtype=torch.bool)
    m[:, 0] = True
    m[4, 2] = True                     # row 4 sees node 2, the others (but 2) do not
    for n in (0, 61, 130):
        c = Case(dt, d_h, [n], T, 2, mask=m, fill=bad, n_max=256, seed=3)
        c.check()
        clean = c.out.clone()
        c.kv.K[0, :, n + 2] = bad
        c.kv.V[0, :, n + 2] = bad
        c.call()
        assert dv.dv_check(c.ws) == (0, 0)
        for t in (0, 1, 3, 5):
            assert torch.equal(c.out[0, t], clean[0, t]), (n, t)
        assert not torch.isfinite(c.out[0, 2]).any()
        c.kv.K[0, :, n + 2] = 0.0      # finite scores, a V that is not finite
        c.call()
        for t in (0, 1, 3, 5):
            assert torch.equal(c.out[0, t], clean[0, t]), (n, t)
        for t in (2, 4):
            assert (torch.isnan(c.out[0, t]) if np.isnan(bad) else c.out[0, t] == bad).all(), (n, t)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_large_and_descending_scores(dt):
    """Scores whose maximum grows tile by tile, and scores far apart: the
    running maximum has to carry the sums along."""
    c = Case(dt, 64, [640], 5, 2, mask="tree", seed=21)
    ramp = torch.linspace(0.05, 6.0, 645, device="cuda").to(DT[dt])
    c.kv.K[:, :, :645] = c.q[:, :1].transpose(1, 2) * ramp[None, None, :, None]   # row 0's scores ascend
    c.check()
    c.kv.K[:, :, :645] = c.kv.K[:, :, :645].flip(2)
    c.check()


def test_tree_attention_offsets_beyond_32_bits():
    """A cache of more than 2^32 bytes and 2^31 elements, used at its end."""
    B, h, n_max, d_h = 17, 1, 2 ** 20, 128          # 17 * 2^20 * 128 elements > 2^31
    K = torch.zeros(B, h, n_max, d_h, dtype=torch.float16, device="cuda")
    V = torch.zeros_like(K)
    c = Case("f16", d_h, [40] * B, 3, h, mask=None, seed=2)
    n = c.kv.K.shape[2]
    ref = Case("f16", d_h, [40] * B, 3, h, mask=None, seed=2)
    ref.call()
    K[:, :, :n], V[:, :, :n] = c.kv.K, c.kv.V
    c.kv = dv.KV(K, V, None, None)
    c.call()
    assert dv.dv_check(c.ws) == (0, 0)
    assert torch.equal(c.out, ref.out)
    # the last positions of the last row
    g = _gen(4)
    K[-1, 0, -2000:] = torch.randn(2000, d_h, generator=g, device="cuda").half()
    V[-1, 0, -2000:] = torch.randn(2000, d_h, generator=g, device="cuda").half()
    ns = [0] * (B - 1) + [n_max - 3]
    c.ns, c.pos = ns, _i32(ns)
    c.check()


def test_device_errors_are_reported_and_contained():
    def fresh(**kw):
        return Case("f16", 64, [20, 30], 4, 3, seed=7, **kw)

    c = fresh()
    good = c.out.clone()
    c.call()
    good.copy_(c.out)
    for pos, st in ((-1, 9), (c.kv.n_max - 3, 9), (2 ** 31 - 2, 9)):
        c.pos = _i32([20, pos])
        c.out.fill_(1.0)
        c.call()
        assert dv.dv_check(c.ws)[0] == st
        assert torch.equal(c.out[0], good[0]) and (c.out[1] == 0).all()
    c = fresh(heads=[[0, 1], [0, 2]])
    c.head_idx[1, 1] = 3
    c.out.fill_(1.0)
    c.call()
    assert dv.dv_check(c.ws) == (5, 3)
    assert torch.equal(c.out[0, :, :2], good[0, :, :2]) and torch.equal(c.out[1, :, 0], good[1, :, 0])
    assert (c.out[1, :, 1:] == 0).all()
    c = fresh(heads=[[0, 1], [0, 2]])
    c.head_count[0] = 5
    c.call()
    assert dv.dv_check(c.ws) == (8, 5)
    assert torch.equal(c.out[0, :, :2], good[0, :, :2])
    c = fresh(nodes=[4, 4])
    c.nodes[0] = 9
    c.call()
    assert dv.dv_check(c.ws) == (8, 9)
    assert torch.equal(c.out, good)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_captured_replayed_and_on_another_stream(dt):
    c = Case(dt, 128, [300, 90], 12, 3, nodes=[12, 7], seed=11)
    c.check()
    want = c.out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    c.call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(c.out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call()
    # lengths, mask and queries are read at replay
    for seed in (12, 13):
        d = Case(dt, 128, [40 * (seed - 11), 200], 12, 3, nodes=[5, 12], n_max=c.kv.n_max, seed=seed)
        for a, b in ((c.q, d.q), (c.kv.K, d.kv.K), (c.kv.V, d.kv.V), (c.pos, d.pos), (c.nodes, d.nodes),
                     (c.mask, d.mask)):
            a.copy_(b)
        c.out.fill_(float("nan"))
        graph.replay()
        d.check()
        assert torch.equal(c.out, d.out)


def test_two_calls_at_once_with_their_own_workspaces():
    a = Case("f16", 128, [900], 16, 8, seed=31)
    b = Case("f16", 64, [1200, 64], 9, 6, seed=32)
    a.check(), b.check()
    wa, wb = a.out.clone(), b.out.clone()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        a.call(stream=s1)
        b.call(stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(a.out, wa) and torch.equal(b.out, wb)


# ------------------------------------------------------------------ moving cache rows

def _cache(L, B, h, n_max, d_h, dt, seed, keep=0.5):
    g = _gen(seed)
    out = []
    for _ in range(L):
        K, V = (torch.randn(B, h, n_max, d_h, generator=g, device="cuda").to(DT[dt]) for _ in range(2))
        X = torch.randn(B, n_max, h * d_h + 8, generator=g, device="cuda").to(DT[dt])
        valid = (torch.rand(B, h, n_max, generator=g, device="cuda") < keep).to(torch.uint8)
        K[valid == 0], V[valid == 0] = float("nan"), float("nan")
        out.append(dv.KV(K, V, X, valid))
    return out


def _copy(kvs):
    return [[t.clone() for t in (c.K, c.V, c.X, c.valid)] for c in kvs]


def _same(kvs, want):
    for l, (c, w) in enumerate(zip(kvs, want)):
        for name, t, r in zip("KVXv", (c.K, c.V, c.X, c.valid), w):
            if name != "v":
                t, r = (x.view(torch.int32 if x.element_size() == 4 else torch.int16) for x in (t, r))
            assert torch.equal(t, r), (l, name)


def _compact_ref(want, b, pos, idx):
    for K, V, X, valid in want:
        for k, u in enumerate(idx):
            have = valid[b, :, pos + u].bool()
            for t in (K, V):
                t[b, have, pos + k] = t[b, have, pos + u].clone()
            X[b, pos + k] = X[b, pos + u].clone()
            valid[b, :, pos + k] = valid[b, :, pos + u].clone()


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("L,h,d_h", [(1, 2, 64), (3, 3, 128), (2, 1, 8), (66, 1, 16)])
def test_compact(dt, L, h, d_h):
    lists = [[0, 1, 2], [2, 3, 7, 9, 12], [5], [], list(range(1, 16))]
    pos = [3, 0, 40, 7, 11]
    B, n_max = 5, 48
    kvs = _cache(L, B, h, n_max, d_h, dt, 40 + L)
    layers, ws = dv.KVLayers(kvs), dv.workspace(256)
    idx = torch.full((B, 16), -1, dtype=torch.int32)
    for b, x in enumerate(lists):
        idx[b, :len(x)] = torch.tensor(x, dtype=torch.int32)
    idx, count, p = idx.cuda(), _i32([len(x) for x in lists]), _i32(pos)
    want = _copy(kvs)
    for b in range(B):
        _compact_ref(want, b, pos[b], lists[b])
    new = torch.zeros_like(p)
    dv.dv_kv_compact(layers, p, idx, count, ws, new_pos=new)
    assert dv.dv_check(ws) == (0, 0)
    _same(kvs, want)
    assert new.tolist() == [a + len(x) for a, x in zip(pos, lists)] and p.tolist() == pos
    # a second call, in place of the positions themselves
    count.zero_()
    dv.dv_kv_compact(layers, p, idx, count, ws, new_pos=p)
    _same(kvs, want)
    assert p.tolist() == pos


def test_compact_advances_positions_in_place_in_a_graph():
    kvs = _cache(2, 2, 2, 64, 64, "f16", 3)
    want = _copy(kvs)
    layers, ws = dv.KVLayers(kvs), dv.workspace(256)
    idx, count, pos = _i32([[1, 3, 4], [0, 2, 0]]), _i32([3, 2]), _i32([5, 6])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dv.dv_kv_compact(layers, pos, idx, count, ws, new_pos=pos)
    for r in range(4):
        graph.replay()
        _compact_ref(want, 0, 5 + 3 * r, [1, 3, 4])
        _compact_ref(want, 1, 6 + 2 * r, [0, 2])
    assert dv.dv_check(ws) == (0, 0)
    _same(kvs, want)
    assert pos.tolist() == [17, 14]


def test_compact_leaves_refused_sequences_alone():
    for bad, pos, st in (([0, 0, 2], 4, 5), ([2, 1, 3], 4, 5), ([-1, 1, 2], 4, 5), ([0, 1, 12], 4, 9), ([0, 1, 2], -1, 9),
                         ([0, 1, 2], 16, 9)):
        kvs = _cache(1, 2, 2, 16, 64, "bf16", 8)
        want = _copy(kvs)
        _compact_ref(want, 1, 2, [1, 2])
        layers, ws = dv.KVLayers(kvs), dv.workspace(256)
        p = _i32([pos, 2])
        dv.dv_kv_compact(layers, p, _i32([bad, [1, 2, 0]]), _i32([3, 2]), ws, new_pos=p)
        assert dv.dv_check(ws)[0] == st
        _same(kvs, want)
        assert p.tolist() == [pos, 4]
    kvs = _cache(1, 1, 2, 16, 64, "f32", 8)
    want = _copy(kvs)
    _compact_ref(want, 0, 2, [1, 2])
    layers, ws = dv.KVLayers(kvs), dv.workspace(256)
    dv.dv_kv_compact(layers, _i32([2]), _i32([[1, 2]]), _i32([5]), ws)
    assert dv.dv_check(ws) == (8, 5)
    _same(kvs, want)


def _reorder_ref(want, S, W, pos, start, parent):
    for l, tensors in enumerate(want):
        old = [t.clone() for t in tensors]
        for s in range(S):
            for w in range(W):
                p = parent[s][w]
                lo, hi = start[s], pos[s * W + p]
                if p == w or hi <= lo:
                    continue
                dst, src = s * W + w, s * W + p
                have = old[3][src, :, lo:hi].bool()
                for t, o in zip(tensors[:2], old[:2]):
                    t[dst, :, lo:hi][have] = o[src, :, lo:hi][have]
                tensors[2][dst, lo:hi] = old[2][src, lo:hi]
                tensors[3][dst, :, lo:hi] = old[3][src, :, lo:hi]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("L,S,W,h,d_h,n_max", [
    (1, 1, 1, 1, 64, 16), (2, 3, 2, 2, 64, 32), (1, 2, 4, 3, 128, 48), (1, 1, 7, 2, 8, 80), (1, 2, 16, 1, 128, 33),
    (1, 1, 32, 2, 64, 40), (65, 1, 3, 1, 16, 16),
])
def test_reorder(dt, L, S, W, h, d_h, n_max):
    cpu = torch.Generator().manual_seed(L * 100 + W)
    kvs = _cache(L, S * W, h, n_max, d_h, dt, W)
    want = _copy(kvs)
    layers, ws = dv.KVLayers(kvs), dv.workspace(256)
    for r in range(3):
        pos = torch.randint(0, n_max + 1, (S * W,), generator=cpu).tolist()
        start = torch.randint(0, n_max // 2, (S,), generator=cpu).tolist() if r else [0] * S
        parent = torch.randint(0, W, (S, W), generator=cpu)
        if r == 2:                                    # a cycle over all beams
            parent = ((torch.arange(W) + 1) % W).expand(S, W)
        dv.dv_kv_reorder(layers, _i32(pos), parent.int().contiguous().cuda(), ws, start=_i32(start) if r else None)
        _reorder_ref(want, S, W, pos, start, parent.tolist())
        assert dv.dv_check(ws) == (0, 0)
        _same(kvs, want)


def test_reorder_leaves_refused_beams_alone():
    kvs = _cache(2, 4, 2, 32, 64, "f16", 5)
    want = _copy(kvs)
    layers, ws = dv.KVLayers(kvs), dv.workspace(256)
    dv.dv_kv_reorder(layers, _i32([20, 20, 20, 20]), _i32([[1, 4, 0, -1]]), ws)
    assert dv.dv_check(ws)[0] == 5
    _reorder_ref(want, 1, 4, [20] * 4, [0], [[1, 1, 0, 3]])
    _same(kvs, want)
    dv.dv_kv_reorder(layers, _i32([20, 33, -1, 20]), _i32([[1, 2, 0, 0]]), ws)
    assert dv.dv_check(ws)[0] == 9
    _reorder_ref(want, 1, 4, [20, 0, 0, 20], [0], [[1, 2, 0, 0]])
    _same(kvs, want)
    # a start behind every position, and one below zero
    for start in ([40], [-3]):
        dv.dv_kv_reorder(layers, _i32([20, 20, 20, 20]), _i32([[1, 1, 0, 2]]), ws, start=_i32(start))
        _reorder_ref(want, 1, 4, [20] * 4, [max(0, start[0])], [[1, 1, 0, 2]])
        assert dv.dv_check(ws) == (0, 0)
        _same(kvs, want)


# ------------------------------------------------------------------ beam selection

def _beam_ref(logits, cum, K, done=None, end=0):
    """Scores in float64, ranked by score and then by flat index."""
    x, cum = logits.double().cpu().numpy(), cum.double().cpu().numpy()
    S, W, V = x.shape
    score, token, beam = np.zeros((S, K)), np.zeros((S, K), int), np.zeros((S, K), int)
    with np.errstate(all="ignore"):
        for s in range(S):
            tot = np.full((W, V), -np.inf)
            for w in range(W):
                c = cum[s, w]
                if done is not None and done[s, w]:
                    tot[w, end] = c if np.isfinite(c) else -np.inf
                    continue
                r = x[s, w]
                if np.isnan(r).any() or np.isposinf(r).any() or np.isneginf(r).all() or not np.isfinite(c):
                    continue
                m = r.max()
                tot[w] = c + (r - (m + np.log(np.exp(r - m).sum())))
            f = tot.reshape(-1)
            best = np.lexsort((np.arange(f.size), -f))[:K]
            score[s], token[s], beam[s] = f[best], best % V, best // V
    return score, token, beam


def _beam_check(logits, cum, K, done=None, end=0):
    """Tokens and beams exactly.  Scores: fp32 rounding (2^-24 relative) and
    the log-sum-exp's error, below 2^-21 (fp32 exponentials, two units in the
    last place each, under a sum in at least that precision)."""
    S, W, V = logits.shape
    ws = dv.workspace(dv.dv_beam_select_workspace_size(S, W, V, K))
    score = torch.full((S, K), float("nan"), device="cuda")
    token, beam = (torch.full((S, K), -1, dtype=torch.int32, device="cuda") for _ in range(2))
    rs, rt, rb = _beam_ref(logits, cum, K, None if done is None else done.cpu().numpy(), end)
    for _ in range(2):
        score.fill_(float("nan"))
        dv.dv_beam_select(logits, cum, score, token, beam, ws, done=done, end_token=end)
        assert dv.dv_check(ws) == (0, 0)
        assert np.array_equal(token.cpu().numpy(), rt) and np.array_equal(beam.cpu().numpy(), rb)
        got = score.double().cpu().numpy()
        fine = np.isfinite(rs)
        assert np.array_equal(fine, np.isfinite(got)) and (got[~fine] == -np.inf).all()
        assert (np.abs(got[fine] - rs[fine]) <= 2.0 ** -24 * np.abs(rs[fine]) + 2.0 ** -21).all()


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("S,W,V,K", [
    (1, 1, 1, 1), (1, 1, 7, 7), (2, 3, 5, 15), (1, 4, 100, 4), (3, 2, 1001, 8), (2, 5, 8191, 10), (2, 4, 8193, 64),
    (1, 32, 20000, 64), (5, 1, 50003, 1), (1, 3, 40007, 6), (40, 2, 333, 3),
])
def test_beam_select(dt, S, W, V, K):
    g = _gen(S * 1000 + V)
    logits = (3 * torch.randn(S, W, V, generator=g, device="cuda")).to(DT[dt])
    cum = -5 * torch.rand(S, W, generator=g, device="cuda")
    _beam_check(logits, cum, K)
    if V > 3:
        logits[:, :, torch.rand(V, generator=g, device="cuda") < 0.3] = -float("inf")
        logits[:, :, V // 2] = 1.0
        done = (torch.rand(S, W, generator=g, device="cuda") < 0.4).to(torch.uint8)
        _beam_check(logits, cum, K, done, V // 3)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [50, 9001])
def test_beam_ties_go_to_the_lower_index(dt, V):
    """Equal logits inside a row, equal rows (whose addresses differ in
    alignment, V being odd), everything equal."""
    g = _gen(V)
    few = torch.randint(0, 4, (2, 4, V), generator=g, device="cuda").to(DT[dt])
    cum = torch.zeros(2, 4, device="cuda")
    _beam_check(few[:, :1].expand(2, 4, V).contiguous(), cum, 20)
    row = torch.randn(1, 1, V, generator=g, device="cuda").to(DT[dt])
    _beam_check(row.expand(2, 4, V).contiguous(), cum, 12)
    _beam_check(torch.zeros(1, 3, V, device="cuda", dtype=DT[dt]), torch.zeros(1, 3, device="cuda"), 64)
    _beam_check(torch.arange(V, device="cuda").float().expand(1, 2, V).div(V).contiguous().to(DT[dt]), cum[:1, :2], 40)
    _beam_check(-torch.arange(V, device="cuda").float().expand(1, 2, V).div(V).contiguous().to(DT[dt]), cum[:1, :2], 40)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_beam_rows_without_finite_candidates(dt):
    inf = float("inf")
    V, K = 300, 12
    x = torch.randn(6, 3, V, generator=_gen(6), device="cuda").to(DT[dt])
    cum = -torch.rand(6, 3, generator=_gen(7), device="cuda")
    x[0, 0, 5], x[1, 1, 17] = float("nan"), inf
    x[2, 2] = -inf
    x[3, :, 3:] = -inf                 # fewer finite tokens than asked for
    cum[4, 0], cum[4, 1], cum[5, 2] = -inf, float("nan"), inf
    _beam_check(x, cum, K)
    x[5] = -inf                        # nothing at all
    _beam_check(x, cum, K)
    low = x.clone()                    # masked with the type's lowest value instead, a whole row of it too
    low[3, :, 3:] = torch.finfo(DT[dt]).min
    low[2, 2] = torch.finfo(DT[dt]).min
    low[1, 0, 7] = torch.finfo(DT[dt]).max / 2
    _beam_check(low, cum, K)
    for end in (0, 7, 299):            # ended beams: one candidate each, then -inf from the lowest token on
        _beam_check(x, cum, K, torch.ones(6, 3, dtype=torch.uint8, device="cuda"), end)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("K", [1, 5, 64])
def test_beam_values_that_crowd_the_threshold(dt, K):
    """Inputs that list many tokens: zeros of both signs, the best tokens of a
    row in the hands of a few threads, rows of -inf but for a few tokens,
    long runs of equal values, ascending and descending rows over several
    chunks."""
    V, inf = 20001, float("inf")
    g = _gen(K)
    cum = torch.tensor([[0.0, -0.25]], device="cuda")
    x = torch.zeros(1, 2, V, device="cuda")
    x[:, :, torch.rand(V, generator=g, device="cuda") < 0.5] = -0.0
    _beam_check(x.to(DT[dt]), cum, K)
    v = torch.arange(V, device="cuda")
    few = torch.where((v // 8) % 256 < 9, 4.0 + torch.randn(1, 2, V, generator=g, device="cuda"), -4.0)
    _beam_check(few.to(DT[dt]), cum, K)
    holes = torch.full((1, 2, V), -inf, device="cuda")
    holes[:, :, [7, 8190, 8191, 8192, 20000]] = torch.randn(1, 2, 5, generator=g, device="cuda")
    _beam_check(holes.to(DT[dt]), cum, K)
    runs = (v // 700 % 5).float().expand(1, 2, V).contiguous()
    _beam_check(runs.to(DT[dt]), cum, K)
    _beam_check((v / V).expand(1, 2, V).contiguous().to(DT[dt]), cum, K)
    _beam_check((-v / V).expand(1, 2, V).contiguous().to(DT[dt]), cum, K)


def test_beam_rows_with_a_stride_and_any_alignment():
    big = torch.randn(2 * 3 * 4099 + 8, generator=_gen(3), device="cuda").half()
    for off in range(8):
        rows = big[off:off + 6 * 4099].view(2, 3, 4099)[:, :, :4001]
        _beam_check(rows, torch.zeros(2, 3, device="cuda"), 9)


def test_beam_select_captured():
    S, W, V, K = 2, 4, 9000, 8
    logits, cum = torch.randn(S, W, V, device="cuda"), torch.zeros(S, W, device="cuda")
    score, token, beam = torch.zeros(S, K, device="cuda"), *(torch.zeros(S, K, dtype=torch.int32, device="cuda") for _ in range(2))
    ws = dv.workspace(dv.dv_beam_select_workspace_size(S, W, V, K))
    dv.dv_beam_select(logits, cum, score, token, beam, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dv.dv_beam_select(logits, cum, score, token, beam, ws)
    for seed in range(3):
        logits.normal_(generator=_gen(seed))
        graph.replay()
        _, rt, rb = _beam_ref(logits, cum, K)
        assert np.array_equal(token.cpu().numpy(), rt) and np.array_equal(beam.cpu().numpy(), rb)


def test_tree_attention_waits_that_run_out_unwind():
    """A 1 ns limit lets waits give up before their copies land (whether one
    does depends on timing).  The call ends, the workspace stays usable, and
    the next call is right."""
    c = Case("f16", 128, [2000, 700], 16, 8, seed=41)
    c.check()
    want = c.out.clone()
    prev = dv.dv_set_wait_limit_ns(1)
    try:
        for _ in range(3):
            c.call()
            st, _ = dv.dv_check(c.ws)
            assert st in (0, 6)
    finally:
        dv.dv_set_wait_limit_ns(prev)
    c.out.zero_()
    c.call()
    assert dv.dv_check(c.ws) == (0, 0)
    assert torch.equal(c.out, want)


# ------------------------------------------------------------------ guard regions

def _guarded_ws(nbytes):
    w = Guarded((max(int(nbytes), 256),), torch.uint8)
    dv.dv_workspace_init(w.t)
    return w


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d_h,T,g", [(64, 5, 1), (128, 70, 2), (64, 1, 1)])
def test_tree_attention_writes_stay_in_bounds(dt, d_h, T, g):
    c = Case(dt, d_h, [300, 0, 77], T, 3, g=g, seed=51, n_max=(300 + T + 15) // 16 * 16)
    out, ws = Guarded(tuple(c.out.shape), DT[dt]), _guarded_ws(dv.dv_tree_attn_workspace_size(3, T, 3, g, d_h))
    c.call()
    want, c.out, c.ws = c.out, out.t, ws.t
    c.call()
    assert dv.dv_check(ws.t) == (0, 0)
    assert torch.equal(out.t, want) and out.intact() and ws.intact()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_cache_moves_stay_in_bounds(dt):
    B, h, n_max, d_h = 4, 3, 32, 64
    shapes = ((B, h, n_max, d_h), (B, h, n_max, d_h), (B, n_max, h * d_h))
    parts = [Guarded(s, DT[dt], fill=1.0) for s in shapes] + [Guarded((B, h, n_max), torch.uint8, fill=1)]
    layers, ws, new = dv.KVLayers([dv.KV(*(p.t for p in parts))]), _guarded_ws(256), Guarded((B,), torch.int32)
    dv.dv_kv_compact(layers, _i32([0, 5, 30, 31]), _i32([[0, 3], [1, 26], [0, 1], [0, 0]]), _i32([2, 2, 2, 1]), ws.t,
                     new_pos=new.t)
    dv.dv_kv_reorder(layers, _i32([32, 32, 7, 0]), _i32([[1, 0, 3, 2]]), ws.t)
    assert dv.dv_check(ws.t) == (0, 0)
    assert all(p.intact() for p in parts) and ws.intact() and new.intact()
    assert new.t.tolist() == [2, 7, 32, 32]


@pytest.mark.parametrize("dt", ["f32", "f16"])
def test_beam_select_writes_stay_in_bounds(dt):
    S, W, V, K = 3, 4, 9001, 8
    logits = torch.randn(S, W, V, generator=_gen(5), device="cuda").to(DT[dt])
    ws = _guarded_ws(dv.dv_beam_select_workspace_size(S, W, V, K))
    score, token, beam = Guarded((S, K), torch.float32), Guarded((S, K), torch.int32), Guarded((S, K), torch.int32)
    cum = torch.zeros(S, W, device="cuda")
    dv.dv_beam_select(logits, cum, score.t, token.t, beam.t, ws.t)
    assert dv.dv_check(ws.t) == (0, 0)
    assert all(x.intact() for x in (ws, score, token, beam))
    _, rt, rb = _beam_ref(logits, cum, K)
    assert np.array_equal(token.t.cpu().numpy(), rt) and np.array_equal(beam.t.cpu().numpy(), rb)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("W,K,end", [(1, 4, 10), (2, 2, 299), (2, 5, 4), (3, 12, 200), (2, 5, 0)])
def test_ended_beams_of_score_minus_infinity(dt, W, K, end):
    """An ended beam at -inf offers its end token at -inf as well: it takes no
    place before lower tokens."""
    logits = torch.randn(2, W, 300, generator=_gen(W + K), device="cuda").to(DT[dt])
    cum = torch.full((2, W), float("-inf"), device="cuda")
    done = torch.ones(2, W, dtype=torch.uint8, device="cuda")
    _beam_check(logits, cum, K, done, end)
    cum[1, W - 1] = -1.5               # one sequence with a candidate
    _beam_check(logits, cum, K, done, end)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_beam_select_unwinds_when_its_waits_run_out(dt):
    """With a wait limit of a nanosecond a scan may give up on a copy: the call
    returns, reports it, writes nothing outside its outputs, and the next call
    is right."""
    S, W, V, K = 6, 8, 60001, 16
    logits = torch.randn(S, W, V, generator=_gen(61), device="cuda").to(DT[dt])
    cum = -torch.rand(S, W, generator=_gen(62), device="cuda")
    score = Guarded((S, K), torch.float32)
    token, beam = Guarded((S, K), torch.int32), Guarded((S, K), torch.int32)
    ws = _guarded_ws(dv.dv_beam_select_workspace_size(S, W, V, K))
    prev = dv.dv_set_wait_limit_ns(1)
    try:
        for _ in range(3):
            dv.dv_beam_select(logits, cum, score.t, token.t, beam.t, ws.t)
            st, _ = dv.dv_check(ws.t)
            assert st in (0, 6)
    finally:
        dv.dv_set_wait_limit_ns(prev)
    dv.dv_beam_select(logits, cum, score.t, token.t, beam.t, ws.t)
    assert dv.dv_check(ws.t) == (0, 0)
    assert score.intact() and token.intact() and beam.intact() and ws.intact()
    _, rt, rb = _beam_ref(logits, cum, K, None, 0)
    assert np.array_equal(token.t.cpu().numpy(), rt) and np.array_equal(beam.t.cpu().numpy(), rb)
