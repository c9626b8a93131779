"""The verify pass where its nodes meet the cache's end, are padding, or share
few heads and neurons; what it leaves alone, and what it keeps."""

import math

import pytest
import torch

from contextual_sparsity_decode_gb300 import binding as dv
from contextual_sparsity_decode_gb300 import stack
from synth import Workload, embeddings, layer_weights
from test_stack_candidates import N_PROMPT, TOL, _close, _decoder, _inputs, _step

pytestmark = pytest.mark.gpu


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _filled(B, pos, **kw):
    """A decoder whose caches hold something in every slot, at positions pos."""
    dec = _decoder(B, **kw)
    g = torch.Generator(device="cuda").manual_seed(17)
    for kv in dec.kv:
        for t in (kv.K, kv.V, kv.X):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda").to(t.dtype))
        kv.valid.fill_(1)
    dec.pos.copy_(_i32(pos))
    return dec


def _tensors(dec):
    return [[t.clone() for t in (kv.K, kv.V, kv.X, kv.valid)] for kv in dec.kv]


def _unchanged(dec, old, b, lo, hi):
    """Slots [lo, hi) of row b hold what they held, in every layer."""
    for l, kv in enumerate(dec.kv):
        for name, t, o in zip("KVXv", (kv.K, kv.V, kv.X, kv.valid), old[l]):
            t, o = (x[b, lo:hi] if name == "X" else x[b, :, lo:hi] for x in (t, o))
            assert torch.equal(t, o), (l, name)


@pytest.mark.parametrize("pos", [64, 62, 70, -2, 2 ** 31 - 2])
def test_a_tree_behind_the_cache_changes_no_row(pos):
    """A tree that does not fit behind its sequence (or a position that is none)
    is reported; no slot of the row changes, and the other row is served."""
    E = _inputs(2, 5, 512, 31)
    dec = _filled(2, [pos, 30])
    old = _tensors(dec)
    got = dec.verify_tree(E)
    with pytest.raises(dv.DvError) as e:
        dec.check()
    assert e.value.status == 9
    _unchanged(dec, old, 0, 0, 64)
    _unchanged(dec, old, 1, 0, 30)
    _unchanged(dec, old, 1, 35, 64)
    ref = _filled(2, [30, 30])
    want = ref.verify_tree(E)
    ref.check()
    _close(got[1], want[1])


def test_padding_nodes_write_nothing():
    """Nodes behind nodes[b] are padding: their slots keep what they hold, also
    where they would lie behind the cache."""
    E = _inputs(3, 5, 512, 32)
    pos, nodes = [60, 40, 20], [2, 1, 0]
    dec = _filled(3, pos)
    old = _tensors(dec)
    got = dec.verify_tree(E, nodes=_i32(nodes))
    dec.check()
    for b in range(3):
        _unchanged(dec, old, b, 0, pos[b])
        _unchanged(dec, old, b, pos[b] + nodes[b], 64)
    for b, n in enumerate(nodes[:2]):
        ref = _filled(3, pos)
        want = ref.verify_tree(E[:, :n])
        ref.check()
        _close(got[b, :n], want[b])
        for kv, k in zip(dec.kv, ref.kv):
            _close(kv.X[b, pos[b]:pos[b] + n], k.X[b, pos[b]:pos[b] + n])
            _close(kv.K[b, :, pos[b]:pos[b] + n], k.K[b, :, pos[b]:pos[b] + n])


def test_more_nodes_than_the_tree_has_are_cut_off():
    E = _inputs(1, 3, 512, 33)
    dec, ref = _filled(1, [20]), _filled(1, [20])
    for d in (dec, ref):
        for kv in d.kv:
            kv.valid[:, :, 20:] = 0
    old = _tensors(dec)
    got = dec.verify_tree(E, nodes=_i32([9]))
    with pytest.raises(dv.DvError) as e:
        dec.check()
    assert e.value.status == 8
    _unchanged(dec, old, 0, 23, 64)
    want = ref.verify_tree(E)
    ref.check()
    _close(got, want)


@pytest.mark.parametrize("T", [3, 5])
def test_a_tree_that_ends_with_the_cache(T):
    """Three nodes fill the last three slots (two more are padding): the same as
    in a longer cache."""
    E = _inputs(1, T, 512, 34)
    dec, ref = _decoder(1), _decoder(1, n_max=80)
    g = torch.Generator(device="cuda").manual_seed(35)
    for a, b in zip(dec.kv, ref.kv):
        X = torch.randn(61, 512, generator=g, device="cuda").to(a.X.dtype)
        a.X[0, :61], b.X[0, :61] = X, X
        a.valid.zero_(), b.valid.zero_()
    dec.pos.fill_(61), ref.pos.fill_(61)
    nodes = _i32([3])
    got, want = dec.verify_tree(E, nodes=nodes), ref.verify_tree(E, nodes=nodes)
    dec.check(), ref.check()
    _close(got[:, :3], want[:, :3])
    for a, b in zip(dec.kv, ref.kv):
        assert a.valid.all()
        _close(a.K, b.K[:, :, :64])
        _close(a.X, b.X[:, :64])


def test_verify_captured_and_replayed():
    """One graph of the pass: streams, lengths and positions are read at replay,
    a tree that does not fit among them."""
    E, nodes = _inputs(2, 4, 512, 39), _i32([4, 2])
    dec, ref = _filled(2, [20, 30]), _filled(2, [20, 30])
    dec.verify_tree(E, nodes=nodes)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = dec.verify_tree(E, nodes=nodes)
    for pos, n, status in (([25, 60], [3, 4], 0), ([0, 33], [0, 4], 0), ([61, 11], [4, 1], 9)):
        for d in (dec, ref):
            for kv, o in zip(d.kv, _filled(2, pos).kv):
                for t, u in ((kv.K, o.K), (kv.V, o.V), (kv.X, o.X), (kv.valid, o.valid)):
                    t.copy_(u)
            d.pos.copy_(_i32(pos))
        nodes.copy_(_i32(n))
        E.copy_(_inputs(2, 4, 512, pos[0]))
        graph.replay()
        want = ref.verify_tree(E, nodes=nodes)
        for d in (dec, ref):
            if status:
                with pytest.raises(dv.DvError) as e:
                    d.check()
                assert e.value.status == status
            else:
                d.check()
        for b in range(2):
            if pos[b] + n[b] <= 64:
                _close(got[b, :n[b]], want[b, :n[b]]) if n[b] else None
            for a, o in zip(dec.kv, ref.kv):
                _close(a.X[b], o.X[b])
                assert torch.equal(a.valid[b], o.valid[b])


@pytest.mark.parametrize("bad", [
    dict(nodes=torch.tensor([3, 2])), dict(nodes=torch.tensor([[3], [2]], dtype=torch.int32)),
    dict(nodes=torch.tensor([3], dtype=torch.int32)), dict(mask=torch.ones(3, 3)),
    dict(mask=torch.ones(3, 4, dtype=torch.bool)), dict(mask=torch.ones(1, 3, 3, dtype=torch.bool)),
    dict(mask=torch.ones(3, 3, dtype=torch.bool).t()), dict(mask=torch.ones(3, 3, dtype=torch.bool), cpu=True),
])
def test_verify_refuses_before_it_writes(bad):
    dec = _filled(2, [30, 30])
    old = _tensors(dec)
    with pytest.raises(ValueError):
        dec.verify_tree(_inputs(2, 3, 512, 36), **{k: t if "cpu" in bad else t.cuda() for k, t in bad.items() if k != "cpu"})
    for b in range(2):
        _unchanged(dec, old, b, 0, 64)
    dec.check()


def test_verify_does_not_inherit_the_launch_policy(monkeypatch):
    """A call right after the predictor that writes its list must not start
    early, whatever level the process is at; the level is left as it was."""
    dec = _decoder(1)
    seen = []

    def level(fn):
        def call(*a, **kw):
            now = dv.dv_set_launch_overlap(0)
            dv.dv_set_launch_overlap(now)
            seen.append(now)
            return fn(*a, **kw)
        return call

    monkeypatch.setattr(stack.dv, "dv_sparse_mlp", level(dv.dv_sparse_mlp))
    prev = dv.dv_set_launch_overlap(1)
    try:
        dec.verify_tree(_inputs(1, 1, 512, 37))
        dec.check()
        after = dv.dv_set_launch_overlap(1)
        monkeypatch.setattr(stack.dv, "dv_kv_repair", None)     # ... also when a call fails
        with pytest.raises(TypeError):
            dec.verify_tree(_inputs(1, 1, 512, 37))
        failed = dv.dv_set_launch_overlap(1)
    finally:
        dv.dv_set_launch_overlap(prev)
    assert seen == [0] * dec.L and after == 1 and failed == 1


def test_buffers_of_many_tree_sizes_stay_bounded():
    """Trees of every size up to 24: what is kept for them is bounded by the
    largest, not by how many sizes there were, and sizes that share buffers
    give the same results."""
    def kept(sizes):
        dec = _decoder(1)
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        for T in sizes:
            dec.verify_tree(_inputs(1, T, 512, T))
        dec.check()
        torch.cuda.synchronize()
        return torch.cuda.memory_allocated() - before

    one = kept([24])
    assert kept([24] + list(range(1, 24))) <= 1.01 * one
    assert kept(range(1, 25)) <= 3 * one
    dec = _decoder(1)
    dec.verify_tree(_inputs(1, 24, 512, 24))
    for T in (1, 5, 16):
        fresh = _decoder(1)
        want, got = fresh.verify_tree(_inputs(1, T, 512, T)), dec.verify_tree(_inputs(1, T, 512, T))
        dec.check(), fresh.check()
        _close(got, want)


def test_verify_refuses_no_nodes():
    dec = _decoder(1)
    with pytest.raises(ValueError):
        dec.verify_tree(torch.zeros(1, 0, 512, device="cuda"))


def test_check_reports_a_failure_once():
    """A refused tree leaves an error in the repair's workspace and in the
    attention's: one check reads and clears both."""
    dec = _filled(1, [62])
    dec.verify_tree(_inputs(1, 5, 512, 40))
    with pytest.raises(dv.DvError) as e:
        dec.check()
    assert e.value.status == 9
    dec.check()


@pytest.mark.parametrize("keep_all", [True, False])
def test_the_output_projection_keeps_its_bits(monkeypatch, keep_all):
    """The streams behind the attention are what the attention gave times Wo, in
    fp32 as in a decode step: 512 products (2^-24 each of the summed magnitudes)
    and two roundings, not one to 16 bits."""
    dec = _decoder(2, keep_all=keep_all)
    E = _inputs(2, 7, 512, 41)
    ln, tree = dv.dv_layernorm, dv.dv_tree_attn
    streams, outs = [], []
    monkeypatch.setattr(stack.dv, "dv_layernorm", lambda x, *a, **kw: (streams.append(x.clone()), ln(x, *a, **kw)))
    monkeypatch.setattr(stack.dv, "dv_tree_attn",
                        lambda *a, **kw: (tree(*a, **kw), outs.append(a[4].clone())))
    dec.verify_tree(E)
    dec.check()
    for l in range(dec.L):
        before, after = streams[2 * l].double(), streams[2 * l + 1].double()
        out, Wo = outs[l].view(14, 512).double(), dec.layers[l]["Wo"].view(512, 512).double()
        want = before + out @ Wo
        tol = 512 * 2.0 ** -24 * (out.abs() @ Wo.abs()) + 2.0 ** -23 * (want.abs() + before.abs())
        assert ((after - want).abs() <= tol).all()


@pytest.mark.parametrize("B,T,tree", [(1, 5, True), (2, 9, False), (3, 20, True)])
def test_sparse_trees_of_several_nodes(monkeypatch, B, T, tree):
    """Few heads and neurons kept, several nodes: the streams against the same
    pass in 64 bits with the sets that the predictor gave.  The sets' inputs are
    checked too: heads from node 0, neurons node by node, both from the layer
    before (layer 0: its own attention input).

    y is rounded to the storage type in both; the pass rounds q, the attention's
    output and its projection as well (see TOL), and a y that falls across a
    rounding moves by a step."""
    dec = _decoder(B, keep_all=False)
    E = _inputs(B, T, 512, 38)
    mask = torch.ones(T, T, dtype=torch.bool).tril()
    if tree:                                  # two chains that share node 0
        odd = torch.arange(T) % 2
        mask &= (odd[:, None] == odd[None, :]) | (torch.arange(T) == 0)[None, :]
    sets = []
    predict = dv.dv_predict

    def spy(y, predictors, *a, **kw):
        predict(y, predictors, *a, **kw)
        (p,) = predictors
        sets.append((y.clone(), p.idx.clone(), p.count.clone()))

    monkeypatch.setattr(stack.dv, "dv_predict", spy)
    got = dec.verify_tree(E, mask=mask.cuda() if tree else None)
    dec.check()
    monkeypatch.undo()
    h, d_h, d = dec.h, dec.d_h, dec.d
    chunks = (B * T + 31) // 32
    assert len(sets) == dec.L * (1 + chunks)

    def ln(r):
        m = r.mean(-1, keepdim=True)
        v = ((r - m) ** 2).mean(-1, keepdim=True)
        return ((r - m) / (v + dec.eps).sqrt()).to(dec.dtype).double()

    def near(y, want):                        # stored values: half a step each, and what came in
        e = float((y.double() - want).norm() / want.norm())
        assert e <= TOL, e

    r, src = E.double().reshape(B * T, d), None
    for l in range(dec.L):
        W = {k: v.double() for k, v in dec.layers[l].items()}
        y = ln(r)
        src = y if l == 0 else src
        calls = sets[l * (1 + chunks):(l + 1) * (1 + chunks)]
        near(calls[0][0], src.view(B, T, d)[:, 0])
        near(torch.cat([c[0] for c in calls[1:]]), src)
        att = torch.zeros(B * T, d, dtype=torch.float64, device="cuda")
        for b in range(B):
            rows = y.view(B, T, d)[b]
            X = torch.cat([dec.kv[l].X[b, :N_PROMPT].double(), rows])
            see = torch.cat([torch.ones(T, N_PROMPT, dtype=torch.bool), mask], 1).cuda()
            idx = calls[0][1][b, :int(calls[0][2][b])].tolist()
            assert len(idx) == dec.k_heads < h
            for i in idx:
                q, k, v = (x @ W["Wqkv"][i, m].T for x, m in ((rows, 0), (X, 1), (X, 2)))
                s = (q @ k.T * dec.scale).masked_fill(~see, -math.inf)
                att.view(B, T, d)[b] += torch.softmax(s, 1) @ v @ W["Wo"][i]
        r = r + att
        ya, y = y, ln(r)
        out = torch.zeros_like(r)
        for n in range(B * T):
            _, idx, cnt = calls[1 + n // 32]
            j = idx[n % 32, :int(cnt[n % 32])].long()
            assert len(j) == dec.k_neurons < dec.N
            out[n] = torch.relu(W["W1n"][j] @ y[n]) @ W["W2n"][j]
        r, src = r + out, ya
    near(got.reshape(B * T, d), r)


def test_the_first_tree_of_a_size_is_not_captured():
    """Buffers made inside a capture would hold nothing until the graph's first
    replay: refused, and nothing is kept of the attempt."""
    dec = _filled(1, [20])
    E = _inputs(1, 3, 512, 42)
    with pytest.raises(RuntimeError):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            dec.verify_tree(E)
    want = _filled(1, [20]).verify_tree(E)
    _close(dec.verify_tree(E), want)
    dec.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = dec.verify_tree(E)
    graph.replay()
    _close(got, want)


@pytest.mark.parametrize("dtype,tol", [("f32", 1e-5), ("bf16", 8 * 2.0 ** -8)])
def test_linear_draft_in_other_types(dtype, tol):
    """As in f16: half-steps of the type per layer, fp32's own sums for f32."""
    w = Workload("cand", 72, d=512, h=8, d_h=64, N=1024, r=64, dtype=dtype, layers=2, n_prompt=N_PROMPT)
    layers = [layer_weights(w, l, device="cuda") for l in range(w.layers)]
    decs = []
    for _ in range(2):
        dec = stack.SparseDecoder(layers, 2, 64, 8, w.N, 0.125)
        dec.prefill([torch.stack([embeddings(w, N_PROMPT, f"X{l}/{b}", device="cuda") for b in range(2)])
                     for l in range(w.layers)], N_PROMPT)
        decs.append(dec)
    E = _inputs(2, 5, 512, 43)
    got = decs[0].verify_tree(E)
    decs[0].check()
    for t in range(5):
        want = _step(decs[1], E[:, t])
        assert float((got[:, t].double() - want.double()).norm() / want.double().norm()) <= tol
