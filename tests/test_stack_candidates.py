"""A decoder stack with several candidates per sequence: drafted trees verified
in one pass, a path of them accepted, beams reordered -- against the same
decoder taking one token at a time.

Tolerance of a verified node's residual stream (relative L2): the verify pass
rounds q, the attention's output and its projection to the storage type where
the decode step keeps fp32, three half-steps per layer (2^-11 relative each in
f16), and what that moves y across a rounding adds one more: 4 per layer, two
layers, 8 half-steps."""

import math

import pytest
import torch

from contextual_sparsity_decode_gb300 import binding as dv
from contextual_sparsity_decode_gb300.stack import SparseDecoder
from synth import Workload, embeddings, layer_weights

pytestmark = pytest.mark.gpu

TOL = 8 * 2.0 ** -11
N_PROMPT = 21


def _decoder(B, d_h=64, h=8, keep_all=True, n_max=64, wid=71):
    w = Workload("cand", wid, d=h * d_h, h=h, d_h=d_h, N=1024, r=64, dtype="f16", layers=2, n_prompt=N_PROMPT)
    dev = "cuda"
    layers = [layer_weights(w, l, device=dev) for l in range(w.layers)]
    dec = SparseDecoder(layers, B, n_max, h if keep_all else 3, w.N if keep_all else 64, 1.0 / math.sqrt(d_h))
    X = [torch.stack([embeddings(w, N_PROMPT, f"X{l}/{b}", device=dev) for b in range(B)]) for l in range(w.layers)]
    dec.prefill(X, N_PROMPT)
    return dec


def _step(dec, e):
    """One decode step from the residual input e [B][d]; returns its output."""
    dec.r_stream.copy_(e)
    dec.step_ops()
    dv.dv_positions_advance(dec.pos, 0, dec.n_max)
    dec.check()
    return dec.r_stream.clone()


def _inputs(B, T, d, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(B, T, d, generator=g, device="cuda")


def _close(a, b):
    e = float((a.double() - b.double()).norm() / b.double().norm())
    assert e <= TOL, e


@pytest.mark.parametrize("B,T,d_h", [(1, 1, 64), (1, 5, 128), (2, 4, 64), (3, 13, 64)])
def test_linear_draft_matches_token_by_token(B, T, d_h):
    E = _inputs(B, T, 8 * d_h, 5)
    dec, ref = _decoder(B, d_h), _decoder(B, d_h)
    got = dec.verify_tree(E)
    dec.check()
    assert dec.pos.tolist() == [N_PROMPT] * B
    for t in range(T):
        _close(got[:, t], _step(ref, E[:, t]))


def test_tree_then_accept_then_decode():
    """Two branches (0-1-3 and 0-2-4) and an odd leaf (5 under 1).  Each node
    matches the decode of its own path; the accepted path 0-2-4 leaves the
    cache as that decode does, and decoding continues from it."""
    B, T = 2, 6
    parent = [-1, 0, 0, 1, 2, 1]
    mask = torch.zeros(T, T, dtype=torch.bool)
    for t, p in enumerate(parent):
        if p >= 0:
            mask[t] = mask[p]
        mask[t, t] = True
    E = _inputs(B, T, 512, 9)
    dec = _decoder(B)
    got = dec.verify_tree(E, mask=mask.cuda())
    for path in ([0, 1, 3], [0, 2, 4], [0, 1, 5]):
        ref = _decoder(B)
        for t in path:
            _close(got[:, t], _step(ref, E[:, t]))
    ref = _decoder(B)
    for t in (0, 2, 4):
        _step(ref, E[:, t])
    idx = torch.tensor([[0, 2, 4], [0, 2, 4]], dtype=torch.int32, device="cuda")
    dec.accept(idx, torch.tensor([3, 3], dtype=torch.int32, device="cuda"))
    dec.check()
    assert dec.pos.tolist() == ref.pos.tolist() == [N_PROMPT + 3] * B
    n = N_PROMPT + 3
    for a, b in zip(dec.kv, ref.kv):
        assert torch.equal(a.valid[:, :, :n], b.valid[:, :, :n])
        _close(a.K[:, :, N_PROMPT:n], b.K[:, :, N_PROMPT:n])
        _close(a.X[:, N_PROMPT:n], b.X[:, N_PROMPT:n])
    nxt = _inputs(B, 1, 512, 10)[:, 0]
    _close(_step(dec, nxt), _step(ref, nxt))
    # ... and a second tree, of another size and not full in the second sequence
    E2 = _inputs(B, 3, 512, 11)
    got = dec.verify_tree(E2, nodes=torch.tensor([3, 2], dtype=torch.int32, device="cuda"))
    dec.check()
    for t in range(3):
        out = _step(ref, E2[:, t])
        _close(got[0, t], out[0])
        if t < 2:
            _close(got[1, t], out[1])


def test_sparse_verify_uses_the_step_s_sets():
    """With few heads and neurons kept, one verified node equals one decode
    step: the same predictions, the same repairs."""
    E = _inputs(2, 1, 512, 13)
    dec, ref = _decoder(2, keep_all=False), _decoder(2, keep_all=False)
    for k in range(3):
        got = dec.verify_tree(E)
        _close(got[:, 0], _step(ref, E[:, 0]))
        dec.accept(torch.zeros(2, 1, dtype=torch.int32, device="cuda"),
                   torch.ones(2, dtype=torch.int32, device="cuda"))
        dec.check()
        E = _inputs(2, 1, 512, 14 + k)
    for a, b in zip(dec.kv, ref.kv):
        assert torch.equal(a.valid[:, :, :N_PROMPT + 3], b.valid[:, :, :N_PROMPT + 3])


def test_beam_search_reorders_the_caches():
    """Beam search over a small vocabulary: select, reorder, step.  After every
    reordering a step of beam w gives what the parent's row would have given
    (2+ rows add partial sums with fp32 atomics: 1e-5 relative)."""
    S, W, V = 2, 3, 211
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    dec, plain = _decoder(S * W), _decoder(S * W)
    same = [b - b % W for b in range(S * W)]           # a sequence's beams share its prompt
    for d in (dec, plain):
        for kv in d.kv:
            for t in (kv.K, kv.V, kv.X, kv.valid):
                t.copy_(t[same])
    emb = torch.randn(V, 512, generator=g, device="cuda")
    head = torch.randn(512, V, generator=g, device="cuda") / 16
    ws = dv.workspace(dv.dv_beam_select_workspace_size(S, W, V, W))
    score, token, beam = torch.zeros(S, W, device="cuda"), *(torch.zeros(S, W, dtype=torch.int32, device="cuda") for _ in range(2))
    start = torch.full((S,), N_PROMPT, dtype=torch.int32, device="cuda")
    r = _step(dec, emb[torch.zeros(S * W, dtype=torch.long, device="cuda")])
    _step(plain, emb[torch.zeros(S * W, dtype=torch.long, device="cuda")])
    cum = torch.full((S, W), -math.inf, device="cuda")
    cum[:, 0] = 0.0                                    # the first step's beams are all the same
    for _ in range(4):
        logits = (r @ head).view(S, W, V)
        dv.dv_beam_select(logits, cum, score, token, beam, ws)
        assert dv.dv_check(ws) == (0, 0)
        assert (score[:, 1:] <= score[:, :-1]).all() and torch.isfinite(score).all()
        cum.copy_(score)
        dec.reorder(beam, start)
        for kv in plain.kv:                            # the same by copies
            rows = (torch.arange(S, device="cuda")[:, None] * W + beam).view(-1).long()
            for t in (kv.K, kv.V, kv.X, kv.valid):
                t.copy_(t[rows])
        e = emb[token.view(-1).long()]
        r, want = _step(dec, e), _step(plain, e)
        assert float((r - want).norm() / want.norm()) <= 1e-5


def test_verify_refuses_other_shapes():
    dec = _decoder(2)
    for bad in (torch.zeros(1, 3, 512, device="cuda"), torch.zeros(2, 3, 256, device="cuda"),
                torch.zeros(2, 3, 512, device="cuda", dtype=torch.float16)):
        with pytest.raises(ValueError):
            dec.verify_tree(bad)


def test_a_tree_behind_the_cache_is_reported():
    dec = _decoder(1)
    dec.pos.fill_(dec.n_max - 3)
    dec.verify_tree(_inputs(1, 5, 512, 1))
    with pytest.raises(dv.DvError) as e:
        dec.check()
    assert e.value.status == 9
