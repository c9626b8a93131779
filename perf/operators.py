"""Measured cases of the operators that answer with several candidates per
sequence: attention of a drafted token tree over the KV cache, compaction of
the accepted nodes, beam selection over beams and vocabulary, and the
reordering of the beams' caches.

``run`` computes an operator in its plain form (elementary torch operations)
while ``own`` is false and through the library's entry points while it is true.

Layouts (as in include/dv.h): K, V [B][h][n_max][d_h], X [B][n_max][d],
valid [B][h][n_max] uint8; a decoder's layers are kept as one allocation per
tensor with the layer in front.
"""

import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_ES = {"f32": 4, "f16": 2, "bf16": 2}


# --------------------------------------------------------------------- cases

def listed():
    return [
        # one sequence, a handful of drafted tokens, every head of an
        # OPT-1.3B-shaped layer: the call whose latency shows
        dict(name="tree_1x8_of_512", op="tree", dt="f16", B=1, h=32, g=1, d_h=64, n=512, T=8, keep=32,
             ragged=False, mask="tree"),
        # contextual sparsity kept in the verify step: 20 % of the heads of an
        # OPT-13B-shaped layer, a linear draft of odd length
        dict(name="tree_1x21_of_1089_sparse", op="tree", dt="f16", B=1, h=40, g=1, d_h=128, n=1089, T=21, keep=8,
             ragged=False, mask="chain"),
        # OPT-175B-shaped layer, batch 8, 64-node trees: the largest
        dict(name="tree_8x64_of_2047", op="tree", dt="f16", B=8, h=96, g=1, d_h=128, n=2047, T=64, keep=96,
             ragged=False, mask="tree"),
        # long contexts of unequal length, five query heads to a K/V head,
        # trees that are not all full
        dict(name="tree_3x25_of_32768_shared", op="tree", dt="bf16", B=3, h=8, g=5, d_h=128, n=32768, T=25, keep=8,
             ragged=True, mask="tree"),
        # 32-bit storage
        dict(name="tree_3x7_of_1000_f32", op="tree", dt="f32", B=3, h=12, g=1, d_h=64, n=1000, T=7, keep=12,
             ragged=True, mask="tree"),
        # a 40-layer OPT-13B-shaped stack keeps 4 of 21 drafted tokens
        dict(name="compact_40_layers", op="compact", dt="f16", L=40, B=1, h=40, d_h=128, n=1024, T=21, cap=8,
             keep=40),
        # OPT-30B-shaped layers, batch 32, half the heads present
        dict(name="compact_8_layers_batch_32", op="compact", dt="bf16", L=8, B=32, h=56, d_h=128, n=600, T=64,
             cap=12, keep=28),
        # one sequence, four beams
        dict(name="beam_1x4_of_32000", op="beam", dt="f16", S=1, W=4, V=32000, K=4, done=False),
        # a small batch in 32 bits, twice as many candidates as beams, odd rows
        dict(name="beam_8x8_of_50257_f32", op="beam", dt="f32", S=8, W=8, V=50257, K=16, done=True),
        # a large batch over a large vocabulary
        dict(name="beam_48x10_of_128001", op="beam", dt="bf16", S=48, W=10, V=128001, K=20, done=True),
        # one layer, one sequence, four short beams
        dict(name="reorder_1x4_of_512", op="reorder", dt="f16", L=1, S=1, W=4, h=32, d_h=64, n=512, start=400,
             keep=32),
        # OPT-30B-shaped layers, four sequences of eight beams, half the heads
        # present, the prompt shared by a sequence's beams
        dict(name="reorder_3_layers_4x8", op="reorder", dt="bf16", L=3, S=4, W=8, h=56, d_h=128, n=1500, start=1003,
             keep=28),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "compact", "beam", "beam", "reorder"])
    dt = rng.choice(["f16", "bf16", "f16", "bf16", "f32"])
    d_h = rng.choice([64, 128])
    if op == "tree":
        g = rng.choice([1, 1, 1, 2, 3, 5, 8])
        h = _log(rng, 4, 96 // g)
        T = _log(rng, 1, min(96 if dt != "f32" else 24, 256 // g))
        B = _log(rng, 1, 16)
        most = 4.0e8 if dt != "f32" else 4.0e7   # bytes of K and V
        n = _log(rng, 1, int(max(2, min(32768, most / (2 * B * h * d_h * _ES[dt])))))
        return dict(op=op, dt=dt, B=B, h=h, g=g, d_h=d_h, n=n, T=T, keep=rng.randint(1, h),
                    ragged=rng.random() < 0.5, mask=rng.choice(["tree", "tree", "chain"]))
    if op == "compact":
        L, B, h = _log(rng, 1, 40), _log(rng, 1, 16), _log(rng, 4, 64)
        T = _log(rng, 1, 64)
        n = _log(rng, 1, int(max(2, min(2000, 1.2e9 / (3 * L * B * h * d_h * _ES[dt])))))
        return dict(op=op, dt=dt, L=L, B=B, h=h, d_h=d_h, n=n, T=T, cap=rng.randint(1, min(T, 16)),
                    keep=rng.randint(1, h))
    if op == "beam":
        S, W = _log(rng, 1, 32), rng.randint(1, 10)
        V = _log(rng, 1000, 128000)
        return dict(op=op, dt=dt, S=S, W=W, V=V, K=rng.choice([W, 2 * W]), done=rng.random() < 0.5)
    L, S, W, h = _log(rng, 1, 8), _log(rng, 1, 4), rng.randint(2, 10), _log(rng, 4, 56)
    n = _log(rng, 16, int(max(17, min(1500, 1.5e9 / (3 * L * S * W * h * d_h * _ES[dt])))))
    return dict(op=op, dt=dt, L=L, S=S, W=W, h=h, d_h=d_h, n=n, start=rng.randint(0, n - 1), keep=rng.randint(1, h))


# ----------------------------------------------------- sizes that a case fixes

def _lengths(c):
    """Positions in each sequence's cache, and nodes of each tree."""
    if not c["ragged"]:
        return [c["n"]] * c["B"], [c["T"]] * c["B"]
    ns = [max(0, c["n"] - (b * 2654435761 % 997) * c["n"] // 2000) for b in range(c["B"])]
    ts = [max(1, c["T"] - (b * 40503 % 7) * c["T"] // 12) for b in range(c["B"])]
    return ns, ts


def _accepted(c):
    return [1 + (b * 7 + 3) % c["cap"] for b in range(c["B"])]


def _beam_lengths(c):
    return [max(1, c["n"] - 3 * s) for s in range(c["S"])]


def _n_max(n):
    return max(16, (n + 15) // 16 * 16)


# -------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 17)
    return g


def _normal(shape, dt, g, std=1.0):
    x = torch.empty(shape, dtype=_DT[dt], device="cuda")
    x.normal_(0.0, std, generator=g)
    return x


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _tree_mask(B, T, g):
    """Ancestor masks of random trees: node u's parent is an earlier node or
    (for a root) the committed sequence."""
    parent = (torch.rand(B, T, device="cuda", generator=g).sqrt() * torch.arange(T, device="cuda")).long() - 1
    m = torch.zeros(B, T + 1, T, dtype=torch.bool, device="cuda")   # row T: a root's empty ancestry
    rows = torch.arange(B, device="cuda")
    for t in range(T):
        p = parent[:, t]
        m[:, t] = m[rows, torch.where(p < 0, T, p)]
        m[:, t, t] = True
    return m[:, :T].contiguous()


def _head_lists(B, h, keep, g):
    idx = torch.rand(B, h, device="cuda", generator=g).argsort(dim=1)[:, :keep].sort(dim=1).values
    return idx.int().contiguous(), torch.full((B,), keep, dtype=torch.int32, device="cuda")


def _caches(c, B, n_max, g):
    """Stacked caches [L][...] with `keep` of the heads present per row."""
    L, h, d_h = c["L"], c["h"], c["d_h"]
    st = dict(K=_normal((L, B, h, n_max, d_h), c["dt"], g), V=_normal((L, B, h, n_max, d_h), c["dt"], g),
              X=_normal((L, B, n_max, h * d_h), c["dt"], g))
    have = torch.rand(L, B, h, device="cuda", generator=g).argsort(dim=2) < c["keep"]
    st["valid"] = have[..., None].expand(L, B, h, n_max).to(torch.uint8).contiguous()
    return st


def _layers(dv, st):
    return dv.KVLayers([dv.KV(st["K"][l], st["V"][l], st["X"][l], st["valid"][l]) for l in range(st["K"].shape[0])])


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = dict(case=case)
    if c["op"] == "tree":
        ns, ts = _lengths(c)
        B, T, h = c["B"], c["T"], c["h"]
        n_max = _n_max(max(ns) + T)
        st.update(q=_normal((B, T, h * c["g"], c["d_h"]), c["dt"], g), K=_normal((B, h, n_max, c["d_h"]), c["dt"], g),
                  V=_normal((B, h, n_max, c["d_h"]), c["dt"], g), pos=_i32(ns), scale=c["d_h"] ** -0.5,
                  nodes=_i32(ts) if c["ragged"] else None,
                  mask=_tree_mask(B, T, g) if c["mask"] == "tree" else None, head_idx=None, head_count=None)
        if c["keep"] < h:
            st["head_idx"], st["head_count"] = _head_lists(B, h, c["keep"], g)
        st["out"] = torch.zeros_like(st["q"])
    elif c["op"] == "compact":
        B, T = c["B"], c["T"]
        n_max = _n_max(c["n"] + T)
        st.update(_caches(c, B, n_max, g))
        count = _accepted(c)
        order = torch.rand(B, T, device="cuda", generator=g).argsort(dim=1)
        idx = torch.zeros(B, c["cap"], dtype=torch.int32, device="cuda")
        for b in range(B):
            idx[b, :count[b]] = order[b, :count[b]].sort().values.int()
        st.update(pos=_i32([c["n"] - b % max(1, c["n"] // 2) for b in range(B)]), idx=idx, count=_i32(count),
                  new_pos=torch.zeros(B, dtype=torch.int32, device="cuda"))
    elif c["op"] == "beam":
        S, W, V, K = c["S"], c["W"], c["V"], c["K"]
        logits = _normal((S, W, V), c["dt"], g, 3.0)
        logits[:, :, torch.randint(0, V, (V // 50 + 1,), device="cuda", generator=g)] = -math.inf   # tokens ruled out
        st.update(logits=logits, cum=-6.0 * torch.rand(S, W, device="cuda", generator=g), end=V // 3,
                  done=(torch.rand(S, W, device="cuda", generator=g) < 0.2).to(torch.uint8) if c["done"] else None,
                  score=torch.zeros(S, K, device="cuda"), token=torch.zeros(S, K, dtype=torch.int32, device="cuda"),
                  beam=torch.zeros(S, K, dtype=torch.int32, device="cuda"))
    else:
        S, W = c["S"], c["W"]
        st.update(_caches(c, S * W, _n_max(c["n"]), g))
        lens = _beam_lengths(c)
        st.update(pos=_i32([n for n in lens for _ in range(W)]), start=_i32([min(c["start"], n) for n in lens]),
                  parent=torch.randint(0, W, (S, W), device="cuda", generator=g).int())
    if own:
        from contextual_sparsity_decode_gb300 import binding as dv
        st["dv"] = dv
        if c["op"] == "tree":
            st["kv"] = dv.KV(st["K"], st["V"], None, None)
            st["ws"] = dv.workspace(dv.dv_tree_attn_workspace_size(c["B"], c["T"], c["h"], c["g"], c["d_h"]))
        elif c["op"] == "beam":
            st["ws"] = dv.workspace(dv.dv_beam_select_workspace_size(c["S"], c["W"], c["V"], c["K"]))
        else:
            st["layers"], st["ws"] = _layers(dv, st), dv.workspace(256)
    return st


# --------------------------------------------------------------- plain forms

def _plain_tree(st):
    q, K, V, pos = st["q"], st["K"], st["V"], st["pos"]
    B, T, hq, d_h = q.shape
    h, n_max = K.shape[1], K.shape[2]
    g = hq // h
    qf = q.float().view(B, T, h, g, d_h).permute(0, 2, 1, 3, 4).reshape(B, h, T * g, d_h)
    Kf, Vf = K.float(), V.float()
    if st["head_idx"] is not None:
        at = st["head_idx"].long()[:, :, None, None]
        qf = qf.gather(1, at.expand(-1, -1, T * g, d_h))
        Kf, Vf = Kf.gather(1, at.expand(-1, -1, n_max, d_h)), Vf.gather(1, at.expand(-1, -1, n_max, d_h))
    nodes = st["nodes"] if st["nodes"] is not None else torch.full_like(pos, T)
    mask = st["mask"]
    if mask is None:
        mask = torch.ones(T, T, dtype=torch.bool, device=q.device).tril().expand(B, T, T)
    j = torch.arange(n_max, device=q.device)
    u = j[None, :] - pos[:, None]                               # slot of the tree, [B][n_max]
    in_tree = (u >= 0) & (u < nodes[:, None])
    seen = mask.gather(2, u.clamp(0, T - 1)[:, None, :].expand(B, T, n_max)) & in_tree[:, None, :]
    seen = seen | (u < 0)[:, None, :]
    seen = seen & (torch.arange(T, device=q.device)[None, :, None] < nodes[:, None, None])
    seen = seen.repeat_interleave(g, dim=1)[:, None]            # [B][1][T g][n_max]
    s = torch.matmul(qf, Kf.transpose(2, 3)) * st["scale"]
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    top = s.amax(dim=3, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(dim=3, keepdim=True)
    o = torch.matmul(p / torch.where(total > 0, total, torch.ones_like(total)), Vf)
    o = o.view(B, -1, T, g, d_h)
    full = torch.zeros(B, h, T, g, d_h, device=q.device)
    if st["head_idx"] is not None:
        full.scatter_(1, st["head_idx"].long()[:, :, None, None, None].expand_as(o), o)
    else:
        full = o
    st["out"].copy_(full.permute(0, 2, 1, 3, 4).reshape(B, T, hq, d_h))
    return st["out"]


def _plain_compact(st):
    K, V, X, valid, pos, idx, count = (st[k] for k in ("K", "V", "X", "valid", "pos", "idx", "count"))
    L, B, h, n_max, d_h = K.shape
    k = torch.arange(idx.shape[1], device=K.device)
    live = k[None, :] < count[:, None]                           # [B][cap]
    dst = (pos[:, None] + k[None, :]).long().clamp(max=n_max - 1)
    src = torch.where(live, (pos[:, None] + idx).long(), dst)
    b = torch.arange(B, device=K.device)[:, None].expand_as(dst)
    sv = valid[:, b, :, src]                                     # [B][cap][L][h]
    for t in (K, V):
        old, new = t[:, b, :, dst], t[:, b, :, src]              # [B][cap][L][h][d_h]
        new = torch.where((live[:, :, None, None] & (sv != 0))[..., None], new, old)
        t[:, b[live], :, dst[live]] = new[live]
    X[:, b[live], dst[live]] = X[:, b[live], src[live]]
    valid[:, b[live], :, dst[live]] = sv[live]
    st["new_pos"].copy_(pos + count)
    return dict(K=K, V=V, X=X, valid=valid, new_pos=st["new_pos"])


def _plain_beam(st):
    x, cum, done = st["logits"].double(), st["cum"].double(), st["done"]
    S, W, V = x.shape
    K = st["score"].shape[1]
    top = x.amax(dim=2, keepdim=True)
    lse = top + torch.exp(x - top).sum(dim=2, keepdim=True).log()
    total = cum[:, :, None] + (x - lse)
    if done is not None:
        ended = torch.full_like(total, -math.inf)
        ended[:, :, st["end"]] = cum
        total = torch.where((done != 0)[:, :, None], ended, total)
    best, at = torch.sort(total.view(S, W * V), dim=1, descending=True, stable=True)
    st["score"].copy_(best[:, :K])
    st["token"].copy_(at[:, :K] % V)
    st["beam"].copy_(at[:, :K] // V)
    return dict(score=st["score"], token=st["token"], beam=st["beam"])


def _plain_reorder(st):
    K, V, X, valid, pos, start, parent = (st[k] for k in ("K", "V", "X", "valid", "pos", "start", "parent"))
    S, W = parent.shape
    src = (torch.arange(S, device=K.device)[:, None] * W + parent).view(-1).long()   # [S W]
    j = torch.arange(K.shape[3], device=K.device)
    moved = (j[None, :] >= start.repeat_interleave(W)[:, None]) & (j[None, :] < pos[src][:, None])
    sv = valid[:, src]
    there = moved[None, :, None, :] & (sv != 0)
    K.copy_(torch.where(there[..., None], K[:, src], K))
    V.copy_(torch.where(there[..., None], V[:, src], V))
    X.copy_(torch.where(moved[None, :, :, None], X[:, src], X))
    valid.copy_(torch.where(moved[None, :, None, :], sv, valid))
    return dict(K=K, V=V, X=X, valid=valid)


def run(state):
    st, op = state, state["case"]["op"]
    if own:
        dv = st["dv"]
        if op == "tree":
            dv.dv_tree_attn(st["q"], st["kv"], st["pos"], st["scale"], st["out"], st["ws"], mask=st["mask"],
                            nodes=st["nodes"], head_idx=st["head_idx"], head_count=st["head_count"])
            return st["out"]
        if op == "compact":
            dv.dv_kv_compact(st["layers"], st["pos"], st["idx"], st["count"], st["ws"], new_pos=st["new_pos"])
            return {k: st[k] for k in ("K", "V", "X", "valid", "new_pos")}
        if op == "beam":
            dv.dv_beam_select(st["logits"], st["cum"], st["score"], st["token"], st["beam"], st["ws"],
                              done=st["done"], end_token=st["end"])
            return {k: st[k] for k in ("score", "token", "beam")}
        dv.dv_kv_reorder(st["layers"], st["pos"], st["parent"], st["ws"], start=st["start"])
        return {k: st[k] for k in ("K", "V", "X", "valid")}
    return {"tree": _plain_tree, "compact": _plain_compact, "beam": _plain_beam, "reorder": _plain_reorder}[op](st)


# ---------------------------------------------------------------------- work

def work(case):
    c, es = case, _ES[case["dt"]]
    if c["op"] == "tree":
        ns, ts = _lengths(c)
        rows = [min(c["T"], t) for t in ts]
        keys = sum(n + t for n, t in zip(ns, ts))
        kv = 2 * c["keep"] * keys * c["d_h"] * es
        q = sum(rows) * c["keep"] * c["g"] * c["d_h"] * es
        out = c["B"] * c["T"] * c["h"] * c["g"] * c["d_h"] * es
        mask = c["B"] * c["T"] * c["T"] if c["mask"] == "tree" else 0
        flops = 4 * c["keep"] * c["g"] * c["d_h"] * sum((n + t) * r for n, t, r in zip(ns, ts, rows))
        return dict(bytes=kv + q + out + mask, flops=flops)
    if c["op"] == "compact":
        rows = sum(_accepted(c))                                 # read once, written once
        row = 2 * c["keep"] * c["d_h"] * es + c["h"] * c["d_h"] * es + c["h"]
        return dict(bytes=2 * c["L"] * rows * row, flops=0)
    if c["op"] == "beam":
        n = c["S"] * c["W"] * c["V"]
        return dict(bytes=n * es + c["S"] * c["K"] * 12, flops=4 * n)
    # a parent drawn at random leaves a beam where it is once in W; the beams
    # that move take their rows from about W (1 - 1/e) distinct parents
    W, rows = c["W"], sum(max(0, n - min(c["start"], n)) for n in _beam_lengths(c))
    written = W - 1
    read = W * (1.0 - (1.0 - 1.0 / W) ** (W - 1))
    row = 2 * c["keep"] * c["d_h"] * es + c["h"] * c["d_h"] * es + c["h"]
    return dict(bytes=int(c["L"] * rows * (read + written) * row), flops=0)


# ---------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    c, st = case, prepare(case, seed)
    if c["op"] == "tree":
        # one (sequence, head) at a time, the softmax taken row by row over
        # exactly the visible positions
        ns, ts = _lengths(c)
        B, T, hq, d_h = st["q"].shape
        out = torch.zeros(B, T, hq, d_h, dtype=torch.float64, device="cuda")
        for b in range(B):
            n, t = ns[b], ts[b]
            low = torch.tril(torch.ones(t, t, device="cuda")) > 0 if st["mask"] is None else st["mask"][b, :t, :t]
            ok = torch.cat([torch.ones(t, n, dtype=torch.bool, device="cuda"), low], dim=1)
            heads = range(c["h"]) if st["head_idx"] is None else st["head_idx"][b].tolist()
            for i in heads:
                k, v = st["K"][b, i, :n + t].double(), st["V"][b, i, :n + t].double()
                for e in range(c["g"]):
                    w = (st["q"][b, :t, i * c["g"] + e].double() @ k.T * st["scale"]).masked_fill(~ok, -math.inf)
                    out[b, :t, i * c["g"] + e] = torch.softmax(w, dim=1) @ v
        return out
    if c["op"] == "compact":
        pos, idx, count = (st[k].tolist() for k in ("pos", "idx", "count"))
        for b in range(c["B"]):
            for k in range(count[b]):                            # ascending: a slot is read before it is written
                to, at = pos[b] + k, pos[b] + idx[b][k]
                there = st["valid"][:, b, :, at].bool()
                for t in (st["K"], st["V"]):
                    t[:, b, :, to][there] = t[:, b, :, at][there]
                st["X"][:, b, to] = st["X"][:, b, at].clone()
                st["valid"][:, b, :, to] = st["valid"][:, b, :, at].clone()
        new = _i32([p + m for p, m in zip(pos, count)])
        return dict(K=st["K"], V=st["V"], X=st["X"], valid=st["valid"], new_pos=new)
    if c["op"] == "beam":
        S, W, V, K = c["S"], c["W"], c["V"], c["K"]
        cum = st["cum"].double().cpu().numpy()
        done = np.zeros((S, W), bool) if st["done"] is None else st["done"].cpu().numpy() != 0
        score, token, beam = np.zeros((S, K)), np.zeros((S, K), np.int32), np.zeros((S, K), np.int32)
        for s in range(S):
            x = st["logits"][s].double()
            logp = torch.log_softmax(x, dim=1)
            # candidates of a beam: everything not below its K-th largest
            kth = torch.topk(logp, min(K, V), dim=1).values[:, -1:]
            rows, cols = (t.cpu().numpy() for t in torch.nonzero(logp >= kth, as_tuple=True))
            vals = cum[s][rows] + logp.cpu().numpy()[rows, cols]
            keep = ~done[s][rows]
            ends = np.flatnonzero(done[s])
            rows, cols, vals = (np.concatenate(p) for p in ((rows[keep], ends), (cols[keep], np.full(len(ends), st["end"])),
                                                            (vals[keep], cum[s][ends])))
            if len(rows) < K:
                return None                                      # fewer candidates than asked for: ties at -inf
            first = np.lexsort((rows * V + cols, -vals))[:K]
            score[s], token[s], beam[s] = vals[first], cols[first], rows[first]
        return dict(score=score, token=token, beam=beam)
    # every beam's row is taken from a copy of the cache as it was
    parent, pos, start = (st[k].tolist() for k in ("parent", "pos", "start"))
    W = c["W"]
    for s in range(c["S"]):
        old = {k: st[k][:, s * W:(s + 1) * W].clone() for k in ("K", "V", "X", "valid")}
        for w in range(W):
            p = parent[s][w]
            lo, hi = start[s], pos[s * W + p]
            if hi <= lo:
                continue
            there = old["valid"][:, p, :, lo:hi].bool()
            for k in ("K", "V"):
                st[k][:, s * W + w, :, lo:hi][there] = old[k][:, p, :, lo:hi][there]
            st["X"][:, s * W + w, lo:hi] = old["X"][:, p, lo:hi]
            st["valid"][:, s * W + w, :, lo:hi] = old["valid"][:, p, :, lo:hi]
    return dict(K=st["K"], V=st["V"], X=st["X"], valid=st["valid"])
