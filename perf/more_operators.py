"""Measured cases of the operators around 4-bit weights and drawn tokens:
quantisation of a matrix to 4 bits with group scales, products of 1 to 32 rows
with such a matrix, the sparse MLP over such matrices, and sampling with
temperature, top-k, top-p and min-p from given random numbers.

``run`` computes an operator in its plain form (elementary torch operations)
while ``own`` is false and through the library's entry points while it is true.

A 4-bit matrix (as in include/dv.h): rows of ceil(d / 128) blocks of 64 bytes;
the 32-bit word w of a block, g = w / 2 and s = w % 2, holds the codes of the
elements 64 s + 8 g + e, e < 8, at bit 4 (e / 2) + 16 (e % 2); an element is
(code - 8) times the scale of its group of 64 or 128 elements.
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
        # a predictor-sized matrix in 32 bits, rows that end inside a block
        dict(name="quantize_1024x1000_f32", op="quantize", dt="f32", N=1024, d=1000, group=64),
        # one MLP matrix of an OPT-13B-shaped layer, as a model is converted
        dict(name="quantize_20480x5120", op="quantize", dt="f16", N=20480, d=5120, group=128),
        # a small projection, one token: the call whose latency shows
        dict(name="matvec_1_2048x2048", op="matvec", dt="f16", B=1, N=2048, d=2048, group=128),
        # the output head of an OPT-13B-shaped model, one token, an odd vocabulary
        dict(name="matvec_1_50257x5120", op="matvec", dt="f16", B=1, N=50257, d=5120, group=128),
        # a ragged matrix in 32 bits, a few rows
        dict(name="matvec_5_5001x5000_f32", op="matvec", dt="f32", B=5, N=5001, d=5000, group=64),
        # an OPT-30B-shaped projection to the neurons, a full batch
        dict(name="matvec_32_28672x7168", op="matvec", dt="bf16", B=32, N=28672, d=7168, group=64),
        # the benchmark's layer: 5 % of the neurons, one token
        dict(name="mlp_1_1024_of_20480x5120", op="mlp", dt="f16", B=1, N=20480, d=5120, k=1024, group=128),
        # half the neurons of an OPT-30B-shaped layer, one token
        dict(name="mlp_1_14336_of_28672x7168", op="mlp", dt="bf16", B=1, N=28672, d=7168, k=14336, group=128),
        # 16 tokens with lists of their own, 5 % each, groups of 64
        dict(name="mlp_16_1434_of_28672x7168", op="mlp", dt="bf16", B=16, N=28672, d=7168, k=1434, group=64),
        # one sequence, all filters
        dict(name="sample_1x32000", op="sample", dt="f16", B=1, V=32000, T="one", k=50, p=0.9, min_p=0.02),
        # a small batch drawn from the whole vocabulary, 32-bit logits of a head
        dict(name="sample_8x50257_f32", op="sample", dt="f32", B=8, V=50257, T="rows", k=0, p=1.0, min_p=0.0),
        # a large batch over a large vocabulary, nucleus sampling
        dict(name="sample_192x128001", op="sample", dt="bf16", B=192, V=128001, T="rows", k=0, p=0.95, min_p=0.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "matvec", "matvec", "mlp", "mlp", "sample", "sample"])
    dt = rng.choice(["f16", "bf16", "f16", "bf16", "f32"])
    group = rng.choice([64, 128])
    if op == "quantize":
        d = 8 * _log(rng, 8, 1024)
        return dict(op=op, dt=dt, N=_log(rng, 64, max(65, int(1.0e8 / d))), d=d, group=group)
    if op == "matvec":
        B, d = rng.choice([1, 1, 1, 2, 3, _log(rng, 4, 32)]), 8 * _log(rng, 32, 1536)
        return dict(op=op, dt=dt, B=B, N=_log(rng, 64, max(65, int(2.0e8 / d))), d=d, group=group)
    if op == "mlp":
        B, d = rng.choice([1, 1, 1, 2, _log(rng, 3, 32)]), 8 * _log(rng, 32, 1536)
        N = _log(rng, 256, 32768)
        most = max(17, int(2.0e8 / (B * d)))
        return dict(op=op, dt=dt, B=B, N=N, d=d, k=min(N, _log(rng, 16, most)), group=group)
    V = _log(rng, 300, 150000)
    return dict(op=op, dt=dt, B=_log(rng, 1, max(2, min(300, int(2.4e7 / V)))), V=V, T=rng.choice(["one", "rows", "rows"]),
                k=rng.choice([0, 0, 1, 20, 50, 200, 1000]), p=rng.choice([1.0, 1.0, 0.5, 0.8, 0.9, 0.95, 0.99]),
                min_p=rng.choice([0.0, 0.0, 0.01, 0.1]))


# -------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 29)
    return g


def _normal(shape, dt, g, std=1.0):
    x = torch.empty(shape, dtype=_DT[dt], device="cuda")
    x.normal_(0.0, std, generator=g)
    return x


def _blocks(d):
    return (d + 127) // 128


def _quantized(W, group):
    """The plain quantisation of W [N][d]: packed codes, scales, and the codes
    less 8 in 64 bits."""
    N, d = W.shape
    groups = (d + group - 1) // group
    x = torch.zeros(N, groups * group, dtype=torch.float64, device=W.device)
    x[:, :d] = W
    x = x.view(N, groups, group)
    scale = (x.abs().amax(dim=2) / 7).to(W.dtype)
    s = scale.double()[:, :, None]
    c = torch.where(s > 0, torch.round(x / torch.where(s > 0, s, 1.0)).clamp(-8, 7), 0.0).view(N, -1)[:, :d]
    code = torch.full((N, _blocks(d) * 128), 8, dtype=torch.int32, device=W.device)
    code[:, :d] = c.to(torch.int32) + 8
    code = code.view(N, _blocks(d), 2, 8, 8).permute(0, 1, 3, 2, 4)       # [N][block][g][s][e]
    at = torch.arange(8, device=W.device)
    word = (code.long() << (4 * (at // 2) + 16 * (at % 2))).sum(dim=4)    # below 2^32
    word = torch.where(word >= 2 ** 31, word - 2 ** 32, word).to(torch.int32).reshape(N, -1)
    return word.view(torch.uint8), scale, c


def _matrix(N, d, dt, group, g):
    """A 4-bit matrix of normal weights, in slices that bound the memory."""
    q = torch.empty(N, _blocks(d) * 64, dtype=torch.uint8, device="cuda")
    s = torch.empty(N, (d + group - 1) // group, dtype=_DT[dt], device="cuda")
    step = max(1, 40_000_000 // d)
    for n in range(0, N, step):
        rows = min(step, N - n)
        q[n:n + rows], s[n:n + rows], _ = _quantized(_normal((rows, d), dt, g, 0.02), group)
    return q, s


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = dict(case=case)
    if c["op"] == "quantize":
        W = _normal((c["N"], c["d"]), c["dt"], g, 0.02)
        st.update(W=W, q=torch.zeros(c["N"], _blocks(c["d"]) * 64, dtype=torch.uint8, device="cuda"),
                  scale=torch.zeros(c["N"], (c["d"] + c["group"] - 1) // c["group"], dtype=W.dtype, device="cuda"),
                  values=torch.zeros_like(W))
    elif c["op"] == "matvec":
        st["q"], st["scale"] = _matrix(c["N"], c["d"], c["dt"], c["group"], g)
        st.update(y=_normal((c["B"], c["d"]), c["dt"], g), out=torch.zeros(c["B"], c["N"], device="cuda"))
    elif c["op"] == "mlp":
        st["q1"], st["s1"] = _matrix(c["N"], c["d"], c["dt"], c["group"], g)
        st["q2"], st["s2"] = _matrix(c["N"], c["d"], c["dt"], c["group"], g)
        idx = torch.rand(c["B"], c["N"], device="cuda", generator=g).argsort(dim=1)[:, :c["k"]].sort(dim=1).values
        st.update(y=_normal((c["B"], c["d"]), c["dt"], g), idx=idx.int().contiguous(),
                  count=torch.full((c["B"],), c["k"], dtype=torch.int32, device="cuda"),
                  out=torch.zeros(c["B"], c["d"], device="cuda"))
    else:
        B, V = c["B"], c["V"]
        logits = _normal((B, V), c["dt"], g, 3.0)
        logits[:, torch.randint(0, V, (V // 50 + 1,), device="cuda", generator=g)] = -math.inf   # tokens ruled out
        T = None
        if c["T"] == "rows":   # requests of their own temperature, every eighth of them greedy
            T = 0.5 + torch.rand(B, device="cuda", generator=g)
            T[::8] = 0.0 if B >= 8 else 0.7
        full = dict(device="cuda")
        st.update(logits=logits, T=T, u=torch.rand(B, generator=g, **full),
                  k=torch.full((B,), c["k"], dtype=torch.int32, **full) if c["k"] else None,
                  p=torch.full((B,), c["p"], **full) if c["p"] < 1 else None,
                  min_p=torch.full((B,), c["min_p"], **full) if c["min_p"] else None,
                  token=torch.zeros(B, dtype=torch.int32, **full), prob=torch.zeros(B, **full))
    if own:
        from contextual_sparsity_decode_gb300 import binding as dv
        st["dv"] = dv
        if c["op"] == "quantize":
            st["W4"] = dv.Q4(st["q"], st["scale"], c["d"], c["group"])
        elif c["op"] == "matvec":
            st["W4"] = dv.Q4(st["q"], st["scale"], c["d"], c["group"])
            st["ws"] = dv.workspace(dv.dv_q4_matvec_workspace_size(c["B"], c["d"], c["N"]))
        elif c["op"] == "mlp":
            st["W1"], st["W2"] = (dv.Q4(st[q], st[s], c["d"], c["group"]) for q, s in (("q1", "s1"), ("q2", "s2")))
            st["ws"] = dv.workspace(dv.dv_q4_sparse_mlp_workspace_size(c["B"], c["d"], c["N"], c["k"]))
        else:
            st["ws"] = dv.workspace(dv.dv_sample_workspace_size(c["B"], c["V"]))
    return st


# --------------------------------------------------------------- plain forms

def _opened(q, scale, d, group):
    """Rows [..., pitch] of packed codes and their scales as fp32 weights."""
    w = q.view(torch.int32)
    at = torch.arange(8, dtype=torch.int32, device=q.device)
    code = (w[..., None] >> (4 * (at // 2) + 16 * (at % 2))) & 15               # [..., words][e]
    code = code.view(*w.shape[:-1], -1, 8, 2, 8).transpose(-3, -2)               # [..., block][s][g][e]
    code = code.reshape(*w.shape[:-1], -1)[..., :d]
    return (code - 8).float() * scale.float().repeat_interleave(group, dim=-1)[..., :d]


def _plain_quantize(st):
    c = st["case"]
    q, scale, code = _quantized(st["W"], c["group"])
    st["q"].copy_(q)
    st["scale"].copy_(scale)
    st["values"].copy_(code * scale.double().repeat_interleave(c["group"], dim=1)[:, :c["d"]])
    return dict(values=st["values"], scale=st["scale"])


def _plain_matvec(st):
    c = st["case"]
    st["out"].copy_(st["y"].float() @ _opened(st["q"], st["scale"], c["d"], c["group"]).T)
    return st["out"]


def _plain_mlp(st):
    c, at = st["case"], st["idx"].long()
    W1 = _opened(st["q1"][at], st["s1"][at], c["d"], c["group"])                 # [B][k][d]
    a = torch.bmm(W1, st["y"].float()[:, :, None]).clamp(min=0)
    W2 = _opened(st["q2"][at], st["s2"][at], c["d"], c["group"])
    st["out"].copy_(torch.bmm(a.transpose(1, 2), W2)[:, 0])
    return st["out"]


def _plain_sample(st):
    x = st["logits"].double()
    B, V = x.shape
    T = torch.ones(B, 1, dtype=torch.float64, device=x.device) if st["T"] is None else st["T"].double()[:, None]
    m = x.amax(dim=1, keepdim=True)
    w = torch.exp((x - m) / torch.where(T > 0, T, 1.0))
    ordered, at = torch.sort(x, dim=1, descending=True, stable=True)
    w = w.gather(1, at)
    rank = torch.arange(V, device=x.device)[None]
    keep = torch.ones_like(w, dtype=torch.bool)
    if st["k"] is not None:
        keep &= rank < st["k"][:, None]
    if st["p"] is not None:
        inside = torch.where(keep, w, 0.0)
        before = inside.cumsum(dim=1) - inside
        keep &= (before < st["p"].double()[:, None] * inside.sum(dim=1, keepdim=True)) | (rank == 0)
    if st["min_p"] is not None:
        keep &= w >= st["min_p"].double()[:, None]
    keep &= (T > 0) | (rank == 0)
    w = torch.zeros_like(w).scatter_(1, at, torch.where(keep, w, 0.0))           # by token again
    upto = w.cumsum(dim=1)
    token = (upto <= st["u"].double()[:, None] * upto[:, -1:]).sum(dim=1, keepdim=True)
    st["token"].copy_(token[:, 0])
    st["prob"].copy_((w.gather(1, token) / upto[:, -1:])[:, 0])
    return dict(token=st["token"], prob=st["prob"])


def run(state):
    st, op = state, state["case"]["op"]
    if own:
        dv = st["dv"]
        if op == "quantize":
            dv.dv_q4_quantize(st["W"], st["W4"], values=st["values"])
            return dict(values=st["values"], scale=st["scale"])
        if op == "matvec":
            dv.dv_q4_matvec(st["y"], st["W4"], st["out"], st["ws"])
            return st["out"]
        if op == "mlp":
            dv.dv_q4_sparse_mlp(st["y"], st["W1"], st["W2"], st["idx"], st["count"], st["out"], st["ws"])
            return st["out"]
        dv.dv_sample(st["logits"], st["u"], st["token"], st["ws"], temperature=st["T"], top_k=st["k"], top_p=st["p"],
                     min_p=st["min_p"], prob=st["prob"])
        return dict(token=st["token"], prob=st["prob"])
    return {"quantize": _plain_quantize, "matvec": _plain_matvec, "mlp": _plain_mlp, "sample": _plain_sample}[op](st)


# ---------------------------------------------------------------------- work

def _row_bytes(c):
    return c["d"] / 2 + (c["d"] + c["group"] - 1) // c["group"] * _ES[c["dt"]]


def work(case):
    c, es = case, _ES[case["dt"]]
    if c["op"] == "quantize":
        return dict(bytes=int(c["N"] * (2 * c["d"] * es + _row_bytes(c))), flops=3 * c["N"] * c["d"])
    if c["op"] == "matvec":
        return dict(bytes=int(c["N"] * _row_bytes(c)) + c["B"] * (c["d"] * es + 4 * c["N"]),
                    flops=2 * c["B"] * c["N"] * c["d"])
    if c["op"] == "mlp":
        # lists are drawn independently: the expected number of neurons in any of them
        union = c["N"] * (1.0 - (1.0 - c["k"] / c["N"]) ** c["B"])
        return dict(bytes=int(2 * union * _row_bytes(c)) + c["B"] * (c["d"] * (es + 4) + 4 * c["k"]),
                    flops=4 * c["B"] * c["k"] * c["d"])
    return dict(bytes=c["B"] * (c["V"] * es + 16), flops=4 * c["B"] * c["V"])


# ---------------------------------------------------- the definition in 64 bits

def _elements(q, scale, c):
    """Weights in 64 bits, element by element from the layout's definition."""
    t = torch.arange(c["d"], device=q.device)
    e, s, g = t % 8, t % 128 // 64, t % 64 // 8
    bit = 4 * (e // 2) + 16 * (e % 2)
    byte = t // 128 * 64 + 4 * (2 * g + s) + bit // 8
    return (((q[:, byte] >> (bit % 8).to(torch.uint8)) & 15).double() - 8) * scale[:, t // c["group"]].double()


def exact(case, seed):
    c, st = case, prepare(case, seed)
    if c["op"] == "quantize":
        values, scales = torch.empty_like(st["W"], dtype=torch.float64), torch.empty_like(st["scale"], dtype=torch.float64)
        for i, t in enumerate(range(0, c["d"], c["group"])):
            W = st["W"][:, t:t + c["group"]].double()
            s = (W.abs().max(dim=1).values / 7).to(st["W"].dtype).double()       # a scale is held in the matrix's type
            scales[:, i] = s
            ratio = W / s[:, None]
            values[:, t:t + c["group"]] = torch.where(s[:, None] > 0, torch.clamp(ratio.round(), -8, 7) * s[:, None], 0.0)
        return dict(values=values, scale=scales)
    if c["op"] == "matvec":
        out = torch.empty(c["B"], c["N"], dtype=torch.float64, device="cuda")
        step = max(1, 50_000_000 // c["d"])
        for n in range(0, c["N"], step):
            out[:, n:n + step] = torch.mm(st["y"].double(), _elements(st["q"][n:n + step], st["scale"][n:n + step], c).T)
        return out
    if c["op"] == "mlp":
        out = torch.zeros(c["B"], c["d"], dtype=torch.float64, device="cuda")
        step = max(1, 50_000_000 // c["d"])
        for b in range(c["B"]):
            for n in range(0, c["k"], step):
                at = st["idx"][b, n:n + step].long()
                a = torch.relu(_elements(st["q1"][at], st["s1"][at], c) @ st["y"][b].double())
                out[b] += a @ _elements(st["q2"][at], st["s2"][at], c)
        return out
    x = st["logits"].double().cpu().numpy()
    u = st["u"].double().cpu().numpy()
    row = lambda t, b, other: other if t is None else float(t[b])  # noqa: E731
    token, prob = np.zeros(c["B"], np.int32), np.zeros(c["B"])
    for b in range(c["B"]):
        T, k, p, least = row(st["T"], b, 1.0), row(st["k"], b, 0), row(st["p"], b, 1.0), row(st["min_p"], b, 0.0)
        best = int(np.argmax(x[b]))
        if T == 0:
            token[b], prob[b] = best, 1.0
            continue
        w = np.exp((x[b] - x[b, best]) / T)
        first = np.argsort(-x[b], kind="stable")
        first = first[:int(k)] if k > 0 else first
        mass = w[first]
        if p < 1:
            ends = np.searchsorted(np.cumsum(mass), p * mass.sum(), side="left")
            first = first[:ends + 1]
        first = np.sort(first[w[first] >= least])
        upto = np.cumsum(w[first])
        i = int(np.searchsorted(upto, u[b] * upto[-1], side="right"))
        token[b], prob[b] = first[i], w[first[i]] / upto[-1]
    return dict(token=token, prob=prob)
