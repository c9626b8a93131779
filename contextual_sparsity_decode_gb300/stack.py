"""Decoder stack driver: one decoded token through L sparse layers, with the
next layer's heads and neurons predicted on a side CUDA stream from the
current layer's attention input ("用Deja Vu来提高 LLM 的推理速度" §3.1, parallel
sparsity prediction; Deja Vu reading notes, "Reducing Overhead with
Asynchronous Execution").

Per layer l (main stream):
    y_a = LN(r)                      dv_layernorm
    (layer 0 only) S_A, S_M = predict(y_a)          dv_predict, synchronous
    wait for layer l's look-ahead sets (event)
    record "y_a of layer l ready"; side stream: dv_lookahead(y_a, P^{l+1})
    r += MHA_{S_A}(y_a)              dv_sparse_attn (append, repair, attend)
    y_m = LN(r);  r += MLP_{S_M}(y_m)    dv_layernorm, dv_sparse_mlp
The whole token (both streams) is captured once into a CUDA graph and
replayed.  This module only orders calls; every step of a token runs in
libdv's kernels.

Several candidates per sequence: ``verify_tree`` runs a drafted token tree
through the layers (dv_tree_attn over the cache), ``accept`` keeps a path of it
(dv_kv_compact), and ``reorder`` lets beams continue others (dv_kv_reorder).

4 bits: a layer's MLP may be held in 4 bits (dv_q4_sparse_mlp in the place of
dv_sparse_mlp), and ``sample`` draws the next tokens through a 4-bit output head
(dv_layernorm, dv_q4_matvec, dv_sample).
"""

from __future__ import annotations

from typing import Dict, List, Optional

import torch

from . import binding as dv


def quantize_mlp(layers: List[Dict[str, torch.Tensor]], group: int = 128) -> List[dict]:
    """The same layers with their MLP in 4 bits (W1q and W2q in the place of
    W1n and W2n; groups of 64 or 128 weights share a scale): a quarter of the
    memory.  Steps over few neurons of one sequence are slower than in 16 bits
    (40 layers of 5120, 5 % of 20480 neurons, groups of 128: 49 us a layer, 41 in
    f16; 8 sequences 158 and 161)."""
    out = []
    for W in layers:
        W = dict(W)
        if "W1n" in W:
            W["W1q"], W["W2q"] = (dv.Q4.of(W.pop(k), group) for k in ("W1n", "W2n"))
        out.append(W)
    return out


class SparseDecoder:
    """Device state of an L-layer sparse decoder for a batch of B sequences.

    layers: per layer a dict of weight tensors in the library layouts
            (Wqkv, Wo, W1n, W2n, PA1t, PA2t, PM1t, PM2t), all of one dtype.
            A layer may hold its MLP in 4 bits, as W1q and W2q (binding.Q4)
            in the place of W1n and W2n: see ``quantize_mlp``.
    trace:  keep a copy of the residual stream before layer 0 (r_in0) and
            after every block of every layer (r_mid[l] after the attention,
            r_out[l] after the MLP), so that each block can be checked on its
            own inputs (plain device copies between the calls).
    """

    def __init__(self, layers: List[Dict[str, torch.Tensor]], B: int, n_max: int,
                 k_heads: int, k_neurons: int, scale: float, eps: float = 1e-5,
                 trace: bool = False):
        W0 = layers[0]
        self.layers = layers
        self.L = len(layers)
        self.h, _, self.d_h, self.d = W0["Wqkv"].shape
        self.N, self.r = W0["PM2t"].shape
        self.B, self.n_max = B, n_max
        self.k_heads, self.k_neurons = k_heads, k_neurons
        self.scale, self.eps = float(scale), float(eps)
        self.dtype = W0["Wqkv"].dtype
        dev = W0["Wqkv"].device
        for W in layers:
            if "W1q" in W and any((q.N, q.d, q.dtype) != (self.N, self.d, self.dtype) for q in (W["W1q"], W["W2q"])):
                raise ValueError(f"4-bit matrices of another shape or type than [{self.N}][{self.d}] of {self.dtype}")
        self.device = dev
        i32 = dict(dtype=torch.int32, device=dev)
        B, d = self.B, self.d
        self.kv = [dv.KV.empty(B, self.h, n_max, self.d_h, d, self.dtype, dev) for _ in layers]
        self.head_idx = [torch.zeros(B, k_heads, **i32) for _ in layers]
        self.head_cnt = [torch.zeros(B, **i32) for _ in layers]
        self.neur_idx = [torch.zeros(B, k_neurons, **i32) for _ in layers]
        self.neur_cnt = [torch.zeros(B, **i32) for _ in layers]
        self.y_a = [torch.zeros(B, d, dtype=self.dtype, device=dev) for _ in layers]
        self.y_m = [torch.zeros(B, d, dtype=self.dtype, device=dev) for _ in layers]
        self.r_stream = torch.zeros(B, d, dtype=torch.float32, device=dev)   # residual
        self.trace = bool(trace)
        if self.trace:
            f32 = dict(dtype=torch.float32, device=dev)
            self.r_in0 = torch.zeros(B, d, **f32)
            self.r_mid = [torch.zeros(B, d, **f32) for _ in layers]
            self.r_out = [torch.zeros(B, d, **f32) for _ in layers]
        self.pos = torch.zeros(B, **i32)
        self.ws_pred_main = dv.workspace(dv.dv_predict_workspace_size(B, 2, self.r, self.N), dev)
        self.ws_pred_side = dv.workspace(dv.dv_predict_workspace_size(B, 2, self.r, self.N), dev)
        self.ws_attn = dv.workspace(
            dv.dv_sparse_attn_workspace_size(B, d, self.h, self.d_h, k_heads, n_max), dev)
        self.ws_mlp, self.ws_mlp_q4 = self._mlp_workspaces(B, k_neurons)
        self.kv_layers = dv.KVLayers(self.kv)
        self.ws_move = dv.workspace(256, dev)
        self._tree: Dict[int, dict] = {}    # buffers of verify_tree by the nodes they hold
        self.head: Optional[dv.Q4] = None   # output head (set_head)
        self.side = torch.cuda.Stream(device=dev)
        self.ev_y = [dv.make_event() for _ in layers]
        self.ev_pred = [dv.make_event() for _ in layers]
        torch.cuda.synchronize(dev)
        self.graph: Optional[torch.cuda.CUDAGraph] = None
        # optional timing of one kernel family inside the step (events recorded
        # around every call of it on the main stream)
        self.timed: Optional[str] = None
        self.t_ev: List[torch.cuda.Event] = []

    def set_keep(self, k_heads: int, k_neurons: int):
        """Change the number of heads and neurons kept per layer (new index
        lists and block workspaces; the KV caches are kept).  Re-capture
        the graph afterwards."""
        dev, B = self.device, self.B
        i32 = dict(dtype=torch.int32, device=dev)
        self.k_heads, self.k_neurons = k_heads, k_neurons
        self.head_idx = [torch.zeros(B, k_heads, **i32) for _ in self.layers]
        self.head_cnt = [torch.zeros(B, **i32) for _ in self.layers]
        self.neur_idx = [torch.zeros(B, k_neurons, **i32) for _ in self.layers]
        self.neur_cnt = [torch.zeros(B, **i32) for _ in self.layers]
        self.ws_attn = dv.workspace(
            dv.dv_sparse_attn_workspace_size(B, self.d, self.h, self.d_h, k_heads, self.n_max), dev)
        self.ws_mlp, self.ws_mlp_q4 = self._mlp_workspaces(B, k_neurons)
        self._tree = {}
        self.graph = None

    # ------------------------------------------------------------------ pieces
    def _mlp_workspaces(self, rows: int, k_neurons: int):
        """For the layers whose MLP is in 16 (or 32) bits and for those in 4
        (None where there are none): a workspace keeps state of its kind of
        call, so the two do not share one."""
        kinds = {"W1q" in W for W in self.layers}
        size = (self.d, self.N, k_neurons)
        return (dv.workspace(dv.dv_sparse_mlp_workspace_size(rows, *size), self.device) if False in kinds else None,
                dv.workspace(dv.dv_q4_sparse_mlp_workspace_size(rows, *size), self.device) if True in kinds else None)

    def _mlp(self, l: int, y, idx, cnt, out, ws, ws_q4):
        """out += the sparse MLP of layer l."""
        W = self.layers[l]
        if "W1q" in W:
            dv.dv_q4_sparse_mlp(y, W["W1q"], W["W2q"], idx, cnt, out, ws_q4, accumulate=True)
        else:
            dv.dv_sparse_mlp(y, W["W1n"], W["W2n"], idx, cnt, out, ws, accumulate=True)

    def predictors(self, l: int):
        W = self.layers[l]
        return [dv.Predictor(W["PA1t"], W["PA2t"], self.head_idx[l], self.head_cnt[l],
                             dv.DV_TOPK, self.k_heads),
                dv.Predictor(W["PM1t"], W["PM2t"], self.neur_idx[l], self.neur_cnt[l],
                             dv.DV_TOPK, self.k_neurons)]

    def prefill(self, X_prompt: List[torch.Tensor], n_prompt: int):
        """Synthetic prompt: X[b][0:n_prompt] = X_prompt[l] for every layer and
        K/V of every head computed from it (dv_kv_repair with all heads)."""
        all_heads = torch.arange(self.h, dtype=torch.int32, device=self.device).repeat(self.B, 1)
        cnt = torch.full((self.B,), self.h, dtype=torch.int32, device=self.device)
        pos = torch.full((self.B,), n_prompt, dtype=torch.int32, device=self.device)
        ws = dv.workspace(dv.dv_sparse_attn_workspace_size(self.B, self.d, self.h, self.d_h, self.h,
                                                           self.n_max), self.device)
        for l in range(self.L):
            kv = self.kv[l]
            kv.valid.zero_()
            kv.X[:, :n_prompt].copy_(X_prompt[l][:, :n_prompt])
            dv.dv_kv_repair(kv, self.layers[l]["Wqkv"], pos, all_heads, cnt, ws)
        self.pos.fill_(n_prompt)
        st, info = dv.dv_check(ws)
        if st != 0:
            raise dv.DvError(st, "prefill", f"info={info}")

    def _dense_ops(self):
        """One prompt position through every layer with all heads and all
        neurons selected (no predictor), on the current stream."""
        if self.trace:
            self.r_in0.copy_(self.r_stream)
        for l in range(self.L):
            W = self.layers[l]
            dv.dv_layernorm(self.r_stream, self.y_a[l], self.eps)
            dv.dv_sparse_attn(self.y_a[l], W["Wqkv"], W["Wo"], self.kv[l], self.pos,
                              self.head_idx[l], self.head_cnt[l], self.scale, self.r_stream,
                              self.ws_attn, accumulate=True)
            if self.trace:
                self.r_mid[l].copy_(self.r_stream)
            dv.dv_layernorm(self.r_stream, self.y_m[l], self.eps)
            self._mlp(l, self.y_m[l], self.neur_idx[l], self.neur_cnt[l], self.r_stream, self.ws_mlp,
                      self.ws_mlp_q4)
            if self.trace:
                self.r_out[l].copy_(self.r_stream)

    def prefill_dense(self, E: torch.Tensor, n_prompt: int, on_position=None):
        """Dense causal prompt pass (Deja Vu reading notes, "Typical LLM
        procedure": the prompt runs through every layer, which builds each
        layer's KV cache; generation then goes token by token).  Positions
        0..n_prompt-1 in order, each through every layer with all heads and
        all neurons selected -- the decode step's own kernels with S = all,
        one CUDA graph replayed per position -- so position t attends over
        positions 0..t (causal attention) and every layer's X, K, V and valid
        flags below n_prompt are the model's own.  E [B][n_prompt][d] (fp32)
        is the residual stream entering layer 0.  Afterwards the decoder
        continues at n_prompt with its keep counts.  ``on_position(t)`` runs
        after position t (the tests read the traced activations there)."""
        keep = (self.k_heads, self.k_neurons)
        dev, B = self.device, self.B
        if n_prompt > self.n_max:
            raise ValueError("prompt longer than the cache")
        self.set_keep(self.h, self.N)
        heads = torch.arange(self.h, dtype=torch.int32, device=dev).repeat(B, 1)
        neurons = torch.arange(self.N, dtype=torch.int32, device=dev).repeat(B, 1)
        for l in range(self.L):
            self.kv[l].valid.zero_()
            self.head_idx[l].copy_(heads)
            self.head_cnt[l].fill_(self.h)
            self.neur_idx[l].copy_(neurons)
            self.neur_cnt[l].fill_(self.N)
        self.pos.zero_()
        graph = torch.cuda.CUDAGraph()
        s = torch.cuda.Stream(device=dev)
        s.wait_stream(torch.cuda.current_stream())
        # every attention / MLP call follows the layernorm that produces its
        # input and no predictor runs: launch overlap holds for all of them
        prev = dv.dv_set_launch_overlap(1)
        try:
            with torch.cuda.stream(s):
                with torch.cuda.graph(graph, stream=s):
                    self._dense_ops()
                    dv.dv_positions_advance(self.pos, 0, self.n_max)
        finally:
            dv.dv_set_launch_overlap(prev)
        torch.cuda.current_stream().wait_stream(s)
        for t in range(n_prompt):
            self.r_stream.copy_(E[:, t])
            graph.replay()
            if on_position is not None:
                on_position(t)
        self.check()
        self.set_keep(*keep)

    def _time(self, kind: str, stream=None):
        """Record a timing event (kept in self.t_ev) when timing ``kind``.
        Events are 'external' so that they are real event records inside a
        captured graph."""
        if self.timed != kind:
            return
        try:
            ev = torch.cuda.Event(enable_timing=True, external=True)
        except TypeError:  # older torch: events still work outside graphs
            ev = torch.cuda.Event(enable_timing=True)
        ev.record(stream if stream is not None else torch.cuda.current_stream())
        self.t_ev.append(ev)

    def step_ops(self):
        """Enqueue one token on the current stream (+ the side stream)."""
        # Every attention / MLP call here directly follows the layernorm that
        # produces its input, except layer 0's attention (after its predictor
        # on the same stream): launch overlap is on for all the others.
        prev = dv.dv_set_launch_overlap(1)
        try:
            self._step_ops()
        finally:
            dv.dv_set_launch_overlap(prev)

    def _step_ops(self):
        main = torch.cuda.current_stream()
        if self.trace:
            self.r_in0.copy_(self.r_stream)
        for l in range(self.L):
            W = self.layers[l]
            self._time("ln")
            dv.dv_layernorm(self.r_stream, self.y_a[l], self.eps)
            self._time("ln")
            if l == 0:
                self._time("predict")
                dv.dv_predict(self.y_a[0], self.predictors(0), self.ws_pred_main)
                self._time("predict")
            else:
                main.wait_event(self.ev_pred[l])
            if l + 1 < self.L:
                self.ev_y[l].record(main)
                if self.timed == "predict":
                    # dv_lookahead spelled out so the timing events bracket
                    # only the predictor kernels on the side stream
                    self.side.wait_event(self.ev_y[l])
                    self._time("predict", self.side)
                    dv.dv_predict(self.y_a[l], self.predictors(l + 1), self.ws_pred_side,
                                  stream=self.side)
                    self._time("predict", self.side)
                    self.ev_pred[l + 1].record(self.side)
                else:
                    dv.dv_lookahead(self.y_a[l], self.predictors(l + 1), self.ws_pred_side,
                                    self.ev_y[l], self.side, self.ev_pred[l + 1])
            self._time("attn")
            if l == 0:
                dv.dv_set_launch_overlap(0)  # the predictor just wrote this call's head list
            dv.dv_sparse_attn(self.y_a[l], W["Wqkv"], W["Wo"], self.kv[l], self.pos,
                              self.head_idx[l], self.head_cnt[l], self.scale, self.r_stream,
                              self.ws_attn, accumulate=True)
            dv.dv_set_launch_overlap(1)
            self._time("attn")
            if self.trace:
                self.r_mid[l].copy_(self.r_stream)
            self._time("ln")
            dv.dv_layernorm(self.r_stream, self.y_m[l], self.eps)
            self._time("ln")
            self._time("mlp")
            self._mlp(l, self.y_m[l], self.neur_idx[l], self.neur_cnt[l], self.r_stream, self.ws_mlp,
                      self.ws_mlp_q4)
            self._time("mlp")
            if self.trace:
                self.r_out[l].copy_(self.r_stream)

    def capture(self, advance: Optional[tuple] = None, host_io: Optional[tuple] = None):
        """Capture one token (optionally followed by pos advance (lo, hi))
        into a CUDA graph.  host_io = (h_in, h_out), pinned host tensors of
        the residual's shape: the graph then starts with the copy of h_in
        into the residual stream and ends with the copy of the result into
        h_out, so a host-driven loop costs one graph launch per token."""
        self.graph = torch.cuda.CUDAGraph()
        s = torch.cuda.Stream(device=self.device)
        s.wait_stream(torch.cuda.current_stream())
        if host_io is not None:
            for t in host_io:
                if t.device.type != "cpu" or not t.is_pinned() or t.shape != self.r_stream.shape \
                        or t.dtype != self.r_stream.dtype:
                    raise ValueError("host_io: pinned host fp32 tensors of the residual's shape")
        with torch.cuda.stream(s):
            with torch.cuda.graph(self.graph, stream=s):
                if host_io is not None:
                    self.r_stream.copy_(host_io[0], non_blocking=True)
                self.step_ops()
                if advance is not None:
                    dv.dv_positions_advance(self.pos, advance[0], advance[1])
                if host_io is not None:
                    host_io[1].copy_(self.r_stream, non_blocking=True)
        torch.cuda.current_stream().wait_stream(s)

    def replay(self):
        self.graph.replay()

    # ------------------------------------------------------------------ the next token
    def set_head(self, head: dv.Q4):
        """The output head of ``sample``: a 4-bit matrix [V][d] (its row v
        scores token v), and the buffers that go with it (a graph that has
        captured ``sample`` is captured again after another head)."""
        if head.d != self.d or head.dtype != self.dtype or head.q.device != self.device:
            raise ValueError(f"a 4-bit matrix with rows of {self.d} of {self.dtype} on {self.device} is wanted")
        dev, B = self.device, self.B
        self.head = head
        self.y_head = torch.zeros(B, self.d, dtype=self.dtype, device=dev)
        self.logits = torch.zeros(B, head.N, dtype=torch.float32, device=dev)
        self.token = torch.zeros(B, dtype=torch.int32, device=dev)
        self.prob = torch.zeros(B, dtype=torch.float32, device=dev)
        self.ws_head = dv.workspace(dv.dv_q4_matvec_workspace_size(B, self.d, head.N), dev)
        self.ws_sample = dv.workspace(dv.dv_sample_workspace_size(B, head.N), dev)

    def sample(self, u, temperature=None, top_k=None, top_p=None, min_p=None):
        """The next token of each sequence and its probability (``token`` and
        ``prob``, [B]), drawn with the numbers u from the head's scores of the
        residual stream that a step leaves: layer norm, ``logits``, dv_sample
        (whose parameters these are).  Can be captured."""
        if self.head is None:
            raise ValueError("sample: set_head first")
        dv.dv_layernorm(self.r_stream, self.y_head, self.eps)
        dv.dv_q4_matvec(self.y_head, self.head, self.logits, self.ws_head)
        dv.dv_sample(self.logits, u, self.token, self.ws_sample, temperature, top_k, top_p, min_p, prob=self.prob)
        return self.token, self.prob

    # ------------------------------------------- several candidates per sequence
    def _tree_buffers(self, T: int) -> dict:
        """Buffers and workspaces of verify_tree for trees of T nodes: the
        smallest set made so far that holds them, or a new one for the next
        power of two (all sets together hold less than twice the largest).  A
        set stays until set_keep: captured graphs hold its addresses."""
        size = min((n for n in self._tree if n >= T), default=0)
        if size:
            return self._tree[size]
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError(f"verify_tree of {T} nodes: run it once before it is captured (its buffers are made then)")
        size = 1 << (T - 1).bit_length()
        dev, B, d, h, d_h = self.device, self.B, self.d, self.h, self.d_h
        rows = B * size
        chunk = min(rows, 32)   # rows of one dv_predict / dv_sparse_mlp call
        i32 = dict(dtype=torch.int32, device=dev)
        t = dict(r=torch.zeros(rows, d, dtype=torch.float32, device=dev),
                 y=torch.zeros(rows, d, dtype=self.dtype, device=dev),
                 y2=torch.zeros(rows, d, dtype=self.dtype, device=dev),
                 y_mlp=torch.zeros(rows, d, dtype=self.dtype, device=dev),
                 y_root=torch.zeros(B, d, dtype=self.dtype, device=dev),
                 out=torch.zeros(rows, h * d_h, dtype=self.dtype, device=dev),
                 head_idx=torch.zeros(B, self.k_heads, **i32), head_cnt=torch.zeros(B, **i32),
                 neur_idx=torch.zeros(chunk, self.k_neurons, **i32), neur_cnt=torch.zeros(chunk, **i32),
                 node=torch.arange(size, **i32)[None], row=torch.arange(B, device=dev)[:, None],
                 head=(torch.arange(B * h, device=dev) * self.n_max).view(B, 1, h),
                 ws_pred=dv.workspace(dv.dv_predict_workspace_size(max(chunk, min(B, 32)), 1, self.r, self.N), dev),
                 ws_tree=dv.workspace(dv.dv_tree_attn_workspace_size(B, size, h, 1, d_h), dev))
        t["ws_mlp"], t["ws_mlp_q4"] = self._mlp_workspaces(chunk, self.k_neurons)
        self._tree[size] = t
        return t

    def verify_tree(self, E: torch.Tensor, mask: Optional[torch.Tensor] = None,
                    nodes: Optional[torch.Tensor] = None) -> torch.Tensor:
        """The residual streams [B][T][d] (fp32) that T drafted tokens per
        sequence leave the last layer with, all nodes in one pass.

        E [B][T][d] (fp32): the streams entering layer 0; mask and nodes as in
        dv_tree_attn (None: a linear draft, full trees).  pos + nodes may be
        n_max at most: a tree behind that changes no row of the cache, and
        ``check`` reports it.  The live nodes' rows are written to the cache
        behind pos, which does not move: ``accept`` keeps a path of them.  The
        pass can be captured once a tree of its size has run (capture it again
        after set_keep or prefill_dense, which make new buffers).  A
        tree's nodes share one set of heads per layer, predicted from node 0;
        neurons are predicted node by node, both from the same inputs as in a
        decode step (layer 0 from its own attention input, layer l from layer
        l - 1's).  The query and output projections are plain library GEMMs
        over every head.  q and the attention's result are rounded to the
        storage type, which dv_tree_attn takes and gives (a decode step keeps
        them in fp32); sums and streams are fp32."""
        B, T, d = E.shape
        if B != self.B or T < 1 or d != self.d or E.dtype != torch.float32:
            raise ValueError(f"E: fp32 [{self.B}][T][{self.d}], T >= 1")
        # before anything is written: the calls below would refuse these too late
        if nodes is not None and (nodes.dtype != torch.int32 or nodes.shape != (B,) or not nodes.is_contiguous()
                                  or nodes.device != self.pos.device):
            raise ValueError(f"nodes: contiguous int32 [{B}] on {self.pos.device}")
        if mask is not None and (mask.dtype not in (torch.bool, torch.uint8) or not mask.is_contiguous()
                                 or mask.shape not in ((T, T), (B, T, T)) or mask.device != self.pos.device):
            raise ValueError(f"mask: contiguous bool or uint8 [T][T] or [{B}][T][T] on {self.pos.device}")
        # the predictors here write their lists right before the calls that read them
        prev = dv.dv_set_launch_overlap(0)
        try:
            return self._verify_ops(E, mask, nodes)
        finally:
            dv.dv_set_launch_overlap(prev)

    def _verify_ops(self, E, mask, nodes):
        B, T, d = E.shape
        t = self._tree_buffers(T)
        h, d_h, rows, chunk = self.h, self.d_h, B * T, min(B * T, 32)
        r, y, before, y_mlp, out = (t[k][:rows] for k in ("r", "y", "y2", "y_mlp", "out"))
        r.copy_(E.reshape(rows, d))
        # Rows of the cache that the nodes take: those of live nodes alone, and
        # none of a tree that does not fit (the calls below report it).  A node
        # without a row of its own repeats its tree's last live one, or, where
        # there is none, writes back what slot 0 holds: every index may be
        # written, and equal ones get equal values.
        live = torch.full_like(self.pos, T) if nodes is None else nodes.clamp(0, T)
        inside = (self.pos >= 0) & (self.pos <= self.n_max)
        end = self.pos + live.where(inside, 0)
        fits = (inside & (self.pos <= self.n_max - live) & (live > 0))[:, None]
        node = torch.minimum(t["node"][:, :T], live[:, None] - 1).clamp_(min=0)
        slot = (self.pos[:, None] + node).where(fits, 0)
        x_row = (t["row"] * self.n_max + slot).view(-1)
        y_row = (t["row"] * T + node).view(-1)
        x_new = fits.expand(B, T).reshape(rows, 1)
        flag = (t["head"] + slot[:, :, None]).view(-1)
        bound = (~fits).to(torch.uint8).mul_(255)[:, :, None].expand(B, T, h).reshape(-1)   # min: cleared, or as it is
        wide = {} if self.dtype == torch.float32 else dict(out_dtype=torch.float32)
        for l in range(self.L):
            W, kv = self.layers[l], self.kv[l]
            dv.dv_layernorm(r, y, self.eps)
            src = before if l else y          # what the predictors read
            t["y_root"].copy_(src.view(B, T, d)[:, 0])
            for b in range(0, B, 32):
                e = min(b + 32, B)
                dv.dv_predict(t["y_root"][b:e], [dv.Predictor(W["PA1t"], W["PA2t"], t["head_idx"][b:e],
                                                             t["head_cnt"][b:e], dv.DV_TOPK, self.k_heads)],
                              t["ws_pred"])
            X = kv.X.view(B * self.n_max, d)
            X.index_copy_(0, x_row, y.index_select(0, y_row).where(x_new, X.index_select(0, x_row)))
            kv.valid.view(-1).scatter_reduce_(0, flag, bound, "amin")
            dv.dv_kv_repair(kv, W["Wqkv"], end, t["head_idx"], t["head_cnt"], self.ws_attn)
            q = torch.bmm(y.expand(h, rows, d), W["Wqkv"][:, 0].transpose(1, 2))         # [h][B T][d_h]
            dv.dv_tree_attn(q.permute(1, 0, 2).contiguous().view(B, T, h, d_h), kv, self.pos, self.scale,
                            out.view(B, T, h, d_h), t["ws_tree"], mask=mask, nodes=nodes, head_idx=t["head_idx"],
                            head_count=t["head_cnt"])
            r += torch.mm(out, W["Wo"].view(h * d_h, d), **wide)
            dv.dv_layernorm(r, y_mlp, self.eps)
            for i in range(0, rows, chunk):
                e = min(i + chunk, rows)
                idx, cnt = t["neur_idx"][:e - i], t["neur_cnt"][:e - i]
                dv.dv_predict(src[i:e], [dv.Predictor(W["PM1t"], W["PM2t"], idx, cnt, dv.DV_TOPK, self.k_neurons)],
                              t["ws_pred"])
                self._mlp(l, y_mlp[i:e], idx, cnt, r[i:e], t["ws_mlp"], t["ws_mlp_q4"])
            y, before = before, y
        return r.view(B, T, d).clone()

    def accept(self, idx: torch.Tensor, count: torch.Tensor):
        """Keep nodes idx[b][0 .. count[b]) of the last verified tree of each
        sequence (int32, ascending: a path of the tree) and advance pos."""
        dv.dv_kv_compact(self.kv_layers, self.pos, idx, count, self.ws_move, new_pos=self.pos)

    def reorder(self, parent: torch.Tensor, start: Optional[torch.Tensor] = None):
        """Let beam w of sequence s (cache row s * width + w) continue beam
        parent[s][w] (int32 [n_seq][width], n_seq * width = B; start as in
        dv_kv_reorder).  The beams of a sequence have the same length."""
        dv.dv_kv_reorder(self.kv_layers, self.pos, parent, self.ws_move, start=start)

    def check(self):
        """Raise the first error that any call has recorded since the last check
        (all workspaces are read and cleared)."""
        used = [self.ws_pred_main, self.ws_pred_side, self.ws_attn, self.ws_mlp, self.ws_mlp_q4, self.ws_move]
        if self.head is not None:
            used += [self.ws_head, self.ws_sample]
        for t in self._tree.values():
            used += [t[k] for k in ("ws_pred", "ws_mlp", "ws_mlp_q4", "ws_tree")]
        found = [dv.dv_check(ws) for ws in used if ws is not None]
        for st, info in found:
            if st != 0:
                raise dv.DvError(st, "decode step", f"info={info}")
