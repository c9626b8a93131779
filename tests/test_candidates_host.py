"""Host-side checks of the operators for several candidates per sequence (no
GPU needed): workspace queries and the refusal of bad arguments before
anything is launched."""

import ctypes

import pytest
import torch

from contextual_sparsity_decode_gb300 import binding as dv

FAKE = 1 << 20  # never dereferenced: validation fails first
INVALID, DTYPE, WORKSPACE, UNSUPPORTED = 1, 2, 3, 7


def _vp(x):
    return None if x is None else ctypes.c_void_p(x)


def _tree(q=FAKE, B=2, T=5, h=4, g=1, d_h=64, K=FAKE, V=FAKE, n_max=64, pos=FAKE, nodes=FAKE, mask=FAKE, idx=FAKE,
          cap=4, count=FAKE, dt=dv.DV_F16, out=FAKE, ws=FAKE, ws_bytes=0, scale=0.125):
    kv = dv.dv_kv(K, V, None, None, n_max)
    return dv.lib().dv_tree_attn(_vp(q), B, T, h, g, d_h, ctypes.byref(kv), _vp(pos), _vp(nodes), _vp(mask), 1,
                                 _vp(idx), cap, _vp(count), scale, dt, _vp(out), _vp(ws), ws_bytes, _vp(0))


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(K=None), dict(V=None), dict(pos=None), dict(out=None), dict(q=FAKE + 8), dict(K=FAKE + 8),
    dict(out=FAKE + 4), dict(pos=FAKE + 2), dict(nodes=FAKE + 1), dict(idx=FAKE + 2), dict(idx=None),
    dict(count=None), dict(cap=0), dict(cap=5), dict(B=0), dict(B=513), dict(T=0), dict(T=1025), dict(h=0),
    dict(h=1025), dict(g=0), dict(g=65), dict(n_max=0), dict(n_max=40), dict(n_max=1048592),
    dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
])
def test_tree_attention_refuses_bad_arguments(kw):
    assert _tree(ws_bytes=1 << 30, **kw) == INVALID


def test_tree_attention_refuses_types_shapes_and_small_workspaces():
    assert _tree(dt=7, ws_bytes=1 << 30) == DTYPE
    assert _tree(d_h=96, ws_bytes=1 << 30) == UNSUPPORTED
    need = dv.dv_tree_attn_workspace_size(2, 5, 4, 1, 64)
    assert _tree(ws_bytes=need - 1) == WORKSPACE
    assert _tree(ws=None, ws_bytes=need) == WORKSPACE
    assert _tree(ws=FAKE + 8, ws_bytes=need) == WORKSPACE


def test_workspace_queries():
    a = dv.dv_tree_attn_workspace_size(1, 8, 32, 1, 64)
    b = dv.dv_tree_attn_workspace_size(1, 64, 32, 1, 128)
    assert 0 < a < b
    # a unit holds at most 128 query rows: longer trees and larger batches need no more
    assert dv.dv_tree_attn_workspace_size(64, 1000, 32, 1, 128) == dv.dv_tree_attn_workspace_size(1, 128, 8, 1, 128)
    for bad in ((0, 8, 32, 1, 64), (1, 0, 32, 1, 64), (1, 8, 0, 1, 64), (1, 8, 32, 65, 64)):
        with pytest.raises(dv.DvError) as e:
            dv.dv_tree_attn_workspace_size(*bad)
        assert e.value.status == INVALID
    with pytest.raises(dv.DvError) as e:
        dv.dv_tree_attn_workspace_size(1, 8, 32, 1, 80)
    assert e.value.status == UNSUPPORTED
    assert 0 < dv.dv_beam_select_workspace_size(1, 4, 32000, 4) < dv.dv_beam_select_workspace_size(8, 4, 32000, 4)
    for bad in ((0, 4, 100, 4), (1, 33, 100, 4), (1, 4, 0, 4), (1, 4, 100, 0), (1, 4, 100, 65), (1, 2, 3, 7),
                (1, 1, 4194305, 1)):
        with pytest.raises(dv.DvError) as e:
            dv.dv_beam_select_workspace_size(*bad)
        assert e.value.status == INVALID


def _kvs(n=2, n_max=(32, 32), K=FAKE):
    return (dv.dv_kv * n)(*[dv.dv_kv(K, FAKE, FAKE, FAKE, n_max[l]) for l in range(n)])


def _compact(kvs=None, n=2, B=2, d=128, h=2, d_h=64, pos=FAKE, idx=FAKE, cap=3, count=FAKE, dt=dv.DV_BF16,
             new_pos=FAKE, ws=FAKE, ws_bytes=256):
    return dv.lib().dv_kv_compact(kvs if kvs is not None else _kvs(), n, B, d, h, d_h, _vp(pos), _vp(idx), cap,
                                  _vp(count), dt, _vp(new_pos), _vp(ws), ws_bytes, _vp(0))


@pytest.mark.parametrize("kw,status", [
    (dict(n=0), INVALID), (dict(n=1025), INVALID), (dict(B=0), INVALID), (dict(B=65536), INVALID),
    (dict(d=100), INVALID), (dict(d_h=60), INVALID), (dict(h=0), INVALID), (dict(pos=None), INVALID),
    (dict(idx=None), INVALID), (dict(count=None), INVALID), (dict(cap=0), INVALID), (dict(new_pos=FAKE + 1), INVALID),
    (dict(dt=9), DTYPE), (dict(ws_bytes=255), WORKSPACE), (dict(ws=None), WORKSPACE),
    (dict(kvs=_kvs(2, (32, 48))), INVALID), (dict(kvs=_kvs(2, (0, 0))), INVALID), (dict(kvs=_kvs(K=FAKE + 8)), INVALID),
    (dict(kvs=_kvs(K=None)), INVALID),
])
def test_compact_refuses_bad_arguments(kw, status):
    assert _compact(**kw) == status


def _reorder(kvs=None, n=2, S=2, W=4, d=128, h=2, d_h=64, pos=FAKE, start=FAKE, parent=FAKE, dt=dv.DV_F32, ws=FAKE,
             ws_bytes=256):
    return dv.lib().dv_kv_reorder(kvs if kvs is not None else _kvs(), n, S, W, d, h, d_h, _vp(pos), _vp(start),
                                  _vp(parent), dt, _vp(ws), ws_bytes, _vp(0))


@pytest.mark.parametrize("kw,status", [
    (dict(n=0), INVALID), (dict(S=0), INVALID), (dict(S=1024), INVALID), (dict(W=0), INVALID), (dict(W=33), INVALID),
    (dict(d=102), INVALID), (dict(d_h=6), INVALID), (dict(pos=None), INVALID), (dict(parent=None), INVALID),
    (dict(start=FAKE + 2), INVALID), (dict(dt=-1), DTYPE), (dict(ws_bytes=0), WORKSPACE),
    (dict(kvs=_kvs(2, (32, 16))), INVALID),
])
def test_reorder_refuses_bad_arguments(kw, status):
    assert _reorder(**kw) == status


def _beam(logits=FAKE, S=2, W=4, V=1000, ld=1000, dt=dv.DV_F16, cum=FAKE, done=FAKE, end=2, K=8, score=FAKE,
          token=FAKE, beam=FAKE, ws=FAKE, ws_bytes=1 << 30):
    return dv.lib().dv_beam_select(_vp(logits), S, W, V, ld, dt, _vp(cum), _vp(done), end, K, _vp(score), _vp(token),
                                   _vp(beam), _vp(ws), ws_bytes, _vp(0))


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), INVALID), (dict(cum=None), INVALID), (dict(score=None), INVALID), (dict(token=None), INVALID),
    (dict(beam=None), INVALID), (dict(logits=FAKE + 1), INVALID), (dict(logits=FAKE + 2, dt=dv.DV_F32), INVALID),
    (dict(cum=FAKE + 2), INVALID), (dict(S=0), INVALID), (dict(S=65536), INVALID), (dict(W=0), INVALID),
    (dict(W=33), INVALID), (dict(V=0), INVALID), (dict(ld=999), INVALID), (dict(K=0), INVALID), (dict(K=65), INVALID),
    (dict(W=1, V=5, K=6), INVALID), (dict(end=-1), INVALID), (dict(end=1000), INVALID), (dict(dt=3), DTYPE),
    (dict(ws_bytes=256), WORKSPACE), (dict(ws=FAKE + 4), WORKSPACE),
])
def test_beam_select_refuses_bad_arguments(kw, status):
    assert _beam(**kw) == status


def test_binding_refuses_shapes_types_and_layouts():
    """Tensors that the kernels would misread are refused before the call (the
    checks look at shapes only: the tensors here are on the CPU)."""
    B, T, h, d_h, n_max = 2, 3, 4, 64, 32
    kv = dv.KV(*(torch.zeros(B, h, n_max, d_h, dtype=torch.float16) for _ in range(2)), None, None)
    pos, ws = torch.zeros(B, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8)
    q = torch.zeros(B, T, h, d_h, dtype=torch.float16)

    def refused(**kw):
        a = dict(q=q, kv=kv, pos=pos, scale=1.0, out=q.clone(), ws=ws)
        a.update(kw)
        with pytest.raises(dv.DvError) as e:
            dv.dv_tree_attn(**a)
        assert e.value.status == INVALID

    refused(q=q.bfloat16())
    refused(q=torch.zeros(B, h, T, d_h, dtype=torch.float16).transpose(1, 2))
    refused(out=torch.zeros(B, T, h, d_h))
    refused(out=torch.zeros(B, T + 1, h, d_h, dtype=torch.float16))
    refused(q=torch.zeros(B, T, h + 1, d_h, dtype=torch.float16), out=torch.zeros(B, T, h + 1, d_h, dtype=torch.float16))
    refused(mask=torch.ones(T, T + 1, dtype=torch.bool))
    refused(mask=torch.ones(B + 1, T, T, dtype=torch.bool))
    refused(mask=torch.ones(T, T))
    with pytest.raises(dv.DvError):
        dv.KVLayers([dv.KV(kv.K, kv.V, torch.zeros(B, n_max, 8), torch.zeros(B, h, n_max, dtype=torch.uint8))])
    X, valid = torch.zeros(B, n_max, 8, dtype=torch.float16), torch.zeros(B, h, n_max, dtype=torch.uint8)
    with pytest.raises(dv.DvError):
        dv.KVLayers([dv.KV(kv.K, kv.V, X, valid), dv.KV(kv.K[:1], kv.V, X, valid)])
    layers = dv.KVLayers([dv.KV(kv.K, kv.V, X, valid)])
    with pytest.raises(dv.DvError):
        dv.dv_kv_reorder(layers, pos, torch.zeros(2, 2, dtype=torch.int32), ws)
    logits = torch.zeros(4, 2, 100).transpose(0, 1)
    with pytest.raises(dv.DvError):
        dv.dv_beam_select(logits, torch.zeros(2, 4), torch.zeros(2, 4), pos, pos, ws)


def _beam_tensors(**kw):
    i32 = dict(dtype=torch.int32)
    t = dict(logits=torch.zeros(2, 3, 50), cum=torch.zeros(2, 3), score=torch.zeros(2, 4),
             token=torch.zeros(2, 4, **i32), beam=torch.zeros(2, 4, **i32), ws=torch.zeros(1 << 16, dtype=torch.uint8),
             done=torch.zeros(2, 3, dtype=torch.uint8))
    t.update(kw)
    dv.dv_beam_select(*(t[k] for k in ("logits", "cum", "score", "token", "beam", "ws")), done=t["done"])


@pytest.mark.parametrize("kw", [
    dict(token=torch.zeros(2, 3, dtype=torch.int32)), dict(beam=torch.zeros(1, 4, dtype=torch.int32)),
    dict(token=torch.zeros(2, 4, dtype=torch.int16)), dict(score=torch.zeros(1, 4)),
    dict(score=torch.zeros(2, 4, dtype=torch.float16)), dict(beam=torch.zeros(4, 2, dtype=torch.int32).t()),
    dict(cum=torch.zeros(2, 2)), dict(cum=torch.zeros(2, 3, dtype=torch.float16)),
    dict(done=torch.zeros(2, 2, dtype=torch.uint8)), dict(done=torch.zeros(2, 3, dtype=torch.int32)),
])
def test_beam_select_refuses_tensors_of_other_sizes(kw):
    with pytest.raises(dv.DvError) as e:
        _beam_tensors(**kw)
    assert e.value.status == INVALID


def _four_layers(B=4):
    kv = dv.KV(*(torch.zeros(B, 2, 16, 8, dtype=torch.float16) for _ in range(2)),
               torch.zeros(B, 16, 16, dtype=torch.float16), torch.zeros(B, 2, 16, dtype=torch.uint8))
    return dv.KVLayers([kv])


@pytest.mark.parametrize("kw", [
    dict(pos=3), dict(idx=(3, 2)), dict(count=5), dict(new_pos=3), dict(dtype=torch.int64),
])
def test_compact_refuses_lists_of_other_sizes(kw):
    i32 = dict(dtype=kw.get("dtype", torch.int32))
    pos, count, new_pos = (torch.zeros(kw.get(k, 4), **i32) for k in ("pos", "count", "new_pos"))
    with pytest.raises(dv.DvError) as e:
        dv.dv_kv_compact(_four_layers(), pos, torch.zeros(kw.get("idx", (4, 2)), **i32), count,
                         torch.zeros(256, dtype=torch.uint8), new_pos=new_pos)
    assert e.value.status == INVALID


@pytest.mark.parametrize("kw", [dict(pos=3), dict(start=1), dict(parent=(2, 3)), dict(dtype=torch.int64)])
def test_reorder_refuses_lists_of_other_sizes(kw):
    i32 = dict(dtype=kw.get("dtype", torch.int32))
    with pytest.raises(dv.DvError) as e:
        dv.dv_kv_reorder(_four_layers(), torch.zeros(kw.get("pos", 4), **i32), torch.zeros(kw.get("parent", (2, 2)), **i32),
                         torch.zeros(256, dtype=torch.uint8), start=torch.zeros(kw.get("start", 2), **i32))
    assert e.value.status == INVALID


@pytest.mark.parametrize("kw", [
    dict(pos=1), dict(nodes=1), dict(count=3), dict(head_idx=(1, 2)), dict(dtype=torch.int64),
])
def test_tree_attention_refuses_lists_of_other_sizes(kw):
    i32 = dict(dtype=kw.get("dtype", torch.int32))
    q = torch.zeros(2, 3, 2, 64, dtype=torch.float16)
    kv = dv.KV(*(torch.zeros(2, 2, 16, 64, dtype=torch.float16) for _ in range(2)), None, None)
    with pytest.raises(dv.DvError) as e:
        dv.dv_tree_attn(q, kv, torch.zeros(kw.get("pos", 2), **i32), 0.125, torch.zeros_like(q),
                        torch.zeros(1 << 26, dtype=torch.uint8), nodes=torch.zeros(kw.get("nodes", 2), **i32),
                        head_idx=torch.zeros(kw.get("head_idx", (2, 2)), **i32),
                        head_count=torch.zeros(kw.get("count", 2), **i32))
    assert e.value.status == INVALID


@pytest.mark.parametrize("scale", [2.4e38, 3.4e38, 3.4028235e38])
def test_tree_attention_refuses_a_scale_that_overflows_to_base_two(scale):
    """scale log2(e) multiplies the scores: infinite, it would make a NaN of 0."""
    need = dv.dv_tree_attn_workspace_size(2, 5, 4, 1, 64)
    assert _tree(ws_bytes=need, scale=scale) == INVALID
    assert _tree(ws_bytes=need - 1, scale=2.3e38) == WORKSPACE      # (refused for its workspace only)
