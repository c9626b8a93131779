"""Host-side checks of the 4-bit matrices (no GPU needed): workspace queries
and the refusal of bad arguments before anything is launched."""

import ctypes

import pytest
import torch

from contextual_sparsity_decode_gb300 import binding as dv

FAKE = 1 << 20  # never dereferenced: validation fails first
INVALID, DTYPE, WORKSPACE, UNSUPPORTED = 1, 2, 3, 7


def _vp(x):
    return None if x is None else ctypes.c_void_p(x)


def _q4(q=FAKE, scale=FAKE, group=128):
    return ctypes.byref(dv.dv_q4(q, scale, group))


def _quantize(W=FAKE, N=4, d=128, dt=dv.DV_F16, group=128, q=FAKE, scale=FAKE, values=FAKE):
    return dv.lib().dv_q4_quantize(_vp(W), N, d, dt, group, _vp(q), _vp(scale), _vp(values), _vp(0))


@pytest.mark.parametrize("kw,status", [
    (dict(W=None), INVALID), (dict(W=FAKE + 8), INVALID), (dict(q=None), INVALID), (dict(q=FAKE + 8), INVALID),
    (dict(scale=None), INVALID), (dict(scale=FAKE + 2), INVALID), (dict(values=FAKE + 4), INVALID), (dict(N=0), INVALID),
    (dict(N=(1 << 24) + 1), INVALID), (dict(d=0), INVALID), (dict(d=100), INVALID), (dict(d=102, dt=dv.DV_F32), INVALID),
    (dict(d=32776), INVALID), (dict(dt=3), DTYPE), (dict(group=32), UNSUPPORTED), (dict(group=0), UNSUPPORTED),
])
def test_quantize_refuses_bad_arguments(kw, status):
    assert _quantize(**kw) == status


def _matvec(y=FAKE, B=2, d=128, N=10, W=None, dt=dv.DV_BF16, out=FAKE, ws=FAKE, ws_bytes=1 << 30):
    return dv.lib().dv_q4_matvec(_vp(y), B, d, N, W if W is not None else _q4(), dt, _vp(out), 0, _vp(ws), ws_bytes, _vp(0))


@pytest.mark.parametrize("kw,status", [
    (dict(y=None), INVALID), (dict(y=FAKE + 8), INVALID), (dict(out=None), INVALID), (dict(out=FAKE + 2), INVALID),
    (dict(B=0), INVALID), (dict(B=33), INVALID), (dict(d=0), INVALID), (dict(d=12), INVALID),
    (dict(d=6, dt=dv.DV_F32), INVALID), (dict(d=32776), INVALID), (dict(N=0), INVALID), (dict(N=(1 << 24) + 1), INVALID),
    (dict(W=_q4(q=None)), INVALID), (dict(W=_q4(scale=None)), INVALID), (dict(W=_q4(q=FAKE + 4)), INVALID),
    (dict(W=_q4(group=96)), UNSUPPORTED), (dict(dt=-1), DTYPE), (dict(ws=None), WORKSPACE), (dict(ws=FAKE + 4), WORKSPACE),
    (dict(ws_bytes=255), WORKSPACE),
])
def test_matvec_refuses_bad_arguments(kw, status):
    assert _matvec(**kw) == status


def _mlp(y=FAKE, B=2, d=128, N=10, W1=None, W2=None, idx=FAKE, cap=4, count=FAKE, dt=dv.DV_F16, out=FAKE, ws=FAKE,
         ws_bytes=1 << 30):
    return dv.lib().dv_q4_sparse_mlp(_vp(y), B, d, N, W1 or _q4(), W2 or _q4(), _vp(idx), cap, _vp(count), dt, _vp(out), 0,
                                     _vp(ws), ws_bytes, _vp(0))


@pytest.mark.parametrize("kw,status", [
    (dict(y=None), INVALID), (dict(y=FAKE + 2), INVALID), (dict(idx=None), INVALID), (dict(idx=FAKE + 1), INVALID),
    (dict(count=None), INVALID), (dict(count=FAKE + 2), INVALID), (dict(out=None), INVALID), (dict(out=FAKE + 1), INVALID),
    (dict(B=0), INVALID), (dict(B=33), INVALID), (dict(N=0), INVALID), (dict(N=65537), INVALID), (dict(cap=0), INVALID),
    (dict(d=20), INVALID), (dict(W1=_q4(q=None)), INVALID), (dict(W2=_q4(scale=FAKE + 1)), INVALID),
    (dict(W1=_q4(group=256)), UNSUPPORTED), (dict(W2=_q4(group=1)), UNSUPPORTED), (dict(dt=5), DTYPE),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=256), WORKSPACE),
])
def test_sparse_mlp_refuses_bad_arguments(kw, status):
    assert _mlp(**kw) == status


def test_workspace_queries():
    a, b = dv.dv_q4_matvec_workspace_size(1, 5120, 100), dv.dv_q4_matvec_workspace_size(32, 5120, 100)
    assert 0 < a < b
    a, b = dv.dv_q4_sparse_mlp_workspace_size(1, 5120, 20480, 1024), dv.dv_q4_sparse_mlp_workspace_size(4, 5120, 20480, 1024)
    assert 0 < a < b
    for bad in ((0, 64, 10), (33, 64, 10), (1, 0, 10), (1, 32769, 10), (1, 64, 0)):
        with pytest.raises(dv.DvError) as e:
            dv.dv_q4_matvec_workspace_size(*bad)
        assert e.value.status == INVALID
    for bad in ((0, 64, 10, 1), (33, 64, 10, 1), (1, 64, 65537, 1), (1, 64, 10, 0)):
        with pytest.raises(dv.DvError) as e:
            dv.dv_q4_sparse_mlp_workspace_size(*bad)
        assert e.value.status == INVALID


def _refused(status, f, *args, **kw):
    with pytest.raises(dv.DvError) as e:
        f(*args, **kw)
    assert e.value.status == status


def test_binding_refuses_tensors_of_other_sizes_and_types():
    f16, f32, u8 = torch.float16, torch.float32, torch.uint8
    Q = dv.Q4.empty(6, 200, f16, 64, "cpu")
    assert Q.q.shape == (6, 128) and Q.scale.shape == (6, 4) and (Q.N, Q.d, Q.dt) == (6, 200, dv.DV_F16)
    _refused(UNSUPPORTED, dv.Q4.empty, 6, 200, f16, 32, "cpu")
    _refused(INVALID, dv.Q4, torch.zeros(6, 64, dtype=u8), Q.scale, 200, 64)
    _refused(INVALID, dv.Q4, torch.zeros(6, 256, dtype=u8)[:, ::2], Q.scale, 200, 64)
    _refused(INVALID, dv.Q4, Q.q, torch.zeros(6, 3, dtype=f16), 200, 64)
    _refused(DTYPE, dv.Q4, Q.q, torch.zeros(6, 4, dtype=torch.float64), 200, 64)
    ws = torch.zeros(1 << 16, dtype=u8)
    _refused(INVALID, dv.dv_q4_quantize, torch.zeros(6, 192, dtype=f16), Q)
    _refused(INVALID, dv.dv_q4_quantize, torch.zeros(6, 200), Q)
    _refused(INVALID, dv.dv_q4_quantize, torch.zeros(6, 200, dtype=f16), Q, torch.zeros(6, 200))
    y, out = torch.zeros(2, 200, dtype=f16), torch.zeros(2, 6)
    _refused(INVALID, dv.dv_q4_matvec, y.float(), Q, out, ws)
    _refused(INVALID, dv.dv_q4_matvec, torch.zeros(2, 192, dtype=f16), Q, out, ws)
    _refused(INVALID, dv.dv_q4_matvec, torch.zeros(2, 400, dtype=f16)[:, ::2], Q, out, ws)
    _refused(INVALID, dv.dv_q4_matvec, y, Q, torch.zeros(2, 7), ws)
    _refused(INVALID, dv.dv_q4_matvec, y, Q, out.half(), ws)
    idx, cnt, o = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(2, 200)
    other = dv.Q4.empty(7, 200, f16, 64, "cpu")
    _refused(INVALID, dv.dv_q4_sparse_mlp, y, Q, other, idx, cnt, o, ws)
    _refused(INVALID, dv.dv_q4_sparse_mlp, y, Q, dv.Q4.empty(6, 200, f32, 64, "cpu"), idx, cnt, o, ws)
    _refused(INVALID, dv.dv_q4_sparse_mlp, y, Q, Q, idx.long(), cnt, o, ws)
    _refused(INVALID, dv.dv_q4_sparse_mlp, y, Q, Q, idx, cnt[:1], o, ws)
    _refused(INVALID, dv.dv_q4_sparse_mlp, y, Q, Q, idx, cnt, torch.zeros(2, 6), ws)
    # what lies on the host never reaches a kernel
    _refused(INVALID, dv.dv_q4_quantize, torch.zeros(6, 200, dtype=f16), Q)
    _refused(INVALID, dv.dv_q4_matvec, y, Q, out, ws)
    _refused(INVALID, dv.dv_q4_sparse_mlp, y, Q, Q, idx, cnt, o, ws)


def _sample(logits=FAKE, B=2, V=100, ld=100, dt=dv.DV_F16, u=FAKE, T=FAKE, k=FAKE, p=FAKE, min_p=FAKE, token=FAKE,
            prob=FAKE, ws=FAKE, ws_bytes=256):
    return dv.lib().dv_sample(_vp(logits), B, V, ld, dt, _vp(u), _vp(T), _vp(k), _vp(p), _vp(min_p), _vp(token),
                              _vp(prob), _vp(ws), ws_bytes, _vp(0))


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), INVALID), (dict(u=None), INVALID), (dict(token=None), INVALID), (dict(logits=FAKE + 1), INVALID),
    (dict(logits=FAKE + 2, dt=dv.DV_F32), INVALID), (dict(u=FAKE + 2), INVALID), (dict(T=FAKE + 1), INVALID),
    (dict(k=FAKE + 2), INVALID), (dict(p=FAKE + 3), INVALID), (dict(min_p=FAKE + 2), INVALID), (dict(token=FAKE + 2), INVALID),
    (dict(prob=FAKE + 2), INVALID), (dict(B=0), INVALID), (dict(B=65536), INVALID), (dict(V=0), INVALID),
    (dict(V=524289, ld=600000), INVALID), (dict(ld=99), INVALID), (dict(dt=4), DTYPE), (dict(ws=None), WORKSPACE),
    (dict(ws_bytes=255), WORKSPACE), (dict(ws=FAKE + 8), WORKSPACE),
])
def test_sample_refuses_bad_arguments(kw, status):
    assert _sample(**kw) == status


def test_sample_binding_refuses_other_tensors():
    f32, i32 = torch.float32, torch.int32
    logits, u, token, ws = torch.zeros(2, 10), torch.zeros(2), torch.zeros(2, dtype=i32), torch.zeros(256, dtype=torch.uint8)
    _refused(INVALID, dv.dv_sample, torch.zeros(2, 20)[:, ::2], u, token, ws)
    _refused(INVALID, dv.dv_sample, logits, u.double(), token, ws)
    _refused(INVALID, dv.dv_sample, logits, torch.zeros(3), token, ws)
    _refused(INVALID, dv.dv_sample, logits, u, token.long(), ws)
    for name, t in (("temperature", torch.zeros(1)), ("top_k", torch.zeros(2)), ("top_p", torch.zeros(2, dtype=torch.float16)),
                    ("min_p", torch.zeros(4)[::2]), ("prob", torch.zeros(2, dtype=torch.float64))):
        _refused(INVALID, dv.dv_sample, logits, u, token, ws, **{name: t})
    _refused(INVALID, dv.dv_sample, logits, u, token, ws)   # on the host
    for bad in ((0, 10), (65536, 10), (1, 0), (1, 524289)):
        with pytest.raises(dv.DvError):
            dv.dv_sample_workspace_size(*bad)
    assert dv.dv_sample_workspace_size(65535, 524288) >= 256
