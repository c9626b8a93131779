"""A matrix quantised on a stream of the caller's: what fills its buffers is ordered
on that stream too, whatever the current one still has to do."""

import contextlib

import pytest
import torch

from contextual_sparsity_decode_gb300 import binding as dv

from dvtest import TORCH


def test_the_buffers_are_made_on_the_callers_stream(monkeypatch):
    """(No GPU: the order of the host's steps.)"""
    current, steps = [None], []

    @contextlib.contextmanager
    def stream(s):
        prev, current[0] = current[0], s
        yield
        current[0] = prev

    class Stream:
        cuda_stream = 77

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: handle or "a new stream")
    zeros = torch.zeros
    monkeypatch.setattr(torch, "zeros", lambda *a, **k: steps.append(("fill", current[0])) or zeros(*a, **k))
    monkeypatch.setattr(dv, "dv_q4_quantize", lambda W, out, stream=None: steps.append(("quantise", dv._stream(stream))))
    W = torch.ones(3, 128)
    dv.Q4.of(W, 128, stream=Stream())
    dv.Q4.of(W, 128, stream=77)
    assert steps == [("fill", 77), ("fill", 77), ("quantise", 77)] * 2
    del steps[:]
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: 0)
    dv.Q4.of(W, 128, stream=0)
    assert steps == [("fill", 0), ("fill", 0), ("quantise", 0)]


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_a_busy_current_stream_does_not_reach_the_codes(dt, handle):
    W = torch.randn(300, 1000, generator=torch.Generator().manual_seed(3)).to(TORCH[dt]).cuda()
    want = dv.Q4.of(W, 64)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    torch.cuda._sleep(200_000_000)   # the current stream is busy for a tenth of a second or so
    got = dv.Q4.of(W, 64, stream=s.cuda_stream if handle else s)
    torch.cuda.synchronize()
    assert torch.equal(got.q, want.q) and torch.equal(got.scale, want.scale)


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True])
def test_the_default_stream_from_a_busy_one(handle):
    W = torch.randn(300, 1000, generator=torch.Generator().manual_seed(3)).half().cuda()
    want = dv.Q4.of(W, 128)
    torch.cuda.synchronize()
    default = torch.cuda.default_stream()
    with torch.cuda.stream(torch.cuda.Stream()):
        torch.cuda._sleep(200_000_000)
        got = dv.Q4.of(W, 128, stream=0 if handle else default)
    torch.cuda.synchronize()
    assert torch.equal(got.q, want.q) and torch.equal(got.scale, want.scale)
