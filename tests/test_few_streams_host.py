"""MoELayer.forward_few's host side without a GPU: which stream's pool its memory comes from,
and what it builds per call.  The library call is replaced by a recorder."""
from __future__ import annotations

from contextlib import contextmanager

import pytest
import torch

from sparse_mixture_experts_21_b200 import _lib as L
from sparse_mixture_experts_21_b200 import layer, synth

W = synth.WORKLOADS["tiny_top2_fp32"]


class Host:
    """A layer on the CPU whose allocations, launches and record_stream calls are noted with the
    stream that was current at the time ("main" outside any stream context)."""

    def __init__(self, monkeypatch):
        self.now, self.allocated, self.launched, self.recorded = "main", [], [], []
        real_empty, real_like = torch.empty, torch.empty_like

        @contextmanager
        def stream(s):
            before, self.now = self.now, s
            yield
            self.now = before

        def note(make):
            def made(*a, **k):
                t = make(*a, **k)
                self.allocated.append((t.data_ptr(), self.now))
                return t
            return made

        self.lay = layer.MoELayer(W, synth.make_inputs(W, "cpu"), "cpu")
        monkeypatch.setattr(torch.cuda, "stream", stream)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: self.now)
        monkeypatch.setattr(torch, "empty", note(real_empty))
        monkeypatch.setattr(torch, "empty_like", note(real_like))
        monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: self.recorded.append((t.data_ptr(), s)))
        monkeypatch.setattr(L, "moe_few_tokens", lambda cfg, x, *a: self.launched.append((cfg, a[-3:])))

    def pool(self, t):
        return [s for p, s in self.allocated if p == t.data_ptr()][-1]


def test_output_and_scratch_come_from_the_launch_streams_pool(monkeypatch):
    """A block of the current stream's pool may still be in use by the current stream's earlier
    work, which a launch on another stream is not ordered after."""
    h = Host(monkeypatch)
    y = h.lay.forward_few(torch.zeros(3, W.d), "side")
    (_, (y_arg, ws, stream)), = h.launched
    assert y_arg is y and stream == "side" and h.now == "main"
    for t in (y, ws, h.lay.few_idx, h.lay.few_w):
        assert h.pool(t) == "side"
    # the caller reads y on the current stream: its block waits for that too
    assert (y.data_ptr(), "main") in h.recorded


def test_without_a_stream_nothing_changes_pools(monkeypatch):
    h = Host(monkeypatch)
    y = h.lay.forward_few(torch.zeros(3, W.d))
    (_, (_, ws, stream)), = h.launched
    assert stream is None and h.pool(y) == h.pool(ws) == "main" and not h.recorded


def test_a_given_output_is_used_as_it_is(monkeypatch):
    h = Host(monkeypatch)
    h.lay.forward_few(torch.zeros(3, W.d))
    n, out = len(h.allocated), torch.zeros(3, W.d)
    assert h.lay.forward_few(torch.zeros(3, W.d), "side", out=out) is out
    assert len(h.allocated) == n and not h.recorded


def test_the_configuration_is_built_once_per_count(monkeypatch):
    """A latency-bound call builds nothing that the call before has left."""
    h = Host(monkeypatch)
    built = []
    real = layer.make_config
    monkeypatch.setattr(layer, "make_config", lambda w, T=None: built.append(T) or real(w, T))
    for n in (3, 3, 5, 3, 5):
        h.lay.forward_few(torch.zeros(n, W.d))
    assert built == [L.FEW_TOKENS_MAX, 3, 5]
    assert [c.T for c, _ in h.launched] == [3, 3, 5, 3, 5]
