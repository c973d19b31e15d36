"""MoELayer.forward_few as callers use it beside other work on the GPU."""
from __future__ import annotations

from dataclasses import replace

import pytest
import torch

from sparse_mixture_experts_21_b200 import _lib as L
from sparse_mixture_experts_21_b200.layer import MoELayer
from sparse_mixture_experts_21_b200.synth import WORKLOADS, make_inputs

pytestmark = pytest.mark.gpu


def small(mode):
    return replace(WORKLOADS["deepseekmoe_16b"], name="serve", T=16, d=512, N=16, f=384, n_shared=1, f_shared=384,
                   dtype="fp32" if mode == "fp32" else "bf16", mxfp4=mode == "mxfp4")


@pytest.mark.parametrize("mode", ["bf16", "fp32", "mxfp4"])
def test_a_side_stream_beside_work_on_freed_blocks(mode):
    """First and later calls on a side stream, without `out`, while the current stream still has
    writes pending to blocks that it has freed."""
    w = small(mode)
    inp = make_inputs(w, "cuda")
    want = MoELayer(w, inp, "cuda", update_bias=False).forward_few(inp["x"]).clone()
    lay = MoELayer(w, inp, "cuda", update_bias=False)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(3):
        torch.cuda._sleep(20_000_000)                       # ~10 ms on the current stream
        for shape, dt in ((inp["x"].shape, inp["x"].dtype), ((1 << 20,), torch.uint8), ((64, w.k), torch.int32)):
            torch.empty(shape, dtype=dt, device="cuda").fill_(3)
        outs.append(lay.forward_few(inp["x"], s))
    torch.cuda.synchronize()
    assert L.moe_device_status() == L.MOE_OK
    assert all(torch.equal(y, want) for y in outs)


def test_an_output_dropped_while_the_current_stream_reads_it():
    """The current stream reads y after waiting for the side stream; y is dropped at once and the
    side stream's next output must not land in it before that read."""
    w = small("bf16")
    inp = make_inputs(w, "cuda")
    lay = MoELayer(w, inp, "cuda", update_bias=False)
    want = lay.forward_few(inp["x"]).clone()
    other = torch.zeros_like(inp["x"])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = lay.forward_few(inp["x"], s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(20_000_000)
    kept = y.clone()
    del y
    lay.forward_few(other, s)
    torch.cuda.synchronize()
    assert torch.equal(kept, want)


def test_a_side_stream_inside_a_capture():
    """A step that forks to a side stream and drops y within the capture, replayed on new inputs."""
    w = small("mxfp4")
    inp = make_inputs(w, "cuda")
    lay = MoELayer(w, inp, "cuda", update_bias=False)
    x, out = inp["x"].clone(), torch.empty_like(inp["x"])
    lay.forward_few(x)
    torch.cuda.synchronize()
    main, side, g = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        for _ in range(2):
            side.wait_stream(main)
            y = lay.forward_few(x, side)
            main.wait_stream(side)
            out.copy_(y)
            del y
    for scale in (1.0, 0.5, 2.0):
        x.copy_(inp["x"] * scale)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, lay.forward_few(x))
    assert L.moe_device_status() == L.MOE_OK
