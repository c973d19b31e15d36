"""What the Python binding of the MXFP4 and few-token operators refuses before it calls the
library (no GPU)."""
from __future__ import annotations

from contextlib import nullcontext
from dataclasses import replace

import pytest
import torch

from sparse_mixture_experts_21_b200 import _lib as L
from sparse_mixture_experts_21_b200 import layer, synth

TINY = replace(synth.WORKLOADS["tiny_top2_fp32"], T=2, n_shared=1, f_shared=128)
MX = replace(synth.WORKLOADS["deepseekmoe_16b"], T=2, N=2, k=1, d=128, f=128, n_shared=1, f_shared=128)


def few_args(w):
    inp = synth.make_inputs(w, "cpu")
    return dict(x=inp["x"], w_gate=inp["w_gate"], off=None, bias=None,
                **{n: inp[n] for n in ("w1", "w3", "w2", "ws1", "ws3", "ws2")}, fs=w.n_shared * w.f_shared,
                idx=torch.zeros(w.T, w.k, dtype=torch.int32), tw=torch.zeros(w.T, w.k), y=torch.zeros_like(inp["x"]),
                ws=torch.zeros(16, dtype=torch.uint8))


@pytest.mark.parametrize("name", ["x", "w_gate", "w1", "w3", "w2", "ws1", "ws3", "ws2", "idx", "tw", "y", "ws"])
def test_a_missing_operand_is_refused(name):
    a = few_args(TINY)
    a[name] = None
    with pytest.raises(ValueError):
        L.moe_few_tokens(layer.make_config(TINY), *a.values())
    a = few_args(MX)
    for n in ("w1", "w3", "w2", "ws1", "ws3", "ws2"):
        m = a[n].reshape(-1, a[n].shape[-1])
        a[n] = (torch.zeros(m.shape[0], m.shape[1] // 2, dtype=torch.uint8), L.mx_scales(*m.shape, "cpu"))
    whole = a[name]
    for gone in (None, (None, whole[1]), (whole[0], None)) if isinstance(whole, tuple) else (None,):
        a[name] = gone
        with pytest.raises(ValueError):
            L.moe_few_tokens_mxfp4(layer.make_config(MX), *a.values())


@pytest.mark.parametrize("at", [0, 1, 2])
def test_quantise_refuses_a_missing_operand(at):
    args = [torch.zeros(4, 128), torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)]
    args[at] = None
    with pytest.raises(ValueError):
        L.moe_quantize_mxfp4(*args)
    with pytest.raises(ValueError):
        L.moe_dequantize_mxfp4(args[1], args[2], args[0])


# ------------------------------------------------------------------ the grouped product
def ffn_args(G=3, rows=200, d=256, f=128):
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    scales = lambda r, c, g=0: L.mx_scales(r, c, "cpu", g)  # noqa: E731
    cfg = layer.make_config(replace(synth.WORKLOADS["deepseek_v3"], d=d, T=rows))
    return cfg, dict(xq=u8(rows, d), xsf=scales(rows, d, G), rows=rows, off=torch.zeros(G + 1, dtype=torch.int32), G=G,
                     w1=u8(G * f, d // 2), s1=scales(G * f, d), w3=u8(G * f, d // 2), s3=scales(G * f, d),
                     w2=u8(G * d, f // 2), s2=scales(G * d, f), f=f, h=u8(rows, f), hs=scales(rows, f, G),
                     y=torch.zeros(rows, d, dtype=torch.bfloat16))


class Reached(Exception):
    pass


@pytest.fixture
def reach(monkeypatch):
    """The binding's checks alone: what passes them ends here instead of in the library."""
    def load():
        raise Reached
    monkeypatch.setattr(L, "load", load)
    monkeypatch.setattr(torch.cuda, "device", lambda d: nullcontext())

    def call(cfg, a):
        L.moe_grouped_ffn_mxfp4(cfg, *a.values())
    return call


def test_grouped_ffn_refuses_operands_that_do_not_fit(reach):
    """Every operand short by its smallest step, of another type, missing, or elsewhere."""
    for name in ("xq", "xsf", "off", "w1", "s1", "w3", "s3", "w2", "s2", "h", "hs", "y"):
        cfg, a = ffn_args()
        if name in ("xsf", "hs"):       # buffers for any split: at worst 2 groups of 1 row and one of 198
            per = 512 * (256 if name == "xsf" else 128) // 128
            short = a[name][:4 * per - 1]
        else:
            short = a[name].reshape(-1)[:-1]
        other = a[name].to(torch.int64 if name == "off" else torch.float16)
        for bad in (short, other, None, a[name].to("meta")):
            with pytest.raises(ValueError):
                reach(cfg, dict(a, **{name: bad}))


@pytest.mark.parametrize("G,rows", [(1, 1), (1, 128), (1, 129), (3, 2), (3, 200), (5, 700), (64, 509)])
def test_grouped_ffn_takes_scale_buffers_that_hold_every_split(reach, G, rows):
    """The fewest 128-row tiles that hold any split of the rows into groups are enough (a plain
    matrix's for one group); one atom less is refused."""
    cfg, a = ffn_args(G, rows)
    # most tiles: as many groups as there are rows for hold one row, the rest fills whole tiles
    worst = max((m + (rows - m) // 128 for m in range(1, min(G, rows) + 1)))
    for name, cols in (("xsf", 256), ("hs", 128)):
        need = worst * cols // 128 * 512
        with pytest.raises(Reached):
            reach(cfg, dict(a, **{name: torch.zeros(need, dtype=torch.uint8)}))
        with pytest.raises(ValueError):
            reach(cfg, dict(a, **{name: torch.zeros(need - 512, dtype=torch.uint8)}))
    if G == 1:
        assert L.mx_scales(rows, 256, "cpu").numel() == worst * 2 * 512


def test_grouped_ffn_takes_rows_of_the_8_bit_type(reach):
    cfg, a = ffn_args()
    for n in ("xq", "h"):
        a[n] = a[n].view(torch.float8_e4m3fn)
    with pytest.raises(Reached):
        reach(cfg, a)


# ------------------------------------------------------------------ the stream's handle
def test_the_current_streams_handle_without_the_private_name(monkeypatch):
    """Every entry point takes the current stream's handle from a private function of torch; a
    torch without it still has the stream object's."""
    class Stream:
        cuda_stream = 77
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 55, raising=False)
    assert L._stream() == 55 and L._stream(Stream) == 77
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    assert L._stream() == 77
