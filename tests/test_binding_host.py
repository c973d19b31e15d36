"""What the Python binding of the MXFP4 and few-token operators refuses before it calls the
library (no GPU)."""
from __future__ import annotations

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
