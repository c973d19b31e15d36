"""Refusals of the few-token layer, before anything touches a GPU."""
import ctypes
from dataclasses import replace

import pytest
import torch

from sparse_mixture_experts_21_b200 import _lib as L
from sparse_mixture_experts_21_b200 import layer, synth

OK = 0x1000000
IA, UN, SMALL = L.MOE_ERR_INVALID_ARG, L.MOE_ERR_UNSUPPORTED, L.MOE_ERR_WORKSPACE_TOO_SMALL
V3 = synth.WORKLOADS["deepseek_v3"].with_tokens(8)


def call(lib, w=V3, fs=2048, mxfp4=False, ws_bytes=1 << 40, cfg=None, **at):
    c = layer.make_config(w) if cfg is None else cfg
    a = {n: OK for n in ("x", "wg", "off", "bias", "w1", "w3", "w2", "ws1", "ws3", "ws2", "idx", "tw", "y", "ws")}
    s = {n: OK for n in ("s1", "s3", "s2", "ss1", "ss3", "ss2")}
    a.update({k: v for k, v in at.items() if k in a})
    s.update({k: v for k, v in at.items() if k in s})
    head = (ctypes.byref(c), a["x"], a["wg"], a["off"], a["bias"])
    tail = (fs, a["idx"], a["tw"], a["y"], a["ws"], ws_bytes, None)
    mats = ("w1", "w3", "w2", "ws1", "ws3", "ws2")
    if mxfp4:
        both = [v for m, sc in zip(mats, s) for v in (a[m], s[sc])]
        return lib.moe_few_tokens_mxfp4(*head, *both, *tail)
    return lib.moe_few_tokens(*head, *(a[m] for m in mats), *tail)


@pytest.mark.parametrize("mxfp4", [False, True])
def test_arguments(lib, mxfp4):
    go = lambda **k: call(lib, mxfp4=mxfp4, **k)  # noqa: E731
    assert go(w=V3.with_tokens(65)) == UN
    assert go(w=V3.with_tokens(0), x=None, ws=None, ws_bytes=0) == L.MOE_OK
    assert go(fs=-8) == IA and go(fs=4) == IA
    assert go(w=replace(V3, f=2044)) == IA
    bad = layer.make_config(V3)
    bad.top_k = 300
    assert go(cfg=bad) == IA
    for name in ("x", "wg", "w1", "w3", "w2", "ws1", "ws3", "ws2", "y"):
        assert go(**{name: None}) == IA
        assert go(**{name: OK + 8}) == IA
    for name in ("idx", "tw"):
        assert go(**{name: None}) == IA
    for name in ("idx", "tw", "off", "bias"):
        assert go(**{name: OK + 2}) == IA
    assert go(ws=None) == IA and go(ws=OK + 8) == IA
    need = L.few_tokens_workspace_size(layer.make_config(V3), 2048)
    assert go(ws_bytes=need - 1) == SMALL


def test_mxfp4_shapes(lib):
    for w in (replace(V3, d=192), replace(V3, f=192), replace(V3, dtype="fp32")):
        assert call(lib, w=w, mxfp4=True) == UN
    assert call(lib, fs=192, mxfp4=True) == UN
    for name in ("s1", "s3", "s2", "ss1", "ss3", "ss2"):
        assert call(lib, mxfp4=True, **{name: None}) == IA
        assert call(lib, mxfp4=True, **{name: OK + 4}) == IA


def test_workspace_size(lib):
    c = layer.make_config(V3)
    out = ctypes.c_size_t()
    assert lib.moe_few_tokens_workspace_size(ctypes.byref(c), 2048, None) == IA
    assert lib.moe_few_tokens_workspace_size(ctypes.byref(c), 12, ctypes.byref(out)) == IA
    assert lib.moe_few_tokens_workspace_size(None, 0, ctypes.byref(out)) == IA
    small = L.few_tokens_workspace_size(c, 0)
    # counters, logits and hidden rows at the least
    assert small >= 256 + 4 * 8 * 256 + 2 * 8 * 8 * 2048
    assert L.few_tokens_workspace_size(c, 2048) >= small + 2 * 8 * 2048
    assert L.few_tokens_workspace_size(layer.make_config(V3.with_tokens(64)), 2048) > L.few_tokens_workspace_size(c, 2048)
    with pytest.raises(L.MoeError):
        L.few_tokens_workspace_size(layer.make_config(V3.with_tokens(65)), 0)


def test_binding_refuses_wrong_buffers():
    w = replace(synth.WORKLOADS["tiny_top2_fp32"], T=2)
    inp = synth.make_inputs(w, "cpu")
    c = layer.make_config(w)
    good = dict(x=inp["x"], wg=inp["w_gate"], w1=inp["w1"], w3=inp["w3"], w2=inp["w2"],
                idx=torch.zeros(2, 2, dtype=torch.int32), tw=torch.zeros(2, 2), y=torch.zeros(2, w.d),
                ws=torch.zeros(16, dtype=torch.uint8))
    wrong = dict(x=good["x"][:1], wg=good["wg"].bfloat16(), w1=good["w1"][:7], w3=good["w3"].double(), w2=good["w2"][:, :3],
                 idx=good["idx"].long(), tw=good["tw"][:1], y=good["y"].bfloat16(), ws=good["ws"].int())
    for name, v in wrong.items():
        a = dict(good, **{name: v})
        with pytest.raises(ValueError):
            L.moe_few_tokens(c, a["x"], a["wg"], None, None, a["w1"], a["w3"], a["w2"], None, None, None, 0, a["idx"],
                             a["tw"], a["y"], a["ws"])


def test_layer_refuses():
    lay = layer.MoELayer(synth.WORKLOADS["tiny_top2_fp32"], {}, "cpu")
    with pytest.raises(ValueError):
        lay.forward_few(torch.zeros(65, 128))
    with pytest.raises(ValueError):
        lay.forward_few(torch.zeros(2, 64))
    for name in ("ec_deepseekmoe_16b",):
        ec = layer.MoELayer.__new__(layer.MoELayer)
        ec.w, ec.weights = synth.WORKLOADS[name], {}
        with pytest.raises(ValueError):
            ec.forward_few(torch.zeros(2, 2048))
    for flag in ("fp8", "mxfp8", "nvfp4"):
        lp = layer.MoELayer.__new__(layer.MoELayer)
        lp.w, lp.weights = replace(V3, **{flag: True}), {}
        with pytest.raises(ValueError):
            lp.forward_few(torch.zeros(2, 7168))


def test_widths_past_the_offsets(lib):
    one = dict(N=1, k=1, n_groups=1, topk_groups=1, group_topn=1)
    big = (1 << 24) + 128
    assert call(lib, w=replace(V3, d=big, **one)) == UN
    assert call(lib, w=replace(V3, f=big, **one)) == UN
    assert call(lib, w=replace(V3, **one), fs=big) == UN
    assert call(lib, w=replace(V3, N=256, f=1 << 23)) == UN            # rows of a stack past 2^31
