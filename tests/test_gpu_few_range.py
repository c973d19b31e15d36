"""The few-token layer at the ends of its number range: results that are finite numbers come out
as such however far apart tokens, hidden rows and weight blocks lie."""
from __future__ import annotations

from dataclasses import replace

import pytest
import torch

from sparse_mixture_experts_21_b200 import _lib as L
from sparse_mixture_experts_21_b200.synth import make_inputs
from tests.test_gpu_few import V3, Few

pytestmark = pytest.mark.gpu

TOKENS = [1, 3, 8, 12, 40]          # columns by token up to 8; one and two passes of 32 beyond


def inputs(T, **change):
    w = replace(V3, T=T, N=16, k=4, n_groups=4, topk_groups=2, bias_std=0.0, **change)
    return w, make_inputs(w, "cuda", T)


def scale(t, e):
    """t 2^e in t's type; exact for the ordinary numbers of make_inputs, in two steps because 2^e
    itself may be out of range."""
    return t.mul_(2.0 ** (e // 2)).mul_(2.0 ** (e - e // 2))


@pytest.mark.parametrize("T", TOKENS)
def test_gate_and_up_of_large_blocks_and_small_tokens(T):
    """Blocks of 2^112 and up under tokens of 2^-114: ordinary hidden rows."""
    w, inp = inputs(T)
    scale(inp["x"], -114)
    for n in ("w_gate", "w1", "w3", "ws1", "ws3"):
        scale(inp[n], 114)
    few = Few(w, mxfp4=True, inp=inp)
    assert int(few.mats["w1"][1].max()) >= 127 + 109
    few.call()
    few.check()


@pytest.mark.parametrize("T", TOKENS)
def test_down_of_large_blocks_and_small_hidden_rows(T):
    """Hidden rows of 2^-110 under blocks of 2^116 and up: outputs of 2^11 or so."""
    w, inp = inputs(T)
    for n, e in (("w3", -110), ("ws3", -110), ("w2", 121), ("ws2", 121)):
        scale(inp[n], e)
    few = Few(w, mxfp4=True, inp=inp)
    few.call()
    few.check()


@pytest.mark.parametrize("T", TOKENS)
def test_one_expert_of_large_blocks_beside_ordinary_ones(T):
    """A routed expert and half of the shared one far from the others, in both products."""
    w, inp = inputs(T)
    for n, e in (("w1", 0), ("w3", -110), ("w2", 110)):
        scale(inp[n][3], e)
    half = w.f_shared // 2
    scale(inp["ws3"][:half], -110)
    scale(inp["ws2"][:, :half], 110)
    inp["ws2"][:, half:] = 0
    inp["logit_offset"] = torch.zeros(w.N, device="cuda")
    inp["logit_offset"][3] = 20.0
    few = Few(w, mxfp4=True, inp=inp)
    few.call()
    # its sigmoid is 1, but a group counts with two scores: another two groups may add up to more
    assert (few.idx[:T] == 3).any()
    few.check()


@pytest.mark.parametrize("T", [2, 9])
def test_small_tokens_beside_an_ordinary_one(T):
    """Columns of large blocks that only the small tokens have numbers in."""
    w, inp = inputs(T)
    half = w.d // 2
    for n in ("w1", "w3", "ws1", "ws3"):
        scale(inp[n][..., half:], 112)
    inp["x"][0, half:] = 0
    scale(inp["x"][1:, half:], -112)
    inp["x"][1:, :half] = 0
    scale(inp["w_gate"][:, half:], 112)
    few = Few(w, mxfp4=True, inp=inp)
    few.call()
    few.check()


@pytest.mark.parametrize("T", [3, 12])
def test_what_is_infinite_stays_so(T):
    """Sums past fp32 beside finite ones: the tokens that overflow, and no others, are not finite."""
    w, inp = inputs(T)
    for n in ("w1", "w3", "ws1", "ws3"):
        scale(inp[n], 114)
    scale(inp["x"][1:], -114)
    few = Few(w, mxfp4=True, inp=inp)
    few.call()
    torch.cuda.synchronize()
    assert L.moe_device_status() == L.MOE_OK
    assert not torch.isfinite(few.y[0]).any() and torch.isfinite(few.y[1:T]).all()


@pytest.mark.parametrize("T", [2, 6, 12])
def test_small_weights_of_small_hidden_rows_under_large_blocks(T):
    """Routing weights of 2^-20 or so, not renormalised, on hidden rows of 2^-117 and blocks of
    2^124 over them: their products add up to ordinary outputs."""
    w, inp = inputs(T, score="softmax", renorm=False, n_shared=0)
    for n, e in (("w3", -117), ("w2", 124)):
        scale(inp[n], e)
    # an expert of zeros takes nearly all of the softmax
    inp["w2"][0] = 0
    inp["logit_offset"] = torch.zeros(w.N, device="cuda")
    inp["logit_offset"][0] = 14.0
    few = Few(w, mxfp4=True, inp=inp)
    few.call()
    few.check(routing=False)          # affinities of 2^-20 are all near ties to the routing check


@pytest.mark.parametrize("T", [3, 12])
def test_a_nan_scale_over_nonzero_codes_is_nan(T):
    """Scale bytes of 255 that another quantiser may leave over nonzero codes: NaN, as
    moe_dequantize_mxfp4 reads them, in what depends on them and nowhere else."""
    w, inp = inputs(T, n_shared=0)
    few = Few(w, mxfp4=True, inp=inp)
    few.call()
    torch.cuda.synchronize()
    want, idx = few.y[:T].clone(), few.idx[:T].clone()
    # W2: column block 1 of row 33 of every expert; rows are 128 to a tile, K = f = 256
    sf = few.mats["w2"][1].view(w.N * w.d // 128, w.f // 128, 512)
    sf[0::w.d // 128, 0, 16 * (33 % 32) + 4 * (33 // 32) + 1] = 255
    few.call()
    torch.cuda.synchronize()
    bad = torch.isnan(few.y[:T])
    assert bad[:, 33].all() and bad.sum() == T
    assert torch.equal(few.y[:T][~bad], want[~bad])
    # W1: every scale of one expert; its tokens lose every output
    few = Few(w, mxfp4=True, inp=inp)
    e = int(idx[0, 0])
    few.mats["w1"][1].view(w.N, -1)[e] = 255
    few.call()
    torch.cuda.synchronize()
    hit = (idx == e).any(1)
    assert hit.any() and torch.isnan(few.y[:T][hit]).all() and torch.equal(few.y[:T][~hit], want[~hit])


@pytest.mark.parametrize("T", [2, 6, 12])
def test_small_weights_of_small_hidden_rows(T):
    """The same with blocks of 2^108: no sum leaves fp32 on the way, and neither the weight nor
    the hidden row's scale may lose bits to the other."""
    w, inp = inputs(T, score="softmax", renorm=False, n_shared=0)
    for n, e in (("w3", -117), ("w2", 108)):
        scale(inp[n], e)
    inp["w2"][0] = 0
    inp["logit_offset"] = torch.zeros(w.N, device="cuda")
    inp["logit_offset"][0] = 14.0
    few = Few(w, mxfp4=True, inp=inp)
    few.call()
    few.check(routing=False)
