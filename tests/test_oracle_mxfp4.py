"""Pins of the oracle's MXFP4 functions, each against something other than the oracle, and
the host-side refusals of the MXFP4 entry points (no GPU)."""
import ctypes
from dataclasses import replace

import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from sparse_mixture_experts_21_b200 import _lib as L
from sparse_mixture_experts_21_b200 import layer, synth
from sparse_mixture_experts_21_b200.ep import EPMoELayer

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


@pytest.mark.parametrize("amax,e", [(6.0, 0), (4.0, 0), (7.99, 0), (8.0, 1), (3.99, -1), (1.0, -2), (2.0 ** -30, -32),
                                    (2.0 ** -126, -127), (0.0, -127)])
def test_scale_hand_cases(amax, e):
    x = np.zeros((1, 32))
    x[0, 5] = -amax
    q, ex = O.quantize_mxfp4(x)
    assert ex[0, 0] == e
    assert q[0, 5] == -min(6.0, np.round(amax * 2.0 ** -e * 2) / 2 if amax * 2.0 ** -e < 2 else
                           GRID[np.argmin(np.abs(GRID - amax * 2.0 ** -e))])


def test_codes_are_the_nearest_grid_point():
    x = np.random.default_rng(0).standard_normal((16, 96)) * 2.0 ** np.random.default_rng(1).integers(-9, 9, (16, 1))
    q, e = O.quantize_mxfp4(x)
    v = np.abs(x) / np.repeat(2.0 ** e, 32, axis=1)
    assert np.all(np.isin(np.abs(q), GRID))
    best = np.min(np.abs(v[:, :, None] - GRID), axis=2)
    assert np.all(np.abs(v - np.abs(q)) <= best)
    amax = np.abs(x).reshape(16, 3, 32).max(2)
    assert np.all((amax / 2.0 ** e >= 4) & (amax / 2.0 ** e < 8))


def test_requantising_is_exact_unless_the_largest_saturated():
    """Values already on the grid with their block's largest at 4 or 6 read back unchanged."""
    rng = np.random.default_rng(2)
    q = rng.choice(np.concatenate([GRID, -GRID]), (8, 64))
    q[:, 0], q[:, 32] = 6.0, -4.0
    x = q * 2.0 ** rng.integers(-20, 20, (8, 1))
    assert np.array_equal(O.dequantize_mxfp4(*O.quantize_mxfp4(x)), x)


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_a_block_that_is_not_finite_reads_back_as_nan(bad):
    x = np.ones((2, 64))
    x[1, 40] = bad
    v = O.dequantize_mxfp4(*O.quantize_mxfp4(x))
    assert np.all(np.isnan(v[1, 32:])) and np.all(v[0] == 1) and np.all(v[1, :32] == 1)


def test_ffn_is_the_dense_ffn_of_the_values_that_the_codes_stand_for():
    """With x, the weights and h already on their grids nothing is lost: one input element and
    one hidden unit that are powers of two."""
    x = np.zeros((1, 32)); x[0, 3] = 2.0
    w1 = np.zeros((32, 32)); w1[0, 3] = 64.0           # gate 128: silu(128) = 128 to 53 bits
    w3 = np.zeros((32, 32)); w3[0, 3] = 0.5            # up 1
    w2 = np.zeros((32, 32)); w2[7, 0] = -1.5
    y = O.swiglu_ffn_mxfp4(x, w1, w3, w2)
    assert y[0, 7] == -192.0 and np.count_nonzero(y) == 1


def test_ffn_close_to_exact():
    """Each weight is off by at most a quarter of its size (a step is half the value at 1, and
    saturation takes at most 2 of 8), each MXFP8 factor by at most an eighth, with signs that
    average out over the sums: well under half of the output's norm."""
    rng = np.random.default_rng(4)
    x, w1, w3 = rng.standard_normal((8, 128)), *(rng.standard_normal((2, 96, 128)) / 128 ** 0.5)
    w2 = rng.standard_normal((128, 96)) / 96 ** 0.5
    exact = O.swiglu_ffn(x, w1, w3, w2)
    y = O.swiglu_ffn_mxfp4(x, w1, w3, w2)
    assert 0.01 < np.linalg.norm(y - exact) / np.linalg.norm(exact) < 0.5


# ------------------------------------------------------------------------------ refusals
def test_mxfp4_argument_checks(lib):
    ok = 0x1000000
    IA, UN = L.MOE_ERR_INVALID_ARG, L.MOE_ERR_UNSUPPORTED
    for fn in (lambda *a: lib.moe_quantize_mxfp4(a[0], a[1], a[2], a[3], a[4], a[5], None),
               lambda *a: lib.moe_dequantize_mxfp4(a[4], a[5], a[2], a[3], a[1], a[0], None)):
        assert fn(ok, 1, 10, 96, ok, ok) == IA              # cols % 128
        assert fn(ok, 1, 10, 0, ok, ok) == IA
        assert fn(ok, 2, 10, 128, ok, ok) == IA             # no such type
        assert fn(ok, 1, -1, 128, ok, ok) == IA
        assert fn(ok + 8, 1, 10, 128, ok, ok) == IA         # misaligned
        assert fn(ok, 1, 10, 128, ok + 4, ok) == IA
        assert fn(ok, 1, 10, 128, ok, ok + 4) == IA
        assert fn(None, 1, 10, 128, ok, ok) == IA
        assert fn(ok, 1, 10, 128, None, ok) == IA
        assert fn(ok, 0, 10, 128, ok, None) == IA
        assert fn(ok, 1, 1 << 40, 128, ok, ok) == UN
        assert fn(None, 1, 0, 128, None, None) == L.MOE_OK  # no rows
    c = layer.make_config(synth.WORKLOADS["deepseek_v3"])

    def ffn(cfg=c, cap=1024, G=4, f=2048, **at):
        a = dict(xq=ok, xsf=ok, off=ok, w1=ok, s1=ok, w3=ok, s3=ok, w2=ok, s2=ok, h=ok, hs=ok, y=ok)
        a.update(at)
        return lib.moe_grouped_ffn_mxfp4(ctypes.byref(cfg), a["xq"], a["xsf"], cap, a["off"], G, a["w1"], a["s1"],
                                         a["w3"], a["s3"], a["w2"], a["s2"], f, a["h"], a["hs"], a["y"], None)
    assert ffn(f=2000) == UN
    assert ffn(cfg=layer.make_config(synth.WORKLOADS["tiny_top2_fp32"])) == UN
    assert ffn(G=0) == IA and ffn(G=513) == IA and ffn(cap=-1) == IA and ffn(f=0) == IA
    assert ffn(off=None) == IA
    assert ffn(cap=1 << 31) == UN
    assert ffn(cap=0, xq=None) == L.MOE_OK
    for name in ("xq", "xsf", "w1", "s1", "w3", "s3", "w2", "s2", "h", "hs", "y"):
        assert ffn(**{name: None}) == IA
        assert ffn(**{name: ok + 8}) == IA
    for name in ("w1", "w3", "w2"):
        assert ffn(**{name: ok + 16}) == IA                 # 4-bit codes: 32-byte bases


def test_binding_refuses_wrong_buffers():
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    q, sf = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    for args in ((x.half(), q, sf), (x, q[:3], sf), (x, q.int(), sf), (x, q, sf[:511])):
        with pytest.raises(ValueError):
            L.moe_quantize_mxfp4(*args)
        with pytest.raises(ValueError):
            L.moe_dequantize_mxfp4(args[1], args[2], args[0])


def test_layers_refuse_what_mxfp4_does_not_cover():
    with pytest.raises(ValueError):
        layer.MoELayer(replace(synth.WORKLOADS["deepseek_v3_mxfp4"], f=1000), {}, "cpu")
    with pytest.raises(ValueError):
        layer.MoELayer(replace(synth.WORKLOADS["ec_deepseekmoe_16b"], mxfp4=True), {}, "cpu")
    with pytest.raises(ValueError):
        EPMoELayer(synth.WORKLOADS["deepseek_v3_mxfp4"], {}, 0, 2, "cpu")
