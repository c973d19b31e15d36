"""MXFP4 on the GPU: quantisation and its inverse bit for bit, the grouped FFN of MXFP8 rows
and MXFP4 weights against 64 bits within bounds counted from roundings, the layer end to end."""
from __future__ import annotations

from dataclasses import replace

import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from sparse_mixture_experts_21_b200 import _lib as L
from sparse_mixture_experts_21_b200.layer import MoELayer, make_config
from sparse_mixture_experts_21_b200.synth import WORKLOADS, make_inputs
from tests.parity_util import (NEAR_TIE, TOL_BF16, expert_weights_fn, f64, i64, mx_scales_rowmajor, oracle_cfg,
                               rel_err, shared_weights)

pytestmark = pytest.mark.gpu

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x):
    rows, cols = x.shape
    q = torch.full((rows, cols // 2), 0xA5, dtype=torch.uint8, device="cuda")
    sf = L.mx_scales(rows, cols, "cuda").fill_(0xA5)
    L.moe_quantize_mxfp4(x, q, sf)
    return q, sf


def values(q):
    """Code values of packed codes, element 2i in the low nibble."""
    b = q.cpu().numpy()
    c = np.stack([b & 15, b >> 4], axis=-1).reshape(b.shape[0], -1)
    return np.where(c >= 8, -1.0, 1.0) * GRID[c & 7]


def weights(gen, rows, cols, dtype):
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    return (x * torch.exp2(torch.randint(-30, 30, (rows, 1), generator=gen, device="cuda").float())).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 128), (127, 128), (129, 640), (300, 1408), (5, 7168)])
def test_quantise_and_back_bit_exact(dtype, rows, cols):
    x = weights(torch.Generator(device="cuda").manual_seed(rows + cols), rows, cols, dtype)
    x[0, :32] = 0
    x[0, 32:64] = torch.arange(32, device="cuda").float() / 4      # every tie between grid points; amax 7.75
    x[0, 64:96] = -x[0, 32:64]
    x[rows - 1, 96:128] = 2.0 ** -126                              # the smallest normal: scale byte 0
    x[rows - 1, 97] = 2.0 ** -130                                  # and a subnormal
    q, sf = quantize(x)
    q_ref, e_ref = O.quantize_mxfp4(f64(x))
    assert np.array_equal(mx_scales_rowmajor(sf, rows, cols).astype(int) - 127, e_ref)
    assert np.array_equal(values(q), q_ref)
    for back in (torch.float32, torch.bfloat16):
        y = torch.full((rows, cols), 7.0, dtype=back, device="cuda")
        L.moe_dequantize_mxfp4(q, sf, y)
        assert np.array_equal(f64(y), O.dequantize_mxfp4(q_ref, e_ref))
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_what_is_not_finite_reads_back_as_nan(dtype):
    x = torch.ones(130, 256, dtype=dtype, device="cuda")
    x[129, 5], x[3, 40], x[3, 255] = float("nan"), float("inf"), -float("inf")
    q, sf = quantize(x)
    y = torch.empty_like(x)
    L.moe_dequantize_mxfp4(q, sf, y)
    want = torch.ones_like(x)
    want[129, :32] = want[3, 32:64] = want[3, 224:] = float("nan")
    assert torch.equal(torch.isnan(y), torch.isnan(want)) and torch.equal(y.nan_to_num(5), want.nan_to_num(5))
    assert torch.all(q[129, :16] == 0)


def test_largest_fp32_values_and_every_scale_byte():
    """Blocks at every binade from subnormal to the largest finite value."""
    x = torch.exp2(torch.arange(-149, 128, dtype=torch.float64)).float().cuda()[:, None].repeat(1, 128)
    x[:, 1::2] *= -1.5
    x = x.nan_to_num(posinf=3e38, neginf=-3e38)
    q, sf = quantize(x)
    q_ref, e_ref = O.quantize_mxfp4(f64(x))
    assert np.array_equal(mx_scales_rowmajor(sf, *x.shape).astype(int) - 127, e_ref)
    assert np.array_equal(values(q), q_ref)


def quantize_rows(x, off, d):
    """MXFP8 codes and group-tiled scales of expert-ordered rows."""
    cap, G = x.shape[0], len(off) - 1
    xq = torch.zeros(cap, d, dtype=torch.uint8, device="cuda")
    xsf = L.mx_scales(cap, d, "cuda", G).fill_(0xFF)      # scales past a group's rows: NaN, to show if they are read
    nkb, tile = d // 128, 0
    for g in range(G):
        n = int(off[g + 1] - off[g])
        if n == 0:
            continue
        nt = (n + 127) // 128
        sg = torch.full((nt * nkb * 512,), 0xFF, dtype=torch.uint8, device="cuda")
        L.moe_quantize_mxfp8(x[off[g]:off[g + 1]].contiguous(), xq[off[g]:off[g + 1]], sg)
        xsf[tile * nkb * 512:(tile + nt) * nkb * 512] = sg
        tile += nt
    return xq, xsf


@pytest.mark.parametrize("d,f,sizes,slack", [
    (128, 128, [1], 0),
    (384, 384, [0, 1, 130, 257, 77], 40),      # empty and 1-row groups, ragged tails, an odd number of K blocks
    (256, 512, [128, 0, 0, 300], 1),
    (2048, 1408, [3] * 7 + [0] + [65], 0),     # f of 11 K blocks, a short last tile of y
    (128, 1408, [260, 5], 3),
    (7168, 2048, [5, 0, 190], 0),
])
def test_grouped_ffn(d, f, sizes, slack):
    G, R = len(sizes), sum(sizes)
    cap = R + slack
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    gen = torch.Generator(device="cuda").manual_seed(d + 3 * f + G)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=gen, device="cuda") * std).to(torch.bfloat16)  # noqa: E731
    x = rnd(cap, d)
    w1, w3, w2 = rnd(G * f, d, std=d ** -0.5), rnd(G * f, d, std=d ** -0.5), rnd(G * d, f, std=f ** -0.5)
    xq, xsf = quantize_rows(x, off, d)
    (w1q, s1), (w3q, s3), (w2q, s2) = (quantize(t) for t in (w1, w3, w2))
    hq = torch.full((cap, f), 3, dtype=torch.uint8, device="cuda")
    hsf = L.mx_scales(cap, f, "cuda", G).fill_(0xFF)
    y = torch.full((cap, d), 7.0, dtype=torch.bfloat16, device="cuda")
    cfg = make_config(replace(WORKLOADS["deepseek_v3"], d=d, T=R))
    L.moe_grouped_ffn_mxfp4(cfg, xq, xsf, cap, torch.tensor(off, device="cuda"), G, w1q, s1, w3q, s3, w2q, s2, f,
                            hq, hsf, y)
    torch.cuda.synchronize()
    assert L.moe_device_status() == L.MOE_OK
    assert torch.all(y[R:] == 7.0) and torch.all(hq[R:] == 3)
    hv = hq[:R].view(torch.float8_e4m3fn).double().cpu().numpy()
    e_h = mx_scales_rowmajor(hsf, R, f, off).astype(np.int64) - 127
    scale = np.repeat(2.0 ** e_h, 32, axis=1)
    xd = O.dequantize_mxfp8(*O.quantize_mxfp8(f64(x[:R])))
    yg = f64(y)
    for g in range(G):
        lo, hi = off[g], off[g + 1]
        if hi == lo:
            continue
        a, b, c = (O.dequantize_mxfp4(*O.quantize_mxfp4(f64(t[g * n:(g + 1) * n]))) for t, n in
                   ((w1, f), (w3, f), (w2, d)))
        xg = xd[lo:hi]
        gate, up = xg @ a.T, xg @ b.T
        h = O.silu(gate) * up
        # each fp32 sum of d exact products is off by at most d steps of its terms' total;
        # silu' < 1.1; the fp32 silu and product add a few relative roundings
        acc = d * 2.0 ** -23
        dh = 1.1 * acc * (np.abs(xg) @ np.abs(a).T) * np.abs(up) + np.abs(O.silu(gate)) * acc * (np.abs(xg) @ np.abs(b).T) \
            + 2.0 ** -18 * np.abs(h)
        # the block's exponent, unless the largest is that close to a power of two
        amax = np.abs(h).reshape(hi - lo, -1, 32).max(2)
        near = dh.reshape(hi - lo, -1, 32).max(2)
        e_lo, e_hi = (np.frexp(np.maximum(v, 0))[1] - 9 for v in (amax - near, amax + near))
        assert np.all((e_h[lo:hi] >= e_lo) & (e_h[lo:hi] <= e_hi))
        # E4M3: half a step is 2^-4 of the value, 2^-10 of the scale below the normals; 448 at most
        s = scale[lo:hi]
        most = np.clip(h, -448 * s, 448 * s)
        assert np.all(np.abs(hv[lo:hi] * s - most) <= 2.0 ** -4 * np.abs(most) + 2.0 ** -10 * s + dh)
        # y from the GPU's own h: the sum's bound and one rounding to bf16
        hd = hv[lo:hi] * s
        ref = hd @ c.T
        tol = f * 2.0 ** -23 * (np.abs(hd) @ np.abs(c).T)
        assert np.all(np.abs(yg[lo:hi] - ref) <= 2.0 ** -8 * (np.abs(ref) + tol) + tol)


def test_weight_scales_far_from_one_and_nan_blocks():
    """Scales of 2^-100 and 2^60 pass through the product exactly; a NaN block spoils its own
    output column alone."""
    d = f = 128
    x = torch.zeros(4, d, device="cuda", dtype=torch.bfloat16)
    x[:, 0], x[:, 1] = 2.0, 0.0
    w1 = torch.zeros(f, d, device="cuda", dtype=torch.bfloat16)
    w1[:, 0] = 20.0                                       # gate 32 or 48 after rounding: silu is linear there
    w3 = torch.zeros_like(w1)
    w3[:, 0] = 2.0 ** -100
    w2 = torch.zeros_like(w1)
    w2[:, 0] = 2.0 ** 60
    w2[9, 1] = float("nan")
    off = np.array([0, 4], np.int32)
    xq, xsf = quantize_rows(x, off, d)
    (w1q, s1), (w3q, s3), (w2q, s2) = (quantize(t) for t in (w1, w3, w2))
    hq, hsf = torch.empty(4, f, dtype=torch.uint8, device="cuda"), L.mx_scales(4, f, "cuda", 1)
    y = torch.empty(4, d, dtype=torch.bfloat16, device="cuda")
    L.moe_grouped_ffn_mxfp4(make_config(replace(WORKLOADS["deepseek_v3"], d=d, T=4)), xq, xsf, 4,
                            torch.tensor(off, device="cuda"), 1, w1q, s1, w3q, s3, w2q, s2, f, hq, hsf, y)
    # silu(32) = 32 / (1 + e^-32) is 32 - 4e-13 in 64 bits and, 1 + e^-32 being 1 in fp32 (e^-32 <
    # 2^-46 < 2^-24), exactly 32 in fp32, where h is formed: a power of two, whose block exponent the
    # 64-bit value just misses.  So the reference rounds h to fp32 before it is re-quantised.
    w2 = w2.nan_to_num()
    _, h = O.swiglu_ffn_mxfp4(f64(x), f64(w1), f64(w3), f64(w2), hidden_out=True)
    hd = O.dequantize_mxfp8(*O.quantize_mxfp8(h.astype(np.float32)))
    want = hd @ O.dequantize_mxfp4(*O.quantize_mxfp4(f64(w2))).T
    ok = np.arange(d) != 9
    assert np.array_equal(f64(y)[:, ok], want[:, ok])     # one product per output, powers of two: exact
    assert np.all(np.isnan(f64(y)[:, 9]))


@pytest.mark.parametrize("overlap", [False, True])
@pytest.mark.parametrize("T", [0, 1, 129, 777])
def test_layer_forward(T, overlap):
    w = replace(WORKLOADS["deepseekmoe_16b"], name="dsmoe_mx4_small", T=T, d=384, N=16, k=6, f=256, n_shared=1,
                f_shared=384, mxfp4=True)
    inp = make_inputs(w, "cuda")
    lay = MoELayer(w, inp, "cuda", update_bias=False, overlap_shared=overlap)
    lay.forward(inp["x"])
    torch.cuda.synchronize()
    assert L.moe_device_status() == L.MOE_OK
    if T == 0:
        return
    r = O.route(f64(inp["x"]), f64(inp["w_gate"]), oracle_cfg(w), None)
    clear = r["margin"] >= NEAR_TIE
    assert np.array_equal(i64(lay.topk_idx)[clear], r["idx"][clear])
    out = O.layer_forward(f64(inp["x"]), None, oracle_cfg(w), expert_weights_fn(inp), shared_weights(inp),
                          routing={"idx": i64(lay.topk_idx), "w": f64(lay.topk_w)}, expert_ffn=O.swiglu_ffn_mxfp4)
    assert rel_err(f64(lay.y[:T]), out["y"]) < TOL_BF16


def test_layer_captured_and_replayed():
    w = replace(WORKLOADS["deepseek_v3"], name="v3_mx4_small", T=300, d=512, N=64, f=256, f_shared=256, mxfp4=True)
    inp = make_inputs(w, "cuda")
    lay = MoELayer(w, inp, "cuda", update_bias=False)
    want = lay.forward(inp["x"]).clone()
    lay.capture(inp["x"])
    lay.y.zero_()
    lay.replay()
    torch.cuda.synchronize()
    assert L.moe_device_status() == L.MOE_OK and torch.equal(lay.y, want)


def test_quantise_on_another_stream():
    s = torch.cuda.Stream()
    x = torch.randn(64, 256, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        q, sf = quantize(x)
    s.synchronize()
    assert np.array_equal(values(q), O.quantize_mxfp4(f64(x))[0])
