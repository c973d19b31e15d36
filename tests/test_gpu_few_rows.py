"""The few-token layer, token by token in the norm of each output row, at the layers' real widths
and with every routing option at the token counts that take different code.

The bounds.  bf16 and MXFP4 weights: the output's rounding is at most 2^-8 of each value, so of
the row's norm; the hidden rows' is at most 2^-8 of each hidden value, whose signs are as good as
random, so it comes out of W2 as about that share of the row again: 2^-7 together.  (fp32 sums add
d 2^-24 of their terms at the very most of random signs, sqrt(d) 2^-24 < 2^-17.)  fp32: the sums of
d terms in the products before and after, two such factors, with a margin: 1e-5.
Each bound has to notice a missing part: what is checked against it is also checked against
the reference without one of its picks, without its shared part, and against zeros."""
from __future__ import annotations

from dataclasses import replace

import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from sparse_mixture_experts_21_b200 import _lib as L
from sparse_mixture_experts_21_b200.synth import WORKLOADS, Workload, make_inputs
from tests.parity_util import NEAR_TIE, f64, i64, oracle_cfg
from tests.test_gpu_few import TINY, V3, Few

pytestmark = pytest.mark.gpu

BOUND = {"bf16": 2.0 ** -7, "mxfp4": 2.0 ** -7, "fp32": 1e-5}


def close(y, ref, bound):
    """Every row's error within `bound` of the row's norm (rows of zeros exactly)."""
    return bool(((y - ref).norm(dim=1) <= bound * ref.norm(dim=1)).all())


class Rows(Few):
    """Few with its parts in 64 bits on the GPU, from its own picks and weights."""

    def wide(self, name, e=None):
        t = self.mats[name]
        if self.mxfp4:
            rows, cols = self.inp[name].shape[-2:]
            q, sf = t
            if e is not None:                            # rows are whole 128-row tiles
                q = q.view(self.w.N, rows, cols // 2)[e]
                sf = sf.view(self.w.N, -1)[e]
            v = torch.empty(rows, cols, device="cuda")
            L.moe_dequantize_mxfp4(q.contiguous(), sf.contiguous(), v)
            return v.double()
        return (t if e is None else t[e]).double()

    def parts(self):
        """[T, k + 1, d]: each pick's share of the output, then the shared experts'."""
        w, T = self.w, self.w.T
        out = torch.zeros(T, w.k + 1, w.d, dtype=torch.float64, device="cuda")
        x, idx, wt = self.inp["x"].double(), self.idx[:T].long(), self.wt[:T].double()
        cap = O.capacity(oracle_cfg(w), T) if w.capacity != "dropless" else T * w.k
        swiglu = lambda g, u: g * torch.sigmoid(g) * u  # noqa: E731
        self.dropped = 0
        for e in idx.unique().tolist():
            t, j = torch.nonzero(idx == e, as_tuple=True)           # tokens ascending
            self.dropped += max(0, len(t) - cap)
            t, j = t[:cap], j[:cap]
            h = swiglu(x[t] @ self.wide("w1", e).T, x[t] @ self.wide("w3", e).T)
            out[t, j] = wt[t, j][:, None] * (h @ self.wide("w2", e).T)
        if self.fs:
            h = swiglu(x @ self.wide("ws1").T, x @ self.wide("ws3").T)
            sw = torch.ones(T, dtype=torch.float64, device="cuda")
            if w.shared_sink:
                r = self.oracle()
                sw = torch.tensor(r["w_shared"], device="cuda")
            out[:, w.k] = sw[:, None] * (h @ self.wide("ws2").T)
        return out

    def oracle(self):
        route = O.route_shared_sink if self.w.shared_sink else O.route
        r = route(f64(self.inp["x"]), f64(self.inp["w_gate"]), oracle_cfg(self.w), bias=f64(self.inp["bias"]),
                  logit_offset=f64(self.inp["logit_offset"]))
        if self.w.shared_sink and not self.w.renorm:       # as moe_route: the affinities themselves
            r["w"], r["w_shared"] = np.take_along_axis(r["s"], r["idx"], axis=1), r["s_shared"]
        return r

    def check_rows(self):
        torch.cuda.synchronize()
        assert L.moe_device_status() == L.MOE_OK
        w, T = self.w, self.w.T
        bound = BOUND["mxfp4" if self.mxfp4 else w.dtype]
        r = self.oracle()
        clear = r["margin"] >= NEAR_TIE
        assert clear.any()
        assert np.array_equal(i64(self.idx[:T])[clear], r["idx"][clear])
        # a logit: each of d additions is off by 2^-24 of a partial sum, which for terms of random
        # signs stays within 4 |x| |w| / sqrt(d); sqrt(d) such errors of random signs.  A weight:
        # twice its logit's and as much of the sum's
        dz = 2.0 ** -24 * 4 * float(self.inp["x"].double().norm(dim=1).max()) * \
            float(self.inp["w_gate"].double().norm(dim=1).max())
        if self.inp["logit_offset"] is not None:           # added in fp32
            dz += 2.0 ** -24 * float(self.inp["logit_offset"].abs().max() + 8)
        assert np.allclose(f64(self.wt[:T])[clear], r["w"][clear], rtol=4 * dz + 2.0 ** -19, atol=0)
        parts = self.parts()
        ref, y = parts.sum(1), self.y[:T].double()
        assert close(y, ref, bound), float(((y - ref).norm(dim=1) / ref.norm(dim=1)).max())
        # and the check itself: a part gone, or all of them
        assert not close(torch.zeros_like(y), ref, bound)
        for j in range(w.k + 1):
            gone = parts[:, j].norm(dim=1) > 0
            assert gone.any() or self.dropped or (j == w.k and not self.fs)
            if gone.any():
                assert not close(y[gone], (ref - parts[:, j])[gone], bound), j


WIDE = [(7168, 32, 8, 2048, 2048), (4096, 8, 2, 1408, 0), (2048, 64, 6, 1408, 2816), (1024, 3, 3, 2176, 384),
        (128, 300, 1, 128, 128)]


@pytest.mark.parametrize("T", [1, 2, 5, 24, 64])
@pytest.mark.parametrize("d,N,k,f,fs", WIDE)
@pytest.mark.parametrize("mode", ["bf16", "mxfp4"])
def test_real_widths(d, N, k, f, fs, T, mode):
    w = Workload("wide", T=T, d=d, N=N, k=k, f=f, n_shared=1 if fs else 0, f_shared=fs, score="sigmoid")
    few = Rows(w, mxfp4=mode == "mxfp4", seed=T)
    few.call()
    few.check_rows()


@pytest.mark.parametrize("T", [1, 2, 5, 24, 64])
@pytest.mark.parametrize("d,N,k,f,fs", [(2048, 16, 4, 1408, 1408), (4096, 8, 2, 1024, 0), (200, 7, 3, 136, 8)])
def test_real_widths_fp32(d, N, k, f, fs, T):
    w = Workload("wide", T=T, d=d, N=N, k=k, f=f, n_shared=1 if fs else 0, f_shared=fs, score="sigmoid", dtype="fp32")
    few = Rows(w, seed=T)
    few.call()
    few.check_rows()


OPTIONS = {
    "sink": dict(shared_sink=True),
    "sink_softmax": dict(shared_sink=True, score="softmax"),
    "sink_no_renorm": dict(shared_sink=True, renorm=False),
    "no_renorm": dict(score="softmax", renorm=False, bias_std=0.0),
    "offset": dict(zipf_s=1.1, score="softmax", bias_std=0.0),
    "offset_sink_no_shared_renorm": dict(zipf_s=0.7, shared_sink=True, renorm=False),
    "top1_groups": dict(n_groups=16, topk_groups=3, group_topn=1),
    "top3_groups": dict(n_groups=4, topk_groups=3, group_topn=3),
    "six_groups": dict(N=48, n_groups=6, topk_groups=3, group_topn=2),
    "floor_capacity": dict(capacity="floor_cf_k_T_over_N", cf=1.0),
}


@pytest.mark.parametrize("T", [1, 2, 3, 7, 37])
@pytest.mark.parametrize("option", OPTIONS)
@pytest.mark.parametrize("mode", ["bf16", "fp32", "mxfp4"])
def test_routing_options_at_every_kind_of_count(option, T, mode):
    """1 and 2 tokens select on every block, 3 and 4 read whole router rows, up to 8 keep a column
    per token in the down pass; a shared weight or an offset enters each of them apart."""
    change = dict(OPTIONS[option], dtype="fp32" if mode == "fp32" else "bf16")
    few = Rows(replace(V3, T=T, **change), mxfp4=mode == "mxfp4", seed=T)
    few.call()
    few.check_rows()


@pytest.mark.parametrize("T", [2, 3, 7, 37])
@pytest.mark.parametrize("sink", [False, True])
@pytest.mark.parametrize("mode", ["bf16", "fp32", "mxfp4"])
def test_dropped_tokens_at_every_kind_of_count(T, sink, mode):
    """A capacity of one token per expert where all tokens want the same few."""
    w = replace(V3, T=T, n_groups=1, k=4, capacity="ceil_cf_T_over_N", cf=0.5, shared_sink=sink, bias_std=0.0,
                dtype="fp32" if mode == "fp32" else "bf16")
    inp = make_inputs(w, "cuda", T)
    inp["logit_offset"] = torch.zeros(w.N, device="cuda")
    inp["logit_offset"][::16] = 3.0
    few = Rows(w, mxfp4=mode == "mxfp4", inp=inp)
    few.call()
    few.check_rows()
    assert few.dropped > 0


@pytest.mark.parametrize("mode", ["bf16", "fp32", "mxfp4"])
@pytest.mark.parametrize("T", [6, 12])
def test_rows_of_far_magnitudes(mode, T):
    """Tokens of 2^60 and of 2^-60 beside ordinary ones and a zero one; hidden values far past fp16's
    range.  Affinities of the large token saturate, so the routing is the kernel's own."""
    w = replace(V3, T=T, bias_std=0.0, dtype="fp32" if mode == "fp32" else "bf16")
    inp = make_inputs(w, "cuda", 2)
    inp["x"][1] *= 2.0 ** 60
    inp["x"][2] *= 2.0 ** -60
    inp["x"][3] = 0
    few = Rows(w, mxfp4=mode == "mxfp4", inp=inp)
    few.call()
    torch.cuda.synchronize()
    ref, y = few.parts().sum(1), few.y[:T].double()
    assert torch.isfinite(ref).all() and float(ref[1].abs().max()) > 2.0 ** 110 and bool((y[3] == 0).all())
    assert float(ref[2].abs().max()) < 2.0 ** -110
    rows = [t for t in range(T) if t != 3]
    assert close(y[rows], ref[rows], BOUND[mode])
