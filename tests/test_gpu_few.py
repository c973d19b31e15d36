"""The few-token layer against 64 bits, within bounds counted from roundings: sizes, types and
routings where it can go wrong, then as it is used (after a prompt, captured, on two streams)."""
from __future__ import annotations

from dataclasses import replace

import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from sparse_mixture_experts_21_b200 import _lib as L
from sparse_mixture_experts_21_b200.layer import MoELayer, make_config
from sparse_mixture_experts_21_b200.synth import WORKLOADS, Workload, make_inputs
from tests.parity_util import NEAR_TIE, TOL_BF16, f64, i64, oracle_cfg, rel_err

pytestmark = pytest.mark.gpu

MATS = ("w1", "w3", "w2", "ws1", "ws3", "ws2")


def pack(t):
    m = t.reshape(-1, t.shape[-1])
    q = torch.empty(m.shape[0], m.shape[1] // 2, dtype=torch.uint8, device="cuda")
    sf = L.mx_scales(m.shape[0], m.shape[1], "cuda")
    L.moe_quantize_mxfp4(m, q, sf)
    return q, sf


class Few:
    """One workload's inputs, buffers and call."""

    def __init__(self, w: Workload, mxfp4=False, seed=0, inp=None):
        self.w, self.mxfp4 = w, mxfp4
        self.inp = make_inputs(w, "cuda", seed) if inp is None else inp
        self.fs = w.n_shared * w.f_shared
        self.mats = {n: pack(self.inp[n]) if mxfp4 else self.inp[n] for n in MATS if n in self.inp}
        self.cfg = make_config(w)
        self.ws = torch.full((L.few_tokens_workspace_size(self.cfg, self.fs),), 0xA5, dtype=torch.uint8, device="cuda")
        self.idx = torch.full((w.T + 1, w.k), -7, dtype=torch.int32, device="cuda")
        self.wt = torch.full((w.T + 1, w.k), -7.0, device="cuda")
        self.y = torch.full((w.T + 2, w.d), 7.0, device="cuda").to(self.inp["x"].dtype)

    def call(self, stream=None, ws=None):
        fn = L.moe_few_tokens_mxfp4 if self.mxfp4 else L.moe_few_tokens
        fn(self.cfg, self.inp["x"], self.inp["w_gate"], self.inp["logit_offset"], self.inp["bias"],
           *(self.mats.get(n) for n in MATS), self.fs, self.idx, self.wt, self.y, self.ws if ws is None else ws, stream)

    def matrix(self, name, e=None):
        t = self.inp[name] if e is None else self.inp[name][e]
        return O.dequantize_mxfp4(*O.quantize_mxfp4(f64(t))) if self.mxfp4 else f64(t)

    def expect(self):
        """y in 64 bits from the GPU's own picks and weights, and how far the kernel's may be."""
        w = self.w
        T, u = w.T, 2.0 ** -24 if w.dtype == "fp32" else 2.0 ** -8       # half a step of x's type
        x, idx, wt = f64(self.inp["x"]), i64(self.idx[:T]), f64(self.wt[:T])
        y, tol = np.zeros((T, w.d)), np.zeros((T, w.d))
        load = np.zeros(w.N, int)
        cap = O.capacity(oracle_cfg(w), T) if w.capacity != "dropless" else T * w.k
        groups = {}
        for t in range(T):
            for j in range(w.k):
                e = idx[t, j]
                if load[e] < cap:
                    groups.setdefault(int(e), []).append((t, wt[t, j]))
                load[e] += 1
        parts = [(toks, [self.matrix(n, e) for n in MATS[:3]]) for e, toks in groups.items()]
        if self.fs:
            sw = np.ones(T)
            if w.shared_sink:
                sw = O.route_shared_sink(x, f64(self.inp["w_gate"]), oracle_cfg(w), bias=f64(self.inp["bias"]),
                                         logit_offset=f64(self.inp["logit_offset"]))["w_shared"]
            parts.append(([(t, sw[t]) for t in range(T)], [self.matrix(n) for n in MATS[3:]]))
        for toks, (a, b, c) in parts:
            t, g = np.array([i for i, _ in toks]), np.array([v for _, v in toks])[:, None]
            xe = x[t]
            gate, up = xe @ a.T, xe @ b.T
            h = O.silu(gate) * up
            # sums of d products in fp32 in any order: d half-steps of their terms' total each;
            # |silu'| < 1.1, the fp32 exponential, quotient and product 2^-18 of h; h to x's type u of it
            acc = w.d * 2.0 ** -24
            dh = 1.1 * acc * (np.abs(xe) @ np.abs(a).T) * np.abs(up) \
                + np.abs(O.silu(gate)) * acc * (np.abs(xe) @ np.abs(b).T) + 2.0 ** -18 * np.abs(h)
            f = c.shape[1]
            dc = 0.0
            if self.mxfp4:
                # x and h as fp16 times a power of two that puts the row's largest at 2^14 or more: bf16's
                # 8 bits are exact there but for what falls below half of fp16's smallest step, 2^-25:
                # 2^-39 of the row's largest
                ex = 2.0 ** -39 * np.abs(xe).max(1, keepdims=True)
                dh = dh + ex * (1.1 * np.abs(up) * np.abs(a).sum(1) + np.abs(O.silu(gate)) * np.abs(b).sum(1))
                dc = 2.0 ** -39 * (np.abs(h) + dh).max(1, keepdims=True) * np.abs(c).sum(1)
            dh = dh + u * (np.abs(h) + dh)
            y[t] += g * (h @ c.T)
            # the down sum: f half-steps, and the weighting, the sum over experts and a shared
            # weight 2^-18 (up to k + 2 roundings of 2^-24 and the shared weight's own)
            tol[t] += np.abs(g) * ((dh + (f * 2.0 ** -24 + 2.0 ** -18) * (np.abs(h) + dh)) @ np.abs(c).T + dc)
        return y, tol + u * (np.abs(y) + tol)

    def check(self, routing=True):
        torch.cuda.synchronize()
        w, T = self.w, self.w.T
        assert L.moe_device_status() == L.MOE_OK
        assert torch.all(self.idx[T] == -7) and torch.all(self.wt[T] == -7) and torch.all(self.y[T:] == 7)
        if routing:
            route = O.route_shared_sink if w.shared_sink else O.route
            r = route(f64(self.inp["x"]), f64(self.inp["w_gate"]), oracle_cfg(w), bias=f64(self.inp["bias"]),
                      logit_offset=f64(self.inp["logit_offset"]))
            clear = r["margin"] >= NEAR_TIE if "margin" in r else np.ones(T, bool)
            assert clear.any()
            assert np.array_equal(i64(self.idx[:T])[clear], r["idx"][clear])
            # a logit is off by at most d half-steps of its terms' total, a weight by twice that of
            # itself (softmax or sigmoid, then the quotient by the sum), and a few roundings
            dz = w.d * 2.0 ** -24 * (np.abs(f64(self.inp["x"])) @ np.abs(f64(self.inp["w_gate"])).T).max()
            assert np.allclose(f64(self.wt[:T])[clear], r["w"][clear], rtol=4 * dz + 2.0 ** -19, atol=1e-30)
        y, tol = self.expect()
        off = np.abs(f64(self.y[:T]) - y)
        assert np.all(off <= tol), float(np.max(off / np.maximum(tol, 1e-300)))


TINY = WORKLOADS["tiny_top2_fp32"]
V3 = replace(WORKLOADS["deepseek_v3"], d=512, N=64, f=256, f_shared=256)
DS = replace(WORKLOADS["deepseekmoe_16b"], d=264, N=16, f=200, f_shared=72, n_shared=2)


@pytest.mark.parametrize("T", [1, 3, 64])
@pytest.mark.parametrize("base", [TINY, replace(TINY, d=200, N=7, k=3, f=136, n_shared=1, f_shared=8),
                                  replace(TINY, d=8, N=1, k=1, f=8, capacity="dropless")])
def test_fp32(base, T):
    f = Few(replace(base, T=T), seed=T)
    f.call()
    f.check()


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 31, 33, 64])
@pytest.mark.parametrize("base", [V3, DS])
def test_bf16(base, T):
    f = Few(replace(base, T=T), seed=T)
    f.call()
    f.check()


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 31, 33, 64])
@pytest.mark.parametrize("base", [V3, replace(DS, d=384, f=640, f_shared=128), replace(DS, d=128, f=1408, n_shared=0)])
def test_mxfp4(base, T):
    f = Few(replace(base, T=T), mxfp4=True, seed=T)
    f.call()
    f.check()


@pytest.mark.parametrize("mxfp4", [False, True])
@pytest.mark.parametrize("d,N,k,f,fs,T", [(128, 512, 16, 128, 0, 64), (128, 300, 1, 128, 128, 5), (4096, 8, 2, 1408, 0, 20),
                                         (7168, 32, 8, 2048, 2048, 1), (2048, 64, 6, 1408, 2816, 40),
                                         (1024, 3, 3, 2176, 384, 13)])
def test_sizes(d, N, k, f, fs, T, mxfp4):
    w = Workload("sizes", T=T, d=d, N=N, k=k, f=f, n_shared=1 if fs else 0, f_shared=fs)
    few = Few(w, mxfp4=mxfp4, seed=N)
    few.call()
    few.check()


@pytest.mark.parametrize("change", [
    dict(score="softmax", renorm=False), dict(score="softmax", bias_std=0.0, n_groups=1),
    dict(zipf_s=1.1, score="softmax"), dict(shared_sink=True), dict(shared_sink=True, score="softmax"),
    dict(capacity="ceil_cf_T_over_N", cf=1.25), dict(capacity="floor_cf_k_T_over_N", cf=1.0),
    dict(capacity="ceil_cf_T_over_N", cf=0.001, n_shared=0), dict(n_groups=16, topk_groups=3, group_topn=1)])
@pytest.mark.parametrize("mxfp4", [False, True])
def test_routing_options(change, mxfp4):
    few = Few(replace(V3, T=37, **change), mxfp4=mxfp4, seed=5)
    few.call()
    few.check()


@pytest.mark.parametrize("kind", ["bf16", "fp32", "mxfp4"])
@pytest.mark.parametrize("T", [40, 64])
def test_every_token_to_the_same_experts(kind, T):
    """Two experts take all tokens (more than one pass of a kernel's token tile); then a capacity
    that keeps the first few, the other tokens' rows are the shared expert's alone, or zero."""
    w = replace(V3, T=T, d=256, N=8, k=2, n_groups=1, dtype="fp32" if kind == "fp32" else "bf16", bias_std=0.0)
    for change in (dict(), dict(capacity="ceil_cf_T_over_N", cf=0.5, n_shared=0)):
        ww = replace(w, **change)
        inp = make_inputs(ww, "cuda", 3)
        inp["logit_offset"] = torch.zeros(8, device="cuda")
        inp["logit_offset"][[5, 2]] = 40.0
        few = Few(ww, mxfp4=kind == "mxfp4", inp=inp)
        few.call()
        few.check(routing=False)
        assert torch.all(few.idx[:T].sort(1).values == torch.tensor([2, 5], device="cuda"))
        if change:
            cap = -(-T // 16)                       # ceil(0.5 T / 8)
            assert torch.all(few.y[cap:T] == 0) and torch.all(few.y[:cap].abs().sum(1) > 0)


@pytest.mark.parametrize("kind", ["bf16", "fp32", "mxfp4"])
def test_bad_tokens_spoil_only_their_own_rows(kind):
    """A token of NaN and one with an infinity among good ones: the good rows' bits do not change."""
    w = replace(V3, T=11, dtype="fp32" if kind == "fp32" else "bf16")
    few = Few(w, mxfp4=kind == "mxfp4", seed=1)
    few.call()
    torch.cuda.synchronize()
    want, idx = few.y[:11].clone(), few.idx[:11].clone()
    few.inp["x"][4] = float("nan")
    few.inp["x"][9, 17] = float("inf")
    few.y.fill_(7)
    few.call()
    torch.cuda.synchronize()
    L.moe_device_status()                               # a NaN token may leave no valid pick: reported, not followed
    good = [t for t in range(11) if t not in (4, 9)]
    assert torch.equal(few.y[good], want[good]) and torch.equal(few.idx[good], idx[good])
    assert torch.all(torch.isnan(few.y[4])) and not torch.isfinite(few.y[9]).any()
    assert torch.all(few.y[11:] == 7)


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
def test_extreme_magnitudes(kind):
    """Rows of 2^60 and of 2^-60 beside ordinary ones, and hidden values far past fp16's range."""
    w = replace(V3, T=6, bias_std=0.0)
    inp = make_inputs(w, "cuda", 2)
    inp["x"][1] *= 2.0 ** 20
    inp["x"][2] *= 2.0 ** -60
    inp["x"][3] = 0
    inp["x"][5, ::2] = 0
    few = Few(w, mxfp4=kind == "mxfp4", inp=inp)
    few.call()
    few.check(routing=False)
    assert torch.all(few.y[3] == 0)


def test_no_tokens_changes_nothing():
    few = Few(replace(V3, T=0))
    few.call()
    torch.cuda.synchronize()
    assert torch.all(few.y == 7) and torch.all(few.idx == -7)


def test_weight_blocks_that_are_nan():
    """A NaN block of W2 spoils its own output column for the tokens of its expert."""
    w = replace(V3, T=9, n_shared=0)
    inp = make_inputs(w, "cuda", 4)
    inp["w2"][:, 33, 40] = float("nan")
    few = Few(w, mxfp4=True, inp=inp)
    few.call()
    torch.cuda.synchronize()
    bad = torch.isnan(few.y[:9])
    assert torch.all(bad[:, 33]) and bad.sum() == 9


@pytest.mark.parametrize("kind", ["bf16", "fp32", "mxfp4"])
@pytest.mark.parametrize("T", [2, 7, 12])
def test_an_expert_that_is_nan_spoils_only_its_own_tokens(kind, T):
    w = replace(V3, T=T, N=16, k=2, n_groups=1, n_shared=0, bias_std=0.0, dtype="fp32" if kind == "fp32" else "bf16")
    inp = make_inputs(w, "cuda", 6)
    few = Few(w, mxfp4=kind == "mxfp4", inp=inp)
    few.call()
    torch.cuda.synchronize()
    want, idx = few.y[:T].clone(), few.idx[:T].clone()
    e = int(idx[0, 0])
    for name in ("w1", "w2"):
        inp[name][e] = float("nan")
    few = Few(w, mxfp4=kind == "mxfp4", inp=inp)
    few.call()
    torch.cuda.synchronize()
    hit = (idx == e).any(1)
    assert hit.any() and not hit.all()
    assert torch.isnan(few.y[:T][hit]).all() and torch.equal(few.y[:T][~hit], want[~hit])


@pytest.mark.parametrize("kind", ["bf16", "fp32", "mxfp4"])
def test_same_bits_every_time_and_on_another_stream(kind):
    few = Few(replace(V3, T=23, dtype="fp32" if kind == "fp32" else "bf16"), mxfp4=kind == "mxfp4")
    few.call()
    torch.cuda.synchronize()
    want = few.y.clone()
    s = torch.cuda.Stream()
    for stream in (None, s, s):
        few.y.fill_(7)
        few.ws.fill_(0xFF)
        torch.cuda.synchronize()
        few.call(stream)
        torch.cuda.synchronize()
        assert torch.equal(few.y, want)


def test_two_graphs_replayed_at_once():
    """Two captured steps with a workspace each, replayed on two streams again and again."""
    a, b = Few(replace(V3, T=3)), Few(replace(V3, T=50), mxfp4=True, seed=9)
    graphs, want = [], []
    for f in (a, b):
        f.call()
        torch.cuda.synchronize()
        want.append(f.y.clone())
        s = torch.cuda.Stream()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            f.call(s)
        graphs.append((g, s))
    for f in (a, b):
        f.y.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert L.moe_device_status() == L.MOE_OK
    assert torch.equal(a.y[:3], want[0][:3]) and torch.equal(b.y[:50], want[1][:50])


@pytest.mark.parametrize("mode", ["bf16", "fp32", "mxfp4"])
def test_a_prompt_and_then_its_next_tokens(mode):
    """One layer object: forward over a prompt, then forward_few steps on the same weights. A few
    tokens through either path differ by roundings, and for MXFP4 by the prompt path's 8-bit rows."""
    w = replace(WORKLOADS["deepseekmoe_16b"], name="serve", T=300, d=512, N=16, f=384, n_shared=1, f_shared=384,
                dtype="fp32" if mode == "fp32" else "bf16", mxfp4=mode == "mxfp4")
    inp = make_inputs(w, "cuda")
    lay = MoELayer(w, inp, "cuda", update_bias=False)
    y = lay.forward(inp["x"])[:300].clone()
    idx = lay.topk_idx.clone()
    # an E4M3 rounding is 2^-4 of a value at most; of a product of two such (x and h) summed with
    # signs that average, no more than 2 * 2^-4 of the output's largest
    tol = {"bf16": TOL_BF16, "fp32": 1e-5, "mxfp4": 2.0 ** -3}[mode]
    for lo, n in ((0, 1), (1, 5), (6, 64), (236, 64), (0, 1)):
        yf = lay.forward_few(inp["x"][lo:lo + n].contiguous())
        torch.cuda.synchronize()
        same = (lay.few_idx == idx[lo:lo + n]).all(1)
        assert same.float().mean() > 0.9
        assert rel_err(f64(yf[same]), f64(y[lo:lo + n][same])) < tol
    assert L.moe_device_status() == L.MOE_OK
    # captured, with new inputs for every replay
    x = inp["x"][:4].clone()
    out = torch.empty_like(x)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        lay.forward_few(x, s, out=out)
    for lo in (8, 100):
        x.copy_(inp["x"][lo:lo + 4])
        g.replay()
        assert torch.equal(out, lay.forward_few(inp["x"][lo:lo + 4].contiguous()))


def test_mxfp4_scale_byte_zero_counts():
    """Blocks of the smallest scale, 2^-127, under tokens large enough that their products are
    ordinary numbers."""
    T, N, d, f = 3, 4, 256, 128
    g = torch.Generator(device="cuda").manual_seed(9)
    x = (torch.randn(T, d, generator=g, device="cuda") * 2.0 ** 100).bfloat16()
    w = Workload("zero", T=T, N=N, k=2, d=d, f=f, n_shared=0, f_shared=0)
    wg = torch.randn(N, d, generator=g, device="cuda") * 2.0 ** -104
    w1 = torch.randn(N * f, d, generator=g, device="cuda") * 2.0 ** -128
    w3 = torch.randn(N * f, d, generator=g, device="cuda") * 2.0 ** -128
    w2 = torch.randn(N * d, f, generator=g, device="cuda") * 2.0 ** 40
    packs = []
    for m in (w1, w3, w2):
        q = torch.empty(m.shape[0], m.shape[1] // 2, dtype=torch.uint8, device="cuda")
        sf = L.mx_scales(m.shape[0], m.shape[1], "cuda")
        L.moe_quantize_mxfp4(m.float(), q, sf)
        packs.append((q, sf))
    assert int((packs[0][1] == 0).sum()) == N * f * d // 32
    c = make_config(w)
    ws = torch.empty(L.few_tokens_workspace_size(c, 0), dtype=torch.uint8, device="cuda")
    idx = torch.empty(T, 2, dtype=torch.int32, device="cuda")
    tw = torch.empty(T, 2, device="cuda")
    y = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    L.moe_few_tokens_mxfp4(c, x, wg, None, None, *packs, None, None, None, 0, idx, tw, y, ws)
    deq = []
    for (q, sf), m in zip(packs, (w1, w3, w2)):
        v = torch.empty_like(m)
        L.moe_dequantize_mxfp4(q, sf, v)
        deq.append(v.double().view(N, -1, m.shape[1]))
    ref = torch.zeros(T, d, dtype=torch.float64, device="cuda")
    for t in range(T):
        for j in range(2):
            e = int(idx[t, j])
            a, b = deq[0][e] @ x[t].double(), deq[1][e] @ x[t].double()
            h = (a * torch.sigmoid(a) * b).bfloat16().double()
            ref[t] += tw[t, j].double() * (deq[2][e] @ h)
    assert float(ref.abs().max()) > 0
    # y rounds to bf16 (2^-8 of itself); h may round the other way (2^-7 of one step of h): with
    # the sums' fp32 error far below, 2^-6 of the row's norm bounds both
    assert float((y.double() - ref).norm()) <= 2.0 ** -6 * float(ref.norm())


def test_mxfp4_codes_at_16_byte_addresses():
    """Codes that start 16 bytes into an allocation: the same results as aligned ones."""
    f = Few(replace(WORKLOADS["deepseekmoe_16b"], T=5, N=8, d=256, f=128, n_shared=1, f_shared=128), mxfp4=True)
    f.call()
    y = f.y.clone()
    keep = []
    for n, (q, sf) in f.mats.items():
        buf = torch.zeros(q.numel() + 64, dtype=torch.uint8, device="cuda")
        view = buf[16:16 + q.numel()].view(q.shape)
        view.copy_(q)
        assert view.data_ptr() % 32 == 16
        keep.append(buf)
        f.mats[n] = (view, sf)
    f.y.fill_(7.0)
    f.call()
    assert torch.equal(f.y, y)
