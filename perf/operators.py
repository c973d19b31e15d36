"""The operators for serving a sparse MoE layer to few tokens and from 4-bit weights.

Three kinds of case:

  few    a whole MoE layer (router, top-k, routed and shared experts, weighted sum) for
         1 to 64 tokens, as one step of token-by-token serving calls it; expert weights
         in bf16, fp32 or MXFP4
  ffn    the grouped SwiGLU FFN of a prompt's expert-ordered rows: MXFP8 rows times
         MXFP4 expert weights
  quant  a matrix to MXFP4 (E2M1 codes, one power-of-two scale per 32 along a row)
         and back, as loading, checking or exporting weights does

`run` computes each in its plain form with elementary torch operations, or, where `own`
is set, through this package's entry points.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------- cases
def _few(name, T, weights, d, N, k, f, fs=0, score="softmax", groups=1, keep=1, bias=0.0, cf=0.0):
    """fs: total width of the shared experts; groups/keep: group-limited selection; cf > 0:
    capacity ceil(cf T / N) per expert, later tokens dropped."""
    return dict(name=name, kind="few", T=T, weights=weights, d=d, N=N, k=k, f=f, fs=fs, score=score, groups=groups,
                keep=keep, bias=bias, cf=cf)


V3 = dict(d=7168, N=256, k=8, f=2048, fs=2048, score="sigmoid", groups=8, keep=4, bias=0.02)
DS16B = dict(d=2048, N=64, k=6, f=1408, fs=2816)


def listed():
    return [
        # the smallest call: 3 tokens of the tiny fp32 layer with a capacity; latency only
        _few("few_tiny_fp32_t3", 3, "fp32", d=128, N=8, k=2, f=256, cf=1.25),
        # one user's next token through a large layer, weights in bf16 and in MXFP4
        _few("few_v3_bf16_t1", 1, "bf16", **V3),
        _few("few_v3_mxfp4_t1", 1, "mxfp4", **V3),
        # a handful of users on a small fine-grained layer; an odd count of tokens
        _few("few_16b_bf16_t7", 7, "bf16", **DS16B),
        # a server's batch of 24 on the large layer with 4-bit weights
        _few("few_v3_mxfp4_t24", 24, "mxfp4", **V3),
        # few large experts: every expert meets about a quarter of the batch
        _few("few_8x7b_bf16_t32", 32, "bf16", d=4096, N=8, k=2, f=14336),
        # the largest call: 64 tokens meet most of the 256 experts
        _few("few_v3_bf16_t64", 64, "bf16", **V3),
        # a short prompt: few rows per expert, some experts empty
        dict(name="ffn_16b_r509", kind="ffn", G=64, rows=509, d=2048, f=1408),
        # an ordinary prompt batch on the small layer, ragged groups
        dict(name="ffn_16b_r24576", kind="ffn", G=64, rows=24576, d=2048, f=1408),
        # a quarter of the large layer's experts (one of four ranks) under a full batch
        dict(name="ffn_v3_r32768", kind="ffn", G=64, rows=32768, d=7168, f=2048),
        # a few activation rows there and back: latency
        dict(name="quant_rows33_bf16", kind="quant", rows=33, cols=7168, dtype="bf16"),
        # 16 experts' matrices of the large layer as they are loaded
        dict(name="quant_weights_bf16", kind="quant", rows=16 * 2048, cols=7168, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["few", "few", "few", "ffn", "quant"])
    if kind == "quant":
        return dict(kind="quant", rows=_log(rng, 1, 60000), cols=128 * rng.randint(1, 56),
                    dtype=rng.choice(["bf16", "bf16", "fp32"]))
    if kind == "ffn":
        return dict(kind="ffn", G=_log(rng, 1, 64), rows=_log(rng, 1, 16384), d=128 * rng.randint(1, 32),
                    f=128 * rng.randint(1, 16))
    weights = rng.choice(["bf16", "bf16", "mxfp4", "mxfp4", "fp32"])
    step = 128 if weights == "mxfp4" else 8
    most = 2048 if weights == "fp32" else 7168
    d, f = step * _log(rng, 256 // step, most // step), step * _log(rng, 128 // step, 2048 // step)
    groups = rng.choice([1, 1, 4, 8])
    N = 8 * _log(rng, 1, 24)
    keep = groups if groups == 1 else rng.randint(groups // 2, groups)
    k = rng.randint(1, min(8, (N // groups) * keep))
    score = rng.choice(["softmax", "sigmoid"])
    return dict(kind="few", T=_log(rng, 1, 64), weights=weights, d=d, N=N, k=k, f=f,
                fs=rng.choice([0, f, 2 * f]), score=score, groups=groups, keep=keep,
                bias=rng.choice([0.0, 0.02]) if score == "sigmoid" else 0.0, cf=rng.choice([0.0, 0.0, 0.0, 4.0]))


def _active(c):
    """Experts that at least one of T tokens picks, under even routing."""
    return c["N"] * (1.0 - (1.0 - c["k"] / c["N"]) ** c["T"])


def work(c):
    if c["kind"] == "quant":
        n, b = c["rows"] * c["cols"], 4 if c["dtype"] == "fp32" else 2
        return {"bytes": n * (2 * b + 2 * (0.5 + 1 / 32)), "flops": 2 * n}
    if c["kind"] == "ffn":
        G, R, d, f = c["G"], c["rows"], c["d"], c["f"]
        w = min(G, R) * 3 * d * f * (0.5 + 1 / 32)
        return {"bytes": w + R * d * (1 + 1 / 32) + R * d * 2, "flops": 6 * R * d * f}
    T, d, f, fs, N, k = c["T"], c["d"], c["f"], c["fs"], c["N"], c["k"]
    b = {"bf16": 2, "fp32": 4, "mxfp4": 0.5 + 1 / 32}[c["weights"]]
    e = 4 if c["weights"] == "fp32" else 2
    return {"bytes": 3 * d * (f * _active(c) + fs) * b + 4 * N * d + 2 * T * d * e,
            "flops": 2 * T * d * (3 * (k * f + fs) + N)}


# -------------------------------------------------------------------------- MXFP4 layout
# Codes: element 2i of a row in the low nibble of byte i.  Scales: rows in tiles of 128; the
# 512 bytes of tile t and 128-wide column block c stand at (t * cols / 128 + c) * 512, in
# which scale j (columns 128 c + 32 j ..) of row m is at byte 16 (m % 32) + 4 (m / 32) + j.
def _to_atoms(s, rows, blocks):
    """Scale bytes [rows, 4 * blocks] -> tile order; rows past the end 0."""
    pad = (-rows) % 128
    s = torch.nn.functional.pad(s, (0, 0, 0, pad)).view(-1, 4, 32, blocks, 4)
    return s.permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def _from_atoms(sf, lead, rows, blocks):
    """Tile-order bytes of `lead` matrices of `rows` (a multiple of 128) -> [lead, rows, 4 * blocks]."""
    s = sf.view(lead, rows // 128, blocks, 32, 4, 4).permute(0, 1, 4, 3, 2, 5)
    return s.reshape(lead, rows, 4 * blocks)


def _exponent_byte(amax, emax):
    """Biased exponent of 2^(floor(log2 amax) - emax), at least 0."""
    ef = (amax.float().view(torch.int32) >> 23) & 0xFF
    return (ef - emax).clamp_min(0)


def _mxfp4(x):
    """x [rows, cols] -> codes [rows, cols] (0..15, sign in bit 3) and scale bytes [rows, cols / 32]."""
    v = x.float().view(x.shape[0], -1, 32)
    b = _exponent_byte(v.abs().amax(-1), 2)
    a = (v * torch.ldexp(torch.ones((), device=x.device), 127 - b)[..., None])
    m = a.abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    code = code | (torch.signbit(a).to(torch.uint8) << 3)
    return code.view(x.shape), b.to(torch.uint8)


def _pack(x):
    """Weights [rows, cols] -> packed codes and tile-order scales, a few rows at a time."""
    rows, cols = x.shape
    q = torch.empty(rows, cols // 2, dtype=torch.uint8, device=x.device)
    s = torch.empty(rows, cols // 32, dtype=torch.uint8, device=x.device)
    for r in range(0, rows, 16384):
        c, s[r:r + 16384] = _mxfp4(x[r:r + 16384])
        q[r:r + 16384] = c[:, 0::2] | (c[:, 1::2] << 4)
    return q, _to_atoms(s, rows, cols // 128)


def _pairs(device):
    """The two values of every code byte, [256, 2]."""
    v = torch.tensor(E2M1 + tuple(-e for e in E2M1), device=device)
    i = torch.arange(256, device=device)
    return torch.stack([v[i & 15], v[i >> 4]], 1)


def _unpack(q, sf, lead, rows, cols):
    """Codes [lead * rows, cols / 2] and tile-order scales -> fp32 [lead, rows, cols]."""
    s = _from_atoms(sf, lead, rows, cols // 128)
    v = _pairs(q.device)[q.view(lead, rows, cols // 2).int()].view(lead, rows, cols // 32, 32)
    return (v * torch.ldexp(torch.ones((), device=q.device), s.int() - 127)[..., None]).view(lead, rows, cols)


# ------------------------------------------------------------------------------ prepare
def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, std=1.0, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype).mul_(std)

    def stack(n, rows, cols, dtype):
        t = torch.empty(n * rows, cols, dtype=dtype, device="cuda")
        for r in range(0, n * rows, 32768):
            t[r:r + 32768] = randn(min(32768, n * rows - r), cols, std=cols ** -0.5)
        return t

    if c["kind"] == "quant":
        # weights' spread, with rows of different size
        x = randn(c["rows"], c["cols"]) * torch.exp2(randn(c["rows"], 1) * 2)
        return {"case": c, "x": x.to(torch.float32 if c["dtype"] == "fp32" else torch.bfloat16)}

    def packed(n, rows, cols):
        q = torch.empty(n * rows, cols // 2, dtype=torch.uint8, device="cuda")
        per = rows * (cols // 32)
        sf = torch.empty(n * per, dtype=torch.uint8, device="cuda")
        for e in range(n):
            q[e * rows:(e + 1) * rows], sf[e * per:(e + 1) * per] = _pack(stack(1, rows, cols, torch.bfloat16))
        return q, sf

    d, f = c["d"], c["f"]
    if c["kind"] == "ffn":
        G, R = c["G"], c["rows"]
        # uneven groups: a fifth of the experts get no rows, the rest shares like exp(N(0, 1))
        share = torch.exp(torch.randn(G, generator=torch.Generator().manual_seed(seed)))
        share[4::5] = 0
        ends = (share.cumsum(0) / share.sum() * R).round().long().tolist()
        ends[-1] = R
        offsets = [0] + ends
        x = randn(R, d)
        # the rows as the quantising permutation leaves them: MXFP8 codes, scales tiled by group
        v = x.to(torch.bfloat16).float().view(R, -1, 32)
        b = _exponent_byte(v.abs().amax(-1), 8)
        xq = (v * torch.ldexp(torch.ones((), device="cuda"), 127 - b)[..., None]).clamp(-448, 448)
        xq = xq.to(torch.float8_e4m3fn).view(torch.uint8).view(R, d)
        b = b.to(torch.uint8)
        xsf = torch.cat([_to_atoms(b[o:e], e - o, d // 128) for o, e in zip(offsets, ends) if e > o])
        room = ((R + 127) // 128 + G) * (d // 128) * 512
        xsf = torch.nn.functional.pad(xsf, (0, room - xsf.numel()))
        return {"case": c, "xq": xq, "xsf": xsf, "ends": ends,
                "offsets": torch.tensor(offsets, dtype=torch.int32, device="cuda"),
                "w1": packed(G, f, d), "w3": packed(G, f, d), "w2": packed(G, d, f)}

    N, fs = c["N"], c["fs"]
    dt = torch.float32 if c["weights"] == "fp32" else torch.bfloat16
    s = {"case": c, "x": randn(c["T"], d).to(dt), "w_gate": randn(N, d, std=d ** -0.5),
         "bias": randn(N, std=c["bias"]) if c["bias"] > 0 else None}
    for name, n, rows, cols in (("w1", N, f, d), ("w3", N, f, d), ("w2", N, d, f),
                                ("ws1", 1, fs, d), ("ws3", 1, fs, d), ("ws2", 1, d, fs)):
        if rows and cols:
            s[name] = packed(n, rows, cols) if c["weights"] == "mxfp4" else stack(n, rows, cols, dt)
    return s


# --------------------------------------------------------------------------- plain forms
def _route(c, x, w_gate, bias):
    """The picks [T, k], their weights and the kept slots, scores in 64 bits."""
    T, N, k = c["T"], c["N"], c["k"]
    z = x.double() @ w_gate.double().T
    s = torch.sigmoid(z) if c["score"] == "sigmoid" else torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
    q = s if bias is None else s + bias.double()
    if c["groups"] > 1:
        by = q.view(T, c["groups"], -1)
        best = torch.sort(by, dim=2, descending=True).values[:, :, :min(2, by.shape[2])].sum(2)
        top = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        on = torch.zeros_like(best, dtype=torch.bool).scatter_(1, top, True)
        q = torch.where(on[:, :, None], by, -math.inf).view(T, N)
    idx = torch.sort(q, dim=1, descending=True, stable=True).indices[:, :k]
    w = s.gather(1, idx)
    w = (w / w.sum(1, keepdim=True)).float()
    kept = torch.ones_like(idx, dtype=torch.bool)
    if c["cf"] > 0:
        cap = math.ceil(c["cf"] * T / N)
        hot = torch.zeros(T, N, dtype=torch.int32, device=x.device).scatter_(1, idx, 1)
        kept = (hot.cumsum(0) - hot).gather(1, idx) < cap
    return idx, w, kept


def _experts(s, name, pick):
    """fp32 matrices [n, rows, cols] of the experts `pick` (a device index) of one stack."""
    c = s["case"]
    rows, cols = (c["d"], c["f"]) if name == "w2" else (c["f"], c["d"])
    if c["weights"] == "mxfp4":
        q, sf = s[name]
        return _unpack(q.view(c["N"], -1)[pick].reshape(-1, cols // 2), sf.view(c["N"], -1)[pick].reshape(-1),
                       pick.numel(), rows, cols)
    return s[name].view(c["N"], rows, cols)[pick].float()


def _swiglu(g, u):
    return g / (1 + torch.exp(-g)) * u


def _plain_few(s):
    c = s["case"]
    T, N, k, d, fs = c["T"], c["N"], c["k"], c["d"], c["fs"]
    x = s["x"].float()
    idx, w, kept = _route(c, s["x"], s["w_gate"], s["bias"])
    gate = w * kept
    y = torch.zeros(T, d, device="cuda")
    if fs:
        if c["weights"] == "mxfp4":
            a1, a3, a2 = (_unpack(*s[n], 1, r, cc)[0] for n, r, cc in (("ws1", fs, d), ("ws3", fs, d), ("ws2", d, fs)))
        else:
            a1, a3, a2 = (s[n].float() for n in ("ws1", "ws3", "ws2"))
        y = _swiglu(x @ a1.T, x @ a3.T) @ a2.T
    if T * k <= N:
        # fewer picks than experts: one pick of every token at a time
        for j in range(k):
            e = idx[:, j]
            h = _swiglu(torch.bmm(_experts(s, "w1", e), x[:, :, None]), torch.bmm(_experts(s, "w3", e), x[:, :, None]))
            y = y + gate[:, j:j + 1] * torch.bmm(_experts(s, "w2", e), h)[:, :, 0]
    else:
        # most experts are met: each once, over all tokens, with weight 0 where not picked
        full = torch.zeros(T, N, device="cuda").scatter_(1, idx, gate)
        for e in torch.arange(N, device="cuda").split(1):
            h = _swiglu(x @ _experts(s, "w1", e)[0].T, x @ _experts(s, "w3", e)[0].T)
            y = y + full[:, e] * (h @ _experts(s, "w2", e)[0].T)
    return {"y": y.to(s["x"].dtype), "topk_idx": idx.int(), "topk_w": w}


def _plain_ffn(s):
    c = s["case"]
    G, R, d, f = c["G"], c["rows"], c["d"], c["f"]
    y = torch.empty(R, d, dtype=torch.bfloat16, device="cuda")
    one = torch.ones((), device="cuda")
    start, at = 0, 0
    # the groups' weights and rows differ in number: one product of each kind per group
    for g, end in enumerate(s["ends"]):
        n = end - start
        if n == 0:
            continue
        tiles = (n + 127) // 128
        size = tiles * (d // 128) * 512
        sx = _from_atoms(s["xsf"][at:at + size], 1, tiles * 128, d // 128)[0, :n].int()
        x = s["xq"][start:end].view(torch.float8_e4m3fn).float().view(n, -1, 32)
        x = (x * torch.ldexp(one, sx - 127)[..., None]).view(n, d)

        def weight(name, rows, cols):
            q, sf = s[name]
            per = rows * cols // 32
            return _unpack(q[g * rows:(g + 1) * rows], sf[g * per:(g + 1) * per], 1, rows, cols)[0]

        h = _swiglu(x @ weight("w1", f, d).T, x @ weight("w3", f, d).T).view(n, -1, 32)
        b = _exponent_byte(h.abs().amax(-1), 8)
        hq = (h * torch.ldexp(one, 127 - b)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).float()
        h = (hq * torch.ldexp(one, b - 127)[..., None]).view(n, f)
        y[start:end] = h @ weight("w2", d, f).T
        start, at = end, at + size
    return y


def _plain_quant(s):
    x = s["x"]
    code, b = _mxfp4(x)
    v = torch.tensor(E2M1 + tuple(-e for e in E2M1), device="cuda")[code.int()].view(x.shape[0], -1, 32)
    return (v * torch.ldexp(torch.ones((), device="cuda"), b.int() - 127)[..., None]).view(x.shape).to(x.dtype)


# ------------------------------------------------------------------- the package's calls
def _own(s):
    from sparse_mixture_experts_21_b200 import _lib as L
    c = s["case"]
    if c["kind"] == "quant":
        x = s["x"]
        rows, cols = x.shape
        q = torch.empty(rows, cols // 2, dtype=torch.uint8, device="cuda")
        sf = L.mx_scales(rows, cols, "cuda")
        y = torch.empty_like(x)
        L.moe_quantize_mxfp4(x, q, sf)
        L.moe_dequantize_mxfp4(q, sf, y)
        return y
    if "call" not in s:          # the call's shape, outputs and scratch, kept as a server keeps them
        cfg = L.MoeConfig()
        cfg.T, cfg.d_model, cfg.d_ff = (c["rows"] if c["kind"] == "ffn" else c["T"]), c["d"], c["f"]
        cfg.n_experts, cfg.top_k = c.get("N", c.get("G")), c.get("k", 1)
        cfg.renorm, cfg.x_dtype = 1, L.DTYPE_F32 if c.get("weights") == "fp32" else L.DTYPE_BF16
        if c["kind"] == "ffn":
            R, u8 = c["rows"], torch.uint8
            s["call"] = (cfg, torch.empty(R, c["f"], dtype=u8, device="cuda"), L.mx_scales(R, c["f"], "cuda", c["G"]),
                         torch.empty(R, c["d"], dtype=torch.bfloat16, device="cuda"))
        else:
            cfg.score_fn = L.SCORE_SIGMOID if c["score"] == "sigmoid" else L.SCORE_SOFTMAX
            cfg.n_groups, cfg.topk_groups, cfg.group_score_topn = c["groups"], c["keep"], min(2, c["N"] // c["groups"])
            if c["cf"] > 0:
                cfg.capacity_mode, cfg.capacity_factor = L.CAP_CEIL_CF_T_OVER_N, c["cf"]
            new = lambda *shape, dtype: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
            s["call"] = (cfg, new(c["T"], c["k"], dtype=torch.int32), new(c["T"], c["k"], dtype=torch.float32),
                         torch.empty_like(s["x"]), new(L.few_tokens_workspace_size(cfg, c["fs"]), dtype=torch.uint8))
    if c["kind"] == "ffn":
        cfg, hq, hsf, y = s["call"]
        L.moe_grouped_ffn_mxfp4(cfg, s["xq"], s["xsf"], c["rows"], s["offsets"], c["G"], *s["w1"], *s["w3"], *s["w2"],
                                c["f"], hq, hsf, y)
        return y
    cfg, idx, w, y, ws = s["call"]
    few = L.moe_few_tokens_mxfp4 if c["weights"] == "mxfp4" else L.moe_few_tokens
    few(cfg, s["x"], s["w_gate"], None, s["bias"], s["w1"], s["w3"], s["w2"], s.get("ws1"), s.get("ws3"),
        s.get("ws2"), c["fs"], idx, w, y, ws)
    return {"y": y, "topk_idx": idx, "topk_w": w}


def run(s):
    if own:
        return _own(s)
    return {"few": _plain_few, "ffn": _plain_ffn, "quant": _plain_quant}[s["case"]["kind"]](s)


# -------------------------------------------------------------------------------- exact
def _decode64(q, sf, rows, cols):
    """One MXFP4 matrix in 64 bits, from the byte addresses of its codes and scales."""
    dev = q.device
    m, col = torch.arange(rows, device=dev)[:, None], torch.arange(cols, device=dev)[None, :]
    byte = q.reshape(rows, cols // 2)[:, torch.arange(cols, device=dev) // 2].long()
    code = torch.where(col % 2 == 1, byte >> 4, byte & 15)
    e, man = (code >> 1) & 3, code & 1
    mag = torch.where(e == 0, 0.5 * man.double(), (1 + 0.5 * man.double()) * torch.exp2(e.double() - 1))
    block = torch.arange(cols // 32, device=dev)[None, :]
    at = ((m // 128) * (cols // 128) + block // 4) * 512 + 16 * (m % 32) + 4 * ((m % 128) // 32) + block % 4
    scale = torch.exp2(sf.reshape(-1)[at].double() - 127)
    return torch.where(code >= 8, -mag, mag) * scale.repeat_interleave(32, dim=1)


def _round64(v, mantissa, emin, most):
    """v in 64 bits to the nearest float with that many mantissa bits (ties to even), saturating."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -1000))).clamp_min(emin)
    e = torch.where(v.abs() >= torch.exp2(e + 1), e + 1, torch.where(v.abs() < torch.exp2(e), (e - 1).clamp_min(emin), e))
    step = torch.exp2(e - mantissa)
    return (torch.round(v / step) * step).clamp(-most, most)


def _blocks64(v, emax, mantissa, emin, most):
    """Every 32 of a row under the scale 2^(floor(log2 amax) - emax)."""
    b = v.reshape(v.shape[0], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.frexp(amax).exponent.double() - 1 - emax
    scale = torch.exp2(torch.where(amax > 0, e, torch.full_like(e, -127.0)).clamp_min(-127))
    return (_round64(b / scale, mantissa, emin, most) * scale).reshape(v.shape)


def exact(c, seed):
    s = prepare(c, seed)
    if c["kind"] == "quant":
        if c["rows"] * c["cols"] > 3e8:
            return None
        return _blocks64(s["x"].double(), 2, 1, 0, 6.0)
    act = lambda a, b: a * torch.sigmoid(a) * b  # noqa: E731
    d, f = c["d"], c["f"]

    def matrix(name, e, rows, cols):
        if c["kind"] == "ffn" or c["weights"] == "mxfp4":
            q, sf = s[name]
            return _decode64(q[e * rows:(e + 1) * rows], sf[e * rows * cols // 32:(e + 1) * rows * cols // 32], rows, cols)
        return s[name][e * rows:(e + 1) * rows].double()

    if c["kind"] == "ffn":
        if 6.0 * c["rows"] * d * f > 1e15:
            return None
        y = torch.zeros(c["rows"], d, dtype=torch.float64, device="cuda")
        start, tile = 0, 0
        for g, end in enumerate(s["ends"]):
            if end > start:
                m, block = torch.arange(end - start, device="cuda")[:, None], torch.arange(d // 32, device="cuda")[None, :]
                at = ((tile + m // 128) * (d // 128) + block // 4) * 512 + 16 * (m % 32) + 4 * ((m % 128) // 32) + block % 4
                x = s["xq"][start:end].view(torch.float8_e4m3fn).double()
                x = x * torch.exp2(s["xsf"][at].double() - 127).repeat_interleave(32, dim=1)
                h = act(x @ matrix("w1", g, f, d).T, x @ matrix("w3", g, f, d).T)
                y[start:end] = _blocks64(h, 8, 3, -6, 448.0) @ matrix("w2", g, d, f).T
                tile += (end - start + 127) // 128
                start = end
        return y

    # the layer, token by token and pick by pick
    T, N, k = c["T"], c["N"], c["k"]
    x = s["x"].double()
    z = (x[:, None, :] * s["w_gate"].double()[None]).sum(-1) if T * N * d < 2e8 else x @ s["w_gate"].double().T
    score = 1 / (1 + torch.exp(-z)) if c["score"] == "sigmoid" else torch.softmax(z, 1)
    pref = (score + (0 if s["bias"] is None else s["bias"].double())).cpu().numpy()
    size = N // c["groups"]
    taken, picks, load = {}, [], [0] * N
    cap = math.ceil(c["cf"] * T / N) if c["cf"] > 0 else T * k
    for t in range(T):
        p = pref[t]
        rank = lambda g: -sum(sorted(p[g * size:(g + 1) * size])[::-1][:min(2, size)])  # noqa: E731
        allowed = set(sorted(range(c["groups"]), key=lambda g: (rank(g), g))[:c["keep"]])
        order = sorted((e for e in range(N) if e // size in allowed), key=lambda e: (-p[e], e))[:k]
        picks.append(order)
        for e in order:
            if load[e] < cap:
                taken.setdefault(e, []).append(t)
            load[e] += 1
    idx = torch.tensor(picks, device="cuda")
    w = score.gather(1, idx)
    w = w / w.sum(1, keepdim=True)
    y = torch.zeros(T, d, dtype=torch.float64, device="cuda")
    for e, tokens in taken.items():
        t = torch.tensor(tokens, device="cuda")
        h = act(x[t] @ matrix("w1", e, f, d).T, x[t] @ matrix("w3", e, f, d).T)
        y[t] += (w[t] * (idx[t] == e)).sum(1, keepdim=True) * (h @ matrix("w2", e, d, f).T)
    if c["fs"]:
        h = act(x @ matrix("ws1", 0, c["fs"], d).T, x @ matrix("ws3", 0, c["fs"], d).T)
        y += h @ matrix("ws2", 0, d, c["fs"]).T
    return {"y": y, "topk_idx": None, "topk_w": w}
