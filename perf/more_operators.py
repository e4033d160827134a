"""Cases of the training step's operators around the FP8 products, for measurement.

Every case is one call of a training step (or, for single tokens, of serving):

  layer_norm            y = (x - mean) rstd * weight + bias, written as the E4M3 operand
                        of the next product (1x128 groups) and, for training, as BF16
  layer_norm_backward   dx, and the sums over all rows that are dweight and dbias
  expert_tokens         activations grouped by expert, ragged: E4M3 codes of x^T in
                        groups of 128 tokens that never straddle experts
  expert_wgrad          dW[e] = dY_e^T X_e for all experts at once, from those codes:
                        products whose inner extent is the expert's number of tokens
  adamw                 one AdamW step over many tensors, moments in 32 bits
  adamw_8bit            the same with moments in E4M3, 128 elements a scale

`own` chooses between the plain form (elementary torch operations in float32)
and the framework's operators.  exact() evaluates the definitions in float64.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
BF16 = torch.bfloat16
GROUP = 128


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # One token of a chat session before its next projection: latency counts.
        {"name": "layer norm, 1 token", "kind": "layer_norm", "M": 1, "N": 7168, "x": "bf16",
         "codes": True, "y": False},
        # A training step's forward: codes for the projection, BF16 y for its weight gradient.
        {"name": "layer norm, 4096 tokens", "kind": "layer_norm", "M": 4096, "N": 7168, "x": "f32",
         "codes": True, "y": True},
        # A training step's backward over the same activations.
        {"name": "layer norm backward, 4096", "kind": "layer_norm_backward", "M": 4096, "N": 7168,
         "x": "f32", "dy": "bf16"},
        # A small batch of a narrow layer whose width is a multiple of nothing.
        {"name": "layer norm backward, odd", "kind": "layer_norm_backward", "M": 777, "N": 1001,
         "x": "bf16", "dy": "bf16"},
        # 512 tokens routed over 8 experts of a narrow layer, some with one token or none.
        {"name": "expert tokens, 512", "kind": "expert_tokens", "G": 8, "M": 512, "K": 2048},
        # 4096 tokens routed to 8 of 256 experts each: 128 tokens an expert, no two alike.
        {"name": "expert tokens, 32768", "kind": "expert_tokens", "G": 256, "M": 32768, "K": 7168},
        # A small mixture's gradient, a few dozen tokens an expert.
        {"name": "expert wgrad, 4 experts", "kind": "expert_wgrad", "G": 4, "M": 200, "N": 512,
         "K": 1024, "out": "bf16"},
        # Gate and up projection of 32 resident experts.
        {"name": "expert wgrad, gate and up", "kind": "expert_wgrad", "G": 32, "M": 8192,
         "N": 4096, "K": 7168, "out": "bf16"},
        # Norms, biases and router rows of a model: many small tensors in one step.
        {"name": "AdamW, 60 small tensors", "kind": "adamw", "count": 60, "lo": 1, "hi": 16384,
         "grad": "f32", "copies": False, "clip": True},
        # The projections of one dense layer, moments in 32 bits.
        {"name": "AdamW, one layer", "kind": "adamw", "count": 3, "lo": 14680064, "hi": 14680064,
         "grad": "bf16", "copies": True, "clip": True},
        # A few uneven tensors whose sizes end inside a scale's group, moments in 8 bits.
        {"name": "AdamW 8-bit, uneven", "kind": "adamw_8bit", "count": 5, "lo": 1000, "hi": 500000,
         "grad": "f32", "copies": True, "clip": False},
        # The experts of a layer, moments in 8 bits.
        {"name": "AdamW 8-bit, experts", "kind": "adamw_8bit", "count": 16, "lo": 14680064,
         "hi": 29360128, "grad": "bf16", "copies": True, "clip": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["layer_norm", "layer_norm_backward", "expert_tokens", "expert_wgrad",
                       "adamw", "adamw_8bit"])
    if kind == "layer_norm":
        codes = rng.random() < 0.6
        N = GROUP * _log(rng, 1, 64) if codes else _log(rng, 64, 8192)
        return {"kind": kind, "M": _log(rng, 1, 29000000 // N), "N": N,
                "x": rng.choice(["bf16", "f32"]), "codes": codes,
                "y": not codes or rng.random() < 0.5}
    if kind == "layer_norm_backward":
        N = _log(rng, 64, 8192)
        return {"kind": kind, "M": _log(rng, 1, 29000000 // N), "N": N,
                "x": rng.choice(["bf16", "f32"]), "dy": rng.choice(["bf16", "f32"])}
    if kind == "expert_tokens":
        G = _log(rng, 2, 256)
        return {"kind": kind, "G": G, "M": G * _log(rng, 1, 32768 // G // 2),
                "K": GROUP * _log(rng, 1, 56)}
    if kind == "expert_wgrad":
        while True:
            G = _log(rng, 2, 64)
            c = {"kind": kind, "G": G, "M": G * _log(rng, 1, 600), "N": GROUP * _log(rng, 1, 56),
                 "K": GROUP * _log(rng, 1, 56), "out": "bf16"}
            w = work(c)
            if w["bytes"] <= 2.2e9 and w["flops"] <= 4.8e11:
                return c
    hi = _log(rng, 100, 4000000)
    return {"kind": kind, "count": _log(rng, 1, 60), "lo": max(1, hi // 1000), "hi": hi,
            "grad": rng.choice(["bf16", "f32"]), "copies": rng.random() < 0.5,
            "clip": rng.random() < 0.5}


def _sizes(c):
    """Elements of each tensor: from hi to lo, evenly over the logarithm, ragged
    (every third as it is, the others with an odd remainder)."""
    n = []
    for i in range(c["count"]):
        f = i / max(1, c["count"] - 1)
        v = int(round(math.exp(math.log(c["hi"]) * (1 - f) + math.log(c["lo"]) * f)))
        n.append(v if i % 3 == 0 else max(1, v - 37 * i % 101))
    return n


def _width(name):
    return 2 if name == "bf16" else 4


def _blocks(c):
    """Most groups of 128 tokens that M rows in G experts can take."""
    return (c["M"] + (GROUP - 1) * min(c["G"], c["M"])) // GROUP


def work(c):
    k = c["kind"]
    if k == "layer_norm":
        M, N = c["M"], c["N"]
        out = (1 + 4 / GROUP) * c["codes"] + 2 * c["y"]
        return {"bytes": M * N * (_width(c["x"]) + out) + 8 * N + 8 * M, "flops": 8 * M * N}
    if k == "layer_norm_backward":
        M, N = c["M"], c["N"]
        return {"bytes": M * N * (2 * _width(c["x"]) + _width(c["dy"])) + 12 * N + 8 * M,
                "flops": 14 * M * N}
    if k == "expert_tokens":
        # rows read; codes and scales of every whole group written, on average
        # half a group of padding an expert
        cols = c["M"] + 64 * c["G"]
        return {"bytes": c["K"] * (2 * c["M"] + cols * (1 + 4 / GROUP)), "flops": 3 * c["M"] * c["K"]}
    if k == "expert_wgrad":
        G, M, N, K = c["G"], c["M"], c["N"], c["K"]
        return {"bytes": (N + K) * M * (1 + 4 / GROUP) + _width(c["out"]) * G * N * K,
                "flops": 2 * M * N * K}
    n = sum(_sizes(c))
    state = 16 if k == "adamw" else 4 + 16 / GROUP
    return {"bytes": n * (8 + _width(c["grad"]) + state + 2 * c["copies"]), "flops": 16 * n}


# ------------------------------------------------------------- making inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _rows(g, M, N, dtype):
    """Residual-stream rows: N(0, 1), an offset of each row, one channel in a
    hundred 20 times as large."""
    x = torch.randn((M, N), generator=g, device=DEV)
    x *= torch.where(torch.rand(N, generator=g, device=DEV) < 0.01, 20.0, 1.0)
    x += 0.5 * torch.randn((M, 1), generator=g, device=DEV)
    return x.to(BF16) if dtype == "bf16" else x


def _offsets(seed, G, M):
    """Rows of each expert: random shares of M, one expert in 25 without any."""
    r = np.random.default_rng([int(seed), 78])
    share = r.gamma(3.0, 1.0, G) * (r.random(G) > 0.04)
    share = share if share.sum() > 0 else np.ones(G)
    n = np.floor(share / share.sum() * M).astype(np.int64)
    n[int(np.argmax(share))] += M - int(n.sum())
    off = np.zeros(G + 1, dtype=np.int32)
    off[1:] = np.cumsum(n)
    return off


def _groups(v):
    """1x128 groups along the last axis of float32 [R][n]: E4M3 values, scales [n/128][R]."""
    R, n = v.shape
    v = v.reshape(R, n // GROUP, GROUP)
    amax = v.abs().amax(dim=2)
    inv = 448.0 / amax
    flush = ~torch.isfinite(inv)
    inv = torch.where(flush, 0.0, inv)
    q = (v * inv[:, :, None]).to(E4M3).reshape(R, n)
    return q, torch.where(flush, 0.0, amax / 448.0).t().contiguous()


def _padded(off):
    """First column of each expert's groups, and the end: [G + 1]."""
    n = off[1:] - off[:-1]
    p = torch.zeros_like(off)
    p[1:] = torch.cumsum((n + (GROUP - 1)) // GROUP * GROUP, 0)
    return p


def _columns(off, cols):
    """Of each of `cols` padded columns: its row of x, and whether it has one."""
    p = _padded(off)
    col = torch.arange(cols, device=off.device)
    e = (torch.searchsorted(p, col, right=True) - 1).clamp_max(off.numel() - 2)
    row = off[e] + col - p[e]
    live = row < off[e + 1]
    return torch.where(live, row, 0), live


def _by_expert(x, off, cols):
    """x[M][K] -> float32 x^T [K][cols], every expert's tokens from a group's start."""
    row, live = _columns(off.long(), cols)
    return torch.where(live[:, None], x.float()[row], 0.0).t().contiguous()


def prepare(case, seed):
    c, g = case, _gen(seed)
    k = c["kind"]
    s = {"case": c}
    if k.startswith("layer_norm"):
        M, N = c["M"], c["N"]
        s["x"] = _rows(g, M, N, c["x"])
        s["weight"] = 1.0 + 0.2 * torch.randn(N, generator=g, device=DEV)
        s["bias"] = 0.1 * torch.randn(N, generator=g, device=DEV)
        s["eps"] = 1e-5
        if k == "layer_norm_backward":
            dy = 0.02 * torch.randn((M, N), generator=g, device=DEV)
            s["dy"] = dy.to(BF16) if c["dy"] == "bf16" else dy
            x = s["x"].double()
            mean = x.mean(dim=1)
            var = (x - mean[:, None]).square().mean(dim=1)
            s["mean"], s["rstd"] = mean.float(), torch.rsqrt(var + s["eps"]).float()
        return s
    if k.startswith("expert"):
        G, M = c["G"], c["M"]
        s["off"] = torch.from_numpy(_offsets(seed, G, M)).to(DEV)
        if k == "expert_tokens":
            s["x"] = _rows(g, M, c["K"], "bf16")
            return s
        cols = GROUP * _blocks(c)
        for name, width, size in (("a", c["N"], 0.02), ("b", c["K"], 1.0)):
            v = _by_expert((size * _rows(g, M, width, "f32")).to(BF16), s["off"], cols)
            q, s[name + "_s"] = _groups(v)
            s[name + "_q"] = q.view(torch.uint8)
        n = s["off"][1:] - s["off"][:-1]
        s["most"] = -(-int(n.max()) // GROUP) * GROUP
        return s
    return _prepare_adamw(c, g, s)


def _prepare_adamw(c, g, s):
    """Flat buffers, each tensor from a multiple of 128 elements on, and the
    tensors as views of them."""
    sizes = _sizes(c)
    room = [-(-n // GROUP) * GROUP for n in sizes]
    start = np.concatenate([[0], np.cumsum(room)])
    total = int(start[-1])
    live = torch.zeros(total, dtype=torch.bool, device=DEV)
    for n, at in zip(sizes, start):
        live[at:at + n] = True
    p = 0.02 * torch.randn(total, generator=g, device=DEV)
    grad = 1e-3 * torch.randn(total, generator=g, device=DEV)
    root = 1e-3 * (0.5 + torch.rand(total, generator=g, device=DEV))
    m = 0.3 * root * torch.randn(total, generator=g, device=DEV)
    for t in (p, grad, root, m):
        t *= live
    del live
    s.update(p=p, g=grad.to(BF16) if c["grad"] == "bf16" else grad, starts=start, sizes=sizes)
    del grad
    if c["kind"] == "adamw":
        s["m"], s["v"] = m, root.square_()
    else:
        for name, t in (("m", m), ("v", root)):
            q, sc = _groups(t.view(1, -1))
            s[name + "_q"], s[name + "_s"] = q.view(torch.uint8).view(-1), sc.view(-1)
    del m, root
    s["copy"] = torch.zeros(total, dtype=BF16, device=DEV) if c["copies"] else None
    s["clip"] = torch.full((1,), 0.7, device=DEV) if c["clip"] else None
    # a step number of its own for each set of inputs
    s["step"] = int(torch.randint(10, 4000, (1,), generator=g, device=DEV))
    s["hyper"] = {"lr": 1e-4, "betas": (0.9, 0.95), "eps": 1e-8, "weight_decay": 0.1}

    def views(t, unit=1):
        return [t[at // unit:at // unit + -(-n // unit)] for n, at in zip(sizes, start)]
    s["tensors"] = {k: views(s[k], GROUP if k.endswith("_s") else 1)
                    for k in ("p", "g", "m", "v", "m_q", "m_s", "v_q", "v_s", "copy")
                    if s.get(k) is not None}
    return s


# ------------------------------------------------------------ the plain forms
def _norm(x, weight, bias, eps):
    x = x.float()
    mean = x.mean(dim=1)
    d = x - mean[:, None]
    rstd = 1.0 / torch.sqrt(d.square().mean(dim=1) + eps)
    return d * rstd[:, None] * weight + bias, mean, rstd


def _plain_norm_backward(s):
    x, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    xhat = (x - s["mean"][:, None]) * rstd
    dz = dy * s["weight"]
    c1 = (dz * xhat).mean(dim=1, keepdim=True)
    c2 = dz.mean(dim=1, keepdim=True)
    dx = rstd * (dz - c2 - xhat * c1)
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xhat).sum(dim=0), "dbias": dy.sum(dim=0)}


def _wide(codes, scales, t=torch.float32):
    """Values of E4M3 codes [R][n] with scales [n/128][R]."""
    R, n = codes.shape
    v = codes.view(E4M3).to(t).reshape(R, n // GROUP, GROUP)
    return (v * scales.t().to(t)[:, :, None]).reshape(R, n)


def _plain_wgrad(s):
    # every expert's columns padded to the longest's, one batched product
    off, most = s["off"].long(), s["most"]
    p = _padded(off)
    j = torch.arange(most, device=DEV)
    live = j[None, :] < (p[1:] - p[:-1])[:, None]
    at = torch.where(live, p[:-1, None] + j[None, :], 0)
    a = _wide(s["a_q"], s["a_s"])[:, at] * live
    b = _wide(s["b_q"], s["b_s"]).t().contiguous()[at]
    w = torch.bmm(a.permute(1, 0, 2).contiguous(), b)
    return {"dw": w.to(BF16) if s["case"]["out"] == "bf16" else w}


def _dither(s):
    """20 bits for each element: of its place in its tensor and of the step."""
    starts = torch.from_numpy(s["starts"]).to(DEV)
    i = torch.arange(int(s["starts"][-1]), device=DEV)
    i -= torch.repeat_interleave(starts[:-1], starts[1:] - starts[:-1], output_size=i.numel())
    return (((i * 0x85EBCA6B + s["step"] * 0x9E3779B1) & 0xFFFFFFFF) >> 12).to(torch.int32)


def _dithered(x, u):
    """x >= 0 rounded to E4M3, up where the 20 bits below its last place and u carry."""
    sub = x < 2.0 ** -6
    y = torch.where(sub, x + 2.0 ** -6, x)
    r = ((y.view(torch.int32) + u) & ~0xFFFFF).view(torch.float32)
    return torch.where(sub, r - 2.0 ** -6, r).clamp_max(448.0)


def _requantize(t, u, keep):
    """(codes, scales) of float32 [n] in groups of 128; `keep`: what is not zero
    does not become zero."""
    v = t.view(-1, GROUP)
    amax = v.abs().amax(dim=1)
    inv = 448.0 / amax
    flush = ~torch.isfinite(inv)
    inv = torch.where(flush, 0.0, inv)
    x = (v * inv[:, None]).view(-1)
    r = _dithered(x.abs(), u)
    if keep:
        r = torch.where((r == 0) & (x > 0), 2.0 ** -9, r)
    return (torch.where(x < 0, -r, r).to(E4M3).view(torch.uint8),
            torch.where(flush, 0.0, amax / 448.0))


def _plain_adamw(s):
    h, t = s["hyper"], s["step"]
    b1, b2 = h["betas"]
    eight = s["case"]["kind"] == "adamw_8bit"
    g = s["g"].float()
    if s["clip"] is not None:
        g = g * s["clip"]
    if eight:
        m = (s["m_q"].view(E4M3).float().view(-1, GROUP) * s["m_s"][:, None]).view(-1)
        r = (s["v_q"].view(E4M3).float().view(-1, GROUP) * s["v_s"][:, None]).view(-1)
        v = r * r
    else:
        m, v = s["m"], s["v"]
    m = m * b1 + g * (1.0 - b1)
    v = v * b2 + (g * g) * (1.0 - b2)
    root = torch.sqrt(v)
    # the corrections in 64 bits: 1 - beta^t cancels
    c1, c2 = -math.expm1(t * math.log(b1)), math.sqrt(-math.expm1(t * math.log(b2)))
    step = (h["lr"] / c1) * m / (root / c2 + h["eps"])
    s["p"].copy_(s["p"] * (1.0 - h["lr"] * h["weight_decay"]) - step)
    if s["copy"] is not None:
        s["copy"].copy_(s["p"])
    if eight:
        u = _dither(s)
        for name, x, w in (("m", m, u), ("v", root, 0xFFFFF - u)):
            q, sc = _requantize(x, w, name == "v")
            s[name + "_q"].copy_(q)
            s[name + "_s"].copy_(sc)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    return _adamw_outputs(s)


def _adamw_outputs(s):
    out = {"p": s["p"]}
    if s["copy"] is not None:
        out["copy"] = s["copy"]
    if s["case"]["kind"] == "adamw_8bit":
        out.update(m=s["m_q"].view(E4M3), m_s=s["m_s"], v=s["v_q"].view(E4M3), v_s=s["v_s"])
    else:
        out.update(m=s["m"], v=s["v"])
    return out


def _plain(s):
    c = s["case"]
    k = c["kind"]
    if k == "layer_norm":
        y, mean, rstd = _norm(s["x"], s["weight"], s["bias"], s["eps"])
        out = {"mean": mean, "rstd": rstd}
        if c["codes"]:
            out["q"], out["s"] = _groups(y)
        if c["y"]:
            out["y"] = y.to(BF16)
        return out
    if k == "layer_norm_backward":
        return _plain_norm_backward(s)
    if k == "expert_tokens":
        q, sc = _groups(_by_expert(s["x"], s["off"], GROUP * _blocks(c)))
        return {"q": q, "s": sc}
    if k == "expert_wgrad":
        return _plain_wgrad(s)
    return _plain_adamw(s)


def run(state):
    s = state
    if not own:
        return _plain(s)
    import fine_grained_block_fp8q_amd as fq
    c = s["case"]
    k = c["kind"]
    if k == "layer_norm":
        if not c["codes"]:
            y, mean, rstd = fq.layer_norm(s["x"], s["weight"], s["bias"], s["eps"])
            return {"y": y, "mean": mean, "rstd": rstd}
        r = fq.layer_norm_quantized(s["x"], s["weight"], s["bias"], s["eps"], save_y=c["y"])
        out = {"q": r[0].view(E4M3), "s": r[1], "mean": r[2], "rstd": r[3]}
        if c["y"]:
            out["y"] = r[4]
        return out
    if k == "layer_norm_backward":
        dx, dw, db = fq.layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"])
        return {"dx": dx, "dweight": dw, "dbias": db}
    if k == "expert_tokens":
        q, sc = fq.grouped_quantize_act_t(s["x"], s["off"])
        return {"q": q.view(E4M3), "s": sc}
    if k == "expert_wgrad":
        return {"dw": fq.grouped_gemm_rowscaled(s["a_q"], s["a_s"], s["b_q"], s["b_s"], s["off"],
                                                out_dtype=BF16)}
    t = s["tensors"]
    if k == "adamw":
        fq.adamw(t["p"], t["g"], t["m"], t["v"], s["step"], grad_scale=s["clip"],
                 copies=t.get("copy"), **s["hyper"])
    else:
        fq.adamw_8bit(t["p"], t["g"], t["m_q"], t["m_s"], t["v_q"], t["v_s"], s["step"],
                      grad_scale=s["clip"], copies=t.get("copy"), **s["hyper"])
    return _adamw_outputs(s)


# ---------------------------------------------------- the definitions, 64 bits
def _e4m3(v, u=None):
    """float64 -> E4M3 values, |v| <= 448: the nearest (ties to even), or with u in
    [0, 1) the next one up where the fraction of a step and u reach 1."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6)))
    step = torch.exp2(e - 3)
    if u is None:
        return torch.round(v / step) * step
    return torch.sign(v) * torch.floor(v.abs() / step + u) * step


def _exact_codes(v, u=None):
    """E4M3 values [R][n] and scales [R][n/128] of float64 [R][n]."""
    R, n = v.shape
    x = v.reshape(R, n // GROUP, GROUP)
    top = x.abs().amax(dim=2)
    some = top > 0
    x = x * torch.where(some, 448.0 / torch.where(some, top, 1.0), 0.0)[:, :, None]
    return _e4m3(x.reshape(R, n), u), top / 448.0


def _exact_expert_rows(off):
    """(expert, first row, end, first padded column) of each expert."""
    at = 0
    for e in range(len(off) - 1):
        yield e, off[e], off[e + 1], at
        at += -(-(off[e + 1] - off[e]) // GROUP) * GROUP


def exact(case, seed):
    c, s = case, prepare(case, seed)
    k, t = c["kind"], torch.float64
    if k.startswith("layer_norm"):
        x, w = s["x"].to(t), s["weight"].to(t)
        if k == "layer_norm":
            mean = x.sum(dim=1) / c["N"]
            var = ((x - mean[:, None]) ** 2).sum(dim=1) / c["N"]
            rstd = (var + s["eps"]) ** -0.5
            y = (x - mean[:, None]) * rstd[:, None] * w + s["bias"].to(t)
            out = {"mean": mean, "rstd": rstd}
            if c["codes"]:
                out["q"], sc = _exact_codes(y)
                out["s"] = sc.t().contiguous()
            if c["y"]:
                out["y"] = y
            return out
        dy, r = s["dy"].to(t), s["rstd"].to(t)[:, None]
        z = (x - s["mean"].to(t)[:, None]) * r
        gz = dy * w
        dx = r * (gz - gz.sum(1, keepdim=True) / c["N"]
                  - z * ((gz * z).sum(1, keepdim=True) / c["N"]))
        return {"dx": dx, "dweight": (dy * z).sum(0), "dbias": dy.sum(0)}
    if k.startswith("expert"):
        off = s["off"].tolist()
        cols = GROUP * _blocks(c)
        if k == "expert_tokens":
            v = torch.zeros((cols, c["K"]), dtype=t, device=DEV)
            for e, lo, hi, at in _exact_expert_rows(off):
                v[at:at + hi - lo] = s["x"][lo:hi].to(t)
            q, sc = _exact_codes(v.t().contiguous())
            return {"q": q, "s": sc.t().contiguous()}
        dw = torch.zeros((c["G"], c["N"], c["K"]), dtype=t, device=DEV)
        for e, lo, hi, at in _exact_expert_rows(off):
            end = at + -(-(hi - lo) // GROUP) * GROUP
            if hi > lo:
                a, b = (s[n + "_q"][:, at:end].contiguous().view(E4M3).to(t)
                        * s[n + "_s"][at // GROUP:end // GROUP].t().to(t).repeat_interleave(GROUP, 1)
                        for n in "ab")
                dw[e] = a @ b.t().contiguous()
        return {"dw": dw}
    h, n = s["hyper"], s["step"]
    b1, b2 = h["betas"]
    g = s["g"].to(t) * (s["clip"].to(t) if s["clip"] is not None else 1.0)
    if k == "adamw":
        m, v = s["m"].to(t), s["v"].to(t)
    else:
        m = s["m_q"].view(E4M3).to(t) * s["m_s"].to(t).repeat_interleave(GROUP)
        v = (s["v_q"].view(E4M3).to(t) * s["v_s"].to(t).repeat_interleave(GROUP)) ** 2
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    p = s["p"].to(t)
    p = p - h["lr"] * h["weight_decay"] * p \
        - h["lr"] * (m / (1 - b1 ** n)) / (torch.sqrt(v / (1 - b2 ** n)) + h["eps"])
    out = {"p": p}
    if s["copy"] is not None:
        out["copy"] = p
    if k == "adamw":
        out.update(m=m, v=v)
        return out
    place = torch.empty(p.numel(), dtype=torch.int64, device=DEV)
    for at, end in zip(s["starts"][:-1].tolist(), s["starts"][1:].tolist()):
        place[at:end] = torch.arange(end - at, device=DEV)
    u = torch.div((place * 0x85EBCA6B + n * 0x9E3779B1) % 2 ** 32, 4096, rounding_mode="floor")
    for name, x, w in (("m", m, u), ("v", v.sqrt(), 2 ** 20 - 1 - u)):
        q, sc = _exact_codes(x.view(1, -1), w.to(t).view(1, -1) / 2 ** 20)
        if name == "v":
            q = torch.where((q == 0) & (x.view(1, -1) > 0), 2.0 ** -9, q)
        out[name], out[name + "_s"] = q.view(-1), sc.view(-1)
    return out
