"""Cases of the 8-bit feed-forward operators, for measurement.

Every case is one call path of the feed-forward layer:

  i8_product      C = (A_q W_q^T) * a_s * w_s (+ bias): 8-bit integers, one scale
                  per token and one per output channel
  i8_linear       the same from BF16 activations: quantized per token, then multiplied
  i8_gated        h = act(gate) * up, [gate | up] the integer product above with
                  gate and up weights stacked
  gated           the gated block on fine-grained block-scaled E4M3 operands
                  (1x128 activation groups, 128x128 weight blocks)
  gated_grouped   the same for routed experts, rows grouped by expert
  gated_backward  [dgate | dup] from dh and the saved [gate | up], quantized to E4M3
                  in 1x128 groups along the features (the operand of the input
                  gradient) and along the tokens (the operand of the weight gradient)

`own` chooses between the plain form (elementary torch operations in float32)
and the framework's operators.  exact() evaluates the definitions in float64.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # One token of a chat session through a 4096 x 7168 projection: latency counts.
        {"name": "i8 product, 1 token", "kind": "i8_product", "M": 1, "N": 4096, "K": 7168,
         "bias": False, "out": "bf16"},
        # A ragged batch through a narrow head with a bias: no size is a power of two.
        {"name": "i8 product, ragged, bias", "kind": "i8_product", "M": 777, "N": 1001, "K": 2000,
         "bias": True, "out": "f32"},
        # A decoding batch of 16 sessions from BF16, a hidden size that is not a multiple of 16.
        {"name": "i8 linear, 16 tokens, odd K", "kind": "i8_linear", "M": 16, "N": 7168, "K": 2043,
         "out": "bf16"},
        # A prompt of 4096 tokens from BF16 activations, quantized on the way.
        {"name": "i8 linear, 4096 tokens", "kind": "i8_linear", "M": 4096, "N": 4096, "K": 7168,
         "out": "bf16"},
        # Gate and up projection of a served block, 32 sessions decoding together.
        {"name": "i8 gated, 32 tokens", "kind": "i8_gated", "M": 32, "F": 2048, "K": 7168,
         "act": "silu"},
        # A large prefill batch through a wider block with a tanh-GELU gate.
        {"name": "i8 gated, 8192 tokens", "kind": "i8_gated", "M": 8192, "F": 4096, "K": 7168,
         "act": "gelu_tanh"},
        # One token through a block-scaled E4M3 gated block.
        {"name": "gated, 1 token", "kind": "gated", "M": 1, "F": 2048, "K": 7168, "act": "silu",
         "save": False},
        # A training step's forward: the pre-activations are kept for the backward pass.
        {"name": "gated, 4096 tokens, saved", "kind": "gated", "M": 4096, "F": 2048, "K": 7168,
         "act": "silu", "save": True},
        # A decoding step over 32 resident experts, from no rows to 256 each.
        {"name": "gated experts, decode", "kind": "gated_grouped", "G": 32, "rows": 4300,
         "cap": 256, "F": 2048, "K": 7168, "act": "silu"},
        # 4096 tokens routed to 8 of 256 experts each.
        {"name": "gated experts, 256", "kind": "gated_grouped", "G": 256, "rows": 32768,
         "cap": 256, "F": 2048, "K": 7168, "act": "silu"},
        # A training step's backward through the activation, a batch that is not
        # a multiple of the 128-token groups.
        {"name": "gated backward, 4000 tokens", "kind": "gated_backward", "M": 4000, "F": 2048,
         "act": "silu"},
        # A small batch with a tanh-GELU gate.
        {"name": "gated backward, 200 tokens", "kind": "gated_backward", "M": 200, "F": 1408,
         "act": "gelu_tanh"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cap(c):
    """Whether a drawn case costs no more than the largest listed ones."""
    w = work(c)
    return w["flops"] <= 1e12 and w["bytes"] <= 2.5e9


def draw(rng):
    while True:
        kind = rng.choice(["i8_product", "i8_linear", "i8_gated", "gated", "gated_grouped",
                           "gated_backward"])
        act = rng.choice(["silu", "gelu_tanh"])
        M = _log(rng, 1, 8192)
        if kind == "i8_product":
            c = {"kind": kind, "M": M, "N": _log(rng, 64, 8192), "K": 16 * _log(rng, 8, 512),
                 "bias": rng.random() < 0.5, "out": rng.choice(["bf16", "f32"])}
        elif kind == "i8_linear":
            c = {"kind": kind, "M": M, "N": _log(rng, 64, 8192), "K": _log(rng, 128, 8192),
                 "out": rng.choice(["bf16", "f32"])}
        elif kind == "i8_gated":
            c = {"kind": kind, "M": M, "F": _log(rng, 64, 4096), "K": 16 * _log(rng, 8, 512),
                 "act": act}
        elif kind == "gated":
            c = {"kind": kind, "M": M, "F": 128 * _log(rng, 1, 32), "K": 128 * _log(rng, 1, 56),
                 "act": act, "save": rng.random() < 0.5}
        elif kind == "gated_grouped":
            G = _log(rng, 2, 64)
            c = {"kind": kind, "G": G, "rows": G * _log(rng, 1, 200), "cap": 256,
                 "F": 128 * _log(rng, 1, 16), "K": 128 * _log(rng, 1, 56), "act": act}
        else:
            c = {"kind": kind, "M": M, "F": 128 * _log(rng, 1, 32), "act": act}
        if _cap(c):
            return c


def work(c):
    k = c["kind"]
    if k == "gated_backward":
        M, F = c["M"], c["F"]
        Mp = -(-M // 128) * 128
        # dh and [gate | up] in; codes along both axes out, and their scales
        return {"bytes": 6 * M * F + 2 * F * (M + Mp) + 8 * F / 128 * M + 8 * F * Mp / 128,
                "flops": 20 * M * F}
    if k in ("i8_product", "i8_linear"):
        M, N, K = c["M"], c["N"], c["K"]
        ob = 2 if c["out"] == "bf16" else 4
        act = M * K if k == "i8_product" else 2 * M * K + M * K
        return {"bytes": act + N * K + 4 * (M + N) + ob * M * N, "flops": 2 * M * N * K}
    if k == "i8_gated":
        M, F, K = c["M"], c["F"], c["K"]
        return {"bytes": M * K + 2 * F * K + 4 * (M + 2 * F) + 2 * M * F, "flops": 4 * M * F * K}
    if k == "gated":
        M, F, K = c["M"], c["F"], c["K"]
        out = 2 * M * F * (3 if c["save"] else 1)
        return {"bytes": (M * K) * (1 + 4 / 128) + 2 * F * K + out, "flops": 4 * M * F * K}
    G, R, F, K = c["G"], c["rows"], c["F"], c["K"]
    return {"bytes": R * K * (1 + 4 / 128) + G * 2 * F * K + 2 * R * F, "flops": 4 * R * F * K}


# ------------------------------------------------------------- making inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _activations(g, M, K):
    """BF16 activations: N(0, 1), one channel in a hundred 30 times as large."""
    x = torch.randn((M, K), generator=g, device=DEV)
    big = torch.rand(K, generator=g, device=DEV) < 0.01
    return (x * torch.where(big, 30.0, 1.0)).to(torch.bfloat16)


def _tokens_i8(x):
    """Per-row symmetric quantization: s = amax/127, q = round(x * (127/amax)),
    rows padded with zeros to a multiple of 16."""
    x = x.float()
    amax = x.abs().amax(dim=1)
    inv = 127.0 / amax
    flush = ~torch.isfinite(inv)
    inv = torch.where(flush, 0.0, inv)
    q = torch.round(x * inv[:, None]).clamp(-127, 127).to(torch.int8)
    pad = -x.shape[1] % 16
    if pad:
        q = torch.nn.functional.pad(q, (0, pad))
    return q, torch.where(flush, 0.0, amax / 127.0)


def _groups_e4m3(x):
    """1x128 groups along the last axis: (E4M3 values, scales [K/128][M])."""
    M, K = x.shape
    v = x.float().reshape(M, K // 128, 128)
    amax = v.abs().amax(dim=2)
    inv = 448.0 / amax
    flush = ~torch.isfinite(inv)
    inv = torch.where(flush, 0.0, inv)
    q = (v * inv[:, :, None]).to(E4M3).reshape(M, K)
    return q, torch.where(flush, 0.0, amax / 448.0).t().contiguous()


def _blocks_e4m3(w):
    """128x128 blocks of [..., N, K]: (E4M3 values, scales [..., N/128, K/128])."""
    N, K = w.shape[-2:]
    v = w.float().reshape(*w.shape[:-2], N // 128, 128, K // 128, 128)
    amax = v.abs().amax(dim=(-3, -1))
    q = (v * (448.0 / amax)[..., :, None, :, None]).to(E4M3)
    return q.reshape(w.shape), amax / 448.0


def _counts(seed, G, rows, cap):
    """Rows of each expert: random shares of `rows`, none above `cap`, some empty."""
    r = np.random.default_rng([int(seed), 77])
    share = r.gamma(4.0, 1.0, G) * (r.random(G) > 0.04)
    if share.sum() == 0:
        share[:] = 1.0
    n = np.minimum(np.floor(share / share.sum() * rows), cap).astype(np.int64)
    left = rows - int(n.sum())
    while left > 0:
        at = np.flatnonzero(n < cap)
        take = r.permutation(at)[:left]
        n[take] += 1
        left -= len(take)
    return n


def prepare(case, seed):
    c, g = case, _gen(seed)
    k = c["kind"]
    s = {"case": c}
    if k == "gated_backward":
        M, F = c["M"], c["F"]
        s["dh"] = (0.01 * torch.randn((M, F), generator=g, device=DEV)).to(torch.bfloat16)
        s["gu"] = (2.0 * torch.randn((M, 2 * F), generator=g, device=DEV)).to(torch.bfloat16)
        return s
    K = c["K"]
    if k.startswith("i8"):
        N = c["N"] if "N" in c else 2 * c["F"]
        w = 0.02 * torch.randn((N, K), generator=g, device=DEV)
        s["w_q"], s["w_s"] = _tokens_i8(w.to(torch.bfloat16))
        x = _activations(g, c["M"], K)
        if k == "i8_linear":
            s["x"] = x
        else:
            s["a_q"], s["a_s"] = _tokens_i8(x)
        s["bias"] = torch.randn(N, generator=g, device=DEV) if c.get("bias") else None
        return s
    F = c["F"]
    if k == "gated":
        w = 0.02 * torch.randn((2 * F, K), generator=g, device=DEV)
        q, s["w_s"] = _blocks_e4m3(w.to(torch.bfloat16))
        rows = c["M"]
    else:
        G = c["G"]
        q = torch.empty((G, 2 * F, K), dtype=E4M3, device=DEV)
        s["w_s"] = torch.empty((G, 2 * F // 128, K // 128), device=DEV)
        step = max(1, (1 << 29) // (2 * F * K))
        for e in range(0, G, step):
            n = min(step, G - e)
            w = 0.02 * torch.randn((n, 2 * F, K), generator=g, device=DEV)
            q[e:e + n], s["w_s"][e:e + n] = _blocks_e4m3(w.to(torch.bfloat16))
        rows = c["rows"]
        off = np.zeros(G + 1, dtype=np.int32)
        off[1:] = np.cumsum(_counts(seed, G, rows, c["cap"]))
        s["off"] = torch.from_numpy(off).to(DEV)
    s["w_q"] = q.view(torch.uint8)
    aq, s["a_s"] = _groups_e4m3(_activations(g, rows, K))
    s["a_q"] = aq.view(torch.uint8)
    return s


# ------------------------------------------------------------ the plain forms
_GELU_A = math.sqrt(2.0 / math.pi)
_GELU_B = 0.044715


def _act(g, act):
    if act == "silu":
        return g / (1.0 + torch.exp(-g))
    return 0.5 * g * (1.0 + torch.tanh(_GELU_A * (g + _GELU_B * g * g * g)))


def _act_grad(g, act):
    if act == "silu":
        t = 1.0 / (1.0 + torch.exp(-g))
        return t * (1.0 + g * (1.0 - t))
    t = torch.tanh(_GELU_A * (g + _GELU_B * g * g * g))
    return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * _GELU_A * (1.0 + 3.0 * _GELU_B * g * g)


def _gate(y, F, act):
    return _act(y[..., :F], act) * y[..., F:]


def _i8_matmul(a_q, a_s, w_q, w_s, t=torch.float32):
    return (a_q.to(t) @ w_q.to(t).t()) * a_s.to(t)[:, None] * w_s.to(t)[None, :]


def _rows_of(codes, scales, t=torch.float32):
    """E4M3 codes [M][K] with scales [K/128][M], as values."""
    M, K = codes.shape
    v = codes.view(E4M3).to(t).reshape(M, K // 128, 128)
    return (v * scales.to(t).t()[:, :, None]).reshape(M, K)


def _blocks_of(codes, scales, t=torch.float32):
    """E4M3 codes [..., N, K] with scales [..., N/128, K/128], as values."""
    N, K = codes.shape[-2:]
    v = codes.view(E4M3).to(t).reshape(*codes.shape[:-2], N // 128, 128, K // 128, 128)
    return (v * scales.to(t)[..., :, None, :, None]).reshape(codes.shape)


def _out(v, out):
    return v.to(torch.bfloat16) if out == "bf16" else v


def _plain(s):
    c = s["case"]
    k = c["kind"]
    if k == "i8_product":
        y = _i8_matmul(s["a_q"], s["a_s"], s["w_q"], s["w_s"])
        if s["bias"] is not None:
            y = y + s["bias"]
        return _out(y, c["out"])
    if k == "i8_linear":
        q, a_s = _tokens_i8(s["x"])
        return {"q": q, "s": a_s, "c": _out(_i8_matmul(q, a_s, s["w_q"], s["w_s"]), c["out"])}
    if k == "i8_gated":
        y = _i8_matmul(s["a_q"], s["a_s"], s["w_q"], s["w_s"])
        return _gate(y, c["F"], c["act"]).to(torch.bfloat16)
    if k == "gated":
        y = _rows_of(s["a_q"], s["a_s"]) @ _blocks_of(s["w_q"], s["w_s"]).t()
        h = _gate(y, c["F"], c["act"]).to(torch.bfloat16)
        return {"h": h, "gu": y.to(torch.bfloat16)} if c["save"] else {"h": h}
    if k == "gated_grouped":
        # every expert's rows padded to `cap`, one batched product W A^T
        off = s["off"].long()
        row = torch.arange(c["cap"], device=DEV)
        n = off[1:] - off[:-1]
        live = row[None, :] < n[:, None]
        at = torch.where(live, off[:-1, None] + row[None, :], 0)
        a = _rows_of(s["a_q"], s["a_s"])
        y = torch.bmm(_blocks_of(s["w_q"], s["w_s"]), a[at].transpose(1, 2).contiguous())
        F = c["F"]
        h = _act(y[:, :F], c["act"]) * y[:, F:]
        return {"h": h.transpose(1, 2)[live].to(torch.bfloat16)}
    return _plain_backward(s["dh"].float(), s["gu"].float(), c)


def _plain_backward(dh, gu, c):
    F, M = c["F"], c["M"]
    g, u = gu[:, :F], gu[:, F:]
    dy = torch.cat([dh * u * _act_grad(g, c["act"]), dh * _act(g, c["act"])], dim=1)
    q, sc = _groups_e4m3(dy)
    pad = -M % 128
    qt, st = _groups_e4m3(torch.nn.functional.pad(dy, (0, 0, 0, pad)).t())
    return {"q": q, "s": sc, "qt": qt, "st": st}


def run(state):
    s = state
    if not own:
        return _plain(s)
    import fine_grained_block_fp8q_amd as fq
    c = s["case"]
    k = c["kind"]
    out = torch.bfloat16 if c.get("out", "bf16") == "bf16" else torch.float32
    if k == "i8_product":
        return fq.gemm_i8(s["a_q"], s["a_s"], s["w_q"], s["w_s"], bias=s["bias"], out_dtype=out)
    if k == "i8_linear":
        q, a_s = fq.quantize_token_i8(s["x"])
        return {"q": q, "s": a_s, "c": fq.gemm_i8(q, a_s, s["w_q"], s["w_s"], out_dtype=out)}
    if k == "i8_gated":
        return fq.gemm_i8_gated(s["a_q"], s["a_s"], s["w_q"], s["w_s"], act=c["act"])
    if k == "gated":
        if c["save"]:
            h, gu = fq.gemm_gated(s["a_q"], s["a_s"], s["w_q"], s["w_s"], act=c["act"],
                                  save_gate_up=True)
            return {"h": h, "gu": gu}
        return {"h": fq.gemm_gated(s["a_q"], s["a_s"], s["w_q"], s["w_s"], act=c["act"])}
    if k == "gated_grouped":
        return {"h": fq.grouped_gemm_gated(s["a_q"], s["a_s"], s["off"], s["w_q"], s["w_s"],
                                           act=c["act"])}
    q, sc, qt, st = fq.gated_backward(s["dh"], s["gu"], act=c["act"])
    return {"q": q.view(E4M3), "s": sc, "qt": qt.view(E4M3), "st": st}


# ---------------------------------------------------- the definitions, 64 bits
def _e4m3_round(v):
    """float64 -> the nearest E4M3 value (ties to even), |v| <= 448."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(v / step) * step


def _exact_groups(v):
    """E4M3 values and scales of groups of 128 along the last axis of [R][n]."""
    R, n = v.shape
    x = v.reshape(R, n // 128, 128)
    top = x.abs().amax(dim=2)
    some = top > 0
    mul = torch.where(some, 448.0 / torch.where(some, top, 1.0), 0.0)
    return _e4m3_round(x * mul[:, :, None]).reshape(R, n), (top / 448.0).t().contiguous()


def _exact_gate(gate, up, act):
    if act == "silu":
        return gate * torch.sigmoid(gate) * up
    z = math.sqrt(2.0 / math.pi) * (gate + 0.044715 * gate ** 3)
    return gate * torch.sigmoid(2.0 * z) * up


def exact(case, seed):
    c, s = case, prepare(case, seed)
    k, t = c["kind"], torch.float64
    if k == "gated_backward":
        M, F, dh = c["M"], c["F"], s["dh"].double()
        g, u = s["gu"][:, :F].double(), s["gu"][:, F:].double()
        if c["act"] == "silu":
            sg = torch.sigmoid(g)
            a, da = g * sg, sg + g * sg * torch.sigmoid(-g)
        else:
            z = math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)
            dz = math.sqrt(2.0 / math.pi) * (1.0 + 3 * 0.044715 * g * g)
            sg = torch.sigmoid(2.0 * z)
            a, da = g * sg, sg + g * 2.0 * dz * sg * torch.sigmoid(-2.0 * z)
        dy = torch.empty((-(-M // 128) * 128, 2 * F), dtype=t, device=DEV).zero_()
        dy[:M, :F] = dh * u * da
        dy[:M, F:] = dh * a
        q, sc = _exact_groups(dy[:M])
        qt, st = _exact_groups(dy.t().contiguous())
        return {"q": q, "s": sc, "qt": qt, "st": st}
    if k == "i8_linear":
        # the codes are whole numbers, held to the plain form's; the product is
        # taken of the codes the rule gives in 64 bits from the same 32-bit multiplier
        x = s["x"].double()
        top = x.abs().amax(dim=1)
        mul = (127.0 / top.float()).double()
        q = torch.round((x * mul[:, None]).float().double())
        y = (q @ s["w_q"][:, :c["K"]].double().t()) * (top / 127.0)[:, None] * s["w_s"].double()
        return {"q": None, "s": top / 127.0, "c": y}
    if k.startswith("i8"):
        y = (s["a_q"].double() @ s["w_q"].double().t()) * s["a_s"].double()[:, None] \
            * s["w_s"].double()
        if k == "i8_gated":
            return _exact_gate(y[:, :c["F"]], y[:, c["F"]:], c["act"])
        return y if s["bias"] is None else y + s["bias"].double()
    F, K = c["F"], c["K"]
    a = s["a_q"].view(E4M3).to(t) * s["a_s"].t().to(t).repeat_interleave(128, dim=1)

    def weights(q, sc):
        return q.view(E4M3).to(t) * sc.to(t).repeat_interleave(128, 0).repeat_interleave(128, 1)
    if k == "gated":
        y = a @ weights(s["w_q"], s["w_s"]).t()
        h = _exact_gate(y[:, :F], y[:, F:], c["act"])
        return {"h": h, "gu": y} if c["save"] else {"h": h}
    off = s["off"].tolist()
    h = torch.empty((c["rows"], F), dtype=t, device=DEV)
    for e in range(c["G"]):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            y = a[lo:hi] @ weights(s["w_q"][e], s["w_s"][e]).t()
            h[lo:hi] = _exact_gate(y[:, :F], y[:, F:], c["act"])
    return {"h": h}
