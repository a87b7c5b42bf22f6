"""Speed cases of the feed-forward sublayer's training and serving operators.

Five operators: the gated feed-forward projection over 2:4 FP8 weights
(forward from the activation, which also returns its 8-bit checkpoint),
its backward pass from that checkpoint, the sparse linear's backward pass
from its checkpoint, and layer norm's forward (straight to FP8 codes, or to
the activation type) and backward passes.

Where ``own`` is false, ``run`` computes them with elementary torch operations
in 32 bits; where it is true, through the package's calls.
"""

import math

import torch

own = False

FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
WIDE = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-5


def listed():
    return [
        # one new token of a served model: gate and up of an 8B model's MLP
        dict(name="gated_decode", op="gated", m=1, n=14336, k=4096, x="bf16", a="e4m3",
             w="e4m3", act="silu", bias=False),
        # a ragged batch through a narrow, odd-width block with every option
        dict(name="gated_ragged", op="gated", m=333, n=5001, k=1408, x="f16", a="e5m2",
             w="e4m3", act="gelu", bias=True),
        # prompt processing, and the forward pass of a training step
        dict(name="gated_prefill", op="gated", m=8192, n=14336, k=4096, x="bf16", a="e4m3",
             w="e4m3", act="silu", bias=False),
        # a small fine-tuning step with biases
        dict(name="gated_backward_small", op="gated_backward", m=250, n=2820, k=1024, a="e4m3",
             w="e4m3", act="gelu", bias=True),
        # the backward pass of a training step at full width
        dict(name="gated_backward_large", op="gated_backward", m=8192, n=14336, k=4096, a="e4m3",
             w="e4m3", act="silu", bias=False),
        # the attention output projection's backward pass
        dict(name="linear_backward", op="linear_backward", m=2048, n=4096, k=4096, a="e4m3",
             w="e4m3", bias=False),
        # odd widths, biases and the other formats
        dict(name="linear_backward_ragged", op="linear_backward", m=777, n=1003, k=1536, a="e5m2",
             w="e5m2", bias=True),
        # the norm before a served model's projections, one step of a batch
        dict(name="norm_decode", op="norm", rows=16, cols=4096, x="bf16", q="e4m3"),
        # the norm before the projections of a prompt or a training step
        dict(name="norm_prefill", op="norm", rows=8192, cols=4096, x="bf16", q="e4m3"),
        # a norm kept in the activation's type, odd width
        dict(name="norm_odd", op="norm", rows=1000, cols=1003, x="f32", q=""),
        # a training step's norm
        dict(name="norm_backward", op="norm_backward", rows=8192, cols=4096, x="bf16"),
        # a small step, odd width
        dict(name="norm_backward_odd", op="norm_backward", rows=777, cols=1003, x="f32"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated", "gated_backward", "linear_backward", "norm", "norm_backward"])
    if op in ("norm", "norm_backward"):
        q = rng.choice(["", "e4m3", "e5m2"]) if op == "norm" else ""
        cols = 16 * _spread(rng, 4, 512) if q else _spread(rng, 1, 8192)
        rows = _spread(rng, 1, 8192)
        case = dict(op=op, rows=rows, cols=cols, x=rng.choice(list(WIDE)))
        if op == "norm":
            case["q"] = q
        # no larger than the largest listed
        while case["rows"] * case["cols"] * BYTES[case["x"]] > 8192 * 4096 * 2:
            case["rows"] = max(1, case["rows"] // 2)
        return case
    case = dict(op=op, m=_spread(rng, 1, 8192), n=_spread(rng, 100, 14336),
                k=128 * _spread(rng, 2, 64), a=rng.choice(list(FP8)), w=rng.choice(list(FP8)),
                bias=rng.random() < 0.5)
    if op == "gated":
        case["x"] = rng.choice(list(WIDE))
    if op != "linear_backward":
        case["act"] = rng.choice(["silu", "gelu"])
    while case["n"] * case["k"] > 14336 * 4096:
        case["n"] = max(100, case["n"] // 2)
    return case


def work(case):
    op = case["op"]
    if op in ("norm", "norm_backward"):
        r, c, b = case["rows"], case["cols"], BYTES[case["x"]]
        if op == "norm":
            return {"bytes": r * c * (b + (1 if case["q"] else b)) + 2 * c * b + r * 12,
                    "flops": 8 * r * c}
        return {"bytes": 3 * r * c * b + c * b + 8 * c + r * 8, "flops": 14 * r * c}
    m, n, k = case["m"], case["n"], case["k"]
    rows = n if op == "linear_backward" else 2 * n
    weight = rows * k * 5 // 8 + 4 * rows   # kept codes, index nibbles, scales
    if op == "gated":
        return {"bytes": m * k * (BYTES[case["x"]] + 1) + 4 * m + weight + 2 * m * n,
                "flops": m * rows * k}       # the kept half of the products
    saved = m * k + 4 * m
    grads = 2 * m * k + 2 * rows * k
    dgrad, wgrad = m * rows * k, 2 * m * rows * k
    if op == "gated_backward":
        # gate and up are computed again from the checkpoint
        return {"bytes": 2 * m * n + saved + weight + grads, "flops": m * rows * k + dgrad + wgrad}
    return {"bytes": 2 * m * rows + saved + weight + grads, "flops": dgrad + wgrad}


# ------------------------------------------------------------------ inputs


def _quantise_rows(x, fmt):
    dtype, top = FP8[fmt]
    amax = x.float().abs().amax(1).clamp_min(1e-12)
    # a tensor divisor: divided, where a Python number would be multiplied by its reciprocal
    s = amax / torch.full_like(amax, top)
    return (x.float() / s[:, None]).to(dtype), s


def _weight(rows, k, fmt, gen):
    """FP8 codes [rows, k] of a normal weight with two kept of each four, and the row scales."""
    w = torch.randn(rows, k // 4, 4, device="cuda", generator=gen) * 0.02
    drop = w.abs().argsort(dim=2, stable=True)[:, :, :2]
    w.scatter_(2, drop, 0.0)
    return _quantise_rows(w.view(rows, k), fmt)


def _inputs(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    op = case["op"]
    if op in ("norm", "norm_backward"):
        r, c, t = case["rows"], case["cols"], WIDE[case["x"]]
        x = (normal(r, c) * (0.5 + normal(r, 1).abs()) + 0.3 * normal(r, 1) + 0.1).to(t)
        d = dict(x=x, weight=(1 + 0.1 * normal(c)).to(t), bias=(0.1 * normal(c)).to(t))
        if op == "norm_backward":
            x64 = x.double()
            mean = x64.mean(1)
            rstd = 1 / ((x64 - mean[:, None]).square().mean(1) + EPS).sqrt()
            d.update(mean=mean.float(), rstd=rstd.float(), dy=normal(r, c).to(t))
        return d
    m, n, k = case["m"], case["n"], case["k"]
    rows = n if op == "linear_backward" else 2 * n
    # rows of a gated weight alternate: gate 0, up 0, gate 1, up 1, ...
    codes, s_w = _weight(rows, k, case["w"], gen)
    d = dict(codes=codes, s_w=s_w, bias=None)
    if case["bias"]:
        # gate's n values, then up's
        d["bias"] = (0.1 * normal(rows)).to(torch.bfloat16)
    x = normal(m, k)
    x[:, ::97] *= 8     # a few channels of an activation are large
    if op == "gated":
        d["x"] = x.to(WIDE[case["x"]])
    else:
        d["a_q"], d["s_a"] = _quantise_rows(x.to(torch.bfloat16), case["a"])
        d["dy"] = (0.01 * normal(m, n)).to(torch.bfloat16)
    return d


def prepare(case, seed):
    state = dict(case=case, **_inputs(case, seed))
    if own:
        import semi_structured_sparse_rowwise_b200 as S
        state["S"] = S
        if "codes" in state:
            # a program keeps the compressed weight, and a workspace for its token count
            codes = state.pop("codes").view(torch.uint8)
            state["packed"] = S.sfp8_compress_24(codes, case["w"])
            args = (case["m"], case["n"], case["k"], "cuda")
            if case["op"] == "gated":
                state["workspace"] = S.new_gated_quant_workspace(*args)
            elif case["op"] == "gated_backward":
                state["workspace"] = S.new_gated_backward_workspace(*args)
            else:
                state["workspace"] = S.new_linear_backward_workspace(*args)
            if "a_q" in state:
                state["a_q"] = state["a_q"].view(torch.uint8)
        elif case["op"] == "norm_backward":
            state["workspace"] = S.new_layernorm_backward_workspace(case["rows"], case["cols"],
                                                                    "cuda")
    return state


# ------------------------------------------------------------------ one pass


def _own(st):
    S, case = st["S"], st["case"]
    op = case["op"]
    if op == "gated":
        h, a_q, s_a = S.sfp8_gated_linear_quant(
            st["x"], case["a"], st["packed"], case["w"], st["s_w"], case["n"], case["k"],
            act=case["act"], bias=st["bias"], workspace=st["workspace"])
        return h, a_q.view(FP8[case["a"]][0]), s_a
    if op == "gated_backward":
        return S.sfp8_gated_linear_backward(
            st["dy"], st["a_q"], case["a"], st["s_a"], st["packed"], case["w"], st["s_w"],
            case["n"], case["k"], act=case["act"], bias=st["bias"], need_dbias=case["bias"],
            workspace=st["workspace"])
    if op == "linear_backward":
        return S.sfp8_sparse_linear_backward(
            st["dy"], st["a_q"], case["a"], st["s_a"], st["packed"], case["w"], st["s_w"],
            case["n"], case["k"], need_dbias=case["bias"], workspace=st["workspace"])
    if op == "norm":
        if case["q"]:
            q, s, mean, rstd = S.sfp8_layernorm_quant(st["x"], st["weight"], st["bias"], EPS,
                                                      case["q"])
            return q.view(FP8[case["q"]][0]), s, mean, rstd
        return S.sfp8_layernorm(st["x"], st["weight"], st["bias"], EPS)
    return S.sfp8_layernorm_backward(st["dy"], st["x"], st["weight"], st["mean"], st["rstd"],
                                     workspace=st["workspace"])


def _gate_up(codes, s_w, bias, a_q, s_a):
    z = (a_q.float() @ codes.float().t()) * (s_a[:, None] * s_w[None, :])
    gate, up = z[:, 0::2], z[:, 1::2]
    if bias is not None:
        n = gate.shape[1]
        gate, up = gate + bias[:n].float(), up + bias[n:].float()
    return gate, up


def _act(g, act):
    """The activation and its derivative."""
    if act == "silu":
        p = 1 / (1 + torch.exp(-g))
        return g * p, p * (1 + g * (1 - p))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 0.134145 * g * g)


def _linear_grads(dz, codes, s_w, a_q, s_a, need_dbias):
    dx = (dz * s_w[None, :]) @ codes.float()
    dw = dz.t() @ (a_q.float() * s_a[:, None])
    db = dz.sum(0).to(torch.bfloat16) if need_dbias else None
    return dx.to(torch.bfloat16), dw, db


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "gated":
        a_q, s_a = _quantise_rows(st["x"], case["a"])
        g, u = _gate_up(st["codes"], st["s_w"], st["bias"], a_q, s_a)
        return (_act(g, case["act"])[0] * u).to(torch.bfloat16), a_q, s_a
    if op == "gated_backward":
        g, u = _gate_up(st["codes"], st["s_w"], st["bias"], st["a_q"], st["s_a"])
        f, df = _act(g, case["act"])
        dy = st["dy"].float()
        dz = torch.stack((dy * u * df, dy * f), 2).view(case["m"], 2 * case["n"])
        dx, dw, db = _linear_grads(dz, st["codes"], st["s_w"], st["a_q"], st["s_a"], case["bias"])
        if db is not None:
            db = torch.cat((db[0::2], db[1::2]))
        # gate's rows, then up's
        return dx, torch.cat((dw[0::2].to(torch.bfloat16), dw[1::2].to(torch.bfloat16))), db
    if op == "linear_backward":
        dx, dw, db = _linear_grads(st["dy"].float(), st["codes"], st["s_w"], st["a_q"], st["s_a"],
                                   case["bias"])
        return dx, dw.to(torch.bfloat16), db
    x = st["x"].float()
    if op == "norm":
        mean = x.mean(1)
        c = x - mean[:, None]
        rstd = 1 / torch.sqrt((c * c).mean(1) + EPS)
        y = c * rstd[:, None] * st["weight"].float() + st["bias"].float()
        if case["q"]:
            return (*_quantise_rows(y, case["q"]), mean, rstd)
        return y.to(st["x"].dtype), mean, rstd
    dy = st["dy"].float()
    xh = (x - st["mean"][:, None]) * st["rstd"][:, None]
    wdy = dy * st["weight"].float()
    dx = (wdy - wdy.mean(1, keepdim=True) - xh * (wdy * xh).mean(1, keepdim=True))
    dx = (dx * st["rstd"][:, None]).to(st["x"].dtype)
    return dx, (dy * xh).sum(0), dy.sum(0)


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ in 64 bits


def _fp8_values(v, fmt):
    """v rounded to the format's grid (nearest, ties to even, saturating), in 64 bits."""
    bits, low, top = (3, -6, 448.0) if fmt == "e4m3" else (2, -14, 57344.0)
    _, e = torch.frexp(v)
    step = torch.exp2((e - 1).clamp_min(low).double() - bits)
    return ((v / step).round() * step).clamp(-top, top)


def _exact_rows(x, fmt):
    top = 448.0 if fmt == "e4m3" else 57344.0
    s = (x.abs().amax(1).clamp_min(float(torch.tensor(1e-12))) / top).float()
    return _fp8_values((x / s.double()[:, None]).float().double(), fmt), s.double()


def _exact_act(g, act):
    if act == "silu":
        p = torch.sigmoid(g)
        return g * p, p + g * p * (1 - p)
    c = math.sqrt(2 / math.pi)
    inner = c * (g + 0.044715 * g ** 3)
    t = torch.tanh(inner)
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t ** 2) * c * (1 + 3 * 0.044715 * g ** 2)


def exact(case, seed):
    d = _inputs(case, seed)
    op = case["op"]
    if op in ("norm", "norm_backward"):
        x, w = d["x"].double(), d["weight"].double()
        if op == "norm":
            var, mean = torch.var_mean(x, 1, unbiased=False)
            rstd = (var + EPS).rsqrt()
            y = torch.addcmul(d["bias"].double(), (x - mean[:, None]) * rstd[:, None], w)
            if case["q"]:
                return (*_exact_rows(y, case["q"]), mean, rstd)
            return y, mean, rstd
        dy = d["dy"].double()
        rstd = d["rstd"].double()[:, None]
        xh = (x - d["mean"].double()[:, None]) * rstd
        wdy = dy * w
        c = case["cols"]
        dx = rstd / c * (c * wdy - wdy.sum(1, keepdim=True) - xh * (wdy * xh).sum(1, keepdim=True))
        return dx, torch.einsum("rc,rc->c", dy, xh), dy.sum(0)
    w = d["codes"].double().mul_(d["s_w"].double()[:, None])
    if op == "gated":
        codes, s_a = _exact_rows(d["x"].double(), case["a"])
    else:
        codes, s_a = d["a_q"].double(), d["s_a"].double()
    a = codes * s_a[:, None]
    n = case["n"]
    if op != "linear_backward":
        b = torch.zeros(2 * n, device="cuda") if d["bias"] is None else d["bias"]
        gate = torch.addmm(b[:n].double(), a, w[0::2].t())
        up = torch.addmm(b[n:].double(), a, w[1::2].t())
        f, df = _exact_act(gate, case["act"])
        if op == "gated":
            return f * up, codes, s_a
        dy = d["dy"].double()
        dg, du = dy * up * df, dy * f
        db = torch.cat((dg.sum(0), du.sum(0))) if case["bias"] else None
        return dg @ w[0::2] + du @ w[1::2], torch.cat((dg.t() @ a, du.t() @ a)), db
    dy = d["dy"].double()
    return dy @ w, dy.t() @ a, (dy.sum(0) if case["bias"] else None)
