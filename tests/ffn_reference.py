"""64-bit references of the feed-forward sublayer's operators (gated block,
backward passes, layer norm) and the seeded inputs their tests share.

Weights and activations are FP8 codes with float32 scales, as the operators
take them; the codes are decoded through torch's own float8 types.
"""
import math

import torch

FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
BF16_HALF_STEP = 2.0 ** -8      # finfo(bfloat16).eps / 2: one rounding, relative


def decode(codes, fmt):
    """uint8 FP8 codes -> float64."""
    return codes.view(FP8[fmt][0]).double()


def quantise_rows(x, fmt):
    """Row-wise codes (uint8) and scales of a float tensor (the library's rule)."""
    amax = x.float().abs().amax(1).clamp_min(1e-12)
    s = amax / torch.full_like(amax, FP8[fmt][1])
    return (x.float() / s[:, None]).to(FP8[fmt][0]).view(torch.uint8), s


def gen(seed, device="cuda"):
    return torch.Generator(device).manual_seed(seed)


def sparse_weight(rows, k, seed, scale=0.02):
    """A [rows, k] bf16 weight with two non-zeros in each group of four."""
    g = gen(seed)
    w = torch.randn(rows, k // 4, 4, device="cuda", generator=g) * scale
    w.scatter_(2, w.abs().argsort(dim=2, stable=True)[:, :, :2], 0.0)
    return w.view(rows, k).to(torch.bfloat16)


def act(g, name):
    """The activation and its derivative, in g's precision."""
    if name == "silu":
        p = torch.sigmoid(g)
        return g * p, p * (1 + g * (1 - p))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 0.134145 * g * g)


def linear_parts(a, s_a, w, s_w, bias=None):
    """z = (a w^T) s_a s_w + bias in 64 bits, and the sum of the products' magnitudes."""
    scale = s_a.double()[:, None] * s_w.double()[None, :]
    z = (a @ w.t()) * scale
    size = (a.abs() @ w.abs().t()) * scale
    if bias is not None:
        z = z + bias.double()
    return z, size


def gated_reference(a, s_a, w_rows, s_w, bias, name):
    """Gate, up and h in 64 bits from the alternating rows, and the bound of
    |h - h_ref|: bias is gate's n values, then up's."""
    n = w_rows.shape[0] // 2
    b = None
    if bias is not None:
        b = torch.stack((bias[:n], bias[n:]), 1).reshape(-1)
    z, size = linear_parts(a, s_a, w_rows, s_w, b)
    gate, up = z[:, 0::2], z[:, 1::2]
    f, _ = act(gate, name)
    h = f * up
    # fp32 accumulation of z: 1e-3 of the products' size covers the tensor
    # core's sums (the linear's own tolerance); |act'| <= 1.13 for both
    # activations, |act(g)| <= |g|.  The fast logistic adds 2^-18, h is
    # rounded once.
    dz = 1e-3 * size
    dg, du = dz[:, 0::2], dz[:, 1::2]
    bound = 1.13 * dg * (up.abs() + du) + (f.abs() + 1.13 * dg) * du
    return gate, up, h, bound + (BF16_HALF_STEP + 2.0 ** -18) * (h.abs() + bound) + 1e-37


def backward_reference(dz, dz_err, a, s_a, w, s_w):
    """dx, dw, db in 64 bits from dz (its own error bound dz_err), each with
    the bound of its difference: the expanded operands are rounded to bf16
    once, the fp32 sums err by well under 2^-12 of the products' size, the
    result is rounded once."""
    ws = w * s_w.double()[:, None]
    xs = a * s_a.double()[:, None]
    out = []
    for p, e, q in ((dz, dz_err, ws), (dz.t(), dz_err.t(), xs)):
        ref = p @ q
        size = (BF16_HALF_STEP + 2.0 ** -12) * (p.abs() @ q.abs()) + 1.01 * (e @ q.abs())
        out.append((ref, size + BF16_HALF_STEP * (ref.abs() + size) + 1e-37))
    ref = dz.sum(0)
    size = 2.0 ** -12 * dz.abs().sum(0) + dz_err.sum(0)
    out.append((ref, size + BF16_HALF_STEP * (ref.abs() + size) + 1e-37))
    return out


def gated_grad_reference(dh, gate, up, z_err, name):
    """dz (alternating columns) in 64 bits and its error bound: gate and up err
    by z_err, act and act' have slopes of at most 1.13 and 0.8 (SiLU's second
    derivative is at most 1/2, GELU's below 0.8), dz is rounded once."""
    f, df = act(gate, name)
    dg, du = z_err[:, 0::2], z_err[:, 1::2]
    d = dh.double()
    dgate, dup = d * up * df, d * f
    e_gate = d.abs() * (du * (df.abs() + 0.8 * dg) + up.abs() * 0.8 * dg + 2.0 ** -18 * up.abs())
    e_up = d.abs() * (1.13 * dg + 2.0 ** -18 * f.abs())
    dz = torch.stack((dgate, dup), 2).reshape(dh.shape[0], -1)
    err = torch.stack((e_gate, e_up), 2).reshape(dh.shape[0], -1)
    return dz, err + BF16_HALF_STEP * (dz.abs() + err) + 1e-37
