"""GPU tests of layer norm, forward (activation type, FP8 codes) and backward,
against the 64-bit formulas, at every row length class and alignment."""
import pytest
import torch

import semi_structured_sparse_rowwise_b200 as S
from ffn_reference import FP8, gen
from gpu_pipeline import ensure_library, requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]

DTYPES = [torch.bfloat16, torch.float16, torch.float32]
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_library()
    yield
    assert S.sfp8_read_device_status(clear=True) == (0, 0)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def inputs(rows, cols, dtype, seed, p_dtype=None):
    g = gen(seed)
    x = (torch.randn(rows, cols, device="cuda", generator=g) * 2
         + torch.randn(rows, 1, device="cuda", generator=g)).to(dtype)
    p_dtype = dtype if p_dtype is None else p_dtype
    w = (1 + 0.2 * torch.randn(cols, device="cuda", generator=g)).to(p_dtype)
    b = (0.2 * torch.randn(cols, device="cuda", generator=g)).to(p_dtype)
    return x, w, b


def reference(x, w, b, eps=EPS):
    x = x.double()
    mean = x.mean(1, keepdim=True)
    rstd = ((x - mean).square().mean(1, keepdim=True) + eps).rsqrt()
    xh = (x - mean) * rstd
    return xh * w.double() + b.double(), mean, rstd, xh


def stats_bound(x, mean, rstd):
    """Bounds of the fp32 mean's and rstd's difference.  A sum of C values in
    a tree of depth below 64 errs by under 64 half steps of sum |x|; the
    deviations by that of the mean, and the variance by 64 half steps again
    (relative; halved by the square root)."""
    u = 64 * 2.0 ** -24
    e_mean = u * x.double().abs().mean(1, keepdim=True)
    dev = (x.double() - mean).abs().mean(1, keepdim=True)
    e_rstd = rstd * (2 * u + e_mean * rstd * rstd * (dev + e_mean))
    return e_mean, e_rstd


def check_forward(y, mean, rstd, x, w, b, dtype):
    ref, m, r, xh = reference(x, w, b)
    e_m, e_r = stats_bound(x, m, r)
    assert bool(((mean.double()[:, None] - m).abs() <= e_m + 1e-30).all())
    assert bool(((rstd.double()[:, None] - r).abs() <= e_r).all())
    e = (xh.abs() * e_r / r + e_m * r) * w.double().abs() + 4 * 2.0 ** -24 * (
        (xh * w.double()).abs() + b.double().abs())
    off = (y.double() - ref).abs()
    bound = e + half_step(dtype) * (ref.abs() + e) + (6e-8 if dtype == torch.float16 else 0)
    assert bool((off <= bound).all()), float((off / bound).max())
    return ref, e


# widths: one element, odd ones, every vector class, and past the registers
WIDTHS = [1, 2, 7, 8, 33, 256, 520, 1000, 1003, 1024, 2048, 4096, 4100, 5000, 8192, 12288, 16385,
          32768, 36872]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("rows", [1, 5, 300])
def test_forward(rows, cols, dtype):
    x, w, b = inputs(rows, cols, dtype, rows + cols)
    y, mean, rstd = S.sfp8_layernorm(x, w, b, EPS)
    assert y.dtype == dtype
    check_forward(y, mean, rstd, x, w, b, dtype)


# eight rows a SM and more: the persistent kernel, at every class of width and
# with a last row that leaves some row groups short
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [264, 520, 1000, 1024, 1032, 2048, 2056, 3000, 4096, 5000, 8192])
@pytest.mark.parametrize("rows", [1187, 2500])
def test_forward_many_rows(rows, cols, dtype):
    x, w, b = inputs(rows, cols, dtype, rows + cols)
    y, mean, rstd = S.sfp8_layernorm(x, w, b, EPS)
    check_forward(y, mean, rstd, x, w, b, dtype)


def fp8_half_step(v, fmt):
    """Half the spacing of the format's values at magnitude v."""
    bits, low = (3, -6) if fmt == "e4m3" else (2, -14)
    _, e = torch.frexp(v)
    return torch.exp2((e - 1).clamp_min(low).double() - bits - 1)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(r, c) for r in (1, 16, 310)
                                       for c in (16, 48, 512, 1024, 4096, 8208, 16384, 40960)]
                         + [(r, c) for r in (1184, 3001) for c in (528, 1024, 2064, 4096, 7680)])
def test_codes(rows, cols, dtype, fmt):
    x, w, b = inputs(rows, cols, dtype, rows + cols)
    y = torch.empty_like(x)
    q, s, mean, rstd = S.sfp8_layernorm_quant(x, w, b, EPS, fmt, out=y)
    ref, e = check_forward(y, mean, rstd, x, w, b, dtype)
    top = FP8[fmt][1]
    want = ref.abs().amax(1) / top
    assert bool(((s.double() - want).abs() <= e.amax(1) / top + 2.0 ** -22 * want).all())
    # The code is the nearest to the fp32 y over s, so its value is within half
    # a step (at that magnitude) of it; the fp32 y is within e of the 64-bit
    # one.  (Counting codes instead would fail near zero: a y of 1e-9 that
    # cancels weight and bias errs by 1e-7 in fp32, many of e5m2's finest
    # steps.)  2^-22 covers the rounding of the quotient itself.
    sc = s.double()[:, None]
    got = q.view(FP8[fmt][0]).double()
    off = (got * sc - ref).abs()
    assert bool((off <= e + sc * fp8_half_step((ref.abs() + e) / sc, fmt) * (1 + 2.0 ** -19)).all())
    exact = (ref / sc).float().clamp(-top, top).to(FP8[fmt][0]).double()
    assert float((got != exact).double().mean()) < 2e-3 + 2.0 / got.numel()
    # each row reaches the largest code: the scale is the row's own
    assert bool((q.view(FP8[fmt][0]).double().abs().amax(1) == top).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_fp32_and_missing_parameters(dtype):
    x, w, b = inputs(40, 1024, dtype, 3, torch.float32)
    y, mean, rstd = S.sfp8_layernorm(x, w, b, EPS)
    check_forward(y, mean, rstd, x, w, b, dtype)
    one, zero = torch.ones_like(w), torch.zeros_like(b)
    for weight, bias in ((None, b), (w, None), (None, None)):
        y, mean, rstd = S.sfp8_layernorm(x, weight, bias, EPS)
        check_forward(y, mean, rstd, x, one if weight is None else weight,
                      zero if bias is None else bias, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("first,ld", [(0, 1040), (8, 1032), (3, 1031)])
def test_strided_rows(dtype, first, ld):
    rows, cols = 33, 1024
    flat = torch.randn(rows * ld + 16, device="cuda", generator=gen(1)).to(dtype)
    x = flat[first:first + rows * ld].view(rows, ld)[:, :cols]
    _, w, b = inputs(1, cols, dtype, 2)
    y, mean, rstd = S.sfp8_layernorm(x, w, b, EPS)
    check_forward(y, mean, rstd, x, w, b, dtype)
    dy = torch.randn(rows, cols + 5, device="cuda", generator=gen(5)).to(dtype)[:, 5:]
    got = S.sfp8_layernorm_backward(dy, x, w, mean, rstd)
    check_backward(got, dy, x, w, mean, rstd, dtype)


def test_constant_rows_and_large_offsets():
    x = torch.full((3, 256), 5.0, device="cuda")
    x[1] = 0
    w, b = torch.ones(256, device="cuda"), torch.full((256,), 0.25, device="cuda")
    y, mean, rstd = S.sfp8_layernorm(x, w, b, EPS)
    assert bool((y == 0.25).all()) and mean.tolist() == [5.0, 0.0, 5.0]
    q, s, _, _ = S.sfp8_layernorm_quant(x, w, torch.zeros_like(b), EPS)
    assert bool((q & 127 == 0).all())       # an all-zero y: the guard scale
    assert torch.equal(s, torch.full((3,), 1e-12, device="cuda") / torch.full((3,), 448.0,
                                                                              device="cuda"))
    x, w, b = inputs(4, 4096, torch.float32, 7)
    x = x + 1e4                              # the variance about the mean, not of squares
    y, mean, rstd = S.sfp8_layernorm(x, w, b, EPS)
    check_forward(y, mean, rstd, x, w, b, torch.float32)


def check_backward(got, dy, x, w, mean, rstd, dtype):
    d, xd, m, r = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    xh = (xd - m) * r
    g = d * w.double()
    a, c = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    u = 2.0 ** -24
    e_xh = 2 * u * (xd.abs() + m.abs()) * r + 2 * u * xh.abs()
    e_a = 64 * u * g.abs().mean(1, keepdim=True)
    e_c = 64 * u * (g * xh).abs().mean(1, keepdim=True) + (g.abs() * e_xh).mean(1, keepdim=True)
    dx = r * (g - a - xh * c)
    e = r * (e_a + xh.abs() * e_c + e_xh * c.abs()) + 4 * u * r * (g.abs() + a.abs()
                                                                   + (xh * c).abs())
    off = (got[0].double() - dx).abs()
    bound = e + half_step(dtype) * (dx.abs() + e) + (6e-8 if dtype == torch.float16 else 0) + 1e-37
    assert bool((off <= bound).all()), float((off / bound).max())
    # sums over rows: at most rows / groups + groups additions in a chain
    depth = x.shape[0] + 2
    for out, terms, extra in ((got[1], d * xh, (d.abs() * e_xh).sum(0)), (got[2], d, 0)):
        bound = depth * u * terms.abs().sum(0) + extra + 1e-37
        off = (out.double() - terms.sum(0)).abs()
        assert out.dtype == torch.float32 and bool((off <= bound).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [1, 3, 8, 200, 256, 512, 1000, 1003, 1024, 2048, 4096, 4099, 5001,
                                  8192, 9000, 16384])
@pytest.mark.parametrize("rows", [1, 37, 700, 1999])
def test_backward(rows, cols, dtype):
    x, w, b = inputs(rows, cols, dtype, rows + cols)
    _, mean, rstd = S.sfp8_layernorm(x, w, b, EPS)
    dy = torch.randn(rows, cols, device="cuda", generator=gen(4)).to(dtype)
    got = S.sfp8_layernorm_backward(dy, x, w, mean, rstd)
    check_backward(got, dy, x, w, mean, rstd, dtype)


@pytest.mark.parametrize("p_dtype", [torch.float32, None])
def test_backward_with_other_parameters(p_dtype):
    x, w, b = inputs(90, 2048, torch.bfloat16, 3, torch.float32)
    weight = w if p_dtype else None
    _, mean, rstd = S.sfp8_layernorm(x, weight, None, EPS)
    dy = torch.randn(90, 2048, device="cuda", generator=gen(4)).to(torch.bfloat16)
    got = S.sfp8_layernorm_backward(dy, x, weight, mean, rstd)
    check_backward(got, dy, x, w if p_dtype else torch.ones_like(w), mean, rstd, torch.bfloat16)


def test_formula_against_differences():
    """The backward formula is the derivative of the forward one (64 bits)."""
    x, w, b = (t.double() for t in inputs(3, 40, torch.float32, 9))
    dy = torch.randn(3, 40, device="cuda", generator=gen(2)).double()
    _, m, r, xh = reference(x, w, b)
    g = dy * w
    dx = r * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    dw, db = (dy * xh).sum(0), dy.sum(0)
    step = 1e-6
    for i, (grad, v) in enumerate(((dx, torch.randn_like(x)), (dw, torch.randn_like(w)),
                                   (db, torch.randn_like(b)))):
        up = [t + step * v if i == j else t for j, t in enumerate((x, w, b))]
        down = [t - step * v if i == j else t for j, t in enumerate((x, w, b))]
        slope = ((reference(*up)[0] - reference(*down)[0]) * dy).sum() / (2 * step)
        assert abs(slope - (grad * v).sum()) <= 1e-6 * (1 + abs(slope))


def test_no_rows():
    x, w, b = inputs(0, 64, torch.bfloat16, 1)
    y, mean, rstd = S.sfp8_layernorm(x, w, b)
    assert y.shape == (0, 64)
    dw, db = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    S.sfp8_layernorm_backward(x, x, w, mean, rstd, dweight=dw, dbias=db)
    assert bool((dw == 0).all() and (db == 0).all())


def test_repeats_captured_and_on_a_side_stream():
    x, w, b = inputs(900, 1024, torch.bfloat16, 5)
    dy = torch.randn(900, 1024, device="cuda", generator=gen(4)).to(torch.bfloat16)
    q, s, mean, rstd = S.sfp8_layernorm_quant(x, w, b)
    want = S.sfp8_layernorm_backward(dy, x, w, mean, rstd)
    ws = S.new_layernorm_backward_workspace(900, 1024, "cuda")
    ws.fill_(255)
    outs = [torch.zeros_like(t) for t in (q, s, mean, rstd, *want)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        S.sfp8_layernorm_quant(x, w, b, q=outs[0], scales=outs[1], mean=outs[2], rstd=outs[3])
        S.sfp8_layernorm_backward(dy, x, w, outs[2], outs[3], dx=outs[4], dweight=outs[5],
                                  dbias=outs[6], workspace=ws)
    for _ in range(2):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, t) for o, t in zip(outs, (q, s, mean, rstd, *want)))


def test_refusals():
    x, w, b = inputs(4, 64, torch.bfloat16, 1)
    mean = torch.zeros(4, device="cuda")
    for bad in (lambda: S.sfp8_layernorm(x.t(), w, b), lambda: S.sfp8_layernorm(x.int(), w, b),
                lambda: S.sfp8_layernorm(x, w[:8], b), lambda: S.sfp8_layernorm(x, w, b.float()),
                lambda: S.sfp8_layernorm(x, w.half(), b.half()),
                lambda: S.sfp8_layernorm(x, w.cpu(), b),
                lambda: S.sfp8_layernorm(x, w, b, out=torch.empty_like(x).float()),
                lambda: S.sfp8_layernorm_quant(x, w, b, q_dtype="bf16"),
                lambda: S.sfp8_layernorm_backward(x[:2], x, w, mean, mean),
                lambda: S.sfp8_layernorm_backward(x.float(), x, w, mean, mean),
                lambda: S.sfp8_layernorm_backward(x, x, w, mean[:2], mean)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: S.sfp8_layernorm(x, w, b, out=x),      # over its input
                lambda: S.sfp8_layernorm(x, w, b, -1.0),
                lambda: S.sfp8_layernorm(x, w, b, float("nan")),
                lambda: S.sfp8_layernorm(x, w, b, float("inf")),
                lambda: S.sfp8_layernorm_quant(x[:, :60], w[:60], b[:60]),
                lambda: S.sfp8_layernorm_backward(x, x, w, mean, mean, workspace=torch.zeros(
                    16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(S.Sfp8Error):
            bad()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [1, 2, 3, 5, 31, 33])
@pytest.mark.parametrize("rows", [1, 9, 3000])
def test_backward_of_narrow_rows(rows, cols, dtype):
    """A row of two has nothing left but eps once its mean and its slope are taken
    out, 1e-5 of the terms: no digit of the fp32 terms' rounding may reach it.
    Up to 32 columns, read by element, dx is the 64-bit value rounded to fp32 and once more to x's
    type (2^-50 of the terms for 64-bit rounding, half of fp16's finest step)."""
    x, w, b = inputs(rows, cols, dtype, rows + cols)
    _, mean, rstd = S.sfp8_layernorm(x, w, b, EPS)
    dy = torch.randn(rows, cols, device="cuda", generator=gen(4)).to(dtype)
    got = S.sfp8_layernorm_backward(dy, x, w, mean, rstd)
    check_backward(got, dy, x, w, mean, rstd, dtype)
    if cols > 32:
        return
    r = rstd.double()[:, None]
    xh = (x.double() - mean.double()[:, None]) * r
    g = dy.double() * w.double()
    a, c = g.mean(1, keepdim=True), xh * (g * xh).mean(1, keepdim=True)
    ref = r * (g - a - c)
    bound = (half_step(dtype) + 2.0 ** -23) * ref.abs() + 2.0 ** -50 * r * (
        g.abs() + a.abs() + c.abs()) + (2.0 ** -25 if dtype == torch.float16 else 2.0 ** -140)
    off = (got[0].double() - ref).abs()
    assert bool((off <= bound).all()), float((off / bound).max())
