"""GPU tests of the backward passes with power at long contractions: sums that
are exact (a lost or doubled term changes bits), gradients that live in the last
rows only, error norms that grow as the terms do; the gated pass on two weight
tiles a block and in every format; infinities and NaN, which stay in their rows."""
import pytest
import torch

import semi_structured_sparse_rowwise_b200 as S
from ffn_reference import (BF16_HALF_STEP, FP8, backward_reference, decode, gated_grad_reference,
                           gated_reference, gen, linear_parts, quantise_rows, sparse_weight)
from gpu_pipeline import ensure_library, requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_library()
    yield
    assert S.sfp8_read_device_status(clear=True) == (0, 0)


def small_integers(seed, *shape):
    return torch.randint(-2, 3, shape, device="cuda", generator=gen(seed)).float()


def powers(seed, count):
    return torch.exp2(torch.randint(-2, 3, (count,), device="cuda", generator=gen(seed)).float())


def exact_operands(m, rows, k, seed, a_fmt, w_fmt):
    """Codes that are integers up to 2 and scales that are powers of two from 1/4
    to 4: every operand is exact in bf16, every product a multiple of 1/4 of at
    most 16, and sums of 2^17 of them stay below 2^24 quarters, exact in fp32 in
    any order."""
    w = small_integers(seed, rows, k).view(rows, k // 4, 4)
    w[:, :, 2:] = 0
    w = torch.gather(w, 2, torch.rand(w.shape, device="cuda", generator=gen(seed + 1)).argsort(2))
    codes = w.reshape(rows, k).to(FP8[w_fmt][0]).view(torch.uint8)
    a_q = small_integers(seed + 2, m, k).to(FP8[a_fmt][0]).view(torch.uint8)
    return a_q, powers(seed + 3, m), codes, powers(seed + 4, rows), S.sfp8_compress_24(codes, w_fmt)


LONG = [(1, 16389, 128), (7, 16390, 128), (31, 16387, 128), (64, 16385, 256), (200, 9001, 384),
        (16387, 1, 128), (16390, 31, 256), (9003, 300, 128), (65, 67, 8192), (129, 4100, 1152),
        # hundreds of tiles in both products, with ragged edges
        (4100, 4001, 4096), (3001, 5000, 2176)]


@pytest.mark.parametrize("m,n,k", LONG)
def test_linear_sums_are_exact(m, n, k):
    a_fmt, w_fmt = ("e4m3", "e5m2") if m % 2 else ("e5m2", "e4m3")
    a_q, s_a, codes, s_w, packed = exact_operands(m, n, k, m + n, a_fmt, w_fmt)
    dy = small_integers(5, m, n).to(torch.bfloat16)
    dx, dw, db = S.sfp8_sparse_linear_backward(dy, a_q, a_fmt, s_a, packed, w_fmt, s_w, n, k,
                                               need_dbias=True)
    d = dy.double()
    w = decode(codes, w_fmt) * s_w.double()[:, None]
    x = decode(a_q, a_fmt) * s_a.double()[:, None]
    # the one rounding is the result's; sums of quarters below 2^24 are fp32 numbers
    for got, ref in ((dx, d @ w), (dw, d.t() @ x), (db, d.sum(0))):
        assert float(ref.abs().max()) < 2 ** 22
        assert torch.equal(got, ref.float().to(torch.bfloat16))


def gated_case(m, n, k, name, bias, a_fmt="e4m3", w_fmt="e4m3", dh=None, seed=0):
    """The gated pass's gradients beside their 64-bit references and bounds."""
    codes, s_w = quantise_rows(sparse_weight(2 * n, k, seed + m + n, 0.05), w_fmt)
    x = torch.randn(m, k, device="cuda", generator=gen(seed + k)).to(torch.bfloat16)
    a_q, s_a = quantise_rows(x, a_fmt)
    b = None
    if bias:
        b = (torch.randn(2 * n, device="cuda", generator=gen(3)) * 0.3).to(torch.bfloat16)
    if dh is None:
        dh = torch.randn(m, n, device="cuda", generator=gen(9)).to(torch.bfloat16)
    got = S.sfp8_gated_linear_backward(dh, a_q, a_fmt, s_a, S.sfp8_compress_24(codes, w_fmt),
                                       w_fmt, s_w, n, k, act=name, bias=b, need_dbias=True)
    a, w = decode(a_q, a_fmt), decode(codes, w_fmt)
    gate, up, _, _ = gated_reference(a, s_a, w, s_w, b, name)
    dz, err = gated_grad_reference(dh, gate, up, 1e-3 * linear_parts(a, s_a, w, s_w)[1], name)
    refs = backward_reference(dz, err, a, s_a, w, s_w)
    order = torch.cat((torch.arange(0, 2 * n, 2), torch.arange(1, 2 * n, 2))).cuda()
    refs = [refs[0], tuple(t[order] for t in refs[1]), tuple(t[order] for t in refs[2])]
    return got, refs


def check(got, refs):
    """Each element within its bound, and each gradient within 2^-7 in the
    2-norm: the terms' roundings (dz to bf16, at most 2^-8 of a term, of either
    sign) add up as the terms themselves do, whose signs are random too, so
    they err by at most 2^-8 of the result's norm, and the result's own rounding
    by 2^-8 again; both are below 0.6 of that for roundings spread over a step,
    which leaves room for the 2^-10 or so of gate's and up's fp32 sums."""
    for g, (ref, bound), what in zip(got, refs, ("dx", "dw", "dbias")):
        off = (g.double() - ref).abs()
        assert bool((off <= bound).all()), (what, float((off / bound).max()))
        rel = float((g.double() - ref).norm() / ref.norm().clamp_min(1e-30))
        assert rel < 2 * BF16_HALF_STEP, (what, rel)


@pytest.mark.parametrize("m,n,k", [
    (520, 6300, 8192),      # two weight tiles a block, two k steps a stage
    (520, 6300, 8320),      # ... and an odd number of k steps: one a stage
    (1, 8195, 128), (31, 8193, 256), (8195, 5, 128), (4100, 66, 384)])
@pytest.mark.parametrize("name,bias", [("silu", False), ("gelu", True)])
def test_gated_backward_norms(m, n, k, name, bias):
    check(*gated_case(m, n, k, name, bias))


@pytest.mark.parametrize("a_fmt,w_fmt", [("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("m,n,k", [(9, 300, 256), (200, 301, 384), (600, 130, 512)])
def test_gated_backward_formats(m, n, k, a_fmt, w_fmt):
    check(*gated_case(m, n, k, "gelu", True, a_fmt, w_fmt))


@pytest.mark.parametrize("m,n,k", [(1, 8195, 128), (33, 8193, 256), (8195, 5, 128),
                                   (4097, 67, 384), (520, 6300, 8192)])
@pytest.mark.parametrize("where", ["units", "tokens"])
def test_gated_gradient_of_the_last_rows(m, n, k, where):
    """dh is zero but in the last hidden unit or token: the bounds shrink to
    those terms, which are the tail of one of the contractions."""
    dh = torch.zeros(m, n, device="cuda", dtype=torch.bfloat16)
    last = torch.randn(m, n, device="cuda", generator=gen(9)).to(torch.bfloat16)
    if where == "units":
        dh[:, -1] = last[:, -1]
    else:
        dh[-1] = last[-1]
    got, refs = gated_case(m, n, k, "silu", True, dh=dh)
    for g, (ref, bound), what in zip(got, refs, ("dx", "dw", "dbias")):
        off = (g.double() - ref).abs()
        assert bool((off <= bound).all()), (what, float((off / bound).max()))
        assert bool((ref != 0).any())


SPECIAL = [float("nan"), float("inf"), float("-inf")]


@pytest.mark.parametrize("value", SPECIAL)
@pytest.mark.parametrize("m,n,k", [(40, 90, 256), (300, 500, 384), (9, 16384, 128)])
def test_special_gradients_stay_in_their_rows(m, n, k, value):
    """A NaN or an infinity in one element of the output's gradient reaches that
    token's dx, that row's dw and that dbias, and nothing else."""
    codes, s_w = quantise_rows(sparse_weight(2 * n, k, 1, 0.05), "e4m3")
    packed = S.sfp8_compress_24(codes, "e4m3")
    a_q, s_a = quantise_rows(torch.randn(m, k, device="cuda", generator=gen(2)), "e4m3")
    token, unit = m - 3, n - 5
    for f, rows, affected in (
            (S.sfp8_sparse_linear_backward, 2 * n, [unit]),
            (S.sfp8_gated_linear_backward, n, [unit, n + unit])):
        dy = torch.randn(m, rows, device="cuda", generator=gen(9)).to(torch.bfloat16)
        args = (a_q, "e4m3", s_a, packed, "e4m3", s_w, rows, k)
        want = f(dy, *args, need_dbias=True)
        dy[token, unit] = value
        got = f(dy, *args, need_dbias=True)
        assert not bool(got[0][token].isfinite().all())
        for t, keep in ((0, [token]), (1, affected), (2, affected)):
            left = torch.ones(got[t].shape[0], dtype=torch.bool, device="cuda")
            left[keep] = False
            assert torch.equal(got[t][left], want[t][left])
            if t:
                assert not bool(got[t][~left].isfinite().all())


@pytest.mark.parametrize("m,n,k", [(5, 64, 256), (40, 333, 384), (600, 130, 512), (16, 128, 8192)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_special_activations_stay_in_their_rows(m, n, k, act):
    """Tokens whose codes or scale are NaN, or whose scale is infinite."""
    codes, s_w = quantise_rows(sparse_weight(2 * n, k, 1, 0.05), "e4m3")
    packed = S.sfp8_compress_24(codes, "e4m3")
    a_q, s_a = quantise_rows(torch.randn(m, k, device="cuda", generator=gen(2)), "e4m3")
    dh = torch.randn(m, n, device="cuda", generator=gen(9)).to(torch.bfloat16)

    def run(a_q, s_a):
        args = (a_q, "e4m3", s_a, packed, "e4m3", s_w, n, k)
        return (S.sfp8_gated_linear(*args, act=act),
                S.sfp8_gated_linear_backward(dh, *args, act=act, need_dw=False)[0])

    want = run(a_q, s_a)
    bad_q, bad_s = a_q.clone(), s_a.clone()
    bad_q[0, k - 1] = 0x7F                   # e4m3's NaN
    bad_q[0, 0:k - 1:3] = 0x7F               # ... among the kept slots of every row
    bad_s[2], bad_s[m - 1] = float("nan"), float("inf")
    got = run(bad_q, bad_s)
    left = torch.ones(m, dtype=torch.bool, device="cuda")
    left[[0, 2, m - 1]] = False
    for g, w in zip(got, want):
        assert torch.equal(g[left], w[left])
        assert not bool(g[~left].isfinite().all(1).any())


@pytest.mark.parametrize("value", SPECIAL)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(9, 64), (40, 1003), (300, 4096), (3000, 2048), (2000, 640),
                                       (20, 20480)])
def test_special_values_in_layer_norm(rows, cols, dtype, value):
    """They reach their own row (and, in the backward pass, their columns'
    sums), whichever kernel takes the sizes."""
    x = torch.randn(rows, cols, device="cuda", generator=gen(1)).to(dtype)
    w = torch.randn(cols, device="cuda", generator=gen(2)).to(dtype)
    dy = torch.randn(rows, cols, device="cuda", generator=gen(3)).to(dtype)
    row, col = rows // 2, cols - 1
    left = torch.ones(rows, dtype=torch.bool, device="cuda")
    left[row] = False
    bad = x.clone()
    bad[row, col] = value
    want, got = S.sfp8_layernorm(x, w), S.sfp8_layernorm(bad, w)
    for a, b in zip(want, got):
        assert torch.equal(a[left], b[left])
    assert bool(got[0][row].isnan().all())
    if cols % 16 == 0:
        for fmt in ("e4m3", "e5m2"):
            want, got = S.sfp8_layernorm_quant(x, w, None, 1e-5, fmt), \
                S.sfp8_layernorm_quant(bad, w, None, 1e-5, fmt)
            for a, b in zip(want, got):
                assert torch.equal(a[left], b[left])
            assert bool(decode(got[0][row], fmt).isnan().all())
    _, mean, rstd = S.sfp8_layernorm(x, w)
    want = S.sfp8_layernorm_backward(dy, x, w, mean, rstd)
    bad = dy.clone()
    bad[row, col] = value
    got = S.sfp8_layernorm_backward(bad, x, w, mean, rstd)
    assert torch.equal(want[0][left], got[0][left])
    assert not bool(got[0][row].isfinite().any())
    keep = torch.arange(cols, device="cuda") != col
    for a, b in zip(want[1:], got[1:]):
        assert torch.equal(a[keep], b[keep]) and not bool(b[col].isfinite())
