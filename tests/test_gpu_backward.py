"""GPU tests of the backward passes from 8-bit checkpoints: the sparse
linear's and the gated block's gradients against the 64-bit formulas and, for
the formulas themselves, against differences."""
import pytest
import torch

import semi_structured_sparse_rowwise_b200 as S
from ffn_reference import (BF16_HALF_STEP, act, backward_reference, decode, gated_grad_reference,
                           gated_reference, gen, linear_parts, quantise_rows, sparse_weight)
from gpu_pipeline import ensure_library, requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_library()
    yield
    assert S.sfp8_read_device_status(clear=True) == (0, 0)


def operands(m, rows, k, seed, a_fmt="e4m3", w_fmt="e4m3"):
    codes, s_w = quantise_rows(sparse_weight(rows, k, seed, 0.05), w_fmt)
    x = torch.randn(m, k, device="cuda", generator=gen(seed + 1)).to(torch.bfloat16)
    a_q, s_a = quantise_rows(x, a_fmt)
    return a_q, s_a, codes, s_w, S.sfp8_compress_24(codes, w_fmt)


def within(got, refs):
    for g, (ref, bound), what in zip(got, refs, ("dx", "dw", "dbias")):
        assert g.shape == ref.shape
        off = (g.double() - ref).abs()
        assert bool((off <= bound).all()), (what, float((off / bound).max()))


SHAPES = [(1, 8, 128), (1, 1, 128), (64, 64, 128), (256, 256, 256), (128, 520, 384),
          (300, 1000, 256), (257, 129, 128), (1000, 77, 640), (20, 5000, 128), (5000, 24, 256),
          (512, 2048, 512), (1500, 768, 1024)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_linear_backward(m, n, k):
    a_q, s_a, codes, s_w, packed = operands(m, n, k, m + n + k)
    dy = torch.randn(m, n, device="cuda", generator=gen(9)).to(torch.bfloat16)
    got = S.sfp8_sparse_linear_backward(dy, a_q, "e4m3", s_a, packed, "e4m3", s_w, n, k,
                                        need_dbias=True)
    d = dy.double()
    within(got, backward_reference(d, torch.zeros_like(d), decode(a_q, "e4m3"), s_a,
                                   decode(codes, "e4m3"), s_w))


@pytest.mark.parametrize("a_fmt,w_fmt", [("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
def test_linear_backward_formats(a_fmt, w_fmt):
    m, n, k = 200, 300, 256
    a_q, s_a, codes, s_w, packed = operands(m, n, k, 4, a_fmt, w_fmt)
    dy = torch.randn(m, n, device="cuda", generator=gen(9)).to(torch.bfloat16)
    got = S.sfp8_sparse_linear_backward(dy, a_q, a_fmt, s_a, packed, w_fmt, s_w, n, k,
                                        need_dbias=True)
    d = dy.double()
    within(got, backward_reference(d, torch.zeros_like(d), decode(a_q, a_fmt), s_a,
                                   decode(codes, w_fmt), s_w))


@pytest.mark.parametrize("n,ld,first", [(64, 96, 8), (61, 64, 0), (61, 67, 3), (61, 72, 8)])
def test_strided_output_gradient(n, ld, first):
    """dy as columns of a wider tensor: read in place or through the copy."""
    m, k = 130, 256
    a_q, s_a, _, s_w, packed = operands(m, n, k, 6)
    wide = torch.randn(m, ld + 8, device="cuda", generator=gen(2)).to(torch.bfloat16)
    dy = wide.view(-1)[first:first + m * ld].view(m, ld)[:, :n]
    args = (a_q, "e4m3", s_a, packed, "e4m3", s_w, n, k)
    got = S.sfp8_sparse_linear_backward(dy, *args, need_dbias=True)
    want = S.sfp8_sparse_linear_backward(dy.contiguous(), *args, need_dbias=True)
    assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_full_width_rows_that_cannot_be_read_in_place_are_refused():
    m, n, k = 130, 64, 256
    a_q, s_a, _, s_w, packed = operands(m, n, k, 6)
    flat = torch.zeros(m * n + 8, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(S.Sfp8Error):
        S.sfp8_sparse_linear_backward(flat[3:3 + m * n].view(m, n), a_q, "e4m3", s_a, packed,
                                      "e4m3", s_w, n, k)


GATED = [(1, 1, 128), (3, 60, 256), (32, 100, 384), (100, 333, 128), (250, 705, 256),
         (513, 130, 640), (800, 1100, 256), (40, 64, 8192), (520, 256, 8192)]


@pytest.mark.parametrize("m,n,k", GATED)
@pytest.mark.parametrize("name,bias", [("silu", False), ("gelu", True)])
def test_gated_backward(m, n, k, name, bias):
    check_gated_backward(m, n, k, name, bias)


def check_gated_backward(m, n, k, name, bias):
    a_q, s_a, codes, s_w, packed = operands(m, 2 * n, k, m + n + k)
    b = None
    if bias:
        b = (torch.randn(2 * n, device="cuda", generator=gen(3)) * 0.3).to(torch.bfloat16)
    dh = torch.randn(m, n + 3, device="cuda", generator=gen(9)).to(torch.bfloat16)[:, 3:]
    got = S.sfp8_gated_linear_backward(dh, a_q, "e4m3", s_a, packed, "e4m3", s_w, n, k, act=name,
                                       bias=b, need_dbias=True)
    a, w = decode(a_q, "e4m3"), decode(codes, "e4m3")
    gate, up, _, _ = gated_reference(a, s_a, w, s_w, b, name)
    z_err = 1e-3 * linear_parts(a, s_a, w, s_w)[1]
    dz, err = gated_grad_reference(dh, gate, up, z_err, name)
    refs = backward_reference(dz, err, a, s_a, w, s_w)
    order = torch.cat((torch.arange(0, 2 * n, 2), torch.arange(1, 2 * n, 2))).cuda()
    refs = [refs[0], tuple(t[order] for t in refs[1]), tuple(t[order] for t in refs[2])]
    within(got, refs)


# Few tokens: tiles and stages of which only some rows exist.
FEW = [(1, 16389, 128), (2, 1003, 2176), (7, 16390, 128), (8, 3280, 640), (9, 1003, 2176),
       (16, 823, 2560), (17, 2051, 1152), (31, 16387, 128), (32, 1640, 1280), (33, 1640, 1280),
       (48, 300, 384), (63, 50, 256), (120, 16, 256), (121, 5, 640),
       (5, 1638, 1280)]


@pytest.mark.parametrize("m,n,k", FEW)
def test_few_tokens(m, n, k):
    a_fmt, w_fmt = ("e4m3", "e5m2") if m % 2 else ("e5m2", "e4m3")
    a_q, s_a, codes, s_w, packed = operands(m, n, k, m + n, a_fmt, w_fmt)
    # rows that end with the allocation, NaN between them
    ld = (n + 7) // 8 * 8 + 8
    flat = torch.full(((m - 1) * ld + n,), float("nan"), device="cuda", dtype=torch.bfloat16)
    dy = flat.as_strided((m, n), (ld, 1))
    dy.copy_(torch.randn(m, n, device="cuda", generator=gen(9)))
    got = S.sfp8_sparse_linear_backward(dy, a_q, a_fmt, s_a, packed, w_fmt, s_w, n, k,
                                        need_dbias=True)
    d = dy.double()
    within(got, backward_reference(d, torch.zeros_like(d), decode(a_q, a_fmt), s_a,
                                   decode(codes, w_fmt), s_w))
    alone = S.sfp8_sparse_linear_backward(dy, a_q, a_fmt, s_a, packed, w_fmt, s_w, n, k,
                                          need_dw=False)
    assert torch.equal(alone[0], got[0])


@pytest.mark.parametrize("m,n,k", [(1, 8195, 128), (6, 1026, 1152), (24, 826, 1280)])
def test_few_tokens_gated(m, n, k):
    check_gated_backward(m, n, k, "gelu", True)


@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_gated_formula_against_differences(name):
    """The 64-bit gradient that the kernels are held to is the derivative of
    the 64-bit forward (central differences), and the kernels' dx follows it."""
    m, n, k = 4, 8, 128
    a_q, s_a, codes, s_w, packed = operands(m, 2 * n, k, 31)
    w = decode(codes, "e4m3") * s_w.double()[:, None]
    x = decode(a_q, "e4m3") * s_a.double()[:, None]
    dh = torch.randn(m, n, device="cuda", generator=gen(1)).to(torch.bfloat16)

    def loss(x, w):
        z = x @ w.t()
        return (act(z[:, 0::2], name)[0] * z[:, 1::2] * dh.double()).sum()

    gate, up, _, _ = gated_reference(decode(a_q, "e4m3"), s_a, decode(codes, "e4m3"), s_w, None,
                                     name)
    dz, _ = gated_grad_reference(dh, gate, up, torch.zeros(m, 2 * n, device="cuda").double(), name)
    step = 1e-5
    for seed in range(4):
        vx = torch.randn(m, k, device="cuda", generator=gen(seed)).double()
        vw = torch.randn(2 * n, k, device="cuda", generator=gen(seed + 9)).double()
        slope = (loss(x + step * vx, w) - loss(x - step * vx, w)) / (2 * step)
        assert abs(slope - ((dz @ w) * vx).sum()) <= 1e-6 * abs(slope) + 1e-6
        slope = (loss(x, w + step * vw) - loss(x, w - step * vw)) / (2 * step)
        assert abs(slope - ((dz.t() @ x) * vw).sum()) <= 1e-6 * abs(slope) + 1e-6
    dx, _, _ = S.sfp8_gated_linear_backward(dh, a_q, "e4m3", s_a, packed, "e4m3", s_w, n, k,
                                            act=name)
    ref = dz @ w
    assert float((dx.double() - ref).norm() / ref.norm()) < 4 * BF16_HALF_STEP


def test_outputs_asked_for_one_at_a_time():
    m, n, k = 70, 90, 256
    a_q, s_a, _, s_w, packed = operands(m, 2 * n, k, 8)
    dh = torch.randn(m, n, device="cuda", generator=gen(9)).to(torch.bfloat16)
    dy = torch.randn(m, 2 * n, device="cuda", generator=gen(9)).to(torch.bfloat16)
    args = (a_q, "e4m3", s_a, packed, "e4m3", s_w)
    for f, d, rows in ((S.sfp8_gated_linear_backward, dh, n),
                       (S.sfp8_sparse_linear_backward, dy, 2 * n)):
        want = f(d, *args, rows, k, need_dbias=True)
        for i in range(3):
            need = dict(zip(("need_dx", "need_dw", "need_dbias"), (i == 0, i == 1, i == 2)))
            got = f(d, *args, rows, k, **need)
            assert [g is not None for g in got] == [i == 0, i == 1, i == 2]
            assert torch.equal(got[i], want[i])
        assert f(d, *args, rows, k, need_dx=False, need_dw=False) == (None, None, None)


@pytest.mark.parametrize("m,n", [(0, 24), (5, 0)])
def test_empty_problems_give_zeros(m, n):
    k = 128
    a_q = torch.zeros(m, k, dtype=torch.uint8, device="cuda")
    s_a = torch.ones(m, device="cuda")
    for f, rows in ((S.sfp8_sparse_linear_backward, n), (S.sfp8_gated_linear_backward, 2 * n)):
        packed = torch.zeros(max(1, rows) * k * 80, dtype=torch.uint8, device="cuda")
        dy = torch.ones(m, n, device="cuda", dtype=torch.bfloat16)
        given = [torch.ones(s, device="cuda", dtype=torch.bfloat16)
                 for s in ((m, k), (rows, k), (rows,))]
        f(dy, a_q, "e4m3", s_a, packed, "e4m3", torch.ones(rows, device="cuda"), n, k,
          dx=given[0], dw=given[1], dbias=given[2])
        assert all(bool((g == 0).all()) for g in given)


def test_repeats_bit_for_bit_and_shares_a_workspace():
    m, n, k = 640, 200, 512
    a_q, s_a, _, s_w, packed = operands(m, 2 * n, k, 12)
    dh = torch.randn(m, n, device="cuda", generator=gen(9)).to(torch.bfloat16)
    ws = S.new_gated_backward_workspace(m, n, k, "cuda")
    ws.fill_(255)      # whatever it holds
    args = (dh, a_q, "e4m3", s_a, packed, "e4m3", s_w, n, k)
    first = S.sfp8_gated_linear_backward(*args, need_dbias=True, workspace=ws)
    for _ in range(3):
        again = S.sfp8_gated_linear_backward(*args, need_dbias=True, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("m,n,k", [(60, 300, 256), (640, 2000, 512)])
def test_calls_that_follow_each_other_on_one_workspace(m, n, k):
    """Passes over different operands, one after the other without a wait, in
    one workspace: each must find the one before it done with the expanded
    operands and dz that it overwrites."""
    ops = [operands(m, 2 * n, k, 20 + i) for i in range(2)]
    dhs = [torch.randn(m, n, device="cuda", generator=gen(i)).to(torch.bfloat16) for i in range(2)]
    ws = S.new_gated_backward_workspace(m, n, k, "cuda")

    def run(i, workspace):
        a_q, s_a, _, s_w, packed = ops[i]
        return S.sfp8_gated_linear_backward(dhs[i], a_q, "e4m3", s_a, packed, "e4m3", s_w, n, k,
                                            need_dbias=True, workspace=workspace)

    want = []
    for i in range(2):
        want.append(run(i, S.new_gated_backward_workspace(m, n, k, "cuda")))
        torch.cuda.synchronize()
    got = [run(i % 2, ws) for i in range(40)]
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2])), i


def test_outputs_and_workspaces_at_any_allowed_alignment():
    """16-byte aligned gradients and workspaces that are not 32-byte aligned,
    with a split contraction (few rows of dx, many weight rows)."""
    m, n, k = 60, 5000, 128
    a_q, s_a, _, s_w, packed = operands(m, n, k, 14)
    dy = torch.randn(m, n, device="cuda", generator=gen(9)).to(torch.bfloat16)
    args = (dy, a_q, "e4m3", s_a, packed, "e4m3", s_w, n, k)
    want = S.sfp8_sparse_linear_backward(*args, need_dbias=True)

    def off(numel, dtype, by):
        return torch.zeros(numel + by, dtype=dtype, device="cuda")[by:]

    ws = S.new_linear_backward_workspace(m, n, k, "cuda")
    got = S.sfp8_sparse_linear_backward(
        *args, dx=off(m * k, torch.bfloat16, 8).view(m, k),
        dw=off(n * k, torch.bfloat16, 8).view(n, k), dbias=off(n, torch.bfloat16, 1),
        workspace=off(ws.numel(), torch.uint8, 16))
    assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_gated_backward_with_zero_rows():
    """All-zero rows of the activation and of both weights: their scales are the
    quantiser's guard, 1e-12 over the format's largest value."""
    m, n, k = 48, 40, 256
    rows = sparse_weight(2 * n, k, 3, 0.05)
    rows[0:6] = 0
    codes, s_w = quantise_rows(rows, "e4m3")
    x = torch.randn(m, k, device="cuda", generator=gen(1)).to(torch.bfloat16)
    x[::5] = 0
    a_q, s_a = quantise_rows(x, "e4m3")
    dh = torch.randn(m, n, device="cuda", generator=gen(9)).to(torch.bfloat16)
    b = (torch.randn(2 * n, device="cuda", generator=gen(3))).to(torch.bfloat16)
    got = S.sfp8_gated_linear_backward(dh, a_q, "e4m3", s_a, S.sfp8_compress_24(codes, "e4m3"),
                                       "e4m3", s_w, n, k, bias=b, need_dbias=True)
    a, w = decode(a_q, "e4m3"), decode(codes, "e4m3")
    gate, up, _, _ = gated_reference(a, s_a, w, s_w, b, "silu")
    dz, err = gated_grad_reference(dh, gate, up, 1e-3 * linear_parts(a, s_a, w, s_w)[1], "silu")
    refs = backward_reference(dz, err, a, s_a, w, s_w)
    order = torch.cat((torch.arange(0, 2 * n, 2), torch.arange(1, 2 * n, 2))).cuda()
    within(got, [refs[0], tuple(t[order] for t in refs[1]), tuple(t[order] for t in refs[2])])
    assert bool((got[0] != 0).any(1).all())       # a zero row of x has an input gradient too


def test_captured_on_a_side_stream():
    m, n, k = 320, 300, 512
    a_q, s_a, _, s_w, packed = operands(m, 2 * n, k, 13)
    dh = torch.randn(m, n, device="cuda", generator=gen(9)).to(torch.bfloat16)
    ws = S.new_gated_backward_workspace(m, n, k, "cuda")
    want = S.sfp8_gated_linear_backward(dh, a_q, "e4m3", s_a, packed, "e4m3", s_w, n, k,
                                        need_dbias=True)
    outs = [torch.zeros_like(w) for w in want]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        S.sfp8_gated_linear_backward(dh, a_q, "e4m3", s_a, packed, "e4m3", s_w, n, k, dx=outs[0],
                                     dw=outs[1], dbias=outs[2], workspace=ws)
    for _ in range(2):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_wrapper_refusals():
    m, n, k = 16, 32, 128
    a_q, s_a, _, s_w, packed = operands(m, n, k, 1)
    dy = torch.zeros(m, n, device="cuda", dtype=torch.bfloat16)
    good = dict(dy=dy, a_q=a_q, a_dtype="e4m3", s_a=s_a, packed=packed, w_dtype="e4m3", s_w=s_w,
                n=n, k=k)
    for bad in (dict(dy=dy[:8]), dict(dy=dy.float()), dict(dy=dy.t().contiguous().t()),
                dict(a_q=a_q[:, :64]), dict(s_a=s_a[:4]), dict(s_w=s_w[:4]),
                dict(packed=packed[:100]), dict(w_dtype="bf16"), dict(dy=dy.cpu()),
                dict(dx=torch.empty(m, k, device="cuda")),
                dict(workspace=torch.zeros(64, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            S.sfp8_sparse_linear_backward(**{**good, **bad})
    with pytest.raises(S.Sfp8Error):
        S.sfp8_sparse_linear_backward(**good, workspace=torch.zeros(64, dtype=torch.uint8,
                                                                    device="cuda"))
