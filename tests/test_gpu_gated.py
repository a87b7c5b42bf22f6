"""GPU tests of the gated feed-forward block's forward: the weight preparation
against the one-weight preparation, h against the 64-bit formula on every
kind of work split, the quantising call against the two steps."""
import pytest
import torch

import semi_structured_sparse_rowwise_b200 as S
from semi_structured_sparse_rowwise_b200 import binding as B
from ffn_reference import decode, gated_reference, gen, quantise_rows, sparse_weight
from gpu_pipeline import ensure_library, requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_library()
    yield
    assert S.sfp8_read_device_status(clear=True) == (0, 0)


def block(m, n, k, seed, a_fmt="e4m3", w_fmt="e4m3", bias=False):
    """A gated block's operands: codes, scales, packed weight, bias."""
    rows = sparse_weight(2 * n, k, seed, 0.05)
    codes, s_w = quantise_rows(rows, w_fmt)
    x = torch.randn(m, k, device="cuda", generator=gen(seed + 1)).to(torch.bfloat16)
    a_q, s_a = quantise_rows(x, a_fmt)
    b = None
    if bias:
        b = (torch.randn(2 * n, device="cuda", generator=gen(seed + 2)) * 0.3).to(torch.bfloat16)
    return x, a_q, s_a, codes, s_w, S.sfp8_compress_24(codes, w_fmt), b


def check(h, a_q, a_fmt, s_a, codes, w_fmt, s_w, bias, act):
    _, _, ref, bound = gated_reference(decode(a_q, a_fmt), s_a, decode(codes, w_fmt), s_w, bias,
                                       act)
    off = (h.double() - ref).abs()
    assert h.shape == ref.shape and bool((off <= bound).all()), float((off / bound).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("n,k", [(1, 128), (65, 256), (300, 4224)])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_prepared_weight_is_that_of_the_alternating_rows(n, k, dtype, fmt):
    big = torch.randn(2, n, k + 16, device="cuda", generator=gen(n + k)).to(dtype)
    gate, up = big[0, :, :k], big[1, :, :k]          # strided rows
    packed, s_w = S.sfp8_prepare_gated_weight_24(gate, up, fmt)
    both = torch.stack((gate, up), 1).reshape(2 * n, k).contiguous()
    want, s_want = S.sfp8_prepare_weight_24(both, fmt)
    assert torch.equal(packed, want) and torch.equal(s_w, s_want)


SHAPES = [(1, 1, 128), (1, 100, 256), (16, 64, 512), (17, 333, 384), (33, 640, 1024),
          (64, 128, 128), (100, 1000, 512), (129, 257, 640), (300, 2000, 256), (513, 65, 128),
          (700, 387, 384), (1030, 2600, 256), (16, 256, 8192), (600, 512, 8192)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("act,bias", [("silu", False), ("gelu", True)])
def test_forward_against_the_formula(m, n, k, act, bias):
    _, a_q, s_a, codes, s_w, packed, b = block(m, n, k, m + n + k, bias=bias)
    h = S.sfp8_gated_linear(a_q, "e4m3", s_a, packed, "e4m3", s_w, n, k, act=act, bias=b)
    check(h, a_q, "e4m3", s_a, codes, "e4m3", s_w, b, act)


@pytest.mark.parametrize("a_fmt,w_fmt", [("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("m,n,k", [(5, 200, 512), (520, 200, 512)])
def test_forward_formats(m, n, k, a_fmt, w_fmt):
    _, a_q, s_a, codes, s_w, packed, b = block(m, n, k, 77, a_fmt, w_fmt, True)
    h = S.sfp8_gated_linear(a_q, a_fmt, s_a, packed, w_fmt, s_w, n, k, bias=b)
    check(h, a_q, a_fmt, s_a, codes, w_fmt, s_w, b, "silu")


@pytest.mark.parametrize("m,n,k", [(16, 256, 2048), (200, 321, 1024)])
def test_every_work_split(m, n, k):
    """The table's entry for (m, 2n, k) is followed, and each one is right."""
    _, a_q, s_a, codes, s_w, packed, b = block(m, n, k, 5, bias=True)
    _, _, ref, bound = gated_reference(decode(a_q, "e4m3"), s_a, decode(codes, "e4m3"), s_w, b,
                                       "gelu")
    try:
        for algo in range(S.sfp8_sparse_linear_algo_count(m, 2 * n, k)):
            S.sfp8_sparse_linear_set_algo(m, 2 * n, k, algo)
            ws = S.new_gated_workspace(m, n, k, "cuda")
            for _ in range(2):      # the second call finds the workspace as the first left it
                h = S.sfp8_gated_linear(a_q, "e4m3", s_a, packed, "e4m3", s_w, n, k, act="gelu",
                                        bias=b, workspace=ws)
                off = (h.double() - ref).abs()
                assert bool((off <= bound).all()), (algo, float((off / bound).max()))
    finally:
        S.sfp8_sparse_linear_set_algo(m, 2 * n, k, 0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("m,n,k", [(1, 320, 512), (16, 320, 512), (40, 333, 256), (600, 128, 384)])
def test_quantising_call_is_the_two_steps(m, n, k, dtype):
    _, _, _, _, s_w, packed, b = block(m, n, k, 11, bias=True)
    x = torch.randn(m, k + 32, device="cuda", generator=gen(3)).to(dtype)[:, :k]
    h, a_q, s_a = S.sfp8_gated_linear_quant(x, "e4m3", packed, "e4m3", s_w, n, k, bias=b)
    q, s = S.sfp8_quantize_rowwise(x, "e4m3")
    want = S.sfp8_gated_linear(q, "e4m3", s, packed, "e4m3", s_w, n, k, bias=b)
    assert torch.equal(a_q, q) and torch.equal(s_a, s) and torch.equal(h, want)


def test_saturated_gates():
    """Gates far outside the activation's curved part: act is 0 or the identity."""
    n, k = 64, 128
    x = torch.full((8, k), 100.0, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(2 * n, k, device="cuda", dtype=torch.bfloat16)
    w[0::4] = -1.0      # every other gate is far below zero
    w.view(2 * n, k // 4, 4)[:, :, 2:] = 0
    codes, s_w = quantise_rows(w, "e4m3")
    a_q, s_a = quantise_rows(x, "e4m3")
    packed = S.sfp8_compress_24(codes, "e4m3")
    for act in ("silu", "gelu"):
        h = S.sfp8_gated_linear(a_q, "e4m3", s_a, packed, "e4m3", s_w, n, k, act=act)
        assert bool((h[:, 0::2] == 0).all())
        check(h, a_q, "e4m3", s_a, codes, "e4m3", s_w, None, act)


def test_empty_problems():
    _, a_q, s_a, _, s_w, packed, _ = block(4, 8, 128, 1)
    h = S.sfp8_gated_linear(a_q[:0], "e4m3", s_a[:0], packed, "e4m3", s_w, 8, 128)
    assert h.shape == (0, 8)
    h = S.sfp8_gated_linear(a_q, "e4m3", s_a, packed, "e4m3", s_w[:0], 0, 128)
    assert h.shape == (4, 0)


def test_captured_and_on_another_stream():
    m, n, k = 16, 512, 1024
    x, a_q, s_a, _, s_w, packed, b = block(m, n, k, 21, bias=True)
    want, _, _ = S.sfp8_gated_linear_quant(x, "e4m3", packed, "e4m3", s_w, n, k, bias=b)
    ws = S.new_gated_quant_workspace(m, n, k, "cuda")
    out = torch.zeros_like(want)
    q, s = torch.empty_like(a_q), torch.empty_like(s_a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for _ in range(3):
            S.sfp8_gated_linear_quant(x, "e4m3", packed, "e4m3", s_w, n, k, bias=b, out=out,
                                      workspace=ws, a_q=q, s_a=s)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_wrapper_refusals():
    x, a_q, s_a, _, s_w, packed, b = block(4, 8, 128, 1, bias=True)
    call = lambda **kw: S.sfp8_gated_linear(**{**dict(
        a_q=a_q, a_dtype="e4m3", s_a=s_a, packed=packed, w_dtype="e4m3", s_w=s_w, n=8, k=128,
        bias=b), **kw})
    for bad in (dict(act="relu"), dict(n=9), dict(k=256), dict(bias=b[:8]), dict(s_w=s_w[:8]),
                dict(packed=packed[:-1]), dict(s_a=s_a[:3]), dict(a_q=a_q[:, :64]),
                dict(out=torch.empty(4, 16, device="cuda", dtype=torch.bfloat16)),
                dict(bias=b.float()), dict(s_w=s_w.cpu()), dict(a_dtype="bf16")):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(ValueError):      # x's last column is not unit stride
        S.sfp8_gated_linear_quant(x.t(), "e4m3", packed, "e4m3", s_w, 8, 128)
    with pytest.raises(S.Sfp8Error):     # h would overwrite x
        big = torch.zeros(4 * 128, device="cuda", dtype=torch.bfloat16)
        S.sfp8_gated_linear_quant(big.view(4, 128), "e4m3", packed, "e4m3", s_w, 8, 128,
                                  out=big[:32].view(4, 8))
    with pytest.raises(S.Sfp8Error):     # h would overwrite the codes
        q = torch.zeros(4 * 128, device="cuda", dtype=torch.uint8)
        call(a_q=q.view(4, 128), out=q[:64].view(torch.bfloat16).view(4, 8))
    with pytest.raises(ValueError):
        S.sfp8_prepare_gated_weight_24(x, x[:, :64])
    assert B.ACTIVATION == {"silu": 0, "gelu": 1}
