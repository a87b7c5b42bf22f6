"""GPU tests of the layers over the feed-forward operators, run together as they
are used: a sublayer's forward, its backward pass from 8-bit checkpoints, a
single-token step, and steps captured in a graph."""
import pytest
import torch

import semi_structured_sparse_rowwise_b200 as S
from ffn_reference import act, decode, gen
from gpu_pipeline import ensure_library, requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_library()
    yield
    assert S.sfp8_read_device_status(clear=True) == (0, 0)


def weights(k, hidden, seed):
    g = gen(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    return dict(norm_weight=(1 + 0.1 * normal(k)).to(torch.bfloat16),
                norm_bias=(0.1 * normal(k)).to(torch.bfloat16),
                w_gate=(normal(hidden, k) * k ** -0.5).to(torch.bfloat16),
                w_up=(normal(hidden, k) * k ** -0.5).to(torch.bfloat16),
                w_down=(normal(k, hidden) * hidden ** -0.5).to(torch.bfloat16))


def dense(layer_packed, s_w, rows, k, fmt):
    """The weight a layer computes with, in 64 bits."""
    codes = S.sfp8_decompress_24(layer_packed, rows, k)
    return decode(codes, fmt) * s_w.double()[:, None]


def near(got, want, steps=4):
    """Within `steps` bf16 half steps in the 2-norm: what the roundings of a few
    bf16 operands and the result add up to."""
    off = float((got.double() - want).norm() / want.norm())
    assert off < steps * 2.0 ** -8, off


@pytest.mark.parametrize("m,k,hidden,name", [(1, 256, 384, "silu"), (40, 512, 640, "gelu"),
                                             (700, 256, 1152, "silu")])
def test_sublayer_forward_and_backward(m, k, hidden, name):
    w = weights(k, hidden, 3)
    block = S.SparseFp8FeedForward(**w, act=name)
    x = (torch.randn(m, k, device="cuda", generator=gen(4)) * 2).to(torch.bfloat16)
    dy = torch.randn(m, k, device="cuda", generator=gen(5)).to(torch.bfloat16)
    y, ckpt = block.forward_checkpoint(x)
    assert torch.equal(y, block(x))
    grads = block.backward(dy, ckpt)

    # The same chain in 64 bits through autograd, straight through the
    # quantisers: each stage starts from the values the layers quantised.
    _, _, _, (a_q, s_a), (h_q, s_h) = ckpt
    gu = dense(block.gated.packed, block.gated.s_w, 2 * hidden, k, "e4m3")
    down = dense(block.down.packed, block.down.s_w, k, hidden, "e4m3").requires_grad_()
    gate, up = gu[0::2].clone().requires_grad_(), gu[1::2].clone().requires_grad_()
    x64 = x.double().requires_grad_()
    nw, nb = (w[t].double().requires_grad_() for t in ("norm_weight", "norm_bias"))
    n64 = torch.nn.functional.layer_norm(x64, (k,), nw, nb, 1e-5)
    a64 = n64 + ((decode(a_q, "e4m3") * s_a.double()[:, None]) - n64).detach()
    h64 = act(a64 @ gate.t(), name)[0] * (a64 @ up.t())
    q64 = h64 + ((decode(h_q, "e4m3") * s_h.double()[:, None]) - h64).detach()
    y64 = q64 @ down.t()
    y64.backward(dy.double())
    near(y, y64.detach(), 2)
    near(grads["w_down"], down.grad)
    near(grads["w_gate"], gate.grad, 6)
    near(grads["w_up"], up.grad, 6)
    near(grads["norm_weight"], nw.grad, 8)
    near(grads["norm_bias"], nb.grad, 8)
    near(grads["dx"], x64.grad, 8)


def test_gated_layer_is_its_calls():
    k, hidden, m = 256, 200, 19
    w = weights(k, hidden, 8)
    bias = [torch.randn(hidden, device="cuda", generator=gen(i)).to(torch.bfloat16) for i in (1, 2)]
    layer = S.SparseFp8GatedLinear(w["w_gate"], w["w_up"], *bias, act="gelu")
    x = torch.randn(m, k, device="cuda", generator=gen(4))
    h, (a_q, s_a) = layer.forward_checkpoint(x)
    assert torch.equal(h, layer(x)) and torch.equal(h, layer.forward_codes(a_q, s_a))
    dh = torch.randn(m, hidden, device="cuda", generator=gen(5)).to(torch.bfloat16)
    dx, dw, db = layer.backward(dh, (a_q, s_a))
    want = S.sfp8_gated_linear_backward(dh, a_q, "e4m3", s_a, layer.packed, "e4m3", layer.s_w,
                                        hidden, k, act="gelu", bias=torch.cat(bias),
                                        need_dbias=True)
    assert torch.equal(dx, want[0]) and torch.equal(dw.reshape(-1, k), want[1])
    assert torch.equal(db.reshape(-1), want[2])
    assert layer.backward(dh, (a_q, s_a), need_dx=False, need_dbias=False)[0::2] == (None, None)


def test_gated_layer_follows_the_algorithm_table():
    k, hidden, m = 1024, 320, 16
    w = weights(k, hidden, 8)
    layer = S.SparseFp8GatedLinear(w["w_gate"], w["w_up"])
    x = torch.randn(m, k, device="cuda", generator=gen(4)).to(torch.bfloat16)
    want = layer(x)
    try:
        for algo in range(S.sfp8_sparse_linear_algo_count(m, 2 * hidden, k)):
            S.sfp8_sparse_linear_set_algo(m, 2 * hidden, k, algo)
            for _ in range(2):
                near(layer(x), want.double(), 1)
        assert len(layer._ws) == 1      # one workspace, however often the table changed
    finally:
        S.sfp8_sparse_linear_set_algo(m, 2 * hidden, k, 0)


def test_linear_layer_backward():
    layer = S.SparseFp8Linear(torch.randn(96, 256, device="cuda", generator=gen(1)) * 0.1,
                              bias=torch.zeros(96, device="cuda"))
    x = torch.randn(50, 256, device="cuda", generator=gen(4)).to(torch.bfloat16)
    y, ckpt = layer.forward_checkpoint(x)
    y2, ckpt2 = layer.forward_checkpoint(x * 2)     # an earlier checkpoint stays
    assert torch.equal(y, layer(x)) and not torch.equal(ckpt[1], ckpt2[1])
    dy = torch.randn(50, 96, device="cuda", generator=gen(5)).to(torch.bfloat16)
    dx, dw, db = layer.backward(dy, ckpt)
    near(dx, dy.double() @ dense(layer.packed, layer.s_w, 96, 256, "e4m3"))
    near(dw, dy.double().t() @ (decode(ckpt[0], "e4m3") * ckpt[1].double()[:, None]))
    near(db, dy.double().sum(0))


def test_training_step_captured():
    """Forward and backward of the sublayer in one graph, replayed on new inputs."""
    m, k, hidden = 130, 256, 384
    block = S.SparseFp8FeedForward(**weights(k, hidden, 3))
    x = torch.randn(m, k, device="cuda", generator=gen(4)).to(torch.bfloat16)
    dy = torch.randn(m, k, device="cuda", generator=gen(5)).to(torch.bfloat16)

    def step():
        y, ckpt = block.forward_checkpoint(x)
        return {"y": y, **block.backward(dy, ckpt)}

    step()      # makes the workspaces
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step()
    for seed in (6, 7):
        x.copy_(torch.randn(m, k, device="cuda", generator=gen(seed)))
        graph.replay()
        torch.cuda.synchronize()
        got = {n: t.clone() for n, t in out.items()}
        want = step()
        assert all(torch.equal(got[n], want[n]) for n in want)


def test_refusals():
    w = weights(256, 384, 3)
    with pytest.raises(ValueError):
        S.SparseFp8FeedForward(**{**w, "w_down": w["w_down"][:, :256].contiguous()})
    with pytest.raises(ValueError):
        S.SparseFp8GatedLinear(w["w_gate"], w["w_up"], bias_gate=w["norm_bias"])
    with pytest.raises(ValueError):
        S.SparseFp8GatedLinear(w["w_gate"], w["w_up"][:100])
