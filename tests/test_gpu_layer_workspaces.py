"""GPU tests of the workspaces that layers keep or take for a call: first used
inside a graph capture, after a change of the algorithm table, for many token
counts and on several streams."""
import pytest
import torch

import semi_structured_sparse_rowwise_b200 as S
from ffn_reference import gen
from gpu_pipeline import ensure_library, requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]

# few weight rows and a long k: the split forms, whose counters have to start at zero
M, N, K = 16, 128, 8192


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_library()
    yield
    assert S.sfp8_read_device_status(clear=True) == (0, 0)


def normal(seed, *shape):
    return torch.randn(*shape, device="cuda", generator=gen(seed)).to(torch.bfloat16)


def linear():
    return S.SparseFp8Linear(normal(1, N, K)), lambda layer, x, out: layer(x, out=out)


def gated():
    return (S.SparseFp8GatedLinear(normal(1, N, K), normal(2, N, K)),
            lambda layer, x, out: layer(x, out=out))


def gated_codes():
    layer, _ = gated()

    def run(layer, x, out):
        a_q, s_a = S.sfp8_quantize_rowwise(x, "e4m3")
        return layer.forward_codes(a_q, s_a, out=out)

    return layer, run


FORWARDS = [linear, gated, gated_codes]


def rows(make):
    return N if make is linear else 2 * N


def nan(*shape):
    return torch.full(shape, float("nan"), device="cuda", dtype=torch.bfloat16)


@pytest.mark.parametrize("make", FORWARDS)
def test_first_call_inside_a_capture(make):
    """The clearing of a workspace made during a capture is recorded, not run:
    no later eager call may find that workspace."""
    layer, run = make()
    x = normal(3, M, K)
    want = run(make()[0], x, None)
    # memory of the graph's pool that holds something
    pool, side = torch.cuda.graph_pool_handle(), torch.cuda.Stream()
    filler, graph = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(filler, pool=pool, stream=side):
        t = [torch.full((size << 20,), 255, dtype=torch.uint8, device="cuda")
             for size in [1] * 16 + [32]]       # small blocks and a large one
        del t
    filler.replay()
    torch.cuda.synchronize()
    captured = nan(M, N)
    with torch.cuda.graph(graph, pool=pool, stream=side):
        run(layer, x, captured)
    eager = run(layer, x, nan(M, N))       # before the graph's first run
    torch.cuda.synchronize()
    assert torch.equal(eager, want)
    for _ in range(2):
        captured.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(captured, want)


@pytest.mark.parametrize("make", FORWARDS)
def test_captured_call_keeps_its_workspace_after_a_table_change(make):
    layer, run = make()
    x = normal(3, M, K)
    want = run(layer, x, None).clone()
    captured = nan(M, N)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        run(layer, x, captured)
    n = rows(make)
    query = (S.sfp8_sparse_linear_workspace_bytes if make is gated_codes else
             S.sfp8_sparse_linear_quant_workspace_bytes)
    try:
        size = query(M, n, K)
        # an entry that needs a workspace of another size: the old one's memory
        # is not given to the new one
        for algo in range(S.sfp8_sparse_linear_algo_count(M, n, K)):
            S.sfp8_sparse_linear_set_algo(M, n, K, algo)
            if (query(M, n, K) + 511) // 512 != (size + 511) // 512:
                break
        run(layer, x, None)                # the layer's workspace follows the table
        torch.cuda.synchronize()
        taken = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
        graph.replay()
        torch.cuda.synchronize()
        assert all(bool((t == 255).all()) for t in taken)
        assert torch.equal(captured, want)
    finally:
        S.sfp8_sparse_linear_set_algo(M, n, K, 0)


def test_workspaces_that_need_no_clearing_are_not_cleared(monkeypatch):
    def cleared(*_, **__):
        raise AssertionError("cleared")

    made = (S.new_linear_backward_workspace, (300, 500, 256), S.new_gated_backward_workspace,
            (300, 500, 256), S.new_layernorm_backward_workspace, (300, 500))
    sizes = [f(*a, "cuda").numel() for f, a in zip(made[0::2], made[1::2])]
    monkeypatch.setattr(torch, "zeros", cleared)
    assert [f(*a, "cuda").numel() for f, a in zip(made[0::2], made[1::2])] == sizes
    monkeypatch.undo()
    # the forward's have to start at zero
    for f in (S.new_gated_workspace, S.new_gated_quant_workspace, S.new_workspace,
              S.new_quant_workspace):
        assert not bool(f(M, N, K, "cuda").any())


def backward_layers():
    k, hidden = 256, 384
    w = dict(norm_weight=normal(1, k), norm_bias=normal(2, k), w_gate=normal(3, hidden, k),
             w_up=normal(4, hidden, k), w_down=normal(5, k, hidden))
    block = S.SparseFp8FeedForward(**w)
    return {"linear": (block.down, hidden, k), "gated": (block.gated, k, hidden),
            "block": (block, k, k)}


def tensors(out):
    return [t for t in (out.values() if isinstance(out, dict) else out) if t is not None]


@pytest.mark.parametrize("kind", ["linear", "gated", "block"])
def test_backward_leaves_no_memory_behind(kind):
    """Nothing in a backward pass's workspace is needed after the call, so the
    layer holds none, however many token counts it has met."""
    layer, k, n = backward_layers()[kind]
    held = []
    for m in (65, 130, 300, 301, 512, 777):
        x, dy = normal(m, m, k), normal(m + 1, m, n)
        _, ckpt = layer.forward_checkpoint(x)
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        grads = layer.backward(dy, ckpt)
        torch.cuda.synchronize()
        del grads, x, dy, ckpt
        held.append(torch.cuda.memory_allocated() - before)
    # with the step's tensors gone, less is allocated than before the call
    assert all(h <= 0 for h in held), held


@pytest.mark.parametrize("kind", ["linear", "gated", "block"])
def test_backward_on_two_streams_at_once(kind):
    layer, k, n = backward_layers()[kind]
    m = 700
    steps = []
    for i in range(2):
        _, ckpt = layer.forward_checkpoint(normal(10 + i, m, k))
        steps.append((normal(20 + i, m, n), ckpt))
    torch.cuda.synchronize()
    want = [[t.clone() for t in tensors(layer.backward(*s))] for s in steps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    got = [[], []]
    for _ in range(30):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(tensors(layer.backward(*steps[i])))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


def host_batches(count):
    xs = [normal(50 + i, M, K).cpu().pin_memory() for i in range(count)]
    return xs, [torch.empty((M, N), dtype=torch.bfloat16).pin_memory() for _ in xs]


def test_pipeline_waits_for_what_made_it():
    """The pipeline's streams come after the work that the making stream still
    has queued: its workspace's clearing, the layer's preparation."""
    layer = S.SparseFp8Linear(normal(1, N, K))
    xs, ys = host_batches(3)
    want = [layer(x.cuda()).cpu() for x in xs]
    size = S.sfp8_sparse_linear_quant_workspace_bytes(M, N, K)
    torch.cuda.synchronize()
    t = [torch.full((max(size, 16),), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    del t
    torch.cuda._sleep(400_000_000)         # keeps the current stream busy for a while
    pipe = S.HostPipeline(layer, M, depth=2)
    for x, y in zip(xs, ys):
        y.fill_(float("nan"))
        pipe.submit(x, y)
    pipe.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(y, w) for y, w in zip(ys, want))


def test_pipeline_captured_after_a_table_change():
    layer = S.SparseFp8Linear(normal(1, N, K))
    xs, ys = host_batches(3)
    want = [layer(x.cuda()).cpu() for x in xs]
    pipe = S.HostPipeline(layer, M, depth=2)
    try:
        S.sfp8_sparse_linear_set_algo(M, N, K, 0)      # counts as a change
        graph = pipe.capture(xs, ys)
        for _ in range(2):
            for y in ys:
                y.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(y, w) for y, w in zip(ys, want))
    finally:
        S.sfp8_sparse_linear_set_algo(M, N, K, 0)
