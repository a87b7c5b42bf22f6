"""The layers a user calls: prepared 2:4 sparse FP8 weights, their forward and,
from 8-bit activation checkpoints, their backward passes.

Weight preparation (once, as the page "Add CUTLASS-based row-wise scaled
sparse FP8 kernel", pytorch/ao pull request 1671, does at ``quantize_()`` time,
its items 1, 3 and 4): 2:4 magnitude prune -> row-wise FP8 quantisation ->
2:4 compression.  Forward (per call): dynamic row-wise FP8 quantisation of the
activation -> sparse FP8 GEMM with the scale/bias epilogue.  Every step is a
kernel of libsfp8.so; torch only provides memory and streams.

``SparseFp8Linear`` is one projection, ``SparseFp8GatedLinear`` the gate/up pair
of a gated feed-forward block, ``SparseFp8FeedForward`` the whole sublayer (layer
norm, gated block, down projection).  Their ``forward_checkpoint`` returns what
the backward pass needs beside the result: the quantised activation and its
scales, one byte per element.  Gradients are straight-through: those of the
weights that were prepared, dense, for the caller's optimiser, whose updated
weights make new layers.  A backward pass takes its workspace from torch's
allocator for the call (0.8 GB for a gated block of 14336 units over 4096 at 8192
tokens), so layers, token counts and streams share one and any number of passes
may be in flight.
"""

import torch

from . import binding as B


def _kept_workspace(cache, key, new, *sizes):
    """cache[key], a forward workspace made by new(*sizes) when it is missing or
    the library's algorithm table has changed since (which may pick a split that
    needs a larger one, with its counters elsewhere).  One made inside a graph
    capture is not kept: its clearing is part of the graph and has not run when
    the capture ends, and its memory is the graph's.  One that a captured call
    takes stays allocated as long as the cache, for the graph's replays, also
    when the table changes."""
    epoch = B.algo_epoch()
    capturing = torch.cuda.is_current_stream_capturing()
    hit = cache.get(key)        # table's state, workspace, those that graphs use
    if hit is None or hit[0] != epoch:
        ws = new(*sizes)
        if capturing:
            return ws
        hit = cache[key] = (epoch, ws, [] if hit is None else hit[2])
    if capturing and all(ws is not hit[1] for ws in hit[2]):
        hit[2].append(hit[1])
    return hit[1]


class SparseFp8Linear:
    """y = (s_a s_w^T) * (A_q W_q^T) + bias with a 2:4 compressed FP8 weight."""

    def __init__(self, weight, bias=None, w_dtype="e4m3", a_dtype="e4m3", prune=True):
        if weight.dim() != 2:
            raise ValueError("weight must be [out_features, in_features]")
        self.n, self.k = weight.shape
        self.w_dtype = w_dtype
        self.a_dtype = a_dtype
        self.device = weight.device
        if prune:
            # prune, quantise and compress in one pass over the weight
            self.packed, self.s_w = B.sfp8_prepare_weight_24(weight.contiguous(), w_dtype)
        else:
            w_q, self.s_w = B.sfp8_quantize_rowwise(weight.contiguous(), w_dtype)
            self.packed = B.sfp8_compress_24(w_q, w_dtype)
        self.bias = None if bias is None else bias.to(torch.bfloat16).contiguous()
        self._ws = {}
        self._act = {}
        self._host = {}

    @classmethod
    def from_compressed(cls, packed, s_w, n, k, bias=None, w_dtype="e4m3", a_dtype="e4m3"):
        """A layer over an already compressed weight (packed, s_w)."""
        self = cls.__new__(cls)
        self.n, self.k = n, k
        self.w_dtype, self.a_dtype = w_dtype, a_dtype
        self.device = packed.device
        self.packed, self.s_w = packed, s_w
        self.bias = None if bias is None else bias.to(torch.bfloat16).contiguous()
        self._ws = {}
        self._act = {}
        self._host = {}
        return self

    def workspace(self, m):
        """The layer's zeroed workspace for m tokens (kept between calls; each
        call leaves its split-K counters at zero).  Re-sized after any change
        of the library's algorithm table."""
        return _kept_workspace(self._ws, m, B.new_quant_workspace, m, self.n, self.k, self.device)

    def autotune(self, x, reps=10, flush_bytes=256 << 20):
        """Times every work split of the GEMM for x's token count on this
        layer's weight (sfp8_sparse_linear_search; a flush_bytes write before
        each timed launch evicts the operands from L2) and stores the fastest
        in the library's shape-keyed table, which every later forward with
        that token count -- of any layer of the same shape on this device --
        uses.  Returns (best algorithm, median microseconds per algorithm)."""
        m = x.shape[0]
        a_q, s_a = B.sfp8_quantize_rowwise(x, self.a_dtype)
        flush = None
        if flush_bytes:
            flush = torch.empty((flush_bytes,), dtype=torch.uint8, device=self.device)
        best, times = B.sfp8_sparse_linear_search(a_q, self.a_dtype, s_a, self.packed,
                                                  self.w_dtype, self.s_w, self.n, self.k,
                                                  bias=self.bias, reps=reps, flush=flush)
        B.sfp8_sparse_linear_set_algo(m, self.n, self.k, best, self.device)
        return best, times

    def forward(self, x, out=None):
        """x [m, k] bf16/f16/f32 on the layer's device -> y [m, n] bf16.

        One library call (sfp8_sparse_linear_quant): the quantiser, then the
        GEMM as its programmatic dependent.  The quantised activation, its
        scales and the workspace are kept per token count, so one forward of
        a layer per token count may be in flight at a time (calls on one
        stream are ordered)."""
        m = x.shape[0]
        a_q, s_a = self._act_buffers(m)
        y, _, _ = B.sfp8_sparse_linear_quant(x, self.a_dtype, self.packed, self.w_dtype,
                                             self.s_w, self.n, self.k, bias=self.bias, out=out,
                                             workspace=self.workspace(m), a_q=a_q, s_a=s_a)
        return y

    __call__ = forward

    def forward_checkpoint(self, x):
        """The forward for training: (y, checkpoint), the checkpoint being the
        quantised activation [m, k] and its scales [m] in buffers of its own
        (any number may be kept at a time), the input of ``backward``.  The
        workspace is the layer's: one forward of a layer per token count in
        flight at a time, as in ``forward``."""
        m = x.shape[0]
        y, a_q, s_a = B.sfp8_sparse_linear_quant(x, self.a_dtype, self.packed, self.w_dtype,
                                                 self.s_w, self.n, self.k, bias=self.bias,
                                                 workspace=self.workspace(m))
        return y, (a_q, s_a)

    def backward(self, dy, checkpoint, need_dx=True, need_dw=True, need_dbias=None):
        """(dx [m, k], dw [n, k], dbias [n]) bf16 from dy [m, n] bf16 and
        ``forward_checkpoint``'s checkpoint; None where not asked for (dbias by
        default: where the layer has a bias)."""
        a_q, s_a = checkpoint
        if need_dbias is None:
            need_dbias = self.bias is not None
        return B.sfp8_sparse_linear_backward(
            dy, a_q, self.a_dtype, s_a, self.packed, self.w_dtype, self.s_w, self.n, self.k,
            need_dx=need_dx, need_dw=need_dw, need_dbias=need_dbias)

    def _act_buffers(self, m):
        """The quantised activation [m, k] and its scales [m] (kept per m)."""
        b = self._act.get(m)
        if b is None:
            b = (torch.empty((m, self.k), dtype=torch.uint8, device=self.device),
                 torch.empty((m,), dtype=torch.float32, device=self.device))
            self._act[m] = b
        return b

    def _host_buffers(self, m, x_dtype):
        """Device buffers of the host path for m tokens (kept): staging x, the
        quantised activation and its scales, staging y."""
        key = (m, x_dtype)
        b = self._host.get(key)
        if b is None:
            a_q, s_a = self._act_buffers(m)
            b = (torch.empty((m, self.k), dtype=x_dtype, device=self.device), a_q, s_a,
                 torch.empty((m, self.n), dtype=torch.bfloat16, device=self.device))
            self._host[key] = b
        return b

    def forward_host(self, x_host, y_host, x_dev=None, y_dev=None):
        """Host-buffer forward: x_host [m, k] (page-locked for an asynchronous
        copy) -> device -> quantise -> sparse linear -> y_host [m, n] bf16, in
        one library call (sfp8_sparse_linear_quant_host) on the current
        stream.  x_dev / y_dev override the layer's staging buffers."""
        m = x_host.shape[0]
        xs, a_q, s_a, ys = self._host_buffers(m, x_host.dtype)
        return B.sfp8_sparse_linear_quant_host(
            x_host, self.a_dtype, self.packed, self.w_dtype, self.s_w, self.n, self.k,
            xs if x_dev is None else x_dev, a_q, s_a, ys if y_dev is None else y_dev, y_host,
            self.workspace(m), bias=self.bias)


class SparseFp8GatedLinear:
    """h = act(x W_gate^T + b_gate) * (x W_up^T + b_up) over one compressed weight
    that holds both, one kernel for the whole block.  ``act`` is "silu" or "gelu",
    the latter in its tanh form (torch's ``approximate="tanh"``)."""

    def __init__(self, w_gate, w_up, bias_gate=None, bias_up=None, act="silu", w_dtype="e4m3",
                 a_dtype="e4m3"):
        if w_gate.dim() != 2:
            raise ValueError("w_gate and w_up must be [hidden, in_features]")
        if (bias_gate is None) != (bias_up is None):
            raise ValueError("give both biases or none")
        self.n, self.k = w_gate.shape
        self.act, self.w_dtype, self.a_dtype = act, w_dtype, a_dtype
        self.device = w_gate.device
        self.packed, self.s_w = B.sfp8_prepare_gated_weight_24(w_gate.contiguous(),
                                                               w_up.contiguous(), w_dtype)
        self.bias = None
        if bias_gate is not None:
            self.bias = torch.cat((bias_gate, bias_up)).to(torch.bfloat16)
        self._ws = {}

    def _workspace(self, kind, m):
        new = B.new_gated_quant_workspace if kind == "quant" else B.new_gated_workspace
        return _kept_workspace(self._ws, (kind, m), new, m, self.n, self.k, self.device)

    def forward_checkpoint(self, x, out=None):
        """(h [m, hidden] bf16, checkpoint) from x [m, k] bf16/f16/f32; the
        checkpoint (codes and scales of x) is the input of ``backward``.  The
        layer keeps one workspace per token count, so one forward call of a
        layer per token count may be in flight at a time (calls on one stream
        are ordered); calls captured in graphs that may run at the same time, or
        beside eager ones, take layers of their own.  (A captured call uses the
        workspace that eager calls have made; where there is none, one of the
        graph's own that the graph clears at each run.)"""
        h, a_q, s_a = B.sfp8_gated_linear_quant(
            x, self.a_dtype, self.packed, self.w_dtype, self.s_w, self.n, self.k, act=self.act,
            bias=self.bias, out=out, workspace=self._workspace("quant", x.shape[0]))
        return h, (a_q, s_a)

    def forward(self, x, out=None):
        """h [m, hidden] bf16."""
        return self.forward_checkpoint(x, out)[0]

    __call__ = forward

    def forward_codes(self, a_q, s_a, out=None):
        """h from an activation that is already quantised to ``a_dtype`` codes
        (by ``sfp8_layernorm_quant``, for instance)."""
        return B.sfp8_gated_linear(a_q, self.a_dtype, s_a, self.packed, self.w_dtype, self.s_w,
                                   self.n, self.k, act=self.act, bias=self.bias, out=out,
                                   workspace=self._workspace("codes", a_q.shape[0]))

    def backward(self, dh, checkpoint, need_dx=True, need_dw=True, need_dbias=None):
        """(dx [m, k], dw [2, hidden, k], dbias [2, hidden]) bf16 from dh [m,
        hidden] bf16: dw[0], dbias[0] are gate's, dw[1], dbias[1] up's; None
        where not asked for (dbias by default: where the layer has biases)."""
        a_q, s_a = checkpoint
        if need_dbias is None:
            need_dbias = self.bias is not None
        dx, dw, db = B.sfp8_gated_linear_backward(
            dh, a_q, self.a_dtype, s_a, self.packed, self.w_dtype, self.s_w, self.n, self.k,
            act=self.act, bias=self.bias, need_dx=need_dx, need_dw=need_dw,
            need_dbias=need_dbias)
        return (dx, None if dw is None else dw.view(2, self.n, self.k),
                None if db is None else db.view(2, self.n))


class SparseFp8FeedForward:
    """The feed-forward sublayer without its residual addition:
    y = down(act(gate(norm(x))) * up(norm(x))), the norm, a layer norm, going
    straight to the FP8 codes that the gated block reads.  One forward call per
    token count may be in flight at a time, as for its two layers; backward
    passes share nothing."""

    def __init__(self, norm_weight, norm_bias, w_gate, w_up, w_down, act="silu", eps=1e-5,
                 w_dtype="e4m3", a_dtype="e4m3"):
        self.norm_weight, self.norm_bias, self.eps = norm_weight, norm_bias, eps
        self.gated = SparseFp8GatedLinear(w_gate, w_up, act=act, w_dtype=w_dtype, a_dtype=a_dtype)
        self.down = SparseFp8Linear(w_down, w_dtype=w_dtype, a_dtype=a_dtype)
        if self.down.k != self.gated.n:
            raise ValueError("w_down must have one column per hidden unit")

    def forward_checkpoint(self, x):
        """(y [m, out] bf16, checkpoint) from x [m, k]; the checkpoint keeps x
        itself (not a copy), the norm's two statistics per row and the
        codes and scales of the two quantised activations."""
        a_q, s_a, mean, rstd = B.sfp8_layernorm_quant(x, self.norm_weight, self.norm_bias,
                                                      self.eps, self.gated.a_dtype)
        h = self.gated.forward_codes(a_q, s_a)
        y, inner = self.down.forward_checkpoint(h)
        return y, (x, mean, rstd, (a_q, s_a), inner)

    def forward(self, x):
        """y [m, out] bf16."""
        return self.forward_checkpoint(x)[0]

    __call__ = forward

    def backward(self, dy, checkpoint):
        """Gradients from dy [m, out] bf16: a dict with dx (x's dtype), norm_weight
        and norm_bias (float32), w_gate, w_up and w_down (bf16)."""
        x, mean, rstd, outer, inner = checkpoint
        dh, dw_down, _ = self.down.backward(dy, inner)
        dn, dw, _ = self.gated.backward(dh, outer)
        # the norm's backward pass takes its gradient in x's type
        dn = dn if dn.dtype == x.dtype else dn.to(x.dtype)
        dx, d_weight, d_bias = B.sfp8_layernorm_backward(dn, x, self.norm_weight, mean, rstd)
        return dict(dx=dx, norm_weight=d_weight, norm_bias=d_bias, w_gate=dw[0], w_up=dw[1],
                    w_down=dw_down)


class HostPipeline:
    """Streams host batches of m tokens through a layer, with the host <->
    device copies of one batch overlapping the compute of its neighbours.

    Copies in run on one CUDA stream, the forward (quantise + sparse linear,
    one library call) on a second, copies out on a third; `depth` sets of
    device buffers rotate, and CUDA events order each batch's three steps and
    the reuse of a set.  With page-locked host buffers every step is
    asynchronous, so a sequence of submits can also be captured in a CUDA
    graph (`capture`) and replayed with no per-batch host work."""

    def __init__(self, layer, m, x_dtype=torch.bfloat16, depth=3):
        dev = layer.device
        self.layer, self.m = layer, m
        self.streams = [torch.cuda.Stream(dev) for _ in range(3)]
        self.slots = []
        for _ in range(depth):
            self.slots.append(dict(
                x=torch.empty((m, layer.k), dtype=x_dtype, device=dev),
                y=torch.empty((m, layer.n), dtype=torch.bfloat16, device=dev),
                a_q=torch.empty((m, layer.k), dtype=torch.uint8, device=dev),
                s_a=torch.empty((m,), dtype=torch.float32, device=dev)))
        self._new_workspace()
        self._reset()

    def _new_workspace(self):
        """A zeroed workspace for the table's present choice.  The pipeline's
        streams come after what the current one has queued, the clearing and the
        layer's preparation among it."""
        L = self.layer
        self._ws_epoch = B.algo_epoch()
        ws = B.new_quant_workspace(self.m, L.n, L.k, L.device)
        for sl in self.slots:
            sl["ws"] = ws
        for s in self.streams:
            s.wait_stream(torch.cuda.current_stream(L.device))

    def _reset(self):
        for sl in self.slots:
            sl.update(used=False, x_in=torch.cuda.Event(), y_done=torch.cuda.Event(),
                      y_out=torch.cuda.Event())
        self.i = 0

    def submit(self, x_host, y_host, layer=None):
        """Enqueue one batch: x_host [m, k] -> y_host [m, n] bf16, through
        `layer` (default: the pipeline's; any layer of the same shape, e.g.
        the next layer of a model).  Returns the event that completes once
        y_host holds the result."""
        s_in, s_comp, s_out = self.streams
        sl = self.slots[self.i % len(self.slots)]
        self.i += 1
        L = self.layer if layer is None else layer
        if (L.n, L.k) != (self.layer.n, self.layer.k):
            raise ValueError("layer shape differs from the pipeline's")
        if self._ws_epoch != B.algo_epoch():
            # the algorithm table changed: the forward may need a larger workspace
            self.synchronize()
            self._new_workspace()
        # the set is free once its previous forward has read x and its
        # previous copy out has read y
        if sl["used"]:
            s_in.wait_event(sl["y_done"])
        with torch.cuda.stream(s_in):
            sl["x"].copy_(x_host, non_blocking=True)
        sl["x_in"].record(s_in)
        s_comp.wait_event(sl["x_in"])
        if sl["used"]:
            s_comp.wait_event(sl["y_out"])
        sl["used"] = True
        with torch.cuda.stream(s_comp):
            B.sfp8_sparse_linear_quant(sl["x"], L.a_dtype, L.packed, L.w_dtype, L.s_w, L.n, L.k,
                                       bias=L.bias, out=sl["y"], workspace=sl["ws"],
                                       a_q=sl["a_q"], s_a=sl["s_a"])
        sl["y_done"].record(s_comp)
        s_out.wait_event(sl["y_done"])
        with torch.cuda.stream(s_out):
            y_host.copy_(sl["y"], non_blocking=True)
        sl["y_out"].record(s_out)
        return sl["y_out"]

    def capture(self, x_hosts, y_hosts, layers=None):
        """A CUDA graph of one submit per (x_host, y_host) pair (page-locked
        host tensors); replay it with .replay().  The pipeline's buffers
        belong to the graph afterwards: use another pipeline for eager
        submits."""
        self.synchronize()
        if self._ws_epoch != B.algo_epoch():
            self._new_workspace()     # now: nothing can be waited for during the capture
        self._reset()
        origin = torch.cuda.Stream(self.layer.device)
        origin.wait_stream(torch.cuda.current_stream(self.layer.device))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=origin):
            for s in self.streams:
                s.wait_stream(origin)
            for j, (xh, yh) in enumerate(zip(x_hosts, y_hosts)):
                self.submit(xh, yh, None if layers is None else layers[j % len(layers)])
            for s in self.streams:
                origin.wait_stream(s)
        torch.cuda.current_stream(self.layer.device).wait_stream(origin)
        return g

    def synchronize(self):
        for s in self.streams:
            s.synchronize()
