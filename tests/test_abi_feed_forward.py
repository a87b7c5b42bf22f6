"""Host-side validation of the feed-forward sublayer's entry points, answered
without a GPU, and their declarations seen from plain C.  Nothing here launches
a kernel."""
import ctypes
import os
import subprocess

import pytest

from semi_structured_sparse_rowwise_b200 import binding, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = ctypes.c_void_p(0x10000)        # never dereferenced: rejected before use
ODD = ctypes.c_void_p(0x10001)
BF16, F16, F32, E4M3, E5M2 = range(5)
INVALID, SHAPE, MISALIGNED, DTYPE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def call(fn, good, **changed):
    args = {**good, **changed}
    return fn(*args.values())


def test_prepare_gated_weight(lib):
    good = dict(gate=FAKE, up=FAKE, dtype=BF16, n=4, k=128, ld=128, q=E4M3, packed=FAKE, s_w=FAKE,
                stream=None)
    f = lib.sfp8_prepare_gated_weight_24
    assert call(f, good, q=BF16) == DTYPE and call(f, good, dtype=E4M3) == DTYPE
    assert call(f, good, n=-1) == INVALID and call(f, good, ld=64) == INVALID
    assert call(f, good, k=100) == SHAPE and call(f, good, n=1 << 30) == SHAPE
    assert call(f, good, up=None) == INVALID and call(f, good, gate=None) == INVALID
    assert call(f, good, up=ODD) == MISALIGNED and call(f, good, ld=132) == MISALIGNED
    assert call(f, good, n=0) == 0


GATED = dict(a_q=FAKE, a_dtype=E4M3, s_a=FAKE, m=4, packed=FAKE, w_dtype=E4M3, s_w=FAKE, n=8,
             k=128, act=0, bias=None, h=FAKE, ws=None, ws_bytes=0, stream=None)


def test_gated_linear(lib):
    f = lib.sfp8_gated_linear
    assert call(f, GATED, act=2) == INVALID and call(f, GATED, act=-1) == INVALID
    assert call(f, GATED, a_dtype=F32) == DTYPE and call(f, GATED, w_dtype=BF16) == DTYPE
    assert call(f, GATED, n=-1) == INVALID and call(f, GATED, m=-1) == INVALID
    assert call(f, GATED, k=100) == SHAPE and call(f, GATED, k=0) == SHAPE
    assert call(f, GATED, n=1 << 30) == SHAPE
    for name in ("a_q", "s_a", "packed", "s_w", "h"):
        assert call(f, GATED, **{name: None}) == INVALID
        assert call(f, GATED, **{name: ODD}) == MISALIGNED
    assert call(f, GATED, bias=ODD) == MISALIGNED
    assert call(f, GATED, m=0) == 0 and call(f, GATED, n=0) == 0
    for q in (lib.sfp8_gated_linear_workspace_bytes, lib.sfp8_gated_linear_quant_workspace_bytes,
              lib.sfp8_gated_linear_backward_workspace_bytes,
              lib.sfp8_sparse_linear_backward_workspace_bytes):
        assert q(0, 8, 128) == q(4, 0, 128) == q(4, 8, 100) == q(-1, 8, 128) == 0


def test_gated_linear_quant(lib):
    good = dict(x=FAKE, x_dtype=BF16, ld=128, a_dtype=E4M3, a_q=ctypes.c_void_p(0x20000),
                s_a=ctypes.c_void_p(0x30000), m=4, packed=FAKE, w_dtype=E4M3, s_w=FAKE, n=8,
                k=128, act=1, bias=None, h=ctypes.c_void_p(0x40000), ws=None, ws_bytes=0,
                stream=None)
    f = lib.sfp8_gated_linear_quant
    assert call(f, good, x_dtype=E4M3) == DTYPE and call(f, good, act=7) == INVALID
    assert call(f, good, ld=64) == INVALID and call(f, good, k=64) == SHAPE
    assert call(f, good, h=FAKE) == INVALID           # h over x
    # h is [m, n], not as wide as the weight's 2n rows: it may end where x begins
    # (what is refused next is the device or, where there is one, the row stride)
    assert call(f, good, ld=132, h=ctypes.c_void_p(0x10000 - 4 * 8 * 2)) not in (0, INVALID)
    assert call(f, good, ld=132, h=ctypes.c_void_p(0x10002 - 4 * 8 * 2)) == INVALID
    assert call(f, good, m=0) == 0


BACK = dict(dy=FAKE, ld=8, a_q=FAKE, a_dtype=E4M3, s_a=FAKE, m=4, packed=FAKE, w_dtype=E4M3,
            s_w=FAKE, n=8, k=128, dx=FAKE, dw=FAKE, dbias=FAKE, ws=FAKE, ws_bytes=0, stream=None)


def test_linear_backward(lib):
    f = lib.sfp8_sparse_linear_backward
    assert call(f, BACK, a_dtype=BF16) == DTYPE and call(f, BACK, w_dtype=F32) == DTYPE
    assert call(f, BACK, ld=7) == INVALID and call(f, BACK, m=-1) == INVALID
    assert call(f, BACK, n=-1, ld=8) == INVALID and call(f, BACK, k=130) == SHAPE
    assert call(f, BACK, m=1 << 31) == SHAPE
    for name in ("dx", "dw", "dbias", "a_q", "s_a", "packed", "s_w"):
        assert call(f, BACK, **{name: ODD}) == MISALIGNED
    for name in ("dy", "a_q", "s_a", "packed", "s_w"):
        assert call(f, BACK, **{name: None}) == INVALID
    assert call(f, BACK, ld=12) == MISALIGNED          # rows that TMA cannot read
    assert call(f, BACK, dy=ctypes.c_void_p(0x10002)) == MISALIGNED
    apart = dict(dx=ctypes.c_void_p(0x20000), dw=ctypes.c_void_p(0x30000),
                 dbias=ctypes.c_void_p(0x40000), ws=ctypes.c_void_p(0x50000))
    for name in ("dx", "dw", "dbias"):                 # a gradient over an input, or another
        assert call(f, BACK, **{**apart, name: FAKE}) == INVALID
        other = "dw" if name == "dx" else "dx"
        assert call(f, BACK, **{**apart, name: apart[other]}) == INVALID
        assert call(f, BACK, **{**apart, name: apart["ws"], "ws_bytes": 64}) == INVALID


def test_gated_backward(lib):
    good = dict(list(BACK.items())[:11] + [("act", 0), ("bias", None)] + list(BACK.items())[11:])
    f = lib.sfp8_gated_linear_backward
    assert call(f, good, act=3) == INVALID and call(f, good, n=1 << 30, ld=1 << 30) == SHAPE
    assert call(f, good, bias=ODD) == MISALIGNED and call(f, good, dy=ODD) == MISALIGNED
    for name in ("dy", "a_q", "s_a", "packed", "s_w"):
        assert call(f, good, **{name: None}) == INVALID
        assert call(f, good, **{name: None}, dx=None, dw=None) == INVALID   # gate and up need all


def test_layernorm(lib):
    good = dict(x=FAKE, dtype=BF16, rows=4, cols=64, ld=64, weight=FAKE, bias=FAKE, p_dtype=BF16,
                eps=1e-5, y=FAKE, q=FAKE, q_dtype=E4M3, scales=FAKE, mean=FAKE, rstd=FAKE,
                stream=None)
    f = lib.sfp8_layernorm
    assert call(f, good, dtype=E4M3) == DTYPE and call(f, good, p_dtype=F16) == DTYPE
    assert call(f, good, q_dtype=F16) == DTYPE
    assert call(f, good, rows=-1) == INVALID and call(f, good, ld=63) == INVALID
    for eps in (-1e-5, float("nan"), float("inf")):
        assert call(f, good, eps=eps) == INVALID
    assert call(f, good, cols=0) == SHAPE and call(f, good, cols=60) == SHAPE
    assert call(f, good, x=None) == INVALID and call(f, good, scales=None) == INVALID
    for name in ("x", "y", "weight", "bias", "mean", "rstd", "q", "scales"):
        assert call(f, good, **{name: ODD}) == MISALIGNED
    assert call(f, good, ld=68) == MISALIGNED          # codes need 16-byte rows
    apart = {n: ctypes.c_void_p(0x20000 + 0x1000 * i)
             for i, n in enumerate(("y", "q", "scales", "mean", "rstd"))}
    for name in apart:
        assert call(f, good, **{**apart, name: FAKE}) == INVALID      # over x
        other = "q" if name == "y" else "y"
        assert call(f, good, **{**apart, name: apart[other]}) == INVALID
    assert call(f, good, rows=0) == 0


def test_layernorm_backward(lib):
    good = dict(dy=FAKE, ld_dy=64, x=FAKE, dtype=BF16, rows=4, cols=64, ld=64, weight=FAKE,
                p_dtype=F32, mean=FAKE, rstd=FAKE, dx=FAKE, dw=FAKE, db=FAKE, ws=FAKE, ws_bytes=0,
                stream=None)
    f = lib.sfp8_layernorm_backward
    assert call(f, good, dtype=E5M2) == DTYPE and call(f, good, p_dtype=F16) == DTYPE
    assert call(f, good, ld_dy=63) == INVALID and call(f, good, cols=-1) == INVALID
    assert call(f, good, cols=0) == SHAPE
    for name in ("dy", "x", "mean", "rstd"):
        assert call(f, good, **{name: None}) == INVALID
        assert call(f, good, **{name: ODD}) == MISALIGNED
    for name in ("dx", "dw", "db", "weight"):
        assert call(f, good, **{name: ODD}) == MISALIGNED
    assert call(f, good, dx=None, dw=None, db=None) == 0     # nothing asked for
    apart = dict(dx=ctypes.c_void_p(0x20000), dw=ctypes.c_void_p(0x30000),
                 db=ctypes.c_void_p(0x40000))
    for name in apart:
        assert call(f, good, **{**apart, name: FAKE}) == INVALID
        assert call(f, good, **{**apart, name: apart["dx" if name == "dw" else "dw"]}) == INVALID
    assert lib.sfp8_layernorm_backward_workspace_bytes(0, 64) == 0


C_PROGRAM = """
#include <stdio.h>
#include "sfp8.h"
typedef void (*any_fn)(void);
int main(void) {
  const any_fn fns[] = {
      (any_fn)sfp8_prepare_gated_weight_24, (any_fn)sfp8_gated_linear,
      (any_fn)sfp8_gated_linear_workspace_bytes, (any_fn)sfp8_gated_linear_quant,
      (any_fn)sfp8_gated_linear_quant_workspace_bytes, (any_fn)sfp8_sparse_linear_backward,
      (any_fn)sfp8_sparse_linear_backward_workspace_bytes, (any_fn)sfp8_gated_linear_backward,
      (any_fn)sfp8_gated_linear_backward_workspace_bytes, (any_fn)sfp8_layernorm,
      (any_fn)sfp8_layernorm_backward, (any_fn)sfp8_layernorm_backward_workspace_bytes};
  for (size_t i = 0; i < sizeof(fns) / sizeof(fns[0]); ++i)
    if (fns[i] == NULL) return 1;
  if (sfp8_gated_linear(NULL, SFP8_E4M3, NULL, 1, NULL, SFP8_E4M3, NULL, 8, 128, SFP8_ACT_GELU,
                        NULL, NULL, NULL, 0, NULL) != SFP8_ERR_INVALID_ARG)
    return 2;
  if (sfp8_layernorm(NULL, SFP8_BF16, 0, 64, 64, NULL, NULL, SFP8_F32, 1e-5f, NULL, NULL,
                     SFP8_E4M3, NULL, NULL, NULL, NULL) != SFP8_OK)
    return 3;
  printf("abi ok\\n");
  return 0;
}
"""


def test_from_plain_c(lib, tmp_path):
    src, exe = tmp_path / "ffn.c", tmp_path / "ffn"
    src.write_text(C_PROGRAM)
    so = binding.library_path()
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-I",
                    os.path.join(ROOT, "include"), str(src), so, "-o", str(exe),
                    "-Wl,-rpath," + os.path.dirname(so)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout == "abi ok\n", (out.returncode, out.stdout)


def test_layernorm_to_codes_wants_aligned_parameters(lib):
    """Codes are made 16 bytes at a time only: what is aligned to its element
    alone is refused, as the header says."""
    good = dict(x=FAKE, dtype=BF16, rows=4, cols=64, ld=64, weight=None, bias=None, p_dtype=F32,
                eps=1e-5, y=None, q=ctypes.c_void_p(0x20000), q_dtype=E4M3,
                scales=ctypes.c_void_p(0x30000), mean=None, rstd=None, stream=None)
    f = lib.sfp8_layernorm
    for name in ("x", "y", "q", "weight", "bias"):
        assert call(f, good, **{name: ctypes.c_void_p(0x40008)}) == MISALIGNED
    assert call(f, good, ld=68) == MISALIGNED
