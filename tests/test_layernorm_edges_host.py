"""Host-side checks of include/delta_layernorm.h at its largest sizes (no GPU needed)."""
import ctypes

import pytest

import chunkwise_delta_rule_chunked_amd as D
from test_layernorm_host import bwd, drop, fwd, lib, no_gpu  # noqa: F401

torch = pytest.importorskip("torch")
TOP = (1 << 34) - 1024   # vectors of eight channels


def dropout(rows, width, dtype=D.BF16):
    """y over x, no residual: with fake addresses far from everything."""
    return D.load_library().delta_layer_dropout(rows, width, dtype, drop(0.1), ctypes.c_void_p(1 << 44), None, ctypes.c_void_p(1 << 44), None)


@pytest.mark.parametrize("rows,width,fits", [
    (TOP >> 3, 64, True), ((TOP >> 3) + 1, 64, False), ((1 << 31) - 1, 57, False), ((1 << 31) - 1, 1 << 20, False), ((1 << 31) - 1, 56, True),
    ((1 << 31) - 1, 1, True), (TOP // (1 << 17), 1 << 20, True), ((1 << 17), 1 << 20, False)])
def test_dropout_refuses_what_one_launch_does_not_reach(lib, no_gpu, monkeypatch, rows, width, fits):  # noqa: F811
    monkeypatch.setenv("DELTA_FAULT", "launch")           # -7: every check passed
    assert dropout(rows, width) == (-7 if fits else -2)


def test_the_norms_walk_over_any_number_of_rows(lib, no_gpu, monkeypatch):  # noqa: F811
    monkeypatch.setenv("DELTA_FAULT", "launch")
    far = lambda i: ctypes.c_void_p((i + 1) << 55)      # further apart than 2^53 bytes
    top = (1 << 31) - 1
    assert fwd(rows=top, width=1 << 20, x=far(0), r=far(1), sum=far(4), y=far(5)) == -7
    assert bwd(rows=top, width=1 << 20, dy=far(0), s=far(1), dsum=far(3), dr=far(4), dx=far(5), dw=None, db=None, ws=None, wbytes=0) == -7
