"""Host-side checks of include/delta_linear.h's workspaces (no GPU needed)."""
import ctypes

import pytest

import chunkwise_delta_rule_chunked_amd as D
from test_linear_host import bwd, lib, no_gpu, shape, size  # noqa: F401

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("gate", [1, 2])
@pytest.mark.parametrize("dv", [32, 160])
def test_a_call_without_gates_gradients_takes_the_size_without_gates(lib, no_gpu, monkeypatch, gate, dv):  # noqa: F811
    sh = shape(L=5000, dv=dv)
    none, full = (size("delta_bwd_lin_workspace_bytes", ctypes.byref(sh), 3, g)[1] for g in (0, gate))
    assert none < full
    monkeypatch.setenv("DELTA_FAULT", "launch")           # -7: every check passed
    assert bwd(sh, gate=gate, dg=None, wbytes=none) == -7 and bwd(sh, gate=gate, dg=None, wbytes=none - 1) == -5
    assert bwd(sh, gate=gate, wbytes=full) == -7 and bwd(sh, gate=gate, wbytes=full - 1) == -5


@pytest.mark.parametrize("dtype", [D.F32, D.BF16])
@pytest.mark.parametrize("B,Hk,H,dk,dv", [(3, 6, 6, 64, 80), (1, 16, 16, 128, 128), (2, 8, 16, 128, 256), (1, 1, 1, 16, 16), (9, 1, 7, 32, 48),
                                          (8, 16, 16, 128, 128), (20, 1, 4, 64, 144)])
def test_workspaces_never_fall_with_the_length(lib, no_gpu, monkeypatch, B, Hk, H, dk, dv, dtype):  # noqa: F811
    """A workspace for the longest sequence serves every shorter one."""
    at = lambda fn, L, *gate: size(fn, ctypes.byref(shape(B=B, L=L, H=H, dk=dk, dv=dv, dtype=dtype)), Hk, *gate)[1]
    lengths = list(range(0, 700, 13)) + list(range(700, 9000, 190)) + [20000, 65536, 65537, 1 << 20]
    for args in (("delta_fwd_lin_workspace_bytes",), *(("delta_bwd_lin_workspace_bytes", g) for g in range(3))):
        sizes = [at(args[0], L, *args[1:]) for L in lengths]
        assert sizes == sorted(sizes), (args, [(a, b, x, y) for a, b, x, y in zip(lengths, lengths[1:], sizes, sizes[1:]) if y < x])
