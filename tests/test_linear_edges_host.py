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
