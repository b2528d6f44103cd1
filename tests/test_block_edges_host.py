"""Host-side checks of include/delta_block.h at the edges of what it says (no GPU needed), in the manner of
test_block_host.py."""
import ctypes

import chunkwise_delta_rule_chunked_amd as D
from test_block_host import EPS, fake, lib, no_gpu, size  # noqa: F401  (fixtures)


def test_rmsnorm_bwd_without_dweight_needs_no_workspace(lib, no_gpu, monkeypatch):  # noqa: F811
    f = [fake(i) for i in range(6)]
    call = lambda dw, ws, n: D.load_library().delta_layer_rmsnorm_bwd(4, 100, D.BF16, EPS, f[0], f[1], f[2], f[3], f[4], dw, ws,
                                                                      ctypes.c_size_t(n), None)
    assert call(f[5], None, 0) == -5
    monkeypatch.setenv("DELTA_FAULT", "launch")              # what passes all checks ends with DELTA_ERR_HIP
    assert call(None, None, 0) == -7 and call(f[5], fake(6), 1 << 20) == -7
    assert call(None, f[4], 1 << 20) == -7                   # nothing of it is written, so it may lie anywhere
