"""Host-side checks of include/delta_block.h at the edges of what it says (no GPU needed), in the manner of
test_block_host.py."""
import ctypes
import random

import chunkwise_delta_rule_chunked_amd as D
from test_block_host import EPS, fake, lib, no_gpu, size, table  # noqa: F401  (fixtures)


def test_rmsnorm_bwd_without_dweight_needs_no_workspace(lib, no_gpu, monkeypatch):  # noqa: F811
    f = [fake(i) for i in range(6)]
    call = lambda dw, ws, n: D.load_library().delta_layer_rmsnorm_bwd(4, 100, D.BF16, EPS, f[0], f[1], f[2], f[3], f[4], dw, ws,
                                                                      ctypes.c_size_t(n), None)
    assert call(f[5], None, 0) == -5
    monkeypatch.setenv("DELTA_FAULT", "launch")              # what passes all checks ends with DELTA_ERR_HIP
    assert call(None, None, 0) == -7 and call(f[5], fake(6), 1 << 20) == -7
    assert call(None, f[4], 1 << 20) == -7                   # nothing of it is written, so it may lie anywhere


def test_clip_workspace_goes_by_the_tensors(lib):  # noqa: F811
    """The same total in one tensor and in many needs different sizes; more tensors or longer ones never need
    less."""
    def need(sizes):
        n, _, s, _ = table(sizes)
        rc, b = size("delta_grad_norm_workspace_bytes", n, s)
        assert rc == 0
        return b

    assert need([1000]) < need([1] * 1000)
    rng = random.Random(3)
    for _ in range(200):
        sizes = [rng.choice([0, 1, 5000, 16384, 16385, 10 ** 6, 10 ** 8]) for _ in range(rng.randint(1, 250))]
        i = rng.randrange(len(sizes))
        more = sizes[:i] + [sizes[i] + rng.choice([1, 16384, 10 ** 7])] + sizes[i + 1:]
        assert need(sizes) <= need(more) and need(sizes) <= need(sizes + [rng.choice([0, 3, 10 ** 6])])


def test_error_texts_name_what_these_entry_points_refuse():
    """delta_fwd_glr refuses a g_log at 4 bytes, delta_clip_grads a negative max_norm, and so on."""
    assert "max_norm" in D.strerror(-2) and "eps" in D.strerror(-2)
    assert "input gate" in D.strerror(-3) and "group" in D.strerror(-3)
    assert "g_log of the delta rule" in D.strerror(-4) and "gradient" in D.strerror(-4)
