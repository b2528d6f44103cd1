"""The residual-block operators (include/delta_block.h) at the edges of their contracts: state in place over
many tiles, values whose intermediate products leave float32's range, gates above 1, NaN gates, rows that
workgroups walk over.  Oracle, inputs and bounds as in test_block_gpu.py.
"""
import numpy as np
import pytest

import test_block_gpu as T
from oracle import block as Bk
from parity import say, to_dev
from test_block_gpu import GATES, HALF, U, check, draw, half_step, host, log_gates

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import chunkwise_delta_rule_chunked_amd as D  # noqa: E402


@pytest.mark.parametrize("L", [20, 129, 5000])
def test_glr_in_place_equals_out_of_place(L):
    """h_final over h0: only a chain's first tile reads the start state, its last one overwrites it."""
    B, H, d = 2, 3, 48
    say("glr in place", L)
    x, g, h0 = (to_dev(v, "f32") for v in (draw(1, (B, L, H, d)), log_gates(2, (B, L, H, d)), draw(3, (B, H, d))))
    O, h, st = D.fwd_glr(x, g, h0, input_gate="norm", want_states=True)
    for _ in range(3):
        s = h0.clone()
        Oi, hi, sti = D.fwd_glr(x, g, s, input_gate="norm", h_final=s, want_states=True)
        assert hi is s and torch.equal(Oi, O) and torch.equal(s, h) and torch.equal(sti, st)
