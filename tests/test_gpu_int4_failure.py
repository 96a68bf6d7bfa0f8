"""Failure detection of the INT4 decode, on the GPU, without faulting it: the test hook makes the next decode leave one bulk
copy unissued, so a bounded wait runs out; the kernel records it, lets its other copies land and returns, and the next call
is right again."""
import numpy as np
import pytest
import torch

from bit_kv_cache_13_gb300 import _lib
from test_gpu_int4 import _Case

pytestmark = pytest.mark.gpu
# one kernel; three, with several CTAs a unit; three, every CTA through several units
FORMS = [(2, [700], 0), (2, [700, 300, 40], 3), (8, [33 + (211 * i) % 900 for i in range(25)], 0), (2, [900, 20, 500], 1)]


@pytest.mark.parametrize("g", [4, 8])
@pytest.mark.parametrize("h_kv,ctxs,splits", FORMS)
@pytest.mark.parametrize("decay", [None, 1.0])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(g, h_kv, ctxs, splits, decay):
    c = _Case(g * h_kv, h_kv, ctxs, seed=8)
    ws = torch.zeros(_lib.kvq_int4_workspace_bytes(c.B, c.h_q, h_kv, c.P, splits, True), dtype=torch.uint8, device="cuda")
    good, w_good = c.run(splits, decay, ws=ws)
    assert c.status == 0
    _lib.kvq_debug_drop_next_copy()
    bad, w_bad = c.run(splits, decay, ws=ws)          # returns: the kernel gave up on its own
    assert c.status == -4                                # KVQ_ERR_CUDA
    assert "timed out" in _lib.load().kvq_last_error().decode()
    assert np.isfinite(bad).all() and not np.array_equal(bad, good)
    assert np.array_equal(bad[-1], good[-1]) or c.B == 1  # (what other CTAs did is whole)
    if decay is not None:
        # tokens that were not attended draw no weight; the others' add up to one for each query head (or to nothing,
        # where a head lost every page)
        drawn = (w_bad - c.w0).sum(-1)
        assert np.all(np.minimum(np.abs(drawn), np.abs(drawn - g)) < 1e-3), drawn   # (fp32 entries below 2, 2^-24 each)
        assert np.array_equal(w_bad[-1], w_good[-1]) or c.B == 1
    again, w_again = c.run(splits, decay, ws=ws)      # the hook is one-shot, tickets and workspace are as before
    assert c.status == 0 and np.array_equal(again, good)
    assert decay is None or np.array_equal(w_again, w_good)
