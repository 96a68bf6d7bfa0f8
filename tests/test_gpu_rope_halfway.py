"""Normed values next to half-way between two bf16 numbers."""
import numpy as np
import pytest

from bit_kv_cache_13_gb300 import _lib
from oracle import int4
from test_gpu_rope import Setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps", [0.01, 1e-4, 1e-6, 0.25])
def test_heads_far_below_eps_go_to_one_of_the_two_nearest(eps):
    """1 / sqrt(eps) is a round number, so that x * weight / sqrt(eps) is often half-way to 2^-53.  Whatever side is taken,
    the distance stays within half a step and 2^-42, and does not depend on the call's size."""
    a, b = (Setup(600, 5, 2, rot=64, seed=4, scale=1e-9) for _ in range(2))
    a.call(eps=eps)
    for i in range(0, 600, 200):
        part = slice(i, i + 200)
        _lib.kvq_append_rope_int4(b.q[part], b.k[part], b.v[part], b.pos[part], b.table, b.slots[part], b.mu, b.rk, b.rv, b.cache,
                                  b.pages, b.q_out[part], b.k_out[part], b.qw, b.kw, eps)
    assert (a.q_out == b.q_out).all() and (a.k_out == b.k_out).all() and (a.cache == b.cache).all()
    for x, w, got in ((a.q, a.qw, a.q_out), (a.k, a.kw, a.k_out)):
        y = int4.norm_rope(x.double().cpu().numpy(), a.pos.cpu().numpy(), a.table.cpu().numpy(), w.double().cpu().numpy(), eps)
        half = np.ldexp(1.0, np.frexp(y)[1] - 9)
        size = np.abs(x.double().cpu().numpy()).max(-1, keepdims=True) * float(w.double().abs().max()) / np.sqrt(eps)   # of any term
        assert (np.abs(got.double().cpu().numpy() - y) <= half + 2.0 ** -41 * size).all()
