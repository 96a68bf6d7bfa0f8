"""GPU parity of the INT4 decode where a CTA walks through many (sequence, KV head) units while its rings wrap: several
times as many units as SMs, of one page to over a hundred, and long ones next to short ones in a given split."""
import numpy as np
import pytest

from oracle import int4
from test_gpu_int4 import _Case, _bf, _rot

pytestmark = pytest.mark.gpu


class _Ragged(_Case):
    """A pool of just the pages in use; what lies past a context in its last page is NaN."""

    def __init__(self, h_q, h_kv, ctxs, seed=0):
        rng = np.random.default_rng([seed, h_q, h_kv, len(ctxs)])
        self.B, self.h_q, self.h_kv = len(ctxs), h_q, h_kv
        self.ctx = np.array(ctxs, np.int32)
        used = (self.ctx + 15) // 16
        self.P, self.num_pages = int(used.max()), int(used.sum())
        self.bt = np.full((self.B, self.P), -1, np.int32)
        order, at = rng.permutation(self.num_pages), 0
        for b, n in enumerate(used):
            self.bt[b, :n] = order[at:at + n]
            at += n
        self.rk, self.rv = _rot(rng, h_kv), _rot(rng, h_kv)
        self.cache = int4.new_cache(self.num_pages, h_kv)
        for side in (0, 1):
            for s in range(16):
                x = rng.standard_normal((self.num_pages, h_kv, 128), np.float32) * rng.uniform(0.3, 2, (self.num_pages, 1, 1))
                int4.write_tokens(self.cache, side, s, *int4.quantize(x))
        self.gpu = self.cache.copy()
        nan = np.full((h_kv, 4), np.nan, np.float16)
        for b, n in enumerate(self.ctx):
            for s in range(int(n) % 16, 16 if n % 16 else 0):
                for side in (0, 1):
                    int4.write_tokens(self.gpu[self.bt[b, n // 16]], side, s, np.full((h_kv, 128), 15, np.uint8), nan, nan)
        self.q = _bf(rng.standard_normal((self.B, h_q, 128)) * 2.5)
        self.w0 = rng.random((self.B, h_kv, self.P * 16)).astype(np.float32)


# 60 x 8 units: of 1, 2, 30, 7, 110, 1 pages, some empty
MANY = [[1, 20, 470, 101, 1751, 16, 0, 5, 480, 48][(3 * i) % 10] for i in range(60)]
# 12 x 3 units: most of 81 pages, two long ones, so that a CTA's equal share holds three and more whole units
LONG = [1290, 1290, 9000, 1281, 1290, 1290, 1296, 1290, 1285, 1290, 9001, 1290]


@pytest.mark.parametrize("g", [4, 8])
@pytest.mark.parametrize("h_kv,ctxs,splits", [(8, MANY, 0), (8, MANY, 1), (3, LONG, 1)], ids=["many", "many-split", "long-split"])
@pytest.mark.parametrize("decay", [None, 0.5])
def test_ctas_of_many_units(g, h_kv, ctxs, splits, decay):
    c = _Ragged(g * h_kv, h_kv, ctxs)
    got, w = c.run(splits, decay)
    assert c.status == 0
    c.check(got, w, decay or 1.0)


@pytest.mark.parametrize("g", [2, 6])
def test_bad_pages_on_the_way(g):
    """Ids outside the pool in several units of a CTA's walk: their tokens are dropped, all others attended."""
    c = _Ragged(g * 8, 8, MANY, seed=1)
    bt = c.bt.copy()
    for (b, p), bad in {(8, 50): -1, (4, 29): c.num_pages, (5, 0): 1 << 30, (14, 0): -7, (18, 109): -1, (30, 0): c.num_pages}.items():
        assert p < (c.ctx[b] + 15) // 16
        bt[b, p] = bad
    got, w = c.run(0, 1.0, bt=bt)
    assert c.status == -5
    c.check(got, w, bt=bt)
