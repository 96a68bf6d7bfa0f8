"""Calls of the INT4 decode that its documentation allows and that are easy to get wrong: the output in the query's place,
pages that sequences share, two streams at once, graphs with a workspace each, a batch of thousands."""
import numpy as np
import pytest
import torch

from bit_kv_cache_13_gb300 import _lib
from test_gpu_int4 import SCALE, _Case, _dev
from test_gpu_int4_segments import _Ragged

pytestmark = pytest.mark.gpu


class _Bound:
    """A case's tensors on the device, a workspace and an output of its own."""

    def __init__(self, c, splits=0, decay=None, out=None):
        self.c, self.splits, self.decay = c, splits, decay
        self.args = [c.q.cuda(), _dev(c.gpu), c.num_pages, _dev(c.bt), _dev(c.ctx), _dev(c.rk), _dev(c.rv), SCALE]
        self.out = torch.full_like(self.args[0], float("nan"))
        self.w = _dev(c.w0.copy())
        self.ws = torch.zeros(_lib.kvq_int4_workspace_bytes(c.B, c.h_q, c.h_kv, c.P, splits, decay is not None),
                              dtype=torch.uint8, device="cuda")

    def __call__(self, out=None, stream=None):
        out = self.out if out is None else out
        if self.decay is None:
            _lib.kvq_decode_attn_int4(*self.args, out, self.ws, self.splits, stream=stream)
        else:
            _lib.kvq_decode_attn_int4_weights(*self.args, out, self.w, self.decay, self.ws, self.splits, stream=stream)

    def check(self, out=None, times=1):
        assert _lib.kvq_workspace_status(self.ws) == 0
        out = self.out if out is None else out
        self.c.check(out.double().cpu().numpy(), self.w.double().cpu().numpy() if self.decay is not None and times == 1 else None)


@pytest.mark.parametrize("g", [4, 8])
@pytest.mark.parametrize("h_kv,ctxs,splits", [(2, [700], 0), (2, [700, 0, 300], 3), (8, [40 * i for i in range(24)], 0)])
@pytest.mark.parametrize("decay", [None, 1.0])
def test_output_in_the_querys_place(g, h_kv, ctxs, splits, decay):
    b = _Bound(_Case(g * h_kv, h_kv, ctxs, seed=9), splits, decay)
    b(out=b.args[0])
    torch.cuda.synchronize()
    b.check(b.args[0])


@pytest.mark.parametrize("splits", [0, 2])
def test_pages_that_sequences_share(splits):
    """A common prefix of 20 pages, one page twice in a sequence."""
    c = _Ragged(16, 2, [900, 700, 330], seed=3)
    c.bt[1, :20], c.bt[2, :20] = c.bt[0, :20], c.bt[0, :20]
    c.bt[1, 21] = c.bt[1, 22]
    b = _Bound(c, splits, 1.0)
    b()
    torch.cuda.synchronize()
    b.check()


@pytest.mark.parametrize("captured", [False, True])
def test_two_at_once(captured):
    """Two batches on two streams (or as two graphs replayed on them), each with a workspace of its own, over and over."""
    pair = [_Bound(_Case(32, 8, [1500, 90, 700], seed=10), 0), _Bound(_Case(16, 4, [3000], seed=11), 0)]
    streams = [torch.cuda.Stream() for _ in pair]
    torch.cuda.synchronize()
    runs = []
    for b, s in zip(pair, streams):
        if captured:
            b()
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                b()
            runs.append(graph.replay)
        else:
            runs.append(lambda b=b, s=s: b(stream=s))
    for b in pair:
        b.out.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(20):
        for run, s in zip(runs, streams):
            with torch.cuda.stream(s):
                run()
    torch.cuda.synchronize()
    for b in pair:
        b.check()


@pytest.mark.parametrize("decay", [None, 1.0])
def test_a_batch_of_thousands(decay):
    rng = np.random.default_rng(12)
    c = _Ragged(4, 2, list(rng.integers(0, 60, 2100)) + [5000, 1], seed=4)
    b = _Bound(c, 0, decay)
    b()
    torch.cuda.synchronize()
    b.check()
