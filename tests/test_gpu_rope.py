"""GPU parity of the append with norms and position rotation: q_out and k_out are the real numbers' nearest bf16 values, and
the cache bytes those of kvq_append_int4 on k_out."""
import numpy as np
import pytest
import torch

from bit_kv_cache_13_gb300 import _lib, inputs
from oracle import int4

pytestmark = pytest.mark.gpu
EPS = 1e-6


def _rot(rng, h):
    return np.stack([np.linalg.qr(rng.standard_normal((128, 128)))[0] for _ in range(h)]).astype(np.float32)


class Setup:
    def __init__(self, n, h_q, h_kv, rot=128, norm=True, interleaved=False, fused=True, seed=0, scale=None, max_pos=5000):
        rng = self.rng = np.random.default_rng(seed + n)
        self.n, self.h_q, self.h_kv, self.interleaved = n, h_q, h_kv, interleaved
        x = rng.standard_normal((n, h_q + 2 * h_kv, 128)) * np.where(rng.random((h_q + 2 * h_kv, 128)) < 0.03, 20.0, 1.0)
        if scale is not None:
            x = x * scale
        self.qkv = torch.as_tensor(x, dtype=torch.float32).bfloat16().cuda()
        parts = self.qkv.split([h_q, h_kv, h_kv], 1)
        self.q, self.k, self.v = parts if fused else [p.contiguous() for p in parts]
        self.table = inputs.rope_table(max_pos, rot, 1e6).cuda()
        self.pos = torch.as_tensor(rng.integers(0, max_pos, n), dtype=torch.int32).cuda()
        w = lambda: torch.as_tensor(1 + 0.3 * rng.standard_normal(128), dtype=torch.float32).bfloat16().cuda()  # noqa: E731
        self.qw, self.kw = (w(), w()) if norm else (None, None)
        self.mu = torch.as_tensor(rng.standard_normal((h_kv, 128)), dtype=torch.float32).cuda()
        self.rk, self.rv = (torch.as_tensor(_rot(rng, h_kv)).cuda() for _ in range(2))
        self.pages = (n + 15) // 16 + 1
        self.slots = torch.as_tensor(rng.permutation(self.pages * 16)[:n], dtype=torch.int32).cuda()
        self.cache = torch.as_tensor(rng.integers(0, 256, (self.pages, h_kv, 2560)), dtype=torch.uint8).cuda()
        self.q_out = torch.full((n, h_q, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        self.k_out = torch.full((n, h_kv, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(self, **kw):
        a = dict(q=self.q, k=self.k, v=self.v, q_out=self.q_out, k_out=self.k_out, clip=1.0, eps=EPS) | kw
        _lib.kvq_append_rope_int4(a["q"], a["k"], a["v"], self.pos, self.table, self.slots, self.mu, self.rk, self.rv, self.cache,
                                  self.pages, a["q_out"], a["k_out"], self.qw, self.kw, a["eps"], self.interleaved, a["clip"], self.err)

    def check(self, clip=1.0, eps=EPS):
        start = self.cache.clone()
        want = {}
        for name, x, w in (("q", self.q, self.qw), ("k", self.k, self.kw)):
            y = int4.norm_rope(x.double().cpu().numpy(), self.pos.cpu().numpy(), self.table.cpu().numpy(),
                               None if w is None else w.double().cpu().numpy(), eps, self.interleaved)
            want[name] = int4.to_bf16(y)
        self.call(clip=clip, eps=eps)
        torch.cuda.synchronize()
        for name, got in (("q", self.q_out), ("k", self.k_out)):
            bad = np.argwhere(got.double().cpu().numpy() != want[name])
            assert len(bad) == 0, (name, len(bad), bad[:5].tolist())
        # the cache: the plain append of k_out and v, where positions are good
        slots = torch.where((self.pos >= 0) & (self.pos < self.table.shape[0]), self.slots, torch.full_like(self.slots, -1))
        _lib.kvq_append_int4(self.k_out, self.v.contiguous(), slots, self.mu, self.rk, self.rv, start, self.pages, clip)
        assert torch.equal(start, self.cache)


@pytest.mark.parametrize("n,h_q,h_kv", [(1, 32, 8), (1, 1, 1), (2, 5, 1), (7, 64, 8), (33, 12, 2), (129, 9, 3), (700, 4, 1), (300, 32, 8)])
@pytest.mark.parametrize("rot,norm,interleaved,fused", [(128, True, False, True), (128, False, False, False), (64, True, True, True),
                                                        (128, False, True, True), (96, True, False, False), (16, False, False, True),
                                                        (48, True, True, False)])
def test_rounded_values_and_cache_bytes(n, h_q, h_kv, rot, norm, interleaved, fused):
    Setup(n, h_q, h_kv, rot, norm, interleaved, fused).check(clip=1.0 if n % 2 else 0.9)


def test_one_norm_alone():
    for drop in ("qw", "kw"):
        s = Setup(40, 8, 2)
        setattr(s, drop, None)
        s.check()


@pytest.mark.parametrize("n,h_q,h_kv", [(40, 5, 1), (3, 7, 3), (500, 9, 3)])
def test_one_norm_alone_where_a_query_shares_its_warp_with_a_key(n, h_q, h_kv):
    """An odd number of query heads: the last one and the first key are one warp's two rows."""
    for drop in ("qw", "kw"):
        for scale in (None, 1e-25):
            s = Setup(n, h_q, h_kv, scale=scale)
            setattr(s, drop, None)
            s.check(eps=EPS if scale is None else 0.0)


@pytest.mark.parametrize("scale", [1e-30, 1e-18, 1e-6, 1e8, 1e18, 1e30])
@pytest.mark.parametrize("norm", [True, False])
def test_values_of_any_size(scale, norm):
    """eps = 0 norms them all to the same size; without a norm the outputs are as small or large (large groups saturate)."""
    Setup(50, 4, 2, norm=norm, scale=scale).check(eps=0.0 if norm else EPS)


def test_mixed_sizes_within_a_head():
    for norm in (True, False):
        s = Setup(64, 4, 1, norm=norm, seed=3)
        x = s.qkv.float() * torch.as_tensor(10.0 ** s.rng.uniform(-25, 8, s.qkv.shape), dtype=torch.float32).cuda()
        x[:, :, 5] = 0.0
        s.qkv.copy_(x.bfloat16())
        s.check()


def test_far_positions_and_the_tables_own_scaling():
    s = Setup(60, 8, 2, max_pos=1000)
    s.table = inputs.rope_table(131072 + 50, 128, 1e6, factor=4.0).cuda()
    s.pos = torch.arange(131072 - 20, 131072 + 40, dtype=torch.int32, device="cuda")
    s.check()


def test_positions_outside_the_table():
    for n in (9, 500):   # both appends
        s = Setup(n, 4, 1)
        s.pos[2], s.pos[4], s.pos[6], s.pos[7] = -1, 5000, 2 ** 31 - 1, -2 ** 31
        s.slots[4], s.slots[1], s.slots[3] = -1, -1, s.pages * 16
        s.check()
        assert s.err.item() == 4     # 2, 6, 7, and 3 for its slot; 4 is padding
        assert not s.q_out[[2, 4, 6, 7]].any() and not s.k_out[[2, 4, 6, 7]].any()


def test_zeros_nan_and_infinities():
    s = Setup(20, 4, 2, norm=False)
    s.qkv[3] = 0.0
    s.qkv[5, :, 10] = float("nan")
    s.qkv[6, 0, 100] = float("inf")
    s.call()
    bad = torch.isnan(s.q_out) | torch.isinf(s.q_out)
    assert not s.q_out[3].any() and not s.k_out[3].any()
    assert bad[5, :, [10, 74]].all() and bad[6, 0, [36, 100]].all()
    bad[5, :, [10, 74]] = False
    bad[6, 0, [36, 100]] = False
    assert not bad.any()


def test_in_place_and_refused_overlaps():
    a, b = Setup(33, 8, 2, fused=False), Setup(33, 8, 2, fused=False)
    a.call()
    b.call(q_out=b.q, k_out=b.k)
    assert torch.equal(a.q_out, b.q) and torch.equal(a.k_out, b.k) and torch.equal(a.cache, b.cache)
    one = Setup(1, 4, 1)   # a single token's view is dense
    two = Setup(1, 4, 1)
    one.call()
    two.call(q_out=two.q, k_out=two.k)
    assert torch.equal(one.q_out, two.q) and torch.equal(one.k_out, two.k)
    for kw in (dict(k_out=b.v), dict(q=b.qkv[:, :8], q_out=b.qkv.view(-1)[: 33 * 8 * 128].view(33, 8, 128))):
        with pytest.raises(_lib.KvqError, match="overlap"):
            b.call(**kw)


def test_bytes_do_not_depend_on_the_calls_size():
    """The same tokens in one call and in pieces: both appends, the same cache and outputs."""
    a, b = Setup(600, 4, 2, seed=9), Setup(600, 4, 2, seed=9)
    a.call()
    at = 0
    for n in (1, 2, 60, 250, 287):
        sl = slice(at, at + n)
        _lib.kvq_append_rope_int4(b.q[sl], b.k[sl], b.v[sl], b.pos[sl], b.table, b.slots[sl], b.mu, b.rk, b.rv, b.cache, b.pages,
                                  b.q_out[sl], b.k_out[sl], b.qw, b.kw, EPS)
        at += n
    assert at == 600 and torch.equal(a.cache, b.cache) and torch.equal(a.q_out, b.q_out) and torch.equal(a.k_out, b.k_out)


def test_captured_and_replayed_on_another_stream_with_other_inputs():
    for n in (1, 70, 700):
        a, b = Setup(n, 7, 3, seed=1), Setup(n, 7, 3, seed=2)
        b.slots.copy_(a.slots)
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            a.call()
            side.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                a.call()
        for x in ("qkv", "pos", "qw", "kw", "mu", "rk", "rv", "cache"):
            getattr(a, x).copy_(getattr(b, x))
        a.pos[n // 2] = b.pos[n // 2] = 10 ** 6      # a bad position in the replay
        for _ in range(2):
            g.replay()
        torch.cuda.synchronize()
        b.check()
        assert torch.equal(a.q_out, b.q_out) and torch.equal(a.k_out, b.k_out) and torch.equal(a.cache, b.cache)
        assert a.err.item() == 2 and b.err.item() == 1


def test_two_streams_at_once():
    s = [Setup(300, 8, 2, seed=i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in s]
    torch.cuda.synchronize()
    start = [x.cache.clone() for x in s]
    torch.cuda.synchronize()
    for _ in range(4):
        for x, stream in zip(s, streams):
            with torch.cuda.stream(stream):
                x.call()
    torch.cuda.synchronize()
    for x, y in zip(s, start):
        got = x.q_out.clone(), x.k_out.clone(), x.cache.clone()
        x.cache.copy_(y)
        x.check()
        assert torch.equal(got[0], x.q_out) and torch.equal(got[1], x.k_out) and torch.equal(got[2], x.cache)
