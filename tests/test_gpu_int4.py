"""GPU parity of the INT4 cache (append, read-back, decode attention, accumulated token weights) against the fp64 oracle.

Tolerances, each from the arithmetic:
* cache bytes and read-back values are equal (codes are decided as the exact rotated vectors decide them).
* out, per query head, in the 2-norm (the output rotation is orthogonal, so it keeps the norm of an error): the bf16
  rounding is at most 2^-8 of each value; p and p * scale are rounded to fp16 at most once each, 2^-11 of a term each, so
  2^-10 of sum_s p_s (15 scale_s + |min_s|) per channel; fp32 sums and logits add at most 2^-12 of the same.
* weights: a logit is an fp32 sum whose terms are bounded by a = sum_i |q'_i| (15 scale + |min|) * scale; chains of fewer
  than 64 roundings of 2^-24 leave 2^-18 a, which p takes as a relative error; 2^-18 more for exp2, the sums and the
  normaliser, and 2^-22 of the entry for its own update (a product, a sum and the oracle's exact fp32 input).
"""
import numpy as np
import pytest
import torch

from bit_kv_cache_13_gb300 import _lib, inputs
from bit_kv_cache_13_gb300.workload import Int4Layer
from oracle import int4

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


def _dev(x, dtype=None):
    return torch.as_tensor(x, dtype=dtype, device="cuda").contiguous()


def _rot(rng, h):
    return np.stack([np.linalg.qr(rng.standard_normal((128, 128)))[0] for _ in range(h)]).astype(np.float32)


def _bf(x):
    return torch.as_tensor(np.asarray(x, np.float32)).to(torch.bfloat16)


def _append(k, v, slots, mu, rk, rv, cache, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    _lib.kvq_append_int4(k.cuda(), v.cuda(), _dev(slots, torch.int32), _dev(mu), _dev(rk), _dev(rv), cache, cache.shape[0],
                         err_count=err, **kw)
    torch.cuda.synchronize()
    return int(err.item())


@pytest.mark.parametrize("n,h_kv,clip", [(1, 1, 1.0), (3, 8, 1.0), (17, 2, 0.9), (100, 1, 1.0), (255, 3, 1.0), (256, 1, 0.75),
                                         (300, 2, 1.0), (1031, 1, 1.0), (501, 1, 0.75), (64, 9, 1.0), (3, 200, 1.0)])
def test_append_bytes_and_read_back(n, h_kv, clip):
    rng = np.random.default_rng(n)
    big = np.where(rng.random((h_kv, 128)) < 0.03, 20.0, 1.0)
    mu = (2 * rng.standard_normal((h_kv, 128))).astype(np.float32)
    k, v = _bf(rng.standard_normal((n, h_kv, 128)) * big + mu), _bf(rng.standard_normal((n, h_kv, 128)) * big)
    rk, rv = _rot(rng, h_kv), _rot(rng, h_kv)
    pages = (n + 15) // 16 + 2
    slots = rng.permutation(pages * 16)[:n].astype(np.int32)
    if n > 10:
        slots[3], slots[7], slots[9] = -1, pages * 16, -5   # skipped; outside the pool twice
    start = rng.integers(0, 256, (pages, h_kv, 2560)).astype(np.uint8)
    cache = _dev(start.copy())
    assert _append(k, v, slots, mu, rk, rv, cache, clip=clip) == (2 if n > 10 else 0)
    want = start.copy()
    int4.append(want, k.double().numpy(), v.double().numpy(), slots, mu, rk, rv, clip)
    assert np.array_equal(cache.cpu().numpy(), want)     # and every other slot's bytes as they were
    kr, vr = (torch.full((n, h_kv, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    _lib.kvq_dequant_int4(cache, pages, h_kv, _dev(slots), kr, vr)
    ok = (slots >= 0) & (slots < pages * 16)
    at = np.where(ok, slots, 0)
    for side, got in ((0, kr), (1, vr)):
        tok = np.where(ok[:, None, None], int4.values(want, side)[at // 16, :, at % 16], 0.0)
        # one fp32 fma, then one bf16 rounding
        assert torch.equal(got.cpu(), torch.as_tensor(tok.astype(np.float32)).to(torch.bfloat16))


def test_append_adversarial_groups():
    """Identity rotation: exact midpoints, constant groups, saturating and vanishing scales, signed zeros."""
    eye = np.eye(128, dtype=np.float32)[None]
    for n in (40, 500):
        k = torch.randn(n, 1, 128, generator=torch.Generator().manual_seed(0)) * 3
        k[0, 0, :32] = 1.5
        k[1, 0, :32] = torch.tensor([0.0, 15.0] + [i + 0.5 for i in range(15)] * 2)
        k[2, 0, 32:64] = 1e5 * torch.sign(torch.randn(32, generator=torch.Generator().manual_seed(1)))
        k[3, 0, 64:96] = torch.linspace(-1e-8, 1e-8, 32)
        k[4, 0, 96:] = torch.linspace(-1, 1, 32)
        k[5, 0, :64] = -0.0
        k[6] = 0.0
        k[7] = torch.randint(0, 31, (128,), generator=torch.Generator().manual_seed(2)) * 0.5   # many midpoints
        k, v = k.to(torch.bfloat16), (-k).to(torch.bfloat16)
        mu = np.zeros((1, 128), np.float32)
        cache, want = torch.zeros((32, 1, 2560), dtype=torch.uint8, device="cuda"), int4.new_cache(32, 1)
        assert _append(k, v, np.arange(n), mu, eye, eye, cache) == 0
        int4.append(want, k.double().numpy(), v.double().numpy(), np.arange(n), mu, eye, eye)
        assert np.array_equal(cache.cpu().numpy(), want)


def test_append_with_a_large_centre_and_huge_values():
    """Key minus centre cancels to a thousandth of either; values up to the end of the type's range."""
    rng = np.random.default_rng(6)
    for n in (5, 500):
        mu = (300 * rng.standard_normal((1, 128))).astype(np.float32)
        k = _bf(mu[None] + rng.standard_normal((n, 1, 128)))
        v = _bf(rng.standard_normal((n, 1, 128)) * 10.0 ** rng.uniform(-37, 37, (n, 1, 1)))
        rk, rv = _rot(rng, 1), _rot(rng, 1)
        cache, want = torch.zeros((32, 1, 2560), dtype=torch.uint8, device="cuda"), int4.new_cache(32, 1)
        _append(k, v, np.arange(n), mu, rk, rv, cache)
        int4.append(want, k.double().numpy(), v.double().numpy(), np.arange(n), mu, rk, rv)
        assert np.array_equal(cache.cpu().numpy(), want)


def test_token_bytes_do_not_depend_on_their_company():
    """A prompt in one call, in two ragged ones, and token by token: the same cache."""
    rng = np.random.default_rng(9)
    n, h = 700, 2
    k, v = _bf(rng.standard_normal((n, h, 128))), _bf(rng.standard_normal((n, h, 128)) * 5)
    mu, rk, rv = rng.standard_normal((h, 128)).astype(np.float32), _rot(rng, h), _rot(rng, h)
    slots = np.arange(n, dtype=np.int32)
    got = []
    for cuts in ([0, n], [0, 333, n], list(range(0, 64)) + [64, n], [0, 150, 300, 450, 600, n]):
        cache = torch.zeros((44, h, 2560), dtype=torch.uint8, device="cuda")
        for a, b in zip(cuts, cuts[1:]):
            _append(k[a:b], v[a:b], slots[a:b], mu, rk, rv, cache)
        got.append(cache.cpu().numpy())
    assert all(np.array_equal(got[0], x) for x in got[1:])


@pytest.mark.parametrize("n", [2, 400])
def test_append_not_finite(n):
    rng = np.random.default_rng(3)
    k, v = _bf(rng.standard_normal((n, 1, 128))), _bf(rng.standard_normal((n, 1, 128)))
    k[1, 0, 5], v[0, 0, 9] = float("nan"), float("inf")
    mu, r = np.zeros((1, 128), np.float32), _rot(rng, 1)
    cache = torch.zeros((26, 1, 2560), dtype=torch.uint8, device="cuda")
    _append(k, v, np.arange(n), mu, r, r, cache)
    kr, vr = (torch.empty((n, 1, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    _lib.kvq_dequant_int4(cache, 26, 1, torch.arange(n, dtype=torch.int32, device="cuda"), kr, vr)
    assert kr[1].isnan().all() and vr[0].isnan().all()
    assert kr[0].isfinite().all() and vr[1:].isfinite().all() and kr[2:].isfinite().all()


# ------------------------------------------------------------------ decode

class _Case:
    """A filled cache with its oracle copy: random tokens written by the oracle, NaN bytes past every context."""

    def __init__(self, h_q, h_kv, ctxs, max_pages=None, seed=0, q_scale=2.5, stale=True):
        rng = np.random.default_rng([seed, h_q, h_kv, len(ctxs), max(ctxs)])
        self.B, self.h_q, self.h_kv = len(ctxs), h_q, h_kv
        self.P = max_pages or max(1, (max(ctxs) + 15) // 16)
        self.num_pages = self.B * self.P + 3
        self.bt = rng.permutation(self.num_pages)[: self.B * self.P].reshape(self.B, self.P).astype(np.int32)
        self.ctx = np.array(ctxs, np.int32)
        self.rk, self.rv = _rot(rng, h_kv), _rot(rng, h_kv)
        n = self.num_pages * 16
        self.cache = int4.new_cache(self.num_pages, h_kv)
        for side in (0, 1):
            quant = int4.quantize(rng.standard_normal((n, h_kv, 128)) * rng.uniform(0.3, 2, (n, 1, 1)))
            for s in range(16):
                int4.write_tokens(self.cache, side, s, *(x[s::16] for x in quant))
        self.gpu = self.cache.copy()
        if stale:
            nan = np.full((h_kv, 4), np.nan, np.float16)
            for b, used in enumerate(self.ctx):
                for p in range(max(0, int(used)) // 16, self.P):
                    for s in range(max(0, int(used) - 16 * p), 16):
                        for side in (0, 1):
                            int4.write_tokens(self.gpu[self.bt[b, p]], side, s, np.full((h_kv, 128), 15, np.uint8), nan, nan)
        self.q = _bf(rng.standard_normal((self.B, h_q, 128)) * q_scale)
        self.w0 = rng.random((self.B, h_kv, self.P * 16 + 5)).astype(np.float32)

    def run(self, splits=0, decay=None, ctx=None, bt=None, ws=None):
        out = torch.full((self.B, self.h_q, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        if ws is None:
            ws = torch.zeros(_lib.kvq_int4_workspace_bytes(self.B, self.h_q, self.h_kv, self.P, splits, decay is not None),
                             dtype=torch.uint8, device="cuda")
        args = (self.q.cuda(), _dev(self.gpu), self.num_pages, _dev(self.bt if bt is None else bt),
                _dev(self.ctx if ctx is None else ctx), _dev(self.rk), _dev(self.rv), SCALE, out)
        w = None
        if decay is None:
            _lib.kvq_decode_attn_int4(*args, ws, splits)
        else:
            w = _dev(self.w0.copy())
            _lib.kvq_decode_attn_int4_weights(*args, w, decay, ws, splits)
        torch.cuda.synchronize()
        self.status = _lib.kvq_workspace_status(ws)
        return out.double().cpu().numpy(), None if w is None else w.double().cpu().numpy()

    def check(self, got, w=None, decay=1.0, ctx=None, bt=None):
        ctx, bt = self.ctx if ctx is None else ctx, self.bt if bt is None else bt
        ref, wref = int4.decode(self.q.double().numpy(), self.cache, bt, ctx, self.rk, self.rv, SCALE, self.w0, decay)
        g = self.h_q // self.h_kv
        for b in range(self.B):
            n = int(ctx[b])
            if n <= 0:
                assert not got[b].any()
                if w is not None:
                    assert np.array_equal(w[b], self.w0[b].astype(np.float64))
                continue
            pages = bt[b][: (n + 15) // 16]
            ok = (pages >= 0) & (pages < self.num_pages)
            live = np.repeat(ok, 16)[:n]
            for h in range(self.h_kv):
                tiles = self.cache[np.where(ok, pages, 0), h]
                kk = int4.values(tiles, 0).reshape(-1, 128)[:n]
                span = []    # 15 scale + |min| of each token's channels
                for side in (0, 1):
                    sc, mn = (x.astype(np.float64) for x in int4.meta(tiles, side))
                    span.append(np.repeat(15 * sc + np.abs(mn), 32, -1).reshape(-1, 128)[:n])
                err_w = np.zeros(n)
                for j in range(h * g, (h + 1) * g):
                    qr = self.q[b, j].double().numpy() @ self.rk[h].astype(np.float64)
                    a = np.where(live, kk @ qr * SCALE, -np.inf)
                    p = np.exp(a - a.max()) if live.any() else np.zeros(n)
                    p /= max(p.sum(), 1e-300)
                    amax = (span[0][live] @ np.abs(qr)).max() * SCALE if live.any() else 0.0
                    spread = np.linalg.norm(p @ span[1])
                    tol = 2.0 ** -8 * np.linalg.norm(ref[b, j]) + (2.0 ** -10 + 2.0 ** -12 + 2.0 ** -17 * amax) * spread
                    err = np.linalg.norm(got[b, j] - ref[b, j])
                    assert err <= tol, (b, j, err, tol)
                    err_w += p * (2.0 ** -18 * amax * 2 + 2.0 ** -18)
                if w is not None:
                    d = np.abs(w[b, h, :n] - wref[b, h, :n])
                    assert np.all(d <= err_w + 2.0 ** -22 * np.abs(wref[b, h, :n])), (b, h, d.max())
                    assert np.array_equal(w[b, h, n:], self.w0[b, h, n:].astype(np.float64))


CASES = [
    (4, 1, [1], 0), (4, 1, [15], 0), (4, 1, [16, 17], 0), (1, 1, [33], 0), (8, 4, [100, 0, 47], 0), (6, 2, [257], 3),
    (8, 2, [300, 129], 1), (10, 2, [64, 500], 0), (7, 1, [700], 5), (16, 2, [31, 1000], 0), (8, 1, [2049], 0),
    (32, 8, [777], 0), (16, 2, [1600, 3], 9), (3, 3, [50], 254), (64, 8, [90, 260, 1, 0, 33], 0), (4, 1, [9000], 0),
]


@pytest.mark.parametrize("h_q,h_kv,ctxs,splits", CASES)
def test_decode_matches_oracle(h_q, h_kv, ctxs, splits):
    c = _Case(h_q, h_kv, ctxs)
    got, _ = c.run(splits)
    assert c.status == 0
    c.check(got)


@pytest.mark.parametrize("h_q,h_kv,ctxs,splits", CASES)
@pytest.mark.parametrize("decay", [1.0, 0.75])
def test_weights_match_oracle(h_q, h_kv, ctxs, splits, decay):
    c = _Case(h_q, h_kv, ctxs, seed=1)
    got, w = c.run(splits, decay)
    assert c.status == 0
    c.check(got, w, decay)


# batches on both sides of where one kernel's CTAs have a unit each: 160 units; 80 with up to 128 pages; 48 of one page;
# two heads of a long and two short sequences; 152 units (a CTA each)
BATCHES = [(16, 8, [(37 * i) % 130 for i in range(20)]), (8, 4, [(811 * i) % 2047 for i in range(20)]),
           (6, 6, [1 + i % 16 for i in range(8)]), (10, 2, [20000, 17, 0]), (38, 19, [3, 90, 16, 0, 40, 1, 17, 200])]


@pytest.mark.parametrize("h_q,h_kv,ctxs", BATCHES)
@pytest.mark.parametrize("decay", [None, 1.0])
def test_batches_match_oracle(h_q, h_kv, ctxs, decay):
    c = _Case(h_q, h_kv, ctxs, seed=2)
    got, w = c.run(0, decay)
    assert c.status == 0
    c.check(got, w, decay or 1.0)


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("g", [4, 8])
def test_bad_pages_in_a_given_split(g, splits):
    c = _Case(2 * g, 2, [500, 40, 20])
    bt = c.bt.copy()
    bt[0, 3], bt[0, 31], bt[1, :], bt[2, 1] = -1, c.num_pages, 1 << 30, -7   # sequence 1 loses every page
    got, w = c.run(splits, 1.0, bt=bt)
    assert c.status == -5
    c.check(got, w, bt=bt)


@pytest.mark.parametrize("g", [4, 8])
def test_bad_pages_are_dropped_and_reported(g):
    c = _Case(2 * g, 2, [500, 40, 20])
    bt = c.bt.copy()
    bt[0, 3], bt[0, 31], bt[1, :], bt[2, 1] = -1, c.num_pages, 1 << 30, -7   # sequence 1 loses every page
    got, w = c.run(0, 1.0, bt=bt)
    assert c.status == -5
    c.check(got, w, bt=bt)
    assert not got[1].any() and np.array_equal(w[1], c.w0[1].astype(np.float64))


def test_context_lengths_outside_the_table_are_clamped():
    c = _Case(8, 2, [64, 64], stale=False)
    got, w = c.run(0, 1.0, ctx=np.array([1000, -3], np.int32))
    c.check(got, w, ctx=np.array([64, 0], np.int32))


@pytest.mark.parametrize("g", [1, 4, 8])
def test_not_finite_tokens_reach_their_own_rows_only(g):
    nan = np.full(4, np.nan, np.float16)
    for side in (0, 1):
        c = _Case(2 * g, 2, [70, 70], stale=False)
        int4.write_tokens(c.gpu[c.bt[0, 2], 1], side, 3, np.zeros(128, np.uint8), nan, nan)   # sequence 0, KV head 1
        got, w = c.run(0, 1.0)
        clean, wc = _Case(2 * g, 2, [70, 70], stale=False).run(0, 1.0)
        assert np.isnan(got[0, g:]).all()
        if side == 0:
            assert np.isnan(w[0, 1, :70]).all()
        else:
            assert np.array_equal(w[0, 1], wc[0, 1])
        assert np.array_equal(got[0, :g], clean[0, :g]) and np.array_equal(got[1], clean[1])
        assert np.array_equal(w[0, 0], wc[0, 0]) and np.array_equal(w[1], wc[1])


def test_large_and_tiny_queries():
    for q_scale in (60.0, 1e-3, 0.0):
        for g in (4, 7):
            c = _Case(2 * g, 2, [300], q_scale=q_scale)
            got, w = c.run(0, 1.0)
            c.check(got, w)


def test_offsets_past_32_bits():
    """Pages at the far end of a pool of more than 4 GiB."""
    c = _Case(8, 8, [200])
    far = 220_000
    pool = torch.empty((far + c.num_pages, 8, 2560), dtype=torch.uint8, device="cuda")
    pool[far:] = _dev(c.gpu)
    out = torch.empty((1, 8, 128), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(_lib.kvq_int4_workspace_bytes(1, 8, 8, c.P), dtype=torch.uint8, device="cuda")
    _lib.kvq_decode_attn_int4(c.q.cuda(), pool, pool.shape[0], _dev(c.bt + far), _dev(c.ctx), _dev(c.rk), _dev(c.rv), SCALE, out, ws)
    c.check(out.double().cpu().numpy())
    for n in (2, 300):   # and appends there
        k = _bf(np.random.default_rng(0).standard_normal((n, 8, 128)))
        slots = far * 16 + np.random.default_rng(1).permutation(c.num_pages * 16)[:n].astype(np.int32) % (c.num_pages * 16)
        slots = slots[: min(n, c.num_pages * 16)]
        _append(k[: len(slots)], k[: len(slots)], slots, np.zeros((8, 128), np.float32), c.rk, c.rv, pool)
        int4.append(c.gpu, k[: len(slots)].double().numpy(), k[: len(slots)].double().numpy(), slots - far * 16, np.zeros((8, 128)), c.rk, c.rv)
        assert np.array_equal(pool[far:].cpu().numpy(), c.gpu)


def test_graph_replay_on_another_stream():
    c = _Case(16, 4, [333, 90], seed=3, stale=False)
    ws = torch.zeros(_lib.kvq_int4_workspace_bytes(2, 16, 4, c.P, 0, True), dtype=torch.uint8, device="cuda")
    q, cache, bt, ctx, rk, rv = c.q.cuda(), _dev(c.gpu), _dev(c.bt), _dev(c.ctx), _dev(c.rk), _dev(c.rv)
    out, w = torch.empty((2, 16, 128), dtype=torch.bfloat16, device="cuda"), _dev(c.w0.copy())
    call = lambda: _lib.kvq_decode_attn_int4_weights(q, cache, c.num_pages, bt, ctx, rk, rv, SCALE, out, w, 1.0, ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call()
    for lens in ([333, 90], [200, 0]):          # the same graph with other lengths
        ctx.copy_(torch.tensor(lens, dtype=torch.int32))
        w.copy_(_dev(c.w0))
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        s.synchronize()
        c.check(out.double().cpu().numpy(), w.double().cpu().numpy(), ctx=np.array(lens, np.int32))


def test_inputs_written_by_the_kernel_just_before():
    """Kernels of the library may start early: query, rotations, lengths and cache written right before the call count."""
    c = _Case(8, 2, [600], seed=5, stale=False)
    ws = torch.zeros(_lib.kvq_int4_workspace_bytes(1, 8, 2, c.P, 0, True), dtype=torch.uint8, device="cuda")
    real = [c.q.cuda(), _dev(c.gpu), _dev(c.bt), _dev(c.ctx), _dev(c.rk), _dev(c.rv), _dev(c.w0)]
    for _ in range(3):
        buf = [torch.zeros_like(x) for x in real]
        out = torch.empty((1, 8, 128), dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        for x, y in zip(buf, real):
            x.copy_(y)
        _lib.kvq_decode_attn_int4_weights(buf[0], buf[1], c.num_pages, *buf[2:6], SCALE, out, buf[6], 1.0, ws)
        torch.cuda.synchronize()
        c.check(out.double().cpu().numpy(), buf[6].double().cpu().numpy())


@pytest.mark.parametrize("n", [30, 900])
@pytest.mark.parametrize("splits", [0, 2])
def test_a_chain_of_calls_without_a_pause(n, splits):
    """Append, decode, append over the same slots, decode: each call sees the one before, on a stream of its own too."""
    rng = np.random.default_rng(n)
    h, P = 2, (n + 15) // 16
    mu, rk, rv = _dev(rng.standard_normal((h, 128)).astype(np.float32)), _dev(_rot(rng, h)), _dev(_rot(rng, h))
    kv = [(_bf(rng.standard_normal((n, h, 128))).cuda(), _bf(rng.standard_normal((n, h, 128))).cuda()) for _ in range(2)]
    q, slots = _bf(2 * rng.standard_normal((1, 8, 128))).cuda(), torch.arange(n, dtype=torch.int32, device="cuda")
    bt, ctx = torch.arange(P, dtype=torch.int32, device="cuda")[None], torch.tensor([n], dtype=torch.int32, device="cuda")
    cache = torch.zeros((P, h, 2560), dtype=torch.uint8, device="cuda")
    ws = torch.zeros(_lib.kvq_int4_workspace_bytes(1, 8, h, P, splits), dtype=torch.uint8, device="cuda")
    outs = [torch.empty((1, 8, 128), dtype=torch.bfloat16, device="cuda") for _ in range(8)]

    def run(outs, pause, stream=None):
        for i, out in enumerate(outs):
            _lib.kvq_append_int4(*kv[i % 2], slots, mu, rk, rv, cache, P, stream=stream)
            pause()
            _lib.kvq_decode_attn_int4(q, cache, P, bt, ctx, rk, rv, SCALE, out, ws, splits, stream=stream)
            pause()

    run(outs[:2], torch.cuda.synchronize)
    own = torch.cuda.Stream()
    run(outs[2:6], lambda: None, own)
    own.synchronize()
    run(outs[6:], lambda: None)
    torch.cuda.synchronize()
    assert not torch.equal(outs[0], outs[1])
    assert all(torch.equal(x, outs[i % 2]) for i, x in enumerate(outs))


def test_repeated_calls_give_the_same_bits():
    for h_q in (32, 64):
        c = _Case(h_q, 8, [1500, 700], seed=4)
        a, wa = c.run(0, 1.0)
        for _ in range(3):
            b, wb = c.run(0, 1.0)
            assert np.array_equal(a, b) and np.array_equal(wa, wb)


def test_one_workspace_serves_calls_of_every_shape():
    """Batches that grow and shrink, with and without weights and a given split, in one workspace: each call's bits are
    those of a call with a workspace of its own."""
    cases = [(_Case(8, 1, [100], seed=6), 3), (_Case(32, 8, [40] * 19, seed=6), 0), (_Case(16, 8, [50] * 30, seed=6), 0),
             (_Case(32, 8, [70] * 9, seed=6), 0), (_Case(8, 1, [900], seed=6), 0), (_Case(64, 8, [33] * 12, seed=6), 0)]
    size = lambda c, s, w: _lib.kvq_int4_workspace_bytes(c.B, c.h_q, c.h_kv, c.P, s, w)  # noqa: E731
    ws = torch.zeros(max(size(c, s, True) for c, s in cases), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        for c, splits in cases:
            for decay in (None, 1.0):
                want, w_want = c.run(splits, decay)
                got, w_got = c.run(splits, decay, ws=ws)
                assert c.status == 0 and np.array_equal(got, want)
                assert decay is None or np.array_equal(w_got, w_want)


def test_prefill_then_decode_through_the_layer():
    spec = inputs.small_spec("int4layer", h_q=16, h_kv=2, batch=2, ctx=321, permute=True)
    layer = Int4Layer(spec, 0)
    layer.prefill()
    k_new, v_new = layer.new_kv()
    layer.append(k_new, v_new, layer.new_slots())
    q, out = layer.queries(), torch.empty((2, 16, 128), dtype=torch.bfloat16, device="cuda")
    ws = layer.workspace()
    layer.decode(q, out, ws, decay=1.0)
    plain, split, split_w = (torch.empty_like(out) for _ in range(3))
    layer.decode(q, plain, ws)
    keep, ws2 = layer.weights.clone(), layer.workspace(2)
    layer.decode(q, split, ws2, 2)
    layer.decode(q, split_w, ws2, 2, decay=1.0)
    layer.weights = keep
    assert torch.equal(split, split_w)  # (the same split: the same sums)
    f = lambda x: x.cpu().double().numpy()  # noqa: E731
    cache = int4.new_cache(layer.num_pages, 2)
    for b in range(2):
        k, v = layer.history_kv(b)
        k, v = torch.cat([k, k_new[b:b + 1]]), torch.cat([v, v_new[b:b + 1]])
        int4.append(cache, f(k), f(v), layer.slots(b, torch.arange(321)).cpu().numpy(), f(layer.mu), f(layer.R_k), f(layer.R_v))
    assert np.array_equal(layer.cache.cpu().numpy(), cache)
    ref = int4.decode(f(q), cache, layer.block_table.cpu().numpy(), [321, 321], f(layer.R_k), f(layer.R_v), layer.scale)
    for b in range(2):
        for j in range(16):
            # 2^-8 for bf16, 2^-10 of terms that are a few times the result
            for o in (out, plain, split):
                assert np.linalg.norm(f(o)[b, j] - ref[b, j]) <= 2.0 ** -7 * np.linalg.norm(ref[b, j])
    # 16 heads of two sequences, each with weights that add up to 1 (two calls of one step: only the first accumulates)
    assert abs(float(layer.weights.double().sum()) - 2 * 16) <= 32 * 2.0 ** -15


def _grown(R, n, g):
    """Inputs along columns of R, from its rows in the order of the first column's magnitudes down: products of one sign
    whose partial sums stay near the bound that the norms give, where a sum that is cut to 24 bits at each step errs most."""
    x = R[:, np.where(np.arange(n) % 2, 0, g.integers(0, 128, n))].T * g.uniform(0.5, 2.0, (n, 1))
    return (x * (1.0 + 0.1 * g.standard_normal(x.shape)))[:, None]


@pytest.mark.parametrize("norm", [1.0, 3.0])
def test_append_of_inputs_along_a_column(norm):
    """A whole prefill's bytes are the oracle's, also where the columns of the matrix have another norm than 1."""
    rng = np.random.default_rng(77)
    R = _rot(rng, 1)[0]
    R = (norm * R[np.argsort(-np.abs(R[:, 0]))]).astype(np.float32)
    n = 4096
    k, v = _bf(_grown(R, n, rng)), _bf(_grown(R, n, rng))
    mu = np.zeros((1, 128), np.float32)
    cache, want = torch.zeros((n // 16, 1, 2560), dtype=torch.uint8, device="cuda"), int4.new_cache(n // 16, 1)
    assert _append(k, v, np.arange(n), mu, R[None], R[None], cache) == 0
    int4.append(want, k.double().numpy(), v.double().numpy(), np.arange(n), mu, R[None], R[None])
    assert np.array_equal(cache.cpu().numpy(), want)
