"""GPU parity of chunk attention and of the sliding decode over the INT4 cache against the fp64 oracle.

Tolerance, per row and query head in the 2-norm (the output rotation is orthogonal): bf16 rounds each output value by at
most 2^-8 of it, and oracle.int4.chunk bounds what the fp16 operands do.  The sliding decode's own arithmetic is exact to
more bits, so it is held to the same."""
import numpy as np
import pytest
import torch

from bit_kv_cache_13_gb300 import _lib
from oracle import int4

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


def _dev(x, dtype=None):
    return torch.as_tensor(x, dtype=dtype, device="cuda").contiguous()


def _rot(rng, h):
    return np.stack([np.linalg.qr(rng.standard_normal((128, 128)))[0] for _ in range(h)]).astype(np.float32)


def _cache(rng, pages, h_kv, size=1.0):
    """Tiles of normal keys and values; `size` scales the values' tokens."""
    tiles = int4.new_cache(pages, h_kv)
    for side in (0, 1):
        x = rng.standard_normal((pages, h_kv, 16, 128)) * (0.5 + rng.random((pages, h_kv, 16, 1)))
        if side:
            x = x * size
        for s in range(16):
            int4.write_tokens(tiles, side, s, *int4.quantize(x[:, :, s]))
    return tiles


class Case:
    def __init__(self, seed, new, ctx, h_q, h_kv, window=0, sinks=0, pad=0, extra=1, peak=2.5, size=1.0):
        rng = self.rng = np.random.default_rng(seed)
        self.new, self.ctx, self.window, self.sinks = new, ctx, window, sinks
        B = len(new)
        per = max(1, max(-(-c // 16) for c in ctx)) + extra
        self.bt = rng.permutation(B * per + 3)[: B * per].reshape(B, per).astype(np.int32)
        self.cache = _cache(rng, B * per + 3, h_kv, size)
        for b, c in enumerate(ctx):           # what stands behind a sequence's last token is anything, NaN too
            for i in range(per):
                n = min(16, max(0, c - 16 * i))
                if n < 16:
                    junk = rng.integers(0, 256, (h_kv, 2560)).astype(np.uint8)
                    for side in (0, 1):
                        for s in range(n):
                            for h in range(h_kv):
                                int4.write_tokens(junk[h], side, s, *int4.read_token(self.cache[self.bt[b, i], h], side, s))
                    self.cache[self.bt[b, i]] = junk
        self.start = np.cumsum([0] + new).astype(np.int32)
        n = int(self.start[-1]) + pad
        self.q = torch.as_tensor(peak * rng.standard_normal((n, h_q, 128)), dtype=torch.float32).bfloat16()
        self.rk, self.rv = _rot(rng, h_kv), _rot(rng, h_kv)
        self.h_q, self.h_kv = h_q, h_kv

    def expect(self):
        return int4.chunk(self.q.double().numpy(), self.start, self.cache, self.bt, self.ctx, self.rk, self.rv, SCALE,
                          self.window, self.sinks)

    def workspace(self):
        return torch.zeros(_lib.kvq_chunk_workspace_bytes(self.q.shape[0], len(self.new), self.h_q, self.h_kv),
                           dtype=torch.uint8, device="cuda")

    def device(self):
        return (_dev(self.q), _dev(self.start), _dev(self.cache), self.cache.shape[0], _dev(self.bt),
                _dev(np.asarray(self.ctx, np.int32)), _dev(self.rk), _dev(self.rv), SCALE)

    def run(self, ws=None, status=0):
        args = self.device()
        out = torch.full(self.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        ws = self.workspace() if ws is None else ws
        _lib.kvq_chunk_attn_int4(*args, out, ws, window=self.window, sinks=self.sinks)
        torch.cuda.synchronize()
        assert _lib.load().kvq_workspace_status(ws.data_ptr(), None) == status
        return out.cpu()

    def check(self, got, rows=None):
        want, bound = self.expect()
        n = int(self.start[-1])
        assert torch.equal(got[n:], torch.full_like(got[n:], 7.0))      # rows behind the last sequence
        got, want, bound = got.double().numpy()[:n], want[:n], bound[:n]
        tol = bound + 2.0 ** -8 * np.linalg.norm(want, axis=-1)
        err = np.linalg.norm(got - want, axis=-1)
        if rows is not None:
            err, tol = err[rows], tol[rows]
        assert (err <= tol).all(), (np.argwhere(~(err <= tol))[:8].tolist(), float(np.nanmax(err / np.maximum(tol, 1e-30))))


CASES = [
    # new, ctx, h_q, h_kv, window, sinks
    ([1], [1], 1, 1, 0, 0),
    ([2], [2], 4, 1, 0, 0),
    ([1], [257], 4, 1, 0, 0),
    ([17], [311], 4, 1, 0, 0),
    ([16], [16], 8, 2, 0, 0),
    ([129], [129], 3, 3, 0, 0),
    ([130], [700], 6, 2, 0, 0),
    ([300], [300], 8, 1, 0, 0),
    ([65], [1500], 8, 2, 0, 0),
    ([5, 5, 5], [100, 1000, 517], 8, 2, 0, 0),
    ([0, 3, 1, 0, 40, 1], [0, 3, 77, 50, 41, 1], 7, 1, 0, 0),
    ([20], [300], 12, 1, 0, 0),                      # a group above eight
    ([33], [90], 64, 1, 0, 0),
    ([4, 2], [3, 0], 4, 2, 0, 0),                    # rows before the first token see nothing
    ([70], [400], 4, 1, 1, 0),                       # only itself
    ([70], [400], 4, 1, 5, 0),
    ([70], [400], 4, 1, 64, 4),
    ([70], [400], 4, 2, 33, 20),
    ([260], [1111], 4, 1, 200, 17),
    ([300], [1000], 2, 2, 128, 128),
    ([40], [300], 4, 1, 100, 5000),                  # more sinks than tokens
    ([40], [300], 4, 1, 5000, 4),                    # a window longer than the context
    ([1, 1, 1], [700, 16, 33], 8, 1, 48, 4),
    ([150, 1, 9], [150, 900, 400], 16, 2, 96, 3),
]


@pytest.mark.parametrize("new,ctx,h_q,h_kv,window,sinks", CASES)
def test_chunk(new, ctx, h_q, h_kv, window, sinks):
    c = Case(7 * sum(new) + h_q + sum(ctx), new, ctx, h_q, h_kv, window, sinks, pad=len(new) % 3)
    c.check(c.run())


def test_long_chunks_and_many_units():
    for new, ctx, h_q, h_kv, window in (([700], [2500], 8, 2, 0), ([512, 3, 256], [513, 4001, 256], 4, 1, 0), ([600], [3000], 4, 1, 777)):
        c = Case(sum(ctx), new, ctx, h_q, h_kv, window, 4)
        c.check(c.run())


def test_output_in_the_queries_place_and_the_same_bits_again():
    c = Case(5, [200, 7], [900, 350], 8, 2)
    args, ws = c.device(), c.workspace()
    first = torch.empty_like(args[0])
    _lib.kvq_chunk_attn_int4(*args, first, ws)
    again = torch.empty_like(first)
    _lib.kvq_chunk_attn_int4(*args, again, ws)
    _lib.kvq_chunk_attn_int4(*args, args[0], ws)
    torch.cuda.synchronize()
    assert torch.equal(first, again) and torch.equal(first, args[0])
    c.check(first.cpu())


def test_bad_pages_are_dropped_and_reported():
    c = Case(6, [40, 3], [400, 100], 4, 2)
    c.bt[0, 3], c.bt[0, 9], c.bt[1, 0] = -1, c.cache.shape[0], 2 ** 31 - 1
    c.check(c.run(status=-5))
    c.bt[0, 3] = c.bt[0, 9] = c.bt[1, 0] = 0
    ws = c.workspace()
    c.check(c.run(ws))
    # a bad entry that no row sees is not read
    c = Case(7, [4], [400], 4, 1, window=32, sinks=16)
    c.bt[0, 5], c.bt[0, -1] = -7, -7
    c.check(c.run())


def test_bad_row_starts_are_reported():
    c = Case(8, [10, 5, 8], [100, 60, 80], 4, 1)
    want, bound = c.expect()
    c.start = np.array([0, 10, 8, 18], np.int32)     # the second one descends
    got = c.run(status=-1)
    one = Case(8, [10, 5, 8], [100, 60, 80], 4, 1)
    one.check(got, rows=slice(0, 8))
    c.start = np.array([0, 10, 15, 24], np.int32)    # past the rows
    got = c.run(status=-1)
    one.check(torch.cat([got[:15], torch.zeros_like(got[15:])]), rows=slice(0, 15))
    assert torch.equal(got[15:], torch.full_like(got[15:], 7.0))


@pytest.mark.parametrize("new,ctx,h_q,h_kv", [([5], [2000], 8, 2), ([1], [3000], 4, 1), ([64], [1000], 4, 2), ([70, 1], [1300, 900], 8, 2)])
def test_small_calls_in_few_and_many_shares(new, ctx, h_q, h_kv):
    """A unit's tiles over several CTAs, whose sums are merged, from one tile up to dozens a share."""
    c = Case(30 + sum(new), new, ctx, h_q, h_kv)
    c.check(c.run())


def test_row_starts_up_and_down_of_a_wide_batch():
    """Every other sequence claims all the rows: far more blocks than the workspace has places for, none written behind it."""
    rows, B = 3000, 40001
    c = Case(20, [rows], [rows], 1, 1, extra=0)
    start = torch.zeros(B + 1, dtype=torch.int32)
    start[1::2] = rows
    q, _, cache, pages, bt, _, rk, rv, scale = c.device()
    n = _lib.kvq_chunk_workspace_bytes(rows, B, 1, 1)
    ws = torch.zeros(n + 4096, dtype=torch.uint8, device="cuda")
    ws[n:] = 99
    out = torch.empty_like(q)
    ctx = torch.zeros(B, dtype=torch.int32)
    _lib.kvq_chunk_attn_int4(q, start.cuda(), cache, pages, bt.expand(B, -1).contiguous(), ctx.cuda(), rk, rv, scale, out, ws[:n])
    torch.cuda.synchronize()
    assert _lib.load().kvq_workspace_status(ws.data_ptr(), None) == -1
    assert (ws[n:] == 99).all()
    assert not out.any()                            # no context: every row of the sequences that count sees nothing
    ctx[0] = rows
    _lib.kvq_chunk_attn_int4(q, torch.full((B + 1,), rows, dtype=torch.int32).index_fill_(0, torch.tensor([0]), 0).cuda(), cache, pages,
                             bt.expand(B, -1).contiguous(), ctx.cuda(), rk, rv, scale, out, ws[:n])
    c.check(out.cpu())
    assert (ws[n:] == 99).all()


def test_windows_of_the_largest_sizes():
    for window, sinks in ((2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (100, 2 ** 31 - 1), (16 * 20 - 1, 1), (16 * 20, 1)):
        c = Case(25, [30, 2], [300, 1], 4, 1, window=window, sinks=sinks)
        c.check(c.run())


def test_pages_past_four_gigabytes():
    c = Case(26, [20, 3], [200, 90], 32, 8, window=64, sinks=20)
    q, start, cache, _, bt, ctx, rk, rv, scale = c.device()
    first = 2 ** 32 // (8 * 2560) + 5
    far = torch.empty((first + cache.shape[0], 8, 2560), dtype=torch.uint8, device="cuda")
    far[first:] = cache
    bt = bt + first
    out, ws = torch.full_like(q, 7.0), c.workspace()
    _lib.kvq_chunk_attn_int4(q, start, far, far.shape[0], bt, ctx, rk, rv, scale, out, ws, window=64, sinks=20)
    c.check(out.cpu())
    # the sequences' last tokens alone, by the sliding decode
    last = (start[1:] - 1).long()
    one = torch.empty_like(q[last])
    ws = torch.zeros(_lib.kvq_int4_workspace_bytes(2, 32, 8, bt.shape[1]), dtype=torch.uint8, device="cuda")
    _lib.kvq_decode_attn_int4_sliding(q[last], far, far.shape[0], bt, ctx, rk, rv, scale, 64, 20, one, ws)
    out[last] = one
    c.check(out.cpu())


def test_nan_in_tokens_that_some_rows_see():
    """A cached group of NaN makes the rows that see it NaN, and no other."""
    for side in (0, 1):
        c = Case(9 + side, [150], [400], 4, 1)
        t = 300                                           # position of row 50
        c.check(c.run())
        tile = c.cache[c.bt[0, t // 16], 0]
        codes, sc, mn = int4.read_token(tile, side, t % 16)
        clean = tile.copy()
        int4.write_tokens(tile, side, t % 16, codes, np.full(4, np.nan, np.float16), np.full(4, np.nan, np.float16))
        got = c.run()
        assert torch.isnan(got[50:150]).all() and not torch.isnan(got[:50]).any()
        c.cache[c.bt[0, t // 16], 0] = clean
        c.check(torch.where(torch.isnan(got), c.run(), got))


def test_values_of_any_size():
    """Sinks with small values and far larger weights, values next to the format's ends."""
    for size in (1e-3, 30.0, 3000.0):
        c = Case(21, [100], [700], 4, 1, size=size)
        c.check(c.run())
    c = Case(22, [100], [700], 4, 1, peak=8.0)
    c.check(c.run())


@pytest.mark.parametrize("B,h_q,h_kv,ctx,window,sinks", [
    (1, 4, 1, [1], 1, 0), (1, 8, 1, [257], 16, 0), (1, 4, 1, [3000], 1000, 4), (1, 32, 8, [5000], 333, 70),
    (3, 6, 2, [700, 0, 31], 48, 4), (3, 8, 1, [1000, 17, 300], 5000, 4), (5, 5, 1, [400, 16, 33, 1, 2000], 17, 33),
    (40, 4, 2, None, 100, 5), (40, 16, 2, None, 30, 0), (2, 4, 2, [900, 800], 1, 900), (170, 1, 1, None, 64, 16),
])
@pytest.mark.parametrize("splits", [0, 3])
def test_sliding(B, h_q, h_kv, ctx, window, sinks, splits):
    rng = np.random.default_rng(B + h_q)
    ctx = [int(x) for x in rng.integers(0, 900, B)] if ctx is None else ctx
    c = Case(B, [1] * B, ctx, h_q, h_kv, window, sinks)
    q, _, *args = c.device()
    ws = torch.zeros(_lib.kvq_int4_workspace_bytes(B, h_q, h_kv, c.bt.shape[1], splits), dtype=torch.uint8, device="cuda")
    out = torch.full(c.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    for _ in range(2):
        _lib.kvq_decode_attn_int4_sliding(q, *args, window, sinks, out, ws, splits)
        torch.cuda.synchronize()
        c.check(out.cpu())
    if window >= max(ctx):   # all tokens: the plain decode's bits, where both take the same split
        plain = torch.empty_like(out)
        _lib.kvq_decode_attn_int4(q, *args, plain, ws, 3)
        _lib.kvq_decode_attn_int4_sliding(q, *args, window, sinks, out, ws, 3)
        assert torch.equal(plain, out)


def test_sliding_skips_bad_pages_and_masks_nan():
    c = Case(31, [1], [900], 4, 1, window=100, sinks=20)
    c.bt[0, 10], c.bt[0, 53] = -4, 10 ** 6               # out of sight; in the window
    for t in (20, 799):                                   # tokens next to the sinks and the window: NaN, not seen
        tile = c.cache[c.bt[0, t // 16], 0]
        for side in (0, 1):
            codes, _, _ = int4.read_token(tile, side, t % 16)
            int4.write_tokens(tile, side, t % 16, codes, np.full(4, np.nan, np.float16), np.full(4, np.nan, np.float16))
    q, _, *args = c.device()
    ws = torch.zeros(_lib.kvq_int4_workspace_bytes(1, 4, 1, c.bt.shape[1]), dtype=torch.uint8, device="cuda")
    out = torch.full(c.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    _lib.kvq_decode_attn_int4_sliding(q, *args, 100, 20, out, ws)
    assert _lib.load().kvq_workspace_status(ws.data_ptr(), None) == -5
    c.check(out.cpu())


@pytest.mark.parametrize("new,ctx", [
    ([100, 0, 0, 1], [333, 0, 7, 50]),              # few rows on the average, four blocks of them in one sequence
    ([65, 1, 1], [65, 300, 129]),                   # the last block of a sequence one row past a tile
    ([32, 32], [200, 32]), ([33, 32], [200, 32]),   # 128 rows on the average, and a token more
    ([1] * 300, [int(x) for x in np.random.default_rng(0).integers(0, 200, 300)]),
    ([3] * 90, [int(x) for x in np.random.default_rng(1).integers(3, 500, 90)]),
])
def test_block_sizes_and_wide_batches(new, ctx):
    c = Case(3 + len(new), new, ctx, 4, 1)
    c.check(c.run())
    if len(new) < 10:
        c = Case(4 + len(new), new, ctx, 8, 2, window=40, sinks=5)
        c.check(c.run())


def test_scales_zero_and_negative_and_queries_of_any_size():
    for scale, peak in ((0.0, 2.5), (-SCALE, 2.5), (SCALE * 1e-6, 2.5e6), (SCALE * 1e30, 2.5e-30)):
        c = Case(41, [70], [300], 4, 1, peak=peak)
        args = list(c.device())
        args[-1] = scale
        out, ws = torch.empty_like(args[0]), c.workspace()
        _lib.kvq_chunk_attn_int4(*args, out, ws)
        want, bound = int4.chunk(c.q.double().numpy(), c.start, c.cache, c.bt, c.ctx, c.rk, c.rv, scale)
        err = np.linalg.norm(out.double().cpu().numpy() - want, axis=-1)
        assert (err <= bound + 2.0 ** -8 * np.linalg.norm(want, axis=-1)).all(), scale


def test_a_late_largest_logit_raises_the_reference():
    """Logits that grow along the context by far more than fp16 holds, slowly and at once, also within a tile."""
    for at in (0, 70, 150, 299):
        c = Case(50 + at, [40], [300], 4, 1, peak=1.0)
        q = c.q.float().numpy()
        for h in range(4):    # a key along the mean query at one token: its logit about 40 above the others
            q[:, h] = q[:, 0]
        q[:] = q[:1]
        c.q = torch.as_tensor(q).bfloat16()
        k = (c.q[0, 0].double().numpy() @ c.rk[0].astype(np.float64))
        tile = c.cache[c.bt[0, at // 16], 0]
        int4.write_tokens(tile, 0, at % 16, *int4.quantize(k * (40 / SCALE / (k @ k))))
        c.check(c.run())
    c = Case(60, [30], [1500], 4, 1, peak=1.0)
    q = c.q.float().numpy()
    q[:] = q[:1, :1]
    c.q = torch.as_tensor(q).bfloat16()
    k = c.q[0, 0].double().numpy() @ c.rk[0].astype(np.float64)
    for t in range(0, 1500, 7):
        int4.write_tokens(c.cache[c.bt[0, t // 16], 0], 0, t % 16, *int4.quantize(k * (0.1 * t / SCALE / (k @ k))))
    c.check(c.run())


def test_a_workspace_serves_calls_of_other_shapes():
    big = Case(71, [200, 60], [700, 300], 8, 2)
    ws = big.workspace()
    for c in (big, Case(72, [3], [40], 4, 1), Case(73, [1] * 20, [100] * 20, 4, 1), big, Case(74, [90], [90], 8, 2)):
        assert _lib.kvq_chunk_workspace_bytes(c.q.shape[0], len(c.new), c.h_q, c.h_kv) <= ws.numel()
        c.check(c.run(ws))
    small = torch.zeros(big.workspace().numel() - 1, dtype=torch.uint8, device="cuda")
    with pytest.raises(_lib.KvqError, match="workspace"):
        big.run(small)


def test_captured_and_replayed_on_another_stream_with_other_inputs():
    c, d = Case(81, [50, 5], [400, 90], 8, 2), Case(82, [50, 5], [400, 90], 8, 2)
    args, ws = list(c.device()), c.workspace()
    out = torch.zeros_like(args[0])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        _lib.kvq_chunk_attn_int4(*args, out, ws)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            _lib.kvq_chunk_attn_int4(*args, out, ws)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    c.check(out.cpu())
    other = d.device()
    for x, y in zip(args, other):
        if torch.is_tensor(x):
            x.copy_(y)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    d.check(out.cpu())
    assert _lib.load().kvq_workspace_status(ws.data_ptr(), None) == 0


def test_two_streams_at_once():
    cases = [Case(91, [120], [900], 8, 2), Case(92, [4, 4, 4], [300, 800, 64], 8, 1)]
    streams = [torch.cuda.Stream() for _ in cases]
    state = [(c.device(), c.workspace(), torch.zeros(c.q.shape, dtype=torch.bfloat16, device="cuda")) for c in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (args, ws, out) in zip(streams, state):
            _lib.kvq_chunk_attn_int4(*args, out, ws, stream=s)
    torch.cuda.synchronize()
    for c, (_, _, out) in zip(cases, state):
        c.check(out.cpu())


def test_an_empty_call_and_refused_tensors():
    c = Case(95, [4], [40], 4, 1)
    q, start, *rest = c.device()
    ws = c.workspace()
    _lib.kvq_chunk_attn_int4(q[:0], start * 0, *rest, q[:0], ws)
    with pytest.raises(ValueError, match="contiguous"):
        _lib.kvq_chunk_attn_int4(q.transpose(0, 1).contiguous().transpose(0, 1), start, *rest, torch.empty_like(q), ws)
    with pytest.raises(ValueError, match="q_start"):
        _lib.kvq_chunk_attn_int4(q, start[:1], *rest, torch.empty_like(q), ws)
    with pytest.raises(ValueError, match="out"):
        _lib.kvq_chunk_attn_int4(q, start, *rest, torch.empty_like(q)[:2], ws)
    with pytest.raises(ValueError, match="bytes"):
        _lib.kvq_chunk_attn_int4(q, start, rest[0], rest[1] + 1, *rest[2:], torch.empty_like(q), ws)


def test_a_copy_that_never_comes_is_reported():
    """The wait for it runs out, the call ends, the status says so, and the next call is right."""
    for new, ctx in (([100], [700]), ([3, 3], [500, 90])):
        c = Case(97 + len(new), new, ctx, 8, 2)
        ws = c.workspace()
        _lib.kvq_debug_drop_next_copy()
        args = c.device()
        _lib.kvq_chunk_attn_int4(*args, torch.empty_like(args[0]), ws)
        torch.cuda.synchronize()
        assert _lib.load().kvq_workspace_status(ws.data_ptr(), None) == -4
        c.check(c.run(ws))
