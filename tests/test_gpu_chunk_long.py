"""Chunk attention over contexts of which one CTA sums more than 64K tokens (a pool of few pages, used again and again)."""
import numpy as np
import pytest
import torch

from bit_kv_cache_13_gb300 import _lib
from oracle import int4
from test_gpu_chunk import SCALE, Case, _cache, _dev, _rot

pytestmark = pytest.mark.gpu
B, H, PAGES = 19, 8, 64      # 152 units: a CTA each, where the sequences are as long as one another


def _call(n, q, cache, bt, ctx, rk, rv):
    args = (_dev(q), _dev(np.arange(0, B * n + 1, n, dtype=np.int32)), _dev(cache), PAGES, _dev(bt), _dev(np.full(B, ctx, np.int32)),
            _dev(rk), _dev(rv), SCALE)
    ws = torch.zeros(_lib.kvq_chunk_workspace_bytes(B * n, B, H, H), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(args[0])
    _lib.kvq_chunk_attn_int4(*args, out, ws)
    torch.cuda.synchronize()
    assert _lib.load().kvq_workspace_status(ws.data_ptr(), None) == 0
    return out.double().cpu().numpy()


@pytest.mark.parametrize("n", [2, 256])          # blocks of one row tile and of two
def test_equal_weights_over_a_million_tokens(n):
    """The output is the values' mean.  What a product cuts off its sum is below one unit of fp32's last place, 2^-23, each
    time: over the 4 * 1024 products of a run at most 2^-11, all to one side.  bf16 rounds 1024 different means to either
    side by at most 2^-8, a third of a percent over the root of them: another 2^-12 is five times that."""
    rng = np.random.default_rng(n)
    ctx = 16384 * 64
    cache = _cache(rng, PAGES, H)
    x = 0.1 * rng.standard_normal((PAGES, H, 16, 128)) + rng.uniform(1.0, 2.0, (H, 1, 128))
    for s in range(16):
        int4.write_tokens(cache, 1, s, *int4.quantize(x[:, :, s]))
    eye = np.broadcast_to(np.eye(128, dtype=np.float32), (H, 128, 128))
    bt = np.broadcast_to(np.arange(ctx // 16, dtype=np.int32) % PAGES, (B, ctx // 16))
    got = _call(n, torch.zeros((B * n, H, 128), dtype=torch.bfloat16), cache, bt, ctx, eye, eye)
    v = int4.values(cache, 1).transpose(1, 0, 2, 3).reshape(H, -1, 128)
    mean = v.mean(1)                              # of a sequence's last token
    ratio = (got.reshape(B, n, H, 128)[:, -1] / mean - 1).mean()
    assert abs(ratio) <= 2.0 ** -11 + 2.0 ** -12, ratio


@pytest.mark.parametrize("n,ctx", [(3, 70000), (256, 66000), (3, 140000), (130, 140001)])
def test_runs_are_joined(n, ctx):
    """Ordinary weights, one largest logit in either run: each unit against the oracle."""
    rng = np.random.default_rng(ctx)
    cache, rk, rv = _cache(rng, PAGES, H), _rot(rng, H), _rot(rng, H)
    P = -(-ctx // 16)
    bt = rng.integers(0, PAGES - 2, (B, P)).astype(np.int32)
    q = torch.as_tensor(2.0 * rng.standard_normal((B * n, H, 128)), dtype=torch.float32).bfloat16()
    for b, at in ((0, 5), (1, P - 9), (2, 4090)):     # a page of its own with a key along a query: in the first run, later, next to the cut
        bt[b, at] = PAGES - 1
    for h in range(H):
        k = q[n - 1, h].double().numpy() @ rk[h].astype(np.float64)
        int4.write_tokens(cache[PAGES - 1, h], 0, 3, *int4.quantize(k * (12 / SCALE / (k @ k))))
    got = _call(n, q, cache, bt, ctx, rk, rv).reshape(B, n, H, 128)
    for b in (0, 1, 2, 18):
        for h in (0, 7):
            rows = slice(b * n, b * n + n)
            want, bound = int4.chunk(q[rows, h:h + 1].double().numpy(), [0, n], cache[:, h:h + 1], bt[b:b + 1], [ctx], rk[h:h + 1], rv[h:h + 1], SCALE)
            err = np.linalg.norm(got[b, :, h] - want[:, 0], axis=-1)
            # (far fewer tokens count than there are: a third of the oracle's bound)
            assert (err <= bound[:, 0] / 3 + 2.0 ** -8 * np.linalg.norm(want[:, 0], axis=-1)).all(), (b, h)


@pytest.mark.parametrize("h_q,h_kv,new,ctx", [(2, 1, [256], [4000]), (4, 1, [5], [9000]), (8, 2, [64, 100], [3000, 5000])])
def test_references_that_rise_in_every_tile(h_q, h_kv, new, ctx):
    """Logits grow by 40 nats a tile for a while, then every third tile: sums are taken down right after the product that
    left them, in either stream and in shares that begin anywhere."""
    c = Case(sum(ctx), new, ctx, h_q, h_kv, peak=1.0)
    q = c.rng.standard_normal(128)
    c.q = torch.as_tensor(np.broadcast_to(q, c.q.shape) * c.rng.uniform(0.7, 1.0, c.q.shape[:2] + (1,)), dtype=torch.float32).bfloat16()
    for h in range(h_kv):
        k = q @ c.rk[h].astype(np.float64)
        for b, n in enumerate(ctx):
            for i, tile in enumerate([*range(1, 30), *range(30, n // 64, 3)]):
                if 64 * tile < n:
                    t = 64 * tile + 17 * i % 64
                    if t < n:
                        int4.write_tokens(c.cache[c.bt[b, t // 16], h], 0, t % 16, *int4.quantize(k * (40 * (i + 1) / SCALE / (k @ k))))
    for _ in range(3):
        c.check(c.run())
