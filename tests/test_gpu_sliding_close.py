"""The sliding decode held to its own arithmetic, not to chunk attention's wider one.

Tolerance, per query head in the 2-norm (as for the decode without a window): the bf16 rounding is at most 2^-8 of each
value; p and p * scale are rounded to fp16 at most once each, so 2^-10 of sum_s p_s (15 scale_s + |min_s|) per channel, and
fp32 sums and logits add at most 2^-12 of the same.  Over a call, the mean square error stays within 1.1 times what bf16's
rounding of the exact output alone makes of it, plus 2 (2^-11)^2 / 3 sum_s p_s^2 (15 scale_s + |min_s|)^2: roundings are
independent of each other, and 2^-11 / sqrt(3) is the most that one leaves in standard deviation."""
import numpy as np
import pytest
import torch

from bit_kv_cache_13_gb300 import _lib
from oracle import int4
from test_gpu_chunk import SCALE, Case

pytestmark = pytest.mark.gpu


def _expect(c):
    """Exact outputs, and per channel the sums of p (15 scale + |min|) and of its square."""
    q = c.q.double().numpy()
    out, first, second = (np.zeros(q.shape) for _ in range(3))
    g = c.h_q // c.h_kv
    for b, n in enumerate(c.ctx):
        if n <= 0:
            continue
        t = np.arange(n)
        t = t[(t >= n - c.window) | (t < c.sinks)]
        pages = c.bt[b][t // 16]
        for h in range(c.h_kv):
            tiles = c.cache[pages, h]
            k, v = (int4.values(tiles, side)[np.arange(len(t)), t % 16] for side in (0, 1))
            sc, mn = (np.repeat(x[np.arange(len(t)), t % 16].astype(np.float64), 32, -1) for x in int4.meta(tiles, 1))
            size = 15 * np.abs(sc) + np.abs(mn)
            rk, rv = c.rk[h].astype(np.float64), c.rv[h].astype(np.float64)
            for j in range(h * g, h * g + g):
                a = k @ (q[b, j] @ rk) * float(np.float32(SCALE))
                p = np.exp(a - a.max())
                p /= p.sum()
                out[b, j], first[b, j], second[b, j] = rv @ (p @ v), p @ size, (p * p) @ (size * size)
    return out, first, second


@pytest.mark.parametrize("h_q,h_kv,ctx,window,sinks", [
    (32, 8, [5000], 1000, 4), (32, 8, [131], 100, 4), (8, 1, [900] * 8, 70, 20), (16, 4, [700, 31, 0, 1], 48, 5),
    (8, 2, [int(x) for x in np.random.default_rng(5).integers(1, 1500, 40)], 333, 0), (5, 1, [600] * 9, 10 ** 9, 0)])
@pytest.mark.parametrize("splits", [0, 3])
def test_sliding_by_its_own_arithmetic(h_q, h_kv, ctx, window, sinks, splits):
    c = Case(len(ctx) + h_q, [1] * len(ctx), ctx, h_q, h_kv, window, sinks)
    q, _, *args = c.device()
    ws = torch.zeros(_lib.kvq_int4_workspace_bytes(len(ctx), h_q, h_kv, c.bt.shape[1], splits), dtype=torch.uint8, device="cuda")
    out = torch.full(c.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    _lib.kvq_decode_attn_int4_sliding(q, *args, min(window, 2 ** 31 - 1), sinks, out, ws, splits)
    got = out.double().cpu().numpy()
    want, first, second = _expect(c)
    norm = lambda x: np.linalg.norm(x, axis=-1)  # noqa: E731
    err = norm(got - want)
    assert (err <= 2.0 ** -8 * norm(want) + (2.0 ** -10 + 2.0 ** -12) * norm(first)).all()
    on = norm(want) > 0
    assert got[on].size >= 2048 and not got[~on].any()
    scale = norm(want)[on] ** 2
    near2 = ((int4.to_bf16(want) - want) ** 2).sum(-1)[on]
    spread2 = 2 * 2.0 ** -22 / 3 * second.sum(-1)[on]
    assert (err[on] ** 2 / scale).sum() <= 1.1 * ((near2 + spread2) / scale).sum()
