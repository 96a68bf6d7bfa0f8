"""The oracle's variance of what fp16 operands do to chunk attention, against the roundings themselves (no GPU)."""
import numpy as np
import pytest

from oracle import int4


@pytest.mark.parametrize("window,sinks,peak", [(0, 0, 2.5), (60, 5, 2.5), (0, 0, 0.5)])
def test_spread_covers_the_roundings_and_not_much_more(window, sinks, peak):
    rng = np.random.default_rng(3)
    n, ctx, scale = 30, 400, 128 ** -0.5
    cache = int4.new_cache(ctx // 16, 1)
    for side in (0, 1):
        for s in range(16):
            int4.write_tokens(cache, side, s, *int4.quantize(rng.standard_normal((ctx // 16, 1, 128))))
    rk, rv = (np.linalg.qr(rng.standard_normal((1, 128, 128)))[0].astype(np.float32) for _ in range(2))
    q = peak * rng.standard_normal((n, 2, 128))
    bt = np.arange(ctx // 16, dtype=np.int32)[None]
    want, var = int4.chunk_spread(q, [0, n], cache, bt, [ctx], rk, rv, scale, window, sinks)
    exact, bound = int4.chunk(q, [0, n], cache, bt, [ctx], rk, rv, scale, window, sinks)
    assert np.array_equal(want, exact)
    half = lambda x: np.asarray(x).astype(np.float16).astype(np.float64)  # noqa: E731
    k, v = (half(int4.values(cache[:, 0], side).reshape(-1, 128)) for side in (0, 1))
    t, p = np.arange(ctx), ctx - n + np.arange(n)[:, None]
    see = (t <= p) & ((window == 0) | (t > p - window) | (t < sinks))
    err2 = np.zeros((n, 2))
    for j in range(2):
        a = np.where(see, half(q[:, j] @ half(rk[0])) @ k.T * scale, -np.inf)
        w = np.exp(a - a.max(1, keepdims=True))
        o = half(half(w) @ v / w.sum(1, keepdims=True)) @ half(rv[0]).T
        err2[:, j] = ((o - want[:, j]) ** 2).sum(-1)
    assert (np.sqrt(err2) <= 6 * np.sqrt(var)).all() and (np.sqrt(err2) <= bound).all()
    assert 0.2 < err2.sum() / var.sum() < 1
