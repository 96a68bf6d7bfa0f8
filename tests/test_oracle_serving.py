"""Pins of the oracle's norms, rotation and chunk attention."""
import numpy as np

from bit_kv_cache_13_gb300 import inputs
from oracle import int4


def test_rotation_is_the_complex_product_and_keeps_norms():
    rng = np.random.default_rng(0)
    x, table = rng.standard_normal((5, 2, 128)), inputs.rope_table(50, 64, 1e4).numpy()
    pos = np.array([0, 3, 49, 50, -1])
    for inter in (False, True):
        y = int4.norm_rope(x, pos, table, interleaved=inter)
        assert np.array_equal(y[0], x[0]) and not y[3:].any()
        assert np.array_equal(y[:3, :, 64:], x[:3, :, 64:])
        assert np.allclose(np.linalg.norm(y[:3], axis=-1), np.linalg.norm(x[:3], axis=-1), rtol=1e-6)
        a, b = (slice(0, 64, 2), slice(1, 64, 2)) if inter else (slice(0, 32), slice(32, 64))
        z = (x[1, :, a] + 1j * x[1, :, b]) * np.exp(1j * 3 * 1e4 ** (-np.arange(32) / 32))
        assert np.allclose(y[1, :, a], z.real, atol=1e-6) and np.allclose(y[1, :, b], z.imag, atol=1e-6)


def test_norm_and_rounding():
    x = np.full((1, 1, 128), 3.0)
    y = int4.norm_rope(x, [0], np.concatenate([np.ones((1, 64)), np.zeros((1, 64))], 1), np.arange(128.0), 7.0)
    assert np.allclose(y[0, 0], np.arange(128.0) * 3 / 4)
    assert int4.to_bf16(1 + 2.0 ** -8) == 1 and int4.to_bf16(1 + 3 * 2.0 ** -8) == 1 + 2.0 ** -6
    assert int4.to_bf16(1 + 2.0 ** -8 + 2.0 ** -40) == 1 + 2.0 ** -7 and int4.to_bf16(0.0) == 0


def test_chunk_is_decode_token_by_token():
    rng = np.random.default_rng(1)
    cache = rng.integers(0, 60, (8, 2, 2560)).astype(np.uint8)   # (halves with a small exponent)
    bt = rng.permutation(8)[None].astype(np.int32)
    rk, rv = (np.stack([np.linalg.qr(rng.standard_normal((128, 128)))[0] for _ in range(2)]) for _ in range(2))
    q = 1e4 * rng.standard_normal((20, 4, 128))
    out, bound = int4.chunk(q, [0, 20], cache, bt, [100], rk, rv, 0.1)
    for i in range(20):
        want = int4.decode(q[i:i + 1], cache, bt, [81 + i], rk, rv, 0.1)
        assert np.allclose(out[i], want[0], rtol=1e-9, atol=1e-12)
    assert (bound > 0).all()
    slid, _ = int4.chunk(q, [0, 20], cache, bt, [100], rk, rv, 0.1, window=100)
    assert np.array_equal(slid, out)
    near, _ = int4.chunk(q, [0, 20], cache, bt, [100], rk, rv, 0.1, window=1)
    v = int4.values(cache[bt[0]], 1).transpose(1, 0, 2, 3).reshape(2, 128, 128)
    assert np.allclose(near[3, 1], rv[0].astype(np.float32) @ v[0, 83], rtol=1e-6, atol=1e-9)
