"""GPU parity of the INT4 decode where the values' sizes and the softmax weights leave the ordinary range: sinks whose own
values are small or zero, values from the smallest normal fp16 scale up to the largest, and both in one context.

Tolerances are those of test_gpu_int4.py (`_Case.check`): relative to sum_s p_s (15 scale_s + |min_s|), whatever the size
of a token's weight or values.
"""
import numpy as np
import pytest
import torch

from oracle import int4
from test_gpu_int4 import SCALE, _Case, _bf, _rot

pytestmark = pytest.mark.gpu


class _Range(_Case):
    """Values of token s scaled by v_size[s] (a number: of all); the first token drew `sink` nats more than the others
    draw on average, and its values are sink_size.  Channels have means of twice their spread, so that what is lost of
    many tokens adds up."""

    def __init__(self, h_q, h_kv, ctxs, v_size=1.0, sink=None, sink_size=0.0, seed=0, q_scale=1.0):
        rng = np.random.default_rng([seed, h_q, h_kv, len(ctxs), max(ctxs)])
        self.B, self.h_q, self.h_kv = len(ctxs), h_q, h_kv
        self.P = (max(ctxs) + 15) // 16
        self.num_pages = self.B * self.P
        self.bt = rng.permutation(self.num_pages).reshape(self.B, self.P).astype(np.int32)
        self.ctx = np.array(ctxs, np.int32)
        self.rk, self.rv = _rot(rng, h_kv), _rot(rng, h_kv)
        g, T = h_q // h_kv, self.P * 16
        # the heads of a group point much the same way, so that one key is a sink of all of them
        q = np.repeat(rng.standard_normal((self.B, h_kv, 128)), g, 1) + 0.1 * rng.standard_normal((self.B, h_q, 128))
        self.q = _bf(q * q_scale)
        self.cache = int4.new_cache(self.num_pages, h_kv)
        mean = 2 * rng.standard_normal((h_kv, 128))
        size = np.broadcast_to(np.asarray(v_size(rng, T) if callable(v_size) else v_size, np.float64), (T,))
        for b in range(self.B):
            k, v = rng.standard_normal((2, T, h_kv, 128))
            v = (v + mean) * size[:, None, None]
            if sink is not None:
                for h in range(h_kv):
                    m = self.q[b, h * g:(h + 1) * g].double().numpy().mean(0) @ self.rk[h].astype(np.float64)
                    k[0, h] = m * sink / SCALE / (m @ m)
                v[0] *= sink_size / size[0]
            tiles = np.zeros((self.P, h_kv, 2560), np.uint8)
            for side, x in ((0, k), (1, v)):
                quant = int4.quantize(x)
                for s in range(16):
                    int4.write_tokens(tiles, side, s, *(y[s::16] for y in quant))
            self.cache[self.bt[b]] = tiles
        self.gpu = self.cache
        self.w0 = rng.random((self.B, h_kv, T + 5)).astype(np.float32)


# (splits 1: a unit's pages all in one CTA of the streaming kernel; 0 for one sequence: the one-kernel form)
@pytest.mark.parametrize("g", [3, 4, 8])
@pytest.mark.parametrize("T,sink,size,sink_size,splits", [
    (4096, 11.0, 0.002, 1e-4, 1), (16384, 12.0, 0.005, 2.5e-4, 1), (32768, 13.0, 0.02, 1e-3, 1), (4096, 11.0, 0.002, 1e-4, 0),
    (5000, 20.0, 1.0, 0.0, 1), (5000, 40.0, 1.0, 0.0, 1), (5000, 40.0, 1.0, 0.0, 0), (3000, 14.0, 300.0, 0.0, 2),
])
def test_sinks_with_small_values(g, T, sink, size, sink_size, splits):
    c = _Range(2 * g if T < 10000 else g, 2 if T < 10000 else 1, [T], size, sink, sink_size)
    got, w = c.run(splits, 1.0)
    plain, _ = c.run(splits)
    assert c.status == 0
    c.check(got, w)
    c.check(plain)


@pytest.mark.parametrize("g", [1, 4, 8])
@pytest.mark.parametrize("size", [3e-4, 1e-3, 1e-2, 1e3, 3e4, 1e6])   # (scales past 65504 saturate when they are stored)
@pytest.mark.parametrize("splits", [0, 1])
def test_values_of_every_size(g, size, splits):
    c = _Range(2 * g, 2, [2500, 40], size, q_scale=3.0, seed=1)
    got, _ = c.run(splits)
    assert c.status == 0
    c.check(got)


@pytest.mark.parametrize("g", [4, 8])
@pytest.mark.parametrize("splits", [0, 1])
def test_sizes_that_differ_from_token_to_token(g, splits):
    """Sizes over nine decades in one context, in any order; and one token of huge values that hardly draws weight."""
    for seed, sizes in enumerate([lambda rng, T: 10.0 ** rng.uniform(-4, 5, T),
                                  lambda rng, T: np.sort(10.0 ** rng.uniform(-4, 5, T)),
                                  lambda rng, T: np.sort(10.0 ** rng.uniform(-4, 5, T))[::-1],
                                  lambda rng, T: np.where(np.arange(T) == 0, 3e4, 2e-3)]):
        sink = dict(sink=-30.0, sink_size=3e4) if seed == 3 else {}
        c = _Range(2 * g, 2, [1800, 333], sizes, q_scale=1.5, seed=seed, **sink)
        got, w = c.run(splits, 1.0)
        assert c.status == 0
        c.check(got, w)


@pytest.mark.parametrize("g", [4, 8])
@pytest.mark.parametrize("splits", [0, 1])
def test_values_times_a_power_of_two(g, splits):
    """Value scales and mins times 2^-6 and 2^8 (all of them normal fp16 numbers): products and sums of the values scale
    exactly, so the output does, to the bit."""
    c = _Range(2 * g, 2, [1500, 90], 1.0, q_scale=2.0, seed=2)
    want, _ = c.run(splits)
    for power in (-6, 8):
        d = _Range(2 * g, 2, [1500, 90], 1.0, q_scale=2.0, seed=2)
        meta = d.gpu[..., 2304:].copy().view(np.float16)
        assert np.abs(meta).min() > 2.0 ** -14 * 2.0 ** max(0, -power) and np.abs(meta).max() < 65504 / 2.0 ** max(0, power)
        d.gpu[..., 2304:] = (meta * np.float16(2.0 ** power)).view(np.uint8)
        got, _ = d.run(splits)
        assert np.array_equal(got, want * 2.0 ** power)


@pytest.mark.parametrize("g", [4, 8])
@pytest.mark.parametrize("splits", [0, 1])
@pytest.mark.parametrize("size", [2e4, 1e5, 3e5])   # of the keys: logits of a million and more
def test_logits_of_millions(g, splits, size):
    """Far apart logits: one token has all the weight, and the output is its values, of whatever size."""
    for v_size in (1e-3, 2e-3, 1.0, 2.0, 1e3, 2e3):
        c = _Range(2 * g, 2, [900, 100], v_size, q_scale=200.0, seed=6)
        meta = c.gpu[..., 1024:1280].copy().view(np.float16)
        c.gpu[..., 1024:1280] = np.clip(meta.astype(np.float64) * size / 10, -65504, 65504).astype(np.float16).view(np.uint8)
        tiles = c.cache[c.bt[0, :56], 0]
        a = int4.values(tiles, 0).reshape(-1, 128) @ (c.q[0, 0].double().numpy() @ c.rk[0].astype(np.float64)) * SCALE
        assert abs(a).max() > 25 * size
        got, _ = c.run(splits)
        assert c.status == 0 and np.isfinite(got).all()
        for b in range(2):
            for h in range(2):
                n = int(c.ctx[b])
                tiles = c.cache[c.bt[b, : (n + 15) // 16], h]
                k, v = (int4.values(tiles, side).reshape(-1, 128)[:n] for side in (0, 1))
                for j in range(h * g, (h + 1) * g):
                    a = k @ (c.q[b, j].double().numpy() @ c.rk[h].astype(np.float64)) * SCALE
                    order = np.argsort(a)
                    if a[order[-1]] - a[order[-2]] < 2.0 ** -15 * abs(a).max() + 20:   # (logits are fp32 numbers)
                        continue
                    want = v[order[-1]] @ c.rv[h].astype(np.float64).T
                    # bf16 2^-8, the two fp16 roundings of the one weight and its products, fp32 sums
                    spread = np.abs(v[order[-1]]).max() * 128 ** 0.5 * 2
                    assert np.linalg.norm(got[b, j] - want) <= 2.0 ** -8 * np.linalg.norm(want) + (2.0 ** -10 + 2.0 ** -16) * spread
