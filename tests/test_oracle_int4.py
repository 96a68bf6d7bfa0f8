"""Pins of the INT4 oracle: rational arithmetic, closed forms and brute force that do not re-derive its formulas (CPU)."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import attention, int4


def _brute(z, sc, mn):
    """Nearest of the 16 levels by rational distance, the lower of two as near."""
    s, m = Fraction(float(sc)), Fraction(float(mn))
    if s == 0:
        return np.zeros(len(z), int)
    return np.array([min(range(16), key=lambda c: (abs(Fraction(float(x)) - m - c * s), c)) for x in z])


@pytest.mark.parametrize("seed", range(20))
def test_codes_are_the_nearest_level(seed):
    rng = np.random.default_rng(seed)
    z = rng.standard_normal(32) * 10.0 ** rng.uniform(-3, 3) + rng.normal(0, 5)
    sc, mn = int4.quant_params(z)
    assert np.array_equal(int4.quant_codes(z, sc, mn), _brute(z, sc, mn))
    # the levels span the group's range up to the rounding of scale and min (half an fp16 step each)
    top = float(mn) + 15 * float(sc)
    slack = 2.0 ** -11 * (abs(float(mn)) + 15 * float(sc)) + 1e-7
    assert abs(float(mn) - z.min()) <= slack and abs(top - z.max()) <= 2 * slack


def test_midpoints_go_low_and_the_ends_saturate():
    sc, mn = np.float16(0.5), np.float16(1.0)
    z = np.array([-9.0, 1.0, 1.25, np.nextafter(1.25, 2), 1.75, 8.25, np.nextafter(8.25, 9), 8.5, 99.0])
    assert int4.quant_codes(z, sc, mn).tolist() == [0, 0, 0, 1, 1, 14, 15, 15, 15]


def test_constant_group_underflow_overflow_and_not_finite():
    sc, mn = int4.quant_params(np.full(32, 3.140625))
    assert float(sc) == 0 and float(mn) == 3.140625 and int4.quant_codes(np.full(32, 3.140625), sc, mn).max() == 0
    assert float(int4.quant_params(np.r_[np.zeros(31), 1e-9])[0]) == 0
    sc, mn = int4.quant_params(np.r_[-1e6, 1e6 * np.ones(31)])
    assert float(sc) == 65504 and float(mn) == -65504
    for bad in (np.nan, np.inf, -np.inf):
        assert all(np.isnan(x) for x in int4.quant_params(np.r_[np.zeros(31), bad]))


def test_clip_scales_the_range_ends():
    z = np.linspace(-3, 6, 32)
    sc, mn = int4.quant_params(z, 0.5)
    assert float(mn) == -1.5 and abs(float(sc) - 0.3) <= 2.0 ** -11 * 0.3
    assert int4.quant_codes(z, sc, mn)[0] == 0 and int4.quant_codes(z, sc, mn)[-1] == 15


def test_every_code_and_meta_byte_of_the_tile_is_used_once():
    hit = np.zeros((int4.TILE_BYTES, 2), int)
    for side in (0, 1):
        for s in range(16):
            for c in range(128):
                byte, low = int4.code_address(side, s, c)
                hit[byte, low // 4] += 1
            for g in range(4):
                for at in int4.meta_address(side, s, g):
                    hit[at:at + 2] += 1
    assert np.all(hit == 1)
    # the word and half of the documented layout, by hand: channel 32*2 + 8*1 + 5 of key slot 3; 32*1 + 4*6 + 2 of value slot 9
    assert int4.code_address(0, 3, 77) == (64 * 3 + 16 * 1 + 4 * 2 + 2, 4)
    assert int4.code_address(1, 9, 58) == (1280 + 128 * 4 + 16 * 6 + 4 * 1 + 2 + 1, 0)


def test_tokens_round_trip_and_neighbours_stay():
    rng = np.random.default_rng(1)
    tile = rng.integers(0, 256, int4.TILE_BYTES).astype(np.uint8)
    before = {(side, s): int4.read_token(tile, side, s) for side in (0, 1) for s in range(16)}
    codes = rng.integers(0, 16, 128).astype(np.uint8)
    sc, mn = rng.standard_normal((2, 4)).astype(np.float16)
    int4.write_tokens(tile, 1, 5, codes, sc, mn)
    got = int4.read_token(tile, 1, 5)
    assert all(np.array_equal(a, b) for a, b in zip(got, (codes, sc, mn)))
    for key, want in before.items():
        if key != (1, 5):
            got = int4.read_token(tile, *key)
            assert all(np.array_equal(a.view(np.uint8), b.view(np.uint8)) for a, b in zip(got, want))


def _lattice(rng, n, h_kv):
    """Vectors whose groups hold 0 and 15 and integers between: the quantiser is the identity on them."""
    x = rng.integers(0, 16, (n, h_kv, 4, 32)).astype(np.float64)
    x[..., 0], x[..., 1] = 0, 15
    return x.reshape(n, h_kv, 128)


def test_lattice_inputs_give_plain_attention_and_its_weights():
    rng = np.random.default_rng(2)
    B, h_q, h_kv, n = 2, 6, 2, 37
    cache, bt = int4.new_cache(6, h_kv), np.array([[4, 0, 2], [1, 5, 3]])
    perm = np.stack([np.eye(128)[rng.permutation(128)] for _ in range(h_kv)])   # rotations that keep the lattice
    k, v = _lattice(rng, n, h_kv), _lattice(rng, n, h_kv)
    kk = np.stack([k[:, h] @ perm[h].T for h in range(h_kv)], 1)   # k = z R^T: rotated it is the lattice again
    vv = np.stack([v[:, h] @ perm[h].T for h in range(h_kv)], 1)
    q = rng.standard_normal((B, h_q, 128)) * 0.05
    lens = [n, 20]
    for b in range(B):
        int4.append(cache, kk, vv, [bt[b, t // 16] * 16 + t % 16 for t in range(n)], np.zeros((h_kv, 128)), perm, perm)
    w0 = rng.random((B, h_kv, 48))
    out, w = int4.decode(q, cache, bt, lens, perm, perm, 0.3, w0, 0.5)
    for b in range(B):
        want = attention.gqa_decode(q[b], kk[:lens[b]], vv[:lens[b]], float(np.float32(0.3)))
        assert np.max(np.abs(out[b] - want)) <= 1e-12
        # the weights of a step add up to the query heads of each KV head, and nothing moves past the context
        assert np.allclose((w[b, :, :lens[b]] - 0.5 * w0[b, :, :lens[b]]).sum(-1), h_q // h_kv, atol=1e-12)
        assert np.array_equal(w[b, :, lens[b]:], w0[b, :, lens[b]:])


def test_attention_does_not_change_with_the_centre_or_the_rotation():
    rng = np.random.default_rng(3)
    k, v = rng.standard_normal((2, 24, 1, 128)) * 0.1
    R = np.linalg.qr(rng.standard_normal((128, 128)))[0][None].astype(np.float32)
    q = rng.standard_normal((1, 2, 128))
    want = attention.gqa_decode(q[0], k, v, 0.1)
    for mu, rot in ((np.zeros((1, 128)), np.eye(128)[None]), (k.mean(0), R)):
        cache = int4.new_cache(2, 1)
        int4.append(cache, k, v, np.arange(24), mu, rot, rot)
        got = int4.decode(q, cache, [[0, 1]], [24], rot, rot, 0.1)
        # a coded value is off by at most half a step of about range / 15: 0.5 * 6 * 0.1 / 15
        assert np.max(np.abs(got[0] - want)) <= 0.02


def test_empty_and_dropped_pages():
    rng = np.random.default_rng(4)
    cache = int4.new_cache(2, 1)
    eye = np.eye(128)[None]
    int4.append(cache, *rng.standard_normal((2, 32, 1, 128)), np.arange(32), np.zeros((1, 128)), eye, eye)
    q = rng.standard_normal((1, 1, 128))
    assert not int4.decode(q, cache, [[0, 1]], [0], eye, eye, 0.1).any()
    full = int4.decode(q, cache, [[1, 0]], [16], eye, eye, 0.1)
    out, w = int4.decode(q, cache, [[1, 7]], [30], eye, eye, 0.1, np.zeros((1, 1, 32)))
    assert np.allclose(out, full, atol=1e-13) and not w[0, 0, 16:].any()


def test_select_by_hand():
    w = np.array([[[9, 0.5, np.nan, 3, 3, -0.0, 0.0, 3, -np.inf, np.inf, 1, 2]]], np.float32)
    # sinks {0}, recent {11}; of the rest the largest five: inf (9), then the 3s (3, 4, 7), then 1 (10)
    keep, new = int4.select(w, [12], 7, 1, 1)
    assert keep[0, 0].tolist() == [0, 3, 4, 7, 9, 10, 11] and new.tolist() == [7]
    # zeros of either sign tie (lower index first); NaN and -inf are last and tie
    keep, _ = int4.select(w, [12], 11, 0, 0)
    assert keep[0, 0].tolist() == [0, 1, 2, 3, 4, 5, 6, 7, 9, 10, 11]
    keep, new = int4.select(w, [3], 7, 1, 1)
    assert keep[0, 0].tolist() == [0, 1, 2, -1, -1, -1, -1] and new.tolist() == [3]


def test_gather_moves_tokens_whole():
    rng = np.random.default_rng(5)
    cache = rng.integers(0, 256, (3, 2, int4.TILE_BYTES)).astype(np.uint8)
    dst = np.zeros((2, 2, int4.TILE_BYTES), np.uint8)
    keep = np.array([[[0, 17, 18, 40], [5, 6, 7, 8]]], np.int32)
    w = rng.random((1, 2, 48)).astype(np.float32)
    wo = int4.gather(cache, np.array([[2, 0, 1]]), keep, [4], dst, np.array([[1]]), w)
    assert not dst[0].any()
    for h in range(2):
        for i in range(4):
            s = keep[0, h, i]
            for side in (0, 1):
                a = int4.read_token(dst[1, h], side, i)
                b = int4.read_token(cache[[2, 0, 1][s // 16], h], side, s % 16)
                assert all(np.array_equal(x.view(np.uint8), y.view(np.uint8)) for x, y in zip(a, b))
            assert wo[0, h, i] == w[0, h, s]
    assert not wo[0, :, 4:].any()
