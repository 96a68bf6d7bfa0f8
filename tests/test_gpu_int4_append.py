"""GPU tests of the INT4 append where the tensor cores' sums lose most: a matrix instruction cuts each of its terms off
at a fixed place below the largest of them, so one dominant product takes the low bits of all the others."""
import numpy as np
import pytest
import torch

from oracle import int4
from test_gpu_int4 import _append, _bf, _rot

pytestmark = pytest.mark.gpu


def _dominated(R, n, g, low):
    """Inputs [n, 1, 128] whose product with column 0 of R has one dominant term, all others with the sign against it and
    just below 2^-low of it (times a power of two's odd neighbour, so that their last bits count)."""
    at = np.argmax(np.abs(R[:, 0]))
    x = -np.sign(R[:, 0]) * 2.0 ** -low / np.maximum(np.abs(R[:, 0]), 1e-3) * abs(R[at, 0])
    x = x[None] * g.uniform(0.5, 1.0, (n, 1)) * (1 + g.integers(0, 2, (n, 128)) / 64)
    x[:, at] = np.sign(R[at, 0]) * g.uniform(1.0, 2.0, n)
    return x[:, None]


@pytest.mark.parametrize("low", [20, 22, 23, 24, 25])
def test_append_of_inputs_with_one_dominant_product(low):
    """A dominant product of one sign, 127 of the other just below its last bits: every group's parameters and codes are
    the oracle's, whichever kernel writes them."""
    rng = np.random.default_rng(low)
    R = _rot(rng, 1)
    n = 8192
    k, v = _bf(_dominated(R[0], n, rng, low)), _bf(_dominated(R[0], n, rng, low))
    mu = np.zeros((1, 128), np.float32)
    cache, want = torch.zeros((n // 16, 1, 2560), dtype=torch.uint8, device="cuda"), int4.new_cache(n // 16, 1)
    assert _append(k, v, np.arange(n), mu, R, R, cache) == 0
    int4.append(want, k.double().numpy(), v.double().numpy(), np.arange(n), mu, R, R)
    got = cache.cpu().numpy()
    assert np.array_equal(got, want), np.count_nonzero((got != want).any(-1))


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("units", [1, 2, 4])
def test_a_min_next_to_a_rounding_boundary_under_a_dominant_product(sign, units):
    """The exact min of every group lies 2^-20 past the middle between two fp16 values, of which 2^-16 to 2^-14 is the sum of
    63 products, each just below `units` steps of where a sum with a term of 8 is cut off (2^-25 of it, 2^-22)."""
    r = np.float32(units * 127 / 128 * 2.0 ** -8)          # times 2^-14: a little below units * 2^-22, a bf16 number
    rest = 63 * float(r) * 2.0 ** -14
    R = np.zeros((1, 128, 128), np.float32)
    for g in range(4):
        edge = 8 + (2 * g + 1 + 16 * units) * 2.0 ** -8     # fp16 numbers lie 2^-7 apart here
        low = np.float32(np.ceil((edge - rest) * 2.0 ** 20) * 2.0 ** -20)   # (an fp32 number: 24 bits)
        assert edge < float(low) + rest <= edge + 2.0 ** -20
        R[0, 0, 32 * g:32 * g + 32] = -sign * np.linspace(-5, 7, 32).astype(np.float32)
        R[0, 0, 32 * g + 3] = -sign * low
        R[0, 1:64, 32 * g + 3] = -sign * r
    n = 512
    scale = 2.0 ** np.arange(-4, 4)[np.arange(n) % 8][:, None]
    x = np.zeros((n, 128))
    x[:, :1], x[:, 1:64] = sign * scale, sign * scale * 2.0 ** -14
    x = _bf((x * np.where(np.arange(n) % 16 < 8, 1, -1)[:, None])[:, None])
    mu = np.zeros((1, 128), np.float32)
    cache, want = torch.zeros((n // 16, 1, 2560), dtype=torch.uint8, device="cuda"), int4.new_cache(n // 16, 1)
    assert _append(x, x, np.arange(n), mu, R, R, cache) == 0
    int4.append(want, x.double().numpy(), x.double().numpy(), np.arange(n), mu, R, R)
    got = cache.cpu().numpy()
    assert np.array_equal(got, want), np.count_nonzero((got != want).any(-1))


@pytest.mark.parametrize("n", [3, 600])
@pytest.mark.parametrize("kind", ["nan", "inf", "huge", "largest", "overflowing sum"])
def test_matrices_with_numbers_that_are_huge_or_not_finite(n, kind):
    """Groups that a matrix entry makes infinite or NaN are NaN in whole, the others are as ever; finite results past fp32
    saturate.  Both kernels write the same bytes."""
    rng = np.random.default_rng(5)
    R = _rot(rng, 1)
    if kind == "nan":
        R[0, 17, 40] = np.nan
    elif kind == "inf":
        R[0, 17, 40] = -np.inf
    elif kind == "huge":
        R[0, :, 40] *= 1e25
    elif kind == "largest":
        R[0, 17, 40] = 3.4e38            # (the nearest bf16 number is infinite)
    else:
        R[0, :, 40] = 3e38 * np.where(np.arange(128) % 2, 1, -1)
    k, v = _bf(rng.standard_normal((n, 1, 128))), _bf(rng.standard_normal((n, 1, 128)) * (1e18 if kind == "huge" else 1.0))
    mu = rng.standard_normal((1, 128)).astype(np.float32)
    pages = (n + 15) // 16
    cache, want = torch.zeros((pages, 1, 2560), dtype=torch.uint8, device="cuda"), int4.new_cache(pages, 1)
    assert _append(k, v, np.arange(n), mu, R, R, cache) == 0
    int4.append(want, k.double().numpy(), v.double().numpy(), np.arange(n), mu, R, R)
    got = cache.cpu().numpy()
    for side in (0, 1):
        a, b = int4.values(got, side).reshape(-1, 128)[:n], int4.values(want, side).reshape(-1, 128)[:n]
        assert np.array_equal(a, b, equal_nan=True)
        assert np.isnan(a[:, 32:64]).all() == (kind in ("nan", "inf")) and np.isfinite(np.delete(a, np.s_[32:64], 1)).all()
    few = torch.zeros_like(cache)
    for i in range(min(n, 40)):
        _append(k[i:i + 1], v[i:i + 1], [i], mu, R, R, few)
    done = min(n, 40) // 16
    assert np.array_equal(few.cpu().numpy()[:done], got[:done])
