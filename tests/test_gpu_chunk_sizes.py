"""GPU accuracy of chunk attention over the INT4 cache where its operands are small, large or of very different sizes.

Tolerance.  oracle.int4.chunk_spread derives the variance of what fp16 operands leave of each output row; the rounding to
bf16 adds the distance of the exact row from the nearest bf16 one, which is known.  Over a call, the squared errors
relative to their rows' squared norms may sum to 1.1 times the sum of both: the variance is an upper bound (every rounding
as at the lower end of its power of two, where it is largest), and the two parts' product, which has no mean, is below
3 % of it at 4096 outputs or more.  Of a single row the bf16 rounding is at most 2^-8 of each value, and the rest is taken at
six standard deviations.

Where all rows' queries lie along one direction and one token's key takes most of their weight, the roundings of both are
the same for all rows, so that the variances do not average out over a call: the sum of that part is a single draw, and may
be 25 times its variance (five standard deviations; the same roundings made in numpy give sums of up to 1.4 times).  The
rounding to bf16 still averages."""
import numpy as np
import pytest
import torch

from bit_kv_cache_13_gb300 import _lib
from oracle import int4
from test_gpu_chunk import SCALE, Case

pytestmark = pytest.mark.gpu


def run(c, scale):
    args = list(c.device())
    args[-1] = scale
    out, ws = torch.full_like(args[0], 7.0), c.workspace()
    _lib.kvq_chunk_attn_int4(*args, out, ws, window=c.window, sinks=c.sinks)
    return out.cpu()


def close(c, got, scale=SCALE, one_draw=False):
    n = int(c.start[-1])
    want, var = int4.chunk_spread(c.q.double().numpy(), c.start, c.cache, c.bt, c.ctx, c.rk, c.rv, scale, c.window, c.sinks)
    want, var, got = want[:n], var[:n], got.double().numpy()[:n]
    size2 = (want * want).sum(-1)
    err2 = ((got - want) ** 2).sum(-1)
    assert (err2[size2 == 0] == 0).all()
    assert (np.sqrt(err2) <= 2.0 ** -8 * np.sqrt(size2) + 6 * np.sqrt(var)).all(), np.nanmax(np.sqrt(err2 / np.maximum(size2, 1e-300)))
    near2 = ((int4.to_bf16(want) - want) ** 2).sum(-1)
    on = size2 > 0
    assert got[on].size >= 4096
    ratio = (err2[on] / size2[on]).sum() / ((near2[on] * 1.1 + var[on] * (25 if one_draw else 1.1)) / size2[on]).sum()
    assert ratio <= 1, ratio


def set_keys(c, size, spread=0.5):
    """Normal keys of that size (0.5 to 1.5 times it, token by token) in every tile."""
    shape = c.cache.shape[:2] + (16,)
    x = size * c.rng.standard_normal(shape + (128,)) * (0.5 + c.rng.random(shape + (1,)))
    for s in range(16):
        int4.write_tokens(c.cache, 0, s, *int4.quantize(x[:, :, s]))


def test_ordinary_inputs():
    for new, ctx, h_q, h_kv, window in (([40], [700], 4, 2, 0), ([130, 5], [500, 90], 4, 1, 0), ([64], [900], 2, 1, 100),
                                        ([6] * 4, [300, 90, 6, 700], 8, 2, 0)):
        c = Case(100 + sum(ctx), new, ctx, h_q, h_kv, window, 4)
        close(c, c.run())


@pytest.mark.parametrize("size", [1e-6, 1e-5, 1e-4, 1e-3, 1e-2, 30.0, 3000.0, 3e4])
def test_keys_of_any_size(size):
    """Queries are as much larger, so that the logits are the same: keys from where the cache's fp16 has few bits left to
    where its values pass fp16's range (groups from a scale of 2^11 on are carried at another power of two)."""
    for new, ctx, h_q in (([40], [500], 2), ([140], [300], 2)):
        c = Case(3, new, ctx, h_q, 1)
        set_keys(c, size)
        c.q = torch.as_tensor(2.5 / size * c.rng.standard_normal(c.q.shape), dtype=torch.float32).bfloat16()
        close(c, c.run())


def test_small_keys_beside_huge_ones():
    """Tokens whose huge keys point away from every query have no weight, and take no bits of the others."""
    c = Case(4, [40], [300], 4, 1)
    set_keys(c, 1e-3)
    q = 2500 * c.rng.standard_normal(128)
    c.q = torch.as_tensor(np.broadcast_to(q, c.q.shape) * c.rng.uniform(0.2, 1.0, c.q.shape[:2] + (1,)), dtype=torch.float32).bfloat16()
    away = -q @ c.rk[0].astype(np.float64)
    for t in (0, 3, 130, 131, 250):
        int4.write_tokens(c.cache[c.bt[0, t // 16], 0], 0, t % 16, *int4.quantize(away * (5e4 / np.abs(away).max())))
    close(c, c.run())


@pytest.mark.parametrize("power,keys", [(-120, 1.0), (-60, 1.0), (60, 1.0), (108, 1.0), (115, 1.0), (117, 1.0), (121, 1e-2), (125, 1e-3)])
def test_queries_up_to_the_ends_of_their_type(power, keys):
    """Queries of 0.5 times 2^power, up to bf16's largest, and a scale that makes their logits ordinary ones."""
    c = Case(6, [40], [300], 4, 1)
    set_keys(c, keys)
    x = np.clip(0.5 * c.rng.standard_normal(c.q.shape), -1.9, 1.9)
    c.q = (torch.as_tensor(x, dtype=torch.float64) * 2.0 ** power).bfloat16()
    scale = float(np.float32(5 * SCALE / keys * 2.0 ** -power))
    close(c, run(c, scale), scale)


@pytest.mark.parametrize("length", [2.0 ** -11, 2.0 ** -8, 15.0, 40.0, 300.0, 2000.0])
def test_rotations_that_shorten_or_lengthen(length):
    """R_k of any norm that the header allows (a scale of the keys' channels may be folded into it)."""
    c = Case(7, [40], [300], 4, 1)
    c.rk = (length * c.rk).astype(np.float32)
    c.q = (c.q.float() / length).bfloat16()
    close(c, c.run())


def set_values(c, size):
    """Normal values, size [pages, H_kv, 16] (or a number) times themselves."""
    x = np.asarray(size)[..., None] * c.rng.standard_normal(c.cache.shape[:2] + (16, 128))
    for s in range(16):
        int4.write_tokens(c.cache, 1, s, *int4.quantize(x[:, :, s]))


def set_sinks(c, tokens, gap, size):
    """Queries along one direction, 0.3 to 1 times; tokens whose keys lie `gap` nats along it, with values of that size."""
    q = c.rng.standard_normal(128)
    c.q = torch.as_tensor(np.broadcast_to(q, c.q.shape) * c.rng.uniform(0.3, 1.0, c.q.shape[:2] + (1,)), dtype=torch.float32).bfloat16()
    for h in range(c.h_kv):
        k = q @ c.rk[h].astype(np.float64)
        for t in tokens:
            tile = c.cache[c.bt[0, t // 16], h]
            int4.write_tokens(tile, 0, t % 16, *int4.quantize(k * (gap / SCALE / (k @ k))))
            int4.write_tokens(tile, 1, t % 16, *int4.quantize(size * c.rng.standard_normal(128)))


@pytest.mark.parametrize("size", [0.0, 1e-6, 1e-3, 0.02, 0.3, 3.0, 100.0])
@pytest.mark.parametrize("gap", [5.0, 12.0, 17.0, 20.0, 24.0, 40.0, 75.0])
def test_sinks(gap, size):
    """A token that draws all of the weight, with values from none to far larger ones than the others': at the front, later
    in the context (where the reference is raised), the whole first tile, in a window's sinks; values of other sizes too."""
    for tokens, new, ctx, window, others in (((0,), [40], 500, 0, 1.0), ((0, 1, 2, 3), [70], 700, 0, 30.0), ((170,), [40], 400, 0, 1.0),
                                             (range(64), [40], 500, 0, 1.0), ((0, 2), [40], 700, 100, 1e-3)):
        c = Case(8, new, [ctx], 4, 1, window, 4 if window else 0)
        set_values(c, others)
        set_sinks(c, tokens, gap, size * others)
        close(c, c.run(), one_draw=True)


def test_values_of_sizes_that_differ_by_token():
    """Sizes spread over 35 powers of two from token to token, page to page, and zeros among them."""
    for seed, new, ctx, h_q in ((1, [60], [500], 4), (2, [300], [900], 2), (3, [20, 20], [300, 64], 4)):
        c = Case(seed, new, ctx, h_q, 1)
        shape = c.cache.shape[:2] + (16,)
        for size in (2.0 ** c.rng.uniform(-20, 15, shape), np.broadcast_to(2.0 ** c.rng.uniform(-20, 15, shape[:2] + (1,)), shape),
                     np.where(c.rng.random(shape) < 0.5, 0.0, 1.0), np.where(c.rng.random(shape[:2] + (1,)) < 0.5, 0.0, np.ones(shape))):
            set_values(c, size)
            close(c, c.run())


def test_values_past_the_type_s_largest():
    """min + 15 scale up to a million, which bf16 holds and fp16 does not."""
    c = Case(9, [40], [300], 4, 1)
    set_values(c, 2e5)
    close(c, c.run())
    set_values(c, np.where(c.rng.random(c.cache.shape[:2] + (16,)) < 0.1, 2e5, 1e-2))
    close(c, c.run())


def test_queries_and_scales_that_are_not_finite():
    """A query of NaN or infinity makes its own row NaN and no other; a scale of NaN every row that sees a token."""
    c = Case(10, [40], [30], 4, 2)               # rows before position 0 see nothing
    clean = c.run()
    for x in (float("nan"), float("inf"), -float("inf")):
        q = c.q.clone()
        q[25, 1, 7] = q[38, 3, 100] = x
        keep, c.q = c.q, q
        got = c.run()
        c.q = keep
        hit = torch.zeros(got.shape[:2], dtype=torch.bool)
        hit[25, 1] = hit[38, 3] = True
        assert torch.isnan(got[hit]).all() and torch.equal(got[~hit], clean[~hit])
    got = run(c, float("nan"))
    assert torch.isnan(got[10:]).all() and not got[:10].any()
