"""GPU accuracy of chunk attention over the INT4 cache where its operands are small, large or of very different sizes.

Tolerance.  oracle.int4.chunk_spread derives the variance of what fp16 operands leave of each output row; the rounding to
bf16 adds the distance of the exact row from the nearest bf16 one, which is known.  Over a call, the squared errors
relative to their rows' squared norms may sum to 1.1 times the sum of both: the variance is an upper bound (every rounding
as at the lower end of its power of two, where it is largest), and the two parts' product, which has no mean, is below
3 % of it at 4096 outputs or more.  Of a single row the bf16 rounding is at most 2^-8 of each value, and the rest is taken at
six standard deviations."""
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


def close(c, got, scale=SCALE):
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
    ratio = (err2[on] / size2[on]).sum() / ((near2[on] + var[on]) / size2[on]).sum()
    assert ratio <= 1.1, ratio


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
