"""GPU parity of the INT4 decode where one CTA attends a long context of values around zero by nearly equal weights: the
output is a small remainder of large sums, so what the sums lose shows.

Tolerance in the 2-norm, with spread = |sum_s p_s (15 scale_s + |min_s|)|: 2^-8 of the output for its bf16 rounding; the
terms' two fp16 roundings, independent and 2^-11 each at most, at 4 times the root of their squares' sum; the sums' fp32
roundings, N a warp and to nearest, which leave about 0.2 sqrt(N) 2^-24 of spread (0.29 an ulp, a third for the growth),
at 8 times that for N = 2731 of the 512K tokens: 84 2^-24 < 2^-17.  (Sums that are cut off lose N 2^-24 and more: they
fail.)
"""
import numpy as np
import pytest
import torch

from bit_kv_cache_13_gb300 import _lib
from oracle import int4
from test_gpu_int4 import SCALE, _bf, _dev, _rot

pytestmark = pytest.mark.gpu
T = 1 << 19


@pytest.fixture(scope="module")
def context():
    rng = np.random.default_rng(0)
    P = T // 16
    tiles = rng.integers(0, 256, (P, 1, 2560), np.uint8)       # any codes
    scale = rng.uniform(0.05, 0.2, (2, P, 16, 4)).astype(np.float16)
    meta = tiles.view(np.float16)[:, 0]                        # [P, 1280]
    low = (scale.astype(np.float64) * -7.5).astype(np.float16)
    for s in range(16):
        for g in range(4):
            for side in (0, 1):
                at, at_min = int4.meta_address(side, s, g)
                meta[:, at // 2], meta[:, at_min // 2] = scale[side, :, s, g], low[side, :, s, g]
    k, v = (int4.values(tiles[:, 0], side).reshape(T, 128) for side in (0, 1))
    span = np.repeat((15 * scale[1].astype(np.float64) + np.abs(low[1].astype(np.float64))).reshape(T, 4), 32, -1)
    return tiles, k, v, span, _rot(rng, 1), _rot(rng, 1)


@pytest.mark.parametrize("g", [4, 8])
def test_sums_of_half_a_million_tokens_in_one_cta(context, g):
    tiles, k, v, span, rk, rv = context
    q = _bf(np.random.default_rng(g).standard_normal((1, g, 128)))
    out, P = torch.empty((1, g, 128), dtype=torch.bfloat16, device="cuda"), T // 16
    ws = torch.zeros(_lib.kvq_int4_workspace_bytes(1, g, 1, P, 1), dtype=torch.uint8, device="cuda")
    _lib.kvq_decode_attn_int4(q.cuda(), _dev(tiles), P, torch.arange(P, dtype=torch.int32, device="cuda")[None],
                              torch.tensor([T], dtype=torch.int32, device="cuda"), _dev(rk), _dev(rv), SCALE, out, ws, 1)
    assert _lib.kvq_workspace_status(ws) == 0
    got = out[0].double().cpu().numpy()
    for j in range(g):
        a = k @ (q[0, j].double().numpy() @ rk[0].astype(np.float64)) * SCALE
        p = np.exp(a - a.max())
        p /= p.sum()
        ref = (p @ v) @ rv[0].astype(np.float64).T
        tol = (2.0 ** -8 * np.linalg.norm(ref) + 4 * 2.0 ** -11 * 2 ** 0.5 * np.sqrt((p ** 2) @ span ** 2).max() * 128 ** 0.5 / 3 ** 0.5
               + 2.0 ** -17 * np.linalg.norm(p @ span))
        assert np.linalg.norm(got[j] - ref) <= tol, (j, np.linalg.norm(got[j] - ref), tol, np.linalg.norm(ref))
