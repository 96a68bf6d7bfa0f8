"""GPU parity of eviction (selection by accumulated weight, move of the kept tokens) against the oracle: indices, moved
bytes and weights are equal, none of them is computed."""
import numpy as np
import pytest
import torch

from bit_kv_cache_13_gb300 import _lib, inputs
from bit_kv_cache_13_gb300.workload import Int4Layer
from oracle import int4

pytestmark = pytest.mark.gpu
I32 = torch.int32


def _c(x):
    return torch.as_tensor(np.ascontiguousarray(x)).cuda()


def _select(w, ctx, budget, sinks, recent):
    B, h, T = w.shape
    keep = torch.full((B, h, budget), 77, dtype=I32, device="cuda")
    new = torch.full((B,), 77, dtype=I32, device="cuda")
    _lib.kvq_evict_select(_c(w), _c(np.asarray(ctx, np.int32)), budget, sinks, recent, keep, new)
    return keep.cpu().numpy(), new.cpu().numpy()


def _weights(rng, kind, shape):
    w = np.exp(2.5 * rng.standard_normal(shape)).astype(np.float32)
    if kind == "ties":
        w = rng.integers(0, 4, shape).astype(np.float32)
    if kind == "equal":
        w[:] = 0.0
    if kind == "special":
        w = rng.choice(np.array([np.nan, np.inf, -np.inf, 0.0, -0.0, -1.5, 2.0, 1e-45, -1e-45], np.float32), shape)
    if kind == "near":   # keys that differ in their last bits only
        w = (np.float32(1.0).view(np.uint32) + rng.integers(0, 300, shape).astype(np.uint32)).view(np.float32)
    return w


@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "special", "near"])
@pytest.mark.parametrize("ctx,budget,sinks,recent", [
    ([1], 1, 0, 0), ([2], 1, 0, 0), ([17, 5], 5, 1, 2), ([100, 0, 33], 32, 4, 8), ([1025], 1024, 4, 128), ([1024, 3000], 777, 0, 0),
    ([500], 8, 4, 4), ([500], 8, 0, 8), ([2049, 700], 1, 1, 0), ([2500, -4, 9000], 2047, 3, 60),
])
def test_select_matches_oracle(kind, ctx, budget, sinks, recent):
    rng = np.random.default_rng([budget, len(ctx)])
    w = _weights(rng, kind, (len(ctx), 2, max(max(ctx), 1) + 3))
    keep, new = _select(w, ctx, budget, sinks, recent)
    want, wnew = int4.select(w, ctx, budget, sinks, recent)
    assert np.array_equal(new, wnew) and np.array_equal(keep, want)


@pytest.mark.parametrize("T,budget", [(40_000, 39_999), (131_072, 8192), (300_001, 1000), (600_000, 50_000), (2_500_000, 7)])
def test_select_long_rows(T, budget):
    rng = np.random.default_rng(T)
    for kind in ("spread", "ties"):
        w = _weights(rng, kind, (1, 1, T))
        keep, _ = _select(w, [T], budget, 4, budget // 8)
        mid = np.arange(4, T - budget // 8)
        best = mid[np.lexsort((mid, -w[0, 0, mid].astype(np.float64)))[: budget - 4 - budget // 8]]
        want = np.sort(np.concatenate([np.arange(4), best, np.arange(T - budget // 8, T)]))
        assert np.array_equal(keep[0, 0], want)


def test_context_past_the_row_is_clamped():
    w = _weights(np.random.default_rng(0), "spread", (1, 1, 64))
    keep, new = _select(w, [1000], 16, 2, 2)
    want, wnew = int4.select(w, [1000], 16, 2, 2)
    assert np.array_equal(keep, want) and new.tolist() == wnew.tolist() == [16]


def test_many_rows():
    rng = np.random.default_rng(11)
    w = _weights(rng, "spread", (40, 8, 700))
    ctx = rng.integers(0, 700, 40)
    keep, new = _select(w, ctx, 128, 4, 16)
    want, wnew = int4.select(w, ctx, 128, 4, 16)
    assert np.array_equal(keep, want) and np.array_equal(new, wnew)


def _move(rng, ctx, budget, h, extra_dst=0):
    B = len(ctx)
    P, Q = max(1, (max(ctx) + 15) // 16), (budget + 15) // 16 + extra_dst
    n = B * P + B * Q + 3
    perm = rng.permutation(n).astype(np.int32)
    pool = rng.integers(0, 256, (n, h, 2560)).astype(np.uint8)
    bt, dbt = perm[: B * P].reshape(B, P), perm[B * P: B * P + B * Q].reshape(B, Q)
    w = rng.random((B, h, P * 16)).astype(np.float32)
    keep, new = int4.select(w, ctx, budget, min(2, budget // 2), budget // 4)
    return pool, bt, dbt, w, keep, new


@pytest.mark.parametrize("ctx,budget,h,extra", [([5], 3, 1, 0), ([40, 7], 16, 2, 0), ([100, 0, 64], 33, 3, 2), ([500], 130, 8, 1),
                                               ([33, 48], 48, 2, 0)])
def test_gather_matches_oracle(ctx, budget, h, extra):
    rng = np.random.default_rng([budget, h])
    pool, bt, dbt, w, keep, new = _move(rng, ctx, budget, h, extra)
    gpu = _c(pool)      # one pool for both: the destination pages are others
    wo = torch.full((len(ctx), h, dbt.shape[1] * 16 + 3), 5.0, device="cuda")
    err = torch.zeros(1, dtype=I32, device="cuda")
    _lib.kvq_evict_gather_int4(gpu, gpu.shape[0], _c(bt), _c(keep), _c(new), gpu, gpu.shape[0], _c(dbt), _c(w), wo, err)
    torch.cuda.synchronize()
    want = pool.copy()
    wref = int4.gather(pool, bt, keep, new, want, dbt, w)
    assert int(err) == 0
    assert np.array_equal(gpu.cpu().numpy(), want)     # slots past new_lens and all other pages untouched
    assert np.array_equal(wo.cpu().numpy()[..., :-3], wref) and bool((wo[..., -3:] == 5.0).all())


def test_gather_without_weights_and_bad_entries():
    rng = np.random.default_rng(8)
    pool, bt, dbt, w, keep, new = _move(rng, [100, 60], 40, 2, 1)
    n = pool.shape[0]
    keep, bt, dbt = keep.copy(), bt.copy(), dbt.copy()
    keep[0, 0, 5], keep[0, 0, 6] = -2, 5000                # indices outside the sequence's pages
    bt[1, 1], dbt[0, 1] = n, -1                            # a source and a destination page outside the pool
    gpu = _c(pool)
    err = torch.zeros(1, dtype=I32, device="cuda")
    wo = torch.full((2, 2, dbt.shape[1] * 16), 5.0, device="cuda")
    _lib.kvq_evict_gather_int4(gpu, n, _c(bt), _c(keep), _c(new), gpu, n, _c(dbt), _c(w), wo, err)
    want, bad, wref = pool.copy(), 0, np.zeros(wo.shape, np.float32)
    for b in range(2):
        for h in range(2):
            for i in range(int(new[b])):
                s = int(keep[b, h, i])
                src = bt[b][s // 16] if 0 <= s < bt.shape[1] * 16 else -1
                to = dbt[b][i // 16]
                if 0 <= src < n:
                    wref[b, h, i] = w[b, h, s]
                if not (0 <= src < n and 0 <= to < n):
                    bad += 1
                    continue
                for side in (0, 1):
                    int4.write_tokens(want[to, h], side, i % 16, *int4.read_token(pool[src, h], side, s % 16))
    assert int(err) == bad > 0
    assert np.array_equal(gpu.cpu().numpy(), want) and np.array_equal(wo.cpu().numpy(), wref)
    gpu2 = _c(pool)
    _lib.kvq_evict_gather_int4(gpu2, n, _c(bt), _c(keep), _c(new), gpu2, n, _c(dbt))
    assert np.array_equal(gpu2.cpu().numpy(), want)


def test_select_refuses_on_the_gpu_too():
    w = torch.zeros((1, 1, 64), device="cuda")
    n, keep = torch.zeros(1, dtype=I32, device="cuda"), torch.zeros((1, 1, 8), dtype=I32, device="cuda")
    with pytest.raises(_lib.KvqError, match="above the budget"):
        _lib.kvq_evict_select(w, n, 8, 5, 4, keep, n.clone())


@pytest.mark.parametrize("captured", [False, True])
def test_a_serving_run(captured):
    """Prefill, steps that append and attend with weights, eviction when the cache is full, more steps: every attention
    equals the oracle's over the tokens that the heads kept."""
    spec = inputs.small_spec("evictrun", h_q=8, h_kv=2, batch=2, ctx=200, permute=True)
    total, free = 2 * 13, 2 * 7
    layer = Int4Layer(spec, 0, block_table=torch.arange(total, dtype=I32).view(2, 13), extra_pages=free)
    layer.prefill()
    layer.context_lens = torch.full((2,), 199, dtype=I32, device="cuda")
    out = torch.empty((2, 8, 128), dtype=torch.bfloat16, device="cuda")
    ws = layer.workspace()
    rng = np.random.default_rng(0)
    wref = np.zeros((2, 2, layer.weights.shape[2]))
    n = lambda x: x.cpu().numpy()  # noqa: E731

    def step():
        nonlocal wref
        pos = layer.context_lens.cpu().long()
        kv = [torch.as_tensor(rng.standard_normal((2, 2, 128)), dtype=torch.bfloat16).cuda() for _ in range(2)]
        slots = torch.stack([layer.block_table[b, pos[b] // 16] * 16 + int(pos[b]) % 16 for b in range(2)]).to(I32)
        layer.append(*kv, slots)
        layer.context_lens += 1
        q = torch.as_tensor(rng.standard_normal((2, 8, 128)) * 2, dtype=torch.bfloat16).cuda()
        layer.decode(q, out, ws, decay=1.0)
        torch.cuda.synchronize()
        want, wref = int4.decode(q.double().cpu().numpy(), n(layer.cache), n(layer.block_table), n(layer.context_lens),
                                 n(layer.R_k), n(layer.R_v), layer.scale, wref, 1.0)
        got = out.double().cpu().numpy()
        for b in range(2):
            for j in range(8):   # bf16 rounding 2^-8, fp16 weights 2^-10 of terms that may be several times the result
                assert np.linalg.norm(got[b, j] - want[b, j]) <= 2.0 ** -7 * np.linalg.norm(want[b, j])
        # six steps of weights below 4, each good to 2^-15
        assert np.max(np.abs(n(layer.weights) - wref)) <= 6 * 4 * 2.0 ** -15

    for _ in range(3):
        step()
    dst = torch.arange(total, total + free, dtype=I32, device="cuda").view(2, 7)
    before, w_before = n(layer.cache), n(layer.weights)
    old_bt, old_n = n(layer.block_table), n(layer.context_lens)
    if captured:
        layer.evict(96, 4, 16, dst)
        layer.block_table, layer.context_lens, layer.weights = _c(old_bt), _c(old_n), _c(w_before)
        layer.cache.copy_(torch.as_tensor(before))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            keep = layer.evict(96, 4, 16, dst)
        graph.replay()
    else:
        keep = layer.evict(96, 4, 16, dst)
    torch.cuda.synchronize()
    want_keep, want_new = int4.select(w_before, old_n, 96, 4, 16)
    assert np.array_equal(n(keep), want_keep) and layer.context_lens.tolist() == want_new.tolist() == [96, 96]
    moved = before.copy()
    wref = int4.gather(before, old_bt, want_keep, want_new, moved, n(dst), w_before).astype(np.float64)
    assert np.array_equal(n(layer.cache), moved)
    ws = layer.workspace()
    for _ in range(3):
        step()
    assert layer.context_lens.tolist() == [99, 99]
