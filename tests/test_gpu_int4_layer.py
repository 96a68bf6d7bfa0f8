"""The calls of one layer in the order of serving: a prompt in pieces from the projection's output (norms, rotation, append,
chunk attention), drafted tokens, then single tokens in a sliding window, on Int4Layer, against the fp64 oracle."""
import numpy as np
import pytest
import torch

from bit_kv_cache_13_gb300 import inputs
from bit_kv_cache_13_gb300.workload import Int4Layer
from oracle import int4

pytestmark = pytest.mark.gpu


def _close(got, want, bound):
    err = np.linalg.norm(got.double().cpu().numpy() - want, axis=-1)
    tol = bound + 2.0 ** -8 * np.linalg.norm(want, axis=-1)
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 4)])
def test_prompt_drafts_and_single_tokens(window, sinks):
    h_q, h_kv, B = 8, 2, 3
    rng = np.random.default_rng(7)
    spec = inputs.small_spec("serve", h_q=h_q, h_kv=h_kv, batch=B, ctx=600)
    pages = 40
    layer = Int4Layer(spec, 0, block_table=torch.as_tensor(rng.permutation(B * pages).reshape(B, pages), dtype=torch.int32))
    layer.mu = torch.as_tensor(rng.standard_normal((h_kv, 128)), dtype=torch.float32).cuda()
    layer.context_lens.zero_()
    table = inputs.rope_table(700, 128, 1e4).cuda()
    weight = [torch.as_tensor(1 + 0.2 * rng.standard_normal(128), dtype=torch.float32).bfloat16().cuda() for _ in range(2)]
    cache = layer.cache.cpu().numpy()
    bt, mu, rk, rv = layer.block_table.cpu().numpy(), layer.mu.cpu().numpy(), layer.R_k.cpu().numpy(), layer.R_v.cpu().numpy()
    lens = np.zeros(B, np.int64)
    for new in ([300, 17, 0], [200, 1, 65], [5, 5, 5], [1, 1, 1], [1, 1, 1]):
        start = np.cumsum([0] + new)
        n = int(start[-1])
        qkv = torch.as_tensor(rng.standard_normal((n, h_q + 2 * h_kv, 128)), dtype=torch.float32).bfloat16()
        pos = np.concatenate([lens[b] + np.arange(x) for b, x in enumerate(new)]).astype(np.int32)
        seq = np.repeat(np.arange(B), new)
        slots = (bt[seq, pos // 16] * 16 + pos % 16).astype(np.int32)
        lens += new
        layer.context_lens.copy_(torch.as_tensor(lens))
        q, k, v = qkv.cuda().split([h_q, h_kv, h_kv], 1)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        q_rot, k_rot = layer.append_rope(q, k, v, torch.as_tensor(pos).cuda(), table, torch.as_tensor(slots).cuda(), *weight, err_count=err)
        x = qkv.double().numpy()
        want_q, want_k = (int4.to_bf16(int4.norm_rope(x[:, a:b], pos, table.cpu().numpy(), w.double().cpu().numpy()))
                          for a, b, w in ((0, h_q, weight[0]), (h_q, h_q + h_kv, weight[1])))
        assert err.item() == 0 and np.array_equal(q_rot.double().cpu().numpy(), want_q) and np.array_equal(k_rot.double().cpu().numpy(), want_k)
        int4.append(cache, want_k, x[:, h_q + h_kv:], slots, mu, rk, rv)
        assert np.array_equal(layer.cache.cpu().numpy(), cache)
        want, bound = int4.chunk(want_q, start, cache, bt, lens, rk, rv, layer.scale, window, sinks)
        q_start = torch.as_tensor(start, dtype=torch.int32).cuda()
        out = torch.empty_like(q_rot)
        layer.chunk(q_rot, q_start, out, layer.chunk_workspace(n), window, sinks)
        _close(out, want, bound)
        if new == [1, 1, 1]:
            single = torch.empty_like(q_rot)
            layer.decode(q_rot, single, layer.workspace(weights=False), window=window, sinks=sinks)
            _close(single, want, bound)
