"""Int4Layer's slots on the host: the step's new token stands at context_lens - 1, before an eviction and after."""
import pytest
import torch

from bit_kv_cache_13_gb300 import inputs
from bit_kv_cache_13_gb300.workload import Int4Layer

I32 = torch.int32


def _layer(ctx=100, pages=9):
    spec = inputs.small_spec("int4slots", h_q=4, h_kv=1, batch=2, ctx=ctx)
    return Int4Layer(spec, 0, device="cpu", block_table=torch.arange(2 * pages, dtype=I32).view(2, pages), extra_pages=8)


def test_new_slots_before_an_eviction():
    layer = _layer()
    assert layer.new_slots().tolist() == [6 * 16 + 3, (9 + 6) * 16 + 3]     # position 99 of either
    assert layer.new_slots().dtype == I32


@pytest.mark.parametrize("table", [4, 9])   # shorter than position ctx - 1, and longer
def test_new_slots_after_an_eviction(table):
    layer = _layer()
    # what evict leaves: another table, the kept lengths; then the step's token is counted
    layer.block_table = torch.arange(18, 18 + 2 * table, dtype=I32).view(2, table)
    layer.context_lens = torch.tensor([48, 7], dtype=I32)
    layer.context_lens += 1
    assert layer.new_slots().tolist() == [(18 + 3) * 16 + 0, (18 + table) * 16 + 7]


def test_new_slots_of_an_empty_sequence_and_past_the_table():
    layer = _layer()
    layer.context_lens = torch.tensor([0, 1], dtype=I32)
    assert layer.new_slots().tolist() == [-1, 9 * 16]         # no token: a slot that an append skips
    layer.context_lens = torch.tensor([1, 9 * 16 + 1], dtype=I32)
    with pytest.raises(IndexError):
        layer.new_slots()


def test_append_rope_takes_the_model_s_eps_and_clip(monkeypatch):
    from bit_kv_cache_13_gb300 import _lib
    layer, seen = _layer(), {}
    layer.mu = torch.zeros(1, 128)
    monkeypatch.setattr(_lib, "kvq_append_rope_int4", lambda *args, **kw: seen.update(kw))
    x = torch.zeros(3, 4, 128, dtype=torch.bfloat16)
    q, k = layer.append_rope(x, x[:, :1], x[:, :1], None, None, None, eps=1e-5, clip=0.9)
    assert q.shape == x.shape and k.shape == (3, 1, 128)
    assert seen["eps"] == 1e-5 and seen["clip"] == 0.9
    layer.append_rope(x, x[:, :1], x[:, :1], None, None, None)
    assert seen["eps"] == 1e-6 and seen["clip"] == 1.0
