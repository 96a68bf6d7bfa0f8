"""Refusals of the INT4 and eviction entry points on the host (no GPU): the C ABI checks its arguments before it touches
CUDA, the binding checks the tensors before it calls the library."""
import os

import pytest
import torch

from bit_kv_cache_13_gb300 import _lib, build

host_only = pytest.mark.skipif(torch.cuda.is_available(), reason="host-only checks with placeholder addresses")
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
A, MIS = 0x10000, 0x10004   # placeholder addresses, never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.load()


def _refused(lib, st, status, text):
    assert st == status and text in lib.kvq_last_error().decode(), lib.kvq_last_error()


@host_only
@pytest.mark.parametrize("kw,status,text", [
    (dict(d=64), UNSUPPORTED, "d=64"), (dict(n=-1), INVALID, "n_tok=-1"), (dict(H_kv=0), INVALID, "H_kv=0"),
    (dict(H_kv=70000), UNSUPPORTED, "too large"), (dict(num_pages=0), INVALID, "num_pages=0"),
    (dict(clip=0.0), INVALID, "clip"), (dict(clip=1.01), INVALID, "clip"), (dict(clip=float("nan")), INVALID, "clip"),
    (dict(k=None), INVALID, "null"), (dict(cache=MIS), INVALID, "aligned"),
    (dict(k=MIS), INVALID, "aligned"),
])
def test_append_refuses(lib, kw, status, text):
    a = dict(k=A, n=4, H_kv=1, d=128, clip=1.0, cache=A, num_pages=4) | kw
    st = lib.kvq_append_int4(a["k"], A, a["n"], a["H_kv"], a["d"], A, A, A, A, a["clip"], a["cache"], a["num_pages"], None,
                             None)
    _refused(lib, st, status, text)


@host_only
def test_empty_append_and_read_are_no_ops(lib):
    assert lib.kvq_append_int4(None, None, 0, 1, 128, None, None, None, None, 1.0, None, 4, None, None) == 0
    assert lib.kvq_dequant_int4(None, 4, 1, 128, None, 0, None, None, None) == 0
    _refused(lib, lib.kvq_dequant_int4(A, 4, 1, 128, A, 3, None, None, None), INVALID, "null")


@host_only
@pytest.mark.parametrize("kw,status,text", [
    (dict(d=64), UNSUPPORTED, "d=64"), (dict(B=0), INVALID, "B=0"), (dict(H_q=6, H_kv=4), INVALID, "H_q=6"),
    (dict(H_q=9), UNSUPPORTED, "group above 8"), (dict(max_pages=1 << 27), UNSUPPORTED, "2^27"),
    (dict(splits=255), INVALID, "above 254"), (dict(B=60000, H_kv=300, H_q=300), UNSUPPORTED, "2^24"),
    (dict(B=60000, splits=100), UNSUPPORTED, "2^22"), (dict(B=60000, max_pages=1 << 26), UNSUPPORTED, "2^36"), (dict(splits=-1), INVALID, "splits=-1"), (dict(q=None), INVALID, "null"),
    (dict(out=MIS), INVALID, "alignment"), (dict(ws=MIS), INVALID, "alignment"), (dict(ws_bytes=64), WORKSPACE, "workspace"),
    (dict(B=70000), UNSUPPORTED, "65535"), (dict(w=None), INVALID, "null"), (dict(stride=63), INVALID, "weights_stride"),
    (dict(decay=-0.5), INVALID, "decay"), (dict(decay=float("nan")), INVALID, "decay"),
    (dict(decay=float("inf")), INVALID, "decay"),
])
def test_decode_refuses(lib, kw, status, text):
    a = dict(q=A, B=1, H_q=4, H_kv=1, d=128, max_pages=4, out=A, w=A, stride=64, decay=1.0, ws=A, ws_bytes=1 << 20,
             splits=0) | kw
    head = (a["q"], a["B"], a["H_q"], a["H_kv"], a["d"], A, 10, A, a["max_pages"], A, A, A, 0.1, a["out"])
    st = lib.kvq_decode_attn_int4_weights(*head, a["w"], a["stride"], a["decay"], a["ws"], a["ws_bytes"], a["splits"], None)
    _refused(lib, st, status, text)
    if not {"w", "stride", "decay"} & set(kw):
        _refused(lib, lib.kvq_decode_attn_int4(*head, a["ws"], a["ws_bytes"], a["splits"], None), status, text)


def test_workspace_bytes(lib):
    small = _lib.kvq_int4_workspace_bytes(1, 8, 2, 100, 0)
    assert 256 < small < _lib.kvq_int4_workspace_bytes(1, 8, 2, 100, 0, True)
    # the weights form holds 16 * 100 logits of every query head more
    assert _lib.kvq_int4_workspace_bytes(1, 8, 2, 100, 3, True) >= _lib.kvq_int4_workspace_bytes(1, 8, 2, 100, 3) + 4 * 8 * 1600
    for bad in ((0, 8, 2, 100, 0), (1, 7, 2, 100, 0), (1, 8, 2, 0, 0), (1, 8, 2, 100, -1), (1, 8, 2, 100, 255),
                (1, 8, 2, 1 << 27, 0), (1, 9, 1, 100, 0), (60000, 300, 300, 1, 0), (60000, 1, 1, 1, 100),
                (60000, 1, 1, 1 << 26, 0), (70000, 1, 1, 1, 0)):
        assert _lib.kvq_int4_workspace_bytes(*bad) == 0
    assert _lib.kvq_int4_tile_bytes(128) == 2560 and _lib.kvq_int4_tile_bytes(64) == 0


@host_only
@pytest.mark.parametrize("kw,status,text", [
    (dict(B=0), INVALID, "B=0"), (dict(budget=0), INVALID, "budget=0"), (dict(sinks=-1), INVALID, "sinks=-1"),
    (dict(recent=-2), INVALID, "recent=-2"), (dict(sinks=5, recent=4), INVALID, "above the budget"),
    (dict(sinks=2**31 - 1, recent=2**31 - 1), INVALID, "above the budget"), (dict(stride=99), INVALID, "weights_stride"),
    (dict(w=None), INVALID, "null"), (dict(B=70000), UNSUPPORTED, "65535"),
    (dict(T=(1 << 30) + 1, stride=1 << 31), UNSUPPORTED, "2^30"),
])
def test_select_refuses(lib, kw, status, text):
    a = dict(w=A, stride=100, B=1, H_kv=1, T=100, budget=8, sinks=1, recent=1) | kw
    _refused(lib, lib.kvq_evict_select(a["w"], a["stride"], a["B"], a["H_kv"], a["T"], A, a["budget"], a["sinks"],
                                       a["recent"], A, A, None), status, text)


@host_only
@pytest.mark.parametrize("kw,status,text", [
    (dict(d=64), UNSUPPORTED, "d=64"), (dict(budget=0), INVALID, "budget=0"), (dict(dst_max=1), INVALID, "destination"),
    (dict(cache=MIS), INVALID, "alignment"), (dict(dst=MIS), INVALID, "alignment"), (dict(keep=None), INVALID, "null"),
    (dict(wo=None), INVALID, "null"), (dict(stride=1), INVALID, "strides"), (dict(wo=A), INVALID, "is weights"),
    (dict(dst_max=1 << 27), UNSUPPORTED, "2^27"), (dict(H_kv=70000), UNSUPPORTED, "65535"),
])
def test_gather_refuses(lib, kw, status, text):
    a = dict(cache=A, keep=A, budget=20, H_kv=1, d=128, dst=A, dst_max=2, w=A, stride=64, wo=2 * A, wo_stride=32) | kw
    _refused(lib, lib.kvq_evict_gather_int4(a["cache"], 4, A, 4, a["keep"], a["budget"], A, 1, a["H_kv"], a["d"], a["dst"], 4,
                                            A, a["dst_max"], a["w"], a["stride"], a["wo"], a["wo_stride"], None, None),
             status, text)


def _t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def test_binding_checks_shapes_types_and_device():
    bf, i32, u8 = torch.bfloat16, torch.int32, torch.uint8
    k, mu, R, slots = _t(3, 2, 128, dtype=bf), _t(2, 128), _t(2, 128, 128), _t(3, dtype=i32)
    cache = _t(4, 2, 2560, dtype=u8)
    for args, text in (((k, k[:2], slots, mu, R, R, cache, 4), "v must have shape"),
                       ((k, k, slots[:2], mu, R, R, cache, 4), "slot_mapping"),
                       ((k, k, slots, mu[:1], R, R, cache, 4), "mu_k"),
                       ((k, k, slots, mu, R, R, cache, 5), "cache holds"),
                       ((k, k, slots, mu, R, R, cache, 4), "CUDA tensor")):
        with pytest.raises(ValueError, match=text):
            _lib.kvq_append_int4(*args)
    q, bt, lens, out, ws = _t(1, 4, 128, dtype=bf), _t(1, 4, dtype=i32), _t(1, dtype=i32), _t(1, 4, 128, dtype=bf), _t(64, dtype=u8)
    for args, text in (((q, cache, 4, bt[0], lens, R, R, 0.1, out, ws), "block_table"),
                       ((q, cache, 4, bt, _t(2, dtype=i32), R, R, 0.1, out, ws), "context_lens"),
                       ((q, cache, 4, bt, lens, R, R[:1], 0.1, out, ws), "R_v"),
                       ((q, cache, 4, bt, lens, R, R, 0.1, out[:, :2], ws), "out")):
        with pytest.raises(ValueError, match=text):
            _lib.kvq_decode_attn_int4(*args)
    with pytest.raises(ValueError, match="weights must have shape"):
        _lib.kvq_decode_attn_int4_weights(q, cache, 4, bt, lens, R, R, 0.1, out, _t(1, 1, 64), 1.0, ws)
    with pytest.raises(ValueError, match="err_count must have"):
        _lib.kvq_append_int4(k, k, slots, mu, R, R, cache, 4, 1.0, _t(0, dtype=i32))
    with pytest.raises(ValueError, match="keep"):
        _lib.kvq_evict_select(_t(1, 2, 64), lens, 8, 0, 0, _t(1, 2, 9, dtype=i32), lens)
    keep = _t(1, 2, 8, dtype=i32)
    for args, text in (((cache, 4, bt, keep, lens, cache, 4, bt, _t(1, 2, 64), None), "go together"),
                       ((cache, 4, bt, keep, lens, cache, 9, bt), "dst_cache holds"),
                       ((cache, 4, bt, keep, _t(2, dtype=i32), cache, 4, bt), "new_lens"),
                       ((cache, 4, bt, keep, lens, cache, 4, _t(2, 4, dtype=i32)), "dst_block_table")):
        with pytest.raises(ValueError, match=text):
            _lib.kvq_evict_gather_int4(*args)
