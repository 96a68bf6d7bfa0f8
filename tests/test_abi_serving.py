"""Refusals of the append with norms and rotation, of chunk attention and of the sliding decode on the host (no GPU)."""
import os

import pytest
import torch

from bit_kv_cache_13_gb300 import _lib, build

host_only = pytest.mark.skipif(torch.cuda.is_available(), reason="host-only checks with placeholder addresses")
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
A, MIS = 0x10000, 0x10004   # placeholder addresses, never dereferenced
Q, K, V, QO, KO = (0x100000 * i for i in range(1, 6))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.load()


def _refused(lib, st, status, text):
    assert st == status and text in lib.kvq_last_error().decode(), lib.kvq_last_error()


@host_only
@pytest.mark.parametrize("kw,status,text", [
    (dict(d=64), UNSUPPORTED, "d=64"), (dict(n=-1), INVALID, "n_tok=-1"), (dict(H_q=0), INVALID, "H_q=0"),
    (dict(H_kv=0), INVALID, "H_kv=0"), (dict(H_q=70000), UNSUPPORTED, "too large"), (dict(num_pages=0), INVALID, "num_pages=0"),
    (dict(max_pos=0), INVALID, "max_pos=0"), (dict(rot=8), INVALID, "rot_dim=8"), (dict(rot=0), INVALID, "rot_dim=0"),
    (dict(rot=144), INVALID, "rot_dim=144"), (dict(rot=40), INVALID, "rot_dim=40"), (dict(eps=-1.0), INVALID, "eps"),
    (dict(eps=float("nan")), INVALID, "eps"), (dict(eps=float("inf")), INVALID, "eps"), (dict(clip=0.0), INVALID, "clip"),
    (dict(q=None), INVALID, "null"), (dict(k=None), INVALID, "null"), (dict(v=None), INVALID, "null"),
    (dict(q_out=None), INVALID, "null"), (dict(k_out=None), INVALID, "null"), (dict(rope=None), INVALID, "null"),
    (dict(positions=None), INVALID, "null"), (dict(q=Q + 4), INVALID, "aligned"), (dict(rope=MIS), INVALID, "aligned"),
    (dict(qw=MIS), INVALID, "aligned"), (dict(k_out=KO + 8), INVALID, "aligned"), (dict(qs=511), INVALID, "stride"),
    (dict(qs=516), INVALID, "stride"), (dict(ks=120), INVALID, "stride"), (dict(vs=132), INVALID, "stride"),
    (dict(qs=1 << 40), INVALID, "stride"), (dict(q_out=Q + 1024), INVALID, "overlap"), (dict(q_out=Q, qs=520), INVALID, "overlap"),
    (dict(k_out=V), INVALID, "overlap"), (dict(q_out=KO), INVALID, "overlap"), (dict(k_out=Q), INVALID, "overlap"),
    (dict(q_out=K), INVALID, "overlap"),
])
def test_append_rope_refuses(lib, kw, status, text):
    a = dict(q=Q, qs=512, k=K, ks=128, v=V, vs=128, n=4, H_q=4, H_kv=1, d=128, positions=A, rope=A, max_pos=10, rot=128, qw=None,
             kw=None, eps=1e-6, clip=1.0, num_pages=4, q_out=QO, k_out=KO) | kw
    st = lib.kvq_append_rope_int4(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["n"], a["H_q"], a["H_kv"], a["d"], a["positions"],
                                  a["rope"], a["max_pos"], a["rot"], 0, a["qw"], a["kw"], a["eps"], A, A, A, A, a["clip"], A,
                                  a["num_pages"], a["q_out"], a["k_out"], None, None)
    _refused(lib, st, status, text)


@host_only
def test_empty_calls_are_no_ops(lib):
    assert lib.kvq_append_rope_int4(None, 0, None, 0, None, 0, 0, 4, 1, 128, None, None, 10, 128, 0, None, None, 1e-6, None, None, None,
                                    None, 1.0, None, 4, None, None, None, None) == 0
    assert lib.kvq_chunk_attn_int4(None, 0, None, 2, 4, 1, 128, None, 4, None, 4, None, None, None, 1.0, 0, 0, None, None, 0, None) == 0


@host_only
@pytest.mark.parametrize("kw,status,text", [
    (dict(d=64), UNSUPPORTED, "d=64"), (dict(n=-1), INVALID, "n_tok=-1"), (dict(B=0), INVALID, "B=0"),
    (dict(H_q=6, H_kv=4), INVALID, "H_q=6"), (dict(H_q=65), UNSUPPORTED, "group above 64"), (dict(B=70000), UNSUPPORTED, "65535"),
    (dict(n=1 << 29), UNSUPPORTED, "2^30"), (dict(max_pages=1 << 27), UNSUPPORTED, "2^27"), (dict(max_pages=0), INVALID, "max_pages=0"),
    (dict(num_pages=0), INVALID, "num_pages=0"), (dict(num_pages=1 << 33), UNSUPPORTED, "2^32"), (dict(window=-1), INVALID, "window=-1"),
    (dict(sinks=-1), INVALID, "sinks=-1"), (dict(q=None), INVALID, "null"), (dict(start=None), INVALID, "null"),
    (dict(out=None), INVALID, "null"), (dict(ws=None), INVALID, "null"), (dict(out=MIS), INVALID, "alignment"),
    (dict(ws=MIS), INVALID, "alignment"), (dict(q=MIS), INVALID, "alignment"), (dict(ws_bytes=255), WORKSPACE, "workspace"),
])
def test_chunk_refuses(lib, kw, status, text):
    a = dict(q=A, n=7, start=A, B=2, H_q=4, H_kv=1, d=128, num_pages=4, max_pages=4, window=0, sinks=0, out=A, ws=A, ws_bytes=1 << 30) | kw
    st = lib.kvq_chunk_attn_int4(a["q"], a["n"], a["start"], a["B"], a["H_q"], a["H_kv"], a["d"], A, a["num_pages"], A, a["max_pages"], A,
                                 A, A, 0.1, a["window"], a["sinks"], a["out"], a["ws"], a["ws_bytes"], None)
    _refused(lib, st, status, text)


@host_only
def test_chunk_workspace_of_refused_sizes(lib):
    assert lib.kvq_chunk_workspace_bytes(7, 2, 4, 1) > 0
    for bad in ((-1, 2, 4, 1), (7, 0, 4, 1), (7, 2, 5, 2), (7, 2, 65, 1), (1 << 29, 1, 4, 1)):
        assert lib.kvq_chunk_workspace_bytes(*bad) == 0


@host_only
@pytest.mark.parametrize("kw,status,text", [
    (dict(window=0), INVALID, "window=0"), (dict(window=-5), INVALID, "window=-5"), (dict(sinks=-1), INVALID, "sinks=-1"),
    (dict(d=64), UNSUPPORTED, "d=64"), (dict(H_q=9), UNSUPPORTED, "group above 8"), (dict(ws_bytes=64), WORKSPACE, "workspace"),
    (dict(out=None), INVALID, "null"), (dict(q=MIS), INVALID, "alignment"),
])
def test_sliding_refuses(lib, kw, status, text):
    a = dict(q=A, B=1, H_q=4, H_kv=1, d=128, window=16, sinks=4, out=A, ws=A, ws_bytes=1 << 30) | kw
    st = lib.kvq_decode_attn_int4_sliding(a["q"], a["B"], a["H_q"], a["H_kv"], a["d"], A, 4, A, 4, A, A, A, 0.1, a["window"], a["sinks"],
                                          a["out"], a["ws"], a["ws_bytes"], 0, None)
    _refused(lib, st, status, text)


@host_only
def test_binding_refuses_tensors(lib):
    x = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        _lib.kvq_chunk_attn_int4(x, None, torch.zeros(4, 1, 2560, dtype=torch.uint8), 4, torch.zeros(1, 4, dtype=torch.int32),
                                 torch.zeros(1, dtype=torch.int32), torch.zeros(1, 128, 128), None, 0.1, x, x)
    with pytest.raises(ValueError, match="contiguous"):
        _lib._heads(torch.zeros(2, 128, 4, dtype=torch.bfloat16).transpose(1, 2), 2, -1, "q")
    with pytest.raises(ValueError, match="shape"):
        _lib._heads(x, 3, -1, "q")


def test_chunk_workspace_serves_smaller_calls(lib):
    """A workspace for the largest call of a shape holds any with fewer tokens or sequences."""
    sizes = [1, 2, 3, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000, 4095, 4096, 30000, 65535]
    for h_q, h_kv in ((1, 1), (4, 1), (32, 8), (64, 8), (64, 1)):
        for fixed in sizes:
            by_tokens = [lib.kvq_chunk_workspace_bytes(n, fixed, h_q, h_kv) for n in sizes]
            by_batch = [lib.kvq_chunk_workspace_bytes(fixed, b, h_q, h_kv) for b in sizes]
            assert by_tokens == sorted(by_tokens) and by_batch == sorted(by_batch), (fixed, h_q, h_kv)
            # where blocks of 256 rows take over from those of 128: 128 rows a sequence
            edge = 128 * fixed // (h_q // h_kv)
            around = [lib.kvq_chunk_workspace_bytes(n, fixed, h_q, h_kv) for n in range(max(edge - 2, 1), edge + 3)]
            assert around == sorted(around), (fixed, h_q, h_kv, around)
