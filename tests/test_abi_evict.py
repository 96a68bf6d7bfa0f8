"""Refusals of the eviction calls on the host (no GPU) where what they write overlaps what they read."""
import os

import pytest
import torch

from bit_kv_cache_13_gb300 import _lib, build

host_only = pytest.mark.skipif(torch.cuda.is_available(), reason="host-only checks with placeholder addresses")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.load()


W, LENS, KEEP, NEW = 0x100000, 0x200000, 0x300000, 0x400000   # placeholder addresses, never dereferenced
B, H, T, STRIDE, BUDGET = 3, 2, 100, 112, 8
W_END, KEEP_END = W + ((B * H - 1) * STRIDE + T) * 4, KEEP + B * H * BUDGET * 4


@host_only
@pytest.mark.parametrize("kw", [
    dict(new=LENS), dict(new=LENS + 4), dict(new=LENS - 8),          # the lengths in place, and partly
    dict(new=W), dict(new=W_END - 4), dict(new=W - 4 * B + 4),
    dict(keep=LENS), dict(keep=LENS - B * H * BUDGET * 4 + 4), dict(keep=W), dict(keep=W_END - 4),
    dict(new=KEEP_END - 4), dict(new=KEEP),
])
def test_overlapping_arguments_are_refused(lib, kw):
    a = dict(new=NEW, keep=KEEP) | kw
    st = lib.kvq_evict_select(W, STRIDE, B, H, T, LENS, BUDGET, 1, 1, a["keep"], a["new"], None)
    assert st == -1 and "overlap" in lib.kvq_last_error().decode()


@host_only
@pytest.mark.parametrize("kw", [dict(new=LENS + 4 * B), dict(new=LENS - 4 * B), dict(new=W_END), dict(keep=W_END), dict(new=KEEP_END)])
def test_neighbours_are_not(lib, kw):
    a = dict(new=NEW, keep=KEEP) | kw
    lib.kvq_evict_select(W, STRIDE, B, H, T, LENS, BUDGET, 1, 1, a["keep"], a["new"], None)
    assert "overlap" not in lib.kvq_last_error().decode()   # (it goes on to the device, of which there is none)


# rows of 64 floats (4 source pages) in, of 32 (2 destination pages) out
def _gather(lib, wo, stride, wo_stride, rows=(3, 2)):
    a, b = 0x800000, 0x900000
    lib.kvq_evict_gather_int4(a, 4, LENS, 4, KEEP, 20, NEW, *rows, 128, b, 4, LENS, 2, W, stride, wo, wo_stride, None, None)
    return "must not overlap weights" in lib.kvq_last_error().decode()


@host_only
@pytest.mark.parametrize("floats,stride,wo_stride", [(1, 64, 32), (5 * 64 + 63, 64, 32), (-5 * 32 - 31, 64, 32), (63, 96, 96), (65, 96, 96),
                                                     (64, 100, 96), (64 - 96, 95, 95)])
def test_weights_out_over_weights_is_refused(lib, floats, stride, wo_stride):
    assert _gather(lib, W + 4 * floats, stride, wo_stride)


@host_only
@pytest.mark.parametrize("floats,stride,wo_stride", [(6 * 64, 64, 32), (-6 * 32, 64, 32), (64, 96, 96), (64 - 2 * 96, 96, 96), (70, 128, 128)])
def test_weights_out_beside_or_between_rows_is_not(lib, floats, stride, wo_stride):
    assert not _gather(lib, W + 4 * floats, stride, wo_stride)
