"""ctypes binding of libkvq.so (include/kvq.h), same names as the C ABI.

Argument marshalling only: tensors are checked for device, dtype and
contiguity, their device pointers and the current CUDA stream are passed to
the library, and a non-zero status raises KvqError with the library's error
text.  Every step of the path runs in the library's kernels; there is no
fallback of any kind.
"""
from __future__ import annotations

import ctypes as C
import os
import re

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libkvq.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "kvq.h")

_lib = None

P, I, I64, SZ, F, D = C.c_void_p, C.c_int, C.c_int64, C.c_size_t, C.c_float, C.c_double

_SIGS = {
    "kvq_last_error": ([], C.c_char_p),
    "kvq_int2_tile_bytes": ([I], SZ),
    "kvq_append_int2": ([P, P, I, I, I, P, P, P, P, P, I64, P, P, P, P], I),
    "kvq_decode_workspace_bytes": ([I, I, I, I, I], SZ),
    "kvq_decode_auto_splits": ([I, I, I, I], I),
    "kvq_decode_attn_int2": ([P, I, I, I, I, P, I64, P, I, P, P, P, F, P, P, SZ, I, P], I),
    "kvq_decode_attn_int2_window": ([P, I, I, I, I, P, I64, P, I, P, P, P, P, P, P, P, I, F, P, P, SZ, I, P], I),
    "kvq_workspace_status": ([P, P], I),
    "kvq_append_int2_clip": ([P, P, I, I, I, P, P, P, P, F, P, I64, P, P, P, P], I),
    "kvq_dequant_int2": ([P, I64, I, I, P, I, P, P, P], I),
    "bgtq_energy_scores": ([P, P, I, I, I, I, P, P, P], I),
    "kvq_decode_attn_int2_noalloc": ([P, I, I, I, I, P, I64, P, I, P, P, P, F, P, I, P], I),
    "kvq_debug_drop_next_copy": ([], None),
    "kvq_decode_step_int2": ([P, P, P, I, I, I, I, P, I64, P, I, P, P, P, P, F, P, P, SZ, I, I, P], I),
    "kvq_int4_tile_bytes": ([I], SZ),
    "kvq_append_int4": ([P, P, I, I, I, P, P, P, P, F, P, I64, P, P], I),
    "kvq_dequant_int4": ([P, I64, I, I, P, I, P, P, P], I),
    "kvq_int4_workspace_bytes": ([I, I, I, I, I, I], SZ),
    "kvq_decode_attn_int4": ([P, I, I, I, I, P, I64, P, I, P, P, P, F, P, P, SZ, I, P], I),
    "kvq_decode_attn_int4_weights": ([P, I, I, I, I, P, I64, P, I, P, P, P, F, P, P, I64, F, P, SZ, I, P], I),
    "kvq_evict_select": ([P, I64, I, I, I, P, I, I, I, P, P, P], I),
    "kvq_evict_gather_int4": ([P, I64, P, I, P, I, P, I, I, I, P, I64, P, I, P, I64, P, I64, P, P], I),
    "bgtq_lloyd_max_codebook": ([I, P], I),
    "bgtq_allocate": ([P, I, I, I, I64, P], I),
    "bgtq_tile_bytes": ([I, I], SZ),
    "bgtq_append": ([P, P, I, I, I, P, P, I, I, P, P, P, P, I64, P, P], I),
    "bgtq_decode_attn": ([P, I, I, I, I, P, I64, P, I, P, P, I, I, P, P, P, F, P, P, SZ, I, P], I),
}

STATUS = {0: "KVQ_OK", -1: "KVQ_ERR_INVALID_ARG", -2: "KVQ_ERR_UNSUPPORTED", -3: "KVQ_ERR_WORKSPACE",
          -4: "KVQ_ERR_CUDA", -5: "KVQ_ERR_BAD_BLOCK_TABLE"}


class KvqError(RuntimeError):
    def __init__(self, status: int, text: str):
        super().__init__(f"{STATUS.get(status, status)}: {text}")
        self.status = status


def header_functions() -> list[str]:
    """Names of the functions include/kvq.h declares."""
    src = open(HEADER).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return re.findall(r"\b(kvq_\w+|bgtq_\w+)\s*\(", src)


def load():
    """Loads the in-tree library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with bit_kv_cache_13_gb300.build.build()")
        lib = C.CDLL(LIB_PATH)
        for name, (args, res) in _SIGS.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
    return _lib


def _check(status: int):
    if status != 0:
        raise KvqError(status, load().kvq_last_error().decode())


def _stream(stream) -> int:
    if stream is None:
        dev = torch.cuda.current_device()
        # the handle itself, where torch has a name for it: making a Stream object of it costs 2.5 us, as much as a launch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        return raw(dev) if raw is not None else torch.cuda.current_stream(dev).cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dev(x: torch.Tensor | None, dtype, name: str):
    if x is None:
        return None
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if x.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {x.dtype}")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return x.data_ptr()


# ------------------------------------------------------------------- INT2

def kvq_int2_tile_bytes(d: int = 128) -> int:
    return load().kvq_int2_tile_bytes(d)


def kvq_append_int2(k, v, slot_mapping, mu_k, R_k, R_v, cache, num_pages: int,
                    dbg_rot_k=None, dbg_rot_v=None, err_count=None, stream=None):
    n_tok, h_kv, d = k.shape
    _check(load().kvq_append_int2(
        _dev(k, torch.bfloat16, "k"), _dev(v, torch.bfloat16, "v"), n_tok, h_kv, d,
        _dev(slot_mapping, torch.int32, "slot_mapping"), _dev(mu_k, torch.float32, "mu_k"),
        _dev(R_k, torch.float32, "R_k"), _dev(R_v, torch.float32, "R_v"),
        _dev(cache, torch.uint8, "cache"), int(num_pages),
        _dev(dbg_rot_k, torch.float32, "dbg_rot_k"), _dev(dbg_rot_v, torch.float32, "dbg_rot_v"),
        _dev(err_count, torch.int32, "err_count"), _stream(stream)))


def kvq_append_int2_clip(k, v, slot_mapping, mu_k, R_k, R_v, clip: float, cache, num_pages: int,
                         dbg_rot_k=None, dbg_rot_v=None, err_count=None, stream=None):
    """kvq_append_int2 with clip ratio c in (0, 1] (c = 1: the plain call)."""
    n_tok, h_kv, d = k.shape
    _check(load().kvq_append_int2_clip(
        _dev(k, torch.bfloat16, "k"), _dev(v, torch.bfloat16, "v"), n_tok, h_kv, d,
        _dev(slot_mapping, torch.int32, "slot_mapping"), _dev(mu_k, torch.float32, "mu_k"),
        _dev(R_k, torch.float32, "R_k"), _dev(R_v, torch.float32, "R_v"), float(clip),
        _dev(cache, torch.uint8, "cache"), int(num_pages),
        _dev(dbg_rot_k, torch.float32, "dbg_rot_k"), _dev(dbg_rot_v, torch.float32, "dbg_rot_v"),
        _dev(err_count, torch.int32, "err_count"), _stream(stream)))


def kvq_dequant_int2(cache, num_pages: int, H_kv: int, slot_mapping, k_rot=None, v_rot=None, stream=None):
    """Dequantised rotated vectors [n, H_kv, d] fp32 of the cached tokens at
    slot_mapping [n]."""
    n = slot_mapping.shape[0]
    _check(load().kvq_dequant_int2(
        _dev(cache, torch.uint8, "cache"), int(num_pages), H_kv, 128, _dev(slot_mapping, torch.int32, "slot_mapping"),
        n, _dev(k_rot, torch.float32, "k_rot"), _dev(v_rot, torch.float32, "v_rot"), _stream(stream)))


def kvq_decode_workspace_bytes(B: int, H_q: int, H_kv: int, max_pages_per_seq: int, num_splits: int = 0) -> int:
    return load().kvq_decode_workspace_bytes(B, H_q, H_kv, max_pages_per_seq, num_splits)


def kvq_decode_auto_splits(B: int, H_q: int, H_kv: int, max_pages_per_seq: int) -> int:
    return load().kvq_decode_auto_splits(B, H_q, H_kv, max_pages_per_seq)


def kvq_decode_attn_int2(q, cache, num_pages: int, block_table, context_lens, R_k, R_v, scale: float,
                         out, workspace, num_splits: int = 0, H_kv: int | None = None, stream=None):
    B, H_q, d = q.shape
    h_kv = R_k.shape[0] if H_kv is None else H_kv
    _check(load().kvq_decode_attn_int2(
        _dev(q, torch.bfloat16, "q"), B, H_q, h_kv, d, _dev(cache, torch.uint8, "cache"), int(num_pages),
        _dev(block_table, torch.int32, "block_table"), block_table.shape[1],
        _dev(context_lens, torch.int32, "context_lens"), _dev(R_k, torch.float32, "R_k"),
        _dev(R_v, torch.float32, "R_v"), float(scale), _dev(out, torch.float32, "out"),
        _dev(workspace, torch.uint8, "workspace"), workspace.numel(), int(num_splits), _stream(stream)))


KVQ_STEP_INPUTS_READY = 1


def kvq_decode_step_int2(q, k_new, v_new, cache, num_pages: int, block_table, context_lens, mu_k, R_k, R_v,
                         scale: float, out, workspace, num_splits: int = 0, flags: int = 0, stream=None):
    """One decode step in one launch: the new token k_new, v_new [B, H_kv, d]
    bf16 is appended at position context_lens[b] - 1 of each sequence, then
    the context_lens[b] tokens are attended.  flags = KVQ_STEP_INPUTS_READY
    declares the rotations, key centre, block table, context lengths and
    cache untouched by the kernel just before (read early)."""
    B, H_q, d = q.shape
    h_kv = k_new.shape[1]
    _check(load().kvq_decode_step_int2(
        _dev(q, torch.bfloat16, "q"), _dev(k_new, torch.bfloat16, "k_new"), _dev(v_new, torch.bfloat16, "v_new"),
        B, H_q, h_kv, d, _dev(cache, torch.uint8, "cache"), int(num_pages),
        _dev(block_table, torch.int32, "block_table"), block_table.shape[1],
        _dev(context_lens, torch.int32, "context_lens"), _dev(mu_k, torch.float32, "mu_k"),
        _dev(R_k, torch.float32, "R_k"), _dev(R_v, torch.float32, "R_v"), float(scale),
        _dev(out, torch.float32, "out"), _dev(workspace, torch.uint8, "workspace"), workspace.numel(),
        int(num_splits), int(flags), _stream(stream)))


def kvq_decode_attn_int2_window(q, cache, num_pages: int, block_table, context_lens, R_k, R_v, mu_k, win_k, win_v,
                                win_lens, scale: float, out, workspace, num_splits: int = 0, H_kv: int | None = None,
                                stream=None):
    """kvq_decode_attn_int2 over the cache plus a BF16 window (win_k, win_v:
    [B, win_max, H_kv, d] bf16; win_lens: [B] int32)."""
    B, H_q, d = q.shape
    h_kv = R_k.shape[0] if H_kv is None else H_kv
    _check(load().kvq_decode_attn_int2_window(
        _dev(q, torch.bfloat16, "q"), B, H_q, h_kv, d, _dev(cache, torch.uint8, "cache"), int(num_pages),
        _dev(block_table, torch.int32, "block_table"), block_table.shape[1],
        _dev(context_lens, torch.int32, "context_lens"), _dev(R_k, torch.float32, "R_k"),
        _dev(R_v, torch.float32, "R_v"), _dev(mu_k, torch.float32, "mu_k"), _dev(win_k, torch.bfloat16, "win_k"),
        _dev(win_v, torch.bfloat16, "win_v"), _dev(win_lens, torch.int32, "win_lens"), win_k.shape[1], float(scale),
        _dev(out, torch.float32, "out"), _dev(workspace, torch.uint8, "workspace"), workspace.numel(),
        int(num_splits), _stream(stream)))


def kvq_decode_attn_int2_noalloc(q, cache, num_pages: int, block_table, context_lens, R_k, R_v, scale: float,
                                 out, num_splits: int = 0, H_kv: int | None = None, stream=None):
    """kvq_decode_attn_int2 with the library's fixed scratch instead of a
    caller workspace (for callers that cannot allocate device memory)."""
    B, H_q, d = q.shape
    h_kv = R_k.shape[0] if H_kv is None else H_kv
    _check(load().kvq_decode_attn_int2_noalloc(
        _dev(q, torch.bfloat16, "q"), B, H_q, h_kv, d, _dev(cache, torch.uint8, "cache"), int(num_pages),
        _dev(block_table, torch.int32, "block_table"), block_table.shape[1],
        _dev(context_lens, torch.int32, "context_lens"), _dev(R_k, torch.float32, "R_k"),
        _dev(R_v, torch.float32, "R_v"), float(scale), _dev(out, torch.float32, "out"), int(num_splits),
        _stream(stream)))


def kvq_debug_drop_next_copy() -> None:
    """Test hook: the next INT2 or INT4 decode launch leaves one bulk copy unissued
    so a bounded wait runs out (the call then reports KVQ_ERR_CUDA)."""
    load().kvq_debug_drop_next_copy()


def kvq_workspace_status(workspace, stream=None) -> int:
    """Returns the status code recorded in a decode workspace (0 = OK) and
    clears it."""
    return load().kvq_workspace_status(_dev(workspace, torch.uint8, "workspace"), _stream(stream))


# ------------------------------------------------------------------- INT4
#
# These calls take a few microseconds on the device for a single token, so each
# tensor is checked in one expression; what fails it is looked at again to say why.

_U8, _I32, _F32, _BF16 = torch.uint8, torch.int32, torch.float32, torch.bfloat16


def _ptr(x, dtype, shape, dev: int, name: str):
    """x's device pointer: a contiguous tensor of this dtype and shape (None: any) on device dev, the current one."""
    if x is None:
        return None
    if x.dtype is dtype and x.get_device() == dev and (shape is None or x.shape == shape) and x.is_contiguous():
        return x.data_ptr()
    if shape is not None and tuple(x.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(x.shape)}")
    _dev(x, dtype, name)
    raise ValueError(f"tensors must be on the current device cuda:{torch.cuda.current_device()}, "
                     f"{name} is on {x.device}")


def _here(x) -> int:
    """The current device, whose stream the call is enqueued on (-1 for a tensor that is not on a GPU)."""
    return torch.cuda.current_device() if x.is_cuda else -1


def _call(fn, dev: int, args, stream):
    if dev < 0:
        raise ValueError("the call's tensors must be CUDA tensors")
    _check(fn(*args, _stream(stream)))


def _pool(cache, num_pages: int, h_kv: int, name: str):
    """A cache pool of at least num_pages pages of h_kv INT4 tiles."""
    if cache.numel() < num_pages * h_kv * 2560:
        raise ValueError(f"{name} holds {cache.numel()} bytes, below {num_pages} pages x {h_kv} heads x 2560")


def _rows(x, lead, name: str, last: str):
    """The last extent of x, whose others are lead."""
    if x.shape[:-1] != lead or x.dim() != len(lead) + 1:
        raise ValueError(f"{name} must have shape ({', '.join(map(str, lead))}, {last}), got {tuple(x.shape)}")
    return x.shape[-1]


def _count(x, dev: int):
    if x is not None and x.numel() == 0:
        raise ValueError("err_count must have an element")
    return _ptr(x, _I32, None, dev, "err_count")


def kvq_int4_tile_bytes(d: int = 128) -> int:
    return load().kvq_int4_tile_bytes(d)


def kvq_append_int4(k, v, slot_mapping, mu_k, R_k, R_v, cache, num_pages: int, clip: float = 1.0, err_count=None,
                    stream=None):
    """Quantise-on-append of k, v [n, H_kv, d] bf16 into the INT4 cache."""
    n_tok, h_kv, d = shape = k.shape
    dev = _here(k)
    _pool(cache, num_pages, h_kv, "cache")
    _call(load().kvq_append_int4, dev, (
        _ptr(k, _BF16, shape, dev, "k"), _ptr(v, _BF16, shape, dev, "v"), n_tok, h_kv, d,
        _ptr(slot_mapping, _I32, (n_tok,), dev, "slot_mapping"), _ptr(mu_k, _F32, (h_kv, d), dev, "mu_k"),
        _ptr(R_k, _F32, (h_kv, d, d), dev, "R_k"), _ptr(R_v, _F32, (h_kv, d, d), dev, "R_v"), float(clip),
        _ptr(cache, _U8, None, dev, "cache"), int(num_pages), _count(err_count, dev)), stream)


def kvq_dequant_int4(cache, num_pages: int, H_kv: int, slot_mapping, k_rot=None, v_rot=None, stream=None):
    """Dequantised rotated vectors [n, H_kv, d] bf16 of the cached tokens at slot_mapping [n]."""
    n, dev = slot_mapping.shape[0], _here(cache)
    _pool(cache, num_pages, H_kv, "cache")
    _call(load().kvq_dequant_int4, dev, (
        _ptr(cache, _U8, None, dev, "cache"), int(num_pages), H_kv, 128,
        _ptr(slot_mapping, _I32, (n,), dev, "slot_mapping"), n,
        _ptr(k_rot, _BF16, (n, H_kv, 128), dev, "k_rot"), _ptr(v_rot, _BF16, (n, H_kv, 128), dev, "v_rot")), stream)


def kvq_int4_workspace_bytes(B: int, H_q: int, H_kv: int, max_pages_per_seq: int, num_splits: int = 0,
                             weights: bool = False) -> int:
    return load().kvq_int4_workspace_bytes(B, H_q, H_kv, max_pages_per_seq, num_splits, int(weights))


def _decode_int4_args(dev, q, cache, num_pages, block_table, context_lens, R_k, R_v, scale, out):
    B, H_q, d = shape = q.shape
    h_kv = R_k.shape[0]
    pages = _rows(block_table, (B,), "block_table", "max_pages")
    _pool(cache, num_pages, h_kv, "cache")
    return (_ptr(q, _BF16, None, dev, "q"), B, H_q, h_kv, d, _ptr(cache, _U8, None, dev, "cache"), int(num_pages),
            _ptr(block_table, _I32, None, dev, "block_table"), pages,
            _ptr(context_lens, _I32, (B,), dev, "context_lens"), _ptr(R_k, _F32, (h_kv, d, d), dev, "R_k"),
            _ptr(R_v, _F32, (h_kv, d, d), dev, "R_v"), float(scale), _ptr(out, _BF16, shape, dev, "out"))


def kvq_decode_attn_int4(q, cache, num_pages: int, block_table, context_lens, R_k, R_v, scale: float, out, workspace,
                         num_splits: int = 0, stream=None):
    """Decode attention of q [B, H_q, d] bf16 over the INT4 cache into out [B, H_q, d] bf16."""
    dev = _here(q)
    _call(load().kvq_decode_attn_int4, dev, (
        *_decode_int4_args(dev, q, cache, num_pages, block_table, context_lens, R_k, R_v, scale, out),
        _ptr(workspace, _U8, None, dev, "workspace"), workspace.numel(), int(num_splits)), stream)


def kvq_decode_attn_int4_weights(q, cache, num_pages: int, block_table, context_lens, R_k, R_v, scale: float, out,
                                 weights, decay: float, workspace, num_splits: int = 0, stream=None):
    """kvq_decode_attn_int4 that also adds each token's attention weight, summed over the query heads of its KV head,
    to weights [B, H_kv, >= 16 max_pages] fp32 (scaled by decay first)."""
    dev = _here(q)
    tokens = _rows(weights, (q.shape[0], R_k.shape[0]), "weights", "tokens")
    _call(load().kvq_decode_attn_int4_weights, dev, (
        *_decode_int4_args(dev, q, cache, num_pages, block_table, context_lens, R_k, R_v, scale, out),
        _ptr(weights, _F32, None, dev, "weights"), tokens, float(decay), _ptr(workspace, _U8, None, dev, "workspace"),
        workspace.numel(), int(num_splits)), stream)


def kvq_evict_select(weights, context_lens, budget: int, sinks: int, recent: int, keep, new_lens, stream=None):
    """Chooses the tokens each (sequence, KV head) keeps by weights [B, H_kv, max_tokens] fp32: their indices, ascending,
    into keep [B, H_kv, budget] int32 (-1 past them) and min(length, budget) into new_lens [B] int32."""
    B, h_kv, max_tokens = weights.shape
    dev = _here(weights)
    _call(load().kvq_evict_select, dev, (
        _ptr(weights, _F32, None, dev, "weights"), max_tokens, B, h_kv, max_tokens,
        _ptr(context_lens, _I32, (B,), dev, "context_lens"), int(budget), int(sinks), int(recent),
        _ptr(keep, _I32, (B, h_kv, budget), dev, "keep"), _ptr(new_lens, _I32, (B,), dev, "new_lens")), stream)


def kvq_evict_gather_int4(cache, num_pages: int, block_table, keep, new_lens, dst_cache, dst_num_pages: int,
                          dst_block_table, weights=None, weights_out=None, err_count=None, stream=None):
    """Moves the tokens of keep [B, H_kv, budget] from the pages of block_table into those of dst_block_table (and their
    weights [B, H_kv, tokens] into weights_out, whose rows are zero past them)."""
    B, h_kv, budget = keep.shape
    dev = _here(cache)
    src_pages = _rows(block_table, (B,), "block_table", "pages")
    dst_pages = _rows(dst_block_table, (B,), "dst_block_table", "pages")
    if (weights is None) != (weights_out is None):
        raise ValueError("weights and weights_out go together")
    w_row, o_row = (0 if x is None else _rows(x, (B, h_kv), name, "tokens")
                    for x, name in ((weights, "weights"), (weights_out, "weights_out")))
    _pool(cache, num_pages, h_kv, "cache")
    _pool(dst_cache, dst_num_pages, h_kv, "dst_cache")
    _call(load().kvq_evict_gather_int4, dev, (
        _ptr(cache, _U8, None, dev, "cache"), int(num_pages),
        _ptr(block_table, _I32, None, dev, "block_table"), src_pages,
        _ptr(keep, _I32, None, dev, "keep"), budget, _ptr(new_lens, _I32, (B,), dev, "new_lens"), B, h_kv, 128,
        _ptr(dst_cache, _U8, None, dev, "dst_cache"), int(dst_num_pages),
        _ptr(dst_block_table, _I32, None, dev, "dst_block_table"), dst_pages, _ptr(weights, _F32, None, dev, "weights"),
        w_row, _ptr(weights_out, _F32, None, dev, "weights_out"), o_row,
        _count(err_count, dev)), stream)


# -------------------------------------------------------------- Block-GTQ

def bgtq_energy_scores(q, k, H_kv: int, scores, paired=None, stream=None):
    """Calibration block energy scores (and the paired AM-GM estimate) of
    q [T, H_q, d] and k [T, H_kv, d] bf16 into fp64 [H_kv, d/2] tensors."""
    T, H_q, d = q.shape
    _check(load().bgtq_energy_scores(
        _dev(q, torch.bfloat16, "q"), _dev(k, torch.bfloat16, "k"), T, H_q, H_kv, d,
        _dev(scores, torch.float64, "scores"), None if paired is None else _dev(paired, torch.float64, "paired"),
        _stream(stream)))

def bgtq_lloyd_max_codebook(b: int):
    import numpy as np
    out = np.zeros(1 << b, dtype=np.float64)
    _check(load().bgtq_lloyd_max_codebook(b, out.ctypes.data))
    return out


def bgtq_allocate(scores, b_min: int, b_max: int, total_bits: int):
    import numpy as np
    s = np.ascontiguousarray(scores, dtype=np.float64)
    w = np.zeros(s.shape[0], dtype=np.int8)
    _check(load().bgtq_allocate(s.ctypes.data, s.shape[0], b_min, b_max, int(total_bits), w.ctypes.data))
    return w


def bgtq_tile_bytes(total_bits: int, v_bits: int) -> int:
    return load().bgtq_tile_bytes(total_bits, v_bits)


def bgtq_append(k, v, slot_mapping, widths, total_bits: int, v_bits: int, pi_table, pi_offsets, codebooks,
                cache, num_pages: int, err_count=None, stream=None):
    n_tok, h_kv, d = k.shape
    _check(load().bgtq_append(
        _dev(k, torch.bfloat16, "k"), _dev(v, torch.bfloat16, "v"), n_tok, h_kv, d,
        _dev(slot_mapping, torch.int32, "slot_mapping"), _dev(widths, torch.int8, "widths"), int(total_bits),
        int(v_bits), _dev(pi_table, torch.float32, "pi_table"), _dev(pi_offsets, torch.int64, "pi_offsets"),
        _dev(codebooks, torch.float64, "codebooks"), _dev(cache, torch.uint8, "cache"), int(num_pages),
        _dev(err_count, torch.int32, "err_count"), _stream(stream)))


def bgtq_decode_attn(q, cache, num_pages: int, block_table, context_lens, widths, total_bits: int, v_bits: int,
                     pi_table, pi_offsets, codebooks, scale: float, out, workspace, num_splits: int = 0,
                     stream=None):
    B, H_q, d = q.shape
    h_kv = widths.shape[0]
    _check(load().bgtq_decode_attn(
        _dev(q, torch.bfloat16, "q"), B, H_q, h_kv, d, _dev(cache, torch.uint8, "cache"), int(num_pages),
        _dev(block_table, torch.int32, "block_table"), block_table.shape[1],
        _dev(context_lens, torch.int32, "context_lens"), _dev(widths, torch.int8, "widths"), int(total_bits),
        int(v_bits), _dev(pi_table, torch.float32, "pi_table"), _dev(pi_offsets, torch.int64, "pi_offsets"),
        _dev(codebooks, torch.float64, "codebooks"), float(scale), _dev(out, torch.float32, "out"),
        _dev(workspace, torch.uint8, "workspace"), workspace.numel(), int(num_splits), _stream(stream)))
