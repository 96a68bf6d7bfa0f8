"""Rotated INT4 KV cache, its decode attention with token weights, and eviction
by those weights (fp64 oracle).

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).

The cache is the INT2 one (rotation, centring, groups of 32 rotated channels,
fp16 scale and min) with 16 levels per group.  A code is decided from the
real-number rotated vector, here an fp64 product, so it does not depend on the
order of a sum.

Tile of one (page, KV head), 2560 bytes:
  [   0, 1024) K codes 16 slots x 64 B   [1024, 1280) K meta 16 x (4 scales, 4 mins)
  [1280, 2304) V codes 8 slot pairs x 128 B
  [2304, 2432) V scales 8 pairs x 4 groups x 2 slots   [2432, 2560) V mins
"""
from __future__ import annotations

import numpy as np

from .fp import f16_rn_sat

PAGE, D, GROUP, N_GROUPS, TILE_BYTES, TOP = 16, 128, 32, 4, 2560, 15


# ------------------------------------------------------------------ quantiser

def quant_params(z, clip: float = 1.0):
    """fp16 (scale, min) per group along the last axis (length 32), fp64 input."""
    z = np.asarray(z, np.float64)
    c = float(np.float32(clip))
    fine = np.isfinite(z).all(axis=-1)   # a group with a value that is not finite is NaN
    lo, hi = np.where(fine, c * z.min(axis=-1), np.nan), np.where(fine, c * z.max(axis=-1), np.nan)
    f32 = lambda x: np.clip(x, -np.finfo(np.float32).max, np.finfo(np.float32).max).astype(np.float32)  # noqa: E731
    return f16_rn_sat(f32((hi - lo) / TOP)), f16_rn_sat(f32(lo))   # (past fp32's range: saturated too)


def quant_codes(z, scale_h, min_h):
    """The number of thresholds min + (c + 1/2) scale, c = 0..14, strictly below z."""
    z = np.asarray(z, np.float64)
    sc = np.asarray(scale_h, np.float16).astype(np.float64)[..., None]
    mn = np.asarray(min_h, np.float16).astype(np.float64)[..., None]
    code = np.zeros(z.shape, np.uint8)
    for c in range(TOP):
        code += (mn + (c + 0.5) * sc < z).astype(np.uint8)
    return np.where(sc > 0.0, code, 0).astype(np.uint8)


def quantize(z, clip: float = 1.0):
    z = np.asarray(z, np.float64)
    g = z.reshape(z.shape[:-1] + (N_GROUPS, GROUP))
    sc, mn = quant_params(g, clip)
    return quant_codes(g, sc, mn).reshape(z.shape), sc, mn


def dequantize(codes, scale_h, min_h):
    c = np.asarray(codes, np.float64).reshape(np.shape(codes)[:-1] + (N_GROUPS, GROUP))
    sc, mn = (np.asarray(x, np.float16).astype(np.float64)[..., None] for x in (scale_h, min_h))
    return (mn + c * sc).reshape(np.shape(codes))


# ------------------------------------------------------------------ layout

def code_address(side: int, s: int, ch: int):
    """(byte, low bit) in the tile of slot s's code of channel ch, side 0 keys, 1 values."""
    g, c = divmod(ch, 32)
    if side == 0:
        t, i = divmod(c, 8)
        return 64 * s + 16 * t + 4 * g + i // 2, 4 * (i % 2)
    r, i = divmod(c, 4)
    return 1280 + 128 * (s // 2) + 16 * r + 4 * g + 2 * (s % 2) + i // 2, 4 * (i % 2)


def meta_address(side: int, s: int, g: int):
    """(byte of the fp16 scale, byte of the fp16 min) of slot s, group g."""
    if side == 0:
        return 1024 + 16 * s + 2 * g, 1024 + 16 * s + 8 + 2 * g
    at = 2304 + 16 * (s // 2) + 4 * g + 2 * (s % 2)
    return at, at + 128


CODE_AT = np.array([[[code_address(side, s, c) for c in range(D)] for s in range(PAGE)] for side in (0, 1)])
META_AT = np.array([[[meta_address(side, s, g) for g in range(N_GROUPS)] for s in range(PAGE)] for side in (0, 1)])


def new_cache(num_pages: int, h_kv: int) -> np.ndarray:
    return np.zeros((num_pages, h_kv, TILE_BYTES), np.uint8)


def write_tokens(tiles, side: int, s: int, codes, sc, mn):
    """Writes slot s of tiles [..., 2560] in place: codes [..., 128], fp16 scale and min [..., 4]."""
    byte, low = CODE_AT[side, s, :, 0], CODE_AT[side, s, :, 1]
    for nib in (0, 4):
        at = low == nib
        tiles[..., byte[at]] = (tiles[..., byte[at]] & (0xF0 if nib == 0 else 0x0F)) | (np.asarray(codes)[..., at].astype(np.uint8) << nib)
    for col, h in ((0, sc), (1, mn)):
        raw = np.ascontiguousarray(h, np.float16).view(np.uint8).reshape(np.shape(h) + (2,))
        for e in range(2):
            tiles[..., META_AT[side, s, :, col] + e] = raw[..., e]


def read_token(tile, side: int, s: int):
    """codes [128], scale [4], min [4] of one slot of a tile [2560]."""
    codes = (tile[CODE_AT[side, s, :, 0]] >> CODE_AT[side, s, :, 1].astype(np.uint8)) & 15
    meta = [np.stack([tile[META_AT[side, s, :, c]], tile[META_AT[side, s, :, c] + 1]], -1).reshape(-1).view(np.float16) for c in (0, 1)]
    return codes.astype(np.uint8), meta[0], meta[1]


def meta(tiles, side: int):
    """fp16 scales and mins [..., 16, 4] of tiles [..., 2560]."""
    return [np.ascontiguousarray(np.stack([tiles[..., META_AT[side, :, :, c]], tiles[..., META_AT[side, :, :, c] + 1]], -1)).view(np.float16)[..., 0]
            for c in (0, 1)]


def values(tiles, side: int):
    """Dequantised fp64 [..., 16, 128] of tiles [..., 2560]."""
    tiles = np.asarray(tiles, np.uint8)
    codes = (tiles[..., CODE_AT[side, :, :, 0]] >> CODE_AT[side, :, :, 1].astype(np.uint8)) & 15
    return dequantize(codes, *meta(tiles, side))


# ------------------------------------------------------------------ append, decode

def append(cache, k, v, slot_mapping, mu32, rk32, rv32, clip: float = 1.0):
    """Quantise-on-append (in place) of k, v [n, H_kv, d] at slot_mapping [n]; negative or outside slots are skipped."""
    k, v = np.asarray(k, np.float64), np.asarray(v, np.float64)
    for h in range(k.shape[1]):
        z = (k[:, h] - np.asarray(mu32[h], np.float64)) @ np.asarray(rk32[h], np.float32).astype(np.float64)
        w = v[:, h] @ np.asarray(rv32[h], np.float32).astype(np.float64)
        for side, x in ((0, z), (1, w)):
            codes, sc, mn = quantize(x, clip)
            for i, slot in enumerate(np.asarray(slot_mapping, np.int64)):
                if 0 <= slot < cache.shape[0] * PAGE:
                    write_tokens(cache[slot // PAGE, h], side, int(slot % PAGE), codes[i], sc[i], mn[i])


def decode(q, cache, block_table, ctx_lens, rk32, rv32, scale, weights=None, decay: float = 1.0):
    """Decode attention: o_j = softmax(<q_j, K^ R_k^T> scale) V^ R_v^T over the first ctx_lens[b] tokens; pages outside the
    pool are dropped.  Returns out [B, H_q, d], and (out, weights) with weights [B, H_kv, T] given:
    weights * decay + the sum over the head's queries of each attended token's softmax weight."""
    q = np.asarray(q, np.float64)
    B, h_q, d = q.shape
    h_kv = cache.shape[1]
    g = h_q // h_kv
    out = np.zeros((B, h_q, d))
    acc = None if weights is None else np.array(weights, np.float64)
    for b in range(B):
        n = int(ctx_lens[b])
        if n <= 0:
            continue
        pages = np.asarray(block_table[b][: (n + PAGE - 1) // PAGE], np.int64)
        ok = (pages >= 0) & (pages < cache.shape[0])
        token_ok = np.repeat(ok, PAGE)[:n]
        for h in range(h_kv):
            tiles = cache[np.where(ok, pages, 0), h]
            kt = values(tiles, 0).reshape(-1, d)[:n] @ np.asarray(rk32[h], np.float32).astype(np.float64).T
            vt = values(tiles, 1).reshape(-1, d)[:n] @ np.asarray(rv32[h], np.float32).astype(np.float64).T
            if acc is not None:
                acc[b, h, :n] *= float(np.float32(decay))
            if not token_ok.any():
                continue
            for j in range(h * g, (h + 1) * g):
                a = kt[token_ok] @ q[b, j] * float(np.float32(scale))
                p = np.exp(a - a.max())
                p /= p.sum()
                out[b, j] = p @ vt[token_ok]
                if acc is not None:
                    acc[b, h, np.nonzero(token_ok)[0]] += p
    return out if acc is None else (out, acc)


# ------------------------------------------------------------------ eviction

def select(weights, ctx_lens, budget: int, sinks: int, recent: int):
    """keep [B, H_kv, budget] (-1 past the kept ones) and new_lens [B]."""
    weights = np.asarray(weights, np.float32)
    B, h_kv, T = weights.shape
    keep = np.full((B, h_kv, budget), -1, np.int32)
    new = np.zeros(B, np.int32)
    for b in range(B):
        n = max(0, min(int(ctx_lens[b]), T))
        new[b] = min(n, budget)
        for h in range(h_kv):
            if n <= budget:
                keep[b, h, :n] = np.arange(n)
                continue
            w = [float(x) if x == x else -np.inf for x in weights[b, h]]
            best = sorted(range(sinks, n - recent), key=lambda s: (-w[s], s))[: budget - sinks - recent]
            keep[b, h] = sorted(list(range(sinks)) + best + list(range(n - recent, n)))
    return keep, new


def gather(cache, block_table, keep, new_lens, dst, dst_block_table, weights=None):
    """Moves kept tokens into dst (in place), token by token; returns the moved weights or None."""
    B, h_kv, _ = keep.shape
    wo = None if weights is None else np.zeros((B, h_kv, dst_block_table.shape[1] * PAGE), np.float32)
    for b in range(B):
        for h in range(h_kv):
            for i in range(int(new_lens[b])):
                s = int(keep[b, h, i])
                src = cache[block_table[b][s // PAGE], h]
                to = dst[dst_block_table[b][i // PAGE], h]
                for side in (0, 1):
                    write_tokens(to, side, i % PAGE, *read_token(src, side, s % PAGE))
                if wo is not None:
                    wo[b, h, i] = weights[b, h, s]
    return wo


# ------------------------------------------------------------------ norms and rotation, more than one new token

def norm_rope(x, positions, table, weight=None, eps: float = 1e-6, interleaved: bool = False):
    """Heads x [n, H, 128] normed (with a weight [128]) and their first channels rotated by positions through table
    [max_pos, rot] (rot/2 cosines, then sines); zeros for a position outside the table.  Not rounded."""
    y = np.array(x, np.float64)
    if weight is not None:
        y = y * np.asarray(weight, np.float64) / np.sqrt((y * y).mean(-1, keepdims=True) + eps)
    table = np.asarray(table, np.float32).astype(np.float64)
    half = table.shape[1] // 2
    pos = np.asarray(positions, np.int64)
    ok = (pos >= 0) & (pos < table.shape[0])
    cos, sin = np.split(table[np.where(ok, pos, 0)][:, None], 2, -1)
    j = np.arange(half)
    first, second = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
    a, b = y[..., first], y[..., second]
    y[..., first], y[..., second] = a * cos - b * sin, b * cos + a * sin
    return np.where(ok[:, None, None], y, 0.0)


def to_bf16(y):
    """fp64 to the nearest bf16 value, ties to even, in one rounding (normal range)."""
    y = np.asarray(y, np.float64)
    ulp = np.ldexp(1.0, np.frexp(y)[1] - 8)
    return np.round(y / ulp) * ulp


def chunk(q, q_start, cache, block_table, ctx_lens, rk32, rv32, scale, window: int = 0, sinks: int = 0):
    """Attention of each sequence's last tokens: row q_start[b] + i at position ctx - n_b + i sees cached tokens t <= it
    (window > 0: t > it - window or t < sinks); pages outside the pool are dropped.  Returns out [n, H_q, d] and the bound
    [n, H_q] on the 2-norm of what rounding to fp16 does to it: of the rotation's entries, the rotated queries and the cached
    keys once each (each at most 2^-11 of a product's term, in standard deviation 2^-11 / sqrt(3); the three are independent
    and taken at six standard deviations), of the weights, the values, the sums and the output rotation's entries at 2^-11."""
    q = np.asarray(q, np.float64)
    h_q, d = q.shape[1:]
    h_kv = cache.shape[1]
    g = h_q // h_kv
    out, bound = np.zeros(q.shape), np.zeros(q.shape[:2])
    sc = float(np.float32(scale))
    for b, ctx in enumerate(np.clip(np.asarray(ctx_lens, np.int64), 0, PAGE * block_table.shape[1])):
        n = int(q_start[b + 1] - q_start[b])
        if n <= 0 or ctx == 0:
            continue
        pages = np.asarray(block_table[b][: -(-int(ctx) // PAGE)], np.int64)
        ok = (pages >= 0) & (pages < cache.shape[0])
        t, p = np.arange(ctx), ctx - n + np.arange(n)[:, None]
        see = (t <= p) & np.repeat(ok, PAGE)[:ctx]
        if window:
            see &= (t > p - window) | (t < sinks)
        rows = slice(int(q_start[b]), int(q_start[b]) + n)
        any_row = see.any(1)
        for h in range(h_kv):
            tiles = cache[np.where(ok, pages, 0), h]
            k, v = (values(tiles, side).reshape(-1, d)[:ctx] for side in (0, 1))
            used = see.any(0)
            k, v = np.where(used[:, None], k, 0.0), np.where(used[:, None], v, 0.0)
            size = np.linalg.norm(v, axis=1)
            rk, rv = (np.asarray(r[h], np.float32).astype(np.float64) for r in (rk32, rv32))
            for j in range(h * g, (h + 1) * g):
                qr = q[rows, j] @ rk
                a = np.where(see, qr @ k.T * sc, -np.inf)
                top = np.where(any_row, a.max(1, initial=-np.inf), 0.0)[:, None]
                w = np.where(see, np.exp(a - top), 0.0)
                w /= np.where(any_row, w.sum(1), 1.0)[:, None]
                o = w @ v
                out[rows, j] = o @ rv.T
                e = 6 * 2.0 ** -11 * abs(sc) * np.sqrt((qr * qr) @ (k * k).T) + 2.0 ** -11
                e = np.where(see, e, 0.0)
                bound[rows, j] = (w * e) @ size + 2.0 ** -11 * (w @ size) + 2.0 ** -10 * np.linalg.norm(o, axis=1) + (w * e).sum(1) * np.linalg.norm(o, axis=1) + 1e-6 * size.max(initial=0.0)
    return out, bound


def chunk_spread(q, q_start, cache, block_table, ctx_lens, rk32, rv32, scale, window: int = 0, sinks: int = 0):
    """What chunk() returns and, instead of its bound, the variance [n, H_q] of the 2-norm of the error that fp16 operands
    leave: each is rounded by at most 2^-11 of itself, in standard deviation u = 2^-11 / sqrt(3) at the most, all of them
    independent.  With weights w_t, logits a_t = sum_j q'_j k_tj scale, q'_j = sum_i q_i R_ij:
      * q'_j and the R_ij move all tokens' logits together: by g_j k_tj with var g_j = u^2 (q'_j^2 + sum_i q_i^2 R_ij^2), and
        an error e_t of logit t moves the output by w_t e_t (v_t - o): sum_j var g_j scale^2 |sum_t w_t k_tj (v_t - o)|^2;
      * a key k_tj by itself: u^2 scale^2 sum_t w_t^2 |v_t - o|^2 sum_j (q'_j k_tj)^2;
      * weights and values: 2 u^2 sum_t w_t^2 |v_t|^2;  the sums and R_v, which is orthogonal: 2 u^2 |o|^2."""
    u2 = 2.0 ** -22 / 3
    out, _ = chunk(q, q_start, cache, block_table, ctx_lens, rk32, rv32, scale, window, sinks)
    q = np.asarray(q, np.float64)
    h_q, d = q.shape[1:]
    h_kv = cache.shape[1]
    g = h_q // h_kv
    var = np.zeros(q.shape[:2])
    sc = float(np.float32(scale))
    for b, ctx in enumerate(np.clip(np.asarray(ctx_lens, np.int64), 0, PAGE * block_table.shape[1])):
        n = int(q_start[b + 1] - q_start[b])
        if n <= 0 or ctx == 0:
            continue
        pages = np.asarray(block_table[b][: -(-int(ctx) // PAGE)], np.int64)
        ok = (pages >= 0) & (pages < cache.shape[0])
        t, p = np.arange(ctx), ctx - n + np.arange(n)[:, None]
        see = (t <= p) & np.repeat(ok, PAGE)[:ctx]
        if window:
            see &= (t > p - window) | (t < sinks)
        rows, used = slice(int(q_start[b]), int(q_start[b]) + n), see.any(0)
        for h in range(h_kv):
            tiles = cache[np.where(ok, pages, 0), h]
            k, v = (np.where(used[:, None], values(tiles, side).reshape(-1, d)[:ctx], 0.0) for side in (0, 1))
            rk = np.asarray(rk32[h], np.float32).astype(np.float64)
            rv = np.asarray(rv32[h], np.float32).astype(np.float64)
            for j in range(h * g, (h + 1) * g):
                qr = q[rows, j] @ rk
                a = np.where(see, qr @ k.T * sc, -np.inf)
                w = np.where(see, np.exp(a - np.where(see.any(1), a.max(1, initial=-np.inf), 0.0)[:, None]), 0.0)
                w /= np.where(see.any(1), w.sum(1), 1.0)[:, None]
                o = out[rows, j] @ rv
                away = (v * v).sum(1) - 2 * o @ v.T + (o * o).sum(1)[:, None]      # |v_t - o|^2
                together = (w[:, None] * k.T) @ v - (w @ k)[:, :, None] * o[:, None]
                var[rows, j] = u2 * (sc * sc * (((qr * qr) + (q[rows, j] ** 2) @ (rk * rk)) * (together ** 2).sum(-1)).sum(1)
                                     + sc * sc * (w * w * np.maximum(away, 0.0) * ((qr * qr) @ (k * k).T)).sum(1)
                                     + 2 * (w * w) @ (v * v).sum(1) + 2 * (o * o).sum(1))
    return out, var
