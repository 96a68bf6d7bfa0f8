"""Operators around the INT4 cache as they are timed: appending with the heads' norms and the position rotation on the
way, attention of a chunk of new tokens over the paged cache, and single-token attention in a sliding window with sinks.

A case is one call of one operator (`op`), or of the two that a user makes together:

  rope     norm and rotate the new tokens' queries and keys, quantise keys and values into the paged cache, then read
           the tokens back (what later attention sees)
  chunk    attention of each sequence's last tokens, causal among themselves, over the packed cache; window > 0: over
           the last `window` tokens before each and the first `sinks`
  sliding  single-token attention over the last `window` tokens and the first `sinks`

`run` with `own` false is their plain form; with `own` true it calls the library.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

D, PAGE, GROUP, NG, TILE = 128, 16, 32, 4, 2560
SCALE = 1.0 / math.sqrt(D)
EPS = 1e-6
PADDING = 3  # rows behind the last sequence of a ragged chunk batch


# ------------------------------------------------------------------ cases

def _rope(T, h_q, h_kv, norm=True, interleaved=False, rot=D, start=0, skip=False):
    return dict(op="rope", T=T, h_q=h_q, h_kv=h_kv, norm=norm, interleaved=interleaved, rot=rot, start=start, skip=skip)


def _chunk(B, n, T, h_q, h_kv, window=0, sinks=0, ragged=False):
    return dict(op="chunk", B=B, n=n, T=T, h_q=h_q, h_kv=h_kv, window=window, sinks=sinks, ragged=ragged)


def _sliding(B, T, h_q, h_kv, window, sinks, ragged=False):
    return dict(op="sliding", B=B, n=1, T=T, h_q=h_q, h_kv=h_kv, window=window, sinks=sinks, ragged=ragged)


def listed():
    return [
        # one new token of one sequence far into its context: the projections' output of a decode step
        dict(_rope(1, 32, 8, start=131071), name="rope_1"),
        # a ragged chunk with padded rows (slot -1), without norms, half of each head rotated in neighbouring pairs
        dict(_rope(1531, 32, 8, norm=False, interleaved=True, rot=64, skip=True), name="rope_1531_padded"),
        # the prefill of an 8K prompt of the 32 q / 8 KV head layer
        dict(_rope(8192, 32, 8), name="rope_8k"),
        # a short turn on a small model: launch latency
        dict(_chunk(1, 17, 311, 4, 1), name="chunk_b1_17_of_311"),
        # verifying four drafted tokens (and the one before) of eight users at 32K
        dict(_chunk(8, 5, 32768, 32, 8), name="chunk_b8_5_of_32k"),
        # prompts in pieces beside single tokens and nothing, 64 q / 8 KV heads
        dict(_chunk(6, 509, 8191, 64, 8, ragged=True), name="chunk_b6_ragged_8k_gqa8"),
        # a whole prompt at once
        dict(_chunk(1, 4096, 4096, 32, 8), name="chunk_b1_prompt_4k"),
        # a piece of a long prompt
        dict(_chunk(1, 2048, 32768, 32, 8), name="chunk_b1_2k_of_32k"),
        # the same of a longer one, in a window with sinks
        dict(_chunk(1, 2048, 65536, 32, 8, window=4096, sinks=4), name="chunk_b1_2k_of_64k_window_4k"),
        # the last piece of a long document
        dict(_chunk(1, 4096, 65536, 32, 8), name="chunk_b1_4k_of_64k"),
        # one user at 128K whose layer looks back 4096 tokens
        dict(_sliding(1, 131072, 32, 8, window=4096, sinks=4), name="sliding_b1_128k_window_4k"),
        # a full batch of the 64 q / 8 KV head layer, lengths from nothing to 8K, a short window and many sinks
        dict(_sliding(32, 8191, 64, 8, window=1000, sinks=70, ragged=True), name="sliding_b32_8k_gqa8_ragged"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "chunk", "chunk", "sliding"])
    h_kv = rng.choice([1, 2, 4, 8])
    h_q = h_kv * rng.randint(1, 8)
    if op == "rope":
        T = _log(rng, 1, 8192)
        return _rope(T, h_q, h_kv, rng.random() < 0.6, rng.random() < 0.4, rng.choice([D, D, 64, 32, 96]),
                     _log(rng, 1, 131072), rng.random() < 0.5)
    B = _log(rng, 1, 32)
    T = _log(rng, 1, 131072 // B)
    window = rng.choice([0, _log(rng, 1, 8192), _log(rng, 64, 8192)]) if op == "chunk" else _log(rng, 1, 8192)
    sinks = rng.choice([0, 4, rng.randint(1, 130)]) if window else 0
    if op == "sliding":
        return _sliding(B, T, h_q, h_kv, window, sinks, rng.random() < 0.5)
    n = _log(rng, 1, max(1, min(T, 4096, (1 << 30) // (B * T * (h_q // h_kv)))))
    return _chunk(B, n, T, h_q, h_kv, window, sinks, rng.random() < 0.5)


def lengths(case):
    """(new tokens, tokens in the cache, those among them) of each sequence.  Of a ragged batch of three or more one is
    empty; a chunk batch also has one with a single new token."""
    B, T, n = case["B"], case["T"], case["n"]
    if not case["ragged"]:
        return [n] * B, [T] * B
    ctx = [max(1, T * (b + 1) // B - (7 * b) % 5) for b in range(B)]
    new = [max(1, n - (n * b) // B - (3 * b) % 4) for b in range(B)]
    if B > 2:
        ctx[1], new[1] = 0, int(case["op"] == "sliding")
        new[2] = 1
    return [min(a, c) if case["op"] == "chunk" else 1 for a, c in zip(new, ctx)], ctx


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rotations(h, g):
    a = torch.randn((h, D, D), generator=g, device="cuda", dtype=torch.float64)
    return torch.linalg.qr(a)[0].float().contiguous()


def _block_table(B, T, g):
    P = max(1, -(-T // PAGE))
    return torch.randperm(B * P, generator=g, device="cuda").to(torch.int32).view(B, P), B * P


def _random_cache(n_pages, h_kv, g):
    """A filled cache: quantised standard normal vectors, a few channels' worth of spread between groups."""
    parts = []
    for _ in range(2):
        x = torch.randn((n_pages, h_kv, PAGE, D), generator=g, device="cuda")
        x *= 0.5 + torch.rand((n_pages, h_kv, PAGE, 1), generator=g, device="cuda")
        codes, sc, mn = _quantise(x)
        parts += [codes, sc, mn]
        del x
    return _tiles(_records(*parts))


def prepare(case, seed):
    g = _gen(seed)
    h_q, h_kv, T = case["h_q"], case["h_kv"], case["T"]
    s = {"case": dict(case)}
    s["R_k"], s["R_v"] = _rotations(h_kv, g), _rotations(h_kv, g)
    if case["op"] == "rope":
        # queries, keys and values as one projection leaves them: rows of all heads; a few large key and value channels
        row = torch.randn((T, h_q + 2 * h_kv, D), generator=g, device="cuda")
        big = torch.where(torch.rand((2 * h_kv, D), generator=g, device="cuda") < 0.03, 12.0, 1.0)
        row[:, h_q:] *= big
        s["qkv"] = row.bfloat16()
        weight = lambda: (1 + 0.3 * torch.randn(D, generator=g, device="cuda")).bfloat16()  # noqa: E731
        s["q_weight"], s["k_weight"] = (weight(), weight()) if case["norm"] else (None, None)
        half = case["rot"] // 2
        angle = torch.arange(case["start"] + T, device="cuda", dtype=torch.float64)[:, None] \
            * 1e6 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
        s["rope"] = torch.cat([angle.cos(), angle.sin()], -1).float()
        s["positions"] = torch.arange(case["start"], case["start"] + T, dtype=torch.int32, device="cuda")
        s["mu"] = 0.5 * torch.randn((h_kv, D), generator=g, device="cuda")
        bt, s["num_pages"] = _block_table(1, T, g)
        t = torch.arange(T, device="cuda")
        slots = bt[0][t // PAGE].long() * PAGE + t % PAGE
        if case["skip"]:
            slots[t % 11 == 5] = -1
        s["slots"] = slots.to(torch.int32)
        s["cache"] = torch.zeros((s["num_pages"], h_kv, TILE), dtype=torch.uint8, device="cuda")
        s["q_out"] = torch.empty((T, h_q, D), dtype=torch.bfloat16, device="cuda")
        s["k_out"], s["k_hat"], s["v_hat"] = (torch.empty((T, h_kv, D), dtype=torch.bfloat16, device="cuda") for _ in range(3))
        return s
    new, ctx = lengths(case)
    s["lens"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    s["bt"], s["num_pages"] = _block_table(case["B"], T, g)
    s["cache"] = _random_cache(s["num_pages"], h_kv, g)
    rows = sum(new) + (PADDING if case["op"] == "chunk" and case["ragged"] else 0)
    s["q_start"] = torch.tensor(np.cumsum([0] + new), dtype=torch.int32, device="cuda")
    # peaked attention: logits of standard deviation about 2.5
    s["q"] = (2.5 * torch.randn((rows, h_q, D), generator=g, device="cuda")).bfloat16()
    s["out"] = torch.zeros_like(s["q"])
    return s


# ------------------------------------------------------------------ the format, plainly

def _quantise(x):
    """codes [..., 128] uint8, fp16 scale and min [..., 4] of rotated vectors [..., 128]."""
    g = x.view(x.shape[:-1] + (NG, GROUP))
    mn, mx = g.amin(-1), g.amax(-1)
    sc = ((mx - mn) / 15).float().clamp(-65504, 65504).half()
    mh = mn.float().clamp(-65504, 65504).half()
    s, m = sc.to(x.dtype).unsqueeze(-1), mh.to(x.dtype).unsqueeze(-1)
    c = torch.where(s > 0, torch.ceil((g - m) / s - 0.5).clamp(0, 15), torch.zeros_like(g))
    return c.to(torch.uint8).view(x.shape), sc, mh


def _values(codes, sc, mn):
    """min + code * scale, fp32 [..., 128]."""
    c = codes.view(codes.shape[:-1] + (NG, GROUP)).float()
    return torch.addcmul(mn.float().unsqueeze(-1), c, sc.float().unsqueeze(-1)).view(codes.shape)


def _records(kc, ks, km, vc, vs, vm):
    """Token records [..., 160] uint8: key codes 64, key scales and mins 16, value codes 64, value scales and mins 16."""
    n = kc.shape[:-1]
    k = kc.view(n + (NG, 4, 8)).transpose(-3, -2).reshape(n + (64, 2))
    v = vc.view(n + (NG, 8, 4)).transpose(-3, -2).reshape(n + (64, 2))
    meta = lambda s, m: torch.cat([s, m], -1).contiguous().view(torch.uint8)  # noqa: E731
    return torch.cat([k[..., 0] | (k[..., 1] << 4), meta(ks, km), v[..., 0] | (v[..., 1] << 4), meta(vs, vm)], -1)


def _unpacked(rec):
    """The inverse of _records: kc, ks, km, vc, vs, vm."""
    n = rec.shape[:-1]
    nib = lambda b: torch.stack([b & 15, b >> 4], -1)  # noqa: E731
    half = lambda b: b.contiguous().view(torch.float16)  # noqa: E731
    kc = nib(rec[..., :64]).view(n + (4, NG, 8)).transpose(-3, -2).reshape(n + (D,))
    vc = nib(rec[..., 80:144]).view(n + (8, NG, 4)).transpose(-3, -2).reshape(n + (D,))
    return (kc, half(rec[..., 64:72]), half(rec[..., 72:80]), vc, half(rec[..., 144:152]), half(rec[..., 152:160]))


def _tiles(rec):
    """Page tiles [..., 2560] of token records [..., 16, 160]: the values' codes, scales and mins of two slots interleaved."""
    n = rec.shape[:-2]
    pair = lambda b, w: b.reshape(n + (8, 2, w, 2)).transpose(-3, -2).reshape(n + (-1,))  # noqa: E731
    return torch.cat([rec[..., :64].reshape(n + (-1,)), rec[..., 64:80].reshape(n + (-1,)), pair(rec[..., 80:144], 32),
                      pair(rec[..., 144:152], 4), pair(rec[..., 152:160], 4)], -1)


def _tokens(tiles):
    """Token records [..., 16, 160] of page tiles."""
    n = tiles.shape[:-1]
    pair = lambda b, w: b.reshape(n + (8, w, 2, 2)).transpose(-3, -2).reshape(n + (PAGE, 2 * w))  # noqa: E731
    return torch.cat([tiles[..., :1024].reshape(n + (PAGE, 64)), tiles[..., 1024:1280].reshape(n + (PAGE, 16)),
                      pair(tiles[..., 1280:2304], 32), pair(tiles[..., 2304:2432], 4), pair(tiles[..., 2432:2560], 4)], -1)


# ------------------------------------------------------------------ plain forms

def _to_bf16(y):
    """float64 to the nearest bfloat16, ties to even, in one rounding."""
    ulp = torch.ldexp(torch.ones_like(y), torch.frexp(y)[1] - 8)
    return (torch.round(y / ulp) * ulp).bfloat16()


def _normed_rotated(s, x, weight):
    """x [T, H, 128] normed (where there is a weight) and rotated by its positions: 64 bits, since what is rounded after it
    decides codes."""
    c, x = s["case"], x.double()
    if weight is not None:
        x = x * weight.double() / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    cos, sin = s["rope"][s["positions"].long()].double().unsqueeze(1).chunk(2, -1)
    rot, rest = x[..., :c["rot"]], x[..., c["rot"]:]
    if c["interleaved"]:
        a, b = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = rot.chunk(2, -1)
        rot = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return _to_bf16(torch.cat([rot, rest], -1))


def _plain_rope(s):
    h_q, h_kv = s["case"]["h_q"], s["case"]["h_kv"]
    q, k, v = s["qkv"].split([h_q, h_kv, h_kv], 1)
    q, k = _normed_rotated(s, q, s["q_weight"]), _normed_rotated(s, k, s["k_weight"])
    z = torch.einsum("thi,hij->thj", k.double() - s["mu"].double(), s["R_k"].double())
    w = torch.einsum("thi,hij->thj", v.double(), s["R_v"].double())
    kq, vq = _quantise(z), _quantise(w)
    at = s["slots"].long()
    used = (at >= 0).nonzero()[:, 0]
    tok = _tokens(s["cache"])
    tok[at[used] // PAGE, :, at[used] % PAGE] = _records(*kq, *vq)[used]
    s["cache"].copy_(_tiles(tok))
    kc, ks, km, vc, vs, vm = _unpacked(tok[at.clamp(min=0) // PAGE, :, at.clamp(min=0) % PAGE])
    there = (at >= 0)[:, None, None]
    return {"q": q, "k": k, "k_hat": (_values(kc, ks, km) * there).bfloat16(), "v_hat": (_values(vc, vs, vm) * there).bfloat16()}


def _visible(p, t, ctx, window, sinks):
    """Whether the token at position p sees the cached token t."""
    see = (t <= p) & (t < ctx)
    return see & ((t > p - window) | (t < sinks)) if window else see


def _plain_attention(s):
    """The batch padded to its longest chunk, a KV head at a time (the logits of all would not fit)."""
    c = s["case"]
    B, n, G = c["B"], c["n"], c["h_q"] // c["h_kv"]
    start, ctx = s["q_start"].long(), s["lens"].long()
    i, new = torch.arange(n, device="cuda"), start[1:] - start[:-1]
    there = i < new[:, None]                                                    # [B, n]
    row = (start[:-1, None] + i)[there]
    p = ctx[:, None] - new[:, None] + i                                         # the tokens' positions
    t = torch.arange(s["bt"].shape[1] * PAGE, device="cuda")
    see = _visible(p[:, :, None], t, ctx[:, None, None], c["window"], c["sinks"]) & there[..., None]
    out = torch.zeros((B, n, c["h_q"], D), device="cuda")
    q = torch.zeros((B, n, c["h_q"], D), device="cuda")
    q[there] = s["q"][row].float()
    for h in range(c["h_kv"]):
        kc, ks, km, vc, vs, vm = _unpacked(_tokens(s["cache"][s["bt"].long(), h]).flatten(1, 2))
        k = _values(kc, ks, km) @ s["R_k"][h].T
        v = (_values(vc, vs, vm) @ s["R_v"][h].T).masked_fill((t >= ctx[:, None])[..., None], 0.0)
        a = q[:, :, h * G:(h + 1) * G].flatten(1, 2) @ k.transpose(-1, -2)       # [B, n G, T]
        a = (a * SCALE).view(B, n, G, -1).masked_fill_(~see[:, :, None], -math.inf)
        m = a.amax(-1, keepdim=True)
        a = a.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
        total = a.sum(-1, keepdim=True)
        o = (a.view(B, n * G, -1) @ v).view(B, n, G, D)
        out[:, :, h * G:(h + 1) * G] = o / torch.where(total > 0, total, torch.ones_like(total))
    s["out"][row] = out[there].bfloat16()
    return {"out": s["out"]}


# ------------------------------------------------------------------ the library's calls

def _own_rope(s):
    from bit_kv_cache_13_gb300 import _lib
    c = s["case"]
    q, k, v = s["qkv"].split([c["h_q"], c["h_kv"], c["h_kv"]], 1)
    _lib.kvq_append_rope_int4(q, k, v, s["positions"], s["rope"], s["slots"], s["mu"], s["R_k"], s["R_v"], s["cache"],
                              s["num_pages"], s["q_out"], s["k_out"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                              interleaved=c["interleaved"])
    _lib.kvq_dequant_int4(s["cache"], s["num_pages"], c["h_kv"], s["slots"], s["k_hat"], s["v_hat"])
    return {"q": s["q_out"], "k": s["k_out"], "k_hat": s["k_hat"], "v_hat": s["v_hat"]}


def _own_chunk(s):
    from bit_kv_cache_13_gb300 import _lib
    c = s["case"]
    if "ws" not in s:  # kept from call to call, as a serving loop keeps it
        s["ws"] = torch.zeros(_lib.kvq_chunk_workspace_bytes(s["q"].shape[0], c["B"], c["h_q"], c["h_kv"]), dtype=torch.uint8,
                              device="cuda")
    _lib.kvq_chunk_attn_int4(s["q"], s["q_start"], s["cache"], s["num_pages"], s["bt"], s["lens"], s["R_k"], s["R_v"], SCALE,
                             s["out"], s["ws"], window=c["window"], sinks=c["sinks"])
    return {"out": s["out"]}


def _own_sliding(s):
    from bit_kv_cache_13_gb300 import _lib
    c = s["case"]
    if "ws" not in s:
        s["ws"] = torch.zeros(_lib.kvq_int4_workspace_bytes(c["B"], c["h_q"], c["h_kv"], s["bt"].shape[1]), dtype=torch.uint8,
                              device="cuda")
    _lib.kvq_decode_attn_int4_sliding(s["q"], s["cache"], s["num_pages"], s["bt"], s["lens"], s["R_k"], s["R_v"], SCALE,
                                      c["window"], c["sinks"], s["out"], s["ws"])
    return {"out": s["out"]}


def run(state):
    op = state["case"]["op"]
    if op == "rope":
        return _own_rope(state) if own else _plain_rope(state)
    if op == "chunk":
        return _own_chunk(state) if own else _plain_attention(state)
    return _own_sliding(state) if own else _plain_attention(state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    h_q, h_kv, T = case["h_q"], case["h_kv"], case["T"]
    rotations = 2 * h_kv * D * D * 4
    if case["op"] == "rope":
        used = (T - len(range(5, T, 11)) if case["skip"] else T) * h_kv
        # q and k in and out, v in, a row of the table and two indices a token; packed records out and in, values out
        return {"bytes": T * (h_q + h_kv) * 512 + used * 256 + T * (case["rot"] * 4 + 8) + used * 2 * 160 + T * h_kv * 512
                + rotations + h_kv * D * 4, "flops": used * 4 * D * D}
    pairs = tokens = 0
    new, ctx = lengths(case)
    for n, c in zip(new, ctx):
        p = np.arange(c - n, c)
        p = p[p >= 0]
        if len(p) == 0:
            continue
        w, sinks = case["window"] or c, case["sinks"]
        low = np.maximum(p - w + 1, 0)
        pairs += int((p + 1 - low + np.minimum(low, sinks)).sum())
        tokens += int(c - low[0] + min(low[0], sinks))
    rows = sum(new)
    return {"bytes": tokens * h_kv * 160 + 4 * -(-tokens // PAGE) + rows * h_q * D * 4 + rotations + 8 * case["B"],
            "flops": pairs * h_q * 4 * D}


# ------------------------------------------------------------------ 64 bits, from the definition

def _exact_levels(cache, side):
    """float64 values [N, H, 16, 128] of the tiles' keys (side 0) or values (side 1), by each code's own byte address."""
    ch, slot = torch.arange(D, device=cache.device)[None, :], torch.arange(PAGE, device=cache.device)[:, None]
    g = ch // 32
    if side == 0:
        t, i = ch % 32 // 8, ch % 8
        code_at, nib = 64 * slot + 16 * t + 4 * g + i // 2, i % 2
        sc_at = 1024 + 16 * slot + 2 * g
        mn_at = sc_at + 8
    else:
        r, i = ch % 32 // 4, ch % 4
        code_at, nib = 1280 + 128 * (slot // 2) + 16 * r + 4 * g + 2 * (slot % 2) + i // 2, i % 2
        sc_at = 2304 + 16 * (slot // 2) + 4 * g + 2 * (slot % 2)
        mn_at = sc_at + 128
    full = lambda x: x.expand(PAGE, D).reshape(-1)  # noqa: E731
    code = cache[..., full(code_at)].to(torch.int32) >> (4 * full(nib)) & 15
    halves = cache.contiguous().view(torch.float16).double()
    v = halves[..., full(mn_at) // 2] + code.double() * halves[..., full(sc_at) // 2]
    return v.view(cache.shape[:-1] + (PAGE, D))


def _exact_rounded(y):
    """float64 cut to bfloat16's eight bits, to nearest even, by its bits."""
    b = y.contiguous().view(torch.int64)
    return ((b + ((1 << 44) - 1) + ((b >> 45) & 1)) & -(1 << 45)).view(torch.float64)


def _exact_rotated(s, x, weight):
    """The rotation as a complex product, pair by pair."""
    c = s["case"]
    y = x.double()
    if weight is not None:
        y = y / ((y ** 2).sum(-1, keepdim=True) / D + EPS).sqrt() * weight.double()
    half = c["rot"] // 2
    j = torch.arange(half, device="cuda")
    first, second = (2 * j, 2 * j + 1) if c["interleaved"] else (j, j + half)
    table = s["rope"].double()[s["positions"].long()]
    z = torch.complex(y[..., first], y[..., second]) * torch.complex(table[:, :half], table[:, half:])[:, None]
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_rope(s):
    """Each cached value by trying all 16 levels of its group and taking the nearest (the lower of two as near)."""
    h_q, h_kv = s["case"]["h_q"], s["case"]["h_kv"]
    out = {"q": _exact_rotated(s, s["qkv"][:, :h_q], s["q_weight"]), "k": _exact_rotated(s, s["qkv"][:, h_q:h_q + h_kv], s["k_weight"])}
    there = (s["slots"] >= 0)[:, None]
    for name, x, R in (("k_hat", _exact_rounded(out["k"]) - s["mu"].double(), s["R_k"]), ("v_hat", s["qkv"][:, h_q + h_kv:].double(), s["R_v"])):
        y = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
        for h in range(h_kv):
            z = (x[:, h] @ R[h].double()).view(-1, NG, GROUP)
            low = z.amin(-1, keepdim=True)
            step = ((z.amax(-1, keepdim=True) - low) / 15).float().clamp(max=65504).half().double()
            low = low.float().clamp(-65504, 65504).half().double()
            level = low.unsqueeze(-1) + step.unsqueeze(-1) * torch.arange(16, device="cuda")
            j = (z.unsqueeze(-1) - level).abs().argmin(-1)
            y[:, h] = (low + step * j).view(-1, D) * there
        out[name] = y
    return out


def _exact_attention(s):
    """A sequence and KV head at a time, 512 new tokens together, over the tokens that any of them sees."""
    c = s["case"]
    G = c["h_q"] // c["h_kv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, ctx) in enumerate(zip(*lengths(c))):
        for h in range(c["h_kv"] if ctx else 0):
            tiles = s["cache"][s["bt"][b].long(), h]
            k = _exact_levels(tiles, 0).reshape(-1, D)[:ctx] @ s["R_k"][h].double().T
            v = _exact_levels(tiles, 1).reshape(-1, D)[:ctx] @ s["R_v"][h].double().T
            for i in range(0, n, 512):
                p = torch.arange(ctx - n + i, ctx - n + min(n, i + 512), device="cuda")
                t = torch.arange(ctx, device="cuda")
                t = t[_visible(p[:, None], t, ctx, c["window"], c["sinks"]).any(0)]
                a = torch.einsum("ijd,td->ijt", s["q"][at + i:at + i + len(p), h * G:(h + 1) * G].double(), k[t]) / math.sqrt(D)
                a[~_visible(p[:, None], t, ctx, c["window"], c["sinks"])[:, None].expand(a.shape)] = -math.inf
                out[at + i:at + i + len(p), h * G:(h + 1) * G] = torch.softmax(a, -1) @ v[t]
        at += n
    return {"out": out}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_rope(s) if case["op"] == "rope" else _exact_attention(s)
