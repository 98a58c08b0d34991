"""Norm and rotation of queries and keys, and the paged cache in 8 bits with its bookkeeping, float64 numpy
(test infrastructure).

    y = x / sqrt(mean(x^2) + eps) * w,  pairs (y_a, y_b) turned by position * inv_freq
    a block of 16 tokens and head: e = the least integer >= -126 with every new value <= 448 * 2^e, or the
    older tokens' e if that is larger; code = e4m3(x 2^-e), older codes re-coded by 2^(e_old - e)

The error bounds are derived here from the roundings that the GPU path makes: half a step of
the output's type (2^-8 bf16, 2^-11 fp16, relative), fp32 inside, fp16 weights in P V.
"""

from __future__ import annotations

import numpy as np

from .attention import _as_f64
from .fp8 import e4m3_decode, e4m3_encode
from .scored import HALF32, _pair

BLOCK = 16
ANGLE = 2.0 ** -21  # cos and sin: the angle to 2^-32 of a turn and to fp32 (pi 2^-24), the functions to 2 steps of 2^-23


# ------------------------------------------------------------------ norm and rotation


def turns(pos, inv_freq):
    """cos and sin [..., rot / 2] of pos * inv_freq; the product in more than 64 bits of fraction."""
    angle = np.asarray(pos).astype(np.longdouble)[..., None] * np.asarray(inv_freq).astype(np.longdouble)
    return np.cos(angle).astype(np.float64), np.sin(angle).astype(np.float64)


def _places(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def _turned(y, c, s, rot, interleaved):
    one, two = _places(rot, interleaved)
    out = np.array(y)
    a, b = y[..., one], y[..., two]
    out[..., one], out[..., two] = a * c - b * s, a * s + b * c
    return out


def _spread(y, rot, interleaved):
    """|y_a| + |y_b| at both places of a pair, |y| elsewhere."""
    one, two = _places(rot, interleaved)
    out = np.abs(y)
    both = out[..., one] + out[..., two]
    out[..., one], out[..., two] = both, both
    return out


def _angles(shape, inv_freq, positions):
    B, _, N, _ = shape
    pos = np.broadcast_to(np.arange(N), (B, N)) if positions is None else np.asarray(positions)
    c, s = turns(pos, inv_freq)
    return c[:, None], s[:, None]


def qk_norm_rope(x, w=None, inv_freq=None, positions=None, eps=1e-6, norm=True, interleaved=False, half=2.0 ** -8):
    """(y, bound on |y error|) of one tensor [B, H, N, d]."""
    x = _as_f64(x)
    d = x.shape[3]
    y, rel = x, 0.0
    if norm:
        y = x / np.sqrt((x * x).mean(axis=3, keepdims=True) + eps)
        y = y if w is None else y * _as_f64(w)
        rel = (d / 2 + 12) * HALF32  # the sum of squares (halved by the root), the root, two products
    err = rel * np.abs(y)
    rot = 0 if inv_freq is None else 2 * len(inv_freq)
    if rot:
        c, s = _angles(x.shape, inv_freq, positions)
        err = (rel + ANGLE + 4 * HALF32) * _spread(y, rot, interleaved)
        y = _turned(y, c, s, rot, interleaved)
    return y, err + half * (np.abs(y) + err) + 2.0 ** -25


def qk_norm_rope_backward(x, dy, w=None, inv_freq=None, positions=None, eps=1e-6, norm=True, interleaved=False, half=2.0 ** -8):
    """((dx, dw or None), (bound, bound or None)) of one tensor."""
    x, g = _as_f64(x), _as_f64(dy)
    d, rot = g.shape[3], 0 if inv_freq is None else 2 * len(inv_freq)
    ge = np.zeros_like(g)
    if rot:
        c, s = _angles(g.shape, inv_freq, positions)
        ge = (ANGLE + 4 * HALF32) * _spread(g, rot, interleaved)
        g = _turned(g, c, -s, rot, interleaved)
    if not norm:
        return (g, None), (ge + half * (np.abs(g) + ge) + 2.0 ** -25, None)
    rel = (d / 2 + 12) * HALF32
    r = 1.0 / np.sqrt((x * x).mean(axis=3, keepdims=True) + eps)
    xh = x * r
    ww = 1.0 if w is None else _as_f64(w)
    h, he = g * ww, ge * np.abs(ww) + HALF32 * np.abs(g * ww)
    mean = (h * xh).mean(axis=3, keepdims=True)
    mean_e = (he * np.abs(xh) + ((d + 4) * HALF32 + rel) * np.abs(h * xh)).mean(axis=3, keepdims=True)
    dx = r * (h - xh * mean)
    de = r * (he + np.abs(xh) * (mean_e + rel * np.abs(mean)) + (rel + 4 * HALF32) * (np.abs(h) + np.abs(xh * mean)))
    dw = we = None
    if w is not None:
        rows = g.shape[0] * g.shape[1] * g.shape[2]
        dw = (g * xh).sum(axis=(0, 1, 2))
        # Each product, and their sum in fp32 in any order.
        we = (ge * np.abs(xh) + (rel + (rows + 2) * HALF32) * np.abs(g * xh)).sum(axis=(0, 1, 2)) + 2.0 ** -126
    return (dx, dw), (de + half * (np.abs(dx) + de) + 2.0 ** -25, we)


# ------------------------------------------------------------------- the cache in 8 bits


def block_exponent(top):
    """The least integer e >= -126 with top <= 448 * 2^e."""
    e = -126
    while top > 448.0 * 2.0 ** e:
        e += 1
    return e


def paged_append_fp8(x, codes, scales, table, lens, cu):
    """(codes, scales) after each sequence's new rows of one tensor are written.

    x: [T, Hkv, d]; codes: uint8 [n_pages, Hkv, page, d]; scales: [n_pages, Hkv, page / 16]."""
    codes, scales = np.array(codes, copy=True), np.array(scales, dtype=np.float64, copy=True)
    x = _as_f64(x)
    n_pages, Hkv, page, _ = codes.shape
    for b in range(len(lens)):
        blocks = {}  # (page, block) -> [(row of x, place in the block)]
        for t in range(int(cu[b]), int(cu[b + 1])):
            pos = int(lens[b]) - (int(cu[b + 1]) - t)
            if 0 <= pos < len(table[b]) * page and 0 <= int(table[b][pos // page]) < n_pages:
                blocks.setdefault((int(table[b][pos // page]), pos % page // BLOCK), []).append((t, pos % BLOCK))
        for (p, blk), rows in blocks.items():
            first, held = blk * BLOCK, rows[0][1]
            for h in range(Hkv):
                new = x[[t for t, _ in rows], h]
                e = block_exponent(np.max(np.abs(new), initial=0.0, where=np.isfinite(new)))
                if held:
                    old = int(np.ceil(np.log2(scales[p, h, blk])))
                    e = max(e, old)
                    if 2.0 ** e != scales[p, h, blk]:
                        codes[p, h, first:first + held] = e4m3_encode(
                            e4m3_decode(codes[p, h, first:first + held]) * (scales[p, h, blk] / 2.0 ** e))
                scales[p, h, blk] = 2.0 ** e
                codes[p, h, first + held:first + held + len(rows)] = e4m3_encode(new / 2.0 ** e)
    return codes, scales


def paged_values(codes, scales):
    """The values that a cache of codes stands for, [n_pages, Hkv, page, d]."""
    return e4m3_decode(codes) * np.repeat(_as_f64(scales), BLOCK, axis=2)[..., None]


def _gather(cache, table, n, fill=0.0):
    n_pages, Hkv, page, d = cache.shape
    out = np.full((Hkv, n, d), fill)
    for j in range(n):
        p = int(table[j // page])
        if 0 <= p < n_pages:
            out[:, j] = cache[p, :, j % page]
    return out


def paged_decode_fp8(q, k_codes, v_codes, k_scales, v_scales, table, lens, scale, cap=0.0, slopes=None, half=2.0 ** -8):
    """(O [B, H, d], LSE [B, H], bounds): attention of each sequence's last token over the values that the cache stands for."""
    q = _as_f64(q)
    B, H, d = q.shape
    page = np.shape(k_codes)[2]
    k_all, v_all = paged_values(k_codes, k_scales), paged_values(v_codes, v_scales)
    sv_all = np.repeat(_as_f64(v_scales), BLOCK, axis=2)[..., None]
    G = H // k_all.shape[1]
    o, lse = np.zeros((B, H, d)), np.full((B, H), -np.inf)
    ob, lb = np.zeros((B, H, d)), np.zeros((B, H))
    for b in range(B):
        n = min(max(int(lens[b]), 0), len(table[b]) * page)
        if n == 0:
            continue
        k, v, sv = _gather(k_all, table[b], n), _gather(v_all, table[b], n), _gather(sv_all, table[b], n)[..., 0]
        back = n - 1 - np.arange(n, dtype=np.float64)
        for h in range(H):
            slope = 0.0 if slopes is None else float(slopes[h])
            kk, vv = k[h // G], v[h // G]
            s, _ = _pair(q[b, h:h + 1], kk, back[None, :], scale, cap, slope)
            top = s.max()
            e = np.exp(s[0] - top)
            P, lse[b, h] = e / e.sum(), top + np.log(e.sum())
            o[b, h] = P @ vv
            size = scale * np.max(np.abs(q[b, h]) @ np.abs(kk).T)
            # What fp16's range loses of q's small entries, and of the weights times V's scales, beside the largest.
            small = np.abs(q[b, h]) * (np.abs(q[b, h]) < 2.0 ** -28 * np.abs(q[b, h]).max())
            lost = scale * np.max(np.abs(kk) @ np.minimum(small, 2.0 ** -39 * np.abs(q[b, h]).max()))
            err = HALF32 * ((d + 12) * size + 8 * min(cap, size) + 8 * abs(slope) * n) + lost + 2e-6
            w = P * sv[h // G]
            w = np.where(w < 2.0 ** -21 * w.max(), np.minimum(w, 2.0 ** -32 * w.max()), 0.0)
            # P times V's scale rounded to fp16, and what it loses.
            ob[b, h] = (2.0 ** -11 + 3 * err) * (P @ np.abs(vv)) * 1.01 + half * np.abs(o[b, h]) + 2.0 ** -24
            ob[b, h] += w @ np.where(sv[h // G][:, None] > 0, np.abs(vv) / np.maximum(sv[h // G], 1e-300)[:, None], 0.0)
            lb[b, h] = 2 * err + 4 * HALF32 * abs(lse[b, h])
    return o, lse, ob, lb


# ------------------------------------------------------------------------ bookkeeping


def paged_resize(table, lens, delta, free, count, page, rows):
    """(lens, cu_new, count, status, table, free, slots, positions), sequence by sequence; `rows`: how many slots are asked for."""
    B, width = len(lens), len(table[0]) if len(table) else 0
    table, free, lens = [list(map(int, r)) for r in table], list(map(int, free)), [int(x) for x in lens]
    delta = [int(x) for x in delta]
    count_in = min(max(int(count), 0), len(free))
    pages = lambda n: -(-n // page)
    unfit = sum(not (0 <= n <= width * page and 0 <= n + x <= width * page) for n, x in zip(lens, delta))
    ok = [0 <= n <= width * page and 0 <= n + x <= width * page for n, x in zip(lens, delta)]
    back = sum(max(pages(n) - pages(n + x), 0) for n, x, y in zip(lens, delta, ok) if y)
    take = sum(max(pages(n + x) - pages(n), 0) for n, x, y in zip(lens, delta, ok) if y)
    new = sum(max(x, 0) for x, y in zip(delta, ok) if y)
    bad = unfit + (count_in + back > len(free)) + (new > 2 ** 31 - 1)
    missing = max(take - count_in - back, 0)
    nothing = ([-1] * rows, [-1] * rows)
    if bad or missing:
        return lens, [0] * (B + 1), int(count), [missing, bad], table, free, *nothing
    pool = free[:count_in]
    for b in range(B):
        pool += table[b][pages(lens[b] + delta[b]):pages(lens[b])]
    free[:len(pool)] = pool
    cu, slots, positions = [0], [], []
    for b in range(B):
        for j in range(pages(lens[b]), pages(lens[b] + delta[b])):
            table[b][j] = pool.pop()
        for p in range(lens[b], lens[b] + delta[b]):
            slots.append(table[b][p // page] * page + p % page)
            positions.append(p)
        cu.append(len(slots))
        lens[b] += delta[b]
    tail = [-1] * rows
    return lens, cu, len(pool), [0, 0], table, free, (slots + tail)[:rows], (positions + tail)[:rows]
