"""Scored attention and its paged decode, float64 numpy (test infrastructure).

The plain definition, one dense matrix per head, with no tiling and no intervals:

    a_ij = scale q_i . k_j
    c_ij = cap tanh(a_ij / cap)          (cap = 0: c = a)
    s_ij = c_ij - slope_h |i - j|        (no slopes: s = c)
    LSE_i = ln sum_{j visible} exp(s_ij), O_i = sum exp(s_ij - LSE_i) v_j

Query head h reads key/value head h // (H // Hkv).  Which keys a query sees is decided
pair by pair from the documents (see ``visible``).  The gradient is the chain rule
applied to that, with dS carried through the cap by 1 - tanh^2; dK and dV sum over the
query heads that share a head.

The error bounds that the tests use are derived here as well, from the roundings the
GPU path makes on purpose (P and dS to bf16 as matrix operands, O, dQ, dK, dV to bf16
at the end, half a step = 2^-8 relative each) and the fp32 rounding of the scores.
"""

from __future__ import annotations

import numpy as np

from .attention import _as_f64

HALF = 2.0 ** -8       # half a bf16 step, relative
HALF32 = 2.0 ** -24    # half an fp32 step, relative


def visible(N: int, causal: bool, cu=None, prefix=None) -> np.ndarray:
    """Truth values [N, N] of one row of the batch: query i sees key j.

    cu: offsets of the row's documents (None: one document of N positions); prefix:
    the documents' prefix lengths (None: 0)."""
    see = np.zeros((N, N), dtype=bool)
    cu = [0, N] if cu is None else [int(x) for x in cu]
    for t, (s, e) in enumerate(zip(cu, cu[1:])):
        p = 0 if prefix is None else max(int(prefix[t]), 0)
        for i in range(s, e):
            see[i, s:e] = True if not causal else np.arange(s, e) < max(i + 1, min(s + p, e))
    return see


def _pair(q, k, i_minus_j, scale, cap, slope):
    """Scores of one head before the mask, and the cap's derivative."""
    a = scale * (q @ k.T)
    bend = np.ones_like(a)
    if cap > 0:
        t = np.tanh(a / cap)
        a, bend = cap * t, 1.0 - t * t
    return a - slope * np.abs(i_minus_j), bend


def _head(q, k, see, scale, cap, slope):
    """(P, LSE, bend) of one head; rows that see nothing get P = 0, LSE = -inf."""
    pos = np.arange(q.shape[0], dtype=np.float64)
    s, bend = _pair(q, k, pos[:, None] - pos[None, :], scale, cap, slope)
    s = np.where(see, s, -np.inf)
    any_key = see.any(axis=1)
    top = np.where(any_key, np.max(s, axis=1, initial=-np.inf), 0.0)
    e = np.where(see, np.exp(s - top[:, None]), 0.0)
    l = e.sum(axis=1)
    with np.errstate(divide="ignore"):
        lse = np.where(any_key, top + np.log(np.where(any_key, l, 1.0)), -np.inf)
    return e / np.where(any_key, l, 1.0)[:, None], lse, bend


def _masks(B, N, causal, cu, prefix):
    return [visible(N, causal, None if cu is None else cu[b], None if prefix is None else prefix[b]) for b in range(B)]


def _score_error(q, k, scale, cap, slope, d):
    """How far a score may be off in fp32: the dot product's d + 1 roundings, the cap's and the
    bias's, and the base-2 exponent's product (8 more half steps of each magnitude)."""
    size = scale * np.max(np.abs(q) @ np.abs(k).T, initial=0.0)
    # The cap itself is evaluated to 8 half steps (absolute) of the cap, or of the largest score if that is smaller.
    return HALF32 * ((d + 8) * size + 8 * min(cap, size) + 8 * slope * q.shape[0]) + 2e-6


def scored_forward(q, k, v, scale, causal, cap=0.0, slopes=None, cu=None, prefix=None):
    """(O, LSE, bound on |O error|, bound on |LSE error|), each for every element."""
    q, k, v = _as_f64(q), _as_f64(k), _as_f64(v)
    B, H, N, d = q.shape
    G = H // k.shape[1]
    o, lse = np.zeros(q.shape), np.zeros((B, H, N))
    ob, lb = np.zeros(q.shape), np.zeros((B, H, N))
    for b, see in enumerate(_masks(B, N, causal, cu, prefix)):
        for h in range(H):
            slope = 0.0 if slopes is None else float(slopes[h])
            P, lse[b, h], _ = _head(q[b, h], k[b, h // G], see, scale, cap, slope)
            vv = v[b, h // G]
            o[b, h] = P @ vv
            err = _score_error(q[b, h], k[b, h // G], scale, cap, abs(slope), d)
            # P rounded to bf16; each weight off by the scores' error, twice (its own and the sum's).
            ob[b, h] = (HALF + 3 * err) * (P @ np.abs(vv)) * 1.01 + HALF * np.abs(o[b, h]) + 1e-30
            lb[b, h] = 2 * err + 4 * HALF32 * np.abs(np.where(np.isfinite(lse[b, h]), lse[b, h], 0.0))
    return o, lse, ob, lb


def scored_backward(q, k, v, do, scale, causal, cap=0.0, slopes=None, cu=None, prefix=None, o_given=True):
    """((dQ, dK, dV), bounds on their errors).

    The bounds assume the GPU path: O (in D = dO . O) carries the forward's bf16
    roundings, P and dS are rounded to bf16 as operands, the results once at the end."""
    q, k, v, do = _as_f64(q), _as_f64(k), _as_f64(v), _as_f64(do)
    B, H, N, d = q.shape
    Hkv = k.shape[1]
    G = H // Hkv
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    bq, bk, bv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    for b, see in enumerate(_masks(B, N, causal, cu, prefix)):
        for h in range(H):
            hk = h // G
            slope = 0.0 if slopes is None else float(slopes[h])
            qq, kk, vv, g = q[b, h], k[b, hk], v[b, hk], do[b, h]
            P, _, bend = _head(qq, kk, see, scale, cap, slope)
            dP = g @ vv.T
            D = (P * dP).sum(axis=1, keepdims=True)
            dS = P * (dP - D) * bend
            dq[b, h] = scale * dS @ kk
            dk[b, hk] += scale * dS.T @ qq
            dv[b, hk] += P.T @ g
            err = _score_error(qq, kk, scale, cap, abs(slope), d)
            # Error of O before its use in D (as in scored_forward), hence of D.
            Oe = (HALF + 3 * err) * (P @ np.abs(vv)) * 1.01 + HALF * np.abs(P @ vv)
            De = (np.abs(g) * Oe).sum(axis=1, keepdims=True)
            # dP and D in fp32 (D enters the matrix product as three bf16 terms of 24 bits).
            sums = (np.abs(g) @ np.abs(vv).T) * (d + 8) * HALF32 + np.abs(D) * 8 * HALF32
            # 1 - tanh^2 in fp32: absolute error of a few half steps of 1.
            dSe = P * ((De + sums) * bend + np.abs(dP - D) * (bend * (HALF + 4 * err) + (16 * HALF32 if cap > 0 else 0.0)))
            bq[b, h] = scale * dSe @ np.abs(kk) * 1.02
            bk[b, hk] += scale * dSe.T @ np.abs(qq) * 1.02
            bv[b, hk] += (HALF + 4 * err) * (P.T @ np.abs(g)) * 1.02
    out = (dq, dk, dv)
    return out, tuple(bd + HALF * np.abs(x) + 1e-30 for bd, x in zip((bq, bk, bv), out))


def paged_gather(cache, table, n):
    """The first n tokens [Hkv, n, d] of a sequence whose pages are table[0], table[1], ...

    cache: [n_pages, Hkv, page, d]; a page index outside the cache reads as zeros."""
    cache = _as_f64(cache)
    n_pages, Hkv, page, d = cache.shape
    out = np.zeros((Hkv, n, d))
    for j in range(n):
        p = int(table[j // page])
        if 0 <= p < n_pages:
            out[:, j] = cache[p, :, j % page]
    return out


def paged_decode(q, k_cache, v_cache, table, lens, scale, cap=0.0, slopes=None, half=HALF):
    """(O [B, H, d], LSE [B, H], bounds): attention of each sequence's last token.

    half: half a step of the 16-bit type (P is rounded to it, and O)."""
    q = _as_f64(q)
    B, H, d = q.shape
    n_pages, Hkv, page, _ = np.shape(k_cache)
    G = H // Hkv
    o, lse = np.zeros((B, H, d)), np.full((B, H), -np.inf)
    ob, lb = np.zeros((B, H, d)), np.zeros((B, H))
    for b in range(B):
        n = min(max(int(lens[b]), 0), len(table[b]) * page)
        if n == 0:
            continue
        k, v = paged_gather(k_cache, table[b], n), paged_gather(v_cache, table[b], n)
        back = n - 1 - np.arange(n, dtype=np.float64)
        for h in range(H):
            slope = 0.0 if slopes is None else float(slopes[h])
            s, _ = _pair(q[b, h:h + 1], k[h // G], back[None, :], scale, cap, slope)
            top = s.max()
            e = np.exp(s[0] - top)
            P, lse[b, h] = e / e.sum(), top + np.log(e.sum())
            o[b, h] = P @ v[h // G]
            size = scale * np.max(np.abs(q[b, h]) @ np.abs(k[h // G]).T)
            err = HALF32 * ((d + 8) * size + 8 * min(cap, size) + 8 * abs(slope) * n) + 2e-6
            ob[b, h] = (half + 3 * err) * (P @ np.abs(v[h // G])) * 1.01 + half * np.abs(o[b, h]) + 2.0 ** -24
            lb[b, h] = 2 * err + 4 * HALF32 * abs(lse[b, h])
    return o, lse, ob, lb


def paged_append(k, k_cache, table, lens, cu):
    """The cache (a copy, the same type) with each sequence's new rows written token by token."""
    cache = np.array(k_cache, copy=True)
    k = np.asarray(k)
    n_pages, _, page, _ = cache.shape
    for b in range(len(lens)):
        for t in range(int(cu[b]), int(cu[b + 1])):
            pos = int(lens[b]) - (int(cu[b + 1]) - t)
            if 0 <= pos < len(table[b]) * page and 0 <= int(table[b][pos // page]) < n_pages:
                cache[int(table[b][pos // page]), :, pos % page] = k[t]
    return cache
