"""Pins of the scored-attention oracle: the plain oracle, a scalar loop, torch's own
differentiation in float64, and finite differences."""

import math

import numpy as np
import pytest
import torch

from oracle import attention_backward, attention_forward, paged_append, paged_decode, scored_backward, scored_forward, visible


def _rand(*shape, seed=0):
    return np.random.default_rng(seed).standard_normal(shape)


def test_without_options_it_is_plain_attention():
    q, k, v, g = (_rand(2, 3, 17, 8, seed=s) for s in range(4))
    for causal in (False, True):
        o, lse, _, _ = scored_forward(q, k, v, 0.3, causal)
        o_ref, lse_ref = attention_forward(q, k, v, 0.3, causal)
        assert np.allclose(o, o_ref, atol=1e-12) and np.allclose(lse, lse_ref, atol=1e-12)
        got, _ = scored_backward(q, k, v, g, 0.3, causal)
        for a, b in zip(got, attention_backward(q, k, v, g, 0.3, causal)):
            assert np.allclose(a, b, atol=1e-12)


def test_visible_by_hand():
    # Documents [1, 4) with prefix 2 and [4, 6) with none; position 0 and 6 are padding.
    see = visible(7, True, [1, 4, 4, 6], [2, 5, 0])
    want = np.array([[0, 0, 0, 0, 0, 0, 0], [0, 1, 1, 0, 0, 0, 0], [0, 1, 1, 0, 0, 0, 0], [0, 1, 1, 1, 0, 0, 0],
                     [0, 0, 0, 0, 1, 0, 0], [0, 0, 0, 0, 1, 1, 0], [0, 0, 0, 0, 0, 0, 0]], dtype=bool)
    assert np.array_equal(see, want)
    both = visible(7, False, [1, 4, 4, 6], None)
    assert both[1:4, 1:4].all() and both[4:6, 4:6].all() and both.sum() == 9 + 4


def test_forward_matches_a_scalar_loop():
    B, H, Hkv, N, d, cap, scale = 1, 4, 2, 9, 4, 1.5, 0.7
    q, k, v = _rand(B, H, N, d, seed=5) * 3, _rand(B, Hkv, N, d, seed=6), _rand(B, Hkv, N, d, seed=7)
    slopes, cu, pre = [0.5, 0.1, 0.0, -0.2], [[0, 5, 8]], [[3, 0]]
    o, lse, _, _ = scored_forward(q, k, v, scale, True, cap, slopes, cu, pre)
    for h in range(H):
        for i in range(N):
            doc = 0 if i < 5 else 1 if i < 8 else None
            js = [] if doc is None else [j for j in range(*((0, 5) if doc == 0 else (5, 8)))
                                         if j <= i or (doc == 0 and j < 3)]
            if not js:
                assert lse[0, h, i] == -math.inf and not o[0, h, i].any()
                continue
            s = [cap * math.tanh(scale * sum(q[0, h, i, c] * k[0, h // 2, j, c] for c in range(d)) / cap)
                 - slopes[h] * abs(i - j) for j in js]
            z = sum(math.exp(x) for x in s)
            assert abs(lse[0, h, i] - math.log(z)) < 1e-12
            for c in range(d):
                assert abs(o[0, h, i, c] - sum(math.exp(x) / z * v[0, h // 2, j, c] for x, j in zip(s, js))) < 1e-12


@pytest.mark.parametrize("cap,bias,causal", [(0.0, False, True), (2.0, False, True), (2.0, True, False), (0.0, True, True)])
def test_backward_matches_torch_and_differences(cap, bias, causal):
    B, H, Hkv, N, d, scale = 2, 4, 2, 11, 4, 0.6
    q, k, v, g = _rand(B, H, N, d, seed=1) * 2, _rand(B, Hkv, N, d, seed=2), _rand(B, Hkv, N, d, seed=3), _rand(B, H, N, d, seed=4)
    slopes = [0.3, 0.2, 0.1, 0.05] if bias else None
    cu, pre = [[0, 4, 10], [2, 2, 11]], [[2, 0], [0, 4]]
    (dq, dk, dv), _ = scored_backward(q, k, v, g, scale, causal, cap, slopes, cu, pre)
    see = torch.from_numpy(np.stack([visible(N, causal, cu[b], pre[b]) for b in range(B)]))[:, None]
    tq, tk, tv = (torch.from_numpy(x).requires_grad_() for x in (q, k, v))
    s = scale * tq @ tk.repeat_interleave(2, 1).transpose(2, 3)
    if cap:
        s = cap * torch.tanh(s / cap)
    if bias:
        pos = torch.arange(N, dtype=torch.float64)
        s = s - torch.tensor(slopes, dtype=torch.float64)[:, None, None] * (pos[:, None] - pos[None]).abs()
    p = torch.softmax(s.masked_fill(~see, -1e300), dim=-1) * see
    (p @ tv.repeat_interleave(2, 1) * torch.from_numpy(g)).sum().backward()
    for a, t in ((dq, tq), (dk, tk), (dv, tv)):
        assert np.allclose(a, t.grad.numpy(), atol=1e-11)
    f = lambda qq, kk, vv: float((scored_forward(qq, kk, vv, scale, causal, cap, slopes, cu, pre)[0] * g).sum())
    rng = np.random.default_rng(9)
    for n, x in enumerate((q, k, v)):
        step = rng.standard_normal(x.shape)
        hi, lo = [q, k, v], [q, k, v]
        hi[n], lo[n] = x + 1e-5 * step, x - 1e-5 * step
        assert abs((f(*hi) - f(*lo)) / 2e-5 - float(((dq, dk, dv)[n] * step).sum())) < 1e-6


def test_paged_decode_is_the_last_row_of_the_dense_form():
    B, H, Hkv, d, page = 3, 4, 2, 8, 16
    lens = [21, 0, 16]
    k, v = (_rand(1, Hkv, 21, d, seed=s) for s in (1, 2))
    q = _rand(B, H, d, seed=3)
    table = [[4, 1], [0, 0], [2, 2]]
    kc, vc = np.full((5, Hkv, page, d), np.nan), np.full((5, Hkv, page, d), np.nan)
    for b in (0, 2):
        kc = paged_append(k[0].transpose(1, 0, 2)[:lens[b]], kc, [table[b]], [lens[b]], [0, lens[b]])
        vc = paged_append(v[0].transpose(1, 0, 2)[:lens[b]], vc, [table[b]], [lens[b]], [0, lens[b]])
    slopes = [0.2, 0.1, 0.3, 0.0]
    o, lse, _, _ = paged_decode(q, kc, vc, table, lens, 0.5, 2.0, slopes)
    assert not o[1].any() and np.isneginf(lse[1]).all()
    for b in (0, 2):
        n = lens[b]
        qq = np.zeros((1, H, n, d))
        qq[0, :, n - 1] = q[b]
        o_ref, lse_ref, _, _ = scored_forward(qq, k[:, :, :n], v[:, :, :n], 0.5, True, 2.0, slopes)
        assert np.allclose(o[b], o_ref[0, :, n - 1], atol=1e-12) and np.allclose(lse[b], lse_ref[0, :, n - 1], atol=1e-12)


def test_paged_append_by_hand():
    cache = np.zeros((3, 1, 16, 1))
    rows = np.arange(1, 6, dtype=np.float64).reshape(5, 1, 1)
    # Sequence 0 gets rows 0-2 at positions 15, 16, 17 (pages 2, 0); sequence 1 nothing; sequence 2
    # row 3 at position 0 of a page outside the cache; row 4 belongs to no sequence.
    out = paged_append(rows, cache, [[2, 0], [1, 1], [7, 1]], [18, 4, 1], [0, 3, 3, 4])
    assert out[2, 0, 15, 0] == 1 and out[0, 0, 0, 0] == 2 and out[0, 0, 1, 0] == 3 and out.sum() == 6
