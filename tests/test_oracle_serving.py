"""The oracle of norm and rotation, of the 8-bit paged cache and of its bookkeeping, against closed forms,
finite differences, hand-worked values and the 16-bit cache's oracle."""

import numpy as np
import pytest

from oracle import (e4m3_decode, e4m3_encode, paged_append_fp8, paged_decode, paged_decode_fp8, paged_resize, paged_values,
                    qk_norm_rope, qk_norm_rope_backward)
from oracle.serving import block_exponent, turns

RNG = lambda s: np.random.default_rng(s)


def _freq(rot, base=10000.0):
    return (base ** (-np.arange(0, rot, 2) / rot)).astype(np.float32)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_depends_on_distances_alone(interleaved):
    q, k = RNG(1).normal(size=(2, 1, 2, 1, 64))
    f = _freq(64)
    dots = []
    for shift in (0, 5, 100000):
        a, _ = qk_norm_rope(q, None, f, [[7 + shift]], norm=False, interleaved=interleaved)
        b, _ = qk_norm_rope(k, None, f, [[3 + shift]], norm=False, interleaved=interleaved)
        assert np.allclose((a * a).sum(-1), (q * q).sum(-1), rtol=1e-12)
        dots.append((a * b).sum(-1))
    assert np.allclose(dots[0], dots[1], atol=1e-9) and np.allclose(dots[0], dots[2], atol=1e-9)


def test_rotation_by_a_quarter_turn():
    x = np.zeros((1, 1, 1, 64))
    x[..., 0], x[..., 1], x[..., 20] = 2.0, 3.0, 7.0
    f = np.zeros(8, dtype=np.float32)
    f[0] = np.float32(np.pi / 2)
    y, _ = qk_norm_rope(x, None, f, [[1]], norm=False)  # pairs (0, 8), ...: 2 at 0 goes to 8
    assert np.allclose(y[0, 0, 0, [0, 8, 1, 20]], [0, 2, 3, 7], atol=1e-6)
    y, _ = qk_norm_rope(x, None, f, [[1]], norm=False, interleaved=True)
    assert np.allclose(y[0, 0, 0, [0, 1, 20]], [-3, 2, 7], atol=1e-6)


def test_norm_of_a_row():
    x = np.zeros((1, 1, 1, 64))
    x[..., 3] = 8.0  # mean square 1
    y, _ = qk_norm_rope(x, np.full(64, 0.5), eps=3.0)
    assert np.allclose(y[..., 3], 8 * 0.5 / 2) and not y[..., :3].any()


def test_angles_of_far_positions():
    # 2^31 - 1 turns by the fp32 number nearest 1: against the product reduced in whole numbers.
    c, s = turns([2 ** 31 - 1, -2 ** 31, 10 ** 6], np.array([1.0, 1.0 / 3], dtype=np.float32))
    two_pi = 6283185307179586476925286766559005768394  # 2 pi * 10^39
    for i, p in enumerate((2 ** 31 - 1, -2 ** 31, 10 ** 6)):
        for j, f in enumerate((1.0, float(np.float32(1.0 / 3)))):
            num, den = f.as_integer_ratio()
            r = (p * num * 10 ** 39) % (two_pi * den) / (10 ** 39 * den)
            assert abs(c[i, j] - np.cos(r)) < 1e-9 and abs(s[i, j] - np.sin(r)) < 1e-9


@pytest.mark.parametrize("rot,interleaved,norm", [(64, False, True), (32, True, True), (0, False, True), (16, False, False)])
def test_gradient_by_differences(rot, interleaved, norm):
    g = RNG(2)
    x, dy, w = g.normal(size=(1, 2, 3, 64)), g.normal(size=(1, 2, 3, 64)), 1 + 0.3 * g.normal(size=64) if norm else None
    f = _freq(rot) if rot else None
    kw = dict(inv_freq=f, positions=[[4, 0, 900]], eps=1e-3, norm=norm, interleaved=interleaved)
    (dx, dw), _ = qk_norm_rope_backward(x, dy, w, **kw)
    loss = lambda x, w: float((qk_norm_rope(x, w, **kw)[0] * dy).sum())
    for _ in range(8):
        u = g.normal(size=x.shape)
        assert abs((loss(x + 1e-5 * u, w) - loss(x - 1e-5 * u, w)) / 2e-5 - (dx * u).sum()) < 1e-7
        if norm:
            u = g.normal(size=64)
            assert abs((loss(x, w + 1e-5 * u) - loss(x, w - 1e-5 * u)) / 2e-5 - (dw * u).sum()) < 1e-7


def test_block_exponent():
    assert block_exponent(448.0) == 0 and block_exponent(448.5) == 1 and block_exponent(224.0) == -1
    assert block_exponent(0.0) == -126 and block_exponent(1.75 * 2.0 ** -20) == -28 and block_exponent(3e38) == 120


def test_append_fp8_by_hand():
    # One head, pages of 16: a token of 448, one of 900 beside it (the first is re-coded to half its code), a third too small to count.
    codes, scales = np.full((2, 1, 16, 64), 0x55, np.uint8), np.full((2, 1, 1), 1e9)
    x = np.zeros((3, 1, 64))
    x[0, 0, 0], x[1, 0, 1], x[2, 0, 2], x[2, 0, 3] = 448.0, 900.0, 2.0 ** -9, 3.0 * 2 ** -9
    c, s = paged_append_fp8(x[:1], codes, scales, [[1]], [1], [0, 1])
    assert s[1, 0, 0] == 1.0 and c[1, 0, 0, 0] == 0x7E and s[0, 0, 0] == 1e9
    c, s = paged_append_fp8(x[1:2], c, s, [[1]], [2], [0, 1])
    # 900 > 2 * 448: the scale is 4; 448 becomes 112 = 1.75 * 2^6, 900 / 4 = 225 rounds to 224.
    assert s[1, 0, 0] == 4.0 and e4m3_decode(c[1, 0, 0, 0]) == 112 and e4m3_decode(c[1, 0, 1, 1]) == 224
    c, s = paged_append_fp8(x[2:], c, s, [[1]], [3], [0, 1])
    # 2^-11 and 3 2^-11 in units of the smallest code, 2^-9: 1/4 and 3/4.
    assert s[1, 0, 0] == 4.0 and c[1, 0, 2, 2] == 0 and e4m3_decode(c[1, 0, 2, 3]) == 2.0 ** -9
    assert (c[1, 0, 3:] == 0x55).all() and (c[0] == 0x55).all()


def test_decode_fp8_is_the_decode_of_the_values():
    g = RNG(3)
    codes = [e4m3_encode(100 * g.normal(size=(5, 2, 32, 64))) for _ in range(2)]
    scales = [2.0 ** g.integers(-8, -5, size=(5, 2, 2)) for _ in range(2)]
    q = g.normal(size=(2, 6, 64))
    args = ([[3, 0], [4, 1]], [45, 7], 0.125, 20.0, 2.0 ** -np.arange(6.0))
    o, lse, _, _ = paged_decode_fp8(q, *codes, *scales, *args)
    ref = paged_decode(q, *(paged_values(c, s) for c, s in zip(codes, scales)), *args)
    assert np.allclose(o, ref[0], rtol=1e-12) and np.allclose(lse, ref[1], rtol=1e-12)


def test_resize_by_hand():
    # Pages of 16.  Sequence 0 gives back its second page (7), 1 ends (pages 4, 5), 2 takes two pages: 5, then 4.
    table = [[3, 7, -1], [4, 5, -1], [6, -1, -1]]
    lens, cu, count, status, table, free, slots, pos = paged_resize(table, [20, 32, 15], [-4, -32, 20], [9, 8, 0, 0, 0, 0], 2, 16, 22)
    assert lens == [16, 0, 35] and cu == [0, 0, 0, 20] and status == [0, 0]
    assert table == [[3, 7, -1], [4, 5, -1], [6, 5, 4]]
    assert free == [9, 8, 7, 4, 5, 0] and count == 3
    assert pos == list(range(15, 35)) + [-1, -1]
    assert slots == [6 * 16 + 15] + list(range(80, 96)) + [64, 65, 66] + [-1, -1]


def test_resize_refuses_as_a_whole():
    table = [[3, 7], [4, 5]]
    out = paged_resize(table, [20, 17], [-20, 40], [1, 2, 0, 0], 2, 16, 3)
    assert out[0] == [20, 17] and out[1] == [0, 0, 0] and out[2] == 2 and out[3] == [0, 1] and out[6] == [-1] * 3
    out = paged_resize([[3, -1, -1, -1]], [10], [54], [1, 2], 2, 16, 0)
    assert out[3] == [1, 0] and out[2] == 2 and out[4] == [[3, -1, -1, -1]]


def test_resize_keeps_every_page():
    g = RNG(4)
    B, page, width = 20, 16, 12
    free, count = list(g.permutation(150)), 150
    table, lens = [[-1] * width for _ in range(B)], [0] * B
    for _ in range(60):
        delta = [int(g.integers(-n, 40)) if n + 40 <= width * page else int(g.integers(-n, 1)) for n in lens]
        lens, cu, count, status, table, free, *_ = paged_resize(table, lens, delta, free, count, page, 0)
        held = [p for r, n in zip(table, lens) for p in r[:-(-n // page)]]
        assert sorted(held + free[:count]) == list(range(150))
