"""The paged cache in 8-bit codes on the GPU, and its bookkeeping, against the float64 oracle."""

import numpy as np
import pytest
import torch

import io_aware_exact_fwd_gb300 as fa
from oracle import e4m3_decode, e4m3_encode, paged_append_fp8, paged_decode_fp8, paged_resize

from gpu_util import host_f64, report

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fa.load_library()
    fa.fa_debug_set_wait_limit_ns(0)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _slopes(H):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=torch.float32, device="cuda")


def _tables(lens, page, g, spare=2):
    need = [max(0, -(-n // page)) for n in lens]
    n_pages, width = sum(need) + spare, max(1, max(need))
    order = torch.randperm(n_pages, generator=g)[:sum(need)].tolist()
    table, at = [], 0
    for n in need:
        table.append(order[at:at + n] + [n_pages + 5] * (width - n))  # unused entries: outside the cache
        at += n
    return table, n_pages


def _codes(shape, layout, g, largest=0x7E):
    """Random codes without NaN, and scales: powers of two and other numbers of very different sizes."""
    n_pages, Hkv, page, d = shape
    c = torch.randint(0, largest + 1, shape, generator=g, dtype=torch.uint8) | (torch.randint(0, 2, shape, generator=g, dtype=torch.uint8) << 7)
    s = torch.exp2(torch.randint(-12, -6, (n_pages, Hkv, page // 16), generator=g).float()) * (1 + 0.4 * torch.rand(n_pages, Hkv, page // 16, generator=g))
    c = c.cuda()
    if layout == "nhd":
        c = c.transpose(1, 2).contiguous().transpose(1, 2)
    return c, s.cuda()


def _cache(lens, Hkv, d, page, seed, layout="hnd", garbage=False):
    """(codes of K and V, scales of K and V, table, lengths); garbage: NaN codes and scales behind each last token."""
    g = torch.Generator().manual_seed(seed)
    table, n_pages = _tables(lens, page, g)
    (kc, ks), (vc, vs) = (_codes((n_pages, Hkv, page, d), layout, g) for _ in range(2))
    if garbage:
        keep, blocks = torch.zeros(n_pages, page, dtype=torch.bool), torch.zeros(n_pages, page // 16, dtype=torch.bool)
        for row, n in zip(table, lens):
            for j in range(n):
                keep[row[j // page], j % page] = True
                blocks[row[j // page], j % page // 16] = True
        for c, s in ((kc, ks), (vc, vs)):
            c.masked_fill_(~keep.cuda()[:, None, :, None], 0x7F)
            s.masked_fill_(~blocks.cuda()[:, None], float("nan"))
    return kc, vc, ks, vs, _ints(table), _ints(lens)


def _as_codes(c):
    return c.view(E4M3)


def _check(got, ref, bound, what):
    got = host_f64(got)
    assert np.array_equal(np.isneginf(got), np.isneginf(ref)), what
    fin = np.isfinite(ref)
    assert np.isfinite(got[fin]).all(), f"{what}: not finite"
    ratio = np.abs(got[fin] - ref[fin]) / np.maximum(bound[fin], 1e-300)
    assert ratio.size == 0 or ratio.max() <= 1.0, f"{what}: error {ratio.max():.3f} of its bound"
    return float(ratio.max(initial=0.0))


def _oracle(q, kc, vc, ks, vs, table, lens, d, cap, slopes, dtype):
    num = lambda t: t.cpu().numpy()
    clean = lambda s: np.nan_to_num(num(s).astype(np.float64))
    strip = lambda c: np.where(num(c) & 0x7F == 0x7F, 0, num(c))
    return paged_decode_fp8(host_f64(q), strip(kc), strip(vc), clean(ks), clean(vs), table.tolist(), lens, d ** -0.5, cap,
                            None if slopes is None else num(slopes), HALF[dtype])


# lens, H, Hkv, d, page, dtype, cap, bias
CASES = [
    ([1], 1, 1, 64, 16, torch.bfloat16, 0.0, False),
    ([0, 3, 0], 2, 1, 128, 16, torch.float16, 30.0, True),
    ([16, 17, 15, 1], 4, 4, 64, 16, torch.bfloat16, 0.0, True),
    ([127, 128, 129, 257], 6, 2, 128, 64, torch.bfloat16, 20.0, False),
    ([500, 0, 77, 1000, 5], 16, 2, 128, 32, torch.float16, 0.0, True),
    ([333, 2000], 24, 1, 64, 48, torch.bfloat16, 50.0, True),
    ([7000], 8, 8, 128, 128, torch.bfloat16, 0.0, False),
    ([4097], 40, 1, 64, 1024, torch.float16, 5.0, False),
    ([1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 300] * 3, 3, 3, 128, 16, torch.bfloat16, 0.0, False),
    ([2500, 2500, 0, 0, 1], 32, 16, 64, 256, torch.bfloat16, 0.0, True),
    ([901, 130], 17, 1, 128, 16, torch.bfloat16, 30.0, False),
    ([190, 40], 130, 1, 128, 16, torch.float16, 0.0, False),
]


def _decode(case, layout, garbage, seed=3):
    lens, H, Hkv, d, page, dtype, cap, bias = case
    kc, vc, ks, vs, table, n = _cache(lens, Hkv, d, page, seed, layout, garbage)
    g = torch.Generator().manual_seed(seed + 1)
    q = (torch.randn(len(lens), H, d, generator=g) * (3.0 if cap else 1.0)).to(dtype).cuda()
    slopes = _slopes(H) if bias else None
    o, lse = fa.fa_paged_decode_fp8(q, _as_codes(kc), _as_codes(vc), ks, vs, table, n, softcap=cap, slopes=slopes)
    fa.fa_sync_check()
    ref = _oracle(q, kc, vc, ks, vs, table, lens, d, cap, slopes, dtype)
    return _check(o, ref[0], ref[2], "O"), _check(lse, ref[1], ref[3], "LSE")


@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_decode(case, layout):
    o, lse = _decode(case, layout, False)
    report(f"decode fp8 {case} {layout} (shares of the bounds)", o=o, lse=lse)


@pytest.mark.parametrize("case", [([300, 0, 77, 129, 1], 10, 10, 64, 32, torch.bfloat16, 30.0, True),
                                  ([1000, 2001], 20, 4, 64, 16, torch.float16, 0.0, True),
                                  ([640, 5], 48, 6, 64, 128, torch.bfloat16, 0.0, False),
                                  ([901, 130, 0, 64, 65], 8, 2, 128, 16, torch.bfloat16, 20.0, False),
                                  ([3000, 63], 20, 4, 128, 1024, torch.float16, 0.0, True),
                                  ([333, 32, 33, 31], 32, 4, 128, 48, torch.bfloat16, 0.0, True),
                                  ([640, 5], 9, 3, 64, 48, torch.bfloat16, 0.0, True),
                                  ([200, 131], 36, 4, 64, 48, torch.float16, 20.0, False)], ids=str)
@pytest.mark.parametrize("garbage", [False, True])
def test_rows_of_two_heads(case, garbage):
    # Heads beside each other: two of them a unit where there are an even number and up to eight query heads each.
    _decode(case, "nhd", garbage)


@pytest.mark.parametrize("case", [([0, 300, 1, 17, 900, 0, 40, 16, 129, 31] * 20, 16, 2, 64, 16, torch.bfloat16, 0.0, True),
                                  ([5, 0, 700, 16, 130] * 10, 80, 4, 128, 64, torch.float16, 30.0, False)], ids=["3200", "4000"])
def test_many_heads(case):
    # More heads than blocks that join their parts: some whole, some in parts, some of empty sequences.
    _decode(case, "nhd", False)


@pytest.mark.parametrize("case", [CASES[2], CASES[3], CASES[4], CASES[5], CASES[7]], ids=str)
def test_what_lies_behind_the_last_token_does_not_matter(case):
    _decode(case, "nhd", True)


def test_page_indices_outside_the_cache_read_as_zeros():
    lens, H, Hkv, d, page = [100, 40, 16], 4, 2, 64, 16
    kc, vc, ks, vs, table, n = _cache(lens, Hkv, d, page, 5)
    table[0, 2], table[0, 3], table[1, 0], table[2, 0] = kc.shape[0], -1, 2 ** 31 - 1, -2 ** 31
    q = torch.randn(3, H, d, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).cuda()
    o, lse = fa.fa_paged_decode_fp8(q, _as_codes(kc), _as_codes(vc), ks, vs, table, n)
    fa.fa_sync_check()
    ref = _oracle(q, kc, vc, ks, vs, table, lens, d, 0.0, None, torch.bfloat16)
    _check(o, ref[0], ref[2], "O")
    _check(lse, ref[1], ref[3], "LSE")
    assert not o[2].any()  # zeros alone


def test_lengths_are_clamped_to_the_table():
    kc, vc, ks, vs, table, n = _cache([64, 64, 64], 2, 64, 16, 7)
    q = torch.randn(3, 4, 64, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).cuda()
    args = (q, _as_codes(kc), _as_codes(vc), ks, vs, table)
    want, want_l = fa.fa_paged_decode_fp8(*args, n)
    got, got_l = fa.fa_paged_decode_fp8(*args, _ints([2 ** 31 - 1, 64, -5]))
    fa.fa_sync_check()
    assert torch.equal(got[:2], want[:2]) and torch.equal(got_l[:2], want_l[:2])
    assert not got[2].any() and torch.isneginf(got_l[2]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_queries_and_scales_of_every_size(dtype):
    """Scores of ordinary size from huge queries and tiny keys, tiny and huge values: nothing overflows on the way."""
    lens, d = [150, 70], 128
    kc, vc, ks, vs, table, n = _cache(lens, 2, d, 16, 9)
    q = torch.randn(2, 4, d, generator=torch.Generator().manual_seed(1))
    big = 2.0 ** 100 if dtype == torch.bfloat16 else 2.0 ** 13
    q = (q * torch.tensor([big, 1 / big])[:, None, None]).to(dtype).cuda()
    # The second sequence's pages get the opposite sizes; a value's size changes from block to block by 2^+-40.
    pages = [table[b, :-(-m // 16)].long() for b, m in enumerate(lens)]
    ks[pages[0]] *= 1 / big
    ks[pages[1]] *= big
    vs[pages[0][::2]] *= 2.0 ** 40
    vs[pages[0][1::2]] *= 2.0 ** -40
    vs[pages[1]] *= 2.0 ** -60
    o, lse = fa.fa_paged_decode_fp8(q, _as_codes(kc), _as_codes(vc), ks, vs, table, n, o=None)
    fa.fa_sync_check()
    ref = _oracle(q, kc, vc, ks, vs, table, lens, d, 0.0, None, dtype)
    _check(lse, ref[1], ref[3], "LSE")
    if dtype == torch.bfloat16:  # (values of 2^40 and 2^-60 are none of fp16's)
        scale = np.array([1.0, 2.0 ** -60])[:, None, None]
        bound = (ref[2] - 2.0 ** -24) + 2.0 ** -24 * scale  # (the oracle's absolute term is meant for ordinary values)
        _check(o, ref[0], bound, "O")


def test_a_value_that_weighs_little_beside_a_large_scale():
    # The block with the largest V scale has next to no weight: the rest keeps its bits.
    d, n = 64, 32
    kc = torch.zeros(2, 1, 16, d, dtype=torch.uint8, device="cuda")
    vc = torch.full_like(kc, 0x38)  # 1.0
    kc[0] = 0xB8  # -1: scores of -80
    ks, vs = torch.ones(2, 1, 1, device="cuda"), torch.tensor([2.0 ** 30, 1.0], device="cuda").view(2, 1, 1)
    q = torch.full((1, 1, d), 10.0, dtype=torch.float16, device="cuda")
    o, lse = fa.fa_paged_decode_fp8(q, _as_codes(kc), _as_codes(vc), ks, vs, _ints([[0, 1]]), _ints([n]), scale=0.125)
    fa.fa_sync_check()
    w = np.exp(-80.0)
    want = (w * 2.0 ** 30 + 1) / (w + 1)
    assert abs(o.double().cpu() - want).max() <= 2.0 ** -10 and abs(lse.item() - np.log(16 * (1 + w))) < 1e-5


def test_a_weight_below_fp32_times_a_scale_far_above_the_others():
    # Weights of e^-88, below fp32's normal range, for values 2^120 times those of weight 1: their share is still 2^-7.
    d = 64
    kc = torch.zeros(2, 1, 16, d, dtype=torch.uint8, device="cuda")
    vc = torch.full_like(kc, 0x38)
    kc[0] = 0xB8
    ks = torch.ones(2, 1, 1, device="cuda")
    for order in ([0, 1], [1, 0]):
        vs = torch.tensor([2.0 ** 60, 2.0 ** -60], device="cuda").view(2, 1, 1)
        q = torch.full((1, 1, d), 11.0, dtype=torch.bfloat16, device="cuda")
        o, lse = fa.fa_paged_decode_fp8(q, _as_codes(kc), _as_codes(vc), ks, vs, _ints([order]), _ints([32]), scale=0.125)
        fa.fa_sync_check()
        w = np.exp(-88.0)
        want = (w * 2.0 ** 60 + 2.0 ** -60) / (1 + w)
        assert abs(want * 2.0 ** 60 - 1.008) < 1e-3
        assert (o.double().cpu() / want - 1).abs().max() <= 2.0 ** -8 and abs(lse.item() - np.log(16)) < 1e-5


def test_nan_stays_in_its_sequence_and_head():
    lens = [40, 40]
    kc, vc, ks, vs, table, n = _cache(lens, 2, 64, 16, 11)
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(2)).half().cuda()
    want, want_l = fa.fa_paged_decode_fp8(q, _as_codes(kc), _as_codes(vc), ks, vs, table, n)
    kc[table[0, 1].long(), 1, 3, 5] = 0x7F
    vc[table[1, 0].long(), 0, 15, 7] = 0xFF
    o, lse = fa.fa_paged_decode_fp8(q, _as_codes(kc), _as_codes(vc), ks, vs, table, n)
    fa.fa_sync_check()
    assert o[0, 2:].isnan().all() and lse[0, 2:].isnan().all()
    assert torch.equal(o[0, :2], want[0, :2]) and torch.equal(o[1, 2:], want[1, 2:])
    assert o[1, :2, 7].isnan().all() and torch.equal(lse[1], want_l[1])
    assert torch.equal(o[1, :2, :7], want[1, :2, :7]) and torch.equal(o[1, :2, 8:], want[1, :2, 8:])


def test_views_of_q_o_and_the_table():
    lens = [70, 33]
    kc, vc, ks, vs, table, n = _cache(lens, 2, 128, 16, 9)
    cache = (_as_codes(kc), _as_codes(vc), ks, vs)
    q = torch.randn(2, 4, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    want, want_l = fa.fa_paged_decode_fp8(q, *cache, table, n)
    qkv = torch.zeros(2, 3, 4, 136, dtype=torch.bfloat16, device="cuda")
    qkv[:, 1, :, :128] = q
    wide = torch.full((2, table.shape[1] + 3), 77, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    obuf = torch.full((2, 5, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    o, lse = fa.fa_paged_decode_fp8(qkv[:, 1, :, :128], *cache, wide[:, :table.shape[1]], n, o=obuf[:, :4])
    fa.fa_sync_check()
    assert torch.equal(o, want) and torch.equal(lse, want_l) and bool((obuf[:, 4] == 9).all())


def test_captured_decode_replays_with_new_lengths():
    kc, vc, ks, vs, table, n = _cache([400, 400, 400], 2, 64, 32, 11)
    q = torch.randn(3, 8, 64, generator=torch.Generator().manual_seed(2)).to(torch.float16).cuda()
    ws = torch.empty(fa.fa_paged_decode_workspace_size(3, 8, 2, 64), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(3, 8, device="cuda")
    call = lambda: fa.fa_paged_decode_fp8(q, _as_codes(kc), _as_codes(vc), ks, vs, table, n, o=o, lse=lse, workspace=ws)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens in ([1, 400, 0], [399, 0, 64]):
        n.copy_(torch.tensor(lens))
        ws.fill_(0xFF)  # the workspace's contents on entry do not matter
        g.replay()
        fa.fa_sync_check()
        ref = _oracle(q, kc, vc, ks, vs, table, lens, 64, 0.0, None, torch.float16)
        _check(o, ref[0], ref[2], "O")
        _check(lse, ref[1], ref[3], "LSE")


def test_two_decodes_at_once():
    sets = [_cache([700, 30], 2, 128, 16, 20 + s) for s in range(2)]
    qs = [torch.randn(2, 16, 128, generator=torch.Generator().manual_seed(s)).to(torch.bfloat16).cuda() for s in range(2)]
    call = lambda q, c: fa.fa_paged_decode_fp8(q, _as_codes(c[0]), _as_codes(c[1]), *c[2:])
    want = [call(q, c) for q, c in zip(qs, sets)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(10):
        got = []
        for q, c, s in zip(qs, sets, streams):
            with torch.cuda.stream(s):
                got.append(call(q, c))
        torch.cuda.synchronize()
        for (a, b), (x, y) in zip(want, got):
            assert torch.equal(a, x) and torch.equal(b, y)


def test_more_sequences_than_threads_of_a_block():
    _decode(([(7 * b) % 61 for b in range(700)], 4, 2, 64, 16, torch.bfloat16, 0.0, True), "nhd", False)


def test_cache_past_32_bit_offsets():
    Hkv, page, d = 1, 16, 64
    stride = 1 << 31
    view = lambda t: t.as_strided((3, Hkv, page, d), (stride, page * d, d, 1))
    kc, vc = (view(torch.empty(2 * stride + Hkv * page * d, dtype=torch.uint8, device="cuda")) for _ in range(2))
    kc.fill_(0)
    vc.fill_(0)
    ks, vs = torch.zeros(3, 1, 1, device="cuda"), torch.zeros(3, 1, 1, device="cuda")
    table, n = _ints([[2, 0]]), _ints([20])
    x = torch.randn(20, 2, d, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
    fa.fa_paged_append_fp8(x[:, :1], x[:, 1:], _as_codes(kc), _as_codes(vc), ks, vs, table, n, _ints([0, 20]))
    q = torch.randn(1, 2, d, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).cuda()
    o, lse = fa.fa_paged_decode_fp8(q, _as_codes(kc), _as_codes(vc), ks, vs, table, n)
    fa.fa_sync_check()
    ref = _oracle(q, kc, vc, ks, vs, table, [20], d, 0.0, None, torch.bfloat16)
    _check(o, ref[0], ref[2], "O")
    _check(lse, ref[1], ref[3], "LSE")
    err = np.abs(host_f64(x[:16, 0]) - e4m3_decode(kc[2, 0].cpu().numpy()) * ks[2, 0, 0].item())
    assert (err <= np.maximum(2.0 ** -4 * np.abs(host_f64(x[:16, 0])), 2.0 ** -10 * ks[2, 0, 0].item())).all()


# ------------------------------------------------------------------------- appending


def _append(new, before, Hkv, d, page, dtype, layout, seed=2, tail=0, factor=None):
    """One call against the oracle, bit by bit; returns the cache."""
    g = torch.Generator().manual_seed(seed)
    lens = [a + b for a, b in zip(new, before)]
    table, n_pages = _tables(lens, page, g)
    (kc, ks), (vc, vs) = (_codes((n_pages, Hkv, page, d), layout, g) for _ in range(2))
    ks, vs = (torch.exp2(torch.randint(-9, -5, s.shape, generator=g).float()).cuda() for s in (ks, vs))
    T = sum(new) + tail
    x = torch.randn(T, 2 * Hkv, d, generator=g)
    x = (x * (torch.exp2(2 * torch.randn(T, 2 * Hkv, 1, generator=g)) if factor is None else factor)).to(dtype).cuda()
    k, v = x[:, :Hkv], x[:, Hkv:]  # views of one projection
    cu = np.concatenate([[0], np.cumsum(new)])
    want = [paged_append_fp8(host_f64(t), c.cpu().numpy(), s.cpu().numpy(), table, lens, cu) for t, c, s in ((k, kc, ks), (v, vc, vs))]
    fa.fa_paged_append_fp8(k, v, _as_codes(kc), _as_codes(vc), ks, vs, _ints(table), _ints(lens), _ints(cu.tolist()))
    fa.fa_sync_check()
    for c, s, (wc, ws) in zip((kc, vc), (ks, vs), want):
        assert np.array_equal(host_f64(s), ws)
        assert np.array_equal(c.cpu().numpy(), wc)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("new,before", [([1, 1, 1], [0, 16, 41]), ([0, 37, 5, 64], [3, 11, 0, 16]), ([100], [0]), ([0, 0, 1], [0, 5, 31]),
                                        ([15, 17, 16], [1, 14, 15])])
def test_append(new, before, layout, dtype):
    _append(new, before, 3, 64, 32, dtype, layout, tail=2)
    _append(new, before, 2, 128, 48, dtype, layout, tail=1, seed=4)


@pytest.mark.parametrize("factor", [0.0, 2.0 ** -130, 2.0 ** 100])
def test_append_of_extreme_sizes(factor):
    _append([20, 3], [5, 16], 2, 64, 16, torch.bfloat16, "hnd", factor=factor)


@pytest.mark.parametrize("Hkv,d", [(1, 64), (5, 128)])
def test_append_of_many_tokens(Hkv, d):
    # Enough that a warp takes runs of 16 rows; sequences and blocks end inside the runs.
    _append([9001, 0, 1, 777, 1, 1, 1, 20, 3], [3, 0, 31, 16, 7, 0, 15, 9, 2], Hkv, d, 48, torch.bfloat16, "hnd", tail=5)


def test_append_of_many_single_tokens():
    _append([1] * 2000, [(5 * b) % 40 for b in range(2000)], 3, 64, 16, torch.float16, "nhd")


def test_append_skips_what_has_no_place():
    Hkv, d, page = 1, 64, 16
    kc, vc = (torch.zeros(3, Hkv, page, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((3, Hkv, 1), 2.0 ** -8, device="cuda") for _ in range(2))
    table, lens, cu = [[0, 9], [1, -4], [2, 2]], [18, 2, 40], [0, 4, 9, 13]
    x = torch.arange(1, 14, dtype=torch.float32)[:, None, None].expand(13, 1, d).contiguous().to(torch.bfloat16).cuda()
    want = paged_append_fp8(host_f64(x), kc.cpu().numpy(), ks.cpu().numpy(), table, lens, cu)
    fa.fa_paged_append_fp8(x, x, _as_codes(kc), _as_codes(vc), ks, vs, _ints(table), _ints(lens), _ints(cu))
    fa.fa_sync_check()
    for c, s in ((kc, ks), (vc, vs)):
        assert np.array_equal(c.cpu().numpy(), want[0]) and np.array_equal(host_f64(s), want[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_append_of_infinities_and_nan(dtype):
    x = torch.ones(5, 2, 64, dtype=dtype)
    x[1, 0, 3], x[2, 0, 4], x[3, 0, 5] = float("inf"), float("-inf"), float("nan")
    x[:, 1] = float("inf")
    x = x.cuda()
    kc, vc = (torch.zeros(1, 2, 16, 64, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(1, 2, 1, device="cuda") for _ in range(2))
    fa.fa_paged_append_fp8(x, x, _as_codes(kc), _as_codes(vc), ks, vs, _ints([[0]]), _ints([5]), _ints([0, 5]))
    fa.fa_sync_check()
    vals = e4m3_decode(kc[0, 0, :5].cpu().numpy())
    assert ks[0, 0, 0].item() == 2.0 ** -8 and vals[1, 3] == 448 and vals[2, 4] == -448 and np.isnan(vals[3, 5])
    assert (np.delete(vals.ravel(), [64 + 3, 128 + 4, 192 + 5]) == 256).all()
    assert ks[0, 1, 0].item() == 2.0 ** -126 and (e4m3_decode(kc[0, 1, :5].cpu().numpy()) == 448).all()
    assert torch.equal(kc, vc) and torch.equal(ks, vs)


# ----------------------------------------------------------------------- bookkeeping


def _resize(lens, delta, page, width, spare, rows, in_place, seed=1, capacity=None):
    g = np.random.default_rng(seed)
    pages = lambda n: -(-n // page)
    used = sum(pages(max(n, 0)) for n in lens)
    order = g.permutation(used + spare).tolist()
    table, at = [], 0
    for n in lens:
        m = min(pages(max(n, 0)), width)
        table.append((order[at:at + m] + [-1] * width)[:width])
        at += m
    free = order[used:] + [-7] * (used + 3 if capacity is None else capacity - spare)
    want = paged_resize(table, lens, delta, free, spare, page, rows)
    t = torch.full((max(len(lens), 1), width + 2), 55, dtype=torch.int32, device="cuda")
    t[:len(lens), :width] = torch.tensor(table, dtype=torch.int32).view(len(lens), width)
    view = t[:len(lens), :width]
    n, d, f, c = _ints(lens), _ints(delta), _ints(free), _ints([spare])
    slots, pos = torch.full((rows,), 5, dtype=torch.int64, device="cuda"), torch.full((rows,), 5, dtype=torch.int32, device="cuda")
    kw = dict(seq_lens_out=n, free_count_out=c) if in_place else {}
    out = fa.fa_paged_resize(view, n, d, f, c, page, slots=slots, positions=pos, **kw)
    fa.fa_sync_check()
    got = (out[0], out[1], out[2], out[3], view, f, slots, pos)
    names = "lens cu count status table free slots positions".split()
    for name, x, y in zip(names, got, want):
        y = [y] if name == "count" else y
        assert np.array_equal(x.cpu().numpy().ravel(), np.array(y, dtype=np.int64).ravel()), name
    assert bool((t[:, width:] == 55).all())
    if not in_place:
        assert n.tolist() == lens and c.item() == spare


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens,delta,page,width,spare,rows", [
    ([], [], 16, 4, 3, 5),
    ([0], [1], 16, 1, 1, 1),
    ([16], [0], 16, 1, 0, 0),
    ([20, 32, 15], [-4, -32, 20], 16, 4, 2, 22),
    ([10, 10], [30, -10], 16, 4, 1, 40),       # the page that comes back is taken in the same call
    ([10, 10], [60, 0], 16, 4, 2, 7),          # pages missing
    ([10, 60], [1, 10], 16, 4, 9, 12),         # past the table
    ([10, 5], [1, -6], 16, 4, 9, 3),           # a negative length
    ([-3, 5], [1, 1], 16, 4, 9, 3),
    ([70, 5], [-10, 1], 16, 4, 9, 3),          # a length that the table never held
    ([5, 5, 5], [40, 40, 40], 48, 3, 9, 60),   # fewer rows asked for than there are new tokens
])
def test_resize(lens, delta, page, width, spare, rows, in_place):
    _resize(lens, delta, page, width, spare, rows, in_place)


def test_resize_of_a_list_without_room():
    _resize([40, 3], [-40, 0], 16, 4, 2, 4, False, capacity=4)


@pytest.mark.parametrize("B,seed", [(33, 1), (700, 2), (1500, 3), (5000, 4)])
def test_resize_of_many(B, seed):
    g = np.random.default_rng(seed)
    lens = g.integers(0, 400, B).tolist()
    delta = [int(g.integers(-n, 1)) if g.random() < 0.4 else int(g.integers(0, 300)) for n in lens]
    new = sum(x for x in delta if x > 0)
    _resize(lens, delta, 16, 50, 20 * B, new + 77, bool(seed % 2), seed)
    _resize(lens, delta, 16, 50, 0, new, False, seed)


@pytest.mark.parametrize("rows", [700, 3000, 400000])  # one block; over the GPU, some rows a warp and many
@pytest.mark.parametrize("B,every,by", [(256, 1, 1), (250, 40, 33), (1000, 1, 1), (1000, 333, 200), (400, 399, 1), (300, 2, -1)])
def test_resize_with_idle_sequences(B, every, by, rows):
    # Rows, and pages, of neighbours far apart, or of many sequences.
    lens = [(7 * i) % 90 for i in range(B)]
    delta = [0 if i % every else by if by > 0 else -lens[i] for i in range(B)]
    _resize(lens, delta, 16, 32, 15 * B, rows, False, B)


def test_captured_resize():
    # In place, replayed: every sequence one token longer each time, from the device's own numbers.
    B, page, width = 5, 16, 6
    lens = [0, 15, 16, 3, 31]
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free, count, n, delta = _ints(list(range(40))), _ints([40]), _ints([0] * B), _ints(lens)
    slots, pos = torch.empty(B, dtype=torch.int64, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    cu, status = _ints([0] * (B + 1)), _ints([0, 0])
    ws = torch.empty(fa.fa_paged_resize_workspace_size(B), dtype=torch.uint8, device="cuda")
    call = lambda: fa.fa_paged_resize(table, n, delta, free, count, page, slots=slots, positions=pos, seq_lens_out=n,
                                      free_count_out=count, cu_new=cu, status=status, workspace=ws)
    ref = paged_resize(table.tolist(), [0] * B, lens, free.tolist(), 40, page, B)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    delta.fill_(1)
    for _ in range(20):
        ref = paged_resize(ref[4], ref[0], [1] * B, ref[5], ref[2], page, B)
        graph.replay()
        fa.fa_sync_check()
        for x, y in zip((n, cu, count, status, table, free, slots, pos), ref):
            assert np.array_equal(x.cpu().numpy().ravel(), np.array(y).ravel())


# --------------------------------------------------------------------- all together


def test_a_server_loop():
    """As a model serves: prompts come in, tokens follow, a sequence ends and another takes its place; every step
    resizes, turns queries and keys by the new positions, appends and attends."""
    H, Hkv, d, page, width, pages, cap = 8, 2, 128, 16, 10, 24, 30.0
    B, g = 3, torch.Generator().manual_seed(4)
    kc, vc = (torch.full((pages, Hkv, page, d), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((pages, Hkv, 1), float("nan"), device="cuda") for _ in range(2))
    table, lens = torch.full((B, width), -1, dtype=torch.int32, device="cuda"), _ints([0] * B)
    free, count = torch.randperm(pages, generator=g).to(torch.int32).cuda(), _ints([pages])
    f = torch.tensor([1e4 ** (-i / d) for i in range(0, d, 2)], dtype=torch.float32, device="cuda")
    qw, kw = ((1 + 0.2 * torch.randn(d, generator=g)).cuda() for _ in range(2))
    history = [[] for _ in range(B)]
    for delta in ([37, 1, 90], [1, 1, 1], [1, 1, 1], [1, 1, -92], [1, 1, 50], [1, 1, 1], [-3, 1, 1], [1, 1, 1]):
        T = sum(max(x, 0) for x in delta)
        pos, slots = torch.empty(T + 2, dtype=torch.int32, device="cuda"), torch.empty(T + 2, dtype=torch.int64, device="cuda")
        _, cu, _, status = fa.fa_paged_resize(table, lens, _ints(delta), free, count, page, slots=slots, positions=pos,
                                              seq_lens_out=lens, free_count_out=count)
        qkv = torch.randn(T + 2, H + 2 * Hkv, d, generator=g).bfloat16().cuda()  # two rows of padding
        x = qkv.transpose(0, 1)[None]
        q, k = fa.fa_qk_norm_rope(x[:, :H], x[:, H:H + Hkv], qw, kw, f, pos[None])
        q, k, v = q[0].transpose(0, 1), k[0].transpose(0, 1), qkv[:, H + Hkv:]
        fa.fa_paged_append_fp8(k, v, _as_codes(kc), _as_codes(vc), ks, vs, table, lens, cu)
        at = cu.tolist()
        assert status.tolist() == [0, 0] and at[-1] == T and (pos[T:] == -1).all()
        for b in range(B):
            if delta[b] < 0:
                history[b] = history[b][:len(history[b]) + delta[b]]
            for t in range(at[b], at[b + 1]):
                history[b].append((q[t], k[t], v[t]))
                assert slots[t] == int(table[b, pos[t] // page]) * page + int(pos[t]) % page
        assert lens.tolist() == [len(h) for h in history]
        last = torch.stack([h[-1][0] if h else torch.zeros_like(q[0]) for h in history])
        o, lse = fa.fa_paged_decode_fp8(last, _as_codes(kc), _as_codes(vc), ks, vs, table, lens, softcap=cap)
        fa.fa_sync_check()
        ref = _oracle(last, kc, vc, ks, vs, table.clamp(min=0), lens.tolist(), d, cap, None, torch.bfloat16)
        _check(o, ref[0], ref[2], "O")
        _check(lse, ref[1], ref[3], "LSE")
        for b, h in enumerate(history):
            if not h:
                assert not o[b].any()
                continue
            if len(h) == 1:  # its only value: e4m3's rounding, 2^-4 of it, or half the smallest code's step of a scale <= 2^-5
                v = np.repeat(host_f64(h[0][2]), H // Hkv, 0)
                assert (np.abs(host_f64(o[b]) - v) <= 1.1 * 2.0 ** -4 * np.abs(v) + 2.0 ** -15).all()
    assert sorted(free[:count.item()].tolist() + [p for b in range(B) for p in table[b, :-(-lens[b].item() // page)].tolist()]) == list(range(pages))


def test_refusals_in_the_binding():
    kc, vc, ks, vs, table, n = _cache([40], 2, 64, 16, 1)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    c = (_as_codes(kc), _as_codes(vc))
    with pytest.raises(TypeError):
        fa.fa_paged_decode_fp8(q, kc, vc, ks, vs, table, n)  # bytes, not e4m3
    with pytest.raises(TypeError):
        fa.fa_paged_decode_fp8(q.float(), *c, ks, vs, table, n)
    with pytest.raises(ValueError):
        fa.fa_paged_decode_fp8(q, *c, ks[:, :1], vs, table, n)
    with pytest.raises(ValueError):
        fa.fa_paged_decode_fp8(q, *c, ks.half(), vs, table, n)
    with pytest.raises(TypeError):
        fa.fa_paged_decode_fp8(q, *c, None, vs, table, n)
    with pytest.raises(TypeError):
        fa.fa_paged_decode(q, *c, table, n)  # the 16-bit call
    with pytest.raises(fa.FAError):
        fa.fa_paged_decode_fp8(q[:, :3].contiguous(), *c, ks, vs, table, n)
    with pytest.raises(fa.FAError):  # rows of 72 codes: not on 16 bytes
        wide = torch.zeros(kc.shape[0], 2, 16, 72, dtype=torch.uint8, device="cuda")[..., :64].view(E4M3)
        fa.fa_paged_decode_fp8(q, wide, wide, ks, vs, table, n)
    k = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError):
        fa.fa_paged_append_fp8(k, k.half(), *c, ks, vs, table, n, _ints([0, 1]))
    with pytest.raises(ValueError):
        fa.fa_paged_append_fp8(k, k, *c, ks, vs, table, n, _ints([0, 1, 1]))
    f, cnt, delta = _ints([1, 2]), _ints([2]), _ints([1])
    with pytest.raises(ValueError):
        fa.fa_paged_resize(table, n, delta.long(), f, cnt, 16)
    with pytest.raises(ValueError):
        fa.fa_paged_resize(table, n, _ints([1, 1]), f, cnt, 16)
    with pytest.raises(ValueError):
        fa.fa_paged_resize(table, n, delta, f, cnt, 16, slots=torch.zeros(3, dtype=torch.int64, device="cuda"), positions=_ints([0, 0]))
    with pytest.raises(TypeError):
        fa.fa_paged_resize(table, n, delta, f, None, 16)
    with pytest.raises(fa.FAError):
        fa.fa_paged_resize(table, n, delta, f, cnt, 8)
    with pytest.raises(fa.FAError):
        fa.fa_paged_resize(table, n, delta, f, cnt, 16, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))


def _append_behind(codes, scale, new):
    """(codes, scales) of one block of 16 tokens of one head of 64: `codes` of its first tokens at `scale`, then `new` appended."""
    held, T = codes.shape[0], new.shape[0]
    cache = torch.full((1, 1, 16, 64), 0x55, dtype=torch.uint8)
    cache[0, 0, :held] = codes
    kc, vc = cache.cuda(), cache.cuda()
    ks, vs = (torch.tensor([[[scale]]], dtype=torch.float32, device="cuda") for _ in range(2))
    x = new[:, None].to(torch.bfloat16).cuda()
    fa.fa_paged_append_fp8(x, x, _as_codes(kc), _as_codes(vc), ks, vs, _ints([[0]]), _ints([held + T]), _ints([0, T]))
    fa.fa_sync_check()
    assert torch.equal(kc, vc) and torch.equal(ks, vs)
    want = paged_append_fp8(host_f64(x), cache.numpy(), np.array([[[scale]]], np.float32), [[0]], [held + T], [0, T])
    return kc.cpu().numpy(), host_f64(ks), want


@pytest.mark.parametrize("scale", [2.0 ** 126, 1.3 * 2.0 ** 126, 2.0 ** 127, 1.5 * 2.0 ** 125, 2.0 ** -126, 1.25 * 2.0 ** -126, 1.5 * 2.0 ** -127])
def test_append_behind_the_largest_and_smallest_scales(scale):
    g = torch.Generator().manual_seed(5)
    codes = torch.randint(0, 0x7F, (5, 64), generator=g, dtype=torch.uint8)
    got, scales, want = _append_behind(codes, scale, min(scale, 1.0) * torch.randn(3, 64, generator=g))
    assert np.array_equal(scales, want[1]) and np.array_equal(got, want[0])


def test_append_behind_a_scale_that_no_power_of_two_reaches():
    # 2^127 is the largest there is: codes grow by what the scale loses, up to the largest code.
    codes = torch.arange(0, 0x7F, dtype=torch.uint8)[:64].repeat(2, 1)
    codes[1] += 0x3F
    got, scales, _ = _append_behind(codes, 1.5 * 2.0 ** 127, torch.ones(1, 64))
    assert scales.item() == 2.0 ** 127 and np.array_equal(got[0, 0, :2], e4m3_encode(1.5 * e4m3_decode(codes.numpy())))
    assert not e4m3_decode(got[0, 0, 2]).any()  # 1 beside 2^127


def test_recoding_rounds_the_exact_product():
    # Scales s in (1/2, 1) whose product with a code's value lies next to the middle between two codes, nearer than fp32
    # tells: the scale becomes 1 and the code that of the exact product.
    values = e4m3_decode(np.arange(0x7F, dtype=np.uint8))
    middles = (values[1:] + values[:-1]) / 2
    tried = 0
    for p in (0x39, 0x3B, 0x3D, 0x45):  # 1.125, 1.375, 1.625, 3.25
        v = values[p]
        for m in middles[(middles > v / 2) & (middles < v)]:
            s = float(np.float32(m / v))
            if s * v == m or float(np.float32(s * v)) != m or e4m3_encode(s * v) == e4m3_encode(m):
                continue
            tried += 1
            codes = torch.full((2, 64), p, dtype=torch.uint8)
            codes[1] |= 0x80
            got, scales, want = _append_behind(codes, s, torch.ones(1, 64))
            assert scales.item() == 1.0 and np.array_equal(got, want[0]), (p, m)
    assert tried >= 4


@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("size", [1.0, 16.0])  # new tokens below the scales, and above some
def test_append_behind_scales_that_are_no_powers_of_two(size, layout):
    g = torch.Generator().manual_seed(12)
    new, before, Hkv, d, page = [1, 20, 0, 5, 40], [3, 31, 7, 12, 17], 2, 64, 32
    lens = [a + b for a, b in zip(new, before)]
    table, n_pages = _tables(lens, page, g)
    (kc, ks), (vc, vs) = (_codes((n_pages, Hkv, page, d), layout, g) for _ in range(2))
    x = (size * torch.randn(sum(new), 2 * Hkv, d, generator=g)).to(torch.bfloat16).cuda()
    k, v = x[:, :Hkv], x[:, Hkv:]
    cu = np.concatenate([[0], np.cumsum(new)])
    want = [paged_append_fp8(host_f64(t), c.cpu().numpy(), s.cpu().numpy(), table, lens, cu) for t, c, s in ((k, kc, ks), (v, vc, vs))]
    fa.fa_paged_append_fp8(k, v, _as_codes(kc), _as_codes(vc), ks, vs, _ints(table), _ints(lens), _ints(cu.tolist()))
    fa.fa_sync_check()
    for c, s, (wc, ws) in zip((kc, vc), (ks, vs), want):
        assert np.array_equal(host_f64(s), ws) and np.array_equal(c.cpu().numpy(), wc)


@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("H,Hkv,d", [(2, 2, 64), (3, 1, 128), (14, 2, 64), (16, 2, 128), (21, 3, 64), (9, 1, 64), (16, 1, 64), (17, 1, 64),
                                     (22, 2, 128), (40, 1, 128)])
def test_decode_in_the_workspace_that_it_asks_for(H, Hkv, d, layout):
    # Of every build: parts of as many rows as a unit has heads, none written past the workspace's end.
    lens = [5000, 0, 700, 1, 9000]
    kc, vc, ks, vs, table, n = _cache(lens, Hkv, d, 16, 43, layout)
    q = torch.randn(5, H, d, generator=torch.Generator().manual_seed(44)).to(torch.bfloat16).cuda()
    size = fa.fa_paged_decode_workspace_size(5, H, Hkv, d)
    buf = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    o, lse = fa.fa_paged_decode_fp8(q, _as_codes(kc), _as_codes(vc), ks, vs, table, n, workspace=buf[:size])
    fa.fa_sync_check()
    ref = _oracle(q, kc, vc, ks, vs, table, lens, d, 0.0, None, torch.bfloat16)
    _check(o, ref[0], ref[2], "O")
    _check(lse, ref[1], ref[3], "LSE")
    assert bool((buf[size:] == 0xA5).all())
    with pytest.raises(fa.FAError):
        fa.fa_paged_decode_fp8(q, _as_codes(kc), _as_codes(vc), ks, vs, table, n, workspace=buf[:size - 1])


@pytest.mark.parametrize("B", [40, 700])  # one block; over the GPU
@pytest.mark.parametrize("which", ["slots", "positions", "neither"])
def test_resize_without_slots_or_positions(B, which):
    lens = [(7 * i) % 90 for i in range(B)]
    delta = [(11 * i) % 60 - min(lens[i], 20) for i in range(B)]
    new = sum(x for x in delta if x > 0)
    page, width, spare = 16, 12, 6 * B
    used = sum(-(-n // page) for n in lens)
    order = torch.randperm(used + spare, generator=torch.Generator().manual_seed(B)).tolist()
    table, at = [], 0
    for n in lens:
        m = -(-n // page)
        table.append((order[at:at + m] + [-1] * width)[:width])
        at += m
    free = order[used:] + [-7] * used
    want = paged_resize(table, lens, delta, free, spare, page, new + 3)
    t, n, d, f, c = _ints(table), _ints(lens), _ints(delta), _ints(free), _ints([spare])
    slots, pos = torch.full((new + 3,), 5, dtype=torch.int64, device="cuda"), torch.full((new + 3,), 5, dtype=torch.int32, device="cuda")
    kw = dict(slots=dict(slots=slots), positions=dict(positions=pos), neither={})[which]
    out = fa.fa_paged_resize(t, n, d, f, c, page, **kw)
    fa.fa_sync_check()
    got = dict(zip("lens cu count status table free".split(), (*out, t, f)))
    for name, x, y in zip(got, got.values(), want):
        assert np.array_equal(x.cpu().numpy().ravel(), np.array([y] if name == "count" else y, dtype=np.int64).ravel()), name
    assert slots.tolist() == (want[6] if which == "slots" else [5] * (new + 3))
    assert pos.tolist() == (want[7] if which == "positions" else [5] * (new + 3))


def test_two_graphs_share_a_workspace():
    # Captured for two batches of other sizes over one workspace and replayed in turn on one stream; one's units are of two heads.
    kc, vc, ks, vs, table, n = _cache([700, 90, 333], 2, 64, 16, 25, "nhd")
    kd, vd = (t.contiguous() for t in (kc, vc))
    q = torch.randn(3, 16, 64, generator=torch.Generator().manual_seed(26)).to(torch.bfloat16).cuda()
    ws = torch.empty(fa.fa_paged_decode_workspace_size(3, 16, 2, 64), dtype=torch.uint8, device="cuda")
    runs = [lambda o, l, w: fa.fa_paged_decode_fp8(q, _as_codes(kc), _as_codes(vc), ks, vs, table, n, o=o, lse=l, workspace=w),
            lambda o, l, w: fa.fa_paged_decode_fp8(q[:1], _as_codes(kd), _as_codes(vd), ks, vs, table[:1], n[:1], o=o, lse=l, workspace=w)]
    want = [run(None, None, None) for run in runs]
    outs = [(torch.zeros_like(o), torch.zeros_like(l)) for o, l in want]
    graphs = []
    for run, out in zip(runs, outs):
        run(*out, ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(*out, ws)
        graphs.append(graph)
    for turn in (0, 1, 1, 0):
        for t in outs[turn]:
            t.fill_(7)
        graphs[turn].replay()
        for a, b in zip(outs[turn], want[turn]):
            assert torch.equal(a, b)
    fa.fa_sync_check()


@pytest.mark.parametrize("n", [5, 200, 5000])
def test_the_largest_values_that_the_sums_take(n):
    # 448 times the scale just below 2^122 / n: their weighted mean is itself.
    d = 64
    e = int(np.floor(113.1 - np.log2(n)))  # log2(448) = 8.81
    pages = -(-n // 16)
    kc = torch.randint(0, 0x50, (pages, 2, 16, d), generator=torch.Generator().manual_seed(3), dtype=torch.uint8).cuda()
    vc = torch.full_like(kc, 0x7E)
    ks, vs = torch.full((pages, 2, 1), 0.02, device="cuda"), torch.full((pages, 2, 1), 2.0 ** e, device="cuda")
    q = torch.randn(1, 6, d, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    o, _ = fa.fa_paged_decode_fp8(q, _as_codes(kc), _as_codes(vc), ks, vs, torch.arange(pages, dtype=torch.int32, device="cuda")[None], _ints([n]))
    fa.fa_sync_check()
    # The weights' fp16 rounding (2^-11) in the sum alone, fp32's few steps, and bf16's of the result.
    assert float((o.double() / (448 * 2.0 ** e) - 1).abs().max()) <= 2.0 ** -8 + 1.1 * 2.0 ** -11


@pytest.mark.parametrize("B", [300, 2500])
def test_append_with_idle_sequences_inside_a_run(B):
    # A warp's run of tokens ends one sequence and begins another far behind it.
    new, before = [0] * B, [(3 * b) % 50 for b in range(B)]
    new[0], new[B // 2], new[B // 2 + 1], new[B - 1] = 4001, 7, 1, 3999
    _append(new, before, 2, 64, 64, torch.bfloat16, "hnd", tail=3)
