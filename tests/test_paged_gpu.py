"""The paged cache on the GPU: appending and one-token attention against the float64 oracle."""

import numpy as np
import pytest
import torch

import io_aware_exact_fwd_gb300 as fa
from oracle import paged_append, paged_decode, scored_forward

from gpu_util import host_f64, report

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fa.load_library()
    fa.fa_debug_set_wait_limit_ns(0)


def _slopes(H):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=torch.float32, device="cuda")


def _cache(lens, Hkv, d, page, dtype, seed, layout="nhd", fill=None):
    """A cache whose pages are shuffled; what lies behind each sequence's last token is `fill`."""
    g = torch.Generator().manual_seed(seed)
    need = [max(0, -(-n // page)) for n in lens]
    n_pages, width = sum(need) + 2, max(1, max(need))
    order = torch.randperm(n_pages, generator=g)[:sum(need)].tolist()
    table, at = [], 0
    for n in need:
        table.append(order[at:at + n] + [n_pages + 5] * (width - n))  # unused entries: outside the cache
        at += n
    shape = (n_pages, page, Hkv, d) if layout == "nhd" else (n_pages, Hkv, page, d)
    kc, vc = (torch.randn(shape, generator=g).to(dtype) for _ in range(2))
    if layout == "nhd":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    if fill is not None:
        keep = torch.zeros(n_pages, page, dtype=torch.bool)
        for row, n in zip(table, lens):
            for j in range(n):
                keep[row[j // page], j % page] = True
        for c in (kc, vc):
            c.masked_fill_(~keep[:, None, :, None], fill)
    cuda = lambda t: t.cuda() if layout != "nhd" else t.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    return cuda(kc), cuda(vc), torch.tensor(table, dtype=torch.int32).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()


def _check(got, ref, bound, what):
    got = host_f64(got)
    assert np.array_equal(np.isneginf(got), np.isneginf(ref)), what
    fin = np.isfinite(ref)
    assert np.isfinite(got[fin]).all(), f"{what}: not finite"
    ratio = np.abs(got[fin] - ref[fin]) / np.maximum(bound[fin], 1e-300)
    assert ratio.size == 0 or ratio.max() <= 1.0, f"{what}: error {ratio.max():.3f} of its bound"
    return float(ratio.max(initial=0.0))


# lens, H, Hkv, d, page, dtype, cap, bias
CASES = [
    ([1], 1, 1, 64, 16, torch.bfloat16, 0.0, False),
    ([0, 3, 0], 2, 1, 128, 16, torch.float16, 30.0, True),
    ([16, 17, 15, 1], 4, 4, 64, 16, torch.bfloat16, 0.0, True),
    ([63, 64, 65, 129], 6, 2, 128, 64, torch.bfloat16, 20.0, False),
    ([500, 0, 77, 1000, 5], 16, 2, 128, 32, torch.float16, 0.0, True),
    ([333, 2000], 24, 1, 64, 48, torch.bfloat16, 50.0, True),
    ([7000], 8, 8, 128, 128, torch.bfloat16, 0.0, False),
    ([4097], 40, 1, 64, 1024, torch.float16, 5.0, False),
    ([1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 300] * 3, 3, 3, 128, 16, torch.bfloat16, 0.0, False),
    ([2500, 2500, 0, 0, 1], 32, 16, 64, 256, torch.bfloat16, 0.0, True),
    ([901, 130], 17, 1, 128, 16, torch.bfloat16, 30.0, False),
    ([190, 40], 130, 1, 64, 16, torch.float16, 0.0, False),
]


def _decode(case, layout, fill, seed=3):
    lens, H, Hkv, d, page, dtype, cap, bias = case
    kc, vc, table, n = _cache(lens, Hkv, d, page, dtype, seed, layout, fill)
    g = torch.Generator().manual_seed(seed + 1)
    q = (torch.randn(len(lens), H, d, generator=g) * (3.0 if cap else 1.0)).to(dtype).cuda()
    slopes = _slopes(H) if bias else None
    o, lse = fa.fa_paged_decode(q, kc, vc, table, n, softcap=cap, slopes=slopes)
    fa.fa_sync_check()
    clean = [host_f64(torch.nan_to_num(c.float(), 0.0, 0.0, 0.0)) for c in (kc, vc)]
    ref = paged_decode(host_f64(q), *clean, table.tolist(), lens, d ** -0.5, cap,
                       None if slopes is None else slopes.cpu().numpy(), HALF[dtype])
    return _check(o, ref[0], ref[2], "O"), _check(lse, ref[1], ref[3], "LSE")


@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_decode(case, layout):
    o, lse = _decode(case, layout, None)
    report(f"decode {case} {layout} (shares of the bounds)", o=o, lse=lse)


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("case", [CASES[2], CASES[3], CASES[5], CASES[4]], ids=str)
def test_what_lies_behind_the_last_token_does_not_matter(case, fill):
    _decode(case, "nhd", fill)


def test_page_indices_outside_the_cache_read_as_zeros():
    lens, H, Hkv, d, page = [100, 40], 4, 2, 64, 16
    kc, vc, table, n = _cache(lens, Hkv, d, page, torch.bfloat16, 5)
    table[0, 2], table[0, 3], table[1, 0] = kc.shape[0], -1, 2 ** 31 - 1
    q = torch.randn(2, H, d, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).cuda()
    o, lse = fa.fa_paged_decode(q, kc, vc, table, n)
    fa.fa_sync_check()
    ref = paged_decode(host_f64(q), host_f64(kc), host_f64(vc), table.tolist(), lens, d ** -0.5)
    _check(o, ref[0], ref[2], "O")
    _check(lse, ref[1], ref[3], "LSE")


def test_lengths_are_clamped_to_the_table():
    kc, vc, table, n = _cache([64, 64, 64], 2, 64, 16, torch.bfloat16, 7)
    q = torch.randn(3, 4, 64, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).cuda()
    want, want_l = fa.fa_paged_decode(q, kc, vc, table, n)
    n2 = torch.tensor([2 ** 31 - 1, 64, -5], dtype=torch.int32, device="cuda")
    got, got_l = fa.fa_paged_decode(q, kc, vc, table, n2)
    fa.fa_sync_check()
    assert torch.equal(got[:2], want[:2]) and torch.equal(got_l[:2], want_l[:2])
    assert not got[2].any() and torch.isneginf(got_l[2]).all()


def test_views_of_q_o_and_the_table():
    lens = [70, 33]
    kc, vc, table, n = _cache(lens, 2, 128, 16, torch.bfloat16, 9)
    q = torch.randn(2, 4, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    want, want_l = fa.fa_paged_decode(q, kc, vc, table, n)
    qkv = torch.zeros(2, 3, 4, 136, dtype=torch.bfloat16, device="cuda")
    qkv[:, 1, :, :128] = q
    wide = torch.full((2, table.shape[1] + 3), 77, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    obuf = torch.full((2, 5, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    o, lse = fa.fa_paged_decode(qkv[:, 1, :, :128], kc, vc, wide[:, :table.shape[1]], n, o=obuf[:, :4])
    fa.fa_sync_check()
    assert torch.equal(o, want) and torch.equal(lse, want_l) and bool((obuf[:, 4] == 9).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("new,before", [([1, 1, 1], [0, 16, 40]), ([0, 37, 5, 64], [3, 11, 0, 16]), ([100], [0]), ([0, 0, 1], [0, 5, 31])])
def test_append(new, before, layout, dtype):
    Hkv, d, page = 3, 64, 16
    lens = [a + b for a, b in zip(new, before)]
    kc, vc, table, n = _cache(lens, Hkv, d, page, dtype, 2, layout)
    T = sum(new) + 2  # two rows of no sequence behind the last
    x = torch.randn(T, 2 * Hkv, d, generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    k, v = x[:, :Hkv], x[:, Hkv:]  # views of one projection
    cu = np.concatenate([[0], np.cumsum(new)])
    want = [paged_append(t.float().cpu().numpy(), c.float().cpu().numpy(), table.tolist(), lens, cu) for t, c in ((k, kc), (v, vc))]
    fa.fa_paged_append(k, v, kc, vc, table, n, torch.tensor(cu, dtype=torch.int32, device="cuda"))
    fa.fa_sync_check()
    for c, w in zip((kc, vc), want):
        assert np.array_equal(c.float().cpu().numpy(), w)


def test_append_skips_what_has_no_place():
    # Positions before the cache, past the table and in a page outside the cache are left out.
    Hkv, d, page = 1, 64, 16
    kc, vc = (torch.zeros(3, Hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.tensor([[0, 9], [1, -4], [2, 2]], dtype=torch.int32, device="cuda")
    lens, cu = [18, 2, 40], [0, 4, 9, 13]
    x = torch.arange(1, 14, dtype=torch.float32)[:, None, None].expand(13, 1, d).contiguous().to(torch.bfloat16).cuda()
    want = paged_append(x.float().cpu().numpy(), kc.float().cpu().numpy(), table.tolist(), lens, cu)
    fa.fa_paged_append(x, x, kc, vc, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                       torch.tensor(cu, dtype=torch.int32, device="cuda"))
    fa.fa_sync_check()
    assert np.array_equal(kc.float().cpu().numpy(), want) and np.array_equal(vc.float().cpu().numpy(), want)


def test_prompt_then_tokens_follow_the_training_form():
    """As a model serves: the prompt's rows go into the cache, then one token after the other; each
    token's output is the causal scored forward's row of the whole sequence."""
    H, Hkv, d, page, cap = 8, 2, 128, 16, 30.0
    prompts, steps = [37, 1, 90], 4
    B = len(prompts)
    g = torch.Generator().manual_seed(4)
    full = [[(torch.randn(n + steps, h, d, generator=g) * f).to(torch.bfloat16).cuda() for h, f in ((H, 3.0), (Hkv, 1.0), (Hkv, 1.0))]
            for n in prompts]
    slopes = _slopes(H)
    width = -(-(max(prompts) + steps) // page)
    kc, vc = (torch.full((B * width, Hkv, page, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.randperm(B * width, generator=g).to(torch.int32).view(B, width).cuda()
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    cu = ints(np.concatenate([[0], np.cumsum(prompts)]).tolist())
    fa.fa_paged_append(torch.cat([s[1][:n] for s, n in zip(full, prompts)]), torch.cat([s[2][:n] for s, n in zip(full, prompts)]),
                       kc, vc, table, ints(prompts), cu)
    ref = []
    for q, k, v in full:  # the training form, one sequence a call
        o, lse = fa.fa_fwd_scored(*(x.transpose(0, 1)[None] for x in (q, k, v)), causal=True, softcap=cap, slopes=slopes)
        ref.append((o[0].transpose(0, 1), lse[0].T))
    for t in range(steps):
        at = [n + t for n in prompts]
        lens = ints([a + 1 for a in at])
        row = lambda c: torch.stack([s[c][a] for s, a in zip(full, at)])
        fa.fa_paged_append(row(1), row(2), kc, vc, table, lens, ints(list(range(B + 1))))
        o, lse = fa.fa_paged_decode(row(0), kc, vc, table, lens, softcap=cap, slopes=slopes)
        fa.fa_sync_check()
        for b, a in enumerate(at):
            x = [host_f64(y[:a + 1].transpose(0, 1)[None]) for y in full[b]]
            o_ref, lse_ref, ob, lb = scored_forward(*x, d ** -0.5, True, cap, slopes.cpu().numpy())
            for got_o, got_l in ((o[b], lse[b]), (ref[b][0][a], ref[b][1][a])):
                _check(got_o, o_ref[0, :, a], ob[0, :, a], "O")
                _check(got_l, lse_ref[0, :, a], lb[0, :, a], "LSE")


def test_captured_decode_replays_with_new_lengths():
    lens = [300, 5, 120]
    kc, vc, table, n = _cache([400, 400, 400], 2, 64, 32, torch.float16, 11)
    n.copy_(torch.tensor(lens))
    q = torch.randn(3, 8, 64, generator=torch.Generator().manual_seed(2)).to(torch.float16).cuda()
    ws = torch.empty(fa.fa_paged_decode_workspace_size(3, 8, 2, 64), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(3, 8, device="cuda")
    call = lambda: fa.fa_paged_decode(q, kc, vc, table, n, o=o, lse=lse, workspace=ws)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens in ([1, 400, 0], [399, 0, 64]):
        n.copy_(torch.tensor(lens))
        ws.fill_(0xFF)  # the workspace's contents on entry do not matter
        g.replay()
        got = o.clone(), lse.clone()
        call()
        fa.fa_sync_check()
        assert torch.equal(got[0], o) and torch.equal(got[1], lse)
        ref = paged_decode(host_f64(q), host_f64(kc), host_f64(vc), table.tolist(), lens, 0.125, half=HALF[torch.float16])
        _check(o, ref[0], ref[2], "O")
        _check(lse, ref[1], ref[3], "LSE")


def test_two_decodes_at_once():
    sets = [_cache([700, 30], 2, 128, 16, torch.bfloat16, 20 + s) for s in range(2)]
    qs = [torch.randn(2, 16, 128, generator=torch.Generator().manual_seed(s)).to(torch.bfloat16).cuda() for s in range(2)]
    want = [fa.fa_paged_decode(q, *c) for q, c in zip(qs, sets)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(10):
        got = []
        for q, c, s in zip(qs, sets, streams):
            with torch.cuda.stream(s):
                got.append(fa.fa_paged_decode(q, *c))
        torch.cuda.synchronize()
        for (a, b), (x, y) in zip(want, got):
            assert torch.equal(a, x) and torch.equal(b, y)


def test_cache_past_32_bit_offsets():
    # A page far behind the first 2^31 elements of the cache (the page stride carries it there).
    Hkv, page, d = 1, 16, 64
    stride = 1 << 30  # elements between pages: the cache spans 3 * 2^30 elements, 6 GB
    kbuf = torch.empty(2 * stride + Hkv * page * d, dtype=torch.bfloat16, device="cuda")
    vbuf = torch.empty_like(kbuf)
    view = lambda t: t.as_strided((3, Hkv, page, d), (stride, page * d, d, 1))
    kc, vc = view(kbuf), view(vbuf)
    kc.fill_(0)
    vc.fill_(0)
    table = torch.tensor([[2, 0]], dtype=torch.int32, device="cuda")
    n = torch.tensor([20], dtype=torch.int32, device="cuda")
    x = torch.randn(20, 2, d, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
    fa.fa_paged_append(x[:, :1], x[:, 1:], kc, vc, table, n, torch.tensor([0, 20], dtype=torch.int32, device="cuda"))
    q = torch.randn(1, 2, d, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).cuda()
    o, lse = fa.fa_paged_decode(q, kc, vc, table, n)
    fa.fa_sync_check()
    assert torch.equal(kc[2, 0], x[:16, 0]) and torch.equal(vc[0, 0, :4], x[16:, 1])
    ref = paged_decode(host_f64(q), host_f64(kc), host_f64(vc), table.tolist(), [20], 0.125)
    _check(o, ref[0], ref[2], "O")
    _check(lse, ref[1], ref[3], "LSE")


def test_refusals_in_the_binding():
    kc, vc, table, n = _cache([40], 2, 64, 16, torch.bfloat16, 1)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError):
        fa.fa_paged_decode(q.half(), kc, vc, table, n)
    with pytest.raises(fa.FAError):
        fa.fa_paged_decode(q[:, :3].contiguous(), kc, vc, table, n)
    with pytest.raises(ValueError):
        fa.fa_paged_decode(q, kc, vc, table.long(), n)
    with pytest.raises(ValueError):
        fa.fa_paged_decode(q, kc, vc, table, n.cpu())
    with pytest.raises(fa.FAError):
        fa.fa_paged_decode(q, kc[:, :, :8], vc[:, :, :8], table, n)  # pages of 8 tokens
    with pytest.raises(fa.FAError):
        fa.fa_paged_decode(q, kc, vc, table, n, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))


def test_sequences_that_share_pages():
    # Three sequences with the same first pages (a common prompt), one page twice in one table.
    kc, vc, table, n = _cache([100, 30, 64], 2, 64, 16, torch.bfloat16, 21)
    table[1, :2] = table[0, :2]
    table[2, :4] = table[0, :4]
    table[2, 3] = table[0, 0]
    q = torch.randn(3, 4, 64, generator=torch.Generator().manual_seed(22)).to(torch.bfloat16).cuda()
    o, lse = fa.fa_paged_decode(q, kc, vc, table, n, softcap=20.0)
    fa.fa_sync_check()
    ref = paged_decode(host_f64(q), host_f64(kc), host_f64(vc), table.tolist(), n.tolist(), 0.125, 20.0)
    _check(o, ref[0], ref[2], "O")
    _check(lse, ref[1], ref[3], "LSE")


def test_more_sequences_than_threads_of_a_block():
    lens = [(7 * b) % 61 for b in range(700)]
    _decode((lens, 4, 2, 64, 16, torch.bfloat16, 0.0, True), "nhd", None)


def test_append_of_many_heads():
    # More 16-byte pieces in a token's row than a warp holds at once, the last of them partial.
    Hkv, d, page = 21, 128, 16
    kc, vc, table, n = _cache([19, 3], Hkv, d, page, torch.bfloat16, 23)
    x = torch.randn(9, 2, Hkv, d, generator=torch.Generator().manual_seed(24)).to(torch.bfloat16).cuda()
    cu = torch.tensor([0, 6, 9], dtype=torch.int32, device="cuda")
    want = [paged_append(host_f64(x[:, i]), host_f64(c), table.tolist(), n.tolist(), cu.tolist()) for i, c in enumerate((kc, vc))]
    fa.fa_paged_append(x[:, 0], x[:, 1], kc, vc, table, n, cu)
    fa.fa_sync_check()
    assert np.array_equal(host_f64(kc), want[0]) and np.array_equal(host_f64(vc), want[1])


@pytest.mark.parametrize("Hkv,d", [(1, 64), (3, 64), (1, 128)])
def test_append_of_many_short_rows(Hkv, d):
    # More tokens than 16 warps an SM take one each: several tokens a warp, their rows' pieces not a
    # multiple of its lanes, sequences and pages ending inside a warp's tokens, and rows of no sequence.
    page, new = 48, [9001, 0, 1, 12345, 77, 3]
    lens = [n + 5 * b for b, n in enumerate(new)]
    kc, vc, table, n = _cache(lens, Hkv, d, page, torch.float16, 29)
    T = sum(new) + 7
    x = torch.randn(T, 2, Hkv, d, generator=torch.Generator().manual_seed(30)).half().cuda()
    cu = np.concatenate([[0], np.cumsum(new)])
    want = [paged_append(host_f64(x[:, i]), host_f64(c), table.tolist(), lens, cu) for i, c in enumerate((kc, vc))]
    fa.fa_paged_append(x[:, 0], x[:, 1], kc, vc, table, n, torch.tensor(cu, dtype=torch.int32, device="cuda"))
    fa.fa_sync_check()
    assert np.array_equal(host_f64(kc), want[0]) and np.array_equal(host_f64(vc), want[1])


def test_two_graphs_share_a_workspace():
    # Captured for two batches of other sizes over one workspace and replayed in turn on one stream.
    kc, vc, table, n = _cache([700, 90, 333], 2, 64, 16, torch.bfloat16, 25)
    q = torch.randn(3, 8, 64, generator=torch.Generator().manual_seed(26)).to(torch.bfloat16).cuda()
    ws = torch.empty(fa.fa_paged_decode_workspace_size(3, 8, 2, 64), dtype=torch.uint8, device="cuda")
    runs = [lambda o, l: fa.fa_paged_decode(q, kc, vc, table, n, o=o, lse=l, workspace=ws),
            lambda o, l: fa.fa_paged_decode(q[:1], kc, vc, table[:1], n[:1], o=o, lse=l, workspace=ws)]
    want = [fa.fa_paged_decode(q, kc, vc, table, n), fa.fa_paged_decode(q[:1], kc, vc, table[:1], n[:1])]
    outs = [(torch.zeros_like(o), torch.zeros_like(l)) for o, l in want]
    graphs = []
    for run, out in zip(runs, outs):
        run(*out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(*out)
        graphs.append(g)
    for turn in (0, 1, 1, 0):
        for t in outs[turn]:
            t.fill_(7)
        graphs[turn].replay()
        for a, b in zip(outs[turn], want[turn]):
            assert torch.equal(a, b)
    fa.fa_sync_check()


def test_a_stream_given_by_the_caller():
    kc, vc, table, n = _cache([3000, 1], 2, 128, 64, torch.float16, 27)
    q = torch.randn(2, 8, 128, generator=torch.Generator().manual_seed(28)).half().cuda()
    want = fa.fa_paged_decode(q, kc, vc, table, n)
    size = fa.fa_paged_decode_workspace_size(2, 8, 2, 128)
    torch.cuda.synchronize()
    s, got = torch.cuda.Stream(), []
    for _ in range(8):
        got.append(fa.fa_paged_decode(q, kc, vc, table, n, stream=s))
        torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    fa.fa_sync_check()
    for o, lse in got:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("below", [20.0, 25.5, 28.0])
def test_many_small_weights_behind_a_dominant_token(dtype, below):
    # The first token weighs 2^below times as much as each of the others and adds nothing to the output,
    # which is theirs alone.  320 sequences over the same pages: more heads than blocks, so that a block's
    # warp meets the first token and a quarter of the rest with one reference.
    B, H, n, d, page = 320, 2, 2055, 64, 16
    pages = -(-n // page)
    g = torch.Generator().manual_seed(31)
    kc = torch.zeros(pages, 1, page, d, dtype=dtype)
    kc[..., 0] = -below * float(np.log(2.0))
    vc = (1.0 + torch.rand(pages, 1, page, d, generator=g)).to(dtype)
    kc[0, 0, 0], vc[0, 0, 0] = 0.0, 0.0
    q = torch.zeros(B, H, d, dtype=dtype)
    q[..., 0] = 1.0
    table = torch.arange(pages, dtype=torch.int32).expand(B, pages).contiguous()
    lens = torch.full((B,), n, dtype=torch.int32)
    o, lse = fa.fa_paged_decode(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), lens.cuda(), scale=1.0)
    fa.fa_sync_check()
    ref = paged_decode(host_f64(q[:1]), host_f64(kc), host_f64(vc), table[:1].tolist(), [n], 1.0, half=HALF[dtype])
    for b in range(B):
        _check(o[b], ref[0][0], ref[2][0], "O")
        _check(lse[b], ref[1][0], ref[3][0], "LSE")


@pytest.mark.parametrize("n", [17, 33, 65, 129, 700])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_tokens_of_weight_zero_alone_in_a_warps_share(n, dtype):
    # The last token's score is -inf (a key with an infinite entry): its weight is 0, also where it is the only
    # token of a warp or of a block.
    H, d, page = 3, 128, 16
    kc, vc, table, lens = _cache([n], 1, d, page, dtype, 36)
    q = torch.randn(1, H, d, generator=torch.Generator().manual_seed(37)).to(dtype).cuda()
    q[:, :, 5] = q[:, :, 5].abs() + 0.5
    kc[table[0, (n - 1) // page].item(), 0, (n - 1) % page, 5] = float("-inf")
    o, lse = fa.fa_paged_decode(q, kc, vc, table, lens)
    fa.fa_sync_check()
    # Its place counts for nothing without a bias: the same without the token.
    ref = paged_decode(host_f64(q), host_f64(torch.nan_to_num(kc, neginf=0.0)), host_f64(vc), table.tolist(), [n - 1], d ** -0.5,
                       half=HALF[dtype])
    _check(o, ref[0], ref[2], "O")
    _check(lse, ref[1], ref[3], "LSE")


@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("at", [0, 64, 699])
def test_nan_in_a_visible_key_comes_through(at, cap):
    # ... to the heads that read it, also from a warp, a block or a part that holds no other token.
    kc, vc, table, lens = _cache([700], 2, 128, 16, torch.bfloat16, 38)
    q = torch.randn(1, 6, 128, generator=torch.Generator().manual_seed(39)).to(torch.bfloat16).cuda()
    kc[table[0, at // 16].item(), 0, at % 16, 5] = float("nan")
    o, lse = fa.fa_paged_decode(q, kc, vc, table, lens, softcap=cap)
    fa.fa_sync_check()
    assert bool(torch.isnan(o[:, :3]).all()) and bool(torch.isnan(lse[:, :3]).all())
    assert bool(torch.isfinite(o[:, 3:]).all()) and bool(torch.isfinite(lse[:, 3:]).all())


@pytest.mark.parametrize("cap", [200.0, 1e4, 1e6, 1e20])
@pytest.mark.parametrize("H,Hkv,d,dtype,bias", [(4, 2, 64, torch.bfloat16, False), (24, 1, 128, torch.float16, True)])
def test_decode_with_caps_far_above_the_scores(H, Hkv, d, dtype, bias, cap):
    # (a cap that hardly bends: its error is relative to the score, not to the cap)
    _decode(([1, 70, 900], H, Hkv, d, 16, dtype, cap, bias), "nhd", None)


@pytest.mark.parametrize("cap", [10.0, 100.0, 300.0])
def test_decode_with_small_and_large_arguments_of_the_cap(cap):
    # Scores from far below the cap to far past it, side by side.
    lens, H, d, page = [300, 40], 8, 64, 16
    kc, vc, table, n = _cache(lens, 2, d, page, torch.bfloat16, 33)
    f = torch.logspace(-2, 2.5, H)[None, :, None]
    q = (torch.randn(2, H, d, generator=torch.Generator().manual_seed(34)) * f).to(torch.bfloat16).cuda()
    o, lse = fa.fa_paged_decode(q, kc, vc, table, n, softcap=cap)
    fa.fa_sync_check()
    ref = paged_decode(host_f64(q), host_f64(kc), host_f64(vc), table.tolist(), lens, d ** -0.5, cap)
    _check(o, ref[0], ref[2], "O")
    _check(lse, ref[1], ref[3], "LSE")


def test_decode_agrees_with_the_forward_at_a_large_cap():
    H, Hkv, N, d, cap = 4, 2, 200, 64, 1e5
    g = torch.Generator().manual_seed(35)
    q, k, v = (torch.randn(1, h, N, d, generator=g).to(torch.bfloat16).cuda() for h in (H, Hkv, Hkv))
    _, want = fa.fa_fwd_scored(q, k, v, causal=True, softcap=cap)
    kc, vc = (torch.zeros(13, Hkv, 16, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    table, n = torch.arange(13, dtype=torch.int32, device="cuda")[None], ints([N])
    fa.fa_paged_append(k[0].transpose(0, 1), v[0].transpose(0, 1), kc, vc, table, n, ints([0, N]))
    _, lse = fa.fa_paged_decode(q[:, :, -1], kc, vc, table, n, softcap=cap)
    fa.fa_sync_check()
    # The bound of either LSE, twice: products of at most 10 (sums of |q k| / 8) to 80 half steps and 2e-6, in
    # the LSE twice, and 4 half steps of the LSE.
    assert float((lse - want[:, :, -1]).abs().max()) <= 2 * (2 * (80 * 10 * 2.0 ** -24 + 2e-6) + 4 * 10 * 2.0 ** -24)


@pytest.mark.parametrize("case", [([0, 300, 1, 17, 900, 0, 40, 16, 129, 31] * 20, 16, 2, 64, 16, torch.bfloat16, 0.0, True),
                                  ([5, 0, 700, 16, 130] * 10, 80, 4, 128, 64, torch.float16, 30.0, False)], ids=["3200", "4000"])
def test_many_heads(case):
    # More heads than blocks that join their parts: some whole, some in parts, some of empty sequences.
    _decode(case, "nhd", None)


@pytest.mark.parametrize("H,Hkv,d", [(16, 2, 64), (8, 1, 128), (64, 2, 64), (40, 1, 128)])
def test_decode_in_the_workspace_that_it_uses(H, Hkv, d):
    # Two parts for each of 32 rows an SM and the tiles before each sequence: what the 8-bit cache's decode needs beside
    # that, this one neither asks for nor writes.
    lens = [3000, 0, 700, 1]
    kc, vc, table, n = _cache(lens, Hkv, d, 16, torch.bfloat16, 41)
    q = torch.randn(4, H, d, generator=torch.Generator().manual_seed(42)).to(torch.bfloat16).cuda()
    want = fa.fa_paged_decode(q, kc, vc, table, n)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    size = (2 * 32 * sms * (d + 2) * 4 + 255) // 256 * 256 + (4 + 2) * 8
    buf = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    got = fa.fa_paged_decode(q, kc, vc, table, n, workspace=buf[:size])
    fa.fa_sync_check()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and bool((buf[size:] == 0xA5).all())
    with pytest.raises(fa.FAError):
        fa.fa_paged_decode(q, kc, vc, table, n, workspace=buf[:size - 1])
    assert fa.fa_paged_decode_workspace_size(4, H, Hkv, d) >= size


@pytest.mark.parametrize("H,Hkv,d", [(32, 8, 128), (24, 24, 64)])
def test_idle_places(H, Hkv, d):
    # A batch of a fixed number of places, most of them idle: zeros and -inf there, nothing written beside them.
    lens = [0] * 997
    lens[5], lens[128], lens[996] = 700, 1, 333
    kc, vc, table, n = _cache(lens, Hkv, d, 16, torch.bfloat16, 51)
    q = torch.randn(997, H, d, generator=torch.Generator().manual_seed(52)).to(torch.bfloat16).cuda()
    buf = torch.full((997, H + 1, d), 9.0, dtype=torch.bfloat16, device="cuda")
    o, lse = fa.fa_paged_decode(q, kc, vc, table, n, o=buf[:, :H])
    live = [5, 128, 996]
    want, want_l = fa.fa_paged_decode(q[live], kc, vc, table[live], n[live])
    fa.fa_sync_check()
    idle = n == 0
    assert not o[idle].any() and torch.isneginf(lse[idle]).all() and bool((buf[:, H] == 9).all())
    # (other shares: the parts' sums in another order; a few fp32 steps, before one of bf16)
    assert (o[live].float() - want.float()).abs().max() <= 2.0 ** -7 * want.abs().max() and (lse[live] - want_l).abs().max() < 1e-4
