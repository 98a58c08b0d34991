"""Scored attention on the GPU against the float64 oracle, element by element.

The bounds are the oracle's (oracle/scored.py): the roundings the path makes on purpose,
2^-8 relative each, carried through the formulas, plus the fp32 error of the scores.
"""

import numpy as np
import pytest
import torch

import io_aware_exact_fwd_gb300 as fa
from oracle import scored_backward, scored_forward

from gpu_util import host_f64, report

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fa.load_library()
    fa.fa_debug_set_fault(0)
    fa.fa_debug_set_wait_limit_ns(0)


def _slopes(H):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=torch.float32, device="cuda")


def _inputs(B, H, Hkv, N, d, seed, qscale=1.0, layout="bhnd"):
    g = torch.Generator().manual_seed(seed)

    def one(n, f=1.0):
        x = (torch.randn(B, N, n, d, generator=g) * f).to(torch.bfloat16).cuda()
        return x.transpose(1, 2) if layout == "bnhd" else x.transpose(1, 2).contiguous()
    return one(H, qscale), one(Hkv), one(Hkv), one(H)


def _docs(cu, prefix, causal, B, N):
    if cu is None and prefix is None:
        return None
    t = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")
    return fa.fa_mask_plan(B, N, t(cu), t(prefix), causal=causal, device="cuda")


def _check(got, ref, bound, what):
    got = host_f64(got)
    same = np.isneginf(got) == np.isneginf(ref)
    assert same.all(), f"{what}: -inf in {int((~same).sum())} places where the oracle has none, or the reverse"
    fin = np.isfinite(ref)
    assert np.isfinite(got[fin]).all(), f"{what}: not finite"
    ratio = np.abs(got[fin] - ref[fin]) / np.maximum(bound[fin], 1e-300)
    assert ratio.size == 0 or ratio.max() <= 1.0, f"{what}: error {ratio.max():.3f} of its bound"
    return float(ratio.max(initial=0.0))


# B, H, Hkv, N, d, causal, cap, bias, documents, prefix
CASES = [
    (1, 1, 1, 1, 64, True, 0.0, False, None, None),
    (1, 2, 1, 1, 128, False, 30.0, True, None, None),
    (1, 2, 2, 127, 64, True, 30.0, False, None, None),
    (1, 2, 2, 128, 128, False, 0.0, True, None, None),
    (1, 3, 1, 129, 128, True, 50.0, True, None, None),
    (2, 4, 2, 257, 64, False, 20.0, False, None, None),
    (1, 2, 2, 600, 128, True, 0.0, True, None, None),
    (1, 2, 1, 700, 64, True, 0.0, False, [[0, 3, 3, 260, 555]], None),
    (2, 2, 1, 300, 128, True, 20.0, True, [[0, 1, 128, 300], [5, 100, 100, 129]], [[1, 40, 90], [95, 3, 0]]),
    (1, 2, 2, 513, 64, False, 0.0, True, [[0, 200, 213, 512]], None),
    (1, 2, 2, 513, 128, False, 8.0, False, [[130, 200, 256, 384]], None),
    (2, 2, 2, 200, 128, True, 30.0, False, [[0, 0], [0, 200]], None),          # one row all padding
    (1, 8, 1, 384, 64, True, 0.0, False, None, [[300]]),                       # a prefix and no documents
    (1, 5, 5, 130, 128, True, 5.0, False, [[0, 130]], [[1000]]),               # the prefix passes the end
    (1, 2, 1, 1100, 128, True, 0.0, True, [[0, 500, 1100]], [[499, 30]]),
    (1, 2, 2, 400, 64, True, 200.0, True, [[0, 130, 390]], [[20, 100]]),       # a cap far above the scores
    (1, 2, 1, 300, 128, False, 80.0, True, None, None),
    (3, 2, 2, 65, 64, True, 0.0, False, [[64, 65, 65], [0, 1, 2], [0, 64, 65]], None),
    (1, 16, 1, 1030, 128, True, 0.0, True, None, None),                        # a key block's steps on 16 blocks
    (1, 24, 2, 515, 64, True, 20.0, False, [[3, 100, 101, 400]], [[10, 1, 200]]),
]


def _kw(case, plan):
    B, H, Hkv, N, d, causal, cap, bias, cu, pre = case
    return dict(causal=causal and plan is None, softcap=cap, slopes=_slopes(H) if bias else None, plan=plan)


@pytest.mark.parametrize("layout", ["bhnd", "bnhd"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_and_gradients(case, layout):
    B, H, Hkv, N, d, causal, cap, bias, cu, pre = case
    q, k, v, do = _inputs(B, H, Hkv, N, d, 11 + N, 3.0 if cap else 1.0, layout)
    plan = _docs(cu, pre, causal, B, N)
    kw = _kw(case, plan)
    slopes = None if not bias else _slopes(H).cpu().numpy()
    o, lse = fa.fa_fwd_scored(q, k, v, **kw)
    fa.fa_sync_check()
    args = (d ** -0.5, causal, cap, slopes, cu, pre)
    x = [host_f64(t) for t in (q, k, v, do)]
    o_ref, lse_ref, ob, lb = scored_forward(*x[:3], *args)
    r = {"o": _check(o, o_ref, ob, "O"), "lse": _check(lse, lse_ref, lb, "LSE")}
    for det in (False, True):
        grads = fa.fa_bwd_scored(q, k, v, o, do, lse, deterministic=det, **kw)
        fa.fa_sync_check()
        refs, bounds = scored_backward(*x, *args)
        for name, a, ref, bd in zip(("dq", "dk", "dv"), grads, refs, bounds):
            r[name] = _check(a, ref, bd, f"{name} deterministic={det}")
    report(f"scored {case} {layout} (shares of the bounds)", **r)


# More tiles and key blocks than the SMs run at once: units of two tiles, taken over by running blocks, and undivided
# key blocks (the cases above are mostly of halved units and divided blocks).
MANY = [
    (2, 32, 32, 700, 64, True, 0.0, False, None, None),
    (2, 32, 8, 700, 128, True, 0.0, True, [[0, 130, 400, 690], [20, 300, 301, 650]], [[100, 3, 0], [0, 1, 200]]),
    (2, 32, 32, 700, 128, True, 20.0, False, [[0, 130, 400, 690], [20, 300, 301, 650]], None),
    (2, 32, 32, 700, 64, True, 20.0, True, None, None),
    (2, 32, 8, 700, 128, True, 60.0, True, None, None),
    (2, 32, 16, 700, 64, True, 0.0, True, [[0, 700], [300, 690]], None),
    (2, 32, 16, 700, 64, True, 30.0, False, [[0, 690], [30, 400]], [[200], [5]]),
    (5, 16, 16, 300, 128, False, 0.0, True, None, None),
    (5, 16, 16, 300, 64, False, 60.0, False, None, None),
    (20, 16, 4, 130, 128, True, 20.0, True, [[5 * (b % 3), 20 + b, 60 + 3 * b, 130 - b] for b in range(20)], None),
]


@pytest.mark.parametrize("case", MANY, ids=str)
def test_many_tiles(case):
    B, H, Hkv, N, d, causal, cap, bias, cu, pre = case
    q, k, v, do = _inputs(B, H, Hkv, N, d, 31 + N, 3.0 if cap else 1.0)
    plan = _docs(cu, pre, causal, B, N)
    kw = _kw(case, plan)
    args = (d ** -0.5, causal, cap, None if not bias else _slopes(H).cpu().numpy(), cu, pre)
    o, lse = fa.fa_fwd_scored(q, k, v, **kw)
    grads = fa.fa_bwd_scored(q, k, v, o, do, lse, **kw)
    fa.fa_sync_check()
    x = [host_f64(t) for t in (q, k, v, do)]
    o_ref, lse_ref, ob, lb = scored_forward(*x[:3], *args)
    r = {"o": _check(o, o_ref, ob, "O"), "lse": _check(lse, lse_ref, lb, "LSE")}
    refs, bounds = scored_backward(*x, *args)
    for name, a, ref, bd in zip(("dq", "dk", "dv"), grads, refs, bounds):
        r[name] = _check(a, ref, bd, name)
    report(f"scored {case[:8]} (shares of the bounds)", **r)


@pytest.mark.parametrize("cap", [0.0, 10.0, 55.0, 60.0, 1000.0])
def test_large_scores_and_slopes(cap):
    # Scores far past the cap on both sides (or without one), and slopes that leave only the nearest
    # keys, or the farthest.
    B, H, N, d = 1, 3, 300, 64
    q, k, v, do = _inputs(B, H, H, N, d, 5, 40.0)
    slopes = torch.tensor([8.0, -0.03, -2.0], device="cuda")
    for causal in (False, True):
        o, lse = fa.fa_fwd_scored(q, k, v, causal=causal, softcap=cap, slopes=slopes)
        fa.fa_sync_check()
        x = [host_f64(t) for t in (q, k, v, do)]
        o_ref, lse_ref, ob, lb = scored_forward(*x[:3], d ** -0.5, causal, cap, slopes.cpu().numpy())
        _check(o, o_ref, ob, "O")
        _check(lse, lse_ref, lb, "LSE")
        grads = fa.fa_bwd_scored(q, k, v, o, do, lse, causal=causal, softcap=cap, slopes=slopes)
        fa.fa_sync_check()
        refs, bounds = scored_backward(*x, d ** -0.5, causal, cap, slopes.cpu().numpy())
        for name, a, ref, bd in zip(("dq", "dk", "dv"), grads, refs, bounds):
            _check(a, ref, bd, name)


@pytest.mark.parametrize("H", [1, 62])
def test_scores_that_fall_and_rise_along_the_keys(H):
    # Row maxima far apart between key blocks, both ways, without a cap: -400 to 400.
    B, N, d = 1, 640, 64
    q, k, v, do = _inputs(B, H, H, N, d, 6)
    ramp = torch.linspace(-1, 1, N, device="cuda")[None, None, :, None]
    for sign in (1.0, -1.0):
        qq = torch.ones_like(q) * 8.0
        kk = (sign * ramp * 50.0 * torch.ones_like(k) + 0.1 * k).to(torch.bfloat16)
        plan = _docs([[0, 333, 600]], None, True, B, N)
        o, lse = fa.fa_fwd_scored(qq, kk, v, plan=plan)
        fa.fa_sync_check()
        x = [host_f64(t) for t in (qq, kk, v, do)]
        o_ref, lse_ref, ob, lb = scored_forward(*x[:3], d ** -0.5, True, 0.0, None, [[0, 333, 600]])
        _check(o, o_ref, ob, "O")
        _check(lse, lse_ref, lb, "LSE")


def test_without_options_it_agrees_with_fa_fwd():
    q, k, v, _ = _inputs(2, 3, 3, 300, 128, 8)
    for causal in (False, True):
        o, lse = fa.fa_fwd_scored(q, k, v, causal=causal)
        o1, lse1 = fa.fa_fwd(q, k, v, causal=causal)
        fa.fa_sync_check()
        # Both are within 2^-8 (P) + 2^-8 (O) of the same value.
        assert float((lse - lse1).abs().max()) <= 1e-5
        assert float((o.float() - o1.float()).abs().max()) <= 2 * 2.0 ** -7 * float(v.float().abs().max())


@pytest.mark.parametrize("H,Hkv", [(4, 2), (64, 32)])
def test_same_bits_on_every_run(H, Hkv):
    q, k, v, do = _inputs(1, H, Hkv, 700, 64, 9, 3.0)
    plan = _docs([[0, 300, 690]], [[20, 50]], True, 1, 700)
    kw = dict(softcap=20.0, slopes=_slopes(H), plan=plan)
    runs = []
    for _ in range(3):
        o, lse = fa.fa_fwd_scored(q, k, v, **kw)
        runs.append((o, lse, *fa.fa_bwd_scored(q, k, v, o, do, lse, deterministic=True, **kw)))
    fa.fa_sync_check()
    for other in runs[1:]:
        for a, b in zip(runs[0], other):
            assert torch.equal(a, b)


@pytest.mark.parametrize("N", [150, 530])  # the longer with each key block's steps divided
def test_outputs_of_another_layout_and_neighbours_untouched(N):
    # o, dq, dk, dv as views of larger buffers: what lies between their rows stays.
    B, H, Hkv, d = 1, 2, 1, 64
    q, k, v, do = _inputs(B, H, Hkv, N, d, 10, layout="bnhd")
    kw = dict(causal=True, softcap=15.0)
    o, lse = fa.fa_fwd_scored(q, k, v, **kw)
    ref = (o, *fa.fa_bwd_scored(q, k, v, o, do, lse, deterministic=True, **kw))
    bufs, views = [], []
    for n in (H, H, Hkv, Hkv):
        buf = torch.full((B, N + 3, n + 1, d + 8), 7.0, dtype=torch.bfloat16, device="cuda")
        bufs.append(buf)
        views.append(buf[:, :N, :n, :d].transpose(1, 2))
    o2, _ = fa.fa_fwd_scored(q, k, v, o=views[0], **kw)
    fa.fa_bwd_scored(q, k, v, o, do, lse, dq=views[1], dk=views[2], dv=views[3], deterministic=True, **kw)
    fa.fa_sync_check()
    for buf, view, want in zip(bufs, views, ref):
        assert torch.equal(view, want)
        rest = buf.clone()
        rest[:, :N, :view.shape[1], :d] = 7.0
        assert torch.equal(rest, torch.full_like(rest, 7.0))


def test_captured_step_replays_with_new_inputs_and_documents():
    # plan, forward and backward in one graph on a side stream; replayed after the inputs and the
    # document offsets changed in place.
    B, H, N, d = 1, 2, 260, 64
    q, k, v, do = _inputs(B, H, H, N, d, 12)
    cu = torch.tensor([[0, 100, 260]], dtype=torch.int32, device="cuda")
    plan = fa.fa_mask_plan(B, N, cu)
    o, lse = torch.empty_like(q), torch.empty(B, H, N, device="cuda")
    dq, dk, dv = (torch.empty_like(q) for _ in range(3))
    ws = torch.empty(fa.fa_bwd_scored_workspace_size(B, H, H, N, d), dtype=torch.uint8, device="cuda")

    def step():
        fa.fa_mask_plan(B, N, cu, plan=plan)
        fa.fa_fwd_scored(q, k, v, o=o, lse=lse, softcap=25.0, plan=plan)
        fa.fa_bwd_scored(q, k, v, o, do, lse, dq=dq, dk=dk, dv=dv, workspace=ws, softcap=25.0, plan=plan, deterministic=True)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    cu.copy_(torch.tensor([[0, 31, 250]], dtype=torch.int32))
    q2, k2, v2, do2 = _inputs(B, H, H, N, d, 13)
    for a, b in ((q, q2), (k, k2), (v, v2), (do, do2)):
        a.copy_(b)
    g.replay()
    got = [t.clone() for t in (o, lse, dq, dk, dv)]
    step()
    fa.fa_sync_check()
    for a, b in zip(got, (o, lse, dq, dk, dv)):
        assert torch.equal(a, b)
    o_ref, lse_ref, ob, lb = scored_forward(*(host_f64(t) for t in (q, k, v)), d ** -0.5, True, 25.0, None, [[0, 31, 250]])
    _check(o, o_ref, ob, "O")
    _check(lse, lse_ref, lb, "LSE")


def test_two_streams_at_once():
    ins = [_inputs(1, 4, 2, 500, 128, 20 + n) for n in range(2)]
    want = []
    for q, k, v, do in ins:
        o, lse = fa.fa_fwd_scored(q, k, v, causal=True, softcap=30.0)
        want.append((o, lse, *fa.fa_bwd_scored(q, k, v, o, do, lse, causal=True, softcap=30.0, deterministic=True)))
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in ins], []
    for (q, k, v, do), s in zip(ins, streams):
        with torch.cuda.stream(s):
            o, lse = fa.fa_fwd_scored(q, k, v, causal=True, softcap=30.0)
            got.append((o, lse, *fa.fa_bwd_scored(q, k, v, o, do, lse, causal=True, softcap=30.0, deterministic=True)))
    torch.cuda.synchronize()
    fa.fa_sync_check()
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_offsets_that_break_the_contract_stay_in_bounds():
    # Decreasing and out-of-range offsets: unspecified values, but finite ones, no error, and no
    # write outside the outputs (canaries around them).
    B, H, N, d = 1, 2, 400, 64
    q, k, v, do = _inputs(B, H, H, N, d, 14)
    for cu in ([[-50, 300, 100, 9999]], [[390, 10, 380, 20]], [[500, 600, 700, 800]], [[-9, -8, -7, -6]]):
        plan = _docs(cu, [[7, -3, 2 ** 31 - 1]], True, B, N)
        buf = torch.full((B, H + 2, N, d), 3.0, dtype=torch.bfloat16, device="cuda")
        o, lse = fa.fa_fwd_scored(q, k, v, o=buf[:, 1:-1], plan=plan)
        fa.fa_bwd_scored(q, k, v, o, do, lse, plan=plan)
        fa.fa_sync_check()
        assert bool((buf[:, 0] == 3).all()) and bool((buf[:, -1] == 3).all())


def test_refusals_in_the_binding():
    q, k, v, do = _inputs(1, 4, 2, 64, 64, 15)
    with pytest.raises(fa.FAError):
        fa.fa_fwd_scored(q, k, v, causal=True, plan=fa.fa_mask_plan(1, 64, device="cuda"))
    with pytest.raises(fa.FAError):
        fa.fa_fwd_scored(q, k, v, plan=fa.fa_mask_plan(1, 32, device="cuda"))  # a plan for fewer positions
    with pytest.raises(fa.FAError):
        fa.fa_fwd_scored(q[:, :3].contiguous(), k, v)
    with pytest.raises(fa.FAError):
        fa.fa_fwd_scored(q, k[:, :1].expand(1, 4, 64, 64), v[:, :1].expand(1, 4, 64, 64))  # a stride of 0
    with pytest.raises(ValueError):
        fa.fa_fwd_scored(q, k, v, slopes=torch.ones(3, device="cuda"))
    with pytest.raises(ValueError):
        fa.fa_fwd_scored(q, k, v, slopes=torch.ones(4))
    with pytest.raises(ValueError):
        fa.fa_fwd_scored(q.transpose(2, 3), k, v)


def test_a_plan_of_other_rows_stays_in_bounds():
    # A plan with the same bytes but longer rows, and arbitrary bytes: an unspecified mask, outputs that are
    # finite, and nothing written outside them.
    B, H, N, d = 2, 2, 192, 64
    q, k, v, do = _inputs(B, H, H, N, d, 16)
    longer = fa.fa_mask_plan(1, 2 * N, device="cuda")
    bytes_ = torch.randint(0, 256, (16 * B * N,), dtype=torch.uint8, generator=torch.Generator().manual_seed(3)).cuda()
    for plan in (longer, bytes_):
        buf = torch.full((B, H + 2, N, d), 3.0, dtype=torch.bfloat16, device="cuda")
        o, lse = fa.fa_fwd_scored(q, k, v, o=buf[:, 1:-1], plan=plan)
        grads = [torch.full((B, H + 2, N, d), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
        fa.fa_bwd_scored(q, k, v, o, do, lse, *(x[:, 1:-1] for x in grads), plan=plan)
        fa.fa_sync_check()
        for x in (buf, *grads):
            assert bool((x[:, 0] == 3).all()) and bool((x[:, -1] == 3).all())


@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("deterministic", [False, True])
def test_what_padding_holds_does_not_matter(cap, deterministic):
    # The largest finite values in padding, alone and opposite in sign: their products pass the range
    # of fp32 and give infinities and NaN, none of which may reach a result.
    B, H, N, d = 1, 2, 300, 64
    q, k, v, do = _inputs(B, H, H, N, d, 17)
    plan = _docs([[40, 150, 220]], None, True, B, N)
    kw = dict(softcap=cap, plan=plan)
    o, lse = fa.fa_fwd_scored(q, k, v, **kw)
    want = (o, lse, *fa.fa_bwd_scored(q, k, v, o, do, lse, deterministic=True, **kw))
    x = [host_f64(t) for t in (q, k, v, do)]
    args = (d ** -0.5, True, cap, None, [[40, 150, 220]], None)
    o_ref, lse_ref, ob, lb = scored_forward(*x[:3], *args)
    refs, bounds = scored_backward(*x, *args)
    big = torch.finfo(torch.bfloat16).max
    for x, f in ((q, big), (k, -big), (v, big), (do, big)):
        for part in (slice(0, 40), slice(220, N)):
            x[:, :, part] = f
            x[:, :, part, ::2] = -f
    o, lse = fa.fa_fwd_scored(q, k, v, **kw)
    got = (o, lse, *fa.fa_bwd_scored(q, k, v, o, do, lse, deterministic=deterministic, **kw))
    fa.fa_sync_check()
    for name, a, b, ref, bound in zip(("o", "lse", "dq", "dk", "dv"), got, want, (o_ref, lse_ref, *refs), (ob, lb, *bounds)):
        _check(a, ref, bound, name)
        # The same bits, but where dq's sum has no fixed order, and with a cap, whose form is chosen by
        # the largest argument of 32 neighbours: padding may send a row to the other form, whose
        # values differ by an fp32 error that the oracle's bounds count.
        if cap == 0.0 and (name != "dq" or deterministic):
            assert torch.equal(a, b), name


def test_a_stream_given_by_the_caller():
    # Everything on `stream`, the workspace made by the call; the current stream's memory churns beside it.
    q, k, v, do = _inputs(1, 4, 2, 700, 64, 18)
    kw = dict(causal=True, softcap=30.0)
    o, lse = fa.fa_fwd_scored(q, k, v, **kw)
    want = fa.fa_bwd_scored(q, k, v, o, do, lse, deterministic=True, **kw)
    size = fa.fa_bwd_scored_workspace_size(1, 4, 2, 700, 64)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = []
    for _ in range(8):
        got.append(fa.fa_bwd_scored(q, k, v, o, do, lse, deterministic=True, stream=s, **kw))
        torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    fa.fa_sync_check()
    for g in got:
        for a, b in zip(g, want):
            assert torch.equal(a, b)


def test_sizes_past_int_are_refused():
    plan = torch.empty(16, dtype=torch.uint8, device="cuda")
    for B, N in ((2 ** 31, 1), (1, 2 ** 31)):
        with pytest.raises(ValueError):
            fa.fa_mask_plan(B, N, plan=plan)
    with pytest.raises(OverflowError):
        fa.fa_mask_plan(2 ** 70, 1, plan=plan)


def test_many_heads_in_runs_agree_with_their_rows_alone():
    # So many heads that the backward works on them in runs (the last one shorter): the bits of the
    # same rows in calls too small for that.
    B, H, N, d = 25, 16, 512, 128
    q, k, v, do = _inputs(B, H, H, N, d, 41)
    o, lse = fa.fa_fwd_scored(q, k, v, causal=True)
    for det in (True, False):
        grads = fa.fa_bwd_scored(q, k, v, o, do, lse, causal=True, deterministic=det)
        for b in range(0, B, 5):
            part = [t[b:b + 5] for t in (q, k, v, o, do, lse)]
            for name, whole, alone in zip(("dq", "dk", "dv"), grads, fa.fa_bwd_scored(*part, causal=True, deterministic=det)):
                if det or name != "dq":  # (dq's fp32 sums have no fixed order)
                    assert torch.equal(whole[b:b + 5], alone), (name, b)
    fa.fa_sync_check()


def _spoil(x, at, value):
    y = x.clone()
    y[at] = value
    return y


# 300 rows of two heads are halved units, 400 rows of 80 heads units of two tiles.
@pytest.mark.parametrize("B,H,N", [(1, 2, 300), (2, 40, 400)])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (0.0, True), (20.0, False), (20.0, True), (60.0, False), (60.0, True)])
@pytest.mark.parametrize("d", [64, 128])
def test_nan_and_infinities_come_through(B, H, N, cap, bias, d):
    # One entry of a key, or of a query, is NaN or infinite.  What the definition makes of it (NaN, or a
    # finite result where the cap or a weight of 0 absorbs an infinity) has to come out in the rows that
    # see it, and in no other.
    from oracle.scored import _score_error

    q, k, v, _ = _inputs(B, H, H, N, d, 51)
    slopes = _slopes(H) if bias else None
    s0 = [float(slopes[0])] if bias else None
    clean = [host_f64(t[:1, :1]) for t in (q, k, v)]
    # The bound of scored_forward, with sum P |v| replaced by the largest |v| (P of the spoilt rows is another).
    err = _score_error(clean[0][0, 0], clean[1][0, 0], d ** -0.5, cap, s0[0] if bias else 0.0, d)
    for name, at in (("key", 77), ("query", 200)):
        for value in (float("nan"), float("inf"), float("-inf")):
            spoilt = [_spoil(t, (0, 0, at, 5), value) if name == n else t for n, t in (("query", q), ("key", k))]
            for causal in (True, False):
                o, lse = fa.fa_fwd_scored(*spoilt, v, causal=causal, softcap=cap, slopes=slopes)
                fa.fa_sync_check()
                with np.errstate(invalid="ignore"):
                    o_ref, lse_ref, _, _ = scored_forward(*(host_f64(t[:1, :1]) for t in (*spoilt, v)), d ** -0.5, causal, cap, s0)
                ob = (2.0 ** -8 + 3 * err) * 1.01 * np.abs(clean[2]).max() + 2.0 ** -8 * np.abs(o_ref)
                lb = 2 * err + 4 * 2.0 ** -24 * np.abs(lse_ref)
                what = f"{name} {value} causal={causal}"
                for got, ref, bound, n in ((o[:1, :1], o_ref, ob, "O"), (lse[:1, :1], lse_ref, lb, "LSE")):
                    got = host_f64(got)
                    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{n} {what}: NaN in other rows than the definition's"
                    fin = ~np.isnan(ref)
                    assert (np.abs(got - ref)[fin] <= bound[fin]).all(), f"{n} {what}"
                assert torch.isfinite(o[-1, -1]).all() and torch.isfinite(lse[-1, -1]).all(), what


@pytest.mark.parametrize("cap,bias", [(0.0, False), (0.0, True), (20.0, False), (20.0, True)])
@pytest.mark.parametrize("H", [1, 64])  # key blocks whose steps are divided, and whole ones
def test_nan_in_a_key_reaches_the_gradients_of_its_document(H, cap, bias):
    # Two documents: every row of the first sees the key, so dK and dV of all its keys are NaN; those of
    # the second keep their values.
    B, N, d, cut = 1, 700, 64, 333
    q, k, v, do = _inputs(B, H, H, N, d, 62)
    plan = _docs([[0, cut, N]], None, False, B, N)
    kw = dict(softcap=cap, slopes=_slopes(H) if bias else None, plan=plan)
    clean = fa.fa_bwd_scored(q, k, v, *_out(q, k, v, do, kw), **kw)
    k[0, 0, 77, 5] = float("nan")
    o, lse = fa.fa_fwd_scored(q, k, v, **kw)
    for det in (False, True):
        _, dk, dv = fa.fa_bwd_scored(q, k, v, o, do, lse, deterministic=det, **kw)
        fa.fa_sync_check()
        assert bool(torch.isnan(lse[0, 0, :cut]).all()) and bool(torch.isfinite(lse[0, 0, cut:]).all())
        for got, want in ((dk, clean[1]), (dv, clean[2])):
            assert bool(torch.isnan(got[0, 0, :cut]).all())
            assert torch.equal(got[0, 0, cut:], want[0, 0, cut:]) and torch.equal(got[0, 1:], want[0, 1:])


def _out(q, k, v, do, kw):
    o, lse = fa.fa_fwd_scored(q, k, v, **kw)
    return o, do, lse


@pytest.mark.parametrize("cap", [30.0, 200.0, 1e4, 1e6, 1e20])
@pytest.mark.parametrize("H,N", [(2, 300), (62, 400)])
def test_biased_scores_on_both_sides_far_below_the_cap(H, N, cap):
    # Keys on both sides of a row take the general form of the bias; the cap's error stays relative to the
    # score there, whatever the cap.
    B, d = 1, 64
    q, k, v, do = _inputs(B, H, H, N, d, 63)
    slopes = _slopes(H)
    o, lse = fa.fa_fwd_scored(q, k, v, softcap=cap, slopes=slopes)
    grads = fa.fa_bwd_scored(q, k, v, o, do, lse, softcap=cap, slopes=slopes)
    fa.fa_sync_check()
    x = [host_f64(t) for t in (q, k, v, do)]
    args = (d ** -0.5, False, cap, slopes.cpu().numpy())
    o_ref, lse_ref, ob, lb = scored_forward(*x[:3], *args)
    _check(o, o_ref, ob, "O")
    _check(lse, lse_ref, lb, "LSE")
    refs, bounds = scored_backward(*x, *args)
    for name, a, ref, bd in zip(("dq", "dk", "dv"), grads, refs, bounds):
        _check(a, ref, bd, name)


@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("H,Hkv", [(2, 1), (64, 32)])  # key blocks whose steps are divided, and whole ones
@pytest.mark.parametrize("what,value", [("k", float("nan")), ("k", float("inf")), ("v", float("nan")), ("do", float("inf"))])
def test_nan_and_infinities_come_through_deterministic_dq(what, value, H, Hkv, cap):
    B, N, d = 1, 700, 64
    t = dict(zip(("q", "k", "v", "do"), _inputs(B, H, Hkv, N, d, 64)))
    t[what][0, 0, 300, 5] = value
    q, k, v, do = t["q"], t["k"], t["v"], t["do"]
    kw = dict(causal=True, softcap=cap, slopes=_slopes(H))
    o, lse = fa.fa_fwd_scored(q, k, v, **kw)
    want = fa.fa_bwd_scored(q, k, v, o, do, lse, **kw)[0]
    got = fa.fa_bwd_scored(q, k, v, o, do, lse, deterministic=True, **kw)[0]
    fa.fa_sync_check()
    bad = ~torch.isfinite(want)
    assert bool(bad.any()) and bool(torch.isnan(got[bad]).all())
    other = slice(H // Hkv, None)  # heads that read another key/value head
    assert bool(torch.isfinite(got[:, other]).all())


@pytest.mark.parametrize("deterministic", [False, True])
@pytest.mark.parametrize("H,Hkv", [(2, 1), (64, 64)])  # key blocks whose steps are divided, and whole ones
def test_masks_that_break_the_contract_give_finite_values_inside_the_outputs(H, Hkv, deterministic):
    # Offsets that decrease or leave the row, a plan of longer rows, arbitrary bytes: any mask, but outputs that
    # are finite (an LSE may be -inf) and nothing written beside them.
    B, N, d = 2, 400, 64
    q, k, v, do = _inputs(B, H, Hkv, N, d, 65)
    plans = [_docs([cu, cu], [[7, -3, 2 ** 31 - 1]] * B, True, B, N)
             for cu in ([-50, 300, 100, 9999], [390, 10, 380, 20], [500, 600, 700, 800], [-9, -8, -7, -6])]
    plans.append(fa.fa_mask_plan(1, B * N, device="cuda"))
    plans.append(torch.randint(0, 256, (16 * B * N,), dtype=torch.uint8, generator=torch.Generator().manual_seed(4)).cuda())
    for plan in plans:
        bufs = [torch.full((B, h + 2, N, d), 3.0, dtype=torch.bfloat16, device="cuda") for h in (H, H, Hkv, Hkv)]
        lbuf = torch.full((B * H * N + 512,), 3.0, device="cuda")
        views = [x[:, 1:-1] for x in bufs]
        o, lse = fa.fa_fwd_scored(q, k, v, o=views[0], lse=lbuf[256:-256].view(B, H, N), plan=plan)
        fa.fa_bwd_scored(q, k, v, o, do, lse, *views[1:], plan=plan, deterministic=deterministic)
        fa.fa_sync_check()
        for x, view in zip(bufs, views):
            assert bool(torch.isfinite(view).all())
            assert bool((x[:, 0] == 3).all()) and bool((x[:, -1] == 3).all())
        assert bool((torch.isfinite(lse) | torch.isneginf(lse)).all())
        assert bool((lbuf[:256] == 3).all()) and bool((lbuf[-256:] == 3).all())
