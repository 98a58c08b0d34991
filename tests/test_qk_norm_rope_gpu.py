"""Norm and rotation of queries and keys on the GPU, and its gradient, against the float64 oracle."""

import numpy as np
import pytest
import torch

import io_aware_exact_fwd_gb300 as fa
from oracle import qk_norm_rope, qk_norm_rope_backward

from gpu_util import host_f64, report

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def _freq(rot, base=10000.0):
    return torch.tensor([base ** (-i / rot) for i in range(0, rot, 2)], dtype=torch.float32, device="cuda") if rot else None


def _pair(case, g, factor=1.0):
    B, N, H, Hkv, d, layout, dtype = (case[x] for x in ("B", "N", "H", "Hkv", "d", "layout", "dtype"))
    rand = lambda *s: (factor * torch.randn(*s, generator=g)).to(dtype).cuda()
    if layout == "qkv":
        x = rand(B, N, H + 2 * Hkv, d).transpose(1, 2)
        return x[:, :H], x[:, H:H + Hkv]
    if layout == "bnhd":
        return rand(B, N, H, d).transpose(1, 2), rand(B, N, Hkv, d).transpose(1, 2)
    return rand(B, H, N, d), rand(B, Hkv, N, d)


def _case(B=1, N=1, H=1, Hkv=1, d=64, rot=None, pairs=False, norm=True, weight="float32", far=0, layout="bhnd",
          dtype=torch.bfloat16, eps=1e-6, factor=1.0):
    return dict(B=B, N=N, H=H, Hkv=Hkv, d=d, rot=d if rot is None else rot, pairs=pairs, norm=norm, weight=weight, far=far,
                layout=layout, dtype=dtype, eps=eps, factor=factor)


CASES = [
    _case(),
    _case(N=7, H=3, d=128, rot=0),
    _case(B=2, N=129, H=4, Hkv=2, rot=32, pairs=True, layout="bnhd"),
    _case(B=3, N=33, H=5, Hkv=5, d=128, rot=16, weight="none", layout="qkv", far=2 ** 31 - 1),
    _case(B=1, N=16, H=8, Hkv=2, far=40000, layout="qkv", dtype=torch.float16),
    _case(B=2, N=65, H=16, Hkv=1, d=128, pairs=True, weight="own", dtype=torch.float16, far=100),
    _case(B=1, N=300, H=2, Hkv=7, d=128, norm=False, weight="none", layout="bnhd"),
    _case(B=2, N=50, H=3, Hkv=3, rot=48, norm=False, weight="none", pairs=True, dtype=torch.float16, far=-5000),
    _case(B=1, N=1500, H=12, Hkv=3, d=128, weight="own", layout="qkv", far=10 ** 6),
    _case(B=1, N=40, H=30, Hkv=10, eps=0.5, factor=0.01, layout="bhnd"),
    _case(B=1, N=2, H=200, Hkv=9, d=128, layout="qkv"),
]


def _state(case, seed=1):
    g = torch.Generator().manual_seed(seed)
    q, k = _pair(case, g, case["factor"])
    gq, gk = _pair(case, g)
    wtype = torch.float32 if case["weight"] == "float32" else case["dtype"]
    qw, kw = (None if case["weight"] == "none" else (1 + 0.3 * torch.randn(case["d"], generator=g)).to(wtype).cuda() for _ in range(2))
    pos = None
    if case["far"]:
        lo, hi = min(case["far"], 0), max(case["far"], 0)
        pos = torch.randint(lo, hi + 1, (case["B"], case["N"]), generator=g, dtype=torch.int64).to(torch.int32)
        pos[0, 0] = case["far"]
        pos = pos.cuda()
    kw_ = dict(q_weight=qw, k_weight=kw, inv_freq=_freq(case["rot"]), positions=pos, eps=case["eps"], norm=case["norm"],
               interleaved=case["pairs"])
    ref = lambda w: dict(w=None if w is None else host_f64(w), inv_freq=None if not case["rot"] else _freq(case["rot"]).cpu().numpy(),
                         positions=None if pos is None else pos.cpu().numpy(), eps=case["eps"], norm=case["norm"],
                         interleaved=case["pairs"], half=HALF[case["dtype"]])
    return q, k, gq, gk, kw_, (ref(qw), ref(kw))


def _within(got, ref, bound, what):
    share = float((np.abs(host_f64(got) - ref) / bound).max(initial=0.0))
    assert share <= 1.0, f"{what}: {share} of its bound"
    return share


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(case):
    q, k, _, _, kw, refs = _state(case)
    got = fa.fa_qk_norm_rope(q, k, **kw)
    fa.fa_sync_check()
    shares = [_within(y, *qk_norm_rope(host_f64(x), **r), what) for y, x, r, what in zip(got, (q, k), refs, "qk")]
    report(f"qk_norm_rope {case} (shares of the bounds)", q=shares[0], k=shares[1])


@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(case):
    q, k, gq, gk, kw, refs = _state(case)
    got = fa.fa_qk_norm_rope_bwd(q, k, gq, gk, **kw)
    again = fa.fa_qk_norm_rope_bwd(q, k, gq, gk, **kw)
    fa.fa_sync_check()
    for i, (x, g, r) in enumerate(((q, gq, refs[0]), (k, gk, refs[1]))):
        (dx, dw), (bx, bw) = qk_norm_rope_backward(host_f64(x), host_f64(g), **r)
        _within(got[i], dx, bx, "dx")
        assert (got[2 + i] is None) == (dw is None)
        if dw is not None:
            _within(got[2 + i], dw, bw, "dw")
            assert got[2 + i].dtype == torch.float32
    assert all(a is b or torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("case", [_case(N=1250, H=12, Hkv=1, d=128), _case(N=2600, H=12, Hkv=3, layout="qkv", dtype=torch.float16),
                                  _case(B=3, N=1667, H=7, Hkv=7), _case(B=2, N=1217, H=24, Hkv=5, layout="bnhd")], ids=str)
def test_tokens_in_rounds(case):
    # As many tokens that warps take some after each other, with all of their heads or a part.
    test_forward(case)
    test_backward(case)


def test_in_place_and_into_views():
    case = _case(B=2, N=70, H=6, Hkv=2, d=128, layout="qkv", rot=64)
    q, k, gq, gk, kw, _ = _state(case)
    want = fa.fa_qk_norm_rope(q, k, **kw)
    back = fa.fa_qk_norm_rope_bwd(q, k, gq, gk, **kw)
    assert want[0].stride() == (70 * 6 * 128, 128, 6 * 128, 1)  # heads beside each other, as they came
    qo = torch.full((2, 8, 70, 136), 3.0, dtype=torch.bfloat16, device="cuda")
    got = fa.fa_qk_norm_rope(q, k, q_out=qo[:, 1:7, :, :128], k_out=torch.empty_like(want[1]), **kw)
    dq = fa.fa_qk_norm_rope_bwd(q, k, gq, gk, dq=gq, dk=gk, **kw)
    fused = q._base if q._base is not None else None
    fa.fa_qk_norm_rope(q, k, q_out=q, k_out=k, **kw)
    fa.fa_sync_check()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and fused is not None
    assert bool((qo[:, 0] == 3).all() and (qo[:, 7] == 3).all() and (qo[..., 128:] == 3).all())
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert all(torch.equal(a, b) for a, b in zip(dq, back))


def test_layouts_give_the_same_bits():
    case = _case(B=2, N=90, H=6, Hkv=3, d=64, rot=32)
    q, k, gq, gk, kw, _ = _state(case)
    other = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in (q, k, gq, gk)]
    a, b = fa.fa_qk_norm_rope(q, k, **kw), fa.fa_qk_norm_rope(*other[:2], **kw)
    c, e = fa.fa_qk_norm_rope_bwd(q, k, gq, gk, **kw), fa.fa_qk_norm_rope_bwd(*other, **kw)
    fa.fa_sync_check()
    assert all(torch.equal(x, y) for x, y in zip(a + c[:2], b + e[:2]))
    assert b[0].stride(1) < b[0].stride(2) and a[0].is_contiguous()


def test_no_tokens_and_no_heads():
    kw = dict(inv_freq=_freq(64), q_weight=torch.ones(64, device="cuda"), k_weight=torch.ones(64, device="cuda"))
    x = lambda *s: torch.randn(*s, dtype=torch.float32, device="cuda").bfloat16()
    q, k = fa.fa_qk_norm_rope(x(2, 3, 0, 64), x(2, 1, 0, 64), **kw)
    assert q.shape == (2, 3, 0, 64) and k.shape == (2, 1, 0, 64)
    for shapes in (((2, 3, 0, 64), (2, 1, 0, 64)), ((0, 3, 5, 64), (0, 1, 5, 64))):
        out = fa.fa_qk_norm_rope_bwd(*(x(*s) for s in shapes + shapes), **kw)
        fa.fa_sync_check()
        assert not out[2].any() and not out[3].any()
    q = x(1, 4, 9, 64)
    both = fa.fa_qk_norm_rope(q, x(1, 1, 9, 64), **kw)
    alone = fa.fa_qk_norm_rope(q, x(1, 0, 9, 64), **kw)
    as_keys = fa.fa_qk_norm_rope(x(1, 0, 9, 64), q, **kw)
    back = fa.fa_qk_norm_rope_bwd(q, x(1, 0, 9, 64), q, x(1, 0, 9, 64), **kw)
    fa.fa_sync_check()
    assert torch.equal(both[0], alone[0]) and torch.equal(both[0], as_keys[1]) and not back[3].any() and back[2].any()


def test_rows_of_zeros_and_of_nan():
    q = torch.zeros(1, 2, 5, 64, dtype=torch.bfloat16, device="cuda")
    q[0, 1, 3] = float("nan")
    k = torch.ones(1, 1, 5, 64, dtype=torch.bfloat16, device="cuda")
    y, z = fa.fa_qk_norm_rope(q, k, inv_freq=_freq(64))
    dq, dk, _, _ = fa.fa_qk_norm_rope_bwd(q, k, torch.ones_like(q), torch.ones_like(k), inv_freq=_freq(64))
    fa.fa_sync_check()
    for t in (y, dq):
        assert t[0, 1, 3].isnan().all() and t.isnan().sum() == 64
    assert not y[0, 0].any() and z.isfinite().all() and dk.isfinite().all()


def test_negative_and_large_frequencies():
    f = torch.tensor([-1.0, 3.0e5, -0.0, 2.0 ** 40, 1e-30, 0.75, 2.5, 1.0], dtype=torch.float32, device="cuda")
    case = _case(N=9, H=2, far=-70000)
    q, k, _, _, kw, refs = _state(case)
    kw["inv_freq"] = f
    got = fa.fa_qk_norm_rope(q, k, **kw)
    fa.fa_sync_check()
    # 2^40 times a position of 17 bits: its angle needs whole-number reduction, so the oracle gets the frequency's rest modulo 2 pi.
    two_pi = 6283185307179586476925286766559005768394338798750211641949889184615632812572  # 2 pi * 10^75
    rest = np.array([float((int(x * 2 ** 60) * 10 ** 75 % (two_pi * 2 ** 60)) / (10 ** 75 * 2 ** 60)) if abs(x) > 1e3 else float(x)
                     for x in f.cpu().tolist()])
    pos = kw["positions"].cpu().numpy()
    for y, x, r in zip(got, (q, k), refs):
        r["inv_freq"] = rest
        ref, bound = qk_norm_rope(host_f64(x), **r)
        # (the rest in 64 bits times positions up to 7e4 and 2 pi: 4e-11, below the bound's angle)
        _within(y, ref, bound, "large frequencies")
    assert pos.min() < -1


def test_captured_and_on_another_stream():
    case = _case(B=1, N=700, H=8, Hkv=2, d=128, layout="bnhd", far=5000)
    q, k, gq, gk, kw, _ = _state(case)
    want = fa.fa_qk_norm_rope(q, k, **kw) + fa.fa_qk_norm_rope_bwd(q, k, gq, gk, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fa.fa_qk_norm_rope(q, k, stream=side, **kw) + fa.fa_qk_norm_rope_bwd(q, k, gq, gk, stream=side, **kw)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fa.fa_qk_norm_rope(q, k, **kw) + fa.fa_qk_norm_rope_bwd(q, k, gq, gk, **kw)
    for _ in range(2):
        for t in got:
            t.fill_(9)
        graph.replay()
        fa.fa_sync_check()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_training_step_with_attention():
    """Norm and rotation, capped attention, and back: the gradients of q, k and the weights through both, against
    differentiating the plain form in 64 bits."""
    B, H, Hkv, N, d, cap = 1, 4, 2, 96, 64, 20.0
    g = torch.Generator().manual_seed(5)
    q, do = (torch.randn(B, N, H, d, generator=g).bfloat16().cuda().transpose(1, 2) for _ in range(2))
    k, v = (torch.randn(B, N, Hkv, d, generator=g).bfloat16().cuda().transpose(1, 2) for _ in range(2))
    qw, kw = ((1 + 0.2 * torch.randn(d, generator=g)).cuda() for _ in range(2))
    prep = dict(q_weight=qw, k_weight=kw, inv_freq=_freq(d))
    qr, kr = fa.fa_qk_norm_rope(q, k, **prep)
    o, lse = fa.fa_fwd_scored(qr, kr, v, causal=True, softcap=cap)
    dqr, dkr, dv = fa.fa_bwd_scored(qr, kr, v, o, do, lse, causal=True, softcap=cap)
    dq, dk, dqw, dkw = fa.fa_qk_norm_rope_bwd(q, k, dqr, dkr, **prep)
    fa.fa_sync_check()
    leaves = [t.double().cpu().requires_grad_() for t in (q, k, v, qw, kw)]
    angle = torch.arange(N).double()[:, None] * _freq(d).double().cpu()
    c, s = torch.cos(angle), torch.sin(angle)

    def plain(x, w):
        y = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w
        a, b = y[..., :d // 2], y[..., d // 2:]
        return torch.cat((a * c - b * s, a * s + b * c), -1)

    kk, vv = (t.repeat_interleave(H // Hkv, 1) for t in (plain(leaves[1], leaves[4]), leaves[2]))
    a = cap * torch.tanh(plain(leaves[0], leaves[3]) @ kk.transpose(2, 3) * d ** -0.5 / cap)
    a = a.masked_fill(torch.ones(N, N, dtype=torch.bool).triu(1), float("-inf"))
    want = torch.autograd.grad(torch.softmax(a, -1) @ vv, leaves, do.double().cpu())
    for got, ref in zip((dq, dk, dv, dqw, dkw), want):
        # Seven bf16 roundings on the way (q, k, P, O, dS, dQ or dK, the result), 2^-8 each of sums that do not exceed the
        # gradient's largest entries by much: the parity bar of the backward, 2e-2 of the largest, takes them.
        assert (got.double().cpu() - ref).abs().max() <= 2e-2 * ref.abs().max()


def test_refusals_in_the_binding():
    q, k = (torch.zeros(1, h, 8, 64, dtype=torch.bfloat16, device="cuda") for h in (4, 2))
    w, f = torch.ones(64, device="cuda"), _freq(64)
    for bad, kind in ((dict(q_weight=w.half()), ValueError), (dict(q_weight=w, k_weight=w.bfloat16()), ValueError),
                      (dict(q_weight=w[:32]), ValueError), (dict(inv_freq=f.double()), ValueError),
                      (dict(inv_freq=f, positions=torch.zeros(1, 8, dtype=torch.int64, device="cuda")), ValueError),
                      (dict(inv_freq=f, positions=torch.zeros(1, 7, dtype=torch.int32, device="cuda")), ValueError),
                      (dict(inv_freq=f.cpu()), ValueError), (dict(q_weight=w, norm=False), fa.FAError),
                      (dict(inv_freq=f[:7]), fa.FAError), (dict(eps=0.0), fa.FAError), (dict(q_out=q.half()), TypeError)):
        with pytest.raises(kind):
            fa.fa_qk_norm_rope(q, k, **bad)
    with pytest.raises(TypeError):
        fa.fa_qk_norm_rope(q.float(), k)
    with pytest.raises(TypeError):
        fa.fa_qk_norm_rope(q, k.half())
    with pytest.raises(ValueError):
        fa.fa_qk_norm_rope(q, k[:, :, :4])
    with pytest.raises(ValueError):
        fa.fa_qk_norm_rope_bwd(q, k, q, k[:, :, :4])
    with pytest.raises(fa.FAError):
        fa.fa_qk_norm_rope_bwd(q, k, q, k, q_weight=w, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))


# Columns past the rotated ones: each is its own, whatever stands in the others.
@pytest.mark.parametrize("d,rot,pairs", [(64, 0, False), (64, 16, False), (64, 16, True), (128, 48, False), (128, 48, True)])
def test_infinities_and_nan_in_columns_that_are_not_rotated(d, rot, pairs):
    g = torch.Generator().manual_seed(7)
    kw = dict(inv_freq=_freq(rot), norm=False, interleaved=pairs)
    clean = [torch.randn(1, h, 9, d, generator=g).bfloat16() for h in (3, 2)]
    x = [t.clone() for t in clean]
    for t, c in zip(x, clean):
        t[0, 0, 1, rot + 3] = float("inf")
        t[0, 1, 2, d - 1] = float("-inf")
        t[0, 0, 4, rot + 8] = float("nan")
        t[0, 1, 5, rot:] = -0.0
        t[0, 1, 6, rot:rot + 2] = torch.tensor([float("inf"), float("nan")])
        c[..., rot:][~torch.isfinite(t[..., rot:])] = 0.0
    x, clean = ([t.cuda() for t in y] for y in (x, clean))
    for call in (lambda q, k: fa.fa_qk_norm_rope(q, k, **kw), lambda q, k: fa.fa_qk_norm_rope_bwd(q, k, q, k, **kw)[:2]):
        got, want = call(*x), call(*clean)
        fa.fa_sync_check()
        for y, z, t in zip(got, want, x):
            nan = t[..., rot:].isnan()
            assert torch.equal(y[..., rot:].isnan(), nan)
            assert torch.equal(y[..., rot:].view(torch.int16)[~nan], t[..., rot:].view(torch.int16)[~nan])
            assert torch.equal(y[..., :rot], z[..., :rot])


@pytest.mark.parametrize("d,rot,pairs", [(64, 0, False), (64, 32, True), (128, 32, False)])
def test_an_infinite_gradient_reaches_its_own_weight_alone(d, rot, pairs):
    case = _case(N=40, H=2, d=d, rot=rot, pairs=pairs)
    q, k, gq, gk, kw, _ = _state(case)
    gq[0, 1, 7, rot + 5], gk[0, 0, 3, d - 1] = 0.0, 0.0
    want = fa.fa_qk_norm_rope_bwd(q, k, gq, gk, **kw)
    gq[0, 1, 7, rot + 5], gk[0, 0, 3, d - 1] = float("inf"), float("nan")
    got = fa.fa_qk_norm_rope_bwd(q, k, gq, gk, **kw)
    fa.fa_sync_check()
    for y, z, at in ((got[2], want[2], rot + 5), (got[3], want[3], d - 1)):
        rest = torch.arange(d, device="cuda") != at
        assert not y[at].isfinite() and torch.equal(y[rest], z[rest])


def test_norm_of_a_row_with_an_infinity():
    # Its mean square is infinite: finite values become 0, the infinity is divided by itself.
    x = torch.ones(1, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    x[0, 0, 1, 40] = float("inf")
    y, _ = fa.fa_qk_norm_rope(x, x, inv_freq=_freq(32))
    fa.fa_sync_check()
    assert y[0, 0, 0].isfinite().all() and y[0, 0, 1, 40].isnan() and y[0, 0, 1].isnan().sum() == 1 and y[0, 0, 1].nansum() == 0


@pytest.mark.parametrize("rows", ["last", "few"])
@pytest.mark.parametrize("case", [_case(N=1250, H=12, Hkv=1, d=128), _case(N=2600, H=12, Hkv=3, layout="qkv", dtype=torch.float16),
                                  _case(B=3, N=1667, H=7, Hkv=7), _case(B=2, N=1217, H=24, Hkv=5, layout="bnhd")], ids=str)
def test_weights_gradient_of_few_rows_among_many(case, rows):
    # One row that is lost, or one that is counted twice, is a large part of what is left: the bound of all rows' sum
    # (2^-24 of it for each) would not see it.
    q, k, gq, gk, kw, refs = _state(case)
    for g in (gq, gk):
        B, H, N, _ = g.shape
        keep = torch.zeros(B, N, H, dtype=torch.bool)  # (tokens first, as warps take them)
        if rows == "last":
            keep[-1, -1, -1] = True
        else:
            keep.view(-1)[::997] = True
        g.masked_fill_(~keep.transpose(1, 2)[..., None].cuda(), 0.0)
    got = fa.fa_qk_norm_rope_bwd(q, k, gq, gk, **kw)
    fa.fa_sync_check()
    for dw, x, g, r in zip(got[2:], (q, k), (gq, gk), refs):
        (_, ref), (_, bound) = qk_norm_rope_backward(host_f64(x), host_f64(g), **r)
        _within(dw, ref, bound, "dw")


@pytest.mark.parametrize("which", ["q_weight", "k_weight"])
def test_one_weight_alone(which):
    case = _case(B=2, N=40, H=4, Hkv=2, weight="own")
    q, k, gq, gk, kw, _ = _state(case)
    both, back = fa.fa_qk_norm_rope(q, k, **kw), fa.fa_qk_norm_rope_bwd(q, k, gq, gk, **kw)
    other = "k_weight" if which == "q_weight" else "q_weight"
    side = 0 if which == "q_weight" else 1
    kw[other] = None
    one, grads = fa.fa_qk_norm_rope(q, k, **kw), fa.fa_qk_norm_rope_bwd(q, k, gq, gk, **kw)
    kw[other] = torch.ones_like(kw[which])
    ones = fa.fa_qk_norm_rope(q, k, **kw)
    fa.fa_sync_check()
    assert torch.equal(one[side], both[side]) and torch.equal(one[1 - side], ones[1 - side])
    assert torch.equal(grads[side], back[side]) and torch.equal(grads[2 + side], back[2 + side]) and grads[3 - side] is None
