"""Refusals of the scored-attention and paged-cache entry points: bad arguments return the
documented status before any device work (the addresses here are never dereferenced)."""

import ctypes
import os

import pytest
import torch

import io_aware_exact_fwd_gb300 as fa

FAKE = 0x10000
INV, UNSUP, MIS, WS = 1, 2, 3, 6
vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fa.library_path()):
        from io_aware_exact_fwd_gb300 import _build

        _build.build()
    return fa.load_library()


def _st(*s):
    return (ctypes.c_int64 * len(s))(*s)


def test_mask_plan(lib):
    def call(cu=FAKE, prefix=FAKE, n=3, plan=FAKE, nb=1 << 20, B=2, N=100, causal=1):
        return lib.fa_mask_plan(vp(cu), vp(prefix), n, vp(plan), nb, B, N, causal, vp(0))
    assert lib.fa_mask_plan_size(2, 100) == 16 * 200
    assert lib.fa_mask_plan_size(0, 100) == 0 and lib.fa_mask_plan_size(1 << 16, 1 << 16) == 0
    assert call(B=-1) == INV and call(N=-1) == INV and call(n=0) == INV and call(causal=2) == INV
    assert call(cu=0, n=2) == INV
    assert call(B=1 << 16, N=1 << 16) == UNSUP
    assert call(plan=0) == WS and call(nb=16 * 200 - 1) == WS
    assert call(plan=FAKE + 8) == MIS and call(cu=FAKE + 2) == MIS and call(prefix=FAKE + 1) == MIS
    assert call(B=0, plan=0) == 0 and call(N=0, plan=0) == 0


BAD_COMMON = [
    (dict(B=-1), INV), (dict(H=-2), INV), (dict(N=-1), INV), (dict(Hkv=0), INV), (dict(Hkv=3), INV), (dict(Hkv=-1), INV),
    (dict(causal=2), INV), (dict(causal=1, plan=FAKE, pb=1 << 30), INV), (dict(d=96), UNSUP), (dict(d=256), UNSUP),
    (dict(scale=0.0), INV), (dict(scale=float("nan")), INV), (dict(cap=-1.0), INV), (dict(cap=float("inf")), INV),
    (dict(cap=float("nan")), INV), (dict(cap=1e-39), INV), (dict(cap=3e38), INV), (dict(plan=FAKE, pb=16 * 200 - 1), WS), (dict(plan=FAKE + 4, pb=1 << 20), MIS),
    (dict(q=0), INV), (dict(v=FAKE + 2), MIS), (dict(lse=FAKE + 2), MIS), (dict(slopes=FAKE + 2), MIS),
    (dict(qs=_st(63, 6400, 25600)), MIS), (dict(qs=_st(56, 6400, 25600)), INV), (dict(qs=_st(64, 0, 25600)), INV),
    (dict(qs=_st(64, -64, 25600)), INV), (dict(B=1 << 16, H=1 << 16), UNSUP), (dict(B=64, H=1 << 14, N=1 << 14), UNSUP),
]


@pytest.mark.parametrize("bad,status", BAD_COMMON)
@pytest.mark.parametrize("which", ["fwd", "bwd"])
def test_scored_refusals(lib, which, bad, status):
    a = dict(q=FAKE, qs=None, k=FAKE, v=FAKE, lse=FAKE, B=2, H=4, Hkv=2, N=100, d=64, plan=0, pb=0, causal=0, scale=0.125,
             cap=0.0, slopes=0, nb=1 << 40, det=0, ws=FAKE * 16, dq=FAKE)
    a.update(bad)
    mask = (a["B"], a["H"], a["Hkv"], a["N"], a["d"], vp(a["plan"]), a["pb"], a["causal"], a["scale"], a["cap"], vp(a["slopes"]))
    if which == "fwd":
        got = lib.fa_fwd_scored(vp(a["q"]), a["qs"], vp(a["k"]), None, vp(a["v"]), None, vp(FAKE), None, vp(a["lse"]), *mask, vp(0))
    else:
        got = lib.fa_bwd_scored(vp(a["q"]), a["qs"], vp(a["k"]), None, vp(a["v"]), None, vp(FAKE), None, vp(FAKE), None,
                                vp(a["lse"]), vp(a["dq"]), None, vp(FAKE), None, vp(FAKE), None, vp(a["ws"]), a["nb"], *mask,
                                a["det"], vp(0))
    assert got == status


def test_scored_backward_workspace(lib):
    need = lib.fa_bwd_scored_workspace_size(2, 4, 2, 100, 64)
    assert need >= 2 * 4 * 100 * 64 * 4
    assert lib.fa_bwd_scored_workspace_size(2, 4, 3, 100, 64) == 0 and lib.fa_bwd_scored_workspace_size(2, 4, 2, 100, 80) == 0

    def call(ws, nb, det=0):
        t = (vp(FAKE), None)
        return lib.fa_bwd_scored(*t, *t, *t, *t, *t, vp(FAKE), *t, *t, *t, vp(ws), nb, 2, 4, 2, 100, 64, vp(0), 0, 0, 0.1, 0.0,
                                 vp(0), det, vp(0))
    assert call(0, need) == WS and call(FAKE, need - 1) == WS and call(FAKE + 16, need) == MIS and call(FAKE, need, 2) == INV


def test_deterministic_backward_of_too_many_heads(lib):
    # (the maxima of a key/value head are a grid's second axis)
    t = (vp(FAKE), None)
    for det, status in ((1, UNSUP), (0, WS)):
        assert lib.fa_bwd_scored(*t, *t, *t, *t, *t, vp(FAKE), *t, *t, *t, vp(0), 0, 1, 65536, 65536, 16, 64, vp(0), 0, 0, 0.1,
                                 0.0, vp(0), det, vp(0)) == status


def test_empty_problems_are_no_ops(lib):
    n = vp(0)
    assert lib.fa_fwd_scored(n, None, n, None, n, None, n, None, n, 0, 4, 2, 10, 64, n, 0, 0, 0.1, 0.0, n, n) == 0
    assert lib.fa_fwd_scored(n, None, n, None, n, None, n, None, n, 2, 4, 2, 0, 64, n, 0, 1, 0.1, 0.0, n, n) == 0
    assert lib.fa_paged_append(n, None, n, None, n, None, n, None, n, 1, n, n, 0, 5, 1, 64, 16, 1, 1, 1, n) == 0
    assert lib.fa_paged_append(n, None, n, None, n, None, n, None, n, 1, n, n, 2, 0, 1, 64, 16, 1, 1, 1, n) == 0
    assert lib.fa_paged_decode(n, None, n, None, n, None, n, 1, n, n, None, n, n, 0, 0, 2, 1, 64, 16, 1, 1, 1, 0.1, 0.0, n, n) == 0


@pytest.mark.parametrize("bad,status", [
    (dict(B=-1), INV), (dict(Hkv=0), INV), (dict(n_pages=0), INV), (dict(max_pages=0), INV), (dict(ts=3), INV),
    (dict(dtype=0), INV), (dict(dtype=3), INV), (dict(d=80), UNSUP), (dict(page=8), UNSUP), (dict(page=24), UNSUP),
    (dict(page=2048), UNSUP), (dict(max_pages=1 << 27, ts=1 << 27), UNSUP), (dict(B=70000), UNSUP), (dict(kc=0), INV),
    (dict(table=0), INV), (dict(lens=0), INV), (dict(kc=FAKE + 8), MIS), (dict(table=FAKE + 2), MIS), (dict(x=0), INV),
    (dict(x=FAKE + 8), MIS), (dict(xs=_st(60, 512)), MIS), (dict(xs=_st(56, 512)), INV), (dict(cs=_st(64, 1024, 0)), INV),
])
@pytest.mark.parametrize("which", ["append", "decode"])
def test_paged_refusals(lib, which, bad, status):
    a = dict(B=2, Hkv=2, d=64, page=16, n_pages=9, max_pages=4, ts=4, dtype=1, kc=FAKE, table=FAKE, lens=FAKE, x=FAKE, xs=None,
             cs=None)
    a.update(bad)
    cache = (vp(a["kc"]), a["cs"], vp(FAKE), None, vp(a["table"]), a["ts"], vp(a["lens"]))
    if which == "append":
        got = lib.fa_paged_append(vp(a["x"]), a["xs"], vp(FAKE), None, *cache, vp(FAKE), a["B"], 5, a["Hkv"], a["d"], a["page"],
                                  a["n_pages"], a["max_pages"], a["dtype"], vp(0))
    else:
        got = lib.fa_paged_decode(vp(a["x"]), a["xs"], *cache, vp(FAKE), None, vp(FAKE), vp(FAKE), 1 << 40, a["B"], 4, a["Hkv"],
                                  a["d"], a["page"], a["n_pages"], a["max_pages"], a["dtype"], 0.1, 0.0, vp(0), vp(0))
    assert got == status


def test_paged_decode_refusals(lib):
    def call(H=4, scale=0.1, cap=0.0, ws=FAKE, nb=1 << 40, o=FAKE, slopes=0, lse=FAKE):
        return lib.fa_paged_decode(vp(FAKE), None, vp(FAKE), None, vp(FAKE), None, vp(FAKE), 4, vp(FAKE), vp(o), None, vp(lse),
                                   vp(ws), nb, 2, H, 2, 64, 16, 9, 4, 1, scale, cap, vp(slopes), vp(0))
    need = lib.fa_paged_decode_workspace_size(2, 4, 2, 64)
    assert need > 0 and lib.fa_paged_decode_workspace_size(2, 3, 2, 64) == 0
    assert call(H=3) == INV and call(H=-4) == INV and call(scale=-1.0) == INV and call(cap=-2.0) == INV
    assert call(cap=1e-40) == INV and call(cap=3.3e38) == INV
    assert call(ws=0) == WS and call(nb=need - 1) == WS and call(ws=FAKE + 16) == MIS
    assert call(o=0) == INV and call(o=FAKE + 2) == MIS and call(lse=FAKE + 2) == MIS and call(slopes=FAKE + 2) == MIS


def test_binding_refuses_before_the_library(lib):
    x = torch.zeros(1, 2, 8, 64)
    with pytest.raises(TypeError):
        fa.fa_fwd_scored(x, x, x)
    with pytest.raises(ValueError):
        fa.fa_fwd_scored(x.bfloat16(), x.bfloat16(), x.bfloat16())  # not on a GPU
    with pytest.raises(ValueError):
        fa.fa_mask_plan(1, 8, torch.zeros(1, 3, dtype=torch.int32))
    with pytest.raises(TypeError):
        fa.fa_paged_decode(torch.zeros(1, 2, 64), x, x, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


@pytest.mark.parametrize("scale,cap", [(0.125, 1e38), (1e-8, 1e31), (1e-30, 1e10), (1e-38, 4.0)])
def test_caps_so_large_that_the_scores_lose_their_bits(lib, scale, cap):
    # 4 scale / softcap would be subnormal or 0 in fp32.
    t = (vp(FAKE), None)
    mask = (2, 4, 2, 100, 64, vp(0), 0, 0, scale, cap, vp(0))
    assert lib.fa_fwd_scored(*t, *t, *t, *t, vp(FAKE), *mask, vp(0)) == INV
    assert lib.fa_bwd_scored(*t, *t, *t, *t, *t, vp(FAKE), *t, *t, *t, vp(FAKE), 1 << 40, *mask, 0, vp(0)) == INV
    assert lib.fa_paged_decode(*t, *t, *t, vp(FAKE), 4, vp(FAKE), *t, vp(FAKE), vp(FAKE), 1 << 40, 2, 4, 2, 64, 16, 9, 4, 1, scale,
                               cap, vp(0), vp(0)) == INV
