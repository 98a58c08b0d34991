"""Refusals of norm and rotation, of the 8-bit paged cache and of its bookkeeping: bad arguments return the
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


@pytest.mark.parametrize("bad,status", [
    (dict(B=-1), INV), (dict(Hkv=0), INV), (dict(n_pages=0), INV), (dict(max_pages=0), INV), (dict(ts=3), INV),
    (dict(dtype=0), INV), (dict(dtype=3), INV), (dict(d=80), UNSUP), (dict(page=8), UNSUP), (dict(page=24), UNSUP),
    (dict(page=2048), UNSUP), (dict(max_pages=1 << 27, ts=1 << 27), UNSUP), (dict(B=70000), UNSUP), (dict(kc=0), INV),
    (dict(table=0), INV), (dict(lens=0), INV), (dict(kc=FAKE + 8), MIS), (dict(table=FAKE + 2), MIS), (dict(x=0), INV),
    (dict(x=FAKE + 8), MIS), (dict(xs=_st(60, 512)), MIS), (dict(xs=_st(56, 512)), INV), (dict(cs=_st(64, 1024, 0)), INV),
    (dict(cs=_st(72, 2048, 4096)), MIS), (dict(cs=_st(64, 1032, 4096)), MIS), (dict(ks=0), INV), (dict(vs=0), INV),
    (dict(ks=FAKE + 2), MIS), (dict(vs=FAKE + 1), MIS),
])
@pytest.mark.parametrize("which", ["append", "decode"])
def test_cache_refusals(lib, which, bad, status):
    a = dict(B=2, Hkv=2, d=64, page=16, n_pages=9, max_pages=4, ts=4, dtype=1, kc=FAKE, table=FAKE, lens=FAKE, x=FAKE, xs=None,
             cs=None, ks=FAKE, vs=FAKE)
    a.update(bad)
    cache = (vp(a["kc"]), a["cs"], vp(FAKE), None, vp(a["ks"]), vp(a["vs"]), vp(a["table"]), a["ts"], vp(a["lens"]))
    if which == "append":
        got = lib.fa_paged_append_fp8(vp(a["x"]), a["xs"], vp(FAKE), None, *cache, vp(FAKE), a["B"], 5, a["Hkv"], a["d"], a["page"],
                                      a["n_pages"], a["max_pages"], a["dtype"], vp(0))
    else:
        got = lib.fa_paged_decode_fp8(vp(a["x"]), a["xs"], *cache, vp(FAKE), None, vp(FAKE), vp(FAKE), 1 << 40, a["B"], 4, a["Hkv"],
                                      a["d"], a["page"], a["n_pages"], a["max_pages"], a["dtype"], 0.1, 0.0, vp(0), vp(0))
    assert got == status


def test_decode_refusals(lib):
    def call(H=4, scale=0.1, cap=0.0, ws=FAKE, nb=1 << 40, o=FAKE, slopes=0, lse=FAKE):
        return lib.fa_paged_decode_fp8(vp(FAKE), None, vp(FAKE), None, vp(FAKE), None, vp(FAKE), vp(FAKE), vp(FAKE), 4, vp(FAKE), vp(o),
                                       None, vp(lse), vp(ws), nb, 2, H, 2, 64, 16, 9, 4, 1, scale, cap, vp(slopes), vp(0))
    need = lib.fa_paged_decode_workspace_size(2, 4, 2, 64)
    assert call(H=3) == INV and call(H=-4) == INV and call(scale=-1.0) == INV and call(cap=-2.0) == INV
    assert call(cap=1e-40) == INV and call(cap=3.3e38) == INV
    assert call(ws=0) == WS and call(nb=need - 1) == WS and call(ws=FAKE + 16) == MIS
    assert call(o=0) == INV and call(o=FAKE + 2) == MIS and call(lse=FAKE + 2) == MIS and call(slopes=FAKE + 2) == MIS


@pytest.mark.parametrize("bad,status", [
    (dict(B=-1), INV), (dict(T=-1), INV), (dict(cap=-1), INV), (dict(width=-1), INV), (dict(width=0), INV), (dict(ts=3), INV),
    (dict(page=8), UNSUP), (dict(page=1040), UNSUP), (dict(B=65536), UNSUP), (dict(width=1 << 27, ts=1 << 27), UNSUP),
    (dict(table=0), INV), (dict(lens=0), INV), (dict(delta=0), INV), (dict(free=0), INV), (dict(count=0), INV), (dict(lo=0), INV),
    (dict(co=0), INV), (dict(cu=0), INV), (dict(status=0), INV), (dict(ws=0), WS), (dict(nb=27), WS), (dict(ws=FAKE + 2), MIS),
    (dict(table=FAKE + 2), MIS), (dict(lens=FAKE + 1), MIS), (dict(slots=FAKE + 4), MIS), (dict(pos=FAKE + 2), MIS),
    (dict(status=FAKE + 2), MIS),
])
def test_resize_refusals(lib, bad, status):
    a = dict(table=FAKE, ts=4, lens=FAKE, delta=FAKE, free=FAKE, cap=9, count=FAKE, lo=FAKE, co=FAKE, cu=FAKE, status=FAKE, slots=0, pos=0,
             T=5, ws=FAKE, nb=28, B=2, page=16, width=4)
    a.update(bad)
    p = lambda n: vp(a[n])
    assert lib.fa_paged_resize_workspace_size(2) == 28
    assert lib.fa_paged_resize(p("table"), a["ts"], p("lens"), p("delta"), p("free"), a["cap"], p("count"), p("lo"), p("co"), p("cu"),
                               p("status"), p("slots"), p("pos"), a["T"], p("ws"), a["nb"], a["B"], a["page"], a["width"], vp(0)) == status


def test_resize_workspace(lib):
    assert lib.fa_paged_resize_workspace_size(-1) == 0 and lib.fa_paged_resize_workspace_size(65536) == 0
    assert lib.fa_paged_resize_workspace_size(0) == 12


BAD_QK = [
    (dict(B=-1), INV), (dict(H=-1), INV), (dict(Hkv=-2), INV), (dict(N=-1), INV), (dict(d=96), UNSUP), (dict(rot=80), INV),
    (dict(rot=-16), INV), (dict(rot=24), UNSUP), (dict(rot=0), INV), (dict(freq=0), INV), (dict(norm=2), INV), (dict(pairs=-1), INV),
    (dict(dtype=0), INV), (dict(dtype=3), INV), (dict(wt=3), INV), (dict(wt=-1), INV), (dict(eps=0.0), INV),
    (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV), (dict(norm=0), INV), (dict(qw=FAKE + 2), MIS),
    (dict(kw=FAKE + 1, wt=1), MIS), (dict(freq=FAKE + 2), MIS), (dict(pos=FAKE + 2), MIS), (dict(q=0), INV), (dict(k=FAKE + 8), MIS),
    (dict(qs=_st(63, 6400, 25600)), MIS), (dict(qs=_st(56, 6400, 25600)), INV), (dict(qs=_st(64, 0, 25600)), INV),
    (dict(out=0), INV), (dict(out=FAKE + 4), MIS), (dict(B=1 << 16, N=1 << 16), UNSUP), (dict(H=1 << 30), UNSUP),
]


def _qk(lib, which, bad):
    a = dict(B=2, H=4, Hkv=2, N=100, d=64, rot=64, qw=FAKE, kw=FAKE, freq=FAKE, pos=0, norm=1, eps=1e-6, wt=0, pairs=0, dtype=1, q=FAKE,
             k=FAKE, qs=None, out=FAKE, ws=FAKE, nb=1 << 30, dqw=FAKE, dkw=FAKE)
    a.update(bad)
    p = lambda n: vp(a[n])
    tail = (a["B"], a["H"], a["Hkv"], a["N"], a["d"], a["rot"], a["norm"], a["eps"], a["wt"], a["pairs"], a["dtype"], vp(0))
    params = (p("qw"), p("kw"), p("freq"), p("pos"))
    if which == "fwd":
        return lib.fa_qk_norm_rope(p("q"), a["qs"], p("k"), None, *params, p("out"), None, vp(FAKE), None, *tail)
    return lib.fa_qk_norm_rope_bwd(p("q"), a["qs"], p("k"), None, vp(FAKE), None, vp(FAKE), None, *params, p("out"), None, vp(FAKE),
                                   None, p("dqw"), p("dkw"), p("ws"), a["nb"], *tail)


@pytest.mark.parametrize("bad,status", BAD_QK)
@pytest.mark.parametrize("which", ["fwd", "bwd"])
def test_qk_refusals(lib, which, bad, status):
    assert _qk(lib, which, bad) == status


@pytest.mark.parametrize("bad,status", [(dict(qw=0), INV), (dict(kw=0), INV), (dict(dqw=FAKE + 2), MIS), (dict(ws=0), WS), (dict(nb=8), WS),
                                        (dict(ws=FAKE + 2), MIS)])
def test_qk_backward_refusals(lib, bad, status):
    assert _qk(lib, "bwd", bad) == status


def test_empty_problems_are_no_ops(lib):
    nothing = dict(q=0, k=0, out=0, qw=0, kw=0, dqw=0, dkw=0, ws=0)
    for sizes in (dict(B=0), dict(N=0), dict(H=0, Hkv=0)):
        assert _qk(lib, "fwd", {**nothing, **sizes}) == 0 and _qk(lib, "bwd", {**nothing, **sizes}) == 0
    n = vp(0)
    assert lib.fa_paged_append_fp8(n, None, n, None, n, None, n, None, n, n, n, 1, n, n, 0, 5, 1, 64, 16, 1, 1, 1, n) == 0
    assert lib.fa_paged_append_fp8(n, None, n, None, n, None, n, None, n, n, n, 1, n, n, 2, 0, 1, 64, 16, 1, 1, 1, n) == 0
    assert lib.fa_paged_decode_fp8(n, None, n, None, n, None, n, n, n, 1, n, n, None, n, n, 0, 0, 2, 1, 64, 16, 1, 1, 1, 0.1, 0.0, n,
                                   n) == 0


def test_workspace_sizes(lib):
    assert lib.fa_qk_norm_rope_bwd_workspace_size(96) == 0
    assert lib.fa_qk_norm_rope_bwd_workspace_size(128) == 2 * lib.fa_qk_norm_rope_bwd_workspace_size(64) > 0


def test_binding_refuses_before_the_library(lib):
    x = torch.zeros(1, 2, 8, 64)
    with pytest.raises(TypeError):
        fa.fa_qk_norm_rope(x, x)
    with pytest.raises(ValueError):
        fa.fa_qk_norm_rope(x.bfloat16(), x.bfloat16())  # not on a GPU
    i = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.fa_paged_resize(i, i[0], i[0], i[0], i[0], 16)
    with pytest.raises(TypeError):
        fa.fa_paged_decode_fp8(torch.zeros(1, 2, 64), x, x, x, x, i, i[0])
    with pytest.raises(TypeError):
        fa.fa_paged_append_fp8(x[0].bfloat16(), x[0].bfloat16(), x, x, x, x, i, i[0], i[0])
