"""Calls on a stream given by the caller, beside a current stream that is still writing memory freed on it.

What a call allocates (outputs, workspaces, plans) has to come from the memory of the stream that
the call runs on: a block that the current stream freed is not idle before that stream gets there.
"""

import pytest
import torch

import io_aware_exact_fwd_gb300 as fa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fa.load_library()
    fa.fa_debug_set_fault(0)
    fa.fa_debug_set_wait_limit_ns(0)


def _randn(*shape, seed, dtype=torch.bfloat16):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def _check(call, *workspaces):
    """call(stream=...) gives the same tensors on a side stream, while the current stream waits to fill freed blocks
    of every output's size (and of each of `workspaces`, in bytes)."""
    want = call(stream=None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(50_000_000)  # some 25 ms of the current stream
    sizes = [t.nbytes for t in want] + list(workspaces)
    freed = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    del freed
    got = call(stream=side)
    torch.cuda.synchronize()
    fa.fa_sync_check()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_scored_attention():
    B, H, Hkv, N, d = 2, 4, 2, 700, 64
    q, k, v, do = (_randn(B, h, N, d, seed=i) for i, h in enumerate((H, Hkv, Hkv, H)))
    cu = torch.tensor([[0, 300, 690], [5, 200, 700]], dtype=torch.int32, device="cuda")
    kw = dict(softcap=20.0, plan=fa.fa_mask_plan(B, N, cu))
    o, lse = fa.fa_fwd_scored(q, k, v, **kw)
    _check(lambda stream: [fa.fa_mask_plan(B, N, cu, stream=stream)])
    _check(lambda stream: fa.fa_fwd_scored(q, k, v, stream=stream, **kw))
    _check(lambda stream: fa.fa_bwd_scored(q, k, v, o, do, lse, deterministic=True, stream=stream, **kw),
           fa.fa_bwd_scored_workspace_size(B, H, Hkv, N, d))


def test_paged_decode():
    B, H, Hkv, d, page = 3, 8, 2, 128, 16
    kc, vc = (_randn(80, Hkv, page, d, seed=i) for i in range(2))
    table = torch.randperm(75, generator=torch.Generator().manual_seed(2)).to(torch.int32).view(B, 25).cuda()
    n = torch.tensor([400, 1, 77], dtype=torch.int32, device="cuda")
    q = _randn(B, H, d, seed=3)
    _check(lambda stream: fa.fa_paged_decode(q, kc, vc, table, n, stream=stream), fa.fa_paged_decode_workspace_size(B, H, Hkv, d))


def _qkvdo(B, H, N, d, dtype=torch.bfloat16):
    return [_randn(B, H, N, d, seed=10 + i, dtype=dtype) for i in range(4)]


def test_forward_and_backward():
    B, H, N, d = 1, 4, 600, 64
    q, k, v, do = _qkvdo(B, H, N, d)
    o, lse = fa.fa_fwd(q, k, v, causal=True)
    _check(lambda stream: fa.fa_fwd(q, k, v, causal=True, stream=stream))
    _check(lambda stream: fa.fa_bwd(q, k, v, o, do, lse, causal=True, deterministic=True, stream=stream),
           fa.fa_bwd_workspace_size(B, H, N, d))


def test_fp8():
    B, H, N, d = 1, 3, 500, 64
    q, k, v, do = _qkvdo(B, H, N, d)
    shape = (B, H, N, d)
    signs = fa.fa_fp8_rotation_signs(7, d).cuda()

    def forward(stream):
        ws = fa.fa_fp8_prepare(q, k, v, signs, stream=stream)
        return fa.fa_fwd_fp8(ws, shape, causal=True, stream=stream)
    o, lse = forward(None)
    ws = fa.fa_fp8_prepare_seeded(q, k, v, 7)
    _check(forward, fa.fa_fp8_workspace_size(*shape))
    _check(lambda stream: fa.fa_fwd_fp8(fa.fa_fp8_prepare_seeded(q, k, v, 7, stream=stream), shape, causal=True, stream=stream),
           fa.fa_fp8_workspace_size(*shape))
    _check(lambda stream: fa.fa_fp8_dequantize(ws, shape, stream=stream))
    _check(lambda stream: fa.fa_bwd_fp8(ws, signs, o, do, lse, causal=True, deterministic=True, stream=stream),
           fa.fa_bwd_fp8_workspace_size(*shape))


def test_split_kv():
    B, H, Nq, Nk, d = 2, 4, 3, 1500, 128
    q, k, v = (_randn(B, H, n, d, seed=20 + i) for i, n in enumerate((Nq, Nk, Nk)))
    parts = fa.fa_fwd_splitkv_partial(q, k, v, 4)
    _check(lambda stream: fa.fa_fwd_splitkv_partial(q, k, v, 4, stream=stream))
    _check(lambda stream: fa.fa_merge_partials(*parts, stream=stream))
    _check(lambda stream: fa.fa_fwd_splitkv(q, k, v, n_split=4, stream=stream), fa.fa_splitkv_workspace_size(B, H, Nq, d, 4))


def test_w4a16():
    M, N, K = 3, 512, 1024
    g = torch.Generator().manual_seed(30)
    x = torch.randn(M, K, generator=g).half().cuda()
    wq = torch.randint(-2 ** 31, 2 ** 31, (N, K // 8), generator=g).to(torch.int32).cuda()
    scales = (torch.rand(K // 128, N, generator=g) * 0.01 + 0.005).half().cuda()
    zeros = torch.randint(0, 16, (K // 128, N), generator=g).to(torch.uint8).cuda()
    _check(lambda stream: [fa.fa_w4a16_gemm(x, wq, scales, zeros, n_split=2, stream=stream)], fa.fa_w4a16_workspace_size(M, N, K, 2))


def test_paged_cache_in_8_bits():
    B, H, Hkv, d, page = 3, 8, 2, 128, 16
    kc, vc = (_randn(80, Hkv, page, d, seed=i).to(torch.float8_e4m3fn) for i in range(2))
    ks, vs = (torch.full((80, Hkv, 1), 0.01, device="cuda") for _ in range(2))
    table = torch.randperm(75, generator=torch.Generator().manual_seed(2)).to(torch.int32).view(B, 25).cuda()
    n = torch.tensor([400, 1, 77], dtype=torch.int32, device="cuda")
    q = _randn(B, H, d, seed=3)
    _check(lambda stream: fa.fa_paged_decode_fp8(q, kc, vc, ks, vs, table, n, stream=stream), fa.fa_paged_decode_workspace_size(B, H, Hkv, d))


@pytest.mark.parametrize("B", [5, 600])
def test_paged_bookkeeping(B):
    # Each sequence a token longer inside its page: the table and the list stay, so that both calls do the same.
    table = torch.arange(2 * B, dtype=torch.int32, device="cuda").view(B, 2)
    n, delta = (torch.full((B,), x, dtype=torch.int32, device="cuda") for x in (17, 1))
    free, count = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    _check(lambda stream: fa.fa_paged_resize(table, n, delta, free, count, 16, stream=stream),
           4 * (2 * B + 4) + fa.fa_paged_resize_workspace_size(B))


def test_norm_and_rotation():
    B, H, Hkv, N, d = 2, 6, 2, 300, 64
    q, k, gq, gk = (_randn(B, h, N, d, seed=i) for i, h in enumerate((H, Hkv, H, Hkv)))
    w, f = torch.ones(d, device="cuda"), torch.tensor([1e4 ** (-i / d) for i in range(0, d, 2)], dtype=torch.float32, device="cuda")
    kw = dict(q_weight=w, k_weight=w, inv_freq=f)
    _check(lambda stream: fa.fa_qk_norm_rope(q, k, stream=stream, **kw))
    _check(lambda stream: fa.fa_qk_norm_rope_bwd(q, k, gq, gk, stream=stream, **kw), 2 * 4 * d, fa.fa_qk_norm_rope_bwd_workspace_size(d))
