"""The workloads by which the scored attention and the paged key-value cache are measured.

Four calls: the scored forward (tanh cap, distance bias, document and prefix masks, shared
key/value heads), a training step of it (forward and gradients), one new token a sequence
over a paged cache, and the writing of new tokens into that cache.
"""

import math
import random

import torch

own = False

BF16, FP16 = "bfloat16", "float16"


# --------------------------------------------------------------------------- cases


def listed():
    return [
        # The smallest call: a short prompt's layer, where latency counts.
        {"name": "fwd small", "op": "fwd", "B": 1, "H": 4, "Hkv": 2, "N": 129, "d": 64, "causal": True, "cap": 30.0,
         "bias": False, "docs": 0, "prefix": False, "pad": 0.0, "layout": "bhnd"},
        # A packed prompt batch with capped scores and shared heads, heads beside tokens as a projection leaves them.
        {"name": "fwd docs cap", "op": "fwd", "B": 2, "H": 16, "Hkv": 4, "N": 8192, "d": 128, "causal": True, "cap": 50.0,
         "bias": False, "docs": 9, "prefix": False, "pad": 0.03, "layout": "bnhd"},
        # A long document whose only positions are the distance bias.
        {"name": "fwd bias long", "op": "fwd", "B": 1, "H": 16, "Hkv": 16, "N": 16384, "d": 128, "causal": True, "cap": 0.0,
         "bias": True, "docs": 0, "prefix": False, "pad": 0.0, "layout": "bhnd"},
        # A training step on a few short rows, both directions visible.
        {"name": "step small", "op": "step", "B": 2, "H": 2, "Hkv": 2, "N": 200, "d": 64, "causal": False, "cap": 20.0,
         "bias": True, "docs": 3, "prefix": False, "pad": 0.1, "layout": "bhnd"},
        # Pretraining on packed documents, capped scores.
        {"name": "step docs cap", "op": "step", "B": 4, "H": 16, "Hkv": 16, "N": 4096, "d": 128, "causal": True, "cap": 30.0,
         "bias": False, "docs": 5, "prefix": False, "pad": 0.02, "layout": "bnhd"},
        # Small heads with a distance bias and shared keys, an odd length.
        {"name": "step bias d64", "op": "step", "B": 2, "H": 32, "Hkv": 8, "N": 2047, "d": 64, "causal": True, "cap": 0.0,
         "bias": True, "docs": 0, "prefix": False, "pad": 0.0, "layout": "bhnd"},
        # Long rows of a few documents, each with a prompt that sees itself both ways.
        {"name": "step prefix", "op": "step", "B": 2, "H": 16, "Hkv": 4, "N": 8192, "d": 128, "causal": True, "cap": 0.0,
         "bias": False, "docs": 2, "prefix": True, "pad": 0.0, "layout": "bhnd"},
        # One user, a short dialogue: a decode step's latency.
        {"name": "decode one", "op": "decode", "B": 1, "H": 16, "Hkv": 4, "d": 128, "page": 16, "least": 900, "most": 900,
         "cap": 0.0, "bias": False, "dtype": BF16},
        # A serving batch of ragged lengths, capped scores.
        {"name": "decode ragged", "op": "decode", "B": 64, "H": 32, "Hkv": 8, "d": 128, "page": 64, "least": 1,
         "most": 16384, "cap": 50.0, "bias": False, "dtype": BF16},
        # One very long context, fp16, distance bias.
        {"name": "decode long", "op": "decode", "B": 1, "H": 16, "Hkv": 16, "d": 64, "page": 128, "least": 131072,
         "most": 131072, "cap": 0.0, "bias": True, "dtype": FP16},
        # The new token of every sequence of a serving batch.
        {"name": "append token", "op": "append", "B": 64, "Hkv": 8, "d": 128, "page": 16, "least": 1, "most": 1,
         "before": 700, "dtype": BF16},
        # Ragged prompts going into the cache.
        {"name": "append prompts", "op": "append", "B": 16, "Hkv": 8, "d": 128, "page": 64, "least": 1, "most": 4096,
         "before": 0, "dtype": BF16},
    ]


def _between(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fwd", "step", "decode", "append"])
    d = rng.choice([64, 128])
    if op in ("fwd", "step"):
        while True:
            Hkv, G = _between(rng, 1, 16), rng.choice([1, 1, 2, 3, 4, 8])
            # (a training row of one token has no gradient but rounding)
            case = {"op": op, "B": _between(rng, 1, 8), "H": Hkv * G, "Hkv": Hkv, "d": d,
                    "N": _between(rng, 1 if op == "fwd" else 16, 16384),
                    "causal": rng.random() < 0.75, "cap": rng.choice([0.0, 20.0, 30.0, 50.0]), "bias": rng.random() < 0.4,
                    "docs": rng.choice([0, 0, 1, 3, 8, 20]), "prefix": rng.random() < 0.3,
                    "pad": rng.choice([0.0, 0.0, 0.05, 0.4]), "layout": rng.choice(["bhnd", "bnhd"])}
            case["docs"] = min(case["docs"], max(1, case["N"] // 16)) if case["docs"] else 0
            case["prefix"] = case["prefix"] and case["causal"] and case["docs"] > 0
            case["pad"] = case["pad"] if case["docs"] else 0.0
            if case["B"] * case["H"] * case["N"] ** 2 * (3.5 if op == "step" else 1.0) <= 16 * 16384 ** 2:
                return case
    dtype, page = rng.choice([BF16, BF16, FP16]), rng.choice([16, 32, 64, 128, 256])
    Hkv = rng.choice([1, 2, 3, 4, 8, 16])
    if op == "decode":
        while True:
            G, most = rng.choice([1, 2, 4, 5, 8, 16, 24]), _between(rng, 1, 65536)
            case = {"op": op, "B": _between(rng, 1, 128), "H": Hkv * G, "Hkv": Hkv, "d": d, "page": page,
                    "least": rng.choice([0, 1, max(1, most // 2), most]), "most": most, "cap": rng.choice([0.0, 30.0, 50.0]),
                    "bias": rng.random() < 0.4, "dtype": dtype}
            if case["B"] * most * Hkv * d <= 64 * 8192 * 8 * 128 and case["B"] * most * case["H"] <= 64 * 8192 * 32:
                return case
    while True:
        most = _between(rng, 1, 4096)
        case = {"op": op, "B": _between(rng, 1, 64), "Hkv": Hkv, "d": d, "page": page, "least": rng.choice([0, 1, most]),
                "most": most, "before": rng.choice([0, 5, 700]), "dtype": dtype}
        if case["B"] * most * Hkv * d <= 16 * 4096 * 8 * 128:
            return case


def _documents(case):
    """Offsets [B][docs + 1] and prefix lengths [B][docs] of a case's documents, from the case alone."""
    rng = random.Random(7 * case["N"] + 31 * case["docs"] + case["B"])
    cu, pre = [], []
    for _ in range(case["B"]):
        end = case["N"] - int(case["pad"] * case["N"] * rng.random())
        cuts = [0] + sorted(rng.randint(0, end) for _ in range(case["docs"] - 1)) + [end]
        cu.append(cuts)
        pre.append([rng.randint(0, max(1, (b - a) // 2)) if case["prefix"] else 0 for a, b in zip(cuts, cuts[1:])])
    return cu, pre


def _pairs(case):
    """(query, key) pairs that see each other, over the batch, for one head."""
    if not case["docs"]:
        n = case["N"]
        return case["B"] * (n * (n + 1) // 2 if case["causal"] else n * n)
    cu, pre = _documents(case)
    total = 0
    for cuts, ps in zip(cu, pre):
        for a, b, p in zip(cuts, cuts[1:], ps):
            n, p = b - a, min(p, b - a)
            total += n * (n + 1) // 2 + p * (p - 1) // 2 if case["causal"] else n * n
    return total


def _lengths(case):
    """Tokens of each sequence, from the case alone; the most and the least are among them."""
    rng = random.Random(3 * case["most"] + 5 * case["B"] + case["page"])
    n = [rng.randint(case["least"], case["most"]) for _ in range(case["B"])]
    n[0] = case["most"]
    if case["B"] > 1:
        n[-1] = case["least"]
    return n


def work(case):
    if case["op"] in ("fwd", "step"):
        B, H, Hkv, N, d = (case[x] for x in ("B", "H", "Hkv", "N", "d"))
        q, kv, lse = 2 * B * H * N * d, 2 * B * Hkv * N * d, 4 * B * H * N
        if case["op"] == "fwd":
            return {"bytes": 2 * q + 2 * kv + lse, "flops": 4 * d * H * _pairs(case)}
        # q, k, v, do in; o, lse, dq, dk, dv out; two products forward, five backward.
        return {"bytes": 4 * q + 4 * kv + lse, "flops": 14 * d * H * _pairs(case)}
    tokens = sum(_lengths(case))
    if case["op"] == "decode":
        return {"bytes": 4 * case["Hkv"] * case["d"] * tokens + 4 * case["B"] * case["H"] * (case["d"] + 1),
                "flops": 4 * case["H"] * case["d"] * tokens}
    return {"bytes": 8 * case["Hkv"] * case["d"] * tokens, "flops": 0}


# ------------------------------------------------------------------------- inputs


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _slopes(H):
    """The geometric slopes 2^(-8 (h + 1) / H) of a distance bias."""
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=torch.float32, device="cuda")


def _normal(shape, g, dtype, factor=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * factor).to(dtype)


def prepare(case, seed):
    g = _generator(seed)
    st = {"case": dict(case)}
    d, Hkv = case["d"], case["Hkv"]
    if case["op"] in ("fwd", "step"):
        B, H, N = case["B"], case["H"], case["N"]

        def heads(n, factor=1.0):  # [B, n, N, d], dense or as a projection's [B, N, n, d] seen by heads
            if case["layout"] == "bnhd":
                return _normal((B, N, n, d), g, torch.bfloat16, factor).transpose(1, 2)
            return _normal((B, n, N, d), g, torch.bfloat16, factor)

        # Capped models have larger scores (here a standard deviation of 3) than plain ones (1).
        st["q"] = heads(H, 3.0 if case["cap"] else 1.0)
        st["k"], st["v"] = heads(Hkv), heads(Hkv)
        if case["op"] == "step":
            st["do"] = heads(H)
        st["slopes"] = _slopes(H) if case["bias"] else None
        st["cu"] = st["prefix"] = st["plan"] = None
        if case["docs"]:
            cu, pre = _documents(case)
            st["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
            st["prefix"] = torch.tensor(pre, dtype=torch.int32, device="cuda") if case["prefix"] else None
        if own:
            import io_aware_exact_fwd_gb300 as fa

            # Made once for a batch and used by every layer of it.
            if case["docs"]:
                st["plan"] = fa.fa_mask_plan(B, N, st["cu"], st["prefix"], causal=case["causal"])
            if case["op"] == "step":
                st["workspace"] = torch.empty(fa.fa_bwd_scored_workspace_size(B, H, Hkv, N, d), dtype=torch.uint8,
                                              device="cuda")
        return st
    dtype = torch.bfloat16 if case["dtype"] == BF16 else torch.float16
    B, page = case["B"], case["page"]
    new = _lengths(case)
    before = case["before"] if case["op"] == "append" else 0
    lens = [n + before for n in new]
    per_seq = max(1, max((n + page - 1) // page for n in lens))
    used = sum((n + page - 1) // page for n in lens)
    pages = used + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[:used].tolist()
    table, at = [], 0
    for n in lens:
        m = (n + page - 1) // page
        table.append(order[at:at + m] + [0] * (per_seq - m))
        at += m
    st["table"] = torch.tensor(table, dtype=torch.int32, device="cuda")
    st["lens"], st["lens_host"] = torch.tensor(lens, dtype=torch.int32, device="cuda"), lens
    # Tokens beside heads inside a page, seen as [pages, heads, page, d].
    st["k_cache"] = _normal((pages, page, Hkv, d), g, dtype).transpose(1, 2)
    st["v_cache"] = _normal((pages, page, Hkv, d), g, dtype).transpose(1, 2)
    if case["op"] == "decode":
        st["q"] = _normal((B, case["H"], d), g, dtype, 3.0 if case["cap"] else 1.0)
        st["slopes"] = _slopes(case["H"]) if case["bias"] else None
        if own:
            import io_aware_exact_fwd_gb300 as fa

            st["workspace"] = torch.empty(fa.fa_paged_decode_workspace_size(B, case["H"], Hkv, d), dtype=torch.uint8,
                                          device="cuda")
    else:
        st["k"], st["v"] = _normal((sum(new), Hkv, d), g, dtype), _normal((sum(new), Hkv, d), g, dtype)
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        st["cu"], st["cu_host"] = torch.tensor(cu, dtype=torch.int32, device="cuda"), cu
    return st


# ---------------------------------------------------------------------- one pass


def run(st):
    case = st["case"]
    if own:
        return _run_own(st, case)
    return {"fwd": _plain_forward, "step": _plain_step, "decode": _plain_decode, "append": _plain_append}[case["op"]](st, case)


def _run_own(st, case):
    import io_aware_exact_fwd_gb300 as fa

    if case["op"] in ("fwd", "step"):
        kw = {"causal": case["causal"] and st["plan"] is None, "softcap": case["cap"], "slopes": st["slopes"],
              "plan": st["plan"]}
        o, lse = fa.fa_fwd_scored(st["q"], st["k"], st["v"], **kw)
        if case["op"] == "fwd":
            return {"o": o, "lse": lse}
        dq, dk, dv = fa.fa_bwd_scored(st["q"], st["k"], st["v"], o, st["do"], lse, workspace=st["workspace"], **kw)
        return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    if case["op"] == "decode":
        o, lse = fa.fa_paged_decode(st["q"], st["k_cache"], st["v_cache"], st["table"], st["lens"],
                                    workspace=st["workspace"], softcap=case["cap"], slopes=st["slopes"])
        return {"o": o, "lse": lse}
    fa.fa_paged_append(st["k"], st["v"], st["k_cache"], st["v_cache"], st["table"], st["lens"], st["cu"])
    return {"k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _visible(case, st, b):
    """Truth values [N, N]: query i sees key j in row b of the batch."""
    N = case["N"]
    i, j = torch.arange(N, device="cuda")[:, None], torch.arange(N, device="cuda")[None, :]
    if not case["docs"]:
        return j <= i if case["causal"] else torch.ones(N, N, dtype=torch.bool, device="cuda")
    ends = st["cu"][b, 1:].contiguous()
    doc = torch.searchsorted(ends, torch.arange(N, device="cuda", dtype=torch.int32), right=True)
    inside = doc < ends.numel()
    see = (doc[:, None] == doc[None, :]) & inside[:, None]
    if case["causal"]:
        ahead = j <= i
        if st["prefix"] is not None:
            safe = doc.clamp(max=ends.numel() - 1)
            reach = (st["cu"][b].gather(0, safe) + st["prefix"][b].gather(0, safe))[None, :]
            ahead = ahead | (j < reach)
        see = see & ahead
    return see


def _plain_weights(case, st, b, h, see):
    """Softmax weights, LSE and the cap's slope 1 - tanh^2 (or None) of one head, in 32 bits."""
    G = case["H"] // case["Hkv"]
    q, k = st["q"][b, h].float(), st["k"][b, h // G].float()
    s = (q @ k.T) * case["d"] ** -0.5
    bend = None
    if case["cap"]:
        t = torch.tanh(s / case["cap"])
        s, bend = case["cap"] * t, 1.0 - t * t
    if case["bias"]:
        pos = torch.arange(case["N"], device="cuda", dtype=torch.float32)
        s = s - st["slopes"][h] * (pos[:, None] - pos[None, :]).abs()
    s = s.masked_fill(~see, float("-inf"))
    top = s.amax(dim=1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(s - top)
    total = p.sum(dim=1, keepdim=True)
    lse = (top + torch.log(total))[:, 0]
    return p / total.clamp(min=1e-30), lse, bend


def _empty_like(t):
    return torch.empty(t.shape, dtype=t.dtype, device="cuda")


def _plain_forward(st, case):
    B, H, N = case["B"], case["H"], case["N"]
    o, lse = _empty_like(st["q"]), torch.empty((B, H, N), dtype=torch.float32, device="cuda")
    for b in range(B):
        see = _visible(case, st, b)
        for h in range(H):
            p, lse[b, h], _ = _plain_weights(case, st, b, h, see)
            o[b, h] = (p @ st["v"][b, h * case["Hkv"] // H].float()).to(o.dtype)
    return {"o": o, "lse": lse}


def _plain_step(st, case):
    B, H, Hkv, N, d = (case[x] for x in ("B", "H", "Hkv", "N", "d"))
    G, scale = H // Hkv, d ** -0.5
    o, lse, dq = _empty_like(st["q"]), torch.empty((B, H, N), dtype=torch.float32, device="cuda"), _empty_like(st["q"])
    dk, dv = _empty_like(st["k"]), _empty_like(st["v"])
    for b in range(B):
        see = _visible(case, st, b)
        for hk in range(Hkv):
            k, v = st["k"][b, hk].float(), st["v"][b, hk].float()
            sum_k, sum_v = torch.zeros_like(k), torch.zeros_like(v)
            for h in range(hk * G, hk * G + G):
                p, lse[b, h], bend = _plain_weights(case, st, b, h, see)
                out, go = p @ v, st["do"][b, h].float()
                o[b, h] = out.to(o.dtype)
                ds = p * (go @ v.T - (go * out).sum(dim=1, keepdim=True))
                if bend is not None:
                    ds = ds * bend
                dq[b, h] = (scale * (ds @ k)).to(dq.dtype)
                sum_k += scale * (ds.T @ st["q"][b, h].float())
                sum_v += p.T @ go
            dk[b, hk], dv[b, hk] = sum_k.to(dk.dtype), sum_v.to(dv.dtype)
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def _plain_decode(st, case):
    B, H, Hkv, d, page = (case[x] for x in ("B", "H", "Hkv", "d", "page"))
    o = torch.zeros((B, H, d), dtype=st["q"].dtype, device="cuda")
    lse = torch.full((B, H), float("-inf"), dtype=torch.float32, device="cuda")
    for b, n in enumerate(st["lens_host"]):
        if n == 0:
            continue
        ids = st["table"][b, :(n + page - 1) // page].long()
        k = st["k_cache"][ids].transpose(0, 1).reshape(Hkv, -1, d)[:, :n].float()
        v = st["v_cache"][ids].transpose(0, 1).reshape(Hkv, -1, d)[:, :n].float()
        s = (st["q"][b].float().view(Hkv, H // Hkv, d) @ k.transpose(1, 2)) * d ** -0.5
        if case["cap"]:
            s = case["cap"] * torch.tanh(s / case["cap"])
        if case["bias"]:
            back = torch.arange(n - 1, -1, -1, device="cuda", dtype=torch.float32)
            s = s - st["slopes"].view(Hkv, H // Hkv, 1) * back
        top = s.amax(dim=2, keepdim=True)
        p = torch.exp(s - top)
        total = p.sum(dim=2, keepdim=True)
        o[b] = ((p @ v) / total).reshape(H, d).to(o.dtype)
        lse[b] = (top + torch.log(total)).reshape(H)
    return {"o": o, "lse": lse}


def _plain_append(st, case):
    page, cu, lens = case["page"], st["cu"].long(), st["lens"].long()
    T = st["k"].shape[0]
    row = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    at = lens[b] - (cu[b + 1] - cu[b]) + (row - cu[b])
    where = st["table"].long()[b, at // page]
    st["k_cache"].transpose(1, 2)[where, at % page] = st["k"]
    st["v_cache"].transpose(1, 2)[where, at % page] = st["v"]
    return {"k_cache": st["k_cache"], "v_cache": st["v_cache"]}


# ------------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("fwd", "step"):
        return _exact_attention(st, case)
    if case["op"] == "decode":
        return _exact_decode(st, case)
    out = {}
    for name, new in (("k_cache", st["k"]), ("v_cache", st["v"])):
        cache = st[name].double()
        for b in range(case["B"]):
            first, last = st["cu_host"][b], st["cu_host"][b + 1]
            t, place = first, st["lens_host"][b] - (last - first)
            while t < last:  # one page at a time
                off = place % case["page"]
                n = min(case["page"] - off, last - t)
                cache[int(st["table"][b, place // case["page"]]), :, off:off + n] = new[t:t + n].double().transpose(0, 1)
                t, place = t + n, place + n
        out[name] = cache
    return out


def _exact_attention(st, case):
    """Document by document, one dense softmax each; gradients by differentiating it."""
    B, H, Hkv, N, d = (case[x] for x in ("B", "H", "Hkv", "N", "d"))
    step = case["op"] == "step"
    o = torch.zeros((B, H, N, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, N), float("-inf"), dtype=torch.float64, device="cuda")
    dq = torch.zeros_like(o)
    dk = torch.zeros((B, Hkv, N, d), dtype=torch.float64, device="cuda")
    dv = torch.zeros_like(dk)
    cu, pre = _documents(case) if case["docs"] else ([[0, N]] * B, [[0]] * B)
    for b in range(B):
        for first, last, p in zip(cu[b], cu[b][1:], pre[b]):
            n = last - first
            if n == 0:
                continue
            place = torch.arange(n, device="cuda", dtype=torch.float64)
            gap = place[:, None] - place[None, :]
            hide = torch.zeros((n, n), dtype=torch.bool, device="cuda")
            if case["causal"]:
                hide = (gap < 0) & (place[None, :] >= p)
            for h in range(H):
                hk = h // (H // Hkv)
                q, k, v = (t.detach().double().requires_grad_(step) for t in (
                    st["q"][b, h, first:last], st["k"][b, hk, first:last], st["v"][b, hk, first:last]))
                s = torch.einsum("id,jd->ij", q, k) / math.sqrt(d)
                if case["cap"]:
                    s = case["cap"] * torch.tanh(s / case["cap"])
                if case["bias"]:
                    s = s - 2.0 ** (-8.0 * (h + 1) / H) * gap.abs()
                s = s.masked_fill(hide, float("-inf"))
                out = torch.softmax(s, dim=1) @ v
                o[b, h, first:last] = out.detach()
                lse[b, h, first:last] = torch.logsumexp(s.detach(), dim=1)
                if step:
                    gq, gk, gv = torch.autograd.grad(out, (q, k, v), st["do"][b, h, first:last].double())
                    dq[b, h, first:last] = gq
                    dk[b, hk, first:last] += gk
                    dv[b, hk, first:last] += gv
                del s, out
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv} if step else {"o": o, "lse": lse}


def _exact_decode(st, case):
    B, H, Hkv, d, page = (case[x] for x in ("B", "H", "Hkv", "d", "page"))
    o = torch.zeros((B, H, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, H), float("-inf"), dtype=torch.float64, device="cuda")
    for b, n in enumerate(st["lens_host"]):
        if n == 0:
            continue
        at = torch.arange(n, device="cuda")
        ids = st["table"][b].long()[at // page]
        for hk in range(Hkv):
            k, v = st["k_cache"][ids, hk, at % page].double(), st["v_cache"][ids, hk, at % page].double()
            for h in range(hk * (H // Hkv), (hk + 1) * (H // Hkv)):
                s = (k * st["q"][b, h].double()).sum(dim=1) / math.sqrt(d)
                if case["cap"]:
                    s = case["cap"] * torch.tanh(s / case["cap"])
                if case["bias"]:
                    s = s - 2.0 ** (-8.0 * (h + 1) / H) * (n - 1 - at).double()
                lse[b, h] = torch.logsumexp(s, dim=0)
                o[b, h] = torch.softmax(s, dim=0) @ v
    return {"o": o, "lse": lse}
