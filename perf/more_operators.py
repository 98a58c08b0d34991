"""The workloads by which the serving of a token from an 8-bit cache and the preparation of queries and keys are measured.

Five calls: the norm of every query and key head with the position rotation, and its
gradient; the bookkeeping of a paged cache on the GPU (page tables, slots and positions
from the sequences' new lengths); new tokens written into a cache of 8-bit codes with a
power-of-two scale for each block of 16 tokens and head; and one new token a sequence
against such a cache.
"""

import math
import random

import torch

own = False

BF16, FP16 = "bfloat16", "float16"
BLOCK = 16  # tokens that share a scale, of one head


# --------------------------------------------------------------------------- cases


def listed():
    return [
        # One decode step of a few sequences: each brings one token; latency counts.
        {"name": "prep step", "op": "prep", "B": 1, "N": 16, "H": 8, "Hkv": 2, "d": 64, "rot": 64, "pairs": False, "norm": True,
         "weight": "float32", "far": 40000, "dtype": FP16, "layout": "qkv"},
        # A packed batch of prompts, heads beside tokens as a fused projection leaves them.
        {"name": "prep prompts", "op": "prep", "B": 2, "N": 8192, "H": 32, "Hkv": 8, "d": 128, "rot": 128, "pairs": False,
         "norm": True, "weight": BF16, "far": 0, "dtype": BF16, "layout": "qkv"},
        # A short training row, half of each head rotated, in neighbouring pairs.
        {"name": "grad small", "op": "grad", "B": 2, "N": 129, "H": 4, "Hkv": 2, "d": 64, "rot": 32, "pairs": True, "norm": True,
         "weight": "float32", "far": 0, "dtype": BF16, "layout": "bhnd"},
        # A layer of a training step.
        {"name": "grad train", "op": "grad", "B": 4, "N": 4096, "H": 16, "Hkv": 16, "d": 128, "rot": 128, "pairs": False,
         "norm": True, "weight": "float32", "far": 0, "dtype": BF16, "layout": "bnhd"},
        # A decode step's new tokens, one a sequence, into half-filled blocks.
        {"name": "append step", "op": "append", "B": 64, "Hkv": 8, "d": 128, "page": 64, "least": 1, "most": 1, "before": 700,
         "dtype": BF16, "layout": "hnd"},
        # Prompts written into the cache.
        {"name": "append prompts", "op": "append", "B": 16, "Hkv": 8, "d": 128, "page": 64, "least": 1, "most": 4096, "before": 5,
         "dtype": BF16, "layout": "hnd"},
        # One sequence in its early tokens.
        {"name": "decode one", "op": "decode", "B": 1, "H": 16, "Hkv": 4, "d": 128, "page": 16, "least": 900, "most": 900,
         "cap": 0.0, "bias": False, "dtype": BF16, "layout": "hnd"},
        # A server's batch: lengths of every size, shared heads, capped scores.
        {"name": "decode batch", "op": "decode", "B": 64, "H": 32, "Hkv": 8, "d": 128, "page": 64, "least": 1, "most": 16384,
         "cap": 50.0, "bias": False, "dtype": BF16, "layout": "hnd"},
        # One very long document, distances as its positions, tokens beside heads in a page.
        {"name": "decode long", "op": "decode", "B": 1, "H": 16, "Hkv": 16, "d": 64, "page": 128, "least": 131072, "most": 131072,
         "cap": 0.0, "bias": True, "dtype": FP16, "layout": "nhd"},
        # Many query heads over one key/value head.
        {"name": "decode shared", "op": "decode", "B": 24, "H": 40, "Hkv": 1, "d": 128, "page": 32, "least": 2000, "most": 8000,
         "cap": 0.0, "bias": False, "dtype": BF16, "layout": "hnd"},
        # A decode step's bookkeeping: every sequence one token longer.
        {"name": "resize step", "op": "resize", "B": 64, "page": 16, "most": 4000, "grow": 1, "shrink": 0.0, "behind": 0},
        # Prompts come in, other sequences end or take tokens back, in one call.
        {"name": "resize mixed", "op": "resize", "B": 1000, "page": 16, "most": 3000, "grow": 2500, "shrink": 0.4, "behind": 1000},
    ]


def _between(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prep", "grad", "append", "decode", "decode", "resize"])
    d, dtype = rng.choice([64, 128]), rng.choice([BF16, BF16, FP16])
    if op in ("prep", "grad"):
        while True:
            Hkv, G = _between(rng, 1, 16), rng.choice([1, 1, 2, 3, 4, 8])
            norm = rng.random() < 0.8
            case = {"op": op, "B": _between(rng, 1, 8), "N": _between(rng, 1, 16384), "H": Hkv * G, "Hkv": Hkv, "d": d,
                    "rot": rng.choice([d, d, d // 2, 16, 0]) if norm else d, "pairs": rng.random() < 0.3, "norm": norm,
                    "weight": rng.choice(["none", "float32", dtype]) if norm else "none", "far": rng.choice([0, 0, 1000, 1000000]),
                    "dtype": dtype, "layout": rng.choice(["bhnd", "bnhd", "qkv"])}
            if case["B"] * case["N"] * (case["H"] + case["Hkv"]) * d <= 16384 * 32 * 128:
                return case
    if op == "resize":
        while True:
            case = {"op": op, "B": _between(rng, 1, 4000), "page": rng.choice([16, 32, 48, 64, 256]), "most": _between(rng, 1, 8000),
                    "grow": _between(rng, 1, 5000), "shrink": rng.choice([0.0, 0.0, 0.2, 0.7]), "behind": rng.choice([0, 0, 1, 77])}
            if case["B"] * (case["most"] + case["grow"]) <= 1000 * 5500:
                return case
    page, Hkv = rng.choice([16, 32, 48, 64, 128, 256]), rng.choice([1, 2, 3, 4, 8, 16])
    if op == "decode":
        while True:
            G, most = rng.choice([1, 2, 4, 5, 8, 16, 24]), _between(rng, 1, 65536)
            case = {"op": op, "B": _between(rng, 1, 128), "H": Hkv * G, "Hkv": Hkv, "d": d, "page": page,
                    "least": rng.choice([0, 1, max(1, most // 2), most]), "most": most, "cap": rng.choice([0.0, 30.0, 50.0]),
                    "bias": rng.random() < 0.4, "dtype": dtype, "layout": rng.choice(["hnd", "hnd", "nhd"])}
            if case["B"] * most * Hkv * d <= 64 * 8192 * 8 * 128 and case["B"] * most * case["H"] <= 64 * 8192 * 32:
                return case
    while True:
        most = _between(rng, 1, 4096)
        case = {"op": op, "B": _between(rng, 1, 64), "Hkv": Hkv, "d": d, "page": page, "least": rng.choice([0, 1, most]),
                "most": most, "before": rng.choice([0, 5, 700]), "dtype": dtype, "layout": rng.choice(["hnd", "hnd", "nhd"])}
        if case["B"] * most * Hkv * d <= 16 * 2048 * 8 * 128:
            return case


def _lengths(case):
    """Tokens of each sequence, from the case alone; the most and the least are among them."""
    rng = random.Random(3 * case["most"] + 5 * case["B"] + case["page"])
    n = [rng.randint(case["least"], case["most"]) for _ in range(case["B"])]
    n[0] = case["most"]
    if case["B"] > 1:
        n[-1] = case["least"]
    return n


def _resizes(case):
    """(tokens, change) of each sequence, from the case alone; a change may take every token away."""
    rng = random.Random(11 * case["most"] + case["B"] + case["grow"])
    lens, delta = [], []
    for _ in range(case["B"]):
        lens.append(rng.randint(0, case["most"]))
        if rng.random() < case["shrink"]:
            delta.append(-rng.choice([lens[-1], rng.randint(0, lens[-1])]))
        else:
            delta.append(rng.randint(1, case["grow"]))
    return lens, delta


def _pages(n, page):
    return (n + page - 1) // page


def work(case):
    if case["op"] in ("prep", "grad"):
        rows, d = case["B"] * case["N"] * (case["H"] + case["Hkv"]), case["d"]
        # x in, y out; with the gradient x and dy in, dx out.  A rotation and a norm are a few operations an element.
        each = 4 if case["op"] == "prep" else 6
        return {"bytes": each * rows * d + 4 * case["B"] * case["N"] + 4 * d, "flops": (8 if each == 4 else 16) * rows * d}
    if case["op"] == "resize":
        lens, delta = _resizes(case)
        new = sum(x for x in delta if x > 0)
        moved = sum(abs(_pages(n + x, case["page"]) - _pages(n, case["page"])) for n, x in zip(lens, delta))
        return {"bytes": 16 * case["B"] + 12 * (new + case["behind"]) + 8 * moved, "flops": 0}
    tokens, Hkv, d = sum(_lengths(case)), case["Hkv"], case["d"]
    scales = 8 * Hkv * sum(_pages(n, BLOCK) for n in _lengths(case))
    if case["op"] == "decode":
        return {"bytes": 2 * Hkv * d * tokens + scales + 4 * case["B"] * case["H"] * (d + 1), "flops": 4 * case["H"] * d * tokens}
    return {"bytes": 6 * Hkv * d * tokens + scales, "flops": 0}


# ------------------------------------------------------------------------- inputs


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _slopes(H):
    """The geometric slopes 2^(-8 (h + 1) / H) of a distance bias."""
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=torch.float32, device="cuda")


def _type(name):
    return {BF16: torch.bfloat16, FP16: torch.float16, "float32": torch.float32}[name]


def _normal(shape, g, dtype, factor=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * factor).to(dtype)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _coded(x):
    """(codes, scales) of values [pages, Hkv, page, d]: a power of two for each block of 16 tokens."""
    pages, Hkv, page, d = x.shape
    blocks = x.float().view(pages, Hkv, page // BLOCK, BLOCK * d)
    scale = _power(_exponent(blocks.abs().amax(dim=3)))
    codes = (blocks / scale[..., None]).to(torch.float8_e4m3fn)
    return codes.view(pages, Hkv, page, d), scale


def _exponent(top):
    """The smallest e of [-126, 126] with top <= 448 * 2^e."""
    m, x = torch.frexp(top)  # top = m 2^x, 1/2 <= m < 1; 448 = 0.875 * 2^9
    e = x - 9 + (m > 0.875).to(x.dtype)
    return torch.where(top > 0, e, torch.full_like(e, -126)).clamp(-126, 126)


def _power(e):
    """2^e, -126 <= e <= 127, exactly."""
    return ((e.int() + 127) << 23).view(torch.float32)


def prepare(case, seed):
    g = _generator(seed)
    st = {"case": dict(case)}
    if case["op"] in ("prep", "grad"):
        B, N, H, Hkv, d, dtype = case["B"], case["N"], case["H"], case["Hkv"], case["d"], _type(case["dtype"])

        def pair():  # [B, H, N, d] and [B, Hkv, N, d]: dense, as projections' [B, N, heads, d], or parts of the fused one's
            if case["layout"] == "qkv":
                x = _normal((B, N, H + 2 * Hkv, d), g, dtype, 2.0).transpose(1, 2)
                return x[:, :H], x[:, H:H + Hkv]
            if case["layout"] == "bnhd":
                return tuple(_normal((B, N, n, d), g, dtype, 2.0).transpose(1, 2) for n in (H, Hkv))
            return tuple(_normal((B, n, N, d), g, dtype, 2.0) for n in (H, Hkv))

        st["q"], st["k"] = pair()
        if case["op"] == "grad":
            st["dq"], st["dk"] = pair()
        st["qw"] = st["kw"] = st["freq"] = st["pos"] = None
        if case["weight"] != "none":
            st["qw"], st["kw"] = ((1.0 + 0.2 * _normal((d,), g, torch.float32)).to(_type(case["weight"])) for _ in range(2))
        if case["rot"]:
            steps = torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda")
            st["freq"] = torch.pow(500000.0, -steps / case["rot"]).float()
        if case["far"]:  # decode steps and packed rows bring positions of their own; else 0 .. N - 1
            st["pos"] = torch.randint(0, case["far"] + 1, (B, N), generator=g, device="cuda", dtype=torch.int32)
        return st
    if case["op"] == "resize":
        page, (lens, delta) = case["page"], _resizes(case)
        had, after = [_pages(n, page) for n in lens], [_pages(n + x, page) for n, x in zip(lens, delta)]
        used, width = sum(had), max(1, max(had + after))
        spare = sum(max(0, b - a) for a, b in zip(had, after)) + 7
        order = torch.randperm(used + spare, generator=g, device="cuda").to(torch.int32)
        table, first = torch.full((case["B"], width), -1, dtype=torch.int32, device="cuda"), 0
        for b, n in enumerate(had):
            table[b, :n] = order[first:first + n]
            first += n
        st["table"], st["lens"], st["delta"] = table, _ints(lens), _ints(delta)
        st["free"] = torch.full((used + spare,), -1, dtype=torch.int32, device="cuda")
        st["free"][:spare] = order[used:]
        st["count"] = _ints([spare])
        rows = sum(x for x in delta if x > 0) + case["behind"]
        st["slots"] = torch.empty(rows, dtype=torch.int64, device="cuda")
        st["positions"] = torch.empty(rows, dtype=torch.int32, device="cuda")
        return st
    dtype, B, page, d, Hkv = _type(case["dtype"]), case["B"], case["page"], case["d"], case["Hkv"]
    new = _lengths(case)
    before = case["before"] if case["op"] == "append" else 0
    lens = [n + before for n in new]
    used, width = sum(_pages(n, page) for n in lens), max(1, max(_pages(n, page) for n in lens))
    order = torch.randperm(used + 3, generator=g, device="cuda").to(torch.int32)[:used].tolist()
    table, at = [], 0
    for n in lens:
        m = _pages(n, page)
        table.append(order[at:at + m] + [0] * (width - m))
        at += m
    st["table"], st["lens"] = _ints(table), _ints(lens)
    st["most"] = max(lens)
    for name in ("k", "v"):
        codes, st[name + "_scales"] = _coded(_normal((used + 3, Hkv, page, d), g, torch.float32))
        if case["layout"] == "nhd":  # tokens beside heads inside a page, seen as [pages, heads, page, d]
            codes = codes.view(torch.uint8).transpose(1, 2).contiguous().transpose(1, 2).view(torch.float8_e4m3fn)
        st[name + "_cache"] = codes
    if case["op"] == "decode":
        st["q"] = _normal((B, case["H"], d), g, dtype, 3.0 if case["cap"] else 1.0)
        st["slopes"] = _slopes(case["H"]) if case["bias"] else None
    else:
        # Some tokens are larger than those before them, so that a half-filled block's scale has to grow.
        size = torch.exp2(torch.randn((sum(new), 1, 1), generator=g, device="cuda"))
        st["k"], st["v"] = ((_normal((sum(new), Hkv, d), g, torch.float32) * size).to(dtype) for _ in range(2))
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        st["cu"] = _ints(cu)
    return st


# ---------------------------------------------------------------------- one pass


def run(st):
    case = st["case"]
    if own:
        return _run_own(st, case)
    return {"prep": _plain_prep, "grad": _plain_grad, "append": _plain_append, "decode": _plain_decode,
            "resize": _plain_resize}[case["op"]](st, case)


def _run_own(st, case):
    import io_aware_exact_fwd_gb300 as fa

    if case["op"] in ("prep", "grad"):
        kw = {"q_weight": st["qw"], "k_weight": st["kw"], "inv_freq": st["freq"], "positions": st["pos"], "norm": case["norm"],
              "interleaved": case["pairs"]}
        if case["op"] == "prep":
            q, k = fa.fa_qk_norm_rope(st["q"], st["k"], **kw)
            return {"q": q, "k": k}
        dq, dk, dqw, dkw = fa.fa_qk_norm_rope_bwd(st["q"], st["k"], st["dq"], st["dk"], **kw)
        return {"dq": dq, "dk": dk, "dqw": dqw, "dkw": dkw}
    if case["op"] == "resize":
        lens, cu, count, status = fa.fa_paged_resize(st["table"], st["lens"], st["delta"], st["free"], st["count"], case["page"],
                                                     slots=st["slots"], positions=st["positions"])
        return {"lens": lens, "cu": cu, "count": count, "status": status, "table": st["table"], "free": st["free"],
                "slots": st["slots"], "positions": st["positions"]}
    cache = (st["k_cache"], st["v_cache"], st["k_scales"], st["v_scales"], st["table"], st["lens"])
    if case["op"] == "decode":
        o, lse = fa.fa_paged_decode_fp8(st["q"], *cache, softcap=case["cap"], slopes=st["slopes"])
        return {"o": o, "lse": lse}
    fa.fa_paged_append_fp8(st["k"], st["v"], *cache, st["cu"])
    return {"k_cache": st["k_cache"], "v_cache": st["v_cache"], "k_scales": st["k_scales"], "v_scales": st["v_scales"]}


def _turns(st, case):
    """cos and sin [B or 1, 1, N, rot / 2] of the rotation's angles; the angles in 64 bits, as far positions need."""
    pos = st["pos"] if st["pos"] is not None else torch.arange(case["N"], device="cuda", dtype=torch.int32)[None]
    angle = pos.double()[:, None, :, None] * st["freq"].double()
    return torch.cos(angle).float(), torch.sin(angle).float()


def _halves(x, case):
    """The two coordinates of every rotated pair (views), and the rest of a head."""
    rot = case["rot"]
    turned = x[..., :rot]
    if case["pairs"]:
        return turned[..., 0::2], turned[..., 1::2], x[..., rot:]
    return turned[..., :rot // 2], turned[..., rot // 2:], x[..., rot:]


def _joined(a, b, rest, case):
    pair = torch.stack((a, b), dim=-1).flatten(-2) if case["pairs"] else torch.cat((a, b), dim=-1)
    return torch.cat((pair, rest), dim=-1)


def _rotated(y, st, case, back):
    if not case["rot"]:
        return y
    c, s = _turns(st, case)
    s = -s if back else s
    a, b, rest = _halves(y, case)
    return _joined(a * c - b * s, a * s + b * c, rest, case)


EPS = 1e-6  # the framework's default


def _plain_prep(st, case):
    def one(x, w):
        y = x.float()
        if case["norm"]:
            y = y * torch.rsqrt((y * y).mean(dim=-1, keepdim=True) + EPS)
            y = y if w is None else y * w.float()
        return _rotated(y, st, case, False).to(x.dtype)

    return {"q": one(st["q"], st["qw"]), "k": one(st["k"], st["kw"])}


def _plain_grad(st, case):
    def one(x, g, w):
        g = _rotated(g.float(), st, case, True)
        if not case["norm"]:
            return g.to(x.dtype), None
        y = x.float()
        r = torch.rsqrt((y * y).mean(dim=-1, keepdim=True) + EPS)
        y = y * r
        h = g if w is None else g * w.float()
        dx = r * (h - y * (h * y).mean(dim=-1, keepdim=True))
        return dx.to(x.dtype), None if w is None else (g * y).double().sum(dim=(0, 1, 2)).float()

    dq, dqw = one(st["q"], st["dq"], st["qw"])
    dk, dkw = one(st["k"], st["dk"], st["kw"])
    return {"dq": dq, "dk": dk, "dqw": dqw, "dkw": dkw}


def _gathered(st, case, name):
    """Tokens [B, Hkv, most, d] of every sequence as 32-bit values, zeros behind its last."""
    page, d, n = case["page"], case["d"], st["most"]
    ids = st["table"].long()[:, :_pages(n, page)]  # [B, pages]
    codes = st[name + "_cache"].float()[ids]       # [B, pages, Hkv, page, d]
    scale = st[name + "_scales"][ids].repeat_interleave(BLOCK, dim=3)[..., None]
    return (codes * scale).transpose(1, 2).reshape(case["B"], case["Hkv"], -1, d)[:, :, :n]


def _plain_decode(st, case):
    B, H, Hkv, d, n = case["B"], case["H"], case["Hkv"], case["d"], st["most"]
    if n == 0:
        return {"o": torch.zeros_like(st["q"]), "lse": torch.full((B, H), float("-inf"), dtype=torch.float32, device="cuda")}
    s = (st["q"].float().view(B, Hkv, H // Hkv, d) @ _gathered(st, case, "k").transpose(2, 3)) * d ** -0.5
    if case["cap"]:
        s = case["cap"] * torch.tanh(s / case["cap"])
    back = st["lens"][:, None] - 1 - torch.arange(n, device="cuda", dtype=torch.int32)
    if case["bias"]:
        s = s - st["slopes"].view(1, Hkv, H // Hkv, 1) * back.float()[:, None, None]
    s = s.masked_fill((back < 0)[:, None, None], float("-inf"))
    top = s.amax(dim=3, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(s - top)
    total = p.sum(dim=3, keepdim=True)
    o = (p @ _gathered(st, case, "v")) / total.clamp(min=1e-30)
    return {"o": o.reshape(B, H, d).to(st["q"].dtype), "lse": (top + torch.log(total)).reshape(B, H)}


def _plain_append(st, case):
    """Every block that gets a new token: its scale from the values that it then holds, its older codes at that scale."""
    page, d, Hkv = case["page"], case["d"], case["Hkv"]
    cu, lens, table = st["cu"].long(), st["lens"].long(), st["table"].long()
    row = torch.arange(st["k"].shape[0], device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    first = lens[b] - (cu[b + 1] - cu[b])  # the sequence's first new position
    pos = first + (row - cu[b])
    block = table[b, pos // page] * (page // BLOCK) + pos % page // BLOCK  # over the whole cache
    old = torch.zeros(st["k_scales"].shape[0] * (page // BLOCK), dtype=torch.int64, device="cuda")
    old[block] = (first - pos // BLOCK * BLOCK).clamp(min=0)  # tokens that the block held before
    touched = torch.zeros(old.shape, dtype=torch.bool, device="cuda")
    touched[block] = True
    out = {}
    for name in ("k", "v"):
        scales = st[name + "_scales"].transpose(1, 2).reshape(-1, Hkv)  # [blocks, Hkv]
        e = torch.where(old[:, None] > 0, torch.frexp(scales)[1] - 1, torch.full_like(scales, -126).to(torch.int32))
        top = torch.zeros_like(scales).index_reduce_(0, block, st[name].float().abs().amax(dim=2), "amax")
        after = _power(torch.where(touched[:, None], torch.maximum(e, _exponent(top)), torch.frexp(scales)[1] - 1))
        codes = st[name + "_cache"].float().transpose(1, 2).reshape(-1, BLOCK, Hkv, d)
        kept = torch.arange(BLOCK, device="cuda")[None] < old[:, None]
        codes = torch.where((kept & touched[:, None])[:, :, None, None], codes * (scales / after)[:, None, :, None], codes)
        codes[block, pos % BLOCK] = st[name].float() / after[block][:, :, None]
        codes = codes.to(torch.float8_e4m3fn).view(-1, page, Hkv, d).transpose(1, 2)
        st[name + "_cache"].view(torch.uint8).copy_(codes.view(torch.uint8))
        st[name + "_scales"].copy_(after.view(-1, page // BLOCK, Hkv).transpose(1, 2))
        out[name + "_cache"], out[name + "_scales"] = st[name + "_cache"], st[name + "_scales"]
    return out


def _plain_resize(st, case):
    page, lens, delta, table, free = case["page"], st["lens"].long(), st["delta"].long(), st["table"], st["free"]
    count, after = st["count"].long(), lens + delta
    had, has = _pages(lens, page), _pages(after, page)
    grow, drop = (has - had).clamp(min=0), (had - has).clamp(min=0)
    col = torch.arange(table.shape[1], device="cuda")[None]
    # Pages given back go behind the free ones, in the sequences' order; new ones come from the end.
    b, c = torch.nonzero((col >= has[:, None]) & (col < had[:, None]), as_tuple=True)
    free[count + (torch.cumsum(drop, 0) - drop)[b] + c - has[b]] = table[b, c]
    total = count + drop.sum()
    b, c = torch.nonzero((col >= had[:, None]) & (col < has[:, None]), as_tuple=True)
    table[b, c] = free[total - 1 - (torch.cumsum(grow, 0) - grow)[b] - (c - had[b])]
    cu = torch.cat((torch.zeros(1, dtype=torch.int64, device="cuda"), torch.cumsum(delta.clamp(min=0), 0)))
    row = torch.arange(st["slots"].shape[0], device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    real = b < case["B"]
    b = b.clamp(max=case["B"] - 1)
    pos = torch.where(real, after[b] - (cu[b + 1] - row), torch.zeros_like(row))
    slots = torch.where(real, table[b, pos // page].long() * page + pos % page, -torch.ones_like(row))
    bad = ((after < 0) | (has > table.shape[1])).sum()[None]
    status = torch.cat(((grow.sum() - total).clamp(min=0), bad))
    return {"lens": after.int(), "cu": cu.int(), "count": (total - grow.sum()).int(), "status": status.int(), "table": table,
            "free": free, "slots": slots, "positions": torch.where(real, pos, -torch.ones_like(pos)).int()}


# ------------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    if case["op"] == "resize":
        return None  # whole numbers, which are equal or wrong
    st = prepare(case, seed)
    return {"prep": _exact_prep, "grad": _exact_prep, "append": _exact_append, "decode": _exact_decode}[case["op"]](st, case)


def _exact_prep(st, case):
    """Pairs as complex numbers, turned by their angles; gradients by differentiating that."""
    grad, out = case["op"] == "grad", {}
    for name in ("q", "k"):
        w = st[name + "w"]
        x = st[name].detach().double().requires_grad_(grad)
        w = None if w is None else w.detach().double().requires_grad_(grad)
        y = x
        if case["norm"]:
            y = x / torch.sqrt(x.square().sum(dim=3, keepdim=True) / case["d"] + EPS)
            y = y if w is None else y * w
        if case["rot"]:
            half = case["rot"] // 2
            i = torch.arange(half, device="cuda")
            one, two = (2 * i, 2 * i + 1) if case["pairs"] else (i, i + half)
            pos = st["pos"].double() if st["pos"] is not None else torch.arange(case["N"], device="cuda").double().expand(case["B"], -1)
            z = torch.complex(y[..., one], y[..., two]) * torch.polar(torch.ones((), dtype=torch.float64, device="cuda").expand(
                case["B"], 1, case["N"], half), (pos[..., None] * st["freq"].double())[:, None])
            y = torch.zeros_like(y).index_add(3, one, z.real).index_add(3, two, z.imag).index_add(
                3, torch.arange(case["rot"], case["d"], device="cuda"), y[..., case["rot"]:])
        if not grad:
            out[name] = y
            continue
        got = torch.autograd.grad(y, (x,) if w is None else (x, w), st["d" + name].double())
        out["d" + name], out["d" + name + "w"] = got[0], None if w is None else got[1]
    return out


def _code(x):
    """The nearest of the 8-bit values (4 bits of exponent, 3 of fraction, up to 448), ties to even."""
    e = (torch.frexp(x.abs())[1] - 1).clamp(min=-6).double()
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _exact_append(st, case):
    """Block by block of every sequence."""
    page, cu, lens, out = case["page"], st["cu"].tolist(), st["lens"].tolist(), {}
    if sum(lens) * case["Hkv"] > 300000:
        return None
    for name in ("k", "v"):
        cache, scales = st[name + "_cache"].float().double(), st[name + "_scales"].double()
        for b in range(case["B"]):
            start = lens[b] - (cu[b + 1] - cu[b])
            for first in range(start // BLOCK * BLOCK, lens[b] if cu[b + 1] > cu[b] else 0, BLOCK):
                p, off = int(st["table"][b, first // page]), first % page
                here = min(BLOCK, lens[b] - first)
                values = torch.zeros((case["Hkv"], here, case["d"]), dtype=torch.float64, device="cuda")
                least = torch.full((case["Hkv"],), -126.0, dtype=torch.float64, device="cuda")
                held = max(0, start - first)
                if held:
                    least = torch.round(torch.log2(scales[p, :, off // BLOCK]))
                    values[:, :held] = cache[p, :, off:off + held] * scales[p, :, off // BLOCK, None, None]
                t = cu[b] + first + held - start
                fresh = st[name][t:t + here - held].double().transpose(0, 1)
                values[:, held:] = fresh
                top = fresh.abs().amax(dim=(1, 2))
                e = torch.round(torch.log2(top / 448.0).clamp(min=-126.0)) - 1.0  # the smallest, or one or two below it
                for _ in range(2):
                    e = torch.where(top > 448.0 * torch.exp2(e), e + 1.0, e)
                e = torch.maximum(e, least)
                scales[p, :, off // BLOCK] = torch.exp2(e)
                cache[p, :, off:off + here] = _code(values / torch.exp2(e)[:, None, None])
        out[name + "_cache"], out[name + "_scales"] = cache, scales
    return out


def _exact_decode(st, case):
    B, H, Hkv, d, page = (case[x] for x in ("B", "H", "Hkv", "d", "page"))
    o = torch.zeros((B, H, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, H), float("-inf"), dtype=torch.float64, device="cuda")
    for b, n in enumerate(st["lens"].tolist()):
        if n == 0:
            continue
        at = torch.arange(n, device="cuda")
        ids = st["table"][b].long()[at // page]
        for hk in range(Hkv):
            k, v = (st[x + "_cache"].view(torch.uint8)[ids, hk, at % page].view(torch.float8_e4m3fn).double() *
                    st[x + "_scales"][ids, hk, at % page // BLOCK].double()[:, None] for x in ("k", "v"))
            for h in range(hk * (H // Hkv), (hk + 1) * (H // Hkv)):
                s = (k * st["q"][b, h].double()).sum(dim=1) / math.sqrt(d)
                if case["cap"]:
                    s = case["cap"] * torch.tanh(s / case["cap"])
                if case["bias"]:
                    s = s - 2.0 ** (-8.0 * (h + 1) / H) * (n - 1 - at).double()
                lse[b, h] = torch.logsumexp(s, dim=0)
                o[b, h] = torch.softmax(s, dim=0) @ v
    return {"o": o, "lse": lse}
