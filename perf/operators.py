"""The operators of a decode step around the expert layers, case by case: what is timed and checked.

Five operators: a residual addition with a root-mean-square norm (bf16 or 8-bit output), a linear
layer of 8-bit activations and 4-bit group-32 weights, writing a paged key/value cache (bf16, int8
or int4), reading rows of it back, and the attention of one new token per sequence over it.

`run` computes a case in plain torch operations (own = False) or with the library's calls
(own = True) on the same state.  `exact` computes the same from the definitions in 64 bits.

Formats (group = 32 consecutive elements, scales in bf16):
  int4 weights   codes int32 [N, K/8], nibble 4j of word w holds q + 8 of element 8w + j; W = s q
  cache          [pages, Hkv, page_size, D] bf16 or int8, or int32 [pages, Hkv, page_size, D/8] in
                 the nibble order above; scales [pages, Hkv, page_size, D/32]; value = s q
                 int8: s = bf16(max|x| / 127), int4: s = bf16(max|x| / 7), q = rint(x / s) within that
"""
import math
import random

import torch

own = False

DEV = "cuda"
GROUP = 32
EPS = 1e-6
LEVELS = {"int8": 127, "int4": 7}


# ------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one request with a short context: the smallest call, launch latency is all of it
        {"name": "attend one short", "op": "attend", "kind": "bf16", "B": 1, "Hq": 8, "Hkv": 2, "D": 64,
         "page": 16, "longest": 257, "ragged": 0, "window": 0, "softcap": 0.0},
        # a serving batch at the library's decode size (64 tokens), lengths of every kind, some empty
        {"name": "attend batch int8", "op": "attend", "kind": "int8", "B": 64, "Hq": 32, "Hkv": 8, "D": 128,
         "page": 32, "longest": 8192, "ragged": 1, "window": 0, "softcap": 0.0},
        # few requests with long documents: the largest, bound by the cache's bytes
        {"name": "attend long bf16", "op": "attend", "kind": "bf16", "B": 4, "Hq": 32, "Hkv": 8, "D": 128,
         "page": 64, "longest": 65536, "ragged": 0, "window": 0, "softcap": 0.0},
        # 4-bit cache, wide heads, a sliding window and capped scores
        {"name": "attend window int4", "op": "attend", "kind": "int4", "B": 48, "Hq": 16, "Hkv": 2, "D": 256,
         "page": 64, "longest": 24000, "ragged": 2, "window": 16384, "softcap": 30.0},
        # a decode step's new rows: one token for each of 64 sequences
        {"name": "write decode int8", "op": "write", "kind": "int8", "T": 64, "Hq": 32, "Hkv": 8, "D": 128, "page": 32},
        # a prompt's rows (the library's prefill size), padded tokens among them
        {"name": "write prompt int4", "op": "write", "kind": "int4", "T": 8192, "Hq": 16, "Hkv": 4, "D": 256, "page": 64},
        # a short shared prefix read back
        {"name": "read short int4", "op": "read", "kind": "int4", "T": 257, "Hkv": 2, "D": 64, "page": 16},
        # long cached prefixes read back for a prompt's attention
        {"name": "read prefix int8", "op": "read", "kind": "int8", "T": 32768, "Hkv": 8, "D": 128, "page": 32},
        # the norm in front of a decode step's linear layers, at the library's hidden size
        {"name": "norm decode 8-bit", "op": "norm", "out": "q8", "T": 64, "H": 2816, "residual": True, "weight": True},
        # the norm in front of a prompt's expert layer
        {"name": "norm prompt bf16", "op": "norm", "out": "bf16", "T": 8192, "H": 2816, "residual": True, "weight": True},
        # the library's dense decode size with 8-bit activations: bound by the weights' bytes
        {"name": "linear decode", "op": "linear", "M": 16, "N": 14336, "K": 4096},
        # a prompt chunk of odd length through a projection of the library's hidden size
        {"name": "linear prompt", "op": "linear", "M": 509, "N": 8192, "K": 2816},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges; its cost stays below the largest listed case's."""
    while True:
        op = rng.choice(["attend", "attend", "write", "read", "norm", "linear"])
        kind = rng.choice(["bf16", "int8", "int4"])
        Hkv, G = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
        D, page = rng.choice([64, 128, 192, 256]), rng.choice([1, 8, 16, 24, 32, 64, 128])
        if op == "attend":
            case = {"op": op, "kind": kind, "B": _log(rng, 1, 256), "Hq": Hkv * G, "Hkv": Hkv, "D": D, "page": page,
                    "longest": _log(rng, 1, 65536), "ragged": rng.randrange(4), "window": rng.choice([0, 0, _log(rng, 1, 8192)]),
                    "softcap": rng.choice([0.0, 0.0, 30.0])}
            # the plain form's 32-bit copies go by the longest sequence
            if case["B"] * case["longest"] * max(Hkv * D, case["Hq"]) > 4 * 65536 * 8 * 128:
                continue
        elif op == "write":
            case = {"op": op, "kind": kind, "T": _log(rng, 1, 8192), "Hq": Hkv * G, "Hkv": Hkv, "D": D, "page": page}
        elif op == "read":
            case = {"op": op, "kind": kind, "T": _log(rng, 1, 32768), "Hkv": Hkv, "D": D, "page": page}
        elif op == "norm":
            case = {"op": op, "out": rng.choice(["bf16", "q8"]), "T": _log(rng, 1, 8192), "H": 8 * _log(rng, 8, 1024),
                    "residual": rng.random() < 0.75, "weight": rng.random() < 0.75}
        else:
            case = {"op": op, "M": _log(rng, 1, 512), "N": _log(rng, 64, 16384), "K": 32 * _log(rng, 4, 256)}
        if work(case)["bytes"] <= 4e8:
            return case


# ------------------------------------------------------------------------------------ the inputs
def _lens(case):
    """The sequences' lengths: a property of the case, so that `work` can count them."""
    if not case["ragged"]:
        return [case["longest"]] * case["B"]
    r = random.Random(case["ragged"])
    lens = [0 if r.random() < 0.05 else _log(r, 1, case["longest"]) if r.random() < 0.5 else r.randint(1, case["longest"])
            for _ in range(case["B"])]
    lens[0] = case["longest"]
    return lens


def _quantise(x, kind):
    """bf16 [..., D] -> (what the cache holds, scales or None), in the formats above."""
    if kind == "bf16":
        return x.clone(), None
    top = LEVELS[kind]
    g = x.float().unflatten(-1, (-1, GROUP))
    s = (g.abs().amax(-1) / top).to(torch.bfloat16)
    sf = s.float().unsqueeze(-1)
    q = torch.where(sf > 0, (g / sf).round().clamp(-top, top), torch.zeros_like(g))
    q = q.flatten(-2).to(torch.int32)
    return (q.to(torch.int8), s) if kind == "int8" else (_pack(q + 8), s)


def _pack(u):
    """Nibbles 0..15 int32 [..., K] -> words int32 [..., K/8]."""
    w = u.unflatten(-1, (-1, 8)) << torch.arange(0, 32, 4, dtype=torch.int32, device=u.device)
    return w.sum(-1).to(torch.int32)


def _nibbles(words):
    """int32 words [..., K/8] -> their codes q in -8..7 as float32 [..., K]."""
    q = (words.unsqueeze(-1) >> torch.arange(0, 32, 4, dtype=torch.int32, device=words.device)) & 15
    return (q - 8).flatten(-2).float()


def _values(codes, scales):
    """What cache rows stand for, float32."""
    if codes.dtype == torch.bfloat16:
        return codes.float()
    q = _nibbles(codes) if codes.dtype == torch.int32 else codes.float()
    return (q.unflatten(-1, (-1, GROUP)) * scales.float().unsqueeze(-1)).flatten(-2)


def _rows(g, T, Hkv, D):
    """Keys or values as a projection gives them: channels of unlike sizes, a few large ones."""
    x = torch.randn((T, Hkv, D), generator=g, device=DEV)
    size = torch.exp(0.4 * torch.randn((Hkv, D), generator=g, device=DEV))
    return (x * size).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]
    if op == "norm":
        T, H = case["T"], case["H"]
        s = {"x": torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16), "residual": None, "weight": None}
        if case["residual"]:
            s["residual"] = (4 * torch.randn((T, H), generator=g, device=DEV)).to(torch.bfloat16)
        if case["weight"]:
            s["weight"] = (1 + 0.3 * torch.randn(H, generator=g, device=DEV)).to(torch.bfloat16)
        if case["out"] == "q8":
            s["values"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    elif op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        x = torch.randn((M, K), generator=g, device=DEV)
        xs = x.abs().amax(-1) / 127
        s = {"xq": (x / xs[:, None]).round().to(torch.int8), "xs": xs,
             "codes": _pack(torch.randint(0, 16, (N, K), generator=g, device=DEV, dtype=torch.int32)),
             "scales": (0.01 * torch.randn((N, K // GROUP), generator=g, device=DEV).abs() + 1e-4).to(torch.bfloat16)}
    elif op == "attend":
        B, Hkv, D, page = case["B"], case["Hkv"], case["D"], case["page"]
        lens = _lens(case)
        need = [-(-n // page) for n in lens]
        pages = sum(need) + 1
        order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        width = max(1, max(need))
        at = torch.arange(width, device=DEV)
        count = torch.tensor(need, device=DEV)
        place = torch.tensor([sum(need[:b]) for b in range(B)], device=DEV)[:, None] + at
        table = torch.where(at < count[:, None], order[place.clamp(max=pages - 1)], torch.full_like(place, -1, dtype=torch.int32))
        s = {"q": torch.randn((B, case["Hq"], D), generator=g, device=DEV).to(torch.bfloat16),
             "page_table": table.contiguous(), "seq_lens": torch.tensor(lens, dtype=torch.int32, device=DEV)}
        for n in "kv":
            x = _rows(g, pages * page, Hkv, D).view(pages, page, Hkv, D).transpose(1, 2)
            s[n], s[n + "_scales"] = _quantise(x.contiguous(), case["kind"])
    else:
        T, Hkv, D, page, kind = case["T"], case["Hkv"], case["D"], case["page"], case["kind"]
        pages = -(-T // page) + 7
        slots = torch.randperm(pages * page, generator=g, device=DEV)[:T]
        if T > 8:
            slots[torch.randperm(T, generator=g, device=DEV)[: T // 50 + 1]] = -1   # padded tokens
        s = {"slots": slots.contiguous()}
        if op == "write":
            # one page more than the call is given: the plain form drops padded tokens there
            shape = (pages + 1, Hkv, page)
            s["qkv"] = _rows(g, T, case["Hq"] + 2 * Hkv, D).view(T, -1)
            wide = {"bf16": (D, torch.bfloat16), "int8": (D, torch.int8), "int4": (D // 8, torch.int32)}[kind]
            for n in "kv":
                s[n] = torch.zeros(shape + (wide[0],), dtype=wide[1], device=DEV)
                s[n + "_scales"] = None if kind == "bf16" else torch.zeros(shape + (D // GROUP,), dtype=torch.bfloat16, device=DEV)
        else:
            for n in "kv":
                x = _rows(g, pages * page, Hkv, D).view(pages, page, Hkv, D).transpose(1, 2)
                s[n], s[n + "_scales"] = _quantise(x.contiguous(), kind)
    s["case"] = case
    return s


def work(case):
    op = case["op"]
    if op == "norm":
        n = case["T"] * case["H"]
        b = n * (2 + (4 if case["residual"] else 0) + (2 if case["out"] == "bf16" else 1)) + (2 * case["H"] if case["weight"] else 0)
        return {"bytes": b + (4 * case["T"] if case["out"] == "q8" else 0), "flops": 6 * n}
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": N * K // 2 + N * K // 16 + M * K + 4 * M + 2 * M * N, "flops": 2 * M * N * K}
    D = case["D"]
    row = {"bf16": 2 * D, "int8": D + D // 16, "int4": D // 2 + D // 16}[case["kind"]]
    if op == "attend":
        seen = sum(min(n, case["window"]) if case["window"] else n for n in _lens(case))
        return {"bytes": 2 * seen * case["Hkv"] * row + 4 * case["B"] * case["Hq"] * D + 8 * case["B"],
                "flops": 4 * seen * case["Hq"] * D}
    n = case["T"] * case["Hkv"]
    return {"bytes": 2 * n * (2 * D + row) + 8 * case["T"], "flops": 6 * n * D}


# ---------------------------------------------------------------------------------- one pass each
def run(s):
    return {"norm": _norm, "linear": _linear, "attend": _attend, "write": _write, "read": _read}[s["case"]["op"]](s)


def _norm(s):
    """h = bf16(x + residual); y = h / sqrt(mean h^2 + eps) * weight, in bf16 or as 8-bit codes with one scale per row."""
    q8 = s["case"]["out"] == "q8"
    if own:
        from w4a16_group_quantized_w4_b200 import api
        if q8:
            q, qs, h = api.w4_rms_add_q8(s["x"], s["residual"], s["weight"], eps=EPS)
            return {"values": torch.mul(q, qs[:, None], out=s["values"]), "scales": qs, "h": h}
        y, h = api.w4_rms_add(s["x"], s["residual"], s["weight"], eps=EPS)
        return {"y": y, "h": h}
    h = s["x"]
    if s["residual"] is not None:
        h = (h.float() + s["residual"].float()).to(torch.bfloat16)
    f = h.float()
    y = f / torch.sqrt(f.square().mean(-1, keepdim=True) + EPS)
    if s["weight"] is not None:
        y = y * s["weight"].float()
    if not q8:
        return {"y": y.to(torch.bfloat16), "h": h}
    qs = y.abs().amax(-1) / 127
    q = torch.where(qs[:, None] > 0, (y / qs[:, None]).round().clamp(-127, 127), torch.zeros_like(y))
    return {"values": torch.mul(q, qs[:, None], out=s["values"]), "scales": qs, "h": h}


def _linear(s):
    """y[m, n] = xs[m] * sum_k xq[m, k] * (scales[n, k/32] * q[n, k])."""
    if own:
        from w4a16_group_quantized_w4_b200 import api
        return api.w4a8_linear(s["xq"], s["xs"], s["codes"], s["scales"])
    return ((s["xq"].float() @ _values(s["codes"], s["scales"]).t()) * s["xs"][:, None]).to(torch.bfloat16)


def _attend(s):
    """Each sequence's one query row over its cached tokens: softmax(cap(q k / sqrt(D))) v per head."""
    case = s["case"]
    if own:
        from w4a16_group_quantized_w4_b200 import api
        return api.kv_cache_attend(s["q"], s["k"], s["v"], s["page_table"], s["seq_lens"], k_scales=s["k_scales"],
                                   v_scales=s["v_scales"], window=case["window"], softcap=case["softcap"])
    B, Hq, D = s["q"].shape
    Hkv, page = case["Hkv"], case["page"]
    pos = torch.arange(s["page_table"].shape[1] * page, device=DEV)
    lens = s["seq_lens"].long()[:, None]
    inside = pos < lens
    if case["window"]:
        inside = inside & (pos >= lens - case["window"])
    at = s["page_table"].long()[:, pos // page].clamp(min=0), pos % page       # [B, L], [L]
    take = lambda t: t[at[0], :, at[1].expand_as(at[0])]                       # noqa: E731  [B, L, Hkv, ...]
    rows = {n: _values(take(s[n]), None if s[n + "_scales"] is None else take(s[n + "_scales"])) for n in "kv"}
    q = s["q"].float().view(B, Hkv, Hq // Hkv, D)
    score = q @ rows["k"].permute(0, 2, 3, 1) / math.sqrt(D)                   # [B, Hkv, G, L]
    if case["softcap"]:
        score = case["softcap"] * torch.tanh(score / case["softcap"])
    score = score.masked_fill(~inside[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    out = (p @ rows["v"].transpose(1, 2)) / torch.where(total > 0, total, torch.ones_like(total))
    return out.reshape(B, Hq, D).to(torch.bfloat16)


def _kv_of(s):
    """The keys' and values' columns of a fused projection's rows (views)."""
    case = s["case"]
    rows = s["qkv"].view(case["T"], -1, case["D"])
    return rows[:, case["Hq"]:case["Hq"] + case["Hkv"]], rows[:, case["Hq"] + case["Hkv"]:]


def _write(s):
    """The tokens' keys and values into their slots (page * page_size + offset; a negative slot is dropped)."""
    k, v = _kv_of(s)
    kind, page = s["case"]["kind"], s["case"]["page"]
    cache = {n: None if s[n] is None else s[n][:-1] for n in ("k", "v", "k_scales", "v_scales")}
    if own:
        from w4a16_group_quantized_w4_b200 import api
        api.kv_cache_write(k, v, s["slots"], cache["k"], cache["v"], k_scales=cache["k_scales"], v_scales=cache["v_scales"])
        return [cache[n] for n in cache if cache[n] is not None]
    last = s["k"].shape[0] - 1
    slot = torch.where(s["slots"] < 0, torch.full_like(s["slots"], last * page), s["slots"])
    for n, x in (("k", k), ("v", v)):
        codes, scales = _quantise(x, kind)
        s[n][slot // page, :, slot % page] = codes
        if scales is not None:
            s[n + "_scales"][slot // page, :, slot % page] = scales
    return [cache[n] for n in cache if cache[n] is not None]


def _read(s):
    """Rows of the cache as bf16 keys and values [T, Hkv, D]; zeros where the slot is negative."""
    if own:
        from w4a16_group_quantized_w4_b200 import api
        return api.kv_cache_read(s["slots"], s["k"], s["v"], k_scales=s["k_scales"], v_scales=s["v_scales"])
    page = s["case"]["page"]
    slot = s["slots"].clamp(min=0)
    keep = (s["slots"] >= 0)[:, None, None]
    out = []
    for n in "kv":
        take = lambda t: t[slot // page, :, slot % page]                       # noqa: E731
        x = _values(take(s[n]), None if s[n + "_scales"] is None else take(s[n + "_scales"]))
        out.append(torch.where(keep, x, torch.zeros_like(x)).to(torch.bfloat16))
    return tuple(out)


# ------------------------------------------------------------------- the definitions in 64 bits
def _exact_codes(words):
    """Packed or int8 codes as float64, one nibble position at a time."""
    if words.dtype != torch.int32:
        return words.double()
    out = torch.empty(words.shape[:-1] + (words.shape[-1] * 8,), dtype=torch.float64, device=words.device)
    for j in range(8):
        out[..., j::8] = ((words >> (4 * j)) & 15).double() - 8
    return out


def _exact_rows(s, n, page, offset):
    """Rows [len, Hkv, D] of cache n at (page, offset), float64."""
    x = _exact_codes(s[n][page, :, offset])
    if s[n + "_scales"] is None:
        return x
    return x * s[n + "_scales"][page, :, offset].double().repeat_interleave(GROUP, dim=-1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        w = _exact_codes(s["codes"]) * s["scales"].double().repeat_interleave(GROUP, dim=-1)
        return (s["xq"].double() * s["xs"].double()[:, None]) @ w.t()
    if op == "norm":
        h = s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double()
        f = h.to(torch.bfloat16).double()           # the norm is of what is stored
        y = f * (f.pow(2).mean(-1, keepdim=True) + EPS).rsqrt()
        y = y if s["weight"] is None else y * s["weight"].double()
        if case["out"] == "bf16":
            return {"y": y, "h": h}
        step = y.abs().max(-1, keepdim=True).values / 127
        return {"values": torch.round(y / step) * step, "scales": step[:, 0], "h": h}
    if op == "attend":
        page, G = case["page"], case["Hq"] // case["Hkv"]
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        for b, n in enumerate(_lens(case)):
            first = max(0, n - case["window"]) if case["window"] else 0
            if n == 0:
                continue
            pos = torch.arange(first, n, device=DEV)
            at = s["page_table"][b].long()[pos // page], pos % page
            for h in range(case["Hkv"]):
                one = {m: s[m][:, h:h + 1] for m in "kv"}
                one.update({m + "_scales": None if s[m + "_scales"] is None else s[m + "_scales"][:, h:h + 1] for m in "kv"})
                k, v = (_exact_rows(one, m, *at)[:, 0] for m in "kv")
                t = s["q"][b, h * G:(h + 1) * G].double() @ k.t() / math.sqrt(case["D"])
                t = t if not case["softcap"] else case["softcap"] * torch.tanh(t / case["softcap"])
                out[b, h * G:(h + 1) * G] = torch.softmax(t, -1) @ v
        return out
    if op == "read":
        keep = s["slots"] >= 0
        slot = s["slots"][keep]
        out = []
        for n in "kv":
            x = torch.zeros((case["T"], case["Hkv"], case["D"]), dtype=torch.float64, device=DEV)
            x[keep] = _exact_rows(s, n, slot // case["page"], slot % case["page"])
            out.append(x)
        return out
    keep = s["slots"] >= 0
    slot = s["slots"][keep]
    found = {}
    for n, x in zip("kv", _kv_of(s)):
        x = x[keep].double()
        if case["kind"] == "bf16":
            whole = torch.zeros(s[n].shape, dtype=torch.float64, device=DEV)
            whole[slot // case["page"], :, slot % case["page"]] = x
            found[n] = whole[:-1]
        else:
            whole = torch.zeros(s[n + "_scales"].shape, dtype=torch.float64, device=DEV)
            whole[slot // case["page"], :, slot % case["page"]] = x.unflatten(-1, (-1, GROUP)).abs().amax(-1) / LEVELS[case["kind"]]
            found[n], found[n + "_scales"] = None, whole[:-1]   # codes are whole numbers
    return [found[n] for n in ("k", "v", "k_scales", "v_scales") if n in found]

