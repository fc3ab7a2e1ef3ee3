"""Measured cases of the key/value-cache operators: `spec_kv_append` (quantise a step's keys and
values into a paged cache), `spec_kv_read` (read them back) and `spec_attend` (the attention of the
verify step's gamma + 1 queries of each sequence, over a prefix that the whole batch shares and the
sequence's own pages).

A cache holds pages [n_pages, Hkv, page, D] of keys and of values, as bfloat16 or as e4m3 with one
power-of-two exponent for each (token, head).  Position p of sequence b is token p of the shared
prefix (p < prefix) or token p - prefix of the sequence's own pages.
"""
import math

import torch

own = False

E_MIN, E_MAX, TOP = -100, 119, 448.0  # range of the stored exponents, largest e4m3 magnitude


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token of one sequence: the smallest write, bound by its launch
        _append("append-token", B=1, gamma=0, Hkv=8, D=128, page=16, lo=700, hi=700),
        # a verify step of a large batch with draft lengths 1..8, keys and values still in float32
        _append("append-ragged", B=512, gamma=8, ragged=True, Hkv=8, D=128, page=64, lo=1, hi=200, src="f32"),
        # two long prompts written at once
        _append("append-prompt", B=2, gamma=16383, Hkv=8, D=128, page=64, lo=0, hi=0),
        # a short odd window read back in float32, across the end of a shared prefix
        _read("read-window", B=4, n=333, Hkv=8, D=80, page=16, prefix=100, lo=150, hi=300, out="f32"),
        # whole long sequences read back, as for moving them to another worker
        _read("read-long", B=16, n=8192, Hkv=8, D=128, page=64, prefix=0, lo=8000, hi=8192, out="bf16"),
        # plain decoding of one sequence: one query token
        _attend("attend-token", B=1, gamma=0, Hq=32, Hkv=8, D=128, page=16, prefix=0, lo=1024, hi=1024),
        # one sequence, four drafts, 200 steps in, unquantised cache, no shared heads
        _attend("attend-single", B=1, gamma=4, Hq=32, Hkv=32, D=80, page=16, prefix=0, lo=200, hi=200, fmt="bf16"),
        # 64 samples of one prompt, four drafts each
        _attend("attend-mixed", B=64, gamma=4, Hq=32, Hkv=8, D=128, page=64, prefix=4096, lo=1, hi=512),
        # few sequences with long own contexts: bound by reading the cache
        _attend("attend-long", B=8, gamma=4, Hq=64, Hkv=8, D=128, page=64, prefix=0, lo=40000, hi=65536),
        # many samples of one long prompt, eight drafts each: bound by the products with the prefix
        _attend("attend-samples", B=256, gamma=8, Hq=32, Hkv=8, D=128, page=64, prefix=8192, lo=1, hi=1024),
        # draft lengths 1..8, small heads, unquantised cache, a prefix that ends inside a page
        _attend("attend-ragged", B=512, gamma=8, ragged=True, Hq=16, Hkv=16, D=64, page=16, prefix=1001,
                lo=0, hi=300, fmt="bf16"),
        # one key/value head for all query heads, odd batch, odd lengths
        _attend("attend-one-head", B=33, gamma=2, Hq=24, Hkv=1, D=96, page=32, prefix=513, lo=7, hi=5001),
    ]


def _append(name, B, gamma, Hkv, D, page, lo, hi, ragged=False, fmt="e4m3", src="bf16"):
    return dict(name=name, op="append", B=B, gamma=gamma, ragged=ragged, Hkv=Hkv, D=D, page=page, prefix=0,
                lo=lo, hi=hi, fmt=fmt, src=src)


def _read(name, B, n, Hkv, D, page, prefix, lo, hi, out, fmt="e4m3"):
    return dict(name=name, op="read", B=B, n=n, Hkv=Hkv, D=D, page=page, prefix=prefix, lo=lo, hi=hi, fmt=fmt, out=out)


def _attend(name, B, gamma, Hq, Hkv, D, page, prefix, lo, hi, ragged=False, fmt="e4m3"):
    return dict(name=name, op="attend", B=B, gamma=gamma, ragged=ragged, Hq=Hq, Hkv=Hkv, D=D, page=page,
                prefix=prefix, lo=lo, hi=hi, fmt=fmt)


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["append", "read", "attend", "attend"])
    page = rng.choice([16, 32, 64, 128])
    D = rng.choice([64, 80, 96, 128])
    fmt = rng.choice(["e4m3", "e4m3", "bf16"])
    while True:
        if op == "append":
            if rng.random() < 0.5:  # verify steps
                c = _append("", B=_log(rng, 1, 512), gamma=rng.randint(0, 8), ragged=False, Hkv=rng.choice([1, 4, 8, 16]),
                            D=D, page=page, lo=0, hi=rng.randint(0, 300), fmt=fmt, src=rng.choice(["bf16", "f32"]))
                c["ragged"] = c["gamma"] > 1 and rng.random() < 0.5
            else:  # prompts
                c = _append("", B=rng.randint(1, 3), gamma=_log(rng, 30, 16000) - 1, Hkv=rng.choice([1, 4, 8]), D=D,
                            page=page, lo=0, hi=rng.randint(0, 300), fmt=fmt, src=rng.choice(["bf16", "f32"]))
        elif op == "read":
            hi = _log(rng, 10, 8000)
            c = _read("", B=_log(rng, 1, 24), n=0, Hkv=rng.choice([1, 4, 8]), D=D, page=page, prefix=rng.choice([0, _log(rng, 1, 2000)]),
                      lo=rng.randint(1, hi), hi=hi, out=rng.choice(["bf16", "f32"]), fmt=fmt)
            c["n"] = c["prefix"] + hi + rng.randint(0, 20)
        else:
            Hkv = rng.choice([1, 2, 8, 16])
            hi = _log(rng, 3, 30000)
            c = _attend("", B=_log(rng, 1, 300), gamma=rng.randint(0, 8), Hq=Hkv * rng.choice([1, 2, 4, 7, 8]), Hkv=Hkv, D=D,
                        page=page, prefix=rng.choice([0, _log(rng, 1, 8000)]), lo=rng.randint(0, hi), hi=hi, fmt=fmt)
            c["ragged"] = c["gamma"] > 1 and rng.random() < 0.4
        w = work(c)
        tokens = c["prefix"] + sum(_lens(c)) + c["B"] * (c.get("gamma", 0) + 1)
        if w["bytes"] < 8e8 and w["flops"] < 2.5e11 and tokens * c["Hkv"] * c["D"] < 6e8 and _scores(c) < 7e8:
            del c["name"]
            return c


def _scores(c):
    if c["op"] != "attend":
        return 0
    return c["B"] * (c["gamma"] + 1) * c["Hq"] * (c["prefix"] + c["hi"] + c["gamma"] + 1)


def _lens(c):
    """Own tokens that each sequence holds before the step (before reading: in all)."""
    B, lo, hi = c["B"], c["lo"], c["hi"]
    return [lo + (hi - lo) * (b * 7919 % 1009) // 1008 if B > 1 else hi for b in range(B)]


def _gammas(c):
    g = c.get("gamma", 0)
    return [1 + (5 * b + 3) % g if c.get("ragged") else g for b in range(c["B"])]


def _own_tokens(c):
    """Own tokens that the cache holds when the operator has run."""
    if c["op"] == "read":
        return _lens(c)
    return [n + g + 1 for n, g in zip(_lens(c), _gammas(c))]


def work(case):
    c = case
    B, Hkv, D, N = c["B"], c["Hkv"], c["D"], c.get("gamma", 0) + 1
    held = Hkv * 2 * (2 * D if c["fmt"] == "bf16" else D + 1)  # bytes of one token in the cache
    pages = lambda n: 4 * sum(-(-x // c["page"]) for x in n)  # noqa: E731
    if c["op"] == "append":
        n = sum(g + 1 for g in _gammas(c))
        return {"bytes": n * (held + Hkv * 2 * D * (4 if c["src"] == "f32" else 2) + 4) + 8 * B, "flops": 2 * n * Hkv * 2 * D}
    if c["op"] == "read":
        n = c["prefix"] + sum(min(x, c["n"] - c["prefix"]) for x in _lens(c))
        out = B * c["n"] * Hkv * 2 * D * (4 if c["out"] == "f32" else 2)
        return {"bytes": n * held + out + pages([c["prefix"]] + _lens(c)) + 4 * B, "flops": B * c["n"] * Hkv * 2 * D}
    n = c["prefix"] + sum(_own_tokens(c))
    q = sum(g + 1 for g in _gammas(c)) * c["Hq"]
    seen = sum((g + 1) * (c["prefix"] + x) + (g + 1) * (g + 2) // 2 for g, x in zip(_gammas(c), _lens(c)))
    return {"bytes": n * held + q * D * 2 + B * N * c["Hq"] * (D * 2 + 4) + pages([c["prefix"]] + _own_tokens(c)) + 8 * B,
            "flops": 4 * seen * c["Hq"] * D}


# ----------------------------------------------------------------- inputs
def _tokens(gen, n, Hkv, D, key):
    """n tokens [n, Hkv, D] in float32: keys have a few strong channels and a token-wise size, values little of either."""
    x = torch.randn((n, Hkv, D), generator=gen, device="cuda")
    channel = torch.exp(torch.randn((Hkv, D), generator=gen, device="cuda") * (0.5 if key else 0.2))
    size = torch.exp(torch.randn((n, 1, 1), generator=gen, device="cuda") * (0.1 if key else 0.5))
    return x.mul_(channel).mul_(size)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B, Hkv, D, page, prefix = c["B"], c["Hkv"], c["D"], c["page"], c["prefix"]
    turn = seed % B
    roll = lambda v: v[turn:] + v[:turn]  # noqa: E731
    lens, gammas, tokens = roll(_lens(c)), roll(_gammas(c)), roll(_own_tokens(c))
    most = max(1, -(-max(tokens) // page))
    shared = -(-prefix // page)
    n_pages = shared + sum(-(-x // page) for x in tokens) + 3
    ids = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros((B, most), dtype=torch.int32)
    order, at = ids.cpu(), shared
    for b, x in enumerate(tokens):
        p = -(-x // page)
        table[b, :p] = order[at:at + p]
        at += p
    int32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    s = dict(case=c, table=table.cuda(), kv_len=int32([prefix + n for n in lens]), prefix=prefix,
             prefix_table=ids[:shared].contiguous(), gamma=int32(gammas) if c.get("ragged") else None)
    cache = []
    for key in (True, False):
        if c["op"] == "append":  # pages in use before: their old contents are overwritten or stay
            x = torch.zeros((n_pages, Hkv, page, D), device="cuda")
        else:
            x = _tokens(gen, n_pages * page, Hkv, D, key).view(n_pages, page, Hkv, D).transpose(1, 2)
        if c["fmt"] == "e4m3":
            e = _exponent(x)
            cache.append(((x * _pow2(-e)[..., None]).to(torch.float8_e4m3fn).contiguous(), e.to(torch.int8).contiguous()))
        else:
            cache.append((x.to(torch.bfloat16).contiguous(), None))
        del x
    (s["k_pages"], s["k_exp"]), (s["v_pages"], s["v_exp"]) = cache
    if c["op"] == "append":
        N = c["gamma"] + 1
        src = torch.float32 if c["src"] == "f32" else torch.bfloat16
        s["k"], s["v"] = (_tokens(gen, B * N, Hkv, D, key).view(B, N, Hkv, D).to(src) for key in (True, False))
    if c["op"] == "attend":
        s["q"] = _tokens(gen, B * (c["gamma"] + 1), c["Hq"], D, True).view(B, c["gamma"] + 1, c["Hq"], D).to(torch.bfloat16)
    if own:  # the handle that a program keeps beside its pages
        import speculative_decoding_verify_03_gb300 as sv
        s["cache"] = sv.KVCache(s["k_pages"], s["v_pages"], s["k_exp"], s["v_exp"])
    return s


# ------------------------------------------------------------------- run
def run(s):
    c = s["case"]
    if own:
        import speculative_decoding_verify_03_gb300 as sv
        if c["op"] == "append":
            sv.spec_kv_append(s["cache"], s["k"], s["v"], s["table"], s["kv_len"], gamma_per_row=s["gamma"])
            return _held(s)
        if c["op"] == "read":
            return sv.spec_kv_read(s["cache"], s["table"], s["kv_len"], c["n"], prefix_table=s["prefix_table"],
                                   prefix_len=s["prefix"], dtype=torch.float32 if c["out"] == "f32" else torch.bfloat16)
        return sv.spec_attend(s["q"], s["cache"], s["table"], s["kv_len"], prefix_table=s["prefix_table"],
                              prefix_len=s["prefix"], gamma_per_row=s["gamma"])
    if c["op"] == "append":
        _plain_append(s, s["k"], s["k_pages"], s["k_exp"])
        _plain_append(s, s["v"], s["v_pages"], s["v_exp"])
        return _held(s)
    if c["op"] == "read":
        return tuple(_plain_read(s, pages, exp) for pages, exp in ((s["k_pages"], s["k_exp"]), (s["v_pages"], s["v_exp"])))
    return _plain_attend(s)


def _held(s):
    return tuple(s[k] for k in ("k_pages", "v_pages", "k_exp", "v_exp") if s[k] is not None)


def _pow2(e):
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _exponent(x):
    """The least integer e in [E_MIN, E_MAX] with max |x| <= 448 * 2^e over the last axis."""
    most = x.abs().amax(-1)
    frac, k = torch.frexp(most)  # most = frac * 2^k, frac in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(frac <= 0.875, k - 9, k - 8)
    return torch.where(most > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)


def _places(s, N):
    """Page and slot of each token of the step, and which tokens there are."""
    c = s["case"]
    t = torch.arange(N, device="cuda")
    pos = s["kv_len"][:, None].long() - s["prefix"] + t
    there = t <= s["gamma"][:, None] if s["gamma"] is not None else torch.ones_like(pos, dtype=torch.bool)
    pos = torch.where(there, pos, torch.zeros_like(pos))
    return torch.gather(s["table"].long(), 1, pos // c["page"]), pos % c["page"], there


def _plain_append(s, x, pages, exp):
    page, slot, there = _places(s, x.shape[1])
    page, slot, x = page[there], slot[there], x[there].float()
    if exp is None:
        pages[page, :, slot] = x.to(torch.bfloat16)
        return
    e = _exponent(x)
    y = (x * _pow2(-e)[..., None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn)
    pages.view(torch.uint8)[page, :, slot] = y.view(torch.uint8)
    exp[page, :, slot] = e.to(torch.int8)


def _gather(pages, exp, table):
    """[..., p] page ids -> float32 [..., Hkv, p * page, D]"""
    t = table.long()
    x = (pages.view(torch.uint8)[t].view(torch.float8_e4m3fn) if exp is not None else pages[t]).float()
    if exp is not None:
        x = x * _pow2(exp[t])[..., None]
    return x.movedim(-3, -4).flatten(-3, -2)


def _plain_read(s, pages, exp):
    c = s["case"]
    B, n, P = c["B"], c["n"], s["prefix"]
    x = _gather(pages, exp, s["table"])[:, :, :n - P]
    if P:
        x = torch.cat([_gather(pages, exp, s["prefix_table"])[None, :, :P].expand(B, -1, -1, -1), x], 2)
    out = torch.zeros((B, c["Hkv"], n, c["D"]), device="cuda")
    out[:, :, :x.shape[2]] = x
    out *= (torch.arange(n, device="cuda") < s["kv_len"][:, None])[:, None, :, None]
    return out.transpose(1, 2).to(torch.float32 if c["out"] == "f32" else torch.bfloat16)


def _plain_attend(s):
    c = s["case"]
    B, N, Hq, Hkv, D, P = c["B"], c["gamma"] + 1, c["Hq"], c["Hkv"], c["D"], s["prefix"]
    G = Hq // Hkv
    q = s["q"].float().view(B, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, D) / math.sqrt(D)
    k, v = (_gather(s[a + "_pages"], s[a + "_exp"], s["table"]) for a in "kv")
    i = torch.arange(N, device="cuda").repeat_interleave(G)
    sees = torch.arange(k.shape[2], device="cuda") <= s["kv_len"][:, None, None] - P + i[:, None]  # [B, N * G, T]
    if s["gamma"] is not None:
        sees &= (i <= s["gamma"][:, None])[:, :, None]
    score = (q @ k.transpose(-1, -2)).masked_fill_(~sees[:, None], -math.inf)
    most = score.amax(-1, keepdim=True)
    if P:  # the prefix's keys and values stand once, for all sequences
        kp, vp = (_gather(s[a + "_pages"], s[a + "_exp"], s["prefix_table"])[:, :P] for a in "kv")
        flat = q.transpose(0, 1).reshape(Hkv, B * N * G, D)
        score_p = (flat @ kp.transpose(-1, -2)).view(Hkv, B, N * G, P).transpose(0, 1)
        most = torch.maximum(most, score_p.amax(-1, keepdim=True))
    most = most.masked_fill(most == -math.inf, 0)
    w = score.sub_(most).exp_()
    total, out = w.sum(-1, keepdim=True), w @ v
    del score, w
    if P:
        w = score_p.sub_(most).exp_()
        total = total + w.sum(-1, keepdim=True)
        out = out + (w.transpose(0, 1).reshape(Hkv, B * N * G, P) @ vp).view(Hkv, B, N * G, D).transpose(0, 1)
    out, lse = out / total, (most + total.log())[..., 0]
    if s["gamma"] is not None:
        none = (i > s["gamma"][:, None])[:, None]
        out, lse = out.masked_fill(none[..., None], 0), lse.masked_fill(none, -math.inf)
    back = lambda x: x.view(B, Hkv, N, G, -1).permute(0, 2, 1, 3, 4).reshape(B, N, Hq, -1)  # noqa: E731
    return back(out).to(torch.bfloat16), back(lse)[..., 0]


# ----------------------------------------------------------------- exact
def _two_to(e):
    """2.0 ** e in float64, exactly (a power function may be off by a unit in the last place)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def exact(case, seed):
    """From the definitions, token by token of the tables, in float64."""
    c, s = case, prepare(case, seed)
    return {"append": _exact_append, "read": _exact_read, "attend": _exact_attend}[c["op"]](c, s)


def _value(s, which, rows):
    """Dequantised [n, Hkv, D] of the cache's tokens rows = (page ids, slots)."""
    page, slot = rows
    x = s[which + "_pages"]
    if s[which + "_exp"] is None:
        return x[page, :, slot].double()
    codes = x.view(torch.uint8)[page, :, slot].long()
    mant, expo = codes & 7, (codes >> 3) & 15
    v = torch.where(expo > 0, (8 + mant).double() * _two_to(expo - 10), mant.double() * 2.0 ** -9)
    v = torch.where(codes >= 128, -v, v)
    return v * _two_to(s[which + "_exp"][page, :, slot])[..., None]


def _rows_of(s, table_row, first, n):
    p = torch.arange(first, first + n, device="cuda")
    return table_row.long()[p // s["case"]["page"]], p % s["case"]["page"]


def _exact_append(c, s):
    out = {k: s[k].to(torch.float64) for k in ("k_pages", "v_pages")}
    exps = {k: s[k] for k in ("k_exp", "v_exp")}
    lens = s["kv_len"].tolist()
    n = [g + 1 for g in (s["gamma"].tolist() if s["gamma"] is not None else [c["gamma"]] * c["B"])]
    for b in range(c["B"]):
        page, slot = _rows_of(s, s["table"][b], lens[b], n[b])
        for a in "kv":
            x = s[a][b, :n[b]].double()
            if c["fmt"] == "bf16":
                out[a + "_pages"][page, :, slot] = x.float().to(torch.bfloat16).double()
                continue
            most = x.abs().amax(-1)
            e = torch.ceil(torch.log2(most / TOP)).clamp(E_MIN, E_MAX)
            e = torch.where(most > TOP * _two_to(e), e + 1, e)
            e = torch.where((most <= TOP * _two_to(e - 1)) & (e > E_MIN), e - 1, e).clamp(E_MIN, E_MAX)
            y = x / _two_to(e)[..., None]
            step = _two_to(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
            out[a + "_pages"][page, :, slot] = torch.round(y / step) * step
            exps[a + "_exp"][page, :, slot] = e.to(torch.int8)
    return tuple(x for x in (out["k_pages"], out["v_pages"], exps["k_exp"], exps["v_exp"]) if x is not None)


def _exact_read(c, s):
    outs = []
    for a in "kv":
        out = torch.zeros((c["B"], c["n"], c["Hkv"], c["D"]), dtype=torch.float64, device="cuda")
        P = s["prefix"]
        for b, held in enumerate(s["kv_len"].tolist()):
            if P:
                out[b, :P] = _value(s, a, _rows_of(s, s["prefix_table"], 0, P))
            m = min(held, c["n"]) - P
            out[b, P:P + m] = _value(s, a, _rows_of(s, s["table"][b], 0, m))
        outs.append(out)
    return tuple(outs)


def _exact_attend(c, s):
    B, N, Hq, Hkv, D, P = c["B"], c["gamma"] + 1, c["Hq"], c["Hkv"], c["D"], s["prefix"]
    if work(c)["flops"] > 4e11:
        return None
    G = Hq // Hkv
    out = torch.zeros((B, N, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, N, Hq), -math.inf, dtype=torch.float64, device="cuda")
    lens = s["kv_len"].tolist()
    gam = s["gamma"].tolist() if s["gamma"] is not None else [c["gamma"]] * B
    kp, vp = (_value(s, a, _rows_of(s, s["prefix_table"], 0, P)) if P else None for a in "kv")
    for b in range(B):
        n, held = gam[b] + 1, lens[b] - P + gam[b] + 1
        k, v = (_value(s, a, _rows_of(s, s["table"][b], 0, held)) for a in "kv")
        if P:
            k, v = torch.cat([kp, k]), torch.cat([vp, v])
        q = s["q"][b, :n].double().view(n, Hkv, G, D)
        z = torch.einsum("nhgd,thd->hngt", q, k) / math.sqrt(D)
        last = lens[b] + torch.arange(n, device="cuda")
        z = torch.where(torch.arange(k.shape[0], device="cuda") <= last[:, None, None], z, torch.full_like(z, -math.inf))
        lse[b, :n] = torch.logsumexp(z, -1).permute(1, 0, 2).reshape(n, Hq)
        out[b, :n] = torch.einsum("hngt,thd->nhgd", torch.softmax(z, -1), v).reshape(n, Hq, D)
    return out, lse
