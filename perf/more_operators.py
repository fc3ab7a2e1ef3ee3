"""Measured cases of the operators for drafted trees and for the sequences around them.

A step of sequence b holds nodes 0 .. gamma_b: node 0 is the last committed token, node j >= 1 is draft
j - 1, whose parent is node parents[b, j - 1] < j (a chain: j - 1).

- `spec_attend_tree`: attention of all nodes over the cache, each seeing what is before the step and the
  nodes of its mask row (its ancestors and itself).
- `spec_tree_mask`, `spec_tree_accept`, `spec_kv_compact`: masks and depths from parents, the walk along the
  tokens that the target drew, and the accepted nodes' cache entries moved to consecutive positions.
- `spec_kv_resize`, `spec_kv_fork`, `spec_kv_copy`: page tables over a pool with reference counts.
- `spec_adjust`: penalties for repeated tokens, biases and grammar masks on the logits of every node.
"""
import math

import torch

own = False

E_MIN, E_MAX, TOP = -100, 119, 448.0  # range of the stored exponents, largest e4m3 magnitude
NO_PAGES = 1 << 9  # status bit of a sequence that the pool has no pages for


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one sequence, a tree of 26 nodes, a thousand tokens in: bound by its launches
        _attend("attend-one", B=1, gamma=25, Hq=32, Hkv=8, D=128, page=16, prefix=0, lo=1024, hi=1024),
        # a batch with trees of 64 nodes over long contexts: bound by the products
        _attend("attend-batch", B=16, gamma=63, Hq=32, Hkv=8, D=128, page=64, prefix=0, lo=2000, hi=8192),
        # small trees of 2..15 nodes for samples of one prompt, unquantised cache, no shared heads
        _attend("attend-shared", B=48, gamma=14, ragged=True, Hq=16, Hkv=16, D=64, page=16, prefix=1001, lo=0,
                hi=300, fmt="bf16"),
        # after the forward pass of one sequence's tree
        _step("step-one", B=1, gamma=25, Hkv=8, D=128, page=16, lo=300, hi=300),
        # of a large batch's, over an unquantised cache
        _step("step-batch", B=256, gamma=63, Hkv=8, D=128, page=64, lo=1, hi=200, fmt="bf16"),
        # room for a step's nine tokens in small pages, and back to what was there
        _pages("pages-step", B=512, page=16, n=9, lo=1, hi=4000, n_pages=98304),
        # long prompts come, and go again, in a pool half of which others hold
        _pages("pages-prompts", B=64, page=16, n=16384, lo=0, hi=0, n_pages=262144),
        # three more samples of one sequence
        _fork("fork-one", B=4, parents=1, Hkv=8, D=128, page=16, lo=1000, hi=1000),
        # 31 samples each of eight sequences, large pages
        _fork("fork-samples", B=256, parents=8, Hkv=8, D=128, page=128, lo=3000, hi=4000),
        # one decoded token of one sequence, penalties alone
        _adjust("adjust-token", B=1, gamma=0, V=50304, dtype="f32", lo=200, hi=200),
        # a verify step of four drafts, penalties and biases
        _adjust("adjust-chain", B=64, gamma=4, V=50304, dtype="f32", lo=100, hi=4000, bias=16),
        # trees of 2..31 nodes of a large vocabulary, a grammar's mask at every node
        _adjust("adjust-tree", B=32, gamma=30, ragged=True, V=152064, dtype="bf16", lo=0, hi=2000, bias=16,
                tree=True, grammar=True),
    ]


def _attend(name, B, gamma, Hq, Hkv, D, page, prefix, lo, hi, ragged=False, fmt="e4m3"):
    return dict(name=name, op="attend", B=B, gamma=gamma, ragged=ragged, Hq=Hq, Hkv=Hkv, D=D, page=page,
                prefix=prefix, lo=lo, hi=hi, fmt=fmt)


def _step(name, B, gamma, Hkv, D, page, lo, hi, ragged=False, fmt="e4m3"):
    return dict(name=name, op="step", B=B, gamma=gamma, ragged=ragged, Hkv=Hkv, D=D, page=page, prefix=0, lo=lo,
                hi=hi, fmt=fmt)


def _pages(name, B, page, n, lo, hi, n_pages):
    return dict(name=name, op="pages", B=B, page=page, n=n, lo=lo, hi=hi, n_pages=n_pages)


def _fork(name, B, parents, Hkv, D, page, lo, hi, fmt="e4m3"):
    return dict(name=name, op="fork", B=B, parents=parents, Hkv=Hkv, D=D, page=page, prefix=0, lo=lo, hi=hi, fmt=fmt)


def _adjust(name, B, gamma, V, dtype, lo, hi, ragged=False, tree=False, bias=0, grammar=False):
    return dict(name=name, op="adjust", B=B, gamma=gamma, ragged=ragged, V=V, dtype=dtype, lo=lo, hi=hi, tree=tree,
                bias=bias, grammar=grammar)


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "step", "pages", "fork", "adjust", "adjust"])
    page = rng.choice([16, 32, 64, 128])
    D = rng.choice([64, 80, 96, 128])
    fmt = rng.choice(["e4m3", "e4m3", "bf16"])
    while True:
        if op == "attend":
            Hkv, hi = rng.choice([1, 2, 8, 16]), _log(rng, 3, 20000)
            c = _attend("", B=_log(rng, 1, 128), gamma=_log(rng, 1, 100), Hq=Hkv * rng.choice([1, 2, 4, 7, 8]), Hkv=Hkv,
                        D=D, page=page, prefix=rng.choice([0, _log(rng, 1, 4000)]), lo=rng.randint(0, hi), hi=hi, fmt=fmt)
            tokens = c["prefix"] + sum(_lens(c)) + c["B"] * (c["gamma"] + 1)
            scores = c["B"] * (c["gamma"] + 1) * c["Hq"] * (c["prefix"] + c["hi"] + c["gamma"] + 1)
            fits = tokens * Hkv * D < 4e8 and scores < 4e8
        elif op == "step":
            hi = _log(rng, 3, 1000)
            c = _step("", B=_log(rng, 1, 300), gamma=_log(rng, 2, 100), Hkv=rng.choice([1, 4, 8]), D=D, page=page,
                      lo=rng.randint(0, hi), hi=hi, fmt=fmt)
            fits = (sum(_lens(c)) + c["B"] * (c["gamma"] + 1)) * c["Hkv"] * D < 4e8 and c["B"] * c["gamma"] < 17000
        elif op == "pages":
            hi = _log(rng, 1, 8000)
            c = _pages("", B=_log(rng, 1, 512), page=page, n=_log(rng, 1, 8000), lo=rng.randint(0, hi), hi=hi, n_pages=0)
            c["n_pages"] = 2 * sum(-(-(x + c["n"]) // page) for x in _lens(c)) + rng.randint(1, 1000)
            fits = c["n_pages"] < 250000
        elif op == "fork":
            hi, parents = _log(rng, 2, 6000), _log(rng, 1, 20)
            c = _fork("", B=parents * rng.randint(2, 17), parents=parents, Hkv=rng.choice([1, 4, 8]), D=D, page=page,
                      lo=rng.randint(1, hi), hi=hi, fmt=fmt)
            fits = (sum(_lens(c)[:parents]) + c["B"] * page) * c["Hkv"] * D < 4e8
        else:
            hi = _log(rng, 10, 8000)
            c = _adjust("", B=_log(rng, 1, 128), gamma=_log(rng, 1, 40) - 1, V=_log(rng, 100, 160000),
                        dtype=rng.choice(["f32", "bf16"]), lo=rng.randint(0, hi), hi=hi, bias=rng.choice([0, 7, 40]),
                        grammar=rng.random() < 0.5)
            c["tree"] = c["gamma"] > 3 and rng.random() < 0.5
            fits = c["B"] * (c["gamma"] + 1) * c["V"] < 1.4e8
        if "ragged" in c:
            c["ragged"] = c["gamma"] > 1 and rng.random() < 0.4
        w = work(c)
        if fits and w["bytes"] < 6e8 and w["flops"] < 8e10:
            del c["name"]
            return c


def _lens(c):
    """Own tokens that each sequence holds before the call."""
    B, lo, hi = c["B"], c["lo"], c["hi"]
    return [lo + (hi - lo) * (b * 7919 % 1009) // 1008 if B > 1 else hi for b in range(B)]


def _gammas(c):
    g = c["gamma"]
    return [1 + (5 * b + 3) % g if c["ragged"] else g for b in range(c["B"])]


def _up(x, y):
    return -(-x // y)


def work(case):
    c = case
    B = c["B"]
    if "Hkv" in c:  # bytes of one token in the cache
        held = c["Hkv"] * 2 * (2 * c["D"] if c["fmt"] == "bf16" else c["D"] + 1)
    if c["op"] == "attend":
        N, D, P = c["gamma"] + 1, c["D"], c["prefix"]
        nodes = [g + 1 for g in _gammas(c)]
        tokens = [x + n for x, n in zip(_lens(c), nodes)]
        seen = sum(n * (P + x) + n * min(n, 8) for n, x in zip(nodes, _lens(c)))  # a node sees some eight of the step
        pages = _up(P, c["page"]) + sum(_up(x, c["page"]) for x in tokens)
        return {"bytes": (P + sum(tokens)) * held + sum(nodes) * c["Hq"] * D * 2 + B * N * c["Hq"] * (D * 2 + 4)
                + sum(nodes) * _up(N, 32) * 4 + 4 * pages + 8 * B, "flops": 4 * seen * c["Hq"] * D}
    if c["op"] == "step":  # some four accepted nodes are moved
        N, n = c["gamma"] + 1, sum(_gammas(c)) + B
        return {"bytes": B * N * (_up(N, 32) + 2) * 4 + n * 12 + B * (16 + 2 * 4 * held), "flops": 4 * n}
    if c["op"] == "pages":
        taken = sum(_up(x + c["n"], c["page"]) - _up(x, c["page"]) for x in _lens(c))
        return {"bytes": taken * 24 + B * 24, "flops": taken}
    if c["op"] == "fork":
        each = B // c["parents"] - 1
        own_tokens = _lens(c)[:c["parents"]]
        full = each * sum(x // c["page"] for x in own_tokens)
        return {"bytes": each * sum(2 * (x % c["page"]) * held for x in own_tokens) + full * 24 + B * 40, "flops": full}
    N, V = c["gamma"] + 1, c["V"]
    return {"bytes": B * N * V * 2 * (4 if c["dtype"] == "f32" else 2) + 4 * sum(_lens(c)) + 4 * B * N
            + (4 * B * N * _up(V, 32) if c["grammar"] else 0) + 8 * B * c["bias"], "flops": B * N * V}


# ----------------------------------------------------------------- inputs
def _tokens(gen, n, Hkv, D, key):
    """n tokens [n, Hkv, D] in float32: keys have a few strong channels and a token-wise size, values little of either."""
    x = torch.randn((n, Hkv, D), generator=gen, device="cuda")
    channel = torch.exp(torch.randn((Hkv, D), generator=gen, device="cuda") * (0.5 if key else 0.2))
    size = torch.exp(torch.randn((n, 1, 1), generator=gen, device="cuda") * (0.1 if key else 0.5))
    return x.mul_(channel).mul_(size)


def _pow2(e):
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _fill_cache(s, c, gen, n_pages):
    """Pages [n_pages, Hkv, page, D] of keys and values, e4m3 with exponents or bfloat16."""
    for a in "kv":
        x = _tokens(gen, n_pages * c["page"], c["Hkv"], c["D"], a == "k").view(n_pages, c["page"], c["Hkv"], c["D"])
        x = x.transpose(1, 2)
        s[a + "_exp"] = None
        if c["fmt"] == "e4m3":
            most = x.abs().amax(-1)
            frac, k = torch.frexp(most)  # most = frac * 2^k; 448 = 0.875 * 2^9
            e = torch.where(frac <= 0.875, k - 9, k - 8).clamp(E_MIN, E_MAX)
            s[a + "_exp"] = e.to(torch.int8).contiguous()
            x = (x * _pow2(-e)[..., None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn)
        else:
            x = x.to(torch.bfloat16)
        s[a + "_pages"] = x.contiguous()
    if own:  # the handle that a program keeps beside its pages
        import speculative_decoding_verify_03_gb300 as sv
        s["cache"] = sv.KVCache(s["k_pages"], s["v_pages"], s["k_exp"], s["v_exp"])


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _trees(B, gamma, seed):
    """Parents [B, gamma] of trees whose nodes stand level by level."""
    g = torch.Generator().manual_seed(seed)
    j = torch.arange(1, gamma + 1)
    p = (torch.rand((B, gamma), generator=g) * j * 0.6).long()
    return p.cummax(1).values if gamma else p


def _reach(parents):
    """[B, N, N] truth values: node j is node i or an ancestor of it."""
    B, N = parents.shape[0], parents.shape[1] + 1
    seen = torch.zeros((B, N, N), dtype=torch.bool)
    seen[:, 0, 0] = True
    rows = torch.arange(B)
    for j in range(1, N):
        seen[:, j] = seen[rows, parents[:, j - 1]]
        seen[:, j, j] = True
    return seen


def _words(bits):
    """Truth values [..., n] -> int32 words [..., ceil(n / 32)], bit i & 31 of word i >> 5."""
    n = bits.shape[-1]
    bits = torch.nn.functional.pad(bits, (0, -n % 32)).unflatten(-1, (-1, 32)).long()
    w = (bits << torch.arange(32, device=bits.device)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def _bits(words, n):
    return (words[..., None] >> torch.arange(32, device=words.device, dtype=torch.int32) & 1).flatten(-2)[..., :n].bool()


def _tables(s, c, gen, tokens):
    """Page tables of sequences with these own tokens behind a shared prefix; the number of pages."""
    B, page, shared = c["B"], c["page"], _up(c["prefix"], c["page"])
    n_pages = shared + sum(_up(x, page) for x in tokens) + 3
    ids = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros((B, max(1, _up(max(tokens), page))), dtype=torch.int32)
    order, at = ids.cpu(), shared
    for b, x in enumerate(tokens):
        table[b, :_up(x, page)] = order[at:at + _up(x, page)]
        at += _up(x, page)
    s["table"], s["prefix_table"] = table.cuda(), ids[:shared].contiguous()
    return n_pages


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    turn = seed % c["B"]
    lens = _lens(c)
    lens = lens[turn:] + lens[:turn]
    s = dict(case=c)
    if "ragged" in c:
        gammas = _gammas(c)
        gammas = gammas[turn:] + gammas[:turn]
        s["gamma"] = _int32(gammas) if c["ragged"] else None
    if c["op"] in ("attend", "step"):
        n_pages = _tables(s, c, gen, [x + g + 1 for x, g in zip(lens, gammas)])
        _fill_cache(s, c, gen, n_pages)
        s["kv_len"] = _int32([c["prefix"] + x for x in lens])
        parents = _trees(c["B"], c["gamma"], seed)
        seen = _reach(parents)
    if c["op"] == "attend":
        N = c["gamma"] + 1
        s["mask"] = _words(seen).cuda()
        s["q"] = _tokens(gen, c["B"] * N, c["Hq"], c["D"], True).view(c["B"], N, c["Hq"], c["D"]).to(torch.bfloat16)
    elif c["op"] == "step":
        _prepare_step(s, c, seed, gammas, parents, seen)
    elif c["op"] == "pages":
        _prepare_pages(s, c, seed, lens)
    elif c["op"] == "fork":
        _prepare_fork(s, c, gen, seed)
    else:
        _prepare_adjust(s, c, gen, seed, lens, gammas)
    return s


def _prepare_step(s, c, seed, gammas, parents, seen):
    """Drafted tokens, and what the target drew: along the way to one node of each tree, something else behind it.
    The path's entries come from behind the places that they go to, or stay, so that a step can be made again."""
    B, N = c["B"], c["gamma"] + 1
    g = torch.Generator().manual_seed(seed + 1)
    draft = torch.randint(0, 50000, (B, N - 1), generator=g)
    target = torch.randint(50000, 50304, (B, N), generator=g)
    depth = seen.sum(-1) - 1
    node = torch.arange(N)
    inside = seen & (node > 0) & (node <= depth[..., None])  # nodes of the path that are places to move to
    stay = inside.sum(-1) == (inside & (inside.cumsum(-1) == node)).sum(-1)
    fits = stay & (node <= torch.tensor(gammas)[:, None])
    end = (torch.rand((B, N), generator=g) * fits + fits).argmax(-1)
    for b in range(B):
        path = seen[b, end[b]].nonzero()[:, 0].tolist()
        for i, j in zip(path, path[1:]):
            target[b, i] = draft[b, j - 1]
    s.update(parents=parents.int().cuda(), draft=draft.int().cuda(), target=target.int().cuda())


def _prepare_pages(s, c, seed, lens):
    """A pool whose pages are held at random by these sequences and by others."""
    g = torch.Generator().manual_seed(seed)
    held = [_up(x, c["page"]) for x in lens]
    wide = max(_up(x + c["n"], c["page"]) for x in lens)
    order = torch.randperm(c["n_pages"], generator=g).int()
    table = torch.full((c["B"], wide), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n]
        at += n
    want = sum(_up(x + c["n"], c["page"]) for x in lens) - at
    others = max(0, min((c["n_pages"] - at) // 2, c["n_pages"] - at - want))
    refs = torch.zeros(c["n_pages"], dtype=torch.int32)
    refs[order[:at + others].long()] = 1
    s.update(refs=refs.cuda(), table=table.cuda(), held=_int32(held), kv_len=_int32(lens))


def _prepare_fork(s, c, gen, seed):
    """`parents` sequences with pages of their own; the other rows of the batch are empty."""
    B, page, n = c["B"], c["page"], c["parents"]
    g = torch.Generator().manual_seed(seed)
    lens = _lens(c)[:n]
    lens = lens[seed % n:] + lens[:seed % n]
    rows = torch.randperm(B, generator=g)
    pages = [_up(x, page) for x in lens]
    n_pages = sum(pages) + B + 5
    order = torch.randperm(n_pages, generator=g).int()
    table = torch.full((B, max(pages)), -1, dtype=torch.int32)
    held, kv_len = torch.zeros(B, dtype=torch.int32), torch.full((B,), -1, dtype=torch.int32)
    at = 0
    for b, x, p in zip(rows.tolist(), lens, pages):
        table[b, :p] = order[at:at + p]
        held[b], kv_len[b] = p, x
        at += p
    refs = torch.zeros(n_pages, dtype=torch.int32)
    refs[order[:at].long()] = 1
    dst = rows[n:]
    src = rows[torch.arange(B - n) % n]
    _fill_cache(s, c, gen, n_pages)
    s.update(refs=refs.cuda(), table=table.cuda(), held=held.cuda(), kv_len=kv_len.cuda(), after=kv_len.clone().cuda(),
             src=src.int().cuda(), dst=dst.int().cuda())


def _prepare_adjust(s, c, gen, seed, lens, gammas):
    B, N, V = c["B"], c["gamma"] + 1, c["V"]
    rand = lambda *shape: torch.rand(shape, generator=gen, device="cuda")  # noqa: E731
    zipf = lambda *shape: torch.exp(rand(*shape) * math.log(V)).long().clamp(max=V - 1).int()  # noqa: E731
    s["logits"] = (torch.randn((B, N, V), generator=gen, device="cuda") * 3).to(
        torch.float32 if c["dtype"] == "f32" else torch.bfloat16)
    s["seq"], s["seq_len"] = zipf(B, max(lens) + N), _int32(lens)
    s["prompt_len"] = (rand(B) * s["seq_len"]).int()
    s["draft"] = zipf(B, N - 1)
    s["mask"] = _words(_reach(_trees(B, N - 1, seed))).cuda() if c["tree"] else None
    s["repetition"], s["presence"], s["frequency"] = 1 + 0.3 * rand(B), rand(B), 0.5 * rand(B)
    s["bias_ids"] = s["bias"] = s["allowed"] = None
    if c["bias"]:  # distinct tokens, none behind a sequence's last
        M = c["bias"]
        first = (rand(B) * V).long()
        ids = (first[:, None] + torch.arange(M, device="cuda") * 7919) % V
        keep = torch.arange(M, device="cuda") < (rand(B, 1) * (M + 1)).long()
        s["bias_ids"] = torch.where(keep, ids, torch.full_like(ids, -1)).int()
        s["bias"] = torch.where(rand(B, M) < 0.2, torch.full((B, M), -100.0, device="cuda"), 10 * rand(B, M) - 5)
    if c["grammar"]:  # half of the sequences are free, the others' nodes allow one token in eight
        w = torch.randint(-2 ** 31, 2 ** 31, (3, B, N, _up(V, 32)), generator=gen, device="cuda").int()
        w = w[0] & w[1] & w[2]
        w[::2] = -1
        s["allowed"] = w


# ------------------------------------------------------------------- run
def run(s):
    c = s["case"]
    if own:
        return _own(c, s)
    if c["op"] == "attend":
        return _plain_attend(c, s)
    if c["op"] == "step":
        return _plain_step(c, s)
    if c["op"] == "pages":
        grown = _plain_resize(s, s["kv_len"], c["n"], c["page"])
        return grown, _plain_resize(s, s["kv_len"], 0, c["page"]), s["refs"], s["table"], s["held"]
    if c["op"] == "fork":
        copies, status = _plain_fork(s, c["page"])
        for name in ("k_pages", "v_pages", "k_exp", "v_exp"):
            if s[name] is not None:
                _plain_copy(s[name], copies)
        back = _plain_resize(s, s["after"], 0, c["page"])
        return (copies, status, back, s["refs"], s["table"], s["held"], s["kv_len"]) + _held(s)
    return _plain_adjust(c, s)


def _own(c, s):
    import speculative_decoding_verify_03_gb300 as sv
    if c["op"] == "attend":
        return sv.spec_attend_tree(s["q"], s["cache"], s["table"], s["kv_len"], s["mask"], prefix_table=s["prefix_table"],
                                   prefix_len=c["prefix"], gamma_per_row=s["gamma"])
    if c["op"] == "step":
        mask, depth = sv.spec_tree_mask(s["parents"], gamma_per_row=s["gamma"])
        accepted, following, path, tokens = sv.spec_tree_accept(s["target"], s["draft"], s["parents"],
                                                                gamma_per_row=s["gamma"])
        sv.spec_kv_compact(s["cache"], s["table"], s["kv_len"], path, accepted)
        return (mask, depth, accepted, following, path, tokens) + _held(s)
    if c["op"] == "pages":
        a = sv.spec_kv_resize(s["refs"], s["table"], s["held"], s["kv_len"], c["n"], c["page"], with_status=True)
        b = sv.spec_kv_resize(s["refs"], s["table"], s["held"], s["kv_len"], 0, c["page"], with_status=True)
        return a, b, s["refs"], s["table"], s["held"]
    if c["op"] == "fork":
        copies, status = sv.spec_kv_fork(s["refs"], s["table"], s["held"], s["kv_len"], s["src"], s["dst"], c["page"],
                                         with_status=True)
        sv.spec_kv_copy(s["cache"], copies)
        back = sv.spec_kv_resize(s["refs"], s["table"], s["held"], s["after"], 0, c["page"], with_status=True)
        return (copies, status, back, s["refs"], s["table"], s["held"], s["kv_len"]) + _held(s)
    return sv.spec_adjust(s["logits"], s["seq"], s["seq_len"], draft_tokens=s["draft"], tree_mask=s["mask"],
                          prompt_len=s["prompt_len"], repetition=s["repetition"], presence=s["presence"],
                          frequency=s["frequency"], bias_ids=s["bias_ids"], bias=s["bias"], allowed=s["allowed"],
                          gamma_per_row=s["gamma"])


def _held(s):
    return tuple(s[k] for k in ("k_pages", "v_pages", "k_exp", "v_exp") if s[k] is not None)


def _gather(pages, exp, table):
    """[..., p] page ids -> float32 [..., Hkv, p * page, D]"""
    t = table.long()
    x = (pages.view(torch.uint8)[t].view(torch.float8_e4m3fn) if exp is not None else pages[t]).float()
    if exp is not None:
        x = x * _pow2(exp[t])[..., None]
    return x.movedim(-3, -4).flatten(-3, -2)


def _plain_attend(c, s):
    B, N, Hq, Hkv, D, P = c["B"], c["gamma"] + 1, c["Hq"], c["Hkv"], c["D"], c["prefix"]
    G = Hq // Hkv
    q = s["q"].float().view(B, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, D) / math.sqrt(D)
    k, v = (_gather(s[a + "_pages"], s[a + "_exp"], s["table"]) for a in "kv")
    own_len = (s["kv_len"] - P).long()
    t = torch.arange(k.shape[2], device="cuda") - own_len[:, None]  # [B, T]: node of the step, below 0: before it
    inside = (t >= 0) & (t < N)
    node = t.clamp(0, N - 1)[:, None].expand(-1, N, -1)
    sees = (t < 0)[:, None] | inside[:, None] & torch.gather(_bits(s["mask"], N), 2, node)  # [B, N, T]
    if s["gamma"] is not None:
        sees &= (torch.arange(N, device="cuda") <= s["gamma"][:, None])[:, :, None]
        sees &= (t <= s["gamma"][:, None])[:, None]
    sees = sees.repeat_interleave(G, 1)
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
        none = (torch.arange(N, device="cuda").repeat_interleave(G) > s["gamma"][:, None])[:, None]
        out, lse = out.masked_fill(none[..., None], 0), lse.masked_fill(none, -math.inf)
    back = lambda x: x.view(B, Hkv, N, G, -1).permute(0, 2, 1, 3, 4).reshape(B, N, Hq, -1)  # noqa: E731
    return back(out).to(torch.bfloat16), back(lse)[..., 0]


def _plain_step(c, s):
    B, N = c["B"], c["gamma"] + 1
    node = torch.arange(N, device="cuda")
    gamma = s["gamma"].long() if s["gamma"] is not None else torch.full((B,), N - 1, device="cuda")
    live = node <= gamma[:, None]
    up = torch.cat([torch.zeros((B, 1), dtype=torch.long, device="cuda"), s["parents"].long()], 1)
    up = torch.where(live, up, node)
    seen = torch.zeros((B, N, N), device="cuda").scatter_(2, up[..., None], 1.0)
    seen[:, node, node] = 1.0
    for _ in range(max(1, (N - 1).bit_length())):  # one link, two, four ...
        seen = (seen @ seen).clamp(max=1.0)
    seen = (seen > 0) & live[..., None]
    depth = (seen.sum(-1) - 1).clamp(min=0)
    # a node stands if it repeats what the target drew at its parent, as the first such child
    draft = torch.cat([torch.full((B, 1), -1, dtype=torch.long, device="cuda"), s["draft"].long()], 1)
    good = (draft == s["target"].long().gather(1, up)) & live & (node > 0)
    twin = (up[:, :, None] == up[:, None]) & (draft[:, :, None] == draft[:, None]) & (node > 0) & (node < node[:, None])
    good &= ~twin.any(-1)
    good[:, 0] = True
    reached = live & ~(seen & ~good[:, None]).any(-1)
    end = torch.where(reached, depth, -1).argmax(-1, keepdim=True)
    accepted = depth.gather(1, end)[:, 0]
    along = torch.gather(seen, 1, end[..., None].expand(-1, 1, N))[:, 0]
    path = torch.full((B, N + 1), -1, dtype=torch.long, device="cuda")
    path.scatter_(1, torch.where(along, depth, N), node.expand(B, N))
    path = path[:, :N]
    tokens = torch.where(path[:, 1:] >= 0, draft.gather(1, path[:, 1:].clamp(min=0)), -1)
    following = s["target"].gather(1, end)[:, 0]
    to = s["kv_len"][:, None].long() + node
    origin = s["kv_len"][:, None].long() + path
    move = (path > node) & (node > 0)
    b = torch.arange(B, device="cuda")[:, None].expand(B, N)[move]
    to, origin = to[move], origin[move]
    table = s["table"].long()
    for x in _held(s):
        x = x.view(torch.uint8) if x.element_size() == 1 else x
        x[table[b, to // c["page"]], :, to % c["page"]] = x[table[b, origin // c["page"]], :, origin % c["page"]]
    return (_words(seen), depth.int(), accepted.int(), following, path.int(), tokens.int()) + _held(s)


def _take(refs, need):
    """The lowest free pages for rows that need so many each, in order: (page of each rank, first rank of each row,
    which rows are served)."""
    free = refs <= 0
    rank = free.cumsum(0) - 1
    pages = torch.zeros(len(refs) + 1, dtype=torch.long, device="cuda")
    pages[torch.where(free, rank, len(refs))] = torch.arange(len(refs), device="cuda")
    last = need.cumsum(0)
    return pages, last - need, last <= free.sum()


def _plain_resize(s, kv_len, n, page):
    refs, table, held = s["refs"], s["table"], s["held"]
    B, wide = table.shape
    want = torch.where(kv_len >= 0, (kv_len.long() + n + page - 1) // page, 0)
    at = torch.arange(wide, device="cuda")
    gone = (at >= want[:, None]) & (at < held[:, None])
    refs.index_add_(0, table.clamp(min=0).flatten().long(), -gone.flatten().int())
    need = (want - held).clamp(min=0)
    pages, first, served = _take(refs, need)
    served &= need > 0
    new = (at < want[:, None]) & (at >= held[:, None]) & served[:, None]
    ids = pages[torch.where(new, first[:, None] + at - held[:, None], 0)]
    table.copy_(torch.where(new, ids, table))
    refs.index_add_(0, torch.where(new, ids, 0).flatten(), torch.where(new, 1 - refs[ids], 0).flatten())
    short = (need > 0) & ~served
    held.copy_(torch.where(short, held, want))
    return torch.where(short, NO_PAGES, 0).int()


def _plain_fork(s, page):
    refs, table, held, kv_len = s["refs"], s["table"], s["held"], s["kv_len"]
    src, dst = s["src"].long(), s["dst"].long()
    tokens = kv_len[src].long()
    full, part = tokens // page, tokens % page
    need = (part > 0).long()
    pages, first, served = _take(refs, need)
    at = torch.arange(table.shape[1], device="cuda")
    shared = (at < full[:, None]) & served[:, None]
    old = table[src]
    new = pages[torch.where(served, first, 0)]
    mine = torch.where((at == full[:, None]) & ((need > 0) & served)[:, None], new[:, None].int(), table[dst])
    table[dst] = torch.where(shared, old, mine)
    refs.index_add_(0, old.clamp(min=0).flatten().long(), shared.flatten().int())
    put = (need > 0) & served
    refs.index_add_(0, torch.where(put, new, 0), torch.where(put, 1 - refs[new], 0))
    held[dst] = torch.where(served, full + need, held[dst]).int()
    kv_len[dst] = torch.where(served, kv_len[src], kv_len[dst])
    origin = old.gather(1, full.clamp(max=table.shape[1] - 1)[:, None])[:, 0].long()
    copies = torch.stack([origin, new, part], 1)
    copies = torch.where(put[:, None], copies, torch.tensor([-1, -1, 0], device="cuda"))
    return copies.int(), torch.where(served, 0, NO_PAGES).int()


def _plain_copy(x, copies):
    """Slots 0 .. n - 1 of page src to page dst, for rows (src, dst, n) of copies."""
    x = x.view(torch.uint8) if x.element_size() == 1 else x
    src, dst, n = copies.long().unbind(1)
    slot = torch.arange(x.shape[2], device="cuda")
    i, at = ((src >= 0)[:, None] & (slot < n[:, None])).nonzero(as_tuple=True)
    x[dst[i], :, at] = x[src[i], :, at]


def _plain_adjust(c, s):
    B, N, V = c["B"], c["gamma"] + 1, c["V"]
    out = torch.empty_like(s["logits"])
    at = torch.arange(s["seq"].shape[1], device="cuda")
    ids = s["seq"].long()
    one = lambda there: there.float()  # noqa: E731
    seen = torch.zeros((B, V), device="cuda").scatter_add_(1, ids, one(at < s["seq_len"][:, None]))
    made = torch.zeros((B, V), device="cuda").scatter_add_(
        1, ids, one((at < s["seq_len"][:, None]) & (at >= s["prompt_len"][:, None])))
    drafts = s["draft"].long()
    node = torch.arange(1, N, device="cuda")
    bias = None
    if s["bias_ids"] is not None:
        bias = torch.zeros((B, V + 1), device="cuda")
        bias = bias.scatter_(1, torch.where(s["bias_ids"] >= 0, s["bias_ids"], V).long(), s["bias"])[:, :V]
    r, f, p = s["repetition"][:, None], s["frequency"][:, None], s["presence"][:, None]
    for i in range(N):
        z = s["logits"][:, i].float()
        path = _bits(s["mask"][:, i], N)[:, 1:] if s["mask"] is not None else (node <= i).expand(B, -1)
        if s["gamma"] is not None:
            path = path & (node <= s["gamma"][:, None])
        count = made.scatter_add(1, drafts, one(path)) if N > 1 else made
        y = torch.where((seen > 0) | (count > 0), torch.where(z > 0, z / r, z * r), z)
        y = y - f * count - p * (count > 0)
        if bias is not None:
            y = y + bias
        if s["allowed"] is not None:
            y = y.masked_fill(~_bits(s["allowed"][:, i], V), -math.inf)
        if s["gamma"] is not None:  # positions behind a sequence's last are as they were
            y = torch.where((i <= s["gamma"])[:, None], y, z)
        out[:, i] = y.to(out.dtype)
    return out


# ----------------------------------------------------------------- exact
def exact(case, seed):
    """From the definitions: sequence by sequence, lists for the tables, float64 for what is computed."""
    c, s = case, prepare(case, seed)
    return {"attend": _exact_attend, "step": _exact_step, "pages": _exact_pages, "fork": _exact_fork,
            "adjust": _exact_adjust}[c["op"]](c, s)


def _two_to(e):
    """2.0 ** e in float64, exactly (a power function may be off by a unit in the last place)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


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


def _rows_of(c, table_row, n):
    p = torch.arange(n, device="cuda")
    return table_row.long()[p // c["page"]], p % c["page"]


def _exact_attend(c, s):
    B, N, Hq, Hkv, D, P = c["B"], c["gamma"] + 1, c["Hq"], c["Hkv"], c["D"], c["prefix"]
    G = Hq // Hkv
    out = torch.zeros((B, N, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, N, Hq), -math.inf, dtype=torch.float64, device="cuda")
    lens = s["kv_len"].tolist()
    gam = s["gamma"].tolist() if s["gamma"] is not None else [c["gamma"]] * B
    words = s["mask"].cpu().tolist()
    for b in range(B):
        n, before = gam[b] + 1, lens[b] - P
        k, v = (_value(s, a, _rows_of(c, s["table"][b], before + n)) for a in "kv")
        if P:
            k, v = (torch.cat([_value(s, a, _rows_of(c, s["prefix_table"], P)), x]) for a, x in (("k", k), ("v", v)))
        sees = [[bool(words[b][i][j // 32] >> (j % 32) & 1) for j in range(n)] for i in range(n)]
        sees = torch.cat([torch.ones((n, P + before), dtype=torch.bool), torch.tensor(sees)], 1).cuda()
        z = torch.einsum("nhgd,thd->hgnt", s["q"][b, :n].double().view(n, Hkv, G, D), k) / math.sqrt(D)
        z = torch.where(sees, z, torch.full_like(z, -math.inf))
        lse[b, :n] = torch.logsumexp(z, -1).permute(2, 0, 1).reshape(n, Hq)
        out[b, :n] = torch.einsum("hgnt,thd->nhgd", torch.softmax(z, -1), v).reshape(n, Hq, D)
    return out, lse


def _exact_step(c, s):
    B, N = c["B"], c["gamma"] + 1
    gam = s["gamma"].tolist() if s["gamma"] is not None else [c["gamma"]] * B
    parents, draft, target = (s[k].tolist() for k in ("parents", "draft", "target"))
    bits = torch.zeros((B, N, N), dtype=torch.bool)
    depth = torch.zeros((B, N), dtype=torch.int32)
    accepted, following = [], []
    path, tokens = torch.full((B, N), -1, dtype=torch.int32), torch.full((B, N - 1), -1, dtype=torch.int32)
    held = [x.double() if x.dtype != torch.int8 else x.clone() for x in _held(s)]
    table, lens, page = s["table"].tolist(), s["kv_len"].tolist(), c["page"]
    for b in range(B):
        for i in range(gam[b] + 1):
            j = i
            bits[b, i, j] = True
            while j > 0:
                j = parents[b][j - 1]
                bits[b, i, j] = True
                depth[b, i] += 1
        at, way = 0, [0]
        while True:
            child = [j for j in range(1, gam[b] + 1) if parents[b][j - 1] == at and draft[b][j - 1] == target[b][at]]
            if not child:
                break
            at = child[0]
            way.append(at)
        accepted.append(len(way) - 1)
        following.append(target[b][at])
        path[b, :len(way)] = torch.tensor(way)
        for d, j in enumerate(way[1:]):
            tokens[b, d] = draft[b][j - 1]
        for d, j in enumerate(way):
            to, origin = lens[b] + d, lens[b] + j
            if to != origin:
                for x in held:
                    x[table[b][to // page], :, to % page] = x[table[b][origin // page], :, origin % page]
    return (_words(bits).cuda(), depth.cuda(), _int32(accepted), _int32(following), path.cuda(), tokens.cuda(), *held)


class _Lists:
    """The pool as lists."""

    def __init__(self, s):
        self.refs, self.table, self.held = (s[k].tolist() for k in ("refs", "table", "held"))

    def free(self):
        return [i for i, r in enumerate(self.refs) if r <= 0]

    def resize(self, kv_len, n, page):
        want = [-(-(x + n) // page) if x >= 0 else 0 for x in kv_len]
        for b, w in enumerate(want):
            for i in range(w, self.held[b]):
                self.refs[self.table[b][i]] -= 1
        free, at, status = self.free(), 0, []
        for b, w in enumerate(want):
            need = max(0, w - self.held[b])
            at += need
            status.append(NO_PAGES if need and at > len(free) else 0)
            if status[-1]:
                continue
            for i in range(need):
                self.table[b][self.held[b] + i] = free[at - need + i]
                self.refs[free[at - need + i]] = 1
            self.held[b] = w
        return _int32(status)

    def tensors(self):
        return _int32(self.refs), _int32(self.table), _int32(self.held)


def _exact_pages(c, s):
    pool, lens = _Lists(s), s["kv_len"].tolist()
    a = pool.resize(lens, c["n"], c["page"])
    return (a, pool.resize(lens, 0, c["page"])) + pool.tensors()


def _exact_fork(c, s):
    pool, lens, page = _Lists(s), s["kv_len"].tolist(), c["page"]
    after = list(lens)
    held = [x.double() if x.dtype != torch.int8 else x.clone() for x in _held(s)]
    free, copies, status = pool.free(), [], []
    for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
        full, part = divmod(lens[a], page)
        status.append(NO_PAGES if part and not free else 0)
        if status[-1]:
            copies.append([-1, -1, 0])
            continue
        for i in range(full):
            pool.table[b][i] = pool.table[a][i]
            pool.refs[pool.table[a][i]] += 1
        copies.append([-1, -1, 0])
        if part:
            new = free.pop(0)
            pool.table[b][full] = new
            pool.refs[new] = 1
            copies[-1] = [pool.table[a][full], new, part]
            for x in held:
                x[new, :, :part] = x[pool.table[a][full], :, :part]
        pool.held[b], lens[b] = full + (part > 0), lens[a]
    back = pool.resize(after, 0, page)
    return (_int32(copies), _int32(status), back) + pool.tensors() + (_int32(lens),) + tuple(held)


def _exact_adjust(c, s):
    B, N, V = c["B"], c["gamma"] + 1, c["V"]
    out = s["logits"].double()
    gam = s["gamma"].tolist() if s["gamma"] is not None else [c["gamma"]] * B
    lens, prompts = s["seq_len"].tolist(), s["prompt_len"].tolist()
    words = s["mask"].cpu().tolist() if s["mask"] is not None else None
    r, f, p = (s[k].double().tolist() for k in ("repetition", "frequency", "presence"))
    for b in range(B):
        seq = s["seq"][b, :lens[b]].long()
        prompt = torch.bincount(seq[:prompts[b]], minlength=V)
        made = torch.bincount(seq[prompts[b]:], minlength=V)
        for i in range(gam[b] + 1):
            path = [j for j in range(1, gam[b] + 1) if (words[b][i][j // 32] >> (j % 32) & 1 if words else j <= i)]
            count = made + torch.bincount(s["draft"][b].long()[torch.tensor(path, dtype=torch.long, device="cuda") - 1],
                                          minlength=V)
            z = out[b, i]
            hit = (count + prompt) > 0
            z[hit & (z > 0)] /= r[b]
            z[hit & (s["logits"][b, i] <= 0)] *= r[b]
            z -= f[b] * count.double()
            z[count > 0] -= p[b]
            if s["bias_ids"] is not None:
                there = s["bias_ids"][b] >= 0
                z[s["bias_ids"][b][there].long()] += s["bias"][b][there].double()
            if s["allowed"] is not None:
                word = s["allowed"][b, i][torch.arange(V, device="cuda") // 32]
                z[(word >> (torch.arange(V, device="cuda") % 32).int() & 1) == 0] = -math.inf
    return out
