"""Trees of drafted tokens on the GPU against their definitions (tree_ref.py):
masks and the accepting walk exactly, the attention within the tolerance that
test_gpu_kv.py derives."""
import numpy as np
import pytest

import kv_ref
import tree_ref
from test_gpu_kv import bf16, check_attend, i32, make_cache, put, sv, tables  # noqa: F401

pytestmark = pytest.mark.gpu


def np_of(t):
    return t.cpu().numpy()


# ------------------------------------------------------------- masks and walk
SHAPES = [(1, 0), (3, 1), (2, 25), (5, 31), (4, 32), (130, 7), (2, 63), (3, 100), (1, 300), (2, 511)]


@pytest.mark.parametrize("B,G", SHAPES)
@pytest.mark.parametrize("shape", ["random", "chain", "star"])
@pytest.mark.parametrize("ragged", [False, True])
def test_mask(sv, B, G, shape, ragged):  # noqa: F811
    rng = np.random.default_rng(B * 1000 + G)
    p = tree_ref.random_parents(rng, B, G)
    if shape == "chain":
        p[:] = np.arange(G)
    if shape == "star":
        p[:] = 0
    g = rng.integers(0, G + 1, B) if ragged else np.full(B, G)
    mask, depth, st = sv.spec_tree_mask(i32(p), i32(g) if ragged else None, with_status=True)
    bits, want = tree_ref.sees(p, g)
    assert (np_of(st) == 0).all()
    assert np.array_equal(np_of(depth), want)
    assert np.array_equal(np_of(mask), tree_ref.words(bits))


def test_mask_errors(sv):  # noqa: F811
    """A bad parent or gamma empties its own row alone; a bad parent past gamma_b is not looked at."""
    rng = np.random.default_rng(1)
    p = tree_ref.random_parents(rng, 6, 40)
    g = np.array([40, 40, 41, -1, 40, 20])
    p[0, 10] = 11  # node 11 its own parent
    p[1, 39] = -1
    p[4, 0] = 1
    p[5, 30] = 1000
    mask, depth, st = sv.spec_tree_mask(i32(p), i32(g), with_status=True)
    bad = [tree_ref.BAD_TREE, tree_ref.BAD_TREE, tree_ref.BAD_GAMMA, tree_ref.BAD_GAMMA, tree_ref.BAD_TREE, 0]
    assert list(np_of(st)) == bad
    assert (np_of(mask)[:5] == 0).all() and (np_of(depth)[:5] == 0).all()
    bits, want = tree_ref.sees(p[5:], g[5:])
    assert np.array_equal(np_of(mask)[5:], tree_ref.words(bits)) and np.array_equal(np_of(depth)[5:], want)


@pytest.mark.parametrize("B,G", SHAPES)
@pytest.mark.parametrize("vocab", [2, 5])
@pytest.mark.parametrize("ragged", [False, True])
def test_accept(sv, B, G, vocab, ragged):  # noqa: F811
    """Few token ids: long ways, and drafts that are alike under one parent."""
    rng = np.random.default_rng(B + G + vocab)
    p = tree_ref.random_parents(rng, B, G, 0.3)
    draft, target = rng.integers(0, vocab, (B, G)), rng.integers(0, vocab, (B, G + 1))
    g = rng.integers(0, G + 1, B) if ragged else np.full(B, G)
    acc, nxt, path, tok, st = sv.spec_tree_accept(i32(target), i32(draft), i32(p), i32(g) if ragged else None,
                                                  with_status=True)
    assert (np_of(st) == 0).all()
    for b in range(B):
        a, t, way = tree_ref.accept(target[b], draft[b], p[b], int(g[b]))
        assert (int(acc[b]), int(nxt[b])) == (a, t)
        assert list(np_of(path)[b]) == way + [-1] * (G + 1 - len(way))
        assert list(np_of(tok)[b]) == [draft[b, j - 1] for j in way[1:]] + [-1] * (G - a)


def test_accept_a_chain_to_its_end(sv):  # noqa: F811
    G = 511
    acc, nxt, path, tok = sv.spec_tree_accept(i32(np.full((1, G + 1), 3)), i32(np.full((1, G), 3)), i32(np.arange(G)[None]))
    assert int(acc) == G and int(nxt) == 3 and np.array_equal(np_of(path)[0], np.arange(G + 1)) and (np_of(tok) == 3).all()


def test_accept_errors(sv):  # noqa: F811
    """Errors of a row: bad gamma, bad tree, a negative token at a visited node
    (elsewhere it does not matter)."""
    p = np.tile(np.array([0, 0, 1]), (6, 1))
    draft, target = np.tile([5, 6, 7], (6, 1)), np.tile([5, 7, 9, 8], (6, 1))
    p[1, 1] = 2
    target[2, 1] = -1   # visited behind node 0
    target[3, 2] = -1   # node 2 is not
    target[5, 0] = -1
    g = [3, 3, 3, 3, 4, 3]
    acc, nxt, path, tok, st = (np_of(x) for x in sv.spec_tree_accept(i32(target), i32(draft), i32(p), i32(g), with_status=True))
    assert list(st) == [0, tree_ref.BAD_TREE, tree_ref.BAD_TOKEN, 0, tree_ref.BAD_GAMMA, tree_ref.BAD_TOKEN]
    assert list(acc) == [2, 0, 0, 2, 0, 0] and list(nxt) == [8, -1, -1, 8, -1, -1]
    for b in range(6):
        assert list(path[b]) == ([0, 1, 3, -1] if b in (0, 3) else [-1] * 4)
        assert list(tok[b]) == ([5, 7, -1] if b in (0, 3) else [-1] * 3)


# ------------------------------------------------------------------ attention
def tree_case(sv, seed, fmt, B, N, Hq, Hkv, D, S, prefix, lens, gammas=None, q_scale=1.0, bits=None, parents=None):  # noqa: F811
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens)
    mp = max(1, -(-(int(lens.max()) + N) // S))
    n, table, pt = tables(rng, B, mp, -(-prefix // S))
    cache, k, v, ke, ve = make_cache(sv, rng, fmt, n, Hkv, S, D)
    q = kv_ref.bf16_bits((rng.standard_normal((B, N, Hq, D)) * q_scale).astype(np.float32))
    g = np.full(B, N - 1) if gammas is None else np.asarray(gammas)
    if bits is None:
        p = tree_ref.random_parents(rng, B, N - 1) if parents is None else parents
        bits = tree_ref.sees(p, np.full(B, N - 1))[0]
    return dict(cache=cache, k=k, v=v, ke=ke, ve=ve, table=table, pt=pt, q=q, lens=lens + prefix, prefix=prefix, S=S,
                N=N, D=D, g=g, ragged=gammas is not None, bits=bits)


def call(sv, s, **kw):  # noqa: F811
    kw = dict(dict(with_status=True, gamma_per_row=i32(s["g"]) if s["ragged"] else None), **kw)
    return sv.spec_attend_tree(bf16(s["q"]), s["cache"], i32(s["table"]), i32(s["lens"]), i32(tree_ref.words(s["bits"])),
                               prefix_table=i32(s["pt"]), prefix_len=s["prefix"], **kw)


def reference(s):
    return tree_ref.attend(kv_ref.bf16_value(s["q"]), kv_ref.cache_value(s["k"], s["ke"]),
                           kv_ref.cache_value(s["v"], s["ve"]), s["table"], s["lens"], s["pt"], s["prefix"], s["g"],
                           s["S"], s["D"] ** -0.5, s["bits"])


def check(sv, s, fmt):  # noqa: F811
    """Beside check_attend's terms, over an e4m3 cache: the weights times 2^e (e the
    exponent of the token's values) are float16 numbers, the row's largest at 2^8 or
    above, spaced 2^-24 at least, so each is off by half of that, 2^-33 of the
    largest at most; the largest is at most 2^-7 here (the exponents of make_cache),
    and a stored value at most 448: 2^-33 3.5 for every token."""
    got, ref = call(sv, s), reference(s)
    least = (int(s["lens"].max()) + s["N"]) * 2.0 ** -33 * 3.5 if fmt == "e4m3" else 0.0
    assert (np_of(got[2]) == 0).all()
    # queries that see nothing have -inf on both sides; a difference of those says nothing
    none = np.isneginf(ref[1]) & (np.arange(s["N"]) <= s["g"][:, None])[:, :, None]
    lse = got[1].clone()
    assert np.isneginf(np_of(lse)[none]).all() and (np_of(got[0].float())[none] == 0).all()
    lse[i32(none).bool()] = 0
    check_attend((got[0], lse), (ref[0], np.where(none, 0, ref[1])) + ref[2:], fmt, s["g"], least=least)
    return got


CASES = [  # B, N, Hq, Hkv, D, S, prefix, own lengths
    (1, 1, 2, 1, 64, 16, 0, [0]),             # the root alone
    (1, 26, 8, 1, 128, 16, 0, [700]),         # 208 rows of one head
    (2, 5, 4, 4, 80, 16, 0, [0, 63]),         # the step across a tile's end
    (3, 8, 6, 2, 96, 32, 1, [0, 64, 130]),
    (2, 33, 14, 2, 128, 64, 65, [1, 62]),     # masks of two words
    (2, 64, 4, 2, 64, 128, 200, [5, 100]),    # 128 rows
    (5, 4, 12, 1, 128, 16, 48, [3, 0, 80, 17, 200]),
    (9, 3, 7, 7, 64, 16, 333, [0, 1, 2, 3, 16, 31, 33, 60, 64]),
    (2, 100, 6, 2, 80, 32, 10, [0, 150]),     # 300 rows, an odd part of the last tile
    (1, 150, 4, 1, 96, 64, 0, [500]),         # 600 rows
    (3, 65, 2, 1, 128, 16, 0, [127, 128, 1]),  # 130 rows: two past a tile of 128
    (1, 512, 1, 1, 64, 64, 0, [70]),          # the largest tree
]


@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=[f"B{c[0]}N{c[1]}q{c[2]}k{c[3]}D{c[4]}S{c[5]}p{c[6]}" for c in CASES])
def test_attend_tree(sv, fmt, case):  # noqa: F811
    check(sv, tree_case(sv, 60, fmt, *case), fmt)


@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
@pytest.mark.parametrize("N,Hq,Hkv,prefix", [(9, 4, 2, 0), (40, 8, 1, 150), (70, 4, 2, 33)])
def test_attend_tree_ragged(sv, fmt, N, Hq, Hkv, prefix):  # noqa: F811
    """Nodes past gamma_b give 0 and -inf, and what stands in their masks and places is not read."""
    B = 7
    g = [0, N - 1, 3, 1, N // 2, 5, N - 2]
    s = tree_case(sv, 61, fmt, B, N, Hq, Hkv, 64, 16, prefix, [0, 40, 300, 7, 128, 255, 13], gammas=g)
    for b in range(B):
        s["bits"][b, g[b] + 1:] = True
        s["bits"][b, :, g[b] + 1:] = True
    check(sv, s, fmt)


@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
@pytest.mark.parametrize("Hq", [2, 16])
@pytest.mark.parametrize("lens", [(0, 0, 5), (0, 130, 64)])
def test_attend_tree_any_mask(sv, fmt, Hq, lens):  # noqa: F811
    """Masks that are no tree's: rows that see nothing of the step (and, without
    tokens before it, nothing at all), later nodes, all nodes."""
    rng = np.random.default_rng(3)
    N = 37
    bits = rng.random((3, N, N)) < 0.3
    bits[:, ::5] = False
    bits[:, 1::7] = True
    s = tree_case(sv, 62, fmt, 3, N, Hq, 1, 128, 32, 0, lens, bits=bits)
    out, lse, _ = check(sv, s, fmt)
    none = ~bits[0].any(-1)
    assert none.sum() == 7 and np.isneginf(np_of(lse)[0][none]).all() and (np_of(out.float())[0][none] == 0).all()


@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
@pytest.mark.parametrize("q_scale", [0.0, 1e-30, 40.0, 1e6])
def test_attend_tree_query_sizes(sv, fmt, q_scale):  # noqa: F811
    check(sv, tree_case(sv, 63, fmt, 2, 30, 8, 2, 64, 16, 0, [200, 31], q_scale=q_scale), fmt)


@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
@pytest.mark.parametrize("N,Hq", [(4, 4), (40, 8)])
def test_attend_tree_of_a_chain_is_attend(sv, fmt, N, Hq):  # noqa: F811
    s = tree_case(sv, 64, fmt, 3, N, Hq, 2, 128, 16, 70, [20, 300, 5], parents=np.tile(np.arange(N - 1), (3, 1)))
    got = sv.spec_attend(bf16(s["q"]), s["cache"], i32(s["table"]), i32(s["lens"]), prefix_table=i32(s["pt"]),
                         prefix_len=70, with_status=True)
    ref = reference(s)
    check_attend(got, ref, fmt, s["g"])
    check_attend(call(sv, s), ref, fmt, s["g"])


MANY = [(40, 20, 16, 2, 64, 16, 0, None), (12, 64, 8, 2, 128, 64, 0, None), (30, 12, 32, 8, 96, 32, 100, None),
        (64, 33, 4, 1, 80, 128, 40, None)]


@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
@pytest.mark.parametrize("case", MANY, ids=[f"B{c[0]}N{c[1]}q{c[2]}k{c[3]}D{c[4]}" for c in MANY])
def test_attend_tree_many_items(sv, fmt, case):  # noqa: F811
    """More items than CTAs, empty sequences among them."""
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 400, case[0])
    lens[::6] = 0
    g = rng.integers(0, case[1], case[0])
    check(sv, tree_case(sv, 65, fmt, *case[:7], lens, gammas=g), fmt)


@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
@pytest.mark.parametrize("N,Hq", [(8, 8), (40, 8)])
@pytest.mark.parametrize("which", ["k", "v"])
def test_attend_tree_nan_stays_where_it_is_seen(sv, fmt, which, N, Hq):  # noqa: F811
    """A NaN in a node's entry reaches those nodes alone that see it; an infinity
    of a value (bfloat16) makes their outputs infinite."""
    s = tree_case(sv, 66, fmt, 3, N, Hq, 2, 64, 16, 37, [20, 63, 125])
    want = reference(s)
    spots = {0: (2, 1, 7), 1: (N - 1, 0, 63), 2: (1, 1, 0)}  # sequence: node, head, element
    for b, (t, h, d) in spots.items():
        p = s["lens"][b] - s["prefix"] + t
        code = 0x7F if fmt == "e4m3" else (0xFF80 if which == "v" and b == 1 else 0x7FC0)
        put(s, which, s["table"][b, p // s["S"]], h, p % s["S"], d, code)
    out, lse, st = (x.float().cpu().numpy() for x in call(sv, s))
    for b, (t, h, d) in spots.items():
        heads = slice(Hq // 2 * h, Hq // 2 * (h + 1))
        hit = np.zeros(out[b].shape, bool)
        hit[np.nonzero(s["bits"][b, :, t])[0], heads, d if which == "v" else slice(None)] = True
        if fmt == "bf16" and which == "v" and b == 1:
            assert np.isneginf(out[b][hit]).all()
        else:
            assert np.isnan(out[b][hit]).all()
        assert np.isfinite(out[b][~hit]).all()
        assert np.abs(out[b] - want[0][b])[~hit].max() < 0.05 * (1 + np.abs(want[0][b]).max())
        assert np.isnan(lse[b, s["bits"][b, :, t], heads]).all() == (which == "k")
        assert np.isfinite(lse[b, ~s["bits"][b, :, t]]).all()
    assert (st == 0).all()


@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
@pytest.mark.parametrize("N,Hq", [(6, 4), (40, 8)])
def test_attend_tree_garbage_past_the_end(sv, fmt, N, Hq):  # noqa: F811
    """NaN and infinities in slots that hold no token, exponents included."""
    g = [N - 1, 2, N - 2]
    s = tree_case(sv, 67, fmt, 3, N, Hq, 2, 128, 16, 0, [20, 63, 5], gammas=g)
    want = reference(s)
    for b, n in enumerate(s["lens"]):
        for p in range(n + g[b] + 1, s["table"].shape[1] * s["S"]):
            pg, sl = s["table"][b, p // s["S"]], p % s["S"]
            for w in "kv":
                for h in range(2):
                    put(s, w, pg, h, sl, slice(None), 0x7F if fmt == "e4m3" else 0x7F80 if sl % 2 else 0x7FC1)
                    if fmt == "e4m3":
                        getattr(s["cache"], w + "_exp")[pg, h, sl] = -128 if sl % 2 else 127
    check_attend(call(sv, s), want, fmt, s["g"])


@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
@pytest.mark.parametrize("N,Hq", [(4, 4), (40, 8)])
def test_attend_tree_error_rows(sv, fmt, N, Hq):  # noqa: F811
    import torch
    g = np.array([N - 1] * 6)
    s = tree_case(sv, 68, fmt, 6, N, Hq, 2, 64, 16, 37, [20, 63, 5, 9, 30, 12], gammas=g)
    want = reference(s)
    s["table"][1, 2] = -7
    s["g"] = g.copy()
    s["g"][2] = N
    s["lens"][4] = s["prefix"] - 1
    got = call(sv, s)
    assert list(np_of(got[2])) == [0, sv.ROW_BAD_PAGE, 16, 0, sv.ROW_BAD_LENGTH, 0]
    for b in (1, 2, 4):
        assert torch.isnan(got[0][b]).all() and torch.isnan(got[1][b]).all()
    good = [0, 3, 5]
    check_attend([x[good] for x in got[:2]], [x[good] for x in want], fmt, g[good])


@pytest.mark.parametrize("off", [0, 1, 8])
@pytest.mark.parametrize("N,Hq", [(6, 4), (40, 8)])
def test_attend_tree_query_strides(sv, off, N, Hq):  # noqa: F811
    import torch
    s = tree_case(sv, 69, "e4m3", 3, N, Hq, 2, 64, 16, 37, [20, 63, 5])
    want = call(sv, s)
    big = torch.zeros((3, N, Hq + 3, 64 + off), dtype=torch.bfloat16, device="cuda")
    view = big[:, :, 1:1 + Hq, off:] if off else big[:, :, 1:1 + Hq]
    view.copy_(bf16(s["q"]))
    got = sv.spec_attend_tree(view, s["cache"], i32(s["table"]), i32(s["lens"]), i32(tree_ref.words(s["bits"])),
                              prefix_table=i32(s["pt"]), prefix_len=37)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_attend_tree_in_a_graph_and_on_a_stream(sv):  # noqa: F811
    """Captured with the workspace left to the call, replayed with new lengths,
    masks and queries; and bitwise the same on another stream, into given tensors."""
    import torch
    s = tree_case(sv, 70, "e4m3", 3, 40, 8, 2, 128, 16, 64, [20, 300, 5])
    q, table, lens, pt, mask = bf16(s["q"]), i32(s["table"]), i32(s["lens"]), i32(s["pt"]), i32(tree_ref.words(s["bits"]))
    kw = dict(prefix_table=pt, prefix_len=64)
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    sv.spec_attend_tree(q, s["cache"], table, lens, mask, **kw)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            out = sv.spec_attend_tree(q, s["cache"], table, lens, mask, **kw)
    for step in range(3):
        lens.copy_(i32(64 + np.array([3 * step, 290 - step, 9])))
        q.mul_(-0.5)
        mask[:, 3] ^= 2
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = sv.spec_attend_tree(q, s["cache"], table, lens, mask, **kw)
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
        into = (torch.empty_like(want[0]), torch.empty_like(want[1]))
        side.wait_stream(torch.cuda.current_stream())
        ws = torch.empty(sv.attend_tree_workspace_bytes(s["cache"], sv.SpecKvBatch(B=3, gamma_max=39, max_pages=table.shape[1],
                         prefix_len=64), 8), dtype=torch.uint8, device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        got = sv.spec_attend_tree(q, s["cache"], table, lens, mask, out=into, workspace=ws, stream=side, **kw)
        side.synchronize()
        assert got[0] is into[0] and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_attend_tree_workspaces_and_outputs_are_checked(sv):  # noqa: F811
    import torch
    s = tree_case(sv, 71, "bf16", 2, 5, 4, 2, 64, 16, 0, [20, 3])
    want = call(sv, s)
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    for bad, error in ((dict(workspace=None), ValueError), (dict(workspace="mine"), ValueError), (dict(workspace=small), sv.SpecError),
                       (dict(workspace=small.cpu()), ValueError), (dict(out=want[0]), TypeError),
                       (dict(out=(want[0], want[0])), ValueError), (dict(out=(want[0].float(), want[1])), ValueError),
                       (dict(scale=float("nan")), sv.SpecError), (dict(scale=-1.0), sv.SpecError)):
        with pytest.raises(error):
            call(sv, s, **bad)
    size = sv.attend_tree_workspace_bytes(s["cache"], sv.SpecKvBatch(B=2, gamma_max=4, max_pages=s["table"].shape[1]), 4)
    for ws in (torch.empty(size, dtype=torch.uint8, device="cuda"), torch.empty(size // 4, dtype=torch.int32, device="cuda")):
        got = call(sv, s, workspace=ws, out=(torch.empty_like(want[0]), torch.empty_like(want[1])))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(call(sv, s, scale=0.125)[0], want[0])  # 64 ** -0.5


@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
@pytest.mark.parametrize("case", [(64, 16, 32, 4, 80, 16, 0), (120, 16, 32, 8, 64, 16, 0), (64, 5, 32, 8, 128, 32, 500),
                                  (30, 9, 32, 8, 96, 64, 0)], ids=str)
def test_attend_tree_many_rows(sv, fmt, case):  # noqa: F811
    """Several rows of a warp in the merge: with as many partial results as most rows
    have, with many (one sequence is long), of sequences with an error, past gamma_b."""
    import torch
    B, N = case[:2]
    rng = np.random.default_rng(6)
    lens = rng.integers(0, 60, B)
    lens[2] = 2500
    g = rng.integers(0, N, B)
    s = tree_case(sv, 72, fmt, *case, lens, gammas=g)
    want = reference(s)
    least = (int(s["lens"].max()) + N) * 2.0 ** -33 * 3.5 if fmt == "e4m3" else 0.0  # as in check
    s["g"] = g.copy()
    s["g"][3] = N
    s["table"][7, 0] = 1 << 30
    s["lens"][7] = s["prefix"] + 5
    got = call(sv, s)
    status = np_of(got[2])
    assert status[3] == 16 and status[7] == sv.ROW_BAD_PAGE and (np.delete(status, [3, 7]) == 0).all()
    for b in (3, 7):
        assert torch.isnan(got[0][b]).all() and torch.isnan(got[1][b]).all()
    good = np.delete(np.arange(B), [3, 7])
    check_attend([x[i32(good).long()] for x in got[:2]], [x[good] for x in want], fmt, g[good], least=least)


@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
@pytest.mark.parametrize("B,N,Hq,Hkv,D,prefix", [(200, 4, 16, 16, 64, 0), (60, 40, 16, 4, 64, 20), (41, 70, 8, 8, 80, 0),
                                                 (50, 17, 32, 4, 128, 0), (2, 300, 64, 32, 64, 0)])
def test_attend_tree_items_of_few_tiles(sv, fmt, B, N, Hq, Hkv, D, prefix):  # noqa: F811
    """More tiles than CTAs, of items that hold one or two: where items count for more
    than their tiles some CTAs have nothing to do.  One long sequence, empty ones."""
    rng = np.random.default_rng(8)
    lens = rng.integers(0, 40, B)
    lens[B // 2], lens[::9] = 1500, 0
    g = rng.integers(0, N, B)
    g[0], g[-1] = N - 1, 0
    check(sv, tree_case(sv, 73, fmt, B, N, Hq, Hkv, D, 16, prefix, lens, gammas=g), fmt)


def test_attend_tree_into_a_list(sv):  # noqa: F811
    """The pair of results may be a list, as spec_attend takes it."""
    import torch
    s = tree_case(sv, 74, "bf16", 2, 5, 4, 2, 64, 16, 0, [20, 3])
    want = call(sv, s)
    into = [torch.empty_like(want[0]), torch.empty_like(want[1])]
    got = call(sv, s, out=into)
    assert got[0] is into[0] and got[1] is into[1] and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for bad in (into[:1], into + into[:1], [into[0], None], {}):
        with pytest.raises(TypeError):
            call(sv, s, out=bad)
