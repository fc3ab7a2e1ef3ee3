"""The key/value cache operators and the attention over the cache on the GPU
against float64 (kv_ref.py).  What is stored and read back is compared bit by
bit; the attention's tolerance is derived in check_attend()."""
import numpy as np
import pytest

import kv_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verify_03_gb300 as m
    m.build()
    return m


def i32(a):
    import torch
    return torch.tensor(np.ascontiguousarray(a), dtype=torch.int32, device="cuda")


def bf16(bits):
    import torch
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def bits_of(t):
    """uint16 bits of a bfloat16 tensor, uint8 codes of a float8 one."""
    import torch
    if t.dtype == torch.bfloat16:
        return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
    return t.contiguous().view(torch.uint8).cpu().numpy()


def make_cache(sv, rng, fmt, n_pages, H, S, D, garbage=True):
    """A cache whose every byte is set: (KVCache, k, v pages and exponents as numpy)."""
    import torch
    out = []
    for _ in range(2):
        if fmt == "bf16":
            x = rng.standard_normal((n_pages, H, S, D)).astype(np.float32)
            out.append((kv_ref.bf16_bits(x), None))
        else:
            codes = rng.integers(0, 256, (n_pages, H, S, D)).astype(np.uint8)
            codes[(codes & 0x7F) == 0x7F] = 0x30
            out.append((codes, rng.integers(-9, -6, (n_pages, H, S)).astype(np.int8)))
    (k, ke), (v, ve) = out
    if fmt == "bf16":
        return sv.KVCache(bf16(k), bf16(v)), k, v, None, None
    f8 = lambda c: torch.from_numpy(c).cuda().view(torch.float8_e4m3fn)  # noqa: E731
    e8 = lambda e: torch.from_numpy(e).cuda()  # noqa: E731
    return sv.KVCache(f8(k.copy()), f8(v.copy()), e8(ke.copy()), e8(ve.copy())), k, v, ke, ve


def tables(rng, B, pages_each, prefix_pages, spare=2):
    n = B * pages_each + prefix_pages + spare
    ids = rng.permutation(n).astype(np.int32)
    return n, ids[: B * pages_each].reshape(B, pages_each), ids[B * pages_each: B * pages_each + prefix_pages]


# ------------------------------------------------------------------- append
@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
@pytest.mark.parametrize("D,S,src,B,N,H", [(64, 16, "f32", 3, 5, 3), (80, 32, "bf16", 2, 1, 1),
                                           (96, 64, "f32", 1, 70, 2), (128, 128, "bf16", 5, 3, 4)])
@pytest.mark.parametrize("ragged", [False, True])
def test_append(sv, fmt, D, S, src, B, N, H, ragged):
    import torch
    rng = np.random.default_rng(D + N + ragged)
    mp = 3 + N // S
    n, table, _ = tables(rng, B, mp, 0)
    cache, k, v, ke, ve = make_cache(sv, rng, fmt, n, H, S, D)
    x, y = (rng.standard_normal((2, B, N, H, D)) * np.exp(rng.normal(0, 3, (2, B, N, H, 1)))).astype(np.float32)
    x[0, 0, 0] = 0.0
    y[0, 0, 0, :4] = [448.0, 17.0, 19.0, 2.0 ** -9]
    if src == "bf16":
        x, y = (kv_ref.bf16_value(kv_ref.bf16_bits(a)).astype(np.float32) for a in (x, y))
    lens = rng.integers(0, mp * S - N + 1, B)
    gam = rng.integers(0, N, B) if ragged else np.full(B, N - 1)
    dev = lambda a: torch.from_numpy(a).cuda().to(torch.float32 if src == "f32" else torch.bfloat16)  # noqa: E731
    st = sv.spec_kv_append(cache, dev(x), dev(y), i32(table), i32(lens),
                           gamma_per_row=i32(gam) if ragged else None, with_status=True)
    for b in range(B):
        for t in range(gam[b] + 1):
            p = lens[b] + t
            pg, sl = table[b, p // S], p % S
            for h in range(H):
                for a, pages, exps in ((x, k, ke), (y, v, ve)):
                    row = a[b, t, h].astype(np.float64)
                    if fmt == "bf16":
                        pages[pg, h, sl] = kv_ref.bf16_bits(a[b, t, h])
                    else:
                        pages[pg, h, sl], exps[pg, h, sl] = kv_ref.quantise(row)
    assert (st.cpu().numpy() == 0).all()
    # every byte: the written ones and, all others, the old ones
    assert np.array_equal(bits_of(cache.k_pages), k) and np.array_equal(bits_of(cache.v_pages), v)
    if fmt == "e4m3":
        assert np.array_equal(cache.k_exp.cpu().numpy(), ke) and np.array_equal(cache.v_exp.cpu().numpy(), ve)


@pytest.mark.parametrize("src", ["f32", "bf16"])
def test_append_extremes(sv, src):
    """Magnitudes over the whole range, ties, subnormal codes, NaN and infinities."""
    import torch
    rng = np.random.default_rng(5)
    N, D = 260, 64
    x = rng.standard_normal((1, N, 1, D)).astype(np.float32)
    for t in range(N):  # row t is of the size 2^(t - 133)
        x[0, t] = np.clip(np.ldexp(x[0, t].astype(np.float64), t - 133), -3.3e38, 3.3e38).astype(np.float32)
    grid = kv_ref.E4M3[:127]
    x[0, 130, 0] = ((grid[60:124] + grid[61:125]) / 2).astype(np.float32)  # midpoints
    x[0, 130, 0, 0] = 448.0
    x[0, 131, 0, :8] = [np.nan, np.inf, -np.inf, -0.0, 0.0, 2.0 ** -30, -(2.0 ** -20), 1.0]
    x[0, 132, 0, :] = np.nan
    if src == "bf16":
        x = np.where(np.isnan(x), np.nan, kv_ref.bf16_value(kv_ref.bf16_bits(x))).astype(np.float32)
    cache, k, v, ke, ve = make_cache(sv, rng, "e4m3", 17, 1, 16, D)
    d = torch.from_numpy(x).cuda().to(torch.float32 if src == "f32" else torch.bfloat16)
    table = np.arange(17)[None]
    sv.spec_kv_append(cache, d, d, i32(table), i32([3]))
    got, exp = bits_of(cache.k_pages).reshape(-1, D), cache.k_exp.cpu().numpy().reshape(-1)
    for t in range(N):
        codes, e = kv_ref.quantise(x[0, t, 0].astype(np.float64))
        bad = np.isnan(kv_ref.E4M3[codes])
        assert exp[3 + t] == e, t
        assert np.array_equal(np.isnan(kv_ref.E4M3[got[3 + t]]), bad), t
        assert np.array_equal(got[3 + t][~bad], codes[~bad]), t
    assert np.array_equal(bits_of(cache.v_pages).reshape(-1, D)[3:3 + N], got[3:3 + N])


def test_append_errors_write_nothing(sv):
    import torch
    rng = np.random.default_rng(6)
    n, table, _ = tables(rng, 7, 2, 0)
    cache, k, v, ke, ve = make_cache(sv, rng, "e4m3", n, 2, 16, 64)
    table[4, 1], table[5, 0] = n, -1
    prefix = 40
    lens = prefix + np.array([0, 0, 30, -1, 14, 3, 28])
    gam = np.array([4, -1, 2, 0, 3, 0, 3])  # rows: bad gamma, bad gamma, length, length, page, page, good
    x = torch.from_numpy(rng.standard_normal((7, 4, 2, 64)).astype(np.float32)).cuda()
    st = sv.spec_kv_append(cache, x, x, i32(table), i32(lens), gamma_per_row=i32(gam), prefix_len=prefix,
                           with_status=True).cpu().numpy()
    G, Ln, Pg = 16, sv.ROW_BAD_LENGTH, sv.ROW_BAD_PAGE
    assert list(st) == [G, G, Ln, Ln, Pg, Pg, 0]
    changed = (bits_of(cache.k_pages) != k).any(axis=(1, 3))
    want = np.zeros_like(changed)
    want[table[6, 1], 12:16] = True
    want[table[4, 0], 14:16] = True  # the tokens that lie on a good page
    assert np.array_equal(changed, want)


@pytest.mark.parametrize("off", [0, 1, 4])
def test_append_strides(sv, off):
    """k and v as views into one projection, heads before tokens, any alignment."""
    import torch
    rng = np.random.default_rng(7)
    B, N, H, D, S = 2, 3, 4, 80, 16
    n, table, _ = tables(rng, B, 2, 0)
    raw = torch.from_numpy(rng.standard_normal((B, H, N, 2 * D + 8)).astype(np.float32)).cuda().bfloat16()
    k = raw[..., off:off + D].transpose(1, 2)
    v = raw[..., D + off:2 * D + off].transpose(1, 2)
    caches = [make_cache(sv, np.random.default_rng(8), "e4m3", n, H, S, D)[0] for _ in range(2)]
    lens = i32([5, 20])
    sv.spec_kv_append(caches[0], k, v, i32(table), lens)
    sv.spec_kv_append(caches[1], k.contiguous(), v.contiguous(), i32(table), lens)
    for a in ("k_pages", "v_pages"):
        assert np.array_equal(bits_of(getattr(caches[0], a)), bits_of(getattr(caches[1], a)))


# --------------------------------------------------------------------- read
@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("D,S,prefix,begin,n", [(64, 16, 0, 0, 40), (80, 32, 33, 7, 77), (96, 64, 64, 60, 9),
                                                (128, 128, 1, 0, 1), (64, 16, 17, 200, 5)])
def test_read(sv, fmt, out, D, S, prefix, begin, n):
    import torch
    rng = np.random.default_rng(D + n)
    B, H = 3, 2
    mp = -(-60 // S)
    np_, table, pt = tables(rng, B, mp, -(-prefix // S))
    cache, k, v, ke, ve = make_cache(sv, rng, fmt, np_, H, S, D)
    lens = prefix + np.array([0, 1, 60 if mp * S >= 60 else mp * S])
    got = sv.spec_kv_read(cache, i32(table), i32(lens), n, begin=begin, prefix_table=i32(pt), prefix_len=prefix,
                          dtype=torch.float32 if out == "f32" else torch.bfloat16, with_status=True)
    assert (got[2].cpu().numpy() == 0).all()
    for g, pages, exps in ((got[0], k, ke), (got[1], v, ve)):
        val = kv_ref.cache_value(pages, exps)
        want = np.zeros((B, n, H, D))
        for b in range(B):
            row = kv_ref.tokens_of(val, table, pt, prefix, S, b, int(lens[b]))[begin:begin + n]
            want[b, : row.shape[0]] = row
        assert np.array_equal(g.float().cpu().numpy(), want.astype(np.float32))  # exact in bfloat16 too


def test_read_errors_give_nan(sv):
    rng = np.random.default_rng(9)
    n, table, pt = tables(rng, 4, 2, 2)
    cache, *_ = make_cache(sv, rng, "e4m3", n, 1, 16, 64)
    table[2, 1] = n + 5
    lens = 20 + np.array([10, -1, 20, 33])
    k, v, st = sv.spec_kv_read(cache, i32(table), i32(lens), 45, prefix_table=i32(pt), prefix_len=20, with_status=True)
    assert list(st.cpu().numpy()) == [0, sv.ROW_BAD_LENGTH, sv.ROW_BAD_PAGE, sv.ROW_BAD_LENGTH]
    nan = np.isnan(k.float().cpu().numpy()).any(axis=(2, 3))
    want = np.zeros((4, 45), bool)
    want[[1, 3]] = True
    want[2, 36:40] = True
    assert np.array_equal(nan, want)
    assert np.array_equal(np.isnan(v.float().cpu().numpy()).any(axis=(2, 3)), want)


# ------------------------------------------------------------------- attend
def check_attend(got, ref, fmt, gammas, least=0.0):
    """out: one rounding to bfloat16 (8 bits: 2^-8 of the result), one of each
    weight (2^-8 of sum w|v| in bfloat16, 2^-11 in float16), and single
    precision: scores summed in at most 32 steps of 2^-23 of
    size = max scale sum|q k| (2^-18 of it), which move a weight and the sum
    by as much each, and 2^-18 for exponentials, sums and the merge.  lse: the
    scores' error and 2^-20 for the exponential and the logarithm.  least: what
    weights in float16's subnormal range are off by in all, where that shows."""
    out, lse = (x.float().cpu().numpy().astype(np.float64) for x in got[:2])
    want, wl, weight, size = ref
    for b, g in enumerate(gammas):
        assert (out[b, g + 1:] == 0).all() and np.isneginf(lse[b, g + 1:]).all()
        o, w, a, z = out[b, : g + 1], want[b, : g + 1], weight[b, : g + 1], size[b, : g + 1, :, None]
        tol = least + 2.0 ** -8 * np.abs(w) + a * ((2.0 ** -8 if fmt == "bf16" else 2.0 ** -11) + 2.0 ** -17 * z + 2.0 ** -18)
        assert (np.abs(o - w) <= tol * 1.01).all(), (b, (np.abs(o - w) / tol).max())
        z = z[..., 0]
        assert (np.abs(lse[b, : g + 1] - wl[b, : g + 1]) <= 2.0 ** -18 * z + 2.0 ** -20 * (1 + np.abs(wl[b, : g + 1]))).all()


def attend_case(sv, seed, fmt, B, N, Hq, Hkv, D, S, prefix, lens, gammas=None, q_scale=1.0, **kw):
    """Runs one case; returns (results, reference, gammas)."""
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens)
    mp = max(1, -(-(int(lens.max()) + N) // S))
    n, table, pt = tables(rng, B, mp, -(-prefix // S))
    cache, k, v, ke, ve = make_cache(sv, rng, fmt, n, Hkv, S, D)
    qb = kv_ref.bf16_bits((rng.standard_normal((B, N, Hq, D)) * q_scale).astype(np.float32))
    g = np.full(B, N - 1) if gammas is None else np.asarray(gammas)
    got = sv.spec_attend(bf16(qb), cache, i32(table), i32(lens + prefix), prefix_table=i32(pt), prefix_len=prefix,
                         gamma_per_row=None if gammas is None else i32(g), with_status=True, **kw)
    assert (got[2].cpu().numpy() == 0).all()
    ref = kv_ref.attend(kv_ref.bf16_value(qb), kv_ref.cache_value(k, ke), kv_ref.cache_value(v, ve), table,
                        lens + prefix, pt, prefix, g, S, kw.get("scale") or D ** -0.5)
    return got, ref, g


CASES = [  # B, N, Hq, Hkv, D, S, prefix, own lengths
    (1, 1, 1, 1, 64, 16, 0, [0]),            # one token in all
    (1, 1, 8, 1, 128, 16, 0, [700]),         # one query row tile, several CTAs
    (2, 5, 4, 4, 80, 16, 0, [0, 63]),        # no shared heads; a tile's end
    (3, 2, 6, 2, 96, 32, 1, [0, 64, 130]),   # a prefix of one token
    (2, 3, 14, 2, 128, 64, 65, [1, 62]),     # 21 rows; a prefix past a tile's end
    (2, 9, 16, 2, 64, 128, 200, [5, 100]),   # 72 rows: two row tiles
    (5, 4, 12, 1, 128, 16, 48, [3, 0, 80, 17, 200]),  # 48 rows
    (9, 3, 7, 7, 64, 16, 333, [0, 1, 2, 3, 16, 31, 33, 60, 64]),  # prefix rows of many sequences
    (2, 70, 2, 1, 64, 16, 10, [0, 30]),      # a long step: causal over several tiles
]


@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=[f"B{c[0]}N{c[1]}q{c[2]}k{c[3]}D{c[4]}S{c[5]}p{c[6]}" for c in CASES])
def test_attend(sv, fmt, case):
    got, ref, g = attend_case(sv, 11, fmt, *case)
    check_attend(got, ref, fmt, g)


@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
@pytest.mark.parametrize("prefix", [0, 150])
def test_attend_ragged(sv, fmt, prefix):
    B = 12
    rng = np.random.default_rng(3)
    gam = rng.integers(0, 9, B)
    got, ref, g = attend_case(sv, 12, fmt, B, 9, 8, 2, 64, 16, prefix, rng.integers(0, 300, B), gammas=gam)
    check_attend(got, ref, fmt, g)


@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
@pytest.mark.parametrize("q_scale", [0.0, 1e-30, 40.0, 1e6])
def test_attend_query_sizes(sv, fmt, q_scale):
    """No scores at all, tiny ones, and a softmax that is one token's."""
    got, ref, g = attend_case(sv, 13, fmt, 2, 2, 4, 2, 64, 16, 20, [50, 7], q_scale=q_scale)
    check_attend(got, ref, fmt, g)


@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
@pytest.mark.parametrize("D,Hq,Hkv,N", [(64, 16, 8, 1), (80, 8, 8, 3), (96, 24, 8, 9), (128, 32, 8, 5)])
def test_attend_many_tiles(sv, fmt, D, Hq, Hkv, N):
    """More key tiles than any number of CTAs takes at once: long items."""
    got, ref, g = attend_case(sv, 15, fmt, 4, N, Hq, Hkv, D, 64, 3000, [7000, 1, 4097, 5500])
    check_attend(got, ref, fmt, g)


@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
@pytest.mark.parametrize("D,Hq,N", [(64, 8, 9), (128, 16, 4)])
def test_attend_many_items(sv, fmt, D, Hq, N):
    """More short items than any number of CTAs takes at once."""
    rng = np.random.default_rng(16)
    B = 200
    got, ref, g = attend_case(sv, 16, fmt, B, N, Hq, 8, D, 16, 130, rng.integers(0, 200, B), gammas=rng.integers(0, N, B))
    check_attend(got, ref, fmt, g)


def test_attend_scale(sv):
    got, ref, g = attend_case(sv, 14, "e4m3", 2, 2, 4, 2, 128, 16, 20, [50, 7], scale=0.25)
    check_attend(got, ref, "e4m3", g)


def build_batch(sv, fmt, seed=21, prefix=37, lens=(20, 63, 5), N=4, Hq=8, Hkv=2, D=64, S=16):
    rng = np.random.default_rng(seed)
    B, lens = len(lens), np.asarray(lens)
    mp = -(-(int(lens.max()) + N) // S)
    n, table, pt = tables(rng, B, mp, -(-prefix // S))
    cache, k, v, ke, ve = make_cache(sv, rng, fmt, n, Hkv, S, D)
    qb = kv_ref.bf16_bits(rng.standard_normal((B, N, Hq, D)).astype(np.float32))
    return dict(cache=cache, k=k, v=v, ke=ke, ve=ve, table=table, pt=pt, q=qb, lens=lens + prefix, prefix=prefix,
                S=S, N=N, D=D)


def call(sv, s, **kw):
    return sv.spec_attend(bf16(s["q"]), s["cache"], i32(s["table"]), i32(s["lens"]), prefix_table=i32(s["pt"]),
                          prefix_len=s["prefix"], with_status=True, **kw)


def reference(s):
    return kv_ref.attend(kv_ref.bf16_value(s["q"]), kv_ref.cache_value(s["k"], s["ke"]),
                         kv_ref.cache_value(s["v"], s["ve"]), s["table"], s["lens"], s["pt"], s["prefix"],
                         np.full(len(s["lens"]), s["N"] - 1), s["S"], s["D"] ** -0.5)


def put(s, which, pg, h, sl, d, code):
    import torch
    t = getattr(s["cache"], which + "_pages")
    raw = t.view(torch.uint8 if t.dtype == torch.float8_e4m3fn else torch.int16)
    raw[pg, h, sl, d] = int(np.int16(np.uint16(code))) if t.dtype == torch.bfloat16 else code
    s[which][pg, h, sl, d] = code


@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
def test_attend_garbage_past_the_end(sv, fmt):
    """NaN and infinities in slots that hold no token, exponents included."""
    s = build_batch(sv, fmt)
    want = reference(s)
    P, S, N = s["prefix"], s["S"], s["N"]
    free = [(s["pt"][-1], sl) for sl in range(P % S, S)]
    for b, n in enumerate(s["lens"]):
        end = n - P + N
        free += [(s["table"][b, p // S], p % S) for p in range(end, s["table"].shape[1] * S)]
    for pg, sl in free:
        for w in "kv":
            for h in range(2):
                put(s, w, pg, h, sl, slice(None), 0x7F if fmt == "e4m3" else 0x7F80 if sl % 2 else 0x7FC1)
                if fmt == "e4m3":
                    getattr(s["cache"], w + "_exp")[pg, h, sl] = -128 if sl % 2 else 127
    check_attend(call(sv, s), want, fmt, np.full(3, N - 1))


@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
@pytest.mark.parametrize("which", ["k", "v"])
def test_attend_masked_nan_stays_where_it_is_seen(sv, fmt, which):
    """A NaN in the entry of the step's token t reaches the queries i >= t
    only; an infinity of a value (bfloat16) makes those outputs infinite."""
    s = build_batch(sv, fmt)
    want = reference(s)
    spots = {0: (2, 1, 7), 1: (3, 0, 63), 2: (1, 1, 0)}  # sequence: token of the step, head, element
    for b, (t, h, d) in spots.items():
        p = s["lens"][b] - s["prefix"] + t
        code = 0x7F if fmt == "e4m3" else (0xFF80 if which == "v" and b == 1 else 0x7FC0)
        put(s, which, s["table"][b, p // s["S"]], h, p % s["S"], d, code)
    out, lse, st = (x.float().cpu().numpy() for x in call(sv, s))
    ref_out = want[0]
    for b, (t, h, d) in spots.items():
        heads = slice(4 * h, 4 * h + 4)
        hit = np.zeros(out[b].shape, bool)
        hit[t:, heads, d if which == "v" else slice(None)] = True
        if fmt == "bf16" and which == "v" and b == 1:
            assert np.isneginf(out[b][hit]).all()
        else:
            assert np.isnan(out[b][hit]).all()
        assert np.isfinite(out[b][~hit]).all()
        assert np.abs(out[b] - ref_out[b])[~hit].max() < 0.05 * (1 + np.abs(ref_out[b]).max())
        assert np.isnan(lse[b, t:, heads]).all() == (which == "k")
        assert np.isfinite(lse[b, :t]).all()
    assert (st == 0).all()


@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
def test_attend_error_rows(sv, fmt):
    import torch
    s = build_batch(sv, fmt, lens=(20, 63, 5, 9, 30, 12))
    want = reference(s)
    s["table"][1, 2] = -7
    s["table"][3, 4] = 10 ** 6  # beyond its tokens: not in use
    good = [0, 3, 5]
    gam = np.array([3, 3, 4, 3, 3, 3])
    s["lens"][4] = s["prefix"] - 1
    got = sv.spec_attend(bf16(s["q"]), s["cache"], i32(s["table"]), i32(s["lens"]), prefix_table=i32(s["pt"]),
                         prefix_len=s["prefix"], gamma_per_row=i32(gam), with_status=True)
    assert list(got[2].cpu().numpy()) == [0, sv.ROW_BAD_PAGE, 16, 0, sv.ROW_BAD_LENGTH, 0]
    for b in (1, 2, 4):
        assert torch.isnan(got[0][b]).all() and torch.isnan(got[1][b]).all()
    check_attend([x[good] for x in got[:2]], [x[good] for x in want], fmt, gam[good])
    s["pt"][1] = -1  # a page of the prefix: every sequence
    got = call(sv, s)
    assert torch.isnan(got[0]).all() and (got[2].cpu().numpy() & sv.ROW_BAD_PAGE).astype(bool)[[0, 1, 2, 3, 5]].all()


@pytest.mark.parametrize("off", [0, 1, 2, 8])
def test_attend_query_strides(sv, off):
    """q as a view into a fused projection with heads before tokens, any alignment."""
    import torch
    s = build_batch(sv, "e4m3")
    q = bf16(s["q"])
    B, N, H, D = q.shape
    raw = torch.full((B, H, N, D + 16), float("nan"), dtype=torch.bfloat16, device="cuda")
    view = raw[..., off:off + D].transpose(1, 2)
    view.copy_(q)
    args = (s["cache"], i32(s["table"]), i32(s["lens"]))
    kw = dict(prefix_table=i32(s["pt"]), prefix_len=s["prefix"])
    a, b = sv.spec_attend(view, *args, **kw), sv.spec_attend(q, *args, **kw)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_attend_strided_pages_and_table(sv):
    """Keys and values in one allocation, a page table with spare columns."""
    import torch
    s = build_batch(sv, "e4m3")
    want = call(sv, s)
    c = s["cache"]
    both = torch.empty((c.n_pages, 2) + c.k_pages.shape[1:], dtype=torch.uint8, device="cuda")
    both[:, 0], both[:, 1] = c.k_pages.view(torch.uint8), c.v_pages.view(torch.uint8)
    both = both.view(torch.float8_e4m3fn)
    c2 = sv.KVCache(both[:, 0], both[:, 1], c.k_exp, c.v_exp)
    wide = torch.full((len(s["lens"]), s["table"].shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    wide[:, : s["table"].shape[1]] = i32(s["table"])
    got = sv.spec_attend(bf16(s["q"]), c2, wide[:, : s["table"].shape[1]], i32(s["lens"]), prefix_table=i32(s["pt"]),
                         prefix_len=s["prefix"])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
def test_attend_prefix_equals_own_tokens(sv, fmt):
    """The same tokens as a prefix or as own pages: the same attention."""
    s = build_batch(sv, fmt, prefix=48, lens=(0, 7, 33))
    a = [x.float().cpu().numpy() for x in call(sv, s)[:2]]
    table = np.concatenate([np.tile(s["pt"], (3, 1)), s["table"]], 1)
    b = [x.float().cpu().numpy() for x in
         sv.spec_attend(bf16(s["q"]), s["cache"], i32(table), i32(s["lens"]))]
    ref = reference(s)
    check_attend(sv.spec_attend(bf16(s["q"]), s["cache"], i32(table), i32(s["lens"])), ref, fmt, np.full(3, 3))
    assert np.abs(a[1] - b[1]).max() < 1e-5
    assert np.abs(a[0] - b[0]).max() <= 2.0 ** -7 * np.abs(b[0]).max()


def test_attend_is_reproducible_and_stream_ordered(sv):
    """Bitwise the same on every call, also on another stream and into given tensors."""
    import torch
    rng = np.random.default_rng(2)
    s = build_batch(sv, "e4m3", prefix=300, lens=tuple(rng.integers(0, 500, 20)), Hq=16, D=128)
    want = call(sv, s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    args = (bf16(s["q"]), s["cache"], i32(s["table"]), i32(s["lens"]))
    pt = i32(s["pt"])
    out = (torch.empty_like(want[0]), torch.empty_like(want[1]))
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = sv.spec_attend(*args, prefix_table=pt, prefix_len=s["prefix"], out=out, stream=side)
        side.synchronize()
        assert got[0] is out[0]
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_attend_in_a_graph(sv):
    """Captured once, replayed with new lengths and queries."""
    import torch
    s = build_batch(sv, "e4m3", prefix=64, lens=(20, 63, 5))
    q, table, lens, pt = bf16(s["q"]), i32(s["table"]), i32(s["lens"]), i32(s["pt"])
    kw = dict(prefix_table=pt, prefix_len=64)
    sv.spec_attend(q, s["cache"], table, lens, **kw)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        sv.spec_attend(q, s["cache"], table, lens, workspace=ws, **kw)
        side.synchronize()
        with torch.cuda.graph(g, stream=side):
            out = sv.spec_attend(q, s["cache"], table, lens, workspace=ws, **kw)
    for step in range(3):
        lens.copy_(i32(64 + np.array([3 * step, 40 - step, 9])))
        q.mul_(-0.5)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = sv.spec_attend(q, s["cache"], table, lens, **kw)
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_offsets_past_32_bits(sv):
    """A pool whose last pages lie beyond 2^32 elements and bytes."""
    import torch
    H, S, D = 8, 128, 128
    n = (1 << 32) // (H * S * D) + 40
    pages = [torch.empty((n, H, S, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    exps = [torch.zeros((n, H, S), dtype=torch.int8, device="cuda") for _ in range(2)]
    big = sv.KVCache(*pages, *exps)
    small = sv.KVCache.empty(6, H, S, D)
    rng = np.random.default_rng(4)
    x, y = (torch.from_numpy(rng.standard_normal((2, 300, H, D)).astype(np.float32)).cuda() for _ in range(2))
    ids = np.arange(6).reshape(2, 3)
    far = ids + n - 6
    zero, lens = i32([0, 0]), i32([296, 299])
    q = torch.from_numpy(rng.standard_normal((2, 1, 16, D)).astype(np.float32)).cuda().bfloat16()
    res = []
    for c, t in ((big, far), (small, ids)):
        sv.spec_kv_append(c, x, y, i32(t), zero)
        res.append(sv.spec_kv_read(c, i32(t), i32([300, 300]), 300) + sv.spec_attend(q, c, i32(t), lens))
    for a, b in zip(*res):
        assert torch.equal(a, b)


def test_append_then_attend_follows_the_step(sv):
    """Two verify steps: rejected drafts' entries are overwritten, and the
    attention sees what the last append left."""
    import torch
    rng = np.random.default_rng(30)
    B, N, H, D, S = 3, 4, 2, 64, 16
    n, table, pt = tables(rng, B, 3, 1)
    cache, k, v, ke, ve = make_cache(sv, rng, "bf16", n, H, S, D)
    t, p = i32(table), i32(pt)
    lens = np.array([10, 25, 13])
    for step in range(2):
        x, y = (torch.from_numpy(rng.standard_normal((B, N, H, D)).astype(np.float32)).cuda().bfloat16() for _ in range(2))
        sv.spec_kv_append(cache, x, y, t, i32(lens), prefix_len=9)
        for b in range(B):
            for j in range(N):
                pos = lens[b] - 9 + j
                k[table[b, pos // S], :, pos % S] = bits_of(x[b, j])
                v[table[b, pos // S], :, pos % S] = bits_of(y[b, j])
        qb = kv_ref.bf16_bits(rng.standard_normal((B, N, 4, D)).astype(np.float32))
        got = sv.spec_attend(bf16(qb), cache, t, i32(lens), prefix_table=p, prefix_len=9)
        ref = kv_ref.attend(kv_ref.bf16_value(qb), kv_ref.cache_value(k, None), kv_ref.cache_value(v, None), table, lens,
                            pt, 9, np.full(B, N - 1), S, D ** -0.5)
        check_attend(got, ref, "bf16", np.full(B, N - 1))
        lens = lens + np.array([1, 3, 2])  # accepted drafts and the new token


# ------------------------------------------- prefixes with many query rows
MANY = [  # B, N, Hq, Hkv, D, S, prefix: more than 64 query rows of a key/value head
    (13, 5, 2, 2, 128, 16, 1),       # 65 rows, one token
    (9, 9, 4, 4, 64, 64, 128),       # 81 rows, a tile's end
    (22, 3, 8, 2, 80, 16, 129),      # 264 rows: more than a row tile; one token past a tile
    (16, 4, 16, 4, 96, 32, 63),      # 256 rows, half a tile less one token
    (30, 9, 4, 2, 128, 128, 700),    # 540 rows
    (70, 1, 6, 3, 64, 16, 2000),     # single tokens
]


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
@pytest.mark.parametrize("case", MANY, ids=[f"B{c[0]}N{c[1]}q{c[2]}k{c[3]}D{c[4]}S{c[5]}p{c[6]}" for c in MANY])
def test_attend_shared_prefix(sv, fmt, case, ragged):
    B, N, Hq, Hkv, D, S, prefix = case
    rng = np.random.default_rng(31)
    gam = rng.integers(0, N, B) if ragged else None
    got, ref, g = attend_case(sv, 32, fmt, B, N, Hq, Hkv, D, S, prefix, rng.integers(0, 20, B), gammas=gam)
    check_attend(got, ref, fmt, g)


@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
@pytest.mark.parametrize("q_scale", [0.0, 1e-30, 40.0, 1e6])
def test_attend_shared_prefix_query_sizes(sv, fmt, q_scale):
    """Weights far below a row's largest: float16 has steps of 2^-24 there, the
    largest weight is 2^11 or more, so each is off by up to 2^-36 of it, times
    the largest value (448 * 2^-7), for 300 tokens of the prefix."""
    got, ref, g = attend_case(sv, 33, fmt, 20, 4, 4, 1, 64, 16, 300, np.arange(20), q_scale=q_scale)
    check_attend(got, ref, fmt, g, least=300 * 2.0 ** -36 * 3.5 if fmt == "e4m3" else 0.0)


def many(sv, fmt, prefix=333, B=24, **kw):
    return build_batch(sv, fmt, prefix=prefix, lens=tuple(np.arange(B) % 7), **kw)  # 24 * 4 * 4 rows a head


@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
def test_attend_shared_prefix_garbage_past_the_end(sv, fmt):
    """NaN and infinities behind the prefix in its last page, exponents included."""
    s = many(sv, fmt, prefix=333, S=64)
    want = reference(s)
    for sl in range(333 % 64, 64):
        for w in "kv":
            for h in range(2):
                put(s, w, s["pt"][-1], h, sl, slice(None), 0x7F if fmt == "e4m3" else 0x7F80 if sl % 2 else 0x7FC1)
                if fmt == "e4m3":
                    getattr(s["cache"], w + "_exp")[s["pt"][-1], h, sl] = -128 if sl % 2 else 127
    check_attend(call(sv, s), want, fmt, np.full(24, 3))


@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("p", [0, 200, 332])
def test_attend_shared_prefix_nan(sv, fmt, which, p):
    """A NaN of the prefix reaches its own head's queries, a value's only its element."""
    s = many(sv, fmt)
    want = reference(s)
    put(s, which, s["pt"][p // 16], 1, p % 16, 5, 0x7F if fmt == "e4m3" else 0x7FC0)
    out, lse, st = (x.float().cpu().numpy() for x in call(sv, s))
    hit = np.zeros(out.shape, bool)
    hit[:, :, 4:, 5 if which == "v" else slice(None)] = True
    assert np.isnan(out[hit]).all() and np.isfinite(out[~hit]).all() and (st == 0).all()
    assert np.isnan(lse[:, :, 4:]).all() == (which == "k") and np.isfinite(lse[:, :, :4]).all()
    assert np.abs(out - want[0])[~hit].max() < 0.05 * (1 + np.abs(want[0]).max())


def test_attend_shared_prefix_exponents(sv):
    """Tokens whose entries differ in size by up to 2^18, and entries of zeros."""
    s = many(sv, "e4m3", prefix=500, D=128)
    rng = np.random.default_rng(34)
    for w in "kv":
        e = getattr(s["cache"], w + "_exp")
        new = rng.integers(-24, -5, e.shape).astype(np.int8)
        zero = rng.random(e.shape) < 0.1
        new[zero] = -100
        s[w][zero] = 0
        s[w + "e"][...] = new
        e.copy_(__import__("torch").from_numpy(new))
        pages = getattr(s["cache"], w + "_pages")
        pages.view(__import__("torch").uint8).copy_(__import__("torch").from_numpy(s[w]))
    check_attend(call(sv, s), reference(s), "e4m3", np.full(24, 3))


def test_attend_shared_prefix_errors(sv):
    """Rows in error among many, and a bad page of the prefix."""
    import torch
    s = many(sv, "e4m3")
    want = reference(s)
    s["table"][3, 0] = -1
    s["lens"][7] = s["prefix"] - 1
    got = call(sv, s)
    st = got[2].cpu().numpy()
    bad = [3, 7]
    good = [b for b in range(24) if b not in bad]
    assert list(st[bad]) == [sv.ROW_BAD_PAGE, sv.ROW_BAD_LENGTH] and (st[good] == 0).all()
    assert torch.isnan(got[0][bad]).all() and torch.isnan(got[1][bad]).all()
    check_attend([x[good] for x in got[:2]], [x[good] for x in want], "e4m3", np.full(22, 3))
    s["pt"][2] = s["cache"].n_pages
    got = call(sv, s)
    assert torch.isnan(got[0]).all() and (got[2].cpu().numpy()[good] == sv.ROW_BAD_PAGE).all()


@pytest.mark.parametrize("off", [0, 1, 8])
def test_attend_shared_prefix_query_strides(sv, off):
    import torch
    s = many(sv, "bf16", D=80)
    q = bf16(s["q"])
    B, N, H, D = q.shape
    raw = torch.full((B, H, N, D + 16), float("nan"), dtype=torch.bfloat16, device="cuda")
    view = raw[..., off:off + D].transpose(1, 2)
    view.copy_(q)
    args = (s["cache"], i32(s["table"]), i32(s["lens"]))
    kw = dict(prefix_table=i32(s["pt"]), prefix_len=s["prefix"])
    a, b = sv.spec_attend(view, *args, **kw), sv.spec_attend(q, *args, **kw)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_attend_workspace_is_reusable(sv):
    """One workspace, not cleared, for calls of other shapes in turn: the same bits."""
    import torch
    runs = [many(sv, "e4m3"), build_batch(sv, "e4m3"), many(sv, "e4m3", prefix=40, D=128)]
    want = [call(sv, s) for s in runs]
    ws = torch.full((1 << 28,), 0xFF, dtype=torch.uint8, device="cuda")
    for k in (0, 1, 2, 1, 0):
        got = call(sv, runs[k], workspace=ws)
        assert all(torch.equal(x, y) for x, y in zip(got, want[k]))


def test_append_and_read_on_another_stream(sv):
    """Ordered on the stream that is given: what is read is what was appended there."""
    import torch
    rng = np.random.default_rng(35)
    H, D, S = 4, 128, 16
    cache = sv.KVCache.empty(40, H, S, D)
    x, y = (torch.from_numpy(rng.standard_normal((2, 300, H, D)).astype(np.float32)).cuda() for _ in range(2))
    table, zero, n = i32(np.arange(40).reshape(2, 20)), i32([0, 0]), i32([300, 300])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    sv.spec_kv_append(cache, x, y, table, zero, stream=side)
    k, v = sv.spec_kv_read(cache, table, n, 300, stream=side)
    side.synchronize()
    # half a step of e4m3: 2^-4 of an element, below its least normal 2^-10 2^e; 224 2^e is less than the largest
    for a, b in ((k, x), (v, y)):
        a, b = a.float().cpu().numpy(), b.cpu().numpy()
        most = np.abs(b).max(-1, keepdims=True)
        assert (np.abs(a - b) <= np.abs(b) * 2.0 ** -4 + most * 2.0 ** -10 / 224).all()


# ----------------------------------------------- values and scores of zero
def zero_values(sv, rows, prefix, fmt="e4m3", keys="random", own="random", heads=None):
    """`rows` query rows of each key/value head over a prefix whose values are
    all zero, as append stores them (e4m3: exponent -100), and own tokens.  So
    many heads that a CTA sums up 1024 tokens of one of them and more."""
    import torch
    B = rows // 4
    heads = heads or -(-9 * 152 * 128 // prefix)
    s = build_batch(sv, fmt, seed=41, prefix=prefix, lens=tuple(np.arange(B) % 5), N=1, Hq=4 * heads, Hkv=heads, S=64)
    pages = s["pt"] if own == "random" else np.arange(s["cache"].n_pages)
    for w in ("k", "v") if keys == "zero" else ("v",):
        s[w][pages] = 0
        p = torch.from_numpy(np.ascontiguousarray(s[w]).view(np.int16 if fmt == "bf16" else np.uint8)).cuda()
        t = getattr(s["cache"], w + "_pages")
        t.view(torch.int16 if fmt == "bf16" else torch.uint8).copy_(p)
        if fmt == "e4m3":
            s[w + "e"][pages] = kv_ref.E_MIN
            getattr(s["cache"], w + "_exp").copy_(torch.from_numpy(s[w + "e"]))
    return s


def check_zero(got, ref, fmt):
    """check_attend's bounds, and for lse 2^-16 more: the largest exponent of the
    weights (-100 and 7 below it) and the logarithm of their sum are then of
    opposite sign and near 2^7, each with a rounding of 2^-17 at most."""
    out, lse = (x.float().cpu().numpy().astype(np.float64) for x in got[:2])
    want, wl, weight, size = ref
    z = size[..., None]
    tol = 2.0 ** -8 * np.abs(want) + weight * ((2.0 ** -8 if fmt == "bf16" else 2.0 ** -11) + 2.0 ** -17 * z + 2.0 ** -18 + 2.0 ** -16)
    assert (np.abs(out - want) <= tol * 1.01).all()
    assert (np.abs(lse - wl) <= 2.0 ** -18 * size + 2.0 ** -20 * (1 + np.abs(wl)) + 2.0 ** -16).all()


@pytest.mark.parametrize("rows,prefix,keys,own", [
    (64, 1024, "zero", "zero"), (64, 8192, "random", "random"), (80, 960, "zero", "random"), (80, 1024, "zero", "random"),
    (80, 1024, "zero", "zero"), (80, 2048, "zero", "random"), (80, 8192, "zero", "zero"), (80, 8192, "random", "random")])
def test_attend_prefix_of_zero_values(sv, rows, prefix, keys, own):
    """The weights of zero values count: an output of 0 from them alone, a share
    of what the own tokens give, and the logarithm of their number."""
    s = zero_values(sv, rows, prefix, keys=keys, own=own)
    got, ref = call(sv, s), reference(s)
    check_zero(got, ref, "e4m3")
    if own == "zero":
        assert (got[0] == 0).all()


def test_attend_zero_values_of_many_tokens(sv):
    """2^21 tokens of equal weight and zero values for each sequence, all of them
    the same page: own tokens that one CTA sums up without an end."""
    import torch
    B, n, S, D = 640, 1 << 21, 128, 64
    cache = sv.KVCache.empty(1, 1, S, D)
    zero = torch.zeros((1, S, 1, D), device="cuda")
    one = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    sv.spec_kv_append(cache, zero, zero, one, i32([0]))
    table = torch.zeros((B, n // S), dtype=torch.int32, device="cuda")
    q = torch.zeros((B, 1, 1, D), dtype=torch.bfloat16, device="cuda")
    out, lse, st = sv.spec_attend(q, cache, table, torch.full((B,), n - 1, dtype=torch.int32, device="cuda"), with_status=True)
    assert (st == 0).all() and (out == 0).all()
    assert (lse.double() - 21 * np.log(2)).abs().max() <= 2.0 ** -16 + 2.0 ** -20 * 16


@pytest.mark.parametrize("rows", [64, 80])
@pytest.mark.parametrize("e", [kv_ref.E_MIN, kv_ref.E_MAX])
def test_attend_values_at_the_ends_of_the_exponents(sv, rows, e):
    """All values with the least or the largest exponent (codes up to 2^3, so
    that sums of some of them are finite)."""
    import torch
    rng = np.random.default_rng(42)
    B = rows // 4
    s = build_batch(sv, "e4m3", seed=43, prefix=700, lens=tuple(np.arange(B) % 90), N=1, Hq=8, Hkv=2, S=64)
    s["v"][...] = rng.integers(0, 0x51, s["v"].shape) | rng.integers(0, 2, s["v"].shape) << 7
    s["ve"][...] = e
    s["cache"].v_pages.view(torch.uint8).copy_(torch.from_numpy(s["v"]))
    s["cache"].v_exp.fill_(e)
    got, ref = call(sv, s), reference(s)
    check_zero(got, ref, "e4m3")
    assert (got[2] == 0).all()


@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
@pytest.mark.parametrize("rows", [64, 80])
@pytest.mark.parametrize("prefix", [100, 128, 192])
@pytest.mark.parametrize("what", ["scale", "zeros"])
def test_attend_no_scores(sv, fmt, rows, prefix, what):
    """scale = 0, and zero queries on zero keys: every token weighs the same, and
    what lies behind the prefix's end still weighs nothing."""
    import torch
    B = rows // 4
    s = build_batch(sv, fmt, seed=44, prefix=prefix, lens=tuple(np.arange(B) % 9), N=1, Hq=8, Hkv=2, S=32)
    if what == "zeros":
        s["q"][...] = 0
        s["k"][...] = 0
        s["cache"].k_pages.view(torch.uint8).zero_()
        if fmt == "e4m3":
            s["ke"][...] = kv_ref.E_MIN
            s["cache"].k_exp.fill_(kv_ref.E_MIN)
    scale = 0.0 if what == "scale" else s["D"] ** -0.5
    got = call(sv, s, scale=scale)
    ref = kv_ref.attend(kv_ref.bf16_value(s["q"]), kv_ref.cache_value(s["k"], s["ke"]), kv_ref.cache_value(s["v"], s["ve"]),
                        s["table"], s["lens"], s["pt"], prefix, np.zeros(B, int), s["S"], scale)
    check_attend(got, ref, fmt, np.zeros(B, int))


# ------------------------------------------------- streams, graphs and workspaces
def test_attend_graph_keeps_its_workspace(sv):
    """A graph captured with the workspace left to the call, replayed behind
    larger calls on the same stream and with the freed memory in use."""
    import torch
    s = build_batch(sv, "e4m3", prefix=64, lens=(20, 63, 5))
    large = many(sv, "e4m3")
    q, table, lens, pt = bf16(s["q"]), i32(s["table"]), i32(s["lens"]), i32(s["pt"])
    kw = dict(prefix_table=pt, prefix_len=64)
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        want = sv.spec_attend(q, s["cache"], table, lens, **kw)
        side.synchronize()
        with torch.cuda.graph(g, stream=side):
            out = sv.spec_attend(q, s["cache"], table, lens, **kw)
        for _ in range(3):
            call(sv, large)
            junk = [torch.full((1 << k,), 0x7F, dtype=torch.uint8, device="cuda") for k in range(12, 26)]
            g.replay()
            side.synchronize()
            assert all((j == 0x7F).all() for j in junk)
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_attend_on_a_stream_while_the_callers_allocates(sv):
    """Calls of growing size on a given stream, the caller's stream filling what
    it gets from the allocator between them."""
    import torch
    runs = [build_batch(sv, "e4m3"), many(sv, "e4m3"), many(sv, "e4m3", prefix=1000, D=128)]
    args = [((bf16(s["q"]), s["cache"], i32(s["table"]), i32(s["lens"])), dict(prefix_table=i32(s["pt"]), prefix_len=s["prefix"]))
            for s in runs]
    want = [sv.spec_attend(*a, **kw) for a, kw in args]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = []
    for _ in range(10):
        for a, kw in args:
            got.append(sv.spec_attend(*a, stream=side, **kw))
            for k in (16, 20, 24, 26):
                torch.full((1 << k,), 0x7F, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for k, g in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(g, want[k % 3])), k


def test_attend_from_threads_on_one_stream(sv):
    """Calls of several threads whose launches may come between one another's."""
    import threading

    import torch
    runs = [build_batch(sv, "e4m3", seed=50 + k, prefix=40 + k) for k in range(4)]
    want = [call(sv, s) for s in runs]
    wrong = []

    def work(k):
        for _ in range(50):
            got = call(sv, runs[k])
            if not all(torch.equal(x, y) for x, y in zip(got, want[k])):
                wrong.append(k)
    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@pytest.mark.parametrize("rows", [0, 64, 80])
@pytest.mark.parametrize("far", [10, 25, 30, 60])
def test_attend_value_exponents_far_apart(sv, rows, far):
    """One token whose values are 2^far times as large as the others', but for an
    element of 0, all tokens of equal weight w.  Over an e4m3 cache a weight
    times 2^e is a float16 number (e the token's exponent), the row's largest
    at 2^8 or above and its last place 2^-24: off by 2^-33 of the largest at
    most, beside 2^-11 of itself.  From 65 rows on e is the tile's largest, the
    row's largest at 2^11 or above (2^-36), and a value u 2^e is a float16
    number times 2^(e - 7) (2^-32 of 2^e at most).  rows = 0: own tokens only."""
    import torch
    B = max(rows, 8) // 4
    prefix = 300 if rows else 0
    s = build_batch(sv, "e4m3", seed=45, prefix=prefix, lens=(150,) * B, N=1, Hq=8, Hkv=2, S=64)
    s["q"][...] = 0
    pg, sl = (s["pt"][2], 5) if rows else (s["table"][1, 1], 5)
    s["ve"][pg, :, sl] = -8 + far
    s["v"][pg, :, sl, 7] = 0
    s["cache"].v_exp.copy_(torch.from_numpy(s["ve"]))
    s["cache"].v_pages.view(torch.uint8).copy_(torch.from_numpy(s["v"]))
    out, lse, st = (x.float().cpu().numpy().astype(np.float64) for x in call(sv, s))
    want, wl, weight, _ = reference(s)
    assert (st == 0).all() and (np.abs(lse - wl) <= 2.0 ** -20 * (1 + np.abs(wl))).all()
    n = prefix + 151
    val = kv_ref.cache_value(s["v"], s["ve"])
    for b in range(B):
        tok = kv_ref.tokens_of(val, s["table"], s["pt"], prefix, 64, b, n)
        e = kv_ref.tokens_of(s["ve"][..., None].astype(np.float64), s["table"], s["pt"], prefix, 64, b, n)[..., 0]
        off, rough = 2.0 ** -33, np.zeros((n, 2))  # the own tokens' bound, which covers a prefix's too
        if rows > 64:
            for t in range(0, prefix, 128):
                e[t:min(t + 128, prefix)] = e[t:min(t + 128, prefix)].max(0)
            rough[:prefix] = 2.0 ** (e[:prefix] - 32)
        for h in range(8):
            u = np.abs(tok[:, h // 4]) * 2.0 ** -e[:, h // 4, None]
            tol = off * (2.0 ** e[:, h // 4].max() / n) * u.sum(0) + rough[:, h // 4].mean()
            tol = tol + 2.0 ** -8 * np.abs(want[b, 0, h]) + weight[b, 0, h] * (2.0 ** -11 + 2.0 ** -18)
            assert (np.abs(out[b, 0, h] - want[b, 0, h]) <= tol * 1.01).all(), (b, h)


@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
@pytest.mark.parametrize("case", [(1, 500, 4, 2, 64, 16, 0, [0]), (2, 300, 2, 1, 128, 64, 70, [0, 130]),
                                  (2, 260, 3, 1, 80, 32, 500, [1, 0])], ids=["begin", "behind", "many"])
def test_attend_prompt(sv, fmt, case):
    """A prompt in one call: hundreds of query tokens, each with one more to see."""
    got, ref, g = attend_case(sv, 46, fmt, *case)
    check_attend(got, ref, fmt, g)
