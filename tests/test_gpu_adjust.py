"""spec_adjust on the GPU against the definition in float64 (tree_ref.adjust)."""
import numpy as np
import pytest

import tree_ref
from test_gpu_kv import i32, sv  # noqa: F401

pytestmark = pytest.mark.gpu

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}  # half a step of the type, relative


def f32(a):
    import torch
    return torch.tensor(np.ascontiguousarray(a), dtype=torch.float32, device="cuda")


def make(seed, B, N, V, dtype, cap=50, M=0, tree=False, grammar=False, ragged=False, penalties=True):
    import torch
    rng = np.random.default_rng(seed)
    s = dict(dtype=dtype, V=V, N=N)
    x = torch.from_numpy((rng.standard_normal((B, N, V)) * 3).astype(np.float32))
    s["logits"] = (x if dtype == "f32" else x.bfloat16()).cuda()
    s["seq"] = np.minimum((V + 2) ** rng.random((B, cap)), V + 1).astype(int) - 1  # V now and then: no token
    s["seq"][rng.random((B, cap)) < 0.05] = -1
    s["seq_len"] = rng.integers(0, cap + 1, B)
    s["prompt_len"] = (rng.random(B) * (s["seq_len"] + 1)).astype(int)
    s["draft"] = np.minimum((V + 1) ** rng.random((B, N - 1)), V).astype(int) - 1
    s["parents"] = tree_ref.random_parents(rng, B, N - 1) if tree else np.tile(np.arange(N - 1), (B, 1))
    s["tree"] = tree
    s["g"] = rng.integers(0, N, B) if ragged else np.full(B, N - 1)
    s["ragged"] = ragged
    s["r"], s["f"], s["p"] = (1 + rng.random(B), rng.normal(0, 0.5, B), rng.normal(0, 1, B)) if penalties else (
        np.ones(B), np.zeros(B), np.zeros(B))
    s["r"], s["f"], s["p"] = (s[k].astype(np.float32) for k in "rfp")
    s["penalties"] = penalties
    s["ids"], s["bias"] = rng.integers(-1, V + 1, (B, M)), rng.normal(0, 4, (B, M)).astype(np.float32)
    s["allowed"] = rng.random((B, N, V)) < 0.5 if grammar else None
    return s


def args(s):
    kw = dict(draft_tokens=i32(s["draft"]), prompt_len=i32(s["prompt_len"]),
              gamma_per_row=i32(s["g"]) if s["ragged"] else None)
    if s["tree"]:
        kw["tree_mask"] = i32(tree_ref.words(tree_ref.sees(s["parents"], np.full(len(s["g"]), s["N"] - 1))[0]))
    if s["penalties"]:
        kw.update(repetition=f32(s["r"]), frequency=f32(s["f"]), presence=f32(s["p"]))
    if s["ids"].shape[1]:
        kw.update(bias_ids=i32(s["ids"]), bias=f32(s["bias"]))
    if s["allowed"] is not None:
        kw["allowed"] = i32(tree_ref.words(s["allowed"]))
    return (i32(s["seq"]), i32(s["seq_len"])), kw


def check(s, got, before=None):
    """Touched logits: at most five roundings in single precision of the largest
    magnitude on the way (division or product, frequency's product, two
    differences, the bias's sum) and one to the type.  Others: bit by bit."""
    z = (s["logits"] if before is None else before).double().cpu().numpy()
    out = got.double().cpu().numpy()
    for b, g in enumerate(s["g"]):
        n = int(s["seq_len"][b])
        ways = tree_ref.ancestors(s["parents"][b], int(g) + 1)
        assert np.array_equal(out[b, g + 1:], z[b, g + 1:])
        for i in range(int(g) + 1):
            y, size, hit = tree_ref.adjust(
                z[b, i], s["seq"][b, :n] if s["penalties"] else [], int(s["prompt_len"][b]),
                [s["draft"][b, j - 1] for j in ways[i][1:]] if s["penalties"] else [], float(s["r"][b]), float(s["f"][b]),
                float(s["p"][b]), zip(s["ids"][b].tolist(), s["bias"][b].tolist()),
                s["allowed"][b, i] if s["allowed"] is not None else None)
            assert np.array_equal(np.isneginf(out[b, i]), np.isneginf(y))
            there = np.isfinite(y)
            tol = np.where(hit, 5 * 2.0 ** -24 * size + HALF[s["dtype"]] * np.abs(y) * 1.01, 0)
            d = np.abs(np.where(there, out[b, i] - np.where(there, y, 0), 0))
            assert (d <= tol).all(), (b, i, (d / np.maximum(tol, 1e-30)).max())


CASES = [  # B, N, V, keywords
    (1, 1, 1, {}), (2, 1, 7, dict(M=3)), (3, 4, 31, dict(grammar=True)), (2, 3, 33, dict(M=5, grammar=True)),
    (4, 5, 1000, dict(M=9)), (2, 9, 5003, dict(ragged=True, grammar=True, M=40)), (3, 2, 20011, dict(cap=3000)),
    (2, 27, 1025, dict(tree=True, M=3, grammar=True)), (5, 70, 301, dict(tree=True, ragged=True)),
    (1, 2, 100003, dict(M=300, cap=500)), (40, 3, 8192, dict(cap=9)), (2, 2, 999, dict(penalties=False, M=4)),
    (2, 2, 999, dict(penalties=False, grammar=True)), (3, 1, 50304, dict(cap=0)), (300, 2, 515, dict(ragged=True)),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=[f"B{c[0]}N{c[1]}V{c[2]}" + "".join(sorted(c[3])) for c in CASES])
def test_adjust(sv, dtype, case):  # noqa: F811
    B, N, V, kw = case
    s = make(B + N + V, B, N, V, dtype, **kw)
    a, k = args(s)
    before = s["logits"].clone()
    out, st = sv.spec_adjust(s["logits"], *a, with_status=True, **k)
    assert (st.cpu().numpy() == 0).all()
    check(s, out)
    assert (s["logits"] == before).all()
    assert sv.spec_adjust(s["logits"], *a, out=s["logits"], **k) is s["logits"]  # in place
    assert (s["logits"] == out).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("off,pad", [(0, 0), (1, 0), (3, 5), (0, 8), (4, 1)])
def test_adjust_strides(sv, dtype, off, pad):  # noqa: F811
    """Rows at any distance from a multiple of 16 bytes, of both tensors alike or
    not; what lies between the rows stays."""
    import torch
    s = make(3, 3, 4, 2021, dtype, M=6, grammar=True, ragged=True)
    a, k = args(s)
    want = sv.spec_adjust(s["logits"], *a, **k)
    t = s["logits"].dtype
    for other in (off, off + 1):
        src = torch.full((3, 4, 2021 + off + pad), 7.0, dtype=t, device="cuda")
        dst = torch.full((3, 4, 2021 + other + pad), 7.0, dtype=t, device="cuda")
        x, y = src[:, :, off:off + 2021], dst[:, :, other:other + 2021]
        x.copy_(s["logits"])
        assert sv.spec_adjust(x, *a, out=y, **k) is y
        assert torch.equal(y, want)
        assert (dst[:, :, :other] == 7).all() and (dst[:, :, other + 2021:] == 7).all()
        sv.spec_adjust(x, *a, out=x, **k)
        assert torch.equal(x, want) and (src[:, :, :off] == 7).all() and (src[:, :, off + 2021:] == 7).all()


def test_adjust_one_mask_for_all(sv):  # noqa: F811
    """A grammar's mask with axes of stride 0, and one of stride more than its words."""
    import torch
    s = make(4, 3, 4, 333, "f32", grammar=True)
    s["allowed"][:] = s["allowed"][:1, :1]
    a, k = args(s)
    want = sv.spec_adjust(s["logits"], *a, **k)
    check(s, want)
    one = k.pop("allowed")[:1, :1]
    wide = torch.zeros((3, 4, 20), dtype=torch.int32, device="cuda")
    wide[:, :, 2:13] = one
    for m in (one.expand(3, 4, -1), wide[:, :, 2:13]):
        assert torch.equal(sv.spec_adjust(s["logits"], *a, allowed=m, **k), want)


def test_adjust_values(sv):  # noqa: F811
    """Infinities, NaN, the type's lowest value and zeros: what no step applies to
    is as it was, masked places are -inf whatever stands there."""
    import torch
    for t in (torch.float32, torch.bfloat16):
        low = torch.finfo(t).min
        z = torch.tensor([float("nan"), float("inf"), float("-inf"), low, 0.0, -0.0, 2.0, -2.0] * 2, dtype=t, device="cuda")
        z = z[None, None].contiguous()
        seq, n = i32([[2, 3, 4, 6, 7, 7]]), i32([6])
        allowed = i32([[[0x00FF]]])
        out = sv.spec_adjust(z, seq, n, repetition=f32([2.0]), frequency=f32([0.5]), presence=f32([1.0]), allowed=allowed)
        o = out[0, 0].float().cpu().numpy()
        assert np.isnan(o[0]) and np.isposinf(o[1]) and np.isneginf(o[2])
        assert o[3] <= low  # twice the lowest value
        assert o[4] == -1.5 and o[5] == 0 and np.signbit(o[5]) and o[6] == -0.5 and o[7] == -6.0
        assert np.isneginf(o[8:]).all()


def test_adjust_bias_listed_twice(sv):  # noqa: F811
    """The last entry of a token counts, in a list longer than a CTA."""
    import torch
    M, V = 1500, 64
    ids = np.tile(np.arange(M) % 10, (2, 1))
    bias = np.arange(2 * M, dtype=np.float32).reshape(2, M)
    out = sv.spec_adjust(torch.zeros((2, 1, V), device="cuda"), i32(np.zeros((2, 0))), i32([0, 0]), bias_ids=i32(ids), bias=f32(bias))
    want = np.zeros((2, V))
    want[:, :10] = bias[:, -10:]
    assert np.array_equal(out[:, 0].cpu().numpy(), want)


def test_adjust_counts(sv):  # noqa: F811
    """One token many times over: counts beyond what 16 bits hold, and the prompt's own not counted."""
    import torch
    n = 70000
    seq = np.zeros((1, n), int)
    seq[0, -1] = 1
    for prompt, want in ((0, n - 1), (100, n - 101), (n - 1, 0)):
        out = sv.spec_adjust(torch.zeros((1, 1, 9), device="cuda"), i32(seq), i32([n]), prompt_len=i32([prompt]),
                             frequency=f32([1.0]))
        assert out[0, 0].cpu().tolist() == [-float(want), -1.0] + [0.0] * 7


def test_adjust_errors(sv):  # noqa: F811
    """A row in error is NaN, past gamma_b and in place too; the others are as without it."""
    import torch
    B = 12
    s = make(5, B, 3, 700, "f32", M=2, ragged=True)
    s["seq_len"] = np.minimum(s["seq_len"], 40)
    a, k = args(s)
    want = sv.spec_adjust(s["logits"], *a, **k)
    seq, n = a
    n, g, pl = n.clone(), k["gamma_per_row"].clone(), k["prompt_len"].clone()
    r, f, p = (k[x].clone() for x in ("repetition", "frequency", "presence"))
    n[0], n[1], pl[2], pl[3] = -1, 51, -1, int(n[3]) + 1
    g[4], g[5] = 3, -1
    r[6], r[7], r[8], f[9], p[10] = 0.0, -1.0, float("nan"), float("inf"), float("nan")
    k.update(gamma_per_row=g, prompt_len=pl, repetition=r, frequency=f, presence=p)
    L, G, Q = tree_ref.BAD_LENGTH, tree_ref.BAD_GAMMA, tree_ref.BAD_PENALTY
    for out in (None, s["logits"]):
        got, st = sv.spec_adjust(s["logits"], seq, n, out=out, with_status=True, **k)
        assert st.cpu().tolist() == [L, L, L, L, G, G, Q, Q, Q, Q, Q, 0]
        assert torch.isnan(got[:11]).all() and torch.equal(got[11], want[11])


def test_adjust_then_sample(sv):  # noqa: F811
    """A mask that allows one token draws it; one that allows nothing is the sampler's error."""
    import torch
    B, V = 4, 5000
    logits = torch.randn((B, 1, V), device="cuda")
    allowed = np.zeros((B, 1, V), bool)
    for b in range(B - 1):
        allowed[b, 0, 17 * b + 3] = True
    out = sv.spec_adjust(logits, i32(np.zeros((B, 0))), i32([0] * B), allowed=i32(tree_ref.words(allowed)))
    tok = sv.spec_sample(out[:, 0], torch.rand(B, device="cuda"), 1.0, top_k=50, top_p=0.9)
    assert tok.cpu().tolist() == [3, 20, 37, -1]


def test_adjust_in_a_graph_and_on_a_stream(sv):  # noqa: F811
    import torch
    s = make(6, 5, 6, 3001, "bf16", M=5, tree=True, grammar=True)
    (seq, n), k = args(s)
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    sv.spec_adjust(s["logits"], seq, n, **k)
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        out = sv.spec_adjust(s["logits"], seq, n, **k)
    for _ in range(3):
        s["logits"].mul_(-0.5)
        n.sub_(1).clamp_(min=0)
        k["prompt_len"].copy_(torch.minimum(k["prompt_len"], n))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = sv.spec_adjust(s["logits"], seq, n, **k)
        side.wait_stream(torch.cuda.current_stream())
        also = sv.spec_adjust(s["logits"], seq, n, stream=side, **k)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(also, want)


def test_adjust_offsets_past_32_bits(sv):  # noqa: F811
    """Rows that begin beyond 2^32 elements of their tensor."""
    import torch
    V = 64
    big = torch.empty((3, (1 << 31) + 8), dtype=torch.bfloat16, device="cuda")
    x = big[:, 8:8 + V].unsqueeze(1)
    x.copy_(torch.randn((3, 1, V), device="cuda"))
    seq, n = i32([[1, 2, 2], [5, 5, 5], [7, 8, 9]]), i32([3, 3, 3])
    kw = dict(repetition=f32([2, 3, 4]), frequency=f32([1, 1, 1]))
    want = sv.spec_adjust(x.clone(), seq, n, **kw)
    assert torch.equal(sv.spec_adjust(x, seq, n, out=x, **kw), want)


@pytest.mark.parametrize("off", [0, 1, 2, 3])
@pytest.mark.parametrize("length", [16383, 16384, 40001])
def test_adjust_long_sequences(sv, off, length):  # noqa: F811
    """Sequences that begin anywhere within 16 bytes, at both sides of the length from which all threads count."""
    import torch
    rng = np.random.default_rng(length + off)
    V, B = 3001, 3
    seq = rng.integers(-1, V + 1, (B, length))
    store = torch.zeros((B, length + 9), dtype=torch.int32, device="cuda")
    view = store[:, off:off + length]
    view.copy_(i32(seq))
    n, prompt = np.array([length, length - 5, 7]), np.array([0, 1000, 3])
    out = sv.spec_adjust(torch.zeros((B, 1, V), device="cuda"), view, i32(n), prompt_len=i32(prompt), frequency=f32([1.0] * B))
    for b in range(B):
        tail = seq[b, prompt[b]:n[b]]
        want = np.bincount(tail[(tail >= 0) & (tail < V)], minlength=V)
        assert np.array_equal(-out[b, 0].cpu().numpy(), want)
