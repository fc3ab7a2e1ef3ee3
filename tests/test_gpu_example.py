"""examples/shared_prompt.py: what it decodes greedily is what the target model
without any cache decodes, up to the rounding of the cache."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "shared_prompt.py")
    spec = importlib.util.spec_from_file_location("shared_prompt", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.sv.build()
    return m


def plain_logits(m, tokens):
    """All positions' logits of one sequence, in float64 and without a cache."""
    import torch
    n = len(tokens)
    x = m.start(tokens[None], torch.arange(n, device="cuda")[None]).double()
    w = lambda t: t.double()  # noqa: E731
    for layer in m.layers:
        y = (m.norm(x) @ w(layer["qkv"])).unflatten(-1, (-1, m.head_dim))[0]
        q, k, v = y.split([m.n_heads, m.n_kv_heads, m.n_kv_heads], 1)
        k, v = (t.repeat_interleave(m.n_heads // m.n_kv_heads, 1) for t in (k, v))
        s = torch.einsum("ihd,jhd->hij", q, k) * m.head_dim ** -0.5
        s = s.masked_fill(torch.ones(n, n, device="cuda").triu(1).bool(), float("-inf"))
        o = torch.einsum("hij,jhd->ihd", s.softmax(-1), v).flatten(1)[None]
        x = x + o @ w(layer["o"])
        x = x + torch.relu(m.norm(x) @ w(layer["up"])) @ w(layer["down"])
    return (m.norm(x) @ m.norm(w(m.embed)).T * x.shape[-1] ** -0.5)[0]


@pytest.mark.parametrize("gamma", [1, 4])
def test_greedy_is_the_targets_choice(ex, gamma):
    """Every token's plain logit is at most `near` below the largest.  An e4m3
    entry is off by up to 2^-4 of itself, a layer's attention output by as much
    at most and the residual stream with it: 2^-3 of the logits' norm for two
    layers, of which a logit (512 of them, of unit vectors' products scaled by
    16) has a share of 512^-1/2 on average, and the difference of two has
    twice a share; six times that covers the largest of all."""
    import torch
    target = ex.Model(layers=2)
    draft = ex.Model(layers=1, like=target)
    prompt = torch.randint(512, (150,), generator=torch.Generator().manual_seed(1)).int().cuda()
    seq, seq_len, steps = ex.decode(target, draft, prompt, 24, 12, gamma=gamma, temperature=0.0)
    assert (seq_len >= 162).all() and 1 <= steps <= 12
    for b in (0, 11, 23):
        toks = seq[b, : int(seq_len[b])]
        logits = plain_logits(target, toks)[149:-1]
        got = logits.gather(1, toks[150:, None].long())[:, 0]
        near = 6 * 2 * 2.0 ** -3 * logits.norm(dim=1) * 512 ** -0.5
        assert (got >= logits.max(1).values - near).all()
    # all samples of a greedy decode are the same
    n = int(seq_len.min())
    assert (seq[:, :n] == seq[0, :n]).all()


def test_sampled_decode_ends(ex):
    import torch
    target = ex.Model(layers=2)
    draft = ex.Model(layers=1, like=target)
    prompt = torch.randint(512, (33,), generator=torch.Generator().manual_seed(2)).int().cuda()
    seq, seq_len, steps = ex.decode(target, draft, prompt, 70, 9, gamma=3, temperature=0.8, top_k=40, top_p=0.9)
    assert ((seq_len >= 42) & (seq_len <= 45)).all()
    assert 2 <= steps <= 8  # 8 tokens behind the first, 1 to 4 a step
    assert ((seq >= 0) & (seq < 512)).all()
