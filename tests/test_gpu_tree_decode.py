"""Greedy decoding with drafted trees, with all of the library's steps for them: page
tables that grow, masks, attention, adjusted logits, the accepting walk, the
cache's compaction, a fork on the way.  What comes out is what the model without
any cache chooses, up to the rounding of the cache."""
import numpy as np
import pytest

import tree_ref
from test_gpu_example import ex, plain_logits  # noqa: F401
from test_gpu_kv import i32

pytestmark = pytest.mark.gpu

PAGE, V, N, PENALTY = 16, 512, 10, 1.3


def adjusted(logits, tokens, prompt):
    """Float64 logits [V] behind tokens, with the penalties of this test."""
    return tree_ref.adjust(logits, tokens, prompt, [], PENALTY, 0.25, 0.125, [(7, -3.0)], None)[0]


def greedy(ex, model, tokens, prompt, n):  # noqa: F811
    """The model's own next n tokens, without a cache."""
    out = list(tokens)
    for _ in range(n):
        z = plain_logits(model, i32(out))[-1].cpu().numpy()
        out.append(int(adjusted(z, out, prompt).argmax()))
    return out[len(tokens):]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_decode_with_trees(ex, fmt):  # noqa: F811
    import torch
    sv, rng = ex.sv, np.random.default_rng(3)
    model = ex.Model(layers=2)
    prompts = [rng.integers(0, V, n).tolist() for n in (40, 5, 77)]
    B, cap, wide = 4, 200, 14  # the last row is a fork's
    dtype = torch.bfloat16 if fmt == "bf16" else torch.float8_e4m3fn
    caches = [sv.KVCache.empty(60, model.n_kv_heads, PAGE, model.head_dim, dtype=dtype) for _ in model.layers]
    refs, table, held = i32(np.zeros(60)), i32(np.full((B, wide), -1)), i32(np.zeros(B))
    seq = torch.zeros((B, cap), dtype=torch.int32, device="cuda")
    for b, p in enumerate(prompts):
        seq[b, :len(p)] = i32(p)
    seq_len, prompt_len = i32([len(p) for p in prompts] + [0]), i32([len(p) for p in prompts] + [0])
    pens = [torch.full((B,), x, device="cuda") for x in (PENALTY, 0.125, 0.25)]
    ids, bias = i32([[7]] * B), torch.full((B, 1), -3.0, device="cuda")

    def forward(tokens, places, kv_len, attend):
        x = model.start(tokens, places)
        for layer, cache in zip(model.layers, caches):
            q, k, v = model.split(layer, x)
            sv.spec_kv_append(cache, k[:len(kv_len)], v[:len(kv_len)], table[:len(kv_len)], kv_len)
            x = model.rest(layer, x, attend(q, cache))
        return model.logits(x)

    # the prompts but for their last tokens, one after the other
    sv.spec_kv_resize(refs, table, held, seq_len - 1, 0, PAGE)
    for b, p in enumerate(prompts):
        zero, one = i32([0]), table[b:b + 1]
        x = model.start(seq[b:b + 1, :len(p) - 1], torch.arange(len(p) - 1, device="cuda")[None])
        for layer, cache in zip(model.layers, caches):
            q, k, v = model.split(layer, x)
            sv.spec_kv_append(cache, k, v, one, zero)
            x = model.rest(layer, x, sv.spec_attend(q, cache, one, zero)[0])
    kv_len = seq_len - 1  # the fork's row: -1, nothing held
    taken = np.zeros(B, int)
    for step in range(7):
        if step == 4:  # the last row becomes a second sample of row 0
            copies = sv.spec_kv_fork(refs, table, held, kv_len, i32([0]), i32([3]), PAGE)
            for cache in caches:
                sv.spec_kv_copy(cache, copies)
            seq[3], seq_len[3], prompt_len[3] = seq[0], seq_len[0], prompt_len[0]
            forked = int(seq_len[0])
        n = B if step >= 4 else B - 1
        assert (sv.spec_kv_resize(refs, table, held, kv_len, N, PAGE, with_status=True)[:n].cpu().numpy() == 0).all()
        parents = tree_ref.random_parents(rng, n, N - 1)
        draft = rng.integers(0, V, (n, N - 1))
        for b in range(n):  # a way through the tree that the model itself would go
            way = tree_ref.ancestors(parents[b], N)[int(rng.integers(1, N))][1:]
            # alike drafts under one parent may lead elsewhere: keep the others off the way's tokens
            own = greedy(ex, model, seq[b, :int(seq_len[b])].tolist(), len(prompts[b % 3]), len(way))
            draft[b][np.isin(draft[b], own)] = V - 1
            for j, t in zip(way, own):
                draft[b, j - 1] = t
        if n == B:
            parents[3], draft[3] = parents[0], draft[0]
        P, D, L = i32(parents), i32(draft), kv_len[:n].contiguous()
        mask, depth = sv.spec_tree_mask(P)
        root = seq[:n].gather(1, L[:, None].long())
        logits = forward(torch.cat([root, D], 1), L[:, None] + depth, L,
                         lambda q, cache: sv.spec_attend_tree(q, cache, table[:n], L, mask)[0])
        rows = lambda t: t[:n].contiguous()  # noqa: E731
        z = sv.spec_adjust(logits, seq[:n], rows(seq_len), D, mask, rows(prompt_len), *(rows(t) for t in pens), rows(ids),
                           rows(bias))
        target = sv.spec_sample(z.view(n * N, V), torch.rand(n * N, device="cuda"), 0.0).view(n, N)
        accepted, following, path, tokens, st = sv.spec_tree_accept(target, D, P, with_status=True)
        assert (st == 0).all()
        for cache in caches:
            assert (sv.spec_kv_compact(cache, table[:n], L, path, accepted, with_status=True) == 0).all()
        length = rows(seq_len)
        after, _ = sv.spec_commit(accepted, following, tokens, seq[:n], length)
        seq_len[:n], kv_len[:n] = length, after
        taken[:n] += accepted.cpu().numpy()
    # a bfloat16 entry, query and output are each off by up to 2^-8 of themselves, an
    # e4m3 entry by 2^-4: 2^-6 and 2^-3 of a layer's output and the residual stream with
    # it, twice that for two layers; a logit has a share of 512^-1/2 of the logits' norm
    # on average, the difference of two twice a share; six times that covers the
    # largest, and the penalty's factor
    share = 6 * 2 * 2 * (2.0 ** -6 if fmt == "bf16" else 2.0 ** -3) * V ** -0.5 * PENALTY
    for b in range(B):
        toks, first = seq[b, :int(seq_len[b])].tolist(), len(prompts[b % 3])
        logits = plain_logits(model, i32(toks)).cpu().numpy()
        if b < 3:
            assert len(toks) - first == 7 + taken[b]  # one of its own draws a step, and the accepted drafts
        for i in range(first, len(toks)):
            y = adjusted(logits[i - 1], toks[:i], first)
            assert y[toks[i]] >= y.max() - share * np.linalg.norm(logits[i - 1]), (b, i)
    assert taken[:3].sum() >= 7  # the ways that the model itself would go are gone, most of the time
    m = min(int(seq_len[0]), int(seq_len[3]))
    assert (seq[3, :m] == seq[0, :m]).all() and m > forked
    # all pages come back
    sv.spec_kv_resize(refs, table, held, i32([-1] * B), 0, PAGE)
    assert (refs == 0).all() and (held == 0).all()
