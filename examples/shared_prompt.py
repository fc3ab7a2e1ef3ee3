"""Speculative decoding of many samples of one prompt, with all of the library's steps.

A small random transformer (target) and a smaller one (draft) each keep a
paged e4m3 cache per layer.  The prompt is appended once, to pages that all
samples share; after that every step is

    draft:  gamma + 1 times  spec_kv_append, spec_attend (one query), spec_sample
    target: spec_kv_append, spec_attend (gamma + 1 queries) in each layer
    spec_verify of the drafts, spec_commit of what is accepted

The entries of rejected drafts stay behind kv_len and are overwritten by the
next step's.  Run: python examples/shared_prompt.py [samples] [new tokens]
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verify_03_gb300 as sv  # noqa: E402


class Model:
    """Attention and MLP layers with random weights; the embedding is the output layer too."""

    def __init__(self, vocab=512, width=256, layers=2, n_heads=8, n_kv_heads=2, head_dim=64, seed=0, like=None):
        g = torch.Generator().manual_seed(seed)
        w = lambda *s: (torch.randn(s, generator=g) * s[-2] ** -0.5).cuda()  # noqa: E731
        self.n_heads, self.n_kv_heads, self.head_dim = n_heads, n_kv_heads, head_dim
        self.embed = w(vocab, width) if like is None else like.embed
        self.place = w(4096, width) if like is None else like.place
        self.layers = like.layers[:layers] if like is not None else [
            dict(qkv=w(width, (n_heads + 2 * n_kv_heads) * head_dim), o=w(n_heads * head_dim, width),
                 up=w(width, 2 * width), down=w(2 * width, width)) for _ in range(layers)]

    def norm(self, x):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)

    def split(self, layer, x):
        """q, k and v [B, n, heads, head_dim]: views into the projection."""
        y = (self.norm(x) @ layer["qkv"]).bfloat16().unflatten(-1, (-1, self.head_dim))
        return y.split([self.n_heads, self.n_kv_heads, self.n_kv_heads], 2)

    def rest(self, layer, x, attended):
        x = x + attended.flatten(2).float() @ layer["o"]
        return x + torch.relu(self.norm(x) @ layer["up"]) @ layer["down"]

    def start(self, tokens, places):
        return self.norm(self.embed[tokens.long()]) + 0.1 * self.norm(self.place[places.long()])

    def logits(self, x):
        return (self.norm(x) @ self.norm(self.embed).T * x.shape[-1] ** -0.5).contiguous()


class Server:
    """A model with its caches: a pool of pages per layer, page tables shared by the layers."""

    def __init__(self, model, prompt, samples, room, page_size=16):
        self.model, self.prefix = model, len(prompt)
        shared, each = -(-len(prompt) // page_size), -(-room // page_size)
        self.caches = [sv.KVCache.empty(shared + samples * each, model.n_kv_heads, page_size, model.head_dim)
                       for _ in model.layers]
        ids = torch.arange(shared + samples * each, dtype=torch.int32, device="cuda")
        self.shared, self.own = ids[:shared], ids[shared:].view(samples, each)
        # the prompt, as one sequence whose own pages are the shared ones
        x = model.start(prompt[None], torch.arange(len(prompt), device="cuda")[None])
        zero = torch.zeros(1, dtype=torch.int32, device="cuda")
        for layer, cache in zip(model.layers, self.caches):
            q, k, v = model.split(layer, x)
            sv.spec_kv_append(cache, k, v, self.shared[None], zero)
            x = model.rest(layer, x, sv.spec_attend(q, cache, self.shared[None], zero)[0])
        self.first = model.logits(x[:, -1])

    def step(self, tokens, kv_len):
        """Logits [B, n, vocab] of tokens [B, n] at positions kv_len[b] .. kv_len[b] + n - 1."""
        n, m = tokens.shape[1], self.model
        x = m.start(tokens, kv_len[:, None] + torch.arange(n, device="cuda"))
        for layer, cache in zip(m.layers, self.caches):
            q, k, v = m.split(layer, x)
            sv.spec_kv_append(cache, k, v, self.own, kv_len, prefix_len=self.prefix)
            out, _ = sv.spec_attend(q, cache, self.own, kv_len, prefix_table=self.shared, prefix_len=self.prefix)
            x = m.rest(layer, x, out)
        return m.logits(x)


def decode(target, draft, prompt, samples, new, gamma=4, temperature=1.0, top_k=0, top_p=1.0, seed=0):
    """`new` tokens or up to gamma more for each of `samples` continuations of
    prompt [n] int32: (sequences int32, their lengths, number of steps)."""
    g = torch.Generator("cuda").manual_seed(seed)
    room = new + 2 * gamma + 2
    big, small = (Server(m, prompt, samples, room) for m in (target, draft))
    law = dict(temperature=temperature, top_k=top_k, top_p=top_p)
    end = len(prompt) + new
    seq = torch.zeros((samples, len(prompt) + room), dtype=torch.int32, device="cuda")
    seq[:, :len(prompt)] = prompt
    first = big.first.expand(samples, -1).contiguous()
    seq[:, len(prompt)] = sv.spec_sample(first, torch.rand(samples, generator=g, device="cuda"), **law)
    seq_len = torch.full((samples,), len(prompt) + 1, dtype=torch.int32, device="cuda")
    steps = 0
    while int(seq_len.min()) < end:
        kv_len = seq_len - 1  # the last token's entry is this step's first
        tokens = torch.empty((samples, gamma + 1), dtype=torch.int32, device="cuda")
        tokens[:, 0] = seq.gather(1, kv_len[:, None].long())[:, 0]
        guess = []
        for i in range(gamma + 1):  # the last one for its entry alone
            guess.append(small.step(tokens[:, i:i + 1], kv_len + i)[:, 0])
            if i < gamma:
                u = torch.rand(samples, generator=g, device="cuda")
                tokens[:, i + 1] = sv.spec_sample(guess[i], u, **law)
        uniforms = torch.rand((samples, gamma + 1, 2), generator=g, device="cuda")
        drafts = tokens[:, 1:].contiguous()
        accepted, following = sv.spec_verify(big.step(tokens, kv_len), torch.stack(guess[:gamma], 1), drafts,
                                             uniforms, **law)
        before = seq_len.clone()
        sv.spec_commit(accepted, following, drafts, seq, seq_len)
        seq_len = torch.where(before >= end, before, seq_len)  # samples that are done stand still
        steps += 1
    return seq, seq_len, steps


def main():
    args = [int(a) for a in sys.argv[1:3]]
    samples, new = args + [64, 64][len(args):]
    sv.build()
    target = Model(layers=3)
    draft = Model(layers=2, like=target)
    prompt = torch.randint(512, (1000,), generator=torch.Generator().manual_seed(1)).int().cuda()
    for gamma in (1, 4):
        _, seq_len, steps = decode(target, draft, prompt, samples, new, gamma=gamma, temperature=0.6)
        got = float((seq_len - len(prompt) - 1).float().mean())
        print(f"gamma {gamma}: {steps} steps, {got / steps:.2f} tokens per step and sample")


if __name__ == "__main__":
    main()
