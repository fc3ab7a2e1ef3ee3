"""spec_adjust with slices of 2049 to 8192 tokens, as large batches have them (a CTA's slice
is the vocabulary over 2432 / B), and the first call of a process."""
import subprocess
import sys

import pytest

import conftest
from test_gpu_kv import sv  # noqa: F401

pytestmark = pytest.mark.gpu

HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8}  # half a step of the type, relative

FIRST = """
import sys
import torch
import speculative_decoding_verify_03_gb300 as sv
sv.build()
for B, V in ((76, 262144), (304, 65536), (76, 262112), (608, 32768)):
    x = torch.randn((B, 1, V), device="cuda").to(getattr(torch, sys.argv[1]))
    seq, n = torch.full((B, 4), V - 1, dtype=torch.int32, device="cuda"), torch.full((B,), 4, dtype=torch.int32, device="cuda")
    y = sv.spec_adjust(x, seq, n, frequency=torch.full((B,), 8.0, device="cuda"))
    assert torch.equal(y[:, :, :-1], x[:, :, :-1]) and ((x[:, :, -1] - 32).float() - y[:, :, -1].float()).abs().max() <= 0.25
"""


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_first_call_of_a_process(sv, dtype):  # noqa: F811
    """Slices of 8192 tokens without biases, 48 KB of shared memory beside the kernel's own
    words, before any larger call of the same kernel.  (x - 32 is off by half a step of
    bfloat16 below 64, 0.125, once in the comparison and once in the result.)"""
    run = subprocess.run([sys.executable, "-c", FIRST, dtype], cwd=conftest.ROOT, capture_output=True, text=True, timeout=600)
    assert run.returncode == 0, run.stderr[-2000:]


CASES = [  # B, N, V, biases
    (76, 1, 262144, 0), (76, 1, 262144, 5), (608, 1, 32768, 0), (608, 1, 32768, 9), (304, 1, 50304, 0), (304, 1, 50304, 3),
    (76, 2, 253952, 0), (200, 3, 50304, 7), (2432, 2, 8192, 0), (2432, 9, 8191, 3), (90, 1, 100003, 300), (1216, 33, 8193, 0),
]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("B,N,V,M", CASES)
def test_wide_slices(sv, dtype, B, N, V, M):  # noqa: F811
    """Chains, against the formula in float64.  Tolerance: five roundings in single precision of
    the largest magnitude on the way (division or product, frequency's product, two differences,
    the bias's sum) and one to the type; what no step applies to, bit by bit."""
    import torch
    g = torch.Generator("cuda").manual_seed(B + N + V + M)
    rand = lambda *s: torch.rand(s, generator=g, device="cuda")  # noqa: E731
    token = lambda *s: (rand(*s) ** 3 * (V + 2)).int() - 1  # noqa: E731 (-1 and V now and then: no tokens)
    cap = 24
    x = ((rand(B, N, V) - 0.5) * 12).to(getattr(torch, dtype))
    seq, draft = token(B, cap), token(B, N - 1)
    n = (rand(B) * (cap + 1)).int()
    prompt = (rand(B) * (n + 1)).int().minimum(n)
    gamma = (rand(B) * N).int().clamp(max=N - 1)
    r, f, p = 1 + rand(B), rand(B) - 0.5, 2 * rand(B) - 1
    kw = dict(draft_tokens=draft, prompt_len=prompt, gamma_per_row=gamma, repetition=r, frequency=f, presence=p)
    bias_of = torch.zeros((B, V + 2), dtype=torch.float64, device="cuda")
    biased = torch.zeros((B, V + 2), dtype=torch.bool, device="cuda")
    if M:
        ids, bias = token(B, M), 4 * rand(B, M) - 2
        kw.update(bias_ids=ids, bias=bias)
        for j in range(M):  # the last entry of a token counts
            bias_of.scatter_(1, ids[:, j:j + 1].long() + 1, bias[:, j:j + 1].double())
            biased.scatter_(1, ids[:, j:j + 1].long() + 1, True)
    out, st = sv.spec_adjust(x, seq, n, with_status=True, **kw)
    assert (st == 0).all()
    at, one = torch.arange(cap, device="cuda"), lambda t: t[:, None].double()
    made, seen = (torch.zeros((B, V + 2), dtype=torch.float64, device="cuda") for _ in range(2))
    seen.scatter_add_(1, seq.long() + 1, (at < n[:, None]).double())
    made.scatter_add_(1, seq.long() + 1, ((at < n[:, None]) & (at >= prompt[:, None])).double())
    for i in range(N):
        if i:
            made.scatter_add_(1, draft[:, i - 1:i].long() + 1, torch.ones((B, 1), dtype=torch.float64, device="cuda"))
        m, b = made[:, 1:-1], bias_of[:, 1:-1]
        was = (seen[:, 1:-1] > 0) | (m > 0)
        z = x[:, i].double()
        y = torch.where(was, torch.where(z > 0, z / one(r), z * one(r)), z)
        size = z.abs().maximum(y.abs()) + (m > 0) * (one(f).abs() * m + one(p).abs()) + b.abs()
        y = torch.where(m > 0, y - one(f) * m - one(p), y) + b
        hit = (was | biased[:, 1:-1]) & (gamma >= i)[:, None]
        tol = 5 * 2.0 ** -24 * size + HALF[dtype] * y.abs() * 1.01
        got = out[:, i]
        assert torch.equal(torch.where(hit, x[:, i], got), x[:, i]), i
        far = torch.where(hit, (got.double() - y).abs() / tol.clamp(min=1e-30), torch.zeros_like(y)).max().item()
        assert far <= 1, (i, far)
    assert sv.spec_adjust(x, seq, n, out=x, **kw) is x and torch.equal(x, out)  # in place
