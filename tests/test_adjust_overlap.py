"""Outputs of spec_adjust that share elements with its logits are refused; views of one
tensor that lie between one another's rows are not."""
import ctypes

import numpy as np
import pytest

import speculative_decoding_verify_03_gb300 as m
from speculative_decoding_verify_03_gb300 import tree
from test_gpu_kv import i32, sv  # noqa: F401

P = 1 << 20  # a fake device address: only calls that are refused are made with it


def elements(B, N, V, row, pos):
    return {b * row + i * pos + v for b in range(B) for i in range(N) for v in range(V)}


def call(B, N, V, logits, out, apart, dtype):
    """logits, out: (row stride, position stride); out begins `apart` elements behind logits."""
    size = 2 if dtype else 4
    a = tree.SpecAdjustParams(B=B, gamma_max=N - 1, V=V, dtype=dtype, capacity=10, n_bias=0, logits_row_stride=logits[0],
                              logits_pos_stride=logits[1], out_row_stride=out[0], out_pos_stride=out[1], seq_row_stride=10,
                              seq=P, seq_len=P, draft_tokens=P)
    return m.lib().spec_adjust(P, ctypes.byref(a), P + apart * size, None, None)


@pytest.mark.parametrize("dtype", [0, 1])
def test_overlapping_outputs_refused(dtype):
    m.build()
    assert call(2, 3, 100, (300, 100), (300, 100), 100, dtype) == 1   # one position on
    assert call(2, 3, 100, (300, 100), (300, 100), -599, dtype) == 1  # one element in common
    assert call(2, 3, 100, (600, 200), (600, 200), 101, dtype) == 1   # between the rows, one element too far
    assert call(1, 1, 100, (0, 0), (0, 0), 99, dtype) == 1
    assert call(3, 2, 100, (0, 0), (200, 100), -599, dtype) == 1      # one row of logits for all
    rng, met = np.random.default_rng(dtype), 0
    while met < 1000:
        B, N, V = (int(x) for x in rng.integers(1, 5, 3))
        out = tuple(int(x) for x in rng.integers(V, 40, 2))
        logits = out if rng.random() < 0.5 else tuple(int(x) for x in rng.integers(0, 40, 2))
        apart = int(rng.integers(-150, 150))
        if apart and {x + apart for x in elements(B, N, V, *out)} & elements(B, N, V, *logits):
            assert call(B, N, V, logits, out, apart, dtype) == 1, (B, N, V, logits, out, apart)
            met += 1


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_views_of_one_tensor(sv, dtype):  # noqa: F811
    """Logits and output side by side in a tensor, and turn about by position or by row: the
    output is that of tensors of their own, the logits and all between them stay."""
    import torch
    B, N, V = 3, 4, 517
    dtype = getattr(torch, dtype)
    z = torch.randn((B, N, V), device="cuda").to(dtype)
    seq, n = i32(np.arange(B * 9).reshape(B, 9)), i32([9, 4, 0])
    kw = dict(draft_tokens=i32([[5, 6, 7]] * B), frequency=torch.full((B,), 0.5, device="cuda"))
    want = sv.spec_adjust(z, seq, n, **kw)
    both = torch.empty((2, B, N, V), dtype=dtype, device="cuda")
    turns = (lambda t: t, lambda t: t.transpose(0, 1).contiguous().transpose(0, 1),
             lambda t: t.permute(1, 2, 0, 3).contiguous().permute(2, 0, 1, 3))
    for turn in turns:
        for x, y in ((0, 1), (1, 0)):
            t = turn(both)
            t.fill_(7)
            t[x].copy_(z)
            assert sv.spec_adjust(t[x], seq, n, out=t[y], **kw).data_ptr() == t[y].data_ptr()
            assert torch.equal(t[y], want) and torch.equal(t[x], z)
    # other strides than the logits': rows of the output between rows of positions one after the other
    store = torch.full((B, 2 * N * V), 7.0, dtype=dtype, device="cuda")
    x, y = store[:, :N * V].view(B, N, V), store[:, N * V:].unflatten(1, (N, V))[:, :, :V - 9]
    x.copy_(z)
    sv.spec_adjust(x[:, :, :V - 9], seq, n, out=y, **kw)
    assert torch.equal(y, want[:, :, :V - 9]) and torch.equal(x, z) and (store[:, N * V:].unflatten(1, (N, V))[:, :, V - 9:] == 7).all()
    wide = torch.full((B, 3 * N, V), 7.0, dtype=dtype, device="cuda")  # positions 0, 1, .. and N, N + 2, ..
    x, y = wide[:, :N], wide[:, N::2]
    x.copy_(z)
    sv.spec_adjust(x, seq, n, out=y, **kw)
    assert torch.equal(y, want) and torch.equal(x, z) and (wide[:, N + 1::2] == 7).all()
    for y in (wide[:, 1:N + 1], wide[:, 3:2 * N + 3:2]):
        with pytest.raises(sv.SpecError):
            sv.spec_adjust(x, seq, n, out=y, **kw)
