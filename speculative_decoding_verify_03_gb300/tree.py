"""Trees of drafted tokens and the logits that they are judged by: the binding of
include/spec_tree.h."""
from __future__ import annotations

import ctypes

import torch

from .kv import _bf16, _byref, _check, _elsewhere, _f32, _i32, _int32, _lib, _on, _ptr, _raw_stream, _status

TREE_MAX = 512
ROW_BAD_TREE, ROW_BAD_PENALTY = 1 << 10, 1 << 11


class SpecAdjustParams(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("B", "gamma_max", "V", "dtype", "capacity", "n_bias")] +
                [(n, ctypes.c_int64) for n in ("logits_row_stride", "logits_pos_stride", "out_row_stride",
                                               "out_pos_stride", "seq_row_stride", "allowed_row_stride",
                                               "allowed_pos_stride")] +
                [(n, ctypes.c_void_p) for n in ("seq", "seq_len", "prompt_len", "draft_tokens", "tree_mask",
                                                "gamma_per_row", "repetition", "presence", "frequency", "bias_ids",
                                                "bias", "allowed")])


def _table(name, t, shape, device):
    """A contiguous int32 tensor of this shape on the device: its address (0 without elements)."""
    if t.dtype is not _i32:
        raise TypeError(f"{name} must be int32")
    if t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {list(shape)} on {device}")
    return t.data_ptr()


def _float(name, t, shape, device):
    """As _table, float32."""
    if t.dtype is not _f32:
        raise TypeError(f"{name} must be float32")
    if t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {list(shape)} on {device}")
    return t.data_ptr()


def spec_tree_mask(parents, gamma_per_row=None, with_status=False, stream=None):
    """What the nodes of drafted trees see (see spec_tree_mask in
    include/spec_tree.h): parents [B, gamma_max] int32, parents[b, j - 1] < j the
    parent of node j = 1 .. gamma_b, node 0 the root.  Returns (mask [B,
    gamma_max + 1, ceil((gamma_max + 1) / 32)] int32, bit j & 31 of word j >> 5
    of row i set if node j is node i or an ancestor of it, depth [B, gamma_max +
    1] int32), and row_status [B] when with_status."""
    dev = parents.device
    if parents.dim() != 2:
        raise ValueError("parents must be [B, gamma_max]")
    B, G = parents.shape
    up = _table("parents", parents, (B, G), dev)
    gam = None if gamma_per_row is None else _int32("gamma_per_row", gamma_per_row, B, dev)
    if _elsewhere(stream, dev):
        return _on(stream, dev, spec_tree_mask, parents, gamma_per_row, with_status)
    mask = torch.empty(B, G + 1, (G + 32) // 32, dtype=_i32, device=dev)
    depth = torch.empty(B, G + 1, dtype=_i32, device=dev)
    st = _status(with_status, B, dev)
    code = _lib().spec_tree_mask(B, G, up, gam, mask.data_ptr(), depth.data_ptr(), _ptr(st), _raw_stream(dev.index))
    if code:
        _check(code)
    return (mask, depth, st) if with_status else (mask, depth)


def spec_tree_accept(target_tokens, draft_tokens, parents, gamma_per_row=None, with_status=False, stream=None):
    """The walk along the target's draws (see spec_tree_accept in
    include/spec_tree.h): target_tokens [B, gamma_max + 1] int32, the token drawn
    at each node, draft_tokens and parents [B, gamma_max] int32.  Returns
    (accepted_len [B], next_token [B], path [B, gamma_max + 1], path_tokens [B,
    gamma_max]) int32, and row_status [B] when with_status: path goes to
    spec_kv_compact; accepted_len, next_token and path_tokens go to spec_commit."""
    dev = target_tokens.device
    if target_tokens.dim() != 2 or target_tokens.shape[1] < 1:
        raise ValueError("target_tokens must be [B, gamma_max + 1]")
    B, N = target_tokens.shape
    tgt = _table("target_tokens", target_tokens, (B, N), dev)
    tok = _table("draft_tokens", draft_tokens, (B, N - 1), dev)
    up = _table("parents", parents, (B, N - 1), dev)
    gam = None if gamma_per_row is None else _int32("gamma_per_row", gamma_per_row, B, dev)
    if _elsewhere(stream, dev):
        return _on(stream, dev, spec_tree_accept, target_tokens, draft_tokens, parents, gamma_per_row, with_status)
    acc = torch.empty(B, dtype=_i32, device=dev)
    nxt = torch.empty(B, dtype=_i32, device=dev)
    path = torch.empty(B, N, dtype=_i32, device=dev)  # sizes one by one: 1 us less each than a shape
    tokens = torch.empty(B, N - 1, dtype=_i32, device=dev)
    st = _status(with_status, B, dev)
    code = _lib().spec_tree_accept(B, N - 1, tgt, tok, up, gam, acc.data_ptr(), nxt.data_ptr(), path.data_ptr(),
                                   tokens.data_ptr(), _ptr(st), _raw_stream(dev.index))
    if code:
        _check(code)
    return (acc, nxt, path, tokens, st) if with_status else (acc, nxt, path, tokens)


def spec_adjust(logits, seq, seq_len, draft_tokens=None, tree_mask=None, prompt_len=None, repetition=None,
                presence=None, frequency=None, bias_ids=None, bias=None, allowed=None, gamma_per_row=None, out=None,
                with_status=False, stream=None):
    """Penalties, biases and a grammar's mask on the logits of a step (see
    spec_adjust in include/spec_tree.h).  logits [B, gamma_max + 1, V] float32 or
    bfloat16 (contiguous vocabulary); position i comes behind seq[b,
    :seq_len[b]] ([B, capacity] int32, its first prompt_len[b] tokens the prompt)
    and behind the drafts on the way to node i (draft_tokens [B, gamma_max]
    int32; tree_mask of spec_tree_mask, or None: a chain, drafts 0 .. i - 1).
    repetition, presence, frequency [B] float32; bias_ids [B, n] int32 and bias
    [B, n] float32; allowed [B, gamma_max + 1, ceil(V / 32)] int32, bit v & 31 of
    word v >> 5 set if v is allowed (axes of stride 0 are fine: one mask for
    all).  Each is optional.  out: None (a new tensor), logits (in place) or a
    tensor of its shape and type that does not overlap it.  Returns out, and
    row_status [B] when with_status."""
    dev = logits.device
    if logits.dim() != 3 or logits.shape[1] < 1 or logits.shape[2] < 1:
        raise ValueError("logits must be [B, gamma_max + 1, V]")
    if logits.dtype is not _f32 and logits.dtype is not _bf16:
        raise TypeError(f"logits must be float32 or bfloat16, got {logits.dtype}")
    B, N, V = logits.shape
    in_row, in_pos, one = logits.stride()
    if one != 1 and V > 1:
        raise ValueError("the vocabulary axis must be contiguous")
    if out is not None and (out.shape != logits.shape or out.dtype != logits.dtype or out.device != dev or
                            (out.stride(2) != 1 and V > 1)):
        raise ValueError("out must be of the logits' shape, type and device, its vocabulary axis contiguous")
    if seq.dtype is not _i32:
        raise TypeError("seq must be int32")
    if seq.dim() != 2 or seq.shape[0] != B or seq.device != dev or (B and seq.shape[1] > 1 and seq.stride(1) != 1):
        raise ValueError(f"seq must be [{B}, capacity] on {dev} with contiguous rows")
    if N > 1 and draft_tokens is None:
        raise ValueError("draft_tokens must be given where there are drafts")
    if (bias_ids is None) != (bias is None):
        raise ValueError("bias_ids and bias go together")
    lens = _int32("seq_len", seq_len, B, dev)
    prompt = None if prompt_len is None else _int32("prompt_len", prompt_len, B, dev)
    gam = None if gamma_per_row is None else _int32("gamma_per_row", gamma_per_row, B, dev)
    drafts = None if draft_tokens is None else _table("draft_tokens", draft_tokens, (B, N - 1), dev)
    tree = None if tree_mask is None else _table("tree_mask", tree_mask, (B, N, (N + 31) // 32), dev)
    rep = None if repetition is None else _float("repetition", repetition, (B,), dev)
    pres = None if presence is None else _float("presence", presence, (B,), dev)
    freq = None if frequency is None else _float("frequency", frequency, (B,), dev)
    n_bias, ids, values = 0, None, None
    if bias is not None:
        n_bias = bias.shape[1] if bias.dim() == 2 else -1
        values = _float("bias", bias, (B, n_bias), dev)
        ids = _table("bias_ids", bias_ids, (B, n_bias), dev)
    words, allowed_row, allowed_pos = None, 0, 0
    if allowed is not None:
        if allowed.dtype is not _i32:
            raise TypeError("allowed must be int32")
        n = (V + 31) // 32
        allowed_row, allowed_pos, one = allowed.stride() if allowed.dim() == 3 else (0, 0, 0)
        if allowed.shape != (B, N, n) or allowed.device != dev or (n > 1 and one != 1):
            raise ValueError(f"allowed must be [{B}, {N}, {n}] on {dev} with contiguous words")
        words = allowed.data_ptr()
    if _elsewhere(stream, dev):
        return _on(stream, dev, spec_adjust, logits, seq, seq_len, draft_tokens, tree_mask, prompt_len, repetition,
                   presence, frequency, bias_ids, bias, allowed, gamma_per_row, out, with_status)
    if out is None:
        out = torch.empty(B, N, V, dtype=logits.dtype, device=dev)
    row, pos, _ = out.stride()
    P = SpecAdjustParams(B, N - 1, V, 0 if logits.dtype is _f32 else 1, seq.shape[1], n_bias, in_row, in_pos, row, pos,
                         seq.stride(0) if B > 1 else seq.shape[1], allowed_row, allowed_pos, seq.data_ptr(), lens, prompt,
                         drafts, tree, gam, rep, pres, freq, ids, values, words)
    st = _status(with_status, B, dev)
    code = _lib().spec_adjust(logits.data_ptr(), _byref(P), out.data_ptr(), _ptr(st), _raw_stream(dev.index))
    if code:
        _check(code)
    return (out, st) if with_status else out
