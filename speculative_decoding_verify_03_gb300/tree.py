"""Trees of drafted tokens and the logits that they are judged by: the binding of
include/spec_tree.h."""
from __future__ import annotations

import ctypes

from .kv import _native, _on

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


def spec_tree_mask(parents, gamma_per_row=None, with_status=False, stream=None):
    """What the nodes of drafted trees see (see spec_tree_mask in
    include/spec_tree.h): parents [B, gamma_max] int32, parents[b, j - 1] < j the
    parent of node j = 1 .. gamma_b, node 0 the root.  Returns (mask [B,
    gamma_max + 1, ceil((gamma_max + 1) / 32)] int32, bit j & 31 of word j >> 5
    of row i set if node j is node i or an ancestor of it, depth [B, gamma_max +
    1] int32), and row_status [B] when with_status."""
    if stream is not None:
        return _on(stream, parents.device, spec_tree_mask, parents, gamma_per_row, with_status)
    return _native().tree_mask(parents, gamma_per_row, with_status)


def spec_tree_accept(target_tokens, draft_tokens, parents, gamma_per_row=None, with_status=False, stream=None):
    """The walk along the target's draws (see spec_tree_accept in
    include/spec_tree.h): target_tokens [B, gamma_max + 1] int32, the token drawn
    at each node, draft_tokens and parents [B, gamma_max] int32.  Returns
    (accepted_len [B], next_token [B], path [B, gamma_max + 1], path_tokens [B,
    gamma_max]) int32, and row_status [B] when with_status: path goes to
    spec_kv_compact; accepted_len, next_token and path_tokens go to spec_commit."""
    if stream is not None:
        return _on(stream, target_tokens.device, spec_tree_accept, target_tokens, draft_tokens, parents, gamma_per_row,
                   with_status)
    return _native().tree_accept(target_tokens, draft_tokens, parents, gamma_per_row, with_status)


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
    if stream is not None:
        return _on(stream, logits.device, spec_adjust, logits, seq, seq_len, draft_tokens, tree_mask, prompt_len,
                   repetition, presence, frequency, bias_ids, bias, allowed, gamma_per_row, out, with_status)
    return _native().adjust(logits, seq, seq_len, draft_tokens, tree_mask, prompt_len, repetition, presence, frequency,
                            bias_ids, bias, allowed, gamma_per_row, out, with_status)
