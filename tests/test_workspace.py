"""The workspaces that the sampler's calls make for themselves, on the CPU."""
import torch

import speculative_decoding_verify_03_gb300 as sv
from test_kv_ref import FakeGpu, Stream


def test_workspaces_are_the_calls_own(monkeypatch):
    """Neither shared by calls whose launches may come between one another's, nor
    replaced under a captured graph; the memory is the launch stream's."""
    sv.build()
    gpu = FakeGpu(monkeypatch)
    monkeypatch.setattr(torch, "zeros", torch.empty)
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    P = sv.SpecParams(B=8, gamma_max=4, V=50304, dtype=0, temperature=1.0, top_p=0.9, top_k=50,
                      target_pos_stride=50304, target_row_stride=5 * 50304, draft_pos_stride=50304,
                      draft_row_stride=4 * 50304)
    a, b = (sv.auto_workspace(P, "cuda:0", s) for s in (None, None))
    assert a.data_ptr() != b.data_ptr() and a.numel() == b.numel() >= sv.workspace_bytes(P)
    c = sv.auto_workspace(P, "cuda:0", Stream(77))
    assert [t.stream for t in (a, b, c)] == [0, 0, 77] and len(gpu.made) == 3
