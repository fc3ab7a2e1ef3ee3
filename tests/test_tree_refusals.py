"""What the operators for trees, page tables and adjusted logits refuse, on the
CPU: arguments are checked before any launch; and the references that the GPU
tests compare with, on cases worked out by hand."""
import ctypes

import numpy as np
import pytest
import torch

import speculative_decoding_verify_03_gb300 as sv
import tree_ref
from speculative_decoding_verify_03_gb300 import kv, tree
from test_kv_ref import BAD, FakeGpu, OnGpu, Stream, _batch, _cache

P = 1 << 20  # a fake, never dereferenced, device address


@pytest.fixture(scope="module")
def L():
    sv.build()
    return sv.lib()


# -------------------------------------------------------------- the references
def test_tree_reference():
    p = np.array([[0, 0, 1, 3]], np.int32)
    bits, depth = tree_ref.sees(p, [4])
    assert depth.tolist() == [[0, 1, 1, 2, 3]]
    assert tree_ref.words(bits)[0, :, 0].tolist() == [1, 3, 5, 11, 27]
    assert tree_ref.accept([7, 8, 9, 6, 5], [7, 7, 8, 6], p[0], 4) == (3, 5, [0, 1, 3, 4])
    assert tree_ref.accept([7, 8, 9, 6, 5], [7, 7, 8, 6], p[0], 2) == (1, 8, [0, 1])
    assert tree_ref.words(np.ones((1, 33), bool)).tolist() == [[-1, 1]]


def test_pool_reference():
    pool = tree_ref.Pool([0] * 6, [[-1] * 4] * 3, [0, 0, 0], 16)
    assert pool.resize([20, 1, -1], 0) == [0, 0, 0] and pool.table[0][:2] == [0, 1] and pool.table[1][0] == 2
    kv_len = [20, 1, -1]
    assert pool.fork(kv_len, [0], [2]) == ([[1, 3, 4]], [0]) and pool.refs == [2, 1, 1, 1, 0, 0] and kv_len == [20, 1, 20]
    assert pool.resize([-1, 50, 20], 0) == [0, 0, 0]  # page 1 comes back, page 0 is shared
    assert pool.table[1][:4] == [2, 1, 4, 5] and pool.refs == [1] * 6
    assert pool.resize([1, 50, 20], 0)[0] == tree_ref.NO_PAGES


def test_adjust_reference():
    y, _, hit = tree_ref.adjust(np.array([2.0, -2.0, 1.0, 0.5]), [0, 1, 1], 1, [1], 2.0, 0.5, 1.0, [(2, 1.0), (2, 3.0)], None)
    assert y.tolist() == [1.0, -4.0 - 1.5 - 1.0, 4.0, 0.5] and hit.tolist() == [True, True, True, False]


# ------------------------------------------------------------------ the C ABI
@pytest.mark.parametrize("cache,batch,code", BAD)
def test_descriptors_refused(L, cache, batch, code):
    c, b = ctypes.byref(_cache(**cache)), ctypes.byref(_batch(**batch))
    s = ctypes.byref((ctypes.c_int64 * 3)(64 * 8 * 4, 64 * 8, 64))
    assert L.spec_attend_tree(c, b, P, P, 16, s, 0.1, P, P, None, P, 1 << 30, None) == code
    assert L.spec_kv_compact(c, b, P, P, None, None) == code
    if not batch and cache != dict(n_pages=-1):
        assert L.spec_kv_copy(c, P, 3, None) == code


def test_attend_tree_arguments(L):
    c, b = ctypes.byref(_cache()), ctypes.byref(_batch())
    s = ctypes.byref((ctypes.c_int64 * 3)(64 * 8 * 4, 64 * 8, 64))
    neg = ctypes.byref((ctypes.c_int64 * 3)(64 * 8 * 4, -64 * 8, 64))
    att = lambda b=b, m=P, q=P, h=16, st=s, sc=0.1, o=P, l=P, ws=P, n=1 << 30: L.spec_attend_tree(  # noqa: E731
        c, b, m, q, h, st, sc, o, l, None, ws, n, None)
    assert att(m=None) == att(m=P + 2) == att(q=None) == att(h=0) == att(h=12) == att(st=None) == att(st=neg) == 1
    assert att(sc=float("nan")) == att(sc=-1.0) == att(o=None) == att(q=P + 1) == att(o=P + 2) == att(l=P + 2) == 1
    need = L.spec_attend_tree_workspace_size(c, b, 16)
    assert need > 0 and att(ws=None) == att(ws=P + 16) == att(n=need - 1) == 3
    assert att(b=ctypes.byref(_batch(gamma_max=512))) == 2 and att(b=ctypes.byref(_batch(gamma_max=512, B=0))) == 2
    assert L.spec_attend_tree_workspace_size(c, ctypes.byref(_batch(gamma_max=512)), 16) == 0
    assert L.spec_attend_tree_workspace_size(c, ctypes.byref(_batch(gamma_max=511)), 16) > 0
    assert att(b=ctypes.byref(_batch(B=0)), m=None) == 0


def test_compact_and_copy_arguments(L):
    c, b = ctypes.byref(_cache()), ctypes.byref(_batch())
    assert L.spec_kv_compact(c, b, None, P, None, None) == L.spec_kv_compact(c, b, P, None, None, None) == 1
    assert L.spec_kv_compact(c, b, P + 2, P, None, None) == L.spec_kv_compact(None, b, P, P, None, None) == 1
    assert L.spec_kv_compact(c, ctypes.byref(_batch(gamma_max=512)), P, P, None, None) == 2
    assert L.spec_kv_compact(c, ctypes.byref(_batch(B=0)), None, None, None, None) == 0
    assert L.spec_kv_copy(c, None, 1, None) == L.spec_kv_copy(c, P + 1, 1, None) == L.spec_kv_copy(c, P, -1, None) == 1
    assert L.spec_kv_copy(None, P, 1, None) == 1 and L.spec_kv_copy(c, P, (1 << 20) + 1, None) == 2
    assert L.spec_kv_copy(c, None, 0, None) == 0
    assert L.spec_kv_compact(c, b, P, P, P + 2, None) == 1  # row_status


def _pool(**kw):
    f = dict(B=2, max_pages=4, n_pages=10, page_size=16, prefix_len=0, table_row_stride=4, refs=P, table=P, held=P)
    f.update(kw)
    return ctypes.byref(kv.SpecKvPool(**f))


POOLS = [(dict(B=-1), 1), (dict(max_pages=-1), 1), (dict(n_pages=-1), 1), (dict(page_size=0), 1), (dict(page_size=24), 2),
         (dict(prefix_len=-1), 1), (dict(table_row_stride=3), 1), (dict(B=4097), 2), (dict(refs=None), 1),
         (dict(table=None), 1), (dict(held=None), 1), (dict(refs=P + 2), 1), (dict(max_pages=1 << 27, table_row_stride=1 << 27), 2)]


@pytest.mark.parametrize("pool,code", POOLS)
def test_pools_refused(L, pool, code):
    assert L.spec_kv_resize(_pool(**pool), P, 1, None, None) == code
    assert L.spec_kv_fork(_pool(**pool), P, P, P, 1, P, None, None) == code


def test_pool_arguments(L):
    assert L.spec_kv_resize(None, P, 1, None, None) == L.spec_kv_resize(_pool(), None, 1, None, None) == 1
    assert L.spec_kv_resize(_pool(), P, -1, None, None) == 1 and L.spec_kv_resize(_pool(), P + 1, 1, None, None) == 1
    assert L.spec_kv_resize(_pool(), P, (1 << 30) + 1, None, None) == 2
    assert L.spec_kv_resize(_pool(B=0, refs=None, table=None, held=None), None, 1, None, None) == 0
    fork = lambda len_=P, s=P, d=P, n=1, c=P: L.spec_kv_fork(_pool(), len_, s, d, n, c, None, None)  # noqa: E731
    assert fork(len_=None) == fork(s=None) == fork(d=None) == fork(c=None) == fork(n=-1) == fork(s=P + 1) == 1
    assert fork(n=4097) == 2 and fork(n=0, s=None, d=None, c=None) == 0
    assert L.spec_kv_resize(_pool(), P, 1, P + 1, None) == L.spec_kv_fork(_pool(), P, P, P, 1, P, P + 2, None) == 1  # status


def test_tree_arguments(L):
    mask = lambda B=2, G=3, p=P, g=None, m=P, d=P: L.spec_tree_mask(B, G, p, g, m, d, None, None)  # noqa: E731
    assert mask(B=-1) == mask(G=-1) == mask(p=None) == mask(m=None) == mask(p=P + 1) == mask(d=P + 2) == mask(g=P + 1) == 1
    assert mask(G=512) == 2 and mask(B=0, m=None) == 0
    acc = lambda B=2, G=3, t=P, d=P, p=P, a=P, n=P, w=P: L.spec_tree_accept(  # noqa: E731
        B, G, t, d, p, None, a, n, w, None, None, None)
    assert acc(B=-1) == acc(G=-1) == acc(t=None) == acc(d=None) == acc(p=None) == acc(a=None) == acc(n=None) == acc(w=P + 1) == 1
    assert acc(G=512) == 2 and acc(B=0, t=None) == 0


def _adjust(L, logits=P, out=2 * P, **kw):
    f = dict(B=2, gamma_max=1, V=100, dtype=0, capacity=10, n_bias=0, logits_row_stride=200, logits_pos_stride=100,
             out_row_stride=200, out_pos_stride=100, seq_row_stride=10, seq=P, seq_len=P, draft_tokens=P)
    f.update(kw)
    return L.spec_adjust(logits, ctypes.byref(tree.SpecAdjustParams(**f)), out, None, None)


@pytest.mark.parametrize("bad,code", [
    (dict(B=-1), 1), (dict(gamma_max=-1), 1), (dict(V=0), 1), (dict(V=(1 << 24) + 1), 1), (dict(dtype=2), 1),
    (dict(capacity=-1), 1), (dict(n_bias=-1), 1), (dict(n_bias=3), 1), (dict(n_bias=3, bias=P), 1), (dict(seq=None), 1),
    (dict(seq_len=None), 1), (dict(draft_tokens=None), 1), (dict(logits=None), 1), (dict(out=None), 1), (dict(logits=P + 2), 1),
    (dict(out=2 * P + 1), 1), (dict(out_pos_stride=99), 1), (dict(out_row_stride=99), 1), (dict(logits_pos_stride=-1), 1),
    (dict(seq_row_stride=-1), 1), (dict(allowed=P, allowed_row_stride=-1), 1), (dict(allowed=P + 2), 1), (dict(tree_mask=P + 1), 1),
    (dict(out=P, logits_pos_stride=200, logits_row_stride=400), 1), (dict(n_bias=65535, bias=P, bias_ids=P), 2),
    (dict(gamma_max=512, tree_mask=P), 2), (dict(gamma_max=5000, presence=P), 2), (dict(gamma_max=1 << 20), 2), (dict(B=0), 0),
    (dict(capacity=1 << 30), 2), (dict(out_row_stride=100, out_pos_stride=100), 1), (dict(out_row_stride=100, out_pos_stride=199), 1),
    (dict(out_row_stride=199, out_pos_stride=100), 1), (dict(out_row_stride=100, out_pos_stride=200, B=0), 0),
])
def test_adjust_arguments(L, bad, code):
    assert _adjust(L, **bad) == code
    assert L.spec_adjust(P, None, P, None, None) == 1


# ---------------------------------------------------------------- the binding
def test_binding_refuses():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    f = lambda *s: torch.zeros(s)  # noqa: E731
    c = sv.KVCache(z(3, 2, 16, 64), z(3, 2, 16, 64))
    with pytest.raises(TypeError):
        sv.spec_attend_tree(z(2, 3, 4, 64), c, i(2, 4), i(2), None)
    for m in (i(2, 3, 2), i(2, 2, 1), i(3, 3, 1), i(2, 3, 2)[:, :, :1]):
        with pytest.raises(ValueError):
            sv.spec_attend_tree(z(2, 3, 4, 64), c, i(2, 4), i(2), m)
    with pytest.raises(TypeError):
        sv.spec_attend_tree(z(2, 3, 4, 64), c, i(2, 4), i(2), i(2, 3, 1).long())
    good = dict(q=z(2, 3, 4, 64), page_table=i(2, 4), kv_len=i(2), mask=i(2, 3, 1))
    for bad in (dict(q=z(2, 3, 3, 64)), dict(q=z(2, 3, 4, 80)), dict(q=z(3, 3, 4, 64)), dict(q=z(2, 0, 4, 64), mask=i(2, 0, 0)),
                dict(q=z(2, 3, 64, 4).transpose(2, 3)), dict(page_table=i(3, 4)), dict(page_table=i(4, 2).t()), dict(kv_len=i(2, 1)),
                dict(gamma_per_row=i(3)), dict(prefix_len=3), dict(prefix_len=17, prefix_table=i(1))):
        with pytest.raises(ValueError):
            sv.spec_attend_tree(cache=c, **dict(good, **bad))
    for bad in (dict(q=z(2, 3, 4, 64).float()), dict(page_table=i(2, 4).long()), dict(scale="1"), dict(prefix_table=[0], prefix_len=1)):
        with pytest.raises(TypeError):
            sv.spec_attend_tree(cache=c, **dict(good, **bad))
    for bad in (dict(path=i(3, 4)), dict(path=i(4, 2).t()), dict(accepted_len=i(3)), dict(kv_len=i(2, 1)), dict(path=i(2, 0))):
        a = dict(page_table=i(2, 4), kv_len=i(2), path=i(2, 4), accepted_len=i(2))
        a.update(bad)
        with pytest.raises(ValueError):
            sv.spec_kv_compact(c, **a)
    for bad in (i(3), i(2, 4), i(3, 2).t()):
        with pytest.raises(ValueError):
            sv.spec_kv_copy(c, bad)
    for bad in (dict(held=i(3)), dict(page_table=i(2)), dict(page_table=i(4, 2).t()), dict(refs=i(2, 5)), dict(kv_len=i(1)),
                dict(page_table=i(1, 4).expand(2, 4))):
        a = dict(refs=i(5), page_table=i(2, 4), held=i(2), kv_len=i(2))
        a.update(bad)
        with pytest.raises(ValueError):
            sv.spec_kv_resize(**a, n_step=1, page_size=16)
        with pytest.raises(ValueError):
            sv.spec_kv_fork(**a, src=i(1), dst=i(1), page_size=16)
    with pytest.raises(ValueError):
        sv.spec_kv_fork(i(5), i(2, 4), i(2), i(2), i(1), i(2), 16)
    with pytest.raises(TypeError):
        sv.spec_tree_mask(f(2, 3))
    with pytest.raises(ValueError):
        sv.spec_tree_mask(i(3, 2).t())
    with pytest.raises(ValueError):
        sv.spec_tree_accept(i(2, 4), i(2, 4), i(2, 3))
    with pytest.raises(ValueError):
        sv.spec_tree_accept(i(2, 0), i(2, 0), i(2, 0))
    good = dict(logits=f(2, 3, 50), seq=i(2, 9), seq_len=i(2), draft_tokens=i(2, 2))
    for bad in (dict(logits=f(2, 50)), dict(logits=f(2, 50, 3).transpose(1, 2)), dict(seq=i(3, 9)), dict(seq=i(9, 2).t()),
                dict(seq_len=i(3)), dict(draft_tokens=None), dict(draft_tokens=i(2, 3)), dict(tree_mask=i(2, 3, 2)),
                dict(repetition=f(3)), dict(presence=f(2, 1)), dict(bias=f(2, 4)), dict(bias=f(2, 4), bias_ids=i(2, 5)),
                dict(allowed=i(2, 3, 3)), dict(allowed=i(2, 2, 3).transpose(1, 2)), dict(out=f(2, 3, 51)),
                dict(out=f(2, 3, 50).bfloat16()), dict(gamma_per_row=i(3)), dict(prompt_len=i(1))):
        with pytest.raises(ValueError):
            sv.spec_adjust(**dict(good, **bad))
    for bad in (dict(logits=f(2, 3, 50).half()), dict(seq=f(2, 9)), dict(repetition=i(2)), dict(bias=i(2, 4), bias_ids=i(2, 4)),
                dict(allowed=f(2, 3, 2)), dict(draft_tokens=f(2, 2))):
        with pytest.raises(TypeError):
            sv.spec_adjust(**dict(good, **bad))


def test_binding_takes_numbers_and_tensors():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    for bad in (dict(n_step=None), dict(n_step=1.5), dict(page_size="16"), dict(refs=None), dict(kv_len=[0, 0]), dict(held=None)):
        with pytest.raises(TypeError):
            sv.spec_kv_resize(**dict(dict(refs=i(5), page_table=i(2, 4), held=i(2), kv_len=i(2), n_step=1, page_size=16), **bad))
    with pytest.raises(OverflowError):
        sv.spec_kv_resize(i(5), i(2, 4), i(2), i(2), 1 << 31, 16)
    with pytest.raises(TypeError):
        sv.spec_tree_mask([[0]])


# ------------------------------------------------- streams and devices, on the CPU
def calls_on(device="cuda:0", B=2):
    z = lambda *s, dt=torch.int32: OnGpu(torch.zeros(s, dtype=dt), device)  # noqa: E731
    bf = torch.bfloat16
    cache = sv.KVCache(z(3, 2, 16, 64, dt=bf), z(3, 2, 16, 64, dt=bf))
    pool = (z(5), z(B, 4), z(B), z(B))
    return {
        "attend_tree": lambda **kw: sv.spec_attend_tree(z(B, 3, 4, 64, dt=bf), cache, z(B, 4), z(B), z(B, 3, 1), with_status=True, **kw),
        "compact": lambda **kw: sv.spec_kv_compact(cache, z(B, 4), z(B), z(B, 3), z(B), with_status=True, **kw),
        "copy": lambda **kw: sv.spec_kv_copy(cache, z(4, 3), **kw),
        "resize": lambda **kw: sv.spec_kv_resize(*pool, 1, 16, with_status=True, **kw),
        "fork": lambda **kw: sv.spec_kv_fork(*pool, z(1), z(1), 16, with_status=True, **kw),
        "mask": lambda **kw: sv.spec_tree_mask(z(B, 3), with_status=True, **kw),
        "accept": lambda **kw: sv.spec_tree_accept(z(B, 4), z(B, 3), z(B, 3), with_status=True, **kw),
        "adjust": lambda **kw: sv.spec_adjust(z(B, 2, 9, dt=torch.float32), z(B, 5), z(B), draft_tokens=z(B, 1), with_status=True, **kw),
    }


OPS = ["attend_tree", "compact", "copy", "resize", "fork", "mask", "accept", "adjust"]


class FakeNative:
    """The host-side binding: notes the stream that is current when it is called, gives a pair back."""

    def __init__(self, gpu):
        self.gpu = gpu

    def __getattr__(self, name):
        def called(*args):
            assert all(getattr(a, "device", None) is not None or a is None or isinstance(a, (int, str)) for a in args)
            self.gpu.calls.append((self.gpu.device, self.gpu.streams.get(self.gpu.device, 0)))
            return torch.empty(3, dtype=torch.int32, device="cuda:0"), torch.empty(3, dtype=torch.int32, device="cuda:0")
        return called


@pytest.fixture
def gpu(monkeypatch):
    monkeypatch.setattr(FakeGpu, "spec_attend_tree", FakeGpu._called, raising=False)
    monkeypatch.setattr(FakeGpu, "spec_attend_tree_workspace_size", FakeGpu.spec_attend_workspace_size, raising=False)
    fake = FakeGpu(monkeypatch)
    native = FakeNative(fake)
    for m in (kv, tree):
        monkeypatch.setattr(m, "_native", lambda: native)
    return fake


@pytest.mark.parametrize("op", OPS)
def test_a_given_stream_is_the_one_of_all_tensors(gpu, op):
    """What a call allocates is the given stream's, and goes back not before the
    caller's stream is done with it."""
    got = calls_on()[op](stream=Stream(77))
    assert gpu.calls[0][-1] == 77 and all(t.stream == 77 for t in gpu.made)
    assert all(t.used_on == [0] for t in got)
    calls_on()[op]()
    assert gpu.calls[1][-1] == 0


@pytest.mark.parametrize("op", OPS)
def test_a_given_streams_device_is_current(gpu, op):
    calls_on("cuda:1")[op](stream=Stream(5, "cuda:1"))
    assert gpu.calls[0][0] == 1 and gpu.calls[0][-1] == 5 and gpu.device == 0


@pytest.mark.parametrize("op", OPS)
def test_streams_of_other_devices_and_host_tensors_are_refused(gpu, op):
    with pytest.raises(ValueError):
        calls_on("cuda:1")[op](stream=Stream(5, "cuda:0"))
    with pytest.raises(sv.SpecError):
        calls_on("cpu")[op](stream=Stream(5, "cuda:0"))
    assert not gpu.calls


def test_host_tensors_are_refused():
    """Without a given stream the host-side binding itself says so, behind its other checks."""
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    z = torch.zeros((3, 2, 16, 64), dtype=torch.bfloat16)
    c = sv.KVCache(z, z)
    for call in (lambda: sv.spec_kv_compact(c, i(2, 4), i(2), i(2, 3), i(2)), lambda: sv.spec_kv_copy(c, i(4, 3)),
                 lambda: sv.spec_kv_resize(i(5), i(2, 4), i(2), i(2), 1, 16),
                 lambda: sv.spec_kv_fork(i(5), i(2, 4), i(2), i(2), i(1), i(1), 16), lambda: sv.spec_tree_mask(i(2, 3)),
                 lambda: sv.spec_tree_accept(i(2, 4), i(2, 3), i(2, 3)),
                 lambda: sv.spec_adjust(torch.zeros(2, 1, 9), i(2, 5), i(2)),
                 lambda: sv.spec_attend_tree(torch.zeros((2, 3, 4, 64), dtype=torch.bfloat16), c, i(2, 4), i(2), i(2, 3, 1))):
        with pytest.raises(sv.SpecError, match="no CPU path"):
            call()
