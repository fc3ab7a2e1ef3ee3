"""The cache reference against identities, and the binding's and the C ABI's
refusals, without a GPU."""
import contextlib
import ctypes

import numpy as np
import pytest
import torch

import kv_ref
import speculative_decoding_verify_03_gb300 as sv
from speculative_decoding_verify_03_gb300 import kv


def test_e4m3_table_matches_the_format():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(np.isnan(codes), np.isnan(kv_ref.E4M3))
    ok = ~np.isnan(codes)
    assert np.array_equal(codes[ok], kv_ref.E4M3[ok])


@pytest.mark.parametrize("size", [1e-30, 1e-3, 1.0, 448.0, 3e38])
def test_quantise_is_the_nearest_code(size):
    rng = np.random.default_rng(1)
    row = (rng.standard_normal(64) * size).clip(-3.4e38, 3.4e38)
    codes, e = kv_ref.quantise(row)
    top = np.abs(row).max()
    assert top <= 448 * 2.0 ** e or e == kv_ref.E_MAX
    assert e == kv_ref.E_MIN or top > 448 * 2.0 ** (e - 1)
    got = kv_ref.E4M3[codes] * 2.0 ** e
    near = np.abs(kv_ref.E4M3[:127][None] * 2.0 ** e - np.abs(row)[:, None]).min(1)
    assert np.array_equal(np.abs(np.abs(got) - np.abs(row)), near)
    assert np.array_equal(np.sign(got)[got != 0], np.sign(row)[got != 0])


def test_quantise_edges():
    assert kv_ref.quantise(np.zeros(4))[1] == kv_ref.E_MIN
    codes, e = kv_ref.quantise(np.array([448.0, 1.0, np.nan, np.inf]))
    assert e == 0 and list(codes) == [0x7E, 0x38, 0x7F, 0x7F]
    assert kv_ref.quantise(np.array([449.0]))[1] == 1
    # ties to even: 17 lies between 16 (mantissa 0) and 18 (mantissa 1)
    codes, e = kv_ref.quantise(np.array([448.0, 17.0, 19.0]))
    assert list(kv_ref.E4M3[codes] * 2.0 ** e) == [448.0, 16.0, 20.0]


def test_attend_reference_on_uniform_scores():
    """Zero queries weigh all visible positions alike."""
    rng = np.random.default_rng(2)
    kval, vval = rng.standard_normal((2, 5, 2, 4, 8))
    table, pt = np.array([[3, 0]]), np.array([4])
    q = np.zeros((1, 2, 4, 8))
    out, lse, weight, size = kv_ref.attend(q, kval, vval, table, [5], pt, 3, [1], 4, 0.3)
    seen = np.concatenate([vval[4, :, :3].transpose(1, 0, 2), vval[3, :, :3].transpose(1, 0, 2)])
    assert np.allclose(lse[0, 0], np.log(6)) and np.allclose(lse[0, 1], np.log(7))
    assert np.allclose(out[0, 0, 2], seen[:, 1].mean(0))
    assert np.allclose(weight[0, 0, 0], np.abs(seen[:, 0]).mean(0)) and (size == 0).all()


# ------------------------------------------------------------------ refusals
P = 1 << 20  # a fake, never dereferenced, device address


@pytest.fixture(scope="module")
def L():
    sv.build()
    return sv.lib()


def _cache(**kw):
    f = dict(k_pages=P, v_pages=P, k_exp=P, v_exp=P, k_page_stride=8 * 16 * 64,
             v_page_stride=8 * 16 * 64, n_pages=4, page_size=16, n_kv_heads=8, head_dim=64, format=1)
    f.update(kw)
    return kv.SpecKvCache(**f)


def _batch(**kw):
    f = dict(B=2, gamma_max=3, max_pages=4, prefix_len=0, table_row_stride=4, page_table=P,
             prefix_table=None, kv_len=P, gamma_per_row=None)
    f.update(kw)
    return kv.SpecKvBatch(**f)


BAD = [
    (dict(format=2), {}, 1), (dict(n_pages=-1), {}, 1), (dict(n_kv_heads=0), {}, 1),
    (dict(head_dim=0), {}, 1), (dict(page_size=0), {}, 1), (dict(head_dim=72), {}, 2),
    (dict(page_size=24), {}, 2), (dict(k_page_stride=8 * 16 * 64 - 16), {}, 1),
    (dict(v_page_stride=8 * 16 * 64 + 8), {}, 1), (dict(k_pages=None), {}, 1),
    (dict(v_pages=P + 8), {}, 1), (dict(k_exp=None), {}, 1), (dict(v_exp=P + 1), {}, 1),
    ({}, dict(B=-1), 1), ({}, dict(max_pages=-1), 1), ({}, dict(prefix_len=-1), 1),
    ({}, dict(table_row_stride=3), 1), ({}, dict(B=4097), 2), ({}, dict(page_table=None), 1),
    ({}, dict(kv_len=None), 1), ({}, dict(prefix_len=5), 1),
]
STEP = [({}, dict(gamma_max=-1), 1)]


def _calls(L, c, b):
    s = ctypes.byref((ctypes.c_int64 * 3)(64 * 8 * 4, 64 * 8, 64))
    c, b = ctypes.byref(c), ctypes.byref(b)
    return {
        "append": L.spec_kv_append(c, b, P, P, 1, s, s, None, None),
        "read": L.spec_kv_read(c, b, 0, 4, 1, P, P, None, None),
        "attend": L.spec_attend(c, b, P, 16, s, 0.1, P, P, None, P, 1 << 30, None),
    }


@pytest.mark.parametrize("cache,batch,code", BAD)
def test_descriptors_refused(L, cache, batch, code):
    assert set(_calls(L, _cache(**cache), _batch(**batch)).values()) == {code}


@pytest.mark.parametrize("cache,batch,code", STEP)
def test_step_refused(L, cache, batch, code):
    got = _calls(L, _cache(**cache), _batch(**batch, B=0))
    assert got["append"] == got["attend"] == code and got["read"] == 0


def test_empty_batch_is_noop(L):
    assert set(_calls(L, _cache(), _batch(B=0)).values()) == {0}
    none = _batch(B=0, page_table=None, kv_len=None)
    assert set(_calls(L, _cache(k_pages=None, v_pages=None), none).values()) == {0}


def test_own_arguments_refused(L):
    c, b = ctypes.byref(_cache()), ctypes.byref(_batch())
    s = ctypes.byref((ctypes.c_int64 * 3)(64 * 8 * 4, 64 * 8, 64))
    neg = ctypes.byref((ctypes.c_int64 * 3)(64 * 8 * 4, -64 * 8, 64))
    assert L.spec_kv_append(None, b, P, P, 1, s, s, None, None) == 1
    assert L.spec_kv_append(c, None, P, P, 1, s, s, None, None) == 1
    assert L.spec_kv_append(c, b, None, P, 1, s, s, None, None) == 1
    assert L.spec_kv_append(c, b, P, P, 2, s, s, None, None) == 1
    assert L.spec_kv_append(c, b, P, P + 1, 1, s, s, None, None) == 1
    assert L.spec_kv_append(c, b, P, P, 1, None, s, None, None) == 1
    assert L.spec_kv_append(c, b, P, P, 1, s, neg, None, None) == 1
    assert L.spec_kv_read(c, b, -1, 4, 1, P, P, None, None) == 1
    assert L.spec_kv_read(c, b, 0, -4, 1, P, P, None, None) == 1
    assert L.spec_kv_read(c, b, 0, 4, 1, P, None, None, None) == 1
    assert L.spec_kv_read(c, b, 0, 4, 0, P + 2, P, None, None) == 1
    assert L.spec_kv_read(c, b, 1 << 30, 4, 1, P, P, None, None) == 1
    assert L.spec_kv_read(c, b, 0, 0, 1, P, P, None, None) == 0
    att = lambda q=P, h=16, st=s, sc=0.1, o=P, l=P, ws=P, n=1 << 30: L.spec_attend(  # noqa: E731
        c, b, q, h, st, sc, o, l, None, ws, n, None)
    assert att(q=None) == att(h=0) == att(h=12) == att(st=None) == att(st=neg) == 1
    assert att(sc=float("nan")) == att(sc=float("inf")) == att(sc=-1.0) == att(o=None) == 1
    assert att(q=P + 1) == att(o=P + 2) == att(l=P + 2) == 1
    need = L.spec_attend_workspace_size(c, b, 16)
    assert need > 0
    assert att(ws=None) == att(ws=P + 16) == att(n=need - 1) == 3


def test_workspace_size(L):
    size = lambda cache, batch, h=16: L.spec_attend_workspace_size(  # noqa: E731
        ctypes.byref(cache), ctypes.byref(batch), h)
    assert size(_cache(), _batch()) == size(_cache(k_pages=None), _batch(kv_len=None, page_table=None))
    assert size(_cache(), _batch(prefix_len=100)) > size(_cache(), _batch())
    assert size(_cache(), _batch(B=400)) > size(_cache(), _batch())
    assert size(_cache(head_dim=72), _batch()) == 0
    assert size(_cache(), _batch(), 12) == 0
    assert L.spec_attend_workspace_size(None, ctypes.byref(_batch()), 16) == 0


def test_binding_refuses():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    c = sv.KVCache(z(3, 2, 16, 64), z(3, 2, 16, 64))
    f8 = torch.float8_e4m3fn
    with pytest.raises(TypeError):
        sv.KVCache(z(3, 2, 16, 64, dt=torch.float32), z(3, 2, 16, 64, dt=torch.float32))
    with pytest.raises(TypeError):
        sv.KVCache(z(3, 2, 16, 64, dt=f8), z(3, 2, 16, 64, dt=f8))
    with pytest.raises(ValueError):
        sv.KVCache(z(3, 2, 16, 64), z(3, 2, 16, 64), z(3, 2, 16, dt=torch.int8), z(3, 2, 16, dt=torch.int8))
    with pytest.raises(ValueError):
        sv.KVCache(z(3, 16, 2, 64).transpose(1, 2), z(3, 2, 16, 64))
    with pytest.raises(ValueError):
        sv.KVCache(z(3, 2, 16, 64, dt=f8), z(3, 2, 16, 64, dt=f8), z(3, 2, 8, dt=torch.int8), z(3, 2, 16, dt=torch.int8))
    t, n = i(2, 4), i(2)
    for bad in (dict(k=z(2, 1, 2, 80)), dict(k=z(2, 1, 4, 64)), dict(k=z(3, 1, 2, 64)),
                dict(k=z(2, 1, 64, 2).transpose(2, 3)), dict(kv_len=i(3)), dict(page_table=i(3, 4)),
                dict(page_table=i(4, 2).t()), dict(gamma_per_row=i(3))):
        a = dict(k=z(2, 1, 2, 64), page_table=t, kv_len=n)
        a.update(bad)
        with pytest.raises(ValueError):
            sv.spec_kv_append(c, a["k"], a["k"], a["page_table"], a["kv_len"], a.get("gamma_per_row"))
    with pytest.raises(TypeError):
        sv.spec_kv_append(c, z(2, 1, 2, 64), z(2, 1, 2, 64), t.long(), n)
    with pytest.raises(TypeError):
        sv.spec_kv_append(c, z(2, 1, 2, 64, dt=torch.float16), z(2, 1, 2, 64, dt=torch.float16), t, n)
    with pytest.raises(TypeError):
        sv.spec_kv_read(c, t, n, 4, dtype=torch.float16)
    with pytest.raises(ValueError):
        sv.spec_kv_read(c, t, n, -1)
    with pytest.raises(ValueError):
        sv.spec_kv_read(c, t, n, 4, prefix_len=17, prefix_table=i(1))
    with pytest.raises(TypeError):
        sv.spec_attend(z(2, 1, 4, 64, dt=torch.float32), c, t, n)
    for q in (z(2, 1, 3, 64), z(2, 1, 4, 80), z(3, 1, 4, 64), z(2, 0, 4, 64), z(2, 1, 64, 4).transpose(2, 3)):
        with pytest.raises(ValueError):
            sv.spec_attend(q, c, t, n)
    with pytest.raises(ValueError):
        sv.spec_attend(z(2, 1, 4, 64), c, t, n, prefix_len=3)


def test_binding_takes_pages_of_one_head():
    """A size of one leaves its stride open: only the order of what is there counts."""
    t = torch.zeros((4, 16, 1, 64), dtype=torch.bfloat16).transpose(1, 2)
    assert sv.KVCache(t, t).n_kv_heads == 1


# --------------------------------------- streams, devices and workspaces, on the CPU
class OnGpu:
    """A CPU tensor that says it lies on a GPU."""

    def __init__(self, t, device="cuda:0", stream=None):
        self.t, self.device, self.stream, self.used_on = t, torch.device(device), stream, []

    def record_stream(self, stream):
        self.used_on.append(stream.cuda_stream)

    def __getattr__(self, name):
        return getattr(self.t, name)

    def __getitem__(self, i):
        return self.t[i]


class FakeGpu:
    """The library and torch's current stream and device, none of them real: what
    is allocated and launched is noted with the stream and device of the moment."""

    def __init__(self, monkeypatch):
        self.device, self.streams, self.made, self.calls, self.hook = 0, {}, [], [], None
        empty = torch.empty

        def new(*size, dtype=None, device=None):
            t = OnGpu(empty(*size, dtype=dtype), device, self.streams.get(torch.device(device).index, 0))
            self.made.append(t)
            return t
        monkeypatch.setattr(torch, "empty", new)
        monkeypatch.setattr(torch.cuda, "stream", self.on_stream)
        monkeypatch.setattr(torch.cuda, "device", self.on_device)
        monkeypatch.setattr(torch.cuda, "current_stream",
                            lambda device=None: Stream(self.streams.get(torch.device(device).index, 0), device))
        monkeypatch.setattr(kv, "_device", lambda: self.device, raising=False)
        monkeypatch.setattr(kv, "_raw_stream", lambda index: self.streams.get(index, 0))
        monkeypatch.setattr(kv, "_library", self)

    @contextlib.contextmanager
    def on_device(self, device):
        before, self.device = self.device, torch.device(device).index
        yield
        self.device = before

    @contextlib.contextmanager
    def on_stream(self, stream):
        with self.on_device(stream.device):
            before = self.streams.get(self.device, 0)
            self.streams[self.device] = stream.cuda_stream
            yield
            self.streams[self.device] = before

    def _called(self, *args):
        self.calls.append((self.device, *args))
        hook, self.hook = self.hook, None
        if hook:
            hook()
        return 0

    spec_kv_append = spec_kv_read = spec_attend = _called

    def spec_attend_workspace_size(self, cache, batch, n_heads):
        return batch._obj.B << 20


class Stream:
    def __init__(self, address, device="cuda:0"):
        self.cuda_stream, self.device = address, torch.device(device)


def step_on(device="cuda:0", B=2):
    """Arguments of the three operators, all on one device."""
    z = lambda *s, dt=torch.bfloat16: OnGpu(torch.zeros(s, dtype=dt), device)  # noqa: E731
    cache = sv.KVCache(z(3, 2, 16, 64), z(3, 2, 16, 64))
    t, n = z(B, 4, dt=torch.int32), z(B, dt=torch.int32)
    return {"append": lambda **kw: sv.spec_kv_append(cache, z(B, 1, 2, 64), z(B, 1, 2, 64), t, n, with_status=True, **kw),
            "read": lambda **kw: sv.spec_kv_read(cache, t, n, 5, with_status=True, **kw),
            "attend": lambda **kw: sv.spec_attend(z(B, 1, 4, 64), cache, t, n, with_status=True, **kw)}


def test_calls_that_overlap_do_not_share_a_workspace(monkeypatch):
    """The launches of a call from another thread may come between two of a call's own."""
    gpu = FakeGpu(monkeypatch)
    gpu.hook = step_on()["attend"]
    step_on()["attend"]()
    outer, inner = (c[-3] for c in gpu.calls)
    assert outer and inner and outer != inner


@pytest.mark.parametrize("op", ["append", "read", "attend"])
def test_a_given_stream_is_the_one_of_all_tensors(monkeypatch, op):
    """What a call allocates goes back to the stream that its kernels run on, and
    what it returns not before the caller's stream is done with it."""
    gpu = FakeGpu(monkeypatch)
    got = step_on()[op](stream=Stream(77))
    assert gpu.calls[0][-1] == 77
    assert gpu.made and all(t.stream == 77 for t in gpu.made)
    assert all(t.used_on == [0] for t in (got if isinstance(got, tuple) else (got,)))
    step_on()[op]()
    assert gpu.calls[1][-1] == 0 and gpu.made[-1].stream == 0


def test_workspaces_do_not_outlive_the_call(monkeypatch):
    """A workspace is the call's own: within a graph's capture it is the graph's."""
    gpu = FakeGpu(monkeypatch)
    for B in (1, 3, 2):
        step_on(B=B)["attend"]()
        work = [t for t in gpu.made if t.dtype == torch.uint8]
        assert [t.numel() for t in work] == [B << 20]
        gpu.made.clear()


@pytest.mark.parametrize("op", ["append", "read", "attend"])
def test_the_launch_is_on_the_caches_device(monkeypatch, op):
    gpu = FakeGpu(monkeypatch)
    for device, stream in ((1, None), (0, None), (1, Stream(5, "cuda:1"))):
        gpu.calls.clear()
        step_on(f"cuda:{device}")[op](stream=stream)
        assert gpu.calls[0][0] == device and gpu.calls[0][-1] == (stream.cuda_stream if stream else 0)
        assert gpu.device == 0


@pytest.mark.parametrize("op", ["append", "read", "attend"])
def test_streams_of_other_devices_and_host_tensors_are_refused(monkeypatch, op):
    gpu = FakeGpu(monkeypatch)
    with pytest.raises(ValueError):
        step_on("cuda:1")[op](stream=Stream(5, "cuda:0"))
    with pytest.raises(sv.SpecError):
        step_on("cpu")[op]()
    with pytest.raises(sv.SpecError):
        step_on("cpu")[op](stream=Stream(5, "cuda:0"))
    assert not gpu.calls


def test_a_given_workspace_is_checked(monkeypatch):
    gpu = FakeGpu(monkeypatch)
    ok = OnGpu(torch.zeros(4096, dtype=torch.uint8))
    step_on()["attend"](workspace=ok)
    assert gpu.calls[0][-3:-1] == (ok.data_ptr(), 4096)
    for bad in (None, torch.zeros(4096, dtype=torch.uint8), OnGpu(torch.zeros(4096, dtype=torch.uint8), "cuda:1"),
                OnGpu(torch.zeros((64, 128), dtype=torch.uint8)[:, ::2])):
        with pytest.raises(ValueError):
            step_on()["attend"](workspace=bad)
    assert len(gpu.calls) == 1


def test_workspace_bytes_by_shapes():
    """What a caller that keeps a workspace needs: the package's names alone."""
    sv.build()
    t = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    cache = sv.KVCache(t, t)
    size = lambda **kw: sv.attend_workspace_bytes(cache, sv.SpecKvBatch(**kw), 16)  # noqa: E731
    want = dict(B=3, gamma_max=4, max_pages=7, prefix_len=100)
    made = kv._batch(cache, torch.zeros((3, 7), dtype=torch.int32), torch.zeros(3, dtype=torch.int32), 4,
                     torch.zeros(7, dtype=torch.int32), 100, None)
    assert size(**want) == sv.attend_workspace_bytes(cache, made, 16) > 0
    assert size(**dict(want, B=300)) > size(**want)


def test_workspace_of_a_shared_prefix(L):
    """Its partial results are those of one CTA per multiprocessor (152) and one
    more for each item of 256 query rows: outputs and a logarithm in float32."""
    cache = _cache(head_dim=128, k_page_stride=8 * 16 * 128, v_page_stride=8 * 16 * 128)
    size = lambda **kw: L.spec_attend_workspace_size(ctypes.byref(cache), ctypes.byref(_batch(**kw)), 32)  # noqa: E731
    for B in (17, 64, 300):  # 4 * 4 query rows of each of 8 heads for a sequence
        items = -(-B * 16 // 256) * 8
        more = size(B=B, prefix_len=1000) - size(B=B)
        assert 0 < more <= (items + 152) * 256 * (128 + 1) * 4 + 1024
