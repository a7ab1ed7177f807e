"""Every launching call of the wrapper runs with its tensors' device current,
on the stream that was asked for, and allocates its output there.  Without a
GPU: the library's calls, the device and the streams are stand-ins that note
what is current when."""

import contextlib
import types

import pytest
import torch

from head_split_kv_decode_b200 import binding as B
from head_split_kv_decode_b200 import cache as C

HERE = torch.device("cuda", 1)  # the cache's; device 0 is current outside


class Fake:
    """A tensor that knows its shape and where it was made."""

    def __init__(self, now, *shape):
        self.now, self.shape, self.device = now, torch.Size(shape), HERE
        self.made = dict(now)

    def data_ptr(self):
        return 1 << 20

    def new_empty(self, shape, dtype=None):
        return Fake(self.now, *shape)


@pytest.fixture
def world(monkeypatch):
    now = {"device": 0, "stream": "default of 0"}
    calls = []

    @contextlib.contextmanager
    def device(d):
        old = dict(now)
        now.update(device=torch.device(d).index, stream="default of %d" % torch.device(d).index)
        yield
        now.update(old)

    @contextlib.contextmanager
    def stream(s):
        old = now["stream"]
        now["stream"] = s.name
        yield
        now["stream"] = old

    def default(d):
        return types.SimpleNamespace(name="default of %d" % d.index, cuda_stream="handle: default of %d" % d.index)

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", default)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now["device"], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: "handle: default of %d" % i, raising=False)
    for name in B.SIGNATURES:
        if hasattr(B, name):
            monkeypatch.setattr(B, name, lambda *a, _n=name: calls.append((_n, dict(now), a[-1])))
    c = object.__new__(C.DuoCache)
    c.handle, c.device, c.batch, c.n_q_heads, c.n_kv_heads, c.head_dim = None, HERE, 2, 8, 2, 128
    c.io_dtype = c.out_dtype = torch.bfloat16
    c.ws_ptr, c.ws_bytes, c.prefill_ws_bytes = 1 << 20, 100, 64
    c._pf_ws = None
    c._check = lambda *a, **k: None
    monkeypatch.setattr(C, "_aligned_buffer", lambda n, d, zero: (Fake(now, n), 0))
    return now, calls, c


def _calls(c, now):
    q, kv, k1 = Fake(now, 2, 8, 128), Fake(now, 2, 5, 2, 128), Fake(now, 2, 2, 128)
    chunk = Fake(now, 2, 5, 8, 128)
    return {
        "duo_append_kv": lambda s: c.append(0, kv, kv, stream=s),
        "duo_append_kv_rows": lambda s: c.append_rows(0, [0, 1], kv, kv, stream=s),
        "duo_decode_attn": lambda s: c.decode(0, q, stream=s),
        "duo_decode_attn_rows": lambda s: c.decode_rows(0, [0, 1], q, stream=s),
        "duo_decode_step": lambda s: c.step(0, q, k1, k1, stream=s),
        "duo_decode_step_rows": lambda s: c.step_rows(0, [0, 1], q, k1, k1, stream=s),
        "duo_prefill_attn": lambda s: c.prefill(0, chunk, kv, kv, stream=s),
        "duo_prefill_attn_rows": lambda s: c.prefill_rows(0, [0, 1], chunk, kv, kv, stream=s),
        "duo_decode_attn_partial": lambda s: c.decode_partial(0, q, stream=s),
    }


NAMES = sorted(_calls(None, {}))


@pytest.mark.parametrize("side", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_call_runs_where_its_cache_lies(world, name, side):
    now, calls, c = world
    stream = types.SimpleNamespace(name="side", cuda_stream="handle: side") if side else None
    out = _calls(c, now)[name](stream)
    want = "side" if side else "default of 1"
    assert [(n, w["device"], w["stream"], h) for n, w, h in calls] == [(name, 1, want, "handle: " + want)]
    for t in (out if isinstance(out, tuple) else (out,)) + (c._pf_ws,):
        if isinstance(t, Fake):
            assert t.made == {"device": 1, "stream": want}
    assert (out is None) == ("append" in name)
    assert now == {"device": 0, "stream": "default of 0"}


def test_given_outputs_are_used(world):
    now, calls, c = world
    out = Fake(now, 2, 8, 128)
    assert c.decode(0, Fake(now, 2, 8, 128), out=out) is out
    o, lse = Fake(now, 2, 8, 128), Fake(now, 2, 8)
    got = c.decode_partial(0, Fake(now, 2, 8, 128), o_part=o, lse_part=lse)
    assert got[0] is o and got[1] is lse


def test_workspace_is_zero_before_the_cache_is_bound(world, monkeypatch):
    """Binding waits for the device, so a first decode on any stream finds the
    workspace's zeros if they were asked for before it."""
    now, calls, _ = world
    order = []

    def buffer(n, device, zero):
        order.append("zeros" if zero else "memory")
        t = Fake(now, n)
        t.__class__ = type("Buffer", (Fake,), {"__getitem__": lambda self, i: self})
        return t, 0
    monkeypatch.setattr(C, "_aligned_buffer", buffer)
    monkeypatch.setattr(B, "duo_cache_create", lambda *a: 1)
    monkeypatch.setattr(B, "duo_cache_required_bytes", lambda h: (100, 100))
    monkeypatch.setattr(B, "duo_cache_bind", lambda *a: order.append("bind on %d" % now["device"]))
    monkeypatch.setattr(B, "duo_prefill_workspace_bytes", lambda h: 0)
    monkeypatch.setattr(B, "duo_cache_destroy", lambda h: None)
    C.DuoCache(1, 1, 2, 1, 128, "bf16", 64, [[1]], 4, 16, device=HERE)
    assert sorted(order[:-1]) == ["memory", "zeros"] and order[-1] == "bind on 1"
