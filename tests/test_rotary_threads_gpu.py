"""One rotation shared by host threads, each with its own cache and stream."""

import threading

import pytest
import torch

from head_split_kv_decode_b200 import synth
from head_split_kv_decode_b200.cache import DuoCache
from head_split_kv_decode_b200.rotary import Rotary, qk_norm_rope

pytestmark = pytest.mark.gpu

BF, D = torch.bfloat16, 128


def test_threads_share_a_rotation(cuda_lib):
    """What each thread gets is what it gets alone, call after call."""
    hq, hkv, steps = 8, 2, 60
    freq = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda()
    rot = Rotary(freq, D, q_norm=torch.linspace(0.5, 1.5, D, device="cuda").to(BF))
    data = [synth.kv_field(i, [0], range(steps), hq + 2 * hkv, D, device="cuda").to(BF) for i in range(3)]

    def work(i, out):
        x = data[i]
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.default_stream())
        with torch.cuda.stream(stream):
            cache = DuoCache(1, 1, hq, hkv, D, "fp8", steps, torch.tensor([[1, 0]]), 4, 16)
            cache.set_decode_reproducible(True)
            for t in range(steps):
                part = x[:, t:t + 1]
                q = cache.append_rope(0, rot, part[:, :, hq:hq + hkv], part[:, :, hq + hkv:], q=part[:, :, :hq])
                pos = torch.full((1, 1), t, device="cuda")
                q2, _ = qk_norm_rope(rot, part[:, :, :hq], part[:, :, hq:hq + hkv], pos)
                out.append((q, q2, cache.decode(0, q[:, 0])))
            stream.synchronize()

    alone, together = [[] for _ in data], [[] for _ in data]
    for i in range(len(data)):
        work(i, alone[i])
    threads = [threading.Thread(target=work, args=(i, together[i])) for i in range(len(data))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for a, b in zip(alone, together):
        assert len(a) == len(b) == steps
        for x, y in zip(a, b):
            assert torch.equal(x[0], x[1]) and all(torch.equal(u, v) for u, v in zip(x, y))
