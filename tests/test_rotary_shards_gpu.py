"""The append with rotation into sequence shards: positions counted from the
sequence's start, whatever part of it a shard keeps."""

import pytest
import torch

from head_split_kv_decode_b200 import synth
from head_split_kv_decode_b200.cache import DuoCache
from head_split_kv_decode_b200.rotary import Rotary, qk_norm_rope

pytestmark = pytest.mark.gpu

BF, D = torch.bfloat16, 128


@pytest.mark.parametrize("kv,paged", [("bf16", False), ("bf16", True), ("int4", False), ("fp8", False), ("fp8", True)])
def test_default_positions_in_a_shard(cuda_lib, kv, paged):
    """The bytes of rotating at the global positions and appending, in shards
    before, around and past the tokens, over chunks that cross their ends."""
    hq, hkv, S, R, n = 4, 2, 3, 40, 400
    freq = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda()
    w = torch.linspace(0.5, 1.5, D, device="cuda").to(BF)
    rot = Rotary(freq, D, k_norm=w, q_norm=w)
    x = synth.kv_field(1, range(2), range(n), hq + 2 * hkv, D, device="cuda").to(BF)
    q, k, v = x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:]
    pos = torch.arange(n, device="cuda").expand(2, n)
    for lo, hi in ((0, 133), (133, 266), (266, 1 << 62), (1000, 2000)):
        kw = dict(pool_blocks=4) if paged else {}
        one, two = (DuoCache(1, 2, hq, hkv, D, kv, 134, torch.tensor([[1, 0]]), S, R, **kw) for _ in range(2))
        for c in (one, two):
            c.set_retrieval_shard(lo, hi)
        for a, b in ((0, 1), (1, 100), (100, 140), (140, 141), (141, 270), (270, n)):
            part = [t[:, a:b].contiguous() for t in (q, k, v)]  # (rows of a slice are not at one stride)
            qr, kr = qk_norm_rope(rot, part[0], part[1], pos[:, a:b].contiguous())
            two.append(0, kr, part[2])
            got = one.append_rope(0, rot, part[1], part[2], q=part[0])
            torch.cuda.synchronize()
            assert torch.equal(got, qr) and torch.equal(one.storage, two.storage), (lo, a, b)


def test_append_repeats_itself(cuda_lib):
    """The same tokens give the same bytes every time: nothing depends on the
    order in which blocks run."""
    hq, hkv, n = 8, 4, 3000
    freq = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda()
    rot = Rotary(freq, D, q_norm=torch.ones(D, dtype=BF, device="cuda"), k_norm=torch.ones(D, dtype=BF, device="cuda"))
    x = synth.kv_field(2, [0], range(n), hq + 2 * hkv, D, device="cuda").to(BF)
    cache = DuoCache(1, 1, hq, hkv, D, "fp8", n, torch.tensor([[1, 1, 0, 1]]), 4, 60, pool_blocks=12)
    seen = []
    for _ in range(5):
        cache.release_rows()
        q = cache.append_rope(0, rot, x[:, :, hq:hq + hkv], x[:, :, hq + hkv:], q=x[:, :, :hq])
        torch.cuda.synchronize()
        seen.append((q, cache.storage.clone()))
    assert all(torch.equal(a, b) for s in seen[1:] for a, b in zip(s, seen[0]))
