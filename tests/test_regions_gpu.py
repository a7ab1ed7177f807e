"""Views of an 8-bit cache's buffers, row by row, packed and paged."""

import pytest
import torch

from head_split_kv_decode_b200 import synth
from head_split_kv_decode_b200.cache import DuoCache

pytestmark = pytest.mark.gpu

BF, D = torch.bfloat16, 128


@pytest.mark.parametrize("paged", [False, True])
def test_gather_rows_of_every_buffer(cuda_lib, paged):
    """Rows of different lengths, appended last row first, so that block ids
    are not row numbers: the tail and the streaming slots are the row's own."""
    batch, S, R = 3, 4, 60
    cache = DuoCache(1, batch, 2, 2, D, "fp8", 600, torch.tensor([[1, 0]]), S, R,
                     **(dict(pool_blocks=9) if paged else {}))
    lens, kept = [70, 300, 545], {}
    for b in (2, 1, 0):
        k, v = (synth.kv_field(10 * i + b, [0], range(lens[b]), 2, D, device="cuda")[0].to(BF) for i in (1, 2))
        cache.append_rows(0, [b], k[None], v[None])
        kept[b] = {"k": k, "v": v}
    torch.cuda.synchronize()
    for b, n in enumerate(lens):
        full = n // 32 * 32
        for name in "kv":
            x = kept[b][name]
            tail = cache.gather_rows(0, "tail_" + name, b, n - full).contiguous().view(BF)
            assert torch.equal(tail[0], x[full:, 0])
            slots = cache.gather_rows(0, "str_" + name, b, S + R).contiguous().view(BF)
            assert torch.equal(slots[0, :S], x[:S, 1])
            p = torch.arange(n - R, n, device="cuda")
            assert torch.equal(slots[0, S + (p - S) % R], x[p, 1])
            assert cache.gather_rows(0, "ret_" + name, b, n).shape == (1, n, D)
