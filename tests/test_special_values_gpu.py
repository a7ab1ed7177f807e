"""NaN, infinities and values at the ends of the types' ranges through the
rotary and 8-bit cache operators.

What a definition makes NaN is NaN, and what it does not touch keeps the bits
of the same call without the special value.
"""

import pytest
import torch

from head_split_kv_decode_b200 import binding as B
from head_split_kv_decode_b200 import synth
from head_split_kv_decode_b200.cache import DuoCache

pytestmark = pytest.mark.gpu

BF, D = torch.bfloat16, 128
NAN, INF = float("nan"), float("inf")


def _seq(seed, n, heads):
    return synth.kv_field(seed, [0], range(n), heads, D, device="cuda")[0].to(BF)


# ------------------------------------------------------------------ split pre-fill


def _prefill(n, C, k, v, q):
    """A chunk of C queries on a history of n tokens; KV head 0 of 2 is a
    retrieval head with 4 query heads, short enough that its tiles are cut
    into runs."""
    cache = DuoCache(1, 1, 8, 2, D, "fp8", n + C, torch.tensor([[1, 0]]), 4, 60)
    cache.append(0, k[None, :n], v[None, :n])
    out = cache.prefill(0, q[None], k[None, n:].contiguous(), v[None, n:].contiguous())[0]
    torch.cuda.synchronize()
    assert B.duo_poll_device_error() == 0
    return out


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("n,C", [(4000, 7), (3001, 300)])
def test_split_prefill_keeps_nan(cuda_lib, n, C, bad):
    """One key, query or value that makes scores or sums NaN: exactly the
    outputs that it reaches are NaN, whichever run of keys holds it."""
    k, v, q = _seq(1, n + C, 2), _seq(2, n + C, 2), _seq(3, C, 8)
    clean = _prefill(n, C, k, v, q)
    assert torch.isfinite(clean.float()).all()
    # a query: its own row and head; q.k sums infinities of both signs or is
    # infinite for some key, and inf - inf is NaN
    q2 = q.clone()
    q2[C // 2, 1, 17] = bad
    out = _prefill(n, C, k, v, q2)
    assert out[C // 2, 1].isnan().all()
    out[C // 2, 1] = clean[C // 2, 1]
    assert torch.equal(out, clean)
    if bad != bad:  # (an infinity in the history takes the largest code)
        for at in (n // 2, 5):
            k2 = k.clone()
            k2[at, 0, 9] = bad
            out = _prefill(n, C, k2, v, q)
            assert out[:, :4].isnan().all()
            assert torch.equal(out[:, 4:], clean[:, 4:])
            v2 = v.clone()
            v2[at, 0, 9] = bad
            out = _prefill(n, C, k, v2, q)
            assert out[:, :4, 9].isnan().all()
            out[:, :4, 9] = clean[:, :4, 9]
            assert torch.equal(out, clean)
    # the chunk's own keys: the queries from that token on
    at = C // 2
    k2 = k.clone()
    k2[n + at, 0, 9] = NAN
    out = _prefill(n, C, k2, v, q)
    assert out[at:, :4].isnan().all()
    assert torch.equal(out[:at], clean[:at]) and torch.equal(out[:, 4:], clean[:, 4:])
