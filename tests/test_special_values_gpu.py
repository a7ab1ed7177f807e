"""NaN, infinities and values at the ends of the types' ranges through the
rotary and 8-bit cache operators.

What a definition makes NaN is NaN, and what it does not touch keeps the bits
of the same call without the special value.
"""

import pytest
import torch

from head_split_kv_decode_b200 import binding as B
from head_split_kv_decode_b200 import synth
from head_split_kv_decode_b200.cache import DuoCache, merge_partials

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


# ------------------------------------------------------------------ decode


@pytest.mark.parametrize("kv", ["fp8", "bf16", "int4"])
@pytest.mark.parametrize("splits", [1, 3, 100])
def test_decode_partials_keep_nan(cuda_lib, kv, splits):
    """A NaN query makes every score of its head NaN: so are its decode, its
    share of a sequence shard, and what the shares merge to."""
    n = 6000
    mask = torch.tensor([[1, 0]])
    k, v, q = _seq(1, n, 2), _seq(2, n, 2), _seq(3, 1, 8)
    q[0, 2, 40] = q[0, 6, 0] = NAN
    live = [h for h in range(8) if h not in (2, 6)]
    parts = []
    for lo, hi in ((0, 2500), (2500, 1 << 62)):
        c = DuoCache(1, 1, 8, 2, D, kv, n, mask, 4, 60)
        c.set_retrieval_shard(lo, hi)
        c.set_decode_splits(splits)
        c.append(0, k[None], v[None])
        o, lse = c.decode_partial(0, q, owns_streaming=lo == 0)
        assert o[0, 2].isnan().all() and lse[0, 2].isnan()
        if lo == 0:
            assert o[0, 6].isnan().all() and lse[0, 6].isnan()
        assert torch.isfinite(o[0, live]).all()
        parts.append((o, lse))
    out = merge_partials(torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts]),
                         torch.empty(1, 8, D, device="cuda"))
    c = DuoCache(1, 1, 8, 2, D, kv, n, mask, 4, 60)
    c.append(0, k[None], v[None])
    c.set_decode_splits(splits)
    for got in (out, c.decode(0, q).float()):
        assert got[0, (2, 6)].isnan().all() and torch.isfinite(got[0, live]).all()
