"""NaN, infinities, values at the ends of the types' ranges, and the bits of a
probability, through the rotary and 8-bit cache operators.

What a definition makes NaN is NaN, and what it does not touch keeps the bits
of the same call without the special value.
"""

import numpy as np
import pytest
import torch

from head_split_kv_decode_b200 import binding as B
from head_split_kv_decode_b200 import synth
from head_split_kv_decode_b200.cache import DuoCache, merge_partials
from head_split_kv_decode_b200.rotary import Rotary, qk_norm_rope
from oracle import attention as OA
from oracle import fp8 as OF

from _util import f64
from test_rotary_gpu import assert_rotated

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


@pytest.mark.parametrize("kv", ["fp8", "bf16", "int4"])
@pytest.mark.parametrize("C", [5, 128, 130, 300])
def test_prefill_rows_do_not_meet(cuda_lib, kv, C):
    """NaN in one row's chunk stays in that row: a key tile that reaches past a
    row's last token does not read the next row's."""
    n = 70
    cache = DuoCache(1, 3, 8, 2, D, kv, n + C, torch.tensor([[1, 0]]), 4, 60)
    k, v, q = (torch.stack([_seq(10 * i + b, n + C, h) for b in range(3)]) for i, h in ((1, 2), (2, 2), (3, 8)))
    cache.append(0, k[:, :n].contiguous(), v[:, :n].contiguous())
    k, v, q = (x[:, n:].contiguous() for x in (k, v, q))
    clean = cache.prefill(0, q, k, v)
    for t in (q, k, v):
        t[1] = NAN
    out = cache.prefill(0, q, k, v)
    torch.cuda.synchronize()
    assert B.duo_poll_device_error() == 0
    assert torch.isfinite(clean.float()).all() and out[1].isnan().all()
    assert torch.equal(out[::2], clean[::2])


@pytest.mark.parametrize("kv", ["fp8", "int4"])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("n,C", [(1, 5), (70, 130), (129, 300), (200, 20), (255, 1), (256, 7), (300, 129), (383, 257)])
def test_prefill_after_a_spoilt_sequence(cuda_lib, kv, paged, n, C):
    """Rows of a coded cache that hold NaN and infinities beside or before a
    sequence, in its blocks, slots, pages or the next ones, do not reach its
    pre-fill."""
    cap = n + C + 300
    kw = dict(pool_blocks=3 * -(-cap // 256)) if paged else {}
    k, v, q = (torch.stack([_seq(10 * i + b, n + C, h) for b in range(3)]) for i, h in ((1, 4), (2, 4), (3, 8)))
    hist, part = [x[:, :n].contiguous() for x in (k, v)], [x[:, n:].contiguous() for x in (q, k, v)]
    outs = []
    for spoilt in (False, True):
        cache = DuoCache(1, 3, 8, 4, D, kv, cap, torch.tensor([[1, 0, 1, 0]]), 4, 500, **kw)
        if spoilt:
            bad = torch.full((3, cap, 4, D), NAN, dtype=BF, device="cuda")
            bad[:, ::3] = INF
            cache.append(0, bad, bad)
            cache.release_rows([0, 2])
        else:
            cache.append_rows(0, [1], *(x[1:2] for x in hist))
        rows = [2, 0]
        cache.append_rows(0, rows, *(x[rows] for x in hist))
        outs.append(cache.prefill_rows(0, rows, *(x[rows] for x in part)))
        torch.cuda.synchronize()
        assert B.duo_poll_device_error() == 0
    assert torch.isfinite(outs[0].float()).all() and torch.equal(outs[0], outs[1])


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


# ------------------------------------------------------------------ the largest values


def _top_block():
    """A block of 32 tokens around bf16's largest value, both signs, with the
    values on either side of the cut and of code 240's neighbours, an infinity
    and a NaN."""
    big = 2.0 ** 120
    vals = [torch.finfo(BF).max, 248 * big, 249 * big, 247 * big, 244 * big, 240 * big, 232 * big, 231 * big, 9 * big,
            1.5 * 2.0 ** 111, 1e30, 0.0, INF, NAN]
    x = torch.zeros(32, 1, D, dtype=torch.float64)
    for i, y in enumerate(vals):
        x[i, 0, i] = y
        x[31 - i, 0, 64 + i] = -y
    return x.to(BF).cuda()


def test_largest_values_are_held_finite(cuda_lib):
    """Every finite bf16 value is held as a finite one, up to the largest:
    codes and scales bit for bit."""
    x = _top_block()
    assert torch.isfinite(x).sum() == x.numel() - 4
    cache = DuoCache(1, 1, 1, 1, D, "fp8", 128, torch.ones(1, 1), 4, 60)
    cache.append(0, x[None], x.flip(0)[None].contiguous())
    torch.cuda.synchronize()
    for name, y in (("k", x), ("v", x.flip(0))):
        held, codes, sc = OF.held(f64(y))
        assert np.isfinite(held[np.isfinite(f64(y))]).all() and np.nanmax(np.abs(held)) < 2.0 ** 128
        got = cache.gather_rows(0, "ret_" + name, 0, 32)[0].cpu().numpy()
        ref, nan = OF.encode_e4m3(codes)[:, 0], np.isnan(codes[:, 0])
        assert np.array_equal(got[~nan], ref[~nan]) and ((got[nan] & 0x7F) == 0x7F).all()
        gs = cache.gather_rows(0, "ret_%s_sz" % name, 0, 1).contiguous().view(torch.float32)
        assert gs.item() == sc[0, 0] == 2.0 ** 120


def test_largest_values_through_the_prefill(cuda_lib):
    """A key or value of bf16's largest magnitude in the history: scores and
    outputs stay finite where the held value makes them so."""
    n, C = 64, 3
    k, v, q = _seq(1, n + C, 1), _seq(2, n + C, 1), torch.zeros(C, 2, D, dtype=BF, device="cuda")
    v[5, 0, 7] = torch.finfo(BF).max
    k[9, 0, 3] = -torch.finfo(BF).max
    cache = DuoCache(1, 1, 2, 1, D, "fp8", n + C, torch.ones(1, 1), 4, 60)
    cache.append(0, k[None, :n], v[None, :n])
    out = cache.prefill(0, q[None], k[None, n:].contiguous(), v[None, n:].contiguous())[0]
    torch.cuda.synchronize()
    # zero queries: every key has the same weight
    held = np.concatenate([OF.held(f64(v[:n]))[0], f64(v[n:])])[:, 0]
    for i in range(C):
        ref = held[:n + i + 1].mean(0)
        # equal probabilities are exact; the mean is rounded once, its fp32 sum is off by 2^-24 a term
        tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -17 * np.abs(held[:n + i + 1]).mean(0)
        assert (np.abs(f64(out[i]) - ref[None]) <= tol[None]).all()


@pytest.mark.parametrize("splits", [0, 3])
def test_large_values_through_the_decode(cuda_lib, splits):
    """Values near the top of fp32's range: the decode's sums hold them as the
    bf16 decode's do (300 keys of up to 2^118: under 2^127)."""
    n = 300
    k = _seq(1, n, 2)
    v = ((1.0 + torch.rand(n, 2, D, generator=torch.Generator().manual_seed(2))) * 2.0 ** 117).to(BF).cuda()
    q = torch.zeros(1, 4, D, dtype=BF, device="cuda")
    cache = DuoCache(1, 1, 4, 2, D, "fp8", n, torch.tensor([[1, 0]]), 4, 290)
    cache.set_decode_output(torch.float32)
    cache.set_decode_splits(splits)
    cache.append(0, k[None], v[None])
    out = f64(cache.decode(0, q)[0])
    # zero queries: every key has the same weight, a power of two, so that only the fp32 sums round
    held = OF.held(f64(v))[0][:, 0], f64(v)[:, 1]
    kept = np.arange(n)[(np.arange(n) < 4) | (np.arange(n) >= n - 290)]
    for h in range(4):
        ref = held[0].mean(0) if h < 2 else held[1][kept].mean(0)
        assert (np.abs(out[h] - ref) <= 2.0 ** -15 * ref).all()


@pytest.mark.parametrize("group", range(1, 9))
def test_decode_keeps_the_probabilities_bits(cuda_lib, group):
    """Every channel holds one key's value, so that each output is one
    probability times it.  Queries have one channel: a score is one exact
    product, |score| log2(e) <= 6, times the scale (4 roundings: 2^-20).  A
    probability is off by that and the exponential's 2^-21, kept to 2^-16 (two
    bf16; two f16 keep more), over a sum of at most 117 (2^-17): 2^-15 in all."""
    n, S, R = 117, 4, 100
    k = _seq(1, n, 2)
    k[:, :, 0] = (8.0 * torch.rand(n, 2, generator=torch.Generator().manual_seed(4)) - 4.0).to(BF).cuda()
    v = torch.zeros(n, 2, D, dtype=BF, device="cuda")
    at = torch.arange(n, device="cuda")
    v[at, :, at] = (1.0 + torch.rand(n, 2, generator=torch.Generator().manual_seed(5))).to(BF).cuda()
    q = torch.zeros(1, 2 * group, D, dtype=BF, device="cuda")
    q[0, :, 0] = torch.linspace(-1.0, 1.0, 2 * group).to(BF).cuda()
    mask = torch.tensor([1, 0])
    cache = DuoCache(1, 1, 2 * group, 2, D, "fp8", n, mask[None], S, R)
    cache.set_decode_output(torch.float32)
    cache.append(0, k[None], v[None])
    kh, vh = f64(k), f64(v)
    kh[:, 0], vh[:, 0] = OF.held(kh)[0][:, 0], OF.held(vh)[0][:, 0]
    ref = OA.decode_reference(f64(q), kh[None], vh[None], mask.numpy(), S, R, 1.0)
    out = f64(cache.decode(0, q, scale=1.0))
    assert (np.abs(out - ref) <= 2.0 ** -15 * ref).all()


# ------------------------------------------------------------------ frequencies


@pytest.mark.parametrize("start", [0, -1000003, 12345678, (1 << 33) - 100])
def test_frequencies_of_every_size(cuda_lib, start):
    """Negative, zero and subnormal frequencies, and many radians a position,
    while |position| * max(|frequency|, 8) < 2^36."""
    n, rot = 33, 64
    f = [4.0, 4.0000005, 7.75, -3.0, -0.3, 0.0, 1e-40, -1e-45, 1.17549435e-38, 1e-20, 5e-7, 1.9999999, 2.0, 3.1415927,
         6.2831855, 1.0 / 3.0]
    f += [100.25, -1000.1, 4096.5, 0.1, 0.2, 0.7, 1e-3, 2.5] if abs(start) < 1 << 24 else [7.9, 0.11] * 4
    f += [0.01 * i for i in range(8)]
    freq = torch.tensor(f, dtype=torch.float32, device="cuda")
    pos = start + torch.arange(n, dtype=torch.int64, device="cuda")
    assert (pos.abs().max().double() * freq.abs().clamp(min=8).max().double()).item() < 2.0 ** 36
    x = _seq(7, n, 3)
    for il in (False, True):
        o, _ = qk_norm_rope(Rotary(freq, D, interleaved=il), x, None, pos)
        torch.cuda.synchronize()
        assert_rotated(o, x, pos.cpu().numpy(), rot, None, 0.0, freq, il, 1.0)


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("il", [False, True])
def test_a_frequency_that_is_not_finite(cuda_lib, il, bad):
    """Its pair is NaN at every position, the others keep their bits; alone and
    on the way into an 8-bit cache, row by row and as whole blocks."""
    n, rot = 40, 64
    freq = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()
    broken = freq.clone()
    broken[5] = bad
    pair = [10, 11] if il else [5, 5 + rot // 2]
    rest = [c for c in range(D) if c not in pair]
    q, k = _seq(8, n, 2), _seq(9, n, 1)
    pos = torch.arange(n, device="cuda")
    ref = qk_norm_rope(Rotary(freq, D, interleaved=il), q, k, pos)
    out = qk_norm_rope(Rotary(broken, D, interleaved=il), q, k, pos)
    for a, b in zip(out, ref):
        assert a[:, :, pair].isnan().all() and torch.equal(a[:, :, rest], b[:, :, rest])
    cache = DuoCache(1, 1, 2, 1, D, "fp8", 128, torch.ones(1, 1), 4, 60)
    r = Rotary(broken, D, interleaved=il)
    for a, b in ((0, 3), (3, n)):
        got = cache.append_rope(0, r, k[None, a:b], k[None, a:b], q=q[None, a:b])[0]
        assert got[:, :, pair].isnan().all() and torch.equal(got[:, :, rest], ref[0][a:b][:, :, rest])
    torch.cuda.synchronize()
    codes = cache.gather_rows(0, "ret_k", 0, 32)[0]
    assert ((codes[:, pair] & 0x7F) == 0x7F).all() and ((codes[:, rest] & 0x7F) != 0x7F).all()
    tail = cache.region(0, "tail_k").view(BF)[0, 0, :n - 32]
    assert tail[:, pair].isnan().all() and torch.equal(tail[:, rest], ref[1][32:, 0][:, rest])
