"""The 8-bit cache against the fp64 oracle: held bytes bit for bit, decode and
pre-fill over exactly what is held.

Tolerance of the decode (float32 outputs): a probability is rounded to f16
(half a step 2^-11 of it) before it meets a coded value, to bf16 (2^-8) before
a bf16 one.  Scores are fp32 sums of exact products: off by at most 128 terms
of 2^-24 * sum|q k|, under 1e-4 here after the scale (sum|q k| * scale < 100),
and the exponential by 2^-21; 3e-4 covers both for numerator and denominator.
So |err| <= sum_j p_j |v_j| (r_j + 3e-4), r_j = 2^-11 or 2^-8 by key, computed
per element by the oracle itself; bf16 outputs add half their step, 2^-8 |ref|.
"""

import numpy as np
import pytest
import torch

from head_split_kv_decode_b200 import binding as B
from head_split_kv_decode_b200 import synth
from head_split_kv_decode_b200.cache import DuoCache, merge_partials
from head_split_kv_decode_b200.rotary import Rotary, qk_norm_rope
from oracle import attention as OA
from oracle import cache as OC
from oracle import fp8 as OF

from _util import assert_parity, f64, seeded_mask

pytestmark = pytest.mark.gpu

BF, D = torch.bfloat16, 128


def _seq(seed, n, heads):
    """[n, heads, D] with outlier channels, one per 40."""
    x = synth.kv_field(seed, [0], range(n), heads, D, device="cuda")[0]
    x[..., 3::40] *= 10.0
    return x.to(BF)


def _cache(batch, hq, hkv, n_ret, cap, S=4, R=60, paged=False, seed=1):
    mask = seeded_mask(seed, hkv, n_ret)
    kw = dict(pool_blocks=batch * -(-cap // 256)) if paged else {}
    c = DuoCache(1, batch, hq, hkv, D, "fp8", cap, mask[None], S, R, **kw)
    c.set_decode_output(torch.float32)
    return c, mask


def _held(x, mask):
    """K or V [n, heads, D] as attention sees it, and each key's rounding unit of p."""
    full = len(x) // OF.BLOCK * OF.BLOCK
    h = OF.held(f64(x))[0]
    m = mask.numpy().astype(bool)
    out = np.where(m[None, :, None], h, f64(x))
    unit = np.full(x.shape[:2], 2.0 ** -8)
    unit[:full, m] = 2.0 ** -11
    return out, unit[..., None]


def _reference(q, k, v, mask, S, R, scale=None):
    """(output, tolerance) [hq, D] of one row's decode."""
    kh, unit = _held(k, mask)
    vh, _ = _held(v, mask)
    args = (mask.numpy(), S, R, scale)
    ref = OA.decode_reference(f64(q)[None], kh[None], vh[None], *args)[0]
    tol = OA.decode_reference(f64(q)[None], kh[None], (np.abs(vh) * (unit + 3e-4))[None], *args)[0]
    return ref, tol


def assert_close(got, ref, tol, what=""):
    g = f64(got)
    if got.dtype == BF:
        tol = tol + 2.0 ** -8 * np.abs(ref)
    err = np.abs(g - ref)
    assert (err <= tol).all(), "%s: worst %.3g, %.3g allowed" % (what, err.max(), tol.flat[(err - tol).argmax()])


def _check_bytes(cache, mask, b, k, v, S, R):
    """Row b's codes, scales, tail and streaming slots bit for bit."""
    n = len(k)
    full = n // OF.BLOCK * OF.BLOCK
    ret = [h for h in range(len(mask)) if mask[h]]
    strm = [h for h in range(len(mask)) if not mask[h]]
    for name, x in (("k", k), ("v", v)):
        if ret:
            _, codes, sc = OF.held(f64(x[:, ret]))
            got = cache.gather_rows(0, "ret_" + name, b, full)
            if full:
                assert np.array_equal(got.cpu().numpy(), OF.encode_e4m3(codes).transpose(1, 0, 2))
                gs = cache.gather_rows(0, "ret_%s_sz" % name, b, full // OF.BLOCK).contiguous().view(torch.float32)
                assert np.array_equal(gs[..., 0].cpu().numpy().astype(np.float64), sc.T)
            tail = cache.region(0, "tail_" + name).view(BF)[b, :, :n - full]
            assert torch.equal(tail, x[full:][:, ret].transpose(0, 1))
        if strm:
            slots = cache.region(0, "str_" + name).view(BF)[b]
            for i, h in enumerate(strm):
                for p in range(n):
                    if p < S or p >= n - R:
                        assert torch.equal(slots[i, OC.ring_slot(p, S, R)], x[p, h]), (name, h, p)


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("chunks", [[1], [31], [32], [33], [64], [1, 31, 1, 31], [300], [257, 3, 64, 1, 200],
                                    [95, 95, 95, 95], [1] * 70], ids=lambda c: "x".join(map(str, c[:4])))
def test_bytes_do_not_depend_on_the_chunks(cuda_lib, paged, chunks):
    S, R = 3, 40
    cache, mask = _cache(2, 8, 4, 2, 600, S, R, paged)
    n = sum(chunks)
    K, V = [_seq(10 + b, n, 4) for b in range(2)], [_seq(20 + b, n, 4) for b in range(2)]
    K[1][n // 2:, :, 7] = 0
    at = 0
    for c in chunks:
        cache.append(0, torch.stack([x[at:at + c] for x in K]), torch.stack([x[at:at + c] for x in V]))
        at += c
    torch.cuda.synchronize()
    for b in range(2):
        _check_bytes(cache, mask, b, K[b], V[b], S, R)
    full = n // 32
    kept, eq = cache.kv_bytes()
    per = full * 2 * (32 * 128 + 4) + n % 32 * 512
    assert kept == 2 * (2 * per + 2 * min(n, S + R) * 512) and eq == 2 * 4 * per


def test_special_values_in_a_block(cuda_lib):
    """Zero blocks, tiny and huge blocks, infinities and NaN, ties to even."""
    cache, mask = _cache(1, 2, 1, 1, 256)
    x = _seq(5, 224, 1)
    x[0:32] = 0
    x[32:64] *= 1e-30
    x[64:96] *= 1e30
    x[96:128, 0, 9] = float("inf")
    x[100, 0, 10] = float("-inf")
    x[128:160, 0, 11] = float("nan")
    x[160:192] = (torch.arange(32 * 128, device="cuda").view(32, 1, 128) % 512 / 2 - 100).to(BF)
    cache.append(0, x[None], x.flip(0)[None].contiguous())
    torch.cuda.synchronize()
    for name, y in (("k", x), ("v", x.flip(0))):
        _, codes, sc = OF.held(f64(y))
        got = cache.gather_rows(0, "ret_" + name, 0, 224)[0].cpu().numpy()
        ref = OF.encode_e4m3(codes)[:, 0]
        nan = np.isnan(codes[:, 0])
        assert np.array_equal(got[~nan], ref[~nan]) and ((got[nan] & 0x7F) == 0x7F).all()
        gs = cache.gather_rows(0, "ret_%s_sz" % name, 0, 7).contiguous().view(torch.float32)[0, :, 0]
        assert np.array_equal(gs.cpu().numpy().astype(np.float64), sc[:, 0])


LENGTHS = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 300, 511, 1024, 1057, 5000, 20011]


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("n", LENGTHS)
def test_decode_lengths(cuda_lib, n, paged):
    cache, mask = _cache(1, 8, 2, 1, n, 64, 256, paged)
    k, v, q = _seq(1, n, 2), _seq(2, n, 2), 1.5 * _seq(3, 1, 8)
    cache.append(0, k[None], v[None])
    ref, tol = _reference(q[0], k, v, mask, 64, 256)
    assert_close(cache.decode(0, q)[0], ref, tol)
    cache.set_decode_output(BF)
    assert_close(cache.decode(0, q)[0], ref, tol, "bf16")


@pytest.mark.parametrize("hq,hkv,n_ret", [(g * 2, 2, r) for g in range(1, 9) for r in (1, 2)]
                         + [(32, 32, 8), (32, 32, 0), (16, 16, 16), (64, 64, 20), (3, 1, 1), (5, 1, 0)])
def test_decode_head_layouts(cuda_lib, hq, hkv, n_ret):
    n = 3333
    cache, mask = _cache(1, hq, hkv, n_ret, n, 4, 60)
    k, v, q = _seq(1, n, hkv), _seq(2, n, hkv), _seq(3, 1, hq)
    cache.append(0, k[None], v[None])
    ref, tol = _reference(q[0], k, v, mask, 4, 60, 0.2)
    assert_close(cache.decode(0, q, scale=0.2)[0], ref, tol)


@pytest.mark.parametrize("splits", [1, 2, 7, 64, 512])
@pytest.mark.parametrize("n", [40, 2500])
def test_decode_splits(cuda_lib, splits, n):
    cache, mask = _cache(1, 8, 2, 1, n)
    k, v, q = _seq(1, n, 2), _seq(2, n, 2), _seq(3, 1, 8)
    cache.append(0, k[None], v[None])
    ref, tol = _reference(q[0], k, v, mask, 4, 60)
    for repro in (False, True):
        cache.set_decode_splits(splits)
        cache.set_decode_reproducible(repro)
        a = cache.decode(0, q)
        assert_close(a[0], ref, tol, "splits %d" % splits)
        if repro:
            assert torch.equal(cache.decode(0, q), a)


@pytest.mark.parametrize("S,R", [(0, 1), (0, 7), (5, 1), (64, 256), (3, 5000), (17, 1000)])
def test_decode_windows(cuda_lib, S, R):
    n = 1500
    cache, mask = _cache(1, 16, 8, 2, n, S, R)
    k, v, q = _seq(1, n, 8), _seq(2, n, 8), _seq(3, 1, 16)
    cache.append(0, k[None], v[None])
    ref, tol = _reference(q[0], k, v, mask, S, R)
    assert_close(cache.decode(0, q)[0], ref, tol)


def test_query_and_key_ranges(cuda_lib):
    """Queries and values far outside f16's range, blocks whose scales differ
    by 2^40, and one query head of zeros."""
    n = 700
    cache, mask = _cache(1, 8, 2, 1, n)
    k, v, q = _seq(1, n, 2), _seq(2, n, 2), _seq(3, 1, 8)
    q[0, 1] *= 2.0 ** 60
    k[:, 0] *= 2.0 ** -60
    k[:, 1] *= 2.0 ** -60
    q[0, 2] *= 2.0 ** -70
    q[0, 3] = 0
    q[0, 5] *= 2.0 ** 60
    v[:300] *= 2.0 ** 30
    v[300:] *= 2.0 ** -10
    cache.append(0, k[None], v[None])
    ref, tol = _reference(q[0], k, v, mask, 4, 60)
    assert_close(cache.decode(0, q)[0], ref, tol)


def test_stale_bytes_of_released_rows_do_not_matter(cuda_lib):
    """A row that held NaN and infinities is released and refilled, shorter."""
    for paged in (False, True):
        cache, mask = _cache(2, 8, 2, 1, 600, paged=paged)
        bad = torch.full((2, 600, 2, D), float("nan"), dtype=BF, device="cuda")
        bad[:, ::3] = float("inf")
        cache.append(0, bad, bad)
        cache.release_rows()
        k, v, q = _seq(1, 77, 2), _seq(2, 77, 2), _seq(3, 20, 8)
        cache.append(0, torch.stack([k, k]), torch.stack([v, v]))
        ref, tol = _reference(q[0], k, v, mask, 4, 60)
        out = cache.decode(0, torch.stack([q[0], q[0]]))
        kc, vc = _seq(4, 20, 2), _seq(5, 20, 2)
        pre = cache.prefill(0, torch.stack([q, q]), torch.stack([kc, kc]), torch.stack([vc, vc]))
        for b in range(2):
            assert_close(out[b], ref, tol)
            assert torch.isfinite(pre[b].float()).all()


def test_rows_of_different_lengths(cuda_lib):
    """A paged batch served row by row: appends, steps, release and reuse; the
    batch is longer than one launch takes."""
    batch, S, R = 130, 4, 60
    cache, mask = _cache(batch, 8, 2, 1, 1400, S, R, paged=True)
    lens = {b: (b * 37) % 900 + 1 for b in range(batch)}
    lens[5], lens[6], lens[128], lens[129] = 1, 32, 31, 1399
    K = {b: _seq(100 + b, lens[b] + 2, 2) for b in range(batch)}
    V = {b: _seq(300 + b, lens[b] + 2, 2) for b in range(batch)}
    Q = {b: _seq(500 + b, 2, 8) for b in range(batch)}
    for b in range(batch):
        cache.append_rows(0, [b], K[b][None, :lens[b]], V[b][None, :lens[b]])
    order = list(range(batch))[::-1]
    step = [b for b in order if b != 129]
    out = cache.step_rows(0, step, torch.stack([Q[b][0] for b in step]),
                          torch.stack([K[b][lens[b]] for b in step]), torch.stack([V[b][lens[b]] for b in step]))
    check = [5, 6, 128, 0, 17, 64, 127, 99]
    for b in check:
        ref, tol = _reference(Q[b][0], K[b][:lens[b] + 1], V[b][:lens[b] + 1], mask, S, R)
        assert_close(out[step.index(b)], ref, tol, "row %d" % b)
    out = cache.decode_rows(0, [129, 6], torch.stack([Q[129][0], Q[6][0]]))
    for i, b in enumerate((129, 6)):
        n = lens[b] + (b != 129)
        ref, tol = _reference(Q[b][0], K[b][:n], V[b][:n], mask, S, R)
        assert_close(out[i], ref, tol)
    cache.release_rows([6])
    assert cache.row_seq_len(0, 6) == 0
    k, v = _seq(900, 1000, 2), _seq(901, 1000, 2)
    cache.append_rows(0, [6], k[None], v[None])
    ref, tol = _reference(Q[6][1], k, v, mask, S, R)
    assert_close(cache.decode_rows(0, [6], Q[6][1:])[0], ref, tol)
    torch.cuda.synchronize()
    _check_bytes(cache, mask, 6, k, v, S, R)
    _check_bytes(cache, mask, 17, K[17][:lens[17] + 1], V[17][:lens[17] + 1], S, R)


def test_long_steps_across_blocks(cuda_lib):
    """70 fused-call steps across three block boundaries equal the oracle at each."""
    cache, mask = _cache(1, 8, 2, 1, 200)
    k, v, q = _seq(1, 100, 2), _seq(2, 100, 2), _seq(3, 100, 8)
    cache.append(0, k[None, :30], v[None, :30])
    for n in range(30, 100):
        out = cache.step(0, q[None, n], k[None, n], v[None, n])
        if n % 32 in (0, 1, 15, 16, 30, 31):
            ref, tol = _reference(q[n], k[:n + 1], v[:n + 1], mask, 4, 60)
            assert_close(out[0], ref, tol, "step %d" % n)


def test_step_refuses_before_appending(cuda_lib):
    cache, mask = _cache(1, 8, 2, 1, 20000)
    k, v, q = _seq(1, 20000, 2), _seq(2, 20000, 2), _seq(3, 1, 8)
    cache.append(0, k[None], v[None])
    out = torch.empty(1, 8, D, device="cuda")
    kn = k[:1].contiguous()
    for ws, wsb, scale in ((None, 0, 0.0), (cache.ws_ptr, 16, 0.0), (cache.ws_ptr, cache.ws_bytes, float("nan"))):
        with pytest.raises(B.DuoError):
            B.duo_decode_step(cache.handle, 0, q.data_ptr(), kn.data_ptr(), kn.data_ptr(), out.data_ptr(), scale, ws, wsb)
        assert cache.seq_len(0) == 20000
    assert cache.capacity == 20000  # the cache rounds up to 20096
    cache.append(0, k[None, :96], v[None, :96])
    with pytest.raises(B.DuoError) as e:
        cache.step(0, q, k[:1], v[:1])
    assert e.value.name == "DUO_ERR_CAPACITY" and cache.seq_len(0) == 20096


def test_static_scratch_decode(cuda_lib):
    n = 9000
    cache, mask = _cache(1, 8, 2, 1, n)
    k, v, q = _seq(1, n, 2), _seq(2, n, 2), _seq(3, 1, 8)
    cache.append(0, k[None], v[None])
    cache.set_decode_reproducible(True)
    assert cache.decode_splits(0) > 1
    ref = cache.decode(0, q)
    out = torch.empty_like(ref)
    for _ in range(2):
        B.duo_decode_attn_static(cache.handle, 0, q.data_ptr(), out.data_ptr(), 0.0)
        torch.cuda.synchronize()
        assert torch.equal(out, ref)


def test_offsets_past_32_bits(cuda_lib):
    """Code buffers of 4.9 GB: the last heads and the last batch row lie past 2^32 bytes."""
    hq = hkv = 64
    cache = DuoCache(1, 2, hq, hkv, D, "fp8", 300000, torch.ones(1, hkv), 4, 60)
    cache.set_decode_output(torch.float32)
    assert cache.region(0, "ret_k").numel() > 1 << 32
    n = 100
    k, v, q = _seq(1, n, hkv), _seq(2, n, hkv), _seq(3, 1, hq)
    cache.append(0, torch.stack([k, k]), torch.stack([v, v]))
    out = cache.decode(0, torch.cat([q, q]))
    ref, tol = _reference(q[0], k, v, torch.ones(hkv, dtype=torch.uint8), 4, 60)
    for b in range(2):
        assert_close(out[b], ref, tol)
    cache.close()


def test_shard_without_keys(cuda_lib):
    """A shard that holds no position yet: retrieval partials empty, streaming heads whole."""
    mask = torch.tensor([1, 0], dtype=torch.uint8)
    k, v, q = _seq(1, 90, 2), _seq(2, 90, 2), _seq(3, 1, 8)
    c = DuoCache(1, 1, 8, 2, D, "fp8", 64, mask[None], 4, 60)
    c.set_retrieval_shard(2000, 1 << 62)
    c.append(0, k[None], v[None])
    for own in (True, False):
        o, lse = c.decode_partial(0, q, owns_streaming=own)
        torch.cuda.synchronize()
        assert (o[0, :4] == 0).all() and (lse[0, :4] == -float("inf")).all()
        assert torch.isfinite(lse[0, 4:]).all() if own else (lse[0, 4:] == -float("inf")).all()
    ref, tol = _reference(q[0], k, v, torch.zeros(2, dtype=torch.uint8), 4, 60)
    o, _ = c.decode_partial(0, q)
    assert_close(o[0, 4:], ref[4:], tol[4:])


def test_captured_steps_and_two_caches(cuda_lib):
    """Append with rotation and decode captured into graphs of two caches that
    share nothing, replayed at the same time on two streams: each replay writes
    the same slots and attends to them, whatever its inputs hold by then."""
    rot = Rotary((10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda(), D)
    work = []
    for i in range(2):
        n = 1000 + 37 * i
        cache, mask = _cache(1, 8, 2, 1, n + 1, paged=bool(i))
        k, v = _seq(10 + i, n + 2, 2), _seq(20 + i, n + 2, 2)
        cache.append(0, k[None, :n], v[None, :n])
        cache.set_decode_reproducible(True)
        x = _seq(30 + i, 2, 12).view(2, 1, 1, 12, D)
        io = x[0].clone()
        cache.decode(0, io[0, :, :8].contiguous())  # launch facts looked up before the capture
        g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            q = cache.append_rope(0, rot, io[:, :, 8:10], io[:, :, 10:], q=io[:, :, :8])
            out = cache.decode(0, q[:, 0])
        work.append((cache, mask, k[:n], v[:n], x, io, g, s, out, n))
    for t in (0, 1):
        for *_, x, io, g, s, out, n in work:
            io.copy_(x[t])
        torch.cuda.synchronize()
        for *_, g, s, out, n in work:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for cache, mask, k, v, x, io, g, s, out, n in work:
            pos = torch.tensor([[n]], device="cuda")
            q1, k1 = qk_norm_rope(rot, x[t][:, :, :8], x[t][:, :, 8:10], pos)
            ref, tol = _reference(q1[0, 0], torch.cat([k, k1[0]]), torch.cat([v, x[t][0, :, 10:]]), mask, 4, 60)
            assert_close(out[0], ref, tol)


def test_side_stream_and_default_stream(cuda_lib):
    """The same calls on a side stream give the same bits as on the current one."""
    rot = Rotary((10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda(), D)
    x = _seq(40, 70, 12).view(1, 70, 12, D)
    outs = []
    for side in (None, torch.cuda.Stream()):
        cache, mask = _cache(1, 8, 2, 1, 100)
        cache.set_decode_reproducible(True)
        torch.cuda.synchronize()
        q = cache.append_rope(0, rot, x[:, :, 8:10], x[:, :, 10:], q=x[:, :, :8], stream=side)
        if side is not None:
            side.synchronize()
        o = cache.decode(0, q[:, -1].contiguous(), stream=side)
        torch.cuda.synchronize()
        outs.append((q, o, cache.storage.clone()))
    assert all(torch.equal(a, b) for a, b in zip(*outs))


@pytest.mark.parametrize("world", [2, 3])
def test_sequence_shards(cuda_lib, world):
    """Shards (odd boundaries: blocks count from the shard's first position),
    merged, equal attention over what the shards hold."""
    n, S, R, hq, hkv = 1001, 4, 60, 8, 4
    mask = seeded_mask(2, hkv, 2)
    k, v, q = _seq(1, n, hkv), _seq(2, n, hkv), _seq(3, 1, hq)
    per = -(-n // world)
    ranges = [(r * per, (r + 1) * per if r < world - 1 else 1 << 62) for r in range(world)]
    parts, kh, vh, unit = [], f64(k), f64(v), np.full((n, hkv, 1), 2.0 ** -8)
    m = mask.numpy().astype(bool)
    for r, (lo, hi) in enumerate(ranges):
        c = DuoCache(1, 1, hq, hkv, D, "fp8", per, mask[None], S, R)
        c.set_retrieval_shard(lo, hi)
        for a, b in ((0, 5), (5, 400), (400, 401), (401, n)):
            c.append(0, k[None, a:b], v[None, a:b])
        parts.append(c.decode_partial(0, q, owns_streaming=r == 0))
        end = min(hi, n)
        kh[lo:end, m] = OF.held(f64(k[lo:end]))[0][:, m]
        vh[lo:end, m] = OF.held(f64(v[lo:end]))[0][:, m]
        unit[lo:lo + (end - lo) // 32 * 32, m] = 2.0 ** -11
    out = torch.empty(1, hq, D, device="cuda")
    merge_partials(torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts]), out)
    ref = OA.decode_reference(f64(q), kh[None], vh[None], mask.numpy(), S, R)
    tol = OA.decode_reference(f64(q), kh[None], (np.abs(vh) * (unit + 3e-4))[None], mask.numpy(), S, R)
    assert_close(out, ref, tol)


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("h,C", [(0, 1), (0, 130), (1, 1), (31, 33), (32, 128), (100, 257), (700, 64)])
def test_prefill(cuda_lib, h, C, paged):
    """Attend-then-append chunks over what the cache holds (bar of the bf16
    pre-fill: the expansion is exact, so it is the same kernel on the same kind of rows)."""
    S, R, hq, hkv = 4, 60, 8, 4
    cache, mask = _cache(2, hq, hkv, 2, 1024, S, R, paged)
    n = h + C

    def plain(seed, n, heads):
        return synth.kv_field(seed, [0], range(n), heads, D, device="cuda")[0].to(BF)
    K, V = [plain(1 + b, n, hkv) for b in range(2)], [plain(3 + b, n, hkv) for b in range(2)]
    q = [plain(5 + b, C, hq) for b in range(2)]
    if h:
        cache.append(0, torch.stack([x[:h] for x in K]), torch.stack([x[:h] for x in V]))
        cache._prefill_ws()
        cache._pf_ws.fill_(0xFF)  # NaN bytes: the workspace needs no initialisation
    out = cache.prefill(0, torch.stack(q), torch.stack([x[h:] for x in K]), torch.stack([x[h:] for x in V]))
    torch.cuda.synchronize()
    for b in range(2):
        kh, vh = (np.concatenate([_held(x[:h], mask)[0], f64(x[h:])]) for x in (K[b], V[b]))
        ref = OA.prefill_reference(f64(q[b])[None], kh[None], vh[None], h, mask.numpy(), S, R)
        assert_parity(out[b:b + 1], ref, "bf16", "row %d" % b)


@pytest.mark.parametrize("lens,C,hq,hkv,n_ret", [
    ([4000], 7, 8, 2, 1), ([3000], 300, 8, 4, 2), ([5000, 40], 20, 4, 2, 1), ([1, 2000, 130], 129, 6, 2, 2),
    ([2500], 1, 16, 2, 1)])
def test_prefill_split(cuda_lib, lens, C, hq, hkv, n_ret):
    """Short chunks on long histories, whose tiles are cut into runs (rows with
    fewer tiles than runs among them), against the oracle."""
    S, R, batch = 4, 60, len(lens)
    cache, mask = _cache(batch, hq, hkv, n_ret, max(lens) + C, S, R, paged=batch > 1)

    def plain(seed, n, heads):
        return synth.kv_field(seed, [0], range(n), heads, D, device="cuda")[0].to(BF)
    K = [plain(10 + b, n + C, hkv) for b, n in enumerate(lens)]
    V = [plain(20 + b, n + C, hkv) for b, n in enumerate(lens)]
    q = [plain(30 + b, C, hq) for b in range(batch)]
    for b, n in enumerate(lens):
        cache.append_rows(0, [b], K[b][None, :n], V[b][None, :n])
    cache._prefill_ws()
    cache._pf_ws.fill_(0xFF)
    out = cache.prefill(0, torch.stack(q), torch.stack([x[n:] for x, n in zip(K, lens)]),
                        torch.stack([x[n:] for x, n in zip(V, lens)]))
    torch.cuda.synchronize()
    assert B.duo_poll_device_error() == 0
    for b, h in enumerate(lens):
        kh, vh = (np.concatenate([_held(x[:h], mask)[0], f64(x[h:])]) for x in (K[b], V[b]))
        ref = OA.prefill_reference(f64(q[b])[None], kh[None], vh[None], h, mask.numpy(), S, R)
        assert_parity(out[b:b + 1], ref, "bf16", "row %d" % b)


def test_calls_refused(cuda_lib):
    cache, mask = _cache(1, 8, 2, 1, 256)
    q = _seq(1, 1, 8)
    with pytest.raises(B.DuoError) as e:
        cache.decode(0, q)
    assert e.value.name == "DUO_ERR_STATE"
    k = _seq(1, 40, 2)
    cache.append(0, k[None], k[None])
    odd = torch.zeros(8 * D + 1, dtype=BF, device="cuda")[1:].view(1, 8, D)  # contiguous, 2 bytes off
    with pytest.raises(B.DuoError) as e:
        cache.decode(0, odd)
    assert e.value.name == "DUO_ERR_ARG"
    with pytest.raises(B.DuoError) as e:
        cache.step(0, odd, k[None, 0], k[None, 0])
    assert e.value.name == "DUO_ERR_ARG" and cache.seq_len(0) == 40
    with pytest.raises(B.DuoError) as e:  # the 8-bit pre-fill needs its workspace
        B.duo_prefill_attn(cache.handle, 0, q.data_ptr(), k.data_ptr(), k.data_ptr(), 1, q.data_ptr(), 0.0, None, 0)
    assert e.value.name == "DUO_ERR_WORKSPACE"
    with pytest.raises(B.DuoError) as e:
        cache.append(0, torch.cat([k] * 6)[None], torch.cat([k] * 6)[None])
    assert e.value.name == "DUO_ERR_CAPACITY" and cache.seq_len(0) == 40


def test_serving_loop(cuda_lib):
    """The operators as a serving loop uses them: a prompt in chunks (norm and
    rotation, pre-fill, append), then tokens (append with rotation, decode),
    two layers, on an 8-bit paged cache; every attention against the oracle."""
    S, R, hq, hkv, layers = 4, 60, 8, 4, 2
    masks = torch.stack([seeded_mask(7 + i, hkv, 2) for i in range(layers)])
    cache = DuoCache(layers, 1, hq, hkv, D, "fp8", 600, masks, S, R, pool_blocks=3)
    cache.set_decode_output(torch.float32)
    freq = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda()
    w = [(1 + 0.2 * _seq(90 + i, 1, 1)[0, 0].float().clamp(-1, 1)).to(BF) for i in range(2)]
    rot = Rotary(freq, D, q_norm=w[0], k_norm=w[1])
    seen = [([], []) for _ in range(layers)]
    at = 0
    for C in (200, 133, 1, 1, 1, 1):
        pos = torch.arange(at, at + C, device="cuda")
        for layer in range(layers):
            x = synth.kv_field(1000 * layer + at, [0], range(C), hq + 2 * hkv, D, device="cuda")[0].to(BF)
            q, k, v = x[None, :, :hq], x[None, :, hq:hq + hkv], x[None, :, hq + hkv:]
            qr, kr = qk_norm_rope(rot, q, k, pos[None])
            ks, vs = seen[layer]
            mask = masks[layer]
            if C > 1:
                out = cache.prefill(layer, qr, kr, v.contiguous())
                cache.append_rope(layer, rot, k, v)
                hist = [torch.cat(y) if y else None for y in (ks, vs)]
                kh, vh = (np.concatenate([_held(a, mask)[0], f64(b)]) if a is not None else f64(b)
                          for a, b in zip(hist, (kr[0], v[0])))
                ref = OA.prefill_reference(f64(qr), kh[None], vh[None], at, mask.numpy(), S, R)
                assert_parity(out, ref, "bf16", "chunk at %d" % at)
                ks.append(kr[0]), vs.append(v[0])
            else:
                q1 = cache.append_rope(layer, rot, k, v, q=q)
                assert torch.equal(q1, qr)
                out = cache.decode(layer, q1[:, 0])
                ks.append(kr[0]), vs.append(v[0])
                ref, tol = _reference(qr[0, 0], torch.cat(ks), torch.cat(vs), mask, S, R)
                assert_close(out[0], ref, tol, "token at %d" % at)
        at += C
    assert B.duo_poll_device_error() == 0
