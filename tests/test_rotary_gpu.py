"""Norm and rotation of queries and keys (duo_qk_norm_rope) and the append with
rotation (duo_append_rope), against the fp64 oracle.

Tolerance.  The result is rounded once to its type: half a step, 2^-8 (bf16)
or 2^-24 (fp32) of it.  Before that the kernel works in fp32; relative to
|y_a| + |y_b| of a channel's pair it is off by at most: the sum of squares
(8 serial and 4 tree additions on D = 128, halved by the root: 6 units of
2^-24) + the root (2) + two products (2) + the turn fraction (2^-32 turn and
the fixed-point rate: 1) + sine and cosine (2 each, the Taylor sums' first
omitted terms among them) + mscale (1) + product and fma (2): under 24 units.
"""

import numpy as np
import pytest
import torch

from head_split_kv_decode_b200 import binding as B
from head_split_kv_decode_b200 import synth
from head_split_kv_decode_b200.cache import DuoCache
from head_split_kv_decode_b200.rotary import Rotary, qk_norm_rope
from oracle import rotary as OR

from _util import f64, seeded_mask

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _inv_freq(rot, base=10000.0):
    return (base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float().cuda()


def _weights(seed, d, dtype):
    return (1.0 + 0.3 * synth.kv_field(seed, [0], range(1), 1, d, device="cuda")[0, 0, 0]).to(dtype)


def _tokens(seed, n, heads, d, dtype):
    return synth.kv_field(seed, [0], range(n), heads, d, device="cuda")[0].to(dtype)


def assert_rotated(got, x, pos, rot, weight, eps, inv_freq, interleaved, mscale, what=""):
    y = OR.norm(f64(x), None if weight is None else f64(weight), eps)
    freq = f64(inv_freq) if rot else np.zeros(0)
    ref = OR.rotate(y, pos, freq, interleaved, mscale) if rot else y
    size = OR.pair_size(y, rot, interleaved, mscale)
    tol = (2.0 ** -8 if got.dtype == BF else 2.0 ** -24) * np.abs(ref) + 24 * 2.0 ** -24 * size
    err = np.abs(f64(got) - ref)
    bad = ~(err <= tol)
    assert not bad.any(), "%s: %d off, worst %.3g of %.3g" % (
        what, bad.sum(), err[bad].max(), tol[bad][err[bad].argmax()])


CASES = [  # tokens, hq, hkv, d, dtype, rot, interleaved, norm, start
    (1, 32, 8, 128, BF, 128, False, "qk", 131071),
    (1, 1, 1, 64, F32, 64, False, "qk", 0),
    (7, 5, 3, 128, BF, 128, False, "q", 1000000),
    (7, 5, 3, 64, BF, 32, True, "k", 3),
    (33, 7, 1, 64, F32, 16, True, "", 999983),
    (5, 9, 2, 128, F32, 48, False, "k", -7),
    (3, 3, 3, 64, BF, 64, True, "q", (1 << 31) - 2),
    (40, 32, 8, 128, BF, 0, False, "qk", 0),
    (11, 2, 0, 128, BF, 112, False, "qk", 5),
    (11, 0, 2, 128, F32, 128, True, "qk", 5),
    (1500, 32, 8, 128, BF, 128, False, "qk", 70000),   # several heads a warp
    (3001, 8, 8, 64, F32, 64, True, "qk", 12345),
    (2500, 13, 5, 64, BF, 32, False, "k", 0),
]


@pytest.mark.parametrize("c", CASES, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
def test_qk_norm_rope(cuda_lib, c):
    n, hq, hkv, d, dt, rot, il, norm, start = c
    q = _tokens(1, n, hq, d, dt) if hq else None
    k = _tokens(2, n, hkv, d, dt) if hkv else None
    wq = _weights(3, d, dt) if "q" in norm else None
    wk = _weights(4, d, dt) if "k" in norm else None
    freq, ms, eps = _inv_freq(rot), 1.25, 1e-5
    pos = start + torch.arange(n, dtype=torch.int64, device="cuda") * 3
    r = Rotary(freq, d, interleaved=il, mscale=ms, q_norm=wq, k_norm=wk, eps=eps)
    qo, ko = qk_norm_rope(r, q, k, pos)
    torch.cuda.synchronize()
    for x, o, w in ((q, qo, wq), (k, ko, wk)):
        if x is None:
            assert o is None
            continue
        assert o.dtype == dt and o.is_contiguous()
        assert_rotated(o, x, pos.cpu().numpy(), rot, w, eps, freq, il, ms)


def test_views_in_place_and_streams(cuda_lib):
    """Slices of one projection, heads in another order, out tensors, in
    place, a batch dimension, and a side stream give the same bits."""
    n, hq, hkv, d = 37, 8, 2, 128
    x = _tokens(5, n, hq + 2 * hkv, d, BF)
    r = Rotary(_inv_freq(128), d, q_norm=_weights(6, d, BF), k_norm=_weights(7, d, BF))
    pos = torch.arange(n, device="cuda")
    q, k = x[:, :hq], x[:, hq:hq + hkv]
    qo, ko = qk_norm_rope(r, q, k, pos)
    dq, dk = q.contiguous(), k.contiguous()
    a = qk_norm_rope(r, dq, dk, pos)
    assert torch.equal(a[0], qo) and torch.equal(a[1], ko)
    grouped = torch.stack([dq.view(n, hkv, hq // hkv, d)[:, :, 0], dk], 2).view(n, 2 * hkv, d)
    b = qk_norm_rope(r, grouped[:, ::2], grouped[:, 1::2], pos)  # heads two apart
    assert torch.equal(b[0], qo.view(n, hkv, hq // hkv, d)[:, :, 0]) and torch.equal(b[1], ko)
    c = qk_norm_rope(r, dq.clone()[None], dk.clone()[None], pos[None])
    assert c[0].shape == (1, n, hq, d) and torch.equal(c[0][0], qo)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    e = qk_norm_rope(r, q, k, pos, stream=s)
    s.synchronize()
    assert torch.equal(e[0], qo) and torch.equal(e[1], ko)
    qk_norm_rope(r, dq, dk, pos, q_out=dq, k_out=dk)  # in place
    assert torch.equal(dq, qo) and torch.equal(dk, ko)
    with pytest.raises(ValueError):
        qk_norm_rope(r, q, k, pos, q_out=torch.empty_like(qo[:-1]))
    with pytest.raises(ValueError):
        qk_norm_rope(r, q, k, pos.int())
    with pytest.raises(ValueError):
        qk_norm_rope(r, q, k)
    with pytest.raises(ValueError):
        qk_norm_rope(r, q.float(), k, pos)
    with pytest.raises(ValueError):
        qk_norm_rope(r, q, k[:-1], pos)
    with pytest.raises(ValueError):
        qk_norm_rope(Rotary(_inv_freq(64), 64), q, k, pos)
    with pytest.raises(ValueError):
        qk_norm_rope(Rotary(None, d, q_norm=_weights(6, d, F32)), q, k, pos)


def test_special_values_stay_in_their_vector(cuda_lib):
    """NaN and infinities touch their own head vector only; a zero vector with eps = 0 gives NaN (0/0)."""
    n, d = 6, 128
    q, k = _tokens(8, n, 4, d, BF), _tokens(9, n, 2, d, BF)
    r = Rotary(_inv_freq(64), d, q_norm=_weights(6, d, BF), k_norm=_weights(7, d, BF))
    pos = torch.arange(n, device="cuda")
    qo, ko = qk_norm_rope(r, q, k, pos)
    q2, k2 = q.clone(), k.clone()
    q2[2, 1, 5], k2[3, 0, 100], k2[4, 1] = float("nan"), float("inf"), 0.0
    a, b = qk_norm_rope(r, q2, k2, pos)
    same_q, same_k = torch.ones(n, 4, dtype=torch.bool), torch.ones(n, 2, dtype=torch.bool)
    same_q[2, 1] = same_k[3, 0] = same_k[4, 1] = False
    assert torch.equal(a[same_q], qo[same_q]) and torch.equal(b[same_k], ko[same_k])
    assert a[2, 1].isnan().all() and (b[4, 1] == 0).all()


@pytest.mark.parametrize("dt,d,rot,il", [(BF, 128, 32, False), (BF, 128, 48, True), (F32, 64, 16, True),
                                         (F32, 128, 112, False), (BF, 64, 48, False)])
def test_channels_past_rot_dim_keep_their_bits(cuda_lib, dt, d, rot, il):
    """Infinities, NaN and negative zeros there neither change nor reach another channel."""
    n = 9
    x = _tokens(17, n, 3, d, dt)
    special = torch.tensor([float("inf"), float("-inf"), float("nan"), -0.0], device="cuda", dtype=dt)
    x[:, :, rot:] = torch.where(torch.arange(d - rot, device="cuda") % 3 == 0, x[:, :, rot:],
                                special[torch.arange(d - rot, device="cuda") % 4])
    pos = torch.arange(n, device="cuda") + 11
    freq = _inv_freq(rot)
    r = Rotary(freq, d, interleaved=il)
    o, _ = qk_norm_rope(r, x, None, pos)
    got, want, bits = o[..., rot:].contiguous(), x[..., rot:].contiguous(), torch.int16 if dt == BF else torch.int32
    assert torch.equal(got.isnan(), want.isnan())  # (a NaN's payload is not kept)
    assert torch.equal(got.view(bits)[~want.isnan()], want.view(bits)[~want.isnan()])
    clean = x.clone()
    clean[:, :, rot:] = 0
    want, _ = qk_norm_rope(r, clean, None, pos)
    assert torch.equal(o[..., :rot], want[..., :rot])


def test_graph_capture_and_replay(cuda_lib):
    n, d = 9, 128
    q, k = _tokens(10, n, 8, d, BF), _tokens(11, n, 2, d, BF)
    r = Rotary(_inv_freq(128), d)
    pos = torch.arange(n, device="cuda")
    ref = [t.clone() for t in qk_norm_rope(r, q, k, pos + 100)]
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qk_norm_rope(r, q, k, pos, q_out=qo, k_out=ko)
    pos += 100
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(qo, ref[0]) and torch.equal(ko, ref[1])


# ------------------------------------------------------------------ append

APPENDS = [  # kv, paged, d, Hq, Hkv, n_ret, rot, interleaved, norm
    ("f32", False, 64, 4, 4, 2, 64, False, "qk"),
    ("f32", False, 128, 4, 2, 1, 32, True, ""),
    ("bf16", False, 64, 8, 4, 2, 64, True, "k"),
    ("bf16", False, 128, 8, 4, 4, 128, False, "qk"),
    ("bf16", True, 128, 8, 4, 2, 64, False, "q"),
    ("int4", False, 64, 4, 4, 2, 32, False, "k"),
    ("int4", False, 128, 8, 4, 1, 128, True, ""),
    ("int4", True, 128, 8, 4, 3, 128, False, "qk"),
    ("fp8", False, 128, 8, 4, 2, 128, False, "qk"),
    ("fp8", True, 128, 8, 4, 3, 64, True, "k"),
    ("fp8", True, 128, 6, 2, 0, 128, False, "qk"),
    ("fp8", False, 128, 6, 2, 2, 128, False, ""),
]


@pytest.mark.parametrize("c", APPENDS, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("S,R", [(4, 20), (0, 700)])
def test_append_rope_equals_rotate_then_append(cuda_lib, c, S, R):
    """The same bytes in the whole cache, the same queries, as duo_qk_norm_rope
    followed by duo_append_kv, over chunks of many sizes; the inputs are slices
    of a projection.  Rows are at different lengths where the layout allows."""
    kv, paged, d, hq, hkv, n_ret, rot, il, norm = c
    dt = F32 if kv == "f32" else BF
    batch, cap = 3, 900
    mask = seeded_mask(1, hkv, n_ret)
    kw = dict(pool_blocks=3 * 4) if paged else {}
    one, two = (DuoCache(1, batch, hq, hkv, d, kv, cap, mask[None], S, R, **kw) for _ in range(2))
    r = Rotary(_inv_freq(rot), d, interleaved=il, q_norm=_weights(3, d, dt) if "q" in norm else None,
               k_norm=_weights(4, d, dt) if "k" in norm else None)
    length, seed = [0] * batch, 20
    for rows, n in (([0, 1, 2], 1), ([1], 31), ([0, 2], 33), ([0, 1, 2], 1), ([2, 0], 95), ([1], 257),
                    ([0, 1, 2], 30), ([0], 2), ([1], 64), ([2], 500), ([2, 1, 0], 1)):
        seed += 1
        x = _tokens(seed, len(rows) * n, hq + 2 * hkv, d, dt).view(len(rows), n, hq + 2 * hkv, d)
        q, k, v = x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:]
        at = torch.tensor([[length[b] + i for i in range(n)] for b in rows], device="cuda")
        pos = None if seed % 2 else at + 100000
        qr, kr = qk_norm_rope(r, q, k, at if pos is None else pos)
        two.append_rows(0, rows, kr, v.contiguous())
        with_q = seed % 3 != 0
        got = one.append_rope_rows(0, rows, r, k, v, q=q if with_q else None, positions=pos)
        assert (torch.equal(got, qr) if with_q else got is None)
        for b in rows:
            length[b] += n
        torch.cuda.synchronize()
        # the pools' and buffers' bytes, block tables included
        for b in range(batch):
            assert one.row_seq_len(0, b) == two.row_seq_len(0, b) == length[b]
        assert torch.equal(one.storage, two.storage), "bytes differ after %s += %d" % (rows, n)


def test_append_rope_whole_batch_and_empty(cuda_lib):
    cache = DuoCache(1, 2, 4, 2, 128, "bf16", 64, torch.tensor([[1, 0]]), 2, 10)
    r = Rotary(_inv_freq(128), 128)
    x = _tokens(1, 2 * 5, 4, 128, BF).view(2, 5, 4, 128)
    q = cache.append_rope(0, r, x[:, :, :2], x[:, :, 2:], q=x)
    assert q.shape == (2, 5, 4, 128) and cache.seq_len(0) == 5
    before = cache.storage.clone()
    cache.append_rope(0, r, x[:, :0, :2], x[:, :0, 2:])  # nothing
    none = cache.append_rope(0, r, x[:, :0, :2], x[:, :0, 2:], q=x[:, :0])
    assert none.shape == (2, 0, 4, 128)
    a, b = qk_norm_rope(r, x[0, :0], x[0, :0, :2], torch.zeros(0, dtype=torch.int64, device="cuda"))
    assert a.shape == (0, 4, 128) and b.shape == (0, 2, 128)
    assert cache.seq_len(0) == 5 and torch.equal(before, cache.storage)


def test_append_rope_refuses(cuda_lib):
    """Each refusal leaves the cache's lengths and bytes as they were."""
    cache = DuoCache(1, 2, 4, 2, 128, "fp8", 128, torch.tensor([[1, 0]]), 2, 10, pool_blocks=2)
    r = Rotary(_inv_freq(128), 128)
    x = _tokens(1, 2 * 129, 8, 128, BF).view(2, 129, 8, 128)
    k, v, q = x[:, :, :2], x[:, :, 2:4], x[:, :, 4:]
    before = cache.storage.clone()
    ok = (k[:1, :4], v[:1, :4])
    for args, kw in (((k[:1, :4], v[:1, :3]), {}), (ok, dict(q=x[:1, :4])), ((k[:1, :4].float(), v[:1, :4]), {}),
                     ((k[:1, :4, :1], v[:1, :4, :1]), {}), (ok, dict(positions=torch.zeros(1, 4, device="cuda"))),
                     (ok, dict(positions=torch.zeros(4, dtype=torch.int64, device="cuda"))),
                     (ok, dict(q_out=torch.zeros(1, 4, 4, 128, dtype=BF, device="cuda"))),
                     ((k[0, :4], v[0, :4]), {}), ((k.cpu()[:1, :4], v[:1, :4]), {})):
        with pytest.raises(ValueError):
            cache.append_rope_rows(0, [0], r, *args, **kw)
    with pytest.raises(ValueError):
        cache.append_rope_rows(0, [0], Rotary(_inv_freq(64), 64), *ok)
    for rows, n, name in (([0, 1], 129, "DUO_ERR_CAPACITY"), ([0, 0], 4, "DUO_ERR_ARG"), ([0, 2], 4, "DUO_ERR_ARG")):
        with pytest.raises(B.DuoError) as e:
            cache.append_rope_rows(0, rows, r, k[:, :n].contiguous(), v[:, :n].contiguous())
        assert e.value.name == name
    with pytest.raises(B.DuoError) as e:
        cache.append_rope_rows(1, [0], r, *ok)
    assert e.value.name == "DUO_ERR_ARG"
    torch.cuda.synchronize()
    assert torch.equal(before, cache.storage) and cache.seq_len(0) == 0 and cache.pool_free_blocks() == 2
