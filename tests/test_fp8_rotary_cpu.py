"""The 8-bit cache and the rotation without a GPU: pins of their oracles,
layout plan and byte accounting, and every refusal of the new calls (made
before anything is enqueued, so bad pointers are never followed)."""

import ctypes

import numpy as np
import pytest
import torch

from head_split_kv_decode_b200 import binding as B
from head_split_kv_decode_b200 import build as BUILD
from head_split_kv_decode_b200 import rotary as RT
from oracle import fp8 as OF
from oracle import rotary as OR


@pytest.fixture(scope="module")
def lib():
    BUILD.build()
    return B.lib()


# ------------------------------------------------------------------ oracles


def test_oracle_codes_match_torch_and_the_value_table():
    """Every byte decodes to its own code, and rounding agrees with an
    independent conversion (torch's float8_e4m3fn) on ties and subnormals."""
    codes = torch.arange(256, dtype=torch.uint8)
    vals = codes.view(torch.float8_e4m3fn).double().numpy()
    fin = np.isfinite(vals)
    assert fin.sum() == 254 and np.nanmax(vals) == 448.0
    assert np.array_equal(OF.encode_e4m3(vals[fin]), codes.numpy()[fin])
    assert OF.encode_e4m3(np.array([np.nan]))[0] & 0x7F == 0x7F
    g = torch.Generator().manual_seed(3)
    x = torch.cat([torch.randn(20000, generator=g) * 100, torch.randn(20000, generator=g) * 0.02]).to(torch.bfloat16)
    x = x.float().clamp(-448, 448)
    assert np.array_equal(OF.nearest_e4m3(x.double().numpy()), x.to(torch.float8_e4m3fn).double().numpy())


@pytest.mark.parametrize("amax,scale", [(448.0, 1.0), (449.0, 2.0), (447.0, 1.0), (224.0, 0.5),
                                        (225.0, 1.0), (1.75, 2.0 ** -8), (0.0, 2.0 ** -120),
                                        (1e-38, 2.0 ** -120), (3e38, 2.0 ** 120)])
def test_oracle_scale_is_the_smallest_power(amax, scale):
    x = np.zeros((OF.BLOCK, 8))
    x[5, 3] = -amax
    assert OF.block_scale(x) == scale
    x[6, 1], x[7, 2] = np.inf, np.nan  # do not set the scale
    assert OF.block_scale(x) == scale


def test_oracle_rotation_pins():
    """Quarter turns by hand; relative positions: <R_m q, R_n k> depends on m - n; norm of ones."""
    y = np.arange(8, dtype=np.float64).reshape(1, 1, 8)
    quarter = [np.pi / 2] * 4
    assert np.allclose(OR.rotate(y, [1], quarter)[0, 0], [-4, -5, -6, -7, 0, 1, 2, 3], atol=1e-15)
    assert np.allclose(OR.rotate(y, [1], quarter, True)[0, 0], [-1, 0, -3, 2, -5, 4, -7, 6], atol=1e-15)
    assert np.allclose(OR.rotate(y, [1], quarter[:2])[0, 0], [-2, -3, 0, 1, 4, 5, 6, 7], atol=1e-15)
    r = np.random.default_rng(0)
    q, k, f = r.normal(size=(1, 1, 16)), r.normal(size=(1, 1, 16)), r.uniform(0, 1, 8)
    for il in (False, True):
        a = (OR.rotate(q, [1007], f, il) * OR.rotate(k, [1000], f, il)).sum()
        b = (OR.rotate(q, [7], f, il) * k).sum()
        assert abs(a - b) < 1e-11
    assert np.allclose(OR.norm(np.full((1, 4), -3.0), [1, 2, 3, 4], 0.0), [[-1, -2, -3, -4]])


# ------------------------------------------------------------------ layout


def _create(**kw):
    args = dict(layers=2, batch=3, n_q_heads=8, n_kv_heads=4, head_dim=128, kv_dtype="fp8",
                capacity=1000, head_mask=[1, 0, 0, 1, 0, 0, 0, 0], S=4, R=60)
    args.update(kw)
    if "pool_blocks" in args:
        return B.duo_cache_create_paged(**args)
    return B.duo_cache_create(**args)


@pytest.mark.parametrize("paged", [False, True])
def test_fp8_layout(lib, paged):
    h = _create(**(dict(pool_blocks=10) if paged else {}))
    try:
        cb, _ = B.duo_cache_required_bytes(h)
        v = B.duo_layout_info(h, 0)
        assert v.capacity == 1024 and v.row_bytes == 128 and v.str_k_sz == v.str_v_sz == -1
        rows = 10 * 2 * 256 if paged else 3 * 2 * 1024
        tk, tv = B.duo_fp8_tail_info(h, 0)
        tail = 3 * 2 * 32 * 256
        regions = [(v.ret_k, rows * 128), (v.ret_v, rows * 128), (v.ret_k_sz, rows // 32 * 4),
                   (v.ret_v_sz, rows // 32 * 4), (v.str_k, 3 * 2 * 64 * 256),
                   (v.str_v, 3 * 2 * 64 * 256), (tk, tail), (tv, tail)]
        v1 = B.duo_layout_info(h, 1)  # no retrieval head: no codes, scales or tails
        assert B.duo_fp8_tail_info(h, 1) == (-1, -1) and v1.ret_k == v1.ret_k_sz == -1
        regions += [(v1.str_k, 3 * 4 * 64 * 256), (v1.str_v, 3 * 4 * 64 * 256)]
        regions.sort()
        assert all(off % 256 == 0 for off, _ in regions)
        for (a, sa), (b, _) in zip(regions, regions[1:]):
            assert a + sa <= b, "regions overlap"
        assert regions[-1][0] + regions[-1][1] <= cb
        assert B.duo_prefill_workspace_bytes(h) > 0
        assert B.duo_kv_bytes(h) == (0, 0)
    finally:
        B.duo_cache_destroy(h)
    other = _create(kv_dtype="bf16")
    try:
        assert B.duo_fp8_tail_info(other, 0) == (-1, -1)
    finally:
        B.duo_cache_destroy(other)


@pytest.mark.parametrize("kw,name", [
    (dict(head_dim=64), "DUO_ERR_UNSUPPORTED"),
    (dict(n_q_heads=36), "DUO_ERR_UNSUPPORTED"),            # 9 query heads per KV head
    (dict(n_q_heads=36, pool_blocks=4), "DUO_ERR_UNSUPPORTED"),
    (dict(pool_blocks=0), "DUO_ERR_ARG"),
    (dict(n_q_heads=10), "DUO_ERR_LAYOUT"),
    (dict(kv_dtype=4), "DUO_ERR_ARG"),
])
def test_fp8_create_refusals(lib, kw, name):
    with pytest.raises(B.DuoError) as e:
        _create(**kw)
    assert e.value.name == name


@pytest.mark.parametrize("group", range(1, 9))
def test_fp8_takes_every_group_size(lib, group):
    h = _create(n_q_heads=4 * group)
    B.duo_cache_destroy(h)


def test_fp8_planner(lib):
    """The 8-bit decode's plan: no more CTAs than SMs for one long row, a
    split per 1024 keys at most, one split for a short row."""
    h = _create(batch=1, layers=1, head_mask=[1, 1, 0, 0], capacity=1 << 20)
    try:
        for n in (1, 31, 32, 1024, 1025, 5000, 131072, 1 << 20):
            splits, pack = B.duo_test_plan_decode(h, 0, [n], 148)
            assert 1 <= splits[0] <= max(1, -(-n // 1024))
            assert 2 * splits[0] + -(-2 // pack) <= 148
        assert B.duo_test_plan_decode(h, 0, [1 << 20], 148)[0][0] >= 72
    finally:
        B.duo_cache_destroy(h)


# ------------------------------------------------------------------ refusals

PTR = 1 << 20  # never followed: every call below is refused


def _rope(**kw):
    args = dict(rot_dim=64, interleaved=0, inv_freq=PTR, mscale=1.0, norm_eps=1e-6, q_norm=None,
                k_norm=None)
    args.update(kw)
    return B.duo_rope_desc(*[args[n] for n, _ in B.duo_rope_desc._fields_])


def _heads(data=PTR, tok=1024, head=128):
    return B.duo_heads(data, tok, head)


BAD_ROPE = [dict(rot_dim=-16), dict(rot_dim=8), dict(rot_dim=144), dict(interleaved=2),
            dict(interleaved=-1), dict(inv_freq=None), dict(inv_freq=PTR + 2),
            dict(mscale=float("nan")), dict(mscale=float("inf")), dict(q_norm=PTR + 8),
            dict(k_norm=PTR + 2), dict(q_norm=PTR, norm_eps=-1e-6),
            dict(k_norm=PTR, norm_eps=float("nan"))]
BAD_HEADS = [None, _heads(data=None), _heads(data=PTR + 8), _heads(tok=1028), _heads(head=4),
             _heads(tok=-1024), _heads(head=-128)]


def _qk(rope=None, **kw):
    args = dict(rope=rope or _rope(), dtype="bf16", n_tokens=4, n_q_heads=8, n_kv_heads=2,
                head_dim=128, q=_heads(), k=_heads(), positions_ptr=PTR, q_out_ptr=PTR, k_out_ptr=PTR)
    args.update(kw)
    B.duo_qk_norm_rope(**args)


@pytest.mark.parametrize("bad", BAD_ROPE)
def test_qk_norm_rope_refuses_descriptions(lib, bad):
    with pytest.raises(B.DuoError) as e:
        _qk(_rope(**bad))
    assert e.value.name == "DUO_ERR_ARG"


@pytest.mark.parametrize("kw", [
    dict(dtype="int4"), dict(dtype="fp8"), dict(head_dim=96), dict(n_tokens=-1), dict(n_q_heads=-1),
    dict(n_kv_heads=-2), dict(n_q_heads=70000), dict(n_tokens=1 << 41), dict(positions_ptr=None),
    dict(positions_ptr=PTR + 4), dict(q_out_ptr=None), dict(k_out_ptr=None), dict(q_out_ptr=PTR + 8),
    dict(k_out_ptr=PTR + 4)] + [dict(q=h) for h in BAD_HEADS] + [dict(k=h) for h in BAD_HEADS])
def test_qk_norm_rope_refuses_arguments(lib, kw):
    with pytest.raises(B.DuoError) as e:
        _qk(**kw)
    assert e.value.name == "DUO_ERR_ARG"


def test_qk_norm_rope_null_description(lib):
    assert lib.duo_qk_norm_rope(None, 1, 4, 8, 2, 128, _heads(), _heads(), PTR, PTR, PTR, None) == 1
    _qk(n_tokens=0, q=None, k=None, positions_ptr=None, q_out_ptr=None, k_out_ptr=None)  # nothing to do
    _qk(n_q_heads=0, n_kv_heads=0, q=None, k=None, q_out_ptr=None, k_out_ptr=None)


def test_append_rope_refusals(lib):
    h = _create()
    try:
        for rows in (None, [0, 2]):
            with pytest.raises(B.DuoError) as e:
                B.duo_append_rope_rows(h, 0, rows, _rope(), _heads(), _heads(), _heads(), PTR, 2, PTR)
            assert e.value.name == "DUO_ERR_STATE"  # not bound
        for layer in (-1, 2):
            assert lib.duo_append_rope(h, layer, _rope(), _heads(), _heads(), _heads(), PTR, 2, PTR, None) == 1
        assert lib.duo_append_rope(None, 0, _rope(), _heads(), _heads(), _heads(), PTR, 2, PTR, None) == 1
    finally:
        B.duo_cache_destroy(h)


def test_rotary_class_refusals():
    f = torch.ones(32)
    for kw in (dict(head_dim=96), dict(mscale=0.0), dict(mscale=float("nan")), dict(eps=-1.0),
               dict(inv_freq=f.double()), dict(inv_freq=torch.ones(12)), dict(inv_freq=torch.ones(72)),
               dict(inv_freq=torch.ones(4, 8)), dict(inv_freq=f),  # a CPU tensor
               dict(inv_freq=None, q_norm=torch.ones(128)), dict(inv_freq=None, k_norm=torch.ones(64))):
        with pytest.raises(ValueError):
            RT.Rotary(**{**dict(inv_freq=None, head_dim=128), **kw})
    r = RT.Rotary(None, 128)
    assert r.rot_dim == 0
    x = torch.zeros(3, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        RT.qk_norm_rope(r, x, x)  # CPU tensors
    with pytest.raises(ValueError):
        RT.qk_norm_rope(r, x.half(), x.half())
    with pytest.raises(ValueError):
        RT.qk_norm_rope(r, x[0], x[0])


def test_heads_view_strides():
    """Views of a projection's output are taken; others are refused."""
    d = torch.device("cpu")
    x = torch.zeros(3, 5, 10, 128, dtype=torch.bfloat16)

    def view(t, dtype=torch.bfloat16):
        h = RT.heads_view(t, tuple(t.shape), "x", dtype, d)
        return h.token_stride, h.head_stride
    assert view(x) == (1280, 128)
    assert view(x[:, :, 2:6]) == (1280, 128)
    assert view(x[:, 2:3]) == (6400, 128)              # one token a row: the rows' stride
    assert view(x[:, :, ::2]) == (1280, 256)
    assert view(x[:1, :, 3:4]) == (1280, 128)          # (one head: its stride is not used)
    assert view(x[:1, :1, :, :].expand(1, 1, 10, 128)) == (6400, 128)
    assert view(x[0]) == (1280, 128) and view(x[0, :1].as_strided((1, 10, 128), (7, 128, 1))) == (0, 128)
    assert view(x.as_strided((2, 3, 1, 128), (3840, 1280, 5, 1))) == (1280, 0)
    assert view(x.view(3, 5, 2, 5, 128)[:, :, 0].unsqueeze(1)) == (1280, 128)
    assert view(x.transpose(1, 2)[:1]) == (128, 1280)
    for bad in (x[:, 1:], x[:, ::2], x.transpose(0, 1), x[..., :64].transpose(2, 3),
                x.flatten()[1:1 + 2 * 1280].view(2, 10, 128)):
        with pytest.raises(ValueError):
            RT.heads_view(bad, tuple(bad.shape), "x", torch.bfloat16, d)
    with pytest.raises(ValueError):
        view(x, torch.float32)
    with pytest.raises(TypeError):
        RT.heads_view(None, (1, 2, 3), "x", torch.float32, d)
    with pytest.raises(ValueError):
        RT.heads_view(x, (3, 5, 10, 64), "x", torch.bfloat16, d)
    with pytest.raises(ValueError):
        RT.heads_view(x, tuple(x.shape), "x", torch.bfloat16, torch.device("meta"))


def test_desc_struct_sizes():
    """The ctypes structures have the header's layout (64-bit pointers)."""
    assert ctypes.sizeof(B.duo_heads) == 24 and ctypes.sizeof(B.duo_rope_desc) == 40
