"""The 8-bit pre-fill at run counts of the test's own choice: one, two, as many
as there are key tiles, and more than a short row has."""

import numpy as np
import pytest
import torch

from head_split_kv_decode_b200 import binding as B
from head_split_kv_decode_b200 import synth
from head_split_kv_decode_b200.cache import DuoCache
from oracle import attention as OA
from oracle import fp8 as OF

from _util import assert_parity, f64, seeded_mask

pytestmark = pytest.mark.gpu

BF, D = torch.bfloat16, 128
S, R = 4, 60


def _plain(seed, n, heads):
    return synth.kv_field(seed, [0], range(n), heads, D, device="cuda")[0].to(BF)


def _history(x, mask):
    return np.where(mask.numpy().astype(bool)[None, :, None], OF.held(f64(x))[0], f64(x))


@pytest.mark.parametrize("lens,C,hq,hkv,n_ret", [
    ([700], 5, 2, 2, 1), ([1000, 33, 0], 130, 4, 4, 2), ([129], 257, 3, 1, 1)])
def test_forced_runs(cuda_lib, lens, C, hq, hkv, n_ret):
    """The same outputs, against the oracle, at every run count; a NaN key of
    the history, wherever its run ends, reaches every query of its head."""
    batch = len(lens)
    mask = seeded_mask(1, hkv, n_ret)
    cache = DuoCache(1, batch, hq, hkv, D, "fp8", max(lens) + C, mask[None], S, R)
    K = [_plain(10 + b, n + C, hkv) for b, n in enumerate(lens)]
    V = [_plain(20 + b, n + C, hkv) for b, n in enumerate(lens)]
    q = torch.stack([_plain(30 + b, C, hq) for b in range(batch)])
    chunk = [torch.stack([x[n:] for x, n in zip(X, lens)]) for X in (K, V)]
    cache._prefill_ws()
    ref = []
    for b, h in enumerate(lens):
        kh, vh = (np.concatenate([_history(x[:h], mask), f64(x[h:])]) for x in (K[b], V[b]))
        ref.append(OA.prefill_reference(f64(q[b])[None], kh[None], vh[None], h, mask.numpy(), S, R))
    head = int(np.flatnonzero(mask.numpy())[0])
    g = hq // hkv
    tiles = -(-max(lens) // 128) + -(-C // 128)
    for nan in (False, True):
        cache.release_rows()
        for b, n in enumerate(lens):
            if n:
                k = K[b][None, :n].clone()
                if nan and b == 0:
                    k[0, n // 2, head, 3] = float("nan")
                cache.append_rows(0, [b], k, V[b][None, :n])
        for runs in sorted({1, 2, 3, tiles - 1, tiles, tiles + 5, 296}):
            B.duo_test_force_prefill_runs(cache.handle, runs)
            cache._pf_ws.fill_(0xFF)
            out = cache.prefill(0, q, *chunk)
            torch.cuda.synchronize()
            assert B.duo_poll_device_error() == 0
            if nan:
                part = out[0, :, head * g:(head + 1) * g]
                assert part.isnan().all(), "%d runs" % runs
                part[:] = torch.from_numpy(ref[0][0][:, head * g:(head + 1) * g]).to(part)
            for b in range(batch):
                assert_parity(out[b:b + 1], ref[b], "bf16", "row %d, %d runs" % (b, runs))
