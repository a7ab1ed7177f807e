"""Norm and position rotation of queries and keys (``duo_qk_norm_rope``), and
the description of it that ``DuoCache.append_rope`` takes.

PyTorch is used for device memory and streams only; the arithmetic runs in the
library's kernels.
"""

import contextlib
import ctypes

import torch

from . import binding as B

_DTYPE = {torch.bfloat16: "bf16", torch.float32: "f32"}


@contextlib.contextmanager
def on_device(device, stream):
    """Make ``device`` (and ``stream``, so that outputs allocated inside belong
    to it) current for a call; yields the stream's handle."""
    if stream is None and device.index == torch.cuda.current_device():
        yield torch.cuda.current_stream(device).cuda_stream
        return
    with torch.cuda.device(device):
        s = stream if stream is not None else torch.cuda.current_stream(device)
        with torch.cuda.stream(s):
            yield s.cuda_stream


def heads_view(t, shape, name, dtype, device):
    """``duo_heads`` of t, a [..., heads, head_dim] view whose leading
    dimensions lie at one stride; raises for what the kernels cannot take."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.dtype != dtype:
        raise ValueError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.numel() == 0:  # nothing to read
        return B.duo_heads(None, 0, 0)
    st = t.stride()
    if st[-1] != 1 and shape[-1] > 1:
        raise ValueError("%s must have contiguous channels" % name)
    # one stride for all tokens: the innermost leading dimension's, which the
    # outer ones have to continue
    tok, count = 0, 1
    for size, stride in zip(reversed(shape[:-2]), reversed(st[:-2])):
        if size == 1:
            continue
        if count == 1:
            tok = stride
        elif stride != tok * count:
            raise ValueError("%s: its tokens must lie at one stride" % name)
        count *= size
    head = st[-2] if shape[-2] > 1 else 0
    step = 16 // t.element_size()
    if t.data_ptr() % 16 or tok % step or head % step:
        raise ValueError("%s must start at, and its tokens and heads lie at, multiples of 16 bytes" % name)
    return B.duo_heads(t.data_ptr(), tok, head)


class Rotary:
    """Per-head RMS norm and position rotation of queries and keys.

    inv_freq: float32 CUDA tensor [rot_dim / 2], radians per position of each
    pair (any frequency scaling is in it); None or empty: no rotation.
    interleaved: pairs (2j, 2j + 1) instead of (j, j + rot_dim / 2).
    mscale: factor on the rotation.  q_norm, k_norm: RMS-norm weights
    [head_dim] in the tensors' type, or None.  The tensors are kept alive here.
    """

    def __init__(self, inv_freq, head_dim, interleaved=False, mscale=1.0, q_norm=None, k_norm=None,
                 eps=1e-6):
        if head_dim not in (64, 128):
            raise ValueError("head_dim must be 64 or 128")
        if inv_freq is not None and inv_freq.numel():
            if inv_freq.dtype != torch.float32 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
                raise ValueError("inv_freq must be a contiguous float32 vector")
            if inv_freq.numel() % 8 or 2 * inv_freq.numel() > head_dim:
                raise ValueError("rot_dim must be a multiple of 16 and at most head_dim")
            if inv_freq.device.type != "cuda":
                raise ValueError("inv_freq must be a CUDA tensor")
        else:
            inv_freq = None
        for name, w in (("q_norm", q_norm), ("k_norm", k_norm)):
            if w is not None and (tuple(w.shape) != (head_dim,) or not w.is_contiguous()
                                  or w.device.type != "cuda"):
                raise ValueError("%s must be a contiguous CUDA vector of head_dim weights" % name)
        if not mscale > 0 or not eps >= 0:
            raise ValueError("mscale must be positive and eps not negative")
        self.head_dim, self.rot_dim = head_dim, 0 if inv_freq is None else 2 * inv_freq.numel()
        self.inv_freq, self.q_norm, self.k_norm = inv_freq, q_norm, k_norm

        def ptr(t):
            return None if t is None else t.data_ptr()

        self._desc = B.duo_rope_desc(self.rot_dim, int(bool(interleaved)), ptr(inv_freq),
                                     float(mscale), float(eps), ptr(q_norm), ptr(k_norm))

    def desc(self, dtype, device):
        """The C description, for tensors of dtype on device."""
        for name, t in (("inv_freq", self.inv_freq), ("q_norm", self.q_norm), ("k_norm", self.k_norm)):
            if t is None:
                continue
            if t.device != device:
                raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
            if name != "inv_freq" and t.dtype != dtype:
                raise ValueError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
        return self._desc


def qk_norm_rope(rotary, q, k, positions=None, q_out=None, k_out=None, stream=None):
    """Norm and rotate q [..., n_q_heads, head_dim] and k [..., n_kv_heads,
    head_dim] (either may be None) of the same tokens, at int64 positions of
    the leading shape.  q and k may be strided views (slices of a projection's
    output) whose tokens lie at one stride.  Returns (q_out, k_out), dense."""
    ref = q if q is not None else k
    if not isinstance(ref, torch.Tensor) or ref.dim() < 3:
        raise ValueError("q or k must be a [..., heads, head_dim] tensor")
    dtype, device, lead = ref.dtype, ref.device, tuple(ref.shape[:-2])
    if dtype not in _DTYPE:
        raise ValueError("q and k must be bfloat16 or float32")
    if device.type != "cuda":
        raise ValueError("q and k must be CUDA tensors")
    desc = rotary.desc(dtype, device)
    n = 1
    for size in lead:
        n *= size
    if positions is not None:
        if (not isinstance(positions, torch.Tensor) or positions.dtype != torch.int64
                or positions.device != device or tuple(positions.shape) != lead
                or not positions.is_contiguous()):
            raise ValueError("positions must be a contiguous int64 tensor %s on %s" % (lead, device))
    elif rotary.rot_dim:
        raise ValueError("positions are needed to rotate")
    with on_device(device, stream) as s:
        views, outs, heads = [], [], []
        for name, t, out in (("q", q, q_out), ("k", k, k_out)):
            if t is None:
                if out is not None:
                    raise ValueError("%s_out without %s" % (name, name))
                views.append(None), outs.append(None), heads.append(0)
                continue
            shape = lead + (t.shape[-2] if t.dim() == ref.dim() else -1, rotary.head_dim)
            views.append(heads_view(t, shape, name, dtype, device))
            if out is None:
                out = torch.empty(shape, dtype=dtype, device=device)
            elif (out.device != device or tuple(out.shape) != shape or out.dtype != dtype
                  or not out.is_contiguous()):
                raise ValueError("%s_out must be a contiguous %s tensor %s on %s" % (name, dtype, shape, device))
            outs.append(out)
            heads.append(t.shape[-2])
        B.duo_qk_norm_rope(desc, _DTYPE[dtype], n, heads[0], heads[1], rotary.head_dim, views[0],
                           views[1], None if positions is None else positions.data_ptr(),
                           None if outs[0] is None else outs[0].data_ptr(),
                           None if outs[1] is None else outs[1].data_ptr(), s)
    return outs[0], outs[1]
