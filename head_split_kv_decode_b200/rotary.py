"""Norm and position rotation of queries and keys (``duo_qk_norm_rope``), and
the description of it that ``DuoCache.append_rope`` takes.

PyTorch is used for device memory and streams only; the arithmetic runs in the
library's kernels.
"""

import torch

from . import binding as B

_DTYPE = {torch.bfloat16: B.DUO_BF16, torch.float32: B.DUO_F32}
_BYTES = {torch.bfloat16: 2, torch.float32: 4}


def run_on(device, stream, call):
    """call(stream handle) with ``device``, and ``stream`` (default the
    device's current one), current: what it allocates belongs to that stream."""
    if stream is None and device.index == torch._C._cuda_getDevice():
        return call(torch._C._cuda_getCurrentRawStream(device.index))
    with torch.cuda.device(device):
        s = stream if stream is not None else torch.cuda.current_stream(device)
        with torch.cuda.stream(s):
            return call(s.cuda_stream)


def heads_view(t, shape, name, dtype, device):
    """``duo_heads`` of t, a [..., heads, head_dim] view whose leading
    dimensions lie at one stride; raises for what the kernels cannot take."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.dtype is not dtype:
        raise ValueError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    ptr, st = t.data_ptr(), t.stride()
    if ptr == 0:  # nothing to read
        return B.duo_heads(None, 0, 0)
    if st[-1] != 1:
        raise ValueError("%s must have contiguous channels" % name)
    size = _BYTES[dtype]
    # the usual forms first: [tokens, heads, d] and [rows, tokens, heads, d]
    head = st[-2]
    if len(st) == 3:
        tok = st[0]
    elif len(st) == 4 and (shape[1] == 1 or st[0] == st[1] * shape[1]):
        tok = st[0] if shape[1] == 1 else st[1]
    else:
        tok = 1  # not aligned: the general form below
    if not (ptr | tok * size | head * size) & 15:
        return B.duo_heads(ptr, tok, head)
    # one stride for all tokens: the innermost leading dimension's, which the
    # outer ones have to continue; dimensions of size 1 have none
    tok, count = 0, 1
    for i in range(len(shape) - 3, -1, -1):
        if shape[i] == 1:
            continue
        if count == 1:
            tok = st[i]
        elif st[i] != tok * count:
            raise ValueError("%s: its tokens must lie at one stride" % name)
        count *= shape[i]
    if shape[-2] == 1:
        head = 0
    if (ptr | tok * size | head * size) & 15:
        raise ValueError("%s must start at, and its tokens and heads lie at, multiples of 16 bytes" % name)
    return B.duo_heads(ptr, tok, head)


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
        self._checked = None  # the last (dtype, device) found right

    def desc(self, dtype, device):
        """The C description, for tensors of dtype on device."""
        if self._checked == (dtype, device):
            return self._desc
        for name, t in (("inv_freq", self.inv_freq), ("q_norm", self.q_norm), ("k_norm", self.k_norm)):
            if t is None:
                continue
            if t.device != device:
                raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
            if name != "inv_freq" and t.dtype != dtype:
                raise ValueError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
        self._checked = dtype, device
        return self._desc


def qk_norm_rope(rotary, q, k, positions=None, q_out=None, k_out=None, stream=None):
    """Norm and rotate q [..., n_q_heads, head_dim] and k [..., n_kv_heads,
    head_dim] (either may be None) of the same tokens, at int64 positions of
    the leading shape.  q and k may be strided views (slices of a projection's
    output) whose tokens lie at one stride.  Returns (q_out, k_out), dense."""
    ref = q if q is not None else k
    if not isinstance(ref, torch.Tensor) or ref.dim() < 3:
        raise ValueError("q or k must be a [..., heads, head_dim] tensor")
    dtype, device, lead = ref.dtype, ref.device, ref.shape[:-2]
    kind = _DTYPE.get(dtype)
    if kind is None:
        raise ValueError("q and k must be bfloat16 or float32")
    if device.type != "cuda":
        raise ValueError("q and k must be CUDA tensors")
    desc = rotary.desc(dtype, device)
    pos_ptr = None
    if positions is not None:
        if (not isinstance(positions, torch.Tensor) or positions.dtype is not torch.int64
                or positions.device != device or positions.shape != lead
                or not positions.is_contiguous()):
            raise ValueError("positions must be a contiguous int64 tensor %s on %s" % (tuple(lead), device))
        pos_ptr = positions.data_ptr()
    elif rotary.rot_dim:
        raise ValueError("positions are needed to rotate")

    def call(handle):
        qh, qo, qp, nq = _side("q", q, q_out, lead, rotary.head_dim, dtype, device)
        kh, ko, kp, nk = _side("k", k, k_out, lead, rotary.head_dim, dtype, device)
        B.duo_qk_norm_rope(desc, kind, lead.numel(), nq, nk, rotary.head_dim, qh, kh, pos_ptr, qp, kp,
                           handle)
        return qo, ko

    return run_on(device, stream, call)


def _side(name, t, out, lead, head_dim, dtype, device):
    """(view, output, its pointer, heads) of q or k; the output is allocated when not given."""
    if t is None:
        if out is not None:
            raise ValueError("%s_out without %s" % (name, name))
        return None, None, None, 0
    heads = t.shape[-2] if t.dim() > 1 else 0
    shape = lead + (heads, head_dim)
    view = heads_view(t, shape, name, dtype, device)
    if out is None:
        out = t.new_empty(shape)
    elif out.device != device or out.shape != shape or out.dtype is not dtype or not out.is_contiguous():
        raise ValueError("%s_out must be a contiguous %s tensor %s on %s" % (name, dtype, tuple(shape), device))
    return view, out, out.data_ptr(), heads
