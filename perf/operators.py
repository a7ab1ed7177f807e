"""Cases of the rotary and 8-bit cache operators, in plain torch and through the framework.

Four calls of a serving loop, between the QKV projection and the attention output:

- ``qk_norm_rope``: per-head RMS norm of queries and keys with the position rotation;
- ``append_rope``: append of a step's or a prompt's K/V to the head-split cache, K normed and
  rotated on the way, with the same tokens' queries;
- ``decode_fp8``: single-token attention over an 8-bit cache (e4m3 codes, one power-of-two scale
  per 32 tokens and KV head; the newest, unfinished block in bf16; streaming heads in bf16);
- ``prefill_fp8``: a chunk's attention over an 8-bit cache's history and the chunk itself.

A cache here has ``n_ret`` retrieval KV heads (the first ones) that keep every token, and the
rest streaming: ``S`` sinks and a ring of the ``R`` newest tokens.
"""

import math

import torch

own = False

BLOCK = 32       # tokens of one scale of the 8-bit cache
PAGE = 256       # tokens of one block of the paged layout
THETA = 500000.0
EPS = 1e-6
E4M3_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases


def _rope(name, tokens, hq, hkv, d, dtype, rot, interleaved, norm, start):
    return {"name": name, "op": "qk_norm_rope", "tokens": tokens, "hq": hq, "hkv": hkv, "d": d,
            "dtype": dtype, "rot": rot, "interleaved": interleaved, "norm": norm, "start": start}


def _append(name, kv, paged, batch, tokens, hq, hkv, n_ret, d, rot, norm, start, S, R):
    return {"name": name, "op": "append_rope", "kv": kv, "paged": paged, "batch": batch,
            "tokens": tokens, "hq": hq, "hkv": hkv, "n_ret": n_ret, "d": d, "rot": rot,
            "norm": norm, "start": start, "S": S, "R": R}


def _decode(name, paged, batch, shortest, longest, hq, hkv, n_ret, S, R):
    return {"name": name, "op": "decode_fp8", "paged": paged, "batch": batch,
            "shortest": shortest, "longest": longest, "hq": hq, "hkv": hkv, "n_ret": n_ret,
            "S": S, "R": R}


def _prefill(name, batch, history, chunk, hq, hkv, n_ret, S, R):
    return {"name": name, "op": "prefill_fp8", "batch": batch, "history": history, "chunk": chunk,
            "hq": hq, "hkv": hkv, "n_ret": n_ret, "S": S, "R": R}


def listed():
    return [
        # one decoded token of one sequence: pure latency
        _rope("rope 1 token", 1, 32, 8, 128, "bf16", 128, False, True, 131071),
        # a pre-fill chunk of a GQA model late in a 128K prompt, q and k as slices of the projection's output
        _rope("rope chunk 4096 gqa", 4096, 32, 8, 128, "bf16", 128, False, True, 120000),
        # a float32 MHA model with a partial, interleaved rotation and no norm, an odd prompt
        _rope("rope 777 f32 d64", 777, 8, 8, 64, "f32", 32, True, False, 0),
        # a decode step of 8 sequences at far positions into a paged bf16 cache
        _append("append step 8 paged bf16", "bf16", True, 8, 1, 32, 8, 4, 128, 128, True, 60001, 64, 256),
        # a long prompt's chunk into a paged 8-bit cache
        _append("append 8192 paged fp8", "fp8", True, 1, 8192, 32, 8, 4, 128, 128, True, 0, 64, 256),
        # four odd-sized prompts at once into a packed bf16 cache, without norms
        _append("append 4x1777 bf16", "bf16", False, 4, 1777, 32, 32, 8, 128, 128, False, 0, 64, 256),
        # a short chat on one sequence: few splits, latency
        _decode("decode 300 fp8", False, 1, 300, 300, 32, 8, 4, 64, 256),
        # the long-context GQA step
        _decode("decode gqa 128k fp8", False, 1, 131075, 131075, 32, 8, 4, 64, 256),
        # the MHA step: many streaming heads
        _decode("decode mha 32k fp8", False, 1, 32768, 32768, 32, 32, 8, 64, 256),
        # a served batch of sequences of mixed lengths, paged
        _decode("decode paged 8x2k-64k fp8", True, 8, 2048, 65536, 32, 8, 4, 64, 256),
        # one million tokens, a quarter of the heads with full history
        _decode("decode gqa 1m fp8", False, 1, 1048576, 1048576, 32, 8, 2, 64, 256),
        # a chunk in the middle of a pre-fill on the 8-bit cache
        _prefill("prefill 1000 on 15000 fp8", 1, 15000, 1000, 32, 8, 4, 64, 256),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk_norm_rope", "append_rope", "decode_fp8", "decode_fp8", "prefill_fp8"])
    hkv = rng.choice([1, 2, 4, 8, 8, 16])
    hq = hkv * rng.choice([1, 2, 4, 4, 8] if hkv <= 8 else [1, 2])
    n_ret = rng.randint(0 if op == "append_rope" else 1, hkv)
    S, R = rng.choice([(64, 256), (4, 64), (0, 100), (16, 1000)])
    if op == "qk_norm_rope":
        dtype, d = rng.choice(["bf16", "bf16", "f32"]), rng.choice([128, 128, 64])
        c = _rope("", _log(rng, 1, 5000), hq, hkv, d, dtype, rng.choice([d, d, d // 2, d // 4]),
                  rng.random() < 0.3, rng.random() < 0.6, rng.choice([0, rng.randint(0, 1000000)]))
    elif op == "append_rope":
        kv = rng.choice(["bf16", "fp8", "fp8", "f32"])
        paged = kv != "f32" and rng.random() < 0.6
        d = 128 if kv == "fp8" or paged else rng.choice([64, 128])
        total = _log(rng, 1, 8192)
        batch = min(rng.choice([1, 1, 3, 8, 40]), total)
        c = _append("", kv, paged, batch, max(1, total // batch), hq, hkv, n_ret, d,
                    rng.choice([d, d, d // 2]), rng.random() < 0.6,
                    rng.choice([0, rng.randint(0, 1000000)]), S, R)
    elif op == "decode_fp8":
        batch = rng.choice([1, 1, 1, 2, 5, 16])
        longest = _log(rng, 1, min(400000, 1500000 // (batch * n_ret)))
        c = _decode("", rng.random() < 0.5, batch, max(1, int(longest * rng.choice([1.0, 0.5, 0.03]))),
                    longest, hq, hkv, n_ret, S, R)
    else:
        chunk = _log(rng, 1, 1000)
        chunk = max(1, min(chunk, 16000 // (n_ret * (hq // hkv))))
        c = _prefill("", 1, _log(rng, 1, 15000), chunk, hq, hkv, n_ret, S, R)
    del c["name"]
    return c


def _lengths(c):
    """The rows' lengths of a decode case: from the shortest to the longest, in geometric steps."""
    b, lo, hi = c["batch"], c["shortest"], c["longest"]
    if b == 1:
        return [hi]
    return [int(round(lo * (hi / lo) ** (i / (b - 1)))) for i in range(b)]


# ------------------------------------------------------------------ inputs


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _inv_freq(rot):
    i = torch.arange(0, rot, 2, dtype=torch.float64, device="cuda")
    return (THETA ** (-i / max(rot, 1))).to(torch.float32)


def _norm_weight(gen, c, dtype):
    if not c["norm"]:
        return None
    return (1.0 + 0.2 * _randn(gen, c["d"])).to(dtype)


def _kv_history(gen, batch, heads, tokens, d):
    """K or V [batch, heads, tokens, d] in bf16, every 100th channel ten times the others'."""
    x = _randn(gen, batch, heads, tokens, d).to(torch.bfloat16)
    x[..., ::100] *= 10.0
    return x


def _decode_inputs(c, seed):
    """Lengths, q [batch, hq, d] and, per KV head, K and V of the longest row's tokens."""
    gen = _generator(seed)
    lens = _lengths(c)
    q = (1.5 * _randn(gen, c["batch"], c["hq"], 128)).to(torch.bfloat16)
    n = max(lens)
    ret = [_kv_history(gen, c["batch"], c["n_ret"], n, 128) for _ in range(2)]
    # streaming heads: the first and the last tokens are all that is ever kept
    few = min(n, 2 * (c["S"] + c["R"]))
    stream = [_kv_history(gen, c["batch"], c["hkv"] - c["n_ret"], few, 128) for _ in range(2)]
    return lens, q, ret, stream


def _prefill_inputs(c, seed):
    gen = _generator(seed)
    n = c["history"] + c["chunk"]
    k, v = (_kv_history(gen, c["batch"], c["hkv"], n, 128) for _ in range(2))
    q = (1.5 * _randn(gen, c["batch"], c["chunk"], c["hq"], 128)).to(torch.bfloat16)
    return q, k, v


def _projection(c, seed, tokens, dtype):
    """What a QKV projection leaves: [tokens, (hq + 2 hkv) * d]; q, k and v are slices of it."""
    gen = _generator(seed)
    x = (1.3 * _randn(gen, tokens, (c["hq"] + 2 * c["hkv"]) * c["d"])).to(dtype)
    x = x.view(tokens, c["hq"] + 2 * c["hkv"], c["d"])
    q, k, v = x[:, :c["hq"]], x[:, c["hq"]:c["hq"] + c["hkv"]], x[:, c["hq"] + c["hkv"]:]
    weights = _norm_weight(gen, c, dtype), _norm_weight(gen, c, dtype)
    return q, k, v, weights


def _mask(c):
    return [1] * c["n_ret"] + [0] * (c["hkv"] - c["n_ret"])


def _slot(p, S, R):
    return torch.where(p < S, p, S + (p - S) % R)


# ------------------------------------------------------------------ the plain 8-bit cache


def _quantise(x):
    """x [batch, heads, blocks * BLOCK, d] -> (codes as float8, scales [batch, heads, blocks])."""
    y = x.float().unflatten(2, (-1, BLOCK))
    top = torch.where(y.isfinite(), y.abs(), torch.zeros_like(y)).amax((-1, -2))
    m, e = torch.frexp(top)  # top = m * 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(top > 0, e - 9 + (m > 0.875).int(), torch.full_like(e, -120)).clamp(min=-120)
    scale, inverse = (((127 + x) << 23).view(torch.float32) for x in (e, -e))  # exact powers of two
    z = (y * inverse[..., None, None]).clamp(-E4M3_MAX, E4M3_MAX)
    return z.to(torch.float8_e4m3fn).flatten(2, 3), scale


def _plain_cache(c, lens, ret, stream_kept):
    """The 8-bit cache as plain tensors: codes and scales of the full blocks, the open blocks."""
    n = torch.tensor(lens, device="cuda")
    full = n // BLOCK * BLOCK
    at = full[:, None] + torch.arange(BLOCK, device="cuda")            # the open block's positions
    blocks = max(lens) // BLOCK
    out = {"n": n, "full": full, "stream": stream_kept}
    for name, x in zip(("k", "v"), ret):
        codes, scale = _quantise(x[:, :, :blocks * BLOCK])
        idx = at.clamp(max=x.shape[2] - 1)[:, None, :, None].expand(-1, x.shape[1], -1, x.shape[3])
        out[name] = codes, scale, x.gather(2, idx)
    return out


# ------------------------------------------------------------------ prepare


def prepare(case, seed):
    c = dict(case)
    return {"qk_norm_rope": _prepare_rope, "append_rope": _prepare_append,
            "decode_fp8": _prepare_decode, "prefill_fp8": _prepare_prefill}[c["op"]](c, seed)


def _prepare_rope(c, seed):
    q, k, _, (wq, wk) = _projection(c, seed, c["tokens"], TYPES[c["dtype"]])
    pos = c["start"] + torch.arange(c["tokens"], dtype=torch.int64, device="cuda")
    st = {"c": c, "q": q, "k": k, "pos": pos, "freq": _inv_freq(c["rot"]), "wq": wq, "wk": wk}
    if own:
        st["rotary"] = _rotary(st)
    return st


def _rotary(st):
    from head_split_kv_decode_b200.rotary import Rotary
    c = st["c"]
    return Rotary(st["freq"], c["d"], interleaved=c.get("interleaved", False), q_norm=st["wq"],
                  k_norm=st["wk"], eps=EPS)


def _prepare_append(c, seed):
    dtype = TYPES["f32" if c["kv"] == "f32" else "bf16"]
    b, n = c["batch"], c["tokens"]
    q, k, v, (wq, wk) = _projection(c, seed, b * n, dtype)
    q, k, v = (x.unflatten(0, (b, n)) for x in (q, k, v))
    pos = c["start"] + torch.arange(n, dtype=torch.int64, device="cuda").expand(b, n).contiguous()
    st = {"c": c, "q": q, "k": k, "v": v, "pos": pos, "freq": _inv_freq(c["rot"]), "wq": wq, "wk": wk}
    pages = -(-n // PAGE)
    if own:
        from head_split_kv_decode_b200.cache import DuoCache
        st["rotary"] = _rotary(st)
        st["cache"] = DuoCache(1, b, c["hq"], c["hkv"], c["d"], c["kv"], n, _mask(c), c["S"], c["R"],
                               pool_blocks=b * pages if c["paged"] else None)
        st["rows"] = list(range(b - 1, -1, -1))
        return st
    # plain buffers of the same layout
    S, R, n_ret, n_str = c["S"], c["R"], c["n_ret"], c["hkv"] - c["n_ret"]
    rows = PAGE if c["paged"] else (n if c["kv"] != "fp8" else -(-n // 128) * 128)
    outer = b * pages if c["paged"] else b
    st["table"] = torch.arange(b * pages, device="cuda").view(b, pages) if c["paged"] else None

    def zeros(*shape, t=dtype):
        return torch.zeros(*shape, dtype=t, device="cuda")

    kind = torch.uint8 if c["kv"] == "fp8" else dtype
    for name in ("k", "v"):
        st["ret_" + name] = zeros(outer, n_ret, rows, c["d"], t=kind)
        st["str_" + name] = zeros(b, n_str, S + R, c["d"])
        if c["kv"] == "fp8":
            st["scale_" + name] = zeros(outer, n_ret, rows // BLOCK, t=torch.float32)
            st["tail_" + name] = zeros(b, n_ret, BLOCK, c["d"])
    return st


def _prepare_decode(c, seed):
    lens, q, ret, stream = _decode_inputs(c, seed)
    st = {"c": c, "q": q}
    n_str = c["hkv"] - c["n_ret"]
    S, R = c["S"], c["R"]
    few = stream[0].shape[2]
    if own:
        from head_split_kv_decode_b200.cache import DuoCache
        pages = sum(-(-n // PAGE) for n in lens)
        cache = DuoCache(1, c["batch"], c["hq"], c["hkv"], 128, "fp8", max(lens), _mask(c), S, R,
                         pool_blocks=pages if c["paged"] else None)
        for b, n in enumerate(lens):
            for at in range(0, n, 65536):
                end = min(n, at + 65536)
                # a streaming head's tokens repeat with the period of what is made of them
                p = torch.arange(at, end, device="cuda")
                src = torch.where(p < S, p, few - 1 - (n - 1 - p) % max(1, few - S)).clamp(min=0)
                kv = [torch.cat([r[b, :, at:end], s[b][:, src]], 0).transpose(0, 1)[None].contiguous()
                      for r, s in zip(ret, stream)]
                cache.append_rows(0, [b], *kv)
        st["cache"] = cache
        return st
    n = torch.tensor(lens, device="cuda")
    j = torch.arange(S + R, device="cuda")
    # the window of each row: sinks, then the R newest positions (those past the sinks)
    p = torch.where(j < S, j, n[:, None] - 1 - (j - S))
    seen = torch.where(j < S, p < n[:, None], p >= S)
    src = torch.where(p < S, p, few - 1 - (n[:, None] - 1 - p) % max(1, few - S)).clamp(min=0)
    idx = src[:, None, :, None].expand(-1, n_str, -1, 128)
    kept = [x.gather(2, idx.clamp(max=few - 1)) for x in stream], seen
    st["cache"] = _plain_cache(c, lens, ret, kept)
    return st


def _prepare_prefill(c, seed):
    q, k, v = _prefill_inputs(c, seed)
    h, n = c["history"], c["history"] + c["chunk"]
    kc, vc = (x[:, :, h:].transpose(1, 2).contiguous() for x in (k, v))
    st = {"c": c, "q": q, "k": kc, "v": vc}
    if own:
        from head_split_kv_decode_b200.cache import DuoCache
        cache = DuoCache(1, c["batch"], c["hq"], c["hkv"], 128, "fp8", n, _mask(c), c["S"], c["R"])
        cache.append(0, *(x[:, :, :h].transpose(1, 2).contiguous() for x in (k, v)))
        st["cache"] = cache
        return st
    r = c["n_ret"]
    st["cache"] = _plain_cache(c, [h] * c["batch"], [x[:, :r, :h] for x in (k, v)], None)
    # streaming heads: the sinks and the newest R tokens, by position
    p = torch.cat([torch.arange(min(c["S"], h), device="cuda"),
                   torch.arange(min(h, max(c["S"], h - c["R"])), h, device="cuda")])
    st["window"] = p, k[:, r:, p], v[:, r:, p]
    return st


# ------------------------------------------------------------------ run


def run(state):
    op = state["c"]["op"]
    if own:
        return _own(state, op)
    if op == "qk_norm_rope":
        c = state["c"]
        return (_plain_rope(c, state["q"], state["pos"], state["freq"], state["wq"]),
                _plain_rope(c, state["k"], state["pos"], state["freq"], state["wk"]))
    if op == "append_rope":
        return _plain_append(state)
    if op == "decode_fp8":
        return _plain_decode(state)
    return _plain_prefill(state)


def _own(st, op):
    if op == "qk_norm_rope":
        from head_split_kv_decode_b200.rotary import qk_norm_rope
        return qk_norm_rope(st["rotary"], st["q"], st["k"], st["pos"])
    cache = st["cache"]
    if op == "append_rope":
        cache.release_rows(st["rows"])  # new sequences take the slots
        q = cache.append_rope(0, st["rotary"], st["k"], st["v"], q=st["q"], positions=st["pos"])
        return _own_contents(st, q)
    if op == "decode_fp8":
        return cache.decode(0, st["q"])
    return cache.prefill(0, st["q"], st["k"], st["v"])


def _own_contents(st, q):
    c, cache = st["c"], st["cache"]
    io = st["k"].dtype
    kind = torch.float8_e4m3fn if c["kv"] == "fp8" else io
    out = {"q": q}
    for name in ("k", "v"):
        if c["n_ret"]:
            out["ret_" + name] = cache.region(0, "ret_" + name).view(kind)
            if c["kv"] == "fp8":
                out["scale_" + name] = cache.region(0, "ret_%s_sz" % name).view(torch.float32)[..., 0]
                out["tail_" + name] = cache.region(0, "tail_" + name).view(io)
        if c["n_ret"] < c["hkv"]:
            out["str_" + name] = cache.region(0, "str_" + name).view(io)
    return out


def _plain_rope(c, x, pos, freq, w):
    """x [..., heads, d] at pos [...], in 32 bits (the angles in 64), rounded once."""
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w.float()
    ang = pos[..., None].double() * freq.double()
    cos, sin = ang.cos().float()[..., None, :], ang.sin().float()[..., None, :]
    rot = c["rot"]
    if c.get("interleaved"):
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        z = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        z = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([z, y[..., rot:]], -1).to(x.dtype)


def _plain_append(st):
    c = st["c"]
    b, n, S, R, n_ret = c["batch"], c["tokens"], c["S"], c["R"], c["n_ret"]
    out = {"q": _plain_rope(c, st["q"], st["pos"], st["freq"], st["wq"])}
    kv = {"k": _plain_rope(c, st["k"], st["pos"], st["freq"], st["wk"]), "v": st["v"]}
    p = torch.arange(n, device="cuda")
    live = torch.cat([p[:min(S, n)], p[max(min(S, n), n - R):]])
    rows = torch.arange(b, device="cuda")
    full = n // BLOCK * BLOCK
    for name in ("k", "v"):
        x = kv[name].transpose(1, 2)                                  # [b, heads, n, d]
        if n_ret:
            ret = x[:, :n_ret]
            keep, codes, scale = n, ret, None
            if c["kv"] == "fp8":
                keep = full
                codes, scale = _quantise(ret[:, :, :full])
                codes = codes.view(torch.uint8)
                st["tail_" + name][:, :, :n - full] = ret[:, :, full:]
            at = p[:keep]
            if c["paged"]:
                page = st["table"][:, at // PAGE]                     # [b, keep]
                st["ret_" + name][page, :, (at % PAGE)[None]] = codes.transpose(1, 2)
                if scale is not None:
                    ab = torch.arange(full // BLOCK, device="cuda")
                    st["scale_" + name][st["table"][:, ab // (PAGE // BLOCK)], :,
                                        (ab % (PAGE // BLOCK))[None]] = scale.transpose(1, 2)
            else:
                st["ret_" + name][:, :, :keep] = codes
                if scale is not None:
                    st["scale_" + name][:, :, :full // BLOCK] = scale
            out["ret_" + name] = st["ret_" + name]
            if scale is not None:
                out["ret_" + name] = st["ret_" + name].view(torch.float8_e4m3fn)
                out["scale_" + name], out["tail_" + name] = st["scale_" + name], st["tail_" + name]
        if n_ret < c["hkv"]:
            st["str_" + name][rows[:, None], :, _slot(live, S, R)[None]] = x[:, n_ret:, live].transpose(1, 2)
            out["str_" + name] = st["str_" + name]
    return out


def _attend(q, k, v, seen):
    """q [b, heads, queries, d], k/v [b, heads, keys, d] in 32 bits; seen broadcasts to the scores."""
    s = q @ k.transpose(-1, -2) / math.sqrt(q.shape[-1])
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    p = torch.exp(s - s.amax(-1, keepdim=True))
    return (p @ v) / p.sum(-1, keepdim=True)


def _expand(cache):
    """K and V of the 8-bit cache's full blocks followed by the open block, in 32 bits."""
    kv = []
    for name in ("k", "v"):
        codes, scale, tail = cache[name]
        x = (codes.float().unflatten(2, (-1, BLOCK)) * scale[..., None, None]).flatten(2, 3)
        kv.append(torch.cat([x, tail.float()], 2))
    full, n = cache["full"], cache["n"]
    pos = torch.arange(kv[0].shape[2] - BLOCK, device="cuda")
    open_ = torch.arange(BLOCK, device="cuda")
    seen = torch.cat([pos < full[:, None], open_ < (n - full)[:, None]], 1)  # [b, keys]
    return kv[0], kv[1], seen


def _plain_decode(st):
    c, cache = st["c"], st["cache"]
    g = c["hq"] // c["hkv"]
    q = st["q"].float().unflatten(1, (c["hkv"], g))
    k, v, seen = _expand(cache)
    out = [_attend(q[:, :c["n_ret"]], k, v, seen[:, None, None])]
    if c["n_ret"] < c["hkv"]:
        (ks, vs), mask = cache["stream"]
        out.append(_attend(q[:, c["n_ret"]:], ks.float(), vs.float(), mask[:, None, None]))
    return torch.cat(out, 1).flatten(1, 2).to(st["q"].dtype)


def _plain_prefill(st):
    c = st["c"]
    r, h, n, g = c["n_ret"], c["history"], c["chunk"], c["hq"] // c["hkv"]
    q = st["q"].float().transpose(1, 2).unflatten(1, (c["hkv"], g)).flatten(2, 3)  # [b, hkv, g * n, d]
    kc, vc = st["k"].float().transpose(1, 2), st["v"].float().transpose(1, 2)
    i = (h + torch.arange(n, device="cuda")).repeat(g)[:, None]                    # query positions
    j = h + torch.arange(n, device="cuda")
    k, v, seen = _expand(st["cache"])
    mask = torch.cat([seen[0].expand(g * n, -1), j <= i], 1)
    out = [_attend(q[:, :r], torch.cat([k, kc[:, :r]], 2), torch.cat([v, vc[:, :r]], 2), mask)]
    if r < c["hkv"]:
        p, ks, vs = st["window"]
        p = torch.cat([p, j])
        mask = (p <= i) & ((p < c["S"]) | (i - p < c["R"]))
        out.append(_attend(q[:, r:], torch.cat([ks.float(), kc[:, r:]], 2),
                           torch.cat([vs.float(), vc[:, r:]], 2), mask))
    out = torch.cat(out, 1).unflatten(2, (g, n)).flatten(1, 2)                     # [b, hq, n, d]
    return out.transpose(1, 2).to(st["q"].dtype).contiguous()


# ------------------------------------------------------------------ work


def _ret_bytes(n, d, kv):
    """Bytes of K and V that one retrieval head holds of n tokens."""
    if kv == "fp8":
        full = n // BLOCK
        return 2 * (full * (BLOCK * d + 4) + (n - full * BLOCK) * d * 2)
    return 2 * n * d * (4 if kv == "f32" else 2)


def work(case):
    c = dict(case)
    if c["op"] == "qk_norm_rope":
        values = c["tokens"] * (c["hq"] + c["hkv"]) * c["d"]
        return {"bytes": 2 * values * (4 if c["dtype"] == "f32" else 2) + 8 * c["tokens"] + 2 * c["rot"],
                "flops": 7 * values}
    if c["op"] == "append_rope":
        b, n, d, io = c["batch"], c["tokens"], c["d"], 4 if c["kv"] == "f32" else 2
        live = min(n, c["S"]) + max(0, n - max(min(n, c["S"]), n - c["R"]))
        n_str = c["hkv"] - c["n_ret"]
        q = 2 * n * c["hq"] * d * io
        kv = c["n_ret"] * (2 * n * d * io + _ret_bytes(n, d, c["kv"])) + n_str * 4 * live * d * io
        return {"bytes": b * (q + kv + 8 * n) + 2 * c["rot"],
                "flops": b * 7 * d * (n * (c["hq"] + c["n_ret"]) + live * n_str)}
    g, n_str, W = c["hq"] // c["hkv"], c["hkv"] - c["n_ret"], c["S"] + c["R"]
    if c["op"] == "decode_fp8":
        lens = _lengths(c)
        kv = sum(c["n_ret"] * _ret_bytes(n, 128, "fp8") + n_str * min(n, W) * 512 for n in lens)
        keys = sum(c["n_ret"] * n + n_str * min(n, W) for n in lens)
        return {"bytes": kv + 2 * c["batch"] * c["hq"] * 128 * 2, "flops": 4 * 128 * g * keys}
    h, n = c["history"], c["chunk"]
    pairs = n * h + n * (n + 1) // 2
    # streaming: query i sees min(i + 1, S) sinks and the rest of its R newest keys
    seen = sum(min(i + 1, c["S"]) + max(0, min(i + 1, c["R"]) - max(0, min(i + 1, c["S"]) - max(0, i + 1 - c["R"])))
               for i in range(h, h + n))
    kv = c["n_ret"] * _ret_bytes(h, 128, "fp8") + n_str * min(h, W) * 512 + 4 * n * c["hkv"] * 128
    return {"bytes": c["batch"] * (kv + 4 * n * c["hq"] * 128),
            "flops": c["batch"] * 4 * 128 * g * (c["n_ret"] * pairs + n_str * seen)}


# ------------------------------------------------------------------ exact (64 bits, written apart)


def exact(case, seed):
    c = dict(case)
    if c["op"] == "qk_norm_rope":
        q, k, _, (wq, wk) = _projection(c, seed, c["tokens"], TYPES[c["dtype"]])
        pos = c["start"] + torch.arange(c["tokens"], device="cuda")
        return _exact_rope(c, q, pos, wq), _exact_rope(c, k, pos, wk)
    if c["op"] == "append_rope":
        return _exact_append(c, seed)
    if c["op"] == "decode_fp8":
        return _exact_decode(c, seed)
    return _exact_prefill(c, seed)


def _exact_rope(c, x, pos, w):
    """As complex numbers: pair i of a head times mscale e^{i angle}, mscale = 1."""
    y = x.to(torch.float64)
    if w is not None:
        norm = torch.linalg.vector_norm(y, dim=-1, keepdim=True) ** 2 / y.shape[-1]
        y = y / torch.sqrt(norm + EPS) * w.to(torch.float64)
    half = c["rot"] // 2
    inv = _inv_freq(c["rot"]).to(torch.float64)
    turn = torch.polar(torch.ones_like(inv), torch.outer(pos.reshape(-1).to(torch.float64), inv).remainder(2 * math.pi))
    turn = turn.view(*pos.shape, 1, half)
    first = list(range(0, c["rot"], 2)) if c.get("interleaved") else list(range(half))
    second = [i + 1 for i in first] if c.get("interleaved") else [i + half for i in first]
    z = torch.complex(y[..., first], y[..., second]) * turn
    out = y.clone()
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _power(e):
    """2^e in 64 bits for whole e: torch.pow on the GPU is off by an ulp at some of them."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_e4m3(x):
    """x [..., BLOCK, d] in 64 bits -> (the code values, the block's scale): the nearest e4m3 to x / scale."""
    top = x.abs().flatten(-2).amax(-1).clamp(min=2.0 ** -200)
    e = torch.ceil(torch.log2(top / 448.0))
    e = torch.where(top <= 448.0 * _power(e - 1), e - 1, e)
    e = torch.where(top > 448.0 * _power(e), e + 1, e).clamp(min=-120)
    z = x / _power(e)[..., None, None]
    size = z.abs().clamp(min=2.0 ** -6)
    at = torch.floor(torch.log2(size))
    at = at - (size < _power(at)).to(at.dtype) + (size >= _power(at + 1)).to(at.dtype)
    step = _power(at - 3)
    return torch.round(z / step) * step, _power(e)


def _exact_held(x):
    """What an 8-bit cache holds of one head's tokens x [n, d]: full blocks as e4m3, the rest as it is."""
    x = x.to(torch.float64)
    full = x.shape[0] // BLOCK * BLOCK
    if full == 0:
        return x
    z, s = _exact_e4m3(x[:full].view(-1, BLOCK, x.shape[1]))
    return torch.cat([(z * s[:, None, None]).view(full, -1), x[full:]])


def _exact_append(c, seed):
    io = TYPES["f32" if c["kv"] == "f32" else "bf16"]
    b, n, d, S, R = c["batch"], c["tokens"], c["d"], c["S"], c["R"]
    q, k, v, (wq, wk) = _projection(c, seed, b * n, io)
    pos = (c["start"] + torch.arange(n, device="cuda")).repeat(b)
    out = {"q": _exact_rope(c, q, pos, wq).view(b, n, c["hq"], d)}
    kv = {"k": _exact_rope(c, k, pos, wk).view(b, n, -1, d), "v": v.to(torch.float64).reshape(b, n, -1, d)}
    pages = -(-n // PAGE)
    for name, x in kv.items():
        if c["n_ret"]:
            ret = x[:, :, :c["n_ret"]].permute(0, 2, 1, 3)
            cap = pages * PAGE if c["paged"] else (n if c["kv"] != "fp8" else -(-n // 128) * 128)
            rows = torch.zeros(b, c["n_ret"], cap, d, dtype=torch.float64, device="cuda")
            if c["kv"] == "fp8":
                # K is held as bf16 before it is coded
                ret = ret.to(torch.bfloat16).to(torch.float64)
                full = n // BLOCK * BLOCK
                scale = torch.zeros(b, c["n_ret"], cap // BLOCK, dtype=torch.float64, device="cuda")
                tail = torch.zeros(b, c["n_ret"], BLOCK, d, dtype=torch.float64, device="cuda")
                if full:
                    z, s = _exact_e4m3(ret[:, :, :full].unflatten(2, (-1, BLOCK)))
                    rows[:, :, :full], scale[:, :, :full // BLOCK] = z.flatten(2, 3), s
                tail[:, :, :n - full] = ret[:, :, full:]
                if c["paged"]:
                    scale = scale.unflatten(2, (pages, -1)).transpose(1, 2).flatten(0, 1)
                out["scale_" + name], out["tail_" + name] = scale, tail
            else:
                rows[:, :, :n] = ret
            if c["paged"]:
                rows = rows.unflatten(2, (pages, PAGE)).transpose(1, 2).flatten(0, 1)
            out["ret_" + name] = rows
        if c["n_ret"] < c["hkv"]:
            ring = torch.zeros(b, c["hkv"] - c["n_ret"], S + R, d, dtype=torch.float64, device="cuda")
            for p in range(n):
                if p < S or p >= n - R:
                    ring[:, :, p if p < S else S + (p - S) % R] = x[:, p, c["n_ret"]:]
            out["str_" + name] = ring
    return out


def _exact_decode(c, seed):
    lens, q, ret, stream = _decode_inputs(c, seed)
    g, S, R = c["hq"] // c["hkv"], c["S"], c["R"]
    few = stream[0].shape[2]
    out = torch.empty(c["batch"], c["hq"], 128, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        for h in range(c["hkv"]):
            if h < c["n_ret"]:
                k, v = (_exact_held(x[b, h, :n]) for x in ret)
            else:
                keep = [p for p in range(min(n, S))] + [p for p in range(max(S, n - R), n)]
                at = [p if p < S else max(0, few - 1 - (n - 1 - p) % max(1, few - S)) for p in keep]
                k, v = (x[b, h - c["n_ret"], at].to(torch.float64) for x in stream)
            s = q[b, h * g:(h + 1) * g].to(torch.float64) @ k.T * 128 ** -0.5
            out[b, h * g:(h + 1) * g] = torch.softmax(s, -1) @ v
    return out


def _exact_prefill(c, seed):
    q, k, v = _prefill_inputs(c, seed)
    h0, n, g = c["history"], c["chunk"], c["hq"] // c["hkv"]
    out = torch.empty(c["batch"], n, c["hq"], 128, dtype=torch.float64, device="cuda")
    i = torch.arange(h0, h0 + n, device="cuda")[:, None]
    j = torch.arange(h0 + n, device="cuda")[None]
    for b in range(c["batch"]):
        for h in range(c["hkv"]):
            kk, vv = k[b, h].to(torch.float64), v[b, h].to(torch.float64)
            hide = j > i
            if h < c["n_ret"]:
                kk, vv = (torch.cat([_exact_held(x[:h0]), x[h0:]]) for x in (kk, vv))
            else:
                hide = hide | ((j >= c["S"]) & (i - j >= c["R"]))
            for m in range(g):
                s = (q[b, :, h * g + m].to(torch.float64) @ kk.T * 128 ** -0.5).masked_fill(hide, -math.inf)
                out[b, :, h * g + m] = torch.softmax(s, -1) @ vv
    return out
