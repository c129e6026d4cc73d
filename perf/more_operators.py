"""Measured calls of four more operators of a paged KV cache, and their plain forms.

  norm    the RMS norm of each q and k head, the rotary positions and the
          scatter of a step's K/V rows into the pools, in one pass
          (``paged_kv_write_norm_rope``)
  window  attention in which a query sees the last ``window`` tokens and the
          first ``sink`` ones (``paged_attention_window_forward``)
  write   the scatter of K/V rows into pools of 8-bit codes with a scale for
          each block and kv head, which grows as rows arrive
          (``paged_kv_write_fp8block``)
  attn8   attention over such pools (``paged_attention_forward_fp8block``)

``run`` computes the plain form in elementary torch operations, or, where
``own`` is true, makes the library's calls.  Sequence lengths are spread evenly
over [min_len, max_len] and shuffled by the seed, so ``work`` is exact.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4, "fp8": 1}
_FP8_SCALE = 8.0 / 448  # spans normed values after their weights
_EPS = 1e-6
_DEV = "cuda"


def _norm(name, tokens, q_heads, kv_heads, head_dim, rotary, interleaved, block, dtype, to, max_pos, fused):
    """``to``: "pool" (of the rows' type), "fp8" (one scale a pool) or "rows" (k as dense rows, no pool)."""
    return {"name": name, "op": "norm", "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "rotary": rotary, "interleaved": interleaved, "block": block, "dtype": dtype,
            "to": to, "max_pos": max_pos, "fused": fused}


def _attend(op, name, seqs, query, ragged, min_len, max_len, q_heads, kv_heads, head_dim, block, dtype, window, sink):
    """``window`` 0: every earlier token is seen."""
    return {"name": name, "op": op, "seqs": seqs, "query": query, "ragged": ragged, "min_len": min_len,
            "max_len": max_len, "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "block": block,
            "dtype": dtype, "window": window, "sink": sink}


def _write(name, seqs, query, ragged, min_len, max_len, kv_heads, head_dim, block, dtype, fused):
    """``query`` new tokens of each sequence (up to that many where ragged), at the end of its tokens."""
    return {"name": name, "op": "write", "seqs": seqs, "query": query, "ragged": ragged, "min_len": min_len,
            "max_len": max_len, "kv_heads": kv_heads, "head_dim": head_dim, "block": block, "dtype": dtype,
            "fused": fused}


def listed():
    return [
        # one decode step of 64 running sequences: latency counts
        _norm("norm-decode", 64, 32, 8, 128, 128, False, 16, "bf16", "pool", 4096, False),
        # a mixed step: 8 prefill chunks of 512 tokens and 120 decodes, rows that are views of a fused projection
        _norm("norm-mixed", 4216, 32, 8, 128, 128, False, 16, "bf16", "pool", 8192, True),
        # a long prompt into FP8 pools, half of each head rotated, interleaved pairs, far positions
        _norm("norm-prompt-fp8", 16384, 32, 8, 128, 64, True, 16, "bf16", "fp8", 131072, False),
        # a small fp32 model's decode step: odd lengths, head_dim 64, a short window
        _attend("window", "window-small-f32", 5, 1, False, 33, 517, 8, 2, 64, 16, "f32", 100, 3),
        # the decode batch at contexts far beyond the window
        _attend("window", "window-decode", 64, 1, False, 2048, 16384, 32, 8, 128, 16, "bf16", 4096, 4),
        # prompt chunks of a layer with a short window: few of the cached keys are seen
        _attend("window", "window-prefill", 8, 512, False, 2560, 8192, 32, 8, 128, 16, "bf16", 1024, 4),
        # one decode step into 8-bit pools: blocks begin, go on and outgrow their scale
        _write("write-decode", 64, 1, False, 1, 47, 8, 128, 16, "bf16", False),
        # the prompts of 8 sequences, their first block partly filled before, rows of a fused projection
        _write("write-prompt", 8, 2048, False, 2048, 2063, 8, 128, 16, "bf16", True),
        # the decode batch: one token each for 64 sequences of 512 to 4096 tokens
        _attend("attn8", "attn8-decode", 64, 1, False, 512, 4096, 32, 8, 128, 16, "bf16", 0, 0),
        # few very long contexts, single tokens
        _attend("attn8", "attn8-long", 4, 1, False, 131072, 131072, 32, 8, 128, 16, "bf16", 0, 0),
        # a verify step of 5 tokens: 40 rows to a kv head
        _attend("attn8", "attn8-verify", 32, 5, False, 8192, 8192, 64, 8, 128, 32, "bf16", 0, 0),
        # prompt chunks of 512 tokens on up to 2048 cached ones
        _attend("attn8", "attn8-prefill", 8, 512, False, 512, 2560, 32, 8, 128, 16, "bf16", 0, 0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "window", "window", "write", "attn8", "attn8"])
    kv_heads = rng.choice([1, 2, 4, 8])
    block = rng.choice([8, 16, 32, 64])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "norm":
        to = rng.choice(["pool", "pool", "fp8", "rows"])
        head_dim = rng.choice([64, 80, 128, 128, 256])
        c = _norm("", _log(rng, 1, 12000), kv_heads * rng.choice([1, 2, 4]), kv_heads, head_dim,
                  rng.choice([head_dim, head_dim // 2]), rng.random() < 0.4, block, dtype, to,
                  rng.choice([4096, 131072]), rng.random() < 0.5)
    elif op == "write":
        query = rng.choice([1, 1, _log(rng, 2, 2500)])
        seqs = _log(rng, 1, min(96, 12000 // query))
        low = query + rng.choice([0, 1, block // 2, 3 * block])
        c = _write("", seqs, query, rng.random() < 0.5, low, low + rng.choice([0, 5, 40]), kv_heads,
                   rng.choice([64, 128]), block, dtype, rng.random() < 0.5)
    else:
        group = rng.choice([1, 2, 3, 4, 7, 8, 12])
        query = rng.choice([1, 1, 1, _log(rng, 2, 300)])
        if op == "attn8":
            dtype, head_dim = "bf16", 128
        else:
            head_dim = rng.choice([64, 128, 128])
            query = min(query, 4) if dtype == "f32" else query
        rows = query * group
        # keys in all, so that neither the rows' logits nor the gathered keys outgrow the largest listed case
        most = min(400000, 250000000 // (rows * kv_heads))
        seqs = _log(rng, 1, 48)
        max_len = max(query + 1, min(_log(rng, 64, 60000), most // seqs))
        window = 0 if op == "attn8" and rng.random() < 0.7 else _log(rng, 16, 8192)
        c = _attend(op, "", seqs, query, rng.random() < 0.5, max(query, max_len // rng.choice([1, 2, 5])), max_len,
                    kv_heads * group, kv_heads, head_dim, block, dtype, window,
                    rng.choice([0, 1, 4, 4, 130]) if window else 0)
    del c["name"]
    return c


def _lens(case):
    n, lo, hi = case["seqs"], case["min_len"], case["max_len"]
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _queries(case, lens):
    """Query tokens of each sequence (in the order of _lens)."""
    if not case["ragged"]:
        return [min(case["query"], L) for L in lens]
    return [min(1 + (7 * i + case["query"] - 1) % case["query"], L) for i, L in enumerate(lens)]


def _pages(case, lens, gen):
    """Block tables of a seeded block order, and the pool's number of blocks."""
    bs = case["block"]
    need = [-(-L // bs) for L in lens]
    total = sum(need) + 4
    order = torch.randperm(total, generator=gen)
    ends = torch.tensor(need).cumsum(0)
    col = torch.arange(max(need))
    at = (ends - torch.tensor(need))[:, None] + col
    tables = torch.where(col < torch.tensor(need)[:, None], order[at.clamp(max=total - 1)], -1)
    return tables.to(torch.int32).to(_DEV), total


def _normal(shape, dtype, seed):
    gen = torch.Generator(_DEV).manual_seed(seed)
    return torch.randn(shape, generator=gen, device=_DEV, dtype=torch.float32).to(_TYPES[dtype])


def _scale_of(top):
    """The least power of two (2^-60 to 2^60) whose 448-fold covers ``top``."""
    m, e = torch.frexp(top)  # top = m 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(top > 0, e, -60).clamp(-60, 60)
    return torch.ldexp(torch.ones_like(top), e)


def _coded_pool(case, num_blocks, seed):
    """Codes and scales of a pool whose blocks and heads have magnitudes of their own."""
    x = _normal((num_blocks, case["block"], case["kv_heads"], case["head_dim"]), "f32", seed)
    gen = torch.Generator(_DEV).manual_seed(seed + 11)
    size = torch.randn((num_blocks, 1, case["kv_heads"], 1), generator=gen, device=_DEV)
    x *= torch.exp(0.5 * size)
    scale = _scale_of(x.abs().amax((1, 3)))
    x /= scale[:, None, :, None]
    return x.to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    gen = torch.Generator().manual_seed(seed)
    bs = case["block"]
    if case["op"] == "norm":
        T, Hq, Hkv, D = case["tokens"], case["q_heads"], case["kv_heads"], case["head_dim"]
        if case["fused"]:  # views of one projection's output
            rows = _normal((T, Hq + 2 * Hkv, D), case["dtype"], seed)
            q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
        else:
            q, k, v = (_normal((T, h, D), case["dtype"], seed + 7919 * i) for i, h in enumerate((Hq, Hkv, Hkv)))
        num_blocks = -(-T // bs) + 2
        shape = (num_blocks, bs, Hkv, D)
        dt = torch.float8_e4m3fn if case["to"] == "fp8" else _TYPES[case["dtype"]]
        r = case["rotary"]
        st = {"case": case, "q": q, "k": k, "v": v, "q_out": torch.empty(T, Hq, D, device=_DEV, dtype=q.dtype),
              "q_weight": (1 + 0.2 * _normal((D,), "f32", seed + 5)).to(q.dtype),
              "k_weight": (1 + 0.2 * _normal((D,), "f32", seed + 6)).to(q.dtype),
              "positions": torch.randint(0, case["max_pos"], (T,), generator=gen).to(_DEV),
              "inv_freq": (10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)).to(_DEV),
              "slots": torch.randperm(num_blocks * bs, generator=gen)[:T].to(_DEV)}
        if case["to"] == "rows":
            st["k_out"] = torch.empty(T, Hkv, D, device=_DEV, dtype=q.dtype)
        else:
            st["k_cache"], st["v_cache"] = (torch.zeros(shape, device=_DEV).to(dt) for _ in range(2))
        return st
    lens = _lens(case)
    order = torch.randperm(len(lens), generator=gen).tolist()
    n = _queries(case, lens)
    lens, n = [lens[i] for i in order], [n[i] for i in order]
    tables, num_blocks = _pages(case, lens, gen)
    qsl = torch.cat([torch.zeros(1, dtype=torch.long), torch.tensor(n).cumsum(0)])
    T, Hkv, D = int(qsl[-1]), case["kv_heads"], case["head_dim"]
    st = {"case": case, "tables": tables, "max_query": max(n), "qsl": qsl.to(torch.int32).to(_DEV),
          "lens": torch.tensor(lens, dtype=torch.int32, device=_DEV)}
    if case["op"] == "window":
        shape = (num_blocks, bs, Hkv, D)
        st["k_cache"], st["v_cache"] = _normal(shape, case["dtype"], seed + 2), _normal(shape, case["dtype"], seed + 3)
    else:
        for i, name in enumerate("kv"):
            st[name + "_cache"], st[name + "_scales"] = _coded_pool(case, num_blocks, seed + 2 + 100 * i)
    if case["op"] == "write":
        # new rows of other magnitudes than their blocks'
        gain = torch.exp(0.7 * torch.randn(T, generator=gen)).to(_DEV)[:, None, None]
        rows = (_normal((T, 2 * Hkv, D), "f32", seed) * gain).to(_TYPES[case["dtype"]])
        k, v = rows[:, :Hkv], rows[:, Hkv:]
        st["k"], st["v"] = (k, v) if case["fused"] else (k.contiguous(), v.contiguous())
        seq = torch.repeat_interleave(torch.arange(len(n)), torch.tensor(n))
        place = torch.arange(T) - qsl[seq] + torch.tensor([L - x for L, x in zip(lens, n)])[seq]
        block = tables.cpu().long()[seq, place // bs]
        st["slots"] = (block * bs + place % bs).to(_DEV)
        return st
    st["q"] = (2 * _normal((T, case["q_heads"], D), "f32", seed)).to(_TYPES[case["dtype"]])
    st["out"] = torch.empty_like(st["q"])
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _turn(x, cos, sin, interleaved):
    """x [T, H, D] in fp32; the first 2 * cos.shape[-1] columns are rotated."""
    r = cos.shape[-1]
    c, s = cos[:, None], sin[:, None]
    head, rest = x[..., :2 * r], x[..., 2 * r:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    else:
        a, b = head[..., :r], head[..., r:]
        turned = torch.cat([a * c - b * s, a * s + b * c], -1)
    return torch.cat([turned, rest], -1)


def _rms(x, weight):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS) * weight.float()


def _plain_norm(st):
    case = st["case"]
    angle = st["positions"].double()[:, None] * st["inv_freq"]
    cos, sin = angle.cos().float(), angle.sin().float()
    st["q_out"].copy_(_turn(_rms(st["q"], st["q_weight"]), cos, sin, case["interleaved"]))
    k = _turn(_rms(st["k"], st["k_weight"]), cos, sin, case["interleaved"])
    if case["to"] == "rows":
        st["k_out"].copy_(k)
        return st["q_out"], st["k_out"]
    v = st["v"].float()
    if case["to"] == "fp8":
        k, v = (k / _FP8_SCALE).clamp(-448, 448), (v / _FP8_SCALE).clamp(-448, 448)
    for pool, rows in ((st["k_cache"], k), (st["v_cache"], v)):
        bits = torch.uint8 if pool.dtype == torch.float8_e4m3fn else pool.dtype
        pool.view(-1, case["kv_heads"], case["head_dim"]).view(bits)[st["slots"]] = rows.to(pool.dtype).view(bits)
    return st["q_out"], st["k_cache"], st["v_cache"]


def _rows_of(pool, scales, tables, width):
    """The sequences' rows [B, width, Hkv, D] in fp32."""
    if scales is None:
        x = pool[tables].float()
    else:
        x = pool.view(torch.uint8)[tables].view(pool.dtype).float() * scales[tables][:, :, None, :, None]
    return x.flatten(1, 2)[:, :width]


def _plain_attention(st):
    case = st["case"]
    B, Hkv, D, width = case["seqs"], case["kv_heads"], case["head_dim"], case["max_len"]
    G, most = case["q_heads"] // Hkv, st["max_query"]
    L, qsl, tables = st["lens"].long(), st["qsl"].long(), st["tables"].long().clamp(min=0)
    n = qsl[1:] - qsl[:-1]
    keys = _rows_of(st["k_cache"], st.get("k_scales"), tables, width)
    i = torch.arange(most, device=_DEV)
    token = (qsl[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    q = st["q"].float()[token].view(B, most, Hkv, G, D).permute(0, 2, 1, 3, 4).flatten(2, 3)
    logits = (q @ keys.permute(0, 2, 3, 1)) * (1 / math.sqrt(D))         # [B, Hkv, rows, keys]
    del keys
    key = torch.arange(width, device=_DEV)
    place = (L - n)[:, None] + i                                         # [B, queries]
    seen = key <= place[..., None]
    if case["window"]:
        seen &= (key > place[..., None] - case["window"]) | (key < case["sink"])
    live = i < n[:, None]
    seen = (seen & live[..., None]).repeat_interleave(G, 1)[:, None]
    logits = logits.masked_fill_(~seen, -math.inf)
    top = logits.amax(-1, keepdim=True).clamp(min=-1e30)
    e = logits.sub_(top).exp_()
    total = e.sum(-1, keepdim=True).clamp(min=1e-30)
    values = _rows_of(st["v_cache"], st.get("v_scales"), tables, width)
    # rows past a sequence's end hold what an earlier one left
    values = torch.where((key < L[:, None])[..., None, None], values, 0.0)
    out = (e @ values.permute(0, 2, 1, 3)) / total                       # [B, Hkv, rows, D]
    out = out.view(B, Hkv, most, G, D).permute(0, 2, 1, 3, 4).flatten(2, 3)
    st["out"].copy_(out[live])
    return st["out"]


def _plain_write(st):
    case = st["case"]
    bs, Hkv, D = case["block"], case["kv_heads"], case["head_dim"]
    slots = st["slots"]
    block, place = slots // bs, slots % bs
    num_blocks = st["k_cache"].shape[0]
    begun = torch.zeros(num_blocks, dtype=torch.bool, device=_DEV)
    begun[block[place == 0]] = True
    written = torch.zeros(num_blocks * bs, dtype=torch.bool, device=_DEV)
    written[slots] = True
    out = []
    for rows, pool, scales in ((st["k"], st["k_cache"], st["k_scales"]), (st["v"], st["v_cache"], st["v_scales"])):
        x = rows.float()
        top = torch.zeros(num_blocks, Hkv, device=_DEV)
        top.scatter_reduce_(0, block[:, None].expand(-1, Hkv), x.abs().amax(-1), "amax")
        touched = torch.zeros(num_blocks, dtype=torch.bool, device=_DEV)
        touched[block] = True
        need = _scale_of(top)
        old = torch.where(begun[:, None], 0.0, scales)
        new = torch.where(touched[:, None], torch.maximum(old, need), scales)
        # the rows that stay, at the block's new scale
        grown = touched & ~begun
        ids = grown.nonzero()[:, 0]
        codes = pool.view(torch.uint8)[ids].view(pool.dtype).float()
        again = (codes * (scales[ids] / new[ids])[:, None, :, None]).to(pool.dtype)
        pool.view(torch.uint8)[ids] = again.view(torch.uint8)
        scales.copy_(new)
        coded = (x / new[block][..., None]).clamp(-448, 448).to(pool.dtype)
        pool.view(-1, Hkv, D).view(torch.uint8)[slots] = coded.view(torch.uint8)
        out += [pool, scales]
    return out


def _own(st):
    import paged_kv_cache_236_gb300 as pkv
    case = st["case"]
    if case["op"] == "norm":
        args = st["q"], st["k"], st["v"], st["q_weight"], st["k_weight"], st["positions"], st["inv_freq"]
        if case["to"] == "rows":
            pkv.paged_kv_write_norm_rope(*args, eps=_EPS, interleaved=case["interleaved"], q_out=st["q_out"],
                                         k_out=st["k_out"])
            return st["q_out"], st["k_out"]
        if case["to"] == "fp8":
            pkv.paged_kv_write_norm_rope_fp8(*args, st["slots"], st["k_cache"], st["v_cache"], _FP8_SCALE, _FP8_SCALE,
                                             eps=_EPS, interleaved=case["interleaved"], q_out=st["q_out"])
        else:
            pkv.paged_kv_write_norm_rope(*args, st["slots"], st["k_cache"], st["v_cache"], eps=_EPS,
                                         interleaved=case["interleaved"], q_out=st["q_out"])
        return st["q_out"], st["k_cache"], st["v_cache"]
    if case["op"] == "write":
        pkv.paged_kv_write_fp8block(st["k"], st["v"], st["slots"], st["k_cache"], st["v_cache"], st["k_scales"],
                                    st["v_scales"])
        return [st["k_cache"], st["k_scales"], st["v_cache"], st["v_scales"]]
    scale = 1 / math.sqrt(case["head_dim"])
    batch = st["tables"], st["lens"], st["qsl"], scale
    if case["op"] == "window":
        return pkv.paged_attention_window_forward(st["q"], st["k_cache"], st["v_cache"], *batch, case["window"],
                                                  case["sink"], out=st["out"], max_query_len=st["max_query"])
    return pkv.paged_attention_forward_fp8block(st["q"], st["k_cache"], st["v_cache"], st["k_scales"], st["v_scales"],
                                                *batch, window=case["window"], num_sink=case["sink"], out=st["out"],
                                                max_query_len=st["max_query"])


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "write": _plain_write, "window": _plain_attention,
            "attn8": _plain_attention}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def _seen(place, window, sink):
    """Keys that the query at ``place`` sees."""
    if not window or place < window:
        return place + 1
    return window + min(sink, place + 1 - window)


def work(case):
    e = _BYTES[case["dtype"]]
    if case["op"] == "norm":
        T, Hq, Hkv, D = case["tokens"], case["q_heads"], case["kv_heads"], case["head_dim"]
        # rows in, rotated q and k (and v) out, a position and a slot a token
        if case["to"] == "rows":
            moved = 2 * (Hq + Hkv) * e
        else:
            moved = (Hq + 2 * Hkv) * e + Hq * e + 2 * Hkv * _BYTES["fp8" if case["to"] == "fp8" else case["dtype"]]
        return {"bytes": T * D * moved + 16 * T + 4 * case["rotary"] + 2 * D * e,
                "flops": T * (Hq + Hkv) * (4 * D + 3 * case["rotary"])}
    lens = _lens(case)
    n = _queries(case, lens)
    Hkv, D, bs = case["kv_heads"], case["head_dim"], case["block"]
    if case["op"] == "write":
        blocks = sum((L - 1) // bs - (L - x) // bs + 1 for L, x in zip(lens, n))
        return {"bytes": sum(n) * (Hkv * D * 2 * (e + 1) + 8) + blocks * Hkv * 2 * 4, "flops": sum(n) * Hkv * D * 4}
    p = e if case["op"] == "window" else 1
    keys = pairs = blocks = 0
    for L, x in zip(lens, n):
        first = L - x if not case["window"] else max(0, L - x - case["window"] + 1)
        some = L if not case["window"] else L - first + min(case["sink"], first)
        keys += some
        blocks += -(-some // bs)
        pairs += sum(_seen(L - x + i, case["window"], case["sink"]) for i in range(x))
    scales = 0 if case["op"] == "window" else blocks * Hkv * 2 * 4
    return {"bytes": keys * Hkv * D * 2 * p + 2 * sum(n) * case["q_heads"] * D * e + 4 * blocks + scales,
            "flops": pairs * case["q_heads"] * 4 * D}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _exact_norm(case, st):
    T, r, D, Hkv = case["tokens"], case["rotary"] // 2, case["head_dim"], case["kv_heads"]
    z = torch.polar(torch.ones(T, r, dtype=torch.float64, device=_DEV),
                    st["positions"].to(torch.float64).unsqueeze(1) * st["inv_freq"].unsqueeze(0))

    def turn(x, weight):
        x = x.to(torch.float64)
        size = torch.linalg.vector_norm(x, dim=-1, keepdim=True) / math.sqrt(D)
        x = x * weight.to(torch.float64) / torch.sqrt(size ** 2 + _EPS)
        lo, hi = (slice(0, 2 * r, 2), slice(1, 2 * r, 2)) if case["interleaved"] else (slice(0, r), slice(r, 2 * r))
        w = torch.complex(x[..., lo], x[..., hi]) * z.unsqueeze(1)
        x[..., lo], x[..., hi] = w.real.clone(), w.imag.clone()
        return x

    q, k = turn(st["q"], st["q_weight"]), turn(st["k"], st["k_weight"])
    if case["to"] == "rows":
        return q, k
    pools = []
    for rows in (k, st["v"].to(torch.float64)):
        pool = torch.zeros(st["k_cache"].numel() // (Hkv * D), Hkv, D, dtype=torch.float64, device=_DEV)
        pool[st["slots"]] = rows / _FP8_SCALE if case["to"] == "fp8" else rows
        pools.append(pool.view(st["k_cache"].shape))
    return q, pools[0], pools[1]


def _exact_write(case, st):
    bs = case["block"]
    slots = st["slots"].cpu()
    order = torch.argsort(slots)
    split = torch.bincount(slots // bs, minlength=st["k_cache"].shape[0]).tolist()
    out = []
    for rows, pool, scales in ((st["k"], st["k_cache"], st["k_scales"]), (st["v"], st["v_cache"], st["v_scales"])):
        codes, scales = pool.cpu().to(torch.float64), scales.cpu().to(torch.float64)
        rows = rows.cpu().to(torch.float64)
        for block, mine in enumerate(torch.split(order, split)):
            if not len(mine):
                continue
            x = rows[mine]
            top = x.abs().amax((0, 2)) / 448
            need = torch.tensor([2.0 ** max(-60, min(60, math.ceil(math.log2(t)))) if t > 0 else 2.0 ** -60
                                 for t in top.tolist()], dtype=torch.float64)
            if (slots[mine] % bs == 0).any():
                new = need
            else:
                new = torch.maximum(need, scales[block])
                codes[block] *= (scales[block] / new)[:, None]
            scales[block] = new
            codes[block, slots[mine] % bs] = x / new[:, None]
        out += [codes.to(_DEV), scales.to(_DEV)]
    return out


def _exact_attention(case, st):
    Hkv, bs, window = case["kv_heads"], case["block"], case["window"]
    G, D = case["q_heads"] // Hkv, case["head_dim"]
    out = torch.empty(st["q"].shape, dtype=torch.float64, device=_DEV)
    lens, qsl = st["lens"].tolist(), st["qsl"].tolist()

    def values(name, blocks):
        pool = st[name + "_cache"]
        if case["op"] == "window":
            return pool[blocks].to(torch.float64).reshape(-1, Hkv, D)
        x = pool.view(torch.uint8)[blocks].view(pool.dtype).to(torch.float64)
        return (x * st[name + "_scales"][blocks].to(torch.float64)[:, None, :, None]).reshape(-1, Hkv, D)

    for s, L in enumerate(lens):
        blocks = st["tables"][s, :-(-L // bs)].long()
        K, V = values("k", blocks)[:L], values("v", blocks)[:L]
        q = st["q"][qsl[s]:qsl[s + 1]].to(torch.float64)
        n = q.shape[0]
        hidden = torch.ones(n, L, dtype=torch.bool, device=_DEV).triu(L - n + 1)
        if window:
            far = torch.ones(n, L, dtype=torch.bool, device=_DEV).tril(L - n - window)
            far[:, :case["sink"]] = False
            hidden |= far
        for h in range(Hkv):
            z = torch.einsum("igd,jd->igj", q[:, h * G:(h + 1) * G], K[:, h]) / math.sqrt(D)
            w = torch.softmax(z.masked_fill(hidden[:, None], -math.inf), -1)
            out[qsl[s]:qsl[s + 1], h * G:(h + 1) * G] = torch.einsum("igj,jd->igd", w, V[:, h])
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(case, st)
    return _exact_write(case, st) if case["op"] == "write" else _exact_attention(case, st)


if __name__ == "__main__":
    for c in listed():
        w = work(c)
        print("%-20s %10.3f MB %10.3f GFLOP" % (c["name"], w["bytes"] / 1e6, w["flops"] / 1e9))
    for k in range(6):
        print(draw(random.Random(k)))
