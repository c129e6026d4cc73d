"""Measured calls of the bounded-cache operators, and their plain forms.

Four operators keep a paged KV cache within a budget while a model serves long
contexts:

  rope     the rotary positions of a step's q and k, and the scatter of its K/V
           rows into the block pools (``paged_kv_write_rope``)
  scores   the attention weight that a step's queries pay to each cached token,
           added to a running score per (sequence, kv head, position)
           (``paged_attention_scores``)
  select   the positions a budget keeps: the first ones, the last ones and the
           highest scores between (``paged_kv_select``)
  compact  the kept tokens' K/V rows and scores moved to the front of their
           sequence's blocks (``paged_kv_compact``)

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
_FP8_SCALE = 4.5 / 448  # spans N(0, 1) values
_DEV = "cuda"


def _rope(name, tokens, q_heads, kv_heads, head_dim, rotary, interleaved, block, dtype, pool, max_pos, fused):
    return {"name": name, "op": "rope", "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "rotary": rotary, "interleaved": interleaved, "block": block, "dtype": dtype,
            "pool": pool, "max_pos": max_pos, "fused": fused}


def _scores(name, seqs, query, ragged, min_len, max_len, q_heads, kv_heads, head_dim, block, dtype, pool, decay):
    return {"name": name, "op": "scores", "seqs": seqs, "query": query, "ragged": ragged, "min_len": min_len,
            "max_len": max_len, "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "block": block,
            "dtype": dtype, "pool": pool, "decay": decay}


def _select(name, seqs, min_len, max_len, kv_heads, budget, sink, recent):
    return {"name": name, "op": "select", "seqs": seqs, "min_len": min_len, "max_len": max_len,
            "kv_heads": kv_heads, "budget": budget, "sink": sink, "recent": recent}


def _compact(name, seqs, min_len, max_len, kv_heads, head_dim, block, dtype, budget, scores):
    return {"name": name, "op": "compact", "seqs": seqs, "min_len": min_len, "max_len": max_len,
            "kv_heads": kv_heads, "head_dim": head_dim, "block": block, "dtype": dtype, "budget": budget,
            "scores": scores}


def listed():
    return [
        # one decode step of 64 running sequences: latency counts
        _rope("rope-decode", 64, 32, 8, 128, 128, False, 16, "bf16", "same", 4096, False),
        # a mixed step: 8 prefill chunks of 512 tokens and 120 decodes, rows that are views of a fused projection
        _rope("rope-mixed", 4216, 32, 8, 128, 128, False, 16, "bf16", "same", 8192, True),
        # a long prompt into FP8 pools, half of each head rotated, interleaved pairs, far positions
        _rope("rope-prompt-fp8", 16384, 32, 8, 128, 64, True, 16, "bf16", "fp8", 131072, False),
        # a small fp32 model's decode step: odd lengths, head_dim 64
        _scores("scores-small-f32", 5, 1, False, 33, 517, 8, 2, 64, 16, "f32", "same", 1.0),
        # the decode batch: one token each for 64 sequences of 512 to 4096 tokens
        _scores("scores-decode", 64, 1, False, 512, 4096, 32, 8, 128, 16, "bf16", "same", 1.0),
        # few very long contexts, single tokens, older weight fading
        _scores("scores-long", 4, 1, False, 131072, 131072, 32, 8, 128, 16, "bf16", "same", 0.98),
        # a verify step of 5 tokens: 40 rows to a kv head
        _scores("scores-verify", 32, 5, False, 8192, 8192, 64, 8, 128, 32, "bf16", "same", 1.0),
        # the last up to 64 queries of 8 prompts score their whole prompt before it is cut to a budget
        _scores("scores-window", 8, 64, True, 6000, 16384, 32, 8, 128, 16, "bf16", "same", 0.0),
        # the decode batch cut to 512 tokens each
        _select("select-batch", 64, 512, 4096, 8, 512, 4, 64),
        # long contexts cut to an eighth
        _select("select-long", 4, 131072, 131072, 8, 16384, 4, 1024),
        # the decode batch's rows moved together
        _compact("compact-batch", 64, 512, 4096, 8, 128, 16, "bf16", 512, True),
        # long contexts in FP8 pools cut to an eighth
        _compact("compact-long-fp8", 4, 100003, 131072, 8, 128, 16, "fp8", 16384, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "scores", "scores", "select", "compact"])
    kv_heads = rng.choice([1, 2, 4, 8])
    head_dim = rng.choice([64, 128])
    block = rng.choice([8, 16, 32, 64])
    if op == "rope":
        pool = rng.choice(["same", "same", "fp8"])
        head_dim = 128 if pool == "fp8" else head_dim
        c = _rope("", _log(rng, 1, 12000), kv_heads * rng.choice([1, 2, 4]), kv_heads, head_dim,
                  rng.choice([head_dim, head_dim // 2]), rng.random() < 0.4, block, rng.choice(["bf16", "bf16", "f32"]),
                  pool, rng.choice([4096, 131072]), rng.random() < 0.5)
    elif op == "scores":
        group = rng.choice([1, 2, 3, 4, 7, 8])
        query = rng.choice([1, 1, 1, _log(rng, 2, 96)])
        rows = query * group
        # keys in all, so that neither the rows' logits nor the gathered keys outgrow the largest listed case
        most = min(400000, 60000000 // (rows * kv_heads))
        seqs = _log(rng, 1, 48)
        max_len = max(query + 1, min(_log(rng, 64, 60000), most // seqs))
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        pool = "fp8" if dtype == "bf16" and head_dim == 128 and rng.random() < 0.25 else "same"
        c = _scores("", seqs, query, rng.random() < 0.5, max(query, max_len // rng.choice([1, 2, 5])), max_len,
                    kv_heads * group, kv_heads, head_dim, block, dtype, pool, rng.choice([0.0, 0.9, 1.0]))
    else:
        seqs = _log(rng, 1, 64)
        max_len = min(_log(rng, 64, 120000), 400000 // seqs)
        budget = max(8, int(max_len * rng.uniform(0.1, 0.7)))
        low = max(1, max_len // rng.choice([1, 2, 6]))
        if op == "select":
            c = _select("", seqs, low, max_len, kv_heads, budget, min(4, budget // 4),
                        int(budget * rng.uniform(0, 0.5)))
        else:
            c = _compact("", seqs, low, max_len, kv_heads, head_dim, block, rng.choice(["bf16", "f32", "fp8"]),
                         budget, rng.random() < 0.5)
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
    order = torch.randperm(total, generator=gen).tolist()
    tables = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        tables[s, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    return tables.to(_DEV), total


def _normal(shape, dtype, seed):
    gen = torch.Generator(_DEV).manual_seed(seed)
    x = torch.randn(shape, generator=gen, device=_DEV, dtype=torch.float32)
    return (x / _FP8_SCALE).to(torch.float8_e4m3fn) if dtype == "fp8" else x.to(_TYPES[dtype])


def prepare(case, seed):
    gen = torch.Generator().manual_seed(seed)
    if case["op"] == "rope":
        T, Hq, Hkv, D, bs = case["tokens"], case["q_heads"], case["kv_heads"], case["head_dim"], case["block"]
        pool = case["dtype"] if case["pool"] == "same" else case["pool"]
        if case["fused"]:  # views of one projection's output
            rows = _normal((T, Hq + 2 * Hkv, D), case["dtype"], seed)
            q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
        else:
            q, k, v = (_normal((T, h, D), case["dtype"], seed + 7919 * i) for i, h in enumerate((Hq, Hkv, Hkv)))
        num_blocks = -(-T // bs) + 2
        shape = (num_blocks, bs, Hkv, D)
        dt = torch.float8_e4m3fn if pool == "fp8" else _TYPES[pool]
        r = case["rotary"]
        return {"case": case, "q": q, "k": k, "v": v, "k_cache": torch.zeros(shape, device=_DEV).to(dt),
                "v_cache": torch.zeros(shape, device=_DEV).to(dt), "q_out": torch.empty(T, Hq, D, device=_DEV, dtype=q.dtype),
                "positions": torch.randint(0, case["max_pos"], (T,), generator=gen).to(_DEV),
                "inv_freq": (10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)).to(_DEV),
                "slots": torch.randperm(num_blocks * bs, generator=gen)[:T].to(_DEV)}
    lens = _lens(case)
    order = torch.randperm(len(lens), generator=gen).tolist()
    if case["op"] == "select":
        lens = [lens[i] for i in order]
        g = torch.Generator(_DEV).manual_seed(seed)
        # accumulated weight: positive, a few tokens far above the rest
        w = torch.rand(case["seqs"], case["kv_heads"], case["max_len"], generator=g, device=_DEV)
        return {"case": case, "scores": w ** 6, "lens": torch.tensor(lens, dtype=torch.int32, device=_DEV),
                "kept": torch.empty(case["seqs"], case["kv_heads"], case["budget"], dtype=torch.int32, device=_DEV)}
    Hkv, D = case["kv_heads"], case["head_dim"]
    if case["op"] == "scores":
        n = _queries(case, lens)
        lens, n = [lens[i] for i in order], [n[i] for i in order]
        tables, num_blocks = _pages(case, lens, gen)
        pool = case["dtype"] if case["pool"] == "same" else case["pool"]
        qsl = [0]
        for x in n:
            qsl.append(qsl[-1] + x)
        shape = (case["seqs"], Hkv, case["max_len"])
        g = torch.Generator(_DEV).manual_seed(seed + 1)
        return {"case": case, "q": (2 * _normal((qsl[-1], case["q_heads"], D), "f32", seed)).to(_TYPES[case["dtype"]]),
                "k_cache": _normal((num_blocks, case["block"], Hkv, D), pool, seed + 2), "tables": tables,
                "lens": torch.tensor(lens, dtype=torch.int32, device=_DEV),
                "qsl": torch.tensor(qsl, dtype=torch.int32, device=_DEV), "max_query": max(n),
                "scores": torch.rand(shape, generator=g, device=_DEV), "out": torch.zeros(shape, device=_DEV)}
    lens = [lens[i] for i in order]
    tables, num_blocks = _pages(case, lens, gen)
    shape = (num_blocks, case["block"], Hkv, D)
    lens_dev = torch.tensor(lens, dtype=torch.int64, device=_DEV)
    budget, most = case["budget"], case["max_len"]
    # a seeded choice of min(L, budget) positions of each (sequence, head), ascending
    g = torch.Generator(_DEV).manual_seed(seed)
    r = torch.rand(case["seqs"], Hkv, most, generator=g, device=_DEV)
    key = torch.arange(most, device=_DEV)
    r = torch.where(key < lens_dev[:, None, None], r, 2.0)
    kept = torch.sort(torch.argsort(r, -1)[..., :budget], -1).values
    kept = torch.where(kept < lens_dev[:, None, None], kept, -1)  # positions past the end sort last
    if kept.shape[-1] < budget:
        kept = torch.nn.functional.pad(kept, (0, budget - kept.shape[-1]), value=-1)
    return {"case": case, "k_cache": _normal(shape, case["dtype"], seed + 3), "v_cache": _normal(shape, case["dtype"], seed + 4),
            "tables": tables, "kept": kept.to(torch.int32).contiguous(),
            "scores": torch.rand(case["seqs"], Hkv, most, generator=g, device=_DEV) if case["scores"] else None}


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _rotate(x, cos, sin, interleaved):
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


def _plain_rope(st):
    case = st["case"]
    angle = st["positions"].double()[:, None] * st["inv_freq"]
    cos, sin = angle.cos().float(), angle.sin().float()
    st["q_out"].copy_(_rotate(st["q"].float(), cos, sin, case["interleaved"]))
    k = _rotate(st["k"].float(), cos, sin, case["interleaved"])
    v = st["v"].float()
    if case["pool"] == "fp8":
        k, v = (k / _FP8_SCALE).clamp(-448, 448), (v / _FP8_SCALE).clamp(-448, 448)
    for pool, rows in ((st["k_cache"], k), (st["v_cache"], v)):
        bits = torch.uint8 if pool.dtype == torch.float8_e4m3fn else pool.dtype
        pool.view(-1, case["kv_heads"], case["head_dim"]).view(bits)[st["slots"]] = rows.to(pool.dtype).view(bits)
    return st["q_out"], st["k_cache"], st["v_cache"]


def _plain_scores(st):
    case = st["case"]
    B, Hkv, D, bs = case["seqs"], case["kv_heads"], case["head_dim"], case["block"]
    G = case["q_heads"] // Hkv
    scale = 1 / math.sqrt(D)
    L, qsl = st["lens"].long(), st["qsl"].long()
    n = qsl[1:] - qsl[:-1]
    width = case["max_len"]
    pool, tables = st["k_cache"], st["tables"].long().clamp(min=0)
    if pool.dtype == torch.float8_e4m3fn:
        keys, scale = pool.view(torch.uint8)[tables].view(torch.float8_e4m3fn).float(), scale * _FP8_SCALE
    else:
        keys = pool[tables].float()
    keys = keys.flatten(1, 2)[:, :width]                                  # [B, keys, Hkv, D]
    i = torch.arange(st["max_query"], device=_DEV)
    token = (qsl[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    q = st["q"].float()[token].view(B, -1, Hkv, G, D)                     # [B, queries, Hkv, G, D]
    q = q.permute(0, 2, 1, 3, 4).flatten(2, 3)                            # [B, Hkv, rows, D]
    logits = (q @ keys.permute(0, 2, 3, 1)) * scale                       # [B, Hkv, rows, keys]
    key = torch.arange(width, device=_DEV)
    seen = key <= (L - n)[:, None, None] + i[:, None]                     # [B, queries, keys]
    seen = (seen & (i < n[:, None])[..., None]).repeat_interleave(G, 1)[:, None]
    logits = logits.masked_fill(~seen, -math.inf)
    top = logits.amax(-1, keepdim=True).clamp(min=-1e30)
    e = torch.exp(logits - top)
    paid = (e / e.sum(-1, keepdim=True).clamp(min=1e-30)).sum(2)          # [B, Hkv, keys]
    if case["decay"] == 0.0:
        new = paid
    else:
        old = (key < (L - n)[:, None])[:, None]
        new = paid + torch.where(old, st["scores"] * case["decay"], 0.0)
    st["out"].copy_(torch.where((key < L[:, None])[:, None], new, st["out"]))
    return st["out"]


def _plain_select(st):
    case = st["case"]
    L = st["lens"].long()[:, None, None]
    pos = torch.arange(case["max_len"], device=_DEV)
    forced = (pos < case["sink"]) | (pos >= L - case["recent"])
    worth = torch.where(forced, math.inf, st["scores"])
    worth = torch.where(pos < L, worth, -math.inf)
    # highest first, ties to the lowest position
    order = torch.sort(worth, dim=-1, descending=True, stable=True).indices[..., :case["budget"]]
    order = torch.where(order < L, order, case["max_len"])  # positions past the end sort last
    kept = torch.sort(order, -1).values
    st["kept"].fill_(-1)
    st["kept"][..., :kept.shape[-1]] = torch.where(kept < L, kept, -1).to(torch.int32)
    return st["kept"]


def _plain_compact(st):
    case = st["case"]
    bs, Hkv = case["block"], case["kv_heads"]
    kept, tables = st["kept"].long(), st["tables"].long().clamp(min=0)
    B, _, budget = kept.shape
    live = kept >= 0
    to = torch.arange(budget, device=_DEV).expand_as(kept)
    to = torch.where(live, to, 0)
    src = torch.where(live, kept, 0)
    s = torch.arange(B, device=_DEV)[:, None, None].expand_as(kept)
    h = torch.arange(Hkv, device=_DEV)[None, :, None].expand_as(kept)
    s, h, src, to = s[live], h[live], src[live], to[live]
    for pool in (st["k_cache"], st["v_cache"]):
        p = pool.view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else pool
        rows = p[tables[s, src // bs], src % bs, h]
        p[tables[s, to // bs], to % bs, h] = rows
    if st["scores"] is not None:
        st["scores"][s, h, to] = st["scores"][s, h, src]
        return st["k_cache"], st["v_cache"], st["scores"]
    return st["k_cache"], st["v_cache"]


def _own(st):
    import paged_kv_cache_236_gb300 as pkv
    case = st["case"]
    if case["op"] == "rope":
        if case["pool"] == "fp8":
            pkv.paged_kv_write_rope_fp8(st["q"], st["k"], st["v"], st["positions"], st["inv_freq"], st["slots"],
                                        st["k_cache"], st["v_cache"], _FP8_SCALE, _FP8_SCALE,
                                        interleaved=case["interleaved"], q_out=st["q_out"])
        else:
            pkv.paged_kv_write_rope(st["q"], st["k"], st["v"], st["positions"], st["inv_freq"], st["slots"],
                                    st["k_cache"], st["v_cache"], interleaved=case["interleaved"], q_out=st["q_out"])
        return st["q_out"], st["k_cache"], st["v_cache"]
    if case["op"] == "scores":
        scale = 1 / math.sqrt(case["head_dim"])
        if case["pool"] == "fp8":
            return pkv.paged_attention_scores_fp8kv(st["q"], st["k_cache"], st["tables"], st["lens"], st["qsl"],
                                                    st["scores"], scale, _FP8_SCALE, decay=case["decay"],
                                                    out=st["out"], max_query_len=st["max_query"])
        return pkv.paged_attention_scores(st["q"], st["k_cache"], st["tables"], st["lens"], st["qsl"], st["scores"],
                                          scale, decay=case["decay"], out=st["out"], max_query_len=st["max_query"])
    if case["op"] == "select":
        return pkv.paged_kv_select(st["scores"], st["lens"], case["budget"], num_sink=case["sink"],
                                   num_recent=case["recent"], out=st["kept"])
    pkv.paged_kv_compact(st["k_cache"], st["v_cache"], st["tables"], st["kept"], scores=st["scores"])
    return (st["k_cache"], st["v_cache"]) + (() if st["scores"] is None else (st["scores"],))


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "scores": _plain_scores, "select": _plain_select,
            "compact": _plain_compact}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "rope":
        T, Hq, Hkv, D = case["tokens"], case["q_heads"], case["kv_heads"], case["head_dim"]
        e = _BYTES[case["dtype"]]
        p = _BYTES[case["dtype"] if case["pool"] == "same" else case["pool"]]
        # rows in, rotated q and the pool rows out, a position and a slot a token
        return {"bytes": T * D * ((Hq + 2 * Hkv) * e + Hq * e + 2 * Hkv * p) + 16 * T + 4 * case["rotary"],
                "flops": 3 * T * (Hq + Hkv) * case["rotary"]}
    lens = _lens(case)
    Hkv = case["kv_heads"]
    if case["op"] == "scores":
        n, D = _queries(case, lens), case["head_dim"]
        G = case["q_heads"] // Hkv
        e = _BYTES[case["dtype"] if case["pool"] == "same" else case["pool"]]
        pairs = sum(x * (L - x) + x * (x + 1) // 2 for L, x in zip(lens, n))  # visible (query, key) pairs
        old = 0 if case["decay"] == 0.0 else sum(L - x for L, x in zip(lens, n))
        return {"bytes": sum(lens) * Hkv * (D * e + 4) + old * Hkv * 4 + sum(n) * Hkv * G * D * _BYTES[case["dtype"]]
                + 4 * sum(-(-L // case["block"]) for L in lens),
                "flops": pairs * Hkv * G * (2 * D + 4)}
    kept = [min(L, case["budget"]) for L in lens]
    if case["op"] == "select":
        return {"bytes": 4 * Hkv * (sum(lens) + case["seqs"] * case["budget"]), "flops": sum(lens) * Hkv}
    # each kept row read and written once, in K and in V
    e = _BYTES[case["dtype"]]
    row = 2 * case["head_dim"] * e + (4 if case["scores"] else 0)
    moved = sum(k for k, L in zip(kept, lens) if L > case["budget"])  # nothing moves where nothing is dropped
    return {"bytes": 2 * moved * Hkv * row + 4 * Hkv * case["seqs"] * case["budget"], "flops": 0}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] in ("select", "compact"):
        return None  # whole numbers; rows that are moved as they are
    st = prepare(case, seed)
    if case["op"] == "rope":
        T, r, D = case["tokens"], case["rotary"] // 2, case["head_dim"]
        z = torch.polar(torch.ones(T, r, dtype=torch.float64, device=_DEV),
                        st["positions"].to(torch.float64).unsqueeze(1) * st["inv_freq"].unsqueeze(0))

        def turn(x):
            x = x.to(torch.float64).clone()
            lo, hi = (slice(0, 2 * r, 2), slice(1, 2 * r, 2)) if case["interleaved"] else (slice(0, r), slice(r, 2 * r))
            w = torch.complex(x[..., lo], x[..., hi]) * z.unsqueeze(1)
            x[..., lo], x[..., hi] = w.real.clone(), w.imag.clone()
            return x

        pools = []
        for rows in (turn(st["k"]), st["v"].to(torch.float64)):
            pool = torch.zeros(st["k_cache"].numel() // (case["kv_heads"] * D), case["kv_heads"], D, dtype=torch.float64,
                               device=_DEV)
            pool[st["slots"]] = rows / _FP8_SCALE if case["pool"] == "fp8" else rows
            pools.append(pool.view(st["k_cache"].shape))
        return turn(st["q"]), pools[0], pools[1]
    Hkv, bs = case["kv_heads"], case["block"]
    G, D = case["q_heads"] // Hkv, case["head_dim"]
    out = st["out"].to(torch.float64)
    lens, qsl = st["lens"].tolist(), st["qsl"].tolist()
    factor = _FP8_SCALE if case["pool"] == "fp8" else 1.0
    for s, L in enumerate(lens):
        blocks = st["tables"][s, :-(-L // bs)].long()
        pool = st["k_cache"]
        pool = pool.view(torch.uint8)[blocks].view(pool.dtype) if case["pool"] == "fp8" else pool[blocks]
        K = pool.to(torch.float64).reshape(-1, Hkv, D)[:L] * factor
        q = st["q"][qsl[s]:qsl[s + 1]].to(torch.float64)
        n = q.shape[0]
        later = torch.ones(n, L, dtype=torch.bool, device=_DEV).triu(L - n + 1)
        for h in range(Hkv):
            z = torch.einsum("igd,jd->igj", q[:, h * G:(h + 1) * G], K[:, h]) / math.sqrt(D)
            z = z.masked_fill(later[:, None], -math.inf)
            w = torch.softmax(z, -1).sum((0, 1))
            if case["decay"] != 0.0:
                w[:L - n] += case["decay"] * st["scores"][s, h, :L - n].to(torch.float64)
            out[s, h, :L] = w
    return out


if __name__ == "__main__":
    for c in listed():
        w = work(c)
        print("%-20s %10.3f MB %10.3f GFLOP" % (c["name"], w["bytes"] / 1e6, w["flops"] / 1e9))
    for k in range(6):
        print(draw(random.Random(k)))
