"""paged_kv_write_norm_rope and its FP8 form against the fp64 definition.

Tolerances.  The squares of at most 1024 elements are summed in fp32 in chains
of at most 48 and joined by at most 32 sums: a relative error under 80 * 2^-24,
half of it in the root; rsqrtf is good to 2 ulp (2^-22), the mean and eps round
twice: together under 46 * 2^-24 < 2.8e-6 of the normed value.  cos and sin are
within 2.2e-7, a factor cos * weight and the rotation round five times more
(5 * 2^-24): under 6e-7 * amplitude * (|z1| + |z2|) with z the normed pair.
Then one rounding to the output's type: half a step.
"""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_236_gb300 as pkv
from gpu_util import to_f64
from oracle import budget as ob
from oracle import fp8, serving

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
REL = 2.8e-6 + 6e-7


def pair_sums(x, rot, interleaved):
    """|x1| + |x2| of each element's pair; past the rotary part the element itself."""
    a = np.abs(x)
    out = a.copy()
    if interleaved:
        out[..., 0:rot:2] = out[..., 1:rot:2] = a[..., 0:rot:2] + a[..., 1:rot:2]
    else:
        out[..., :rot // 2] = out[..., rot // 2:rot] = a[..., :rot // 2] + a[..., rot // 2:rot]
    return out


def expect(x, w, eps, pos, inv, interleaved, amp):
    z = serving.head_norm(to_f64(x.contiguous()), None if w is None else to_f64(w), eps)
    want = ob.rope(z, pos.cpu().numpy(), inv.cpu().numpy(), interleaved, amp)
    return want, REL * amp * pair_sums(z, 2 * len(inv), interleaved)


def near(got, want, tol, step):
    err = np.abs(to_f64(got) - want)
    assert np.all(err <= tol + step * (np.abs(want) + tol)), float((err / (tol + step * np.abs(want) + 1e-300)).max())


def make(seed, T, Hq, Hkv, D, dtype, fused):
    g = torch.Generator().manual_seed(seed)
    size = torch.exp(2 * torch.randn(T, 1, 1, generator=g))  # tokens of very different magnitude
    rows = (size * torch.randn(T, Hq + 2 * Hkv, D, generator=g)).to(dtype).cuda()
    q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
    return (q, k, v) if fused else (q.contiguous(), k.contiguous(), v.contiguous())


CASES = [  # T, Hq, Hkv, D, rot, interleaved, bs, fused, skipped slots
    (1, 1, 1, 64, 64, False, 16, False, False),
    (1, 32, 8, 128, 128, False, 16, False, False),
    (7, 8, 2, 128, 64, True, 8, True, True),
    (64, 6, 3, 64, 32, False, 32, True, True),
    (33, 4, 4, 128, 128, True, 64, False, True),
    (5, 3, 1, 80, 48, False, 16, False, False),      # five places of a head: lanes left over
    (5, 7, 5, 80, 48, True, 16, True, False),
    (6, 5, 3, 256, 256, False, 16, True, True),
    (3, 3, 2, 1024, 512, False, 16, False, False),   # more places than lanes
    (3, 2, 2, 1024, 1024, True, 16, True, False),
    (9, 2, 2, 10, 6, False, 16, False, True),        # rows of 20 or 40 bytes: by the element
    (9, 5, 2, 18, 2, True, 16, False, True),
    (40, 12, 4, 128, 100, False, 16, True, True),    # halves of 50: by the element, more places than lanes
    (1300, 4, 2, 64, 64, False, 16, False, True),
]
IDS = lambda c: "-".join(map(str, c))  # noqa: E731


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_pools_and_rows(case, dtype):
    T, Hq, Hkv, D, rot, inter, bs, fused, skips = case
    q, k, v = make(T + D, T, Hq, Hkv, D, dtype, fused)
    g = torch.Generator().manual_seed(T)
    NB = T // bs + 3
    slots = torch.randperm(NB * bs, generator=g)[:T].cuda()
    if skips:
        slots[::3] = -1
    pos = torch.randint(0, 200000, (T,), generator=g).cuda()
    inv = pkv.rope_frequencies(rot)
    wdtype = torch.float32 if T % 2 else dtype
    qw, kw = ((1 + 0.3 * torch.randn(D, generator=g)).to(wdtype).cuda() for _ in range(2))
    if T == 64:
        kw = None
    amp, eps = (1.0, 1e-6) if T % 2 else (1.25, 1e-2)
    kc = torch.full((NB, bs, Hkv, D), float("nan"), dtype=dtype, device="cuda")
    vc = kc.clone()
    k_out = torch.empty(T, Hkv, D, dtype=dtype, device="cuda")
    out = pkv.paged_kv_write_norm_rope(q, k, v, qw, kw, pos, inv, slots, kc, vc, eps=eps, interleaved=inter,
                                       amplitude=amp, k_out=k_out)
    step = HALF_STEP[dtype]
    near(out, *expect(q, qw, eps, pos, inv, inter, amp), step)
    near(k_out, *expect(k, kw, eps, pos, inv, inter, amp), step)
    live = slots >= 0
    flat_k, flat_v = kc.view(-1, Hkv, D), vc.view(-1, Hkv, D)
    assert torch.equal(flat_k[slots[live]], k_out[live]) and torch.equal(flat_v[slots[live]], v[live])
    untouched = torch.ones(NB * bs, dtype=torch.bool, device="cuda")
    untouched[slots[live]] = False
    assert torch.isnan(flat_k[untouched]).all() and torch.isnan(flat_v[untouched]).all()
    # without pools, and in place
    q2, k2 = q.clone(memory_format=torch.contiguous_format), k.clone(memory_format=torch.contiguous_format)
    assert pkv.paged_kv_write_norm_rope(q2, k2, None, qw, kw, pos, inv, eps=eps, interleaved=inter, amplitude=amp,
                                        q_out=q2, k_out=k2) is q2
    assert torch.equal(q2, out) and torch.equal(k2, k_out)
    assert pkv.device_errors() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", [c for c in CASES if c[0] < 1000], ids=IDS)
def test_fp8_pools(case, dtype):
    T, Hq, Hkv, D, rot, inter, bs, fused, skips = case
    q, k, v = make(T + D + 1, T, Hq, Hkv, D, dtype, fused)
    g = torch.Generator().manual_seed(T + 1)
    NB = T // bs + 3
    slots = torch.randperm(NB * bs, generator=g)[:T].cuda()
    if skips:
        slots[1::4] = -7
    pos = torch.randint(0, 200000, (T,), generator=g).cuda()
    inv = pkv.rope_frequencies(rot)
    kw = (1 + 0.3 * torch.randn(D, generator=g)).to(dtype).cuda()
    kc = torch.full((NB, bs, Hkv, D), 0x7F, dtype=torch.uint8, device="cuda")
    vc = kc.clone()
    ks, vs = 0.004, 0.02
    out = pkv.paged_kv_write_norm_rope_fp8(q, k, v, None, kw, pos, inv, slots, kc, vc, ks, vs, interleaved=inter)
    near(out, *expect(q, None, 1e-6, pos, inv, inter, 1.0), HALF_STEP[dtype])
    want, tol = expect(k, kw, 1e-6, pos, inv, inter, 1.0)
    live = (slots >= 0).cpu().numpy()
    at = slots.cpu().numpy()[live]
    got = fp8.dequantize(kc.cpu().numpy(), ks).reshape(-1, Hkv, D)[at]
    err = np.abs(got - np.clip(want, -448 * ks, 448 * ks)[live])
    # half a step of E4M3: 2^-4 of the value, 2^-10 scale below the smallest normal; the division rounds once
    assert np.all(err <= (tol + (2.0 ** -4 + 2.0 ** -23) * (np.abs(want) + tol) + 2.0 ** -10 * ks)[live])
    rows = v.contiguous().float().cpu().numpy()
    assert np.array_equal(vc.cpu().numpy().reshape(-1, Hkv, D)[at], fp8.quantize(rows, vs)[live])
    untouched = np.ones(NB * bs, bool)
    untouched[at] = False
    assert np.all(kc.cpu().numpy().reshape(-1, Hkv, D)[untouched] == 0x7F)
    assert pkv.device_errors() == 0


def test_zero_rows_and_slots_past_the_pool():
    q = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(3, 1, 64, dtype=torch.bfloat16, device="cuda")
    kc = torch.full((1, 16, 1, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    pos = torch.tensor([0, 1, 2], device="cuda")
    slots = torch.tensor([2, 16, -1], device="cuda")
    out = pkv.paged_kv_write_norm_rope(q, k, k, None, None, pos, pkv.rope_frequencies(64), slots, kc, vc)
    assert pkv.device_errors() == pkv.DEVERR["slot_out_of_range"]
    assert torch.all(out == 0) and torch.all(kc[0, 2] == 0)
    kc[0, 2] = 5.0
    assert torch.all(kc == 5.0)


def test_refusals():
    q, k, v = make(1, 4, 4, 2, 64, torch.bfloat16, False)
    pos, inv = torch.arange(4, device="cuda"), pkv.rope_frequencies(64)
    slots = torch.arange(4, device="cuda")
    kc = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    f = pkv.paged_kv_write_norm_rope
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    k_out = torch.empty_like(k)
    bad = [
        lambda: f(q, k, v, w, w, pos, inv),                                   # nowhere to write
        lambda: f(q, k, None, w, w, pos, inv, slots, kc, kc.clone()),
        lambda: f(q, k, v, w, w, pos, inv, slots, kc),
        lambda: f(q, k, v, w[:32], w, pos, inv, slots, kc, kc.clone()),
        lambda: f(q, k, v, w, w.half(), pos, inv, slots, kc, kc.clone()),
        lambda: f(q, k, v, w, w.float(), pos, inv, slots, kc, kc.clone()),
        lambda: f(q, k, v, w, w, pos, inv, slots, kc.float(), kc.float()),
        lambda: f(q, k, v, w, w, pos.int(), inv, slots, kc, kc.clone()),
        lambda: f(q, k, v, w, w, pos, inv.float(), slots, kc, kc.clone()),
        lambda: f(q, k, v, w, w, pos, inv, slots[:3], kc, kc.clone()),
        lambda: f(q[:1].expand(4, -1, -1), k, v, w, w, pos, inv, slots, kc, kc.clone()),
        lambda: f(q, k, v, w, w, pos, inv, slots, kc, kc.clone(), k_out=k_out[:2]),
        lambda: f(q, k, v, w, w.cpu(), pos, inv, slots, kc, kc.clone()),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for eps in (0.0, -1.0, math.nan, math.inf):
        with pytest.raises(pkv.LibraryError):
            f(q, k, v, w, w, pos, inv, slots, kc, kc.clone(), eps=eps)
    assert f(q[:0], k[:0], v[:0], w, w, pos[:0], inv, slots[:0], kc, kc.clone()).shape[0] == 0
