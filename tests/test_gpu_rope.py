"""paged_kv_write_rope and its FP8 form against the fp64 definition.

Tolerances.  cos and sin are those of a half-turn count rounded to fp32 (off
by at most 2^-25 half turns, pi * 2^-25 radians < 1e-7) from a sincospif good
to 2 ulp (2 * 2^-24), so each is within 2.2e-7; two products and a sum round
three times (3 * 2^-24 of |x1| + |x2|).  Together under 4.1e-7 * amplitude *
(|x1| + |x2|); then one rounding to the output's type: half a step.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_236_gb300 as pkv
from gpu_util import to_f64
from oracle import budget as ob
from oracle import fp8

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def pair_sums(x, rot, interleaved):
    """|x1| + |x2| of each element's pair (0 past the rotary part)."""
    a = np.abs(x)
    out = np.zeros_like(a)
    if interleaved:
        s = a[..., 0:rot:2] + a[..., 1:rot:2]
        out[..., 0:rot:2] = out[..., 1:rot:2] = s
    else:
        s = a[..., :rot // 2] + a[..., rot // 2:rot]
        out[..., :rot // 2] = out[..., rot // 2:rot] = s
    return out


def make(seed, T, Hq, Hkv, D, dtype, fused=False, pad=0):
    g = torch.Generator().manual_seed(seed)
    if fused:
        rows = torch.randn(T, Hq + 2 * Hkv, D + pad, generator=g).to(dtype).cuda()[..., :D] if pad == 0 else None
        return rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
    return tuple(torch.randn(T, h, D, generator=g).to(dtype).cuda() for h in (Hq, Hkv, Hkv))


def check(q, k, v, pos, inv, slots, kc, vc, out, kc0, vc0, rot, interleaved, amp, scales=None):
    step = HALF_STEP[q.dtype]
    qf, kf = to_f64(q.contiguous()), to_f64(k.contiguous())
    p, f = pos.cpu().numpy(), inv.cpu().numpy()
    want = ob.rope(qf, p, f, interleaved, amp)
    tol = 4.1e-7 * amp * pair_sums(qf, rot, interleaved)
    err = np.abs(to_f64(out) - want)
    assert np.all(err <= tol + step * (np.abs(want) + tol)), float((err - tol - step * np.abs(want)).max())
    assert np.array_equal(to_f64(out)[..., rot:], qf[..., rot:])
    want_k = ob.rope(kf, p, f, interleaved, amp)
    tol_k = 4.1e-7 * amp * pair_sums(kf, rot, interleaved)
    s = slots.cpu().numpy()
    live = (s >= 0) & (s < kc.shape[0] * kc.shape[1])
    shape = (-1,) + tuple(kc.shape[2:])
    if scales is None:
        got_k, got_v = to_f64(kc).reshape(shape)[s[live]], to_f64(vc).reshape(shape)[s[live]]
        err = np.abs(got_k - want_k[live])
        assert np.all(err <= (tol_k + step * (np.abs(want_k) + tol_k))[live])
        assert np.array_equal(got_v, to_f64(v.contiguous())[live])
    else:
        ks, vs = scales
        got_k = fp8.dequantize(kc.cpu().numpy(), ks).reshape(shape)[s[live]]
        err = np.abs(got_k - np.clip(want_k[live], -448 * ks, 448 * ks))
        # half a step of E4M3: 2^-4 of the value, 2^-10 scale below the smallest normal; the division rounds once
        assert np.all(err <= (tol_k + (2.0 ** -4 + 2.0 ** -23) * (np.abs(want_k) + tol_k) + 2.0 ** -10 * ks)[live])
        vrows = v.contiguous().float().cpu().numpy()
        assert np.array_equal(vc.cpu().numpy().reshape(shape)[s[live]], fp8.quantize(vrows, vs)[live])
    untouched = np.ones(kc.shape[0] * kc.shape[1], bool)
    untouched[s[live]] = False
    as_bits = lambda t: (t.view(torch.int16) if t.dtype == torch.bfloat16 else t).cpu().numpy().reshape(shape)  # noqa: E731
    assert np.array_equal(as_bits(kc)[untouched], as_bits(kc0)[untouched], equal_nan=kc.dtype == torch.float32)
    assert np.array_equal(as_bits(vc)[untouched], as_bits(vc0)[untouched], equal_nan=kc.dtype == torch.float32)


CASES = [  # T, Hq, Hkv, D, rot, interleaved, bs, fused, skipped slots
    (1, 1, 1, 64, 64, False, 16, False, False),
    (1, 32, 8, 128, 128, False, 16, False, False),
    (7, 8, 2, 128, 64, True, 8, True, True),
    (64, 6, 3, 64, 32, False, 32, True, True),
    (33, 4, 4, 128, 128, True, 64, False, True),
    (5, 3, 1, 80, 48, False, 16, False, False),
    (5, 3, 1, 80, 48, True, 16, True, False),
    (9, 2, 2, 10, 6, False, 16, False, True),      # rows of 20 or 40 bytes: the element path
    (9, 5, 2, 18, 2, True, 16, False, True),
    (300, 12, 4, 128, 100, False, 16, True, True),  # halves of 50: the element path
    (2600, 4, 2, 64, 64, False, 16, False, True),   # several tokens to a block
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_rope_write(case, dtype):
    T, Hq, Hkv, D, rot, inter, bs, fused, skips = case
    q, k, v = make(T + D, T, Hq, Hkv, D, dtype, fused)
    g = torch.Generator().manual_seed(T)
    NB = T // bs + 3
    slots = torch.randperm(NB * bs, generator=g)[:T].cuda()
    if skips:
        slots[::3] = -1
    pos = torch.randint(0, 200000, (T,), generator=g).cuda()
    pos[-1] = 0
    inv = pkv.rope_frequencies(rot)
    kc = torch.full((NB, bs, Hkv, D), float("nan"), dtype=dtype, device="cuda")
    vc = kc.clone()
    kc0, vc0 = kc.clone(), vc.clone()
    amp = 1.0 if T % 2 else 1.25
    out = pkv.paged_kv_write_rope(q, k, v, pos, inv, slots, kc, vc, interleaved=inter, amplitude=amp)
    check(q, k, v, pos, inv, slots, kc, vc, out, kc0, vc0, rot, inter, amp)
    assert pkv.device_errors() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", [c for c in CASES if c[0] < 1000], ids=lambda c: "-".join(map(str, c)))
def test_rope_write_fp8(case, dtype):
    T, Hq, Hkv, D, rot, inter, bs, fused, skips = case
    q, k, v = make(T + D + 1, T, Hq, Hkv, D, dtype, fused)
    g = torch.Generator().manual_seed(T + 1)
    NB = T // bs + 3
    slots = torch.randperm(NB * bs, generator=g)[:T].cuda()
    if skips:
        slots[1::4] = -7
    pos = torch.randint(0, 200000, (T,), generator=g).cuda()
    inv = pkv.rope_frequencies(rot)
    kc = torch.full((NB, bs, Hkv, D), 0x7F, dtype=torch.uint8, device="cuda")
    vc = kc.clone()
    out = pkv.paged_kv_write_rope_fp8(q, k, v, pos, inv, slots, kc, vc, 0.004, 0.02, interleaved=inter)
    check(q, k, v, pos, inv, slots, kc, vc, out, torch.full_like(kc, 0x7F), torch.full_like(kc, 0x7F), rot, inter,
          1.0, (0.004, 0.02))
    assert pkv.device_errors() == 0


def test_far_and_negative_positions():
    """Angles stay exact: positions of 2^24, of 2^40 with a frequency whose
    multiples of a turn are known, and below zero."""
    pos = torch.tensor([1 << 24, -(1 << 24), -5, 3], dtype=torch.int64, device="cuda")
    q, k, v = make(3, 4, 2, 1, 64, torch.float32)
    inv = pkv.rope_frequencies(64)
    kc = torch.zeros(1, 8, 1, 64, device="cuda")
    vc = kc.clone()
    slots = torch.arange(4, device="cuda")
    out = pkv.paged_kv_write_rope(q, k, v, pos, inv, slots, kc, vc)
    # the frequency in turns is rounded to 2^-53 of itself (and once more by 1 / 2 pi): 2^24 * 2^-52 radians, below 1e-8
    want = ob.rope(to_f64(q), pos.cpu().numpy(), inv.cpu().numpy())
    tol = 4.2e-7 * pair_sums(to_f64(q), 64, False)
    assert np.all(np.abs(to_f64(out) - want) <= tol + 2.0 ** -24 * np.abs(want))
    eighth = torch.full((1,), 2 * np.pi / 8, dtype=torch.float64, device="cuda")
    pos = torch.tensor([(1 << 40) + 2, 8 << 33], dtype=torch.int64, device="cuda")
    x = torch.tensor([1.0, 2.0] + [0.0] * 62, device="cuda").expand(2, 1, 64).contiguous()
    y = pkv.paged_kv_write_rope(x, x, x, pos, eighth, slots[:2], kc, vc, interleaved=True).cpu()
    # 2 pi / 8 and 1 / (2 pi) are each rounded to 2^-53: 2^40 positions are at most 2^-11 radians off
    assert np.allclose(y[0, 0, :2], [-2, 1], atol=3 * 2.0 ** -11)
    assert np.allclose(y[1, 0, :2], [1, 2], atol=3 * 2.0 ** -11)


def test_in_place_and_out_of_range_slots():
    q, k, v = make(8, 40, 4, 2, 64, torch.bfloat16)
    pos = torch.arange(40, device="cuda")
    inv = pkv.rope_frequencies(64)
    kc = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    kc0 = kc.clone()
    slots = torch.arange(40, device="cuda")
    slots[7], slots[9] = 48, 1 << 40
    want = pkv.paged_kv_write_rope(q, k, v, pos, inv, slots, kc, vc)
    assert pkv.device_errors() == pkv.DEVERR["slot_out_of_range"]
    check(q, k, v, pos, inv, slots, kc, vc, want, kc0, kc0.clone(), 64, False, 1.0)
    q2 = q.clone()
    same = pkv.paged_kv_write_rope(q2, k, v, pos, inv, slots.clamp(max=47), kc, vc, q_out=q2)
    assert same.data_ptr() == q2.data_ptr() and torch.equal(same.view(torch.int16), want.view(torch.int16))
    pkv.device_errors()


def test_equals_separate_write_for_rotated_rows():
    """The pools hold what paged_kv_write puts there for k rotated by itself
    (position 0 turns nothing) and the attention that follows reads them."""
    q, k, v = make(9, 20, 8, 2, 128, torch.bfloat16)
    slots = torch.randperm(64, device="cuda")[:20]
    a, b, c, d = (torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    out = pkv.paged_kv_write_rope(q, k, v, torch.zeros(20, dtype=torch.int64, device="cuda"),
                                  pkv.rope_frequencies(128), slots, a, b)
    pkv.paged_kv_write(k, v, slots, c, d)
    assert torch.equal(a, c) and torch.equal(b, d) and torch.equal(out, q)


def test_refusals():
    q, k, v = make(10, 4, 4, 2, 64, torch.bfloat16)
    pos, slots = torch.arange(4, device="cuda"), torch.arange(4, device="cuda")
    inv = pkv.rope_frequencies(64)
    kc = torch.zeros(1, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    call = lambda **o: pkv.paged_kv_write_rope(**{**dict(q=q, k=k, v=v, positions=pos, inv_freq=inv, slot_mapping=slots,  # noqa: E731
                                                         k_cache=kc, v_cache=vc), **o})
    for bad in (dict(q=q.float()), dict(q=q[:3]), dict(q=q.transpose(1, 2)), dict(k=k[:, :1]), dict(v=v.float()),
                dict(positions=pos.int()), dict(positions=pos[:3]), dict(inv_freq=inv.float()),
                dict(inv_freq=pkv.rope_frequencies(128)), dict(slot_mapping=slots.int()), dict(k_cache=kc.float()),
                dict(q_out=q.float()), dict(q=q.cpu()), dict(v_cache=vc[..., :32])):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(pkv.LibraryError):
        call(amplitude=0.0)
    empty = call(q=q[:0], k=k[:0], v=v[:0], positions=pos[:0], slot_mapping=slots[:0])
    assert empty.shape == (0, 4, 64)


def test_stream_and_graph():
    q, k, v = make(11, 16, 4, 2, 64, torch.bfloat16)
    pos, slots = torch.arange(16, device="cuda"), torch.arange(16, device="cuda")
    inv = pkv.rope_frequencies(64)
    kc = torch.zeros(1, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    want = pkv.paged_kv_write_rope(q, k, v, pos, inv, slots, kc, vc)
    want_k = kc.clone()
    torch.cuda.synchronize()
    g, out = torch.cuda.CUDAGraph(), torch.empty_like(q)
    with torch.cuda.graph(g):
        pkv.paged_kv_write_rope(q, k, v, pos, inv, slots, kc, vc, q_out=out)
    pos += 3
    kc.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert not torch.equal(out, want)
    pos -= 3
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(kc, want_k)


def test_one_token_of_any_stride_and_repeated_rows():
    """A lone token's stride does not matter; one row repeated over several
    tokens (a stride of 0, which the C call takes for dense) is refused."""
    kc = torch.zeros(2, 16, 2, 64, device="cuda")
    vc = torch.zeros_like(kc)
    f = pkv.rope_frequencies(64)
    i64 = lambda x: torch.tensor(x, dtype=torch.int64, device="cuda")  # noqa: E731
    row = torch.randn(1, 2, 64, device="cuda")
    want = pkv.paged_kv_write_rope(row, row, row, i64([5]), f, i64([3]), kc, vc)
    lone = row.as_strided((1, 2, 64), (0, 64, 1))
    assert torch.equal(pkv.paged_kv_write_rope(lone, lone, lone, i64([5]), f, i64([4]), kc, vc), want)
    assert torch.equal(kc[0, 3], kc[0, 4]) and torch.equal(vc[0, 4], row[0])
    many, dense = row.expand(3, 2, 64), row.repeat(3, 1, 1)
    for at in range(3):
        rows = [many if i == at else dense for i in range(3)]
        with pytest.raises(ValueError):
            pkv.paged_kv_write_rope(*rows, i64([0, 1, 2]), f, i64([0, 1, 2]), kc, vc)


def _turns(positions, inv_freq):
    """Fractions of a turn of positions x frequencies, in integers: 1 / (2 pi) to
    400 bits by Machin's formula, frequencies as the rationals they are."""
    one = 1 << 400

    def arctan_of_1_over(x):
        total = term = one // x
        n, sign = 3, -1
        while term:
            term //= x * x
            total += sign * (term // n)
            n, sign = n + 2, -sign
        return total
    two_pi = 8 * (4 * arctan_of_1_over(5) - arctan_of_1_over(239))
    out = np.empty((len(positions), len(inv_freq)))
    for i, f in enumerate(inv_freq):
        num, den = float(f).as_integer_ratio()
        for t, p in enumerate(positions):
            turns = ((int(p) * num * one << 400) // (den * two_pi)) % one
            out[t, i] = turns / one
    return out


@pytest.mark.parametrize("interleaved", [False, True])
def test_positions_of_any_size(interleaved):
    """Every int64 position, to its ends, and frequencies up to 2^31, of either
    sign: the bound of the near positions."""
    pos = [1 << 31, (1 << 40) + 12345, 1 << 50, -(1 << 50) - 7, 3 * (1 << 60) + 99, (1 << 63) - 1, -(1 << 63), -(1 << 62) + 1]
    inv = pkv.rope_frequencies(64)
    inv[1], inv[5], inv[9], inv[13], inv[17] = 1e-300, 0.0, -0.3, 1000.1, float(2 ** 31) + 0.7
    n = len(pos)
    q, k, v = make(17, n, 3, 2, 64, torch.float32)
    kc = torch.zeros(1, 16, 2, 64, device="cuda")
    out = pkv.paged_kv_write_rope(q, k, v, torch.tensor(pos, dtype=torch.int64, device="cuda"), inv,
                                  torch.arange(n, device="cuda"), kc, kc.clone(), interleaved=interleaved)
    a = 2 * np.pi * _turns(pos, inv.cpu().numpy())
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    first, second = (slice(0, 64, 2), slice(1, 64, 2)) if interleaved else (slice(0, 32), slice(32, 64))
    for got, x in ((to_f64(out), to_f64(q)), (to_f64(kc)[0, :n], to_f64(k))):
        want = np.empty_like(x)
        want[..., first] = x[..., first] * c - x[..., second] * s
        want[..., second] = x[..., second] * c + x[..., first] * s
        # 2^31 * 2^-63 of a turn more than near positions, below 2e-9 radians
        tol = 4.2e-7 * pair_sums(x, 64, interleaved)
        assert np.all(np.abs(got - want) <= tol + 2.0 ** -24 * np.abs(want))
