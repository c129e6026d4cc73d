"""paged_attention_forward_fp8block at the ends of its ranges: q, K's scales and
the logit scale by powers of two apart, and rows of q that are not finite.

Powers of two that cancel leave every logit what it was, so the tolerances are
those of the operator's other tests.  They follow from weights of 9 bits or more
(2^-9 of each), q's split (2^-17 of a row's largest |q|, below 9, in each of 128
products with values of K below 16, of random sign, times 2^-3.5: below 2^-9 of a
unit of logit) and the output's rounding (2^-8), of values up to 4.5: below 3.6e-2,
taken as 4e-2; the mean error, of random signs, a tenth.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_236_gb300 as pkv
from gpu_util import to_f64
from test_gpu_fp8block_attention import Batch

pytestmark = pytest.mark.gpu

QUERIES = [[1, 1], [3, 4], [64, 5]]


def apart(seed, n, q, k, scale):
    """A batch whose q, K scales and logit scale are 2^q, 2^k and 2^scale times the usual."""
    b = Batch(seed, [600, 300], n, 8, 2, 16)
    assert np.nanmax(b.scales[0]) * 2.0 ** k <= 2.0 ** 60 and np.nanmin(b.scales[0]) * 2.0 ** k >= 2.0 ** -60
    b.q = b.q * 2.0 ** q
    b.scales[0] = (b.scales[0].astype(np.float64) * 2.0 ** k).astype(np.float32)
    b.scale *= 2.0 ** scale
    b.up()
    return b


@pytest.mark.parametrize("n", QUERIES)
@pytest.mark.parametrize("q,k,scale", [(-60, 60, 0), (-64, 64, 0), (-64, 0, 64), (-110, 60, 50), (-40, 0, 40),
                                       (48, -48, 0), (60, 0, -60), (96, -48, -48), (0, 60, -60), (0, -48, 48)])
def test_powers_of_two_that_cancel(q, k, scale, n):
    b = apart(31, n, q, k, scale)
    b.check(pkv.paged_attention_forward_fp8block(*b.args))
    b.check(pkv.paged_attention_forward_fp8block(*b.args, window=200, num_sink=3), 200, 3)
    assert pkv.device_errors() == 0


@pytest.mark.parametrize("n", QUERIES)
def test_rows_of_q_of_every_magnitude(n):
    """Tokens from 2^-110 to 2^0 side by side over K of 2^60 and a small logit scale: most see
    logits of next to nothing, and a mean of V."""
    b = apart(32, n, 0, 60, -60)
    size = torch.exp2(-10.0 * (torch.arange(b.q.shape[0]) % 12))
    b.q = (b.q.float() * size[:, None, None]).to(torch.bfloat16)
    b.up()
    b.check(pkv.paged_attention_forward_fp8block(*b.args))


@pytest.mark.parametrize("n", QUERIES)
def test_rows_of_q_that_are_not_finite(n):
    """A NaN makes its row NaN, an infinity its row what it will: no other row moves."""
    b = Batch(33, [600, 300], n, 8, 2, 16)
    want = pkv.paged_attention_forward_fp8block(*b.args)
    b.check(want)
    q = b.args[0].clone()
    last = q.shape[0] - 1
    q[0, 1, 5], q[last, 6, 127], q[last, 2, 0] = float("nan"), float("inf"), float("-inf")
    got = pkv.paged_attention_forward_fp8block(q, *b.args[1:])
    assert pkv.device_errors() == 0
    assert torch.isnan(got[0, 1]).all()
    for t, h in ((0, 1), (last, 6), (last, 2)):
        got[t, h] = want[t, h]
    assert torch.equal(got, want)


@pytest.mark.parametrize("n", [1, 64])
@pytest.mark.parametrize("part", [0.5, 0.75, 1.0, 1.25, 1.5, 2.5, 3.0])
def test_the_split_of_q_at_its_bound(n, part):
    """An element of part * 2^-17 beside a largest one of 1 meets a large K: the logit is off by at
    most 2^-17 |k|.  Two keys with V of 1 and 0, so that the output is the sigmoid of the logit; a
    sixteenth for the roundings of the weights and the output (2^-7 of p, over 1 - p >= 0.2)."""
    one = torch.tensor([448.0, 1.0]).to(torch.float8_e4m3fn).view(torch.uint8)
    codes = torch.zeros(2, 1, 16, 1, 128, dtype=torch.uint8)
    codes[0, 0, 0, 0, 1], codes[1, 0, 0] = one[0], one[1]
    kc, vc = codes.cuda()
    k_scale, v_scale = torch.full((1, 1), 2.0 ** 7, device="cuda"), torch.ones(1, 1, device="cuda")
    q = torch.zeros(n, 8, 128, dtype=torch.bfloat16)
    q[..., 0], q[..., 1] = 1.0, part * 2.0 ** -17
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    # n queries of two keys each: n sequences, or one of many rows with the mask left out
    k = 448 * 2.0 ** 7
    if n == 1:
        args = i32(0).view(1, 1), i32(2), i32(0, 1)
        out = pkv.paged_attention_forward_fp8block(q.cuda(), kc, vc, k_scale, v_scale, *args, 1.0)
        p = to_f64(out)
        logit = np.log(p / (1 - p))
    else:  # keys 2 .. n - 1 are zeros too: the first key's odds against n - 1 others
        blocks = n // 16
        kc, vc = (torch.cat([c] + [torch.zeros_like(c)] * (blocks - 1)) for c in (kc, vc))
        k_scale, v_scale = k_scale.repeat(blocks, 1), v_scale.repeat(blocks, 1)
        vc[0, 0] = int(one[1])
        args = i32(*range(blocks)).view(1, blocks), i32(n), i32(0, n)
        out = pkv.paged_attention_forward_fp8block(q.cuda(), kc, vc, k_scale, v_scale, *args, 1.0, False)
        p = to_f64(out)
        logit = np.log(p * (n - 1) / (1 - p))
    true = part * 2.0 ** -17 * k
    assert np.all(np.abs(logit - true) <= 2.0 ** -17 * k + 1 / 16), (logit.min(), logit.max(), true)
