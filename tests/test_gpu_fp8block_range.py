"""paged_attention_forward_fp8block at the ends of its ranges: q, K's scales and
the logit scale by powers of two apart.

Powers of two that cancel leave every logit what it was, so the tolerances are
those of the operator's other tests: weights of 9 bits or more (2^-9 of each), q's
split (2^-17 of a row's largest |q| in each of 128 products, of random sign: below
2^-7 of a unit of logit), the output's half step (2^-9 below a power of two), of
values up to 4.5: below 4e-2 in all, the mean error, of random signs, a tenth.
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
