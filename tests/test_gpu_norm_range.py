"""paged_kv_write_norm_rope at the ends of its range: elements just below 2^60,
where the squares of a long head add up past fp32's.

Tolerances are those of the operator's other tests: 2.8e-6 + 6e-7 of the two
normed values of a pair for the fp32 arithmetic (80 roundings of the sum of
squares, half of that in the root, five more of the factors), and half a step
of the output's type.  An eighth of a lane's sum is exact.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_236_gb300 as pkv
from gpu_util import to_f64
from oracle import budget as ob
from oracle import serving

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TOP = {torch.bfloat16: 2.0 ** 60 * (1 - 2.0 ** -8), torch.float32: 2.0 ** 60 * (1 - 2.0 ** -24)}
REL = 2.8e-6 + 6e-7

CASES = [  # T, Hq, Hkv, D, rot, interleaved
    (3, 2, 1, 128, 128, False),
    (3, 2, 1, 256, 256, True),
    (3, 2, 1, 512, 512, False),
    (3, 2, 1, 512, 6, False),      # halves of 3: by the element
    (3, 2, 1, 1024, 1024, False),
    (2, 3, 2, 1024, 64, True),
    (2, 1, 1, 1024, 2, True),      # by the element
    (4, 2, 1, 1000, 1000, True),
    (1300, 1, 1, 512, 512, False),  # tokens enough for bulk copies
    (1300, 1, 1, 512, 64, True),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_heads_of_the_largest_elements(case, dtype):
    T, Hq, Hkv, D, rot, inter = case
    g = torch.Generator().manual_seed(D + T)
    sign = lambda h: (2.0 * torch.randint(0, 2, (T, h, D), generator=g) - 1).double()  # noqa: E731
    q, k = ((sign(h) * TOP[dtype]).to(dtype).cuda() for h in (Hq, Hkv))
    pos = torch.arange(T).cuda()
    inv = pkv.rope_frequencies(rot)
    w = (1 + 0.3 * torch.randn(D, generator=g)).cuda()
    k_out = torch.empty_like(k)
    q_out = pkv.paged_kv_write_norm_rope(q, k, None, w, None, pos, inv, interleaved=inter, k_out=k_out)
    for x, weight, got in ((q, w, q_out), (k, None, k_out)):
        z = serving.head_norm(to_f64(x), None if weight is None else to_f64(weight), 1e-6)
        want = ob.rope(z, pos.cpu().numpy(), inv.cpu().numpy(), inter, 1.0)
        tol = REL * 2 * np.abs(z).max(-1, keepdims=True)
        err = np.abs(to_f64(got) - want)
        assert np.all(err <= tol + HALF_STEP[dtype] * (np.abs(want) + tol)), float(err.max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_small_elements_follow_eps(dtype):
    """Squares far below eps, and below fp32's normal numbers: x / sqrt(eps)."""
    x = torch.full((2, 1, 1024), 2.0 ** -70, dtype=dtype, device="cuda")
    k_out = torch.empty_like(x)
    q_out = pkv.paged_kv_write_norm_rope(x, x, None, None, None, torch.zeros(2, dtype=torch.int64, device="cuda"),
                                         pkv.rope_frequencies(2), eps=2.0 ** -40, k_out=k_out)
    assert torch.equal(k_out, q_out)
    assert float((q_out.double() * 2.0 ** 50 - 1).abs().max()) <= REL + HALF_STEP[dtype]
