"""Rows of one tile whose running maximum rises at different key tiles.

The multi-token kernel keeps a row's reference maximum until a tile exceeds it
by 8 in log2 units; here that happens in every key tile, for some rows of a
warp and not for others.  Tolerance as the other bf16 attention tests'.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_236_gb300 as pkv
from gpu_util import check_close, to_f64
from oracle import paged_oracle as po

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,L", [(64, 640), (33, 515), (300, 300)])
def test_some_rows_raise_their_maximum(n, L, D):
    Hq, Hkv, bs = 8, 2, 16
    g = torch.Generator().manual_seed(n)
    blocks = -(-L // bs)
    kc = torch.randn(blocks + 1, bs, Hkv, D, generator=g)
    vc = torch.randn(blocks + 1, bs, Hkv, D, generator=g)
    q = torch.randn(n, Hq, D, generator=g)
    # one component carries a logit that climbs by 10 a tile for the even heads and falls for the odd ones
    scale = D ** -0.5
    tile = (torch.arange((blocks + 1) * bs) // 128).view(blocks + 1, bs, 1)
    kc[..., 0] = 2.0 * tile
    q[..., 0] = 5.0 / scale * torch.tensor([1.0, -1.0]).repeat(Hq // 2)
    kc, vc, q = (t.to(torch.bfloat16).cuda() for t in (kc, vc, q))
    tables = torch.arange(blocks, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    qsl = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    out = pkv.paged_attention_forward(q, kc, vc, tables, lens, qsl, scale)
    want = po.paged_attention(to_f64(q), to_f64(kc), to_f64(vc), tables.cpu().numpy(), [L], [0, n], scale, True)
    check_close(to_f64(out), want, "bf16")
    assert pkv.device_errors() == 0
    assert np.isfinite(want).all()
