"""paged_kv_write_fp8block into blocks whose scales the caller put there.

The rule is stated in fp32 operations (a product with the reciprocal of the
scale, both rounded once), which are made here one by one: codes and scales are
equal, nothing to tolerate.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_236_gb300 as pkv
from oracle import fp8, serving

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [40, 600])  # both ways of finding a block's rows
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_any_scale_that_was_there(T, dtype):
    g = torch.Generator().manual_seed(T)
    bs, Hkv, D, NB = 16, 2, 64, T // 4
    put = [0.7, 0.01, 1e-3, 3.0, 0.0, -2.0, float("nan"), 1e-8, 0.25, 1.1e4]
    scales = torch.tensor(put)[torch.randint(0, len(put), (2, NB, Hkv), generator=g)]
    codes = torch.randint(0, 256, (2, NB, bs, Hkv, D), generator=g, dtype=torch.int32).to(torch.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0
    rows = (torch.exp(2 * torch.randn(T, 1, 1, generator=g)) * torch.randn(T, 2 * Hkv, D, generator=g)).to(dtype)
    blocks = torch.arange(T) // 4
    slots = blocks * bs + 1 + torch.randint(0, 3, (T,), generator=g) + 3 * (torch.arange(T) % 4)  # never the first
    dev = [t.cuda() for t in (rows[:, :Hkv], rows[:, Hkv:], slots)]
    kc, vc, ks, vs = codes[0].cuda(), codes[1].cuda(), scales[0].cuda(), scales[1].cuda()
    pkv.paged_kv_write_fp8block(*dev, kc, vc, ks, vs)
    one = np.float32(1)
    for x, c, s, got_c, got_s in ((rows[:, :Hkv], codes[0], scales[0], kc, ks), (rows[:, Hkv:], codes[1], scales[1], vc, vs)):
        x, c, s = x.float().numpy(), c.numpy().copy(), s.numpy()
        want_s = s.copy()
        for b in range(NB):
            mine = np.arange(4 * b, 4 * b + 4)
            for h in range(Hkv):
                old = s[b, h] if s[b, h] > 0 else np.float32(0)
                now = max(old, np.float32(serving.block_scale(float(np.abs(x[mine, h]).max()))))
                by = one / now
                if now > old:
                    values = fp8.dequantize(c[b, :, h], 1.0).astype(np.float32)
                    c[b, :, h] = fp8.e4m3_encode(values * (old * by))
                for t in mine:
                    c[b, int(slots[t]) % bs, h] = fp8.e4m3_encode(x[t, h] * by)
                want_s[b, h] = now
        assert np.array_equal(got_s.cpu().numpy(), want_s)
        assert np.array_equal(got_c.cpu().numpy(), c)
    assert pkv.device_errors() == 0
