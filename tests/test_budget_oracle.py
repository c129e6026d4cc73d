"""Pins of the fp64 definitions in oracle/budget.py: closed forms, brute force
and torch as a black box."""
import math

import numpy as np
import pytest
import torch

from oracle import budget as ob


def test_rope_quarter_turn_and_copy():
    x = np.arange(1.0, 7.0).reshape(1, 1, 6)
    y = ob.rope(x, np.array([1]), np.array([math.pi / 2, math.pi]))
    # pairs (1, 3) by a quarter turn, (2, 4) by a half turn; 5, 6 copied
    assert np.allclose(y[0, 0], [-3, -2, 1, -4, 5, 6], atol=1e-15)
    y = ob.rope(x, np.array([1]), np.array([math.pi / 2, math.pi]), interleaved=True, amplitude=2.0)
    assert np.allclose(y[0, 0], [-4, 2, -6, -8, 5, 6], atol=1e-14)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_scores_depend_on_distance(interleaved):
    rng = np.random.default_rng(3)
    f = 10000.0 ** (-np.arange(0, 16, 2) / 16)
    q, k = rng.standard_normal((2, 1, 1, 16))
    at = lambda x, p: ob.rope(x, np.array([p]), f, interleaved)[0, 0]  # noqa: E731
    base = at(q, 7) @ at(k, 3)
    assert at(q, 107) @ at(k, 103) == pytest.approx(base, abs=1e-11)
    assert np.linalg.norm(at(q, 99)) == pytest.approx(np.linalg.norm(q), rel=1e-13)
    assert np.array_equal(at(q, 0), q[0, 0])


def test_rope_equals_complex_product():
    rng = np.random.default_rng(4)
    x = rng.standard_normal((5, 3, 8))
    pos = np.array([0, 1, 17, 4096, 131071])
    f = 500000.0 ** (-np.arange(0, 8, 2) / 8)
    z = np.exp(1j * pos[:, None] * f)[:, None]
    w = (x[..., 0::2] + 1j * x[..., 1::2]) * z
    y = ob.rope(x, pos, f, True)
    assert np.allclose(y[..., 0::2], w.real, atol=1e-10) and np.allclose(y[..., 1::2], w.imag, atol=1e-10)


def test_scores_closed_forms():
    # equal keys: every visible key gets the same weight
    K = np.ones((6, 2, 4))
    q = np.random.default_rng(0).standard_normal((2, 4, 4))
    w = ob.scores_update(q, K, np.zeros((2, 6)), 0.5)
    assert np.allclose(w, [[2 / 5 + 2 / 6] * 5 + [2 / 6]] * 2)
    w = ob.scores_update(q, K, np.zeros((2, 6)), 0.5, causal=False)
    assert np.allclose(w, 4 / 6)
    # a row's weights sum to one, old weight counts below the step's tokens only
    old = np.arange(12.0).reshape(2, 6)
    w2 = ob.scores_update(q, K, old, 0.5, decay=0.25)
    assert np.allclose(w2[:, :4], [[2 / 5 + 2 / 6] * 4] * 2 + 0.25 * old[:, :4]) and np.allclose(w2[:, 5], 2 / 6)
    assert np.array_equal(ob.scores_update(q[:0], K, old, 0.5), old)


def test_scores_equal_softmax():
    rng = np.random.default_rng(5)
    n, L, Hq, Hkv, D = 3, 9, 4, 2, 8
    q, K = rng.standard_normal((n, Hq, D)), rng.standard_normal((L, Hkv, D))
    got = ob.scores_update(q, K, np.zeros((Hkv, L)), 0.3)
    z = torch.einsum("ihd,jhd->hij", torch.from_numpy(q), torch.from_numpy(K).repeat_interleave(2, 1)) * 0.3
    z = z.masked_fill(torch.ones(n, L, dtype=torch.bool).triu(L - n + 1), -math.inf)
    want = torch.softmax(z, -1).sum(1).view(Hkv, 2, L).sum(1).numpy()
    assert np.allclose(got, want, atol=1e-14)


def test_select_by_hand_and_brute_force():
    s = np.array([5, 1, 9, 9, 2, 9, 0, 0.5])
    assert ob.select(s, 8, 5, 1, 1) == [0, 2, 3, 5, 7]
    assert ob.select(s, 8, 4, 1, 1) == [0, 2, 3, 7]      # of the equal 9s the lower positions
    assert ob.select(s, 4, 4, 1, 1) == [0, 1, 2, 3] and ob.select(s, 0, 4) == []
    assert ob.select(s, 8, 2, 1, 1) == [0, 7]
    s[2] = np.nan
    assert ob.select(s, 8, 4, 1, 1) == [0, 3, 5, 7]
    assert ob.select(np.array([-np.inf, np.nan, -0.0, 0.0]), 4, 1) == [2]
    rng = np.random.default_rng(1)
    for _ in range(50):
        L, b = int(rng.integers(1, 20)), int(rng.integers(1, 20))
        s = rng.integers(0, 4, L).astype(float)
        kept = ob.select(s, L, b)
        assert len(kept) == min(L, b) and kept == sorted(set(kept))
        gone = sorted(set(range(L)) - set(kept))
        assert not gone or not kept or min(s[kept]) >= max(s[gone])
        for j in gone:  # an equal score that was kept sits lower
            assert all(i < j for i in kept if s[i] == s[j])


def test_compact_moves_rows_in_order():
    pool = np.arange(4 * 2 * 2 * 1).reshape(4, 2, 2, 1)
    was = pool.copy()
    table = [3, 1, 0]
    ob.compact_head(pool, table, table, [0, 3, 4], 1)
    assert pool[3, 0, 1] == was[3, 0, 1] and pool[3, 1, 1] == was[1, 1, 1] and pool[1, 0, 1] == was[0, 0, 1]
    assert np.array_equal(pool[:, :, 0], was[:, :, 0])
