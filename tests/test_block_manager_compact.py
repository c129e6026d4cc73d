"""BlockManager.compact: the C++ manager against the reference model call by
call, the content of every live sequence through its table after each call
(rows moved in a host pool as paged_kv_compact would), block accounting, and
the refusals.  Host code only."""
import numpy as np
import pytest

from oracle import budget as ob
from oracle.block_manager import BlockManagerModel, OutOfBlocks as ModelOOB


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_236_gb300 import build
    build.build()
    import paged_kv_cache_236_gb300 as p
    return p


class Pair:
    """The two managers in step, and a host pool of one value a slot."""

    def __init__(self, pkv, nb, bs, mb):
        self.pkv, self.bs, self.nb = pkv, bs, nb
        self.c, self.m = pkv.BlockManager(nb, bs, mb), BlockManagerModel(nb, bs, mb)
        self.pool = np.full((nb, bs, 1, 1), -1, dtype=np.int64)
        self.rows = {}      # seq -> values its cache holds, in order
        self.next = 0       # values are never reused

    def both(self, name, *args):
        try:
            want = getattr(self.m, name)(*args)
        except ModelOOB:
            with pytest.raises(self.pkv.OutOfBlocks):
                getattr(self.c, name)(*args)
            self.same()
            return None
        got = getattr(self.c, name)(*args)
        self.same()
        return got, want

    def same(self):
        assert self.c.stats() == self.m.stats()
        for s in self.m.tables:
            assert self.c.block_table(s) == self.m.block_table(s)

    def check(self):
        for s, rows in self.rows.items():
            t = self.c.block_table(s)
            got = [int(self.pool[t[j // self.bs], j % self.bs, 0, 0]) for j in range(len(rows))]
            assert got == rows, s
        held = [b for s in self.rows for b in self.c.block_table(s)]
        assert len(set(held)) == self.c.stats()["in_use"]

    def put(self, seq, slots, copies):
        for a, b in np.asarray(copies).reshape(-1, 2):
            self.pool[b] = self.pool[a]
        for x in slots:
            self.pool[x // self.bs, x % self.bs] = self.next
            self.rows[seq].append(self.next)
            self.next += 1

    def step(self, seqs, n):
        r = self.both("step", seqs, n)
        if r is None:
            return
        got, want = r
        for k in want:
            assert np.array_equal(got[k], want[k]), k
        at = 0
        for a, b in got["copies"]:
            self.pool[b] = self.pool[a]
        for s, k in zip(seqs, n):
            self.rows.setdefault(s, [])
            self.put(s, got["slot_mapping"][at:at + k], [])
            at += k

    def compact(self, rng, seqs, keep):
        r = self.both("compact", seqs, keep)
        if r is None:
            return
        got, want = r
        for k, w in zip(("block_tables", "dst_block_tables", "context_lens"), want):
            assert np.array_equal(got[k], w), k
        was = self.pool.copy()
        for i, (s, n) in enumerate(zip(seqs, keep)):
            L = len(self.rows[s])
            kept = sorted(rng.choice(L, min(L, n), replace=False).tolist()) if L > n else list(range(L))
            assert got["context_lens"][i] == len(kept)
            ob.compact_head(self.pool, got["block_tables"][i], got["dst_block_tables"][i], kept, 0, was)
            self.rows[s] = [self.rows[s][j] for j in kept]
            assert np.all(got["dst_block_tables"][i][-(-len(kept) // self.bs):] == -1)


@pytest.mark.parametrize("seed,nb,bs,mb", [(1, 60, 4, 12), (2, 30, 2, 16), (3, 200, 8, 20), (4, 24, 1, 20), (5, 40, 16, 6)])
def test_streams(pkv, seed, nb, bs, mb):
    rng = np.random.default_rng(seed)
    p = Pair(pkv, nb, bs, mb)
    tokens = {}   # of sequences never compacted, as the prefix cache takes them
    done = 0
    for it in range(500):
        live = list(p.rows)
        kind = rng.choice(["new", "step", "step", "fork", "free", "add", "compact", "compact"])
        if kind == "new" or not live:
            s = 1000 + it
            prompt = rng.integers(0, 2, int(rng.integers(1, bs * mb // 2 + 1))).tolist()
            got, want = p.both("try_get_prefix_blocks", s, prompt)
            assert got == want
            t = p.c.block_table(s)
            p.rows[s] = [int(p.pool[t[j // bs], j % bs, 0, 0]) for j in range(got)]
            r = p.both("update", s, len(prompt) - got)
            if r is None:
                p.both("free", s)
                del p.rows[s]
            else:
                assert list(r[0][0]) == list(r[1][0])
                p.put(s, r[0][0], r[0][1])
                tokens[s] = prompt
        elif kind == "step":
            seqs = [s for s in live if rng.random() < 0.5 and len(p.rows[s]) + 3 <= bs * mb]
            n = [int(rng.integers(0, 4)) for _ in seqs]
            before = {s: len(p.rows[s]) for s in seqs}
            p.step(seqs, n)
            for s, k in zip(seqs, n):
                if s in tokens and len(p.rows[s]) == before[s] + k:
                    tokens[s] = tokens[s] + [7] * k
        elif kind == "fork":
            s = live[rng.integers(len(live))]
            p.both("fork", s, 100000 + it)
            p.rows[100000 + it] = list(p.rows[s])
            if s in tokens:
                tokens[100000 + it] = tokens[s]
        elif kind == "free" and len(live) > 2:
            s = live[rng.integers(len(live))]
            p.both("free", s)
            del p.rows[s]
            tokens.pop(s, None)
        elif kind == "add":
            s = live[rng.integers(len(live))]
            if s in tokens:
                p.both("add_prefix", s, tokens[s])
            else:
                with pytest.raises(pkv.LibraryError):
                    p.c.add_prefix(s, p.rows[s])
                with pytest.raises(ValueError):
                    p.m.add_prefix(s, p.rows[s])
        elif kind == "compact":
            seqs = [s for s in live if rng.random() < 0.6]
            keep = [int(rng.integers(0, bs * mb)) if rng.random() < 0.5 else int(rng.integers(0, bs + 2)) for _ in seqs]
            short = [s for s, n in zip(seqs, keep) if n < len(p.rows[s])]
            old = {s: len(p.rows[s]) for s in short}
            p.compact(rng, seqs, keep)
            for s in short:
                if len(p.rows[s]) < old[s]:
                    tokens.pop(s, None)
                    done += 1
        p.check()
    assert done > 50


def test_shared_and_cached_blocks_keep_their_rows(pkv):
    """Two sequences on one cached prefix, both compacted in one call, and a
    third that still reads it."""
    p = Pair(pkv, 40, 4, 10)
    p.step([1], [16])
    p.both("add_prefix", 1, list(range(16)))
    for s in (2, 3):
        p.both("try_get_prefix_blocks", s, list(range(16)) + [99])
        p.rows[s] = list(p.rows[1])
        p.step([s], [6])
    shared = p.c.block_table(1)
    p.compact(np.random.default_rng(0), [2, 3], [9, 22])   # 3 is not shortened
    assert p.c.block_table(1) == shared and p.c.block_table(3)[:4] == shared
    assert not set(p.c.block_table(2)) & set(shared)
    p.check()
    p.compact(np.random.default_rng(1), [1, 3], [5, 5])
    p.check()
    # the cached prefix is still found, with its rows
    got, _ = p.both("try_get_prefix_blocks", 9, list(range(16)) + [99])
    assert got == 16 and p.c.block_table(9) == shared
    assert [int(p.pool[b, i, 0, 0]) for b in shared for i in range(4)] == list(range(16))


def test_refusals_change_nothing(pkv):
    m = pkv.BlockManager(4, 4, 4)
    m.update(1, 12)
    m.fork(1, 2)
    before = (m.stats(), m.block_table(1), m.block_table(2))
    with pytest.raises(pkv.OutOfBlocks):          # three shared blocks to replace, one free
        m.compact([1], 9)
    for bad in (([1, 1], [2, 2]), ([7], [2]), ([1], [-1])):
        with pytest.raises(pkv.LibraryError):
            m.compact(*bad)
    with pytest.raises(ValueError):
        m.compact([1, 2], [1])
    assert before == (m.stats(), m.block_table(1), m.block_table(2))
    r = m.compact([1], 4)                          # one block suffices
    assert r["context_lens"].tolist() == [4] and m.block_table(1) == [3] and m.num_tokens(1) == 4
    assert r["block_tables"][0].tolist() == before[1] + [-1] and r["dst_block_tables"][0].tolist() == [3, -1, -1, -1]
    assert m.compact([], [])["context_lens"].size == 0
    with pytest.raises(pkv.LibraryError):
        m.add_prefix(1, [1, 2, 3, 4])
    m.add_prefix(2, list(range(12)))
