"""Pins of the page oracle (oracle/kv_pages.py): worked examples by hand, and
the invariant that the counts always equal what the table holds."""
import numpy as np
import pytest

from oracle import attention, kv_pages


def counts(table, pages):
    return np.bincount(table[table >= 0].ravel(), minlength=pages)


def test_fork_reserve_release_by_hand():
    # one sequence of 5 positions on pages of 4: pages 2, 0; page 1 and 3..5 free
    table = np.array([[2, 0, -1], [-1, -1, -1], [-1, -1, -1]], dtype=np.int32)
    ref = np.array([1, 0, 1, 0, 0, 0], dtype=np.int32)
    seq_len = np.array([5, 0, 0], dtype=np.int32)
    pool = np.arange(6 * 4, dtype=np.int32).reshape(1, 6, 4, 1)
    assert not kv_pages.fork(np.array([0, 0]), np.array([1, 2]), seq_len, table, ref, 4)
    assert table.tolist() == [[2, 0, -1]] * 3 and ref.tolist() == [3, 0, 3, 0, 0, 0] and seq_len.tolist() == [5] * 3
    assert not kv_pages.reserve(np.array([4, 1, 1]), seq_len, table, ref, pool, 4)
    # sequence 0 writes 5..8: its own copy of the partial page (1) and a new page (3); 1 copies (4); 2 keeps page 0
    assert table.tolist() == [[2, 1, 3], [2, 4, -1], [2, 0, -1]]
    assert ref.tolist() == [1, 1, 3, 1, 1, 0]
    assert pool[0, 1, 0, 0] == pool[0, 4, 0, 0] == pool[0, 0, 0, 0] == 0 and pool[0, 1, 1, 0] == 5
    assert not kv_pages.release(np.array([-1, 0, 4]), seq_len, table, ref, 4)
    assert table.tolist() == [[2, 1, 3], [-1, -1, -1], [2, -1, -1]]
    assert ref.tolist() == [0, 1, 2, 1, 0, 0] and seq_len.tolist() == [5, 0, 4]
    errors, live = kv_pages.compact(table, ref, pool)
    assert not errors and live == 3
    assert table.tolist() == [[2, 1, 0], [-1, -1, -1], [2, -1, -1]] and ref.tolist() == [1, 1, 2, 0, 0, 0]


def test_reserve_is_all_or_nothing():
    table = np.full((2, 4), -1, dtype=np.int32)
    ref = np.zeros(3, dtype=np.int32)
    before = table.copy()
    assert kv_pages.reserve(np.array([4, 4]), np.zeros(2, int), table, ref, np.zeros((1, 3, 2, 1)), 2) == {"POOL"}
    assert (table == before).all() and not ref.any()


@pytest.mark.parametrize("seed", range(5))
def test_counts_follow_the_table(seed):
    rng = np.random.default_rng(seed)
    B, cols, P, ps = 6, 8, 40, 3
    table = np.full((B, cols), -1, dtype=np.int32)
    ref = np.zeros(P, dtype=np.int32)
    seq_len = np.zeros(B, dtype=np.int32)
    pool = rng.integers(0, 100, (2, P, ps, 2))
    told = {b: [] for b in range(B)}      # what every position of every sequence should hold
    for step in range(60):
        need = rng.integers(0, 4, B).astype(np.int32)
        if not kv_pages.reserve(need, seq_len, table, ref, pool, ps):
            for b in range(B):
                for _ in range(need[b]):
                    x = int(rng.integers(100, 10**6))
                    pool[:, table[b, seq_len[b] // ps], seq_len[b] % ps] = x
                    told[b].append(x)
                    seq_len[b] += 1
        cut = np.where(rng.random(B) < 0.3, rng.integers(0, seq_len + 1), -1)
        assert not kv_pages.release(cut, seq_len, table, ref, ps)
        for b in range(B):
            if cut[b] >= 0:
                told[b] = told[b][:cut[b]]
        s, d = rng.permutation(B)[:2]
        if not kv_pages.fork(np.array([s]), np.array([d]), seq_len, table, ref, ps):
            told[d] = list(told[s])
        if step % 7 == 0:
            errors, live = kv_pages.compact(table, ref, pool)
            assert not errors and live == (ref > 0).sum() == (ref[:live] > 0).sum()
        assert (counts(table, P) == ref).all()
        for b in range(B):
            got = [pool[0, table[b, i // ps], i % ps, 0] for i in range(seq_len[b])]
            assert got == told[b]


def test_path_in_place_equals_staged():
    rng = np.random.default_rng(3)
    B, N, ps = 3, 9, 4
    table = rng.permutation(B * 8).reshape(B, 8).astype(np.int32)
    seq_len = np.array([0, 5, 11], dtype=np.int32)
    path = np.full((B, N), -1, dtype=np.int32)
    path[0, :3], path[1, :2] = [1, 4, 8], [3, 5]
    n = np.array([3, 2, -1])
    pool = rng.integers(0, 100, (2, B * 8, ps, 3))
    staged = np.zeros((2, B, N, 3), dtype=pool.dtype)
    for b in range(B):
        for i in range(N):
            pos = seq_len[b] + i
            staged[:, b, i] = pool[:, table[b, pos // ps], pos % ps]
    one, two, l1, l2 = pool.copy(), pool.copy(), seq_len.copy(), seq_len.copy()
    assert not kv_pages.commit_path(n, path, l1, table, one, None, ps)
    assert not kv_pages.commit_path(n, path, l2, table, two, staged, ps)
    assert (one == two).all() and (l1 == l2).all() and l1.tolist() == [4, 8, 11]
    path[0, 1] = 1
    assert kv_pages.commit_path(n, path, l1, table, one, None, ps) == {"PATH"}


def test_attention_oracle_by_hand():
    q = np.array([[[1.0, 0.0]], [[0.0, 2.0]]])
    k = np.array([[[1.0, 0.0]], [[0.0, 1.0]], [[5.0, 5.0]]])
    v = np.array([[[1.0, 2.0]], [[3.0, 4.0]], [[np.nan, np.inf]]])
    see = np.array([[True, False, False], [True, True, False]])
    out, lse, _, _ = attention.rows(q, k, v, see, 0.5)
    assert out[0, 0].tolist() == [1.0, 2.0] and lse[0, 0] == 0.5
    w = np.exp([0.0, 1.0]) / np.exp([0.0, 1.0]).sum()
    assert np.allclose(out[1, 0], w @ v[:2, 0]) and np.isclose(lse[1, 0], np.log(1 + np.e))
    out, lse, _, _ = attention.rows(q, k, v, np.zeros((2, 3), bool), 0.5)
    assert not out.any() and (lse == -np.inf).all()
    assert attention.ancestors([-1, 0, 0, 1]).tolist() == [[1, 0, 0, 0], [1, 1, 0, 0], [1, 0, 1, 0], [1, 1, 0, 1]]
    assert attention.chain_mask(2, 4).tolist() == [[1, 1, 1, 0], [1, 1, 1, 1]]
    assert attention.chain_mask(3, 1).tolist() == [[0], [0], [1]]


def test_compact_reports_an_entry_of_a_page_that_is_filled():
    # pages 3 and 4 are live and move to 0 and 1; sequence 1 names page 1, free before and another's afterwards
    table = np.array([[3, 4], [1, -1]], dtype=np.int32)
    ref = np.array([0, 0, 0, 1, 1, 0], dtype=np.int32)
    pool = np.arange(6).reshape(1, 6, 1, 1)
    assert kv_pages.compact(table, ref, pool) == ({"PAGE"}, 2)
    assert table.tolist() == [[0, 1], [1, -1]] and ref.tolist() == [1, 1, 0, 0, 0, 0]
    assert kv_pages.compact(table[:1], ref, pool) == (set(), 2)
