"""Page operators and the tree path commit on the GPU against the serial oracle
(oracle/kv_pages.py): tables, counts, lengths and pool contents bit-exact."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_67_gb300 as sv
from oracle import kv_pages

pytestmark = pytest.mark.gpu

BITS = dict(CAPACITY=1, PAGE=2, LENGTH=4, PATH=8, REF=16, PAIR=32, BUSY=64, POOL=128)


def word(errors):
    return sum(BITS[e] for e in errors)


class State:
    """The same cache on the GPU and in the oracle."""

    def __init__(self, B, cols, pages, page_size, layers=2, width=8, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.ps = page_size
        self.table = np.full((B, cols), -1, dtype=np.int32)
        self.ref = np.zeros(pages, dtype=np.int32)
        self.seq_len = np.zeros(B, dtype=np.int32)
        self.pool = torch.randint(-30000, 30000, (layers, pages, page_size, width), generator=g,
                                  dtype=torch.int16).numpy()
        self.upload()
        self.ws = sv.kv_pages_workspace(self.d_table, self.d_ref)

    def upload(self):
        self.d_table, self.d_ref, self.d_len, self.d_pool = (
            torch.from_numpy(x.copy()).cuda() for x in (self.table, self.ref, self.seq_len, self.pool))

    def check(self, errors):
        assert sv.kv_pages_read_error(self.ws) == word(errors)
        assert np.array_equal(self.d_table.cpu().numpy(), self.table)
        assert np.array_equal(self.d_ref.cpu().numpy(), self.ref)
        assert np.array_equal(self.d_len.cpu().numpy(), self.seq_len)
        assert np.array_equal(self.d_pool.cpu().numpy(), self.pool)

    def release(self, new_len):
        e = kv_pages.release(new_len, self.seq_len, self.table, self.ref, self.ps)
        d = None if new_len is None else dev(new_len)
        sv.spec_kv_release(d, self.d_len, self.d_table, self.d_ref, self.ps, workspace=self.ws)
        self.check(e)
        return e

    def fork(self, src, dst):
        src, dst = np.asarray(src, dtype=np.int32), np.asarray(dst, dtype=np.int32)
        e = kv_pages.fork(src, dst, self.seq_len, self.table, self.ref, self.ps)
        sv.spec_kv_fork(dev(src), dev(dst), self.d_len, self.d_table, self.d_ref, self.ps, workspace=self.ws)
        self.check(e)
        return e

    def reserve(self, need):
        need = np.asarray(need, dtype=np.int32)
        e = kv_pages.reserve(need, self.seq_len, self.table, self.ref, self.pool, self.ps)
        sv.spec_kv_reserve(dev(need), self.d_len, self.d_table, self.d_ref, self.d_pool, workspace=self.ws)
        self.check(e)
        return e

    def compact(self):
        e, live = kv_pages.compact(self.table, self.ref, self.pool)
        out = torch.full((1,), -5, dtype=torch.int32, device="cuda")
        sv.spec_kv_compact(self.d_table, self.d_ref, self.d_pool, out_num_live=out, workspace=self.ws)
        assert int(out) == live
        self.check(e)
        return e

    def grow(self, by):
        self.seq_len += np.asarray(by, dtype=np.int32)
        self.d_len.copy_(torch.from_numpy(self.seq_len))


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


@pytest.mark.parametrize("B,cols,pages,ps,layers,width", [(1, 3, 4, 1, 1, 8), (7, 9, 50, 3, 2, 520),
                                                          (40, 6, 300, 16, 3, 2048), (1100, 4, 5000, 2, 1, 8)])
def test_random_rounds(B, cols, pages, ps, layers, width):
    rng = np.random.default_rng(B + pages)
    st = State(B, cols, pages, ps, layers, width, seed=B)
    for step in range(12):
        need = rng.integers(0, 2 * ps + 1, B)
        need = np.minimum(need, cols * ps - st.seq_len)
        if not st.reserve(need):
            st.grow(need)
        st.release(np.where(rng.random(B) < 0.3, rng.integers(0, st.seq_len + 1), -1))
        if B > 1:
            perm = rng.permutation(B)
            n = max(1, B // 4)
            st.release(np.where(np.isin(np.arange(B), perm[:n]), 0, -1))
            st.fork(perm[n + np.arange(n) % max(1, B - n)], perm[:n])
        if step % 3 == 2:
            st.compact()
        if step % 4 == 3:
            st.release(None)
    st.release(np.zeros(B, dtype=np.int32))
    assert not st.ref.any() and (st.table == -1).all()


def test_shared_partial_page_with_every_number_of_writers():
    for writers in range(1, 6):
        st = State(5, 4, 30, 8, seed=writers)
        st.reserve([5, 0, 0, 0, 0])
        st.grow([5, 0, 0, 0, 0])
        st.fork([0] * 4, [1, 2, 3, 4])
        st.reserve([3 if b >= 5 - writers else 0 for b in range(5)])
        st.reserve([9] * 5)


def test_refusals_leave_the_sequence_alone():
    st = State(6, 4, 40, 4)
    st.reserve([6, 6, 6, 6, 0, 0])
    st.grow([6, 6, 6, 6, 0, 0])
    assert st.reserve([100, -1, 1, 0, 0, 0]) == {"CAPACITY", "LENGTH"}
    assert st.release(np.array([7, -1, 2, -1, 0, 0])) == {"LENGTH"}
    assert st.fork([0, 1, 9, 3, 4, 4], [4, 4, 5, 3, 0, 0]) == {"PAIR"}
    assert st.fork([0], [1]) == {"BUSY"}
    assert st.fork([0, 1], [4, 5]) == set()
    assert st.fork([4, 0], [5, 4]) == {"PAIR", "BUSY"}
    # a page id behind the pool, a missing page under committed positions, a count below 1, a negative length
    st.table[0, 1], st.table[1, 1], st.seq_len[3] = 40, -1, -2
    st.ref[st.table[2, 0]] = 0
    st.upload()
    assert st.reserve([1, 1, 1, 1, 0, 0]) == {"PAGE", "REF", "LENGTH"}
    assert st.release(np.array([0, -1, 0, 0, -1, -1])) == {"PAGE", "REF", "LENGTH"}
    # the error word is the latest call's
    assert st.reserve([0] * 6) == set()


def test_reserve_refuses_as_a_whole():
    st = State(3, 50, 10, 4)
    assert st.reserve([30, 30, 1]) == {"POOL"}
    assert st.reserve([36, 0, 4]) == set()
    assert st.reserve([0, 1, 0]) == {"POOL"}


def test_exactly_the_last_page_and_pools_wider_than_a_scan_step():
    for pages in (1, 31, 32, 33, 16384, 16385, 40000):
        st = State(2, pages, pages, 1, layers=1)
        assert st.reserve([pages, 0]) == set()
        assert st.reserve([0, 1]) == {"POOL"}


def test_compact_with_stray_entries():
    st = State(4, 3, 20, 2, layers=3, width=72)
    st.ref[[3, 19, 12, 7]] = [1, 2, 1, 1]
    st.table[0], st.table[1], st.table[2] = [19, 3, -1], [19, 12, 7], [15, 25, -7]   # 15 is free, 25 no page
    st.upload()
    assert st.compact() == {"PAGE"}
    assert sorted(np.nonzero(st.ref)[0].tolist()) == [0, 1, 2, 3]
    st.table[2] = -1
    st.upload()
    assert st.compact() == set()


def test_round_on_another_stream_and_captured():
    """Release, fork and reserve in a captured graph on a side stream, replayed."""
    B, ps = 8, 4
    st = State(B, 12, 120, ps, layers=2, width=264, seed=5)
    roots = np.array([0, 0, 0, 0, 0, 0, 1, 1])
    st.reserve(roots * 10)
    st.grow(roots * 10)
    drop = np.array([0] * 6 + [-1, -1])
    src, dst, need = [6, 6, 6, 7, 7, 7], [0, 1, 2, 3, 4, 5], [5] * B
    d = [dev(x) for x in (drop, np.array(src), np.array(dst), np.array(need))]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())

    def calls():
        sv.spec_kv_release(d[0], st.d_len, st.d_table, st.d_ref, ps, workspace=st.ws, stream=stream)
        sv.spec_kv_fork(d[1], d[2], st.d_len, st.d_table, st.d_ref, ps, workspace=st.ws, stream=stream)
        sv.spec_kv_reserve(d[3], st.d_len, st.d_table, st.d_ref, st.d_pool, workspace=st.ws, stream=stream)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        calls()
        with torch.cuda.graph(graph, stream=stream):
            calls()
        graph.replay()
    stream.synchronize()
    for _ in range(2):
        kv_pages.release(drop, st.seq_len, st.table, st.ref, ps)
        kv_pages.fork(np.array(src), np.array(dst), st.seq_len, st.table, st.ref, ps)
        assert not kv_pages.reserve(np.array(need), st.seq_len, st.table, st.ref, st.pool, ps)
    st.check(set())


# ---------------------------------------------------------------- tree path
def path_case(B, N, ps, layers, width, seed, cols=40):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, cols * ps - N + 1, B).astype(np.int32)
    table = rng.permutation(B * cols).reshape(B, cols).astype(np.int32)
    n = rng.integers(-1, min(N, 6), B).astype(np.int32)
    n[0] = N - 1                                     # the whole tree is one path
    path = np.full((B, N), -1, dtype=np.int32)
    for b in range(B):
        if n[b] > 0:
            path[b, :n[b]] = np.sort(rng.permutation(N - 1)[:n[b]] + 1)
    pool = rng.integers(-30000, 30000, (layers, B * cols, ps, width)).astype(np.int16)
    staged = rng.integers(-30000, 30000, (layers, B, N, width)).astype(np.int16)
    return lens, table, n, path, pool, staged


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,N,ps,layers,width", [(1, 1, 1, 1, 8), (3, 16, 7, 2, 264), (9, 40, 16, 5, 2048),
                                                 (2, 256, 8, 3, 72), (700, 4, 2, 1, 16)])
def test_path_commit(B, N, ps, layers, width, in_place):
    cols = -(-N // ps) + 5
    lens, table, n, path, pool, staged = path_case(B, N, ps, layers, width, seed=B + N, cols=cols)
    d_len, d_pool = dev(lens), torch.from_numpy(pool.copy()).cuda()
    st = None if in_place else staged
    ws = sv.kv_path_workspace(B)
    for call in range(2):                            # the second call on the advanced lengths
        errors = kv_pages.commit_path(n, path, lens, table, pool, st, ps)
        sv.spec_kv_commit_path(dev(n), dev(path), d_len, dev(table), d_pool,
                               None if in_place else torch.from_numpy(staged).cuda(), workspace=ws)
        assert sv.kv_pages_read_error(ws) == word(errors)
        assert np.array_equal(d_len.cpu().numpy(), lens)
        assert np.array_equal(d_pool.cpu().numpy(), pool)


def test_path_commit_refusals():
    lens, table, n, path, pool, staged = path_case(8, 6, 4, 2, 16, seed=2, cols=6)
    n[:] = 2
    path[:, :2] = [2, 4]
    path[1, 1] = 2            # not ascending
    path[2, 0] = 0            # the root again
    path[3, 1] = 6            # no such node
    n[4] = 6                  # longer than the tree allows
    lens[5] = -1
    lens[6] = 6 * 4 - 2       # runs past the table
    table[7] = 999
    for st in (staged, None):
        d_len, d_pool = dev(lens), torch.from_numpy(pool.copy()).cuda()
        want_len, want_pool = lens.copy(), pool.copy()
        errors = kv_pages.commit_path(n, path, want_len, table, want_pool, st, 4)
        assert errors == {"PATH", "LENGTH", "CAPACITY", "PAGE"}
        ws = sv.spec_kv_commit_path(dev(n), dev(path), d_len, dev(table), d_pool,
                                    None if st is None else torch.from_numpy(staged).cuda())
        assert sv.kv_pages_read_error(ws) == word(errors)
        assert np.array_equal(d_len.cpu().numpy(), want_len)
        assert np.array_equal(d_pool.cpu().numpy(), want_pool)


def test_compact_reports_entries_of_free_pages_on_either_side():
    """An entry that names a free page stays as it is and is reported, whether the page lies behind the live ones or is
    one of the holes that are filled; entries of live pages, moved or not, are not."""
    for stray, flagged in ((15, True), (25, True), (1, True), (0, True), (2, True), (3, False), (19, False), (-1, False)):
        st = State(3, 3, 20, 2, layers=2, width=72, seed=stray + 1)
        st.ref[[3, 19, 12, 7]] = [2, 2, 1, 1]
        st.table[0], st.table[1], st.table[2] = [19, 3, -1], [19, 12, 7], [-1, stray, -1]
        st.upload()
        assert st.compact() == ({"PAGE"} if flagged else set())
        if flagged:
            assert int(st.d_table[2, 1]) == stray


def test_reserve_where_a_sequence_holds_a_page_twice():
    """Columns of one sequence that share a page are told apart like those of two: the last one that is written keeps it."""
    st = State(3, 4, 20, 4, layers=2, width=72, seed=3)
    st.table[0, :3], st.ref[5], st.ref[6] = [5, 5, 6], 2, 1
    st.seq_len[0] = 2
    st.upload()
    assert st.reserve([9, 0, 0]) == set()
    assert st.table[0, :3].tolist() == [0, 5, 6]
    st = State(3, 4, 20, 4, layers=2, width=72, seed=4)
    st.table[0, :3], st.table[1, :2], st.table[2, :2] = [5, 5, 5], [5, 7], [7, 7]
    st.ref[[5, 7]] = [4, 3]
    st.seq_len[:] = [3, 1, 2]
    st.upload()
    assert st.reserve([5, 7, 6]) == set()                # sequence 0 leaves its third column
    assert st.table.tolist() == [[0, 1, 5, -1], [2, 3, -1, -1], [4, 7, -1, -1]]
    st = State(2, 6, 20, 2, seed=5)
    st.table[0, :6], st.table[1, :2] = [3, 9, 3, 9, 9, 3], [9, 9]
    st.ref[[3, 9]] = [3, 5]
    st.seq_len[:] = [1, 0]
    st.upload()
    assert st.reserve([11, 4]) == set()
