"""Attention over the paged cache and over packed prompts on the GPU against
the fp64 definition (oracle/attention.py).

Tolerance, per element, from the arithmetic of include/spec_attention.h.  With
u = eps/2 of the type (half a step, relative) and f = 2^-24 (f32):
  * a score s = scale * q.k accumulates at most D + 2 f32 roundings of terms
    whose magnitudes sum to at most `reach`: |ds| <= (D + 2) f reach; its exponent
    (s - m) log2 e is one more rounding of a value of at most 2 reach log2 e:
    in all |ds| <= (D + 8) f reach on the score's own scale;
  * exp2 is good to 2^-22 relative, rescalings by exp(m_old - m_new) and the
    sums add less than 2^-17 in all for up to 2^7 blocks' partial results, and
    the f32 sums over n keys at most n f;
  * each weight is rounded to the type for the product: u;
  * the result is rounded once: u |out|.
A relative error e of every weight moves sum w v / sum w by at most 2 e sum w|v| /
sum w = 2 e weight, the rounding of the weights (numerator only) by u weight.
So |d out| <= u |out| + (u + 2 ((D + 8) f reach + n f + 2^-17)) weight, and
|d lse| <= (D + 8) f reach + n f + 2^-17 + 2 f |lse|.  A subnormal fp16 weight
(below 2^-14) is rounded by at most 2^-25 absolutely instead: the sum over n
keys adds n 2^-25 max|v|."""
import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_67_gb300 as sv
from oracle import attention

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def limits(out, lse, weight, reach, n, D, dtype, vmax):
    u, f = torch.finfo(dtype).eps / 2, 2.0 ** -24
    rel = (D + 8) * f * reach + n * f + 2.0 ** -17
    tiny = n * 2.0 ** -25 * vmax if dtype == torch.float16 else 0.0
    least = torch.finfo(dtype).tiny * u              # results below the normal range
    return (u * np.abs(out) + (u + 2 * rel[..., None]) * weight + tiny + least,
            rel + 2 * f * np.where(np.isfinite(lse), np.abs(lse), 0))


def check(got, got_lse, want, D, dtype, keys, vmax):
    out, lse, weight, reach = want
    a, b = limits(out, lse, weight, reach, keys, D, dtype, vmax)
    got = got.double().cpu().numpy()
    far = np.abs(got - out) - a
    assert np.isfinite(got).all()
    assert (far <= 0).all(), (far.max(), np.unravel_index(far.argmax(), far.shape))
    if got_lse is not None:
        got_lse = got_lse.double().cpu().numpy()
        assert np.array_equal(np.isinf(got_lse), np.isinf(lse))
        ok = np.isfinite(lse)
        assert (np.abs(got_lse - lse)[ok] <= b[ok]).all()


def np64(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------- paged cache
class Cache:
    def __init__(self, lens, S, heads, kv_heads, D, dtype, page, staged, seed=0, spare=3, scale=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        B, self.S, self.D, self.page, self.dtype = len(lens), S, D, page, dtype
        held = [-(-(n + S) // page) for n in lens]
        pages = sum(held) + spare
        entry = 2 * kv_heads * D
        rand = lambda *s: (torch.randn(s, generator=g, device="cuda") * scale).to(dtype)  # noqa: E731
        self.q, self.pool = rand(B, S, heads, D), rand(pages, page, entry)
        self.staged = rand(B, S, entry) if staged else None
        table = np.full((B, max(held) + 1), -1, dtype=np.int32)
        perm = rng.permutation(pages)
        at = 0
        for b, n in enumerate(held):
            table[b, :n] = perm[at:at + n]
            at += n
        self.table, self.seq_len = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
        self.lens, self.kv_heads, self.heads = list(lens), kv_heads, heads

    def entries(self, b, S=None):
        """[L + S][entry] in fp64, as the operator is to see them."""
        S, L, table = self.S if S is None else S, self.lens[b], self.table[b].cpu().numpy()
        n = L if self.staged is not None else L + S
        flat = [int(table[p // self.page]) * self.page + p % self.page for p in range(n)]
        rows = self.pool.view(-1, self.pool.shape[-1])[torch.tensor(flat, dtype=torch.int64, device="cuda")]
        if self.staged is not None:
            rows = torch.cat([rows, self.staged[b, :S]])
        return np64(rows)

    def want(self, b, parents=None, S=None, scale=None):
        S, L, D = self.S if S is None else S, self.lens[b], self.D
        kv = self.entries(b, S)
        among = np.tril(np.ones((S, S), bool)) if parents is None else attention.ancestors(parents[:S])
        see = np.concatenate([np.ones((S, L), bool), among], 1)
        w = self.kv_heads * D
        return attention.rows(np64(self.q[b, :S]), kv[:, :w].reshape(-1, self.kv_heads, D),
                              kv[:, w:].reshape(-1, self.kv_heads, D), see, scale or 1 / math.sqrt(D))

    def run(self, **kw):
        out = torch.full_like(self.q, 7.0)
        lse = torch.full(self.q.shape[:3], 7.0, device="cuda")
        ws = kw.pop("workspace", None)
        if ws is None:
            ws = sv.kv_attention_workspace(self.q, self.pool)
        got = sv.spec_kv_attention(kw.pop("q", self.q), self.pool, self.table, self.seq_len, self.staged, out=out,
                                   out_lse=lse, workspace=ws, **kw)
        assert got is out
        return out, lse, sv.attention_read_error(ws)

    def vmax(self):
        return max(float(x.abs().nan_to_num(0, 0, 0).max()) for x in (self.pool, self.staged) if x is not None)

    def check(self, parents=None, **kw):
        out, lse, err = self.run(parents=None if parents is None else
                                 torch.tensor([parents] * len(self.lens), dtype=torch.int32).cuda(), **kw)
        assert err == 0
        for b in range(len(self.lens)):
            check(out[b], lse[b], self.want(b, parents, scale=kw.get("scale")), self.D, self.dtype,
                  self.lens[b] + self.S, self.vmax())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("staged", [False, True])
@pytest.mark.parametrize("page", [1, 7, 16, 128, 300])
@pytest.mark.parametrize("D,heads,kv_heads", [(64, 3, 1), (128, 8, 2), (128, 7, 1), (64, 8, 8)])
def test_one_token(dtype, staged, page, D, heads, kv_heads):
    c = Cache([0, 1, 127, 128, 129, 255, 256, 700], 1, heads, kv_heads, D, DTYPES[dtype], page, staged, seed=page + D)
    c.check()


@pytest.mark.parametrize("staged", [False, True])
@pytest.mark.parametrize("S", [2, 5, 9, 33])
@pytest.mark.parametrize("D,heads,kv_heads,dtype", [(128, 8, 2, "bf16"), (64, 6, 2, "fp16"), (128, 64, 1, "bf16")])
def test_chain(staged, S, D, heads, kv_heads, dtype):
    c = Cache([0, 3, 125, 300], S, heads, kv_heads, D, DTYPES[dtype], 16, staged, seed=S)
    c.check()


TREES = {"bush": [-1, 0, 0, 0, 1, 1, 2, 3, 4, 7], "star": [-1] + [0] * 20, "line": list(range(-1, 39)),
         "wide": [-1] + [i // 3 for i in range(69)]}


@pytest.mark.parametrize("staged", [False, True])
@pytest.mark.parametrize("tree", sorted(TREES))
@pytest.mark.parametrize("D,heads,kv_heads,dtype", [(128, 4, 1, "bf16"), (64, 3, 3, "fp16")])
def test_tree(staged, tree, D, heads, kv_heads, dtype):
    p = TREES[tree]
    c = Cache([0, 50, 120, 257], len(p), heads, kv_heads, D, DTYPES[dtype], 24, staged, seed=len(p))
    c.check(parents=p)


@pytest.mark.parametrize("staged", [False, True])
def test_largest_tree_and_group(staged):
    rng = np.random.default_rng(0)
    p = [-1] + [int(rng.integers(0, i)) for i in range(1, 256)]
    Cache([200], 256, 4, 2, 64, torch.bfloat16, 16, staged, seed=1).check(parents=p)
    Cache([90, 0], 3, 64, 1, 64, torch.float16, 16, staged, seed=2).check()


@pytest.mark.parametrize("B,L", [(1, 5000), (3, 2999), (40, 300)])
def test_lengths_split_over_the_grid(B, L):
    """Caches longer than a CTA's share, ragged."""
    Cache([max(0, L - 37 * b) for b in range(B)], 1, 4, 2, 128, torch.bfloat16, 16, False, seed=B).check()


def test_ragged_rows_and_rows_left_alone():
    c = Cache([40, 300, 17, 0], 5, 4, 2, 64, torch.bfloat16, 16, True, seed=4)
    n = [5, 2, 0, 1]
    out, lse, err = c.run(q_len=torch.tensor(n, dtype=torch.int32).cuda())
    assert err == 0
    for b, k in enumerate(n):
        if k:
            check(out[b, :k], lse[b, :k], c.want(b, S=k), c.D, c.dtype, c.lens[b] + k, c.vmax())
        assert (out[b, k:] == 7).all() and (lse[b, k:] == 7).all()


def test_strided_queries_scale_and_defaults():
    c = Cache([33, 260], 3, 4, 2, 64, torch.float16, 8, False, seed=6)
    wide = torch.randn((2, 3, 4 + 4, 64), device="cuda").half()
    c.q = wide[:, :, :4]
    out, lse, err = c.run(scale=0.3)
    assert err == 0
    for b in range(2):
        check(out[b], lse[b], c.want(b, scale=0.3), c.D, c.dtype, c.lens[b] + 3, c.vmax())
    alone = sv.spec_kv_attention(c.q, c.pool, c.table, c.seq_len, scale=0.3)
    assert torch.equal(alone, out)


@pytest.mark.parametrize("staged", [False, True])
def test_garbage_that_nobody_sees(staged):
    """NaN and infinity behind the lengths, in unused pages, and in the entries of nodes that are not ancestors."""
    for parents in (None, [-1, 0, 0, 1]):
        c = Cache([5, 130, 64], 4, 4, 2, 64, torch.bfloat16, 16, staged, seed=9)
        seen = torch.zeros(c.pool.shape[:2], dtype=torch.bool, device="cuda")
        for b, L in enumerate(c.lens):
            for p in range(L + (0 if staged else 4)):
                seen[int(c.table[b, p // 16]), p % 16] = True
        bad = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda").bfloat16()
        c.pool[~seen] = bad[torch.arange(c.pool.shape[2], device="cuda") % 3]
        # new entry 3 is seen by row 3 alone (chain), and not by rows 0..2 (tree): spoil it
        for b, L in enumerate(c.lens):
            if staged:
                c.staged[b, 3] = float("nan")
            else:
                c.pool[int(c.table[b, (L + 3) // 16]), (L + 3) % 16] = float("nan")
        p = None if parents is None else torch.tensor([parents] * 3, dtype=torch.int32).cuda()
        out, lse, err = c.run(parents=p)
        assert err == 0
        for b in range(3):
            want = c.want(b, parents)
            check(out[b, :3], lse[b, :3], [x[:3] for x in want], 64, c.dtype, c.lens[b] + 4, c.vmax())
            assert out[b, 3].isnan().all() and lse[b, 3].isnan().all()


def test_infinite_values_that_are_seen():
    """A value of +inf reaches exactly the rows and columns that see it; a key of -inf score weighs nothing."""
    c = Cache([20, 200], 3, 2, 1, 64, torch.bfloat16, 16, False, seed=12)
    b, L = 1, 200
    where = lambda p: (int(c.table[b, p // 16]), p % 16)  # noqa: E731
    c.pool[where(L + 1)][64 + 5] = float("inf")        # value column 5 of the second new token
    c.pool[where(7)][64 + 9] = -float("inf")           # value column 9 of a committed one
    out, lse, err = c.run()
    assert err == 0 and lse.isfinite().all()
    assert torch.isfinite(out[0]).all()
    o = out[1]
    assert torch.isfinite(o[0, :, 5]).all() and (o[1:, :, 5] == float("inf")).all()
    assert (o[:, :, 9] == -float("inf")).all()
    rest = [i for i in range(64) if i not in (5, 9)]
    assert torch.isfinite(o[:, :, rest]).all()
    for p in (L + 1, 7):                               # the finite columns are what they are without the infinities
        c.pool[where(p)][64:] = torch.where(c.pool[where(p)][64:].isinf(), torch.zeros_like(c.pool[where(p)][64:]),
                                            c.pool[where(p)][64:])
    want = c.want(1)
    check(o[:, :, rest], lse[1], [want[0][..., rest], want[1], want[2][..., rest], want[3]], 64, c.dtype, 203,
          c.vmax())


def test_far_scores():
    """Scores of several hundreds: weights of one key or of exact ties."""
    Cache([300, 129], 2, 4, 2, 128, torch.bfloat16, 16, False, seed=3, scale=6.0).check()
    c = Cache([256], 1, 2, 1, 64, torch.float16, 16, False, seed=3)
    c.pool[..., :64] = c.pool[:1, :1, :64]              # every key the same: the mean of the values
    c.check()


def test_bad_sequences_are_flagged_and_zero():
    c = Cache([50, 60, 70, 80, 90, 20], 3, 4, 2, 64, torch.bfloat16, 16, False, seed=5)
    c.seq_len[0] = -1
    c.seq_len[1] = c.table.shape[1] * 16 - 1
    c.table[2, 1] = 10 ** 6
    c.table[3, 0] = -1
    q_len = torch.tensor([3, 3, 3, 3, 4, 3], dtype=torch.int32).cuda()
    out, lse, err = c.run(q_len=q_len)
    assert err == sv.ATTN_DEVERR_LENGTH | sv.ATTN_DEVERR_CAPACITY | sv.ATTN_DEVERR_PAGE
    assert not out[:5].any() and (lse[:5] == -float("inf")).all()
    check(out[5], lse[5], c.want(5), 64, c.dtype, 23, c.vmax())
    parents = torch.tensor([[-1, 0, 0], [0, 0, 0], [-1, 1, 0], [-1, 0, -1], [-1, 0, 2], [-1, 0, 1]],
                           dtype=torch.int32).cuda()
    c = Cache([50, 60, 70, 80, 90, 20], 3, 4, 2, 64, torch.bfloat16, 16, True, seed=5)
    ws = sv.kv_attention_workspace(c.q, c.pool)
    out, lse, err = c.run(parents=parents, workspace=ws)
    assert err == sv.ATTN_DEVERR_TREE
    assert not out[1:5].any()
    for b in (0, 5):
        check(out[b], lse[b], c.want(b, parents[b].tolist()), 64, c.dtype, 93, c.vmax())
    out, lse, err = c.run(workspace=ws)                 # the error word is the latest call's
    assert err == 0


def test_equal_calls_give_equal_bits_and_graphs_replay():
    c = Cache([1000, 3, 511], 4, 8, 2, 128, torch.bfloat16, 16, False, seed=8)
    ws = sv.kv_attention_workspace(c.q, c.pool)
    first, lse, _ = c.run(workspace=ws)
    again, lse2, _ = c.run(workspace=ws)
    assert torch.equal(first, again) and torch.equal(lse, lse2)
    out = torch.empty_like(first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        sv.spec_kv_attention(c.q, c.pool, c.table, c.seq_len, out=out, workspace=ws)
    c.q.copy_(torch.randn_like(c.q, dtype=torch.float32))
    c.seq_len.copy_(torch.tensor([400, 0, 500], dtype=torch.int32))
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    c.lens = [400, 0, 500]
    fresh, lse, _ = c.run()
    assert torch.equal(out, fresh)
    for b in range(3):
        check(out[b], None, c.want(b), 128, c.dtype, c.lens[b] + 4, c.vmax())


def test_own_stream_without_a_workspace():
    c = Cache([900, 40], 2, 8, 2, 64, torch.float16, 16, True, seed=10)
    want, _, _ = c.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [sv.spec_kv_attention(c.q, c.pool, c.table, c.seq_len, c.staged, stream=s) for _ in range(3)]
    s.synchronize()
    assert all(torch.equal(g, want) for g in got)


# ----------------------------------------------------------------- prompts
def prompts(lens, extra, heads, kv_heads, D, dtype, seed=0, strided=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    keys = [n + e for n, e in zip(lens, extra)]
    rand = lambda n, h: torch.randn((n, h, D), generator=g, device="cuda").to(dtype)  # noqa: E731
    if strided:       # one fused projection of queries, keys and values
        qkv = rand(sum(lens), heads + 2 * kv_heads)
        q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:]
    else:
        q, k, v = rand(sum(lens), heads), rand(sum(keys), kv_heads), rand(sum(keys), kv_heads)
    cu = lambda x: torch.tensor([0] + list(np.cumsum(x)), dtype=torch.int32).cuda()  # noqa: E731
    return q, k, v, cu(lens), cu(keys)


def check_prompts(q, k, v, cu_q, cu_k, out, lse, dtype, rows=None, scale=None):
    cq, ck, D = cu_q.tolist(), cu_k.tolist(), q.shape[2]
    for b in range(len(cq) - 1):
        n, m = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
        see = attention.chain_mask(n, m)
        at = np.arange(n) if rows is None else np.unique(np.clip(rows, 0, n - 1)) if n else np.arange(0)
        if n == 0:
            continue
        sl, kl = slice(cq[b], cq[b + 1]), slice(ck[b], ck[b + 1])
        want = attention.rows(np64(q[sl])[at], np64(k[kl]), np64(v[kl]), see[at], scale or 1 / math.sqrt(D))
        check(out[sl][torch.from_numpy(at).cuda()], None if lse is None else lse[sl][torch.from_numpy(at).cuda()], want,
              D, dtype, m, float(v.abs().nan_to_num(0, 0, 0).max()))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D,heads,kv_heads", [(64, 2, 2), (128, 4, 1), (128, 3, 1), (64, 14, 2)])
def test_packed_prompts(dtype, D, heads, kv_heads):
    lens = [1, 0, 5, 127, 128, 129, 64, 300, 2]
    q, k, v, cq, ck = prompts(lens, [0] * 9, heads, kv_heads, D, DTYPES[dtype], seed=D + heads)
    lse = torch.empty(q.shape[:2], device="cuda")
    ws = sv.prompt_attention_workspace(q, k, len(lens))
    out = sv.spec_prompt_attention(q, k, v, cq, out_lse=lse, workspace=ws)
    assert sv.attention_read_error(ws) == 0
    check_prompts(q, k, v, cq, ck, out, lse, DTYPES[dtype])


@pytest.mark.parametrize("strided", [False, True])
def test_long_prompts_sampled_rows(strided):
    lens = [1500, 700, 33]
    q, k, v, cq, ck = prompts(lens, [0] * 3, 8, 2, 128, torch.bfloat16, seed=1, strided=strided)
    out = sv.spec_prompt_attention(q, k, v, cq)
    check_prompts(q, k, v, cq, ck, out, None, torch.bfloat16,
                  rows=np.array([0, 1, 31, 32, 63, 64, 127, 128, 255, 256, 600, 699, 1023, 1024, 1498, 1499]))


def test_pieces_of_prompts_and_rows_without_a_key():
    lens, extra = [40, 1, 130, 9, 5, 3], [100, 513, 7, -4, -5, -3]   # the last three have fewer keys than queries
    q, k, v, cq, ck = prompts(lens, extra, 4, 2, 64, torch.float16, seed=2)
    lse = torch.empty(q.shape[:2], device="cuda")
    out = sv.spec_prompt_attention(q, k, v, cq, ck, out_lse=lse, scale=0.2)
    check_prompts(q, k, v, cq, ck, out, lse, torch.float16, scale=0.2)
    assert not out[cq[3]:cq[3] + 4].any() and (lse[cq[3]:cq[3] + 4] == -float("inf")).all()
    assert out[cq[3] + 4:cq[4]].any()


def test_rows_of_no_sequence_and_bad_offsets():
    q, k, v, _, _ = prompts([300], [0], 4, 2, 64, torch.bfloat16, seed=3)
    cq = torch.tensor([10, 100, 90, 200, 260, 301], dtype=torch.int32).cuda()
    out = torch.full_like(q, 7.0)
    ws = sv.prompt_attention_workspace(q, k, 5)
    sv.spec_prompt_attention(q, k, v, cq, out=out, workspace=ws)
    assert sv.attention_read_error(ws) == sv.ATTN_DEVERR_LENGTH
    assert (out[:10] == 7).all() and (out[260:] == 7).all()
    for a, z in ((10, 100), (90, 200), (200, 260)):
        good = torch.tensor([0, z - a], dtype=torch.int32).cuda()
        alone = sv.spec_prompt_attention(q[a:z], k[a:z], v[a:z], good)
        sure = slice(0, z - a) if a != 10 else slice(0, 80)
        sure = slice(10, z - a) if a == 90 else sure
        check_prompts(q[a:z], k[a:z], v[a:z], good, good, alone, None, torch.bfloat16)
        assert torch.allclose(out[a:z][sure].float(), alone[sure].float(), atol=0.02)
    sv.spec_prompt_attention(q, k, v, torch.tensor([0, 300], dtype=torch.int32).cuda(), out=out, workspace=ws)
    assert sv.attention_read_error(ws) == 0
    sv.spec_prompt_attention(q, k, v, torch.tensor([-1, 300], dtype=torch.int32).cuda(), workspace=ws)
    assert sv.attention_read_error(ws) == sv.ATTN_DEVERR_LENGTH


def test_prompt_garbage_stays_where_it_is():
    """NaN in a later token, in the neighbours in the pack, and behind the last sequence."""
    lens = [70, 200, 64]
    q, k, v, cq, ck = prompts(lens + [20], [0] * 4, 4, 2, 64, torch.bfloat16, seed=4)
    cq, ck = cq[:4].contiguous(), ck[:4].contiguous()
    bad = slice(int(cq[1]) + 150, int(cq[1]) + 155)     # tokens 150..154 of the second prompt
    k[bad], v[bad] = float("nan"), float("inf")
    k[int(cq[3]):], v[int(cq[3]):] = float("nan"), float("nan")
    out = sv.spec_prompt_attention(q, k, v, cq, out=torch.zeros_like(q))
    for b, rows in ((0, 70), (1, 150), (2, 64)):
        a, z = int(cq[b]), int(cq[b]) + rows
        c = torch.tensor([0, rows], dtype=torch.int32).cuda()
        check_prompts(q[a:z], k[a:z], v[a:z], c, c, out[a:z], None, torch.bfloat16)
    a = int(cq[1])
    assert out[a + 150:a + 200].isnan().all()
    v[bad] = float("nan")
    k[bad] = 0.5                                          # finite scores, values not a number
    out = sv.spec_prompt_attention(q, k, v, cq, out=torch.zeros_like(q))
    assert torch.isfinite(out[a:a + 150]).all() and out[a + 150:a + 200].isnan().all()
    assert torch.isfinite(out[a + 200:int(cq[3])]).all()


def test_prompt_infinite_value_column():
    q, k, v, cq, ck = prompts([300], [0], 4, 1, 64, torch.float16, seed=7)
    v[140, 0, 3] = float("inf")
    out = sv.spec_prompt_attention(q, k, v, cq)
    assert torch.isfinite(out[:140]).all() and (out[140:, :, 3] == float("inf")).all()
    assert torch.isfinite(out[:, :, :3]).all() and torch.isfinite(out[:, :, 4:]).all()


def test_prompt_graph_and_equal_bits():
    q, k, v, cq, _ = prompts([513, 100, 7], [0] * 3, 8, 4, 128, torch.bfloat16, seed=5)
    ws = sv.prompt_attention_workspace(q, k, 3)
    first = sv.spec_prompt_attention(q, k, v, cq, workspace=ws)
    out = torch.empty_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.spec_prompt_attention(q, k, v, cq, out=out, workspace=ws)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)


def test_more_sequences_than_a_block_has_threads():
    lens = [(i * 7) % 5 for i in range(3000)]
    q, k, v, cq, ck = prompts(lens, [0] * 3000, 2, 1, 64, torch.bfloat16, seed=6)
    out = sv.spec_prompt_attention(q, k, v, cq)
    check_prompts(q, k, v, cq, ck, out, None, torch.bfloat16)
    c = Cache([i % 9 for i in range(2000)], 1, 2, 1, 64, torch.bfloat16, 4, True, seed=1)
    c.check()


def test_as_many_sequences_as_a_call_takes():
    """65535 sequences of one key or none: weight 1, so a row is its value, bit for bit."""
    B = 65535
    lens = (torch.arange(B) % 3 != 1).int()
    cu = torch.cat([torch.zeros(1, dtype=torch.int32), lens.cumsum(0).int()]).cuda()
    n = int(cu[-1])
    q, v = (torch.randn((n, h, 64), device="cuda").bfloat16() for h in (2, 1))
    assert torch.equal(sv.spec_prompt_attention(q, v, v, cu), v.expand(n, 2, 64))
    entry = torch.randn((B, 1, 128), device="cuda").bfloat16()
    pool = torch.randn((2, 4, 128), device="cuda").bfloat16()
    table = torch.zeros((B, 1), dtype=torch.int32, device="cuda")
    qc = torch.randn((B, 1, 2, 64), device="cuda").bfloat16()
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    out = torch.full_like(qc, 7.0)
    sv.spec_kv_attention(qc, pool, table, zero, entry, q_len=lens.cuda(), out=out)
    want = torch.where(lens.cuda().bool()[:, None, None, None], entry[:, :, None, 64:].expand(B, 1, 2, 64),
                       torch.full_like(qc, 7.0))
    assert torch.equal(out, want)


# ---------------------------------------------------------------- together
def test_a_speculative_round_on_the_cache():
    """A prompt's attention and its entries, two continuations that share them, a tree round on either: the rows
    of the tree attention equal the prompt operator's on the same tokens written out, and after the commit of an
    accepted path a plain token reads the cache it left."""
    D, heads, kv_heads, ps, layers, P = 64, 4, 2, 8, 2, 45
    E = 2 * kv_heads * D
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    B, pages, parents = 3, 60, [-1, 0, 0, 1, 1, 2]
    N = len(parents)
    table = torch.full((B, 12), -1, dtype=torch.int32, device="cuda")
    ref = torch.zeros(pages, dtype=torch.int32, device="cuda")
    seq_len = torch.zeros(B, dtype=torch.int32, device="cuda")
    pool = rand(layers, pages, ps, E)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    # prompt: attention, then its entries into the cache of sequence 0
    q, kv = rand(P, heads, D), rand(layers, P, E)
    k, v = kv[1].view(P, 2, kv_heads, D)[:, 0], kv[1].view(P, 2, kv_heads, D)[:, 1]
    cu = i32(0, P)
    o = sv.spec_prompt_attention(q, k, v, cu)
    check_prompts(q, k, v, cu, cu, o, None, torch.bfloat16)
    ws = sv.kv_pages_workspace(table, ref)
    sv.spec_kv_reserve(i32(P, 0, 0), seq_len, table, ref, pool, workspace=ws)
    staged = torch.zeros((layers, B, P, E), dtype=pool.dtype, device="cuda")
    staged[:, 0] = kv
    sv.spec_kv_commit(i32(P - 1, -1, -1), seq_len, table, pool, staged)
    # two continuations of it
    sv.spec_kv_fork(i32(0, 0), i32(1, 2), seq_len, table, ref, ps, workspace=ws)
    sv.spec_kv_reserve(i32(N, N, N), seq_len, table, ref, pool, workspace=ws)
    assert sv.kv_pages_read_error(ws) == 0 and seq_len.tolist() == [P] * 3
    # the tree pass writes its entries in place (another tree for each sequence) and attends
    tree = rand(layers, B, N, E)
    for b in range(B):
        for i in range(N):
            pool[:, int(table[b, (P + i) // ps]), (P + i) % ps] = tree[:, b, i]
    tq = rand(B, N, heads, D)
    got = sv.spec_kv_attention(tq, pool[1], table, seq_len, parents=i32(*parents).repeat(B, 1))
    also = sv.spec_kv_attention(tq, pool[1], table, seq_len, tree[1].contiguous(),
                                parents=i32(*parents).repeat(B, 1))
    line = attention.ancestors(parents)
    for b in range(B):
        for i in range(N):
            on = np.nonzero(line[i])[0]
            keys = torch.cat([kv[1], tree[1, b, torch.from_numpy(on).cuda()]]).view(-1, 2, kv_heads, D)
            want = attention.rows(np64(tq[b, i:i + 1]), np64(keys[:, 0]), np64(keys[:, 1]),
                                  np.ones((1, len(keys)), bool), D ** -0.5)
            for x in (got, also):
                check(x[b, i:i + 1], None, want, D, torch.bfloat16, len(keys), float(pool.abs().max()))
    # accepted: 0-1-4 on sequence 0, nothing on 1, a flagged row on 2
    path = torch.full((B, N), -1, dtype=torch.int32, device="cuda")
    path[0, :2] = i32(1, 4)
    pws = sv.spec_kv_commit_path(i32(2, 0, -1), path, seq_len, table, pool)
    assert sv.kv_pages_read_error(pws) == 0 and seq_len.tolist() == [P + 3, P + 1, P]
    sv.spec_kv_release(None, seq_len, table, ref, ps, workspace=ws)
    sv.spec_kv_release(i32(-1, -1, 0), seq_len, table, ref, ps, workspace=ws)
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    sv.spec_kv_compact(table, ref, pool, out_num_live=live, workspace=ws)
    assert sv.kv_pages_read_error(ws) == 0 and int(live) == int((ref > 0).sum()) == int(table.max()) + 1
    # the next token of sequences 0 and 1
    sv.spec_kv_reserve(i32(1, 1, 0), seq_len, table, ref, pool, workspace=ws)
    new, nq = rand(B, 1, E), rand(B, 1, heads, D)
    got = sv.spec_kv_attention(nq, pool[1], table, seq_len, new, q_len=i32(1, 1, 0))
    for b, nodes in ((0, [0, 1, 4]), (1, [0])):
        keys = torch.cat([kv[1], tree[1, b, torch.tensor(nodes).cuda()], new[b]]).view(-1, 2, kv_heads, D)
        want = attention.rows(np64(nq[b]), np64(keys[:, 0]), np64(keys[:, 1]), np.ones((1, len(keys)), bool),
                              D ** -0.5)
        check(got[b], None, want, D, torch.bfloat16, len(keys), float(pool.abs().max()))


# --------------------------------------------------------------- the far ends
def test_nothing_to_do():
    c = Cache([40, 9], 3, 4, 2, 64, torch.bfloat16, 16, True, seed=2)
    out, lse, err = c.run(q_len=torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert err == 0 and (out == 7).all() and (lse == 7).all()
    q, k, v, _, _ = prompts([5], [0], 4, 2, 64, torch.float16)
    out = torch.full_like(q, 7.0)
    sv.spec_prompt_attention(q, k, v, torch.zeros(4, dtype=torch.int32, device="cuda"), out=out)
    assert (out == 7).all()


def test_pool_beyond_32_bits_of_bytes_and_elements():
    """Pages at the far end of a pool of 9.7 GB; pages named by two sequences, and twice by one."""
    kv_heads, D, page, entry = 8, 128, 16, 2048
    pages = 148000
    pool = torch.empty((pages, page, entry), dtype=torch.bfloat16, device="cuda")
    used = list(range(pages - 12, pages)) + [0, 1]
    pool[used] = torch.randn((len(used), page, entry), device="cuda").bfloat16()
    c = Cache([150, 150, 100], 2, 8, kv_heads, D, torch.bfloat16, page, False, seed=1)
    c.pool = pool
    table = torch.full((3, 11), -1, dtype=torch.int32)
    table[0, :10] = torch.tensor(used[:10])
    table[1, :10] = torch.tensor(used[:9] + [used[10]])
    table[2, :7] = torch.tensor([used[12], used[13], used[12], used[3], used[4], used[5], used[11]])
    c.table = table.cuda()
    out, lse, err = c.run()
    assert err == 0
    for b in range(3):
        check(out[b], lse[b], c.want(b), D, c.dtype, 152, 6.0)


def test_most_heads_and_single_token_strides():
    c = Cache([20, 150], 1, 1024, 1024, 64, torch.bfloat16, 16, True, seed=3)
    out, lse, err = c.run()
    assert err == 0
    for b in range(2):
        check(out[b], lse[b], c.want(b), 64, c.dtype, c.lens[b] + 1, c.vmax())
    c = Cache([20, 150, 3], 1, 4, 2, 128, torch.float16, 16, False, seed=4)
    wide = torch.randn((3, 1, 12, 128), device="cuda").half()
    c.q = wide[:, :, 4:8]
    out, lse, err = c.run()
    assert err == 0
    for b in range(3):
        check(out[b], lse[b], c.want(b), 128, c.dtype, c.lens[b] + 1, c.vmax())


def test_two_calls_at_once():
    """Calls on two streams, each with its own workspace, over and over."""
    a = Cache([700, 30], 1, 8, 2, 128, torch.bfloat16, 16, False, seed=5)
    q, k, v, cq, _ = prompts([300, 200], [0, 0], 8, 2, 128, torch.bfloat16, seed=6)
    want_a, _, _ = a.run()
    want_p = sv.spec_prompt_attention(q, k, v, cq)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    wa, wp = sv.kv_attention_workspace(a.q, a.pool), sv.prompt_attention_workspace(q, k, 2)
    torch.cuda.synchronize()
    got_a, got_p = [], []
    for _ in range(10):
        got_a.append(sv.spec_kv_attention(a.q, a.pool, a.table, a.seq_len, workspace=wa, stream=s1))
        got_p.append(sv.spec_prompt_attention(q, k, v, cq, workspace=wp, stream=s2))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want_a) for x in got_a) and all(torch.equal(x, want_p) for x in got_p)


def test_spoiled_first_blocks_and_many_spoiled_rows():
    """NaN and infinite values in the only block of an item, and in all of a block's later tokens."""
    q, k, v, cq, ck = prompts([100, 260], [0, 0], 2, 1, 128, torch.bfloat16, seed=8)
    v[20] = float("inf")
    v[100 + 130:] = float("nan")
    out = sv.spec_prompt_attention(q, k, v, cq)
    check_prompts(q[:20], k[:20], v[:20], cq[:2].clamp(max=20), cq[:2].clamp(max=20), out[:20], None, torch.bfloat16)
    assert (out[20:100] == float("inf")).all()
    assert torch.isfinite(out[100:230]).all() and out[230:].isnan().all()
    c = torch.tensor([0, 130], dtype=torch.int32, device="cuda")
    check_prompts(q[100:230], k[100:230], v[100:230], c, c, out[100:230], None, torch.bfloat16)


@pytest.mark.parametrize("staged", [False, True])
def test_rising_scores(staged):
    """Every block's scores far above the last one's, and far below: the reference moves, or stays."""
    for sign in (1.0, -1.0):
        c = Cache([1000], 2, 2, 1, 64, torch.bfloat16, 16, staged, seed=9)
        c.q[:] = 1.0
        ramp = torch.arange(1000, device="cuda") // 100 * sign * 0.5
        for p in range(1000):
            c.pool[int(c.table[0, p // 16]), p % 16, :64] += ramp[p].to(torch.bfloat16)
        c.check()
    for dtype in (torch.bfloat16, torch.float16):
        q, k, v, cq, ck = prompts([600], [0], 2, 2, 64, dtype, seed=10)
        q[:] = 1.0
        k += (torch.arange(600, device="cuda") // 60).to(dtype)[:, None, None]
        out = sv.spec_prompt_attention(q, k, v, cq)
        check_prompts(q, k, v, cq, ck, out, None, dtype, rows=np.arange(0, 600, 7))


@pytest.mark.parametrize("D,n", [(128, 400), (64, 1040)])
def test_hidden_values_after_an_item_with_one_row_tile(D, n):
    """The last item of a head has one row tile of 16 tokens and more blocks than the ring of K and V tiles holds (4 at
    128, 9 at 64); the next head's first item has two, and its first block is masked.  One infinite value in the upper
    half of the columns of an early key reaches the rows that see it and no other."""
    B, heads, kv_heads, key, column = 12, 32, 8, 40, D - 3
    q, k, v, cq, _ = prompts([n] * B, [0] * B, heads, kv_heads, D, torch.bfloat16, seed=21)
    v.view(B, n, kv_heads, D)[:, key, :, column] = float("inf")
    ws = sv.prompt_attention_workspace(q, k, B)
    out = sv.spec_prompt_attention(q, k, v, cq, workspace=ws)
    assert sv.attention_read_error(ws) == 0
    o = out.view(B, n, heads, D)
    assert torch.isfinite(o[:, :key]).all() and (o[:, key:, :, column] == float("inf")).all()
    assert torch.isfinite(o[..., [c for c in range(D) if c != column]]).all()
    for b in range(B):
        a = b * n
        c = torch.tensor([0, key], dtype=torch.int32).cuda()
        rows = slice(a, a + key)
        check_prompts(q[rows], k[rows], v[rows], c, c, out[rows], None, torch.bfloat16)
    for _ in range(5):
        assert torch.equal(sv.spec_prompt_attention(q, k, v, cq, workspace=ws), out)


@pytest.mark.parametrize("staged", [False, True])
@pytest.mark.parametrize("L,S", [(300, 1), (1000, 1), (1000, 5), (20000, 1), (20000, 5)])
def test_a_query_that_is_not_a_number_however_its_cache_is_cut(L, S, staged):
    """The heads that hold a NaN give NaN, with a few pieces to join and with many; the others what they give alone."""
    c = Cache([L], S, 4, 1, 64, torch.bfloat16, 16, staged, seed=L + S)
    c.q[0, S - 1, 1, 7] = float("nan")
    out, lse, err = c.run()
    assert err == 0
    assert out[0, S - 1, 1].isnan().all() and lse[0, S - 1, 1].isnan()
    sure = torch.ones((S, 4), dtype=torch.bool)
    sure[S - 1, 1] = False
    want = [x[sure.numpy()] for x in c.want(0)]
    check(out[0][sure.cuda()], lse[0][sure.cuda()], want, 64, c.dtype, L + S, c.vmax())


@pytest.mark.parametrize("L", [1000, 20000])
def test_keys_that_are_not_numbers_in_a_piece_of_their_own(L):
    """A staged NaN key is one token's last block; NaN keys may fill whole blocks: neither may drop out."""
    c = Cache([L], 1, 4, 2, 128, torch.float16, 16, True, seed=L)
    c.staged[0, 0, 3] = float("nan")                       # a key of the first head, seen by heads 0 and 1
    out, lse, err = c.run()
    assert err == 0 and out[0, 0, :2].isnan().all() and lse[0, 0, :2].isnan().all()
    want = [x[:, 2:] for x in c.want(0)]
    check(out[0, :, 2:], lse[0, :, 2:], want, 128, c.dtype, L + 1, float(c.pool.abs().max()))
    for first, n in ((384, 128), (0, 256), (L - 104, 104)):
        c = Cache([L], 1, 4, 2, 128, torch.float16, 16, False, seed=L)
        for p in range(first, first + n):
            c.pool[int(c.table[0, p // 16]), p % 16, 3] = float("nan")
        out, lse, err = c.run()
        assert err == 0 and out[0, 0, :2].isnan().all() and lse[0, 0, :2].isnan().all()
        assert out[0, 0, 2:].isfinite().all() and lse[0, 0, 2:].isfinite().all()


def test_a_prompt_row_that_is_not_a_number():
    q, k, v, cq, ck = prompts([3000, 500], [0, 0], 4, 2, 128, torch.bfloat16, seed=13)
    rows = [0, 5, 700, 1499, 2999, 3100]
    q[rows, 2, 1] = float("nan")
    lse = torch.empty(q.shape[:2], device="cuda")
    out = sv.spec_prompt_attention(q, k, v, cq, out_lse=lse)
    assert out[rows, 2].isnan().all() and lse[rows, 2].isnan().all()
    rest = torch.ones(q.shape[:2], dtype=torch.bool, device="cuda")
    rest[rows, 2] = False
    assert out[rest].isfinite().all() and lse[rest].isfinite().all()


@pytest.mark.parametrize("L", [300, 1000, 20000])
def test_an_infinite_value_of_a_key_far_below_the_others(L):
    """Its weight is positive by definition, so the result is not finite, whichever piece the key is in."""
    for p in (0, 130, 290):
        c = Cache([L], 1, 2, 1, 64, torch.bfloat16, 16, False, seed=L)
        c.q[:] = 1.0
        c.pool[..., :64] = 4.0
        where = (int(c.table[0, p // 16]), p % 16)
        c.pool[where][:64] = -60.0                          # (512 lower on the scores' scale)
        c.pool[where][64 + 5] = float("inf")
        out, lse, err = c.run()
        assert err == 0 and not out[..., 5].isfinite().any()
        assert out[..., :5].isfinite().all() and out[..., 6:].isfinite().all() and lse.isfinite().all()
    c = Cache([L], 1, 2, 1, 64, torch.bfloat16, 16, True, seed=L)   # a staged entry is a block of its own
    c.q[:] = 1.0
    c.pool[..., :64] = 4.0
    c.staged[0, 0, :64] = -60.0
    c.staged[0, 0, 64 + 5] = float("inf")
    out, lse, err = c.run()
    assert err == 0 and not out[..., 5].isfinite().any()
    assert out[..., :5].isfinite().all() and out[..., 6:].isfinite().all() and lse.isfinite().all()


def test_one_workspace_for_calls_of_different_batches():
    """A workspace serves calls of any batch it is large enough for, of either operator, one after the other: what one
    leaves in it marks no sequence of the next as bad."""
    few = Cache([40, 300, 17, 1000, 60, 7, 129, 500], 2, 4, 2, 64, torch.bfloat16, 16, False, seed=31)
    many = Cache([5 + b for b in range(200)], 2, 4, 2, 64, torch.bfloat16, 16, False, seed=32)
    q, k, v, cq, _ = prompts([300, 40, 129], [0] * 3, 4, 2, 64, torch.bfloat16, seed=33)
    want_few, want_many, want_prompts = few.run()[0], many.run()[0], sv.spec_prompt_attention(q, k, v, cq)
    ws = max((sv.kv_attention_workspace(many.q, many.pool), sv.prompt_attention_workspace(q, k, 3),
              sv.kv_attention_workspace(few.q, few.pool)), key=torch.numel)
    for _ in range(2):
        for b in (0, 199, 100):
            assert torch.equal(few.run(workspace=ws)[0], want_few)
            assert torch.equal(sv.spec_prompt_attention(q, k, v, cq, workspace=ws), want_prompts)
            was = int(many.seq_len[b])
            many.seq_len[b] = -1
            out, lse, err = many.run(workspace=ws)
            many.seq_len[b] = was
            assert err == sv.ATTN_DEVERR_LENGTH
            good = [i for i in range(200) if i != b]
            assert not out[b].any() and (lse[b] == -float("inf")).all()
            assert torch.equal(out[good], want_many[good])
            few.seq_len[3] = -1
            out, lse, err = few.run(workspace=ws)
            few.seq_len[3] = 1000
            good = [i for i in range(8) if i != 3]
            assert err == sv.ATTN_DEVERR_LENGTH and not out[3].any() and torch.equal(out[good], want_few[good])


@pytest.mark.parametrize("dtype,powers", [("fp16", [(7, 8), (11, 12), (14, 14), (15, 15)]),
                                          ("bf16", [(10, 10), (16, 16), (20, 30), (40, 45)])])
@pytest.mark.parametrize("scale", [0.3, 0.7])
def test_scores_beyond_24_bits(dtype, powers, scale):
    """Scores up to 2^84: the weights are one key's or those of exact ties, wherever the largest score stands, rising
    and falling, negative, and beside rows of small scores.  (Queries and keys of a few bits, so that products are exact
    in f32; those with the scale are not: by 2^-8 to 2^7 and more in the exponent of a weight.)  The weights that stay
    are equal, so a result is off by the rounding of the weights (u) and its own (u), and by the sums' and exponentials'
    share 2^-17 as above; half a step of 2^-24 for the score with its scale, for the sum with the logarithm and for their
    product is three for the log-sum-exp."""
    u = torch.finfo(DTYPES[dtype]).eps / 2
    g = np.random.default_rng(5)
    for a, b in powers:
        for kind in ("one", "ties", "up", "down", "negative"):
            n = 700
            m = {"one": np.full(n, 0.25), "ties": np.full(n, 0.25), "up": 0.25 * (1 + np.arange(n) // 200),
                 "down": 0.25 * (4 - np.arange(n) // 200), "negative": np.full(n, -1.0)}[kind]
            best = g.integers(0, n)
            m[best] = 1.0 if kind != "negative" else -0.25
            if kind == "ties":
                m[g.integers(0, n)] = 1.0
            c = Cache([n], 2, 4, 2, 64, DTYPES[dtype], 16, False, seed=a + b)
            c.q[:] = 0
            c.q[..., 0] = 1.171875 * 2.0 ** a
            c.q[:, :, 1] = c.q[:, :, 1] * 2.0 ** -a            # a row of small scores in the same warp
            flat = [int(c.table[0, p // 16]) * 16 + p % 16 for p in range(n)]
            keys = c.pool.view(-1, 256)
            keys[:, :128] = 0
            col = torch.from_numpy(m * 1.3046875 * 2.0 ** b).to(keys).cuda()
            keys[torch.tensor(flat).cuda(), 0] = col
            keys[torch.tensor(flat).cuda(), 64] = col
            q, k, v, cq, ck = prompts([n], [0], 4, 2, 64, DTYPES[dtype], seed=a)
            q[:], k[:] = 0, 0
            q[..., 0], k[:, :, 0] = 1.171875 * 2.0 ** a, col[:, None]
            q[:, 1] = q[:, 1] * 2.0 ** -a
            got, lse, err = c.run(scale=scale)
            assert err == 0
            lse_p = torch.empty(q.shape[:2], device="cuda")
            got_p = sv.spec_prompt_attention(q, k, v, cq, scale=scale, out_lse=lse_p)
            rows = np.array([0, 1, 127, 128, 250, 500, 699])
            want_p = attention.rows(np64(q)[rows], np64(k), np64(v), attention.chain_mask(n, n)[rows],
                                    float(np.float32(scale)))
            for x, y, w in ((got[0], lse[0], c.want(0, scale=float(np.float32(scale)))),
                            (got_p[rows], lse_p[rows], want_p)):
                x, y = np64(x), np64(y)
                assert np.isfinite(x).all() and np.isfinite(y).all(), (a, b, kind)
                far = np.abs(x - w[0]) - (u * np.abs(w[0]) + (u + 2.0 ** -17) * w[2] + 2.0 ** -25)
                assert (far <= 0).all(), (a, b, kind, far.max(), np.unravel_index(far.argmax(), far.shape))
                assert (np.abs(y - w[1]) <= 2.0 ** -16 + 3 * 2.0 ** -24 * np.abs(w[1])).all(), (a, b, kind)


def test_small_fp16_weights_beside_a_large_one():
    """One key far above thousands of others, whose weights of 1.5e-8 (2^-26) together are 1e-4 of the sum and whose
    values are 1 where that key's is 0.  Weights relative to the reference are rounded with 2^7 of room (at the reference
    itself 2^7 stands in fp16, and the row's sum is at least that): one below the normal range is off by at most 2^-25,
    2^-32 of the sum, instead of 2^-25."""
    n, B = 8000, 160
    c = Cache([n], 1, 2, 1, 64, torch.float16, 16, False, seed=41)
    c.q[:] = 0
    c.q[..., 0] = 4.5
    c.pool[..., :64] = 0
    c.pool[..., 64:] = 1
    c.pool[int(c.table[0, 0]), 0, 0] = 4.0                 # position 0: score 18, value 0
    c.pool[int(c.table[0, 0]), 0, 64:] = 0
    want = c.want(0, scale=1.0)
    assert 1e-4 < want[0].min() and want[0].max() < 1.4e-4
    out, lse, err = c.run(scale=1.0)                       # cut into pieces
    assert err == 0
    check(out[0], lse[0], want, 64, c.dtype, n + 1, 2.0 ** -7)
    q, table = c.q.expand(B, 1, 2, 64).contiguous(), c.table.expand(B, -1).contiguous()
    out = sv.spec_kv_attention(q, c.pool, table, c.seq_len.expand(B).contiguous(), scale=1.0)   # one piece each
    for b in (0, 77, B - 1):
        check(out[b], None, want, 64, c.dtype, n + 1, 2.0 ** -7)
    q, k, v, cq, ck = prompts([2000] * 6, [0] * 6, 16, 4, 64, torch.float16, seed=42)
    q[:], k[:], v[:] = 0, 0, 1
    q[..., 0] = 4.5
    k[::2000, :, 0], v[::2000] = 4.0, 0
    out = sv.spec_prompt_attention(q, k, v, cq, scale=1.0)
    for b in (0, 5):
        rows = [0, 1, 600, 1999]
        want = attention.rows(np64(q[2000 * b:2000 * b + 2000])[rows], np64(k[2000 * b:2000 * b + 2000]),
                              np64(v[2000 * b:2000 * b + 2000]), attention.chain_mask(2000, 2000)[rows], 1.0)
        check(out[2000 * b:2000 * b + 2000][rows], None, want, 64, torch.float16, 2000, 2.0 ** -7)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("fill", [float("nan"), float("inf"), 60000.0])
def test_queries_that_are_not_asked_for(dtype, fill):
    """Rows behind q_len, and rows of q that no sequence names, may hold anything: the others keep their bits."""
    for staged in (False, True):
        c = Cache([700, 40, 300], 9, 6, 2, 64, DTYPES[dtype], 16, staged, seed=51)
        n = torch.tensor([3, 9, 1], dtype=torch.int32).cuda()
        want, lse, _ = c.run(q_len=n)
        for b, k in enumerate(n.tolist()):
            c.q[b, k:] = fill
        got, lse2, err = c.run(q_len=n)
        assert err == 0 and torch.equal(got, want) and torch.equal(lse, lse2)
    q, k, v, _, _ = prompts([900], [0], 6, 2, 128, DTYPES[dtype], seed=52)
    cq = torch.tensor([5, 430, 430, 800], dtype=torch.int32).cuda()
    want = sv.spec_prompt_attention(q, k, v, cq)
    q[:5], q[800:] = fill, fill
    assert torch.equal(sv.spec_prompt_attention(q, k, v, cq), want)


@pytest.mark.parametrize("dtype,power", [("bf16", 20), ("bf16", 60), ("fp16", 15)])
def test_scores_beyond_24_bits_beside_values_that_are_not_finite(dtype, power):
    """Both slow ways in one block: rows that do not see the values are one key's value, to a rounding of the weight and
    of the result and 2^-17; rows that see one are not finite in its column only."""
    u, n, D = torch.finfo(DTYPES[dtype]).eps / 2, 300, 64
    m = np.where(np.arange(n) % 50 == 7, 0.25 + np.arange(n) / 512, 0.125) * 1.3046875   # a larger key every 50 tokens
    q, k, v, cq, _ = prompts([n], [0], 4, 2, D, DTYPES[dtype], seed=61)
    q[:], k[:] = 0, 0
    q[..., 0], k[:, :, 0] = 1.171875 * 2.0 ** power, torch.from_numpy(m * 2.0 ** power).to(k).cuda()[:, None]
    c = Cache([0], n - 100, 4, 2, D, DTYPES[dtype], 16, True, seed=62)                   # the same as new tokens
    c.q[0], c.staged[0, :, :2 * D], c.staged[0, :, 2 * D:] = (
        x[:n - 100].reshape(n - 100, *s) for x, s in ((q, (4, D)), (k, (-1,)), (v, (-1,))))
    clean = np64(v).copy()
    v[150, :, 3], v[290, :, 60] = float("inf"), float("nan")
    c.staged.view(1, n - 100, 2, 2, D)[0, 150, 1, :, 3] = float("inf")
    out = np64(sv.spec_prompt_attention(q, k, v, cq, scale=0.7))
    got, _, err = c.run(scale=0.7)
    assert err == 0
    want = attention.rows(np64(q), np64(k), clean, attention.chain_mask(n, n), float(np.float32(0.7)))
    for x, w in ((out, want), (np64(got[0]), [y[:n - 100] for y in want])):
        bad = np.zeros(x.shape, bool)
        bad[150:, :, 3] = True
        bad[290:, :, 60] = True
        assert np.array_equal(np.isfinite(x), ~bad)
        far = np.abs(x - w[0]) - (u * np.abs(w[0]) + (u + 2.0 ** -17) * w[2] + 2.0 ** -25)
        assert (far[~bad] <= 0).all()
