"""Host-side refusals of the attention, page and path entry points: returned
before any CUDA call, so these run without a GPU."""
import ctypes

import pytest
import torch

import speculative_decoding_verification_67_gb300 as sv
from speculative_decoding_verification_67_gb300 import _build

ARG, DIMS, ALIGN, WORKSPACE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return sv.library()


def at(addr):
    return ctypes.c_void_p(addr)


GOOD, NULL, OFF8, OFF2 = at(0x10000), at(None), at(0x10008), at(0x10002)
KV = dict(B=4, S=5, heads=8, kv_heads=2, head_dim=128, page_size=16, num_pages=100, max_pages=10, dtype=0,
          q_stride=1024)
PROMPT = dict(B=4, heads=8, kv_heads=2, head_dim=128, total_q=100, total_k=120, dtype=1, q_stride=1024, k_stride=256,
              v_stride=256)


def kv_dims(**kw):
    d = dict(KV, **kw)
    return sv.SpecKvAttnDims(*(d[n] for n, _ in sv.SpecKvAttnDims._fields_))


def prompt_dims(**kw):
    d = dict(PROMPT, **kw)
    return sv.SpecPromptDims(*(d[n] for n, _ in sv.SpecPromptDims._fields_))


KV_BAD = [dict(B=0), dict(B=65536), dict(S=0), dict(S=257), dict(heads=7), dict(heads=0), dict(kv_heads=0),
          dict(heads=130, kv_heads=2, q_stride=130 * 128), dict(heads=2048, kv_heads=1024, q_stride=2048 * 128),
          dict(head_dim=96), dict(head_dim=256), dict(page_size=0), dict(num_pages=0), dict(max_pages=0),
          dict(max_pages=1 << 30, page_size=4), dict(num_pages=1 << 30, page_size=4), dict(dtype=2), dict(dtype=-1),
          dict(q_stride=1023), dict(q_stride=1016), dict(q_stride=1028), dict(B=65535, S=257)]


@pytest.mark.parametrize("bad", KV_BAD)
def test_kv_attention_sizes(lib, bad):
    assert lib.spec_kv_attention_workspace_bytes(kv_dims(**bad)) == 0
    assert lib.spec_kv_attention(GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, 0.1, GOOD, GOOD, kv_dims(**bad), GOOD,
                                 1 << 40, NULL) == DIMS


def test_kv_attention_arguments(lib):
    n = lib.spec_kv_attention_workspace_bytes(kv_dims())
    assert n > 0

    def call(q=GOOD, pool=GOOD, bt=GOOD, sl=GOOD, st=NULL, par=NULL, ql=NULL, scale=0.1, out=GOOD, lse=NULL,
             ws=GOOD, size=n):
        return lib.spec_kv_attention(q, pool, bt, sl, st, par, ql, scale, out, lse, kv_dims(), ws, size, NULL)

    for name in ("q", "pool", "bt", "sl", "out", "ws"):
        assert call(**{name: NULL}) == ARG, name
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=scale) == ARG
    for name in ("q", "pool", "st", "out", "ws"):
        assert call(**{name: OFF8}) == ALIGN, name
    for name in ("bt", "sl", "par", "ql", "lse"):
        assert call(**{name: OFF2}) == ALIGN, name
    assert call(size=n - 1) == WORKSPACE


@pytest.mark.parametrize("bad", [dict(B=0), dict(B=65536), dict(heads=9), dict(kv_heads=0), dict(head_dim=80),
                                 dict(total_q=0), dict(total_q=(1 << 24) + 1), dict(total_k=0), dict(dtype=3),
                                 dict(q_stride=1020), dict(k_stride=248), dict(v_stride=252)])
def test_prompt_attention_sizes(lib, bad):
    assert lib.spec_prompt_attention_workspace_bytes(prompt_dims(**bad)) == 0
    assert lib.spec_prompt_attention(GOOD, GOOD, GOOD, GOOD, GOOD, 0.1, GOOD, GOOD, prompt_dims(**bad), GOOD, 1 << 40,
                                     NULL) == DIMS


def test_prompt_attention_arguments(lib):
    n = lib.spec_prompt_attention_workspace_bytes(prompt_dims())
    assert n > 0

    def call(q=GOOD, k=GOOD, v=GOOD, cq=GOOD, ck=NULL, scale=0.1, out=GOOD, lse=NULL, ws=GOOD, size=n):
        return lib.spec_prompt_attention(q, k, v, cq, ck, scale, out, lse, prompt_dims(), ws, size, NULL)

    for name in ("q", "k", "v", "cq", "out", "ws"):
        assert call(**{name: NULL}) == ARG, name
    assert call(scale=0.0) == ARG and call(scale=float("nan")) == ARG
    for name in ("q", "k", "v", "out", "ws"):
        assert call(**{name: OFF8}) == ALIGN, name
    for name in ("cq", "ck", "lse"):
        assert call(**{name: OFF2}) == ALIGN, name
    assert call(size=n - 1) == WORKSPACE


def pages(B=4, max_pages=8, num_pages=100, page_size=16):
    return sv.SpecKvPagesDims(B, max_pages, num_pages, page_size)


def test_page_operators(lib):
    n = lib.spec_kv_pages_workspace_bytes(pages())
    assert n >= 256 + 16 * 4 + 4 * 4 * 100
    bad = [pages(B=0), pages(B=65536), pages(max_pages=0), pages(num_pages=0), pages(page_size=0),
           pages(max_pages=1 << 28), pages(num_pages=1 << 28)]
    for d in bad:
        assert lib.spec_kv_pages_workspace_bytes(d) == 0

    def release(new=NULL, sl=GOOD, bt=GOOD, ref=GOOD, d=pages(), ws=GOOD, size=n):
        return lib.spec_kv_release(new, sl, bt, ref, d, ws, size, NULL)

    def fork(src=GOOD, dst=GOOD, k=2, sl=GOOD, bt=GOOD, ref=GOOD, d=pages(), ws=GOOD, size=n):
        return lib.spec_kv_fork(src, dst, k, sl, bt, ref, d, ws, size, NULL)

    def reserve(need=GOOD, sl=GOOD, bt=GOOD, ref=GOOD, pool=GOOD, layers=2, entry=64, d=pages(), ws=GOOD, size=n):
        return lib.spec_kv_reserve(need, sl, bt, ref, pool, layers, entry, d, ws, size, NULL)

    def compact(bt=GOOD, ref=GOOD, pool=GOOD, layers=2, entry=64, live=NULL, d=pages(), ws=GOOD, size=n):
        return lib.spec_kv_compact(bt, ref, pool, layers, entry, live, d, ws, size, NULL)

    for fn, need in ((release, "sl bt ref ws"), (fork, "src dst sl bt ref ws"), (reserve, "need sl bt ref pool ws"),
                     (compact, "bt ref pool ws")):
        for name in need.split():
            assert fn(**{name: NULL}) == ARG, (fn, name)
        for d in bad:
            assert fn(d=d) == DIMS
        assert fn(ws=OFF8) == ALIGN and fn(bt=OFF2) == ALIGN and fn(ref=OFF2) == ALIGN
        assert fn(size=n - 1) == WORKSPACE
    assert release(new=OFF2) == ALIGN and fork(src=OFF2) == ALIGN and reserve(need=OFF2) == ALIGN
    assert compact(live=OFF2) == ALIGN
    assert fork(k=0) == DIMS and fork(k=65536) == DIMS
    for fn in (reserve, compact):
        assert fn(pool=OFF8) == ALIGN
        for kw in (dict(layers=0), dict(layers=65536), dict(entry=0), dict(entry=24)):
            assert fn(**kw) == DIMS


def test_path_commit(lib):
    d = sv.SpecKvDims(4, 16, 2, 16, 100, 10, 4096)
    n = lib.spec_kv_path_workspace_bytes(d)
    assert n >= 256 + 4 * 4
    assert lib.spec_kv_path_workspace_bytes(sv.SpecKvDims(4, 257, 2, 16, 100, 10, 4096)) == 0

    def call(num=GOOD, path=GOOD, sl=GOOD, bt=GOOD, st=NULL, pool=GOOD, dims=d, ws=GOOD, size=n):
        return lib.spec_kv_commit_path(num, path, sl, bt, st, pool, dims, ws, size, NULL)

    for name in ("num", "path", "sl", "bt", "pool", "ws"):
        assert call(**{name: NULL}) == ARG, name
    assert call(dims=sv.SpecKvDims(4, 16, 2, 16, 100, 10, 24)) == DIMS
    assert call(st=OFF8) == ALIGN and call(pool=OFF8) == ALIGN and call(path=OFF2) == ALIGN
    assert call(size=n - 1) == WORKSPACE


def test_binding_refuses_host_tensors_types_and_shapes(lib):
    q = torch.zeros((2, 3, 4, 64), dtype=torch.bfloat16)
    pool = torch.zeros((5, 16, 256), dtype=torch.bfloat16)
    bt, sl = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        sv.spec_kv_attention(q, pool, bt, sl)
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        sv.spec_kv_attention(q.float(), pool.float(), bt, sl)
    with pytest.raises(ValueError, match="share a dtype"):
        sv.spec_kv_attention(q, pool.half(), bt, sl)
    with pytest.raises(ValueError, match="entry"):
        sv.spec_kv_attention(q, pool[..., :200].contiguous(), bt, sl)
    with pytest.raises(ValueError, match="heads of a token"):
        sv.spec_kv_attention(q.transpose(2, 3), pool, bt, sl)
    with pytest.raises(ValueError, match="evenly"):
        sv.spec_kv_attention(torch.zeros((2, 6, 4, 64), dtype=q.dtype)[:, :3], pool, bt, sl)
    with pytest.raises(ValueError, match="block_table"):
        sv.spec_kv_attention(q, pool, bt[0], sl)
    p = torch.zeros((7, 4, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="total_q"):
        sv.spec_prompt_attention(p, p, p[:6], sl)
    with pytest.raises(ValueError, match="cu_q"):
        sv.spec_prompt_attention(p, p, p, sl[:1])
    with pytest.raises(ValueError, match="CUDA"):
        sv.spec_prompt_attention(p, p, p, sl)
    ref = torch.zeros(9, dtype=torch.int32)
    for fn in (lambda: sv.kv_pages_workspace(bt, ref), lambda: sv.spec_kv_release(None, sl, bt, ref, 16),
               lambda: sv.spec_kv_fork(sl, sl, sl, bt, ref, 16),
               lambda: sv.spec_kv_reserve(sl, sl, bt, ref, torch.zeros((1, 9, 16, 8))),
               lambda: sv.spec_kv_compact(bt, ref, torch.zeros((1, 9, 16, 8))),
               lambda: sv.spec_kv_commit_path(sl, bt, sl, bt, torch.zeros((1, 9, 16, 8)))):
        with pytest.raises(ValueError, match="CUDA"):
            fn()
    with pytest.raises(ValueError, match="block_table"):
        sv.spec_kv_release(None, sl, bt[0], ref, 16)


def test_an_attention_workspace_does_not_depend_on_the_batch(lib):
    """One workspace serves calls of any batch: what has to be zero lies at the same place for all."""
    assert len({lib.spec_kv_attention_workspace_bytes(kv_dims(B=b)) for b in (1, 4, 200, 65535)}) == 1
    assert len({lib.spec_prompt_attention_workspace_bytes(prompt_dims(B=b)) for b in (1, 4, 200, 65535)}) == 1


@pytest.mark.parametrize("scale", [2.36e38, 3.4e38])
def test_scales_whose_product_with_log2_e_is_infinite(lib, scale):
    """(0 times it would not be a number: a row of zero scores is the mean of its values.)"""
    kv, pr = kv_dims(), prompt_dims()
    assert lib.spec_kv_attention(GOOD, GOOD, GOOD, GOOD, NULL, NULL, NULL, scale, GOOD, NULL, kv, GOOD, 1 << 40,
                                 NULL) == ARG
    assert lib.spec_prompt_attention(GOOD, GOOD, GOOD, GOOD, NULL, scale, GOOD, NULL, pr, GOOD, 1 << 40, NULL) == ARG
