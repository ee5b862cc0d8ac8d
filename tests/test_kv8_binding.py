"""What the binding of the 8-bit cache and of sampling says before it looks for a device; runs without a GPU."""
import warnings

import pytest
import torch

import speculative_decoding_verification_67_gb300 as sv


@pytest.mark.parametrize("dtype", [torch.float8_e4m3fn, torch.float8_e5m2])
def test_pages_of_a_float8_pool_without_scales(dtype):
    """A warning, as calls with a pool whose scales lie elsewhere go on to work."""
    pool = torch.zeros((1, 9, 16, 128), dtype=torch.uint8)
    table, ref, one = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(9, dtype=torch.int32), \
        torch.zeros(2, dtype=torch.int32)
    scales = torch.zeros(1, 9, 2, 1)
    calls = (lambda p, **kw: sv.spec_kv_reserve(one, one, table, ref, p, **kw),
             lambda p, **kw: sv.spec_kv_compact(table, ref, p, **kw))
    for call in calls:
        with pytest.warns(UserWarning, match="scales"), pytest.raises(ValueError, match="CUDA"):
            call(pool.view(dtype))
        for args, kw in (((pool,), {}), ((pool.view(dtype),), dict(scales=scales)), ((pool.to(torch.bfloat16),), {})):
            with warnings.catch_warnings(), pytest.raises(ValueError, match="CUDA"):
                warnings.simplefilter("error")
                call(*args, **kw)


@pytest.mark.parametrize("top_k,want", [(0, 0), (7, 7), (-5, -5), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1),
                                        (2 ** 32 + 5, 2 ** 31 - 1), (-2 ** 40 + 3, -2 ** 31)])
def test_top_k_beyond_32_bits(monkeypatch, top_k, want):
    """The setting that reaches the ABI keeps its meaning (2^32 + 5 is not 5)."""
    seen = []
    struct = sv.SpecSampleParams
    monkeypatch.setattr(sv, "SpecSampleParams", lambda *a: seen.append(struct(*a)) or seen[0])
    with pytest.raises(ValueError, match="CUDA"):
        sv.spec_sample(torch.zeros(3, 50), torch.zeros(3), top_k=top_k)
    assert seen[0].top_k == want
    with pytest.raises(TypeError):
        sv.spec_sample(torch.zeros(3, 50), torch.zeros(3), top_k=2.0)
