"""Filtered logits where 512 T is small beside the largest logit: what was removed weighs nothing all the same.

Tokens and rows are compared with oracle/sample.py as in test_gpu_sample.py."""
import math

import pytest
import torch

import _helpers as H
import oracle
import speculative_decoding_verification_67_gb300 as sv
from test_gpu_sample import check, rows

pytestmark = pytest.mark.gpu


def weightless(z, out, T):
    """Every removed token's logit lies 380 T and more below the largest."""
    gone = (out != z) & (z > -math.inf) | (z == -math.inf)
    far = (z.amax(1, keepdim=True).double() - out.double()) / T
    assert gone.any() and (far[gone] >= 380).all()


@pytest.mark.parametrize("T", [0.0, 1e-6, 1e-9, 1e-20, 1e-30, 1e-37])
@pytest.mark.parametrize("size", [20.0, 5e4, 1e10, 0.0])
def test_low_temperatures(T, size):
    z, u = rows(5, 20000, seed=21)
    z = (z * 4).round() / 4 + size                            # (many equals at the largest)
    z[1, ::3] = -math.inf
    z[2, 7:30] = z[2].max() + max(size, 1.0) * 2.0 ** -20
    # (0.37113 of 20000, 30, 23 and few equals is nowhere near a whole number)
    for kw in (dict(top_k=2), dict(top_p=0.37113), dict(top_k=30, top_p=0.37113), dict(min_p=0.5)):
        check(z, u, T=T, most_near=1, **kw)
    if T:
        out = torch.empty_like(z)
        sv.spec_sample(z, None, T, top_k=1, out_logits=out)
        weightless(z, out, float(torch.tensor(T)))


@pytest.mark.parametrize("T", [1e-6, 1e-9, 1e-20])
def test_equals_that_were_removed_through_the_verify_step(T):
    """None of them is emitted.  (The verify step's exponents are z log2(e) / T in f32 pairs: 23 * 1.44 / 1e-9 = 3e10 is beyond
    2^24, where their steps exceed 1, and it reports such rows instead.)"""
    B, K, V = 24, 3, 2000
    g = torch.Generator(device="cuda").manual_seed(22)
    zp = torch.randint(0, 4, (B * (K + 1), V), generator=g, device="cuda").float() + 20
    zq = zp.view(B, K + 1, V)[:, :K].clone()
    zq[:, ::2, :9] = 23.0                                     # (other equals come first in some draft rows)
    zq = zq.reshape(B * K, V)
    fp, fq = torch.empty_like(zp), torch.empty_like(zq)
    sv.spec_sample(zp, None, T, top_k=3, out_logits=fp)
    drafts = sv.spec_sample(zq, torch.rand(B * K, generator=g, device="cuda"), T, top_k=3, out_logits=fq)
    u = torch.rand((B, K + 1), generator=g, device="cuda")
    tok, acc = sv.spec_verify_from_logits(fp, fq, drafts.view(B, K), u, T)
    if T >= 1e-6:
        ref = oracle.verify_sampling(H.np64(fp).reshape(B, K + 1, V), H.np64(fq).reshape(B, K, V),
                                     H.np_int(drafts).reshape(B, K), H.np64(u), H.t32(T))
        H.compare_sampling(H.np_int(tok), H.np_int(acc), ref, K)
    keeps = torch.zeros_like(zp, dtype=torch.bool)
    first = torch.where(zp == 23, torch.arange(V, device="cuda"), V).sort(1)[0][:, :3]
    keeps.scatter_(1, first, True)
    for b in range(B):
        for j in range(int(acc[b]) + 1):
            assert keeps[b * (K + 1) + j, int(tok[b, j])]


@pytest.mark.parametrize("T", [1.0, 1e-9, 1e-20])
@pytest.mark.parametrize("V,R", [(300001, 3), (200000, 300)])
def test_in_place_beyond_shared_memory(V, R, T):
    """What a draw reads again from memory is not overwritten before it is through; -FLT_MAX takes the place of nothing."""
    z, u = rows(R, V, seed=23, sd=1.0)
    z = (z * 4).round() / 4 + 50
    z[0] = -torch.finfo(torch.float32).max                    # (equals that no value lies below)
    for kw in (dict(top_k=1000), dict(top_p=0.37113), dict(min_p=0.9)):
        want = torch.empty_like(z)
        tok = sv.spec_sample(z, u, T, out_logits=want, **kw)
        for _ in range(3):
            same = z.clone()
            assert torch.equal(sv.spec_sample(same, u, T, out_logits=same, **kw), tok)
            assert torch.equal(same, want)
