"""Attention over the 8-bit cache where its weights are very unequal, against the fp64 definition.

Tolerance, per element, from include/spec_kv8.h.  With u = eps/2 of the type and f = 2^-24:
  * scores: a query element is good to 2^-27 of its row's largest, products accumulate in f32:
    2^-27 scale max|q| sum|k| + (D + 16) f reach, reach = 1.1 scale sum |q||k|; exp2 and rescalings 2^-17
  * sums: a thread adds a weight of each block (nb of them) and 16 sums are joined, (nb + 16) f; the products take 32 keys
    a step, 4 a block, and may be cut off instead of rounded: (4 nb + 8) 2^-23
  * a cached weight times its value's scale: 2^-11 of itself, or 2^-18 of the largest in its block of 128 keys (`fine`
    blocks 2^-23: there the largest is 8 at least, as the block sets the row's reference), or 2^-50 of the row's largest
    (new entries count with a scale of 1); times the code
  * a new entry's weight: u of itself
  * the result: u of itself, half the smallest subnormal at least."""
import math

import pytest
import torch

import speculative_decoding_verification_67_gb300 as sv
from test_gpu_kv8 import F8, Cache8

pytestmark = pytest.mark.gpu


def limits(c, S, b=0, hidden=(), fine=(), scale=None):
    """out, lse and their limits, [S][heads][D] and [S][heads], of a chain; `hidden`: new entries that score -infinity."""
    scale = scale or float(torch.tensor(1 / math.sqrt(c.D), dtype=torch.float32))
    old, vs = c.entries(b)
    L = len(old)
    new = c.staged[b, :S].double().view(S, 2, c.kv, c.D).clone()
    sees = torch.cat([torch.ones((S, L), dtype=torch.bool), torch.ones((S, S), dtype=torch.bool).tril()], 1).cuda()
    for i in hidden:
        sees[:, L + i] = False
        new[i] = 0
    u, f, nb = torch.finfo(c.dtype).eps / 2, 2.0 ** -24, -(-L // 128) + -(-S // 128)
    block = torch.arange(L, device="cuda") // 128
    outs = []
    for h in range(c.heads):
        kvh = h // (c.heads // c.kv)
        q = c.q[b, :S, h].double()
        k, v = (torch.cat([old[:, i, kvh], new[:, i, kvh]]) for i in (0, 1))
        s = (q @ k.T * scale).masked_fill(~sees, -math.inf)
        top = s.amax(1, keepdim=True)
        w = torch.exp(s - top)
        total = w.sum(1, keepdim=True)
        out, lse = w @ v / total, (top + total.log())[:, 0]
        reach = 1.1 * scale * (q.abs() @ k.abs().T).masked_fill(~sees, 0).amax(1, keepdim=True)
        rel = (c.D + 16) * f * reach + scale * 2.0 ** -27 * q.abs().amax(1, keepdim=True) * k.abs().sum(1).amax() + 2.0 ** -17
        scaled = w[:, :L] * vs[:, kvh]
        codes = torch.where(vs[:, kvh, None] > 0, old[:, 1, kvh].abs() / vs[:, kvh, None], 0)
        coarse = 2.0 ** -50 * torch.cat([scaled, w[:, L:]], 1).amax(1, keepdim=True) * codes.sum(0)
        if L:
            size = int(block[-1]) + 1
            most = torch.nn.functional.pad(scaled, (0, size * 128 - L)).view(S, size, 128).amax(2)
            step = torch.full((size,), 2.0 ** -18, dtype=torch.float64, device="cuda")
            step[list(fine)] = 2.0 ** -23
            sums = torch.zeros((size, c.D), dtype=torch.float64, device="cuda").index_add_(0, block, codes)
            coarse = coarse + (most * step) @ sums
        weight = w @ v.abs() / total
        lim = (u * out.abs() + (2.0 ** -11 + 2 * rel + (4 * nb + 8) * 2.0 ** -23 + (nb + 16) * f) * weight +
               u * (w[:, L:] @ v[L:].abs()) / total + coarse / total + torch.finfo(c.dtype).tiny * u)
        outs.append((out, lse, lim, (rel + (nb + 16) * f)[:, 0] + 2 * f * lse.abs()))
    return [torch.stack(x, 1) for x in zip(*outs)]


def check(c, S, b=0, got=None, **kw):
    if got is None:
        out, lse, err = c.run()
        assert err == 0
        got = out[b], lse[b]
    out, lse, lim, lim_lse = limits(c, S, b, **kw)
    assert torch.isfinite(got[0]).all() and torch.isfinite(got[1]).all()
    far = ((got[0].double() - out).abs() / lim)
    assert far.max() <= 1, (far.max(), (far == far.max()).nonzero()[0].tolist())
    assert ((got[1].double() - lse).abs() <= lim_lse).all()


def alone(c, B=None):
    """The call with so many sequences (the first one again and again) that a CTA walks a whole item; the first one's rows."""
    if B is None:
        B = -(-torch.cuda.get_device_properties(0).multi_processor_count // c.kv)
    more = lambda x: x[:1].expand(B, *x.shape[1:]).contiguous()  # noqa: E731
    q = more(c.q)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    ws = sv.kv8_attention_workspace(q, c.scales)
    sv.spec_kv8_attention(q, c.pool, c.scales, more(c.table), more(c.seq_len), more(c.staged), out=out, out_lse=lse,
                          workspace=ws)
    assert sv.kv8_read_error(ws) == 0
    return out[0], lse[0]


# ---------------------------------------------- blocks in which a row sees nothing
def low_scores(lens, S, heads, kv, first, last, dtype="bf16", seed=31):
    """Queries of about 1 and keys of -1: scores (natural logarithms) from `first` to `last` along each cache."""
    c = Cache8(lens, S, heads, kv, 64, 16, "e4m3", dtype, seed=seed, spread=0.0)
    c.q.copy_(1 + 2.0 ** -6 * c.q.float().clamp(-3, 3))
    c.pool.view(torch.uint8)[..., :kv * 64] = 0xb8
    c.scales[:, 1] = 1.0
    for b, n in enumerate(lens):
        held = -(-n // 16)
        c.scales[c.table[b, :held].long(), 0] = torch.linspace(-first / 8, -last / 8, held, device="cuda")[:, None]
    return c


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("first,last", [(-56.0, -55.0), (-90.0, -55.0), (-83.0, -83.0), (-60.0, -85.0)])
@pytest.mark.parametrize("L", [5, 300, 1000])
def test_a_new_entry_of_minus_infinity_before_low_scores(first, last, L, dtype):
    c = low_scores([L], 1, 4, 2, first, last, dtype)
    c.staged[..., :128] = -math.inf
    check(c, 1, hidden=[0])
    check(c, 1, got=alone(c), hidden=[0])


@pytest.mark.parametrize("first,last", [(-56.0, -55.0), (-90.0, -55.0), (-83.0, -83.0)])
def test_a_second_block_of_new_entries_before_low_scores(first, last):
    """Pieces of an item that begin with new entries 128 and more, which rows before them do not see."""
    lens = [250, 300, 413, 520, 640, 777, 900, 1100]
    c = low_scores(lens, 256, 4, 2, first, last)
    c.staged[..., :128] = -8.0                                # scores of about -64
    out, lse, err = c.run()
    assert err == 0
    for b in range(len(lens)):
        check(c, 256, b, (out[b], lse[b]))
