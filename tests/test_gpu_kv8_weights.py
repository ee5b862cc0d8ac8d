"""Attention over the 8-bit cache where its weights are very unequal, against the fp64 definition.

Tolerance, per element, from include/spec_kv8.h.  With u = eps/2 of the type and f = 2^-24:
  * scores: a query element is good to 2^-27 of its row's largest, products accumulate in f32:
    2^-27 scale max|q| sum|k| + (D + 16) f reach, reach = 1.1 scale sum |q||k|; exp2 and rescalings 2^-17
  * sums: a thread adds a weight of each block (nb of them) and 16 sums are joined, (nb + 16) f; the products take 32 keys
    a step, 4 a block, and may be cut off instead of rounded: (4 nb + 8) 2^-23
  * a cached weight times its value's scale: 2^-11 of itself, or half the last part's step, 2^-25 in units in which the row's
    largest is 2 at least where references were set: 2^-26 of it (new entries count with a scale of 1); times the code.
    Where references rose by 2^10 or more, or were set at first, the next cached block's largest is 2^-8 at least; in tests
    whose blocks are alike from there on (within 2^2 of one another) that is `step` = 2^-15 of each block's largest
  * a new entry's weight: u of itself
  * the result: u of itself, half the smallest subnormal at least."""
import math

import pytest
import torch

import speculative_decoding_verification_67_gb300 as sv
from test_gpu_kv8 import F8, Cache8

pytestmark = pytest.mark.gpu


def limits(c, S, b=0, hidden=(), step=None, first=None, scale=None):
    """out, lse and their limits, [S][heads][D] and [S][heads], of a chain; `hidden`: new entries that score -infinity;
    `step`: of each block's largest weight times scale (`first`: of the first block's), None: 2^-26 of the row's."""
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
        if step is None:
            coarse = 2.0 ** -26 * torch.cat([scaled, w[:, L:]], 1).amax(1, keepdim=True) * codes.sum(0)
        else:
            size = int(block[-1]) + 1
            most = torch.nn.functional.pad(scaled, (0, size * 128 - L)).view(S, size, 128).amax(2) * step
            if first is not None:
                most[:, 0] *= first / step
            coarse = most @ torch.zeros((size, c.D), dtype=torch.float64, device="cuda").index_add_(0, block, codes)
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


# --------------------------------------------------------- small weights beside large ones
def common_mean(L, log_scale, dtype, D=64, S=1, heads=4, seed=41):
    """Scores of standard deviation 1/2, values of mean 1/2 and standard deviation 1, whose scale is given."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = Cache8([L], S, heads, heads, D, 16, "e4m3", dtype, seed=seed, spread=0.0, spare=0)
    shape = c.pool.shape[:2] + (heads * D,)
    keys = 0.5 * torch.randn(shape, generator=g, device="cuda")
    values = 0.5 + torch.randn(shape, generator=g, device="cuda")
    c.scales[:, 0], c.scales[:, 1] = 2.0 ** -6, 2.0 ** log_scale
    c.pool.copy_(torch.cat([keys * 2.0 ** 6, (values * 2.0 ** -log_scale).clamp(-448, 448)], 2).to(F8["e4m3"]))
    return c


def want_score(c, share, skip=0):
    """[heads]: the score with which a key has that share beside the cached ones from `skip` on, for the first token."""
    k = c.entries(0)[0][skip:, 0]
    s = torch.einsum("hd,lhd->hl", c.q[0, 0].double(), k) / math.sqrt(c.D)
    return s.logsumexp(1) + math.log(share / (1 - share))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("L,share", [(8191, 0.9), (32000, 0.5), (32000, 0.8), (60000, 0.8), (60000, 0.98)])
@pytest.mark.parametrize("log_scale", [-8, -7, -6])
def test_a_new_token_with_most_of_the_weight(L, share, log_scale, dtype):
    """Cached weights of 2^-15 to 2^-22 of the new token's, before their values' scale."""
    c = common_mean(L, log_scale, dtype)
    c.q.mul_(4).clamp_(-4, 4)
    c.scales[:, 0] *= 0.25
    q = c.q[0, 0].double()
    new = want_score(c, share)[:, None] * math.sqrt(c.D) / q.square().sum(1, keepdim=True) * q
    c.staged[0, 0, :c.kv * c.D] = new.to(c.dtype).flatten()
    c.staged[0, 0, c.kv * c.D:] *= 2.0 ** -8                  # (its own values are small, so that the cached ones count)
    check(c, 1, got=alone(c), step=2.0 ** -15)


def test_new_entries_of_large_values_whose_weight_is_large():
    """What they leave in O grows when the reference is set anew for the cached keys."""
    c = common_mean(3000, -7, "bf16")
    q = c.q[0, 0].double()
    new = want_score(c, 0.99999)[:, None] * math.sqrt(c.D) / q.square().sum(1, keepdim=True) * q
    c.staged[0, 0, :c.kv * c.D] = new.to(c.dtype).flatten()
    c.staged[0, 0, c.kv * c.D:] *= 2.0 ** 60
    check(c, 1, got=alone(c), step=2.0 ** -15)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("L,share", [(8000, 0.99), (32000, 0.99), (8000, 0.999), (32000, 0.999)])
@pytest.mark.parametrize("S", [1, 6])
def test_a_cached_key_with_most_of_the_weight_and_no_value(L, share, S, dtype):
    """The first key's block sets the reference (the new tokens' own scores are far below it), the others come behind it."""
    c = common_mean(L, -7, dtype, S=S)
    q = c.q[0, 0].double()
    c.q[0] = c.q[0, :1]                                       # (rows of a chain that ask for the same)
    c.staged[..., :c.kv * c.D] = 0
    c.staged[..., c.kv * c.D:] *= 2.0 ** -10
    key = want_score(c, share, 1)[:, None] * math.sqrt(c.D) / q.square().sum(1, keepdim=True) * q
    page = int(c.table[0, 0])
    first = c.pool[page, 0].float()
    first[:c.kv * c.D] = (key.flatten() * 2.0 ** 6).float()
    first[c.kv * c.D:] = 2.0 ** -9
    c.pool[page, 0] = first.clamp(-448, 448).to(F8["e4m3"])
    s = torch.einsum("hd,lhd->hl", q, c.entries(0)[0][:, 0]) / math.sqrt(c.D)
    assert (s.softmax(1)[:, 0] > 1 - 3 * (1 - share)).all()
    check(c, S, got=alone(c), step=2.0 ** -15, first=2.0 ** -26)


@pytest.mark.parametrize("S,heads,D", [(1, 8, 64), (5, 8, 128), (4, 12, 64), (40, 2, 128), (130, 2, 64)])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("drop", [12, 20, 30, 44])
def test_a_page_of_zeros_and_smaller_ones_behind_it(S, heads, D, fmt, drop):
    """The first block's values are zeros of a large scale, the others' scales are 2^-drop of it."""
    c = Cache8([1500], S, heads, 2, D, 64, fmt, "fp16", seed=51, spread=0.0)
    order, kv = c.table[0, :24].long(), 2 * D
    c.scales[:, 0] *= 0.25
    c.scales[order, 1] = 2.0 ** (drop - 6 if fmt == "e4m3" else drop - 14)
    c.scales[order[2:], 1] *= 2.0 ** -drop
    c.pool.view(torch.uint8)[order[:2], :, kv:] = 0
    c.staged[..., kv:] = 0
    c.staged[..., :kv] *= 0.25
    # (what is in O grows by 2^32 at most: the others' largest is 2^(2 - 44 + 32) then, less 2 and one for the rounding)
    step = 2.0 ** -15 if drop <= 30 else 2.0 ** -12
    first = 2.0 ** -26
    if S * heads <= 8:
        check(c, S, got=alone(c), step=step, first=first)
    check(c, S, step=step, first=first)


@pytest.mark.parametrize("S,heads,D", [(1, 8, 64), (1, 32, 128), (4, 12, 64), (40, 2, 128), (9, 9, 64)])
@pytest.mark.parametrize("spread", [6, 12, 30])
@pytest.mark.parametrize("seed", range(3))
def test_blocks_of_very_different_size(S, heads, D, spread, seed):
    """Blocks whose values' scales differ by any powers of two up to 2^60; the heaviest half holds zeros."""
    kv = 3 if heads == 9 else 2
    c = Cache8([3000], S, heads, kv, D, 128, "e4m3", "fp16", seed=60 + seed, spread=0.0)
    g = torch.Generator().manual_seed(seed)
    order = c.table[0, :24].long()
    size = torch.randint(-spread, spread + 1, (24,), generator=g)
    # (the lightest half's values are of the size of its heaviest block, so that results are not below fp16's range)
    c.scales[order, 1] = torch.exp2((size - size.median()).float() - 12).cuda()[:, None]
    c.pool.view(torch.uint8)[order[(size > size.median()).cuda()], :, kv * D:] = 0
    c.staged[..., kv * D:] = 0
    check(c, S)
    if S * heads <= 32:
        check(c, S, got=alone(c))


@pytest.mark.parametrize("S,heads", [(1, 4), (12, 4)])
def test_scores_that_fall_and_rise(S, heads):
    """Keys that point along the queries by turns more and less, values' scales that fall with them or rise."""
    for sign in (1, -1):
        # (values of up to 448 2^(24 - 9) or so: bf16, as fp16 ends at 65504)
        c = Cache8([2500], S, heads, 2, 64, 16, "e4m3", "bf16", seed=71, spread=0.0)
        order = c.table[0, :157].long()
        wave = 3 * torch.sin(torch.arange(157, device="cuda") / 3.0) + torch.linspace(0, 3, 157, device="cuda")
        c.scales[order, 0] *= torch.exp2(wave - 3)[:, None]
        c.scales[order, 1] *= torch.exp2(sign * 4 * wave)[:, None]
        check(c, S)
        check(c, S, got=alone(c))
