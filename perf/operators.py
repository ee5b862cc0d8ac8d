"""What the cache operators are measured on: the cases, their inputs, their plain form and their work.

Four operators around the paged key-value cache of a speculative round:

* attention of a sequence's newest tokens over its cache pages (``spec_kv_attention``): one token, a drafted
  chain, or a tree of candidates;
* attention over packed prompts (``spec_prompt_attention``);
* the cache's pages (``spec_kv_release``, ``spec_kv_fork``, ``spec_kv_reserve``, ``spec_kv_compact``);
* the commit of an accepted tree path (``spec_kv_commit_path``).

An entry of the cache is one layer's key and value of one position, ``[2][kv_heads][head_dim]``.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _sv():
    import speculative_decoding_verification_67_gb300 as sv
    return sv


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # One sequence decoding one token: the smallest call of a serving loop, where latency is what counts.
        dict(name="token_B1_L1000", op="attention", dtype="bf16", B=1, S=1, heads=32, kv_heads=8, head_dim=128,
             page=16, lo=1000, hi=1000, staged=False, tree="", lse=False),
        # A full decoding batch of a large model: ragged caches up to 8191 positions, one token each, the token's
        # entry still staged.
        dict(name="token_B64_L8191", op="attention", dtype="bf16", B=64, S=1, heads=64, kv_heads=8, head_dim=128,
             page=16, lo=512, hi=8191, staged=True, tree="", lse=False),
        # The target pass over four drafts and the pending token (K = 4), entries in place; a page size that does
        # not divide the kernel's tiles.
        dict(name="chain_B8_K4_L4095", op="attention", dtype="fp16", B=8, S=5, heads=32, kv_heads=8, head_dim=128,
             page=24, lo=512, hi=4095, staged=False, tree="", lse=True),
        # The tree pass over 40 candidates with a small model's heads: groups of three, odd pages.
        dict(name="tree_B4_N40_L2500", op="attention", dtype="bf16", B=4, S=40, heads=12, kv_heads=4, head_dim=64,
             page=7, lo=777, hi=2500, staged=True, tree="3,3,3", lse=False),
        # The last pieces of three prompts whose first parts are already processed: few rows, longer keys.
        dict(name="pieces_B3_T97", op="prompt", dtype="fp16", B=3, lo=11, hi=97, before=301, heads=16, kv_heads=16,
             head_dim=64, lse=True),
        # A prefill batch: prompts of very different lengths packed behind each other.
        dict(name="prompts_B16_T2047", op="prompt", dtype="bf16", B=16, lo=1, hi=2047, before=0, heads=32,
             kv_heads=8, head_dim=128, lse=False),
        # One long prompt.
        dict(name="prompt_T12301", op="prompt", dtype="bf16", B=1, lo=12301, hi=12301, before=0, heads=32,
             kv_heads=8, head_dim=128, lse=False),
        # Sampling four continuations of each of two prompts: drop the losers, share the winner's pages, make room
        # for the next round.
        dict(name="pages_B8_layers32", op="pages", B=8, fan=4, n=5, layers=32, entry=4096, page=16, lo=40, hi=200),
        # The same for 16 prompts on a model of 80 layers.
        dict(name="pages_B64_layers80", op="pages", B=64, fan=4, n=9, layers=80, entry=4096, page=16, lo=64, hi=400),
        # After sequences have left: the live pages move to the front of the pool.
        dict(name="compact_P1501", op="compact", B=32, layers=32, entry=4096, page=16, pages=1501, percent=61),
        # The accepted path of 64 trees of 16 candidates, from staged entries.
        dict(name="path_B64_N16_layers80", op="path", B=64, N=16, layers=80, entry=4096, page=16, staged=True,
             depth=3, lo=512, hi=8191),
        # The same where the tree pass wrote its entries in place.
        dict(name="path_B8_N57_layers32", op="path", B=8, N=57, layers=32, entry=4096, page=16, staged=False,
             depth=3, lo=512, hi=4095),
    ]


def _log(rng, a, b):
    return min(b, max(a, int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "prompt", "prompt", "prompt", "pages", "compact", "path"])
    if op == "attention":
        kv = rng.choice([1, 2, 4, 8])
        tree = rng.choice(["", "", "", "3,2,1", "3,3,3", "8,2,2", "2,1"])
        S = _tree_size(tree) if tree else rng.choice([1, 1, 1, 2, 3, 5, 9])
        B = _log(rng, 1, 64)
        hi = min(_log(rng, 1, 8191), 400000 // (B * kv))
        lo = rng.randint(0, hi)
        return dict(op=op, dtype=rng.choice(["bf16", "fp16"]), B=B, S=S, heads=kv * rng.choice([1, 2, 3, 4, 7, 8]),
                    kv_heads=kv, head_dim=rng.choice([64, 128]), page=rng.choice([1, 5, 8, 16, 24, 32, 64, 100, 128]),
                    lo=lo, hi=hi, staged=rng.random() < 0.5, tree=tree, lse=rng.random() < 0.5)
    if op == "prompt":
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 3, 4, 7])
        hi = _log(rng, 1, 4000)
        B = min(_log(rng, 1, 16), max(1, (1 << 29) // (heads * hi * hi)))
        return dict(op=op, dtype=rng.choice(["bf16", "fp16"]), B=B, lo=rng.randint(1, hi), hi=hi,
                    before=rng.choice([0, 0, rng.randint(1, 500)]), heads=heads, kv_heads=kv,
                    head_dim=rng.choice([64, 128]), lse=rng.random() < 0.5)
    layers, entry = rng.choice([1, 7, 32, 60]), rng.choice([256, 1040, 4096])
    if op == "pages":
        fan = rng.choice([1, 2, 3, 4])
        lo = _log(rng, 1, 200)
        return dict(op=op, B=fan * _log(rng, 1, 16), fan=fan, n=rng.choice([1, 2, 5, 9, 40]), layers=layers,
                    entry=entry, page=rng.choice([1, 3, 8, 16, 32]), lo=lo, hi=lo + rng.randint(0, 150))
    if op == "compact":
        return dict(op=op, B=_log(rng, 1, 64), layers=layers, entry=entry, page=rng.choice([1, 3, 8, 16]),
                    pages=_log(rng, 2, 1200), percent=rng.randint(1, 100))
    return dict(op=op, B=_log(rng, 1, 64), N=rng.choice([10, 16, 40, 57]), layers=layers, entry=entry,
                page=rng.choice([1, 3, 8, 16, 32]), staged=rng.random() < 0.5, depth=rng.choice([1, 2, 3, 4]),
                lo=0, hi=_log(rng, 1, 8191))


def _lengths(case):
    """The batch's lengths, spread over [lo, hi]; prepare() deals them out in another order for each seed."""
    span = case["hi"] - case["lo"] + 1
    return [case["lo"] + int(span * (((b + 1) * 0.6180339887498949) % 1.0)) for b in range(case["B"])]


def _tree_parents(tree):
    parents, level = [-1], [0]
    for k in (int(x) for x in tree.split(",")):
        nxt = []
        for p in level:
            for _ in range(k):
                parents.append(p)
                nxt.append(len(parents) - 1)
        level = nxt
    return parents


def _tree_size(tree):
    return len(_tree_parents(tree))


def _cells(n, page):
    return -(-n // page)


# ----------------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    return {"attention": _prepare_attention, "prompt": _prepare_prompt, "pages": _prepare_pages,
            "compact": _prepare_compact, "path": _prepare_path}[case["op"]](case, seed)


def _gens(seed):
    return torch.Generator(device="cuda").manual_seed(seed), torch.Generator().manual_seed(seed), random.Random(seed)


def _normal(shape, dtype, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _dealt(case, rng):
    lens = _lengths(case)
    rng.shuffle(lens)
    return lens


def _table(lens, cols, pages, cpu):
    """int32 [B][cols]: distinct pages, in shuffled order, over the first lens[b] columns; -1 behind."""
    perm = torch.randperm(pages, generator=cpu).tolist()
    table = torch.full((len(lens), cols), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        table[b, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
        at += n
    return table.cuda()


def _prepare_attention(case, seed):
    g, cpu, rng = _gens(seed)
    dt, B, S, page = _DT[case["dtype"]], case["B"], case["S"], case["page"]
    lens = _dealt(case, rng)
    held = [_cells(n + S, page) for n in lens]
    pages, entry = sum(held), 2 * case["kv_heads"] * case["head_dim"]
    table = _table(held, max(held), pages, cpu)
    st = dict(case=case, table=table, seq_len=torch.tensor(lens, dtype=torch.int32).cuda(),
              pool=_normal((pages, page, entry), dt, g), staged=None, parents=None, longest=max(lens))
    st["q"] = _normal((B, S, case["heads"], case["head_dim"]), dt, g)
    if case["staged"]:
        st["staged"] = _normal((B, S, entry), dt, g)
    if case["tree"]:
        st["parents"] = torch.tensor(_tree_parents(case["tree"]), dtype=torch.int32).repeat(B, 1).cuda()
    return st


def _prepare_prompt(case, seed):
    g, _, rng = _gens(seed)
    dt, D = _DT[case["dtype"]], case["head_dim"]
    lens = _dealt(case, rng)
    keys = [n + case["before"] for n in lens]
    cu = lambda x: torch.tensor([0] + x, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()  # noqa: E731
    return dict(case=case, cu_q=cu(lens), cu_k=cu(keys), longest=max(lens), longest_k=max(keys),
                q=_normal((sum(lens), case["heads"], D), dt, g), k=_normal((sum(keys), case["kv_heads"], D), dt, g),
                v=_normal((sum(keys), case["kv_heads"], D), dt, g))


def _bytes(shape, g):
    return torch.randint(-30000, 30000, shape, generator=g, device="cuda", dtype=torch.int16)


def _prepare_pages(case, seed):
    """Rows 0 .. B - B/fan - 1 are continuations, the last B/fan rows the sequences they continue."""
    g, cpu, rng = _gens(seed)
    B, fan, n, page = case["B"], case["fan"], case["n"], case["page"]
    roots = B // fan
    lens = _dealt(dict(case, B=roots), rng)
    cols = _cells(max(lens) + n, page)
    pages = sum(_cells(x, page) for x in lens) + B * (_cells(n, page) + 1)
    kids = B - roots
    held = [0] * kids + [_cells(x, page) for x in lens]
    table = _table(held, cols, pages, cpu)
    ref = torch.zeros(pages, dtype=torch.int32)
    ref[table.cpu()[table.cpu() >= 0].long()] = 1
    seq_len = torch.tensor([0] * kids + lens, dtype=torch.int32).cuda()
    src = torch.tensor([kids + i // max(1, fan - 1) for i in range(kids)], dtype=torch.int32).cuda()
    dst = torch.arange(kids, dtype=torch.int32).cuda()
    drop = torch.tensor([0] * kids + [-1] * roots, dtype=torch.int32).cuda()
    st = dict(case=case, table=table, ref=ref.cuda(), seq_len=seq_len, src=src, dst=dst, drop=drop,
              need=torch.full((B,), n, dtype=torch.int32).cuda(),
              pool=_bytes((case["layers"], pages, page, case["entry"] // 2), g))
    _plain_pages(st)  # the round before: the continuations hold their pages
    return st


def _prepare_compact(case, seed):
    g, cpu, _ = _gens(seed)
    P, B = case["pages"], case["B"]
    live = max(1, P * case["percent"] // 100)
    ids = torch.randperm(P, generator=cpu)[:live].to(torch.int32)
    cols = _cells(live, B)
    table = torch.full((B * cols,), -1, dtype=torch.int32)
    table[:live] = ids
    ref = torch.zeros(P, dtype=torch.int32)
    ref[ids.long()] = 1
    table, ref = table.view(B, cols).cuda(), ref.cuda()
    return dict(case=case, table0=table, ref0=ref, table=table.clone(), ref=ref.clone(),
                pool=_bytes((case["layers"], P, case["page"], case["entry"] // 2), g))


def _accepted(case):
    """Accepted candidates of each sequence: 0 to `depth`."""
    return [(b * 7 + 3) % (case["depth"] + 1) for b in range(case["B"])]


def _prepare_path(case, seed):
    g, cpu, rng = _gens(seed)
    B, N, page = case["B"], case["N"], case["page"]
    lens = _dealt(case, rng)
    n = _accepted(case)
    rng.shuffle(n)
    # Accepted nodes lie behind the first `depth` ones, so that a path written in place can be written again.
    path = [sorted(rng.sample(range(case["depth"] + 1, N), k)) + [-1] * (N - k) for k in n]
    cols = _cells(max(lens) + N, page)
    first, last = [x // page for x in lens], [(x + N - 1) // page for x in lens]
    perm, at = torch.randperm(sum(b - a + 1 for a, b in zip(first, last)), generator=cpu) + 1, 0
    table = torch.zeros((B, cols), dtype=torch.int32)  # pages of earlier positions are not touched: page 0
    for b in range(B):
        k = last[b] - first[b] + 1
        table[b, first[b]:last[b] + 1] = perm[at:at + k].to(torch.int32)
        at += k
    width = case["entry"] // 2
    return dict(case=case, seq_len0=torch.tensor(lens, dtype=torch.int32).cuda(),
                seq_len=torch.tensor(lens, dtype=torch.int32).cuda(), table=table.cuda(),
                n=torch.tensor(n, dtype=torch.int32).cuda(), path=torch.tensor(path, dtype=torch.int32).cuda(),
                pool=_bytes((case["layers"], at + 1, page, width), g),
                staged=_bytes((case["layers"], B, N, width), g) if case["staged"] else None)


# --------------------------------------------------------------------------------------------- one pass
def run(st):
    op = st["case"]["op"]
    if own:
        return {"attention": _own_attention, "prompt": _own_prompt, "pages": _own_pages, "compact": _own_compact,
                "path": _own_path}[op](st)
    return {"attention": _plain_attention, "prompt": _plain_prompt, "pages": _plain_pages, "compact": _plain_compact,
            "path": _plain_path}[op](st)


def _kept(st, name, make):
    """What a user's program makes once and keeps: workspaces and output buffers."""
    if name not in st:
        st[name] = make()
    return st[name]


def _own_attention(st):
    sv, q = _sv(), st["q"]
    out = _kept(st, "out", lambda: torch.empty_like(q))
    lse = _kept(st, "lse", lambda: torch.empty(q.shape[:3], dtype=torch.float32, device="cuda")) \
        if st["case"]["lse"] else None
    ws = _kept(st, "ws", lambda: sv.kv_attention_workspace(q, st["pool"]))
    sv.spec_kv_attention(q, st["pool"], st["table"], st["seq_len"], st["staged"], parents=st["parents"], out=out,
                         out_lse=lse, workspace=ws)
    return [out] if lse is None else [out, lse]


def _own_prompt(st):
    sv, q = _sv(), st["q"]
    out = _kept(st, "out", lambda: torch.empty_like(q))
    lse = _kept(st, "lse", lambda: torch.empty(q.shape[:2], dtype=torch.float32, device="cuda")) \
        if st["case"]["lse"] else None
    ws = _kept(st, "ws", lambda: sv.prompt_attention_workspace(q, st["k"], st["case"]["B"]))
    sv.spec_prompt_attention(q, st["k"], st["v"], st["cu_q"], st["cu_k"], out=out, out_lse=lse, workspace=ws)
    return [out] if lse is None else [out, lse]


def _own_pages(st):
    sv, page = _sv(), st["case"]["page"]
    ws = _kept(st, "ws", lambda: sv.kv_pages_workspace(st["table"], st["ref"]))
    sv.spec_kv_release(st["drop"], st["seq_len"], st["table"], st["ref"], page, workspace=ws)
    if len(st["src"]):
        sv.spec_kv_fork(st["src"], st["dst"], st["seq_len"], st["table"], st["ref"], page, workspace=ws)
    sv.spec_kv_reserve(st["need"], st["seq_len"], st["table"], st["ref"], st["pool"], workspace=ws)
    return [st["table"], st["ref"], st["seq_len"], st["pool"]]


def _own_compact(st):
    sv = _sv()
    ws = _kept(st, "ws", lambda: sv.kv_pages_workspace(st["table"], st["ref"]))
    st["table"].copy_(st["table0"])  # the scheduler's tables
    st["ref"].copy_(st["ref0"])
    live = _kept(st, "live", lambda: torch.empty(1, dtype=torch.int32, device="cuda"))
    sv.spec_kv_compact(st["table"], st["ref"], st["pool"], out_num_live=live, workspace=ws)
    return [st["table"], st["ref"], live, st["pool"]]


def _own_path(st):
    sv = _sv()
    st["seq_len"].copy_(st["seq_len0"])  # the scheduler's lengths
    ws = _kept(st, "ws", lambda: sv.kv_path_workspace(st["case"]["B"]))
    sv.spec_kv_commit_path(st["n"], st["path"], st["seq_len"], st["table"], st["pool"], st["staged"], workspace=ws)
    return [st["seq_len"], st["pool"]]


# ------------------------------------------------------------------------------------------ plain forms
def _weights(s, visible):
    """exp(s - max) over the visible keys and their sum; rows without one weigh nothing. Overwrites s."""
    s.masked_fill_(~visible, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    w = s.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    return w, total, (top + total.log()).squeeze(-1)


def _plain_attention(st):
    c, q, table, L = st["case"], st["q"], st["table"].long(), st["seq_len"].long()
    B, S, H, G, D, page = c["B"], c["S"], c["kv_heads"], c["heads"] // c["kv_heads"], c["head_dim"], c["page"]
    dev, longest = q.device, st["longest"]
    old = torch.arange(longest, device=dev).expand(B, longest)
    new = torch.arange(S, device=dev)

    def entries(pos):
        at = table.gather(1, (pos // page).clamp_(max=table.shape[1] - 1)).clamp_(min=0)
        return st["pool"][at, pos % page]

    fresh = st["staged"] if st["staged"] is not None else entries(L[:, None] + new)
    kv = torch.cat([entries(old), fresh], 1).float().view(B, longest + S, 2, H, D)
    k, v = kv[:, :, 0].permute(0, 2, 3, 1), kv[:, :, 1].transpose(1, 2)          # [B,H,D,T], [B,H,T,D]
    if st["parents"] is None:
        among = (new[None, :] <= new[:, None]).expand(B, S, S)
    else:  # ancestors: paths of any length in the parent relation
        step = torch.eye(S, device=dev) + (st["parents"].long()[:, :, None] == new).float()
        among = torch.linalg.matrix_power(step, S) > 0
    visible = torch.cat([(old < L[:, None])[:, None].expand(B, S, longest), among], -1)   # [B,S,T]
    rows = q.float().view(B, S, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, S * G, D)
    s = torch.matmul(rows, k) * (1.0 / math.sqrt(D))
    w, total, lse = _weights(s, visible.repeat_interleave(G, 1)[:, None])
    o = torch.matmul(w, v) / total
    back = lambda x, *t: x.view(B, H, S, G, *t).transpose(1, 2).reshape(B, S, H * G, *t)  # noqa: E731
    out = back(o, D).to(q.dtype)
    return [out, back(lse)] if c["lse"] else [out]


def _plain_prompt(st):
    c, q, cu_q, cu_k = st["case"], st["q"], st["cu_q"].long(), st["cu_k"].long()
    B, H, G, D = c["B"], c["kv_heads"], c["heads"] // c["kv_heads"], c["head_dim"]
    dev, T, U = q.device, st["longest"], st["longest_k"]
    n, m = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    i, j = torch.arange(T, device=dev), torch.arange(U, device=dev)
    rows = (cu_q[:-1, None] + i).clamp_(max=q.shape[0] - 1)
    cells = (cu_k[:-1, None] + j).clamp_(max=st["k"].shape[0] - 1)
    qs = q[rows].float().view(B, T, H, G, D).permute(0, 2, 3, 1, 4)               # [B,H,G,T,D]
    k = st["k"][cells].float().permute(0, 2, 3, 1)[:, :, None]                     # [B,H,1,D,U]
    v = st["v"][cells].float().transpose(1, 2)[:, :, None]
    visible = (j[None, None, :] <= (i[None, :] + (m - n)[:, None])[:, :, None]) & (j < m[:, None])[:, None, :]
    s = torch.matmul(qs, k).mul_(1.0 / math.sqrt(D))
    w, total, lse = _weights(s, visible[:, None, None])
    o = torch.where(total > 0, torch.matmul(w, v) / total, torch.zeros((), device=dev))
    inside = i[None, :] < n[:, None]
    out = o.permute(0, 3, 1, 2, 4).reshape(B, T, H * G, D)[inside].to(q.dtype)
    return [out, lse.permute(0, 3, 1, 2).reshape(B, T, H * G)[inside]] if c["lse"] else [out]


def _plain_release(new_len, seq_len, table, ref, page):
    cols = torch.arange(table.shape[1], device=table.device)
    gone = (cols >= ((new_len + page - 1) // page)[:, None]) & (table >= 0) & (new_len >= 0)[:, None]
    ref.scatter_add_(0, table.clamp(min=0).long().flatten(), -gone.int().flatten())
    table.masked_fill_(gone, -1)
    seq_len.copy_(torch.where(new_len >= 0, new_len, seq_len))


def _plain_fork(src, dst, seq_len, table, ref, page):
    src, dst = src.long(), dst.long()
    cols = torch.arange(table.shape[1], device=table.device)
    used = cols < ((seq_len[src] + page - 1) // page)[:, None]
    rows = torch.where(used, table[src], torch.full_like(table[src], -1))
    ref.scatter_add_(0, rows.clamp(min=0).long().flatten(), used.int().flatten())
    table[dst] = rows
    seq_len[dst] = seq_len[src]


def _plain_reserve(need, seq_len, table, ref, pool):
    B, cols, page = table.shape[0], table.shape[1], pool.shape[2]
    c = torch.arange(cols, device=table.device)
    inside = (c >= (seq_len // page)[:, None]) & (c <= ((seq_len + need - 1) // page)[:, None]) & (need > 0)[:, None]
    held = table >= 0
    old = table.clamp(min=0).long()
    writes = (inside & held).int().flatten()
    row = torch.arange(B, dtype=torch.int32, device=table.device)[:, None].expand(B, cols)
    many = torch.zeros_like(ref).scatter_add_(0, old.flatten(), writes)
    last = torch.full_like(ref, -1).scatter_reduce_(0, old.flatten(), torch.where(writes.bool(), row.flatten(), -1),
                                                    "amax")
    stays = (many >= ref)[old] & (last[old] == row)          # every holder writes: the last one keeps the page
    copied = inside & held & (ref[old] > 1) & ~stays
    fresh = inside & (~held | copied)
    free = torch.argsort((ref > 0).int(), stable=True)        # free pages, lowest first
    rank = (fresh.flatten().cumsum(0) - 1).clamp_(min=0, max=len(ref) - 1).view(B, cols)
    page_of = free[rank]
    slots = torch.arange(page, device=table.device)
    moved = (copied & (c == (seq_len // page)[:, None]))[:, :, None] & (slots < (seq_len % page)[:, None])[:, None]
    b, col, slot = moved.nonzero(as_tuple=True)
    pool[:, page_of[b, col], slot] = pool[:, old[b, col], slot]
    ref.scatter_add_(0, old.flatten(), -copied.int().flatten())
    ref.scatter_add_(0, page_of.flatten(), fresh.int().flatten())
    table.copy_(torch.where(fresh, page_of.int(), table))


def _plain_pages(st):
    page = st["case"]["page"]
    _plain_release(st["drop"], st["seq_len"], st["table"], st["ref"], page)
    _plain_fork(st["src"], st["dst"], st["seq_len"], st["table"], st["ref"], page)
    _plain_reserve(st["need"], st["seq_len"], st["table"], st["ref"], st["pool"])
    return [st["table"], st["ref"], st["seq_len"], st["pool"]]


def _plain_compact(st):
    table, ref, pool = st["table"], st["ref"], st["pool"]
    table.copy_(st["table0"])
    ref.copy_(st["ref0"])
    live = ref > 0
    ids = torch.arange(len(ref), device=ref.device)
    count = live.sum()
    holes, movers = (~live & (ids < count)).nonzero()[:, 0], (live & (ids >= count)).nonzero()[:, 0]
    pool[:, holes] = pool[:, movers]
    to = ids.clone()
    to[movers] = holes
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].int(), table))
    ref[holes] = ref[movers]
    ref[movers] = 0
    return [table, ref, count.int().view(1), pool]


def _plain_path(st):
    pool, table, page = st["pool"], st["table"].long(), st["case"]["page"]
    st["seq_len"].copy_(st["seq_len0"])
    L, n = st["seq_len"].long(), st["n"].long()
    B, N = st["path"].shape
    node = torch.cat([torch.zeros((B, 1), dtype=torch.int64, device=table.device), st["path"][:, :-1].long()], 1)
    i = torch.arange(N, device=table.device)
    b, at = (i <= n[:, None]).nonzero(as_tuple=True)
    node = node[b, at]
    spot = lambda pos: (table[b, pos // page], pos % page)  # noqa: E731
    to = spot(L[b] + at)
    if st["staged"] is not None:
        pool[:, to[0], to[1]] = st["staged"][:, b, node]
    else:
        come = spot(L[b] + node)
        pool[:, to[0], to[1]] = pool[:, come[0], come[1]]
    st["seq_len"].add_(st["n"] + 1)
    return [st["seq_len"], pool]


# --------------------------------------------------------------------------------------------- 64 bits
def _exact_rows(q, k, v, sees):
    """Attention of q [n][heads][D] over k, v [m][kv_heads][D] with sees [n][m], by the definition in 64 bits."""
    n, heads, D = q.shape
    share = heads // k.shape[1]
    out = torch.empty((heads, n, D), dtype=torch.float64, device=q.device)
    lse = torch.empty((heads, n), dtype=torch.float64, device=q.device)
    for h in range(heads):
        a = (q[:, h].double() @ k[:, h // share].double().T) / math.sqrt(D)
        a = a.masked_fill(~sees, -math.inf)
        lse[h] = torch.logsumexp(a, -1)
        out[h] = torch.nan_to_num(torch.exp(a - lse[h][:, None]), nan=0.0) @ v[:, h // share].double()
    return out.transpose(0, 1), lse.T


def exact(case, seed):
    if case["op"] not in ("attention", "prompt"):
        return None  # copies and whole numbers
    st = prepare(case, seed)
    outs, lses = [], []
    if case["op"] == "prompt":
        cq, ck = st["cu_q"].tolist(), st["cu_k"].tolist()
        for b in range(case["B"]):
            q, k, v = st["q"][cq[b]:cq[b + 1]], st["k"][ck[b]:ck[b + 1]], st["v"][ck[b]:ck[b + 1]]
            sees = torch.ones((len(q), len(k)), dtype=torch.bool, device="cuda").tril(len(k) - len(q))
            o, s = _exact_rows(q, k, v, sees)
            outs.append(o)
            lses.append(s)
        res = [torch.cat(outs), torch.cat(lses)]
    else:
        S, page, D, H = case["S"], case["page"], case["head_dim"], case["kv_heads"]
        up = _tree_parents(case["tree"]) if case["tree"] else list(range(-1, S - 1))
        among = torch.zeros((S, S), dtype=torch.bool)
        for i in range(S):
            a = i
            while a >= 0:
                among[i, a] = True
                a = up[a]
        table = st["table"].cpu()
        for b, L in enumerate(st["seq_len"].tolist()):
            total = L if case["staged"] else L + S
            flat = [int(table[b, p // page]) * page + p % page for p in range(total)]
            rows = st["pool"].view(-1, st["pool"].shape[-1])[torch.tensor(flat, dtype=torch.int64, device="cuda")]
            if case["staged"]:
                rows = torch.cat([rows, st["staged"][b]])
            sees = torch.cat([torch.ones((S, L), dtype=torch.bool), among], 1).cuda()
            o, s = _exact_rows(st["q"][b], rows[:, :H * D].view(-1, H, D), rows[:, H * D:].view(-1, H, D), sees)
            outs.append(o)
            lses.append(s)
        res = [torch.stack(outs), torch.stack(lses)]
    return res if case["lse"] else res[:1]


# ------------------------------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op in ("attention", "prompt"):
        heads, kv, D, lens = case["heads"], case["kv_heads"], case["head_dim"], _lengths(case)
        if op == "attention":
            S = case["S"]
            up = _tree_parents(case["tree"]) if case["tree"] else list(range(-1, S - 1))
            depth = [0] * S
            for i in range(S):
                depth[i] = 1 + (depth[up[i]] if up[i] >= 0 else 0)
            rows, keys = case["B"] * S, sum(n + S for n in lens)
            pairs = sum(n * S for n in lens) + case["B"] * sum(depth)
            extra = 4 * sum(_cells(n + S, case["page"]) for n in lens) + 4 * case["B"]
        else:
            rows, keys = sum(lens), sum(n + case["before"] for n in lens)
            pairs = sum(n * case["before"] + n * (n + 1) // 2 for n in lens)
            extra = 8 * (case["B"] + 1)
        nbytes = 2 * (2 * rows * heads * D + 2 * keys * kv * D) + extra + (4 * rows * heads if case["lse"] else 0)
        return {"bytes": nbytes, "flops": 4 * heads * D * pairs}
    if op == "pages":
        page, roots = case["page"], case["B"] // case["fan"]
        lens = _lengths(dict(case, B=roots))
        slots = sum((case["fan"] - 1) * (n % page) for n in lens)
        cells = sum(case["fan"] * _cells(n + case["n"], page) for n in lens)
        return {"bytes": 2 * slots * case["layers"] * case["entry"] + 16 * cells, "flops": 0}
    if op == "compact":
        live = max(1, case["pages"] * case["percent"] // 100)
        moved = live * (case["pages"] - live) / case["pages"]  # expected: the live pages lie anywhere
        return {"bytes": 2 * moved * case["layers"] * case["page"] * case["entry"] + 12 * case["pages"] + 8 * live,
                "flops": 0}
    kept = sum(_accepted(case)) + (case["B"] if case["staged"] else 0)
    return {"bytes": 2 * kept * case["layers"] * case["entry"] + 16 * case["B"], "flops": 0}
