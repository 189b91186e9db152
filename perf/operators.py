"""What is measured of the packed-prompt, draft-tree and paged-cache operators.

A serving program holds its K/V cache as pages [P, G, page, d_h] that block
tables hand out to sequences.  Per prompt batch it attends over the packed
prompts and writes their K/V into pages; per speculative step it reserves
pages, appends the drafted tokens' K/V, scores the drafted tree against the
cache, and keeps the accepted path; per beam step it drops the beams that
lost, forks the ones that won and makes the pages they are about to write
their own.

Cases are dicts of plain values; "op" says which operator a case runs:
  prefill  causal attention over packed prompts of different lengths
  tree     attention of a tree of drafted tokens over a paged (page > 0) or
           dense (page = 0) cache; n = 1 is the single-token step
  append   new K/V rows into the pages (or the dense cache)
  compact  the accepted path's rows moved to the front of the drafted ones
  pages    one beam step of the page pool: release, fork, reserve with
           copy-on-write
Lengths follow from the case alone (seqs, lo, hi, mix); values from the seed.
"""
from __future__ import annotations

import math
import random

import torch

own = False

BF16 = torch.bfloat16


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a handful of chat turns arriving together: launch latency counts
        dict(name="prefill_chat_turns", op="prefill", seqs=4, lo=5, hi=211, mix=1, H=32, G=8, d=128, window=0),
        # many short prompts, three query heads per group, d_h 64
        dict(name="prefill_many_short", op="prefill", seqs=96, lo=1, hi=700, mix=2, H=24, G=8, d=64, window=0),
        # documents with short prompts between them: the compute-bound end
        dict(name="prefill_documents", op="prefill", seqs=4, lo=1900, hi=8192, mix=3, H=32, G=8, d=128, window=0),
        # one conversation verifying a small tree
        dict(name="tree_one_chat", op="tree", seqs=1, lo=777, hi=777, mix=4, n=8, ragged=False, page=16, H=32, G=8,
             d=128),
        # a serving batch, 16 drafts a sequence over ragged lengths (128 query rows per KV head)
        dict(name="tree_batch", op="tree", seqs=32, lo=1024, hi=8192, mix=5, n=16, ragged=True, page=64, H=64, G=8,
             d=128),
        # long contexts, the widest tree (256 query rows per KV head), dense cache
        dict(name="tree_long_context", op="tree", seqs=4, lo=131000, hi=131000, mix=6, n=64, ragged=False, page=0,
             H=32, G=8, d=128),
        # drafts of a batch appended: small and scattered
        dict(name="append_drafts", op="append", seqs=32, lo=1024, hi=4096, mix=7, new_lo=1, new_hi=16, page=16, G=8,
             d=128, f32=False),
        # prompts appended after prefill: bandwidth
        dict(name="append_prompts", op="append", seqs=24, lo=0, hi=0, mix=8, new_lo=200, new_hi=8000, page=64, G=8,
             d=128, f32=False),
        # accepted paths of a batch kept
        dict(name="compact_batch", op="compact", seqs=32, lo=1024, hi=4096, mix=9, m=16, page=16, G=8, d=128,
             f32=False),
        # many sequences and wide trees
        dict(name="compact_wide", op="compact", seqs=256, lo=100, hi=2048, mix=10, m=64, page=64, G=8, d=128,
             f32=False),
        # four beams each for a few requests
        dict(name="pages_few_beams", op="pages", seqs=4, forks=12, lo=100, hi=900, mix=11, new=1, page=16, spare=64,
             G=8, d=128, f32=False),
        # a full pool: 128 requests forked into two beams each, long tables
        dict(name="pages_full_pool", op="pages", seqs=128, forks=128, lo=500, hi=3000, mix=12, new=24, page=16,
             spare=2000, G=8, d=128, f32=False),
    ]


def draw(rng):
    def logint(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))

    op = rng.choice(["prefill", "prefill", "tree", "tree", "tree", "append", "compact", "pages"])
    d = rng.choice([64, 128])
    G = rng.choice([1, 2, 4, 8, 8])
    c = dict(op=op, mix=rng.randrange(1 << 20), G=G, d=d)
    if op == "prefill":
        r = rng.choice([1, 2, 3, 4, 5, 7, 8])
        hi = logint(8, 4096)
        c.update(seqs=logint(1, max(1, min(64, 16384 // hi))), lo=rng.choice([0, 1, max(1, hi // 8)]), hi=hi, H=G * r,
                 window=rng.choice([0, 0, logint(1, 2048)]))
    elif op == "tree":
        r = rng.choice([1, 2, 3, 4, 6, 8, 16])
        hi = logint(16, 32768)
        c.update(seqs=logint(1, max(1, min(64, 131072 // hi))), lo=rng.choice([0, 1, max(1, hi // 8)]), hi=hi,
                 n=rng.choice([1, 1, 2, 5, 8, 13, 16, 32, 64]), ragged=rng.random() < 0.5, H=G * r,
                 page=rng.choice([0, 16, 32, 64, 128, 256]))
    elif op == "append":
        hi = logint(16, 4096)
        new = logint(1, 4000)
        c.update(seqs=logint(1, max(1, min(64, 65536 // max(hi, new)))), lo=0, hi=hi, new_lo=0, new_hi=new,
                 page=rng.choice([0, 16, 32, 64, 128]), f32=rng.random() < 0.25)
    elif op == "compact":
        hi = logint(16, 4096)
        c.update(seqs=logint(1, max(1, min(256, 262144 // hi))), lo=0, hi=hi, m=rng.choice([1, 3, 8, 16, 40, 64]),
                 page=rng.choice([0, 16, 32, 64, 128]), f32=rng.random() < 0.25)
    else:
        hi = logint(16, 4096)
        seqs = logint(1, max(1, min(64, 131072 // hi)))
        c.update(seqs=seqs, forks=logint(1, 64), lo=1, hi=hi, new=rng.choice([1, 5, 16, 64]),
                 page=rng.choice([16, 32, 64]), spare=logint(1, 4000), f32=rng.random() < 0.25)
    return c


def spread(case, lo, hi, count, salt=0):
    """`count` lengths in [lo, hi], the largest among them, spread over their logarithm."""
    rng = random.Random(case["mix"] * 7919 + salt)
    got = [hi] + [int(math.exp(rng.uniform(math.log(lo + 1), math.log(hi + 2)))) - 1 for _ in range(count - 1)]
    got = [max(lo, min(hi, x)) for x in got]
    rng.shuffle(got)
    return got


def lengths(case):
    return spread(case, case["lo"], case["hi"], case["seqs"])


def draft_counts(case):
    n, B = case["n"], case["seqs"]
    return spread(case, 1, n, B, 1) if case["ragged"] else [n] * B


def new_counts(case):
    return spread(case, case["new_lo"], case["new_hi"], case["seqs"], 2)


def keep_counts(case):
    return spread(case, 0, case["m"], case["seqs"], 3)


def fork_sources(case):
    """Which of the live sequences each fork copies (fork i goes to row seqs + i)."""
    return [i % case["seqs"] for i in range(case["forks"])]


# ------------------------------------------------------------------ inputs

def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cu(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return _ints(at)


def _pool(case, need, gen, dtype):
    """K, V pools and a block table whose row b lists enough pages for need[b] positions, in random
    order over the pool (page = 0: a dense cache [B, G, T_cap, d_h] and no table)."""
    B, G, d, page = len(need), case["G"], case["d"], case["page"]
    if page == 0:
        shape, table = (B, G, max(need), d), None
    else:
        per = [-(-x // page) for x in need]
        total = sum(per)
        pages = total + total // 8 + 1
        perm = torch.randperm(pages, generator=gen, device="cuda")[:total].to(torch.int32)
        table = torch.full((B, max(max(per), 1)), -1, dtype=torch.int32, device="cuda")
        where = torch.arange(table.shape[1], device="cuda")[None] < torch.tensor(per, device="cuda")[:, None]
        table[where] = perm
        shape = (pages, G, page, d)
    k = torch.randn(shape, generator=gen, device="cuda", dtype=dtype)
    v = torch.randn(shape, generator=gen, device="cuda", dtype=dtype)
    return k, v, table


def _tree_masks(B, n, gen):
    """Ancestor bit masks [B, n] of random trees: node 0 is the root, node j hangs under one of the
    few nodes before it; bit i of mask j says that j sees i (itself among them)."""
    back = torch.randint(1, 5, (B, n), generator=gen, device="cuda")
    masks = torch.ones((B, n), dtype=torch.int64, device="cuda")
    for j in range(1, n):
        parent = (j - back[:, j]).clamp(min=0)
        masks[:, j] = masks.gather(1, parent[:, None])[:, 0] | (torch.ones_like(parent) << j)
    return masks


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    G, d = case["G"], case["d"]

    def randn(*shape, dtype=BF16):
        return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)

    lens = lengths(case)
    s = dict(op=op, case=dict(case))
    if op == "prefill":
        N = max(1, sum(lens))
        s.update(q=randn(N, case["H"], d), k=randn(N, G, d), v=randn(N, G, d), cu=_cu(lens), scale=1 / math.sqrt(d),
                 longest=max(1, max(lens)), out=torch.zeros((N, case["H"], d), dtype=BF16, device="cuda"))
    elif op == "tree":
        B, n = case["seqs"], case["n"]
        k, v, table = _pool(case, [t + n for t in lens], gen, BF16)
        s.update(q=randn(B, n, case["H"], d), k=k, v=v, table=table, seqlens=_ints(lens), masks=_tree_masks(B, n, gen),
                 counts=_ints(draft_counts(case)) if case["ragged"] else None, scale=1 / math.sqrt(d),
                 longest=max(lens) + n, out=torch.zeros((B, n, case["H"], d), dtype=BF16, device="cuda"))
    elif op == "append":
        dtype = torch.float32 if case["f32"] else BF16
        counts = new_counts(case)
        N = max(1, sum(counts))
        k, v, table = _pool(case, [max(1, t + n) for t, n in zip(lens, counts)], gen, dtype)
        s.update(k_new=randn(N, G, d, dtype=dtype), v_new=randn(N, G, d, dtype=dtype), cu=_cu(counts), k=k, v=v,
                 table=table, seqlens=_ints(lens))
    elif op == "compact":
        dtype = torch.float32 if case["f32"] else BF16
        B, m = case["seqs"], case["m"]
        k, v, table = _pool(case, [t + 64 for t in lens], gen, dtype)
        # ascending draft indices, as a root-to-leaf path has them
        order = torch.rand((B, 64), generator=gen, device="cuda").argsort(1)[:, :m].sort(1).values.to(torch.int32)
        s.update(k=k, v=v, table=table, seqlens=_ints(lens), keep=order.contiguous(), n_keep=_ints(keep_counts(case)))
    else:
        dtype = torch.float32 if case["f32"] else BF16
        B, F, page, new = case["seqs"], case["forks"], case["page"], case["new"]
        rows = B + F
        held = [-(-t // page) for t in lens]
        src = fork_sources(case)
        tails = 2 * (rows + 1) + sum(-(-(lens[b] + new) // page) - lens[b] // page for b in list(range(B)) + src)
        pages = sum(held) + tails + case["spare"]
        table = torch.full((rows, max(-(-(t + new) // page) for t in lens)), -1, dtype=torch.int32, device="cuda")
        perm = torch.randperm(pages, generator=gen, device="cuda")[:sum(held)].to(torch.int32)
        where = torch.arange(table.shape[1], device="cuda")[None] < torch.tensor(held + [0] * F, device="cuda")[:, None]
        table[where] = perm
        refcount = torch.zeros(pages, dtype=torch.int32, device="cuda")
        refcount[perm.long()] = 1
        s.update(k=randn(pages, G, page, d, dtype=dtype), v=randn(pages, G, page, d, dtype=dtype), table=table,
                 refcount=refcount, seqlens=_ints(lens + [0] * F), n_new=_ints([new] * rows),
                 hold=_ints(lens + [0] * F), src=_ints(src), dst=_ints(list(range(B, rows))))
    return s


# ------------------------------------------------------------------ the operators, plainly

def _plain_prefill(s):
    q, k, v, cu = s["q"], s["k"], s["v"], s["cu"].long()
    (N, H, d), G, L, w = q.shape, k.shape[1], s["longest"], s["case"]["window"]
    at = torch.arange(L, device="cuda")
    lens = cu[1:] - cu[:-1]
    inside = at[None] < lens[:, None]                                   # [B, L]
    rows = (cu[:-1, None] + at[None]).clamp(max=N - 1)                  # padded batch of the packed rows
    Q = q[rows].float().unflatten(2, (G, H // G)).permute(0, 2, 3, 1, 4)  # [B, G, r, L, d]
    K = k[rows].float().permute(0, 2, 3, 1)[:, :, None]                 # [B, G, 1, d, L]
    V = v[rows].float().permute(0, 2, 1, 3)[:, :, None]                 # [B, G, 1, L, d]
    p = torch.matmul(Q, K).mul_(s["scale"])
    hidden = (at[None] > at[:, None]) | ((at[None] <= at[:, None] - w) if w else False)
    p.masked_fill_(hidden[None, None, None] | ~inside[:, None, None, None], -math.inf)
    p.sub_(p.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    o = torch.matmul(p, V) / p.sum(-1, keepdim=True)
    out = s["out"]
    out[rows[inside]] = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[inside].to(out.dtype)
    return out


def _rows_of(table, page, b, pos):
    """(page, row) of position pos of sequence b; a dense cache is one page per sequence."""
    if table is None:
        return b, pos
    return table.long()[b, pos // page], pos % page


def _gathered(cache, table, L):
    """Positions 0..L-1 of every sequence as [B, G, L, d] in 32 bits."""
    if table is None:
        return cache[:, :, :L].float()
    x = cache[table.long().clamp(min=0)]                                # [B, M, G, page, d]
    return x.transpose(1, 2).flatten(2, 3)[:, :, :L].float()


def _plain_tree(s):
    q, T, masks = s["q"], s["seqlens"].long(), s["masks"]
    (B, n, H, d), G, L = q.shape, s["k"].shape[1], s["longest"]
    Q = q.float().unflatten(2, (G, H // G)).permute(0, 2, 1, 3, 4).flatten(2, 3)      # [B, G, n r, d]
    K, V = _gathered(s["k"], s["table"], L), _gathered(s["v"], s["table"], L)
    rel = torch.arange(L, device="cuda")[None] - T[:, None]                           # [B, L]
    bit = (masks[:, :, None] >> rel.clamp(0, 63)[:, None]) & 1                        # [B, n, L]
    sees = (rel[:, None] < 0) | ((rel[:, None] < n) & (bit != 0))
    p = torch.matmul(Q, K.transpose(2, 3)).mul_(s["scale"]).unflatten(2, (n, H // G))
    p.masked_fill_(~sees[:, None, :, None], -math.inf)
    p.sub_(p.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    o = torch.matmul(p.flatten(2, 3), V).unflatten(2, (n, H // G)) / p.sum(-1, keepdim=True)
    o = o.permute(0, 2, 1, 3, 4).flatten(2, 3)                                        # [B, n, H, d]
    if s["counts"] is not None:
        o = torch.where((torch.arange(n, device="cuda")[None] < s["counts"][:, None])[:, :, None, None], o,
                        s["out"].float())
    return o.to(BF16)


def _plain_append(s):
    k, v, cu, T = s["k"], s["v"], s["cu"].long(), s["seqlens"].long()
    tok = torch.arange(s["k_new"].shape[0], device="cuda")
    if int(s["case"]["new_hi"]) == 0:
        return k, v, s["seqlens"] + 0
    b = (tok[:, None] >= cu[None, 1:]).sum(1)
    page, row = _rows_of(s["table"], s["case"]["page"], b, T[b] + tok - cu[b])
    k[page, :, row] = s["k_new"]
    v[page, :, row] = s["v_new"]
    return k, v, (T + cu[1:] - cu[:-1]).to(torch.int32)


def _plain_compact(s):
    k, v, T = s["k"], s["v"], s["seqlens"].long()
    B, m = s["keep"].shape
    j = torch.arange(m, device="cuda")[None].expand(B, m)
    taken = torch.where(j < s["n_keep"][:, None], s["keep"].long(), j)   # the rest stay where they are
    b = torch.arange(B, device="cuda")[:, None].expand(B, m)
    page = s["case"]["page"]
    p0, r0 = _rows_of(s["table"], page, b, T[:, None] + taken)
    p1, r1 = _rows_of(s["table"], page, b, T[:, None] + j)
    k[p1, :, r1] = k[p0, :, r0]
    v[p1, :, r1] = v[p0, :, r0]
    return k, v, s["seqlens"] + s["n_keep"]


def _plain_pages(s):
    k, v, table, ref, T, page = s["k"], s["v"], s["table"], s["refcount"], s["seqlens"], s["case"]["page"]
    M = table.shape[1]
    at = torch.arange(M, device="cuda")[None]
    # release: entries past the pages that the lengths to hold need
    gone = (at >= (s["hold"][:, None] + page - 1) // page) & (table >= 0)
    ref.index_add_(0, table[gone].long(), torch.full_like(table[gone], -1))
    table[gone] = -1
    # fork: the rows dst share the pages of the rows src
    src, dst = s["src"].long(), s["dst"].long()
    T[dst] = T[src]
    got = torch.where(at < (T[src][:, None] + page - 1) // page, table[src], -1)
    table[dst] = got
    ref.index_add_(0, got[got >= 0].long(), torch.ones_like(got[got >= 0]))
    # reserve: positions [T, T + new) become each row's own; lowest free pages, in table order
    lo, hi = T // page, (T + s["n_new"] + page - 1) // page
    inside = (at >= lo[:, None]) & (at < hi[:, None]) & (s["n_new"] > 0)[:, None]
    shared = inside & (table >= 0) & (ref[table.long().clamp(min=0)] > 1)
    takes = inside & (table < 0) | shared
    free = (ref == 0).nonzero()[:, 0].to(torch.int32)
    old = table[shared].long()
    tail = shared & (at == lo[:, None]) & (T % page > 0)[:, None]
    b = tail.nonzero()[:, 0]
    before = table[tail].long()
    new = free[: int(takes.sum())]
    table[takes] = new
    ref[new.long()] = 1
    ref.index_add_(0, old, torch.full_like(s["refcount"][: old.numel()], -1))
    row = torch.arange(page, device="cuda")
    which, r = (row[None] < (T[b] % page)[:, None]).nonzero(as_tuple=True)
    to = table[tail].long()
    k[to[which], :, r] = k[before[which], :, r]
    v[to[which], :, r] = v[before[which], :, r]
    return table, ref, T, k, v


def run(s):
    op = s["op"]
    if not own:
        plain = {"prefill": _plain_prefill, "tree": _plain_tree, "append": _plain_append, "compact": _plain_compact,
                 "pages": _plain_pages}
        return plain[op](s)
    import kv_cache_decode_04_b200 as gqa

    if op == "prefill":
        return gqa.prefill_packed(s["q"], s["k"], s["v"], s["cu"], scale=s["scale"], window=s["case"]["window"],
                                  out=s["out"])
    if op == "tree":
        return gqa.decode_tree(s["q"], s["k"], s["v"], s["seqlens"], tree_mask=s["masks"], n_draft=s["counts"],
                               block_table=s["table"], scale=s["scale"], out=s["out"])
    if op == "append":
        return s["k"], s["v"], gqa.cache_append(s["k_new"], s["v_new"], s["cu"], s["seqlens"], s["k"], s["v"],
                                                block_table=s["table"])
    if op == "compact":
        return s["k"], s["v"], gqa.cache_compact(s["k"], s["v"], s["seqlens"], s["keep"], n_keep=s["n_keep"],
                                                 block_table=s["table"])
    gqa.pages_release(s["table"], s["refcount"], s["hold"], page_size=s["case"]["page"])
    gqa.pages_fork(s["table"], s["refcount"], s["seqlens"], s["src"], s["dst"], page_size=s["case"]["page"])
    gqa.pages_reserve(s["table"], s["refcount"], s["seqlens"], s["n_new"], s["k"], s["v"])
    return s["table"], s["refcount"], s["seqlens"], s["k"], s["v"]


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op, G, d = case["op"], case["G"], case["d"]
    lens = lengths(case)
    B = case["seqs"]
    if op == "prefill":
        H, w, N = case["H"], case["window"], sum(lens)
        pairs = sum(x * (x + 1) // 2 if not w or w >= x else w * (w + 1) // 2 + (x - w) * w for x in lens)
        return {"bytes": 2 * N * d * (2 * H + 2 * G) + 4 * (B + 1), "flops": 4 * H * d * pairs}
    if op == "tree":
        H, counts = case["H"], draft_counts(case)
        keys = sum(t + n for t, n in zip(lens, counts))
        pairs = sum(n * (t + 1) for t, n in zip(lens, counts))
        return {"bytes": 4 * keys * G * d + sum(counts) * (4 * H * d + 8) + 8 * B, "flops": 4 * H * d * pairs}
    size = 4 if case["f32"] else 2
    if op == "append":
        return {"bytes": 4 * size * sum(new_counts(case)) * G * d + 12 * B, "flops": 0}
    if op == "compact":
        kept = sum(keep_counts(case))
        return {"bytes": 4 * size * kept * G * d + 4 * kept + 12 * B, "flops": 0}
    page, new = case["page"], case["new"]
    src = fork_sources(case)
    forked = set(src)
    rows = lens + [lens[i] for i in src]
    shared = [b in forked for b in range(B)] + [True] * len(src)
    copied = sum(t % page for t, f in zip(rows, shared) if f)
    entries = sum(-(-(t + new) // page) for t in rows)
    return {"bytes": 4 * size * copied * G * d + 8 * entries + 4 * entries, "flops": 0}


# ------------------------------------------------------------------ the definitions in 64 bits

def _attend64(q, K, V, sees, scale):
    """softmax over the keys that `sees` [rows, keys] lets through; a row that sees none is zero."""
    x = (q @ K.T) * scale
    x[~sees] = -math.inf
    top = x.max(1, keepdim=True).values
    e = torch.exp(x - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    z = e.sum(1, keepdim=True)
    return (e @ V) / torch.where(z > 0, z, torch.ones_like(z))


def _place(table, page, b, pos):
    return (b, pos) if table is None else (table[b][pos // page], pos % page)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "prefill":
        out = s["out"].double()
        H, r, w, cu = case["H"], case["H"] // case["G"], case["window"], s["cu"].tolist()
        for a, z in zip(cu[:-1], cu[1:]):
            for lo in range(a, z, 1024):
                hi = min(z, lo + 1024)
                i, j = torch.arange(lo, hi, device="cuda")[:, None], torch.arange(a, hi, device="cuda")[None]
                sees = (j <= i) & (j > i - w) if w else j <= i
                for h in range(H):
                    out[lo:hi, h] = _attend64(s["q"][lo:hi, h].double(), s["k"][a:hi, h // r].double(),
                                              s["v"][a:hi, h // r].double(), sees, s["scale"])
        return out
    T = s["seqlens"].tolist()
    page, table = case["page"], None if s["table"] is None else s["table"].tolist()
    if op == "tree":
        out = s["out"].double()
        n, r, counts = case["n"], case["H"] // case["G"], draft_counts(case)
        masks = s["masks"].tolist()
        for b, t in enumerate(T):
            c = counts[b]
            sees = torch.ones((c, t + c), dtype=torch.bool)
            for i in range(c):
                for j in range(c):
                    sees[i, t + j] = bool((masks[b][i] >> j) & 1)
            sees = sees.cuda()
            for g in range(case["G"]):
                if table is None:
                    K, V = s["k"][b, g, : t + c], s["v"][b, g, : t + c]
                else:
                    held = torch.tensor(table[b], device="cuda")
                    held = held[held >= 0]
                    K, V = s["k"][held, g].flatten(0, 1)[: t + c], s["v"][held, g].flatten(0, 1)[: t + c]
                K, V = K.double(), V.double()
                for h in range(g * r, (g + 1) * r):
                    out[b, :c, h] = _attend64(s["q"][b, :c, h].double(), K, V, sees, s["scale"])
        return out
    k, v = s["k"].double(), s["v"].double()
    if op in ("append", "compact"):
        grow, moves = [0] * len(T), []
        if op == "append":
            cu = s["cu"].tolist()
            for b, t in enumerate(T):
                grow[b] = cu[b + 1] - cu[b]
                moves += [(cu[b] + i, _place(table, page, b, t + i)) for i in range(grow[b])]
            if moves:
                src = torch.tensor([m[0] for m in moves], device="cuda")
                at = torch.tensor([m[1] for m in moves], device="cuda")
                k[at[:, 0], :, at[:, 1]] = s["k_new"].double()[src]
                v[at[:, 0], :, at[:, 1]] = s["v_new"].double()[src]
        else:
            keep, grow = s["keep"].tolist(), s["n_keep"].tolist()
            for b, t in enumerate(T):
                moves += [(_place(table, page, b, t + keep[b][j]), _place(table, page, b, t + j)) for j in range(grow[b])]
            if moves:
                a, z = (torch.tensor([m[i] for m in moves], device="cuda") for i in (0, 1))
                k[z[:, 0], :, z[:, 1]] = k[a[:, 0], :, a[:, 1]].clone()
                v[z[:, 0], :, z[:, 1]] = v[a[:, 0], :, a[:, 1]].clone()
        return k, v, torch.tensor([t + n for t, n in zip(T, grow)], dtype=torch.int32)
    # pages, on lists
    ref, hold, new = s["refcount"].tolist(), s["hold"].tolist(), case["new"]
    for b, t in enumerate(hold):
        for i in range(-(-t // page), len(table[b])):
            if table[b][i] >= 0:
                ref[table[b][i]] -= 1
                table[b][i] = -1
    for a, z in zip(s["src"].tolist(), s["dst"].tolist()):
        T[z] = T[a]
        for i in range(-(-T[a] // page)):
            table[z][i] = table[a][i]
            ref[table[a][i]] += 1
    counted, free = list(ref), [p for p, n in enumerate(ref) if n == 0]
    took = 0
    for b, t in enumerate(T):
        for i in range(t // page, -(-(t + new) // page)):
            was = table[b][i]
            if was >= 0 and counted[was] < 2:
                continue
            table[b][i] = free[took]
            ref[free[took]] = 1
            took += 1
            if was >= 0:
                ref[was] -= 1
                if i == t // page and t % page:
                    k[table[b][i], :, : t % page] = k[was, :, : t % page]
                    v[table[b][i], :, : t % page] = v[was, :, : t % page]
    return (torch.tensor(table, dtype=torch.int32), torch.tensor(ref, dtype=torch.int32), torch.tensor(T, dtype=torch.int32),
            k, v)
