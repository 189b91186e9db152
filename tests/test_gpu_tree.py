"""Attention of drafted trees over dense and paged caches (gqa_decode_tree) vs the 64-bit definition.

The bound is derived in paged_reference.py.  Cache rows past a sequence's end, and pages nobody lists,
hold NaN; rows past a sequence's drafts keep what they held.
"""
import pytest
import torch

import paged_reference as ref

pytestmark = pytest.mark.gpu


def tree_masks(B, n, gen):
    m = torch.zeros((B, n), dtype=torch.int64)
    for b in range(B):
        for j in range(n):
            up = 0 if j == 0 else int(m[b, max(0, j - 1 - int(torch.randint(0, 4, (1,), generator=gen)))])
            bit = up | (1 << j)
            m[b, j] = bit - (1 << 64) if bit >= 1 << 63 else bit
    return m


class Case:
    def __init__(self, B, n, H, G, d, page, lens, counts=None, seed=0, spare=3, M=None):
        gen = torch.Generator().manual_seed(seed)
        self.q = torch.randn((B, n, H, d), generator=gen).to(torch.bfloat16)
        self.seqlens = list(lens)
        self.counts = counts
        ends = [t + (n if counts is None else c) for t, c in zip(lens, counts or [n] * B)]
        self.mask = tree_masks(B, n, gen)
        if page:
            per = [-(-e // page) for e in ends]
            P = sum(per) + spare
            M = M or max(max(per), 1) + 1
            perm = torch.randperm(P, generator=gen).tolist()
            self.table = torch.full((B, M), -1, dtype=torch.int32)
            for b in range(B):
                for i in range(per[b]):
                    self.table[b, i] = perm.pop()
            shape = (P, G, page, d)
        else:
            self.table, shape = None, (B, G, max(ends) + spare, d)
        self.k, self.v = (torch.full(shape, float("nan")).to(torch.bfloat16) for _ in range(2))
        for b, e in enumerate(ends):
            for c in (self.k, self.v):
                rows = torch.randn((e, G, d), generator=gen).to(torch.bfloat16)
                for t in range(e):
                    p, i = ref.place(self.table, page, b, t)
                    c[p, :, i] = rows[t]
        self.scale = d ** -0.5

    def args(self, mask=True):
        i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
        return (self.q.cuda(), self.k.cuda(), self.v.cuda(), i32(self.seqlens)), dict(
            tree_mask=self.mask.cuda() if mask else None, n_draft=i32(self.counts),
            block_table=None if self.table is None else self.table.cuda())


def run(gqa, x, mask=True):
    a, kw = x.args(mask)
    out = torch.full(x.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    gqa.decode_tree(*a, out=out, **kw)
    gqa.get_status()
    return out.cpu()


def compare(got, x, mask=True):
    r, w = ref.decode_tree(x.q, x.k, x.v, x.table, x.seqlens, x.mask if mask else None, x.counts, x.scale)
    inside = ~torch.isnan(r[:, :, 0, 0])
    ref.check(got[inside], r[inside], w[inside])
    assert (got[~inside] == 7.0).all()


@pytest.mark.parametrize("n,H,G,d", [(1, 4, 4, 64), (1, 8, 1, 128), (3, 6, 2, 128), (8, 32, 8, 128), (16, 8, 1, 64),
                                     (17, 8, 1, 128), (64, 2, 2, 64), (64, 4, 1, 128), (64, 7, 1, 64), (5, 40, 1, 64),
                                     (3, 128, 1, 64), (64, 16, 1, 64)])
@pytest.mark.parametrize("page", [0, 16, 48, 64, 256])
def test_shapes_and_pages(gqa, n, H, G, d, page):
    x = Case(3, n, H, G, d, page, [0, 130, 301], seed=n + H + page)
    compare(run(gqa, x), x)


@pytest.mark.parametrize("lens", [[0], [1], [63], [64], [127], [128], [129], [255, 256, 257]])
@pytest.mark.parametrize("n", [1, 2, 64])
def test_ends_around_tile_borders(gqa, lens, n):
    x = Case(len(lens), n, 4, 2, 64, 32, lens, seed=n + lens[0])
    compare(run(gqa, x), x)


@pytest.mark.parametrize("n,H,G", [(16, 4, 1), (64, 4, 1), (64, 16, 1)])
def test_ragged_drafts_and_empty_sequences(gqa, n, H, G):
    counts = [0, 1, n, 3, 0, n // 2, n - 1]
    x = Case(7, n, H, G, 64, 16, [10, 0, 333, 129, 0, 64, 200], counts=counts, seed=n)
    compare(run(gqa, x), x)


def test_no_mask_is_a_chain(gqa):
    x = Case(2, 9, 4, 2, 128, 16, [5, 140], seed=12)
    compare(run(gqa, x, mask=False), x, mask=False)


def test_rows_that_see_nothing_are_zero(gqa):
    x = Case(2, 4, 4, 2, 64, 16, [0, 50], seed=13)
    x.mask[0, 1] = 0
    x.mask[0, 2] = 1 << 40  # only bits past the drafts
    x.mask[1, 3] = 0        # sees the cache alone
    got = run(gqa, x)
    compare(got, x)
    assert (got[0, 1] == 0).all() and (got[0, 2] == 0).all()


@pytest.mark.parametrize("n,H,G,T", [(8, 4, 2, 100), (40, 8, 1, 115), (64, 8, 1, 0), (33, 2, 2, 127)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_drafts_that_no_mask_names_may_hold_anything(gqa, n, H, G, T, value):
    """Padded places of a tree whose K/V were never written."""
    x = Case(2, n, H, G, 64, 16, [T, 300], seed=n + T)
    for b, gone in enumerate(([1, n - 1], [n // 2])):
        clear = ~sum(1 << j for j in gone)
        for i in range(n):
            m = int(x.mask[b, i]) & clear & ((1 << 64) - 1)
            x.mask[b, i] = m - (1 << 64) if m >= 1 << 63 else m
        for j in gone:
            p, r = ref.place(x.table, 16, b, x.seqlens[b] + j)
            x.k[p, :, r] = value
            x.v[p, :, r] = value
    got = run(gqa, x)
    for b, gone in enumerate(([1, n - 1], [n // 2])):
        for j in gone:
            p, r = ref.place(x.table, 16, b, x.seqlens[b] + j)
            x.k[p, :, r] = 0  # (the definition's own 0 * NaN)
            x.v[p, :, r] = 0
    compare(got, x)


def test_no_drafts_at_all_and_the_largest_batch(gqa):
    x = Case(3, 2, 4, 2, 64, 16, [5, 0, 70], counts=[0, 0, 0], seed=31)
    compare(run(gqa, x), x)
    B = 8000
    q = torch.randn((B, 1, 2, 64), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    k, v = (torch.randn((B, 1, 5, 64), generator=torch.Generator().manual_seed(s)).to(torch.bfloat16).cuda()
            for s in (2, 3))
    lens = [b % 5 for b in range(B)]
    got = gqa.decode_tree(q, k, v, torch.tensor(lens, dtype=torch.int32).cuda()).cpu()
    gqa.get_status()
    for b in (0, 1, 4, 3999, 7998, 7999):
        for h in range(2):
            r, w = ref.attend(q[b, :, h].cpu(), k[b, 0, :lens[b] + 1].cpu(), v[b, 0, :lens[b] + 1].cpu(),
                              torch.ones(1, lens[b] + 1, dtype=torch.bool), 64 ** -0.5)
            ref.check(got[b, :, h], r, w)


def test_one_draft_is_a_decode_step(gqa):
    """A single token over a dense cache: what gqa_decode gives over the lengths with that token."""
    x = Case(3, 1, 8, 2, 128, 0, [700, 1, 64], seed=14)
    a, kw = x.args()
    got = gqa.decode_tree(*a, **kw)
    T = x.k.shape[2]
    want = gqa.decode(a[0][:, 0], a[1], a[2], a[3] + 1)
    gqa.get_status()
    assert T > 700
    r, w = ref.decode_tree(x.q, x.k, x.v, None, x.seqlens, None, None, x.scale)
    ref.check(got, r, w)
    ref.check(want, r[:, 0], w[:, 0])


@pytest.mark.parametrize("B,n,H,G,lens", [(1, 8, 8, 1, [9000]), (1, 64, 4, 1, [9000]), (40, 4, 8, 2, None),
                                          (40, 33, 8, 2, None), (600, 1, 2, 1, None)])
def test_cut_and_whole_segments(gqa, B, n, H, G, lens):
    """Segments cut over many CTAs, and many segments to a CTA; the same bits twice."""
    if lens is None:
        gen = torch.Generator().manual_seed(B)
        lens = torch.randint(0, 2000 if B < 100 else 300, (B,), generator=gen).tolist()
    x = Case(B, n, H, G, 64, 64, lens, seed=15)
    got = run(gqa, x)
    assert torch.equal(got, run(gqa, x))
    compare(got, x)


@pytest.mark.parametrize("scale", [1e-3, 4.0])
@pytest.mark.parametrize("n", [4, 64])
def test_large_scores_move_the_maximum(gqa, scale, n):
    x = Case(1, n, 4, 1, 64, 16, [700], seed=16)
    ramp = torch.linspace(0.01, 1, 700 + n)
    for t in range(700 + n):
        p, i = ref.place(x.table, 16, 0, t)
        x.k[p, :, i] = (x.k[p, :, i].float() * ramp[t]).to(torch.bfloat16)
    a, kw = x.args()
    got = gqa.decode_tree(*a, scale=scale, **kw).cpu()
    gqa.get_status()
    r, w = ref.decode_tree(x.q, x.k, x.v, x.table, x.seqlens, x.mask, None, scale)
    # scores up to 2^8 in log2 units: 2^2 times what the bound's fp32 part assumes
    d = (got.double() - r).abs()
    assert (d <= ref.bound(r, w) + 4 * ref.FP32_PART * w).all()


def test_missing_pages_read_as_zeros_and_are_flagged(gqa):
    for bad in (-1, 1 << 20, -(1 << 31)):
        x = Case(2, 4, 4, 2, 64, 32, [100, 200], seed=17)
        x.table[1, 3] = bad
        a, kw = x.args()
        out = gqa.decode_tree(*a, **kw)
        with pytest.raises(gqa.GQAError) as e:
            gqa.get_status()
        assert e.value.code == -9
        r, w = ref.decode_tree(x.q, x.k, x.v, x.table, x.seqlens, x.mask, None, x.scale)
        ref.check(out, r, w)


def test_lengths_out_of_range_are_clamped_and_flagged(gqa):
    x = Case(2, 4, 4, 2, 64, 0, [100, 100], seed=18, spare=0)
    for lens, counts in (([-3, 100], None), ([100, 101], None), ([100, 1 << 30], None), ([10, 10], [5, 4]),
                         ([10, 10], [-1, 4])):
        y = Case(2, 4, 4, 2, 64, 0, [100, 100], seed=18, spare=0)
        y.seqlens, y.counts = lens, counts
        a, kw = y.args()
        gqa.decode_tree(*a, **kw)
        with pytest.raises(gqa.GQAError) as e:
            gqa.get_status()
        assert e.value.code == -7
        y.seqlens = [min(max(t, 0), 100) for t in lens]
        y.counts = None if counts is None else [min(max(c, 0), 4) for c in counts]
        compare(run(gqa, y), y)


def test_graphs_that_share_a_workspace_and_two_streams(gqa):
    xs = [Case(4, 8, 8, 2, 64, 16, [3, 500, 64, 1000], seed=19 + i) for i in range(2)]
    calls = [x.args() for x in xs]
    want = [gqa.decode_tree(*a, **kw) for a, kw in calls]
    ws = torch.empty(gqa.decode_tree_workspace_bytes(4, 8, 8, 2, 64), dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(w) for w in want]
    graphs = []
    for (a, kw), out in zip(calls, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            gqa.decode_tree(*a, workspace=ws, out=out, **kw)
        graphs.append(g)
    for _ in range(5):
        for o in outs:
            o.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[gqa.decode_tree(*a, stream=s, **kw) for _ in range(10)] for (a, kw), s in zip(calls, streams)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(y, w) for y in g)
    gqa.get_status()


@pytest.mark.parametrize("n,H,G,d", [(1, 4, 4, 64), (1, 8, 1, 128), (8, 8, 2, 128), (16, 8, 1, 64), (64, 2, 2, 64),
                                     (64, 4, 1, 128), (33, 7, 1, 64)])
@pytest.mark.parametrize("page", [0, 48])
def test_short_contexts_carry_p_as_two_terms(gqa, n, H, G, d, page):
    """Sequences of at most 256 positions, drafts included."""
    x = Case(5, n, H, G, d, page, [0, 3, 100, 150, 256 - n], seed=n + H + page)
    got = run(gqa, x)
    r, w = ref.decode_tree(x.q, x.k, x.v, x.table, x.seqlens, x.mask, x.counts, x.scale)
    ref.check(got, r, w, split=True)


@pytest.mark.parametrize("n,H,G", [(4, 4, 2), (64, 4, 1), (1, 2, 2)])
@pytest.mark.parametrize("T,at", [(50, 20), (900, 899), (9000, 4000)])
def test_a_row_that_sees_a_score_that_is_not_finite_says_so(gqa, n, H, G, T, at):
    """In whole segments and in ones cut over many CTAs: a visible NaN or +inf score gives NaN, one of
    -inf counts for nothing, and the other heads, rows and sequences are what they were."""
    nan, inf = float("nan"), float("inf")
    for where, value in (("q", nan), ("q", inf), ("cached", nan), ("cached", inf), ("cached", -inf), ("draft", nan)):
        x = Case(2, n, H, G, 64, 64, [T, 70], seed=15)
        if where == "q":
            x.q[0, n // 2, 0, 5] = value
        else:
            p, i = ref.place(x.table, 64, 0, T + n // 2 if where == "draft" else at)
            x.k[p, 0, i, 5] = value
        got = run(gqa, x).double()
        r, w = ref.decode_tree(x.q, x.k, x.v, x.table, x.seqlens, x.mask, x.counts, x.scale)
        assert torch.equal(torch.isnan(got), torch.isnan(r)), (where, value)
        fine = torch.isfinite(r)
        ref.check(got[fine], r[fine], w[fine])


def test_a_workspace_that_overlaps_is_refused(gqa):
    x = Case(2, 4, 4, 2, 64, 16, [5, 40], seed=33)
    a, kw = x.args()
    size = gqa.decode_tree_workspace_bytes(2, 4, 4, 2, 64)
    out = torch.empty(x.q.numel() * 2 + size, dtype=torch.uint8, device="cuda")
    rows = out[:x.q.numel() * 2].view(torch.bfloat16).view(x.q.shape)
    gqa.decode_tree(*a, out=rows, workspace=out[x.q.numel() * 2:], **kw)
    want = rows.clone()
    with pytest.raises(gqa.GQAError) as e:
        gqa.decode_tree(*a, out=rows, workspace=out[x.q.numel() * 2 - 256:], **kw)
    assert e.value.code == -1
    gqa.get_status()
    assert torch.equal(rows, want)
