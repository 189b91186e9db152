"""Rows and pages of a cache: append, compact, reserve, fork, release, against plain lists.

Everything here moves or counts, so every comparison is exact.
"""
import pytest
import torch

import paged_reference as ref

pytestmark = pytest.mark.gpu

I32 = torch.int32


def i32(x):
    return torch.tensor(x, dtype=I32).cuda()


def caches(B, G, d, page, cap, dtype, seed=0):
    """Random caches and a scattered table of full capacity (page 0: dense)."""
    gen = torch.Generator().manual_seed(seed)
    if page:
        M = -(-cap // page)
        P = B * M + 2
        table = torch.randperm(P, generator=gen)[: B * M].reshape(B, M).to(I32)
        shape = (P, G, page, d)
    else:
        table, shape = None, (B, G, cap, d)
    k, v = (torch.randn(shape, generator=gen).to(dtype) for _ in range(2))
    return k, v, table


def same(a, b):
    return torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))


def expect(gqa, code):
    with pytest.raises(gqa.GQAError) as e:
        gqa.get_status()
    assert e.value.code == code
    gqa.get_status()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page,G,d", [(0, 3, 64), (7, 1, 128), (16, 8, 128), (64, 2, 64)])
@pytest.mark.parametrize("lens,counts", [([0], [1]), ([3, 0, 60, 17], [0, 64, 5, 1]), ([10] * 40, [1] * 40)])
def test_append(gqa, dtype, page, G, d, lens, counts):
    B = len(lens)
    k, v, table = caches(B, G, d, page, 80, dtype, seed=B + d)
    gen = torch.Generator().manual_seed(1)
    N = sum(counts)
    kn, vn = (torch.randn((N, G, d), generator=gen).to(dtype) for _ in range(2))
    cu = [sum(counts[:b]) for b in range(B + 1)]
    kd, vd = k.cuda(), v.cuda()
    got = gqa.cache_append(kn.cuda(), vn.cuda(), i32(cu), i32(lens), kd, vd,
                           block_table=None if table is None else table.cuda())
    gqa.get_status()
    for b in range(B):
        for i in range(counts[b]):
            p, r = ref.place(table, page, b, lens[b] + i)
            k[p, :, r], v[p, :, r] = kn[cu[b] + i], vn[cu[b] + i]
    assert same(kd, k) and same(vd, v)
    assert got.tolist() == [t + c for t, c in zip(lens, counts)]


def test_append_without_room_or_page(gqa):
    k, v, table = caches(4, 2, 64, 16, 64, torch.bfloat16, seed=3)
    kn = torch.ones((40, 2, 64), dtype=torch.bfloat16)
    # sequence 1 has no room for its 10 rows; the others are written
    kd, vd = k.cuda(), v.cuda()
    lens = [0, 60, 54, -1]
    got = gqa.cache_append(kn.cuda(), kn.cuda(), i32([0, 10, 20, 30, 40]), i32(lens), kd, vd, block_table=table.cuda())
    expect(gqa, -7)
    assert got.tolist() == [10, 60, 64, -1]
    for b in (0, 2):
        for i in range(10):
            p, r = ref.place(table, 16, b, lens[b] + i)
            k[p, :, r], v[p, :, r] = kn[0], kn[0]
    assert same(kd, k) and same(vd, v)
    # a missing page: its rows are not written
    for bad in (-1, 1 << 30):
        holes = table.clone()
        holes[0, 1] = bad
        gqa.cache_append(kn.cuda(), kn.cuda(), i32([0, 40, 40, 40, 40]), i32([0, 0, 0, 0]), kd, vd,
                         block_table=holes.cuda())
        expect(gqa, -9)
        for i in list(range(16)) + list(range(32, 40)):
            p, r = ref.place(table, 16, 0, i)
            k[p, :, r], v[p, :, r] = kn[0], kn[0]
        assert same(kd, k) and same(vd, v)
    # offsets that fall or leave [0, N] write nothing out of place
    before = kd.clone()
    gqa.cache_append(kn.cuda(), kn.cuda(), i32([0, 41, 20, -3, 1 << 30]), i32([0, 0, 0, 0]), kd, vd,
                     block_table=table.cuda())
    expect(gqa, -7)
    assert same(kd, before.cpu())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page,G,d", [(0, 2, 64), (5, 3, 128), (16, 8, 128), (64, 1, 64)])
@pytest.mark.parametrize("m", [1, 7, 64])
def test_compact(gqa, dtype, page, G, d, m):
    B = 6
    gen = torch.Generator().manual_seed(m)
    lens = [0, 1, 15, 16, 63, 30]
    k, v, table = caches(B, G, d, page, 128, dtype, seed=m + d)
    keep = torch.randint(0, 64, (B, m), generator=gen).to(I32)  # any order, repeated entries
    keep[1] = torch.arange(m)                                   # nothing moves
    keep[2] = torch.randperm(64, generator=gen)[:m].sort().values
    n_keep = [m, m, m // 2, 0, 1, m]
    for counts in (n_keep, None):
        kd, vd = k.cuda(), v.cuda()
        got = gqa.cache_compact(kd, vd, i32(lens), keep.cuda(), n_keep=None if counts is None else i32(counts),
                                block_table=None if table is None else table.cuda())
        gqa.get_status()
        wk, wv = k.clone(), v.clone()
        for b in range(B):
            c = m if counts is None else counts[b]
            for j in range(c):
                p0, r0 = ref.place(table, page, b, lens[b] + int(keep[b, j]))
                p1, r1 = ref.place(table, page, b, lens[b] + j)
                wk[p1, :, r1], wv[p1, :, r1] = k[p0, :, r0], v[p0, :, r0]
        assert same(kd, wk) and same(vd, wv)
        assert got.tolist() == [t + (m if counts is None else c) for t, c in zip(lens, counts or [m] * B)]


def test_compact_skips_what_it_cannot_do(gqa):
    k, v, table = caches(5, 2, 64, 16, 64, torch.bfloat16, seed=5)
    kd, vd = k.cuda(), v.cuda()
    keep = i32([[3, 1], [64, 0], [0, -1], [2, 5], [1, 2]])
    lens = [10, 10, 10, 60, -2]
    got = gqa.cache_compact(kd, vd, i32(lens), keep, block_table=table.cuda())
    expect(gqa, -7)
    assert got.tolist() == [12, 10, 10, 60, -2]
    wk = k.clone()
    for j, f in enumerate((3, 1)):
        p0, r0 = ref.place(table, 16, 0, 10 + f)
        p1, r1 = ref.place(table, 16, 0, 10 + j)
        wk[p1, :, r1] = k[p0, :, r0]
    assert same(kd, wk)
    holes = table.clone()
    holes[0, 1] = -1
    kd, vd = k.cuda(), v.cuda()
    got = gqa.cache_compact(kd, vd, i32([10] * 5), i32([[6, 7]] * 5), n_keep=i32([2, 0, 0, 0, 0]),
                            block_table=holes.cuda())
    expect(gqa, -9)
    assert got.tolist() == [10] * 5 and same(kd, k)
    got = gqa.cache_compact(kd, vd, i32([10] * 5), i32([[6, 7]] * 5), n_keep=i32([3, -1, 0, 0, 0]),
                            block_table=table.cuda())
    expect(gqa, -7)
    assert got.tolist() == [10] * 5 and same(kd, k)


class Both:
    """A pool on the device and on lists."""

    def __init__(self, gqa, rows, live, page, M, P, G=2, d=64, dtype=torch.bfloat16, seed=0):
        gen = torch.Generator().manual_seed(seed)
        perm = torch.randperm(P, generator=gen).tolist()
        table, ref_ = [[-1] * M for _ in range(rows)], [0] * P
        T = live + [0] * (rows - len(live))
        for b, t in enumerate(T):
            for i in range(-(-t // page)):
                table[b][i] = perm.pop()
                ref_[table[b][i]] = 1
        self.gqa, self.page = gqa, page
        self.want = ref.Pool(table, ref_, T, page)
        self.k, self.v = (torch.randn((P, G, page, d), generator=gen).to(dtype) for _ in range(2))
        self.kd, self.vd = self.k.cuda(), self.v.cuda()
        self.table, self.ref, self.T = i32(table), i32(ref_), i32(T)

    def release(self, lengths):
        self.gqa.pages_release(self.table, self.ref, i32(lengths), page_size=self.page)
        self.want.release(lengths)

    def fork(self, src, dst):
        self.gqa.pages_fork(self.table, self.ref, self.T, i32(src), i32(dst), page_size=self.page)
        self.want.fork(src, dst)

    def reserve(self, new):
        self.gqa.pages_reserve(self.table, self.ref, self.T, i32(new), self.kd, self.vd)
        self.want.reserve(new)
        for e, p, rows in self.want.copies:
            self.k[p, :, :rows], self.v[p, :, :rows] = self.k[e, :, :rows], self.v[e, :, :rows]
        self.want.copies = []

    def check(self):
        assert self.table.tolist() == self.want.table
        assert self.ref.tolist() == self.want.ref
        assert self.T.tolist() == self.want.T
        assert same(self.kd, self.k) and same(self.vd, self.v)


@pytest.mark.parametrize("page", [16, 7, 64])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_beam_steps(gqa, page, dtype):
    """Rounds of fork, reserve, grow and release, as a beam search makes them."""
    x = Both(gqa, 12, [5, 64, 33, 128], page, 40, 400, dtype=dtype, seed=page)
    for step in range(4):
        x.fork([0, 0, 1, 2, 3, 3], [4, 5, 6, 7, 8, 9])
        x.check()
        new = [1, 3, 17, 0, 2, 40, 1, 1, 1, 16, 0, 0]
        x.reserve(new)
        x.check()
        grown = [t + n for t, n in zip(x.want.T, new)]
        x.T.copy_(i32(grown))
        x.want.T = grown
        x.release([grown[0], 20 + step, grown[2], grown[3], 0, 0, 0, 0, 0, 0, 0, 0])
        x.T[1], x.want.T[1] = 20 + step, 20 + step
        x.T[4:10] = 0
        x.want.T[4:10] = [0] * 6
        x.check()
    gqa.get_status()


def test_reserve_after_a_cut_into_a_shared_page(gqa):
    """Two rows share pages; one is cut back into the middle of a shared page and writes on."""
    x = Both(gqa, 3, [70], 16, 8, 30, seed=1)
    x.fork([0], [1])
    x.release([70, 37, 0])
    x.T[1], x.want.T[1] = 37, 37
    x.reserve([0, 20, 0])
    x.check()
    assert x.want.table[1][:2] == x.want.table[0][:2] and x.want.table[1][2] != x.want.table[0][2]
    gqa.get_status()


@pytest.mark.parametrize("per_row", [300, 400])
def test_reserve_large_and_long(gqa, per_row):
    """Many rows, many pages: several steps of the free-page scan, prompts of hundreds of pages.  The
    rows need about 264,000 pages: too many for a pool of 300 a row, and nothing changes then."""
    gen = torch.Generator().manual_seed(2)
    live = torch.randint(0, 300, (700,), generator=gen).tolist()
    x = Both(gqa, 800, live, 1, 700, per_row * 800, G=1, seed=3)
    x.reserve(torch.randint(0, 400, (800,), generator=gen).tolist())
    x.check()
    assert x.want.flagged == (per_row == 300)
    if x.want.flagged:
        expect(gqa, -9)
    gqa.get_status()


def test_reserve_all_or_nothing(gqa):
    x = Both(gqa, 3, [16, 16], 16, 4, 6, seed=4)
    x.reserve([40, 33, 0])  # six pages, four are free
    x.check()
    expect(gqa, -9)
    x.reserve([33, 1, 0])   # exactly four
    x.check()
    gqa.get_status()


def test_reserve_ranges_and_bad_entries(gqa):
    x = Both(gqa, 4, [16, 16, 5], 16, 3, 20, seed=5)
    x.reserve([33, 3, -1, 48])  # beyond capacity, fine, negative, the whole row
    x.check()
    expect(gqa, -7)
    x = Both(gqa, 3, [20, 20, 20], 16, 3, 20, seed=6)
    x.table[0, 1], x.want.table[0][1] = 999, 999          # out of range: replaced
    x.ref[x.want.table[1][1]] = 0                           # listed but not counted: replaced
    x.want.ref[x.want.table[1][1]] = 0
    x.reserve([1, 1, 1])
    x.check()
    expect(gqa, -9)


def test_fork_refuses_what_clashes(gqa):
    x = Both(gqa, 10, [40, 17, 8], 16, 4, 30, seed=7)
    x.want.table[2][0], x.table[2, 0] = 77, 77             # row 2's page is out of range
    x.fork([0, 1, 0, 1, 9, -1, 0, 10, 2, 3], [4, 5, 4, 1, 0, 6, 2, 7, 8, 9])
    x.check()
    expect(gqa, -9)
    # rows 0 and 1 are also some pair's dst there: no pair may run
    assert all(x.want.table[b] == [-1] * 4 for b in range(3, 10))
    x.fork([0, 1, 0, 9, -1, 10, 2, 3, 1], [4, 5, 4, 3, 6, 7, 8, 9, 7])
    x.check()
    expect(gqa, -9)
    assert x.want.table[4][:3] == x.want.table[0][:3] and x.want.table[5][:2] == x.want.table[1][:2]
    assert x.want.table[8] == [-1] * 4 and x.want.table[3] == [-1] * 4


def test_release_flags_bad_entries(gqa):
    x = Both(gqa, 3, [40, 17, 8], 16, 4, 30, seed=8)
    x.want.table[0][3], x.table[0, 3] = 1000, 1000
    x.want.ref[x.want.table[1][1]], x.ref[x.want.table[1][1]] = 0, 0
    x.release([16, 0, -4])
    x.check()
    expect(gqa, -9)
    x.release([0, 0, 1 << 30])
    x.check()
    gqa.get_status()


def test_a_pool_step_replays(gqa):
    """Release, fork and reserve captured once and replayed: the lists after as many steps."""
    x = Both(gqa, 6, [21, 40], 16, 8, 64, seed=9)
    hold, src, dst, new = [21, 40, 0, 0, 0, 0], [0, 0, 1, 1], [2, 3, 4, 5], [5, 1, 2, 3, 30, 6]
    dev = [i32(v) for v in (hold, src, dst, new)]
    ws = torch.empty(int(gqa.lib.gqa_pages_reserve_workspace_bytes(6, 64)), dtype=torch.uint8, device="cuda")

    def step():
        gqa.pages_release(x.table, x.ref, dev[0], page_size=16)
        gqa.pages_fork(x.table, x.ref, x.T, dev[1], dev[2], page_size=16)
        gqa.pages_reserve(x.table, x.ref, x.T, dev[3], x.kd, x.vd, workspace=ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(6):
        graph.replay()
        x.want.release(hold)
        x.want.fork(src, dst)
        x.want.reserve(new)
        for e, p, rows in x.want.copies:
            x.k[p, :, :rows], x.v[p, :, :rows] = x.k[e, :, :rows], x.v[e, :, :rows]
        x.want.copies = []
    torch.cuda.synchronize()
    x.check()
    gqa.get_status()


def broken(counts, N, gen, spots):
    """Offsets of these counts with `spots` entries replaced by anything from -2 to N + 2."""
    cu = [sum(counts[:b]) for b in range(len(counts) + 1)]
    for _ in range(spots):
        at = int(torch.randint(0, len(cu), (1,), generator=gen))
        cu[at] = int(torch.randint(-2, N + 3, (1,), generator=gen))
    return cu


@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("cu,lens", [([0, 40, 20], [3, 5]), ([0, 10, 5, 15], [0, 1, 2]), ([20, 0, 40], [0, 0]),
                                     (5, None), (70, None), (300, None)])
def test_append_offsets_that_fall(gqa, page, cu, lens):
    """A sequence is served, all its rows and its length, unless its own range is bad or begins below an
    earlier offset; no length counts a row that was not written."""
    G, d, cap = 2, 64, 80
    gen = torch.Generator().manual_seed(1 if lens else cu)
    trials = [(cu, lens)]
    if lens is None:
        trials = []
        for spots in (1, 2, 3, 8):
            counts = torch.randint(0, 9, (cu,), generator=gen).tolist()
            trials.append((broken(counts, sum(counts), gen, spots),
                           torch.randint(0, cap - 4, (cu,), generator=gen).tolist()))
    for offsets, T in trials:
        B = len(T)
        N = max(1, min(max(offsets), 2000))
        k, v, table = caches(B, G, d, page, cap, torch.bfloat16, seed=B)
        kn, vn = (torch.randn((N, G, d), generator=gen).to(torch.bfloat16) for _ in range(2))
        kd, vd = k.cuda(), v.cuda()
        got = gqa.cache_append(kn.cuda(), vn.cuda(), i32(offsets), i32(T), kd, vd,
                               block_table=None if table is None else table.cuda())
        want, bad = list(T), False
        for b in range(B):
            lo, hi = offsets[b], offsets[b + 1]
            if not (0 <= lo <= hi <= N and lo >= max(offsets[:b + 1]) and T[b] + hi - lo <= cap):
                bad = True
                continue
            want[b] += hi - lo
            for i in range(hi - lo):
                p, r = ref.place(table, page, b, T[b] + i)
                k[p, :, r], v[p, :, r] = kn[lo + i], vn[lo + i]
        assert got.tolist() == want
        assert same(kd, k) and same(vd, v)
        if bad:
            expect(gqa, -7)
        gqa.get_status()


def test_fork_of_a_page_that_nobody_holds(gqa):
    """Row 1 lists a page whose count is 0: its pair is skipped and flagged, the others run, and no page
    ends with fewer references than rows that list it."""
    x = Both(gqa, 7, [40, 40, 17], 16, 4, 30, seed=10)
    lost = x.want.table[1][2]
    x.ref[lost] = 0
    before = x.table.clone()
    counts = x.ref.clone()
    gqa.pages_fork(x.table, x.ref, x.T, i32([0, 1, 1, 2]), i32([3, 4, 5, 6]), page_size=16)
    expect(gqa, -9)
    for a, z in ((0, 3), (2, 6)):
        held = -(-x.want.T[a] // 16)
        before[z, :held] = before[a, :held]
        counts[before[a, :held].long()] += 1
        x.want.T[z] = x.want.T[a]
    assert torch.equal(x.table, before) and torch.equal(x.ref, counts) and x.T.tolist() == x.want.T


def test_append_of_no_rows(gqa):
    k, v, table = caches(3, 2, 64, 16, 64, torch.bfloat16, seed=6)
    kn = torch.ones((5, 2, 64), dtype=torch.bfloat16)
    kd, vd = k.cuda(), v.cuda()
    for cu in ([0, 0, 0, 0], [5, 5, 5, 5], [2, 2, 2, 2]):
        got = gqa.cache_append(kn.cuda(), kn.cuda(), i32(cu), i32([0, 64, 7]), kd, vd, block_table=table.cuda())
        assert got.tolist() == [0, 64, 7] and same(kd, k) and same(vd, v)
    gqa.get_status()


@pytest.mark.parametrize("page", [0, 16])
def test_rows_on_another_stream_and_replayed(gqa, page):
    """Append and compact queued on a side stream, with lengths that they allocate, and captured: each
    replay takes the lengths that it finds."""
    B, G, d = 3, 2, 64
    k, v, table = caches(B, G, d, page, 96, torch.bfloat16, seed=11)
    gen = torch.Generator().manual_seed(12)
    kn, vn = (torch.randn((12, G, d), generator=gen).to(torch.bfloat16) for _ in range(2))
    cu, lens, keep, n_keep = [0, 5, 6, 12], [3, 40, 15], [[0, 2, 4], [0, 0, 0], [5, 1, 3]], [3, 1, 2]
    bt = None if table is None else table.cuda()
    args = kn.cuda(), vn.cuda(), i32(cu)
    T, kp, nk = i32(lens), i32(keep), i32(n_keep)

    def step(kd, vd, T, stream=None):
        gqa.cache_append(*args, T, kd, vd, block_table=bt, stream=stream)
        return gqa.cache_compact(kd, vd, T, kp, n_keep=nk, block_table=bt, stream=stream)

    def model(T):
        for b in range(B):
            for i in range(cu[b + 1] - cu[b]):
                p, r = ref.place(table, page, b, T[b] + i)
                k[p, :, r], v[p, :, r] = kn[cu[b] + i], vn[cu[b] + i]
            rows = [ref.place(table, page, b, T[b] + j) for j in keep[b][:n_keep[b]]]
            was = [(k[p, :, r].clone(), v[p, :, r].clone()) for p, r in rows]
            for j, (x, y) in enumerate(was):
                p, r = ref.place(table, page, b, T[b] + j)
                k[p, :, r], v[p, :, r] = x, y
        return [t + c for t, c in zip(T, n_keep)]

    kd, vd = k.cuda(), v.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(kd, vd, T, side)
    side.synchronize()
    lens = model(lens)
    assert got.tolist() == lens and same(kd, k) and same(vd, v)
    T.copy_(got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(kd, vd, T)
    for _ in range(4):
        graph.replay()
        T.copy_(got)
        lens = model(lens)
        assert T.tolist() == lens and same(kd, k) and same(vd, v)
    gqa.get_status()


def test_pool_calls_on_another_stream(gqa):
    x = Both(gqa, 4, [21, 40], 16, 6, 40, seed=13)
    side = torch.cuda.Stream()
    hold, src, dst, new = i32([21, 33, 0, 0]), i32([0, 1]), i32([2, 3]), i32([1, 2, 3, 20])
    side.wait_stream(torch.cuda.current_stream())
    gqa.pages_release(x.table, x.ref, hold, page_size=16, stream=side)
    gqa.pages_fork(x.table, x.ref, x.T, src, dst, page_size=16, stream=side)
    gqa.pages_reserve(x.table, x.ref, x.T, new, x.kd, x.vd, stream=side)
    side.synchronize()
    x.want.release([21, 33, 0, 0])
    x.want.fork([0, 1], [2, 3])
    x.want.reserve([1, 2, 3, 20])
    for e, p, rows in x.want.copies:
        x.k[p, :, :rows], x.v[p, :, :rows] = x.k[e, :, :rows], x.v[e, :, :rows]
    x.check()
    gqa.get_status()
