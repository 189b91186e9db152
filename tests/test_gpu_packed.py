"""Causal prefill over packed prompts (gqa_prefill_packed) vs the 64-bit definition.

The bound is derived in paged_reference.py; rows of no sequence keep what they held, bit for bit, and
NaN around and between sequences reaches nobody.
"""
import pytest
import torch

import paged_reference as ref

pytestmark = pytest.mark.gpu


def inputs(cu, H, G, d, N=None, seed=0, std=1.0):
    gen = torch.Generator().manual_seed(seed)
    N = N or max(1, cu[-1])
    q, k, v = (torch.randn((N, h, d), generator=gen).mul_(std).to(torch.bfloat16) for h in (H, G, G))
    return q, k, v


def offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def run(gqa, q, k, v, cu, **kw):
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    got = gqa.prefill_packed(q.cuda(), k.cuda(), v.cuda(), torch.tensor(cu, dtype=torch.int32).cuda(), out=out, **kw)
    gqa.get_status()
    assert got is out
    return out.cpu()


def compare(got, r, w, q):
    inside = ~torch.isnan(r[:, 0, 0])
    # rows of at most 128 keys carry P as two terms, but which tile a row is in is the kernel's
    # affair: the one-term bound holds for all
    ref.check(got[inside], r[inside], w[inside])
    assert (got[~inside] == 7.0).all()


@pytest.mark.parametrize("H,G,d", [(4, 4, 64), (4, 2, 128), (6, 2, 64), (8, 2, 128), (5, 1, 128), (7, 1, 64),
                                   (16, 1, 128), (64, 1, 64), (65, 1, 64), (128, 1, 64)])
@pytest.mark.parametrize("lens", [[1], [5, 1, 0, 130, 64], [300, 17], [0, 0, 129, 128, 127, 0]])
def test_groups_and_lengths(gqa, H, G, d, lens):
    cu = offsets(lens)
    q, k, v = inputs(cu, H, G, d, seed=sum(lens) + H)
    got = run(gqa, q, k, v, cu)
    r, w = ref.prefill_packed(q, k, v, cu, d ** -0.5)
    compare(got, r, w, q)


@pytest.mark.parametrize("window", [1, 2, 31, 128, 200, 257, 1000])
@pytest.mark.parametrize("H,G", [(2, 2), (6, 2), (8, 1)])
def test_windows(gqa, window, H, G):
    cu = offsets([3, 700, 129])
    q, k, v = inputs(cu, H, G, 64, seed=window)
    got = run(gqa, q, k, v, cu, window=window)
    r, w = ref.prefill_packed(q, k, v, cu, 64 ** -0.5, window)
    compare(got, r, w, q)


def test_rows_outside_sequences_are_untouched_and_unread(gqa):
    """cu_seqlens that starts late and ends early; the rows outside hold NaN."""
    cu = [37, 167, 167, 300]
    q, k, v = inputs(cu, 8, 2, 128, N=450, seed=3)
    for x in (q, k, v):
        x[:37] = float("nan")
        x[300:] = float("nan")
    got = run(gqa, q, k, v, cu)
    r, w = ref.prefill_packed(q, k, v, cu, 128 ** -0.5)
    compare(got, r, w, q)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_poisoned_sequence_poisons_no_other(gqa, value):
    cu = offsets([70, 50, 200])
    q, k, v = inputs(cu, 4, 1, 64, seed=4)
    k[70:120] = value
    v[70:120] = value
    got = run(gqa, q, k, v, cu)
    r, w = ref.prefill_packed(q, k, v, cu, 64 ** -0.5)
    for a, z in ((0, 70), (120, 320)):
        ref.check(got[a:z], r[a:z], w[a:z])


def test_many_sequences_match_the_dense_call_and_themselves(gqa):
    """200 prompts of 1 to 400 tokens; each against a call of its own, and twice the same bits."""
    gen = torch.Generator().manual_seed(5)
    lens = torch.randint(1, 401, (200,), generator=gen).tolist()
    cu = offsets(lens)
    q, k, v = inputs(cu, 8, 2, 64, seed=6)
    got, again = run(gqa, q, k, v, cu), run(gqa, q, k, v, cu)
    assert torch.equal(got, again)
    r, w = ref.prefill_packed(q, k, v, cu, 64 ** -0.5)
    compare(got, r, w, q)
    for b in (0, 77, 199):
        a, z = cu[b], cu[b + 1]
        dense = gqa.prefill_causal(*(x[a:z][None].cuda() for x in (q, k, v)))[0].cpu()
        ref.check(dense, r[a:z], w[a:z])


def test_the_largest_batch(gqa):
    """8192 sequences, every third empty."""
    lens = [0 if b % 3 == 0 else b % 7 + 1 for b in range(8192)]
    cu = offsets(lens)
    q, k, v = inputs(cu, 2, 1, 64, seed=12)
    got = run(gqa, q, k, v, cu)
    for b in (0, 1, 2, 4000, 4001, 8189, 8190, 8191):
        a, z = cu[b], cu[b + 1]
        r, w = ref.prefill_packed(q[a:z], k[a:z], v[a:z], [0, z - a], 64 ** -0.5)
        ref.check(got[a:z], r, w)


def test_long_sequences_sampled(gqa):
    """3000 + 5000 + 1 tokens: rows across all key tiles."""
    cu = offsets([3001, 1, 5000])
    q, k, v = inputs(cu, 8, 2, 128, seed=8)
    got = run(gqa, q, k, v, cu)
    for s in (0, 127, 128, 1500, 3000, 3001, 3002, 5555, 8001):
        a = max(c for c in cu if c <= s)
        for h in (0, 3, 7):
            r, w = ref.attend(q[s:s + 1, h], k[a:s + 1, h // 4], v[a:s + 1, h // 4],
                              torch.ones(1, s + 1 - a, dtype=torch.bool), 128 ** -0.5)
            ref.check(got[s:s + 1, h], r, w)


@pytest.mark.parametrize("scale", [1e-3, 0.5, 4.0])
def test_scales_and_large_scores(gqa, scale):
    """The running maximum moves by far more than the rescale threshold."""
    cu = offsets([513])
    q, k, v = inputs(cu, 2, 1, 64, seed=9)
    k = (k.float() * torch.linspace(0.01, 1, 513)[:, None, None]).to(torch.bfloat16)
    got = run(gqa, q, k, v, cu, scale=scale)
    r, w = ref.prefill_packed(q, k, v, cu, scale)
    # scores reach sum |q k| * scale ~ 64 * 0.64 * 4 * 1.44 < 2^8 in log2 units, 2^2 times what the
    # bound's fp32 part assumes
    d = (got.double() - r).abs()
    assert (d <= ref.bound(r, w) + 4 * ref.FP32_PART * w).all()


def test_bad_offsets_are_clamped_and_flagged(gqa):
    q, k, v = inputs([0, 300], 4, 2, 64, seed=10)
    for cu in ([0, 200, 100, 300], [-5, 300], [0, 301], [0, 1 << 30]):
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        gqa.prefill_packed(q.cuda(), k.cuda(), v.cuda(), torch.tensor(cu, dtype=torch.int32).cuda(), out=out)
        with pytest.raises(gqa.GQAError) as e:
            gqa.get_status()
        assert e.value.code == -7
        gqa.get_status()


def test_captured_replayed_and_on_another_stream(gqa):
    cu = torch.tensor([0, 100, 333], dtype=torch.int32).cuda()
    q, k, v = (x.cuda() for x in inputs([0, 333], 8, 2, 128, seed=11))
    want = gqa.prefill_packed(q, k, v, cu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = gqa.prefill_packed(q, k, v, cu, stream=side)
    side.synchronize()
    assert torch.equal(want, other)
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gqa.prefill_packed(q, k, v, cu, out=out)
    cu.copy_(torch.tensor([0, 200, 333], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, gqa.prefill_packed(q, k, v, cu))
    gqa.get_status()


@pytest.mark.parametrize("cu,held", [
    ([-5, 300], [0, 300]), ([0, 301], [0, 300]), ([0, 1 << 30], [0, 300]), ([0, 200, 100, 300], [0, 200, 200, 300]),
    ([50, 20, 10, 250], [50, 50, 50, 250]), ([0, 1 << 30, 5, 300], [0, 300, 300, 300]),
    ([-5, 100, -7, 200], [0, 100, 100, 200]), ([0, 150, 0, 150, 0, 290], [0, 150, 150, 150, 150, 290]),
    ([0, 60, 130] + [129, 131] * 200 + [280], [0, 60, 130] + [130] + [131] * 399 + [280])])
@pytest.mark.parametrize("H,G", [(4, 2), (3, 1)])
def test_bad_offsets_count_as_the_largest_before_them(gqa, H, G, cu, held):
    """Offsets are forced into [0, N] and then up to the largest before them: no row has two sequences."""
    q, k, v = inputs([0, 300], H, G, 64, seed=13)
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    gqa.prefill_packed(q.cuda(), k.cuda(), v.cuda(), torch.tensor(cu, dtype=torch.int32).cuda(), out=out)
    with pytest.raises(gqa.GQAError) as e:
        gqa.get_status()
    assert e.value.code == -7
    gqa.get_status()
    r, w = ref.prefill_packed(q, k, v, held, 64 ** -0.5)
    compare(out.cpu(), r, w, q)


def test_offsets_that_fall_in_the_largest_batch(gqa):
    lens = [b % 4 for b in range(8192)]
    cu = offsets(lens)
    q, k, v = inputs(cu, 2, 1, 64, seed=16)
    bad = list(cu)
    bad[1] = 700
    bad[4000] = bad[6000] = 5
    held = [max(bad[:b + 1]) for b in range(8193)]
    want = run(gqa, q, k, v, held)
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    gqa.prefill_packed(q.cuda(), k.cuda(), v.cuda(), torch.tensor(bad, dtype=torch.int32).cuda(), out=out)
    with pytest.raises(gqa.GQAError) as e:
        gqa.get_status()
    assert e.value.code == -7
    assert torch.equal(out.cpu(), want)
    gqa.get_status()


@pytest.mark.parametrize("H,G,d", [(4, 4, 64), (2, 2, 128), (4, 2, 128), (6, 2, 64), (8, 2, 64), (5, 1, 128),
                                   (6, 1, 64), (7, 1, 64), (64, 1, 64), (100, 1, 64)])
def test_first_rows_carry_p_as_two_terms(gqa, H, G, d):
    """Positions 0 to 127 of every prompt, whatever its length and group size."""
    cu = offsets([300, 1, 128, 129, 57, 700])
    q, k, v = inputs(cu, H, G, d, seed=H + d)
    got = run(gqa, q, k, v, cu)
    r, w = ref.prefill_packed(q, k, v, cu, d ** -0.5)
    compare(got, r, w, q)
    for a, z in zip(cu[:-1], cu[1:]):
        z = min(z, a + 128)
        ref.check(got[a:z], r[a:z], w[a:z], split=True)


@pytest.mark.parametrize("window", [1, 2, 3, 31, 127, 128, 200, 256])
@pytest.mark.parametrize("H,G,d", [(2, 2, 128), (6, 2, 64), (8, 1, 64)])
def test_narrow_windows_carry_p_as_two_terms(gqa, window, H, G, d):
    cu = offsets([3, 700, 129])
    q, k, v = inputs(cu, H, G, d, seed=window)
    got = run(gqa, q, k, v, cu, window=window)
    r, w = ref.prefill_packed(q, k, v, cu, d ** -0.5, window)
    ref.check(got, r, w, split=True)


@pytest.mark.parametrize("where", ["q", "k", "v"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("H,G", [(2, 2), (6, 2)])
def test_a_row_that_sees_a_value_that_is_not_finite_says_so(gqa, where, value, H, G):
    """One element of one position is not finite: the rows that see it are what the formula makes of it
    (a score of +inf is NaN, one of -inf counts for nothing), the rows before it what they were."""
    cu = offsets([40, 400])
    q, k, v = inputs(cu, H, G, 64, seed=14)
    at = 40 + 230
    for x, name in ((q, "q"), (k, "k"), (v, "v")):
        if name == where:
            x[at, 0, 5] = value
    got = run(gqa, q, k, v, cu).double()
    r, w = ref.prefill_packed(q, k, v, cu, 64 ** -0.5)
    for b in range(2):
        for s in range(cu[b], cu[b + 1]):
            # (0 * NaN: V's own column, in rows before the position)
            if where == "v" and s < at:
                r[s, : H // G, 5] = got[s, : H // G, 5]
                w[s, : H // G, 5] = 0
    assert torch.equal(torch.isnan(got), torch.isnan(r))
    assert torch.equal(got[torch.isinf(r)], r[torch.isinf(r)])
    fine = torch.isfinite(r) & torch.isfinite(got)
    assert fine.sum() > 0.4 * r.numel() and torch.equal(torch.isfinite(got), torch.isfinite(r))
    ref.check(got[fine], r[fine], w[fine])


def test_no_tokens_at_all(gqa):
    for cu in ([0, 0], [3, 3, 3], [0] * 2000):
        q, k, v = inputs([0, 3], 4, 2, 64, seed=17)
        assert (run(gqa, q, k, v, cu) == 7.0).all()
