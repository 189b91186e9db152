"""Packed, tree and paged calls at their limits: offsets past 32 bits, the largest batches at d_h 128, ragged
chains, calls captured with memory of their own, tensors that are refused on the GPU."""
import pytest
import torch

import paged_reference as ref

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def test_pages_behind_32_bits(gqa):
    """Pools of 2.25e9 elements; the sequences live in the last pages."""
    P, G, page, d, H = 2_200_000, 1, 16, 64, 4
    free, _ = torch.cuda.mem_get_info()
    if free < 12 << 30:
        pytest.skip("needs 12 GB")
    kp, vp = (torch.empty((P, G, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert kp.numel() > 1 << 31
    gen = torch.Generator().manual_seed(1)
    k, v = (torch.randn((150, G, d), generator=gen).to(torch.bfloat16) for _ in range(2))
    table = torch.full((2, 8), -1, dtype=torch.int32)
    table[0, :7] = torch.arange(P - 1, P - 8, -1)
    table[1, :3] = torch.arange(P - 10, P - 13, -1)
    table = table.cuda()
    T = gqa.cache_append(k.cuda(), v.cuda(), i32([0, 110, 150]), i32([0, 0]), kp, vp, block_table=table)
    assert T.tolist() == [110, 40]
    assert torch.equal(kp[P - 1, 0].cpu(), k[:16, 0]) and torch.equal(vp[P - 12, 0, :8].cpu(), v[142:150, 0])
    q = torch.randn((2, 5, H, d), generator=gen).to(torch.bfloat16)
    got = gqa.decode_tree(q.cuda(), kp, vp, i32([105, 35]), block_table=table)
    gqa.get_status()
    for b, (a, n) in enumerate(((0, 110), (110, 40))):
        sees = torch.ones((5, n), dtype=torch.bool).tril(n - 5)
        for h in range(H):
            r, w = ref.attend(q[b, :, h], k[a:a + n, 0], v[a:a + n, 0], sees, d ** -0.5)
            ref.check(got[b, :, h], r, w)
    gqa.cache_compact(kp, vp, i32([105, 35]), i32([[2, 4], [1, 3]]), block_table=table)
    gqa.get_status()
    assert torch.equal(kp[P - 7, 0, 9:11].cpu(), k[[107, 109], 0])
    # a shared page high up is copied to a free one higher still
    count = torch.ones(P, dtype=torch.int32, device="cuda")
    count[P - 2:] = 0
    count[P - 12] = 2
    both = torch.full((1, 8), -1, dtype=torch.int32)
    both[0, :3] = torch.tensor([P - 10, P - 11, P - 12])
    both = both.cuda()
    gqa.pages_reserve(both, count, i32([37]), i32([4]), kp, vp)
    gqa.get_status()
    assert both.tolist()[0][:3] == [P - 10, P - 11, P - 2] and int(count[P - 12]) == 1
    assert torch.equal(kp[P - 2, 0, :5], kp[P - 12, 0, :5]) and torch.equal(vp[P - 2, 0, :5], vp[P - 12, 0, :5])


def test_largest_batch_at_128(gqa):
    B, H, d = 8000, 2, 128
    gen = torch.Generator().manual_seed(2)
    q = torch.randn((B, 1, H, d), generator=gen).to(torch.bfloat16).cuda()
    k, v = (torch.randn((B, 1, 4, d), generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    lens = [b % 4 for b in range(B)]
    got = gqa.decode_tree(q, k, v, i32(lens)).cpu()
    gqa.get_status()
    for b in (0, 1, 2, 3, 4000, 7998, 7999):
        keys = lens[b] + 1
        for h in range(H):
            r, w = ref.attend(q[b, :, h].cpu(), k[b, 0, :keys].cpu(), v[b, 0, :keys].cpu(),
                              torch.ones((1, keys), dtype=torch.bool), d ** -0.5)
            ref.check(got[b, :, h], r, w)


def test_two_row_tiles_in_the_largest_batch(gqa):
    B, H, d, n = 8000, 64, 64, 3  # 192 rows
    gen = torch.Generator().manual_seed(3)
    q = torch.randn((B, n, H, d), generator=gen).to(torch.bfloat16).cuda()
    k, v = (torch.randn((B, 1, 6, d), generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    lens = [b % 4 for b in range(B)]
    got = gqa.decode_tree(q, k, v, i32(lens)).cpu()
    gqa.get_status()
    for b in (0, 1, 3, 5001, 7999):
        keys = lens[b] + n
        sees = torch.ones((n, keys), dtype=torch.bool).tril(lens[b])
        for h in (0, 63):
            r, w = ref.attend(q[b, :, h].cpu(), k[b, 0, :keys].cpu(), v[b, 0, :keys].cpu(), sees, d ** -0.5)
            ref.check(got[b, :, h], r, w)


def test_packed_largest_batch_at_128(gqa):
    lens = [b % 4 for b in range(8192)]
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    gen = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn((cu[-1], h, 128), generator=gen).to(torch.bfloat16) for h in (2, 1, 1))
    got = gqa.prefill_packed(q.cuda(), k.cuda(), v.cuda(), i32(cu)).cpu()
    gqa.get_status()
    for b in (1, 2, 3, 4097, 8190, 8191):
        a, z = cu[b], cu[b + 1]
        r, w = ref.prefill_packed(q[a:z], k[a:z], v[a:z], [0, z - a], 128 ** -0.5)
        ref.check(got[a:z], r, w)


@pytest.mark.parametrize("H,G", [(8, 2), (64, 1)])
def test_ragged_chains(gqa, H, G):
    """Draft counts without masks."""
    from test_gpu_tree import Case, compare, run

    x = Case(4, 20, H, G, 64, 32, [0, 50, 200, 117], counts=[20, 0, 7, 12], seed=5)
    compare(run(gqa, x, mask=False), x, mask=False)


def test_captured_with_memory_of_its_own(gqa):
    """Workspaces and outputs that the calls allocate themselves, inside a capture."""
    from test_gpu_tree import Case

    x = Case(3, 6, 8, 2, 64, 16, [40, 300, 7], seed=6)
    a, kw = x.args()
    want = gqa.decode_tree(*a, **kw)
    table, count = torch.full((2, 4), -1, dtype=torch.int32, device="cuda"), torch.zeros(9, dtype=torch.int32,
                                                                                         device="cuda")
    zero, five = i32([0, 0]), i32([5, 20])
    kp = torch.zeros((9, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    gqa.pages_reserve(table, count, zero, zero, kp, vp)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = gqa.decode_tree(*a, **kw)
        gqa.pages_reserve(table, count, zero, five, kp, vp)
    for _ in range(3):
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    assert table.tolist() == [[0, -1, -1, -1], [1, 2, -1, -1]] and count.tolist() == [1, 1, 1] + [0] * 6
    gqa.get_status()


def test_tensors_that_are_refused(gqa):
    q = torch.zeros((8, 4, 64), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((8, 2, 64), dtype=torch.bfloat16, device="cuda")
    cu = i32([0, 8])
    with pytest.raises(ValueError, match="contiguous"):
        gqa.prefill_packed(torch.zeros((4, 8, 64), dtype=torch.bfloat16, device="cuda").transpose(0, 1), k, k, cu,
                           out=q)
    with pytest.raises(TypeError, match="cu_seqlens"):
        gqa.prefill_packed(q, k, k, cu.cpu(), out=q.clone())
    with pytest.raises(gqa.GQAError) as e:
        gqa.prefill_packed(q, k, k, cu, out=q)
    assert e.value.code == -1
    with pytest.raises(gqa.GQAError) as e:  # k is not 16-byte aligned
        flat = torch.zeros(8 * 2 * 64 + 1, dtype=torch.bfloat16, device="cuda")
        gqa.prefill_packed(q, flat[1:].view(8, 2, 64), k, cu)
    assert e.value.code == -3
    with pytest.raises(OverflowError):
        gqa.prefill_packed(q, k, k, cu, window=1 << 40)
    with pytest.raises(AttributeError):
        gqa.pages_release([1], cu, cu, page_size=16)
    gqa.get_status()
