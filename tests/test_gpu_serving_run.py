"""The packed, tree and paged calls together, as a serving loop uses them.

Prompts are prefilled packed and their K/V appended into pages; then rounds of: reserve, append the drafts,
attend, keep an accepted path, trim.  Beside it the sequences grow as plain lists of K/V rows.  Every
attention output is held to the 64-bit definition over those lists, and at the end every page holds what
the lists say.
"""
import pytest
import torch

import paged_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page,H,G,d", [(16, 8, 2, 64), (64, 6, 3, 128)])
def test_speculative_serving(gqa, page, H, G, d):
    gen = torch.Generator().manual_seed(page)
    prompts = [37, 1, 130, 200]
    B, n, M, P = len(prompts), 12, 24, 140
    scale = d ** -0.5

    def rows(N, heads):
        return torch.randn((N, heads, d), generator=gen).to(torch.bfloat16)

    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    kp = torch.full((P, G, page, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vp = kp.clone()
    table = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
    count = torch.zeros(P, dtype=torch.int32, device="cuda")
    T = torch.zeros(B, dtype=torch.int32, device="cuda")

    # prompts
    N = sum(prompts)
    q, k, v = rows(N, H), rows(N, G), rows(N, G)
    cu = [sum(prompts[:b]) for b in range(B + 1)]
    out = gqa.prefill_packed(q.cuda(), k.cuda(), v.cuda(), i32(cu))
    r, w = ref.prefill_packed(q, k, v, cu, scale)
    ref.check(out, r, w)
    gqa.pages_reserve(table, count, T, i32(prompts), kp, vp)
    T = gqa.cache_append(k.cuda(), v.cuda(), i32(cu), T, kp, vp, block_table=table)
    K = [k[cu[b]:cu[b + 1]] for b in range(B)]
    V = [v[cu[b]:cu[b + 1]] for b in range(B)]
    gqa.get_status()

    for step in range(6):
        drafts = torch.randint(1, n + 1, (B,), generator=gen).tolist()
        gqa.pages_reserve(table, count, T, i32(drafts), kp, vp)
        N = sum(drafts)
        kd, vd = rows(N, G), rows(N, G)
        at = [sum(drafts[:b]) for b in range(B + 1)]
        gqa.cache_append(kd.cuda(), vd.cuda(), i32(at), T, kp, vp, block_table=table)
        q = torch.randn((B, n, H, d), generator=gen).to(torch.bfloat16)
        mask, paths = torch.zeros((B, n), dtype=torch.int64), []
        for b in range(B):
            parents = [-1] + [int(torch.randint(max(0, j - 3), j, (1,), generator=gen)) for j in range(1, n)]
            for j in range(n):
                mask[b, j] = (1 << j) | (int(mask[b, parents[j]]) if j else 0)
            leaf = int(torch.randint(0, drafts[b], (1,), generator=gen))
            paths.append([j for j in range(n) if (int(mask[b, leaf]) >> j) & 1])
        got = gqa.decode_tree(q.cuda(), kp, vp, T, tree_mask=mask.cuda(), n_draft=i32(drafts), block_table=table)
        gqa.get_status()
        for b in range(B):
            c = drafts[b]
            kb, vb = torch.cat([K[b], kd[at[b]:at[b + 1]]]), torch.cat([V[b], vd[at[b]:at[b + 1]]])
            sees = torch.ones((c, len(kb)), dtype=torch.bool)
            for i in range(c):
                for j in range(c):
                    sees[i, len(K[b]) + j] = bool((int(mask[b, i]) >> j) & 1)
            for h in range(H):
                g = h // (H // G)
                r, w = ref.attend(q[b, :c, h], kb[:, g], vb[:, g], sees, scale)
                ref.check(got[b, :c, h], r, w)
            kept = [len(K[b]) + j for j in paths[b]]
            K[b], V[b] = torch.cat([K[b], kb[kept]]), torch.cat([V[b], vb[kept]])
        keep = torch.zeros((B, n), dtype=torch.int32)
        for b, path in enumerate(paths):
            keep[b, :len(path)] = torch.tensor(path)
        T = gqa.cache_compact(kp, vp, T, keep.cuda(), n_keep=i32([len(x) for x in paths]), block_table=table)
        gqa.pages_release(table, count, T, page_size=page)
        gqa.get_status()
        assert T.tolist() == [len(x) for x in K]

    held = table.cpu()
    assert int(count.sum()) == sum(-(-len(x) // page) for x in K) and int(count.max()) == 1
    for b in range(B):
        assert torch.equal(ref.rows_of(kp.cpu(), held, b, len(K[b])), K[b].transpose(0, 1))
        assert torch.equal(ref.rows_of(vp.cpu(), held, b, len(V[b])), V[b].transpose(0, 1))


def test_a_layer_cache_takes_drafts(gqa):
    """The dense cache that the layer step appends to serves the tree call as it is."""
    import gqa_inputs as gi

    x = gi.qkv_inputs(2, 256, 8, 2, 64, 40, seed=5, seqlens=[20, 3])
    kc, vc, sl = x.k_cache.cuda(), x.v_cache.cuda(), x.seqlens.cuda()
    qt, T = gqa.qkv_append(x.h.cuda(), x.W_Q.cuda(), x.W_K.cuda(), x.W_V.cuda(), kc, vc, sl)
    # the appended token as one draft behind the old lengths
    got = gqa.decode_tree(qt[:, None], kc, vc, sl)
    want = gqa.decode(qt, kc, vc, T)
    gqa.get_status()
    r, w = ref.decode_tree(qt[:, None].cpu(), kc.cpu(), vc.cpu(), None, [20, 3], None, None, 64 ** -0.5)
    ref.check(got, r, w)
    ref.check(want, r[:, 0], w[:, 0])
