"""Arguments that the packed, tree and paged calls refuse on the host (no GPU needed)."""
import pytest
import torch

import kv_cache_decode_04_b200 as gqa

L = gqa.lib
A, BB, C, D, E, F, G_, H_ = (i << 32 for i in range(1, 9))  # addresses far apart


def packed(**kw):
    a = dict(q=A, k=BB, v=C, cu=D, out=E, B=2, N=100, H=8, G=2, d_h=64, scale=0.1, window=0, dt=gqa.GQA_BF16)
    a.update(kw)
    return L.gqa_prefill_packed(a["q"], a["k"], a["v"], a["cu"], a["out"], a["B"], a["N"], a["H"], a["G"], a["d_h"],
                                a["scale"], a["window"], a["dt"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(G=3), -1), (dict(B=0), -1), (dict(N=0), -1), (dict(window=-1), -1), (dict(q=None), -1), (dict(cu=None), -1),
    (dict(scale=0.0), -1), (dict(scale=float("inf")), -1), (dict(dt=gqa.GQA_F32), -2), (dict(d_h=96), -2),
    (dict(H=258, G=2), -2), (dict(B=8193), -2), (dict(N=1 << 30), -2), (dict(k=BB + 8), -3), (dict(cu=D + 2), -3),
    (dict(out=A), -1), (dict(out=BB + 16), -1)])
def test_prefill_packed(kw, code):
    assert packed(**kw) == code


def tree(**kw):
    a = dict(q=A, k=BB, v=C, table=D, sl=E, mask=F, nd=None, scale=0.1, out=G_, B=2, n=4, H=8, G=2, d_h=64, page=16,
             P=10, M=5, dt=gqa.GQA_BF16, ws=H_, wsb=1 << 30)
    a.update(kw)
    return L.gqa_decode_tree(a["q"], a["k"], a["v"], a["table"], a["sl"], a["mask"], a["nd"], a["scale"], a["out"],
                             a["B"], a["n"], a["H"], a["G"], a["d_h"], a["page"], a["P"], a["M"], a["dt"], a["ws"],
                             a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(G=3), -1), (dict(n=0), -1), (dict(n=65), -1), (dict(sl=None), -1), (dict(scale=-1.0), -1),
    (dict(scale=float("nan")), -1), (dict(dt=gqa.GQA_F32), -2), (dict(dt=9), -2), (dict(d_h=32), -2),
    (dict(H=258, G=2), -2), (dict(page=24), -2), (dict(page=0), -1), (dict(M=0), -1), (dict(M=1 << 28), -2),
    (dict(table=None), -1), (dict(B=8193), -2), (dict(mask=F + 4), -3), (dict(out=A), -1), (dict(q=A + 2), -3),
    (dict(M=1 << 26, B=8000), -2)])
def test_decode_tree(kw, code):
    assert tree(**kw) == code
    assert gqa.lib.gqa_last_error_string()


def append(**kw):
    a = dict(kn=A, vn=BB, cu=C, sl=D, slo=E, k=F, v=G_, table=None, B=2, N=8, G=2, d_h=64, page=100, P=2, M=1,
             dt=gqa.GQA_F32)
    a.update(kw)
    return L.gqa_cache_append(a["kn"], a["vn"], a["cu"], a["sl"], a["slo"], a["k"], a["v"], a["table"], a["B"], a["N"],
                              a["G"], a["d_h"], a["page"], a["P"], a["M"], a["dt"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(N=0), -1), (dict(B=0), -1), (dict(kn=None), -1), (dict(P=3), -1), (dict(slo=D + 4), -1), (dict(v=F), -1),
    (dict(kn=F), -1), (dict(dt=5), -2), (dict(d_h=80), -2), (dict(kn=A + 4), -3), (dict(sl=D + 1), -3)])
def test_cache_append(kw, code):
    assert append(**kw) == code


def compact(**kw):
    a = dict(k=A, v=BB, table=C, sl=D, keep=E, nk=F, slo=G_, B=2, m=4, G=2, d_h=64, page=16, P=9, M=3,
             dt=gqa.GQA_BF16)
    a.update(kw)
    return L.gqa_cache_compact(a["k"], a["v"], a["table"], a["sl"], a["keep"], a["nk"], a["slo"], a["B"], a["m"],
                               a["G"], a["d_h"], a["page"], a["P"], a["M"], a["dt"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(m=0), -1), (dict(m=65), -1), (dict(keep=None), -1), (dict(slo=D), -1), (dict(slo=E), -1), (dict(v=A), -1),
    (dict(d_h=256), -2), (dict(k=A + 8), -3), (dict(nk=F + 2), -3)])
def test_cache_compact(kw, code):
    assert compact(**kw) == code


def test_pages():
    def reserve(**kw):
        a = dict(t=A, r=BB, sl=C, n=D, k=E, v=F, B=2, G=2, d_h=64, page=16, P=10, M=5, dt=gqa.GQA_BF16, ws=G_,
                 wsb=1 << 20)
        a.update(kw)
        return L.gqa_pages_reserve(a["t"], a["r"], a["sl"], a["n"], a["k"], a["v"], a["B"], a["G"], a["d_h"],
                                   a["page"], a["P"], a["M"], a["dt"], a["ws"], a["wsb"], None)

    for kw, code in [(dict(t=None), -1), (dict(r=A), -1), (dict(P=0), -1), (dict(v=E), -1), (dict(dt=3), -2),
                     (dict(ws=None), -5), (dict(wsb=10), -5), (dict(ws=G_ + 16), -3), (dict(n=None), -1)]:
        assert reserve(**kw) == code, kw
    assert L.gqa_pages_fork(A, BB, C, D, E, 0, 4, 16, 10, 5, None) == -1
    assert L.gqa_pages_fork(A, BB, C, D, E, 8193, 4, 16, 10, 5, None) == -2
    assert L.gqa_pages_fork(A, BB, C, None, E, 2, 4, 16, 10, 5, None) == -1
    assert L.gqa_pages_fork(A, BB, C + 1, D, E, 2, 4, 16, 10, 5, None) == -3
    assert L.gqa_pages_release(A, BB, None, 4, 16, 10, 5, None) == -1
    assert L.gqa_pages_release(A, BB, C, 4, 0, 10, 5, None) == -1
    assert L.gqa_pages_release(A, BB, C, 4, 1 << 28, 10, 64, None) == -2


def test_the_binding_checks_shapes_types_and_devices():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        gqa.prefill_packed(z(8, 4, 64), z(9, 2, 64), z(9, 2, 64), i(2))
    with pytest.raises(ValueError):
        gqa.prefill_packed(z(8, 4, 64), z(8, 2, 64), z(8, 2, 64), torch.zeros(2, dtype=torch.int64))
    with pytest.raises(TypeError):
        gqa.prefill_packed(z(8, 4, 64), z(8, 2, 64), z(8, 2, 64, dt=torch.float32), i(2))
    with pytest.raises(TypeError):  # not a CUDA tensor
        gqa.prefill_packed(z(8, 4, 64), z(8, 2, 64), z(8, 2, 64), i(2))
    with pytest.raises(ValueError):  # tree_mask of another type
        gqa.decode_tree(z(2, 3, 4, 64), z(2, 2, 9, 64), z(2, 2, 9, 64), i(2), tree_mask=i(2, 3))
    with pytest.raises(ValueError):  # a dense cache of another batch
        gqa.decode_tree(z(2, 3, 4, 64), z(5, 2, 9, 64), z(5, 2, 9, 64), i(2))
    with pytest.raises(ValueError):
        gqa.decode_tree(z(2, 3, 4, 64), z(5, 2, 16, 64), z(5, 2, 16, 64), i(2), block_table=i(3, 4))
    with pytest.raises(TypeError):
        gqa.cache_append(z(4, 2, 64), z(4, 2, 64), i(3), i(2), z(2, 2, 9, 64, dt=torch.float32),
                         z(2, 2, 9, 64, dt=torch.float32))
    with pytest.raises(ValueError):
        gqa.cache_compact(z(2, 2, 9, 64), z(2, 2, 9, 64), i(2), i(3, 4))
    with pytest.raises(ValueError):
        gqa.pages_reserve(i(2, 4), i(6), i(2), i(2), z(5, 2, 16, 64), z(5, 2, 16, 64))
    with pytest.raises(ValueError):
        gqa.pages_fork(i(2, 4), i(6), i(2), i(2), i(1), page_size=16)


def test_pages_reserve_page_of_2g_pieces():
    # the copy of a shared page counts its 16-byte pieces, 16 a row here, in 32 bits
    big = dict(k=1 << 41, v=1 << 42, B=2, G=8, d_h=128, P=2, M=1)

    def reserve(page):
        return L.gqa_pages_reserve(A, BB, C, D, big["k"], big["v"], big["B"], big["G"], big["d_h"], page, big["P"],
                                   big["M"], gqa.GQA_BF16, G_, 0, None)

    assert reserve(1 << 24) == -2
    assert reserve(1 << 23) == -5  # only the workspace is missing


def test_decode_tree_line_of_2g_tiles():
    # 2^29 segments of one tile, each counted as four
    kw = dict(q=1 << 48, k=1 << 49, v=1 << 50, out=1 << 51, B=1 << 12, n=1, P=1, M=1, page=16, wsb=0)
    assert tree(**kw, H=1 << 17, G=1 << 17) == -2


def test_pages_reserve_table_of_2g_entries():
    # the plan counts the entries that need a page in 32 bits
    def reserve(B, M, page=16):
        return L.gqa_pages_reserve(1 << 50, 1 << 51, C, D, 1 << 52, 1 << 53, B, 2, 64, page, 10, M, gqa.GQA_BF16, G_, 0,
                                   None)

    assert reserve(17, 134217711) == -2
    assert reserve(8192, 1 << 18, 1) == -2
    assert reserve(8192, (1 << 18) - 1, 1) == -5  # only the workspace is missing
    assert reserve(1, 134217711) == -5


def test_what_is_written_overlaps_nothing():
    """Each call with one tensor at the beginning or end of one that it writes."""
    ints = 2 * 5 * 4                       # block_table [2, 5]
    rows = 2 * 4 * 8 * 64 * 2              # q, out [2, 4, 8, 64] bf16
    pool = 10 * 2 * 16 * 64 * 2            # [10, 2, 16, 64] bf16
    for name in ("table", "sl", "mask", "nd"):
        assert tree(**{name: G_ + rows - 8}) == -1, name
    dense = 2 * 2 * 100 * 64 * 4           # [2, 2, 100, 64] fp32
    for kw in (dict(cu=F + dense - 4), dict(sl=G_ + dense - 4), dict(slo=F + dense - 8), dict(slo=A), dict(slo=C + 8)):
        assert append(**kw) == -1, kw
    assert append(table=E, M=5) == -1 and append(table=F, M=5) == -1
    for kw in (dict(sl=A + 16), dict(keep=BB), dict(nk=A), dict(table=G_), dict(slo=A + 64), dict(table=BB)):
        assert compact(**kw) == -1, kw

    def reserve(t=A, r=BB, sl=C, n=D, k=E, v=F, ws=G_):
        return L.gqa_pages_reserve(t, r, sl, n, k, v, 2, 2, 64, 16, 10, 5, gqa.GQA_BF16, ws, 1 << 20, None)

    for kw in (dict(sl=A + ints - 4), dict(n=BB + 36), dict(t=E + pool - 32), dict(r=F), dict(sl=E), dict(ws=A),
               dict(ws=BB), dict(ws=C), dict(ws=D), dict(ws=E + pool - 256), dict(ws=F)):
        assert reserve(**kw) == -1, kw
    for args in ((A, BB, A + ints - 4, D, E), (A, BB, BB, D, E), (A, BB, C, A, E), (A, BB, C, D, BB + 36), (A, BB, C, C, E)):
        assert L.gqa_pages_fork(*args, 2, 2, 16, 10, 5, None) == -1, args
    for lengths in (A + ints - 4, BB):
        assert L.gqa_pages_release(A, BB, lengths, 2, 16, 10, 5, None) == -1


def test_the_tree_workspace_is_sized_for_the_tensors_device(monkeypatch):
    """Its size is kept by device and shape: it is asked of that device, not of the current one."""
    import contextlib

    current = [0]

    @contextlib.contextmanager
    def device(index):
        was, current[0] = current[0], index
        yield
        current[0] = was

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(gqa, "decode_tree_workspace_bytes", lambda *shape: 1000 + current[0])
    gqa._tree_workspace.cache_clear()
    assert gqa._tree_workspace(5, 1, 2, 4, 2, 64) == 1005
    assert gqa._tree_workspace(0, 1, 2, 4, 2, 64) == 1000
    gqa._tree_workspace.cache_clear()
