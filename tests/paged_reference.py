"""Plain 64-bit definitions of the packed-prompt, draft-tree and paged-cache calls, for the tests.

Attention returns (out, weight): ``weight`` is the softmax-weighted sum of |v|, the quantity the error
bounds are stated in.  Everything runs on the CPU in float64 and, for the page pool, on Python lists.

Error bound of the attention kernels (``bound``).  With u = 2^-8, half a bf16 step relative to the value:
  - the output is rounded once to bf16: at most u |ref|;
  - P is rounded to bf16 before P.V, each p_t by at most u p_t, which moves the output by at most
    u sum_t p_t |v_t| / l = u weight; where P is carried as two bf16 terms that is u^2 weight;
  - q.k over d_h <= 128 bf16 products in fp32 (relative 2^-23 a step, 128 steps): the scores of these
    tests stay below 2^5 in sum_d |q_d k_d| * scale * log2(e) < 2^6, so p is off by at most
    128 * 2^-23 * 2^6 * ln 2 < 2^-10 of itself in the worst case of every rounding one way, which random
    signs bring to about 2^-10 / sqrt(128) < 2^-13; the running sums, the exponential (2^-22) and the merge
    weights add less.  2^-12 weight covers them.
A first-order bound; 1.01 leaves room for the products of these terms.
"""
import math

import torch

U = torch.finfo(torch.bfloat16).eps / 2
FP32_PART = 2.0 ** -12


def attend(q, K, V, sees, scale):
    """q [rows, d], K/V [keys, d], sees [rows, keys]: (softmax(scale q K^T) V, softmax . |V|)."""
    q, K, V = q.double(), K.double(), V.double()
    x = (q @ K.T) * scale
    x = x.masked_fill(~sees, -math.inf)
    top = x.max(1, keepdim=True).values if x.shape[1] else torch.zeros(x.shape[0], 1, dtype=torch.float64)
    e = torch.exp(x - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    z = e.sum(1, keepdim=True)
    w = e / torch.where(z > 0, z, torch.ones_like(z))
    return w @ V, w @ V.abs()


def bound(ref, weight, split=False):
    return 1.01 * (U * ref.abs() + ((U * U if split else U) + FP32_PART) * weight)


def check(got, ref, weight, split=False):
    d = (got.detach().double().cpu() - ref).abs()
    assert torch.isfinite(got.double()).all(), "non-finite output"
    over = d - bound(ref, weight, split)
    assert (over <= 0).all(), "max excess %g at %s" % (over.max().item(), (over > 0).nonzero()[:4].tolist())


def prefill_packed(q, k, v, cu, scale, window=0):
    """(out, weight) [N, H, d]; rows of no sequence are NaN."""
    N, H, d = q.shape
    r = H // k.shape[1]
    out = torch.full((N, H, d), math.nan, dtype=torch.float64)
    weight = out.clone()
    for a, z in zip(cu[:-1], cu[1:]):
        i, j = torch.arange(a, z)[:, None], torch.arange(a, z)[None]
        sees = (j <= i) & ((j > i - window) if window else True)
        for h in range(H):
            out[a:z, h], weight[a:z, h] = attend(q[a:z, h], k[a:z, h // r], v[a:z, h // r], sees, scale)
    return out, weight


def rows_of(cache, table, b, count):
    """Positions 0..count-1 of sequence b of a paged (table [B, M]) or dense cache, [G, count, d]."""
    if table is None:
        return cache[b, :, :count]
    page = cache.shape[2]
    held = [int(e) for e in table[b][: -(-count // page)]]
    zero = torch.zeros_like(cache[0])
    return torch.cat([cache[e] if 0 <= e < cache.shape[0] else zero for e in held], 1)[:, :count] if held \
        else cache[0, :, :0]


def decode_tree(q, k, v, table, seqlens, mask, n_draft, scale):
    """(out, weight) [B, n, H, d]; rows past n_draft are NaN."""
    B, n, H, d = q.shape
    G = k.shape[1]
    r = H // G
    out = torch.full((B, n, H, d), math.nan, dtype=torch.float64)
    weight = out.clone()
    for b in range(B):
        T = int(seqlens[b])
        c = n if n_draft is None else int(n_draft[b])
        if c == 0:
            continue
        sees = torch.ones((c, T + c), dtype=torch.bool)
        for i in range(c):
            for j in range(c):
                sees[i, T + j] = j <= i if mask is None else bool((int(mask[b, i]) >> j) & 1)
        K, V = rows_of(k, table, b, T + c), rows_of(v, table, b, T + c)
        for h in range(H):
            out[b, :c, h], weight[b, :c, h] = attend(q[b, :c, h], K[h // r], V[h // r], sees, scale)
    return out, weight


def place(table, page, b, pos):
    return (b, pos) if table is None else (int(table[b][pos // page]), pos % page)


class Pool:
    """The page pool on lists: table rows, reference counts, lengths, and K/V page contents as a dict
    page -> list of rows (any values)."""

    def __init__(self, table, ref, seqlens, page):
        self.table, self.ref, self.T = [list(r) for r in table], list(ref), list(seqlens)
        self.page, self.copies = page, []
        self.flagged = False

    def release(self, lengths):
        for b, L in enumerate(lengths):
            if L < 0:
                self.flagged = True
                continue
            for k in range(-(-L // self.page), len(self.table[b])):
                e = self.table[b][k]
                if e < 0:
                    continue
                self.table[b][k] = -1
                if e >= len(self.ref) or self.ref[e] <= 0:
                    self.flagged = True
                else:
                    self.ref[e] -= 1

    def fork(self, src, dst):
        B, M = len(self.table), len(self.table[0])
        for i, (a, z) in enumerate(zip(src, dst)):
            ok = 0 <= a < B and 0 <= z < B and z not in src and z not in dst[:i] and a not in dst
            if ok:
                T = self.T[a]
                ok = 0 <= T <= M * self.page and all(e < 0 for e in self.table[z])
                need = -(-T // self.page) if ok else 0
                ok = ok and all(0 <= e < len(self.ref) for e in self.table[a][:need])
            if not ok:
                self.flagged = True
                continue
            for k in range(need):
                self.table[z][k] = self.table[a][k]
                self.ref[self.table[a][k]] += 1
            self.T[z] = T

    def reserve(self, new):
        B, M, P = len(self.table), len(self.table[0]), len(self.ref)
        before = list(self.ref)
        takes = []
        for b in range(B):
            T, n = self.T[b], new[b]
            if T < 0 or n < 0 or T + n > M * self.page:
                self.flagged = True
                continue
            if n == 0:
                continue
            for k in range(T // self.page, -(-(T + n) // self.page)):
                e = self.table[b][k]
                if e >= P or (e >= 0 and before[e] < 1):
                    self.flagged = True
                if not (0 <= e < P and before[e] == 1):
                    takes.append((b, k, e))
        free = [p for p in range(P) if before[p] == 0]
        if len(free) < len(takes):
            self.flagged = True
            return
        for (b, k, e), p in zip(takes, free):
            self.table[b][k] = p
            self.ref[p] = 1
            if 0 <= e < P and before[e] > 1:
                self.ref[e] -= 1
                if k == self.T[b] // self.page and self.T[b] % self.page:
                    self.copies.append((e, p, self.T[b] % self.page))
