// decode_tree.cu -- attention of a tree of drafted tokens over a dense or
// paged K/V cache, on the 5th-generation tensor cores (sm_100a).
//
// What is computed: sequence b holds T_b cached positions followed by its n_b
// drafts' keys and values (positions T_b .. T_b + n_b - 1).  Draft i with query
// head h, g = h / (H/G), sees every cached position and the drafts j < n_b
// whose bit j is set in its 64-bit mask (its ancestors and itself; without
// masks, the drafts j <= i):
//     out[b,i,h] = sum_t softmax_t(scale * q[b,i,h] . K[b,g,t]) V[b,g,t].
// n = 1 is the single-token step over pages.
//
// Rows are (draft, head of the group) pairs, 128 to a tensor-core tile, so a
// cached position is read once for all drafts and all heads of its group.  The
// pipeline is attend.cuh's: with at most 128 rows one row tile and alternate
// key tiles (PAIR = 0), with more two row tiles, 256 rows, that share every key
// tile (PAIR = 1).  Drafts beyond that form further row blocks, each with its
// own pass over the keys.
//
// Partition.  The key tiles of all (sequence, KV head, row block) segments are
// laid end to end and cut into equal shares, one per CTA (persistent, one per
// SM), so ragged batches balance.  A segment counts kSegCost tiles more than it
// has, for what a piece costs beside its tiles (its first scores, the merge and
// the output).  A segment that lies in one share is written to `out` directly.
// The others leave one partial record (max, sum, unnormalised O) per piece: a
// share has at most one piece that begins inside its segment (slot 2 cta) and
// one that is cut off by the share's end (slot 2 cta + 1).  The CTA that holds
// the second piece of a cut segment describes the segment to
// decode_tree_combine, which merges its records.
//
// A page is loaded in boxes of up to 128 positions; lane i of a TMA warp looks
// up and loads box i.  Boxes past the sequence's end, and pages that the table
// lacks, are asked for outside the pool, which TMA fills with zeros.
#include <climits>

#include "attend.cuh"
#include "decode_common.cuh"

namespace gqa {

namespace {

using namespace att;

// A segment cut by share boundaries, described by the share whose beginning is
// the first cut: its sequence (-1: no such segment), KV head, row block, last
// share, and the length of the whole line.
struct Cut {
    int b, g, rb, last, W, nd, pad[2];  // nd: drafts of the sequence
};

struct TreeParams {
    const int32_t *seqlens;
    const int64_t *mask;     // null: draft i sees drafts j <= i
    const int32_t *n_draft;  // null: n
    void *out;
    Cut *ws_cut;    // [C]
    float2 *ws_ml;  // [slots][rows]
    float *ws_o;    // [slots][D][rows]
    unsigned *status;
    float scale_log2;
    CacheView c;
    int n, H, r;
    int pt;   // drafts per row tile, floor(128 / r)
    int pb;   // drafts per row block, pt or 2 pt
    int box;  // positions per K/V load
    int C;    // CTAs of the split kernel
    unsigned long long timeout_ns;
};

// Tiles that a segment counts beyond its own.  A piece costs about 3.5 us
// beside its tiles of 1.3 us (one row tile), and less against tiles of 2.3 us.
template <int PAIR>
constexpr int kSegCost = PAIR ? 1 : 3;

// Cached positions and drafts of sequence b, forced into range.
__device__ __forceinline__ int2 seq_state(const TreeParams &p, int b, bool *bad = nullptr) {
    const int nd0 = p.n_draft ? p.n_draft[b] : p.n;
    const int nd = min(max(nd0, 0), min(p.n, p.c.cap));
    const int T0 = p.seqlens[b];
    const int T = min(max(T0, 0), p.c.cap - nd);
    if (bad) *bad = nd != nd0 || T != T0;
    return make_int2(T, nd);
}

__device__ __forceinline__ int share_begin(int c, int W, int C) { return (int)((long long)c * W / C); }

// Bits of `mask` (draft visibility) as the visibility of 32 keys from `rel` on,
// rel counted from the first draft: keys before it are all visible.
__device__ __forceinline__ uint32_t visible_word(uint64_t mask, int rel) {
    if (rel <= -32) return 0xffffffffu;
    if (rel >= 64) return 0u;
    if (rel >= 0) return (uint32_t)(mask >> rel);
    return ((uint32_t)mask << -rel) | ((1u << -rel) - 1u);
}

template <int D, int PAIR_>
struct TreePolicy {
    static constexpr int PAIR = PAIR_;
    static constexpr int kCost = kSegCost<PAIR>;
    using Lay = Layout<D, PAIR>;

    const TreeParams &p;
    const CUtensorMap *tmq, *tmk, *tmv;
    const int *cu;  // [B + 1] weighted tiles before each sequence's segments
    int u_begin, u_end;
    unsigned *status;
    float scale_log2;
    __nv_bfloat16 *out;
    uint64_t timeout_ns;
    uint64_t pol_kv;

    // The key tiles [j0, j1) of segment (b, g, row block rb) that lie in the share.
    struct Piece : PieceBase {
        int b, g, rb, T, nd, j0;
        int slot;  // record slot, -1: the segment is whole
        bool two_terms;
        __device__ bool split(int) const { return two_terms; }
    };
    struct Row {
        uint64_t bits;  // drafts that the row sees
        uint64_t seen;  // drafts that some row of the row block sees
        int out_row;
    };

    struct Iter {
        const TreePolicy &pol;
        int u, b;
        __device__ Iter(const TreePolicy &pol_, bool) : pol(pol_), u(pol_.u_begin) {
            int lo = 0, hi = pol.p.c.B - 1;  // the last b with cu[b] <= u
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (pol.cu[mid] <= u) lo = mid; else hi = mid - 1;
            }
            b = lo;
        }
        __device__ bool next(Piece &q) {
            const TreeParams &p = pol.p;
            while (u < pol.u_end) {
                while (pol.cu[b + 1] <= u) ++b;
                const int2 s = seq_state(p, b);
                const int n_tok = s.x + s.y, nt = (n_tok + kKeys - 1) / kKeys, len = nt + kCost;
                const int off = u - pol.cu[b], seg = off / len, r0 = off - seg * len;
                const int r1 = min(len, r0 + (pol.u_end - u));
                u += r1 - r0;
                const int j0 = max(0, r0 - kCost), j1 = max(0, r1 - kCost);
                if (j1 <= j0) continue;  // nothing but (a part of) the extra cost
                const int blocks = (s.y + p.pb - 1) / p.pb;
                q.b = b;
                q.T = s.x;
                q.nd = s.y;
                q.g = seg / blocks;
                q.rb = seg - q.g * blocks;
                q.j0 = j0;
                q.slot = j0 > 0 ? 2 * (int)blockIdx.x : j1 < nt ? 2 * (int)blockIdx.x + 1 : -1;
                const int keys = min(n_tok, j1 * kKeys) - j0 * kKeys;
                q.k0 = keys;
                q.k1 = PAIR && s.y - q.rb * p.pb > p.pt ? keys : 0;
                // as in the dense decode: P as two terms for at most 256 positions
                q.two_terms = n_tok <= 256;
                return true;
            }
            return false;
        }
        __device__ void done() {}
    };

    // Page (outside the pool when there is nothing to read) and row of this lane's box.
    struct Where {
        int page, row;
    };
    __device__ Where kv_look(const Piece &q, int j, int lane) const {
        Where w = {p.c.num_pages, 0};
        const int pos = (q.j0 + j) * kKeys + lane * p.box;
        if (lane * p.box < kKeys && pos < q.T + q.nd) {
            if (p.c.table) {
                const int k = pos / p.c.page;
                const int e = p.c.table[(size_t)q.b * p.c.M + k];
                w.row = pos - k * p.c.page;
                if (e >= 0 && e < p.c.num_pages) w.page = e;
                else set_status(status, STATUS_PAGES);
            } else {
                w.page = q.b;
                w.row = pos;
            }
        }
        return w;
    }
    __device__ void kv(const Piece &q, int, Where w, bool is_k, uint8_t *dst, uint64_t *bar, int lane) const {
        if (lane * p.box < kKeys)
            for (int half = 0; half < Lay::HALVES; ++half)
                tma_load_4d(dst + half * kHalf + lane * p.box * 128, is_k ? tmk : tmv, bar, half * 64, w.row, q.g,
                            w.page, pol_kv);
    }
    __device__ int q_bytes() const { return p.pt * p.r * 128; }
    __device__ void q(const Piece &q, int hh, uint8_t *dst, uint64_t *bar) const {
        for (int half = 0; half < Lay::HALVES; ++half)
            tma_load_3d(dst + half * kHalf, tmq, bar, half * 64, q.g * p.r, q.b * p.n + q.rb * p.pb + hh * p.pt,
                        pol_kv);
    }
    __device__ Row row(const Piece &q, int hh, int t) const {
        const int tok = t / p.r, head = t - tok * p.r;
        const int i = q.rb * p.pb + hh * p.pt + tok;  // draft
        Row w = {0, 0, -1};
        const int d0 = q.rb * p.pb, d1 = min(q.nd, d0 + p.pb);  // the row block's drafts
        if (p.mask) {
            for (int k = d0 + (t & 31); k < d1; k += 32) w.seen |= (uint64_t)p.mask[(size_t)q.b * p.n + k];
            w.seen = (uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)w.seen) |
                     (uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)(w.seen >> 32)) << 32;
        } else {
            w.seen = ~0ull >> (64 - d1);
        }
        w.seen &= ~0ull >> (64 - q.nd);
        if (tok < p.pt && i < q.nd && index_ok(q.b < p.c.B && i < p.n && q.g * p.r + head < p.H, status)) {
            w.bits = p.mask ? (uint64_t)p.mask[(size_t)q.b * p.n + i] : ~0ull >> (63 - i);
            w.bits &= ~0ull >> (64 - q.nd);
            w.out_row = (q.b * p.n + i) * p.H + q.g * p.r + head;
        }
        return w;
    }
    __device__ bool masked(const Piece &q, int, int j) const { return (q.j0 + j + 1) * kKeys > q.T; }
    __device__ uint32_t words(const Piece &q, const Row &w, int j, int c) const {
        return visible_word(w.bits, (q.j0 + j) * kKeys + c * 32 - q.T);
    }
    // From the first draft on when there is one that nobody sees (a padded place that was never
    // written, say), else from the sequence's end on.
    __device__ int clear_from(const Piece &q, const Row &w, int j) const {
        const bool gap = w.seen != (~0ull >> (64 - q.nd));
        return max(0, q.T + (gap ? 0 : q.nd) - (q.j0 + j) * kKeys);
    }
    __device__ bool clears(const Piece &q, const Row &w, int j, int r) const {
        const int rel = (q.j0 + j) * kKeys + r - q.T;
        return rel >= 64 || !((w.seen >> rel) & 1u);
    }
    __device__ float *record(const Piece &q) const {
        return q.slot < 0 ? nullptr : p.ws_o + (size_t)q.slot * D * kRows * (PAIR + 1);
    }
    __device__ float2 *record_ml(const Piece &q) const { return p.ws_ml + (size_t)q.slot * kRows * (PAIR + 1); }

    // Once, by warp 11: describes the segment that this share's beginning cuts first: the share
    // begins behind the segment's first tile and the share before it does not.  (An empty
    // share, of which there are some when the tiles are fewer than the CTAs, may do so.)
    bool described = false;
    __device__ void side(int lane) {
        if (lane != 0 || described) return;
        described = true;
        Cut cut = {-1, 0, 0, 0, cu[p.c.B], 0, {0, 0}};
        const int W = cut.W, c = blockIdx.x;
        if (u_begin > 0 && u_begin < W) {
            const int b = Iter(*this, false).b;
            const int2 s = seq_state(p, b);
            const int nt = (s.x + s.y + kKeys - 1) / kKeys, len = nt + kCost;
            const int off = u_begin - cu[b], seg = off / len, s0 = cu[b] + seg * len;
            const int blocks = (s.y + p.pb - 1) / p.pb;
            if (u_begin > s0 + kCost && share_begin(c - 1, W, p.C) <= s0 + kCost) {
                cut.b = b;
                cut.g = seg / blocks;
                cut.rb = seg % blocks;
                cut.nd = s.y;
                cut.last = (int)(((long long)(s0 + len) * p.C - 1) / W);
            }
        }
        p.ws_cut[c] = cut;
    }
};

template <int D, int PAIR>
size_t tree_smem(int B) {
    return Layout<D, PAIR>::SMEM + (size_t)(B + 1) * 4 + 32 * 4;
}

template <int D, int PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    decode_tree_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                       const __grid_constant__ CUtensorMap tmv, const TreeParams p) {
    using Lay = Layout<D, PAIR>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const Barriers<D, PAIR> bar(sm);
    int *cu = reinterpret_cast<int *>(sm + Lay::OFF_POLICY);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        bar.init();
        fence_barrier_init();
    }
    if (threadIdx.x == 256) {
        tma_prefetch_desc(&tmq);
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
    }
    if (warp == 9) tc::tmem_alloc(bar.tmem_slot, kTmemCols);
    tc::fence_before();
    pdl_wait_primary();
    const int W = block_prefix(p.c.B, cu, cu + p.c.B + 1, [&](int b) {
        bool bad;
        const int2 s = seq_state(p, b, &bad);
        if (bad && blockIdx.x == 0) set_status(p.status, STATUS_SEQLEN);
        return ((s.x + s.y + kKeys - 1) / kKeys + kSegCost<PAIR>) * ((s.y + p.pb - 1) / p.pb) * p.c.G;
    });
    pdl_launch_dependents();
    tc::fence_after();
    const uint32_t tmem = *bar.tmem_slot;
    TreePolicy<D, PAIR> pol{p, &tmq, &tmk, &tmv, cu, share_begin(blockIdx.x, W, p.C),
                            share_begin(blockIdx.x + 1, W, p.C), p.status, p.scale_log2,
                            static_cast<__nv_bfloat16 *>(p.out), p.timeout_ns, l2_policy_evict_first()};
    attend<D, PAIR>(pol, sm, tmem);
    tc::fence_before();
    __syncthreads();
    if (warp == 9) {
        tc::fence_after();
        tc::tmem_dealloc(tmem, kTmemCols);
    }
}

// Merges the records of the segment cut at the start of share c = blockIdx.x:
// M = max m_i, out = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i.  One thread per
// record row, columns [8 y, 8 y + 8) of d_h; reads are coalesced (column-major
// records).  Latency-bound: all that it needs of the segment comes in one load,
// four records are asked for at a time, and the blocks fit the GPU at once.
template <int D, int PAIR>
__global__ void __launch_bounds__(kRows *(PAIR + 1)) decode_tree_combine(const TreeParams p) {
    constexpr int kRecRows = kRows * (PAIR + 1);
    const int t = threadIdx.x;
    const int hh = t >> 7, tok = (t & 127) / p.r, head = (t & 127) - tok * p.r;
    const int col = blockIdx.y * 8;
    pdl_wait_primary();
    const int4 *desc = reinterpret_cast<const int4 *>(p.ws_cut + blockIdx.x);
    const int4 d0 = desc[0], d1 = desc[1];
    const int b = d0.x, g = d0.y, rb = d0.z, last = d0.w, W = d1.x, nd = d1.y;
    const int i = rb * p.pb + hh * p.pt + tok;
    if (b < 0 || tok >= p.pt || i >= nd) return;
    // the records: slot 2 c - 1 (the end of the share before), then slot 2 c of each share
    // up to the last that is not empty
    const int first = blockIdx.x, n = last - first + 2;
    float M = -INFINITY, L = 0.f, acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    for (int k0 = 0; k0 < n; k0 += 4) {
        float2 v[4];
        float o[4][8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = k0 + j, c = first + k - 1;
            v[j] = make_float2(-INFINITY, 0.f);
            if (k >= n || (k > 0 && W < p.C && share_begin(c, W, p.C) == share_begin(c + 1, W, p.C))) continue;
            const size_t slot = 2 * (size_t)c + (k == 0 ? 1 : 0);
            v[j] = p.ws_ml[slot * kRecRows + t];
            const float *src = p.ws_o + (slot * D + col) * kRecRows + t;
#pragma unroll
            for (int e = 0; e < 8; ++e) o[j][e] = src[(size_t)e * kRecRows];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (v[j].x == -INFINITY) {  // no record, or nothing seen yet (0); all that was seen is NaN (NaN)
                L += v[j].y;
                continue;
            }
            const float Mn = fmaxf(M, v[j].x);
            const float a = fast_exp2(M - Mn), w = fast_exp2(v[j].x - Mn);
            L = L * a + w * v[j].y;
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = acc[e] * a + w * o[j][e];
            M = Mn;
        }
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    uint32_t pk[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) pk[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) +
                               (((size_t)b * p.n + i) * p.H + g * p.r + head) * D + col) =
        make_uint4(pk[0], pk[1], pk[2], pk[3]);
}

template <int D, int PAIR>
struct TreeTag {};

template <int D, int PAIR>
cudaError_t run_tree(const TreeParams &p, const CUtensorMap *tmq, const CUtensorMap *tmk, const CUtensorMap *tmv,
                     cudaStream_t st) {
    auto kern = decode_tree_kernel<D, PAIR>;
    cudaError_t e = once_per_device<TreeTag<D, PAIR>>([&] {
        cudaFuncAttributes fa;
        cudaError_t r = cudaFuncGetAttributes(&fa, kern);
        if (r != cudaSuccess) return r;
        if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidKernelImage;  // register split would not hold
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    });
    if (e != cudaSuccess) return e;
    e = dec::launch_pdl(kern, dim3(p.C), dim3(kThreads), tree_smem<D, PAIR>(p.c.B), st, *tmq, *tmk, *tmv, p);
    if (e != cudaSuccess) return e;
    return dec::launch_pdl(decode_tree_combine<D, PAIR>, dim3(p.C, D / 8), dim3(kRows * (PAIR + 1)), 0, st, p);
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// Two row tiles when one does not hold all of a KV head's rows.
bool tree_pair(int n, int r) { return n > kRows / r; }

}  // namespace

size_t decode_tree_workspace(int n, int r, int d_h, int num_sms) {
    const size_t rows = (size_t)kRows * (tree_pair(n, r) ? 2 : 1), slots = 2 * (size_t)num_sms;
    return up256((size_t)num_sms * sizeof(Cut)) + up256(slots * rows * 8) + up256(slots * rows * d_h * 4);
}

cudaError_t launch_decode_tree(const TreeArgs &a, const CUtensorMap *tmq, const CUtensorMap *tmk,
                               const CUtensorMap *tmv, cudaStream_t st) {
    TreeParams p = {};
    p.seqlens = a.seqlens;
    p.mask = a.mask;
    p.n_draft = a.n_draft;
    p.out = a.out;
    p.status = a.status;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.c = a.cache;
    p.n = a.n;
    p.H = a.H;
    p.r = a.H / a.cache.G;
    p.pt = kRows / p.r;
    const bool pair = tree_pair(a.n, p.r);
    p.pb = pair ? 2 * p.pt : p.pt;
    p.box = a.box;
    p.C = a.num_sms;
    p.timeout_ns = a.timeout_ns;
    const size_t rows = (size_t)kRows * (pair ? 2 : 1), slots = 2 * (size_t)a.num_sms;
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    p.ws_cut = reinterpret_cast<Cut *>(ws);
    ws += up256((size_t)a.num_sms * sizeof(Cut));
    p.ws_ml = reinterpret_cast<float2 *>(ws);
    ws += up256(slots * rows * 8);
    p.ws_o = reinterpret_cast<float *>(ws);
    if (a.d_h == 128) return pair ? run_tree<128, 1>(p, tmq, tmk, tmv, st) : run_tree<128, 0>(p, tmq, tmk, tmv, st);
    if (a.d_h == 64) return pair ? run_tree<64, 1>(p, tmq, tmk, tmv, st) : run_tree<64, 0>(p, tmq, tmk, tmv, st);
    return cudaErrorInvalidValue;
}

}  // namespace gqa
