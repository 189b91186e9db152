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
// Rows are (draft, head of the group) pairs, 128 to a tensor-core tile
// (attend.cuh), so a cached position is read once for all drafts and all heads
// of its group: HBM-bound while the rows are few.  Two layouts (PAIR):
//   PAIR = 0, n (H/G) <= 128 rows: one row tile; the two softmax warpgroups
//     take alternate key tiles, each with its own running maximum, sum and O.
//     They are merged in tensor memory's order at the end of a piece.  With one
//     warpgroup the softmax of a tile (~1500 cycles) and its tensor work would
//     follow each other within the ~2850 cycles HBM needs for the tile.
//   PAIR = 1, more rows: two row tiles (256 rows) share every key tile.
//     Drafts beyond that form further row blocks, each with its own pass.
//
// Partition.  The key tiles of all (sequence, KV head, row block) segments are
// laid end to end and cut into equal shares, one per CTA (persistent, one per
// SM), so ragged batches balance to within a tile.  A segment that lies in one
// share is written to `out` directly.  The others leave one partial record
// (max, sum, unnormalised O) per piece: a share has at most one piece that
// begins at its start (slot 2 cta) and one cut off by its end (slot 2 cta + 1).
// decode_tree_combine merges each cut segment's records.
//
// Roles (384 threads):
//   warps 0-3, 4-7  softmax + epilogue of row tile / key parity 0, 1
//   warp 8          K tiles and Q rows by TMA     warp 11  V tiles by TMA
//   warp 9          tcgen05.mma                   warp 10  clears V rows past the end
// A page is loaded in boxes of up to 128 positions; lane i of a TMA warp looks
// up and loads box i.  Boxes past the sequence's end, and pages that the table
// lacks, are asked for outside the pool, which TMA fills with zeros.
#include <climits>

#include "attend.cuh"
#include "decode_common.cuh"

namespace gqa {

namespace {

using namespace att;

template <int D, int PAIR>
struct TreeLay {
    static constexpr int HALVES = D / 64;
    static constexpr int TILE = HALVES * kHalf;  // [128 x D] bf16
    static constexpr int NQ = PAIR ? 1 : 2;      // Q buffers (of PAIR + 1 tiles)
    static constexpr int OFF_Q = 0;              // 2 tiles either way
    static constexpr int OFF_K = 2 * TILE;       // 2 stages
    static constexpr int OFF_V = 4 * TILE;       // 2 stages
    static constexpr int OFF_BAR = 6 * TILE;
    static constexpr int OFF_ML = OFF_BAR + 256;       // [2][128] (m, l) of the two key parities
    static constexpr int OFF_CU = OFF_ML + 2 * 128 * 8;  // cu[B + 1], scratch[32]
};

template <int D, int PAIR>
size_t tree_smem(int B) {
    return 1024 + (size_t)TreeLay<D, PAIR>::OFF_CU + (size_t)(B + 1) * 4 + 32 * 4;
}

struct TreeParams {
    const int32_t *seqlens;
    const int64_t *mask;     // null: draft i sees drafts j <= i
    const int32_t *n_draft;  // null: n
    void *out;
    int *ws_cu;     // [B + 1] tile prefix
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

// Cached positions and drafts of sequence b, forced into range.
__device__ __forceinline__ int2 seq_state(const TreeParams &p, int b, bool *bad = nullptr) {
    const int nd0 = p.n_draft ? p.n_draft[b] : p.n;
    const int nd = min(max(nd0, 0), min(p.n, p.c.cap));
    const int T0 = p.seqlens[b];
    const int T = min(max(T0, 0), p.c.cap - nd);
    if (bad) *bad = nd != nd0 || T != T0;
    return make_int2(T, nd);
}

// A piece: the key tiles [j0, j1) of segment (b, g, row block rb) that lie in
// one share.
struct Piece {
    int b, g, rb, T, nd, nt, j0, j1;
    bool at_start;  // begins where the share begins
};

// Walks a share's pieces in order.
struct PieceWalk {
    int u, u_end, u_begin, b;
    __device__ PieceWalk(const TreeParams &p, const int *cu, int ub, int ue) : u(ub), u_end(ue), u_begin(ub) {
        int lo = 0, hi = p.c.B - 1;  // the last b with cu[b] <= u
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (cu[mid] <= u) lo = mid; else hi = mid - 1;
        }
        b = lo;
    }
    __device__ bool next(const TreeParams &p, const int *cu, Piece &q) {
        if (u >= u_end) return false;
        while (cu[b + 1] <= u) ++b;
        const int2 s = seq_state(p, b);
        q.b = b;
        q.T = s.x;
        q.nd = s.y;
        q.nt = (s.x + s.y + kKeys - 1) / kKeys;
        const int off = u - cu[b], seg = off / q.nt, blocks = (s.y + p.pb - 1) / p.pb;
        q.j0 = off - seg * q.nt;
        q.g = seg / blocks;
        q.rb = seg - q.g * blocks;
        q.at_start = u == u_begin;
        q.j1 = min(q.nt, q.j0 + (u_end - u));
        u += q.j1 - q.j0;
        return true;
    }
};

// cu[b] = key tiles of the segments of all sequences before b; returns the
// whole.  Every thread of the block calls it; scratch holds 32 ints.
__device__ int tree_prefix(const TreeParams &p, int *cu, int *scratch, bool report) {
    const int nthr = blockDim.x, tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int chunk = (p.c.B + nthr - 1) / nthr;
    const int b0 = min(p.c.B, tid * chunk), b1 = min(p.c.B, b0 + chunk);
    bool bad = false;
    auto tiles = [&](int b) {
        bool wrong;
        const int2 s = seq_state(p, b, &wrong);
        bad |= wrong;
        return ((s.x + s.y + kKeys - 1) / kKeys) * ((s.y + p.pb - 1) / p.pb) * p.c.G;
    };
    int local = 0;
    for (int b = b0; b < b1; ++b) local += tiles(b);
    if (bad && report) set_status(p.status, STATUS_SEQLEN);
    int incl = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) scratch[wid] = incl;
    __syncthreads();
    if (wid == 0) {
        const int nw = nthr >> 5;
        int w = lane < nw ? scratch[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += v;
        }
        if (lane < nw) scratch[lane] = w;
        if (lane == nw - 1) cu[p.c.B] = w;
    }
    __syncthreads();
    int run = incl - local + (wid > 0 ? scratch[wid - 1] : 0);
    for (int b = b0; b < b1; ++b) {
        cu[b] = run;
        run += tiles(b);
    }
    __syncthreads();
    return cu[p.c.B];
}

// Bits of `mask` (draft visibility) as the visibility of 32 keys from `rel` on,
// rel counted from the first draft: keys before it are all visible.
__device__ __forceinline__ uint32_t visible_word(uint64_t mask, int rel) {
    if (rel <= -32) return 0xffffffffu;
    if (rel >= 64) return 0u;
    if (rel >= 0) return (uint32_t)(mask >> rel);
    return ((uint32_t)mask << -rel) | ((1u << -rel) - 1u);
}

template <int D, int PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    decode_tree_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                       const __grid_constant__ CUtensorMap tmv, const TreeParams p) {
    using Lay = TreeLay<D, PAIR>;
    constexpr int HALVES = Lay::HALVES, kTile = Lay::TILE, NQ = Lay::NQ;
    constexpr int kRecRows = kRows * (PAIR + 1);
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + Lay::OFF_BAR);
    uint64_t *q_full = bars + 0;    // [2] (NQ used)
    uint64_t *q_empty = bars + 2;   // [2]
    uint64_t *k_full = bars + 4;    // [2]
    uint64_t *k_empty = bars + 6;   // [2]
    uint64_t *v_full = bars + 8;    // [2]
    uint64_t *v_empty = bars + 10;  // [2]
    uint64_t *s_full = bars + 12;   // [2] per softmax warpgroup
    uint64_t *p_ready = bars + 14;  // [2]
    uint64_t *o_done = bars + 16;   // a piece's last P.V is complete
    uint64_t *ep_bar = bars + 17;   // the two warpgroups meet (PAIR = 0)
    uint64_t *drain = bars + 18;
    uint64_t *tail_go = bars + 19;  // [2] a segment's last V tile is on its way to stage i ...
    uint64_t *v_clean = bars + 21;  // [2] ... and its rows past the end are zero
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 23);
    int *abort_flag = reinterpret_cast<int *>(tmem_slot + 1);
    float2 *ml = reinterpret_cast<float2 *>(sm + Lay::OFF_ML);
    int *cu = reinterpret_cast<int *>(sm + Lay::OFF_CU);
    int *scratch = cu + p.c.B + 1;
    volatile int *vabort = abort_flag;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&q_full[s], 1);
            mbar_init(&q_empty[s], 1);
            mbar_init(&k_full[s], 1);
            mbar_init(&k_empty[s], 1);
            mbar_init(&v_full[s], 1);
            mbar_init(&v_empty[s], 1);
            mbar_init(&s_full[s], 1);
            mbar_init(&p_ready[s], 128);
            mbar_init(&tail_go[s], 1);
            mbar_init(&v_clean[s], 1);
        }
        mbar_init(o_done, 1);
        mbar_init(ep_bar, 256);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 8 && lane == 0) {
        tma_prefetch_desc(&tmq);
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
    }
    if (warp == 9) tc::tmem_alloc(tmem_slot, kTmemCols);
    tc::fence_before();
    pdl_wait_primary();
    const int W = tree_prefix(p, cu, scratch, blockIdx.x == 0);  // syncs the block
    pdl_launch_dependents();
    tc::fence_after();
    const uint32_t tmem = *tmem_slot;
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b <= p.c.B; b += kThreads) p.ws_cu[b] = cu[b];
    const int u_begin = (int)((long long)blockIdx.x * W / p.C);
    const int u_end = (int)((long long)(blockIdx.x + 1) * W / p.C);
    const int n_tiles = u_end - u_begin;

    if (n_tiles == 0) {
        // an empty share
    } else if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLowRegs));
        if (warp == 8 || warp == 11) {
            // ------------------------------------------------ TMA producers
            const bool is_k = warp == 8;
            const CUtensorMap *tm = is_k ? &tmk : &tmv;
            uint64_t *full = is_k ? k_full : v_full, *empty = is_k ? k_empty : v_empty;
            uint8_t *ring = sm + (is_k ? Lay::OFF_K : Lay::OFF_V);
            const uint64_t pol = l2_policy_evict_first();
            const int boxes = kKeys / p.box, boxes_bytes = p.box * 128;
            PieceWalk w(p, cu, u_begin, u_end);
            Piece q;
            bool ok = true;
            int it = 0, piece = 0;
            while (ok && w.next(p, cu, q)) {
                const int n_tok = q.T + q.nd;
                for (int j = q.j0; j < q.j1 && ok; ++j, ++it) {
                    const int st = it & 1;
                    // this lane's box: its page (outside the pool when there is nothing to
                    // read) and row, looked up while the stage drains
                    const int pos = j * kKeys + lane * p.box;
                    int page = p.c.num_pages, row = 0;
                    if (lane < boxes && pos < n_tok) {
                        if (p.c.table) {
                            const int k = pos / p.c.page;
                            const int e = p.c.table[(size_t)q.b * p.c.M + k];
                            row = pos - k * p.c.page;
                            if (e >= 0 && e < p.c.num_pages) page = e;
                            else set_status(p.status, STATUS_PAGES);
                        } else {
                            page = q.b;
                            row = pos;
                        }
                    }
                    if (__any_sync(0xffffffffu, *vabort != 0) || !warp_wait(&empty[st], ((it >> 1) & 1) ^ 1, p.timeout_ns)) {
                        if (lane == 0) set_status(p.status, STATUS_TIMEOUT);
                        *vabort = 1;
                        ok = false;
                        break;
                    }
                    if (lane == 0) mbar_arrive_expect_tx(&full[st], kTile);
                    __syncwarp();
                    if (lane < boxes)
                        for (int half = 0; half < HALVES; ++half)
                            tma_load_4d(ring + st * kTile + half * kHalf + lane * boxes_bytes, tm, &full[st], half * 64,
                                        row, q.g, page, pol);
                    if (!is_k && lane == 0 && j == q.nt - 1 && q.nt * kKeys > n_tok) mbar_arrive(&tail_go[st]);
                    if (is_k && j == q.j0) {
                        // the piece's query rows, into the buffer its predecessor's scores released
                        const int qb = piece % NQ;
                        const int d0 = q.rb * p.pb, nh = PAIR && q.nd - d0 > p.pt ? 2 : 1;
                        if (!warp_wait(&q_empty[qb], ((piece / NQ) & 1) ^ 1, p.timeout_ns)) {
                            if (lane == 0) set_status(p.status, STATUS_TIMEOUT);
                            *vabort = 1;
                            ok = false;
                        } else if (lane == 0) {
                            mbar_arrive_expect_tx(&q_full[qb], nh * HALVES * p.pt * p.r * 128);
                            for (int hh = 0; hh < nh; ++hh)
                                for (int half = 0; half < HALVES; ++half)
                                    tma_load_3d(sm + Lay::OFF_Q + (PAIR ? hh : qb) * kTile + half * kHalf, &tmq,
                                                &q_full[qb], half * 64, q.g * p.r, q.b * p.n + d0 + hh * p.pt, pol);
                        }
                        __syncwarp();
                        ++piece;
                    }
                }
            }
            // no copy is in flight when the CTA leaves, whatever the other warps did
            for (int i = max(0, it - 2); i < it; ++i) warp_wait(&full[i & 1], (i >> 1) & 1, p.timeout_ns);
            if (is_k)
                for (int i = max(0, piece - NQ); i < piece; ++i)
                    warp_wait(&q_full[i % NQ], (i / NQ) & 1, p.timeout_ns);
        } else if (warp == 9) {
            // ------------------------------------------------ MMA issuer
            if (lane == 0) {
                constexpr uint32_t idesc_s = tc::idesc_bf16(128, 128, false, false);
                constexpr uint32_t idesc_o = tc::idesc_bf16(128, D, false, true);
                bool issued = false, ok = true;
                auto wait = [&](uint64_t *bar, uint32_t par, bool spin = false) {
                    if (!ok || *vabort ||
                        !(spin ? mbar_wait_spin(bar, par, p.timeout_ns) : mbar_wait(bar, par, p.timeout_ns))) {
                        if (ok) set_status(p.status, STATUS_TIMEOUT);
                        ok = false;
                        *vabort = 1;
                    }
                    return ok;
                };
                const uint64_t dq = tc::sdesc_sw128(smem_u32(sm + Lay::OFF_Q), 16, 1024);
                const uint64_t dk = tc::sdesc_sw128(smem_u32(sm + Lay::OFF_K), 16, 1024);
                const uint64_t dv = tc::sdesc_sw128(smem_u32(sm + Lay::OFF_V), kHalf, 1024);
                auto mma_s = [&](int sb, int qt, int ks) {  // S block sb = Q tile qt times K stage ks
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
                        tc::mma_ss(tmem + sb * 128, dq + ((qt * kTile) >> 4) + off, dk + ((ks * kTile) >> 4) + off,
                                   idesc_s, kk > 0 ? 1u : 0u);
                    }
                    issued = true;
                };
                auto mma_pv = [&](int sb, int vs, bool acc, bool split) {
                    const int passes = split ? 2 : 1;
#pragma unroll 1
                    for (int ps = 0; ps < passes; ++ps)
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            tc::mma_ts(tmem + 256 + sb * 128, tmem + sb * 128 + ps * 64 + kk * 8,
                                       dv + ((vs * kTile + kk * 2048) >> 4), idesc_o,
                                       (acc || ps > 0 || kk > 0) ? 1u : 0u);
                };
                // The scores run ahead of P.V (two tiles for PAIR = 0, one for PAIR = 1), across
                // pieces: S block i is rewritten only behind the P.V that read its P.
                PieceWalk sw(p, cu, u_begin, u_end), vw(p, cu, u_begin, u_end);
                Piece sq, vq;
                int s_it = 0, s_j = 0, s_piece = -1, cnt[2] = {0, 0}, tails[2] = {0, 0};
                bool s_new = true, s_two = false;
                // advances the score walk to the next tile and waits for its inputs
                auto s_next = [&]() {
                    if (s_new) {
                        sw.next(p, cu, sq);
                        ++s_piece;
                        s_j = sq.j0;
                        s_two = PAIR && sq.nd - sq.rb * p.pb > p.pt;
                        if (!wait(&q_full[s_piece % NQ], (s_piece / NQ) & 1)) return false;
                        s_new = false;
                    }
                    return wait(&k_full[s_it & 1], (s_it >> 1) & 1);
                };
                // closes the tile: its K stage, and after a piece's last tile its Q buffer
                auto s_close = [&]() {
                    tc::commit(&k_empty[s_it & 1]);
                    if (++s_j == sq.j1) {
                        tc::commit(&q_empty[s_piece % NQ]);
                        s_new = true;
                    }
                    ++s_it;
                };
                if constexpr (!PAIR) {
                    auto s_tile = [&]() {
                        if (!s_next()) return;
                        mma_s(s_it & 1, s_piece & 1, s_it & 1);
                        tc::commit(&s_full[s_it & 1]);
                        s_close();
                    };
                    s_tile();
                    if (ok && n_tiles > 1) s_tile();
                    int it = 0;
                    while (ok && vw.next(p, cu, vq)) {
                        const bool split = vq.T + vq.nd <= 2 * kKeys, tail = vq.nt * kKeys > vq.T + vq.nd;
                        for (int j = vq.j0; j < vq.j1 && ok; ++j, ++it) {
                            const int st = it & 1;
                            if (!wait(&v_full[st], (it >> 1) & 1)) break;
                            if (tail && j == vq.nt - 1 && !wait(&v_clean[st], tails[st]++ & 1)) break;
                            if (!wait(&p_ready[st], cnt[st]++ & 1, true)) break;
                            tc::fence_after();
                            mma_pv(st, st, j - vq.j0 >= 2, split);
                            tc::commit(&v_empty[st]);
                            if (j + 1 == vq.j1) tc::commit(o_done);
                            if (s_it < n_tiles) s_tile();
                        }
                    }
                } else {
                    bool two = false;
                    if (s_next()) {
                        mma_s(0, 0, 0);
                        tc::commit(&s_full[0]);
                        two = s_two;
                        if (two) {
                            mma_s(1, 1, 0);
                            tc::commit(&s_full[1]);
                        }
                        s_close();
                    }
                    int it = 0;
                    while (ok && vw.next(p, cu, vq)) {
                        const bool split = vq.T + vq.nd <= 2 * kKeys, tail = vq.nt * kKeys > vq.T + vq.nd;
                        for (int j = vq.j0; j < vq.j1 && ok; ++j, ++it) {
                            const int st = it & 1;
                            const bool more = it + 1 < n_tiles, now_two = two;
                            if (!wait(&v_full[st], (it >> 1) & 1)) break;
                            if (tail && j == vq.nt - 1 && !wait(&v_clean[st], tails[st]++ & 1)) break;
                            if (!wait(&p_ready[0], cnt[0]++ & 1, true)) break;
                            tc::fence_after();
                            mma_pv(0, st, j > vq.j0, split);
                            if (more) {
                                if (!s_next()) break;
                                mma_s(0, 0, s_it & 1);
                                tc::commit(&s_full[0]);
                                two = s_two;
                            }
                            if (now_two) {
                                if (!wait(&p_ready[1], cnt[1]++ & 1, true)) break;
                                tc::fence_after();
                                mma_pv(1, st, j > vq.j0, split);
                            }
                            tc::commit(&v_empty[st]);
                            if (j + 1 == vq.j1) tc::commit(o_done);
                            if (more) {
                                if (two) {
                                    mma_s(1, 1, s_it & 1);
                                    tc::commit(&s_full[1]);
                                }
                                s_close();
                            }
                        }
                    }
                }
                if (issued && !ok) {  // let MMAs already issued finish before TMEM is freed
                    tc::commit(drain);
                    mbar_wait(drain, 0, p.timeout_ns);
                }
            }
            __syncwarp();
        } else if (warp == 10) {
            // ------------------------------------------------ V rows past the end
            // Waits for tail_go of the stage first: until the load is issued the stage's
            // v_full may stand two phases back, which its parity alone cannot tell apart.
            // A stage's next tail comes only after the P.V that waits for v_clean.
            PieceWalk w(p, cu, u_begin, u_end);
            Piece q;
            int it = 0, tails[2] = {0, 0};
            while (w.next(p, cu, q)) {
                it += q.j1 - q.j0;
                const int last = it - 1, st = last & 1, n_tok = q.T + q.nd;
                if (q.j1 < q.nt || q.nt * kKeys == n_tok) continue;
                if (!warp_wait(&tail_go[st], tails[st]++ & 1, p.timeout_ns) ||
                    !warp_wait(&v_full[st], (last >> 1) & 1, p.timeout_ns))
                    break;
                zero_tail_rows<D>(sm + Lay::OFF_V + st * kTile, n_tok - (q.nt - 1) * kKeys, lane);
                if (lane == 0) mbar_arrive(&v_clean[st]);
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kHighRegs));
        // ------------------------------------------------ softmax + epilogue
        const int hh = warp >> 2;          // row tile (PAIR) or key-tile parity
        const int t = threadIdx.x & 127;   // row = tensor-memory lane
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_off + hh * 128;
        const uint32_t tO = tmem + lane_off + 256 + hh * 128;
        const int tok = t / p.r, head = t - tok * p.r;
        PieceWalk w(p, cu, u_begin, u_end);
        Piece q;
        bool ok = true;
        int it = 0, cnt = 0, piece = 0, ep_phase = 0;
        auto meet = [&]() {  // both warpgroups (bounded: false when the wait ran out)
            mbar_arrive(ep_bar);
            return warp_wait(ep_bar, ep_phase++ & 1, p.timeout_ns);
        };
        while (ok && w.next(p, cu, q)) {
            const int n_tok = q.T + q.nd;
            const int d0 = q.rb * p.pb + (PAIR ? hh * p.pt : 0);
            const int i = d0 + tok;  // draft of this row
            const bool valid = tok < p.pt && i < q.nd;
            const bool active = !PAIR || d0 < q.nd;  // the row tile has rows
            uint64_t bits = 0;
            if (valid) {
                bits = p.mask ? (uint64_t)p.mask[(size_t)q.b * p.n + i] : ~0ull >> (63 - i);
                bits &= ~0ull >> (64 - q.nd);
            }
            const bool split = n_tok <= 2 * kKeys;
            float m = -INFINITY, l = 0.f;
            bool first = true;
            for (int j = q.j0; j < q.j1; ++j, ++it) {
                if (PAIR ? !active : (it & 1) != hh) continue;
                const bool aborted = __any_sync(0xffffffffu, *vabort != 0);
                if (aborted || !warp_wait(&s_full[hh], cnt & 1, p.timeout_ns)) {
                    ok = false;
                    break;
                }
                ++cnt;
                tc::fence_after();
                const int rel = j * kKeys - q.T;  // the tile's first key, from the first draft
                softmax_step<D>(tS, tO, p.scale_log2, first, split, m, l, [&](uint32_t(&sr)[4][32]) {
                    if (rel + kKeys > 0) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const uint32_t word = visible_word(bits, rel + c * 32);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!((word >> e) & 1u)) sr[c][e] = __float_as_uint(-INFINITY);
                        }
                    }
                });
                first = false;
                tc::fence_before();
                mbar_arrive(&p_ready[hh]);
            }
            if (!ok) break;
            if (!warp_wait(o_done, piece & 1, p.timeout_ns)) {
                ok = false;
                break;
            }
            ++piece;
            tc::fence_after();
            const bool whole = q.j0 == 0 && q.j1 == q.nt;
            const size_t slot = 2 * (size_t)blockIdx.x + (q.at_start ? 0 : 1);
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) +
                                 (((size_t)q.b * p.n + i) * p.H + q.g * p.r + head) * D;
            // the record is column-major so that a warp's stores are 128 bytes in a row
            const int rec_row = (PAIR ? hh * kRows : 0) + t;
            float *rec = p.ws_o + slot * D * kRecRows + rec_row;
            // columns [c0, c1) of O, or of the merge of both parities' O
            float w0 = 1.f, w1 = 0.f, M = m, L = l;
            uint32_t tA = tO, tB = tO;
            int c0 = 0, c1 = D;
            if constexpr (!PAIR) {
                ml[hh * kRows + t] = make_float2(m, l);
                if (!meet()) {
                    ok = false;
                    break;
                }
                const float2 a = ml[t], b2 = ml[kRows + t];
                M = fmaxf(a.x, b2.x);
                w0 = a.x == -INFINITY ? 0.f : fast_exp2(a.x - M);
                w1 = b2.x == -INFINITY ? 0.f : fast_exp2(b2.x - M);
                L = w0 * a.y + w1 * b2.y;
                tA = tmem + lane_off + 256;
                tB = tA + 128;
                c0 = hh * (D / 2);
                c1 = c0 + D / 2;
            }
            if (active) {
                const float inv = whole ? (L > 0.f ? 1.f / L : 0.f) : 1.f;
#pragma unroll 1
                for (int c = c0; c < c1; c += 16) {
                    uint32_t oa[16], ob[16];
                    tc::ld16(tA + c, oa);
                    if constexpr (!PAIR) tc::ld16(tB + c, ob);
                    tc::wait_ld();
                    float v[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        // a parity without a key holds an O that was never written
                        v[e] = w0 != 0.f ? w0 * __uint_as_float(oa[e]) : 0.f;
                        if constexpr (!PAIR)
                            if (w1 != 0.f) v[e] = fmaf(w1, __uint_as_float(ob[e]), v[e]);
                    }
                    if (whole) {
                        uint32_t pk[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) pk[e] = pack_bf16x2(v[2 * e] * inv, v[2 * e + 1] * inv);
                        if (valid) {
                            uint4 *d4 = reinterpret_cast<uint4 *>(dst + c);
                            d4[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                            d4[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e) rec[(size_t)(c + e) * kRecRows] = v[e];
                    }
                }
                if (!whole && (PAIR || hh == 0)) p.ws_ml[slot * kRecRows + rec_row] = make_float2(M, L);
            }
            tc::fence_before();
            if constexpr (!PAIR) {  // both have read both O before either is written again
                if (!meet()) {
                    ok = false;
                    break;
                }
            }
        }
        if (!ok && lane == 0) {
            set_status(p.status, STATUS_TIMEOUT);
            *vabort = 1;
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 9) {
        tc::fence_after();
        tc::tmem_dealloc(tmem, kTmemCols);
    }
}

// Merges the records of each segment that a share boundary cut.  Block (c, y):
// the segment holding the boundary of share c = blockIdx.x + 1, unless an
// earlier boundary already lies inside that segment; columns [16 y, 16 y + 16);
// one thread per record row.
template <int D, int PAIR>
__global__ void __launch_bounds__(kRows *(PAIR + 1)) decode_tree_combine(const TreeParams p) {
    constexpr int kRecRows = kRows * (PAIR + 1);
    pdl_wait_primary();
    const int *cu = p.ws_cu;
    const long long W = cu[p.c.B];
    const int c1 = blockIdx.x + 1;
    const int u = (int)((long long)c1 * W / p.C);
    if (u >= W || u == 0) return;
    int lo = 0, hi = p.c.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= u) lo = mid; else hi = mid - 1;
    }
    const int b = lo;
    const int2 s = seq_state(p, b);
    const int nt = (s.x + s.y + kKeys - 1) / kKeys, blocks = (s.y + p.pb - 1) / p.pb;
    const int off = u - cu[b], seg = off / nt;
    const int s0 = cu[b] + seg * nt, s1 = s0 + nt;
    if (u == s0 || (int)((long long)(c1 - 1) * W / p.C) > s0) return;  // not cut here, or not the first cut
    const int g = seg / blocks, rb = seg - g * blocks;
    const int t = threadIdx.x & 127, hh = threadIdx.x >> 7;
    const int tok = t / p.r, head = t - tok * p.r;
    const int i = rb * p.pb + (PAIR ? hh * p.pt : 0) + tok;
    if (tok >= p.pt || i >= s.y) return;
    const int col = blockIdx.y * 16;
    // pieces: the one before the first cut, then one for each share that begins inside the segment
    int c = c1 - 1;
    float M = -INFINITY, L = 0.f, acc[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = 0.f;
    for (;; ++c) {
        const int ub = (int)((long long)c * W / p.C), ue = (int)((long long)(c + 1) * W / p.C);
        if (ub >= s1) break;
        if (ub == ue) continue;
        const size_t slot = 2 * (size_t)c + (ub >= s0 ? 0 : 1);
        const float2 v = p.ws_ml[slot * kRecRows + threadIdx.x];
        const float *src = p.ws_o + (slot * D + col) * kRecRows + threadIdx.x;
        float o[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = src[(size_t)e * kRecRows];
        const float Mn = fmaxf(M, v.x);
        if (Mn == -INFINITY) continue;  // nothing seen yet
        const float a = fast_exp2(M - Mn), w = fast_exp2(v.x - Mn);
        L = L * a + w * v.y;
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[e] = acc[e] * a + w * o[e];
        M = Mn;
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
    uint32_t pk[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) pk[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    uint4 *d4 = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) +
                                          (((size_t)b * p.n + i) * p.H + g * p.r + head) * D + col);
    d4[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
    d4[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
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
    if (p.C < 2) return cudaSuccess;
    return dec::launch_pdl(decode_tree_combine<D, PAIR>, dim3(p.C - 1, D / 16), dim3(kRows * (PAIR + 1)), 0, st, p);
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// Row tiles a CTA works on at once: two when one tile does not hold all of a
// KV head's rows.
bool tree_pair(int n, int r) { return n > kRows / r; }

}  // namespace

size_t decode_tree_workspace(int B, int n, int r, int d_h, int num_sms) {
    const size_t rows = (size_t)kRows * (tree_pair(n, r) ? 2 : 1), slots = 2 * (size_t)num_sms;
    return up256((size_t)(B + 1) * 4) + up256(slots * rows * 8) + up256(slots * rows * d_h * 4);
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
    p.ws_cu = reinterpret_cast<int *>(ws);
    ws += up256((size_t)(a.cache.B + 1) * 4);
    p.ws_ml = reinterpret_cast<float2 *>(ws);
    ws += up256(slots * rows * 8);
    p.ws_o = reinterpret_cast<float *>(ws);
    if (a.d_h == 128) return pair ? run_tree<128, 1>(p, tmq, tmk, tmv, st) : run_tree<128, 0>(p, tmq, tmk, tmv, st);
    if (a.d_h == 64) return pair ? run_tree<64, 1>(p, tmq, tmk, tmv, st) : run_tree<64, 0>(p, tmq, tmk, tmv, st);
    return cudaErrorInvalidValue;
}

}  // namespace gqa
