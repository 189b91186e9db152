// attend.cuh -- the attention pipeline that the packed prefill and the
// draft-tree decode share (sm_100a): rows of (token, query head) packed into
// M = 128 tensor-core tiles, pieces of key tiles streamed through shared
// memory, online softmax in tensor memory, persistent CTAs.
//
// Row packing.  The r = H/G query heads of a group read the same K/V head, so
// the rows of one tile are the (token, head) pairs of PT = floor(128 / r)
// consecutive tokens: row = token * r + head.  One TMA box of [64 dims x r
// heads x PT tokens] lays them out in that order.  A few tokens then fill a
// tile as well as many do, whatever r is.
//
// A piece is one or two row tiles against a run of consecutive 128-key tiles.
// A CTA works through pieces that a policy hands to every role in the same
// order, and nothing waits for a piece to end but the row tile's own threads:
// the next piece's Q, K and V are loaded, and its first scores computed, while
// the last one's output is written.
//   PAIR = 1: two row tiles (the two softmax warpgroups, one each) share every
//     key tile.
//   PAIR = 0: one row tile; the warpgroups take alternate key tiles, each with
//     its own maximum, sum and O, merged at the end of the piece.
//
// Roles (384 threads):
//   warps 0-3, 4-7  softmax and epilogue of row tile / key parity 0, 1: one
//                   thread per row = tensor-memory lane
//   warp 8          K tiles and Q rows by TMA
//   warp 11         V tiles by TMA, and what the policy has to do on the side
//   warps 9, 10     tcgen05.mma of row tile / key parity 0, 1: one lane of each issues.
//                   An issuing thread spends a third of a tile's time in checks of
//                   barriers and on instructions between its MMAs; with two of them
//                   one's MMAs fill the other's gaps.
// Tensor memory: S0/P0, S1/P1 (128 columns each), O0, O1 (128 each).  P (bf16)
// overwrites its S block; the S of a later tile is issued behind the P.V that
// reads that P, and MMAs of one thread complete in order.
//
// What bounds it (d_h = 128): one key tile of two row tiles is 2,048 cycles of
// tensor time and takes 3,990, two groups of 16 MMAs at 80-125 cycles each
// beside the other row tile's softmax: 970-973 TFLOP/s on 2 x 8192 tokens and 64
// heads under the power cap (1,113 before it), where prefill.cu has 965-967
// (1,095).  With one row tile the two parities overlap and
// a tile takes the 2,430 cycles that HBM needs for its 64 KB (7.4 TB/s).
#pragma once

#include "common.cuh"
#include "internal.h"
#include "tc.cuh"

namespace gqa {
namespace att {

constexpr int kRows = 128;               // query rows per tile (tensor-memory lanes)
constexpr int kKeys = 128;               // keys per K/V tile
constexpr int kHalf = 128 * 64 * 2;      // one [128 rows x 64 bf16] swizzled box
constexpr int kThreads = 384;            // 3 warpgroups: two of softmax, one of TMA and MMA
// Register split (setmaxnreg): the launch gives every thread kLaunchRegs; the
// TMA/MMA warpgroup drops to kLowRegs, the softmax warpgroups rise to
// kHighRegs.  The launchers check the compiled count, since an .inc beyond the
// launch's total would wait forever.
constexpr int kLaunchRegs = 168;
constexpr int kLowRegs = 136;
constexpr int kHighRegs = 184;
static_assert(2 * 128 * kHighRegs + 128 * kLowRegs <= kThreads * kLaunchRegs, "register split");
constexpr uint32_t kTmemCols = 512;

// Shared memory of the pipeline: NQ buffers of PAIR + 1 Q tiles, ST-stage K
// and V rings, barriers, the (m, l) exchange.  192 KB or less of tiles leaves
// room for the policies' lists.
template <int D, int PAIR>
struct Layout {
    static constexpr int HALVES = D / 64;
    static constexpr int TILE = HALVES * kHalf;  // [128 x D] bf16
    // two Q buffers wherever they fit beside the rings: the next piece's rows then
    // never wait for the last scores of this one
    static constexpr int NQ = (D == 128 && PAIR) ? 1 : 2;
    static constexpr int ST = D == 128 ? 2 : 4;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = NQ * (PAIR + 1) * TILE;
    static constexpr int OFF_V = OFF_K + ST * TILE;
    static constexpr int OFF_BAR = OFF_V + ST * TILE;
    static constexpr int OFF_ML = OFF_BAR + 400;              // [2][128] (m, l) of the two parities
    static constexpr int OFF_POLICY = OFF_ML + (PAIR ? 0 : 2 * 128 * 8);  // what the policy keeps
    static constexpr int SMEM = 1024 + OFF_POLICY;
};

__device__ __forceinline__ void tma_load_4d(void *dst, const void *tmap, uint64_t *bar, int x, int y,
                                            int z, int w, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w),
        "l"(policy)
        : "memory");
}

__device__ __forceinline__ uint64_t f32x2_pack(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void f32x2_unpack(uint64_t v, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t f32x2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t f32x2_add(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Warp-uniform bounded wait: every lane polls; the warp agrees on the result.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, uint64_t limit) {
    const bool ok = mbar_wait(bar, parity, limit);
    return __all_sync(0xffffffffu, ok);
}

// Online softmax of this thread's query row (its tensor-memory lane) over one
// tile of scores at tS: moves the running maximum m (log2 units) and the sum l
// and writes P = 2^(s - m) as bf16 pairs over the scores.
//   - The maximum moves (and O at tO is rescaled) only when it grows by more
//     than 8, so p <= 2^8: numerator and denominator use the same stale one.
//   - `first`: O holds nothing of this row yet.  Otherwise the P.V that last
//     wrote O is complete, because the S just read was issued behind it.
//   - m = -inf (no key seen yet): every score is -inf and p = 0.
//   - The row sum adds the unrounded p in fp32.
// softmax_whole and softmax_part below do this for the two kinds of tile.

// Moves the maximum to cover mx (log2 units) and rescales l and O with it.
template <int D>
__device__ __forceinline__ void move_max(uint32_t tO, float mx, bool first, float &m, float &l) {
    if (first) {
        m = mx;
        l = 0.f;
        return;
    }
    const float mn = fmaxf(m, mx);
    const bool need = mn > m + 8.f;
    if (!__any_sync(0xffffffffu, need)) return;
    float alpha = 1.f;
    if (need) {
        alpha = fast_exp2(m - mn);
        m = mn;
        l *= alpha;
    }
#pragma unroll 1
    for (int c = 0; c < D / 16; ++c) {
        uint32_t orow[16];
        tc::ld16(tO + c * 16, orow);
        tc::wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) orow[e] = __float_as_uint(__uint_as_float(orow[e]) * alpha);
        tc::st16(tO + c * 16, orow);
    }
}

// exp of 32 raw scores and their sum in rs2 (four packed partial sums); bf16 pairs.
__device__ __forceinline__ void exp_chunk(const uint32_t (&sr)[32], uint64_t sc2, uint64_t nm2, uint64_t (&rs2)[4],
                                          uint64_t (*keep)[16], uint32_t (&pk)[16]) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const uint64_t x2 =
            f32x2_fma(f32x2_pack(__uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1])), sc2, nm2);
        float x0, x1;
        f32x2_unpack(x2, x0, x1);
        const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
        const uint64_t p2 = f32x2_pack(p0, p1);
        rs2[e & 3] = f32x2_add(rs2[e & 3], p2);
        if (keep) (*keep)[e] = p2;
        pk[e] = pack_bf16x2(p0, p1);
    }
}

__device__ __forceinline__ float sum_of(const uint64_t (&rs2)[4]) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a0, a1;
        f32x2_unpack(rs2[i], a0, a1);
        sum += a0 + a1;
    }
    return sum;
}

__device__ __forceinline__ float max_chunk(const uint32_t (&sr)[32], float mx) {
    float m4[4] = {mx, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int e = 0; e < 32; ++e) m4[e & 3] = fmaxf(m4[e & 3], __uint_as_float(sr[e]));
    return fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
}

// A whole tile that every row sees; P in columns [0, 64).
template <int D>
__device__ __forceinline__ void softmax_whole(uint32_t tS, uint32_t tO, float scale_log2, bool first, float &m,
                                              float &l) {
    uint32_t sr[4][32];
#pragma unroll
    for (int c = 0; c < 4; ++c) tc::ld32(tS + c * 32, sr[c]);
    tc::wait_ld();
#pragma unroll
    for (int c = 0; c < 4; ++c) tc::hold32(sr[c]);
    float mx4[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) mx4[c] = max_chunk(sr[c], -INFINITY);
    const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * scale_log2;
    const float m0 = first ? mx : m;
    // (the rescale of O, when there is one, comes after P is written: P is what the tensor core waits for)
    const float mn = first ? mx : fmaxf(m, mx);
    const bool need = mn > m0 + 8.f;
    const bool rescale = __any_sync(0xffffffffu, need);
    float alpha = 1.f;
    if (need) alpha = fast_exp2(m0 - mn);
    m = need ? mn : m0;
    const float mu = m == -INFINITY ? 0.f : m;
    const uint64_t sc2 = f32x2_pack(scale_log2, scale_log2), nm2 = f32x2_pack(-mu, -mu);
    uint64_t rs2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint32_t pk[16];
        exp_chunk(sr[c], sc2, nm2, rs2, nullptr, pk);
        tc::st16(tS + c * 16, pk);
    }
    if (rescale) {
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
            uint32_t orow[16];
            tc::ld16(tO + c * 16, orow);
            tc::wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) orow[e] = __float_as_uint(__uint_as_float(orow[e]) * alpha);
            tc::st16(tO + c * 16, orow);
        }
    }
    l = (first ? 0.f : l * alpha) + sum_of(rs2);
    tc::wait_st();
}

// Any other tile: only its first 32 * nch keys, of which bit e of words(c)
// says whether the row sees key 32 c + e.  P of chunk c stays in the chunk's
// own 32 columns: P_hi in the first 16 and, with `split`, P_lo = p - P_hi in
// the next 16 (two bf16 terms, about 16 significant bits: for rows that see so
// few keys that the rounding of P does not average out).  Two passes over the
// chunks in a rolled loop: a short tile costs what it holds, and the code stays
// small (unrolled, these paths were 38 KB of instructions, which every launch
// fetched anew).
template <int D, typename Words>
__device__ __forceinline__ void softmax_part(uint32_t tS, uint32_t tO, float scale_log2, bool first, bool split,
                                             int nch, float &m, float &l, Words words) {
    auto load = [&](int c, uint32_t (&sr)[32]) {
        tc::ld32(tS + c * 32, sr);
        const uint32_t w = words(c);
        tc::wait_ld();
        tc::hold32(sr);
#pragma unroll
        for (int e = 0; e < 32; ++e)
            if (!((w >> e) & 1u)) sr[e] = __float_as_uint(-INFINITY);
    };
    float mx = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < nch; ++c) {
        uint32_t sr[32];
        load(c, sr);
        mx = max_chunk(sr, mx);
    }
    move_max<D>(tO, mx * scale_log2, first, m, l);
    const float mu = m == -INFINITY ? 0.f : m;
    const uint64_t sc2 = f32x2_pack(scale_log2, scale_log2), nm2 = f32x2_pack(-mu, -mu);
    uint64_t rs2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll 1
    for (int c = 0; c < nch; ++c) {
        uint32_t sr[32], pk[16];
        uint64_t p2[16];
        load(c, sr);
        exp_chunk(sr, sc2, nm2, rs2, &p2, pk);
        tc::st16(tS + c * 32, pk);
        if (split) {
            const uint64_t minus1 = f32x2_pack(-1.f, -1.f);
#pragma unroll
            for (int e = 0; e < 16; ++e) {  // p - P_hi is exact in fp32
                const uint64_t hi = f32x2_pack(__uint_as_float(pk[e] << 16), __uint_as_float(pk[e] & 0xffff0000u));
                float r0, r1;
                f32x2_unpack(f32x2_fma(hi, minus1, p2[e]), r0, r1);
                pk[e] = pack_bf16x2(r0, r1);
            }
            tc::st16(tS + c * 32 + 16, pk);
        }
    }
    l += sum_of(rs2);
    tc::wait_st();
}

// Writes 8 NP values of each lane's row (bf16 pairs in w, NP pieces of 16
// bytes) to out + row * D + col; row < 0: nothing.  NP lanes first exchange
// their pieces (a transpose by shuffles), so that each store instruction
// covers 16 NP consecutive bytes of a row: one thread storing its own row
// touches 32 lines per instruction, and those stores took 2.2 us of a
// [2 x 128 x 128] epilogue.
template <int D, int NP>
__device__ __forceinline__ void store_rows(__nv_bfloat16 *out, int row, int col, uint32_t (&w)[4 * NP]) {
    const int lane = threadIdx.x & 31, a = lane & (NP - 1);
#pragma unroll
    for (int s = 1; s < NP; s <<= 1) {
        const bool up = (lane & s) != 0;
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            if (k & s) continue;
            // pieces k and k | s: this lane keeps the one on its side and gives the other
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t &lo = w[4 * k + i], &hi = w[4 * (k | s) + i];
                const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? lo : hi, s);
                if (up) lo = got; else hi = got;
            }
        }
    }
    // piece k now is piece a of the row of lane (lane & ~(NP - 1)) + k
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        const int rk = __shfl_sync(0xffffffffu, row, (lane & ~(NP - 1)) + k);
        if (rk >= 0)
            *reinterpret_cast<uint4 *>(out + (size_t)rk * D + col + a * 8) =
                make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
    }
}

// What the pipeline needs to know of a piece; policies add their own.
struct PieceBase {
    // keys of row tile 0 and 1, from the first key of the piece's first tile on (0:
    // the tile has no rows).  Row tile i visits ceil(k_i / 128) tiles.
    int k0, k1;
    __device__ int tiles() const { return (max(k0, k1) + kKeys - 1) / kKeys; }
};

__device__ __forceinline__ int chunks_of(int keys, int j) {  // 32-key chunks of tile j that hold keys
    return min(4, (keys - j * kKeys + 31) / 32);
}

template <int D, int PAIR>
struct Barriers {
    static constexpr int ST = Layout<D, PAIR>::ST;
    // Arrivals that release a K or V stage: both issuers use every tile of a pair
    // (one that has nothing to do with a tile arrives without an MMA), one uses a
    // tile otherwise.
    static constexpr int USERS = PAIR ? 2 : 1;
    uint64_t *q_full, *q_empty;                          // [2] (NQ used)
    uint64_t *k_full, *k_empty, *v_full, *v_empty;       // [ST]
    uint64_t *s_full, *p_ready;                          // [2] per softmax warpgroup
    // [2] a piece's last P.V of row tile / parity i is complete; only for pieces that have
    // one.  No later phase can complete before both warpgroups have seen this one, since it
    // takes a P that warpgroup i writes after this piece's epilogue.
    uint64_t *o_done;
    uint64_t *meet;                                      // the two warpgroups (PAIR = 0)
    uint64_t *drain;                                     // [2] one per issuer
    uint64_t *turn;                                      // [2] issuer i may go on
    uint64_t *policy;                                    // [16]
    uint32_t *tmem_slot;
    int *abort_flag;
    __device__ explicit Barriers(uint8_t *sm) {
        uint64_t *b = reinterpret_cast<uint64_t *>(sm + Layout<D, PAIR>::OFF_BAR);
        q_full = b;
        q_empty = b + 2;
        s_full = b + 4;
        p_ready = b + 6;
        o_done = b + 8;
        meet = b + 10;
        drain = b + 46;
        k_full = b + 12;
        k_empty = k_full + ST;
        v_full = k_empty + ST;
        v_empty = v_full + ST;
        policy = b + 28;
        tmem_slot = reinterpret_cast<uint32_t *>(b + 44);
        abort_flag = reinterpret_cast<int *>(b + 45);
        turn = b + 48;
    }
    __device__ void init() const {  // one thread
        for (int s = 0; s < 2; ++s) {
            mbar_init(&q_full[s], 1);
            mbar_init(&q_empty[s], 2);
            mbar_init(&drain[s], 1);
            mbar_init(&turn[s], 1);
            mbar_init(&s_full[s], 1);
            mbar_init(&p_ready[s], 128);
            mbar_init(&o_done[s], 1);
        }
        for (int s = 0; s < ST; ++s) {
            mbar_init(&k_full[s], 1);
            mbar_init(&k_empty[s], USERS);
            mbar_init(&v_full[s], 1);
            mbar_init(&v_empty[s], USERS);
        }
        mbar_init(meet, 256);
        *abort_flag = 0;
    }
};

// Everything after set-up: all threads of the CTA, tensor memory allocated at
// `tmem`.  Pol is the policy:
//   Pol::Piece                    a PieceBase with more: split(row tile) says whether its P is carried
//                                 as two bf16 terms
//   Pol::Iter(pol, whole_warp)    walks the CTA's pieces: bool next(Piece &), the same for all lanes
//                                 when a whole warp calls it, and done() when the calling role is
//                                 through with a piece (one call per piece)
//   pol.kv(piece, tile, K or V, stage address, barrier, lane)  loads of a tile, by a whole warp
//   pol.kv_look(piece, tile, lane)  what kv() needs from memory, asked for before the stage is free
//   pol.q(piece, row tile, address, barrier)  loads of Q rows, by one lane; pol.q_bytes() each
//   pol.masked(piece, row tile, tile)  whether some row does not see all of a key tile
//   pol.row(piece, row tile, row)  -> Pol::Row, the thread's row; its out_row: row of `out`, or -1
//   pol.words(piece, row, tile, c)  what the row sees of the 32 keys of chunk c, as bits
//   pol.clear_from(piece, row, tile), pol.clears(piece, row, tile, key)  V rows of the tile that
//                                 nobody sees: the first that may be one (128: none), and which are
//   pol.side(lane)                called by warp 11 before each of its pieces
//   pol.record(piece)             null, or where this piece's partial results go (D x rows floats,
//                                 column-major), and pol.record_ml(piece)
template <int D, int PAIR, typename Pol>
__device__ __forceinline__ void attend(Pol &pol, uint8_t *sm, uint32_t tmem) {
    using Lay = Layout<D, PAIR>;
    using Piece = typename Pol::Piece;
    constexpr int HALVES = Lay::HALVES, kTile = Lay::TILE, NQ = Lay::NQ, ST = Lay::ST;
    constexpr int kRecRows = kRows * (PAIR + 1);
    const Barriers<D, PAIR> bar(sm);
    volatile int *vabort = bar.abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint64_t limit = pol.timeout_ns;

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLowRegs));
        if (warp == 8 || warp == 11) {
            // ------------------------------------------------ TMA producers
            const bool is_k = warp == 8;
            uint64_t *full = is_k ? bar.k_full : bar.v_full, *empty = is_k ? bar.k_empty : bar.v_empty;
            uint8_t *ring = sm + (is_k ? Lay::OFF_K : Lay::OFF_V);
            typename Pol::Iter walk(pol, true);
            Piece q;
            bool ok = true;
            int it = 0, piece = 0;
            for (;;) {
                if (!is_k) pol.side(lane);
                if (!ok || !walk.next(q)) break;
                const int n = q.tiles();
                for (int j = 0; j < n && ok; ++j, ++it) {
                    const int st = it % ST;
                    const auto where = pol.kv_look(q, j, lane);
                    if (__any_sync(0xffffffffu, *vabort != 0) || !warp_wait(&empty[st], ((it / ST) & 1) ^ 1, limit)) {
                        if (lane == 0) set_status(pol.status, STATUS_TIMEOUT);
                        *vabort = 1;
                        ok = false;
                        break;
                    }
                    if (lane == 0) mbar_arrive_expect_tx(&full[st], kTile);
                    __syncwarp();
                    pol.kv(q, j, where, is_k, ring + st * kTile, &full[st], lane);
                    if (is_k && j == 0) {
                        // the piece's query rows, into the buffer that the scores of NQ pieces ago released
                        const int qb = piece % NQ;
                        if (!warp_wait(&bar.q_empty[qb], ((piece / NQ) & 1) ^ 1, limit)) {
                            if (lane == 0) set_status(pol.status, STATUS_TIMEOUT);
                            *vabort = 1;
                            ok = false;
                        } else {
                            if (lane == 0) {
                                const int nh = PAIR && q.k1 > 0 ? 2 : 1;
                                mbar_arrive_expect_tx(&bar.q_full[qb], nh * HALVES * pol.q_bytes());
                                for (int hh = 0; hh < nh; ++hh)
                                    pol.q(q, hh, sm + Lay::OFF_Q + (qb * (PAIR + 1) + hh) * kTile, &bar.q_full[qb]);
                            }
                            ++piece;
                        }
                        __syncwarp();
                    }
                }
                walk.done();
            }
            // no copy is in flight when the CTA leaves, whatever the other warps did
            for (int i = max(0, it - ST); i < it; ++i) warp_wait(&full[i % ST], (i / ST) & 1, limit);
            if (is_k)
                for (int i = max(0, piece - NQ); i < piece; ++i)
                    warp_wait(&bar.q_full[i % NQ], (i / NQ) & 1, limit);
        } else if (lane == 0) {
            // ------------------------------------------------ MMA issuers, warps 9 and 10
            const int hh = warp - 9;
            constexpr uint32_t idesc_s = tc::idesc_bf16(128, 128, false, false);
            constexpr uint32_t idesc_o = tc::idesc_bf16(128, D, false, true);
            bool issued = false, ok = true;
            // Spins (a suspended thread resumed ~600 cycles late); the abort flag and the time are
            // looked at only while there is something to wait for.
            auto wait = [&](uint64_t *b, uint32_t par) {
                if (mbar_test_wait(b, par)) return true;
                const uint64_t t0 = global_timer_ns();
                for (;;) {
                    for (int i = 0; i < 64; ++i)
                        if (mbar_test_wait(b, par)) return true;
                    if (*vabort || global_timer_ns() - t0 > limit) break;
                }
                set_status(pol.status, STATUS_TIMEOUT);
                ok = false;
                *vabort = 1;
                return false;
            };
            const uint64_t dq = tc::sdesc_sw128(smem_u32(sm + Lay::OFF_Q), 16, 1024);
            const uint64_t dk = tc::sdesc_sw128(smem_u32(sm + Lay::OFF_K), 16, 1024);
            const uint64_t dv = tc::sdesc_sw128(smem_u32(sm + Lay::OFF_V), kHalf, 1024);
            const uint32_t tS = tmem + hh * 128, tO = tmem + 256 + hh * 128;
            // Two walks over the tiles: the scores' runs ahead of P.V's by LOOK tiles, across
            // pieces.  Round k issues P.V of tile k - LOOK and S of tile k, where they are this
            // issuer's.  What the round needs is looked up and waited for before its wait for P:
            // from there to the S is on every tile's critical path.
            // In pieces of kTurnTiles or more the issuers of a pair take turns, a group [P.V of one
            // tile, S of the next] each.  Left to themselves they fall into step: both softmaxes
            // then share the SM's issue slots, both groups the tensor core, and neither overlaps the
            // other (4,800 cycles a tile against 3,990; passing the turn on before the S took 4,300,
            // one thread for both row tiles 4,400).  In short pieces the order only costs (89 against
            // 87 us for 96 short prompts).  With alternate key tiles each round is one issuer's.
            constexpr int kTurnTiles = 4;
            constexpr int LOOK = PAIR ? 1 : 2;
            typename Pol::Iter sw(pol, false), vw(pol, false);
            Piece sq, vq;
            int s_j = 0, s_n = 0, s_piece = -1, v_j = 0, v_n = 0, cnt = 0, turns = 0;
            bool more = true;
            for (int k = 0; ok; ++k) {
                const int it = k - LOOK, vs = it & (ST - 1), ks = k & (ST - 1);
                bool pv = it >= 0, mine = false, last = false;
                int nch = 0;
                if (pv) {
                    if (v_j == v_n) {
                        if (!vw.next(vq)) break;
                        v_j = 0;
                        v_n = vq.tiles();
                    }
                    const int keys = PAIR && hh ? vq.k1 : vq.k0;
                    mine = PAIR ? keys > v_j * kKeys : (it & 1) == hh;
                    last = PAIR ? keys <= (v_j + 1) * kKeys : v_j + 2 >= v_n;
                    // how P lies in its S block: 0 as softmax_whole left it, else softmax_part's chunks
                    nch = chunks_of(keys, v_j);
                    if (nch == 4 && !vq.split(PAIR ? hh : 0) && !pol.masked(vq, PAIR ? hh : 0, v_j)) nch = 0;
                    if ((PAIR || mine) && !wait(&bar.v_full[vs], (it / ST) & 1)) break;
                }
                // the next scores, unless they open a piece: its Q may still be on its way, and
                // P.V does not wait for that
                bool s_ready = more && s_j < s_n;
                const bool act = PAIR || (k & 1) == hh;  // this issuer's round
                if (s_ready && act && !wait(&bar.k_full[ks], (k / ST) & 1)) break;
                if (mine && !wait(&bar.p_ready[hh], cnt++ & 1)) break;
                const bool turn = PAIR ? pv && v_n >= kTurnTiles : act;  // the same for both
                if (turn && (hh == 1 || turns > 0) && !wait(&bar.turn[hh], (turns - 1 + hh) & 1)) break;
                if (mine) {
                    tc::fence_after();
                    const uint64_t d = dv + ((vs * kTile) >> 4);
                    const bool acc = PAIR ? v_j > 0 : v_j >= 2;
                    // O += P V, two K-steps of 16 keys per chunk
                    if (nch == 0) {
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            tc::mma_ts(tO, tS + kk * 8, d + ((kk * 2048) >> 4), idesc_o, (acc || kk > 0) ? 1u : 0u);
                    } else {
#pragma unroll 1
                        for (int lo = 0; lo <= (vq.split(PAIR ? hh : 0) ? 16 : 0); lo += 16)
#pragma unroll 1
                            for (int kk = 0; kk < 2 * nch; ++kk)
                                tc::mma_ts(tO, tS + (kk >> 1) * 32 + (kk & 1) * 8 + lo, d + ((kk * 2048) >> 4),
                                           idesc_o, (acc || lo > 0 || kk > 0) ? 1u : 0u);
                    }
                    if (last) tc::commit(&bar.o_done[hh]);
                }
                // S = Q K^T of tile k: D / 16 K-steps over d_h.  A piece's first one comes after the
                // turn is passed on, since it may have to wait.
                const bool opens = !s_ready;
                if (opens) {
                    if (turn) mbar_arrive(&bar.turn[hh ^ 1]);
                    if (more) more = sw.next(sq);
                    if (more) {
                        ++s_piece;
                        s_j = 0;
                        s_n = sq.tiles();
                        if (!wait(&bar.q_full[s_piece % NQ], (s_piece / NQ) & 1)) break;
                        if (act && !wait(&bar.k_full[ks], (k / ST) & 1)) break;
                        s_ready = true;
                    }
                }
                if (s_ready) {
                    const bool on = PAIR ? (hh ? sq.k1 : sq.k0) > s_j * kKeys : act;
                    if (on) {
                        const uint64_t q = dq + ((((s_piece % NQ) * (PAIR + 1) + (PAIR ? hh : 0)) * kTile) >> 4);
                        const uint64_t kd = dk + ((ks * kTile) >> 4);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
                            tc::mma_ss(tS, q + off, kd + off, idesc_s, kk > 0 ? 1u : 0u);
                        }
                        tc::commit(&bar.s_full[hh]);
                        issued = true;
                        tc::commit(&bar.k_empty[ks]);
                    } else if (PAIR) {
                        mbar_arrive(&bar.k_empty[ks]);
                    }
                    if (++s_j == s_n) tc::commit(&bar.q_empty[s_piece % NQ]);
                }
                if (turn) {
                    if (!opens) mbar_arrive(&bar.turn[hh ^ 1]);
                    ++turns;
                }
                if (pv) {
                    if (mine) tc::commit(&bar.v_empty[vs]);
                    else if (PAIR) mbar_arrive(&bar.v_empty[vs]);
                    if (++v_j == v_n) vw.done();
                }
            }
            if (issued && !ok) {  // let MMAs already issued finish before TMEM is freed
                tc::commit(&bar.drain[hh]);
                mbar_wait(&bar.drain[hh], 0, limit);
            }
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kHighRegs));
        // ------------------------------------------------ softmax + epilogue
        const int hh = warp >> 2;          // row tile (PAIR) or key-tile parity
        const int t = threadIdx.x & 127;   // row = tensor-memory lane
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_off + hh * 128;
        const uint32_t tO = tmem + lane_off + 256 + hh * 128;
        float2 *ml = reinterpret_cast<float2 *>(sm + Lay::OFF_ML);
        typename Pol::Iter walk(pol, true);
        bool ok = true;
        int it = 0, cnt = 0, met = 0, now_it = 0, now_n = 0;
        int done[2] = {0, 0};  // pieces seen through o_done
        auto both_meet = [&]() {  // bounded: false when the wait ran out
            mbar_arrive(bar.meet);
            return warp_wait(bar.meet, met++ & 1, limit);
        };
        // Writes a piece's output, or its partial record; sets ok when a wait runs out.
        auto epilogue = [&](const Piece &now, int out_row, float m, float l) {
            const int keys = PAIR && hh ? now.k1 : now.k0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                // the row tile's own last P.V, or both parities' where the piece has them
                if (PAIR ? i != hh || keys == 0 : now_n < 2 && (now_it & 1) != i) continue;
                if (!warp_wait(&bar.o_done[i], done[i]++ & 1, limit)) {
                    ok = false;
                    return;
                }
            }
            tc::fence_after();
            float *rec = pol.record(now);
            // columns [c0, c0 + NC) of O, or of the merge of both parities' O
            constexpr int NC = PAIR ? D : D / 2, CH = NC < 64 ? NC : 64;
            float w0 = 1.f, w1 = 0.f, M = m, L = l;
            uint32_t tA = tO;
            int c0 = 0;
            if constexpr (!PAIR) {
                ml[hh * kRows + t] = make_float2(m, l);
                if (!both_meet()) {
                    ok = false;
                    return;
                }
                const float2 a = ml[t], b = ml[kRows + t];
                M = fmaxf(a.x, b.x);
                w0 = a.x == -INFINITY ? 0.f : fast_exp2(a.x - M);
                w1 = b.x == -INFINITY ? 0.f : fast_exp2(b.x - M);
                L = w0 * a.y + w1 * b.y;
                tA = tmem + lane_off + 256;
                c0 = hh * NC;
            }
            if (!PAIR || keys > 0) {
                if (!rec) {
                    // (L = 0: the row sees nothing; a NaN, from a score that is NaN or +inf, stays one)
                    const float inv = L == 0.f ? 0.f : 1.f / L;
                    w0 *= inv;
                    w1 *= inv;
                }
#pragma unroll 1
                for (int c = c0; c < c0 + NC; c += CH) {
                    uint32_t pk[CH / 2];
#pragma unroll
                    for (int cc = 0; cc < CH; cc += 32) {
                        uint32_t oa[32], ob[32];
                        tc::ld32(tA + c + cc, oa);
                        if constexpr (!PAIR) tc::ld32(tA + 128 + c + cc, ob);
                        tc::wait_ld();
                        tc::hold32(oa);
                        if constexpr (!PAIR) tc::hold32(ob);
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            // (a parity without a key holds an O that was never written)
                            float v0 = w0 != 0.f ? w0 * __uint_as_float(oa[e]) : 0.f;
                            float v1 = w0 != 0.f ? w0 * __uint_as_float(oa[e + 1]) : 0.f;
                            if constexpr (!PAIR) {
                                v0 = w1 != 0.f ? fmaf(w1, __uint_as_float(ob[e]), v0) : v0;
                                v1 = w1 != 0.f ? fmaf(w1, __uint_as_float(ob[e + 1]), v1) : v1;
                            }
                            if (rec) {
                                // column-major: a warp's stores are 128 bytes in a row
                                float *d = rec + (size_t)(c + cc + e) * kRecRows + (PAIR ? hh * kRows : 0) + t;
                                if (out_row >= 0) {
                                    d[0] = v0;
                                    d[kRecRows] = v1;
                                }
                            }
                            pk[(cc + e) / 2] = pack_bf16x2(v0, v1);
                        }
                    }
                    if (!rec) store_rows<D, CH / 8>(pol.out, out_row, c, pk);
                }
                if (rec && (PAIR || hh == 0) && out_row >= 0)
                    pol.record_ml(now)[(PAIR ? hh * kRows : 0) + t] = make_float2(M, L);
            }
            walk.done();
            tc::fence_before();
            if constexpr (!PAIR) {  // both have read both O before either is written again
                if (!both_meet()) ok = false;
            }
        };
        Piece q, now;
        typename Pol::Row row = {};
        int out_row = -1;
        float m = -INFINITY, l = 0.f;
        bool open = false;  // `now` waits for its epilogue
        while (ok) {
            // the next piece and its row are looked up while the last P.V of the one before runs
            const bool have = walk.next(q);
            if (have) row = pol.row(q, PAIR ? hh : 0, t);
            if (open) epilogue(now, out_row, m, l);
            open = have && ok;
            if (!open) break;
            const int n = q.tiles(), keys = PAIR && hh ? q.k1 : q.k0;
            now_it = it;
            now_n = n;
            m = -INFINITY;
            l = 0.f;
            bool first = true;
            for (int j = 0; j < n; ++j, ++it) {
                if (PAIR ? j * kKeys >= keys : (it & 1) != hh) continue;
                const bool aborted = __any_sync(0xffffffffu, *vabort != 0);
                if (aborted || !warp_wait(&bar.s_full[hh], cnt & 1, limit)) {
                    ok = false;
                    break;
                }
                ++cnt;
                tc::fence_after();
                const int nch = chunks_of(keys, j);
                if (nch == 4 && !q.split(PAIR ? hh : 0) && !pol.masked(q, PAIR ? hh : 0, j)) {
                    softmax_whole<D>(tS, tO, pol.scale_log2, first, m, l);
                } else {
                    softmax_part<D>(tS, tO, pol.scale_log2, first, q.split(PAIR ? hh : 0), nch, m, l,
                                    [&](int c) { return pol.words(q, row, j, c); });
                    // V rows that no row of the piece sees, those past the sequence's end among them:
                    // P is 0 there, but 0 times what they hold must stay 0.  Each warpgroup clears
                    // those that its P.V reads, ahead of it (both may write zeros over zeros); the
                    // stage cannot be refilled before that P.V.
                    const int r0 = pol.clear_from(q, row, j), r1 = 32 * nch;
                    if (r0 < r1) {
                        if (!warp_wait(&bar.v_full[it % ST], (it / ST) & 1, limit)) {
                            ok = false;
                            break;
                        }
                        uint8_t *tile = sm + Lay::OFF_V + (it % ST) * kTile;
                        for (int i = t; i < (r1 - r0) * HALVES * 8; i += 128) {
                            const int rr = r0 + i / (HALVES * 8), rem = i % (HALVES * 8);
                            if (!pol.clears(q, row, j, rr)) continue;
                            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(
                                             smem_u32(tile + (rem >> 3) * kHalf + rr * 128 + (rem & 7) * 16)),
                                         "r"(0u)
                                         : "memory");
                        }
                        fence_proxy_async_smem();
                    }
                }
                first = false;
                tc::fence_before();
                mbar_arrive(&bar.p_ready[hh]);
            }
            now = q;
            out_row = row.out_row;
        }
        if (!ok && lane == 0) {
            set_status(pol.status, STATUS_TIMEOUT);
            *vabort = 1;
        }
    }
}

// Exclusive sums cu[0..n) of f(i), and the whole in cu[n], by all kThreads
// threads of the block; scratch holds 32 ints.  Ends with a barrier.
template <typename F>
__device__ __forceinline__ int block_prefix(int n, int *cu, int *scratch, F f) {
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int chunk = (n + kThreads - 1) / kThreads;
    const int i0 = min(n, tid * chunk), i1 = min(n, i0 + chunk);
    int local = 0;
    for (int i = i0; i < i1; ++i) {
        const int x = f(i);
        cu[i] = x;
        local += x;
    }
    int incl = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) scratch[wid] = incl;
    __syncthreads();
    int run = incl - local;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) run += w < wid ? scratch[w] : 0;
    for (int i = i0; i < i1; ++i) {
        const int x = cu[i];
        cu[i] = run;
        run += x;
    }
    if (tid == kThreads - 1) cu[n] = run;
    __syncthreads();
    return cu[n];
}

}  // namespace att
}  // namespace gqa
