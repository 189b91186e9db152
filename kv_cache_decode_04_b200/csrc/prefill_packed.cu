// prefill_packed.cu -- causal GQA attention over prompts of different lengths
// packed into one token axis, on the 5th-generation tensor cores (sm_100a).
//
// What is computed: with sequence b = positions [cu[b], cu[b+1]) of the packed
// axis, for each of its positions s and query head i, g = i / (H/G),
//     out[s,i] = sum_{cu[b] <= t <= s} softmax_t(scale * q[s,i] . k[t,g]) v[t,g]
// (with a window W > 0: s - W < t <= s).
//
// The pipeline is attend.cuh's with two row tiles (PAIR = 1): a piece is 2 *
// floor(128 / r) consecutive positions of one sequence, all r heads of one
// group, against the key tiles that they see.
//
// Work list.  The lengths are on the device, so warp 11 of each CTA finds the
// CTA's pieces from cu as it goes and passes them to the other roles through a
// ring in shared memory.  Pieces are ordered by their index x within the
// sequence, the largest first, so that the ones with the most keys start first
// whatever sequence they belong to, and dealt out in turns, forward and
// backward alternately, so that no CTA gets the longest of every turn.  With
// the pieces of each sequence counted once in shared memory, a step from one
// index to the next is one warp-wide count of the sequences that reach it.
#include <climits>

#include "attend.cuh"
#include "decode_common.cuh"

namespace gqa {

namespace {

using namespace att;

constexpr int kRing = 8;   // pieces between the list and the slowest role
constexpr int kAhead = 3;  // entries filled ahead of warp 11's own

struct PackedParams {
    const int32_t *cu;
    void *out;
    unsigned *status;
    float scale_log2;
    int B, N, H, G, r;
    int pt;  // positions per 128-row tile, floor(128 / r)
    unsigned long long timeout_ns;
    int window;
};

template <int D>
struct PackedPolicy {
    static constexpr int PAIR = 1;
    using Lay = Layout<D, PAIR>;

    const PackedParams &p;
    const CUtensorMap *tmq, *tmk, *tmv;
    int4 *ring;           // [kRing] (first packed position, length, first position, group); group < 0: no more
    uint64_t *filled, *taken;  // [kRing]
    int *counts;          // [B] pieces of each sequence (per group)
    bool falls;           // some entry of cu is below the one before it
    volatile int *vabort;
    unsigned *status;
    float scale_log2;
    __nv_bfloat16 *out;
    uint64_t timeout_ns;
    uint64_t pol_q, pol_kv;

    struct Piece : PieceBase {
        int start, len, s0, g, j_lo;
        bool split0, split1;
        __device__ bool split(int hh) const { return hh ? split1 : split0; }
    };
    struct Row {
        int pos, key_lo, out_row;
    };

    // Start and length of sequence b: offsets are forced into [0, N] and, where some fall, up to
    // the largest before them, so that no row belongs to two sequences.
    static __device__ __forceinline__ int2 span(const PackedParams &p, int b, bool falls) {
        int a = min(max(p.cu[b], 0), p.N);
        if (falls) {
#pragma unroll 1
            for (int i = 0; i < b; ++i) a = max(a, min(p.cu[i], p.N));
        }
        return make_int2(a, max(min(p.cu[b + 1], p.N), a) - a);
    }

    // The consumers of a ring entry: the two TMA warps, the two MMA threads, the softmax warps.
    static constexpr int kConsumers = 12;

    struct Iter {
        PackedPolicy &pol;
        const bool whole;
        int i = 0, finished = 0;
        __device__ Iter(PackedPolicy &pol_, bool whole_warp) : pol(pol_), whole(whole_warp) {}
        __device__ bool next(Piece &q) {
            const PackedParams &p = pol.p;
            const int slot = i % kRing;
            bool ok = *pol.vabort == 0 && mbar_wait(&pol.filled[slot], (i / kRing) & 1, pol.timeout_ns);
            if (whole) ok = __all_sync(0xffffffffu, ok);
            if (!ok) {
                set_status(pol.status, STATUS_TIMEOUT);
                *pol.vabort = 1;
                return false;
            }
            const int4 e = pol.ring[slot];
            if (e.w < 0) return false;
            ++i;
            q.start = e.x;
            q.len = e.y;
            q.s0 = e.z;
            q.g = e.w;
            // keys from the first one that the window leaves to the first row, on a tile border
            q.j_lo = p.window > 0 ? max(0, q.s0 - p.window + 1) / kKeys : 0;
            const int base = q.j_lo * kKeys;
            q.k0 = min(q.len, q.s0 + p.pt) - base;
            q.k1 = q.s0 + p.pt < q.len ? min(q.len, q.s0 + 2 * p.pt) - base : 0;
            // as in the dense prefill: P as two terms for the rows of positions 0 to 127 (a tile
            // that holds one of them) and in narrow windows
            const bool narrow = p.window > 0 && p.window <= 256;
            q.split0 = q.s0 < kKeys || narrow;
            q.split1 = q.s0 + p.pt < kKeys || narrow;
            return true;
        }
        __device__ void done() {
            if ((threadIdx.x & 31) == 0) mbar_arrive(&pol.taken[finished % kRing]);
            ++finished;
        }
    };

    struct Where {};
    __device__ Where kv_look(const Piece &, int, int) { return {}; }
    __device__ void kv(const Piece &q, int j, Where, bool is_k, uint8_t *dst, uint64_t *bar, int lane) {
        if (lane == 0)
            for (int half = 0; half < Lay::HALVES; ++half)
                tma_load_3d(dst + half * kHalf, is_k ? tmk : tmv, bar, half * 64, q.g,
                            q.start + (q.j_lo + j) * kKeys, pol_kv);
    }
    __device__ int q_bytes() const { return p.pt * p.r * 128; }
    __device__ void q(const Piece &q, int hh, uint8_t *dst, uint64_t *bar) {
        for (int half = 0; half < Lay::HALVES; ++half)
            tma_load_3d(dst + half * kHalf, tmq, bar, half * 64, q.g * p.r, q.start + q.s0 + hh * p.pt, pol_q);
    }
    __device__ Row row(const Piece &q, int hh, int t) const {
        const int tok = t / p.r, head = t - tok * p.r;
        Row w;
        w.pos = q.s0 + hh * p.pt + tok;
        w.key_lo = p.window > 0 ? w.pos - p.window + 1 : INT_MIN;
        const bool ok = tok < p.pt && w.pos < q.len &&
                        index_ok(q.start + w.pos < p.N && q.g * p.r + head < p.H, status);
        w.out_row = ok ? (q.start + w.pos) * p.H + q.g * p.r + head : -1;
        return w;
    }
    __device__ bool masked(const Piece &q, int hh, int j) const {
        const int key0 = (q.j_lo + j) * kKeys, first = q.s0 + hh * p.pt;
        return key0 + kKeys - 1 > first || (p.window > 0 && key0 < first + p.pt - p.window);
    }
    __device__ uint32_t words(const Piece &q, const Row &w, int j, int c) const {
        const int key0 = (q.j_lo + j) * kKeys + c * 32;
        const int hi = w.pos - key0, lo = max(w.key_lo, 0) - key0;  // keys [lo, hi] of the chunk
        uint32_t bits = hi < 0 ? 0u : hi >= 31 ? 0xffffffffu : (2u << hi) - 1u;
        if (lo > 0) bits &= lo > 31 ? 0u : 0xffffffffu << lo;
        return bits;
    }
    // keys past the sequence's end
    __device__ int clear_from(const Piece &q, const Row &, int j) const { return q.len - (q.j_lo + j) * kKeys; }
    __device__ bool clears(const Piece &, const Row &, int, int) const { return true; }
    __device__ float *record(const Piece &) const { return nullptr; }
    __device__ float2 *record_ml(const Piece &) const { return nullptr; }

    // The list's state, in warp 11.
    struct List {
        int i = 0;      // entries filled
        int x, at;      // the level: pieces of index x; how many sequences (of one group) have one
        int below = 0;  // pieces of the levels before
        int b0 = 0, seen = 0;  // the level's scan: sequences before b0, `seen` of them in the level
        bool begun = false, ended = false;
    } list;

    // Keeps the ring a few entries ahead of warp 11's own walk.  (Filling entry i waits
    // until every role is through with entry i - kRing, which none of them needs this
    // warp for: it has long loaded that piece.)
    __device__ void side(int lane) {
        const int p2 = 2 * p.pt, B = p.B, C = gridDim.x;
        auto reach = [&](int x) {  // sequences with a piece of index x
            int n = 0;
            for (int b = lane; b < B; b += 32) n += counts[b] > x ? 1 : 0;
            return (int)__reduce_add_sync(0xffffffffu, n);
        };
        List &s = list;
        if (!s.begun) {
            int top = 0;
            for (int b = lane; b < B; b += 32) top = max(top, counts[b]);
            s.x = __reduce_max_sync(0xffffffffu, top) - 1;
            s.at = s.x >= 0 ? reach(s.x) : 0;
        }
        const int until = s.begun ? s.i + 1 : kAhead;
        s.begun = true;
        for (; s.i < until && !s.ended; ++s.i) {
            const int i = s.i;
            // the CTA's i-th piece: turns run forward and backward
            const int u = i * C + ((i & 1) ? C - 1 - (int)blockIdx.x : (int)blockIdx.x);
            const int v = u / p.G;
            while (s.x >= 0 && v >= s.below + s.at) {
                s.below += s.at;
                --s.x;
                s.at = s.x >= 0 ? reach(s.x) : 0;
                s.b0 = s.seen = 0;
            }
            // the (v - below)-th sequence of the level: the lane that holds it writes the entry
            int4 e = make_int4(0, 0, 0, -1);
            bool found = false;
            while (s.x >= 0) {  // (ends: the level has more than v - below sequences)
                const int b = s.b0 + lane;
                const unsigned has = __ballot_sync(0xffffffffu, b < B && counts[b] > s.x);
                const int n = __popc(has), k = v - s.below - s.seen;
                if (k < n) {
                    found = ((has >> lane) & 1u) && __popc(has & ((1u << lane) - 1u)) == k;
                    if (found) {
                        const int2 w = span(p, b, falls);
                        e = make_int4(w.x, w.y, s.x * p2, u - v * p.G);
                    }
                    break;
                }
                s.seen += n;
                s.b0 += 32;
            }
            s.ended = s.x < 0;
            const int slot = i % kRing;
            if (i >= kRing) {
                const bool ok = *vabort == 0 && mbar_wait(&taken[slot], ((i / kRing) & 1) ^ 1, timeout_ns);
                if (!__all_sync(0xffffffffu, ok)) {
                    if (lane == 0) set_status(status, STATUS_TIMEOUT);
                    *vabort = 1;
                    s.ended = true;
                    return;
                }
            }
            if (found || (s.ended && lane == 0)) {
                ring[slot] = e;
                mbar_arrive(&filled[slot]);
            }
            __syncwarp();
        }
    }
};

template <int D>
constexpr size_t packed_smem(int B) {
    return Layout<D, 1>::SMEM + kRing * sizeof(int4) + (size_t)B * 4;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_packed_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                          const __grid_constant__ CUtensorMap tmv, const PackedParams p) {
    using Lay = Layout<D, 1>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const Barriers<D, 1> bar(sm);
    int4 *ring = reinterpret_cast<int4 *>(sm + Lay::OFF_POLICY);
    int *counts = reinterpret_cast<int *>(ring + kRing);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        bar.init();
        for (int s = 0; s < kRing; ++s) {
            mbar_init(&bar.policy[s], 1);
            mbar_init(&bar.policy[kRing + s], PackedPolicy<D>::kConsumers);
        }
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
    auto count = [&](int b, bool falls) {
        return (PackedPolicy<D>::span(p, b, falls).y + 2 * p.pt - 1) / (2 * p.pt);
    };
    bool falls = false;
    for (int b = threadIdx.x; b < p.B; b += kThreads) {
        const int a = p.cu[b], z = p.cu[b + 1];
        counts[b] = count(b, false);
        falls = falls || z < a;
        if (blockIdx.x == 0 && (a < 0 || z < a || z > p.N)) set_status(p.status, STATUS_SEQLEN);
    }
    falls = __syncthreads_or(falls);
    if (falls) {
        for (int b = threadIdx.x; b < p.B; b += kThreads) counts[b] = count(b, true);
        __syncthreads();
    }
    tc::fence_after();
    const uint32_t tmem = *bar.tmem_slot;
    PackedPolicy<D> pol{p, &tmq, &tmk, &tmv, ring, bar.policy, bar.policy + kRing, counts, falls, bar.abort_flag,
                        p.status, p.scale_log2, static_cast<__nv_bfloat16 *>(p.out), p.timeout_ns,
                        l2_policy_evict_first(), l2_policy_evict_last()};
    attend<D, 1>(pol, sm, tmem);
    tc::fence_before();
    __syncthreads();
    if (warp == 9) {
        tc::fence_after();
        tc::tmem_dealloc(tmem, kTmemCols);
    }
}

template <int D>
struct PackedTag {};

template <int D>
cudaError_t run_packed(const PackedParams &p, int grid, const CUtensorMap *tmq, const CUtensorMap *tmk,
                       const CUtensorMap *tmv, cudaStream_t st) {
    auto kern = prefill_packed_kernel<D>;
    cudaError_t e = once_per_device<PackedTag<D>>([&] {
        cudaFuncAttributes fa;
        cudaError_t r = cudaFuncGetAttributes(&fa, kern);
        if (r != cudaSuccess) return r;
        if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidKernelImage;  // register split would not hold
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    });
    if (e != cudaSuccess) return e;
    return dec::launch_pdl(kern, dim3(grid), dim3(kThreads), packed_smem<D>(p.B), st, *tmq, *tmk, *tmv, p);
}

static_assert(packed_smem<128>(8192) <= 227 * 1024, "the counts of 8192 sequences fit");

}  // namespace

cudaError_t launch_prefill_packed(const PackedArgs &a, const CUtensorMap *tmq, const CUtensorMap *tmk,
                                  const CUtensorMap *tmv, cudaStream_t st) {
    PackedParams p = {};
    p.cu = a.cu;
    p.out = a.out;
    p.status = a.status;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.B = a.B;
    p.N = a.N;
    p.H = a.H;
    p.G = a.G;
    p.r = a.H / a.G;
    p.pt = kRows / p.r;
    p.window = a.window;
    p.timeout_ns = a.timeout_ns;
    // one CTA per SM, or fewer when there cannot be that many pieces
    const long long pieces = ((long long)a.N / (2 * p.pt) + a.B) * a.G;
    const int grid = (int)(pieces < a.num_sms ? pieces : a.num_sms);
    if (a.d_h == 64) return run_packed<64>(p, grid, tmq, tmk, tmv, st);
    if (a.d_h == 128) return run_packed<128>(p, grid, tmq, tmk, tmv, st);
    return cudaErrorInvalidValue;
}

}  // namespace gqa
