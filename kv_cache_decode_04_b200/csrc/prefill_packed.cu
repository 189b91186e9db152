// prefill_packed.cu -- causal GQA attention over prompts of different lengths
// packed into one token axis, on the 5th-generation tensor cores (sm_100a).
//
// What is computed: with sequence b = positions [cu[b], cu[b+1]) of the packed
// axis, for each of its positions s and query head i, g = i / (H/G),
//     out[s,i] = sum_{cu[b] <= t <= s} softmax_t(scale * q[s,i] . k[t,g]) v[t,g]
// (with a window W > 0: s - W < t <= s).
//
// One CTA = 2 tiles of 128 rows, a row being a (position, head of the group)
// pair (attend.cuh): 2 * floor(128 / r) consecutive positions of one sequence,
// all r heads of one group.  Each K/V tile that it loads serves both.  Roles
// and tensor-memory layout are those of prefill.cu: warp 8 TMA, warp 9 MMA,
// warps 0-3 and 4-7 the softmax of one tile each (a thread per row), warp 10
// clears V rows past a sequence's end.
//
// Work list.  The lengths are on the device, so the grid is an upper bound
// (sum_b ceil(len_b / P2) <= N / P2 + B tiles) and each CTA finds its tile
// from cu: tiles are ordered by their index within the sequence, the largest
// first, so that the ones with the most keys start first whatever sequence
// they belong to.  With C(x) = sum_b max(0, tiles_b - x) tiles of index >= x,
// tile u has the index x with C(x+1) <= u < C(x): a binary search whose every
// step is one warp-wide sum.
#include <climits>

#include "attend.cuh"
#include "decode_common.cuh"

namespace gqa {

namespace {

using namespace att;

template <int D>
struct PackLay {
    static constexpr int HALVES = D / 64;
    static constexpr int TILE = HALVES * kHalf;  // [128 x D] bf16
    static constexpr int OFF_Q = 0;              // 2 tiles
    static constexpr int OFF_K = 2 * TILE;       // 2 stages
    static constexpr int OFF_V = 4 * TILE;       // 2 stages
    static constexpr int OFF_BAR = 6 * TILE;
    static constexpr size_t SMEM = 1024 + OFF_BAR + 256;
};

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

// Start and length of sequence b, forced into [0, N].
__device__ __forceinline__ int2 seq_span(const PackedParams &p, int b) {
    const int a = min(max(p.cu[b], 0), p.N);
    return make_int2(a, min(max(p.cu[b + 1], a), p.N) - a);
}

// The tile of rank u (see the head of the file): its sequence and index.  One
// warp; false when there are not so many.
__device__ bool find_tile(const PackedParams &p, int u, int lane, int &seq, int &index) {
    const int p2 = 2 * p.pt;
    auto tiles = [&](int b) { return (seq_span(p, b).y + p2 - 1) / p2; };
    // a warp's batches are few in most calls, and the lengths stay in L1
    auto at_least = [&](int x) {  // tiles of index >= x
        int n = 0;
        for (int b = lane; b < p.B; b += 32) n += max(0, tiles(b) - x);
        return __reduce_add_sync(0xffffffffu, n);
    };
    int top = 0;
    for (int b = lane; b < p.B; b += 32) top = max(top, tiles(b));
    top = __reduce_max_sync(0xffffffffu, top);
    if (u >= at_least(0)) return false;
    int lo = 0, hi = top - 1;  // the largest x with C(x) > u
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (at_least(mid) > u) lo = mid; else hi = mid - 1;
    }
    // the k-th sequence that has a tile of this index
    int k = u - at_least(lo + 1);
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int b = b0 + lane;
        const unsigned has = __ballot_sync(0xffffffffu, b < p.B && tiles(b) > lo);
        const int n = __popc(has);
        if (k < n) {
            unsigned bits = has;
            for (int i = 0; i < k; ++i) bits &= bits - 1;
            seq = b0 + __ffs(bits) - 1;
            index = lo;
            return true;
        }
        k -= n;
    }
    return false;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_packed_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                          const __grid_constant__ CUtensorMap tmv, const PackedParams p) {
    using Lay = PackLay<D>;
    constexpr int HALVES = Lay::HALVES, kTile = Lay::TILE;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + Lay::OFF_BAR);
    uint64_t *bar_q = bars + 0;
    uint64_t *k_full = bars + 1;    // [2]
    uint64_t *k_empty = bars + 3;   // [2]
    uint64_t *v_full = bars + 5;    // [2]
    uint64_t *v_empty = bars + 7;   // [2]
    uint64_t *s_full = bars + 9;    // [2] one per row tile
    uint64_t *p_ready = bars + 11;  // [2]
    uint64_t *o_done = bars + 13;
    uint64_t *drain = bars + 14;
    uint64_t *tail_go = bars + 15;  // the last V tile is on its way ...
    uint64_t *v_clean = bars + 16;  // ... and its rows past the sequence's end are zero
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 17);
    int *abort_flag = reinterpret_cast<int *>(tmem_slot + 1);
    int *unit = abort_flag + 1;  // [2] sequence (or -1), tile index
    volatile int *vabort = abort_flag;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(bar_q, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&k_full[s], 1);
            mbar_init(&k_empty[s], 1);
            mbar_init(&v_full[s], 1);
            mbar_init(&v_empty[s], 1);
            mbar_init(&s_full[s], 1);
            mbar_init(&p_ready[s], 128);
        }
        mbar_init(o_done, 1);
        mbar_init(drain, 1);
        mbar_init(tail_go, 1);
        mbar_init(v_clean, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    pdl_wait_primary();
    if (warp == 8) {
        int seq = -1, index = 0;
        if (!find_tile(p, blockIdx.x / p.G, lane, seq, index)) seq = -1;
        if (lane == 0) {
            unit[0] = seq;
            unit[1] = index;
        }
        if (blockIdx.x == 0) {  // once per call: lengths out of range
            bool bad = false;
            for (int b = lane; b <= p.B; b += 32) {
                const int c = p.cu[b];
                bad |= c < 0 || c > p.N || (b > 0 && c < p.cu[b - 1]);
            }
            if (__any_sync(0xffffffffu, bad) && lane == 0) set_status(p.status, STATUS_SEQLEN);
        }
    }
    if (warp == 9) tc::tmem_alloc(tmem_slot, kTmemCols);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *tmem_slot;
    const int b = unit[0];
    const int g = blockIdx.x % p.G;
    const int h0 = g * p.r;
    const int2 span = seq_span(p, max(b, 0));
    const int start = span.x, len = b < 0 ? 0 : span.y;
    const int s0 = unit[1] * 2 * p.pt;  // first position of the CTA within its sequence
    // the debug build's check of the unit (uniform over the CTA)
    const bool go = b >= 0 && index_ok(s0 < len && start + len <= p.N && h0 + p.r <= p.H, p.status);
    // Key tiles: j_lo..j_hi[hh] for row tile hh, whose positions start at s0 + hh pt.
    // The second may need one tile more than the first, or have no position at all.
    const int nh = go ? (s0 + p.pt < len ? 2 : 1) : 0;
    const int j_lo = p.window > 0 ? max(0, s0 - p.window + 1) / kKeys : 0;
    const int j_hi0 = (min(len, s0 + p.pt) - 1) / kKeys;
    const int j_hi = nh == 2 ? (min(len, s0 + 2 * p.pt) - 1) / kKeys : j_hi0;
    const int n_kv = go ? j_hi - j_lo + 1 : 0;
    const int n_kv0 = go ? j_hi0 - j_lo + 1 : 0;  // tiles the first row tile visits (n_kv or fewer)
    const bool tail = (j_hi + 1) * kKeys > len;   // the last key tile runs past the sequence
    const bool split_p = j_hi == 0 || (p.window > 0 && p.window <= 256);

    if (!go) {
        // no tile for this CTA
    } else if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLowRegs));
        if (warp == 8) {
            // ------------------------------------------------ TMA producer
            if (lane == 0) {
                const uint64_t pol_q = l2_policy_evict_first(), pol_kv = l2_policy_evict_last();
                mbar_arrive_expect_tx(bar_q, nh * HALVES * p.pt * p.r * 128);
                for (int hh = 0; hh < nh; ++hh)
                    for (int half = 0; half < HALVES; ++half)
                        tma_load_3d(sm + Lay::OFF_Q + hh * kTile + half * kHalf, &tmq, bar_q, half * 64, h0,
                                    start + s0 + hh * p.pt, pol_q);
                int nk = 0, nv = 0;  // tiles asked for
                for (int jj = 0; jj < n_kv; ++jj) {
                    const int st = jj & 1, row = start + (j_lo + jj) * kKeys;
                    const uint32_t ph = (jj >> 1) & 1;
                    if (*vabort || !mbar_wait(&k_empty[st], ph ^ 1, p.timeout_ns)) {
                        set_status(p.status, STATUS_TIMEOUT);
                        *vabort = 1;
                        break;
                    }
                    mbar_arrive_expect_tx(&k_full[st], kTile);
                    for (int half = 0; half < HALVES; ++half)
                        tma_load_3d(sm + Lay::OFF_K + st * kTile + half * kHalf, &tmk, &k_full[st], half * 64, g, row,
                                    pol_kv);
                    nk = jj + 1;
                    if (*vabort || !mbar_wait(&v_empty[st], ph ^ 1, p.timeout_ns)) {
                        set_status(p.status, STATUS_TIMEOUT);
                        *vabort = 1;
                        break;
                    }
                    mbar_arrive_expect_tx(&v_full[st], kTile);
                    for (int half = 0; half < HALVES; ++half)
                        tma_load_3d(sm + Lay::OFF_V + st * kTile + half * kHalf, &tmv, &v_full[st], half * 64, g, row,
                                    pol_kv);
                    nv = jj + 1;
                    if (tail && nv == n_kv) mbar_arrive(tail_go);
                }
                // whatever the other warps did, no copy is in flight when the CTA leaves
                mbar_wait(bar_q, 0, p.timeout_ns);
                for (int jj = max(0, nk - 2); jj < nk; ++jj) mbar_wait(&k_full[jj & 1], (jj >> 1) & 1, p.timeout_ns);
                for (int jj = max(0, nv - 2); jj < nv; ++jj) mbar_wait(&v_full[jj & 1], (jj >> 1) & 1, p.timeout_ns);
            }
            __syncwarp();
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
                // S_hh = Q_hh K^T: D/16 K-steps over d_h
                auto issue_s = [&](int hh, int ks) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
                        tc::mma_ss(tmem + hh * 128, dq + ((hh * kTile) >> 4) + off, dk + ((ks * kTile) >> 4) + off,
                                   idesc_s, kk > 0 ? 1u : 0u);
                    }
                };
                // O_hh += P_hh V: 8 K-steps of 16 keys (a second pass adds P_lo)
                auto issue_pv = [&](int hh, int vs, bool acc) {
                    const int passes = split_p ? 2 : 1;
#pragma unroll 1
                    for (int ps = 0; ps < passes; ++ps)
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            tc::mma_ts(tmem + 256 + hh * 128, tmem + hh * 128 + ps * 64 + kk * 8,
                                       dv + ((vs * kTile + kk * 2048) >> 4), idesc_o,
                                       (acc || ps > 0 || kk > 0) ? 1u : 0u);
                };
                const bool two = nh == 2;
                if (wait(bar_q, 0) && wait(&k_full[0], 0)) {
                    issue_s(0, 0);
                    tc::commit(&s_full[0]);
                    if (two) {
                        issue_s(1, 0);
                        tc::commit(&s_full[1]);
                    }
                    tc::commit(&k_empty[0]);
                    issued = true;
                    for (int j = 0; j < n_kv && ok; ++j) {  // j counts visited tiles
                        const int st = j & 1, st2 = (j + 1) & 1;
                        const uint32_t ph = (j >> 1) & 1, ph2 = ((j + 1) >> 1) & 1;
                        const bool on0 = j < n_kv0, next0 = j + 1 < n_kv0, next = j + 1 < n_kv;
                        if (!wait(&v_full[st], ph)) break;
                        if (tail && j == n_kv - 1 && !wait(v_clean, 0)) break;
                        if (on0) {
                            if (!wait(&p_ready[0], j & 1, true)) break;
                            tc::fence_after();
                            issue_pv(0, st, j > 0);
                        }
                        if (next) {
                            if (!wait(&k_full[st2], ph2)) break;
                            if (next0) {
                                issue_s(0, st2);
                                tc::commit(&s_full[0]);
                            }
                        }
                        if (two) {
                            if (!wait(&p_ready[1], j & 1, true)) break;
                            tc::fence_after();
                            issue_pv(1, st, j > 0);
                        }
                        tc::commit(&v_empty[st]);
                        if (next) {
                            if (two) {
                                issue_s(1, st2);
                                tc::commit(&s_full[1]);
                            }
                            tc::commit(&k_empty[st2]);
                        }
                    }
                    tc::commit(o_done);
                }
                if (issued && !ok) {  // let MMAs already issued finish before TMEM is freed
                    tc::commit(drain);
                    mbar_wait(drain, 0, p.timeout_ns);
                }
            }
            __syncwarp();
        } else if (warp == 10 && tail) {
            // ------------------------------------------------ V rows past the end
            // (tail_go first: before the load is issued the stage's barrier may stand
            // two phases back, which a wait on the parity alone cannot tell apart)
            const int last = n_kv - 1;
            if (warp_wait(tail_go, 0, p.timeout_ns) &&
                warp_wait(&v_full[last & 1], (last >> 1) & 1, p.timeout_ns)) {
                zero_tail_rows<D>(sm + Lay::OFF_V + (last & 1) * kTile, len - j_hi * kKeys, lane);
                if (lane == 0) mbar_arrive(v_clean);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kHighRegs));
        // ------------------------------------------------ softmax + epilogue
        const int hh = warp >> 2;          // row tile
        const int t = threadIdx.x & 127;   // row = tensor-memory lane
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_off + hh * 128;
        const uint32_t tO = tmem + lane_off + 256 + hh * 128;
        const int tok = t / p.r, head = t - tok * p.r;
        const int first_pos = s0 + hh * p.pt;
        const int pos = first_pos + tok;
        const int key_lo = p.window > 0 ? pos - p.window + 1 : INT_MIN;
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        const int my_kv = hh >= nh ? 0 : (hh == 0 ? n_kv0 : n_kv);
        for (int jj = 0; jj < my_kv; ++jj) {
            const int key0 = (j_lo + jj) * kKeys;
            const bool aborted = __any_sync(0xffffffffu, *vabort != 0);
            if (aborted || !warp_wait(&s_full[hh], jj & 1, p.timeout_ns)) {
                if (lane == 0) set_status(p.status, STATUS_TIMEOUT);
                *vabort = 1;
                ok = false;
                break;
            }
            tc::fence_after();
            // a tile with keys after some row's position, or before its window
            const bool masked = key0 + kKeys - 1 > first_pos || (p.window > 0 && key0 < first_pos + p.pt - p.window);
            softmax_step<D>(tS, tO, p.scale_log2, jj == 0, split_p, m, l, [&](uint32_t(&sr)[4][32]) {
                if (masked) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const int key = key0 + c * 32 + e;
                            if (key > pos || key < key_lo) sr[c][e] = __float_as_uint(-INFINITY);
                        }
                }
            });
            tc::fence_before();
            mbar_arrive(&p_ready[hh]);
        }
        // epilogue: O / l -> bf16 -> out[start + pos, h0 + head, :]
        const bool run = __all_sync(0xffffffffu, ok && *vabort == 0);
        if (hh >= nh) {
            // no rows: nothing to store
        } else if (run && warp_wait(o_done, 0, p.timeout_ns)) {
            tc::fence_after();
            const float inv = l > 0.f ? 1.f / l : 0.f;
            const bool store = tok < p.pt && pos < len;
            __nv_bfloat16 *dst =
                static_cast<__nv_bfloat16 *>(p.out) + ((size_t)(start + pos) * p.H + h0 + head) * D;
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
                uint32_t orow[16];
                tc::ld16(tO + c * 16, orow);
                tc::wait_ld();
                uint32_t pk[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    pk[e] = pack_bf16x2(__uint_as_float(orow[2 * e]) * inv, __uint_as_float(orow[2 * e + 1]) * inv);
                if (store) {
                    uint4 *d4 = reinterpret_cast<uint4 *>(dst + c * 16);
                    d4[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    d4[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
                }
            }
        } else if (lane == 0) {
            set_status(p.status, STATUS_TIMEOUT);
        }
    }
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
cudaError_t run_packed(const PackedParams &p, unsigned grid, const CUtensorMap *tmq, const CUtensorMap *tmk,
                       const CUtensorMap *tmv, cudaStream_t st) {
    constexpr size_t smem = PackLay<D>::SMEM;
    cudaError_t e = once_per_device<PackedTag<D>>([] {
        cudaFuncAttributes fa;
        cudaError_t r = cudaFuncGetAttributes(&fa, prefill_packed_kernel<D>);
        if (r != cudaSuccess) return r;
        if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidKernelImage;  // register split would not hold
        return cudaFuncSetAttribute(prefill_packed_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    });
    if (e != cudaSuccess) return e;
    return dec::launch_pdl(prefill_packed_kernel<D>, dim3(grid), dim3(kThreads), smem, st, *tmq, *tmk, *tmv, p);
}

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
    const long long grid = ((long long)a.N / (2 * p.pt) + a.B) * a.G;
    if (grid <= 0 || grid >= (1ll << 31)) return cudaErrorInvalidConfiguration;
    if (a.d_h == 64) return run_packed<64>(p, (unsigned)grid, tmq, tmk, tmv, st);
    if (a.d_h == 128) return run_packed<128>(p, (unsigned)grid, tmq, tmk, tmv, st);
    return cudaErrorInvalidValue;
}

}  // namespace gqa
