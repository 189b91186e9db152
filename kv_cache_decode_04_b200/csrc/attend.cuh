// attend.cuh -- what the packed prefill and the draft-tree decode share: rows
// of (token, query head) packed into M = 128 tensor-core tiles, and the online
// softmax of one [128 x 128] score tile held in tensor memory.
//
// Row packing.  The r = H/G query heads of a group read the same K/V head, so
// the rows of one tile are the (token, head) pairs of PT = floor(128 / r)
// consecutive tokens: row = token * r + head.  One TMA box of [64 dims x r
// heads x PT tokens] lays them out in that order.  A few tokens then fill a
// tile as well as many do, whatever r is.
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
constexpr uint32_t kTmemCols = 512;  // S0/P0, S1/P1 (128 columns each), O0, O1 (128 each)

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

// One online-softmax step for this thread's query row (its tensor-memory lane):
// reads the 128 scores at tS, lets `mask(sr)` set hidden ones to -inf, moves
// the running maximum m (log2 units) and the sum l, and writes P = 2^(s - m)
// as bf16 pairs over the first 64 columns at tS.
//   - The maximum moves (and O at tO is rescaled) only when it grows by more
//     than 8, so p <= 2^8: numerator and denominator use the same stale one.
//   - `first`: O holds nothing of this row yet.  Otherwise the P.V that last
//     wrote O is complete, because the S just read was issued behind it.
//   - split_p: P is carried as P_hi + P_lo, two bf16 terms (about 16
//     significant bits), P_lo in columns 64..127.  For rows that see so few
//     keys that the rounding of P does not average out.
//   - m = -inf (no key seen yet): every score is -inf and p = 0.
// The row sum adds the unrounded p in fp32.
template <int D, typename Mask>
__device__ __forceinline__ void softmax_step(uint32_t tS, uint32_t tO, float scale_log2, bool first, bool split_p,
                                             float &m, float &l, Mask mask) {
    uint32_t sr[4][32];
#pragma unroll
    for (int c = 0; c < 4; ++c) tc::ld32(tS + c * 32, sr[c]);
    tc::wait_ld();
#pragma unroll
    for (int c = 0; c < 4; ++c) tc::hold32(sr[c]);
    mask(sr);
    // row maximum of the raw scores (the scale is positive), eight partial maxima
    float mx8[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) mx8[i] = -INFINITY;
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int e = 0; e < 32; ++e) mx8[e & 7] = fmaxf(mx8[e & 7], __uint_as_float(sr[c][e]));
    const float mx = fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                           fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7]))) * scale_log2;
    float alpha = 1.f;
    bool rescale = false;
    if (first) {
        m = mx;
    } else {
        const float mn = fmaxf(m, mx);
        const bool need = mn > m + 8.f;
        rescale = __any_sync(0xffffffffu, need);
        if (need) {
            alpha = fast_exp2(m - mn);
            m = mn;
            l *= alpha;
        }
    }
    const float mu = m == -INFINITY ? 0.f : m;
    const uint64_t sc2 = f32x2_pack(scale_log2, scale_log2), nm2 = f32x2_pack(-mu, -mu);
    uint64_t rs2[4] = {0ull, 0ull, 0ull, 0ull};
    if (!split_p) {
#pragma unroll
        for (int c4 = 0; c4 < 4; ++c4) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const uint64_t x2 = f32x2_fma(
                    f32x2_pack(__uint_as_float(sr[c4][2 * e]), __uint_as_float(sr[c4][2 * e + 1])), sc2, nm2);
                float x0, x1;
                f32x2_unpack(x2, x0, x1);
                const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
                rs2[e & 3] = f32x2_add(rs2[e & 3], f32x2_pack(p0, p1));
                pk[e] = pack_bf16x2(p0, p1);
            }
            tc::st16(tS + c4 * 16, pk);
        }
    } else {
#pragma unroll
        for (int c4 = 0; c4 < 4; ++c4) {
#pragma unroll
            for (int e4 = 0; e4 < 4; ++e4) {
                uint32_t ph[4], pl[4];
#pragma unroll
                for (int e1 = 0; e1 < 4; ++e1) {
                    const int e = e4 * 4 + e1;
                    const float p0 = fast_exp2(fmaf(__uint_as_float(sr[c4][2 * e]), scale_log2, -mu));
                    const float p1 = fast_exp2(fmaf(__uint_as_float(sr[c4][2 * e + 1]), scale_log2, -mu));
                    rs2[e1] = f32x2_add(rs2[e1], f32x2_pack(p0, p1));
                    ph[e1] = pack_bf16x2(p0, p1);
                    const float2 h = unpack_bf16x2(ph[e1]);
                    pl[e1] = pack_bf16x2(p0 - h.x, p1 - h.y);
                }
                tc::st4(tS + c4 * 16 + e4 * 4, ph);
                tc::st4(tS + 64 + c4 * 16 + e4 * 4, pl);
            }
        }
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
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a0, a1;
        f32x2_unpack(rs2[i], a0, a1);
        sum += a0 + a1;
    }
    l = first ? sum : l + sum;
    tc::wait_st();
}

// Zeroes rows [r0, 128) of a [128 x D] V tile (D / 64 swizzled boxes): P is 0
// there, but 0 times what lies past a sequence's end must stay 0.  One warp;
// the fence makes the writes visible to the tensor core's reads.
template <int D>
__device__ __forceinline__ void zero_tail_rows(uint8_t *tile, int r0, int lane) {
    const int n = (kKeys - r0) * (D / 64) * 8;  // 16-byte pieces
    for (int i = lane; i < n; i += 32) {
        const int row = r0 + i / ((D / 64) * 8), rem = i % ((D / 64) * 8);
        asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(
                         smem_u32(tile + (rem >> 3) * kHalf + row * 128 + (rem & 7) * 16)),
                     "r"(0u)
                     : "memory");
    }
    fence_proxy_async_smem();
    __syncwarp();
}

}  // namespace att
}  // namespace gqa
