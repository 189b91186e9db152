// cache.cu -- rows and pages of the K/V cache: append, compact, and the page
// pool's reserve (with copy-on-write), fork and release (sm_100a).
//
// A cache is either dense, [B, G, T_cap, d_h], or paged: pools of pages
// [P, G, page, d_h] and a block table [B, M] whose entry k names the page that
// holds positions [k page, (k+1) page) of the sequence (-1: none).  A dense
// cache is the paged one with page = T_cap and the identity table, and the
// kernels treat it so.  Nothing here computes on the values: rows are moved as
// 16-byte pieces, so fp32 and bf16 caches take the same code.
//
// A bad length, count or table entry never reaches an address: it sets a bit
// of the status word and the row, sequence or pair it belongs to is skipped.
#include <climits>

#include "common.cuh"
#include "decode_common.cuh"
#include "internal.h"

namespace gqa {

namespace {

// Page and row of position `pos` of sequence b; false when no page holds it.
__device__ __forceinline__ bool locate(const CacheView &c, int b, int pos, int &page, int &row) {
    if (!c.table) {
        page = b;
        row = pos;
        return true;
    }
    const int k = pos / c.page;
    row = pos - k * c.page;
    page = c.table[(size_t)b * c.M + k];
    return page >= 0 && page < c.num_pages;
}

// 16-byte piece `i` of the row (page, g, row) in pieces of the cache.
__device__ __forceinline__ size_t piece_of(const CacheView &c, int page, int g, int row) {
    return (((size_t)page * c.G + g) * c.page + row) * c.row16;
}

// ------------------------------------------------------------------ append

constexpr int kAppendWarps = 8;
constexpr int kAppendHeld = 4;  // pieces of K and of V that a lane has in flight

// Whether some entry of cu[0 .. B] is below the one before it: each thread of
// the block looks at its part.  Four entries a load, the next thread's first by
// shuffle, since at 8192 sequences what the blocks of an SM read here adds up.
__device__ __forceinline__ bool any_falls(const int32_t *cu, int B) {
    const bool wide = (reinterpret_cast<uintptr_t>(cu) & 15) == 0;
    bool falls = false;
    for (int base = 0; base <= B; base += blockDim.x * 4) {
        const int i = base + threadIdx.x * 4;
        int4 x = make_int4(INT_MAX, INT_MAX, INT_MAX, INT_MAX);  // entries behind the last
        if (wide && i + 3 <= B) {
            x = *reinterpret_cast<const int4 *>(cu + i);
        } else {
            if (i <= B) x.x = cu[i];
            if (i + 1 <= B) x.y = cu[i + 1];
            if (i + 2 <= B) x.z = cu[i + 2];
            if (i + 3 <= B) x.w = cu[i + 3];
        }
        int next = __shfl_down_sync(0xffffffffu, x.x, 1);
        if ((threadIdx.x & 31) == 31) next = i + 4 <= B ? cu[i + 4] : INT_MAX;
        falls = falls || x.y < x.x || x.z < x.y || x.w < x.z || next < x.w;
    }
    return falls;
}

// One warp per new token: it finds the token's sequence in cu_seqlens (a
// binary search over B + 1 entries), then moves the token's G rows of K and of
// V, all loads of a round before its stores.  HBM-bound for prompts: each byte
// is read once and written once.
//
// A sequence is served, all its rows and its length, or left alone: it is left
// alone when its range is bad, when it has no room, or when it begins below an
// earlier offset, so the served ranges never share a row.  Offsets that fall
// are rare and found by every block at its start (the entries are the ones the
// search then reads); only then is an earlier offset looked for, and the search
// linear: a range that is served holds tok exactly when the first offset above
// tok is its end.  24 prompts of 200 to 8,000 tokens (G 8, d_h 128): 73.3 us,
// 6.2 TB/s; 32 sequences' drafts 2.9 in a graph; one row each of 8,192 sequences
// 13.5, of which the look at the offsets is 1.6.
__global__ void __launch_bounds__(kAppendWarps * 32)
    cache_append_kernel(const uint4 *__restrict__ k_new, const uint4 *__restrict__ v_new, const int32_t *cu,
                        const int32_t *seqlens, int32_t *seqlens_out, uint4 *__restrict__ k_cache,
                        uint4 *__restrict__ v_cache, const CacheView c, int N, unsigned *status) {
    pdl_wait_primary();
    const int lane = threadIdx.x & 31;
    const int gid = blockIdx.x * blockDim.x + threadIdx.x;
    const bool falls = __syncthreads_or(any_falls(cu, c.B));
    auto served = [&](int b, int lo, int hi, int T) {
        if (lo < 0 || hi < lo || hi > N || T < 0 || hi - lo > c.cap || T > c.cap - (hi - lo)) return false;
        if (falls)
            for (int i = 0; i < b; ++i)
                if (cu[i] > lo) return false;
        return true;
    };
    // lengths after the append (once, here)
    for (int b = gid; b < c.B; b += gridDim.x * blockDim.x) {
        const int lo = cu[b], hi = cu[b + 1], T = seqlens[b];
        const bool ok = served(b, lo, hi, T);
        if (!ok) set_status(status, STATUS_SEQLEN);
        seqlens_out[b] = ok ? T + (hi - lo) : T;
    }
    const int end = falls ? N : min(N, max(0, cu[c.B]));
    const int pieces = c.G * c.row16;
    const int shift = __ffs(c.row16) - 1;  // pieces of a row: 8, 16 or 32
    for (int tok = gid >> 5; tok < end; tok += (gridDim.x * blockDim.x) >> 5) {
        int lo = 0, hi = c.B - 1;  // the last b with cu[b] <= tok
        if (falls) {
            while (lo < c.B && cu[lo + 1] <= tok) ++lo;  // cu[0] > tok: its range does not hold tok
            if (lo == c.B) continue;
            hi = lo;
        }
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (cu[mid] <= tok) lo = mid; else hi = mid - 1;
        }
        const int first = cu[lo], last = cu[lo + 1], T = seqlens[lo];
        if (tok < first || tok >= last || !served(lo, first, last, T)) continue;
        int page, row;
        if (!locate(c, lo, T + tok - first, page, row)) {
            if (lane == 0) set_status(status, STATUS_PAGES);
            continue;
        }
        const size_t src = (size_t)tok * pieces;
        for (int i0 = lane; i0 < pieces; i0 += 32 * kAppendHeld) {
            uint4 k[kAppendHeld], v[kAppendHeld];
#pragma unroll
            for (int j = 0; j < kAppendHeld; ++j) {
                const int i = i0 + j * 32;
                if (i < pieces) {
                    k[j] = __ldcs(k_new + src + i);
                    v[j] = __ldcs(v_new + src + i);
                }
            }
#pragma unroll
            for (int j = 0; j < kAppendHeld; ++j) {
                const int i = i0 + j * 32;
                if (i < pieces) {
                    const size_t dst = piece_of(c, page, i >> shift, row) + (i & (c.row16 - 1));
                    k_cache[dst] = k[j];
                    v_cache[dst] = v[j];
                }
            }
        }
    }
}

// ------------------------------------------------------------------ compact

constexpr int kCompactThreads = 256;
constexpr int kKeepMax = 64;

// One block per (sequence, KV head, K or V).  All kept rows are read into
// registers before any is written, so any order of `keep`, repeated entries
// included, gives the rows as they were before the call.  Latency-bound: three
// dependent loads (lengths and entries, pages, rows), so blocks should be many:
// with ROW16 = 8 or 16 pieces a row 30 registers let eight share an SM, with 32
// (fp32, d_h = 128) a thread holds eight pieces, 48 registers, and five do.
// 32 sequences of 16 rows: 2.1 us in a graph, 256 of 64: 6.6 (bf16, G 8, d_h 128).
template <int ROW16>
__global__ void __launch_bounds__(kCompactThreads)
    cache_compact_kernel(uint4 *k_cache, uint4 *v_cache, const int32_t *seqlens, const int32_t *keep,
                         const int32_t *n_keep, int32_t *seqlens_out, const CacheView c, int m, unsigned *status) {
    constexpr int kHeld = kKeepMax * ROW16 / kCompactThreads;  // pieces a thread holds
    __shared__ size_t src[kKeepMax], dst[kKeepMax];
    __shared__ int moves[kKeepMax];
    pdl_wait_primary();
    const int b = blockIdx.x / (2 * c.G), rem = blockIdx.x % (2 * c.G);
    const int g = rem >> 1;
    uint4 *cache = (rem & 1) ? v_cache : k_cache;
    const int j = threadIdx.x;
    const int from = j < m ? keep[(size_t)b * m + j] : 0;
    const int T = seqlens[b];
    const int n = n_keep ? n_keep[b] : m;
    bool ok = T >= 0 && T <= c.cap && n >= 0 && n <= m;
    bool paged = true;
    if (ok && j < n) {
        ok = from >= 0 && from < kKeepMax && T <= c.cap - 1 - max(from, j);
        if (ok) {
            int p0, r0, p1, r1;
            paged = locate(c, b, T + from, p0, r0);
            paged = locate(c, b, T + j, p1, r1) && paged;
            if (paged) {
                src[j] = piece_of(c, p0, g, r0);
                dst[j] = piece_of(c, p1, g, r1);
            }
            moves[j] = from != j;
        }
    }
    const bool all_ok = __syncthreads_and(ok), all_paged = __syncthreads_and(paged);
    const bool go = all_ok && all_paged;
    if (rem == 0 && threadIdx.x == 0) {
        seqlens_out[b] = go ? T + n : T;
        if (!all_ok) set_status(status, STATUS_SEQLEN);
        if (!all_paged) set_status(status, STATUS_PAGES);
    }
    if (!go) return;
    uint4 held[kHeld];
    const int pieces = n * ROW16;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        const int p = i * kCompactThreads + threadIdx.x;
        if (p < pieces && moves[p / ROW16]) held[i] = cache[src[p / ROW16] + p % ROW16];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        const int p = i * kCompactThreads + threadIdx.x;
        if (p < pieces && moves[p / ROW16]) cache[dst[p / ROW16] + p % ROW16] = held[i];
    }
}

// ------------------------------------------------------------------ release

constexpr int kPageThreads = 128;

// One block per sequence: entries past the pages that lengths[b] positions
// need give up their reference and become -1.
__global__ void __launch_bounds__(kPageThreads)
    pages_release_kernel(int32_t *table, int32_t *refcount, const int32_t *lengths, int M, int page, int P,
                         unsigned *status) {
    pdl_wait_primary();
    const int b = blockIdx.x;
    const int len = lengths[b];
    if (len < 0) {
        if (threadIdx.x == 0) set_status(status, STATUS_SEQLEN);
        return;
    }
    const long long first = ((long long)len + page - 1) / page;
    int32_t *row = table + (size_t)b * M;
    for (long long k = first + threadIdx.x; k < M; k += blockDim.x) {
        const int e = row[k];
        if (e < 0) continue;
        row[k] = -1;
        // a page out of range, or one that nobody held: the counts stay as they were
        if (e >= P) {
            set_status(status, STATUS_PAGES);
        } else if (atomicSub(&refcount[e], 1) <= 0) {
            atomicAdd(&refcount[e], 1);
            set_status(status, STATUS_PAGES);
        }
    }
}

// ------------------------------------------------------------------ fork

// One block per pair: row dst[i] comes to list the pages that hold the
// seqlens[src[i]] positions of row src[i], each with one more reference.
// Which pairs run depends on the inputs alone, so the order of the blocks does
// not matter: a pair is skipped and flagged when an index is out of range, its
// dst is also some pair's src or its src some pair's dst, an earlier pair has the
// same dst, dst's row is not empty, src's length is out of range, or src's table
// lacks a page or lists one that nobody holds (with one reference for two rows, a
// reserve would take the page for either row's own).
__global__ void __launch_bounds__(kPageThreads)
    pages_fork_kernel(int32_t *table, int32_t *refcount, int32_t *seqlens, const int32_t *src, const int32_t *dst,
                      int n, int B, int M, int page, int P, unsigned *status) {
    pdl_wait_primary();
    const int i = blockIdx.x;
    const int a = src[i], z = dst[i];
    bool ok = a >= 0 && a < B && z >= 0 && z < B;
    int T = 0;
    if (ok) {
        // (what a row that another pair writes holds here does not matter: this pair is skipped below)
        T = seqlens[a];
#pragma unroll 4
        for (int k = threadIdx.x; k < M; k += blockDim.x) {  // (no branches: the loads of a round go out together)
            const int old = table[(size_t)z * M + k], e = table[(size_t)a * M + k];
            const int held = e >= 0 && e < P ? refcount[e] : 0;  // (counts only rise in this kernel)
            ok &= old < 0 && ((long long)k * page >= T || held > 0);
        }
        ok = ok && T >= 0 && T <= (long long)M * page;
    }
    for (int k = threadIdx.x; k < n; k += blockDim.x) {
        const int zk = dst[k];
        ok = ok && zk != a && src[k] != z && (k >= i || zk != z);
    }
    if (__syncthreads_and(ok)) {
        for (int k = threadIdx.x; (long long)k * page < T; k += blockDim.x) {
            const int e = table[(size_t)a * M + k];
            table[(size_t)z * M + k] = e;
            atomicAdd(&refcount[e], 1);
        }
        if (threadIdx.x == 0) seqlens[z] = T;
        return;
    }
    if (threadIdx.x == 0) set_status(status, STATUS_PAGES);
}

// ------------------------------------------------------------------ reserve

constexpr int kPlanThreads = 1024;
constexpr int kPlanLanes = 4;    // lanes that share a sequence
constexpr int kScanInts = 16;    // refcounts a thread looks at per step of the free-page scan

// Exclusive sum over the block; `total` gets the whole sum.  Every thread calls it.
__device__ __forceinline__ int block_scan(int x, int *warp_sums, int &total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sums[w] = incl;
    __syncthreads();
    if (w == 0) {
        int s = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += v;
        }
        warp_sums[lane] = s;
    }
    __syncthreads();
    total = warp_sums[31];
    const int r = incl - x + (w ? warp_sums[w - 1] : 0);
    __syncthreads();
    return r;
}

// Entries [lo, hi) of row b that the positions [T, T + n) lie in; empty when
// there is nothing to reserve or the request is out of range (then ok is false).
__device__ __forceinline__ void span(int T, int n, int page, int M, int &lo, int &hi, bool &ok) {
    ok = T >= 0 && n >= 0 && (long long)T + n <= (long long)M * page;
    lo = hi = 0;
    if (ok && n > 0) {
        lo = T / page;
        hi = (int)(((long long)T + n + page - 1) / page);
    }
}

// An entry has to get a page (in the plan below: held != 1) when it has none,
// when it shares one, and when it is out of range or names a page that nobody
// holds, which is flagged.
// The plan, one block: which entries take a page (decided on the reference
// counts before the call), the lowest free pages for them in table order, the
// new table and counts, and per sequence the copy that the second kernel makes.
// All or nothing: with too few free pages nothing changes.
// ws: free pages [P], references to drop [P], jobs [B] (int4).
// Latency-bound: a chain of dependent loads (lengths, entries, counts) and the
// scan.  Each group of lanes keeps what it read of its first sequence's first
// entries, so that up to 256 sequences of a few entries are read once (256 rows
// over 15,000 pages: 7.5 us; read again in step 4, with eight lanes a sequence,
// 12.8 us).  The scan starts at page 0 and ends when it has enough: 0.1 us per
// 1,000 pages in front of the last one taken.  With 1,000 free pages at the end of
// 100,000, a million and two million pages the call takes 18, 113 and 216 us.
__global__ void __launch_bounds__(kPlanThreads)
    pages_reserve_plan(int32_t *table, int32_t *refcount, const int32_t *seqlens, const int32_t *n_new, int B, int M,
                       int page, int P, int32_t *ws_free, int32_t *ws_drop, int4 *ws_job, unsigned *status) {
    extern __shared__ int need[];  // [B], then exclusive sums
    __shared__ int sums[32];
    pdl_wait_primary();
    const int tid = threadIdx.x;
    const int sub = tid & (kPlanLanes - 1), group = tid / kPlanLanes;
    constexpr int kGroups = kPlanThreads / kPlanLanes;
    const int base_lane = (tid & 31) & ~(kPlanLanes - 1);
    const unsigned gmask = ((1u << kPlanLanes) - 1) << base_lane;
    // this lane's first entry of the group's first sequence
    int T0 = 0, n0 = 0, e0 = -1, r0 = 0;
    // 1. how many pages each sequence takes
    for (int b = group; b < B; b += kGroups) {
        int lo, hi, count = 0;
        bool ok;
        const int T = seqlens[b], n = n_new[b];
        span(T, n, page, M, lo, hi, ok);
        if (!ok && sub == 0) set_status(status, STATUS_SEQLEN);
        for (int k = lo + sub; k < hi; k += kPlanLanes) {
            const int e = table[(size_t)b * M + k];
            const int held = e >= 0 && e < P ? refcount[e] : 0;
            if (e >= P || (e >= 0 && held < 1)) set_status(status, STATUS_PAGES);
            count += held != 1 ? 1 : 0;
            if (k == lo + sub && b == group) {
                e0 = e;
                r0 = held;
            }
        }
        if (b == group) {
            T0 = T;
            n0 = n;
        }
#pragma unroll
        for (int o = kPlanLanes / 2; o > 0; o >>= 1) count += __shfl_xor_sync(gmask, count, o);
        if (sub == 0) need[b] = count;
    }
    __syncthreads();
    // 2. their exclusive sums
    const int chunk = (B + kPlanThreads - 1) / kPlanThreads;
    const int b0 = min(B, tid * chunk), b1 = min(B, b0 + chunk);
    int mine = 0, total = 0;
    for (int b = b0; b < b1; ++b) mine += need[b];
    int run = block_scan(mine, sums, total);
    for (int b = b0; b < b1; ++b) {
        const int n = need[b];
        need[b] = run;
        run += n;
    }
    // 3. the `total` lowest free pages
    int found = 0;
    const bool wide = (reinterpret_cast<uintptr_t>(refcount) & 15) == 0;
    for (int base = 0; base < P && found < total; base += kPlanThreads * kScanInts) {
        const int p0 = base + tid * kScanInts;
        unsigned bits = 0;
        if (wide && p0 + kScanInts <= P) {
#pragma unroll
            for (int i = 0; i < kScanInts / 4; ++i) {
                const int4 v = *reinterpret_cast<const int4 *>(refcount + p0 + 4 * i);
                bits |= ((v.x == 0 ? 1u : 0u) | (v.y == 0 ? 2u : 0u) | (v.z == 0 ? 4u : 0u) | (v.w == 0 ? 8u : 0u))
                        << (4 * i);
            }
        } else {
            for (int i = 0; i < kScanInts; ++i)
                if (p0 + i < P && refcount[p0 + i] == 0) bits |= 1u << i;
        }
        int here;
        int at = found + block_scan(__popc(bits), sums, here);
        for (; bits && at < total; bits &= bits - 1) ws_free[at++] = p0 + __ffs(bits) - 1;
        found += here;
    }
    __syncthreads();  // (block_scan ends with one; this orders the last writes of ws_free and need)
    const bool enough = found >= total;
    if (!enough && tid == 0) set_status(status, STATUS_PAGES);
    // 4. the new entries; references that they drop are only noted, since other
    //    sequences' decisions still read the counts
    for (int b = group; b < B; b += kGroups) {
        int lo, hi;
        bool ok;
        const bool first = b == group;
        const int T = first ? T0 : seqlens[b];
        span(T, first ? n0 : n_new[b], page, M, lo, hi, ok);
        int at = need[b];
        int4 job = make_int4(0, 0, 0, 0);
        for (int k0 = lo; k0 < hi && enough; k0 += kPlanLanes) {
            const int k = k0 + sub;
            int e = -1, held = 1;
            if (first && k0 == lo) {
                e = e0;
                held = k < hi ? r0 : 1;
            } else if (k < hi) {
                e = table[(size_t)b * M + k];
                held = e >= 0 && e < P ? refcount[e] : 0;
            }
            const bool take = held != 1;
            const unsigned votes = (__ballot_sync(gmask, take) & gmask) >> base_lane;
            if (take) {
                const int slot = at + __popc(votes & ((1u << sub) - 1));
                const int fresh = ws_free[slot];
                ws_drop[slot] = held > 1 ? e : -1;
                table[(size_t)b * M + k] = fresh;
                if (held > 1 && k == lo) job = make_int4(e, fresh, T - lo * page, 0);
            }
            at += __popc(votes);
        }
        // (entry lo belongs to lane 0 of the group, which holds the job)
        if (sub == 0) ws_job[b] = job;
    }
    __syncthreads();
    // 5. the counts
    if (enough)
        for (int i = tid; i < total; i += kPlanThreads) {
            refcount[ws_free[i]] = 1;
            if (ws_drop[i] >= 0) atomicSub(&refcount[ws_drop[i]], 1);
        }
}

// Copies the rows [0, rows) of every KV head from the page a sequence shared
// to its own.  Grid: (sequence, K or V).
__global__ void __launch_bounds__(256)
    pages_copy_rows(uint4 *k_pages, uint4 *v_pages, const int4 *ws_job, int G, int page, int row16) {
    pdl_wait_primary();
    const int4 job = ws_job[blockIdx.x];
    if (job.z <= 0) return;
    uint4 *pool = blockIdx.y ? v_pages : k_pages;
    const int per = job.z * row16;  // pieces per KV head
    const size_t stride = (size_t)page * row16;
    const uint4 *from = pool + (size_t)job.x * G * stride;
    uint4 *to = pool + (size_t)job.y * G * stride;
    for (int i = threadIdx.x; i < G * per; i += blockDim.x) {
        const int g = i / per, e = i - g * per;
        to[g * stride + e] = from[g * stride + e];
    }
}

}  // namespace

cudaError_t launch_cache_append(const void *k_new, const void *v_new, const int32_t *cu, const int32_t *seqlens,
                                int32_t *seqlens_out, void *k_cache, void *v_cache, const CacheView &c, int N,
                                int num_sms, unsigned *status, cudaStream_t st) {
    const long long blocks = ((long long)N + kAppendWarps - 1) / kAppendWarps;
    const int grid = (int)(blocks < 1 ? 1 : blocks > num_sms * 64ll ? num_sms * 64ll : blocks);
    return dec::launch_pdl(cache_append_kernel, dim3(grid), dim3(kAppendWarps * 32), 0, st,
                           static_cast<const uint4 *>(k_new), static_cast<const uint4 *>(v_new), cu, seqlens,
                           seqlens_out, static_cast<uint4 *>(k_cache), static_cast<uint4 *>(v_cache), c, N, status);
}

cudaError_t launch_cache_compact(void *k_cache, void *v_cache, const int32_t *seqlens, const int32_t *keep,
                                 const int32_t *n_keep, int32_t *seqlens_out, const CacheView &c, int m,
                                 unsigned *status, cudaStream_t st) {
    auto launch = [&](auto kern) {
        return dec::launch_pdl(kern, dim3(c.B * c.G * 2), dim3(kCompactThreads), 0, st, static_cast<uint4 *>(k_cache),
                               static_cast<uint4 *>(v_cache), seqlens, keep, n_keep, seqlens_out, c, m, status);
    };
    switch (c.row16) {  // d_h 64 or 128, bf16 or fp32
    case 8: return launch(cache_compact_kernel<8>);
    case 16: return launch(cache_compact_kernel<16>);
    default: return launch(cache_compact_kernel<32>);
    }
}

cudaError_t launch_pages_release(int32_t *table, int32_t *refcount, const int32_t *lengths, int B, int M, int page,
                                 int P, unsigned *status, cudaStream_t st) {
    return dec::launch_pdl(pages_release_kernel, dim3(B), dim3(kPageThreads), 0, st, table, refcount, lengths, M, page,
                           P, status);
}

cudaError_t launch_pages_fork(int32_t *table, int32_t *refcount, int32_t *seqlens, const int32_t *src,
                              const int32_t *dst, int n, int B, int M, int page, int P, unsigned *status,
                              cudaStream_t st) {
    return dec::launch_pdl(pages_fork_kernel, dim3(n), dim3(kPageThreads), 0, st, table, refcount, seqlens, src, dst,
                           n, B, M, page, P, status);
}

size_t pages_reserve_workspace(int B, int P) {
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    return up((size_t)B * sizeof(int4)) + 2 * up((size_t)P * 4);
}

cudaError_t launch_pages_reserve(int32_t *table, int32_t *refcount, const int32_t *seqlens, const int32_t *n_new,
                                 void *k_pages, void *v_pages, int B, int G, int M, int page, int P, int row16,
                                 void *workspace, unsigned *status, cudaStream_t st) {
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    int4 *jobs = reinterpret_cast<int4 *>(ws);
    int32_t *free_pages = reinterpret_cast<int32_t *>(ws + up((size_t)B * sizeof(int4)));
    int32_t *drops = reinterpret_cast<int32_t *>(ws + up((size_t)B * sizeof(int4)) + up((size_t)P * 4));
    cudaError_t e = dec::launch_pdl(pages_reserve_plan, dim3(1), dim3(kPlanThreads), (size_t)B * 4, st, table,
                                    refcount, seqlens, n_new, B, M, page, P, free_pages, drops, jobs, status);
    if (e != cudaSuccess) return e;
    return dec::launch_pdl(pages_copy_rows, dim3(B, 2), dim3(256), 0, st, static_cast<uint4 *>(k_pages),
                           static_cast<uint4 *>(v_pages), (const int4 *)jobs, G, page, row16);
}

}  // namespace gqa
