// decode_sparse.cu -- Polar Attention decode over the pages that a cheap score
// selects for each (sequence, kv head).
//
// A page's key bounds (smallest and largest key of each dimension) give the
// largest product any key of the page can have with a query q:
//
//   score(q) = sum_d max(q_d lo_d, q_d hi_d)
//
// A kv group's score is the largest of its query heads'.  The newest page is
// always read, then the pages with the highest scores (lower page on a tie),
// `keep` in all.  Selected pages go through the same streaming state as the
// other decodes (decode_rows.cuh).
#include <algorithm>
#include <atomic>

#include "decode_rows.cuh"
#include "polar_internal.h"
#include "tc_common.cuh"

namespace polar {
namespace {

constexpr int kSmem = kRingStages * kStageBytes + 1024;  // + alignment slack
constexpr int kScoreThreads = 256;
constexpr int kSelThreads = 512;
constexpr int kSelKeys = 10240;  // keys that the selection holds in shared memory (40 KB)
constexpr int kScorePages = 512;   // pages of a score block at most
constexpr int kScoreRing = 8;      // pages that a lane has in flight
constexpr int kFusedPages = 1024;  // rows up to which the selection's block scores its pages itself
constexpr int kMaxCluster = 8;

__device__ __forceinline__ bool valid_len(int len, int max_pages) {
    return len >= 1 && len <= static_cast<long long>(max_pages) * kPage;
}

// Scores as unsigned keys in the order of the values; NaN above everything
// but the newest page, so that a page that is not comparable is read.
__device__ __forceinline__ uint32_t score_key(float x) {
    if (x != x) return 0xfffffffeu;
    const uint32_t b = __float_as_uint(x + 0.0f);  // -0 ties with 0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// The score of a key (a NaN for the highest, which no score has).
__device__ __forceinline__ float key_score(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// A page's score in 64 bits, rounded once: what the pages are ordered by.  By a
// warp: lane (head of four, eight dimensions).
template <int G>
__device__ __forceinline__ uint32_t exact_key(const uint4 *__restrict__ q,
                                              const uint4 *__restrict__ b, int lane) {
    const int c = lane & 7;
    const uint4 lo = __ldg(b + c), hi = __ldg(b + 8 + c);
    const uint32_t lw[4] = {lo.x, lo.y, lo.z, lo.w}, hw[4] = {hi.x, hi.y, hi.z, hi.w};
    uint32_t best = 0;
#pragma unroll
    for (int h0 = 0; h0 < G; h0 += 4) {
        const int h = min(h0 + (lane >> 3), G - 1);
        const uint4 x = __ldg(q + h * 8 + c);
        const uint32_t qw[4] = {x.x, x.y, x.z, x.w};
        double s = 0.0;
#pragma unroll
        for (int d = 0; d < 8; ++d) {
            const float qd = __uint_as_float(d & 1 ? qw[d >> 1] & 0xffff0000u : qw[d >> 1] << 16);
            const uint32_t e = qd < 0.f ? lw[d >> 1] : hw[d >> 1];
            s = fma(static_cast<double>(qd),
                    static_cast<double>(__uint_as_float(d & 1 ? e & 0xffff0000u : e << 16)), s);
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) s += __shfl_xor_sync(~0u, s, o);
        best = max(best, score_key(static_cast<float>(s)));
    }
    return __reduce_max_sync(~0u, best);
}

__device__ __forceinline__ void copy_async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
                 : "memory");
}

// Scores of pages 0 .. count - 1 of one (sequence, kv head), by a block of
// kThreads, in fp32 with a bound on each one's error, from which the selection
// sees where 64 bits are needed: sink(page, score, bound) in one thread per page.
// phys(p) is the pool's page, or -1 (ranks last).  ring: kScoreRing * 2 * kThreads
// vectors of shared memory.
//
// Eight lanes take a page for up to four query heads, eight dimensions each (a
// group of eight heads takes sixteen lanes).  A lane copies its part of a page's
// bounds into its own places of the ring, kScoreRing pages ahead, so that the
// copies in flight cost no registers and nothing waits for another thread.
// A product of two bf16 is exact in fp32 (a subnormal one aside), so a score is
// at most 4 roundings in a lane, one to join its two sums and 3 across lanes
// from the exact sum: off by at most 8 * 2^-24 * sum_d max_h |q_d| max(|lo_d|,
// |hi_d|), which with that sum's own roundings is below 12 * 2^-24 of it, and
// 2^-100 for subnormals.
template <int G, int kThreads, typename Phys, typename Sink>
__device__ __forceinline__ void score_pages(const uint4 *__restrict__ q,
                                            const uint4 *__restrict__ bounds, int g, int Hkv,
                                            int count, uint4 *ring, Phys &&phys, Sink &&sink) {
    constexpr int GH = G < 4 ? G : 4;       // heads of a lane
    constexpr int kLanes = 8 * (G / GH);    // lanes of a page
    constexpr int kStep = kThreads / kLanes;
    const int tid = threadIdx.x, c = tid & 7, part = tid % kLanes / 8;
    float2 qf[GH][4], qm[4];
#pragma unroll
    for (int d = 0; d < 4; ++d) qm[d] = make_float2(0.f, 0.f);
#pragma unroll
    for (int h = 0; h < GH; ++h) {
        const uint4 x = __ldg(q + (part * GH + h) * 8 + c);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const float2 v = make_float2(__uint_as_float(w[d] << 16),
                                         __uint_as_float(w[d] & 0xffff0000u));
            qf[h][d] = v;
            qm[d] = make_float2(fmaxf(qm[d].x, fabsf(v.x)), fmaxf(qm[d].y, fabsf(v.y)));
        }
    }
    const int p0 = tid / kLanes, steps = (count + kStep - 1) / kStep;
    auto fetch = [&](int step) {
        const int p = p0 + step * kStep, x = p < count ? phys(p) : -1;
        if (x >= 0) {
            const uint4 *b = bounds + (static_cast<size_t>(x) * Hkv + g) * 16 + c;
            uint4 *dst = ring + step % kScoreRing * 2 * kThreads + tid;
            copy_async16(dst, b);
            copy_async16(dst + kThreads, b + 8);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int e = 0; e < kScoreRing - 1; ++e) fetch(e);
    for (int step = 0; step < steps; ++step) {  // the same number in every lane: it shuffles
        fetch(step + kScoreRing - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kScoreRing - 1) : "memory");
        const int p = p0 + step * kStep;
        const uint4 *src = ring + step % kScoreRing * 2 * kThreads + tid;
        const uint4 lo4 = src[0], hi4 = src[kThreads];
        const uint32_t lw[4] = {lo4.x, lo4.y, lo4.z, lo4.w};
        const uint32_t hw[4] = {hi4.x, hi4.y, hi4.z, hi4.w};
        float2 acc[GH], mag = make_float2(0.f, 0.f);
#pragma unroll
        for (int h = 0; h < GH; ++h) acc[h] = make_float2(0.f, 0.f);
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const float2 lo = make_float2(__uint_as_float(lw[d] << 16),
                                          __uint_as_float(lw[d] & 0xffff0000u));
            const float2 hi = make_float2(__uint_as_float(hw[d] << 16),
                                          __uint_as_float(hw[d] & 0xffff0000u));
            const float2 m = make_float2(fmaxf(fabsf(lo.x), fabsf(hi.x)),
                                         fmaxf(fabsf(lo.y), fabsf(hi.y)));
            mag = f2_fma(qm[d], m, mag);
#pragma unroll
            for (int h = 0; h < GH; ++h)
                acc[h] = f2_add(acc[h], make_float2(fmaxf(qf[h][d].x * lo.x, qf[h][d].x * hi.x),
                                                    fmaxf(qf[h][d].y * lo.y, qf[h][d].y * hi.y)));
        }
        // Sum over the eight lanes; where a lane has several heads, each step
        // halves them instead of repeating the sum.
        float err = mag.x + mag.y, best;
        float s[GH];
#pragma unroll
        for (int h = 0; h < GH; ++h) s[h] = acc[h].x + acc[h].y;
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1)  // over both halves of eight heads: an upper bound
            err = o < 8 ? err + __shfl_xor_sync(~0u, err, o)
                        : fmaxf(err, __shfl_xor_sync(~0u, err, o));
        if constexpr (GH == 4) {
            const bool up = c & 4, up2 = c & 2;
            const float s0 = (up ? s[2] : s[0]) + __shfl_xor_sync(~0u, up ? s[0] : s[2], 4);
            const float s1 = (up ? s[3] : s[1]) + __shfl_xor_sync(~0u, up ? s[1] : s[3], 4);
            best = (up2 ? s1 : s0) + __shfl_xor_sync(~0u, up2 ? s0 : s1, 2);
            best += __shfl_xor_sync(~0u, best, 1);
            best = fmaxf(best, __shfl_xor_sync(~0u, best, 2));
            best = fmaxf(best, __shfl_xor_sync(~0u, best, 4));
        } else if constexpr (GH == 2) {
            const bool up = c & 4;
            best = (up ? s[1] : s[0]) + __shfl_xor_sync(~0u, up ? s[0] : s[1], 4);
            best += __shfl_xor_sync(~0u, best, 2);
            best += __shfl_xor_sync(~0u, best, 1);
            best = fmaxf(best, __shfl_xor_sync(~0u, best, 4));
        } else {
            best = s[0] + __shfl_xor_sync(~0u, s[0], 4);
            best += __shfl_xor_sync(~0u, best, 2);
            best += __shfl_xor_sync(~0u, best, 1);
        }
        if constexpr (kLanes == 16) best = fmaxf(best, __shfl_xor_sync(~0u, best, 8));
        // Bounds that are not finite make err so, too: 64 bits then decide.
        if (tid % kLanes == 0 && p < count) {
            const bool ok = phys(p) >= 0;
            sink(p, ok ? best : -INFINITY, ok ? fmaf(err, 12.0f * 0x1p-24f, 0x1p-100f) : 0.f);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// Block (pages, kv head, sequence) of long rows.
template <int G>
__global__ void __launch_bounds__(kScoreThreads, 3)
sparse_score_kernel(const uint4 *__restrict__ q, const uint4 *__restrict__ bounds,
                    const int32_t *__restrict__ page_table, const int32_t *__restrict__ seqlens,
                    float2 *__restrict__ scores, int num_pages, int max_pages, int Hkv, int keep,
                    int pages_per_block) {
    extern __shared__ uint4 score_ring[];
    __shared__ int pages[kScorePages];
    const int g = blockIdx.y, seq = blockIdx.z;
    const int len = seqlens[seq];
    if (!valid_len(len, max_pages)) return;  // reported by the selection
    const int npg = (len + kPage - 1) / kPage;
    const int first = blockIdx.x * pages_per_block, count = min(npg - first, pages_per_block);
    if (npg <= keep || count <= 0) return;  // every page is read, or none is here
    const int32_t *pt = page_table + static_cast<size_t>(seq) * max_pages + first;
    for (int p = threadIdx.x; p < count; p += kScoreThreads) {
        const int x = pt[p];
        pages[p] = x >= 0 && x < num_pages ? x : -1;
    }
    __syncthreads();
    const size_t row = static_cast<size_t>(seq) * Hkv + g;
    float2 *out = scores + row * max_pages + first;
    score_pages<G, kScoreThreads>(q + row * G * 8, bounds, g, Hkv, count, score_ring,
                                  [&](int p) { return pages[p]; },
                                  [&](int p, float s, float e) { out[p] = make_float2(s, e); });
}

struct SelectArgs {
    const uint4 *q, *bounds;
    const float2 *scores;
    const int32_t *page_table, *seqlens;
    int32_t *selected;  // [num_seqs, Hkv, keep]: ascending pages, then -1
    uint32_t *keys;     // per (sequence, head) row of max_pages: past kSelKeys pages
    int num_pages, max_pages, Hkv, keep;
    int *status;
};

// Block (kv head, sequence): the pages with the highest scores, ascending.
//
// A radix selection over keys in the scores' order finds the k-th highest.
// Scores lie close together, so its digits begin at the highest bit in which
// two keys differ, and it ends as soon as a bin is taken whole.  Scores come in
// fp32 with error bounds; with E the largest of them and T the k-th highest
// score, the k-th highest exact score is within E of T, so a page above T + 2E
// is taken and one below T - 2E is not, whatever the roundings.  Where the pages
// between are not all taken, they get their exact scores, and the selection
// runs once more on (taken, exact, not taken).
//
// kScores: the block scores its pages itself, for rows short enough that a
// launch costs more than one block's reading them (measured at 512 pages, one
// sequence: XXX us against XXX with a launch of its own).
template <int G, bool kScores>
__global__ void __launch_bounds__(kSelThreads) sparse_select_kernel(const SelectArgs a) {
    extern __shared__ uint4 score_ring[];  // kScores: the ring, then the pages and the keys
    constexpr int kRingVecs = kScores ? kScoreRing * 2 * kSelThreads : 0;
    int *pages = reinterpret_cast<int *>(score_ring + kRingVecs);
    uint32_t *held = reinterpret_cast<uint32_t *>(pages) + (kScores ? kFusedPages : 0);
    __shared__ int hist[256];
    __shared__ uint32_t ends[4][kSelThreads / 32];
    __shared__ int counts[2][kSelThreads / 32];
    __shared__ int s_bin, s_left, s_whole;
    const int g = blockIdx.x, seq = blockIdx.y, tid = threadIdx.x;
    const int lane = tid & 31, w = tid >> 5;
    constexpr int kWarps = kSelThreads / 32;
    const int len = a.seqlens[seq];
    wait_for_previous_kernel();  // every block, so that a later kernel's wait covers the scores
    if (!valid_len(len, a.max_pages)) {
        if (g == 0 && tid == 0) record_error(a.status, POLAR_ERR_BAD_SEQLEN);
        return;
    }
    const int npg = (len + kPage - 1) / kPage;
    const size_t row = static_cast<size_t>(seq) * a.Hkv + g;
    int32_t *out = a.selected + row * a.keep;
    if (npg <= a.keep) {
        for (int i = tid; i < a.keep; i += kSelThreads) out[i] = i < npg ? i : -1;
        return;
    }
    if (tid == 0) out[a.keep - 1] = npg - 1;  // the newest page, without a score
    if (a.keep == 1) return;
    const int n = npg - 1, take = a.keep - 1;
    uint32_t *keys = n <= kSelKeys ? held : a.keys + row * a.max_pages;

    uint32_t err = 0;  // as bits: in the order of the values, and a NaN above all
    if constexpr (kScores) {
        const int32_t *pt = a.page_table + static_cast<size_t>(seq) * a.max_pages;
        for (int p = tid; p < n; p += kSelThreads) {
            const int x = pt[p];
            pages[p] = x >= 0 && x < a.num_pages ? x : -1;
        }
        __syncthreads();
        score_pages<G, kSelThreads>(a.q + row * G * 8, a.bounds, g, a.Hkv, n, score_ring,
                                    [&](int p) { return pages[p]; },
                                    [&](int p, float s, float e) {
                                        keys[p] = score_key(s);
                                        err = max(err, __float_as_uint(e) & 0x7fffffffu);
                                    });
    } else {
        const float2 *scores = a.scores + row * a.max_pages;
#pragma unroll 8
        for (int p = tid; p < n; p += kSelThreads) {
            const float2 x = scores[p];
            keys[p] = score_key(x.x);
            err = max(err, __float_as_uint(x.y) & 0x7fffffffu);
        }
    }
    if (tid < 256) hist[tid] = 0;

    // Keys above floor_key are taken, and the first `left` of those equal to it;
    // `open`: low bits that do not count.
    uint32_t floor_key = 0, open = 0;
    int left = 0;
    auto radix = [&]() {
        uint32_t all_and = ~0u, all_or = 0u;
        for (int p = tid; p < n; p += kSelThreads) {
            all_and &= keys[p];
            all_or |= keys[p];
        }
        all_and = __reduce_and_sync(~0u, all_and);
        all_or = __reduce_or_sync(~0u, all_or);
        if (lane == 0) {
            ends[0][w] = all_and;
            ends[1][w] = all_or;
        }
        __syncthreads();
        for (int i = 0; i < kWarps; ++i) {
            all_and &= ends[0][i];
            all_or |= ends[1][i];
        }
        int bits = 32 - __clz(static_cast<int>(all_and ^ all_or));
        floor_key = bits == 32 ? 0u : all_and >> bits << bits;
        left = take;
        while (bits > 0) {
            const int shift = max(bits - 8, 0);
            const uint32_t digit = (1u << (bits - shift)) - 1;
            for (int p = tid; p < n; p += kSelThreads) {
                const uint32_t k = keys[p];
                if (bits == 32 || (k ^ floor_key) >> bits == 0)
                    atomicAdd(&hist[k >> shift & digit], 1);
            }
            __syncthreads();
            if (w == 0) {  // the left-th key's bin from above: lane l has bins 255-8l .. 248-8l
                int h[8], sum = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) sum += h[e] = hist[255 - 8 * lane - e];
                int upto = sum;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(~0u, upto, o);
                    if (lane >= o) upto += y;
                }
                int before = upto - sum;
                if (before < left && left <= upto) {
                    bool found = false;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if (!found && left <= before + h[e]) {
                            s_bin = 255 - 8 * lane - e;
                            s_left = left - before;
                            s_whole = left - before == h[e];
                            found = true;
                        }
                        before += h[e];
                    }
                }
            }
            __syncthreads();
            if (tid < 256) hist[tid] = 0;
            floor_key |= static_cast<uint32_t>(s_bin) << shift;
            left = s_left;
            const bool whole = s_whole != 0;
            bits = shift;
            __syncthreads();
            if (whole) break;
        }
        open = bits > 0 ? (1u << bits) - 1 : 0u;
    };
    __syncthreads();
    radix();

    // The pages whose place the roundings could change.
    err = __reduce_max_sync(~0u, err);
    if (lane == 0) ends[2][w] = err;
    // T: the lowest key that is taken (with a bin taken whole, the lowest in it).
    uint32_t lowest = ~0u;
    for (int p = tid; p < n; p += kSelThreads) {
        const uint32_t k = keys[p];
        if ((k & ~open) >= floor_key) lowest = min(lowest, k);
    }
    lowest = __reduce_min_sync(~0u, lowest);
    if (lane == 0) ends[3][w] = lowest;
    __syncthreads();
    for (int i = 0; i < kWarps; ++i) {
        lowest = min(lowest, ends[3][i]);
        err = max(err, ends[2][i]);
    }
    const float E = __uint_as_float(err);
    const float T = key_score(lowest);
    // Rounded outwards by more than the sums' own roundings and the exact
    // scores' rounding to fp32.
    const float reach = 2.0f * E + (fabsf(T) + E) * 0x1p-22f;
    const float above = T + reach, below = T - reach;
    // Where nothing can change, ties included, the fp32 keys' choice stands.
    auto place = [&](uint32_t k) {  // 2: taken, 0: not taken, 1: to be seen
        const float x = key_score(k);
        return x > above ? 2 : x < below ? 0 : 1;
    };
    int mid = 0, sure = 0;
    for (int p = tid; p < n; p += kSelThreads) {
        const int c = place(keys[p]);
        mid += c == 1;
        sure += c == 2;
    }
    mid = __reduce_add_sync(~0u, mid);
    sure = __reduce_add_sync(~0u, sure);
    if (lane == 0) {
        counts[0][w] = mid;
        counts[1][w] = sure;
    }
    __syncthreads();
    mid = sure = 0;
    for (int i = 0; i < kWarps; ++i) {
        mid += counts[0][i];
        sure += counts[1][i];
    }
    if (sure + mid != take) {
        const int32_t *pt = a.page_table + static_cast<size_t>(seq) * a.max_pages;
        const uint4 *q = a.q + row * G * 8;
        for (int first = 32 * w; first < n; first += kSelThreads) {
            const int p = first + lane, c = p < n ? place(keys[p]) : 0;
            const int phys = c == 1 ? pt[p] : -1;
            uint32_t k = c == 2 ? 0xffffffffu : 0u;
            for (uint32_t todo = __ballot_sync(~0u, phys >= 0 && phys < a.num_pages); todo;
                 todo &= todo - 1) {
                const int who = __ffs(todo) - 1;
                const size_t page = __shfl_sync(~0u, phys, who);
                const uint32_t e = exact_key<G>(q, a.bounds + (page * a.Hkv + g) * 16, lane);
                if (lane == who) k = e;
            }
            if (p < n) keys[p] = k;
        }
        __syncthreads();
        radix();
    } else {  // all of `mid` are taken
        floor_key = lowest;
        open = 0;
        left = n;
    }

    // Ascending order: warp w has pages w * per .. w * per + per - 1.
    const int per = (n + kSelThreads - 1) / kSelThreads * 32;
    const int p0 = min(w * per, n), p1 = min(p0 + per, n);
    int gs = 0, es = 0;
    for (int p = p0 + lane; p < p0 + per; p += 32) {
        const uint32_t k = p < p1 ? keys[p] & ~open : 0u;
        gs += __popc(__ballot_sync(~0u, p < p1 && k > floor_key));
        es += __popc(__ballot_sync(~0u, p < p1 && k == floor_key));
    }
    __syncthreads();  // the counts above are read
    if (lane == 0) {
        counts[0][w] = gs;
        counts[1][w] = es;
    }
    __syncthreads();
    gs = es = 0;
    for (int i = 0; i < w; ++i) {
        gs += counts[0][i];
        es += counts[1][i];
    }
    const uint32_t below_me = (1u << lane) - 1;
    for (int p = p0 + lane; p < p0 + per; p += 32) {
        const uint32_t k = p < p1 ? keys[p] & ~open : 0u;
        const bool gt = p < p1 && k > floor_key, eq = p < p1 && k == floor_key;
        const uint32_t mg = __ballot_sync(~0u, gt), me = __ballot_sync(~0u, eq);
        const int gi = gs + __popc(mg & below_me), ei = es + __popc(me & below_me);
        if (gt || (eq && ei < left)) out[gi + min(ei, left)] = p;
        gs += __popc(mg);
        es += __popc(me);
    }
}

struct SparseArgs {
    const int32_t *page_table, *seqlens, *selected;
    const __nv_bfloat16 *q;
    const float *u;
    __nv_bfloat16 *out;
    float *neff, *partials;
    int *status;
    int num_pages, max_pages, Hq, Hkv, keep, splits;
    Epilogue ep;
};

// Positions of the selected pages: all are full but the newest.
__device__ __forceinline__ int selected_tokens(int len, int keep) {
    const int npg = (len + kPage - 1) / kPage;
    return (min(npg, keep) - 1) * kPage + len - (npg - 1) * kPage;
}

// CTA (part of the selected pages, kv head, sequence): the parts are equal
// shares of what is selected.  A cluster along x merges its CTAs' states; with
// one cluster per (kv head, sequence) it writes the rows, else a partial.
template <int G>
__global__ void __launch_bounds__(kRowThreads)
sparse_split_kernel(const __grid_constant__ CUtensorMap kv_map, const SparseArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) PageRing ring;
    const int g = blockIdx.y, seq = blockIdx.z;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gq = lane >> 2, tq = lane & 3;

    const int len = a.seqlens[seq];
    if (!valid_len(len, a.max_pages)) {  // the whole cluster; reported by the selection
        wait_for_previous_kernel();
        return;
    }
    const int npg = (len + kPage - 1) / kPage;
    const int nsel = min(npg, a.keep), per = (nsel + gridDim.x - 1) / gridDim.x;
    const int p0 = min(static_cast<int>(blockIdx.x) * per, nsel);
    const int np = min(nsel, p0 + per) - p0;

    RowTile<1> tile[1];
    tile[0].clear();
    if (w < kRowWarps)
        tile[0].load_row(0,
                         gq < G ? a.q + (static_cast<size_t>(seq) * a.Hq + g * G + gq) * kHeadDim
                                : nullptr,
                         tq,
                         a.ep.s * length_temperature(
                             static_cast<float>(selected_tokens(len, a.keep)), a.ep.alpha,
                             a.ep.L) * kLog2e);
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&kv_map);
        init_ring(ring);
    }
    wait_for_previous_kernel();
    {
        const int32_t *pt = a.page_table + static_cast<size_t>(seq) * a.max_pages;
        const int32_t *sel = a.selected + (static_cast<size_t>(seq) * a.Hkv + g) * a.keep + p0;
        for (int i = threadIdx.x; i < np; i += kRowThreads) {
            const int x = pt[sel[i]];
            ring.page[i] = x >= 0 && x < a.num_pages ? x : -1;
            if (ring.page[i] < 0) record_error(a.status, POLAR_ERR_BAD_PAGE);
        }
    }
    __syncthreads();
    const uint32_t sbase = smem_u32(smem);
    if (w == kRowWarps) {
        if (lane == 0)
            copy_steps(ring, np, a.status, [&](int kk, int st, uint64_t *bar) {
                const int phys = ring.page[kk];
                if (phys < 0) {
                    mbar_arrive(bar);
                    return;
                }
                mbar_arrive_expect_tx(bar, kStageBytes);
                const int row = (phys * 2 * a.Hkv + g) * kPage;  // K block of the kv head
                tma_load_2d(smem + st * kStageBytes, &kv_map, 0, row, bar);
                tma_load_2d(smem + st * kStageBytes + kChunkBytes, &kv_map, 0,
                            row + a.Hkv * kPage, bar);
            });
        __syncwarp();
    } else {
        // The newest page is the last that is selected; all others are full.
        const uint64_t newest = first_tokens(len - (npg - 1) * kPage);
        compute_steps(ring, np, lane, a.status, [&](int kk, int st) {
            const uint32_t kb = sbase + st * kStageBytes;
            if (ring.page[kk] >= 0)
                page_step<1, 1>(tile, kb, kb + kChunkBytes, w, lane,
                                p0 + kk == nsel - 1 ? newest : ~0ull);
        });
    }
    let_next_kernel_start();
    reduce_rows<1, 1>(tile, reinterpret_cast<float *>(smem), G, w, lane,
                      [&](int r, bool real, const RowState &x) {
        const size_t row = static_cast<size_t>(seq) * a.Hq + g * G + r;
        if (a.splits > 1)
            store_part(x, a.partials + (row * a.splits + blockIdx.x / cluster_size()) *
                                           kPartialFloats, real);
        else
            finish_row(x, selected_tokens(len, a.keep), a.ep, a.u + (g * G + r) * kHeadDim,
                       a.out + row * kHeadDim, a.neff ? a.neff + row : nullptr, real);
    });
}

// Eight lanes per (sequence, query head).
__global__ void __launch_bounds__(128) sparse_merge_kernel(const SparseArgs a, int rows) {
    int row = blockIdx.x * 16 + (threadIdx.x >> 3);
    bool real = row < rows;
    row = min(row, rows - 1);
    const int len = a.seqlens[row / a.Hq];
    real = real && valid_len(len, a.max_pages);
    wait_for_previous_kernel();
    const float *base = a.partials + static_cast<size_t>(row) * a.splits * kPartialFloats;
    finish_row(merge_parts(a.splits, [&](int k) { return base + k * kPartialFloats; }),
               selected_tokens(len, a.keep), a.ep, a.u + (row % a.Hq) * kHeadDim,
               a.out + static_cast<size_t>(row) * kHeadDim, a.neff ? a.neff + row : nullptr, real);
}

constexpr int kScoreSmem = kScoreRing * 2 * kScoreThreads * 16;
constexpr int kFusedSmem = kScoreRing * 2 * kSelThreads * 16 + 2 * kFusedPages * 4;

struct Layout {  // the workspace: scores, keys (long rows), selected pages, partials
    size_t keys, selected, partials, total;
    int cluster, splits;  // CTAs of a cluster, clusters of a (sequence, kv head)
};

Layout layout(int num_seqs, int max_pages, int keep, int Hq, int Hkv) {
    Layout l;
    const int pages = std::min(keep, max_pages);
    const long long heads = static_cast<long long>(num_seqs) * Hkv;
    // Enough CTAs for four on each of 148 SMs, of at least two pages each.
    l.cluster = 1;
    while (l.cluster < kMaxCluster && heads * l.cluster < 148 * 4 && l.cluster * 4 <= pages)
        l.cluster *= 2;
    l.splits = 1;
    while ((heads * l.cluster * l.splits * 2 <= 148 * 4 && l.cluster * l.splits * 16 <= pages) ||
           l.cluster * l.splits * kMaxSteps < pages)
        l.splits *= 2;
    auto pad = [](size_t x) { return (x + 15) / 16 * 16; };
    l.keys = pad(heads * max_pages * 8);
    l.selected = l.keys + (max_pages > kSelKeys ? pad(heads * max_pages * 4) : 0);
    l.partials = l.selected + pad(heads * keep * 4);
    l.total = l.partials + (l.splits > 1 ? static_cast<size_t>(num_seqs) * Hq * l.splits *
                                               kPartialFloats * sizeof(float) : 0);
    return l;
}

template <int G>
cudaError_t launch_all(const SparseLaunch &a, const CUtensorMap &map, const Layout &l) {
    static std::atomic<uint64_t> configured{0};  // one bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(configured.load() & bit)) {
        e = cudaFuncSetAttribute(sparse_split_kernel<G>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kSmem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(sparse_score_kernel<G>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, kScoreSmem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(sparse_select_kernel<G, true>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, kFusedSmem);
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit);
    }
    char *ws = static_cast<char *>(a.workspace);
    float2 *scores = reinterpret_cast<float2 *>(ws);
    int32_t *sel = a.selected ? a.selected : reinterpret_cast<int32_t *>(ws + l.selected);
    const uint4 *q = static_cast<const uint4 *>(a.q), *bounds = static_cast<const uint4 *>(a.bounds);
    // Rows that may hold more pages than are kept are scored: long ones by a
    // kernel of many blocks, short ones by the selection's own block.
    const bool scored = a.max_pages > a.keep, fused = scored && a.max_pages <= kFusedPages;
    if (scored && !fused) {
        // Three blocks fit an SM; about six, since lengths differ.  A step is 32
        // pages (16 for groups of eight heads).
        const int step = kScoreThreads / (G == 8 ? 16 : 8);
        const long long all = static_cast<long long>(a.num_seqs) * a.Hkv *
                              ((a.max_pages + step - 1) / step);
        const int per = step * static_cast<int>(
            std::clamp<long long>(all / (148 * 6), 1, kScorePages / step));
        sparse_score_kernel<G><<<dim3((a.max_pages + per - 1) / per, a.Hkv, a.num_seqs),
                                 kScoreThreads, kScoreSmem, a.stream>>>(
            q, bounds, a.page_table, a.seqlens, scores, a.num_pages, a.max_pages, a.Hkv, a.keep,
            per);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        count_launches(1);
    }
    SelectArgs s{q, bounds, scores, a.page_table, a.seqlens, sel,
                 reinterpret_cast<uint32_t *>(ws + l.keys), a.num_pages, a.max_pages, a.Hkv,
                 a.keep, a.status};
    if (fused)
        e = launch_ex(sparse_select_kernel<G, true>, dim3(a.Hkv, a.num_seqs), kSelThreads,
                      kFusedSmem, 1, false, a.stream, s);
    else
        e = launch_ex(sparse_select_kernel<G, false>, dim3(a.Hkv, a.num_seqs), kSelThreads,
                      std::min(a.max_pages, kSelKeys) * sizeof(uint32_t), 1, scored, a.stream, s);
    if (e != cudaSuccess) return e;
    SparseArgs p;
    p.page_table = a.page_table; p.seqlens = a.seqlens; p.selected = sel;
    p.q = static_cast<const __nv_bfloat16 *>(a.q); p.u = a.u;
    p.out = static_cast<__nv_bfloat16 *>(a.out); p.neff = a.neff;
    p.partials = reinterpret_cast<float *>(ws + l.partials);
    p.status = a.status; p.num_pages = a.num_pages; p.max_pages = a.max_pages;
    p.Hq = a.Hq; p.Hkv = a.Hkv; p.keep = a.keep; p.splits = l.splits;
    const float L = static_cast<float>(a.L);
    p.ep = Epilogue{a.s, a.alpha, L, a.beta, 1.0f / logf(L)};
    e = launch_ex(sparse_split_kernel<G>, dim3(l.cluster * l.splits, a.Hkv, a.num_seqs), kRowThreads,
                  kSmem, l.cluster, true, a.stream, map, p);
    if (e != cudaSuccess) return e;
    count_launches(2);
    if (l.splits > 1) {
        const int rows = a.num_seqs * a.Hq;
        e = launch_ex(sparse_merge_kernel, dim3((rows + 15) / 16), 128, 0, 1, true, a.stream, p,
                      rows);
        if (e != cudaSuccess) return e;
        count_launches(1);
    }
    return cudaSuccess;
}

}  // namespace

size_t sparse_workspace_bytes(int num_seqs, int max_pages, int keep, int Hq, int Hkv) {
    return layout(num_seqs, max_pages, keep, Hq, Hkv).total;
}

cudaError_t launch_decode_sparse(const SparseLaunch &a) {
    CUtensorMap map;
    if (!page_pool_map(&map, a.kv_pages, a.num_pages, a.Hkv)) return cudaErrorInvalidValue;
    const Layout l = layout(a.num_seqs, a.max_pages, a.keep, a.Hq, a.Hkv);
    switch (a.Hq / a.Hkv) {
        case 1: return launch_all<1>(a, map, l);
        case 2: return launch_all<2>(a, map, l);
        case 4: return launch_all<4>(a, map, l);
        case 8: return launch_all<8>(a, map, l);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace polar
