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
constexpr int kSelThreads = 256;
constexpr int kSelCluster = 8;
constexpr int kFew = 64;  // pages in doubt that are ranked by comparing all
constexpr int kSelKeys = 10240;  // keys that the selection holds in shared memory (40 KB)
constexpr int kScorePages = 512;  // page ids that a block holds
constexpr int kScoreRing = 2;     // pages that a lane has in flight
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
// kThreads, with a bound on each one's error, from which the selection sees where
// 64 bits are needed: sink(page, score, bound) in one thread per page.  phys(p)
// is the pool's page, or -1 (ranks last).  ring: kScoreRing * 4 * kThreads vectors
// of shared memory.
//
// With q = q+ + q-, max(q lo, q hi) is q+ hi + q- lo, so the scores are a product
// of the heads' [q+ q-] with the pages' [hi lo], which a warp forms for eight
// pages by mma.sync (bf16 in, fp32 accumulate); the same of absolute values is
// the sum of the terms' magnitudes.  The order of the 128 terms is free: a lane's
// operands are the 16-byte pieces that it copies itself, a step ahead, so that
// nothing waits for another thread.  (In fp32 on the CUDA cores the scores of 16
// sequences of 1024 to 4096 pages took 30 us, bound by the instructions; this
// 24 us, 42 MB being 6.4 us.)  Products are exact; an instruction adds 16 of them
// and the sum so far, each cut off at 2^-23 of the largest at worst, eight times:
// at most 8 * 17 * 2^-23 of the terms' magnitudes, of which 256 * 2^-23 is taken,
// and 2^-100 for subnormals.
template <int G, int kThreads, typename Phys, typename Sink>
__device__ __forceinline__ void score_pages(const uint4 *__restrict__ q,
                                            const uint4 *__restrict__ bounds, int g, int Hkv,
                                            int count, uint4 *ring, Phys &&phys, Sink &&sink) {
    constexpr int kStep = kThreads / 4;  // pages of a step: eight a warp
    const int tid = threadIdx.x, n = tid & 31, c = n & 3, head = n >> 2;
    uint32_t qp[2][4], qn[2][4];  // the row's positive and negative parts, dims 8 (c + 4 j) ..
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint4 x = head < G ? __ldg(q + head * 8 + c + 4 * j) : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t negative = (w[e] >> 15 & 0x00010001u) * 0xffffu;
            qp[j][e] = w[e] & ~negative;
            qn[j][e] = w[e] & negative;
        }
    }
    const int p0 = tid / 4, steps = (count + kStep - 1) / kStep;
    auto fetch = [&](int step) {
        const int p = p0 + step * kStep, x = p < count ? phys(p) : -1;
        if (x >= 0) {
            const uint4 *b = bounds + (static_cast<size_t>(x) * Hkv + g) * 16 + c;
            uint4 *dst = ring + step % kScoreRing * 4 * kThreads + tid;
#pragma unroll
            for (int e = 0; e < 4; ++e) copy_async16(dst + e * kThreads, b + 4 * e);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int e = 0; e < kScoreRing - 1; ++e) fetch(e);
    for (int step = 0; step < steps; ++step) {  // the same number in every lane: it shuffles
        fetch(step + kScoreRing - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kScoreRing - 1) : "memory");
        __syncwarp();  // lanes without a page or a score to store come back: mma is the warp's
        const uint4 *src = ring + step % kScoreRing * 4 * kThreads + tid;
        float s[4] = {0.f, 0.f, 0.f, 0.f}, m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // lo, lo, hi, hi
            const uint4 x = src[e * kThreads];
            const uint32_t(&a)[4] = e < 2 ? qn[e] : qp[e - 2];
            constexpr uint32_t kAbs = 0x7fff7fffu;
            mma_bf16(s, a[0], 0u, a[1], 0u, x.x, x.y);
            mma_bf16(s, a[2], 0u, a[3], 0u, x.z, x.w);
            mma_bf16(m, a[0] & kAbs, 0u, a[1] & kAbs, 0u, x.x & kAbs, x.y & kAbs);
            mma_bf16(m, a[2] & kAbs, 0u, a[3] & kAbs, 0u, x.z & kAbs, x.w & kAbs);
        }
        // Row `head`, pages 2 c and 2 c + 1 of the warp's eight: the heads' largest.
        // What is not finite makes m so, too: 64 bits then decide.
#pragma unroll
        for (int o = 1; o < G; o <<= 1)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                s[e] = fmaxf(s[e], __shfl_xor_sync(~0u, s[e], 4 * o));
                const uint32_t y = __float_as_uint(m[e]);  // in bit order: a NaN stays
                m[e] = __uint_as_float(max(y, __shfl_xor_sync(~0u, y, 4 * o)));
            }
        if (head == 0) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int p = step * kStep + (tid >> 5) * 8 + 2 * c + e;
                if (p < count) {
                    const bool ok = phys(p) >= 0;
                    sink(p, ok ? s[e] : -INFINITY, ok ? fmaf(m[e], 0x1p-15f, 0x1p-100f) : 0.f);
                }
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

struct SelectArgs {
    const uint4 *q, *bounds;
    const int32_t *page_table, *seqlens;
    int32_t *selected;  // [num_seqs, Hkv, keep]: ascending pages, then -1
    uint32_t *keys;     // per (sequence, head) row of max_pages: past kSelKeys pages
    int num_pages, max_pages, Hkv, keep;
    int *status;
};

// Cluster along x per (kv head, sequence): the pages with the highest scores,
// ascending.  The blocks score a share of the pages each and write the keys to
// the first block's shared memory (past kSelKeys pages: to the workspace), which
// selects.  One launch: a kernel for the scores and one for the selection took
// 25.6 us a call where one sequence has 512 pages and 85 us at 16 sequences of
// 1024 to 4096, this took 22.4 and 83.
//
// A radix selection over keys in the scores' order finds the k-th highest.
// Scores lie close together, so its digits begin at the highest bit in which
// two keys differ, and it ends as soon as a bin is taken whole.  Scores come
// with error bounds; with E the largest of them and T the k-th highest
// score, the k-th highest exact score is within E of T, so a page above T + 2E
// is taken and one below T - 2E is not, whatever the roundings.  Where the pages
// between are not all taken, they get their exact scores, and the selection
// runs once more on (taken, exact, not taken).
template <int G>
__global__ void __launch_bounds__(kSelThreads) sparse_select_kernel(const SelectArgs a) {
    extern __shared__ uint4 score_ring[];  // then the keys
    uint32_t *held = reinterpret_cast<uint32_t *>(score_ring + kScoreRing * 4 * kSelThreads);
    __shared__ int pages[kScorePages];
    __shared__ int hist[256];
    __shared__ uint32_t ends[3][kSelThreads / 32];
    __shared__ int counts[2][kSelThreads / 32];
    __shared__ int s_bin, s_left, s_whole;
    __shared__ uint32_t s_err;
    __shared__ int2 few[kFew];  // page, exact key
    const int g = blockIdx.y, seq = blockIdx.z, tid = threadIdx.x;
    const int lane = tid & 31, w = tid >> 5;
    const int C = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
    constexpr int kWarps = kSelThreads / 32;
    const int len = a.seqlens[seq];
    if (!valid_len(len, a.max_pages)) {
        if (rank == 0 && g == 0 && tid == 0) record_error(a.status, POLAR_ERR_BAD_SEQLEN);
        return;
    }
    const int npg = (len + kPage - 1) / kPage;
    const size_t row = static_cast<size_t>(seq) * a.Hkv + g;
    int32_t *out = a.selected + row * a.keep;
    if (npg <= a.keep) {
        if (rank == 0)
            for (int i = tid; i < a.keep; i += kSelThreads) out[i] = i < npg ? i : -1;
        return;
    }
    if (rank == 0 && tid == 0) out[a.keep - 1] = npg - 1;  // the newest page, without a score
    if (a.keep == 1) return;
    const int n = npg - 1, take = a.keep - 1;
    uint32_t *keys = n <= kSelKeys ? held : a.keys + row * a.max_pages;
    if (tid == 0) s_err = 0;
    if (tid < 256) hist[tid] = 0;
    if (C > 1) cluster_sync(); else __syncthreads();

    // This block's share of the scores.
    uint32_t err = 0;  // as bits: in the order of the values, and a NaN above all
    const uint4 *q = a.q + row * G * 8;
    const int32_t *pt = a.page_table + static_cast<size_t>(seq) * a.max_pages;
    uint32_t *to = n <= kSelKeys ? const_cast<uint32_t *>(cluster_map(held, 0)) : keys;
    const int share = (n + C - 1) / C, last = min(n, (rank + 1) * share);
    for (int first = rank * share; first < last; first += kScorePages) {
        const int count = min(last - first, kScorePages);
        __syncthreads();  // the pages before are done
        for (int p = tid; p < count; p += kSelThreads) {
            const int x = pt[first + p];
            pages[p] = x >= 0 && x < a.num_pages ? x : -1;
        }
        __syncthreads();
        score_pages<G, kSelThreads>(q, a.bounds, g, a.Hkv, count, score_ring,
                                    [&](int p) { return pages[p]; },
                                    [&](int p, float s, float e) {
                                        to[first + p] = score_key(s);
                                        err = max(err, __float_as_uint(e) & 0x7fffffffu);
                                    });
    }
    err = __reduce_max_sync(~0u, err);
    if (lane == 0 && err) atomicMax(const_cast<uint32_t *>(cluster_map(&s_err, 0)), err);
    if (C > 1) cluster_sync(); else __syncthreads();
    if (rank > 0) return;
    err = s_err;

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
    radix();

    // The pages whose place the roundings could change.
    // T: the lowest key that is taken (with a bin taken whole, the lowest in it).
    uint32_t lowest = ~0u;
    for (int p = tid; p < n; p += kSelThreads) {
        const uint32_t k = keys[p];
        if ((k & ~open) >= floor_key) lowest = min(lowest, k);
    }
    lowest = __reduce_min_sync(~0u, lowest);
    if (lane == 0) ends[2][w] = lowest;
    __syncthreads();
    for (int i = 0; i < kWarps; ++i) {
        lowest = min(lowest, ends[2][i]);
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
    if (sure + mid == take) {  // all of `mid` are taken
        floor_key = lowest;
        open = 0;
        left = n;
    } else if (mid <= kFew) {  // the usual case: they are ranked among themselves
        if (tid == 0) s_left = 0;
        __syncthreads();
        for (int p = tid; p < n; p += kSelThreads) {
            const int c = place(keys[p]);
            if (c == 1) few[atomicAdd(&s_left, 1)].x = p;  // in any order
            keys[p] = c == 2 ? 0xffffffffu : 0u;
        }
        __syncthreads();
        for (int i = w; i < mid; i += kWarps) {
            const int phys = pt[few[i].x];
            const bool ok = phys >= 0 && phys < a.num_pages;
            const size_t at = (static_cast<size_t>(ok ? phys : 0) * a.Hkv + g) * 16;
            const uint32_t k = ok ? exact_key<G>(q, a.bounds + at, lane) : 0u;
            if (lane == 0) few[i].y = static_cast<int>(k);
        }
        __syncthreads();
        if (tid < mid) {
            const uint32_t k = few[tid].y;
            int before = 0;
            for (int i = 0; i < mid; ++i) {
                const uint32_t o = few[i].y;
                before += o > k || (o == k && few[i].x < few[tid].x);
            }
            if (before < take - sure) keys[few[tid].x] = 0xffffffffu;
        }
        __syncthreads();
        floor_key = 0xffffffffu;
        open = 0;
        left = n;
    } else {
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

    RowTile<1> tile;
    tile.clear();
    if (w < kRowWarps)
        tile.load_row(0,
                      gq < G ? a.q + (static_cast<size_t>(seq) * a.Hq + g * G + gq) * kHeadDim
                             : nullptr,
                      tq,
                      a.ep.s * length_temperature(static_cast<float>(selected_tokens(len, a.keep)),
                                                  a.ep.alpha, a.ep.L) * kLog2e);
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
                page_step(tile, kb, kb + kChunkBytes, w, lane,
                          p0 + kk == nsel - 1 ? newest : ~0ull);
        });
    }
    let_next_kernel_start();
    reduce_rows(tile, reinterpret_cast<float *>(smem), G, w, lane,
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

constexpr int kRingBytes = kScoreRing * 4 * kSelThreads * 16;

struct Layout {  // the workspace: keys (long rows), selected pages, partials
    size_t selected, partials, total;
    int cluster, splits;  // CTAs of a cluster, clusters of a (sequence, kv head)
};

Layout layout(int num_seqs, int max_pages, int keep, int Hq, int Hkv) {
    Layout l;
    const int pages = std::min(keep, max_pages);
    const long long heads = static_cast<long long>(num_seqs) * Hkv;
    // Enough CTAs for four on each of 148 SMs, of at least two pages each.  Clusters
    // merge what else needs a kernel (1 sequence, 32 pages: 18.7 us, without
    // clusters 20.8; 16 sequences, 256 pages: 86 and 93).
    l.cluster = 1;
    while (l.cluster < kMaxCluster && heads * l.cluster < 148 * 4 && l.cluster * 4 <= pages)
        l.cluster *= 2;
    l.splits = 1;
    while ((heads * l.cluster * l.splits * 2 <= 148 * 4 && l.cluster * l.splits * 16 <= pages) ||
           l.cluster * l.splits * kMaxSteps < pages)
        l.splits *= 2;
    auto pad = [](size_t x) { return (x + 15) / 16 * 16; };
    l.selected = max_pages > kSelKeys ? pad(heads * max_pages * 4) : 0;
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
        e = cudaFuncSetAttribute(sparse_split_kernel<G>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(sparse_select_kernel<G>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kRingBytes + kSelKeys * sizeof(uint32_t));
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit);
    }
    char *ws = static_cast<char *>(a.workspace);
    int32_t *sel = a.selected ? a.selected : reinterpret_cast<int32_t *>(ws + l.selected);
    const uint4 *q = static_cast<const uint4 *>(a.q);
    const uint4 *bounds = static_cast<const uint4 *>(a.bounds);
    SelectArgs s{q, bounds, a.page_table, a.seqlens, sel, reinterpret_cast<uint32_t *>(ws),
                 a.num_pages, a.max_pages, a.Hkv, a.keep, a.status};
    // Blocks of a row, with two steps of the scores each (one block a row: 512 pages
    // 10.6 us, 4 blocks 7.9; 16 sequences of 1024 to 4096 pages 66 us, 8 blocks 35).
    const int step = kSelThreads / 4;
    int blocks = 1;
    while (blocks < kSelCluster && blocks * step * 2 < a.max_pages && a.max_pages > a.keep)
        blocks *= 2;
    const size_t held = std::min(a.max_pages, kSelKeys) * sizeof(uint32_t);
    e = launch_ex(sparse_select_kernel<G>, dim3(blocks, a.Hkv, a.num_seqs), kSelThreads,
                  kRingBytes + held, blocks, false, a.stream, s);
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
    e = launch_ex(sparse_split_kernel<G>, dim3(l.cluster * l.splits, a.Hkv, a.num_seqs),
                  kRowThreads, kSmem, l.cluster, true, a.stream, map, p);
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
