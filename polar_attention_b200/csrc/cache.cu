// cache.cu -- the paged KV cache's own operations: growth with copy on write,
// appending tokens with their pages' key bounds, forking and freeing rows, and
// moving live pages together.  All state (tables, lengths, reference counts)
// stays on the device.
#include <algorithm>

#include "launch.cuh"
#include "polar_common.cuh"
#include "polar_internal.h"

namespace polar {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kRowVecs = kHeadDim / 8;  // 16-byte vectors of one key or value row

__device__ __forceinline__ int pages_of(int len) { return (len + kPage - 1) / kPage; }

// Inclusive sum over the block's threads; `scratch` holds one value per warp.
// Returns this thread's inclusive prefix; *total gets the block's sum.
template <typename T>
__device__ __forceinline__ T block_scan(T x, T *scratch, T *total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // scratch may still be read from the call before
    if (lane == 31) scratch[w] = x;
    __syncthreads();
    T before = 0, sum = 0;
    for (int i = 0; i < nw; ++i) {
        const T s = scratch[i];
        before += i < w ? s : 0;
        sum += s;
    }
    *total = sum;
    return x + before;
}

// ------------------------------------------------------------------ grow ---

constexpr int kPlanRows = 1024;   // rows whose plan is held in shared memory
constexpr int kPlanFresh = 2048;  // and new pages
constexpr int kFusedRows = 128;   // rows up to which one cluster plans and copies
constexpr int kFusedCluster = 8;

struct ReserveArgs {
    int32_t *refs, *table, *lens, *granted;
    const int32_t *grow;
    uint4 *kv, *bounds;
    int num_pages, max_pages, num_seqs, Hkv;
    // Workspace: per page the last growing row that writes it and how many do;
    // the free pages found, in order, used past kPlanFresh; per row the running
    // sum of pages taken and the page that it copies (-1: none), used past
    // kPlanRows; the copies.
    int *owner, *sharers, *fresh, *end, *copy;
    int3 *copies;    // source page, its copy, rows
    int *num_copies;
    int *status;
};

// Plan of a growth step, by a block's threads.  Which rows copy their last page;
// how many pages each row takes (a running sum over the rows); the lowest free
// ids (a running count over the reference counts that stops once there are
// enough); then every taken page finds its row by a search in the running sums.
// What bounds it is the chain of dependent loads, so the first stretch of
// reference counts is on its way before the rows are looked at, rows and new
// pages are held in shared memory, and the passes over shared pages run only
// where a last page is shared.  copies/num_copies get the copies (num_copies is
// in shared memory), in any order.
__device__ __forceinline__ void reserve_plan(const ReserveArgs &a, int3 *copies, int *num_copies) {
    __shared__ int scratch[kPlanThreads / 32];
    __shared__ long long wide[kPlanThreads / 32];
    __shared__ int s_end[kPlanRows], s_copy[kPlanRows], s_len[kPlanRows], s_fresh[kPlanFresh];
    const int tid = threadIdx.x, N = a.num_seqs;
    int *const end_of = N <= kPlanRows ? s_end : a.end;
    int *const copy_of = N <= kPlanRows ? s_copy : a.copy;
    if (tid == 0) *num_copies = 0;

    constexpr int kPer = 16;
    int r[kPer];
    auto fetch = [&](int p) {  // reference counts of pages p .. p + 15; past the pool: taken
        const bool whole = p + kPer <= a.num_pages &&
                           (reinterpret_cast<uintptr_t>(a.refs) & 15u) == 0;
#pragma unroll
        for (int e = 0; e < kPer; e += 4) {
            int4 x = make_int4(1, 1, 1, 1);
            if (whole) {
                x = *reinterpret_cast<const int4 *>(a.refs + p + e);
            } else {
                if (p + e < a.num_pages) x.x = a.refs[p + e];
                if (p + e + 1 < a.num_pages) x.y = a.refs[p + e + 1];
                if (p + e + 2 < a.num_pages) x.z = a.refs[p + e + 2];
                if (p + e + 3 < a.num_pages) x.w = a.refs[p + e + 3];
            }
            r[e] = x.x; r[e + 1] = x.y; r[e + 2] = x.z; r[e + 3] = x.w;
        }
    };
    fetch(tid * kPer);

    // A row before it grows: its length, its growth and, where it has a partly
    // filled last page to write, that page and its references.
    struct Row {
        int len, g, page, refs, bad;
    };
    auto row = [&](int i) {
        Row x{a.lens[i], a.grow[i], -1, 0, 0};
        const long long cap = static_cast<long long>(a.max_pages) * kPage;
        if (x.len < 0 || x.len > cap || x.g < 0 || x.len + static_cast<long long>(x.g) > cap) {
            x.bad = POLAR_ERR_BAD_SEQLEN;
        } else if (x.g > 0 && x.len % kPage != 0) {
            x.page = a.table[static_cast<size_t>(i) * a.max_pages + x.len / kPage];
            if (x.page < 0 || x.page >= a.num_pages) {
                x.bad = POLAR_ERR_BAD_PAGE;
                x.page = -1;
            } else {
                x.refs = a.refs[x.page];
            }
        }
        return x;
    };
    Row mine{0, 0, -1, 0, 0};  // row tid: all that is needed up to kPlanThreads rows
    if (tid < N) mine = row(tid);
    bool shared = mine.refs > 1;
    for (int i = tid + kPlanThreads; i < N; i += kPlanThreads) shared |= row(i).refs > 1;
    if (__syncthreads_or(shared)) {
        for (int i = tid; i < N; i += kPlanThreads) {
            const Row x = i == tid ? mine : row(i);
            if (x.refs > 1) {
                a.owner[x.page] = -1;
                a.sharers[x.page] = 0;
            }
        }
        __syncthreads();
        for (int i = tid; i < N; i += kPlanThreads) {
            const Row x = i == tid ? mine : row(i);
            if (x.refs > 1) {
                atomicMax(&a.owner[x.page], i);
                atomicAdd(&a.sharers[x.page], 1);
            }
        }
        __syncthreads();
    }

    // Sums in 64 bits: many rows may ask for far more than the pool has.
    long long asked = 0;
    for (int i0 = 0; i0 < N; i0 += kPlanThreads) {
        const int i = i0 + tid;
        long long need = 0;
        int copy = -1;
        if (i < N) {
            const Row x = i0 == 0 ? mine : row(i);
            if (x.bad) {
                record_error(a.status, x.bad);
            } else {
                need = pages_of(x.len + x.g) - pages_of(x.len);
                if (x.refs > 1 &&
                    !(__ldcg(&a.sharers[x.page]) == x.refs && __ldcg(&a.owner[x.page]) == i)) {
                    copy = x.page;
                    ++need;
                }
            }
        }
        long long total;
        const long long end = asked + block_scan(need, wide, &total);
        asked += total;
        if (i < N) {
            end_of[i] = static_cast<int>(min(end, 0x7fffffffll));
            copy_of[i] = copy;
            if (N <= kPlanRows) s_len[i] = mine.len;
        }
    }

    const int wanted = static_cast<int>(min(asked, 0x7ffffffell));
    int *const fresh = wanted <= kPlanFresh ? s_fresh : a.fresh;
    int found = 0;
    for (int p0 = 0; p0 < a.num_pages && found < wanted; p0 += kPlanThreads * kPer) {
        const int p = p0 + tid * kPer;
        if (p0 > 0) fetch(p);
        int free = 0;
#pragma unroll
        for (int e = 0; e < kPer; ++e) free += r[e] == 0;
        int total;
        int at = found + block_scan(free, scratch, &total) - free;
#pragma unroll
        for (int e = 0; e < kPer; ++e)
            if (r[e] == 0) {
                if (at < wanted) fresh[at] = p + e;
                ++at;
            }
        found += total;
    }
    __syncthreads();

    // Each taken page, by its place in the running sums: its row is the first
    // whose sum is past it; the row's copy comes before its new pages.  Rows
    // are served up to the first whose sum is past the pages found.
    for (int k = tid; k < min(found, wanted); k += kPlanThreads) {
        int lo = 0, hi = N - 1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (end_of[mid] > k) hi = mid; else lo = mid + 1;
        }
        if (end_of[lo] > found) break;  // not served, nor any page after
        const int j = k - (lo > 0 ? end_of[lo - 1] : 0), copy = copy_of[lo], id = fresh[k];
        const int len = N <= kPlanRows ? s_len[lo] : a.lens[lo];
        const bool is_copy = copy >= 0 && j == 0;
        const int c = is_copy ? len / kPage : pages_of(len) + j - (copy >= 0);
        a.table[static_cast<size_t>(lo) * a.max_pages + c] = id;
        a.refs[id] = 1;
        if (is_copy) {
            atomicSub(&a.refs[copy], 1);
            copies[atomicAdd(num_copies, 1)] = make_int3(copy, id, len % kPage);
        }
    }
    __syncthreads();  // the lengths above are the old ones
    for (int i = tid; i < N; i += kPlanThreads) {
        const int len = i == tid ? mine.len : a.lens[i], g = i == tid ? mine.g : a.grow[i];
        const int bad = i == tid ? mine.bad : row(i).bad;
        const bool served = !bad && end_of[i] <= found;
        if (!served && !bad && g > 0) record_error(a.status, POLAR_ERR_NO_PAGES);
        a.granted[i] = served ? g : 0;
        if (served) a.lens[i] = len + g;
    }
}

// One 8 KB block (K|V and head) of a copied page, by a warp: its valid rows, and
// its share of the page's bounds.
__device__ __forceinline__ void copy_block(uint4 *kv, uint4 *bounds, int3 c, int blk, int Hkv,
                                           int lane) {
    const size_t step = static_cast<size_t>(2) * Hkv;
    const size_t src = c.x * step + blk, dst = c.y * step + blk;
    const uint4 *from = kv + src * (kPage * kRowVecs);
    uint4 *to = kv + dst * (kPage * kRowVecs);
    const int vecs = c.z * kRowVecs;
    for (int e0 = lane; e0 < vecs; e0 += 32 * 8) {
        uint4 x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (e0 + 32 * k < vecs) x[k] = from[e0 + 32 * k];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (e0 + 32 * k < vecs) to[e0 + 32 * k] = x[k];
    }
    if (bounds && lane < kRowVecs)
        bounds[dst * kRowVecs + lane] = bounds[src * kRowVecs + lane];
}

// A growth step of few rows: one cluster, whose first block plans and hands the
// copies to all.  One launch instead of two, since a loop of such calls spends its
// time on the launches (append step of 64 rows: 43 us, with two kernels 46).  On
// the GPU the two kernels are the faster ones, the more so the more rows copy.
// Replayed from a graph, two kernels and this, for 1, 16, 64 and 128 rows: without
// copies 5.2, 4.7, 4.6, 4.9 us and 5.1, 5.5, 5.2, 5.2; where every row copies its
// tail 10.2, 10.4, 10.2, 10.6 and 10.9, 12.6, 15.5, 21.8.
__global__ void __launch_bounds__(kPlanThreads)
cache_reserve_fused_kernel(const ReserveArgs a) {
    __shared__ int3 copies[kFusedRows];
    __shared__ int num_copies;
    const int rank = static_cast<int>(cluster_rank());
    if (rank == 0) reserve_plan(a, copies, &num_copies);
    cluster_sync();
    const int n = *cluster_map(&num_copies, 0), per = 2 * a.Hkv;
    const int3 *list = cluster_map(copies, 0);
    for (int u = rank * (kPlanThreads / 32) + (threadIdx.x >> 5); u < n * per;
         u += kFusedCluster * (kPlanThreads / 32))
        copy_block(a.kv, a.bounds, list[u / per], u % per, a.Hkv, threadIdx.x & 31);
    cluster_sync();  // the first block stays while its list is read
}

__global__ void __launch_bounds__(kPlanThreads) cache_reserve_plan_kernel(const ReserveArgs a) {
    __shared__ int num_copies;
    reserve_plan(a, a.copies, &num_copies);
    __syncthreads();
    if (threadIdx.x == 0) *a.num_copies = num_copies;
}

__global__ void __launch_bounds__(128) cache_reserve_copy_kernel(const ReserveArgs a) {
    wait_for_previous_kernel();
    const int n = *a.num_copies, per = 2 * a.Hkv;
    for (int u = blockIdx.x * 4 + (threadIdx.x >> 5); u < n * per; u += gridDim.x * 4)
        copy_block(a.kv, a.bounds, a.copies[u / per], u % per, a.Hkv, threadIdx.x & 31);
}

// ---------------------------------------------------------------- append ---

struct AppendArgs {
    const uint4 *k, *v;
    uint4 *kv, *bounds;
    const int32_t *refs, *pick, *counts, *table, *lens;
    int src_tokens, tokens, num_pages, max_pages, Hkv;
    int *status;
};

__device__ __forceinline__ uint32_t bmin2(uint32_t a, uint32_t b) {
    __nv_bfloat162 r = __hmin2_nan(reinterpret_cast<__nv_bfloat162 &>(a),
                                   reinterpret_cast<__nv_bfloat162 &>(b));
    return reinterpret_cast<uint32_t &>(r);
}
__device__ __forceinline__ uint32_t bmax2(uint32_t a, uint32_t b) {
    __nv_bfloat162 r = __hmax2_nan(reinterpret_cast<__nv_bfloat162 &>(a),
                                   reinterpret_cast<__nv_bfloat162 &>(b));
    return reinterpret_cast<uint32_t &>(r);
}
__device__ __forceinline__ uint4 bmin8(uint4 a, uint4 b) {
    return make_uint4(bmin2(a.x, b.x), bmin2(a.y, b.y), bmin2(a.z, b.z), bmin2(a.w, b.w));
}
__device__ __forceinline__ uint4 bmax8(uint4 a, uint4 b) {
    return make_uint4(bmax2(a.x, b.x), bmax2(a.y, b.y), bmax2(a.z, b.z), bmax2(a.w, b.w));
}
__device__ __forceinline__ uint4 shfl8(uint4 a, int o) {
    return make_uint4(__shfl_xor_sync(0xffffffffu, a.x, o), __shfl_xor_sync(0xffffffffu, a.y, o),
                      __shfl_xor_sync(0xffffffffu, a.z, o), __shfl_xor_sync(0xffffffffu, a.w, o));
}

// Block (touched page of the row and kv head, row): thread (row r0 of 16, vector
// c of 8) moves rows r0, r0 + 16, ... of the page.  The heads of a page are
// neighbours, since a token's rows of all heads lie together in k and v.  Rows
// before the first new token are read back where the bounds need them.  Bound by
// memory: 405 MB in 71 us (5.7 TB/s), the rows read and written once and so kept
// out of the caches' way (plain loads and stores: 73.2 us; without the bound on
// registers, 8 or 16 blocks an SM: 73.6, 77 and 74.5).
__global__ void __launch_bounds__(128, 12) cache_append_kernel(const AppendArgs a) {
    __shared__ uint4 part[2][4][kRowVecs];
    const int i = blockIdx.y, g = blockIdx.x % a.Hkv, touched = blockIdx.x / a.Hkv;
    const int len = a.lens[i], cnt = a.counts ? a.counts[i] : a.tokens;
    if (cnt < 0 || cnt > a.tokens || len < cnt ||
        len > static_cast<long long>(a.max_pages) * kPage) {
        if (blockIdx.x == 0 && threadIdx.x == 0) record_error(a.status, POLAR_ERR_BAD_SEQLEN);
        return;
    }
    const int first = len - cnt;  // position of the first new token
    const int lp = first / kPage + touched;
    if (cnt == 0 || lp >= pages_of(len)) return;
    const int page = a.table[static_cast<size_t>(i) * a.max_pages + lp];
    if (page < 0 || page >= a.num_pages || (a.refs && a.refs[page] != 1)) {
        if (g == 0 && threadIdx.x == 0) record_error(a.status, POLAR_ERR_BAD_PAGE);
        return;
    }
    const int lo = max(first - lp * kPage, 0), hi = min(len - lp * kPage, kPage);
    const int c = threadIdx.x & 7, r0 = threadIdx.x >> 3;
    uint4 *kp = a.kv + (static_cast<size_t>(page) * 2 * a.Hkv + g) * (kPage * kRowVecs);
    uint4 *vp = kp + static_cast<size_t>(a.Hkv) * (kPage * kRowVecs);

    uint4 kx[4], vx[4];
    bool write[4], have[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int r = r0 + 16 * e;
        write[e] = r >= lo && r < hi;
        have[e] = r < hi && (write[e] || a.bounds != nullptr);
        kx[e] = vx[e] = make_uint4(0, 0, 0, 0);
        if (write[e]) {
            const int t = lp * kPage + r - first;
            const int from = a.pick ? a.pick[static_cast<size_t>(i) * a.tokens + t] : t;
            if (from < 0 || from >= a.src_tokens) {
                record_error(a.status, POLAR_ERR_BAD_SLOT);
                write[e] = false;  // the row stays as it is, and its key counts as it is
            } else {
                const size_t at =
                    ((static_cast<size_t>(i) * a.src_tokens + from) * a.Hkv + g) * kRowVecs + c;
                kx[e] = __ldcs(a.k + at);
                vx[e] = __ldcs(a.v + at);
            }
        }
        if (have[e] && !write[e] && a.bounds) kx[e] = kp[r * kRowVecs + c];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (write[e]) {
            __stcs(kp + (r0 + 16 * e) * kRowVecs + c, kx[e]);
            __stcs(vp + (r0 + 16 * e) * kRowVecs + c, vx[e]);
        }
    if (!a.bounds) return;
    const uint32_t inf = 0x7f807f80u, ninf = 0xff80ff80u;
    uint4 mn = make_uint4(inf, inf, inf, inf), mx = make_uint4(ninf, ninf, ninf, ninf);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (have[e]) {
            mn = bmin8(mn, kx[e]);
            mx = bmax8(mx, kx[e]);
        }
#pragma unroll
    for (int o = 8; o <= 16; o <<= 1) {  // the warp's four rows of each vector
        mn = bmin8(mn, shfl8(mn, o));
        mx = bmax8(mx, shfl8(mx, o));
    }
    const int w = threadIdx.x >> 5;
    if ((threadIdx.x & 31) < kRowVecs) {
        part[0][w][c] = mn;
        part[1][w][c] = mx;
    }
    __syncthreads();
    if (threadIdx.x < 2 * kRowVecs) {
        const int which = threadIdx.x >> 3;
        uint4 x = part[which][0][c];
#pragma unroll
        for (int k = 1; k < 4; ++k)
            x = which ? bmax8(x, part[1][k][c]) : bmin8(x, part[0][k][c]);
        a.bounds[(static_cast<size_t>(page) * a.Hkv + g) * 2 * kRowVecs + threadIdx.x] = x;
    }
}

// ----------------------------------------------------------- fork, free ---

__global__ void __launch_bounds__(256)
cache_fork_kernel(int32_t *__restrict__ refs, int num_pages,
                  const int32_t *__restrict__ src_table, const int32_t *__restrict__ src_lens,
                  int num_src, const int32_t *__restrict__ src_rows,
                  int32_t *__restrict__ dst_table, int32_t *__restrict__ dst_lens, int max_pages,
                  int *status) {
    const int i = blockIdx.y;
    const bool says = blockIdx.x == 0 && threadIdx.x == 0;
    const int src = src_rows[i];
    if (src < 0) return;
    if (src >= num_src) {
        if (says) record_error(status, POLAR_ERR_BAD_SLOT);
        return;
    }
    const int len = src_lens[src];
    if (len < 0 || len > static_cast<long long>(max_pages) * kPage) {
        if (says) record_error(status, POLAR_ERR_BAD_SEQLEN);
        return;
    }
    if (says) dst_lens[i] = len;
    const int n = pages_of(len);
    for (int c = blockIdx.x * 256 + threadIdx.x; c < n; c += gridDim.x * 256) {
        const int p = src_table[static_cast<size_t>(src) * max_pages + c];
        dst_table[static_cast<size_t>(i) * max_pages + c] = p;
        if (p >= 0 && p < num_pages)
            atomicAdd(&refs[p], 1);
        else
            record_error(status, POLAR_ERR_BAD_PAGE);
    }
}

// One block per row, so that the row's length is read by all its threads
// before it changes.
__global__ void __launch_bounds__(256)
cache_free_kernel(int32_t *__restrict__ refs, int num_pages, int32_t *__restrict__ table,
                  int max_pages, int32_t *__restrict__ lens, const int32_t *__restrict__ keep,
                  int *status) {
    const int i = blockIdx.x;
    const int len = lens[i], kept = keep ? keep[i] : 0;
    __syncthreads();
    if (len < 0 || len > static_cast<long long>(max_pages) * kPage) {
        if (threadIdx.x == 0) record_error(status, POLAR_ERR_BAD_SEQLEN);
        return;
    }
    if (kept < 0 || kept >= len) return;
    if (threadIdx.x == 0) lens[i] = kept;
    int32_t *pt = table + static_cast<size_t>(i) * max_pages;
    for (int c = pages_of(kept) + threadIdx.x; c < pages_of(len); c += 256) {
        const int p = pt[c];
        pt[c] = -1;
        if (p < 0 || p >= num_pages) {
            record_error(status, POLAR_ERR_BAD_PAGE);
        } else if (atomicSub(&refs[p], 1) <= 0) {
            atomicAdd(&refs[p], 1);
            record_error(status, POLAR_ERR_BAD_PAGE);
        }
    }
}

// --------------------------------------------------------------- compact ---

constexpr int kCompactCluster = 8;

struct CompactArgs {
    int32_t *refs, *table, *used;
    const int32_t *lens;
    uint4 *kv, *bounds;
    int num_pages, max_pages, num_seqs, Hkv;
    // Workspace: [0] pages that move; per page its rank among the movers (-1:
    // free, -2: stays); the movers and their places, by rank.
    int *head, *rank, *src, *dst;
    int *status;
};

// With n live pages and L(x) live pages below id x: a live page p >= n is the
// (L(p) - L(n))-th mover, a free id p < n the (p - L(p))-th place.  One cluster;
// each block counts its stretch of the pool, the blocks exchange their counts,
// and each writes the ranks of its stretch.
__global__ void __launch_bounds__(kPlanThreads) cache_compact_plan_kernel(const CompactArgs a) {
    __shared__ int scratch[kPlanThreads / 32];
    __shared__ int counts[2];  // live pages of this block's stretch; of them, those below n
    constexpr int kPer = 8;
    const int tid = threadIdx.x, block = static_cast<int>(cluster_rank());
    const int stretch = ((a.num_pages + kCompactCluster - 1) / kCompactCluster + 3) / 4 * 4;
    const int lo = min(block * stretch, a.num_pages), hi = min(lo + stretch, a.num_pages);
    auto live_in = [&](int from, int to) {
        int mine = 0, total;
        for (int p = from + tid; p < to; p += kPlanThreads) mine += a.refs[p] > 0;
        block_scan(mine, scratch, &total);
        return total;
    };
    const int own = live_in(lo, hi);
    if (tid == 0) counts[0] = own;
    cluster_sync();
    int n = 0, upto = 0;  // upto: L at the place that is next
    for (int b = 0; b < kCompactCluster; ++b) {
        const int x = cluster_map(counts, b)[0];
        n += x;
        upto += b < block ? x : 0;
    }
    const int below = n >= hi ? own : n <= lo ? 0 : live_in(lo, n);
    if (tid == 0) counts[1] = below;
    cluster_sync();
    int live_below = 0;  // L(n)
    for (int b = 0; b < kCompactCluster; ++b) live_below += cluster_map(counts, b)[1];

    for (int q0 = lo; q0 < hi; q0 += kPlanThreads * kPer) {
        const int p0 = q0 + tid * kPer;
        bool live[kPer];
        int count = 0, total;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            live[e] = p0 + e < hi && a.refs[p0 + e] > 0;
            count += live[e];
        }
        int at = upto + block_scan(count, scratch, &total) - count;  // L(p0)
        upto += total;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int p = p0 + e;
            if (p < hi) {
                if (p < n) {
                    a.rank[p] = live[e] ? -2 : -1;
                    if (!live[e]) a.dst[p - at] = p;
                } else {
                    a.rank[p] = live[e] ? at - live_below : -1;
                    if (live[e]) a.src[at - live_below] = p;
                }
            }
            at += live[e];
        }
    }
    if (block == 0 && tid == 0) {
        a.head[0] = n - live_below;
        a.used[0] = n;
    }
    cluster_sync();  // no block leaves while its counts are read
}

// Copies the movers' pages, laid end to end, 32 KB at a time (eight vectors a
// thread in flight), then rewrites references and tables.  Bound by memory: 1.07 GB
// moved and read in 168 us (6.4 TB/s).  Many short blocks: 8 an SM that loop took
// 178 us, 32 an SM 171, 256 an SM 172.
__global__ void __launch_bounds__(256) cache_compact_move_kernel(const CompactArgs a) {
    wait_for_previous_kernel();
    const int moves = a.head[0];
    const int units = moves * a.Hkv;  // of 16 KB: Hkv of them a page
    for (int u0 = 2 * blockIdx.x; u0 < units; u0 += 2 * gridDim.x) {
        uint4 x[2][4];
        size_t to[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int u = min(u0 + h, units - 1), k = u / a.Hkv, at = u % a.Hkv;
            const uint4 *from = a.kv + (static_cast<size_t>(a.src[k]) * a.Hkv + at) * 1024;
            to[h] = (static_cast<size_t>(a.dst[k]) * a.Hkv + at) * 1024 + threadIdx.x;
#pragma unroll
            for (int e = 0; e < 4; ++e) x[h][e] = __ldcs(from + 256 * e + threadIdx.x);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (u0 + h < units)
#pragma unroll
                for (int e = 0; e < 4; ++e) __stcs(a.kv + to[h] + 256 * e, x[h][e]);
    }
    const int per = 2 * a.Hkv * kRowVecs;  // vectors of a page's bounds
    for (long long u = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
         u < static_cast<long long>(moves) * per; u += static_cast<long long>(gridDim.x) * 256) {
        const int k = static_cast<int>(u / per), e = static_cast<int>(u % per);
        if (a.bounds)
            a.bounds[static_cast<size_t>(a.dst[k]) * per + e] =
                a.bounds[static_cast<size_t>(a.src[k]) * per + e];
        if (e == 0) {
            a.refs[a.dst[k]] = a.refs[a.src[k]];
            a.refs[a.src[k]] = 0;
        }
    }
    const long long entries = static_cast<long long>(a.num_seqs) * a.max_pages;
    for (long long e = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; e < entries;
         e += static_cast<long long>(gridDim.x) * 256) {
        const int i = static_cast<int>(e / a.max_pages), c = static_cast<int>(e % a.max_pages);
        const int len = a.lens[i];
        if (len < 0 || len > static_cast<long long>(a.max_pages) * kPage) {
            if (c == 0) record_error(a.status, POLAR_ERR_BAD_SEQLEN);
            continue;
        }
        if (c >= pages_of(len)) continue;
        const int p = a.table[e];
        const int r = p >= 0 && p < a.num_pages ? a.rank[p] : -1;
        if (r == -1)
            record_error(a.status, POLAR_ERR_BAD_PAGE);
        else if (r >= 0)
            a.table[e] = a.dst[r];
    }
}

}  // namespace

size_t cache_workspace_bytes(int num_pages, int num_seqs) {
    // Three ints a page (reserve: owner, sharers, fresh; compact: rank, src,
    // dst), five a row, and one more.
    return (3 * static_cast<size_t>(num_pages) + 5 * static_cast<size_t>(num_seqs) + 4) *
           sizeof(int);
}

cudaError_t launch_cache_reserve(const CacheLaunch &a, const int32_t *grow, int32_t *granted) {
    int *ws = static_cast<int *>(a.workspace);
    ReserveArgs r;
    r.refs = a.refs; r.table = a.table; r.lens = a.lens; r.grow = grow; r.granted = granted;
    r.num_pages = a.num_pages; r.max_pages = a.max_pages; r.num_seqs = a.num_seqs;
    r.owner = ws; r.sharers = ws + a.num_pages; r.fresh = ws + 2 * static_cast<size_t>(a.num_pages);
    const size_t n = a.num_seqs;
    int *rows = ws + 3 * static_cast<size_t>(a.num_pages);
    r.end = rows; r.copy = rows + n;
    r.copies = reinterpret_cast<int3 *>(rows + 2 * n);
    r.num_copies = rows + 5 * n;
    r.kv = static_cast<uint4 *>(a.kv); r.bounds = static_cast<uint4 *>(a.bounds); r.Hkv = a.Hkv;
    r.status = a.status;
    if (a.num_seqs <= kFusedRows) {
        count_launches(1);
        return launch_ex(cache_reserve_fused_kernel, dim3(kFusedCluster), kPlanThreads, 0,
                         kFusedCluster, false, a.stream, r);
    }
    cache_reserve_plan_kernel<<<1, kPlanThreads, 0, a.stream>>>(r);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    count_launches(2);
    return launch_ex(cache_reserve_copy_kernel, dim3(std::min(a.num_seqs, 148 * 8)), 128, 0, 1,
                     true, a.stream, r);
}

cudaError_t launch_cache_append(const CacheLaunch &a, const void *k, const void *v, int src_tokens,
                                const int32_t *pick, int tokens, const int32_t *counts) {
    AppendArgs p;
    p.k = static_cast<const uint4 *>(k); p.v = static_cast<const uint4 *>(v);
    p.kv = static_cast<uint4 *>(a.kv); p.bounds = static_cast<uint4 *>(a.bounds);
    p.refs = a.refs; p.pick = pick; p.counts = counts; p.table = a.table; p.lens = a.lens;
    p.src_tokens = src_tokens; p.tokens = tokens; p.num_pages = a.num_pages;
    p.max_pages = a.max_pages; p.Hkv = a.Hkv; p.status = a.status;
    // Pages that `tokens` new tokens can touch, from any offset in a page.
    const long long touched =
        std::min<long long>(a.max_pages, (tokens - 1ll + kPage - 1) / kPage + 1);
    if (touched * a.Hkv > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    count_launches(1);
    return launch_ex(cache_append_kernel, dim3(static_cast<unsigned>(touched * a.Hkv), a.num_seqs),
                     128, 0, 1, false, a.stream, p);
}

cudaError_t launch_cache_fork(const CacheLaunch &a, const int32_t *src_table,
                              const int32_t *src_lens, int num_src, const int32_t *src_rows) {
    const int blocks = std::min((a.max_pages + 255) / 256, 64);
    count_launches(1);
    return launch_ex(cache_fork_kernel, dim3(blocks, a.num_seqs), 256, 0, 1, false, a.stream,
                     a.refs, a.num_pages, src_table, src_lens, num_src, src_rows, a.table, a.lens,
                     a.max_pages, a.status);
}

cudaError_t launch_cache_free(const CacheLaunch &a, const int32_t *keep) {
    count_launches(1);
    return launch_ex(cache_free_kernel, dim3(a.num_seqs), 256, 0, 1, false, a.stream, a.refs,
                     a.num_pages, a.table, a.max_pages, a.lens, keep, a.status);
}

cudaError_t launch_cache_compact(const CacheLaunch &a, int32_t *used) {
    int *ws = static_cast<int *>(a.workspace);
    CompactArgs c;
    c.refs = a.refs; c.table = a.table; c.lens = a.lens; c.used = used;
    c.kv = static_cast<uint4 *>(a.kv); c.bounds = static_cast<uint4 *>(a.bounds);
    c.num_pages = a.num_pages; c.max_pages = a.max_pages; c.num_seqs = a.num_seqs; c.Hkv = a.Hkv;
    c.rank = ws; c.src = ws + a.num_pages; c.dst = ws + 2 * static_cast<size_t>(a.num_pages);
    c.head = ws + 3 * static_cast<size_t>(a.num_pages);
    c.status = a.status;
    cudaError_t e = launch_ex(cache_compact_plan_kernel, dim3(kCompactCluster), kPlanThreads, 0,
                              kCompactCluster, false, a.stream, c);
    if (e != cudaSuccess) return e;
    count_launches(2);
    // At most half of the pages move.
    const int blocks = static_cast<int>(
        std::min<long long>(148 * 64, static_cast<long long>(a.num_pages) * a.Hkv / 4 + 1));
    return launch_ex(cache_compact_move_kernel, dim3(blocks), 256, 0, 1, true, a.stream, c);
}

}  // namespace polar
