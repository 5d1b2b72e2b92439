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

namespace polar {
namespace {

constexpr int kStages = 3;
constexpr int kSmem = kStages * kStageBytes + 1024;  // + alignment slack
constexpr int kScorePages = 64;  // pages per block of the score kernel
constexpr int kSelThreads = 512;

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

// Block (pages, kv head, sequence); eight lanes per page, eight dimensions
// each.  Products of two bf16 are exact in fp32; their sum is formed in 64
// bits and rounded once, so that the order of the pages does not depend on the
// order of the sum.
template <int G>
__global__ void __launch_bounds__(256)
sparse_score_kernel(const __nv_bfloat16 *__restrict__ q, const uint4 *__restrict__ bounds,
                    const int32_t *__restrict__ page_table, const int32_t *__restrict__ seqlens,
                    uint32_t *__restrict__ keys, int num_pages, int max_pages, int Hq, int Hkv,
                    int keep, int *status) {
    const int g = blockIdx.y, seq = blockIdx.z;
    const int len = seqlens[seq];
    if (!valid_len(len, max_pages)) return;  // reported by the selection
    const int npg = (len + kPage - 1) / kPage;
    if (npg <= keep) return;  // every page is read
    const int c = threadIdx.x & 7;
    float qf[G][8];
    const __nv_bfloat16 *qp =
        q + (static_cast<size_t>(seq) * Hq + static_cast<size_t>(g) * G) * kHeadDim + 8 * c;
#pragma unroll
    for (int h = 0; h < G; ++h)
#pragma unroll
        for (int d = 0; d < 8; ++d) qf[h][d] = __bfloat162float(qp[h * kHeadDim + d]);
    const int32_t *pt = page_table + static_cast<size_t>(seq) * max_pages;
    uint32_t *out = keys + (static_cast<size_t>(seq) * Hkv + g) * max_pages;
    const int end = min(npg, (static_cast<int>(blockIdx.x) + 1) * kScorePages);
    for (int p = blockIdx.x * kScorePages + (threadIdx.x >> 3); p < end; p += 32) {
        const int phys = pt[p];
        float best = -INFINITY;
        bool nan = false;
        if (phys >= 0 && phys < num_pages) {  // uniform over the page's eight lanes
            const uint4 *b = bounds + (static_cast<size_t>(phys) * Hkv + g) * 16;
            const uint4 lo4 = __ldg(b + c), hi4 = __ldg(b + 8 + c);
            const uint32_t lw[4] = {lo4.x, lo4.y, lo4.z, lo4.w};
            const uint32_t hw[4] = {hi4.x, hi4.y, hi4.z, hi4.w};
            const uint32_t group = 0xffu << (threadIdx.x & 24);
#pragma unroll
            for (int h = 0; h < G; ++h) {
                double acc = 0.0;
#pragma unroll
                for (int d = 0; d < 8; ++d) {
                    const uint32_t lb = d & 1 ? lw[d >> 1] & 0xffff0000u : lw[d >> 1] << 16;
                    const uint32_t hb = d & 1 ? hw[d >> 1] & 0xffff0000u : hw[d >> 1] << 16;
                    acc += static_cast<double>(
                        fmaxf(qf[h][d] * __uint_as_float(lb), qf[h][d] * __uint_as_float(hb)));
                }
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) acc += __shfl_xor_sync(group, acc, o);
                const float s = static_cast<float>(acc);
                nan |= s != s;
                best = fmaxf(best, s);
            }
        }
        if (c == 0) out[p] = nan ? 0xfffffffeu : score_key(best);
    }
}

struct SelectArgs {
    const uint32_t *keys;
    const int32_t *seqlens;
    int32_t *selected;  // [num_seqs, Hkv, keep]: ascending pages, then -1
    int max_pages, Hkv, keep;
    int *status;
};

// Block (kv head, sequence): the keep highest keys by a radix selection, then
// the pages in ascending order.
__global__ void __launch_bounds__(kSelThreads) sparse_select_kernel(const SelectArgs a) {
    __shared__ int hist[256];
    __shared__ int scratch[2][kSelThreads / 32];
    __shared__ uint32_t s_prefix;
    __shared__ int s_left;
    const int g = blockIdx.x, seq = blockIdx.y, tid = threadIdx.x;
    const int len = a.seqlens[seq];
    if (!valid_len(len, a.max_pages)) {
        if (g == 0 && tid == 0) record_error(a.status, POLAR_ERR_BAD_SEQLEN);
        return;
    }
    const int npg = (len + kPage - 1) / kPage;
    int32_t *out = a.selected + (static_cast<size_t>(seq) * a.Hkv + g) * a.keep;
    if (npg <= a.keep) {
        for (int i = tid; i < a.keep; i += kSelThreads) out[i] = i < npg ? i : -1;
        return;
    }
    const uint32_t *keys = a.keys + (static_cast<size_t>(seq) * a.Hkv + g) * a.max_pages;
    auto key = [&](int p) { return p == npg - 1 ? 0xffffffffu : keys[p]; };

    // The keep-th highest key, byte by byte.
    uint32_t prefix = 0;
    int left = a.keep;  // still to be taken among the keys with this prefix
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        for (int p = tid; p < npg; p += kSelThreads) {
            const uint32_t k = key(p);
            if (shift == 24 || (k >> (shift + 8)) == prefix >> (shift + 8))
                atomicAdd(&hist[k >> shift & 255u], 1);
        }
        __syncthreads();
        if (tid == 0) {
            int b = 255;
            while (left > hist[b]) left -= hist[b--];
            s_prefix = prefix | static_cast<uint32_t>(b) << shift;
            s_left = left;
        }
        __syncthreads();
        prefix = s_prefix;
        left = s_left;
    }

    // Keys above it, and the first `left` equal to it, in ascending order.
    int above = 0, equal = 0;  // in the pages before this step
    const int lane = tid & 31, w = tid >> 5;
    for (int p0 = 0; p0 < npg; p0 += kSelThreads) {
        const int p = p0 + tid;
        const uint32_t k = p < npg ? key(p) : 0u;
        const bool gt = p < npg && k > prefix, eq = p < npg && k == prefix;
        const uint32_t mg = __ballot_sync(0xffffffffu, gt), me = __ballot_sync(0xffffffffu, eq);
        if (lane == 0) {
            scratch[0][w] = __popc(mg);
            scratch[1][w] = __popc(me);
        }
        __syncthreads();
        const uint32_t below = (1u << lane) - 1;
        int ng = above + __popc(mg & below), ne = equal + __popc(me & below);
        for (int i = 0; i < kSelThreads / 32; ++i) {
            if (i < w) {
                ng += scratch[0][i];
                ne += scratch[1][i];
            }
            above += scratch[0][i];
            equal += scratch[1][i];
        }
        if (gt || (eq && ne < left)) out[ng + min(ne, left)] = p;
        __syncthreads();
    }
}

struct SparseArgs {
    const int32_t *page_table, *seqlens, *selected;
    const __nv_bfloat16 *q;
    float *partials;
    int *status;
    int num_pages, max_pages, Hq, Hkv, keep, pages_per_split, max_splits;
    float s, alpha, L;
};

// Positions of the selected pages: all are full but the newest.
__device__ __forceinline__ int selected_tokens(int len, int keep) {
    const int npg = (len + kPage - 1) / kPage;
    return (min(npg, keep) - 1) * kPage + len - (npg - 1) * kPage;
}

// CTA (split of the selected pages, kv head, sequence).
template <int G>
__global__ void __launch_bounds__(128)
sparse_split_kernel(const __grid_constant__ CUtensorMap kv_map, const SparseArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) uint64_t full_bar[kStages];
    __shared__ float mst[4][8][6];
    float(*macc)[8][kHeadDim] = reinterpret_cast<float(*)[8][kHeadDim]>(smem);
    const int split = blockIdx.x, g = blockIdx.y, seq = blockIdx.z;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gq = lane >> 2, tq = lane & 3;

    const int len = a.seqlens[seq];
    if (!valid_len(len, a.max_pages)) return;
    const int npg = (len + kPage - 1) / kPage;
    const int p0 = split * a.pages_per_split, nsel = min(npg, a.keep);
    if (p0 >= nsel) return;
    const int np = min(nsel, p0 + a.pages_per_split) - p0;
    const int32_t *pt = a.page_table + static_cast<size_t>(seq) * a.max_pages;
    const int32_t *sel = a.selected + (static_cast<size_t>(seq) * a.Hkv + g) * a.keep + p0;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&kv_map);
        for (int st = 0; st < kStages; ++st) mbar_init(&full_bar[st], 1);
        fence_barrier_init();
    }
    __syncthreads();
    auto issue = [&](int kk) {
        const int st = kk % kStages, phys = pt[sel[kk]];
        if (phys >= 0 && phys < a.num_pages) {
            mbar_arrive_expect_tx(&full_bar[st], kStageBytes);
            const int row = (phys * 2 * a.Hkv + g) * kPage;  // K block of the kv head
            tma_load_2d(smem + st * kStageBytes, &kv_map, 0, row, &full_bar[st]);
            tma_load_2d(smem + st * kStageBytes + kChunkBytes, &kv_map, 0, row + a.Hkv * kPage,
                        &full_bar[st]);
        } else {
            record_error(a.status, POLAR_ERR_BAD_PAGE);
            mbar_arrive(&full_bar[st]);
        }
    };
    if (threadIdx.x == 0)
        for (int kk = 0; kk < min(kStages, np); ++kk) issue(kk);

    RowTile<1> tile[1];
    tile[0].clear();
    tile[0].load_row(0,
                     gq < G ? a.q + (static_cast<size_t>(seq) * a.Hq + g * G + gq) * kHeadDim
                            : nullptr,
                     tq,
                     a.s * length_temperature(static_cast<float>(selected_tokens(len, a.keep)),
                                              a.alpha, a.L) * kLog2e);
    int issued = min(kStages, np), consumed = 0;
    bool ok = true;
    const uint32_t sbase = smem_u32(smem);
    for (int kk = 0; kk < np; ++kk) {
        const int st = kk % kStages;
        const bool ready = mbar_wait(&full_bar[st], (kk / kStages) & 1, a.status);
        if (!__syncthreads_and(ready)) { ok = false; break; }
        consumed = kk + 1;
        const int page = sel[kk], phys = pt[page];
        if (phys >= 0 && phys < a.num_pages)
            page_step<1, 1>(tile, sbase + st * kStageBytes, sbase + st * kStageBytes + kChunkBytes,
                            w, lane, first_tokens(len - page * kPage));
        __syncthreads();  // every warp is done with stage st
        if (threadIdx.x == 0 && issued < np) issue(issued++);
    }
    if (!ok) {
        // Bounded drain of copies still in flight before shared memory is released.
        if (threadIdx.x == 0)
            for (int kk = consumed; kk < issued; ++kk)
                mbar_wait(&full_bar[kk % kStages], (kk / kStages) & 1, a.status);
        __syncthreads();
        return;
    }
    merge_warps<1, 1>(tile, mst, macc, w, lane, [&](int r) -> float * {
        if (r >= G) return nullptr;
        return a.partials + ((static_cast<size_t>(seq) * a.Hq + g * G + r) * a.max_splits + split) *
                                kPartialFloats;
    });
}

// One warp per (sequence, query head).
__global__ void __launch_bounds__(128)
sparse_merge_kernel(const float *__restrict__ partials, const int32_t *__restrict__ seqlens,
                    const float *__restrict__ u, __nv_bfloat16 *__restrict__ out,
                    float *__restrict__ neff_out, long long rows, int Hq, int max_pages, int keep,
                    int pages_per_split, int max_splits, float s, float alpha, float L, float beta,
                    float inv_ln_L) {
    const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (row >= rows) return;
    const int len = seqlens[row / Hq];
    if (!valid_len(len, max_pages)) return;
    const int nsel = min((len + kPage - 1) / kPage, keep);
    merge_splits(partials + row * max_splits * kPartialFloats,
                 (nsel + pages_per_split - 1) / pages_per_split, selected_tokens(len, keep), s,
                 alpha, L, beta, inv_ln_L, u + (row % Hq) * kHeadDim, threadIdx.x & 31,
                 out + row * kHeadDim, neff_out ? neff_out + row : nullptr);
}

int pages_per_split(int num_seqs, int pages, int Hkv) {
    const long long work = static_cast<long long>(num_seqs) * Hkv * pages;
    int n = 64;
    while (n > 2 && work / n < 148ll * 3 * 4) n >>= 1;
    return n;
}

struct Layout {  // the workspace: keys, selected pages, partials
    size_t selected, partials, total;
    int pps, splits;
};

Layout layout(int num_seqs, int max_pages, int keep, int Hq, int Hkv) {
    Layout l;
    const int pages = std::min(keep, max_pages);
    l.pps = pages_per_split(num_seqs, pages, Hkv);
    l.splits = (pages + l.pps - 1) / l.pps;
    auto pad = [](size_t x) { return (x + 15) / 16 * 16; };
    const size_t heads = static_cast<size_t>(num_seqs) * Hkv;
    l.selected = pad(heads * max_pages * 4);
    l.partials = l.selected + pad(heads * keep * 4);
    l.total = l.partials +
              static_cast<size_t>(num_seqs) * Hq * l.splits * kPartialFloats * sizeof(float);
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
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit);
    }
    char *ws = static_cast<char *>(a.workspace);
    uint32_t *keys = reinterpret_cast<uint32_t *>(ws);
    int32_t *sel = a.selected ? a.selected : reinterpret_cast<int32_t *>(ws + l.selected);
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q);
    if (a.max_pages > a.keep) {
        sparse_score_kernel<G><<<dim3((a.max_pages + kScorePages - 1) / kScorePages, a.Hkv,
                                      a.num_seqs), 256, 0, a.stream>>>(
            q, static_cast<const uint4 *>(a.bounds), a.page_table, a.seqlens, keys, a.num_pages,
            a.max_pages, a.Hq, a.Hkv, a.keep, a.status);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        count_launches(1);
    }
    SelectArgs s{keys, a.seqlens, sel, a.max_pages, a.Hkv, a.keep, a.status};
    sparse_select_kernel<<<dim3(a.Hkv, a.num_seqs), kSelThreads, 0, a.stream>>>(s);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    SparseArgs p;
    p.page_table = a.page_table; p.seqlens = a.seqlens; p.selected = sel; p.q = q;
    p.partials = reinterpret_cast<float *>(ws + l.partials);
    p.status = a.status; p.num_pages = a.num_pages; p.max_pages = a.max_pages;
    p.Hq = a.Hq; p.Hkv = a.Hkv; p.keep = a.keep;
    p.pages_per_split = l.pps; p.max_splits = l.splits;
    p.s = a.s; p.alpha = a.alpha; p.L = static_cast<float>(a.L);
    sparse_split_kernel<G><<<dim3(l.splits, a.Hkv, a.num_seqs), 128, kSmem, a.stream>>>(map, p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const long long rows = static_cast<long long>(a.num_seqs) * a.Hq;
    sparse_merge_kernel<<<static_cast<unsigned>((rows + 3) / 4), 128, 0, a.stream>>>(
        p.partials, a.seqlens, a.u, static_cast<__nv_bfloat16 *>(a.out), a.neff, rows, a.Hq,
        a.max_pages, a.keep, l.pps, l.splits, a.s, a.alpha, p.L, a.beta, 1.0f / logf(p.L));
    count_launches(3);
    return cudaGetLastError();
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
