// decode_tree.cu -- Polar Attention for a tree of drafted tokens over the
// paged cache.
//
// Node t of a sequence sees every cached position and the drafted nodes whose
// bits its mask has; the drafted keys and values come as dense rows, so that a
// rejected node never touches the cache.  A row is a (node, query head of the
// kv group) pair; rows that share a kv head share its page reads.  The work of
// a sequence is its cached pages and, behind them, one step for the drafted
// rows (at most 64, laid out like a page); splits of it go to CTAs of their
// own, and a second kernel merges their states exactly.
#include <algorithm>
#include <atomic>

#include "decode_rows.cuh"
#include "polar_internal.h"
#include "tc_common.cuh"

namespace polar {
namespace {

constexpr int kStages = 3;
constexpr int kSmem = kStages * kStageBytes + 1024;  // + alignment slack

struct TreeArgs {
    const int32_t *page_table, *seqlens, *tree_lens;
    const uint64_t *mask;
    const __nv_bfloat16 *q;
    float *partials;
    int *status;
    int num_pages, max_pages, Hq, Hkv, tree, steps_per_split, max_splits, row_tiles;
    float s, alpha, L;
};

// Number of drafted nodes of a sequence, or -1 if its lengths are out of range.
__device__ __forceinline__ int tree_nodes(const int32_t *seqlens, const int32_t *tree_lens, int seq,
                                          int tree, int max_pages) {
    const int len = seqlens[seq], n = tree_lens ? tree_lens[seq] : tree;
    const bool ok = len >= 0 && len <= static_cast<long long>(max_pages) * kPage && n >= 0 &&
                    n <= tree;
    return ok ? n : -1;
}

__device__ __forceinline__ bool not_finite(uint32_t half_bits) {
    return (half_bits & 0x7f80u) == 0x7f80u;
}

// CTA (row tile within split, kv head, sequence).
template <int G, int MT, int kHR>
__global__ void __launch_bounds__(128)
tree_split_kernel(const __grid_constant__ CUtensorMap kv_map,
                  const __grid_constant__ CUtensorMap k_map,
                  const __grid_constant__ CUtensorMap v_map, const TreeArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    constexpr int kRows = 8 * kHR * MT;
    __shared__ __align__(8) uint64_t full_bar[kStages];
    __shared__ float mst[4][kRows][6];
    // The warps' value sums, in the page ring once every page is consumed.
    static_assert(4 * kRows * kHeadDim * sizeof(float) <= kStages * kStageBytes, "ring too small");
    float(*macc)[kRows][kHeadDim] = reinterpret_cast<float(*)[kRows][kHeadDim]>(smem);

    const int split = blockIdx.x / a.row_tiles, rt = blockIdx.x % a.row_tiles;
    const int g = blockIdx.y, seq = blockIdx.z;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gq = lane >> 2, tq = lane & 3;

    const int nodes = tree_nodes(a.seqlens, a.tree_lens, seq, a.tree, a.max_pages);
    if (nodes <= 0) {
        if (nodes < 0 && blockIdx.x == 0 && g == 0 && threadIdx.x == 0)
            record_error(a.status, POLAR_ERR_BAD_SEQLEN);
        return;
    }
    const int R = G * nodes, row0 = rt * kRows;
    if (row0 >= R) return;
    const int len = a.seqlens[seq];
    const int npg = (len + kPage - 1) / kPage;
    const int p0 = split * a.steps_per_split;
    if (p0 > npg) return;  // step npg is the drafted rows
    const int np = min(npg + 1, p0 + a.steps_per_split) - p0;
    const int32_t *pt = a.page_table + static_cast<size_t>(seq) * a.max_pages + p0;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&kv_map);
        for (int st = 0; st < kStages; ++st) mbar_init(&full_bar[st], 1);
        fence_barrier_init();
    }
    __syncthreads();

    // Producer: thread 0 fills a stage with the K and V blocks of one step.  A
    // page id outside the pool is reported and replaced by a plain arrive.
    auto usable = [&](int kk) {
        return p0 + kk == npg || (pt[kk] >= 0 && pt[kk] < a.num_pages);
    };
    auto issue = [&](int kk) {
        const int st = kk % kStages;
        uint8_t *dst = smem + st * kStageBytes;
        if (p0 + kk == npg) {
            mbar_arrive_expect_tx(&full_bar[st], kStageBytes);
            tma_load_3d(dst, &k_map, 0, g, seq * a.tree, &full_bar[st]);
            tma_load_3d(dst + kChunkBytes, &v_map, 0, g, seq * a.tree, &full_bar[st]);
        } else if (usable(kk)) {
            mbar_arrive_expect_tx(&full_bar[st], kStageBytes);
            const int row = (pt[kk] * 2 * a.Hkv + g) * kPage;  // K block of the kv head
            tma_load_2d(dst, &kv_map, 0, row, &full_bar[st]);
            tma_load_2d(dst + kChunkBytes, &kv_map, 0, row + a.Hkv * kPage, &full_bar[st]);
        } else {
            record_error(a.status, POLAR_ERR_BAD_PAGE);
            mbar_arrive(&full_bar[st]);
        }
    };
    if (threadIdx.x == 0)
        for (int kk = 0; kk < min(kStages, np); ++kk) issue(kk);

    const uint64_t drafted = first_tokens(nodes);
    const uint64_t *masks = a.mask + static_cast<size_t>(seq) * a.tree;
    RowTile<kHR> tile[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        tile[m].clear();
#pragma unroll
        for (int hr = 0; hr < kHR; ++hr) {
            const int r = row0 + m * 8 * kHR + 8 * hr + gq;
            const int t = r / G, hh = r % G;
            const bool real = r < R;
            const int n = real ? len + __popcll(masks[t] & drafted) : 0;
            tile[m].load_row(hr,
                             real ? a.q + ((static_cast<size_t>(seq) * a.tree + t) * a.Hq + g * G +
                                           hh) * kHeadDim
                                  : nullptr,
                             tq,
                             a.s * length_temperature(static_cast<float>(n), a.alpha, a.L) * kLog2e);
        }
    }

    int issued = min(kStages, np), consumed = 0;
    bool ok = true;
    const uint32_t sbase = smem_u32(smem);
    for (int kk = 0; kk < np; ++kk) {
        const int st = kk % kStages;
        const bool ready = mbar_wait(&full_bar[st], (kk / kStages) & 1, a.status);
        if (!__syncthreads_and(ready)) { ok = false; break; }
        consumed = kk + 1;
        const uint32_t kb = sbase + st * kStageBytes, vb = kb + kChunkBytes;
        if (p0 + kk < npg) {
            if (usable(kk))
                page_step<MT, kHR>(tile, kb, vb, w, lane, first_tokens(len - (p0 + kk) * kPage));
        } else {
            // The drafted rows: a mask for each row.  A value row that is not
            // finite may count only for the rows that see it, and a product
            // with a zero weight would not be zero: such values are left out
            // of the product and added to the rows that see them (their sum
            // is not finite either way).
            uint32_t kf[2][2][4];
            load_keys(kb, w, lane, kf);
            const uint32_t tok4 = lane_tokens(drafted, w, tq);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                uint32_t bits[kHR];
#pragma unroll
                for (int hr = 0; hr < kHR; ++hr) {
                    const int r = row0 + m * 8 * kHR + 8 * hr + gq;
                    bits[hr] = r < R ? lane_tokens(masks[r / G] & drafted, w, tq) : 0u;
                }
                tile[m].template score<false>(kf, bits);
            }
            bool odd = false;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t v[4];
                load_values(vb, w, lane, i, v);
                mask_values(v, tok4);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool lo = not_finite(v[e]), hi = not_finite(v[e] >> 16);
                    odd |= lo | hi;
                    v[e] = mask_pair(v[e], !lo, !hi);
                }
#pragma unroll
                for (int m = 0; m < MT; ++m) tile[m].weigh(i, v);
            }
            if (__any_sync(0xffffffffu, odd)) {
                const uint8_t *vs = smem + st * kStageBytes + kChunkBytes;
                for (int j = 16 * w; j < min(16 * w + 16, nodes); ++j)
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int hr = 0; hr < kHR; ++hr) {
                            const int r = row0 + m * 8 * kHR + 8 * hr + gq;
                            if (r >= R || !(masks[r / G] >> j & 1)) continue;
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const uint32_t x = *reinterpret_cast<const uint32_t *>(
                                    vs + swz(j, i) + 4 * tq);
                                if (not_finite(x))
                                    tile[m].acc[i][2 * hr] += __uint_as_float(x << 16);
                                if (not_finite(x >> 16))
                                    tile[m].acc[i][2 * hr + 1] += __uint_as_float(x & 0xffff0000u);
                            }
                        }
            }
        }
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
    merge_warps<MT, kHR>(tile, mst, macc, w, lane, [&](int r) -> float * {
        r += row0;
        if (r >= R) return nullptr;
        return a.partials + (((static_cast<size_t>(seq) * a.tree + r / G) * a.Hq + g * G + r % G) *
                                 a.max_splits + split) * kPartialFloats;
    });
}

// One warp per (sequence, node, query head).
__global__ void __launch_bounds__(128)
tree_merge_kernel(const float *__restrict__ partials, const int32_t *__restrict__ seqlens,
                  const int32_t *__restrict__ tree_lens, const uint64_t *__restrict__ mask,
                  const float *__restrict__ u, __nv_bfloat16 *__restrict__ out,
                  float *__restrict__ neff_out, long long rows, int Hq, int tree, int max_pages,
                  int steps_per_split, int max_splits, float s, float alpha, float L, float beta,
                  float inv_ln_L) {
    const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (row >= rows) return;
    const int lane = threadIdx.x & 31;
    const int h = static_cast<int>(row % Hq);
    const long long node = row / Hq;  // seq * tree + t
    const int seq = static_cast<int>(node / tree), t = static_cast<int>(node % tree);
    const int nodes = tree_nodes(seqlens, tree_lens, seq, tree, max_pages);
    if (t >= nodes) return;  // also a sequence out of range (-1)
    const int len = seqlens[seq];
    const int n = len + __popcll(mask[node] & first_tokens(nodes));
    const int steps = (len + kPage - 1) / kPage + 1;
    merge_splits(partials + row * max_splits * kPartialFloats,
                 (steps + steps_per_split - 1) / steps_per_split, n, s, alpha, L, beta, inv_ln_L,
                 u + static_cast<size_t>(h) * kHeadDim, lane, out + row * kHeadDim,
                 neff_out ? neff_out + row : nullptr);
}

template <int G, int MT, int kHR>
cudaError_t launch_split(const CUtensorMap &kv, const CUtensorMap &k, const CUtensorMap &v,
                         TreeArgs &t, int num_seqs, cudaStream_t stream) {
    static std::atomic<uint64_t> configured{0};  // one bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(configured.load() & bit)) {
        e = cudaFuncSetAttribute(tree_split_kernel<G, MT, kHR>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit);
    }
    t.row_tiles = (G * t.tree + 8 * kHR * MT - 1) / (8 * kHR * MT);
    tree_split_kernel<G, MT, kHR><<<dim3(t.max_splits * t.row_tiles, t.Hkv, num_seqs), 128, kSmem,
                                    stream>>>(kv, k, v, t);
    return cudaGetLastError();
}

template <int G>
cudaError_t launch_split_rows(const CUtensorMap &kv, const CUtensorMap &k, const CUtensorMap &v,
                              TreeArgs &t, int num_seqs, cudaStream_t stream) {
    if (G * t.tree <= 8) return launch_split<G, 1, 1>(kv, k, v, t, num_seqs, stream);
    if (G * t.tree <= 16) return launch_split<G, 1, 2>(kv, k, v, t, num_seqs, stream);
    return launch_split<G, 2, 2>(kv, k, v, t, num_seqs, stream);
}

// Steps (pages, and the drafted rows) per split.
int steps_per_split(int num_seqs, int max_pages, int Hkv) {
    const long long work = static_cast<long long>(num_seqs) * Hkv * (max_pages + 1);
    int n = 64;
    while (n > 2 && work / n < 148ll * 3 * 4) n >>= 1;
    return n;
}

}  // namespace

size_t tree_workspace_bytes(int num_seqs, int max_pages, int tree, int Hq, int Hkv) {
    const int per = steps_per_split(num_seqs, max_pages, Hkv);
    const size_t splits = (static_cast<size_t>(max_pages) + per) / per;
    return static_cast<size_t>(num_seqs) * tree * Hq * splits * kPartialFloats * sizeof(float);
}

bool page_pool_map(CUtensorMap *map, const void *kv_pages, int num_pages, int Hkv) {
    const uint64_t dims[2] = {static_cast<uint64_t>(kHeadDim),
                              static_cast<uint64_t>(num_pages) * 2 * Hkv * kPage};
    const uint64_t strides[1] = {kHeadDim * 2};
    const uint32_t box[2] = {kHeadDim, kPage};
    return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(kv_pages),
                        dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) == CUDA_SUCCESS;
}

cudaError_t launch_decode_tree(const TreeLaunch &a) {
    CUtensorMap kv, k, v;
    // Drafted rows as (dim, head, node): 64 nodes of one head are a page's block.
    const uint64_t dims[3] = {static_cast<uint64_t>(kHeadDim), static_cast<uint64_t>(a.Hkv),
                              static_cast<uint64_t>(a.num_seqs) * a.tree};
    const uint64_t strides[2] = {kHeadDim * 2, static_cast<uint64_t>(a.Hkv) * kHeadDim * 2};
    const uint32_t box[3] = {kHeadDim, 1, kPage};
    if (!page_pool_map(&kv, a.kv_pages, a.num_pages, a.Hkv) ||
        encode_tiled(&k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(a.k), dims,
                     strides, box, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS ||
        encode_tiled(&v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(a.v), dims,
                     strides, box, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    TreeArgs t;
    t.page_table = a.page_table; t.seqlens = a.seqlens; t.tree_lens = a.tree_lens; t.mask = a.mask;
    t.q = static_cast<const __nv_bfloat16 *>(a.q);
    t.partials = static_cast<float *>(a.workspace);
    t.status = a.status; t.num_pages = a.num_pages; t.max_pages = a.max_pages;
    t.Hq = a.Hq; t.Hkv = a.Hkv; t.tree = a.tree;
    t.steps_per_split = steps_per_split(a.num_seqs, a.max_pages, a.Hkv);
    t.max_splits = (a.max_pages + t.steps_per_split) / t.steps_per_split;
    t.s = a.s; t.alpha = a.alpha; t.L = static_cast<float>(a.L);
    cudaError_t e;
    switch (a.Hq / a.Hkv) {
        case 1: e = launch_split_rows<1>(kv, k, v, t, a.num_seqs, a.stream); break;
        case 2: e = launch_split_rows<2>(kv, k, v, t, a.num_seqs, a.stream); break;
        case 4: e = launch_split_rows<4>(kv, k, v, t, a.num_seqs, a.stream); break;
        case 8: e = launch_split_rows<8>(kv, k, v, t, a.num_seqs, a.stream); break;
        default: return cudaErrorInvalidValue;
    }
    if (e != cudaSuccess) return e;
    const long long rows = static_cast<long long>(a.num_seqs) * a.tree * a.Hq;
    tree_merge_kernel<<<static_cast<unsigned>((rows + 3) / 4), 128, 0, a.stream>>>(
        t.partials, a.seqlens, a.tree_lens, a.mask, a.u, static_cast<__nv_bfloat16 *>(a.out),
        a.neff, rows, a.Hq, a.tree, a.max_pages, t.steps_per_split, t.max_splits, a.s, a.alpha,
        static_cast<float>(a.L), a.beta, 1.0f / logf(static_cast<float>(a.L)));
    count_launches(2);
    return cudaGetLastError();
}

}  // namespace polar
