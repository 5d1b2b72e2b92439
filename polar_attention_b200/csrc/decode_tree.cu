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

#include "decode_tree.cuh"
#include "polar_internal.h"
#include "tc_common.cuh"

namespace polar {
namespace {

constexpr int kSmem = kRingStages * kStageBytes + 1024;  // + alignment slack
constexpr int kMaxCluster = 8;
constexpr int kTcSteps = 8192;

// CTA (part and row tile, kv head, sequence); the parts are equal shares of the
// sequence's steps.  A cluster along x merges its CTAs' states; with one
// cluster per row tile it writes the rows, else partials.  Tiles of 8 or 16
// rows: 32 rows read a page half as often but left half as many CTAs for the
// same work (1 sequence of 1500 tokens, 64 rows: 16.5 us, 16 rows 12.4).
template <int G, int kHR>
__global__ void __launch_bounds__(kRowThreads, kHR == 2 ? 3 : 4)
tree_split_kernel(const __grid_constant__ CUtensorMap kv_map,
                  const __grid_constant__ CUtensorMap k_map,
                  const __grid_constant__ CUtensorMap v_map, const TreeArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    constexpr int kRows = 8 * kHR;
    __shared__ __align__(8) PageRing ring;
    // The rows' states go to the page ring once every page is consumed.
    static_assert(5 * kRows * kPartialFloats * sizeof(float) <= kRingStages * kStageBytes,
                  "ring too small");

    const int C = static_cast<int>(cluster_size()), group = blockIdx.x / C;
    const int rt = group % a.row_tiles, split = group / a.row_tiles;
    const int part = split * C + static_cast<int>(cluster_rank());
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
    // Of npg + 1 steps: the drafted rows last.
    const int per = (npg + a.splits * C) / (a.splits * C);
    const int p0 = min(part * per, npg + 1);
    const int np = min(npg + 1, p0 + per) - p0;
    const int32_t *pt = a.page_table + static_cast<size_t>(seq) * a.max_pages + p0;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&kv_map);
        init_ring(ring);
    }
    // A page id outside the pool is reported and its step skipped.
    for (int i = threadIdx.x; i < np; i += kRowThreads) {
        const int x = p0 + i == npg ? 0 : pt[i];
        ring.page[i] = x >= 0 && x < a.num_pages ? x : -1;
        if (ring.page[i] < 0) record_error(a.status, POLAR_ERR_BAD_PAGE);
    }
    __syncthreads();

    const uint32_t sbase = smem_u32(smem);
    const uint64_t drafted = first_tokens(nodes);
    const uint64_t *masks = a.mask + static_cast<size_t>(seq) * a.tree;
    RowTile<kHR> tile;
    if (w == kRowWarps) {
        if (lane == 0)
            copy_steps(ring, np, a.status, [&](int kk, int st, uint64_t *bar) {
                uint8_t *dst = smem + st * kStageBytes;
                const int phys = ring.page[kk];
                if (phys < 0) {
                    mbar_arrive(bar);
                    return;
                }
                mbar_arrive_expect_tx(bar, kStageBytes);
                if (p0 + kk == npg) {
                    tma_load_3d(dst, &k_map, 0, g, seq * a.tree, bar);
                    tma_load_3d(dst + kChunkBytes, &v_map, 0, g, seq * a.tree, bar);
                } else {
                    const int row = (phys * 2 * a.Hkv + g) * kPage;  // K block of the kv head
                    tma_load_2d(dst, &kv_map, 0, row, bar);
                    tma_load_2d(dst + kChunkBytes, &kv_map, 0, row + a.Hkv * kPage, bar);
                }
            });
        __syncwarp();
    }
    const bool computes = w < kRowWarps;
    tile.clear();
#pragma unroll
    for (int hr = 0; hr < kHR; ++hr) {
        const int r = row0 + 8 * hr + gq;
        const int t = r / G, hh = r % G;
        const bool real = computes && r < R;
        const int n = real ? len + __popcll(masks[t] & drafted) : 0;
        tile.load_row(hr,
                      real ? a.q + ((static_cast<size_t>(seq) * a.tree + t) * a.Hq + g * G + hh) *
                                       kHeadDim
                           : nullptr,
                      tq,
                      a.ep.s * length_temperature(static_cast<float>(n), a.ep.alpha, a.ep.L) *
                          kLog2e);
    }

    if (computes) compute_steps(ring, np, lane, a.status, [&](int kk, int st) {
        const uint32_t kb = sbase + st * kStageBytes, vb = kb + kChunkBytes;
        if (p0 + kk < npg) {
            if (ring.page[kk] >= 0)
                page_step(tile, kb, vb, w, lane, first_tokens(len - (p0 + kk) * kPage));
        } else {
            // The drafted rows: a mask for each row.  A value row that is not
            // finite may count only for the rows that see it, and a product
            // with a zero weight would not be zero: such values are left out
            // of the product and added to the rows that see them (their sum
            // is not finite either way).
            uint32_t kf[2][2][4];
            load_keys(kb, w, lane, kf);
            const uint32_t tok4 = lane_tokens(drafted, w, tq);
            uint32_t bits[kHR];
#pragma unroll
            for (int hr = 0; hr < kHR; ++hr) {
                const int r = row0 + 8 * hr + gq;
                bits[hr] = r < R ? lane_tokens(masks[r / G] & drafted, w, tq) : 0u;
            }
            tile.template score<false>(kf, bits);
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
                tile.weigh(i, v);
            }
            if (__any_sync(0xffffffffu, odd)) {
                const uint8_t *vs = smem + st * kStageBytes + kChunkBytes;
                for (int j = 16 * w; j < min(16 * w + 16, nodes); ++j)
#pragma unroll
                    for (int hr = 0; hr < kHR; ++hr) {
                        const int r = row0 + 8 * hr + gq;
                        if (r >= R || !(masks[r / G] >> j & 1)) continue;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const uint32_t x =
                                *reinterpret_cast<const uint32_t *>(vs + swz(j, i) + 4 * tq);
                            if (not_finite(x))
                                tile.acc[i][2 * hr] += __uint_as_float(x << 16);
                            if (not_finite(x >> 16))
                                tile.acc[i][2 * hr + 1] += __uint_as_float(x & 0xffff0000u);
                        }
                    }
            }
        }
    });
    let_next_kernel_start();
    reduce_rows(tile, reinterpret_cast<float *>(smem), min(kRows, R - row0), w, lane,
                [&](int r, bool real, const RowState &x) {
        const int t = (row0 + r) / G, h = g * G + (row0 + r) % G;
        const size_t row = (static_cast<size_t>(seq) * a.tree + t) * a.Hq + h;
        if (a.splits > 1)
            store_part(x, a.partials + (row * a.splits + split) * kPartialFloats, real);
        else
            finish_row(x, len + __popcll(masks[t] & drafted), a.ep, a.u + h * kHeadDim,
                       a.out + row * kHeadDim, a.neff ? a.neff + row : nullptr, real);
    });
}

// Eight lanes per (sequence, node, query head).
__global__ void __launch_bounds__(128) tree_merge_kernel(const TreeArgs a, long long rows) {
    long long row = static_cast<long long>(blockIdx.x) * 16 + (threadIdx.x >> 3);
    bool real = row < rows;
    row = min(row, rows - 1);
    const int h = static_cast<int>(row % a.Hq);
    const long long node = row / a.Hq;  // seq * tree + t
    const int seq = static_cast<int>(node / a.tree), t = static_cast<int>(node % a.tree);
    const int nodes = tree_nodes(a.seqlens, a.tree_lens, seq, a.tree, a.max_pages);
    real = real && t < nodes;  // not of a sequence out of range (-1)
    const int n = real ? a.seqlens[seq] + __popcll(a.mask[node] & first_tokens(nodes)) : 0;
    wait_for_previous_kernel();
    const float *base = a.partials + row * a.splits * kPartialFloats;
    finish_row(merge_parts(real ? a.splits : 0, [&](int k) { return base + k * kPartialFloats; }),
               n, a.ep, a.u + h * kHeadDim, a.out + row * kHeadDim,
               a.neff ? a.neff + row : nullptr, real);
}

template <int G, int kHR>
cudaError_t launch_split(const CUtensorMap &kv, const CUtensorMap &k, const CUtensorMap &v,
                         const TreeArgs &t, const TreePlan &plan, int num_seqs,
                         cudaStream_t stream) {
    static std::atomic<uint64_t> configured{0};  // one bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(configured.load() & bit)) {
        e = cudaFuncSetAttribute(tree_split_kernel<G, kHR>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit);
    }
    return launch_ex(tree_split_kernel<G, kHR>,
                     dim3(plan.cluster * plan.splits * plan.row_tiles, t.Hkv, num_seqs),
                     kRowThreads, kSmem, plan.cluster, false, stream, kv, k, v, t);
}

template <int G>
cudaError_t launch_split_rows(const CUtensorMap &kv, const CUtensorMap &k, const CUtensorMap &v,
                              const TreeArgs &t, const TreePlan &plan, int num_seqs,
                              cudaStream_t stream) {
    if (plan.tile_rows == 8) return launch_split<G, 1>(kv, k, v, t, plan, num_seqs, stream);
    return launch_split<G, 2>(kv, k, v, t, plan, num_seqs, stream);
}

TreePlan tree_plan(int num_seqs, int max_pages, int tree, int Hq, int Hkv) {
    TreePlan p;
    const int R = Hq / Hkv * tree;
    p.tile_rows = R <= 8 ? 8 : 16;
    p.row_tiles = (R + p.tile_rows - 1) / p.tile_rows;
    const long long tiles = static_cast<long long>(num_seqs) * Hkv * p.row_tiles;
    const int steps = max_pages + 1;
    p.cluster = 1;
    // No more CTAs than fit at once: 512 of which 444 fit took 19.4 us, 256 of them
    // 10.3 (16 sequences of 200 .. 400 tokens, 16 rows).
    const int at_once = 148 * (p.tile_rows == 8 ? 4 : 3);
    while (p.cluster < kMaxCluster && tiles * p.cluster * 2 <= at_once && p.cluster * 2 <= steps)
        p.cluster *= 2;
    p.splits = 1;
    while ((tiles * p.cluster * p.splits * 2 <= at_once && p.cluster * p.splits * 16 <= steps) ||
           p.cluster * p.splits * kMaxSteps < steps)
        p.splits *= 2;
    return p;
}

// Rows of more than one m16 tile read every page again here; the 128-row tiles of
// tcgen05 read it once, though most of a tile may be padding and its pipeline
// takes longer to fill.  Up to 16 rows this kernel is faster at any size (16
// sequences of 4096 .. 16384 tokens, 4 kv heads, 16 rows: 55 us, tcgen05 65).
// Above, it depends on the steps over all m16 tiles (us here, us by tcgen05):
//   rows 32, 1 sequence of 1500: 10.7, 20.5; of 16000 (4000 steps): 22.6, 24.4
//   rows 128, 1 sequence of 8000 (4100): 21.4, 24.7; of 16000 (8000): 32.8, 28.8
//   rows 64, 16 sequences of 500 .. 2000 (8400): 30.8, 31.4
//   rows 24, 1 sequence of 60000 (7500): 33.0, 37.0; rows 64 (15000): 54, 43
//   rows 32, 16 sequences of 4096 .. 16384 (33000): 98, 65.
bool uses_tc(int num_seqs, int max_pages, int tree, int Hq, int Hkv) {
    const int R = Hq / Hkv * tree;
    return R > 16 &&
           static_cast<long long>(num_seqs) * Hkv * ((R + 15) / 16) * (max_pages + 1) >= kTcSteps;
}

}  // namespace

size_t tree_workspace_bytes(int num_seqs, int max_pages, int tree, int Hq, int Hkv) {
    if (uses_tc(num_seqs, max_pages, tree, Hq, Hkv))
        return tree_tc_workspace_bytes(num_seqs, max_pages, tree, Hq, Hkv);
    const TreePlan p = tree_plan(num_seqs, max_pages, tree, Hq, Hkv);
    if (p.splits == 1) return 16;  // none of it is touched
    return static_cast<size_t>(num_seqs) * tree * Hq * p.splits * kPartialFloats * sizeof(float);
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
    const TreePlan plan = tree_plan(a.num_seqs, a.max_pages, a.tree, a.Hq, a.Hkv);
    TreeArgs t;
    t.page_table = a.page_table; t.seqlens = a.seqlens; t.tree_lens = a.tree_lens; t.mask = a.mask;
    t.q = static_cast<const __nv_bfloat16 *>(a.q); t.v = static_cast<const __nv_bfloat16 *>(a.v);
    t.u = a.u; t.out = static_cast<__nv_bfloat16 *>(a.out); t.neff = a.neff;
    t.partials = static_cast<float *>(a.workspace);
    t.status = a.status; t.num_pages = a.num_pages; t.max_pages = a.max_pages;
    t.Hq = a.Hq; t.Hkv = a.Hkv; t.tree = a.tree; t.num_seqs = a.num_seqs;
    t.splits = plan.splits; t.row_tiles = plan.row_tiles;
    const float L = static_cast<float>(a.L);
    t.ep = Epilogue{a.s, a.alpha, L, a.beta, 1.0f / logf(L)};
    cudaError_t e;
    if (uses_tc(a.num_seqs, a.max_pages, a.tree, a.Hq, a.Hkv)) {
        count_launches(2);
        return launch_tree_tc(kv, k, v, t,
                              tree_tc_ctas(a.num_seqs, a.max_pages, a.tree, a.Hq, a.Hkv), a.stream);
    }
    switch (a.Hq / a.Hkv) {
        case 1: e = launch_split_rows<1>(kv, k, v, t, plan, a.num_seqs, a.stream); break;
        case 2: e = launch_split_rows<2>(kv, k, v, t, plan, a.num_seqs, a.stream); break;
        case 4: e = launch_split_rows<4>(kv, k, v, t, plan, a.num_seqs, a.stream); break;
        case 8: e = launch_split_rows<8>(kv, k, v, t, plan, a.num_seqs, a.stream); break;
        default: return cudaErrorInvalidValue;
    }
    if (e != cudaSuccess) return e;
    count_launches(1);
    if (plan.splits > 1) {
        const long long rows = static_cast<long long>(a.num_seqs) * a.tree * a.Hq;
        e = launch_ex(tree_merge_kernel, dim3(static_cast<unsigned>((rows + 15) / 16)), 128, 0, 1,
                      true, a.stream, t, rows);
        if (e != cudaSuccess) return e;
        count_launches(1);
    }
    return cudaSuccess;
}

}  // namespace polar
