// decode_tree.cuh -- what the drafted tree's kernels share: their arguments, the
// launch plan and the checks of a sequence's lengths.
#pragma once

#include "decode_rows.cuh"

namespace polar {

struct TreeArgs {
    const int32_t *page_table, *seqlens, *tree_lens;
    const uint64_t *mask;
    const __nv_bfloat16 *q, *v;
    const float *u;
    __nv_bfloat16 *out;
    float *neff, *partials;
    int *status;
    int num_seqs, num_pages, max_pages, Hq, Hkv, tree;
    int splits;     // clusters per row tile
    int row_tiles;  // row tiles per (sequence, kv head)
    Epilogue ep;
};

struct TreePlan {  // the mma.sync kernel's grid
    int tile_rows;  // 8 or 16
    int row_tiles, cluster, splits;
};

// The tcgen05 kernel (128-row tiles): its CTAs, the workspace they need, and
// the launch, given the tensor maps over the page pool and the drafted rows.
int tree_tc_ctas(int num_seqs, int max_pages, int tree, int Hq, int Hkv);
size_t tree_tc_workspace_bytes(int num_seqs, int max_pages, int tree, int Hq, int Hkv);
cudaError_t launch_tree_tc(const CUtensorMap &kv, const CUtensorMap &k, const CUtensorMap &v,
                           const TreeArgs &t, int ctas, cudaStream_t stream);

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

}  // namespace polar
