// decode_tree_tc.cu -- the drafted tree's decode on the tensor cores (tcgen05),
// for trees whose rows (node, query head of the kv group) fill a good part of
// a 128-row tile.
//
// A CTA has one row tile of a (sequence, kv head) and a share of its steps: the
// cached pages and, last, the drafted rows.  Per step of 64 keys:
//   S = Q K^T   tcgen05.mma M=128 N=64 K=64, both operands in shared memory
//   P, stats    one thread per row reads its 64 scores from tensor memory,
//               keeps max, l, l2, S1 and S2 in registers and writes the weights
//               back as bf16
//   O += P V    tcgen05.mma M=128 N=64 K=64, P from tensor memory
// S is double-buffered (P lies in its S's columns), so that the next scores are
// formed while the softmax warps work.  The reference max of a row moves only
// when a logit exceeds it by more than 2^8 (kRescaleThreshold); O is then
// rescaled in tensor memory by the row's thread, behind the products in flight.
//
// Tensor memory: 256 columns (S0 S1 O: 64 fp32 columns each), so two CTAs share
// an SM and one's softmax covers the other's waits.  Four warps do the softmax,
// one copies, one issues the products.
#include <algorithm>
#include <atomic>

#include "decode_tree.cuh"
#include "polar_internal.h"
#include "tc_common.cuh"

namespace polar {
namespace {

constexpr int kTileRows = 128;
constexpr int kStagesTc = 5;
constexpr int kTcThreads = 192;
constexpr int kQBytes = kTileRows * kHeadDim * 2;
constexpr int kSmemTc = kQBytes + kStagesTc * kStageBytes + 1024;  // + alignment slack
constexpr uint32_t kColS = 0, kColO = 128, kTmemCols = 256;
static_assert(kTileRows * kPartialFloats * 4 <= kStagesTc * kStageBytes, "ring too small");

__device__ __forceinline__ void tmem_alloc_256(uint32_t *dst_smem) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 256;" ::"r"(
                     smem_u32(dst_smem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_256(uint32_t taddr) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 256;" ::"r"(taddr) : "memory");
}

struct RowStats {  // one row's streaming state, in its thread
    float m_ref, m_raw, l, l2, s1, s2;
};

// Max and raw sums of a row's 64 scores; masked scores (bit clear) do not count.
template <bool kAll>
__device__ __forceinline__ float raw_stats(uint32_t (&sr)[2][32], uint64_t mask, RowStats &x) {
    float mx[2] = {-INFINITY, -INFINITY};
    float2 a1 = make_float2(0.f, 0.f), a2 = a1;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t m = static_cast<uint32_t>(mask >> (32 * h));
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
            float2 v = make_float2(__uint_as_float(sr[h][e]), __uint_as_float(sr[h][e + 1]));
            if (!kAll) {
                const bool v0 = m >> e & 1u, v1 = m >> (e + 1) & 1u;
                mx[(e >> 1) & 1] = max3(mx[(e >> 1) & 1], v0 ? v.x : -INFINITY, v1 ? v.y : -INFINITY);
                v.x = v0 ? v.x : 0.f;
                v.y = v1 ? v.y : 0.f;
            } else {
                mx[(e >> 1) & 1] = max3(mx[(e >> 1) & 1], v.x, v.y);
            }
            a1 = f2_add(a1, v);
            a2 = f2_fma(v, v, a2);
        }
    }
    x.s1 += a1.x + a1.y;
    x.s2 += a2.x + a2.y;
    return fmaxf(mx[0], mx[1]);
}

// Weights 2^(cl2 S - m_ref) as packed bf16, and their sums l and l2 (of the
// unrounded weights; the bf16 operand is off by at most 2^-9 of itself).
template <bool kAll>
__device__ __forceinline__ void weights(const uint32_t (&sr)[2][32], uint64_t mask, float cl2,
                                        RowStats &x, uint32_t (&pk)[32]) {
    const float ref = x.m_ref == -INFINITY ? 0.f : x.m_ref;  // nothing seen yet: weights are zero
    const float2 sc = make_float2(cl2, cl2), nm = make_float2(-ref, -ref);
    float2 la = make_float2(0.f, 0.f), l2a = la;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t m = static_cast<uint32_t>(mask >> (32 * h));
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
            const float2 v = make_float2(__uint_as_float(sr[h][e]), __uint_as_float(sr[h][e + 1]));
            const float2 z = f2_fma(v, sc, nm);
            float2 p = make_float2(ex2(z.x), ex2(z.y));
            if (!kAll) {
                p.x = m >> e & 1u ? p.x : 0.f;
                p.y = m >> (e + 1) & 1u ? p.y : 0.f;
            }
            la = f2_add(la, p);
            l2a = f2_fma(p, p, l2a);
            pk[16 * h + (e >> 1)] = pack_bf16(p.x, p.y);
        }
    }
    x.l += la.x + la.y;
    x.l2 += l2a.x + l2a.y;
}

template <int G>
__global__ void __launch_bounds__(kTcThreads, 2)
tree_tc_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap kv_map,
               const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
               const TreeArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *ring = smem + kQBytes;
    __shared__ __align__(8) uint64_t q_full, full[kStagesTc], empty[kStagesTc];
    __shared__ __align__(8) uint64_t s_full[2], p_ready[2], pv_done, mma_done;
    __shared__ unsigned long long odd_nodes;  // drafted nodes with values that are not finite
    __shared__ uint32_t tmem_base_sh;
    __shared__ int page[kMaxSteps];

    const int C = static_cast<int>(cluster_size()), group = blockIdx.x / C;
    const int rt = group % a.row_tiles, split = group / a.row_tiles;
    const int part = split * C + static_cast<int>(cluster_rank());
    const int g = blockIdx.y, seq = blockIdx.z;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const int nodes = tree_nodes(a.seqlens, a.tree_lens, seq, a.tree, a.max_pages);
    if (nodes <= 0) {
        if (nodes < 0 && blockIdx.x == 0 && g == 0 && threadIdx.x == 0)
            record_error(a.status, POLAR_ERR_BAD_SEQLEN);
        return;
    }
    const int R = G * nodes, row0 = rt * kTileRows;
    if (row0 >= R) return;
    const int len = a.seqlens[seq];
    const int npg = (len + kPage - 1) / kPage;
    const int per = (npg + a.splits * C) / (a.splits * C);  // of npg + 1 steps: the drafted rows last
    const int p0 = min(part * per, npg + 1);
    const int np = min(npg + 1, p0 + per) - p0;
    const int32_t *pt = a.page_table + static_cast<size_t>(seq) * a.max_pages + p0;

    if (threadIdx.x == 0) {
        mbar_init(&q_full, 1);
        for (int st = 0; st < kStagesTc; ++st) {
            mbar_init(&full[st], 1);
            mbar_init(&empty[st], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&s_full[b], 1);
            mbar_init(&p_ready[b], 4);
        }
        mbar_init(&pv_done, 1);
        mbar_init(&mma_done, 1);
        odd_nodes = 0;
        fence_barrier_init();
    }
    if (w == 5) tmem_alloc_256(&tmem_base_sh);
    // A page id outside the pool is reported; its step reads page 0 and counts no key.
    for (int i = threadIdx.x; i < np; i += kTcThreads) {
        const int x = p0 + i == npg ? 0 : pt[i];
        page[i] = x >= 0 && x < a.num_pages ? x : -1;
        if (page[i] < 0) record_error(a.status, POLAR_ERR_BAD_PAGE);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_sh;
    const uint64_t drafted = first_tokens(nodes);
    const uint64_t *masks = a.mask + static_cast<size_t>(seq) * a.tree;

    // This thread's row (softmax warps).
    const int row = row0 + static_cast<int>(threadIdx.x);
    const bool active = w < 4 && row0 + 32 * w < R;  // the warp has a row at all
    const uint64_t seen = w < 4 && row < R ? masks[row / G] & drafted : 0ull;
    const int n = w < 4 && row < R ? len + __popcll(seen) : 0;
    RowStats x{-INFINITY, -INFINITY, 0.f, 0.f, 0.f, 0.f};

    if (w == 4) {
        if (lane == 0 && np > 0) {
            tma_prefetch_desc(&q_map);
            tma_prefetch_desc(&kv_map);
            mbar_arrive_expect_tx(&q_full, kQBytes);
            tma_load_3d(smem, &q_map, 0, g * G, seq * a.tree + row0 / G, &q_full);
            int kk = 0;
            for (; kk < np; ++kk) {
                const int st = kk % kStagesTc;
                if (kk >= kStagesTc && !mbar_wait(&empty[st], ((kk / kStagesTc) - 1) & 1, a.status))
                    break;
                uint8_t *dst = ring + st * kStageBytes;
                mbar_arrive_expect_tx(&full[st], kStageBytes);
                if (p0 + kk == npg) {
                    tma_load_3d(dst, &k_map, 0, g, seq * a.tree, &full[st]);
                    tma_load_3d(dst + kChunkBytes, &v_map, 0, g, seq * a.tree, &full[st]);
                } else {
                    const int at = (max(page[kk], 0) * 2 * a.Hkv + g) * kPage;
                    tma_load_2d(dst, &kv_map, 0, at, &full[st]);
                    tma_load_2d(dst + kChunkBytes, &kv_map, 0, at + a.Hkv * kPage, &full[st]);
                }
            }
            // Every copy lands before shared memory is reused or released.
            mbar_wait(&q_full, 0, a.status);
            for (int j = max(0, kk - kStagesTc); j < kk; ++j)
                mbar_wait(&full[j % kStagesTc], (j / kStagesTc) & 1, a.status);
        }
        __syncwarp();
    } else if (w == 5) {
        if (lane == 0 && np > 0) {
            constexpr uint32_t idesc_qk = idesc_bf16(kTileRows, kPage, false);
            constexpr uint32_t idesc_pv = idesc_bf16(kTileRows, kHeadDim, true);
            // Q and K are K-major (SBO 1024), V is MN-major (one 64-column atom).
            const uint32_t q_lo = sdesc_lo(smem_u32(smem), 16);
            const uint32_t k_lo = sdesc_lo(smem_u32(ring), 16);
            const uint32_t v_lo = sdesc_lo(smem_u32(ring) + kChunkBytes, 8192);
            constexpr uint32_t hi = kSdescHi128B, kStep = kStageBytes >> 4;
            bool ok = mbar_wait(&q_full, 0, a.status);
            for (int i = 0; i <= np && ok; ++i) {
                if (i < np) {
                    const int st = i % kStagesTc;
                    // S_i overwrites P_(i-2): its product is done.
                    if (i >= 2 && !(ok = mbar_wait(&pv_done, (i - 2) & 1, a.status))) break;
                    if (!(ok = mbar_wait(&full[st], (i / kStagesTc) & 1, a.status))) break;
                    tc_fence_after();
                    const uint32_t d = tmem + kColS + (i & 1) * 64, ka = k_lo + st * kStep;
                    mma_ss2<0>(d, q_lo, hi, ka, hi, idesc_qk);
                    mma_ss2<1>(d, q_lo + 2, hi, ka + 2, hi, idesc_qk);
                    mma_ss2<1>(d, q_lo + 4, hi, ka + 4, hi, idesc_qk);
                    mma_ss2<1>(d, q_lo + 6, hi, ka + 6, hi, idesc_qk);
                    tc_commit(&s_full[i & 1]);
                }
                if (i >= 1) {
                    const int j = i - 1, st = j % kStagesTc;
                    if (!(ok = mbar_wait(&p_ready[j & 1], (j >> 1) & 1, a.status))) break;
                    tc_fence_after();
                    const uint32_t va = v_lo + st * kStep, pa = tmem + kColS + (j & 1) * 64;
                    mma_ts2(tmem + kColO, pa, va, hi, idesc_pv, j > 0);
#pragma unroll
                    for (int kk = 1; kk < kPage / 16; ++kk)
                        mma_ts2(tmem + kColO, pa + 8 * kk, va + 128 * kk, hi, idesc_pv, 1u);
                    tc_commit(&empty[st]);
                    tc_commit(&pv_done);
                }
            }
            // All products complete before tensor memory is freed.
            tc_commit(&mma_done);
            mbar_wait(&mma_done, 0, a.status);
        }
        __syncwarp();
    } else {
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(32 * w) << 16);
        const uint32_t tO = lane_base + kColO;
        const float cl2 = a.ep.s * length_temperature(static_cast<float>(n), a.ep.alpha, a.ep.L) *
                          kLog2e;
        bool ok = true;
        for (int i = 0; i < np; ++i) {
            ok = mbar_wait(&s_full[i & 1], (i >> 1) & 1, a.status);
            if (!__all_sync(~0u, ok)) { ok = false; break; }
            tc_fence_after();
            const bool draft = p0 + i == npg;
            const int left = len - (p0 + i) * kPage;  // cached tokens of this step
            // The step's keys: a full page, or a mask.
            const uint64_t mask = draft ? seen : page[i] < 0 ? 0ull : first_tokens(left);
            const bool all = !draft && page[i] >= 0 && left >= kPage;
            if (!all) {
                // Value rows that no row may see are zeroed, since a zero weight
                // does not silence what is not finite; drafted values that are
                // not finite are zeroed and added to the rows that see them at
                // the end.
                const int st = i % kStagesTc;
                const bool landed = mbar_wait(&full[st], (i / kStagesTc) & 1, a.status);
                const uint64_t keep = draft ? drafted : mask;
                uint32_t odd = 0;
                if (landed)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int r = 16 * w + 4 * e + (lane >> 3);
                        uint4 *v = reinterpret_cast<uint4 *>(ring + st * kStageBytes + kChunkBytes +
                                                             r * 128) + (lane & 7);
                        if (!(keep >> r & 1)) {
                            *v = make_uint4(0, 0, 0, 0);
                        } else if (draft) {
                            uint4 y = *v;
                            uint32_t *word = reinterpret_cast<uint32_t *>(&y);
                            bool bad = false;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const bool lo = not_finite(word[k]), up = not_finite(word[k] >> 16);
                                bad |= lo | up;
                                word[k] = mask_pair(word[k], !lo, !up);
                            }
                            if (bad) {
                                *v = y;
                                odd |= 1u << (4 * e + (lane >> 3));
                            }
                        }
                    }
                if (odd) atomicOr(&odd_nodes, static_cast<unsigned long long>(odd) << (16 * w));
                fence_proxy_async_smem();
                __syncwarp();
            }
            if (active) {
                const uint32_t tS = lane_base + kColS + (i & 1) * 64;
                uint32_t sr[2][32], pk[32];
                tmem_ld32(tS, sr[0]);
                tmem_ld32(tS + 32, sr[1]);
                tmem_wait_ld();
                const float tmax = all ? raw_stats<true>(sr, mask, x) : raw_stats<false>(sr, mask, x);
                x.m_raw = fmaxf(x.m_raw, tmax);
                const float zmax = tmax * cl2;
                const bool need = zmax > x.m_ref + kRescaleThreshold;
                if (__any_sync(~0u, need)) {
                    const float r = need ? exp2f(x.m_ref - zmax) : 1.f;  // 0 where nothing was seen
                    x.l *= r;
                    x.l2 *= r * r;
                    if (need) x.m_ref = zmax;
                    if (i > 0) {  // O *= r, once the products before are done
                        ok = mbar_wait(&pv_done, (i - 1) & 1, a.status);
                        if (!__all_sync(~0u, ok)) { ok = false; break; }
                        tc_fence_after();
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t o[32];
                            tmem_ld32(tO + 32 * h, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * r);
                            tmem_st32(tO + 32 * h, o);
                        }
                    }
                }
                if (all)
                    weights<true>(sr, mask, cl2, x, pk);
                else
                    weights<false>(sr, mask, cl2, x, pk);
                tmem_st32(tS, pk);
                tmem_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_ready[i & 1]);
        }
        // Rows without a step keep the empty state.
        if (ok && np > 0) ok = mbar_wait(&pv_done, (np - 1) & 1, a.status);
        ok = __all_sync(~0u, ok) && np > 0;
        tc_fence_after();
        // The copies of this CTA have all been consumed: its ring takes the rows' states.
        float *own = reinterpret_cast<float *>(ring) + threadIdx.x * kPartialFloats;
        named_barrier(1, 128);  // every softmax warp is past the last product
        if (active) {
            // Where it counts, drafted values that are not finite.
            const uint64_t extra = ok ? odd_nodes & seen : 0ull;
            const __nv_bfloat16 *vrow = a.v + (static_cast<size_t>(seq) * a.tree * a.Hkv + g) *
                                                  kHeadDim;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t o[32];
                if (ok) {
                    tmem_ld32(tO + 32 * h, o);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0u;
                }
                for (uint64_t todo = extra; todo; todo &= todo - 1) {
                    const int j = __ffsll(static_cast<long long>(todo)) - 1;
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float y = __bfloat162float(
                            vrow[static_cast<size_t>(j) * a.Hkv * kHeadDim + 32 * h + e]);
                        if (!(fabsf(y) < INFINITY))
                            o[e] = __float_as_uint(__uint_as_float(o[e]) + y);
                    }
                }
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    *reinterpret_cast<uint4 *>(own + 32 * h + e) =
                        make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
            if (!ok) x = RowStats{-INFINITY, -INFINITY, 0.f, 0.f, 0.f, 0.f};
            *reinterpret_cast<float4 *>(own + 64) = make_float4(x.m_ref, x.m_raw, x.l, x.l2);
            *reinterpret_cast<float2 *>(own + 68) = make_float2(x.s1, x.s2);
        }
        tc_fence_before();
    }
    let_next_kernel_start();
    __syncthreads();
    tc_fence_after();
    if (w == 5) tmem_dealloc_256(tmem);

    // The cluster's states of a row: eight lanes merge them and finish the row.
    const float *parts = reinterpret_cast<const float *>(ring);
    const int nrows = min(kTileRows, R - row0), rank = static_cast<int>(cluster_rank());
    if (C > 1) cluster_sync();
    for (int r0 = w < 4 ? 4 * (w * C + rank) : nrows; r0 < nrows; r0 += 16 * C) {
        const int r = min(r0 + (lane >> 3), nrows - 1);
        const bool real = r0 + (lane >> 3) < nrows;
        const RowState st = merge_parts(C, [&](int k) {
            const float *p = parts + r * kPartialFloats;
            return C > 1 ? cluster_map(p, k) : p;
        });
        const int t = (row0 + r) / G, h = g * G + (row0 + r) % G;
        const size_t out_row = (static_cast<size_t>(seq) * a.tree + t) * a.Hq + h;
        if (a.splits > 1)
            store_part(st, a.partials + (out_row * a.splits + split) * kPartialFloats, real);
        else
            finish_row(st, len + __popcll(masks[t] & drafted), a.ep, a.u + h * kHeadDim,
                       a.out + out_row * kHeadDim, a.neff ? a.neff + out_row : nullptr, real);
    }
    if (C > 1) cluster_sync();  // no CTA leaves while its states are read
}

template <int G>
cudaError_t launch_tc(const CUtensorMap &q, const CUtensorMap &kv, const CUtensorMap &k,
                      const CUtensorMap &v, const TreeArgs &t, const TreePlan &plan, int num_seqs,
                      cudaStream_t stream) {
    static std::atomic<uint64_t> configured{0};  // one bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(configured.load() & bit)) {
        e = cudaFuncSetAttribute(tree_tc_kernel<G>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kSmemTc);
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit);
    }
    return launch_ex(tree_tc_kernel<G>, dim3(plan.cluster * plan.splits * plan.row_tiles, t.Hkv,
                                             num_seqs),
                     kTcThreads, kSmemTc, plan.cluster, false, stream, q, kv, k, v, t);
}

}  // namespace

cudaError_t launch_tree_tc(const CUtensorMap &kv, const CUtensorMap &k, const CUtensorMap &v,
                           const TreeArgs &t, const TreePlan &plan, int num_seqs,
                           cudaStream_t stream) {
    CUtensorMap q;
    const int G = t.Hq / t.Hkv;
    // Query rows as (dim, head, node): a tile is the group's heads of 128 / G nodes.
    const uint64_t dims[3] = {static_cast<uint64_t>(kHeadDim), static_cast<uint64_t>(t.Hq),
                              static_cast<uint64_t>(num_seqs) * t.tree};
    const uint64_t strides[2] = {kHeadDim * 2, static_cast<uint64_t>(t.Hq) * kHeadDim * 2};
    const uint32_t box[3] = {kHeadDim, static_cast<uint32_t>(G),
                             static_cast<uint32_t>(kTileRows / G)};
    if (encode_tiled(&q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16 *>(t.q), dims,
                     strides, box, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    switch (G) {
        case 1: return launch_tc<1>(q, kv, k, v, t, plan, num_seqs, stream);
        case 2: return launch_tc<2>(q, kv, k, v, t, plan, num_seqs, stream);
        case 4: return launch_tc<4>(q, kv, k, v, t, plan, num_seqs, stream);
        case 8: return launch_tc<8>(q, kv, k, v, t, plan, num_seqs, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace polar
