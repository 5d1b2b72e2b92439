// decode_tree_tc.cu -- the drafted tree's decode on the tensor cores (tcgen05),
// for trees whose rows (node, query head of the kv group) fill a good part of
// a 128-row tile.
//
// Work.  A tile is 128 rows of one (sequence, kv head); its steps are the
// cached pages and, last, the drafted rows, 64 keys each.  All steps of all
// tiles in a row, cut into equal shares, are the CTAs' work: whatever the
// sequences' lengths, the CTAs end together, and tiles that read the same pages
// do so at the same time.  A CTA goes through its share tile by tile; a tile it
// holds whole it finishes, of a tile it shares it stores the rows' states, which
// tree_tc_merge_kernel joins (at most two such tiles a CTA: its first and last).
//
// A step is a page, 64 keys:
//   S = Q K^T   tcgen05.mma M=128 N=64 K=64, operands in shared memory
//   P, stats    one thread per row reads its scores from tensor memory 32 at a
//               time, keeps max, l, l2, S1 and S2 in registers and writes the
//               weights back as bf16 (P lies in S's columns)
//   O += P V    tcgen05.mma M=128 N=64 K=64, P from tensor memory
// A CTA's step is one chain; 128 columns (S, O) and two 16 KB stages are all it
// needs, so four CTAs share an SM and cover each other's waits.
//
// What bounds it (64 nodes, 8 sequences of 32K-64K, 221-250 us): the four chains of an
// SM wait for one another.  The products' pipe is busy for 34 % of the time,
// exponentials 45 %, issue slots 48 %.  Measured while the raw scores were summed
// without means (215-232 us): per SM and step of a full tile about 1100 clocks; a
// chain alone on its SM 2100 for a step, 270 and 180 of them to issue the products,
// about 300 until each is seen, 900 for the weights and sums, of which 512 are
// exponentials (16 an SM and clock), 200 to reach tensor memory and back.  Loads do
// not bound it (half of them left out, or all from one page: the same time).  Tried
// then: two threads a row in clusters of eight CTAs, two an SM, 310-330 us; equal
// shares with a 64-key buffer and one thread for copies and products 268 us, with
// two 32-key buffers 255 us, with 128-key steps and two CTAs an SM 283 us; two
// 64-key buffers and two CTAs an SM 235 us; three chains with the next scores formed
// during a step's weights (160 columns a chain, one CTA of 480 threads) 230-240 us.
//
// The reference max of a row moves only when a logit exceeds it by more than
// 2^24 (kTcThreshold), and then to a whole number of log2 units: weights are
// formed against the one at hand in the pass that finds the scores' max, and only
// where that was too low they are formed again, and O and the step's weights so
// far multiplied by a power of two in tensor memory by the row's thread.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "decode_tree.cuh"
#include "polar_attn_selftest.h"
#include "polar_internal.h"
#include "tc_common.cuh"

namespace polar {
namespace {

constexpr int kTileRows = 128;
constexpr int kStagesTc = 2;
constexpr int kTcThreads = 192;  // four softmax warps, one that copies, one that issues products
constexpr int kTcPerSm = 4;
constexpr int kQBytes = kTileRows * kHeadDim * 2;
constexpr int kSmemTc = kQBytes + kStagesTc * kStageBytes + 1024;  // + alignment slack
constexpr uint32_t kColS = 0, kColO = 64;
// How far (log2 units) a logit may exceed a row's reference before it moves: up
// to 2^24 times 2^18 keys, squared, stays far inside fp32, and bf16 weights keep
// their relative precision, so a row rarely moves it after its first keys.
constexpr float kTcThreshold = 24.0f;
constexpr int kSlotFloats = kTileRows * kPartialFloats;

__device__ __forceinline__ void tmem_alloc_128(uint32_t *dst_smem) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 128;" ::"r"(
                     smem_u32(dst_smem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_128(uint32_t taddr) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 128;" ::"r"(taddr) : "memory");
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one != 0;
}

// Steps that a share has at least (4 sequences of 4000-5000 tokens, 128 rows: at
// least 1 36.8 us, 4 28.8, 12 32.9).
constexpr int kMinShare = 4;
constexpr int kMergeThreads = 256;

// Tiles that the sequences can have.
long long num_tiles(int num_seqs, int tree, int Hq, int Hkv) {
    return static_cast<long long>(num_seqs) * Hkv * ((Hq / Hkv * tree + kTileRows - 1) / kTileRows);
}

constexpr size_t record_bytes(long long tiles) {
    return (static_cast<size_t>(tiles) * 3 * sizeof(int) + 15) / 16 * 16;
}

// One pass over a thread's 32 scores against its reference max: the weights
// 2^(cl2 S - m_ref) as packed bf16 (operands of the second product, off by at
// most half a step, 2^-8 of themselves; the sums take them unrounded), their
// sums, the max and the raw scores' sums.  Scores whose mask bit is clear do not
// count.
struct TileSums {
    float top, s1, s2, l, l2;
};
template <bool kAll>
__device__ __forceinline__ TileSums tile_pass(const uint32_t (&sr)[32], uint32_t mask, float cl2,
                                              float m_ref, uint32_t (&pk)[16]) {
    const float2 sc = make_float2(cl2, cl2), nm = make_float2(-m_ref, -m_ref);
    float mx[2] = {-INFINITY, -INFINITY};
    float2 a1 = make_float2(0.f, 0.f), a2 = a1, la = a1, l2a = a1;
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
        float2 v = make_float2(__uint_as_float(sr[e]), __uint_as_float(sr[e + 1]));
        const bool v0 = kAll || (mask >> e & 1u), v1 = kAll || (mask >> (e + 1) & 1u);
        const float2 z = f2_fma(v, sc, nm);
        mx[(e >> 1) & 1] = max3(mx[(e >> 1) & 1], v0 ? v.x : -INFINITY, v1 ? v.y : -INFINITY);
        if (!kAll) v = make_float2(v0 ? v.x : 0.f, v1 ? v.y : 0.f);
        a1 = f2_add(a1, v);
        a2 = f2_fma(v, v, a2);
        float2 p = make_float2(ex2(z.x), ex2(z.y));
        if (!kAll) p = make_float2(v0 ? p.x : 0.f, v1 ? p.y : 0.f);
        la = f2_add(la, p);
        l2a = f2_fma(p, p, l2a);
        pk[e >> 1] = pack_bf16(p.x, p.y);
    }
    return TileSums{fmaxf(mx[0], mx[1]), a1.x + a1.y, a2.x + a2.y, la.x + la.y, l2a.x + l2a.y};
}

// Sum of squares of a thread's 32 scores about `mean`, of those that count.
__device__ __forceinline__ float squares_about(const uint32_t (&sr)[32], uint32_t mask,
                                               float mean) {
    const float2 off = make_float2(-mean, -mean);
    float2 a = make_float2(0.f, 0.f);
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
        float2 d = f2_add(make_float2(__uint_as_float(sr[e]), __uint_as_float(sr[e + 1])), off);
        d = make_float2(mask >> e & 1u ? d.x : 0.f, mask >> (e + 1) & 1u ? d.y : 0.f);
        a = f2_fma(d, d, a);
    }
    return a.x + a.y;
}

// 16 n columns of fp32 of this thread's lane of tensor memory, times r.  The stores
// are complete on return: the second half of a step may load the columns again.
__device__ __forceinline__ void scale_columns(uint32_t t, int n, float r) {
#pragma unroll 1
    for (int c = 0; c < n; ++c) {
        uint32_t o[16];
        tmem_ld16(t + 16 * c, o);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * r);
        tmem_st16(t + 16 * c, o);
    }
    tmem_wait_st();
}

// The weights of a step's first half (16 columns of bf16 pairs), times a power
// of two.
__device__ __forceinline__ void scale_weights(uint32_t t, float r) {
    uint32_t o[16];
    tmem_wait_st();
    tmem_ld16(t, o);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 16; ++e)
        o[e] = pack_bf16(__uint_as_float(o[e] << 16) * r, __uint_as_float(o[e] & 0xffff0000u) * r);
    tmem_st16(t, o);
}

struct RowStats {  // one row's streaming state, in its thread
    float m_ref, m_raw, l, l2;
    Moments dots;
};

// What the CTA in which a tile begins leaves to the merge.
struct SharedTile {
    int parts;      // CTAs that hold steps of the tile; 1: it is finished
    int cta, slot;  // part 0 is in this slot, part j > 0 in slot 2 (cta + j)
};

// A share of the steps, tile by tile.
template <int G>
struct Walk {
    const TreeArgs &a;
    int seq, tile, step;      // tile: head * tiles per head + row tile
    int nodes, len, per_tile, tiles;  // of the sequence
    long long left;

    __device__ __forceinline__ int tiles_per_head() const {
        return (G * nodes + kTileRows - 1) / kTileRows;
    }
    __device__ __forceinline__ void enter(int s) {
        seq = s;
        nodes = tree_nodes(a.seqlens, a.tree_lens, s, a.tree, a.max_pages);
        len = a.seqlens[s];
        per_tile = (len + kPage - 1) / kPage + 1;
        tiles = nodes > 0 ? tiles_per_head() * a.Hkv : 0;
    }
    __device__ __forceinline__ int head() const { return tile / tiles_per_head(); }
    __device__ __forceinline__ int row0() const { return tile % tiles_per_head() * kTileRows; }
    // First quarter of the 128 lanes that the tile's rows take.  A tile that does
    // not fill them moves about with the tile's number: a quarter of the lanes
    // belongs to one scheduler, and all four get their share of such tiles.
    __device__ __forceinline__ int quarter() const {
        const int used = (min(G * nodes - row0(), kTileRows) + 31) / 32;
        return (seq + tile) % (5 - used);
    }
    // Steps of the current tile in this share.
    __device__ __forceinline__ int count() const {
        return static_cast<int>(min(left, static_cast<long long>(per_tile - step)));
    }
    __device__ __forceinline__ void next() {
        left -= count();
        step = 0;
        if (++tile == tiles && left > 0) {
            tile = 0;
            do enter(seq + 1); while (tiles == 0);
        }
    }
};

// The copying thread's way through a share: a tile's queries once the tile before
// has formed its last scores, then its steps, each once its stage is free again.
// A wait that runs out ends it.  Every copy has landed on return, whichever way it
// ended: of each barrier, the phase of its last load is waited for.
#pragma nv_exec_check_disable
template <typename Share, typename Port>
__host__ __device__ __forceinline__ void copy_share(Share &share, Port &port) {
    int tiles = 0, it = 0;  // loads so far
    bool ok = true;
    for (; ok && share.left > 0; share.next()) {
        if (tiles > 0 && !(ok = port.queries_free((tiles - 1) & 1))) break;
        port.load_queries(share);
        ++tiles;
        const int n = share.count();
        for (int j = 0; j < n; ++j, ++it) {
            const int st = it % kStagesTc;
            if (it >= kStagesTc && !(ok = port.stage_free(st, (it / kStagesTc - 1) & 1))) break;
            port.load_step(share, j, st);
        }
    }
    if (tiles > 0) port.queries_landed((tiles - 1) & 1);
    for (int j = it > kStagesTc ? it - kStagesTc : 0; j < it; ++j)
        port.step_landed(j % kStagesTc, (j / kStagesTc) & 1);
}

template <int G>
__device__ __forceinline__ long long steps_of(const TreeArgs &a, int seq) {
    const int nodes = tree_nodes(a.seqlens, a.tree_lens, seq, a.tree, a.max_pages);
    if (nodes <= 0) return 0;
    return static_cast<long long>((a.seqlens[seq] + kPage - 1) / kPage + 1) * a.Hkv *
           ((G * nodes + kTileRows - 1) / kTileRows);
}

template <int G>
__global__ void __launch_bounds__(kTcThreads, kTcPerSm)
tree_tc_kernel(const __grid_constant__ CUtensorMap q_map,
               const __grid_constant__ CUtensorMap kv_map,
               const __grid_constant__ CUtensorMap k_map,
               const __grid_constant__ CUtensorMap v_map,
               const TreeArgs a, SharedTile *__restrict__ shared_tiles) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *ring = smem + kQBytes;
    __shared__ __align__(8) uint64_t q_full, q_empty, full[kStagesTc], empty[kStagesTc], s_full,
        p_ready, pv_done, mma_done;
    __shared__ unsigned long long odd_nodes;  // drafted nodes with values that are not finite
    __shared__ uint32_t tmem_base_sh;
    __shared__ long long wide[kTcThreads / 32];
    __shared__ int s_seq;
    __shared__ long long s_offset;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;

    if (threadIdx.x == 0) {
        mbar_init(&q_full, 1);
        mbar_init(&q_empty, 1);
        for (int st = 0; st < kStagesTc; ++st) {
            mbar_init(&full[st], 1);
            mbar_init(&empty[st], 1);
        }
        mbar_init(&s_full, 1);
        mbar_init(&p_ready, 4);
        mbar_init(&pv_done, 1);
        mbar_init(&mma_done, 1);
        odd_nodes = 0;
        fence_barrier_init();
    }
    // This CTA's share: steps cta * share .. of all sequences' steps in a row.
    long long all = 0;
    for (int s = threadIdx.x; s < a.num_seqs; s += kTcThreads) {
        if (cta == 0 && tree_nodes(a.seqlens, a.tree_lens, s, a.tree, a.max_pages) < 0)
            record_error(a.status, POLAR_ERR_BAD_SEQLEN);
        all += steps_of<G>(a, s);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(~0u, all, o);
    if (lane == 0) wide[w] = all;
    __syncthreads();
    all = 0;
    for (int i = 0; i < kTcThreads / 32; ++i) all += wide[i];
    const long long share =
        max((all + gridDim.x - 1) / gridDim.x, static_cast<long long>(kMinShare));
    const long long first = min(cta * share, all), count = min(share, all - first);
    if (count == 0) return;
    long long before = 0;
    for (int s0 = 0; s0 < a.num_seqs; s0 += kTcThreads) {
        const int s = s0 + threadIdx.x;
        const long long mine = s < a.num_seqs ? steps_of<G>(a, s) : 0;
        long long upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(~0u, upto, o);
            if (lane >= o) upto += y;
        }
        __syncthreads();  // `wide` was read
        if (lane == 31) wide[w] = upto;
        __syncthreads();
        for (int i = 0; i < w; ++i) upto += wide[i];
        upto += before;
        if (upto - mine <= first && first < upto) {
            s_seq = s;
            s_offset = first - (upto - mine);
        }
        for (int i = 0; i < kTcThreads / 32; ++i) before += wide[i];
        if (before > first) break;  // uniform
    }
    __syncwarp();  // instructions on tensor memory are for whole warps
    if (w == 5) tmem_alloc_128(&tmem_base_sh);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_sh;
    Walk<G> walk{a};
    walk.left = count;
    walk.enter(s_seq);
    walk.tile = static_cast<int>(s_offset / walk.per_tile);
    walk.step = static_cast<int>(s_offset % walk.per_tile);
    if (threadIdx.x == 0) {
        // The tiles that begin here.
        Walk<G> x = walk;
        long long done = 0;
        for (; x.left > 0; x.next()) {
            if (x.step == 0) {
                const long long end = first + done + x.per_tile;  // the step behind the tile
                const SharedTile t{static_cast<int>((end - 1) / share) - cta + 1, cta,
                                   2 * cta + (done > 0)};
                shared_tiles[(static_cast<size_t>(x.seq) * a.Hkv + x.head()) * a.row_tiles +
                             x.row0() / kTileRows] = t;
            }
            done += x.count();
        }
    }

    int it = 0;     // steps so far, for the barriers' phases
    if (w == 4) {
        // -------------------------------------------- copies (one thread)
        if (lane == 0) {
            tma_prefetch_desc(&q_map);
            tma_prefetch_desc(&kv_map);
            struct Port {
                const CUtensorMap &q_map, &kv_map, &k_map, &v_map;
                const TreeArgs &a;
                uint8_t *smem, *ring;
                uint64_t *q_full, *q_empty, *full, *empty;
                const int32_t *pt;            // the tile's page ids from its first step on
                int npg, g, seq, s0, n, id;   // id: the next step's page

                __device__ __forceinline__ bool queries_free(uint32_t parity) {
                    return mbar_wait(q_empty, parity, a.status);
                }
                __device__ __forceinline__ void load_queries(const Walk<G> &x) {
                    npg = x.per_tile - 1;
                    g = x.head();
                    seq = x.seq;
                    s0 = x.step;
                    n = x.count();
                    pt = a.page_table + static_cast<size_t>(seq) * a.max_pages + s0;
                    id = s0 < npg ? pt[0] : 0;
                    mbar_arrive_expect_tx(q_full, kQBytes);
                    tma_load_3d(smem, &q_map, 0, g * G,
                                seq * a.tree + (x.row0() - 32 * x.quarter()) / G, q_full);
                }
                __device__ __forceinline__ bool stage_free(int st, uint32_t parity) {
                    return mbar_wait(&empty[st], parity, a.status);
                }
                __device__ __forceinline__ void load_step(const Walk<G> &, int j, int st) {
                    int phys = id;
                    id = j + 1 < n && s0 + j + 1 < npg ? pt[j + 1] : 0;
                    // A page id outside the pool is reported; its step reads page
                    // 0 and counts no key.
                    if (phys < 0 || phys >= a.num_pages) {
                        record_error(a.status, POLAR_ERR_BAD_PAGE);
                        phys = 0;
                    }
                    uint8_t *dst = ring + st * kStageBytes;
                    mbar_arrive_expect_tx(&full[st], kStageBytes);
                    if (s0 + j == npg) {
                        tma_load_3d(dst, &k_map, 0, g, seq * a.tree, &full[st]);
                        tma_load_3d(dst + kChunkBytes, &v_map, 0, g, seq * a.tree, &full[st]);
                    } else {
                        const int at = (phys * 2 * a.Hkv + g) * kPage;  // K block of the kv head
                        tma_load_2d(dst, &kv_map, 0, at, &full[st]);
                        tma_load_2d(dst + kChunkBytes, &kv_map, 0, at + a.Hkv * kPage, &full[st]);
                    }
                }
                __device__ __forceinline__ void queries_landed(uint32_t parity) {
                    mbar_wait(q_full, parity, a.status);
                }
                __device__ __forceinline__ void step_landed(int st, uint32_t parity) {
                    mbar_wait(&full[st], parity, a.status);
                }
            };
            Port port{q_map, kv_map, k_map, v_map, a, smem, ring, &q_full, &q_empty, full, empty,
                      nullptr, 0, 0, 0, 0, 0, 0};
            copy_share(walk, port);
        }
        __syncwarp();
    } else if (w == 5) {
        // ---------------------------------------------------------- products
        // The warp goes through the loop as one, so that what the instructions
        // take from its registers is the same in all lanes, and one lane issues: two
        // products of four instructions take 450 clocks to issue (in a branch of one
        // lane 760).
        constexpr uint32_t idesc_qk = idesc_bf16(kTileRows, kPage, false);
        constexpr uint32_t idesc_pv = idesc_bf16(kTileRows, kHeadDim, true);
        // Q and K are K-major (SBO 1024), V is MN-major (one 64-column atom).
        const uint32_t q_lo = sdesc_lo(smem_u32(smem), 16);
        const uint32_t k_lo = sdesc_lo(smem_u32(ring), 16);
        const uint32_t v_lo = sdesc_lo(smem_u32(ring) + kChunkBytes, 8192);
        constexpr uint32_t hi = kSdescHi128B, kStep = kStageBytes >> 4;
        const uint32_t t = __shfl_sync(~0u, tmem, 0), o = t + kColO;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            return __all_sync(~0u, mbar_wait(bar, parity, a.status)) != 0;
        };
        bool ok = true;
        int tiles = 0;
        int st = 0, phase = 0;  // stage and parity of step `it`
        for (; ok && walk.left > 0; walk.next(), ++tiles) {
            const int n = walk.count();
            if (!(ok = wait(&q_full, tiles & 1))) break;
            for (int j = 0; j < n; ++j, ++it) {
                if (!(ok = wait(&full[st], phase))) break;
                // The scores overwrite the weights of the step before.
                if (it > 0 && !(ok = wait(&pv_done, (it - 1) & 1))) break;
                tc_fence_after();
                const uint32_t d = t + kColS, ka = k_lo + st * kStep, va = v_lo + st * kStep;
                if (elect_one()) {
                    mma_ss2<0>(d, q_lo, hi, ka, hi, idesc_qk);
                    mma_ss2<1>(d, q_lo + 2, hi, ka + 2, hi, idesc_qk);
                    mma_ss2<1>(d, q_lo + 4, hi, ka + 4, hi, idesc_qk);
                    mma_ss2<1>(d, q_lo + 6, hi, ka + 6, hi, idesc_qk);
                    tc_commit(&s_full);
                    if (j == n - 1) tc_commit(&q_empty);
                }
                __syncwarp();
                if (!(ok = wait(&p_ready, it & 1))) break;
                tc_fence_after();
                if (elect_one()) {
                    mma_ts2(o, d, va, hi, idesc_pv, j > 0);
                    mma_ts2(o, d + 8, va + 128, hi, idesc_pv, 1u);
                    mma_ts2(o, d + 16, va + 256, hi, idesc_pv, 1u);
                    mma_ts2(o, d + 24, va + 384, hi, idesc_pv, 1u);
                    tc_commit(&pv_done);
                    tc_commit(&empty[st]);
                }
                __syncwarp();
                if (++st == kStagesTc) {
                    st = 0;
                    phase ^= 1;
                }
            }
        }
        // All products complete before tensor memory is freed.
        if (elect_one()) tc_commit(&mma_done);
        __syncwarp();
        wait(&mma_done, 0);
    } else {
        // ------------------------------------------------- softmax warps
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(32 * w) << 16);
        const uint32_t tS = lane_base + kColS, tO = lane_base + kColO;
        bool ok = true;
        int segment = 0;
        for (; ok && walk.left > 0; walk.next(), ++segment) {
            const int npg = walk.per_tile - 1, g = walk.head();
            const int r_tile = static_cast<int>(threadIdx.x) - 32 * walk.quarter();  // may be none
            const int row = walk.row0() + r_tile;
            const int s0 = walk.step, cnt = walk.count(), nodes = walk.nodes, len = walk.len;
            const int R = G * nodes;
            const bool real = r_tile >= 0 && row < R;
            const bool active = __any_sync(~0u, real);  // the warp has a row at all
            const uint64_t drafted = first_tokens(nodes);
            const size_t node0 = static_cast<size_t>(walk.seq) * a.tree;
            const uint64_t seen = real ? a.mask[node0 + row / G] & drafted : 0ull;
            const int n = real ? len + __popcll(seen) : 0;
            const float cl2 = a.ep.s * length_temperature(static_cast<float>(n), a.ep.alpha,
                                                          a.ep.L) * kLog2e;
            const int32_t *pt = a.page_table + static_cast<size_t>(walk.seq) * a.max_pages;
            RowStats x{-INFINITY, -INFINITY, 0.f, 0.f, {0.f, 0.f, 0.f}};
            // Step `it` (`first`: the tile's, O holds nothing yet).  kAll: every row
            // sees all of its keys; else the bits of `mask`.
            auto soft_step = [&](auto kAll, uint64_t mask, bool first) {
                ok = mbar_wait(&s_full, it & 1, a.status);
                if (!__all_sync(~0u, ok)) { ok = false; return; }
                tc_fence_after();
                Moments step;  // where all keys count
                if (active) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t pk[16];
                        TileSums t;
                        while (true) {
                            uint32_t sr[32];
                            tmem_ld32(tS + 32 * h, sr);
                            tmem_wait_ld();
                            const float ref = x.m_ref == -INFINITY ? 0.f : x.m_ref;
                            t = tile_pass<decltype(kAll)::value>(
                                sr, static_cast<uint32_t>(mask >> (32 * h)), cl2, ref, pk);
                            const float zmax = t.top * cl2;
                            const bool need = zmax > x.m_ref + kTcThreshold;
                            if (!__any_sync(~0u, need)) break;
                            // The reference was too low for some row: move it,
                            // rescale what it holds, by a power of two (0 where
                            // nothing was seen before), and form the weights again.
                            const float to = ceilf(zmax);
                            const float r = need ? exp2f(x.m_ref - to) : 1.f;
                            x.l *= r;
                            x.l2 *= r * r;
                            if (need) x.m_ref = to;
                            // (The product before is done: its weights lay where
                            // these scores do.)
                            if (!first) scale_columns(tO, 4, r);
                            if (h > 0) scale_weights(tS, r);
                        }
                        x.m_raw = fmaxf(x.m_raw, t.top);
                        // The squares about the half step's mean: off the sum of
                        // squares where that leaves at least 1/64 of it (at most
                        // six bits lost), else summed again.  (To sum about one of
                        // the scores always took 72 us instead of 69 for 26 nodes,
                        // 248 instead of 239 for 64.)
                        const uint32_t half = static_cast<uint32_t>(mask >> (32 * h));
                        const float k = decltype(kAll)::value ? 32.f
                                                              : static_cast<float>(__popc(half));
                        const float mean = decltype(kAll)::value ? t.s1 * (1.f / 32)
                                                                 : t.s1 / fmaxf(k, 1.f);
                        float m2 = fmaf(-t.s1, mean, t.s2);
                        const bool lost = real && m2 * 64.f < t.s2;
                        if (__any_sync(~0u, lost)) {
                            uint32_t sr[32];
                            tmem_ld32(tS + 32 * h, sr);
                            tmem_wait_ld();
                            const float y = squares_about(sr, half, mean);
                            if (lost) m2 = y;
                        }
                        if (!decltype(kAll)::value) {
                            x.dots.template join<true>(k, mean, m2);
                        } else if (h == 0) {
                            step = Moments{32.f, mean, m2};
                        } else {
                            const float d = mean - step.mean;
                            step = Moments{64.f, fmaf(0.5f, d, step.mean),
                                           fmaf(16.f * d, d, step.m2 + m2)};
                        }
                        x.l += t.l;
                        x.l2 += t.l2;
                        tmem_st16(tS + 16 * h, pk);
                    }
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_ready);
                if (decltype(kAll)::value && active)  // while the product runs
                    x.dots.template join<false>(64.f, step.mean, step.m2);
            };
            for (int j0 = 0; ok && j0 < cnt; j0 += 32) {
                const int p = s0 + j0 + lane;
                const int id = j0 + lane < cnt && p < npg ? pt[p] : 0;
                const uint32_t bad = __ballot_sync(~0u, id < 0 || id >= a.num_pages);
                const int j1 = min(j0 + 32, cnt), full_pages = len / kPage - s0;
                for (int j = j0; ok && j < j1; ++j, ++it) {
                    const bool skip = bad >> (j - j0) & 1u;  // a page outside the pool
                    if (j < full_pages && !skip) {
                        soft_step(std::true_type{}, ~0ull, j == 0);
                        continue;
                    }
                    const bool draft = s0 + j == npg;
                    const uint64_t mask =
                        draft ? seen : skip ? 0ull : first_tokens(len - (s0 + j) * kPage);
                    // Value rows that no row may see are zeroed, since a zero
                    // weight does not silence what is not finite; drafted
                    // values that are not finite are zeroed and added to the
                    // rows that see them at the end.
                    const int st = it % kStagesTc;
                    ok = mbar_wait(&full[st], (it / kStagesTc) & 1, a.status);
                    if (!__all_sync(~0u, ok)) { ok = false; break; }
                    const uint64_t keep = draft ? drafted : mask;
                    uint32_t odd = 0;
#pragma unroll 1
                    for (int e = 0; e < 4; ++e) {
                        const int r = 16 * w + 4 * e + (lane >> 3);
                        uint4 *v = reinterpret_cast<uint4 *>(ring + st * kStageBytes + kChunkBytes +
                                                             r * 128) + (lane & 7);
                        if (!(keep >> r & 1)) {
                            *v = make_uint4(0, 0, 0, 0);
                        } else if (draft) {
                            const uint4 y = *v;
                            uint32_t word[4] = {y.x, y.y, y.z, y.w};
                            bool found = false;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const bool lo = not_finite(word[k]), up = not_finite(word[k] >> 16);
                                found |= lo | up;
                                word[k] = mask_pair(word[k], !lo, !up);
                            }
                            if (found) {
                                *v = make_uint4(word[0], word[1], word[2], word[3]);
                                odd |= 1u << (4 * e + (lane >> 3));
                            }
                        }
                    }
                    if (odd) atomicOr(&odd_nodes, static_cast<unsigned long long>(odd) << (16 * w));
                    fence_proxy_async_smem();
                    __syncwarp();
                    soft_step(std::false_type{}, mask, j == 0);
                }
            }
            if (!ok) break;
            // The tile's last product.
            ok = mbar_wait(&pv_done, (it - 1) & 1, a.status);
            if (!__all_sync(~0u, ok)) { ok = false; break; }
            tc_fence_after();
            if (!active) continue;
            // Drafted values that are not finite, where they count.
            const uint64_t extra = s0 + cnt > npg ? odd_nodes & seen : 0ull;
            const __nv_bfloat16 *vrow = a.v + (node0 * a.Hkv + g) * kHeadDim;
            auto column = [&](int c, uint32_t (&o)[16]) {  // O's columns 16c .. 16c + 15
                __syncwarp();  // lanes that had values to add, or no row to write, come back
                tmem_ld16(tO + 16 * c, o);
                tmem_wait_ld();
                for (uint64_t todo = extra; todo; todo &= todo - 1) {
                    const int j = __ffsll(static_cast<long long>(todo)) - 1;
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float y = __bfloat162float(
                            vrow[static_cast<size_t>(j) * a.Hkv * kHeadDim + 16 * c + e]);
                        if (!(fabsf(y) < INFINITY))
                            o[e] = __float_as_uint(__uint_as_float(o[e]) + y);
                    }
                }
            };
            if (s0 > 0 || s0 + cnt <= npg) {  // a shared tile: its state for the merge
                const size_t slot = 2 * cta + (segment > 0);
                float *part = a.partials + slot * kSlotFloats + r_tile * kPartialFloats;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t o[16];
                    column(c, o);
#pragma unroll
                    for (int e = 0; e < 16; e += 4)
                        *reinterpret_cast<uint4 *>(part + 16 * c + e) =
                            make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                }
                *reinterpret_cast<float4 *>(part + 64) = make_float4(x.m_ref, x.m_raw, x.l, x.l2);
                *reinterpret_cast<float4 *>(part + 68) =
                    make_float4(x.dots.n, x.dots.mean, x.dots.m2, 0.f);
            } else {
                float sq = 0.f, ne = 0.f, mag = 0.f;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t o[16];
                    column(c, o);
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        sq = fmaf(__uint_as_float(o[e]), __uint_as_float(o[e]), sq);
                }
                if (n > 0)
                    mag = row_magnitude(x.l, x.l2, x.m_raw, x.dots, static_cast<float>(n), a.ep,
                                        &ne);
                const float inv = n > 0 ? 1.0f / fmaxf(sqrtf(sq), 1e-30f) : 0.f;
                const int h = g * G + row % G;
                const size_t out_row = (node0 + row / G) * a.Hq + h;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t o[16];
                    column(c, o);
                    if (!real) continue;
                    uint32_t y[8];
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const float2 uu = *reinterpret_cast<const float2 *>(a.u + h * kHeadDim +
                                                                            16 * c + e);
                        const float y0 = fmaf(mag, uu.x, __uint_as_float(o[e]) * inv);
                        const float y1 = fmaf(mag, uu.y, __uint_as_float(o[e + 1]) * inv);
                        y[e >> 1] = n > 0 ? pack_bf16(y0, y1) : 0u;
                    }
                    uint4 *dst = reinterpret_cast<uint4 *>(a.out + out_row * kHeadDim + 16 * c);
                    dst[0] = make_uint4(y[0], y[1], y[2], y[3]);
                    dst[1] = make_uint4(y[4], y[5], y[6], y[7]);
                }
                if (real && a.neff) a.neff[out_row] = ne;
            }
            tc_fence_before();  // O is read before the next tile's first product
        }
    }
    let_next_kernel_start();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (w == 5) tmem_dealloc_128(tmem);
}

// Rows of the tiles that several CTAs share: block (tile, some of its rows).
// A row's parts go to `shares` groups of eight lanes, whose states are then
// joined; the host takes more shares where there are few tiles of many parts, so
// that about as many blocks do the work (1 sequence of 60000 tokens, 48 rows: one
// group of eight lanes per row 94 us in all, this 43).
template <int G>
__global__ void __launch_bounds__(kMergeThreads)
tree_tc_merge_kernel(const TreeArgs a, const SharedTile *__restrict__ shared_tiles, int shares) {
    constexpr int kGroups = kMergeThreads / 8;
    __shared__ __align__(16) float joined[kGroups][kPartialFloats];
    const int tile = blockIdx.x, rt = tile % a.row_tiles, head = tile / a.row_tiles % a.Hkv;
    const int seq = tile / a.row_tiles / a.Hkv, row0 = rt * kTileRows;
    const int nodes = tree_nodes(a.seqlens, a.tree_lens, seq, a.tree, a.max_pages);
    const int per_block = kGroups / shares, r0 = per_block * blockIdx.y;
    const int rows = min(G * nodes - row0, kTileRows);
    wait_for_previous_kernel();
    if (r0 >= rows) return;  // also a tile that no sequence has
    const SharedTile t = shared_tiles[tile];
    if (t.parts == 1) return;
    const int group = threadIdx.x >> 3, share = group / per_block, r = r0 + group % per_block;
    const int row = min(r, rows - 1);
    const int node = (row0 + row) / G, h = head * G + (row0 + row) % G;
    const size_t seq_node = static_cast<size_t>(seq) * a.tree + node;
    const int n = a.seqlens[seq] + __popcll(a.mask[seq_node] & first_tokens(nodes));
    RowState x = merge_parts(share < t.parts ? (t.parts - share + shares - 1) / shares : 0,
                             [&](int k) {
        const int j = shares * k + share;
        const size_t slot = j == 0 ? t.slot : 2 * (t.cta + j);
        return a.partials + slot * kSlotFloats + row * kPartialFloats;
    });
    if (shares > 1) {
        store_part(x, joined[group], true);
        __syncthreads();
        x = merge_parts(shares, [&](int k) { return joined[group % per_block + k * per_block]; });
    }
    finish_row(x, n, a.ep, a.u + h * kHeadDim, a.out + (seq_node * a.Hq + h) * kHeadDim,
               a.neff ? a.neff + seq_node * a.Hq + h : nullptr, share == 0 && r < rows);
}

template <int G>
cudaError_t launch_tc(const CUtensorMap &q, const CUtensorMap &kv, const CUtensorMap &k,
                      const CUtensorMap &v, const TreeArgs &t, int ctas, cudaStream_t stream) {
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
    // The workspace: the tiles' records, then two slots of row states for each CTA.
    const long long tiles = num_tiles(t.num_seqs, t.tree, t.Hq, t.Hkv);
    SharedTile *records = reinterpret_cast<SharedTile *>(t.partials);
    TreeArgs a = t;
    a.partials = t.partials + record_bytes(tiles) / sizeof(float);
    a.row_tiles = (G * t.tree + kTileRows - 1) / kTileRows;
    e = launch_ex(tree_tc_kernel<G>, dim3(ctas), kTcThreads, kSmemTc, 1, false, stream, q, kv, k, v,
                  a, records);
    if (e != cudaSuccess) return e;
    int shares = 1;  // of the parts of a row: four each
    while (shares < kMergeThreads / 8 && shares * 8 * tiles <= ctas) shares *= 2;
    const int rows = std::min(G * t.tree, kTileRows), per_block = kMergeThreads / 8 / shares;
    const dim3 grid(static_cast<unsigned>(tiles), (rows + per_block - 1) / per_block);
    return launch_ex(tree_tc_merge_kernel<G>, grid, kMergeThreads, 0, 1, true, stream, a,
                     static_cast<const SharedTile *>(records), shares);
}

}  // namespace

int tree_tc_ctas(int num_seqs, int max_pages, int tree, int Hq, int Hkv) {
    const long long most = (num_tiles(num_seqs, tree, Hq, Hkv) * (max_pages + 1) + kMinShare - 1) /
                           kMinShare;
    return static_cast<int>(std::min<long long>(148 * kTcPerSm, most));
}

size_t tree_tc_workspace_bytes(int num_seqs, int max_pages, int tree, int Hq, int Hkv) {
    return record_bytes(num_tiles(num_seqs, tree, Hq, Hkv)) +
           static_cast<size_t>(2 * tree_tc_ctas(num_seqs, max_pages, tree, Hq, Hkv)) * kSlotFloats *
               sizeof(float);
}

cudaError_t launch_tree_tc(const CUtensorMap &kv, const CUtensorMap &k, const CUtensorMap &v,
                           const TreeArgs &t, int ctas, cudaStream_t stream) {
    CUtensorMap q;
    const int G = t.Hq / t.Hkv;
    // Query rows as (dim, head, node): a tile is the group's heads of 128 / G nodes.
    const uint64_t dims[3] = {static_cast<uint64_t>(kHeadDim), static_cast<uint64_t>(t.Hq),
                              static_cast<uint64_t>(t.num_seqs) * t.tree};
    const uint64_t strides[2] = {kHeadDim * 2, static_cast<uint64_t>(t.Hq) * kHeadDim * 2};
    const uint32_t box[3] = {kHeadDim, static_cast<uint32_t>(G),
                             static_cast<uint32_t>(kTileRows / G)};
    if (encode_tiled(&q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16 *>(t.q),
                     dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    switch (G) {
        case 1: return launch_tc<1>(q, kv, k, v, t, ctas, stream);
        case 2: return launch_tc<2>(q, kv, k, v, t, ctas, stream);
        case 4: return launch_tc<4>(q, kv, k, v, t, ctas, stream);
        case 8: return launch_tc<8>(q, kv, k, v, t, ctas, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace polar

namespace {

// copy_share()'s port on the host: counts loads and waits; the wait number
// `fail_at` runs out.
struct CountingPort {
    int fail_at, waits = 0, queries = 0, steps[polar::kStagesTc] = {};
    int missed = 0;  // waits at the end that are not for a barrier's last load

    bool wait() { return waits++ != fail_at; }
    bool queries_free(uint32_t) { return wait(); }
    bool stage_free(int, uint32_t) { return wait(); }
    template <typename Share> void load_queries(const Share &) { ++queries; }
    template <typename Share> void load_step(const Share &, int, int st) { ++steps[st]; }
    void queries_landed(uint32_t parity) { landed(queries, parity); }
    void step_landed(int st, uint32_t parity) { landed(steps[st], parity); }
    void landed(int &loads, uint32_t parity) {  // a barrier's loads have parities 0, 1, 0, ..
        if (loads == 0 || ((loads - 1) & 1u) != parity) ++missed;
        loads = 0;
    }
};

struct CountedShare {
    const int *steps;
    int left;  // tiles
    int count() const { return *steps; }
    void next() { ++steps, --left; }
};

}  // namespace

int polar_attn_selftest_tree_copies(const int *steps, int tiles, int fail_at, int *waits) {
    if (!steps || !waits || tiles < 0) return -1;
    for (int i = 0; i < tiles; ++i)
        if (steps[i] < 1) return -1;
    CountedShare share{steps, tiles};
    CountingPort port{fail_at};
    polar::copy_share(share, port);
    *waits = port.waits;
    port.missed += port.queries != 0;
    for (int x : port.steps) port.missed += x != 0;
    return port.missed;
}
