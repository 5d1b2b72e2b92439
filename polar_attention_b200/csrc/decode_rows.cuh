// decode_rows.cuh -- the streaming state of a tile of query rows over cached
// pages, shared by the tree and the page-selecting decode.
//
// A CTA has four computing warps; warp w takes tokens 16w .. 16w+15 of every page that
// the CTA streams, for all of the CTA's rows.  Rows sit in an m16 tile of
// mma.sync m16n8k16 (bf16 in, fp32 accumulate): lane (gq, tq) owns row gq and,
// with two row sets, gq + 8.  Each row keeps the method's state:
// reference max m_ref (log2 units, moved lazily), l, l2 (rescaled by r and
// r^2 when it moves), the raw dots' number, mean, sum of squared deviations and
// max, and the value accumulator.  The S fragments are the P operand of the
// second product.
//
// The null floor takes the spread of a row's raw dots.  Where keys are alike it is
// a small part of their mean, and S2/n - (S1/n)^2 of sums in fp32 loses it (a chain
// of 65536 dots of 0.77: 0.004 instead of 0, which at a scale of 16 is 0.07 of the
// gate).  So deviations are summed about means: each step's own, joined to the
// row's by the number of dots on both sides (Chan, Golub and LeVeque's update), and
// parts of a row about their common mean: nothing large cancels.  Replayed from a
// graph, with the plain sums and with these: 8 nodes of one sequence 9.0 and 9.6 us,
// 32 pages of one long sequence 16.0 and 16.4, 256 of 16 sequences 85.7 and 86.2;
// tcgen05 with 26 nodes 66.4 and 70.3, with 64 nodes 216 and 224.
#pragma once

#include "launch.cuh"
#include "mma_common.cuh"

namespace polar {

struct Moments {  // of n raw dots: mean, sum of squared deviations from it
    float n, mean, m2;

    // Joins k more dots (kMaybeNone: possibly none, then of mean 0).
    template <bool kMaybeNone>
    __device__ __forceinline__ void join(float k, float k_mean, float k_m2) {
        const float all = n + k, d = k_mean - mean;
        const float f = kMaybeNone && k == 0.f ? 0.f : __fdividef(k, all);
        mean = fmaf(d, f, mean);
        m2 += fmaf(d * d, n * f, k_m2);
        n = all;
    }
};

template <int kHR>
struct RowTile {
    uint32_t qa[kHR][4][2];
    float cl2[kHR], m_ref[kHR], m_raw[kHR], l[kHR], l2[kHR];
    Moments dots[kHR];
    float acc[8][4];
    uint32_t pa[kHR][2];  // this page's weights, the A operand of P V

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int hr = 0; hr < kHR; ++hr) {
            m_ref[hr] = m_raw[hr] = -INFINITY;
            l[hr] = l2[hr] = 0.f;
            dots[hr] = Moments{0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
    }

    // Query row of row set hr (null: zero padding) and its exponent scale.
    __device__ __forceinline__ void load_row(int hr, const __nv_bfloat16 *q, int tq, float scale) {
        const uint32_t *qrow = reinterpret_cast<const uint32_t *>(q);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            qa[hr][kk][0] = q ? __ldg(qrow + 8 * kk + tq) : 0u;
            qa[hr][kk][1] = q ? __ldg(qrow + 8 * kk + 4 + tq) : 0u;
        }
        cl2[hr] = scale;
    }

    // Scores of this warp's 16 tokens (key fragments kf: [n-tile][k half]),
    // the streaming statistics and the weights.  bits[hr]: which of the lane's
    // four tokens (2 nt + e) the row sees; kAll: all of them.
    template <bool kAll>
    __device__ __forceinline__ void score(const uint32_t (&kf)[2][2][4],
                                          const uint32_t (&bits)[kHR]) {
        __syncwarp();  // the products, here and in weigh(), are the whole warp's
        float sc[2][4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
            sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
                mma_bf16(sc[nt], qa[0][ks][0], kHR == 2 ? qa[kHR - 1][ks][0] : 0u, qa[0][ks][1],
                         kHR == 2 ? qa[kHR - 1][ks][1] : 0u, kf[nt][ks >> 1][2 * (ks & 1)],
                         kf[nt][ks >> 1][2 * (ks & 1) + 1]);
        }
#pragma unroll
        for (int hr = 0; hr < kHR; ++hr) {
            bool vld[2][2];
            float tmax = -INFINITY, ts1 = 0.f, ts2 = 0.f, seen = 4.f;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    vld[nt][e] = kAll || (bits[hr] >> (2 * nt + e) & 1u);
                    const float x = vld[nt][e] ? sc[nt][2 * hr + e] : 0.f;
                    tmax = fmaxf(tmax, vld[nt][e] ? x : -INFINITY);
                    ts1 += x;
                }
            if (!kAll) seen = static_cast<float>(__popc(bits[hr] & 15u));
            const float mean = kAll ? 0.25f * ts1 : seen > 0.f ? __fdividef(ts1, seen) : 0.f;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float d = vld[nt][e] ? sc[nt][2 * hr + e] - mean : 0.f;
                    ts2 = fmaf(d, d, ts2);
                }
            dots[hr].template join<!kAll>(seen, mean, ts2);
            tmax = fmaxf(tmax, __shfl_xor_sync(0xffffffffu, tmax, 1));
            tmax = fmaxf(tmax, __shfl_xor_sync(0xffffffffu, tmax, 2));
            m_raw[hr] = fmaxf(m_raw[hr], tmax);
            const float zmax = tmax * cl2[hr];
            if (zmax > m_ref[hr] + kRescaleThreshold) {  // uniform over the quad of the row
                const float r = exp2f(m_ref[hr] - zmax);
                l[hr] *= r;
                l2[hr] *= r * r;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    acc[i][2 * hr] *= r;
                    acc[i][2 * hr + 1] *= r;
                }
                m_ref[hr] = zmax;
            }
            float pv[2][2];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float p =
                        vld[nt][e] ? exp2f(fmaf(sc[nt][2 * hr + e], cl2[hr], -m_ref[hr])) : 0.f;
                    pv[nt][e] = p;
                    l[hr] += p;
                    l2[hr] = fmaf(p, p, l2[hr]);
                }
            // bf16 operand of the second product: at most half a step (2^-8
            // relative) per weight, as in the other decode kernels; l and l2
            // sum the unrounded weights.
            pa[hr][0] = pack_bf16x2(pv[0][0], pv[0][1]);
            pa[hr][1] = pack_bf16x2(pv[1][0], pv[1][1]);
        }
        __syncwarp();  // quads whose row moved its reference come back
    }

    // acc += P V for value columns 16i .. 16i+15 (v: transposed fragments).
    __device__ __forceinline__ void weigh(int i, const uint32_t (&v)[4]) {
        mma_bf16(acc[2 * i], pa[0][0], kHR == 2 ? pa[kHR - 1][0] : 0u, pa[0][1],
                 kHR == 2 ? pa[kHR - 1][1] : 0u, v[0], v[1]);
        mma_bf16(acc[2 * i + 1], pa[0][0], kHR == 2 ? pa[kHR - 1][0] : 0u, pa[0][1],
                 kHR == 2 ? pa[kHR - 1][1] : 0u, v[2], v[3]);
    }
};

// The lane's four tokens (2 nt + e) of warp w in a page's 64-bit token mask.
__device__ __forceinline__ uint32_t lane_tokens(uint64_t page_mask, int w, int tq) {
    const uint32_t x = static_cast<uint32_t>(page_mask >> (16 * w + 2 * tq));
    return (x & 3u) | ((x >> 6) & 12u);
}

// Mask of the first n tokens of a page (n >= 1; 64 and more: all).
__device__ __forceinline__ uint64_t first_tokens(int n) {
    return n >= kPage ? ~0ull : (1ull << n) - 1;
}

__device__ __forceinline__ void load_keys(uint32_t kb, int w, int lane, uint32_t (&kf)[2][2][4]) {
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
        const int tok = 16 * w + 8 * nt + (lane & 7);
        ldsm_x4(kb + swz(tok, lane >> 3), kf[nt][0]);
        ldsm_x4(kb + swz(tok, 4 + (lane >> 3)), kf[nt][1]);
    }
}

__device__ __forceinline__ void load_values(uint32_t vb, int w, int lane, int i,
                                            uint32_t (&v)[4]) {
    const int row = 16 * w + 8 * ((lane >> 3) & 1) + (lane & 7);
    ldsm_x4_t(vb + swz(row, 2 * i + (lane >> 4)), v);
}

// Value fragments with the rows of tokens outside `tok4` (the lane's four)
// zeroed, so that no stale value enters the product.
__device__ __forceinline__ void mask_values(uint32_t (&v)[4], uint32_t tok4) {
    v[0] = mask_pair(v[0], tok4 & 1u, tok4 & 2u);
    v[1] = mask_pair(v[1], tok4 & 4u, tok4 & 8u);
    v[2] = mask_pair(v[2], tok4 & 1u, tok4 & 2u);
    v[3] = mask_pair(v[3], tok4 & 4u, tok4 & 8u);
}

// One page over the CTA's rows.  mask: the page's valid tokens (the same for
// every row).
template <int kHR>
__device__ __forceinline__ void page_step(RowTile<kHR> &tile, uint32_t kb, uint32_t vb, int w,
                                          int lane, uint64_t mask) {
    uint32_t kf[2][2][4];
    load_keys(kb, w, lane, kf);
    const bool all = mask == ~0ull;
    const uint32_t tok4 = lane_tokens(mask, w, lane & 3);
    uint32_t bits[kHR];
#pragma unroll
    for (int hr = 0; hr < kHR; ++hr) bits[hr] = tok4;
    if (all)
        tile.template score<true>(kf, bits);
    else
        tile.template score<false>(kf, bits);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t v[4];
        load_values(vb, w, lane, i, v);
        if (!all) mask_values(v, tok4);
        tile.weigh(i, v);
    }
}

// --------------------------------------------------------- page streaming ---

constexpr int kRingStages = 3;       // steps in flight per CTA (16 KB each; four CTAs an SM)
constexpr int kRowWarps = 4;         // warps that compute
constexpr int kRowThreads = 160;     // and one that copies
constexpr int kMaxSteps = 512;       // steps of a CTA: their page ids are held in shared memory

struct PageRing {
    uint64_t full[kRingStages], empty[kRingStages];
    int page[kMaxSteps];  // physical page of each step; -1: skipped
};

__device__ __forceinline__ void init_ring(PageRing &r) {
    for (int st = 0; st < kRingStages; ++st) {
        mbar_init(&r.full[st], 1);
        mbar_init(&r.empty[st], kRowWarps);
    }
    fence_barrier_init();
}

// The copying warp's part: load(kk, stage, barrier) starts the copies of step kk
// (16 KB) or arrives on the barrier without any.  Every copy has landed on
// return, unless a wait ran out.
template <typename Load>
__device__ __forceinline__ void copy_steps(PageRing &r, int np, int *status, Load &&load) {
    int kk = 0;
    for (; kk < np; ++kk) {
        const int st = kk % kRingStages;
        if (kk >= kRingStages && !mbar_wait(&r.empty[st], ((kk / kRingStages) - 1) & 1, status))
            break;
        load(kk, st, &r.full[st]);
    }
    for (int j = max(0, kk - kRingStages); j < kk; ++j)
        mbar_wait(&r.full[j % kRingStages], (j / kRingStages) & 1, status);
}

// A computing warp's part: step(kk, stage) on each step as its copies land.
template <typename Step>
__device__ __forceinline__ void compute_steps(PageRing &r, int np, int lane, int *status,
                                              Step &&step) {
    for (int kk = 0; kk < np; ++kk) {
        const int st = kk % kRingStages;
        if (!__all_sync(~0u, mbar_wait(&r.full[st], (kk / kRingStages) & 1, status))) break;
        step(kk, st);
        __syncwarp();
        if (lane == 0) mbar_arrive(&r.empty[st]);
    }
}

// A row's merged state, spread over eight lanes: lane j of them holds value
// columns 8j .. 8j + 7; the statistics are the same in all.
struct RowState {
    float M, m_raw, l, l2;
    Moments dots;
    float4 o[2];
};

// Exact merge of `count` partial states of a row by eight lanes (four rows a
// warp; all lanes of the warp are here); part(k) is the k-th (kPartialFloats
// layout).  M = -inf: no key seen so far.
template <typename Part>
__device__ __forceinline__ RowState merge_parts(int count, Part &&part) {
    const int j = threadIdx.x & 7;
    RowState x;
    x.M = x.m_raw = -INFINITY;
    x.l = x.l2 = 0.f;
    x.dots = Moments{0.f, 0.f, 0.f};
    x.o[0] = x.o[1] = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
    for (int k = j; k < count; k += 8) {
        const float *p = part(k);
        const float2 dots = *reinterpret_cast<const float2 *>(p + 68);
        x.M = fmaxf(x.M, p[64]);
        x.dots.n += dots.x;
        sum = fmaf(dots.x, dots.y, sum);
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
        x.M = fmaxf(x.M, __shfl_xor_sync(~0u, x.M, o));
        x.dots.n += __shfl_xor_sync(~0u, x.dots.n, o);
        sum += __shfl_xor_sync(~0u, sum, o);
    }
    x.dots.mean = x.dots.n > 0.f ? __fdividef(sum, x.dots.n) : 0.f;
#pragma unroll 4
    for (int k = 0; k < count; ++k) {
        const float *p = part(k);
        const float4 st = *reinterpret_cast<const float4 *>(p + 64);
        const float4 dots = *reinterpret_cast<const float4 *>(p + 68);  // n, mean, m2
        const float4 a = *reinterpret_cast<const float4 *>(p + 8 * j);
        const float4 b = *reinterpret_cast<const float4 *>(p + 8 * j + 4);
        const float r = x.M == -INFINITY ? 0.f : exp2f(st.x - x.M);  // st.x: reference max, log2
        x.l = fmaf(st.z, r, x.l);
        x.l2 = fmaf(st.w, r * r, x.l2);
        x.o[0] = make_float4(fmaf(a.x, r, x.o[0].x), fmaf(a.y, r, x.o[0].y),
                             fmaf(a.z, r, x.o[0].z), fmaf(a.w, r, x.o[0].w));
        x.o[1] = make_float4(fmaf(b.x, r, x.o[1].x), fmaf(b.y, r, x.o[1].y),
                             fmaf(b.z, r, x.o[1].z), fmaf(b.w, r, x.o[1].w));
        const float d = dots.y - x.dots.mean;
        x.dots.m2 += fmaf(dots.x * d, d, dots.z);
        x.m_raw = fmaxf(x.m_raw, st.y);
    }
    return x;
}

__device__ __forceinline__ void store_part(const RowState &x, float *dst, bool real) {
    const int j = threadIdx.x & 7;
    if (!real) return;
    *reinterpret_cast<float4 *>(dst + 8 * j) = x.o[0];
    *reinterpret_cast<float4 *>(dst + 8 * j + 4) = x.o[1];
    if (j == 0) *reinterpret_cast<float4 *>(dst + 64) = make_float4(x.M, x.m_raw, x.l, x.l2);
    if (j == 1)
        *reinterpret_cast<float4 *>(dst + 68) = make_float4(x.dots.n, x.dots.mean, x.dots.m2, 0.f);
}

struct Epilogue {  // the method's constants at a row's end
    float s, alpha, L, beta, inv_ln_L;
};

// The magnitude of a row of n visible keys (n > 0) and its n_eff.  The gate depends
// on how far the largest dot lies above the mean and on the spread alone, so the
// mean is taken off first.
__device__ __forceinline__ float row_magnitude(float l, float l2, float m_raw, const Moments &dots,
                                               float n, const Epilogue &e, float *neff) {
    return polar_magnitude(l, l2, m_raw - dots.mean, 0.f, dots.m2,
                           e.s * length_temperature(n, e.alpha, e.L), n, e.beta, e.inv_ln_L, neff);
}

// out = content + count and n_eff of a row of n visible keys, by eight lanes
// (all lanes of the warp are here; rows that are not `real` are not written).
// A row that sees nothing gives zeros.
__device__ __forceinline__ void finish_row(const RowState &x, int n, const Epilogue &e,
                                           const float *__restrict__ u, __nv_bfloat16 *out,
                                           float *neff_out, bool real) {
    const int j = threadIdx.x & 7;
    float ne = 0.f, mag = 0.f;
    if (n > 0) mag = row_magnitude(x.l, x.l2, x.m_raw, x.dots, static_cast<float>(n), e, &ne);
    float o[8] = {x.o[0].x, x.o[0].y, x.o[0].z, x.o[0].w, x.o[1].x, x.o[1].y, x.o[1].z, x.o[1].w};
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sq = fmaf(o[i], o[i], sq);
#pragma unroll
    for (int k = 1; k < 8; k <<= 1) sq += __shfl_xor_sync(~0u, sq, k);
    if (!real) return;
    const float inv = 1.0f / fmaxf(sqrtf(sq), 1e-30f);
    const float4 ua = *reinterpret_cast<const float4 *>(u + 8 * j);
    const float4 ub = *reinterpret_cast<const float4 *>(u + 8 * j + 4);
    const float uu[8] = {ua.x, ua.y, ua.z, ua.w, ub.x, ub.y, ub.z, ub.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = n > 0 ? fmaf(mag, uu[i], o[i] * inv) : 0.f;
    *reinterpret_cast<uint4 *>(out + 8 * j) =
        make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]),
                   pack_bf16x2(o[6], o[7]));
    if (neff_out && j == 0) *neff_out = ne;
}

// Writes each warp's states of all the CTA's rows to shared memory, one partial
// per (row, warp): parts [rows][4][kPartialFloats].
template <int kHR>
__device__ __forceinline__ void spill_states(RowTile<kHR> &t, float *parts, int w, int lane) {
    const int gq = lane >> 2, tq = lane & 3;
#pragma unroll
    for (int hr = 0; hr < kHR; ++hr) {
        float n = t.dots[hr].n, sum = n * t.dots[hr].mean;
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) {
            t.l[hr] += __shfl_xor_sync(0xffffffffu, t.l[hr], o);
            t.l2[hr] += __shfl_xor_sync(0xffffffffu, t.l2[hr], o);
            n += __shfl_xor_sync(0xffffffffu, n, o);
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            t.m_raw[hr] = fmaxf(t.m_raw[hr], __shfl_xor_sync(0xffffffffu, t.m_raw[hr], o));
        }
        const float mean = n > 0.f ? __fdividef(sum, n) : 0.f, d = t.dots[hr].mean - mean;
        float m2 = fmaf(t.dots[hr].n * d, d, t.dots[hr].m2);
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) m2 += __shfl_xor_sync(0xffffffffu, m2, o);
        float *p = parts + ((8 * hr + gq) * 4 + w) * kPartialFloats;
        if (tq == 0) {
            *reinterpret_cast<float4 *>(p + 64) =
                make_float4(t.m_ref[hr], t.m_raw[hr], t.l[hr], t.l2[hr]);
            *reinterpret_cast<float4 *>(p + 68) = make_float4(n, mean, m2, 0.f);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            *reinterpret_cast<float2 *>(p + 8 * i + 2 * tq) =
                make_float2(t.acc[i][2 * hr], t.acc[i][2 * hr + 1]);
    }
}

// Reduces the rows' states over the CTA's warps and the cluster's CTAs and
// hands each of the first nrows rows to fin(row, real, state) in eight lanes of
// the cluster (lanes past the last row get it with real = false).  parts:
// 5 * kRows partials of shared memory, at the same place in every CTA; all
// threads of the cluster are here.
template <int kHR, typename Final>
__device__ __forceinline__ void reduce_rows(RowTile<kHR> &tile, float *parts, int nrows, int w,
                                            int lane, Final &&fin) {
    constexpr int kRows = 8 * kHR;
    __syncthreads();  // the page ring is free
    if (w < kRowWarps) spill_states(tile, parts, w, lane);
    __syncthreads();
    float *own = parts + kRows * 4 * kPartialFloats;
    const int C = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
    for (int r0 = w < kRowWarps ? 4 * w : nrows; r0 < nrows; r0 += 4 * kRowWarps) {
        const int r = min(r0 + (lane >> 3), nrows - 1);
        const bool real = r0 + (lane >> 3) < nrows;
        const RowState x = merge_parts(
            4, [&](int k) { return parts + (r * 4 + k) * kPartialFloats; });
        if (C == 1)
            fin(r, real, x);
        else
            store_part(x, own + r * kPartialFloats, real);
    }
    if (C == 1) return;
    cluster_sync();
    for (int r0 = w < kRowWarps ? 4 * (w * C + rank) : nrows; r0 < nrows; r0 += 4 * kRowWarps * C) {
        const int r = min(r0 + (lane >> 3), nrows - 1);
        const bool real = r0 + (lane >> 3) < nrows;
        fin(r, real,
            merge_parts(C, [&](int k) { return cluster_map(own + r * kPartialFloats, k); }));
    }
    cluster_sync();  // no CTA leaves while its states are read
}

}  // namespace polar
