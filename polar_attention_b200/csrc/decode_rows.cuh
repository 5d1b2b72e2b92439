// decode_rows.cuh -- the streaming state of a tile of query rows over cached
// pages, shared by the tree and the page-selecting decode.
//
// A CTA has four warps; warp w takes tokens 16w .. 16w+15 of every page that
// the CTA streams, for all of the CTA's rows.  Rows sit in m16 tiles of
// mma.sync m16n8k16 (bf16 in, fp32 accumulate): lane (gq, tq) of a tile owns
// rows gq and, with two row sets, gq + 8.  Each row keeps the method's state:
// reference max m_ref (log2 units, moved lazily), l, l2 (rescaled by r and
// r^2 when it moves), the raw dots' sums S1, S2 and max, and the value
// accumulator.  The S fragments are the P operand of the second product.
#pragma once

#include "mma_common.cuh"

namespace polar {

template <int kHR>
struct RowTile {
    uint32_t qa[kHR][4][2];
    float cl2[kHR], m_ref[kHR], m_raw[kHR], l[kHR], l2[kHR], s1[kHR], s2[kHR];
    float acc[8][4];
    uint32_t pa[kHR][2];  // this page's weights, the A operand of P V

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int hr = 0; hr < kHR; ++hr) {
            m_ref[hr] = m_raw[hr] = -INFINITY;
            l[hr] = l2[hr] = s1[hr] = s2[hr] = 0.f;
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
            float tmax = -INFINITY, ts1 = 0.f, ts2 = 0.f;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    vld[nt][e] = kAll || (bits[hr] >> (2 * nt + e) & 1u);
                    const float x = vld[nt][e] ? sc[nt][2 * hr + e] : 0.f;
                    tmax = fmaxf(tmax, vld[nt][e] ? x : -INFINITY);
                    ts1 += x;
                    ts2 = fmaf(x, x, ts2);
                }
            tmax = fmaxf(tmax, __shfl_xor_sync(0xffffffffu, tmax, 1));
            tmax = fmaxf(tmax, __shfl_xor_sync(0xffffffffu, tmax, 2));
            s1[hr] += ts1;
            s2[hr] += ts2;
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
            // bf16 operand of the second product: half a step (2^-9 relative)
            // per weight, as in the other decode kernels; l and l2 sum the
            // unrounded weights.
            pa[hr][0] = pack_bf16x2(pv[0][0], pv[0][1]);
            pa[hr][1] = pack_bf16x2(pv[1][0], pv[1][1]);
        }
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

// One page over the CTA's tiles.  mask: the page's valid tokens (the same for
// every row).
template <int MT, int kHR>
__device__ __forceinline__ void page_step(RowTile<kHR> (&tile)[MT], uint32_t kb, uint32_t vb, int w,
                                          int lane, uint64_t mask) {
    uint32_t kf[2][2][4];
    load_keys(kb, w, lane, kf);
    const bool all = mask == ~0ull;
    const uint32_t tok4 = lane_tokens(mask, w, lane & 3);
    uint32_t bits[kHR];
#pragma unroll
    for (int hr = 0; hr < kHR; ++hr) bits[hr] = tok4;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        if (all)
            tile[m].template score<true>(kf, bits);
        else
            tile[m].template score<false>(kf, bits);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t v[4];
        load_values(vb, w, lane, i, v);
        if (!all) mask_values(v, tok4);
#pragma unroll
        for (int m = 0; m < MT; ++m) tile[m].weigh(i, v);
    }
}

// Merges the four warps' states exactly (mst: [4][rows][6], macc:
// [4][rows][64], both shared) and writes the partials of the CTA's rows;
// dest(r) is row r's partial, or null.  The caller's threads are all here.
template <int MT, int kHR, typename Dest>
__device__ __forceinline__ void merge_warps(RowTile<kHR> (&tile)[MT],
                                            float (*mst)[8 * kHR * MT][6],
                                            float (*macc)[8 * kHR * MT][kHeadDim], int w, int lane,
                                            Dest &&dest) {
    const int gq = lane >> 2, tq = lane & 3;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int hr = 0; hr < kHR; ++hr) {
            RowTile<kHR> &t = tile[m];
#pragma unroll
            for (int o = 1; o <= 2; o <<= 1) {
                t.l[hr] += __shfl_xor_sync(0xffffffffu, t.l[hr], o);
                t.l2[hr] += __shfl_xor_sync(0xffffffffu, t.l2[hr], o);
                t.s1[hr] += __shfl_xor_sync(0xffffffffu, t.s1[hr], o);
                t.s2[hr] += __shfl_xor_sync(0xffffffffu, t.s2[hr], o);
                t.m_raw[hr] = fmaxf(t.m_raw[hr], __shfl_xor_sync(0xffffffffu, t.m_raw[hr], o));
            }
            const int r = m * 8 * kHR + 8 * hr + gq;
            if (tq == 0) {
                mst[w][r][0] = t.m_ref[hr];
                mst[w][r][1] = t.m_raw[hr];
                mst[w][r][2] = t.l[hr];
                mst[w][r][3] = t.l2[hr];
                mst[w][r][4] = t.s1[hr];
                mst[w][r][5] = t.s2[hr];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                *reinterpret_cast<float2 *>(&macc[w][r][8 * i + 2 * tq]) =
                    make_float2(t.acc[i][2 * hr], t.acc[i][2 * hr + 1]);
        }
    __syncthreads();
    for (int r = w; r < 8 * kHR * MT; r += 4) {
        float *dst = dest(r);
        if (!dst) continue;
        float M = -INFINITY;
#pragma unroll
        for (int k = 0; k < 4; ++k) M = fmaxf(M, mst[k][r][0]);
        float2 o = make_float2(0.f, 0.f);
        float ml = 0.f, ml2 = 0.f, ms1 = 0.f, ms2 = 0.f, mraw = -INFINITY;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float rr = M == -INFINITY ? 0.f : exp2f(mst[k][r][0] - M);
            const float2 x = *reinterpret_cast<const float2 *>(&macc[k][r][2 * lane]);
            o.x = fmaf(x.x, rr, o.x);
            o.y = fmaf(x.y, rr, o.y);
            ml = fmaf(mst[k][r][2], rr, ml);
            ml2 = fmaf(mst[k][r][3], rr * rr, ml2);
            ms1 += mst[k][r][4];
            ms2 += mst[k][r][5];
            mraw = fmaxf(mraw, mst[k][r][1]);
        }
        reinterpret_cast<float2 *>(dst)[lane] = o;
        if (lane == 0) {
            reinterpret_cast<float4 *>(dst + 64)[0] = make_float4(M, mraw, ml, ml2);
            reinterpret_cast<float2 *>(dst + 68)[0] = make_float2(ms1, ms2);
        }
    }
}

// Exact merge of a row's split partials and the epilogue, by one warp (lane
// owns columns 2 lane, 2 lane + 1).  A row that sees nothing gives zeros.
__device__ __forceinline__ void merge_splits(const float *__restrict__ base, int nsplit, int n,
                                             float s, float alpha, float L, float beta,
                                             float inv_ln_L, const float *__restrict__ u, int lane,
                                             __nv_bfloat16 *out, float *neff_out) {
    float M = -INFINITY;
    for (int sp = lane; sp < nsplit; sp += 32) M = fmaxf(M, base[sp * kPartialFloats + 64]);
    M = warp_max(M);
    float l = 0.f, l2 = 0.f, s1 = 0.f, s2 = 0.f, m_raw = -INFINITY, a0 = 0.f, a1 = 0.f;
#pragma unroll 4
    for (int sp = 0; sp < nsplit; ++sp) {
        const float *p = base + static_cast<size_t>(sp) * kPartialFloats;
        const float4 st = *reinterpret_cast<const float4 *>(p + 64);
        const float2 ss = *reinterpret_cast<const float2 *>(p + 68);
        const float2 ac = reinterpret_cast<const float2 *>(p)[lane];
        const float r = M == -INFINITY ? 0.f : exp2f(st.x - M);
        l = fmaf(st.z, r, l);
        l2 = fmaf(st.w, r * r, l2);
        a0 = fmaf(ac.x, r, a0);
        a1 = fmaf(ac.y, r, a1);
        s1 += ss.x;
        s2 += ss.y;
        m_raw = fmaxf(m_raw, st.y);
    }
    float ne = 0.f, mag = 0.f;
    if (n > 0) {
        const float nf = static_cast<float>(n);
        const float c = s * length_temperature(nf, alpha, L);
        mag = polar_magnitude(l, l2, m_raw, s1, s2, c, nf, beta, inv_ln_L, &ne);
    }
    const float nrm = sqrtf(warp_sum(a0 * a0 + a1 * a1));
    const float inv = 1.0f / fmaxf(nrm, 1e-30f);
    const float2 uu = reinterpret_cast<const float2 *>(u)[lane];
    float2 o = make_float2(fmaf(mag, uu.x, a0 * inv), fmaf(mag, uu.y, a1 * inv));
    if (n <= 0) o = make_float2(0.f, 0.f);
    reinterpret_cast<__nv_bfloat162 *>(out)[lane] = __floats2bfloat162_rn(o.x, o.y);
    if (neff_out && lane == 0) *neff_out = ne;
}

}  // namespace polar
