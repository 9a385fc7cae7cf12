// Rebuilding the rows of cached pages on the warps' tensor cores (bf16 stores):
// blocks of 128 positions of one KV head, keys or values, as fp32 accumulator
// tiles.  Shared by the kernels that stage operand images and that read rows.
//
// A block's pages lie in shared memory, page s at s * page_bytes: the key (LK,
// RK) or value (LVt, RVt) part of a factorized page's record, as stored, or a
// dense page's rows, swizzled as in the dense pool.  INT4 records arrive in a
// fetch buffer of their own and are expanded from there to the same matrices in
// fp16: codes as they are (exact), only L_K's times their rank's scale, whose
// products need two fp16 (high part and residual) because the scale sits inside
// the contraction.  The other scales multiply the finished rows.
#pragma once
#include "common.cuh"
#include "kernels.h"

namespace pkv {

constexpr int BLOCK = 128;            // positions of a block
constexpr int STAGE_THREADS = 512;    // two warps to 16 positions

// Where a page's matrices lie and how they arrive.
struct BlockLayout {
    uint32_t page_bytes;    // a page's place: its larger factor part, or its dense rows
    uint32_t kR, vR;        // offsets of RK and RVt in it (LK, LVt at 0; INT4: L_K's residuals behind LK)
    uint32_t fetch_bytes;   // INT4: a page's place in the fetch buffer,
    uint32_t scales;        // and the offset of its scale vectors there
    __host__ __device__ explicit BlockLayout(const Layout &y) {
        const uint32_t lk = (uint32_t)(y.P * y.rkp * 2), rk = (uint32_t)(y.rkp * y.d * 2);
        const uint32_t lv = (uint32_t)(y.P * y.rvp * 2), rv = (uint32_t)(y.rvp * y.d * 2);
        kR = y.q4 ? 2 * lk : lk;
        vR = lv;
        const uint32_t kpart = kR + rk, vpart = vR + rv, part = kpart > vpart ? kpart : vpart;
        page_bytes = part > y.dense_half_bytes ? part : (uint32_t)y.dense_half_bytes;
        const uint32_t ks = (uint32_t)y.q_off_V, vs = (uint32_t)(y.q_off_sRK - y.q_off_V);
        scales = ks > vs ? ks : vs;
        fetch_bytes = (scales + (uint32_t)(y.rec_bytes - y.q_off_sRK) + 127) & ~127u;
        if (!y.q4) fetch_bytes = page_bytes;
    }
    // Shared memory for two fetch buffers of `pages` pages (INT4: and the expanded pages).
    __host__ __device__ uint32_t smem(const Layout &y, int pages) const {
        return 2 * pages * fetch_bytes + (y.q4 ? pages * page_bytes : 0);
    }
};

// A block of `pages` pages from page pg0 on: which of them are factorized, and
// where their parts lie.
struct BlockPages {
    int pg0, lo, hi;  // pages [lo, hi) of the block are factorized
    __device__ __forceinline__ BlockPages(const Layout &y, int pages, int pg0_, int fw, int kv) : pg0(pg0_) {
        lo = max(0, min(pages, y.sink_pages - pg0));
        hi = max(0, min(pages, fw - pg0));
        if (hi < lo) hi = lo;
    }
    // One thread: start the copies of the factorized pages' parts (`extra`: bytes expected in vain).
    template <bool Q4>
    __device__ __forceinline__ void fetch(const Layout &y, const BlockLayout &bl, const char *factor_pool, int layer, int b, int h,
                                          int kv, unsigned char *buf, uint64_t *bar, uint32_t extra) const {
        if (lo == hi) return;
        const size_t off = kv ? (Q4 ? y.q_off_V : y.off_LV) : 0;
        const uint32_t part = (uint32_t)((kv ? (Q4 ? y.q_off_sRK : y.rec_bytes) : (Q4 ? y.q_off_V : y.off_LV)) - off);
        const uint32_t tail = Q4 ? (uint32_t)(y.rec_bytes - y.q_off_sRK) : 0;
        mbar_arrive_expect_tx(bar, (uint32_t)(hi - lo) * (part + tail) + extra);
        const char *src = factor_pool + y.record_offset(layer, b, h, pg0 + lo);
        for (int s = lo; s < hi; ++s, src += y.rec_bytes) {
            bulk_g2s(buf + s * bl.fetch_bytes, src + off, part, bar);
            if (Q4) bulk_g2s(buf + s * bl.fetch_bytes + bl.scales, src + y.q_off_sRK, tail, bar);
        }
    }
    // INT4: the factorized pages' matrices from their codes, a warp to a slab of
    // eight registers per lane.  All threads; a barrier follows.
    __device__ __forceinline__ void expand(const Layout &y, const BlockLayout &bl, int kv, const unsigned char *buf,
                                           unsigned char *pages) const {
        const int K1 = kv ? y.P : y.d, r = kv ? y.rvp : y.rkp, N2 = kv ? y.d : y.P;
        const int n1 = q4_operand_regs(K1, r), n = n1 + q4_operand_regs(r, N2), slabs = (n + 7) / 8;
        const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
        // registers of a 16-wide k-step, and their reciprocals (exact for the few hundred registers there are)
        const int step1 = r / 4, step2 = N2 / 4;
        const uint32_t inv1 = (65536 + step1 - 1) / step1, inv2 = (65536 + step2 - 1) / step2;
        // R_K [dim][rank] -> RK[rank][dim], L_V [token][rank] -> LVt[rank][token]
        const SwzRows first((kv ? 0u : bl.kR) + 4 * c, g, K1 * 2);
        // L_K [rank][token] -> LK[token][rank], R_V [rank][dim] -> RVt[dim][rank]
        const SwzRows second((kv ? bl.vR : 0u) + 4 * c, g, r * 2);
        for (int u = threadIdx.x >> 5; u < (hi - lo) * slabs; u += STAGE_THREADS / 32) {
            int s = lo, slab = u;
            for (; slab >= slabs; slab -= slabs) ++s;
            const unsigned char *src = buf + s * bl.fetch_bytes;
            unsigned char *dst = pages + s * bl.page_bytes;
            const uint2 words = *reinterpret_cast<const uint2 *>(src + (slab * 32 + lane) * 8);
            const uint32_t *sLK =
                reinterpret_cast<const uint32_t *>(src + bl.scales + (y.q_off_sLK - y.q_off_sRK)) + c * (r / 8);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int m = 8 * slab + j;
                if (m >= n) break;
                const uint32_t x = q4_reg(j < 4 ? words.x : words.y, j & 3);
                const bool one = m < n1;
                const int k = one ? m : m - n1, ks = (int)((k * (one ? inv1 : inv2)) >> 16), rem = k - ks * (one ? step1 : step2);
                const bool wide = 16 * ks + 16 <= (one ? K1 : r);  // else the last step, eight wide
                const int tile = wide ? rem >> 1 : rem, chunk = 2 * ks + (wide ? rem & 1 : 0);
                if (one) {
                    *reinterpret_cast<uint32_t *>(dst + first(tile, chunk)) = x;
                } else if (kv) {
                    *reinterpret_cast<uint32_t *>(dst + second(tile, chunk)) = x;
                } else {
                    uint32_t hi16, lo16;
                    mul_split_f16(x, sLK[chunk], hi16, lo16);
                    *reinterpret_cast<uint32_t *>(dst + second(tile, chunk)) = hi16;
                    *reinterpret_cast<uint32_t *>(dst + y.P * r * 2 + second(tile, chunk)) = lo16;
                }
            }
        }
    }
    // INT4: scales of page s: s_RK or s_RV of head dimensions dim, dim + 1 (dim even), s_LV of tokens t, t + 1 (t even).
    __device__ __forceinline__ float2 dim_scales(const Layout &y, const BlockLayout &bl, const unsigned char *buf, int s, int kv, int dim) const {
        const unsigned char *at = buf + s * bl.fetch_bytes + bl.scales + (kv ? y.q_off_sRV - y.q_off_sRK : 0);
        return __half22float2(*reinterpret_cast<const __half2 *>(at + 2 * q4_dscale_index(dim)));
    }
    __device__ __forceinline__ float2 token_scales(const Layout &y, const BlockLayout &bl, const unsigned char *buf, int s, int t) const {
        const unsigned char *at = buf + s * bl.fetch_bytes + bl.scales + (y.q_off_sLV - y.q_off_sRK);
        return __half22float2(*reinterpret_cast<const __half2 *>(at + 2 * q4_scale_index(y.P, t)));
    }
};

// The other rows of the block into the buffer: position pos < T0 from the dense
// pool, pos < T1 from row `row0 + pos - T0` of a chunk ([rows][H][D]), zeros past.
// Infinities and NaN in a chunk's values become zeros: earlier tokens weigh them
// by zero, which they would turn into NaN.  Returns whether the thread met any.
// All threads; a barrier follows.
template <int P, int D>
__device__ __forceinline__ int fetch_dense(const Layout &y, const BlockPages &bp, const char *dense_pool, const char *chunk,
                                            int row0, int layer, int b, int h, int kv, int T0, int T1, unsigned char *buf,
                                            uint32_t page_bytes) {
    constexpr int CH = D / 8;  // 16-byte chunks of a row
    constexpr int PER = BLOCK * CH / STAGE_THREADS;
    uint4 v[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int e = threadIdx.x + k * STAGE_THREADS, row = e / CH, ch = e % CH, s = row / P, pos = bp.pg0 * P + row;
        v[k] = make_uint4(0, 0, 0, 0);
        if ((s >= bp.lo && s < bp.hi) || pos >= T1) continue;
        const char *src = pos >= T0 ? chunk + ((size_t)(row0 + pos - T0) * y.H + h) * (D * 2) + 16 * ch
                                    : dense_pool + y.dense_offset(layer, b, y.dense_slot(bp.pg0 + s), h, kv) +
                                          swz_offset(row % P, 16 * ch, D * 2);
        v[k] = *reinterpret_cast<const uint4 *>(src);
    }
    int bad = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int e = threadIdx.x + k * STAGE_THREADS, row = e / CH, ch = e % CH, s = row / P;
        if (s >= bp.lo && s < bp.hi) continue;
        if (kv && bp.pg0 * P + row >= T0)
            v[k] = make_uint4(finite_pair(v[k].x, bad), finite_pair(v[k].y, bad), finite_pair(v[k].z, bad), finite_pair(v[k].w, bad));
        *reinterpret_cast<uint4 *>(buf + s * page_bytes + swz_offset(row % P, 16 * ch, D * 2)) = v[k];
    }
    return bad;
}

// Two accumulator registers pairs from bf16 pairs: of row g, and of row g + 8.
__device__ __forceinline__ void put_pairs(uint32_t r0, uint32_t r1, float *d) {
    d[0] = bf16_lo_to_f32(r0);
    d[1] = bf16_hi_to_f32(r0);
    d[2] = bf16_lo_to_f32(r1);
    d[3] = bf16_hi_to_f32(r1);
}

// Positions 16 w .. 16 w + 15 (w = warp % 8) and half of the columns of a
// block: tile j = columns 8 nt(j) .. + 7.  Column pairs that RoPE turns (i, i +
// D / 2) stay with one lane, in tiles j and j + KT / 2.
template <int P, int D>
struct RowTile {
    static constexpr int KT = D / 16;
    int lane, w, half, s, t0;
    __device__ __forceinline__ RowTile() {
        lane = threadIdx.x & 31;
        const int warp = threadIdx.x >> 5;
        w = warp & 7;
        half = warp >> 3;
        s = 16 * w / P;
        t0 = 16 * w % P;
    }
    __device__ __forceinline__ int nt(int j) const { return j % (KT / 2) + KT / 2 * half + KT * (j / (KT / 2)); }

    // += L R, L row-major (keys: at `base`) or transposed (values), R at `R`.
    template <bool VALUES, bool H16>
    __device__ __forceinline__ void product(float (&acc)[8][4], const Layout &y, uint32_t base, uint32_t R) const {
        const int rp = VALUES ? y.rvp : y.rkp, pitch = rp * 2, half8 = (lane >> 3) & 1, row8 = (lane & 7) + 8 * (lane >> 4);
        const SwzRows rows16(VALUES ? R : base, VALUES ? row8 : t0 + (lane & 15), pitch);  // the matrix of run-time pitch
        const SwzRows rows8(VALUES ? R : base, VALUES ? lane & 15 : t0 + (lane & 15), pitch);
        int k0 = 0;
        for (; k0 + 16 <= rp; k0 += 16) {
            uint32_t a0, a1, a2, a3;
            if (VALUES)
                ldsm_x4_t(base + swz_offset(k0 + row8, 2 * t0 + 16 * half8, P * 2), a0, a1, a2, a3);
            else
                ldsm_x4(rows16(0, k0 / 8 + (lane >> 4)), a0, a1, a2, a3);
#pragma unroll
            for (int j = 0; j < KT; j += 2) {
                uint32_t b0, b1, b2, b3;
                if (VALUES)
                    ldsm_x4(rows16(nt(j), k0 / 8 + half8), b0, b1, b2, b3);
                else
                    ldsm_x4_t(R + swz_offset(k0 + (lane & 15), 16 * nt(j) + 16 * (lane >> 4), D * 2), b0, b1, b2, b3);
                Ops<H16>::mma(acc[j], a0, a1, a2, a3, b0, b1);
                Ops<H16>::mma(acc[j + 1], a0, a1, a2, a3, b2, b3);
            }
        }
        if (k0 < rp) {  // eight ranks left
            uint32_t a0, a1;
            if (VALUES)
                ldsm_x2_t(base + swz_offset(k0 + (lane & 7), 2 * t0 + 16 * half8, P * 2), a0, a1);
            else
                ldsm_x2(rows8(0, k0 / 8), a0, a1);
#pragma unroll
            for (int j = 0; j < KT; j += 2) {
                uint32_t b0, b1;
                if (VALUES)
                    ldsm_x2(rows8(nt(j), k0 / 8), b0, b1);
                else
                    ldsm_x2_t(R + swz_offset(k0 + (lane & 7), 16 * nt(j) + 16 * half8, D * 2), b0, b1);
                Ops<H16>::mma8(acc[j], a0, a1, b0);
                Ops<H16>::mma8(acc[j + 1], a0, a1, b1);
            }
        }
    }
    // The dense page's rows at `base`.
    __device__ __forceinline__ void rows(float (&acc)[8][4], uint32_t base) const {
#pragma unroll
        for (int j = 0; j < KT; j += 2) {
            uint32_t r0, r1, r2, r3;
            ldsm_x4(base + swz_offset(t0 + (lane & 15), 16 * nt(j) + 16 * (lane >> 4), D * 2), r0, r1, r2, r3);
            put_pairs(r0, r1, acc[j]);
            put_pairs(r2, r3, acc[j + 1]);
        }
    }
    // The tile's rows of the block whose pages lie at `pages` (INT4 codes and scales at `fetched`).
    template <bool Q4>
    __device__ __forceinline__ void rebuild(float (&acc)[8][4], const Layout &y, const BlockLayout &bl, const BlockPages &bp, int kv,
                                            const unsigned char *pages, const unsigned char *fetched) const {
#pragma unroll
        for (int j = 0; j < KT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
        const uint32_t base = smem_u32(pages + s * bl.page_bytes);
        if (s < bp.lo || s >= bp.hi) {
            rows(acc, base);
            return;
        }
        if (kv) {
            product<true, Q4>(acc, y, base, base + bl.vR);
        } else {
            product<false, Q4>(acc, y, base, base + bl.kR);
            if (Q4) product<false, Q4>(acc, y, base + (uint32_t)(y.P * y.rkp * 2), base + bl.kR);
        }
        if (Q4) {
            const int g = lane >> 2, c = lane & 3;
            float row[2] = {1.f, 1.f};
            if (kv)
                for (int r2 = 0; r2 < 2; ++r2) {
                    const int t = t0 + g + 8 * r2;
                    const float2 f = bp.token_scales(y, bl, fetched, s, t & ~1);
                    row[r2] = t & 1 ? f.y : f.x;
                }
#pragma unroll
            for (int j = 0; j < KT; ++j) {
                const float2 f = bp.dim_scales(y, bl, fetched, s, kv, 8 * nt(j) + 2 * c);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j][e] *= row[e >> 1] * (e & 1 ? f.y : f.x);
            }
        }
    }
    // Turn keys stored before RoPE by their positions pg P + t0 + row (the page
    // start's angle plus the offset's); rows at positions T1 and past are zeros.
    __device__ __forceinline__ void turn(float (&acc)[8][4], const float2 *rope_base, const float2 *rope_delta, int pg, int T1) const {
        if (pg * P + t0 >= T1) return;  // perhaps past the tables
        const int g = lane >> 2, c = lane & 3;
#pragma unroll
        for (int j = 0; j < KT / 2; ++j) {
            const int i = 8 * nt(j) + 2 * c;  // angles i and i + 1
            const float4 a = *reinterpret_cast<const float4 *>(rope_base + (size_t)pg * (D / 2) + i);
#pragma unroll
            for (int r2 = 0; r2 < 2; ++r2) {
                const float4 o = *reinterpret_cast<const float4 *>(rope_delta + (t0 + g + 8 * r2) * (D / 2) + i);
                auto one = [&](float ax, float ay, float ox, float oy, float &x0, float &x1) {
                    const float cs = ax * ox - ay * oy, sn = ay * ox + ax * oy;
                    const float u0 = x0 * cs - x1 * sn, u1 = x1 * cs + x0 * sn;
                    x0 = u0;
                    x1 = u1;
                };
                one(a.x, a.y, o.x, o.y, acc[j][2 * r2], acc[j + KT / 2][2 * r2]);
                one(a.z, a.w, o.z, o.w, acc[j][2 * r2 + 1], acc[j + KT / 2][2 * r2 + 1]);
            }
        }
    }
};

}  // namespace pkv
