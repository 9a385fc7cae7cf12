// Rebuilding the rows of cached pages on the warps' tensor cores (bf16 stores):
// blocks of 128 positions of one KV head, keys or values, as fp32 accumulator
// tiles.  Shared by the kernels that stage operand images and that read rows.
//
// A block's pages lie in a fetch buffer, page s at s * stage_page_bytes: the
// key (LK, RK) or value (LVt, RVt) part of a factorized page's record, as stored,
// or a dense page's rows, swizzled as in the dense pool.
#pragma once
#include "common.cuh"
#include "kernels.h"

namespace pkv {

constexpr int BLOCK = 128;            // positions of a block
constexpr int STAGE_THREADS = 512;    // two warps to 16 positions

// Bytes of a page's place in a fetch buffer: the larger factor part of a record,
// or the page's dense rows.
__host__ __device__ inline uint32_t stage_page_bytes(const Layout &y) {
    const size_t kpart = y.off_LV, vpart = y.rec_bytes - y.off_LV, part = kpart > vpart ? kpart : vpart;
    return (uint32_t)(part > y.dense_half_bytes ? part : y.dense_half_bytes);
}

// A block of `pages` pages from page pg0 on: which of them are factorized, and
// where their parts lie.
struct BlockPages {
    int pg0, lo, hi;  // pages [lo, hi) of the block are factorized
    uint32_t part;    // bytes of one part
    __device__ __forceinline__ BlockPages(const Layout &y, int pages, int pg0_, int fw, int kv) : pg0(pg0_) {
        lo = max(0, min(pages, y.sink_pages - pg0));
        hi = max(0, min(pages, fw - pg0));
        if (hi < lo) hi = lo;
        part = (uint32_t)(kv ? y.rec_bytes - y.off_LV : y.off_LV);
    }
    // One thread: start the copies of the factorized pages' parts.
    __device__ __forceinline__ void fetch(const Layout &y, const char *factor_pool, int layer, int b, int h, int kv,
                                          unsigned char *buf, uint32_t page_bytes, uint64_t *bar) const {
        if (lo == hi) return;
        mbar_arrive_expect_tx(bar, (uint32_t)(hi - lo) * part);
        const char *src = factor_pool + y.record_offset(layer, b, h, pg0 + lo) + (kv ? y.off_LV : 0);
        for (int s = lo; s < hi; ++s, src += y.rec_bytes) bulk_g2s(buf + s * page_bytes, src, part, bar);
    }
};

// The other rows of the block into the buffer: position pos < T0 from the dense
// pool, pos < T1 from row `row0 + pos - T0` of a chunk ([rows][H][D]), zeros past.
// All threads; a barrier follows.
template <int P, int D>
__device__ __forceinline__ void fetch_dense(const Layout &y, const BlockPages &bp, const char *dense_pool, const char *chunk,
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
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int e = threadIdx.x + k * STAGE_THREADS, row = e / CH, ch = e % CH, s = row / P;
        if (s >= bp.lo && s < bp.hi) continue;
        *reinterpret_cast<uint4 *>(buf + s * page_bytes + swz_offset(row % P, 16 * ch, D * 2)) = v[k];
    }
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

    // L R of the page at `base`, L row-major (keys) or transposed with the
    // values' operand order.
    template <bool VALUES>
    __device__ __forceinline__ void product(float (&acc)[8][4], const Layout &y, uint32_t base) const {
        const int rp = VALUES ? y.rvp : y.rkp, pitch = rp * 2, half8 = (lane >> 3) & 1, row8 = (lane & 7) + 8 * (lane >> 4);
        const uint32_t R = base + (uint32_t)(VALUES ? y.off_RV - y.off_LV : y.off_RK);
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
                mma16816(acc[j], a0, a1, a2, a3, b0, b1);
                mma16816(acc[j + 1], a0, a1, a2, a3, b2, b3);
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
                mma1688(acc[j], a0, a1, b0);
                mma1688(acc[j + 1], a0, a1, b1);
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
    // Turn keys stored before RoPE by their positions pg P + t0 + row (the page
    // start's angle plus the offset's); rows at positions T1 and past are zeros.
    __device__ __forceinline__ void turn(float (&acc)[8][4], const float2 *rope_base, const float2 *rope_delta, int pg, int T1) const {
        const int g = lane >> 2, c = lane & 3;
#pragma unroll
        for (int r2 = 0; r2 < 2; ++r2) {
            const int t = t0 + g + 8 * r2;
            if (pg * P + t >= T1) continue;
#pragma unroll
            for (int j = 0; j < KT / 2; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = 8 * nt(j) + 2 * c + e;
                    const float2 a = rope_base[(size_t)pg * (D / 2) + i], o = rope_delta[t * (D / 2) + i];
                    const float cs = a.x * o.x - a.y * o.y, sn = a.y * o.x + a.x * o.y;
                    float &x0 = acc[j][2 * r2 + e], &x1 = acc[j + KT / 2][2 * r2 + e];
                    const float u0 = x0 * cs - x1 * sn, u1 = x1 * cs + x0 * sn;
                    x0 = u0;
                    x1 = u1;
                }
        }
    }
};

}  // namespace pkv
