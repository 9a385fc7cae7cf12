// Chunk attention on the fifth-generation tensor cores ("PuzzleKV: Page-Wise
// Low-Rank Decomposition for KV Cache Compression", §3.3 ④, eqs. (4)-(5)).
//
// One pass over the keys in blocks of 128 for 256 query rows at a time: S = Q
// K^T into tensor memory, the online softmax in registers (one row per
// thread), P back into tensor memory as the next product's operand, O += P V.
#include <algorithm>
#include <cfloat>

#include "kernels.h"
#include "rebuild.cuh"
#include "tcgen05.cuh"

namespace pkv {

namespace {

// Three warpgroups.  Launched with 168 registers a thread (384 x 168 = 64,512),
// the two softmax warpgroups, which hold a score row each thread, take 224 and
// the third keeps 56: 2 x 224 + 56 = 3 x 168.
constexpr int FLASH_THREADS = 384;
constexpr int RING = 5;  // key / value images in flight: what is left of shared memory beside two query tiles

// The pieces of one CTA's share of the units, in order.
struct Pieces {
    const FlashParams &p;
    long long left;
    int i, h, pair, b0;
    // the current piece: blocks [cb0, cb1) of cnb; the share's first piece?
    int ci, ch, cpair, cb0, cb1, cnb;
    bool cfirst;
    __device__ __forceinline__ Pieces(const FlashParams &p_, int cta) : p(p_), cfirst(false), cnb(0) {
        const FlashParams::Share &s = p.share[cta];
        left = s.units;
        i = s.i; h = s.h; pair = s.pair; b0 = s.b0;
    }
    __device__ __forceinline__ bool next() {
        if (left <= 0) return false;
        cfirst = cnb == 0;
        ci = i; ch = h; cpair = pair; cb0 = b0;
        cnb = flash_blocks(p.T[i], p.n[i], p.G, pair);
        cb1 = (int)min((long long)cnb, b0 + left);
        left -= cb1 - cb0;
        b0 = 0;
        if ((pair + 1) * FLASH_ROWS < p.n[i] * p.G) {
            ++pair;
        } else {
            pair = 0;
            if (++h == p.H) {
                h = 0;
                ++i;
            }
        }
        return true;
    }
    __device__ __forceinline__ int rows() const { return p.n[ci] * p.G; }
    __device__ __forceinline__ long long image(int b) const {
        const int nblk = p.blk_off[ci + 1] - p.blk_off[ci];
        return (long long)p.blk_off[ci] * p.H + (long long)ch * nblk + b;
    }
};

struct FlashShared {
    uint64_t kv_full[RING], kv_empty[RING], q_full[2], s_full[2], p_full[2], o_full[2];
    uint32_t tmem;
    volatile int failed;
};

// Bounded wait of one role; when it gives up, or another role has, every role leaves.
__device__ __forceinline__ bool role_wait(FlashShared &s, uint64_t *bar, uint32_t parity, const FlashParams &p) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 15) == 0) {
            if (s.failed) return false;
            if (global_ns() - t0 > p.hook.limit()) break;
        }
    }
    s.failed = 1;
    atomicOr(p.status + STATUS_TIMEOUT, 1);
    return false;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// A power of two exponent e with |x| 2^-e in [2^12, 2^13) for the largest
// finite |x| = m (0 for m = 0): fp16 then holds x 2^-e with 11 bits down to
// 2^-27 of m.  2^e and 2^-e stay normal fp32 numbers.
__device__ __forceinline__ int fp16_exponent(float m) {
    if (!(m > 0.f)) return 0;
    const int e = (int)((__float_as_uint(m) >> 23) & 255) - 127 - 12;
    return max(-110, min(e, 115));
}
// The power of a value block: a multiple of four, so that the blocks of a
// sequence mostly share it, with the largest finite |x| = m in [2^11, 2^15): 11
// bits down to 2^-25 of m or less, whatever the size of the values.  A block of
// zeros has none.
constexpr int NO_VALUES = -120;
__device__ __forceinline__ int value_exponent(float m) {
    if (!(m > 0.f)) return NO_VALUES;
    const int e = (int)((__float_as_uint(m) >> 23) & 255) - 127 - 11;
    return max(-108, e & ~3);
}
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
__device__ __forceinline__ float finite_abs(float x) {
    const float a = fabsf(x);
    return a <= 3.4028235e38f ? a : 0.f;  // an infinity or NaN sets no scale
}

}  // namespace

// ---------------------------------------------------------------- operand images

// Item (entry, head, block of 128 positions; keys or values): one image.  A
// factorized page's rows are L_K R_K and (transposed) R_V^T L_V^T, products of
// the stored bf16 factors with fp32 sums (m16n8k16 on the warps: each product
// is tiny and its operands lie as stored); dense rows and the chunk's come as
// they are.  The rows are rounded once, to fp16 scaled by a power of two per
// block: 11 bits against bf16's 8, because a key's rounding moves its score,
// and the scores' errors, unlike the output's rounding, grow with |s|.
// (Rebuilt keys and values in bf16 left 6e-3 of the output's norm at 32K tokens,
// 3.5 times the output's own rounding; fp16 leaves 1.8e-3 there and 1.9e-3 at
// 128K, the bf16 output's own rounding being 1.7e-3.)  The powers follow each
// block's largest element, so ordinary spreads inside a block (columns of unlike
// sizes) lose nothing; a value's power is a multiple of four (value_exponent).
//
// HBM-bound: 47 % of the image bytes are read, all are written.  Every step of
// an item is short and waits on the one before, so CTAs stay and loop over
// items: the next item's factors arrive and the last image leaves while one is
// computed.  32K tokens x 8 heads, ranks 16 and 24: 51 us (3.9 TB/s; 82 us with a
// CTA per block and 8 warps); INT4 records, whose codes are expanded first, take
// about 95 us, keys before RoPE, turned here, 68.
struct StageItem {
    int i, b, T0, T1, fw, h, blk, kv;
    StageItem() = default;
    __device__ __forceinline__ StageItem(const StageParams &p, int item) {
        kv = item & 1;
        int u = item >> 1;
        i = 0;
        while (u >= p.blk_off[i + 1] * p.y.H) ++i;
        const int nblk = p.blk_off[i + 1] - p.blk_off[i];
        u -= p.blk_off[i] * p.y.H;
        h = u / nblk;
        blk = u - h * nblk;
        b = p.seqs[i];
        T0 = p.T[i];
        T1 = T0 + p.n[i];
        fw = p.fw[i];
    }
};

template <int P, int D, bool Q4>
__global__ void __launch_bounds__(STAGE_THREADS, 2) stage_kernel(const StageParams p) {
    extern __shared__ __align__(128) unsigned char sm[];
    __shared__ uint64_t bars[2];
    __shared__ StageItem its[2];
    __shared__ float red[STAGE_THREADS / 32];
    constexpr int NP = FLASH_KEYS / P, IMG = FLASH_KEYS * D * 2;
    const Layout &y = p.y;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int items = 2 * p.blk_off[p.nseq] * y.H;
    const BlockLayout bl(y);
    unsigned char *img = sm;
    if (tid == 0) {
        mbar_init(&bars[0], 1);
        mbar_init(&bars[1], 1);
        fence_barrier_init();
    }
    grid_dependency_wait();  // the launch before may still write pages, or read the images
    __syncthreads();
    auto buffer = [&](int buf) { return sm + IMG + buf * NP * bl.fetch_bytes; };
    auto fetch = [&](int item, int buf) {  // one thread: an item's place and its factors
        const StageItem it = its[buf] = StageItem(p, item);
        BlockPages(y, NP, it.blk * NP, it.fw, it.kv)
            .fetch<Q4>(y, bl, p.factor_pool, p.layer, it.b, it.h, it.kv, buffer(buf), &bars[buf], item == 0 ? p.hook.extra() : 0);
    };
    if (tid == 0 && (int)blockIdx.x < items) fetch(blockIdx.x, 0);
    grid_launch_dependents();  // the attention may be set up
    __syncthreads();
    uint32_t phase = 0;  // bit of each buffer's barrier
    int buf = 0;
    for (int item = blockIdx.x; item < items; item += gridDim.x, buf ^= 1) {
        const int next = item + gridDim.x;
        if (tid == 0 && next < items) fetch(next, buf ^ 1);
        const StageItem it = its[buf];
        const BlockPages bp(y, NP, it.blk * NP, it.fw, it.kv);
        unsigned char *pages = Q4 ? buffer(2) : buffer(buf);
        int bad = 0;
        if (bp.lo > 0 || bp.hi < NP)
            bad = __syncthreads_or(fetch_dense<P, D>(y, bp, p.dense_pool, it.kv ? p.v_new : p.k_new, p.off[it.i], p.layer, it.b,
                                                     it.h, it.kv, it.T0, it.T1, pages, bl.page_bytes));
        if (bp.lo < bp.hi) {
            const bool ok = __syncthreads_and(mbar_wait_bounded(&bars[buf], (phase >> buf) & 1, p.status, p.hook.limit()) ? 1 : 0) != 0;
            if (!ok) {  // let the copies land, then leave the images as they are
                if (tid == 0) {
                    mbar_wait_bounded(&bars[buf], (phase >> buf) & 1, nullptr);
                    if (next < items) {
                        const StageItem nx = its[buf ^ 1];
                        const BlockPages nb(y, NP, nx.blk * NP, nx.fw, nx.kv);
                        if (nb.lo < nb.hi) mbar_wait_bounded(&bars[buf ^ 1], (phase >> (buf ^ 1)) & 1, nullptr);
                    }
                }
                break;
            }
            phase ^= 1u << buf;
            if (Q4) {
                bp.expand(y, bl, it.kv, buffer(buf), pages);
                __syncthreads();
            }
        }
        float acc[8][4];
        // the largest finite |acc| of the CTA; also past the last image's store
        auto block_max = [&](int tiles) {
            float m = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < tiles)
#pragma unroll
                    for (int e = 0; e < 4; ++e) m = fmaxf(m, finite_abs(acc[j][e]));
            m = warp_max(m);
            if (lane == 0) red[warp] = m;
            if (tid == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            __syncthreads();
            m = lane < STAGE_THREADS / 32 ? red[lane] : 0.f;
            return warp_max(m);
        };
        int scale;  // the image's power of two
        if (it.kv == 0) {
            const RowTile<P, D> rt;
            constexpr int KT = RowTile<P, D>::KT;
            rt.template rebuild<Q4>(acc, y, bl, bp, 0, pages, buffer(buf));
            if (y.rope) rt.turn(acc, p.rope_base, p.rope_delta, bp.pg0 + rt.s, it.T1);
            scale = fp16_exponent(block_max(KT));
            const float f = pow2i(-scale);
#pragma unroll
            for (int j = 0; j < KT; ++j)
#pragma unroll
                for (int r2 = 0; r2 < 2; ++r2) {
                    const int r = 16 * rt.w + g + 8 * r2, nt = rt.nt(j);
                    *reinterpret_cast<uint32_t *>(img + (nt / 8) * (FLASH_KEYS * 128) + r * 128 + (((nt & 7) ^ (r & 7)) << 4) + 4 * c) =
                        pack_f16(acc[j][2 * r2] * f, acc[j][2 * r2 + 1] * f);
                }
        } else {
            // transposed; warp: 16 head dimensions, KR positions
            constexpr int KR = D == 128 ? 64 : 32, PK = P < KR ? P : KR, PT = PK / 8;
            const int d0 = 16 * (warp % (D / 16)), key0 = KR * (warp / (D / 16));
#pragma unroll
            for (int j = 0; j < KR / 8; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
#pragma unroll
            for (int s2 = 0; s2 < KR / PK; ++s2) {
                const int s = (key0 + s2 * PK) / P, off = (key0 + s2 * PK) % P;  // page, its first position here
                const uint32_t base = smem_u32(pages + s * bl.page_bytes);
                if (s >= bp.lo && s < bp.hi) {
                    const SwzRows RV(base + bl.vR, d0 + (lane & 15), y.rvp * 2);
                    int k0 = 0;
                    for (; k0 + 16 <= y.rvp; k0 += 16) {
                        uint32_t a0, a1, a2, a3;
                        ldsm_x4(RV(0, k0 / 8 + (lane >> 4)), a0, a1, a2, a3);
#pragma unroll
                        for (int j = 0; j < PT; j += 2) {
                            uint32_t b0, b1, b2, b3;
                            ldsm_x4_t(base + swz_offset(k0 + (lane & 15), 2 * off + 16 * j + 16 * (lane >> 4), P * 2), b0, b1, b2, b3);
                            Ops<Q4>::mma(acc[s2 * PT + j], a0, a1, a2, a3, b0, b1);
                            Ops<Q4>::mma(acc[s2 * PT + j + 1], a0, a1, a2, a3, b2, b3);
                        }
                    }
                    if (k0 < y.rvp) {
                        uint32_t a0, a1;
                        ldsm_x2(RV(0, k0 / 8), a0, a1);
#pragma unroll
                        for (int j = 0; j < PT; j += 2) {
                            uint32_t b0, b1;
                            ldsm_x2_t(base + swz_offset(k0 + (lane & 7), 2 * off + 16 * j + 16 * ((lane >> 3) & 1), P * 2), b0, b1);
                            Ops<Q4>::mma8(acc[s2 * PT + j], a0, a1, b0);
                            Ops<Q4>::mma8(acc[s2 * PT + j + 1], a0, a1, b1);
                        }
                    }
                    if (Q4) {
                        float dim[2];
                        for (int r2 = 0; r2 < 2; ++r2) {
                            const int n = d0 + g + 8 * r2;
                            const float2 f = bp.dim_scales(y, bl, buffer(buf), s, 1, n & ~1);
                            dim[r2] = n & 1 ? f.y : f.x;
                        }
#pragma unroll
                        for (int j = 0; j < PT; ++j) {
                            const float2 f = bp.token_scales(y, bl, buffer(buf), s, off + 8 * j + 2 * c);
#pragma unroll
                            for (int e = 0; e < 4; ++e) acc[s2 * PT + j][e] *= dim[e >> 1] * (e & 1 ? f.y : f.x);
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < PT; j += 2) {
                        uint32_t r0, r1, r2, r3;
                        ldsm_x4_t(base + swz_offset(off + 8 * j + (lane & 7) + 8 * (lane >> 4), 2 * d0 + 16 * ((lane >> 3) & 1), D * 2),
                                  r0, r1, r2, r3);
                        put_pairs(r0, r1, acc[s2 * PT + j]);
                        put_pairs(r2, r3, acc[s2 * PT + j + 1]);
                    }
                }
            }
            scale = value_exponent(block_max(KR / 8));
            const float f = pow2i(-scale);
#pragma unroll
            for (int j = 0; j < KR / 8; ++j)
#pragma unroll
                for (int r2 = 0; r2 < 2; ++r2) {
                    const int r = d0 + g + 8 * r2, key = key0 + 8 * j;
                    *reinterpret_cast<uint32_t *>(img + (key / 64) * (D * 128) + r * 128 + ((((key & 63) >> 3) ^ (r & 7)) << 4) +
                                                  4 * c) = pack_f16(acc[j][2 * r2] * f, acc[j][2 * r2 + 1] * f);
                }
        }
        fence_proxy_async_shared();  // the image is written, the fetch buffer is read
        __syncthreads();
        if (tid == 0) {
            asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(p.images + (size_t)item * IMG),
                         "r"(smem_u32(img)), "r"((uint32_t)IMG)
                         : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            reinterpret_cast<float *>(p.scales)[item] = (float)scale + (!bad ? 0.f : scale < 0 ? -0.25f : 0.25f);
        }
    }
    if (tid == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // the images are written
}

// ---------------------------------------------------------------- attention

// Warps 0-3 and 4-7: the softmax of one 128-row tile each (thread = row); warp
// 8: the matrix products; warp 9: the copies.  Tensor memory: the tiles' S (128
// columns each; P overwrites it as fp16 in the first 64), then their O.
//
// Order of the products: S0(0) S1(0), then per block PV0 S0' PV1 S1', so that
// while one tile's softmax runs, the other tile's two products do.  A commit
// covers every product issued before it: when a tile's S is complete, so is
// its previous P V, and its threads may rescale O.
//
// Bound by the softmax and the products together: a unit of 2 x 128 x 128 takes
// 3,180 cycles, its products 2,048, each tile's softmax 1,550 (exponentials and
// packing 975 of them).  2,048 tokens over 30K, 32 / 8 heads: 670 to 690 us, 1.55
// PFLOP/s, tensor cores active 70 %.  Slower: two threads to a row (the exchange of maxima
// costs what the halves save), a warp per tile for the products (they interleave),
// a share of the exponentials as polynomials (the special-function unit is not the
// bound).
template <int D>
__global__ void __launch_bounds__(FLASH_THREADS, 1) flash_kernel(const FlashParams p) {
    extern __shared__ unsigned char sm_raw[];
    __shared__ FlashShared s;
    constexpr int IMG = FLASH_KEYS * D * 2;  // a key image, a value image, a query tile
    unsigned char *sm = sm_raw + ((1024 - (smem_u32(sm_raw) & 1023)) & 1023);
    unsigned char *Qs = sm, *ring = sm + 2 * IMG;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int k = 0; k < RING; ++k) {
            mbar_init(&s.kv_full[k], 1);
            mbar_init(&s.kv_empty[k], 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&s.q_full[t], 128);
            mbar_init(&s.s_full[t], 1);
            mbar_init(&s.p_full[t], 128);
            mbar_init(&s.o_full[t], 1);
        }
        s.failed = 0;
        fence_barrier_init();
    }
    __syncwarp();  // the allocation is the whole warp's
    if (warp == 0) tmem_alloc(&s.tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_dependency_wait();  // the images are written
    const uint32_t tmem = s.tmem;
    Pieces pc(p, blockIdx.x);

    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        const int t = warp >> 2, w4 = warp & 3, row = 32 * w4 + lane;
        const uint32_t lanes = (uint32_t)(32 * w4) << 16;
        const uint32_t tS = tmem + lanes + 128 * t, tO = tmem + lanes + 256 + 128 * t;
        unsigned char *q_tile = Qs + t * IMG;
        uint32_t s_phase = 0, o_phase = 0;
        while (pc.next()) {
            const int R = pc.rows(), r0 = pc.cpair * FLASH_ROWS + 128 * t;
            if (r0 >= R) continue;
            const int r = r0 + row, i = pc.ci, G = p.G;
            const bool live = r < R;
            const int tok = (live ? r : R - 1) / G, lim = p.T[i] + tok;
            // the query row: fp16, scaled by a power of two of its own
            float qs;
            {
                uint4 v[D / 8];
                const uint4 *src = reinterpret_cast<const uint4 *>(
                    p.q + (((size_t)(p.off[i] + tok) * p.Hq + pc.ch * G + (live ? r % G : 0)) * D) * 2);
                float m = 0.f;
#pragma unroll
                for (int k = 0; k < D / 8; ++k) v[k] = live ? src[k] : make_uint4(0, 0, 0, 0);
                auto each = [&](uint32_t w) {
                    m = fmaxf(m, fmaxf(finite_abs(bf16_lo_to_f32(w)), finite_abs(bf16_hi_to_f32(w))));
                };
#pragma unroll
                for (int k = 0; k < D / 8; ++k) {
                    each(v[k].x);
                    each(v[k].y);
                    each(v[k].z);
                    each(v[k].w);
                }
                const int e = fp16_exponent(m);
                const float f = pow2i(-e);
                qs = pow2i(e) * p.scale_log2;
                auto cv = [&](uint32_t w) { return pack_f16(bf16_lo_to_f32(w) * f, bf16_hi_to_f32(w) * f); };
#pragma unroll
                for (int k = 0; k < D / 8; ++k)
                    *reinterpret_cast<uint4 *>(q_tile + (k / 8) * (128 * 128) + row * 128 + (((k & 7) ^ (row & 7)) << 4)) =
                        make_uint4(cv(v[k].x), cv(v[k].y), cv(v[k].z), cv(v[k].w));
            }
            fence_proxy_async_shared();
            tc_fence_before();  // the previous piece's O has been read
            mbar_arrive(&s.q_full[t]);
            float m = -INFINITY, l = 0.f;
            int E = 0, top = 0;  // O is in units of 2^E; the largest E so far
            const float2 *scales = p.scales + pc.image(0);
            float2 sc = scales[pc.cb0];
            const int full = (p.T[i] + r0 / G + 1) / FLASH_KEYS;  // blocks before it are seen whole by every row of the tile
            bool ok = true;
            for (int blk = pc.cb0; blk < pc.cb1; ++blk) {
                // a positive normal number whatever the operands' sizes: masked scores
                // are minus infinity and others may be zero, times this factor
                const float cf = fminf(fmaxf(qs * pow2i((int)sc.x), FLT_MIN), FLT_MAX);
                const int ev = (int)sc.y;
                if (blk + 1 < pc.cb1) sc = scales[blk + 1];
                // a warp leaves as one: tensor-memory accesses are whole-warp operations
                if (!(ok = __all_sync(0xffffffffu, role_wait(s, &s.s_full[t], s_phase, p)))) break;
                s_phase ^= 1;
                tc_fence_after();
                uint32_t x[4][32];
#pragma unroll
                for (int k = 0; k < 4; ++k) tmem_ld32(tS + 32 * k, x[k]);
                tc_wait_ld();
                if (blk >= full) {
                    const int last = lim - blk * FLASH_KEYS;  // last column this row sees
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (32 * k + e > last) x[k][e] = 0xff800000u;
                }
                float mx;
                {  // eight short chains of three-input maxima
                    float a[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) a[j] = __uint_as_float(x[0][j]);
#pragma unroll
                    for (int e = 8; e < 120; e += 16)
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            a[j] = max3(a[j], __uint_as_float(x[(e + j) / 32][(e + j) & 31]),
                                        __uint_as_float(x[(e + 8 + j) / 32][(e + 8 + j) & 31]));
#pragma unroll
                    for (int j = 0; j < 8; ++j) a[j] = fmaxf(a[j], __uint_as_float(x[3][24 + j]));
                    mx = fmaxf(max3(max3(a[0], a[1], a[2]), a[3], a[4]), max3(a[5], a[6], a[7]));
                }
                mx *= cf;
                // The reference m moves only when a score exceeds it by 2^8, so O is
                // rescaled rarely.  The weights are 2^7 times 2^(s - m), up to 2^15: fp16
                // holds them in full down to 2^-21 of the reference's and to a step
                // of 2^-31 below, so that a long tail still counts.  A value block
                // whose power is above E, or two steps below, rescales O as well,
                // exactly: a block's weights are never more than one step short of
                // their bits.  (A power 2^60 below the largest stays short: O, at
                // most 2^30 T units, must not overflow.)
                float f = 1.f;
                if (blk == pc.cb0) {
                    m = mx;
                    E = top = ev;
                } else {
                    if (mx > m + 8.f) {
                        f = m == -INFINITY ? 1.f : ex2(m - mx);
                        m = mx;
                        l *= f;
                    }
                    const int to = ev > E ? ev : ev < E - 4 && ev != NO_VALUES ? max(ev, min(E, top - 60)) : E;
                    f *= pow2i(max(E - to, -126));
                    E = to;
                    top = max(top, E);
                    if (__any_sync(0xffffffffu, f != 1.f)) {
                        for (int k = 0; k < D / 32; ++k) {
                            uint32_t o[32];
                            tmem_ld32(tO + 32 * k, o);
                            tc_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st32(tO + 32 * k, o);
                        }
                    }
                }
                // 2^up: this block's values in units of O (2^-41 of any weight is zero in fp16)
                const float up = ev == NO_VALUES ? 0.f : (float)max(ev - E, -41);
                const float off = (m == -INFINITY ? 0.f : m) - up - 7.f;
                uint64_t sum[2] = {0, 0};  // pairs of zeros
                const uint64_t cf2 = pair(cf, cf), off2 = pair(-off, -off);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint32_t w[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const uint32_t *xx = &x[2 * k + e / 16][(2 * e) & 31];
                        float p0, p1;
                        unpair(fma2(pair(__uint_as_float(xx[0]), __uint_as_float(xx[1])), cf2, off2), p0, p1);
                        p0 = ex2(p0);
                        p1 = ex2(p1);
                        sum[e & 1] = add2(sum[e & 1], pair(p0, p1));
                        w[e] = pack_f16(p0, p1);
                    }
                    tmem_st32(tS + 32 * k, w);
                }
                float ls, ls1;
                unpair(add2(sum[0], sum[1]), ls, ls1);
                ls += ls1;
                l += up == 0.f ? ls : ls * ex2(-up);
                tc_wait_st();
                tc_fence_before();
                mbar_arrive(&s.p_full[t]);
            }
            if (!ok || !__all_sync(0xffffffffu, role_wait(s, &s.o_full[t], o_phase, p))) break;
            o_phase ^= 1;
            tc_fence_after();
            const float unit = pow2i(E);
            const bool whole = pc.cb0 == 0 && pc.cb1 == pc.cnb;
            const float f = whole ? unit / l : unit;
            float *part = nullptr;
            if (!whole) {
                part = p.partials + ((size_t)(2 * blockIdx.x + (pc.cfirst ? 0 : 1)) * FLASH_ROWS + 128 * t + row) * (D + 4);
                if (live) *reinterpret_cast<float4 *>(part) = make_float4(m, l, 0.f, 0.f);
            }
            char *out = p.out + (((size_t)(p.off[i] + tok) * p.Hq + pc.ch * G + r % G) * D) * 2;
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
                uint32_t o[32];
                __syncwarp();  // the read is the whole warp's, the stores are the live rows'
                tmem_ld32(tO + 32 * k, o);
                tc_wait_ld();
                if (live && whole) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        auto pk = [&](int a) {
                            return pack_bf16(__uint_as_float(o[e + a]) * f, __uint_as_float(o[e + a + 1]) * f);
                        };
                        *reinterpret_cast<uint4 *>(out + (32 * k + e) * 2) = make_uint4(pk(0), pk(2), pk(4), pk(6));
                    }
                } else if (live) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<float4 *>(part + 4 + 32 * k + e) =
                            make_float4(__uint_as_float(o[e]) * f, __uint_as_float(o[e + 1]) * f,
                                        __uint_as_float(o[e + 2]) * f, __uint_as_float(o[e + 3]) * f);
                }
            }
        }
    } else {
        // One instruction for the whole warpgroup, before its warps part.
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 8) {
            // One elected lane issues, but the whole warp runs the loop: addresses
            // and descriptors then stay in uniform registers.  With a single lane
            // in the loop each product took 90-107 cycles to issue against the 64
            // it runs for.
            const uint32_t leader = elect_one();
            const uint64_t dq = tc_desc(smem_u32(Qs)), dr = tc_desc(smem_u32(ring));
            constexpr uint32_t ID_S = tc_idesc_f16(128, FLASH_KEYS), ID_O = tc_idesc_f16(128, D);
            uint32_t x = 0, q_phase[2] = {0, 0}, p_phase[2] = {0, 0};
            bool ok = true;
            auto wait = [&](uint64_t *bar, uint32_t parity) { return __all_sync(0xffffffffu, role_wait(s, bar, parity, p)) != 0; };
            auto full = [&](uint32_t n) { return wait(&s.kv_full[n % RING], (n / RING) & 1); };
            auto scores = [&](int t, uint32_t n) {
                const uint64_t a = dq + t * (IMG >> 4), b = dr + (n % RING) * (IMG >> 4);
                if (leader) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        tc_mma_ss(tmem + 128 * t, a + (k / 4) * (128 * 128 >> 4) + (k % 4) * 2,
                                  b + (k / 4) * (FLASH_KEYS * 128 >> 4) + (k % 4) * 2, ID_S, k > 0);
                    tc_commit(&s.s_full[t]);
                }
                __syncwarp();
            };
            auto values = [&](int t, uint32_t n, bool acc) {
                const uint64_t b = dr + (n % RING) * (IMG >> 4);
                if (leader) {
#pragma unroll
                    for (int k = 0; k < FLASH_KEYS / 16; ++k)
                        tc_mma_ts(tmem + 256 + 128 * t, tmem + 128 * t + 8 * k, b + (k / 4) * (D * 128 >> 4) + (k % 4) * 2, ID_O,
                                  acc || k > 0);
                }
                __syncwarp();
            };
            auto commit = [&](uint64_t *bar) {
                if (leader) tc_commit(bar);
                __syncwarp();
            };
            while (ok && pc.next()) {
                const int tiles = pc.cpair * FLASH_ROWS + 128 < pc.rows() ? 2 : 1, nb = pc.cb1 - pc.cb0;
                for (int t = 0; t < tiles && ok; ++t) {
                    ok = wait(&s.q_full[t], q_phase[t]);
                    q_phase[t] ^= 1;
                }
                ok = ok && full(x);
                if (!ok) break;
                tc_fence_after();
                for (int t = 0; t < tiles; ++t) scores(t, x);
                commit(&s.kv_empty[x % RING]);
                for (int j = 0; j < nb && ok; ++j) {
                    const uint32_t v = x + 1 + 2 * j;
                    const bool more = j + 1 < nb;
                    ok = full(v) && (!more || full(v + 1));
                    for (int t = 0; t < tiles && ok; ++t) {
                        ok = wait(&s.p_full[t], p_phase[t]);
                        if (!ok) break;
                        p_phase[t] ^= 1;
                        tc_fence_after();
                        values(t, v, j > 0);
                        if (more)
                            scores(t, v + 1);
                        else
                            commit(&s.o_full[t]);
                    }
                    commit(&s.kv_empty[v % RING]);
                    if (more) commit(&s.kv_empty[(v + 1) % RING]);
                }
                x += 2 * nb;
            }
            if (!ok)  // products still in flight end before the tensor memory is freed
                for (int k = 0; k < 1000; ++k) __nanosleep(1000);
        } else if (warp == 9 && lane == 0) {
            uint32_t x = 0;
            bool ok = true;
            while (ok && pc.next()) {
                const char *src = p.images + (size_t)pc.image(pc.cb0) * (2 * IMG);
                for (int k = 0; k < 2 * (pc.cb1 - pc.cb0) && ok; ++k, ++x) {
                    ok = role_wait(s, &s.kv_empty[x % RING], ((x / RING) & 1) ^ 1, p);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&s.kv_full[x % RING], IMG + (x == 0 ? p.hook.extra() : 0));
                    bulk_g2s(ring + (x % RING) * IMG, src + (size_t)k * IMG, IMG, &s.kv_full[x % RING]);
                }
            }
            // copies still in flight land before the CTA ends, also where another
            // role gives up after the last of them was started
            for (uint32_t k = x < RING ? 0 : x - RING; k < x; ++k)
                mbar_wait_bounded(&s.kv_full[k % RING], (k / RING) & 1, nullptr);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_free(tmem, 512);
}

// Join the states of the pairs cut between CTAs, eq. (5).  Block (boundary,
// group of 8 rows): the boundary of shares c and c + 1, if it cuts a pair and is
// the first that does; one warp per row, the pieces' o summed in order, the same in
// every launch.
template <int D>
__global__ void __launch_bounds__(256) flash_merge_kernel(const FlashParams p) {
    grid_dependency_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const FlashParams::Share &cut = p.share[blockIdx.x + 1], &before = p.share[blockIdx.x];
    // units from the pair's first on: cut.b0 before the boundary
    if (cut.b0 == 0 || before.units < cut.b0) return;
    const int i = cut.i, h = cut.h, pr = cut.pair;
    const int nb = flash_blocks(p.T[i], p.n[i], p.G, pr);
    const int c0 = blockIdx.x;  // the CTA that begins the pair
    int c1 = c0 + 1;            // and the one that ends it
    for (long long at = cut.b0 + cut.units; at < nb; at += p.share[c1].units) ++c1;
    const int np = c1 - c0 + 1, slot0 = before.units == cut.b0 ? 2 * c0 : 2 * c0 + 1;
    const int R = p.n[i] * p.G;
    constexpr int V = D / 32;
    {
        const int rr = 8 * blockIdx.y + warp, r = pr * FLASH_ROWS + rr;
        if (r >= R) return;
        auto row = [&](int c) { return p.partials + ((size_t)(c == 0 ? slot0 : 2 * (c0 + c)) * FLASH_ROWS + rr) * (D + 4); };
        // the first 32 (m, l) and the first eight o come in one trip to memory
        float2 ml = lane < np ? *reinterpret_cast<const float2 *>(row(lane)) : make_float2(-INFINITY, 0.f);
        float o[8][V];
        auto fetch = [&](int c0) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int e = 0; e < V; ++e) o[j][e] = c0 + j < np ? row(c0 + j)[4 + lane * V + e] : 0.f;
        };
        fetch(0);
        float M = ml.x;
        for (int c = lane + 32; c < np; c += 32) M = fmaxf(M, row(c)[0]);
        M = warp_max(M);
        float L = 0.f, acc[V] = {};
        for (int cb = 0; cb < np; cb += 32) {
            if (cb) ml = cb + lane < np ? *reinterpret_cast<const float2 *>(row(cb + lane)) : make_float2(-INFINITY, 0.f);
            const float f = ex2(ml.x - M);
            L = fmaf(f, ml.y, L);
            for (int c = 0; c < 32 && cb + c < np; c += 8) {
                if (cb + c) fetch(cb + c);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float fj = __shfl_sync(0xffffffffu, f, c + j);
#pragma unroll
                    for (int e = 0; e < V; ++e) acc[e] = fmaf(fj, o[j][e], acc[e]);
                }
            }
        }
        const float il = 1.f / warp_sum(L);
        __nv_bfloat16 *dst = reinterpret_cast<__nv_bfloat16 *>(p.out) +
                             ((size_t)(p.off[i] + r / p.G) * p.Hq + h * p.G + r % p.G) * D;
#pragma unroll
        for (int e = 0; e < V; ++e) dst[lane * V + e] = __float2bfloat16_rn(acc[e] * il);
    }
}

// What nonfinite_kernel needs of FlashParams, whose 9 KB make a launch 3 us longer.
struct NonfiniteParams {
    int H, Hq, G;
    const char *v_new;
    char *out;
    const float2 *scales;
    int T[MAX_CALL_BATCH], n[MAX_CALL_BATCH], off[MAX_CALL_BATCH], blk_off[MAX_CALL_BATCH + 1];
};

// Block (entry, head), a thread to a column: infinities and NaN among the chunk's
// values, left out of the images, into the outputs that see them: the weights
// are positive, so each takes over its column from its token on.  Nearly always
// nothing: the blocks' marks are read and that is all (2 to 8 us of a call; a
// function called by the attention kernel took 4 % of its time, reached or not).
template <int D>
__global__ void __launch_bounds__(D) nonfinite_kernel(const NonfiniteParams p) {
    grid_dependency_wait();
    const int i = blockIdx.x, h = blockIdx.y, c = threadIdx.x, nblk = p.blk_off[i + 1] - p.blk_off[i];
    const float2 *scales = p.scales + (size_t)p.blk_off[i] * p.H + (size_t)h * nblk;
    int bad = 0;
    for (int blk = p.T[i] / FLASH_KEYS + c; blk < nblk; blk += D) bad |= scales[blk].y != truncf(scales[blk].y);
    if (!__syncthreads_or(bad)) return;
    const __nv_bfloat16 *v = reinterpret_cast<const __nv_bfloat16 *>(p.v_new) + ((size_t)p.off[i] * p.H + h) * D + c;
    __nv_bfloat16 *out = reinterpret_cast<__nv_bfloat16 *>(p.out) + ((size_t)p.off[i] * p.Hq + h * p.G) * D + c;
    float seen = 0.f;  // the sum of those up to token t
#pragma unroll 8
    for (int t = 0; t < p.n[i]; ++t) {
        const float x = __bfloat162float(v[(size_t)t * p.H * D]);
        if (!isfinite(x)) seen += x;
        if (seen != 0.f)
            for (int g = 0; g < p.G; ++g) {
                __nv_bfloat16 &o = out[((size_t)t * p.Hq + g) * D];
                o = __float2bfloat16_rn(__bfloat162float(o) + seen);
            }
    }
}

template <int P, int D, bool Q4>
static cudaError_t stage_t(const StageParams &p, int num_sms, cudaStream_t st) {
    const int smem = FLASH_KEYS * D * 2 + (int)BlockLayout(p.y).smem(p.y, FLASH_KEYS / P);  // at most 32 + 2 x 41 KB
    cudaError_t e = allow_smem<stage_kernel<P, D, Q4>>(smem);
    if (e != cudaSuccess) return e;
    const int items = 2 * p.blk_off[p.nseq] * p.y.H, resident = std::min(2, 227 * 1024 / (smem + 1024));
    return launch_dependent(stage_kernel<P, D, Q4>, dim3((unsigned)std::min(items, num_sms * resident)), STAGE_THREADS, smem, st, p);
}

cudaError_t launch_stage(const StageParams &p, int num_sms, cudaStream_t st) {
    if (p.blk_off[p.nseq] == 0) return cudaSuccess;
#define PKV_STAGE_CASE(PP, DD) \
    if (p.y.P == PP && p.y.d == DD) return p.y.q4 ? stage_t<PP, DD, true>(p, num_sms, st) : stage_t<PP, DD, false>(p, num_sms, st);
    PKV_STAGE_CASE(16, 64)
    PKV_STAGE_CASE(32, 64)
    PKV_STAGE_CASE(64, 64)
    PKV_STAGE_CASE(16, 128)
    PKV_STAGE_CASE(32, 128)
    PKV_STAGE_CASE(64, 128)
#undef PKV_STAGE_CASE
    return cudaErrorInvalidValue;
}

template <int D>
static cudaError_t flash_t(const FlashParams &p, cudaStream_t st) {
    constexpr int smem = (2 + RING) * FLASH_KEYS * D * 2 + 1024;
    cudaError_t e = allow_smem<flash_kernel<D>>(smem);
    if (e != cudaSuccess) return e;
    e = launch_dependent(flash_kernel<D>, dim3((unsigned)p.ctas), FLASH_THREADS, smem, st, p);
    if (e == cudaSuccess && p.ctas > 1) {
        int most = 0;
        for (int i = 0; i < p.nseq; ++i) most = std::max(most, std::min(FLASH_ROWS, p.n[i] * p.G));
        e = launch_dependent(flash_merge_kernel<D>, dim3((unsigned)(p.ctas - 1), (unsigned)((most + 7) / 8)), 256, 0, st, p);
    }
    if (e != cudaSuccess) return e;
    NonfiniteParams np;
    np.H = p.H; np.Hq = p.Hq; np.G = p.G;
    np.v_new = p.v_new;
    np.out = p.out;
    np.scales = p.scales;
    for (int i = 0; i <= p.nseq; ++i) np.blk_off[i] = p.blk_off[i];
    for (int i = 0; i < p.nseq; ++i) {
        np.T[i] = p.T[i]; np.n[i] = p.n[i]; np.off[i] = p.off[i];
    }
    return launch_dependent(nonfinite_kernel<D>, dim3((unsigned)p.nseq, (unsigned)p.H), D, 0, st, np);
}

cudaError_t launch_flash(const FlashParams &p, int d, cudaStream_t st) {
    if (p.units == 0) return cudaSuccess;
    return d == 64 ? flash_t<64>(p, st) : flash_t<128>(p, st);
}

}  // namespace pkv
