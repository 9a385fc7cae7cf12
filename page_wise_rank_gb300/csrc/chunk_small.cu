// Chunk attention of a few tokens per sequence ("PuzzleKV: Page-Wise Low-Rank
// Decomposition for KV Cache Compression", §3.3 ④, eqs. (4)-(5)): drafted
// tokens being verified, or single tokens beside longer chunks.
//
// HBM-bound: the pages are read once, as stored, for all query rows of the KV
// head.  A factorized page contributes s = (q R_K^T) L_K^T and o = (p L_V) R_V,
// the small factors contracted first (no page is rebuilt).  Rebuilding pages
// for the tensor-memory kernel (chunk_flash.cu) costs three times their bytes
// and pays only when hundreds of rows share a page.
//
// 6 tokens over 32.7K, 32 / 8 heads, ranks 16 and 24: 23 us, 2.7 TB/s (floor 9.5); the
// SMs' slots take half of the bytes and fill in 4 to 5 us, then each warp has about
// seven pages of dependent products.
//
// The products run as m16n8k16 on 16-row tiles of the queries: they are too
// narrow (ranks of 16 to 24, 16 to 128 rows) to fill a 128-row tensor-memory
// tile, and the intermediates feed the next product from registers.  The
// intermediates (q R_K^T, the weights, and their product with L_V) are split
// into bf16 high parts and residuals, two products on one operand, so that no
// step rounds to fewer than 16 bits; the output is rounded once.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace pkv {

namespace {

constexpr int SMALL_WARPS = 8;
constexpr int SMALL_SLOTS = 16;

struct SmallShared {
    uint64_t full[SMALL_SLOTS], empty[SMALL_SLOTS];
    int failed;
    int bad;  // the chunk's values hold infinities or NaN
};

__device__ __forceinline__ float ex2s(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One warp's running state for its 16 query rows: lane 4g + c holds rows g and
// g + 8, columns 8 t + 2c, + 1 of every tile t.
template <int D>
struct RowState {
    uint32_t q[D / 16][4];
    float o[D / 8][4];
    float m[2], l[2];
};

// Fold the scores of NT token tiles (in units of 1 / scale log2) into the
// state; they become weights.
template <int NT, int D>
__device__ __forceinline__ void fold(RowState<D> &w, float (&s)[NT][4], float scale) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        float mx = -INFINITY;
#pragma unroll
        for (int t = 0; t < NT; ++t) mx = fmaxf(mx, fmaxf(s[t][2 * r], s[t][2 * r + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // The reference moves only when a score exceeds it by 2^8: the weights
        // are split to 16 bits whatever their size, and o is rescaled rarely.
        const float top = mx * scale;
        const bool move = top > w.m[r] + 8.f;
        if (__any_sync(0xffffffffu, move)) {
            const float f = move ? ex2s(w.m[r] - top) : 1.f;
            if (move) w.m[r] = top;
            w.l[r] *= f;
#pragma unroll
            for (int t = 0; t < D / 8; ++t) {
                w.o[t][2 * r] *= f;
                w.o[t][2 * r + 1] *= f;
            }
        }
        const float base = w.m[r] == -INFINITY ? 0.f : w.m[r];
        float ls = 0.f;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                s[t][2 * r + e] = ex2s(fmaf(s[t][2 * r + e], scale, -base));
                ls += s[t][2 * r + e];
            }
        w.l[r] += ls;  // this lane's columns; the quad's sums join at the end
    }
}

// A operand (high parts and residuals) of two adjacent accumulator tiles.
__device__ __forceinline__ void split_tiles(const float *t0, const float *t1, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
    split_bf16(t0[0], t0[1], hi[0], lo[0]);
    split_bf16(t0[2], t0[3], hi[1], lo[1]);
    split_bf16(t1[0], t1[1], hi[2], lo[2]);
    split_bf16(t1[2], t1[3], hi[3], lo[3]);
}

// NT tiles += (hi + lo) b: the high parts' products, then the residuals', so
// that products on one tile are NT apart.
template <int NT>
__device__ __forceinline__ void both(float (*acc)[4], const uint32_t (&hi)[4], const uint32_t (&lo)[4],
                                     const uint32_t (&b)[NT / 2][4]) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
        mma16816(acc[n], hi[0], hi[1], hi[2], hi[3], b[n / 2][2 * (n & 1)], b[n / 2][2 * (n & 1) + 1]);
#pragma unroll
    for (int n = 0; n < NT; ++n)
        mma16816(acc[n], lo[0], lo[1], lo[2], lo[3], b[n / 2][2 * (n & 1)], b[n / 2][2 * (n & 1) + 1]);
}

// A factorized page, eq. (4).
template <int P, int D>
__device__ __forceinline__ void page_unit(RowState<D> &w, const Layout &y, uint32_t rec, float scale, int lane) {
    constexpr int NT = P / 8;
    const int row8 = (lane & 7) + 8 * (lane >> 4), half = (lane >> 3) & 1;
    float s[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
    {
        const uint32_t RK = rec + (uint32_t)y.off_RK;
        const SwzRows LK(rec, row8, y.rkp * 2), LK8(rec, lane & 15, y.rkp * 2);
        int k0 = 0;
#pragma unroll 1
        for (; k0 + 16 <= y.rkp; k0 += 16) {
            float t[4][4];  // even and odd steps apart: shorter chains
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                uint32_t b0, b1, b2, b3;
                ldsm_x4(RK + swz_offset(k0 + row8, 32 * ks + 16 * half, D * 2), b0, b1, b2, b3);
                if (ks < 2) {
                    mma16816_first(t[2 * ks], w.q[ks][0], w.q[ks][1], w.q[ks][2], w.q[ks][3], b0, b1);
                    mma16816_first(t[2 * ks + 1], w.q[ks][0], w.q[ks][1], w.q[ks][2], w.q[ks][3], b2, b3);
                } else {
                    mma16816(t[2 * (ks & 1)], w.q[ks][0], w.q[ks][1], w.q[ks][2], w.q[ks][3], b0, b1);
                    mma16816(t[2 * (ks & 1) + 1], w.q[ks][0], w.q[ks][1], w.q[ks][2], w.q[ks][3], b2, b3);
                }
            }
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                t[0][e] += t[2][e];
                t[1][e] += t[3][e];
            }
            split_tiles(t[0], t[1], hi, lo);
            uint32_t b[NT / 2][4];
#pragma unroll
            for (int n = 0; n < NT / 2; ++n) ldsm_x4(LK(2 * n, k0 / 8 + half), b[n][0], b[n][1], b[n][2], b[n][3]);
            both<NT>(s, hi, lo, b);
        }
        if (k0 < y.rkp) {  // eight ranks left
            float t[2][4] = {};
#pragma unroll
            for (int ks = 0; ks < D / 16; ks += 2) {
                uint32_t b0, b1, b2, b3;
                ldsm_x4(RK + swz_offset(k0 + (lane & 7), 32 * ks + 16 * (lane >> 3), D * 2), b0, b1, b2, b3);
                mma16816(t[0], w.q[ks][0], w.q[ks][1], w.q[ks][2], w.q[ks][3], b0, b1);
                mma16816(t[1], w.q[ks + 1][0], w.q[ks + 1][1], w.q[ks + 1][2], w.q[ks + 1][3], b2, b3);
            }
            uint32_t h0, h1, l0, l1;
            split_bf16(t[0][0] + t[1][0], t[0][1] + t[1][1], h0, l0);
            split_bf16(t[0][2] + t[1][2], t[0][3] + t[1][3], h1, l1);
#pragma unroll
            for (int n = 0; n < NT; n += 2) {
                uint32_t b0, b1;
                ldsm_x2(LK8(n, k0 / 8), b0, b1);
                mma1688(s[n], h0, h1, b0);
                mma1688(s[n + 1], h0, h1, b1);
                mma1688(s[n], l0, l1, b0);
                mma1688(s[n + 1], l0, l1, b1);
            }
        }
    }
    fold<NT, D>(w, s, scale);
    uint32_t ph[P / 16][4], pl[P / 16][4];
#pragma unroll
    for (int k = 0; k < P / 16; ++k) split_tiles(s[2 * k], s[2 * k + 1], ph[k], pl[k]);
    const uint32_t LV = rec + (uint32_t)y.off_LV;
    const SwzRows RV(rec + (uint32_t)y.off_RV, row8, y.rvp * 2), RV8(rec + (uint32_t)y.off_RV, lane, y.rvp * 2);
    int k0 = 0;
#pragma unroll 1
    for (; k0 + 16 <= y.rvp; k0 += 16) {
        float u[4][4];  // weights' high parts and residuals apart
#pragma unroll
        for (int k = 0; k < P / 16; ++k) {
            uint32_t b0, b1, b2, b3;
            ldsm_x4(LV + swz_offset(k0 + row8, 32 * k + 16 * half, P * 2), b0, b1, b2, b3);
            if (k == 0) {
                mma16816_first(u[0], ph[k][0], ph[k][1], ph[k][2], ph[k][3], b0, b1);
                mma16816_first(u[1], ph[k][0], ph[k][1], ph[k][2], ph[k][3], b2, b3);
                mma16816_first(u[2], pl[k][0], pl[k][1], pl[k][2], pl[k][3], b0, b1);
                mma16816_first(u[3], pl[k][0], pl[k][1], pl[k][2], pl[k][3], b2, b3);
                continue;
            }
            mma16816(u[0], ph[k][0], ph[k][1], ph[k][2], ph[k][3], b0, b1);
            mma16816(u[1], ph[k][0], ph[k][1], ph[k][2], ph[k][3], b2, b3);
            mma16816(u[2], pl[k][0], pl[k][1], pl[k][2], pl[k][3], b0, b1);
            mma16816(u[3], pl[k][0], pl[k][1], pl[k][2], pl[k][3], b2, b3);
        }
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            u[0][e] += u[2][e];
            u[1][e] += u[3][e];
        }
        split_tiles(u[0], u[1], hi, lo);
#pragma unroll
        for (int n0 = 0; n0 < D / 8; n0 += 8) {
            uint32_t b[4][4];
#pragma unroll
            for (int n = 0; n < 4; ++n) ldsm_x4(RV(n0 + 2 * n, k0 / 8 + half), b[n][0], b[n][1], b[n][2], b[n][3]);
            both<8>(w.o + n0, hi, lo, b);
        }
    }
    if (k0 < y.rvp) {
        float u[2][4] = {};
#pragma unroll
        for (int k = 0; k < P / 16; ++k) {
            uint32_t b0, b1;
            ldsm_x2(LV + swz_offset(k0 + (lane & 7), 32 * k + 16 * half, P * 2), b0, b1);
            mma16816(u[0], ph[k][0], ph[k][1], ph[k][2], ph[k][3], b0, b1);
            mma16816(u[1], pl[k][0], pl[k][1], pl[k][2], pl[k][3], b0, b1);
        }
        uint32_t h0, h1, l0, l1;
        split_bf16(u[0][0] + u[1][0], u[0][1] + u[1][1], h0, l0);
        split_bf16(u[0][2] + u[1][2], u[0][3] + u[1][3], h1, l1);
#pragma unroll
        for (int n = 0; n < D / 8; n += 4) {
            uint32_t b0, b1, b2, b3;
            ldsm_x4(RV8(n, k0 / 8), b0, b1, b2, b3);
            mma1688(w.o[n], h0, h1, b0);
            mma1688(w.o[n + 1], h0, h1, b1);
            mma1688(w.o[n + 2], h0, h1, b2);
            mma1688(w.o[n + 3], h0, h1, b3);
            mma1688(w.o[n], l0, l1, b0);
            mma1688(w.o[n + 1], l0, l1, b1);
            mma1688(w.o[n + 2], l0, l1, b2);
            mma1688(w.o[n + 3], l0, l1, b3);
        }
    }
}

// UR dense rows at `rows` (keys, then values UR rows further), of which row g
// (g + 8) of the tile sees the first see[0] (see[1]) and `valid` hold anything.
template <int UR, int D>
__device__ __forceinline__ void dense_unit(RowState<D> &w, uint32_t rows, int see0, int see1, int valid, float scale, int lane) {
    constexpr int NT = UR / 8;
    const int c = lane & 3, row8 = (lane & 7) + 8 * (lane >> 4), half = (lane >> 3) & 1;
    float s[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
            uint32_t b0, b1, b2, b3;
            ldsm_x4(rows + swz_offset(8 * n + row8, 32 * ks + 16 * half, D * 2), b0, b1, b2, b3);
            mma16816(s[n], w.q[ks][0], w.q[ks][1], w.q[ks][2], w.q[ks][3], b0, b1);
            mma16816(s[n + 1], w.q[ks][0], w.q[ks][1], w.q[ks][2], w.q[ks][3], b2, b3);
        }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int col = 8 * t + 2 * c + (e & 1);
            if (col >= (e < 2 ? see0 : see1)) s[t][e] = -INFINITY;
        }
    fold<NT, D>(w, s, scale);
    const uint32_t V = rows + UR * D * 2;
#pragma unroll
    for (int k = 0; k < UR / 16; ++k) {
        uint32_t hi[4], lo[4];
        split_tiles(s[2 * k], s[2 * k + 1], hi, lo);
        // rows past `valid` hold old values, whatever they are: read as zero
        auto keep = [&](int t) { return (t < valid ? 0xffffu : 0u) | (t + 1 < valid ? 0xffff0000u : 0u); };
        const uint32_t k0 = keep(16 * k + 2 * c), k1 = keep(16 * k + 8 + 2 * c);
#pragma unroll
        for (int n0 = 0; n0 < D / 8; n0 += 8) {
            uint32_t b[4][4];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                ldsm_x4_t(V + swz_offset(16 * k + (lane & 15), 16 * (n0 + 2 * n) + 16 * (lane >> 4), D * 2), b[n][0], b[n][1],
                          b[n][2], b[n][3]);
                b[n][0] &= k0;
                b[n][1] &= k1;
                b[n][2] &= k0;
                b[n][3] &= k1;
            }
            both<8>(w.o + n0, hi, lo, b);
        }
    }
}

}  // namespace

// Eight warps: RT row tiles (16 rows each) x PG page groups.  A group's warps
// work on the same unit, a factorized page or UR rows of a dense page, each for
// its rows; the groups take the CTA's units in turn and stream them through
// slots of their own, filled by bulk copies that the group's first warp issues
// as soon as all its warps have left the slot.
template <int P, int D>
__global__ void __launch_bounds__(32 * SMALL_WARPS, 1) small_kernel(const SmallParams p) {
    extern __shared__ __align__(128) unsigned char sm[];
    __shared__ SmallShared sh;
    constexpr int UR = P / 2 < 16 ? 16 : P / 2, UP = P / UR;  // rows of a dense unit, units of a page
    constexpr uint32_t HALF = UR * D * 2;                    // its key (or value) bytes
    const Layout &y = p.y;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int h = blockIdx.y;
    int i = 0;
    while ((int)blockIdx.x >= p.boff[i + 1] - (i + 1)) ++i;
    const int sp = (int)blockIdx.x - (p.boff[i] - i), ns = p.ns[i];
    const int G = y.G, n = p.n[i], R = n * G, T = p.T[i], b = p.seqs[i];
    const int tiles = (R + 15) / 16, RT = tiles <= 1 ? 1 : tiles <= 2 ? 2 : tiles <= 4 ? 4 : 8;
    const int PG = min(SMALL_WARPS / RT, p.slots / 2), SPG = p.slots / PG;
    const int rt = warp % RT, pg = warp / RT;
    // the CTA's units: dense sink pages, factorized pages, dense window pages
    const int p0 = p.bounds[p.boff[i] + sp], p1 = p.bounds[p.boff[i] + sp + 1];
    const int n_pages = (T + P - 1) / P, fw = max(p.fw[i], 0), fs = min(y.sink_pages, n_pages);
    auto dense_units = [&](int a, int z) {  // units of the dense pages [a, z)
        return a < z ? UP * (z - a) - (z == n_pages ? UP - (T - (n_pages - 1) * P + UR - 1) / UR : 0) : 0;
    };
    const int a1 = min(p1, fs), f0 = max(p0, fs), f1 = max(f0, min(p1, fw)), w0 = max(f1, max(p0, fs));
    const int uA = dense_units(p0, a1), uF = f1 - f0, uW = w0 < p1 ? dense_units(w0, p1) : 0;
    const int units = uA + uF + uW;
    // unit u: page and, for dense pages, first row in the page (factorized: -1)
    auto unit = [&](int u, int &page, int &row) {
        if (u < uA) {
            page = p0 + u / UP;
            row = u % UP * UR;
        } else if (u < uA + uF) {
            page = f0 + u - uA;
            row = -1;
        } else {
            const int k = u - uA - uF;
            page = w0 + k / UP;
            row = k % UP * UR;
        }
    };
    if (tid == 0) {
        for (int k = 0; k < p.slots; ++k) {
            mbar_init(&sh.full[k], 1);
            mbar_init(&sh.empty[k], RT);
        }
        sh.failed = sh.bad = 0;
        fence_barrier_init();
    }
    grid_dependency_wait();  // the launch before may still write pages or queries
    __syncthreads();
    const int slot0 = pg * SPG;
    const bool active = pg < PG, leader = active && rt == 0 && lane == 0;
    auto slot_of = [&](int k) { return slot0 + k % SPG; };
    const char *records = p.factor_pool + y.record_offset(p.layer, b, h, 0);
    const char *dense = p.dense_pool + y.dense_offset(p.layer, b, 0, h, 0);
    const uint32_t rec_bytes = (uint32_t)y.rec_bytes;
    const size_t slot_bytes = (size_t)y.H * 2 * y.dense_half_bytes;
    // Leader: the group's k-th unit into its slot.
    auto issue = [&](int k) {
        const int u = pg + k * PG;
        if (u >= units) return true;
        const int sl = slot_of(k);
        if (k >= SPG && !mbar_wait_bounded(&sh.empty[sl], (k / SPG - 1) & 1, p.status, p.hook.limit())) return false;
        int page, row;
        unit(u, page, row);
        unsigned char *dst = sm + (size_t)sl * p.unit_bytes;
        const uint32_t extra = u == 0 ? p.hook.extra() : 0;
        if (row < 0) {
            mbar_arrive_expect_tx(&sh.full[sl], rec_bytes + extra);
            bulk_g2s(dst, records + (size_t)page * rec_bytes, rec_bytes, &sh.full[sl]);
        } else {
            const char *src = dense + y.dense_slot(page) * slot_bytes + (size_t)row * D * 2;
            mbar_arrive_expect_tx(&sh.full[sl], 2 * HALF + extra);
            bulk_g2s(dst, src, HALF, &sh.full[sl]);
            bulk_g2s(dst + HALF, src + y.dense_half_bytes, HALF, &sh.full[sl]);
        }
        return true;
    };
    bool ok = true;
    int issued = 0;
    if (leader)
        for (; issued < SPG; ++issued) issue(issued);
    // the chunk's rows, swizzled, zeros past the last: units of UR rows; infinities
    // and NaN among the values wait until the end, since earlier tokens weigh
    // them by zero, which they would turn into NaN
    unsigned char *chunk = sm + (size_t)p.slots * p.unit_bytes;
    const int cu = sp == ns - 1 ? (n + UR - 1) / UR : 0;
    constexpr int CH = D / 8, AHEAD = 8;  // 16-byte chunks of a row; loads in flight
    for (int e0 = tid; e0 < cu * UR * 2 * CH; e0 += AHEAD * 32 * SMALL_WARPS) {
        uint4 v[AHEAD];
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            const int e = e0 + a * 32 * SMALL_WARPS, ch = e % CH, kv = e / CH % 2, t = e / (2 * CH);
            v[a] = make_uint4(0, 0, 0, 0);
            if (t < n) v[a] = reinterpret_cast<const uint4 *>((kv ? p.v_new : p.k_new) + ((size_t)(p.off[i] + t) * y.H + h) * (D * 2))[ch];
        }
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            const int e = e0 + a * 32 * SMALL_WARPS, ch = e % CH, kv = e / CH % 2, t = e / (2 * CH);
            if (kv) {
                int bad = 0;
                v[a] = make_uint4(finite_pair(v[a].x, bad), finite_pair(v[a].y, bad), finite_pair(v[a].z, bad), finite_pair(v[a].w, bad));
                if (bad) sh.bad = 1;
            }
            if (t < cu * UR)
                *reinterpret_cast<uint4 *>(chunk + (size_t)(t / UR) * 2 * HALF + kv * HALF + swz_offset(t % UR, 16 * ch, D * 2)) = v[a];
        }
    }
    // the warp's query rows
    RowState<D> w;
    const int r0 = 16 * rt + g;
#pragma unroll
    for (int a = 0; a < 2; ++a) {
        const int r = r0 + 8 * a, tok = r / G;
        const bool in = active && r < R;
        const uint32_t *src = reinterpret_cast<const uint32_t *>(p.q) +
                              (((size_t)(p.off[i] + (in ? tok : 0)) * y.Hq + h * G + (in ? r - tok * G : 0)) * D) / 2 + c;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            w.q[k][a] = in ? src[8 * k] : 0u;
            w.q[k][2 + a] = in ? src[8 * k + 4] : 0u;
        }
    }
#pragma unroll
    for (int t = 0; t < D / 8; ++t) w.o[t][0] = w.o[t][1] = w.o[t][2] = w.o[t][3] = 0.f;
    w.m[0] = w.m[1] = -INFINITY;
    w.l[0] = w.l[1] = 0.f;
    grid_launch_dependents();  // the merge may be set up
    if (cu) __syncthreads();  // the chunk is in place (the same in every thread)
    if (active) {
        for (int u = pg; u < cu; u += PG)
            dense_unit<UR, D>(w, smem_u32(chunk + (size_t)u * 2 * HALF), r0 / G + 1 - u * UR, (r0 + 8) / G + 1 - u * UR, UR,
                              p.scale_log2, lane);
        for (int k = 0; pg + k * PG < units; ++k) {
            const int sl = slot_of(k);
            // a warp leaves as one
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.full[sl], (k / SPG) & 1, p.status, p.hook.limit())) != 0;
            if (!ok) break;
            // the slot of the unit before is free, or nearly: the next copy goes there
            if (leader && k > 0 && (ok = issue(issued))) ++issued;
            __syncwarp();  // the products below are the whole warp's
            int page, row;
            unit(pg + k * PG, page, row);
            const uint32_t at = smem_u32(sm + (size_t)sl * p.unit_bytes);
            if (row < 0) {
                page_unit<P, D>(w, y, at, p.scale_log2, lane);
            } else {
                const int valid = min(UR, T - page * P - row);
                dense_unit<UR, D>(w, at, valid, valid, valid, p.scale_log2, lane);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.empty[sl]);
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
            if (!ok) break;
        }
        if (!ok) {
            if (leader)  // copies still in flight land before the CTA ends
                for (int k = max(0, issued - SPG); k < issued; ++k)
                    if (pg + k * PG < units) mbar_wait_bounded(&sh.full[slot_of(k)], (k / SPG) & 1, nullptr);
            if (lane == 0) atomicExch(&sh.failed, 1);
        }
    }
    __syncthreads();  // every copy has landed and every slot is read
    if (sh.failed) return;
    // the groups' states side by side, then joined row by row, eq. (5)
    constexpr int S = D + 4;
    float *comb = reinterpret_cast<float *>(sm);
    if (active) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            w.l[r] += __shfl_xor_sync(0xffffffffu, w.l[r], 1);
            w.l[r] += __shfl_xor_sync(0xffffffffu, w.l[r], 2);
            float *row = comb + ((size_t)pg * RT * 16 + r0 + 8 * r) * S;
            if (c == 0) *reinterpret_cast<float2 *>(row) = make_float2(w.m[r], w.l[r]);
#pragma unroll
            for (int t = 0; t < D / 8; ++t)
                *reinterpret_cast<float2 *>(row + 4 + 8 * t + 2 * c) = make_float2(w.o[t][2 * r], w.o[t][2 * r + 1]);
        }
    }
    __syncthreads();
    for (int e = tid; e < R * (D / 4); e += blockDim.x) {
        const int r = e / (D / 4), j = e % (D / 4);
        float M = -INFINITY;
        for (int k = 0; k < PG; ++k) M = fmaxf(M, comb[((size_t)k * RT * 16 + r) * S]);
        float L = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < PG; ++k) {
            const float *row = comb + ((size_t)k * RT * 16 + r) * S;
            const float f = row[0] == -INFINITY ? 0.f : ex2s(row[0] - M);
            const float4 v = *reinterpret_cast<const float4 *>(row + 4 + 4 * j);
            L = fmaf(f, row[1], L);
            o.x = fmaf(f, v.x, o.x);
            o.y = fmaf(f, v.y, o.y);
            o.z = fmaf(f, v.z, o.z);
            o.w = fmaf(f, v.w, o.w);
        }
        if (sh.bad)  // those that the row sees, each into its column (the weights are positive)
            for (int t = 0; t <= r / G; ++t) {
                const uint2 x = *reinterpret_cast<const uint2 *>(p.v_new + (((size_t)(p.off[i] + t) * y.H + h) * D + 4 * j) * 2);
                int bad = 0;
                const uint2 z = make_uint2(finite_pair(x.x, bad), finite_pair(x.y, bad));
                if (!bad) continue;
                if ((x.x ^ z.x) & 0xFFFFu) o.x += bf16_lo_to_f32(x.x);
                if ((x.x ^ z.x) >> 16) o.y += bf16_hi_to_f32(x.x);
                if ((x.y ^ z.y) & 0xFFFFu) o.z += bf16_lo_to_f32(x.y);
                if ((x.y ^ z.y) >> 16) o.w += bf16_hi_to_f32(x.y);
            }
        if (ns == 1) {
            const float il = 1.f / L;
            *reinterpret_cast<uint2 *>(p.out + ((((size_t)(p.off[i] + r / G) * y.Hq + h * G + r % G) * D) + 4 * j) * 2) =
                make_uint2(pack_bf16(o.x * il, o.y * il), pack_bf16(o.z * il, o.w * il));
        } else {
            float *row = p.partials + (size_t)(p.poff[i] + (long long)(h * ns + sp) * R + r) * S;
            if (j == 0) *reinterpret_cast<float4 *>(row) = make_float4(M, L, 0.f, 0.f);
            *reinterpret_cast<float4 *>(row + 4 + 4 * j) = o;
        }
    }
}

static int small_unit_bytes(const Layout &y) {
    const int ur = y.P / 2 < 16 ? 16 : y.P / 2;
    return (int)((std::max(y.rec_bytes, (size_t)ur * y.d * 4) + 127) & ~(size_t)127);
}
// Shared memory: slots, the chunk's rows; the states of eight row tiles reuse it.
static int small_slots(const Layout &y, int most_tokens, int &chunk_bytes) {
    const int ur = y.P / 2 < 16 ? 16 : y.P / 2;
    chunk_bytes = (most_tokens + ur - 1) / ur * ur * y.d * 4;
    const int room = 226 * 1024 - (int)sizeof(SmallShared) - chunk_bytes;
    return std::min(SMALL_SLOTS, room / small_unit_bytes(y));
}

size_t small_smem_bytes(const Layout &y, int most_tokens) {
    int chunk = 0;
    const int slots = small_slots(y, most_tokens, chunk);
    if (slots < 2) return 0;
    return std::max((size_t)slots * small_unit_bytes(y) + chunk, (size_t)SMALL_ROWS * (y.d + 4) * 4);
}

template <int P, int D>
static cudaError_t small_t(const SmallParams &p, size_t smem, cudaStream_t st) {
    cudaError_t e = allow_smem<small_kernel<P, D>>(smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(small_kernel<P, D>, dim3((unsigned)(p.boff[p.nseq] - p.nseq), (unsigned)p.y.H), 32 * SMALL_WARPS, smem,
                            st, p);
}

cudaError_t launch_small(SmallParams &p, cudaStream_t st) {
    if (p.nseq == 0) return cudaSuccess;
    int most = 0;
    for (int i = 0; i < p.nseq; ++i) most = std::max(most, p.n[i]);
    const size_t smem = small_smem_bytes(p.y, most);
    if (smem == 0) return cudaErrorInvalidValue;
    p.slots = small_slots(p.y, most, p.chunk_bytes);
    p.unit_bytes = small_unit_bytes(p.y);
    if (p.y.d == 64) {
        if (p.y.P == 16) return small_t<16, 64>(p, smem, st);
        if (p.y.P == 32) return small_t<32, 64>(p, smem, st);
        return small_t<64, 64>(p, smem, st);
    }
    if (p.y.P == 16) return small_t<16, 128>(p, smem, st);
    if (p.y.P == 32) return small_t<32, 128>(p, smem, st);
    return small_t<64, 128>(p, smem, st);
}

}  // namespace pkv
