// Rows in and out of the paged cache: reading rows as attention sees them,
// appending a chunk of tokens, and placing plain factors in a store's records
// ("PuzzleKV: Page-Wise Low-Rank Decomposition for KV Cache Compression",
// §3.3 ③-⑤).  Page kinds follow page_kind() in layout.h.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "rebuild.cuh"

namespace pkv {

// Block (page of a call entry, head, K/V): the page's rows inside the entry's
// range, a thread to 16 bytes of a row.  fp32 factorized pages are rebuilt as L
// R in fp32; bf16 calls take dense and chunk rows only (read_kernel rebuilds).
template <typename T>
__global__ void __launch_bounds__(256) rows_kernel(const RowsParams p) {
    extern __shared__ __align__(128) unsigned char sm[];
    constexpr int VE = 16 / sizeof(T);  // elements of a thread
    const Layout &y = p.y;
    const int P = y.P, d = y.d, h = blockIdx.y, kv = blockIdx.z;
    int i = 0;
    while ((int)blockIdx.x >= p.page_off[i + 1]) ++i;
    const int lo = p.lo[i], hi = lo + p.n[i], T0 = p.T[i], b = p.seqs[i];
    const int pg = lo / P + (int)blockIdx.x - p.page_off[i];
    const int r0 = max(lo, pg * P), r1 = min(hi, pg * P + P);
    const bool factored = pg * P < T0 && page_kind(pg, T0, P, y.sink_tokens, y.W) == KIND_FACTORED;
    const int rp = kv == 0 ? y.rkp : y.rvp;
    float *Ls = reinterpret_cast<float *>(sm), *Rs = Ls + P * rp;  // L [P][rp], R [rp][d]
    if constexpr (sizeof(T) == 4) {
        if (factored) {
            const char *rec = p.factor_pool + y.record_offset(p.layer, b, h, pg);
            for (int e = threadIdx.x; e < P * rp; e += blockDim.x)
                Ls[e] = kv == 0 ? *swz_ptr<float>(rec, e / rp, e % rp, rp) : *swz_ptr<float>(rec + y.off_LV, e % rp, e / rp, P);
            for (int e = threadIdx.x; e < rp * d; e += blockDim.x)
                Rs[e] = kv == 0 ? *swz_ptr<float>(rec + y.off_RK, e / d, e % d, d)
                                : *swz_ptr<float>(rec + y.off_RV, e % d, e / d, rp);
            __syncthreads();
        }
    }
    const char *page = p.dense_pool + y.dense_offset(p.layer, b, y.dense_slot(pg), h, kv);
    const T *chunk = reinterpret_cast<const T *>(kv == 0 ? p.k_new : p.v_new);
    T *out = reinterpret_cast<T *>(kv == 0 ? p.k_out : p.v_out);
    const int nv = d / VE;
    for (int e = threadIdx.x; e < (r1 - r0) * nv; e += blockDim.x) {
        const int r = r0 + e / nv, c = e % nv * VE, t = r - pg * P;
        uint4 x;
        if (factored) {
            float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
            if constexpr (sizeof(T) == 4)
                for (int j = 0; j < rp; ++j) {
                    const float l = Ls[t * rp + j];
                    const float4 v = *reinterpret_cast<const float4 *>(Rs + j * d + c);
                    f = make_float4(fmaf(l, v.x, f.x), fmaf(l, v.y, f.y), fmaf(l, v.z, f.z), fmaf(l, v.w, f.w));
                }
            x = make_uint4(__float_as_uint(f.x), __float_as_uint(f.y), __float_as_uint(f.z), __float_as_uint(f.w));
        } else if (r < T0) {
            x = *reinterpret_cast<const uint4 *>(swz_ptr<T>(page, t, c, d));
        } else {
            x = *reinterpret_cast<const uint4 *>(chunk + ((size_t)(p.coff[i] + r - T0) * y.H + h) * d + c);
        }
        *reinterpret_cast<uint4 *>(out + (size_t)(p.off[i] + r - lo) * p.row_stride + (size_t)h * p.head_stride + c) = x;
    }
}

// Rows of bf16 stores, HBM-bound: a factorized row is 0.47 of its bytes as
// factors, and all of them are written.  CTAs stay and loop over items (128
// positions of an entry, head, K/V): the next item's factors arrive while one is
// computed on the warps' tensor cores (fp32 sums, rounded once) and written a
// whole row per sixteen lanes.  32K tokens x 8 heads, ranks 16 and 24: 52 us (3.8
// TB/s; 277 us with scalar products, a block per page); a CTA's item is a chain of
// short steps, and two CTAs of 16 warps fill the registers.
struct ReadItem {
    int i, b, h, kv, pg0, lo, hi, off, fw;
    ReadItem() = default;
    __device__ __forceinline__ ReadItem(const RowsParams &p, int item, int pages) {
        kv = item & 1;
        h = (item >> 1) % p.y.H;
        int blk = (item >> 1) / p.y.H;
        i = 0;
        while (blk >= p.page_off[i + 1]) ++i;
        blk -= p.page_off[i];
        lo = p.lo[i];
        hi = lo + p.n[i];
        pg0 = lo / p.y.P + blk * pages;
        b = p.seqs[i];
        off = p.off[i];
        fw = min(p.fw[i], (hi + p.y.P - 1) / p.y.P);  // factorized pages that hold asked rows
    }
};

template <int P, int D, bool Q4>
__global__ void __launch_bounds__(STAGE_THREADS, 2) read_kernel(const RowsParams p) {
    extern __shared__ __align__(128) unsigned char sm[];
    __shared__ uint64_t bars[2];
    __shared__ ReadItem its[2];
    constexpr int NP = BLOCK / P, TILE = BLOCK * D * 2, CH = D / 8;
    const Layout &y = p.y;
    const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int items = 2 * p.page_off[p.nseq] * y.H;  // page_off: blocks here
    const BlockLayout bl(y);
    if (tid == 0) {
        mbar_init(&bars[0], 1);
        mbar_init(&bars[1], 1);
        fence_barrier_init();
    }
    grid_dependency_wait();  // the launch before may still write pages
    __syncthreads();
    auto buffer = [&](int buf) { return sm + TILE + buf * NP * bl.fetch_bytes; };
    auto fetch = [&](int item, int buf) {  // one thread: an item's place and its factors
        const ReadItem it = its[buf] = ReadItem(p, item, NP);
        BlockPages(y, NP, it.pg0, it.fw, it.kv)
            .fetch<Q4>(y, bl, p.factor_pool, p.layer, it.b, it.h, it.kv, buffer(buf), &bars[buf], item == 0 ? p.hook.extra() : 0);
    };
    if (tid == 0 && (int)blockIdx.x < items) fetch(blockIdx.x, 0);
    __syncthreads();
    uint32_t phase = 0;
    int buf = 0;
    const RowTile<P, D> rt;
    for (int item = blockIdx.x; item < items; item += gridDim.x, buf ^= 1) {
        const int next = item + gridDim.x;
        if (tid == 0 && next < items) fetch(next, buf ^ 1);
        const ReadItem it = its[buf];
        const int lo = it.lo, hi = it.hi;
        const BlockPages bp(y, NP, it.pg0, it.fw, it.kv);
        unsigned char *pages = Q4 ? buffer(2) : buffer(buf);
        if (bp.lo > 0 || bp.hi < NP) {
            // rows past the asked ones are not read: pages of this block past
            // `hi` may be factorized and have no dense rows
            fetch_dense<P, D>(y, bp, p.dense_pool, nullptr, 0, p.layer, it.b, it.h, it.kv, hi, hi, pages, bl.page_bytes);
            __syncthreads();
        }
        if (bp.lo < bp.hi) {
            const bool ok = __syncthreads_and(mbar_wait_bounded(&bars[buf], (phase >> buf) & 1, p.status, p.hook.limit()) ? 1 : 0) != 0;
            if (!ok) {
                if (tid == 0) {
                    mbar_wait_bounded(&bars[buf], (phase >> buf) & 1, nullptr);
                    if (next < items) {
                        const ReadItem nx = its[buf ^ 1];
                        const BlockPages nb(y, NP, nx.pg0, nx.fw, nx.kv);
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
        rt.template rebuild<Q4>(acc, y, bl, bp, it.kv, pages, buffer(buf));
        if (y.rope && it.kv == 0) rt.turn(acc, p.rope_base, p.rope_delta, it.pg0 + rt.s, hi);
#pragma unroll
        for (int j = 0; j < rt.KT; ++j)
#pragma unroll
            for (int r2 = 0; r2 < 2; ++r2)
                *reinterpret_cast<uint32_t *>(sm + swz_offset(16 * rt.w + g + 8 * r2, 16 * rt.nt(j) + 4 * c, D * 2)) =
                    pack_bf16(acc[j][2 * r2], acc[j][2 * r2 + 1]);
        fence_proxy_async_shared();  // the fetch buffer is read
        __syncthreads();
        __nv_bfloat16 *out = reinterpret_cast<__nv_bfloat16 *>(it.kv ? p.v_out : p.k_out) + (size_t)it.h * p.head_stride;
#pragma unroll
        for (int k = 0; k < BLOCK * CH / STAGE_THREADS; ++k) {
            const int e = tid + k * STAGE_THREADS, row = e / CH, ch = e % CH, pos = it.pg0 * P + row;
            if (pos >= lo && pos < hi)
                reinterpret_cast<uint4 *>(out + (size_t)(it.off + pos - lo) * p.row_stride)[ch] =
                    *reinterpret_cast<const uint4 *>(sm + swz_offset(row, 16 * ch, D * 2));
        }
        __syncthreads();  // the tile is read
    }
}

// Block (group of 16 rows, head, call entry): rows that stay in a dense page.
// A row of the chunk whose page has already left the ring at the new length is
// not written (its page is factorized from the caller's rows).  Block (0, 0,
// entry) also writes the entry's length and the page kinds from its first page
// that was dense on.
template <typename T>
__global__ void append_chunk_kernel(const AppendChunkParams p) {
    const Layout &y = p.y;
    const int i = blockIdx.z, h = blockIdx.y, b = p.seqs[i];
    const int T0 = p.T[i], T1 = T0 + p.n[i];
    if (T1 == T0) return;
    const int last = (T1 - 1) / y.P;
    if (h == 0 && blockIdx.x == 0) {
        if (threadIdx.x == 0) p.lengths[y.len_index(b, p.layer)] = T1;
        const int first = max(0, (T0 - y.W) / y.P - 1);
        for (int pg = first + threadIdx.x; pg <= last; pg += blockDim.x)
            p.desc[y.desc_index(b, p.layer, pg)] =
                page_kind(pg, T1, y.P, y.sink_tokens, y.W) == KIND_DENSE ? (KIND_DENSE << KIND_SHIFT) | y.dense_slot(pg) : pg;
    }
    const T *src[2] = {reinterpret_cast<const T *>(p.k), reinterpret_cast<const T *>(p.v)};
    constexpr int VE = 16 / sizeof(T);  // elements of a 16-byte chunk
    const int nv = y.d / VE, per_row = 2 * nv;
    const int j0 = blockIdx.x * 16, j1 = min(p.n[i], j0 + 16);
    for (int e = threadIdx.x; e < (j1 - j0) * per_row; e += blockDim.x) {
        const int j = j0 + e / per_row, kv = (e % per_row) / nv, c = e % nv;
        const int pg = (T0 + j) / y.P, row = (T0 + j) % y.P;
        if (pg >= y.sink_pages && pg <= last - y.ring) continue;
        char *dst = p.dense_pool + y.dense_offset(p.layer, b, y.dense_slot(pg), h, kv);
        *reinterpret_cast<uint4 *>(swz_ptr<T>(dst, row, c * VE, y.d)) =
            reinterpret_cast<const uint4 *>(src[kv] + ((size_t)(p.off[i] + j) * y.H + h) * y.d)[c];
    }
}

// Block (call entry, layer): the length, and the kinds of the pages the old
// length described (pages past the new length become 0).
__global__ void truncate_kernel(const TruncateParams p) {
    const Layout &y = p.y;
    const int i = blockIdx.x, layer = blockIdx.y, b = p.seqs[i], T = p.T[i];
    if (threadIdx.x == 0) p.lengths[y.len_index(b, layer)] = T;
    const int n = (T + y.P - 1) / y.P;
    for (int pg = max(0, (T - y.W) / y.P - 1) + threadIdx.x; pg < p.had[i]; pg += blockDim.x) {
        int v = 0;
        if (pg < n)
            v = page_kind(pg, T, y.P, y.sink_tokens, y.W) == KIND_DENSE ? (KIND_DENSE << KIND_SHIFT) | y.dense_slot(pg) : pg;
        p.desc[y.desc_index(b, layer, pg)] = v;
    }
}

// Block (page, head): the four factors into the record, ranks padded with zeros.
template <typename T>
__global__ void load_factors_kernel(const LoadFactorsParams p) {
    const Layout &y = p.y;
    const int P = y.P, d = y.d, h = blockIdx.y;
    char *rec = p.factor_pool + y.record_offset(p.layer, p.seq, h, p.page0 + blockIdx.x);
    const size_t pg = (size_t)h * p.n + blockIdx.x;
    const T *LK = reinterpret_cast<const T *>(p.LK) + pg * P * y.rk, *RK = reinterpret_cast<const T *>(p.RK) + pg * y.rk * d;
    const T *LV = reinterpret_cast<const T *>(p.LV) + pg * P * y.rv, *RV = reinterpret_cast<const T *>(p.RV) + pg * y.rv * d;
    const T zero = Elem<T>::from_f32(0.f);
    for (int e = threadIdx.x; e < P * y.rkp; e += blockDim.x) {
        const int t = e / y.rkp, j = e % y.rkp;
        *swz_ptr<T>(rec, t, j, y.rkp) = j < y.rk ? LK[t * y.rk + j] : zero;
    }
    for (int e = threadIdx.x; e < y.rkp * d; e += blockDim.x) {
        const int j = e / d, c = e % d;
        *swz_ptr<T>(rec + y.off_RK, j, c, d) = j < y.rk ? RK[j * d + c] : zero;
    }
    for (int e = threadIdx.x; e < y.rvp * P; e += blockDim.x) {
        const int j = e / P, t = e % P;
        *swz_ptr<T>(rec + y.off_LV, j, t, P) = j < y.rv ? LV[t * y.rv + j] : zero;
    }
    for (int e = threadIdx.x; e < d * y.rvp; e += blockDim.x) {
        const int c = e / y.rvp, j = e % y.rvp;
        *swz_ptr<T>(rec + y.off_RV, c, j, y.rvp) = j < y.rv ? RV[j * d + c] : zero;
    }
}

template <int P, int D, bool Q4>
static cudaError_t read_t(const RowsParams &p, int num_sms, cudaStream_t st) {
    const int smem = BLOCK * D * 2 + (int)BlockLayout(p.y).smem(p.y, BLOCK / P);
    cudaError_t e = allow_smem<read_kernel<P, D, Q4>>(smem);
    if (e != cudaSuccess) return e;
    const int items = 2 * p.page_off[p.nseq] * p.y.H, resident = std::min(2, 227 * 1024 / (smem + 1024));
    return launch_dependent(read_kernel<P, D, Q4>, dim3((unsigned)std::min(items, num_sms * resident)), STAGE_THREADS, smem, st, p);
}

cudaError_t launch_read(RowsParams &p, int num_sms, cudaStream_t st) {
    const Layout &y = p.y;
    if (y.dtype != 1) return launch_rows(p, st);
    const int np = BLOCK / y.P;
    p.page_off[0] = 0;
    for (int i = 0; i < p.nseq; ++i) {
        const int pages = p.n[i] > 0 ? (p.lo[i] + p.n[i] - 1) / y.P - p.lo[i] / y.P + 1 : 0;
        p.page_off[i + 1] = p.page_off[i] + (pages + np - 1) / np;
    }
    if (p.page_off[p.nseq] == 0) return cudaSuccess;
#define PKV_READ_CASE(PP, DD) \
    if (y.P == PP && y.d == DD) return y.q4 ? read_t<PP, DD, true>(p, num_sms, st) : read_t<PP, DD, false>(p, num_sms, st);
    PKV_READ_CASE(16, 64)
    PKV_READ_CASE(32, 64)
    PKV_READ_CASE(64, 64)
    PKV_READ_CASE(16, 128)
    PKV_READ_CASE(32, 128)
    PKV_READ_CASE(64, 128)
#undef PKV_READ_CASE
    return cudaErrorInvalidValue;
}

cudaError_t launch_rows(RowsParams &p, cudaStream_t st) {
    const Layout &y = p.y;
    p.page_off[0] = 0;
    for (int i = 0; i < p.nseq; ++i)
        p.page_off[i + 1] = p.page_off[i] + (p.n[i] > 0 ? (p.lo[i] + p.n[i] - 1) / y.P - p.lo[i] / y.P + 1 : 0);
    if (p.page_off[p.nseq] == 0) return cudaSuccess;
    const size_t smem = (size_t)(y.P + y.d) * (y.rkp > y.rvp ? y.rkp : y.rvp) * 4;  // at most 48 KB
    const dim3 grid((unsigned)p.page_off[p.nseq], (unsigned)y.H, 2);
    if (y.dtype == 1)
        rows_kernel<__nv_bfloat16><<<grid, 256, smem, st>>>(p);
    else
        rows_kernel<float><<<grid, 256, smem, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_append_chunk(const AppendChunkParams &p, cudaStream_t st) {
    int most = 0;
    for (int i = 0; i < p.nseq; ++i) most = p.n[i] > most ? p.n[i] : most;
    if (most == 0) return cudaSuccess;
    const dim3 grid((unsigned)((most + 15) / 16), (unsigned)p.y.H, (unsigned)p.nseq);
    if (p.y.dtype == 1)
        append_chunk_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(p);
    else
        append_chunk_kernel<float><<<grid, 256, 0, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_truncate(const TruncateParams &p, cudaStream_t st) {
    truncate_kernel<<<dim3((unsigned)p.nseq, (unsigned)p.y.L), 128, 0, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_load_factors(const LoadFactorsParams &p, cudaStream_t st) {
    const dim3 grid((unsigned)p.n, (unsigned)p.y.H);
    if (p.y.dtype == 1)
        load_factors_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(p);
    else
        load_factors_kernel<float><<<grid, 256, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace pkv
