// Attention of a chunk of query tokens over densely laid out fp32 keys and
// values in CUDA-core arithmetic (fp32 stores), and the merge of split softmax states
// ("PuzzleKV: Page-Wise Low-Rank Decomposition for KV Cache Compression",
// §3.3 ④, eq. (5)).
//
// With m the running maximum (log2 units) of a row's scores s = q k / sqrt(d),
//   l = sum 2^(s - m),  o = sum 2^(s - m) v,  out = o / l,
// one pass over the keys; query token j of a sequence with T cached tokens
// sees keys 0 .. T + j.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace pkv {

constexpr int CS_ROWS = 32, CS_KEYS = 32;  // query rows and keys of a tile

__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }

// Block (tile of 32 query rows of one (entry, KV head), split): 128 threads,
// eight to a pair of rows.  A thread scores 2 rows x 4 keys and accumulates
// 2 rows x D/8 columns, so that a shared-memory vector feeds two rows.  Bound by
// shared-memory reads where there is much work, by its few dependent tiles where
// there is little (37 tokens over 1K, d = 64: 13 us).
template <int D>
__global__ void __launch_bounds__(128) chunk_simple_kernel(const ChunkAttnParams p) {
    extern __shared__ __align__(16) float sm[];
    constexpr int PQ = D + 4;  // row pitch: the four row groups of a warp start on distinct banks
    float *Qs = sm, *Ks = Qs + CS_ROWS * PQ, *Vs = Ks + CS_KEYS * PQ, *Ps = Vs + CS_KEYS * PQ;
    const int tid = threadIdx.x, tx = tid & 7, ty = tid >> 3;
    int i = 0;
    while ((int)blockIdx.x >= p.tile_off[i + 1]) ++i;
    const int G = p.G, R = p.n[i] * G, tiles = (R + CS_ROWS - 1) / CS_ROWS, ns = p.ns[i];
    int u = (int)blockIdx.x - p.tile_off[i];
    const int sp = u % ns;
    u /= ns;
    const int h = u / tiles, row0 = (u % tiles) * CS_ROWS;
    const int Tk = p.T[i] + p.n[i], nkb = (Tk + CS_KEYS - 1) / CS_KEYS;
    const int kb0 = (int)((long long)nkb * sp / ns), kb1 = (int)((long long)nkb * (sp + 1) / ns);
    const float *q = reinterpret_cast<const float *>(p.q);
    constexpr int PER = CS_KEYS * D / 4 / 128;  // groups of four elements of a tile per thread
    {
        float4 v[PER];
#pragma unroll
        for (int a = 0; a < PER; ++a) {
            const int e = tid + 128 * a, r = row0 + e / (D / 4), tok = r / G;
            v[a] = r < R ? load4(q + ((size_t)(p.off[i] + tok) * p.Hq + h * G + r - tok * G) * D + e % (D / 4) * 4)
                         : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int a = 0; a < PER; ++a) {
            const int e = tid + 128 * a;
            *reinterpret_cast<float4 *>(Qs + e / (D / 4) * PQ + e % (D / 4) * 4) =
                make_float4(v[a].x * p.scale_log2, v[a].y * p.scale_log2, v[a].z * p.scale_log2, v[a].w * p.scale_log2);
        }
    }
    int lim[2];  // last key each of the thread's rows sees (-1: no such row)
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[2][D / 8];
#pragma unroll
    for (int a = 0; a < 2; ++a) {
        const int r = row0 + 2 * ty + a;
        lim[a] = r < R ? p.T[i] + r / G : -1;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) o[a][c] = 0.f;
    }
    const int last_key = p.T[i] + (min(row0 + CS_ROWS, R) - 1) / G;
    const float *K = reinterpret_cast<const float *>(p.K) + (size_t)p.koff[i] * p.H * D + (size_t)h * D;
    const float *V = reinterpret_cast<const float *>(p.V) + (size_t)p.koff[i] * p.H * D + (size_t)h * D;
    for (int kb = kb0; kb < kb1 && kb * CS_KEYS <= last_key; ++kb) {
        float4 kr[PER], vr[PER];  // in flight together, past the last tile's arithmetic
#pragma unroll
        for (int a = 0; a < PER; ++a) {
            const int e = tid + 128 * a, t = kb * CS_KEYS + e / (D / 4);
            const size_t at = (size_t)t * p.H * D + e % (D / 4) * 4;
            kr[a] = t < Tk ? load4(K + at) : make_float4(0.f, 0.f, 0.f, 0.f);
            vr[a] = t < Tk ? load4(V + at) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        __syncthreads();
#pragma unroll
        for (int a = 0; a < PER; ++a) {
            const int e = tid + 128 * a, at = e / (D / 4) * PQ + e % (D / 4) * 4;
            *reinterpret_cast<float4 *>(Ks + at) = kr[a];
            *reinterpret_cast<float4 *>(Vs + at) = vr[a];
        }
        __syncthreads();
        float s[2][4] = {};
        for (int c = 0; c < D; c += 4) {
            float4 qa = *reinterpret_cast<const float4 *>(Qs + (2 * ty) * PQ + c);
            float4 qb = *reinterpret_cast<const float4 *>(Qs + (2 * ty + 1) * PQ + c);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 kv = *reinterpret_cast<const float4 *>(Ks + (tx + 8 * j) * PQ + c);
                s[0][j] = fmaf(qa.x, kv.x, fmaf(qa.y, kv.y, fmaf(qa.z, kv.z, fmaf(qa.w, kv.w, s[0][j]))));
                s[1][j] = fmaf(qb.x, kv.x, fmaf(qb.y, kv.y, fmaf(qb.z, kv.z, fmaf(qb.w, kv.w, s[1][j]))));
            }
        }
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (kb * CS_KEYS + tx + 8 * j > lim[a]) s[a][j] = -INFINITY;
                mx = fmaxf(mx, s[a][j]);
            }
#pragma unroll
            for (int x = 1; x < 8; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
            const float mn = fmaxf(m[a], mx), base = mn == -INFINITY ? 0.f : mn;
            const float f = exp2f(m[a] - base);
            float ls = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float w = exp2f(s[a][j] - base);
                ls += w;
                Ps[(2 * ty + a) * (CS_KEYS + 1) + tx + 8 * j] = w;
            }
            l[a] = fmaf(l[a], f, ls);
            m[a] = mn;
#pragma unroll
            for (int c = 0; c < D / 8; ++c) o[a][c] *= f;
        }
        __syncwarp();  // a row's eight threads share a warp
        for (int k = 0; k < CS_KEYS; ++k) {
            const int t = kb * CS_KEYS + k;
            float w[2];
#pragma unroll
            for (int a = 0; a < 2; ++a) w[a] = Ps[(2 * ty + a) * (CS_KEYS + 1) + k];
#pragma unroll
            for (int c4 = 0; c4 < D / 32; ++c4) {
                const float4 v = *reinterpret_cast<const float4 *>(Vs + k * PQ + 32 * c4 + 4 * tx);
#pragma unroll
                for (int a = 0; a < 2; ++a)
                    if (t <= lim[a]) {  // a key the row does not see adds nothing, whatever its value holds
                        o[a][4 * c4] = fmaf(w[a], v.x, o[a][4 * c4]);
                        o[a][4 * c4 + 1] = fmaf(w[a], v.y, o[a][4 * c4 + 1]);
                        o[a][4 * c4 + 2] = fmaf(w[a], v.z, o[a][4 * c4 + 2]);
                        o[a][4 * c4 + 3] = fmaf(w[a], v.w, o[a][4 * c4 + 3]);
                    }
            }
        }
        __syncwarp();
    }
#pragma unroll
    for (int a = 0; a < 2; ++a) {
#pragma unroll
        for (int x = 1; x < 8; x <<= 1) l[a] += __shfl_xor_sync(0xffffffffu, l[a], x);
        const int r = row0 + 2 * ty + a;
        if (r >= R) continue;
        if (ns == 1) {
            const float il = 1.f / l[a];
            float *dst = reinterpret_cast<float *>(p.out) + ((size_t)(p.off[i] + r / G) * p.Hq + h * G + r % G) * D;
#pragma unroll
            for (int c4 = 0; c4 < D / 32; ++c4)
                *reinterpret_cast<float4 *>(dst + 32 * c4 + 4 * tx) =
                    make_float4(o[a][4 * c4] * il, o[a][4 * c4 + 1] * il, o[a][4 * c4 + 2] * il, o[a][4 * c4 + 3] * il);
        } else {
            float *row = p.partials + (size_t)(p.poff[i] + (long long)(h * ns + sp) * R + r) * (D + 4);
            if (tx == 0) *reinterpret_cast<float4 *>(row) = make_float4(m[a], l[a], 0.f, 0.f);
#pragma unroll
            for (int c4 = 0; c4 < D / 32; ++c4)
                *reinterpret_cast<float4 *>(row + 4 + 32 * c4 + 4 * tx) =
                    make_float4(o[a][4 * c4], o[a][4 * c4 + 1], o[a][4 * c4 + 2], o[a][4 * c4 + 3]);
        }
    }
}

// Warp per query row of an entry with several splits: the states joined in
// split order (the same sums whatever the launch), eq. (5).
template <typename T, int D>
__global__ void __launch_bounds__(128) chunk_merge_kernel(const ChunkAttnParams p) {
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    int i = 0;
    while (i < p.nseq && w >= p.tile_off[i + 1]) ++i;
    if (i >= p.nseq) return;
    const int G = p.G, R = p.n[i] * G, ns = p.ns[i];
    const int u = (int)(w - p.tile_off[i]), h = u / R, r = u % R;
    const float *rows = p.partials + (size_t)(p.poff[i] + (long long)h * ns * R + r) * (D + 4);
    const size_t pitch = (size_t)R * (D + 4);
    constexpr int V = D / 32;
    // the first 32 (m, l) and the first eight o come in one trip to memory
    float2 ml = lane < ns ? *reinterpret_cast<const float2 *>(rows + lane * pitch) : make_float2(-INFINITY, 0.f);
    float o[8][V];
    auto fetch = [&](int s0) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int k = 0; k < V; ++k) o[j][k] = s0 + j < ns ? rows[(s0 + j) * pitch + 4 + lane * V + k] : 0.f;
    };
    fetch(0);
    float M = ml.x;
    for (int s = lane + 32; s < ns; s += 32) M = fmaxf(M, rows[s * pitch]);
    M = warp_max(M);
    float L = 0.f, acc[V] = {};
    for (int sb = 0; sb < ns; sb += 32) {
        if (sb) ml = sb + lane < ns ? *reinterpret_cast<const float2 *>(rows + (sb + lane) * pitch) : make_float2(-INFINITY, 0.f);
        const float f = exp2f(ml.x - M);
        L = fmaf(f, ml.y, L);
        for (int s = 0; s < 32 && sb + s < ns; s += 8) {
            if (sb + s) fetch(sb + s);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float fj = __shfl_sync(0xffffffffu, f, s + j);
#pragma unroll
                for (int k = 0; k < V; ++k) acc[k] = fmaf(fj, o[j][k], acc[k]);
            }
        }
    }
    L = warp_sum(L);
    const float il = 1.f / L;
    T *dst = reinterpret_cast<T *>(p.out) + ((size_t)(p.off[i] + r / G) * p.Hq + h * G + r % G) * D;
#pragma unroll
    for (int k = 0; k < V; ++k) dst[lane * V + k] = Elem<T>::from_f32(acc[k] * il);
}

template <int D>
static cudaError_t simple_t(ChunkAttnParams &p, cudaStream_t st) {
    constexpr int smem = ((CS_ROWS + 2 * CS_KEYS) * (D + 4) + CS_ROWS * (CS_KEYS + 1)) * 4;
    cudaError_t e = allow_smem<chunk_simple_kernel<D>>(smem);
    if (e != cudaSuccess) return e;
    chunk_simple_kernel<D><<<(unsigned)p.tile_off[p.nseq], 128, smem, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_chunk_simple(ChunkAttnParams &p, cudaStream_t st) {
    p.tile_off[0] = 0;
    for (int i = 0; i < p.nseq; ++i)
        p.tile_off[i + 1] = p.tile_off[i] + p.H * ((p.n[i] * p.G + CS_ROWS - 1) / CS_ROWS) * p.ns[i];
    if (p.tile_off[p.nseq] == 0) return cudaSuccess;
    return p.d == 64 ? simple_t<64>(p, st) : simple_t<128>(p, st);
}

cudaError_t launch_chunk_merge(const ChunkAttnParams &q, int dtype, cudaStream_t st) {
    ChunkAttnParams p = q;
    p.tile_off[0] = 0;
    for (int i = 0; i < p.nseq; ++i) p.tile_off[i + 1] = p.tile_off[i] + (p.ns[i] > 1 ? p.H * p.n[i] * p.G : 0);
    const int rows = p.tile_off[p.nseq];
    if (rows == 0) return cudaSuccess;
    const unsigned grid = (unsigned)((rows + 3) / 4);
    if (dtype == 1)
        return p.d == 64 ? launch_dependent(chunk_merge_kernel<__nv_bfloat16, 64>, grid, 128, 0, st, p)
                         : launch_dependent(chunk_merge_kernel<__nv_bfloat16, 128>, grid, 128, 0, st, p);
    return p.d == 64 ? launch_dependent(chunk_merge_kernel<float, 64>, grid, 128, 0, st, p)
                     : launch_dependent(chunk_merge_kernel<float, 128>, grid, 128, 0, st, p);
}

}  // namespace pkv
