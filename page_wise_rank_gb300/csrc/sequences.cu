// Copies of whole sequences inside a store: forks (one prompt, several
// samples), reordered beams, compaction of slots.
//
// A sequence slot owns the same byte offsets in both pools as every other
// slot, shifted by a constant per layer.  So all the pairs of a call can be
// copied "at once" with no scratch in HBM: a CTA takes one small tile of
// offsets, brings that tile of every distinct source into shared memory, and
// only then writes the destinations' tiles; no other CTA touches those bytes,
// so permutations and cycles need no order between pairs.  Each source byte
// is read once however many destinations it has.  HBM-bound: 81 MB read and 242 MB
// written (one sequence to three) in 52 us, 6.2 TB/s.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace pkv {

constexpr int COPY_SMEM = 96 * 1024;  // most staging per CTA (many sources)
constexpr int COPY_TILE = 16 * 1024;  // a tile of few sources: many CTAs per SM keep copies in flight

// Tiles of one layer: per head the factor records of pages [sink_pages,
// max_upto), cut in tiles of p.tile bytes; then every dense slot that some
// source uses ([head][K|V][P][d], contiguous), cut the same way.
struct CopyTiles {
    size_t head_bytes, slot_bytes;
    int per_head, per_slot, nslots, per_layer;
    __host__ __device__ explicit CopyTiles(const CopyParams &p) {
        const Layout &y = p.y;
        head_bytes = p.max_upto > y.sink_pages ? (size_t)(p.max_upto - y.sink_pages) * y.rec_bytes : 0;
        slot_bytes = (size_t)y.H * 2 * y.dense_half_bytes;
        per_head = (int)((head_bytes + p.tile - 1) / p.tile);
        per_slot = (int)((slot_bytes + p.tile - 1) / p.tile);
        nslots = 0;
        for (unsigned long long m = p.any_slots; m; m &= m - 1) ++nslots;
        per_layer = y.H * per_head + nslots * per_slot;
    }
};

__global__ void __launch_bounds__(32) copy_sequences_kernel(const CopyParams p) {
    extern __shared__ __align__(128) char stage[];
    __shared__ uint64_t bar;
    const Layout &y = p.y;
    const CopyTiles t(p);
    // page table of the destinations, from the sources' lengths
    for (int e = blockIdx.x; e < p.npair * y.L; e += gridDim.x) {
        const int i = e / y.L, l = e % y.L, b = p.dst[i], T = p.T[p.pair_src[i]];
        const int n = (T + y.P - 1) / y.P;
        if (threadIdx.x == 0) p.lengths[y.len_index(b, l)] = T;
        for (int pg = threadIdx.x; pg < (n > p.had[i] ? n : p.had[i]); pg += 32) {
            int v = 0;
            if (pg < n)
                v = page_kind(pg, T, y.P, y.sink_tokens, y.W) == KIND_DENSE
                        ? (KIND_DENSE << KIND_SHIFT) | y.dense_slot(pg) : pg;
            p.desc[y.desc_index(b, l, pg)] = v;
        }
    }
    if (threadIdx.x != 0) return;
    mbar_init(&bar, 1);
    fence_barrier_init();
    uint32_t phase = 0;
    const int total = t.per_layer * y.L;
    for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
        const int l = tile / t.per_layer;
        int r = tile % t.per_layer;
        char *pool;
        size_t base, stride, off, end;  // slot b's region starts at base + b * stride; the tile is [off, end) of it
        int slot = -1;
        if (r < y.H * t.per_head) {
            const int h = r / t.per_head;
            pool = p.factor_pool;
            base = y.record_offset(l, 0, h, y.sink_pages);
            stride = (size_t)y.H * y.n_pg_max * y.rec_bytes;
            off = (size_t)(r % t.per_head) * p.tile;
            end = off + p.tile < t.head_bytes ? off + p.tile : t.head_bytes;
        } else {
            r -= y.H * t.per_head;
            unsigned long long m = p.any_slots;
            for (int k = r / t.per_slot; k > 0; --k) m &= m - 1;
            slot = __ffsll((long long)m) - 1;
            pool = p.dense_pool;
            base = y.dense_offset(l, 0, slot, 0, 0);
            stride = (size_t)y.dslots * t.slot_bytes;
            off = (size_t)(r % t.per_slot) * p.tile;
            end = off + p.tile < t.slot_bytes ? off + p.tile : t.slot_bytes;
        }
        // bytes of this tile that source j holds
        auto bytes_of = [&](int j) -> uint32_t {
            size_t e = end;
            if (slot >= 0) {
                if (!((p.slots[j] >> slot) & 1)) return 0;
            } else {
                const size_t live = p.upto[j] > y.sink_pages ? (size_t)(p.upto[j] - y.sink_pages) * y.rec_bytes : 0;
                if (live < e) e = live;
            }
            return e > off ? (uint32_t)(e - off) : 0;
        };
        uint32_t tx = 0;
        for (int j = 0; j < p.nsrc; ++j) tx += bytes_of(j);
        if (tx == 0) continue;
        // the previous tile's stores have read the stage
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        mbar_arrive_expect_tx(&bar, tx + (tile == 0 ? p.hook.extra() : 0));
        for (int j = 0; j < p.nsrc; ++j) {
            const uint32_t nb = bytes_of(j);
            if (nb) bulk_g2s(stage + (size_t)j * p.tile, pool + base + (size_t)p.src[j] * stride + off, nb, &bar);
        }
        if (!mbar_wait_bounded(&bar, phase, p.status, p.hook.limit())) {  // give up: let the copies land, write nothing more
            mbar_wait_bounded(&bar, phase, nullptr);
            break;
        }
        phase ^= 1;
        for (int i = 0; i < p.npair; ++i) {
            const int j = p.pair_src[i];
            const uint32_t nb = bytes_of(j);
            if (nb)
                asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                                 pool + base + (size_t)p.dst[i] * stride + off),
                             "r"(smem_u32(stage + (size_t)j * p.tile)), "r"(nb)
                             : "memory");
        }
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

cudaError_t launch_copy(CopyParams &p, int num_sms, cudaStream_t st) {
    p.max_upto = 0;
    p.any_slots = 0;
    for (int j = 0; j < p.nsrc; ++j) {
        p.max_upto = p.upto[j] > p.max_upto ? p.upto[j] : p.max_upto;
        p.any_slots |= p.slots[j];
    }
    p.tile = COPY_SMEM / p.nsrc < COPY_TILE ? (COPY_SMEM / p.nsrc) & ~511 : COPY_TILE;
    const CopyTiles t(p);
    const long total = (long)t.per_layer * p.y.L;
    const long work = total > (long)p.npair * p.y.L ? total : (long)p.npair * p.y.L;
    const int smem = p.tile * p.nsrc;
    cudaError_t e = allow_smem<copy_sequences_kernel>(COPY_SMEM);
    if (e != cudaSuccess) return e;
    const long most = (long)num_sms * std::min(16, 220 * 1024 / (smem + 1024));
    const long grid = work < most ? work : most;
    copy_sequences_kernel<<<(unsigned)grid, 32, smem, st>>>(p);
    return cudaGetLastError();
}

}  // namespace pkv
