// C ABI of the calls that work on several tokens or whole sequences at once
// (declared in include/puzzlekv.h): chunk attention, chunk append, reading
// rows, loading factors, copying and cutting back sequences.  Every argument
// is checked on the host before anything is launched, the host mirror decides
// which pages are dense, and scratch memory is the caller's.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <exception>
#include <vector>

#include "../../include/puzzlekv.h"
#include "kernels.h"
#include "layout.h"
#include "store.h"

using namespace pkv;

namespace {

// Run an entry point's body; a C++ exception (host memory) becomes a status.
template <typename F>
puzzlekv_status guarded(F body) {
    try {
        return body();
    } catch (const std::exception &e) {
        return fail(PUZZLEKV_ERR_INVALID_ARG, "host-side failure: %s", e.what());
    } catch (...) {
        return fail(PUZZLEKV_ERR_INVALID_ARG, "host-side failure");
    }
}

int length_of(const puzzlekv_store *s, int b, int l) { return std::max(0, s->len[(size_t)b * s->y.L + l]); }

// A call that changes the host mirror cannot be captured: a replay would
// repeat the device work without the bookkeeping.
puzzlekv_status refuse_capture(cudaStream_t strm) {
    cudaStreamCaptureStatus c = cudaStreamCaptureStatusNone;
    const cudaError_t e = cudaStreamIsCapturing(strm, &c);
    if (e != cudaSuccess) return cuda_fail(e, "cudaStreamIsCapturing");
    if (c != cudaStreamCaptureStatusNone)
        return fail(PUZZLEKV_ERR_UNSUPPORTED, "this call changes the store's host state and cannot be captured");
    return PUZZLEKV_OK;
}

// A captured call cannot wait for background work queued outside the capture:
// a batch must have been waited for, and by the captured stream unless it has
// finished since.
puzzlekv_status refuse_pending(const puzzlekv_store *s, cudaStream_t strm) {
    bool pending = false;
    for (const auto &cb : s->batches) pending |= cb.pending;
    if (!pending) return PUZZLEKV_OK;
    cudaStreamCaptureStatus c = cudaStreamCaptureStatusNone;
    const cudaError_t e = cudaStreamIsCapturing(strm, &c);
    if (e != cudaSuccess) return cuda_fail(e, "cudaStreamIsCapturing");
    if (c == cudaStreamCaptureStatusNone) return PUZZLEKV_OK;
    for (const auto &cb : s->batches) {
        if (!cb.pending) continue;
        bool here = false;
        for (const auto &w : cb.waited) here |= w.stream == strm;
        if (!here && (cb.waited.empty() || !batch_finished(cb)))
            return fail(PUZZLEKV_ERR_UNSUPPORTED, "background conversions are pending: call puzzlekv_wait_background before the capture");
    }
    return PUZZLEKV_OK;
}

puzzlekv_status check_list(const puzzlekv_store *s, const int32_t *ids, int32_t B, const char *what) {
    if (!s) return fail(PUZZLEKV_ERR_INVALID_ARG, "store is NULL");
    if (B < 1 || B > MAX_CALL_BATCH) return fail(PUZZLEKV_ERR_INVALID_ARG, "B must be in [1, %d]", MAX_CALL_BATCH);
    if (!ids) return fail(PUZZLEKV_ERR_INVALID_ARG, "%s is NULL", what);
    for (int i = 0; i < B; ++i) {
        if (ids[i] < 0 || ids[i] >= s->y.Bmax) return fail(PUZZLEKV_ERR_INVALID_ARG, "%s: slot %d out of range", what, ids[i]);
        for (int j = 0; j < i; ++j)
            if (ids[j] == ids[i]) return fail(PUZZLEKV_ERR_INVALID_ARG, "%s: slot %d listed twice", what, ids[i]);
    }
    return PUZZLEKV_OK;
}

// The list of a chunk call: counts >= 0, no sequence past its capacity.
puzzlekv_status check_chunk(const puzzlekv_store *s, int32_t layer, const int32_t *seq_ids, const int32_t *counts, int32_t B) {
    const puzzlekv_status st = check_list(s, seq_ids, B, "seq_ids");
    if (st != PUZZLEKV_OK) return st;
    if (layer < 0 || layer >= s->y.L) return fail(PUZZLEKV_ERR_INVALID_ARG, "layer %d out of range", layer);
    if (!counts) return fail(PUZZLEKV_ERR_INVALID_ARG, "counts is NULL");
    for (int i = 0; i < B; ++i) {
        if (counts[i] < 0) return fail(PUZZLEKV_ERR_INVALID_ARG, "counts[%d] is negative", i);
        const int T = length_of(s, seq_ids[i], layer);
        if (counts[i] > s->y.Tmax - T)
            return fail(PUZZLEKV_ERR_CAPACITY, "sequence %d: %d + %d tokens exceed max_tokens_per_seq=%d", seq_ids[i], T,
                        counts[i], s->y.Tmax);
    }
    return PUZZLEKV_OK;
}

// The test hook's request for this kernel, if there is one: consumed by the launch.
WaitHook take_hook(puzzlekv_store *s, int kernel) {
    WaitHook h;
    if (s->fail_chunk != kernel) return h;
    h.inject = 1;
    h.wait_ns = s->fail_chunk_ns;
    s->fail_chunk = FAIL_NONE;
    return h;
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// First dense page past the sink of a T-token sequence (pages [sink, it) are factorized).
int first_window_page(const Layout &y, int T) {
    int fw = (T + y.P - 1) / y.P;
    while (fw > y.sink_pages && page_kind(fw - 1, T, y.P, y.sink_tokens, y.W) == KIND_DENSE) --fw;
    return fw;
}

// What a chunk attention call runs and places in its workspace.
struct AttnPlan {
    int nseq = 0;                      // entries with new tokens, and their cached lengths
    int seqs[MAX_CALL_BATCH], lens[MAX_CALL_BATCH];
    SmallParams s{};                   // bf16 stores: entries of few query rows
    FlashParams f{};                   // bf16 stores: the others (staged as `g`)
    StageParams g{};
    ChunkAttnParams a{};               // fp32 stores, rebuilt by `r`; the merge of split states
    RowsParams r{};
    size_t images = 0, scales = 0, flash_parts = 0, keys = 0, values = 0, parts = 0, bytes = 0;  // offsets, total
};

void rows_params(const puzzlekv_store *s, int layer, RowsParams &rp) {
    rp = RowsParams{};
    rp.y = s->y;
    rp.factor_pool = s->factor_pool;
    rp.dense_pool = s->dense_pool;
    rp.status = reinterpret_cast<int *>(s->workspace);
    rp.rope_base = reinterpret_cast<const float2 *>(s->workspace + s->y.rope_base_offset);
    rp.rope_delta = reinterpret_cast<const float2 *>(s->workspace + s->y.rope_delta_offset);
    rp.layer = layer;
}

// Splits of the few-token path's entries over the SMs (one CTA each): every KV
// head's CTAs go to the entries in proportion to what they cost, the bytes they
// stream, times 1.6, 3.2 or 6.4 where two, four or eight row tiles make the
// arithmetic of a page (about 1,050 cycles a row-tile pair) longer than its
// 670 cycles of memory time.  One wave of CTAs is best when the shares come out even;
// lists of unequal lengths fill the SMs better with up to four.  A CTA's start
// and merge cost about as much as streaming 110 KB.
void split_small(const puzzlekv_store *s, SmallParams &p) {
    const Layout &y = s->y;
    constexpr double kCta = 110e3;
    const long long rec = (long long)y.rec_bytes, half = (long long)y.P * y.d * y.esz;
    std::vector<double> cost(p.nseq);
    double total = 0, best = 0;
    for (int i = 0; i < p.nseq; ++i) {
        const PageSplit ps(p.T[i], y.P, y.sink_pages, y.sink_tokens, y.W, rec, half, 1);
        const int tiles = (p.n[i] * y.G + 15) / 16;
        cost[i] = ((double)ps.total + (double)p.n[i] * y.d * 2 * y.esz) * (tiles <= 1 ? 1.0 : tiles <= 2 ? 1.6 : tiles <= 4 ? 3.2 : 6.4);
        total += cost[i];
    }
    std::vector<int> ns(p.nseq), pick(p.nseq, 1);
    for (int waves = 1; waves <= 4; ++waves) {
        const int want = std::min(700, std::max(1, s->num_sms * waves / y.H));
        double most = 0;
        int ctas = 0;
        for (int i = 0; i < p.nseq; ++i) {
            const int pages = (p.T[i] + y.P - 1) / y.P;
            ns[i] = std::max(1, std::min({pages, MAX_SPLITS, (int)std::lround(cost[i] * want / total)}));
            most = std::max(most, cost[i] / ns[i]);
            ctas += ns[i] * y.H;
        }
        const int rounds = (ctas + s->num_sms - 1) / s->num_sms;
        const double t = std::max(most + kCta, total * y.H / s->num_sms) + kCta * rounds + (rounds - 1) * most / 2;
        if (waves == 1 || t < best) {
            best = t;
            pick = ns;
        }
    }
    for (int i = 0; i < p.nseq; ++i) {
        p.ns[i] = pick[i];
        const PageSplit ps(p.T[i], y.P, y.sink_pages, y.sink_tokens, y.W, rec, half, p.ns[i]);
        for (int r = 0; r <= p.ns[i]; ++r) p.bounds[p.boff[i] + r] = ps.begin(r);
        p.boff[i + 1] = p.boff[i] + p.ns[i] + 1;
    }
}

// The shares of the tensor-memory path's CTAs.  A piece costs its blocks and
// about kPiece more (queries in, output out, an empty pipeline at both ends), so
// the shares are cut where the costs come out even: without that, a CTA of many
// short pieces (first chunks of prompts) took three times as long as one of
// long pieces.
void split_flash(const puzzlekv_store *s, FlashParams &f) {
    constexpr int kPiece = 4;
    // costs and blocks before each pair of every entry, one head
    struct Before {
        long long cost, blocks;
    };
    std::vector<std::vector<Before>> pairs(f.nseq);
    std::vector<Before> heads;  // before (entry, head), in order
    Before all{0, 0};
    for (int j = 0; j < f.nseq; ++j) {
        Before u{0, 0};
        for (int p = 0; (long long)p * FLASH_ROWS < (long long)f.n[j] * f.G; ++p) {
            pairs[j].push_back(u);
            const int nb = flash_blocks(f.T[j], f.n[j], f.G, p);
            u.cost += nb + kPiece;
            u.blocks += nb;
        }
        for (int h = 0; h < f.H; ++h, all.cost += u.cost, all.blocks += u.blocks) heads.push_back(all);
    }
    f.units = all.blocks;
    const int most = (int)std::min<long long>(std::min(s->num_sms, FLASH_MAX_CTAS), all.blocks);
    auto below = [](long long x, const Before &e) { return x < e.cost; };
    f.ctas = 0;
    long long last = -1;
    for (int c = 0; c < most; ++c) {
        const long long x = all.cost * c / most;
        const int eh = (int)(std::upper_bound(heads.begin(), heads.end(), x, below) - heads.begin()) - 1;
        const std::vector<Before> &u = pairs[eh / f.H];
        const long long r = x - heads[eh].cost;
        const int pair = (int)(std::upper_bound(u.begin(), u.end(), r, below) - u.begin()) - 1;
        const int b0 = (int)std::max<long long>(0, r - u[pair].cost - kPiece);
        const long long at = heads[eh].blocks + u[pair].blocks + b0;
        if (at == last) continue;  // no empty shares
        if (f.ctas) f.share[f.ctas - 1].units = at - last;
        f.share[f.ctas++] = {eh / f.H, eh % f.H, pair, b0, 0};
        last = at;
    }
    f.share[f.ctas - 1].units = all.blocks - last;
}

void plan_attention(const puzzlekv_store *s, int32_t layer, const int32_t *seq_ids, const int32_t *counts, int32_t B,
                    AttnPlan &pl) {
    const Layout &y = s->y;
    const float scale = (float)(1.4426950408889634074 / std::sqrt((double)y.d));
    const bool tensor = y.dtype == 1;
    int most_small = 0;
    if (tensor && !y.rope && !y.q4)
        for (int i = 0; i < B; ++i)
            if (counts[i] <= SMALL_ROWS / y.G) most_small = std::max(most_small, counts[i]);
    const int small_tokens = most_small && small_smem_bytes(y, most_small) ? most_small : 0;
    ChunkAttnParams &a = pl.a;
    a.H = y.H; a.Hq = y.Hq; a.G = y.G; a.d = y.d;
    a.scale_log2 = scale;
    pl.s.y = y;
    pl.s.scale_log2 = scale;
    pl.s.layer = layer;
    FlashParams &f = pl.f;
    f.H = y.H; f.Hq = y.Hq; f.G = y.G;
    f.scale_log2 = scale;
    rows_params(s, layer, pl.r);
    StageParams &g = pl.g;
    g.y = y;
    g.factor_pool = s->factor_pool;
    g.dense_pool = s->dense_pool;
    g.rope_base = pl.r.rope_base;
    g.rope_delta = pl.r.rope_delta;
    g.layer = layer;
    long tiles = 0;
    long long rows = 0, parts = 0;
    int off = 0;
    for (int i = 0; i < B; off += counts[i], ++i) {
        const int n = counts[i], T = length_of(s, seq_ids[i], layer), fw = first_window_page(y, T);
        if (n == 0) continue;
        pl.seqs[pl.nseq] = seq_ids[i];
        pl.lens[pl.nseq++] = T;
        if (n <= small_tokens) {
            SmallParams &p = pl.s;
            const int j = p.nseq++;
            p.seqs[j] = seq_ids[i]; p.T[j] = T; p.n[j] = n; p.off[j] = off; p.fw[j] = fw;
        } else if (tensor) {
            const int j = f.nseq++;
            f.T[j] = g.T[j] = T;
            f.n[j] = g.n[j] = n;
            f.off[j] = g.off[j] = off;
            g.seqs[j] = seq_ids[i];
            g.fw[j] = fw;
            f.blk_off[j + 1] = g.blk_off[j + 1] = f.blk_off[j] + (T + n + FLASH_KEYS - 1) / FLASH_KEYS;
        } else {
            const int j = a.nseq++;
            a.T[j] = T; a.n[j] = n; a.off[j] = off;
            a.koff[j] = rows;
            RowsParams &r = pl.r;
            r.seqs[j] = seq_ids[i]; r.T[j] = T; r.n[j] = T + n; r.off[j] = (int)rows; r.coff[j] = off;
            rows += T + n;
            tiles += (long)y.H * ((n * (long)y.G + 31) / 32);
        }
    }
    g.nseq = f.nseq;
    pl.r.nseq = a.nseq;
    size_t at = 0;
    if (pl.s.nseq) {
        SmallParams &p = pl.s;
        split_small(s, p);
        a.nseq = p.nseq;  // merged by the same kernel
        for (int j = 0; j < p.nseq; ++j) {
            a.T[j] = p.T[j]; a.n[j] = p.n[j]; a.off[j] = p.off[j];
            a.ns[j] = p.ns[j];
            a.poff[j] = p.poff[j] = parts;
            if (p.ns[j] > 1) parts += (long long)y.H * p.ns[j] * p.n[j] * y.G;
        }
    }
    if (f.nseq) {
        split_flash(s, f);
        const size_t blocks = (size_t)f.blk_off[f.nseq] * y.H;
        pl.images = at;
        pl.scales = pl.images + blocks * (2 * FLASH_KEYS * y.d * 2);
        pl.flash_parts = pl.scales + up256(blocks * sizeof(float2));
        at = pl.flash_parts + (f.ctas > 1 ? up256((size_t)2 * f.ctas * FLASH_ROWS * (y.d + 4) * 4) : 0);
    }
    if (rows) {
        // few query tiles: cut the keys so that about four CTAs land on every SM
        const int want = (int)std::max(1L, 4L * s->num_sms / tiles);
        for (int j = 0; j < a.nseq; ++j) {
            a.ns[j] = std::max(1, std::min(want, (a.T[j] + a.n[j]) / 64));
            a.poff[j] = parts;
            if (a.ns[j] > 1) parts += (long long)y.H * a.ns[j] * a.n[j] * y.G;
        }
        const size_t bytes = up256((size_t)rows * y.H * y.d * y.esz);
        pl.keys = at;
        pl.values = at + bytes;
        at += 2 * bytes;
    }
    pl.parts = at;
    pl.bytes = at + up256((size_t)parts * (y.d + 4) * 4);
}

// Pages of an appended sequence that leave the dense region without factors.
struct LeavePlan {
    std::vector<int> pages;
    bool gather = false;  // some page's rows are not all in the ring once the chunk is in
};

void plan_leaving(const puzzlekv_store *s, int b, int layer, int n, LeavePlan &lp) {
    const Layout &y = s->y;
    const int T0 = length_of(s, b, layer), T1 = T0 + n;
    lp.pages.clear();
    lp.gather = false;
    if (n == 0) return;
    const int last = (T1 - 1) / y.P;
    for (int p = std::max(y.sink_pages, (T0 - y.W) / y.P - 1); p <= last; ++p) {
        if (page_kind(p, T1, y.P, y.sink_tokens, y.W) == KIND_DENSE) continue;
        if (p * y.P < T0 && page_kind(p, T0, y.P, y.sink_tokens, y.W) == KIND_FACTORED) continue;
        if (T0 > 0 && has_factors(s, b, layer, p)) continue;
        lp.pages.push_back(p);
        if (p <= last - y.ring) lp.gather = true;
    }
}

size_t gather_bytes(const Layout &y, const LeavePlan &lp) {
    if (!lp.gather) return 0;
    const size_t rows = (size_t)(lp.pages.back() - lp.pages.front() + 1) * y.P;
    return 2 * up256(rows * y.H * y.d * y.esz);
}

// Do [a, a + na) and [b, b + nb) share a byte?
bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), z = reinterpret_cast<uintptr_t>(b);
    return na > 0 && nb > 0 && x < z + nb && z < x + na;
}

puzzlekv_status check_work(const void *work, size_t have, size_t need) {
    if (need == 0) return PUZZLEKV_OK;
    if (!work || (reinterpret_cast<uintptr_t>(work) & 255u) != 0)
        return fail(PUZZLEKV_ERR_INVALID_ARG, "the workspace must be non-NULL and 256-byte aligned");
    if (have < need) return fail(PUZZLEKV_ERR_INVALID_ARG, "the workspace holds %zu bytes, this call needs %zu", have, need);
    return PUZZLEKV_OK;
}

}  // namespace

extern "C" {

puzzlekv_status puzzlekv_chunk_workspace(const puzzlekv_store *s, int32_t layer, const int32_t *seq_ids,
                                         const int32_t *counts, int32_t B, size_t *attention_bytes,
                                         size_t *append_bytes) {
    return guarded([&]() -> puzzlekv_status {
        puzzlekv_status st = check_chunk(s, layer, seq_ids, counts, B);
        if (st != PUZZLEKV_OK) return st;
        if (attention_bytes) {
            AttnPlan pl;
            plan_attention(s, layer, seq_ids, counts, B, pl);
            *attention_bytes = pl.bytes;
        }
        if (append_bytes) {
            *append_bytes = 0;
            LeavePlan lp;
            for (int i = 0; i < B; ++i) {
                plan_leaving(s, seq_ids[i], layer, counts[i], lp);
                *append_bytes += gather_bytes(s->y, lp);
            }
        }
        return PUZZLEKV_OK;
    });
}

puzzlekv_status puzzlekv_chunk_attention(puzzlekv_store *s, int32_t layer, const void *q, const void *k, const void *v,
                                         void *out, const int32_t *seq_ids, const int32_t *counts, int32_t B,
                                         void *work, size_t work_bytes, void *stream) {
    NvtxRange nvtx_range("puzzlekv_chunk_attention");
    return guarded([&]() -> puzzlekv_status {
        puzzlekv_status st = check_chunk(s, layer, seq_ids, counts, B);
        if (st != PUZZLEKV_OK) return st;
        if (!q || !k || !v || !out || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out))
            return fail(PUZZLEKV_ERR_INVALID_ARG, "q, k, v and out must be non-NULL and 16-byte aligned");
        const Layout &y = s->y;
        AttnPlan pl;
        plan_attention(s, layer, seq_ids, counts, B, pl);
        if (pl.nseq == 0) return PUZZLEKV_OK;
        st = check_work(work, work_bytes, pl.bytes);
        if (st != PUZZLEKV_OK) return st;
        // A row of out is written after its own row of q is read, but beside reads
        // of the others and of the chunk's keys and values.
        size_t tokens = 0;
        for (int i = 0; i < B; ++i) tokens += counts[i];
        const size_t qb = tokens * y.Hq * y.d * y.esz, kb = tokens * y.H * y.d * y.esz;
        if (overlap(out, qb, k, kb) || overlap(out, qb, v, kb) || (out != q && overlap(out, qb, q, qb)))
            return fail(PUZZLEKV_ERR_INVALID_ARG, "out must not overlap k, v or (unless it is q) q");
        if (overlap(work, pl.bytes, q, qb) || overlap(work, pl.bytes, k, kb) || overlap(work, pl.bytes, v, kb) ||
            overlap(work, pl.bytes, out, qb))
            return fail(PUZZLEKV_ERR_INVALID_ARG, "the workspace must not overlap q, k, v or out");
        cudaStream_t strm = static_cast<cudaStream_t>(stream);
        st = refuse_pending(s, strm);
        if (st != PUZZLEKV_OK) return st;
        char *w = static_cast<char *>(work);
        wait_conversions(s, strm, pl.seqs, pl.lens, pl.nseq);
        s->after_decode = false;
        cudaError_t e = cudaSuccess;
        if (pl.f.nseq) {
            pl.g.k_new = static_cast<const char *>(k);
            pl.g.v_new = static_cast<const char *>(v);
            pl.g.images = w + pl.images;
            pl.g.scales = reinterpret_cast<float2 *>(w + pl.scales);
            pl.g.status = status_ptr(s);
            pl.f.q = static_cast<const char *>(q);
            pl.f.v_new = pl.g.v_new;
            pl.f.out = static_cast<char *>(out);
            pl.f.images = pl.g.images;
            pl.f.scales = pl.g.scales;
            pl.f.partials = reinterpret_cast<float *>(w + pl.flash_parts);
            pl.f.status = status_ptr(s);
            pl.g.hook = take_hook(s, FAIL_STAGE);
            pl.f.hook = take_hook(s, FAIL_FLASH);
            e = launch_stage(pl.g, s->num_sms, strm);
            if (e == cudaSuccess) e = launch_flash(pl.f, y.d, strm);
        }
        ChunkAttnParams &a = pl.a;
        a.q = static_cast<const char *>(q);
        a.out = static_cast<char *>(out);
        a.partials = reinterpret_cast<float *>(w + pl.parts);
        if (pl.s.nseq && e == cudaSuccess) {
            pl.s.factor_pool = s->factor_pool;
            pl.s.dense_pool = s->dense_pool;
            pl.s.q = a.q;
            pl.s.k_new = static_cast<const char *>(k);
            pl.s.v_new = static_cast<const char *>(v);
            pl.s.out = a.out;
            pl.s.partials = a.partials;
            pl.s.status = status_ptr(s);
            pl.s.hook = take_hook(s, FAIL_SMALL);
            e = launch_small(pl.s, strm);
        }
        if (pl.r.nseq && e == cudaSuccess) {
            RowsParams &r = pl.r;
            r.k_new = static_cast<const char *>(k);
            r.v_new = static_cast<const char *>(v);
            r.k_out = w + pl.keys;
            r.v_out = w + pl.values;
            r.row_stride = (size_t)y.H * y.d;
            r.head_stride = y.d;
            a.K = r.k_out;
            a.V = r.v_out;
            e = launch_rows(r, strm);
            if (e == cudaSuccess) e = launch_chunk_simple(a, strm);
        }
        if (a.nseq && e == cudaSuccess) e = launch_chunk_merge(a, y.dtype, strm);
        if (e != cudaSuccess) return cuda_fail(e, "chunk attention launch");
        return PUZZLEKV_OK;
    });
}

puzzlekv_status puzzlekv_append_chunk(puzzlekv_store *s, int32_t layer, const void *k, const void *v,
                                      const int32_t *seq_ids, const int32_t *counts, int32_t B, void *work,
                                      size_t work_bytes, void *stream) {
    NvtxRange nvtx_range("puzzlekv_append_chunk");
    return guarded([&]() -> puzzlekv_status {
        puzzlekv_status st = check_chunk(s, layer, seq_ids, counts, B);
        if (st != PUZZLEKV_OK) return st;
        if (!k || !v || !aligned16(k) || !aligned16(v))
            return fail(PUZZLEKV_ERR_INVALID_ARG, "k and v must be non-NULL and 16-byte aligned");
        const Layout &y = s->y;
        cudaStream_t strm = static_cast<cudaStream_t>(stream);
        std::vector<LeavePlan> leave(B);
        AppendChunkParams ap{};
        ap.y = y;
        ap.lengths = lengths_ptr(s);
        ap.desc = desc_ptr(s);
        ap.dense_pool = s->dense_pool;
        ap.k = static_cast<const char *>(k);
        ap.v = static_cast<const char *>(v);
        ap.layer = layer;
        ap.nseq = B;
        size_t need = 0;
        int grown[MAX_CALL_BATCH], off = 0;
        for (int i = 0; i < B; ++i) {
            plan_leaving(s, seq_ids[i], layer, counts[i], leave[i]);
            need += gather_bytes(y, leave[i]);
            ap.seqs[i] = seq_ids[i];
            ap.T[i] = length_of(s, seq_ids[i], layer);
            ap.n[i] = counts[i];
            ap.off[i] = off;
            grown[i] = ap.T[i] + counts[i];
            off += counts[i];
        }
        if (off == 0) return PUZZLEKV_OK;
        st = check_work(work, work_bytes, need);
        const size_t kb = (size_t)off * y.H * y.d * y.esz;
        if (st == PUZZLEKV_OK && (overlap(work, need, k, kb) || overlap(work, need, v, kb)))
            st = fail(PUZZLEKV_ERR_INVALID_ARG, "the workspace must not overlap k or v");
        if (st == PUZZLEKV_OK) st = refuse_capture(strm);
        if (st != PUZZLEKV_OK) return st;
        // a page converted in the background becomes factorized, or its ring
        // slot is written, only past its batch's deadline
        wait_conversions(s, strm, seq_ids, grown, B);
        s->after_decode = false;
        FactorParams fp{};
        fp.max_ql_iter = 30;
        fp.status = status_ptr(s);
        fp.y = y;
        fp.P = y.P;
        fp.d = y.d;
        fp.x_esz = y.esz;
        fp.factor_pool = s->factor_pool;
        cudaError_t e = cudaSuccess;
        // pages whose rows the ring will not hold: from a copy of their rows
        // (old rows of the ring, then the chunk's) made before the ring changes
        size_t at = 0;
        for (int i = 0; i < B && e == cudaSuccess; ++i) {
            const LeavePlan &lp = leave[i];
            if (!lp.gather) continue;
            const int lo = lp.pages.front(), rows = (lp.pages.back() - lo + 1) * y.P;
            const size_t half = gather_bytes(y, lp) / 2;
            RowsParams rp;
            rows_params(s, layer, rp);
            rp.k_new = ap.k;
            rp.v_new = ap.v;
            rp.k_out = static_cast<char *>(work) + at;
            rp.v_out = rp.k_out + half;
            rp.row_stride = y.d;
            rp.head_stride = (size_t)rows * y.d;
            rp.nseq = 1;
            rp.seqs[0] = seq_ids[i];
            rp.T[0] = ap.T[i];
            rp.lo[0] = lo * y.P;
            rp.n[0] = rows;
            rp.coff[0] = ap.off[i];
            e = launch_rows(rp, strm);
            fp.mode = FACT_MODE_PREFILL;
            const size_t shift = (size_t)lo * y.P * y.d * y.esz;  // page lo is the copy's first
            fp.k_src = rp.k_out - shift;
            fp.v_src = rp.v_out - shift;
            fp.seq = seq_ids[i];
            fp.T = rows;
            fp.layer0 = layer;
            fp.n_layers = 1;
            for (size_t a = 0; a < lp.pages.size() && e == cudaSuccess;) {  // runs of consecutive pages
                size_t z = a + 1;
                while (z < lp.pages.size() && lp.pages[z] == lp.pages[z - 1] + 1) ++z;
                fp.p_lo = lp.pages[a];
                fp.p_hi = lp.pages[z - 1] + 1;
                fp.n_jobs = (long)y.H * 2 * (fp.p_hi - fp.p_lo);
                e = launch_factorize(fp, s->num_sms, strm);
                a = z;
            }
            at += 2 * half;
        }
        if (e == cudaSuccess) e = launch_append_chunk(ap, strm);
        // the other leaving pages are whole in the ring
        fp.mode = FACT_MODE_CONVERT;
        fp.dense_pool = s->dense_pool;
        fp.layer = layer;
        fp.n_conv = 0;
        auto flush = [&]() {
            if (fp.n_conv == 0 || e != cudaSuccess) return;
            fp.n_jobs = (long)fp.n_conv * y.H * 2;
            e = launch_factorize(fp, s->num_sms, strm);
            fp.n_conv = 0;
        };
        for (int i = 0; i < B; ++i) {
            if (leave[i].gather) continue;
            for (int p : leave[i].pages) {
                if (fp.n_conv == MAX_CALL_BATCH) flush();
                fp.conv_seq[fp.n_conv] = seq_ids[i];
                fp.conv_page[fp.n_conv++] = p;
            }
        }
        flush();
        if (e != cudaSuccess) return cuda_fail(e, "chunk append launch");
        for (int i = 0; i < B; ++i) {
            if (counts[i] == 0) continue;
            const int b = seq_ids[i];
            if (ap.T[i] == 0) {
                reset_factors(s, b, layer, y.sink_pages);
                s->dense_lo[(size_t)b * y.L + layer] = y.sink_pages;
            }
            for (int p : leave[i].pages) set_factors(s, b, layer, p);
            grow_dense(s, b, layer, s->len[(size_t)b * y.L + layer] = grown[i]);
        }
        return PUZZLEKV_OK;
    });
}

puzzlekv_status puzzlekv_read_tokens(puzzlekv_store *s, int32_t layer, const int32_t *seq_ids, const int32_t *starts,
                                     const int32_t *counts, int32_t B, void *k, void *v, void *stream) {
    NvtxRange nvtx_range("puzzlekv_read_tokens");
    return guarded([&]() -> puzzlekv_status {
        puzzlekv_status st = check_list(s, seq_ids, B, "seq_ids");
        if (st != PUZZLEKV_OK) return st;
        const Layout &y = s->y;
        if (layer < 0 || layer >= y.L) return fail(PUZZLEKV_ERR_INVALID_ARG, "layer %d out of range", layer);
        if (!starts || !counts) return fail(PUZZLEKV_ERR_INVALID_ARG, "starts and counts must be non-NULL");
        if (!k || !v || !aligned16(k) || !aligned16(v))
            return fail(PUZZLEKV_ERR_INVALID_ARG, "k and v must be non-NULL and 16-byte aligned");
        RowsParams rp;
        rows_params(s, layer, rp);
        int lens[MAX_CALL_BATCH], off = 0;
        for (int i = 0; i < B; ++i) {
            const int T = length_of(s, seq_ids[i], layer);
            if (starts[i] < 0 || counts[i] < 0 || starts[i] > T || counts[i] > T - starts[i])
                return fail(PUZZLEKV_ERR_INVALID_ARG, "entry %d: rows [%d, %d + %d) of a sequence of %d tokens", i, starts[i],
                            starts[i], counts[i], T);
            rp.seqs[i] = seq_ids[i];
            lens[i] = rp.T[i] = T;
            rp.fw[i] = first_window_page(y, T);
            rp.lo[i] = starts[i];
            rp.n[i] = counts[i];
            rp.off[i] = off;
            off += counts[i];
        }
        if (off == 0) return PUZZLEKV_OK;
        const size_t kb = (size_t)off * y.H * y.d * y.esz;
        if (overlap(k, kb, v, kb)) return fail(PUZZLEKV_ERR_INVALID_ARG, "k and v must not overlap");
        rp.nseq = B;
        rp.k_out = static_cast<char *>(k);
        rp.v_out = static_cast<char *>(v);
        rp.row_stride = (size_t)y.H * y.d;
        rp.head_stride = y.d;
        cudaStream_t strm = static_cast<cudaStream_t>(stream);
        st = refuse_pending(s, strm);
        if (st != PUZZLEKV_OK) return st;
        wait_conversions(s, strm, seq_ids, lens, B);
        s->after_decode = false;
        rp.hook = take_hook(s, FAIL_READ);
        const cudaError_t e = launch_read(rp, s->num_sms, strm);
        if (e != cudaSuccess) return cuda_fail(e, "row read launch");
        return PUZZLEKV_OK;
    });
}

puzzlekv_status puzzlekv_load_factors(puzzlekv_store *s, int32_t layer, int32_t seq, int32_t page0, int32_t n,
                                      const void *LK, const void *RK, const void *LV, const void *RV, void *stream) {
    NvtxRange nvtx_range("puzzlekv_load_factors");
    return guarded([&]() -> puzzlekv_status {
        puzzlekv_status st = check_list(s, &seq, 1, "seq");
        if (st != PUZZLEKV_OK) return st;
        const Layout &y = s->y;
        if (layer < 0 || layer >= y.L) return fail(PUZZLEKV_ERR_INVALID_ARG, "layer %d out of range", layer);
        if (y.q4) return fail(PUZZLEKV_ERR_UNSUPPORTED, "INT4 records take no plain factors");
        const int complete = length_of(s, seq, layer) / y.P;
        if (n < 0 || page0 < y.sink_pages || page0 > complete || n > complete - page0)
            return fail(PUZZLEKV_ERR_INVALID_ARG, "pages [%d, %d + %d): sequence %d has complete pages [%d, %d) past its sink",
                        page0, page0, n, seq, y.sink_pages, complete);
        if (n == 0) return PUZZLEKV_OK;
        if (!LK || !RK || !LV || !RV || !aligned16(LK) || !aligned16(RK) || !aligned16(LV) || !aligned16(RV))
            return fail(PUZZLEKV_ERR_INVALID_ARG, "factors must be non-NULL and 16-byte aligned");
        cudaStream_t strm = static_cast<cudaStream_t>(stream);
        st = refuse_capture(strm);
        if (st != PUZZLEKV_OK) return st;
        wait_conversions(s, strm, nullptr, nullptr, 0, true);  // a pending batch may hold one of the pages
        s->after_decode = false;
        LoadFactorsParams p{};
        p.y = y;
        p.factor_pool = s->factor_pool;
        p.LK = static_cast<const char *>(LK);
        p.RK = static_cast<const char *>(RK);
        p.LV = static_cast<const char *>(LV);
        p.RV = static_cast<const char *>(RV);
        p.layer = layer;
        p.seq = seq;
        p.page0 = page0;
        p.n = n;
        const cudaError_t e = launch_load_factors(p, strm);
        if (e != cudaSuccess) return cuda_fail(e, "factor load launch");
        for (int g = page0; g < page0 + n; ++g) set_factors(s, seq, layer, g);
        return PUZZLEKV_OK;
    });
}

puzzlekv_status puzzlekv_copy_sequences(puzzlekv_store *s, const int32_t *src_ids, const int32_t *dst_ids, int32_t n,
                                        void *stream) {
    NvtxRange nvtx_range("puzzlekv_copy_sequences");
    return guarded([&]() -> puzzlekv_status {
        puzzlekv_status st = check_list(s, dst_ids, n, "dst_ids");
        if (st != PUZZLEKV_OK) return st;
        if (!src_ids) return fail(PUZZLEKV_ERR_INVALID_ARG, "src_ids is NULL");
        const Layout &y = s->y;
        CopyParams p{};
        p.y = y;
        p.factor_pool = s->factor_pool;
        p.dense_pool = s->dense_pool;
        p.lengths = lengths_ptr(s);
        p.desc = desc_ptr(s);
        p.status = status_ptr(s);
        for (int i = 0; i < n; ++i) {
            const int b = src_ids[i];
            if (b < 0 || b >= y.Bmax) return fail(PUZZLEKV_ERR_INVALID_ARG, "src_ids: slot %d out of range", b);
            const int T = length_of(s, b, 0);
            if (T < 1) return fail(PUZZLEKV_ERR_INVALID_ARG, "src_ids: sequence %d holds no tokens", b);
            for (int l = 1; l < y.L; ++l)
                if (length_of(s, b, l) != T)
                    return fail(PUZZLEKV_ERR_INVALID_ARG, "src_ids: sequence %d has layers of different lengths", b);
            if (b == dst_ids[i]) continue;
            int j = 0;
            while (j < p.nsrc && p.src[j] != b) ++j;
            if (j == p.nsrc) {
                p.src[j] = b;
                p.T[j] = T;
                const int pages = (T + y.P - 1) / y.P;
                int lo = pages;  // first page past the sink that some layer still holds densely
                for (int l = 0; l < y.L; ++l) {
                    const size_t x = (size_t)b * y.L + l;
                    int upto = s->conv_upto[x];
                    for (int g = (int)s->marked[x].size() - 1; g >= upto; --g)
                        if (s->marked[x][g]) {
                            upto = g + 1;
                            break;
                        }
                    p.upto[j] = std::max(p.upto[j], upto);
                    lo = std::min(lo, std::max(s->dense_lo[x], y.sink_pages));
                }
                for (int g = 0; g < std::min(y.sink_pages, pages); ++g) p.slots[j] |= 1ull << y.dense_slot(g);
                for (int g = lo; g < pages; ++g) p.slots[j] |= 1ull << y.dense_slot(g);
                ++p.nsrc;
            }
            p.dst[p.npair] = dst_ids[i];
            p.pair_src[p.npair] = j;
            for (int l = 0; l < y.L; ++l)
                p.had[p.npair] = std::max(p.had[p.npair], (length_of(s, dst_ids[i], l) + y.P - 1) / y.P);
            ++p.npair;
        }
        if (p.npair == 0) return PUZZLEKV_OK;
        cudaStream_t strm = static_cast<cudaStream_t>(stream);
        st = refuse_capture(strm);
        if (st != PUZZLEKV_OK) return st;
        // the sources' bookkeeping before any destination's changes
        std::vector<int> len, upto, lo;
        std::vector<std::vector<uint8_t>> marked;
        for (int j = 0; j < p.nsrc; ++j)
            for (int l = 0; l < y.L; ++l) {
                const size_t x = (size_t)p.src[j] * y.L + l;
                len.push_back(s->len[x]);
                upto.push_back(s->conv_upto[x]);
                lo.push_back(s->dense_lo[x]);
                marked.push_back(s->marked[x]);
            }
        wait_conversions(s, strm, nullptr, nullptr, 0, true);
        s->after_decode = false;
        p.hook = take_hook(s, FAIL_COPY);
        const cudaError_t e = launch_copy(p, s->num_sms, strm);
        if (e != cudaSuccess) return cuda_fail(e, "sequence copy launch");
        for (int i = 0; i < p.npair; ++i)
            for (int l = 0; l < y.L; ++l) {
                const size_t x = (size_t)p.dst[i] * y.L + l, z = (size_t)p.pair_src[i] * y.L + l;
                s->len[x] = len[z];
                s->conv_upto[x] = upto[z];
                s->dense_lo[x] = lo[z];
                s->marked[x] = marked[z];
            }
        return PUZZLEKV_OK;
    });
}

puzzlekv_status puzzlekv_truncate_sequences(puzzlekv_store *s, const int32_t *seq_ids, const int32_t *lengths, int32_t B,
                                            void *stream) {
    NvtxRange nvtx_range("puzzlekv_truncate_sequences");
    return guarded([&]() -> puzzlekv_status {
        puzzlekv_status st = check_list(s, seq_ids, B, "seq_ids");
        if (st != PUZZLEKV_OK) return st;
        if (!lengths) return fail(PUZZLEKV_ERR_INVALID_ARG, "lengths is NULL");
        const Layout &y = s->y;
        TruncateParams p{};
        p.y = y;
        p.lengths = lengths_ptr(s);
        p.desc = desc_ptr(s);
        p.nseq = B;
        for (int i = 0; i < B; ++i) {
            const int b = seq_ids[i], T = lengths[i];
            if (T < 0) return fail(PUZZLEKV_ERR_INVALID_ARG, "lengths[%d] is negative", i);
            const int pages = (T + y.P - 1) / y.P, fw = first_window_page(y, T);
            for (int l = 0; l < y.L; ++l) {
                const int have = length_of(s, b, l);
                if (T > have)
                    return fail(PUZZLEKV_ERR_INVALID_ARG, "sequence %d holds %d tokens in layer %d, fewer than %d", b, have, l, T);
                if (T < have && fw < pages && fw >= y.sink_pages && fw < s->dense_lo[(size_t)b * y.L + l])
                    return fail(PUZZLEKV_ERR_INVALID_ARG,
                                "sequence %d cannot go back to %d tokens: page %d would be dense and its rows are gone "
                                "(kept from page %d on)", b, T, fw, s->dense_lo[(size_t)b * y.L + l]);
                p.had[i] = std::max(p.had[i], (have + y.P - 1) / y.P);
            }
            p.seqs[i] = b;
            p.T[i] = T;
        }
        cudaStream_t strm = static_cast<cudaStream_t>(stream);
        st = refuse_capture(strm);
        if (st != PUZZLEKV_OK) return st;
        wait_conversions(s, strm, nullptr, nullptr, 0, true);  // a pending batch may hold a page that is cut off
        s->after_decode = false;
        const cudaError_t e = launch_truncate(p, strm);
        if (e != cudaSuccess) return cuda_fail(e, "truncate launch");
        for (int i = 0; i < B; ++i)
            for (int l = 0; l < y.L; ++l) {
                const size_t x = (size_t)p.seqs[i] * y.L + l;
                const int T = p.T[i], complete = T / y.P;
                s->len[x] = T > 0 ? T : -1;
                if (T == 0) {
                    reset_factors(s, p.seqs[i], l, y.sink_pages);
                    s->dense_lo[x] = y.sink_pages;
                    continue;
                }
                // pages from the cut on are written anew: they will be in the ring
                s->dense_lo[x] = std::min(s->dense_lo[x], std::max(y.sink_pages, complete));
                // a page cut into is filled again with other tokens: its factors are void
                s->conv_upto[x] = std::max(y.sink_pages, std::min(s->conv_upto[x], complete));
                std::vector<uint8_t> &m = s->marked[x];
                for (size_t g = complete; g < m.size(); ++g) m[g] = 0;
            }
        return PUZZLEKV_OK;
    });
}

}  // extern "C"
