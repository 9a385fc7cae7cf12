// The host handle of a store and what the C ABI's entry points share (private
// to the library): errors, the length mirror and its bookkeeping, and the
// ordering of background conversions.
#pragma once
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>
#include <stdint.h>

#include <algorithm>
#include <vector>

#include "../../include/puzzlekv.h"
#include "layout.h"

namespace pkv {

// Record the calling thread's error message; both return the status to pass on.
puzzlekv_status fail(puzzlekv_status st, const char *fmt, ...);
puzzlekv_status cuda_fail(cudaError_t e, const char *what);

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// An NVTX range around a call of the C ABI, seen by profilers (free when
// none is attached).
struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange &) = delete;
    NvtxRange &operator=(const NvtxRange &) = delete;
};

}  // namespace pkv

struct puzzlekv_store {
    puzzlekv_config cfg;
    pkv::Layout y;
    char *dense_pool, *factor_pool, *page_table, *workspace;
    std::vector<int> len;    // host mirror [seq][layer]; -1 = empty slot
    // Which pages have factor records, per (seq, layer): every page in
    // [sink_pages, conv_upto) and, above it, the pages marked in `marked`
    // (factorized out of order by a page-list call).
    std::vector<int> conv_upto;                   // [seq][layer]
    std::vector<std::vector<uint8_t>> marked;     // [seq][layer][page], allocated on first use
    // First page past the sink whose rows the dense ring still holds, per
    // (seq, layer): a prompt's first dense page, then, as the ring comes
    // round, the oldest page not overwritten.  A sequence can be cut back to
    // any length whose dense pages start at or after it.
    std::vector<int> dense_lo;                    // [seq][layer]
    std::vector<int2> job_host;  // staging of the batched-conversion job list
    bool after_decode = false;   // the store's latest launch was a decode launch
    int fail_next = 0;           // failure-path test hook for the next decode launch (0 = off)
    uint64_t fail_wait_ns = 0;   // its waits' limit
    int fail_chunk = 0;          // the same for the next launch of one chunk kernel (FAIL_* in kernels.h)
    uint64_t fail_chunk_ns = 0;
    int num_sms;
    // Batched conversions run on an internal low-priority stream.  A batch's
    // factor records are first read when one of its pages becomes
    // factorized, i.e. when its sequence reaches deadline[seq] tokens; every
    // stream whose calls attend at or past that length waits for the batch,
    // until it is known to have finished.
    struct ConvBatch {
        cudaEvent_t done = nullptr;
        bool pending = false;       // queued, and not known to have finished
        // The streams ordered after it.  Ids, unlike handles, are not used again
        // for later streams, but a captured stream's cannot be asked for.
        struct Waiter {
            unsigned long long id;
            cudaStream_t stream;
        };
        std::vector<Waiter> waited;
        std::vector<int> deadline;  // [seq]: length at which the batch's first page is factorized
        std::vector<char> uses;     // [seq][layer]: the batch writes factor records of that layer
    };
    cudaStream_t conv_stream = nullptr;
    cudaEvent_t conv_ready = nullptr;  // caller's stream position a batch starts after
    std::vector<ConvBatch> batches;    // ring
    int next_batch = 0;
    ~puzzlekv_store() {
        if (conv_stream) cudaStreamSynchronize(conv_stream);
        for (auto &cb : batches)
            if (cb.done) cudaEventDestroy(cb.done);
        if (conv_ready) cudaEventDestroy(conv_ready);
        if (conv_stream) cudaStreamDestroy(conv_stream);
    }
};

namespace pkv {

inline int *lengths_ptr(puzzlekv_store *s) { return reinterpret_cast<int *>(s->page_table); }
inline int *desc_ptr(puzzlekv_store *s) { return reinterpret_cast<int *>(s->page_table + s->y.desc_offset); }
inline int *status_ptr(puzzlekv_store *s) { return reinterpret_cast<int *>(s->workspace); }

// Factor-record bookkeeping of (seq b, layer l).
inline bool has_factors(const puzzlekv_store *s, int b, int l, int p) {
    const size_t i = (size_t)b * s->y.L + l;
    if (p < s->conv_upto[i]) return p >= s->y.sink_pages;
    const std::vector<uint8_t> &m = s->marked[i];
    return (size_t)p < m.size() && m[p] != 0;
}
inline void set_factors(puzzlekv_store *s, int b, int l, int p) {
    const size_t i = (size_t)b * s->y.L + l;
    int &upto = s->conv_upto[i];
    std::vector<uint8_t> &m = s->marked[i];
    if (p < upto) return;
    if (m.size() < (size_t)s->y.n_pg_max) m.assign(s->y.n_pg_max, 0);
    m[p] = 1;
    while (upto < s->y.n_pg_max && m[upto]) m[upto++] = 0;  // extend the prefix over marked pages
}
inline void reset_factors(puzzlekv_store *s, int b, int l, int upto) {
    const size_t i = (size_t)b * s->y.L + l;
    s->conv_upto[i] = upto;
    std::vector<uint8_t>().swap(s->marked[i]);
}
// Sequence b of layer l has grown to T tokens, rows written in its ring.
inline void grow_dense(puzzlekv_store *s, int b, int l, int T) {
    int &lo = s->dense_lo[(size_t)b * s->y.L + l];
    lo = std::max(lo, (T - 1) / s->y.P - s->y.ring + 1);
}

// Has the batch finished on the device?  (Also while some stream is captured.)
bool batch_finished(const puzzlekv_store::ConvBatch &cb);
// Make `strm` wait for a batch, unless it has finished or `strm` has waited
// already.  Returns true if a wait was inserted.
bool wait_batch(puzzlekv_store::ConvBatch &cb, cudaStream_t strm);
// Make `strm` wait for every pending background conversion batch that the
// listed sequences (at the given lengths) reach, or for all of them when
// `all` is set.  Returns true if a wait was inserted.
bool wait_conversions(puzzlekv_store *s, cudaStream_t strm, const int32_t *seq_ids, const int *lens, int B,
                      bool all = false);

}  // namespace pkv
