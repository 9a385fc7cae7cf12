// Kernel parameter blocks and launchers (private to the library).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "layout.h"

namespace pkv {

enum { FACT_MODE_BATCH = 0, FACT_MODE_PREFILL = 1, FACT_MODE_CONVERT = 2, FACT_MODE_CONVERT_LIST = 3,
       FACT_MODE_BATCH_Q4 = 4 };

struct FactorParams {
    int mode;
    long n_jobs;
    int max_ctas;  // grid size cap (0: the default, a few CTAs per SM looping over the jobs)
    int max_ql_iter;  // QL iterations allowed per eigenvalue
    int *status;  // device status words (may be null in batch mode)
    // batch mode: X[n][P][d] -> L[n][P][r], R[n][r][d], sigma[n][P]
    const char *x_base;
    int x_esz, out_esz, P, d, r;
    char *L_out, *R_out;
    float *sigma;
    // store modes
    Layout y;
    char *factor_pool;
    const char *dense_pool;
    // prefill: pages [p_lo, p_hi) of sequence `seq`, layers layer0 ..
    // layer0 + n_layers - 1, from k_src / v_src ([n_layers][H][T][d])
    const char *k_src, *v_src;
    int seq, T, p_lo, p_hi, layer0, n_layers;
    // convert: one page per call entry of `layer`
    int layer, n_conv;
    int conv_seq[MAX_CALL_BATCH], conv_page[MAX_CALL_BATCH];
    // convert list: device int2 {seq << 8 | layer, page} per page, 2 H jobs each
    const int2 *conv_list;
    // batch INT4 mode: pages X[n][P][d] (x_base) of one kind (0 key, 1 value)
    // -> INT4 records q4_records[n][y.rec_bytes] (that kind's code stream and
    // scales), and optionally the absorbed fp32 factors the codes quantize,
    // q4_L[n][P][rank padded to 8] and q4_R[n][rank padded][d]
    int q4_kind;
    char *q4_records;
    float *q4_L, *q4_R;
};

constexpr int MAX_BOUNDS = 384;  // page bounds of all CTAs of one bf16 decode launch

struct DecodeParams {
    Layout y;
    const char *factor_pool, *dense_pool;
    const int *lengths, *desc;
    const char *q;      // [B][Hq][d] storage dtype
    float *partials;    // workspace split partials
    int *tickets;       // workspace split tickets, zero between launches
    int wait_first;     // bf16 kernel: the preceding launch may have written factor records
    // failure-path test hook (0 = off): 1 = the first unit of CTA (0, 0, 0)
    // expects bytes no copy delivers, 2 = so does every split merge; the waits
    // of this launch give up after wait_ns (0 = the library's limit)
    int inject;
    unsigned long long wait_ns;
    float *out;         // [B][Hq][d]
    int *status;
    int layer, chunk, nseq;
    int stages;         // shared-memory ring depth (bf16 kernel)
    int seqs[MAX_CALL_BATCH];
    int lens[MAX_CALL_BATCH];       // tokens attended per call entry (host mirror, after any append)
    // fused append (decode step): the token at position lens - 1 comes from
    // k_new / v_new ([B][H][d]); the kernel writes it into its dense page and
    // updates the device page table (new page, page converted before launch)
    const char *k_new, *v_new;
    int append;
    int conv_page[MAX_CALL_BATCH];  // page converted before this launch, or -1
    // bf16 kernel, filled by its launcher: CTA r of call entry i streams pages
    // [bounds[boff[i] + r], bounds[boff[i] + r + 1]) (PageSplit), of which
    // [fs[i], fw[i]) are the sequence's factorized pages
    int boff[MAX_CALL_BATCH], fs[MAX_CALL_BATCH], fw[MAX_CALL_BATCH];
    int nsplit[MAX_CALL_BATCH];     // CTAs per (sequence, KV head) of call entry i
    int bounds[MAX_BOUNDS];
    int *lengths_out, *desc_out;    // device page table (written when append)
    const float2 *rope_base, *rope_delta;  // keys stored before RoPE: (cos, sin) tables (Layout)
};

constexpr int MAX_DENSE_PAGES = 64;  // dense pages of one sequence (sink + window + filling)

struct SeqInitParams {
    Layout y;
    int *lengths, *desc;
    char *dense_pool;
    const char *k_src, *v_src;  // [n_layers][H][T][d]: layers layer0 .. layer0 + n_layers - 1
    int seq, T, n_dense, layer0, n_layers;
    int dense_pages[MAX_DENSE_PAGES];
};

struct AppendParams {
    Layout y;
    int *lengths, *desc;
    char *dense_pool;
    const char *k, *v;  // [B][H][d]
    int layer, nseq;
    int seqs[MAX_CALL_BATCH];
    int pos[MAX_CALL_BATCH];       // token position written (old length)
    int conv_page[MAX_CALL_BATCH]; // page converted by this call, or -1
};

// Failure-path test hook of the chunk kernels: with `inject` set, the first
// barrier that the launch's first CTA fills expects 16 bytes that no copy
// delivers, and waits give up after `wait_ns` (0: the library's limit).
enum { FAIL_NONE = 0, FAIL_SMALL = 1, FAIL_STAGE = 2, FAIL_FLASH = 3, FAIL_READ = 4, FAIL_COPY = 5 };
struct WaitHook {
    int inject = 0;
    uint64_t wait_ns = 0;
#if defined(__CUDACC__)
    __device__ __forceinline__ uint32_t extra() const { return inject && blockIdx.x == 0 && blockIdx.y == 0 ? 16u : 0u; }
    __device__ __forceinline__ uint64_t limit() const { return wait_ns ? wait_ns : WAIT_NS; }
#endif
};

// Rows of the cache of a list of sequences, as attention sees them: row t of
// call entry i comes from the store for t < T[i] (factorized pages rebuilt as
// L R, by launch_read with keys stored before RoPE turned) and from the chunk
// k_new / v_new ([sum n][H][d], entry i's tokens from row coff[i] on) beyond.
// Rows lo[i] .. lo[i] + n[i] - 1 go to k_out / v_out: row r of the call's rows
// (entry i's from off[i] on) at element r * row_stride + head * head_stride.
struct RowsParams {
    Layout y;
    const char *factor_pool, *dense_pool;
    const float2 *rope_base, *rope_delta;
    const char *k_new, *v_new;
    char *k_out, *v_out;
    int *status;
    size_t row_stride, head_stride;  // elements
    int layer, nseq;
    int seqs[MAX_CALL_BATCH], T[MAX_CALL_BATCH], lo[MAX_CALL_BATCH], n[MAX_CALL_BATCH];
    int off[MAX_CALL_BATCH], coff[MAX_CALL_BATCH];
    int fw[MAX_CALL_BATCH];  // launch_read: page after the last factorized one
    int page_off[MAX_CALL_BATCH + 1];  // pages touched by the entries before (filled by the launcher)
    WaitHook hook;
};

// Chunk append: rows T[i] .. T[i] + n[i] - 1 of entry i, from k / v ([sum
// n][H][d], entry i's from off[i] on), into the dense pages still in the
// sink or the ring at length T[i] + n[i]; lengths and page kinds follow.
struct AppendChunkParams {
    Layout y;
    int *lengths, *desc;
    char *dense_pool;
    const char *k, *v;
    int layer, nseq;
    int seqs[MAX_CALL_BATCH], T[MAX_CALL_BATCH], n[MAX_CALL_BATCH], off[MAX_CALL_BATCH];
};

// Lengths and page kinds of the listed sequences at a new (shorter) length T[i]
// in every layer; had[i] is the number of pages described before.
struct TruncateParams {
    Layout y;
    int *lengths, *desc;
    int nseq;
    int seqs[MAX_CALL_BATCH], T[MAX_CALL_BATCH], had[MAX_CALL_BATCH];
};

// Plain factors of n pages from page0 on into their records: LK [H][n][P][rk],
// RK [H][n][rk][d], LV [H][n][P][rv], RV [H][n][rv][d], storage dtype.
struct LoadFactorsParams {
    Layout y;
    char *factor_pool;
    const char *LK, *RK, *LV, *RV;
    int layer, seq, page0, n;
};

// Every listed destination slot takes its source's pages, as if all were
// copied at once: src[j] are the distinct sources; pair i copies source
// pair_src[i] (an index into src) to slot dst[i].
struct CopyParams {
    Layout y;
    char *factor_pool, *dense_pool;
    int *lengths, *desc;
    int *status;
    int nsrc, npair;
    int src[MAX_CALL_BATCH], T[MAX_CALL_BATCH];          // per source: slot, length
    int upto[MAX_CALL_BATCH];                            // page after its last factor record
    unsigned long long slots[MAX_CALL_BATCH];            // its dense slots in use
    int dst[MAX_CALL_BATCH], pair_src[MAX_CALL_BATCH];
    int had[MAX_CALL_BATCH];                             // pages the destination's table described
    // filled by the launcher
    int max_upto, tile;
    unsigned long long any_slots;
    WaitHook hook;
};

// Attention of a chunk of queries over rows laid out densely, and the merge
// of split states.  Entry i holds n[i] tokens (rows off[i] .. of q and out,
// [sum n][Hq][d]); its T[i] + n[i] key / value rows start at row koff[i] of K /
// V ([rows][H][d]); query token j sees the first T[i] + j + 1.  Row r of the
// n G query rows of (entry, KV head) is token r / G, head r % G.  With ns[i] >
// 1 the keys are cut into ns[i] ranges whose states (m in log2 units, l, two
// pad floats, o[d]) go to row poff[i] + (head ns[i] + split) n[i] G + r of
// `partials`.
struct ChunkAttnParams {
    int H, Hq, G, d, nseq;
    float scale_log2;  // log2(e) / sqrt(d)
    const char *q;
    const char *K, *V;
    char *out;
    float *partials;
    int T[MAX_CALL_BATCH], n[MAX_CALL_BATCH], off[MAX_CALL_BATCH], ns[MAX_CALL_BATCH];
    long long koff[MAX_CALL_BATCH], poff[MAX_CALL_BATCH];
    int tile_off[MAX_CALL_BATCH + 1];  // CTAs of the entries before (filled by the launcher)
};

constexpr int FLASH_ROWS = 256, FLASH_KEYS = 128;  // query rows of a pair of tiles, keys of a block

// Chunk attention on the fifth-generation tensor cores (bf16 stores).  The
// entries' rows 0 .. T + n - 1 are laid out as fp16 operand images, one pair
// (keys [128][d], values transposed [d][128], both K-major in the 128-byte
// swizzle) per KV head and block of 128 positions: entry i, head h, block b at
// index (blk_off[i] H + h nblk(i) + b), nblk(i) = ceil((T[i] + n[i]) / 128).
// scales holds each block's powers of two (key, value): row = image 2^scale.  A
// value block whose chunk rows held infinities or NaN (zeros in the image) has a
// quarter added to the magnitude of its power.
struct StageParams {
    Layout y;
    const char *factor_pool, *dense_pool;
    const float2 *rope_base, *rope_delta;
    const char *k_new, *v_new;
    char *images;
    float2 *scales;
    int *status;
    int layer, nseq;
    int seqs[MAX_CALL_BATCH], T[MAX_CALL_BATCH], n[MAX_CALL_BATCH], off[MAX_CALL_BATCH];
    int fw[MAX_CALL_BATCH];  // page after the last factorized one (pages [sink_pages, fw) are)
    int blk_off[MAX_CALL_BATCH + 1];
    WaitHook hook;
};

// The query rows of (entry, KV head) are cut into pairs of 128-row tiles; pair
// p attends blocks 0 .. flash_blocks() - 1.  All (entry, head, pair, block)
// units in this order are shared out evenly over ctas CTAs; the states of
// pairs cut between CTAs go to partials ([2 ctas][256][d + 4]).
constexpr int FLASH_MAX_CTAS = 256;
struct FlashParams {
    int H, Hq, G, nseq, ctas;
    float scale_log2;
    const char *q;
    const char *v_new;
    char *out;
    const char *images;
    const float2 *scales;
    float *partials;
    int *status;
    int T[MAX_CALL_BATCH], n[MAX_CALL_BATCH], off[MAX_CALL_BATCH], blk_off[MAX_CALL_BATCH + 1];
    long long units;  // of all entries
    // share of CTA c: units[c] units from block b0 of (entry, head, pair) on
    struct Share {
        int i, h, pair, b0;
        long long units;
    } share[FLASH_MAX_CTAS];
    WaitHook hook;
};

// Blocks that pair p of an entry of T cached and n new tokens attends.
PKV_HD int flash_blocks(int T, int n, int G, int p) {
    const int last = (p + 1) * FLASH_ROWS < n * G ? (p + 1) * FLASH_ROWS : n * G;
    return (T + (last - 1) / G) / FLASH_KEYS + 1;
}

// Attention of a few tokens per sequence straight over the pages (bf16 stores
// with keys as stored): CTA (split, KV head) streams the units of its entry's
// pages [bounds[boff + split], bounds[boff + split + 1]) for all the entry's
// query rows; the last split also takes the chunk.  States of entries with
// several splits go to the rows of ChunkAttnParams::partials.
constexpr int SMALL_ROWS = 128;        // query rows per (entry, KV head)
constexpr int SMALL_BOUNDS = 1024;
struct SmallParams {
    Layout y;
    const char *factor_pool, *dense_pool;
    const char *q, *k_new, *v_new;
    char *out;
    float *partials;
    int *status;
    float scale_log2;
    int layer, nseq;
    int slots, unit_bytes, chunk_bytes;  // filled by the launcher
    int seqs[MAX_CALL_BATCH], T[MAX_CALL_BATCH], n[MAX_CALL_BATCH], off[MAX_CALL_BATCH], ns[MAX_CALL_BATCH];
    int fw[MAX_CALL_BATCH];
    int boff[MAX_CALL_BATCH + 1];  // first bound of each entry; split numbers run boff[i] - i ..
    long long poff[MAX_CALL_BATCH];
    int bounds[SMALL_BOUNDS];
    WaitHook hook;
};
// Shared memory that a launch for these entries would take (0: they do not fit).
size_t small_smem_bytes(const Layout &y, int most_tokens);
cudaError_t launch_small(SmallParams &p, cudaStream_t st);

cudaError_t launch_stage(const StageParams &p, int num_sms, cudaStream_t st);
cudaError_t launch_flash(const FlashParams &p, int d, cudaStream_t st);

// fp32 stores: any rows.  bf16 stores: dense and chunk rows, keys as stored.
cudaError_t launch_rows(RowsParams &p, cudaStream_t st);
// Rows of the cache alone (no chunk rows), any store.
cudaError_t launch_read(RowsParams &p, int num_sms, cudaStream_t st);
cudaError_t launch_append_chunk(const AppendChunkParams &p, cudaStream_t st);
cudaError_t launch_truncate(const TruncateParams &p, cudaStream_t st);
cudaError_t launch_load_factors(const LoadFactorsParams &p, cudaStream_t st);
cudaError_t launch_copy(CopyParams &p, int num_sms, cudaStream_t st);
cudaError_t launch_chunk_simple(ChunkAttnParams &p, cudaStream_t st);  // fp32
cudaError_t launch_chunk_merge(const ChunkAttnParams &p, int dtype, cudaStream_t st);

cudaError_t launch_factorize(const FactorParams &p, int num_sms, cudaStream_t st);
cudaError_t launch_seq_init(const SeqInitParams &p, cudaStream_t st);
cudaError_t launch_append(const AppendParams &p, cudaStream_t st);
// Chooses pages per CTA (p.chunk) for one wave over total_pages pages
// (all listed sequences and KV heads), then launches.
cudaError_t launch_decode(DecodeParams &p, long total_pages, int max_pages, int num_sms, cudaStream_t st);
// Dynamic shared memory the tensor-core decode kernel of this layout's path
// needs in its runtime-rank form (0 for fp32 stores).
size_t decode_smem_bytes(const Layout &y);
constexpr size_t MAX_DECODE_SMEM = 227 * 1024;  // opt-in shared memory per CTA on sm_103a

}  // namespace pkv
