/*
 * bgtq.h -- C ABI of the Block-GTQ packed KV-cache library for B200 (sm_100a).
 *
 * Block-GTQ ("RoPE-Aware Bit Allocation for KV-Cache Quantization", Liang,
 * Zhang, Jia; arXiv 2606.24033 abstract and the blockgtq README) quantises
 * the key cache per RoPE 2-D frequency block: a label-free Q/K energy score
 * per block, greedy integer bit widths by marginal gain under a fixed
 * average, then the TurboQuant-MSE (TQ-MSE) encoder; a packed-cache serving
 * path decodes attention straight from the codes.  This library implements
 * that hot path:
 *
 *   bgtq_allocate       energy score per block + greedy allocation + tables
 *   bgtq_encode_append  rotate, normalise, Lloyd-Max quantise, bit-pack K/V
 *   bgtq_encode_append_rope  the same from K before RoPE (RoPE fused in)
 *   bgtq_rotate_query   the query in each width group's rotated basis
 *   bgtq_decode_attn    one GQA decode step over the packed cache
 *   bgtq_decode_step    encode_append of a step's rows + decode_attn in one call
 *   bgtq_decode_attn_buffered  decode with fp16 sink / recent-window rows
 *   bgtq_decode_step_buffered  the same after a step's appends, in one call
 *   bgtq_logit_mae      per-layer logit error of the packed keys (diagnostic)
 *   bgtq_set_block_table  page table of a paged cache
 *
 * Beside the packed cache, an 8-bit one for layers that 4 bits do not hold:
 *
 *   bgtq_byte_append       e4m3 or int8 codes, one scale per 64 positions and head
 *   bgtq_byte_decode_attn  attention over it for 1..16 tokens a sequence, with
 *                          capped, distance-biased, windowed, prefix- and
 *                          document-masked scores
 *
 * For both caches:
 *
 *   bgtq_copy_pages / _fork_sequences / _resize_sequences / _compact_pages
 *                          pages of a paged cache shared, copied, freed,
 *                          reserved and moved together
 *   bgtq_rope_axes         rotary positions over one or several axes for the
 *                          query and key rows of a step
 *
 * Conventions
 *  - Every function returns 0 (BGTQ_OK) or a negative BGTQ_ERR_* code and
 *    never throws or aborts.  Argument checks happen before any launch; a
 *    call that fails its checks launches nothing.
 *  - Device buffers are owned by the caller (allocated e.g. with torch); the
 *    library never allocates or frees device memory.  Host memory for the
 *    tables is owned by the state and freed by bgtq_destroy.
 *  - "stream" is a cudaStream_t passed as void* (NULL = legacy default
 *    stream).  Calls marked ASYNC only enqueue work on that stream; calls
 *    marked SYNC wait for their own work before returning.
 *  - K and Q arrive after RoPE; the library never applies RoPE.  head_dim
 *    must be 128 (64 RoPE blocks).  Softmax scale is 1/sqrt(head_dim).
 *    Query head h reads KV head h / G, G = n_q_heads / n_kv_heads.
 *  - fp16 tensors are IEEE binary16, row-major, densely packed, 16-byte
 *    aligned.
 *  - A state belongs to the CUDA device that was current at bgtq_create
 *    (its buffers live there).  Every call that launches work or copies
 *    returns BGTQ_ERR_INVALID_ARG, launching nothing, when another device
 *    is current.
 *  - A state is not thread-safe: call it from one host thread at a time.
 *    Its decode calls share the workspace's scratch (rotated queries, split
 *    partials, arrival counters), so two of its calls must not overlap
 *    on the GPU: issue them on one stream, or order the streams.
 *
 * Cache layout inside d_cache (offsets from bgtq_cache_offsets, each
 * 256-byte aligned; L layers, B = max_batch, H = n_kv_heads, T =
 * ceil(capacity / 64) tiles of 64 positions per (layer, sequence, head)):
 *   K tiles    uint8 [L][B][H][T][1024*k_avg_bits]  codes of 64 positions,
 *              laid out for the tensor-core decode (per lane, the nibble
 *              selectors of its mma A-fragments as bit planes; width groups
 *              widest first; see the tile-format definition shipped with
 *              the tests' CPU oracle)
 *   K norms    fp16  [L][B][H][T*64][4]   slot i = norm of group i (width
 *              descending); unused slots 0
 *   V tiles    uint8 [L][B][H][T][1024*v_avg_bits]  same scheme, one group
 *   V norms    fp16  [L][B][H][T*64]
 * Paged cache (page_pool_tiles = P > 0; PagedAttention's block table,
 * cited by the blockgtq pages): the same four arrays with [L][H][P] in place
 * of [L][B][H][T], and the caller's block table (bgtq_set_block_table)
 * mapping tile t of sequence b to a page id, the same for every layer and
 * KV head.  Sequences of a ragged batch then hold only the pages they use.
 * Codebook: the N(0,1) Lloyd-Max levels for 1..4 bits rounded once to
 * binary16; thresholds are the exact midpoints of those levels.
 */
#ifndef BGTQ_H
#define BGTQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum {
  BGTQ_OK = 0,
  BGTQ_ERR_INVALID_ARG = -1,   /* a size, index or config field out of range */
  BGTQ_ERR_NULL = -2,          /* a required pointer is NULL */
  BGTQ_ERR_CUDA = -3,          /* a CUDA runtime call failed (launch or copy) */
  BGTQ_ERR_BUFFER_SIZE = -4,   /* a caller buffer is smaller than required */
  BGTQ_ERR_NOT_READY = -5,     /* no allocation set yet (allocate/set_allocation first) */
  BGTQ_ERR_DEVICE = -6,        /* a kernel raised its error flag (see bgtq_get_device_error) */
  BGTQ_ERR_HOST_ALLOC = -7,    /* host malloc failed */
  BGTQ_ERR_ALIGNMENT = -8      /* a device pointer is not 16-byte aligned */
};

/* Device error flag bits, reported by bgtq_get_device_error. */
enum {
  BGTQ_DEVERR_CAPACITY = 1,    /* encode_append, byte_append: start + count > capacity (rows skipped) */
  BGTQ_DEVERR_SEQ_LEN = 2,     /* decode: a seq_len < 0 or > capacity (sequence skipped, output 0), or a pos_lo /
                                  buf_count out of range (clamped); page operations: a length out of range */
  BGTQ_DEVERR_ARG = 4,         /* encode_append, byte_append: start < 0 or count < 0 or count > n; fork_sequences: a
                                  parent out of range */
  BGTQ_DEVERR_NONFINITE = 8,   /* allocate: a calibration value is Inf or NaN; byte_append: a row's element is
                                  (stored as the largest code, NaN as 0) */
  BGTQ_DEVERR_TIMEOUT = 16,    /* decode: a wait for a tile copy gave up (bounded spin); page operations: a page
                                  copy's wait did, and pages to be written may hold parts of either content */
  BGTQ_DEVERR_PAGE = 32,       /* paged cache: a block-table entry outside [0, page_pool_tiles) (encode and byte_append
                                  skip the tile, decode reads page 0 instead, logit MAE skips the tile); page
                                  operations: a page id in use outside it, or one that is free (compact_pages) */
  BGTQ_DEVERR_POOL = 64        /* fork_sequences, resize_sequences: no free page was left for some row */
};

typedef struct {
  int32_t n_layers;          /* 1..65535 (a call's layers are a launch grid dimension) */
  int32_t n_kv_heads;        /* >= 1 */
  int32_t n_q_heads;         /* multiple of n_kv_heads; G = n_q_heads / n_kv_heads <= 16 */
  int32_t head_dim;          /* must be 128 */
  int32_t max_batch;         /* >= 1 */
  int32_t k_avg_bits;        /* average K bits per dim, 1..4 (record = 16*k bytes) */
  int32_t v_avg_bits;        /* V bits per dim, 1..4 */
  int32_t b_min;             /* smallest K width, 0..4 (0: a block may store nothing) */
  int32_t b_max;             /* largest K width, b_min..4, b_min <= k_avg_bits <= b_max */
  int32_t rope_pairing;      /* 0: block j = dims (j, j+64) (rotate_half); 1: (2j, 2j+1) */
  int32_t max_splits;        /* split-K slots per (layer, seq, KV head); 0 = 256 */
  int32_t page_pool_tiles;   /* 0: contiguous cache; > 0: paged cache with this many
                                64-position pages per (layer, KV head), addressed
                                through bgtq_set_block_table */
  int64_t capacity_tokens;   /* cached tokens per sequence, >= 1 */
  uint64_t seed;             /* seeds the Haar rotations */
} bgtq_config;

typedef struct bgtq_state bgtq_state;

/* Bytes of the two caller-owned device buffers for a config.
 * cache_bytes: the packed K/V cache (layout above).  workspace_bytes: the
 * device tables plus scratch (energy partial sums, rotated queries, split-K
 * partials, error flag).  A config whose cache or workspace would reach
 * 2^56 bytes is rejected with BGTQ_ERR_INVALID_ARG.  SYNC (host only). */
int bgtq_required_bytes(const bgtq_config* cfg, size_t* cache_bytes, size_t* workspace_bytes);

/* Creates a state over caller buffers of at least the required sizes (both
 * 256-byte aligned).  The state keeps the pointers; the buffers must outlive
 * it.  Uploads the Lloyd-Max codebooks and clears the error flag on
 * "stream".  No allocation is set: call bgtq_allocate or
 * bgtq_set_allocation before encoding.  SYNC. */
int bgtq_create(const bgtq_config* cfg, void* d_cache, size_t cache_bytes,
                void* d_workspace, size_t workspace_bytes, void* stream, bgtq_state** out);

/* Frees the host-side state (never the caller's device buffers). NULL is a no-op. */
void bgtq_destroy(bgtq_state* st);

/* Block-GTQ allocation (abstract: per layer and KV head, a label-free energy
 * score for every RoPE block, then integer widths handed out greedily by
 * marginal gain).  Score of block j: s_j = EQ_j * EK_j with
 * EQ_j = sum over rows and the G query heads of the group of ||q_j||^2 and
 * EK_j = sum over rows of ||k_j||^2, accumulated exactly on the GPU (fp16 x
 * 2^24 is an integer; 128-bit sums).  Greedy: every block starts at b_min;
 * each step gives one bit to the block with the largest s_j*(Dist(b_j) -
 * Dist(b_j+1)) below b_max (ties: lowest block), until sum_j b_j =
 * k_avg_bits * 64.  Dist(b) = N(0,1) Lloyd-Max MSE {1, .363380, .117482,
 * .034548, .009497}.  Then builds the per-(layer, KV head) group layout and
 * Haar rotations and uploads them.
 *   d_calib_q  fp16 [n_layers][nq][n_q_heads][128]
 *   d_calib_k  fp16 [n_layers][nk][n_kv_heads][128]
 * nq, nk >= 1.  SYNC (copies the exact sums back, runs the greedy on the host). */
int bgtq_allocate(bgtq_state* st, const void* d_calib_q, int32_t nq,
                  const void* d_calib_k, int32_t nk, void* stream);

/* Sets the widths directly (e.g. uniform TQ-MSE: every block = k_avg_bits)
 * and builds/uploads the tables as bgtq_allocate does.
 *   h_widths int8 [n_layers][n_kv_heads][64], each in [b_min, b_max],
 *            each (layer, head) summing to 64 * k_avg_bits.  SYNC. */
int bgtq_set_allocation(bgtq_state* st, const int8_t* h_widths, void* stream);

/* Copies the current widths out (int8 [n_layers][n_kv_heads][64]). SYNC. */
int bgtq_get_allocation(const bgtq_state* st, int8_t* h_widths);

/* The exact energies of the last bgtq_allocate as 128-bit integers in units
 * of 2^-48, little-endian (lo, hi) uint64 pairs:
 *   h_eq, h_ek  uint64 [n_layers][n_kv_heads][64][2].  SYNC. */
int bgtq_get_energy(const bgtq_state* st, uint64_t* h_eq, uint64_t* h_ek);

/* The Lloyd-Max codebook for bits in 1..4 (TurboQuant's scalar quantiser on
 * N(0,1)) as stored: h_centroids[2^bits] (binary16 values as floats),
 * h_thresholds[2^bits - 1] (their midpoints). */
int bgtq_get_codebook(int32_t bits, float* h_centroids, float* h_thresholds);

/* Group layout of (layer, kv_head): *n_groups, per group its width and size
 * (h_width[4], h_size[4]; unused 0) and h_perm[128] = the original dim at
 * each record position.  SYNC (host tables). */
int bgtq_get_layout(const bgtq_state* st, int32_t layer, int32_t kv_head, int32_t* n_groups,
                    int32_t* h_width, int32_t* h_size, int32_t* h_perm);

/* The fp32 Haar rotation of one group (kind 0 = K, group index 0..n_groups-1)
 * or of V (kind 1, group ignored), row-major d x d, y = R x.  *d receives
 * the size; h_out must hold 128*128 floats.  SYNC (host tables). */
int bgtq_get_rotation(const bgtq_state* st, int32_t layer, int32_t kv_head, int32_t kind,
                      int32_t group, float* h_out, int32_t* d);

/* Byte offsets of the four cache arrays inside d_cache:
 * out[0] K tiles, out[1] K norms, out[2] V tiles, out[3] V norms. */
int bgtq_cache_offsets(const bgtq_state* st, size_t* out);

/* TQ-MSE encode + bit-pack of new rows into the cache.  Source: the
 * Block-GTQ abstract (the allocator's widths feed the TurboQuant-MSE
 * encoder, and the serving path keeps a packed cache) and the blockgtq
 * README's method blurb (integer widths on top of the TQ-MSE encoder) and
 * packed-cache deployment path; TurboQuant (arXiv 2504.19874, cited on the
 * mlsanity index page) for the encoder itself: a random rotation, then the
 * Lloyd-Max scalar quantiser of each rotated coordinate.  For each layer
 * l in [layer, layer + layer_count), sequence b < batch, row r < count[b]:
 * the K and V rows at d_k/d_v[l - layer][b][r][h][:] go to cache position
 * start[b] + r of (l, b, h).  Per K width group g (dims D_g, d = |D_g|):
 * n = ||x[D_g]|| (float64), y = R_g x[D_g] (fp32), u = sqrt(d) y / n,
 * code = #{thresholds <= u}; stored norm = fp16(n).  V: one group of 128.
 *   d_k, d_v   fp16 [layer_count][batch][n][n_kv_heads][128]
 *   d_start    int32 [batch]  first cache position written
 *   d_count    int32 [batch]  rows of this sequence, 0..n
 * Rows with start + r >= capacity are skipped and set BGTQ_DEVERR_CAPACITY.
 * ASYNC. */
int bgtq_encode_append(bgtq_state* st, int32_t layer, int32_t layer_count,
                       const void* d_k, const void* d_v, const int32_t* d_start,
                       const int32_t* d_count, int32_t batch, int32_t n, void* stream);

/* The fused RoPE + encode: bgtq_encode_append with the K rows taken before
 * RoPE (the key projection's output).  Row r of sequence b is turned by
 * RoPE at its cache position p = start[b] + r before it is encoded: block j
 * of the config's rope_pairing (dims (j, j+64) or (2j, 2j+1)) becomes
 * (a cos t - b sin t, a sin t + b cos t) with t = p * rope_base^(-2j/128),
 * the product in fp64 reduced to [-pi, pi], sin and cos in fp32.  The
 * turned values are encoded in fp32 without rounding to fp16.  Groups hold
 * whole RoPE blocks, so a group's norm is that of the row as given, up to
 * the rounding of the turned values.
 * V rows are encoded as in bgtq_encode_append.  rope_base: finite, > 1
 * (BGTQ_ERR_INVALID_ARG otherwise).  Arguments, layouts and device errors
 * otherwise as bgtq_encode_append.  ASYNC. */
int bgtq_encode_append_rope(bgtq_state* st, int32_t layer, int32_t layer_count,
                            const void* d_k, const void* d_v, const int32_t* d_start,
                            const int32_t* d_count, int32_t batch, int32_t n, double rope_base,
                            void* stream);

/* The query in each K width group's rotated basis.  Source: TurboQuant's
 * encoder (arXiv 2504.19874, cited on the mlsanity index page) rotates each
 * group of a key by R_g, and R_g is orthogonal, so q . R_g^T y = (R_g q) . y:
 * the logits of the Block-GTQ abstract's packed-cache serving path can be
 * taken from the codes once q is rotated, one rotation per width group.
 * q~ in record order: per K group g, (1/sqrt(128)) (1/sqrt(d_g)) R_g q[D_g].
 *   d_q     fp16 [layer_count][batch][n_q_heads][128]
 *   d_qrot  fp32 [layer_count][batch][n_q_heads][128]
 * Also writes the tensor-core operand form of q~ into the workspace.  ASYNC. */
int bgtq_rotate_query(bgtq_state* st, int32_t layer, int32_t layer_count, const void* d_q,
                      int32_t batch, float* d_qrot, void* stream);

/* One decode step over the packed cache.  Source: the Block-GTQ abstract's
 * packed-cache serving path (attention at 128K-512K context straight from
 * the packed K3V3 cache) and the blockgtq README's decode benchmark and
 * backend table (a fused decode kernel reading the packed cache); split-K
 * decoding after FlashAttention / FlashAttention-2 (arXiv 2205.14135,
 * 2307.08691, cited on the mlsanity index page).
 * For each layer in [layer, layer + layer_count), sequence
 * b < batch and query head h,
 *   out = sum_t softmax_t(q . k_hat_t / sqrt(128)) v_hat_t over cache
 *   positions t < seq_lens[b],
 * taken in the rotated domain (logits from q~ and the codes; V accumulated
 * in V's rotated basis and rotated back once).  seq_lens[b] = 0 gives 0.
 *   d_q        fp16 [layer_count][batch][n_q_heads][128]
 *   d_seq_lens int32 [batch], 0..capacity
 *   d_out      fp16 [layer_count][batch][n_q_heads][128]
 * Uses the workspace for q~ and split-K partials, so calls on one state
 * must not overlap on the GPU.  ASYNC. */
int bgtq_decode_attn(bgtq_state* st, int32_t layer, int32_t layer_count, const void* d_q,
                     const int32_t* d_seq_lens, int32_t batch, void* d_out, void* stream);

/* One decode step of a layer range as a serving loop runs it: the step's
 * new K/V rows go into the packed cache, then attention reads it (the
 * Block-GTQ abstract's packed-cache serving path; the blockgtq README's
 * decode benchmark, which times decode steps at a given context length).
 * bgtq_encode_append of the step's new
 * rows followed by bgtq_decode_attn, with the same arguments, results and
 * errors as those two calls in that order (seq_lens should count the new
 * rows).  With 1 <= n <= 16 rows per sequence the appends and the query
 * rotation run in one launch (they are independent), so a step takes three
 * launches instead of four.  n = 0 appends nothing (d_k, d_v, d_start and
 * d_count may then be NULL).  ASYNC. */
int bgtq_decode_step(bgtq_state* st, int32_t layer, int32_t layer_count, const void* d_k, const void* d_v,
                     const int32_t* d_start, const int32_t* d_count, int32_t n, const void* d_q,
                     const int32_t* d_seq_lens, int32_t batch, void* d_out, void* stream);

/* Decode with an fp16 buffer: the Block-GTQ README's "withbuffer" setting
 * (AIME commands: a few sink positions and a recent window kept
 * unquantised).  For each layer, sequence b and query head h, attention runs
 * over the packed positions [pos_lo[b], seq_lens[b]) and the sequence's
 * first buf_count[b] buffered rows, with one softmax:
 *   out = sum_t softmax_t(q . k_t / sqrt(128)) v_t
 * over both sets (the packed rows dequantised as for bgtq_decode_attn, the
 * buffered rows as given).  Which positions the buffered rows stand for is
 * the caller's business (typically [0, n_sink) and [len - n_window, len),
 * with pos_lo = n_sink and seq_lens = len - n_window).
 *   d_q, d_out   fp16 [layer_count][batch][n_q_heads][128]
 *   d_seq_lens   int32 [batch]  end of the packed range, 0..capacity
 *   d_pos_lo     int32 [batch]  start of the packed range, 0..seq_lens[b]
 *   d_buf_k/v    fp16 [layer_count][batch][n_buf][n_kv_heads][128]
 *   d_buf_count  int32 [batch]  buffered rows used, 0..n_buf
 *   n_buf        1..1024 (BGTQ_ERR_INVALID_ARG outside)
 * An empty packed range and no buffered row give 0.  Out-of-range
 * lengths set BGTQ_DEVERR_SEQ_LEN and are clamped.  The buffered rows of a
 * (sequence, KV head) are attended by one more CTA of the split pass,
 * beside the packed ones.  Uses the workspace like bgtq_decode_attn.
 * ASYNC. */
int bgtq_decode_attn_buffered(bgtq_state* st, int32_t layer, int32_t layer_count, const void* d_q,
                              const int32_t* d_seq_lens, const int32_t* d_pos_lo, int32_t batch, const void* d_buf_k,
                              const void* d_buf_v, const int32_t* d_buf_count, int32_t n_buf, void* d_out,
                              void* stream);

/* Per-layer logit MAE of the packed keys: the Block-GTQ abstract's logit
 * fidelity diagnostic and the blockgtq README's per-layer kernel MAE
 * (bit allocation section, `--window-M 1024`), comparing Block-GTQ with
 * uniform TQ-MSE at the same average width (two states, one allocated and
 * one with bgtq_set_allocation, holding the same keys).  Only K is
 * involved.  Over a window of m cached positions w0 .. w0+m-1 of sequence
 * seq, with the queries at the same positions, for every causal pair
 * (query i, key j), 0 <= j <= i < m, and each query head h:
 *   d_mae[l][h] = mean |q_{i,h} . k_hat_j - q_{i,h} . k_j| / sqrt(128)
 * where q . k_hat is the logit exactly as the decode computes it from the
 * packed cache and k the exact key.  A layer's MAE is the mean over its
 * heads.
 *   d_q    fp16 [layer_count][m][n_q_heads][128]   queries (post-RoPE)
 *   d_k    fp16 [layer_count][m][n_kv_heads][128]  the exact keys the cache
 *          holds (encoded) at positions w0 .. w0+m-1 of sequence seq
 *   d_mae  double [layer_count][n_q_heads], written by the call
 * 0 <= seq < max_batch, m >= 1, w0 >= 0, w0 + m <= capacity_tokens,
 * else BGTQ_ERR_INVALID_ARG.  The per-head sums use fp64 atomics, so the
 * last bits can vary between runs.  Does not touch the workspace's decode
 * scratch.  ASYNC. */
int bgtq_logit_mae(bgtq_state* st, int32_t layer, int32_t layer_count, int32_t seq, int32_t w0, int32_t m,
                   const void* d_q, const void* d_k, double* d_mae, void* stream);

/* bgtq_encode_append of a step's new rows followed by
 * bgtq_decode_attn_buffered, as one call (the appends and the query rotation
 * share a launch for 1..16 rows per sequence): same arguments, results and
 * errors as those two calls in that order.  In the withbuffer setting the
 * rows appended are typically those leaving the recent fp16 window.  n = 0
 * appends nothing (d_k, d_v, d_start and d_count may then be NULL).  ASYNC. */
int bgtq_decode_step_buffered(bgtq_state* st, int32_t layer, int32_t layer_count, const void* d_k, const void* d_v,
                              const int32_t* d_start, const int32_t* d_count, int32_t n, const void* d_q,
                              const int32_t* d_seq_lens, const int32_t* d_pos_lo, int32_t batch,
                              const void* d_buf_k, const void* d_buf_v, const int32_t* d_buf_count, int32_t n_buf,
                              void* d_out, void* stream);

/* The two stages of bgtq_decode_attn after bgtq_rotate_query, for callers
 * that time or schedule them separately (same arguments and results):
 * bgtq_decode_split runs the split-K pass over the packed cache from the
 * rotated queries d_qrot (fp32 [layer_count][batch][n_q_heads][128], as
 * written by bgtq_rotate_query) into the workspace's partials, and
 * bgtq_decode_combine merges them into d_out.  Both must see the same
 * layer, layer_count, batch, split setting and length values.  The combine
 * reads d_seq_lens as soon as the work queued before it on the stream lets
 * it start, so it must follow its bgtq_decode_split on the stream with no
 * kernel of the caller's in between.  ASYNC. */
int bgtq_decode_split(bgtq_state* st, int32_t layer, int32_t layer_count, const float* d_qrot,
                      const int32_t* d_seq_lens, int32_t batch, void* stream);
int bgtq_decode_combine(bgtq_state* st, int32_t layer, int32_t layer_count, const int32_t* d_seq_lens,
                        int32_t batch, void* d_out, void* stream);

/* No Block-GTQ counterpart on the pages: a library convenience.
 *
 * Same computation, arguments and results as bgtq_decode_attn, for callers
 * that cannot allocate device memory themselves: code that issues work from
 * inside a CUDA stream capture (allocation is not a capturable operation),
 * or a runtime whose device memory is fully reserved up front by its own
 * pool.  This call needs no caller-provided scratch: the rotated queries
 * and split-K partials live in one static device array inside the library
 * of BGTQ_STATIC_SCRATCH_BYTES (16 MiB), which every GPU that loads the
 * library holds until the process exits.  The call allocates nothing.
 *
 * The scratch needed is 64 KiB of arrival counters plus rows * (512 +
 * n_splits * 528 + 8 * 528) bytes, rows = layer_count * max_batch *
 * n_q_heads, plus 6 KiB per (layer, sequence, KV head, block of 8 query
 * heads), with n_splits the most split CTAs a unit can get as for
 * bgtq_decode_attn (see bgtq_set_split_tokens); a call needing more
 * returns BGTQ_ERR_BUFFER_SIZE before launching anything.
 *
 * The first call on a device looks up the array's device address (once per
 * device, with that device current); make that first call before any
 * stream capture.  The address is kept for the life of the process: after
 * cudaDeviceReset (a new primary context) it is stale, so no call may
 * follow a reset of a device the library has used.  Every call on a device
 * shares the one array and reads
 * only what the same call wrote: calls that overlap on the GPU (different
 * streams, or different states at once) race on it.  ASYNC after the first
 * call. */
#define BGTQ_STATIC_SCRATCH_BYTES (16u << 20)
int bgtq_decode_attn_static_scratch(bgtq_state* st, int32_t layer, int32_t layer_count, const void* d_q,
                                    const int32_t* d_seq_lens, int32_t batch, void* d_out, void* stream);

/* Paged cache only (page_pool_tiles > 0): the block table, int32
 * [max_batch][ceil(capacity / 64)] in device memory, caller-owned: entry
 * [b][t] = the page holding positions 64 t .. 64 t + 63 of sequence b, in
 * 0 .. page_pool_tiles - 1.  Entries are read by the kernels when they run
 * (so the caller may fill in new pages between calls, also under graph
 * replay); only the tiles a call reads or writes need valid entries.  Two
 * sequences must not share a page they write.  Until a table is set, calls
 * that touch the cache return BGTQ_ERR_NOT_READY; on a contiguous cache
 * this call returns BGTQ_ERR_INVALID_ARG.  NULL clears the table.  SYNC
 * (host only). */
int bgtq_set_block_table(bgtq_state* st, const int32_t* d_block_table);

/* Split-K width for the decode calls: 0 = automatic (one wave of resident
 * CTAs spread over all (layer, sequence, KV head) units in proportion to
 * their lengths, so that the sequences of a ragged batch finish together;
 * at most twice a unit's even share and max_splits), else a multiple of 64
 * (one tile): a sequence of len positions then gets ceil(len / tokens) <=
 * max_splits split CTAs per unit.  The split counts are computed on the GPU
 * from the lengths.  Results do not depend on the setting beyond
 * floating-point reassociation. */
int bgtq_set_split_tokens(bgtq_state* st, int32_t tokens);

/* Test hook for the bounded waits (no fault is involved): while tile >= 0,
 * the split pass issues no copy for cache tile `tile` of any unit, so the
 * warp that waits for it gives up after about a second of polls, raises
 * BGTQ_DEVERR_TIMEOUT, lets its other copies land and posts empty partials
 * for its CTA; the output then leaves that CTA's positions out.  -1 turns the
 * hook off (the default).  SYNC (host only). */
int bgtq_test_drop_tile_copies(bgtq_state* st, int32_t tile);

/* Selects the decode calls' kernels: fused = 1 asks for the fused launch
 * (query rotation, split-K pass, split merge and inverse V rotation in one
 * kernel of 4- or 8-CTA clusters, whichever holds more CTAs at once), taken
 * where the GPU can co-schedule such a cluster for the config; fused = 0 (the
 * default) runs the query rotation, the split pass and the combine as three
 * launches.  Both compute the same
 * attention up to the order of the split merge.  Other values:
 * BGTQ_ERR_INVALID_ARG.  SYNC (host only). */
int bgtq_set_decode_path(bgtq_state* st, int32_t fused);

/* Which kernels the decode calls of this state launch, and how many CTAs
 * the automatic split plan spreads over a call (*h_ctas: the CTAs the GPU
 * holds at once for that kernel).  *h_fused = 1 when
 * bgtq_decode_attn, bgtq_decode_step and bgtq_decode_attn_static_scratch run
 * as one fused launch per call (query rotation, split-K pass, split merge and
 * inverse V rotation in thread-block clusters of 4 or 8 CTAs; bgtq_decode_step
 * launches the appends before it); 0 when they run the query rotation, the
 * split pass and the combine as three launches (as the buffered and stage
 * calls always do): the fused path was not selected, or this GPU cannot
 * co-schedule its cluster for the config.  Both compute the same attention.
 * SYNC (host only; the first call may query the GPU's occupancy). */
int bgtq_get_decode_path(bgtq_state* st, int32_t* h_fused, int32_t* h_ctas);

/* ---- The 8-bit cache ---------------------------------------------------
 *
 * A cache of 8-bit codes beside the packed one: for layers, heads or models
 * that 1..4 bits do not hold, with the packed cache's 64-position blocks,
 * layouts, paging and call conventions.  No calibration, rotation or
 * allocation comes before it.  A state made by bgtq_byte_create works with
 * bgtq_destroy, bgtq_cache_offsets, bgtq_set_block_table,
 * bgtq_test_drop_tile_copies, bgtq_get_device_error, the page operations and
 * the calls below; the packed cache's other calls answer BGTQ_ERR_NOT_READY or
 * BGTQ_ERR_INVALID_ARG for it, and the bgtq_byte_* calls
 * BGTQ_ERR_INVALID_ARG for a packed state.
 *
 * Arrays (bgtq_cache_offsets: K codes, K scales, V codes, V scales), with
 * slots [L][B][H][T] contiguous or [L][H][P] paged as for the packed cache:
 *   codes   uint8 [slots][64][128]  e4m3 (OCP, no infinities) or int8, row p
 *                                   = position 64 t + p, plain order
 *   scales  fp32 [slots]            a power of two, at least 2^-100
 * The value of a code is code * scale.  One scale for the 64 positions of a
 * (layer, sequence or page, KV head) block, K and V apart.  Device pointers of
 * the bgtq_byte_* calls are 16-byte aligned. */
enum { BGTQ_CODE_E4M3 = 0, BGTQ_CODE_INT = 1 };       /* int: int8, -127 .. 127 */
enum { BGTQ_DTYPE_HALF = 0, BGTQ_DTYPE_BFLOAT = 1 };  /* fp16, bf16 */

typedef struct {
  int32_t n_layers;          /* 1..65535 */
  int32_t n_kv_heads;        /* >= 1 */
  int32_t n_q_heads;         /* multiple of n_kv_heads; G = n_q_heads / n_kv_heads <= 16 */
  int32_t head_dim;          /* must be 128 */
  int32_t max_batch;         /* >= 1 */
  int32_t code;              /* BGTQ_CODE_* */
  int32_t dtype;             /* BGTQ_DTYPE_* of appended rows, queries and outputs */
  int32_t max_q_tokens;      /* most query tokens of a sequence in one call, 1..16 */
  int32_t page_pool_tiles;   /* 0: contiguous; > 0: paged, this many 64-position pages per (layer, KV head) */
  int32_t reserved;          /* 0 */
  int64_t capacity_tokens;   /* cached tokens per sequence, 1..2^30 */
} bgtq_byte_config;

/* Bytes of the two caller-owned device buffers.  A config of 2^31 - 64 or
 * more positions over all layers, heads and sequences (or pages), or of more
 * than 2^24 query rows a sequence (n_q_heads x max_q_tokens), is rejected with
 * BGTQ_ERR_INVALID_ARG.  SYNC (host only). */
int bgtq_byte_required_bytes(const bgtq_byte_config* cfg, size_t* cache_bytes, size_t* workspace_bytes);

/* Creates a state over caller buffers (256-byte aligned, at least the
 * required sizes; they must outlive it).  The cache's contents are left as
 * they are: a zeroed buffer holds zeros.  SYNC. */
int bgtq_byte_create(const bgtq_byte_config* cfg, void* d_cache, size_t cache_bytes, void* d_workspace,
                     size_t workspace_bytes, void* stream, bgtq_state** out);

/* Quantises and stores new rows: for each layer l in [layer, layer +
 * layer_count), sequence b < batch, row r < count[b], the K and V rows go to
 * position start[b] + r.  Per block, K and V apart: a = the largest finite
 * magnitude of the call's rows in it, Qmax = 448 (e4m3) or 127 (int8), e_new
 * = the least integer >= -100 with a <= Qmax 2^e_new.  A call that writes the
 * block's first position starts the block anew: e = e_new, and its other
 * positions keep bytes that mean nothing until they are written.  Otherwise e
 * = max(e_old, e_new), e_old = -100 where the block's scale is no power of two
 * (a buffer never written; a recycled page's scale is one); where e grew, the block's other codes are rescaled
 * (round(code 2^(e_old - e)), ties to even).  New codes are round(x 2^-e),
 * ties to even; the scale is 2^e.  Infinities become the largest code and
 * NaN 0, with BGTQ_DEVERR_NONFINITE.
 *   d_k, d_v   fp16 or bf16 [layer_count][batch][n][n_kv_heads][128]; n = 0
 *              appends nothing (they may then be NULL)
 *   d_start    int32 [batch]
 *   d_count    int32 [batch], 0..n
 * Positions at or past the capacity are skipped and set
 * BGTQ_DEVERR_CAPACITY; start < 0 or count outside 0..n skips the sequence
 * and sets BGTQ_DEVERR_ARG; a page id outside the pool skips the block and
 * sets BGTQ_DEVERR_PAGE.  Two sequences must not write one page.  One launch.
 * ASYNC. */
int bgtq_byte_append(bgtq_state* st, int32_t layer, int32_t layer_count, const void* d_k, const void* d_v,
                     const int32_t* d_start, const int32_t* d_count, int32_t batch, int32_t n, void* stream);

/* How bgtq_byte_decode_attn scores query i of sequence b, at position
 * p = seq_lens[b] - n_q + i, against position t.  In this order:
 *   x = scale q . k_t
 *   x <- softcap tanh(x / softcap)
 *   x <- x - slopes[query head] (p - t)
 * t is visible if t < min(prefix[b], seq_lens[b]), or if
 * max(doc_start[b][i], p - window + 1, 0) <= t <= p.  The prefix is seen by all
 * of the call's queries, before and behind their own position, whatever the
 * window and the document (attention sinks, a prompt attended both ways). */
typedef struct {
  double scale;                /* 0: 1/sqrt(128); else 0 < scale <= 16384 */
  double softcap;              /* 0: none; else 1e-30..1e30 */
  int32_t window;              /* 0: none; else a query sees its own position and the window - 1 before it */
  int32_t reserved;            /* not read */
  const float* d_slopes;       /* fp32 [n_q_heads], finite; NULL: no bias */
  const int32_t* d_prefix;     /* int32 [batch]; NULL: 0 (values clamped to 0..seq_lens) */
  const int32_t* d_doc_start;  /* int32 [batch][n_q]; NULL: 0 */
} bgtq_score;

/* Attention of the last n_q tokens of each sequence (1: a decode step; more:
 * tokens drafted or verified together, causal among themselves) over the
 * 8-bit cache, which holds their own rows too.
 *   d_q, d_out   fp16 or bf16 [layer_count][batch][n_q][n_q_heads][128]
 *   d_seq_lens   int32 [batch], 0..capacity, the new tokens counted
 *   n_q          1..max_q_tokens
 *   score        host memory, read before the call returns; NULL: the defaults
 * Positions that no query of the call sees may hold anything (codes and
 * scales of a buffer never written); the others hold what an append stored,
 * which is never a NaN code.
 * Scores, softmax statistics and sums are fp32 (scale q . k past 2^57, which
 * only bf16 rows reach, may count as less than it is, but past 2^57; a
 * slope past 2^95 counts as 2^95; sums of weighted values overflow where more
 * than 65536 positions share the weight of values near bf16's largest); the
 * softmax weights are rounded to fp16 before they meet the (exact) codes.  A
 * query that sees nothing gives 0; one before position 0 (where n_q >
 * seq_lens[b]) sees the prefix alone.  A length out of range sets
 * BGTQ_DEVERR_SEQ_LEN and counts as 0; a page id outside the pool sets
 * BGTQ_DEVERR_PAGE and page 0 is read.
 * Results do not depend on the batch's other sequences beyond the order of
 * floating-point sums, and are the same each time.  Uses the workspace: two
 * such calls on one state must not overlap on the GPU (captured graphs that
 * hold one included).  Two launches.  ASYNC. */
int bgtq_byte_decode_attn(bgtq_state* st, int32_t layer, int32_t layer_count, const void* d_q,
                          const int32_t* d_seq_lens, int32_t batch, int32_t n_q, const bgtq_score* score, void* d_out,
                          void* stream);

/* ---- Pages of a paged cache, packed or 8-bit ------------------------------
 *
 * A page id names the same 64 positions' slots in every layer and KV head.
 * The caller keeps, in device memory, the block table int32 [batch][ceil(
 * capacity / 64)], the lengths int32 [batch] (row b holds its table's first
 * ceil(lens[b] / 64) entries) and reference counts int32 [page_pool_tiles]:
 * how many rows hold a page, and one more for every other owner (a prompt
 * kept for later requests); 0: free.  Entries behind a row's last page are
 * neither read nor written, but for those that a resize frees.  The calls
 * work on a state of either kind with page_pool_tiles > 0
 * (BGTQ_ERR_INVALID_ARG otherwise), whether or not a block table is set, and
 * for the packed cache before or after an allocation.  They take pages from
 * the lowest free id up, in the order of the rows, so the same inputs give
 * the same tables.  Pointers are 4-byte aligned; outputs lie apart from the
 * inputs and one another, except where "may be" says so
 * (BGTQ_ERR_INVALID_ARG).  1 <= batch <= max_batch.  d_scratch: device memory of
 * bgtq_page_scratch_bytes bytes whose contents are lost; calls that overlap on
 * the GPU need one each (captured graphs included).
 * A length out of 0..capacity sets BGTQ_DEVERR_SEQ_LEN and counts as 0; a page
 * id in use out of 0..page_pool_tiles - 1 sets BGTQ_DEVERR_PAGE. */

/* Bytes of d_scratch (16 a row and 12 a page of the pool).  SYNC (host only). */
int bgtq_page_scratch_bytes(const bgtq_state* st, size_t* bytes);

/* Copies page src[i] to page dst[i], i < n, for every layer and KV head
 * (codes, norms or scales as they are).  A page may be copied to several, but
 * no page may be in d_dst twice, nor in both lists (i = i aside, which does
 * nothing): which bytes it then holds is not defined.  A pair with an id
 * outside the pool is skipped and sets BGTQ_DEVERR_PAGE.  One launch.  ASYNC. */
int bgtq_copy_pages(bgtq_state* st, const int32_t* d_src, const int32_t* d_dst, int32_t n, void* stream);

/* Row b becomes a fork of row parent[b], -1: empty (freed).  Beam search,
 * parallel samples of a prompt, rows leaving.  Whole pages are shared; a page
 * that a row fills partly, which it will write next, ends up with one holder:
 * of the rows that take it over the first keeps it (unless a row or owner
 * besides them holds it too), the others get copies.
 *   d_parent     int32 [batch], -1..batch - 1 (else BGTQ_DEVERR_ARG, taken as -1)
 *   d_table, d_refs, d_lens            before
 *   d_table_out, d_refs_out, d_lens_out  after; refs_out may be refs, lens_out
 *                lens; table_out is another table (copy it back, or point
 *                bgtq_set_block_table to it)
 * Where the pool has no page left for a copy: BGTQ_DEVERR_POOL, the row's entry
 * is -1 and its length that of its whole pages.  Two launches.  ASYNC. */
int bgtq_fork_sequences(bgtq_state* st, const int32_t* d_parent, const int32_t* d_table, const int32_t* d_refs,
                        const int32_t* d_lens, int32_t batch, int32_t* d_table_out, int32_t* d_refs_out,
                        int32_t* d_lens_out, void* d_scratch, void* stream);

/* Takes row b from lens[b] to new_lens[b] positions.  Shorter (drafted tokens
 * rejected; 0: freed): the pages behind its last one are given back, their
 * entries -1.  Longer: it gets pages for all of its positions, and where its
 * last page is filled partly and shared, a copy of it (by the same rule as a
 * fork), so that positions lens[b] .. new_lens[b] - 1 may be written.  Pages
 * given back in the call are handed out in the same call.
 *   d_table, d_refs   before and after
 *   d_lens_out        the lengths granted; may be d_lens or d_new_lens
 * Where the pool runs out: BGTQ_DEVERR_POOL, and lens_out[b] is the length the
 * row got pages for (lens[b] where no page was left to copy its last one to).
 * A new length out of range sets BGTQ_DEVERR_SEQ_LEN and changes nothing for
 * its row.  Two launches.  ASYNC. */
int bgtq_resize_sequences(bgtq_state* st, int32_t* d_table, int32_t* d_refs, const int32_t* d_lens,
                          const int32_t* d_new_lens, int32_t batch, int32_t* d_lens_out, void* d_scratch,
                          void* stream);

/* Moves the live pages (refs > 0) to ids 0 .. n_live - 1: the k-th live page
 * from n_live on goes to the k-th free one below.
 *   d_table_out  the rows' entries renamed; may be d_table
 *   d_refs_out   the counts at the new ids; may be d_refs
 *   d_map        int32 [page_pool_tiles]: each page's new id, -1 for a free one
 *                (for owners besides the table's rows)
 *   d_n_live     int32 [1]
 * An entry that names a free page becomes -1 and sets BGTQ_DEVERR_PAGE.  Two
 * launches.  ASYNC. */
int bgtq_compact_pages(bgtq_state* st, const int32_t* d_table, const int32_t* d_refs, const int32_t* d_lens,
                       int32_t batch, int32_t* d_table_out, int32_t* d_refs_out, int32_t* d_map, int32_t* d_n_live,
                       void* d_scratch, void* stream);

/* ---- Rotary positions over several axes ----------------------------------- */

typedef struct {
  int32_t n_q_heads;         /* >= 0, <= 65536 */
  int32_t n_kv_heads;        /* >= 0, <= 65536; one of both > 0 */
  int32_t head_dim;          /* must be 128 */
  int32_t pairing;           /* as bgtq_config's rope_pairing */
  int32_t dtype;             /* BGTQ_DTYPE_* */
  int32_t n_axes;            /* 1..64 (time, height, width: 3; 1: plain RoPE) */
  uint8_t axis[64];          /* block j turns with axis[j] < n_axes */
  double base;               /* finite, > 1 */
} bgtq_rope_config;

/* Turns query and key rows before they meet a cache: block j of token n by
 * the angle pos[axis[j]][n] base^(-2j/128), (a, b) -> (a cos - b sin, a sin +
 * b cos).  Angles in fp64, sines and products in fp32, one rounding.
 *   cfg            host memory, read before the call returns
 *   d_q, d_q_out   fp16 or bf16, n_q_heads x 128 in a row a token, the tokens
 *                  `stride` elements apart (a multiple of 8, up to 2^30): a
 *                  slice of a projection's output will do
 *   d_k, d_k_out   likewise with n_kv_heads; not read where that is 0
 *   d_pos          int32 [n_axes][tokens], any values
 * An output may be its input (same pointer and stride); else outputs lie apart
 * from the inputs and one another (slices of the same rows do).  Rows are
 * 16-byte aligned, d_pos 4.  0 <= tokens <= 2^30.  Works on the current
 * device, whose memory the pointers must be.  One launch.  ASYNC. */
int bgtq_rope_axes(const bgtq_rope_config* cfg, const void* d_q, int32_t q_stride, const void* d_k, int32_t k_stride,
                   const int32_t* d_pos, int32_t tokens, void* d_q_out, int32_t q_out_stride, void* d_k_out,
                   int32_t k_out_stride, void* stream);

/* Synchronises "stream", reads the device error flag into *h_flags
 * (BGTQ_DEVERR_* bits) and clears it.  SYNC. */
int bgtq_get_device_error(bgtq_state* st, void* stream, int32_t* h_flags);

/* Static description of a status code. */
const char* bgtq_error_string(int32_t status);

#ifdef __cplusplus
}
#endif

#endif /* BGTQ_H */
