/* sv.h -- batch-invariant block verify for greedy speculative decoding (sm_103a).
 *
 * One context holds one sequence of a decoder-only transformer whose weights
 * live in device memory.  Its committed prefix is kept in a paged K/V cache
 * (page size 16, block table, pages from a fixed pool).  Every call runs the
 * same hand-written CUDA kernels on the context's stream:
 *   embed -> per layer [RMSNorm+QKV linear with QK-norm, RoPE and paged K/V
 *   write fused in its epilogue; split-KV paged attention (row r of a call sees
 *   pos+r+1 positions); attention projection + residual; RMSNorm+gate|up
 *   linear with SwiGLU/GeGLU; down projection + residual] -> final RMSNorm +
 *   LM head with per-tile argmax -> argmax/accept/truncate.
 *
 * Verify semantics follow "Phase 23: Speculative Verify Parity" section 2:
 * write the window's K/V into the committed cache in one shot (step 1), give
 * each row its own context length (step 2), compute rows with the same
 * rounding path as single-token decode (step 3), keep the K/V on acceptance
 * (step 4), truncate to the accepted prefix on rejection (step 5).  The
 * acceptance rule is the greedy one of "Shape and cache history in Gemma block
 * verification", section "Mechanism and failure": a draft is kept only while it
 * equals the target's greedy token after the same preceding ids; the
 * correction token is the target's greedy token at the first mismatch.
 *
 * Batch invariance: row r of any call is bit-identical to a single-token
 * decode at the same prefix, and results do not depend on how the cache was
 * built (one-token commits, block commits, one prefill) or on which physical
 * pages hold it.  Logits are returned as fp32 holding bf16 values; argmax ties
 * go to the lowest token id.
 *
 * The pending token: after every commit the library knows the target's
 * greedy token after the committed sequence (sv_prefill's next_token,
 * sv_decode's next_token, sv_verify's correction_token).  A verify window
 * starts with it ("Phase 23" section 2: the window is the known-correct next
 * token plus the drafts), so sv_verify and sv_decode reject any other
 * tokens[0] with SV_E_STATE and change nothing.  Committing tokens the model
 * did not choose (a prompt, forced ids) is sv_prefill's job.  After
 * sv_truncate to a shorter length the pending token is not known, and the
 * next window may start with any id.
 *
 * Conventions for every call:
 *   - Return 0 (SV_OK) or a negative SV_E_* code; sv_last_error() then gives a
 *     message.  On SV_E_INVAL / SV_E_NOMEM / SV_E_STATE the sequence state is
 *     unchanged.
 *     SV_E_CUDA means a CUDA call or a kernel's own bounds/timeout check
 *     failed; the context should then be destroyed.
 *   - Host pointers are read or written before the call returns; device
 *     pointers must stay valid until the work on the context's stream is done.
 *   - Calls on one context must not overlap (one host thread at a time).
 */
#ifndef SV_H
#define SV_H
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SV_OK 0
#define SV_E_INVAL (-1)       /* bad argument or unsupported shape */
#define SV_E_NOMEM (-2)       /* page pool or device memory exhausted */
#define SV_E_CUDA (-3)        /* CUDA error or a kernel reported a failed check */
#define SV_E_STATE (-4)       /* call not valid in the current state (asynchronous work
                                 pending, or tokens[0] not the pending greedy token) */

#define SV_PAGE_SIZE 16       /* positions per KV page */
#define SV_MAX_K 32           /* most rows in one verify step */
#define SV_MAX_PREFILL_ROWS 128 /* most rows in one prefill block (tcgen05 linears) */
#define SV_KV_BF16 0          /* cache formats: bf16 values */
#define SV_KV_E4M3 1          /* e4m3 codes with power-of-two scales */

typedef struct sv_ctx sv_ctx;

/* Model shape and context limits.
 *   hidden % 128 == 0; ffn % 64 == 0; (n_q_heads + 2 n_kv_heads) head_dim % 128
 *   == 0; head_dim in {64, 128, 256}; qk_norm requires head_dim <= 128;
 *   n_q_heads % n_kv_heads == 0 and 16 % (n_q_heads / n_kv_heads) == 0.
 *   act: 0 = SwiGLU silu(gate)*up, 1 = GeGLU with tanh-approximated GELU.
 *   page_size must be 16.  max_k in [1, 32].  max_seq: longest sequence
 *   (committed + window), in [max_k, 1048576]; max_pages: KV pool size in
 *   pages (>= max_seq/16 for one full sequence). */
typedef struct {
  int32_t n_layers, hidden, n_q_heads, n_kv_heads, head_dim, ffn, vocab;
  float rms_eps, rope_theta;
  int32_t qk_norm, act, tie_embeddings;
  int32_t page_size, max_pages, max_k, max_seq;
  /* kv_delayed: when to write a verify window's K/V into the cache.
   *   0 = write-then-truncate: the step writes every window row into the
   *       cache pages and, after acceptance, zeroes the rejected rows.
   *   1 = delayed write-through ("Phase B decision — post-v4", section
   *       "Phase C gating item (new)", candidate C0 "Delayed KV write-through":
   *       verify produces its logits without committing K/V; K/V are committed
   *       once acceptance is decided): the window is written into three
   *       scratch pages per layer (seeded with the committed rows of its pages)
   *       and only the accepted rows are copied into the cache.  Rejected
   *       drafts never reach the cache pages.
   *   Both give bit-identical logits, argmax, acceptance and cache contents;
   *   1 costs 3 more pages per layer and one copy kernel per verify step.
   *   Prefill and decode steps commit every row and take path 0 either way. */
  int32_t kv_delayed;
  /* kv_format: SV_KV_BF16 (0), or SV_KV_E4M3 (1) for a cache in 8 bits with one
   * exponent for each kv head and position (scale_block 1 of the paged caches
   * below): half the cache's bytes and traffic, one kernel more a layer, which
   * rounds the step's rows as it writes them.  Not together with kv_delayed.
   * window, sinks: with window > 0 the row at position t attends only to the
   * positions p > t - window and p < sinks (a model trained so; the cache
   * keeps every position).
   *   Either runs the attention of sv_attend below, with the same batch
   * invariance: a verify row is bit-identical to single-token decode, and
   * results do not depend on how the cache was built.  The context holds that
   * attention's workspace for 128 rows over max_seq, whatever the window (281
   * MB for 32768 positions and 32 query heads of 128). */
  int32_t kv_format, window, sinks;
} sv_config;

/* Device pointers to bf16 weights, row-major, borrowed for the context's
 * lifetime (the caller keeps them allocated and unchanged).  Each must be
 * 16-byte aligned.  Per-layer fields are HOST arrays of n_layers device
 * pointers (read during sv_create only).  sv_create also copies every linear
 * weight (wqkv, wo, w_gate_up, w_down, the LM head) into a tiled layout the
 * context owns and streams from: each 64-column k-block of a 128-row tile one
 * contiguous 16 KB run (the same memory again, 15.1 GB for the 8B shape);
 * SV_NO_TILED=1 streams the borrowed row-major weights instead.
 *   embed, lm_head [vocab, hidden] (lm_head may equal embed); final_norm [hidden]
 *   attn_norm, ffn_norm [hidden]; q_norm, k_norm [head_dim] (ignored if !qk_norm)
 *   wqkv [(n_q_heads + 2 n_kv_heads) head_dim, hidden]: q heads, k heads, v heads
 *   wo [hidden, n_q_heads head_dim]
 *   w_gate_up [2 ffn, hidden]: gate rows then up rows
 *   w_down [hidden, ffn]                                                        */
typedef struct {
  const void *embed, *lm_head, *final_norm;
  const void *const *attn_norm, *const *wqkv, *const *q_norm, *const *k_norm;
  const void *const *wo, *const *ffn_norm, *const *w_gate_up, *const *w_down;
} sv_weights;

/* Create a context on the current CUDA device.  cuda_stream: the caller's
 * stream (cudaStream_t), or NULL for the legacy stream.  A stream of the
 * caller's (not NULL, cudaStreamLegacy or cudaStreamPerThread) is the one
 * every call of the context runs on; it must outlive the context.  For the
 * default streams, which take no stream capture or programmatic dependent
 * launch, the library runs on a stream of its own, ordered after the
 * caller's stream at the start of each call and the caller's stream after
 * the library's work at the end.  Allocates the KV pool, block
 * table, activations, workspaces and the tiled weight copies (all owned by
 * the context); it synchronises the device first, since it reads the
 * weights.
 *
 * Environment switches, read here (results are bit-identical whichever are
 * set, the last one excepted; they change only how the work is launched):
 *   SV_NO_TC=1        steps of 9..32 rows use the mma.sync linear instead of
 *                     the tcgen05 one;
 *   SV_NO_GRAPHS=1    launch every step's kernels directly instead of through
 *                     a CUDA graph per (rows, mode, logits buffer);
 *   SV_NO_PDL=1       no programmatic dependent launch between a step's kernels;
 *   SV_NO_TILED=1     no tiled weight copies: the linears read the borrowed
 *                     row-major weights (less memory, slower streaming);
 *   SV_L2_PREFETCH=n  1: each linear prefetches the next one's first k-blocks
 *                     into L2; 2: only the QKV linear does, for the attention
 *                     projection (off by default: it measured slower);
 *   SV_TEST_WITHHOLD_PARTIAL=c  failure-detection test only: in the first
 *                     linear of every step (steps of at most 8 rows), CTA c
 *                     never hands its split-tile partial to the CTA that
 *                     finishes the tile, whose bounded wait (2 s) then gives
 *                     up: the call returns SV_E_CUDA (status bit 1, timeout)
 *                     and the context must be destroyed.  Results are then
 *                     wrong; never set it otherwise. */
int sv_create(const sv_config* cfg, const sv_weights* w, void* cuda_stream, sv_ctx** out);
void sv_destroy(sv_ctx* ctx);

/* Commit n tokens (host array) at positions len .. len+n-1, processed in the
 * row blocks sv_prefill_blocks gives (whatever max_k is; each block streams
 * every weight once).  last_logits_dev: device fp32 [vocab] for the logits
 * after the last token, or NULL.  next_token: the greedy token after the
 * last one (the new pending token).  Any ids may be committed.  The K/V of
 * every position are bit-identical to those of one-token commits, whatever
 * the block sizes ("Shape and cache history in Gemma block verification",
 * section "Same-prefix controls": one fresh prefill of the committed prefix
 * is one of the three cache histories that must agree).  Synchronous. */
int sv_prefill(sv_ctx* ctx, const int32_t* tokens_host, int n, float* last_logits_dev,
               int32_t* next_token);

/* Commit the pending token and return the greedy next token; logits_dev
 * [vocab] or NULL.  Identical to sv_verify with K = 1 (the single-token
 * decode every verify row must equal: "Phase 23" section 2 step 3), including
 * the SV_E_STATE check of `token`.  Synchronous. */
int sv_decode(sv_ctx* ctx, int32_t token, float* logits_dev, int32_t* next_token);

/* Block verify of K rows (host array) [pending, d_1 .. d_{K-1}] at positions
 * pos .. pos+K-1 (pos = current length): the window's K/V go into the cache
 * in one shot and row r attends to pos+r+1 positions ("Phase 23" section 2
 * steps 1-2).  Row 0 is always committed; drafts are accepted while d_{j+1}
 * equals the argmax of row j (the greedy rule of the Gemma page, section
 * "Mechanism and failure").  On return n_accepted in [0, K-1],
 * correction_token = argmax of row n_accepted (the new pending token), the
 * length is pos + 1 + n_accepted, and the K/V of rejected rows are zeroed
 * ("Phase 23" section 2 steps 4-5).  tokens[0] must be the pending token
 * when one is known (else SV_E_STATE, nothing changed).  logits_dev: device
 * fp32 [K, vocab] or NULL.  Synchronous. */
int sv_verify(sv_ctx* ctx, const int32_t* tokens_host, int K, float* logits_dev,
              int32_t* n_accepted, int32_t* correction_token);

/* Asynchronous verify with device-resident input and output, for callers that
 * keep drafts on the GPU (the same step as sv_verify).  tokens_dev: int32 [K];
 * result_dev: int32 [4] = {n_accepted, correction_token, new_length, status
 * (0 = ok)}; both memory of the context's device (else SV_E_INVAL, nothing
 * queued), 4-byte aligned, read and written by the step's kernels themselves
 * (so they must stay valid until the step is done).  The sequence length and
 * pending token are tracked on the device; pages must already cover every
 * position the call writes (see sv_reserve), otherwise the kernels skip the
 * writes and report a nonzero status.  A step whose tokens[0] is not the pending token commits nothing:
 * its result is {-1, pending, old length, status | 8}, and the next sv_sync
 * returns SV_E_STATE.  Call sv_sync before any synchronous call. */
int sv_verify_async(sv_ctx* ctx, const int32_t* tokens_dev, int K, float* logits_dev,
                    int32_t* result_dev);

/* Make pages cover positions [0, len) (page-table bookkeeping of the paged
 * cache that "Phase 23" section 2 step 1 writes into).  Synchronous. */
int sv_reserve(sv_ctx* ctx, int len);

/* Wait for asynchronous calls, read the device length and pending token back
 * and report any kernel status error (SV_E_CUDA) or a rejected window
 * (SV_E_STATE, see sv_verify_async).  Pages beyond the length are released
 * by the next synchronous call that changes the length. */
int sv_sync(sv_ctx* ctx);

/* Roll the sequence back to new_len <= length: zero the K/V of the removed
 * positions and release their pages ("Phase 23" section 2 step 5: truncate
 * the target cache to the accepted prefix).  A shorter length forgets the
 * pending token.  Synchronous. */
int sv_truncate(sv_ctx* ctx, int new_len);

/* Greedy speculative generation: `draft` proposes, `target` verifies.
 * (Phase 23: Speculative Verify Parity, section 2: drafts are checked by one
 * batched target forward, the longest matching prefix is accepted and the
 * rejected tail rolled back.)  Both contexts hold the same committed tokens
 * (e.g. one prompt prefilled into each) and share the vocabulary; `pending`
 * is the target's greedy token after them (sv_prefill's next_token).  Each
 * round the drafter decodes K-1 tokens after the pending one, the target
 * verifies the K-row block [pending, drafts], and the drafter is rolled back
 * (or advanced) to the target's length.  Rounds run until at least n_new
 * tokens are committed.  The tokens are the target's own greedy continuation,
 * whatever the drafter proposes.
 *   K in [1, target max_k]; K = 1 is plain decoding.  Both contexts need
 *   max_seq >= length + n_new + K.
 *   out_tokens: host int32 [n_new + K - 1]; *n_out (n_new .. n_new + K - 1)
 *   of them are written: every token committed, in order, starting with
 *   `pending`.  *next_pending: the target's greedy token after them.
 *   stats (or NULL): int32 [3] = {verify steps, drafts accepted, drafts
 *   proposed}.
 * Errors: SV_E_INVAL (arguments), SV_E_STATE (lengths differ or asynchronous
 * work pending), or those of the calls it makes (a drafter's error is
 * reported through the target's sv_last_error).  Synchronous. */
int sv_spec_generate(sv_ctx* target, sv_ctx* draft, int32_t pending, int K, int n_new,
                     int32_t* out_tokens, int32_t* n_out, int32_t* next_pending, int32_t* stats);

/* Current committed length (as of the last synchronous call or sv_sync). */
int sv_seq_len(const sv_ctx* ctx);

/* Test read of the paged cache ("Phase 23" section 2 step 1 is what writes
 * it).  Copies the cached K and V of positions [first, first+count) of one
 * layer into two device buffers k_dst_dev, v_dst_dev, each bf16 [count,
 * n_kv_heads, head_dim].  Positions may run to the end of the last page the
 * sequence holds, past its length: every slot there is zero (rejected rows
 * and truncated positions are zeroed), which tests check.  An 8-bit cache is
 * read as the values its codes stand for, and past the length as zeros.
 * Synchronous. */
int sv_kv_read(sv_ctx* ctx, int layer, int first, int count, void* k_dst_dev, void* v_dst_dev);

/* Shuffle the order in which free pages are handed out (seeded).  Results
 * must not depend on it; tests use it to build the same prefix on different
 * physical pages (a cache-history change in the sense of the Gemma page,
 * section "Same-prefix controls"). */
int sv_shuffle_pages(sv_ctx* ctx, uint64_t seed);

/* Test hook for per-layer comparisons.  While hidden_dev is not NULL, every
 * step of at most max_rows rows (1..32) also copies its residual stream into
 * hidden_dev, bf16 [n_layers + 1][rows][hidden]: entry 0 holds the embedded
 * rows, entry l + 1 the output of layer l (the last one is the input of the
 * final RMSNorm).  Such steps run without CUDA graphs or programmatic
 * dependent launch; results are bit-identical either way.  NULL turns it off.
 * The buffer must stay valid while it is set. */
int sv_trace_hidden(sv_ctx* ctx, void* hidden_dev, int max_rows);

/* Number of kernel launches in one step of K rows: with_head = 1 counts a
 * verify step (LM head and acceptance, and for kv_delayed with K > 1 the
 * window copy; an 8-bit cache's write is counted in each layer), 0 a prefill block without the LM head (a block of more than
 * 32 rows is embedded 32 rows a launch).  Steps of more than 8 rows on the
 * tcgen05 form add one row normalisation before each QKV, gate|up and LM
 * head linear. */
int sv_step_kernel_count(const sv_ctx* ctx, int K, int with_head);

/* The row blocks sv_prefill cuts n tokens into, in order, written to
 * sizes[0 .. count-1]; returns count, or SV_E_INVAL if n < 1 or more than
 * max_blocks blocks would be needed (sizes may be NULL to ask for the count
 * only, with max_blocks 0).  The last block holds the 1..SV_MAX_K rows left
 * over; the others hold SV_MAX_K rows, or with use_tc (the tcgen05 linears,
 * the default unless SV_NO_TC=1 was set when the context was created) up to
 * SV_MAX_PREFILL_ROWS rows, always a multiple of SV_MAX_K.  Host only: needs
 * no context and no GPU. */
int sv_prefill_blocks(int n, int use_tc, int32_t* sizes, int max_blocks);

/* Measurement hook for the dominant kernel class.  Launches one linear of the
 * model for K rows, once per layer (distinct weights, so every launch streams
 * from HBM), `reps` times after one untimed pass, chained as inside a step on
 * the context's stream, and timed with CUDA events on that stream.
 *   which: SV_LIN_O, SV_LIN_GATE_UP, SV_LIN_DOWN or SV_LIN_LM_HEAD
 *   avg_us: mean device time per launch
 *   bytes_per_launch (or NULL): algorithmic bytes of one launch = weight bytes
 *     + input rows + output rows (bf16)
 * Overwrites the step's scratch activations; the sequence and its cache are
 * untouched.  Synchronous. */
#define SV_LIN_O 1
#define SV_LIN_GATE_UP 2
#define SV_LIN_DOWN 3
#define SV_LIN_LM_HEAD 4
int sv_time_linear(sv_ctx* ctx, int which, int K, int reps, float* avg_us, double* bytes_per_launch);

/* LM-head step that allocates no device memory.  There is no counterpart to
 * this call on the pages the library follows; it exists for callers that may
 * not call cudaMalloc: code running in a process whose GPU memory is already
 * reserved by another allocator (a serving runtime's pool, or a plugin inside
 * one), and latency-critical code that cannot accept the device-wide
 * synchronisation an allocation may cause.
 *
 * Computes, for M rows x (bf16 [M, hidden], device):
 *   logits = bf16(RMSNorm(x; gain, eps) . W^T)   as fp32 [M, vocab] (device)
 *   argmax[m] = greedy token of row m (largest logit, lowest id on ties)
 * with the same K split and rounding as the context's LM head.  It runs the
 * mma.sync form of the batch-invariant linear for every M; the context runs
 * that form up to 8 rows and the tcgen05 form for 9-32 rows, and the two are
 * bit-identical, so for a model with no layers this call's logits and argmax
 * equal sv_verify's bit for bit at every M.
 *   gain: bf16 [hidden]; W: bf16 [vocab, hidden]; all inputs 16-byte aligned.
 *   argmax_dev: int32 [M] or NULL; status_dev: int32 [1] or NULL, set to 0, or
 *     to the kernels' failure bits (1 timeout).  When the call returns non-zero,
 *     logits_dev, argmax_dev and status_dev are undefined (work already queued
 *     may or may not have written them).
 *   cuda_stream: the stream to run on (NULL = legacy stream).  Asynchronous.
 * Scratch: the split-K partials (one slot per CTA), the argmax partials and
 * the row statistics live in one fixed 8 MiB device array inside the library
 * (held on every GPU that loads it until the process exits).  Shapes whose
 * scratch would not fit return SV_E_NOMEM; the scratch is about
 *   8 * M * ceil(vocab/128) + 4 * G * 128 * (8, 16 or 32 for M <= 8, 16, 32)
 *   bytes, G <= the SM count (one CTA per SM, equal shares of W): with 152
 *   SMs a vocabulary of up to about 2.9 million ids fits at any M.
 * Other limits: 1 <= M <= 32, hidden % 128 == 0 (else SV_E_INVAL).
 * The first call on a device looks up the array's address and sets kernel
 * attributes for that device; make that first call before any stream capture.
 * Every call uses the same array: calls that overlap on the GPU (other
 * streams, other threads) race and must be serialised by the caller. */
int sv_lm_head_noalloc(const void* x_dev, const void* gain_dev, const void* w_dev, int M, int hidden,
                       int vocab, float eps, float* logits_dev, int32_t* argmax_dev,
                       int32_t* status_dev, void* cuda_stream);

/* ---------------------------------------------------------------- paged caches
 * Operators on a paged K/V cache of the caller's, for a batch of sequences:
 * write rows of K and V, fetch them back, and attend to them.  The contexts
 * above run the same kernels on their own pools (sv_config.kv_format, window).
 *
 * A pool holds codes k, v [n_pages, n_kv_heads, 16, head_dim], device memory
 * aligned to 16 bytes.  head_dim is 64, 128 or 256; n_pages * n_kv_heads * 16
 * is below 2^31 - 1.  format:
 *   SV_KV_BF16  the codes are the bf16 values (k_exp, v_exp, scale_block unused);
 *   SV_KV_E4M3  8 bits: e4m3 codes, and for each kv head and block of
 *     scale_block = 1 or 16 positions one e8m0 exponent byte b, the value
 *     2^(b - 127), in k_exp, v_exp [n_pages, n_kv_heads, 16 / scale_block]
 *     (16-byte aligned).  A block whose largest magnitude is a has the smallest
 *     exponent e >= -100 with a <= 448 * 2^e; its values are rounded to the
 *     nearest code, ties to even.  So a value x of a block comes back within
 *     2^-4 |x| (half a step of e4m3's four significant bits) or within
 *     2^-10 * 2^e near zero (e > -100: a > 224 * 2^e, so 2^-17.8 a).  A block with an
 *     infinity or NaN has byte 255 and codes of zero: it reads back as NaN
 *     throughout.  (A value that rounds up to 2^128 comes back as infinity.)
 *   scale_block 1: an append never touches what is stored, so the cache's
 *     bytes do not depend on how the positions were cut into calls.
 *   scale_block 16: one exponent a page.  A write that begins inside a page
 *     keeps the page's exponent or raises it; when it rises the page's
 *     earlier codes are rounded again.  A page whose first position is
 *     written starts anew.
 * The NaN codes 0x7f, 0xff, the exponent bytes 248 to 254, and 0 to 26 beside
 * codes that are not zero, are not written; where a caller's own pool holds them
 * at positions a row sees, that row's result is not defined (NaN or a number),
 * other rows' are not affected.
 * Zeroed exponents and codes are zeros, as written zeros are.
 *
 * The rows of a call: sequence s brings rows row_start[s] .. row_start[s+1] - 1
 * (device int32 [n_seq + 1], not decreasing (sv_attend raises status bit 2 and
 * leaves the outputs undefined where it does); NULL: n_rows / n_seq rows each),
 * which stand at positions first[s], first[s] + 1, ... (device int32 [n_seq],
 * read as within -2^30 .. 2^30).
 * Position p lies in page block_table[s * table_stride + p / 16] at slot p % 16
 * (device int32 [n_seq, table_stride], at most 2^23 positions).  n_rows: rows
 * of the buffers (at most 2^28); those behind the last sequence's are not
 * touched.  max_rows: the most rows of a sequence where the caller knows it
 * (0: n_rows); only speed depends on it.
 * The device arrays are read when the kernels run: a captured graph may be
 * replayed with other lengths, tables and rows.
 *   Rows at negative positions are padding: not written, fetched as zeros,
 * and attending to nothing.  A page that the table does not reach or that is
 * not of the pool is passed over (nothing written, zeros fetched, its
 * positions unseen) and status bit 2 raised.
 *   In one sv_kv_write call no two rows may lie at the same place of the pool,
 * with scale_block 16 no rows of two sequences in the same page (its exponent
 * is one). Pages may be shared between sequences otherwise (a common prefix).
 *
 * Conventions: device pointers of the current device; strides in elements,
 * multiples of 8, between rows whose heads lie side by side (rows of a fused
 * projection will do); row buffers 16-byte aligned.  status_dev: int32 the
 * kernels OR their failure bits into (1 timeout, 2 bad page), or NULL.
 * cuda_stream: the stream to run on (NULL = legacy stream).  Asynchronous, no
 * allocation, no synchronisation: may be captured into a graph (the first
 * sv_attend of a process on a device sets kernel attributes).  Returns SV_OK,
 * SV_E_INVAL (nothing launched), SV_E_NOMEM (workspace too small, nothing
 * launched) or SV_E_CUDA. */
typedef struct {
  int32_t format, n_pages, n_kv_heads, head_dim, scale_block;
  void *k, *v;
  uint8_t *k_exp, *v_exp;
} sv_kv_pool;
typedef struct {
  int32_t n_seq, n_rows, max_rows, table_stride;
  const int32_t *block_table, *first, *row_start;
} sv_row_batch;

/* Put the rows' K and V (bf16 [n_rows, n_kv_heads, head_dim]) into their places. */
int sv_kv_write(const sv_kv_pool* pool, const sv_row_batch* rows, const void* k_dev, int64_t k_stride,
                const void* v_dev, int64_t v_stride, int32_t* status_dev, void* cuda_stream);

/* The reverse: K and V of the rows' positions as bf16. */
int sv_kv_fetch(const sv_kv_pool* pool, const sv_row_batch* rows, void* k_dev, int64_t k_stride, void* v_dev,
                int64_t v_stride, int32_t* status_dev, void* cuda_stream);

/* Attention of the rows over the pool: the row at position t sees positions
 * p <= t, or with window > 0 those with p > t - window or p < sinks, and
 *   out = softmax(scale * q . k) v,  lse = ln(sum exp(scale * q . k)).
 * The rows' own K and V are taken from the pool: write them first.
 *   q, out: bf16 [n_rows, n_q_heads, head_dim], query head h reads kv head
 *   h / (n_q_heads / n_kv_heads) (n_q_heads a multiple of n_kv_heads);
 *   lse_dev: fp32 [n_rows, n_q_heads] or NULL.  A row that sees nothing gives
 *   zeros and -infinity.  What lies in places a row does not see has no effect on it.
 * An infinity among the values of a bf16 cache that a row sees is the row's
 * output in that column; a NaN, or infinities of both signs, make it NaN.
 * Softmax sums and accumulators are fp32.  Over a bf16 cache the sum of up to
 * 256 positions is taken with weights of up to 2^8: values beyond 2^112 may
 * come out as infinities.  Over an 8-bit cache a weight times
 * its value block's scale is rounded to f16 relative to the row's largest such
 * product (2^-11 of itself, at least 2^-25 of the largest).  A row's result depends on its own
 * query, position, window and cache alone, bit for bit: not on the other
 * rows or sequences of the call, nor on the pages that hold the cache.
 * n_seq is at most 1024.
 *   workspace_dev: sv_attend_workspace bytes (256-byte aligned) that the call
 *   may overwrite; calls that may run at the same time (other streams,
 *   captured graphs replayed beside one another), or that two threads issue
 *   on one stream, need one each.  It holds n_q_heads * (4 head_dim + 8) bytes
 *   for every row and every 256 positions that the block table reaches (128 of
 *   the first 1024).  Calls that would need more than 512 MB run in blocks of
 *   rows, one behind the other, and need that much (64 rows are kept together
 *   as far as 4 GB: decode with a table cut for the longest context). */
int sv_attend_workspace(const sv_kv_pool* pool, const sv_row_batch* rows, int n_q_heads, int64_t* bytes);
int sv_attend(const sv_kv_pool* pool, const sv_row_batch* rows, int n_q_heads, const void* q_dev, int64_t q_stride,
              void* out_dev, int64_t out_stride, float* lse_dev, int window, int sinks, float scale,
              void* workspace_dev, int64_t workspace_bytes, int32_t* status_dev, void* cuda_stream);

const char* sv_last_error(const sv_ctx* ctx);

#ifdef __cplusplus
}
#endif
#endif
