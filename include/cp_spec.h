/*
 * cp_spec.h -- C ABI of the GB300 CodePredictor speculative-decoding library.
 *
 * The library runs the inner RVQ loop of a Qwen3-TTS / Qwen3-Omni style
 * CodePredictor: per audio frame, given the talker hidden x and the first
 * code c_0, it emits the residual codes c_1..c_{G-1}, either one decoder pass
 * per code (autoregressive, verify_window = 0) or by speculative rounds
 * ("CodePredictor Speculative Decoding", section "How a round works"):
 *   1. draft: lm_head_{s+1..s+N-1} applied to the current hidden h_s
 *      (section "Why the draft is free"), top-k / temperature sampling;
 *   2. verify: one causal decoder pass over the committed code and the
 *      N-1 drafts against the per-stream KV cache;
 *   3. accept: exact speculative sampling, min(1, p/q), residual
 *      norm(max(0, p - q)) at the first rejection, bonus code when every
 *      draft is accepted ("Speculative Decoding, Beyond Text", section 02);
 *      greedy (temperature 0) is exact argmax equality;
 *   4. reconcile: the KV cache keeps positions 0..s' (s' = last committed
 *      depth); rejected entries stay in memory but are never read (section 07).
 * Two options change only the drafts, so the committed codes keep the
 * autoregressive law: position-aware draft offsets (the draft of lookahead t
 * reads head_{s+t} on h_s + b_t; "RVQ Position Aware Speculative Decoding for
 * On Device TTS", section 2.2) and an adaptive window per stream chosen from
 * its acceptance by offset ("Speculative Decoding, Beyond Text", runtime
 * policies).
 *
 * Sequence layout of one frame: position 0 holds x, position j >= 1 holds
 * the embedding E_{j-1}(c_{j-1}); the decoder output at position j, through
 * the final RMSNorm and head_j, gives the law p_j of c_j ("RVQ Position Aware
 * Speculative Decoding for On Device TTS", Figure 1 and section 2.1).
 *
 * Conventions for every entry point:
 *  - Pointers named d_* are DEVICE pointers, h_* are HOST pointers.  The
 *    caller owns all device memory (weights, workspace, inputs, outputs) and
 *    must keep it alive while work it was passed to is in flight.  The
 *    library never allocates device memory.  A context (cp_spec_ctx) is host
 *    memory owned by the library until cp_spec_destroy.
 *  - Every device pointer must be 16-byte aligned; otherwise the call
 *    returns CP_SPEC_E_INVALID.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *    stream).  Calls enqueue work on it and return without synchronising,
 *    except where stated.  Argument errors are returned synchronously and
 *    enqueue nothing.  Device-side errors (bad code index, a weight tile
 *    copy that did not land in time) are recorded in a device status word and reported by
 *    cp_spec_status_word() or by the next call on the same context.
 *  - Randomness is Philox4x32-10 (Salmon et al., SC'11) with counter
 *    (stream id, frame index, depth, purpose) and key = (seed mod 2^32,
 *    seed >> 32); purpose DRAFT = 0, ACCEPT = 1, TARGET = 2.  u = (word0 >> 8)
 *    * 2^-24.  Results are therefore reproducible bit for bit and
 *    independent of batching or of how streams are split across calls.
 *  - No entry point ever traps, asserts or spins without a bound on the GPU.
 */
#ifndef CP_SPEC_H
#define CP_SPEC_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define CP_SPEC_MAX_LAYERS 64
#define CP_SPEC_MAX_WINDOW 8
#define CP_SPEC_MAX_CODE_GROUPS 64
#define CP_SPEC_MAX_VOCAB 8192
/* Size of the library-owned scratch of cp_spec_decode_frames_static (8 MiB). */
#define CP_SPEC_STATIC_SCRATCH_BYTES (8u << 20)

typedef enum {
  CP_SPEC_OK = 0,
  CP_SPEC_W_AR_FALLBACK = 1,       /* warning: speculation disabled, runs the AR loop */
  CP_SPEC_E_INVALID = -1,          /* bad argument (range, null, alignment)           */
  CP_SPEC_E_UNSUPPORTED = -2,      /* shape outside what the kernels implement        */
  CP_SPEC_E_CUDA = -3,             /* a CUDA runtime call failed                      */
  CP_SPEC_E_WORKSPACE = -4,        /* workspace smaller than cp_spec_workspace_bytes  */
  CP_SPEC_E_DEVICE_TIMEOUT = -5,   /* a bounded device-side wait gave up              */
  CP_SPEC_E_STATE = -6,            /* call out of order (e.g. round before begin)     */
  CP_SPEC_E_DEVICE = -7            /* device-side check failed (e.g. code out of range) */
} cp_spec_status;

/* Decoder shape.  dtype: 0 = float32 weights, 1 = bfloat16 weights.
 * Norm gains are always float32.  Requirements: hidden % 8 == 0,
 * ffn % 8 == 0, n_q_heads * head_dim % 8 == 0, head_dim even and <= 256,
 * n_q_heads % n_kv_heads == 0, 1 <= n_layers <= 64,
 * 2 <= num_code_groups <= 64, 2 <= vocab <= 8192. */
typedef struct {
  int32_t hidden, n_layers, n_q_heads, n_kv_heads, head_dim, ffn, vocab, num_code_groups;
  int32_t dtype;
  float rope_theta; /* rotary base, rotate-half pairing (i, i + head_dim/2) */
  float rms_eps;    /* RMSNorm epsilon                                       */
} cp_spec_model;

/* Device pointers to the weights (borrowed, read-only, row-major).
 * embed:   [G-1][V][H]   table j (0-based) embeds c_j as the input of position j+1.
 * lm_head: [G-1][V][H]   index j-1 is head_j (scores c_j).
 * Per layer l: wq [nq*d][H], wk [nkv*d][H], wv [nkv*d][H], wo [H][nq*d],
 * w_gate [F][H], w_up [F][H], w_down [H][F]; attn_norm, ffn_norm [H] fp32.
 * final_norm [H] fp32.  The blocks are pre-norm: h += Wo attn(RMSNorm(h));
 * h += Wdown (silu(Wgate b) * Wup b) with b = RMSNorm(h).
 * draft_offset: [K][H] fp32 position-aware draft offsets b_1..b_K, K =
 * config.draft_offsets (NULL when K = 0).  The draft of lookahead t reads
 * head_{s+t} on h_s + b_t for t <= K, and h_s alone beyond K, where h_s is
 * the final-normed hidden the target head_s reads; the target heads never see
 * an offset, so the committed codes keep the autoregressive law ("RVQ
 * Position Aware Speculative Decoding for On Device TTS", section 2.2 and
 * Figure 3).  The library reads b once, in cp_spec_init (and in every
 * cp_spec_decode_frames_static call), and keeps the products head_j . b_t
 * in the workspace: later changes to the values behind the pointer are not
 * seen by an existing context. */
typedef struct {
  const void* embed;
  const void* lm_head;
  const float* final_norm;
  const float* attn_norm[CP_SPEC_MAX_LAYERS];
  const void* wq[CP_SPEC_MAX_LAYERS];
  const void* wk[CP_SPEC_MAX_LAYERS];
  const void* wv[CP_SPEC_MAX_LAYERS];
  const void* wo[CP_SPEC_MAX_LAYERS];
  const float* ffn_norm[CP_SPEC_MAX_LAYERS];
  const void* w_gate[CP_SPEC_MAX_LAYERS];
  const void* w_up[CP_SPEC_MAX_LAYERS];
  const void* w_down[CP_SPEC_MAX_LAYERS];
  const float* draft_offset;
} cp_spec_weights;

/* verify_window: 0 = autoregressive loop; 2..8 = one committed depth plus
 * N-1 drafted depths ("CodePredictor Speculative Decoding", "Options": 1 is
 * rejected because it leaves no draft slot).  top_k: 1..vocab, the default
 * for every stream and the maximum any stream may use.  temperature: 0 =
 * greedy, else in [1e-3, 100].  max_streams: streams the workspace is sized
 * for (>= 1).  draft_offsets: K, the number of position-aware draft offset
 * vectors in weights.draft_offset, 0..7 (0 = the heads are reused without
 * offsets); offsets beyond verify_window - 1 are never read.
 * adapt_accept_pct, adapt_min_reached: the adaptive window ("Speculative
 * Decoding, Beyond Text", runtime policies).  0 = off: every round drafts
 * min(verify_window - 1, codes left).  With pct in 1..100, each stream picks
 * the window of its next frame from its acceptance by offset earlier in the
 * same cp_spec_decode_frames call: offsets t = 1, 2, ... are kept while each
 * has fewer than adapt_min_reached (>= 1) drafts reached by the left-to-right
 * test, or accepted at least pct percent of them (100 * accepted >= pct *
 * reached); the window is 1 + the kept leading offsets.  Window 1 runs the
 * frame without drafts, one row per pass.  The choice depends only on
 * earlier frames, so the committed codes keep the autoregressive law.  Each
 * call (and each cp_spec_begin_frame) starts with no history, i.e. with the
 * full window. */
typedef struct {
  int32_t verify_window;
  int32_t top_k;
  float temperature;
  uint64_t seed;
  int32_t max_streams;
  int32_t draft_offsets;
  int32_t adapt_accept_pct;
  int32_t adapt_min_reached;
} cp_spec_config;

/* Counters accumulated since init (or the last cp_spec_reset_stats).
 * committed = codes c_1..c_{G-1} emitted; passes = decoder passes (frame
 * prefills + rounds, or AR steps); accepted/drafted_by_offset[t] = drafts at
 * offset t (1..8) accepted / reached by the left-to-right test (every draft
 * up to and including the first rejection; "report acceptance by offset",
 * "Speculative Decoding, Beyond Text", section 06).  weight_bytes and
 * kv_bytes count the algorithmic HBM bytes of all decoder passes (every
 * layer matrix once per pass, each distinct lm_head applied in the pass
 * once, the KV positions each pass reads). */
typedef struct {
  int64_t frames, passes, rounds, committed, bonus, rejections;
  int64_t drafted_by_offset[9];
  int64_t accepted_by_offset[9];
  int64_t weight_bytes, kv_bytes, heads_applied;
  /* Pass kernels executed on the device (5 per layer, 6 with a 4-bit KV cache,
   * + lm_heads, top-k and accept, per pass; counted by the accept kernel). */
  int64_t kernel_launches;
  int64_t reserved[7];
} cp_spec_stats;

typedef struct cp_spec_ctx cp_spec_ctx;

/* Bytes of device workspace cp_spec_init needs for this model/config
 * (KV cache, activations, logits, sampling lists, per-stream state).
 * Returns 0 if the arguments are invalid. */
size_t cp_spec_workspace_bytes(const cp_spec_model* model, const cp_spec_config* config);

/* Validate, carve the caller's workspace (d_workspace, >= the size above),
 * initialise device state on the current device (synchronously) and return a
 * context in *out.  Returns CP_SPEC_W_AR_FALLBACK (and a usable context in AR
 * mode) when verify_window >= 2 but num_code_groups < 3, i.e. there is no
 * draft slot after the first code ("CodePredictor Speculative Decoding",
 * "Limitations": automatic fallback).  vocab above CP_SPEC_MAX_VOCAB returns
 * CP_SPEC_E_UNSUPPORTED: there is no second backend and no CPU fallback. */
cp_spec_status cp_spec_init(const cp_spec_model* model, const cp_spec_weights* weights,
                            const cp_spec_config* config, void* d_workspace, size_t workspace_bytes,
                            cp_spec_ctx** out);

/* Sparse draft tree ("RVQ Position Aware Speculative Decoding for On Device
 * TTS", section 2.2 "tree attention / sparse tree attention", Figure 2).
 * HOST arrays of n entries (1 <= n <= 62), nodes listed parents first:
 * parent[i] is -1 for a child of the committed code, else an earlier node;
 * rank[i] is the rank of the node's token among the draft logits of its
 * depth (value descending, index ascending; 0 = the largest), below
 * min(top_k rounded up to a multiple of 4, vocab).  Siblings come in
 * ascending rank without repeats; depth at most CP_SPEC_MAX_WINDOW - 1.
 * The arrays are read during the call only. */
typedef struct {
  int32_t n;
  const int32_t* parent;
  const int32_t* rank;
} cp_spec_tree;

/* Workspace bytes of a tree context (0 if the arguments are invalid). */
size_t cp_spec_workspace_bytes_tree(const cp_spec_model* model, const cp_spec_config* config,
                                    const cp_spec_tree* tree);

/* cp_spec_init for tree rounds instead of chain rounds: every round drafts
 * the tree's nodes (node i carries the rank[i]-th draft logit of head_{s+d}
 * on h_s, d its depth; nodes deeper than the codes left are dropped),
 * verifies the committed code and every node short of the frame end in one
 * pass (each node attends to the prefix and to its own ancestors), and walks
 * the tree from the committed code: the children of a node are tested in
 * rank order as point-mass drafts against the node's target law (accept
 * child c iff u < p'(c), p' the remaining mass renormalised; Philox purpose
 * 4 + the child's index among those tested), and one code is drawn from what
 * remains when none is accepted (purpose TARGET).  Every committed code keeps
 * the autoregressive law; under temperature 0 the codes equal greedy
 * autoregressive decoding.  config->verify_window, adapt_accept_pct and
 * adapt_min_reached are ignored (the tree fixes the drafts); draft_offsets
 * applies to depths 1..K.  The accepted path's K/V rows are copied from the
 * nodes' slots to their positions: the one place a round moves cache data.
 * Decode with cp_spec_decode_frames / cp_spec_begin_frame + cp_spec_round as
 * for chain contexts.  Errors as cp_spec_init, plus CP_SPEC_E_INVALID for a
 * malformed tree or fewer than 3 code groups. */
cp_spec_status cp_spec_init_tree(const cp_spec_model* model, const cp_spec_weights* weights,
                                 const cp_spec_config* config, const cp_spec_tree* tree, void* d_workspace,
                                 size_t workspace_bytes, cp_spec_ctx** out);

/* Contexts over 4-bit weights.  The matrices (wq, wk, wv, wo, w_gate, w_up,
 * w_down, lm_head) are given packed by cp_spec_w4_pack, each with groups of
 * `group` along its rows; lm_head as one matrix [(G-1) * V][H].  embed stays in
 * the model's dtype, the norms and draft offsets in float32.  Everything else
 * is as for cp_spec_init (tree NULL) or cp_spec_init_tree: decoding, rounds,
 * sampling, offsets, the adaptive window, counters (weight_bytes counts packed
 * bytes).  The committed law is that of the decoder with the values that the
 * packed weights stand for, computed in float32 (inputs count with 22 bits).
 * kv_bits 32 keeps the float32 KV cache; 4 holds each stream's frame in a
 * 4-bit cache (cp_spec_kv4_append, cp_spec_kv4_attention: one page per stream
 * and layer) of 0.14 of its bytes, at the price of the keys' and values' own
 * rounding; greedy codes of different windows may then differ where a value
 * lies as close to a rounding border as float32 sums differ.  Made for few
 * rows per pass: every block of 8 rows reads the weights again, so packed and
 * bfloat16 weights are about even at 8 streams and bfloat16 ones 3 to 4.5 times
 * faster at 64.  The 4-bit cache saves memory, not time (N = 4, one stream: 186
 * against 159 us per pass).
 * Limits beside cp_spec_init's: head_dim a multiple of 32, vocab of 16; kv_bits
 * 4 needs head_dim 64, 128 or 256 and chain rounds. */
typedef struct {
  int32_t group;   /* 32, 64 or 128 */
  int32_t kv_bits; /* 32 or 4 */
} cp_spec_quant;

/* Workspace bytes of such a context (0 if the arguments are invalid). */
size_t cp_spec_workspace_bytes_w4(const cp_spec_model* model, const cp_spec_config* config, const cp_spec_tree* tree,
                                  const cp_spec_quant* quant);
cp_spec_status cp_spec_init_w4(const cp_spec_model* model, const cp_spec_weights* weights, const cp_spec_config* config,
                               const cp_spec_tree* tree, const cp_spec_quant* quant, void* d_workspace, size_t workspace_bytes,
                               cp_spec_ctx** out);

/* Per-stream sampling overrides, HOST arrays of n entries (n <= max_streams):
 * top_k in 1..config.top_k, temperature 0 (greedy) or in [1e-3, 100].
 * Synchronous (small host-to-device copy). */
cp_spec_status cp_spec_set_stream_sampling(cp_spec_ctx* ctx, int32_t n, const int32_t* h_top_k,
                                           const float* h_temperature);

/* Decode n_frames frames for streams 0..n_streams-1 (n_streams <= max_streams).
 * d_x: [n_frames][n_streams][H] float32 talker hiddens; d_c0: [n_frames][n_streams]
 * int32 first codes; d_codes (out): [n_frames][n_streams][G] int32, with
 * d_codes[f][b][0] = c_0.  Frame f uses Philox frame index first_frame + f.
 * One launch of the context's call graph on `stream` (a setup kernel, then
 * a device-controlled loop of decoder passes, 5 L + 3 kernels each (6 L + 3
 * with a 4-bit KV cache), until
 * every stream has finished its frames; the graph is built and instantiated
 * on the first call, in host memory); streams advance through their frames
 * independently.  Asynchronous. */
cp_spec_status cp_spec_decode_frames(cp_spec_ctx* ctx, int32_t n_streams, int32_t n_frames,
                                     int32_t first_frame, const float* d_x, const int32_t* d_c0,
                                     int32_t* d_codes, void* stream);

/* Step-wise API.  cp_spec_begin_frame stages one frame for every stream
 * (d_x [n_streams][H], d_c0 [n_streams], both read by later rounds and kept
 * alive by the caller until the frame completes).  Each cp_spec_round runs
 * one decoder pass for every unfinished stream: the first is the frame
 * prefill (rows x, E_0(c_0); commits c_1), later ones are speculative
 * rounds (or AR steps).  d_codes [n_streams][G] receives codes as they are
 * committed; d_committed [n_streams] (optional) receives s+1, the number of
 * codes of the frame known so far (G when the frame is complete).
 * Asynchronous. */
cp_spec_status cp_spec_begin_frame(cp_spec_ctx* ctx, int32_t n_streams, const float* d_x,
                                   const int32_t* d_c0, int32_t frame_idx, void* stream);
cp_spec_status cp_spec_round(cp_spec_ctx* ctx, int32_t* d_codes, int32_t* d_committed, void* stream);

/* Teacher-forced logits, for checking the decoder numerics: rows x,
 * E_0(c_0), ..., E_{P-2}(c_{P-2}) at positions 0..P-1 (2 <= P <= G) for each
 * stream, run through the same verify-pass kernels in chunks of at most
 * max(verify_window, 2) rows.  d_codes [n_streams][P-1]; d_logits (out)
 * [n_streams][P-1][V] = head_j at position j; d_draft_logits (optional, out,
 * speculative configs only) [n_streams][P-1][N-1][V] = head_{j+t} at
 * position j (zero where j+t > G-1).  Asynchronous. */
cp_spec_status cp_spec_teacher_logits(cp_spec_ctx* ctx, int32_t n_streams, int32_t P, const float* d_x,
                                      const int32_t* d_codes, float* d_logits, float* d_draft_logits,
                                      void* stream);

/* Acceptance kernels alone (no model): R independent rounds of N-1 drafts
 * verified against N target rows (2 <= N <= 8, 2 <= V <= 8192).
 * mode 0: d_target [R][N][V] and d_draft [R][N-1][V] are float32 logits,
 *         processed with top_k / temperature as in the full path;
 * mode 1: they are already-processed float32 probabilities (each row's
 *         non-zero entries are its support; top_k/temperature ignored,
 *         temperature 0 not allowed).
 * Draft t (1..N-1) is drawn from draft row t-1 with Philox (r, 0, t, DRAFT),
 * accepted with (r, 0, t, ACCEPT); residual / bonus draws use (r, 0, t,
 * TARGET).  Outputs: d_tokens [R][N] committed codes, -1 padded;
 * d_n_accepted [R]; d_drafts [R][N-1] (optional).  Asynchronous; needs no
 * context and no workspace. */
cp_spec_status cp_spec_accept_batch(int32_t R, int32_t N, int32_t V, int32_t top_k, float temperature,
                                    uint64_t seed, int32_t mode, const float* d_target,
                                    const float* d_draft, int32_t* d_tokens, int32_t* d_n_accepted,
                                    int32_t* d_drafts, void* stream);

/* ------------------------------------------------------ 4-bit operators
 * Products with 4-bit weights, a KV cache held in 4 bits, and attention over
 * it: the decoder's own operators for models whose weights and caches should
 * take a quarter of the memory.  Context-free like cp_spec_accept_batch:
 * nothing kept between calls, asynchronous, safe to capture into a
 * graph and to call from several threads and streams at once.  They run on the
 * current device, which must be the pointers' and the stream's.
 *
 * The format.  A value is s * c, with c one of the sixteen E2M1 numbers +-0,
 * 0.5, 1, 1.5, 2, 3, 4, 6 and s the bfloat16 scale of a group of consecutive
 * elements: s = bf16(max |x| * r), r the float32 number nearest to 1/6, c the
 * E2M1 number nearest to x / s, ties to the even code, saturating at 6.  A
 * group that holds an infinity or a NaN reads back as NaN; one whose scale
 * rounds to zero reads back as zeros.
 * Any finite x is held like that; the product and the attention are made for
 * weights, keys and values of at most 2^100 in magnitude (beyond, a group's sum
 * may overflow where the result would not, and small weights of a softmax drop out).
 *
 * Element types (dtype, out_dtype): 0 float32, 1 bfloat16, 2 float16.  Row
 * strides count elements; a row itself is dense. */
#define CP_SPEC_MAX_W4_K 32768
#define CP_SPEC_MAX_KV4_ROWS 64

/* Bytes of a packed matrix [n][k] (rows padded to 16, columns to 128 by
 * zeros), 0 if the arguments are invalid.  n >= 1, 1 <= k <= CP_SPEC_MAX_W4_K,
 * group 32, 64 or 128. */
size_t cp_spec_w4_bytes(int32_t n, int32_t k, int32_t group);

/* Quantises d_w [n][k] (row stride w_stride >= k) into d_packed
 * (cp_spec_w4_bytes, 16-byte aligned), in groups along k.  Once per matrix;
 * the layout is the library's own. */
cp_spec_status cp_spec_w4_pack(int32_t n, int32_t k, int32_t group, int32_t dtype, const void* d_w, int64_t w_stride,
                               void* d_packed, void* stream);

/* The values a packed matrix stands for, rounded once to dtype: d_w (out) [n][k]. */
cp_spec_status cp_spec_w4_unpack(int32_t n, int32_t k, int32_t group, int32_t dtype, const void* d_packed, void* d_w,
                                 void* stream);

/* y[r][i] = sum_j x[r][j] w[i][j] for `rows` rows (0 .. 65535) of x: the
 * product of a decoder pass, made for the few rows of a verify window or a
 * batch of streams (up to 32 rows, 16 of float32, share one read of w).
 * d_x [rows][k] of dtype with row stride x_stride >= k, d_y (out) [rows][n] of
 * out_dtype (dtype, or 0) with row stride y_stride >= n; nothing between the
 * rows of d_y is written.  Sums in float32; float32 inputs count with 22 bits,
 * the 16-bit types exactly, neither finer than 2^-39 of the largest of the 128
 * neighbours (columns 128 j ..) that an input has.
 * The order of the sums depends on the shape only: a row's result does not
 * depend on the values of the rows beside it. */
cp_spec_status cp_spec_w4_gemv(int32_t rows, int32_t n, int32_t k, int32_t group, int32_t dtype, int32_t out_dtype,
                               const void* d_x, int64_t x_stride, const void* d_packed, void* d_y, int64_t y_stride,
                               void* stream);

/* A KV cache in 4 bits: n_pages pages of page_size token slots (a multiple of
 * 16) for n_kv_heads heads of head_dim channels (64, 128 or 256), one scale
 * per 32 channels of a token and head, keys and values together.  The caller
 * owns the memory (cp_spec_kv4_bytes, 16-byte aligned) and need not clear it.
 *
 * d_pages [n_seqs][max_pages] int32 maps page j of sequence b to a page of the
 * cache; NULL: sequence b owns pages b * max_pages .. (needs n_seqs *
 * max_pages <= n_pages).  max_pages * page_size < 2^31.  An entry outside
 * [0, n_pages) is never followed: its positions are not written, read back as
 * zeros, and are left out of the attention.  So are positions past max_pages *
 * page_size. */
typedef struct {
  int32_t n_pages, page_size, n_kv_heads, head_dim;
} cp_spec_kv4;

/* Bytes of the cache, 0 if the shape is invalid or the cache would pass 2^48 bytes. */
size_t cp_spec_kv4_bytes(const cp_spec_kv4* shape);

/* Quantises rows of keys and values as they are written: row i of sequence b
 * goes to position d_pos[b] + i, for i < d_rows[b] (clamped to 0 .. rows; NULL:
 * rows).  d_k, d_v [n_seqs * rows][n_kv_heads][head_dim] with row strides
 * k_stride, v_stride >= n_kv_heads * head_dim (slices of a fused projection
 * work).  Other slots keep their values.  Two rows written to one slot by
 * calls or sequences that overlap in time leave it undefined; neighbouring
 * slots may be written at the same time. */
cp_spec_status cp_spec_kv4_append(const cp_spec_kv4* shape, void* d_cache, const int32_t* d_pages, int32_t max_pages,
                                  int32_t n_seqs, int32_t rows, const int32_t* d_pos, const int32_t* d_rows, int32_t dtype,
                                  const void* d_k, int64_t k_stride, const void* d_v, int64_t v_stride, void* stream);

/* The values the cache holds for positions 0 .. length - 1 of each sequence,
 * rounded once to dtype: d_k, d_v (out) [n_seqs][length][n_kv_heads][head_dim].
 * Positions at or past d_len[b] (NULL: length) read as zeros. */
cp_spec_status cp_spec_kv4_read(const cp_spec_kv4* shape, const void* d_cache, const int32_t* d_pages, int32_t max_pages,
                                int32_t n_seqs, int32_t length, const int32_t* d_len, int32_t dtype, void* d_k, void* d_v,
                                void* stream);

/* Attention of a window of rows over the held cache.  Sequence b has
 * d_kv_len[b] positions (clamped to 0 .. max_pages * page_size), the last
 * d_rows[b] of them (clamped to 0 .. rows; NULL: rows; rows <=
 * CP_SPEC_MAX_KV4_ROWS) the window's own, already appended.  With base =
 * d_kv_len[b] - d_rows[b], row i sees every position below base, and of the
 * window the positions base .. base + i (d_mask NULL: causal) or base + j for
 * every bit j of d_mask[b][i] (uint64; the nodes of a sparse tree set their
 * ancestors' bits and their own).  Negative positions do not exist (base may
 * be negative).
 *   o = softmax(scale * q k^T) v,  scale finite,
 * d_q, d_o (out) [n_seqs * rows][n_q_heads][head_dim] of dtype with row strides
 * q_stride, o_stride >= n_q_heads * head_dim; query head e reads KV head
 * e / (n_q_heads / n_kv_heads).  d_lse (optional, out) [n_seqs][rows][n_q_heads]
 * float32: the log of the sum of the exponentials.  A row that sees nothing
 * gives zeros and -infinity; a position that a row does not see cannot reach it,
 * whatever is stored there, not by a bit.  Rows at or past d_rows[b] are left as
 * they were.  Scores and sums are float32 (float32 queries count with 22 bits); a
 * weight times a value's scale counts with 11 bits (bfloat16) or 22 (float16,
 * float32), and with a weight of 1 standing for the row's largest never finer
 * than 2^-31 of the largest value scale that the row sees in any channel of the
 * head (of 2^-80 where all are smaller): channels or positions far smaller than
 * that lose bits.
 * Results do not depend on timing or on the other sequences' contents, but
 * max_pages and the numbers of sequences, heads and rows choose how a long
 * sequence is split, which moves them within rounding.
 * d_work: cp_spec_kv4_attention_bytes of scratch (NULL where that is 0), used
 * during the call's work only; calls that overlap in time need their own. */
cp_spec_status cp_spec_kv4_attention(const cp_spec_kv4* shape, const void* d_cache, const int32_t* d_pages, int32_t max_pages,
                                     int32_t n_seqs, int32_t rows, int32_t n_q_heads, const int32_t* d_kv_len,
                                     const int32_t* d_rows, const uint64_t* d_mask, float scale, int32_t dtype,
                                     const void* d_q, int64_t q_stride, void* d_o, int64_t o_stride, float* d_lse,
                                     void* d_work, size_t work_bytes, void* stream);

/* Workspace of that call on the current device: 0 unless sequences are split
 * (few sequences and heads, long tables); also 0 if the arguments are invalid. */
size_t cp_spec_kv4_attention_bytes(const cp_spec_kv4* shape, int32_t max_pages, int32_t n_seqs, int32_t rows,
                                   int32_t n_q_heads, int32_t dtype);

/* --------------------------------------------- 16-bit paged KV cache
 * The operators of an outer model's step over a cache in its own 16-bit type:
 * page tables and slot maps made on the device from request lengths, rotary
 * embedding over several position axes (alone, or as rows are written into the
 * cache), and attention over the cache for prompts, single tokens, verify
 * windows and draft trees, with an optional sliding window whose first tokens
 * stay visible.  Context-free like the 4-bit operators and under the same rules:
 * nothing kept between calls, asynchronous, safe to capture and to call from
 * several threads and streams, on the current device.
 *
 * Rows are packed: the rows of all sequences one after the other, sequence b
 * those from d_row_start[b] to d_row_start[b + 1] - 1.  n_rows is the room of the
 * call; rows behind the last sequence are padding and are left as they were. */
#define CP_SPEC_MAX_PLAN_SEQS 4096
#define CP_SPEC_MAX_TREE_ROWS 64
#define CP_SPEC_MAX_KV16_ROWS (1 << 24)

/* One step of a pool of pages.  The pool has n_pages pages of page_size slots (a
 * multiple of 16), used by any cache of that shape.  Its state, all device memory
 * of the caller's and changed in place: d_free [n_pages] with d_n_free [1], a stack
 * of the free pages (the top is entry n_free - 1); d_pages [n_seqs][max_pages], the
 * page tables; d_held [n_seqs], the pages that each sequence holds.
 *
 * Sequence b keeps its first d_len[b] tokens and adds d_new[b] rows (NULL: none;
 * negative numbers count as 0), so it needs ceil((len + new) / page_size) pages.
 * First all pages past the need go back to the stack and their table entries
 * become -1; then lacking pages are taken, sequence by sequence, from its top.
 * (What is given back goes last sequence and last page first: giving back what the
 * call before took restores the stack.)  A draft that is rejected, or a request
 * that ends, gives its pages back by a smaller length.
 *
 * d_refused[b] (optional): 0, or why the sequence gets no rows: 1 too few free
 * pages (the lacks of all sequences up to b exceed them; a sequence that lacks
 * none is served), 2 more pages than max_pages, 3 the new rows of all sequences
 * up to b exceed n_rows.  A refused sequence takes no pages (with 2 it gives none
 * back either) and keeps min(d_len[b], what its pages hold) tokens.
 *
 * Out: d_kv_len [n_seqs] tokens with the new rows, d_row_start [n_seqs + 1], and
 * for each of the n_rows rows d_pos, its position, and d_slot, its slot in the
 * cache (page * page_size + offset): what cp_spec_kv16_append and
 * cp_spec_kv16_attention take (the tables serve the 4-bit cache too).  Padding has
 * position 0 and slot -1; a row whose table entry is no page has slot -1.
 * n_rows may be 0 (d_pos, d_slot NULL).  Whole numbers throughout: results do not
 * depend on timing.  n_seqs <= CP_SPEC_MAX_PLAN_SEQS, max_pages * page_size and
 * n_seqs * max_pages below 2^31.  Inputs and outputs must not overlap. */
cp_spec_status cp_spec_kv_plan(int32_t n_seqs, int32_t max_pages, int32_t page_size, int32_t n_pages, const int32_t* d_len,
                               const int32_t* d_new, int32_t* d_pages, int32_t* d_held, int32_t* d_free, int32_t* d_n_free,
                               int32_t n_rows, int32_t* d_kv_len, int32_t* d_row_start, int32_t* d_pos, int64_t* d_slot,
                               int32_t* d_refused, void* stream);

/* A rotary embedding: pair i (channels i and i + rot_dim / 2 of a head, the
 * rotate-half pairing of cp_spec_model) turns by the position on its axis times
 * theta^(-2 i / rot_dim), i counted over all axes; channels from rot_dim on stay.  Filled by
 * cp_spec_rope_init, a host function without device work; the struct is read
 * during the calls that take it.  Another rule (frequencies that begin anew at each
 * axis, as image encoders have, or scaled ones) is written into turns and axis
 * after that: any turns, and axis below n_axes. */
typedef struct {
  int32_t rot_dim, n_axes;
  uint8_t axis[128];   /* axis of each pair                                      */
  uint64_t turns[128]; /* frequency of each pair: turns per position, times 2^64 */
} cp_spec_rope;

/* rot_dim: a multiple of 16 up to 256; 1 <= theta <= 1e30; n_axes 1..4 (time,
 * height, width, ...).  HOST sections [n_axes]: pairs of each axis, rot_dim / 2 in
 * all (NULL with one axis).  interleaved 0: the first sections[0] pairs belong to
 * axis 0, the next to axis 1, and so on; 1: pair i belongs to axis a = i mod n_axes
 * where a > 0 and i < n_axes * sections[a], else to axis 0. */
cp_spec_status cp_spec_rope_init(cp_spec_rope* rope, int32_t rot_dim, double theta, int32_t n_axes, const int32_t* sections,
                                 int32_t interleaved);

/* Rotates rows of queries and keys: d_q [n_rows][n_q_heads][head_dim], d_k
 * [n_rows][n_k_heads][head_dim] of dtype (0 float32, 1 bfloat16, 2 float16), row
 * strides in elements, a row dense; into d_q_out, d_k_out (which may be the inputs,
 * with their stride).  n_q_heads or n_k_heads may be 0.  d_pos [n_axes][pos_stride]
 * int32, any sign; pos_stride 0: all axes have the same positions.  head_dim: a
 * multiple of 16 up to 256, >= rot_dim.  A position times its frequency (53 bits)
 * is reduced to a turn exactly, and the result is rounded once. */
cp_spec_status cp_spec_rope_rows(const cp_spec_rope* rope, int32_t n_rows, int32_t head_dim, int32_t dtype, const int32_t* d_pos,
                                 int64_t pos_stride, int32_t n_q_heads, const void* d_q, int64_t q_stride, void* d_q_out,
                                 int64_t q_out_stride, int32_t n_k_heads, const void* d_k, int64_t k_stride, void* d_k_out,
                                 int64_t k_out_stride, void* stream);

/* A KV cache of 16-bit elements (dtype 1 bfloat16, 2 float16): keys, then values,
 * each [n_pages][n_kv_heads][page_size][head_dim] and dense.  page_size: a power of
 * two from 16 to 1024; head_dim 64, 128 or 256; n_kv_heads up to 1024, n_kv_heads *
 * page_size * n_pages below 2^40.  The caller owns the memory
 * (cp_spec_kv16_bytes, 16-byte aligned). */
typedef struct {
  int32_t n_pages, page_size, n_kv_heads, head_dim, dtype;
} cp_spec_kv16;

/* Bytes of the cache, 0 if the shape is invalid. */
size_t cp_spec_kv16_bytes(const cp_spec_kv16* shape);

/* Writes rows of keys and values [n_rows][n_kv_heads][head_dim] of the cache's
 * type to slots d_slot [n_rows] (page * page_size + offset).  With rope (d_pos,
 * pos_stride as in cp_spec_rope_rows) the keys are rotated as they are written, and
 * queries d_q [n_rows][n_q_heads][head_dim] (n_q_heads may be 0) into d_q_out, all
 * in one kernel.  A row whose slot is outside the cache (padding) is left out
 * whole, its queries too.  Two rows with one slot leave it undefined. */
cp_spec_status cp_spec_kv16_append(const cp_spec_kv16* shape, void* d_cache, int32_t n_rows, const int64_t* d_slot, const void* d_k,
                                   int64_t k_stride, const void* d_v, int64_t v_stride, const cp_spec_rope* rope,
                                   const int32_t* d_pos, int64_t pos_stride, int32_t n_q_heads, const void* d_q, int64_t q_stride,
                                   void* d_q_out, int64_t q_out_stride, void* stream);

/* Attention of rows over the cache.  d_pages [n_seqs][max_pages] as for the 4-bit
 * cache (NULL: sequence b owns pages b * max_pages ..; positions whose entry is
 * outside [0, n_pages) are left out; max_pages * page_size at most 2^31 - 1024).
 * Sequence b has d_kv_len[b] positions (clamped to 0 .. max_pages * page_size), the
 * last m of them its rows, already appended: m =
 * d_row_start[b + 1] - d_row_start[b], at most max_rows, and 0 where that range does
 * not lie in 0 .. n_rows.  Row i is at position p = base + i, base = d_kv_len[b] - m
 * (which may be negative; positions below 0 do not exist), and sees the positions
 * j <= p with j > p - window or j < sinks (window 0: all of them).
 * With d_mask [n_rows] uint64 (max_rows <= CP_SPEC_MAX_TREE_ROWS) the rows are the
 * nodes of a sparse tree: of its sequence's own rows, a row sees base + j for every
 * bit j of its mask (ancestors and itself), and of the positions below base those
 * that window and sinks leave for p = base + (bits set) - 1, the node's depth.
 *   o = softmax(scale q k^T) v,  scale of magnitude at most 2^127,
 * d_q, d_o (out) [n_rows][n_q_heads][head_dim] of the cache's type, row strides in
 * elements; query head e reads KV head e / (n_q_heads / n_kv_heads).  d_lse
 * (optional, out) [n_rows][n_q_heads] float32: the log of the sum of the
 * exponentials.  A row that sees nothing gives zeros and -infinity.  What is stored
 * at a position that a row does not see cannot reach it, not by a bit; an infinity
 * or NaN among the values reaches every row that sees it.
 * Scores, sums and the softmax are float32; sums of finite values stay finite, and
 * values down to 2^-100 keep their bits.  A weight enters the product with the
 * values as a sum of two numbers of the cache's type, or, where many rows of a
 * sequence share the tiles of the tensor cores, as one; an fp16 weight far below
 * its row's largest is off by up to 2^-40 of that largest besides, as one number by
 * 2^-32, or 2^-38 where those around it are as small.  Results do not depend on
 * timing or on the other sequences' contents, but the call's sizes choose the
 * kernel and how a long sequence is split, which moves them within rounding.
 * d_work: cp_spec_kv16_attention_bytes of scratch (NULL where that is 0), used
 * during the call's work only; calls that overlap in time need their own.
 * d_status (optional, device, one int32, 4-byte aligned): set to
 * CP_SPEC_E_DEVICE_TIMEOUT if it was 0 and a bounded wait of a kernel ran out (the
 * outputs are then incomplete); else left as it is. */
cp_spec_status cp_spec_kv16_attention(const cp_spec_kv16* shape, const void* d_cache, const int32_t* d_pages, int32_t max_pages,
                                      int32_t n_seqs, int32_t n_rows, int32_t max_rows, int32_t n_q_heads, const int32_t* d_kv_len,
                                      const int32_t* d_row_start, const uint64_t* d_mask, int32_t window, int32_t sinks, float scale,
                                      const void* d_q, int64_t q_stride, void* d_o, int64_t o_stride, float* d_lse, void* d_work,
                                      size_t work_bytes, int32_t* d_status, void* stream);

/* Workspace of that call on the current device (tree: whether it has masks): 0
 * unless sequences are split; also 0 if the arguments are invalid. */
size_t cp_spec_kv16_attention_bytes(const cp_spec_kv16* shape, int32_t max_pages, int32_t n_seqs, int32_t n_rows, int32_t max_rows,
                                    int32_t n_q_heads, int32_t window, int32_t sinks, int32_t tree);

/* Decode without any allocation: cp_spec_decode_frames for a one-off job,
 * with no context and no caller workspace.  The pages describe no such call;
 * it exists for callers that cannot allocate device memory when they decode:
 * a runtime with no device allocator of its own, a host whose memory pool is
 * frozen after start-up, or one that must keep its device footprint fixed.
 * The KV cache, activations, sampling lists and stream state live instead in
 * a library-owned array of CP_SPEC_STATIC_SCRATCH_BYTES in the module's
 * global memory, reserved by the CUDA runtime when the library's module is
 * loaded (one copy per device).
 *
 * Arguments are those of cp_spec_init plus cp_spec_decode_frames (same
 * layouts; streams 0..n_streams-1, n_streams <= config->max_streams).  The
 * workspace it needs is cp_spec_workspace_bytes(model, config); above
 * CP_SPEC_STATIC_SCRATCH_BYTES the call returns CP_SPEC_E_WORKSPACE and
 * enqueues nothing (lower max_streams).  d_status (optional, device, one
 * int32, 4-byte aligned; the other device pointers need 16 bytes) receives
 * the device status word after the decode: CP_SPEC_OK,
 * CP_SPEC_E_DEVICE_TIMEOUT or CP_SPEC_E_DEVICE.
 *
 * Every call clears the scratch, resets it to the state cp_spec_init leaves
 * (on `stream`, before the decode) and decodes: results equal those of a
 * fresh context with the same config, bit for bit.  Per-stream sampling
 * overrides and counters are not available.  Asynchronous; returns
 * CP_SPEC_W_AR_FALLBACK under the same condition as cp_spec_init.
 *
 * The first call on each device looks up the scratch address
 * (cudaGetSymbolAddress, which may load the module) and caches it; make that
 * first call before any stream capture begins.  The decode runs as a call
 * graph (host objects, no device allocation by the library) that is cached
 * per device and rebuilt, after a device synchronisation, when the model,
 * weights or configuration change.  All calls on one device share
 * the one scratch array: calls whose work overlaps in time (different
 * streams, or threads without ordering) race on it and give wrong results.
 * Order them on one stream.  Launches count in the context-free counter of
 * cp_spec_launch_count(NULL). */
cp_spec_status cp_spec_decode_frames_static(const cp_spec_model* model, const cp_spec_weights* weights,
                                            const cp_spec_config* config, int32_t n_streams, int32_t n_frames,
                                            int32_t first_frame, const float* d_x, const int32_t* d_c0,
                                            int32_t* d_codes, int32_t* d_status, void* stream);

/* Synchronise `stream` and return the device status word of the context:
 * CP_SPEC_OK, CP_SPEC_E_DEVICE_TIMEOUT or CP_SPEC_E_DEVICE.  Clears it. */
cp_spec_status cp_spec_status_word(cp_spec_ctx* ctx, void* stream);

/* Synchronise `stream` and copy the counters to *h_stats. */
cp_spec_status cp_spec_read_stats(cp_spec_ctx* ctx, cp_spec_stats* h_stats, void* stream);
cp_spec_status cp_spec_reset_stats(cp_spec_ctx* ctx, void* stream);

/* Diagnostic hook for tests (the pages have no counterpart).
 * wait_limit_ns (1e4 .. 6e10; default 2e9) bounds every device-side wait of
 * the context's kernels (a weight or input copy that has not landed): after
 * it the kernel records CP_SPEC_E_DEVICE_TIMEOUT in the status word, waits
 * (with the same bound) for its own copies still in flight and returns; the
 * pass loop then stops.  flags (0 .. 3):
 *   bit 0 (1): one wait of the first decoder kernel of every pass (CTA 0)
 *     never completes, so that wait always runs out;
 *   bit 1 (2): after each decision the accept kernel writes NaN into every
 *     KV slot of the stream that the next pass must not read (positions past
 *     the committed depth, the tree nodes' slots, and at a frame's end the
 *     whole cache), so a pass that read a stale slot would show NaN
 *     ("Speculative Decoding, Beyond Text", section 07: the logical length
 *     and the valid-position mask).
 * 0 restores normal operation.  Nothing traps or spins without a bound.
 * Packed weights have no bounded wait (bit 0) and a 4-bit cache no float slots
 * (bit 1): CP_SPEC_E_UNSUPPORTED there.
 * ctx NULL: the waits of cp_spec_kv16_attention, in all later calls of the process;
 * flags 1: the last copy of every CTA is not made, 2: none is, so that the waits
 * for it run out and the call's d_status says so.
 * Synchronises the device if the context's call graph exists (it is rebuilt
 * on the next call). */
cp_spec_status cp_spec_test_hooks(cp_spec_ctx* ctx, uint64_t wait_limit_ns, int32_t flags);

/* Number of launches the library has enqueued on this context: kernels
 * launched directly, plus one per launch of the context's call graph (whose
 * pass kernels are counted on the device: cp_spec_stats.kernel_launches).
 * cp_spec_accept_batch, the 4-bit operators, those of the 16-bit cache and
 * cp_spec_decode_frames_static count in a process-wide counter, ctx = NULL. */
int64_t cp_spec_launch_count(const cp_spec_ctx* ctx);

/* Last error message of the context, or (ctx NULL) of the last call without a
 * context that the calling thread made and that was refused; valid until that
 * thread's next refused call.  Never NULL. */
const char* cp_spec_last_error(const cp_spec_ctx* ctx);

/* Release the host context.  Does not touch the caller's device memory. */
void cp_spec_destroy(cp_spec_ctx* ctx);

#ifdef __cplusplus
}
#endif
#endif /* CP_SPEC_H */
