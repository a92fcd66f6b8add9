/*
 * gocr.h - C ABI of the GB300 self-speculative block decoder.
 *
 * The library runs the decode round of a decoder trained for both AR and
 * block-diffusion decoding (GravityOCR, "Diffusion Drafts, AR Verifies"):
 *
 *   draft   one forward of [x0, M x B]: the boundary token x0 reads the cache
 *           causally and yields a0; the B [M] rows read the cache and the whole
 *           window bidirectionally and yield drafts d1..dB
 *           (GravityOCR review, §3.2 "Self-Speculative Decoding");
 *   verify  one token-causal forward of [a0, d1..dB] yields a1..a(B+1) and
 *           overwrites the draft's KV slots with causal state in place
 *           (review, Appendix B.2 "Self-Speculative Decoding and KV-Cache Update");
 *   accept  A = longest prefix with d_j == a_j; commit a0, d1..dA, a(A+1);
 *           the rejected suffix is rolled back (velog review, inference section).
 *
 * Everything runs on one GPU in hand-written sm_103a kernels.  All entry points
 * return GOCR_OK (0) or a negative GOCR_E* code; nothing throws across the ABI.
 * A handle is not thread-safe: calls on one handle must not overlap.
 *
 * Layouts: every matrix is row-major [out, in] (y = x W^T), elements in the
 * handle's dtype (fp32, or bf16 as uint16 bit patterns).  Norm gains are fp32.
 */
#ifndef GOCR_H
#define GOCR_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ---------------------------------------------------- */
#define GOCR_OK          0
#define GOCR_EINVAL     (-1) /* bad argument: null pointer, size out of range   */
#define GOCR_ECAPACITY  (-2) /* KV capacity, rows or block size over the limit  */
#define GOCR_ECUDA      (-3) /* a CUDA runtime call failed (see gocr_last_error) */
#define GOCR_EDEVICE    (-4) /* a kernel raised its error word (NaN logits ...)  */
#define GOCR_ETIMEOUT   (-5) /* the on-device round loop hit its round limit     */
#define GOCR_ENOMEM     (-6) /* allocation failed                                */
#define GOCR_ESTATE     (-7) /* call order: decode before prefill, and the like  */

enum { GOCR_DTYPE_F32 = 0, GOCR_DTYPE_BF16 = 1 };
/* decode modes: AR greedy (one token per forward), self-speculative rounds,
 * and (gocr_decode_ex) direct block diffusion and self-speculative rounds
 * with a refined draft */
enum { GOCR_MODE_AR = 0, GOCR_MODE_SELFSPEC = 1, GOCR_MODE_DIFFUSION = 2, GOCR_MODE_REFINED = 3 };
/* single-forward kinds for gocr_debug_forward */
enum { GOCR_FWD_AR = 0, GOCR_FWD_DRAFT = 1, GOCR_FWD_VERIFY = 2 };

#define GOCR_MAX_BLOCK 64      /* largest block size B */
#define GOCR_LAYER_TENSORS 9   /* wq wk wv wo wg wu wd g_attn g_mlp */

/* Model and capacity.  q_dim = n_q_heads*head_dim and kv_dim =
 * n_kv_heads*head_dim must be multiples of 128, head_dim 64 or 128, ffn a
 * multiple of 64, hidden and vocab multiples of 128, n_q_heads a multiple of
 * n_kv_heads. */
typedef struct gocr_config {
  int32_t n_layers, hidden, n_q_heads, n_kv_heads, head_dim, ffn, vocab;
  int32_t dtype;          /* GOCR_DTYPE_F32 | GOCR_DTYPE_BF16 */
  float rms_eps;          /* RMSNorm epsilon (1e-6) */
  float rope_theta;       /* rotary base (1e4) */
  int32_t max_ctx;        /* KV positions per request: >= P + max_new + B + 2 */
  int32_t max_block;      /* largest B the handle will be asked for (<= 64) */
  int32_t max_requests;   /* request slots (KV caches) */
  int32_t eos_id;         /* stop token, -1 = none */
} gocr_config;

/* Device pointers to the weights.  The caller owns them and keeps them alive
 * until gocr_free; the handle copies the projections it re-packs (QKV fused,
 * gate/up interleaved) at create time and reads the others in place. */
typedef struct gocr_weights {
  const void* embed;        /* [vocab, hidden] dtype */
  const void* mask_embed;   /* [hidden] dtype: the single [M] row */
  const void* lm_head;      /* [vocab, hidden] dtype (untied) */
  const float* g_final;     /* [hidden] fp32 */
  /* host array of n_layers * GOCR_LAYER_TENSORS device pointers, per layer:
   * wq [Hq*d, h], wk [Hkv*d, h], wv [Hkv*d, h], wo [h, Hq*d], wg [F, h],
   * wu [F, h], wd [h, F] (dtype), g_attn [h], g_mlp [h] (fp32) */
  const void* const* layer;
} gocr_weights;

/* Decode statistics (review §4.1 eq. 5: TPF = committed / forwards, the
 * prefill excluded; a round with A accepted drafts commits A + 2 tokens). */
typedef struct gocr_stats {
  int64_t rounds;           /* self-spec rounds, or AR steps                  */
  int64_t forwards;         /* draft + verify forwards (AR: one per token)    */
  int64_t committed;        /* decode-committed tokens (prefill token not in) */
  int64_t accepted_drafts;  /* sum of A over rounds                          */
  int32_t accept_hist[GOCR_MAX_BLOCK + 1]; /* rounds per accepted count A    */
  double device_ms;         /* device time of the decode call (CUDA events)  */
} gocr_stats;

/* Optional device allocator (for example backed by PyTorch's caching
 * allocator).  Must return 256-byte-aligned device memory or NULL. */
typedef void* (*gocr_alloc_fn)(size_t bytes, void* user);
typedef void (*gocr_free_fn)(void* ptr, void* user);

typedef struct gocr_handle gocr_handle;

/* Create a decoder on the current CUDA device.
 *   stream      cudaStream_t every launch goes to (NULL = legacy default).
 *   alloc/free  device allocator; both NULL = cudaMalloc/cudaFree.
 * Returns GOCR_EINVAL for an unsupported shape (including more than 64 q
 * heads per kv head, or more than 2^20 attention rows (token, q head) in one
 * forward: max(max_ctx, max_requests x (max_block + 1)) x q heads per kv
 * head), GOCR_ENOMEM, GOCR_ECUDA. */
int gocr_create(const gocr_config* cfg, const gocr_weights* w, void* stream,
                gocr_alloc_fn alloc, gocr_free_fn free_fn, void* alloc_user,
                gocr_handle** out);

/* Causal prefill of request slot `req` from P prefix embeddings (the image +
 * prompt prefix, [P, hidden] in dtype; host or device pointer, copied before
 * the call returns).  Resets the slot: the argmax of the last row becomes
 * out[0] and the boundary token x0; the cache holds positions 0..P-1.
 * GOCR_ECAPACITY if P + 1 > max_ctx. */
int gocr_prefill(gocr_handle* h, int req, const void* prefix_embeds, int P);

/* Decode request `req` until max_new tokens are in out (out[0], the prefill
 * token, counts) or eos.  mode GOCR_MODE_AR commits one token per forward;
 * GOCR_MODE_SELFSPEC runs draft/verify/accept rounds of block size B.  The
 * whole loop runs on the device (a CUDA graph with a device-side while loop,
 * no host synchronisation between rounds); the call blocks until it ends and
 * then copies out_tokens (host, caller-owned, >= max_new entries) and stats
 * (may be NULL).  GOCR_ECAPACITY if P + max_new + B + 2 > max_ctx. */
int gocr_decode(gocr_handle* h, int req, int mode, int B, int max_new,
                int32_t* out_tokens, gocr_stats* stats);

/* Batched decode of n_req prefilled request slots in one round loop: every
 * forward concatenates the requests' windows (ragged caches, one position
 * sequence per request).  max_new[i] per request; out_tokens[i] host buffers;
 * stats: array of n_req or NULL.  Finished requests stop committing while
 * the others continue. */
int gocr_decode_batch(gocr_handle* h, int n_req, const int32_t* reqs, int mode, int B,
                      const int32_t* max_new, int32_t* const* out_tokens, gocr_stats* stats);

/* Options of the block-step decodes. */
typedef struct gocr_decode_opts {
  float tau;            /* DIFFUSION: the confidence threshold tau_c; REFINED: the
                           draft-side threshold.  Confidence = the largest softmax
                           probability of a row; a value equal to tau passes. */
  int32_t draft_steps;  /* REFINED: draft forwards per round at most, 1..64 */
  float temperature;    /* AR, SELFSPEC: 0 = greedy; > 0 = sampling from
                           softmax(logits / temperature) (see below) */
  uint32_t reserved;    /* 0 */
  uint64_t seed;        /* sampling: key of the random numbers */
} gocr_decode_opts;

/* gocr_decode_batch with every mode, one forward per device-loop iteration
 * for the two block-step modes (opts required for them, ignored otherwise):
 *
 *   GOCR_MODE_DIFFUSION  direct block-diffusion decoding (GravityOCR review,
 *     §2 "Block Diffusion" and Appendix B.1 "Direct Block-Diffusion
 *     Decoding"): a block of B slots at positions p+1..p+B starts as [M];
 *     each denoising step forwards the draft window [x0, slots] (x0 causal,
 *     the slots reading the cache and the whole window) and fixes every masked
 *     slot whose confidence reaches tau (slot s takes the argmax of the row at
 *     position p+s-1, the shift-by-one convention), or else the single most
 *     confident masked slot (the lowest slot among equals).  A finished block
 *     commits its B tokens (cut at max_new and after the first eos); unless
 *     decoding stops there, a token-causal cache-write forward of [x0,
 *     y_1..y_B] at p..p+B follows, the cache keeps positions 0..p+B-1 and
 *     y_B becomes the boundary.  Stats: rounds = blocks, forwards = denoising
 *     steps + cache writes, accept_hist[k] = blocks finished in k steps,
 *     accepted_drafts = 0.
 *   GOCR_MODE_REFINED  self-speculative rounds whose draft runs up to
 *     draft_steps denoising forwards (review Appendix D, "Draft Schedule"):
 *     each step fixes slots by the rule above with the draft-side threshold;
 *     after the last step (or when every slot is fixed) the verify window is
 *     [slot 1..slot B, the last step's prediction at position p+B+1], unfixed
 *     slots taking the last step's predictions; verify, accept and rollback
 *     are those of GOCR_MODE_SELFSPEC, so the output equals AR greedy.
 *     draft_steps = 1 is the one-shot round (the same tokens, stats and bits
 *     as GOCR_MODE_SELFSPEC).  Stats: forwards = draft steps + verifies.
 *
 *   Sampling (GOCR_MODE_AR or GOCR_MODE_SELFSPEC with temperature > 0): the
 *     decode tokens are drawn from softmax(logits / temperature) (the
 *     prefill token stays the greedy argmax).  Self-speculative rounds then
 *     use the speculative acceptance-rejection rule (review §2 "Speculative
 *     Decoding"; the blog: the rule preserves the AR distribution): a0 is
 *     drawn from the boundary row, d_j from [M] row j (draft distribution
 *     q_j); verify row j - 1 gives the target p_j; d_j is accepted when a
 *     uniform u_j < min(1, p_j(d_j) / q_j(d_j)); the first rejection draws
 *     the replacement from max(0, p_j - q_j) renormalised, B acceptances
 *     draw the bonus from verify row B; commit and rollback as in the greedy
 *     round.  Random numbers: Philox4x32-10 (Salmon et al., SC 2011), key
 *     (seed low word, seed high word), counter (v / 4, position, purpose,
 *     request slot), lane v % 4, uniform ((x >> 9) + 0.5) / 2^23; a draw is
 *     a Gumbel-max, argmax of score_v - log(-log u_v) with the lowest index
 *     among equals; purposes 0 a target token at its position (AR steps, a0,
 *     the bonus), 1 a draft token, 2 an acceptance uniform (v = 0), 3 a
 *     replacement; the token at absolute position t uses position t.
 *
 * No forced-acceptance override applies to the block-step modes or to
 * sampling.  Errors as gocr_decode_batch; GOCR_EINVAL for a NaN threshold,
 * draft_steps out of range, a negative or NaN temperature, or a temperature
 * with the block-step modes. */
int gocr_decode_ex(gocr_handle* h, int n_req, const int32_t* reqs, int mode, int B, const gocr_decode_opts* opts,
                   const int32_t* max_new, int32_t* const* out_tokens, gocr_stats* stats);

/* Forced-acceptance hook for request `req` (host arrays, copied):  in round r
 * with c tokens committed, drafts become d_j = ref[c+j] for j <= G_r and
 * d_(G_r+1) = (ref[c+G_r+1] + 1) mod vocab, G_r = schedule[r] (rounds past
 * n_rounds use G = 0; positions past n_ref keep the model's draft).
 * n_ref = 0 removes the hook.  Applied between draft and verify. */
int gocr_set_draft_override(gocr_handle* h, int req, const int32_t* ref_tokens, int n_ref,
                            const int32_t* schedule, int n_rounds);

/* One forward at the request's current state, for parity checks; nothing is
 * committed and cache_len is unchanged (KV slots at and after cache_len are
 * written).  kind AR: tokens = [x], n = 1, at position cache_len.  DRAFT:
 * tokens[0] = x0 and n = B + 1 (rows 1..B are [M]), positions cache_len.. .
 * VERIFY: tokens = [a0, d1..dB], n = B + 1, positions cache_len+1.. (call it
 * after a DRAFT at the same state, which wrote x0's slot).  logits_out: host
 * [n, vocab] fp32, or NULL. */
int gocr_debug_forward(gocr_handle* h, int req, int kind, const int32_t* tokens, int n,
                       float* logits_out);

/* gocr_debug_forward over n_req prefilled request slots in one batched
 * forward, as gocr_decode_batch runs its rounds: request i's window is rows
 * [i n, (i + 1) n) with tokens[i n .. (i + 1) n) (same per-kind meaning as
 * above, each at its own request's cache length), and logits_out (host, or
 * NULL) receives [n_req n, vocab] fp32 in that row order.  The requests are
 * distinct; GOCR_ECAPACITY when a window does not fit its cache. */
int gocr_debug_forward_batch(gocr_handle* h, int n_req, const int32_t* reqs, int kind, const int32_t* tokens,
                             int n, float* logits_out);

/* Copy n cached positions from pos0 of layer `layer` to host buffers
 * k_out/v_out, each [n, n_kv_heads, head_dim] fp32 (keys are stored rotated;
 * bf16 models keep the cache as bf16 hi + lo planes, returned as their sum). */
int gocr_read_kv(gocr_handle* h, int req, int layer, int pos0, int n, float* k_out, float* v_out);

/* Current cache length (position of the boundary token) and boundary token. */
int gocr_get_state(gocr_handle* h, int req, int32_t* cache_len, int32_t* x0);

/* Read-only handle properties.
 *   GOCR_OPT_ATTENTION  the tensor-core attention kernels of a bf16 handle,
 *                     fixed at create time:
 *     GOCR_ATTN_MMA_SYNC  64-row tiles on mma.sync;
 *     GOCR_ATTN_TCGEN05  128-row tiles with both contractions on tcgen05 and
 *       their accumulators in tensor memory.
 *   A handle takes TCGEN05 when its key-chunk ranks average at least four
 *   32-key chunks at full capacity (batched handles), MMA_SYNC otherwise;
 *   GOCR_ATTN=tc or GOCR_ATTN=mma in the environment at create time
 *   overrides (gocr_op_attention reads it per call; MMA_SYNC by default).
 *   The two round differently; each is bit-consistent across its own
 *   forwards.
 *   GOCR_OPT_ATTN_RANKS  key-chunk ranks of the handle's attention (the
 *                     split of a row's keys, fixed at create time).
 * GOCR_EINVAL for an unknown option. */
enum { GOCR_OPT_ATTENTION = 5, GOCR_OPT_ATTN_RANKS = 6 };
enum { GOCR_ATTN_TCGEN05 = 0, GOCR_ATTN_MMA_SYNC = 1 };
int gocr_get_option(const gocr_handle* h, int option, int* value);

/* Timeline of the last debug forward (a profiling aid; GOCR_ESTATE when the
 * trace is off).  out: host, at least n_words words.
 *   GOCR_TRACE_KERNELS  one record per launch of a debug forward (on with
 *     GOCR_OP_TRACE=1 in the environment at create time): n_words >=
 *     8 * (5 * n_layers + 1), laid out [launch][8] in forward order (per
 *     layer QKV, attention, O, gate/up, down; then the LM head); a record is
 *     (first CTA start, first and last release from the dependency wait,
 *     last CTA end, last mainloop end, last split-K exchange end, 0, 0),
 *     globaltimer ns (the last two marks for GEMMs only). */
/*   GOCR_TRACE_CTAS  the same launches with one record per CTA (on with
 *     GOCR_OP_TRACE=2): n_words >= 8 * 2048 * (5 * n_layers + 1), laid out
 *     [launch][CTA slot][8]; CTA c of a kernel (linear block index) fills slot
 *     c, the attention merge kernel's CTAs slots 1024 + c; a record is (start,
 *     release from the dependency wait, GEMM epilogue start, end, then as the
 *     launch records: mainloop end, split-K exchange end, cluster barrier
 *     passed, accumulator drained; attention: first chunk ready, chunk loop
 *     done, merge start), zero where a CTA did not reach a mark. */
enum { GOCR_TRACE_KERNELS = 1, GOCR_TRACE_CTAS = 2 };
int gocr_read_trace(gocr_handle* h, int which, uint64_t* out, size_t n_words);

/* Last error message of the handle (or of the library when h is NULL). */
const char* gocr_last_error(const gocr_handle* h);

void gocr_free(gocr_handle* h);

/* ---- single-kernel entry points (parity tests, device pointers) --------- */

/* y[T, N] (fp32) = x[T, K] w[N, K]^T, the decoder's weight-streaming GEMM with
 * its fixed split-K reduction (the split count depends on N and K only, so a
 * row's result does not depend on T).  x and w in dtype, K % 8 == 0.
 * workspace: device, >= gocr_op_linear_workspace(T, N, K) bytes, all zero
 * before the first call (the kernel leaves it ready for the next call). */
size_t gocr_op_linear_workspace(int T, int N, int K);
int gocr_op_linear(int dtype, const void* x, const void* w, float* y, int T, int N, int K,
                   void* workspace, size_t workspace_bytes, void* stream);

/* y[T, N] (fp32) = (x_hi + x_lo)[T, K] w[N, K]^T with bf16 planes x_hi,
 * x_lo and bf16 w: the decoder's GEMM on the hi + lo activation planes its
 * epilogues write (each K chunk takes the hi and the lo products as separate
 * tensor-core accumulators, adds them, and the chunk sums are added in chunk
 * order).  Up to two 128-row token slices split each tile's K chunks over a
 * thread-block cluster; more rows run them in one CTA per 64-token slice.
 * Either way a row's bits depend on neither T nor the kernel that ran it.  K % 8 == 0; x_hi, x_lo,
 * w 16-byte aligned.  workspace: as gocr_op_linear.
 * flags: 0, or GOCR_OP_OVERLAP: launched as the decoder launches it, with
 * programmatic dependent launch, so that it may start while the stream's
 * previous kernel finishes.  It then fetches w before that kernel has
 * completed (x_hi, x_lo and y only after): w must not be written by it.
 * Errors: GOCR_EINVAL (null pointer, shape, flags), GOCR_ECAPACITY
 * (workspace), GOCR_ECUDA (launch). */
#define GOCR_OP_OVERLAP 1u
int gocr_op_linear_planes(const void* x_hi, const void* x_lo, const void* w, float* y, int T, int N, int K,
                          void* workspace, size_t workspace_bytes, unsigned flags, void* stream);

/* Grouped-query attention of one request window against a KV cache, the
 * decoder's kernel for that dtype.  Operands are planes, as the decoder keeps
 * them: for GOCR_DTYPE_BF16, bf16 hi and lo arrays with v = hi + lo (tensor
 * cores, about 16 significant bits); for GOCR_DTYPE_F32, fp32 arrays in *_hi
 * with the lo pointers NULL.  q [T, Hq, d], k and v [Hkv, cap, d] (device);
 * o [T, Hq, d] fp32 (device); lim: device int32[T], row t reads keys
 * 0..lim[t] (draft: row 0 = p, rows 1..B = p+B; verify/AR: the row's own
 * position).  d in {64, 128}; Hq / Hkv <= 64 and T x Hq / Hkv <= 2^20
 * (GOCR_EINVAL otherwise).  GOCR_DTYPE_BF16 reads K and V by TMA: the four
 * K/V planes must be 16-byte aligned (GOCR_EINVAL otherwise).  GOCR_DTYPE_BF16 keeps its partial rows in a
 * device scratch buffer of the library (one per device, allocated or grown
 * by the first call that needs more): calls that overlap on the GPU race. */
int gocr_op_attention(int dtype, const void* q_hi, const void* q_lo, const void* k_hi, const void* k_lo,
                      const void* v_hi, const void* v_lo, float* o, const int32_t* lim, int T, int Hq, int Hkv,
                      int d, int cap, void* stream);

/* gocr_op_attention with a second key interval per row: row t reads keys
 * 0..lim[t] and lo2[t]..hi2[t] (none when hi2[t] < lo2[t]); lo2, hi2:
 * device int32[T], both NULL = the plain call.  With lo2/hi2 given, the
 * bf16 path splits each row tile's keys over fewer ranks as T grows (at most
 * two waves of the kernel's resident CTAs) and runs the tcgen05 kernel when
 * its ranks average at least four 32-key chunks, else the mma.sync kernel
 * (GOCR_ATTN=tc / mma forces one): a row's result then depends on T in its
 * last bits (the plain call's does not).  Key chunks masked for every row of
 * a tile are skipped, which changes no bits. */
int gocr_op_attention_ranges(int dtype, const void* q_hi, const void* q_lo, const void* k_hi, const void* k_lo,
                             const void* v_hi, const void* v_lo, float* o, const int32_t* lim, const int32_t* lo2,
                             const int32_t* hi2, int T, int Hq, int Hkv, int d, int cap, void* stream);

/* Row key intervals of the joint AR / block-diffusion training attention
 * (GravityOCR review §3.1 "Joint AR-Diffusion Training"; the Trillion Labs
 * blog's three-stream figure): one forward over the packed sequence
 * [prefix (P), clean response (N), corrupted stream 1 (N), corrupted stream
 * 2 (N)], responses cut into blocks of B tokens.  The prefix (image and
 * prompt, never corrupted) and the clean stream are causal; a token of block
 * b of a corrupted stream reads the prefix, the clean blocks before b and
 * the whole of its own corrupted block b (bidirectional), and nothing of the
 * other corrupted stream, of its own stream's other blocks, or of clean
 * block b and later.  Host outputs, [P + 3 N] each: lim, lo2, hi2 as
 * gocr_op_attention_ranges reads them, and pos (or NULL) the rotary
 * position of each row (a stream's response token i sits at P + i).
 * GOCR_EINVAL for negative sizes, B < 1, or a null output. */
int gocr_three_stream_ranges(int P, int N, int B, int32_t* lim, int32_t* lo2, int32_t* hi2, int32_t* pos);

/* ---- training and scoring operators (device pointers) -------------------
 *
 * The two ends of a decoder's training step and its attention over packed
 * sequences, forward (which also scores and prefills) and backward.  For all
 * of them: row-major arrays, device memory of the current device, `stream` a
 * stream of the current device (GOCR_EINVAL otherwise); bf16 operands, the
 * embedding's arrays and workspaces aligned to 16 bytes, other int32 and fp32
 * arrays to 4; nothing is allocated, kept between calls or synchronised, so a call
 * can be captured into a graph; a workspace need not be cleared and belongs to
 * one call at a time (for calls of several shapes: the largest of their sizes,
 * which need not be that of the largest shape).  The same inputs give the same
 * bits.  Outputs must not overlap inputs.  Zero rows (T = 0) are allowed:
 * gradients of weights are then zero.  Errors: GOCR_EINVAL (null pointer, shape,
 * alignment, stream), GOCR_ECAPACITY (workspace), GOCR_ECUDA (launch). */

/* y[T, H] = scale * row(ids[t]), rounded once to dtype: row(id) is embed[id]
 * for 0 <= id < V, mask_embed for id = -1 (the [M] row; zero when mask_embed
 * is NULL), and zero for every other id (padding).  embed [V, H], mask_embed
 * [H] and y in dtype, ids int32[T] (device).  H % 8 == 0, H <= 2^20, T and
 * V <= 2^28. */
int gocr_op_embed(int dtype, const void* embed, const void* mask_embed, const int32_t* ids, void* y, int T, int H,
                  int V, float scale, void* stream);

/* Gradient of gocr_op_embed: d_embed[V, H] (dense: rows of tokens that do not
 * occur are zero) and d_mask[H] (NULL: not wanted) from dy[T, H], all in
 * dtype.  Positions are sorted by token; a row's sum is in fp32, in an order
 * that follows from ids alone, and is rounded once. */
size_t gocr_op_embed_backward_workspace(int T, int H);
int gocr_op_embed_backward(int dtype, const void* dy, const int32_t* ids, void* d_embed, void* d_mask, int T, int H,
                           int V, float scale, void* workspace, size_t workspace_bytes, void* stream);

/* Causal attention over packed sequences with grouped heads, bf16: sequence s
 * is rows cu_seqlens[s] .. cu_seqlens[s+1] - 1 (device int32[n_seq + 1],
 * non-decreasing, within 0..T; empty sequences allowed; the values stay on the
 * device), and row i of a sequence reads its rows 0..i: o = softmax(scale q
 * k^T) v, lse = the log of the row's sum of exponentials.  q [T, Hq, d] with
 * rows ldq elements apart, k and v [T, Hkv, d] with rows ldk and ldv apart (so
 * the three may be column ranges of one fused projection; pitches % 8 == 0);
 * o [T, Hq, d] bf16 and lse [Hq, T] fp32 dense.  d 64 or 128, Hq % Hkv == 0,
 * 0 < scale <= 1e30, Hq <= 1024, n_seq <= 2^20, T <= 2^24, (n_seq + T) (Hq + Hkv)
 * <= 2^31 - 1, pitches <= 2^32.  exp(scale q k^T - m), with m within 2^8 of the
 * row's maximum so far, is rounded to bf16 for the product with v; scores,
 * softmax statistics and sums are in fp32.  Rows that belong to no
 * sequence are not read into any result, whatever they hold, and their o and
 * lse are left as they were; nothing of one sequence reaches another,
 * non-finite values included.  Within a sequence a non-finite v may reach the
 * rows before it, too, that share its block of 128; a non-finite q or k does not. */
int gocr_op_attention_packed(const void* q, const void* k, const void* v, void* o, float* lse,
                             const int32_t* cu_seqlens, int n_seq, int T, int Hq, int Hkv, int d, long long ldq,
                             long long ldk, long long ldv, float scale, void* stream);

/* Gradient of gocr_op_attention_packed from d_o [T, Hq, d] and the forward
 * call's o and lse: dq [T, Hq, d], dk and dv [T, Hkv, d] bf16, dense (rows that
 * belong to no sequence are left as they were).  dk and dv sum over the q
 * heads of the group; all sums are in fp32, in a fixed order.  P = exp(S - lse)
 * and dS = P (do v^T - delta) are rounded to bf16 for the products with do, q and
 * k.  delta = do . o takes o as it was rounded to bf16; for the first 32 rows of a
 * sequence, which see few keys, it is summed from P and do v^T instead.  Within a
 * sequence a non-finite q, k, v or do may reach all gradients of its block of
 * 128 rows, beside those that depend on it. */
size_t gocr_op_attention_packed_backward_workspace(int T, int Hq);
int gocr_op_attention_packed_backward(const void* d_o, const void* q, const void* k, const void* v, const void* o,
                                      const float* lse, const int32_t* cu_seqlens, void* dq, void* dk, void* dv,
                                      int n_seq, int T, int Hq, int Hkv, int d, long long ldq, long long ldk,
                                      long long ldv, float scale, void* workspace, size_t workspace_bytes,
                                      void* stream);

/* Softmax cross entropy of a linear head: z = x w^T with x [T, H] and w [V, H]
 * in bf16 (fp32 sums), lse[t] = log sum_v exp z[t, v], loss[t] = lse[t] -
 * z[t, labels[t]].  A label outside 0..V-1 marks a row without a target: its
 * loss is zero (lse is written all the same).  The logits are not stored.  H %
 * 8 == 0, H <= 2^15, T and V <= 2^22. */
size_t gocr_op_linear_ce_workspace(int T, int V);
int gocr_op_linear_ce(const void* x, const void* w, const int32_t* labels, float* loss, float* lse, int T, int V,
                      int H, void* workspace, size_t workspace_bytes, void* stream);

/* Gradient of sum_t dloss[t] loss[t]: dx[T, H] and dw[V, H] in bf16, from the
 * forward call's lse.  dloss[t] is the row's weight in the training loss (of a
 * clean or a corrupted stream's mean, say); rows without a target add nothing
 * (their dloss, lse and x count for nothing, whatever they hold).  z is computed
 * again in pieces of the vocabulary; (softmax - one-hot) dloss / u is rounded to
 * bf16 for the products, whose sums are in fp32 and are multiplied by u.  u
 * follows from the smallest and the largest mantissa among the targets' weights
 * and is such that bf16 holds both nearly exactly in units of it: the weight of
 * a mean is no common rounding error, those of two streams' means hardly ever
 * one above 2^-10 (2^-9 at worst).  Weights between the two are rounded as they
 * come, and a row's last bits depend on them. */
/* Bytes: a piece of the softmax gradient (T times the larger of 4,096 columns and
 * 2^25 / T, at most V, in bf16), the fp32 parts of dx and a copy of x; for short
 * calls and small vocabularies more than the logits would take. */
size_t gocr_op_linear_ce_backward_workspace(int T, int V, int H);
int gocr_op_linear_ce_backward(const float* dloss, const void* x, const void* w, const int32_t* labels,
                               const float* lse, void* dx, void* dw, int T, int V, int H, void* workspace,
                               size_t workspace_bytes, void* stream);

/* The same with the forward call's loss[T], too (NULL: without it).  The
 * label's softmax - 1 is -(1 - exp(-loss)) then, with the loss's relative
 * precision.  Without the loss it is the difference of z and lse, of which the
 * rounding of both (about 1e-6 to 1e-5 for logits of tens) is left: rows whose
 * loss is below 1e-3 want the loss. */
int gocr_op_linear_ce_backward_with_loss(const float* dloss, const void* x, const void* w, const int32_t* labels,
                                         const float* loss, const float* lse, void* dx, void* dw, int T, int V, int H,
                                         void* workspace, size_t workspace_bytes, void* stream);

/* ---- paged KV cache (device pointers) -----------------------------------
 *
 * Requests of any length share one pool of pages: the page step hands pages
 * out and takes them back, the write puts a forward's rotated keys and its
 * values into them, and the attention reads them.  One forward of a program
 * that keeps its requests this way is gocr_op_page_step once and, in each
 * layer, gocr_op_kv_write_paged and gocr_op_attention_paged.  The rules of the
 * operators above (stream, alignment, errors, nothing kept, outputs apart from
 * inputs) hold here, too.
 *
 * A request is a row of the block table [n_req, max_pages] (int32, device):
 * position x of request r lies in page table[r, x / page_size], at offset x %
 * page_size; its slot is page * page_size + offset.  page_size is 16, 32, 64,
 * 128 or 256, n_pages * page_size <= 2^31 - 1, max_pages * page_size <= 2^24,
 * n_req <= 4096.  A page belongs to one request. */

/* One layer's cache, bf16: element (page, head, offset, c) of k at k + page *
 * k_page + head * k_head + offset * k_token + c, and of v likewise; strides in
 * elements, multiples of 8, no more than 2^32, and such that no two elements
 * share a place (of a dimension of one entry the stride counts for nothing).
 * Pages that hold a head's tokens together and pages that hold a token's heads
 * together are both served, and pages of several layers or of k and v may be
 * interleaved.  k and v 16-byte aligned. */
typedef struct gocr_paged_kv {
  void* k;
  void* v;
  int64_t k_page, k_head, k_token;
  int64_t v_page, v_head, v_token;
  int32_t n_pages, page_size, n_kv_heads, head_dim;
} gocr_paged_kv;

/* Block tables, row positions and slots of the next forward, from the
 * requests' lengths.  Request r holds the pages of positions 0..held[r]-1; its
 * rows of the forward are positions start[r]..end[r]-1, and afterwards it
 * holds the pages of positions 0..end[r]-1: pages are taken where end needs
 * more, and given back where it needs fewer.  So with p positions cached a
 * draft window is (held, start, end) = (p, p, p+B+1), the verify window over it
 * (p+B+1, p+1, p+B+2), its rollback to A accepted drafts (p+B+2, p+A+2,
 * p+A+2), and the end of a request (held, 0, 0).
 *
 * free_pages[n_pages] is a stack, its lowest *n_free entries the free pages.
 * The pages given back go onto it first, the first one (by request, then by
 * position) on top; then pages are taken from the top, the first need first.
 * Growth that is rolled back leaves the stack as it was, in order.  Pages go to
 * requests in their order: from the first one on whose need, with the needs of
 * those before it, is more than there is, requests that need pages are refused.
 * Refused too are a request whose lengths do not satisfy 0 <= start <= held, start
 * <= end and held, end <= max_pages * page_size (it has no rows), and, from the
 * first one on whose rows end behind row T, all requests, those without rows
 * among them: an end or a rollback behind it gives nothing back, and is asked for
 * again with held_out as held.
 *
 * Outputs: table (in place: entries of pages taken; the others, those of pages
 * given back among them, stay as they were), free_pages (in place, entries at
 * and above *n_free), and
 *   n_free_out[1]       the new *n_free;
 *   held_out[n_req]     end, or held where refused: the next call's held;
 *   kv_len[n_req]       end, or 0 where refused: gocr_op_attention_paged's;
 *   cu_rows[n_req + 1]  request r's rows are cu_rows[r]..cu_rows[r+1]-1, <= T;
 *   pos[T], slots[T]    of each row; -1 of refused requests' rows and of rows
 *                       behind the last one.
 * All int32, on the device; T <= 2^24.  Lengths, tables and stacks that contradict one
 * another give meaningless pages, but no access outside the arrays. */
int gocr_op_page_step(const int32_t* held, const int32_t* start, const int32_t* end, int n_req, int32_t* table,
                      int max_pages, int page_size, int32_t* free_pages, int n_pages, const int32_t* n_free,
                      int32_t* n_free_out, int32_t* held_out, int32_t* kv_len, int32_t* cu_rows, int32_t* pos,
                      int32_t* slots, int T, void* stream);

/* Rotary embedding of a forward's q and k rows and the write of k and v into
 * the cache: for row t at position x = pos[t] and i < d / 2,
 *   (y[i], y[i+d/2]) = (c u[i] - s u[i+d/2], c u[i+d/2] + s u[i]),
 * c and s the cosine and sine of x theta^(-2i/d), for each head of q (into
 * q_out[T, Hq, d], dense) and of k (into the cache at slots[t]); v is copied.
 * The angle is exact to 2^-25 turns up to position 2^24, values are rounded once
 * to bf16.  q, k and v bf16 with rows ldq, ldk and ldv elements apart, as in
 * gocr_op_attention_packed; pos and slots int32[T] (device).  A row whose slot
 * is outside 0..n_pages*page_size-1 is skipped: whatever it holds, nothing is
 * written for it, and its q_out row is left as it was.  The slots of a call are distinct (of two rows with
 * one slot, parts of either may be left).  Hq <= 1024, Hq % Hkv == 0, d 64 or
 * 128, T <= 2^24, 1 <= theta <= 1e30. */
int gocr_op_kv_write_paged(const void* q, const void* k, const void* v, const int32_t* pos, const int32_t* slots,
                           void* q_out, const gocr_paged_kv* kv, int T, int Hq, long long ldq, long long ldk,
                           long long ldv, float theta, void* stream);

/* Attention of each request's new rows over its pages, the new rows' keys
 * among them: request r's rows are q rows cu_rows[r]..cu_rows[r+1]-1 (device
 * int32[n_req+1], non-decreasing, within 0..T), n of them; row i is at position
 * p_i = kv_len[r] - n + i and reads keys 0..p_i: single tokens, verify windows,
 * prompts prefilled whole or in chunks.  With kind GOCR_FWD_DRAFT the rows of a
 * request are a draft window: its first row reads keys 0..p_0 and the others
 * keys 0..kv_len[r]-1 (for GOCR_FWD_AR and GOCR_FWD_VERIFY: as above).  o[T, Hq, d]
 * bf16 = softmax(scale q k^T) v and lse[Hq, T] fp32 = log of the row's sum of
 * exponentials; o = 0 and lse = -infinity for a row without a key (p_i < 0).
 * q [T, Hq, d] with rows ldq elements apart; q head h reads kv head h / (Hq /
 * Hkv).  Rows that belong to no request are left as they were.  Keys behind
 * kv_len, of other requests and of other pages reach nothing, whatever they
 * hold; within a request a non-finite v may reach rows before it, too, that
 * are of the same call.  kv_len above max_pages * page_size is taken for that;
 * table entries outside 0..n_pages-1 read as pages of zeros.  Hq / Hkv <= 64, Hq <=
 * 1024, d 64 or 128, T <= 2^24, T Hq <= 2^31 - 1, pitch and scale as in
 * gocr_op_attention_packed; (T / (2 floor(128 Hkv / Hq)) + n_req) Hkv
 * (max_pages page_size / 128 + 5) <= 2^29; page and head strides of a cache such
 * that its extent has fewer than 2^31 of their greatest common divisor.
 * Scores, softmax statistics, sums and the parts of a split key axis are in
 * fp32; exp(scale q k^T - m), with m within 2^8 of the maximum so far, is
 * rounded to bf16 for the product with v.  The keys of all requests are cut into
 * equal pieces, so a row's last bits depend on the lengths of all requests of the
 * call (on nothing that the others hold; the same call gives the same bits): the row of
 * a verify window need not equal that of a single token bit for bit, as the rows of
 * the decoder's own forwards do.  The workspace takes up to 304 (2 floor(128
 * Hkv / Hq) Hq / Hkv) (4 d + 8) bytes, 40 MB with heads of 128, and less for
 * fewer rows. */
size_t gocr_op_attention_paged_workspace(int T, int Hq, int Hkv, int d);
int gocr_op_attention_paged(const void* q, const gocr_paged_kv* kv, const int32_t* table, int max_pages,
                            const int32_t* cu_rows, const int32_t* kv_len, int kind, void* o, float* lse, int n_req,
                            int T, int Hq, long long ldq, float scale, void* workspace, size_t workspace_bytes,
                            void* stream);

/* Waits for `stream` and reports whether a kernel of these operators on the
 * current device gave up a wait (they do after two seconds) since the calling
 * thread last asked, or, at its first question, since the library was loaded:
 * GOCR_EDEVICE; the outputs of such a call are not valid, and no other call
 * reports it.  The kernels count, and nothing is cleared, so threads take no
 * report from one another; which stream's kernel it was is not recorded.
 * GOCR_EINVAL while `stream` is being captured. */
int gocr_op_status(void* stream);

/* For tests of a program's handling of gocr_op_status: one warp that waits for
 * something that does not come, gives up after so many microseconds (1 to
 * 1,000,000) and reports it as the operators' kernels do. */
int gocr_op_wait_probe(int microseconds, void* stream);

/* ---- allocation-free GEMM ------------------------------------------------ */

/* Bytes of the device scratch array behind gocr_op_linear_static (per GPU). */
#define GOCR_STATIC_SCRATCH_BYTES (16u << 20)

/* gocr_op_linear for callers that cannot allocate device memory: a plug-in
 * whose host application owns every allocation, a real-time loop that may not
 * enter the allocator, a sandbox that forbids cudaMalloc.  Same arguments,
 * layouts and results as gocr_op_linear, but no workspace: the split-K partial
 * sums and tile counters live in one file-scope device array of
 * GOCR_STATIC_SCRATCH_BYTES that every GPU loading this library keeps until
 * the process exits.  GravityOCR has no counterpart: this is a deployment
 * convenience of this library.
 *   - Calls nothing that allocates (no cudaMalloc/cudaFree, no library
 *     allocator): it clears the counters with cudaMemsetAsync and launches.
 *   - GOCR_ECAPACITY when gocr_op_linear_workspace(T, N, K) exceeds
 *     GOCR_STATIC_SCRATCH_BYTES (message in gocr_last_error(NULL)).
 *   - The first call on a device looks up the array's device address with
 *     that device current and caches it; make that first call before any
 *     stream capture.  Under lazy module loading (the CUDA default) that
 *     first call is also where the driver reserves the array on the device,
 *     and it fails with GOCR_ECUDA if the device has no room for it; from
 *     the second call on, nothing is reserved.
 *   - `stream` must belong to the current device (GOCR_EINVAL otherwise).
 *   - All calls on a device share the array and it keeps the last call's
 *     contents: calls that overlap on the GPU (other streams, other threads)
 *     race; order them on one stream. */
int gocr_op_linear_static(int dtype, const void* x, const void* w, float* y, int T, int N, int K,
                          void* stream);

#ifdef __cplusplus
}
#endif
#endif /* GOCR_H */
