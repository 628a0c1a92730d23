/*
 * fm.h -- C ABI of libfm.so, a GB300 (sm_103a) implementation of the forward
 * pass of a block-parallel speculative-decoding drafter of the FlashMap /
 * DFlash kind.  One process, one GPU; every compute step runs in the
 * library's own CUDA kernels.
 *
 * Sources (page title, file, section):
 *   [FM]  diskformer 0.5.4 -> 0.6.6, package/engines/flashmap_drafter.js
 *   [MTP] diskformer 0.5.3 -> 0.6.4, package/engines/ternary_bonsai_2_mtp.js
 *   [DF]  mlx-bun 0.4.0 -> 1.0.0, package/src/spec/dspark/module-dflash.ts
 *
 * Conventions
 *   - Pointers named *_dev are device pointers; *_host are host pointers.
 *     "stream" is a cudaStream_t passed as void* (NULL = legacy stream).
 *   - Every call checks its arguments on the host before it launches anything
 *     and returns an fm_status; nothing aborts and no C++ exception crosses the
 *     ABI.  On failure fm_last_error(h) holds a one-line reason.
 *   - All device work is ordered on the given stream; no call synchronises the
 *     host except fm_debug_copy (it copies to host memory), fm_synchronize and
 *     fm_create.
 *   - A handle is not thread-safe: one host thread at a time per handle.
 */
#ifndef FM_H_
#define FM_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define FM_ABI_VERSION 1

/* exported from libfm.so; everything else in the library is hidden */
#if defined(__GNUC__)
#define FM_API __attribute__((visibility("default")))
#else
#define FM_API
#endif

typedef enum fm_status {
  FM_OK = 0,
  FM_ERR_INVALID_ARG = 1,   /* a null/misaligned pointer, a size or index out of range, a bad tensor */
  FM_ERR_UNSUPPORTED = 2,   /* a configuration the kernels do not handle (see fm_config) */
  FM_ERR_OOM = 3,           /* a device or pinned-host allocation failed */
  FM_ERR_CONTEXT_FULL = 4,  /* start + n_rows + block + 1 > max_ctx ([FM] extendContext's check) */
  FM_ERR_STATE = 5,         /* the call does not fit the sequence state (pos != length, start > length) */
  FM_ERR_CUDA = 6,          /* a CUDA runtime error; fm_last_error has the CUDA message */
  FM_ERR_TIMEOUT = 7        /* a bounded device-side wait gave up (reported, never hung) */
} fm_status;

/* fm_config.variant */
#define FM_VARIANT_FLASHMAP 0 /* adaLN DiT drafter with context injection [FM] */
#define FM_VARIANT_DFLASH 1   /* KV-injection drafter, Eq 2 / Eq 3 [DF] */

/* fm_config.lm_format: storage of the tied token table E [vocab][target_dim] */
#define FM_LM_BF16 0
#define FM_LM_Q8_0 1 /* GGUF Q8_0: per 32 values a little-endian f16 scale then 32 int8 (34 bytes) [MTP] */

/* fm_tensor.dtype */
#define FM_DTYPE_BF16 0
#define FM_DTYPE_Q8_0 1
#define FM_DTYPE_F32 2
#define FM_DTYPE_F16 3  /* rows of the 4-bit cache's calls */

typedef struct fm_config {
  int32_t variant;     /* FM_VARIANT_* */
  int32_t dim;         /* draft width D (multiple of 128) */
  int32_t n_heads;     /* D = n_heads * head_dim */
  int32_t head_dim;    /* 64 or 128 */
  int32_t n_layers;    /* DiT / backbone layers (1..64) */
  int32_t ff_dim;      /* MLP width (multiple of 128) */
  int32_t block;       /* draft slots: 16 for [FM], gamma for [DF]; 1..16 */
  int32_t target_dim;  /* the target's hidden width Ht (multiple of 64) */
  int32_t n_taps;      /* tapped target layers; feature rows are n_taps * target_dim wide */
  int32_t vocab;       /* rows of the token table */
  int32_t lm_format;   /* FM_LM_* */
  int32_t max_ctx;     /* cache rows per sequence (positions 0 .. max_ctx-1) */
  int32_t max_seqs;    /* independent sequences the handle holds caches for (>= 1) */
  float rope_theta;    /* RoPE base ([FM] CFG.theta) */
  float ln_eps;        /* adaLN LayerNorm eps ([FM] CFG.lnEps) */
  float rms_eps;       /* RMSNorm eps ([FM] CFG.rmsEps; [DF] the target's eps) */
  float qk_eps;        /* per-head q/k RMSNorm eps ([FM] CFG.qkEps) */
} fm_config;

/*
 * One named weight.  Names, shapes and layouts ([out][in] for [FM], [in][out]
 * for [DF]) are those of the drafter checkpoints:
 *   [FM]: fc.weight, hidden_norm.weight, anchor_proj.{weight,bias},
 *         anchor_norm.weight, state_norm.weight, x_embed.{weight,bias},
 *         layers.{l}.{self_attn,cross_attn}.{q,k,v,o}_proj.weight,
 *         layers.{l}.{self_attn,cross_attn}.{q,k}_norm.weight,
 *         layers.{l}.mlp.fc{1,2}.{weight,bias}, head.{weight,bias},
 *         token_embd.weight (the tied table; FM_DTYPE_Q8_0 or FM_DTYPE_BF16).
 *         A missing bias is read as zero.
 *   [DF]: bb.{i}.{attn_norm,q,k,v,o,ff_norm,gate,up,down}, W_c, ctx_norm,
 *         tok_proj, mask_emb, block_pos, out_norm, out_proj, token_embd.weight.
 * data is host memory (on_device = 0) or device memory (on_device = 1); the
 * library copies (and repacks) every tensor during fm_create, so the caller may
 * free it when fm_create returns.  nbytes must equal the tensor's size.
 */
typedef struct fm_tensor {
  const char *name;
  const void *data;
  int64_t nbytes;
  int32_t dtype;      /* FM_DTYPE_* */
  int32_t on_device;  /* 0 host, 1 device */
} fm_tensor;

typedef struct fm_handle fm_handle;

/*
 * fm_create -- take the configuration and the weights, build the device state
 * ([FM] FlashMapDrafter.load / upload / init; [DF] DflashDrafter.load).
 *   modulation_host: [FM] the adaLN table [(3*n_layers+1) * 3 * dim] f32 in
 *     blocks [scale dim | shift dim | gate dim] for (self, cross, mlp) of every
 *     layer and the final norm ([FM] timeConditioning output, e.g. from
 *     fm_time_conditioning); host or device memory; NULL for [DF].
 *   On success *out owns: the repacked weights, per-sequence caches of max_ctx
 *   rows, work buffers, and the constant start row h0 = x_embed(state_norm(
 *   mean row of E)) ([FM] init).  Synchronises the stream before returning.
 * Errors: FM_ERR_INVALID_ARG (null pointer, unknown/missing/mis-sized tensor,
 *   wrong dtype), FM_ERR_UNSUPPORTED (dims outside the limits above), FM_ERR_OOM,
 *   FM_ERR_CUDA.  *out is NULL on failure.
 */
FM_API fm_status fm_create(const fm_config *cfg, const fm_tensor *weights, int32_t n_weights,
                    const float *modulation_host, void *stream, fm_handle **out);

/*
 * fm_time_conditioning -- the adaLN table fm_create takes for [FM], computed
 * from the checkpoint's time-conditioning linears for the jump s -> t of the
 * flow map ([FM] timeConditioning; the page drafts with s = 0, t = 1):
 *   e(x) = [cos a_i | sin a_i], a_i = x * time_scale * exp(-ln(10000) i / half),
 *   half = time_dim / 2 ([FM] CFG.timeDim, CFG.timeScale);
 *   ts = time_embed.linear_2(SiLU(time_embed.linear_1(e(s)))), tj likewise with
 *   jump_embed and e(t); cond = SiLU(ts + tj), SiLU(x) = x / (1 + exp(-x));
 *   block n of the table = adaLN linear n of cond, n over
 *   layers.{l}.{self_attn_adaln,cross_attn_adaln,mlp_adaln}.linear then
 *   final_adaln.linear, each [scale dim | shift dim | gate dim].
 * weights: bf16 tensors (host or device) time_embed.linear_{1,2}.{weight,bias},
 *   jump_embed.linear_{1,2}.{weight,bias} (linear_1 [cond_dim][time_dim],
 *   linear_2 [cond_dim][cond_dim]) and every adaLN linear .weight
 *   [3 dim][cond_dim] / .bias [3 dim]; a missing bias is read as zero.  Other
 *   tensors in the list are ignored, so the full checkpoint list may be passed.
 * table_dev: device f32 [(3 n_layers + 1) * 3 * dim], caller-owned; pass it to
 *   fm_create as the modulation table (device memory is accepted there).
 * Set-up: allocates temporary device buffers and synchronises the stream.
 * Errors: FM_ERR_INVALID_ARG (null or misaligned pointer, odd time_dim,
 *   missing / mis-sized tensor, not [FM]), FM_ERR_OOM, FM_ERR_CUDA; the reason
 *   is in fm_last_error(NULL).
 */
FM_API fm_status fm_time_conditioning(const fm_config *cfg, const fm_tensor *weights, int32_t n_weights,
                                      int32_t time_dim, int32_t cond_dim, float time_scale, float s, float t,
                                      float *table_dev, void *stream);

/*
 * fm_context_append -- context injection ([FM] extendContext; [DF] Eq 2 and
 * projectContextRows): the target's tapped feature rows feats_dev
 * [n_rows][n_taps * target_dim] f32 (device, row-major, 16-byte aligned)
 * become cache rows start_pos .. start_pos + n_rows - 1 of sequence seq.
 *   [FM]: c = fc(f); cn = RMSNorm(c; hidden_norm); per layer k = RoPE(k_norm(
 *         k_proj cn)) at the row's position, v = v_proj cn; stored as f16.
 *   [DF]: H = RMSNorm(f W_c; ctx_norm); per layer K = attn_norm(H) W_k,
 *         V = attn_norm(H) W_v; stored as f16.
 * start_pos <= length is required; writing below the length rewinds (the
 * verify step re-appends from the anchor slot).  Afterwards length =
 * start_pos + n_rows.  n_rows may be 0 (only moves the length).
 * Errors: FM_ERR_INVALID_ARG (seq out of range, n_rows < 0, null feats with
 *   n_rows > 0), FM_ERR_STATE (start_pos > length or < 0),
 *   FM_ERR_CONTEXT_FULL (start_pos + n_rows + block + 1 > max_ctx), FM_ERR_CUDA.
 */
FM_API fm_status fm_context_append(fm_handle *h, int32_t seq, const float *feats_dev, int32_t n_rows,
                            int32_t start_pos, void *stream);

/*
 * fm_context_append_batched -- fm_context_append for several sequences in one
 * call.  Dense appends (>= 128 rows) run one after another through the
 * tensor-core prefill.  The shorter appends of 4 or more sequences, on a
 * FlashMap handle with max_seqs >= 2 and head_dim 128, share each weight
 * read: all their rows go through one fc GEMM and one K/V GEMM (per-row
 * sequence and position), in chunks of at most 16384 rows; otherwise each
 * runs on its sequence's own stream, concurrently (each reading the weights
 * itself).  feats_dev holds the rows of seq_ids[0], then seq_ids[1], ...;
 * n_rows_host[i] and start_host[i] are per sequence (host arrays of n_seqs).
 * Same checks per sequence; nothing is launched if any check fails.
 * Sequence ids must be distinct.  Batched calls on one handle run in stream
 * order on one stream (they share the handle's batched-pass buffers).
 */
FM_API fm_status fm_context_append_batched(fm_handle *h, int32_t n_seqs, const int32_t *seq_ids_host,
                                    const float *feats_dev, const int32_t *n_rows_host,
                                    const int32_t *start_host, void *stream);

/*
 * fm_draft -- draft `block` tokens after each anchor ([FM] draft; [DF]
 * forwardRows with the greedy argmax).  For sequence seq_ids[i] the anchor
 * token anchors[i] sits at position pos[i], which must equal that sequence's
 * length.  [FM] writes the anchor's own context slot (cache row pos) as the
 * page does; the length is unchanged (a later append from pos overwrites it).
 * tokens_dev: device int32 [n_seqs][block], written in stream order.
 * Host arrays: seq_ids, anchors, pos (n_seqs each; distinct seq ids).
 * Four or more sequences on a FlashMap handle with max_seqs >= 2 and
 * head_dim 128 draft together, in passes of up to 32: each pass runs every
 * product over all the pass's slot rows as one tensor-core GEMM (f16
 * operands), so each weight and the token table are read once per pass, and
 * one attention launch per layer serves every sequence's cache.  Fewer
 * sequences, or other handles, run one chain per sequence on the sequences'
 * own streams.
 * Errors: FM_ERR_INVALID_ARG (anchor outside [0, vocab), bad seq id, n_seqs
 *   outside [1, max_seqs], null tokens), FM_ERR_STATE (pos != length),
 *   FM_ERR_CONTEXT_FULL (pos + block + 1 > max_ctx), FM_ERR_CUDA.
 */
FM_API fm_status fm_draft(fm_handle *h, int32_t n_seqs, const int32_t *seq_ids_host, const int32_t *anchors_host,
                   const int32_t *pos_host, int32_t *tokens_dev, void *stream);

/*
 * Host-buffer forms of the three calls above, for callers whose feature rows
 * arrive in, and whose drafted tokens go to, host memory.  Each copies on the
 * stream with cudaMemcpyAsync: the rows into a handle-owned device staging
 * buffer (grown when a call needs more; it waits for the previous
 * host-buffer call's work before it is reused), then runs the device-pointer
 * call, whose checks, behaviour and errors it shares; fm_draft_host then
 * copies the tokens back.  With pinned host memory every copy is
 * asynchronous to the host: the rows must stay unchanged, and tokens_host
 * must not be read, until the stream has passed the call (fm_synchronize).
 * With pageable memory the runtime makes the copies synchronous instead.
 *   feats_host: host f32 rows laid out as in the device-pointer call (no
 *     alignment requirement).
 *   tokens_host: host int32 [n_seqs][block].
 * Errors: those of the device-pointer call; FM_ERR_INVALID_ARG (null
 *   feats_host with rows, null tokens_host); FM_ERR_OOM (the staging buffer
 *   could not grow); FM_ERR_CUDA (a copy failed).
 */
FM_API fm_status fm_context_append_host(fm_handle *h, int32_t seq, const float *feats_host, int32_t n_rows,
                                        int32_t start_pos, void *stream);
FM_API fm_status fm_context_append_batched_host(fm_handle *h, int32_t n_seqs, const int32_t *seq_ids_host,
                                                const float *feats_host, const int32_t *n_rows_host,
                                                const int32_t *start_host, void *stream);
FM_API fm_status fm_draft_host(fm_handle *h, int32_t n_seqs, const int32_t *seq_ids_host,
                               const int32_t *anchors_host, const int32_t *pos_host, int32_t *tokens_host,
                               void *stream);

/*
 * fm_draft_pruned -- [DF] the greedy draft of one sequence through the
 * sequential logit head, with the confidence head and confidence pruning
 * (module-dflash.ts: ``#markov`` (Eq 5), ``#rnn`` (Eq 6), ``#confidence`` and
 * the pruning of Alg 1 in ``forwardRows``).  Needs weights that hold
 * markov.w1 [V][r] (r <= 512, vocab % 8 == 0) and markov.w2 [r][V], or the RNN
 * head (rnn.wH [r][r], rnn.bH [r], rnn.wO [r][V]); conf.w [dim + r] and
 * conf.b [1] for conf_dev and any threshold.  With such weights fm_draft also
 * drafts through the sequential head (no pruning).
 * Position k (prev = anchor for k = 0, else token k - 1; e1 = markov.w1[prev]):
 *   Markov bias = e1 markov.w2; RNN s_k = tanh(s_{k-1} rnn.wH + e1 + rnn.bH),
 *   s_{-1} = 0, bias = s_k rnn.wO;  token_k = argmax(base logits_k + bias),
 *   ties to the lower index;  conf_k = sigmoid([out_norm(row k), e1] conf.w
 *   + conf.b).
 * Pruning: the threshold of position k is thresholds_host[k] (host float
 * [block], or NULL) unless that is NaN, else min_conf (NaN: none), as the
 * page's per-position lookup falls back to its uniform override.  The block ends at the
 * first k >= 1 with conf_k below its threshold (length = k).  Entries
 * 0 .. min(length, block - 1) of tokens_dev and conf_dev are written (the
 * cut position's own, whose confidence decided the cut, included); later
 * positions are not drafted and their entries are left as they were.
 * tokens_dev: device int32 [block]; conf_dev: device float [block] or NULL;
 * length_dev: device int32 [1] or NULL, the positions kept (block without
 * pruning).  All written in stream order.  Same argument checks as fm_draft;
 * FM_ERR_UNSUPPORTED without a sequential head, or without a confidence head
 * when conf_dev or a threshold is given.
 */
FM_API fm_status fm_draft_pruned(fm_handle *h, int32_t seq, int32_t anchor, int32_t pos,
                                 const float *thresholds_host, float min_conf, int32_t *tokens_dev,
                                 float *conf_dev, int32_t *length_dev, void *stream);

/*
 * fm_accept -- greedy acceptance ([FM] specGenerate verify step; [MTP] the
 * same rule): n_accepted = the longest prefix i < k with draft[i] == target[i];
 * bonus = target[n_accepted].  draft_host has k entries, target_host k + 1.
 * Pure host function.  Errors: FM_ERR_INVALID_ARG (null pointer, k < 0).
 */
FM_API fm_status fm_accept(const int32_t *draft_host, const int32_t *target_host, int32_t k, int32_t *n_accepted,
                    int32_t *bonus);

/*
 * fm_accept_batched -- fm_accept for n_seqs sequences on the device:
 * draft_dev [n_seqs][block], target_dev [n_seqs][block + 1], k_dev [n_seqs]
 * (each clamped to [0, block]); writes n_accepted_dev[n_seqs], bonus_dev[n_seqs].
 * Errors: FM_ERR_INVALID_ARG (null pointer, n_seqs < 1), FM_ERR_CUDA.
 */
FM_API fm_status fm_accept_batched(fm_handle *h, int32_t n_seqs, const int32_t *draft_dev, const int32_t *target_dev,
                            const int32_t *k_dev, int32_t *n_accepted_dev, int32_t *bonus_dev, void *stream);

/*
 * fm_lm_head_argmax_noalloc -- fm_draft's fused lm_head + per-row argmax on
 * rows the caller supplies: tokens[t] = argmax_v sum_k y[t][k] E[v][k]
 * (ties -> lowest v) over the handle's token table E.  The paper has no
 * counterpart to this entry point.  It is for callers that may not allocate
 * device memory while they run -- a serving loop whose memory is all handed
 * out up front by its own pool, or code running where cudaMalloc would stall
 * the device or could fail under memory pressure.  It allocates nothing: the
 * cross-CTA partial bests and the completion ticket live in a fixed 64 KB
 * block of static device memory inside the library, which every GPU that
 * loads the library keeps until the process exits.  That block holds at
 * most 255 CTAs of partials; larger grids are rejected with
 * FM_ERR_UNSUPPORTED.  The first call on a device looks up the block's
 * address and zeroes the ticket on the stream, so make that first call
 * before any stream capture.  Every call shares the block: calls that
 * overlap on the GPU (other streams, other handles on the same device) race
 * and must be serialised by the caller.
 * y_dev: device f32 [n_rows][target_dim], row-major, 16-byte aligned.
 * tokens_dev: device int32 [n_rows], 4-byte aligned, written in stream
 * order.  Both stay owned by the caller.  The handle's device must be the
 * current device.
 * Errors: FM_ERR_INVALID_ARG (null or misaligned pointer, n_rows outside
 *   1..16, the current device is not the handle's), FM_ERR_UNSUPPORTED (grid
 *   beyond the static block), FM_ERR_CUDA.  A device-side bounded wait that
 *   gives up inside the kernel is reported late: the call has already
 *   returned FM_OK, tokens_dev is then undefined, and the next
 *   fm_synchronize (or fm_debug_copy) on the handle returns FM_ERR_TIMEOUT.
 */
FM_API fm_status fm_lm_head_argmax_noalloc(fm_handle *h, const float *y_dev, int32_t n_rows, int32_t *tokens_dev,
                                    void *stream);

/*
 * fm_synchronize -- wait for the work on stream, then report whether a
 * device-side bounded wait gave up in any call since the last check (a wait
 * that exceeds its clock budget raises an error word on the device and its
 * kernel returns instead of hanging).  Clears the word.
 * Errors: FM_ERR_TIMEOUT (a wait gave up: the outputs of those calls are
 *   undefined; the handle stays usable), FM_ERR_CUDA, FM_ERR_INVALID_ARG.
 */
FM_API fm_status fm_synchronize(fm_handle *h, void *stream);

/*
 * fm_selftest_wait_timeout -- exercise the failure path of the bounded waits:
 * launches one CTA whose mbarrier wait can never complete, with a budget of
 * budget_us microseconds (1 .. 1e6); the wait gives up, raises the handle's
 * device error word and the kernel returns.  A following fm_synchronize
 * returns FM_ERR_TIMEOUT.  Nothing hangs and nothing faults.
 * Errors: FM_ERR_INVALID_ARG (budget out of range), FM_ERR_CUDA.
 */
FM_API fm_status fm_selftest_wait_timeout(fm_handle *h, int32_t budget_us, void *stream);

/*
 * The verify-length and fallback policy of the speculative loop ([FM]
 * specGenerate): a caller-owned record and four host functions, no device
 * work.  Per step of the loop fm_policy_next says whether to run a draft round
 * verifying k drafts (FM_ACT_ROUND), a step of a plain-decoding stretch
 * (FM_ACT_PLAIN: report it with fm_policy_after_plain), or a plain step at the
 * drafter's context limit (FM_ACT_PLAIN_LIMIT: position + 2 block + 2 >
 * max_ctx; no statistics).  After a round, fm_policy_after_round takes the
 * accepted count and the round's time.
 *   k: adaptive (verify = 0): block when the acceptance average >= 5, else 7;
 *      fixed: min(block, verify).
 *   averages: acceptance 0.6 / 0.4 (starts at 4), tokens per round
 *      0.75 / 0.25 of accepted + 1 (starts at 5), round time 0.6 / 0.4 (the
 *      first round after a stretch whose rows were handed to the drafter is left
 *      out), plain-step time 0.7 / 0.3 (starts at 30 ms).
 *   fallback: from the fourth round on, when tokens per round x plain-step time
 *      < 0.85 x round time, a plain stretch of probe_every steps starts (then
 *      one round probes again).
 * Errors: FM_ERR_INVALID_ARG (null pointer, block < 1, verify < 0,
 *   probe_every < 1, accepted < 0, a plain report outside a stretch).
 */
typedef struct fm_verify_policy {
  int32_t block, verify, fallback, probe_every;
  double ema;          /* acceptance average */
  double ema_tokens;   /* tokens-per-round average */
  double round_ms;     /* round-time average, < 0 until the first round */
  double step_ms;      /* plain-step time average */
  int32_t plain_left;  /* steps left in the current plain stretch */
  int32_t rounds;      /* rounds so far */
  int32_t catch_up;    /* the next round's time is left out of the average */
  int32_t pad;
} fm_verify_policy;
#define FM_ACT_ROUND 0
#define FM_ACT_PLAIN 1
#define FM_ACT_PLAIN_LIMIT 2
FM_API fm_status fm_policy_init(fm_verify_policy *p, int32_t block, int32_t verify, int32_t fallback,
                                int32_t probe_every);
FM_API fm_status fm_policy_next(const fm_verify_policy *p, int32_t position, int32_t max_ctx, int32_t *action,
                                int32_t *k);
FM_API fm_status fm_policy_after_round(fm_verify_policy *p, int32_t accepted, double ms);
FM_API fm_status fm_policy_after_plain(fm_verify_policy *p, double ms, int32_t rows_handed);

/* fm_debug_copy selectors ([FM] readOut / peek: look at working buffers) */
#define FM_DEBUG_HIDDEN 0   /* index = layer: the block's hidden rows after that layer [block][dim] f32 (last draft) */
#define FM_DEBUG_HEAD_OUT 1 /* the head output Y [block][target_dim] f32 (last draft of seq) */
#define FM_DEBUG_LOGITS 2   /* logits [block][vocab] f32 of the last draft's Y, recomputed without argmax */
#define FM_DEBUG_CACHE_K 3  /* index = layer: cache K of seq, [n_heads][max_ctx][head_dim] as f16 bits */
#define FM_DEBUG_CACHE_V 4  /* index = layer: cache V, same layout */
#define FM_DEBUG_H0 5       /* [FM] the constant start row h0 [dim] f32 */
#define FM_DEBUG_STEP_TRACE 6 /* [FM] persistent step trace of the last traced draft: u64 [phases][CTAs][8]
                                 (CTAs = the step's clusters x 8) globaltimer ns: 0 phase start, 1 staged,
                                 2 done, 3 last copy issued, 4 last MMA committed, 5 partials published,
                                 6 epilogues done; 0 = no event */

/*
 * fm_debug_copy -- copy nbytes of the selected buffer, starting at byte
 * offset, to dst_host.  Synchronises the stream.  After a batched draft,
 * FM_DEBUG_HEAD_OUT and FM_DEBUG_LOGITS read the sequence's rows of the last
 * pass of the last batched call (the logits recomputed by the batched
 * lm_head's product); a sequence of an earlier pass, or of an earlier batched
 * call, has no kept head output until its next draft (FM_ERR_UNSUPPORTED).
 * FM_DEBUG_HIDDEN is kept by single-sequence drafts only.
 * Errors: FM_ERR_INVALID_ARG (unknown selector, index or range outside the
 * buffer), FM_ERR_UNSUPPORTED (above), FM_ERR_CUDA, FM_ERR_TIMEOUT (a bounded
 * wait gave up in an earlier call).
 */
FM_API fm_status fm_debug_copy(fm_handle *h, int32_t what, int32_t seq, int32_t index, int64_t offset, void *dst_host,
                        int64_t nbytes, void *stream);

/* fm_set_debug flags */
#define FM_DEBUG_KEEP_HIDDEN 1 /* keep every layer's block hidden rows for FM_DEBUG_HIDDEN (adds copies) */
#define FM_DEBUG_PROFILE 2     /* bracket every kernel launch with CUDA events (serialises the chain) */
#define FM_DEBUG_TRACE 4       /* record per-phase timestamps of the persistent draft step (FM_DEBUG_STEP_TRACE) */

/* Debug switches for later calls (0 = the plain hot path).  Errors: FM_ERR_INVALID_ARG. */
FM_API fm_status fm_set_debug(fm_handle *h, int32_t flags);

/* Per-kernel timings gathered while FM_DEBUG_PROFILE is set: one entry per
 * kernel name, with the launches, their summed device time and the summed
 * algorithmic bytes they move (weights once, activations once); for the
 * tensor-core GEMMs (names containing "gemm") the field holds their summed
 * floating-point operations instead (2 M N K each).  Reading synchronises the
 * stream of the recorded launches and resets the record.
 * Errors: FM_ERR_INVALID_ARG (null pointers, cap < 0), FM_ERR_CUDA. */
typedef struct fm_kernel_time {
  char name[32];
  int32_t launches;
  float ms;
  double bytes;
} fm_kernel_time;
FM_API fm_status fm_profile_read(fm_handle *h, fm_kernel_time *out, int32_t cap, int32_t *n);

/* Current context length of a sequence.  Errors: FM_ERR_INVALID_ARG. */
FM_API fm_status fm_get_length(const fm_handle *h, int32_t seq, int32_t *length);

/* Device bytes the handle holds ([FM] gpuBytes). */
FM_API fm_status fm_memory_bytes(const fm_handle *h, int64_t *bytes);

/* Kernel launches issued by the last fm_context_append / fm_draft / batched call. */
FM_API fm_status fm_last_launch_count(const fm_handle *h, int32_t *count);

FM_API const char *fm_status_str(fm_status s);
FM_API const char *fm_last_error(const fm_handle *h);   /* never NULL; "" when no error; NULL h: the last failed
                                                            fm_create / fm_time_conditioning on this thread */

/* Free everything the handle owns.  NULL is ignored. */
FM_API void fm_destroy(fm_handle *h);

/* ------------------------------------------------------------------------
 * The MTP draft head ([MTP] ternary_bonsai_2_mtp.js: the header's graph,
 * MCFG, MTPHead.forward and its kernels, MTPRunner's draft loop): one
 * Qwen-style decoder layer with Q8_0 weights, chained in depth.  A second
 * drafter, with its own handle.
 *
 * One pass over M <= max_rows rows (tokens x at positions pos0 .. pos0+M-1,
 * each with h, the normed hidden of its previous position):
 *   Xc = [rms(E[x]; enorm) | rms(h; hnorm)];  X = eh_proj Xc
 *   A = rms(X; attn_norm);  [q | gate] per q head = attn_q A;  k, v = attn_k A, attn_v A
 *   per head RMSNorm over head_dim (attn_q_norm / attn_k_norm), NEOX RoPE on the
 *   first rot_dims (pairs i, i + rot_dims/2, angle pos * theta^(-2i/rot_dims));
 *   k, v rows stored in the head's own f32 cache at their positions
 *   O = softmax(q k^T / sqrt(head_dim)) v over cache rows kv_lo .. pos (KV head
 *   h / (n_heads / n_kv_heads)), times sigmoid(gate)
 *   X += attn_output O;  X += ffn_down(silu(ffn_gate A') * ffn_up A'), A' = rms(X; post_attention_norm)
 *   h' = rms(X; shared_head_norm);  draft = argmax(lm_head h'), ties to the lower index
 * ------------------------------------------------------------------------ */
typedef struct fm_mtp_config {
  int32_t hidden;      /* H (MCFG.H 5120); a multiple of 128 */
  int32_t inter;       /* I (17408); a multiple of 128 */
  int32_t n_heads;     /* q heads (24) */
  int32_t n_kv_heads;  /* KV heads (4); divides n_heads */
  int32_t head_dim;    /* 256; a multiple of 32, <= 256 */
  int32_t rot_dims;    /* NEOX-rotated dims per head (64); even, <= head_dim */
  float theta;         /* RoPE base (1e7) */
  float eps;           /* RMSNorm eps (1e-6) */
  int32_t vocab;       /* lm_head rows (248320) */
  int32_t kv_cap;      /* cache rows (positions) the head keeps */
  int32_t max_rows;    /* M per pass, <= 8 (MCFG.MAXM) */
} fm_mtp_config;

typedef struct fm_mtp fm_mtp;

/*
 * fm_mtp_create -- load the head.  weights (host or device, copied):
 *   Q8_0 (GGUF rows [N][K/32 * 34]): eh_proj [H][2H], attn_q [n_heads*2*head_dim][H]
 *     (per head the query rows, then its gate rows), attn_k / attn_v
 *     [n_kv_heads*head_dim][H], attn_output [H][n_heads*head_dim], ffn_gate /
 *     ffn_up [I][H], ffn_down [H][I], lm_head [vocab][H];
 *   FM_DTYPE_F32: enorm, hnorm, attn_norm, post_attention_norm, shared_head_norm [H],
 *     attn_q_norm, attn_k_norm [head_dim];
 *   FM_DTYPE_BF16: token_embd [vocab][H] (the rows the drafted tokens are embedded with).
 * Every 2-D product's N must be a multiple of 128 and its K of 64.
 * Errors: FM_ERR_INVALID_ARG (null, missing / mis-sized tensor, wrong dtype),
 *   FM_ERR_UNSUPPORTED (dims outside the limits above), FM_ERR_OOM, FM_ERR_CUDA.
 *   *out is NULL on failure; the reason is in fm_mtp_last_error(NULL).
 */
FM_API fm_status fm_mtp_create(const fm_mtp_config *cfg, const fm_tensor *weights, int32_t n_weights, void *stream,
                               fm_mtp **out);

/*
 * fm_mtp_forward -- MTPHead.forward: one pass over n_rows rows.  tokens_dev:
 * device int32 [n_rows]; hn_dev: device f32 [n_rows][H] (the normed hidden of
 * each row's previous position); writes cache rows pos0 .. pos0+n_rows-1 and,
 * when hout_dev is not NULL, h' (device f32 [n_rows][H]).  Attention reads rows
 * kv_lo .. pos; rows below pos0 must have been written by earlier passes.
 * drafts_dev (device int32 [n_rows] or NULL) receives argmax(lm_head h') per row.
 * Errors: FM_ERR_INVALID_ARG (n_rows outside [1, max_rows], null tokens / hn,
 *   kv_lo outside [0, pos0], pos0 + n_rows > kv_cap), FM_ERR_CUDA.
 */
FM_API fm_status fm_mtp_forward(fm_mtp *m, int32_t n_rows, const int32_t *tokens_dev, const float *hn_dev,
                                int32_t pos0, int32_t kv_lo, float *hout_dev, int32_t *drafts_dev, void *stream);

/*
 * fm_mtp_draft -- MTPRunner's draft: a pass over the n_rows pending rows (as
 * fm_mtp_forward), the draft of its last row, then depth - 1 single-row passes
 * at pos0 + n_rows, ..., each on the previous draft (embedded on the device)
 * and the previous pass's last h'.  drafts_dev: device int32 [depth].  No host
 * round trip between the passes.  Errors: as fm_mtp_forward, and depth outside
 * [1, kv_cap - pos0 - n_rows + 1].
 */
FM_API fm_status fm_mtp_draft(fm_mtp *m, int32_t n_rows, const int32_t *tokens_dev, const float *hn_dev,
                              int32_t pos0, int32_t kv_lo, int32_t depth, int32_t *drafts_dev, void *stream);

/* Copy the head's K (which = 0) or V (which = 1) cache rows [0, rows) ([rows][n_kv_heads * head_dim] f32,
   host or device dst) after the stream's work (synchronises it); for tests.  Also reports what the device
   raised since the last check: FM_ERR_INVALID_ARG for a token outside [0, vocab) that reached the embedding
   (row 0 was read instead), FM_ERR_TIMEOUT for a bounded wait that gave up.  Errors: FM_ERR_INVALID_ARG,
   FM_ERR_CUDA. */
FM_API fm_status fm_mtp_cache(fm_mtp *m, int32_t which, int32_t rows, float *dst, void *stream);

/* Kernel launches issued by the last fm_mtp_forward / fm_mtp_draft. */
FM_API fm_status fm_mtp_last_launch_count(const fm_mtp *m, int32_t *count);
FM_API const char *fm_mtp_last_error(const fm_mtp *m);   /* never NULL; NULL m: the last failed fm_mtp_create */
FM_API void fm_mtp_destroy(fm_mtp *m);

/* ------------------------------------------------------------------------
 * A KV cache held in 4 bits: rows in (fm_kvq_append) and out (fm_kvq_read),
 * attention over it (fm_kvq_attend) that can keep count of the attention
 * weight each row collects, and eviction by that weight (fm_kvq_evict).  The
 * pages keep their caches in f16 and f32 and hold every row; this cache has no
 * counterpart there.  It stands by itself, or holds the MTP head's rows
 * (fm_mtp_use_kvq).
 *
 * A row of a KV head is cut into groups of 32 values; a group is held as an
 * f16 scale d and 32 codes c in 0 .. 15 (4.5 bits a value) and stands for
 * d (c - 8):  d = f16(m / -8), m the group's value of largest magnitude (the
 * negative one where +m and -m tie); c = clamp(rint(x / d) + 8, 0, 15), ties
 * to even, 8 where d = 0.  NaN is stored as 0; infinities and values beyond
 * 8 * 65504 saturate.
 *
 * Each (layer, sequence) has its own length, kept on the host by the calls.
 * Rows behind it are never read as values and left as they are.  Host arrays
 * (seq_ids, counts) have n_seqs entries, 1 <= n_seqs <= config.n_seqs.
 * Calls allocate nothing and may be captured into a graph, which then repeats
 * the call at the lengths it was captured with.  Eager calls on different
 * streams are put in the order they were issued in (they share a workspace
 * and the weights); a captured call is not, so graphs that use one cache are
 * replayed one after another, and ordered with eager calls, by the caller, and
 * not after fm_kvq_destroy.  The cache's device must be the current device.
 * Device pointers are 16-byte aligned, and row strides (ld, ldq, ldo: elements
 * between rows) whole multiples of 16 bytes; pointers to weights and kept rows are
 * 4-byte aligned (FM_ERR_INVALID_ARG otherwise).  One host thread at a time per
 * cache.
 * ------------------------------------------------------------------------ */
typedef struct fm_kvq_config {
  int32_t n_layers;    /* 1 .. 1024 */
  int32_t n_seqs;      /* sequences (slots) per layer: 1 .. 65536 */
  int32_t n_kv_heads;  /* 1 .. 256 */
  int32_t head_dim;    /* 64, 128 or 256 */
  int32_t max_rows;    /* rows per sequence and layer: 1 .. 2^24 */
} fm_kvq_config;

typedef struct fm_kvq fm_kvq;

/*
 * fm_kvq_create -- an empty cache on the current device.  Synchronises the
 * stream.  Errors: FM_ERR_INVALID_ARG, FM_ERR_UNSUPPORTED (head_dim),
 * FM_ERR_OOM, FM_ERR_CUDA; *out is NULL on failure and the reason is in
 * fm_kvq_last_error(NULL).
 */
FM_API fm_status fm_kvq_create(const fm_kvq_config *cfg, void *stream, fm_kvq **out);

/*
 * fm_kvq_append -- rows k_dev, v_dev [sum n_rows][n_kv_heads][head_dim] of
 * dtype FM_DTYPE_F32 / F16 / BF16, row stride ld, packed in the order of
 * seq_ids, become rows start .. start + n_rows - 1 of their sequence in layer.
 * start <= length; writing below the length rewinds.  Afterwards length =
 * start + n_rows (n_rows may be 0: only moves the length).  The new rows'
 * weights are 0.  Sequence ids are distinct.
 * Errors: FM_ERR_INVALID_ARG, FM_ERR_STATE (start > length or < 0),
 *   FM_ERR_CONTEXT_FULL (start + n_rows > max_rows), FM_ERR_CUDA; nothing is
 *   launched if a check fails.
 */
FM_API fm_status fm_kvq_append(fm_kvq *c, int32_t layer, int32_t n_seqs, const int32_t *seq_ids_host,
                               const int32_t *n_rows_host, const int32_t *start_host, const void *k_dev,
                               const void *v_dev, int32_t dtype, int64_t ld, void *stream);

/*
 * fm_kvq_read -- the values that rows row .. row + n_rows - 1 stand for,
 * rounded once to dtype, into k_dev and v_dev (laid out as in fm_kvq_append;
 * either may be NULL), and their weights into weights_dev (f32
 * [n_seqs][n_kv_heads][ldw], entry r = row + r's; or NULL).
 * Errors: FM_ERR_INVALID_ARG (rows outside the length, ...), FM_ERR_CUDA.
 */
FM_API fm_status fm_kvq_read(fm_kvq *c, int32_t layer, int32_t n_seqs, const int32_t *seq_ids_host,
                             const int32_t *row_host, const int32_t *n_rows_host, void *k_dev, void *v_dev,
                             int32_t dtype, int64_t ld, float *weights_dev, int64_t ldw, void *stream);

/*
 * fm_kvq_attend -- attention of n_rows[i] query rows (a draft block, a verify
 * step's rows, one token) of each sequence over its cache:
 *   out[r][h] = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q[r][h] . k_j),
 * head h reading KV head h / (n_heads / n_kv_heads), over the rows
 * first_row <= j < length, and with causal != 0 only j <= length - n_rows + t
 * for the sequence's row t (its n_rows rows are the cache's last).  A row that
 * sees nothing (length 0, first_row past the end, more query rows than cached
 * ones) gives zeros.  q_dev and out_dev: [sum n_rows][n_heads][head_dim] of
 * dtype, row strides ldq and ldo, packed in the order of seq_ids; they may not
 * overlap (out_dev == q_dev is refused).
 *
 * Scores, softmax and sums are f32.  The cache's values enter exactly as stored,
 * f32 queries to ~22 bits (f16 and bf16 ones as they are).  Products are summed
 * to f32's precision in f32 calls and in the scores of calls that count weights;
 * the other sums of f16 and bf16 calls keep ~2^-17 of their largest term, below
 * the outputs' own rounding (so the same queries may give other last bits with
 * weights than without).  A probability times its row's V scale is kept to ~21
 * bits for f32 outputs, rounded to f16's 11 once for f16 ones and twice for bf16
 * ones, and a key's part to 2^-24 of the largest |v| of its KV head that the call
 * sees.  Rows that the call does not see (behind the length, ahead of first_row,
 * overwritten or evicted) have no part in any of it.  A query row with a NaN or an infinity
 * gives NaN, and one with values past 2^97 may.
 *
 * decay >= 0 also counts the attention weight each cache row collects, per KV
 * head:  w_j = decay w_j + sum over the call's rows and the KV head's query
 * heads of p_j / sum p  (decay 1: plain accumulation; 0: this call's weights
 * alone), for the rows 0 .. length - 1 of every sequence with n_rows > 0, and
 * writes the new weights to weights_dev (f32 [n_seqs][n_kv_heads][ldw]) unless
 * that is NULL.  decay < 0: weights are left alone.
 * Sequence ids are distinct where weights are counted.
 * Errors: FM_ERR_INVALID_ARG (also: over 65,536 query rows of a sequence or over
 *   1,024 query heads a KV head), FM_ERR_UNSUPPORTED (a sequence's rows make
 *   units of 32 query rows x heads of a KV head: over 2^15 units, or over
 *   2^31 - 1 stages in them, a unit having one for each 128 cache rows from
 *   first_row on, or 64 with head_dim 256, and four more), FM_ERR_CUDA.  A bounded device wait that gives up is
 *   reported by fm_kvq_synchronize.
 */
FM_API fm_status fm_kvq_attend(fm_kvq *c, int32_t layer, int32_t n_seqs, const int32_t *seq_ids_host,
                               const int32_t *n_rows_host, const void *q_dev, int32_t dtype, int32_t n_heads,
                               int64_t ldq, float scale, int32_t causal, int32_t first_row, void *out_dev,
                               int64_t ldo, float decay, float *weights_dev, int64_t ldw, void *stream);

/* fm_kvq_set_weights -- the weights of rows 0 .. length - 1 from weights_dev (f32 [n_seqs][n_kv_heads][ldw]): a
   saved state, or a measure of the caller's own to evict by.  Sequence ids are distinct.  Errors:
   FM_ERR_INVALID_ARG, FM_ERR_CUDA. */
FM_API fm_status fm_kvq_set_weights(fm_kvq *c, int32_t layer, int32_t n_seqs, const int32_t *seq_ids_host,
                                    const float *weights_dev, int64_t ldw, void *stream);

/*
 * fm_kvq_evict -- bring sequences down to `keep` rows: per KV head the last
 * `recent` rows stay, and of the rows before them the keep - recent with the
 * largest weight (ties: the lowest row; NaN ranks below every number), in their
 * order.  The kept rows, with their weights, become rows 0 .. of sequence
 * dst_ids[i], whose length is then min(keep, length); a sequence of at most
 * keep rows keeps all.  dst_ids[i] may be src_ids[i] (in place), or another
 * sequence, whose rows are replaced and whose source stays as it is (a branch).  Destinations are distinct, and none
 * is the source of another entry.  kept_dev: int32 [n_seqs][n_kv_heads][keep]
 * or NULL receives the rows kept; entries past min(keep, length) are left as
 * they were.  0 <= recent <= keep <= max_rows.
 * After an eviction the heads of a sequence hold different rows of the past, in
 * one order: causal calls and first_row go by the place in the cache.
 * Errors: FM_ERR_INVALID_ARG, FM_ERR_CUDA.
 */
FM_API fm_status fm_kvq_evict(fm_kvq *c, int32_t layer, int32_t n_seqs, const int32_t *src_ids_host,
                              const int32_t *dst_ids_host, int32_t keep, int32_t recent, int32_t *kept_dev,
                              void *stream);

/* The rows a (layer, sequence) holds.  Errors: FM_ERR_INVALID_ARG. */
FM_API fm_status fm_kvq_length(const fm_kvq *c, int32_t layer, int32_t seq, int32_t *length);
/* The configuration the cache was made with.  Errors: FM_ERR_INVALID_ARG. */
FM_API fm_status fm_kvq_get_config(const fm_kvq *c, fm_kvq_config *cfg);
/* Kernel launches issued by the last call that completed. */
FM_API fm_status fm_kvq_last_launch_count(const fm_kvq *c, int32_t *count);
/* Device bytes the cache holds (rows, weights, workspace). */
FM_API fm_status fm_kvq_memory_bytes(const fm_kvq *c, int64_t *bytes);
/* Wait for the stream; FM_ERR_TIMEOUT if a bounded device wait gave up since the last check (cleared). */
FM_API fm_status fm_kvq_synchronize(fm_kvq *c, void *stream);
/* fm_selftest_wait_timeout for a cache: a bounded wait that gives up after budget_us (1 .. 1e6) raises the cache's error
   word, which the next fm_kvq_synchronize reports.  Errors: FM_ERR_INVALID_ARG, FM_ERR_CUDA. */
FM_API fm_status fm_kvq_selftest_wait_timeout(fm_kvq *c, int32_t budget_us, void *stream);
FM_API const char *fm_kvq_last_error(const fm_kvq *c);   /* never NULL; NULL c: the last failed fm_kvq_create */
/* Free everything the cache owns, once the calls issued so far are done.  NULL is ignored; a capture in progress goes on. */
FM_API void fm_kvq_destroy(fm_kvq *c);

/*
 * fm_mtp_use_kvq -- keep the MTP head's rows in (layer, seq) of the 4-bit cache
 * c from the next pass on (c NULL: in the head's own f32 cache again, which
 * holds what it held).  A pass stores its rows by fm_kvq_append and attends by
 * fm_kvq_attend; the rows a position may have are c's, not kv_cap's (kv_cap
 * may be 1 on a head that only ever uses c).  c has the head's n_kv_heads and
 * head_dim, stays the caller's and outlives its use.
 *   next_pos: the position after the cache's last row (the length, unless
 *     rows were evicted before).  A pass at pos0 <= next_pos rewinds
 *     next_pos - pos0 rows and appends its own.  Rows evicted between passes
 *     (fm_kvq_evict, in place) are the older ones as long as `recent` covers
 *     what a pass may rewind; kv_lo is then 0.
 *   decay: >= 0 counts the attention weights in every pass (fm_kvq_attend),
 *     for an eviction; < 0 does not.
 * Passes then also fail with FM_ERR_STATE (pos0 > next_pos, or a rewind past
 * the rows that are left), FM_ERR_CONTEXT_FULL (the rows do not fit c),
 * FM_ERR_INVALID_ARG (positions past 2^31 - 1, another current device) and
 * FM_ERR_UNSUPPORTED (kv_lo > 0 after an eviction); nothing is launched then.
 * fm_mtp_cache with rows > 0 answers FM_ERR_STATE; with rows = 0 it also reports
 * (and clears) a bounded wait of c's that gave up, as fm_kvq_synchronize does.
 * Errors: FM_ERR_INVALID_ARG (another device, other heads or head_dim, no such layer or
 *   sequence, next_pos below the length, decay not finite), FM_ERR_OOM.
 */
FM_API fm_status fm_mtp_use_kvq(fm_mtp *m, fm_kvq *c, int32_t layer, int32_t seq, int64_t next_pos, float decay);

/* ------------------------------------------------------------------------
 * A KV cache in pages: a batch's new rows are written to it with the per-head
 * norms and the position rotation in the same pass (fm_paged_write), and
 * attended over from there (fm_paged_attend), with or without a sliding window
 * and a few first rows that stay visible.  The pages keep one contiguous cache
 * a sequence; this one has no counterpart there.  It stands by itself, or holds
 * the MTP head's rows (fm_mtp_use_paged).
 *
 * The pool is the caller's: K and V apart, each
 * [n_layers][n_pages][n_kv_heads][page_rows][head_dim] of dtype, 16-byte
 * aligned, alive and in place as long as the handle is used.  What lies in it
 * is plain values, so pages may be shared, copied and handed round.
 *
 * A batch (fm_paged_batch) says which rows are new and where sequences lie.
 * Its numbers are on the device: a captured call reads them again at every
 * replay.  (A table's rows are at least table_pages entries apart, one sequence's
 * too.)  Sequence i's new rows are rows starts[i] .. starts[i + 1] - 1 of the
 * packed rows; lengths[i] rows are in the cache once they are written, the new
 * ones the last, so a new row t of n has position lengths[i] - n + t.  Row j of
 * the sequence is row j % page_rows of page table[i][j / page_rows].  Several
 * sequences may name one page to read from; a row that a call writes is named
 * once.  Packed rows behind starts[n_seqs] and rows that no call names are left
 * as they are.
 * A sequence whose starts or length point outside the packed rows or the table
 * is left out of the call; a page outside the pool that is needed is read as
 * zeros and not written; fm_paged_synchronize reports both.  Starts that fall
 * within the packed rows are not looked for: whose rows are written is then open.
 *
 * Calls allocate and copy nothing and change nothing in the handle: several
 * may run at once, from several host threads, on several streams and in
 * several graphs, as long as each has its own workspace and what they write is
 * apart.  The cache's device must be the current device.  Row pointers are
 * 16-byte aligned, their strides whole multiples of 16 bytes; a row's head_dim
 * values are contiguous.  Strides of an axis of one entry are not looked at.
 * ------------------------------------------------------------------------ */
#define FM_ROPE_INTERLEAVED 0   /* pairs (2 i, 2 i + 1) */
#define FM_ROPE_HALF 1          /* pairs (i, i + rot_dims / 2) */
#define FM_ROPE_PLAIN 0         /* angle pos f_i, f_i = theta^(-2 i / rot_dims) */
#define FM_ROPE_LINEAR 1        /* f_i / rope_factor */
#define FM_ROPE_BY_PARTS 2      /* f_i (r + (1 - r) / rope_factor), r = clamp((rope_rows f_i / 2 pi - rope_low) / (rope_high - rope_low), 0, 1):
                                   pairs that turn at least rope_high times over rope_rows rows keep their angle, those
                                   that turn at most rope_low times are stretched.  The ramp between is over turns, as the
                                   method's paper has it; implementations that ramp over the pair's index between borders
                                   rounded to whole pairs give the middle pairs other angles, which are not to be had here */

typedef struct fm_paged_config {
  int32_t n_layers;      /* 1 .. 1024 */
  int32_t n_pages;       /* pages a layer */
  int32_t page_rows;     /* 16, 32, 64, 128 or 256 */
  int32_t n_heads;       /* query heads, a multiple of n_kv_heads, at most 128 times as many */
  int32_t n_kv_heads;    /* 1 .. 256 */
  int32_t head_dim;      /* 64, 128 or 256 */
  int32_t dtype;         /* FM_DTYPE_F16 or FM_DTYPE_BF16: the pool's, and the attention's rows' */
  int32_t rot_dims;      /* rotated dims of a head, the first ones: a multiple of 16, 0 for none */
  int32_t rot_layout;    /* FM_ROPE_INTERLEAVED or FM_ROPE_HALF */
  int32_t rope_scaling;  /* FM_ROPE_PLAIN, FM_ROPE_LINEAR or FM_ROPE_BY_PARTS */
  int32_t rope_rows;     /* BY_PARTS: the context the angles were made for */
  float theta;           /* RoPE base, at least 1 */
  float rope_factor;     /* LINEAR, BY_PARTS: at least 1 */
  float rope_low, rope_high;   /* BY_PARTS: turns */
  float rope_gain;       /* the rotated dims are multiplied by it (1; scaled contexts may want more) */
  float eps;             /* of the norms */
} fm_paged_config;       /* (the rope fields and theta are not looked at where rot_dims is 0) */

typedef struct fm_paged_batch {
  const int32_t *starts;    /* device [n_seqs + 1], never falling */
  const int32_t *lengths;   /* device [n_seqs] */
  const int32_t *table;     /* device [n_seqs][table_pages], rows table_ld entries apart */
  int64_t table_ld;
  int32_t n_seqs;           /* 0 .. 65536 */
  int32_t n_tokens;         /* packed rows that q, k, v and out hold (starts[n_seqs] of them at most are new) */
  int32_t table_pages;      /* pages a sequence may have; at most 2^30 rows */
  int32_t max_new;          /* the most new rows a sequence may have: chooses the attention kernel and its workspace
                               (more of them than that are attended over all the same) */
} fm_paged_batch;

/* Rows [n_tokens][heads][head_dim]: data, and elements between tokens and between heads. */
typedef struct fm_paged_rows {
  void *data;
  int64_t token_stride, head_stride;
} fm_paged_rows;

typedef struct fm_paged fm_paged;

/*
 * fm_paged_create -- a cache over the caller's pool, on the current device (the pool's).  Synchronises the stream.
 * Errors: FM_ERR_INVALID_ARG, FM_ERR_UNSUPPORTED (head_dim, page_rows, heads a
 *   KV head, a pool of over 2^31 - 257 rows of heads), FM_ERR_OOM, FM_ERR_CUDA; *out is NULL on
 *   failure and the reason is in fm_paged_last_error(NULL).
 */
FM_API fm_status fm_paged_create(const fm_paged_config *cfg, void *k_pool_dev, void *v_pool_dev, void *stream,
                                 fm_paged **out);

/*
 * fm_paged_write -- per new row and head: q and k are divided by their root
 * mean square, sqrt(mean x^2 + eps), and multiplied by q_norm / k_norm (f32
 * [head_dim], 16-byte aligned; NULL: no norm), rotated at the row's position,
 * and rounded once to the pool's type; q goes to q_out, k and v (v as it is) to
 * the row's place in layer's pages.  q and q_out may be NULL (rows of context),
 * or k and v (queries alone; the pages are then not looked at).  dtype:
 * FM_DTYPE_F32 or the pool's.  Norms and rotation are f32; a position's angle
 * is taken from 64-bit turns, so far positions lose nothing.  q_out may be q
 * itself (the same type and strides).  Rows with a negative position (more new
 * rows than the length) are not written, and reported.
 * Errors: FM_ERR_INVALID_ARG, FM_ERR_UNSUPPORTED (limits above, 2^31 - 1 rows of heads in
 *   a batch), FM_ERR_CUDA.
 */
FM_API fm_status fm_paged_write(fm_paged *c, int32_t layer, const fm_paged_batch *batch, const fm_paged_rows *q,
                                const fm_paged_rows *k, const fm_paged_rows *v, int32_t dtype,
                                const float *q_norm_dev, const float *k_norm_dev, const fm_paged_rows *q_out,
                                void *stream);

/*
 * fm_paged_attend -- per new row (position p) and query head h:
 *   out = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale q . k_j),
 * over KV head h / (n_heads / n_kv_heads) and the rows j < length that it sees:
 * all of them; with causal != 0 those with j <= p; with a window > 0 (causal
 * only) those of them with j > p - window, and the first `sinks` (those with
 * j <= p).  A row that sees nothing gives zeros, one that sees only scores of minus
 * infinity NaN (0 / 0).  q and out are of the pool's type and do not overlap
 * (out->data == q->data is refused); scale is 1e-30 to 1e30.
 * Scores, weights' sums and outputs are summed in f32; each weight is rounded
 * once to the pool's type where it multiplies v, the output once at the end.  A
 * row that is not seen has no part in the result, whatever it holds (pages
 * outside every window of the call's rows are not read, their table entries
 * may be stale).  Of a key whose weight is below 2^-24 (f16) of the largest one
 * the part may be lost.  scale q . k past f32's range counts as infinite; past
 * 2^24, where a score's last bit is a factor of two or more, weights below the
 * largest are as rough as that.
 * Infinities and NaN of V that some rows of a unit see and others do not take a
 * slow path (1 us and up a key tile); in rows that none sees they cost nothing.
 * workspace_dev: fm_paged_workspace_bytes(c, batch->max_new) bytes on the device, 16-byte
 * aligned, its contents of no matter; no other call may use it until this one is done.
 * Errors: FM_ERR_INVALID_ARG, FM_ERR_UNSUPPORTED, FM_ERR_CUDA.  A bounded
 *   device wait that gives up is reported by fm_paged_synchronize.
 */
FM_API fm_status fm_paged_attend(fm_paged *c, int32_t layer, const fm_paged_batch *batch, const fm_paged_rows *q,
                                 const fm_paged_rows *out, float scale, int32_t causal, int32_t window,
                                 int32_t sinks, void *workspace_dev, int64_t workspace_bytes, void *stream);

/* The workspace of calls with batches of at most max_new new rows a sequence.  Errors: FM_ERR_INVALID_ARG. */
FM_API fm_status fm_paged_workspace_bytes(const fm_paged *c, int32_t max_new, int64_t *bytes);
/* The configuration the cache was made with.  Errors: FM_ERR_INVALID_ARG. */
FM_API fm_status fm_paged_get_config(const fm_paged *c, fm_paged_config *cfg);
/* Kernel launches issued by this host thread's last write or attend. */
FM_API fm_status fm_paged_last_launch_count(const fm_paged *c, int32_t *count);
/* Wait for the stream; FM_ERR_TIMEOUT if a bounded device wait gave up, FM_ERR_INVALID_ARG if a batch's numbers pointed
   outside, since the last check.  What it reports is cleared, the first of the two ahead of the second, which the next call
   reports; what other streams still run may raise them again. */
FM_API fm_status fm_paged_synchronize(fm_paged *c, void *stream);
/* fm_selftest_wait_timeout for a paged cache.  Errors: FM_ERR_INVALID_ARG, FM_ERR_CUDA. */
FM_API fm_status fm_paged_selftest_wait_timeout(fm_paged *c, int32_t budget_us, void *stream);
FM_API const char *fm_paged_last_error(const fm_paged *c);   /* never NULL; this host thread's last failed fm_paged call */
/* Free what the handle owns (not the pool).  NULL is ignored; a capture in progress goes on.  Graphs that hold its calls
   are not replayed afterwards. */
FM_API void fm_paged_destroy(fm_paged *c);

/*
 * fm_mtp_use_paged -- keep the MTP head's rows in layer of the paged cache c
 * from the next pass on (c NULL: in the head's own f32 cache again, which holds
 * what it held; fm_mtp_use_kvq and this call replace each other).  A pass
 * writes its rows by fm_paged_write, norms and rotation with them, and attends
 * by fm_paged_attend in the pool's type (f16 or bf16: the rows' roundings).  The
 * row of position p is row p of the sequence whose pages table_dev (device
 * int32 [table_pages], read when passes run, its pages changed only between
 * them) names; rows below a pass's pos0 were written by earlier passes or by
 * fm_paged_write.  The table's rows, not kv_cap, bound the positions (kv_cap
 * may be 1).  window, sinks: as fm_paged_attend's (0, 0: every row is seen).
 * c has the head's n_heads, n_kv_heads, head_dim, rot_dims, theta and eps, the half layout, and any
 * scaling of the angles; it stays the caller's and outlives its use.
 * Passes then also fail with FM_ERR_CONTEXT_FULL (positions past the table),
 * FM_ERR_UNSUPPORTED (kv_lo > 0) and FM_ERR_INVALID_ARG (another current
 * device); nothing is launched then.  fm_mtp_cache with rows > 0 answers
 * FM_ERR_STATE; with rows = 0 it also reports what fm_paged_synchronize does.
 * Errors: FM_ERR_INVALID_ARG (another device, configuration or layer, table, window or
 *   sinks), FM_ERR_OOM.
 */
FM_API fm_status fm_mtp_use_paged(fm_mtp *m, fm_paged *c, int32_t layer, const int32_t *table_dev,
                                  int32_t table_pages, int32_t window, int32_t sinks);

#ifdef __cplusplus
}
#endif
#endif /* FM_H_ */
