/* llmq — GB300-native per-token decode step of a Llama/Qwen-style decoder with
 * group-64 4-bit weights (W4A16), behind a plain C ABI.
 *
 * The operation is the decode step the aot-llm page ("p10node/aot-llm") draws
 * in its sequence diagram and "static pipeline": embedding -> [RMSNorm ->
 * q/k/v matvec -> RoPE -> attention over the KV cache -> o matvec + residual
 * -> RMSNorm -> gate/up -> SwiGLU -> down + residual] x L -> RMSNorm -> logits
 * -> greedy choice. Weights are "packed group-64 W4A16" (llmopt page); the KV
 * cache is bf16 appended from f32 (zynfer page, stage M4). The shape of the
 * API follows aot-llm's C library section (open a model, evaluate tokens, read
 * n_vocab logits, reset a context) and the pytensor-ml issue's "immutable
 * model, mutable context" and "fail at load with the missing capability named".
 *
 * Conventions for every entry point:
 *   - returns LLM_OK (0) or a negative llm_status; llm_last_error() then holds
 *     a one-line reason. LLM_ERR_CUDA and LLM_ERR_TIMEOUT poison the model
 *     (every later call returns the same error); all other errors leave it
 *     usable.
 *   - a model is not thread-safe: the caller serialises calls on one model.
 *   - output pointers marked "host or device" may point to either; the call
 *     is synchronous when any output is in host memory.
 *   - all device memory is owned by the library and allocated once, in
 *     llm_model_create; no call in the token loop allocates.
 */
#ifndef LLMQ_H
#define LLMQ_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define LLMQ_ABI_VERSION 1

typedef enum {
  LLM_OK = 0,
  LLM_ERR_INVALID_ARG = -1,   /* null pointer, out-of-range index, bad size */
  LLM_ERR_UNSUPPORTED = -2,   /* config the kernels do not cover; message names it */
  LLM_ERR_OOM = -3,           /* device allocation failed at create */
  LLM_ERR_CTX_FULL = -4,      /* position would reach max_seq */
  LLM_ERR_CUDA = -5,          /* CUDA runtime error (poisons the model) */
  LLM_ERR_TIMEOUT = -6,       /* a device-side wait hit its limit (poisons the model) */
  LLM_ERR_NAN = -7,           /* the logit reduction saw a NaN */
  LLM_ERR_NOT_FOUND = -8      /* tensor name unknown */
} llm_status;

typedef enum { LLM_F32 = 0, LLM_BF16 = 1, LLM_F16 = 2, LLM_Q4G64 = 3,
               LLM_Q8G32 = 4 /* int8 codes with one fp16 scale per 32 values (llm_kv_view) */ } llm_dtype;

/* llm_config.flags */
#define LLM_NO_GRAPH 1u       /* launch the step's kernels one by one (debugging) */
#define LLM_NO_PDL   2u       /* no programmatic dependent launch between kernels */
#define LLM_MULTI_KERNEL 4u   /* one kernel per phase instead of the persistent step kernel */
#define LLM_TEST_EXPIRE_WAIT 0x80000000u  /* test only: every grid barrier of the persistent step
                                 waits for one arrival too many with a 1 ms limit, so the first one
                                 expires; the call returns LLM_ERR_TIMEOUT (nothing faults or hangs) */
#define LLM_DEBUG_BATCH_HIDDEN 16u  /* keep every layer's residual of the last batched decode step
                                 for llm_debug_hidden_batch (adds L+1 device copies to the step) */
#define LLM_W4A8 64u          /* 4-bit weights x int8 activations in the batch-1 paths: every 4-bit GEMV
                                 input quantized once per 32-input block (fp16 scale amax/127, codes
                                 round(x/scale) clamped to +-127) and dotted in integers; the batched
                                 kernels keep their fp16 tensor-core inputs. Not with LLM_DATAFLOW_STEP */
#define LLM_KV_Q8 128u        /* grouped int8 K/V cache (llmopt README, "Current compiler and runtime":
                                 grouped-Q8 attention state): each 32 values of a (position, kv head)
                                 row stored as int8 codes with one fp16 scale fp16(amax/127), codes
                                 round(x/scale) half away from zero clamped to +-127, decided in fp32;
                                 attention reads the codes and scales. Persistent step only (not with
                                 LLM_MULTI_KERNEL or LLM_DATAFLOW_STEP); llm_kv_write quantizes its bf16
                                 rows the same way, llm_kv_read_q8 reads codes and scales */
#define LLM_DATAFLOW_STEP 8u  /* greedy batch-1 steps on the flag-synchronised persistent kernel (phases
                                 wait on flagged words instead of grid barriers; slower than the
                                 default grid-barrier step on GB300, kept for comparison) */

typedef struct {
  int32_t abi_version;        /* must equal LLMQ_ABI_VERSION */
  int32_t dim, n_layers, n_heads, n_kv_heads, head_dim, ffn_dim, vocab;
  float   norm_eps;           /* RMSNorm epsilon */
  int32_t rope_neox;          /* 0: rotate pairs (2i, 2i+1); 1: pairs (i, i + head_dim/2) */
  double  rope_theta;         /* RoPE base: theta_i = base^(-2i/head_dim) */
  int32_t qk_norm;            /* 1: per-head RMSNorm of q and k before RoPE (Qwen3) */
  int32_t tied_embedding;     /* 1: LM head is the bf16 embedding table */
  int32_t max_seq;            /* KV capacity per sequence (positions) */
  int32_t max_batch;          /* number of sequences (independent caches) */
  uint32_t flags;             /* LLM_NO_GRAPH | LLM_NO_PDL | LLM_MULTI_KERNEL | LLM_DATAFLOW_STEP |
                                 LLM_DEBUG_BATCH_HIDDEN | LLM_W4A8 | LLM_KV_Q8 | LLM_TEST_EXPIRE_WAIT */
} llm_config;

/* One input tensor in the canonical layout, host memory, caller-owned, only
 * read during llm_model_create (the caller may free it afterwards).
 *   LLM_Q4G64 linear [rows=out][cols=in], cols % 64 == 0:
 *       codes  uint8 [rows][cols/2], element 2j in the low nibble of byte j,
 *                    element 2j+1 in the high nibble;
 *       scales fp16  [rows][cols/64];  mins fp16 [rows][cols/64];
 *       weight w[r][c] = scale[r][c/64] * q + min[r][c/64].
 *   LLM_F32 / LLM_BF16 dense [rows][cols] in `data` (norm weights: rows = 1).
 * Names: "embed" (f32, or bf16 when tied) [vocab][dim]; "final_norm";
 * per layer l: "L{l}.attn_norm", "L{l}.ffn_norm", "L{l}.q_norm", "L{l}.k_norm"
 * (qk_norm only, [head_dim]); q4 "L{l}.wq" [n_heads*head_dim][dim],
 * "L{l}.wk", "L{l}.wv" [n_kv_heads*head_dim][dim], "L{l}.wo"
 * [dim][n_heads*head_dim], "L{l}.w_gate", "L{l}.w_up" [ffn_dim][dim],
 * "L{l}.w_down" [dim][ffn_dim]; "lm_head" q4 [vocab][dim] when untied. */
typedef struct {
  const char* name;
  int32_t dtype;              /* llm_dtype */
  int64_t rows, cols;
  const void* codes;          /* LLM_Q4G64 */
  const void* scales;
  const void* mins;
  const void* data;           /* LLM_F32 / LLM_BF16 */
} llm_tensor;

typedef struct llm_model llm_model;

typedef struct {
  int64_t device_bytes;       /* all device memory owned by the model */
  int64_t weight_stream_bytes;/* repacked weight bytes read per decode step */
  int64_t kv_bytes_per_pos;   /* bf16 K+V bytes per cached position, all layers */
  int32_t kernels_per_step;   /* kernel nodes in one batch-1 step */
  int32_t n_sm;               /* SMs of the device the model lives on */
} llm_stats;

/* Validate the config, repack the 4-bit weights into the GPU tile layout, copy
 * everything to the device, size all buffers and capture the step graph.
 * cuda_stream: cudaStream_t to run on, or NULL for a stream the model owns.
 * Errors: INVALID_ARG, UNSUPPORTED (head_dim not 64/128, cols % 64, heads not
 * divisible, missing tensor...), NOT_FOUND, OOM, CUDA. On error *out = NULL.
 * Source: aot-llm README, "Library output" and its C example (aot_open: the model opened once, weights
 * ready); pytensor-ml issue #53, "Acceptance rules that apply to every PR" (fail at load with the
 * missing capability named). */
int llm_model_create(const llm_config* cfg, const llm_tensor* tensors, int32_t n_tensors,
                     void* cuda_stream, llm_model** out);

/* Free every device allocation of the model. NULL is accepted.
 * Source: no page counterpart: the model owns its device memory (pytensor-ml issue #53, "Already
 * here": immutable model, mutable context). */
void llm_model_destroy(llm_model* m);

/* Append n tokens (host array) to sequence seq at positions len..len+n-1 and
 * return the last position's fp32 logits [vocab] and greedy token. Runs n
 * decode steps. logits_out / argmax_out: host or device, may be NULL.
 * Errors: INVALID_ARG, CTX_FULL (len + n > max_seq), NAN, CUDA, TIMEOUT.
 * Source: aot-llm README C example (aot_eval of n prompt tokens, then aot_logits: n_vocab floats); the
 * static pipeline emitted for every model (aot-llm README) run once per token. */
int llm_prefill(llm_model* m, int32_t seq, const int32_t* tokens, int32_t n,
                float* logits_out, int32_t* argmax_out);

/* The same contract as llm_prefill, computed as batched prompt processing
 * (aot-llm "Batched prompt processing": each weight row read once per chunk of
 * tokens; llmopt "prefill-style GEMM"): chunks of up to 32 tokens go through
 * the batched pipeline (4-bit skinny GEMMs on the tensor cores, fp32
 * accumulation) with the chunk's rows appending their k, v to the cache first
 * and then attending causally over it. Equal to token-by-token prefill within
 * floating-point tolerance (a different summation order); the greedy token is
 * the argmax of the returned logits. llm_debug_hidden is not updated.
 * Errors as llm_prefill. */
int llm_prefill_batched(llm_model* m, int32_t seq, const int32_t* tokens, int32_t n,
                        float* logits_out, int32_t* argmax_out);

/* One decode step of sequence seq for `token` at position len; len += 1.
 * logits_out [vocab] fp32 and argmax_out (lowest index wins ties): host or
 * device, may be NULL. Errors as llm_prefill.
 * Source: aot-llm README, "The static pipeline emitted for every model" and its C example (one token
 * through aot_eval, aot_logits); pytensor-ml issue #53 (one-token append to the cache). */
int llm_decode_step(llm_model* m, int32_t seq, int32_t token, float* logits_out,
                    int32_t* argmax_out);

/* n_steps greedy steps starting from first_token; each step's argmax feeds the
 * next step on the device (no host round trip per step). tokens_out
 * [n_steps] (host or device) receives the token chosen at each step.
 * Source: zynfer PR #100, stage M3 (one command buffer per forward, 2 waits per token instead of 476:
 * the step runs on the device without a host round trip). */
int llm_decode_greedy(llm_model* m, int32_t seq, int32_t first_token, int32_t n_steps,
                      int32_t* tokens_out);

/* Sampled instead of greedy next-token choice for the batch-1 calls
 * (llm_prefill, llm_prefill_batched, llm_decode_step, llm_decode_greedy), from
 * the options the aot-llm page lists ("Generated binary options": temperature,
 * 0 = greedy; top-k; top-p; seed). Keep the top_k largest logits (ties: lower
 * token id), p = softmax((l - l_max) / temperature), keep the shortest prefix
 * whose cumulative probability reaches top_p, and take the first token whose
 * cumulative probability exceeds u times the prefix total. The draw u for the
 * token after position pos of sequence seq is Philox4x32-10 (Salmon et al.,
 * SC 2011) of counter (pos, seq, 0, 0) and key (seed low, seed high word):
 * u = (x0 >> 8) / 2^24, reproducible from the seed. The chosen token is what
 * argmax_out / tokens_out return and what llm_decode_greedy feeds back.
 * temperature 0 restores the greedy choice. llm_decode_step_batch stays
 * greedy. Errors: INVALID_ARG (temperature < 0 or not finite; when sampling,
 * top_k outside 1..64 or top_p outside (0, 1]). */
int llm_set_sampling(llm_model* m, float temperature, int32_t top_k, float top_p, uint64_t seed);

/* One decode step for sequences 0..n_seq-1 at once (n_seq == max_batch >= 2,
 * at most 32), each at its own position (its cache may come from
 * llm_kv_write or llm_prefill). The 4-bit matvecs become skinny GEMMs (fp32
 * register tiles, each weight dequantised once for every sequence); attention
 * runs over every sequence's own cache length. tokens [n_seq] (host or
 * device), or NULL to continue every sequence from its previous greedy token
 * on the device; logits_out [n_seq][vocab] and argmax_out [n_seq]: host or
 * device, may be NULL. Synchronous when tokens or an output are host memory.
 * Errors: UNSUPPORTED (max_batch < 2), INVALID_ARG, CTX_FULL, NAN, CUDA.
 * Source: no page decodes several sequences at once; this applies the batched prompt path of the
 * aot-llm README ("Batched prompt processing": each weight row read once for a chunk of tokens) to one
 * token of each sequence. */
int llm_decode_step_batch(llm_model* m, const int32_t* tokens, int32_t n_seq,
                          float* logits_out, int32_t* argmax_out);

/* Forget the cache of sequence seq (-1: all); its length becomes 0.
 * Source: aot-llm README C example (aot_ctx_reset). */
int llm_kv_reset(llm_model* m, int32_t seq);

/* Copy bf16 keys/values [n][n_kv_heads][head_dim] (host or device) into
 * positions pos0..pos0+n-1 of one layer of sequence seq; keys are stored as
 * given (already rotated). The sequence length becomes max(len, pos0 + n).
 * Errors: INVALID_ARG, CTX_FULL.
 * Source: aot-llm README (aot_ctx_save / aot_ctx_load move a conversation's cache between processes);
 * zynfer PR #100, stage M4 (bf16 KV cache appended from f32). */
int llm_kv_write(llm_model* m, int32_t seq, int32_t layer, int32_t pos0, int32_t n,
                 const uint16_t* k_bf16, const uint16_t* v_bf16);

/* Read back bf16 keys/values [n][n_kv_heads][head_dim] (host or device).
 * Source: as llm_kv_write. */
int llm_kv_read(llm_model* m, int32_t seq, int32_t layer, int32_t pos0, int32_t n,
                uint16_t* k_bf16, uint16_t* v_bf16);

/* Read back an int8 cache (LLM_KV_Q8 models): codes k, v [n][n_kv_heads][head_dim]
 * and fp16 scale bits ks, vs [n][n_kv_heads][head_dim / 32], host or device.
 * Source: llmopt README, "Current compiler and runtime" (grouped-Q8 attention state). */
int llm_kv_read_q8(llm_model* m, int32_t seq, int32_t layer, int32_t pos0, int32_t n, int8_t* k, uint16_t* ks,
                   int8_t* v, uint16_t* vs);

/* Current cache length of sequence seq, or a negative llm_status.
 * Source: pytensor-ml issue #53, "Already here" (the cache and its one-token append). */
int llm_kv_len(const llm_model* m, int32_t seq);

/* Residual stream after the embedding and after every layer of the last
 * batch-1 step: out [(n_layers+1)][dim] fp32, host or device.
 * Source: pytensor-ml issue #53, "Acceptance rules that apply to every PR" (an independent oracle, the
 * cached output checked at every step). */
int llm_debug_hidden(llm_model* m, float* out);

/* Residual stream of every sequence after the embedding and after every layer
 * of the last llm_decode_step_batch: out [(n_layers+1)][max_batch][dim] fp32,
 * host or device. Needs a model created with LLM_DEBUG_BATCH_HIDDEN
 * (else LLM_ERR_UNSUPPORTED).
 * Source: as llm_debug_hidden. */
int llm_debug_hidden_batch(llm_model* m, float* out);

/* Undo the repack of one 4-bit tensor: write its canonical codes [rows][cols/2],
 * scales and mins [rows][cols/64] (host) from the device copy.
 * Source: aot-llm README, testing section (every dot product and weight type checked against a scalar
 * reference). */
int llm_debug_unpack(llm_model* m, const char* name, uint8_t* codes, uint16_t* scales,
                     uint16_t* mins);

/* Test hook: the nth device allocation (counted from 1) made by the models
 * created after this call fails as if cudaMalloc had run out of memory, so
 * llm_model_create returns LLM_ERR_OOM naming the buffer and frees what it
 * had allocated. nth <= 0 disarms it. Process-wide; returns LLM_OK.
 * Source: zynfer PR #100, stage M6 (allocation behaviour tested with a failing allocator). */
int llm_debug_fail_alloc(int32_t nth);

/* Test hook: on != 0 makes a wait of each CTA of the llm_tree_attention,
 * llm_prefix_attention and plain llm_token_probs calls launched from then on
 * (llm_decode_tree's among them) run out, after 1 ms; their outputs are not valid, and llm_tree_status, or the model's
 * call, reports TIMEOUT. Process-wide; returns LLM_OK.
 * Source: as llm_debug_fail_alloc. */
int llm_debug_expire_waits(int32_t on);

/* Sizes and counts of the model (host struct).
 * Source: zynfer PR #100, stages M2-M4 (bytes per token for the roofline estimate). */
int llm_model_stats(const llm_model* m, llm_stats* out);

/* One launch of a decode step, as timed by llm_profile_step. */
typedef struct {
  int32_t kind;               /* 0 4-bit GEMV, 1 bf16 GEMV, 2 attention, 3 logits/argmax */
  int32_t layer;              /* -1 for the LM head and the argmax */
  int64_t bytes;              /* algorithmic HBM bytes: weight units, or K/V rows read */
  float   ms;                 /* CUDA-event duration on the model's stream */
} llm_kernel_time;

/* Run one decode step of `token` like llm_decode_step, but eagerly and
 * without programmatic dependent launch, with a CUDA event pair around every
 * kernel. Writes up to max_out records (launch order) and returns the number
 * of launches, or a negative llm_status. Meant for measurement, not the token
 * loop (it creates and destroys events).
 * Source: zynfer PR #100, stage M2 (per-family timing and a roofline JSON). */
int llm_profile_step(llm_model* m, int32_t seq, int32_t token, llm_kernel_time* out, int32_t max_out);

/* Time back-to-back launches of the batch-1 step's kernels of sequence seq
 * (programmatic dependent launch between them, CUDA events on the model's
 * stream) on the buffers the last step left. which = 0 q|k|v GEMV, 1
 * attention, 2 o GEMV, 3 gate|up GEMV, 4 down GEMV: that kernel for `layer`,
 * or for every layer in turn when layer = -1 (so that a weight set larger than
 * L2 is streamed); 5 the LM-head GEMV; 6 every 4-bit/bf16 GEMV of one step in
 * step order. The list is launched n times. Attention launches re-append the
 * last position with the values already there. Writes the mean milliseconds
 * per launch and the mean algorithmic bytes per launch. Needs at least one
 * completed step of seq.
 * Source: as llm_profile_step. */
int llm_time_kernel(llm_model* m, int32_t seq, int32_t which, int32_t layer, int32_t n, float* ms,
                    int64_t* bytes);

/* On a model without LLM_DATAFLOW_STEP, in a library built with
 * LLMQ_PHASE_STAMPS=1 (else LLM_ERR_UNSUPPORTED): one step (n_steps = 1) of
 * the grid-barrier persistent step, recording per (phase, CTA) the clock64
 * stamps 0 phase start, 1 grid barrier passed, 2 input built, 3 weight units
 * done, 4 arrival issued (0 where a phase has no such point), and with
 * LLMQ_UNIT_STAMPS=1 also 5..8 the largest and summed per-warp cycles waiting
 * for units and in unit dots; values 12..15 of phase 0's records hold
 * (%globaltimer, clock64) at each CTA's start and end; out [phases][n_sm][16].
 * Otherwise: run n_steps (1..8) greedy steps of sequence seq from first_token through the
 * flag-synchronised step kernel in one launch and record, for every (step,
 * phase, CTA), 16 values: the SM cycle counter (clock64) when the phase's
 * input build starts, when its inputs have all arrived, when the build is
 * done, when the phase's weight units are done and when its outputs are
 * published (the LM head's stays 0); the largest and the summed per-warp
 * cycles spent waiting for weight units and computing unit dots; values 12..15
 * of the CTA's (step 0, phase 0) record hold (%globaltimer ns, clock64) at the
 * kernel's start and end, which map its cycles onto one time line.
 * out [n_steps][phases][n_sm][16] (host); phases are the four GEMVs of every
 * layer (q|k|v, o with the attention in its build, gate|up, down) and the LM
 * head. Returns the number of records (n_steps * phases * n_sm) or a negative
 * llm_status (UNSUPPORTED when the step kernel does not cover these
 * positions). len += n_steps. For measurement, not the token loop.
 * Source: as llm_profile_step. */
int llm_phase_times(llm_model* m, int32_t seq, int32_t first_token, int32_t n_steps, uint64_t* out,
                    int64_t max_out);

/* Wait for all queued work of the model and report device-side errors.
 * Source: pytensor-ml issue #53, "Acceptance rules that apply to every PR" (errors reported, not
 * swallowed). */
int llm_sync(llm_model* m);

/* Last error text of the model (m may be NULL: the last error of this thread
 * in a create or in a call without a model). Never NULL; owned by the library.
 * Source: as llm_sync. */
const char* llm_last_error(const llm_model* m);

/* Kernel-level check: y = W x through the same repack and dequant-GEMV kernel
 * the decode step uses (plain store epilogue). w: one LLM_Q4G64 or LLM_BF16
 * tensor (host, cols a multiple of 64 up to 8192); x [cols], y [rows] fp32
 * host arrays. Allocates and frees its
 * own device memory; not for the token loop.
 * Source: aot-llm README, testing section (every matrix product against a float reference). */
int llm_op_matvec(const llm_tensor* w, const float* x, float* y);

/* llm_op_matvec in the W4A8 numerics of LLM_W4A8 (Q4G64 tensors only): x is
 * quantized per 32-input block to int8 with an fp16 scale (aot-llm README,
 * implementation notes: the f32 activation vector quantized once to Q8_0,
 * integer dot products scaled back to f32), each block's integer sums
 * scaled by its d and the group's scale and min. */
int llm_op_matvec_w4a8(const llm_tensor* w, const float* x, float* y);

/* y = W x with one weight matrix already resident in model m, without any
 * device allocation. No page has a counterpart: it exists for callers that
 * cannot call cudaMalloc at this point -- a process whose device memory was
 * handed to its own pool at start-up (a new cudaMalloc would fail or bypass
 * the pool's accounting), or a latency-critical loop where cudaMalloc/cudaFree
 * would stall (cudaFree synchronises the device). The caller passes x [cols]
 * and y [rows] as fp32 device buffers (y must not overlap x) on the model's
 * device, which must be the current device; `name` is a 4-bit tensor stored
 * as a contiguous row range ("L{l}.wq", "L{l}.wk", "L{l}.wv", "L{l}.wo",
 * "L{l}.w_down", "lm_head") or "embed" for a tied bf16 LM head.
 * Scratch (split-row-tile partial sums, arrival counters, a status word) lives
 * in one file-scope device array of 4 MiB + 128 KiB + 256 B that every GPU
 * loading the library keeps until exit; a matrix needing more partial-sum or
 * counter space is rejected with LLM_ERR_UNSUPPORTED naming both sizes (the
 * model stays usable). The first call on a device looks up the array's device
 * address (cudaGetSymbolAddress) and keeps it for the process: it does not
 * survive cudaDeviceReset, after which this call must not be used again.
 * Every call shares the array and clears its counters and status on
 * `cuda_stream` (NULL: the legacy default stream) before the kernel: calls
 * whose work overlaps on the GPU race on it, so serialise them. The call is
 * synchronous -- it reads the status word back and synchronises
 * `cuda_stream`, returning after y is written -- so it cannot be captured
 * into a graph: on a capturing stream it returns LLM_ERR_INVALID_ARG without
 * touching the stream or the model. Device ordinals of 64 and above:
 * LLM_ERR_UNSUPPORTED. */
int llm_matvec_noalloc(const llm_model* m, const char* name, const float* x, float* y, void* cuda_stream);

/* ---- tree decoding ---------------------------------------------------------
 * Operators of a decoding step that verifies a tree of drafted tokens: node 0
 * is the root (the last chosen token), every other node a draft whose parent
 * has a lower index. llm_tree_attention scores all nodes over the cache in one
 * pass, llm_token_probs turns logits into the sampler's probabilities,
 * llm_verify_tree decides which drafts are kept, llm_commit_tree moves the
 * kept nodes' K/V rows into the cache; llm_decode_tree runs all of them for a
 * model's own sequence.
 *
 * Each of the four works on the caller's device buffers on the current device
 * and on `cuda_stream` (NULL: the legacy default stream). They are
 * asynchronous, allocate nothing, keep nothing between calls and can be
 * captured into a graph; calls on different streams share no state. Errors
 * (INVALID_ARG, UNSUPPORTED, CUDA) are returned before any launch, with their
 * reason in llm_last_error(NULL) of the calling thread. Buffers must stay
 * valid, and outputs must not overlap inputs where not said otherwise. Lengths,
 * counts, paths and tokens are read on the device: values outside their range
 * never lead out of a buffer (they are clamped or their node is skipped).
 * Source: no page drafts tokens; the cache formats are llm_kv_write's. */

/* K and V rows in device memory, [seq][layer][head][row][head_dim] at any
 * strides (in elements, multiples of 16 bytes, below 2^38; a row is contiguous;
 * k and v 16-byte aligned and laid out alike; a sequence or head stride of 0
 * shares the rows). LLM_BF16, or LLM_Q8G32: int8 codes and
 * fp16 scales [..][head_dim / 32] at the scale strides (multiples of
 * head_dim / 32, aligned to a row of scales). head_dim 64 or 128. */
typedef struct {
  int32_t dtype;
  int32_t n_seq, n_layers, n_heads, rows, head_dim;
  void *k, *v, *k_scales, *v_scales;
  int64_t seq_stride, layer_stride, head_stride, row_stride;
  int64_t scale_seq_stride, scale_layer_stride, scale_head_stride, scale_row_stride;
} llm_kv_view;

typedef struct {
  int32_t dtype;                /* of q and out: LLM_BF16 or LLM_F32 */
  int32_t n_seq, n_nodes, n_heads;  /* n_nodes 1..64; n_heads a multiple of the cache's heads */
  const void* q;                /* [n_seq][n_nodes][n_heads][head_dim], already rotated */
  void* out;                    /* the same shape; rows of nodes at or past counts[b] are left as they were */
  int64_t q_strides[3], out_strides[3];  /* elements (seq, node, head), multiples of 16 bytes */
  const llm_kv_view* cache;     /* one layer; the first n_seq sequences */
  const llm_kv_view* tree;      /* the nodes' own rows (node j at row j), or NULL: the cache alone */
  const int32_t* lens;          /* [n_seq] cache rows that every node sees (clamped to 0..rows) */
  const uint64_t* mask;         /* [n_seq][n_nodes] bit j: the node sees tree row j (not read when tree is NULL) */
  const int32_t* counts;        /* [n_seq] nodes of each sequence (clamped to 0..n_nodes), or NULL: n_nodes */
  float scale;                  /* of the scores, usually 1/sqrt(head_dim) */
} llm_tree_attention_args;

/* out = softmax(scale q K^T over the visible rows) V; query head h reads kv
 * head h / (n_heads / cache heads). Products on the tensor cores, sums in
 * fp32 (for fp32 queries the tensor cores, which cut off, add up 256 rows at
 * most); fp32 queries and their probabilities carry 24 bits, for bf16 queries
 * the probabilities and int8 rows' values 16. Over bf16 rows, where a CTA takes
 * 128 query rows (more than 64 of a kv head's nodes x heads, in a batch that
 * fills the GPU), bf16 queries' probabilities carry 8: the error is then 1.41
 * times that of an exact output rounded to bf16, and so depends on the batch.
 * Scores may have any finite size. A node that sees no row gets zeros. A row that
 * a node does not see has no influence on it, whatever it holds. With n_nodes = 1
 * and tree = NULL this is one decode token's attention over a cache that already
 * holds its row. */
int llm_tree_attention(const llm_tree_attention_args* args, void* cuda_stream);

/* Wait for `cuda_stream` and report whether a device-side wait of a
 * llm_tree_attention, llm_prefix_attention or llm_token_probs on the current device passed its limit
 * (2 s) since the last call (TIMEOUT: the outputs of that call are not valid). */
int llm_tree_status(void* cuda_stream);

/* probs[r] = the distribution the sampler of llm_set_sampling draws from:
 * the top_k largest logits (1..64, ties to the lower id; 0: all of them), of
 * softmax(logit / temperature) over them the shortest prefix whose mass reaches
 * top_p, renormalised; every other token 0. fp32 rows at the given strides
 * (elements); probs may be logits itself. A NaN logit counts as -inf, +inf as the
 * largest finite value, a row without a finite logit gives zeros.
 * With a top_k, a row takes time quadratic in the number of its largest logits
 * where they crowd at fewer than top_k of the 128 places (j mod 512) / 4 of a
 * slice of it (9 ms for half of 151936 tokens). UNSUPPORTED: top_p < 1 without
 * a top_k, vocab over 524288 (819200 without top_k). */
int llm_token_probs(const float* logits, int64_t logits_stride, float* probs, int64_t probs_stride, int32_t n_rows,
                    int32_t vocab, float temperature, int32_t top_k, float top_p, void* cuda_stream);

typedef struct {
  int32_t n_seq, n_nodes, vocab;  /* n_nodes 1..64 */
  const int32_t* tokens;          /* [n_seq][n_nodes]; the root's is not tested */
  const int32_t* parents;         /* [n_seq][n_nodes] a lower node's index; other values: the node is never reached */
  const int32_t* counts;          /* [n_seq] or NULL, as in llm_tree_attention */
  const float* uniforms;          /* [n_seq][n_nodes] in [0, 1): entry i >= 1 tests node i, entry 0 draws the last token */
  const float* probs;             /* [n_seq][n_nodes][vocab] target probabilities after each node */
  int64_t probs_strides[2];       /* elements (seq, node) */
  const float* draft_probs;       /* the same shape: what each node's children were drawn from (independently), or
                                     NULL: the children are fixed choices (a top-k tree, a lookup) */
  int64_t draft_strides[2];
  const int32_t* targets;         /* [n_seq][n_nodes] greedy mode instead of probs: the target's choice after each node */
  int32_t* path;                  /* [n_seq][n_nodes] out: kept nodes from the root on, then -1 */
  int32_t* n_path;                /* [n_seq] out: how many (at least 1, the root) */
  int32_t* next;                  /* [n_seq] out: the token that follows the last kept node */
} llm_verify_tree_args;

/* Speculative sampling over a tree; the tokens that come out are distributed
 * as the target's own. From the root, the current node's children are tested
 * in index order. r = probs[node], m = 1; child i with token x is kept when
 * u_i q(x) < r(x) / m and becomes the current node; otherwise r becomes
 * max(r/m - q, 0) and m its sum (a rejection that leaves nothing does not
 * count). Without draft_probs q(x) = 1 and a rejected token loses its
 * probability: r(x) becomes 0, and m, from 1 on, less by it (rows are taken to
 * sum to 1 up to their rounding). When no child is left, next is the first token
 * where the running sum of r exceeds u_0 times r's sum (vocab - 1 if probs[node]
 * has no mass). Decisions are made with sums of at least 45 bits. Negative and
 * NaN probabilities count as 0; a token outside 0..vocab-1 is never kept.
 * counts[b] = 0: path all -1, n_path 0, next -1. Greedy mode: a child is kept
 * when its token equals targets[current]; next = targets[last]. */
int llm_verify_tree(const llm_verify_tree_args* args, void* cuda_stream);

/* cache row lens[b] + k = tree row path[b][k] for k < n_path[b], in every layer
 * and head, K, V and scales; new_lens[b] = lens[b] + n_path[b] (new_lens may be
 * lens). Rows past the cache's end are dropped and new_lens stops there;
 * entries of path outside 0..rows-1 leave their cache row as it was. The tree's rows
 * are no rows of the cache (not a draft area behind lens). path [n_seq][n_nodes]. */
int llm_commit_tree(const llm_kv_view* cache, const llm_kv_view* tree, int32_t n_seq, int32_t n_nodes,
                    const int32_t* lens, const int32_t* path, const int32_t* n_path, int32_t* new_lens,
                    void* cuda_stream);

/* One decoding step of sequence seq over a drafted tree of n nodes (1..32):
 * tokens[0] is the token that follows the cache (the last chosen one),
 * parents[i] < i for every other node; both host or device. All nodes run
 * through the batched pipeline at once (node i at position len + its depth,
 * seeing the cache, its ancestors and itself), then the drafts are verified
 * (llm_verify_tree): greedily, or with sampling on (llm_set_sampling) against
 * the sampler's distribution with `uniforms` [n] in [0, 1) (host or device) and
 * `draft_probs` [n][vocab] (device, or NULL: fixed choices; read behind the work
 * that the legacy default stream has at the call: work on a stream that does not
 * synchronize with it has to have ended, or to be on the model's). The kept nodes'
 * K/V rows are appended and the sequence grows by their number. path_out [n]
 * receives the kept nodes (then -1), n_path_out their number, next_out the
 * token after them (the next tree's root), logits_out (may be NULL) the [n][vocab] logits of
 * every node: host or device. Synchronous. With greedy choices the tokens are
 * those of llm_decode_greedy within floating-point tolerance. An error leaves
 * the sequence as it was. Errors: INVALID_ARG, UNSUPPORTED (n; with sampling on,
 * a vocab over 524288), CTX_FULL (len + n > max_seq), NAN, CUDA, TIMEOUT.
 * Source: no page drafts tokens; the pipeline is llm_prefill_batched's. */
int llm_decode_tree(llm_model* m, int32_t seq, const int32_t* tokens, const int32_t* parents, int32_t n,
                    const float* draft_probs, const float* uniforms, int32_t* path_out, int32_t* n_path_out,
                    int32_t* next_out, float* logits_out);

/* ---- serving ---------------------------------------------------------------
 * Operators of a decoding step of a served batch on the caller's own tensors:
 * llm_append_kv norms and rotates new tokens' heads and writes their rows,
 * llm_prefix_attention attends behind prefixes that sequences share,
 * llm_sample_tokens draws the next tokens, llm_read_kv reads rows back. The
 * conventions are those of the tree-decoding operators above (streams, errors,
 * captures, values read on the device); they follow one another and those on one
 * stream: llm_append_kv writes rows of the views that the attentions read.
 * Source: as the tree-decoding operators; the formats are llm_kv_write's, the
 * options llm_set_sampling's. */

typedef struct {
  int32_t dtype;                /* of q, k and v: LLM_BF16 or LLM_F32 */
  int32_t out_dtype;            /* of q_out: LLM_BF16 or LLM_F32 */
  int32_t n_tokens, n_heads;    /* n_heads: of q (0 with q NULL); k and v have the cache's heads */
  const void *q, *k, *v;        /* [token][head][head_dim]; q may be NULL */
  void* q_out;                  /* [token][head][head_dim]; may be q itself (same type and strides) */
  int64_t q_strides[2], k_strides[2], v_strides[2], out_strides[2];  /* elements (token, head), multiples of 16 bytes */
  const llm_kv_view* cache;     /* one layer */
  const int32_t* seqs;          /* [n_tokens] sequence and */
  const int32_t* rows;          /* [n_tokens] row that a token's k and v go to; out of range: they go nowhere */
  const int32_t* positions;     /* [n_tokens] of the rotation, any int32; NULL: rows */
  const float *q_norm, *k_norm; /* [head_dim] RMSNorm weights of a head (16-byte aligned), or NULL: no norm */
  float norm_eps;
  double rope_theta;            /* base, at least 2^-10; 0: no rotation */
  int32_t rope_neox;            /* as in llm_config */
} llm_append_kv_args;

/* Per token and head: q and k normed (x / sqrt(mean(x^2) + eps) * weight) and
 * rotated by position * rope_theta^(-2i/head_dim), q to q_out, k and v (as they
 * are) to the cache's row in its format: bf16, or int8 codes and scales with the
 * roundings of LLM_KV_Q8. Computed in fp32, angles in 64-bit fixed point (2^-30 of a
 * turn at position 2^20, of bases from 1/4 on), rounded once into the outputs. Int8 rows: values past
 * 65504 * 127 saturate, a NaN makes its 32 values NaN. With q, norms and rope_theta
 * left out it writes rows as they are, quantised for an int8 cache. The (seq, row)
 * pairs of a call differ; of two equal ones the row holds parts of either. */
int llm_append_kv(const llm_append_kv_args* args, void* cuda_stream);

/* k[l][t], v[l][t] = the values of row rows[t] of sequence seqs[t] in every layer
 * and head, as LLM_BF16 or LLM_F32 (int8 rows: code times scale, rounded once);
 * zeros where seqs[t] or rows[t] is out of range. Both outputs, each in memory of its
 * own, lie at out_strides (elements: layer, token, head; multiples of 16 bytes). */
int llm_read_kv(const llm_kv_view* cache, int32_t n_tokens, const int32_t* seqs, const int32_t* rows, int32_t out_dtype,
                void* k, void* v, const int64_t* out_strides, void* cuda_stream);

typedef struct {
  llm_tree_attention_args attention;  /* the queries, every sequence's own rows, its new tokens (tree, mask), the output */
  const llm_kv_view* prefix;    /* one layer, alike the cache: rows of its sequence g are those that group g shares */
  int32_t n_groups;             /* up to the prefix view's sequences */
  const int32_t* starts;        /* [n_groups + 1] ascending: sequences starts[g] .. starts[g + 1] - 1 are group g
                                 * (of others, the rows are whatever they come to; nothing else is written) */
  const int32_t* prefix_lens;   /* [n_groups] rows of each prefix (clamped to 0..rows) */
  void* workspace;              /* device memory, 32-byte aligned; calls that may overlap have one each */
  int64_t workspace_bytes;      /* at least llm_prefix_workspace's */
} llm_prefix_attention_args;

/* llm_tree_attention where every node sees, before its sequence's own rows, the
 * first prefix_lens[g] rows of its group's prefix; those are read and multiplied
 * once for all sequences of the group. Sequences outside of starts[0] ..
 * starts[n_groups] - 1 see no prefix. What llm_tree_attention says of types,
 * precision, counts, masks and empty rows holds here too (bf16 queries over bf16
 * prefix rows: the probabilities carry 8 bits where the batch has more than 64 query
 * rows, n_seq x n_nodes x heads, of a kv head). One decode token: n_nodes = 1, its row already in the cache and
 * tree NULL, or its row as the tree's. llm_tree_status reports waits that ran out.
 * The host chooses kernels and splits and does not know the lengths: it goes by the rows
 * of the views. Views narrowed to the batch's longest length are faster than ones of a
 * cache's whole room (32 sequences of 20 rows, 16/8 heads x 128, behind 2048: 16 us in
 * bf16 views of 20 rows, 28 of 4096; int8 prefixes of 2048 rows 19 us, in a view of 32768
 * 37). */
int llm_prefix_attention(const llm_prefix_attention_args* args, void* cuda_stream);

/* Bytes of llm_prefix_attention's workspace, or a negative llm_status. Nothing in it
 * has to be set, or is kept for another call. */
int64_t llm_prefix_workspace(int32_t n_seq, int32_t n_nodes, int32_t n_heads, int32_t head_dim);

typedef struct {
  const float* logits;          /* [n_rows][vocab] at logits_stride (elements) */
  int64_t logits_stride;
  int32_t n_rows, vocab;
  const float* uniforms;        /* [n_rows] in [0, 1) (others are clamped) */
  const float* temperature;     /* [n_rows]; 0 (or below, NaN): the largest logit; NULL: 1 */
  const int32_t* top_k;         /* [n_rows]; 0 (or below) or NULL: off; up to vocab */
  const float* top_p;           /* [n_rows]; 1 (or above, NaN) or NULL: off */
  const float* min_p;           /* [n_rows]; 0 (or below, NaN) or NULL: off */
  int32_t* tokens;              /* [n_rows] out */
  float* probs;                 /* [n_rows] out: what the token was drawn with, or NULL */
} llm_sample_args;

/* The next token of every row, under options of its own, read on the device. In
 * the order of llm_set_sampling (the largest logit first, ties by id) the options
 * keep, of p = softmax(logit / temperature): the first top_k tokens; of those the
 * shortest prefix whose mass reaches top_p of theirs; of those the ones with p >=
 * min_p times the largest p. The token is the first whose cumulative probability
 * exceeds uniforms[r] times the kept ones' total, as llm_set_sampling chooses it from
 * the same draw; probs[r] is its share of that total. Borders are decided with
 * 64-bit sums of weights of 34 bits, 28 below 1/16 of the largest: with errors of either
 * sign a border is off by 2^-34 of the row's mass, by 2^-28 at most (thousands of equal
 * logits below 1/16). A NaN logit counts as -inf, +inf as the
 * largest finite value; a row without a finite logit gives -1. The same call gives
 * the same tokens every time; a row in another batch gives the same one, but for
 * borders that lie within those sums' last bits. Rows with thousands of logits around a
 * border (untrained ones, high temperatures) take up to three times as long. Rows with
 * crowds of equal logits around it take 8 to 25 times (151936 equal ones 0.17 ms, 256 rows
 * of them 2.9 ms), rows whose largest logit is 22713 temperatures or more from 0 (20 at a
 * temperature of 0.00088) 4 to 12 times (0.09 and 1.5 ms; a temperature of 0 takes the
 * usual time). UNSUPPORTED: vocab over 524288. */
int llm_sample_tokens(const llm_sample_args* args, void* cuda_stream);

#ifdef __cplusplus
}
#endif
#endif /* LLMQ_H */
