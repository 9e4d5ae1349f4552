/*
 * msk.h - C ABI of the persistent MoE verify-step kernel library (libmsk.so).
 *
 * One call of msk_decode_step runs the verify pass of a speculative decode
 * step at batch size one: T (<= 16) tokens through every decoder layer of a
 * sliding-window / global-attention mixture-of-experts transformer, one
 * persistent kernel launch per layer.  Sources, by page title and section:
 *   [newruntime] "Muse Spark Open Ultrafast: Pushing beyond 1,000 Tokens per
 *                second" (newruntime.com), "What happened": 62 decoder
 *                layers (46 sliding-window over the previous 2,048 tokens,
 *                16 global), 8 of 256 experts per token, NVFP4 experts with
 *                some layers in bf16, 16 tokens verified in one pass.
 *   [orcarouter] "Muse Spark Open: 1.109 token al secondo sono un cambiamento
 *                di kernel, non un cambiamento di modello" (orcarouter.ai),
 *                "Dove si colloca il confine del kernel": each launch covers
 *                one layer's attention through the next layer's QKV
 *                projection and KV write; a pooler shrinks each token vector
 *                before the experts and an unpooler restores it; fp4 after
 *                the first expert GEMM, bf16 after the second.
 *   [ai4snews]   "Muse Spark Open decoding passes 1,000 tokens per second..."
 *                (ai4snews.wisdomeyes.cn), "Interpretation": speculative L2
 *                prefetch of the 14 experts the previous step used most.
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers unless a comment says host.
 *   - The caller owns every buffer it passes.  The library copies what it
 *     needs from weights during msk_load_layer (repacking them into its own
 *     device memory); caller weight buffers may be freed after that call.
 *   - Work is enqueued on the given stream.  msk_layer_step and
 *     msk_decode_step synchronise that stream before returning, to read the
 *     device error word; they return MSK_ERR_TIMEOUT if a bounded device
 *     wait ran out (the device context stays usable and the next call
 *     re-initialises the device synchronisation state).  With the
 *     environment variable MSK_VERBOSE_ERRORS set, the device error word
 *     (code, phase, block) is also printed to stderr.
 *   - No C++ exception crosses this boundary.  A model is not thread-safe;
 *     use one model per host thread / stream.
 *   - Requires an sm_103 device (GB300); otherwise MSK_ERR_UNSUPPORTED_DEVICE.
 */
#ifndef MSK_H_
#define MSK_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MSK_OK = 0,
  MSK_ERR_INVALID_ARG = 1,      /* null pointer, bad index, inconsistent sizes */
  MSK_ERR_SHAPE = 2,            /* a dimension the kernels do not support */
  MSK_ERR_ALIGNMENT = 3,        /* a pointer or stride not 16-byte aligned */
  MSK_ERR_BAD_SCALE = 4,        /* an E4M3 block scale is NaN or negative */
  MSK_ERR_UNSUPPORTED_DEVICE = 5,
  MSK_ERR_OOM = 6,
  MSK_ERR_CUDA = 7,             /* a CUDA runtime call failed */
  MSK_ERR_TIMEOUT = 8,          /* a device wait exceeded its time budget */
  MSK_ERR_NOT_LOADED = 9        /* a layer's weights were never loaded */
} msk_status;

typedef struct msk_model msk_model; /* opaque, library-owned */

/* Model configuration.  Supported: hidden, pooled and inter multiples of 128;
 * head_dim 64 or 128; n_q_heads a multiple of n_kv_heads with
 * (n_q_heads / n_kv_heads) * verify_tokens <= 64; verify_tokens <= 16;
 * top_k <= 8; n_experts <= 256 (a multiple of 8); pooled, inter <= 2048;
 * hidden <= 4096.
 * Anything else: msk_create returns MSK_ERR_SHAPE. */
typedef struct {
  int32_t n_layers;
  int32_t hidden;          /* D */
  int32_t n_q_heads;       /* Hq */
  int32_t n_kv_heads;      /* Hkv; query head h reads kv head h / (Hq/Hkv) */
  int32_t head_dim;        /* d */
  int32_t pooled;          /* P: pooler output width, expert input width */
  int32_t n_experts;       /* E */
  int32_t top_k;           /* k */
  int32_t inter;           /* I: expert intermediate width */
  int32_t verify_tokens;   /* T */
  int32_t max_seq;         /* KV cache capacity per layer */
  int32_t prefetch_experts; /* experts prefetched into L2 per layer (14) */
  const uint8_t* layer_is_global; /* HOST [n_layers]: 1 global, 0 sliding */
  int32_t window;          /* sliding window W: keys [p - W + 1, p] */
  float rms_eps;           /* RMSNorm epsilon (1e-6) */
  float rope_theta;        /* RoPE base (1e6) */
  uint64_t wait_budget_ns; /* bound on every device-side wait; 0 = 200 ms */
} msk_model_config;

/* A bf16 matrix [rows][cols], row-major; ld_elems = elements between rows
 * (>= cols, a multiple of 8; 0 means cols). */
typedef struct {
  const void* data;
  int64_t rows, cols, ld_elems;
} msk_bf16_desc;

/* An NVFP4 matrix [rows][cols] (cols a multiple of 128, unless a call says otherwise):
 *   packed: [rows][cols/2] bytes, element 2i in the low nibble of byte i,
 *           element 2i+1 in the high nibble; E2M1 codes (bit 3 = sign);
 *   scales: [rows][cols/16] E4M3 codes, one per 16 consecutive elements
 *           along a row (sign bit must be 0, NaN codes are rejected);
 *   tensor_scale: fp32 multiplier of the whole matrix.
 * Value w[r][c] = fp32(e2m1 * e4m3) * tensor_scale. */
typedef struct {
  const uint8_t* packed;
  const uint8_t* scales;
  float tensor_scale;
  int64_t rows, cols;
} msk_nvfp4_desc;

/* One layer's weights.  Dense weights are [out][in] (K-major).
 *   attn_norm, moe_norm : [1][hidden] RMSNorm gains;
 *   w_qkv   : [(Hq + 2 Hkv) d][hidden], rows [q heads | k heads | v heads];
 *   w_o     : [hidden][Hq d];  w_pool : [pooled][hidden];
 *   w_router: [n_experts][pooled];  router_bias : fp32 [n_experts];
 *   w_unpool: [hidden][pooled];
 *   w_gate, w_up : HOST arrays [n_experts] of [inter][pooled] NVFP4;
 *   w_down  : HOST array [n_experts] of [pooled][inter] NVFP4. */
typedef struct {
  msk_bf16_desc attn_norm, moe_norm, w_qkv, w_o, w_pool, w_unpool, w_router;
  const float* router_bias;
  const msk_nvfp4_desc* w_gate;
  const msk_nvfp4_desc* w_up;
  const msk_nvfp4_desc* w_down;
} msk_layer_weights;

/* Creates a model: validates the configuration, checks the device, and
 * allocates the library's scratch (activations between phases, attention
 * partials, synchronisation words).  *out is NULL on failure. */
msk_status msk_create(const msk_model_config* cfg, msk_model** out);

/* Copies layer `layer`'s weights into the library's tiled layouts on the
 * device: dense rows in mma-fragment order, expert codes and block scales
 * interleaved per 16-row unit.  Validates shapes, 16-byte alignment and every
 * E4M3 block scale (MSK_ERR_BAD_SCALE).  Synchronises `stream`.  Loading a
 * layer again replaces it. */
msk_status msk_load_layer(msk_model* m, int32_t layer, const msk_layer_weights* w,
                          void* stream /* cudaStream_t */);

/* Runs ONE persistent launch: attention(layer) .. MoE(layer) .. and, unless
 * `layer` is the last, QKV(layer + 1) with its KV write.
 *   hidden     : [T][hidden] bf16, in: the layer input h; out: h2.
 *   kv_cache   : [n_layers][2 (K, V)][n_kv_heads][max_seq][head_dim] bf16;
 *                K is stored after RoPE.  Rows at the verify positions of
 *                layer `layer` must already be written (by the previous
 *                launch, or by run_prologue on this one).
 *   positions  : HOST [T], positions[t] == positions[0] + t, the last one
 *                < max_seq.  The cached length is positions[0].
 *   prev_routing: [T][top_k] int32 experts this layer chose in the previous
 *                step, or NULL (no speculative prefetch).  Only moves data
 *                into L2: results never depend on it.
 *   routing_out: [T][top_k] int32, or NULL.  Rank order: logit descending,
 *                index ascending on ties.
 *   run_prologue: nonzero = first compute layer `layer`'s own QKV and KV
 *                write from `hidden` (what the previous launch would have
 *                done).
 * The query vectors of the next layer are kept inside the model between
 * calls.  Returns after the stream has completed the launch. */
msk_status msk_layer_step(msk_model* m, int32_t layer, void* hidden, void* kv_cache,
                          const int32_t* positions, const int32_t* prev_routing,
                          int32_t* routing_out, int32_t run_prologue, void* stream);

/* The whole verify step: the prologue of layer 0, then one launch per layer.
 *   prev_routing: [n_layers][T][top_k] int32 or NULL; routing_out:
 *   [n_layers][T][top_k] int32 or NULL.  hidden holds the last layer's h2
 *   (no final norm) on return; the KV rows of every layer are written at
 *   the verify positions. */
msk_status msk_decode_step(msk_model* m, void* hidden, void* kv_cache, const int32_t* positions,
                           const int32_t* prev_routing, int32_t* routing_out, void* stream);

/* The same two calls for a TREE of candidate tokens instead of a chain
 * ([orcarouter] on the draft: the verified block is a tree of candidates
 * generated by the draft model, not a linear chain).
 *   cache_len : S, the number of cached tokens (every position < S holds a
 *               K/V row); S + T <= max_seq.
 *   parents   : HOST [T]; parents[t] is the verify slot of t's parent, an
 *               earlier slot (0 <= parents[t] < t), or -1 for a child of the
 *               last cached token.  parents[t] == t - 1 for every t is the
 *               chain, i.e. msk_layer_step / msk_decode_step with
 *               positions S + t.
 * Slot t has position S + depth(t) (depth = number of verify ancestors),
 * which sets its RoPE angle and its sliding window; its K/V rows are
 * written at cache row S + t (slot order, so that the caller can compact
 * the accepted path afterwards); it attends to the cached keys inside its
 * window and to the verify rows of its ancestors and itself (those whose
 * positions fall inside its window).  MSK_ERR_INVALID_ARG for a parent out
 * of range or S out of range. */
msk_status msk_layer_step_tree(msk_model* m, int32_t layer, void* hidden, void* kv_cache, int32_t cache_len,
                               const int32_t* parents, const int32_t* prev_routing, int32_t* routing_out,
                               int32_t run_prologue, void* stream);
msk_status msk_decode_step_tree(msk_model* m, void* hidden, void* kv_cache, int32_t cache_len,
                                const int32_t* parents, const int32_t* prev_routing, int32_t* routing_out,
                                void* stream);

/* The whole step as one CUDA graph.  The pages run the draft, the verify
 * and the accept of a decode step as one CUDA graph with 97 launches
 * ([newruntime] "What happened"; the plugin's README in [orcarouter]); this
 * is the verify part.
 * msk_step_graph_capture records the n_layers launches of a step (as
 * msk_decode_step would enqueue them) into a graph owned by the model, on a
 * stream of the library's own; nothing runs.  The buffers given here are
 * baked into the graph: every replay reads and writes these same `hidden`,
 * `kv_cache`, `prev_routing` ([n_layers][T][top_k] or NULL) and
 * `routing_out` ([n_layers][T][top_k] or NULL).  Capturing again replaces
 * the graph.  Must not be called while another capture is active on the
 * calling thread.
 * msk_step_graph_launch replays it for one step on `stream`: the cached
 * length `cache_len` and the candidate tree `parents` (HOST [T], as in
 * msk_decode_step_tree; NULL = the chain) are copied to a small device
 * record that every launch reads at its start, so one graph serves every
 * step.  Results are bit-identical to msk_decode_step_tree /
 * msk_decode_step with the same inputs.  Synchronises `stream`; returns
 * MSK_ERR_NOT_LOADED if nothing was captured, MSK_ERR_INVALID_ARG for a bad
 * cache_len or tree.  Launch timing and the phase timeline are not recorded
 * for replays. */
msk_status msk_step_graph_capture(msk_model* m, void* hidden, void* kv_cache, const int32_t* prev_routing,
                                  int32_t* routing_out);
msk_status msk_step_graph_launch(msk_model* m, int32_t cache_len, const int32_t* parents, void* stream);

/* Per-phase device timestamps (%globaltimer, ns) of the most recent call,
 * recorded only while timing is enabled (msk_set_timing).  Layout:
 * [launches][ctas][MSK_TIMELINE_SLOTS], launches in the call's order (one
 * launch, of the layer given, after msk_layer_step); *n receives the number
 * of uint64 written (at most cap). */
#define MSK_TIMELINE_SLOTS 64
msk_status msk_set_timing(msk_model* m, int32_t enable);
msk_status msk_get_timeline(msk_model* m, uint64_t* host_out, size_t cap, size_t* n,
                            int32_t* n_launches, int32_t* n_ctas);

/* Per-launch device durations.  While enabled, msk_layer_step and
 * msk_decode_step record a CUDA event pair on the call's stream around
 * every layer launch; msk_get_launch_ms returns the durations (ms) of the
 * most recent call's launches, in launch order (*n = number written). */
msk_status msk_set_launch_timing(msk_model* m, int32_t enable);
msk_status msk_get_launch_ms(msk_model* m, float* host_out, int32_t cap, int32_t* n);

/* Test hooks (not needed in production).
 * msk_set_wait_budget: device wait bound in ns (0 restores the default).
 * msk_set_fault_injection: CTA `cta` skips its arrival at grid barrier number
 *   `barrier` (counted from 1 within a launch) of every launch; -1 disables.
 *   Used to check that a missing producer ends in MSK_ERR_TIMEOUT. */
msk_status msk_set_wait_budget(msk_model* m, uint64_t ns);
msk_status msk_set_fault_injection(msk_model* m, int32_t barrier, int32_t cta);

/* Copies an intermediate of the most recent launch (device to device) for
 * tests: 0 q stash [T][Hq][d] bf16, 1 attention output [T][Hq d] bf16,
 * 2 h1 [T][D] bf16, 3 pooled [T][P] bf16, 4 router logits [T][E] fp32,
 * 5 fp4 intermediate codes [T k][I/2] (E2M1, element 2i in the low nibble
 * of byte i), 6 its E4M3 scales [T k][I/16],
 * 7 expert outputs [T k][P] bf16 (slot t*k + r), 8 combined expert output
 * [T][P] bf16, 9 the experts ranked for the speculative L2 prefetch [33]
 * int32 (count n, then n expert ids, most used in prev_routing first).  Copies min(bytes, size of the buffer); *copied = that. */
msk_status msk_debug_scratch(msk_model* m, int32_t which, void* dst, size_t bytes, size_t* copied,
                             void* stream);

/* Dequantises expert `expert`'s matrix `which` (0 gate, 1 up, 2 down) of a
 * loaded layer by reading the library's repacked layout, into out
 * ([rows][cols] fp32, device).  Bit-exact with fp32(e2m1*e4m3)*tensor_scale. */
msk_status msk_debug_dequant(msk_model* m, int32_t layer, int32_t expert, int32_t which,
                             float* out, void* stream);

/* Test hook: the E2M1 code (round-to-nearest-even, saturating; sign bit
 * kept for negative values that round to zero) and the E4M3 code (same rules)
 * of each of the n DEVICE floats in x, written to the DEVICE byte arrays e2m1
 * and e4m3, through the very conversion routines the kernels use for the
 * activation quantiser.  Synchronises `stream`. */
msk_status msk_debug_convert(const float* x, int64_t n, uint8_t* e2m1, uint8_t* e4m3, void* stream);

/* Runs the kernel's activation quantiser on x ([rows][cols] fp32, cols a
 * multiple of 16, device): writes E2M1 codes (one per byte) to codes
 * [rows][cols] and E4M3 scales to scales [rows][cols/16].  Standalone (no
 * model). */
msk_status msk_debug_quantize(const float* x, int64_t rows, int64_t cols, uint8_t* codes,
                              uint8_t* scales, void* stream);

/* Test hook: one block-scaled NVFP4 tile on the tensor cores (tcgen05
 * kind::mxf4nvf4, the instruction the expert GEMMs use), through the same
 * shared-memory operand layouts and scale-factor placement as the layer
 * kernel:  d[128][16] = A[128][K] * B[b_rows][K]^T in fp32, rows of B past
 * b_rows taken as zero.
 *   a_codes : [128][K/2] E2M1 codes, element 2i in the low nibble of byte i;
 *   a_scales: [128][K/16] E4M3 block scales (one per 16 elements of K);
 *   b_codes, b_scales: the same for B's b_rows (1..16) rows;
 *   K: 128..2048, a multiple of 128; d: [128][16] fp32.  All DEVICE.
 * Value of an element: e2m1 * e4m3 (no tensor scale).  Allocates a 4-byte
 * error word; synchronises `stream`. */
msk_status msk_debug_fp4_gemm(const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* b_codes,
                              const uint8_t* b_scales, int32_t b_rows, int32_t K, float* d, void* stream);

/* Split-KV GQA attention of one layer (the layer kernel's attention stage)
 * as a standalone call that allocates no device memory.  The pages describe
 * no such call: it is here for callers that cannot allocate when they need
 * attention, e.g. code drawing all device memory from a serving framework's
 * pre-sized pool, or code that must not allocate while work is being
 * recorded for later replay.
 *   q        : [tokens][n_q_heads][head_dim] bf16, rotated queries;
 *   kv_layer : [2 (K, V)][n_kv_heads][max_seq][head_dim] bf16, one layer's
 *              cache, keys after RoPE, rows up to pos0 + tokens - 1 written;
 *   window   : 0 for global attention, else keys [p - window + 1, p];
 *   out      : [tokens][n_q_heads * head_dim] bf16.
 * Token t sits at position pos0 + t and sees keys up to its own position.
 * Supported: head_dim 64 or 128, tokens <= 16, (n_q_heads / n_kv_heads) *
 * tokens <= 64, n_q_heads * head_dim <= 4096, n_kv_heads <= the device's SM
 * count (each kv head needs at least one block); else MSK_ERR_SHAPE.
 * Scratch (per-block partial results and synchronisation words) lives in
 * one fixed 6 MiB array inside the library on every GPU that loads it, kept
 * until the process exits; a call whose shape needs more (SM count * 64 *
 * (head_dim + 2) * 4 bytes + 512) returns MSK_ERR_SHAPE.  The first call on
 * a device looks up that array's device address and sets the kernels'
 * shared-memory limit (guarded by a mutex, so first calls from several host
 * threads are safe).  All calls share the array: calls that overlap on the
 * GPU race, so serialise them.  The synchronisation words are cleared at the
 * start of every call.  The call synchronises `stream` before returning (to
 * read the device error word: MSK_ERR_TIMEOUT if a device wait ran out), so
 * it cannot run while `stream` is being captured into a CUDA graph. */
msk_status msk_attention_noalloc(const void* q, const void* kv_layer, int32_t tokens, int32_t n_q_heads,
                                 int32_t n_kv_heads, int32_t head_dim, int32_t max_seq, int32_t pos0,
                                 int32_t window, void* out, void* stream);

/* ---------------------------------------------------------------------------
 * Operators around the step, each a call of its own on the caller's buffers:
 * a KV cache held in 4 bits, products with 4-bit weights, and the log
 * probabilities that accept or reject the verified tokens.  The pages
 * describe none of them; they serve the same batch-one verify pass.
 *
 * They differ from the step's calls in three ways: they take no model, they
 * ENQUEUE their work on `stream` and return without waiting for it, and they
 * may be captured into a CUDA graph.  They keep nothing between calls but the
 * record of a device wait that ran out (msk_ops_check).  Where a call
 * takes a workspace, the caller owns it: calls that may overlap on the GPU
 * (two streams, two graphs) need one each.  Its contents are of no meaning
 * before or after a call.
 * The device must be the current one of the calling thread. */
typedef enum { MSK_BF16 = 0, MSK_FP16 = 1, MSK_FP32 = 2 } msk_dtype;

/* One layer's KV cache in the step's order, NVFP4:
 *   codes : [2 (K, V)][n_kv_heads][max_seq][head_dim / 2] E2M1 codes, element
 *           2i in the low nibble of byte i;
 *   scales: [2][n_kv_heads][max_seq][head_dim / 16] E4M3 block scales.
 * Value = e2m1 * e4m3 * k_scale (keys) or v_scale (values); both positive.
 * Both pointers 16-byte aligned; head_dim 64 or 128; max_seq up to 2^30. */
typedef struct {
  uint8_t* codes;
  uint8_t* scales;
  int32_t n_kv_heads, head_dim, max_seq;
  float k_scale, v_scale;
} msk_kv4_desc;

/* Quantises `tokens` rows of K and V into cache rows pos0 .. pos0 + tokens - 1.
 *   k, v: element (t, h, i) at t * token_stride + h * head_stride + i, of type
 *         dtype (any of the three): rows of a QKV projection and layers of the
 *         bf16 cache alike.  Rows and strides are multiples of 16 bytes.
 *   pos0_dev: NULL, or a DEVICE int32 that is read instead of pos0 when the
 *         kernel runs (for graphs); clamped to [0, max_seq - tokens].
 * The activation quantiser of the step (see msk_debug_quantize) on
 * fp32(x / k_scale): block scale E4M3_RN(amax / 6), codes E2M1_RN(x / scale).
 * A value beyond 2688 * k_scale saturates; an infinity counts as such a
 * value; a NaN does not count for its block's scale and is stored as 6 times
 * it.  tokens == 0 does nothing. */
msk_status msk_kv4_write(const msk_kv4_desc* cache, const void* k, const void* v, int32_t dtype, int32_t tokens,
                         int64_t token_stride, int64_t head_stride, int32_t pos0, const int32_t* pos0_dev,
                         void* stream);

/* The reverse: rows pos0 .. pos0 + tokens - 1 of the cache as values of type
 * dtype (exact in bf16 and fp16 where the tensor's scale is 1, else rounded
 * once), to k and v laid out as above; their rows must not overlap (a stride
 * of 0 is refused). */
msk_status msk_kv4_read(const msk_kv4_desc* cache, int32_t pos0, int32_t tokens, void* k, void* v, int32_t dtype,
                        int64_t token_stride, int64_t head_stride, void* stream);

/* GQA attention of `tokens` (1..16) queries over a 4-bit cache: what
 * msk_attention_noalloc computes, and its tree form.
 *   q      : element (t, h, i) at t * q_stride + h * head_dim + i, bf16 or
 *            fp16, after RoPE; q_stride a multiple of 8, 16-byte aligned;
 *   out    : [tokens][n_q_heads * head_dim], the type of q, 16-byte aligned;
 *   cache_len: S, cached rows; the tokens' own K/V sit at rows S + t, written
 *            before; S + tokens <= max_seq;
 *   cache_len_dev: NULL, or a DEVICE int32 that is read instead of cache_len
 *            when the kernels run (for graphs); clamped to
 *            [0, max_seq - tokens].  The call is then laid out for the
 *            longest length, which costs a short one 1 to 3 us;
 *   parents: HOST [tokens] as in msk_decode_step_tree, or NULL for the chain
 *            (read during the call, so a graph keeps the tree it was captured
 *            with);
 *   window : 0 for global attention, else keys [p - window + 1, p];
 *   softmax_scale: factor of the scores, 0 for 1 / sqrt(head_dim); with k_scale
 *            and log2(e) a finite fp32 number.
 * n_q_heads a multiple of cache->n_kv_heads, any quotient.  Cache rows that no
 * query sees are not read, or do not count whatever they hold.
 * Queries enter the products in fp16 after a scaling of each row by a power of
 * two (elements above 2^-31 of the row's greatest without rounding, smaller ones
 * off by at most 2^-39 of it), softmax weights as two fp16 numbers (22 bits, below
 * that 2^-32 of a row's greatest), keys and values without rounding; sums are fp32.
 * workspace: at least msk_attention_kv4_workspace bytes (0 for few keys, when
 * it may be NULL), 16-byte aligned; for a call with cache_len_dev the bytes for
 * max_seq - tokens. */
size_t msk_attention_kv4_workspace(int32_t tokens, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                                   int32_t window, int32_t cache_len);
msk_status msk_attention_kv4(const void* q, int32_t dtype, int64_t q_stride, const msk_kv4_desc* cache,
                             int32_t tokens, int32_t n_q_heads, int32_t cache_len, const int32_t* cache_len_dev,
                             const int32_t* parents, int32_t window, float softmax_scale, void* out,
                             void* workspace, size_t workspace_bytes, void* stream);

/* y[t][n] = sum_k x[t][k] w[n][k] for `tokens` (1..16) rows: a projection or
 * vocabulary head whose weights are NVFP4 and whose activations are not
 * quantised.
 *   x: [tokens][cols], bf16 or fp16, x_stride elements between rows (a
 *      multiple of 8), 16-byte aligned;
 *   w: rows arbitrary, cols a multiple of 128 up to 32768, codes and scales
 *      16-byte aligned, read where they are (no repacking);
 *   y: [tokens][rows] of y_dtype (bf16, fp16 or fp32), y_stride elements
 *      between rows, aligned to its element.
 * Weights enter without rounding (the products e2m1 * e4m3), x in fp16 after a
 * scaling of each row by a power of two (elements above 2^-31 of the row's
 * greatest without rounding, smaller ones off by at most 2^-39 of it), sums are
 * fp32.  A NaN block scale makes the
 * outputs of its row NaN.  tokens == 0 or rows == 0 does nothing. */
msk_status msk_linear_fp4(const void* x, int32_t x_dtype, int64_t x_stride, const msk_nvfp4_desc* w, int32_t tokens,
                          void* y, int32_t y_dtype, int64_t y_stride, void* stream);

/* Synchronises `stream` (so not under capture) and tells whether a bounded
 * device wait of these operators ran out on the current device since the last
 * call of this function: MSK_ERR_TIMEOUT (the outputs of the calls since then are
 * not to be used), else MSK_OK.  Such waits are in msk_linear_fp4, in
 * msk_experts_fp4 and in msk_attention_kv4 for more than 16 query rows of a kv
 * head; the other kernels
 * wait for nothing that may stay away.  There is one record for a device: a check
 * clears it, and takes note of other threads' and streams' calls too, so of several
 * users of a device one has to check for all. */
msk_status msk_ops_check(void* stream);

/* Log probabilities under softmax(logits / temperature), one pass per row:
 *   logits : [rows][vocab] of dtype (any of the three), ld elements between
 *            rows (>= vocab, no alignment asked beyond the element's);
 *   tokens : int32 [rows] given tokens, or NULL (then logprob and rank are
 *            NULL too).  A token outside [0, vocab) marks a padded row: its
 *            logprob is 0 and its rank -1;
 *   temperature: 1e-30 to 1e30;
 *   logprob: fp32 [rows], log softmax at the given token;
 *   rank   : int32 [rows], how many logits are greater than the given one;
 *   entropy: fp32 [rows], in nats;
 *   top    : 0..32 alternatives (at most vocab): top_ids int32 [rows][top] and
 *            top_logprobs fp32 [rows][top], greatest first, of equal logits
 *            the lowest index first.
 * Any output may be NULL.  Logits of -inf are barred tokens (probability 0).
 * A row with a NaN or +inf, or with nothing but -inf, has no distribution: its
 * logprob, entropy and top_logprobs are NaN, its ids in range.
 * rows == 0 does nothing. */
msk_status msk_token_logprobs(const void* logits, int32_t dtype, int64_t rows, int64_t vocab, int64_t ld,
                              const int32_t* tokens, float temperature, int32_t top, float* logprob, int32_t* rank,
                              float* entropy, int32_t* top_ids, float* top_logprobs, void* stream);

/* ---------------------------------------------------------------------------
 * The experts of a whole prompt: what the step does for 16 tokens inside its
 * launch, as operators for any number.  In the order of their use:
 *   msk_moe_route     router logits -> each token's experts and gates
 *   msk_moe_sort      the tokens' slots by expert
 *   msk_quantize_fp4  rows to 4 bits (as the step quantises activations)
 *   msk_experts_fp4   gate and up projections with SwiGLU; once more for the
 *                     down projection, on rows quantised again
 *   msk_moe_combine   outputs back at their tokens, weighted and summed
 * A token's slots are its experts by rank: slot = token * top_k + rank.  The
 * slots in sorted order are at places 0, 1, ...  The conventions are those of
 * the operators above: calls enqueue on `stream` and return, may be captured,
 * and keep nothing between calls; none takes a workspace.
 * Experts' weights are the caller's, row-major as msk_load_layer is given them.  The
 * model's own copy is laid out for the step and serves the step alone: a program that
 * verifies and sends prompts through the same experts keeps both, 9/16 of a byte for
 * each weight once more (256 experts of 3 x 1024 x 2048: 0.9 GB a layer). */

/* The step's router on any number of tokens: x = fp32(logits) + bias, the
 * top_k greatest, of equal ones the lowest index first, and their softmax.
 *   logits : [tokens][n_experts] of dtype (any of the three), ld elements
 *            between rows (>= n_experts, no alignment asked beyond the element's);
 *   bias   : fp32 [n_experts] or NULL;
 *   experts: int32 [tokens][top_k], gates: fp32 [tokens][top_k], by rank.
 * n_experts up to 1024, top_k up to 32 and n_experts.  An x of -inf or NaN is a
 * barred expert; where fewer than top_k are left the ranks behind them get expert
 * -1 and gate 0.  A token with an x of +inf has gates of NaN.  tokens == 0 does
 * nothing. */
msk_status msk_moe_route(const void* logits, int32_t dtype, int64_t tokens, int32_t n_experts, int64_t ld,
                         const float* bias, int32_t top_k, int32_t* experts, float* gates, void* stream);

/* Sorts n slots by expert, within an expert by slot.
 *   experts: int32 [n]; one outside [0, n_experts) (-1, say) drops its slot;
 *   offsets: int32 [n_experts + 1]: expert e has places offsets[e] ..
 *            offsets[e + 1] - 1;
 *   slots  : int32 [n]: the slot at a place, -1 from offsets[n_experts] on;
 *   places : int32 [n]: the place of a slot, -1 for a dropped one.
 * n_experts up to 1024, n up to 2^30.  n == 0 writes offsets of 0. */
msk_status msk_moe_sort(const int32_t* experts, int64_t n, int32_t n_experts, int32_t* offsets, int32_t* slots,
                        int32_t* places, void* stream);

/* Rows to 4 bits: x ([rows][cols] of dtype, any of the three, x_stride elements
 * between rows) to codes [rows][cols / 2] and scales [rows][cols / 16] as in
 * msk_nvfp4_desc.  The activation quantiser of the step (see msk_debug_quantize)
 * on fp32(x / tensor_scale); what msk_kv4_write says of values that saturate, of
 * infinities and of NaN holds here too.  cols a multiple of 16 up to 2^24; x,
 * its rows, codes and scales 16-byte aligned; tensor_scale positive.  rows == 0
 * does nothing. */
msk_status msk_quantize_fp4(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t x_stride,
                            float tensor_scale, uint8_t* codes, uint8_t* scales, void* stream);

/* The reverse: values of type dtype (exact in bf16 and fp16 where tensor_scale is
 * 1, else rounded once behind fp32) into rows of x, which must not overlap. */
msk_status msk_dequantize_fp4(const uint8_t* codes, const uint8_t* scales, float tensor_scale, int64_t rows,
                              int64_t cols, void* x, int32_t dtype, int64_t x_stride, void* stream);

/* One matrix of each expert, all of one size: packed [n_experts][rows][cols / 2],
 * scales [n_experts][rows][cols / 16] as in msk_nvfp4_desc (16-byte aligned, read
 * where they are), tensor_scales: DEVICE fp32 [n_experts], or NULL for 1. */
typedef struct {
  const uint8_t* packed;
  const uint8_t* scales;
  const float* tensor_scales;
  int32_t n_experts;
  int64_t rows, cols;
  const void* maps; /* NULL, or what msk_fp4_experts_maps has made of these weights (HOST) */
} msk_fp4_experts;

/* The copy engine's descriptors of the weights, which msk_experts_fp4 makes anew at
 * every call that is not given them (0.13 us each, two a matrix): into
 * MSK_FP4_MAPS_BYTES of HOST memory, 128-byte aligned, that the caller keeps with
 * the weights.  w->maps is not read.  They hold for these addresses and sizes: a
 * call with others in the struct beside them is MSK_ERR_INVALID_ARG. */
#define MSK_FP4_MAPS_BYTES 384
msk_status msk_fp4_experts_maps(const msk_fp4_experts* w, void* maps);

/* Products of quantised rows with their experts' weights: for every place p of
 * expert e
 *   y[p][i] = sum_j x[row(p)][j] w[e][i][j],  or with `up`
 *   y[p][i] = silu(sum_j x[row(p)][j] w[e][i][j]) * sum_j x[row(p)][j] up[e][i][j].
 *   x      : quantised rows (both 4-bit operands enter the tensor cores as they
 *            are; sums are fp32); x->rows any number, 16-byte aligned;
 *   slots  : NULL: row(p) = p; else int32 [n] as from msk_moe_sort:
 *            row(p) = slots[p] / top_k, so that a token's row is read where it
 *            is by all of its experts (rows outside x are taken as its nearest);
 *   n      : number of places, x->rows at most where slots is NULL;
 *   offsets: DEVICE int32 [n_experts + 1], ascending, as from msk_moe_sort;
 *            what goes beyond [0, n] or back is cut off;
 *   up     : NULL, or weights of w's size;
 *   y      : [n][w->rows] of y_dtype (any of the three), y_stride elements between
 *            rows, aligned to its element; places of no expert are left as
 *            they were.
 * One expert (offsets {0, n}) is a plain product.  cols a multiple of 64, 64 to
 * 131072; n_experts up to 1024, rows up to 2^24, n_experts * rows below 2^31 - 256;
 * n up to 2^30.  A NaN block scale makes its row's outputs NaN.  silu is off by some
 * 2^-21 of its value, and 0 for a gate below some -87.3 (where it is under 2^-119 in
 * magnitude).  Any tensor scales: results in fp32's range are not lost to products of
 * scales out of it.  n == 0 or rows == 0 does nothing.  Waits on the device are
 * bounded: see msk_ops_check. */
msk_status msk_experts_fp4(const msk_nvfp4_desc* x, const int32_t* slots, int32_t top_k, int64_t n,
                           const int32_t* offsets, const msk_fp4_experts* w, const msk_fp4_experts* up, void* y,
                           int32_t y_dtype, int64_t y_stride, void* stream);

/* Test hook (not needed in production), for the calls of msk_experts_fp4 that follow in
 * this process: of tile number `tile` of each pair of blocks (0 its first; -1: of none)
 * nobody is told that its sums are complete, and waits are bounded by wait_ns (up to 200
 * ms; 0: these) and the time for each step.  Used to check that a signal which stays away
 * ends in MSK_ERR_TIMEOUT from msk_ops_check; what such calls write is not to be used. */
msk_status msk_debug_experts_fault(int32_t tile, uint64_t wait_ns);

/* out[t] = sum over ranks r of gates[t][r] * y[places[t][r]], in order of rank, in
 * fp32, rounded once.
 *   y     : [y_rows][cols] of y_dtype, y_stride elements between rows;
 *   places: int32 [tokens][top_k] as from msk_moe_sort; one outside [0, y_rows)
 *           is a dropped slot: nothing of it is read;
 *   gates : fp32 [tokens][top_k], or NULL for 1;
 *   out   : [tokens][cols] of out_dtype, out_stride elements between rows.
 * Everything aligned to its element (rows of 16-byte pieces are faster).
 * tokens == 0 or cols == 0 does nothing. */
msk_status msk_moe_combine(const void* y, int32_t y_dtype, int64_t y_rows, int64_t y_stride, const int32_t* places,
                           const float* gates, int64_t tokens, int32_t top_k, int64_t cols, void* out,
                           int32_t out_dtype, int64_t out_stride, void* stream);

/* Number of SMs (= CTAs per launch) the model uses, and bytes of device
 * memory it owns. */
msk_status msk_get_info(msk_model* m, int32_t* n_ctas, int64_t* device_bytes);

const char* msk_status_string(msk_status s);
void msk_destroy(msk_model* m);

#ifdef __cplusplus
}
#endif
#endif /* MSK_H_ */
