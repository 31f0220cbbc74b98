/*
 * mk.h -- C ABI of the GB300 persistent MoE decode-layer library (libmk.so).
 *
 * One call runs the batch-1 speculative-verify decode step (T <= 16 tokens) of
 * one decoder layer as ONE persistent kernel launch; a stack call chains one
 * launch per layer with programmatic dependent launch.
 *
 * What a launch computes (page "Muse Spark Open: 1,109 Tokens a Second Is a
 * Kernel Change, Not a Model Change", section "Where the kernel boundary sits,
 * and why it stops there"): a layer's attention through the next layer's qkv
 * projection and KV write -- GQA attention over a bf16 KV cache (sliding window
 * of 2,048 tokens or global), o-proj + residual, RMSNorm, router (top-k of E
 * experts), the pooler projection, NVFP4 expert gate/up/down with SiLU, the
 * weighted combine (section "What the 5.9 ms is still spent on"), the
 * unpooler + residual, and optionally the next layer's RMSNorm + QKV
 * projection + KV write.  The first layer of a chain runs its own RMSNorm +
 * QKV + KV write first ("The first and last layers have slightly different
 * operations", same section).  The dense variant (page "LMSYS Details SGLang
 * Megakernel ...", "Key Takeaways": the draft's dense layers, one launch each)
 * replaces router..unpooler with a bf16 SwiGLU MLP.
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers on the device that was current
 *     when the layer was created.  Layouts are row-major, "out x in" for
 *     weights (the input dimension is contiguous), element types as stated.
 *   - Ownership: the caller owns every weight, KV cache, activation and output
 *     buffer and keeps them alive while a layer that uses them exists or a
 *     step is in flight.  Weights are borrowed and never written.  The library
 *     owns and frees its own scratch, counters, repacked scale factors and
 *     status word.
 *   - Errors: every call returns an mk_status; no call aborts, throws or
 *     prints (unless MK_LOG=1 in the environment, at create time).  Argument
 *     and shape errors are reported before anything is launched.  Launch
 *     failures return MK_ERR_CUDA.  Device-side timeouts are reported by
 *     mk_layer_status / mk_stack_status after the caller synchronises.
 *   - Steps are asynchronous on the caller's stream; the library never
 *     synchronises a stream.  One step may be in flight per layer / stack
 *     object at a time.
 */
#ifndef MK_H_
#define MK_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MK_OK = 0,
  MK_ERR_INVALID_ARG = 1,   /* null pointer, bad size, misaligned buffer        */
  MK_ERR_UNSUPPORTED = 2,   /* shape/flag combination not built, wrong GPU arch */
  MK_ERR_CUDA = 3,          /* a CUDA runtime/driver call or launch failed      */
  MK_ERR_OOM = 4,           /* library-owned allocation failed                  */
  MK_ERR_TIMEOUT = 5,       /* a bounded device-side wait expired               */
  MK_ERR_DEVICE_FAULT = 6   /* device reported an inconsistent state            */
} mk_status;

typedef enum {
  MK_FFN_MOE_NVFP4 = 0,           /* router + pooler + NVFP4 experts + unpooler */
  MK_FFN_DENSE_SWIGLU_BF16 = 1    /* bf16 SwiGLU MLP                            */
} mk_ffn_kind;

/* mk_layer_config.flags */
#define MK_FIRST_LAYER   0x1u  /* run RMSNorm + QKV + KV write on x_in first     */
#define MK_FUSE_NEXT_QKV 0x2u  /* end with the next layer's RMSNorm+QKV+KV write;
                                  it projects bf16(x_out * gain) and multiplies
                                  the sum by the RMS factor, so that it can start
                                  per 128-column tile of x_out: the same map as
                                  RMSNorm-then-QKV, with the bf16 rounding of the
                                  normalised input moved                          */
#define MK_TOPK_RENORM   0x4u  /* combine weights renormalised over the top-k    */
#define MK_PREFETCH_NEXT_KV 0x8u /* in a stack (mk_stack_step), fetch the next
                                    layer's old KV rows -- those its verify tokens
                                    will see, when K and V together are at most
                                    16 MB -- into L2 while this layer runs its
                                    last weight phases (page "Muse Spark Open:
                                    1,109 Tokens a Second ...", section "What the
                                    5.9 ms is still spent on": the next layer's
                                    old KV is prefetched into L2 before its launch
                                    lands); ignored by mk_decode_step           */

typedef struct mk_layer_config {
  int32_t hidden;         /* H, a multiple of 256                                */
  int32_t n_q_heads;      /* Hq; must equal 4 * n_kv_heads                        */
  int32_t n_kv_heads;     /* Hkv                                                 */
  int32_t head_dim;       /* d: 64 or 128                                        */
  int32_t window;         /* 0 = global; else key j visible to the query at
                             position p iff j <= p and p - j < window            */
  int32_t ffn_kind;       /* mk_ffn_kind                                         */
  int32_t n_experts;      /* E (MoE), <= 256                                     */
  int32_t top_k;          /* k (MoE), <= 8                                       */
  int32_t pooled_dim;     /* P (MoE): pooler output / expert input, % 128 == 0   */
  int32_t expert_inter;   /* I (MoE): expert intermediate, % 128 == 0            */
  int32_t dense_inter;    /* F (dense): SwiGLU intermediate, % 128 == 0          */
  int32_t max_tokens;     /* <= 16                                               */
  int32_t max_ctx;        /* KV capacity in positions (rows of each cache)       */
  float rms_eps;          /* RMSNorm epsilon; 0 selects 1e-6                      */
  uint32_t flags;         /* MK_FIRST_LAYER | MK_FUSE_NEXT_QKV | MK_TOPK_RENORM
                             | MK_PREFETCH_NEXT_KV                               */
  int32_t prefetch_experts; /* MoE, 0..16: while the router picks this step's
                               experts, the weights of the previous step's N
                               most-used experts are fetched into L2 (page
                               "Muse Spark Open: 1,109 Tokens a Second ...",
                               section "Three bills a kernel this big has to
                               pay": the 14 most-used experts); 0 = off       */
  uint64_t wait_timeout_ns; /* bound on every device-side wait; 0 -> 200 ms      */
} mk_layer_config;

/* Weights: borrowed device pointers, never written.  bf16 unless stated.
 * hidden must be a multiple of 64; Hq*d and every "in" size of a bf16 matrix a
 * multiple of 64; NVFP4 "in" sizes a multiple of 64.                          */
typedef struct mk_layer_weights {
  const void* attn_norm_w;  /* [H]            (MK_FIRST_LAYER only)             */
  const void* w_qkv;        /* [Hq*d + 2*Hkv*d, H] q heads, k heads, v heads     */
  const void* w_o;          /* [H, Hq*d]                                         */
  const void* ffn_norm_w;   /* [H]                                               */
  /* MoE */
  const void* w_router;     /* [E, H]                                            */
  const void* w_pool;       /* [P, H]                                            */
  const void* w_unpool;     /* [H, P]                                            */
  const void* exp_gate_q;   /* uint8 [E, I, P/2]: E2M1 codes, element 2i in the
                               low nibble of byte i, bit 3 = sign               */
  const void* exp_gate_s;   /* uint8 [E, I, P/16]: E4M3 scale per 16 inputs      */
  const float* exp_gate_ts; /* float [E]: tensor scale per expert matrix         */
  const void* exp_up_q;     /* uint8 [E, I, P/2]                                 */
  const void* exp_up_s;     /* uint8 [E, I, P/16]                                */
  const float* exp_up_ts;   /* float [E]                                         */
  const void* exp_down_q;   /* uint8 [E, P, I/2]                                 */
  const void* exp_down_s;   /* uint8 [E, P, I/16]                                */
  const float* exp_down_ts; /* float [E]                                         */
  /* dense */
  const void* w_gate;       /* [F, H]                                            */
  const void* w_up;         /* [F, H]                                            */
  const void* w_down;       /* [H, F]                                            */
  /* MK_FUSE_NEXT_QKV: the next layer's norm gain and QKV weight */
  const void* next_attn_norm_w; /* [H]                                           */
  const void* next_w_qkv;       /* [Hq*d + 2*Hkv*d, H]                           */
} mk_layer_weights;

/* Per-step buffers of a single-layer step (all device pointers). */
typedef struct mk_step_io {
  int32_t n_tokens;       /* T, 1..max_tokens; verify token i sits at ctx + i   */
  int32_t ctx_len;        /* positions [0, ctx) of the caches are valid          */
  const void* x_in;       /* bf16 [T, H]                                         */
  void* x_out;            /* bf16 [T, H] (must not alias x_in)                   */
  const void* q_in;       /* bf16 [T, Hq*d]; required iff !MK_FIRST_LAYER, and
                             then rows ctx..ctx+T-1 of the caches must be written */
  void* k_cache;          /* bf16 [max_ctx, Hkv, d], this layer                  */
  void* v_cache;          /* bf16 [max_ctx, Hkv, d]                              */
  void* next_k_cache;     /* MK_FUSE_NEXT_QKV: next layer's caches; rows
                             ctx..ctx+T-1 are written                            */
  void* next_v_cache;
  void* q_out;            /* MK_FUSE_NEXT_QKV: bf16 [T, Hq*d] next layer's q     */
  int32_t* topk_idx_out;  /* optional (may be NULL), MoE: int32 [T, k]           */
  float* topk_w_out;      /* optional (may be NULL), MoE: float [T, k]           */
  const uint16_t* tree_mask; /* optional HOST pointer to T uint16, read during the
                             call: token-tree verification (page "sgl-muse-mega:
                             Meta's Megakernel ...", section "What the README says
                             the kernels do": the draft's candidates form a
                             tree).  Bit j of tree_mask[i] is set iff verify
                             token j is token i itself or an ancestor of i;
                             tokens in topological order, so every mask holds
                             bit i and no bit above i, and the ancestors of an
                             ancestor are in the mask too (MK_ERR_INVALID_ARG
                             otherwise).  Token i sits at sequence position
                             ctx + depth_i (depth = its ancestors' count) and
                             keeps its K/V row at ctx + i; it sees the prefix
                             positions j < ctx with ctx + depth_i - j < window
                             and its ancestors-or-self a with depth_i - depth_a
                             < window (window 0: no limit).  NULL = the causal
                             chain (token i's ancestors are 0 .. i-1).           */
} mk_step_io;

typedef struct mk_layer mk_layer;
typedef struct mk_stack mk_stack;

/* Create a layer: validates the configuration, checks the current device is a
 * compute-capability 10.3 GPU, allocates library-owned scratch, repacks the
 * NVFP4 block scales into the tensor-core layout (library-owned copy) and
 * encodes the TMA descriptors of the weights.  Synchronous.  *out is NULL on
 * error. */
mk_status mk_layer_create(const mk_layer_config* cfg, const mk_layer_weights* w,
                          mk_layer** out);

/* Run one decode step of one layer as one persistent launch on `stream`
 * (a cudaStream_t; NULL = legacy default stream).  Asynchronous. */
mk_status mk_decode_step(mk_layer* layer, const mk_step_io* io, void* stream);

/* Device status of the layer's last step(s): MK_OK, or MK_ERR_TIMEOUT if a
 * bounded wait expired (the step's outputs are then undefined).  Reads a
 * device word synchronously; call after synchronising the step's stream.
 * The status is sticky until mk_layer_clear_status. */
mk_status mk_layer_status(mk_layer* layer);
mk_status mk_layer_clear_status(mk_layer* layer);

/* Frees library-owned memory only.  NULL is ignored. */
void mk_layer_destroy(mk_layer* layer);

/* Stacks: layers[0] must have MK_FIRST_LAYER; layers[0..n-2] must have
 * MK_FUSE_NEXT_QKV with next_w_qkv == layers[l+1]'s w_qkv and
 * next_attn_norm_w == layers[l+1]'s attn_norm_w; layers[n-1] must not fuse.
 * All layers share shapes except the window.  The stack borrows the layers
 * (destroy the stack before them). */
mk_status mk_stack_create(mk_layer* const* layers, int32_t n_layers, mk_stack** out);

typedef struct mk_stack_io {
  int32_t n_tokens;
  int32_t ctx_len;
  const void* x_in;           /* bf16 [T, H]                                   */
  void* x_out;                /* bf16 [T, H]                                   */
  void* const* k_caches;      /* host array of n_layers device pointers        */
  void* const* v_caches;      /* host array of n_layers device pointers        */
  int32_t* topk_idx_out;      /* optional: int32 [n_layers, T, k]              */
  float* topk_w_out;          /* optional: float [n_layers, T, k]              */
  const uint16_t* tree_mask;  /* optional HOST [T]: as mk_step_io.tree_mask, for
                                 every layer                                   */
} mk_stack_io;

/* One decode step through every layer: one launch per layer on `stream`,
 * chained with programmatic dependent launch.  Asynchronous. */
mk_status mk_stack_step(mk_stack* stack, const mk_stack_io* io, void* stream);
mk_status mk_stack_status(mk_stack* stack);
void mk_stack_destroy(mk_stack* stack);

/* Expert-prefetch statistics of a layer (MoE, prefetch_experts > 0), summed
 * over its steps since creation: `predicted` experts prefetched, `active`
 * experts the steps routed to, `hits` prefetched experts that were active.
 * hits / active is the share of expert weights that the prefetch covered.
 * Reads device counters synchronously: call after synchronising. */
typedef struct mk_prefetch_stats {
  uint64_t steps;
  uint64_t predicted;
  uint64_t active;
  uint64_t hits;
} mk_prefetch_stats;
mk_status mk_layer_prefetch_stats(mk_layer* layer, mk_prefetch_stats* out);
/* The same summed over the stack's layers. */
mk_status mk_stack_prefetch_stats(mk_stack* stack, mk_prefetch_stats* out);

/* Human-readable name of a status code (static storage). */
const char* mk_status_string(mk_status s);

/* Launch geometry chosen at create time (for reporting). */
typedef struct mk_layer_info {
  int32_t grid;            /* CTAs (one per SM)                                */
  int32_t threads;         /* threads per CTA                                  */
  int32_t smem_bytes;      /* dynamic shared memory per CTA                    */
  int32_t tmem_cols;       /* tensor-memory columns per CTA                    */
  int64_t scratch_bytes;   /* library-owned device bytes                       */
} mk_layer_info;
mk_status mk_layer_get_info(mk_layer* layer, mk_layer_info* info);

/* Self-timing (page "Muse Spark Open: 1,109 Tokens a Second ...", section
 * "What the 5.9 ms is still spent on": the kernel times itself with
 * %globaltimer stamps written by one lane per block).  Enabled for layers
 * created while the environment holds MK_TIMESTAMPS=1 (else this returns
 * MK_ERR_UNSUPPORTED).  Copies min(n, grid * 160) u64 of the layer's last
 * step to host memory: per CTA, 10 rows of 16 -- rows 0..8 are the phases
 * (QKV, attention, merge, o-proj, router+pool, expert gate/up, expert down,
 * unpool, next QKV) with %globaltimer stamps (epilogue start, epilogue end,
 * last MMA issued, last weight tile issued) followed by nanoseconds spent
 * (producer waiting for a free stage, MMA waiting for weights, for the token
 * operand, for a free accumulator, stager waiting for a free operand buffer,
 * stager working, epilogue waiting for an accumulator, epilogue working,
 * MMA issuing) and three more stamps (MMA starts the phase's units, stagers'
 * input dependency met, epilogue starts the phase's units);
 * row 9 starts with (kernel start, inputs ready, kernel end, this CTA's
 * router top-k start and its routing arrival -- CTAs 0..T-1 select one token
 * each --, router logits complete (in the CTA that finished the last router
 * tile), p complete seen by this CTA's stagers, its share of the p image
 * written).  All values are of the last step; stamps of
 * unused phases read 0.  Each CTA keeps them in shared memory and writes them
 * out when it exits, so that timing costs little.  Synchronous. */
mk_status mk_get_timestamps(mk_layer* layer, uint64_t* host_buf, size_t n);

/* One decode step of one layer, like mk_layer_create + mk_decode_step, but
 * allocating nothing: for callers that cannot call cudaMalloc -- code that
 * runs where device allocation is not allowed or not wanted, such as a
 * process whose device memory is handed out by another allocator or pool, or
 * one that must not grow its footprint after start-up.  (The pages describe
 * no counterpart; this is an addition of this library.)
 *
 * Every library-owned buffer of the step -- split-K and attention partials,
 * intermediates, counters, the repacked NVFP4 scale factors -- is carved out
 * of one static device array of 16 MiB that every GPU loading the library
 * holds until the process exits.  The caller still passes the weights, KV
 * caches, inputs and outputs, exactly as for mk_layer_create/mk_decode_step.
 * Layers whose buffers do not fit (roughly: small shapes such as hidden 256
 * with 16 small experts fit; the 4096-hidden, 256-expert shapes do not) are
 * rejected with MK_ERR_UNSUPPORTED before anything is launched (with
 * MK_LOG=1 a line on stderr says why); the attention split uses at most 32
 * chunks per KV head.  cfg->prefetch_experts is ignored: the shared array
 * keeps no routing history from one call to the next.
 *
 * The first call on a device performs a one-time set-up with that device
 * current (it looks up the array's device address); make that first call
 * before any stream capture.  The call is asynchronous on `stream`; every
 * call re-zeroes the counters it needs and re-derives the scale factors, and
 * all calls share the one array, so calls whose work overlaps on the GPU
 * (other streams, other threads) race and give undefined results.  A
 * device-side wait timeout leaves the outputs undefined and is not reported
 * by this call.  Same argument rules and errors as mk_layer_create and
 * mk_decode_step. */
mk_status mk_decode_step_noalloc(const mk_layer_config* cfg, const mk_layer_weights* w,
                                 const mk_step_io* io, void* stream);

/* ====================================================================
 * Batched decoding over a paged KV cache with a shared prefix
 *
 * The layer calls above run one sequence over a contiguous cache.  The calls
 * below are the operators of a step over several requests: mk_build_slots
 * gives every new token its position and its place in the cache,
 * mk_rope_apply rotates q and k and writes k and v there, mk_prefix_attn
 * attends.  A layer that ends with MK_FUSE_NEXT_QKV can be given positions
 * as well: mk_rope_apply rotates its q_out and the cache rows it wrote in
 * place, before the next layer (without MK_FIRST_LAYER) starts from them.
 *
 * The paged cache is a pool of pages, bf16 or fp16
 * [n_pages, page_size, n_kv_heads, head_dim] for K and the same for V; a slot
 * is page * page_size + offset.  A contiguous cache [max_ctx, Hkv, d] of the
 * layer calls is such a pool.  "Rows" are the new tokens of a step, request
 * after request: row r belongs to request b iff cu_rows[b] <= r <
 * cu_rows[b + 1].
 *
 * These calls keep no device memory: outputs and workspaces are the
 * caller's.  They are asynchronous on `stream`, never synchronise, may be
 * captured into a graph and may run at the same time on several streams as
 * long as their outputs and workspaces are distinct.  All tensors lie on the
 * device that is current during the call (MK_ERR_INVALID_ARG where the
 * library can tell otherwise) and `stream` belongs to it.
 * ==================================================================== */

typedef enum { MK_BF16 = 0, MK_FP16 = 1 } mk_dtype;

/* Block tables and slot maps from request lengths.
 *
 * Request b holds cached_lens[b] tokens of its own in the pages that its row
 * of block_table names, behind a prefix of prefix_len tokens that is not in
 * its table, and brings new_lens[b] tokens.  It needs
 *   ceil((cached + new) / page_size) - ceil(cached / page_size)
 * pages, which it gets from free_pages[*free_head ..] in batch order.  A
 * request is refused, and changes nothing of its table, if a length is
 * negative, cached + new is beyond max_pages pages, its rows end behind
 * n_rows, or -- where it needs pages -- its pages and those of the requests
 * before it are more than the list holds.  free_head outside 0..n_free is
 * taken as the nearer end.
 *
 * Outputs: rows keep their place whether a request is refused or not.  For
 * row i of request b the position is prefix_len + cached + i (at most
 * INT32_MAX) and the slot
 * table[b][(cached + i) / page_size] * page_size + (cached + i) % page_size;
 * the slot is -1 for a refused request and for a page outside 0..n_pages-1.
 * Rows behind the last request get position 0, slot -1, request -1.
 * Calling again with the same inputs gives the same outputs; inputs and
 * outputs (free_head and summary, cached_lens and lens among them) must not
 * overlap (MK_ERR_INVALID_ARG).  */
typedef struct mk_slots_io {
  int32_t n_requests;         /* B, 0 .. 65536                                    */
  int32_t n_rows;             /* length of the row outputs                        */
  int32_t page_size;          /* tokens per page, >= 1                            */
  int32_t max_pages;          /* pages per row of block_table;
                                 prefix_len + (max_pages + 1) * page_size < 2^31   */
  int64_t table_stride;       /* entries between rows of block_table, >= max_pages */
  int32_t n_pages;            /* pages in the pool                                */
  int32_t n_free;             /* length of free_pages                             */
  int32_t prefix_len;         /* >= 0                                             */
  const int32_t* cached_lens; /* [B]                                              */
  const int32_t* new_lens;    /* [B]                                              */
  const int32_t* free_pages;  /* [n_free]; NULL iff n_free is 0                   */
  const int32_t* free_head;   /* optional [1]: first entry not taken; NULL = 0    */
  int32_t* block_table;       /* [B, max_pages]: new pages are written            */
  int32_t* cu_rows;           /* [B + 1]: sums of new_lens (negative ones as 0),
                                 at most n_rows                                   */
  int32_t* lens;              /* [B]: cached + new, or cached where refused
                                 (then brought into 0 .. max_pages * page_size)   */
  int32_t* positions;         /* [n_rows]                                         */
  int64_t* slots;             /* [n_rows]                                         */
  int32_t* row_request;       /* optional [n_rows]                                */
  int32_t* summary;           /* [4]: free_head after the step; rows in use;
                                 requests refused; pages that the requests not
                                 refused for lengths or rows need together (at
                                 most INT32_MAX)                                  */
} mk_slots_io;
mk_status mk_build_slots(const mk_slots_io* io, void* stream);

/* Rotary positions.
 *
 * Of each head the first rot_dim values are rotated in pairs i = 0 ..
 * rot_dim/2 - 1 by the angle position * f_i:
 *   y_a = m (x_a cos - x_b sin),  y_b = m (x_b cos + x_a sin),
 * with (a, b) = (i, i + rot_dim/2) (MK_ROPE_HALF) or (2i, 2i + 1)
 * (MK_ROPE_INTERLEAVED); the other values pass.  f_i = theta^(-2i / rot_dim)
 * is scaled for contexts beyond the trained orig_ctx by `factor`:
 *   MK_ROPE_SCALE_NONE    f_i
 *   MK_ROPE_SCALE_LINEAR  f_i / factor (positions interpolated)
 *   MK_ROPE_SCALE_BASE    theta' = theta factor^(rot_dim / (rot_dim - 2))
 *   MK_ROPE_SCALE_PARTS   f_i (g + (1 - g) / factor), where g rises from 0 to 1
 *                         as the turns over orig_ctx, orig_ctx f_i / 2 pi, go
 *                         from beta_slow to beta_fast
 * and m = attn_factor, or where that is 0: 0.1 ln(factor) + 1 for
 * MK_ROPE_SCALE_PARTS, else 1.  Angles are held as 64-bit fractions of a turn
 * (exact modulo whole turns at any int32 position), values in 32 bits, and
 * each result is rounded once. */
typedef enum { MK_ROPE_HALF = 0, MK_ROPE_INTERLEAVED = 1 } mk_rope_layout;
typedef enum {
  MK_ROPE_SCALE_NONE = 0,
  MK_ROPE_SCALE_LINEAR = 1,
  MK_ROPE_SCALE_BASE = 2,
  MK_ROPE_SCALE_PARTS = 3
} mk_rope_scaling;

typedef struct mk_rope_config {
  int32_t head_dim;    /* d, a multiple of 8, <= 256                              */
  int32_t rot_dim;     /* 8 .. d; a multiple of 16 (MK_ROPE_HALF) or 8            */
  int32_t layout;      /* mk_rope_layout                                          */
  int32_t scaling;     /* mk_rope_scaling                                         */
  double theta;        /* >= 1                                                    */
  double factor;       /* >= 1; 1 for MK_ROPE_SCALE_NONE                          */
  int32_t orig_ctx;    /* MK_ROPE_SCALE_PARTS: > 0                                */
  double beta_fast;    /* MK_ROPE_SCALE_PARTS: > beta_slow; both 0 selects 32, 1  */
  double beta_slow;
  double attn_factor;  /* m; 0 = the scaling's own                                */
} mk_rope_config;

typedef struct mk_rope mk_rope;

/* Host memory only: a mk_rope serves every device, stream and thread. */
mk_status mk_rope_create(const mk_rope_config* cfg, mk_rope** out);
void mk_rope_destroy(mk_rope* rope);  /* NULL is ignored */

/* Rotates q into q_out and k into the cache and copies v into the cache.
 * Strides are in elements between rows (heads are contiguous, head_dim values
 * each), multiples of 8; tensors are 16-byte aligned.  q, k and v may be views
 * of one projection output.  q_out may be q itself (same stride), and k and v
 * may be the very cache rows that slots names for them; any other overlap
 * of an input with an output is not allowed.  A row whose slot is outside
 * 0 .. n_slots-1 writes nothing to the caches.  Slots are distinct: of rows
 * with the same slot either one's values stay, in pieces of 16 bytes. */
typedef struct mk_rope_io {
  int32_t n_rows;            /* >= 0; with 0 every pointer may be NULL            */
  int32_t n_q_heads;         /* 0 iff q is NULL                                   */
  int32_t n_kv_heads;        /* 0 iff k is NULL                                   */
  int32_t head_dim;          /* d: the one the mk_rope was created for            */
  int32_t dtype;             /* mk_dtype, of every tensor                         */
  const void* q;             /* [n_rows, n_q_heads, d]; optional                  */
  int64_t q_stride;
  void* q_out;               /* [n_rows, n_q_heads, d]                            */
  int64_t q_out_stride;
  const void* k;             /* [n_rows, n_kv_heads, d]; optional                 */
  int64_t k_stride;
  const void* v;             /* [n_rows, n_kv_heads, d]; optional: v_cache is
                                left as it is                                     */
  int64_t v_stride;
  const int32_t* positions;  /* [n_rows]                                          */
  const int64_t* slots;      /* [n_rows]; required with k                         */
  void* k_cache;             /* [n_slots, n_kv_heads, d]; required with k         */
  void* v_cache;             /* the same; required with v                         */
  int64_t n_slots;
} mk_rope_io;
mk_status mk_rope_apply(const mk_rope* rope, const mk_rope_io* io, void* stream);

/* Attention of a batch whose requests share a prefix.
 *
 * Request b has n_b = cu_rows[b+1] - cu_rows[b] rows and lens[b] keys of its
 * own, the last n_b of which are its rows' own; every row sees the
 * prefix_len keys of the prefix too.  With base = max(0, lens[b] - n_b), row
 * i has the position p = prefix_len + base + i and sees
 *   the prefix keys j (at position j),
 *   its request's keys j < lens[b] with j <= base + i (at prefix_len + j);
 * with tree_mask p = prefix_len + base + popcount(mask) - 1 and, of the
 * request's keys, those with j < base and those j >= base whose bit j - base is
 * set (bits of keys that are not there are ignored);
 * and of all these, with window > 0, only keys at positions > p - window.
 *   out = sum_j softmax_j(scale q.k_j) v_j,  lse = ln sum_j exp(scale q.k_j).
 * A row that sees no key gets out = 0 and lse = -infinity.  Rows before
 * cu_rows[0] and from cu_rows[B] on are left as they are.  Keys that no row sees
 * do not count: they may hold anything.  A key that some row sees must be finite.
 * A row of q that holds a NaN gets NaN, if it sees a key, and no other row does.
 * The prefix is read once per kv head and 256 / group rows of the batch, whichever
 * requests they are of, not once per request (and from HBM once as long as it fits
 * the L2 cache).
 *
 * Scores and sums are held in 32 bits, for scores scale q.k up to 2^26; the
 * softmax weights are rounded to the tensors' type before they multiply v (the
 * layer calls keep 16 bits of them).  Two calls on the same inputs give the
 * same bits.  Work is planned in 32 bits: MK_ERR_UNSUPPORTED where n_kv_heads *
 * (n_rows / (256 / group) + n_requests) * (128-key tiles of prefix and table
 * together) comes to 2^29 or more.  lens outside 0 .. max_pages * page_size
 * and cu_rows outside 0 .. n_rows are taken as the nearer end, and a page
 * outside 0 .. n_pages-1 reads as zeros.  A cu_rows that falls leaves out and
 * lse undefined: see mk_prefix_attn_status. */
typedef struct mk_prefix_attn_io {
  int32_t n_requests;          /* B, 1 .. 65536                                   */
  int32_t n_rows;              /* rows of q, >= 0                                 */
  int32_t n_q_heads;           /* a multiple of n_kv_heads, at most 64 per kv head */
  int32_t n_kv_heads;
  int32_t head_dim;            /* d: 64 or 128                                    */
  int32_t dtype;               /* mk_dtype of q, the caches and out               */
  int32_t page_size;           /* a power of two, 16 .. 65536                     */
  int32_t n_pages;             /* n_pages * page_size < 2^31                      */
  int32_t prefix_len;          /* >= 0                                            */
  int32_t max_pages;           /* pages per row of block_table, >= 0              */
  int64_t table_stride;        /* entries between rows of block_table             */
  int32_t window;              /* 0 = every key; with tree_mask 0 or >= 64        */
  float scale;                 /* of the scores; 0 selects 1 / sqrt(d)            */
  const void* q;               /* [n_rows, n_q_heads, d], 16-byte aligned         */
  int64_t q_stride;            /* elements between rows, a multiple of 8          */
  const void* k_cache;         /* [n_pages, page_size, n_kv_heads, d]             */
  const void* v_cache;
  const int32_t* prefix_pages; /* [ceil(prefix_len / page_size)]                  */
  const int32_t* block_table;  /* [B, max_pages]                                  */
  const int32_t* lens;         /* [B]                                             */
  const int32_t* cu_rows;      /* [B + 1]                                         */
  const uint64_t* tree_mask;   /* optional [n_rows]: bit j of row i's word says
                                  that it sees row j of its request, itself
                                  always among them; a request has at most 64
                                  rows then (a 65th would be seen by none)        */
  void* out;                   /* [n_rows, n_q_heads, d]; not q                   */
  int64_t out_stride;          /* elements between rows, a multiple of 8          */
  float* lse;                  /* optional [n_rows, n_q_heads]                    */
} mk_prefix_attn_io;

/* Bytes of workspace that mk_prefix_attn needs for every call with these
 * n_requests, n_rows, heads and head_dim (pointers are not looked at), on the
 * current device.  Grows with n_rows and n_requests. */
mk_status mk_prefix_attn_workspace(const mk_prefix_attn_io* io, int64_t* bytes);

/* workspace: device memory, 256-byte aligned, its content does not matter; one
 * call in flight per workspace. */
mk_status mk_prefix_attn(const mk_prefix_attn_io* io, void* workspace, int64_t workspace_bytes,
                         void* stream);

/* Device status of the last mk_prefix_attn that used `workspace`: MK_OK, or
 * MK_ERR_TIMEOUT if a bounded device-side wait expired (2 s for a hand-off),
 * MK_ERR_INVALID_ARG if its cu_rows falls; out and lse are then undefined, and the
 * next call on the workspace is well.  Reads a device word synchronously: call
 * after synchronising. */
mk_status mk_prefix_attn_status(const void* workspace);

/* ====================================================================
 * The attention half of a batched layer over a paged cache in 4 bits
 *
 * mk_linear makes q, k and v of the batch's rows, mk_qkv_append norms and
 * rotates them and writes k and v into a paged cache, mk_kvq_attn attends,
 * mk_linear projects back onto the residual stream.  Slots, positions, lens,
 * cu_rows and block tables are those of mk_build_slots (prefix_len 0: a prefix
 * that requests share stands in each of their tables).  The conventions are
 * those of the batched calls above.
 *
 * A cache in 4 bits: of each token and kv head the head_dim values lie in groups
 * of 16; each group has an E4M3 scale s, each head a power of two 2^e, and the
 * code n (0 .. 15) stands for (n - 8) s 2^e.  Pools, in order of
 *   codes   uint8 [n_pages, n_kv_heads, page_size, head_dim / 2], value 2i in the
 *           low nibble of byte i
 *   scales  uint8 [n_pages, n_kv_heads, page_size, head_dim / 16]
 * The slot page * page_size + offset is the row (page, :, offset).
 * ==================================================================== */

typedef struct mk_kvq_cache {
  int32_t n_pages;        /* n_pages * page_size < 2^31                           */
  int32_t page_size;      /* a power of two, 16 .. 65536                          */
  int32_t n_kv_heads;     /* <= 4096                                              */
  int32_t head_dim;       /* d: a multiple of 16, <= 256                          */
  void* k_codes;          /* the pools; 16-byte aligned                           */
  void* k_scales;
  void* v_codes;
  void* v_scales;
  const int32_t* k_exp;   /* optional [n_kv_heads]: e of each head's keys, -64 ..
                             64 (others count as the nearer end); NULL = 0        */
  const int32_t* v_exp;   /* the same of its values                               */
} mk_kvq_cache;

/* Norms of q and k, rotary positions and the K/V write in one pass.
 *
 * Of each head x (with a norm weight w):
 *   n_i = x_i w_i / sqrt(mean_j x_j^2 + eps),
 * then the rotation of mk_rope_apply by the row's position (rope NULL: none).
 * q goes to q_out, rounded once.  k and v (v as it is) go to the row's slot: with
 * bits 16 into k_cache and v_cache as in mk_rope_apply, rounded once; with bits 4
 * into kvq: of each group z_i = y_i 2^-e of 16 values
 *   s = E4M3(max |z| / 7) to nearest even, at most 448,
 *   n_i = min(max(rint(z_i / s), -8), 7) + 8   (8 where s is 0).
 * These are the codes of the formula: sums and angles are held in 32 bits, and
 * where a value comes so near a border between two codes or scales that this
 * could tell, the group is worked out again in 64 bits.  A group that holds a NaN
 * gets the scale NaN (0x7F) and the codes 8; infinities saturate.
 * A row whose slot is outside the pool writes nothing there; slots are distinct.
 * mean x^2 + eps has to be a normal number in 32 bits (squares up to 3e38).
 * q_out may be q itself (same stride); any other overlap of an output with an input or
 * another output is refused, each counted as the stretch from its first value to its
 * last, with two exceptions: q_out may lie between the rows of k and v (at their stride),
 * and with bits 16 k may be in the k_cache, v in the v_cache, in the very rows that slots
 * names. */
typedef struct mk_qkv_append_io {
  int32_t n_rows;            /* >= 0; with 0 every tensor of rows may be NULL      */
  int32_t n_q_heads;         /* 0 iff q is NULL; <= 4096                           */
  int32_t n_kv_heads;        /* 0 iff k is NULL; <= 4096                           */
  int32_t head_dim;          /* d: a multiple of 8 (bits 4: 16), <= 256            */
  int32_t dtype;             /* mk_dtype of q, k, v, the norm weights, the caches
                                in 16 bits                                         */
  int32_t bits;              /* 16 or 4: the cache's                               */
  float eps;                 /* >= 0; looked at with a norm weight only            */
  const void* q;             /* [n_rows, n_q_heads, d]; optional                   */
  int64_t q_stride;          /* elements between rows, a multiple of 8             */
  void* q_out;               /* [n_rows, n_q_heads, d]                             */
  int64_t q_out_stride;
  const void* k;             /* [n_rows, n_kv_heads, d]; optional                  */
  int64_t k_stride;
  const void* v;             /* [n_rows, n_kv_heads, d]; optional: the cache's
                                values are left as they are                        */
  int64_t v_stride;
  const int32_t* positions;  /* [n_rows]; required with rope                       */
  const int64_t* slots;      /* [n_rows]; required with k                          */
  const void* q_norm;        /* optional [d]: w of the q heads                     */
  const void* k_norm;        /* optional [d]: w of the k heads                     */
  void* k_cache;             /* bits 16: [n_slots, n_kv_heads, d]                  */
  void* v_cache;
  int64_t n_slots;           /* bits 16                                            */
  mk_kvq_cache kvq;          /* bits 4                                             */
} mk_qkv_append_io;
mk_status mk_qkv_append(const mk_rope* rope, const mk_qkv_append_io* io, void* stream);

/* The values that rows of a cache in 4 bits stand for, in 16 bits: row i of k_out
 * and v_out is slot slots[i], or slot i where slots is NULL (then n_rows is at most
 * the pool's slots).  A slot outside the pool reads as zeros.  bf16 holds every
 * (n - 8) s exactly, fp16 as well; 2^e may round or overflow there. */
typedef struct mk_kvq_read_io {
  mk_kvq_cache kvq;
  int32_t n_rows;            /* >= 0                                               */
  int32_t dtype;             /* mk_dtype of k_out and v_out                        */
  const int64_t* slots;      /* optional [n_rows]                                  */
  void* k_out;               /* [n_rows, n_kv_heads, d], contiguous; optional       */
  void* v_out;               /* the same; optional                                 */
} mk_kvq_read_io;
mk_status mk_kvq_read(const mk_kvq_read_io* io, void* stream);

/* Attention over a paged cache in 4 bits.
 *
 * Request b has n_b = cu_rows[b+1] - cu_rows[b] rows and lens[b] keys, the last
 * n_b of which are its rows' own.  With base = max(0, lens[b] - n_b) its row i has
 * the position p = base + i and sees the keys j < lens[b] with j <= p; with
 * tree_mask p = base + popcount(mask) - 1 and it sees the keys j < base and those
 * j >= base whose bit j - base is set (bits of keys that are not there are
 * ignored); and of all these, with window > 0, only keys at positions > p - window
 * (key j is at position j).
 *   out = sum_j softmax_j(scale q.k_j) v_j,  lse = ln sum_j exp(scale q.k_j).
 * A row that sees no key gets out = 0 and lse = -infinity.  Rows before cu_rows[0]
 * and from cu_rows[B] on are left as they are.  Keys that no row sees do not count:
 * their codes and scales may be anything.  A key that some row sees must have
 * finite scales.  A row of q that holds a NaN gets NaN, if it sees a key, and no
 * other row does.
 *
 * Keys and values come into the products exactly; q is held in 11 bits relative to
 * its row's largest value or better; the softmax weights are rounded to fp16 (11
 * bits) before they multiply v, and those below 2^-31 of a row's largest count in its
 * sum only; scores, maxima, sums and out are held in 32 bits and out is rounded once.  Two calls on the same inputs give the same bits.
 * lens outside 0 .. max_pages * page_size and cu_rows outside 0 .. n_rows are
 * taken as the nearer end, and a page outside 0 .. n_pages-1 reads as zeros.  A
 * cu_rows that falls leaves out and lse undefined.  Scores up to 2^26 are held to.
 * A page's codes (n_kv_heads * page_size * d / 2 bytes) are less than 2^31.  No
 * output may overlap an input; a tensor of rows counts from its first value to its
 * last, what lies between its rows included.
 * A call goes through one kernel, by its requests' rows per kv head on average (up to 8,
 * up to 16, more): single tokens beside long chunks take less time in a call of their
 * own. */
typedef struct mk_kvq_attn_io {
  int32_t n_requests;          /* B, 1 .. 65536                                   */
  int32_t n_rows;              /* rows of q, >= 0                                 */
  int32_t n_q_heads;           /* a multiple of kvq.n_kv_heads, at most 64 per kv
                                  head                                            */
  int32_t dtype;               /* mk_dtype of q and out                           */
  int32_t max_pages;           /* pages per row of block_table, >= 0              */
  int32_t window;              /* 0 = every key; with tree_mask 0 or >= 64        */
  float scale;                 /* of the scores; 0 selects 1 / sqrt(d)            */
  int64_t table_stride;        /* entries between rows of block_table             */
  mk_kvq_cache kvq;            /* head_dim 64 or 128                              */
  const void* q;               /* [n_rows, n_q_heads, d], 16-byte aligned         */
  int64_t q_stride;            /* elements between rows, a multiple of 8          */
  const int32_t* block_table;  /* [B, max_pages]                                  */
  const int32_t* lens;         /* [B]                                             */
  const int32_t* cu_rows;      /* [B + 1]                                         */
  const uint64_t* tree_mask;   /* optional [n_rows], as for mk_prefix_attn; here a
                                  word may leave its own row out or be empty, as
                                  of a padded row                                 */
  void* out;                   /* [n_rows, n_q_heads, d]; not q                   */
  int64_t out_stride;          /* elements between rows, a multiple of 8          */
  float* lse;                  /* optional [n_rows, n_q_heads]                    */
} mk_kvq_attn_io;

/* Bytes of workspace for every call with these n_requests, n_rows, heads and
 * head_dim (pointers are not looked at), on the current device. */
mk_status mk_kvq_attn_workspace(const mk_kvq_attn_io* io, int64_t* bytes);

/* workspace: device memory, 256-byte aligned, its content does not matter; one
 * call in flight per workspace. */
mk_status mk_kvq_attn(const mk_kvq_attn_io* io, void* workspace, int64_t workspace_bytes,
                      void* stream);

/* Device status of the last mk_kvq_attn that used `workspace`: MK_OK, or
 * MK_ERR_TIMEOUT if a bounded device-side wait expired (out and lse are then
 * undefined).  Reads a device word synchronously: call after synchronising. */
mk_status mk_kvq_attn_status(const void* workspace);

/* Projection with bias, activation and residual:
 *   out = act(x w^T + bias) + residual,
 * summed in 32 bits and rounded once; an activation's result below 2^-119 may be 0.
 * MK_ACT_SILU: y / (1 + e^-y); MK_ACT_GELU: y (1 + erf(y / sqrt 2)) / 2;
 * MK_ACT_GELU_TANH: y (1 + tanh(sqrt(2 / pi) (y + 0.044715 y^3))) / 2.  residual may be
 * out itself (same stride); any other overlap of an input with out, counted as for
 * mk_kvq_attn, is not allowed.  Two calls on the same inputs give the same bits. */
typedef enum { MK_ACT_NONE = 0, MK_ACT_SILU = 1, MK_ACT_GELU = 2, MK_ACT_GELU_TANH = 3 } mk_act;

typedef struct mk_linear_io {
  int32_t n_rows;          /* >= 0; with 0 x, residual and out may be NULL        */
  int32_t n_in;            /* a multiple of 8, >= 8                               */
  int32_t n_out;           /* >= 1                                                */
  int32_t dtype;           /* mk_dtype, of every tensor                           */
  int32_t act;             /* mk_act                                              */
  const void* x;           /* [n_rows, n_in], 16-byte aligned                     */
  int64_t x_stride;        /* elements between rows, a multiple of 8              */
  const void* w;           /* [n_out, n_in], 16-byte aligned                      */
  int64_t w_stride;        /* the same                                            */
  const void* bias;        /* optional [n_out]                                    */
  const void* residual;    /* optional [n_rows, n_out]                            */
  int64_t residual_stride; /* elements between rows, >= n_out                     */
  void* out;               /* [n_rows, n_out]                                     */
  int64_t out_stride;      /* elements between rows, >= n_out                     */
} mk_linear_io;

/* Bytes of workspace for every call with these sizes (pointers and strides are not
 * looked at), on the current device. */
mk_status mk_linear_workspace(const mk_linear_io* io, int64_t* bytes);

/* workspace: as for mk_kvq_attn. */
mk_status mk_linear(const mk_linear_io* io, void* workspace, int64_t workspace_bytes, void* stream);

/* Device status of the last mk_linear that used `workspace`: as mk_kvq_attn_status. */
mk_status mk_linear_status(const void* workspace);

#ifdef __cplusplus
}
#endif
#endif /* MK_H_ */
