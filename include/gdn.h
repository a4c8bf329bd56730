/*
 * gdn.h — C ABI of libgdn: the Gated DeltaNet (GDN) decode step on NVIDIA B200 (sm_100a).
 *
 * The operation is the single-token (or short multi-token) decode of one GDN
 * linear-attention layer, as dispatched on the page
 * "spark_model/forward/qwen3_5/linear_attention.rs" (Atlas), steps 3 to 8 plus the
 * SiLU(z) gate of the fused steps 9+10+11:
 *
 *   conv   : per channel, a depthwise causal conv of width W over the stored W-1 raw
 *            inputs and the new ones (no bias), SiLU; per-head L2 norm of the Q and K
 *            channels, x / sqrt(sum x^2 + l2_eps); q additionally times q_scale
 *   gate   : g = -exp(A_log) * softplus(a + dt_bias), alpha = exp(g); beta = sigmoid(b)
 *   update : per (sequence, v-head h) with k-head h / (Hv/Hk), FP32 state S[dk][dv]:
 *            S <- alpha S;  S <- S + beta k (v - S^T k)^T;  o = S^T q
 *   norm   : out = o / sqrt(mean_j o_j^2 + rms_eps) * norm_w * silu(z)
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Pointers. Every tensor argument is a DEVICE pointer owned by the caller,
 *   contiguous, row-major in the layout stated, and 16-byte aligned. bf16 values are
 *   passed as their uint16_t bit patterns. The library allocates nothing, keeps no
 *   state between calls and never synchronizes; it only enqueues kernels on `stream`
 *   (a cudaStream_t; NULL means the legacy default stream). Outputs must not alias
 *   inputs or one another.
 * Shapes. Hk = num_k_heads, Hv = num_v_heads (a multiple of Hk, Hv/Hk <= 8),
 *   dk = head_k_dim, dv = head_v_dim (each 16, 32, 64 or 128), W = conv_width (2..8),
 *   C = 2*Hk*dk + Hv*dv qkv channels ordered Q | K | V, head-major inside each block.
 *   B = sequences in this call (B = 0 is a no-op), T = tokens per sequence (1..16),
 *   P = pool_slots.
 * Pools. conv_pool [P][W-1][C] bf16 holds each slot's last W-1 raw (pre-conv) inputs,
 *   row 0 the oldest; state_pool [P][Hv][dk][dv] fp32. Sequence b uses slot slots[b]
 *   of both pools; slots[] (int32, device) must hold distinct values. Pools are
 *   updated in place; slots that no sequence names are never read or written.
 * Multi-token calls (T > 1) are defined as T single-token calls in order.
 * Errors. Every argument check runs on the host before anything is enqueued, so a
 *   call that returns an error has written nothing. Slot VALUES live on the device:
 *   a sequence whose slot is outside [0, P) is skipped entirely (its pools and
 *   outputs untouched) and, when err_flag is non-NULL, the bit
 *   GDN_DEVICE_ERR_SLOT_RANGE is OR-ed into *err_flag (the caller zeroes it; the
 *   library never clears it). Duplicate slots are not detected on the device and
 *   give undefined results; gdn_check_slots_host() checks a host copy. Every wait
 *   inside a kernel is bounded: a CTA whose staged state copy has not landed after
 *   2e9 cycles of its SM's clock (a second at the top clock) gives up, ORs
 *   GDN_DEVICE_ERR_TIMEOUT into *err_flag and writes neither that state tile nor its
 *   outputs (their values are then unspecified).
 *   A failed launch returns GDN_ERR_CUDA.
 */
#ifndef GDN_H_
#define GDN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    GDN_OK = 0,
    GDN_ERR_INVALID_ARGUMENT = 1, /* null pointer, negative size, eps < 0, bad pool size */
    GDN_ERR_UNSUPPORTED = 2,      /* a shape outside the supported set above */
    GDN_ERR_MISALIGNED = 3,       /* a tensor pointer not 16-byte aligned */
    GDN_ERR_SLOT_RANGE = 4,       /* gdn_check_slots_host: slot out of range or repeated */
    GDN_ERR_CUDA = 5              /* the CUDA launch itself failed */
} gdn_status;

/* Bits a kernel ORs into *err_flag. */
#define GDN_DEVICE_ERR_SLOT_RANGE 1 /* a sequence's slot is outside [0, pool_slots) */
#define GDN_DEVICE_ERR_TIMEOUT 2    /* a bounded wait inside the kernel ran out */
#define GDN_DEVICE_ERR_SEQLEN 4     /* a token count (varlen) or accepted count (spec commit) out of range */
#define GDN_DEVICE_ERR_BATCH 8      /* gdn_decode_step_device_batch: *B_dev outside [0, B_max] */
#define GDN_DEVICE_ERR_PAGE 16      /* a page number outside the pool, no free page left, or a table row in use */

typedef struct {
    int32_t num_k_heads; /* Hk */
    int32_t num_v_heads; /* Hv, a multiple of Hk */
    int32_t head_k_dim;  /* dk */
    int32_t head_v_dim;  /* dv */
    int32_t conv_width;  /* W */
    float l2_eps;        /* q/k L2-norm epsilon (inside the root); the page uses 1e-6 */
    float rms_eps;       /* output RMSNorm epsilon (inside the root) */
    float q_scale;       /* factor on the normalised q; 0 selects 1/sqrt(dk) */
} gdn_config;

/*
 * Stage 1 — step 3 of the page, "fused causal_conv1d_update_l2norm", with the
 * 1/sqrt(d_k) q scale it applies at the kernel output, and the Q|K|V split of step 6.
 *   qkv     [B][T][C] bf16        this call's raw projections
 *   conv_w  [C][W] bf16           tap W-1 multiplies the current token
 *   conv_pool, pool_slots, slots  as above; the slot's history is rolled in place
 *   q_out   [B][T][Hk][dk] fp32   L2-normalised, times q_scale
 *   k_out   [B][T][Hk][dk] fp32   L2-normalised
 *   v_out   [B][T][Hv][dv] fp32   SiLU output, no norm
 *   err_flag nullable device int32
 */
gdn_status gdn_conv_update(const gdn_config* cfg, int32_t B, int32_t T, const uint16_t* qkv,
                           const uint16_t* conv_w, uint16_t* conv_pool, int32_t pool_slots,
                           const int32_t* slots, float* q_out, float* k_out, float* v_out,
                           int32_t* err_flag, void* stream);

/*
 * Stage 2 — steps 4, 5 and 7 of the page: the gate, beta and
 * "gated_delta_rule_decode" on the FP32 state pool, one pass over each state.
 *   q, k    [B][T][Hk][dk] fp32   as produced by gdn_conv_update (q already scaled)
 *   v       [B][T][Hv][dv] fp32
 *   a, b    [B][T][Hv] bf16       raw gate and beta projections
 *   A_log, dt_bias [Hv] fp32
 *   state_pool, pool_slots, slots as above; each named state is read once and
 *                                 written once (after all T tokens)
 *   o       [B][T][Hv][dv] fp32   S^T q with S after the token's update
 */
gdn_status gdn_recurrent_step(const gdn_config* cfg, int32_t B, int32_t T, const float* q,
                              const float* k, const float* v, const uint16_t* a, const uint16_t* b,
                              const float* A_log, const float* dt_bias, float* state_pool,
                              int32_t pool_slots, const int32_t* slots, float* o,
                              int32_t* err_flag, void* stream);

/*
 * Stage 3 — step 8 of the page (per-head RMSNorm over dv with one weight vector
 * shared by all heads) and the SiLU(z) gate of steps 9+10+11.
 *   rows     number of (sequence, token, v-head) rows, i.e. B*T*Hv
 *   o        [rows][dv] fp32
 *   z        [rows][dv] bf16
 *   norm_w   [dv] bf16
 *   out_bf16 [rows][dv] bf16      round-to-nearest-even of the fp32 result
 *   out_f32  [rows][dv] fp32      nullable; the same result before rounding
 */
gdn_status gdn_gated_rmsnorm(const gdn_config* cfg, int32_t rows, const float* o, const uint16_t* z,
                             const uint16_t* norm_w, uint16_t* out_bf16, float* out_f32,
                             void* stream);

/*
 * The fused decode step: the three stages above in ONE kernel launch. Each state
 * tile is streamed from HBM once and written back in place; the conv history of
 * every channel is read and rolled by exactly one CTA; q, k, v, the gates and o
 * never leave the chip.
 *   qkv [B][T][C], a [B][T][Hv], b [B][T][Hv], z [B][T][Hv][dv]   bf16 inputs
 *   conv_w [C][W] bf16, A_log [Hv] fp32, dt_bias [Hv] fp32, norm_w [dv] bf16
 *   conv_pool, state_pool, pool_slots, slots                     as above
 *   out_bf16 [B][T][Hv][dv] bf16
 *   out_f32  [B][T][Hv][dv] fp32, nullable (the unrounded output, for parity checks)
 *   err_flag nullable device int32
 *   workspace nullable device buffer of gdn_decode_workspace_bytes() bytes, zeroed by
 *            the caller once before its first use; every call leaves it zeroed again.
 *            With it, large single-token batches are spread over the SMs dynamically
 *            (faster SMs take more sequences); without it the split is static. The
 *            results are the same bits either way. Calls that may run at the same
 *            time on the GPU need separate workspaces.
 * The first call on a device (per shape) queries the device once and sets a kernel
 * attribute; make it before capturing the call into a CUDA graph.
 * The launch allows programmatic stream serialization: the kernel may begin while the
 * kernel before it in the stream drains, but it reads nothing (inputs, pools, slots,
 * workspace) before that kernel has completed; until then it only issues L2 prefetch
 * hints for the first state tiles it will read.
 */
gdn_status gdn_decode_step(const gdn_config* cfg, int32_t B, int32_t T, const uint16_t* qkv,
                           const uint16_t* a, const uint16_t* b, const uint16_t* z,
                           const uint16_t* conv_w, const float* A_log, const float* dt_bias,
                           const uint16_t* norm_w, uint16_t* conv_pool, float* state_pool,
                           int32_t pool_slots, const int32_t* slots, uint16_t* out_bf16,
                           float* out_f32, int32_t* err_flag, void* workspace, void* stream);

/* Bytes of the optional workspace of gdn_decode_step (a multiple of 16). */
size_t gdn_decode_workspace_bytes(void);

/*
 * gdn_decode_step with the batch count in DEVICE memory, for CUDA-graph replay. The
 * launch is sized for B_max sequences; each kernel reads *B_dev (int32, 4-byte
 * aligned) after the work before it in the stream has completed and processes
 * sequences 0 .. *B_dev - 1 only, exactly as gdn_decode_step with B = *B_dev would
 * (the results may differ from that call in the last bits where B_max selects
 * another kernel than B would). Sequences *B_dev .. B_max - 1: pools and outputs
 * untouched. A captured call therefore serves every batch up to B_max: before each
 * replay write the count to *B_dev and the inputs and slots of that many sequences
 * to the captured buffers (the counterpart of the layer graph hooks on the page
 * "metrale_model_arch/glm5next_dsa/layer.rs", which read the replayed step's
 * positions from device memory). All other arguments are those of gdn_decode_step
 * with B = B_max (tensors sized for B_max). A value of *B_dev outside [0, B_max]
 * runs no sequence and ORs GDN_DEVICE_ERR_BATCH into *err_flag. The host-side
 * kernel choice and device queries happen on the first call per shape: make it
 * before the capture.
 */
gdn_status gdn_decode_step_device_batch(const gdn_config* cfg, const int32_t* B_dev, int32_t B_max, int32_t T,
                                        const uint16_t* qkv, const uint16_t* a, const uint16_t* b, const uint16_t* z,
                                        const uint16_t* conv_w, const float* A_log, const float* dt_bias,
                                        const uint16_t* norm_w, uint16_t* conv_pool, float* state_pool,
                                        int32_t pool_slots, const int32_t* slots, uint16_t* out_bf16, float* out_f32,
                                        int32_t* err_flag, void* workspace, void* stream);

/*
 * The fused decode step for a batch whose sequences bring different numbers of tokens
 * (a chunk of a prompt for some, one token for others) in ONE kernel launch. The
 * pages launch per sequence and have no such layout; each sequence's tokens are
 * processed exactly as gdn_decode_step processes T tokens (steps 3 to 8 and the
 * SiLU(z) gate of steps 9+10+11, the tokens in order, the state on chip in between).
 * The tokens of all sequences are packed row after row:
 *   cu_seqlens [B+1] int32 device, 4-byte aligned: sequence i owns the n_i =
 *            cu_seqlens[i+1] - cu_seqlens[i] rows cu_seqlens[i] .. cu_seqlens[i+1]-1;
 *            cu_seqlens[0] = 0 and cu_seqlens[B] = total_tokens are expected
 *   T_max    the largest n_i, 1..16 (sizes the kernel's on-chip buffers)
 *   total_tokens  rows of the packed tensors (>= 0; only checked on the host)
 *   qkv [total][C], a [total][Hv], b [total][Hv], z [total][Hv][dv]   bf16 inputs
 *   out_bf16 [total][Hv][dv] bf16, out_f32 [total][Hv][dv] fp32 nullable
 *   the weights, pools, slots and err_flag as for gdn_decode_step.
 * A sequence with n_i = 0 is left untouched. A sequence with n_i < 0, n_i > T_max or
 * rows outside [0, total_tokens) is skipped (pools and outputs untouched) and
 * GDN_DEVICE_ERR_SEQLEN is OR-ed into *err_flag; a slot outside [0, pool_slots) is
 * handled as in gdn_decode_step. Rows that no sequence owns are neither read nor
 * written. total_tokens = 0 returns GDN_OK without launching. Launched like
 * gdn_decode_step (programmatic stream serialization, no allocation, no
 * synchronization).
 */
gdn_status gdn_decode_step_varlen(const gdn_config* cfg, int32_t B, const int32_t* cu_seqlens,
                                  int32_t T_max, int32_t total_tokens, const uint16_t* qkv,
                                  const uint16_t* a, const uint16_t* b, const uint16_t* z,
                                  const uint16_t* conv_w, const float* A_log, const float* dt_bias,
                                  const uint16_t* norm_w, uint16_t* conv_pool, float* state_pool,
                                  int32_t pool_slots, const int32_t* slots, uint16_t* out_bf16,
                                  float* out_f32, int32_t* err_flag, void* stream);

/*
 * The projections on either side of the decode step, as GEMMs on the tensor cores
 * (tcgen05, bf16 inputs, fp32 accumulation, bf16 outputs rounded to nearest even).
 * Token rows: rows = B*T <= 256; hidden: the model width, a multiple of 8.
 *
 * gdn_in_proj — step 2 of the page (in_proj_qkv, in_proj_z and the dual-output
 * in_proj_a / in_proj_b, all reading the same normalised input) as ONE GEMM over the
 * four weights stacked row-wise:
 *   x     [rows][hidden] bf16                      the normalised layer input
 *   w_in  [C + Hv*dv + 2*Hv][hidden] bf16          rows: in_proj_qkv (C rows), in_proj_z
 *                                                  (Hv*dv), in_proj_a (Hv), in_proj_b (Hv)
 *   qkv [rows][C], z [rows][Hv*dv], a [rows][Hv], b [rows][Hv] bf16 outputs, laid out as
 *                                                  gdn_decode_step takes them (T = 1 rows,
 *                                                  or [B][T] flattened)
 *   out_f32 [rows][C + Hv*dv + 2*Hv] fp32, nullable: the stacked outputs before rounding
 * gdn_out_proj — the GEMV of the page's fused steps 9+10+11, out = out_proj @ y, on the
 * decode step's output y (already normalised and gated by SiLU(z)):
 *   y     [rows][Hv*dv] bf16, w_out [hidden][Hv*dv] bf16, out [rows][hidden] bf16
 *   out_f32 [rows][hidden] fp32, nullable
 * The first call per shape queries the device (kernel attribute, co-resident clusters,
 * which set how K is split); make it before capturing the call into a CUDA graph.
 * Errors: rows > 256 or hidden not a multiple of 8 give GDN_ERR_UNSUPPORTED; other
 * checks as above, all before anything is enqueued. Every wait inside the kernel is
 * bounded; on expiry GDN_DEVICE_ERR_TIMEOUT is OR-ed into *err_flag (nullable) and
 * the outputs are unspecified. Launched with programmatic stream serialization.
 */
gdn_status gdn_in_proj(const gdn_config* cfg, int32_t hidden, int32_t rows, const uint16_t* x,
                       const uint16_t* w_in, uint16_t* qkv, uint16_t* z, uint16_t* a, uint16_t* b, float* out_f32,
                       int32_t* err_flag, void* stream);
gdn_status gdn_out_proj(const gdn_config* cfg, int32_t hidden, int32_t rows, const uint16_t* y,
                        const uint16_t* w_out, uint16_t* out, float* out_f32, int32_t* err_flag, void* stream);

/*
 * Speculative decoding: verify T drafted tokens, then keep the state after the
 * accepted prefix only. The GDN analogue of the rewind of a rejected speculative
 * draft on the page "metrale_model_arch/glm5next_dsa/layer.rs" (its lockstep check
 * and rewind_to(seq_len) on a rejected draft): a linear-attention state cannot be
 * rewound by truncation, so the verify call leaves both pools as they were and
 * records, per token, the factors of that token's state update; the commit call
 * applies the first n_accept[b] of them.
 *
 * gdn_spec_verify takes the arguments of gdn_decode_step (T = the drafted tokens,
 * 1..16) and writes exactly the outputs a T-token gdn_decode_step would write
 * (steps 3 to 8 and the SiLU(z) gate, the tokens in order), but neither conv_pool nor
 * state_pool is written. Instead, for token t of sequence b:
 *   spec_k     [B][T][Hk][dk] fp32  the normalised key k_t (L2 norm of step 3)
 *   spec_delta [B][T][Hv][dv] fp32  the write delta_t = beta_t (v_t - alpha_t S_{t-1}^T k_t)
 *   spec_alpha [B][T][Hv]     fp32  the decay alpha_t = exp(g_t)
 * so that the state after token t is S_t = alpha_t S_{t-1} + k_t delta_t^T
 * (v-head h uses k-head h / (Hv/Hk)). All three buffers are caller-owned device
 * memory, 16-byte aligned, written in full for every sequence that is not skipped.
 * Skipping (slot out of range) and err_flag are as in gdn_decode_step. Launched
 * like gdn_decode_step (programmatic stream serialization, no allocation).
 */
gdn_status gdn_spec_verify(const gdn_config* cfg, int32_t B, int32_t T, const uint16_t* qkv, const uint16_t* a,
                           const uint16_t* b, const uint16_t* z, const uint16_t* conv_w, const float* A_log,
                           const float* dt_bias, const uint16_t* norm_w, const uint16_t* conv_pool,
                           const float* state_pool, int32_t pool_slots, const int32_t* slots, uint16_t* out_bf16,
                           float* out_f32, float* spec_k, float* spec_delta, float* spec_alpha, int32_t* err_flag,
                           void* stream);

/*
 * Commits the accepted prefix of a gdn_spec_verify call: sequence b keeps its first
 * n = n_accept[b] drafted tokens. Its state becomes S_n (the updates of tokens
 * 0..n-1 applied in order to the state the verify call read) and its conv history
 * becomes the last W-1 raw inputs of [history, qkv tokens 0..n-1], bit for bit. The
 * result equals that of a gdn_decode_step over the first n tokens only.
 *   n_accept   [B] int32 device; 0 leaves the sequence's pools untouched
 *   T          the T of the verify call (the layout of qkv and the spec buffers)
 *   qkv        [B][T][C] bf16, the verify call's input (for the conv history)
 *   spec_k, spec_delta, spec_alpha  as written by the verify call
 *   conv_pool, state_pool, pool_slots, slots  the verify call's pools and slots
 * A sequence whose n_accept is outside [0, T] is skipped and GDN_DEVICE_ERR_SEQLEN
 * is OR-ed into *err_flag; a slot outside [0, pool_slots) is handled as in
 * gdn_decode_step. Each named state is read once and written once (when n > 0).
 */
gdn_status gdn_spec_commit(const gdn_config* cfg, int32_t B, int32_t T, const int32_t* n_accept,
                           const uint16_t* qkv, uint16_t* conv_pool, float* state_pool, int32_t pool_slots,
                           const int32_t* slots, const float* spec_k, const float* spec_delta,
                           const float* spec_alpha, int32_t* err_flag, void* stream);

/*
 * gdn_decode_step for callers that cannot allocate device memory. The pages have
 * no counterpart of this entry point; it exists for the library's users.
 *
 * Some callers cannot provide even the small workspace of gdn_decode_step: code
 * that runs inside a host framework which owns the device allocator, plugins with a
 * fixed memory budget, or latency-critical paths that must not call cudaMalloc
 * (which can synchronize the device). This entry point takes the same arguments as
 * gdn_decode_step without `workspace`, allocates nothing (no cudaMalloc, cudaFree
 * or allocating library call) and uses a fixed scratch array that the library
 * itself places in device memory instead: gdn_decode_static_scratch_bytes() bytes
 * on every GPU that loads the library, held until the process exits.
 *   - The first call on a device looks up that array's device address once (with
 *     the device current); make that first call before any stream capture.
 *   - Each call clears the part of the array it needs with an asynchronous memset
 *     on `stream`, then launches as gdn_decode_step does. The results are the same.
 *   - All calls on a device share the one array, which keeps the last call's
 *     contents: calls that overlap on the GPU (other streams, other threads) race
 *     on it. Serialize them, or use gdn_decode_step with one workspace each.
 *   - If the scratch this build needs exceeds the array, the call returns
 *     GDN_ERR_UNSUPPORTED before doing anything.
 */
gdn_status gdn_decode_step_static_scratch(const gdn_config* cfg, int32_t B, int32_t T,
                                          const uint16_t* qkv, const uint16_t* a,
                                          const uint16_t* b, const uint16_t* z,
                                          const uint16_t* conv_w, const float* A_log,
                                          const float* dt_bias, const uint16_t* norm_w,
                                          uint16_t* conv_pool, float* state_pool,
                                          int32_t pool_slots, const int32_t* slots,
                                          uint16_t* out_bf16, float* out_f32, int32_t* err_flag,
                                          void* stream);

/* Size in bytes of the fixed scratch array of gdn_decode_step_static_scratch. */
size_t gdn_decode_static_scratch_bytes(void);

/*
 * ---------------------------------------------------------------------------------
 * The softmax-attention layers that alternate with GDN layers in a hybrid model, on a
 * paged key/value cache ("metrale_model_layers/forward/qwen3_5/full_attention.rs": the
 * per-head q/k RMSNorm, the rotary positions, the KV append, the decode attention and
 * the sigmoid output gate). The conventions above hold, with these additions.
 *
 * Cache. k_pages, v_pages [num_pages][page_size][Hkv][d], bf16 or e4m3, one pair per
 *   layer. page_table [table_rows][max_pages] int32 and seq_lens [table_rows] int32 are
 *   shared by all layers and indexed by SLOT like the GDN pools: the token at position
 *   p of slot s is row p % page_size of page page_table[s][p / page_size]. Entries that
 *   hold no page are -1, behind those that hold one. seq_lens[s] is the number of tokens stored BEFORE the step:
 *   gdn_qk_rope_append writes positions seq_lens[s] .. and gdn_attn_decode reads them
 *   too, and neither changes seq_lens, so every layer of the step sees the same lengths;
 *   the caller advances them once per step (by the accepted count after a speculative
 *   step: positions past seq_lens are rewritten by the next append, which is all that
 *   rewinding takes. A sequence that was forked, or is a fork, is not rewound below the
 *   last page boundary at or before the length that it then had: pages before that are
 *   shared, and an append to them would write into every holder's).
 * Rows. With cu_seqlens NULL sequence i owns T token rows i*T ..; otherwise T is the
 *   largest count (1..16) and sequence i owns rows cu_seqlens[i] .. cu_seqlens[i+1]-1,
 *   as in gdn_decode_step_varlen (0 tokens: left untouched, which also serves padded
 *   batches in a captured graph; counts or rows out of range: skipped,
 *   GDN_DEVICE_ERR_SEQLEN). total_tokens: rows of the packed tensors (B*T without
 *   cu_seqlens). A sequence whose slot is outside [0, table_rows) is skipped and
 *   flagged GDN_DEVICE_ERR_SLOT_RANGE, one whose length is negative or does not fit
 *   max_pages * page_size positions is skipped and flagged GDN_DEVICE_ERR_SEQLEN.
 *   A page number outside [0, num_pages) is flagged GDN_DEVICE_ERR_PAGE and neither
 *   read nor written. Slots of one gdn_qk_rope_append call are distinct (two sequences
 *   would write the same places); gdn_attn_decode may be given a slot twice.
 */
enum { GDN_KV_BF16 = 0, GDN_KV_E4M3 = 1 };

typedef struct {
    int32_t num_q_heads;      /* Hq, a multiple of Hkv, Hq/Hkv <= 16; query head h reads kv head h / (Hq/Hkv) */
    int32_t num_kv_heads;     /* Hkv */
    int32_t head_dim;         /* d: 64, 128 or 256 */
    int32_t rotary_dim;       /* R: the leading R dimensions of each head are rotated; even, 0..d */
    int32_t rope_interleaved; /* 0: pairs (i, i + R/2); 1: pairs (2i, 2i + 1) */
    int32_t page_size;        /* tokens per page, 1..65536 */
    int32_t kv_dtype;         /* GDN_KV_BF16 or GDN_KV_E4M3 */
    int32_t window;           /* 0: none; W: a token attends the last W positions, its own among them */
    float norm_eps;           /* epsilon of the q/k RMSNorm, inside the root */
    float norm_offset;        /* the norm's weight is norm_offset + w (0, or 1 for weights stored around zero) */
    float rope_scale;         /* factor on cos and sin (long-context scaling); 0 selects 1 */
    float sm_scale;           /* factor on q.k; 0 selects 1/sqrt(d) */
    float softcap;            /* 0: none; c: a score x becomes c tanh(x / c), off by c 2^-21 at most (c <= 64), else x 2^-20 */
    float k_scale, v_scale;   /* e4m3: a stored value times this is the value; 0 selects 1. bf16: 0 or 1 */
} gdn_attn_config;

typedef struct {
    void* k_pages; /* [num_pages][page_size][Hkv][d] */
    void* v_pages;
    int32_t num_pages;
    const int32_t* page_table; /* [table_rows][max_pages], 4-byte aligned */
    int32_t table_rows;
    int32_t max_pages;
    const int32_t* seq_lens; /* [table_rows], 4-byte aligned */
} gdn_kv_cache;

/* Heads of token rows that need not be contiguous (slices of one projection): element
 * (row, head, i) at ptr[row * row_stride + head * head_stride + i]. Strides in elements,
 * multiples of 8, not negative (0: one row or head for all); ptr 16-byte aligned. */
typedef struct {
    const uint16_t* ptr;
    int64_t row_stride;
    int64_t head_stride;
} gdn_heads;

/*
 * RMSNorm of each q and k head, rotary positions and the cache append, one launch:
 *   x <- x / sqrt(mean x^2 + norm_eps) * (norm_offset + w)        (w NULL: no norm)
 *   pair (x_i, x_j) at position p, angle p * inv_freq[i], c and s its cosine and sine
 *   times rope_scale: (x_i c - x_j s, x_j c + x_i s)
 *   q [rows][Hq][d], k, v [rows][Hkv][d]   bf16
 *   q_norm_w, k_norm_w [d] bf16            nullable
 *   inv_freq [R/2] fp32                    may be NULL when R = 0
 *   q_out [rows][Hq][d] bf16               contiguous
 * k and v go to the cache (e4m3: value / scale, saturated, round to nearest even). The
 * angle is formed and reduced in 64 bits, so positions of millions of tokens keep full
 * precision. A token whose page is flagged still gets its q_out row.
 */
gdn_status gdn_qk_rope_append(const gdn_attn_config* cfg, const gdn_kv_cache* cache, int32_t B, int32_t T,
                              const int32_t* cu_seqlens, int32_t total_tokens, const gdn_heads* q, const gdn_heads* k,
                              const gdn_heads* v, const uint16_t* q_norm_w, const uint16_t* k_norm_w,
                              const float* inv_freq, const int32_t* slots, uint16_t* q_out, int32_t* err_flag,
                              void* stream);

/*
 * Attention of the new tokens over the cache (theirs included: append first): one
 * launch, or two where a key/value head has many query rows T * Hq / Hkv (a bf16 cache with
 * a page_size that is a multiple of 8, more than 16, 32 or 64 rows at d = 256, 128 or 64:
 * products on the fifth-generation tensor cores and a second launch that joins the parts of
 * split sequences). Token t of a sequence at position p = seq_lens[slot] + t attends positions
 * 0..p (the last `window` of them): x = sm_scale q.k (capped), P = softmax(x),
 *   out = (sum_j P_j v_j) * sigmoid(gate)                          (gate NULL: no gate)
 *   lse [rows][Hq] fp32 nullable: the natural logarithm of the sum of exp(x)
 *   q, gate [rows][Hq][d] bf16; out [rows][Hq][d] bf16, contiguous
 *   workspace of gdn_attn_decode_workspace_bytes(cfg, B, T) bytes, zeroed by the caller
 *            once before its first use; every call leaves its counters zeroed again.
 *            Calls that may run at the same time on the GPU need separate workspaces;
 *            one that is large enough serves any configuration. After a call that
 *            raised GDN_DEVICE_ERR_TIMEOUT it has to be zeroed again, and the call's
 *            outputs are unspecified.
 * Values of keys and values past a sequence's end are never used (they may be NaN), and
 * a non-finite value of a later drafted token does not reach the rows before it. Pages
 * that lie wholly before every row's window are not read. B <= 2048, and B times a
 * sequence's places at most 2^31 - 2^16 (GDN_ERR_UNSUPPORTED): its places are Hkv x (row
 * tiles) x (token tiles + 13), of max_pages * page_size tokens (or window + T, if fewer) in
 * tiles of 8192 / (d * element bytes), and of T * Hq / Hkv rows in tiles of 8, 16, 32 or 64
 * (the smallest that holds them, else 64); with many rows tiles are 64 tokens by 128 rows
 * (rounded down to a multiple of Hq / Hkv). Results do not
 * depend on timing: the split of the work and the order of every sum follow from the
 * lengths alone. A sequence with a flagged page has unspecified outputs.
 */
gdn_status gdn_attn_decode(const gdn_attn_config* cfg, const gdn_kv_cache* cache, int32_t B, int32_t T,
                           const int32_t* cu_seqlens, int32_t total_tokens, const gdn_heads* q, const gdn_heads* gate,
                           const int32_t* slots, uint16_t* out, float* lse, int32_t* err_flag, void* workspace,
                           void* stream);

/* Bytes of the workspace of gdn_attn_decode for B sequences of up to T tokens (0 for a
 * configuration it refuses). They depend on head_dim, kv_dtype, page_size, Hq/Hkv and T. */
size_t gdn_attn_decode_workspace_bytes(const gdn_attn_config* cfg, int32_t B, int32_t T);

/*
 * Host: rotation speeds inv_freq[i], i < rotary_dim/2, for gdn_qk_rope_append and the
 * factor for gdn_attn_config.rope_scale.
 *   factor 1: theta^(-2i/R).   linear (yarn = 0): the same divided by factor.
 *   yarn = 1 (Peng et al., "YaRN", 2023): pairs that turn less than once over
 *   original_len tokens are divided by factor, those that turn more than 32 times are
 *   kept, a ramp in between; *rope_scale = 0.1 ln(factor) + 1 (1 otherwise).
 */
gdn_status gdn_rope_inv_freq_host(int32_t rotary_dim, double theta, double factor, int32_t yarn, int32_t original_len,
                                  float* inv_freq, float* rope_scale);

/*
 * Page tables kept on the device. page_refs [num_pages] int32 counts the table entries
 * that hold each page (0: free). A new page is always the lowest free one, given in the
 * order of the call's sequences, so tables are reproducible. Tables start as -1,
 * counters and lengths as 0. Slots of one call are distinct (children of a fork among
 * themselves and from all parents; one parent may appear many times). page_table,
 * seq_lens and page_refs are updated in place; copy lists are written in full.
 * A bad slot is skipped and flagged GDN_DEVICE_ERR_SLOT_RANGE, a bad length or count
 * GDN_DEVICE_ERR_SEQLEN, and GDN_DEVICE_ERR_PAGE flags a sequence that was skipped
 * because no free page was left for it (then every later one of the call that needs
 * pages is skipped too) or because its table row is in use.
 * n (sequences of a call) <= 2048, num_pages and max_pages < 2^31 - 2^15.
 *
 * reserve: gives slot i the pages for its next n_tokens[i] tokens (n_tokens NULL: T).
 * fork:    child dst[i] becomes a copy of parent src[i]: whole pages are shared, a
 *          partly filled last page is replaced by a new one, and copy_src[i], copy_dst[i]
 *          [n] say which page to copy where (-1, -1: none; a skipped child's copy_dst
 *          is -2). The child's row must be empty. Reserved pages past the parent's length are not inherited.
 * free:    releases every page of the rows and sets their lengths to 0 (a slot listed
 *          twice is released once).
 * compact: moves the pages in use to the front of the pool: copy_src, copy_dst
 *          [num_pages] get the *n_copies moves (the rest -1; sources and destinations
 *          never overlap), remap [num_pages] each page's new number (-1 for a free one),
 *          and every row of the table and the counters follow.
 */
gdn_status gdn_pages_reserve(int32_t page_size, int32_t n, const int32_t* slots, const int32_t* n_tokens, int32_t T,
                             int32_t* page_table, int32_t table_rows, int32_t max_pages, const int32_t* seq_lens,
                             int32_t* page_refs, int32_t num_pages, int32_t* err_flag, void* stream);
gdn_status gdn_pages_fork(int32_t page_size, int32_t n, const int32_t* src, const int32_t* dst, int32_t* page_table,
                          int32_t table_rows, int32_t max_pages, int32_t* seq_lens, int32_t* page_refs,
                          int32_t num_pages, int32_t* copy_src, int32_t* copy_dst, int32_t* err_flag, void* stream);
gdn_status gdn_pages_free(int32_t n, const int32_t* slots, int32_t* page_table, int32_t table_rows, int32_t max_pages,
                          int32_t* seq_lens, int32_t* page_refs, int32_t num_pages, int32_t* err_flag, void* stream);
gdn_status gdn_pages_compact(int32_t* page_table, int32_t table_rows, int32_t max_pages, int32_t* page_refs,
                             int32_t num_pages, int32_t* copy_src, int32_t* copy_dst, int32_t* n_copies,
                             int32_t* remap, int32_t* err_flag, void* stream);

/*
 * Copies rows of up to 64 buffers at once, one launch: for each pair i < n (n_dev
 * non-NULL: i < min(*n_dev, n)) row dst_ids[i] of every buffer becomes row src_ids[i].
 * A buffer is an array of `rows` rows of row_bytes bytes (a multiple of 16): the pages of
 * every layer's cache after a fork or a compaction, or the slots of the GDN state and
 * conv pools. Pairs with a negative id are skipped, ids >= rows are skipped and flagged
 * GDN_DEVICE_ERR_SLOT_RANGE (*n_dev outside [0, n]: GDN_DEVICE_ERR_BATCH, nothing
 * copied). Destinations are distinct and none is a source.
 */
typedef struct {
    void* base;
    int64_t row_bytes;
} gdn_copy_buffer;
gdn_status gdn_copy_rows(const gdn_copy_buffer* buffers, int32_t n_buffers, int32_t rows, int32_t n,
                         const int32_t* src_ids, const int32_t* dst_ids, const int32_t* n_dev, int32_t* err_flag,
                         void* stream);

/*
 * Self-test of the bounded waits inside every kernel of this library (the pages have no
 * counterpart): one GPU thread waits on a barrier phase that nothing completes, gives up
 * after limit_cycles cycles of its SM's clock (1 .. 2^40) and ORs GDN_DEVICE_ERR_TIMEOUT
 * into *err_flag (device int32, required). `cycles` (nullable, device uint64) receives
 * the cycles the wait took. Nothing else is touched; the context stays usable.
 */
gdn_status gdn_selftest_wait_timeout(uint64_t limit_cycles, int32_t* err_flag, uint64_t* cycles, void* stream);

/*
 * Host-side check of a HOST copy of slots[]: GDN_OK when all B values are distinct
 * and in [0, pool_slots), GDN_ERR_SLOT_RANGE otherwise, GDN_ERR_INVALID_ARGUMENT for
 * a null pointer or negative size. Touches no device.
 */
gdn_status gdn_check_slots_host(const int32_t* slots_host, int32_t B, int32_t pool_slots);

/* A static, human-readable name for a status code. */
const char* gdn_status_string(gdn_status status);

/* ABI version of this header: (major << 16) | minor. */
#define GDN_ABI_VERSION ((1 << 16) | 5)
int32_t gdn_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H_ */
