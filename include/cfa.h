/*
 * cfa.h -- C ABI of the cluster-fused decode-attention library (libcfa.so).
 *
 * One call runs one decode step of a decoder attention block for a batch of
 * B sequences on one GPU, in a single kernel launch:
 *
 *   1. QKV projection of the new token      qkv[b] = x[b] . W_qkv
 *   2. KV append                            k_cache[b,h,ctx_len] = k[b,h]
 *                                           v_cache[b,h,ctx_len] = v[b,h]
 *   3. single-query attention with a max-subtracted softmax over the
 *      ctx_len cached keys plus the new one (scale 1/sqrt(head_dim))
 *   4. output projection                    out[b] = concat_h(attn[b,h]) . W_o
 *
 * This is the decoder block of the page "ClusterFusion框架解析：LLM推理优化的集群
 * 通信革命" (ClusterFusion framework analysis): the three stages of its §1.1,
 * fused the way its §3.2 describes (one thread-block cluster per head, the
 * cluster's blocks splitting head_dim and the KV length, q/k/v shared by a
 * cluster gather and the softmax statistics and partial outputs combined by
 * cluster reductions over distributed shared memory, §3.1). The page merges
 * its partial output projections with atomicAdd; this library merges them in
 * a fixed head order instead, so results are bitwise reproducible.
 *
 * Conventions shared by every call:
 *   - All tensors are bf16 (IEEE binary32 with the low 16 bits dropped),
 *     dense, row-major, and live in device memory owned by the caller. All
 *     arithmetic accumulates in fp32. Results are rounded to bf16 with
 *     round-to-nearest-even.
 *   - Weights are [in, out] and applied as x . W (the page's
 *     torch.mm(hidden_states, W_qkv) form, §1.1):
 *       W_qkv [hidden, 3*hidden]: columns [0,H) are Q, [H,2H) K, [2H,3H) V;
 *                                 head h owns columns [h*d, (h+1)*d) of each.
 *       W_o   [hidden, hidden]:   row block [h*d, (h+1)*d) multiplies head h.
 *   - Caches are [B, n_heads, max_ctx, head_dim]. Positions [0, ctx_len) are
 *     read; position ctx_len is written; all other positions are neither read
 *     nor written.
 *   - Every device pointer must be 16-byte aligned. `out` must not overlap an
 *     input. ctx_len is shared by all B sequences.
 *   - Calls are asynchronous on the given CUDA stream (NULL = legacy default
 *     stream) unless stated otherwise. A plan owns a small device workspace,
 *     so one plan must not run concurrently on two streams; use one plan per
 *     stream.
 *   - Functions that return cfa_status never abort the process. Host-side
 *     argument checks happen before anything is launched; an error leaves
 *     every buffer untouched.
 *
 * Supported shapes: hidden == n_heads * head_dim, head_dim in {64, 128},
 * 1 <= B <= 16, hidden a multiple of 64, 1 <= max_ctx <= 1<<22. Other shapes
 * return CFA_ERR_UNSUPPORTED.
 */
#ifndef CFA_H
#define CFA_H

#ifdef __cplusplus
extern "C" {
#endif

typedef struct cfa_plan cfa_plan; /* opaque */

typedef enum cfa_status {
    CFA_OK = 0,
    CFA_ERR_INVALID_ARG = 1, /* NULL plan or pointer, ctx_len out of range, ... */
    CFA_ERR_UNSUPPORTED = 2, /* a shape or cluster size this build does not run */
    CFA_ERR_CUDA = 3,        /* a CUDA runtime call failed (no device, launch, ...) */
    CFA_ERR_TIMEOUT = 4,     /* a bounded device-side wait gave up (see cfa_plan_status) */
    CFA_ERR_ALIGNMENT = 5,   /* a pointer is not 16-byte aligned */
    CFA_ERR_NO_PAGES = 6     /* a page pool ran out (see cfa_paged_status) */
} cfa_status;

/*
 * Create a plan for batch B, hidden size `hidden` = n_heads * head_dim and a
 * cache capacity of max_ctx positions, on the current CUDA device.
 * Chooses the cluster size (blocks per head) and the pipeline depth: of the
 * sizes whose whole grid is resident on the GPU at once, the smallest whose
 * grid gives every SM a block, else the largest; if no size is co-resident,
 * the largest that runs. Sets the kernel attributes, and allocates the plan's workspace (fp32 per-head
 * output-projection partials [n_heads, B, hidden], arrival counters of the
 * cross-head merge, a status word, and device staging
 * for cfa_decode_step_host).
 * Returns NULL on failure; cfa_last_error() then says why.
 */
cfa_plan *cfa_plan_create(int B, int hidden, int n_heads, int head_dim, int max_ctx);

/* Release the plan and its workspace. Synchronizes the device first. NULL is a no-op. */
void cfa_plan_destroy(cfa_plan *plan);

/*
 * One decode step (steps 1-4 above), launched on `stream` (a cudaStream_t).
 *   x       bf16 [B, hidden]               read
 *   W_qkv   bf16 [hidden, 3*hidden]        read
 *   W_o     bf16 [hidden, hidden]          read
 *   k_cache bf16 [B, n_heads, max_ctx, head_dim]  rows [0,ctx_len) read, row ctx_len written
 *   v_cache bf16 [B, n_heads, max_ctx, head_dim]  same
 *   ctx_len number of cached positions before this token, 0 <= ctx_len < max_ctx
 *   out     bf16 [B, hidden]               written
 * Re-running a step with the same ctx_len rewrites the same cache row with
 * the same value, so a step is idempotent.
 * The step is one kernel launch, or two when the plan merges the heads'
 * partial output projections in a separate kernel (large batches; see
 * cfa_plan_describe).
 * Launch overlap (on by default, see cfa_plan_set_overlap): the step is
 * launched with programmatic stream serialization, so it may be scheduled
 * while the previous kernel on the stream is still running. Before that
 * kernel has finished it only initialises shared memory and prefetches
 * weight tiles; x and the caches are read, and every buffer is written, only
 * afterwards. The weights must therefore not be written by kernels still in
 * flight on the stream.
 * Errors: CFA_ERR_INVALID_ARG (NULL pointer, ctx_len out of range),
 * CFA_ERR_ALIGNMENT, CFA_ERR_CUDA (launch failure). Faults raised while the
 * kernel runs surface at the next synchronizing call, as with any CUDA kernel.
 */
cfa_status cfa_decode_step(cfa_plan *plan, const void *x, const void *W_qkv,
                           const void *W_o, void *k_cache, void *v_cache,
                           int ctx_len, void *out, void *stream);

/*
 * The decode step with one context length per sequence and, optionally, a
 * rotary position embedding of the new token's q and k. This widens the
 * page's block (which names no positional encoding, §1.1) toward a
 * Llama2-style layer:
 *   ctx_lens   host array [B]: cached positions of sequence b before this
 *              token, each in [0, max_ctx); row ctx_lens[b] of sequence b is
 *              written, rows [0, ctx_lens[b]) are read.
 *   rope_theta 0 disables the rotation; > 0 rotates dims i and i + d/2 of
 *              q and k_new by ctx_lens[b] * rope_theta^(-2i/d) (rotate-half
 *              form; e.g. 10000 for Llama2). Cached keys are taken as
 *              already rotated, and the appended k row is the rotated one.
 * Other arguments as cfa_decode_step, which equals this call with every
 * ctx_lens[b] = ctx_len and rope_theta = 0. Errors: CFA_ERR_INVALID_ARG
 * also for a NULL ctx_lens, a length out of range or a negative theta.
 */
cfa_status cfa_decode_step_ex(cfa_plan *plan, const void *x, const void *W_qkv,
                              const void *W_o, void *k_cache, void *v_cache,
                              const int *ctx_lens, double rope_theta, void *out,
                              void *stream);

/*
 * The same step for a caller whose token activations live in host memory:
 * takes x_host (bf16 [B, hidden]) to the GPU, runs the step of
 * cfa_decode_step on `stream`, brings the result back to out_host
 * (bf16 [B, hidden]) and synchronizes `stream` before returning. Weights and
 * caches stay device pointers. With page-locked, device-mapped host buffers
 * (cudaHostAlloc / cudaHostRegister, 16-byte aligned) there is no DMA
 * transfer: the step writes out_host itself, and reads x_host itself at
 * B <= 2 (at B >= 3 a small copy kernel first stages x in the plan's device
 * buffer, which the step's tensor-map loads read). Other host memory goes
 * through cudaMemcpyAsync and the plan's staging buffers, and is slower.
 * Errors as cfa_decode_step.
 */
cfa_status cfa_decode_step_host(cfa_plan *plan, const void *x_host, const void *W_qkv,
                                const void *W_o, void *k_cache, void *v_cache,
                                int ctx_len, void *out_host, void *stream);

/*
 * The same decode step for callers that cannot allocate device memory while
 * they run: engines whose device memory is owned and budgeted by a host
 * framework (plugins that receive only their input and output buffers), and
 * serving loops that forbid cudaMalloc after start-up because it may
 * synchronize the device and may fail under memory pressure. The paper has no
 * counterpart to this entry point; it exists only for such callers.
 *
 * No plan is involved: the shape is passed directly, with the same meaning,
 * limits and cluster-size choice as cfa_plan_create, and the arguments after
 * it mean what they mean for cfa_decode_step. Nothing is allocated: the
 * kernel's scratch (arrival counters, status word and the fp32 per-head
 * output-projection partials) lives in one fixed array inside the library,
 * 8 MiB + 16.25 KiB, which every GPU that loads the library keeps until the
 * process exits. Shapes with n_heads * B * hidden > 2^21 do not fit and
 * return CFA_ERR_UNSUPPORTED before anything is launched.
 *
 * The first call on a device sets the array up (looks up its device address
 * and zeroes its counters, synchronizing that device once); make that first
 * call before any stream capture. If that set-up fails (CFA_ERR_CUDA), the
 * device is not marked as set up and the next call tries again. Every call then clears the counters with an
 * asynchronous memset on `stream` and launches the kernel (and the separate
 * head merge, where the plan would use one) there, without launch overlap. All calls on a device share the one array, so calls whose
 * kernels may run at the same time on that device (other streams, other host
 * threads) race and must be serialized by the caller. Device-side wait
 * timeouts are not reported by this entry point.
 * Errors: as cfa_plan_create and cfa_decode_step.
 */
cfa_status cfa_decode_step_noalloc(int B, int hidden, int n_heads, int head_dim, int max_ctx,
                                   const void *x, const void *W_qkv, const void *W_o,
                                   void *k_cache, void *v_cache, int ctx_len, void *out,
                                   void *stream);

/*
 * Override the cluster size (thread blocks per head): 1, 2, 4, 8 or 16.
 * CFA_ERR_UNSUPPORTED if the shape does not split evenly at that size, the
 * device cannot co-schedule such a cluster, or its shared memory does not fit.
 * The plan is unchanged on error.
 */
cfa_status cfa_plan_set_cluster_size(cfa_plan *plan, int cluster_size);

/*
 * Override the pipeline depth (number of 16 KB shared-memory stages per
 * block); 0 restores the automatic choice. CFA_ERR_UNSUPPORTED if the shared
 * memory does not fit or the depth is outside [2, 64]. The plan is unchanged
 * on error.
 */
cfa_status cfa_plan_set_stages(cfa_plan *plan, int stages);

/*
 * How the blocks of a head's cluster share their partial q, k and v (the
 * ClusterGather step, CF section 3.1.2 "QKV向量共享"). mode 0: every block
 * sends its whole partial [B][3][64] to every peer and each sums all of them
 * (one round of pushes; the receive buffer holds C partials). mode 1:
 * reduce-scatter then all-gather -- each block sums one slice of the columns
 * over the blocks of its column group and sends the sum to every peer (two
 * rounds; the receive buffer holds 2 partials whatever C, which leaves more
 * shared memory for pipeline stages). Both sum in the same order, so the
 * results are bit for bit the same. mode -1 (the default): mode 1 where it
 * fits more blocks on an SM than mode 0, or, at the same blocks per SM,
 * gives more stages and either the batch runs its projections on the tensor
 * cores (B >= 3) or mode 0 leaves fewer than 4 stages; else mode 0.
 * CFA_ERR_INVALID_ARG for another mode; CFA_ERR_UNSUPPORTED if the layout
 * does not fit. The plan is unchanged on error.
 */
cfa_status cfa_plan_set_qkv_exchange(cfa_plan *plan, int mode);

/*
 * Enable (1, the default) or disable (0) launch overlap for the following
 * steps. With overlap on, a step's prologue and first weight loads run under
 * the tail of the previous kernel in the stream (see cfa_decode_step); with
 * it off, the step starts only after that kernel has finished.
 */
cfa_status cfa_plan_set_overlap(cfa_plan *plan, int enable);

/* Current cluster size of the plan, or -1 for NULL. */
int cfa_plan_cluster_size(const cfa_plan *plan);

/*
 * Write a one-line JSON description of the plan (shape, cluster size, grid,
 * block, shared memory per block, pipeline stages, stage bytes, co-resident
 * clusters, the form of the cross-head merge -- "flat": the last head to
 * finish a column chunk sums every head's partials inside the fused kernel;
 * "separate": a second kernel, launched behind it on the same stream, sums
 * them, chosen when the flat form would read more than 256 KB through one
 * block -- "launches_per_step", 1 or 2, and "qkv_exchange", "gather" or
 * "reduce_scatter") into buf (NUL-terminated, truncated to len).
 * CFA_ERR_INVALID_ARG for NULL arguments.
 */
cfa_status cfa_plan_describe(const cfa_plan *plan, char *buf, int len);

/*
 * The layout a plan of this shape would use with cluster size C on a device
 * with the given limits, computed on the host with no device, no allocation
 * and no CUDA call: the same arithmetic as cfa_plan_create and
 * cfa_plan_set_cluster_size after they have read the device's attributes
 * (num_sms = multiprocessor count; smem_per_sm, smem_optin, smem_reserved =
 * shared memory per multiprocessor, the per-block opt-in maximum and the
 * per-block reservation, in bytes). exchange and stages are as in
 * cfa_plan_set_qkv_exchange (-1 automatic) and cfa_plan_set_stages (0
 * automatic). C itself is the caller's: the plan's automatic choice also
 * needs the device's answer on how many clusters of each size fit at once.
 * Writes one JSON line into buf (len >= 256): cluster_size, grid,
 * blocks_per_sm (the blocks an SM is sized to hold), stages, smem_bytes,
 * qkv_exchange, tensor_cores (1: the projections run on tcgen05, B >= 3),
 * tmem_cols, proj_rows_per_block, proj_tile_rows, out_cols_per_block and
 * merge ("flat" or "separate"). Errors: shapes as cfa_plan_create;
 * CFA_ERR_INVALID_ARG for out-of-range limits, exchange, stages or buffer;
 * CFA_ERR_UNSUPPORTED when C does not divide the work or the layout does not
 * fit the shared memory.
 */
cfa_status cfa_plan_layout(int B, int hidden, int n_heads, int head_dim, int max_ctx, int C,
                           int exchange, int stages, int num_sms, int smem_per_sm,
                           int smem_optin, int smem_reserved, char *buf, int len);

/*
 * Device-side status of the plan: synchronizes the device, reads and clears
 * the status word the kernels set when a bounded wait gives up. CFA_OK when
 * nothing happened, CFA_ERR_TIMEOUT after a timed-out wait,
 * CFA_ERR_INVALID_ARG after a device-resident position out of range (layer
 * stack), CFA_ERR_CUDA if the read itself fails.
 */
cfa_status cfa_plan_status(cfa_plan *plan);

/* Status of the last failed call on this thread (plan creation included). */
cfa_status cfa_last_error(void);

/* Static, human-readable name of a status code. */
const char *cfa_status_string(cfa_status status);

/*
 * Self-test of the bounded-wait mechanism every in-kernel wait uses: launches
 * one block that waits on a shared-memory barrier nothing ever arrives on,
 * giving up after limit_us microseconds, then reports through a status word.
 * Synchronizes `stream`. Returns CFA_ERR_TIMEOUT when the wait gave up as it
 * must, CFA_OK if it (wrongly) completed, CFA_ERR_CUDA on a CUDA error.
 * limit_us must be in [1, 1<<20]. No GPU fault or hang is involved.
 */
cfa_status cfa_selftest_wait_timeout(int limit_us, void *stream);

/* ==========================================================================
 * Decoder layers around the attention block, and the multi-layer decode loop.
 *
 * The page reports time per output token of a whole Llama2-7B decoder
 * [§3.3, §5.1] but describes only the attention block of a layer (§1.1). The
 * rest of a layer follows the Llama2 arrangement (a reading, not the page):
 *
 *   xn = bf16( rmsnorm(x; attn_norm) )
 *   h  = bf16( x + attention_block(xn) )          (the fused step above)
 *   hn = bf16( rmsnorm(h; mlp_norm) )
 *   y  = bf16( h + (bf16(silu(hn . W_gate) * (hn . W_up))) . W_down )
 *
 * rmsnorm(v; g)_i = g_i v_i / sqrt(mean_j v_j^2 + eps), silu(z) = z/(1+e^-z).
 * Same conventions as above: bf16 row-major tensors in caller-owned device
 * memory, weights [in, out] applied as v . W, fp32 accumulation, 16-byte
 * aligned pointers, asynchronous on `stream`, fixed-order (bitwise
 * reproducible) reductions.
 * ========================================================================== */

typedef struct cfa_mlp cfa_mlp;     /* opaque */
typedef struct cfa_stack cfa_stack; /* opaque */

/*
 * y[b] = bf16(g * x[b] / sqrt(mean(x[b]^2) + eps)) for b < B; x, y [B, n],
 * g [n]. n a multiple of 8 in [8, 1<<20], B in [1, 65535], eps >= 0 finite;
 * y must not overlap x or g. CFA_ERR_INVALID_ARG / CFA_ERR_ALIGNMENT before
 * any launch, CFA_ERR_CUDA if the launch fails.
 */
cfa_status cfa_rmsnorm(int B, int n, const void *x, const void *g, float eps, void *y,
                       void *stream);

/*
 * Plan for the MLP half of a layer at batch B: hidden a multiple of 64
 * (<= 65536), ffn a multiple of 128 (<= 1<<18), 1 <= B <= 16
 * (CFA_ERR_UNSUPPORTED otherwise). Allocates the [B, ffn] SwiGLU buffer, the
 * fp32 split partials and arrival counters of its two GEMVs, and a status
 * word. NULL on failure; cfa_last_error() says why.
 */
cfa_mlp *cfa_mlp_create(int B, int hidden, int ffn);

/* Release the plan (synchronizes the device first). NULL is a no-op. */
void cfa_mlp_destroy(cfa_mlp *mlp);

/*
 * y = h + down(silu(gate(hn)) * up(hn)) with hn = bf16(rmsnorm(h; norm_w)):
 *   h, y [B, hidden]; norm_w [hidden]; W_gate, W_up [hidden, ffn];
 *   W_down [ffn, hidden].
 * Two kernel launches (RMSNorm + gate/up + SwiGLU; down + residual). y must
 * not overlap h, norm_w or a weight. One plan must not run on two streams at
 * once. Errors as cfa_rmsnorm.
 */
cfa_status cfa_mlp_step(cfa_mlp *mlp, const void *h, const void *norm_w, float eps,
                        const void *W_gate, const void *W_up, const void *W_down, void *y,
                        void *stream);

/*
 * Override the MLP kernels' occupancy (blocks per SM, 1..4) and pipeline depth
 * (16 KB stages per block, 2..12); 0 keeps the automatic choice. For sweeps.
 * CFA_ERR_UNSUPPORTED if it does not fit (the plan is then unchanged).
 */
cfa_status cfa_mlp_set_pipeline(cfa_mlp *mlp, int blocks_per_sm, int stages);

/*
 * Choose the kernel of the MLP's two GEMVs: path -1 = by batch size (the
 * tcgen05 tensor-core kernel from B = 2 on, the CUDA-core kernel at B = 1), 0 =
 * CUDA cores, 1 = tensor cores. The result is the same to within fp32
 * summation order. Keeps the pipeline overrides of cfa_mlp_set_pipeline.
 * CFA_ERR_INVALID_ARG for another path; CFA_ERR_UNSUPPORTED if the shape does
 * not fit the kernel (the plan is then unchanged).
 */
cfa_status cfa_mlp_set_path(cfa_mlp *mlp, int path);

/* Synchronizes, reads and clears the plan's device status word (as cfa_plan_status). */
cfa_status cfa_mlp_status(cfa_mlp *mlp);

/* One-line JSON description of the plan's two GEMVs (grid, units, stages, shared memory). */
cfa_status cfa_mlp_describe(const cfa_mlp *mlp, char *buf, int len);

/*
 * A stack of n_layers decoder layers (shapes as cfa_plan_create and
 * cfa_mlp_create) for the decode loop. Owns one attention plan, one MLP plan
 * and three [B, hidden] activation buffers; the layers' weights and caches
 * stay the caller's. NULL on failure; cfa_last_error() says why.
 */
cfa_stack *cfa_stack_create(int n_layers, int B, int hidden, int n_heads, int head_dim, int ffn,
                            int max_ctx);

/* Release the stack (synchronizes the device first). NULL is a no-op. */
void cfa_stack_destroy(cfa_stack *stack);

/*
 * Bind layer `layer` (0-based) to its weights and caches: attn_norm,
 * mlp_norm [hidden]; W_qkv [hidden, 3*hidden]; W_o [hidden, hidden]; caches
 * [B, n_heads, max_ctx, head_dim]; W_gate, W_up [hidden, ffn]; W_down
 * [ffn, hidden]. The pointers must stay valid while the stack is used.
 * Rebinding a layer invalidates a recorded graph (it is recorded again on
 * the next cfa_stack_step_graph).
 */
cfa_status cfa_stack_set_layer(cfa_stack *stack, int layer, const void *attn_norm,
                               const void *W_qkv, const void *W_o, void *k_cache, void *v_cache,
                               const void *mlp_norm, const void *W_gate, const void *W_up,
                               const void *W_down);

/*
 * One token through every layer: x [B, hidden] in, out [B, hidden] out (x and
 * out may be the same buffer). positions: device int [B], the cached length
 * of every sequence, read by each layer's attention kernel on the device
 * (so a recorded graph serves every position); each must lie in
 * [0, max_ctx - 1]. A value outside that range is not caught on the host: the
 * kernels flag it in the status word (cfa_stack_status then returns
 * CFA_ERR_INVALID_ARG), read no cache rows and append nothing for that
 * sequence. advance != 0 adds 1 to every position after the last layer (the
 * decode loop's next token). rope_theta > 0 rotates q and the new k as in
 * cfa_decode_step_ex; eps is the RMSNorm epsilon. All layers must be bound.
 * 4 kernels per layer (+1 with advance).
 */
cfa_status cfa_stack_step(cfa_stack *stack, const void *x, int *positions, double rope_theta,
                          float eps, int advance, void *out, void *stream);

/*
 * The same token step, recorded into a CUDA graph on the first call (and
 * again whenever x, out, positions, rope_theta, eps, advance, the stream or a
 * layer binding changes) and replayed with one graph launch afterwards.
 * `stream` must not be the legacy default stream (CFA_ERR_INVALID_ARG).
 */
cfa_status cfa_stack_step_graph(cfa_stack *stack, const void *x, int *positions,
                                double rope_theta, float eps, int advance, void *out,
                                void *stream);

/* Synchronizes and reads (and clears) the status of both plans of the stack. */
cfa_status cfa_stack_status(cfa_stack *stack);

/* One-line JSON description (layers, launches per token, both plans). */
cfa_status cfa_stack_describe(const cfa_stack *stack, char *buf, int len);

/* ==========================================================================
 * Multi-head latent attention (MLA), the DeepSeek variant the page adapts
 * ClusterFusion to: the latent key/value cache partitioned across clusters,
 * combined by a sparse cluster reduction (§5.2). The page gives no formula or
 * dimension; the block is DeepSeek-V2/V3's attention with their widths:
 * latent 512, per-head nope / rope / value 128 / 64 / 128 (fixed here).
 *
 * One step for B sequences at positions ctx_lens[b] (weights [in, out]):
 *   a   = bf16(x . W_a)                    W_a  [hidden, q_lora + 576]
 *   q   = bf16(bf16(rmsnorm(a[:q_lora]; g_q)) . W_uq)     W_uq [q_lora, n_heads*192]
 *         per head: [q_nope (128) | q_rope (64)]
 *   row = [bf16(rmsnorm(a[q_lora:q_lora+512]; g_kv)) | bf16(rope(a[q_lora+512:], L))]
 *         appended to the latent cache at L    cache [B, max_ctx, 576]
 *   per head h, with W_kvb [512, n_heads*256] holding per head [W_k (128) | W_v (128)]:
 *     keys    k_t = [c_t . W_k,h | k_rope_t], values v_t = c_t . W_v,h  (c_t = latent of row t)
 *     o_h     = softmax_t((q_nope . k_nope_t + rope(q_rope) . k_rope_t) / sqrt(192)) . v
 *   out = bf16(bf16(concat_h o_h) . W_o)   W_o  [n_heads*128, hidden]
 * rope is the rotate-half form of cfa_decode_step_ex over the 64 rope dims
 * (rope_theta 0 disables it); rmsnorm as cfa_rmsnorm. The attention runs in
 * absorbed form (q_nope folded into W_k, values projected after the sum), one
 * thread-block cluster per (sequence, group of 16 heads) -- or two or four,
 * each over its share of the latent rows ("row splits", §5.2's cache
 * partitioned across clusters), chosen per step when that grid still fits on
 * the GPU at once; the last of them to finish combines them in split order,
 * so a given shape's results are bitwise reproducible.
 * ========================================================================== */

typedef struct cfa_mla cfa_mla; /* opaque */

/*
 * Plan for batch B (1..16), hidden a multiple of 64, n_heads even (the
 * cluster holds the largest power-of-two group of heads up to 16 that divides
 * n_heads), q_lora a multiple of 64, max_ctx latent rows per sequence.
 * Allocates the intermediate a, q, v buffers, GEMV workspace and status words.
 * NULL on failure; cfa_last_error() says why.
 */
cfa_mla *cfa_mla_create(int B, int hidden, int n_heads, int q_lora, int max_ctx);

/* Release the plan (synchronizes the device first). NULL is a no-op. */
void cfa_mla_destroy(cfa_mla *mla);

/*
 * One MLA decode step (4 kernel launches). ctx_lens: host array [B], each in
 * [0, max_ctx - 1]; row ctx_lens[b] of the cache is written, rows below it are
 * read. out must not overlap x, the cache or W_o. Errors as cfa_decode_step.
 */
cfa_status cfa_mla_step(cfa_mla *mla, const void *x, const void *W_a, const void *g_q,
                        const void *g_kv, const void *W_uq, const void *W_kvb, const void *W_o,
                        void *cache, const int *ctx_lens, double rope_theta, float eps,
                        void *out, void *stream);

/* Synchronizes, reads and clears the plan's device status words. */
cfa_status cfa_mla_status(cfa_mla *mla);

/* One-line JSON description (cluster shape, row splits, grid, shared memory,
 * GEMV grids). */
cfa_status cfa_mla_describe(const cfa_mla *mla, char *buf, int len);

/*
 * Fix the number of row splits (1, 2 or 4 clusters per sequence and head
 * group, each over its share of the latent rows) for every later step; the
 * cluster size becomes the largest whose grid then fits on the GPU at once.
 * 0 restores the default, a choice per step: of the shapes that fit at once,
 * the one with the least estimated attention time for the step's longest
 * sequence (long contexts split further). Synchronizes the device first.
 * CFA_ERR_INVALID_ARG for other values; CFA_ERR_UNSUPPORTED if no cluster size
 * fits.
 */
cfa_status cfa_mla_set_row_splits(cfa_mla *mla, int splits);

/* ==========================================================================
 * Paged caches: block tables and slot maps built on the GPU, rotary embedding
 * with the append to the cache, and attention of a ragged batch over a prefix
 * that all its requests share and each request's own pages. A widening of the
 * page's block (§1.1, one contiguous cache per sequence) to batches whose
 * requests come and go, have several query tokens each (drafted tokens, prompt
 * chunks) and start with the same tokens.
 *
 * Cache layout: k_pages and v_pages are bf16 [n_pages, n_kv_heads, page_size,
 * head_dim]; row `off` of page `id` is slot id * page_size + off. A contiguous
 * cache [B, n_heads, max_ctx, head_dim] of the calls above is such a cache
 * with page_size = max_ctx and sequence b in page b (where max_ctx is an
 * allowed page size). n_heads is a multiple of n_kv_heads: query heads
 * [g G, (g + 1) G) read key head g, G = n_heads / n_kv_heads.
 *
 * Requests' lengths, offsets, tables and slots are device arrays (int32), read
 * by the kernels on the device, so that a recorded graph serves every step. A
 * value out of range is found there: it is flagged in the status word
 * (cfa_paged_status) and nothing is read or written out of bounds. Results are
 * bitwise reproducible. Conventions otherwise as above; integer arrays are
 * 4-byte aligned, the bf16 ones 16-byte aligned.
 *
 * A plan owns a workspace: one plan must not run on two streams at once, nor
 * in two graphs that may run at the same time. Calls are asynchronous: arrays live
 * until the stream has passed the call.
 * ========================================================================== */

typedef struct cfa_paged cfa_paged; /* opaque */

/*
 * Plan on the current device for at most max_seqs (1..1024) requests and
 * max_tokens (1..131072) new tokens per call. head_dim 64 or 128, n_heads <=
 * 1024, page_size 16, 32 or a multiple of 64 up to 1<<22
 * (CFA_ERR_UNSUPPORTED otherwise; CFA_ERR_INVALID_ARG for non-positive values
 * or n_heads not a multiple of n_kv_heads). No rotation until
 * cfa_paged_set_rope. With R = min(max_tokens G, 128 max_seqs) and G = n_heads /
 * n_kv_heads the workspace holds 2 n_kv_heads R + 512 SMs rows of head_dim + 2
 * floats, and the plan of a call 64 + 32 (SMs + R) bytes. NULL on failure;
 * cfa_last_error() says why.
 */
cfa_paged *cfa_paged_create(int max_seqs, int max_tokens, int n_heads, int n_kv_heads,
                            int head_dim, int page_size);

/* Release the plan (synchronizes its device first). NULL is a no-op. */
void cfa_paged_destroy(cfa_paged *paged);

/* Scaling of the rotary frequencies for long contexts. */
enum {
    CFA_ROPE_PLAIN = 0,    /* f_i = theta^(-2i / rotary_dim) */
    CFA_ROPE_LINEAR = 1,   /* f_i / factor */
    CFA_ROPE_BY_PARTS = 2  /* between f_i and f_i / factor by the turns in original_ctx */
};

/*
 * The rotation of the following cfa_paged_append and cfa_paged_layer calls:
 * pair i of the first rotary_dim dims of a head at position n turns by n f_i,
 * and its cosine and sine are multiplied by `magnitude` (1: a rotation). The
 * pair is dims (i, i + rotary_dim/2), or (2i, 2i + 1) where interleaved != 0;
 * dims from rotary_dim on pass through. rotary_dim is a multiple of 16 up to
 * head_dim; 0 turns the rotation off. scaling is one of the three above;
 * by parts, with r = original_ctx f_i / 2 pi turns over the original context
 * and g = clamp((r - low_turns) / (high_turns - low_turns), 0, 1), the
 * frequency is g f_i + (1 - g) f_i / factor: linear in the turns. Code that ramps
 * linearly in the pair's index i instead, between the indices at which a pair makes
 * high_turns and low_turns (rounded down and up), has other frequencies for the pairs
 * between, and no arguments here give those: check which of the two a checkpoint was
 * trained on. Needs theta >= 1, factor >= 1, 0 < magnitude <= 1e6, all finite, and by
 * parts 0 <= low_turns < high_turns and
 * original_ctx >= 1 (CFA_ERR_INVALID_ARG; a rotary_dim that is no multiple of
 * 16 or above head_dim: CFA_ERR_UNSUPPORTED). Held on the host: a recorded
 * graph keeps the rotation it was recorded with.
 */
cfa_status cfa_paged_set_rope(cfa_paged *paged, double theta, int rotary_dim, int interleaved,
                              int scaling, double factor, double low_turns, double high_turns,
                              int original_ctx, double magnitude);

/*
 * Tables and slot maps of one step, in one kernel. Request b has lens[b]
 * tokens in its pages and brings fresh[b] more (0 allowed):
 *   - it is given the pages it lacks: tables[b][j] for
 *     ceil(lens/page_size) <= j < ceil((lens + fresh)/page_size) are written with
 *     free_pages[pool[0]], free_pages[pool[0] + 1], ... in the order of b and j
 *     (free_pages [n_free]; pool[0] entries are taken so far, pool[1] <= n_free
 *     there are). Other table entries are not written; those below are read.
 *   - cu [n_seqs + 1] gets the first token row of every request and the total;
 *   - token i of request b, in row cu[b] + i, gets position
 *     base + lens[b] + i and slot id * page_size + (lens[b] + i) % page_size of its
 *     page; rows from the total up to n_slots get position 0 and slot -1;
 *   - lens_out [n_seqs] = lens + fresh, pool_out = {pool[0] + pages taken, pool[1]}
 *     (lens_out may be lens and pool_out may be pool; no other overlap).
 * A page id below 0 or with slots above 2^31 - 1 gives slot -1 and is flagged
 * (CFA_ERR_INVALID_ARG from cfa_paged_status). tables is [n_seqs, table_width]
 * (table_width <= 1<<18, table_width * page_size and base <= 1<<30, here and
 * below). All or nothing: a negative length or pool counter, a total above n_slots,
 * a request longer than table_width * page_size (then cfa_paged_status returns
 * CFA_ERR_INVALID_ARG) or too few free pages (CFA_ERR_NO_PAGES) leave the tables as
 * they were, lens_out = lens, pool_out = pool, every cu 0, every slot -1 and every
 * position 0.
 * Errors: CFA_ERR_INVALID_ARG (NULL, sizes out of the plan's range, overlaps),
 * CFA_ERR_ALIGNMENT, CFA_ERR_CUDA.
 */
cfa_status cfa_paged_tables(cfa_paged *paged, int n_seqs, int base, const int *lens,
                            const int *fresh, const int *free_pages, int n_free, const int *pool,
                            int *tables, int table_width, int *lens_out, int *pool_out, int *cu,
                            int *positions, int *slots, int n_slots, void *stream);

/*
 * Rotate q and k by positions [n_tokens] and put k and v into the cache, in
 * one kernel: q_out[t] = rotated q[t] (bf16 [n_tokens, n_heads, head_dim]),
 * row slots[t] of k_pages = rotated k[t], of v_pages = v[t]. q, k and v are
 * rows of heads (dense within a row) with strides of q_stride, k_stride and
 * v_stride elements (multiples of 8), so that they may be slices of one fused
 * projection. q_out may be q where q_stride = n_heads * head_dim; it must not
 * overlap q otherwise, nor k, v or the pages. Rows with a negative slot are
 * skipped: their q_out row stays as it was. A slot of n_pages * page_size or
 * more is skipped too and flagged (CFA_ERR_INVALID_ARG from cfa_paged_status).
 * Two tokens with the same slot leave in its row pieces of either. With
 * n_tokens 0 this call and the next two do nothing (pointers may then be NULL).
 */
cfa_status cfa_paged_append(cfa_paged *paged, int n_tokens, const void *q, long long q_stride,
                            const void *k, long long k_stride, const void *v, long long v_stride,
                            const int *positions, const int *slots, int n_pages, void *k_pages,
                            void *v_pages, void *q_out, void *stream);

/*
 * Attention of n_tokens query rows q (bf16, heads dense, row stride q_stride
 * elements) of n_seqs requests: rows [cu[b], cu[b + 1]) are the last tokens
 * of request b. Each attends every key of the prefix (prefix_len positions in
 * the pages prefix_table lists; may be 0) and, of the lens[b] keys in the pages
 * of tables[b] (its new tokens' own keys among them), those up to its own
 * position: row cu[b] + i sees lens[b] - (cu[b + 1] - cu[b]) + i + 1 of them.
 *   out  bf16 [n_tokens, n_heads, head_dim] = softmax(scale q . k) v; the weights
 *        are rounded to bf16 (to nearest) for the product with v, everything else
 *        up to the result is held in 32 bits
 *   lse  fp32 [n_tokens, n_heads], the natural logarithm of the sum of
 *        exp(scale q . k), or NULL
 * A row that sees no key gets 0 and lse -inf. Rows outside [cu[0], cu[n_seqs])
 * stay as they were. scale 0 means 1/sqrt(head_dim); scale times log2 e must be
 * finite in 32 bits. Keys and values that a row does not see do not change it,
 * whatever they hold, NaN included (values that are not finite and that only some of a
 * request's rows see take a slow pass behind the call). Flagged in the status word as CFA_ERR_INVALID_ARG: offsets cu that
 * are not ascending within [0, n_tokens], or more than some 2^27 blocks of
 * 128 keys over all key heads and tiles of 256 rows (nothing is written then); a
 * length outside [0, table_width * page_size] (taken as 0); a page id outside
 * [0, n_pages) where a key is read (its keys and values count as zeros).
 * out and lse must not overlap an input or each other.
 */
cfa_status cfa_paged_attention(cfa_paged *paged, int n_tokens, int n_seqs, const void *q,
                               long long q_stride, const int *cu, const int *prefix_table,
                               int prefix_len, const int *tables, int table_width,
                               const int *lens, int n_pages, const void *k_pages,
                               const void *v_pages, float scale, void *out, float *lse,
                               void *stream);

/*
 * The attention half of one layer: cfa_paged_append (q rotated into q_out,
 * which may be q), then cfa_paged_attention on q_out. Arguments as theirs; the
 * requests' rows and slots as cfa_paged_tables made them, once per step for all layers.
 * Nothing that the call writes may overlap cu, lens, tables or prefix_table, and out and
 * lse not positions or slots either.
 */
cfa_status cfa_paged_layer(cfa_paged *paged, int n_tokens, int n_seqs, const void *q,
                           long long q_stride, const void *k, long long k_stride, const void *v,
                           long long v_stride, const int *positions, const int *slots,
                           const int *cu, const int *prefix_table, int prefix_len,
                           const int *tables, int table_width, const int *lens, int n_pages,
                           void *k_pages, void *v_pages, float scale, void *q_out, void *out,
                           float *lse, void *stream);

/* Synchronizes, reads and clears the plan's device status word (as
 * cfa_plan_status; CFA_ERR_NO_PAGES after a refused cfa_paged_tables). */
cfa_status cfa_paged_status(cfa_paged *paged);

/* One-line JSON description (shape, rotation, SMs used, shared memory; on the
 * device, workspace_bytes of records and plan_bytes of a call's plan). */
cfa_status cfa_paged_describe(const cfa_paged *paged, char *buf, int len);

/* ==========================================================================
 * Paged latent caches: multi-head latent attention (the formulas and widths of
 * cfa_mla: latent 512, per head 128 unrotated + 64 rotated query dims, 128 value dims) for the
 * ragged batches of the paged caches. A cache row is a token's normed latent and
 * rotated key, 576 bf16, which all heads share:
 *   pages bf16 [n_pages, page_size, 576]; row `off` of page `id` is slot id * page_size + off,
 * so cfa_paged_tables of a plan with the same page_size makes tables, offsets, positions and
 * slots for it too. Per layer and step:
 *   cfa_latent_append     norm, rotation, rows into their slots; queries rotated
 *   decode, drafted tokens (absorbed form: a head's products with W_kvb on the query's side)
 *     cfa_latent_fold       queries into the latent space
 *     cfa_latent_attention  over the cached rows
 *     cfa_latent_unfold     results back to the value dims
 *   prompts (expanded form)
 *     cfa_latent_expanded   over keys and values that the caller has expanded (latents . W_kvb)
 * W_kvb is cfa_mla's: [512, n_heads * 256], per head [W_k (128) | W_v (128)]. Device arrays,
 * values out of range, alignment and streams as in the paged caches above (a plan's workspace
 * serves cfa_latent_attention and cfa_latent_expanded).
 * ========================================================================== */

typedef struct cfa_latent cfa_latent; /* opaque */

/*
 * Plan on the current device for at most max_seqs (1..1024) requests and max_tokens
 * (1..131072) new tokens per call, n_heads 1..1024, page_size 16, 32 or a multiple of 64 up
 * to 1<<22 (CFA_ERR_UNSUPPORTED otherwise; CFA_ERR_INVALID_ARG for non-positive values). No
 * rotation until cfa_latent_set_rope. The workspace holds the records of cut tiles, SMs x 128
 * rows of 512 + 4 floats. NULL on failure; cfa_last_error() says why.
 */
cfa_latent *cfa_latent_create(int max_seqs, int max_tokens, int n_heads, int page_size);

/* Release the plan (synchronizes its device first). NULL is a no-op. */
void cfa_latent_destroy(cfa_latent *latent);

/*
 * The rotation of the following cfa_latent_append and cfa_latent_layer calls, over the 64
 * rotated dims; arguments as cfa_paged_set_rope. theta 0 turns it off. magnitude multiplies the
 * rotated dims of queries and keys, so those dims' part of a score by its square. A model whose
 * magnitude belongs to the whole score, all 192 dims, has magnitude 1 here and the square of its own in
 * the attention's scale (magnitude^2 / sqrt(192)).
 */
cfa_status cfa_latent_set_rope(cfa_latent *latent, double theta, int interleaved, int scaling,
                               double factor, double low_turns, double high_turns,
                               int original_ctx, double magnitude);

/*
 * A token's cache row from the down projection's row a (576 bf16: latent, then the key to
 * rotate; rows a_stride elements apart) and its rotated queries:
 *   row = [bf16(rmsnorm(a[:512]; g_kv)) | bf16(rope(a[512:], positions[t]))] to slots[t]
 *   q_out[t, h] = [q[t, h, :128] | bf16(rope(q[t, h, 128:], positions[t]))]
 * q rows of n_heads * 192, q_stride elements apart (both strides multiples of 8); q_out
 * [n_tokens, n_heads, 192] may be q where q_stride = n_heads * 192 (then only the rotated
 * dims are touched), and must not overlap q otherwise. rmsnorm as cfa_rmsnorm; g_kv [512]; eps >= 0, finite.
 * Rows with a negative slot are skipped: their q_out row stays as it was. A slot of
 * n_pages * page_size or more is skipped too and flagged (CFA_ERR_INVALID_ARG from
 * cfa_latent_status). Two tokens with the same slot leave in its row pieces of either. With
 * n_tokens 0 this call and the next ones do nothing (pointers may then be NULL).
 */
cfa_status cfa_latent_append(cfa_latent *latent, int n_tokens, const void *a, long long a_stride,
                             const void *g_kv, float eps, const void *q, long long q_stride,
                             const int *positions, const int *slots, int n_pages, void *pages,
                             void *q_out, void *stream);

/*
 * Queries into the latent space: q_lat [n_tokens, n_heads, 576],
 *   q_lat[t, h] = [bf16(W_k,h . q[t, h, :128]) | q[t, h, 128:]]
 * q as cfa_latent_append wrote it (q_stride elements between tokens, a multiple of 8). fp32 sums.
 */
cfa_status cfa_latent_fold(cfa_latent *latent, int n_tokens, const void *q, long long q_stride,
                           const void *W_kvb, void *q_lat, void *stream);

/*
 * Results out of the latent space: out [n_tokens, n_heads, 128],
 *   out[t, h] = bf16(o_lat[t, h] . W_v,h), o_lat [n_tokens, n_heads, 512].
 */
cfa_status cfa_latent_unfold(cfa_latent *latent, int n_tokens, const void *o_lat,
                             const void *W_kvb, void *out, void *stream);

/*
 * Attention of folded queries q_lat [n_tokens, n_heads, 576] of n_seqs requests over their
 * cached rows: tokens [cu[b], cu[b + 1]) are the last of request b, whose lens[b] rows (its
 * new tokens' own among them) lie in the pages of tables[b]. Token cu[b] + i sees the first
 * lens[b] - (cu[b + 1] - cu[b]) + i + 1 of them.
 *   o_lat bf16 [n_tokens, n_heads, 512] = sum_j softmax_j(scale q_lat . row_j) row_j[:512];
 *         the weights are rounded to bf16 for the product with the rows, everything else up to the
 *         result is held in 32 bits
 *   lse   fp32 [n_tokens, n_heads], the natural logarithm of the sum of exp(scale q_lat . row_j),
 *         or NULL
 * A token that sees no row gets 0 and lse -inf. Tokens outside [cu[0], cu[n_seqs]) stay as
 * they were. scale 0 means 1/sqrt(192); scale times log2 e must be finite in 32 bits. Rows
 * that a token does not see do not change it, whatever they hold. A score that is NaN or +inf makes
 * its token's head NaN; whether a row with such values and score -inf (weight 0) does is not defined. Where all
 * scores are -inf the result is that of a token that sees no row, or NaN. Flagged in the status word
 * as CFA_ERR_INVALID_ARG: offsets cu that are not ascending within [0, n_tokens], or 2^30 - 1 units or
 * more, a tile of 128 of a request's token heads having two and one for each block of 128 rows that its
 * last token sees (nothing is written then); a length outside
 * [0, table_width * page_size] (taken as 0); a page id outside [0, n_pages) where a row is read
 * (it counts as zeros). o_lat and lse must not overlap an input or each other.
 */
cfa_status cfa_latent_attention(cfa_latent *latent, int n_tokens, int n_seqs, const void *q_lat,
                                const int *cu, const int *tables, int table_width,
                                const int *lens, int n_pages, const void *pages, float scale,
                                void *o_lat, float *lse, void *stream);

/*
 * Attention of prompts over expanded keys and values: request b has query tokens
 * [cu[b], cu[b + 1]) of q (n_heads * 192 a token, q_stride elements apart) and keys
 * [cu_k[b], cu_k[b + 1]) of kv [n_keys, n_heads, 256] (per head [key (128) | value (128)], rows
 * kv_stride elements apart: the product of normed latents with W_kvb) and k_rope (64 a key, shared by the
 * heads, rows k_rope_stride apart: cache rows from dim 512 on, for instance). Its query tokens
 * are the last of its keys' tokens: with n query tokens and L keys, token i sees the first
 * L - n + i + 1 keys.
 *   out bf16 [n_tokens, n_heads, 128], lse fp32 [n_tokens, n_heads] or NULL, as cfa_latent_attention
 *   computes them from k = [key | k_rope] and value, scale and unseen keys as there. Values that are not
 *   finite stay in their dim; where only some tokens of a request see one, a pass over the keys of the
 *   tokens beside them, behind the attention, adds it to those. An infinite value whose weight is 0 in 32 bits
 *   shows as infinity or NaN, one or the other by where its key lies. A key with score -inf and finite values
 *   has weight 0, and a token's head with no other keys gets 0 and lse -inf.
 * q_stride a multiple of 8, kv_stride and k_rope_stride too. A token that sees no key gets 0 and lse
 * -inf; tokens outside the requests stay as they were. Flagged (CFA_ERR_INVALID_ARG from
 * cfa_latent_status, nothing written): cu or cu_k that are not ascending within [0, n_tokens]
 * and [0, n_keys]. n_keys up to 1<<30; with 0 kv and k_rope may be NULL.
 */
cfa_status cfa_latent_expanded(cfa_latent *latent, int n_tokens, int n_keys, int n_seqs,
                               const void *q, long long q_stride, const void *kv,
                               long long kv_stride, const void *k_rope, long long k_rope_stride,
                               const int *cu, const int *cu_k, float scale, void *out, float *lse,
                               void *stream);

/*
 * The attention of one layer's decode step: cfa_latent_append (queries rotated into q_out,
 * which may be q), cfa_latent_fold to q_lat, cfa_latent_attention to o_lat, cfa_latent_unfold
 * to out [n_tokens, n_heads, 128]. Arguments as theirs. Nothing that the call writes may overlap what
 * a later part of it reads, but for these four arrays' own part.
 */
cfa_status cfa_latent_layer(cfa_latent *latent, int n_tokens, int n_seqs, const void *a,
                            long long a_stride, const void *g_kv, float eps, const void *q,
                            long long q_stride, const int *positions, const int *slots,
                            const int *cu, const int *tables, int table_width, const int *lens,
                            int n_pages, void *pages, const void *W_kvb, float scale, void *q_out,
                            void *q_lat, void *o_lat, float *lse, void *out, void *stream);

/* Synchronizes, reads and clears the plan's device status word (as cfa_plan_status). */
cfa_status cfa_latent_status(cfa_latent *latent);

/* One-line JSON description (shape, rotation, grid, shared memory, workspace_bytes). */
cfa_status cfa_latent_describe(const cfa_latent *latent, char *buf, int len);

#ifdef __cplusplus
}
#endif

#endif /* CFA_H */
