/*
 * edge_ops.h -- C ABI of the GB300 fused decode-seam operator library
 * (libedge_ops.so, sm_103a).
 *
 * Four operators from the fused decode seams of small transformer decoders:
 *   edge_qk_norm_rope  per-head QK-RMSNorm + rotary embedding prologue
 *   edge_add_rmsnorm   residual add followed by RMSNorm of the rounded sum
 *   edge_rmsnorm       RMSNorm, with or without a weight
 *   edge_glu_act       SiLU / tanh-GELU gated activation of a merged gate+up
 * Each op can write a static-scale FP8 E4M3 output instead of the activation
 * dtype.  Beside them: the rotary embedding alone, LayerNorm, quantization, the
 * QKV split with its KV-cache write, and what a paged KV cache needs next to
 * that write:
 *   edge_paged_attention   attention of new tokens over the cache's pages
 *   edge_*_axes            rotary positions with several axes
 *   edge_pages_*           copying, freeing, forking and compacting pages
 * And linear layers in 8 bits with a scale for each token and output channel:
 *   edge_*_q8              norm, gate and quantization that find the scale of
 *                          each row, and the matrix product that reads them
 *
 * Sources, by page and section:
 *   "thox-edge-ops v2: fused decode kernels for small models on THOX edge
 *     hardware": section 3 (tensor contract; R1 numerics; R2 conventions;
 *     R5 safety), section 5.1 (operators), section 5.4 (fused QK-norm+RoPE),
 *     section 5.5 (validation before pointer arithmetic).
 *   ninfer pull request "Register the text profile of ops::rmsnorm_rope ...":
 *     "Implementation" (out-of-place partial-rotary text profile) and the
 *     review (pass eps and theta, keep the shape dispatch inside the op).
 *   FlashRT "optimization-details": the static-scale FP8 fused kernels, the
 *     static calibration and the no-weight RMSNorm.
 *
 * Common contract (all entry points):
 *   - Every tensor pointer is a caller-owned CUDA device pointer to a dense,
 *     row-major (contiguous) array.  The library allocates nothing, caches
 *     no tensor, never synchronizes the device or the stream, and copies
 *     nothing between host and device.  Every call can be captured into a
 *     CUDA graph.
 *   - `stream` is a cudaStream_t, or NULL for the legacy default stream.
 *     The kernel is enqueued on it, and the call returns once it is enqueued.
 *   - `dt` is the activation dtype: EDGE_F32, EDGE_F16 or EDGE_BF16.  Norm
 *     weights have dtype `dt`.  The output dtype `out_dt` is either `dt` or
 *     EDGE_FP8_E4M3.
 *   - Arithmetic is fp32 with one rounding of each output, to nearest even
 *     (R1).  With an FP8 output, the fp32 result y is multiplied by
 *     `inv_scale` in fp32 and converted to E4M3 with saturation to +-448.
 *     Here inv_scale = 1 / scale, and scale = amax / 448 comes from a
 *     calibration pass.  `inv_scale` is ignored unless out_dt is FP8.
 *   - Validation happens before any pointer arithmetic or launch.  An
 *     invalid call launches nothing and returns a nonzero edge_status.  A
 *     call with zero rows or tokens returns EDGE_OK and launches nothing.
 *   - Pointers must be aligned to their element size (EDGE_ERR_ALIGN
 *     otherwise).  16-byte aligned tensors whose rows are multiples of 16
 *     bytes take the vectorized path; other valid layouts take a scalar GPU
 *     path.  There is never a CPU fallback.
 *   - An output may alias its input exactly (in place) where stated.  Any
 *     other overlap between a written buffer and another buffer is rejected
 *     with EDGE_ERR_ALIAS.  An FP8 output must not alias an input.
 *   - A launch failure returns EDGE_ERR_CUDA.  edge_last_cuda_error() then
 *     gives the cudaError_t of the calling thread's last failure.
 */
#ifndef EDGE_OPS_H
#define EDGE_OPS_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    EDGE_F32 = 0,
    EDGE_F16 = 1,
    EDGE_BF16 = 2,
    EDGE_FP8_E4M3 = 3, /* 8-bit results and operands: OCP E4M3 "fn", saturating */
    EDGE_INT8 = 4      /* 8-bit results and operands of the edge_*_q8 calls */
} edge_dtype;

typedef enum {
    EDGE_OK = 0,
    EDGE_ERR_NULL = 1,        /* a required pointer is NULL */
    EDGE_ERR_DTYPE = 2,       /* unknown dtype, or out_dt not dt / FP8 */
    EDGE_ERR_SHAPE = 3,       /* negative or inconsistent sizes */
    EDGE_ERR_ALIGN = 4,       /* a pointer not aligned to its element size */
    EDGE_ERR_ALIAS = 5,       /* a written buffer overlaps another buffer */
    EDGE_ERR_UNSUPPORTED = 6, /* valid but beyond this build's limits */
    EDGE_ERR_CUDA = 7,        /* the launch failed (see edge_last_cuda_error) */
    EDGE_ERR_VALUE = 8        /* bad scalar: eps, inv_scale, flag or enum */
} edge_status;

typedef enum {
    EDGE_ROPE_ROTATE_HALF = 0, /* pairs (j, j + rotary_dim/2), GPT-NeoX */
    EDGE_ROPE_INTERLEAVED = 1  /* pairs (2j, 2j + 1), GPT-J */
} edge_rope_layout;

typedef enum {
    EDGE_ACT_SILU = 0,     /* silu(g) = g / (1 + e^-g) */
    EDGE_ACT_GELU_TANH = 1 /* 0.5 g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) */
} edge_act;

/*
 * RMSNorm ("thox-edge-ops v2", section 5.1; FlashRT no-weight RMSNorm).
 *
 *   out[t, i] = x[t, i] * r_t * (w[i] + weight_offset),
 *   r_t = 1 / sqrt(mean_i(x[t, i]^2) + eps).
 *
 * x:    [rows, hidden] of dt.
 * w:    [hidden] of dt, or NULL for the no-weight form out = x * r.
 *       weight_offset 0 applies w directly (Llama).  weight_offset 1
 *       applies 1 + w in fp32 (Gemma, zero-centred weight).
 * out:  [rows, hidden] of out_dt.  out == x is allowed when out_dt == dt.
 * eps:  finite and >= 0; it sits inside the root.
 * Errors: NULL x/out; rows < 0 or hidden <= 0; eps or weight_offset invalid;
 * partial overlap.
 */
edge_status edge_rmsnorm(void* out, edge_dtype out_dt, const void* x, const void* w,
                         edge_dtype dt, int64_t rows, int64_t hidden, float eps,
                         int weight_offset, float inv_scale, void* stream);

/*
 * Fused residual-add RMSNorm ("thox-edge-ops v2", R1 and sections 5.1 and
 * 5.2; FlashRT residual_add_rms_norm_fp8_static).
 *
 *   residual[t, i] <- round_dt(fp32(x[t, i]) + fp32(residual[t, i]))
 *   out[t, i]       = RMSNorm(residual[t, :])[i]
 *
 * The sum is widened, added in fp32 and rounded once to dt.  The result is
 * bit-identical to an eager add of the two tensors.  The norm (same
 * arguments as edge_rmsnorm) is taken of the rounded sum.
 * x:        [rows, hidden] of dt (read).
 * residual: [rows, hidden] of dt (read, then overwritten with the sum).
 * out:      [rows, hidden] of out_dt.  out == x is allowed when out_dt == dt.
 *           out must not overlap residual.
 */
edge_status edge_add_rmsnorm(void* out, edge_dtype out_dt, const void* x, void* residual,
                             const void* w, edge_dtype dt, int64_t rows, int64_t hidden,
                             float eps, int weight_offset, float inv_scale, void* stream);

/*
 * Gated activation of a merged gate+up projection ("thox-edge-ops v2",
 * section 5.1; FlashRT gate_geglu_merged_fp8).
 *
 *   out[t, i] = act(gate_up[t, i]) * gate_up[t, d + i],  0 <= i < d
 *
 * The gate is the first half of each row and the up projection the second.
 * gate_up: [rows, 2*d] of dt.   out: [rows, d] of out_dt (no overlap).
 * act: EDGE_ACT_SILU or EDGE_ACT_GELU_TANH.
 */
edge_status edge_glu_act(void* out, edge_dtype out_dt, const void* gate_up, edge_dtype dt,
                         int64_t rows, int64_t d, edge_act act, float inv_scale, void* stream);

/*
 * Fused per-head QK-RMSNorm + RoPE prologue ("thox-edge-ops v2", sections
 * 5.1 and 5.4; ninfer text profile, "Implementation").
 *
 * For every token t and every head h of q (weight wq) and of k (weight wk):
 *   m = round_dt(RMSNorm(head) with the head's weight)   (as edge_rmsnorm)
 *   if 0 <= positions[t] < cache_len, rotate the first rotary_dim channels
 *   of m.  For pair j < rotary_dim/2 with members (a, b), c = cos[p, j] and
 *   s = sin[p, j]:
 *        a' = a c - b s,   b' = b c + a s   (fp32, then one rounding)
 *   Channels at or past rotary_dim carry m.  A token whose position is
 *   negative or >= cache_len is normalized but not rotated, and no cache row
 *   at that position is read (R5), so no device synchronization is needed:
 *   every cache read lies inside [0, cache_len).
 *
 * q, k:        [tokens, q_heads, head_dim] and [tokens, k_heads, head_dim]
 *              of dt.  This is the innermost-first [head_dim, heads, tokens]
 *              of the ninfer profile.
 * q_out,k_out: same shapes, of out_dt.  q_out == q and k_out == k are allowed
 *              (in place) when out_dt == dt.
 * wq, wk:      [head_dim] of dt each, or NULL for unit weight.
 * rotary_dim:  even, 0 <= rotary_dim <= head_dim (0: no rotation).
 * layout:      EDGE_ROPE_ROTATE_HALF or EDGE_ROPE_INTERLEAVED.
 * positions:   [tokens] int64, device.  It may be NULL only if rotary_dim == 0
 *              or cache_len == 0.
 * cos, sin:    [cache_len, rotary_dim/2] fp32, device.  Row p holds the
 *              angles of position p, so theta is the caller's.  They may be
 *              NULL only if rotary_dim == 0 or cache_len == 0.
 * The FP8 epilogue quantizes the rotated value and the rounded m of the
 * channels that do not rotate.
 */
edge_status edge_qk_norm_rope(void* q_out, void* k_out, edge_dtype out_dt, const void* q,
                              const void* k, const void* wq, const void* wk, edge_dtype dt,
                              int64_t tokens, int32_t q_heads, int32_t k_heads, int32_t head_dim,
                              int32_t rotary_dim, edge_rope_layout layout,
                              const int64_t* positions, const float* cos, const float* sin,
                              int64_t cache_len, float eps, int weight_offset, float inv_scale,
                              void* stream);

/*
 * One-read LayerNorm (FlashRT "optimization-details": siglip_layernorm_1read,
 * a single pass over a register-cached row instead of three).
 *
 *   out[t, i] = (x[t, i] - mu_t) / sqrt(var_t + eps) * gamma[i] + beta[i]
 *   mu_t = mean_i x[t, i],  var_t = mean_i (x[t, i] - mu_t)^2  (biased)
 *
 * x: [rows, hidden] of dt.  gamma, beta: [hidden] of dt, each nullable (1, 0).
 * out: [rows, hidden] of out_dt; out == x is allowed when out_dt == dt.
 * fp32 arithmetic, one rounding (or the FP8 epilogue).
 */
edge_status edge_layernorm(void* out, edge_dtype out_dt, const void* x, const void* gamma,
                           const void* beta, edge_dtype dt, int64_t rows, int64_t hidden,
                           float eps, float inv_scale, void* stream);

/*
 * Standalone static-scale FP8 quantization (FlashRT "optimization-details":
 * quantize_fp8_static).  out[i] = E4M3(fl32(x[i]) * inv_scale), to nearest
 * even with saturation to +-448.  x: n elements of dt.  out: n bytes, which
 * must not overlap x.  inv_scale must be finite and > 0.
 */
edge_status edge_quantize_fp8(void* out, const void* x, edge_dtype dt, int64_t n, float inv_scale,
                              void* stream);

/*
 * Fused QKV split + QK-norm + RoPE + KV-cache write (FlashRT
 * "optimization-details": qkv_split_rope_kvcache; "thox-edge-ops v2",
 * roadmap item 4: a KV write fused into the prologue).
 *
 * qkv:   [tokens, (q_heads + 2 kv_heads) head_dim] of dt.  Row t holds q_heads
 *        query heads, then kv_heads key heads, then kv_heads value heads
 *        (the output of a fused QKV projection).
 * q_out: [tokens, q_heads, head_dim] of dt: the query heads after the prologue
 *        of edge_qk_norm_rope (per-head RMSNorm when normalize = 1, rounded to
 *        dt; the rotation of the first rotary_dim channels by cos/sin row
 *        positions[t]).
 * k_cache, v_cache: [num_slots, kv_heads, head_dim] of dt.  Row slots[t]
 *        receives the key heads of token t after the same prologue, and the
 *        value heads unchanged.  A token whose slot is negative or
 *        >= num_slots writes no cache row, so the cache is never written out
 *        of bounds; the other rows are left untouched.  When two tokens name
 *        the same slot, which token's row remains there is unspecified.
 * slots: [tokens] int64, device.  Caches and slots may be NULL when
 *        kv_heads == 0 or num_slots == 0.
 * slots == NULL with num_slots == 0 writes no cache row at all (the query
 * heads are still produced).
 * Output dtype is dt (no FP8 epilogue).  Outputs must not overlap each other
 * or any input.  Element-aligned tensors of any head size up to 2048 are
 * served: a vector path when head_dim * size(dt) is a power-of-two multiple
 * of 16 up to 512 bytes, the tensors are 16-byte aligned and the rotary width
 * suits 16-byte vectors, else a scalar path.  EDGE_ERR_UNSUPPORTED: head_dim
 * above 2048, or tokens * (q_heads + 2 kv_heads) above 2^31 - 1.
 */
edge_status edge_qkv_rope_cache(void* q_out, void* k_cache, void* v_cache, const void* qkv,
                                const void* wq, const void* wk, edge_dtype dt, int64_t tokens,
                                int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                int32_t rotary_dim, edge_rope_layout layout,
                                const int64_t* positions, const float* cos, const float* sin,
                                int64_t cache_len, const int64_t* slots, int64_t num_slots,
                                float eps, int weight_offset, int normalize, void* stream);

/* Flags of edge_qk_norm_rope_ex. */
enum {
    /* Rotate the fp32 normalized value and round once after the rotation,
     * instead of rotating its rounding to dt.  This is the variant the
     * ninfer review asks for (item 1).  Channels that do not rotate are
     * unchanged (they carry round_dt of the normalized value either way). */
    EDGE_QK_ROTATE_UNROUNDED = 1
};

/*
 * edge_qk_norm_rope with option flags (EDGE_QK_* above; 0 gives exactly
 * edge_qk_norm_rope).  Unknown flags return EDGE_ERR_VALUE.
 */
edge_status edge_qk_norm_rope_ex(void* q_out, void* k_out, edge_dtype out_dt, const void* q,
                                 const void* k, const void* wq, const void* wk, edge_dtype dt,
                                 int64_t tokens, int32_t q_heads, int32_t k_heads,
                                 int32_t head_dim, int32_t rotary_dim, edge_rope_layout layout,
                                 const int64_t* positions, const float* cos, const float* sin,
                                 int64_t cache_len, float eps, int weight_offset, float inv_scale,
                                 uint32_t flags, void* stream);

/*
 * Standalone rotary embedding ("thox-edge-ops v2", section 5.1, the rotary
 * operator: query and key in one launch).  For every head of q and k of token
 * t with 0 <= positions[t] < cache_len, pair j < rotary_dim/2 (rotate-half or
 * interleaved, as in edge_qk_norm_rope) becomes a' = a c - b s, b' = b c + a s
 * in fp32, rounded once (or the FP8 epilogue).  Other channels, and every
 * channel of a token outside the cache, are copied unchanged.  Same layout,
 * aliasing and error rules as edge_qk_norm_rope, with no weights and no eps.
 */
edge_status edge_rope(void* q_out, void* k_out, edge_dtype out_dt, const void* q, const void* k,
                      edge_dtype dt, int64_t tokens, int32_t q_heads, int32_t k_heads,
                      int32_t head_dim, int32_t rotary_dim, edge_rope_layout layout,
                      const int64_t* positions, const float* cos, const float* sin,
                      int64_t cache_len, float inv_scale, void* stream);

/* How the pairs of a rotary embedding with several axes belong to the axes. */
typedef enum {
    EDGE_AXES_BLOCKS = 0, /* sections[0] pairs of axis 0, then those of axis 1, ... */
    EDGE_AXES_CYCLED = 1  /* dealt in turn: pair j to axis j mod axes while that axis has
                           * pairs left (j / axes < sections[j mod axes]), else to axis 0 */
} edge_axis_order;

/*
 * Rotary positions with several axes (time, height and width of images and
 * video; text tokens carry the same position on every axis).  The forms of
 * edge_qk_norm_rope_ex, edge_rope and edge_qkv_rope_cache in which pair j of
 * the rotary channels turns by cos/sin row positions[axis(j)][t], column j.
 *
 * positions: [axes, tokens] int64, device.  A token with any of its positions
 *            negative or >= cache_len does not rotate, and no cache row is read
 *            for it.
 * axes:      1 to 4.
 * sections:  [axes] pairs of each axis, HOST memory, read during the call;
 *            together rotary_dim / 2.  EDGE_AXES_CYCLED needs every pair of the
 *            axes behind the first to exist: (sections[a] - 1) * axes + a <
 *            rotary_dim / 2.
 * Otherwise the arguments, results and errors of the forms with one position;
 * equal positions on every axis give the same values (up to the rounding of the
 * normalized head, where the two forms take different kernels).  EDGE_ERR_NULL:
 * sections NULL.  EDGE_ERR_SHAPE: axes or sections that do not fit.  EDGE_ERR_VALUE: an
 * unknown order.
 */
edge_status edge_qk_norm_rope_axes(void* q_out, void* k_out, edge_dtype out_dt, const void* q,
                                   const void* k, const void* wq, const void* wk, edge_dtype dt,
                                   int64_t tokens, int32_t q_heads, int32_t k_heads,
                                   int32_t head_dim, int32_t rotary_dim, edge_rope_layout layout,
                                   const int64_t* positions, int32_t axes, const int32_t* sections,
                                   edge_axis_order order, const float* cos, const float* sin,
                                   int64_t cache_len, float eps, int weight_offset,
                                   float inv_scale, uint32_t flags, void* stream);
edge_status edge_rope_axes(void* q_out, void* k_out, edge_dtype out_dt, const void* q,
                           const void* k, edge_dtype dt, int64_t tokens, int32_t q_heads,
                           int32_t k_heads, int32_t head_dim, int32_t rotary_dim,
                           edge_rope_layout layout, const int64_t* positions, int32_t axes,
                           const int32_t* sections, edge_axis_order order, const float* cos,
                           const float* sin, int64_t cache_len, float inv_scale, void* stream);
edge_status edge_qkv_rope_cache_axes(void* q_out, void* k_cache, void* v_cache, const void* qkv,
                                     const void* wq, const void* wk, edge_dtype dt, int64_t tokens,
                                     int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                     int32_t rotary_dim, edge_rope_layout layout,
                                     const int64_t* positions, int32_t axes,
                                     const int32_t* sections, edge_axis_order order,
                                     const float* cos, const float* sin, int64_t cache_len,
                                     const int64_t* slots, int64_t num_slots, float eps,
                                     int weight_offset, int normalize, void* stream);

/*
 * Attention of a chunk of new tokens over a paged KV cache (the reader of the
 * cache that edge_qkv_rope_cache writes).  A chunk of one token per sequence is
 * the decode step; causal = 0 is cross attention to cached states of any
 * length.
 *
 * Sequence b has lens[b] keys in the cache.  Its new tokens are the rows
 * [q_starts[b], q_starts[b + 1]) of q, n of them, and they are the last n of
 * its positions: query i sits at position lens[b] - n + i.  Key j of the
 * sequence is in slot block_table[b][j / page_size] * page_size + j % page_size.
 * For query head h, which reads key head h / (q_heads / kv_heads):
 *   s_j   = scale * (q . k_j)  over the keys the query sees,
 *   out   = sum_j softmax(s)_j v_j,   lse = ln(sum_j e^(s_j)).
 * A query sees key j when 0 <= j < lens[b], the page number is inside
 * [0, num_slots / page_size), and, if causal, j <= its position and (window
 * > 0) position - j < window.  What the cache holds at other keys does not
 * matter.  A query that sees no key, or only keys of score -infinity, gives
 * out 0 and lse -infinity; NaN and infinities in the query and in the keys and
 * values that it sees reach its row.
 *
 * q:           [tokens, q_heads, head_dim] of dt.
 * k_cache, v_cache: [num_slots, kv_heads, head_dim] of dt (NULL allowed when
 *              num_slots == 0).
 * out:         [tokens, q_heads, head_dim] of out_dt.  Rows that belong to no
 *              sequence are left as they were (in lse as well).
 * lse:         [tokens, q_heads] fp32, or NULL.
 * block_table: [num_seqs, max_pages] int32.   lens: [num_seqs] int32, clamped
 *              to [0, max_pages * page_size].
 * q_starts:    [num_seqs + 1] int32, not decreasing, inside [0, tokens]
 *              (values outside are clamped); NULL for one token per sequence,
 *              with tokens == num_seqs.
 * scale:       finite and > 0.  window: 0 for none; 0 when causal == 0.
 * workspace:   device memory of at least edge_paged_attention_workspace bytes,
 *              16-byte aligned, overwritten by the call.  It needs no clearing
 *              and holds nothing between calls; calls that may run at the same
 *              time need one each.
 * Scores, maxima, sums and outputs are held in fp32.  16-bit calls round the
 * weights to dt for the product with the values; with at most 16 packed rows
 * (tokens * q_heads / kv_heads) per sequence on average, sequences of at most 8
 * keep what that rounding leaves over as well.  The output is rounded once.
 * Results are the same from run to run.  Waits inside the kernel are limited to
 * two seconds; should one run out, which correct operation never does, the rows
 * that it concerns (out and lse) are NaN.
 * One kernel serves all sequences of a call, chosen by their average number of
 * rows; a short chunk among many decode tokens does better in a call of its own.
 * EDGE_ERR_SHAPE: q_heads not a multiple of kv_heads, or a workspace that is
 * too small.  EDGE_ERR_UNSUPPORTED: head_dim above 256, or tokens * q_heads or
 * max_pages * page_size above 2^30.
 */
edge_status edge_paged_attention(void* out, edge_dtype out_dt, float* lse, const void* q,
                                 const void* k_cache, const void* v_cache, edge_dtype dt,
                                 int64_t tokens, int32_t q_heads, int32_t kv_heads,
                                 int32_t head_dim, int64_t num_slots, int32_t page_size,
                                 const int32_t* block_table, int32_t num_seqs, int32_t max_pages,
                                 const int32_t* lens, const int32_t* q_starts, float scale,
                                 int causal, int32_t window, float inv_scale, void* workspace,
                                 int64_t workspace_bytes, void* stream);

/*
 * Bytes of workspace that edge_paged_attention needs on the current device for
 * any number of tokens, sequences and keys; -1 for arguments that it refuses.
 */
int64_t edge_paged_attention_workspace(edge_dtype dt, int32_t q_heads, int32_t kv_heads,
                                       int32_t head_dim);

/*
 * Pages of a KV cache.  A pool of num_pages pages is common to num_caches caches
 * (the key and value caches of every layer); page p of a cache is its bytes
 * [p * page_bytes, (p + 1) * page_bytes), that is slots [p * page_size, (p + 1)
 * * page_size).  Sequence b holds the pages named in row b of block_table
 * (entries outside [0, num_pages) name none), and refs[p] counts the entries
 * that name page p; a page is free when refs[p] <= 0.
 *
 * caches:      [num_caches] device pointers in HOST memory, read during the
 *              call, of any alignment (16-byte aligned caches and pages take the
 *              vector path).  num_caches = 0 moves no data.
 * block_table: [num_seqs, max_pages] int32.   lens: [num_seqs] int32.
 * refs:        [num_pages] int32.   All index arrays are device memory.
 * Written buffers must not overlap each other or any other buffer.  Results do
 * not depend on timing.  EDGE_ERR_UNSUPPORTED: page_bytes of 2^31 or more, or
 * more than 2^31 pieces of 1024 bytes in one cache's moves.  Numbers from the
 * device are checked there: no call reads or writes outside its buffers.
 *
 * edge_pages_copy copies page src[i] to page dst[i] in every cache, for i < n.
 *   Pairs with a page outside the pool, or with src[i] == dst[i], are passed
 *   over.  Of the other pairs with the same destination the last is carried
 *   out, and a pair whose source is the destination of another is not.  Pairs
 *   are held against each other, which takes n^2 steps: calls of some thousand
 *   pairs each do better than one of many.
 * EDGE_ERR_UNSUPPORTED: n above 65536.
 */
edge_status edge_pages_copy(void* const* caches, int32_t num_caches, int64_t page_bytes,
                            int32_t num_pages, const int32_t* src, const int32_t* dst, int32_t n,
                            void* stream);

/*
 * edge_pages_free gives back the pages of the sequences seqs[i], i < n: every
 *   entry of the row is taken out (-1) and its page's count lowered, and the
 *   length becomes 0.  Numbers outside [0, num_seqs) are passed over, and a
 *   sequence that is named twice is freed once.
 */
edge_status edge_pages_free(int32_t* block_table, int32_t num_seqs, int32_t max_pages,
                            int32_t* lens, int32_t* refs, int32_t num_pages, const int32_t* seqs,
                            int32_t n, void* stream);

/*
 * edge_pages_fork makes sequence children[i] a copy of parents[i], for i < n:
 *   it shares the parent's full pages (their counts are raised), and a last page
 *   that is filled in part is copied, in every cache, into the lowest free page;
 *   forks take pages in the order of i.
 * status: [n]: 0 forked; 1 no free page was left (the child stays as it was);
 *         2 refused: a number outside [0, num_seqs), a child whose row holds a
 *         page or whose length is not 0, or a child that the call names as a
 *         parent or earlier as a child.
 * pairs:  [2 n]: source and destination of each page copied, -1 -1 where none.
 * lens are read clamped to [0, max_pages * page_size].
 * EDGE_ERR_UNSUPPORTED: n above 8192, or max_pages * page_size above 2^30.
 */
edge_status edge_pages_fork(void* const* caches, int32_t num_caches, int64_t page_bytes,
                            int32_t num_pages, int32_t page_size, int32_t* block_table,
                            int32_t num_seqs, int32_t max_pages, int32_t* lens, int32_t* refs,
                            const int32_t* parents, const int32_t* children, int32_t n,
                            int32_t* status, int32_t* pairs, void* stream);

/*
 * edge_pages_compact moves the L pages in use to the first L numbers: the k-th
 *   page in use from L on moves to the k-th free page below L, in every cache.
 *   block_table_out and refs_out (each may be its input) receive the table with
 *   the new numbers (entries that name a free page become -1, entries outside
 *   the pool stay) and the counts.
 * workspace: at least edge_pages_compact_workspace(num_pages) bytes, 16-byte
 *   aligned.  After the call its first num_pages int32 hold the new number of
 *   each page, -1 for a page that was free.
 */
edge_status edge_pages_compact(void* const* caches, int32_t num_caches, int64_t page_bytes,
                               int32_t num_pages, int32_t* block_table_out,
                               const int32_t* block_table, int32_t num_seqs, int32_t max_pages,
                               int32_t* refs_out, const int32_t* refs, void* workspace,
                               int64_t workspace_bytes, void* stream);
int64_t edge_pages_compact_workspace(int32_t num_pages);

/*
 * Rows in 8 bits with a scale for each row (token), found from the row itself: the
 * inputs of edge_matmul_q8.  code[t, i] * scales[t] stands for the value.
 *
 *   edge_rmsnorm_q8, edge_add_rmsnorm_q8:  p_i = s_i (w[i] + weight_offset), s = x or
 *       the rounded sum x + residual, which replaces residual
 *   edge_glu_act_q8:   p_i = act(gate_up[t, i]) * gate_up[t, n + i]
 *   edge_quantize_q8:  p_i = x[t, i]
 *   m = max_i |p_i|,  Q = 127 (EDGE_INT8) or 448 (EDGE_FP8_E4M3),
 *   code_i = round(p_i * inv) to nearest even,  inv = min(Q / m, 2^126)  (the product
 *       is rounded to fp32 first; inv is an fp32 number for E4M3, and for int8 is held
 *       to 2^-44 of itself, so that a value halfway between two codes takes the even
 *       one),
 *   scales[t] = step, or r_t * step for the norms (r_t as in edge_rmsnorm),
 *   step = max(m / Q, 2^-126),
 * all in fp32 but for that, the divisions IEEE.  The factor r_t of the norm is common to the
 * row, so it enters the scale alone; int8 codes lie in -127 .. 127.
 * A row with a NaN or an infinity among its products has a scale that is NaN or
 * infinite (the norms: NaN), and codes without a meaning.
 *
 * out:    [rows, n] bytes of q_dt (EDGE_INT8 or EDGE_FP8_E4M3).
 * scales: [rows] fp32.
 * The other arguments and the errors as in edge_rmsnorm, edge_add_rmsnorm,
 * edge_glu_act and edge_quantize_fp8; out and scales must not overlap each other
 * or any other buffer.  EDGE_ERR_UNSUPPORTED: n above 2^24.
 */
edge_status edge_rmsnorm_q8(void* out, edge_dtype q_dt, float* scales, const void* x,
                            const void* w, edge_dtype dt, int64_t rows, int64_t n, float eps,
                            int weight_offset, void* stream);
edge_status edge_add_rmsnorm_q8(void* out, edge_dtype q_dt, float* scales, const void* x,
                                void* residual, const void* w, edge_dtype dt, int64_t rows,
                                int64_t n, float eps, int weight_offset, void* stream);
edge_status edge_glu_act_q8(void* out, edge_dtype q_dt, float* scales, const void* gate_up,
                            edge_dtype dt, int64_t rows, int64_t n, edge_act act, void* stream);
edge_status edge_quantize_q8(void* out, edge_dtype q_dt, float* scales, const void* x,
                             edge_dtype dt, int64_t rows, int64_t n, void* stream);

/*
 * Matrix product of 8-bit operands with a scale for each token and each output
 * channel (the reader of the calls above).
 *
 *   out[t, j] = round((sum_i a[t, i] w[j, i]) * a_scales[t] * w_scales[j] + bias[j])
 *
 * a:        [tokens, k] of q_dt (EDGE_INT8 or EDGE_FP8_E4M3).
 * w:        [n, k] of q_dt, a row for each output channel.
 * a_scales: [tokens] fp32.   w_scales: [n] fp32.
 * bias:     [n] of out_dt, or NULL.
 * out:      [tokens, n] of out_dt (EDGE_F32, EDGE_F16 or EDGE_BF16); it must not
 *           overlap any other buffer.
 * int8 sums are exact (every int8 value is allowed, -128 too).  E4M3 sums are
 * held in fp32; a NaN code makes the sums it enters NaN.  The sum, rounded to
 * fp32, is multiplied by a_scales[t], then by w_scales[j], and the bias is added,
 * in fp32; then the output is rounded once.  Results are the same from run to run.
 * Operands with k a multiple of 16 whose addresses are multiples of 16 take the
 * tensor-memory and streaming paths; others a slower one.  Waits inside the kernel
 * are limited to two seconds; should one run out, which correct operation never
 * does, the outputs that it concerns are NaN.
 * EDGE_ERR_SHAPE: tokens < 0, n or k < 1.  EDGE_ERR_UNSUPPORTED: k above 131,071
 * (the largest whose int8 sums fit 32 bits), or tokens or n above 2^24.
 */
edge_status edge_matmul_q8(void* out, edge_dtype out_dt, const void* a, const void* w,
                           edge_dtype q_dt, const float* a_scales, const float* w_scales,
                           const void* bias, int64_t tokens, int64_t n, int64_t k, void* stream);

/*
 * Plain device copy of `bytes` bytes from src to dst, in the launch form of the
 * operators above (a one-shot grid of 16-byte vectors, each CTA's source span
 * prefetched into L2 before the dependent-launch wait).  It computes nothing:
 * it is the yardstick the measurements set each operator against, the time a
 * kernel of that form needs to move the same number of bytes.  No page defines
 * it.  dst and src are device pointers of any alignment (16-byte aligned ones
 * take the vector path); the ranges must not overlap (EDGE_ERR_ALIAS).
 * bytes < 0: EDGE_ERR_SHAPE; bytes == 0 launches nothing.
 */
edge_status edge_copy(void* dst, const void* src, int64_t bytes, void* stream);

/* A static, NUL-terminated description of a status code. */
const char* edge_status_str(edge_status status);

/* The cudaError_t of the calling thread's last EDGE_ERR_CUDA (0 if none). */
int edge_last_cuda_error(void);

/* Library version: major * 10000 + minor * 100 + patch. */
int edge_version(void);

#ifdef __cplusplus
}
#endif

#endif /* EDGE_OPS_H */
