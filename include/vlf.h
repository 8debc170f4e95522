/*
 * vlf.h -- C ABI of libvlf.so: fused variable-length flash attention (forward and backward)
 * for NVIDIA GB300 (sm_103a).
 *
 * The operation is the one the mtlattn 0.3.0 page defines for its varlen_attention call
 * (section "Use"):
 *   q [total_q, H_q, D_qk], k [total_kv, H_kv, D_qk], v [total_kv, H_kv, D_v], packed by
 *   cumulative sequence lengths cu_seqlens_q / cu_seqlens_kv (int32 [num_seqs + 1]), no padding;
 *   query head h reads kv head h / (H_q / H_kv) (GQA / MQA);
 *   logit(i, j) = scale * (q_i . k_j) + bias[global row i, h or 0, sequence-local key j];
 *   causal (end-aligned): row i sees key j iff j <= i + (kv_len - q_len);
 *   window W > 0: row i sees only the last W keys up to that diagonal,
 *                 j >= i + (kv_len - q_len) - W + 1;
 *   out_i = softmax_j(logit(i, .)) v, accumulated in fp32 without materialising the L x L
 *   score matrix (online softmax, mtlattn 0.3.0 header; triton-msl part 1, "What works").
 * The asymmetric latent-attention head (D_qk = 192 = 128 "nope" ++ 64 "rope", D_v = 128) is the
 * one of triton-msl part 2, "Latent attention".
 *
 * Conventions for every entry point
 *   - All tensors are dense, row-major (C-contiguous) device buffers owned by the caller; the
 *     library never allocates, frees or synchronises inside vlf_attn_varlen_fwd/_bwd and only
 *     enqueues work on `stream` (mtlattn 0.3.0, "Notes": work is ordered on the caller's stream
 *     without a per-call host sync).
 *   - Element types: q, k, v, out, dout, dq, dk, dv share `dtype` (VLF_F16, VLF_BF16, VLF_F32);
 *     bias, lse and the workspace are fp32.  Accumulation is fp32 for every dtype; each output is
 *     rounded once (round-to-nearest-even) to its storage type.
 *   - Every pointer must be 16-byte aligned.
 *   - Correct-or-refuse (triton-msl part 1, "Correct-or-refuse"): an argument the library cannot
 *     handle returns a negative vlf_status before anything is enqueued; nothing is silently
 *     approximated.  Errors found on the device (bad cu_seqlens, a pipeline wait that ran out of
 *     time) are recorded in a per-device error word and returned by vlf_check_error().  The
 *     kernels never trap.
 *   - Indices into q/k/v/out/bias are 64-bit: bias tensors beyond 2^32 elements are supported.
 */
#ifndef VLF_H
#define VLF_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t; NULL is the legacy default stream. */
struct CUstream_st;
typedef struct CUstream_st *vlf_stream_t;

typedef enum { VLF_F16 = 0, VLF_BF16 = 1, VLF_F32 = 2 } vlf_dtype;

typedef enum {
  VLF_OK = 0,
  VLF_ERR_INVALID = -1,     /* null pointer, negative size, H_q % H_kv != 0, bias_heads not 1/H_q */
  VLF_ERR_UNSUPPORTED = -2, /* a valid problem this build does not implement (e.g. head width) */
  VLF_ERR_ALIGN = -3,       /* a pointer is not 16-byte aligned (device: a kernel's shared window
                               is not 1024-byte aligned) */
  VLF_ERR_LAUNCH = -4,      /* the CUDA runtime refused a launch or a query */
  VLF_ERR_TIMEOUT = -5,     /* device: a pipeline wait exceeded its time limit (kernel bailed out) */
  VLF_ERR_BAD_SEQLENS = -6, /* device: cu_seqlens not in [0, total], decreasing, or longer than max_seqlen */
  VLF_ERR_WORKSPACE = -7,   /* a workspace missing or smaller than its size query returns */
  VLF_ERR_BAD_PAGES = -8    /* device: a page outside the pool, or tables and counts that disagree */
} vlf_status;

/* Extended-call flags (vlf_attn_varlen_fwd_ex / _bwd_ex). */
#define VLF_FLAG_NO_SKIP 1u    /* visit every KV tile, masking per element (tile-skip check) */
#define VLF_FLAG_FORCE_SIMT 2u /* use the SIMT fp32-FMA kernels even where a tensor-core one exists */
#define VLF_FLAG_NO_PACK 4u    /* forward: never pack a kv head's query heads into one tile (the
                                  decode-size layout); results are identical either way */
#define VLF_FLAG_TEST_TIMEOUT 8u /* testing the failure path: the tensor-core forward's producer
                                    never loads the query tile, so every CTA's pipeline waits run
                                    out after their time limit (2 s); the kernel records
                                    VLF_ERR_TIMEOUT, drains, frees its TMEM and returns, and the
                                    device stays usable (out is not written) */

/*
 * Forward.  mtlattn 0.3.0, section "Use" (varlen_attention with scale, causal, window, attn_bias).
 *
 *   q            [total_q, h_q, d_qk]      dtype
 *   k            [total_kv, h_kv, d_qk]    dtype
 *   v            [total_kv, h_kv, d_v]     dtype
 *   cu_seqlens_q / cu_seqlens_kv           device int32 [num_seqs + 1], cu[0] = 0,
 *                                          non-decreasing, cu[num_seqs] = total_q / total_kv
 *   max_seqlen_q / max_seqlen_kv           host ints >= every sequence's q_len / kv_len
 *                                          (size the launch grid; max_seqlen_kv is also the
 *                                          row length of `bias`)
 *   h_q % h_kv == 0
 *   scale        softmax scale; <= 0 selects 1/sqrt(d_qk)
 *   causal       0/1, end-aligned
 *   window       <= 0: none; else the number of keys each row sees up to its diagonal
 *   bias         NULL or fp32 [total_q, bias_heads, max_seqlen_kv], bias_heads in {1, h_q};
 *                row = global query row, column = sequence-local key; -inf masks the pair
 *   out          [total_q, h_q, d_v]       dtype (written)
 *   lse          NULL or fp32 [h_q, total_q]: natural-log log-sum-exp of each row's logits,
 *                -inf for a row that sees no key (its out row is 0).  Required by the backward.
 * Supported: dtype F16/BF16 with any 1 <= d_qk, d_v <= 256 (tensor-core kernels for
 * (d_qk, d_v) in {(64,64), (96,96), (128,128), (192,128), (256,256)}); dtype F32 with d_qk,
 * d_v <= 256 (tensor-core kernels for (32,32) and (64,64), products in three tf32 passes with
 * fp32 accumulation; fp32 FMA otherwise).
 */
int vlf_attn_varlen_fwd(const void *q, const void *k, const void *v,
                        const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_kv, int num_seqs,
                        int total_q, int total_kv, int max_seqlen_q, int max_seqlen_kv,
                        int h_q, int h_kv, int d_qk, int d_v, int dtype,
                        float scale, int causal, int window,
                        const float *bias, int bias_heads,
                        void *out, float *lse, vlf_stream_t stream);

/*
 * As vlf_attn_varlen_fwd, plus `flags` (VLF_FLAG_*) and `bias_bands`: NULL, or the result of
 * vlf_bias_bands for this bias (below), which lets the kernels skip the KV tiles the bias masks
 * for every row of a query tile.
 */
int vlf_attn_varlen_fwd_ex(const void *q, const void *k, const void *v,
                           const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_kv, int num_seqs,
                           int total_q, int total_kv, int max_seqlen_q, int max_seqlen_kv,
                           int h_q, int h_kv, int d_qk, int d_v, int dtype,
                           float scale, int causal, int window,
                           const float *bias, int bias_heads,
                           void *out, float *lse, vlf_stream_t stream, unsigned flags,
                           const void *bias_bands);

/*
 * Split-KV forward, for problems whose (query tile, head) CTAs are too few to fill the GPU --
 * small batches of decode steps (one query row per sequence against a long cache; the
 * end-aligned causal rule serves cached decode, mtlattn 0.3.0, "Use") or short queries against
 * long keys.
 * Each CTA's KV band is cut into num_splits contiguous parts computed in parallel; each part
 * writes its normalised fp32 result and its log-sum-exp L_s to the workspace, and a combine
 * kernel writes out = sum_s exp(L_s - LSE) out_s and lse = LSE = log sum_s exp(L_s) -- the
 * same softmax, summed in another order (results agree with vlf_attn_varlen_fwd to rounding).
 *
 *   arguments as vlf_attn_varlen_fwd_ex, plus
 *   num_splits   0: the library's choice (vlf_fwd_num_splits); 1: unsplit; 2..64: that many
 *                parts (some may be empty); num_splits * num_seqs <= 65535
 *   workspace    device buffer of at least vlf_attn_varlen_fwd_split_workspace_size(total_q,
 *                h_q, d_v, num_splits) bytes, owned by the caller, clobbered; may be NULL when
 *                the call runs unsplit
 * Shapes that cannot split (dtype F32, (d_qk, d_v) other than (64,64), (96,96), (128,128),
 * (256,256)) run the unsplit forward.  Returns VLF_ERR_WORKSPACE when a split call's workspace is missing or
 * too small.
 */
int vlf_attn_varlen_fwd_split(const void *q, const void *k, const void *v,
                              const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_kv,
                              int num_seqs, int total_q, int total_kv, int max_seqlen_q,
                              int max_seqlen_kv, int h_q, int h_kv, int d_qk, int d_v, int dtype,
                              float scale, int causal, int window,
                              const float *bias, int bias_heads,
                              void *out, float *lse, int num_splits,
                              void *workspace, size_t workspace_bytes, vlf_stream_t stream,
                              unsigned flags, const void *bias_bands);

/*
 * The number of parts vlf_attn_varlen_fwd_split uses for num_splits = 0 (1: no split).  Pure
 * host arithmetic on the launch shape, with the CTAs resident per SM (two; one at width 256)
 * as the "slots" of a wave:
 * a grid below one wave is split into as many parts as keep it within one wave, each part at
 * least 256 keys (at most 64 parts); a grid of one to three waves whose last wave is under 95%
 * full gets 2 or 3 parts, whichever fills its waves better (the fewer on a tie), each at least
 * 1024 keys; larger grids are not split.  num_sms <= 0 takes the current device's SM count
 * (returns 1 if it cannot be queried).
 */
int vlf_fwd_num_splits(int num_seqs, int max_seqlen_q, int max_seqlen_kv, int h_q, int h_kv,
                       int d_qk, int d_v, int dtype, unsigned flags, int num_sms);

/*
 * Bytes of workspace vlf_attn_varlen_fwd_split needs: fp32 parts [num_splits, total_q, h_q, d_v]
 * and their log-sum-exps [num_splits, h_q, total_q], each rounded up to 256 bytes; 0 when
 * num_splits < 2.  Pure host arithmetic.
 */
size_t vlf_attn_varlen_fwd_split_workspace_size(int total_q, int h_q, int d_v, int num_splits);

/*
 * Bytes of fp32 workspace vlf_attn_varlen_bwd needs: the row dot products D = rowsum(dO o O),
 * [h_q, total_q] fp32 (rounded up to 256 bytes).  Pure host arithmetic; never fails (returns 0
 * for invalid sizes).
 */
size_t vlf_attn_varlen_bwd_workspace_size(int total_q, int total_kv, int h_q, int h_kv,
                                          int d_qk, int d_v, int dtype);

/*
 * Backward.  The gradients of sum(out * dout) with respect to q, k, v, the bias held constant
 * (mtlattn 0.3.0, "Use": the bias is treated as constant; triton-msl part 2, "Beyond softmax":
 * a tiled FlashAttention-2 backward).  Same shapes and conventions as the forward, plus
 *   out, lse     the forward's outputs for the same inputs
 *   dout         [total_q, h_q, d_v]       dtype
 *   dq           [total_q, h_q, d_qk]      dtype (written)
 *   dk, dv       [total_kv, h_kv, d_qk], [total_kv, h_kv, d_v] dtype (written; each kv head
 *                sums the contributions of its h_q / h_kv query heads)
 *   workspace    device buffer of at least vlf_attn_varlen_bwd_workspace_size(...) bytes,
 *                owned by the caller, contents need not be initialised; clobbered.
 */
int vlf_attn_varlen_bwd(const void *q, const void *k, const void *v, const void *out,
                        const float *lse, const void *dout,
                        const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_kv, int num_seqs,
                        int total_q, int total_kv, int max_seqlen_q, int max_seqlen_kv,
                        int h_q, int h_kv, int d_qk, int d_v, int dtype,
                        float scale, int causal, int window,
                        const float *bias, int bias_heads,
                        void *dq, void *dk, void *dv,
                        void *workspace, size_t workspace_bytes, vlf_stream_t stream);

/*
 * As vlf_attn_varlen_bwd, plus `flags`, optional per-stage timing events and the bias bands
 * (NULL, or vlf_bias_bands's result for this bias, as in vlf_attn_varlen_fwd_ex).  When
 * stage_events is not NULL it holds n_stage_events >= VLF_BWD_STAGES + 1 cudaEvent_t handles
 * (created by the caller); event 0 is recorded on `stream` before the first kernel and event
 * s+1 after stage s, stages being, in order: 0 the dO.O row-dot pre-pass, 1 the dK/dV kernel,
 * 2 the dQ kernel.  Recording adds no synchronisation.
 */
#define VLF_BWD_STAGES 3
int vlf_attn_varlen_bwd_ex(const void *q, const void *k, const void *v, const void *out,
                           const float *lse, const void *dout,
                           const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_kv, int num_seqs,
                           int total_q, int total_kv, int max_seqlen_q, int max_seqlen_kv,
                           int h_q, int h_kv, int d_qk, int d_v, int dtype,
                           float scale, int causal, int window,
                           const float *bias, int bias_heads,
                           void *dq, void *dk, void *dv,
                           void *workspace, size_t workspace_bytes, vlf_stream_t stream,
                           unsigned flags, void *const *stage_events, int n_stage_events,
                           const void *bias_bands);

/*
 * Bias bands.  An additive bias often masks whole stretches of each row (mtlattn 0.3.0, "Use":
 * -inf masks a pair and a boolean mask becomes a 0 / -inf bias; a prefix-LM mask hides every key
 * past the prefix and the diagonal).  This pass records, for each bias head and query row, the
 * keys from the first to the last finite value among the row's first kv_len columns, and whether
 * the bias is exactly 0 throughout them; and the same, combined, for each block of 64 rows of
 * each sequence.  Given to the _ex calls, it lets the tensor-core kernels (16-bit data, widths
 * up to 128, one query tile per CTA) skip the KV tiles and query items that hold only -inf bias
 * values for their rows -- the skipped pairs contribute exact zeros -- and mask by interval
 * without reading the bias where every row of a tile is such a 0 / -inf interval.  The results
 * equal those computed without the bands within the stated tolerances (the bias values of a pure
 * interval are 0; the masked pairs are the same).  The bands must come from this bias (same
 * tensor, unmodified since): stale bands give wrong results.
 *   bias, bias_heads, cu_seqlens_q / _kv, num_seqs, total_q, max_seqlen_kv   as in the forward
 *   bands        device buffer of at least vlf_bias_bands_size(total_q, bias_heads) bytes,
 *                16-byte aligned, owned by the caller, written: two int32x4 tables of
 *                [bias_heads][total_q] entries -- per row {lo, hi, pure, 0} (keys [lo, hi) from
 *                the first to the last finite value, lo = hi = 0 if none; pure 1 when the bias
 *                is 0 throughout them), then per 64-row block of each sequence, at the block's
 *                first row, {lo, hi, ilo, ihi}: the union of its rows' intervals and, when all
 *                its rows are pure, their intersection (-1, -1 otherwise)
 * Enqueued on `stream`; no synchronisation.  Returns VLF_OK or a negative status (invalid
 * arguments, VLF_ERR_WORKSPACE for a missing or short buffer).
 */
size_t vlf_bias_bands_size(int total_q, int bias_heads);
int vlf_bias_bands(const float *bias, int bias_heads, const int32_t *cu_seqlens_q,
                   const int32_t *cu_seqlens_kv, int num_seqs, int total_q, int max_seqlen_kv,
                   void *bands, size_t bands_bytes, vlf_stream_t stream);

/*
 * Latent attention with split operands (triton-msl part 2, "Latent attention": the score is the
 * sum of two query-key products over different widths, a 128-wide "nope" part and a 64-wide
 * "rope" part, so the contraction is 192 wide while the output stays 128 wide).  The parts are
 * passed as they are produced, without concatenation, and the rope key may be one tensor shared
 * by every head:
 *   logit(i, j) = scale * (q_nope_i . k_nope_j + q_rope_i . k_rope_j) + bias,
 * with head h reading k_nope / v of kv head h / (h_q / h_kv) and k_rope of that kv head, or of
 * the single rope head when rope_heads = 1.  Results equal vlf_attn_varlen_fwd / _bwd on the
 * concatenated operands q = [q_nope | q_rope], k = [k_nope | k_rope broadcast over kv heads]
 * (the same kernels, the same arithmetic).
 *
 *   q_nope  [total_q, h_q, 128]   q_rope [total_q, h_q, 64]          dtype
 *   k_nope  [total_kv, h_kv, 128] k_rope [total_kv, rope_heads, 64]  dtype, rope_heads in {1, h_kv}
 *   v       [total_kv, h_kv, 128]                                     dtype
 *   d_nope, d_rope, d_v must be 128, 64, 128 (VLF_ERR_UNSUPPORTED otherwise, and for dtype F32
 *   or VLF_FLAG_FORCE_SIMT: there is no SIMT kernel for split operands); other arguments and
 *   outputs as vlf_attn_varlen_fwd / _bwd.  scale <= 0 selects 1/sqrt(192).
 * Backward outputs (written): dq_nope / dq_rope like q_nope / q_rope, dk_nope like k_nope, dv
 * like v, dk_rope like k_rope -- for a shared rope key (rope_heads = 1) the sum over every head
 * of its gradient, accumulated in fp32 in kv-head order (deterministic) and rounded once.  The
 * workspace (caller-owned, clobbered) holds the row dot products and, for a shared rope key with
 * h_kv > 1, the per-kv-head fp32 rope gradients [h_kv, total_kv, 64].
 */
int vlf_attn_varlen_fwd_latent(const void *q_nope, const void *q_rope, const void *k_nope,
                               const void *k_rope, const void *v,
                               const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_kv,
                               int num_seqs, int total_q, int total_kv, int max_seqlen_q,
                               int max_seqlen_kv, int h_q, int h_kv, int rope_heads,
                               int d_nope, int d_rope, int d_v, int dtype,
                               float scale, int causal, int window,
                               const float *bias, int bias_heads,
                               void *out, float *lse, vlf_stream_t stream, unsigned flags);

/* Bytes of workspace vlf_attn_varlen_bwd_latent needs (pure host arithmetic; 0 for invalid
 * sizes). */
size_t vlf_attn_varlen_bwd_latent_workspace_size(int total_q, int total_kv, int h_q, int h_kv,
                                                 int rope_heads, int dtype);

int vlf_attn_varlen_bwd_latent(const void *q_nope, const void *q_rope, const void *k_nope,
                               const void *k_rope, const void *v, const void *out,
                               const float *lse, const void *dout,
                               const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_kv,
                               int num_seqs, int total_q, int total_kv, int max_seqlen_q,
                               int max_seqlen_kv, int h_q, int h_kv, int rope_heads,
                               int d_nope, int d_rope, int d_v, int dtype,
                               float scale, int causal, int window,
                               const float *bias, int bias_heads,
                               void *dq_nope, void *dq_rope, void *dk_nope, void *dk_rope,
                               void *dv, void *workspace, size_t workspace_bytes,
                               vlf_stream_t stream, unsigned flags,
                               void *const *stage_events, int n_stage_events);

/*
 * Number of kernels this library has launched in this process (all devices, all streams),
 * counted on the host at each successful launch.  For benchmarks that report their launches.
 */
uint64_t vlf_launch_count(void);

/*
 * Which kernel family the forward / backward would use for this problem: 1 tensor-core
 * (tcgen05), 0 SIMT fp32 FMA, negative status if the problem is refused.  Host only.
 */
int vlf_fwd_path(int h_q, int h_kv, int d_qk, int d_v, int dtype, int bias_heads, unsigned flags);
int vlf_bwd_path(int h_q, int h_kv, int d_qk, int d_v, int dtype, int bias_heads, unsigned flags);

/*
 * Synchronises `stream`, then returns and clears the current device's error word (VLF_OK,
 * VLF_ERR_TIMEOUT or VLF_ERR_BAD_SEQLENS), or VLF_ERR_LAUNCH if the CUDA runtime reports an
 * error.  The only entry point that blocks the host.
 */
int vlf_check_error(vlf_stream_t stream);

/* Static description of a status code. */
const char *vlf_status_string(int status);

/*
 * Tile scheduler (host-callable, no GPU needed).  For sequence-local query rows [r0, r1) of a
 * sequence with q_len queries and kv_len keys, the key range [*lo, *hi) that holds every key
 * any of those rows may see under the causal/window rules above; keys outside it are skipped
 * whole (mtlattn 0.3.0, "Use": fully masked KV tiles are skipped, window jumps to its band).
 * Returns VLF_OK or VLF_ERR_INVALID.
 */
int vlf_sched_kv_band(int r0, int r1, int q_len, int kv_len, int causal, int window,
                      int *lo, int *hi);

/* The query rows [*lo, *hi) that may see any key of [j0, j1) (the backward's dK/dV band). */
int vlf_sched_q_band(int j0, int j1, int q_len, int kv_len, int causal, int window,
                     int *lo, int *hi);

/*
 * Backward that allocates nothing.  The pages have no counterpart to this entry point; it exists
 * for callers that cannot allocate device memory at call time -- a plugin whose enqueue hook may
 * not allocate, a service that reserves its memory budget up front, or code that must not
 * trigger the device-wide synchronisation cudaMalloc / cudaFree can cause.  Same arguments and
 * results as vlf_attn_varlen_bwd without the workspace: the row dot products live in a
 * fixed-size array inside the library's own device memory instead.
 *   - Size limit: h_q * total_q <= 8,388,608 (vlf_noalloc_scratch_bytes() bytes of fp32);
 *     larger problems return VLF_ERR_UNSUPPORTED before anything is enqueued.
 *   - Every GPU that loads the library holds that array (32 MiB) until the process exits.
 *   - Calls on one device share the array and it keeps the last call's contents (nothing in it
 *     needs to start at zero).  Calls whose work overlaps on the GPU race on it: order them on
 *     one stream, or with events.
 *   - The first call on each device looks up the array's device address; make that first call
 *     before any stream capture begins.  The address is kept for the life of the process and is
 *     not valid after a cudaDeviceReset of that device: do not call this entry point on a
 *     device after resetting it.
 *   - No cudaMalloc, cudaFree or other allocating routine is called.
 */
int vlf_attn_varlen_bwd_noalloc(const void *q, const void *k, const void *v, const void *out,
                                const float *lse, const void *dout,
                                const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_kv,
                                int num_seqs, int total_q, int total_kv, int max_seqlen_q,
                                int max_seqlen_kv, int h_q, int h_kv, int d_qk, int d_v, int dtype,
                                float scale, int causal, int window,
                                const float *bias, int bias_heads,
                                void *dq, void *dk, void *dv, vlf_stream_t stream);

/* Bytes of the fixed array vlf_attn_varlen_bwd_noalloc uses as its workspace. */
size_t vlf_noalloc_scratch_bytes(void);

/*
 * Decoding on a bounded cache: rotary positions, attention behind a shared prefix, the weight each
 * cached key received, and the cache cut down by it.  The pages have no counterpart to these entry
 * points (they stop at "cached decode" with the end-aligned causal rule, mtlattn 0.3.0, "Use", and
 * at a head with a "rope" part, triton-msl part 2, "Latent attention"); they are what a program
 * that serves with the calls above runs next to them.
 *
 * total_q and total_kv are below 2^31 - 2^16 in them (VLF_ERR_UNSUPPORTED).  max_seqlen_q and max_seqlen_kv
 * may be any upper bounds, but how the work is cut goes by them: pass them tight where time counts
 * (a bound of the longest cache for a batch of short ones costs shared-prefix attention its split).
 */

/*
 * Rotary positions with several axes, of packed queries and keys together.
 *   q [total, h_q, d], k [total, h_k, d]   dtype; the heads and columns of a token are dense, tokens
 *                are q_stride / k_stride elements apart (slices of a fused projection's output are
 *                taken as they are); k may be NULL with h_k = 0
 *   q_out, k_out as q, k, with strides of their own (at least h * d).  An output may be its input
 *                (same pointer and stride); otherwise outputs overlap no input.
 *   positions    device int32 [n_axes, total], any values
 *   n_axes       1..4; sections: host int [n_axes], how many consecutive pairs each axis turns
 *                (>= 0, their sum is rot / 2); NULL with n_axes = 1
 *   inv_freq     device fp32 [rot / 2], finite: the radians pair c turns per unit of its position
 *   rot          even, 0..d: the columns that turn; the others pass through
 *   interleaved  0: pair c is columns (c, c + rot / 2); 1: columns (2 c, 2 c + 1)
 *   inverse      0: y_a = x_a cos t - x_b sin t, y_b = x_b cos t + x_a sin t with
 *                t = positions[axis(c)][token] * inv_freq[c]; 1: by -t, which is the gradient of
 *                the rotation (and undoes it)
 * The angle is taken in 64-bit fixed point, off by at most |position| (|inv_freq| 2^-55 + 2^-64) turns
 * whatever the position; sines, cosines and products are fp32, the result is rounded once.
 */
int vlf_rope(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
             const int32_t *positions, int n_axes, const int *sections, const float *inv_freq,
             int total, int h_q, int h_k, int d, int rot, int dtype, int interleaved, int inverse,
             void *q_out, int64_t q_out_stride, void *k_out, int64_t k_out_stride,
             vlf_stream_t stream);

/*
 * Attention of a batch whose sequences all start with the same keys (a shared system prompt or
 * document): sequence s attends over the prefix_len prefix keys followed by its own kv_len keys, and
 * out / lse are those of vlf_attn_varlen_fwd on the concatenated keys (the causal and window rules
 * count all prefix_len + kv_len keys; row i stands at key i + prefix_len + kv_len - q_len).  The
 * prefix is held and read once for the batch: where it pays, rows of all sequences share its tiles.
 *   k_prefix [prefix_len, h_kv, d_qk], v_prefix [prefix_len, h_kv, d_v]   dtype; prefix_len >= 0,
 *                with the longest own length, min(max_seqlen_kv, total_kv), below 2^31 - 2^16
 *   workspace    device buffer of at least vlf_attn_varlen_fwd_prefix_workspace_size(...) bytes,
 *                owned by the caller, clobbered (two calls that may overlap need two); may be NULL
 *                where that is 0
 *   flags        VLF_FLAG_FORCE_SIMT; others are ignored
 * Other arguments as vlf_attn_varlen_fwd (no bias); dtypes and widths as there, with tensor-core
 * kernels for F16 / BF16 and (d_qk, d_v) in {(64,64), (96,96), (128,128)}.  Keys and values of other
 * sequences never reach a row, whatever they hold; a value of its own sequence or of the prefix that
 * is not finite may also reach rows that do not see its key (a weight of 0 times it), as in
 * vlf_attn_varlen_fwd.  A row that sees a NaN logit is NaN, and so is its lse.  No backward.
 */
int vlf_attn_varlen_fwd_prefix(const void *q, const void *k_prefix, const void *v_prefix,
                               int prefix_len, const void *k, const void *v,
                               const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_kv,
                               int num_seqs, int total_q, int total_kv, int max_seqlen_q,
                               int max_seqlen_kv, int h_q, int h_kv, int d_qk, int d_v, int dtype,
                               float scale, int causal, int window, void *out, float *lse,
                               void *workspace, size_t workspace_bytes, vlf_stream_t stream,
                               unsigned flags);

/* Bytes of workspace vlf_attn_varlen_fwd_prefix needs: a rule on these sizes and the SM count
 * (num_sms <= 0: the current device's); 0 for invalid sizes. */
size_t vlf_attn_varlen_fwd_prefix_workspace_size(int num_seqs, int total_q, int max_seqlen_q,
                                                 int max_seqlen_kv, int prefix_len, int h_q,
                                                 int h_kv, int d_qk, int d_v, int dtype,
                                                 unsigned flags, int num_sms);

/*
 * The attention weight that each key received:
 *   weights[g, j] = prev[g, j] + sum of exp(scale * q_i,h . k_j,g - lse[h, i]) over the query rows
 *                   i of j's sequence that see j (causal and window rules as in the forward) and
 *                   the heads h of kv head g,
 * the column sums of the attention matrix whose row log-sum-exps the forward returned.  With the
 * lse of vlf_attn_varlen_fwd_prefix it gives the own keys' weights, and, called with the prefix as
 * the one sequence's keys (cu_seqlens {0, total_q} and {0, prefix_len}, no causal rule or window),
 * the prefix keys' over the batch.
 *   q, k, sequences, scale, causal, window   as the forward that returned lse
 *   lse          fp32 [h_q, total_q]; a row with -inf gives nothing
 *   prev         NULL (zeros) or fp32 [h_kv, total_kv]; may be weights
 *   weights      fp32 [h_kv, total_kv] (written)
 *   workspace    at least vlf_attn_key_weights_workspace_size(...) bytes, as above
 *   flags        VLF_FLAG_FORCE_SIMT; others are ignored
 * Sums are fp32, each in a fixed order.  Tensor-core kernels for F16 / BF16 and d in {64, 96, 128,
 * 192}; any d <= 256 otherwise.
 */
int vlf_attn_key_weights(const void *q, const void *k, const float *lse,
                         const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_kv, int num_seqs,
                         int total_q, int total_kv, int max_seqlen_q, int max_seqlen_kv, int h_q,
                         int h_kv, int d, int dtype, float scale, int causal, int window,
                         const float *prev, float *weights, void *workspace,
                         size_t workspace_bytes, vlf_stream_t stream, unsigned flags);

/* Bytes of workspace vlf_attn_key_weights needs, a rule as above. */
size_t vlf_attn_key_weights_workspace_size(int num_seqs, int total_kv, int max_seqlen_q,
                                           int max_seqlen_kv, int h_q, int h_kv, int d, int dtype,
                                           unsigned flags, int num_sms);

/*
 * Cache eviction.  Of each sequence's L keys n = min(L, budget) stay: all of them, or the first
 * `sink`, the last `recent`, and of the keys between them the budget - sink - recent with the
 * largest weight (of equal weights the lower index; -0 equals +0, a NaN is below every number).
 * Each kv head chooses for itself; kept keys keep their order.
 *   k [total_kv, h_kv, d_qk], v [total_kv, h_kv, d_v]   dtype
 *   weights      fp32 [h_kv, total_kv]
 *   budget >= 0, sink >= 0, recent >= 0, sink + recent <= budget
 *   total_out    rows of the outputs, at least the sum of the n (else VLF_ERR_BAD_SEQLENS on the
 *                device, and the sequences that do not fit are not written); rows behind the last
 *                kept one are left as they were
 *   k_out [total_out, h_kv, d_qk], v_out [total_out, h_kv, d_v], weights_out fp32 [h_kv, total_out]
 *   index_out    int32 [h_kv, total_out]: the sequence-local key each row came from
 *   cu_out       int32 [num_seqs + 1]: the cu_seqlens of the outputs (-1 behind a sequence that had
 *                an error; neither it nor the next one is copied).  With num_seqs = 0 nothing is
 *                enqueued, and the one entry is the caller's to set to 0
 * Outputs overlap neither an input nor one another (VLF_ERR_INVALID).  d_qk, d_v <= 256.
 */
int vlf_cache_evict(const void *k, const void *v, const float *weights,
                    const int32_t *cu_seqlens_kv, int num_seqs, int total_kv, int max_seqlen_kv,
                    int h_kv, int d_qk, int d_v, int dtype, int budget, int sink, int recent,
                    int total_out, void *k_out, void *v_out, float *weights_out,
                    int32_t *index_out, int32_t *cu_out, vlf_stream_t stream);

/*
 * Serving from a cache of pages in 8 bits: the norm of queries and keys with their positions, the pages
 * that hold keys and values, attention over them, and the tables that say which sequence has which
 * pages.  The pages have no counterpart to these entry points either.
 *
 * The cache of a layer:
 *   k_pages      e4m3 (one byte: sign, 4 exponent and 3 mantissa bits, no infinities, 0x7f and 0xff are
 *                NaN) [num_pages, h_kv, page, d_qk]; v_pages the same with d_v
 *   k_scale, v_scale   fp32 [num_pages, h_kv]: a value is its byte's times its page's and head's scale.
 *                Scales are powers of two from 2^-64 on (those that vlf_pages_write leaves)
 *   page         16, 32, 64, 128 or 256 tokens (VLF_ERR_UNSUPPORTED otherwise)
 *   page_table   int32 [num_seqs, max_pages]: key j of sequence s is slot j % page of page
 *                page_table[s][j / page]; entries behind a sequence's last page are not looked at
 *   seqlens_kv   int32 [num_seqs], at most max_pages * page
 * max_pages * page and the numbers of tokens are below 2^31 - 2^16; d_qk, d_v <= 256.  A page that is needed
 * and lies outside 0..num_pages - 1 records VLF_ERR_BAD_PAGES and is passed over (nothing is written for it, and
 * rows do not see its keys), a sequence whose lengths are out of range VLF_ERR_BAD_SEQLENS.
 */

/*
 * Root-mean-square norm of each head of q and k, and the rotary positions of vlf_rope, in one pass:
 *   y = R(t) (w o x / sqrt(mean(x^2) + eps)),
 * the mean over the head's d columns.
 *   q_weight, k_weight   [d] of type weight_dtype (`dtype` or VLF_F32), for every head; NULL: ones
 *   eps          >= 0, finite
 *   others       as in vlf_rope (rot = 0, positions and inv_freq NULL: the norm alone)
 * The arithmetic is fp32 (a row's sum of squares too: elements are below 2^59 in size), the result is rounded once.
 */
int vlf_norm_rope(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                  const void *q_weight, const void *k_weight, int weight_dtype, float eps,
                  const int32_t *positions, int n_axes, const int *sections, const float *inv_freq,
                  int total, int h_q, int h_k, int d, int rot, int dtype, int interleaved,
                  void *q_out, int64_t q_out_stride, void *k_out, int64_t k_out_stride,
                  vlf_stream_t stream);

/*
 * Its gradients: of sum(q_out o dq_out) + sum(k_out o dk_out) with respect to q, k and the weights.
 *   dq_out, dk_out   gradients of the outputs, dtype, with strides of their own
 *   dq, dk       as q, k (written); may be dq_out / dk_out or q / k (same pointer and stride)
 *   dq_weight, dk_weight   [d] of type weight_dtype (written), or NULL: not wanted.  The sums over tokens
 *                and heads are fp32, in a fixed order, rounded once (0 where there are none)
 *   workspace    at least vlf_norm_rope_bwd_workspace_size(d) bytes where a weight's gradient is
 *                wanted; owned by the caller, clobbered (two calls that may overlap need two)
 */
int vlf_norm_rope_bwd(const void *dq_out, int64_t dq_out_stride, const void *dk_out,
                      int64_t dk_out_stride, const void *q, int64_t q_stride, const void *k,
                      int64_t k_stride, const void *q_weight, const void *k_weight, int weight_dtype,
                      float eps, const int32_t *positions, int n_axes, const int *sections,
                      const float *inv_freq, int total, int h_q, int h_k, int d, int rot, int dtype,
                      int interleaved, void *dq, int64_t dq_stride, void *dk, int64_t dk_stride,
                      void *dq_weight, void *dk_weight, void *workspace, size_t workspace_bytes,
                      vlf_stream_t stream);
size_t vlf_norm_rope_bwd_workspace_size(int d);

/*
 * New tokens into their pages.  Token i of sequence s becomes key seqlens_kv[s] - n + i of it, n =
 * cu_seqlens[s + 1] - cu_seqlens[s]: seqlens_kv counts the new tokens, and the same two tensors describe
 * the queries of these tokens to vlf_attn_varlen_fwd_pages.
 *   k [total, h_kv, d_qk], v [total, h_kv, d_v]   dtype; heads and columns of a token are dense, tokens
 *                k_stride / v_stride elements apart
 * A page's scale (each head's for itself) is the smallest power of two, 2^-64 at least, times which 448
 * holds the largest new value of the page, or the scale that the page has where that is larger: then the
 * bytes of the page that are not written anew are multiplied by old / new and rounded again, which costs
 * them nothing but what falls below e4m3's least step.  A call that writes slot 0 of a page begins
 * it: the scale that it had does not count, and its other bytes stay as they are.  Values are rounded to
 * nearest, ties to even.  A value that is not finite is held as a NaN and does not count for the scale.
 * Each page that is written belongs to one sequence (vlf_pages_fork sees to it); where two tokens of a
 * call reach the same slot, either may be left.
 */
int vlf_pages_write(const void *k, int64_t k_stride, const void *v, int64_t v_stride, void *k_pages,
                    void *v_pages, float *k_scale, float *v_scale, const int32_t *page_table,
                    const int32_t *cu_seqlens, const int32_t *seqlens_kv, int num_seqs, int total,
                    int max_pages, int num_pages, int page, int h_kv, int d_qk, int d_v, int dtype,
                    vlf_stream_t stream);

/*
 * Attention over the pages: out and lse are those of vlf_attn_varlen_fwd on the keys and values that the
 * bytes stand for, without a bias.
 *   q, cu_seqlens_q, total_q, max_seqlen_q, heads, dtype, scale, causal, window, out, lse   as there
 *   workspace    at least vlf_attn_varlen_fwd_pages_workspace_size(...) bytes, owned by the caller,
 *                clobbered (two calls that may overlap need two); may be NULL where that is 0
 *   flags        VLF_FLAG_FORCE_SIMT; others are ignored
 * Pages of which no row of a sequence sees a key (in front of the window) are not looked at and may be
 * outside the pool.  What other bytes of a page hold never reaches a row, but a value of its own sequence
 * that is NaN may also reach rows that do not see its key.  A row that sees a NaN logit is NaN, and so is
 * its lse; a query that holds an infinity or a NaN has NaN logits alone (vlf_attn_varlen_fwd takes infinite
 * ones as they are, and a row of minus infinities for one that sees no key).  Tensor-core kernels for
 * F16 / BF16 and d_qk = d_v in {64, 128}; fp32 FMA otherwise.  On the tensor cores a weight times its page's
 * value scale is held to 11 bits, and to 2^-24 of the largest such product of the keys that the row sees; a
 * value scale more than 2^100 below that key's may cost the key its part of the lse.  Scales of pages that a
 * row does not see do not matter to it.  Logits are below 2^26 in size there (fp32 holds them to whole units
 * from 2^24 on, and from 2^27 on weights pass what fp16 holds: the row may be NaN).
 * max_seqlen_q decides which kernel runs: more than 32 rows of a kv head's group (max_seqlen_q * h_q / h_kv)
 * take the one for many rows, so a loose bound makes single rows slower (2.4 times, in large batches), never
 * wrong.  No backward.
 */
int vlf_attn_varlen_fwd_pages(const void *q, const void *k_pages, const void *v_pages,
                              const float *k_scale, const float *v_scale, const int32_t *page_table,
                              const int32_t *cu_seqlens_q, const int32_t *seqlens_kv, int num_seqs,
                              int total_q, int max_seqlen_q, int max_pages, int num_pages, int page,
                              int h_q, int h_kv, int d_qk, int d_v, int dtype, float scale, int causal,
                              int window, void *out, float *lse, void *workspace,
                              size_t workspace_bytes, vlf_stream_t stream, unsigned flags);

/* Bytes of workspace vlf_attn_varlen_fwd_pages needs: a rule on these sizes and the SM count
 * (num_sms <= 0: the current device's); 0 for invalid sizes. */
size_t vlf_attn_varlen_fwd_pages_workspace_size(int num_seqs, int total_q, int max_seqlen_q, int h_q,
                                                int h_kv, int d_qk, int d_v, int dtype, unsigned flags,
                                                int num_sms);

/*
 * Pages copied: page src[i] (keys, values and scales of every head) over page dst[i], for each i with
 * src[i] >= 0.  A page is in dst at most once and not in src as well (what it then holds is not
 * defined).  src and dst are int32 [n], on the device: the lists of the two calls below.
 */
int vlf_pages_copy(void *k_pages, void *v_pages, float *k_scale, float *v_scale, const int32_t *src,
                   const int32_t *dst, int n, int num_pages, int page, int h_kv, int d_qk, int d_v,
                   vlf_stream_t stream);

/*
 * The page tables of the next step.  New row s follows the old row parents[s] (the same row: it goes on;
 * several with one parent: it forks; a row that is no one's parent: its pages are released), or none
 * (parents[s] < 0: it begins empty), and gets room for grow[s] more tokens.
 *   page_table [num_in, max_pages], seqlens [num_in]   the old rows
 *   refs         int32 [num_pages]: how many hold each page: old rows, and others (a prompt kept for
 *                later); 0: the page is free
 *   parents, grow   int32 [num_out], grow >= 0
 *   table_out    [num_out, max_pages] (-1 behind a row's last page); seqlens_out [num_out], the parent's
 *                plus grow; refs_out [num_pages], in which new rows stand for the old ones
 *   src, dst     int32 [num_out]: the copies to make before anything is written, for vlf_pages_copy of
 *                each layer (-1: none)
 *   left         int32 [1]: free pages left
 * Whole pages are shared.  A page that is not full has one holder: the first new row that goes on in it
 * keeps it, if no one else holds it, and every other gets a copy.  New pages are the free ones in
 * ascending order, for the rows in order, a row's copy first.
 * Where more pages are needed than are free, left is negative (their number) and nothing else happens:
 * table_out is -1 throughout, seqlens_out 0, refs_out is refs, src and dst are -1.  So it is, with left =
 * INT32_MIN, after an error: VLF_ERR_BAD_SEQLENS (a length or grow negative or beyond max_pages * page),
 * VLF_ERR_BAD_PAGES (a parent or page out of range, refs below the old rows' holds).
 *   workspace    at least vlf_pages_fork_workspace_size(num_pages, num_out) bytes, owned by the caller,
 *                clobbered (two calls that may overlap need two)
 * Outputs overlap no input and not one another (VLF_ERR_INVALID).
 */
int vlf_pages_fork(const int32_t *page_table, const int32_t *seqlens, const int32_t *refs,
                   const int32_t *parents, const int32_t *grow, int num_in, int num_out, int max_pages,
                   int num_pages, int page, int32_t *table_out, int32_t *seqlens_out, int32_t *refs_out,
                   int32_t *src, int32_t *dst, int32_t *left, void *workspace, size_t workspace_bytes,
                   vlf_stream_t stream);
size_t vlf_pages_fork_workspace_size(int num_pages, int num_out);

/*
 * The U pages in use (refs > 0) moved into the first U of the pool: those behind move into the free ones
 * among the first U, in order.
 *   page_table [num_seqs, max_pages], refs [num_pages]   as above
 *   table_out    the tables afterwards: entries that name a page in use follow it, others become -1
 *   refs_out [num_pages]; to int32 [num_pages]: where each page in use is afterwards (-1: it was free)
 *   src, dst     int32 [num_pages / 2]: the copies to make, for vlf_pages_copy of each layer; -1 behind them
 *   used         int32 [1]: U
 *   workspace    at least vlf_pages_compact_workspace_size(num_pages) bytes, as above
 * Outputs overlap no input and not one another (VLF_ERR_INVALID).
 */
int vlf_pages_compact(const int32_t *page_table, const int32_t *refs, int num_seqs, int max_pages,
                      int num_pages, int32_t *table_out, int32_t *refs_out, int32_t *to, int32_t *src,
                      int32_t *dst, int32_t *used, void *workspace, size_t workspace_bytes,
                      vlf_stream_t stream);
size_t vlf_pages_compact_workspace_size(int num_pages);

/* Library version, major * 10000 + minor * 100 + patch. */
int vlf_version(void);

#ifdef __cplusplus
}
#endif

#endif /* VLF_H */
