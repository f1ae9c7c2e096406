/*
 * libmla.h -- C ABI of libmla: Multi-head Latent Attention (MLA) decode over
 * a paged latent KV cache, for NVIDIA GB300 (sm_103a).
 *
 * The two operations follow the interface on the FlashMLA-PyTorch page
 * (flash_mla_interface.py: get_mla_metadata and flash_mla_with_kvcache) and
 * the vLLM page "vllm.attention.ops.flashmla" (same functions, parameter
 * and return tables):
 *
 *   mla_get_metadata  -- split-KV load-balancing schedule over the SMs
 *                        (get_mla_metadata: tile_scheduler_metadata of shape
 *                        (num_sm_parts, TileSchedulerMetaDataSize) and
 *                        num_splits of shape (batch_size + 1), both int32)
 *   mla_decode_fwd    -- the decode (flash_mla_with_kvcache / fwd_kvcache_mla):
 *                        out (batch, s_q, h_q, head_dim_v) and the fp32
 *                        softmax_lse (batch, h_q, s_q)
 *
 * Conventions shared by every call
 *   - Every tensor argument is a plain pointer owned by the caller (device
 *     memory, except the host buffers of mla_decode_fwd_host); libmla keeps
 *     no reference to it after the call returns.  libmla allocates device
 *     memory only for calls that pass no workspace and for
 *     mla_decode_fwd_host (stream-ordered, released by mla_shutdown).
 *   - All work is enqueued on `stream` (a cudaStream_t; NULL is the legacy
 *     default stream) and runs asynchronously; no call synchronizes the host
 *     except mla_check_device_error.
 *   - Every call returns an int status (MLA_OK or one of MLA_ERR_*); the
 *     detail of the last failure on the calling thread is available from
 *     mla_last_error().  A failing call enqueues nothing.
 *   - Layouts use element strides; the last dimension of every tensor must
 *     be contiguous.  bf16 tensors are IEEE bfloat16 bit patterns.
 *
 * The workspace convention (query the size, then pass caller-owned scratch)
 * mirrors the two-phase C API on the Ascend ATB "MLA" page
 * (AtbMLAGetWorkspaceSize, then AtbMLA).
 */
#ifndef LIBMLA_H
#define LIBMLA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *mla_stream_t; /* same handle as cudaStream_t */

/* Status codes. */
enum {
    MLA_OK = 0,
    MLA_ERR_ARG = 1,         /* invalid argument: shape, stride, alignment or NULL pointer   */
    MLA_ERR_UNSUPPORTED = 2, /* valid request outside what libmla implements (see each call) */
    MLA_ERR_ARCH = 3,        /* current device is not compute capability 10.3 (sm_103)       */
    MLA_ERR_CUDA = 4,        /* a CUDA runtime or driver call failed                          */
    MLA_ERR_WORKSPACE = 5,   /* workspace pointer NULL or smaller than mla_workspace_size     */
    MLA_ERR_DEVICE = 6       /* a kernel reported an error (see mla_check_device_error)       */
};

/* Device-side error bits, reported by mla_check_device_error. */
enum {
    MLA_DEVERR_TIMEOUT = 1,     /* a bounded wait inside a kernel gave up; outputs are invalid */
    MLA_DEVERR_BAD_BLOCK = 2    /* a needed block_table entry was outside [0, num_blocks)       */
};

/* int32 entries per tile_scheduler_metadata row (TileSchedulerMetaDataSize). */
#define MLA_METADATA_SIZE 8

/* Fixed dimensions of the MLA decode this library implements. */
#define MLA_HEAD_DIM 576        /* 512 latent + 64 RoPE dims of q and of each cache row */
#define MLA_HEAD_DIM_V 512      /* V = the first 512 dims of each cache row             */
#define MLA_PAGE_BLOCK_SIZE 64  /* cache rows per physical block                        */

/*
 * Problem description for mla_decode_fwd / mla_workspace_size.
 *
 *   q            (batch, s_q, h_q, head_dim) bf16;        q_stride   = {batch, token, head}
 *   k_cache      (num_blocks, page_block_size, h_k, head_dim) bf16;
 *                                                          k_stride   = {block, row, kv-head}
 *   block_table  (batch, max_blocks_per_seq) int32;        bt_stride  = elements per row
 *   out          (batch, s_q, h_q, head_dim_v) bf16;       out_stride = {batch, token, head}
 *   softmax_lse  (batch, h_q, s_q) fp32, contiguous.
 *
 * Requirements (else MLA_ERR_ARG): batch >= 0, s_q >= 1, h_k >= 1,
 * h_q % h_k == 0, head_dim == 576, head_dim_v == 512, page_block_size == 64,
 * num_blocks >= 1, max_blocks_per_seq >= 1, num_sm_parts >= 1; every stride a
 * multiple of 8 elements and every bf16 base pointer 16-byte aligned.
 * Limits (else MLA_ERR_UNSUPPORTED): s_q * h_q / h_k <= 1024 query rows per
 * KV head; batch <= 65535.
 */
typedef struct {
    int32_t batch;
    int32_t s_q;
    int32_t h_q;
    int32_t h_k;
    int32_t head_dim;
    int32_t head_dim_v;
    int32_t page_block_size;
    int32_t num_blocks;
    int32_t max_blocks_per_seq;
    int32_t num_sm_parts;      /* rows of tile_scheduler_metadata */
    int64_t q_stride[3];
    int64_t k_stride[3];
    int64_t bt_stride;
    int64_t out_stride[3];
} mla_shape_t;

/*
 * Number of scheduler parts (rows of tile_scheduler_metadata) that fill
 * `device` for the given head configuration: the number of two-CTA clusters
 * of the decode kernel that can be resident at once, divided by the number
 * of 128-row blocks per KV head and by num_heads_k (at least 1).
 * num_heads_per_head_k = s_q * h_q / h_k (vLLM page, get_mla_metadata
 * parameter table).  Errors: MLA_ERR_ARG (non-positive argument),
 * MLA_ERR_ARCH, MLA_ERR_CUDA.
 */
int mla_get_num_sm_parts(int device, int num_heads_per_head_k, int num_heads_k, int *num_sm_parts);

/*
 * Split-KV schedule (get_mla_metadata).  Reads cache_seqlens (device, int32,
 * `batch` entries) on the device and writes
 *   tile_scheduler_metadata  (num_sm_parts, MLA_METADATA_SIZE) int32, device
 *   num_splits               (batch + 1) int32, device: exclusive prefix sum
 *                            of the number of parts each sequence is split over
 * Record of part p: [begin_b, begin_blk, end_b, end_blk, first_slot,
 * num_blocks, 0, 0]; the part processes, for b in [begin_b, end_b], blocks
 * [b == begin_b ? begin_blk : 0, b == end_b ? end_blk : ceil(L_b / 64)).
 * Policy: greedy contiguous walk over (sequence, block) with a fixed cost of
 * c blocks per segment and a per-part target of
 * ceil((W + (num_sm_parts - 1) * c) / num_sm_parts), W = sum(n_b + c), where
 * c (the decode kernel's fixed work per segment in page times) is 6 for
 * num_heads_per_head_k >= 64 and 4 below, for a bf16 cache.
 * Errors: MLA_ERR_ARG (NULL pointer, batch < 0, num_sm_parts < 1,
 * num_heads_per_head_k < 1, num_heads_k < 1), MLA_ERR_UNSUPPORTED
 * (batch > 16384 or num_sm_parts > 1024), MLA_ERR_CUDA.
 */
int mla_get_metadata(const int32_t *cache_seqlens, int batch, int num_heads_per_head_k,
                     int num_heads_k, int num_sm_parts, int32_t *tile_scheduler_metadata,
                     int32_t *num_splits, mla_stream_t stream);

/*
 * mla_get_metadata for a cache of kv_bytes-byte elements (2: bf16, 1: e4m3,
 * for mla_decode_fwd_fp8): the segment cost c is one block more for e4m3,
 * whose pages take less time against the same fixed work.  Any schedule is
 * valid for either call; this one balances the parts for that cache.
 * Errors: as mla_get_metadata, and MLA_ERR_ARG for kv_bytes other than 1 or 2.
 */
int mla_get_metadata_ex(const int32_t *cache_seqlens, int batch, int num_heads_per_head_k,
                        int num_heads_k, int kv_bytes, int num_sm_parts, int32_t *tile_scheduler_metadata,
                        int32_t *num_splits, mla_stream_t stream);

/*
 * Bytes of workspace mla_decode_fwd needs for `shape`: fp32 partial outputs
 * and log-sum-exps of the sequences the schedule splits, for up to
 * batch + num_sm_parts splits.  Errors: MLA_ERR_ARG.
 */
int mla_workspace_size(const mla_shape_t *shape, size_t *bytes);

/*
 * Paged MLA decode (flash_mla_with_kvcache / fwd_kvcache_mla).  For every
 * sequence b, query token i < s_q and head h, with hk = h / (h_q / h_k),
 * L = cache_seqlens[b] and n = causal ? L - s_q + 1 + i : L (clamped to
 * [0, L]; bottom-right alignment):
 *   s_t = softmax_scale * q[b,i,h,:] . k[t, hk, :]       t < n, all 576 dims
 *   out[b,i,h,:]      = sum_t softmax(s)_t * k[t, hk, 0:512]   (V aliases K)
 *   softmax_lse[b,h,i] = ln sum_t exp(s_t)
 * where k[t] is row t % 64 of physical block block_table[b][t / 64].
 * Rows with n == 0 get out = 0 and softmax_lse = -inf.
 * softmax_scale <= 0 or NaN selects the default 1/sqrt(head_dim) (the
 * interface's default of q.shape[-1] ** -0.5).
 *
 * tile_scheduler_metadata / num_splits must come from mla_get_metadata on
 * the same cache_seqlens and num_sm_parts (not checked).  block_table
 * entries past ceil(L / 64) are never read; needed entries outside
 * [0, num_blocks) are not dereferenced and raise MLA_DEVERR_BAD_BLOCK.
 * workspace: device scratch of at least mla_workspace_size bytes, 256-byte
 * aligned, not used concurrently by another call.  workspace == NULL with
 * workspace_bytes == 0 selects the library's own stream-ordered workspace:
 * one buffer per (device, stream), allocated and grown with cudaMallocAsync
 * on `stream` (calls on one stream share it; calls on different streams get
 * different buffers) and released by mla_shutdown (the workspace
 * convention of the FlashMLA-PyTorch / vLLM pages leaves the scratch to the
 * library; the Ascend ATB page's size query plus caller buffer is the
 * explicit form).
 * Errors: MLA_ERR_ARG, MLA_ERR_UNSUPPORTED, MLA_ERR_ARCH, MLA_ERR_WORKSPACE,
 * MLA_ERR_CUDA.  Launches two kernels: mla_decode_splitkv then
 * mla_decode_combine, with the same arguments.
 */
int mla_decode_fwd(const mla_shape_t *shape, const void *q, const void *k_cache,
                   const int32_t *block_table, const int32_t *cache_seqlens,
                   const int32_t *tile_scheduler_metadata, const int32_t *num_splits,
                   float softmax_scale, int causal, void *out, float *softmax_lse,
                   void *workspace, size_t workspace_bytes, mla_stream_t stream);

/*
 * The first of the two launches of mla_decode_fwd: the persistent split-KV
 * decode.  Sequences the schedule does not split are finished here (out and
 * softmax_lse written); split ones leave fp32 partials in the workspace.
 */
int mla_decode_splitkv(const mla_shape_t *shape, const void *q, const void *k_cache,
                       const int32_t *block_table, const int32_t *cache_seqlens,
                       const int32_t *tile_scheduler_metadata, const int32_t *num_splits,
                       float softmax_scale, int causal, void *out, float *softmax_lse,
                       void *workspace, size_t workspace_bytes, mla_stream_t stream);

/*
 * The second launch of mla_decode_fwd: merges the partials of every split
 * sequence by log-sum-exp weighting (lse = ln sum_s exp(lse_s),
 * out = sum_s exp(lse_s - lse) * out_s) and writes out / softmax_lse for
 * them, and out = 0, softmax_lse = -inf for empty sequences.
 * Same arguments as mla_decode_fwd (q, k_cache and block_table unused).
 */
int mla_decode_combine(const mla_shape_t *shape, const void *q, const void *k_cache,
                       const int32_t *block_table, const int32_t *cache_seqlens,
                       const int32_t *tile_scheduler_metadata, const int32_t *num_splits,
                       float softmax_scale, int causal, void *out, float *softmax_lse,
                       void *workspace, size_t workspace_bytes, mla_stream_t stream);

/*
 * Size of the scratch built into the library for mla_decode_fwd_noalloc:
 * 64 MiB of device memory on every GPU that loads the library, held until
 * the process exits.
 */
#define MLA_NOALLOC_SCRATCH_BYTES (64u * 1024u * 1024u)

/*
 * mla_decode_fwd without a workspace argument, for callers that cannot
 * allocate device memory themselves: code whose device memory is owned by
 * another allocator (an inference server's pool, say) or a latency-critical
 * loop that cannot afford the device-wide synchronisation cudaMalloc or
 * cudaFree may cause.  The split partials go to a scratch array built into
 * the library (MLA_NOALLOC_SCRATCH_BYTES); this call allocates nothing.
 * The pages this library follows have no counterpart of this call.
 *
 * Arguments, results and errors as mla_decode_fwd, plus MLA_ERR_UNSUPPORTED
 * (with a message giving both sizes) when mla_workspace_size(shape) exceeds
 * MLA_NOALLOC_SCRATCH_BYTES.  The first call on a device looks up the
 * scratch's device address with that device current; make it before any
 * stream capture (and again after mla_shutdown, which forgets it).  All calls share the one scratch array: calls whose
 * kernels may overlap on the GPU (unordered streams) race on it and must not
 * be issued.  Nothing in the scratch needs clearing between calls.
 */
int mla_decode_fwd_noalloc(const mla_shape_t *shape, const void *q, const void *k_cache,
                           const int32_t *block_table, const int32_t *cache_seqlens,
                           const int32_t *tile_scheduler_metadata, const int32_t *num_splits,
                           float softmax_scale, int causal, void *out, float *softmax_lse,
                           mla_stream_t stream);

/*
 * Strides (elements) of the RoPE tensors of mla_decode_fwd_split.
 */
typedef struct {
    int64_t q_rope_stride[3];   /* q_rope (batch, s_q, h_q, 64): {batch, token, head}            */
    int64_t krope_stride[3];    /* krope (num_blocks, 64, h_k, 64): {block, row, kv-head}          */
} mla_rope_strides_t;

/*
 * mla_decode_fwd on split inputs: the latent and RoPE parts of the query and
 * of the cache in separate tensors, the layout of the Ascend ATB MLA page
 * (parameter table: qNope, qRope, ctKV, kRope; cacheMode 1, separate
 * caches).  The result is that of mla_decode_fwd on the concatenations
 * q = [q_nope | q_rope] and k_cache = [ctkv | krope] along the last
 * dimension; V is ctkv.
 *   q_nope  (batch, s_q, h_q, 512) bf16   strides shape->q_stride
 *   q_rope  (batch, s_q, h_q, 64) bf16    strides rope->q_rope_stride
 *   ctkv    (num_blocks, 64, h_k, 512) bf16  strides shape->k_stride
 *   krope   (num_blocks, 64, h_k, 64) bf16   strides rope->krope_stride
 * shape->head_dim stays 576 (the logical q . k length).  Every pointer
 * 16-byte aligned, every stride a positive multiple of 8 elements, head
 * strides at least the head's dims.  Everything else (schedule, workspace,
 * errors, the two launches) as mla_decode_fwd.  Both calls read the same
 * bytes from HBM for the same problem.
 */
int mla_decode_fwd_split(const mla_shape_t *shape, const mla_rope_strides_t *rope,
                         const void *q_nope, const void *q_rope, const void *ctkv, const void *krope,
                         const int32_t *block_table, const int32_t *cache_seqlens,
                         const int32_t *tile_scheduler_metadata, const int32_t *num_splits,
                         float softmax_scale, int causal, void *out, float *softmax_lse,
                         void *workspace, size_t workspace_bytes, mla_stream_t stream);

/*
 * mla_decode_fwd over an e4m3 (FP8, 1 sign, 4 exponent, 3 mantissa bits)
 * query and latent cache, with the two fused product scales of the FlashInfer
 * page (trtllm_batch_decode_with_kv_cache_mla, the note on bmm1_scale and
 * bmm2_scale):
 *   s_t = bmm1_scale * sum_{d < 576} q[d] * k[t][d]
 *   out = bmm2_scale * sum_t softmax(s)_t * k[t][0:512]      (bf16)
 *   softmax_lse = ln sum_t exp(s_t)                           (fp32)
 * with q and k the e4m3 values as stored.  bmm1_scale folds the query and key
 * dequantisation scales into the softmax scale; bmm2_scale is the value
 * dequantisation scale.
 *   q        (batch, s_q, h_q, 576) e4m3 bytes      strides shape->q_stride (elements = bytes)
 *   k_cache  (num_blocks, 64, h_k, 576) e4m3 bytes  strides shape->k_stride
 *   out      (batch, s_q, h_q, 512) bf16, softmax_lse (batch, h_q, s_q) fp32, as mla_decode_fwd
 * Masking, schedule (mla_get_metadata), workspace (NULL = internal) and the
 * two launches are those of mla_decode_fwd.
 *
 * Accuracy.  The probabilities are rounded to e4m3 for the PV product (the
 * denominator sums them unrounded): each weight errs by up to 2^-4 of itself, and below 2^-6 of its
 * row's largest by up to 2^-10 of that one, so that many keys 7 nats or more below a few others may
 * lose their part.
 * With more than 32 query rows per KV head the two halves of each logit,
 * s_0 and s_1 (latent dims 0-255 + RoPE dims 512-543, and the rest), are
 * rounded to bf16 before they are added, which moves a logit by at most
 * bmm1_scale * 2^-8 * (|s_0| + |s_1|) and softmax_lse by at most the
 * probability-weighted mean of those moves.
 *
 * Errors: as mla_decode_fwd, and MLA_ERR_ARG when bmm1_scale is not positive
 * and finite, bmm2_scale not finite, or a q / k_cache stride is not a
 * multiple of 16 bytes.
 */
int mla_decode_fwd_fp8(const mla_shape_t *shape, const void *q, const void *k_cache,
                       const int32_t *block_table, const int32_t *cache_seqlens,
                       const int32_t *tile_scheduler_metadata, const int32_t *num_splits,
                       float bmm1_scale, float bmm2_scale, int causal, void *out, float *softmax_lse,
                       void *workspace, size_t workspace_bytes, mla_stream_t stream);

/*
 * The first of the two launches of mla_decode_fwd_fp8 (the e4m3 split-KV
 * decode), with its arguments; the second is mla_decode_combine on the same
 * workspace, which merges split sequences exactly as for bf16 inputs (the
 * partials already carry bmm2_scale).  A NULL workspace selects the same
 * internal one for both calls on one stream.
 */
int mla_decode_splitkv_fp8(const mla_shape_t *shape, const void *q, const void *k_cache,
                           const int32_t *block_table, const int32_t *cache_seqlens,
                           const int32_t *tile_scheduler_metadata, const int32_t *num_splits,
                           float bmm1_scale, float bmm2_scale, int causal, void *out, float *softmax_lse,
                           void *workspace, size_t workspace_bytes, mla_stream_t stream);

/*
 * One whole decode step from host buffers: copies q, block_table and
 * cache_seqlens to the device, computes the schedule (mla_get_metadata with
 * shape->num_sm_parts parts), decodes (mla_decode_fwd) and returns out and
 * softmax_lse to host memory, all enqueued on `stream` -- the sequence of the
 * FlashMLA-PyTorch page's usage (get_mla_metadata from cache_seqlens, then
 * flash_mla_with_kvcache) with the host transfers around it.  The results are in
 * the host buffers once `stream` has completed; the inputs must stay
 * unchanged until then.
 *   q_host              host, bf16, laid out by shape->q_stride
 *   block_table_host    host, int32, row stride shape->bt_stride
 *   cache_seqlens_host  host, int32, batch entries
 *   k_cache             DEVICE (the cache stays resident), as mla_decode_fwd
 *   out_host            host, bf16 (batch, s_q, h_q, 512), contiguous:
 *                       shape->out_stride must be {s_q*h_q*512, h_q*512, 512}
 *   softmax_lse_host    host, fp32 (batch, h_q, s_q), contiguous
 * Host buffers should be page-locked (cudaHostAlloc, cudaHostRegister) for
 * the copies to be asynchronous; pageable memory works, with copies that
 * block the host.  When out_host / softmax_lse_host are page-locked and
 * mapped into the device's address space, the kernels store the results
 * there directly and no device-to-host copy is made; otherwise they are
 * staged in device memory and copied back.  The schedule runs on a second,
 * library-owned stream while q is copied, and `stream` waits for it before
 * the decode, so work enqueued on `stream` afterwards is ordered after the
 * whole step.
 * Device staging (inputs, schedule, workspace, output staging) is one
 * buffer per (device, stream), allocated and grown with cudaMallocAsync on
 * `stream`, and released, with the second stream, by mla_shutdown.
 * batch == 0 enqueues nothing (the pointers may then be NULL).
 * Errors: as mla_decode_fwd and mla_get_metadata (MLA_ERR_UNSUPPORTED for
 * batch > 16384 or num_sm_parts > 1024), plus MLA_ERR_ARG for a
 * non-contiguous out.  A CUDA failure after the first copy was enqueued
 * returns MLA_ERR_CUDA with part of the step enqueued.
 */
int mla_decode_fwd_host(const mla_shape_t *shape, const void *q_host, const void *k_cache,
                        const int32_t *block_table_host, const int32_t *cache_seqlens_host,
                        float softmax_scale, int causal, void *out_host, float *softmax_lse_host,
                        mla_stream_t stream);

/* Element types of the rotary, append and chunk calls. */
enum {
    MLA_DTYPE_BF16 = 0,
    MLA_DTYPE_F16 = 1,
    MLA_DTYPE_F32 = 2,
    MLA_DTYPE_E4M3 = 3   /* 8-bit float as in mla_decode_fwd_fp8; values are rounded to it saturating at +-448 */
};

/* Scaling of the rotary frequencies for contexts longer than the trained one. */
enum {
    MLA_ROPE_PLAIN = 0,
    MLA_ROPE_LINEAR = 1,   /* every frequency divided by `factor` */
    MLA_ROPE_YARN = 2      /* frequencies by parts, see mla_rope_init */
};

typedef struct {
    int32_t kind;                  /* MLA_ROPE_* */
    double factor;                 /* >= 1 */
    double original_max_position;  /* trained context (yarn) */
    double beta_fast, beta_slow;   /* turns over the trained context between which the ramp lies (yarn) */
    double mscale, mscale_all_dim; /* factor on cos and sin (yarn): see mla_rope_init */
} mla_rope_scaling_t;

#define MLA_ROPE_MAX_PAIRS 128

/* What the rotating calls need of a rotary embedding, filled by mla_rope_init; passed by
 * value to the kernels, so it lives in host memory and needs no device copy. */
typedef struct {
    int32_t rotary_dim;                    /* rotated dims of a head */
    int32_t interleaved;                   /* 1: pairs (2i, 2i + 1); 0: pairs (i, i + rotary_dim / 2) */
    float factor;                          /* on cos and sin */
    int32_t reserved;
    uint64_t turns[MLA_ROPE_MAX_PAIRS];    /* frequency of each pair, turns per position times 2^64 */
} mla_rope_plan_t;

/*
 * Fills *plan.  Pair i of rotary_dim / 2 has the frequency f_i = theta^(-2i / rotary_dim)
 * radians per position; scaling (NULL: MLA_ROPE_PLAIN) changes it:
 *   MLA_ROPE_LINEAR  f_i / factor
 *   MLA_ROPE_YARN    f_i (1 - r_i) + f_i / factor * r_i, where r_i rises from 0 to 1 between the
 *                    pairs lo and hi: with c(t) = rotary_dim ln(original_max_position / (2 pi t)) / (2 ln theta),
 *                    lo = max(floor(c(beta_fast)), 0), hi = min(ceil(c(beta_slow)), rotary_dim - 1),
 *                    r_i = clamp((i - lo) / max(hi - lo, 0.001), 0, 1); cos and sin are multiplied by
 *                    (1 + 0.1 mscale ln factor) / (1 + 0.1 mscale_all_dim ln factor).
 * Host only, no CUDA call.  Errors: MLA_ERR_ARG (rotary_dim odd or outside [2, 256], theta < 1
 * or not finite, factor < 1, an invalid scaling).
 */
int mla_rope_init(mla_rope_plan_t *plan, int rotary_dim, int interleaved, double theta,
                  const mla_rope_scaling_t *scaling);

/*
 * Shape of mla_rope: x and out (batch, tokens, heads, head_dim), positions (batch, tokens)
 * contiguous int32.  Strides in elements of the tensor's own type, {batch, token, head}; the
 * last dimension is contiguous.  Any alignment of whole elements works; rows whose addresses
 * and dims are multiples of 16 bytes take the wide path.
 */
typedef struct {
    int32_t batch, tokens, heads, head_dim;
    int32_t rope_offset;   /* first rotated dim of a head */
    int32_t dtype;         /* of x: MLA_DTYPE_BF16, _F16 or _F32 */
    int32_t out_dtype;     /* dtype, or MLA_DTYPE_E4M3 */
    int64_t x_stride[3], out_stride[3];
} mla_rope_shape_t;

/*
 * Rotary positions: out = x with the dims [rope_offset, rope_offset + rotary_dim) of every head
 * rotated, (a, b) -> factor * (a cos t - b sin t, b cos t + a sin t), t = position * frequency
 * (inverse != 0: -t, which is also the gradient of the forward call; it undoes that call where factor is 1).
 * The reduction modulo one turn is exact for every int32 position; the frequency is a 64-bit float's, which
 * leaves an angle off by up to |position * frequency| * 2^-52; cos and sin are fp32; each value is rounded
 * once, to out_dtype.  e4m3 values are multiplied by out_scale first (1 for the other types).
 * out == x (same type and strides) rotates in place and leaves the other dims alone; otherwise
 * they are copied, and x and out must not overlap in any other way.
 * What is written (whole rows, in place their rotated dims) must not overlap itself: of the dimensions with more
 * than one entry, by rising stride, each steps past all that those before it span (else MLA_ERR_ARG).
 * One launch.  Errors: MLA_ERR_ARG, MLA_ERR_UNSUPPORTED (batch * tokens * heads above 2^31 - 1025),
 * MLA_ERR_ARCH, MLA_ERR_CUDA.
 */
int mla_rope(const mla_rope_plan_t *plan, const mla_rope_shape_t *shape, const void *x, const int32_t *positions,
             int inverse, void *out, float out_scale, mla_stream_t stream);

/*
 * Shape of mla_cache_append.  latent (total_tokens, h_k, 512) and k_rope (total_tokens, h_k, 64)
 * bf16 with strides {token, KV head}; the cache as mla_decode_fwd's (strides {block, row, KV head}),
 * or latent and RoPE parts in two tensors as mla_decode_fwd_split's.
 */
typedef struct {
    int32_t batch, total_tokens, h_k;
    int32_t page_block_size, num_blocks, max_blocks_per_seq;
    int32_t kv_dtype;            /* MLA_DTYPE_BF16 or MLA_DTYPE_E4M3 */
    int64_t latent_stride[2], k_rope_stride[2];
    int64_t k_stride[3];         /* of k_cache */
    int64_t krope_stride[3];     /* of krope_cache (ignored when it is NULL) */
    int64_t bt_stride;
} mla_append_shape_t;

/*
 * Writes the cache rows of new tokens.  Sequence b's new tokens are cu_seqlens_q[b] ..
 * cu_seqlens_q[b + 1] - 1 (device, batch + 1 entries, non-decreasing, from 0), or with
 * cu_seqlens_q == NULL total_tokens / batch each; they are its last ones:  token i of n goes to
 * position cache_seqlens[b] - n + i (cache_seqlens includes them), i.e. row position % 64 of
 * physical block block_table[b][position / 64].  The 512 latent dims are stored as they are, the
 * 64 rotary dims rotated by plan (rotary_dim 64) at that position, or at positions[token] when
 * positions is not NULL.  k_cache holds rows of 576 dims when krope_cache is NULL, else 512 dims
 * with the rotated 64 in krope_cache.  An e4m3 cache takes the values times kv_scale, saturating
 * at +-448; a bf16 one needs kv_scale == 1.  Every value is rounded once.
 * Tokens outside every sequence are padding and are skipped.  A position that is negative or past
 * the block table, or a block outside [0, num_blocks), is not stored and raises
 * MLA_DEVERR_BAD_BLOCK.  (An e4m3 cache in two tensors is for readers of the caller's own: the split calls of this
 * library take bf16 alone.)  All other cache rows stay as they are.  Two tokens that the table sends
 * to one row leave either's values.  One launch.
 * Alignment: latent and k_rope 16 bytes, caches 16 (e4m3: 8), strides multiples of 8 elements.
 * The caches' rows must not overlap: as mla_rope's.
 * Errors: MLA_ERR_ARG, MLA_ERR_UNSUPPORTED (total_tokens * h_k above 2^31 - 65), MLA_ERR_ARCH,
 * MLA_ERR_CUDA.
 */
int mla_cache_append(const mla_append_shape_t *shape, const mla_rope_plan_t *plan, const void *latent,
                     const void *k_rope, const int32_t *block_table, const int32_t *cu_seqlens_q,
                     const int32_t *cache_seqlens, const int32_t *positions, void *k_cache, void *krope_cache,
                     float kv_scale, mla_stream_t stream);

/*
 * Shape of the chunk attention: a ragged batch of new tokens over the paged cache.
 *   q            (total_q, h_q, 576) bf16;   q_stride = {token, head}
 *   k_cache      (num_blocks, 64, h_k, 576) bf16; k_stride = {block, row, kv-head}
 *   block_table  (batch, max_blocks_per_seq) int32; bt_stride = elements per row
 *   out          (total_q, h_q, 512) bf16;   out_stride = {token, head}
 *   softmax_lse  (total_q, h_q) fp32, contiguous
 * Requirements (else MLA_ERR_ARG): as mla_shape_t's, and the rows of out must not overlap (as mla_rope's); no limit on
 * the query rows per KV head.
 * Limits (else MLA_ERR_UNSUPPORTED): batch <= 16384, num_parts <= 1024,
 * max_blocks_per_seq <= 2^24, total_q * h_q <= 2^31 - 1025.
 */
typedef struct {
    int32_t batch, total_q;
    int32_t h_q, h_k, head_dim, head_dim_v;
    int32_t page_block_size, num_blocks, max_blocks_per_seq;
    int32_t num_parts;         /* rows of chunk_metadata */
    int64_t q_stride[2];
    int64_t k_stride[3];
    int64_t bt_stride;
    int64_t out_stride[2];
} mla_chunk_shape_t;

/* Parts (rows of chunk_metadata) that fill `device`.  Errors: as mla_get_num_sm_parts. */
int mla_chunk_get_num_parts(int device, int *num_parts);

/*
 * Schedule of the chunk attention: reads cu_seqlens_q (batch + 1) and cache_seqlens (batch) on the
 * device and writes chunk_metadata (num_parts, MLA_METADATA_SIZE) int32.  The query rows of each
 * (sequence, KV head) are cut into blocks of 128 and the keys a block sees into tiles of 128; part
 * p's record [begin_b, begin_block, begin_tile, end_b, end_block, end_tile, 0, 0] gives it the tiles
 * from the first triple up to the second (blocks of a sequence count KV head by KV head).  The
 * stretches are contiguous, in order, cover everything once and cost about the same.  One call per
 * step serves every layer.  Any schedule is valid for any lengths; this one balances these.
 * Errors: MLA_ERR_ARG, MLA_ERR_UNSUPPORTED (the limits above), MLA_ERR_ARCH, MLA_ERR_CUDA.
 */
int mla_chunk_get_metadata(const int32_t *cu_seqlens_q, const int32_t *cache_seqlens, int batch, int total_q, int h_q,
                           int h_k, int causal, int num_parts, int32_t *chunk_metadata, mla_stream_t stream);

/* Bytes of workspace for `shape`: fp32 partials of two blocks per part.  Errors: MLA_ERR_ARG, MLA_ERR_UNSUPPORTED. */
int mla_chunk_workspace_size(const mla_chunk_shape_t *shape, size_t *bytes);

/*
 * Attention of a ragged batch of chunks of new tokens over the paged cache (which holds their own
 * keys: mla_cache_append comes first).  Sequence b's queries are the n_b tokens cu_seqlens_q[b] ..
 * cu_seqlens_q[b + 1] - 1, the last of its L = cache_seqlens[b] positions.  Token i and head h see
 * n = causal ? L - n_b + 1 + i : L keys, clamped to [0, L], and out, softmax_lse, the default scale,
 * rows without a key, bad blocks and reads of the cache are as in mla_decode_fwd.  Sequences may
 * have no new tokens or no keys.  Tokens outside every sequence are padding: their rows of out and
 * softmax_lse stay as they are.  A cache length past the block table raises MLA_DEVERR_BAD_BLOCK and
 * is cut to it.  Cache rows at and past L may hold anything.  A NaN or an infinity in a row below L is the
 * sequence's own: it may reach every query of a block of 128 rows in which one sees that key, also those
 * that the causal mask keeps from it (weight 0 times NaN).  out and softmax_lse must not overlap the inputs.
 * Two launches: the attention, and the merge of blocks that the schedule cuts.
 * workspace: mla_chunk_workspace_size bytes, 256-byte aligned, not used concurrently by another
 * call; NULL with workspace_bytes == 0 selects the library's own of (device, stream), which a call
 * captured into a graph must not use (MLA_ERR_WORKSPACE).  It is the decode's too: threads that share a
 * stream, and callers that put work between mla_decode_splitkv and mla_decode_combine, bring their own.
 * Errors: MLA_ERR_ARG, MLA_ERR_UNSUPPORTED, MLA_ERR_ARCH, MLA_ERR_WORKSPACE, MLA_ERR_CUDA.
 */
int mla_chunk_fwd(const mla_chunk_shape_t *shape, const void *q, const void *k_cache, const int32_t *block_table,
                  const int32_t *cu_seqlens_q, const int32_t *cache_seqlens, const int32_t *chunk_metadata,
                  float softmax_scale, int causal, void *out, float *softmax_lse, void *workspace,
                  size_t workspace_bytes, mla_stream_t stream);

/* Strides (elements) of the RoPE tensors of mla_chunk_fwd_split. */
typedef struct {
    int64_t q_rope_stride[2];   /* q_rope (total_q, h_q, 64): {token, head}              */
    int64_t krope_stride[3];    /* krope (num_blocks, 64, h_k, 64): {block, row, kv-head} */
} mla_chunk_rope_strides_t;

/* mla_chunk_fwd on split inputs, as mla_decode_fwd_split is to mla_decode_fwd: q_nope
 * (total_q, h_q, 512), q_rope (total_q, h_q, 64), ctkv (num_blocks, 64, h_k, 512), krope
 * (num_blocks, 64, h_k, 64), all bf16. */
int mla_chunk_fwd_split(const mla_chunk_shape_t *shape, const mla_chunk_rope_strides_t *rope, const void *q_nope,
                        const void *q_rope, const void *ctkv, const void *krope, const int32_t *block_table,
                        const int32_t *cu_seqlens_q, const int32_t *cache_seqlens, const int32_t *chunk_metadata,
                        float softmax_scale, int causal, void *out, float *softmax_lse, void *workspace,
                        size_t workspace_bytes, mla_stream_t stream);

/* mla_chunk_fwd over an e4m3 query and cache, with the product scales of mla_decode_fwd_fp8
 * (logits bmm1_scale * q.k, out times bmm2_scale).  Strides of q and k_cache are multiples of 16
 * elements.
 * Accuracy.  For the second product a softmax weight is held to 2^-8 of itself down to 2^-10.5 of its
 * row's largest weight or less.  Smaller ones have fewer bits and are rounded up or down so that each is right in the
 * mean to 2^-8 of itself, down to 2^-29 of the largest: a single one is off by less than a quarter of itself (or 2^-20
 * of the largest), the sum over many by much less.  The rounding depends on the row, the key's place and the schedule
 * alone: the same call gives the same bits.  softmax_lse has unrounded weights. */
int mla_chunk_fwd_fp8(const mla_chunk_shape_t *shape, const void *q, const void *k_cache, const int32_t *block_table,
                      const int32_t *cu_seqlens_q, const int32_t *cache_seqlens, const int32_t *chunk_metadata,
                      float bmm1_scale, float bmm2_scale, int causal, void *out, float *softmax_lse, void *workspace,
                      size_t workspace_bytes, mla_stream_t stream);

/*
 * Releases the internal workspaces that calls without a workspace allocated
 * and the staging buffers and streams of mla_decode_fwd_host (synchronizing
 * each device that holds one first).  Later such calls
 * allocate again.  It also forgets what the library set up per device
 * (kernel attributes, the device addresses of its error word and of the
 * built-in scratch of mla_decode_fwd_noalloc, cache tensor maps), which the
 * next call on each device sets up again: call it before resetting a device
 * (cudaDeviceReset), since the reset may reload the library's module at
 * other addresses.  Not to be called while another thread uses the library.
 * Errors: MLA_ERR_CUDA.
 */
int mla_shutdown(void);

/*
 * Synchronizes the current device, then stores in *bits the OR of the
 * MLA_DEVERR_* bits kernels of this library raised on it since the last
 * clear, and clears them when `clear` is non-zero.  Returns MLA_OK, or
 * MLA_ERR_CUDA when synchronization itself failed.
 */
int mla_check_device_error(int *bits, int clear);

/* Static description of a status code. */
const char *mla_status_string(int status);

/* Detail message of the last failing call on the calling thread ("" if none). */
const char *mla_last_error(void);

/* Library version, as major * 10000 + minor * 100 + patch. */
int mla_version(void);

#ifdef __cplusplus
}
#endif

#endif /* LIBMLA_H */
