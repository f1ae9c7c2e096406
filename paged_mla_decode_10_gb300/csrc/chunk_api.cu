// chunk_api.cu -- entry points of the chunk attention: checks, schedule, launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "api_internal.h"
#include "chunk_common.cuh"

namespace mla {
__global__ void mla_chunk_metadata_kernel(const int32_t *cu, const int32_t *seqlens, int batch, int total_q, int h_k, int hpk,
                                          int causal, int parts, int32_t *md);
size_t chunk_metadata_smem_bytes(int batch);
uint32_t chunk_metadata_threads();
int launch_chunk_combine(const ChunkParams &p, cudaStream_t stream);
namespace chunk_bf16 {
int launch(const ChunkParams &p, const void *latent, const int64_t *l_s, const void *rope, const int64_t *r_s, cudaStream_t stream);
}
namespace chunk_f8 {
int launch(const ChunkParams &p, const void *latent, const int64_t *l_s, const void *rope, const int64_t *r_s, cudaStream_t stream);
}
}  // namespace mla

namespace {

using namespace mla;

constexpr int kMaxChunkBatch = 16384;
constexpr int kMaxChunkParts = 1024;

int check_chunk_shape(const mla_chunk_shape_t *sh) {
    if (!sh) return report_error(MLA_ERR_ARG, "shape is NULL");
    if (sh->batch < 0 || sh->total_q < 0) return report_errorf(MLA_ERR_ARG, "batch %d or total_q %d < 0", sh->batch, sh->total_q);
    if (sh->h_q < 1 || sh->h_k < 1 || sh->h_q % sh->h_k)
        return report_errorf(MLA_ERR_ARG, "h_q %d must be a positive multiple of h_k %d", sh->h_q, sh->h_k);
    if (sh->head_dim != MLA_HEAD_DIM || sh->head_dim_v != MLA_HEAD_DIM_V)
        return report_errorf(MLA_ERR_ARG, "head_dim must be 576 and head_dim_v 512 (got %d, %d)", sh->head_dim, sh->head_dim_v);
    if (sh->page_block_size != MLA_PAGE_BLOCK_SIZE)
        return report_errorf(MLA_ERR_ARG, "page_block_size must be 64 (got %d)", sh->page_block_size);
    if (sh->num_blocks < 1 || sh->max_blocks_per_seq < 1)
        return report_error(MLA_ERR_ARG, "num_blocks and max_blocks_per_seq must be >= 1");
    if (sh->max_blocks_per_seq > (1 << 24)) return report_errorf(MLA_ERR_UNSUPPORTED, "max_blocks_per_seq %d > 2^24", sh->max_blocks_per_seq);
    if (sh->num_parts < 1) return report_error(MLA_ERR_ARG, "num_parts must be >= 1");
    if (sh->batch > kMaxChunkBatch) return report_errorf(MLA_ERR_UNSUPPORTED, "batch %d > %d", sh->batch, kMaxChunkBatch);
    if (sh->num_parts > kMaxChunkParts) return report_errorf(MLA_ERR_UNSUPPORTED, "num_parts %d > %d", sh->num_parts, kMaxChunkParts);
    if ((int64_t)sh->total_q * sh->h_q > 0x7fffffffll - 1024)
        return report_error(MLA_ERR_UNSUPPORTED, "total_q * h_q exceeds 2^31 - 1025");
    for (int i = 0; i < 2; ++i)
        if (sh->q_stride[i] <= 0 || sh->q_stride[i] % 8 || sh->out_stride[i] <= 0 || sh->out_stride[i] % 8)
            return report_error(MLA_ERR_ARG, "strides must be positive multiples of 8 elements");
    for (int i = 0; i < 3; ++i)
        if (sh->k_stride[i] <= 0 || sh->k_stride[i] % 8) return report_error(MLA_ERR_ARG, "strides must be positive multiples of 8 elements");
    // rows of out are written: they must not overlap
    const int64_t n[2] = {sh->total_q, sh->h_q};
    if (!rows_apart(n, sh->out_stride, 2, MLA_HEAD_DIM_V))
        return report_error(MLA_ERR_ARG, "out rows overlap (a stride smaller than what the other spans)");
    if (sh->bt_stride < sh->max_blocks_per_seq) return report_error(MLA_ERR_ARG, "bt_stride < max_blocks_per_seq");
    return MLA_OK;
}

size_t chunk_workspace(int parts, size_t *lse_off) {
    const size_t rows = (size_t)parts * kSlotsPerPart * kBlockRows;
    const size_t o = rows * MLA_HEAD_DIM_V * sizeof(float);   // a multiple of 256
    if (lse_off) *lse_off = o;
    return o + rows * sizeof(float);
}

// Where the query and the cache come from: rows of 576 dims, or separate latent and RoPE parts.
struct ChunkSource {
    int elem = 2;
    const void *q, *q_rope, *latent, *rope;
    int64_t q_s[2], qr_s[2], l_s[3], r_s[3];
    bool split = false;
};

int chunk_run(const mla_chunk_shape_t *sh, const ChunkSource &src, const int32_t *block_table, const int32_t *cu,
              const int32_t *seqlens, const int32_t *md, float scale, float out_scale, int causal, void *out, float *lse,
              void *ws, size_t ws_bytes, mla_stream_t stream) {
    if (sh->total_q == 0 || sh->batch == 0) return MLA_OK;   // no token, or padding only
    if (!src.q || !src.q_rope || !src.latent || !src.rope || !block_table || !cu || !seqlens || !md || !out || !lse)
        return report_error(MLA_ERR_ARG, "NULL tensor pointer");
    if (!is_aligned(src.q, 16) || !is_aligned(src.q_rope, 16) || !is_aligned(src.latent, 16) || !is_aligned(src.rope, 16))
        return report_error(MLA_ERR_ARG, "query and cache must be 16-byte aligned");
    if (!is_aligned(out, 16)) return report_error(MLA_ERR_ARG, "out must be 16-byte aligned");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    size_t lse_off = 0;
    const size_t need = chunk_workspace(sh->num_parts, &lse_off);
    DeviceInfo di;
    int st = device_info(&di);
    if (st != MLA_OK) return st;
    if (!ws && ws_bytes == 0) {
        // a captured graph would keep the address of a buffer that later calls may free or share
        cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
        const cudaError_t e = cudaStreamIsCapturing(s, &cap);
        if (e != cudaSuccess) return report_cuda(e, "cudaStreamIsCapturing");
        if (cap != cudaStreamCaptureStatusNone)
            return report_errorf(MLA_ERR_WORKSPACE, "pass a workspace (%zu bytes) to a call that is captured into a graph", need);
        if ((st = stream_workspace(need, s, &ws, &ws_bytes)) != MLA_OK) return st;
    }
    if (!ws) return report_errorf(MLA_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", need);
    if (!is_aligned(ws, 256)) return report_error(MLA_ERR_WORKSPACE, "workspace not 256-byte aligned");
    if (ws_bytes < need) return report_errorf(MLA_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", ws_bytes, need);

    ChunkParams p;
    memset(&p, 0, sizeof p);
    p.block_table = block_table;
    p.bt_stride = sh->bt_stride;
    p.cu = cu;
    p.seqlens = seqlens;
    p.md = md;
    p.q = src.q;
    p.q_rope = src.q_rope;
    p.q_s0 = src.q_s[0]; p.q_s1 = src.q_s[1];
    p.qr_s0 = src.qr_s[0]; p.qr_s1 = src.qr_s[1];
    p.out = static_cast<uint16_t *>(out);
    p.o_s0 = sh->out_stride[0]; p.o_s1 = sh->out_stride[1];
    p.lse = lse;
    p.ws_o = static_cast<float *>(ws);
    p.ws_lse = reinterpret_cast<float *>(static_cast<char *>(ws) + lse_off);
    p.err = di.err_word;
    p.batch = sh->batch; p.total_q = sh->total_q; p.h_q = sh->h_q; p.h_k = sh->h_k; p.hpk = sh->h_q / sh->h_k;
    int log2 = 0;
    while ((1ll << log2) < p.hpk) ++log2;
    p.hpk_shift = 31 + log2;
    p.hpk_mul = (uint32_t)(((1ull << p.hpk_shift) + p.hpk - 1) / p.hpk);
    p.num_blocks = sh->num_blocks;
    p.max_blocks = sh->max_blocks_per_seq;
    p.num_parts = sh->num_parts;
    p.causal = causal ? 1 : 0;
    p.rope_x0 = src.split ? 0 : MLA_HEAD_DIM_V;
    p.scale_log2 = (float)((double)scale * 1.4426950408889634);
    p.out_scale = out_scale;
    // a concatenated cache's RoPE boxes come through a map over whole rows, from its base
    const void *rope = src.split ? src.rope : src.latent;
    st = src.elem == 1 ? chunk_f8::launch(p, src.latent, src.l_s, rope, src.r_s, s)
                       : chunk_bf16::launch(p, src.latent, src.l_s, rope, src.r_s, s);
    if (st != MLA_OK) return st;
    const int e = launch_chunk_combine(p, s);
    return e == 0 ? MLA_OK : report_cuda((cudaError_t)e, "chunk combine launch");
}

// Rows of 576 dims: the RoPE parts lie 512 elements behind the latent ones.
ChunkSource concat_rows(const mla_chunk_shape_t *sh, const void *q, const void *k, int elem) {
    ChunkSource c;
    c.elem = elem;
    c.q = q;
    c.latent = k;
    c.q_rope = q ? static_cast<const char *>(q) + MLA_HEAD_DIM_V * elem : nullptr;
    c.rope = k ? static_cast<const char *>(k) + MLA_HEAD_DIM_V * elem : nullptr;
    for (int i = 0; i < 2; ++i) c.q_s[i] = c.qr_s[i] = sh->q_stride[i];
    for (int i = 0; i < 3; ++i) c.l_s[i] = c.r_s[i] = sh->k_stride[i];
    return c;
}

float default_scale(float scale) {
    return scale > 0.f && std::isfinite(scale) ? scale : 1.0f / std::sqrt((float)MLA_HEAD_DIM);
}

}  // namespace

extern "C" {

int mla_chunk_get_num_parts(int device, int *num_parts) {
    if (!num_parts) return report_error(MLA_ERR_ARG, "num_parts is NULL");
    // one part per two-CTA cluster of the attention kernel: as many as the decode's with one row block
    return mla_get_num_sm_parts(device, 1, 1, num_parts);
}

int mla_chunk_get_metadata(const int32_t *cu_seqlens_q, const int32_t *cache_seqlens, int batch, int total_q, int h_q,
                           int h_k, int causal, int num_parts, int32_t *chunk_metadata, mla_stream_t stream) {
    if (batch < 0 || total_q < 0 || h_k < 1 || h_q < 1 || h_q % h_k || num_parts < 1)
        return report_error(MLA_ERR_ARG, "mla_chunk_get_metadata: bad argument");
    if (!chunk_metadata || (batch > 0 && (!cu_seqlens_q || !cache_seqlens)))
        return report_error(MLA_ERR_ARG, "mla_chunk_get_metadata: NULL pointer");
    if (batch > kMaxChunkBatch) return report_errorf(MLA_ERR_UNSUPPORTED, "batch %d > %d", batch, kMaxChunkBatch);
    if (num_parts > kMaxChunkParts) return report_errorf(MLA_ERR_UNSUPPORTED, "num_parts %d > %d", num_parts, kMaxChunkParts);
    if ((int64_t)total_q * h_q > 0x7fffffffll - 1024)
        return report_error(MLA_ERR_UNSUPPORTED, "total_q * h_q exceeds 2^31 - 1025");
    DeviceInfo di;
    int st = device_info(&di);
    if (st != MLA_OK) return st;
    const size_t smem = chunk_metadata_smem_bytes(batch);
    cudaError_t e = cudaFuncSetAttribute(mla_chunk_metadata_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)chunk_metadata_smem_bytes(kMaxChunkBatch));
    if (e != cudaSuccess) return report_cuda(e, "cudaFuncSetAttribute(chunk metadata)");
    mla_chunk_metadata_kernel<<<1, chunk_metadata_threads(), smem, reinterpret_cast<cudaStream_t>(stream)>>>(
        cu_seqlens_q, cache_seqlens, batch, total_q, h_k, h_q / h_k, causal ? 1 : 0, num_parts, chunk_metadata);
    e = cudaGetLastError();
    return e == cudaSuccess ? MLA_OK : report_cuda(e, "chunk metadata launch");
}

int mla_chunk_workspace_size(const mla_chunk_shape_t *shape, size_t *bytes) {
    if (!bytes) return report_error(MLA_ERR_ARG, "bytes is NULL");
    int st = check_chunk_shape(shape);
    if (st != MLA_OK) return st;
    *bytes = chunk_workspace(shape->num_parts, nullptr);
    return MLA_OK;
}

int mla_chunk_fwd(const mla_chunk_shape_t *shape, const void *q, const void *k_cache, const int32_t *block_table,
                  const int32_t *cu_seqlens_q, const int32_t *cache_seqlens, const int32_t *chunk_metadata,
                  float softmax_scale, int causal, void *out, float *softmax_lse, void *workspace,
                  size_t workspace_bytes, mla_stream_t stream) {
    int st = check_chunk_shape(shape);
    if (st != MLA_OK) return st;
    return chunk_run(shape, concat_rows(shape, q, k_cache, 2), block_table, cu_seqlens_q, cache_seqlens, chunk_metadata,
                     default_scale(softmax_scale), 1.0f, causal, out, softmax_lse, workspace, workspace_bytes, stream);
}

int mla_chunk_fwd_split(const mla_chunk_shape_t *shape, const mla_chunk_rope_strides_t *rope, const void *q_nope,
                        const void *q_rope, const void *ctkv, const void *krope, const int32_t *block_table,
                        const int32_t *cu_seqlens_q, const int32_t *cache_seqlens, const int32_t *chunk_metadata,
                        float softmax_scale, int causal, void *out, float *softmax_lse, void *workspace,
                        size_t workspace_bytes, mla_stream_t stream) {
    int st = check_chunk_shape(shape);
    if (st != MLA_OK) return st;
    if (!rope) return report_error(MLA_ERR_ARG, "rope strides are NULL");
    ChunkSource c;
    c.split = true;
    c.q = q_nope;
    c.q_rope = q_rope;
    c.latent = ctkv;
    c.rope = krope;
    for (int i = 0; i < 2; ++i) {
        if (rope->q_rope_stride[i] <= 0 || rope->q_rope_stride[i] % 8)
            return report_error(MLA_ERR_ARG, "rope strides must be positive multiples of 8 elements");
        c.q_s[i] = shape->q_stride[i];
        c.qr_s[i] = rope->q_rope_stride[i];
    }
    for (int i = 0; i < 3; ++i) {
        if (rope->krope_stride[i] <= 0 || rope->krope_stride[i] % 8)
            return report_error(MLA_ERR_ARG, "rope strides must be positive multiples of 8 elements");
        c.l_s[i] = shape->k_stride[i];
        c.r_s[i] = rope->krope_stride[i];
    }
    return chunk_run(shape, c, block_table, cu_seqlens_q, cache_seqlens, chunk_metadata, default_scale(softmax_scale),
                     1.0f, causal, out, softmax_lse, workspace, workspace_bytes, stream);
}

int mla_chunk_fwd_fp8(const mla_chunk_shape_t *shape, const void *q, const void *k_cache, const int32_t *block_table,
                      const int32_t *cu_seqlens_q, const int32_t *cache_seqlens, const int32_t *chunk_metadata,
                      float bmm1_scale, float bmm2_scale, int causal, void *out, float *softmax_lse, void *workspace,
                      size_t workspace_bytes, mla_stream_t stream) {
    int st = check_chunk_shape(shape);
    if (st != MLA_OK) return st;
    if (!(bmm1_scale > 0.f) || !std::isfinite(bmm1_scale) || !std::isfinite(bmm2_scale))
        return report_error(MLA_ERR_ARG, "bmm1_scale must be positive and finite, bmm2_scale finite");
    for (int i = 0; i < 3; ++i)
        if ((i < 2 && shape->q_stride[i] % 16) || shape->k_stride[i] % 16)
            return report_error(MLA_ERR_ARG, "e4m3 q and k_cache strides must be multiples of 16 elements");
    return chunk_run(shape, concat_rows(shape, q, k_cache, 1), block_table, cu_seqlens_q, cache_seqlens, chunk_metadata,
                     bmm1_scale, bmm2_scale, causal, out, softmax_lse, workspace, workspace_bytes, stream);
}

}  // extern "C"
