// append.cu -- new tokens into the paged latent cache (mla_cache_append).
//
// Token i of sequence b's n new ones sits at position L - n + i of the
// sequence (L: its length with them), i.e. in row (position % 64) of physical
// block block_table[b][position / 64].  The kernel writes its 512 latent dims
// as they are and its 64 rotary dims rotated by that position, rounded once to
// the cache's type (e4m3: after the factor kv_scale, saturating at 448).
//
// Bound by memory: 1152 bytes read and 1152 (e4m3: 576) written per row; for a
// decode step's few rows by the chain launch -> lengths -> block table -> store.
// A block takes a few consecutive rows.  Every thread asks for its values first; then
// the first warp finds the rows' sequences (a 32-way search of the offsets, two or
// three rounds) and slots, and the angles follow, while the values are on their way.
// Measured: 65536 rows into split bf16 caches 31 us (4.9 TB/s; a plain copy of as many
// bytes takes 26), 8192 rows of 13 sequences into e4m3 6.6 us, a decode step's 64 rows
// 3.9 us.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "api_internal.h"
#include "decode_common.cuh"
#include "rope.cuh"
#include "sm103.cuh"

namespace mla {

int check_rope_plan(const mla_rope_plan_t *plan);

namespace {

constexpr int kRope = kDqk - kDv;        // 64 rotary dims of a cache row
constexpr int kPairs = kRope / 2;
constexpr int kThreads = 288;            // 4 rows of 72 chunks of 8 values
constexpr int kRowsAtOnce = 4;
constexpr int kMaxRows = 16;             // rows of a block

struct AppendParams {
    const __nv_bfloat16 *latent, *k_rope;
    int64_t lat_s[2], rope_s[2];         // token, KV head
    const int32_t *block_table, *cu, *seqlens, *positions;
    int64_t bt_stride;
    void *cache, *krope_cache;           // krope_cache: dims 512.. of a row when the cache is concatenated
    int64_t c_s[3], kr_s[3];             // block, row, KV head
    int *err;
    int batch, tokens, h_k, num_blocks, max_blocks, per_seq, rows_per_block;
    float scale, factor;
    uint64_t turns[kPairs];
};

// Sequence of token t: the last b with cu[b] <= t.  Whole warp.
__device__ __forceinline__ int find_sequence(const int32_t *cu, int batch, int t, int lane) {
    int lo = 0, n = batch;   // the answer lies in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int at = lane * step;
        const bool le = at < n && (at == 0 || __ldg(cu + lo + at) <= t);
        const int k = 31 - __clz(__ballot_sync(0xffffffffu, le));
        lo += k * step;
        n = min(step, n - k * step);
    }
    return lo;
}

template <bool E4M3>
__device__ __forceinline__ void store8(uint8_t *row, int dim, const float (&v)[8]) {
    if constexpr (E4M3) {
        *reinterpret_cast<uint2 *>(row + dim) =
            make_uint2(pack_e4m3x4(v[0], v[1], v[2], v[3]), pack_e4m3x4(v[4], v[5], v[6], v[7]));
    } else {
        *reinterpret_cast<uint4 *>(row + 2 * dim) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                               pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    }
}

__device__ __forceinline__ void unpack8(const uint4 &w, float (&v)[8]) {
    const __nv_bfloat16 *e = reinterpret_cast<const __nv_bfloat16 *>(&w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __bfloat162float(e[i]);
}

template <bool E4M3, bool HALVES>
__global__ void __launch_bounds__(kThreads) mla_append_kernel(const __grid_constant__ AppendParams p) {
    __shared__ float2 cs[kMaxRows][kPairs];
    __shared__ int64_t slot[kMaxRows], rslot[kMaxRows];   // element offset of the row in its cache, < 0: not stored
    __shared__ int pos_of[kMaxRows];
    const int tid = threadIdx.x, lane = tid & 31;
    const int row0 = blockIdx.x * p.rows_per_block;       // row = token * h_k + KV head
    const int nrows = min(p.rows_per_block, p.tokens * p.h_k - row0);
    // this thread's 16-byte chunk (latent dims 8c, or rotary dims 8 (c - 64)) of up to four rows
    const int c = tid % 72, r0 = tid / 72;
    uint4 x[kMaxRows / kRowsAtOnce], y[HALVES ? kMaxRows / kRowsAtOnce : 1];   // y: the partners of halves
#pragma unroll
    for (int k = 0; k < kMaxRows / kRowsAtOnce; ++k) {
        const int r = r0 + k * kRowsAtOnce;
        if (r < nrows) {
            const int row = row0 + r, t = p.h_k > 1 ? row / p.h_k : row, hk = row - t * p.h_k;
            if (c < 64) {
                x[k] = __ldg(reinterpret_cast<const uint4 *>(p.latent + (int64_t)t * p.lat_s[0] + (int64_t)hk * p.lat_s[1] + 8 * c));
            } else {
                const uint4 *src = reinterpret_cast<const uint4 *>(p.k_rope + (int64_t)t * p.rope_s[0] + (int64_t)hk * p.rope_s[1]);
                x[k] = __ldg(src + (c - 64));
                if (HALVES) y[k] = __ldg(src + ((c - 64) ^ 4));
            }
        }
    }
    if (tid < 32) {
        int lo = 0, hi = 0;
        if (p.cu) {
            lo = find_sequence(p.cu, p.batch, row0 / p.h_k, lane);
            const int last = (row0 + nrows - 1) / p.h_k;
            hi = last != row0 / p.h_k ? find_sequence(p.cu, p.batch, last, lane) : lo;
        }
        if (lane < nrows) {
            const int t = (row0 + lane) / p.h_k, hk = (row0 + lane) - t * p.h_k;
            int b, first, n;
            bool in;
            if (p.cu) {
                while (lo < hi) {   // the last b in [lo, hi] with cu[b] <= t
                    const int mid = (lo + hi + 1) >> 1;
                    if (__ldg(p.cu + mid) <= t) lo = mid;
                    else hi = mid - 1;
                }
                b = lo;
                first = __ldg(p.cu + b);
                n = __ldg(p.cu + b + 1) - first;
                in = t >= first && t < first + n;   // tokens before the first or behind the last sequence are padding
            } else {
                b = t / p.per_seq;
                first = b * p.per_seq;
                n = p.per_seq;
                in = true;
            }
            int64_t at = -1, rat = -1;
            int pos = 0;
            if (in) {
                pos = __ldg(p.seqlens + b) - n + (t - first);
                const int blk = pos >> 6;
                if (pos < 0 || blk >= p.max_blocks) {
                    atomicOr(p.err, kErrBadBlock);
                } else {
                    const int phys = __ldg(p.block_table + (int64_t)b * p.bt_stride + blk);
                    if (phys < 0 || phys >= p.num_blocks) {
                        atomicOr(p.err, kErrBadBlock);
                    } else {
                        at = (int64_t)phys * p.c_s[0] + (int64_t)(pos & 63) * p.c_s[1] + (int64_t)hk * p.c_s[2];
                        rat = (int64_t)phys * p.kr_s[0] + (int64_t)(pos & 63) * p.kr_s[1] + (int64_t)hk * p.kr_s[2];
                    }
                }
                if (p.positions) pos = __ldg(p.positions + t);
            }
            slot[lane] = at;
            rslot[lane] = rat;
            pos_of[lane] = pos;
        }
    }
    __syncthreads();
    for (int i = tid; i < nrows * kPairs; i += kThreads)
        cs[i / kPairs][i % kPairs] = rope_cos_sin(p.turns[i % kPairs], pos_of[i / kPairs], p.factor);
    __syncthreads();
    constexpr int kEl = E4M3 ? 1 : 2;
#pragma unroll
    for (int k = 0; k < kMaxRows / kRowsAtOnce; ++k) {
        const int r = r0 + k * kRowsAtOnce;
        if (r >= nrows || slot[r] < 0) continue;
        if (c < 64) {
            uint8_t *row = static_cast<uint8_t *>(p.cache) + slot[r] * kEl;
            if constexpr (E4M3) {
                float v[8];
                unpack8(x[k], v);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] *= p.scale;
                store8<true>(row, 8 * c, v);
            } else {
                *reinterpret_cast<uint4 *>(row + 16 * c) = x[k];
            }
        } else {
            float v[8];
            unpack8(x[k], v);
            const int q = c - 64;   // dims [8q, 8q + 8)
            float o[8];
            if constexpr (HALVES) {
                float w[8];
                unpack8(y[k], w);
                const float sign = q < 4 ? -1.f : 1.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 a = cs[r][8 * (q & 3) + i];
                    o[i] = (v[i] * a.x + sign * (w[i] * a.y)) * p.scale;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 a = cs[r][4 * q + i];
                    o[2 * i] = (v[2 * i] * a.x - v[2 * i + 1] * a.y) * p.scale;
                    o[2 * i + 1] = (v[2 * i + 1] * a.x + v[2 * i] * a.y) * p.scale;
                }
            }
            store8<E4M3>(static_cast<uint8_t *>(p.krope_cache) + rslot[r] * kEl, 8 * q, o);
        }
    }
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" int mla_cache_append(const mla_append_shape_t *shape, const mla_rope_plan_t *plan, const void *latent,
                                const void *k_rope, const int32_t *block_table, const int32_t *cu_seqlens_q,
                                const int32_t *cache_seqlens, const int32_t *positions, void *k_cache,
                                void *krope_cache, float kv_scale, mla_stream_t stream) {
    if (!shape) return report_error(MLA_ERR_ARG, "shape is NULL");
    int st = check_rope_plan(plan);
    if (st != MLA_OK) return st;
    const mla_append_shape_t &sh = *shape;
    if (plan->rotary_dim != kRope) return report_errorf(MLA_ERR_ARG, "the cache's rotary part has 64 dims, the plan %d", plan->rotary_dim);
    if (sh.batch < 0 || sh.total_tokens < 0 || sh.h_k < 1 || sh.num_blocks < 1 || sh.max_blocks_per_seq < 1)
        return report_error(MLA_ERR_ARG, "batch and total_tokens must be >= 0; h_k, num_blocks, max_blocks_per_seq >= 1");
    if (sh.page_block_size != MLA_PAGE_BLOCK_SIZE)
        return report_errorf(MLA_ERR_ARG, "page_block_size must be 64 (got %d)", sh.page_block_size);
    if (sh.kv_dtype != MLA_DTYPE_BF16 && sh.kv_dtype != MLA_DTYPE_E4M3)
        return report_error(MLA_ERR_ARG, "kv_dtype must be bf16 or e4m3");
    const bool e4m3 = sh.kv_dtype == MLA_DTYPE_E4M3;
    if (!std::isfinite(kv_scale) || (!e4m3 && kv_scale != 1.0f))
        return report_error(MLA_ERR_ARG, "kv_scale must be finite, and 1 for a bf16 cache");
    if (sh.bt_stride < sh.max_blocks_per_seq) return report_error(MLA_ERR_ARG, "bt_stride < max_blocks_per_seq");
    const int64_t rows = (int64_t)sh.total_tokens * sh.h_k;
    if (rows > 0x7fffffffll - 64) return report_error(MLA_ERR_UNSUPPORTED, "total_tokens * h_k exceeds 2^31 - 65");
    if (rows > 0 && !cu_seqlens_q && (sh.batch == 0 || sh.total_tokens % sh.batch))
        return report_error(MLA_ERR_ARG, "without cu_seqlens_q, total_tokens must be a multiple of batch");
    if (rows == 0 || sh.batch == 0) return MLA_OK;   // nothing, or padding only
    if (!latent || !k_rope || !block_table || !cache_seqlens || !k_cache) return report_error(MLA_ERR_ARG, "NULL tensor pointer");
    for (int i = 0; i < 2; ++i)
        if (sh.latent_stride[i] <= 0 || sh.latent_stride[i] % 8 || sh.k_rope_stride[i] <= 0 || sh.k_rope_stride[i] % 8)
            return report_error(MLA_ERR_ARG, "strides must be positive multiples of 8 elements");
    const int64_t dims = krope_cache ? kDv : kDqk;
    for (int i = 0; i < 3; ++i) {
        if (sh.k_stride[i] <= 0 || sh.k_stride[i] % 8 || (krope_cache && (sh.krope_stride[i] <= 0 || sh.krope_stride[i] % 8)))
            return report_error(MLA_ERR_ARG, "strides must be positive multiples of 8 elements");
        // the cache's rows are written: they must not overlap
        if (sh.k_stride[i] < dims || (krope_cache && sh.krope_stride[i] < kRope))
            return report_error(MLA_ERR_ARG, "cache strides smaller than a row");
    }
    const int64_t n[3] = {sh.num_blocks, sh.page_block_size, sh.h_k};
    if (!rows_apart(n, sh.k_stride, 3, dims) || (krope_cache && !rows_apart(n, sh.krope_stride, 3, kRope)))
        return report_error(MLA_ERR_ARG, "cache rows overlap (a stride smaller than what the others span)");
    const uintptr_t out_align = e4m3 ? 8 : 16;
    if (!is_aligned(latent, 16) || !is_aligned(k_rope, 16) || !is_aligned(k_cache, out_align) ||
        (krope_cache && !is_aligned(krope_cache, out_align)))
        return report_errorf(MLA_ERR_ARG, "latent and k_rope must be 16-byte aligned, the caches %d-byte", (int)out_align);
    DeviceInfo di;
    if ((st = device_info(&di)) != MLA_OK) return st;
    AppendParams p;
    p.latent = static_cast<const __nv_bfloat16 *>(latent);
    p.k_rope = static_cast<const __nv_bfloat16 *>(k_rope);
    for (int i = 0; i < 2; ++i) {
        p.lat_s[i] = sh.latent_stride[i];
        p.rope_s[i] = sh.k_rope_stride[i];
    }
    p.block_table = block_table;
    p.cu = cu_seqlens_q;
    p.seqlens = cache_seqlens;
    p.positions = positions;
    p.bt_stride = sh.bt_stride;
    p.cache = k_cache;
    p.krope_cache = krope_cache ? krope_cache : static_cast<uint8_t *>(k_cache) + kDv * (e4m3 ? 1 : 2);
    for (int i = 0; i < 3; ++i) {
        p.c_s[i] = sh.k_stride[i];
        p.kr_s[i] = krope_cache ? sh.krope_stride[i] : sh.k_stride[i];
    }
    p.err = di.err_word;
    p.batch = sh.batch;
    p.tokens = sh.total_tokens;
    p.h_k = sh.h_k;
    p.num_blocks = sh.num_blocks;
    p.max_blocks = sh.max_blocks_per_seq;
    p.per_seq = cu_seqlens_q ? 0 : sh.total_tokens / sh.batch;
    p.scale = kv_scale;
    p.factor = plan->factor;
    for (int i = 0; i < kPairs; ++i) p.turns[i] = plan->turns[i];
    // four rows a block while that leaves SMs idle, sixteen for large calls
    p.rows_per_block = rows <= 4ll * di.sm_count * kRowsAtOnce ? kRowsAtOnce : kMaxRows;
    const unsigned grid = (unsigned)((rows + p.rows_per_block - 1) / p.rows_per_block);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (e4m3) {
        if (plan->interleaved) mla_append_kernel<true, false><<<grid, kThreads, 0, s>>>(p);
        else mla_append_kernel<true, true><<<grid, kThreads, 0, s>>>(p);
    } else {
        if (plan->interleaved) mla_append_kernel<false, false><<<grid, kThreads, 0, s>>>(p);
        else mla_append_kernel<false, true><<<grid, kThreads, 0, s>>>(p);
    }
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? MLA_OK : report_cuda(e, "append launch");
}
