// rope.cu -- rotary positions (mla_rope_init, mla_rope).
//
//   (a, b) -> (a c - b s, b c + a s),  c, s = factor * cos, sin(position * frequency_i)
//
// over the pairs of `rotary_dim` dims of every head, neighbours (2i, 2i + 1)
// or halves (i, i + rotary_dim / 2).  The inverse turns the other way; it is
// also the gradient, since the rotation is linear and its transpose is the
// rotation by the opposite angle (times the same factor).
//
// Bound by memory (3 FMAs per element), and at small sizes by the launch.  A
// block takes a run of (token, head) rows, computes the angles of the tokens it
// touches once into shared memory, where all heads of a token share them, and
// moves 16 bytes per load.  A thread keeps its chunk of the row and takes several
// rows at a time (32 to 64 bytes in flight), whose loads are issued ahead of the angles;
// addresses advance by additions.  Measured: 8191 x 20 rows of 128 fp32 values
// 27 us (6.1 TB/s; a plain copy of as many bytes takes 28), 2051 x 16 rows of 576
// bf16 values into e4m3 10.9 us (5.2 TB/s), the 64 rotary dims of 4096 x 128 rows
// between two wider tensors 24.8 us (5.4 TB/s), a decode step's 64 x 128 rows 2.8 us.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "api_internal.h"
#include "rope.cuh"
#include "sm103.cuh"

namespace mla {
namespace {

struct RopeParams {
    const void *x;
    void *out;
    const int32_t *positions;
    int64_t x_s[3], o_s[3];      // elements: batch, token, head
    uint32_t rows, tokens, heads;   // rows = batch * tokens * heads; tokens per batch entry
    int32_t off, dim;            // first rotated dim, dims of a head
    int32_t pairs;
    int32_t copy;                // also copy the dims that are not rotated
    int32_t rows_per_block;
    // blockDim.y rows on: as tokens and heads, and as elements, to which the others add when the
    // heads run over into the next token, and the tokens into the next batch entry
    uint32_t step_tokens, step_heads;
    int64_t x_step, o_step, x_token, o_token, x_batch, o_batch;
    float out_scale, factor;     // factor carries the plan's; sin_sign the direction
    float sin_sign;
    uint64_t turns[MLA_ROPE_MAX_PAIRS];
};

constexpr int kRows = 4;   // rows of a thread, of one 16-byte load each

template <typename T> __device__ __forceinline__ T from_float(float x);
template <> __device__ __forceinline__ float from_float<float>(float x) { return x; }
template <> __device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

struct E4m3 { uint8_t v; };
template <> __device__ __forceinline__ E4m3 from_float<E4m3>(float x) {
    return E4m3{(uint8_t)pack_e4m3x4(x, 0.f, 0.f, 0.f)};
}

// V consecutive elements, and the way back from floats: 16-byte accesses for V >= 4, single elements
// otherwise.
template <typename T, int V>
struct alignas(V >= 4 ? 16 : sizeof(T)) Chunk {
    T e[V];
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (V >= 4) {
#pragma unroll
            for (int i = 0; i < V * (int)sizeof(T) / 16; ++i)
                reinterpret_cast<uint4 *>(e)[i] = reinterpret_cast<const uint4 *>(p)[i];
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) e[i] = p[i];
        }
    }
    __device__ __forceinline__ float operator[](int i) const { return to_float(e[i]); }
};
template <typename T, int V>
__device__ __forceinline__ void store_vec(T *p, const float (&v)[V], float scale) {
    alignas(16) T e[V];
    if constexpr (sizeof(T) == 1 && V >= 4) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i)
            reinterpret_cast<uint32_t *>(e)[i] = pack_e4m3x4(v[4 * i] * scale, v[4 * i + 1] * scale, v[4 * i + 2] * scale, v[4 * i + 3] * scale);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) e[i] = from_float<T>(sizeof(T) == 1 ? v[i] * scale : v[i]);
    }
    if constexpr (V * sizeof(T) == 16) *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(e);
    else if constexpr (V >= 4 && V * sizeof(T) == 4) *reinterpret_cast<uint32_t *>(p) = *reinterpret_cast<const uint32_t *>(e);
    else {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = e[i];
    }
}

// Elements of a chunk on the wide path: 16 bytes, or 16 16-bit values that become 16 bytes of e4m3 (with 8,
// the address arithmetic of the kernel took more time than its memory traffic).
template <typename TI, typename TO>
__host__ __device__ constexpr int wide_chunk() {
    return sizeof(TO) == 1 && sizeof(TI) == 2 ? 16 : 16 / (int)sizeof(TI);
}

// Blocks an SM: a block waits once for its loads and once for its angles, so several have to be there.  With a row's
// two halves of 16 bytes in flight a thread, six fit; with two rows (and four blocks) 4096 x 128 rows of 64
// bf16 values took 26.4 us instead of 24.8.
template <typename TI, typename TO, bool HALVES>
__host__ __device__ constexpr int blocks_per_sm() {
    return HALVES && wide_chunk<TI, TO>() * sizeof(TI) == 16 ? 6 : 4;
}

// WIDE: whole chunks; otherwise element accesses (rows of any alignment).
template <typename TI, typename TO, bool HALVES, bool WIDE>
__global__ void __launch_bounds__(256, (blocks_per_sm<TI, TO, HALVES>())) mla_rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int V = WIDE ? wide_chunk<TI, TO>() : (HALVES ? 1 : 2);
    // rows of a thread in flight: 64 bytes for pairs of neighbours, one row for halves
    constexpr int R = HALVES ? 1 : kRows / (V * sizeof(TI) > 16 ? 2 : 1);
    extern __shared__ float2 cs[];   // [tokens of the block][pairs]
    const uint32_t row0 = blockIdx.x * (uint32_t)p.rows_per_block;
    const uint32_t row_end = min(row0 + (uint32_t)p.rows_per_block, p.rows);
    const uint32_t tok0 = row0 / p.heads, ntok = (row_end - 1) / p.heads - tok0 + 1;
    // chunks of a row: the rotated ones first (HALVES: V pairs, two runs of V elements;
    // else V / 2 pairs, one run), then the dims before and behind them
    const int rot_chunks = HALVES ? p.pairs / V : 2 * p.pairs / V;
    const int pre = p.copy ? (p.off + V - 1) / V : 0;
    const int post_at = p.off + 2 * p.pairs;
    const int chunks = rot_chunks + pre + (p.copy ? (p.dim - post_at + V - 1) / V : 0);

    int c = threadIdx.x, d0 = 0, end = 0;   // the thread's chunk; its first dim, and where its run of dims ends
    bool rot = false;
    uint32_t row = row_end, tok = 0, h = 0, b_end = 0;   // b_end: tokens up to the batch entry's end
    const TI *src = nullptr;
    TO *dst = nullptr;
    Chunk<TI, V> x[R], y[R];                // y: the partners of halves
    TO *at[R];
    uint32_t angle[R];
    int n = 0;
    const auto first_row = [&]() {
        rot = c < rot_chunks;
        const bool front = c < rot_chunks + pre;
        d0 = rot ? p.off + c * V : front ? (c - rot_chunks) * V : post_at + (c - rot_chunks - pre) * V;
        end = rot ? post_at : front ? p.off : p.dim;
        row = row0 + threadIdx.y;
        tok = row / p.heads;
        h = row - tok * p.heads;
        const uint32_t b = tok / p.tokens, i = tok - b * p.tokens;
        b_end = (b + 1) * p.tokens;
        src = static_cast<const TI *>(p.x) + (int64_t)b * p.x_s[0] + (int64_t)i * p.x_s[1] + (int64_t)h * p.x_s[2] + d0;
        dst = static_cast<TO *>(p.out) + (int64_t)b * p.o_s[0] + (int64_t)i * p.o_s[1] + (int64_t)h * p.o_s[2] + d0;
    };
    const auto load_rows = [&]() {
        n = 0;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if (row < row_end) {
                at[k] = dst;
                angle[k] = (tok - tok0) * (uint32_t)p.pairs + (uint32_t)(HALVES ? c * V : c * V / 2);
                if (d0 + V <= end) {
                    x[k].load(src);
                    if (HALVES && rot) y[k].load(src + p.pairs);
                } else {
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        if (d0 + j < end) x[k].e[j] = src[j];
                }
                n = k + 1;
            }
            row += blockDim.y;
            tok += p.step_tokens;
            h += p.step_heads;
            src += p.x_step;
            dst += p.o_step;
            if (h >= p.heads) {
                h -= p.heads;
                ++tok;
                src += p.x_token;
                dst += p.o_token;
            }
            while (tok >= b_end) {
                b_end += p.tokens;
                src += p.x_batch;
                dst += p.o_batch;
            }
        }
    };
    if (c < chunks) {
        first_row();
        load_rows();
    }
    // the angles, while those loads are on their way
    const int tid = threadIdx.y * blockDim.x + threadIdx.x, nthr = blockDim.x * blockDim.y;
    for (uint32_t i = tid; i < ntok * (uint32_t)p.pairs; i += nthr) {
        const uint32_t t = i / (uint32_t)p.pairs, k = i - t * (uint32_t)p.pairs;
        float2 v = rope_cos_sin(p.turns[k], __ldg(p.positions + tok0 + t), p.factor);
        v.y *= p.sin_sign;
        cs[i] = v;
    }
    __syncthreads();
    while (c < chunks) {
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if (k >= n) break;
            TO *o = at[k];
            float r[V];
            if (!rot) {
#pragma unroll
                for (int j = 0; j < V; ++j) r[j] = x[k][j];
                if (d0 + V <= end) {
                    store_vec<TO, V>(o, r, p.out_scale);
                } else {
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        if (d0 + j < end) {
                            const float one[1] = {r[j]};
                            store_vec<TO, 1>(o + j, one, p.out_scale);
                        }
                }
            } else if constexpr (HALVES) {
                float q[V];
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float2 t = cs[angle[k] + j];
                    r[j] = x[k][j] * t.x - y[k][j] * t.y;
                    q[j] = y[k][j] * t.x + x[k][j] * t.y;
                }
                store_vec<TO, V>(o, r, p.out_scale);
                store_vec<TO, V>(o + p.pairs, q, p.out_scale);
            } else {
#pragma unroll
                for (int j = 0; j < V / 2; ++j) {
                    const float2 t = cs[angle[k] + j];
                    r[2 * j] = x[k][2 * j] * t.x - x[k][2 * j + 1] * t.y;
                    r[2 * j + 1] = x[k][2 * j + 1] * t.x + x[k][2 * j] * t.y;
                }
                store_vec<TO, V>(o, r, p.out_scale);
            }
        }
        if (row >= row_end) {
            c += blockDim.x;
            if (c >= chunks) break;
            first_row();
        }
        load_rows();
    }
}

constexpr uint32_t kMaxAngles = 4096;   // entries of a block's angle table (32 KB)

template <typename TI, typename TO>
int launch(const RopeParams &p, bool halves, bool wide, dim3 grid, dim3 block, size_t smem, cudaStream_t s) {
    if (halves) {
        if (wide) mla_rope_kernel<TI, TO, true, true><<<grid, block, smem, s>>>(p);
        else mla_rope_kernel<TI, TO, true, false><<<grid, block, smem, s>>>(p);
    } else {
        if (wide) mla_rope_kernel<TI, TO, false, true><<<grid, block, smem, s>>>(p);
        else mla_rope_kernel<TI, TO, false, false><<<grid, block, smem, s>>>(p);
    }
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? MLA_OK : report_cuda(e, "rotary launch");
}

template <typename TI>
int launch_out(const RopeParams &p, bool e4m3, bool halves, bool wide, dim3 grid, dim3 block, size_t smem, cudaStream_t s) {
    return e4m3 ? launch<TI, E4m3>(p, halves, wide, grid, block, smem, s)
                : launch<TI, TI>(p, halves, wide, grid, block, smem, s);
}

int dtype_bytes(int t) {
    return t == MLA_DTYPE_F32 ? 4 : t == MLA_DTYPE_BF16 || t == MLA_DTYPE_F16 ? 2 : t == MLA_DTYPE_E4M3 ? 1 : 0;
}

}  // namespace

int check_rope_plan(const mla_rope_plan_t *plan) {
    if (!plan) return report_error(MLA_ERR_ARG, "rotary plan is NULL");
    if (plan->rotary_dim < 2 || plan->rotary_dim > 2 * MLA_ROPE_MAX_PAIRS || plan->rotary_dim % 2 ||
        (plan->interleaved != 0 && plan->interleaved != 1) || !std::isfinite(plan->factor))
        return report_error(MLA_ERR_ARG, "rotary plan not set up by mla_rope_init");
    return MLA_OK;
}

}  // namespace mla

using namespace mla;

extern "C" {

int mla_rope_init(mla_rope_plan_t *plan, int rotary_dim, int interleaved, double theta,
                  const mla_rope_scaling_t *scaling) {
    if (!plan) return report_error(MLA_ERR_ARG, "rotary plan is NULL");
    if (rotary_dim < 2 || rotary_dim > 2 * MLA_ROPE_MAX_PAIRS || rotary_dim % 2)
        return report_errorf(MLA_ERR_ARG, "rotary_dim must be even and in [2, %d] (got %d)", 2 * MLA_ROPE_MAX_PAIRS,
                             rotary_dim);
    if (!(theta >= 1.0) || !std::isfinite(theta)) return report_error(MLA_ERR_ARG, "theta must be finite and >= 1");
    const int kind = scaling ? scaling->kind : MLA_ROPE_PLAIN;
    if (kind != MLA_ROPE_PLAIN && kind != MLA_ROPE_LINEAR && kind != MLA_ROPE_YARN)
        return report_errorf(MLA_ERR_ARG, "unknown rotary scaling %d", kind);
    if (kind != MLA_ROPE_PLAIN && (!(scaling->factor >= 1.0) || !std::isfinite(scaling->factor)))
        return report_error(MLA_ERR_ARG, "rotary scaling factor must be finite and >= 1");
    double lo = 0, hi = 0, factor = 1.0;
    const double pi = 3.14159265358979323846;
    if (kind == MLA_ROPE_YARN) {
        if (!(scaling->original_max_position >= 1.0) || !std::isfinite(scaling->original_max_position) ||
            !(scaling->beta_slow > 0.0) || !(scaling->beta_fast >= scaling->beta_slow) ||
            !std::isfinite(scaling->beta_fast) || !std::isfinite(scaling->mscale) ||
            !std::isfinite(scaling->mscale_all_dim) || !(theta > 1.0))
            return report_error(MLA_ERR_ARG, "yarn needs theta > 1, original_max_position >= 1, beta_fast >= beta_slow > 0 "
                                             "and finite mscale values");
        // the pair whose wavelength fits `turns` times into the original context
        auto pair_of = [&](double turns) {
            return rotary_dim * std::log(scaling->original_max_position / (turns * 2.0 * pi)) / (2.0 * std::log(theta));
        };
        lo = std::fmax(std::floor(pair_of(scaling->beta_fast)), 0.0);
        hi = std::fmin(std::ceil(pair_of(scaling->beta_slow)), rotary_dim - 1.0);
        const double lf = 0.1 * std::log(scaling->factor);
        factor = (lf * scaling->mscale + 1.0) / (lf * scaling->mscale_all_dim + 1.0);
        if (!std::isfinite(factor)) return report_error(MLA_ERR_ARG, "yarn: mscale_all_dim gives no finite factor");
    }
    plan->rotary_dim = rotary_dim;
    plan->interleaved = interleaved ? 1 : 0;
    plan->factor = (float)factor;
    plan->reserved = 0;
    for (int i = 0; i < MLA_ROPE_MAX_PAIRS; ++i) plan->turns[i] = 0;
    for (int i = 0; i < rotary_dim / 2; ++i) {
        double f = std::pow(theta, -2.0 * i / rotary_dim);
        if (kind == MLA_ROPE_LINEAR) f /= scaling->factor;
        if (kind == MLA_ROPE_YARN) {
            const double ramp = std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 1e-3), 0.0), 1.0);
            f = f * (1.0 - ramp) + f / scaling->factor * ramp;
        }
        // f <= 1 radian a position: below a sixth of a turn, so the fraction fits
        plan->turns[i] = (uint64_t)std::llrint(std::ldexp(f / (2.0 * pi), 63)) * 2u;
    }
    return MLA_OK;
}

int mla_rope(const mla_rope_plan_t *plan, const mla_rope_shape_t *shape, const void *x, const int32_t *positions,
             int inverse, void *out, float out_scale, mla_stream_t stream) {
    int st = check_rope_plan(plan);
    if (st != MLA_OK) return st;
    if (!shape) return report_error(MLA_ERR_ARG, "shape is NULL");
    const mla_rope_shape_t &sh = *shape;
    if (sh.batch < 0 || sh.tokens < 0 || sh.heads < 1 || sh.head_dim < 1)
        return report_error(MLA_ERR_ARG, "batch and tokens must be >= 0, heads and head_dim >= 1");
    if (sh.rope_offset < 0 || (int64_t)sh.rope_offset + plan->rotary_dim > sh.head_dim)
        return report_errorf(MLA_ERR_ARG, "rotated dims [%d, %d + %d) outside head_dim %d", sh.rope_offset, sh.rope_offset,
                             plan->rotary_dim, sh.head_dim);
    const int bi = dtype_bytes(sh.dtype), bo = dtype_bytes(sh.out_dtype);
    if ((sh.dtype != MLA_DTYPE_BF16 && sh.dtype != MLA_DTYPE_F16 && sh.dtype != MLA_DTYPE_F32) ||
        (sh.out_dtype != sh.dtype && sh.out_dtype != MLA_DTYPE_E4M3))
        return report_error(MLA_ERR_ARG, "dtype must be bf16, fp16 or fp32, out_dtype the same or e4m3");
    const bool e4m3 = sh.out_dtype == MLA_DTYPE_E4M3;
    if (!std::isfinite(out_scale) || (!e4m3 && out_scale != 1.0f))
        return report_error(MLA_ERR_ARG, "out_scale must be finite, and 1 unless out_dtype is e4m3");
    for (int i = 0; i < 3; ++i)
        if (sh.x_stride[i] < 0 || sh.out_stride[i] < 0) return report_error(MLA_ERR_ARG, "negative stride");
    const int64_t rows = (int64_t)sh.batch * sh.tokens * sh.heads;
    if (rows > 0x7fffffffll - 1024) return report_error(MLA_ERR_UNSUPPORTED, "batch * tokens * heads exceeds 2^31 - 1025");
    if (rows == 0) return MLA_OK;
    if (!x || !out || !positions) return report_error(MLA_ERR_ARG, "NULL tensor pointer");
    const int64_t n[3] = {sh.batch, sh.tokens, sh.heads};
    const bool in_place = x == out;
    // What different threads write must lie apart: whole rows, or in place their rotated dims.
    if (!rows_apart(n, sh.out_stride, 3, in_place ? plan->rotary_dim : sh.head_dim))
        return report_error(MLA_ERR_ARG, "out rows overlap (a stride smaller than what the others span)");
    if (!is_aligned(x, bi) || !is_aligned(out, bo) || !is_aligned(positions, 4))
        return report_error(MLA_ERR_ARG, "pointer not aligned to its element");
    if (in_place) {
        bool same = !e4m3;
        for (int i = 0; i < 3; ++i) same = same && (n[i] == 1 || sh.x_stride[i] == sh.out_stride[i]);
        if (!same) return report_error(MLA_ERR_ARG, "in place needs out's type and strides to be x's");
    }
    DeviceInfo di;
    if ((st = device_info(&di)) != MLA_OK) return st;

    RopeParams p;
    p.x = x;
    p.out = out;
    p.positions = positions;
    const int pairs = plan->rotary_dim / 2, v = e4m3 && bi == 2 ? 16 : 16 / bi;
    bool wide = is_aligned(x, 16) && is_aligned(out, (uintptr_t)(v * bo)) && sh.rope_offset % v == 0 &&
                (plan->interleaved ? plan->rotary_dim % v == 0 : pairs % v == 0) && (in_place || sh.head_dim % v == 0);
    for (int i = 0; i < 3; ++i) {
        p.x_s[i] = sh.x_stride[i];
        p.o_s[i] = sh.out_stride[i];
        wide = wide && (n[i] == 1 || (sh.x_stride[i] % v == 0 && sh.out_stride[i] % v == 0));
    }
    // One run of tokens where the strides allow it (always with one token each): a step that crosses many
    // batch entries walks them one by one.
    int64_t tokens = sh.tokens;
    if (tokens == 1) {
        p.x_s[1] = p.x_s[0];
        p.o_s[1] = p.o_s[0];
        tokens = sh.batch;
    } else if (p.x_s[0] == tokens * p.x_s[1] && p.o_s[0] == tokens * p.o_s[1]) {
        tokens *= sh.batch;
    }
    p.rows = (uint32_t)rows;
    p.tokens = (uint32_t)tokens;
    p.heads = (uint32_t)sh.heads;
    p.off = sh.rope_offset;
    p.dim = sh.head_dim;
    p.pairs = pairs;
    p.copy = in_place ? 0 : 1;
    p.out_scale = out_scale;
    p.factor = plan->factor;
    p.sin_sign = inverse ? -1.f : 1.f;
    for (int i = 0; i < MLA_ROPE_MAX_PAIRS; ++i) p.turns[i] = plan->turns[i];

    const int vv = wide ? v : (plan->interleaved ? 2 : 1);
    const int chunks = (plan->interleaved ? 2 * pairs : pairs) / vv +
                       (p.copy ? (sh.rope_offset + vv - 1) / vv + (sh.head_dim - sh.rope_offset - 2 * pairs + vv - 1) / vv : 0);
    const int bx = chunks < 256 ? chunks : 256, by = 256 / bx;
    // four rows a thread when that still fills the GPU twice over, else one; a block's rows
    // may touch as many tokens as its angle table holds
    int64_t rpb = kRows * by;
    if (rows < 2ll * di.sm_count * rpb) rpb = by;
    const int64_t most = (int64_t)(kMaxAngles / pairs);
    if (sh.heads < most && rpb > (most - 1) * sh.heads) rpb = (most - 1) * sh.heads;
    p.rows_per_block = (int)rpb;
    p.step_tokens = (uint32_t)(by / sh.heads);
    p.step_heads = (uint32_t)(by % sh.heads);
    const int64_t *xs = p.x_s, *os = p.o_s;
    p.x_step = p.step_tokens * xs[1] + p.step_heads * xs[2];
    p.o_step = p.step_tokens * os[1] + p.step_heads * os[2];
    p.x_token = xs[1] - sh.heads * xs[2];
    p.o_token = os[1] - sh.heads * os[2];
    p.x_batch = xs[0] - tokens * xs[1];
    p.o_batch = os[0] - tokens * os[1];
    const int64_t ntok = (rpb + sh.heads - 2) / sh.heads + 1;
    const size_t smem = (size_t)ntok * pairs * sizeof(float2);
    const dim3 grid((unsigned)((rows + rpb - 1) / rpb)), block(bx, by);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool halves = !plan->interleaved;
    switch (sh.dtype) {
    case MLA_DTYPE_BF16: return launch_out<__nv_bfloat16>(p, e4m3, halves, wide, grid, block, smem, s);
    case MLA_DTYPE_F16: return launch_out<__half>(p, e4m3, halves, wide, grid, block, smem, s);
    default: return launch_out<float>(p, e4m3, halves, wide, grid, block, smem, s);
    }
}

}  // extern "C"
