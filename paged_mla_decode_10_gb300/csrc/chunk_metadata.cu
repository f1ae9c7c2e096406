// chunk_metadata.cu -- the schedule of the chunk attention (mla_chunk_get_metadata).
//
// Cost of a block: its tiles plus kBlockCost.  The blocks of all sequences, in
// order, form one line of W cost units; part p takes the stretch
// [p S, (p + 1) S) with S = max(ceil(W / parts), kMinShare).  A cut inside a
// block is moved to the block's start or end when it would leave fewer than
// kMinPiece tiles on that side.  A cut depends on its position alone, so the
// end of one part is the start of the next, and part 0 starts at (0, 0, 0) and
// the last at (batch, 0, 0).
//
// The sum of a run of blocks is closed.  With B = L - n + 1 and h heads a KV
// head, block k < R - 1 sees B + floor((128 k + 127) / h) keys, so its tiles are
//   ceil(that / 128) = floor((k + beta) / h),  beta = floor((127 + (B + 127) h) / 128)
// (or 0 if that is negative), and sum_{i < x} floor(i / h) = h q (q - 1) / 2 + q r
// for x = q h + r.  The last block sees all L keys.
//
// One block of 1024 threads: a thread per sequence for its cost, a scan over the
// sequences, then a thread per cut, which finds its sequence and its block by
// bisection.  The call runs once per step, shared by all layers: 5 us for a few
// sequences, 9 us for one of 8192 new tokens at 128 heads, 14 us for 4096 sequences.
#include <cuda_runtime.h>

#include <cstdint>

#include "chunk_common.cuh"

namespace mla {

namespace {
constexpr int kThreads = 1024, kWarps = kThreads / 32;

// Costs of the blocks of one (sequence, KV head).
struct HeadCost {
    long long beta;
    int hpk, blocks, causal, all;   // all: tiles over every key

    __device__ __forceinline__ HeadCost(const ChunkSeq &s, int hpk_, int causal_)
        : hpk(hpk_), blocks(s.row_blocks), causal(causal_), all(tiles_of(s.L)) {
        const long long a = 127 + (long long)(s.L - s.n + 128) * hpk;
        beta = a >> 7;   // towards minus infinity
    }
    __device__ __forceinline__ long long quotients(long long x) const {   // sum of floor(i / hpk), i < x
        if (x <= 0) return 0;
        const long long q = x / hpk, r = x - q * hpk;
        return hpk * (q * (q - 1) / 2) + q * r;
    }
    // Cost of the blocks before block j < blocks.
    __device__ __forceinline__ long long before(int j) const {
        const long long tiles = causal ? quotients(j + beta) - quotients(beta) : (long long)j * all;
        return tiles + (long long)j * kBlockCost;
    }
    __device__ __forceinline__ long long total() const {
        return blocks > 0 ? before(blocks - 1) + all + kBlockCost : 0;
    }
};
}  // namespace

__global__ void __launch_bounds__(kThreads) mla_chunk_metadata_kernel(const int32_t *cu, const int32_t *seqlens, int batch,
                                                                      int total_q, int h_k, int hpk, int causal, int parts,
                                                                      int32_t *md) {
    extern __shared__ long long line[];   // [batch + 1]: cost before each sequence
    __shared__ long long warp_tot[kWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) line[0] = 0;
    // inclusive scan of the sequences' costs into line[1..batch], in runs of kThreads
    long long carry = 0;
    for (int base = 0; base < batch; base += kThreads) {
        const int i = base + tid;
        long long v = 0;
        if (i < batch) {
            ChunkSeq s;
            s.load(cu, seqlens, i, total_q, hpk, 1 << 24, nullptr);
            v = HeadCost(s, hpk, causal).total() * h_k;
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        if (lane == 31) warp_tot[warp] = v;
        __syncthreads();
        long long before = carry, all = 0;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += warp_tot[w];
            all += warp_tot[w];
        }
        if (i < batch) line[i + 1] = v + before;
        carry += all;
        __syncthreads();
    }
    const long long W = carry;   // not from shared memory: without a sequence no barrier has come since line[0] was set
    long long share = (W + parts - 1) / parts;
    if (share < kMinShare) share = kMinShare;
    // cut p lies between parts p - 1 and p
    for (int p = tid; p <= parts; p += kThreads) {
        int cb = batch, cj = 0, ct = 0;
        const long long g = (long long)p * share;
        if (p == 0) {
            cb = 0;
        } else if (p < parts && g < W) {
            int lo = 0, hi = batch - 1;   // the last sequence with line[b] <= g
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (line[mid] <= g) lo = mid;
                else hi = mid - 1;
            }
            ChunkSeq s;
            s.load(cu, seqlens, lo, total_q, hpk, 1 << 24, nullptr);
            const HeadCost head(s, hpk, causal);
            long long at = g - line[lo];
            const long long per_head = head.total();
            const int hk = (int)(at / per_head);
            at -= hk * per_head;
            int j = 0, last = s.row_blocks - 1;   // the last block with before(j) <= at
            while (j < last) {
                const int mid = (j + last + 1) >> 1;
                if (head.before(mid) <= at) j = mid;
                else last = mid - 1;
            }
            const int tiles = tiles_of(s.block_keys(last_row(j) / hpk, causal));
            const int cut = (int)(at - head.before(j)) - kBlockCost;   // tiles before the cut
            cb = lo;
            cj = hk * s.row_blocks + j;
            if (cut >= kMinPiece && tiles - cut >= kMinPiece) {
                ct = cut;
            } else if (cut >= kMinPiece && ++cj == s.row_blocks * h_k) {   // the next block, or sequence
                ++cb;
                cj = 0;
            }
        }
        if (p < parts) {
            md[p * kMdSize + 0] = cb; md[p * kMdSize + 1] = cj; md[p * kMdSize + 2] = ct;
            md[p * kMdSize + 6] = 0; md[p * kMdSize + 7] = 0;
        }
        if (p > 0) {
            md[(p - 1) * kMdSize + 3] = cb; md[(p - 1) * kMdSize + 4] = cj; md[(p - 1) * kMdSize + 5] = ct;
        }
    }
}

size_t chunk_metadata_smem_bytes(int batch) { return (size_t)(batch + 1) * sizeof(long long); }
uint32_t chunk_metadata_threads() { return kThreads; }

}  // namespace mla
