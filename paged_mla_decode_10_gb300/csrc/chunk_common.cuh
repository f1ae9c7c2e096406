// chunk_common.cuh -- work units and schedule records of the chunk attention.
//
// The query rows of one (sequence, KV head) -- its n new tokens times the
// hpk = h_q / h_k heads, token by token -- are cut into blocks of 128 rows, the
// keys a block sees into tiles of 128.  A schedule record gives each part a
// contiguous run of (sequence, block, tile); a block that starts and ends
// inside one part is finished there, the pieces of any other leave fp32
// partials that the combine merges.
#pragma once

#include <cstdint>

#include "decode_common.cuh"

namespace mla {

constexpr int kTileKeys = 128;          // keys of a tile: two cache pages
constexpr int kTilePages = kTileKeys / kPage;
constexpr int kBlockRows = 128;         // query rows of a block
constexpr int kSlotsPerPart = 2;        // partials a part can leave: of its first and of its last block
// Fixed work of opening a block (query load, pipeline fill, output), in tiles: an estimate.  A change of block was
// measured since at 4 to 4.5 tiles' time in bf16 and 4.5 to 5.5 in e4m3; other values have not been timed.
constexpr int kBlockCost = 3;
// A part takes at least this much work, and a cut leaves at least kMinPiece tiles on either side:
// splitting a block costs a second block's fixed work and the partials' way through memory.
constexpr int kMinShare = 8, kMinPiece = 2;

struct ChunkParams {
    const int32_t *block_table;
    int64_t bt_stride;
    const int32_t *cu, *seqlens, *md;
    const void *q, *q_rope;          // latent and RoPE query dims (q_rope: q's dims 512.. when concatenated)
    int64_t q_s0, q_s1, qr_s0, qr_s1;   // token, head; elements
    uint16_t *out;                   // bf16 (total_q, h_q, 512)
    int64_t o_s0, o_s1;
    float *lse;                      // (total_q, h_q)
    float *ws_o, *ws_lse;            // partials: (slot, 128 rows, 512), (slot, 128 rows)
    int *err;
    int batch, total_q, h_q, h_k, hpk, num_blocks, max_blocks, num_parts, causal;
    int rope_x0;                     // first RoPE dim in the RoPE tensor map (512 on a concatenated cache, else 0)
    float scale_log2, out_scale;
    uint32_t hpk_mul, hpk_shift;     // ceil(2^hpk_shift / hpk), hpk_shift = 31 + ceil(log2 hpk)

    // row / hpk, exact for 0 <= row < 2^31: the multiplier is less than hpk <= 2^(hpk_shift - 31) above the
    // quotient times hpk, so the product is off by less than 2^hpk_shift in units of hpk
    __device__ __forceinline__ int token_of(int row) const {
        return (int)(((uint64_t)(uint32_t)row * hpk_mul) >> hpk_shift);
    }
};

__host__ __device__ constexpr int tiles_of(int keys) { return (keys + kTileKeys - 1) / kTileKeys; }
// Last row of block rb; below 2^31, as total_q * h_q <= 2^31 - 1025.
__host__ __device__ constexpr int last_row(int rb) { return rb * kBlockRows + (kBlockRows - 1); }

// One sequence's share of the batch.
struct ChunkSeq {
    int first, n, L;      // first query token, query tokens, cache length with them
    int row_blocks;       // 128-row blocks per KV head

    // Reads sequence b's lengths; offsets outside [0, total_q] are cut to it, so that a
    // wrong array never leads out of the query, and a length past the block table to its end.
    __device__ __forceinline__ void load(const int32_t *cu, const int32_t *seqlens, int b, int total_q, int hpk,
                                         int max_blocks, int *err) {
        int lo = __ldg(cu + b), hi = __ldg(cu + b + 1);
        lo = lo < 0 ? 0 : (lo > total_q ? total_q : lo);
        hi = hi < lo ? lo : (hi > total_q ? total_q : hi);
        first = lo;
        n = hi - lo;
        L = __ldg(seqlens + b);
        L = L < 0 ? 0 : L;
        if (L > max_blocks * (int64_t)kPage) {
            if (err) atomicOr(err, kErrBadBlock);
            L = max_blocks * kPage;
        }
        row_blocks = (int)(((int64_t)n * hpk + kBlockRows - 1) / kBlockRows);
    }
    // Keys that query token i sees (bottom-right alignment), clamped to [0, L].
    __device__ __forceinline__ int visible(int i, int causal) const {
        const int v = causal ? L - n + 1 + i : L;
        return v < 0 ? 0 : (v > L ? L : v);
    }
    // Keys that a block sees, whose last row belongs to token `last` (or past the end).
    __device__ __forceinline__ int block_keys(int last, int causal) const {
        return visible(last < n ? last : n - 1, causal);
    }
};

// A run of tiles of one block.
struct ChunkPiece {
    int b, hk, rb;        // sequence, KV head, row block
    int keys;             // keys that the block's last row sees
    int lo, hi, tiles;    // tiles [lo, hi) of the block's `tiles`
    int slot;             // partial slot, or -1 for a block that this piece finishes
    ChunkSeq seq;
};

// Walks a part's record; every role of a CTA runs its own copy and sees the same pieces.
// Any record sequence that runs from (0, 0, 0) to (batch, 0, 0) without gaps covers every
// block exactly once, whatever lengths it was computed for.
struct ChunkWalk {
    int b, j, b1, j1, t0, t1, part, max_seq_blocks;
    bool first;

    __device__ __forceinline__ void init(const int32_t *md, int p) {
        const int32_t *rec = md + (int64_t)p * kMdSize;
        b = rec[0]; j = rec[1]; t0 = rec[2];
        b1 = rec[3]; j1 = rec[4]; t1 = rec[5];
        if (b < 0) { b = 0; j = 0; t0 = 0; }
        if (j < 0) { j = 0; t0 = 0; }
        part = p;
        first = true;
    }
    __device__ __forceinline__ bool next(const ChunkParams &p, ChunkPiece &w) {
        while (b < p.batch && (b < b1 || (b == b1 && (j < j1 || (j == j1 && t1 > 0))))) {
            w.seq.load(p.cu, p.seqlens, b, p.total_q, p.hpk, p.max_blocks, p.err);
            if (j >= w.seq.row_blocks * p.h_k) {
                ++b;
                j = 0;
                first = false;
                continue;
            }
            w.b = b;
            w.hk = p.h_k > 1 ? j / w.seq.row_blocks : 0;
            w.rb = j - w.hk * w.seq.row_blocks;
            w.keys = w.seq.block_keys(p.token_of(last_row(w.rb)), p.causal);
            w.tiles = tiles_of(w.keys);
            w.lo = first && t0 > 0 ? t0 : 0;
            w.hi = (b == b1 && j == j1 && t1 < w.tiles) ? t1 : w.tiles;
            first = false;
            ++j;
            if (w.lo > 0 && w.lo >= w.hi) continue;   // the part before finished this block
            w.slot = w.lo > 0 ? kSlotsPerPart * part : (w.hi < w.tiles ? kSlotsPerPart * part + 1 : -1);
            return true;
        }
        return false;
    }
};

}  // namespace mla
