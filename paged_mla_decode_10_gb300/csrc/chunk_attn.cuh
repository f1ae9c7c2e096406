// chunk_attn.cuh -- attention of ragged chunks of new tokens over the paged latent cache.
//
// Included twice, with MLA_CHUNK_F8 0 (bf16 query and cache) and 1 (e4m3).
//
// Work split.  A cluster of two CTAs takes the pieces of one schedule part: runs of 128-key tiles of
// a block of 128 query rows.  The output accumulator of a row is 512 fp32 dims, 2 KB, so a CTA's 256 KB
// of TMEM could hold that of 128 rows and nothing else.  The pair therefore runs tcgen05 with
// cta_group::2 at M = 128: each CTA owns 64 of the rows with all their dims (half its TMEM) and the
// tensor cores of both work on one product, each CTA keeping half of its B operand in shared memory:
//   S = Q K^T   N = 128 keys: CTA c holds the keys of page c of the tile, all 576 dims
//   O += P V    N = 2 x 256 dims: CTA c holds dims [256 h + 128 c, + 128), h = 0, 1, of both pages
// No logit crosses between the CTAs, and the softmax of a row is done once.  The two products want the
// cache rows cut in different ways, so V comes by copies of its own (from L2).
//
// In TMEM a row's accumulators lie in two lanes: lane r holds the first half of the N columns of row
// r, lane 64 + r the second.  Two warps share each quarter of the lanes, so four threads have 32 keys of
// a row each; they meet over the row's maximum in shared memory.  (With four warps instead of eight the
// softmax took 2700 cycles a tile on e4m3, more than its products.)
//
// One thread issues at most one MMA per 62 cycles, a QK^T step of N = 128 takes the pipe 32 and a PV
// step 64, and a wait behind MMAs of the same thread returns only once they are issued (all measured).
// So four threads issue: two take the QK^T of alternate tiles (and S buffers), two the halves h of PV.
//
// Per CTA:
//   TMEM  [0, 256) O (h = 0, 1: 128 columns each)   [256, 320) S0   [320, 384) S1   [384, 512) Q: its
//         first dims (bf16 256, e4m3 512), each row in both of its lanes
//   smem  the rest of Q | P | RoPE box of a K tile | ring of K units | ring of V units (16 KB each) | on
//         e4m3, where Q passes on its way to TMEM
//   warps 0-7   Q of a piece into TMEM and shared memory, softmax, epilogue: warp w has TMEM lanes
//               32 (w % 4) on, that is rows 32 (w % 2) on and key half (w % 4) / 2, and of these 64 keys
//               and of the output columns the half w / 4
//   warp  8     TMA producer of K     warp 9  TMA producer of V; TMEM allocation
//   warps 10, 11  QK^T issuers (CTA 0)  warps 12, 13  PV issuers (CTA 0)
//
// The issuing threads sit in CTA 0, so the "full" barriers of CTA 0 collect both CTAs' copies and
// arrivals, and completions are committed to both CTAs' barriers.
//
// Rows past the sequence's end may hold anything.  Their logits are masked; PV stops after the K step
// with the last visible key, and the V producer zeroes that step's rows past the end (0 * NaN).
//
// Every wait is bounded; a timeout sets MLA_DEVERR_TIMEOUT, drains copies and MMAs and returns.
//
// Bound by the tensor cores.  A bf16 tile is 2182 cycles of MMAs alone and takes 2470 to 2700; an e4m3 one
// 1740 (P's remainder is a second PV product) and about 2230; between two blocks of rows pass 10000 to
// 12000 cycles without products (last weights -> last PV -> next Q -> output -> first weights).  Tensor pipe
// active 74 % (bf16) and 75 % (e4m3) of 512 x 128 rows over 6k keys.  Measured with both launches, single calls between
// pauses: 1024 x 128 rows over 15k keys 2.45 to 2.5 ms (1760 to 1809 TFLOP/s; one after another 2.75 ms, 1610, as the
// power limit lowers the clock), 24 ragged sequences with 23 decoding 313 us (1300), 61 x 16 rows over 65k keys 117 us
// (1180; their keys come from HBM, 1.8 times, and tiles of the farther die take 10 % longer), e4m3 2 x 500 x 128 rows
// over up to 7.8k keys 457 to 465 us (2100; one after another 500, 1940), 17 x 16 rows over 300 keys 20 us.

namespace mla {
namespace MLA_CHUNK_NS {

#if MLA_CHUNK_F8
constexpr int kElem = 1;
constexpr int kKUnits = 2;        // K units of a tile: 64 keys x 256 dims
constexpr int kVUnits = 1;        // V units of a page: 64 keys x (128 + 128) dims
constexpr int kStepKeys = 32;     // keys of a PV step
constexpr int kQTmemDims = 512;
constexpr uint32_t kQBoxes = 0;   // whole latent Q boxes in shared memory
constexpr uint32_t kRopeRow = 64;
#else
constexpr int kElem = 2;
constexpr int kKUnits = 4;        // 64 keys x 128 dims
constexpr int kVUnits = 2;        // 64 keys x 128 dims, one for each h
constexpr int kStepKeys = 16;
constexpr int kQTmemDims = 256;
constexpr uint32_t kQBoxes = 4;
constexpr uint32_t kRopeRow = 128;
#endif
constexpr int kBoxDims = 128 / kElem;             // dims of a 128-byte box row
constexpr int kUnitDims = 2 * kBoxDims;           // dims of a K unit
constexpr int kStepsPerUnit = 8;                  // MMA K steps (32 bytes) of a K unit
constexpr int kRopeSteps = (int)kRopeRow / 32;
constexpr int kKStages = 5, kVStages = 4;
static_assert(kVStages % kVUnits == 0, "a V stage belongs to one PV thread");
constexpr uint32_t kUnitBytes = 16384;
constexpr uint32_t kRopeBytes = 64 * kRopeRow;
constexpr uint32_t OFF_Q = 0;                                    // Q boxes of 64 rows x 128 bytes
constexpr uint32_t OFF_QR = OFF_Q + kQBoxes * 8192u;             // Q RoPE box
constexpr uint32_t OFF_P = OFF_QR + 8192u;
constexpr uint32_t OFF_KR = OFF_P + 2 * 16384u;                      // RoPE box of a K tile
constexpr uint32_t OFF_K = OFF_KR + 8192u;
constexpr uint32_t OFF_V = OFF_K + kKStages * kUnitBytes;
// where Q's part for TMEM passes through: the P buffers, or (e4m3) 32 KB of its own
constexpr uint32_t OFF_QS = MLA_CHUNK_F8 ? OFF_V + kVStages * kUnitBytes : OFF_P;
constexpr uint32_t OFF_BAR = OFF_V + kVStages * kUnitBytes + (MLA_CHUNK_F8 ? 32768u : 0u);
constexpr uint32_t OFF_STAT = OFF_BAR + 64 * 8;                  // maxima [3][64], then denominators [4][64] of a row's threads
constexpr uint32_t OFF_MISC = OFF_STAT + 4 * 64 * 4;
constexpr uint32_t kSmemBytes = OFF_MISC + 64 + 1024;
static_assert(kSmemBytes <= 232448, "shared memory budget");
constexpr int kThreads = 448;
constexpr uint32_t TM_O = 0, TM_S = 256, TM_Q = 384;
#if MLA_CHUNK_F8
// P is held as two 8-bit floats, e4m3 and the e5m2 of what that leaves.  A row's maximum stands between 2^4.5 and
// 2^8.5 (e4m3 ends at 448).  A smaller headroom would hold smaller weights but raise the reference, and rescale O, on
// most tiles: with 2^7 and 2^8 (and a remainder taken in fp32) 686 us, so 559, on 2 x 500 x 128 over 7.8k keys.
//
// Weights from 2^-6 on are held to the nearest of 8 significant bits, 2^-8 of their binade.  Smaller ones have fewer
// (2^-14 is off at worst).  Against the row's large weights that is little for one key; but the many keys 7 nats or more
// below a few large ones may all round the same way, while the denominator sums them as they are: 65,000 equal ones 10
// nats down would lose 4 % of their mass, below 2^-17 all of it.  So what 8 bits leave of a remainder beyond e5m2's
// three is rounded up or down by thresholds that take every value equally often (dithering): the 32 keys of a thread have
// 32 thresholds evenly spread over the step, in bit-reversed order, and a byte that changes with the row and the thread's
// keys is XORed to all.  Each weight is then right in the mean, to 2^-8 or fp16's 2^-25, and the sum over many keys to a
// part of a step.  It costs 3 % (450 -> 462 us on 2 x 500 x 128 rows).  A remainder in e4m3 would end at 2^-10,
// 2^-14.5 of the largest weight: 40,000 keys 10.5 nats below one, half of the mass, came out as 0.
constexpr float kRescaleThreshold = 4.0f, kPExp = 4.5f;
#else
constexpr float kRescaleThreshold = 8.0f, kPExp = 0.0f;
#endif

// barriers; "0": used in CTA 0 alone, where both CTAs arrive; "c": committed to both CTAs
// (a wait tells a barrier's last two phases apart, so each waiting thread must see every phase: what two
// threads take in turn has a barrier for either)
constexpr int B_KFULL = 0;                        // 0, for even tiles, then for odd ones
constexpr int B_KEMPTY = B_KFULL + 2 * kKStages;  // c
constexpr int B_VFULL = B_KEMPTY + kKStages;      // 0
constexpr int B_VEMPTY = B_VFULL + kVStages;      // c
constexpr int B_RFULL = B_VEMPTY + kVStages;      // 0, for even tiles and for odd ones
constexpr int B_REMPTY = B_RFULL + 2;             // c
constexpr int B_SFULL = B_REMPTY + 1;             // c, two buffers
constexpr int B_SREAD = B_SFULL + 2;              // 0, two buffers: the softmax warps have read S
constexpr int B_PFULL = B_SREAD + 2;              // 0, two buffers
constexpr int B_PVDONE = B_PFULL + 2;             // c, tiles alternate over two
constexpr int B_OFREE = B_PVDONE + 2;             // 0: O has been read out
constexpr int B_QREADY = B_OFREE + 1;             // 0
constexpr int B_QFREE = B_QREADY + 1;             // c
constexpr int B_DRAIN = B_QFREE + 1;              // c: the QK^T thread's MMAs
constexpr int B_DRAINPV = B_DRAIN + 1;            // c: the PV thread's
constexpr int B_TAIL = B_DRAINPV + 1;             // a last page's V, before its rows past the end are zeroed
constexpr int B_PAIR = B_TAIL + 1;                // two: the four warps that hold the same rows
constexpr int B_ALL = B_PAIR + 2;                 // the eight softmax warps
constexpr int B_COUNT = B_ALL + 1;
static_assert(B_COUNT <= 64, "barrier area");

// Barrier `i` of CTA 0, as an address of the cluster's shared memory.
__device__ __forceinline__ uint32_t lead(const Ctx &c, int i) { return mapa_shared(bar_addr(c, i), 0); }

// After a timeout copies may still be on their way and no role counts them any more.  The roles that
// gave up had waited far longer than a copy takes; the few issued since land within microseconds, so
// ten milliseconds (at 2 GHz) before the CTAs leave are ample, and they end.
__device__ void drain_after_abort() {
    const long long t0 = clock64();
    while (clock64() - t0 < 20000000ll) {}
}

// Arrival on CTA 0's barrier for data that this CTA's threads left in this CTA's shared memory or TMEM
// and that this SM's tensor core reads: the threads' fences (proxy, tcgen05) order the data before it
// within the SM, so it releases at CTA scope.  That argues from the machine: the PTX memory model gives a release at
// CTA scope no effect on a thread of the other CTA, which issues the product.  At cluster scope each arrival held its
// warp up for 1350 cycles (311 -> 423 us on 24 ragged sequences, e4m3 463 -> 719 on 2 x 500 x 128 rows); by way of one
// warp of CTA 1 that passes its CTA's arrivals on at cluster scope they took 323 and 487.
__device__ __forceinline__ void mbar_arrive_lead(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" :: "r"(cluster_bar) : "memory");
}

// Walks a sequence's physical blocks, 32 table entries per coalesced load (whole warp).
struct PageTable {
    int base = -1, mine = 0;
    __device__ __forceinline__ int phys(const ChunkParams &p, int b, int page, int pages, bool fresh, int lane) {
        if (fresh || base < 0 || page < base || page >= base + 32) {
            base = page & ~31;
            mine = 0;
            if (base + lane < pages) {
                mine = __ldg(p.block_table + (int64_t)b * p.bt_stride + base + lane);
                if (mine < 0 || mine >= p.num_blocks) {
                    // only entries that are needed count
                    if (base + lane >= page) atomicOr(p.err, kErrBadBlock);
                    mine = 0;
                }
            }
        }
        return __shfl_sync(0xffffffffu, mine, page - base);
    }
};

// Query row `row` of a piece's (sequence, KV head): its latent or its RoPE dims.
__device__ __forceinline__ const uint8_t *q_row(const ChunkParams &p, const ChunkPiece &w, int row, bool rope) {
    const int i = p.token_of(row), h = w.hk * p.hpk + row - i * p.hpk;
    const int64_t t = w.seq.first + i;
    return rope ? static_cast<const uint8_t *>(p.q_rope) + (t * p.qr_s0 + (int64_t)h * p.qr_s1) * kElem
                : static_cast<const uint8_t *>(p.q) + (t * p.q_s0 + (int64_t)h * p.q_s1) * kElem;
}

// Asks L2 for this CTA's query rows of the piece after the one that `walk` gave last, so that their
// loads at the switch are short (whole warp).
__device__ __forceinline__ void prefetch_next_q(const ChunkParams &p, ChunkWalk walk, int cta, int lane) {
    ChunkPiece n;
    if (!walk.next(p, n) || n.lo >= n.hi) return;
    const int row0 = n.rb * kBlockRows + 64 * cta;
    for (int r = lane; r < 64 && (int64_t)row0 + r < (int64_t)n.seq.n * p.hpk; r += 32) {
        bulk_prefetch_l2(q_row(p, n, row0 + r, false), kDv * kElem);
        bulk_prefetch_l2(q_row(p, n, row0 + r, true), (kDqk - kDv) * kElem);
    }
}

// ----------------------------------------------------------------------------
// K producer: page `cta` of every tile, RoPE box first, then the latent units.
// ----------------------------------------------------------------------------
__device__ void k_producer(const Ctx &c, const ChunkParams &p, ChunkWalk walk, ChunkPiece w, bool have_piece, const CUtensorMap *km,
                           const CUtensorMap *kr, int cta, int lane, uint64_t policy) {
    PageTable pt;
    uint32_t it = 0, ku = 0, g = 0;   // tiles, units, blocks with products
    bool ok = true;
    for (; ok && have_piece; have_piece = walk.next(p, w)) {
        if (w.lo < w.hi) ++g;
        const int pages = (w.keys + kPage - 1) / kPage;   // that the block sees
        bool fresh = true;
        for (int t = w.lo; t < w.hi && ok; ++t, ++it) {
            const int page = kTilePages * t + cta;
            const bool have = page < pages;   // a tile's second page may not exist: its logits are masked
            int phys = 0;
            if (have) {
                phys = pt.phys(p, w.b, page, pages, fresh, lane);
                fresh = false;
            }
            if (lane == 0) {
                ok = wait_bar(c, bar_addr(c, B_REMPTY), (it & 1u) ^ 1u);
                if (ok) {
                    const uint32_t full = lead(c, B_RFULL + (it & 1u));
                    if (have) {
                        mbar_arrive_expect_tx_remote(full, kRopeBytes);
                        tma_load_4d_pair(c.base + OFF_KR, kr, full, p.rope_x0, w.hk, 0, phys, policy);
                    } else {
                        mbar_arrive_remote_relaxed(full);
                    }
                }
                for (int u = 0; u < kKUnits && ok; ++u) {
                    const uint32_t n = ku + (uint32_t)u, st = n % kKStages;
                    ok = wait_bar(c, bar_addr(c, B_KEMPTY + st), ((n / kKStages) & 1u) ^ 1u);
                    if (!ok) break;
                    const uint32_t full = lead(c, B_KFULL + (it & 1u) * kKStages + st), dst = c.base + OFF_K + st * kUnitBytes;
                    if (have) {
                        mbar_arrive_expect_tx_remote(full, kUnitBytes);
                        tma_load_4d_pair(dst, km, full, kUnitDims * u, w.hk, 0, phys, policy);
                        tma_load_4d_pair(dst + 8192u, km, full, kUnitDims * u + kBoxDims, w.hk, 0, phys, policy);
                    } else {
                        mbar_arrive_remote_relaxed(full);
                    }
                }
            }
            ku += kKUnits;
            ok = __shfl_sync(0xffffffffu, ok, 0);
        }
    }
    // every copy issued has been consumed, hence has landed, and every completion has come in before the CTA may exit
    if (lane == 0) {
        for (uint32_t n = ku > (uint32_t)kKStages ? ku - kKStages : 0u; n < ku && !*c.abort_flag; ++n)
            drain_bar(c, bar_addr(c, B_KEMPTY + n % kKStages), (n / kKStages) & 1u);
        if (it > 0 && !*c.abort_flag) drain_bar(c, bar_addr(c, B_REMPTY), (it - 1u) & 1u);
        if (g > 0 && !*c.abort_flag) drain_bar(c, bar_addr(c, B_QFREE), (g - 1u) & 1u);
    }
}

// ----------------------------------------------------------------------------
// V producer: this CTA's dims of both pages of every tile.
// ----------------------------------------------------------------------------
__device__ void v_producer(const Ctx &c, const ChunkParams &p, ChunkWalk walk, ChunkPiece w, bool have_piece, const CUtensorMap *km,
                           int cta, int lane, uint64_t policy) {
    PageTable pt;
    uint32_t vu = 0, tails = 0;
    bool ok = true;
    for (; ok && have_piece; have_piece = walk.next(p, w)) {
        prefetch_next_q(p, walk, cta, lane);
        const int pages = (w.keys + kPage - 1) / kPage;   // that the block sees
        bool fresh = true;
        for (int page = kTilePages * w.lo; page < min(kTilePages * w.hi, pages) && ok; ++page) {
            const int phys = pt.phys(p, w.b, page, pages, fresh, lane);
            fresh = false;
            // rows of the page's last PV step that lie past the sequence
            const int used = min(w.keys - page * kPage, kPage);
            const int z0 = max(w.seq.L - page * kPage, 0), z1 = (used + kStepKeys - 1) / kStepKeys * kStepKeys;
            for (int u = 0; u < kVUnits && ok; ++u, ++vu) {
                const uint32_t st = vu % kVStages, dst = c.base + OFF_V + st * kUnitBytes;
                const bool zero = z0 < z1;
                if (lane == 0) {
                    ok = wait_bar(c, bar_addr(c, B_VEMPTY + st), ((vu / kVStages) & 1u) ^ 1u);
                    if (ok) {
                        const uint32_t full = zero ? mapa_shared(bar_addr(c, B_TAIL), (uint32_t)cta) : lead(c, B_VFULL + st);
                        mbar_arrive_expect_tx_remote(full, kUnitBytes);
#if MLA_CHUNK_F8
                        tma_load_4d_pair(dst, km, full, 128 * cta, w.hk, 0, phys, policy);
                        tma_load_4d_pair(dst + 8192u, km, full, 256 + 128 * cta, w.hk, 0, phys, policy);
#else
                        tma_load_4d_pair(dst, km, full, 256 * u + 128 * cta, w.hk, 0, phys, policy);
                        tma_load_4d_pair(dst + 8192u, km, full, 256 * u + 128 * cta + 64, w.hk, 0, phys, policy);
#endif
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (ok && zero) {
                    // whole 128-byte box rows, so the swizzle does not matter
                    ok = __all_sync(0xffffffffu, wait_bar(c, bar_addr(c, B_TAIL), tails & 1u));
                    ++tails;
                    if (!ok) break;
                    uint8_t *g = reinterpret_cast<uint8_t *>(__cvta_shared_to_generic(dst));
                    const int n = (z1 - z0) * 16;
                    for (int i = lane; i < n; i += 32)
                        *reinterpret_cast<uint4 *>(g + ((i >> 3) & 1) * 8192 + (z0 + (i >> 4)) * 128 + (i & 7) * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_lead(lead(c, B_VFULL + st));
                }
            }
        }
    }
    if (lane == 0) {
        for (uint32_t n = vu > (uint32_t)kVStages ? vu - kVStages : 0u; n < vu && !*c.abort_flag; ++n)
            drain_bar(c, bar_addr(c, B_VEMPTY + n % kVStages), (n / kVStages) & 1u);
    }
}

// ----------------------------------------------------------------------------
// QK^T issuers (CTA 0): tiles alternate over two threads, each with an S buffer sb of its own.
// ----------------------------------------------------------------------------
__device__ void qk_role(const Ctx &c, const ChunkParams &p, ChunkWalk walk, ChunkPiece w, bool have_piece, uint32_t tmem, uint32_t sb,
                        int lane) {
    uint32_t it = 0, g = 0;
    uint32_t phases = 0;   // of this thread's barrier of each K stage
    bool ok = true;
#if MLA_CHUNK_F8
    constexpr uint32_t idS = make_idesc_e4m3(128, kTileKeys, false, false);
#else
    constexpr uint32_t idS = make_idesc_bf16(128, kTileKeys, false, false);
#endif
    for (; ok && have_piece; have_piece = walk.next(p, w)) {
        if (w.lo >= w.hi) continue;   // a block that sees no key: no product
        ok = __all_sync(0xffffffffu, wait_bar(c, bar_addr(c, B_QREADY), g & 1u));
        if (!ok) break;
        const uint32_t dS = tmem + TM_S + 64u * sb;
        for (int t = w.lo; t < w.hi && ok; ++t, ++it) {
            if ((it & 1u) != sb) continue;
            uint32_t ku = it * kKUnits;
            ok = __all_sync(0xffffffffu, wait_bar(c, bar_addr(c, B_SREAD + sb), ((it >> 1) & 1u) ^ 1u));
            if (!ok) break;
            ok = __all_sync(0xffffffffu, wait_bar(c, bar_addr(c, B_RFULL + sb), (it >> 1) & 1u));
            if (!ok) break;
            tc_fence_after();
            if (lane == 0) {
#if MLA_CHUNK_F8
                const uint64_t a = make_sdesc(c.base + OFF_QR, 16, 512, kSwizzle64B), b = make_sdesc(c.base + OFF_KR, 16, 512, kSwizzle64B);
#else
                const uint64_t a = make_sdesc(c.base + OFF_QR, 16, 1024, kSwizzle128B), b = make_sdesc(c.base + OFF_KR, 16, 1024, kSwizzle128B);
#endif
#pragma unroll
                for (int k = 0; k < kRopeSteps; ++k) umma2_ss<MLA_CHUNK_F8>(dS, a + 2u * k, b + 2u * k, idS, k > 0 ? 1u : 0u);
                umma2_commit(bar_addr(c, B_REMPTY));
            }
            __syncwarp();
#pragma unroll 1
            for (int u = 0; u < kKUnits; ++u, ++ku) {
                const uint32_t st = ku % kKStages;
                ok = __all_sync(0xffffffffu, wait_bar(c, bar_addr(c, B_KFULL + sb * kKStages + st), (phases >> st) & 1u));
                phases ^= 1u << st;
                if (!ok) break;
                tc_fence_after();
                if (lane == 0) {
                    const uint64_t b = make_sdesc(c.base + OFF_K + st * kUnitBytes, 16, 1024, kSwizzle128B);
                    if (u * kUnitDims < kQTmemDims) {
                        const uint32_t a = tmem + TM_Q + 8u * kStepsPerUnit * (uint32_t)u;
#pragma unroll
                        for (int k = 0; k < kStepsPerUnit; ++k)   // +32 bytes a step, +8 KB a box
                            umma2_ts<MLA_CHUNK_F8>(dS, a + 8u * k, b + (uint64_t)((k >> 2) * 512 + (k & 3) * 2), idS, 1u);
                    } else {
                        const uint64_t a = make_sdesc(c.base + OFF_Q + (uint32_t)(u * kUnitDims - kQTmemDims) / kBoxDims * 8192u, 16,
                                                      1024, kSwizzle128B);
#pragma unroll
                        for (int k = 0; k < kStepsPerUnit; ++k)
                            umma2_ss<MLA_CHUNK_F8>(dS, a + (uint64_t)((k >> 2) * 512 + (k & 3) * 2),
                                                   b + (uint64_t)((k >> 2) * 512 + (k & 3) * 2), idS, 1u);
                    }
                    umma2_commit(bar_addr(c, B_KEMPTY + st));
                    if (u == kKUnits - 1) umma2_commit(bar_addr(c, B_SFULL + sb));
                }
                __syncwarp();
            }
        }
        if (!ok) break;
        if (lane == 0) umma2_commit(bar_addr(c, B_QFREE));   // of this thread's products; the other commits its own
        __syncwarp();
        ++g;
    }
    if (lane == 0) umma2_commit(bar_addr(c, B_DRAIN));
    __syncwarp();
    // the arrivals for this thread's last tile have come: none is on its way when the CTA leaves
    const uint32_t mine = (it + 1u - sb) >> 1;   // tiles of this thread
    if (ok && mine > 0) wait_bar(c, bar_addr(c, B_SREAD + sb), (mine - 1u) & 1u);
}

// ----------------------------------------------------------------------------
// PV issuers (CTA 0): output dims [256 h, 256 h + 256).
// ----------------------------------------------------------------------------
__device__ void pv_role(const Ctx &c, const ChunkParams &p, ChunkWalk walk, ChunkPiece w, bool have_piece, uint32_t tmem, int h,
                        int lane) {
    uint32_t it = 0, vp = 0, g = 0;   // tiles, pages, pieces
    bool ok = true;
#if MLA_CHUNK_F8
    constexpr uint32_t idPV = make_idesc_e4m3(128, 256, false, true), idLow = idPV | kIdescAE5m2;
#else
    constexpr uint32_t idPV = make_idesc_bf16(128, 256, false, true);
#endif
    const uint32_t d = tmem + TM_O + 128u * (uint32_t)h;
    for (; ok && have_piece; have_piece = walk.next(p, w)) {
        if (w.lo >= w.hi) continue;
        for (int t = w.lo; t < w.hi && ok; ++t, ++it) {
            ok = __all_sync(0xffffffffu, wait_bar(c, bar_addr(c, B_PFULL + (it & 1u)), (it >> 1) & 1u));
            if (ok && t == w.lo) ok = __all_sync(0xffffffffu, wait_bar(c, bar_addr(c, B_OFREE), (g & 1u) ^ 1u));
            const uint32_t pbuf = c.base + OFF_P + (it & 1u) * 16384u;
            for (int pg = 0; pg < kTilePages && ok; ++pg, ++vp) {
                const int used = min(w.keys - (kTilePages * t + pg) * kPage, kPage);
                if (used <= 0) break;
                const int steps = (used + kStepKeys - 1) / kStepKeys;
                const uint32_t vu = vp * kVUnits + (kVUnits > 1 ? (uint32_t)h : 0u), st = vu % kVStages;
                ok = __all_sync(0xffffffffu, wait_bar(c, bar_addr(c, B_VFULL + st), (vu / kVStages) & 1u));
                if (!ok) break;
                tc_fence_after();
                if (lane == 0) {
                    const uint32_t acc = t > w.lo || pg > 0 ? 1u : 0u;
#if MLA_CHUNK_F8
                    // P: 128 keys a row, e4m3 parts, then e5m2 remainders 8 KB on; V: a box of 128 dims for each h
                    const uint64_t a = make_sdesc(pbuf, 16, 1024, kSwizzle128B) + 4u * pg;
                    const uint64_t b = make_sdesc(c.base + OFF_V + st * kUnitBytes + 8192u * (uint32_t)h, 8192, 1024, kSwizzle128B);
#pragma unroll
                    for (int k = 0; k < kPage / kStepKeys; ++k) {   // +32 keys: +4096 bytes of V
                        if (k < steps) {
                            umma2_ss<1>(d, a + 2u * k, b + 256u * k, idPV, k > 0 ? 1u : acc);
                            umma2_ss<1>(d, a + 512u + 2u * k, b + 256u * k, idLow, 1u);
                        }
                    }
#else
                    const uint64_t a = make_sdesc(pbuf + 8192u * (uint32_t)pg, 16, 1024, kSwizzle128B);
                    const uint64_t b = make_sdesc(c.base + OFF_V + st * kUnitBytes, 8192, 1024, kSwizzle128B);
#pragma unroll
                    for (int k = 0; k < kPage / kStepKeys; ++k)     // +16 keys: +2048 bytes of V
                        if (k < steps) umma2_ss<0>(d, a + 2u * k, b + 128u * k, idPV, k > 0 ? 1u : acc);
#endif
                    umma2_commit(bar_addr(c, B_VEMPTY + st));
                }
                __syncwarp();
            }
            if (ok && lane == 0) umma2_commit(bar_addr(c, B_PVDONE + (it & 1u)));
            __syncwarp();
        }
        ++g;
    }
    if (lane == 0) umma2_commit(bar_addr(c, B_DRAINPV));
    __syncwarp();
    if (ok && g > 0) wait_bar(c, bar_addr(c, B_OFREE), (g - 1u) & 1u);   // the last block's, as for QK^T
}

// Warps meet (the four that hold the same rows, or all eight): what any wrote to shared memory before is
// visible to all after.  Bounded, unlike a named barrier.
struct Meet {
    uint32_t bar, phase;
    __device__ __forceinline__ bool operator()(const Ctx &c, int lane) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
        const bool ok = __all_sync(0xffffffffu, wait_bar(c, bar, phase));
        phase ^= 1u;
        return ok;
    }
};

// All products of the CTA's first `it` tiles are in O, and the P buffers free (whole warp).
__device__ __forceinline__ bool wait_output(const Ctx &c, uint32_t it) {
    const bool ok = __all_sync(0xffffffffu, wait_bar(c, bar_addr(c, B_PVDONE + ((it - 1u) & 1u)), ((it - 1u) >> 1) & 1u));
    tc_fence_after();
    return ok;
}

// The products of the CTA's first g pieces are done with Q (whole warp).
__device__ __forceinline__ bool q_free(const Ctx &c, uint32_t g) {
    const bool ok = __all_sync(0xffffffffu, wait_bar(c, bar_addr(c, B_QFREE), (g & 1u) ^ 1u));
    tc_fence_after();
    return ok;
}

// ----------------------------------------------------------------------------
// Q of a piece, by the softmax warps: this CTA's 64 rows, the first kQTmemDims dims (512 bytes) into
// TMEM (lanes r and 64 + r alike), the others into shared memory.  Rows past the block's end are zero.
// All copies are asynchronous and in whole lines; the part for TMEM passes through shared memory (each lane loading
// its row's bytes itself took 32 lines an instruction, and 7000 cycles instead of 3000 for it all).  Everything
// else has to be free of the piece before (q_free); on e4m3 that is awaited here.  g pieces were loaded before.
// ----------------------------------------------------------------------------
__device__ __forceinline__ bool load_q(const Ctx &c, const ChunkParams &p, const ChunkPiece &w, uint32_t tmem, int cta, Meet &all,
                                       uint32_t g) {
    const int tid = threadIdx.x, lane = tid & 31, quarter = (tid >> 5) & 3, part = tid >> 7;
    const int rows = (int)min((int64_t)w.seq.n * p.hpk - (int64_t)w.rb * kBlockRows - 64 * cta, (int64_t)64);   // of this CTA
    const int row0 = w.rb * kBlockRows + 64 * cta;
    constexpr int kLatCh = kDv * kElem / 16;   // 16-byte chunks of a row's latent dims
    const int ch = tid % kLatCh;
    const uint32_t dst = c.base + (ch < 32 ? OFF_QS : OFF_Q + (uint32_t)((ch - 32) >> 3) * 8192u);
#pragma unroll 4
    for (int r = tid / kLatCh; r < 64; r += 256 / kLatCh)
        cp_async_16(dst + (ch < 32 ? (uint32_t)r * 512u + (uint32_t)((ch ^ (r & 7)) << 4) : swz128_offset(r, ch & 7)),
                    q_row(p, w, r < rows ? row0 + r : row0, false) + 16 * ch, r < rows);
#if MLA_CHUNK_F8
    if (!q_free(c, g)) return false;
#endif
    constexpr int kCh = (int)kRopeRow / 16;
#pragma unroll
    for (int i = tid; i < 64 * kCh; i += 256) {
        const int r = i / kCh, k = i % kCh;
        cp_async_16(c.base + OFF_QR + (kRopeRow == 128 ? swz128_offset(r, k) : swz64_offset(r, k)),
                    q_row(p, w, r < rows ? row0 + r : row0, true) + 16 * k, r < rows);
    }
    cp_async_wait_all();
    if (!all(c, lane)) return false;
    const int r = (32 * quarter + lane) & 63;
    const uint8_t *src = reinterpret_cast<const uint8_t *>(__cvta_shared_to_generic(c.base)) + OFF_QS + r * 512;
    uint32_t x[64];   // 256 bytes of the row
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const uint4 t = *reinterpret_cast<const uint4 *>(src + (((16 * part + j) ^ (r & 7)) << 4));
        x[4 * j] = t.x; x[4 * j + 1] = t.y; x[4 * j + 2] = t.z; x[4 * j + 3] = t.w;
    }
    tmem_st_32x32b_x64(tmem + ((uint32_t)quarter << 21) + TM_Q + 64u * (uint32_t)part, x);
    tmem_st_wait();
    fence_proxy_async_smem();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive_lead(lead(c, B_QREADY));
    return true;
}

// ----------------------------------------------------------------------------
// Softmax and epilogue (warps 0-7).
// ----------------------------------------------------------------------------
__device__ __forceinline__ float max32(const float (&v)[32]) {   // three-input maxima: 32 -> 11 -> 4 -> 1
    float t[11];
#pragma unroll
    for (int i = 0; i < 10; ++i) t[i] = fmax3(v[3 * i], v[3 * i + 1], v[3 * i + 2]);
    t[10] = fmaxf(v[30], v[31]);
    return fmax3(fmax3(t[0], t[1], t[2]), fmax3(t[3], t[4], t[5]), fmax3(fmax3(t[6], t[7], t[8]), t[9], t[10]));
}
// Floats as whole numbers in the same order, and back.
__device__ __forceinline__ int ordered(float x) {
    const int i = __float_as_int(x);
    return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float from_ordered(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }

#if MLA_CHUNK_F8
// Two weights: `hi` as an e4m3 pair, and what is left as e5m2 in the upper byte of each half of the result.  By way of
// fp16 (2^-11 of a weight's binade).  The remainder passes through a sum with 8 hi, which keeps 8 significant bits
// of the weight; where hi is a normal number that leaves the remainder three, which e5m2 holds.  An fp16 value's upper
// byte is an e5m2 value: a threshold (a byte) added to the lower one carries into it if the two pass 255.
__device__ __forceinline__ uint32_t split_e4m3x2(float2 p, uint16_t &hi, uint32_t threshold) {
    uint32_t h, back, rest;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(p.y), "f"(p.x));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(hi) : "r"(h));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(hi));
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(rest) : "r"(back), "r"(0x47004700u), "r"(h));      // 8 back + (h - back)
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(rest) : "r"(back), "r"(0xc800c800u), "r"(rest));   // - 8 back
    return rest + threshold;
}
// Thresholds of the keys 2i and 2i + 1 of a thread's 32: 8 * (key's five bits reversed) + 4, in either half.
__host__ __device__ constexpr uint32_t dither_of(int key) {
    uint32_t v = 0;
    for (int i = 0; i < 5; ++i) v |= (uint32_t)((key >> i) & 1) << (7 - i);
    return v + 4u;
}
__host__ __device__ constexpr uint32_t dither_pair(int i) { return dither_of(2 * i) | dither_of(2 * i + 1) << 16; }
#endif

__device__ void softmax_role(const Ctx &c, const ChunkParams &p, ChunkWalk walk, ChunkPiece w, bool have_piece, uint32_t tmem,
                             int cta) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int quarter = warp & 3, part = warp >> 2;
    const int r = 32 * (quarter & 1) + lane, kh = quarter >> 1;
    const uint32_t lane_base = (uint32_t)quarter << 21;
    uint8_t *smem = reinterpret_cast<uint8_t *>(__cvta_shared_to_generic(c.base));
    // Row maxima of three tiles in turn.  A tile's word is reset in the tile before, ahead of that tile's
    // meeting, when every thread has read what the word held two tiles earlier.
    int *const top = reinterpret_cast<int *>(smem + OFF_STAT) + r;
    float *const den = reinterpret_cast<float *>(smem + OFF_STAT) + r;   // denominators [4][64], between pieces
    const int lowest = ordered(-INFINITY);
    Meet meet{bar_addr(c, B_PAIR + (warp & 1)), 0u}, all{bar_addr(c, B_ALL), 0u};
    const uint32_t sread[2] = {lead(c, B_SREAD), lead(c, B_SREAD + 1)};
    const uint32_t pfull[2] = {lead(c, B_PFULL), lead(c, B_PFULL + 1)}, ofree = lead(c, B_OFREE);
    const float c2 = p.scale_log2;

    uint32_t it = 0, g = 0;   // tiles; pieces whose Q is loaded
    bool ok = true;
    if (have_piece && w.lo < w.hi) {
        ok = load_q(c, p, w, tmem, cta, all, g);
        ++g;
    }
    while (ok && have_piece) {
        const int64_t row64 = (int64_t)w.rb * kBlockRows + 64 * cta + r;
        const bool row_real = row64 < (int64_t)w.seq.n * p.hpk;
        const int row = (int)row64, qi = p.token_of(row);
        const int n_vis = row_real ? w.seq.visible(qi, p.causal) : 0;
        const bool any = w.hi > w.lo;
        float m_ref = -INFINITY, l_sum = 0.f;
        uint32_t slot = 0;
        if (any) {   // words of the first tile; the denominators that shared the place have been read
            if (part == 0 && kh == 0) top[0] = lowest;
            ok = meet(c, lane);
        }
        for (int t = w.lo; t < w.hi && ok; ++t, ++it) {
            const uint32_t sb = it & 1u;
            ok = __all_sync(0xffffffffu, wait_bar(c, bar_addr(c, B_SFULL + sb), (it >> 1) & 1u));
            if (!ok) break;
            tc_fence_after();
            float sv[32];
            {
                uint32_t raw[32];
                tmem_ld_32x32b_x32(tmem + lane_base + TM_S + 64u * sb + 32u * (uint32_t)part, raw);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j) sv[j] = __uint_as_float(raw[j]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote_relaxed(sread[sb]);
            const int nv = n_vis - (t * kTileKeys + 64 * kh + 32 * part);   // this thread's visible keys
            if (__any_sync(0xffffffffu, nv < 32)) {
#pragma unroll
                for (int j = 0; j < 32; ++j) sv[j] = j < nv ? sv[j] : -INFINITY;
            }
            const uint32_t next_slot = slot == 2u ? 0u : slot + 1u;
            atomicMax(top + 64 * slot, ordered(max32(sv)));
            if (part == 0 && kh == 0) top[64 * next_slot] = lowest;
            ok = meet(c, lane);
            if (!ok) break;
            const float mt = from_ordered(top[64 * slot]) * c2;
            slot = next_slot;
            const bool o_live = m_ref != -INFINITY;
            const bool raise = mt > m_ref + kRescaleThreshold;   // true for the first finite tile
            float factor = 1.f;
            if (raise) {
                if (o_live) factor = ex2_approx(m_ref - mt);
                m_ref = mt;
                l_sum *= factor;
            }
            const float neg_m = m_ref == -INFINITY ? 0.f : kPExp - m_ref;
            float2 ps[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#if MLA_CHUNK_F8
            const uint32_t shift = ((4u * (uint32_t)t + (uint32_t)(2 * kh + part) + 61u * (uint32_t)row) * 0x9e3779b1u >> 24) * 0x00010001u;
            uint32_t pk[8], pl[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 a01 = __ffma2_rn(make_float2(sv[4 * j], sv[4 * j + 1]), make_float2(c2, c2), make_float2(neg_m, neg_m));
                const float2 a23 = __ffma2_rn(make_float2(sv[4 * j + 2], sv[4 * j + 3]), make_float2(c2, c2), make_float2(neg_m, neg_m));
                const float2 p01 = make_float2(ex2_approx(a01.x), ex2_approx(a01.y));
                const float2 p23 = make_float2(ex2_approx(a23.x), ex2_approx(a23.y));
                uint16_t h0, h1;
                const uint32_t r0 = split_e4m3x2(p01, h0, dither_pair(2 * j) ^ shift);
                const uint32_t r1 = split_e4m3x2(p23, h1, dither_pair(2 * j + 1) ^ shift);
                pk[j] = (uint32_t)h0 | ((uint32_t)h1 << 16);
                pl[j] = __byte_perm(r0, r1, 0x7531);
                ps[0] = __fadd2_rn(ps[0], p01);
                ps[1] = __fadd2_rn(ps[1], p23);
            }
#else
            uint32_t pk[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float2 a = __ffma2_rn(make_float2(sv[2 * j], sv[2 * j + 1]), make_float2(c2, c2), make_float2(neg_m, neg_m));
                const float2 pp = make_float2(ex2_approx(a.x), ex2_approx(a.y));
                pk[j] = pack_bf16x2(pp.x, pp.y);
                ps[j & 1] = __fadd2_rn(ps[j & 1], pp);   // the denominator sums the unrounded weights
            }
#endif
            l_sum += (ps[0].x + ps[0].y) + (ps[1].x + ps[1].y);
            // the P buffer is free once the PV that read it has completed
            if (it >= 2) {
                ok = __all_sync(0xffffffffu, wait_bar(c, bar_addr(c, B_PVDONE + sb), ((it >> 1) & 1u) ^ 1u));
                if (!ok) break;
            }
            uint8_t *const pb = smem + OFF_P + sb * 16384u;
#if MLA_CHUNK_F8
#pragma unroll
            for (int ch = 0; ch < 2; ++ch) {
                const uint32_t o = swz128_offset(r, 4 * kh + 2 * part + ch);
                *reinterpret_cast<uint4 *>(pb + o) = make_uint4(pk[4 * ch], pk[4 * ch + 1], pk[4 * ch + 2], pk[4 * ch + 3]);
                *reinterpret_cast<uint4 *>(pb + 8192u + o) = make_uint4(pl[4 * ch], pl[4 * ch + 1], pl[4 * ch + 2], pl[4 * ch + 3]);
            }
#else
#pragma unroll
            for (int ch = 0; ch < 4; ++ch)
                *reinterpret_cast<uint4 *>(pb + 8192u * kh + swz128_offset(r, 4 * part + ch)) =
                    make_uint4(pk[4 * ch], pk[4 * ch + 1], pk[4 * ch + 2], pk[4 * ch + 3]);
#endif
            if (__any_sync(0xffffffffu, raise && o_live)) {   // O is complete up to the tile before
                ok = __all_sync(0xffffffffu, wait_bar(c, bar_addr(c, B_PVDONE + (sb ^ 1u)), ((it - 1) >> 1) & 1u));
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {   // the lane's columns h = part
                    const uint32_t col = tmem + lane_base + TM_O + 128u * (uint32_t)part + 32u * (uint32_t)q;
                    uint32_t o[32];
                    tmem_ld_32x32b_x32(col, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const float2 v = __fmul2_rn(make_float2(__uint_as_float(o[j]), __uint_as_float(o[j + 1])), make_float2(factor, factor));
                        o[j] = __float_as_uint(v.x);
                        o[j + 1] = __float_as_uint(v.y);
                    }
                    tmem_st_32x32b_x32(col, o);
                }
                tmem_st_wait();
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_lead(pfull[sb]);
        }
        if (!ok) break;

        ChunkPiece n;
        const bool have_next = walk.next(p, n);
        // The next piece's Q first: its first QK^T runs during the epilogue.  On e4m3 it is fetched while O is
        // being completed (444 us instead of 452); on bf16 it passes through the P buffers, which are free after that.
#if !MLA_CHUNK_F8
        if (any) {
            ok = wait_output(c, it);
            if (!ok) break;
        }
#endif
        if (have_next && n.lo < n.hi) {
#if !MLA_CHUNK_F8
            ok = q_free(c, g);
            if (!ok) break;
#endif
            ok = load_q(c, p, n, tmem, cta, all, g);
            if (!ok) break;
            ++g;
        }
#if MLA_CHUNK_F8
        if (any) {
            ok = wait_output(c, it);
            if (!ok) break;
        }
#endif

        // ---- epilogue.  The row's denominator is the sum of its four threads', in one order for all.
        ok = meet(c, lane);               // every maximum has been read, and the rows' part of the P buffers
        if (ok && any) {
            den[64 * (2 * kh + part)] = l_sum;
            ok = meet(c, lane);
            l_sum = (den[0] + den[64]) + (den[128] + den[192]);
        }
        if (!ok) break;
        const bool live = l_sum != 0.f;   // NaN among a row's inputs stays NaN
        const bool direct = w.slot < 0;
        const float inv = live ? (direct ? p.out_scale : 1.f) / l_sum : 0.f;
        if (row_real && kh == 0 && part == 0) {
            float lse = -INFINITY;
            if (live) {
                float lg;
                asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(lg) : "f"(l_sum));
                lse = (m_ref - kPExp + lg) * 0.6931471805599453f;
            }
            if (direct) p.lse[(int64_t)(w.seq.first + qi) * p.h_q + w.hk * p.hpk + row - qi * p.hpk] = lse;
            else p.ws_lse[w.slot * kBlockRows + 64 * cta + r] = lse;
        }
        // This thread's dims: [256 part + 128 kh, + 128), a column of TMEM each, in passes of 128 bytes (64
        // bf16 values, or 32 of a partial's fp32).  A pass goes through shared memory, [32 rows of the group]
        // [4 threads x 128 bytes], 16-byte chunks swizzled by row, so that a store instruction writes four
        // whole lines of one row instead of a piece of 32 rows' each.  A block's output takes 4000 to 6000 cycles, as
        // the stores of all SMs come together; the next block's Q and first two products of QK^T pass meanwhile.
        const int passes = direct ? 2 : 4;
        uint8_t *const stage = smem + OFF_P + (quarter & 1) * 16384;
        const int mine = kh + 2 * part;   // which of the row's four threads, and of the group's four warps
        // the rows that this warp stores: eight of its group, from the block's row `first`
        const int64_t first = (int64_t)w.rb * kBlockRows + 64 * cta + 32 * (quarter & 1) + 8 * mine;
        const int orows = (int)min((int64_t)w.seq.n * p.hpk - first, (int64_t)8);
        const int otoken = p.token_of((int)first), ohead = (int)first - otoken * p.hpk;
        const int64_t orow = (int64_t)(w.seq.first + otoken) * p.o_s0 + (int64_t)(w.hk * p.hpk + ohead) * p.o_s1;
#pragma unroll 1
        for (int q = 0; q < passes && ok; ++q) {
            uint32_t o[32];
            if (!any) {
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] = 0u;
            } else if (direct) {
                uint32_t y[64];
                tmem_ld_32x32b_x64(tmem + lane_base + TM_O + 128u * (uint32_t)part + 64u * (uint32_t)q, y);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] = pack_bf16x2(__uint_as_float(y[2 * j]) * inv, __uint_as_float(y[2 * j + 1]) * inv);
            } else {
                tmem_ld_32x32b_x32(tmem + lane_base + TM_O + 128u * (uint32_t)part + 32u * (uint32_t)q, o);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * inv);
            }
#pragma unroll
            for (int ch = 0; ch < 8; ++ch)   // a row without a visible key gives zeros, whatever its products left
                *reinterpret_cast<uint4 *>(stage + lane * 512 + mine * 128 + ((ch ^ (lane & 7)) << 4)) =
                    live ? make_uint4(o[4 * ch], o[4 * ch + 1], o[4 * ch + 2], o[4 * ch + 3]) : make_uint4(0u, 0u, 0u, 0u);
            ok = meet(c, lane);
            if (!ok) break;
            if (q == passes - 1 && any) {    // O may be written again
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote_relaxed(ofree);
            }
            const int seg = lane >> 3, ch = lane & 7;   // of a row: the part of thread `seg`
            uint4 v[8];                                 // the warp's eight rows of the group
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[k] = *reinterpret_cast<const uint4 *>(stage + (8 * mine + k) * 512 + seg * 128 + ((ch ^ k) << 4));
            if (direct) {
                uint16_t *dst = p.out + orow + 256 * (seg >> 1) + 128 * (seg & 1) + 64 * q + 8 * ch;
                int hd = ohead;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    if (k < orows) *reinterpret_cast<uint4 *>(dst) = v[k];
                    dst += p.o_s1;
                    if (++hd == p.hpk) {
                        hd = 0;
                        dst += p.o_s0 - p.hpk * p.o_s1;
                    }
                }
            } else {
                float *dst = p.ws_o + ((int64_t)w.slot * kBlockRows + 64 * cta + 32 * (quarter & 1) + 8 * mine) * kDv +
                             256 * (seg >> 1) + 128 * (seg & 1) + 32 * q + 4 * ch;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k < orows) *reinterpret_cast<uint4 *>(dst + k * kDv) = v[k];
            }
            if (q < passes - 1) ok = meet(c, lane);     // the rows' part of the stage has been read
        }
        ok = ok && all(c, lane);                        // and all of it, before the next weights are stored there
        w = n;
        have_piece = have_next;
    }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
mla_chunk_kernel(const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap kr, const __grid_constant__ ChunkParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    Ctx c;
    c.base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (c.base - raw);
    c.bars = c.base + OFF_BAR;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + OFF_MISC);
    c.abort_flag = reinterpret_cast<volatile int *>(smem + OFF_MISC + 4);
    c.err = p.err;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cta = (int)cluster_ctarank();
    if (threadIdx.x == 0) {
        *c.abort_flag = 0;
        for (int i = 0; i < kKStages; ++i) {
            mbar_init(bar_addr(c, B_KFULL + i), 2);
            mbar_init(bar_addr(c, B_KFULL + kKStages + i), 2);
            mbar_init(bar_addr(c, B_KEMPTY + i), 1);
        }
        for (int i = 0; i < kVStages; ++i) {
            mbar_init(bar_addr(c, B_VFULL + i), 2);
            mbar_init(bar_addr(c, B_VEMPTY + i), kVUnits > 1 ? 1 : 2);   // e4m3: both PV threads read a unit
        }
        mbar_init(bar_addr(c, B_RFULL), 2);
        mbar_init(bar_addr(c, B_RFULL + 1), 2);
        mbar_init(bar_addr(c, B_REMPTY), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar_addr(c, B_PFULL + i), 16);
            mbar_init(bar_addr(c, B_SFULL + i), 1);
            mbar_init(bar_addr(c, B_SREAD + i), 16);   // the softmax warps of both CTAs
            mbar_init(bar_addr(c, B_PVDONE + i), 2);   // the two PV threads
        }
        mbar_init(bar_addr(c, B_OFREE), 16);
        mbar_init(bar_addr(c, B_QREADY), 16);
        mbar_init(bar_addr(c, B_QFREE), 2);
        mbar_init(bar_addr(c, B_DRAIN), 2);
        mbar_init(bar_addr(c, B_DRAINPV), 2);
        mbar_init(bar_addr(c, B_TAIL), 1);
        mbar_init(bar_addr(c, B_PAIR), 4);
        mbar_init(bar_addr(c, B_PAIR + 1), 4);
        mbar_init(bar_addr(c, B_ALL), 8);
        fence_mbar_init();
    }
    if (warp == 8 && lane == 0) {
        tma_prefetch_desc(&km);
        tma_prefetch_desc(&kr);
    }
    if (warp == 9) {
        tmem_alloc_pair(smem_u32(tmem_slot), 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    cluster_arrive();   // barriers of both CTAs are set up before any remote arrival
    // The launch may come while the kernel before it on the stream still runs: setting up does not wait for
    // that kernel, what reads or writes global memory does.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // every role walks the part's pieces by itself; the first one's lengths come during the cluster's barrier
    ChunkWalk walk;
    walk.init(p.md, blockIdx.x >> 1);
    ChunkPiece w;
    const bool have = walk.next(p, w);
    cluster_wait();
    const uint32_t tmem = *tmem_slot;

    if (warp < 8) {
        softmax_role(c, p, walk, w, have, tmem, cta);
    } else if (warp == 8) {
        k_producer(c, p, walk, w, have, &km, &kr, cta, lane, l2_policy_evict_last());
    } else if (warp == 9) {
        v_producer(c, p, walk, w, have, &km, cta, lane, l2_policy_evict_last());
    } else if (warp < 12) {
        if (cta == 0) qk_role(c, p, walk, w, have, tmem, (uint32_t)(warp - 10), lane);
    } else {
        if (cta == 0) pv_role(c, p, walk, w, have, tmem, warp - 12, lane);
    }
    __syncthreads();
    // both issuers' products are over, in this CTA too
    if (threadIdx.x == 0) {
        drain_bar(c, bar_addr(c, B_DRAIN), 0);
        drain_bar(c, bar_addr(c, B_DRAINPV), 0);
        if (*c.abort_flag) drain_after_abort();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // Neither CTA leaves, nor frees TMEM, while the other's work may touch it.  Execution alone: each role has
    // seen what the other CTA sends it, and a releasing barrier would wait 4000 cycles for the output stores.
    cluster_arrive_relaxed();
    cluster_wait();
    if (warp == 9) tmem_dealloc_pair(tmem, 512);
}

}  // namespace MLA_CHUNK_NS
}  // namespace mla
