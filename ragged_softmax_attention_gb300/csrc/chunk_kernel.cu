// Attention of chunks of new tokens over a paged KV cache, sm_103a: token t of a
// request with d new tokens and n keys (the chunk included) sees the keys lo_t ..
// hi_t - 1, hi_t = n - d + t + 1 (causal) or n, lo_t = max(0, n - d + t - window) or 0.
//
// The (token, head) rows that share a KV head's keys fill the MMA M axis, whole
// tokens, up to 128 rows a row tile, as in the tree decode:
//   S [128 x 128]  = Q_tile * K_tile^T          (tcgen05, FP32 in TMEM)
//   O [128 x D]   += P [128 x 128] * V_tile      (tcgen05, P and O in TMEM)
// with a thread to a row and a conditional rescale (the base of the exponentials moves
// when a maximum rose by more than 8 log2 units).
//
// A unit is (request, KV head, NT consecutive row tiles).  Units are laid end to end by
// weight -- the keys that they walk and what it costs to start one -- and every CTA takes
// an equal contiguous range, so one long request, many short ones and a mixed batch all
// fill the GPU; a unit that a range's border cuts leaves partial rows, at most two pieces
// a CTA whatever the batch, which a second launch merges.  A unit's weight is linear in
// its number within the request (but for the window's start), so sums over units are
// closed forms: every CTA works out its range from the lengths by itself, one pass over
// the requests and one binary search, and no planning launch is needed.
//
// D = 128 with more than a row tile a request: NT = 2, two row tiles take turns on the
// tensor core over shared K and V tiles, each with its own MMA-issuing thread, softmax
// warpgroup, S buffer and O.  D = 256 with more than a row tile runs on pairs of CTAs
// (another file).  Otherwise NT = 1 with three S buffers (two at D = 256), QK and PV issued
// by a thread each.
//
// FP8 caches: QK is kind::f8f6f4 on the bytes as they land, with each query row split in place
// into two E4M3 terms (as in the tree decode; two terms of K = 32 take the tensor core as long
// as one BF16 pass); PV is the BF16 kernel's, on values that four warps widen (exactly) into a
// ring of two slots, so that most of shared memory is for copies in flight.  (Keys and values
// widened in place, in a ring of BF16 slots: 811 us for 761 below.)  Their softmax warpgroups
// have 160 registers, which the whole row of S does not fit, and read it twice.
//
// Measured (GB300): 2,048 tokens on 32,768 keys, 40/8 heads, 907 us, 1.56 PFLOP/s, bound by
// the chain of a row tile (2,800 cycles a key tile of two, 2,048 of them products); 16
// prompts of 300 .. 5,000 tokens, 32/8 heads, 797 us, 1.24 PFLOP/s, and 500 .. 2,000 tokens
// with a window of 1,023 keys 144 us, where the ends of units (7,300 cycles) and masked tiles
// take the rest; 48 requests of which 40 bring one token 322 us, 61 % of DRAM; FP8, 256 ..
// 1,024 tokens on 2,048 .. 16,384 keys, 755 us, 1.23 PFLOP/s, 3,800 cycles a key tile, to which
// everything adds (one QK term less would take 75 us off, the widening 32, the second
// reading 20); 24 tokens on 700 keys 14.6 us, 6 of them before the first scores.
//
// Warp roles: warp 0 copies K and V tiles, warps 1 and 2 issue the MMAs, warp 3 works out
// the pieces and copies the queries, then NT warpgroups of softmax, then (FP8) a
// warpgroup that widens.
#include "chunk_common.cuh"

namespace fw {
namespace {

using namespace chunk;

template <int D_, int NT_, bool KV8_>
struct ChunkCfg {
    static constexpr int D = D_, NT = NT_;
    static constexpr bool KV8 = KV8_;
    // S buffers of a stream, i.e. key tiles QK runs ahead: what O leaves of TMEM.
    static constexpr int kSB = NT == 2 ? 1 : D == 128 ? 3 : 2;
    static constexpr int kTileSlots = D / 128;                  // ring slots of one K or V tile
    static constexpr int kChunkBytes = 128 * 128;               // 128 rows x 64 bf16 columns
    static constexpr int kSlotBytes = 2 * kChunkBytes;          // 128 rows x 128 columns
    static constexpr int kQBytes = 128 * D * 2;
    // FP8: two slots of widened values, the rest is for keys and values as they land.
    static constexpr int kSlots = KV8 ? 2 : (229376 - NT * kQBytes) / kSlotBytes;
    static constexpr int kRawSlots = KV8 ? (229376 - NT * kQBytes - kSlots * kSlotBytes) / kChunkBytes / 2 : 0;      // of each
    static constexpr int kOffQ = 0;
    static constexpr int kOffRing = NT * kQBytes;
    static constexpr int kOffRaw = kOffRing + kSlots * kSlotBytes;      // keys, then values
    static constexpr int kOffBar = kOffRaw + 2 * kRawSlots * kChunkBytes;
    static constexpr int kSched = !KV8 ? 4 : NT == 2 ? 2 : 3;       // unit records in flight (FP8: what there is room for)
    static constexpr int kBarSlotFull = 0;
    static constexpr int kBarSlotEmpty = kBarSlotFull + kSlots;
    static constexpr int kBarRawFull = kBarSlotEmpty + kSlots;  // FP8: keys [kRawSlots], then values
    static constexpr int kBarRawEmpty = kBarRawFull + 2 * kRawSlots;
    static constexpr int kBarQFull = kBarRawEmpty + 2 * kRawSlots;
    static constexpr int kBarQEmpty = kBarQFull + 1;
    static constexpr int kBarQReady = kBarQEmpty + 1;           // [kQSets], FP8: the queries are split
    static constexpr int kQSets = KV8 ? kSched : 0;             // rows' exponents, beside the unit's record
    static constexpr int kBarSFull = kBarQReady + kQSets;       // [NT][kSB]
    static constexpr int kBarPHalf = kBarSFull + NT * kSB;      // [NT][kSB]
    static constexpr int kBarPFull = kBarPHalf + NT * kSB;      // [NT][kSB]
    static constexpr int kBarPvDone = kBarPFull + NT * kSB;     // [NT][kSB]
    static constexpr int kBarIssued = kBarPvDone + NT * kSB;    // [NT]
    static constexpr int kBarDrain = kBarIssued + NT;           // [2]
    static constexpr int kBarSchedFull = kBarDrain + 2;
    static constexpr int kBarSchedEmpty = kBarSchedFull + kSched;
    static constexpr int kBarNever = kBarSchedEmpty + kSched;   // test hook: no thread ever arrives on it
    static constexpr int kNumBars = kBarNever + 1;
    static constexpr int kOffSched = (kOffBar + kNumBars * 8 + 63) / 64 * 64;
    static constexpr int kOffBad = kOffSched + kSched * 64;
    static constexpr int kOffPlan = (kOffBad + kBadUnits * kBadUnitWords * 4 + 15) / 16 * 16;
    static constexpr int kOffScan = kOffPlan + 32;              // [16] warp sums
    static constexpr int kOffMisc = kOffScan + 128;
    static constexpr int kOffExp = kOffMisc + 16;               // [kQSets][NT][128]
    static constexpr int kSmemBytes = kOffExp + kQSets * NT * 128 + 1024;
    static_assert(kSmemBytes <= 232448, "shared memory budget of one CTA exceeded");
    static constexpr int kThreads = 128 + NT * 128 + (KV8 ? 128 : 0);
    static constexpr int kSchedReaders = 3 + 4 * NT + (KV8 ? 4 : 0);    // issuers, the producer, softmax, widening warps
    // NT = 2: launched at 168 registers (FP8: 128) a thread; after the split
    // 128 x 80 + 256 x 208 = 63488 <= 384 x 168, FP8 128 x (72 + 120) + 256 x 160 = 512 x 128 (72 + 104
    // and 168: 771 us for 761, 80 + 64 and 184: 837).
    static constexpr uint32_t kRegsControl = KV8 ? 72 : 80, kRegsSoftmax = KV8 ? 160 : 208, kRegsWiden = 120;
    static_assert(kRegsControl < 128 && kRegsWiden < 128 && kRegsSoftmax > (KV8 ? 128 : 168), "which way each goes");
    static_assert(NT == 1 || KV8 || 128 * kRegsControl + 256 * kRegsSoftmax <= 384 * 168, "register split");
    static_assert(NT == 1 || !KV8 || 128 * (kRegsControl + kRegsWiden) + 256 * kRegsSoftmax <= 512 * 128, "register split");
    static constexpr uint32_t kIdescQK = KV8 ? kIdescF8QK : idesc_bf16_f32(128, kKvTile, false, false);
    static constexpr uint32_t kIdescPV = idesc_bf16_f32(128, 128, false, true);
    __device__ static constexpr uint32_t s_col(int x, int buf) { return (uint32_t)(x * kSB + buf) * 128u; }
    __device__ static constexpr uint32_t o_col(int x) { return (uint32_t)(NT * kSB + x) * 128u; }
    // Ring positions, in whole K or V tiles, of a piece of n key tiles: two streams take
    // K_j and V_j in turn; one runs QK kSB tiles ahead.  FP8: a ring each.
    static constexpr int kPerTile = KV8 ? 1 : 2 * kTileSlots;   // positions of a key tile
    __device__ static __forceinline__ int ring_k(int j, int n) { return KV8 ? j : NT == 2 ? 2 * j : pos_k<kSB>(j, n); }
    __device__ static __forceinline__ int ring_v(int j, int n) { return KV8 ? j : NT == 2 ? 2 * j + 1 : pos_v<kSB>(j, n); }
};

// Four E4M3 bytes as BF16 (exact; NaN stays NaN).
__device__ __forceinline__ uint2 widen4_bf16(uint32_t w) {
    uint32_t h0, h1;
    widen4(w, h0, h1);
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&h0));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&h1));
    return make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(b.x, b.y));
}

template <int D, int NT, bool KV8>
__global__ void __launch_bounds__(ChunkCfg<D, NT, KV8>::kThreads, 1)
chunk_kernel(const __grid_constant__ ChunkParams p, const __grid_constant__ CUtensorMap tm_q,
             const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
    using C = ChunkCfg<D, NT, KV8>;
    constexpr int kSB = C::kSB, TS = C::kTileSlots;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sQ = smem + C::kOffQ;
    uint8_t *sRing = smem + C::kOffRing;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
    uint64_t *slot_full = bars + C::kBarSlotFull;
    uint64_t *slot_empty = bars + C::kBarSlotEmpty;
    uint64_t *raw_full = bars + C::kBarRawFull;
    uint64_t *raw_empty = bars + C::kBarRawEmpty;
    uint64_t *q_full = bars + C::kBarQFull;
    uint64_t *q_empty = bars + C::kBarQEmpty;
    uint64_t *q_ready = bars + C::kBarQReady;
    uint64_t *s_full = bars + C::kBarSFull;
    uint64_t *p_half = bars + C::kBarPHalf;
    uint64_t *p_full = bars + C::kBarPFull;
    uint64_t *pv_done = bars + C::kBarPvDone;
    uint64_t *issued = bars + C::kBarIssued;
    uint64_t *drain = bars + C::kBarDrain;
    uint64_t *sched_full = bars + C::kBarSchedFull;
    uint64_t *sched_empty = bars + C::kBarSchedEmpty;
    ChunkUnit *sched = reinterpret_cast<ChunkUnit *>(smem + C::kOffSched);
    uint32_t *bad = reinterpret_cast<uint32_t *>(smem + C::kOffBad);
    long long *plan = reinterpret_cast<long long *>(smem + C::kOffPlan);
    long long *scan = reinterpret_cast<long long *>(smem + C::kOffScan);
    int8_t *q_exp = reinterpret_cast<int8_t *>(smem + C::kOffExp);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kOffMisc + 4);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kSlots; ++i) {
            mbar_init(&slot_full[i], KV8 ? 4 : 1); mbar_init(&slot_empty[i], NT);
        }
        for (int i = 0; i < 2 * C::kRawSlots; ++i) {
            mbar_init(&raw_full[i], 1); mbar_init(&raw_empty[i], i < C::kRawSlots ? NT : 4);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, NT);
        for (int i = 0; i < C::kQSets; ++i) mbar_init(&q_ready[i], 4);
        for (int i = 0; i < NT * kSB; ++i) {
            mbar_init(&s_full[i], 1); mbar_init(&p_half[i], 4); mbar_init(&p_full[i], 4); mbar_init(&pv_done[i], 1);
        }
        for (int i = 0; i < NT; ++i) mbar_init(&issued[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&drain[i], 1);
        for (int i = 0; i < C::kSched; ++i) { mbar_init(&sched_full[i], 1); mbar_init(&sched_empty[i], C::kSchedReaders); }
        mbar_init(bars + C::kBarNever, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tm_q); tma_prefetch_desc(&tm_k); tma_prefetch_desc(&tm_v);
    }
    if (warp == 1) { tmem_alloc(tmem_slot, 512); tmem_relinquish(); }
    pdl_launch_dependents();                       // the merge may take its place; it waits for this grid
    chunk_plan<NT>(p, blockIdx.x, plan, scan);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const WaitCtx wc{p.status, p.timeout_ns, abort_flag};
    auto wait_unit = [&](int k) -> const ChunkUnit * {
        const int sl = k % C::kSched;
        return mbar_wait(&sched_full[sl], (k / C::kSched) & 1, wc) ? &sched[sl] : nullptr;
    };
    auto free_unit = [&](int k) { mbar_arrive(&sched_empty[k % C::kSched]); };
    // A unit record for a whole warp; b < 0 at the end.
    auto warp_unit = [&](int k) -> ChunkUnit {
        const ChunkUnit *ur = wait_unit(k);
        ChunkUnit u;
        u.b = -1;
        if (ur) u = *ur;
        __syncwarp();
        if (lane == 0) free_unit(k);
        return u;
    };

    if (warp < 4) {
      if constexpr (NT == 2) setmaxnreg_dec<C::kRegsControl>();
      if (warp == 0) {
        // ------------------------------------------------------------ producer
        const int box_rows = p.ps < kKvTile ? p.ps : kKvTile;
        uint32_t rp = 0;                                  // slots filled so far; FP8: key tiles of earlier pieces
        uint32_t raw[2] = {0, 0};                         // FP8: slots of keys and of values filled so far
        // Test hook for the bounded waits: before it copies anything, this warp waits on
        // a barrier that nothing completes.  Nor do products then begin; the other roles
        // wind down over the units at hand.
        bool ok = !p.test_stall || warp_wait(bars + C::kBarNever, 0, wc, lane);
        for (int k = 0; ok; ++k) {
            const ChunkUnit u = warp_unit(k);
            if (!__all_sync(0xffffffffu, u.b >= 0)) break;
            auto copy_tile = [&](int j, int entry, bool is_v) -> bool {
                const int key0 = (u.tile0 + j) * kKvTile;
                const int slot0 = p.ps < kKvTile ? 0 : p.ps_shift >= 0 ? key0 & (p.ps - 1) : key0 % p.ps;
                const bool mine = lane < 16 && page_copied(p, u, j, lane) &&
                                  (p.ps >= kKvTile || key0 + (lane + 1) * p.ps > u.lo);
                const unsigned who = __ballot_sync(0xffffffffu, mine);
                const uint32_t bytes = (uint32_t)(__popc(who) * box_rows * (KV8 ? 128 : 256));
                if constexpr (KV8) {
                    const uint32_t r = rp + j;
                    const int sl = r % C::kRawSlots + (is_v ? C::kRawSlots : 0);
                    if (!warp_wait(&raw_empty[sl], ((r / C::kRawSlots) & 1) ^ 1, wc, lane)) return false;
                    if (lane == 0) mbar_arrive_expect_tx(&raw_full[sl], bytes);
                    __syncwarp();
                    if (is_v) raw[1] = r + 1;
                    else raw[0] = r + 1;
                    if (mine)
                        tma_load_4d(smem_u32(smem + C::kOffRaw + sl * C::kChunkBytes + lane * box_rows * 128),
                                    is_v ? (const void *)&tm_v : (const void *)&tm_k, &raw_full[sl], 0, u.g, slot0, checked_page(p, entry));
                } else {
#pragma unroll
                    for (int s = 0; s < TS; ++s, ++rp) {
                        const int sl = rp % C::kSlots;
                        if (!warp_wait(&slot_empty[sl], ((rp / C::kSlots) & 1) ^ 1, wc, lane)) return false;
                        if (lane == 0) mbar_arrive_expect_tx(&slot_full[sl], bytes);
                        __syncwarp();
                        if (mine) {
                            const int phys = checked_page(p, entry);
                            const void *map = is_v ? (const void *)&tm_v : (const void *)&tm_k;
#pragma unroll
                            for (int c = 0; c < 2; ++c)
                                tma_load_4d(smem_u32(sRing + sl * C::kSlotBytes + c * C::kChunkBytes + lane * box_rows * 128), map,
                                            &slot_full[sl], s * 128 + c * 64, u.g, slot0, phys);
                        }
                    }
                }
                return true;
            };
            PageWindow table;
            table.open(p, u);
            if constexpr (NT == 2) {
                for (int j = 0; j < u.ntiles && ok; ++j) {
                    const int entry = table.at(p, u, j);
                    ok = copy_tile(j, entry, false) && copy_tile(j, entry, true);
                }
            } else {
                int entries[kSB];                         // of the tiles whose V copy is to come
#pragma unroll
                for (int j = 0; j < kSB; ++j) {
                    if (j >= u.ntiles || !ok) continue;
                    entries[j] = table.at(p, u, j);
                    ok = copy_tile(j, entries[j], false);
                }
                for (int j = 0; j < u.ntiles && ok; ++j) {
                    ok = copy_tile(j, entries[0], true);
#pragma unroll
                    for (int i = 0; i + 1 < kSB; ++i) entries[i] = entries[i + 1];
                    if (ok && j + kSB < u.ntiles) {
                        entries[kSB - 1] = table.at(p, u, j + kSB);
                        ok = copy_tile(j + kSB, entries[kSB - 1], false);
                    }
                }
            }
            if constexpr (KV8) rp += u.ntiles;
        }
        if (lane == 0) {
            // The copies land before the CTA leaves.
            auto drain = [&](uint64_t *full, uint32_t slots, uint32_t filled) {
                for (uint32_t i = 0; i < slots && i < filled; ++i) {
                    const uint32_t r = filled - 1 - i;
                    mbar_wait_drain(&full[r % slots], (r / slots) & 1, wc);
                }
            };
            if constexpr (KV8) {
                drain(raw_full, C::kRawSlots, raw[0]);
                drain(raw_full + C::kRawSlots, C::kRawSlots, raw[1]);
            } else {
                drain(slot_full, C::kSlots, rp);
            }
        }
        __syncwarp();
      } else if (warp < 3) {
        // ----------------------------------------------------------------- MMA
        if (lane == 0) {
            const int x = NT == 2 ? warp - 1 : 0;
            uint32_t rp = 0;                              // ring slots of earlier pieces
            uint32_t steps = 0;                           // this stream's key tiles of earlier pieces
            uint32_t turns = 0;                           // shared steps of earlier pieces (both streams present)
            const SDesc q_d = sdesc_sw128_split(smem_u32(sQ + x * C::kQBytes), 16, 1024);
            const SDesc k_d = sdesc_sw128_split(smem_u32(KV8 ? smem + C::kOffRaw : sRing), 16, 1024);
            const SDesc v_d = sdesc_sw128_split(smem_u32(sRing), C::kChunkBytes, 1024);
            auto wait_tile = [&](uint32_t r) -> bool {
#pragma unroll
                for (int s = 0; s < TS; ++s)
                    if (!mbar_wait(&slot_full[(r + s) % C::kSlots], ((r + s) / C::kSlots) & 1, wc)) return false;
                return true;
            };
            auto wait_keys = [&](uint32_t r) -> bool {
                if constexpr (KV8) return mbar_wait(&raw_full[r % C::kRawSlots], (r / C::kRawSlots) & 1, wc);
                return wait_tile(r);
            };
            auto wait_queries = [&](int k) -> bool {
                if constexpr (KV8) return mbar_wait(&q_ready[k % C::kQSets], (k / C::kQSets) & 1, wc);
                return mbar_wait(q_full, k & 1, wc);
            };
            auto release_tile = [&](uint32_t r) {
#pragma unroll
                for (int s = 0; s < TS; ++s) mma_commit(&slot_empty[(r + s) % C::kSlots]);
            };
            auto release_keys = [&](uint32_t r) {
                if constexpr (KV8) mma_commit(&raw_empty[r % C::kRawSlots]);
                else release_tile(r);
            };
            const uint32_t idesc_qk = C::kIdescQK | (p.scale_log2 < 0.f ? kIdescNegateA : 0u);
            auto push_qk = [&](uint32_t r, int buf) {
                if constexpr (KV8) {
                    const SDesc kd{k_d.lo + (r % C::kRawSlots) * (C::kChunkBytes >> 4), k_d.hi};
#pragma unroll
                    for (int term = 0; term < 2; ++term)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_f8_ss(tmem + C::s_col(x, buf), sdesc_at(q_d, term * C::kChunkBytes + kk * 32),
                                      sdesc_at(kd, kk * 32), idesc_qk, term + kk > 0 ? 1u : 0u);
                } else {
#pragma unroll
                    for (int s = 0; s < TS; ++s) {
                        const SDesc kd{k_d.lo + ((r + s) % C::kSlots) * (C::kSlotBytes >> 4), k_d.hi};
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk) {
                            const uint32_t off = (kk >> 2) * C::kChunkBytes + (kk & 3) * 32;
                            mma_bf16_ss(tmem + C::s_col(x, buf), sdesc_at(q_d, s * C::kSlotBytes + off), sdesc_at(kd, off),
                                        idesc_qk, s + kk > 0 ? 1u : 0u);
                        }
                    }
                }
            };
            // P of a key tile lies over the first 64 columns of its S buffer
            // (two BF16 a column); each half of 64 keys goes out as it comes.
            auto push_pv_half = [&](uint32_t r, int buf, int half, bool first) {
#pragma unroll
                for (int s = 0; s < TS; ++s) {
                    const SDesc vd{v_d.lo + ((r + s) % C::kSlots) * (C::kSlotBytes >> 4), v_d.hi};
#pragma unroll
                    for (int k4 = 0; k4 < 4; ++k4) {
                        const int kk = half * 4 + k4;
                        mma_bf16_ts(tmem + C::o_col(x) + s * 128, tmem + C::s_col(x, buf) + kk * 8,
                                    sdesc_at(vd, kk * 16 * 128), C::kIdescPV, (first && kk == 0) ? 0u : 1u);
                    }
                }
            };
            bool ok = true;
            for (int k = 0; ok; ++k) {
                const ChunkUnit *ur = wait_unit(k);
                const bool got = ur && ur->b >= 0;
                const int n = got ? ur->ntiles : 0;
                const int nrt = got ? ur->nrt : 0;
                free_unit(k);
                if (!got) break;
                const uint32_t r0 = rp;
                rp += (uint32_t)(n * C::kPerTile);
                auto rk = [&](int j) { return r0 + (uint32_t)(C::ring_k(j, n) * TS); };
                auto rv = [&](int j) { return r0 + (uint32_t)(C::ring_v(j, n) * TS); };
                if constexpr (NT == 1) {
                    // QK from one thread (warp 2), PV from the other: neither's waits hold up
                    // the other's products.  Each waits for the other's step first: what lay
                    // in the ring slot before its tile has then landed, as a parity wait
                    // needs (K_j comes at most kSB tiles before V_j, less than the ring).
                    if (warp == 2 && !wait_queries(k)) break;
                    for (int j = 0; j < n && ok; ++j) {
                        const uint32_t st = steps + j;
                        const int buf = st % kSB;
                        const uint32_t ph = (st / kSB) & 1;
                        if (warp == 2) {
                            // The buffer's last P has gone through the tensor core.
                            ok = (st < kSB || mbar_wait(&pv_done[buf], ph ^ 1, wc)) && wait_keys(rk(j));
                            if (!ok) break;
                            tc_fence_after();
                            push_qk(rk(j), buf);
                            mma_commit(&s_full[buf]);
                            release_keys(rk(j));
                            if (j == n - 1) mma_commit(q_empty);
                        } else {
                            ok = mbar_wait(&p_half[buf], ph, wc) && wait_tile(rv(j));
                            if (!ok) break;
                            tc_fence_after();
                            push_pv_half(rv(j), buf, 0, j == 0);
                            ok = mbar_wait(&p_full[buf], ph, wc);
                            if (!ok) break;
                            tc_fence_after();
                            push_pv_half(rv(j), buf, 1, false);
                            mma_commit(&pv_done[buf]);
                            release_tile(rv(j));
                        }
                    }
                    steps += n;
                } else {
                    if (!wait_queries(k)) break;
                    if (x >= nrt) {
                        // No row tile for this stream: it still sees every copy land and
                        // hands every slot back, so that its phases stay in step.
                        mbar_arrive(q_empty);
                        for (uint32_t r = r0; r < rp && ok; ++r) {
                            if constexpr (KV8) {
                                ok = wait_keys(r);
                                if (ok) mbar_arrive(&raw_empty[r % C::kRawSlots]);
                                if (!ok) break;
                            }
                            ok = mbar_wait(&slot_full[r % C::kSlots], (r / C::kSlots) & 1, wc);
                            if (ok) mbar_arrive(&slot_empty[r % C::kSlots]);
                        }
                        continue;
                    }
                    if (!wait_keys(rk(0))) break;
                    tc_fence_after();
                    push_qk(rk(0), 0);
                    mma_commit(&s_full[x]);
                    release_keys(rk(0));
                    if (n == 1) mma_commit(q_empty);
                    for (int j = 0; j < n && ok; ++j) {
                        const uint32_t ph = (steps + j) & 1;
                        if (nrt == 2) {
                            // Turns: stream 1 follows stream 0's step j, stream 0 stream 1's
                            // step j - 1, so that one's products run under the other's softmax.
                            // (Steps count on across pieces, so neither gets two phases ahead.)
                            const uint32_t dep = turns + j + x;
                            if (dep > 0 && !mbar_wait(&issued[1 - x], (dep - 1) & 1, wc)) { ok = false; break; }
                        }
                        // A wait between pushes lets the tensor pipe run dry: the tiles of the
                        // whole step first.  (K_{j+1} needs only older slots handed back.)
                        const bool next = j + 1 < n;
                        if (!wait_tile(rv(j)) || (next && !wait_keys(rk(j + 1))) || !mbar_wait(&p_half[x], ph, wc)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        push_pv_half(rv(j), 0, 0, j == 0);
                        if (!mbar_wait(&p_full[x], ph, wc)) { ok = false; break; }
                        tc_fence_after();
                        push_pv_half(rv(j), 0, 1, false);
                        // The turn goes over while this step's QK is still being pushed: the
                        // other issuer's waits overlap that, and its PV queues right behind.
                        if (nrt == 2) mbar_arrive(&issued[x]);
                        if (next) push_qk(rk(j + 1), 0);
                        else mma_commit(&pv_done[x]);
                        release_tile(rv(j));
                        if (next) {
                            mma_commit(&s_full[x]);
                            release_keys(rk(j + 1));
                            if (j + 2 == n) mma_commit(q_empty);
                        }
                    }
                    if (!ok) break;
                    steps += n;
                    if (nrt == 2) turns += n;
                }
            }
            mma_commit(&drain[warp - 1]);
            mbar_wait_drain(&drain[warp - 1], 0, wc);
        }
        __syncwarp();
      } else if (warp == 3) {
        // ----------------------------------------------- the pieces; queries
        ChunkWalk<NT> walk;
        walk.init(p, blockIdx.x, plan);
        for (int k = 0;; ++k) {
            ChunkUnit u;
            walk.next(p, u);
            const int sl = k % C::kSched;
            bool ok = warp_wait(&sched_empty[sl], ((k / C::kSched) & 1) ^ 1, wc, lane);
            if (ok && lane == 0) { sched[sl] = u; mbar_arrive(&sched_full[sl]); }
            __syncwarp();
            ok = ok && u.b >= 0 && warp_wait(q_empty, (k & 1) ^ 1, wc, lane);
            if (!ok) {
                // The copies land before the CTA leaves.
                if (lane == 0 && k > 0) mbar_wait_drain(q_full, (k - 1) & 1, wc);
                break;
            }
            if (lane == 0) {
                const uint32_t qrows = p.head_chunks > 1 ? 128u : (uint32_t)(p.G * p.tile_tokens);
                mbar_arrive_expect_tx(q_full, (uint32_t)u.nrt * (D / 64) * qrows * 128u);
                for (int x = 0; x < u.nrt; ++x) {
                    const int rt = u.rt0 + x;
                    int h0 = u.g * p.G, t0 = rt * p.tile_tokens;
                    if (p.head_chunks > 1) { t0 = rt / p.head_chunks; h0 += (rt - t0 * p.head_chunks) * 128; }
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
                        tma_load_3d(smem_u32(sQ + x * C::kQBytes + c * C::kChunkBytes), &tm_q, q_full, c * 64, h0, u.q0 + t0);
                }
            }
            __syncwarp();
        }
        if (lane == 0) p.cuts[blockIdx.x] = walk.cut;
        __syncwarp();
      }
    } else if (KV8 && warp >= 4 + 4 * NT) {
        if constexpr (KV8) {
            // ------------------------------------------------------ widening
            // A unit's queries first, into two E4M3 terms in place; then its values, from where
            // they landed to a slot that the products read.  Eight lanes take four 16-byte units
            // of two rows whose numbers differ in bits 0 and 2: their swizzled places then fall on
            // different banks, read and written.  (The barrier among them has no limit: they wait
            // together, and a wait that ran out does not part them.)
            if constexpr (NT == 2) setmaxnreg_dec<C::kRegsWiden>();
            const int r = (lane >> 3) ^ (lane & 4 ? 5 : 0), row0 = (warp & 3) * 32 + r, c = 2 * (lane & 3);
            const uint32_t from0 = row0 * 128 + (((lane & 3) ^ r) << 4);
            const uint32_t from1 = row0 * 128 + (((lane & 3) + 4) ^ r) * 16;
            const uint32_t to0 = row0 * 128 + ((c ^ r) << 4), to1 = row0 * 128 + (((c + 1) ^ r) << 4);
            auto put = [&](uint8_t *at, const uint4 &b) {
                const uint2 x0 = widen4_bf16(b.x), x1 = widen4_bf16(b.y), x2 = widen4_bf16(b.z), x3 = widen4_bf16(b.w);
                *reinterpret_cast<uint4 *>(at + to0) = make_uint4(x0.x, x0.y, x1.x, x1.y);
                *reinterpret_cast<uint4 *>(at + to1) = make_uint4(x2.x, x2.y, x3.x, x3.y);
            };
            uint32_t rp = 0;
            for (int k = 0;; ++k) {
                const ChunkUnit u = warp_unit(k);
                if (!named_bar_all(2, 128, u.b >= 0)) break;
                mbar_wait(q_full, k & 1, wc);
                __syncwarp();
                const int set = k % C::kQSets;
                for (int x = 0; x < u.nrt; ++x)
                    split_rows<C::kChunkBytes>(sQ + x * C::kQBytes, p.head_chunks > 1 ? 128 : p.G * p.tile_tokens, warp & 3, lane,
                                               [&](int r, int8_t e) { q_exp[(set * NT + x) * 128 + r] = e; });
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&q_ready[set]);
                for (int i = 0; i < u.ntiles; ++i, ++rp) {
                    const int rl = C::kRawSlots + rp % C::kRawSlots, sl = rp % C::kSlots;
                    // (Every lane waits: those that only hear of it from one that did may have read before.)
                    mbar_wait(&raw_full[rl], (rp / C::kRawSlots) & 1, wc);
                    mbar_wait(&slot_empty[sl], ((rp / C::kSlots) & 1) ^ 1, wc);
                    __syncwarp();
                    const uint8_t *from = smem + C::kOffRaw + rl * C::kChunkBytes;
                    uint8_t *at = sRing + sl * C::kSlotBytes;
#pragma unroll
                    for (int it = 0; it < 4; it += 2) {
                        const uint4 b0 = *reinterpret_cast<const uint4 *>(from + it * 1024 + from0);
                        const uint4 b1 = *reinterpret_cast<const uint4 *>(from + it * 1024 + from1);
                        const uint4 b2 = *reinterpret_cast<const uint4 *>(from + it * 1024 + 1024 + from0);
                        const uint4 b3 = *reinterpret_cast<const uint4 *>(from + it * 1024 + 1024 + from1);
                        put(at + it * 1024, b0);
                        put(at + C::kChunkBytes + it * 1024, b1);
                        put(at + it * 1024 + 1024, b2);
                        put(at + C::kChunkBytes + it * 1024 + 1024, b3);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) { mbar_arrive(&raw_empty[rl]); mbar_arrive(&slot_full[sl]); }
                }
            }
        }
    } else {
        if constexpr (NT == 2) {
            setmaxnreg_inc<C::kRegsSoftmax>();
        }
        // ------------------------------------------------- softmax / epilogue
        // The named barriers below have no limit, so the warps that share them never part:
        // a failed wait inside a unit does not change the control flow, and a unit that
        // not all of them see (a wait for its record ran out) is taken by none.
        const int x = (warp - 4) >> 2;
        const int q4 = warp & 3;
        const int row = q4 * 32 + lane;
        const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
        const float scale_all = fabsf(p.scale_log2);  // the MMA negates Q for a negative one
        auto wait_pv = [&](uint32_t step) { mbar_wait(&pv_done[x * kSB + step % kSB], (step / kSB) & 1, wc); };
        uint32_t steps = 0, pieces = 0, rp = 0;
        for (int k = 0;; ++k) {
            ChunkUnit u;
            float scale = scale_all;
            if constexpr (KV8) {
                // The row's exponent is read before the record goes back: the unit that
                // reuses its place cannot come before that.  (Bounded from below: a scale of
                // zero, or a small one times the 2^-126 of a row of zeros, would turn the -inf
                // of hidden keys into NaN.  Sums here stay below 2^24, so under the bound every
                // score is zero to the exponential.)
                const ChunkUnit *ur = wait_unit(k);
                u.b = -1;
                if (ur) u = *ur;
                const int set = k % C::kQSets;
                if (u.b >= 0) mbar_wait(&q_ready[set], (k / C::kQSets) & 1, wc);
                scale = fmaxf(scale * __int_as_float((127 - q_exp[(set * NT + x) * 128 + row]) << 23), 1e-37f);
                __syncwarp();
                if (lane == 0) free_unit(k);
            } else {
                u = warp_unit(k);
            }
            if (!(x == 0 ? named_bar_all(1, 128, u.b >= 0) : __all_sync(0xffffffffu, u.b >= 0) != 0)) break;
            const uint32_t r0 = rp;
            rp += (uint32_t)(u.ntiles * C::kPerTile);
            if (x >= u.nrt) continue;
            uint32_t *marks = bad + k % kBadUnits * kBadUnitWords;
            if (x == 0) {
                if (row < kBadUnitWords) marks[row] = 0;
                named_bar_sync(1, 128);
            }
            int t, h;
            const bool live = chunk_tile_row(p, u.rt0 + x, u.g, u.d, row, t, h);
            const bool warp_live = __any_sync(0xffffffffu, live);
            const int lo = live ? key_lo(p, u, t) : 0, hi = live ? key_hi(p, u, t) : 0;
            // Keys that every row of the unit sees, and that some row does: [all_lo, all_hi) and
            // [any_lo, any_hi).
            int t0 = u.rt0 * p.tile_tokens, t1 = min(u.d, (u.rt0 + u.nrt) * p.tile_tokens) - 1;
            if (p.head_chunks > 1) t0 = t1 = u.rt0 / p.head_chunks;
            const int all_lo = key_lo(p, u, t1), all_hi = key_hi(p, u, t0);
            const int any_lo = key_lo(p, u, t0), any_hi = key_hi(p, u, t1);
            float m_ref = kNegInf, l_sum = 0.f;
            for (int j = 0; j < u.ntiles; ++j, ++steps) {
                const int buf = steps % kSB;
                const int key0 = (u.tile0 + j) * kKvTile;
                const bool masked = key0 < all_lo || key0 + kKvTile > all_hi;
                // In such a tile stream 0 sees to the values, for both streams (stream 1's
                // product follows stream 0's).
                const bool values = masked && x == 0;
                uint32_t bits[4] = {0, 0, 0, 0};              // the keys this row sees
                if (masked) {
#pragma unroll
                    for (int w = 0; w < 4; ++w) bits[w] = range_bits(lo, hi, key0 + 32 * w);
                }
                mbar_wait(&s_full[x * kSB + buf], (steps / kSB) & 1, wc);
                tc_fence_after();
                if (warp_live) {                          // else rows of padding: whatever lies there
                    const uint32_t sa = tmem + lane_off + C::s_col(x, buf);
                    auto read_s = [&](int half, float *v) {
                        tmem_ld32(sa + half * 64, v);
                        tmem_ld32(sa + half * 64 + 32, v + 32);
                    };
                    auto hide = [&](int half, float *v) {
                        const uint32_t b0 = half == 0 ? bits[0] : bits[2], b1 = half == 0 ? bits[1] : bits[3];
#pragma unroll
                        for (int i = 0; i < 64; ++i)
                            if (!((i < 32 ? b0 : b1) >> (i & 31) & 1)) v[i] = kNegInf;
                    };
                    // Two streams read the row of S once.  One stream, and streams over FP8 caches,
                    // which have no registers for it (854 us for 768), read it twice, for its maximum
                    // and for P, 64 keys at a time in rolled loops, whose code stays small (unrolled
                    // 831 for 771; 32 keys at a time 804 for 761).
                    float sv[NT == 2 && !KV8 ? kKvTile : 1], ext = kNegInf;
                    if constexpr (NT == 2 && !KV8) {
                        read_s(0, sv);
                        read_s(1, sv + 64);
                        tmem_wait_ld();
                        if (masked) { hide(0, sv); hide(1, sv + 64); }
                        ext = max_of<kKvTile>(sv);
                    } else {
#pragma unroll 1
                        for (int half = 0; half < 2; ++half) {
                            float v[64];
                            read_s(half, v);
                            tmem_wait_ld();
                            if (masked) hide(half, v);
                            ext = fmaxf(ext, max_of<64>(v));
                        }
                    }
                    const float m_tile = live ? ext * scale : kNegInf;    // -inf when it sees none of these keys
                    const bool up = m_tile > m_ref + kRescaleSlack;   // also the first visible tile: m_ref = -inf
                    if (__any_sync(0xffffffffu, up)) {
                        float alpha = 1.f;
                        if (up) {
                            alpha = ex2_approx(m_ref - m_tile);
                            l_sum *= alpha;
                            m_ref = m_tile;
                        }
                        if (j > 0) {
                            // With one S buffer, S_j there means PV_{j-1} is done; with more
                            // it may still run.
                            if constexpr (kSB > 1) {
                                wait_pv(steps - 1);
                                tc_fence_after();
                            }
#pragma unroll 1
                            for (int c = 0; c < D / 32; ++c) {
                                float o[32];
                                const uint32_t oa = tmem + lane_off + C::o_col(x) + c * 32;
                                tmem_ld32(oa, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 32; ++i) o[i] *= alpha;
                                tmem_st32(oa, o);
                            }
                            tmem_wait_st();
                        }
                    }
                    // P = 2^(s * scale * log2 e - m_ref), rounded to BF16 (the MMA's A
                    // operand shares V's type); the row sum takes it unrounded.
                    const float mu = m_ref == kNegInf ? 0.f : m_ref;
                    uint64_t sum[4] = {0, 0, 0, 0};
                    auto put_half = [&](int half, float *v) {
                        uint32_t pk[32];
                        exp_64(v, scale, -mu, sum);
#pragma unroll
                        for (int i = 0; i < 64; i += 2) pk[i >> 1] = pack_bf16x2(v[i], v[i + 1]);
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            tmem_st16u(sa + half * 32 + c * 16, *reinterpret_cast<const uint32_t(*)[16]>(pk + c * 16));
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0 && !values) mbar_arrive(half == 0 ? &p_half[x * kSB + buf] : &p_full[x * kSB + buf]);
                    };
                    if constexpr (NT == 2 && !KV8) {
                        put_half(0, sv);
                        put_half(1, sv + 64);
                    } else {
#pragma unroll 1
                        for (int half = 0; half < 2; ++half) {
                            float v[64];
                            read_s(half, v);
                            tmem_wait_ld();
                            if (masked) hide(half, v);
                            put_half(half, v);
                        }
                    }
                    l_sum += sum_of(sum);
                }
                if (values) {
                    // Values of keys that nobody sees must not meet a zero weight: they may be
                    // NaN; nor those that are not finite the weights of rows that do not see
                    // them.  A thread looks after one key, when its row of P is done: the values
                    // have landed meanwhile.
                    const uint32_t r = r0 + (uint32_t)(C::ring_v(j, u.ntiles) * TS);      // (FP8: of widened values)
                    // A parity wait needs the slot's copy before V_j to have landed.
                    // S_j there proves that for all copies up to K_j; with two slots
                    // to a tile the one before V_j's may be V_{j-1}, which its
                    // finished product proves.
                    // So does that of V_{j-2} for two slots of widened values.
                    static_assert(TS == 2 || NT == 2 || KV8 || C::kSlots >= 2 * kSB, "the ring holds what QK runs ahead");
                    if constexpr (TS == 2) {
                        if (steps > 0) wait_pv(steps - 1);
                    }
                    if constexpr (KV8 && NT == 1) {
                        if (steps > 1) wait_pv(steps - 2);
                    }
                    const int key = key0 + row;
                    const bool seen = key >= any_lo && key < any_hi;
#pragma unroll 1
                    for (int s = 0; s < TS; ++s) {
                        const uint32_t sl = (r + s) % C::kSlots;
                        mbar_wait(&slot_full[sl], ((r + s) / C::kSlots) & 1, wc);
                        uint8_t *vr = sRing + sl * C::kSlotBytes + row * 128;
                        uint32_t wild = 0;                // an exponent of all ones carries into the sign's place
                        if (seen) {
#pragma unroll 1
                            for (int c = 0; c < 2; ++c)
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    const uint4 w = reinterpret_cast<const uint4 *>(vr + c * C::kChunkBytes)[i ^ (row & 7)];
                                    wild |= ((w.x & 0x7f807f80u) + 0x00800080u) | ((w.y & 0x7f807f80u) + 0x00800080u) |
                                            ((w.z & 0x7f807f80u) + 0x00800080u) | ((w.w & 0x7f807f80u) + 0x00800080u);
                                }
                            wild &= 0x80008000u;
                            if (wild) {
                                atomicOr(bad_words(marks, u.tile0 + j, any_lo, all_hi) + (row >> 5), 1u << (row & 31));
                                atomicOr(marks, 1u);
                            }
                        }
                        if (!seen || wild) {
#pragma unroll 1
                            for (int c = 0; c < 2; ++c)
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    reinterpret_cast<uint4 *>(vr + c * C::kChunkBytes)[i ^ (row & 7)] = make_uint4(0, 0, 0, 0);
                        }
                    }
                    fence_proxy_async_smem();
                }
                if (values || !warp_live) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) { mbar_arrive(&p_half[x * kSB + buf]); mbar_arrive(&p_full[x * kSB + buf]); }
                }
            }
            // ------------------------------------------------------ epilogue
            ++pieces;
            if constexpr (NT == 1) {
#pragma unroll
                for (int i = kSB; i >= 1; --i)
                    if (steps >= (uint32_t)i) wait_pv(steps - i);
            } else {
                mbar_wait(&pv_done[x], (pieces - 1) & 1, wc);
            }
            tc_fence_after();
            if (warp_live) {
                bool poison = false;
                if (__builtin_expect(*reinterpret_cast<volatile uint32_t *>(marks) != 0, 0)) {
#pragma unroll 1
                    for (int j = 0; j < u.ntiles; ++j) {
                        const int key0 = (u.tile0 + j) * kKvTile;
                        if (key0 >= all_lo && key0 + kKvTile <= all_hi) continue;
                        const uint32_t *words = bad_words(marks, u.tile0 + j, any_lo, all_hi);
                        for (int w = 0; w < 4; ++w) poison |= (words[w] & range_bits(lo, hi, key0 + 32 * w)) != 0;
                    }
                }
                write_row_at<D, NT>(p, u, x, row, live, (int64_t)(u.q0 + t) * p.out_stride[0] + h * p.out_stride[1],
                                    (int64_t)(u.q0 + t) * p.lse_stride[0] + h * p.lse_stride[1],
                                    m_ref, l_sum, live && poison,
                                    [&](int c, float (&o)[32]) {
                    tmem_ld32(tmem + lane_off + C::o_col(x) + c * 32, o);
                    tmem_wait_ld();
                });
            }
            tc_fence_before();
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// Merges the pieces of the units that CTA ranges cut, as the tree decode's merge does:
// with weighted sums o_i, row sums l_i and bases m_i, M = max m_i, out = sum 2^(m_i - M)
// o_i / sum 2^(m_i - M) l_i.  The pieces of the unit whose first one ended CTA c's range
// opened the following ranges.  Block (chunk, c) takes 32 rows of that unit, a lane a row
// and a warp an equal share of the columns, and turns the result round in shared memory.
// The rows of units that see no key are written here too.
// More threads have more pieces' loads on their way; two row tiles of 128 columns, whose
// blocks are the most, fit the GPU better in blocks of four warps (as the tree's).
template <int D, int NT>
constexpr int kMergeThreads = D == 128 && NT == 2 ? 128 : 256;

template <int D, int NT>
__global__ void __launch_bounds__(kMergeThreads<D, NT>) chunk_merge_kernel(const __grid_constant__ ChunkParams p) {
    constexpr int kThreads = kMergeThreads<D, NT>;
    constexpr int kUnits = D / 4 / (kThreads / 32);   // 16-byte FP32 units of a warp's columns
    constexpr int kPieces = 16 / kUnits;
    __shared__ uint4 stage[32][D / 8 + 1];           // BF16 rows
    __shared__ long long offset[32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // Zeros and -inf, a warp to a request; these wait for nothing.
    const int nwarps = gridDim.x * gridDim.y * (kThreads / 32);
    for (int b = (blockIdx.y * gridDim.x + blockIdx.x) * (kThreads / 32) + warp; b < p.B; b += nwarps) {
        const ChunkRow r = chunk_row<NT>(p, b);
        const int64_t empty = min((int64_t)r.d, (int64_t)r.v0 * step_tokens<NT>(p));
        for (int64_t i = lane; i < empty * p.Hq * (D / 8); i += 32) {
            const int64_t t = i / (p.Hq * (D / 8));
            const int c = (int)(i - t * (p.Hq * (D / 8)));
            reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(p.out) + (r.q0 + t) * p.out_stride[0] +
                                      (c / (D / 8)) * p.out_stride[1])[c % (D / 8)] = make_uint4(0, 0, 0, 0);
        }
        if (p.lse)
            for (int64_t i = lane; i < empty * p.Hq; i += 32) {
                const int64_t t = i / p.Hq;
                p.lse[(r.q0 + t) * p.lse_stride[0] + (i - t * p.Hq) * p.lse_stride[1]] = kNegInf;
            }
    }
    pdl_wait();                                      // the pieces are written
    const ChunkCut cut = p.cuts[blockIdx.y];
    const int x = blockIdx.x / 4, row = (blockIdx.x & 3) * 32 + lane;
    if (cut.count == 0 || x >= cut.nrt) return;
    int t, h;
    const bool live = chunk_tile_row(p, cut.rt0 + x, cut.g, cut.d, row, t, h);
    if (!__syncthreads_or(live)) return;
    const int step = p.ride ? p.Hkv : 1;
    auto slot = [&](int k) -> int64_t { return k == 0 ? 2 * blockIdx.y + 1 : 2 * (blockIdx.y + k * step); };
    float4 acc[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f, m = kNegInf;
    if (live) {
        for (int k0 = 0; k0 < cut.count; k0 += kPieces) {
            float2 ml[kPieces];
            float4 v[kPieces][kUnits];
#pragma unroll
            for (int k = 0; k < kPieces; ++k) {
                ml[k] = make_float2(kNegInf, 0.f);
                if (k0 + k >= cut.count) continue;
                const int64_t sl = slot(k0 + k);
                ml[k] = p.part_ml[sl * (NT * 128) + x * 128 + row];
#pragma unroll
                for (int i = 0; i < kUnits; ++i) v[k][i] = *part_unit<D, NT>(p, sl, warp * kUnits + i, x * 128 + row);
            }
            float mn = m;
#pragma unroll
            for (int k = 0; k < kPieces; ++k)
                if (ml[k].y != 0.f) mn = fmaxf(mn, ml[k].x);
            const float mu = mn == kNegInf ? 0.f : mn;       // nothing visible so far, or NaN scores alone
            const float alpha = ex2_approx(m - mu);
            m = mn;
            l *= alpha;
#pragma unroll
            for (int i = 0; i < kUnits; ++i) { acc[i].x *= alpha; acc[i].y *= alpha; acc[i].z *= alpha; acc[i].w *= alpha; }
#pragma unroll
            for (int k = 0; k < kPieces; ++k) {
                if (ml[k].y == 0.f) continue;
                const float w = ex2_approx(ml[k].x - mu);
                l = fmaf(w, ml[k].y, l);
#pragma unroll
                for (int i = 0; i < kUnits; ++i) {
                    acc[i].x = fmaf(w, v[k][i].x, acc[i].x);
                    acc[i].y = fmaf(w, v[k][i].y, acc[i].y);
                    acc[i].z = fmaf(w, v[k][i].z, acc[i].z);
                    acc[i].w = fmaf(w, v[k][i].w, acc[i].w);
                }
            }
        }
    }
    const float inv = l != 0.f ? p.out_scale / l : 0.f;
#pragma unroll
    for (int i = 0; i < kUnits; i += 2)
        stage[lane][(warp * kUnits + i) / 2] =
            make_uint4(pack_bf16x2(acc[i].x * inv, acc[i].y * inv), pack_bf16x2(acc[i].z * inv, acc[i].w * inv),
                       pack_bf16x2(acc[i + 1].x * inv, acc[i + 1].y * inv), pack_bf16x2(acc[i + 1].z * inv, acc[i + 1].w * inv));
    if (warp == 0) {
        offset[lane] = live ? (int64_t)(cut.q0 + t) * p.out_stride[0] + h * p.out_stride[1] : -1;
        if (live && p.lse)
            p.lse[(int64_t)(cut.q0 + t) * p.lse_stride[0] + h * p.lse_stride[1]] =
                l != 0.f ? (m + log2f(l)) * 0.69314718055994531f : kNegInf;
    }
    __syncthreads();
    for (int i = tid; i < 32 * (D / 8); i += kThreads) {
        const int r = i / (D / 8), c = i % (D / 8);
        if (offset[r] >= 0)
            reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(p.out) + offset[r])[c] = stage[r][c];
    }
}

template <int D, int NT, bool KV8>
cudaError_t launch_t(const ChunkParams &p, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                     cudaStream_t stream, int *launches) {
    using C = ChunkCfg<D, NT, KV8>;
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!configured[dev & 63]) {
        e = cudaFuncSetAttribute(chunk_kernel<D, NT, KV8>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
        if (e != cudaSuccess) return e;
        configured[dev & 63] = true;
    }
    chunk_kernel<D, NT, KV8><<<p.grid, C::kThreads, C::kSmemBytes, stream>>>(p, tq, tk, tv);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    ++*launches;
    e = launch_chunk_merge(p, stream);
    if (e != cudaSuccess) return e;
    ++*launches;
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_chunk_merge(const ChunkParams &p, cudaStream_t stream) {
    const dim3 grid(p.row_tiles * 4, p.workers);
    auto launch = [&](auto kernel, int threads) { return launch_after_previous(kernel, grid, dim3(threads), 0, stream, p); };
    if (p.D == 256 && p.row_tiles == 2) return launch(chunk_merge_kernel<256, 2>, kMergeThreads<256, 2>);
    if (p.D == 256) return launch(chunk_merge_kernel<256, 1>, kMergeThreads<256, 1>);
    if (p.row_tiles == 2) return launch(chunk_merge_kernel<128, 2>, kMergeThreads<128, 2>);
    return launch(chunk_merge_kernel<128, 1>, kMergeThreads<128, 1>);
}

// (A pair of CTAs has two pieces of two row tiles where two CTAs have four of one.)
size_t chunk_workspace_bytes(int head_dim, int grid) {
    const int rows = head_dim == 128 ? 256 : 128;
    return (size_t)grid * (2 * (size_t)rows * (head_dim * 4 + 8) + sizeof(ChunkCut));
}

void chunk_place_workspace(ChunkParams *p, void *ws) {
    const int64_t rows = p->D == 128 ? 256 : 128;
    char *at = static_cast<char *>(ws);
    p->part_o = reinterpret_cast<float *>(at);
    at += (int64_t)p->grid * 2 * rows * p->D * 4;
    p->part_ml = reinterpret_cast<float2 *>(at);
    at += (int64_t)p->grid * 2 * rows * 8;
    p->cuts = reinterpret_cast<ChunkCut *>(at);
}

cudaError_t launch_chunk(const ChunkParams &p, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                         cudaStream_t stream, int *launches) {
    *launches = 0;
    if (p.D == 256 && p.row_tiles == 2) return launch_chunk_pair(p, tq, tk, tv, stream, launches);
    if (p.D == 256) return launch_t<256, 1, false>(p, tq, tk, tv, stream, launches);
    if (p.kv8)
        return p.row_tiles == 2 ? launch_t<128, 2, true>(p, tq, tk, tv, stream, launches)
                                : launch_t<128, 1, true>(p, tq, tk, tv, stream, launches);
    return p.row_tiles == 2 ? launch_t<128, 2, false>(p, tq, tk, tv, stream, launches)
                            : launch_t<128, 1, false>(p, tq, tk, tv, stream, launches);
}

}  // namespace fw
