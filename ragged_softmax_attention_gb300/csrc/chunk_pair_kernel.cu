// Attention of chunks over a paged cache at head dim 256, sm_103a: pairs of CTAs.
//
// A unit is two row tiles, as at head dim 128, but S, O and the operands of 256 columns
// leave a CTA room for one: the tiles of a unit run on the two CTAs of a cluster, with
// tcgen05.mma.cta_group::2 issued by CTA 0 for both,
//   S [256 x 128]  = Q [256 x 256] * K_tile^T
//   O [256 x 256] += P [256 x 128] * V_tile
// Each CTA holds its own row tile and its 128 rows of S (two buffers) and O in TMEM; the
// B operands are split: CTA r copies keys 64 r .. 64 r + 63 of a K tile and columns 128 r
// .. 128 r + 127 of a V tile.  An SM so moves 64 KiB a step of 128 keys instead of 128
// KiB, which its share of L2 delivers in the 2,048 cycles of the step's products only
// just (a CTA by itself: 4,300 cycles a step).
//
// Measured (GB300): 200 .. 1,100 tokens on 1,024 .. 6,000 keys, 4 requests of 16/16 heads, 149 us
// (0.76 PFLOP/s, 41 % of DRAM; a CTA a row tile: 195), 2.7 units a pair, whose starts and uneven
// ends are what is left; with the next tiles fetched into L2 ahead 157.
//
// Both CTAs work out the same pieces, each for itself.  Copies of both complete on CTA 0's
// barriers, CTA 0's commits arrive on both CTAs'; P is handed over by CTA 0's four softmax
// warps and one thread of CTA 1, after its warps have met.  Values in tiles that some row
// does not see whole are looked after by the CTA that holds their columns, once the issuer
// has seen them land and said so; what is not finite is marked in both CTAs.  A mark stands
// in both before P of its tile is handed over (a fence at cluster scope behind it, on that
// path alone), so before that tile's product begins, and is read after a wait at cluster
// scope for the unit's last product: the case below as before, 149 us.  (An arrival of the
// issuer's at cluster scope for every unit that may have marks took 161.)
//
// Warp roles: warp 0 copies K and V halves, warp 1 of CTA 0 issues the MMAs, warp 3 works
// out the pieces and copies the queries, warps 4 .. 7 run the softmax.
#include "chunk_common.cuh"
#include "fw_pair.cuh"

namespace fw {
namespace {

using namespace chunk;

constexpr int D = 256, NT = 2;
constexpr int kThreads = 256;
constexpr int kSlots = 5;
constexpr int kSlotBytes = 32768;              // half a K tile (64 x 256) or half a V tile (128 x 128)
constexpr int kQBytes = 128 * D * 2;
constexpr int kOffRing = kQBytes;
constexpr int kOffBar = kOffRing + kSlots * kSlotBytes;
constexpr int kSched = 4;                      // unit records in flight
constexpr int kBarSlotFull = 0;                // CTA 0's count both CTAs' copies
constexpr int kBarSlotEmpty = kBarSlotFull + kSlots;
constexpr int kBarQFull = kBarSlotEmpty + kSlots;
constexpr int kBarQEmpty = kBarQFull + 1;
constexpr int kBarSFull = kBarQEmpty + 1;      // [2]
constexpr int kBarPFull = kBarSFull + 2;       // [2], CTA 0's: its 4 warps and one arrival of CTA 1
constexpr int kBarPvDone = kBarPFull + 2;      // [2]
constexpr int kBarValues = kBarPvDone + 2;     // the values of a tile to be looked at are there
constexpr int kBarDrain = kBarValues + 1;
constexpr int kBarSchedFull = kBarDrain + 1;
constexpr int kBarSchedEmpty = kBarSchedFull + kSched;
constexpr int kBarNever = kBarSchedEmpty + kSched;        // test hook: no thread ever arrives on it
constexpr int kNumBars = kBarNever + 1;
constexpr int kOffSched = (kOffBar + kNumBars * 8 + 63) / 64 * 64;
// Marks of eight units: a CTA writes its partner's too, and may be two steps, so two units,
// ahead of it or behind; a unit's words are cleared three units early.
constexpr int kMarkUnits = 8, kMarksAhead = 3;
constexpr int kOffBad = kOffSched + kSched * 64;
constexpr int kOffPlan = (kOffBad + kMarkUnits * kBadUnitWords * 4 + 15) / 16 * 16;
constexpr int kOffScan = kOffPlan + 32;        // [8] warp sums
constexpr int kOffMisc = kOffScan + 64;
constexpr int kSmemBytes = kOffMisc + 16 + 1024;
static_assert(kSmemBytes <= 232448, "shared memory budget of one CTA exceeded");
constexpr uint32_t kIdescQK = idesc_bf16_f32(256, 128, false, false);
constexpr uint32_t kIdescPV = idesc_bf16_f32(256, 256, false, true);
constexpr uint32_t kOCol = 256;                // TMEM: two S buffers of 128 columns, then O

__device__ __forceinline__ void or_cluster(uint32_t addr, uint32_t v) {
    asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ void fence_cluster() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
chunk_pair_kernel(const __grid_constant__ ChunkParams p, const __grid_constant__ CUtensorMap tm_q,
                  const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sQ = smem;
    uint8_t *sRing = smem + kOffRing;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kOffBar);
    uint64_t *slot_full = bars + kBarSlotFull;
    uint64_t *slot_empty = bars + kBarSlotEmpty;
    uint64_t *q_full = bars + kBarQFull;
    uint64_t *q_empty = bars + kBarQEmpty;
    uint64_t *s_full = bars + kBarSFull;
    uint64_t *p_full = bars + kBarPFull;
    uint64_t *pv_done = bars + kBarPvDone;
    uint64_t *values_there = bars + kBarValues;
    uint64_t *drain = bars + kBarDrain;
    uint64_t *sched_full = bars + kBarSchedFull;
    uint64_t *sched_empty = bars + kBarSchedEmpty;
    ChunkUnit *sched = reinterpret_cast<ChunkUnit *>(smem + kOffSched);
    uint32_t *bad = reinterpret_cast<uint32_t *>(smem + kOffBad);
    long long *plan = reinterpret_cast<long long *>(smem + kOffPlan);
    long long *scan = reinterpret_cast<long long *>(smem + kOffScan);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kOffMisc + 4);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();
    const int worker = blockIdx.x >> 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kSlots; ++i) { mbar_init(&slot_full[i], 1); mbar_init(&slot_empty[i], 1); }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int i = 0; i < 2; ++i) { mbar_init(&s_full[i], 1); mbar_init(&p_full[i], 5); mbar_init(&pv_done[i], 1); }
        mbar_init(values_there, 1);
        mbar_init(drain, 1);
        // Readers: the producer, four softmax warps, and in CTA 0 the issuer.
        for (int i = 0; i < kSched; ++i) { mbar_init(&sched_full[i], 1); mbar_init(&sched_empty[i], rank == 0 ? 6 : 5); }
        mbar_init(bars + kBarNever, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    for (int i = threadIdx.x; i < kMarkUnits * kBadUnitWords; i += kThreads) bad[i] = 0;
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tm_q); tma_prefetch_desc(&tm_k); tma_prefetch_desc(&tm_v);
    }
    if (warp == 1) { tmem_alloc_pair(tmem_slot, 512); tmem_relinquish_pair(); }
    pdl_launch_dependents();                       // the merge may take its place; it waits for this grid
    chunk_plan<NT>(p, worker, plan, scan);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();                            // both CTAs' barriers exist before any remote use
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const WaitCtx wc{p.status, p.timeout_ns, abort_flag};
    auto wait_unit = [&](int k) -> const ChunkUnit * {
        const int sl = k % kSched;
        return mbar_wait(&sched_full[sl], (k / kSched) & 1, wc) ? &sched[sl] : nullptr;
    };
    auto free_unit = [&](int k) { mbar_arrive(&sched_empty[k % kSched]); };
    // A unit record for a whole warp; b < 0 at the end.
    auto warp_unit = [&](int k) -> ChunkUnit {
        const ChunkUnit *ur = wait_unit(k);
        ChunkUnit u;
        u.b = -1;
        if (ur) u = *ur;
        __syncwarp();
        if (lane == 0) free_unit(k);
        __syncwarp();
        return u;
    };
    // Keys that every row of the unit sees, and that some row does: [all_lo, all_hi) and
    // [any_lo, any_hi).  A tile outside the first has its values looked after.
    struct Seen { int all_lo, all_hi, any_lo, any_hi; };
    auto seen_of = [&](const ChunkUnit &u) {
        int t0 = u.rt0 * p.tile_tokens, t1 = min(u.d, (u.rt0 + u.nrt) * p.tile_tokens) - 1;
        if (p.head_chunks > 1) t0 = t1 = u.rt0 / p.head_chunks;
        return Seen{key_lo(p, u, t1), key_hi(p, u, t0), key_lo(p, u, t0), key_hi(p, u, t1)};
    };
    auto masked_tile = [&](const Seen &s, int tile) {
        return tile * kKvTile < s.all_lo || tile * kKvTile + kKvTile > s.all_hi;
    };

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        const int krows = p.ps < 64 ? p.ps : 64, vrows = p.ps < kKvTile ? p.ps : kKvTile;
        uint32_t rp = 0;                                  // slots filled so far
        // Test hook for the bounded waits: before it copies anything, this warp waits on
        // a barrier that nothing completes.
        bool ok = !p.test_stall || warp_wait(bars + kBarNever, 0, wc, lane);
        for (int k = 0; ok; ++k) {
            const ChunkUnit u = warp_unit(k);
            if (!__all_sync(0xffffffffu, u.b >= 0)) break;
            // This CTA's half of K_j or V_j, as one ring item.  (CTA 0 announces both halves.)
            auto copy_half = [&](int j, int entry, bool is_v) -> bool {
                const int key0 = (u.tile0 + j) * kKvTile;
                const int slot0 = p.ps < kKvTile ? 0 : p.ps_shift >= 0 ? key0 & (p.ps - 1) : key0 % p.ps;
                const bool page = lane < 16 && page_copied(p, u, j, lane) &&
                                  (p.ps >= kKvTile || key0 + (lane + 1) * p.ps > u.lo);
                // Whether lane's page has keys of half h of a K tile that are to be copied.
                auto in_half = [&](int h) {
                    return page && (p.ps >= kKvTile ? key0 + 64 * h < u.n : (lane * p.ps) / 64 == h);
                };
                const unsigned both = __popc(__ballot_sync(0xffffffffu, page));
                const unsigned halves = __popc(__ballot_sync(0xffffffffu, in_half(0))) + __popc(__ballot_sync(0xffffffffu, in_half(1)));
                const bool mine = is_v ? page : in_half(rank);
                const int sl = rp % kSlots;
                if (!warp_wait(&slot_empty[sl], ((rp / kSlots) & 1) ^ 1, wc, lane)) return false;
                if (rank == 0 && lane == 0)
                    mbar_arrive_expect_tx(&slot_full[sl], is_v ? 2u * both * vrows * 256u : halves * krows * 512u);
                __syncwarp();
                if (mine) {
                    const int phys = checked_page(p, entry);
                    const uint32_t full0 = cluster_addr(&slot_full[sl], 0);
                    const uint32_t dst = smem_u32(sRing + sl * kSlotBytes);
                    if (is_v) {
#pragma unroll
                        for (int c = 0; c < 2; ++c)        // 128 keys x 64 columns
                            tma_load_4d_pair(dst + c * 128 * 128 + lane * vrows * 128, &tm_v, full0, rank * 128 + c * 64, u.g,
                                             slot0, phys);
                    } else {
                        const int at = p.ps >= 64 ? 0 : lane * p.ps - 64 * rank;
#pragma unroll
                        for (int c = 0; c < 4; ++c)        // 64 keys x 64 columns
                            tma_load_4d_pair(dst + c * 64 * 128 + at * 128, &tm_k, full0, c * 64, u.g,
                                             p.ps >= kKvTile ? slot0 + 64 * rank : 0, phys);
                    }
                }
                ++rp;
                return true;
            };
            PageWindow table;
            table.open(p, u);
            int entries[2];                               // of the tiles whose V copy is to come
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (j >= u.ntiles || !ok) continue;
                entries[j] = table.at(p, u, j);
                ok = copy_half(j, entries[j], false);
            }
            for (int j = 0; j < u.ntiles && ok; ++j) {
                ok = copy_half(j, entries[0], true);
                entries[0] = entries[1];
                if (ok && j + 2 < u.ntiles) {
                    entries[1] = table.at(p, u, j + 2);
                    ok = copy_half(j + 2, entries[1], false);
                }
            }
        }
        // CTA 0's phases complete once both CTAs' copies have landed; it waits for them
        // before the pair's last meeting, so neither CTA leaves with a copy in flight.
        if (rank == 0 && lane == 0) {
            for (uint32_t i = 0; i < (uint32_t)kSlots && i < rp; ++i) {
                const uint32_t r = rp - 1 - i;
                mbar_wait_drain(&slot_full[r % kSlots], (r / kSlots) & 1, wc);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // -------------------------------------------------- MMA (CTA 0 only)
        if (rank == 0 && lane == 0) {
            uint32_t rp = 0, qk = 0, pv = 0;              // ring items, products issued
            const SDesc q_d = sdesc_sw128_split(smem_u32(sQ), 16, 1024);
            const SDesc k_d = sdesc_sw128_split(smem_u32(sRing), 16, 1024);
            const SDesc v_d = sdesc_sw128_split(smem_u32(sRing), 128 * 128, 1024);
            const uint32_t idesc_qk = kIdescQK | (p.scale_log2 < 0.f ? kIdescNegateA : 0u);
            auto wait_slot = [&](uint32_t r) { return mbar_wait(&slot_full[r % kSlots], (r / kSlots) & 1, wc); };
            auto push_qk = [&](uint32_t r) {
                const SDesc kd{k_d.lo + (r % kSlots) * (kSlotBytes >> 4), k_d.hi};
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_pair_ss(tmem + (qk & 1u) * 128u, sdesc_at(q_d, (kk >> 2) * 128 * 128 + (kk & 3) * 32),
                                sdesc_at(kd, (kk >> 2) * 64 * 128 + (kk & 3) * 32), idesc_qk, kk > 0 ? 1u : 0u);
            };
            auto commit_qk = [&](uint32_t r) {
                mma_commit_pair(&s_full[qk & 1u]);
                ++qk;
                mma_commit_pair(&slot_empty[r % kSlots]);
            };
            // P sits over the first 64 columns of the tile's S buffer, two BF16 a column.
            auto push_pv = [&](uint32_t r, bool first) {
                const SDesc vd{v_d.lo + (r % kSlots) * (kSlotBytes >> 4), v_d.hi};
#pragma unroll
                for (int kk = 0; kk < kKvTile / 16; ++kk)
                    mma_pair_ts(tmem + kOCol, tmem + (pv & 1u) * 128u + kk * 8, sdesc_at(vd, kk * 16 * 128), kIdescPV,
                                (first && kk == 0) ? 0u : 1u);
            };
            bool ok = true;
            for (int k = 0; ok; ++k) {
                const ChunkUnit *ur = wait_unit(k);
                ChunkUnit u;
                u.b = -1;
                if (ur) u = *ur;
                free_unit(k);
                if (u.b < 0) break;
                const int n = u.ntiles;
                const Seen seen = seen_of(u);
                const uint32_t r0 = rp;
                rp += (uint32_t)(2 * n);
                auto rk = [&](int j) { return r0 + (uint32_t)pos_k<2>(j, n); };
                auto rv = [&](int j) { return r0 + (uint32_t)pos_v<2>(j, n); };
                if (!mbar_wait(q_full, k & 1, wc)) break;
                for (int j = 0; j < 2 && j < n && ok; ++j) {
                    ok = wait_slot(rk(j));
                    if (!ok) break;
                    tc_fence_after();
                    push_qk(rk(j));
                    commit_qk(rk(j));
                    if (j == n - 1) mma_commit_pair(q_empty);
                }
                for (int j = 0; j < n && ok; ++j) {
                    const bool next = j + 2 < n;
                    ok = wait_slot(rv(j));
                    if (!ok) break;
                    if (masked_tile(seen, u.tile0 + j)) {
                        mbar_arrive(values_there);
                        mbar_arrive_cluster(cluster_addr(values_there, 1));
                    }
                    ok = (!next || wait_slot(rk(j + 2))) && mbar_wait_cluster(&p_full[pv & 1u], (pv >> 1) & 1u, wc);
                    if (!ok) break;
                    tc_fence_after();
                    push_pv(rv(j), j == 0);
                    if (next) push_qk(rk(j + 2));
                    mma_commit_pair(&pv_done[pv & 1u]);
                    ++pv;
                    mma_commit_pair(&slot_empty[rv(j) % kSlots]);
                    if (next) {
                        commit_qk(rk(j + 2));
                        if (j + 2 == n - 1) mma_commit_pair(q_empty);
                    }
                }
            }
            // No MMA of the pair may still run when the pair frees TMEM.
            mma_commit_pair(drain);
            mbar_wait_drain(drain, 0, wc);
        }
        __syncwarp();
    } else if (warp == 3) {
        // ----------------------------------------------- the pieces; queries
        ChunkWalk<NT> walk;
        walk.init(p, worker, plan);
        const uint32_t q_full0 = cluster_addr(q_full, 0);
        for (int k = 0;; ++k) {
            ChunkUnit u;
            walk.next(p, u);
            const int sl = k % kSched;
            bool ok = warp_wait(&sched_empty[sl], ((k / kSched) & 1) ^ 1, wc, lane);
            if (ok && lane == 0) { sched[sl] = u; mbar_arrive(&sched_full[sl]); }
            __syncwarp();
            ok = ok && u.b >= 0 && warp_wait(q_empty, (k & 1) ^ 1, wc, lane);
            if (!ok) {
                // The copies land before the pair parts.
                if (rank == 0 && lane == 0 && k > 0) mbar_wait_drain(q_full, (k - 1) & 1, wc);
                break;
            }
            if (lane == 0) {
                const uint32_t qrows = p.head_chunks > 1 ? 128u : (uint32_t)(p.G * p.tile_tokens);
                if (rank == 0) mbar_arrive_expect_tx(q_full, 2u * (D / 64) * qrows * 128u);
                // (A CTA without a row tile takes its partner's: its rows are not written.)
                const int rt = u.rt0 + (rank < u.nrt ? rank : 0);
                int h0 = u.g * p.G, t0 = rt * p.tile_tokens;
                if (p.head_chunks > 1) { t0 = rt / p.head_chunks; h0 += (rt - t0 * p.head_chunks) * 128; }
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                    tma_load_3d_pair(smem_u32(sQ + c * 128 * 128), &tm_q, q_full0, c * 64, h0, u.q0 + t0);
            }
            __syncwarp();
        }
        if (rank == 0 && lane == 0) p.cuts[worker] = walk.cut;
        __syncwarp();
    } else if (warp >= 4) {
        // ------------------------------------------------- softmax / epilogue
        // The named barriers below have no limit, so the warps that share them never part:
        // a failed wait inside a unit does not change the control flow, and a unit that
        // not all of them see (a wait for its record ran out) is taken by none.
        const int q4 = warp & 3;
        const int row = q4 * 32 + lane;
        const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
        const float scale = fabsf(p.scale_log2);      // the MMA negates Q for a negative one
        const uint32_t p_full0[2] = {cluster_addr(&p_full[0], 0), cluster_addr(&p_full[1], 0)};
        auto wait_pv = [&](uint32_t i) { mbar_wait(&pv_done[i & 1u], (i >> 1) & 1u, wc); };
        uint32_t steps = 0, rp = 0, looks = 0;
        for (int k = 0;; ++k) {
            const ChunkUnit u = warp_unit(k);
            if (!named_bar_all(2, 128, u.b >= 0)) break;
            const uint32_t r0 = rp;
            rp += (uint32_t)(2 * u.ntiles);
            if (row < kBadUnitWords) bad[(k + kMarksAhead) % kMarkUnits * kBadUnitWords + row] = 0;
            uint32_t *marks = bad + k % kMarkUnits * kBadUnitWords;
            int t, h;
            const bool live = chunk_tile_row(p, u.rt0 + rank, u.g, u.d, row, t, h) && rank < u.nrt;
            const int lo = live ? key_lo(p, u, t) : 0, hi = live ? key_hi(p, u, t) : 0;
            const Seen seen = seen_of(u);
            float m_ref = kNegInf, l_sum = 0.f;
            for (int j = 0; j < u.ntiles; ++j, ++steps) {
                const uint32_t sb = steps & 1u;
                const int key0 = (u.tile0 + j) * kKvTile;
                const bool masked = masked_tile(seen, u.tile0 + j);
                uint32_t bits[4] = {0, 0, 0, 0};              // the keys this row sees
                if (masked) {
#pragma unroll
                    for (int w = 0; w < 4; ++w) bits[w] = range_bits(lo, hi, key0 + 32 * w);
                }
                mbar_wait(&s_full[sb], (steps >> 1) & 1u, wc);
                tc_fence_after();
                const uint32_t sa = tmem + lane_off + sb * 128u;
                float sv[kKvTile];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(sa + c * 32, sv + c * 32);
                tmem_wait_ld();
                if (masked) {
#pragma unroll
                    for (int i = 0; i < kKvTile; ++i)
                        if (!(bits[i >> 5] >> (i & 31) & 1)) sv[i] = kNegInf;
                }
                const float m_tile = live ? max_of<kKvTile>(sv) * scale : kNegInf;
                const bool up = m_tile > m_ref + kRescaleSlack;   // also the first visible tile: m_ref = -inf
                if (__any_sync(0xffffffffu, up)) {
                    float alpha = 1.f;
                    if (up) {
                        alpha = ex2_approx(m_ref - m_tile);
                        l_sum *= alpha;
                        m_ref = m_tile;
                    }
                    if (j > 0) {
                        wait_pv(steps - 1);
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            float o[32];
                            const uint32_t oa = tmem + lane_off + kOCol + c * 32;
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
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t pk[32];
                    exp_64(sv + half * 64, scale, -mu, sum);
#pragma unroll
                    for (int i = 0; i < 64; i += 2) pk[i >> 1] = pack_bf16x2(sv[half * 64 + i], sv[half * 64 + i + 1]);
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        tmem_st16u(sa + half * 32 + c * 16, *reinterpret_cast<const uint32_t(*)[16]>(pk + c * 16));
                }
                tmem_wait_st();
                l_sum += sum_of(sum);
                if (masked) {
                    // This CTA's columns of the values: those of keys that nobody sees are
                    // cleared, and so are those of a key with one that is not finite, which is
                    // marked.  A thread looks after one key, when its row of P is done.
                    mbar_wait_cluster(values_there, looks & 1u, wc);
                    ++looks;
                    const uint32_t sl = (r0 + (uint32_t)pos_v<2>(j, u.ntiles)) % kSlots;
                    const int key = key0 + row;
                    const bool some = key >= seen.any_lo && key < seen.any_hi;
                    uint8_t *vr = sRing + sl * kSlotBytes + row * 128;
                    uint32_t wild = 0;                    // an exponent of all ones carries into the sign's place
                    if (some) {
#pragma unroll 1
                        for (int c = 0; c < 2; ++c)
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const uint4 w = reinterpret_cast<const uint4 *>(vr + c * 128 * 128)[i ^ (row & 7)];
                                wild |= ((w.x & 0x7f807f80u) + 0x00800080u) | ((w.y & 0x7f807f80u) + 0x00800080u) |
                                        ((w.z & 0x7f807f80u) + 0x00800080u) | ((w.w & 0x7f807f80u) + 0x00800080u);
                            }
                        wild &= 0x80008000u;
                        if (wild) {
                            uint32_t *word = bad_words(marks, u.tile0 + j, seen.any_lo, seen.all_hi) + (row >> 5);
                            for (uint32_t cta = 0; cta < 2; ++cta) {
                                or_cluster(cluster_addr(word, cta), 1u << (row & 31));
                                or_cluster(cluster_addr(marks, cta), 1u);
                            }
                            fence_cluster();
                        }
                    }
                    if (!some || wild) {
#pragma unroll 1
                        for (int c = 0; c < 2; ++c)
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                reinterpret_cast<uint4 *>(vr + c * 128 * 128)[i ^ (row & 7)] = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                }
                tc_fence_before();
                __syncwarp();
                // One cluster-wide release a step from CTA 1, not four.
                if (rank == 0) {
                    if (lane == 0) mbar_arrive(&p_full[sb]);
                } else {
                    named_bar_sync(1, 128);
                    if (warp == 4 && lane == 0) mbar_arrive_cluster(p_full0[sb]);
                }
                __syncwarp();
            }
            // ------------------------------------------------------ epilogue
            mbar_wait_cluster(&pv_done[(steps - 1) & 1u], ((steps - 1) >> 1) & 1u, wc);      // the marks, too
            tc_fence_after();
            bool poison = false;
            if (__builtin_expect(*reinterpret_cast<volatile uint32_t *>(marks) != 0, 0)) {
#pragma unroll 1
                for (int j = 0; j < u.ntiles; ++j) {
                    if (!masked_tile(seen, u.tile0 + j)) continue;
                    const volatile uint32_t *words = bad_words(marks, u.tile0 + j, seen.any_lo, seen.all_hi);
                    for (int w = 0; w < 4; ++w) poison |= (words[w] & range_bits(lo, hi, (u.tile0 + j) * kKvTile + 32 * w)) != 0;
                }
            }
            if (rank < u.nrt)
                write_row_at<D, NT>(p, u, rank, row, live, (int64_t)(u.q0 + t) * p.out_stride[0] + h * p.out_stride[1],
                                    (int64_t)(u.q0 + t) * p.lse_stride[0] + h * p.lse_stride[1], m_ref, l_sum, live && poison,
                                    [&](int c, float (&o)[32]) {
                    tmem_ld32(tmem + lane_off + kOCol + c * 32, o);
                    tmem_wait_ld();
                });
            tc_fence_before();
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync_all();                            // no MMA, copy or remote arrival of the pair is left
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

}  // namespace

cudaError_t launch_chunk_pair(const ChunkParams &p, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                              cudaStream_t stream, int *launches) {
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!configured[dev & 63]) {
        e = cudaFuncSetAttribute(chunk_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
        if (e != cudaSuccess) return e;
        configured[dev & 63] = true;
    }
    chunk_pair_kernel<<<2 * p.workers, kThreads, kSmemBytes, stream>>>(p, tq, tk, tv);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    ++*launches;
    e = launch_chunk_merge(p, stream);
    if (e != cudaSuccess) return e;
    ++*launches;
    return cudaSuccess;
}

}  // namespace fw
