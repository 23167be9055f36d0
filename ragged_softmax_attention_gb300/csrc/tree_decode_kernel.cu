// Paged decode of a tree of drafted tokens, sm_103a: draft t of request b sees
// the committed keys 0 .. n - d - 1 and the drafts its mask row names.
//
// With d drafts of G query heads each, the rows that share a KV head's keys
// fill the MMA M axis (a decode of a few tokens, which puts the keys there,
// has too few): a row tile is up to 128 (draft, head) rows, whole drafts,
//   S [128 x 128]  = Q_tile * K_tile^T          (tcgen05, FP32 in TMEM)
//   O [128 x D]   += P [128 x 128] * V_tile      (tcgen05, P and O in TMEM)
// and one softmax thread owns one row, so maxima and sums need no exchange.
// A row tile costs 1,024 MMA cycles per 128-key tile at D = 128 whether it
// holds 8 rows or 128; an SM's share of HBM delivers such a K/V tile in ~2,700,
// so up to two row tiles per CTA the cache, not the products, sets the time.
//
// A unit is (request, KV head, up to NT row tiles); units are laid end to end
// in the order of their key tiles, each preceded by a few empty slots for the
// cost of starting it, and every CTA takes one equal contiguous range, so the
// partial results of a call take two slots per CTA whatever the batch: the
// piece a range begins with and the one it ends with.  Ranges follow from the
// lengths alone, and every CTA works them out for itself (a block-wide sum of
// the requests' slots), which saves a planning launch.
//
// Streams.  D = 128 with more than 128 rows: two row tiles, each with its own
// MMA-issuing thread, softmax warpgroup, S buffer and O, take turns on the
// tensor core while they share every K/V load (NT = 2).  Otherwise one row
// tile with three S buffers (two at D = 256): the products of the next key tiles
// run under the softmax of this one (NT = 1).
//
// Measured (GB300, GPU time of the two launches, `of copy` against a measured
// 6,782 GB/s): 16 requests of 512 .. 8,192 keys, 16 drafts of 40/8 heads (NT = 1)
// 279 MB in 56 us, 0.74 of copy: inside a piece HBM is the bound, the rest is the
// first tile's way (6 us), uneven ends and the merge.  Head dim 256, 8 requests, 24
// drafts of 16/16 heads: 512 MB in 99 us, 0.76.  64 requests of up to 32,768 keys, 32
// drafts (NT = 2): 4.84 GB in 860 .. 955 us by machine, 0.75 .. 0.83; a step takes
// 3,060 cycles, the chain S, softmax (1,390), PV, next QK of two streams in turn,
// where HBM's share is 2,700.  16 requests with 121 drafts of 32/8 heads (NT = 2):
// 134 GFLOP in 128 us, 1.05 PFLOP/s: the same chain takes 95 us of it, the first
// scores 8, pieces' ends 10, the last CTA and the merge 14.
//
// Warp roles: warp 0 copies (Q, then K and V tiles through a ring of 32 KiB
// slots in the order the MMAs take them), warps 1 and 2 issue the MMAs (of a
// stream each, or of QK and PV),
// warp 3 works out the pieces and copies the queries, warps 4.. run the softmax.
#include "tree_common.cuh"

namespace fw {
namespace {

using namespace tree;

template <int D_, int NT_>
struct TreeCfg {
    static constexpr int D = D_, NT = NT_;
    // S buffers of a stream, i.e. key tiles QK runs ahead: what O leaves of TMEM.
    static constexpr int kSB = NT == 2 ? 1 : D == 128 ? 3 : 2;
    static constexpr int kTileSlots = D / 128;                  // ring slots of one K or V tile
    static constexpr int kChunkBytes = 128 * 128;               // 128 rows x 64 bf16 columns
    static constexpr int kSlotBytes = 2 * kChunkBytes;          // 128 rows x 128 columns
    static constexpr int kQBytes = 128 * D * 2;
    static constexpr int kSlots = (229376 - NT * kQBytes) / kSlotBytes;
    static constexpr int kOffQ = 0;
    static constexpr int kOffRing = NT * kQBytes;
    static constexpr int kOffBar = kOffRing + kSlots * kSlotBytes;
    static constexpr int kSched = 4;                            // unit records in flight
    static constexpr int kBarSlotFull = 0;
    static constexpr int kBarSlotEmpty = kBarSlotFull + kSlots;
    static constexpr int kBarQFull = kBarSlotEmpty + kSlots;
    static constexpr int kBarQEmpty = kBarQFull + 1;
    static constexpr int kBarSFull = kBarQEmpty + 1;            // [NT][kSB]
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
    static constexpr int kOffSeen = kOffSched + kSched * 64;    // [2][4 warps][4 words]
    static constexpr int kOffBad = kOffSeen + 128;              // drafts whose values are not finite
    static constexpr int kOffPlan = kOffBad + kBadUnits * kBadWords * 4;        // long long: total, start of row b0; int b0
    static constexpr int kOffScan = kOffPlan + 32;              // [12] warp sums
    static constexpr int kOffMisc = kOffScan + 96;
    static constexpr int kSmemBytes = kOffMisc + 16 + 1024;
    static_assert(kSmemBytes <= 232448, "shared memory budget of one CTA exceeded");
    static constexpr int kThreads = 128 + NT * 128;
    static constexpr int kSchedReaders = 3 + 4 * NT;            // issuers, the producer, softmax warps
    // NT = 2: 384 threads launched at 168 registers; 128 x 80 + 256 x 208 = 63488 <= 64512.
    static constexpr uint32_t kRegsControl = 80, kRegsSoftmax = 208;
    static_assert(NT == 1 || 128 * kRegsControl + 256 * kRegsSoftmax <= 384 * 168, "register split");
    static constexpr uint32_t kIdescQK = idesc_bf16_f32(128, kKvTile, false, false);
    static constexpr uint32_t kIdescPV = idesc_bf16_f32(128, 128, false, true);
    __device__ static constexpr uint32_t s_col(int x, int buf) { return (uint32_t)(x * kSB + buf) * 128u; }
    __device__ static constexpr uint32_t o_col(int x) { return (uint32_t)(NT * kSB + x) * 128u; }
};

template <int D, int NT>
__global__ void __launch_bounds__(TreeCfg<D, NT>::kThreads, 1)
tree_decode_kernel(const __grid_constant__ TreeParams p, const __grid_constant__ CUtensorMap tm_q,
                   const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
    using C = TreeCfg<D, NT>;
    constexpr int kSB = C::kSB, TS = C::kTileSlots;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sQ = smem + C::kOffQ;
    uint8_t *sRing = smem + C::kOffRing;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
    uint64_t *slot_full = bars + C::kBarSlotFull;
    uint64_t *slot_empty = bars + C::kBarSlotEmpty;
    uint64_t *q_full = bars + C::kBarQFull;
    uint64_t *q_empty = bars + C::kBarQEmpty;
    uint64_t *s_full = bars + C::kBarSFull;
    uint64_t *p_half = bars + C::kBarPHalf;
    uint64_t *p_full = bars + C::kBarPFull;
    uint64_t *pv_done = bars + C::kBarPvDone;
    uint64_t *issued = bars + C::kBarIssued;
    uint64_t *drain = bars + C::kBarDrain;
    uint64_t *sched_full = bars + C::kBarSchedFull;
    uint64_t *sched_empty = bars + C::kBarSchedEmpty;
    TreeUnit *sched = reinterpret_cast<TreeUnit *>(smem + C::kOffSched);
    uint32_t *seen_words = reinterpret_cast<uint32_t *>(smem + C::kOffSeen);
    uint32_t *bad = reinterpret_cast<uint32_t *>(smem + C::kOffBad);
    long long *plan = reinterpret_cast<long long *>(smem + C::kOffPlan);
    long long *scan = reinterpret_cast<long long *>(smem + C::kOffScan);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kOffMisc + 4);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kSlots; ++i) { mbar_init(&slot_full[i], 1); mbar_init(&slot_empty[i], NT); }
        mbar_init(q_full, 1);
        mbar_init(q_empty, NT);
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
    plan_range<NT>(p, plan, scan);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const WaitCtx wc{p.status, p.timeout_ns, abort_flag};
    auto wait_unit = [&](int k) -> const TreeUnit * {
        const int sl = k % C::kSched;
        return mbar_wait(&sched_full[sl], (k / C::kSched) & 1, wc) ? &sched[sl] : nullptr;
    };
    auto free_unit = [&](int k) { mbar_arrive(&sched_empty[k % C::kSched]); };

    if (warp < 4) {
      if constexpr (NT == 2) setmaxnreg_dec<C::kRegsControl>();
      if (warp == 0) {
        // ------------------------------------------------------------ producer
        const int box_rows = p.ps < kKvTile ? p.ps : kKvTile;
        uint32_t rp = 0;                                  // ring slots filled so far
        // Test hook for the bounded waits: before it copies anything, this warp waits on
        // a barrier that nothing completes.  Nor do products then begin; the other roles
        // wind down over the units at hand.
        bool ok = !p.test_stall || warp_wait(bars + C::kBarNever, 0, wc, lane);
        for (int k = 0; ok; ++k) {
            const TreeUnit *ur = wait_unit(k);
            TreeUnit u;
            u.b = -1;
            if (ur) u = *ur;
            __syncwarp();
            if (lane == 0) free_unit(k);
            if (!__all_sync(0xffffffffu, u.b >= 0)) break;
            // ---- K and V tiles in the order the MMAs take them
            auto copy_tile = [&](int j, int entry, bool is_v) -> bool {
                const int key0 = (u.tile0 + j) * kKvTile;
                const int slot0 = p.ps < kKvTile ? 0 : p.ps_shift >= 0 ? key0 & (p.ps - 1) : key0 % p.ps;
                const bool mine = lane < 16 && page_copied(p, u, j, lane);
                const unsigned who = __ballot_sync(0xffffffffu, mine);
                const uint32_t bytes = (uint32_t)(__popc(who) * box_rows * 256);
#pragma unroll
                for (int s = 0; s < TS; ++s, ++rp) {
                    const int sl = rp % C::kSlots;
                    if (!warp_wait(&slot_empty[sl], ((rp / C::kSlots) & 1) ^ 1, wc, lane)) return false;
                    if (lane == 0) mbar_arrive_expect_tx(&slot_full[sl], bytes);
                    __syncwarp();
                    if (mine) {
                        const int phys = checked_page(p, entry);
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            tma_load_4d(smem_u32(sRing + sl * C::kSlotBytes + c * C::kChunkBytes + lane * box_rows * 128),
                                        is_v ? (const void *)&tm_v : (const void *)&tm_k, &slot_full[sl],
                                        s * 128 + c * 64, u.g, slot0, phys);
                    }
                }
                return true;
            };
            PageWindow table;
            table.open(p, u);
            int entries[kSB];                             // of the tiles whose V copy is to come
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
        if (lane == 0) {
            for (uint32_t i = 0; i < (uint32_t)C::kSlots && i < rp; ++i) {
                const uint32_t r = rp - 1 - i;
                mbar_wait_drain(&slot_full[r % C::kSlots], (r / C::kSlots) & 1, wc);
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
            const SDesc k_d = sdesc_sw128_split(smem_u32(sRing), 16, 1024);
            const SDesc v_d = sdesc_sw128_split(smem_u32(sRing), C::kChunkBytes, 1024);
            auto wait_tile = [&](uint32_t r) -> bool {
#pragma unroll
                for (int s = 0; s < TS; ++s)
                    if (!mbar_wait(&slot_full[(r + s) % C::kSlots], ((r + s) / C::kSlots) & 1, wc)) return false;
                return true;
            };
            auto tile_there = [&](uint32_t r) -> bool {
                bool there = true;
#pragma unroll
                for (int s = 0; s < TS; ++s)
                    there &= mbar_try_wait(smem_u32(&slot_full[(r + s) % C::kSlots]), ((r + s) / C::kSlots) & 1);
                return there;
            };
            auto release_tile = [&](uint32_t r) {
#pragma unroll
                for (int s = 0; s < TS; ++s) mma_commit(&slot_empty[(r + s) % C::kSlots]);
            };
            const uint32_t idesc_qk = C::kIdescQK | (p.scale_log2 < 0.f ? kIdescNegateA : 0u);
            auto push_qk = [&](uint32_t r, int buf) {
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
            if constexpr (NT == 1) {
                // QK and PV from a thread each: neither's waits hold up the other's
                // products (one thread for both spent 2,200 cycles a key tile, 1,024 of
                // them on products).  Each waits for the other's step first: what lay
                // in the ring slot before its tile has then landed, as a parity wait
                // needs (K_j comes at most kSB tiles before V_j, less than the ring).
                for (int k = 0; ok; ++k) {
                    const TreeUnit *ur = wait_unit(k);
                    const bool got = ur && ur->b >= 0;
                    const int n = got ? ur->ntiles : 0;
                    free_unit(k);
                    if (!got) break;
                    const uint32_t r0 = rp;
                    rp += (uint32_t)(2 * n * TS);
                    if (warp == 2 && !mbar_wait(q_full, k & 1, wc)) break;
                    for (int j = 0; j < n && ok; ++j) {
                        const uint32_t st = steps + j;
                        const int buf = st % kSB;
                        const uint32_t ph = (st / kSB) & 1;
                        if (warp == 2) {
                            const uint32_t r = r0 + (uint32_t)(pos_k<kSB>(j, n) * TS);
                            // The buffer's last P has gone through the tensor core.
                            ok = (st < kSB || mbar_wait(&pv_done[buf], ph ^ 1, wc)) && wait_tile(r);
                            if (!ok) break;
                            tc_fence_after();
                            push_qk(r, buf);
                            mma_commit(&s_full[buf]);
                            release_tile(r);
                            if (j == n - 1) mma_commit(q_empty);
                        } else {
                            const uint32_t r = r0 + (uint32_t)(pos_v<kSB>(j, n) * TS);
                            ok = mbar_wait(&p_half[buf], ph, wc) && wait_tile(r);
                            if (!ok) break;
                            tc_fence_after();
                            push_pv_half(r, buf, 0, j == 0);
                            ok = mbar_wait(&p_full[buf], ph, wc);
                            if (!ok) break;
                            tc_fence_after();
                            push_pv_half(r, buf, 1, false);
                            mma_commit(&pv_done[buf]);
                            release_tile(r);
                        }
                    }
                    steps += n;
                }
            } else {
                for (int k = 0; ok; ++k) {
                    const TreeUnit *ur = wait_unit(k);
                    const bool got = ur && ur->b >= 0;
                    const int n = got ? ur->ntiles : 0;
                    const int nrt = got ? ur->nrt : 0;
                    free_unit(k);
                    if (!got) break;
                    const uint32_t r0 = rp;
                    rp += (uint32_t)(2 * n * TS);
                    if (!mbar_wait(q_full, k & 1, wc)) break;
                    if (x >= nrt) {
                        // No row tile for this stream: it still sees every copy land and
                        // hands every slot back, so that its phases stay in step.
                        mbar_arrive(q_empty);
                        for (uint32_t r = r0; r < rp && ok; ++r) {
                            ok = mbar_wait(&slot_full[r % C::kSlots], (r / C::kSlots) & 1, wc);
                            if (ok) mbar_arrive(&slot_empty[r % C::kSlots]);
                        }
                        continue;
                    }
                    tc_fence_after();
                    auto rk = [&](int j) { return r0 + (uint32_t)(pos_k<kSB>(j, n) * TS); };
                    auto rv = [&](int j) { return r0 + (uint32_t)(pos_v<kSB>(j, n) * TS); };
                    for (int j = 0; j < kSB && j < n && ok; ++j) {
                        ok = wait_tile(rk(j));
                        if (!ok) break;
                        tc_fence_after();
                        push_qk(rk(j), (steps + j) % kSB);
                        mma_commit(&s_full[x * kSB + (steps + j) % kSB]);
                        release_tile(rk(j));
                        if (j == n - 1) mma_commit(q_empty);
                    }
                    for (int j = 0; j < n && ok; ++j) {
                        const uint32_t st = steps + j;
                        const int buf = st % kSB;
                        const uint32_t ph = (st / kSB) & 1;
                        if (nrt == 2) {
                            // Turns: stream 1 follows stream 0's step j, stream 0 stream 1's
                            // step j - 1, so that one's products run under the other's softmax.
                            // (Steps count on across pieces, so neither gets two phases ahead.)
                            const uint32_t dep = turns + j + x;
                            if (dep > 0 && !mbar_wait(&issued[1 - x], (dep - 1) & 1, wc)) { ok = false; break; }
                        }
                        if (!wait_tile(rv(j)) || !mbar_wait(&p_half[x * kSB + buf], ph, wc)) { ok = false; break; }
                        const bool next = j + kSB < n;
                        const bool paired = next && tile_there(rk(j + kSB));
                        tc_fence_after();
                        push_pv_half(rv(j), buf, 0, j == 0);
                        if (!mbar_wait(&p_full[x * kSB + buf], ph, wc)) { ok = false; break; }
                        tc_fence_after();
                        push_pv_half(rv(j), buf, 1, false);
                        if (nrt == 2) mbar_arrive(&issued[x]);
                        // With the next K tile there, its product goes straight behind
                        // (a wait between pushes lets the tensor pipe run dry); else
                        // this tile's V is handed back first.
                        if (paired) push_qk(rk(j + kSB), buf);
                        if (j == n - 1) mma_commit(&pv_done[x]);
                        release_tile(rv(j));
                        if (next) {
                            if (!paired) {
                                if (!wait_tile(rk(j + kSB))) { ok = false; break; }
                                tc_fence_after();
                                push_qk(rk(j + kSB), buf);
                            }
                            mma_commit(&s_full[x * kSB + buf]);
                            release_tile(rk(j + kSB));
                            if (j + kSB == n - 1) mma_commit(q_empty);
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
        // A warp of their own: the next piece is worked out, and its keys copied,
        // while this one's products run.  (Where the copying warp did it, a piece's
        // end cost 10,000 cycles, most of them for instructions gone from the cache.)
        TreeWalk<NT> walk;
        walk.init(p, plan);
        for (int k = 0;; ++k) {
            TreeUnit u;
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
            if (lane == 0) copy_queries<D, NT>(p, u, tm_q, sQ, C::kQBytes, C::kChunkBytes, q_full);
            __syncwarp();
        }
        if (lane == 0) p.cuts[blockIdx.x] = walk.cut;
        __syncwarp();
      }
    } else {
        if constexpr (NT == 2) setmaxnreg_inc<C::kRegsSoftmax>();
        // ------------------------------------------------- softmax / epilogue
        // The named barriers below have no limit, so the warps that share them never part:
        // a failed wait inside a unit does not change the control flow, and a unit that
        // not all of them see (a wait for its record ran out) is taken by none.
        const int x = (warp - 4) >> 2;
        const int q4 = warp & 3;
        const int row = q4 * 32 + lane;
        const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
        const float scale = fabsf(p.scale_log2);      // the MMA negates Q for a negative one
        // PV of step i completes phase i / kSB of its S buffer's barrier.  (One barrier
        // for all steps could be a phase behind or a phase ahead of a wait, which a
        // parity does not tell apart.)
        auto wait_pv = [&](uint32_t step) { mbar_wait(&pv_done[x * kSB + step % kSB], (step / kSB) & 1, wc); };
        uint32_t steps = 0, pieces = 0, rp = 0;
        for (int k = 0;; ++k) {
            const TreeUnit *ur = wait_unit(k);
            TreeUnit u;
            u.b = -1;
            if (ur) u = *ur;
            __syncwarp();
            if (lane == 0) free_unit(k);
            if (!(x == 0 ? named_bar_all(1, 128, u.b >= 0) : __all_sync(0xffffffffu, u.b >= 0) != 0)) break;
            const uint32_t r0 = rp;
            rp += (uint32_t)(2 * u.ntiles * TS);
            if (x >= u.nrt) continue;
            if (x == 0 && row < kBadWords) bad[k % kBadUnits * kBadWords + row] = 0;
            int t, h;
            const bool live = tree_tile_row(p, u.rt0 + x, u.g, u.d, row, t, h);
            const bool warp_live = __any_sync(0xffffffffu, live);
            const int base = u.n - u.d;                   // committed keys
            const int32_t *mrow = p.mask + u.b * p.mask_stride[0] + (live ? t : 0) * p.mask_stride[1];
            float m_ref = kNegInf, l_sum = 0.f;
            for (int j = 0; j < u.ntiles; ++j, ++steps) {
                const int buf = steps % kSB;
                const int key0 = (u.tile0 + j) * kKvTile;
                const bool drafts = key0 + kKvTile > base;    // the tile reaches past the committed keys
                // What the masks say of the tile is worked out while its scores are (131 us
                // against 134 at 242 rows).
                // With drafts in the tile, stream 0 sees to its values, for both streams
                // (stream 1's product follows stream 0's).
                const bool values = drafts && x == 0;
                uint32_t mine = 0;                            // this warp's keys that somebody sees
                uint32_t bits[4] = {0, 0, 0, 0};              // the keys this row sees
                if (drafts) {
                    if (x == 0) {
                        uint32_t *words = seen_words + (j & 1) * 16;
                        seen_keys(p, u, key0, row, 1, words);
                        mine = seen_word(words, q4);
                    }
#pragma unroll
                    for (int w = 0; w < 4; ++w) bits[w] = live ? draft_bits(mrow, key0 + 32 * w - base, u.d) : 0u;
                }
                mbar_wait(&s_full[x * kSB + buf], (steps / kSB) & 1, wc);
                tc_fence_after();
                if (warp_live) {                          // else rows of padding: whatever lies there
                    const uint32_t sa = tmem + lane_off + C::s_col(x, buf);
                    // One stream: the row of S is read twice, for its maximum and for P, 64 keys
                    // at a time in rolled loops, whose code stays small (dim 256: two us of 100
                    // less; dim 128 the same).  Two streams hide less and read it once (130 us
                    // against 142 for 121-draft trees).
                    auto read_s = [&](int half, float *v) {
                        tmem_ld32(sa + half * 64, v);
                        tmem_ld32(sa + half * 64 + 32, v + 32);
                    };
                    auto hide = [&](int half, float *v) {
                        const uint32_t lo = half == 0 ? bits[0] : bits[2], hi = half == 0 ? bits[1] : bits[3];
#pragma unroll
                        for (int i = 0; i < 64; ++i)
                            if (!((i < 32 ? lo : hi) >> (i & 31) & 1)) v[i] = kNegInf;
                    };
                    float sv[NT == 2 ? kKvTile : 1], ext = kNegInf;
                    if constexpr (NT == 2) {
                        read_s(0, sv);
                        read_s(1, sv + 64);
                        tmem_wait_ld();
                        if (drafts) { hide(0, sv); hide(1, sv + 64); }
                        ext = max_of<kKvTile>(sv);
                    } else {
#pragma unroll 1
                        for (int half = 0; half < 2; ++half) {
                            float v[64];
                            read_s(half, v);
                            tmem_wait_ld();
                            if (drafts) hide(half, v);
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
                    if constexpr (NT == 2) {
                        put_half(0, sv);
                        put_half(1, sv + 64);
                    } else {
#pragma unroll 1
                        for (int half = 0; half < 2; ++half) {
                            float v[64];
                            read_s(half, v);
                            tmem_wait_ld();
                            if (drafts) hide(half, v);
                            put_half(half, v);
                        }
                    }
                    l_sum += sum_of(sum);
                }
                if (values) {
                    // Values of keys nobody sees must not meet a zero weight: they may be
                    // NaN; nor a draft's that are not finite the weights of rows that do
                    // not see it.  A thread looks after one key, when its row of P is done:
                    // the values have landed meanwhile.  (Before it: 106 us against 99 at dim 256;
                    // by the copying warp 130.)
                    const uint32_t r = r0 + (uint32_t)(pos_v<kSB>(j, u.ntiles) * TS);
                    // A parity wait needs the slot's copy before V_j to have landed.
                    // S_j there proves that for all copies up to K_j; with two slots
                    // to a tile the one before V_j's may be V_{j-1}, which its
                    // finished product proves.
                    if constexpr (TS == 2) {
                        if (steps > 0) wait_pv(steps - 1);
                    }
                    const bool seen = mine >> lane & 1;
                    const int draft = key0 + row - base;
#pragma unroll 1
                    for (int s = 0; s < TS; ++s) {
                        const uint32_t sl = (r + s) % C::kSlots;
                        mbar_wait(&slot_full[sl], ((r + s) / C::kSlots) & 1, wc);
                        uint8_t *vr = sRing + sl * C::kSlotBytes + row * 128;
                        uint32_t wild = 0;                // an exponent of all ones carries into the sign's place
                        if (seen && draft >= 0) {
#pragma unroll 1
                            for (int c = 0; c < 2; ++c)
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    const uint4 w = reinterpret_cast<const uint4 *>(vr + c * C::kChunkBytes)[i ^ (row & 7)];
                                    wild |= ((w.x & 0x7f807f80u) + 0x00800080u) | ((w.y & 0x7f807f80u) + 0x00800080u) |
                                            ((w.z & 0x7f807f80u) + 0x00800080u) | ((w.w & 0x7f807f80u) + 0x00800080u);
                                }
                            wild &= 0x80008000u;
                            if (wild) mark_bad(bad, k, draft);
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
            if (warp_live)
                write_row<D, NT>(p, u, x, row, live, t, h, m_ref, l_sum, live && sees_bad(bad, u, k, mrow),
                                 [&](int c, float (&o)[32]) {
                    tmem_ld32(tmem + lane_off + C::o_col(x) + c * 32, o);
                    tmem_wait_ld();
                });
            tc_fence_before();
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// Merges the pieces of the units that CTA ranges cut: with weighted sums o_i,
// row sums l_i and bases m_i, M = max m_i, out = sum 2^(m_i - M) o_i /
// sum 2^(m_i - M) l_i.  The pieces of the unit whose first one ended CTA c's
// range opened the following ranges.  Block (chunk, c) takes 32 rows of that
// unit, a lane a row and a warp an equal share of the columns, as the pieces lie, and
// turns the result round in shared memory.  Pieces are read four at once where a
// lane's share of one is 64 bytes, two where it is 128 (four: 1.3 us more at dim 256).
// Two row tiles, whose partials are the most, take blocks of four warps, of which
// more are there when the last CTA ends (129 -> 127 us for 16 requests with 121
// drafts; one row tile, often of more pieces, is better off with eight: 13.4 us
// against 14.1 for one request).  The rows past a request's drafts are written here
// too.
template <int NT>
constexpr int kMergeThreads = NT == 2 ? 128 : 256;

template <int D, int NT>
__global__ void __launch_bounds__(kMergeThreads<NT>) tree_merge_kernel(const __grid_constant__ TreeParams p) {
    constexpr int kThreads = kMergeThreads<NT>;
    constexpr int kUnits = D / 4 / (kThreads / 32);   // 16-byte FP32 units of a warp's columns
    constexpr int kPieces = 16 / kUnits;
    __shared__ uint4 stage[32][D / 8 + 1];           // BF16 rows
    __shared__ long long offset[32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // Zeros and -inf, a warp to a draft; these wait for nothing.
    const int nwarps = gridDim.x * gridDim.y * (kThreads / 32);
    for (int i = (blockIdx.y * gridDim.x + blockIdx.x) * (kThreads / 32) + warp; i < p.B * p.T; i += nwarps) {
        const int b = i / p.T, pt = i - b * p.T;
        int n, d;
        tree_row(p, b, n, d);
        if (pt < d) continue;
        __nv_bfloat16 *o = reinterpret_cast<__nv_bfloat16 *>(p.out) + b * p.out_stride[0] + pt * p.out_stride[1];
        for (int c = lane; c < p.Hq * (D / 8); c += 32)
            reinterpret_cast<uint4 *>(o + (c / (D / 8)) * p.out_stride[2])[c % (D / 8)] = make_uint4(0, 0, 0, 0);
        if (p.lse)
            for (int ph = lane; ph < p.Hq; ph += 32)
                p.lse[b * p.lse_stride[0] + pt * p.lse_stride[1] + ph * p.lse_stride[2]] = kNegInf;
    }
    pdl_wait();                                      // the pieces are written
    const TreeCut cut = p.cuts[blockIdx.y];
    const int x = blockIdx.x / 4, row = (blockIdx.x & 3) * 32 + lane;
    if (cut.count == 0 || x >= cut.nrt) return;
    int t, h;
    const bool live = tree_tile_row(p, cut.rt0 + x, cut.g, cut.d, row, t, h);
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
        offset[lane] = live ? cut.b * p.out_stride[0] + t * p.out_stride[1] + h * p.out_stride[2] : -1;
        if (live && p.lse)
            p.lse[cut.b * p.lse_stride[0] + t * p.lse_stride[1] + h * p.lse_stride[2]] =
                l != 0.f ? (m + log2f(l)) * 0.69314718055994531f : kNegInf;
    }
    __syncthreads();
    for (int i = tid; i < 32 * (D / 8); i += kThreads) {
        const int r = i / (D / 8), c = i % (D / 8);
        if (offset[r] >= 0)
            reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(p.out) + offset[r])[c] = stage[r][c];
    }
}

template <int D, int NT>
cudaError_t launch_bf16(const TreeParams &p, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                        cudaStream_t stream, int *launches) {
    using C = TreeCfg<D, NT>;
    static bool configured[64] = {};
    return launch_pieces(tree_decode_kernel<D, NT>, NT, C::kThreads, C::kSmemBytes, p, tq, tk, tv, stream, configured,
                         launches);
}

}  // namespace

cudaError_t launch_tree_merge(const TreeParams &p, int row_tiles, cudaStream_t stream) {
    const dim3 grid(row_tiles * 4, p.grid), block(row_tiles == 2 ? kMergeThreads<2> : kMergeThreads<1>);
    if (p.D == 256) return launch_after_previous(tree_merge_kernel<256, 1>, grid, block, 0, stream, p);
    if (row_tiles == 2) return launch_after_previous(tree_merge_kernel<128, 2>, grid, block, 0, stream, p);
    return launch_after_previous(tree_merge_kernel<128, 1>, grid, block, 0, stream, p);
}

size_t tree_workspace_bytes(int head_dim, int grid) {
    const int rows = head_dim == 128 ? 256 : 128;
    return (size_t)grid * (2 * (size_t)rows * (head_dim * 4 + 8) + sizeof(TreeCut));
}

void tree_place_workspace(TreeParams *p, void *ws) {
    const int64_t rows = p->D == 128 ? 256 : 128;
    char *at = static_cast<char *>(ws);
    p->part_o = reinterpret_cast<float *>(at);
    at += (int64_t)p->grid * 2 * rows * p->D * 4;
    p->part_ml = reinterpret_cast<float2 *>(at);
    at += (int64_t)p->grid * 2 * rows * 8;
    p->cuts = reinterpret_cast<TreeCut *>(at);
}

cudaError_t launch_tree_decode(const TreeParams &p, const CUtensorMap &tq, const CUtensorMap &tk,
                               const CUtensorMap &tv, cudaStream_t stream, int *launches) {
    *launches = 0;
    if (p.kv8) return launch_tree_decode_fp8(p, tq, tk, tv, stream, launches);
    if (p.D == 256) return launch_bf16<256, 1>(p, tq, tk, tv, stream, launches);
    if (p.row_tiles > 1) return launch_bf16<128, 2>(p, tq, tk, tv, stream, launches);
    return launch_bf16<128, 1>(p, tq, tk, tv, stream, launches);
}

}  // namespace fw
