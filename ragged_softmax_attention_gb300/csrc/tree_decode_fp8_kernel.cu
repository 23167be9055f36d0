// Paged decode of a tree of drafted tokens over an FP8 E4M3 cache, sm_103a.
// Units, ranges, pieces and the merge are those of the BF16 kernel
// (tree_decode_kernel.cu); head dim 128.
//
// An SM's share of HBM delivers an E4M3 K/V tile of 128 keys (32 KiB) in ~1,350
// cycles, half a BF16 tile's, so neither the tensor core nor shared memory can
// afford to widen both caches:
//   S = Q K^T   kind::f8f6f4 on the E4M3 bytes as they land.  Each BF16 query
//               row is scaled by a power of two (largest magnitude in
//               [128, 256)) and carried as two E4M3 terms, hi + mid, exact for
//               every element down to 2^-10 of the row's largest; below, an
//               element is off by at most 2^-17 of the largest.  Two terms of
//               K = 32 products take the tensor core as long as one BF16 pass.
//   O += P V    kind::f16 on FP16: four warps widen each V tile (exact in FP16),
//               64 keys at a time, from the slot it landed in to one the products
//               read; the small second ring leaves most of shared memory to the
//               copies in flight.  P is rounded
//               to FP16, scaled by 2^7 so that weights down to 2^-21 of the
//               largest keep 11 bits (base slack of 2^8 and that factor stay below
//               FP16's 2^16).
// The same warps split the queries, ahead of the softmax, and write zeros for
// the values of keys nobody sees.
//
// Measured: 32 requests of 512 .. 16,384 keys, 16 drafts of 40/8 heads, 529 MB in
// 134.5 us, 0.58 of the measured copy rate; with 32 drafts (two row tiles) 227 us.  A
// key tile takes some 1,900 cycles (3,480): the widened V tile's round (convert
// 1,100, PV behind QK, the slot back) and the softmax of two warpgroups in turn, 103
// us in all; starts and ends of pieces take 18, the way to the first scores 8 of them
// (13 with two row tiles, whose queries the converting warps split as well).  More
// slots for widened values make it slower (139 us), P as two E4M3 terms would need no
// widening but loses the weights below 2^-17 of the largest.
//
// Warp roles: 0 copies keys and values, 1 and 2 issue MMAs, 3 works out the
// pieces and copies queries, 4-7 convert, 8-15 softmax (a warpgroup per stream, or two for one:
// a tile's softmax takes some 2,000 cycles of a warpgroup, more than the tile's
// share of HBM).
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "tree_common.cuh"

namespace fw {
namespace {

using namespace tree;

constexpr int D = 128;
constexpr float kPShift = 7.0f;     // P carries 2^7

// kind::f8f6f4, A and B E4M3 K-major, FP32 accumulation.
constexpr uint32_t kIdescQK = (1u << 4) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
// kind::f16, A and B FP16, B MN-major, FP32 accumulation.
constexpr uint32_t kIdescPV = (1u << 4) | (1u << 16) | ((128u >> 3) << 17) | ((128u >> 4) << 24);

template <int NT_>
struct F8TreeCfg {
    static constexpr int NT = NT_;
    static constexpr int kSB = NT == 2 ? 1 : 3;                 // S buffers of a stream
    static constexpr int kWG = 2;                               // softmax warpgroups, NT = 1: every other tile each
    static constexpr int kQBytes = 128 * D * 2;                 // BF16 rows, then their two E4M3 terms in place
    static constexpr int kKBytes = 128 * D;
    static constexpr int kHalf = 128 * 128;                     // 64 columns of the BF16 rows; one term
    static constexpr int kVChunk = 64 * 128;                    // 64 keys x 64 FP16 columns
    static constexpr int kVBytes = 2 * kVChunk;                 // FP16 values of half a tile's keys
    static constexpr int kKSlots = NT == 2 ? 3 : 4;
    static constexpr int kRSlots = NT == 2 ? 4 : 5;             // E4M3 values as they land
    static constexpr int kVSlots = NT == 2 ? 3 : 2;
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + NT * kQBytes;
    static constexpr int kOffR = kOffK + kKSlots * kKBytes;
    static constexpr int kOffV = kOffR + kRSlots * kKBytes;
    static constexpr int kOffBar = kOffV + kVSlots * kVBytes;
    static constexpr int kSched = 4;
    static constexpr int kBarKFull = 0;
    static constexpr int kBarKEmpty = kBarKFull + kKSlots;
    static constexpr int kBarRFull = kBarKEmpty + kKSlots;      // E4M3 values landed
    static constexpr int kBarREmpty = kBarRFull + kRSlots;      // and read
    static constexpr int kBarVFull = kBarREmpty + kRSlots;      // widened
    static constexpr int kBarVEmpty = kBarVFull + kVSlots;
    static constexpr int kBarQFull = kBarVEmpty + kVSlots;
    static constexpr int kBarQEmpty = kBarQFull + 1;
    static constexpr int kBarQReady = kBarQEmpty + 1;           // [kSched] terms and exponents of unit k written
    static constexpr int kBarSFull = kBarQReady + kSched;       // [NT][kSB]
    static constexpr int kBarPHalf = kBarSFull + NT * kSB;
    static constexpr int kBarPFull = kBarPHalf + NT * kSB;
    static constexpr int kBarPvDone = kBarPFull + NT * kSB;
    static constexpr int kBarIssued = kBarPvDone + NT * kSB;    // [NT]
    static constexpr int kBarDrain = kBarIssued + NT;           // [2]
    static constexpr int kBarBase = kBarDrain + 2;              // [2] base of the rows after a tile (NT = 1)
    static constexpr int kBarOFree = kBarBase + 2;              // O read by both warpgroups (NT = 1)
    static constexpr int kBarSchedFull = kBarOFree + 1;
    static constexpr int kBarSchedEmpty = kBarSchedFull + kSched;
    static constexpr int kBarNever = kBarSchedEmpty + kSched;   // test hook: no thread ever arrives on it
    static constexpr int kNumBars = kBarNever + 1;
    static constexpr int kOffSched = (kOffBar + kNumBars * 8 + 63) / 64 * 64;
    static constexpr int kOffSeen = kOffSched + kSched * 64;    // [2][16 words]
    static constexpr int kOffBad = kOffSeen + 128;              // drafts whose values are NaN
    static constexpr int kOffQScale = kOffBad + kBadUnits * kBadWords * 4;   // [kSched][NT][128 bytes]: exponents of the rows
    static constexpr int kOffPlan = kOffQScale;                 // the plan is used up before the first of them
    static constexpr int kOffScan = kOffPlan + 32;              // [16]
    static constexpr int kOffBase = kOffQScale + kSched * NT * 128;   // NT = 1: [2][128] bases, [2][2][128] row sums
    static constexpr int kOffMisc = kOffBase + (NT == 1 ? (2 + 4) * 128 * 4 : 0);
    static constexpr int kSmemBytes = kOffMisc + 16 + 1024;
    static_assert(kSmemBytes <= 232448, "shared memory budget of one CTA exceeded");
    static constexpr int kThreads = 256 + kWG * 128;
    static constexpr int kSchedReaders = 3 + 4 + 4 * kWG;            // issuers, the producer, converters, softmax
    // 512 threads launched at 128 registers: 128 x 72 + 128 x 96 + 256 x 168 =
    // 64512 <= 65536.
    static constexpr uint32_t kRegsControl = 72, kRegsConvert = 96, kRegsSoftmax = 168, kRegsLaunch = 128;
    static_assert(128 * kRegsControl + 128 * kRegsConvert + kWG * 128 * kRegsSoftmax <= kThreads * kRegsLaunch,
                  "register split");
    __device__ static constexpr uint32_t s_col(int x, int buf) { return (uint32_t)(x * kSB + buf) * 128u; }
    __device__ static constexpr uint32_t o_col(int x) { return (uint32_t)(NT * kSB + x) * 128u; }
};

// Four E4M3 values (one word) as four FP16 values, two words.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
}

// Two BF16 values (one word) times `up` as hi + mid, two E4M3 values each.
__device__ __forceinline__ void split2(uint32_t w, float up, uint32_t &hi, uint32_t &mid) {
    const float a = __uint_as_float(w << 16) * up, b = __uint_as_float(w & 0xffff0000u) * up;
    hi = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const float2 h = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)hi, __NV_E4M3)));
    mid = __nv_cvt_float2_to_fp8x2(make_float2(a - h.x, b - h.y), __NV_SATFINITE, __NV_E4M3);
}

// -inf in place of the scores of hidden keys.
__device__ __forceinline__ void hide(float (&v)[64], uint32_t lo, uint32_t hi) {
#pragma unroll
    for (int i = 0; i < 64; ++i)
        if (!((i < 32 ? lo : hi) >> (i & 31) & 1)) v[i] = kNegInf;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

template <int NT>
__global__ void __launch_bounds__(F8TreeCfg<NT>::kThreads, 1)
tree_decode_fp8_kernel(const __grid_constant__ TreeParams p, const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
    using C = F8TreeCfg<NT>;
    constexpr int kSB = C::kSB;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sQ = smem + C::kOffQ;
    uint8_t *sK = smem + C::kOffK;
    uint8_t *sR = smem + C::kOffR;
    uint8_t *sV = smem + C::kOffV;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
    uint64_t *k_full = bars + C::kBarKFull;
    uint64_t *k_empty = bars + C::kBarKEmpty;
    uint64_t *r_full = bars + C::kBarRFull;
    uint64_t *r_empty = bars + C::kBarREmpty;
    uint64_t *v_full = bars + C::kBarVFull;
    uint64_t *v_empty = bars + C::kBarVEmpty;
    uint64_t *q_full = bars + C::kBarQFull;
    uint64_t *q_empty = bars + C::kBarQEmpty;
    uint64_t *q_ready = bars + C::kBarQReady;
    uint64_t *s_full = bars + C::kBarSFull;
    uint64_t *p_half = bars + C::kBarPHalf;
    uint64_t *p_full = bars + C::kBarPFull;
    uint64_t *pv_done = bars + C::kBarPvDone;
    uint64_t *issued = bars + C::kBarIssued;
    uint64_t *drain = bars + C::kBarDrain;
    uint64_t *base_set = bars + C::kBarBase;
    uint64_t *o_free = bars + C::kBarOFree;
    uint64_t *sched_full = bars + C::kBarSchedFull;
    uint64_t *sched_empty = bars + C::kBarSchedEmpty;
    TreeUnit *sched = reinterpret_cast<TreeUnit *>(smem + C::kOffSched);
    uint32_t *seen_words = reinterpret_cast<uint32_t *>(smem + C::kOffSeen);
    uint32_t *bad = reinterpret_cast<uint32_t *>(smem + C::kOffBad);
    long long *plan = reinterpret_cast<long long *>(smem + C::kOffPlan);
    long long *scan = reinterpret_cast<long long *>(smem + C::kOffScan);
    float *bases = reinterpret_cast<float *>(smem + C::kOffBase);      // [2][128], NT = 1
    float *sums = bases + 256;                                         // [2][2][128], NT = 1
    int8_t *q_exp = reinterpret_cast<int8_t *>(smem + C::kOffQScale);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kOffMisc + 4);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kKSlots; ++i) { mbar_init(&k_full[i], 1); mbar_init(&k_empty[i], NT); }
        for (int i = 0; i < C::kRSlots; ++i) { mbar_init(&r_full[i], 1); mbar_init(&r_empty[i], 4); }
        for (int i = 0; i < C::kVSlots; ++i) { mbar_init(&v_full[i], 4); mbar_init(&v_empty[i], NT); }
        mbar_init(q_full, 1);
        mbar_init(q_empty, NT);
        for (int i = 0; i < NT * kSB; ++i) {
            mbar_init(&s_full[i], 1); mbar_init(&p_half[i], 4); mbar_init(&p_full[i], 4); mbar_init(&pv_done[i], 1);
        }
        for (int i = 0; i < NT; ++i) mbar_init(&issued[i], 1);
        for (int i = 0; i < 2; ++i) { mbar_init(&drain[i], 1); mbar_init(&base_set[i], 4); }
        mbar_init(o_free, 4 * C::kWG);
        for (int i = 0; i < C::kSched; ++i) {
            mbar_init(&q_ready[i], 4); mbar_init(&sched_full[i], 1); mbar_init(&sched_empty[i], C::kSchedReaders);
        }
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
      setmaxnreg_dec<C::kRegsControl>();
      if (warp == 0) {
        // ------------------------------------------------------------ producer
        const int box_rows = p.ps < kKvTile ? p.ps : kKvTile;
        uint32_t ik = 0, iv = 0;                          // K and V tiles issued
        // Test hook for the bounded waits, as in the BF16 kernel.
        bool ok = !p.test_stall || warp_wait(bars + C::kBarNever, 0, wc, lane);
        for (int k = 0; ok; ++k) {
            const TreeUnit *ur = wait_unit(k);
            TreeUnit u;
            u.b = -1;
            if (ur) u = *ur;
            __syncwarp();
            if (lane == 0) free_unit(k);
            if (!__all_sync(0xffffffffu, u.b >= 0)) break;
            // K tile i and V tile i - kSB go out together, a half warp each: one
            // after the other, a copy's barrier and copy instructions take this warp
            // 1,100 cycles beside the others, and a tile two of them.
            PageWindow table;
            table.open(p, u);
            const bool is_v = lane >= 16;
            const int l = lane & 15;
            int entries[kSB + 1];                         // of the last tiles: V comes kSB later
#pragma unroll
            for (int i = 0; i <= kSB; ++i) entries[i] = 0;
            for (int i = 0; i < u.ntiles + kSB && ok; ++i) {
#pragma unroll
                for (int e = 0; e < kSB; ++e) entries[e] = entries[e + 1];
                if (i < u.ntiles) entries[kSB] = table.at(p, u, i);
                const int j = is_v ? i - kSB : i;
                const bool there = j >= 0 && j < u.ntiles;
                const uint32_t slots = is_v ? C::kRSlots : C::kKSlots;
                const uint32_t c = is_v ? iv : ik, sl = c % slots;
                uint64_t *full = is_v ? &r_full[sl] : &k_full[sl];
                const bool mine = there && page_copied(p, u, j, l);
                const unsigned who = __ballot_sync(0xffffffffu, mine) & (is_v ? 0xffff0000u : 0xffffu);
                bool landed = true;
                if (l == 0 && there) landed = mbar_wait(is_v ? &r_empty[sl] : &k_empty[sl], ((c / slots) & 1) ^ 1, wc);
                ok = __all_sync(0xffffffffu, landed);
                if (!ok) break;
                if (l == 0 && there) mbar_arrive_expect_tx(full, (uint32_t)(__popc(who) * box_rows * 128));
                __syncwarp();
                if (mine) {
                    const int key0 = (u.tile0 + j) * kKvTile;
                    const int slot0 = p.ps < kKvTile ? 0 : p.ps_shift >= 0 ? key0 & (p.ps - 1) : key0 % p.ps;
                    tma_load_4d(smem_u32((is_v ? sR : sK) + sl * C::kKBytes + l * box_rows * 128),
                                is_v ? (const void *)&tm_v : (const void *)&tm_k, full, 0, u.g, slot0,
                                checked_page(p, is_v ? entries[0] : entries[kSB]));
                }
                if (i < u.ntiles) ++ik;
                if (i >= kSB) ++iv;
            }
        }
        if (lane == 0) {
            for (uint32_t i = 0; i < (uint32_t)C::kKSlots && i < ik; ++i)
                mbar_wait_drain(&k_full[(ik - 1 - i) % C::kKSlots], ((ik - 1 - i) / C::kKSlots) & 1, wc);
            for (uint32_t i = 0; i < (uint32_t)C::kRSlots && i < iv; ++i)
                mbar_wait_drain(&r_full[(iv - 1 - i) % C::kRSlots], ((iv - 1 - i) / C::kRSlots) & 1, wc);
        }
        __syncwarp();
      } else if (warp < 3) {
        // ----------------------------------------------------------------- MMA
        if (lane == 0) {
            const int x = NT == 2 ? warp - 1 : 0;
            uint32_t tiles = 0;                           // K (and V) tiles of earlier pieces
            uint32_t steps = 0;                           // this stream's among them
            uint32_t turns = 0;                           // those both streams took part in
            const SDesc q_d = sdesc_sw128_split(smem_u32(sQ + x * C::kQBytes), 16, 1024);
            const SDesc k_d = sdesc_sw128_split(smem_u32(sK), 16, 1024);
            const SDesc v_d = sdesc_sw128_split(smem_u32(sV), C::kVChunk, 1024);
            auto wait_k = [&](uint32_t i) { return mbar_wait(&k_full[i % C::kKSlots], (i / C::kKSlots) & 1, wc); };
            // Half `half` of V tile i is number 2 i + half of the second ring.
            auto wait_v = [&](uint32_t i, int half) {
                const uint32_t h = 2 * i + half;
                return mbar_wait(&v_full[h % C::kVSlots], (h / C::kVSlots) & 1, wc);
            };
            auto release_v = [&](uint32_t i, int half) { mma_commit(&v_empty[(2 * i + half) % C::kVSlots]); };
            auto k_there = [&](uint32_t i) {
                return mbar_try_wait(smem_u32(&k_full[i % C::kKSlots]), (i / C::kKSlots) & 1);
            };
            const uint32_t idesc_qk = kIdescQK | (p.scale_log2 < 0.f ? kIdescNegateA : 0u);
            auto push_qk = [&](uint32_t i, int buf) {
                const SDesc kd{k_d.lo + (i % C::kKSlots) * (C::kKBytes >> 4), k_d.hi};
#pragma unroll
                for (int term = 0; term < 2; ++term)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_f8_ss(tmem + C::s_col(x, buf), sdesc_at(q_d, term * C::kHalf + kk * 32),
                                  sdesc_at(kd, kk * 32), idesc_qk, term + kk > 0 ? 1u : 0u);
            };
            auto push_pv_half = [&](uint32_t i, int buf, int half, bool first) {
                const SDesc vd{v_d.lo + ((2 * i + half) % C::kVSlots) * (C::kVBytes >> 4), v_d.hi};
#pragma unroll
                for (int k4 = 0; k4 < 4; ++k4)
                    mma_bf16_ts(tmem + C::o_col(x), tmem + C::s_col(x, buf) + (half * 4 + k4) * 8,
                                sdesc_at(vd, k4 * 16 * 128), kIdescPV, (first && half + k4 == 0) ? 0u : 1u);
            };
            bool ok = true;
            if constexpr (NT == 1) {
                // QK and PV from a thread each, as in the BF16 kernel.
                for (int k = 0; ok; ++k) {
                    const TreeUnit *ur = wait_unit(k);
                    const bool got = ur && ur->b >= 0;
                    const int n = got ? ur->ntiles : 0;
                    free_unit(k);
                    if (!got) break;
                    if (warp == 2) ok = mbar_wait(&q_ready[k % C::kSched], (k / C::kSched) & 1, wc);
                    else if (k > 0) ok = mbar_wait(o_free, (k - 1) & 1, wc);   // the last piece's O is read
                    for (int j = 0; j < n && ok; ++j, ++steps) {
                        const int buf = steps % kSB;
                        const uint32_t ph = (steps / kSB) & 1;
                        if (warp == 2) {
                            ok = wait_k(steps) && (steps < kSB || mbar_wait(&pv_done[buf], ph ^ 1, wc));
                            if (!ok) break;
                            tc_fence_after();
                            push_qk(steps, buf);
                            mma_commit(&s_full[buf]);
                            mma_commit(&k_empty[steps % C::kKSlots]);
                            if (j == n - 1) mma_commit(q_empty);
                        } else {
                            ok = wait_v(steps, 0) && mbar_wait(&p_half[buf], ph, wc);
                            if (!ok) break;
                            tc_fence_after();
                            push_pv_half(steps, buf, 0, j == 0);
                            release_v(steps, 0);
                            ok = wait_v(steps, 1) && mbar_wait(&p_full[buf], ph, wc);
                            if (!ok) break;
                            tc_fence_after();
                            push_pv_half(steps, buf, 1, false);
                            mma_commit(&pv_done[buf]);
                            release_v(steps, 1);
                        }
                    }
                }
            } else {
                for (int k = 0; ok; ++k) {
                    const TreeUnit *ur = wait_unit(k);
                    const bool got = ur && ur->b >= 0;
                    const int n = got ? ur->ntiles : 0;
                    const int nrt = got ? ur->nrt : 0;
                    free_unit(k);
                    if (!got) break;
                    const uint32_t i0 = tiles;
                    tiles += (uint32_t)n;
                    if (!mbar_wait(&q_ready[k % C::kSched], (k / C::kSched) & 1, wc)) break;
                    if (x >= nrt) {
                        // No row tile for this stream: it still sees every tile come and
                        // hands every slot back, so that its phases stay in step.
                        mbar_arrive(q_empty);
                        for (uint32_t i = i0; i < tiles && ok; ++i) {
                            ok = wait_k(i);
                            if (ok) mbar_arrive(&k_empty[i % C::kKSlots]);
                            for (int half = 0; half < 2 && ok; ++half) {
                                ok = wait_v(i, half);
                                if (ok) mbar_arrive(&v_empty[(2 * i + half) % C::kVSlots]);
                            }
                        }
                        continue;
                    }
                    tc_fence_after();
                    for (int j = 0; j < kSB && j < n && ok; ++j) {
                        ok = wait_k(i0 + j);
                        if (!ok) break;
                        tc_fence_after();
                        push_qk(i0 + j, (steps + j) % kSB);
                        mma_commit(&s_full[x * kSB + (steps + j) % kSB]);
                        mma_commit(&k_empty[(i0 + j) % C::kKSlots]);
                        if (j == n - 1) mma_commit(q_empty);
                    }
                    for (int j = 0; j < n && ok; ++j) {
                        const uint32_t st = steps + j;
                        const int buf = st % kSB;
                        const uint32_t ph = (st / kSB) & 1;
                        const uint32_t iv = i0 + j, ik = i0 + j + kSB;
                        if (nrt == 2) {
                            // Turns, as in the BF16 kernel.
                            const uint32_t dep = turns + j + x;
                            if (dep > 0 && !mbar_wait(&issued[1 - x], (dep - 1) & 1, wc)) { ok = false; break; }
                        }
                        if (!wait_v(iv, 0) || !mbar_wait(&p_half[x * kSB + buf], ph, wc)) { ok = false; break; }
                        const bool next = j + kSB < n;
                        const bool paired = next && k_there(ik);
                        tc_fence_after();
                        push_pv_half(iv, buf, 0, j == 0);
                        if (!wait_v(iv, 1) || !mbar_wait(&p_full[x * kSB + buf], ph, wc)) { ok = false; break; }
                        tc_fence_after();
                        push_pv_half(iv, buf, 1, false);
                        if (nrt == 2) mbar_arrive(&issued[x]);
                        if (paired) push_qk(ik, buf);
                        if (j == n - 1) mma_commit(&pv_done[x]);
                        release_v(iv, 0);
                        release_v(iv, 1);
                        if (next) {
                            if (!paired) {
                                if (!wait_k(ik)) { ok = false; break; }
                                tc_fence_after();
                                push_qk(ik, buf);
                            }
                            mma_commit(&s_full[x * kSB + buf]);
                            mma_commit(&k_empty[ik % C::kKSlots]);
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
            if (lane == 0) copy_queries<D, NT>(p, u, tm_q, sQ, C::kQBytes, C::kHalf, q_full);
            __syncwarp();
        }
        if (lane == 0) p.cuts[blockIdx.x] = walk.cut;
        __syncwarp();
      }
    } else if (warp < 8) {
        if constexpr (C::kRegsConvert < C::kRegsLaunch) setmaxnreg_dec<C::kRegsConvert>();
        // ------------------------------------------------------------ converters
        // Thread = query row of a tile, then = key of a tile.  After an abort
        // every wait returns at once and the bounded loops run out; the four warps,
        // which share a named barrier, take or leave a unit together, as do the softmax
        // warps below.
        const int row = threadIdx.x - 128;
        uint32_t i = 0;                                   // V tiles converted
        for (int k = 0;; ++k) {
            const TreeUnit *ur = wait_unit(k);
            TreeUnit u;
            u.b = -1;
            if (ur) u = *ur;
            __syncwarp();
            if (lane == 0) free_unit(k);
            if (!named_bar_all(3, 128, u.b >= 0)) break;
            if (row < kBadWords) bad[k % kBadUnits * kBadWords + row] = 0;
            mbar_wait(q_full, k & 1, wc);
            for (int x = 0; x < u.nrt; ++x) {
                // BF16 row * 2^e = hi + mid, both E4M3, over the row's own bytes: 16 lanes
                // hold a row's 16-byte units, eight rows a pass (each pass waits for its
                // reads and its maxima once), all read before any is written.
                uint8_t *q0 = sQ + x * C::kQBytes;
                const int rows = p.head_chunks > 1 ? 128 : p.G * p.tile_tokens;
                const int un = lane & 15;
#pragma unroll 1
                for (int rb = 8 * (warp - 4); rb < rows; rb += 32) {
                    const int r0 = rb + (lane >> 4);
                    uint4 w[4];
                    uint32_t big[4];                      // largest magnitude, as the bits of an FP32
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = r0 + 2 * i;
                        w[i] = *reinterpret_cast<const uint4 *>(q0 + (un >> 3) * C::kHalf + r * 128 + (((un & 7) ^ (r & 7)) << 4));
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        auto top = [](uint32_t v) { return max((v << 16) & 0x7fff0000u, v & 0x7fff0000u); };
                        big[i] = max(max(top(w[i].x), top(w[i].y)), max(top(w[i].z), top(w[i].w)));
                    }
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1)
#pragma unroll
                        for (int i = 0; i < 4; ++i) big[i] = max(big[i], __shfl_xor_sync(0xffffffffu, big[i], o));
                    __syncwarp();                         // the rows are read
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = r0 + 2 * i;
                        const int e = min(126, max(-120, 134 - (int)(big[i] >> 23)));   // 7 - (exponent - 127)
                        if (un == 0) q_exp[(k % C::kSched * NT + x) * 128 + r] = (int8_t)e;
                        // An infinite or NaN element makes the row's scores NaN.
                        const float up = __int_as_float(big[i] >= 0x7f800000u ? 0x7fc00000 : (127 + e) << 23);
                        uint32_t hi[4], mid[4];
                        split2(w[i].x, up, hi[0], mid[0]);
                        split2(w[i].y, up, hi[1], mid[1]);
                        split2(w[i].z, up, hi[2], mid[2]);
                        split2(w[i].w, up, hi[3], mid[3]);
                        uint8_t *to = q0 + r * 128 + (((un >> 1) ^ (r & 7)) << 4) + (un & 1) * 8;
                        *reinterpret_cast<uint2 *>(to) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
                        *reinterpret_cast<uint2 *>(to + C::kHalf) = make_uint2(mid[0] | mid[1] << 16, mid[2] | mid[3] << 16);
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_ready[k % C::kSched]);
            const int base = u.n - u.d;
            for (int j = 0; j < u.ntiles; ++j, ++i) {
                const int key0 = (u.tile0 + j) * kKvTile;
                uint32_t *words = seen_words + (j & 1) * 16;
                const bool drafts = key0 + kKvTile > base;
                if (drafts) seen_keys(p, u, key0, row, 3, words);
                const uint32_t rl = i % C::kRSlots;
                mbar_wait(&r_full[rl], (i / C::kRSlots) & 1, wc);
                if (drafts) {
                    // Values of keys nobody sees must not meet a zero weight: they may be
                    // NaN; nor a draft's NaN the weights of rows that do not see it.  A
                    // thread looks after one key, in the slot it landed in.
                    const bool seen = seen_word(words, row >> 5) >> (row & 31) & 1;
                    const int draft = key0 + row - base;
                    uint4 *vr = reinterpret_cast<uint4 *>(sR + rl * C::kKBytes + row * 128);
                    uint32_t wild = 0;                    // the bits of a NaN carry into the sign's place
                    if (seen && draft >= 0) {
#pragma unroll 1
                        for (int c = 0; c < 8; ++c) {
                            const uint4 w = vr[c ^ (row & 7)];
                            wild |= ((w.x & 0x7f7f7f7fu) + 0x01010101u) | ((w.y & 0x7f7f7f7fu) + 0x01010101u) |
                                    ((w.z & 0x7f7f7f7fu) + 0x01010101u) | ((w.w & 0x7f7f7f7fu) + 0x01010101u);
                        }
                        wild &= 0x80808080u;
                        if (wild) mark_bad(bad, k, draft);
                    }
                    if (!seen || wild) {
#pragma unroll 1
                        for (int c = 0; c < 8; ++c) vr[c ^ (row & 7)] = make_uint4(0, 0, 0, 0);
                    }
                    named_bar_sync(3, 128);
                }
                // Keys key and 64 + key, columns 64 ch .. 64 ch + 63 of each.  (Rolled:
                // unrolled, this and the softmax evict each other from the instruction
                // cache, which more than doubled both.)
                const int key = row & 63, ch = row >> 6;
                const uint32_t sw = key & 7;
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    const uint32_t hv = 2 * i + half, sl = hv % C::kVSlots;
                    const uint8_t *from = sR + rl * C::kKBytes + (half * 64 + key) * 128;
                    uint8_t *to = sV + sl * C::kVBytes + ch * C::kVChunk + key * 128;
                    uint4 w[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) w[c] = *reinterpret_cast<const uint4 *>(from + (((ch * 4 + c) ^ sw) << 4));
                    mbar_wait(&v_empty[sl], ((hv / C::kVSlots) & 1) ^ 1, wc);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {         // 16 values: two units of FP16
                        uint4 a, b;
                        widen4(w[c].x, a.x, a.y);
                        widen4(w[c].y, a.z, a.w);
                        widen4(w[c].z, b.x, b.y);
                        widen4(w[c].w, b.z, b.w);
                        *reinterpret_cast<uint4 *>(to + (((2 * c) ^ sw) << 4)) = a;
                        *reinterpret_cast<uint4 *>(to + (((2 * c + 1) ^ sw) << 4)) = b;
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (half == 1) mbar_arrive(&r_empty[rl]);
                        mbar_arrive(&v_full[sl]);
                    }
                }
            }
        }
    } else {
        setmaxnreg_inc<C::kRegsSoftmax>();
        // ------------------------------------------------- softmax / epilogue
        // One stream: the two warpgroups take every other key tile.  A row's base
        // passes from tile to tile through shared memory, each keeps the sum of its
        // own tiles, and both write half of the outputs.
        const int wg = (warp - 8) >> 2;
        const int x = NT == 2 ? wg : 0;
        const int q4 = warp & 3;
        const int row = q4 * 32 + lane;
        const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
        uint32_t steps = 0, pieces = 0;
        auto wait_pv = [&](uint32_t step) { mbar_wait(&pv_done[x * kSB + step % kSB], (step / kSB) & 1, wc); };
        for (int k = 0;; ++k) {
            const TreeUnit *ur = wait_unit(k);
            TreeUnit u;
            u.b = -1;
            if (ur) u = *ur;
            // The row's exponent is read before the record goes back: unit k + 4,
            // which reuses its place, cannot come before that.
            if (u.b >= 0) mbar_wait(&q_ready[k % C::kSched], (k / C::kSched) & 1, wc);
            // (Bounded from below: a scale of zero, or a small one times the 2^-126 of a row
            // of zeros, would turn the -inf of hidden keys into NaN.  Sums here
            // stay below 2^24, so under the bound every score is zero to the exponential.)
            const float rs = fmaxf(fabsf(p.scale_log2) *
                                       __int_as_float((127 - q_exp[(k % C::kSched * NT + x) * 128 + row]) << 23),
                                   1e-37f);
            __syncwarp();
            if (lane == 0) free_unit(k);
            if (!(NT == 1 ? named_bar_all(4, 128 * C::kWG, u.b >= 0) : __all_sync(0xffffffffu, u.b >= 0) != 0)) break;
            if (x >= u.nrt) continue;
            int t, h;
            const bool live = tree_tile_row(p, u.rt0 + x, u.g, u.d, row, t, h);
            const bool warp_live = __any_sync(0xffffffffu, live);
            const int base = u.n - u.d;
            const int32_t *mrow = p.mask + u.b * p.mask_stride[0] + (live ? t : 0) * p.mask_stride[1];
            float m_ref = kNegInf, l_sum = 0.f;           // l_sum relative to m_ref
            constexpr int kEvery = NT == 2 ? 1 : C::kWG;
            for (int j = NT == 2 ? 0 : (int)((steps ^ (uint32_t)wg) & 1); j < u.ntiles; j += kEvery) {
                const uint32_t st = steps + j;
                const int buf = st % kSB;
                const int key0 = (u.tile0 + j) * kKvTile;
                const bool drafts = key0 + kKvTile > base;
                uint32_t bits[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
                if (drafts) {
#pragma unroll
                    for (int w = 0; w < 4; ++w) bits[w] = live ? draft_bits(mrow, key0 + 32 * w - base, u.d) : 0u;
                }
                mbar_wait(&s_full[x * kSB + buf], (st / kSB) & 1, wc);
                tc_fence_after();
                if (!warp_live) {                         // rows of padding: whatever lies there
                    // The last tile's base is waited for all the same: this warp must not
                    // stand in for one of the next phase's arrivals.
                    if (NT == 1 && j > 0) mbar_wait(&base_set[(st - 1) & 1], ((st - 1) >> 1) & 1, wc);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (NT == 1) mbar_arrive(&base_set[st & 1]);
                        mbar_arrive(&p_half[x * kSB + buf]);
                        mbar_arrive(&p_full[x * kSB + buf]);
                    }
                    continue;
                }
                const uint32_t sa = tmem + lane_off + C::s_col(x, buf);
                // The row of S is read twice, for its maximum and for P, 64 keys at a
                // time: two streams' softmax warps have no registers for all of it, and
                // the rolled loops keep the code small.
                float ext = kNegInf;
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {
                    float v[64];
                    tmem_ld32(sa + c * 64, v);
                    tmem_ld32(sa + c * 64 + 32, v + 32);
                    tmem_wait_ld();
                    if (drafts) hide(v, c == 0 ? bits[0] : bits[2], c == 0 ? bits[1] : bits[3]);
                    ext = fmaxf(ext, max_of<64>(v));
                }
                const float m_tile = ext == kNegInf || !live ? kNegInf : ext * rs;
                float m_prev = m_ref;                     // the rows' base so far
                if constexpr (NT == 1) {
                    if (j == 0) {
                        m_prev = kNegInf;
                    } else {
                        mbar_wait(&base_set[(st - 1) & 1], ((st - 1) >> 1) & 1, wc);
                        m_prev = bases[((st - 1) & 1) * 128 + row];
                    }
                }
                const bool up = m_tile > m_prev + kRescaleSlack;
                const float m_new = up ? m_tile : m_prev;
                if (__any_sync(0xffffffffu, up) && j > 0) {
                    const float alpha = up ? ex2_approx(m_prev - m_new) : 1.f;
                    if constexpr (kSB > 1) {
                        wait_pv(st - 1);
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
                if constexpr (NT == 1) {
                    bases[(st & 1) * 128 + row] = m_new;
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&base_set[st & 1]);
                }
                if (m_new != m_ref) {
                    l_sum *= ex2_approx(m_ref - m_new);
                    m_ref = m_new;
                }
                // P = 2^(s * rs - m_ref + 7), rounded to FP16; the row sum takes it
                // unrounded.
                const float mu = (m_ref == kNegInf ? 0.f : m_ref) - kPShift;
                uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    float v[64];
                    uint32_t pk[32];
                    tmem_ld32(sa + half * 64, v);
                    tmem_ld32(sa + half * 64 + 32, v + 32);
                    tmem_wait_ld();
                    if (drafts) hide(v, half == 0 ? bits[0] : bits[2], half == 0 ? bits[1] : bits[3]);
                    exp_64(v, rs, -mu, sum);
#pragma unroll
                    for (int i = 0; i < 64; i += 2) pk[i >> 1] = pack_half2(v[i], v[i + 1]);
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        tmem_st16u(sa + half * 32 + c * 16, *reinterpret_cast<const uint32_t(*)[16]>(pk + c * 16));
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(half == 0 ? &p_half[x * kSB + buf] : &p_full[x * kSB + buf]);
                }
                l_sum += sum_of(sum);
            }
            // ------------------------------------------------------ epilogue
            ++pieces;
            steps += u.ntiles;
            if constexpr (NT == 1) {
                const uint32_t last = steps - 1;
                float *sum = sums + (k & 1) * 256;
                if (warp_live) {
                    mbar_wait(&base_set[last & 1], (last >> 1) & 1, wc);
                    const float m_end = bases[(last & 1) * 128 + row];
                    if (m_end != m_ref) l_sum *= ex2_approx(m_ref - m_end);
                    m_ref = m_end;
                    sum[wg * 128 + row] = l_sum;
                }
                named_bar_sync(4, 128 * C::kWG);
                l_sum = sum[row] + sum[128 + row];
#pragma unroll
                for (int i = kSB; i >= 1; --i)
                    if (steps >= (uint32_t)i) wait_pv(steps - i);
            } else {
                mbar_wait(&pv_done[x], (pieces - 1) & 1, wc);
            }
            tc_fence_after();
            if (warp_live)
                write_row<D, NT>(p, u, x, row, live, t, h, m_ref - kPShift, l_sum, live && sees_bad(bad, u, k, mrow),
                                 [&](int c, float (&o)[32]) {
                    tmem_ld32(tmem + lane_off + C::o_col(x) + c * 32, o);
                    tmem_wait_ld();
                }, NT == 1 ? 2 * wg : 0, NT == 1 ? 2 * wg + 2 : D / 32);
            if constexpr (NT == 1) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(o_free);
            }
            tc_fence_before();
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int NT>
cudaError_t launch_fp8(const TreeParams &p, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                       cudaStream_t stream, int *launches) {
    using C = F8TreeCfg<NT>;
    static bool configured[64] = {};
    return launch_pieces(tree_decode_fp8_kernel<NT>, NT, C::kThreads, C::kSmemBytes, p, tq, tk, tv, stream, configured,
                         launches);
}

}  // namespace

cudaError_t launch_tree_decode_fp8(const TreeParams &p, const CUtensorMap &tq, const CUtensorMap &tk,
                                   const CUtensorMap &tv, cudaStream_t stream, int *launches) {
    return p.row_tiles > 1 ? launch_fp8<2>(p, tq, tk, tv, stream, launches) : launch_fp8<1>(p, tq, tk, tv, stream, launches);
}

}  // namespace fw
