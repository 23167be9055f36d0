// What the tree-decode kernels (BF16 and FP8 caches) share: the rows of a unit,
// the walk over a CTA's range of the planned sequence, mask bits, the merge of
// the pieces of cut units.  The chunk kernels take the softmax's arithmetic, the
// page windows and the way rows are written from here (Params, Unit: theirs or the
// tree's).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "decode_common.cuh"
#include "fw_internal.h"
#include "fw_ptx.cuh"

namespace fw {
namespace tree {

using dec::ceil_div_i;
using dec::warp_wait;
constexpr float kNegInf = -__builtin_huge_valf();
// The base of a row's exponentials moves only when its maximum rose by more
// than this many log2 units, so every weight is at most 2^8.
constexpr float kRescaleSlack = 8.0f;
// Instruction descriptor bit: A enters negated (scores of a negative scale).
constexpr uint32_t kIdescNegateA = 1u << 13;
constexpr int kErrInvalid = 1;     // FW_ERR_INVALID_ARG

// One piece: a unit's key tiles inside one CTA range.  64 bytes.
struct alignas(16) TreeUnit {
    int b;             // request, -1 ends the CTA's work
    int g;             // KV head
    int rt0, nrt;      // first row tile and how many
    int n, d;          // keys and drafts of the request
    int tile0, ntiles; // key tiles
    int part;          // partial slot, -1: the whole unit, written to the outputs
    int pad_[7];
};
static_assert(sizeof(TreeUnit) == 64, "a unit record fills one 64-byte slot");

// Keys and drafts of request b, both within what the call can hold.
__device__ __forceinline__ void tree_row(const TreeParams &p, int b, int &n, int &d) {
    n = min(max(__ldg(p.seq_lens + b), 0), p.max_pages * p.ps);
    d = p.draft_lens ? min(max(__ldg(p.draft_lens + b), 0), p.T) : p.T;
    d = min(d, n);
}

// Units of a request in the planned sequence (of one KV head when the heads
// ride on the CTA index).
template <int NT>
__device__ __forceinline__ int tree_units(const TreeParams &p, int d) {
    const int tiles = p.head_chunks > 1 ? d * p.head_chunks : ceil_div_i(d, p.tile_tokens);
    return ceil_div_i(tiles, NT) * (p.ride ? 1 : p.Hkv);
}

// The (draft, head) of row r of row tile rt; false for padding.
__device__ __forceinline__ bool tree_tile_row(const TreeParams &p, int rt, int g, int d, int r, int &t, int &h) {
    if (p.head_chunks > 1) {
        t = rt / p.head_chunks;
        const int hh = (rt - t * p.head_chunks) * 128 + r;
        h = g * p.G + hh;
        return hh < p.G && t < d;
    }
    const int tt = r / p.G;
    t = rt * p.tile_tokens + tt;
    h = g * p.G + (r - tt * p.G);
    return tt < p.tile_tokens && t < d;
}

// Bits of the 32 keys from draft ds on (ds < 0: committed keys first) that the
// mask row shows, among the request's d drafts.
__device__ __forceinline__ uint32_t draft_bits(const int32_t *row, int ds, int d) {
    if (ds <= -32) return 0xffffffffu;
    if (ds >= d) return 0u;
    uint32_t v;
    if (ds < 0) {
        v = ((uint32_t)__ldg(row) << -ds) | ((1u << -ds) - 1u);
    } else {
        const int w = ds >> 5;
        const uint32_t lo = (uint32_t)__ldg(row + w);
        const uint32_t hi = (w + 1) * 32 < d ? (uint32_t)__ldg(row + w + 1) : 0u;
        v = __funnelshift_r(lo, hi, ds & 31);
    }
    const int left = d - ds;
    return left < 32 ? v & ((1u << left) - 1u) : v;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
}

// The softmax's instructions, not its latencies, set a tile's time once several
// warps share a scheduler: maxima of three, and products and sums in pairs.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ void split_pair(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// Largest of N values.
template <int N>
__device__ __forceinline__ float max_of(const float *v) {
    float m[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int i = 4; i + 1 < N; i += 2) m[(i >> 1) & 3] = max3(m[(i >> 1) & 3], v[i], v[i + 1]);
    return fmaxf(max3(m[0], m[1], m[2]), m[3]);
}
// 2^(v * scale + shift) of 64 values, in place, their sum added to four pairs.
__device__ __forceinline__ void exp_64(float *v, float scale, float shift, uint64_t (&sum)[4]) {
    const uint64_t sc = pair_of(scale, scale), sh = pair_of(shift, shift);
#pragma unroll
    for (int i = 0; i < 64; i += 2) {
        float a, b;
        split_pair(fma_pair(pair_of(v[i], v[i + 1]), sc, sh), a, b);
        v[i] = ex2_approx(a);
        v[i + 1] = ex2_approx(b);
        sum[(i >> 1) & 3] = add_pair(sum[(i >> 1) & 3], pair_of(v[i], v[i + 1]));
    }
}
__device__ __forceinline__ float sum_of(const uint64_t (&sum)[4]) {
    float a, b;
    split_pair(add_pair(add_pair(sum[0], sum[1]), add_pair(sum[2], sum[3])), a, b);
    return a + b;
}

// Ring positions, in units of whole K or V tiles, of a piece of n key tiles
// when QK runs L tiles ahead of PV: K_0 .. K_{L-1}, then V_j K_{j+L}.
template <int L>
__device__ __forceinline__ int pos_v(int j, int n) { return min(L, n) + j + min(j, max(0, n - L)); }
template <int L>
__device__ __forceinline__ int pos_k(int j, int n) { return j < L ? j : pos_v<L>(j - L, n) + 1; }


// The planned sequence: request b takes units * (piece_cost + tiles) slots.
// Every thread sums a run of requests; the one whose run holds this CTA's first
// slot looks the request up.  plan[0] = slots in all, plan[1], plan[2] = start
// and number of the request holding the CTA's first slot, plan[3] = span.
// Ends with every thread past a barrier but plan not yet published.
template <int NT>
__device__ __forceinline__ void plan_range(const TreeParams &p, long long *plan, long long *scan) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nthreads = blockDim.x;
    const int per = (p.B + nthreads - 1) / nthreads;
    auto row_slots = [&](int b) -> long long {
        int n, d;
        tree_row(p, b, n, d);
        return (long long)tree_units<NT>(p, d) * (p.piece_cost + ceil_div_i(n, kKvTile));
    };
    long long mine = 0;
    const int b0 = threadIdx.x * per;
    for (int i = 0; i < per && b0 + i < p.B; ++i) mine += row_slots(b0 + i);
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    long long before = incl - mine, total = 0;
    for (int w = 0; w < nthreads / 32; ++w) {
        if (w < warp) before += scan[w];
        total += scan[w];
    }
    const int nranges = p.ride ? (int)gridDim.x / p.Hkv : (int)gridDim.x;
    const long long span = max((long long)p.min_span, (total + nranges - 1) / nranges);
    const long long first = span * (p.ride ? (int)blockIdx.x / p.Hkv : (int)blockIdx.x);
    if (mine > 0 && first >= before && first < before + mine) {
        int b = b0;
        for (long long s; first >= before + (s = row_slots(b)); ++b) before += s;
        plan[1] = before;
        plan[2] = b;
    }
    if (threadIdx.x == 0) { plan[0] = total; plan[3] = span; }
}

// Walks the pieces of this CTA's range (one warp, all lanes alike).  It
// stands at slot `vl` of unit `ui` of request b, so that a step divides nothing.
template <int NT>
struct TreeWalk {
    long long span, left, row0;                       // slots left in the range; the request's first slot
    int range, b, n, d, units, tiles, ui, vl;
    TreeCut cut;

    __device__ void open_row(const TreeParams &p) {
        tree_row(p, b, n, d);
        units = tree_units<NT>(p, d);
        tiles = ceil_div_i(n, kKvTile);
    }
    __device__ void init(const TreeParams &p, const long long *plan) {
        span = plan[3];
        range = p.ride ? (int)blockIdx.x / p.Hkv : (int)blockIdx.x;
        const long long pos = span * range;
        left = min(plan[0], pos + span) - pos;
        cut = TreeCut{};
        if (left > 0) {
            row0 = plan[1];
            b = (int)plan[2];
            open_row(p);
            ui = (int)((pos - row0) / (p.piece_cost + tiles));
            vl = (int)(pos - row0 - (long long)ui * (p.piece_cost + tiles));
        }
    }
    __device__ void next(const TreeParams &p, TreeUnit &u) {     // u.b = -1 at the end
        u.b = -1;
        while (left > 0) {
            if (ui >= units) {                        // on to the next request
                row0 += (long long)units * (p.piece_cost + tiles);
                ++b;
                ui = 0;
                open_row(p);
                continue;
            }
            if (vl < p.piece_cost) {
                left -= p.piece_cost - vl;
                vl = p.piece_cost;
                continue;
            }
            const int tl = vl - p.piece_cost;
            const int th = (int)min((long long)tiles, tl + left);
            u.b = b;
            const int per_head = p.ride ? units : units / p.Hkv;
            u.g = p.ride ? (int)blockIdx.x % p.Hkv : ui / per_head;
            const int rts = p.head_chunks > 1 ? d * p.head_chunks : ceil_div_i(d, p.tile_tokens);
            u.rt0 = (p.ride ? ui : ui - u.g * per_head) * NT;
            u.nrt = min(NT, rts - u.rt0);
            u.n = n;
            u.d = d;
            u.tile0 = tl;
            u.ntiles = th - tl;
            u.part = -1;
            if (tl > 0) {
                u.part = 2 * blockIdx.x;
            } else if (th < tiles) {
                u.part = 2 * blockIdx.x + 1;
                const long long last = row0 + (long long)ui * (p.piece_cost + tiles) + p.piece_cost + tiles - 1;
                cut.count = (int)(last / span) - range + 1;
                cut.b = b; cut.g = u.g; cut.rt0 = u.rt0; cut.nrt = u.nrt; cut.d = d;
            }
            left -= th - tl;
            vl += th - tl;
            if (th == tiles) { ++ui; vl = 0; }
            return;
        }
    }
};

// The queries of a unit (one lane): `nrt` row tiles of 128-byte-swizzled 64-column
// chunks, `chunk` bytes apart.
template <int D, int NT>
__device__ __forceinline__ void copy_queries(const TreeParams &p, const TreeUnit &u, const CUtensorMap &tm_q, uint8_t *sQ,
                                             uint32_t tile_bytes, uint32_t chunk, uint64_t *q_full) {
    const uint32_t qrows = p.head_chunks > 1 ? 128u : (uint32_t)(p.G * p.tile_tokens);
    mbar_arrive_expect_tx(q_full, (uint32_t)u.nrt * (D / 64) * qrows * 128u);
    for (int x = 0; x < u.nrt; ++x) {
        const int rt = u.rt0 + x;
        int h0 = u.g * p.G, t0 = rt * p.tile_tokens;
        if (p.head_chunks > 1) { t0 = rt / p.head_chunks; h0 += (rt - t0 * p.head_chunks) * 128; }
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
            tma_load_4d(smem_u32(sQ + x * tile_bytes + c * chunk), &tm_q, q_full, c * 64, h0, t0, u.b);
    }
}

// Whether page `l` of key tile j of a unit is copied: a tile has up to 16 pages,
// one to a lane.
template <typename Params, typename Unit>
__device__ __forceinline__ bool page_copied(const Params &p, const Unit &u, int j, int l) {
    const int key = (u.tile0 + j) * kKvTile + (p.ps < kKvTile ? l * p.ps : 0);
    return l * p.ps < kKvTile && (l == 0 || p.ps < kKvTile) && j < u.ntiles && key < u.n;
}
// The block-table entries of a piece, 64 at a time in two registers a lane; the
// next 32 are fetched while these are in use.  (Fetched tile by tile, an entry's
// latency is the least a tile can take, some 1,000 cycles: an E4M3 tile's share
// of HBM is 1,350, and the two add up.)
struct PageWindow {
    const int32_t *row;
    int win, last, cur, nxt;

    template <typename Params>
    __device__ __forceinline__ int page_number(const Params &p, int key) const {
        return p.ps_shift >= 0 ? key >> p.ps_shift : key / p.ps;
    }
    __device__ __forceinline__ int entry(int lp) const { return lp <= last ? __ldg(row + lp) : 0; }
    template <typename Params, typename Unit>
    __device__ __forceinline__ void open(const Params &p, const Unit &u) {
        const int lane = threadIdx.x & 31;
        row = p.block_table + (int64_t)u.b * p.bt_stride;
        win = page_number(p, u.tile0 * kKvTile);
        last = page_number(p, min(u.n, (u.tile0 + u.ntiles) * kKvTile) - 1);
        cur = entry(win + lane);
        nxt = entry(win + 32 + lane);
    }
    // The entry of page lane % 16 of key tile j (tiles in order; all lanes call).
    template <typename Params, typename Unit>
    __device__ __forceinline__ int at(const Params &p, const Unit &u, int j) {
        const int lane = threadIdx.x & 31;
        const int lp = page_number(p, (u.tile0 + j) * kKvTile);
        if (lp >= win + 32) {
            win += 32;
            cur = nxt;
            nxt = entry(win + 32 + lane);
        }
        const int idx = lp + (lane & 15) - win;        // < 64 for the pages copied
        const int a = __shfl_sync(0xffffffffu, cur, idx & 31), b = __shfl_sync(0xffffffffu, nxt, idx & 31);
        return idx < 32 ? a : b;
    }
};
// The page to copy, inside the pool whatever the table says.
template <typename Params>
__device__ __forceinline__ int checked_page(const Params &p, int phys) {
    if ((unsigned)phys < (unsigned)p.num_pages) return phys;
    record_error(p.status, kErrInvalid);
    return 0;
}

// Which keys of a 128-key tile some draft of the request sees: bit l of word w is
// key 32 w + l.  128 threads (`id`: their named barrier) share the drafts; `words`
// is 16 words of shared memory that nobody else writes before the next call but
// one.  seen_word reads a word of the result.
__device__ __forceinline__ void seen_keys(const TreeParams &p, const TreeUnit &u, int key0, int thread, uint32_t id,
                                          uint32_t *words) {
    const int lane = thread & 31, w4 = thread >> 5, base = u.n - u.d;
    uint32_t seen[4] = {0, 0, 0, 0};
    for (int t = thread; t < u.d; t += 128) {
        const int32_t *mr = p.mask + u.b * p.mask_stride[0] + t * p.mask_stride[1];
#pragma unroll
        for (int w = 0; w < 4; ++w) seen[w] |= draft_bits(mr, key0 + 32 * w - base, u.d);
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        seen[w] = __reduce_or_sync(0xffffffffu, seen[w]);
        if (lane == 0) words[w4 * 4 + w] = seen[w];
    }
    named_bar_sync(id, 128);
}
__device__ __forceinline__ uint32_t seen_word(const uint32_t *words, int w) {
    return words[w] | words[4 + w] | words[8 + w] | words[12 + w];
}

// Values that are not finite.  A committed key's reach every row as they are.  Those
// of a draft, which some rows see and others do not, must not meet the others' zero
// weights: they are cleared before the products, and the rows that see that draft
// come out as NaN.  A bit to a draft, in the words of unit k % kBadUnits; the unit
// records keep a writer at most four units ahead of a reader.  Cleared when a unit
// begins; the writers meet in seen_keys before the first bit.
constexpr int kBadUnits = 5, kBadWords = 8;
__device__ __forceinline__ void mark_bad(uint32_t *bad, int k, int draft) {
    atomicOr(bad + k % kBadUnits * kBadWords + (draft >> 5), 1u << (draft & 31));
}
__device__ __forceinline__ bool sees_bad(const uint32_t *bad, const TreeUnit &u, int k, const int32_t *mrow) {
    if ((u.tile0 + u.ntiles) * kKvTile <= u.n - u.d) return false;     // no drafts in this piece
    const uint4 *words = reinterpret_cast<const uint4 *>(bad + k % kBadUnits * kBadWords);
    const uint4 a = words[0], b = words[1];
    if (__builtin_expect((a.x | a.y | a.z | a.w | b.x | b.y | b.z | b.w) == 0, 1)) return false;
    uint32_t hit = 0;
#pragma unroll 1
    for (int w = 0; 32 * w < u.d; ++w) hit |= bad[k % kBadUnits * kBadWords + w] & (uint32_t)__ldg(mrow + w);
    return hit != 0;
}

// ------------------------------------------------------------ 8-bit caches
constexpr float kPShift = 7.0f;     // FP16 weights carry 2^7

// kind::f8f6f4, A and B E4M3 K-major, FP32 accumulation.
constexpr uint32_t kIdescF8QK = (1u << 4) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
// kind::f16, A and B FP16, B MN-major, FP32 accumulation.
constexpr uint32_t kIdescF16PV = (1u << 4) | (1u << 16) | ((128u >> 3) << 17) | ((128u >> 4) << 24);

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

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// BF16 row * 2^e = hi + mid, both E4M3, over the row's own bytes (two blocks of 128 bytes a
// row, HALF apart, swizzled): 16 lanes hold a row's 16-byte units, four warps eight rows a pass
// each (each pass waits for its reads and its maxima once), all read before any is written.
// put_exp(r, e) keeps row r's e.
template <int HALF, typename PutExp>
__device__ __forceinline__ void split_rows(uint8_t *q0, int rows, int warp, int lane, PutExp put_exp) {
    const int un = lane & 15;
#pragma unroll 1
    for (int rb = 8 * warp; rb < rows; rb += 32) {
        const int r0 = rb + (lane >> 4);
        uint4 w[4];
        uint32_t big[4];                      // largest magnitude, as the bits of an FP32
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = r0 + 2 * i;
            w[i] = *reinterpret_cast<const uint4 *>(q0 + (un >> 3) * HALF + r * 128 + (((un & 7) ^ (r & 7)) << 4));
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
            if (un == 0) put_exp(r, (int8_t)e);
            // An infinite or NaN element makes the row's scores NaN.
            const float up = __int_as_float(big[i] >= 0x7f800000u ? 0x7fc00000 : (127 + e) << 23);
            uint32_t hi[4], mid[4];
            split2(w[i].x, up, hi[0], mid[0]);
            split2(w[i].y, up, hi[1], mid[1]);
            split2(w[i].z, up, hi[2], mid[2]);
            split2(w[i].w, up, hi[3], mid[3]);
            uint8_t *to = q0 + r * 128 + (((un >> 1) ^ (r & 7)) << 4) + (un & 1) * 8;
            *reinterpret_cast<uint2 *>(to) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
            *reinterpret_cast<uint2 *>(to + HALF) = make_uint2(mid[0] | mid[1] << 16, mid[2] | mid[3] << 16);
        }
    }
}

// A piece's partial rows: 16-byte units of four columns, the rows of a unit side by
// side, so that a warp whose lanes are rows writes and reads whole lines.  (Row by
// row, 32 lanes touch 32 lines a store, and a piece's end took 8,000 cycles.)
template <int D, int NT, typename Params>
__device__ __forceinline__ float4 *part_unit(const Params &p, int64_t slot, int unit, int row) {
    return reinterpret_cast<float4 *>(p.part_o) + (slot * (D / 4) + unit) * (NT * 128) + row;
}

// This thread's row of a finished piece: its output and LSE, or its partial.
// `out_at` and `lse_at` say where its output and LSE lie, as numbers or as what works them
// out where they are needed (the tree decode's: numbers took a batch of FP8 trees 136 us for 133);
// `load` reads 32 columns of O (warp-collective); columns 32 c0 .. 32 c1.
template <typename At>
__device__ __forceinline__ long long place_of(At at) {
    if constexpr (std::is_integral_v<At>) return at;
    else return at();
}
template <int D, int NT, typename Params, typename Unit, typename OutAt, typename LseAt, typename Load>
__device__ __forceinline__ void write_row_at(const Params &p, const Unit &u, int x, int row, bool live, OutAt out_at,
                                             LseAt lse_at, float base2, float l_sum, bool poison, Load load,
                                             int c0 = 0,
                                             int c1 = D / 32) {
    const int lane = threadIdx.x & 31;
    // (A NaN sum is not zero: a NaN that the row sees comes out as NaN.)
    const bool some = l_sum != 0.f;
    const float inv = poison ? __int_as_float(0x7fc00000) : some ? p.out_scale / l_sum : 0.f;
    // Outputs: four lanes exchange their rows' four 16-byte units of a chunk, so that
    // each store writes 64 bytes of a row.
    const long long at = live ? place_of(out_at) : -1;
    long long to[4];
    if (u.part < 0) {
#pragma unroll
        for (int k = 0; k < 4; ++k) to[k] = __shfl_sync(0xffffffffu, at, (lane & ~3) + k);
    }
#pragma unroll 1
    for (int c = c0; c < c1; ++c) {
        float o[32];
        load(c, o);
        if (u.part < 0) {
            uint32_t v[4][4];
#pragma unroll
            for (int w = 0; w < 4; ++w)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[w][i] = some ? pack_bf16x2(o[8 * w + 2 * i] * inv, o[8 * w + 2 * i + 1] * inv) : 0u;
#pragma unroll
            for (int s = 1; s <= 2; s <<= 1) {
                const bool hi = lane & s;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (k & s) continue;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t got = __shfl_xor_sync(0xffffffffu, hi ? v[k][i] : v[k | s][i], s);
                        if (hi) v[k][i] = got; else v[k | s][i] = got;
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (to[k] >= 0)
                    *reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(p.out) + to[k] + c * 32 + (lane & 3) * 8) =
                        make_uint4(v[k][0], v[k][1], v[k][2], v[k][3]);
        } else if (live) {
            if (poison) {
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = inv;
            }
#pragma unroll
            for (int w = 0; w < 8; ++w)
                *part_unit<D, NT>(p, u.part, c * 8 + w, x * 128 + row) =
                    make_float4(o[4 * w], o[4 * w + 1], o[4 * w + 2], o[4 * w + 3]);
        }
    }
    if (!live || c0 > 0) return;
    if (u.part >= 0) p.part_ml[(int64_t)u.part * (NT * 128) + x * 128 + row] = make_float2(base2, l_sum);
    else if (p.lse) p.lse[place_of(lse_at)] = some ? (base2 + log2f(l_sum)) * 0.69314718055994531f : kNegInf;
}
template <int D, int NT, typename Load>
__device__ __forceinline__ void write_row(const TreeParams &p, const TreeUnit &u, int x, int row, bool live, int t,
                                          int h, float base2, float l_sum, bool poison, Load load,
                                          int c0 = 0,
                                          int c1 = D / 32) {
    write_row_at<D, NT>(
        p, u, x, row, live, [&] { return u.b * p.out_stride[0] + t * p.out_stride[1] + h * p.out_stride[2]; },
        [&] { return u.b * p.lse_stride[0] + t * p.lse_stride[1] + h * p.lse_stride[2]; }, base2, l_sum, poison, load, c0, c1);
}

// One launch for the pieces, one for the merge of cut units.
template <typename Kernel>
inline cudaError_t launch_pieces(Kernel kernel, int NT, int threads, size_t smem, const TreeParams &p,
                                 const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                                 cudaStream_t stream, bool (&configured)[64], int *launches) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!configured[dev & 63]) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        configured[dev & 63] = true;
    }
    kernel<<<p.grid, threads, smem, stream>>>(p, tq, tk, tv);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    ++*launches;
    e = launch_tree_merge(p, NT, stream);
    if (e != cudaSuccess) return e;
    ++*launches;
    return cudaSuccess;
}

}  // namespace tree
}  // namespace fw
