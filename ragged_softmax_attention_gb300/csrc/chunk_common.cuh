// What the chunk kernels (a CTA, or a pair of CTAs at head dim 256) share: the plan of
// units and ranges, the walk over a range, masks, and what becomes of values that are not
// finite.
#pragma once

#include "tree_common.cuh"

namespace fw {
namespace chunk {

using namespace tree;

// One piece: a unit's key tiles inside one CTA range.  64 bytes.
struct alignas(16) ChunkUnit {
    int b;             // request, -1 ends the CTA's work
    int g;             // KV head
    int rt0, nrt;      // first row tile and how many
    int n, d, q0;      // keys and new tokens of the request, its first packed row
    int tile0, ntiles; // key tiles
    int part;          // partial slot, -1: the whole unit, written to the outputs
    int lo;            // first key that a row sees: pages wholly before it are not copied
    int pad_[5];
};
static_assert(sizeof(ChunkUnit) == 64, "a unit record fills one 64-byte slot");

// ------------------------------------------------------------------ the plan

// A request's units: `steps` runs of tokens (the first `v0` of which see nothing) times
// `reps` (KV heads, and parts of a token's heads).  All weights in keys.
struct ChunkRow {
    int n, d, q0, steps, v0, reps;
};
template <int NT>
__device__ __forceinline__ int step_tokens(const ChunkParams &p) { return p.head_chunks > 1 ? 1 : NT * p.tile_tokens; }

template <int NT>
__device__ __forceinline__ ChunkRow chunk_row(const ChunkParams &p, int b) {
    ChunkRow r;
    r.q0 = __ldg(p.cu + b);
    const int end = __ldg(p.cu + b + 1);
    const bool ok = r.q0 >= 0 && end >= r.q0 && end <= p.total_q;
    if (!ok && blockIdx.x == 0) record_error(p.status, kErrInvalid);
    r.d = ok ? end - r.q0 : 0;
    r.n = min(max(__ldg(p.seq_lens + b), 0), p.max_pages * p.ps);
    const int s = step_tokens<NT>(p);
    r.steps = ceil_div_i(r.d, s);
    r.v0 = r.n == 0 ? r.steps : p.causal && r.d > r.n ? (r.d - r.n) / s : 0;
    r.reps = (p.head_chunks > 1 ? ceil_div_i(p.head_chunks, NT) : 1) * (p.ride ? 1 : p.Hkv);
    return r;
}
// Weight of step v, and of steps v0 .. v - 1.
template <int NT>
__device__ __forceinline__ long long step_weight(const ChunkParams &p, const ChunkRow &r, int v) {
    const long long s = step_tokens<NT>(p), base = r.n - r.d;
    const long long hi = p.causal ? base + (v + 1) * s : r.n;
    const long long lo = p.window < 0 ? 0 : max(0ll, base - p.window + v * s);
    return p.piece_cost + 128 + hi - lo;
}
template <int NT>
__device__ __forceinline__ long long steps_weight(const ChunkParams &p, const ChunkRow &r, int v) {
    const long long s = step_tokens<NT>(p), base = r.n - r.d, m = v - r.v0;
    auto sum = [](long long a, long long e) { return (e - a) * (a + e - 1) / 2; };      // a + .. + e - 1
    long long w = m * (p.piece_cost + 128);
    w += p.causal ? m * (base + s) + s * sum(r.v0, v) : m * r.n;
    if (p.window >= 0) {
        const long long z = base - p.window;                     // lo = z + i s where that is above zero
        const long long first = max((long long)r.v0, z >= 0 ? 0 : -z / s + 1);
        if (first < v) w -= (v - first) * z + s * sum(first, v);
    }
    return w;
}

// The range of `worker` (a CTA, or a pair of them).  plan[0] = weight in all, plan[1],
// plan[2] = start and number of the request that holds the range's first key, plan[3] = span.  Ends with every thread past a barrier but plan not
// yet published.
template <int NT>
__device__ __forceinline__ void chunk_plan(const ChunkParams &p, int worker, long long *plan, long long *scan) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nthreads = blockDim.x;
    const int per = (p.B + nthreads - 1) / nthreads;
    auto weight = [&](int b) -> long long {
        const ChunkRow r = chunk_row<NT>(p, b);
        return r.v0 < r.steps ? r.reps * steps_weight<NT>(p, r, r.steps) : 0;
    };
    long long mine = 0;
    const int b0 = threadIdx.x * per;
    for (int i = 0; i < per && b0 + i < p.B; ++i) mine += weight(b0 + i);
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
    const int nranges = p.ride ? p.workers / p.Hkv : p.workers;
    const long long span = max((long long)p.min_span, (total + nranges - 1) / nranges);
    const long long first = span * (p.ride ? worker / p.Hkv : worker);
    if (mine > 0 && first >= before && first < before + mine) {
        int b = b0;
        for (long long s; first >= before + (s = weight(b)); ++b) before += s;
        plan[1] = before;
        plan[2] = b;
    }
    if (threadIdx.x == 0) { plan[0] = total; plan[3] = span; }
}

// Walks the pieces of a worker's range (one warp, all lanes alike).  A border at weight
// x of a unit cuts it before tile (x - cost) / 128, for the ranges on both sides alike;
// a piece without tiles is none.
template <int NT>
struct ChunkWalk {
    long long span, pos, end, start;                  // the range; start of the unit
    int worker, range, b, rep, v;
    ChunkRow r;
    ChunkCut cut;

    __device__ int tile_at(const ChunkParams &p, long long x, int tiles) const {
        x -= p.piece_cost;
        return x <= 0 ? 0 : (int)min((long long)tiles, x >> 7);
    }
    __device__ void init(const ChunkParams &p, int who, const long long *plan) {
        worker = who;
        span = plan[3];
        range = p.ride ? worker / p.Hkv : worker;
        pos = span * range;
        end = min(plan[0], pos + span);
        cut = ChunkCut{};
        start = end;
        if (pos >= end) return;
        b = (int)plan[2];
        r = chunk_row<NT>(p, b);
        const long long all = steps_weight<NT>(p, r, r.steps);
        rep = (int)((pos - plan[1]) / all);
        const long long off = pos - plan[1] - rep * all;
        int lo = r.v0, hi = r.steps - 1;              // the last step that starts at or before off
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (steps_weight<NT>(p, r, mid) <= off) lo = mid; else hi = mid - 1;
        }
        v = lo;
        start = plan[1] + rep * all + steps_weight<NT>(p, r, v);
    }
    __device__ void next(const ChunkParams &p, ChunkUnit &u) {   // u.b = -1 at the end
        u.b = -1;
        const int s = step_tokens<NT>(p);
        while (start < end) {
            if (v >= r.steps) {                       // the next KV head, the next request
                v = r.v0;
                if (v >= r.steps || ++rep >= r.reps) {
                    if (++b >= p.B) return;           // (weight is left, so there is one)
                    r = chunk_row<NT>(p, b);
                    rep = 0;
                    v = r.v0;
                }
                continue;
            }
            const long long w = step_weight<NT>(p, r, v);
            const int t0 = v * s, t1 = min(r.d, t0 + s) - 1;
            const int lo = p.window < 0 ? 0 : (int)max(0ll, (long long)r.n - r.d + t0 - p.window);
            const int hi = p.causal ? r.n - r.d + t1 + 1 : r.n;
            const int tile0 = lo / kKvTile, tiles = ceil_div_i(hi, kKvTile) - tile0;
            const int a = tile_at(p, pos - start, tiles);
            const int e = end >= start + w ? tiles : tile_at(p, end - start, tiles);
            const long long at = start;
            const int step = v;
            start += w;
            ++v;
            if (a >= e) continue;
            const int parts = p.head_chunks > 1 ? ceil_div_i(p.head_chunks, NT) : 1;
            const int g = rep / parts, part = rep - g * parts;
            u.b = b;
            u.g = p.ride ? worker % p.Hkv : g;
            u.rt0 = p.head_chunks > 1 ? step * p.head_chunks + part * NT : step * NT;
            u.nrt = min(NT, p.head_chunks > 1 ? p.head_chunks - part * NT : ceil_div_i(r.d, p.tile_tokens) - u.rt0);
            u.n = r.n;
            u.d = r.d;
            u.q0 = r.q0;
            u.tile0 = tile0 + a;
            u.ntiles = e - a;
            u.lo = lo;
            u.part = -1;
            if (a > 0) {
                u.part = 2 * worker;
            } else if (e < tiles) {
                u.part = 2 * worker + 1;
                const long long last = min((at + p.piece_cost + 128ll * tiles + span - 1) / span, (at + w + span - 1) / span);
                cut.count = (int)last - range;
                cut.g = u.g; cut.rt0 = u.rt0; cut.nrt = u.nrt; cut.d = r.d; cut.q0 = r.q0;
            }
            return;
        }
    }
};

// The (token, head) of row r of row tile rt; false for padding.
__device__ __forceinline__ bool chunk_tile_row(const ChunkParams &p, int rt, int g, int d, int r, int &t, int &h) {
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

// First and last key that token t sees, as [lo, hi).
__device__ __forceinline__ int key_lo(const ChunkParams &p, const ChunkUnit &u, int t) {
    return p.window < 0 ? 0 : (int)max(0ll, (long long)u.n - u.d + t - p.window);
}
__device__ __forceinline__ int key_hi(const ChunkParams &p, const ChunkUnit &u, int t) {
    return p.causal ? max(0, u.n - u.d + t + 1) : u.n;
}
// The bits lo .. hi - 1 of 32 keys from `key` on.
__device__ __forceinline__ uint32_t range_bits(int lo, int hi, int key) {
    lo = max(lo - key, 0);
    hi = min(hi - key, 32);
    if (lo >= hi) return 0u;
    return (0xffffffffu >> (32 - (hi - lo))) << lo;
}

// Values that are not finite, in tiles that some row of the unit does not see whole: they
// must not meet the zero weights of rows that do not see them.  They are cleared before
// the products, and the rows that see them come out as NaN.  Such tiles are few, for a
// unit's 256 tokens at most three at either end: bits of a tile's keys in the words of unit
// k % kBadUnits (a writer is at most four units ahead of a reader), behind a word that
// says whether there are any.
constexpr int kBadUnitWords = 4 + 8 * 4;
__device__ __forceinline__ uint32_t *bad_words(uint32_t *marks, int tile, int any_lo, int all_hi) {
    const int upper = tile - all_hi / kKvTile;            // >= 0: reaches past what the first row sees
    return marks + 4 + 4 * ((upper >= 0 ? 4 + upper : tile - any_lo / kKvTile) & 7);
}

}  // namespace chunk
}  // namespace fw
