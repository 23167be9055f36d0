// Around the tree decode, sm_103a: the ancestor masks of drafted trees, the
// page tables and slot map of a step, and the move of the accepted path's
// cache rows.
#include "fw_internal.h"
#include "fw_ptx.cuh"

namespace fw {
namespace {

constexpr int kErrInvalid = 1;     // FW_ERR_INVALID_ARG
constexpr int kErrWorkspace = 3;   // FW_ERR_WORKSPACE

// ---------------------------------------------------------------- tree masks
//
// mask(t) = {t} + mask(parent(t)), depth(t) = depth(parent(t)) + 1.  One block
// per tree, one thread per node, by pointer doubling: with up(t) the 2^r-th
// ancestor and m_r(t) the first 2^r nodes of the way up from t,
//   m_{r+1}(t) = m_r(t) | m_r(up(t)),   up'(t) = up(up(t)),
// which a tree of depth d finishes after ceil(log2 d) rounds.  The launch bounds
// it: 1,024 trees of 121 nodes read 0.5 MB, write 2.4 MB.  (Walking up node by
// node spends some 25 instructions a step, and a thread's step is its warp's:
// 8.6 us at that size, against 4.1.)

constexpr int kMaxTree = 256;

template <int W>                                     // words of a node's mask kept, T <= 32 W
__global__ void __launch_bounds__(kMaxTree) tree_mask_kernel(const __grid_constant__ TreeMaskParams p) {
    __shared__ uint32_t words[2][32 * W][W];
    __shared__ int up[2][32 * W], steps[2][32 * W];
    const int b = blockIdx.x, t = threadIdx.x;
    const int d = p.draft_lens ? min(max(__ldg(p.draft_lens + b), 0), p.T) : p.T;
    uint32_t w[W];
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = 0;
    int u = -1, n = 0;                               // the next node to take in, nodes taken
    if (t < d) {
        u = __ldg(p.parents + b * p.parent_stride + t);
        if (u < -1 || u >= t) {
            record_error(p.status, kErrInvalid);
            u = -1;
        }
#pragma unroll
        for (int i = 0; i < W; ++i)
            if (t >> 5 == i) w[i] = 1u << (t & 31);
        n = 1;
    }
    for (int r = 0; __syncthreads_or(u >= 0); r ^= 1) {
#pragma unroll
        for (int i = 0; i < W; ++i) words[r][t][i] = w[i];
        up[r][t] = u;
        steps[r][t] = n;
        __syncthreads();
        if (u >= 0) {
#pragma unroll
            for (int i = 0; i < W; ++i) w[i] |= words[r][u][i];
            n += steps[r][u];
            u = up[r][u];
        }
    }
    if (t >= p.T) return;
    int32_t *row = p.mask + b * p.mask_stride[0] + t * p.mask_stride[1];
    if (W == 4 && p.W == 4 && ((reinterpret_cast<uintptr_t>(row) & 15) == 0)) {
        *reinterpret_cast<uint4 *>(row) = make_uint4(w[0], w[W > 1 ? 1 : 0], w[W > 2 ? 2 : 0], w[W > 3 ? 3 : 0]);
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i)
            if (i < p.W) row[i] = (int32_t)w[i];
        for (int i = W; i < p.W; ++i) row[i] = 0;
    }
    if (p.depths) p.depths[b * p.depth_stride + t] = n - 1;
}

// --------------------------------------------------------------- page tables
//
// need(b) = max(0, ceil(seq/ps) - held), back(b) = max(0, held - ceil(seq/ps));
// their exclusive prefix sums over the requests (and those of new_lens) place
// every page and every token, so all entries can be written at once: entry k
// of a list belongs to the last request whose prefix is <= k.  Every block
// computes the three prefixes for itself, which takes less time than a second
// launch that waits for a first, and writes one contiguous share of each list,
// so that its searches span a few requests.  Measured: a decode step of 32 requests
// 5.0 us, all of it latencies; the maps of 2,048 prompts (7.9 M places, 0.5 M pages)
// 17.4 us, of which the sums take 3.6, the stores of 32 MB 8.

struct TableRow {
    int seq, fresh, held, want;
    bool ok;
};

// x / page size.  (A 64-bit division, which the sums below could call for too,
// takes a microsecond.)
__device__ __forceinline__ uint32_t pages_of(const PageTableParams &p, uint32_t x) {
    return p.ps_shift >= 0 ? x >> p.ps_shift : x / (uint32_t)p.ps;
}

__device__ __forceinline__ TableRow table_row(const PageTableParams &p, int b) {
    TableRow r;
    r.seq = __ldg(p.seq_lens + b);
    r.fresh = __ldg(p.new_lens + b);
    r.held = __ldg(p.held + b);
    r.ok = r.seq >= 0 && r.seq <= (int64_t)p.max_pages * p.ps && r.fresh >= 0 && r.fresh <= r.seq && r.held >= 0 &&
           r.held <= p.max_pages && !(p.padded && r.fresh > p.L);
    r.want = r.ok ? (int)pages_of(p, (uint32_t)r.seq + (uint32_t)(p.ps - 1)) : r.held;
    return r;
}

// Exclusive prefix over the block's threads of three sums, and their totals.
__device__ void block_prefix3(long long (&v)[3], long long (&total)[3], long long *warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    long long incl[3];
#pragma unroll
    for (int c = 0; c < 3; ++c) {
        incl[c] = v[c];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, incl[c], o);
            if (lane >= o) incl[c] += u;
        }
        if (lane == 31) warp_sums[c * 32 + warp] = incl[c];
    }
    __syncthreads();
    if (warp < 3) {
        long long w = lane < nwarps ? warp_sums[warp * 32 + lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += u;
        }
        warp_sums[warp * 32 + lane] = w;
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 3; ++c) {
        total[c] = warp_sums[c * 32 + 31];
        v[c] = incl[c] - v[c] + (warp > 0 ? warp_sums[c * 32 + warp - 1] : 0);
    }
}

__device__ __forceinline__ int clamp31(long long v) { return v > 0x7fffffffll ? 0x7fffffff : (int)v; }

// Last index b in [lo, hi] with prefix[b] <= k, prefix[lo] <= k.
__device__ __forceinline__ int prefix_row(const int *prefix, int lo, int hi, int k) {
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= k) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// A block's share [begin, end) of n entries, in whole octets, and the rows
// its first and last entry belong to: the threads then search between those.
struct Share {
    int begin, end, row0, row1;
};
__device__ __forceinline__ Share block_share(const int *prefix, int B, int n) {
    Share s;
    const uint32_t per = (((uint32_t)n + gridDim.x - 1) / gridDim.x + 7) & ~7u;
    s.begin = (int)min((uint64_t)n, (uint64_t)per * blockIdx.x);
    s.end = (int)min((uint64_t)n, (uint64_t)per * (blockIdx.x + 1));
    s.row0 = s.row1 = 0;
    if (gridDim.x == 1) {
        s.row1 = B - 1;
    } else if (s.begin < s.end) {
        s.row0 = prefix_row(prefix, 0, B - 1, s.begin);
        s.row1 = prefix_row(prefix, s.row0, B - 1, s.end - 1);
    }
    return s;
}
constexpr int kTableThreads = 1024;                 // most of a block

// kFill: writes the table, the ring and the slots; write_state: writes held_out
// and range_out.
template <bool kFill>
__global__ void __launch_bounds__(kTableThreads) page_table_kernel(const __grid_constant__ PageTableParams p,
                                                                   int write_state, int octets) {
    extern __shared__ int smem_i[];
    int *tok = smem_i;                 // [B + 1] exclusive prefixes
    int *need = tok + p.B + 1;         // [B + 1]
    int *back = need + p.B + 1;        // [B + 1]
    int *first = back + p.B + 1;       // [B] position of the request's first new token
    int *kept = first + p.B;           // [B] pages held before, -1: no slots
    __shared__ long long warp_sums[96];
    __shared__ int s_taken, s_back;
    const int tid = threadIdx.x, nthreads = blockDim.x;
    int head = __ldg(p.range), count = __ldg(p.range + 1);
    const bool range_ok = head >= 0 && head < p.F && count >= 0 && count <= p.F;
    const int room = range_ok ? p.F - count : 0;
    const int head0 = head, count0 = count;
    if (!range_ok) { head = 0; count = 0; }
    const int per = (p.B + nthreads - 1) / nthreads;
    long long v[3] = {0, 0, 0}, total[3];
    bool bad = !range_ok;
#pragma unroll 1
    for (int b = tid * per; b < min(p.B, (tid + 1) * per); ++b) {
        const TableRow r = table_row(p, b);
        bad |= !r.ok;
        v[0] += max(r.fresh, 0);
        v[1] += max(r.want - r.held, 0);
        v[2] += max(r.held - r.want, 0);
    }
    if (tid == 0) { s_taken = 0; s_back = 0; }
    block_prefix3(v, total, warp_sums);
    int taken = 0, given = 0;
#pragma unroll 1
    for (int b = tid * per; b < min(p.B, (tid + 1) * per); ++b) {
        const TableRow r = table_row(p, b);
        // (Padded places need the rows' own counts alone, which wrapped sums still give
        // behind a contradictory count.)
        tok[b] = p.padded ? (int)v[0] : clamp31(v[0]);
        if (kFill && p.cu_new && blockIdx.x == 0) p.cu_new[b] = clamp31(v[0]);
        need[b] = clamp31(v[1]);
        back[b] = clamp31(v[2]);
        v[0] += max(r.fresh, 0);
        v[1] += max(r.want - r.held, 0);
        v[2] += max(r.held - r.want, 0);
        const bool served = r.want <= r.held || v[1] <= count;
        first[b] = r.seq - r.fresh;
        kept[b] = r.ok && served ? r.held : -1;
        if (r.want > r.held && served) taken = clamp31(v[1]);
        if (r.want < r.held && v[2] <= room) given = clamp31(v[2]);
        bad |= r.want < r.held && v[2] > room;
        if (!served && range_ok && blockIdx.x == 0 && kFill) record_error(p.status, kErrWorkspace);
    }
    if (taken) atomicMax(&s_taken, taken);
    if (given) atomicMax(&s_back, given);
    if (tid == 0) {
        tok[p.B] = p.padded ? (int)total[0] : clamp31(total[0]);
        if (kFill && p.cu_new && blockIdx.x == 0) p.cu_new[p.B] = clamp31(total[0]);
        need[p.B] = clamp31(total[1]);
        back[p.B] = clamp31(total[2]);
        bad |= !p.padded && total[0] > p.N;
    }
    if (bad && blockIdx.x == 0 && kFill) record_error(p.status, kErrInvalid);
    __syncthreads();
    taken = s_taken;
    given = s_back;

    if constexpr (kFill) {
        // (Everything below is rolled: a launch runs each loop a few times, and
        // instructions not yet in the SM's cache cost more than those executed.)
        const int limit = 0x7fffffff / p.ps;          // a page whose slots all fit in 32 bits is below it
        auto wrapped = [&](uint32_t e) -> int {       // e < 3 F
            while (e >= (uint32_t)p.F) e -= p.F;
            return (int)e;
        };
        // Page l of request b after the step.
        auto page_of = [&](int b, int l) -> int {
            const int h = kept[b];
            return l < h ? p.table[b * p.table_stride + l] : p.queue[wrapped((uint32_t)head + need[b] + (l - h))];
        };
        auto slot_of = [&](int i, int b) -> int {     // place i, in request b
            const int j = p.padded ? i - b * p.L : i - tok[b];
            if (kept[b] < 0 || j >= (p.padded ? tok[b + 1] - tok[b] : p.N)) return -1;
            const int pos = first[b] + j, lp = (int)pages_of(p, (uint32_t)pos);
            const int page = page_of(b, lp);
            if (page >= 0 && page < limit) return page * p.ps + (pos - lp * p.ps);
            record_error(p.status, kErrInvalid);
            return -1;
        };
        const int live = p.padded ? p.N : min(p.N, tok[p.B]);      // behind it: no token
        // A warp takes a run of a list, so that its rows follow one another and the
        // search is repeated only where a row ends (a search an entry took 18.6 us for
        // the maps of 2,048 prompts, this 17.4; a decode step's 6.1, this 5.0).  The
        // last warps take the first pages, the first warps the first places: a short
        // step's two lookups then wait side by side.
        const int lane = tid & 31, warp = tid >> 5, nwarps = nthreads >> 5;
        if (taken > 0) {
            const Share s = block_share(need, p.B, taken);
            const int run = ((s.end - s.begin + nwarps - 1) / nwarps + 31) & ~31;
            const int k0 = s.begin + (nwarps - 1 - warp) * run, k1 = min(s.end, k0 + run);
            int b = s.row0, upto = s.begin, at = 0;
            int64_t row = 0;
#pragma unroll 1
            for (int k = k0 + lane; k < k1; k += 32) {
                if (k >= upto) {
                    b = prefix_row(need, b, s.row1, k);
                    upto = need[b + 1];
                    at = kept[b] - need[b];
                    row = b * p.table_stride;
                }
                p.table[row + at + k] = p.queue[wrapped((uint32_t)head + k)];
            }
        }
        if (given > 0) {
            const Share s = block_share(back, p.B, given);
#pragma unroll 1
            for (int k = s.begin + tid; k < s.end; k += nthreads) {
                const int b = prefix_row(back, s.row0, s.row1, k);
                p.queue[wrapped((uint32_t)head + count + k)] =
                    p.table[b * p.table_stride + table_row(p, b).want + (k - back[b])];
            }
        }
        if (!octets) {
#pragma unroll 1
            for (int i = blockIdx.x * nthreads + tid; i < p.N; i += gridDim.x * nthreads) {
                int slot = -1;
                if (i < live) slot = slot_of(i, p.padded ? i / p.L : prefix_row(tok, 0, p.B - 1, i));
                p.slots[i] = slot;
            }
        } else {
            // Eight places to a thread, one 32-byte store: within one request they lie
            // in at most two pages.  (With four places to a thread 11 us for 7.9 M, with
            // eight 7 to 8, 4 TB/s of stores, which more lookups in flight do not
            // raise.)  An octet that a request ends in is left to a second pass, a
            // thread to a place; one by one are done those with a page that cannot be
            // named, and the last of all.
            const Share s = block_share(tok, p.padded ? 0 : p.B, live);
            const int run = ((s.end - s.begin + nwarps - 1) / nwarps + 7) & ~7;
            const int i0 = s.begin + warp * run, i1 = min(s.end, i0 + run);
            int b = s.row0, upto = 0, from = 0, h = 0, fresh = 0, at = 0;
#pragma unroll 1
            for (int i = i0 + 8 * lane; i < i1; i += 256) {
                if (i >= upto) {
                    b = p.padded ? i / p.L : prefix_row(tok, b, s.row1, i);
                    from = p.padded ? b * p.L : tok[b];
                    upto = p.padded ? from + p.L : tok[b + 1];
                    fresh = tok[b + 1] - tok[b];
                    h = kept[b];
                    at = first[b];
                }
                const int j = i - from;
                const int left = fresh - j;                           // tokens of the request from here on
                if (left < 8 && i + 8 <= s.end && !p.padded) continue;
                if (h >= 0 && left >= 8) {
                    const int pos = at + j, lp = (int)pages_of(p, (uint32_t)pos);
                    const int off = pos - lp * p.ps, in = p.ps - off;    // places in the first page
                    const int page = page_of(b, lp);
                    const int page2 = in < 8 ? page_of(b, lp + 1) : page;
                    if (page >= 0 && page < limit && page2 >= 0 && page2 < limit) {
                        const int x = page * p.ps + off, y = page2 * p.ps - in;
                        int o[8];
#pragma unroll
                        for (int q = 0; q < 8; ++q) o[q] = (q < in ? x : y) + q;
                        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p.slots + i),
                                     "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                                     : "memory");
                        continue;
                    }
                }
#pragma unroll 1
                for (int q = i; q < min(i + 8, s.end); ++q)
                    p.slots[q] = slot_of(q, p.padded ? b : prefix_row(tok, b, s.row1, q));
            }
            if (!p.padded && s.begin < s.end) {
#pragma unroll 1
                for (int k = 8 * s.row0 + tid; k < 8 * (s.row1 + 1); k += nthreads) {
                    const int b = k >> 3;
                    const int i = ((tok[b + 1] - 1) & ~7) + (k & 7);
                    if (tok[b + 1] == tok[b] || i < s.begin || i >= s.end) continue;
                    p.slots[i] = slot_of(i, prefix_row(tok, s.row0, s.row1, i));
                }
            }
            // Behind the last token.
            const uint32_t per_block = ((uint32_t)(p.N - live) + gridDim.x - 1) / gridDim.x;
            const int64_t b0 = live + (int64_t)per_block * blockIdx.x;
#pragma unroll 1
            for (int64_t i = b0 + tid; i < min((int64_t)p.N, b0 + per_block); i += nthreads) p.slots[i] = -1;
        }
    }
    if (write_state && blockIdx.x == 0) {
        if constexpr (!kFill) pdl_wait();             // the fill has read what this overwrites
        __syncthreads();
        // Every value is read before the barrier that precedes the writes:
        // the outputs may be the inputs.
#pragma unroll 1
        for (int b0 = 0; b0 < p.B; b0 += nthreads) {
            const int b = b0 + tid;
            int h = 0;
            if (b < p.B) {
                const TableRow r = table_row(p, b);
                const bool grown = r.want > r.held && need[b + 1] <= count;
                const bool shrunk = r.want < r.held && back[b + 1] <= room;
                h = grown || shrunk ? r.want : r.held;
            }
            __syncthreads();
            if (b < p.B) p.held_out[b] = h;
        }
        if (tid == 0) {
            int h = head + taken;
            if (range_ok && h >= p.F) h -= p.F;
            p.range_out[0] = range_ok ? h : head0;
            p.range_out[1] = range_ok ? count - taken + given : count0;
        }
    }
}

// ---------------------------------------------------------------- path commit
//
// Row base + i takes row base + path[i], i ascending: path[i] >= i and the path
// increases, so a row is read before anything is moved into it as long as one
// thread moves a 16-byte column's rows in order -- and it may read rows i .. i + 3
// before it writes them, since row base + path[i + 3] is written later still, if
// at all.  A block checks one request's path and looks its pages up once, then
// takes every gridDim.y-th layer, two at a time: a thread has up to eight rows in
// flight.  Measured: 192 requests, 6 accepted drafts, 32 layers of 8 heads of dim
// 128, 101 MB read and written, 24.5 us out of L2, 0.61 of the measured copy rate
// (19.4 us over again on one cache, which L2 holds most of): two or three rounds of
// layers a block, each a round trip to memory behind path, table and lengths; 8
// requests in one layer 3.9 us, the launch and three dependent reads.

constexpr int kCommitThreads = 256;
constexpr int kCommitRows = 256;                     // longest path

struct Move {
    int src_page, src_off, dst_page, dst_off;        // page < 0: stays where it is
};

__global__ void __launch_bounds__(kCommitThreads) kv_commit_kernel(const __grid_constant__ CommitParams p) {
    __shared__ Move moves[kCommitRows];
    __shared__ int count;
    const int b = blockIdx.x, tid = threadIdx.x;
    const int base = __ldg(p.base_lens + b);
    const int m = __ldg(p.path_lens + b);
    const int32_t *path = p.path + b * p.path_stride;
    const int32_t *table = p.table + b * p.table_stride;
    const int64_t cap = (int64_t)p.max_pages * p.ps;
    bool ok = base >= 0 && m >= 0 && m <= p.A;
    if (ok && tid < m) {
        const int s = __ldg(path + tid);
        const int before = tid > 0 ? __ldg(path + tid - 1) : -1;
        ok = s > before && (int64_t)base + s < cap;
        Move mv;
        mv.src_page = -1;
        if (ok && s != tid) {
            const int from = base + s, to = base + tid;
            mv.src_page = __ldg(table + from / p.ps);
            mv.src_off = from % p.ps;
            mv.dst_page = __ldg(table + to / p.ps);
            mv.dst_off = to % p.ps;
            ok = mv.src_page >= 0 && mv.src_page < p.layer_pages && mv.dst_page >= 0 && mv.dst_page < p.layer_pages;
        }
        moves[tid] = mv;
    }
    // The rows at the path's start that are in place need no move: since the path
    // increases, they are the first ones.
    if (tid == 0) count = 0;
    ok = __syncthreads_and(ok);
    if (tid == 0 && blockIdx.y == 0 && blockIdx.z == 0) {
        if (p.new_lens) p.new_lens[b] = ok ? base + m : base;
        if (!ok) record_error(p.status, kErrInvalid);
    }
    if (!ok) return;
    if (tid < m && moves[tid].src_page < 0) atomicAdd(&count, 1);
    __syncthreads();
    const int first = count;
    if (first >= m) return;
    const int kcols = p.Hkv * p.k_units, cols = kcols + p.Hkv * p.v_units;
    const int c = blockIdx.z * kCommitThreads + tid;
    if (c >= cols) return;
    const bool isv = c >= kcols;
    const int units = isv ? p.v_units : p.k_units;
    const int cc = isv ? c - kcols : c;
    const int h = cc / units;
    const int64_t st0 = isv ? p.vc_stride[0] : p.kc_stride[0], st1 = isv ? p.vc_stride[1] : p.kc_stride[1];
    char *col = static_cast<char *>(isv ? p.v_cache : p.k_cache) + h * (isv ? p.vc_stride[2] : p.kc_stride[2]) +
                (int64_t)(cc - h * units) * 16;
    const int64_t next = (int64_t)gridDim.y * p.layer_pages * st0;      // to the block's next layer
    for (int layer = blockIdx.y; layer < p.layers; layer += 2 * gridDim.y) {
        char *at = col + (int64_t)layer * p.layer_pages * st0;
        const bool two = layer + (int)gridDim.y < p.layers;
        for (int i = first; i < m; i += 4) {
            uint4 v[2][4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i + k < m) {
                    const char *src = at + moves[i + k].src_page * st0 + moves[i + k].src_off * st1;
                    v[0][k] = *reinterpret_cast<const uint4 *>(src);
                    if (two) v[1][k] = *reinterpret_cast<const uint4 *>(src + next);
                }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i + k < m) {
                    char *dst = at + moves[i + k].dst_page * st0 + moves[i + k].dst_off * st1;
                    *reinterpret_cast<uint4 *>(dst) = v[0][k];
                    if (two) *reinterpret_cast<uint4 *>(dst + next) = v[1][k];
                }
        }
    }
}

}  // namespace

cudaError_t launch_tree_mask(const TreeMaskParams &p, cudaStream_t stream) {
    const int threads = (p.T + 31) / 32 * 32;
    if (threads <= 32) tree_mask_kernel<1><<<p.B, threads, 0, stream>>>(p);
    else if (threads <= 64) tree_mask_kernel<2><<<p.B, threads, 0, stream>>>(p);
    else if (threads <= 128) tree_mask_kernel<4><<<p.B, threads, 0, stream>>>(p);
    else tree_mask_kernel<8><<<p.B, threads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_page_tables(const PageTableParams &p, cudaStream_t stream, int *launches) {
    *launches = 0;
    const size_t smem = ((size_t)5 * p.B + 3) * sizeof(int);
    static bool configured[64] = {};                 // by device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!configured[dev & 63]) {
        const int most = (5 * kMaxTableRows + 3) * (int)sizeof(int);
        e = cudaFuncSetAttribute(page_table_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(page_table_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e != cudaSuccess) return e;
        configured[dev & 63] = true;
    }
    // A place to a thread as long as the GPU's blocks have enough of them (the
    // shortest way for the maps of a decode step); beyond, octets where they can
    // be stored as vectors.  Pages are a list of their own: a step that takes
    // or returns many for few places needs the blocks too.
    const int threads = p.N <= 256 && p.B <= 256 ? 256 : kTableThreads;
    const int64_t pages = (int64_t)p.B * p.max_pages < p.F ? (int64_t)p.B * p.max_pages : p.F;
    int64_t blocks = ((int64_t)p.N + threads - 1) / threads;
    const int octets = blocks > p.num_sms && p.ps >= 8 && (!p.padded || p.L % 8 == 0) &&
                       reinterpret_cast<uintptr_t>(p.slots) % 32 == 0;
    if (blocks < (pages + 65535) / 65536) blocks = (pages + 65535) / 65536;
    const unsigned grid = (unsigned)(blocks < 1 ? 1 : blocks > p.num_sms ? p.num_sms : blocks);
    // With one block the reads of the outputs' old values are over before the
    // writes; several blocks read them at their own time, so the state is then
    // written by a launch that waits for the fill.
    const bool split = p.in_place && grid > 1;
    page_table_kernel<true><<<grid, threads, smem, stream>>>(p, split ? 0 : 1, octets);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    ++*launches;
    if (split) {
        e = launch_after_previous(page_table_kernel<false>, dim3(1), dim3(threads), smem, stream, p, 1, 0);
        if (e != cudaSuccess) return e;
        ++*launches;
    }
    return cudaSuccess;
}

cudaError_t launch_kv_commit(const CommitParams &p, cudaStream_t stream) {
    const int cols = p.Hkv * (p.k_units + p.v_units);
    const int z = (cols + kCommitThreads - 1) / kCommitThreads;
    const int64_t fill = 8ll * p.num_sms;             // blocks of 256 threads the GPU holds
    int64_t y = (fill + (int64_t)p.B * z - 1) / ((int64_t)p.B * z);
    if (y > p.layers) y = p.layers;
    kv_commit_kernel<<<dim3(p.B, (unsigned)y, z), kCommitThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace fw
