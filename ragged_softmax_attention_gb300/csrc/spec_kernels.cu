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
// per tree, one thread per node, each walking up its ancestors.

constexpr int kMaxTree = 256;

__global__ void __launch_bounds__(kMaxTree) tree_mask_kernel(const __grid_constant__ TreeMaskParams p) {
    __shared__ int parent[kMaxTree];
    const int b = blockIdx.x, t = threadIdx.x;
    const int d = p.draft_lens ? min(max(__ldg(p.draft_lens + b), 0), p.T) : p.T;
    if (t < p.T) {
        int u = __ldg(p.parents + b * p.parent_stride + t);
        if (u < -1 || u >= t) {
            if (t < d) record_error(p.status, kErrInvalid);
            u = -1;
        }
        parent[t] = u;
    }
    __syncthreads();
    if (t >= p.T) return;
    uint32_t w[kMaxTree / 32];
#pragma unroll
    for (int i = 0; i < kMaxTree / 32; ++i) w[i] = 0;
    int depth = -1;
    if (t < d) {
        for (int u = t; u >= 0; u = parent[u], ++depth) {
#pragma unroll
            for (int i = 0; i < kMaxTree / 32; ++i)
                if (u >> 5 == i) w[i] |= 1u << (u & 31);
        }
    }
    int32_t *row = p.mask + b * p.mask_stride[0] + t * p.mask_stride[1];
#pragma unroll
    for (int i = 0; i < kMaxTree / 32; ++i)
        if (i < p.W) row[i] = (int32_t)w[i];
    for (int i = kMaxTree / 32; i < p.W; ++i) row[i] = 0;
    if (p.depths) p.depths[b * p.depth_stride + t] = depth;
}

// --------------------------------------------------------------- page tables
//
// need(b) = max(0, ceil(seq/ps) - held), back(b) = max(0, held - ceil(seq/ps));
// their exclusive prefix sums over the requests (and those of new_lens) place
// every page and every token, so all entries can be written at once: entry k
// of a list belongs to the last request whose prefix is <= k.  Every block
// computes the three prefixes for itself, which takes less time than a second
// launch that waits for a first.

struct TableRow {
    int seq, fresh, held, want;
    bool ok;
};

__device__ __forceinline__ TableRow table_row(const PageTableParams &p, int b) {
    TableRow r;
    r.seq = __ldg(p.seq_lens + b);
    r.fresh = __ldg(p.new_lens + b);
    r.held = __ldg(p.held + b);
    r.ok = r.seq >= 0 && r.seq <= (int64_t)p.max_pages * p.ps && r.fresh >= 0 && r.fresh <= r.seq && r.held >= 0 &&
           r.held <= p.max_pages && !(p.padded && r.fresh > p.L);
    r.want = r.ok ? (int)(((int64_t)r.seq + p.ps - 1) / p.ps) : r.held;
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

// Last index b in [0, n) with prefix[b] <= k (prefix[0] = 0).
__device__ __forceinline__ int prefix_row(const int *prefix, int n, int k) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= k) lo = mid; else hi = mid - 1;
    }
    return lo;
}

constexpr int kTableThreads = 1024;

// kFill: writes the table, the ring and the slots; write_state: writes held_out
// and range_out.
template <bool kFill>
__global__ void __launch_bounds__(kTableThreads) page_table_kernel(const __grid_constant__ PageTableParams p,
                                                                   int write_state) {
    extern __shared__ int smem_i[];
    int *tok = smem_i;                 // [B + 1] exclusive prefixes
    int *need = tok + p.B + 1;
    int *back = need + p.B + 1;
    __shared__ long long warp_sums[96];
    __shared__ int s_taken, s_back;
    const int tid = threadIdx.x;
    int head = __ldg(p.range), count = __ldg(p.range + 1);
    const bool range_ok = head >= 0 && head < p.F && count >= 0 && count <= p.F;
    const int room = range_ok ? p.F - count : 0;
    const int head0 = head, count0 = count;
    if (!range_ok) { head = 0; count = 0; }
    const int per = (p.B + kTableThreads - 1) / kTableThreads;
    long long v[3] = {0, 0, 0}, total[3];
    bool bad = !range_ok;
    for (int i = 0; i < per; ++i) {
        const int b = tid * per + i;
        if (b >= p.B) break;
        const TableRow r = table_row(p, b);
        bad |= !r.ok;
        v[0] += max(r.fresh, 0);
        v[1] += max(r.want - r.held, 0);
        v[2] += max(r.held - r.want, 0);
    }
    if (tid == 0) { s_taken = 0; s_back = 0; }
    block_prefix3(v, total, warp_sums);
    int taken = 0, given = 0;
    for (int i = 0; i < per; ++i) {
        const int b = tid * per + i;
        if (b >= p.B) break;
        const TableRow r = table_row(p, b);
        tok[b] = clamp31(v[0]);
        need[b] = clamp31(v[1]);
        back[b] = clamp31(v[2]);
        v[0] += max(r.fresh, 0);
        v[1] += max(r.want - r.held, 0);
        v[2] += max(r.held - r.want, 0);
        if (r.want > r.held && v[1] <= count) taken = clamp31(v[1]);
        if (r.want < r.held && v[2] <= room) given = clamp31(v[2]);
        bad |= r.want < r.held && v[2] > room;
        if (r.want > r.held && v[1] > count && range_ok && blockIdx.x == 0 && kFill)
            record_error(p.status, kErrWorkspace);
    }
    if (taken) atomicMax(&s_taken, taken);
    if (given) atomicMax(&s_back, given);
    if (tid == 0) {
        tok[p.B] = clamp31(total[0]);
        need[p.B] = clamp31(total[1]);
        back[p.B] = clamp31(total[2]);
        bad |= !p.padded && total[0] > p.N;
    }
    if (bad && blockIdx.x == 0 && kFill) record_error(p.status, kErrInvalid);
    __syncthreads();
    taken = s_taken;
    given = s_back;

    if constexpr (kFill) {
        const int nthreads = gridDim.x * kTableThreads;
        const int gt = blockIdx.x * kTableThreads + tid;
        for (int k = gt; k < taken; k += nthreads) {
            const int b = prefix_row(need, p.B, k);
            int e = head + k;
            if (e >= p.F) e -= p.F;
            p.table[b * p.table_stride + __ldg(p.held + b) + (k - need[b])] = p.queue[e];
        }
        for (int k = gt; k < given; k += nthreads) {
            const int b = prefix_row(back, p.B, k);
            int e = head + count + k;                 // < 3 F: the ring's end, then the returned pages
            while (e >= p.F) e -= p.F;
            p.queue[e] = p.table[b * p.table_stride + table_row(p, b).want + (k - back[b])];
        }
        const int limit = 0x7fffffff / p.ps;          // a page whose slots all fit in 32 bits is below it
        for (int64_t i = gt; i < p.N; i += nthreads) {
            int b, j;
            if (p.padded) {
                b = (int)(i / p.L);
                j = (int)(i - (int64_t)b * p.L);
            } else if (i < tok[p.B]) {
                b = prefix_row(tok, p.B, (int)i);
                j = (int)i - tok[b];
            } else {                                  // behind the last token (every place when B = 0)
                p.slots[i] = -1;
                continue;
            }
            const TableRow r = table_row(p, b);
            int slot = -1;
            if (j < r.fresh && r.ok && (r.want <= r.held || need[b + 1] <= count)) {
                const int pos = r.seq - r.fresh + j;
                const int lp = pos / p.ps;
                int page;
                if (lp < r.held) {
                    page = p.table[b * p.table_stride + lp];
                } else {
                    int e = head + need[b] + lp - r.held;
                    if (e >= p.F) e -= p.F;
                    page = p.queue[e];
                }
                if (page >= 0 && page < limit) slot = page * p.ps + (pos - lp * p.ps);
                else record_error(p.status, kErrInvalid);
            }
            p.slots[i] = slot;
        }
        if (blockIdx.x == 0 && p.cu_new)
            for (int b = tid; b <= p.B; b += kTableThreads) p.cu_new[b] = tok[b];
    }
    if (write_state && blockIdx.x == 0) {
        if constexpr (!kFill) pdl_wait();             // the fill has read what this overwrites
        __syncthreads();
        // Every value is read before the barrier that precedes the writes:
        // the outputs may be the inputs.
        for (int b0 = 0; b0 < p.B; b0 += kTableThreads) {
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
// Row base + i takes row base + path[i], i ascending: path[i] >= i, so a row is
// read before anything is moved into it as long as one thread moves a column's
// rows in order.  One block per (request, layer); one thread per 16-byte
// column of the K or V rows.

constexpr int kCommitThreads = 256;

__global__ void __launch_bounds__(kCommitThreads) kv_commit_kernel(const __grid_constant__ CommitParams p) {
    const int b = blockIdx.x, layer = blockIdx.y;
    const int base = __ldg(p.base_lens + b);
    const int m = __ldg(p.path_lens + b);
    const int32_t *path = p.path + b * p.path_stride;
    const int32_t *table = p.table + b * p.table_stride;
    const int64_t cap = (int64_t)p.max_pages * p.ps;
    bool ok = base >= 0 && m >= 0 && m <= p.A;
    if (ok) {
        for (int i = threadIdx.x; i < m; i += kCommitThreads) {
            const int s = __ldg(path + i);
            bool good = s >= i && (i == 0 || __ldg(path + i - 1) < s) && (int64_t)base + s < cap;
            if (good && s != i) {
                const int ps_ = __ldg(table + (base + s) / p.ps), pd = __ldg(table + (base + i) / p.ps);
                good = ps_ >= 0 && ps_ < p.layer_pages && pd >= 0 && pd < p.layer_pages;
            }
            ok &= good;
        }
    }
    ok = __syncthreads_and(ok);
    if (threadIdx.x == 0 && layer == 0 && blockIdx.z == 0) {
        if (p.new_lens) p.new_lens[b] = ok ? base + m : base;
        if (!ok) record_error(p.status, kErrInvalid);
    }
    if (!ok) return;
    const int kcols = p.Hkv * p.k_units, cols = kcols + p.Hkv * p.v_units;
    for (int c = blockIdx.z * kCommitThreads + threadIdx.x; c < cols; c += gridDim.z * kCommitThreads) {
        const bool isv = c >= kcols;
        const int units = isv ? p.v_units : p.k_units;
        const int cc = isv ? c - kcols : c;
        const int h = cc / units;
        const int64_t *st = isv ? p.vc_stride : p.kc_stride;
        char *col = static_cast<char *>(isv ? p.v_cache : p.k_cache) + (int64_t)layer * p.layer_pages * st[0] +
                    h * st[2] + (int64_t)(cc - h * units) * 16;
        for (int i = 0; i < m; ++i) {
            const int s = __ldg(path + i);
            if (s == i) continue;
            const int from = base + s, to = base + i;
            const int64_t src = __ldg(table + from / p.ps) * st[0] + (from % p.ps) * st[1];
            const int64_t dst = __ldg(table + to / p.ps) * st[0] + (to % p.ps) * st[1];
            *reinterpret_cast<uint4 *>(col + dst) = *reinterpret_cast<const uint4 *>(col + src);
        }
    }
}

}  // namespace

cudaError_t launch_tree_mask(const TreeMaskParams &p, cudaStream_t stream) {
    tree_mask_kernel<<<p.B, (p.T + 31) / 32 * 32, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_page_tables(const PageTableParams &p, cudaStream_t stream, int *launches) {
    *launches = 0;
    const size_t smem = (size_t)3 * (p.B + 1) * sizeof(int);
    static bool configured = false;
    if (!configured) {
        const int most = 3 * (16384 + 1) * (int)sizeof(int);
        cudaError_t e = cudaFuncSetAttribute(page_table_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(page_table_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e != cudaSuccess) return e;
        configured = true;
    }
    const int64_t blocks = ((int64_t)p.N + 4 * kTableThreads - 1) / (4 * kTableThreads);
    const unsigned grid = (unsigned)(blocks < 1 ? 1 : blocks > p.num_sms ? p.num_sms : blocks);
    // With one block the reads of the outputs' old values are over before the
    // writes; several blocks read them at their own time, so the state is then
    // written by a launch that waits for the fill.
    const bool split = p.in_place && grid > 1;
    page_table_kernel<true><<<grid, kTableThreads, smem, stream>>>(p, split ? 0 : 1);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    ++*launches;
    if (split) {
        e = launch_after_previous(page_table_kernel<false>, dim3(1), dim3(kTableThreads), smem, stream, p, 1);
        if (e != cudaSuccess) return e;
        ++*launches;
    }
    return cudaSuccess;
}

cudaError_t launch_kv_commit(const CommitParams &p, cudaStream_t stream) {
    const int cols = p.Hkv * (p.k_units + p.v_units);
    const int z = (cols + kCommitThreads - 1) / kCommitThreads;
    kv_commit_kernel<<<dim3(p.B, p.layers, z), kCommitThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace fw
