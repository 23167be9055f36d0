// Verification of drafted trees against the target's probabilities, sm_103a.
//
// At a node with the target's row p and the draft model's row q, its children are
// tried in order: child c is accepted with probability min(1, R(c) / (S q(c))),
// where R is what is left of p and S its sum; after a rejection
//   R <- max(R - S q, 0),  S <- sum R        (at first R = p, S = 1),
// and the walk goes on from the accepted child.  Where no child is accepted the next
// token is drawn from R: the first x with R(0) + .. + R(x) > u sum R.  Drafts so
// verified are distributed as the target's own samples (rejection sampling, one
// draft after another).  Without a draft model's rows a draft is taken as proposed
// with certainty, and R loses the token.
//
// A draw compares u with one of V running sums, and sums in 32 bits, or in an order
// that a split changes, would move the borders between neighbours by more than
// tokens of 1e-7 are wide.  Probabilities are therefore added as 64-bit integers in
// units of 2^-60 (a float of 2^-37 or more is held exactly): sums are exact, whatever
// their order, up to 4, where they stop.
//
// A cluster of CTAs takes a request.  What the walk compares, u, p and q at the drafts,
// is fetched at once and walked through by one thread; a whole row is only needed
// where a draft is rejected and at the end of the path, and is then summed by all
// CTAs, a segment to a warp, with the segments' sums left in shared memory, so that
// the draw looks again at one segment alone.  The walking thread tells the other CTAs
// what to do, so that they meet the same number of times whatever they read.
#include "fw_internal.h"
#include "fw_ptx.cuh"

namespace fw {
namespace {

constexpr int kErrInvalid = 1;     // FW_ERR_INVALID_ARG
constexpr int kVerifyThreads = 512, kVerifyWarps = kVerifyThreads / 32;
constexpr int kMaxDrafts = 256;
constexpr int kMaxCluster = 8;
typedef unsigned long long u64;
constexpr u64 kOne = 1ull << 60, kMost = 1ull << 62;

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// Stores to the same variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t remote(const void *p, uint32_t rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ void store_remote(const u64 *p, uint32_t rank, u64 v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(remote(p, rank)), "l"(v) : "memory");
}

// A probability in units of 2^-60; NaN and what is negative count as 0, more than 1 as 1.
__device__ __forceinline__ u64 fixed(float v) {
    if (!(v > 0.f)) return 0;
    if (v >= 1.f) return kOne;
    const uint32_t b = __float_as_uint(v);
    const int e = (int)(b >> 23) - 90;                    // 2^(exponent - 127 - 23) / 2^-60
    const u64 m = (b & 0x7fffffu) | 0x800000u;            // (a subnormal's is lost either way)
    return e >= 0 ? m << e : e > -24 ? m >> -e : 0;
}
__device__ __forceinline__ float clamped(float v) { return v > 0.f ? fminf(v, 1.f) : 0.f; }
// A uniform number in units of 2^-64.
__device__ __forceinline__ u64 fraction(float u) {
    if (!(u > 0.f)) return 0;
    return u >= 1.f ? ~0ull : __double2ull_rz((double)u * 18446744073709551616.0);
}
// What is left of p after n rejections, S[i] the sum before the i-th (S[0] = 1).
__device__ __forceinline__ u64 left_of(float p, float q, int n, const u64 *S) {
    u64 r = fixed(p);
    if (n > 0) {
        const u64 f = fixed(q);
        r = r > f ? r - f : 0;
        for (int i = 1; i < n; ++i) {
            const u64 s = __umul64hi(S[i] << 2, f << 2);
            r = r > s ? r - s : 0;
        }
    }
    return r;
}
__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = min(v + __shfl_xor_sync(0xffffffffu, v, o), kMost);
    return v;
}

// What the walking thread asks of the cluster.
struct Order {
    u64 row;               // row of the probabilities
    u64 n;                 // rejections there (with a draft model's rows)
    u64 sum;               // S[n - 1], n > 0
    u64 sweep;             // 1: the row's sums are wanted
    u64 last;              // 1: the path ends here, draw; 2: no row to draw from
    u64 gone[4];           // without a draft model's rows: drafts whose tokens are out, a bit each
};
constexpr int kOrderWords = sizeof(Order) / 8;

struct Shared {
    Order order;
    u64 sums[2][kMaxCluster];          // per CTA, of the last two sweeps
    u64 seg[kVerifyWarps];             // per warp, of the last sweep
    u64 S[kMaxDrafts + 1];
    u64 scan[kVerifyWarps];
    int token[kMaxDrafts], parent[kMaxDrafts], path[kMaxDrafts];
    float u[kMaxDrafts + 1], p[kMaxDrafts], q[kMaxDrafts];
    int count;
};

// A row as groups of four floats on 16-byte boundaries: group g holds x = 4 g - shift
// .. + 3.  Whole groups are one load where the draft model's row lies as the target's.
struct Rows {
    const float *p, *q;
    int V, shift, groups;
    bool q_wide;
    __device__ Rows(const VerifyParams &a, int b, int row) {
        p = a.target + b * a.target_stride[0] + row * a.target_stride[1];
        q = a.draft ? a.draft + b * a.draft_stride[0] + row * a.draft_stride[1] : nullptr;
        V = a.V;
        shift = (int)(reinterpret_cast<uintptr_t>(p) >> 2 & 3);
        q_wide = (int)(reinterpret_cast<uintptr_t>(q) >> 2 & 3) == shift;
        groups = (V + shift + 3) >> 2;
    }
    __device__ __forceinline__ float4 load(const float *r, bool wide, int g) const {
        const int x = 4 * g - shift;
        if (wide && x >= 0 && x + 3 < V) return __ldg(reinterpret_cast<const float4 *>(r + x));
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (x >= 0 && x < V) v.x = __ldg(r + x);
        if (x + 1 >= 0 && x + 1 < V) v.y = __ldg(r + x + 1);
        if (x + 2 >= 0 && x + 2 < V) v.z = __ldg(r + x + 2);
        if (x + 3 >= 0 && x + 3 < V) v.w = __ldg(r + x + 3);
        return v;
    }
};

// The walk, by one thread: runs until it needs a row's sums or has reached its end.
struct Walk {
    int t, cur, count, n;                  // next draft, node, accepted drafts, rejections at the node
    bool stuck;                            // nothing would be left: rejections change nothing more
    int pending;                           // the rejected child whose sums are under way, -1: none
    u64 total, full;                       // S; without a draft model's rows the row's sum
    u64 gone[4];
    int have_row, have_n;                  // what the segments' sums are of

    __device__ void enter(int node) {
        cur = node;
        n = 0;
        stuck = false;
        total = kOne;
        have_row = have_n = -1;
        for (int w = 0; w < 4; ++w) gone[w] = 0;
    }
    __device__ bool is_out(const Shared &sh, int tok) const {
        for (int w = 0; w < 4; ++w)
            for (u64 m = gone[w]; m; m &= m - 1)
                if (sh.token[64 * w + __ffsll((long long)m) - 1] == tok) return true;
        return false;
    }
    // Child c's token leaves R (no draft model's rows).
    __device__ void take_out(const Shared &sh, int c) {
        const u64 x = is_out(sh, sh.token[c]) ? 0 : fixed(sh.p[c]);
        if (full <= x) return;
        full -= x;
        total = full;
        if (x > 0) gone[c >> 6] |= 1ull << (c & 63);
    }
    __device__ void run(const VerifyParams &a, Shared &sh, int T, const u64 *sums, int C, Order &o) {
        o = Order{};
        if (pending >= 0) {
            u64 s = 0;
            for (int r = 0; r < C; ++r) s = min(s + sums[r], kMost);
            if (a.draft) {
                if (s > 0) sh.S[++n] = total = s;
                else stuck = true;
            } else {
                full = s;
                take_out(sh, pending);
            }
            pending = -1;
        }
        for (; t < T && count < a.A; ++t) {
            if (sh.parent[t] != cur || sh.token[t] < 0) continue;
            const double q = sh.q[t];
            double left = sh.p[t];
            if (a.draft) {
                if (n > 0) left = (double)left_of(sh.p[t], sh.q[t], n, sh.S) / (double)total;
            } else if (have_row >= 0) {
                left = is_out(sh, sh.token[t]) ? 0.0 : left * (double)kOne / (double)total;
            }
            if ((double)sh.u[t] * q < left) {
                sh.path[count++] = t;
                enter(t);
                continue;
            }
            if (!a.draft && have_row >= 0) {
                take_out(sh, t);
            } else if (!stuck) {
                pending = t++;
                have_row = cur + a.context;
                have_n = a.draft ? n + 1 : 0;
                o.row = have_row;
                o.n = have_n;
                o.sum = total;
                o.sweep = 1;
                return;
            }
        }
        o.row = cur + a.context;
        o.n = n;
        o.sum = n > 0 ? sh.S[n - 1] : 0;
        o.sweep = have_row < 0 || have_n != n;
        o.last = 1;
        for (int w = 0; w < 4; ++w) o.gone[w] = gone[w];
    }
};

__global__ void __launch_bounds__(kVerifyThreads) verify_kernel(const __grid_constant__ VerifyParams a) {
    __shared__ Shared sh;
    const uint32_t rank = cluster_rank(), C = cluster_size();
    const int b = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int T = a.draft_lens ? min(max(__ldg(a.draft_lens + b), 0), a.T) : a.T;

    // The drafts, and u, p and q where they are compared.
    for (int t = tid; t < T; t += kVerifyThreads) {
        int par = __ldg(a.parents + b * a.parent_stride + t), tok = __ldg(a.tokens + b * a.token_stride + t);
        if (par < -1 || par >= t) {
            if (rank == 0) record_error(a.status, kErrInvalid);
            par = -1;
        }
        if (tok < 0 || tok >= a.V) {
            if (rank == 0) record_error(a.status, kErrInvalid);
            tok = -1;
        }
        const int row = par + a.context;                   // -1: without a context row nobody's child
        const bool tested = row >= 0 && tok >= 0;
        sh.token[t] = tok;
        sh.parent[t] = row < 0 ? -2 : par;
        sh.u[t] = __ldg(a.uniforms + b * a.uniform_stride + t);
        sh.p[t] = tested ? clamped(__ldg(a.target + b * a.target_stride[0] + row * a.target_stride[1] + tok)) : 0.f;
        sh.q[t] = !tested ? 0.f : !a.draft ? 1.f
                : clamped(__ldg(a.draft + b * a.draft_stride[0] + row * a.draft_stride[1] + tok));
    }
    if (tid == 0) {
        sh.u[kMaxDrafts] = __ldg(a.uniforms + b * a.uniform_stride + a.T);
        sh.S[0] = kOne;
    }
    cluster_sync();                                        // also: every CTA of the cluster is there

    Walk walk;
    walk.enter(-1);
    walk.t = walk.count = 0;
    walk.pending = -1;
    walk.full = 0;
    if (!a.context && T > 0) {                             // draft 0 is the token that the last step drew
        if (rank == 0 && tid == 0) sh.path[0] = 0;
        walk.enter(0);
        walk.count = walk.t = 1;
    }
    int sweeps = 0;
    Order o;
    for (;;) {
        if (rank == 0) {
            if (tid == 0) {
                walk.run(a, sh, T, sh.sums[(sweeps - 1) & 1], (int)C, o);
                if (!a.context && T == 0) o = Order{0, 0, 0, 0, 2, {0, 0, 0, 0}};
                sh.order = o;
                if (o.last) {
                    sh.count = walk.count;
                    a.next_tokens[b] = -1;                 // the drawing CTA writes it after the barrier
                    if (o.last == 2) record_error(a.status, kErrInvalid);
                }
            }
            __syncthreads();
            for (int i = tid; i < (int)(C - 1) * kOrderWords; i += kVerifyThreads) {
                const int w = i % kOrderWords;
                store_remote(reinterpret_cast<u64 *>(&sh.order) + w, i / kOrderWords + 1,
                             reinterpret_cast<const u64 *>(&sh.order)[w]);
            }
        }
        cluster_sync();
        o = sh.order;
        if (o.last == 2) break;
        const Rows rows(a, b, (int)o.row);
        const int n = (int)o.n;
        const int per = (rows.groups + (int)C - 1) / (int)C, seg = (per + kVerifyWarps - 1) / kVerifyWarps;
        const int first = (int)rank * per, end = min(rows.groups, first + per);
        if (o.sweep) {
            if (n > 0 && tid == 0) sh.S[n - 1] = o.sum;
            __syncthreads();
            const int g1 = min(end, first + (warp + 1) * seg);
            u64 s = 0;
            for (int g0 = first + warp * seg; g0 < g1; g0 += 128) {
                float4 p[4], q[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int g = g0 + 32 * i + lane;
                    p[i] = q[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (g >= g1) continue;
                    p[i] = rows.load(rows.p, true, g);
                    if (n > 0) q[i] = rows.load(rows.q, rows.q_wide, g);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s = min(s + (left_of(p[i].x, q[i].x, n, sh.S) + left_of(p[i].y, q[i].y, n, sh.S) +
                                 left_of(p[i].z, q[i].z, n, sh.S) + left_of(p[i].w, q[i].w, n, sh.S)), kMost);
            }
            s = warp_sum(s);
            if (lane == 0) sh.seg[warp] = s;
            __syncthreads();
            if (warp == 0) {
                s = warp_sum(lane < kVerifyWarps ? sh.seg[lane] : 0);
                if (lane < (int)C) store_remote(&sh.sums[sweeps & 1][rank], lane, s);
            }
            cluster_sync();
            ++sweeps;
        }
        if (o.last) break;
    }

    if (o.last == 1) {
        // The draw.  Tokens that went out leave the sums first.
        const Rows rows(a, b, (int)o.row);
        const int n = (int)o.n;
        const int per = (rows.groups + (int)C - 1) / (int)C, seg = (per + kVerifyWarps - 1) / kVerifyWarps;
        const int first = (int)rank * per, end = min(rows.groups, first + per);
        u64 *sums = sh.sums[(sweeps - 1) & 1];
        const bool some_out = (o.gone[0] | o.gone[1] | o.gone[2] | o.gone[3]) != 0;
        if (some_out && tid == 0) {
            for (int w = 0; w < 4; ++w)
                for (u64 m = o.gone[w]; m; m &= m - 1) {
                    const int c = 64 * w + __ffsll((long long)m) - 1;
                    const int g = (sh.token[c] + rows.shift) >> 2;
                    const u64 x = fixed(sh.p[c]);
                    sums[g / per] -= min(x, sums[g / per]);
                    if (g >= first && g < end) {
                        u64 &z = sh.seg[(g - first) / seg];
                        z -= min(x, z);
                    }
                }
        }
        __syncthreads();
        u64 S = 0, before = 0;
        for (uint32_t r = 0; r < C; ++r) {
            if (r < rank) before += sums[r];
            S += sums[r];
        }
        if (rank == 0 && tid == 0 && (S == 0 || S >= kMost)) record_error(a.status, kErrInvalid);
        const u64 want = __umul64hi(fraction(sh.u[kMaxDrafts]), S);
        if (S > 0 && want >= before && want - before < sums[rank]) {
            u64 rest = want - before;                      // the first x whose running sum passes it
            int w = 0;
            while (w < kVerifyWarps - 1 && rest >= sh.seg[w]) rest -= sh.seg[w++];
            const int g1 = min(end, first + (w + 1) * seg);
            for (int g0 = first + w * seg; g0 < g1; g0 += kVerifyThreads) {
                const int g = g0 + tid;
                u64 v[4] = {0, 0, 0, 0};
                if (g < g1) {
                    const float4 p = rows.load(rows.p, true, g);
                    const float4 q = n > 0 ? rows.load(rows.q, rows.q_wide, g) : p;
                    v[0] = left_of(p.x, q.x, n, sh.S);
                    v[1] = left_of(p.y, q.y, n, sh.S);
                    v[2] = left_of(p.z, q.z, n, sh.S);
                    v[3] = left_of(p.w, q.w, n, sh.S);
                    if (some_out) {
                        for (int k = 0; k < 4; ++k)
                            for (u64 m = o.gone[k]; m; m &= m - 1) {
                                const int x = sh.token[64 * k + __ffsll((long long)m) - 1] + rows.shift - 4 * g;
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    if (x == i) v[i] = 0;
                            }
                    }
                }
                const u64 own = v[0] + v[1] + v[2] + v[3];
                u64 incl = own;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const u64 y = __shfl_up_sync(0xffffffffu, incl, d);
                    if (lane >= d) incl = min(incl + y, kMost);
                }
                if (lane == 31) sh.scan[warp] = incl;
                __syncthreads();
                u64 lead = 0, all = 0;
                for (int i = 0; i < kVerifyWarps; ++i) {
                    if (i < warp) lead += sh.scan[i];
                    all += sh.scan[i];
                }
                lead += incl - own;
                if (rest >= lead && rest - lead < own) {
                    u64 r = rest - lead;
                    int i = 0;
                    while (i < 3 && r >= v[i]) r -= v[i++];
                    a.next_tokens[b] = 4 * g - rows.shift + i;
                }
                if (rest < all) break;
                rest -= all;
                __syncthreads();
            }
        }
    }
    if (rank == 0) {
        const int count = sh.count;
        for (int i = tid; i < a.A; i += kVerifyThreads)
            a.path[b * a.path_stride + i] = i < count ? sh.path[i] : -1;
        if (tid == 0) a.path_lens[b] = count;
    }
}

}  // namespace

cudaError_t launch_verify(const VerifyParams &p, cudaStream_t stream) {
    // As many CTAs to a request as leave all requests on the GPU at once (each SM takes
    // four of these blocks), eight at most.
    int C = kMaxCluster;
    while (C > 1 && (int64_t)p.B * C > 4ll * p.num_sms) C /= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)p.B * C));
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, verify_kernel, p);
}

}  // namespace fw
