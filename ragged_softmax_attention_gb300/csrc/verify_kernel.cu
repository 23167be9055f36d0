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
//
// Measured (GB300): 64 trees of 24 drafts over 152,000 tokens, one to six sweeps each, 71 us;
// a sweep takes a CTA of eight 6.3 us, bound by its instructions (some 40 an element where
// a product is subtracted), and the request with the most sweeps 54 us.  With every
// rejection gone through for each element 137 us.  A chain of 6 over 32,000 tokens: 9.8 us,
// launch, two rounds of loads, three meetings of the cluster.
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
// The 24-bit significand stands above the place of 1 and moves down by the exponent (a
// shift past 63 gives 0: zeros, subnormals and what is below 2^-61).
__device__ __forceinline__ u64 fixed(float v) {
    const uint32_t b = __float_as_uint(__saturatef(v));
    const u64 m = (u64)((b & 0x7fffffu) | 0x800000u) << 37;
    u64 r;
    asm("shr.u64 %0, %1, %2;" : "=l"(r) : "l"(m), "r"(127u - (b >> 23)));
    return r;
}
__device__ __forceinline__ float clamped(float v) { return v > 0.f ? fminf(v, 1.f) : 0.f; }
// A uniform number in units of 2^-64.
__device__ __forceinline__ u64 fraction(float u) {
    if (!(u > 0.f)) return 0;
    return u >= 1.f ? ~0ull : __double2ull_rz((double)u * 18446744073709551616.0);
}
// What is left of p after n rejections: R_n = max(p - c_n q, 0) with c_1 = 1, c_{n+1} = c_n +
// S_n (an element that a rejection took to 0 stays there), so no element needs to go
// through the earlier ones.  c comes in units of 2^-52; its product with q's 24-bit
// significand keeps 43 bits or more.
__device__ __forceinline__ u64 times(float q, u64 c) {
    const uint32_t b = __float_as_uint(__saturatef(q)), e = b >> 23;
    const uint32_t m = (b & 0x7fffffu) | 0x800000u;
    const u64 h = (u64)m * (uint32_t)(c >> 32) + ((u64)m * (uint32_t)c >> 32);      // c q 2^(170 - e)
    u64 up, down;                                         // (a negative shift is a large one, and gives 0)
    asm("shl.b64 %0, %1, %2;" : "=l"(up) : "l"(h), "r"(e - 110u));
    asm("shr.u64 %0, %1, %2;" : "=l"(down) : "l"(h), "r"(110u - e));
    return up | down;
}
template <int N>                                          // 0, 1, 2: that many or more
__device__ __forceinline__ u64 left_of(float p, float q, u64 c, float rough) {
    const u64 r = fixed(p);
    if (N == 0) return r;
    const u64 t = N == 1 ? fixed(q) : times(q, c);
    // (With c q far above p the product may not fit: nothing is left then.)
    return r > t && (N == 1 || rough * __saturatef(q) < 1.001f * p) ? r - t : 0;
}
__device__ __forceinline__ float rough_of(u64 c) { return (float)c * 2.220446e-16f; }      // 2^-52

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = min(v + __shfl_xor_sync(0xffffffffu, v, o), kMost);
    return v;
}

// What the walking thread asks of the cluster.
struct Order {
    u64 row;               // row of the probabilities
    u64 n;                 // rejections there (with a draft model's rows)
    u64 c;                 // c_n in units of 2^-52
    u64 sweep;             // 1: the row's sums are wanted
    u64 last;              // 1: the path ends here, draw; 2: no row to draw from
    u64 gone[4];           // without a draft model's rows: drafts whose tokens are out, a bit each
};
constexpr int kOrderWords = sizeof(Order) / 8;

struct Shared {
    Order order;
    u64 sums[2][kMaxCluster];          // per CTA, of the last two sweeps
    u64 seg[kVerifyWarps];             // per warp, of the last sweep
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

// Sum of what is left in the groups g0 .. g1 - 1 of a row, a lane's share.
template <int N>
__device__ __forceinline__ u64 sweep(const Rows &rows, int g0, int g1, u64 c) {
    const int lane = threadIdx.x & 31;
    const float rough = rough_of(c);
    u64 s = 0;
    auto add = [&](const float4 &p, const float4 &q) {
        s = min(s + (left_of<N>(p.x, q.x, c, rough) + left_of<N>(p.y, q.y, c, rough) + left_of<N>(p.z, q.z, c, rough) +
                     left_of<N>(p.w, q.w, c, rough)), kMost);
    };
    const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
    for (; g0 < g1; g0 += 128) {
        float4 p[4], q[4];
        if (g0 > 0 && g0 + 128 <= min(g1, rows.groups - 1) && (N == 0 || rows.q_wide)) {      // whole groups all
            const float4 *pp = reinterpret_cast<const float4 *>(rows.p + 4 * g0 - rows.shift) + lane;
            const float4 *qq = reinterpret_cast<const float4 *>(rows.q + 4 * g0 - rows.shift) + lane;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[i] = __ldg(pp + 32 * i);
                if (N > 0) q[i] = __ldg(qq + 32 * i);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) add(p[i], N > 0 ? q[i] : none);
        } else {
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
                const int g = g0 + 32 * i + lane;
                if (g >= g1) continue;
                add(rows.load(rows.p, true, g), N > 0 ? rows.load(rows.q, rows.q_wide, g) : none);
            }
        }
    }
    return s;
}

// The walk, by one thread: runs until it needs a row's sums or has reached its end.
struct Walk {
    int t, cur, count, n;                  // next draft, node, accepted drafts, rejections at the node
    bool stuck;                            // nothing would be left: rejections change nothing more
    int pending;                           // the rejected child whose sums are under way, -1: none
    u64 total, full;                       // S; without a draft model's rows the row's sum
    u64 c;                                 // c_n in units of 2^-52
    int have_row, have_n;                  // what the segments' sums are of

    __device__ void enter(int node) {
        cur = node;
        n = 0;
        stuck = false;
        total = kOne;
        c = 0;
        have_row = have_n = -1;
    }
    // Without a draft model's rows: whether a token is out, and child `d`'s going out.
    __device__ static bool is_out(const Shared &sh, int tok) {
        for (int w = 0; w < 4; ++w)
            for (u64 m = sh.order.gone[w]; m; m &= m - 1)
                if (sh.token[64 * w + __ffsll((long long)m) - 1] == tok) return true;
        return false;
    }
    __device__ void take_out(Shared &sh, int d) {
        const u64 x = is_out(sh, sh.token[d]) ? 0 : fixed(sh.p[d]);
        if (full <= x) return;
        full -= x;
        total = full;
        if (x > 0) sh.order.gone[d >> 6] |= 1ull << (d & 63);
    }
    __device__ void run(const VerifyParams &a, Shared &sh, int T, const u64 *sums, int C) {
        Order &o = sh.order;
        if (pending >= 0) {
            u64 s = 0;
            for (int r = 0; r < C; ++r) s = min(s + sums[r], kMost);
            if (a.draft) {
                if (s > 0) {
                    c += total >> 8;                       // 2^-60 to 2^-52
                    ++n;
                    total = s;
                } else {
                    stuck = true;
                }
            } else {
                full = s;
                take_out(sh, pending);
            }
            pending = -1;
        }
        for (; t < T && count < a.A; ++t) {
            if (sh.parent[t] != cur || sh.token[t] < 0) continue;
            // u q < R / S
            bool yes;
            if (total == kOne && n == 0 && have_row < 0) {
                yes = (double)sh.u[t] * (double)sh.q[t] < (double)sh.p[t];
            } else {
                const u64 left = a.draft ? left_of<2>(sh.p[t], sh.q[t], c, rough_of(c)) : is_out(sh, sh.token[t]) ? 0 : fixed(sh.p[t]);
                yes = (double)sh.u[t] * (double)sh.q[t] * (double)total < (double)left;
            }
            if (yes) {
                sh.path[count++] = t;
                enter(t);
                if (!a.draft) o.gone[0] = o.gone[1] = o.gone[2] = o.gone[3] = 0;
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
                o.c = c + (total >> 8);
                o.sweep = 1;
                o.last = 0;
                return;
            }
        }
        o.row = cur + a.context;
        o.n = n;
        o.c = c;
        o.sweep = have_row < 0 || have_n != n;
        o.last = 1;
    }
};

__global__ void __launch_bounds__(kVerifyThreads, 2) verify_kernel(const __grid_constant__ VerifyParams a) {
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
        sh.order = Order{};
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
                walk.run(a, sh, T, sh.sums[(sweeps - 1) & 1], (int)C);
                if (!a.context && T == 0) sh.order.last = 2;
                if (sh.order.last) {
                    sh.count = walk.count;
                    a.next_tokens[b] = -1;                 // the drawing CTA writes it after the barrier
                    if (sh.order.last == 2) record_error(a.status, kErrInvalid);
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
            const int g0 = first + warp * seg, g1 = min(end, g0 + seg);
            u64 s = n == 0 ? sweep<0>(rows, g0, g1, 0) : n == 1 ? sweep<1>(rows, g0, g1, o.c) : sweep<2>(rows, g0, g1, o.c);
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
                    const float4 q = n > 0 ? rows.load(rows.q, rows.q_wide, g) : make_float4(0.f, 0.f, 0.f, 0.f);
                    const float rough = rough_of(o.c);
                    v[0] = n > 1 ? left_of<2>(p.x, q.x, o.c, rough) : left_of<1>(p.x, q.x, o.c, rough);
                    v[1] = n > 1 ? left_of<2>(p.y, q.y, o.c, rough) : left_of<1>(p.y, q.y, o.c, rough);
                    v[2] = n > 1 ? left_of<2>(p.z, q.z, o.c, rough) : left_of<1>(p.z, q.z, o.c, rough);
                    v[3] = n > 1 ? left_of<2>(p.w, q.w, o.c, rough) : left_of<1>(p.w, q.w, o.c, rough);
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
    // Eight CTAs to a request (what a portable cluster holds) while that is no more than
    // twice what the GPU takes at once: requests differ in what they reject, and short ones
    // make room (64 trees of 24 drafts: 71 us at eight, 82 at four).
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
