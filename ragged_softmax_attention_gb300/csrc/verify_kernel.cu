// Verification of drafted trees against the target's probabilities, sm_103a.
//
// At a node with the target's row p and the draft model's row q, its children are
// tried in order: child c is accepted with probability min(1, R(c) / (S q(c))),
// where R is what is left of p and S its sum; after a rejection
//   R <- max(R - S q, 0),  S <- sum R        (at first R = p, S = 1),
// and the walk goes on from the accepted child.  Where no child is accepted the next
// token is drawn from R: the first x with R(0) + .. + R(x) > u sum R.  Drafts so
// verified are distributed as the target's own samples (rejection sampling, one
// draft after another; a node's children are independent draws).  Without a draft model's
// rows a draft is taken as proposed with certainty, and R loses the token.
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
// Measured (GB300): 64 trees of 24 drafts over 152,000 tokens, one to six sweeps each, 54 us;
// a sweep takes 3 to 8 us of it, by how many long requests share an SM, each meeting of the
// cluster with its walk 1.5, and the request with the most sweeps 52.  The longest requests
// bound it: the SMs issue in 36 % of their cycles.  (Sums of 64-bit integers, loads straight
// into registers and CTAs of 512 threads: 71; every rejection gone through for each element:
// 137.)  A chain of 6 over 32,000 tokens: 8.6 us, launch, two rounds of loads, three meetings.
// A warp that walks as one, by ballots, is no faster than one thread (59 and 9.9 us).
#include "fw_internal.h"
#include "fw_ptx.cuh"

namespace fw {
namespace {

constexpr int kErrInvalid = 1;     // FW_ERR_INVALID_ARG
// Three CTAs of 256 threads an SM: two of 512 meet more slowly (64 trees: 64 us for 54).
constexpr int kVerifyThreads = 256, kVerifyWarps = kVerifyThreads / 32;
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
// Threads that wrote nothing for the others since they last met the threads of their CTA
// arrive without a release (the writers' release covers what came before that meeting).
__device__ __forceinline__ void cluster_sync(bool wrote) {
    __syncwarp();
    if (wrote) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    else asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
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

typedef uint64_t f32x2;
__device__ __forceinline__ f32x2 two(float lo, float hi) {
    f32x2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ float2 both(f32x2 v) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ f32x2 minus(f32x2 a, f32x2 b) { return fma2(b, two(-1.f, -1.f), a); }
__device__ __forceinline__ float clamped(float v) { return v > 0.f ? fminf(v, 1.f) : 0.f; }
// A uniform number in units of 2^-64.
__device__ __forceinline__ u64 fraction(float u) {
    if (!(u > 0.f)) return 0;
    return u >= 1.f ? ~0ull : __double2ull_rz((double)u * 18446744073709551616.0);
}
// What is left of p after n rejections: R_n = max(p - c_n q, 0) with c_1 = 1, c_{n+1} = c_n +
// S_n (an element that a rejection took to 0 stays there), so no element needs to go
// through the earlier ones.  c comes in units of 2^-52 and is taken as two floats, 48 bits.
//
// The difference is held as a float and the float that it lacks (what one step rounds away
// is a float itself), and leaves as integers of 2^-20, 2^-40 and 2^-60: adding 3 2^(22 - k)
// to a small float rounds it to a multiple of 2^-k that stands in the sum's low bits, and
// these are added as they are.  Two elements go through one instruction.  NaN and what is
// negative count as 0, more than 1 as 1.  In 64-bit integers an element takes twice the
// instructions (the trees above: 64 us against 54).
struct Scale {
    f32x2 c, neg, neg_low;                                // c's leading 24 bits, minus them, minus the rest
    __device__ __forceinline__ explicit Scale(u64 n) {
        const float h = __ull2float_rn(n), l = __ll2float_rn((long long)(n - __float2ull_rn(h)));
        const float unit = 2.220446049250313e-16f;        // 2^-52
        c = two(h * unit, h * unit);
        neg = two(-h * unit, -h * unit);
        neg_low = two(-l * unit, -l * unit);
    }
};
constexpr uint32_t kRound0 = 0x41400000u, kRound1 = 0x37400000u, kRound2 = 0x2d400000u;      // 3 2^2, 3 2^-18, 3 2^-38
struct Parts {
    f32x2 v[4];            // of 2^-20, 2^-40, 2^-40 (0 where N = 0), 2^-60
};
__device__ __forceinline__ f32x2 round_to(f32x2 &x, uint32_t by) {      // the multiple; x keeps the rest
    const float m = __uint_as_float(by);
    const f32x2 t = add2(x, two(m, m));
    x = minus(x, add2(t, two(-m, -m)));
    return t;
}
template <int N>                                          // 0, 1, 2: that many or more
__device__ __forceinline__ Parts left_of(float p0, float p1, float q0, float q1, const Scale &s) {
    p0 = __saturatef(p0);
    p1 = __saturatef(p1);
    const f32x2 p = two(p0, p1);
    f32x2 hi = p, lo = 0;
    if (N == 1) {
        const f32x2 q = two(fminf(__saturatef(q0), p0), fminf(__saturatef(q1), p1));
        hi = minus(p, q);
        lo = minus(minus(p, hi), q);
    }
    if (N == 2) {
        const f32x2 q = two(__saturatef(q0), __saturatef(q1));
        const f32x2 t = mul2(q, s.neg);                                // -c q and what it lacks
        const f32x2 low = fma2(q, s.neg_low, fma2(q, s.neg, mul2(q, s.c)));
        const f32x2 d = add2(p, t), rest = add2(add2(minus(p, d), t), low);
        hi = add2(d, rest);
        lo = minus(rest, minus(hi, d));
        const float2 h = both(hi), l = both(lo);
        hi = two(fmaxf(h.x, 0.f), fmaxf(h.y, 0.f));
        lo = two(h.x > 0.f ? l.x : 0.f, h.y > 0.f ? l.y : 0.f);
    }
    Parts r;
    r.v[0] = round_to(hi, kRound0);
    r.v[1] = round_to(hi, kRound1);
    r.v[2] = 0;
    if (N > 0) {
        r.v[2] = round_to(lo, kRound1);
        hi = add2(hi, lo);
    }
    const float m = __uint_as_float(kRound2);
    r.v[3] = add2(hi, two(m, m));
    return r;
}
__device__ __forceinline__ u64 join(uint32_t a, uint32_t b, uint32_t c) {
    return ((long long)(int)a << 40) + ((long long)(int)b << 20) + (int)c;
}
// Two elements in units of 2^-60, where few are asked for.  (c = 0 takes nothing out and
// c = 1 what one rejection does, to the last bit, so one form does for all n.)
__device__ __forceinline__ ulonglong2 left_units(float p0, float p1, float q0, float q1, u64 c) {
    const Parts r = left_of<2>(p0, p1, q0, q1, Scale(c));
    return make_ulonglong2(
        join((uint32_t)r.v[0] - kRound0, (uint32_t)r.v[1] + (uint32_t)r.v[2] - 2 * kRound1, (uint32_t)r.v[3] - kRound2),
        join((uint32_t)(r.v[0] >> 32) - kRound0, (uint32_t)(r.v[1] >> 32) + (uint32_t)(r.v[2] >> 32) - 2 * kRound1,
             (uint32_t)(r.v[3] >> 32) - kRound2));
}
__device__ __forceinline__ u64 left_one(float p, float q, u64 c) { return left_units(p, 0.f, q, 0.f, c).x; }
// Sums of up to 2^10 elements.
template <int N>
struct Sum {
    uint32_t a = 0, b = 0, c = 0, pairs = 0;
    __device__ __forceinline__ void add(const Parts &r) {
        a += (uint32_t)r.v[0] + (uint32_t)(r.v[0] >> 32);
        b += (uint32_t)r.v[1] + (uint32_t)(r.v[1] >> 32);
        if (N > 0) b += (uint32_t)r.v[2] + (uint32_t)(r.v[2] >> 32);
        c += (uint32_t)r.v[3] + (uint32_t)(r.v[3] >> 32);
        ++pairs;
    }
    __device__ __forceinline__ void add(const float4 &p, const float4 &q, const Scale &s) {
        add(left_of<N>(p.x, p.y, q.x, q.y, s));
        add(left_of<N>(p.z, p.w, q.z, q.w, s));
    }
    __device__ __forceinline__ u64 value() const {
        const uint32_t most = 4u << 20, x = a - 2 * pairs * kRound0;
        return x > most ? kMost : min(join(x, b - (N > 0 ? 4 : 2) * pairs * kRound1, c - 2 * pairs * kRound2), kMost);
    }
};

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
static_assert((kMaxCluster - 1) * kOrderWords <= 64, "two warps tell the others");

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

// Groups on their way to shared memory: each lane copies, awaits and reads its own, so
// that no thread waits for another, and kStages - 1 of its loads are under way.
constexpr int kStages = 4, kGroups = 2;                   // groups a stage (8 of 1: 55 us for 54)
constexpr int kStageBytes = kGroups * 2 * 16 * kVerifyThreads, kCopyBytes = kStages * kStageBytes;
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t to, const void *from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(BYTES) : "memory");
}
__device__ __forceinline__ float4 load_shared(uint32_t at) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
    return v;
}

// Sum of what is left in the groups g0 .. g1 - 1 of a row, a lane's share.
template <int N>
__device__ __forceinline__ u64 sweep(const Rows &rows, int g0, int g1, u64 c, uint32_t copies) {
    const int lane = threadIdx.x & 31;
    const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
    if (g0 >= g1) return 0;
    const int e0 = g0 == 0 && rows.shift != 0 ? g0++ : -1;                       // groups that are not whole
    const int e1 = g1 == rows.groups && g0 < g1 && ((rows.V + rows.shift) & 3) != 0 ? --g1 : -1;
    const float4 *pp = reinterpret_cast<const float4 *>(rows.p - rows.shift);
    const float *qq = rows.q - rows.shift;
    copies += threadIdx.x * 16;
    auto start = [&](int g, int stage) {
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int x = g + 32 * i;
            const uint32_t to = copies + stage * kStageBytes + i * 32 * kVerifyThreads;
            if (x < g1) {
                copy_async<16>(to, pp + x);
                if (N > 0 && rows.q_wide) copy_async<16>(to + 16 * kVerifyThreads, qq + 4 * x);
                if (N > 0 && !rows.q_wide) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) copy_async<4>(to + 16 * kVerifyThreads + 4 * j, qq + 4 * x + j);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int i = 0; i < kStages - 1; ++i) start(g0 + lane + 32 * kGroups * i, i);
    const Scale scale(c);
    u64 s = 0;
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
        const int e = i ? e1 : e0;
        if (e < 0 || lane != 0) continue;
        Sum<N> sum;
        sum.add(rows.load(rows.p, true, e), N > 0 ? rows.load(rows.q, rows.q_wide, e) : none, scale);
        s += sum.value();
    }
    int stage = 0;
    while (g0 < g1) {
        Sum<N> sum;
#pragma unroll 1
        for (int k = 0; k < 256 / kGroups && g0 < g1; ++k, g0 += 32 * kGroups) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
            float4 p[kGroups], q[kGroups];
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                const uint32_t from = copies + stage * kStageBytes + i * 32 * kVerifyThreads;
                p[i] = q[i] = none;
                if (g0 + lane + 32 * i >= g1) continue;
                p[i] = load_shared(from);
                if (N > 0) q[i] = load_shared(from + 16 * kVerifyThreads);
            }
            // The stage read a step ago is free.
            start(g0 + lane + 32 * kGroups * (kStages - 1), (stage + kStages - 1) % kStages);
            stage = (stage + 1) % kStages;
#pragma unroll
            for (int i = 0; i < kGroups; ++i) sum.add(p[i], q[i], scale);
        }
        s = min(s + sum.value(), kMost);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
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
        const u64 x = is_out(sh, sh.token[d]) ? 0 : left_one(sh.p[d], 0.f, 0);
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
            if (s >= kMost) record_error(a.status, kErrInvalid);
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
                const u64 left = a.draft ? left_one(sh.p[t], sh.q[t], c)
                                         : is_out(sh, sh.token[t]) ? 0 : left_one(sh.p[t], 0.f, 0);
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

__global__ void __launch_bounds__(kVerifyThreads, 3) verify_kernel(const __grid_constant__ VerifyParams a) {
    __shared__ Shared sh;
    extern __shared__ __align__(16) uint8_t copied[];
    const uint32_t copies = smem_u32(copied);
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
    __syncthreads();
    cluster_sync(warp == 0);                               // every CTA of the cluster is there

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
        cluster_sync(warp < 2);
        o = sh.order;
        if (o.last == 2) break;
        const Rows rows(a, b, (int)o.row);
        const int n = (int)o.n;
        const int per = (rows.groups + (int)C - 1) / (int)C, seg = (per + kVerifyWarps - 1) / kVerifyWarps;
        const int first = (int)rank * per, end = min(rows.groups, first + per);
        if (o.sweep) {
            const int g0 = first + warp * seg, g1 = min(end, g0 + seg);
            u64 s = n == 0 ? sweep<0>(rows, g0, g1, 0, copies) : n == 1 ? sweep<1>(rows, g0, g1, 0, copies)
                  : sweep<2>(rows, g0, g1, o.c, copies);
            s = warp_sum(s);
            if (lane == 0) sh.seg[warp] = s;
            __syncthreads();
            if (warp == 0) {
                s = warp_sum(lane < kVerifyWarps ? sh.seg[lane] : 0);
                if (lane < (int)C) store_remote(&sh.sums[sweeps & 1][rank], lane, s);
            }
            cluster_sync(warp == 0);
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
                    const u64 x = left_one(sh.p[c], 0.f, 0);
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
            if (r < rank) before = min(before + sums[r], kMost);
            S = min(S + sums[r], kMost);
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
                    const ulonglong2 x = left_units(p.x, p.y, q.x, q.y, o.c), y = left_units(p.z, p.w, q.z, q.w, o.c);
                    v[0] = x.x, v[1] = x.y, v[2] = y.x, v[3] = y.y;
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
                    if (i < warp) lead = min(lead + sh.scan[i], kMost);
                    all = min(all + sh.scan[i], kMost);
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
    // Eight CTAs to a request (what a portable cluster holds) while a launch has no more than
    // four an SM: requests differ in what they reject, and short ones make room for others (24
    // drafts over 152,000 tokens, 64 trees: 54 us at eight, 64 at four; over 50,000 tokens,
    // 200 trees: 56 us at two, 81 at eight).
    int C = kMaxCluster;
    while (C > 1 && (int64_t)p.B * C > 4ll * p.num_sms) C /= 2;
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!configured[dev & 63]) {
        e = cudaFuncSetAttribute(verify_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kCopyBytes);
        if (e != cudaSuccess) return e;
        configured[dev & 63] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)p.B * C));
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.dynamicSmemBytes = kCopyBytes;
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
