// Norms of queries and keys for each head with the position rotation in the
// same pass, sm_103a; keys (and values) optionally go straight to their cache
// slots:
//   y = x * rsqrt(mean(x^2) + eps) * w
//   (y_i, y_i') -> (y_i cos a - y_i' sin a, y_i' cos a + y_i sin a),  a = pos * inv_freq_i
// with i' = i + rot / 2 (halves) or the odd neighbour (interleaved).
//
// Every element is read and written once: DRAM bounds it from a few thousand
// tokens on, latencies below.  A head takes D / 16 lanes, and a lane's sixteen
// elements are eight whole pairs, so the rotation needs no exchange and the sum of
// squares log2(D / 16) shuffles (eight elements a lane cost a third more instructions;
// kept for rotations of an odd number of eights).  A warp has a token, or a share of one's
// heads, to itself: it works out the cosines and sines once, a lane's share of them times
// the weights stays in registers over all heads, and copies run ahead through a ring of
// shared memory, past the end of the token, in which a lane reads what it copied itself,
// so that nothing waits for another warp.
//
// Measured (GB300): 8,191 tokens of 40/8 heads into an FP8 cache, 218 MB in 36 us, 0.90 of
// copy; 5,000 of 32/8 heads with three axes, 102 MB in 19.7, 0.76; 48 tokens 3.9, all of it
// round trips.  On the way, first case: every warp that shares a token working out its
// angles, loads by round 85 us; a block's tokens together 64; copies ahead 57; a warp to a
// token 47; the head groups of all tokens in equal runs, codes without division 36.
//
// An angle is needed modulo one turn, and pos * inv_freq in 32 bits loses it (1e5
// radians are good to 0.008).  inv_freq / 2 pi is kept as a 64-bit fraction of a
// turn; the integer product with the position drops whole turns by itself, exactly, for
// either sign.  The fraction is worked out once a block, in integers, since a position of
// 2^31 multiplies what it lacks (a double leaves 2^-25 of a turn for a frequency of 1, 2^-19
// for 40; two doubles do, and take 0.3 us more of the 48 tokens above).  The product's leading
// 32 bits would not fit a float either; less the nearest quarter turn they do to 2^-28 of
// a turn (keys of the first case above that come out as another E4M3 code than in 64 bits: 11
// of 8.4 million; 22 with the angle rounded as it was).
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "fw_internal.h"
#include "fw_ptx.cuh"

namespace fw {
namespace {

constexpr int kErrInvalid = 1;     // FW_ERR_INVALID_ARG
constexpr int kRopeWarps = 8;
constexpr int kRopeThreads = kRopeWarps * 32;
constexpr int kRopeBlocks = 2;     // resident blocks an SM
constexpr int kStages = 6;         // head groups of a warp on their way or in hand
typedef uint64_t f32x2;
__device__ __forceinline__ f32x2 two(float lo, float hi) {
    f32x2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ float2 both(f32x2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
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
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
}
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// E4M3 codes of v / scale, as the append divides.  With inv = 1 / scale rounded to nearest,
// q = v * inv is off by two roundings, and q + (v - q scale) inv, the remainder being
// exact, by less than 2^-46 before its own rounding (Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", section 8), as long as nothing over-
// or underflows: for scales of 2^-60 .. 2^60 and quotients below 2^10; those so small that
// the remainder is not exact have code 0, and their sign is put back.  Other scales (inv =
// 0), and lanes with a quotient that large or infinite, divide; a NaN stays one without.
// (Division alone: 115 us for 4,864 tokens of 128 key and value heads, 94 so.)
template <int N>
__device__ __forceinline__ void codes(const float *v, float scale, float inv, uint32_t *out) {
    float r[N], most = 0.f;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const f32x2 x = two(v[i], v[i + 1]), y = two(inv, inv), q = mul2(x, y);
        const float2 a = both(q), z = both(fma2(fma2(q, two(-scale, -scale), x), y, q));
        // (fmaxf drops a NaN; a sum would not, but inf - inf may come of one.)
        most = fmaxf(most, fmaxf(fabsf(a.x), fabsf(a.y)));
        r[i] = __uint_as_float(__float_as_uint(z.x) | (__float_as_uint(v[i]) & 0x80000000u));
        r[i + 1] = __uint_as_float(__float_as_uint(z.y) | (__float_as_uint(v[i + 1]) & 0x80000000u));
    }
    if (__builtin_expect(!(most < 1024.f) || inv == 0.f, 0)) {
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] = __fdiv_rn(v[i], scale);
    }
#pragma unroll
    for (int i = 0; i < N; i += 4)
        out[i / 4] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(r[i], r[i + 1]), __NV_SATFINITE, __NV_E4M3) |
                     (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(r[i + 2], r[i + 3]), __NV_SATFINITE, __NV_E4M3) << 16;
}

// A run of half a lane's elements, as it lies in memory: E / 2 BF16 values.
template <int E> struct Run;
template <> struct Run<8> { uint2 w; __device__ uint32_t at(int i) const { return i ? w.y : w.x; } };
template <> struct Run<16> {
    uint4 w;
    __device__ uint32_t at(int i) const { return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w; }
};

template <int E>
__device__ __forceinline__ void copy_run(Run<E> *to, const uint16_t *from) {
    if constexpr (E == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}

// A lane's E elements of a head: run 0 and run 1.  Pair i is element i of either run
// (halves), or neighbours (interleaved); a[] and b[] are the pairs' parts, two pairs each.
template <int E, bool kInter>
struct Pairs {
    static constexpr int P = E / 4;
    f32x2 a[P], b[P];
    __device__ __forceinline__ void unpack(const Run<E> &r0, const Run<E> &r1) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            if (kInter) {
                const Run<E> &r = i < P / 2 ? r0 : r1;
                const uint32_t w0 = r.at(2 * i % P), w1 = r.at(2 * i % P + 1);
                a[i] = two(low(w0), low(w1));
                b[i] = two(high(w0), high(w1));
            } else {
                a[i] = two(low(r0.at(i)), high(r0.at(i)));
                b[i] = two(low(r1.at(i)), high(r1.at(i)));
            }
        }
    }
    __device__ __forceinline__ void values(float (&v)[E]) const {             // run 0, then run 1
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float2 x = both(a[i]), y = both(b[i]);
            if (kInter) { v[4 * i] = x.x; v[4 * i + 1] = y.x; v[4 * i + 2] = x.y; v[4 * i + 3] = y.y; }
            else { v[2 * i] = x.x; v[2 * i + 1] = x.y; v[E / 2 + 2 * i] = y.x; v[E / 2 + 2 * i + 1] = y.y; }
        }
    }
    __device__ __forceinline__ float squares() const {
        f32x2 s = mul2(a[0], a[0]), t = mul2(b[0], b[0]);
#pragma unroll
        for (int i = 1; i < P; ++i) { s = fma2(a[i], a[i], s); t = fma2(b[i], b[i], t); }
        const float2 x = both(s), y = both(t);
        return (x.x + x.y) + (y.x + y.y);
    }
};
template <int E>
__device__ __forceinline__ void store_bf16(char *to, const float *v) {
    if constexpr (E == 16)
        *reinterpret_cast<uint4 *>(to) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                                    pack_bf16x2(v[6], v[7]));
    else
        *reinterpret_cast<uint2 *>(to) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}
template <int E>
__device__ __forceinline__ void store_codes(char *to0, char *to1, const float *v, float scale, float inv) {
    uint32_t w[E / 4];
    codes<E>(v, scale, inv, w);
    if constexpr (E == 16) {
        *reinterpret_cast<uint2 *>(to0) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2 *>(to1) = make_uint2(w[2], w[3]);
    } else {
        *reinterpret_cast<uint32_t *>(to0) = w[0];
        *reinterpret_cast<uint32_t *>(to1) = w[1];
    }
}

// f / 2 pi modulo 1 in units of 2^-64, rounded towards zero: f is m 2^e, and of 1 / 2 pi only
// the digits count that m 2^e takes to between 2^-1 and 2^-128; those before make whole turns
// (Payne and Hanek, "Radian reduction for trigonometric functions", 1983).  256 digits
// do for every float.
__device__ __forceinline__ uint64_t turn_of(float freq) {
    const uint32_t w = __float_as_uint(freq), exponent = w >> 23 & 255;
    const uint64_t m = exponent ? (w & 0x7fffffu) | 0x800000u : w & 0x7fffffu;
    const int at = (int)max(exponent, 1u) - 150 + 192, i = at >> 6, r = at & 63;       // e + 192 >= 43
    auto digits = [](int k) -> uint64_t {                                 // 64 of them, after 192 zeros
        return k == 3 ? 0x28be60db9391054aull : k == 4 ? 0x7f09d5f47d4d3770ull : k == 5 ? 0x36d8a5664f10e410ull
             : k == 6 ? 0x7f9458eaf7aef158ull : 0;
    };
    const uint64_t a = digits(i), b = digits(i + 1), c = digits(i + 2);
    const uint64_t t = m * (a << r | b >> 1 >> (63 - r)) + __umul64hi(m, b << r | c >> 1 >> (63 - r));
    return w >> 31 ? 0 - t : t;
}

template <int D, int E, bool kInter, bool kPartial>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
    constexpr int L = D / E, H = E / 2, P = E / 4;   // lanes of a head; elements and f32x2s of a run
    constexpr int HPW = 32 / L;                      // heads of a warp, a group
    constexpr int kAngles = D / 64;                  // of a lane
    __shared__ uint64_t turn[D / 2];                 // inv_freq / 2 pi in 2^-64 turns
    __shared__ int axis[D / 2];
    __shared__ __align__(16) float weight[2][D];     // the first parts of the pairs in order, then the second
    __shared__ __align__(16) float cosine[kRopeWarps][D / 2], sine[kRopeWarps][D / 2];
    extern __shared__ __align__(16) uint8_t ring_bytes[];
    Run<E> (*ring)[2][kRopeThreads] = reinterpret_cast<Run<E> (*)[2][kRopeThreads]>(ring_bytes);      // [kStages]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, half = p.rot / 2;
    // This lane's elements of a head: two runs, o0 and o1 on; its pairs' numbers begin at
    // H j (elements that do not turn make pairs of their own).
    const int j = lane % L, sub = lane / L;
    const bool rotates = !kPartial || E * j < p.rot;
    const int o0 = kInter || !rotates ? E * j : H * j;
    const int o1 = kInter || !rotates ? E * j + H : half + H * j;

    // A token's head groups are queries, keys, values in that order; those of all tokens,
    // end to end, go to the warps in equal runs.
    const int nq = (p.Hq + HPW - 1) / HPW, nk = (p.Hkv + HPW - 1) / HPW;
    const int groups = nq + nk + (p.v ? nk : 0);
    const int64_t total = p.N * groups, warps = (int64_t)gridDim.x * kRopeWarps;
    const int64_t me = (int64_t)blockIdx.x * kRopeWarps + warp;
    const int64_t from = total / warps * me + min(me, total % warps);     // the first total % warps take one more
    const int64_t count = total / warps + (me < total % warps);
    const int64_t n_first = from / groups;
    const int g_first = (int)(from - n_first * groups);

    // The copies, kStages - 1 groups ahead.
    int64_t f_n = n_first, f_rest = count, f_step = 0;
    int f_kind = 0, f_left = 0, f_heads = 0, f_stage = 0, f_g = g_first;
    const uint16_t *f_src = nullptr;
    auto fetch = [&]() {
        if (f_left == 0 && f_rest > 0) {                  // the next kind of heads, the next token
            if (f_g == groups) { f_g = 0; ++f_n; }
            f_kind = f_g < nq ? 0 : f_g < nq + nk ? 1 : 2;
            const int begin = f_kind == 0 ? 0 : f_kind == 1 ? nq : nq + nk, end = f_kind == 0 ? nq : f_kind == 1 ? nq + nk : groups;
            f_left = (int)min((int64_t)(end - f_g), f_rest);
            const int h = (f_g - begin) * HPW + sub;
            f_g += f_left;
            f_rest -= f_left;
            const int64_t step = f_kind == 0 ? p.q_stride[1] : f_kind == 1 ? p.k_stride[1] : p.v_stride[1];
            f_src = (f_kind == 0 ? p.q + f_n * p.q_stride[0] : f_kind == 1 ? p.k + f_n * p.k_stride[0] : p.v + f_n * p.v_stride[0]) +
                    h * step + (f_kind == 2 ? E * j : o0);
            f_step = step * HPW;
            f_heads = (f_kind == 0 ? p.Hq : p.Hkv) - h;
        }
        if (f_left > 0) {
            if (f_heads > 0) {
                copy_run(&ring[f_stage][0][tid], f_src);
                copy_run(&ring[f_stage][1][tid], f_src + (f_kind == 2 ? H : o1 - o0));
            }
            --f_left;
            f_heads -= HPW;
            f_src += f_step;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        f_stage = f_stage + 1 == kStages ? 0 : f_stage + 1;
    };
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) fetch();

    // What the next token's angles and place need, on its way while this one goes through.
    int32_t pos[kAngles], slot = -1;
    auto look = [&](int64_t n) {
        if (n >= p.N) return;
#pragma unroll
        for (int k = 0; k < kAngles; ++k) {
            const int f = lane + 32 * k;
            pos[k] = f < half ? __ldg(p.positions + (p.axes > 1 ? axis[f] * p.pos_stride : 0) + n) : 0;
        }
        slot = p.slots ? __ldg(p.slots + n) : -1;
    };
    // The block's tables, their loads (and the first token's) all on their way before the
    // first is used: with few tokens these round trips are most of the time.
    static_assert(D <= kRopeThreads, "a thread to a table entry");
    const float freq = tid < half ? __ldg(p.inv_freq + tid) : 0.f;
    const int on_axis = tid < half && p.axis_map ? __ldg(p.axis_map + tid) : 0;
    float w_of[2] = {1.f, 1.f};                               // pair tid / 2's first or second part
    if (tid < D) {
        const int pr = tid >> 1, lj = pr / H;
        const int e = kInter ? tid : E * lj >= p.rot ? E * lj + pr % H + H * (tid & 1) : pr + (tid & 1) * half;
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
            const void *w = p.weight[kind];
            if (w) w_of[kind] = p.weight_f32[kind] ? __ldg(static_cast<const float *>(w) + e)
                                                   : __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t *>(w) + e) << 16);
        }
    }
    if (p.axes == 1) look(n_first);
    if (tid < half) {
        turn[tid] = turn_of(freq);
        if ((unsigned)on_axis >= (unsigned)p.axes) record_error(p.status, kErrInvalid);
        axis[tid] = (unsigned)on_axis < (unsigned)p.axes ? on_axis : 0;
    }
    if (tid < D) {
        weight[0][(tid >> 1) + (tid & 1) * (D / 2)] = w_of[0];
        weight[1][(tid >> 1) + (tid & 1) * (D / 2)] = w_of[1];
    }
    __syncthreads();
    if (p.axes > 1) look(n_first);

    int stage = 0, g = g_first;
    int64_t rest = count;
    for (int64_t token = n_first; rest > 0; ++token, g = 0) {
        const int last = (int)min((int64_t)groups, g + rest);
        rest -= last - g;
        __syncwarp();
#pragma unroll
        for (int k = 0; k < kAngles; ++k) {
            const int f = lane + 32 * k;
            float c = 1.f, s = 0.f;
            if (f < half) {
                // The nearest quarter turn and what is left, which a float holds to 2^-28 of a turn.
                const uint32_t at = (uint32_t)((uint64_t)(int64_t)pos[k] * turn[f] >> 32) + 0x20000000u;
                const int quarter = at >> 30, rest_of = (int)(at & 0x3fffffffu) - 0x20000000;
                float s0, c0;
                sincospif((float)rest_of * 4.656612873077393e-10f, &s0, &c0);       // 2^-31: half turns
                c = quarter & 1 ? s0 : c0;
                s = quarter & 1 ? c0 : s0;
                if ((quarter + 1) & 2) c = -c;
                if (quarter & 2) s = -s;
            }
            cosine[warp][f] = c;
            sine[warp][f] = s;
        }
        __syncwarp();
        // The token's cache row, if it has one.
        int64_t kdst = -1, vdst = -1;
        if (p.slots && last > nq) {
            const int64_t row = p.layer_base + slot;
            if (slot >= 0 && row < p.cache_rows) {
                const int64_t page = p.ps_shift >= 0 ? row >> p.ps_shift : row / p.ps;
                const int64_t off = row - page * p.ps;
                kdst = page * p.kc_stride[0] + off * p.kc_stride[1];
                vdst = page * p.vc_stride[0] + off * p.vc_stride[1];
            } else if (slot >= 0 && lane == 0) {
                record_error(p.status, kErrInvalid);
            }
        }
        if (rest > 0) look(token + 1);
#pragma unroll 1
        for (int kind = 0; kind < 3; ++kind) {
            const int end = min(last, kind == 0 ? nq : kind == 1 ? nq + nk : groups);
            if (g >= end) continue;
            int left = end - g;
            int h = (g - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk)) * HPW + sub;
            g = end;
            const bool code = kind > 0 && p.slots && p.kv8;
            const float scale = kind == 1 ? p.k_scale : p.v_scale, inv = kind == 1 ? p.k_inv : p.v_inv;
            int64_t step;                                     // bytes
            char *dst;
            if (kind == 0) {
                step = 2 * p.qo_stride[1];
                dst = reinterpret_cast<char *>(p.q_out + token * p.qo_stride[0]);
            } else if (!p.slots) {
                step = 2 * p.ko_stride[1];
                dst = reinterpret_cast<char *>(p.k_out + token * p.ko_stride[0]);
            } else {
                const int size = p.kv8 ? 1 : 2;
                step = size * (kind == 1 ? p.kc_stride[2] : p.vc_stride[2]);
                dst = static_cast<char *>(kind == 1 ? p.k_cache : p.v_cache) + size * (kind == 1 ? kdst : vdst);
            }
            dst += h * step;
            step *= HPW;
            h = (kind == 0 ? p.Hq : p.Hkv) - h;               // > 0: this lane's head is one
            if (kind > 0 && p.slots && kdst < 0) h = 0;       // a token without a slot
            if (kind == 2) {
                // Values: as they came, or as codes.
#pragma unroll 1
                for (; left > 0; --left, h -= HPW, dst += step) {
                    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
                    const Run<E> r0 = ring[stage][0][tid], r1 = ring[stage][1][tid];
                    stage = stage + 1 == kStages ? 0 : stage + 1;
                    fetch();
                    if (h <= 0) continue;
                    if (code) {
                        float v[E];
#pragma unroll
                        for (int i = 0; i < P; ++i) {
                            v[2 * i] = low(r0.at(i));     v[2 * i + 1] = high(r0.at(i));
                            v[H + 2 * i] = low(r1.at(i)); v[H + 2 * i + 1] = high(r1.at(i));
                        }
                        store_codes<E>(dst + E * j, dst + E * j + H, v, scale, inv);
                    } else {
                        *reinterpret_cast<Run<E> *>(dst + 2 * E * j) = r0;
                        *reinterpret_cast<Run<E> *>(dst + 2 * E * j + E) = r1;
                    }
                }
                continue;
            }
            // What a pair's parts are multiplied by: a' = a ca - b sb, b' = b cb + a sa.
            f32x2 ca[P], sb[P], cb[P], sa[P];
#pragma unroll
            for (int i = 0; i < P; i += 2) {
                const float4 wa = *reinterpret_cast<const float4 *>(&weight[kind][H * j + 2 * i]);
                const float4 wb = *reinterpret_cast<const float4 *>(&weight[kind][D / 2 + H * j + 2 * i]);
                const float4 c = *reinterpret_cast<const float4 *>(&cosine[warp][H * j + 2 * i]);
                const float4 s = *reinterpret_cast<const float4 *>(&sine[warp][H * j + 2 * i]);
                ca[i] = mul2(two(wa.x, wa.y), two(c.x, c.y));   ca[i + 1] = mul2(two(wa.z, wa.w), two(c.z, c.w));
                cb[i] = mul2(two(wb.x, wb.y), two(c.x, c.y));   cb[i + 1] = mul2(two(wb.z, wb.w), two(c.z, c.w));
                sa[i] = mul2(two(wa.x, wa.y), two(s.x, s.y));   sa[i + 1] = mul2(two(wa.z, wa.w), two(s.z, s.w));
                sb[i] = mul2(two(wb.x, wb.y), two(-s.x, -s.y)); sb[i + 1] = mul2(two(wb.z, wb.w), two(-s.z, -s.w));
            }
            const bool norm = p.weight[kind] != nullptr;
#pragma unroll 1
            for (; left > 0; --left, h -= HPW, dst += step) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
                Pairs<E, kInter> x;
                x.unpack(ring[stage][0][tid], ring[stage][1][tid]);
                stage = stage + 1 == kStages ? 0 : stage + 1;
                fetch();
                float r = 1.f;
                if (norm) {
                    float sq = x.squares();
#pragma unroll
                    for (int o = L / 2; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
                    r = rsqrtf(sq * (1.f / D) + p.eps);
                }
                const f32x2 rr = two(r, r);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    // (A lane of elements that do not turn leaves its pairs' other parts out.)
                    const f32x2 u = mul2(x.a[i], ca[i]), w = mul2(x.b[i], cb[i]);
                    const f32x2 ya = rotates ? fma2(x.b[i], sb[i], u) : u, yb = rotates ? fma2(x.a[i], sa[i], w) : w;
                    x.a[i] = mul2(ya, rr);
                    x.b[i] = mul2(yb, rr);
                }
                if (h <= 0) continue;
                float v[E];
                x.values(v);
                if (code) {
                    store_codes<E>(dst + o0, dst + o1, v, scale, inv);
                } else {
                    store_bf16<E>(dst + 2 * o0, v);
                    store_bf16<E>(dst + 2 * o1, v + H);
                }
            }
        }
    }
}

template <int D, int E>
cudaError_t launch_dim(const NormRopeParams &p, cudaStream_t stream) {
    constexpr int HPW = 32 * E / D;
    NormRopeParams a = p;
    const int nk = (p.Hkv + HPW - 1) / HPW;
    const int groups = (p.Hq + HPW - 1) / HPW + nk + (p.v ? nk : 0);
    // As many warps as fit, or as there are head groups.
    const int64_t most = (int64_t)p.num_sms * kRopeBlocks, blocks = (p.N * groups + kRopeWarps - 1) / kRopeWarps;
    const unsigned grid = (unsigned)(blocks < most ? blocks : most);
    auto usual = [](float x) { return x >= 8.67e-19f && x <= 1.15e18f; };      // 2^-60 .. 2^60
    a.k_inv = p.kv8 && usual(p.k_scale) ? 1.f / p.k_scale : 0.f;
    a.v_inv = p.kv8 && usual(p.v_scale) ? 1.f / p.v_scale : 0.f;
    const int which = 2 * (p.interleaved ? 1 : 0) + (p.rot < D ? 1 : 0);
    auto kernel = p.interleaved ? norm_rope_kernel<D, E, true, true> : norm_rope_kernel<D, E, false, true>;
    if constexpr (E == 16)
        if (p.rot == D) kernel = p.interleaved ? norm_rope_kernel<D, E, true, false> : norm_rope_kernel<D, E, false, false>;
    const int smem = kStages * 2 * kRopeThreads * (int)sizeof(Run<E>);
    static bool configured[64][4] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!configured[dev & 63][which]) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        configured[dev & 63][which] = true;
    }
    kernel<<<grid, kRopeThreads, smem, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams &p, cudaStream_t stream) {
    // Sixteen elements a lane where the rotated part divides so.
    if (p.rot % 16)
        return p.D == 64 ? launch_dim<64, 8>(p, stream) : p.D == 128 ? launch_dim<128, 8>(p, stream) : launch_dim<256, 8>(p, stream);
    return p.D == 64 ? launch_dim<64, 16>(p, stream) : p.D == 128 ? launch_dim<128, 16>(p, stream) : launch_dim<256, 16>(p, stream);
}

}  // namespace fw
