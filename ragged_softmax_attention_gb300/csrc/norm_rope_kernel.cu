// Norms of queries and keys for each head with the position rotation in the
// same pass, sm_103a; keys (and values) optionally go straight to their cache
// slots:
//   y = x * rsqrt(mean(x^2) + eps) * w
//   (y_i, y_i') -> (y_i cos a - y_i' sin a, y_i' cos a + y_i sin a),  a = pos * inv_freq_i
// with i' = i + rot / 2 (halves) or the odd neighbour (interleaved).
//
// Every element is read and written once: DRAM bounds it from a few thousand
// tokens on, latencies below.  A head takes D / 8 lanes, and a lane's eight
// elements are four whole pairs, so the rotation needs no exchange and the sum of
// squares log2(D / 8) shuffles; angles are a token's, so a warp keeps a lane's four
// cosines and sines in registers over all heads that it takes of a token.
//
// An angle is needed modulo one turn, and pos * inv_freq in 32 bits loses it (1e5
// radians are good to 0.008).  inv_freq / 2 pi is kept as a 64-bit fraction of a
// turn, worked out in 64 bits once a block; the integer product with the position
// drops whole turns by itself, exactly, for either sign.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "fw_internal.h"
#include "fw_ptx.cuh"

namespace fw {
namespace {

constexpr int kErrInvalid = 1;     // FW_ERR_INVALID_ARG
constexpr int kRopeWarps = 8;
constexpr int kAhead = 4;          // heads of a lane in flight

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
}
__device__ __forceinline__ uint2 pack_bf16x4(const float *v) {
    return make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}
// Codes of v / scale as the append stores them.
__device__ __forceinline__ uint32_t pack_e4m3x4(const float *v, float scale) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(v[0], scale), __fdiv_rn(v[1], scale)),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(v[2], scale), __fdiv_rn(v[3], scale)),
                                                 __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}
__device__ __forceinline__ void unpack_bf16x4(uint2 w, float *v) {
    v[0] = __uint_as_float(w.x << 16);
    v[1] = __uint_as_float(w.x & 0xffff0000u);
    v[2] = __uint_as_float(w.y << 16);
    v[3] = __uint_as_float(w.y & 0xffff0000u);
}

template <int D, bool kInter>
__global__ void __launch_bounds__(kRopeWarps * 32, 4) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
    constexpr int L = D / 8, HPW = 32 / L;           // lanes of a head, heads of a warp
    __shared__ uint64_t turn[D / 2];                 // inv_freq / 2 pi in 2^-64 turns
    __shared__ int axis[D / 2];
    __shared__ __align__(16) float weight[2][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < p.rot / 2; i += blockDim.x) {
        const double t = (double)__ldg(p.inv_freq + i) * 0.15915494309189533577;
        turn[i] = __double2ull_rn((t - floor(t)) * 18446744073709551616.0);
        int a = p.axis_map ? __ldg(p.axis_map + i) : 0;
        if ((unsigned)a >= (unsigned)p.axes) {
            record_error(p.status, kErrInvalid);
            a = 0;
        }
        axis[i] = a;
    }
    for (int i = threadIdx.x; i < 2 * D; i += blockDim.x) {
        const void *w = p.weight[i / D];
        if (w) weight[i / D][i % D] = p.weight_f32[i / D] ? static_cast<const float *>(w)[i % D]
                                                          : __bfloat162float(static_cast<const __nv_bfloat16 *>(w)[i % D]);
    }
    __syncthreads();

    // This lane's elements of a head: two runs of four, o0 and o1 on; as pairs
    // (o0 + i, o1 + i) for halves, neighbours when interleaved.
    const int j = lane % L, sub = lane / L;
    const bool rotates = 8 * j < p.rot;
    const int o0 = kInter || !rotates ? 8 * j : 4 * j;
    const int o1 = kInter || !rotates ? 8 * j + 4 : p.rot / 2 + 4 * j;
    const int nq = (p.Hq + HPW - 1) / HPW, nk = (p.Hkv + HPW - 1) / HPW;
    const int groups = nq + nk + (p.v ? nk : 0);
    const int64_t items = p.N * p.parts;
    for (int64_t item = (int64_t)blockIdx.x * kRopeWarps + warp; item < items; item += (int64_t)gridDim.x * kRopeWarps) {
        int64_t n = item;
        int part = 0;
        if (p.parts > 1) {
            n = item < (1ll << 31) ? (int64_t)((uint32_t)item / (uint32_t)p.parts) : item / p.parts;
            part = (int)(item - n * p.parts);
        }
        const int g0 = (int)((int64_t)groups * part / p.parts), g1 = (int)((int64_t)groups * (part + 1) / p.parts);
        // The token's cache row, if it has one.
        int64_t kdst = -1, vdst = -1;
        if (p.slots && g1 > nq) {
            const int s = __ldg(p.slots + n);
            const int64_t row = p.layer_base + s;
            if (s >= 0 && row < p.cache_rows) {
                const int64_t page = p.ps_shift >= 0 ? row >> p.ps_shift : row / p.ps;
                const int64_t off = row - page * p.ps;
                kdst = page * p.kc_stride[0] + off * p.kc_stride[1];
                vdst = page * p.vc_stride[0] + off * p.vc_stride[1];
            } else if (s >= 0 && lane == 0) {
                record_error(p.status, kErrInvalid);
            }
        }
        float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
        if (rotates && g0 < nq + nk) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t pos = __ldg(p.positions + axis[4 * j + i] * p.pos_stride + n);
                const int32_t frac = (int32_t)((uint64_t)pos * turn[4 * j + i] >> 32);
                sincospif((float)frac * 4.656612873077393e-10f, &s[i], &c[i]);      // 2^-31: half turns
            }
        }
        for (int g = g0; g < g1; g += kAhead) {
            uint2 in[kAhead][2];
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                const int gg = g + a;
                if (gg >= g1) continue;
                const int kind = gg < nq ? 0 : gg < nq + nk ? 1 : 2;
                const int h = (gg - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk)) * HPW + sub;
                if (h >= (kind == 0 ? p.Hq : p.Hkv)) continue;
                const uint16_t *src = kind == 0 ? p.q + n * p.q_stride[0] + h * p.q_stride[1]
                                    : kind == 1 ? p.k + n * p.k_stride[0] + h * p.k_stride[1]
                                                : p.v + n * p.v_stride[0] + h * p.v_stride[1];
                in[a][0] = *reinterpret_cast<const uint2 *>(src + o0);
                in[a][1] = *reinterpret_cast<const uint2 *>(src + o1);
            }
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                const int gg = g + a;
                if (gg >= g1) break;
                const int kind = gg < nq ? 0 : gg < nq + nk ? 1 : 2;
                const int h = (gg - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk)) * HPW + sub;
                const bool live = h < (kind == 0 ? p.Hq : p.Hkv);
                if (kind > 0 && p.slots && kdst < 0) continue;          // a token without a slot
                float v[8];
                unpack_bf16x4(in[a][0], v);
                unpack_bf16x4(in[a][1], v + 4);
                if (kind < 2) {
                    if (p.weight[kind]) {
                        float sq = 0.f;
#pragma unroll
                        for (int i = 0; i < 8; ++i) sq = fmaf(v[i], v[i], sq);
#pragma unroll
                        for (int o = L / 2; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
                        const float r = rsqrtf(sq * (1.f / D) + p.eps);
                        const float4 w0 = *reinterpret_cast<const float4 *>(&weight[kind][o0]);
                        const float4 w1 = *reinterpret_cast<const float4 *>(&weight[kind][o1]);
                        v[0] *= r * w0.x; v[1] *= r * w0.y; v[2] *= r * w0.z; v[3] *= r * w0.w;
                        v[4] *= r * w1.x; v[5] *= r * w1.y; v[6] *= r * w1.z; v[7] *= r * w1.w;
                    }
                    if (rotates) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int x = kInter ? 2 * i : i, y = kInter ? 2 * i + 1 : i + 4;
                            const float a0 = v[x], b0 = v[y];
                            v[x] = fmaf(a0, c[i], -b0 * s[i]);
                            v[y] = fmaf(b0, c[i], a0 * s[i]);
                        }
                    }
                }
                if (!live) continue;
                if (kind > 0 && p.kv8) {
                    const float scale = kind == 1 ? p.k_scale : p.v_scale;
                    uint8_t *dst = kind == 1 ? static_cast<uint8_t *>(p.k_cache) + kdst + h * p.kc_stride[2]
                                             : static_cast<uint8_t *>(p.v_cache) + vdst + h * p.vc_stride[2];
                    *reinterpret_cast<uint32_t *>(dst + o0) = pack_e4m3x4(v, scale);
                    *reinterpret_cast<uint32_t *>(dst + o1) = pack_e4m3x4(v + 4, scale);
                } else {
                    uint16_t *dst = kind == 0 ? p.q_out + n * p.qo_stride[0] + h * p.qo_stride[1]
                                  : kind == 2 ? static_cast<uint16_t *>(p.v_cache) + vdst + h * p.vc_stride[2]
                                  : p.slots   ? static_cast<uint16_t *>(p.k_cache) + kdst + h * p.kc_stride[2]
                                              : p.k_out + n * p.ko_stride[0] + h * p.ko_stride[1];
                    // Values go through as they came (their bits: a NaN's too).
                    *reinterpret_cast<uint2 *>(dst + o0) = kind == 2 ? in[a][0] : pack_bf16x4(v);
                    *reinterpret_cast<uint2 *>(dst + o1) = kind == 2 ? in[a][1] : pack_bf16x4(v + 4);
                }
            }
        }
    }
}

template <int D>
cudaError_t launch_dim(const NormRopeParams &p, cudaStream_t stream) {
    constexpr int HPW = 256 / D;
    NormRopeParams a = p;
    const int nk = (p.Hkv + HPW - 1) / HPW;
    const int groups = (p.Hq + HPW - 1) / HPW + nk + (p.v ? nk : 0);
    // A token's heads are shared out among so many warps that each SM has some 32 with
    // a few rounds each; with many tokens a warp takes a token whole.
    const int64_t warps = (int64_t)p.num_sms * 32;
    const int64_t parts = (4 * warps + p.N - 1) / p.N;
    a.parts = (int)(parts < groups ? parts : groups);
    if (a.parts < 1) a.parts = 1;
    const int64_t blocks = (p.N * a.parts + kRopeWarps - 1) / kRopeWarps;
    const int64_t most = (int64_t)p.num_sms * 4;
    const unsigned grid = (unsigned)(blocks < most ? blocks : most);
    if (p.interleaved) norm_rope_kernel<D, true><<<grid, kRopeWarps * 32, 0, stream>>>(a);
    else norm_rope_kernel<D, false><<<grid, kRopeWarps * 32, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams &p, cudaStream_t stream) {
    if (p.D == 64) return launch_dim<64>(p, stream);
    if (p.D == 128) return launch_dim<128>(p, stream);
    return launch_dim<256>(p, stream);
}

}  // namespace fw
