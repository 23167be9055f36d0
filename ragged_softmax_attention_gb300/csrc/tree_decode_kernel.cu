// Paged decode of a tree of drafted tokens, sm_103a: draft t of request b sees
// the committed keys 0 .. n - d - 1 and the drafts its mask row names.
//
// One block per (request, draft, query head): the keys pass in chunks of 128,
// one per thread, through an online softmax in base 2.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "decode_common.cuh"
#include "fw_internal.h"
#include "fw_ptx.cuh"

namespace fw {
namespace {

using dec::warp_max;
using dec::warp_sum;
constexpr float kNegInf = -__builtin_huge_valf();

template <bool kKv8>
__device__ __forceinline__ float cache_value(const void *base, int64_t i) {
    if constexpr (kKv8) {
        const __nv_fp8_e4m3 v = reinterpret_cast<const __nv_fp8_e4m3 *>(base)[i];
        return (float)v;
    } else {
        return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(base)[i]);
    }
}

template <int D, bool kKv8>
__global__ void __launch_bounds__(128) tree_decode_simple_kernel(const __grid_constant__ TreeParams p) {
    __shared__ float sq[D], sp[128], red[4];
    __shared__ int64_t vrow[128];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = blockIdx.x % p.Hq, t = (blockIdx.x / p.Hq) % p.T, b = blockIdx.x / (p.Hq * p.T);
    const int g = h / p.G;
    const int n = min(max(__ldg(p.seq_lens + b), 0), p.max_pages * p.ps);
    const int d = min(min(p.draft_lens ? max(__ldg(p.draft_lens + b), 0) : p.T, p.T), n);
    float o[D / 128], m = kNegInf, l = 0.f;
#pragma unroll
    for (int i = 0; i < D / 128; ++i) o[i] = 0.f;
    const uint16_t *qr = p.q + b * p.q_stride[0] + t * p.q_stride[1] + h * p.q_stride[2];
    for (int i = tid; i < D; i += 128) sq[i] = __uint_as_float((uint32_t)qr[i] << 16);
    __syncthreads();
    if (t < d) {
        const int32_t *mrow = p.mask + b * p.mask_stride[0] + t * p.mask_stride[1];
        for (int k0 = 0; k0 < n; k0 += 128) {
            const int key = k0 + tid, j = key - (n - d);
            const bool seen = key < n && (j < 0 || (__ldg(mrow + (j >> 5)) >> (j & 31)) & 1);
            float s = kNegInf;
            vrow[tid] = -1;
            if (seen) {
                int page = __ldg(p.block_table + b * p.bt_stride + key / p.ps);
                if ((unsigned)page >= (unsigned)p.num_pages) { record_error(p.status, 1); page = 0; }
                const int64_t kr = page * p.kc_stride[0] + (key % p.ps) * p.kc_stride[1] + g * p.kc_stride[2];
                vrow[tid] = page * p.vc_stride[0] + (key % p.ps) * p.vc_stride[1] + g * p.vc_stride[2];
                float a = 0.f;
                for (int i = 0; i < D; ++i) a = fmaf(sq[i], cache_value<kKv8>(p.k_cache, kr + i), a);
                s = a * p.scale_log2;
            }
            float x = warp_max(s);
            if (lane == 0) red[warp] = x;
            __syncthreads();
            const float mn = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
            const float mu = mn == kNegInf ? 0.f : mn;
            const float alpha = exp2f(m - mu);
            m = mn;
            const float pr = exp2f(s - mu);
            sp[tid] = pr;
            x = warp_sum(pr);
            __syncthreads();
            if (lane == 0) red[warp] = x;
            __syncthreads();
            l = l * alpha + ((red[0] + red[1]) + (red[2] + red[3]));
#pragma unroll
            for (int i = 0; i < D / 128; ++i) {
                float a = o[i] * alpha;
                for (int k = 0; k < 128; ++k)
                    if (vrow[k] >= 0) a = fmaf(sp[k], cache_value<kKv8>(p.v_cache, vrow[k] + i * 128 + tid), a);
                o[i] = a;
            }
            __syncthreads();
        }
    }
    __nv_bfloat16 *orow = reinterpret_cast<__nv_bfloat16 *>(p.out) + b * p.out_stride[0] + t * p.out_stride[1] +
                          h * p.out_stride[2];
#pragma unroll
    for (int i = 0; i < D / 128; ++i)
        orow[i * 128 + tid] = __float2bfloat16_rn(l > 0.f ? o[i] * (p.out_scale / l) : 0.f);
    if (tid == 0 && p.lse)
        p.lse[b * p.lse_stride[0] + t * p.lse_stride[1] + h * p.lse_stride[2]] =
            l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : kNegInf;
}

}  // namespace

cudaError_t launch_tree_decode(const TreeParams &p, cudaStream_t stream, int *launches) {
    const unsigned grid = (unsigned)((int64_t)p.B * p.T * p.Hq);
    if (p.D == 128 && p.kv8) tree_decode_simple_kernel<128, true><<<grid, 128, 0, stream>>>(p);
    else if (p.D == 128) tree_decode_simple_kernel<128, false><<<grid, 128, 0, stream>>>(p);
    else if (p.D == 256) tree_decode_simple_kernel<256, false><<<grid, 128, 0, stream>>>(p);
    else return cudaErrorInvalidValue;
    *launches = 1;
    return cudaGetLastError();
}

}  // namespace fw
