// attn.cu -- attention of one new token per sequence over the paged cache.
//
// One warp per (sequence, query head): the keys one after another, the
// running maximum and sum of the softmax in fp32, the output vector in
// registers (lane l holds elements 4l .. 4l+3).
#include "common.cuh"
#include "kv.h"

namespace moe {

namespace {

__device__ __forceinline__ void load4(const uint8_t* base, size_t row, int D, int lane, int e4m3, float f, float (&x)[4])
{
    if (e4m3) {
        const uint32_t u = *reinterpret_cast<const uint32_t*>(base + row * D + 4 * lane);
#pragma unroll
        for (int i = 0; i < 4; i++)
            x[i] = __half2float(__half(__nv_cvt_fp8_to_halfraw((uint8_t)(u >> (8 * i)), __NV_E4M3))) * f;
    } else {
        const uint2 u = *reinterpret_cast<const uint2*>(base + (row * D + 4 * lane) * 2);
        x[0] = __uint_as_float(u.x << 16);
        x[1] = __uint_as_float(u.x & 0xFFFF0000u);
        x[2] = __uint_as_float(u.y << 16);
        x[3] = __uint_as_float(u.y & 0xFFFF0000u);
    }
}

// 2^(s - 127); 255 is the NaN scale
__device__ __forceinline__ float ue8m0_value(uint32_t s)
{
    return __uint_as_float(s == 0 ? 0x00400000u : s == 255 ? 0x7FFFFFFFu : s << 23);
}

__global__ void __launch_bounds__(128) k_attn(AttnArgs a)
{
    pdl_wait();
    const int w = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (w >= a.B * a.hq) return;
    const int b = w / a.hq, hq = w % a.hq, h = hq / (a.hq / a.hkv);
    const bool in = 4 * lane < a.D;
    int n = a.lens[b];
    const int cap = a.row * a.page_size;
    if ((n < 0 || n > cap) && lane == 0) atomicOr(a.status, kStatusBadIndex);
    n = min(max(n, 0), cap);
    const int first = a.window > 0 ? max(0, n - a.window) : 0;
    float q[4] = {}, o[4] = {}, m = -INFINITY, l = 0.0f;
    if (in) load4((const uint8_t*)a.q, (size_t)b * a.hq + hq, a.D, lane, 0, 1.0f, q);
    for (int j = first; j < n; j++) {
        const int page = a.table[(size_t)b * a.row + j / a.page_size];
        if (page < 0 || page >= a.num_pages) {
            if (lane == 0) atomicOr(a.status, kStatusBadIndex);
            continue;
        }
        const size_t row = ((size_t)page * a.hkv + h) * a.page_size + j % a.page_size;
        float x[4] = {};
        if (in) load4(a.pool.k, row, a.D, lane, a.e4m3, a.e4m3 ? ue8m0_value(a.pool.ks[row]) : 1.0f, x);
        float s = warp_sum(q[0] * x[0] + q[1] * x[1] + q[2] * x[2] + q[3] * x[3]) * a.scale;
        if (a.softcap > 0.0f) s = a.softcap * tanhf(s / a.softcap);
        const float m1 = fmaxf(m, s), down = expf(m - m1), p = expf(s - m1);
        l = l * down + p;
        if (in) load4(a.pool.v, row, a.D, lane, a.e4m3, a.e4m3 ? ue8m0_value(a.pool.vs[row]) : 1.0f, x);
#pragma unroll
        for (int i = 0; i < 4; i++) o[i] = o[i] * down + p * x[i];
        m = m1;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    if (in) {
        const size_t at = ((size_t)b * a.hq + hq) * a.D + 4 * lane;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if (a.out_f32) ((float*)a.out)[at + i] = o[i] * inv;
            else ((__nv_bfloat16*)a.out)[at + i] = __float2bfloat16_rn(o[i] * inv);
        }
    }
    if (lane == 0 && a.lse) a.lse[(size_t)b * a.hq + hq] = l == 0.0f ? -INFINITY : m + logf(l);
}

}  // namespace

cudaError_t launch_attn(const AttnArgs& a, cudaStream_t s)
{
    if (a.B == 0) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.B * a.hq + 3) / 4));
    cfg.blockDim = dim3(128);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_attn, a);
}

}  // namespace moe
