// norm.cu -- root-mean-square norm of rows, with the residual's addition ahead of it
// and the block formats behind it, in one pass: a row stays in the registers of the
// threads that hold it, so that it is read once and everything made of it is
// written once.
#include "common.cuh"
#include "lin.h"
#include "mx.cuh"

namespace moe {

namespace {

constexpr int kNormWarps = 4;       // rows of a CTA where a warp holds a row

// (a plain load: the row may be written in place)
__device__ __forceinline__ uint4 load_once(const void* p)
{
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}

template <int F32>
__device__ __forceinline__ void load8(const void* p, size_t i, float (&v)[8])
{
    if (F32) {
        const uint4 a = load_once((const float*)p + i), b = load_once((const float*)p + i + 4);
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = __uint_as_float(w[j]);
    } else {
        unpack8(load_once((const uint16_t*)p + i), v);
    }
}

__device__ __forceinline__ uint4 bf16x8(const float (&v)[8])
{
    return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

// RES: 0 none, 1 bf16, 2 fp32.  CODES: 0 none, 1 E4M3, 2 E2M1.  V: groups of eight
// elements a thread holds.  ROW: 1 if a warp holds a row, else the CTA does.
template <int XF32, int RES, int CODES, int V, int ROW>
__global__ void __launch_bounds__(ROW ? 32 * kNormWarps : 1024) k_norm(NormArgs a)
{
    __shared__ float s_sum[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tid = ROW ? lane : (int)threadIdx.x, step = ROW ? 32 : (int)blockDim.x;
    const long long t = ROW ? (long long)blockIdx.x * kNormWarps + warp : (long long)blockIdx.x;
    const int groups = a.n / 8;
    pdl_trigger();
    pdl_wait();
    if (ROW && t >= a.T) return;
    const size_t base = (size_t)t * a.n;
    float v[V][8];
    uint4 w[V];
#pragma unroll
    for (int j = 0; j < V; j++) {
        const int g = j * step + tid;
        if (g < groups) {
            load8<XF32>(a.x, base + 8 * g, v[j]);
            if (a.weight) w[j] = __ldg(reinterpret_cast<const uint4*>(a.weight) + g);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) v[j][i] = 0.0f;
        }
    }
    if (RES) {
#pragma unroll
        for (int j = 0; j < V; j++) {
            const int g = j * step + tid;
            if (g >= groups) continue;
            float r[8];
            load8<RES == 2>(a.res, base + 8 * g, r);
#pragma unroll
            for (int i = 0; i < 8; i++) v[j][i] += r[i];
            if (RES == 1) {
                // the norm is of the residual that is stored
                const uint4 b = bf16x8(v[j]);
                unpack8(b, v[j]);
                if (a.res_out) *reinterpret_cast<uint4*>((uint16_t*)a.res_out + base + 8 * g) = b;
            } else if (a.res_out) {
                float4* o = reinterpret_cast<float4*>((float*)a.res_out + base + 8 * g);
                o[0] = make_float4(v[j][0], v[j][1], v[j][2], v[j][3]);
                o[1] = make_float4(v[j][4], v[j][5], v[j][6], v[j][7]);
            }
        }
    }
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < V; j++)
#pragma unroll
        for (int i = 0; i < 8; i++) ss = fmaf(v[j][i], v[j][i], ss);
    ss = warp_sum(ss);
    if (!ROW) {
        if (lane == 0) s_sum[warp] = ss;
        __syncthreads();
        ss = warp_sum(lane < (int)(blockDim.x >> 5) ? s_sum[lane] : 0.0f);
    }
    const float inv = 1.0f / sqrtf(ss / (float)a.n + a.eps);
#pragma unroll
    for (int j = 0; j < V; j++) {
        const int g = j * step + tid;
        const bool in = g < groups;
        float wf[8];
        if (a.weight && in) {
            unpack8(w[j], wf);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) wf[i] = 1.0f;
        }
#pragma unroll
        for (int i = 0; i < 8; i++) v[j][i] = v[j][i] * inv * wf[i];
        // the codes are those of the bf16 output
        const uint4 u = bf16x8(v[j]);
        if (a.out && in) *reinterpret_cast<uint4*>(a.out + base + 8 * g) = u;
        if (CODES == 0) continue;
        if (in) {
            unpack8(u, v[j]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) v[j][i] = 0.0f;
        }
        int s;
        if (CODES == 1) {
            const uint2 c = e4m3_codes8(v[j], s);
            if (!in) continue;
            *reinterpret_cast<uint2*>(a.codes + base + 8 * g) = c;
            if (g % 16 == 0) a.scales[(size_t)t * ((a.n + 127) / 128) + g / 16] = (uint8_t)s;
        } else {
            const uint32_t c = e2m1_codes8(v[j], s);
            if (!in) continue;
            *reinterpret_cast<uint32_t*>(a.codes + (base + 8 * g) / 2) = c;
            if (g % 4 == 0) a.scales[(size_t)t * (a.n / 32) + g / 4] = (uint8_t)s;
        }
    }
}

template <int XF32, int RES, int CODES>
const void* pick(int v, bool row)
{
    if (row)
        return v == 1   ? (const void*)k_norm<XF32, RES, CODES, 1, 1>
               : v == 2 ? (const void*)k_norm<XF32, RES, CODES, 2, 1>
                        : (const void*)k_norm<XF32, RES, CODES, 4, 1>;
    return v == 1   ? (const void*)k_norm<XF32, RES, CODES, 1, 0>
           : v == 2 ? (const void*)k_norm<XF32, RES, CODES, 2, 0>
                    : (const void*)k_norm<XF32, RES, CODES, 4, 0>;
}

template <int XF32, int RES>
const void* pick(int codes, int v, bool row)
{
    return codes == 0 ? pick<XF32, RES, 0>(v, row) : codes == 1 ? pick<XF32, RES, 1>(v, row) : pick<XF32, RES, 2>(v, row);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a0, cudaStream_t s)
{
    NormArgs a = a0;
    const int groups = a.n / 8;
    const bool row = groups <= 128;
    int v, threads;
    if (row) {
        v = groups <= 32 ? 1 : groups <= 64 ? 2 : 4;
        threads = 32 * kNormWarps;
    } else {
        v = groups <= 512 ? 1 : groups <= 1024 ? 2 : 4;
        threads = ((groups + v - 1) / v + 31) / 32 * 32;
    }
    const int codes = !a.codes ? 0 : a.e2m1 ? 2 : 1, res = !a.res ? 0 : a.res_f32 ? 2 : 1;
    const void* fn = a.x_f32 ? (res == 0 ? pick<1, 0>(codes, v, row) : res == 1 ? pick<1, 1>(codes, v, row) : pick<1, 2>(codes, v, row))
                             : (res == 0 ? pick<0, 0>(codes, v, row) : res == 1 ? pick<0, 1>(codes, v, row) : pick<0, 2>(codes, v, row));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(row ? (a.T + kNormWarps - 1) / kNormWarps : a.T));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* args[] = {&a};
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace moe
