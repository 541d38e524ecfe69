// mxquant.cu -- rows to the block formats (E2M1, E4M3, ue8m0 scales) and back, and the
// packing of a linear layer's weights.
//
// Bound by HBM: 16384 x 4096 to E2M1 27.2 us (92 % of the copy rate), to E4M3 32.2 (93 %), back
// 26.6 and 30.6.  Eight elements a thread, so that a warp's loads and stores are whole lines;
// a block's maximum takes three instructions and two or four shuffles, two bf16 at a time, and
// its scale byte is read off the maximum's bits without branches.
#include "common.cuh"
#include "lin.h"
#include "mx.cuh"

namespace moe {

namespace {

cudaError_t launch(const void* fn, long long blocks, int threads, cudaStream_t s, void** args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

// Eight elements a thread and turn: four threads to a block of 32 (E2M1), sixteen to one of
// 128 (E4M3).  A row of `groups` threads begins with a block of its own; E4M3 rows that end
// inside a block have threads without elements there.
// LOADS: of 16 bytes that a thread has in flight.
template <int E2M1, int LOADS>
__global__ void __launch_bounds__(256) k_mx_quant(MxQuantArgs a)
{
    pdl_trigger();
    pdl_wait();
    const int have = a.n / 8, groups = E2M1 ? have : (a.n + 127) / 128 * 16;
    const size_t all = (size_t)a.rows * groups, i0 = (size_t)blockIdx.x * (256 * LOADS) + threadIdx.x;
    uint4 u[LOADS];
    size_t at[LOADS];             // of the group among the rows' groups
    bool in[LOADS];
#pragma unroll
    for (int j = 0; j < LOADS; j++) {
        const size_t i = i0 + 256 * j;
        at[j] = i;
        in[j] = i < all;
        if (!E2M1 && groups != have) {
            const uint32_t row = (uint32_t)(i / groups);
            const int g = (int)(i - (size_t)row * groups);
            in[j] = in[j] && g < have;
            at[j] = (size_t)row * have + g;
        }
        u[j] = make_uint4(0, 0, 0, 0);
        if (in[j]) u[j] = ldg_stream_v4(a.x + 8 * at[j]);
    }
#pragma unroll
    for (int j = 0; j < LOADS; j++) {
        const size_t i = i0 + 256 * j;
        int s;
        if (E2M1) {
            const uint32_t c = e2m1_quantise(u[j], s);
            if (!in[j]) continue;
            reinterpret_cast<uint32_t*>(a.codes)[i] = c;
            if (i % 4 == 0) a.scales[i / 4] = (uint8_t)s;
        } else {
            const uint2 c = e4m3_quantise(u[j], s);
            if (!in[j]) continue;
            reinterpret_cast<uint2*>(a.codes)[at[j]] = c;
            if (i % 16 == 0) a.scales[i / 16] = (uint8_t)s;
        }
    }
}

// Eight elements a thread and turn, in rows of `groups` of them.
constexpr int kValuesTurns = 4;
template <int E2M1, int F32>
__global__ void __launch_bounds__(256) k_mx_values(MxValuesArgs a)
{
    pdl_trigger();
    pdl_wait();
    const int groups = a.n / 8, per = E2M1 ? 4 : 16;     // of a row, and of a scale
    const size_t all = (size_t)a.rows * groups, i0 = (size_t)blockIdx.x * (256 * kValuesTurns) + threadIdx.x;
    uint2 q[kValuesTurns];
    int s[kValuesTurns];
#pragma unroll
    for (int j = 0; j < kValuesTurns; j++) {
        const size_t i = i0 + 256 * j;
        if (i >= all) continue;
        if (E2M1)
            q[j].x = reinterpret_cast<const uint32_t*>(a.codes)[i];
        else
            q[j] = reinterpret_cast<const uint2*>(a.codes)[i];
        if (groups % per == 0) {
            s[j] = a.scales[i / per];
        } else {
            const uint32_t row = (uint32_t)(i / groups);
            s[j] = a.scales[(size_t)row * ((groups + per - 1) / per) + (int)(i - (size_t)row * groups) / per];
        }
    }
#pragma unroll
    for (int j = 0; j < kValuesTurns; j++) {
        const size_t i = i0 + 256 * j;
        if (i >= all) continue;
        const float up = ue8m0_value(s[j]);
        float v[8];
        if (E2M1) {
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const float2 f = e2m1x2_to_f32x2(q[j].x >> (8 * e));
                v[2 * e] = f.x * up;
                v[2 * e + 1] = f.y * up;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; e++) v[e] = e4m3_value((e < 4 ? q[j].x : q[j].y) >> (8 * (e & 3))) * up;
        }
        if (F32) {
            float4* out = reinterpret_cast<float4*>(a.out) + i * 2;
            out[0] = make_float4(v[0], v[1], v[2], v[3]);
            out[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            reinterpret_cast<uint4*>(a.out)[i] =
                make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
        }
    }
}

// One block a unit: thread r copies row r's 128 bytes of codes and its 8 scale bytes.
__global__ void __launch_bounds__(kLinRows) k_mx_pack(MxPackArgs a, int units)
{
    // (dependents start after the end: the product reads weights before it waits)
    pdl_wait();
    const int u = (int)(blockIdx.x % (unsigned)units), r = threadIdx.x;
    const long long row = (long long)(blockIdx.x / (unsigned)units) * kLinRows + r;
    uint8_t* out = a.packed + (size_t)blockIdx.x * kLinUnitBytes;
    const int k0 = u * kLinUnitK, k1 = min(a.K, k0 + kLinUnitK);
    const bool in = row < a.N;
    for (int c = 0; c < 8; c++) {
        const int k = k0 + 32 * c;
        uint4 v = make_uint4(0, 0, 0, 0);
        uint8_t s = 0;
        if (in && k < k1) {
            v = *reinterpret_cast<const uint4*>(a.codes + ((size_t)row * a.K + k) / 2);
            s = a.scales[(size_t)row * (a.K / 32) + k / 32];
        }
        *reinterpret_cast<uint4*>(out + r * 128 + c * 16) = v;
        out[kLinCodeBytes + (c / 4) * kLinAtom + (r % 32) * 16 + (r / 32) * 4 + c % 4] = s;
    }
}

}  // namespace

cudaError_t launch_mx_quant(const MxQuantArgs& a0, cudaStream_t s)
{
    MxQuantArgs a = a0;
    void* args[] = {&a};
    // two loads a thread where that leaves every SM many blocks (16384 x 4096 to E4M3 32.2 us, with
    // one 44, with four 34.4), else one (77 x 2880, quantisation and values, 2.9 us, with four 3.5)
    const long long groups = (long long)a.rows * (a.e2m1 ? a.n / 8 : (a.n + 127) / 128 * 16);
    const bool many = groups > 4096LL * a.sms;
    const void* fn = a.e2m1 ? (many ? (const void*)k_mx_quant<1, 2> : (const void*)k_mx_quant<1, 1>)
                            : (many ? (const void*)k_mx_quant<0, 2> : (const void*)k_mx_quant<0, 1>);
    const int per = many ? 512 : 256;
    return launch(fn, (groups + per - 1) / per, 256, s, args);
}

cudaError_t launch_mx_values(const MxValuesArgs& a0, cudaStream_t s)
{
    MxValuesArgs a = a0;
    void* args[] = {&a};
    const void* fn = a.e2m1 ? (a.out_f32 ? (const void*)k_mx_values<1, 1> : (const void*)k_mx_values<1, 0>)
                            : (a.out_f32 ? (const void*)k_mx_values<0, 1> : (const void*)k_mx_values<0, 0>);
    const long long per = 256 * kValuesTurns;
    return launch(fn, ((long long)a.rows * a.n / 8 + per - 1) / per, 256, s, args);
}

cudaError_t launch_mx_pack(const MxPackArgs& a0, cudaStream_t s)
{
    MxPackArgs a = a0;
    int units = lin_units(a.K);
    void* args[] = {&a, &units};
    return launch((const void*)k_mx_pack, (long long)lin_tiles(a.N) * units, kLinRows, s, args);
}

}  // namespace moe
