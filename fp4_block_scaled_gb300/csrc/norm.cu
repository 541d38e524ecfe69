// norm.cu -- root-mean-square norm of rows, with the residual's addition ahead of it
// and the block formats behind it, in one pass: a row stays in the registers of the
// threads that hold it, so that it is read once and everything made of it is
// written once.
//
// u = r / sqrt(mean(r^2) + eps) * w with r = x + residual: the sum of squares is the only thing
// that the threads of a row exchange (shuffles, and one barrier where a CTA holds the row).
// Bound by HBM: 16384 rows of 4096, bf16 with a bf16 residual, to bf16 and E4M3, 91 us (98 % of
// the copy rate); 16384 of 4096 without a residual 43 us (92 %); 4099 of 2880 14.6 us (84 %: 2.7
// rows a CTA); a million of 128 93 us (85 %); 11040 of 5760 without a residual to bf16 and
// E4M3 52 us (90 %).  One row of 4096 takes 1.7 us, 128 rows 3.3: a launch, a trip to memory, two exchanges.
#include <algorithm>

#include "common.cuh"
#include "lin.h"
#include "mx.cuh"

namespace moe {

namespace {

constexpr int kNormThreads = 2048;  // of an SM, at most
constexpr int kNormWarps = 4;       // of a CTA where a warp or a part of one holds a row

// (a plain load: the row may be written in place)
__device__ __forceinline__ uint4 load_once(const void* p)
{
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}

// Eight elements as they lie in memory.
template <int F32>
struct Raw8 {
    uint4 u[F32 ? 2 : 1];

    __device__ __forceinline__ void load(const void* p, size_t i)
    {
        const uint8_t* at = (const uint8_t*)p + i * (F32 ? 4 : 2);
#pragma unroll
        for (int j = 0; j < (F32 ? 2 : 1); j++) u[j] = load_once(at + 16 * j);
    }

    __device__ __forceinline__ void unpack(float (&v)[8]) const
    {
        if (F32) {
            const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[F32].x, u[F32].y, u[F32].z, u[F32].w};
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] = __uint_as_float(w[j]);
        } else {
            unpack8(u[0], v);
        }
    }
};

__device__ __forceinline__ uint4 bf16x8(const float (&v)[8])
{
    return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

// Eight elements of the row that a thread holds: as floats, or, where they are of bf16, as
// they lie in memory, in half the registers.
template <int PACKED>
struct Held8;

template <>
struct Held8<0> {
    float v[8];

    __device__ __forceinline__ void hold(const float (&f)[8], const uint4&)
    {
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = f[i];
    }

    __device__ __forceinline__ void get(float (&f)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 8; i++) f[i] = v[i];
    }
};

template <>
struct Held8<1> {
    uint4 u;

    __device__ __forceinline__ void hold(const float (&)[8], const uint4& b) { u = b; }
    __device__ __forceinline__ void get(float (&f)[8]) const { unpack8(u, f); }
};

// RES: 0 none, 1 bf16, 2 fp32.  CODES: 0 none, 1 E4M3, 2 E2M1.  V: groups of eight
// elements a thread holds.  ROW: the lanes that hold a row (8, 16 or 32), 0 if the CTA does.
// A CTA takes rows in turn and, but for those of four groups a thread, loads the next ones before
// it computes the present ones.
template <int XF32, int RES, int CODES, int V, int ROW>
__global__ void __launch_bounds__(ROW ? 32 * kNormWarps : 1024) k_norm(NormArgs a)
{
    __shared__ float s_sum[2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kLanes = ROW ? ROW : 32;
    const int tid = ROW ? (int)threadIdx.x % kLanes : (int)threadIdx.x, step = ROW ? ROW : (int)blockDim.x;
    const int rows = ROW ? 32 * kNormWarps / kLanes : 1, sub = ROW ? (int)threadIdx.x / kLanes : 0;
    const int groups = a.n / 8;
    // A CTA of up to 1024 threads has 64 registers a thread, which hold no row of four groups, the
    // next one and the weights.  So there a row of bf16 is kept as such, weights are read from L1 for
    // each row where the next one takes their place, and of four groups no row comes ahead (spilled
    // instead, 2048 rows of 32768 in bf16 with an fp32 residual took 201 us, so 142; in fp32 257, so 164;
    // 16384 of 4096 in bf16 with an fp32 residual 134, so 132).
    constexpr bool kRow32 = RES == 0 ? XF32 : RES == 2;
    constexpr bool kAhead = ROW || V < 4;
    constexpr bool kWeights = ROW || V == 1 || (V == 2 && RES <= !XF32);
    constexpr int kPacked = !ROW && V > 1 && !kRow32;
    pdl_trigger();
    pdl_wait();
    uint4 w[kWeights ? V : 1];
    Raw8<XF32> x[V];
    Raw8<RES == 2> res[V];
    // (threads behind the row's end or the last row take part in the shuffles, with zeros)
    auto load = [&](long long t) {
#pragma unroll
        for (int j = 0; j < V; j++) {
            const int g = j * step + tid;
            if (g < groups && t < a.T) {
                x[j].load(a.x, (size_t)t * a.n + 8 * g);
                if (RES) res[j].load(a.res, (size_t)t * a.n + 8 * g);
            } else {
                x[j] = Raw8<XF32>{};
                res[j] = Raw8<RES == 2>{};
            }
        }
    };
    long long first = (long long)blockIdx.x * rows;
    if (kAhead) load(first + sub);
#pragma unroll
    for (int j = 0; j < V; j++)
        if (kWeights && a.weight && j * step + tid < groups) w[kWeights ? j : 0] = __ldg(reinterpret_cast<const uint4*>(a.weight) + j * step + tid);
    for (int buf = 0; first < a.T; first += (long long)gridDim.x * rows, buf ^= 1) {
        const long long t = first + sub;
        const size_t base = (size_t)t * a.n;
        Held8<kPacked> row[V];
        float ss = 0.0f;
        if (!kAhead) load(t);
#pragma unroll
        for (int j = 0; j < V; j++) {
            const int g = j * step + tid;
            const bool in = g < groups && t < a.T;
            float v[8];
            uint4 b = x[j].u[0];
            x[j].unpack(v);
            if (RES) {
                float r[8];
                res[j].unpack(r);
#pragma unroll
                for (int i = 0; i < 8; i++) v[i] += r[i];
            }
            if (RES == 1) {
                // the norm is of the residual that is stored
                b = bf16x8(v);
                unpack8(b, v);
                if (a.res_out && in) *reinterpret_cast<uint4*>((uint16_t*)a.res_out + base + 8 * g) = b;
            } else if (RES == 2 && a.res_out && in) {
                float4* o = reinterpret_cast<float4*>((float*)a.res_out + base + 8 * g);
                o[0] = make_float4(v[0], v[1], v[2], v[3]);
                o[1] = make_float4(v[4], v[5], v[6], v[7]);
            }
            row[j].hold(v, b);
#pragma unroll
            for (int i = 0; i < 8; i++) ss = fmaf(v[i], v[i], ss);
        }
        const long long next = first + (long long)gridDim.x * rows;
        if (kAhead && next < a.T) load(next + sub);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        if (!ROW) {
            if (lane == 0) s_sum[buf][warp] = ss;
            __syncthreads();
            ss = warp_sum(lane < (int)(blockDim.x >> 5) ? s_sum[buf][lane] : 0.0f);
        }
        const float inv = 1.0f / sqrtf(ss / (float)a.n + a.eps);
#pragma unroll
        for (int j = 0; j < V; j++) {
            const int g = j * step + tid;
            const bool in = g < groups && t < a.T;
            float v[8];
            row[j].get(v);
            if (a.weight && in) {
                float wf[8];
                unpack8(kWeights ? w[kWeights ? j : 0] : __ldg(reinterpret_cast<const uint4*>(a.weight) + g), wf);
#pragma unroll
                for (int i = 0; i < 8; i++) v[i] = v[i] * inv * wf[i];
            } else {
#pragma unroll
                for (int i = 0; i < 8; i++) v[i] *= inv;
            }
            // the codes are those of the bf16 output
            uint4 u = bf16x8(v);
            if (a.out && in) *reinterpret_cast<uint4*>(a.out + base + 8 * g) = u;
            if (CODES == 0) continue;
            if (!in) u = make_uint4(0, 0, 0, 0);
            int s;
            if (CODES == 1) {
                const uint2 c = e4m3_quantise(u, s);
                if (!in) continue;
                *reinterpret_cast<uint2*>(a.codes + base + 8 * g) = c;
                if (g % 16 == 0) a.scales[(size_t)t * ((a.n + 127) / 128) + g / 16] = (uint8_t)s;
            } else {
                const uint32_t c = e2m1_quantise(u, s);
                if (!in) continue;
                *reinterpret_cast<uint32_t*>(a.codes + (base + 8 * g) / 2) = c;
                if (g % 4 == 0) a.scales[(size_t)t * (a.n / 32) + g / 4] = (uint8_t)s;
            }
        }
    }
}

template <int XF32, int RES, int CODES>
const void* pick(int v, int row)
{
    if (row)
        return row == 8    ? (const void*)k_norm<XF32, RES, CODES, 1, 8>
               : row == 16 ? (const void*)k_norm<XF32, RES, CODES, 1, 16>
               : v == 1    ? (const void*)k_norm<XF32, RES, CODES, 1, 32>
                           : (const void*)k_norm<XF32, RES, CODES, 2, 32>;
    return v == 1   ? (const void*)k_norm<XF32, RES, CODES, 1, 0>
           : v == 2 ? (const void*)k_norm<XF32, RES, CODES, 2, 0>
                    : (const void*)k_norm<XF32, RES, CODES, 4, 0>;
}

template <int XF32, int RES>
const void* pick(int codes, int v, int row)
{
    return codes == 0 ? pick<XF32, RES, 0>(v, row) : codes == 1 ? pick<XF32, RES, 1>(v, row) : pick<XF32, RES, 2>(v, row);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a0, cudaStream_t s)
{
    NormArgs a = a0;
    const int groups = a.n / 8, codes = !a.codes ? 0 : a.e2m1 ? 2 : 1, res = !a.res ? 0 : a.res_f32 ? 2 : 1;
    const int row = groups > 64 ? 0 : groups > 16 ? 32 : groups > 8 || (a.codes && !a.e2m1) ? 16 : 8;
    int v, threads;
    if (row) {
        v = groups <= row ? 1 : 2;
        threads = 32 * kNormWarps;
    } else {
        // one group a thread where the rows then run at once (128 rows of 4096 3.2 us, with two
        // 4.1) and for the most bytes a group, fp32 rows with fp32 residuals (11040 of 7872 173 us, with
        // two 182); else two (11040 of 4096 in bf16 37 us, with one 43)
        const int one = (groups + 31) / 32 * 32;
        v = groups <= 1024 && (a.T <= (long long)a.sms * (kNormThreads / one) || (a.x_f32 && res == 2)) ? 1 : groups <= 2048 ? 2 : 4;
        threads = ((groups + v - 1) / v + 31) / 32 * 32;
    }
    const void* fn = a.x_f32 ? (res == 0 ? pick<1, 0>(codes, v, row) : res == 1 ? pick<1, 1>(codes, v, row) : pick<1, 2>(codes, v, row))
                             : (res == 0 ? pick<0, 0>(codes, v, row) : res == 1 ? pick<0, 1>(codes, v, row) : pick<0, 2>(codes, v, row));
    cudaLaunchConfig_t cfg = {};
    const int rows = row ? threads / row : 1;       // of a CTA
    // CTAs that take rows in turn: as many as run at once (11040 rows of 5760 in bf16 51.7 us, with
    // a third more 57.9), and with a residual or fp32 rows up to eight times as many, two rows
    // or more each, since some SMs are faster then (11040 of 4096 in bf16 with a residual 59 us,
    // with as many as run 65; not where an SM has one CTA, whose rows then do not overlap).
    long long grid = (a.T + rows - 1LL) / rows;
    if (grid > a.sms) {
        int at_once = 0;
        const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&at_once, fn, threads, 0);
        if (e != cudaSuccess) return e;
        const long long slots = (long long)a.sms * at_once;
        const long long times = at_once == 1 || (!a.res && !a.x_f32) ? 1 : std::max(1LL, std::min(8LL, grid / (2 * slots)));
        grid = std::min(grid, slots * times);
    }
    cfg.gridDim = dim3((unsigned)grid);
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
