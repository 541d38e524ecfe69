// rope.cu -- rotary positions, and a step's keys and values on their way into
// the paged cache (moe_rope, moe_kv_append).
//
// The angle of pair i at position p is p f_i radians.  With F_i = f_i / 2 pi as
// a fraction of 2^64, p F_i modulo 2^64 is the angle's fraction of a turn,
// exact for every position (F_i's own rounding moves it by p 2^-65 turns), for
// one 64-bit product: no 64-bit floating point, and no range reduction of a
// large argument.  The top 32 bits give the nearest quarter turn and the rest
// r in [-1/8, 1/8] turns; sin and cos of 2 pi r, |2 pi r| <= pi / 4, are their
// Taylor sums to the 9th and 10th power (remainders below 2e-9 and 2e-10).
#include <cuda_fp8.h>

#include "common.cuh"
#include "kv.h"

namespace moe {

namespace {

struct Turn {
    float c, s;
};

// scale * (cos, sin) of the angle p F turns
__device__ __forceinline__ Turn turn_of(uint64_t F, uint32_t p, float scale)
{
    const int32_t t = (int32_t)(uint32_t)((F * (uint64_t)p) >> 32);      // turns * 2^32
    const int32_t q = (int32_t)(((uint32_t)t + 0x20000000u) >> 30);      // nearest quarter turn, mod 4
    const int32_t r = (int32_t)((uint32_t)t - ((uint32_t)q << 30));      // [-2^29, 2^29)
    const float x = (float)r * 1.46291807926716e-09f;                    // 2 pi / 2^32
    const float y = x * x;
    float s = fmaf(y, 2.75573192e-6f, -1.98412698e-4f);                  // 1/9!, -1/7!
    s = fmaf(s, y, 8.33333333e-3f);
    s = fmaf(s, y, -1.66666667e-1f);
    s = fmaf(s * y, x, x);
    float c = fmaf(y, -2.75573192e-7f, 2.48015873e-5f);                  // -1/10!, 1/8!
    c = fmaf(c, y, -1.38888889e-3f);
    c = fmaf(c, y, 4.16666667e-2f);
    c = fmaf(c, y, -0.5f);
    c = fmaf(c, y, 1.0f);
    const float cc = (q & 1) ? s : c, ss = (q & 1) ? c : s;
    Turn o;
    o.c = ((q + 1) & 2) ? -cc * scale : cc * scale;
    o.s = (q & 2) ? -ss * scale : ss * scale;
    return o;
}

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

__device__ __forceinline__ uint2 quant8(const float (&f)[8], float down)
{
    uint32_t o[2];
#pragma unroll
    for (int i = 0; i < 2; i++)
        o[i] = (uint32_t)e4m3_rn_sat(f[4 * i] * down) | ((uint32_t)e4m3_rn_sat(f[4 * i + 1] * down) << 8) |
               ((uint32_t)e4m3_rn_sat(f[4 * i + 2] * down) << 16) | ((uint32_t)e4m3_rn_sat(f[4 * i + 3] * down) << 24);
    return make_uint2(o[0], o[1]);
}

// One lane holds 16 elements of a head, as two runs of 8: with MOE_ROPE_HALF
// the rotated lanes hold a pair's halves (8 e and rot / 2 + 8 e), all others 16
// elements in a row.  GL lanes (a power of two) hold a head.
template <int GL>
__global__ void __launch_bounds__(256) k_rope(RopeArgs a, int split)
{
    pdl_wait();
    const int e = threadIdx.x & (GL - 1);
    const long long g = ((long long)blockIdx.x * blockDim.x + threadIdx.x) / GL;
    const int t = (int)(g / split), u0 = (int)(g % split);
    const bool in = t < a.T && 16 * e < a.D;
    const int pos = t < a.T ? a.pos[t] : -1;
    // no shuffle crosses a group, and a group's lanes leave together
    if (pos < 0) return;
    const bool rotated = a.freqs && 16 * e < a.rot;
    const bool half = rotated && a.layout == MOE_ROPE_HALF;
    const int c0 = half ? 8 * e : 16 * e, c1 = half ? a.rot / 2 + 8 * e : 16 * e + 8;
    Turn w[8];
    if (rotated) {
#pragma unroll
        for (int i = 0; i < 8; i++) w[i] = turn_of(a.freqs[8 * e + i], (uint32_t)pos, a.scale);
    }
    long long slot = -1;                // (page, offset) of the token, as a row of the pool without its heads
    int page = 0, off = 0;
    if (a.append) {
        const int sq = a.seq ? a.seq[t] : t;
        const int pi = pos / a.page_size;
        bool ok = sq >= 0 && sq < a.max_seqs && pi < a.row;
        if (ok) {
            page = a.table[(size_t)sq * a.row + pi];
            ok = page >= 0 && page < a.num_pages;
        }
        off = pos - pi * a.page_size;
        if (ok) slot = 0;
        else if (e == 0 && u0 == 0) atomicOr(a.status, kStatusBadIndex);
    }
    const int units = a.hq + a.hk + a.hv;
    for (int u = u0; u < units; u += split) {
        const int kind = u < a.hq ? 0 : u < a.hq + a.hk ? 1 : 2;
        const int h = kind == 0 ? u : kind == 1 ? u - a.hq : u - a.hq - a.hk;
        const uint16_t* src = kind == 0 ? a.q + (size_t)t * a.ldq : kind == 1 ? a.k + (size_t)t * a.ldk : a.v + (size_t)t * a.ldv;
        src += (size_t)h * a.D;
        const bool turn = rotated && kind != 2;
        const int i0 = turn ? c0 : 16 * e, i1 = turn ? c1 : 16 * e + 8;
        float x0[8] = {}, x1[8] = {};
        uint4 r0 = make_uint4(0, 0, 0, 0), r1 = r0;
        if (in) {
            r0 = *reinterpret_cast<const uint4*>(src + i0);
            r1 = *reinterpret_cast<const uint4*>(src + i1);
        }
        if (turn) {
            unpack8(r0, x0);
            unpack8(r1, x1);
            float y0[8], y1[8];
            if (a.layout == MOE_ROPE_HALF) {
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    y0[i] = x0[i] * w[i].c - x1[i] * w[i].s;
                    y1[i] = x1[i] * w[i].c + x0[i] * w[i].s;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    y0[2 * i] = x0[2 * i] * w[i].c - x0[2 * i + 1] * w[i].s;
                    y0[2 * i + 1] = x0[2 * i + 1] * w[i].c + x0[2 * i] * w[i].s;
                    y1[2 * i] = x1[2 * i] * w[4 + i].c - x1[2 * i + 1] * w[4 + i].s;
                    y1[2 * i + 1] = x1[2 * i + 1] * w[4 + i].c + x1[2 * i] * w[4 + i].s;
                }
            }
            r0 = pack8(y0);
            r1 = pack8(y1);
        }
        if (kind == 0 || !a.append) {
            uint16_t* dst = kind == 0 ? a.q_out + (size_t)t * a.ldq_out : a.k_out + (size_t)t * a.ldk_out;
            dst += (size_t)h * a.D;
            if (in) {
                *reinterpret_cast<uint4*>(dst + i0) = r0;
                *reinterpret_cast<uint4*>(dst + i1) = r1;
            }
            continue;
        }
        if (slot < 0) continue;
        const size_t prow = ((size_t)page * a.hk + h) * a.page_size + off;
        uint8_t* pool = kind == 1 ? a.pool.k : a.pool.v;
        if (!a.e4m3) {
            uint16_t* dst = reinterpret_cast<uint16_t*>(pool) + prow * a.D;
            if (in) {
                *reinterpret_cast<uint4*>(dst + i0) = r0;
                *reinterpret_cast<uint4*>(dst + i1) = r1;
            }
            continue;
        }
        // the bf16 row quantized: amax over the head's lanes, then 16 codes
        unpack8(r0, x0);
        unpack8(r1, x1);
        float amax = 0.0f;
        bool nan = false;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            amax = fmaxf(amax, fmaxf(fabsf(x0[i]), fabsf(x1[i])));
            nan |= x0[i] != x0[i] || x1[i] != x1[i];
        }
        if (nan) amax = __int_as_float(0x7F800000);          // a non-finite maximum, like an infinite one
        const uint32_t gmask = GL == 32 ? 0xFFFFFFFFu : ((1u << GL) - 1u) << ((threadIdx.x & 31) / GL * GL);
#pragma unroll
        for (int o = GL / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(gmask, amax, o));
        const int s = ue8m0_for_amax_bits(amax);
        uint2 q0 = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu), q1 = q0;
        if (s != 255) {
            const float down = __uint_as_float((uint32_t)(254 - s) << 23);       // 2^(127 - s)
            q0 = quant8(x0, down);
            q1 = quant8(x1, down);
        }
        if (in) {
            *reinterpret_cast<uint2*>(pool + prow * a.D + i0) = q0;
            *reinterpret_cast<uint2*>(pool + prow * a.D + i1) = q1;
        }
        if (e == 0) (kind == 1 ? a.pool.ks : a.pool.vs)[prow] = (uint8_t)s;
    }
}

template <int GL>
cudaError_t launch_gl(const RopeArgs& a, cudaStream_t s)
{
    const int units = a.hq + a.hk + a.hv;
    const int split = units;
    const long long threads = (long long)a.T * split * GL;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((threads + 255) / 256));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_rope<GL>, a, split);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s)
{
    if (a.T == 0 || a.hq + a.hk + a.hv == 0) return cudaSuccess;
    if (a.D <= 16) return launch_gl<1>(a, s);
    if (a.D <= 32) return launch_gl<2>(a, s);
    if (a.D <= 64) return launch_gl<4>(a, s);
    return launch_gl<8>(a, s);
}

}  // namespace moe
