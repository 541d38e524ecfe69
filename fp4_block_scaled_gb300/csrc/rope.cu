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

// Eight bf16 values times `down`, as E4M3.
__device__ __forceinline__ uint2 quant8(const uint4& u, float down)
{
    float f[8];
    unpack8(u, f);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; i++)
        o[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(f[2 * i] * down, f[2 * i + 1] * down), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
}

// The largest magnitude of eight bf16 values, both halves (bf16 magnitudes
// order as integers, a NaN above all).
__device__ __forceinline__ uint32_t amax8(const uint4& u)
{
    constexpr uint32_t kAbs = 0x7FFF7FFFu;
    return __vmaxu2(__vmaxu2(u.x & kAbs, u.y & kAbs), __vmaxu2(u.z & kAbs, u.w & kAbs));
}

// GL lanes (a power of two) hold a token's head, 16 elements a lane as two runs
// of 8: with MOE_ROPE_HALF the rotated lanes hold a pair's halves (8 e and
// rot / 2 + 8 e), all others 16 elements in a row; either way a lane needs the
// same eight angles for every head, and computes them once.  The token's heads
// (q, k, v one after another) are dealt to gridDim.y blocks.
// AHEAD: heads whose loads a lane has in flight.  BLOCKS: blocks of an SM.  For the
// queries and keys of 16383 tokens (40 heads of 128), whose bytes alone take
// 49.5 us: 53.9 us with four heads and three blocks, 58.4 with two, 69 with one,
// 55.1 with two heads and four blocks, 68 with four.  The E4M3 append, with more
// to compute per byte, is the other way round: 16000 tokens 66.3 us with four
// heads and three blocks, 63.9 with two and four (bytes 53.2).
template <int GL, int AHEAD, int BLOCKS>
__global__ void __launch_bounds__(256, BLOCKS) k_rope(const __grid_constant__ RopeArgs a)
{
    const int e = threadIdx.x & (GL - 1);
    const int t = (int)(((size_t)blockIdx.x * 256 + threadIdx.x) / GL);
    const bool in = t < a.T && 16 * e < a.D;
    const bool rotated = a.freqs && 16 * e < a.rot;
    const bool half = rotated && a.layout == MOE_ROPE_HALF;
    const int units = a.hq + a.hk + a.hv, split = gridDim.y;
    pdl_wait();
    const int pos = t < a.T ? a.pos[t] : -1;
    const int sq = a.append && a.seq && t < a.T ? a.seq[t] : t;
    uint4 r0[AHEAD], r1[AHEAD];
    // heads [0, hq) are q's, then k's, then v's: where unit u's lane elements lie in its head
    auto turns = [&](int u) { return rotated && u < a.hq + a.hk; };
    auto at0 = [&](int u) { return turns(u) && half ? 8 * e : 16 * e; };
    auto at1 = [&](int u) { return turns(u) && half ? a.rot / 2 + 8 * e : 16 * e + 8; };
    auto load = [&](int i, int u) {
        r0[i] = r1[i] = make_uint4(0, 0, 0, 0);
        if (u >= units || !in) return;
        const uint16_t* src = u < a.hq          ? a.q + (size_t)t * a.ldq + (size_t)u * a.D
                              : u < a.hq + a.hk ? a.k + (size_t)t * a.ldk + (size_t)(u - a.hq) * a.D
                                                : a.v + (size_t)t * a.ldv + (size_t)(u - a.hq - a.hk) * a.D;
        r0[i] = *reinterpret_cast<const uint4*>(src + at0(u));
        r1[i] = *reinterpret_cast<const uint4*>(src + at1(u));
    };
#pragma unroll
    for (int i = 0; i < AHEAD; i++) load(i, blockIdx.y + i * split);
    uint64_t F[8];
    if (rotated) {
#pragma unroll
        for (int i = 0; i < 8; i++) F[i] = a.freqs[8 * e + i];
    }
    // a group's lanes share t and leave together; no shuffle crosses a group
    if (pos < 0) return;
    Turn w[8];
    if (rotated) {
#pragma unroll
        for (int i = 0; i < 8; i++) w[i] = turn_of(F[i], (uint32_t)pos, a.scale);
    }
    bool placed = false;
    size_t row = 0;             // the token's row in the pool, of head 0
    if (a.append) {
        const int pi = pos / a.page_size;
        int page = -1;
        if (sq >= 0 && sq < a.max_seqs && pi < a.row) page = a.table[(size_t)sq * a.row + pi];
        placed = page >= 0 && page < a.num_pages;
        if (placed) row = (size_t)page * a.hk * a.page_size + (pos - pi * a.page_size);
        else if (e == 0 && blockIdx.y == 0) atomicOr(a.status, kStatusBadIndex);
    }
    for (int u0 = blockIdx.y; u0 < units; u0 += AHEAD * split) {
#pragma unroll
        for (int i = 0; i < AHEAD; i++) {
            const int u = u0 + i * split;
            if (u >= units) break;
            if (turns(u)) {
                float x0[8], x1[8], y0[8], y1[8];
                unpack8(r0[i], x0);
                unpack8(r1[i], x1);
                if (a.layout == MOE_ROPE_HALF) {
#pragma unroll
                    for (int k = 0; k < 8; k++) {
                        y0[k] = x0[k] * w[k].c - x1[k] * w[k].s;
                        y1[k] = x1[k] * w[k].c + x0[k] * w[k].s;
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        y0[2 * k] = x0[2 * k] * w[k].c - x0[2 * k + 1] * w[k].s;
                        y0[2 * k + 1] = x0[2 * k + 1] * w[k].c + x0[2 * k] * w[k].s;
                        y1[2 * k] = x1[2 * k] * w[4 + k].c - x1[2 * k + 1] * w[4 + k].s;
                        y1[2 * k + 1] = x1[2 * k + 1] * w[4 + k].c + x1[2 * k] * w[4 + k].s;
                    }
                }
                r0[i] = pack8(y0);
                r1[i] = pack8(y1);
            }
            const int i0 = at0(u), i1 = at1(u);
            if (u < a.hq || !a.append) {
                uint16_t* dst = u < a.hq ? a.q_out + (size_t)t * a.ldq_out + (size_t)u * a.D
                                         : a.k_out + (size_t)t * a.ldk_out + (size_t)(u - a.hq) * a.D;
                if (in) {
                    *reinterpret_cast<uint4*>(dst + i0) = r0[i];
                    *reinterpret_cast<uint4*>(dst + i1) = r1[i];
                }
            } else if (placed) {
                const bool key = u < a.hq + a.hk;
                const size_t prow = row + (size_t)(u - a.hq - (key ? 0 : a.hk)) * a.page_size;
                uint8_t* pool = key ? a.pool.k : a.pool.v;
                if (!a.e4m3) {
                    uint16_t* dst = reinterpret_cast<uint16_t*>(pool) + prow * a.D;
                    if (in) {
                        *reinterpret_cast<uint4*>(dst + i0) = r0[i];
                        *reinterpret_cast<uint4*>(dst + i1) = r1[i];
                    }
                } else {
                    // the bf16 row quantized: its largest magnitude over the head's lanes, then the codes
                    uint32_t top = __vmaxu2(amax8(r0[i]), amax8(r1[i]));
                    top = max(top & 0xFFFFu, top >> 16);
                    const uint32_t group = ((1u << GL) - 1u) << ((threadIdx.x & 31) / GL * GL);
#pragma unroll
                    for (int o = GL / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(group, top, o));
                    const int s = ue8m0_for_amax_bits(__uint_as_float(top << 16));
                    uint2 q0 = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu), q1 = q0;
                    if (s != 255) {
                        const float down = __uint_as_float((uint32_t)(254 - s) << 23);       // 2^(127 - s)
                        q0 = quant8(r0[i], down);
                        q1 = quant8(r1[i], down);
                    }
                    if (in) {
                        *reinterpret_cast<uint2*>(pool + prow * a.D + i0) = q0;
                        *reinterpret_cast<uint2*>(pool + prow * a.D + i1) = q1;
                    }
                    if (e == 0) (key ? a.pool.ks : a.pool.vs)[prow] = (uint8_t)s;
                }
            }
            load(i, u + AHEAD * split);        // the next round's
        }
    }
}

template <int GL, int AHEAD, int BLOCKS>
cudaError_t launch_gl(const RopeArgs& a, cudaStream_t s)
{
    const int units = a.hq + a.hk + a.hv;
    const long long lanes = (long long)a.T * GL;
    // How many lanes share a token's heads.  Few tokens: enough for 512 lanes an
    // SM, up to one head each (measured, 48 heads of 128: 8 tokens 2.0 us with 48
    // sharers and 4.1 with 6; 900 tokens 5.0 us with 10, 6.4 with 6, 8.6 with 48).
    // Many tokens: eight heads each on one set of angles (16383 tokens: 63.6 us with
    // 6 sharers, 67 with 10, 79 with 1; 40 heads of them half rotated: 53.9 with 5, 58
    // with 10, 66 with 1; the E4M3 append of 16000: 63.6 with 6, 67.5 with 10, 67.8
    // with 1).
    const long long fit = (long long)a.sms * 512 / lanes;
    const int least = (units + 7) / 8;
    const int split = (int)(fit < least ? least : fit > units ? units : fit);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((lanes + 255) / 256), (unsigned)split);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_rope<GL, AHEAD, BLOCKS>, a);
}

}  // namespace

cudaError_t rope_init_device()
{
    cudaFuncAttributes at;                      // loads them, so that a first call may be captured
    const void* all[] = {(const void*)k_rope<1, 4, 3>, (const void*)k_rope<2, 4, 3>, (const void*)k_rope<4, 4, 3>,
                         (const void*)k_rope<8, 4, 3>, (const void*)k_rope<2, 2, 4>, (const void*)k_rope<4, 2, 4>,
                         (const void*)k_rope<8, 2, 4>};
    cudaError_t e = cudaSuccess;
    for (const void* k : all)
        if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, k);
    return e;
}

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s)
{
    if (a.T == 0 || a.hq + a.hk + a.hv == 0) return cudaSuccess;
    if (a.append && a.e4m3)                     // D is a multiple of 32
        return a.D <= 32 ? launch_gl<2, 2, 4>(a, s) : a.D <= 64 ? launch_gl<4, 2, 4>(a, s) : launch_gl<8, 2, 4>(a, s);
    if (a.D <= 16) return launch_gl<1, 4, 3>(a, s);
    if (a.D <= 32) return launch_gl<2, 4, 3>(a, s);
    return a.D <= 64 ? launch_gl<4, 4, 3>(a, s) : launch_gl<8, 4, 3>(a, s);
}

}  // namespace moe
