// mx.cuh -- the library's block formats in registers: eight consecutive elements a
// thread, the blocks' maxima by shuffles between neighbouring threads.
#pragma once
#include "common.cuh"

namespace moe {

__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; j++) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}

// 2^(s - 127); 255 is NaN.
__device__ __forceinline__ float ue8m0_value(int s)
{
    return s == 255 ? __uint_as_float(0x7FC00000u) : s == 0 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)s << 23);
}

__device__ __forceinline__ float e4m3_value(uint32_t code)
{
    return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)(code & 0xFF), __NV_E4M3)));
}

// The largest magnitude of the LANES x 8 elements of a block of bf16, two at a time as they
// lie in memory, as the bits of a float: of finite values and infinities their order is
// that of the bits, and a NaN is above every number.
template <int LANES>
__device__ __forceinline__ uint32_t block_amax(const uint4& u)
{
    constexpr uint32_t kAbs = 0x7FFF7FFFu;
    uint32_t m = __vmaxu2(__vmaxu2(u.x & kAbs, u.y & kAbs), __vmaxu2(u.z & kAbs, u.w & kAbs));
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    return max(m << 16, m & 0xFFFF0000u);
}

// The scale byte of a block whose largest magnitude has the bits m: k + 127 with k the
// least integer such that amax <= top 2^k; with amax = f 2^E, k is E less top's exponent, and
// one more where f is above top's fraction, which a sum carries into the exponent.  0: 127;
// not finite: 255.
__device__ __forceinline__ int e2m1_scale_of(uint32_t m)
{
    if (m >= 0x7F800000u) return 255;
    return m == 0 ? 127 : max(1, (int)((m + 0x3FFFFFu) >> 23) - 2);     // top = 1.5 * 2^2
}

__device__ __forceinline__ int e4m3_scale_of(uint32_t m)
{
    if (m >= 0x7F800000u) return 255;
    return m == 0 ? 127 : max(0, (int)((m + 0x1FFFFFu) >> 23) - 8);     // top = 1.75 * 2^8
}

// Codes of eight elements under the scale byte s, the first in the lowest bits.  Under 255
// they are +6, or NaN.
__device__ __forceinline__ uint32_t e2m1_codes8(const float (&v)[8], int s)
{
    if (s == 255) return 0x77777777u;
    const float down = exp2i(127 - s);
    uint32_t c = 0;
#pragma unroll
    for (int j = 0; j < 4; j++) c |= f32x2_to_e2m1x2(v[2 * j] * down, v[2 * j + 1] * down) << (8 * j);
    return c;
}

__device__ __forceinline__ uint2 e4m3_codes8(const float (&v)[8], int s)
{
    if (s == 255) return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
    const float down = __uint_as_float((uint32_t)(254 - s) << 23);
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; j++)
        c[j] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * j] * down, v[2 * j + 1] * down), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// Eight elements of bf16 in a block that neighbouring threads hold, four of them (E2M1) or
// sixteen (E4M3): their codes, and the block's scale byte.  Every thread of the warp calls it.
__device__ __forceinline__ uint32_t e2m1_quantise(const uint4& u, int& s)
{
    float v[8];
    unpack8(u, v);
    s = e2m1_scale_of(block_amax<4>(u));
    return e2m1_codes8(v, s);
}

__device__ __forceinline__ uint2 e4m3_quantise(const uint4& u, int& s)
{
    float v[8];
    unpack8(u, v);
    s = e4m3_scale_of(block_amax<16>(u));
    return e4m3_codes8(v, s);
}

}  // namespace moe
