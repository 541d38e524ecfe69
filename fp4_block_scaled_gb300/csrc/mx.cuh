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

// The largest magnitude of the LANES x 8 elements of a block, as bits: of finite values
// and infinities their order is that of the bits, and a NaN is above every number.
template <int LANES>
__device__ __forceinline__ float block_amax(const float (&v)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; j++) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    return __uint_as_float(m);
}

// Eight elements of a block of 32 that four neighbouring threads hold: their codes (the
// first in the lowest nibble) and the block's scale byte.  A block with an element that
// is not finite has the byte 255 and codes of +6.  Every thread of the warp calls it.
__device__ __forceinline__ uint32_t e2m1_codes8(const float (&v)[8], int& s)
{
    const float amax = block_amax<4>(v);
    if (!(amax < __uint_as_float(0x7F800000u))) {
        s = 255;
        return 0x77777777u;
    }
    s = e2m1_scale_byte(amax);
    const float down = exp2i(127 - s);
    uint32_t c = 0;
#pragma unroll
    for (int j = 0; j < 4; j++) c |= f32x2_to_e2m1x2(v[2 * j] * down, v[2 * j + 1] * down) << (8 * j);
    return c;
}

// Eight elements of a block of 128 that sixteen neighbouring threads hold.  A block with
// an element that is not finite has the byte 255 and codes of NaN.
__device__ __forceinline__ uint2 e4m3_codes8(const float (&v)[8], int& s)
{
    const float amax = block_amax<16>(v);
    s = amax < __uint_as_float(0x7F800000u) ? ue8m0_for_amax_bits(amax) : 255;
    if (s == 255) return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
    const float down = __uint_as_float((uint32_t)(254 - s) << 23);
    uint32_t c[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; j++) c[j / 4] |= (uint32_t)e4m3_rn_sat(v[j] * down) << (8 * (j & 3));
    return make_uint2(c[0], c[1]);
}

}  // namespace moe
