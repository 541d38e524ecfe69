// linear.cuh -- what the two kernels of the dense product share: operand descriptors,
// TMA and cluster helpers, the scales of token rows.
#pragma once
#include <cuda.h>

#include "common.cuh"
#include "lin.h"
#include "mx.cuh"

namespace moe {

constexpr uint32_t kLinSmemMax = 227 * 1024, kLinSmemTwo = 113 * 1024;     // of a CTA, and of each of two on an SM

// K-major operand of 128-byte rows in TMA's 128-byte swizzle, groups of 8 rows of 1 KB.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr)
{
    return (uint64_t)((saddr >> 4) & 0x3FFF) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}

__device__ __forceinline__ void tma_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
                     smem_u32(dst)),
                 "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void tma_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
                     smem_u32(dst)),
                 "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// size: a multiple of 16
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t size)
{
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(size) : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// Every thread of every CTA of the cluster.
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// The same without making memory visible: it does not wait for the stores before it.
__device__ __forceinline__ void cluster_meet()
{
    asm volatile("barrier.cluster.arrive.relaxed;\n\tbarrier.cluster.wait;" ::: "memory");
}

// Bulk copy from this CTA's shared memory to the same place's of another CTA of the
// cluster, completing on its barrier.
__device__ __forceinline__ void bulk_to_peer(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar, uint32_t rank)
{
    asm volatile(
        "{\n\t.reg .b32 d, b;\n\tmapa.shared::cluster.u32 d, %0, %4;\n\tmapa.shared::cluster.u32 b, %3, %4;\n\t"
        "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [d], [%1], %2, [b];\n\t}" ::"r"(dst),
        "r"(src), "r"(bytes), "r"(bar), "r"(rank)
        : "memory");
}

// One lane of a converged warp.  (The compiler knows by it that a single thread runs what
// follows, and keeps the operands of the tensor core's instructions in uniform registers.)
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Whether v holds in each of the `threads` threads that meet at named barrier `id`.
__device__ __forceinline__ bool all_of(int id, int threads, bool v)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbarrier.cta.red.and.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"(id), "r"(threads), "r"((uint32_t)v)
                 : "memory");
    return r != 0;
}

__device__ __forceinline__ void give_up(const LinearArgs& a, int* abort)
{
    atomicOr(a.status, kStatusTimeout);
    *(volatile int*)abort = 1;
}

__device__ __forceinline__ void store(const LinearArgs& a, long long t, long long n, float v)
{
    const size_t i = (size_t)t * a.N + n;
    if (a.out_f32)
        ((float*)a.y)[i] = v;
    else
        ((__nv_bfloat16*)a.y)[i] = __float2bfloat16_rn(v);
}

// Four features from n, a multiple of 4.
__device__ __forceinline__ void store4(const LinearArgs& a, long long t, long long n, const float4& v)
{
    if (a.N % 4 == 0) {
        if (n >= a.N) return;
        const size_t i = (size_t)t * a.N + n;
        if (a.out_f32)
            *reinterpret_cast<float4*>((float*)a.y + i) = v;
        else
            *reinterpret_cast<uint2*>((uint16_t*)a.y + i) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
        return;
    }
    const float w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; j++)
        if (n + j < a.N) store(a, t, n + j, w[j]);
}

// Warp-collective, without waiting: 32 consecutive columns of this warp's 32 lanes.
__device__ __forceinline__ void tc_ld32_nowait(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

// The scales of a stage's token rows, by one warp: lane l holds those of the rows l, l +
// 32, ...  E2M1: eight bytes, and where a row's number is no multiple of four, so that they begin
// anywhere, the three aligned words around them, all on their way at once (byte after byte, 9000
// tokens by 4832 x 4096, quantised, took 112.6 us, so 80.0; 4864 is 75.0.  A path for both kinds
// cost the aligned ones 3 %).  E4M3: the row's byte.
template <int E2M1, int ROWS>
struct Scales {
    uint32_t w[ROWS / 32][E2M1 ? 3 : 1];

    // rows of the tile from t0, `rows` of them
    __device__ __forceinline__ void load(const LinearArgs& a, int rows, int t0, int step, int lane)
    {
        const int n = E2M1 ? a.K / 32 : (a.K + 127) / 128;
        if (E2M1 && n % 4) {
            load_anywhere(a, rows, t0, step, lane, n);
            return;
        }
#pragma unroll
        for (int i = 0; i < ROWS / 32; i++) {
            if (32 * i >= rows) break;
            const int r = lane + 32 * i;
            const bool in = r < rows && t0 + r < a.T;
            const uint8_t* row = a.scales + (size_t)(t0 + r) * n;
            if (E2M1) {
                w[i][0] = in ? *reinterpret_cast<const uint32_t*>(row + 8 * step) : 0u;
                w[i][E2M1] = in && 8 * step + 4 < n ? *reinterpret_cast<const uint32_t*>(row + 8 * step + 4) : 0u;
            } else {
                w[i][0] = in ? row[step] : 0u;
            }
        }
    }

    // (words that hold a byte of the array, and of the last no byte behind it)
    __device__ __forceinline__ void load_anywhere(const LinearArgs& a, int rows, int t0, int step, int lane, int n)
    {
        const size_t size = (size_t)a.T * n;
#pragma unroll
        for (int i = 0; i < ROWS / 32; i++) {
            if (32 * i >= rows) break;
            const int r = lane + 32 * i;
            const size_t from = ((size_t)(t0 + r) * n & ~(size_t)3) + 8 * step;
            const int left = r < rows && t0 + r < a.T ? (int)min(size - from, (size_t)12) : 0;      // bytes of the array
            const uint32_t* p = reinterpret_cast<const uint32_t*>(a.scales + from);
            w[i][0] = left >= 4 ? p[0] : 0u;
            w[i][E2M1] = left >= 8 ? p[1] : 0u;
            w[i][2 * E2M1] = left >= 12 ? p[2] : 0u;
            if (left % 4) {
                // the array's last word is not whole
                uint32_t v = 0;
                for (int b = 0; b < left % 4; b++) v |= (uint32_t)a.scales[size - left % 4 + b] << 8 * b;
                w[i][0] = left < 4 ? v : w[i][0];
                w[i][E2M1] = left / 4 == 1 ? v : w[i][E2M1];
                w[i][2 * E2M1] = left / 4 == 2 ? v : w[i][2 * E2M1];
            }
        }
    }

    // (of the same rows and step)
    __device__ __forceinline__ void store(const LinearArgs& a, int rows, int t0, int step, uint8_t* atoms, int lane) const
    {
        const int per = rows > 128 ? 2 : 1, n = a.K / 32;
        if (E2M1 && n % 4) {
            const int have = n - 8 * step;
            const uint32_t lo = have < 4 ? ~(~0u << 8 * have) : ~0u, hi = have <= 4 ? 0u : have < 8 ? ~(~0u << 8 * (have - 4)) : ~0u;
#pragma unroll
            for (int i = 0; i < ROWS / 32; i++) {
                if (32 * i >= rows) break;
                uint8_t* at = atoms + (i / 4) * kLinAtom + lane * 16 + i % 4 * 4;
                const uint32_t by = (uint32_t)(t0 + lane + 32 * i) * (uint32_t)n % 4 * 8;
                *reinterpret_cast<uint32_t*>(at) = __funnelshift_r(w[i][0], w[i][E2M1], by) & lo;
                *reinterpret_cast<uint32_t*>(at + per * kLinAtom) = __funnelshift_r(w[i][E2M1], w[i][2 * E2M1], by) & hi;
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < ROWS / 32; i++) {
            if (32 * i >= rows) break;
            uint8_t* at = atoms + (i / 4) * kLinAtom + lane * 16 + i % 4 * 4;
            if (E2M1) {
                *reinterpret_cast<uint32_t*>(at) = w[i][0];
                *reinterpret_cast<uint32_t*>(at + per * kLinAtom) = w[i][E2M1];
            } else {
                *reinterpret_cast<uint32_t*>(at) = w[i][0] * 0x01010101u;
            }
        }
    }
};

// A tensor map for TMA loads of 128-byte rows in the 128-byte swizzle.
cudaError_t linear_map(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* base, const cuuint64_t* dims,
                       const cuuint64_t* strides, const cuuint32_t* box);

}  // namespace moe
