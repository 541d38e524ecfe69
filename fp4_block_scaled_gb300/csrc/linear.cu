// linear.cu -- the product of rows in E2M1 or E4M3 with E2M1 weights, both with
// ue8m0 scales: y[t][n] = sum_k x[t][k] w[n][k], on block-scaled tcgen05.mma
// (kind::mxf4, K = 64 a step, or kind::mxf8f6f4, K = 32).
//
// A tile is 128 output features (the MMA's rows) by nt tokens (its columns, a
// multiple of 16).  A stage of the ring is 128 bytes of K of both operands, which TMA
// brings in the 128-byte swizzle that the MMA reads: 256 elements of E2M1, or 128 of
// E4M3, for which TMA expands the weights to a byte an element on their way.
#include <cuda.h>

#include <algorithm>

#include "common.cuh"
#include "lin.h"
#include "mx.cuh"

namespace moe {

namespace {

constexpr int kRing = 16;                  // stages, at most
constexpr int kSplitMax = 8;               // CTAs of a cluster along K, at most (the portable size)
constexpr int kWarpProd = 4, kWarpMma = 5, kWarpLoad = 6, kLoadWarps = 4;
constexpr int kThreads = (kWarpLoad + kLoadWarps) * 32;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint32_t kSmemMax = 227 * 1024;

struct __align__(1024) Control {
    uint64_t full[kRing], empty[kRing], acc_full[2], acc_empty[2], drain;
    uint32_t tmem;
    int abort;
};

struct Plan {
    int nt, ttiles, rtiles;     // token columns of a tile, tiles along T and N
    int steps;                  // stages along K
    int units;                  // of the packed weights along K
    int split;                  // CTAs along K
    int width;                  // columns that each of them sums
    int ring;
    // Warps that load scales, a stage each in turn: no more than the ring has stages, or a
    // warp could wait for a slot that is two rounds behind it, whose barrier has the parity
    // of the round that it waits for.
    int loaders;
    uint32_t b, sfa, sfb, stage;        // byte offsets in a stage, and its size
    uint32_t part;                      // byte offset of the partial sums
    uint32_t smem;
    int sfcols;                 // tensor memory columns of a stage's scales
};

__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr)
{
    return (uint64_t)((saddr >> 4) & 0x3FFF) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}

template <int E2M1>
__device__ __forceinline__ uint32_t idesc(uint32_t n, uint32_t sf)
{
    const uint32_t type = E2M1 ? (1u << 7) | (1u << 10) : (5u << 7);
    return type | ((n >> 3) << 17) | (1u << 23) | ((uint32_t)(kLinRows >> 4) << 24) | (sf << 29) | (sf << 4);
}

template <int E2M1>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t sfa, uint32_t sfb, uint32_t acc)
{
    if (E2M1)
        tc_mma_mxf4(d, a, b, id, sfa, sfb, acc);
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(id), "r"(acc), "r"(sfa), "r"(sfb)
            : "memory");
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

__device__ __forceinline__ void st_cluster(uint32_t saddr, uint32_t rank, float v)
{
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\tst.shared::cluster.f32 [a], %2;\n\t}" ::"r"(saddr),
                 "r"(rank), "f"(v)
                 : "memory");
}

__device__ __forceinline__ void give_up(const LinearArgs& a, Control& ctl)
{
    atomicOr(a.status, kStatusTimeout);
    *(volatile int*)&ctl.abort = 1;
}

__device__ __forceinline__ void store(const LinearArgs& a, long long t, long long n, float v)
{
    const size_t i = (size_t)t * a.N + n;
    if (a.out_f32)
        ((float*)a.y)[i] = v;
    else
        ((__nv_bfloat16*)a.y)[i] = __float2bfloat16_rn(v);
}

// Four scale bytes of a row from `at`, 0 behind its end.
__device__ __forceinline__ uint32_t scale_word(const uint8_t* row, int at, int n)
{
    if (n % 4 == 0) return at < n ? *reinterpret_cast<const uint32_t*>(row + at) : 0u;
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; i++)
        if (at + i < n) w |= (uint32_t)row[at + i] << (8 * i);
    return w;
}

// The scales of a stage's token rows into their atoms, by one warp.
template <int E2M1>
__device__ __forceinline__ void load_scales(const LinearArgs& a, const Plan& p, uint8_t* sfb, int t0, int step, int lane)
{
    const int atoms = p.nt > 128 ? 2 : 1, n = E2M1 ? a.K / 32 : (a.K + 127) / 128;
    for (int r = lane; r < p.nt; r += 32) {
        uint8_t* at = sfb + (r / 128) * kLinAtom + (r % 32) * 16 + (r % 128) / 32 * 4;
        const bool in = t0 + r < a.T;
        const uint8_t* row = a.scales + (size_t)(t0 + r) * n;
        if (E2M1) {
            *reinterpret_cast<uint32_t*>(at) = in ? scale_word(row, 8 * step, n) : 0u;
            *reinterpret_cast<uint32_t*>(at + atoms * kLinAtom) = in ? scale_word(row, 8 * step + 4, n) : 0u;
        } else {
            *reinterpret_cast<uint32_t*>(at) = in ? row[step] * 0x01010101u : 0u;
        }
    }
}

template <int E2M1>
__global__ void __launch_bounds__(kThreads, 1)
    k_linear(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap, LinearArgs a, Plan p)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    Control& ctl = *reinterpret_cast<Control*>(smem);
    uint8_t* ring = smem + sizeof(Control);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kRing; s++) {
            mbar_init(&ctl.full[s], 2);
            mbar_init(&ctl.empty[s], 1);
        }
        for (int b = 0; b < 2; b++) {
            mbar_init(&ctl.acc_full[b], 1);
            mbar_init(&ctl.acc_empty[b], 4);
        }
        mbar_init(&ctl.drain, 1);
        ctl.abort = 0;
        mbar_fence_init();
    }
    if (warp == kWarpMma) tmem_alloc(&ctl.tmem, 512);
    tc_fence_before();
    if (p.split > 1)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem;
    pdl_trigger();
    pdl_wait();

    const uint32_t rank = p.split > 1 ? cluster_rank() : 0;
    const int k0 = (int)((long long)p.steps * rank / p.split), k1 = (int)((long long)p.steps * (rank + 1) / p.split);
    const int tiles = p.ttiles * p.rtiles, first = (int)blockIdx.x / p.split, stride = (int)gridDim.x / p.split;
    uint32_t c = 0, it = 0;

    if (warp == kWarpProd) {
        if (lane == 0) {
            bool ok = true;
            for (int i = first; i < tiles && ok; i += stride) {
                const int rt = i % p.rtiles, t0 = i / p.rtiles * p.nt;
                for (int k = k0; k < k1; k++, c++) {
                    const uint32_t slot = c % p.ring;
                    if (!mbar_wait_or_abort(&ctl.empty[slot], (c / p.ring & 1) ^ 1, &ctl.abort, kWaitNs)) {
                        give_up(a, ctl);
                        ok = false;
                        break;
                    }
                    uint8_t* st = ring + slot * p.stage;
                    uint64_t* bar = &ctl.full[slot];
                    const int z = rt * p.units + (E2M1 ? k : k / 2), half = E2M1 ? 0 : k & 1;
                    const uint32_t sf = E2M1 ? 2 * kLinAtom : kLinAtom;
                    mbar_arrive_expect_tx(bar, (E2M1 ? kLinCodeBytes : kLinCodeBytes / 2) + sf + p.nt * 128);
                    tma_3d(st, &wmap, half * 128, 0, z, bar);
                    bulk_g2s(st + p.sfa, a.packed + (size_t)z * kLinUnitBytes + kLinCodeBytes + half * kLinAtom, sf, bar);
                    tma_2d(st + p.b, &xmap, k * 128, t0, bar);
                }
            }
            // no copy may be in flight into this CTA's memory at its end
            for (uint32_t m = c > (uint32_t)p.ring ? c - p.ring : 0; m < c; m++)
                if (!mbar_wait_or_abort(&ctl.full[m % p.ring], m / p.ring & 1, &ctl.abort, kWaitNs))
                    mbar_wait_bounded(&ctl.full[m % p.ring], m / p.ring & 1, kWaitNs / 64);
        }
    } else if (warp == kWarpMma) {
        if (lane == 0) {
            bool ok = true;
            for (int i = first; i < tiles && ok; i += stride, it++) {
                const uint32_t buf = it & 1;
                ok = mbar_wait_or_abort(&ctl.acc_empty[buf], (it >> 1 & 1) ^ 1, &ctl.abort, kWaitNs);
                const uint32_t acc = tmem + buf * p.nt;
                for (int k = k0; k < k1 && ok; k++, c++) {
                    const uint32_t slot = c % p.ring;
                    ok = mbar_wait_or_abort(&ctl.full[slot], c / p.ring & 1, &ctl.abort, kWaitNs);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t st = smem_u32(ring + slot * p.stage);
                    const uint32_t sfa = tmem + 2 * p.nt + slot * p.sfcols, sfb = sfa + (E2M1 ? 8 : 4);
                    const int atoms = p.nt > 128 ? 2 : 1;
                    for (int h = 0; h < (E2M1 ? 2 : 1); h++) {
                        tc_cp_sf(sfa + 4 * h, umma_desc(st + p.sfa + h * kLinAtom, 16, 128));
                        for (int m = 0; m < atoms; m++)
                            tc_cp_sf(sfb + 4 * (atoms * h + m), umma_desc(st + p.sfb + (atoms * h + m) * kLinAtom, 16, 128));
                    }
                    const uint64_t ad = desc_sw128(st), bd = desc_sw128(st + p.b);
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const int h = E2M1 ? j / 2 : 0;
                        mma<E2M1>(acc, ad + 2 * j, bd + 2 * j, idesc<E2M1>(p.nt, E2M1 ? 2 * (j & 1) : j), sfa + 4 * h,
                                  sfb + 4 * atoms * h, k > k0 || j > 0);
                    }
                    tc_commit(&ctl.empty[slot]);
                }
                if (ok) tc_commit(&ctl.acc_full[buf]);
            }
            if (!ok) {
                // (else the epilogue has waited for the last product)
                give_up(a, ctl);
                tc_commit(&ctl.drain);
                mbar_wait_bounded(&ctl.drain, 0, kWaitNs);
            }
        }
    } else if (warp >= kWarpLoad) {
        bool ok = true;
        for (int i = first; i < tiles && ok; i += stride) {
            const int t0 = i / p.rtiles * p.nt;
            for (int k = k0; k < k1; k++, c++) {
                if (c % p.loaders != (uint32_t)(warp - kWarpLoad)) continue;
                const uint32_t slot = c % p.ring;
                ok = mbar_wait_or_abort(&ctl.empty[slot], (c / p.ring & 1) ^ 1, &ctl.abort, kWaitNs);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                load_scales<E2M1>(a, p, ring + slot * p.stage + p.sfb, t0, k, lane);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.full[slot]);
            }
        }
        if (!ok && lane == 0) give_up(a, ctl);
    } else {
        for (int i = first; i < tiles; i += stride, it++) {
            const long long t0 = (long long)(i / p.rtiles) * p.nt, n = (long long)(i % p.rtiles) * kLinRows + 32 * warp + lane;
            const uint32_t buf = it & 1;
            bool ok = mbar_wait_or_abort(&ctl.acc_full[buf], it >> 1 & 1, &ctl.abort, kWaitNs);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) {
                if (lane == 0) give_up(a, ctl);
                break;
            }
            tc_fence_after();
            const int cols = (int)min((long long)p.nt, a.T - t0);
            const uint32_t from = tmem + buf * p.nt + ((uint32_t)(32 * warp) << 16);
            for (int c0 = 0; c0 < cols; c0 += 16) {
                float v[16];
                tc_ld16(from + c0, v);
                if (p.split == 1) {
#pragma unroll
                    for (int j = 0; j < 16; j++)
                        if (c0 + j < cols && n < a.N) store(a, t0 + c0 + j, n, v[j]);
                } else {
#pragma unroll
                    for (int j = 0; j < 16; j++) {
                        const int col = c0 + j, owner = col / p.width;
                        if (col < cols)
                            st_cluster(smem_u32(smem + p.part) + (((rank * p.width + col - owner * p.width) * kLinRows) + 32 * warp + lane) * 4,
                                       owner, v[j]);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.acc_empty[buf]);
        }
    }
    __syncwarp();
    if (p.split > 1) {
        // (one tile a cluster)
        cluster_sync();
        if (warp < 4 && !*(volatile int*)&ctl.abort) {
            const long long t0 = (long long)(first / p.rtiles) * p.nt, n = (long long)(first % p.rtiles) * kLinRows + 32 * warp + lane;
            const float* part = reinterpret_cast<const float*>(smem + p.part) + 32 * warp + lane;
            const int cols = (int)min((long long)p.nt, a.T - t0);
            for (int j = 0; j < p.width; j++) {
                const int col = (int)rank * p.width + j;
                if (col >= cols) break;
                float v = 0.0f;
                for (int s = 0; s < p.split; s++) v += part[(s * p.width + j) * kLinRows];
                if (n < a.N) store(a, t0 + col, n, v);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWarpMma) tmem_dealloc(tmem, 512);
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled g_encode = nullptr;

cudaError_t encode(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* base, const cuuint64_t* dims,
                   const cuuint64_t* strides, const cuuint32_t* box)
{
    const cuuint32_t ones[3] = {1, 1, 1};
    return g_encode(map, type, (cuuint32_t)rank, (void*)base, dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

Plan make_plan(const LinearArgs& a)
{
    Plan best{};
    double least = 0;
    const int rtiles = lin_tiles(a.N), steps = a.e2m1 ? lin_units(a.K) : (a.K + 127) / 128;
    const int j0 = (a.T + 191) / 192;
    for (int j = j0; j < j0 + 4; j++) {
        Plan p{};
        p.nt = ((a.T + j - 1) / j + 15) / 16 * 16;
        p.ttiles = (a.T + p.nt - 1) / p.nt;
        p.rtiles = rtiles;
        p.steps = steps;
        p.units = lin_units(a.K);
        const long long tiles = (long long)p.ttiles * rtiles;
        p.split = (int)std::max(1LL, std::min({(long long)kSplitMax, a.sms / tiles, (long long)steps}));
        const double waves = (double)((tiles * p.split + a.sms - 1) / a.sms);
        const double cost = waves * (((steps + p.split - 1) / p.split) * std::max(p.nt, 64) + 512.0) + p.split * 64.0;
        if (j == j0 || cost < least) {
            least = cost;
            best = p;
        }
    }
    Plan p = best;
    const uint32_t sf = p.nt > 128 ? 2 : 1, h = a.e2m1 ? 2 : 1;
    p.b = kLinCodeBytes;
    p.sfa = p.b + p.nt * 128;
    p.sfb = p.sfa + h * kLinAtom;
    p.stage = (p.sfb + h * sf * kLinAtom + 1023) / 1024 * 1024;
    p.width = (p.nt + p.split - 1) / p.split;
    const uint32_t part = p.split > 1 ? p.split * p.width * kLinRows * 4 : 0;
    p.sfcols = 4 * h * (1 + sf);
    p.ring = std::min({kRing, (int)((kSmemMax - sizeof(Control) - part) / p.stage), (512 - 2 * p.nt) / p.sfcols,
                       std::max(2, (int)(p.split > 1 ? (steps + p.split - 1) / p.split : kRing))});
    p.loaders = std::min(kLoadWarps, p.ring);
    p.part = sizeof(Control) + p.ring * p.stage;
    // (more than half an SM's, so that no two CTAs of clusters share one and wait for each other's tensor memory)
    p.smem = std::max(p.part + part, kSmemMax / 2 + 2048);
    return p;
}

}  // namespace

bool linear_takes_bf16(int) { return false; }

cudaError_t linear_init_device()
{
    if (!g_encode) {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult got;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12080, cudaEnableDefault, &got);
        if (e != cudaSuccess) return e;
        if (got != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
        g_encode = (EncodeTiled)fn;
    }
    for (const void* fn : {(const void*)k_linear<0>, (const void*)k_linear<1>}) {
        const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMax);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_linear(const LinearArgs& a0, cudaStream_t s)
{
    LinearArgs a = a0;
    Plan p = make_plan(a);
    CUtensorMap wmap, xmap;
    const cuuint64_t wd[3] = {a.e2m1 ? 128u : 256u, kLinRows, (cuuint64_t)p.rtiles * p.units};
    const cuuint64_t ws[2] = {128, kLinUnitBytes};
    const cuuint32_t wb[3] = {128, kLinRows, 1};
    cudaError_t e = encode(&wmap, a.e2m1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 3, a.packed, wd, ws, wb);
    if (e != cudaSuccess) return e;
    const cuuint64_t width = a.e2m1 ? a.K / 2 : a.K;
    const cuuint64_t xd[2] = {width, (cuuint64_t)a.T}, xs[1] = {width};
    const cuuint32_t xb[2] = {128, (cuuint32_t)p.nt};
    e = encode(&xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.codes, xd, xs, xb);
    if (e != cudaSuccess) return e;
    const long long tiles = (long long)p.ttiles * p.rtiles;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.split > 1 ? tiles * p.split : std::min(tiles, (long long)a.sms)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = p.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.split > 1 ? 2 : 1;
    void* args[] = {&wmap, &xmap, &a, &p};
    return cudaLaunchKernelExC(&cfg, a.e2m1 ? (const void*)k_linear<1> : (const void*)k_linear<0>, args);
}

}  // namespace moe
