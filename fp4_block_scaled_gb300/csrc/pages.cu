// pages.cu -- pages of the cache copied inside every layer's pool
// (moe_kv_copy_pages).
//
// One CTA per (pair, layer, part) where the parts are k, v and their scales.
#include "common.cuh"
#include "kv.h"

namespace moe {

namespace {

__global__ void __launch_bounds__(256) k_copy_pages(const __grid_constant__ CopyArgs a)
{
    pdl_wait();
    const int part = blockIdx.y & 3, layer = blockIdx.y >> 2;
    const int src = a.pairs[2 * (size_t)blockIdx.x], dst = a.pairs[2 * (size_t)blockIdx.x + 1];
    if (src < 0 || src >= a.num_pages || dst < 0 || dst >= a.num_pages) {
        if (blockIdx.y == 0 && threadIdx.x == 0) atomicOr(a.status, kStatusBadIndex);
        return;
    }
    const KvPool& p = a.pool[layer];
    uint8_t* base = part == 0 ? p.k : part == 1 ? p.v : part == 2 ? p.ks : p.vs;
    const size_t bytes = part < 2 ? a.kv_bytes : a.scale_bytes;
    if (bytes == 0 || src == dst) return;
    const uint4* from = reinterpret_cast<const uint4*>(base + (size_t)src * bytes);
    uint4* to = reinterpret_cast<uint4*>(base + (size_t)dst * bytes);
    for (size_t i = threadIdx.x; i < bytes / 16; i += blockDim.x) to[i] = from[i];
}

}  // namespace

cudaError_t launch_copy_pages(const CopyArgs& a, cudaStream_t s)
{
    if (a.n == 0 || a.layers == 0) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.n, (unsigned)(4 * a.layers));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_copy_pages, a);
}

}  // namespace moe
