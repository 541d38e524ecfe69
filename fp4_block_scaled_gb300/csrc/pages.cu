// pages.cu -- pages of the cache copied inside every layer's pool
// (moe_kv_copy_pages).
//
// Bound: HBM, each byte read and written once.  A CTA copies a piece of one
// page's k, v or scales in one layer, all its loads in flight before its first
// store; the pieces of all pairs and layers are one grid, so that a few forked
// pages and a whole pool's compaction both fill the machine.  Measured: 512 pages
// of 262 KB in 8 layers, 2.15 GB read and written, 314 us (6.83 TB/s; a plain copy's
// rate is 6.78).
#include "common.cuh"
#include "kv.h"

namespace moe {

namespace {

// Bytes of a CTA's piece, at VEC 16-byte loads a thread.
template <int VEC>
constexpr size_t kPiece = (size_t)256 * 16 * VEC;

// blockIdx: x the pair, y the part (k, v, k scales, v scales) of a layer, z the piece
template <int VEC>
__global__ void __launch_bounds__(256) k_copy_pages(const __grid_constant__ CopyArgs a)
{
    pdl_wait();
    const int parts = a.scale_bytes ? 4 : 2;
    const int part = blockIdx.y % parts, layer = blockIdx.y / parts;
    const size_t bytes = part < 2 ? a.kv_bytes : a.scale_bytes, from = blockIdx.z * kPiece<VEC>;
    if (from >= bytes) return;
    const int src = a.pairs[2 * (size_t)blockIdx.x], dst = a.pairs[2 * (size_t)blockIdx.x + 1];
    if (src < 0 || src >= a.num_pages || dst < 0 || dst >= a.num_pages) {
        if (blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) atomicOr(a.status, kStatusBadIndex);
        return;
    }
    if (src == dst) return;
    const KvPool& p = a.pool[layer];
    uint8_t* base = (part == 0 ? p.k : part == 1 ? p.v : part == 2 ? p.ks : p.vs) + from;
    const uint4* s = reinterpret_cast<const uint4*>(base + (size_t)src * bytes);
    uint4* d = reinterpret_cast<uint4*>(base + (size_t)dst * bytes);
    const int n = (int)((bytes - from < kPiece<VEC> ? bytes - from : kPiece<VEC>) / 16);
    uint4 v[VEC];
#pragma unroll
    for (int i = 0; i < VEC; i++)
        if (i * 256 + (int)threadIdx.x < n) v[i] = __ldcg(s + i * 256 + threadIdx.x);
#pragma unroll
    for (int i = 0; i < VEC; i++)
        if (i * 256 + (int)threadIdx.x < n) d[i * 256 + threadIdx.x] = v[i];
}

template <int VEC>
cudaError_t launch(const CopyArgs& a, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.n, (unsigned)((a.scale_bytes ? 4 : 2) * a.layers), (unsigned)((a.kv_bytes + kPiece<VEC> - 1) / kPiece<VEC>));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_copy_pages<VEC>, a);
}

}  // namespace

cudaError_t copy_init_device()
{
    cudaFuncAttributes at;                      // loads them, so that a first call may be captured
    const cudaError_t e = cudaFuncGetAttributes(&at, k_copy_pages<4>);
    return e == cudaSuccess ? cudaFuncGetAttributes(&at, k_copy_pages<8>) : e;
}

cudaError_t launch_copy_pages(const CopyArgs& a, cudaStream_t s)
{
    if (a.n == 0 || a.layers == 0) return cudaSuccess;
    // Pieces of 16 KB for a short copy, which ends sooner the more CTAs share it (21 MB
    // moved: 3.4 us, 3.9 with 32 KB), of 32 KB for a long one (262 MB: 41 us, 45 with
    // 16 KB; 2.1 GB: 315 and 332 us).
    const double moved = 4.0 * a.n * a.layers * (double)(a.kv_bytes + a.scale_bytes);
    return moved < 128e6 ? launch<4>(a, s) : launch<8>(a, s);
}

}  // namespace moe
