// kv.h -- interfaces between the cache's C ABI (kv.cu) and its kernel files.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/moe_ffn.h"
#include "internal.h"

namespace moe {

// One layer's pool as the kernels see it.
struct KvPool {
    uint8_t* k;
    uint8_t* v;
    uint8_t* ks;                // ue8m0 bytes per row (E4M3), else null
    uint8_t* vs;
};

struct RopeArgs {
    const uint64_t* freqs;      // [rot / 2] turns per position * 2^64; null: no rotation
    int rot, layout;
    float scale;
    const int32_t* pos;
    int T, D, hq, hk, hv;       // heads of q, k, v this call has (0: none)
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    uint16_t* q_out;
    uint16_t* k_out;            // moe_rope; the append writes the pool instead
    long long ldq, ldk, ldv, ldq_out, ldk_out;     // token strides in elements
    // append
    int append, e4m3;
    KvPool pool;
    const int32_t* seq;         // null: token t is of sequence t
    const int32_t* table;
    int num_pages, page_size, row, max_seqs;
    int* status;
    int sms;
};

struct AttnArgs {
    KvPool pool;
    const uint16_t* q;
    const int32_t* lens;
    const int32_t* table;
    int B, hq, hkv, D;
    int num_pages, page_size, row;
    int e4m3, out_f32;
    float scale, softcap;
    int window;
    void* out;
    float* lse;
    int* status;
    int sms, max_seqs;
    uint8_t* ws;                // attn_workspace's bytes
};

// The split attention's workspace: byte offsets and the size.
struct AttnWorkspace {
    size_t tickets, frags, parts, bytes;
};
constexpr int kAttnMaxSeqs = 2048;
AttnWorkspace attn_workspace(int max_seqs, int hq, int hkv, int D, int sms);
cudaError_t attn_init_device(int hq, int hkv, int D, bool e4m3, bool f32);

constexpr int kCopyLayers = 64;
struct CopyArgs {
    KvPool pool[kCopyLayers];
    int layers;
    const int32_t* pairs;
    int n, num_pages;
    size_t kv_bytes, scale_bytes;      // of a page's k (and v), of its k scales (and v scales)
    int* status;
};

cudaError_t rope_init_device();
cudaError_t copy_init_device();
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s);
cudaError_t launch_attn(const AttnArgs& a, cudaStream_t s);
cudaError_t launch_copy_pages(const CopyArgs& a, cudaStream_t s);

}  // namespace moe
