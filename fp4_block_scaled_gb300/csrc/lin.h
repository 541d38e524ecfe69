// lin.h -- interfaces between the C ABI of the dense projections and norms
// (lin.cu) and their kernel files.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/moe_lin.h"
#include "internal.h"

namespace moe {

// Packed weights of a linear layer (mxquant.cu makes them, linear.cu and linear_pair.cu
// stream them): tiles of 128 output features, each cut along K into units of 256 elements,
// in that order.  A unit is 128 rows of 128 bytes of codes (row-major, so that a tensor
// map can read it as E2M1 bytes or expand it to a byte an element) and then its two scale
// atoms of 512 bytes, one for 128 elements each: byte (row % 32) * 16 + (row / 32)
// * 4 + b holds the scale of row `row`'s block b, the order that tcgen05.cp moves
// into tensor memory.  Rows behind N and elements behind K have codes and scales of 0.
constexpr int kLinRows = 128;
constexpr int kLinUnitK = 256;
constexpr int kLinCodeBytes = kLinRows * kLinUnitK / 2;
constexpr int kLinAtom = 512;
constexpr int kLinUnitBytes = kLinCodeBytes + 2 * kLinAtom;

inline int lin_tiles(int n) { return (n + kLinRows - 1) / kLinRows; }
inline int lin_units(int k) { return (k + kLinUnitK - 1) / kLinUnitK; }

struct MxPackArgs {
    const uint8_t* codes;       // [N][K / 2]
    const uint8_t* scales;      // [N][K / 32]
    uint8_t* packed;
    int N, K;
};
cudaError_t launch_mx_pack(const MxPackArgs& a, cudaStream_t s);

struct MxQuantArgs {
    const uint16_t* x;          // bf16 [rows][n]
    int rows, n;
    int e2m1;                   // else E4M3
    int sms;
    uint8_t* codes;             // [rows][n / 2], or [rows][n]
    uint8_t* scales;            // [rows][n / 32], or [rows][ceil(n / 128)]
};
cudaError_t launch_mx_quant(const MxQuantArgs& a, cudaStream_t s);

struct MxValuesArgs {
    const uint8_t* codes;
    const uint8_t* scales;
    int rows, n;
    int e2m1, out_f32;
    void* out;                  // [rows][n]
};
cudaError_t launch_mx_values(const MxValuesArgs& a, cudaStream_t s);

struct NormArgs {
    const void* x;              // [T][n]
    const void* res;            // or null
    void* res_out;              // or null
    const uint16_t* weight;     // bf16 [n] or null
    uint16_t* out;              // bf16 [T][n] or null
    uint8_t* codes;             // or null
    uint8_t* scales;
    int T, n;
    int x_f32, res_f32;
    int e2m1;                   // the codes' format
    float eps;
    int sms;
};
constexpr int kNormMaxN = 32768;
cudaError_t launch_norm(const NormArgs& a, cudaStream_t s);

// What a product's plan goes by on its device, asked once for a handle.
constexpr int kLinClusterMax = 8;       // CTAs of a cluster along K, at most (the portable size)
struct LinDevice {
    int sms;
    int pairs;                          // pairs of CTAs (linear_pair.cu) that run at once
    int clusters[kLinClusterMax + 1];   // clusters of each size (linear.cu) that run at once
};

struct LinearArgs {
    const uint8_t* packed;
    const uint8_t* codes;       // rows of x: [T][K / 2] E2M1 or [T][K] E4M3
    const uint8_t* scales;      // [T][K / 32] or [T][ceil(K / 128)]
    const uint16_t* x;          // bf16 [T][K], quantised in the kernel (codes null)
    int T, N, K;
    int e2m1;
    void* y;                    // [T][N]
    int out_f32;
    int* status;
    uint32_t wait_ns;           // limit of every bounded wait in the kernels
    int withhold;               // test hook: the first CTA never reports its first stage's scales
};
constexpr uint32_t kLinWaitNs = 2000000000u;
// With the device current: its figures, and the kernels' shared-memory limits.
cudaError_t linear_init_device(LinDevice& dev);
cudaError_t linear_pair_init_device(LinDevice& dev);
// Whether the kernel quantises bf16 rows itself; else they are quantised ahead of it.
bool linear_takes_bf16(const LinearArgs& a, const LinDevice& dev);
cudaError_t launch_linear(const LinearArgs& a, const LinDevice& dev, cudaStream_t s);
// Many tokens on pairs of CTAs (linear_pair.cu).
size_t linear_pair_smem(bool e2m1);
cudaError_t launch_linear_pair(const LinearArgs& a, const LinDevice& dev, cudaStream_t s);
// The plan that launch_linear makes, for tests (no device is asked).
void linear_plan(const LinearArgs& a, const LinDevice& dev, moe_lin_test_plan_t* plan);

}  // namespace moe
