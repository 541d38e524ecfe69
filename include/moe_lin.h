/*
 * moe_lin.h -- C ABI of the dense projections and the norms of a decode layer
 * ([A100] §然后又发现每 token 启动 2000 次内核 lists RMSNorm and the quantizers
 * around the experts): what lies between moe_attn_decode, the router and
 * moe_ffn_forward, in the same library.  The conventions, error codes and
 * types of moe_ffn.h hold here.  The weights are in the experts' format, E2M1 with one ue8m0 scale per 32, and
 * the rows in the activation formats MOE_ACT_E4M3_UE8M0_128 or
 * MOE_ACT_E2M1_UE8M0_32.  The pages give none of these formulas; they are the
 * usual ones, stated here.
 *
 * Rows of codes lie as moe_ffn_act_quant lays them:
 *   E4M3  codes uint8 [rows][n],     scales uint8 [rows][ceil(n / 128)]
 *   E2M1  codes uint8 [rows][n / 2] (low nibble = even element), scales uint8
 *         [rows][n / 32]
 * and stand for code * 2^(scale - 127) (a scale of 255: NaN).  n is a multiple
 * of 32. */
#ifndef MOE_LIN_H
#define MOE_LIN_H

#include "moe_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct moe_lin_s* moe_lin_t;

typedef struct {
    int max_tokens;         /* largest T and in_features that moe_linear is     */
    int max_in;             /* given as bf16 rows (a multiple of 32); 0: none   */
} moe_lin_config;

/* Select `device`, allocate the workspace (max_tokens rows of codes) and
 * return a handle.  Errors: INVALID_ARG, UNSUPPORTED, OOM, CUDA. */
int moe_lin_create(moe_lin_t* out, const moe_lin_config* cfg, int device);

/* Wait for `stream`, then return and clear the handle's sticky device status:
 * MOE_OK or MOE_ERR_DEVICE_TIMEOUT. */
int moe_lin_status(moe_lin_t h, void* stream);

/* Free the workspace (no call of the handle may be pending, and graphs that
 * captured its calls may not run again).  NULL is a no-op. */
void moe_lin_destroy(moe_lin_t h);

/* Root-mean-square norm of T rows, the residual added first:
 *   r = x + residual, rounded to residual_dtype     (without a residual: x)
 *   u = bf16(r / sqrt(mean(r^2) + eps) * weight)
 * and u's codes: those that moe_mx_quant gives for u.  Computed in fp32, the
 * squares too: a row whose squares sum beyond its range (elements from about
 * 1e19) comes out as zeros, and one whose squares vanish (below 1e-23) is
 * divided by sqrt(eps).
 *   d          host struct
 *   x          device [T][n] of x_dtype
 *   residual   device [T][n] of residual_dtype, or NULL
 *   residual_out  device [T][n] of residual_dtype: r; NULL: not written.  It
 *              may be residual (in place).
 *   out        device bf16 [T][n]: u; NULL: not written.  It may be x, if that
 *              is bf16.
 *   act_mode   MOE_ACT_BF16: no codes (codes and scales NULL); else the format
 *              of codes and scales, device memory
 * Outputs overlap no input, nor each other, but as said.  n is a multiple of 8
 * (with codes: of 32), at most 32768. */
typedef struct {
    const void* weight;     /* DEVICE bf16 [n], or NULL: ones                   */
    int n;
    float eps;              /* >= 0                                             */
    int x_dtype;            /* MOE_OUT_*                                        */
    int residual_dtype;     /* MOE_OUT_*                                        */
} moe_norm_desc;
int moe_rms_norm(moe_lin_t h, const moe_norm_desc* d, const void* x, const void* residual, int T, void* residual_out,
                 void* out, int act_mode, uint8_t* codes, uint8_t* scales, void* stream);

/* Rows of bf16 to codes and scales.  MOE_ACT_E4M3_UE8M0_128: as
 * moe_ffn_act_quant.  MOE_ACT_E2M1_UE8M0_32: per 32 elements the scale 2^k
 * with k the least integer such that amax <= 6 * 2^k, within -126 .. 127 (0
 * for a block of zeros), and codes to nearest even; a block with an element
 * that is not finite has the scale byte 255.  Bit-exact and deterministic.
 *   x  device bf16 [rows][n];  codes, scales  device, apart from x */
int moe_mx_quant(moe_lin_t h, const void* x, int rows, int n, int act_mode, uint8_t* codes, uint8_t* scales,
                 void* stream);

/* Codes and scales back to what they stand for, device [rows][n] of out_dtype
 * (rounded to nearest even; a bf16 holds every value from 2^-126 exactly). */
int moe_mx_values(moe_lin_t h, int act_mode, const uint8_t* codes, const uint8_t* scales, int rows, int n,
                  int out_dtype, void* out, void* stream);

/* A linear layer's weights, E2M1 [out_features][in_features] as moe_mx_quant
 * lays them, packed once at load time into the order the kernel streams.
 *   packed  device, moe_linear_packed_bytes bytes, 128-byte aligned, apart
 *           from the inputs
 * packed_bytes is 0 for sizes out of range: in_features a multiple of 32 up to
 * 2^20, out_features 1 .. 2^24. */
size_t moe_linear_packed_bytes(int out_features, int in_features);
int moe_linear_pack(moe_lin_t h, const uint8_t* codes, const uint8_t* scales, int out_features, int in_features,
                    void* packed, void* stream);

/* y[t][o] = sum_i x[t][i] * w[o][i] over T rows, for the rows and weights that
 * the codes stand for: exact products, sums in the tensor core's fp32, rounded
 * once to out_dtype.
 *   w         host struct
 *   x         device: codes of act_mode's format, with x_scales; or, x_scales
 *             NULL, bf16 [T][in_features], which the call quantises as
 *             moe_mx_quant does (T and in_features within the handle's config)
 *   y         device [T][out_features] of out_dtype, apart from the inputs
 * Deterministic.  Scales whose product with a code leaves fp32's range make
 * infinities and NaN as they would there.  The kernel reads `packed` before it
 * waits for the stream's previous kernel (programmatic dependent launch), as
 * moe_ffn_forward does its routing: packed must be written by an ordinary kernel
 * or copy, or by moe_linear_pack, not by a kernel that lets its dependents
 * launch early. */
typedef struct {
    const void* packed;     /* DEVICE, made by moe_linear_pack */
    int out_features;
    int in_features;
} moe_linear_desc;
int moe_linear(moe_lin_t h, const moe_linear_desc* w, int act_mode, const void* x, const uint8_t* x_scales, int T,
               void* y, int out_dtype, void* stream);

/* Test hook, as moe_ffn_test_set_wait: later products on h give up every
 * bounded device-side wait after wait_ns nanoseconds (at 2 GHz SM clock; at
 * most the default, 2 s, which 0 restores), and with withhold != 0 the first CTA
 * never reports the first scales it has loaded, so that its waits run out: the
 * call completes, y is incomplete, and moe_lin_status returns
 * MOE_ERR_DEVICE_TIMEOUT.  Errors: INVALID_ARG. */
int moe_lin_test_set_wait(moe_lin_t h, unsigned long long wait_ns, int withhold);

/* Test hook: the plan of moe_linear for these sizes on a device with the figures
 * given, the pure host function that the call itself uses (no handle, no GPU).
 * bf16_rows != 0: of a call without x_scales. */
typedef struct {
    int sms;
    int pairs;              /* pairs of CTAs that run at once                   */
    int clusters[9];        /* [c]: clusters of c = 2 .. 8 CTAs that do         */
} moe_lin_test_device;
typedef struct {
    int tokens;             /* of a tile; 0: tiles of pairs of CTAs             */
    int tiles;              /* (of pairs: 0, as are split and ring)             */
    int split;              /* CTAs of the cluster that cut K for a tile        */
    int ring;               /* stages                                           */
    int smem;               /* bytes of shared memory of a CTA                  */
    int tmem;               /* columns of tensor memory of a CTA                */
} moe_lin_test_plan_t;
int moe_lin_test_plan(const moe_lin_test_device* dev, int act_mode, int bf16_rows, int T, int out_features, int in_features,
                      int out_dtype, moe_lin_test_plan_t* plan);

/* Calls above with their arguments as one array of 64-bit words, in their
 * order: the same call, for language bindings that pay for every argument.
 * INVALID_ARG: an unknown op, no array, an integer outside its type. */
enum { MOE_LIN_CALL_RMS_NORM = 0, MOE_LIN_CALL_QUANT = 1, MOE_LIN_CALL_VALUES = 2, MOE_LIN_CALL_LINEAR = 3 };
int moe_lin_call(int op, const int64_t* words);

#ifdef __cplusplus
}
#endif
#endif /* MOE_LIN_H */
