// lin.cu -- the C ABI of the dense projections and norms: validation, the handle
// and its workspace, launches, status.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <new>

#include "lin.h"

using namespace moe;

struct moe_lin_s {
    moe_lin_config cfg;
    int device;
    LinDevice dev;
    int* status;
    uint32_t wait_ns;
    int withhold;
    uint8_t* codes;             // bf16 rows quantised ahead of a product, in the same allocation
    uint8_t* scales;
};

namespace {

struct LinGuard {
    int prev = -1;
    explicit LinGuard(int dev)
    {
        if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
        if (prev != dev) cudaSetDevice(dev);
    }
    ~LinGuard()
    {
        int cur;
        if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
    }
};

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

int cuda_rc(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

bool overlap(const void* p, size_t np, const void* q, size_t nq)
{
    const char *a = (const char*)p, *b = (const char*)q;
    return p && q && a < b + nq && b < a + np;
}

bool is_type(int t) { return t == MOE_OUT_BF16 || t == MOE_OUT_F32; }
size_t type_bytes(int t) { return t == MOE_OUT_F32 ? 4 : 2; }
bool is_codes(int mode) { return mode == MOE_ACT_E4M3_UE8M0_128 || mode == MOE_ACT_E2M1_UE8M0_32; }
size_t code_bytes(int mode, size_t rows, int n) { return rows * (mode == MOE_ACT_E2M1_UE8M0_32 ? n / 2 : n); }
size_t scale_bytes(int mode, size_t rows, int n) { return rows * (mode == MOE_ACT_E2M1_UE8M0_32 ? n / 32 : (n + 127) / 128); }

constexpr int kMaxRows = 1 << 24;       // rows of a call, and output features
constexpr int kMaxWidth = 1 << 20;      // elements of a row

int check_rows(int rows, int n)
{
    if (rows < 0 || n <= 0 || n % 32) return MOE_ERR_INVALID_ARG;
    return rows > kMaxRows || n > kMaxWidth ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

cudaError_t quantise(int sms, const void* x, int rows, int n, int mode, uint8_t* codes, uint8_t* scales, cudaStream_t s)
{
    return launch_mx_quant(MxQuantArgs{(const uint16_t*)x, rows, n, mode == MOE_ACT_E2M1_UE8M0_32, sms, codes, scales}, s);
}

// The words of a moe_lin_call, in order.
struct Words {
    const int64_t* w;
    bool ok = true;
    template <class P>
    P p()
    {
        return (P)(uintptr_t)*w++;
    }
    int i()
    {
        ok = ok && *w >= INT32_MIN && *w <= INT32_MAX;
        return (int)*w++;
    }
};

}  // namespace

extern "C" {

int moe_lin_create(moe_lin_t* out, const moe_lin_config* cfg, int device)
{
    if (!out) return MOE_ERR_INVALID_ARG;
    *out = nullptr;
    if (!cfg || cfg->max_tokens < 0 || cfg->max_in < 0 || cfg->max_in % 32) return MOE_ERR_INVALID_ARG;
    if (cfg->max_tokens > kMaxRows || cfg->max_in > kMaxWidth) return MOE_ERR_UNSUPPORTED;
    int ndev = 0;
    if (cudaGetDeviceCount(&ndev) != cudaSuccess || device < 0 || device >= ndev)
        return ndev ? MOE_ERR_INVALID_ARG : MOE_ERR_CUDA;
    LinGuard guard(device);
    moe_lin_s* h = new (std::nothrow) moe_lin_s();
    if (!h) return MOE_ERR_OOM;
    h->cfg = *cfg;
    h->device = device;
    h->wait_ns = kLinWaitNs;
    if (cudaDeviceGetAttribute(&h->dev.sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess ||
        linear_init_device(h->dev) != cudaSuccess) {
        cudaGetLastError();
        delete h;
        return MOE_ERR_CUDA;
    }
    const size_t codes = up256((size_t)cfg->max_tokens * cfg->max_in), scales = up256((size_t)cfg->max_tokens * (cfg->max_in / 32));
    void* ws = nullptr;
    if (lib_malloc(&ws, 256 + codes + scales) != cudaSuccess) {
        cudaGetLastError();
        delete h;
        return MOE_ERR_OOM;
    }
    if (lib_zero(ws, 256) != cudaSuccess) {
        cudaFree(ws);
        delete h;
        return MOE_ERR_CUDA;
    }
    h->status = (int*)ws;
    h->codes = (uint8_t*)ws + 256;
    h->scales = h->codes + codes;
    *out = h;
    return MOE_OK;
}

int moe_lin_status(moe_lin_t h, void* stream)
{
    if (!h) return MOE_ERR_INVALID_ARG;
    LinGuard guard(h->device);
    int v = 0;
    if (lib_take_status(h->status, (cudaStream_t)stream, &v) != cudaSuccess) return MOE_ERR_CUDA;
    return v & kStatusTimeout ? MOE_ERR_DEVICE_TIMEOUT : MOE_OK;
}

void moe_lin_destroy(moe_lin_t h)
{
    if (!h) return;
    LinGuard guard(h->device);
    cudaFree(h->status);
    delete h;
}

int moe_rms_norm(moe_lin_t h, const moe_norm_desc* d, const void* x, const void* residual, int T, void* residual_out, void* out,
                 int act_mode, uint8_t* codes, uint8_t* scales, void* stream)
{
    if (!h || !d || T < 0 || d->n <= 0 || !is_type(d->x_dtype) || !is_type(d->residual_dtype) || !(d->eps >= 0.0f) || !isfinite(d->eps))
        return MOE_ERR_INVALID_ARG;
    const bool coded = act_mode != MOE_ACT_BF16;
    if (coded && !is_codes(act_mode)) return MOE_ERR_INVALID_ARG;
    if (coded != (codes != nullptr) || coded != (scales != nullptr) || (residual_out && !residual)) return MOE_ERR_INVALID_ARG;
    if (d->n % (coded ? 32 : 8)) return MOE_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(residual_out, 16) || !aligned(out, 16) || !aligned(codes, 16) ||
        !aligned(scales, 16) || !aligned(d->weight, 16))
        return MOE_ERR_INVALID_ARG;
    if (d->n > kNormMaxN || T > kMaxRows) return MOE_ERR_UNSUPPORTED;
    if (T == 0) return MOE_OK;
    if (!x || (!out && !codes && !residual_out)) return MOE_ERR_INVALID_ARG;
    const size_t all = (size_t)T * d->n, nx = all * type_bytes(d->x_dtype), nr = all * type_bytes(d->residual_dtype);
    // every output apart from every input and output, but that x and out, or the two
    // residuals, may be one array
    struct {
        const void* p;
        size_t n;
    } in[] = {{x, nx}, {residual, nr}, {d->weight, (size_t)d->n * 2}},
      made[] = {{residual_out, nr}, {out, all * 2}, {codes, code_bytes(act_mode, T, d->n)}, {scales, scale_bytes(act_mode, T, d->n)}};
    for (const auto& o : made) {
        for (const auto& i : in) {
            const bool same = o.p == i.p && ((o.p == out && i.p == x && d->x_dtype == MOE_OUT_BF16) || (o.p == residual_out && i.p == residual));
            if (!same && overlap(o.p, o.n, i.p, i.n)) return MOE_ERR_INVALID_ARG;
        }
        for (const auto& q : made)
            if (&q != &o && overlap(o.p, o.n, q.p, q.n)) return MOE_ERR_INVALID_ARG;
    }
    NormArgs a{};
    a.x = x;
    a.res = residual;
    a.res_out = residual_out;
    a.weight = (const uint16_t*)d->weight;
    a.out = (uint16_t*)out;
    a.codes = codes;
    a.scales = scales;
    a.T = T;
    a.n = d->n;
    a.x_f32 = d->x_dtype == MOE_OUT_F32;
    a.res_f32 = d->residual_dtype == MOE_OUT_F32;
    a.e2m1 = act_mode == MOE_ACT_E2M1_UE8M0_32;
    a.eps = d->eps;
    a.sms = h->dev.sms;
    LinGuard guard(h->device);
    return cuda_rc(launch_norm(a, (cudaStream_t)stream));
}

int moe_mx_quant(moe_lin_t h, const void* x, int rows, int n, int act_mode, uint8_t* codes, uint8_t* scales, void* stream)
{
    if (!h || !is_codes(act_mode)) return MOE_ERR_INVALID_ARG;
    const int rc = check_rows(rows, n);
    if (rc) return rc;
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 16)) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!x || !codes || !scales) return MOE_ERR_INVALID_ARG;
    const size_t nx = (size_t)rows * n * 2, nc = code_bytes(act_mode, rows, n), ns = scale_bytes(act_mode, rows, n);
    if (overlap(codes, nc, x, nx) || overlap(scales, ns, x, nx) || overlap(codes, nc, scales, ns)) return MOE_ERR_INVALID_ARG;
    LinGuard guard(h->device);
    return cuda_rc(quantise(h->dev.sms, x, rows, n, act_mode, codes, scales, (cudaStream_t)stream));
}

int moe_mx_values(moe_lin_t h, int act_mode, const uint8_t* codes, const uint8_t* scales, int rows, int n, int out_dtype, void* out,
                  void* stream)
{
    if (!h || !is_codes(act_mode) || !is_type(out_dtype)) return MOE_ERR_INVALID_ARG;
    const int rc = check_rows(rows, n);
    if (rc) return rc;
    if (!aligned(out, 16) || !aligned(codes, 16) || !aligned(scales, 16)) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!out || !codes || !scales) return MOE_ERR_INVALID_ARG;
    const size_t no = (size_t)rows * n * type_bytes(out_dtype);
    if (overlap(out, no, codes, code_bytes(act_mode, rows, n)) || overlap(out, no, scales, scale_bytes(act_mode, rows, n)))
        return MOE_ERR_INVALID_ARG;
    LinGuard guard(h->device);
    return cuda_rc(launch_mx_values(
        MxValuesArgs{codes, scales, rows, n, act_mode == MOE_ACT_E2M1_UE8M0_32, out_dtype == MOE_OUT_F32, out}, (cudaStream_t)stream));
}

size_t moe_linear_packed_bytes(int out_features, int in_features)
{
    if (out_features <= 0 || check_rows(out_features, in_features) != MOE_OK) return 0;
    return (size_t)lin_tiles(out_features) * lin_units(in_features) * kLinUnitBytes;
}

int moe_linear_pack(moe_lin_t h, const uint8_t* codes, const uint8_t* scales, int out_features, int in_features, void* packed, void* stream)
{
    if (!h || out_features <= 0) return MOE_ERR_INVALID_ARG;
    const int rc = check_rows(out_features, in_features);
    if (rc) return rc;
    if (!codes || !scales || !packed || !aligned(codes, 16) || !aligned(scales, 16) || !aligned(packed, 128)) return MOE_ERR_INVALID_ARG;
    const size_t n = moe_linear_packed_bytes(out_features, in_features), nc = code_bytes(MOE_ACT_E2M1_UE8M0_32, out_features, in_features),
                 ns = scale_bytes(MOE_ACT_E2M1_UE8M0_32, out_features, in_features);
    if (overlap(packed, n, codes, nc) || overlap(packed, n, scales, ns)) return MOE_ERR_INVALID_ARG;
    if ((long long)lin_tiles(out_features) * lin_units(in_features) > INT32_MAX) return MOE_ERR_UNSUPPORTED;
    LinGuard guard(h->device);
    return cuda_rc(launch_mx_pack(MxPackArgs{codes, scales, (uint8_t*)packed, out_features, in_features}, (cudaStream_t)stream));
}

int moe_linear(moe_lin_t h, const moe_linear_desc* w, int act_mode, const void* x, const uint8_t* x_scales, int T, void* y, int out_dtype,
               void* stream)
{
    if (!h || !w || !is_codes(act_mode) || !is_type(out_dtype) || w->out_features <= 0) return MOE_ERR_INVALID_ARG;
    const int N = w->out_features, K = w->in_features;
    int rc = check_rows(T, K);
    if (!rc) rc = check_rows(N, K);
    if (rc) return rc;
    if (!w->packed || !aligned(w->packed, 128) || !aligned(x, 16) || !aligned(x_scales, 16) || !aligned(y, 16)) return MOE_ERR_INVALID_ARG;
    if (!x_scales && (T > h->cfg.max_tokens || K > h->cfg.max_in)) return MOE_ERR_INVALID_ARG;
    if ((double)T * N > 1e13 || (long long)lin_tiles(N) * lin_units(K) > INT32_MAX) return MOE_ERR_UNSUPPORTED;
    if (T == 0) return MOE_OK;
    if (!x || !y) return MOE_ERR_INVALID_ARG;
    const size_t ny = (size_t)T * N * type_bytes(out_dtype);
    if (overlap(y, ny, x, x_scales ? code_bytes(act_mode, T, K) : (size_t)T * K * 2) ||
        overlap(y, ny, x_scales, scale_bytes(act_mode, T, K)) || overlap(y, ny, w->packed, moe_linear_packed_bytes(N, K)))
        return MOE_ERR_INVALID_ARG;
    LinearArgs a{};
    a.packed = (const uint8_t*)w->packed;
    a.codes = x_scales ? (const uint8_t*)x : h->codes;
    a.scales = x_scales ? x_scales : h->scales;
    a.T = T;
    a.N = N;
    a.K = K;
    a.e2m1 = act_mode == MOE_ACT_E2M1_UE8M0_32;
    a.y = y;
    a.out_f32 = out_dtype == MOE_OUT_F32;
    a.status = h->status;
    a.wait_ns = h->wait_ns;
    a.withhold = h->withhold;
    LinGuard guard(h->device);
    if (!x_scales) {
        if (linear_takes_bf16(a, h->dev)) {
            a.codes = a.scales = nullptr;
            a.x = (const uint16_t*)x;
        } else {
            const cudaError_t e = quantise(h->dev.sms, x, T, K, act_mode, h->codes, h->scales, (cudaStream_t)stream);
            if (e != cudaSuccess) return MOE_ERR_CUDA;
        }
    }
    return cuda_rc(launch_linear(a, h->dev, (cudaStream_t)stream));
}

int moe_lin_test_set_wait(moe_lin_t h, unsigned long long wait_ns, int withhold)
{
    if (!h || wait_ns > kLinWaitNs) return MOE_ERR_INVALID_ARG;
    h->wait_ns = wait_ns ? (uint32_t)wait_ns : kLinWaitNs;
    h->withhold = withhold != 0;
    return MOE_OK;
}

int moe_lin_test_plan(const moe_lin_test_device* dev, int act_mode, int bf16_rows, int T, int out_features, int in_features, int out_dtype,
                      moe_lin_test_plan_t* plan)
{
    if (!dev || !plan || dev->sms <= 0 || dev->pairs <= 0 || !is_codes(act_mode) || !is_type(out_dtype) || T <= 0 || out_features <= 0)
        return MOE_ERR_INVALID_ARG;
    int rc = check_rows(T, in_features);
    if (!rc) rc = check_rows(out_features, in_features);
    if (rc) return rc;
    LinDevice d{dev->sms, dev->pairs, {}};
    for (int i = 2; i <= kLinClusterMax; i++) d.clusters[i] = dev->clusters[i];
    LinearArgs a{};
    a.T = T;
    a.N = out_features;
    a.K = in_features;
    a.e2m1 = act_mode == MOE_ACT_E2M1_UE8M0_32;
    a.out_f32 = out_dtype == MOE_OUT_F32;
    // (never read: a plan only asks whether there are codes)
    const uint8_t codes = 0;
    if (!bf16_rows || !linear_takes_bf16(a, d)) a.codes = &codes;
    linear_plan(a, d, plan);
    return MOE_OK;
}

int moe_lin_call(int op, const int64_t* words)
{
    if (!words) return MOE_ERR_INVALID_ARG;
    Words a{words};
    if (op == MOE_LIN_CALL_RMS_NORM) {
        const auto h = a.p<moe_lin_t>();
        const auto d = a.p<const moe_norm_desc*>();
        const auto x = a.p<const void*>(), residual = a.p<const void*>();
        const int T = a.i();
        const auto residual_out = a.p<void*>(), out = a.p<void*>();
        const int mode = a.i();
        const auto codes = a.p<uint8_t*>(), scales = a.p<uint8_t*>();
        const auto stream = a.p<void*>();
        return a.ok ? moe_rms_norm(h, d, x, residual, T, residual_out, out, mode, codes, scales, stream) : MOE_ERR_INVALID_ARG;
    }
    if (op == MOE_LIN_CALL_QUANT) {
        const auto h = a.p<moe_lin_t>();
        const auto x = a.p<const void*>();
        const int rows = a.i(), n = a.i(), mode = a.i();
        const auto codes = a.p<uint8_t*>(), scales = a.p<uint8_t*>();
        const auto stream = a.p<void*>();
        return a.ok ? moe_mx_quant(h, x, rows, n, mode, codes, scales, stream) : MOE_ERR_INVALID_ARG;
    }
    if (op == MOE_LIN_CALL_VALUES) {
        const auto h = a.p<moe_lin_t>();
        const int mode = a.i();
        const auto codes = a.p<const uint8_t*>(), scales = a.p<const uint8_t*>();
        const int rows = a.i(), n = a.i(), type = a.i();
        const auto out = a.p<void*>(), stream = a.p<void*>();
        return a.ok ? moe_mx_values(h, mode, codes, scales, rows, n, type, out, stream) : MOE_ERR_INVALID_ARG;
    }
    if (op == MOE_LIN_CALL_LINEAR) {
        const auto h = a.p<moe_lin_t>();
        const auto w = a.p<const moe_linear_desc*>();
        const int mode = a.i();
        const auto x = a.p<const void*>();
        const auto scales = a.p<const uint8_t*>();
        const int T = a.i();
        const auto y = a.p<void*>();
        const int type = a.i();
        const auto stream = a.p<void*>();
        return a.ok ? moe_linear(h, w, mode, x, scales, T, y, type, stream) : MOE_ERR_INVALID_ARG;
    }
    return MOE_ERR_INVALID_ARG;
}

}  // extern "C"
