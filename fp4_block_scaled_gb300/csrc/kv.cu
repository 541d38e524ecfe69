// kv.cu -- the C ABI of the paged key-value cache: validation, the handle and
// its workspace, the rotary table, launches, status.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <new>

#include "kv.h"

using namespace moe;

struct moe_kv_s {
    moe_kv_config cfg;
    int device;
    int sms;
    int* status;
    uint8_t* attn_ws;           // the attention's workspace, in the same allocation
};

namespace {

struct KvGuard {
    int prev = -1;
    explicit KvGuard(int dev)
    {
        if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
        if (prev != dev) cudaSetDevice(dev);
    }
    ~KvGuard()
    {
        int cur;
        if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
    }
};

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

int cuda_rc(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

int check_kv_cfg(const moe_kv_config* c)
{
    if (!c) return MOE_ERR_INVALID_ARG;
    if (c->num_q_heads <= 0 || c->num_kv_heads <= 0 || c->num_q_heads % c->num_kv_heads || c->head_dim <= 0 ||
        c->page_size <= 0 || c->num_pages <= 0 || c->max_seqs <= 0 || c->max_pages_per_seq <= 0)
        return MOE_ERR_INVALID_ARG;
    if (c->kv_dtype != MOE_KV_BF16 && c->kv_dtype != MOE_KV_E4M3_UE8M0) return MOE_ERR_INVALID_ARG;
    if (c->out_dtype != MOE_OUT_BF16 && c->out_dtype != MOE_OUT_F32) return MOE_ERR_INVALID_ARG;
    if (c->num_q_heads > 512 || c->head_dim > 128 || c->head_dim % (c->kv_dtype == MOE_KV_BF16 ? 16 : 32) ||
        c->page_size % 16 || c->page_size > 1024 || c->max_seqs > kAttnMaxSeqs)
        return MOE_ERR_UNSUPPORTED;
    const long long cap = (long long)c->max_pages_per_seq * c->page_size;      // tokens of a sequence: int32 positions
    if (cap > INT32_MAX - 4096) return MOE_ERR_UNSUPPORTED;
    // the attention counts a batch's tiles of 16 keys, in all rows, in 32 bits (with some for each row)
    if ((double)((cap + 15) / 16) * c->max_seqs * c->num_q_heads > 4280000000.0) return MOE_ERR_UNSUPPORTED;
    // and pool places in blocks of 16 rows
    if ((double)c->num_pages * c->num_kv_heads * (c->page_size / 16) > 4294967294.0) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

size_t page_kv_bytes(const moe_kv_config& c)
{
    return (size_t)c.num_kv_heads * c.page_size * c.head_dim * (c.kv_dtype == MOE_KV_BF16 ? 2 : 1);
}

size_t page_scale_bytes(const moe_kv_config& c)
{
    return c.kv_dtype == MOE_KV_BF16 ? 0 : (size_t)c.num_kv_heads * c.page_size;
}

int check_pool(const moe_kv_s* h, const moe_kv_pool* p)
{
    if (!p || !p->k || !p->v || !aligned(p->k, 16) || !aligned(p->v, 16)) return MOE_ERR_INVALID_ARG;
    const bool scaled = h->cfg.kv_dtype != MOE_KV_BF16;
    if (scaled != (p->k_scales != nullptr) || scaled != (p->v_scales != nullptr)) return MOE_ERR_INVALID_ARG;
    if (!aligned(p->k_scales, 16) || !aligned(p->v_scales, 16)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

KvPool pool_of(const moe_kv_pool& p) { return KvPool{(uint8_t*)p.k, (uint8_t*)p.v, p.k_scales, p.v_scales}; }

int check_rope(const moe_kv_s* h, const moe_rope_desc* r)
{
    if (!r->freqs || !aligned(r->freqs, 8) || r->rot_dim < 16 || r->rot_dim % 16 || r->rot_dim > h->cfg.head_dim)
        return MOE_ERR_INVALID_ARG;
    if (r->layout != MOE_ROPE_HALF && r->layout != MOE_ROPE_INTERLEAVED) return MOE_ERR_INVALID_ARG;
    return isfinite(r->scale) ? MOE_OK : MOE_ERR_INVALID_ARG;
}

// The token stride of a bf16 tensor of `heads` heads of D, 0 standing for a
// contiguous one; -1 if it is none.
long long token_stride(long long ld, int heads, int D)
{
    const long long need = (long long)heads * D;
    if (ld == 0) return need;
    return ld >= need && ld % 8 == 0 && ld <= (1LL << 32) ? ld : -1;
}

struct Span {
    const char* lo;
    const char* hi;
    Span(const void* p, long long ld, int heads, int D, int T)
        : lo((const char*)p), hi(p ? lo + ((size_t)(T - 1) * ld + (size_t)heads * D) * 2 : lo)
    {
    }
    Span(const void* p, size_t bytes) : lo((const char*)p), hi(p ? lo + bytes : lo) {}
    bool overlaps(const Span& o) const { return lo < o.hi && o.lo < hi; }
};

// Whether a token of x (`heads` heads of D, every ld elements) may share an
// element with one of y.  Parts of one projection's rows interleave: with one
// stride they are apart if they are so within a row.
bool clash(const Span& x, int hx, long long ldx, const Span& y, int hy, long long ldy, int D)
{
    if (!x.overlaps(y)) return false;
    if (ldx != ldy) return true;
    const long long off = ((y.lo - x.lo) / 2 % ldx + ldx) % ldx;       // where y's part of a row begins, from x's
    return off < (long long)hx * D || off + (long long)hy * D > ldx;
}

constexpr int kMaxTokens = 1 << 24;     // of one moe_rope or moe_kv_append call

// Numbers of about 104 bits, the sum of two doubles, for the rotary table, whose
// entries are 64-bit fractions: errors below 2^-84 of an entry, exp's doublings
// included.
struct Wide {
    double hi, lo = 0.0;
};

Wide fast_sum(double a, double b)       // |a| >= |b|, or a = 0
{
    const double s = a + b;
    return {s, b - (s - a)};
}

Wide operator+(Wide x, Wide y)
{
    const double s = x.hi + y.hi, b = s - x.hi, e = (x.hi - (s - b)) + (y.hi - b);
    return fast_sum(s, e + (x.lo + y.lo));
}

Wide operator-(Wide x) { return {-x.hi, -x.lo}; }

Wide operator*(Wide x, Wide y)
{
    const double p = x.hi * y.hi;
    return fast_sum(p, fma(x.hi, y.lo, fma(x.lo, y.hi, fma(x.hi, y.hi, -p))));
}

Wide operator/(Wide x, double d)
{
    const double q = x.hi / d;
    return fast_sum(q, (fma(-q, d, x.hi) + x.lo) / d);
}

Wide operator/(Wide x, Wide y)
{
    const double q = x.hi / y.hi;
    const Wide rest = x + -(y * Wide{q});
    return fast_sum(q, rest.hi / y.hi);
}

// e^x for |x| < 2^11: the series at x / 2^n below 2^-7, squared n times
Wide wide_exp(Wide x)
{
    int n = 0;
    frexp(x.hi, &n);
    n = x.hi == 0.0 || n < -7 ? 0 : n + 7;
    const Wide r = {ldexp(x.hi, -n), ldexp(x.lo, -n)};
    Wide s = {1.0};
    for (int i = 13; i > 0; i--) s = Wide{1.0} + r * s / (double)i;
    for (; n > 0; n--) s = s * s;
    return s;
}

// ln of m in [1/2, 2]: the logarithm of doubles and one step of Newton's
Wide wide_log_near_one(double m)
{
    const Wide y = {log(m)};
    return y + (Wide{m} * wide_exp(-y) + Wide{-1.0});
}

Wide wide_log(double x)                 // x >= 1
{
    int e;
    const double m = frexp(x, &e);
    return wide_log_near_one(m) + wide_log_near_one(2.0) * Wide{(double)e};
}

}  // namespace

extern "C" {

int moe_kv_pool_bytes(const moe_kv_config* cfg, size_t* kv_bytes, size_t* scale_bytes)
{
    if (!kv_bytes || !scale_bytes) return MOE_ERR_INVALID_ARG;
    *kv_bytes = *scale_bytes = 0;
    const int rc = check_kv_cfg(cfg);
    if (rc) return rc;
    *kv_bytes = (size_t)cfg->num_pages * page_kv_bytes(*cfg);
    *scale_bytes = (size_t)cfg->num_pages * page_scale_bytes(*cfg);
    return MOE_OK;
}

int moe_kv_create(moe_kv_t* out, const moe_kv_config* cfg, int device)
{
    if (!out) return MOE_ERR_INVALID_ARG;
    *out = nullptr;
    const int rc = check_kv_cfg(cfg);
    if (rc) return rc;
    int ndev = 0;
    if (cudaGetDeviceCount(&ndev) != cudaSuccess || device < 0 || device >= ndev)
        return ndev ? MOE_ERR_INVALID_ARG : MOE_ERR_CUDA;
    KvGuard guard(device);
    moe_kv_s* h = new (std::nothrow) moe_kv_s();
    if (!h) return MOE_ERR_OOM;
    h->cfg = *cfg;
    h->device = device;
    void* ws = nullptr;
    if (cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess ||
        attn_init_device(cfg->num_q_heads, cfg->num_kv_heads, cfg->head_dim, cfg->kv_dtype != MOE_KV_BF16,
                         cfg->out_dtype == MOE_OUT_F32) != cudaSuccess ||
        rope_init_device() != cudaSuccess || copy_init_device() != cudaSuccess) {
        delete h;
        return MOE_ERR_CUDA;
    }
    const AttnWorkspace w = attn_workspace(cfg->max_seqs, cfg->num_q_heads, cfg->num_kv_heads, cfg->head_dim, h->sms);
    if (lib_malloc(&ws, 256 + w.bytes) != cudaSuccess) {
        cudaGetLastError();
        delete h;
        return MOE_ERR_OOM;
    }
    // the status word and the attention's tickets are zero before any stream can use them
    if (lib_zero(ws, 256 + w.frags) != cudaSuccess) {
        cudaFree(ws);
        delete h;
        return MOE_ERR_CUDA;
    }
    h->status = (int*)ws;
    h->attn_ws = (uint8_t*)ws + 256;
    *out = h;
    return MOE_OK;
}

int moe_kv_status(moe_kv_t h, void* stream)
{
    if (!h) return MOE_ERR_INVALID_ARG;
    KvGuard guard(h->device);
    int v = 0;
    if (lib_take_status(h->status, (cudaStream_t)stream, &v) != cudaSuccess) return MOE_ERR_CUDA;
    return v & kStatusBadIndex ? MOE_ERR_BAD_INDEX : MOE_OK;
}

void moe_kv_destroy(moe_kv_t h)
{
    if (!h) return;
    KvGuard guard(h->device);
    cudaFree(h->status);
    delete h;
}

int moe_rope_table(int rot_dim, double base, int kind, double factor, int trained_len, uint64_t* turns, float* scale)
{
    if (!turns || !scale || rot_dim < 2 || rot_dim % 2 || rot_dim > 1024) return MOE_ERR_INVALID_ARG;
    if (!(base > 1.0) || !isfinite(base)) return MOE_ERR_INVALID_ARG;
    if (kind < MOE_ROPE_SCALE_NONE || kind > MOE_ROPE_SCALE_YARN) return MOE_ERR_INVALID_ARG;
    if (kind != MOE_ROPE_SCALE_NONE && (!(factor >= 1.0) || !isfinite(factor))) return MOE_ERR_INVALID_ARG;
    if (kind == MOE_ROPE_SCALE_NTK && rot_dim < 4) return MOE_ERR_INVALID_ARG;
    if (kind == MOE_ROPE_SCALE_YARN && trained_len <= 0) return MOE_ERR_INVALID_ARG;
    const Wide two_pi = {6.283185307179586, 2.4492935982947064e-16};
    const double r = rot_dim;
    Wide ln_base = wide_log(base);
    if (kind == MOE_ROPE_SCALE_NTK) ln_base = ln_base + wide_log(factor) * Wide{r} / (r - 2.0);
    double lo = 0.0, hi = 0.0;
    if (kind == MOE_ROPE_SCALE_YARN) {
        auto pair_of = [&](double t) { return r * log(trained_len / (t * two_pi.hi)) / (2.0 * log(base)); };
        lo = fmax(floor(pair_of(32.0)), 0.0);
        hi = fmin(ceil(pair_of(1.0)), r - 1.0);
    }
    for (int i = 0; i < rot_dim / 2; i++) {
        Wide f = wide_exp(ln_base * Wide{-2.0 * i} / r);
        if (kind == MOE_ROPE_SCALE_LINEAR) f = f / factor;
        if (kind == MOE_ROPE_SCALE_YARN) {
            const Wide ramp = i <= lo ? Wide{0.0} : i >= hi ? Wide{1.0} : Wide{i - lo} / (hi - lo);
            f = f * (ramp / factor + (Wide{1.0} + -ramp));
        }
        f = f / two_pi;
        // f 2^64, below 2^62, to the nearest whole number
        const double whole = floor(ldexp(f.hi, 64)), rest = ldexp(f.hi, 64) - whole + ldexp(f.lo, 64);
        turns[i] = (uint64_t)((int64_t)whole + (int64_t)floor(rest + 0.5));
    }
    *scale = kind == MOE_ROPE_SCALE_YARN ? (float)(0.1 * log(factor) + 1.0) : 1.0f;
    return MOE_OK;
}

int moe_rope(moe_kv_t h, const moe_rope_desc* rope, const int32_t* pos, int T, const void* q, long long ldq,
             void* q_out, const void* k, long long ldk, void* k_out, void* stream)
{
    if (!h || !rope || T < 0 || (q == nullptr) != (q_out == nullptr) || (k == nullptr) != (k_out == nullptr))
        return MOE_ERR_INVALID_ARG;
    const moe_kv_config& c = h->cfg;
    int rc = check_rope(h, rope);
    if (rc) return rc;
    const long long lq = token_stride(ldq, c.num_q_heads, c.head_dim), lk = token_stride(ldk, c.num_kv_heads, c.head_dim);
    if (lq < 0 || lk < 0) return MOE_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(q_out, 16) || !aligned(k, 16) || !aligned(k_out, 16) || !aligned(pos, 4))
        return MOE_ERR_INVALID_ARG;
    if (T > kMaxTokens) return MOE_ERR_UNSUPPORTED;
    if (T == 0 || (!q && !k)) return MOE_OK;
    if (!pos) return MOE_ERR_INVALID_ARG;
    RopeArgs a{};
    a.freqs = rope->freqs;
    a.rot = rope->rot_dim;
    a.layout = rope->layout;
    a.scale = rope->scale;
    a.pos = pos;
    a.T = T;
    a.D = c.head_dim;
    a.hq = q ? c.num_q_heads : 0;
    a.hk = k ? c.num_kv_heads : 0;
    a.q = (const uint16_t*)q;
    a.k = (const uint16_t*)k;
    a.q_out = (uint16_t*)q_out;
    a.k_out = (uint16_t*)k_out;
    a.ldq = lq;
    a.ldk = lk;
    a.ldq_out = q == q_out ? lq : (long long)c.num_q_heads * c.head_dim;
    a.ldk_out = k == k_out ? lk : (long long)c.num_kv_heads * c.head_dim;
    a.sms = h->sms;
    // an output overlaps no input but the one it is
    const Span sq(q, lq, a.hq, a.D, T), sk(k, lk, a.hk, a.D, T);
    const Span oq(q_out, a.ldq_out, a.hq, a.D, T), ok(k_out, a.ldk_out, a.hk, a.D, T);
    if (q != q_out && (oq.overlaps(sq) || oq.overlaps(sk))) return MOE_ERR_INVALID_ARG;
    if (k != k_out && (ok.overlaps(sk) || ok.overlaps(sq))) return MOE_ERR_INVALID_ARG;
    if (q && k && (q != q_out || k != k_out) && oq.overlaps(ok)) return MOE_ERR_INVALID_ARG;
    if ((q == q_out || k == k_out) && clash(sq, a.hq, lq, sk, a.hk, lk, a.D)) return MOE_ERR_INVALID_ARG;
    KvGuard guard(h->device);
    return cuda_rc(launch_rope(a, (cudaStream_t)stream));
}

int moe_kv_append(moe_kv_t h, const moe_kv_pool* pool, const void* k, long long ldk, const void* v, long long ldv,
                  const int32_t* pos, const int32_t* seq, const int32_t* page_table, int T,
                  const moe_rope_desc* rope, const void* q, long long ldq, void* q_out, void* stream)
{
    if (!h || T < 0 || (q == nullptr) != (q_out == nullptr) || (q && !rope)) return MOE_ERR_INVALID_ARG;
    const moe_kv_config& c = h->cfg;
    int rc = check_pool(h, pool);
    if (!rc && rope) rc = check_rope(h, rope);
    if (rc) return rc;
    const long long lq = token_stride(ldq, c.num_q_heads, c.head_dim), lk = token_stride(ldk, c.num_kv_heads, c.head_dim),
                    lv = token_stride(ldv, c.num_kv_heads, c.head_dim);
    if (lq < 0 || lk < 0 || lv < 0) return MOE_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(q_out, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(pos, 4) ||
        !aligned(seq, 4) || !aligned(page_table, 4))
        return MOE_ERR_INVALID_ARG;
    if (!seq && T > c.max_seqs) return MOE_ERR_INVALID_ARG;
    if (T > kMaxTokens) return MOE_ERR_UNSUPPORTED;
    if (T == 0) return MOE_OK;
    if (!k || !v || !pos || !page_table) return MOE_ERR_INVALID_ARG;
    RopeArgs a{};
    if (rope) {
        a.freqs = rope->freqs;
        a.rot = rope->rot_dim;
        a.layout = rope->layout;
        a.scale = rope->scale;
    }
    a.pos = pos;
    a.T = T;
    a.D = c.head_dim;
    a.hq = q ? c.num_q_heads : 0;
    a.hk = a.hv = c.num_kv_heads;
    a.q = (const uint16_t*)q;
    a.k = (const uint16_t*)k;
    a.v = (const uint16_t*)v;
    a.q_out = (uint16_t*)q_out;
    a.ldq = lq;
    a.ldk = lk;
    a.ldv = lv;
    a.ldq_out = q == q_out ? lq : (long long)c.num_q_heads * c.head_dim;
    a.append = 1;
    a.e4m3 = c.kv_dtype != MOE_KV_BF16;
    a.pool = pool_of(*pool);
    a.seq = seq;
    a.table = page_table;
    a.num_pages = c.num_pages;
    a.page_size = c.page_size;
    a.row = c.max_pages_per_seq;
    a.max_seqs = c.max_seqs;
    a.status = h->status;
    a.sms = h->sms;
    const Span sq(q, lq, a.hq, a.D, T), sk(k, lk, a.hk, a.D, T), sv(v, lv, a.hv, a.D, T), oq(q_out, a.ldq_out, a.hq, a.D, T);
    if (q && q != q_out && (oq.overlaps(sq) || oq.overlaps(sk) || oq.overlaps(sv))) return MOE_ERR_INVALID_ARG;
    if (q && q == q_out && (clash(sq, a.hq, lq, sk, a.hk, lk, a.D) || clash(sq, a.hq, lq, sv, a.hv, lv, a.D)))
        return MOE_ERR_INVALID_ARG;
    KvGuard guard(h->device);
    return cuda_rc(launch_rope(a, (cudaStream_t)stream));
}

int moe_attn_decode(moe_kv_t h, const moe_kv_pool* pool, const void* q, const int32_t* seq_lens,
                    const int32_t* page_table, int B, float scale, float softcap, int window, void* out, float* lse,
                    void* stream)
{
    if (!h || B < 0 || B > h->cfg.max_seqs || window < 0 || !(fabsf(scale) <= 0x1p32f) ||
        (softcap != 0.0f && !(softcap >= 0x1p-32f && softcap <= 0x1p32f)))
        return MOE_ERR_INVALID_ARG;
    const int rc = check_pool(h, pool);
    if (rc) return rc;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(seq_lens, 4) || !aligned(page_table, 4) || !aligned(lse, 4))
        return MOE_ERR_INVALID_ARG;
    if (B == 0) return MOE_OK;
    if (!q || !seq_lens || !page_table || !out) return MOE_ERR_INVALID_ARG;
    const moe_kv_config& c = h->cfg;
    const size_t heads = (size_t)B * c.num_q_heads, n = heads * c.head_dim;
    const Span sq(q, n * 2), so(out, n * (c.out_dtype == MOE_OUT_F32 ? 4 : 2)), sl(lse, heads * 4);
    if (so.overlaps(sq) || sl.overlaps(sq) || sl.overlaps(so)) return MOE_ERR_INVALID_ARG;
    AttnArgs a{};
    a.pool = pool_of(*pool);
    a.q = (const uint16_t*)q;
    a.lens = seq_lens;
    a.table = page_table;
    a.B = B;
    a.hq = c.num_q_heads;
    a.hkv = c.num_kv_heads;
    a.D = c.head_dim;
    a.num_pages = c.num_pages;
    a.page_size = c.page_size;
    a.row = c.max_pages_per_seq;
    a.e4m3 = c.kv_dtype != MOE_KV_BF16;
    a.out_f32 = c.out_dtype == MOE_OUT_F32;
    a.scale = scale != 0.0f ? scale : 1.0f / sqrtf((float)c.head_dim);
    a.softcap = softcap;
    a.window = window;
    a.out = out;
    a.lse = lse;
    a.status = h->status;
    a.sms = h->sms;
    a.max_seqs = c.max_seqs;
    a.ws = h->attn_ws;
    KvGuard guard(h->device);
    return cuda_rc(launch_attn(a, (cudaStream_t)stream));
}

int moe_kv_copy_pages(moe_kv_t h, const moe_kv_pool* pools, int num_pools, const int32_t* pairs, int n, void* stream)
{
    if (!h || num_pools < 0 || n < 0 || n > h->cfg.num_pages || !aligned(pairs, 4)) return MOE_ERR_INVALID_ARG;
    if (num_pools > 0 && !pools) return MOE_ERR_INVALID_ARG;
    for (int l = 0; l < num_pools; l++) {
        const int rc = check_pool(h, pools + l);
        if (rc) return rc;
    }
    if (num_pools == 0 || n == 0) return MOE_OK;
    if (!pairs) return MOE_ERR_INVALID_ARG;
    CopyArgs a{};
    a.pairs = pairs;
    a.n = n;
    a.num_pages = h->cfg.num_pages;
    a.kv_bytes = page_kv_bytes(h->cfg);
    a.scale_bytes = page_scale_bytes(h->cfg);
    a.status = h->status;
    KvGuard guard(h->device);
    cudaError_t e = cudaSuccess;
    for (int l0 = 0; l0 < num_pools && e == cudaSuccess; l0 += kCopyLayers) {
        a.layers = std::min(kCopyLayers, num_pools - l0);
        for (int l = 0; l < a.layers; l++) a.pool[l] = pool_of(pools[l0 + l]);
        e = launch_copy_pages(a, (cudaStream_t)stream);
    }
    return cuda_rc(e);
}

namespace {

// The words of a moe_kv_call, in order.
struct Words {
    const int64_t* w;
    bool ok = true;
    void* p() { return (void*)(uintptr_t)*w++; }
    long long ll() { return *w++; }
    int i()
    {
        ok = ok && *w >= INT32_MIN && *w <= INT32_MAX;
        return (int)*w++;
    }
    float f()
    {
        double d;
        memcpy(&d, w++, 8);
        ok = ok && (d == 0.0 || (float)d != 0.0f);      // 0 stands for a default
        return (float)d;
    }
};

}  // namespace

int moe_kv_call(int op, const int64_t* words)
{
    if (!words) return MOE_ERR_INVALID_ARG;
    Words a{words};
    if (op == MOE_KV_CALL_ROPE) {
        auto h = (moe_kv_t)a.p();
        auto rope = (const moe_rope_desc*)a.p();
        auto pos = (const int32_t*)a.p();
        const int T = a.i();
        const void* q = a.p();
        const long long ldq = a.ll();
        void* q_out = a.p();
        const void* k = a.p();
        const long long ldk = a.ll();
        void* k_out = a.p();
        void* stream = a.p();
        return a.ok ? moe_rope(h, rope, pos, T, q, ldq, q_out, k, ldk, k_out, stream) : MOE_ERR_INVALID_ARG;
    }
    if (op == MOE_KV_CALL_APPEND) {
        auto h = (moe_kv_t)a.p();
        auto pool = (const moe_kv_pool*)a.p();
        const void* k = a.p();
        const long long ldk = a.ll();
        const void* v = a.p();
        const long long ldv = a.ll();
        auto pos = (const int32_t*)a.p();
        auto seq = (const int32_t*)a.p();
        auto table = (const int32_t*)a.p();
        const int T = a.i();
        auto rope = (const moe_rope_desc*)a.p();
        const void* q = a.p();
        const long long ldq = a.ll();
        void* q_out = a.p();
        void* stream = a.p();
        return a.ok ? moe_kv_append(h, pool, k, ldk, v, ldv, pos, seq, table, T, rope, q, ldq, q_out, stream) : MOE_ERR_INVALID_ARG;
    }
    if (op == MOE_KV_CALL_ATTN_DECODE) {
        auto h = (moe_kv_t)a.p();
        auto pool = (const moe_kv_pool*)a.p();
        const void* q = a.p();
        auto lens = (const int32_t*)a.p();
        auto table = (const int32_t*)a.p();
        const int B = a.i();
        const float scale = a.f(), softcap = a.f();
        const int window = a.i();
        void* out = a.p();
        auto lse = (float*)a.p();
        void* stream = a.p();
        return a.ok ? moe_attn_decode(h, pool, q, lens, table, B, scale, softcap, window, out, lse, stream) : MOE_ERR_INVALID_ARG;
    }
    if (op == MOE_KV_CALL_COPY_PAGES) {
        auto h = (moe_kv_t)a.p();
        auto pools = (const moe_kv_pool*)a.p();
        const int num = a.i();
        auto pairs = (const int32_t*)a.p();
        const int n = a.i();
        void* stream = a.p();
        return a.ok ? moe_kv_copy_pages(h, pools, num, pairs, n, stream) : MOE_ERR_INVALID_ARG;
    }
    return MOE_ERR_INVALID_ARG;
}

}  // extern "C"
