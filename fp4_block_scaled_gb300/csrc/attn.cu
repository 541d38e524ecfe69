// attn.cu -- attention of one new token per sequence over the paged cache, in
// one launch.
//
// The work is cut into tiles of TT keys of one row, a row being a (sequence,
// key head, group of up to NROW query heads); the rows' tiles in order are one
// line, and every warp of the grid takes an equal stretch of it, so the split
// along the cache follows the lengths by itself: a long sequence spreads over
// many warps, short ones share one (where warps would idle, short rows are kept in
// one CTA instead).  A warp keeps the running maximum and sum
// of the softmax and its output rows in registers while it stays in a row
// (softmax(s)_j v_j summed with weights 2^(s_j - m), rescaled when m moves), and
// writes the rows that lie inside its stretch itself.  What is left of a row
// at the two ends of a stretch is merged in the CTA, and across CTAs by the
// last of them to finish the row (a ticket per row; it adds the parts in CTA
// order, so the sums do not depend on which CTA is last, and no CTA waits).
//
// Bound: HBM -- the keys and values are read once, 4 to 16 flops a byte.  So a
// warp streams its tiles through a ring of its own in shared memory (cp.async,
// 16 bytes a lane, two of three 8 KB tiles in flight: 128 KB an SM), with no
// barrier between warps, and fetches ahead what a tile's address needs (the
// page ids of the next 32 tiles; prefetching the next row's queries too gains
// nothing, and its instructions cost one sequence 0.1 us).  The products are
// mma.sync m16n8k16, which are busy 14 to 31 % of the time: a tile of one
// token's 8 query heads fills half of an MMA's 16 rows (the other half carries
// the weights' low terms), and a tcgen05 MMA would want 128 keys in one place and
// a round trip through tensor memory per tile for the same bytes.
//
// Measured (GPU time, back to back; 6783 GB/s is the rate of a plain copy):
//   64 sequences of up to 8000 keys, 8 x 128, bf16:   164 us, 6.43 TB/s
//   2 of up to 131071:                                138 us, 6.45 TB/s
//   128 of up to 8000, E4M3, 8 query heads a key head: 175 us, 5.94 TB/s
//   48 windows of 1000 keys, 16 x 64, capped scores:   37 us, 4.65 TB/s
//   one sequence of 1000 keys:                        7.9 us (of 16: 4.2, 100: 5.4; a launch
//     takes 2.1; then lengths, page ids, keys, the ticket and the join: five round trips)
// While the rings are full the SMs take in 25 bytes a cycle each, the memory's
// rate; what is lost is 3.4 us before them, the tenth by which SMs with a
// slower way to memory end later than others (dealing out the last eighth of
// the line at run time evened that out, but the many parts it left cost the
// join as much), and 2 to 4 us of merging.
#include <type_traits>

#include "common.cuh"
#include "kv.h"

namespace moe {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

// The softmax's reference is moved when a score passes it by more than this
// (in powers of two): weights stay below 2^8, and most tiles rescale nothing.
constexpr float kSlack = 8.0f;

// Keys of a tile: 8 KB of k and v rows; with tiles of half the keys E4M3 rows of 64
// take 37.9 us instead of 34.9 (32 sequences of up to 8000).
__host__ __device__ constexpr int tile_keys(int DP, bool F8) { return F8 && DP <= 64 ? 64 : F8 || DP <= 64 ? 32 : 16; }
__host__ __device__ constexpr int row_bytes(int DP, bool F8) { return DP * (F8 ? 1 : 2); }
// a tile in the ring: k rows, v rows, then (E4M3) their scale bytes
__host__ __device__ constexpr int stage_bytes(int DP, bool F8)
{
    return 2 * tile_keys(DP, F8) * row_bytes(DP, F8) + (F8 ? 2 * tile_keys(DP, F8) : 0);
}
constexpr int kStages = 3;      // tiles of a warp's ring

// A part of a row: NROW output rows (not divided by the sums), the powers of
// two that the sums of weights are multiples of, the sums, and (E4M3) the whole
// powers of two by which the output's lie above theirs.  The
// rows are spaced so that a warp's stores of an MMA result (8 rows, 2 or 4
// columns a lane) meet no bank twice.
__host__ __device__ constexpr int part_row(int DP, bool F8) { return DP + (F8 ? 16 : 8); }
__host__ __device__ constexpr int part_floats(int DP, bool F8, int NROW) { return NROW * part_row(DP, F8) + (F8 ? 3 : 2) * NROW; }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// bf16 rows as they are; E4M3 rows as f16
template <bool F8>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    if (F8) mma_f16(d, a0, a1, a2, a3, b0, b1);
    else mma_bf16(d, a0, a1, a2, a3, b0, b1);
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}

// p as bf16 terms: hi = bf16(p), lo = bf16(p - hi), together 16 significant
// bits (bf16 alone would put an error of up to 2^-8 on every weight), enough for a
// bf16 output; the rest, bf16(p - hi - lo), brings 24 for an fp32 one, whose error
// two terms would leave at 1.3e-6 of the output's norm.
__device__ __forceinline__ void split_pair(float p0, float p1, uint32_t& hi, uint32_t& lo, uint32_t& rest)
{
    hi = pack_bf16(p0, p1);
    const float r0 = p0 - __uint_as_float(hi << 16), r1 = p1 - __uint_as_float(hi & 0xFFFF0000u);
    lo = pack_bf16(r0, r1);
    rest = pack_bf16(r0 - __uint_as_float(lo << 16), r1 - __uint_as_float(lo & 0xFFFF0000u));
}

template <bool F8>
__device__ __forceinline__ void split(float w0, float w1, uint32_t& hi, uint32_t& lo, uint32_t& rest);

// Four E4M3 codes as two pairs of f16 (exact: 4 significant bits, exponents
// -9 .. 8), bytes (0, 1) and (2, 3).
__device__ __forceinline__ void e4m3_to_f16(uint32_t r, uint32_t& lo, uint32_t& hi)
{
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(r));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// w as two f16 terms of 11 bits: its upper bits, which f16 holds exactly above
// 2^-14, and the rest; below, f16's steps of 2^-24 remain, 2^-39 of the largest
// weight that can occur.
__device__ __forceinline__ void split_pair_f16(float w0, float w1, uint32_t& hi, uint32_t& lo)
{
    const float t0 = __uint_as_float(__float_as_uint(w0) & 0xFFFFE000u), t1 = __uint_as_float(__float_as_uint(w1) & 0xFFFFE000u);
    hi = pack_f16(t0, t1);
    lo = pack_f16(w0 - t0, w1 - t1);
}

template <>
__device__ __forceinline__ void split<false>(float w0, float w1, uint32_t& hi, uint32_t& lo, uint32_t& rest)
{
    split_pair(w0, w1, hi, lo, rest);
}

template <>
__device__ __forceinline__ void split<true>(float w0, float w1, uint32_t& hi, uint32_t& lo, uint32_t&)
{
    split_pair_f16(w0, w1, hi, lo);
}

// Chunk c of row r of a tile, swizzled so that eight rows' chunks of one
// column lie in different banks.
template <int ROWB>
__device__ __forceinline__ uint32_t at_chunk(uint32_t base, int r, int c)
{
    const int x = ROWB >= 128 ? (r & 7) : ((r >> 1) & 3);
    return base + (uint32_t)(r * ROWB + ((c ^ x) << 4));
}

// Rows of up to kWhole keys stay with one warp where every warp has a tile and
// the rows are short on the average (at most kShort tiles): a part costs more
// than the few tiles it moves.  256 sequences of up to 30 and 100 keys: 13.4 and
// 21.3 us when split, 10.4 and 19.2 when not; E4M3 of 100: 19.3 and 17.4.  Where
// warps would idle splitting wins: one E4M3 sequence of 100 keys 6.7 us, 9.7 whole.
constexpr int kWhole = 128;
constexpr int kShort = 16;

// A join across CTAs takes 2.3 us, so where CTAs would idle, rows of up to this many
// tiles have one to themselves: 32 (E4M3, whose tiles take twice the instructions:
// 16), and twice that where more than half the CTAs have a row anyway (8 key heads
// of 128, bf16, sequences x keys, without and with it: 1 x 100 7.8 and 5.3 us,
// 1 x 512 7.8 and 7.7, 8 x 500 9.1 and 8.0, 16 x 600 14.4 and 11.5, 18 x 1000 20.5 and
// 17.2; beyond it, 1 x 600 would take 8.4 for 7.7 and one E4M3 sequence of 1000 11.9
// for 9.4; ragged batches gain less, 16 of up to 1000 11.7 and 11.1, or lose, 10 of
// up to 1000 10.1 and 10.8).  More rows than CTAs: see snap (20 x 100 8.7 and 7.9, 40 x 48
// 8.9 and 7.3, 30 x 30, which had no join, 6.0 and 6.2).  The choice costs a line that
// is full 0.2 us (1 x 3000: 9.0 and 9.2).
__device__ __forceinline__ uint32_t one_cta_tiles(bool f8, uint32_t rows) { return (f8 ? 16u : 32u) << (2 * rows > gridDim.x ? 1 : 0); }

// What a row itself (queries, output, places) costs a warp, in tiles, when the
// line is shared out: without it the warps with many short rows end last (128
// E4M3 sequences of up to 8000 keys, some of one key: 188 us, 177 with it; 256 of
// up to 1000: 75.7 and 55.7; 48 windows of 1000 keys: 43.8 and 36.8).
constexpr uint32_t kRowCost = 2;

struct SplitArgs {
    AttnArgs a;
    int G, chunks, R;           // query heads per key head, groups of NROW of them, rows per sequence
    int ps_shift;               // log2 of the page size, -1 if it is no power of two
    int pair_shift;             // 2^it pairs of heads hold a row's
    float* frags;               // [grid][kWarps] parts
    float* parts;               // [grid][2] parts
    int* tickets;               // [max_seqs * R], zero between launches
};

// DP: the elements of a row's place in the ring, CW <= DP those that are computed
// with.  FINE: for fp32 outputs, a third term of the weights over bf16 rows, and a
// tile's sums rounded into the row's.
template <int DP, int CW, bool F8, int NROW, bool FINE>
struct Kernel {
    static constexpr int TT = tile_keys(DP, F8), ROWB = row_bytes(DP, F8), NT = TT / 8, KS = CW / 16, ND = CW / 8;
    static constexpr int C2 = row_bytes(CW, F8) / 32;        // pairs of chunks computed with
    static constexpr int CPR = ROWB / 16, RPI = 32 / CPR, STAGE = stage_bytes(DP, F8), STAGES = kStages;
    static constexpr int PART = part_floats(DP, F8, NROW), PROW = part_row(DP, F8), PHEAD = NROW * PROW;
    static constexpr int SCALES = F8 ? 8 * TT : 0;           // a tile's scales as numbers
    static constexpr int REGION = STAGES * STAGE + SCALES;   // a warp's ring, and at the end its parts
    static_assert(REGION % 16 == 0 && PART % 4 == 0 && 4 * (2 * PART + 4 * 2 * kWarps * NROW) <= REGION,
                  "a warp's parts, and the merge's tables, fit its ring");
    static_assert(STAGES * (TT / 16) <= 32, "the ring's tiles have a bit per 16 keys in one word");
    static constexpr int QR = NROW == 8 ? 2 : 4;

    // ---- a row's state in one warp: lane 4 g + j holds row g (and g + 8 for
    // NROW 16), columns 2j, 2j + 1 of every 8
    // o 2^m is the row's sum of weights times values, l 2^m its sum of weights.
    // E4M3: the values' scales 2^(s - 127) enter o's weights as exponents, so o's
    // reference is m + whole(up): apart from m by a whole number, so that a score
    // less m is rounded once, for o and l alike.  (With a reference of its own,
    // rounded like the scores, one key's output came out off by 2.6e-6 of itself
    // at scores of tens and by 1e-5 at hundreds; now it is the value.)
    float o[ND][4];
    float m[2], l[2], up[2];
    uint32_t q[KS][QR];
    float qf[2];                // score factor of a row: E4M3 queries are scaled

    __device__ __forceinline__ void reset()
    {
#pragma unroll
        for (int i = 0; i < ND; i++)
#pragma unroll
            for (int k = 0; k < 4; k++) o[i][k] = 0.0f;
        m[0] = m[1] = up[0] = up[1] = -INFINITY;
        l[0] = l[1] = 0.0f;
    }

    // (scores pass the references by at most kSlack; o's lies 2^7 lower, so that
    // its weights, up to 2^15, use f16's range)
    static constexpr float kLift = 7.0f;

    // up as o's reference has it; -inf before the first key
    __device__ __forceinline__ static float whole(float up) { return up == -INFINITY ? 0.0f : floorf(up); }

    // Query rows as the A operand.  E4M3: the contraction index runs as
    // e4m3_to_f16 yields the keys' elements, (4j, 4j + 1), (4j + 2, 4j + 3) of 16, and a
    // row is scaled by the power of two that brings its largest element to
    // [2^14, 2^15): f16 holds the bf16 elements exactly down to 2^-31 of that.
    __device__ __forceinline__ void load_q(const SplitArgs& s, int b, int row, int lane)
    {
        const int g = lane >> 2, j = lane & 3, D = s.a.D;
        const int h = s.chunks == 1 ? row : row / s.chunks, c = row - h * s.chunks;
#pragma unroll
        for (int half = 0; half < NROW / 8; half++) {
            const int hg = c * NROW + g + 8 * half;
            const bool in = hg < s.G;
            const uint16_t* src = s.a.q + ((size_t)b * s.a.hq + h * s.G + (in ? hg : 0)) * D;
#pragma unroll
            for (int ks = 0; ks < KS; ks++) {
                uint32_t x = 0, y = 0;
                if (in && 16 * ks < D) {
                    if (F8) {
                        const uint2 u = *reinterpret_cast<const uint2*>(src + 16 * ks + 4 * j);
                        x = u.x;
                        y = u.y;
                    } else {
                        x = *reinterpret_cast<const uint32_t*>(src + 16 * ks + 2 * j);
                        y = *reinterpret_cast<const uint32_t*>(src + 16 * ks + 2 * j + 8);
                    }
                }
                q[ks][NROW == 8 ? 0 : half] = x;
                q[ks][NROW == 8 ? 1 : 2 + half] = y;
            }
        }
    }

    // What load_q left, ready for the products.
    __device__ __forceinline__ void ready_q(const SplitArgs& s)
    {
        const float f = s.a.softcap > 0.0f ? s.a.scale / s.a.softcap : s.a.scale * 1.4426950408889634f;
#pragma unroll
        for (int half = 0; half < NROW / 8; half++) {
            qf[half] = f;
            if (F8) {
                const int qx = NROW == 8 ? 0 : half, qy = NROW == 8 ? 1 : 2 + half;
                uint32_t top = 0;               // bf16 magnitudes order as integers
#pragma unroll
                for (int ks = 0; ks < KS; ks++) top = __vmaxu2(top, __vmaxu2(q[ks][qx] & 0x7FFF7FFFu, q[ks][qy] & 0x7FFF7FFFu));
                top = max(top & 0xFFFFu, top >> 16);
                top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                const int e = min(14 - ((int)(top >> 7) - 127), 126);
                const float up = exp2i(e);
                qf[half] = f * exp2i(-e);
#pragma unroll
                for (int ks = 0; ks < KS; ks++) {
                    const uint32_t x = q[ks][qx], y = q[ks][qy];
                    q[ks][qx] = pack_f16(__uint_as_float(x << 16) * up, __uint_as_float(x & 0xFFFF0000u) * up);
                    q[ks][qy] = pack_f16(__uint_as_float(y << 16) * up, __uint_as_float(y & 0xFFFF0000u) * up);
                }
            }
        }
    }

    __device__ __forceinline__ void mma_q(float (&d)[4], int ks, uint32_t b0, uint32_t b1)
    {
        if (NROW == 8) mma<F8>(d, q[ks][0], 0u, q[ks][1], 0u, b0, b1);
        else mma<F8>(d, q[ks][0], q[ks][1], q[ks][2], q[ks][3], b0, b1);
    }

    // The weights of 16 keys as A operands: high terms, low terms and (FINE, bf16)
    // the rest, rows g and g + 8 of the first and the last 8 keys.
    struct Terms {
        uint32_t h[4], l[4], t[4];

        __device__ __forceinline__ void make(const float (&a)[4], const float (&b)[4])
        {
            h[1] = h[3] = l[1] = l[3] = t[1] = t[3] = 0;
            split<F8>(a[0], a[1], h[0], l[0], t[0]);
            split<F8>(b[0], b[1], h[2], l[2], t[2]);
            if (NROW == 16) {
                split<F8>(a[2], a[3], h[1], l[1], t[1]);
                split<F8>(b[2], b[3], h[3], l[3], t[3]);
            }
        }

        __device__ __forceinline__ void times(float (&d)[4], uint32_t b0, uint32_t b1) const
        {
            if (NROW == 8) {
                mma<F8>(d, h[0], l[0], h[2], l[2], b0, b1);
            } else {
                mma<F8>(d, h[0], h[1], h[2], h[3], b0, b1);
                mma<F8>(d, l[0], l[1], l[2], l[3], b0, b1);
            }
            if (FINE && !F8) mma<F8>(d, t[0], t[1], t[2], t[3], b0, b1);
        }
    };

    // Weights times 16 keys' values, the 32 bytes of their rows at `addr`.
    __device__ __forceinline__ static void values(float (&d)[F8 ? 4 : 2][4], const Terms& w, uint32_t addr)
    {
        uint32_t r[4];
        ldsm4t(r, addr);
        if (F8) {
            // chunk 2 c2 (r0, r1) and 2 c2 + 1 (r2, r3), 16 columns each: even ones, odd ones
#pragma unroll
            for (int c = 0; c < 2; c++) {
                uint32_t e0, d0, e1, d1;
                e4m3_to_f16(__byte_perm(r[2 * c], 0, 0x3120), e0, d0);
                e4m3_to_f16(__byte_perm(r[2 * c + 1], 0, 0x3120), e1, d1);
                w.times(d[F8 ? 2 * c : 0], e0, e1);
                w.times(d[F8 ? 2 * c + 1 : 1], d0, d1);
            }
        } else {
            w.times(d[0], r[0], r[1]);
            w.times(d[1], r[2], r[3]);
        }
    }

    // o times `down`, a factor a row
    __device__ __forceinline__ void shrink(const float (&down)[2])
    {
#pragma unroll
        for (int i = 0; i < ND; i++) {
            o[i][0] *= down[0];
            o[i][1] *= down[0];
            o[i][2] *= NROW == 8 ? down[0] : down[1];                // NROW 8: the low terms' sums
            o[i][3] *= NROW == 8 ? down[0] : down[1];
        }
    }

    // E4M3: new references m and up, and x, the scores less the old one, r, less the
    // new one; w0 is the old whole(up) and then the new; t: the largest of a row's x.
    __device__ __forceinline__ void rebase(float (&x)[NT][4], const float (&t)[2], const float (&r)[2], float (&w0)[2], const float* sc,
                                           int j)
    {
        constexpr int NV = NROW == 8 ? 2 : 4;
        float d[2] = {0.0f, 0.0f}, ty[2] = {-INFINITY, -INFINITY}, down[2] = {1.0f, 1.0f};
        bool none[2] = {true, true};            // no key yet: nothing to bring along
#pragma unroll
        for (int k = 0; k < NV / 2; k++) {
            none[k] = m[k] == -INFINITY;
            m[k] = fmaxf(m[k], r[k] + t[k]);
            d[k] = r[k] - (m[k] == -INFINITY ? 0.0f : m[k]);
        }
#pragma unroll
        for (int n = 0; n < NT; n++) {
            const float2 e = *reinterpret_cast<const float2*>(sc + TT + 8 * n + 2 * j);
#pragma unroll
            for (int k = 0; k < NV; k++) {
                x[n][k] += d[k >> 1];
                ty[k >> 1] = fmaxf(ty[k >> 1], x[n][k] + ((k & 1) ? e.y : e.x));
            }
        }
#pragma unroll
        for (int i = 1; i <= 2; i++)
#pragma unroll
            for (int k = 0; k < NV / 2; k++) ty[k] = fmaxf(ty[k], __shfl_xor_sync(0xFFFFFFFFu, ty[k], i));
#pragma unroll
        for (int k = 0; k < NV / 2; k++) {
            const float w = w0[k];
            up[k] = fmaxf(up[k] + d[k], ty[k] - kLift);
            w0[k] = whole(up[k]);
            // (the sum rounds by 2^-24 of itself, which counts for little where it is large:
            // what it is the exponent of is small beside the new keys' then)
            l[k] *= none[k] ? 0.0f : ex2(d[k]);
            down[k] = none[k] ? 0.0f : ex2(d[k] + (w - w0[k]));
        }
        shrink(down);
    }

    // One tile: `lo`, `hi` are the first and one past the last key of it that
    // count; bad: a bit per 16 keys left out.
    __device__ __forceinline__ void tile(const SplitArgs& s, uint32_t st, const uint8_t* stp, float* sc, int lane, int lo, int hi,
                                         uint32_t bad)
    {
        const int j = lane & 3;
        float top_scale = 0.0f;                 // E4M3: log2 of the largest of v's scales
        if (F8) {
            // a key a lane: k's scale as a number, v's as an exponent, bytes of 255 as
            // NaN, those of keys that do not count as 0 (2^-127)
            uint32_t top = 0;
#pragma unroll
            for (int i = lane; i < TT; i += 32) {
                const uint8_t* b = stp + 2 * TT * ROWB + i;
                const bool in = i >= lo && i < hi && !((bad >> (i / 16)) & 1);
                const uint32_t kb = in ? b[0] : 0, vb = in ? b[TT] : 0;
                // the exponent field alone is zero for 0 and infinity for 255
                sc[i] = __uint_as_float(kb << 23 | (kb == 0 || kb == 255 ? 1u << 22 : 0u));
                sc[TT + i] = vb == 255 ? __uint_as_float(0x7FC00000u)
                                       : __uint_as_float(0x4B000000u | vb) - 8388735.0f;    // 2^23 + byte, less 2^23 + 127
                top = max(top, vb);
            }
            __syncwarp();
            top_scale = (float)(int)__reduce_max_sync(0xFFFFFFFFu, top) - 127.0f;
        }
        const uint32_t kb = st, vb = st + TT * ROWB;
        float x[NT][4];
#pragma unroll
        for (int i = 0; i < NT; i++)
#pragma unroll
            for (int k = 0; k < 4; k++) x[i][k] = 0.0f;
        // scores: 16 keys x 32 bytes of their rows per load
        const int kr = (lane & 7) + ((lane >> 4) & 1) * 8, kc = (lane >> 3) & 1;
#pragma unroll
        for (int c2 = 0; c2 < C2; c2++) {
#pragma unroll
            for (int n2 = 0; n2 < NT / 2; n2++) {
                uint32_t r[4];
                ldsm4(r, at_chunk<ROWB>(kb, 16 * n2 + kr, 2 * c2 + kc));
                if (F8) {
                    uint32_t e, d;
                    e4m3_to_f16(r[0], e, d);
                    mma_q(x[2 * n2], 2 * c2, e, d);
                    e4m3_to_f16(r[2], e, d);
                    mma_q(x[2 * n2 + 1], 2 * c2, e, d);
                    e4m3_to_f16(r[1], e, d);
                    mma_q(x[2 * n2], 2 * c2 + 1, e, d);
                    e4m3_to_f16(r[3], e, d);
                    mma_q(x[2 * n2 + 1], 2 * c2 + 1, e, d);
                } else {
                    mma_q(x[2 * n2], c2, r[0], r[1]);
                    mma_q(x[2 * n2 + 1], c2, r[2], r[3]);
                }
            }
        }
        // the softmax works in powers of two: x = s log2(e)
        constexpr float kLog2e = 1.4426950408889634f;
        constexpr int NV = NROW == 8 ? 2 : 4;
#pragma unroll
        for (int n = 0; n < NT; n++) {
            float2 f = make_float2(1.0f, 1.0f);
            if (F8) f = *reinterpret_cast<const float2*>(sc + 8 * n + 2 * j);
#pragma unroll
            for (int k = 0; k < NV; k++) x[n][k] *= F8 ? qf[k >> 1] * ((k & 1) ? f.y : f.x) : qf[k >> 1];
        }
        if (s.a.softcap > 0.0f) {
            const float cap = s.a.softcap * kLog2e;
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int k = 0; k < NV; k++) x[n][k] = cap * tanhf(x[n][k]);
        }
        // E4M3: x less the reference from here on
        float r[2] = {0.0f, 0.0f}, w0[2] = {0.0f, 0.0f};
        if (F8) {
#pragma unroll
            for (int k = 0; k < NV / 2; k++) {
                r[k] = m[k] == -INFINITY ? 0.0f : m[k];
                w0[k] = whole(up[k]);
            }
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int k = 0; k < NV; k++) x[n][k] -= r[k >> 1];
        }
        if (lo > 0 || hi < TT || bad) {
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int k = 0; k < NV; k++) {
                    const int at = 8 * n + 2 * j + (k & 1);
                    if (at < lo || at >= hi || ((bad >> (n / 2)) & 1)) x[n][k] = -INFINITY;
                }
        }
        float t[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int k = 0; k < NV; k++) t[k >> 1] = fmaxf(t[k >> 1], x[n][k]);
#pragma unroll
        for (int d = 1; d <= 2; d++)
#pragma unroll
            for (int k = 0; k < NV / 2; k++) t[k] = fmaxf(t[k], __shfl_xor_sync(0xFFFFFFFFu, t[k], d));
        if (F8) {
            // o's weights stay below 2^(kLift + kSlack) if even the largest scale meets
            // the largest score, which only now and then moves a reference for nothing
            bool move = false;
#pragma unroll
            for (int k = 0; k < NV / 2; k++)
                move = move || t[k] > (m[k] == -INFINITY ? -INFINITY : kSlack) || t[k] + (top_scale - w0[k]) > kLift + kSlack;
            if (__any_sync(0xFFFFFFFFu, move)) rebase(x, t, r, w0, sc, j);
#pragma unroll
            for (int n = 0; n < NT; n++) {
                const float2 e = *reinterpret_cast<const float2*>(sc + TT + 8 * n + 2 * j);
#pragma unroll
                for (int k = 0; k < NV; k++) {
                    const float y = x[n][k] + (((k & 1) ? e.y : e.x) - w0[k >> 1]);
                    l[k >> 1] += ex2(x[n][k]);
                    x[n][k] = ex2(y);
                }
            }
        } else {
            const bool move = t[0] > m[0] + kSlack || (NROW == 16 && t[1] > m[1] + kSlack);
            if (__any_sync(0xFFFFFFFFu, move)) {
                float down[2] = {1.0f, 1.0f};
#pragma unroll
                for (int k = 0; k < NV / 2; k++) {
                    const float to = fmaxf(m[k], t[k]);
                    if (to != m[k]) down[k] = ex2(m[k] - to);        // 0 from -inf
                    m[k] = to;
                    l[k] *= down[k];
                }
                shrink(down);
            }
#pragma unroll
            for (int k = 0; k < 2; k++)         // before the first key the reference is -inf, and every x as well
                r[k] = m[k] == -INFINITY ? 0.0f : m[k];
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int k = 0; k < NV; k++) {
                    x[n][k] = ex2(x[n][k] - r[k >> 1]);
                    l[k >> 1] += x[n][k];
                }
        }
        // values: 16 keys x 32 bytes of their rows per load.  NROW 8: rows 0..7 of
        // the A operand hold the weights' high terms and rows 8..15 their low
        // terms, so one MMA multiplies both; NROW 16 takes two.
        const int vr = (lane & 7) + ((lane >> 3) & 1) * 8, vc = lane >> 4;
        Terms w[FINE ? NT / 2 : 1];
        if (FINE) {
            // The tensor core cuts the sums it keeps to 24 bits, so a long row's would
            // drift by 2^-25 a product of 16 keys (up to 6e-6 of a row's norm): a
            // tile's sums are made alone and added, rounded, to the row's.
#pragma unroll
            for (int n2 = 0; n2 < NT / 2; n2++) w[n2].make(x[2 * n2], x[2 * n2 + 1]);
#pragma unroll
            for (int c2 = 0; c2 < C2; c2++) {
                constexpr int M = F8 ? 4 : 2;
                float d[M][4];
#pragma unroll
                for (int i = 0; i < M; i++) d[i][0] = d[i][1] = d[i][2] = d[i][3] = 0.0f;
#pragma unroll
                for (int n2 = 0; n2 < NT / 2; n2++) values(d, w[n2], at_chunk<ROWB>(vb, 16 * n2 + vr, 2 * c2 + vc));
#pragma unroll
                for (int i = 0; i < M; i++)
#pragma unroll
                    for (int k = 0; k < 4; k++) o[M * c2 + i][k] += d[i][k];
            }
        } else {
#pragma unroll
            for (int n2 = 0; n2 < NT / 2; n2++) {
                w[0].make(x[2 * n2], x[2 * n2 + 1]);
#pragma unroll
                for (int c2 = 0; c2 < C2; c2++)
                    values(*reinterpret_cast<float(*)[F8 ? 4 : 2][4]>(&o[(F8 ? 4 : 2) * c2]), w[0],
                           at_chunk<ROWB>(vb, 16 * n2 + vr, 2 * c2 + vc));
            }
        }
    }

    // The sums over the row's four lanes, and (NROW 8) the two terms' rows added.
    __device__ __forceinline__ void close()
    {
#pragma unroll
        for (int k = 0; k < NROW / 8; k++) {
            l[k] += __shfl_xor_sync(0xFFFFFFFFu, l[k], 1);
            l[k] += __shfl_xor_sync(0xFFFFFFFFu, l[k], 2);
        }
        if (NROW == 8) {
#pragma unroll
            for (int i = 0; i < ND; i++) {
                o[i][0] += o[i][2];
                o[i][1] += o[i][3];
            }
        }
    }

    // 2^k / l, the factor from o to the output (k within +-160, in two factors: l may
    // be what brings it into range); 0 for a row without keys
    __device__ __forceinline__ static float quotient(float l, float k)
    {
        if (l == 0.0f) return 0.0f;
        if (!F8) return 1.0f / l;
        const int e = (int)k, a = e >> 1;
        return 1.0f / l * exp2i(a) * exp2i(e - a);
    }

    // Column of o[i][k] (k = 0, 1), and of the pair (i, k), (i + 1, k) in E4M3.
    __device__ __forceinline__ static int column(int i, int k, int j)
    {
        return F8 ? 16 * (i / 2) + 4 * j + 2 * k + (i & 1) : 8 * i + 2 * j + k;
    }

    __device__ __forceinline__ void store_part(float* p, int lane) const
    {
        const int g = lane >> 2, j = lane & 3;
#pragma unroll
        for (int half = 0; half < NROW / 8; half++) {
            float* r = p + (g + 8 * half) * PROW;
            if (F8) {           // four columns in a row from an even and an odd MMA column block
#pragma unroll
                for (int i = 0; i < ND; i += 2)
                    *reinterpret_cast<float4*>(r + column(i, 0, j)) =
                        make_float4(o[i][2 * half], o[i + 1][2 * half], o[i][2 * half + 1], o[i + 1][2 * half + 1]);
            } else {
#pragma unroll
                for (int i = 0; i < ND; i++)
                    *reinterpret_cast<float2*>(r + column(i, 0, j)) = make_float2(o[i][2 * half], o[i][2 * half + 1]);
            }
            if (j == 0) {
                p[PHEAD + g + 8 * half] = m[half];
                p[PHEAD + NROW + g + 8 * half] = l[half];
                if (F8) p[PHEAD + 2 * NROW + g + 8 * half] = whole(up[half]);
            }
        }
    }

    __device__ __forceinline__ void store_out(const SplitArgs& s, int b, int row, int lane) const
    {
        const int g = lane >> 2, j = lane & 3;
        const int h = s.chunks == 1 ? row : row / s.chunks, c = row - h * s.chunks;
#pragma unroll
        for (int half = 0; half < NROW / 8; half++) {
            const int hg = c * NROW + g + 8 * half;
            if (hg >= s.G) continue;
            const size_t at = (size_t)b * s.a.hq + h * s.G + hg;
            const float inv = quotient(l[half], F8 ? whole(up[half]) : 0.0f);
            const size_t out = at * s.a.D;
            if (F8) {           // four columns in a row from an even and an odd MMA column block
#pragma unroll
                for (int i = 0; i < ND; i += 2) {
                    const int d = column(i, 0, j);
                    if (d < s.a.D)
                        put4(s.a, out + d, o[i][2 * half] * inv, o[i + 1][2 * half] * inv, o[i][2 * half + 1] * inv,
                             o[i + 1][2 * half + 1] * inv);
                }
            } else {
#pragma unroll
                for (int i = 0; i < ND; i++) {
                    const int d = column(i, 0, j);
                    if (d < s.a.D) put2(s.a, out + d, o[i][2 * half] * inv, o[i][2 * half + 1] * inv);
                }
            }
            if (j == 0) put_lse(s.a, at, m[half], l[half]);
        }
    }

    __device__ __forceinline__ static void put2(const AttnArgs& a, size_t at, float x, float y)
    {
        if (a.out_f32) *reinterpret_cast<float2*>(reinterpret_cast<float*>(a.out) + at) = make_float2(x, y);
        else *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(a.out) + at) = pack_bf16(x, y);
    }

    __device__ __forceinline__ static void put4(const AttnArgs& a, size_t at, float x, float y, float z, float w)
    {
        if (a.out_f32) *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + at) = make_float4(x, y, z, w);
        else *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + at) = make_uint2(pack_bf16(x, y), pack_bf16(z, w));
    }

    __device__ __forceinline__ static void put_lse(const AttnArgs& a, size_t at, float m, float l)
    {
        if (a.lse) a.lse[at] = l == 0.0f ? -INFINITY : m * 0.6931471805599453f + logf(l);
    }

    static constexpr int VEC = DP / 32;         // columns a lane in a merge

    // far: another CTA's
    __device__ __forceinline__ static void load_vec(float (&v)[VEC], const float* p, bool far)
    {
        if (VEC == 4) {
            const float4 x = far ? __ldcg(reinterpret_cast<const float4*>(p)) : *reinterpret_cast<const float4*>(p);
            v[0] = x.x;
            v[1] = x.y;
            v[VEC - 2] = x.z;
            v[VEC - 1] = x.w;
        } else {
            const float2 x = far ? __ldcg(reinterpret_cast<const float2*>(p)) : *reinterpret_cast<const float2*>(p);
            v[0] = x.x;
            v[1] = x.y;
        }
    }

    // A merged row's VEC columns a lane, to its part `to` or as the row's output.
    __device__ __forceinline__ static void finish(const SplitArgs& s, int b, int row, int g, int lane, const float (&acc)[VEC],
                                                  float top, float sum, float k, float* to)
    {
        const int d = lane * VEC;
        if (to) {
            if (VEC == 4) *reinterpret_cast<float4*>(to + g * PROW + d) = make_float4(acc[0], acc[1], acc[VEC - 2], acc[VEC - 1]);
            else *reinterpret_cast<float2*>(to + g * PROW + d) = make_float2(acc[0], acc[1]);
            if (lane == 0) {
                to[PHEAD + g] = top;
                to[PHEAD + NROW + g] = sum;
                if (F8) to[PHEAD + 2 * NROW + g] = k;
            }
            return;
        }
        const int h = s.chunks == 1 ? row : row / s.chunks, hg = (row - h * s.chunks) * NROW + g;
        if (hg >= s.G) return;
        const size_t out = (size_t)b * s.a.hq + h * s.G + hg;
        const float inv = quotient(sum, k);
        if (d < s.a.D) {
            if (VEC == 4) put4(s.a, out * s.a.D + d, acc[0] * inv, acc[1] * inv, acc[VEC - 2] * inv, acc[VEC - 1] * inv);
            else put2(s.a, out * s.a.D + d, acc[0] * inv, acc[1] * inv);
        }
        if (lane == 0) put_lse(s.a, out, top, sum);
    }

    // A row's parts in this CTA, `mem`, at most one a warp (bit 2 w or 2 w + 1,
    // at near(w, 1 or 2)): their weights to tab[bit][NROW], the row's references
    // and sum to tab[16 ..][f][NROW].
    template <class Near>
    __device__ __forceinline__ static void weigh(unsigned mem, Near near, int f, int g, float* tab)
    {
        float m[kWarps], l[kWarps], k[kWarps];
        float top = -INFINITY, above = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; w++) {
            // a place is read whether it holds a part or not, so that no load waits for a branch
            const unsigned is = (mem >> (2 * w)) & 3u;
            const float* e = near(w, is) + PHEAD + g;
            const float a = e[0], b = e[NROW], c = F8 ? e[2 * NROW] : 0.0f;
            m[w] = is ? a : -INFINITY;
            l[w] = is ? b : 0.0f;
            k[w] = is ? c : 0.0f;
        }
#pragma unroll
        for (int w = 0; w < kWarps; w++) top = fmaxf(top, m[w]);
        // -inf before the first key: nothing to bring to the new references
        const float rt = top == -INFINITY ? 0.0f : top;
        if (F8) {
#pragma unroll
            for (int w = 0; w < kWarps; w++) above = fmaxf(above, m[w] + k[w]);
        }
        const float kt = F8 ? whole(above - rt) : 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; w++) {
            const unsigned is = (mem >> (2 * w)) & 3u;
            const float by = ex2(m[w] - rt);
            if (is) tab[(2 * w + (is >> 1)) * NROW + g] = F8 ? ex2(m[w] - rt + (k[w] - kt)) : by;
            sum += by * l[w];
        }
        float* t = tab + (2 * kWarps + f) * NROW + g;
        t[0] = top;
        t[2 * kWarps * NROW] = sum;
        t[4 * kWarps * NROW] = kt;
    }

    // A row's parts of several CTAs merged by one warp: lane i holds part i's
    // numbers, every lane VEC columns of all, and 16 parts' loads are in flight at a
    // time.  at(i) is part i, i < n.
    template <class At>
    __device__ __forceinline__ static void join(const SplitArgs& s, int n, At at, int b, int row, int g, int lane)
    {
        constexpr int N = 16;
        float acc[VEC], top = -INFINITY, kt = 0.0f, sum = 0.0f;
#pragma unroll
        for (int k = 0; k < VEC; k++) acc[k] = 0.0f;
        for (int i0 = 0; i0 < n; i0 += 32) {
            float m = -INFINITY, l = 0.0f, pk = 0.0f;
            if (i0 + lane < n) {
                const float* e = at(i0 + lane) + PHEAD + g;
                m = __ldcg(e);
                l = __ldcg(e + NROW);
                if (F8) pk = __ldcg(e + 2 * NROW);
            }
            float v[N][VEC];
#pragma unroll
            for (int i = 0; i < N; i++) {
#pragma unroll
                for (int k = 0; k < VEC; k++) v[i][k] = 0.0f;
                if (i0 + i < n) load_vec(v[i], at(i0 + i) + g * PROW + lane * VEC, true);
            }
            float t = m, above = m + pk;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, o));
                if (F8) above = fmaxf(above, __shfl_xor_sync(0xFFFFFFFFu, above, o));
            }
            t = fmaxf(t, top);
            above = fmaxf(above, top + kt);
            const float rt = t == -INFINITY ? 0.0f : t;
            float down = ex2(top - rt), w = ex2(m - rt);
            sum = sum * down + warp_sum(w * l);
            if (F8) {
                const float k = whole(above - rt);
                down = ex2(top - rt + (kt - k));
                w = ex2(m - rt + (pk - k));
                kt = k;
            }
            top = t;
#pragma unroll
            for (int k = 0; k < VEC; k++) acc[k] *= down;
#pragma unroll
            for (int h = 0; h < 2; h++) {
#pragma unroll
                for (int i = 0; i < N; i++) {
                    const float f = __shfl_sync(0xFFFFFFFFu, w, N * h + i);
                    if (i0 + N * h + i < n) {
#pragma unroll
                        for (int k = 0; k < VEC; k++) acc[k] = fmaf(f, v[i][k], acc[k]);
                    }
                    if (h == 0 && i0 + N + i < n) load_vec(v[i], at(i0 + N + i) + g * PROW + lane * VEC, true);
                }
            }
        }
        finish(s, b, row, g, lane, acc, top, sum, kt, nullptr);
    }
};

// A part that a warp leaves behind: 2 w + 0 from its first row, 2 w + 1 from its last.
struct Frag {
    int b, row;                 // b < 0: none
    int from_start, to_end;     // the part holds the row's first tile, its last tile
};

// A CTA's sequence, where every row has CTAs of its own: the tiles and the CTAs of
// each of its rows, and the CTAs before its first.
struct Apart {
    int b;
    uint32_t tiles, ctas, before;
};

// A place on the line of tiles.
struct Place {
    int b, row, t, tiles;
};

template <int DP, int CW, bool F8, int NROW, bool FINE>
__global__ void __launch_bounds__(kThreads, 1) k_attn(const __grid_constant__ SplitArgs s)
{
    using K = Kernel<DP, CW, F8, NROW, FINE>;
    constexpr int TT = K::TT;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint32_t s_warp[2][kWarps];
    __shared__ Apart s_own;
    __shared__ int s_apart[2];                  // apart: the first of this row's CTAs and their number, else -1
    __shared__ Frag s_frag[2 * kWarps];
    __shared__ int s_first[2], s_count[2];
    uint8_t* ring = smem;
    uint32_t* pre = reinterpret_cast<uint32_t*>(smem + kWarps * K::REGION);   // [B + 1]
    int* slen = reinterpret_cast<int*>(pre + s.a.B + 1);                               // [B]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int B = s.a.B, ps = s.a.page_size, cap = s.a.row * ps;
    pdl_wait();

    // tiles before each sequence (of one row), by a scan over the lengths
    uint32_t base = 0;
    auto tiles_of = [&](int i) {
        if (i >= B) return 0u;
        int n = s.a.lens[i];
        if ((n < 0 || n > cap) && blockIdx.x == 0) atomicOr(s.a.status, kStatusBadIndex);
        n = min(max(n, 0), cap);
        slen[i] = n;
        const int first = s.a.window > 0 ? max(0, n - s.a.window) : 0;
        return (uint32_t)max(1, (n + TT - 1) / TT - first / TT);
    };
    auto scan = [&](uint32_t x) {               // over B lanes, if they are fewer than a warp's
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            if (d >= B) break;
            const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, d);
            if (lane >= d) x += y;
        }
        return x;
    };
    // Few rows: CTAs of their own, one for a row of up to one_cta tiles, else one for
    // every kWarps tiles; `own` is this CTA's sequence.
    const uint32_t R = (uint32_t)s.R, one_cta = one_cta_tiles(F8, (uint32_t)B * R);
    auto ctas_of = [&](uint32_t tiles) { return tiles <= one_cta ? min(tiles, 1u) : (tiles + kWarps - 1) / kWarps; };
    bool apart = false;
    uint32_t ctas = 0;          // of all rows
    Apart own = {};
    if (B <= 32) {              // every warp by itself, all writing the same
        const uint32_t mine = tiles_of(lane), x = scan(mine), n = ctas_of(mine), y = scan(n);
        if (lane < B) pre[lane + 1] = x;
        if (lane == 0) pre[0] = 0;
        base = __shfl_sync(0xFFFFFFFFu, x, B - 1);
        ctas = __shfl_sync(0xFFFFFFFFu, y, B - 1) * R;
        apart = ctas <= gridDim.x;
        if (apart) {
            own.b = min(__popc(__ballot_sync(0xFFFFFFFFu, lane < B && y * R <= blockIdx.x)), B - 1);
            own.tiles = __shfl_sync(0xFFFFFFFFu, mine, own.b);
            own.ctas = __shfl_sync(0xFFFFFFFFu, n, own.b);
            own.before = (__shfl_sync(0xFFFFFFFFu, y, own.b) - own.ctas) * R;
        }
        __syncwarp();
    } else {
        const bool few = (uint32_t)B * R <= gridDim.x;          // so that B < kThreads
        for (int i0 = 0; i0 < B; i0 += kThreads) {
            const uint32_t mine = tiles_of(i0 + tid), n = ctas_of(mine), x = scan(mine), y = few ? scan(n) : 0u;
            if (lane == 31) {
                s_warp[0][warp] = x;
                s_warp[1][warp] = y;
            }
            __syncthreads();
            uint32_t before = base, all = base, ctas_before = 0;
            ctas = 0;
#pragma unroll
            for (int w = 0; w < kWarps; w++) {
                if (w < warp) {
                    before += s_warp[0][w];
                    ctas_before += s_warp[1][w];
                }
                all += s_warp[0][w];
                ctas += s_warp[1][w];
            }
            if (i0 + tid < B) pre[i0 + tid + 1] = before + x;
            base = all;
            ctas *= R;
            apart = few && ctas <= gridDim.x;
            const uint32_t end = (ctas_before + y) * R, begin = end - n * R;
            if (apart && begin <= blockIdx.x && blockIdx.x < end) s_own = Apart{tid, mine, n, begin};
            __syncthreads();
        }
        if (tid == 0) pre[0] = 0;
        __syncthreads();
        if (apart && blockIdx.x < ctas) own = s_own;
    }
    // The line in units: a row's tiles, and kRowCost for the row itself where warps
    // have several rows.  The CTAs' stretches are equal to one unit, and the warps'
    // within them; fewer CTAs where they would not have a tile for every warp.
    const uint32_t tiles_all = base * R;
    const bool full = !apart && tiles_all >= gridDim.x * kWarps;
    const uint32_t V = full ? kRowCost : 0, W = tiles_all + V * (uint32_t)B * R;
    const uint32_t grid = apart ? ctas : min(gridDim.x, (W + kWarps - 1) / kWarps);
    if (blockIdx.x >= grid) return;
    // a / b; of small numbers (a line that is not full has below 2^14 units) by way
    // of floats: (a + 1/2) / b is 1 / 2b or more from an integer, and off by far less
    auto div = [&](uint32_t a, uint32_t b) {
        return full ? a / b : (uint32_t)__fdividef((float)a + 0.5f, (float)b);
    };
    const uint32_t wq = div(W, grid), wr = W - wq * grid;
    auto cta_of = [&](uint32_t at) { return at < wr * (wq + 1) ? at / (wq + 1) : wr + (at - wr * (wq + 1)) / wq; };
    auto units_before = [&](int b) { return (pre[b] + V * (uint32_t)b) * R; };
    auto seq_of = [&](uint32_t at) {            // the last sequence that begins at or before `at`
        if (B <= 32) return __popc(__ballot_sync(0xFFFFFFFFu, lane < B - 1 && units_before(lane + 1) <= at));
        int lo = 0, hi = B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (units_before(mid) <= at) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    };
    // A CTA's stretch; where warps would idle it does not begin or end inside a
    // row of up to one_cta tiles, but at its end (cta_of still holds for longer rows).
    auto snap = [&](uint32_t at) {
        if (at >= W) return at;
        const int b = seq_of(at);
        const uint32_t tiles = pre[b + 1] - pre[b], in = at - units_before(b), t = in - div(in, tiles) * tiles;
        return tiles <= one_cta && t ? at + tiles - t : at;
    };
    Place begin = {};
    uint32_t lo, hi, row0 = 0;
    if (apart) {
        const uint32_t in = blockIdx.x - own.before, row = div(in, own.ctas);
        const uint32_t piece = in - row * own.ctas;
        if (tid == 0) {
            s_apart[0] = (int)(blockIdx.x - piece);
            s_apart[1] = (int)own.ctas;
        }
        row0 = pre[own.b] * R + row * own.tiles;
        lo = row0 + piece * kWarps;
        hi = own.ctas == 1 ? row0 + own.tiles : min(lo + kWarps, row0 + own.tiles);
        begin.b = own.b;
        begin.row = (int)row;
        begin.tiles = (int)own.tiles;
    } else {
        if (tid == 0) s_apart[0] = -1;
        lo = blockIdx.x * wq + min((uint32_t)blockIdx.x, wr);
        hi = lo + wq + (blockIdx.x < wr ? 1u : 0u);
        if (!full) {
            lo = snap(lo);
            hi = snap(hi);
        }
    }
    const uint32_t per = (hi - lo) / kWarps, left = (hi - lo) % kWarps;
    const uint32_t from = lo + warp * per + min((uint32_t)warp, left);
    const uint32_t to = from + per + ((uint32_t)warp < left ? 1u : 0u);

    // The place where a stretch that ends or begins at unit `at` is cut, and the
    // tiles before it.  The units of the row itself come first and hold no tile; a
    // cut inside a row that is not split moves to its end.
    const bool whole_rows = full && base <= (uint32_t)B * kShort;
    auto cut = [&](uint32_t at, uint32_t& tiles) {
        Place p;
        p.b = seq_of(at);
        p.tiles = (int)(pre[p.b + 1] - pre[p.b]);
        const uint32_t units = (uint32_t)p.tiles + V, in = at - units_before(p.b);
        p.row = (int)div(in, units);
        const uint32_t t = in - (uint32_t)p.row * units;
        p.t = (int)(t - min(t, V));
        tiles = at - V * ((uint32_t)p.b * R + (uint32_t)p.row) - min(t, V);
        if (whole_rows && p.tiles <= kWhole / TT && p.t > 0) {
            tiles += (uint32_t)(p.tiles - p.t);
            p.t = 0;
            if (++p.row == s.R) {
                p.row = 0;
                p.b++;
                p.tiles = p.b < B ? (int)(pre[p.b + 1] - pre[p.b]) : 0;
            }
        }
        return p;
    };
    auto advance = [&](Place& p) {
        if (++p.t < p.tiles) return;
        p.t = 0;
        if (++p.row < s.R) return;
        p.row = 0;
        p.b++;
        if (p.b < B) p.tiles = (int)(pre[p.b + 1] - pre[p.b]);
    };
    uint32_t u = tiles_all, end = to;           // in tiles from here on
    if (apart) {
        begin.t = (int)(from - row0);
        if (from < to) u = from;
    } else if (from < to) {
        begin = cut(from, u);
    }
    if (to >= W) end = tiles_all;       // (apart: the last CTA's last warp, where W is tiles_all)
    else if (full) cut(to, end);
    auto first_key = [&](int b) { return s.a.window > 0 ? max(0, slen[b] - s.a.window) : 0; };

    if (lane < 2) s_frag[2 * warp + lane].b = -1;
    __syncwarp();
    K k;
    if (u < end) {
        uint8_t* my = ring + warp * K::REGION;
        const uint32_t my32 = smem_u32(my);
        // The producer's side: a window of 32 tiles' places in the pool, one a lane
        // (in blocks of 16 rows of one head: a page is a whole number of them), and
        // the page ids of the window that comes next, on their way.
        const int hblk = ps / 16;
        int wb = -1, wt = 0, nb = -1, nt = 0;
        uint32_t blk[TT / 16];
        int ids[TT / 16];
        auto page_of = [&](int key) { return s.ps_shift >= 0 ? key >> s.ps_shift : key / ps; };
        auto fetch = [&](int b, int t) {
            nb = b;
            nt = t;
#pragma unroll
            for (int i = 0; i < TT / 16; i++) {
                const int key = (t + lane) * TT + 16 * i;
                ids[i] = key < slen[b] ? s.a.table[(size_t)b * s.a.row + page_of(key)] : 0;
            }
        };
        auto install = [&]() {
            wb = nb;
            wt = nt;
            const int n = slen[wb], first = first_key(wb);
#pragma unroll
            for (int i = 0; i < TT / 16; i++) {
                const int key = (wt + lane) * TT + 16 * i;
                const bool ok = ids[i] >= 0 && ids[i] < s.a.num_pages;
                blk[i] = key < n && ok ? (uint32_t)ids[i] * (uint32_t)(s.a.hkv * hblk) + (uint32_t)((key - page_of(key) * ps) / 16)
                                       : 0xFFFFFFFFu;
                if (key < n && !ok && key + 16 > first) atomicOr(s.a.status, kStatusBadIndex);
            }
        };
        constexpr int BB = TT / 16;             // a tile's bits of badq
        uint32_t badq = 0;
        Place pp = begin, cp = begin;
        uint32_t up = u;
        const int rb = s.a.D * (F8 ? 1 : 2);    // bytes of a cached row
        const int c = lane % K::CPR, r0 = lane / K::CPR;
        const bool cin = c * 16 < rb;
        // a lane's places in the pool's first row block
        const uint8_t* klane = s.a.pool.k + (cin ? (size_t)r0 * rb + c * 16 : 0);
        const uint8_t* vlane = s.a.pool.v + (cin ? (size_t)r0 * rb + c * 16 : 0);
        const uint8_t* slane = lane ? s.a.pool.vs : s.a.pool.ks;

        auto issue = [&](int stage) {
            const int n = slen[pp.b], first = first_key(pp.b), t0 = first / TT, tile = t0 + pp.t;
            if (pp.b != wb || tile < wt || tile >= wt + 32) {
                if (nb != pp.b || nt != tile) fetch(pp.b, tile);
                install();
                // what comes next: the rest of the row, else the next row's (or, where
                // this window holds a whole row, the next sequence's) beginning
                if (pp.t + 32 < pp.tiles) {
                    fetch(pp.b, tile + 32);
                } else if (pp.row + 1 < s.R && (pp.t > 0 || pp.tiles > 32)) {
                    fetch(pp.b, t0);
                } else if (pp.b + 1 < B) {
                    fetch(pp.b + 1, first_key(pp.b + 1) / TT);
                }
            }
            const uint32_t st = my32 + stage * K::STAGE;
            const int h = s.chunks == 1 ? pp.row : pp.row / s.chunks;
            const int lo = first - tile * TT, hi = n - tile * TT;           // keys [lo, hi) of the tile count
            uint32_t at[TT / 16], bad = 0;
#pragma unroll
            for (int i = 0; i < TT / 16; i++) {
                at[i] = __shfl_sync(0xFFFFFFFFu, blk[i], tile - wt);
                bad |= at[i] == 0xFFFFFFFFu ? 1u << i : 0u;
            }
            if (rb == K::ROWB && lo <= 0 && hi >= TT && !bad) {
                // the common tile: every address is one of two and a constant
#pragma unroll
                for (int i = 0; i < TT / 16; i++) {
                    const size_t row = ((size_t)at[i] + (uint32_t)(h * hblk)) * 16;
                    const uint8_t* ksrc = klane + row * K::ROWB;
                    const uint8_t* vsrc = vlane + row * K::ROWB;
#pragma unroll
                    for (int r = 0; r < 16; r += K::RPI) {
                        cp_async16(at_chunk<K::ROWB>(st, 16 * i + r + r0, c), ksrc + r * K::ROWB, 16);
                        cp_async16(at_chunk<K::ROWB>(st + TT * K::ROWB, 16 * i + r + r0, c), vsrc + r * K::ROWB, 16);
                    }
                    if (F8 && lane < 2) cp_async16(st + 2 * TT * K::ROWB + lane * TT + 16 * i, slane + row, 16);
                }
            } else {
#pragma unroll
                for (int i = 0; i < TT / 16; i++) {
                    const bool ok = !((bad >> i) & 1);
                    const size_t row = ok ? ((size_t)at[i] + (uint32_t)(h * hblk)) * 16 : 0;
#pragma unroll
                    for (int r = 0; r < 16; r += K::RPI) {
                        const int rr = 16 * i + r + r0;
                        // rows that no key has are zeros, whatever the pool holds there
                        const bool in = ok && cin && rr >= lo && rr < hi;
                        const size_t off = in ? row * rb + (size_t)r * rb : 0;
                        cp_async16(at_chunk<K::ROWB>(st, rr, c), klane + off, in ? 16 : 0);
                        cp_async16(at_chunk<K::ROWB>(st + TT * K::ROWB, rr, c), vlane + off, in ? 16 : 0);
                    }
                    if (F8 && lane < 2) cp_async16(st + 2 * TT * K::ROWB + lane * TT + 16 * i, slane + row, ok ? 16 : 0);
                }
            }
            badq = (badq & ~(((1u << BB) - 1u) << (BB * stage))) | (bad << (BB * stage));
            up++;
            if (up < end) advance(pp);
        };

        // the first page ids and queries, ahead of the ring's first loads
        fetch(pp.b, first_key(pp.b) / TT + pp.t);
        k.load_q(s, cp.b, cp.row, lane);
#pragma unroll 1
        for (int i = 0; i < K::STAGES - 1; i++) {
            if (up < end) issue(i);
            cp_async_commit();
        }
        int start = cp.t, first_seg = 1, stage = 0;
        k.ready_q(s);
        k.reset();
        while (true) {
            if (up < end) issue(stage == 0 ? K::STAGES - 1 : stage - 1);
            cp_async_commit();
            cp_async_wait<K::STAGES - 1>();
            __syncwarp();
            const int n = slen[cp.b], first = first_key(cp.b), at = (first / TT + cp.t) * TT;
            k.tile(s, my32 + stage * K::STAGE, my + stage * K::STAGE, reinterpret_cast<float*>(my + K::STAGES * K::STAGE), lane, max(0, first - at), min(TT, n - at),
                   (badq >> (BB * stage)) & ((1u << BB) - 1u));
            __syncwarp();
            stage = stage + 1 == K::STAGES ? 0 : stage + 1;
            u++;
            const bool row_done = cp.t + 1 == cp.tiles;
            if (!row_done && u < end) {
                cp.t++;
                continue;
            }
            k.close();
            if (row_done && start == 0) {
                k.store_out(s, cp.b, cp.row, lane);
            } else {
                // A part: the last one of the stretch goes to the warp's ring, which is
                // drained then; one that ends a row before waits in global memory.
                const bool far = u != end;
                k.store_part(far ? s.frags + ((size_t)blockIdx.x * kWarps + warp) * K::PART
                                 : reinterpret_cast<float*>(my) + (first_seg ? 0 : K::PART), lane);
                if (lane == 0) {
                    Frag& f = s_frag[2 * warp + (first_seg ? 0 : 1)];
                    f.b = cp.b;
                    f.row = cp.row;
                    f.from_start = start == 0;
                    f.to_end = row_done;
                }
            }
            if (u == end) {
                if (!first_seg && s_frag[2 * warp].b >= 0) {
                    // the first row's part comes to the ring, too
                    const float* from = s.frags + ((size_t)blockIdx.x * kWarps + warp) * K::PART;
                    for (int i = lane; i < K::PART / 4; i += 32) cp_async16(my32 + 16 * i, from + 4 * i, 16);
                    cp_async_commit();
                    cp_async_wait<0>();
                }
                break;
            }
            advance(cp);
            start = 0;
            first_seg = 0;
            k.load_q(s, cp.b, cp.row, lane);
            k.ready_q(s);
            k.reset();
        }
    }
    pdl_trigger();
    __syncthreads();

    // Parts of one row in this CTA, at most one a warp.  Every warp reads the
    // parts' heads at once, a lane each, and finds the rows' first parts by votes.
    Frag fr;
    fr.b = -1;
    fr.row = fr.from_start = fr.to_end = 0;
    if (lane < 2 * kWarps) fr = s_frag[lane];
    const unsigned there = __ballot_sync(0xFFFFFFFFu, fr.b >= 0);
    const unsigned before = there & ((1u << lane) - 1u);
    const int prev = before ? 31 - __clz(before) : lane;
    const int pb = __shfl_sync(0xFFFFFFFFu, fr.b, prev), pr = __shfl_sync(0xFFFFFFFFu, fr.row, prev);
    const unsigned heads = __ballot_sync(0xFFFFFFFFu, fr.b >= 0 && (!before || pb != fr.b || pr != fr.row));
    const unsigned starts = __ballot_sync(0xFFFFFFFFu, fr.from_start), ends = __ballot_sync(0xFFFFFFFFu, fr.to_end);
    const int heads_in = min(NROW, s.G);
    auto last_of = [&](int f) {                 // the last part of the row whose first is f
        const unsigned after = heads & ~((2u << f) - 1u);
        return 31 - __clz(there & (after ? (after & -after) - 1u : 0xFFFFFFFFu));
    };
    auto members = [&](int f) { return there & ((2u << last_of(f)) - 1u) & ~((1u << f) - 1u); };
    auto near = [&](int w, unsigned is) {
        return reinterpret_cast<const float*>(ring + w * K::REGION) + (is == 1 ? 0 : K::PART);
    };
    float* tab = reinterpret_cast<float*>(ring) + 2 * K::PART;
    // rows that began before this CTA, that go on after it: their first parts here
    int open[2] = {-1, -1};
    if (heads) {
        const int f = __ffs(heads) - 1, l = 31 - __clz(heads);
        if (!((starts >> f) & 1)) open[0] = f;
        if (((starts >> l) & 1) && !((ends >> last_of(l)) & 1)) open[1] = l;
    }
    // first the weights, a thread a head of a row; then the sums, a warp two heads
    for (int i = tid; i < 2 * kWarps * heads_in; i += kThreads)
        if ((heads >> (i % (2 * kWarps))) & 1) K::weigh(members(i % (2 * kWarps)), near, i % (2 * kWarps), i / (2 * kWarps), tab);
    __syncthreads();
    for (int e = warp; e < __popc(heads) << s.pair_shift; e += kWarps) {
        const int g = 2 * (e & ((1 << s.pair_shift) - 1));
        if (g >= heads_in) continue;
        unsigned rest = heads;
        for (int i = e >> s.pair_shift; i > 0; i--) rest &= rest - 1;
        const int f = __ffs(rest) - 1, last = last_of(f);
        const int slot = (starts >> f) & 1;
        const bool whole = slot && ((ends >> last) & 1);
        const unsigned mem = members(f);
        float acc[2][K::VEC];
#pragma unroll
        for (int k = 0; k < K::VEC; k++) acc[0][k] = acc[1][k] = 0.0f;
        for (unsigned rest = mem; rest;) {      // four parts' loads at a time
            float2 by[4];
            float v[4][2][K::VEC];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                // past the last part: the first one again, without weight
                const int x = rest ? __ffs(rest) - 1 : f;
                by[i] = *reinterpret_cast<const float2*>(tab + x * NROW + g);
                if (!rest) by[i] = make_float2(0.0f, 0.0f);
                rest &= rest - 1;
#pragma unroll
                for (int r = 0; r < 2; r++)
                    K::load_vec(v[i][r], near(x >> 1, 1u + (x & 1)) + (g + r) * K::PROW + lane * K::VEC, false);
            }
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int k = 0; k < K::VEC; k++) {
                    acc[0][k] = fmaf(by[i].x, v[i][0][k], acc[0][k]);
                    acc[1][k] = fmaf(by[i].y, v[i][1][k], acc[1][k]);
                }
        }
        float* to = whole ? nullptr : s.parts + ((size_t)blockIdx.x * 2 + slot) * K::PART;
#pragma unroll
        for (int r = 0; r < 2; r++) {
            const float* t = tab + (2 * kWarps + f) * NROW + g + r;
            if (g + r < heads_in)
                K::finish(s, s_frag[f].b, s_frag[f].row, g + r, lane, acc[r], t[0], t[2 * kWarps * NROW], t[4 * kWarps * NROW], to);
        }
    }
    if (open[0] < 0 && open[1] < 0) return;

    // Rows that other CTAs hold parts of, too: the last CTA to finish joins them.
    __syncthreads();
    if (tid < 2) {
        const int f = tid ? open[1] : open[0];
        int first = -1, count = 0;
        if (f >= 0) {
            // the CTA's part was written before the barrier; its release and the
            // others' acquisition are the ticket's
            const int b = s_frag[f].b, row = s_frag[f].row;
            int* ticket = s.tickets + (size_t)b * s.R + row;
            int old;
            asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(old) : "l"(ticket) : "memory");
            // meanwhile, the CTAs that hold the row
            const uint32_t tiles = pre[b + 1] - pre[b], r0 = units_before(b) + (uint32_t)row * (tiles + V) + V;
            int c0 = s_apart[0];
            if (c0 >= 0) {
                count = s_apart[1];
            } else {
                c0 = (int)cta_of(r0);
                count = (int)cta_of(r0 + tiles - 1) - c0 + 1;
            }
            if (old == count - 1) {
                *ticket = 0;
                first = c0;
            }
        }
        s_first[tid] = first;
        s_count[tid] = count;
    }
    __syncthreads();
    for (int e = warp; e < 2 * heads_in; e += kWarps) {
        const int slot = e >= heads_in, g = slot ? e - heads_in : e, c0 = s_first[slot], n = s_count[slot];
        if (c0 < 0) continue;
        // c0 holds the row's beginning, in its slot 1; the others' parts are in slot 0
        K::join(s, n, [&](int x) { return s.parts + ((size_t)(c0 + x) * 2 + (x == 0 ? 1 : 0)) * K::PART; }, s_frag[open[slot]].b,
                s_frag[open[slot]].row, g, lane);
    }
}

template <int DP, int CW, bool F8, int NROW, bool FINE>
cudaError_t launch(const SplitArgs& s, cudaStream_t st)
{
    using K = Kernel<DP, CW, F8, NROW, FINE>;
    const size_t smem = (size_t)kWarps * K::REGION + (2 * (size_t)s.a.B + 1) * 4;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)s.a.sms);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_attn<DP, CW, F8, NROW, FINE>, s);
}

// The kernel of a handle's configuration: f(its template parameters).
template <class F>
cudaError_t dispatch(int D, bool e4m3, int G, bool f32, F f)
{
    using std::bool_constant;
    using std::integral_constant;
    using C64 = integral_constant<int, 64>;
    using C96 = integral_constant<int, 96>;
    using C128 = integral_constant<int, 128>;
    using N8 = integral_constant<int, 8>;
    using N16 = integral_constant<int, 16>;
    using E4m3 = bool_constant<true>;
    using Bf16 = bool_constant<false>;
    using Fine = bool_constant<true>;
    using Plain = bool_constant<false>;
    auto type = [&](auto dp, auto cw, auto f8, auto rows) {
        return f32 ? f(dp, cw, f8, rows, Fine()) : f(dp, cw, f8, rows, Plain());
    };
    if (D <= 64) {
        if (e4m3) return G <= 8 ? type(C64(), C64(), E4m3(), N8()) : type(C64(), C64(), E4m3(), N16());
        return G <= 8 ? type(C64(), C64(), Bf16(), N8()) : type(C64(), C64(), Bf16(), N16());
    }
    if (!e4m3) return G <= 8 ? type(C128(), C128(), Bf16(), N8()) : type(C128(), C128(), Bf16(), N16());
    // E4M3 rows of up to 96 are computed 96 wide (32 sequences of up to 8000: 47.8 us, 52.4
    // with 128); for bf16, which waits for memory, it makes no difference (71.3, 72.5)
    if (D <= 96) return G <= 8 ? type(C128(), C96(), E4m3(), N8()) : type(C128(), C96(), E4m3(), N16());
    // the order of the finer sums is the faster one for E4M3 rows of 128 and up to 8 heads
    // (128 sequences of up to 8000: 176 us, 180 without), and the slower one for more heads
    // (32 sequences: 71.7 and 65.0 us) and shorter rows (96: 48.5 and 47.8)
    return G <= 8 ? f(C128(), C128(), E4m3(), N8(), Fine()) : type(C128(), C128(), E4m3(), N16());
}

int rows_of(int hq, int hkv)
{
    const int G = hq / hkv;
    return hkv * (G <= 8 ? 1 : (G + 15) / 16);
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

AttnWorkspace attn_workspace(int max_seqs, int hq, int hkv, int D, int sms)
{
    const size_t part = (size_t)part_floats(D <= 64 ? 64 : 128, true, hq / hkv <= 8 ? 8 : 16) * sizeof(float);
    AttnWorkspace w;
    w.tickets = 0;
    w.frags = align256((size_t)max_seqs * rows_of(hq, hkv) * sizeof(int));
    w.parts = w.frags + align256((size_t)sms * kWarps * part);
    w.bytes = w.parts + align256((size_t)sms * 2 * part);
    return w;
}

cudaError_t attn_init_device(int hq, int hkv, int D, bool e4m3, bool f32)
{
    return dispatch(D, e4m3, hq / hkv, f32, [](auto dp, auto cw, auto f8, auto nrow, auto fine) {
        using K = Kernel<dp(), cw(), f8(), nrow(), fine()>;
        return cudaFuncSetAttribute(k_attn<dp(), cw(), f8(), nrow(), fine()>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kWarps * K::REGION + (2 * kAttnMaxSeqs + 1) * 4);
    });
}

cudaError_t launch_attn(const AttnArgs& a, cudaStream_t st)
{
    if (a.B == 0) return cudaSuccess;
    SplitArgs s;
    s.a = a;
    s.G = a.hq / a.hkv;
    s.chunks = s.G <= 8 ? 1 : (s.G + 15) / 16;
    s.R = a.hkv * s.chunks;
    s.ps_shift = a.page_size & (a.page_size - 1) ? -1 : __builtin_ctz((unsigned)a.page_size);
    s.pair_shift = s.G <= 2 ? 0 : s.G <= 4 ? 1 : s.G <= 8 ? 2 : 3;
    const AttnWorkspace w = attn_workspace(a.max_seqs, a.hq, a.hkv, a.D, a.sms);
    s.tickets = reinterpret_cast<int*>(a.ws + w.tickets);
    s.frags = reinterpret_cast<float*>(a.ws + w.frags);
    s.parts = reinterpret_cast<float*>(a.ws + w.parts);
    return dispatch(a.D, a.e4m3, s.G, a.out_f32, [&](auto dp, auto cw, auto f8, auto nrow, auto fine) {
        return launch<dp(), cw(), f8(), nrow(), fine()>(s, st);
    });
}

}  // namespace moe
