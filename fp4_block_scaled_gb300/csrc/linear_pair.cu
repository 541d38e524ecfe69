// linear_pair.cu -- the dense product for many tokens: pairs of CTAs
// (tcgen05 cta_group::2), one tile of 256 tokens by 256 features a pair.
//
// The tokens are the MMA's rows here, 128 of each CTA, so that a thread of the epilogue
// holds consecutive features of one token; each CTA brings its own tokens and half of
// the features, a packed tile of 128, and the tensor cores read the other half from the
// other CTA's shared memory: 32 KB a CTA and stage for 256 x 256 outputs, which is what L2 can
// feed (tiles of 128 x 192 by single CTAs were bound by that and by their epilogue).  The CTAs
// stay and take tiles in turn; the epilogue of one overlaps the products of the next, for
// which two accumulators of 256 columns would leave no tensor memory to the scales: they
// share 48 columns.  Outputs leave through shared memory by TMA stores of whole lines (32-byte
// stores of single rows cost 12 % of the time).
//
// Bounds (GB300): 16384 tokens by 4096 x 6144 in E2M1 take 121 us from codes, 6.8 PFLOP/s, 90 %
// of four times the measured bf16 rate (the K = 64 steps' nominal ratio); 8191 by 4096 x 5760 in
// E4M3 109 us, 3.5 PFLOP/s, 94 % of twice that rate.  The tensor pipe is active 77 % and 89 % of
// the time (ncu), the rest is the first stage of a tile behind the last of the one before, and
// the last round of tiles.  What counted: arrivals at the other CTA's barriers that do not wait
// for memory (with a release at cluster scope each took 1600 cycles, a stage 1750 in all),
// one barrier a stage, the scales of a tile's first stage copied while the tile before is
// emptied.
#include <algorithm>
#include <type_traits>

#include "linear.cuh"

namespace moe {

namespace {

constexpr int kRing = 6;
constexpr int kTokens = 256, kFeatures = 256;
constexpr int kWarpProd = 4, kWarpMma = 5, kWarpLoad = 6, kLoadWarps = 4;
constexpr int kThreads = (kWarpLoad + kLoadWarps) * 32;
constexpr uint32_t kOutBytes = 32 * 128;        // of an epilogue warp's box
// Tensor memory: the accumulators of two tiles in turn, which share kShared columns, and
// behind them the scales of two stages (E4M3: four).  The epilogue empties the shared columns
// first, and then the next tile's products may begin.
constexpr int kShared = 48, kScaleCols = 2 * kFeatures - kShared;

struct __align__(1024) Control {
    uint64_t full[kRing], empty[kRing], acc_full, acc_empty, drain;
    uint32_t tmem;
    int abort;
};

template <int E2M1>
struct Stage {
    static constexpr int kAtoms = E2M1 ? 2 : 1;                 // of 128 elements
    static constexpr uint32_t b = 128 * 128, sfa = 2 * b, sfb = sfa + kAtoms * kLinAtom;
    static constexpr uint32_t bytes = (sfb + 2 * kAtoms * kLinAtom + 1023) / 1024 * 1024;
    static constexpr int cols = 12 * kAtoms, slots = kShared / cols;
    static_assert(sizeof(Control) + kRing * bytes + 4 * kOutBytes <= kLinSmemMax && kLoadWarps <= kRing && slots >= 2, "sizes");
};

// Arrives at a barrier of CTA `rank` of the pair: released at this CTA's scope alone, for at
// the cluster's it waited for the memory of the whole CTA (1600 cycles).  That is enough because
// whoever waits there reads nothing of this CTA's by loads of its own.  What follows in the
// other CTA are tcgen05 instructions, of which this CTA's half is carried out here: on shared
// memory that TMA wrote, or that this CTA's threads wrote and fenced to the async proxy ahead of
// the barrier of their own CTA; and into columns that their warp has read (tcgen05.wait::ld,
// tcgen05.fence).  A plain load of the other CTA's shared memory behind such a barrier
// would need .release.cluster here and .acquire.cluster there.
__device__ __forceinline__ void arrive_at(uint64_t* bar, uint32_t rank)
{
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\tmbarrier.arrive.shared::cluster.b64 _, [a];\n\t}" ::"r"(
                     smem_u32(bar)),
                 "r"(rank)
                 : "memory");
}

__device__ __forceinline__ void commit_both(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
                 "h"((uint16_t)3)
                 : "memory");
}

__device__ __forceinline__ void cp_scales(uint32_t taddr, uint64_t desc)
{
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

template <int E2M1>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t sfa, uint32_t sfb, uint32_t acc)
{
    if (E2M1)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(id), "r"(acc), "r"(sfa), "r"(sfb)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(id), "r"(acc), "r"(sfa), "r"(sfb)
            : "memory");
}

// A: the rows (E2M1 1, or E4M3 0); B: the weights (E2M1, 1 of kind::mxf4 and 5 of
// kind::mxf8f6f4); ue8m0 scales, whose bytes `sf` selects.
template <int E2M1>
__device__ __forceinline__ constexpr uint32_t idesc(uint32_t sf)
{
    return (E2M1 ? (1u << 7) | (1u << 10) : (5u << 10)) | ((uint32_t)(kFeatures >> 3) << 17) | (1u << 23) |
           ((uint32_t)(kTokens >> 4) << 24) | (sf << 29) | (sf << 4);
}

__device__ __forceinline__ void tma_store(const CUtensorMap* map, int x, int y, const void* src)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];\n\tcp.async.bulk.commit_group;" ::"l"(map),
                 "r"(x), "r"(y), "r"(smem_u32(src))
                 : "memory");
}

// 32 tokens (a lane each) by 128 bytes of features from n, by one warp: through its 4 KB of
// shared memory, in TMA's swizzle, to whole lines of y.
__device__ __forceinline__ void stage_box(uint8_t* out, int lane, const uint32_t (&w)[32])
{
    // (the box before has left)
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; j++)
        *reinterpret_cast<uint4*>(out + lane * 128 + ((j ^ (lane & 7)) << 4)) = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
}

// Where y's rows do not begin on 16 bytes, which TMA needs, plain stores of the 16 bytes
// that are aligned: each row is turned round by its s elements behind such a boundary, so that
// seven of its eight pieces lie as they do in y, and the eighth holds its first and last
// elements, which go singly.  8192 tokens by 256 x 9727 take 48 us in bf16 and 93 in f32, where
// TMA's by 9728 take 31 and 51 (each read after the store before it 54 and 113; a row's words
// after the other 100 cycles a row, twice that again).
template <int F32>
__device__ __forceinline__ void store_rows(const LinearArgs& a, uint8_t* out, int t, int n, int lane, const uint32_t (&box)[32])
{
    using Value = std::conditional_t<F32, uint32_t, uint16_t>;
    constexpr int kPiece = 16 / sizeof(Value), kRow = 128 / sizeof(Value);
    uint32_t w[32];
    auto turn = [&](int r) { return (int)((uint32_t)(t + r) * (uint32_t)a.N) & (kPiece - 1); };
    const int s = turn(lane), words = F32 ? s : s >> 1;
#pragma unroll
    for (int j = 0; j < 32; j++) w[j] = F32 ? box[j] : __funnelshift_l(box[(j + 31) & 31], box[j], s % 2 * 16);
#pragma unroll
    for (int by = 1; by <= 2; by *= 2) {
        uint32_t v[32];
#pragma unroll
        for (int j = 0; j < 32; j++) v[j] = words & by ? w[(j + 32 - by) & 31] : w[j];
#pragma unroll
        for (int j = 0; j < 32; j++) w[j] = v[j];
    }
    stage_box(out, lane, w);
    __syncwarp();
    // Rows r0, r0 + 4, ... (every read is on its way before the first store; of the rows' turns
    // there are two, one after the other, so that little is computed for each)
    const int have = min(kRow, a.N - n), r0 = lane / 8, c = lane % 8, rows = a.T - t - r0;
    uint4 v[8];
    Value one[8];
#pragma unroll
    for (int b = 0; b < 8; b++) v[b] = *reinterpret_cast<const uint4*>(out + (4 * b + r0) * 128 + ((c ^ ((4 * b + r0) & 7)) << 4));
#pragma unroll
    for (int b = 0; b < 8; b++) one[b] = *reinterpret_cast<const Value*>(out + (4 * b + r0) * 128 + (((4 * b + r0) & 7) << 4) + c % kPiece * sizeof(Value));
    const size_t next = 8 * (size_t)a.N;
#pragma unroll
    for (int h = 0; h < 2; h++) {
        const int sr = turn(r0 + 4 * h), first = kPiece * c - sr;      // of the box's features
        const int at = c < sr ? kRow + c - sr : c - sr;
        const bool whole = first >= 0 && first + kPiece <= have, single = c < kPiece && sr > 0 && at < have;
        Value* y = (Value*)a.y + (size_t)(t + r0 + 4 * h) * a.N + n;
        Value *to = y + first, *end = y + at;
#pragma unroll
        for (int b = h; b < 8; b += 2, to += next, end += next) {
            if (whole && 4 * b < rows) *reinterpret_cast<uint4*>(to) = v[b];
            if (single && 4 * b < rows) *end = one[b];
        }
        if (first < 0 || first >= have || whole) continue;
        // the piece that y's last feature is in
        to = y + first;
#pragma unroll
        for (int b = h; b < 8; b += 2, to += next) {
            const uint32_t u[4] = {v[b].x, v[b].y, v[b].z, v[b].w};
#pragma unroll
            for (int k = 0; k < kPiece; k++)
                if (4 * b < rows && first + k < have) to[k] = (Value)(F32 ? u[k % 4] : u[k / 2 % 4] >> k % 2 * 16);
        }
    }
}

template <int F32>
__device__ __forceinline__ void store_box(const LinearArgs& a, const CUtensorMap* ymap, bool tma, uint8_t* out, int t, int n, int lane,
                                          const uint32_t (&w)[32])
{
    if (!tma) {
        store_rows<F32>(a, out, t, n, lane, w);
        return;
    }
    stage_box(out, lane, w);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) tma_store(ymap, n, t, out);
}

// The thread of the pair that issues for both CTAs.  (Little is computed between its
// instructions, as in linear.cu.)
template <int E2M1>
__device__ __forceinline__ bool multiply(const LinearArgs& a, Control& ctl, uint8_t* ring, uint32_t tmem, int steps, int first, int tiles, int stride)
{
    using S = Stage<E2M1>;
    constexpr uint32_t kUnit = kLinAtom / 16;
    const uint64_t ad0 = desc_sw128(smem_u32(ring)), sd0 = umma_desc(smem_u32(ring) + S::sfa, 16, 128);
    const uint32_t sf0 = tmem + kScaleCols;
    uint32_t slot = 0, parity = 0, cols = 0, it = 0;
    // the stage whose products are the last to read the scales' columns that come next
    uint32_t before = (uint32_t)kRing - S::slots, before_parity = 1;
    for (int i = first; i < tiles; i += stride, it++) {
        const uint32_t acc = tmem + (it & 1) * (kFeatures - kShared);
        for (int k = 0; k < steps; k++) {
            if (!mbar_wait_or_abort(&ctl.full[slot], parity, &ctl.abort, a.wait_ns)) return false;
            if (!mbar_wait_or_abort(&ctl.empty[before], before_parity, &ctl.abort, a.wait_ns)) return false;
            tc_fence_after();
            const uint64_t ad = ad0 + slot * (S::bytes / 16), sd = sd0 + slot * (S::bytes / 16);
            const uint32_t sfa = sf0 + cols, sfb = sfa + 4 * S::kAtoms;
#pragma unroll
            for (int h = 0; h < S::kAtoms; h++) cp_scales(sfa + 4 * h, sd + h * kUnit);
#pragma unroll
            for (int h = 0; h < 2 * S::kAtoms; h++) cp_scales(sfb + 4 * h, sd + (S::kAtoms + h) * kUnit);
            // the tile before has left the shared columns (and with them the one before it everything)
            if (k == 0 && it > 0 && !mbar_wait_or_abort(&ctl.acc_empty, (it - 1) & 1, &ctl.abort, a.wait_ns)) return false;
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const int h = E2M1 ? j / 2 : 0;
                mma<E2M1>(acc, ad + 2 * j, ad + S::b / 16 + 2 * j, idesc<E2M1>(E2M1 ? 2 * (j & 1) : j), sfa + 4 * h, sfb + 8 * h, k > 0 || j > 0);
            }
            commit_both(&ctl.empty[slot]);
            if (++slot == (uint32_t)kRing) {
                slot = 0;
                parity ^= 1;
            }
            if (++before == (uint32_t)kRing) {
                before = 0;
                before_parity ^= 1;
            }
            cols = cols + S::cols == (uint32_t)(S::slots * S::cols) ? 0 : cols + S::cols;
        }
        commit_both(&ctl.acc_full);
    }
    return true;
}

// The other CTA's: tells the first that its half of a stage is there.
template <int E2M1>
__device__ __forceinline__ bool relay(const LinearArgs& a, Control& ctl, int steps, int first, int tiles, int stride)
{
    uint32_t slot = 0, parity = 0;
    for (int i = first; i < tiles; i += stride)
        for (int k = 0; k < steps; k++) {
            if (!mbar_wait_or_abort(&ctl.full[slot], parity, &ctl.abort, a.wait_ns)) return false;
            arrive_at(&ctl.full[slot], 0);
            if (++slot == (uint32_t)kRing) {
                slot = 0;
                parity ^= 1;
            }
        }
    return true;
}

template <int E2M1, int F32>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    k_linear_pair(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                  const __grid_constant__ CUtensorMap ymap, LinearArgs a, int ftiles, int units, int tma)
{
    using S = Stage<E2M1>;
    extern __shared__ __align__(1024) uint8_t smem[];
    Control& ctl = *reinterpret_cast<Control*>(smem);
    uint8_t* ring = smem + sizeof(Control);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < kRing; s++) {
            mbar_init(&ctl.full[s], rank == 0 ? 3 : 2);     // copies, scales; the other CTA's full
            mbar_init(&ctl.empty[s], 1);
        }
        mbar_init(&ctl.acc_full, 1);
        mbar_init(&ctl.acc_empty, 8);
        mbar_init(&ctl.drain, 1);
        ctl.abort = 0;
        mbar_fence_init();
    }
    if (warp == kWarpProd && elect_one()) {
        prefetch_map(&wmap);
        prefetch_map(&xmap);
    }
    if (warp == kWarpMma) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ctl.tmem)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncwarp();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem;
    pdl_trigger();

    const int steps = E2M1 ? units : (a.K + 127) / 128;
    const int tiles = (int)((a.T + kTokens - 1LL) / kTokens) * ftiles, first = (int)blockIdx.x / 2, stride = (int)gridDim.x / 2;
    const int rtiles = (a.N + kLinRows - 1) / kLinRows;
    const int early = min(steps, kRing);        // stages whose weights come before the kernel ahead is done
    uint32_t c = 0, it = 0;

    if (warp == kWarpProd) {
        if (elect_one()) {
            bool ok = true, waited = false;
            for (int i = first; i < tiles && ok; i += stride) {
                const int f = i % ftiles, t0 = i / ftiles * kTokens + (int)rank * 128;
                // (a pair's second tile of weights may be behind the last: its features are not stored)
                const int w0 = min(2 * f, rtiles - 1) * units, w1 = min(2 * f + 1, rtiles - 1) * units;
                for (int k = 0; k < steps; k++, c++) {
                    const uint32_t slot = c % kRing;
                    if (k == early && !waited) {
                        pdl_wait();
                        waited = true;
                    }
                    if (!mbar_wait_or_abort(&ctl.empty[slot], (c / kRing & 1) ^ 1, &ctl.abort, a.wait_ns)) {
                        give_up(a, &ctl.abort);
                        ok = false;
                        break;
                    }
                    uint8_t* st = ring + slot * S::bytes;
                    uint64_t* bar = &ctl.full[slot];
                    const int u = E2M1 ? k : k / 2, half = E2M1 ? 0 : k & 1;
                    const uint32_t sf = S::kAtoms * kLinAtom;
                    // (expanded weights count as the bytes that were read)
                    mbar_arrive_expect_tx(bar, 128 * 128 + (E2M1 ? 128 * 128 : 128 * 64) + 2 * sf);
                    if (waited) tma_2d(st, &xmap, k * 128, t0, bar);        // (else the MMA's thread does)
                    tma_3d(st + S::b, &wmap, half * 128, 0, (rank ? w1 : w0) + u, bar);
                    const uint8_t* scales = a.packed + kLinCodeBytes + half * kLinAtom;
#pragma unroll
                    for (int h = 0; h < S::kAtoms; h++) {
                        // atom h of both tiles of weights, side by side
                        bulk_g2s(st + S::sfb + 2 * h * kLinAtom, scales + (size_t)(w0 + u) * kLinUnitBytes + h * kLinAtom, kLinAtom, bar);
                        bulk_g2s(st + S::sfb + (2 * h + 1) * kLinAtom, scales + (size_t)(w1 + u) * kLinUnitBytes + h * kLinAtom, kLinAtom, bar);
                    }
                }
                if (!waited) pdl_wait();
                waited = true;
            }
            for (uint32_t m = c > (uint32_t)kRing ? c - kRing : 0; m < c; m++)
                if (!mbar_wait_or_abort(&ctl.full[m % kRing], m / kRing & 1, &ctl.abort, a.wait_ns))
                    mbar_wait_bounded(&ctl.full[m % kRing], m / kRing & 1, a.wait_ns / 64);
        }
    } else if (warp == kWarpMma) {
        if (elect_one()) {
            // (their bytes may be there before the weights' thread expects them: it is its arrival
            // that the barrier's phase waits for)
            pdl_wait();
            for (int e = 0; e < early && first < tiles; e++)
                tma_2d(ring + e * S::bytes, &xmap, e * 128, first / ftiles * kTokens + (int)rank * 128, &ctl.full[e]);
            const bool ok = rank == 0 ? multiply<E2M1>(a, ctl, ring, tmem, steps, first, tiles, stride)
                                      : relay<E2M1>(a, ctl, steps, first, tiles, stride);
            if (!ok) {
                give_up(a, &ctl.abort);
                if (rank == 0) {
                    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(&ctl.drain)) : "memory");
                    mbar_wait_bounded(&ctl.drain, 0, a.wait_ns);
                }
            }
        }
    } else if (warp >= kWarpLoad) {
        pdl_wait();
        bool ok = true;
        for (int i = first; i < tiles && ok; i += stride) {
            const int t0 = i / ftiles * kTokens + (int)rank * 128;
            for (int k = 0; k < steps; k++, c++) {
                if (c % kLoadWarps != (uint32_t)(warp - kWarpLoad)) continue;
                const uint32_t slot = c % kRing;
                Scales<E2M1, 128> sc;
                sc.load(a, 128, t0, k, lane);
                ok = mbar_wait_or_abort(&ctl.empty[slot], (c / kRing & 1) ^ 1, &ctl.abort, a.wait_ns);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                sc.store(a, 128, t0, k, ring + slot * S::bytes + S::sfa, lane);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0 && !(a.withhold && blockIdx.x == 0 && k == 0)) mbar_arrive(&ctl.full[slot]);
            }
        }
        if (!ok && lane == 0) give_up(a, &ctl.abort);
    } else {
        pdl_wait();
        uint8_t* out = ring + kRing * S::bytes + warp * kOutBytes;
        for (int i = first; i < tiles; i += stride, it++) {
            const int n0 = i % ftiles * kFeatures;
            const int t = i / ftiles * kTokens + (int)rank * 128 + 32 * warp;
            bool ok = mbar_wait_or_abort(&ctl.acc_full, it & 1, &ctl.abort, a.wait_ns);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) {
                if (lane == 0) give_up(a, &ctl.abort);
                break;
            }
            tc_fence_after();
            const uint32_t from = tmem + (it & 1) * (kFeatures - kShared) + ((uint32_t)(32 * warp) << 16);
            // The shared columns lie in the first or the last of four groups of 64.
            const int g0 = it & 1 ? 0 : 3;
            for (int g = 0; g < 4; g++) {
                const int n = 64 * ((g + g0) & 3);
                uint32_t r[2][32];
                tc_ld32_nowait(from + n, r[0]);
                tc_ld32_nowait(from + n + 32, r[1]);
                tc_wait_ld();
                tc_ld_fence_regs<32>(r[0]);
                tc_ld_fence_regs<32>(r[1]);
                if (g == 0) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_at(&ctl.acc_empty, 0);
                }
                if (t >= a.T || n0 + n >= a.N) continue;
                if (F32) {
                    store_box<1>(a, &ymap, tma, out, t, n0 + n, lane, r[0]);
                    if (n0 + n + 32 < a.N) store_box<1>(a, &ymap, tma, out, t, n0 + n + 32, lane, r[1]);
                } else {
                    uint32_t w[32];
#pragma unroll
                    for (int j = 0; j < 32; j++)
                        w[j] = pack_bf16(__uint_as_float(r[j / 16][2 * j % 32]), __uint_as_float(r[j / 16][2 * j % 32 + 1]));
                    store_box<0>(a, &ymap, tma, out, t, n0 + n, lane, w);
                }
            }
            tc_fence_before();
        }
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    __syncwarp();
    tc_fence_before();
    cluster_meet();     // no product still reads the other's memory, and no arrival is on its way
    tc_fence_after();
    if (warp == kWarpMma) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

const void* kernel(bool e2m1, bool f32)
{
    return e2m1 ? (f32 ? (const void*)k_linear_pair<1, 1> : (const void*)k_linear_pair<1, 0>)
                : (f32 ? (const void*)k_linear_pair<0, 1> : (const void*)k_linear_pair<0, 0>);
}

}  // namespace

size_t linear_pair_smem(bool e2m1) { return sizeof(Control) + kRing * (e2m1 ? Stage<1>::bytes : Stage<0>::bytes) + 4 * kOutBytes; }

cudaError_t linear_pair_init_device(LinDevice& dev)
{
    for (int i = 0; i < 4; i++) {
        const cudaError_t e = cudaFuncSetAttribute(kernel(i & 1, i & 2), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)linear_pair_smem(i & 1));
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = linear_pair_smem(true);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(&dev.pairs, kernel(true, false), &cfg);
}

cudaError_t launch_linear_pair(const LinearArgs& a0, const LinDevice& dev, cudaStream_t s)
{
    LinearArgs a = a0;
    int units = lin_units(a.K), ftiles = (a.N + kFeatures - 1) / kFeatures;
    CUtensorMap wmap, xmap, ymap{};
    const cuuint64_t wd[3] = {a.e2m1 ? 128u : 256u, kLinRows, (cuuint64_t)lin_tiles(a.N) * units};
    const cuuint64_t ws[2] = {128, kLinUnitBytes};
    const cuuint32_t wb[3] = {128, kLinRows, 1};
    cudaError_t e = linear_map(&wmap, a.e2m1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 3, a.packed, wd, ws, wb);
    if (e != cudaSuccess) return e;
    const cuuint64_t width = a.e2m1 ? a.K / 2 : a.K;
    const cuuint64_t xd[2] = {width, (cuuint64_t)a.T}, xs[1] = {width};
    const cuuint32_t xb[2] = {128, 128};
    e = linear_map(&xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.codes, xd, xs, xb);
    if (e != cudaSuccess) return e;
    const cuuint64_t size = a.out_f32 ? 4 : 2;
    int tma = a.N * size % 16 == 0;
    if (tma) {
        const cuuint64_t yd[2] = {(cuuint64_t)a.N, (cuuint64_t)a.T}, ys[1] = {a.N * size};
        const cuuint32_t yb[2] = {(cuuint32_t)(128 / size), 32};
        e = linear_map(&ymap, a.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.y, yd, ys, yb);
        if (e != cudaSuccess) return e;
    }
    const long long tiles = (a.T + kTokens - 1LL) / kTokens * ftiles;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * std::min(tiles, (long long)dev.pairs)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = linear_pair_smem(a.e2m1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* args[] = {&wmap, &xmap, &ymap, &a, &ftiles, &units, &tma};
    return cudaLaunchKernelExC(&cfg, kernel(a.e2m1, a.out_f32), args);
}

}  // namespace moe
