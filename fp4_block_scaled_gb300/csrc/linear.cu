// linear.cu -- the product of rows in E2M1 or E4M3 with E2M1 weights, both with
// ue8m0 scales: y[t][n] = sum_k x[t][k] w[n][k], on block-scaled tcgen05.mma
// (kind::mxf4, K = 64 a step, or kind::mxf8f6f4, K = 32).
//
// A tile is 128 output features (the MMA's rows) by nt tokens (its columns, a
// multiple of 16).  A stage of the ring is 128 bytes of K of both operands, which TMA
// brings in the 128-byte swizzle that the MMA reads: 256 elements of E2M1, or 128 of
// E4M3, for which TMA expands the weights to a byte an element on their way (HBM and L2
// hold them packed).  Scales lie beside them as the atoms that tcgen05.cp moves; the
// weights' were packed so, the tokens' are gathered from their rows by warps of their own,
// or made there from a few tokens of bf16.
//
// Few tiles are cut along K between the CTAs of a cluster, which send one another their sums
// by bulk copies between their shared memories and add them in a fixed order: a join
// through global memory would cost a ticket's round trip more.
//
// Roles: warps 0-3 epilogue, 4 TMA, 5 MMA, 6-13 the tokens' scales.  The weights of a CTA's
// first stages are fetched before the kernel ahead has finished, its tokens after it.
//
// Bounds (GB300, in CUDA graphs of such products with other weights each): a single token by
// 4096 x 6144 in E2M1 takes 4.5 us where its 13.4 MB are 2.0 at the copy rate, 64 tokens by
// 4096 x 4096 in E4M3 6.8 from codes: the latencies of a start (dependency wait, tokens, first
// product: 0.9 us), of the stages (0.2 us each, or 2.2 to 2.8 cycles a row of a TMA box), of
// the sums' way to their CTA (0.7 us and more) and of the end.  What counted: operands of tcgen05
// instructions in uniform registers (elect.sync; with a lane chosen by its number each took 120
// cycles, not 40), scales loaded ahead of the wait for their slot, weights before the dependency
// wait and the first tokens by another thread beside them, no divisions in the roles' loops.  For
// many tokens pairs of CTAs (linear_pair.cu) are faster.
#include <math.h>

#include <algorithm>

#include "linear.cuh"

namespace moe {

namespace {

constexpr int kRing = 16;                  // stages, at most
constexpr int kMaxNt = 192;                // tokens of a tile, at most
constexpr int kSplitMax = kLinClusterMax;
constexpr int kWarpProd = 4, kWarpMma = 5, kWarpLoad = 6, kLoadWarps = 8;
constexpr int kThreads = (kWarpLoad + kLoadWarps) * 32;

struct __align__(1024) Control {
    uint64_t full[kRing], empty[kRing], acc_full[2], acc_empty[2], drain, red;
    uint32_t tmem;
    int abort;
};

struct Plan {
    int nt, ttiles, rtiles;     // token columns of a tile, tiles along T and N
    int steps;                  // stages along K
    int units;                  // of the packed weights along K
    int split;                  // CTAs along K
    int width;                  // columns that each of them sums
    int group, groups;          // CTAs whose columns leave together, and how many times
    int ring;
    // Warps that load scales, a stage each in turn: no more than the ring has stages, or a
    // warp could wait for a slot that is two rounds behind it, whose barrier has the parity
    // of the round that it waits for.
    int loaders;
    uint32_t b, sfa, sfb, stage;        // byte offsets in a stage, and its size
    uint32_t part;                      // byte offset of the partial sums
    uint32_t smem;
    int sfcols;                 // tensor memory columns of a stage's scales
    int tmem;                   // columns in all
    int acc;                    // column of the second accumulator (0: there is one)
};

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

// The tokens' scales into the atoms of every loaders-th stage, by one warp.
template <int E2M1>
__device__ __forceinline__ bool gather_scales(const LinearArgs& a, const Plan& p, Control& ctl, uint8_t* ring, int k0, int k1, int first, int tiles,
                                              int stride, int warp, int lane)
{
    if (warp >= p.loaders) return true;
    uint32_t slot = warp, parity = 1;
    int k = k0 + warp;
    for (int i = first; i < tiles; i += stride, k -= k1 - k0) {
        const int t0 = i / p.rtiles * p.nt;
        for (; k < k1; k += p.loaders) {
            Scales<E2M1, kMaxNt> sc;
            sc.load(a, p.nt, t0, k, lane);
            const bool ok = mbar_wait_or_abort(&ctl.empty[slot], parity, &ctl.abort, a.wait_ns);
            if (!__all_sync(0xFFFFFFFFu, ok)) return false;
            sc.store(a, p.nt, t0, k, ring + slot * p.stage + p.sfb, lane);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0 && !(a.withhold && blockIdx.x == 0 && k == 0)) mbar_arrive(&ctl.full[slot]);
            slot += p.loaders;
            if (slot >= (uint32_t)p.ring) {
                slot -= p.ring;
                parity ^= 1;
            }
        }
    }
    return true;
}

// Up to 16 token rows quantised from bf16 into the swizzled operand and the atoms, by eight
// warps: a turn is 256 elements of a stage, a row of E2M1 or two rows of E4M3, and a warp has
// one or two turns of every stage, or with few rows, of every second or fourth.
constexpr int kQuantRows = 16;
struct QuantShare {
    int rows, turns, stages;    // warps that share a stage's rows, turns of each, stages from one of its own to the next
    __host__ __device__ QuantShare(bool e2m1, int T, int ring)
    {
        const int all = e2m1 ? T : (T + 1) / 2;
        rows = all < kLoadWarps ? all : kLoadWarps;
        turns = (all + kLoadWarps - 1) / kLoadWarps;
        // (no more than the ring has, as for the scales' warps)
        stages = rows <= 2 && ring >= 4 ? 4 : rows <= 4 ? 2 : 1;
    }
};

template <int E2M1>
__device__ __forceinline__ bool quantise_rows(const LinearArgs& a, const Plan& p, Control& ctl, uint8_t* ring, int k0, int k1, int first, int tiles,
                                              int stride, int warp, int lane)
{
    constexpr int kBatch = 4;           // turns whose rows are loaded ahead
    const QuantShare share(E2M1, a.T, p.ring);
    const int w = warp % share.rows, turns = share.turns, l = E2M1 ? lane : lane % 16;
    if (warp >= share.rows * share.stages) return true;
    uint32_t slot = warp / share.rows, parity = 1;
    int from = k0 + (int)slot;
    for (int i = first; i < tiles; i += stride) {
        const int n = (k1 - from + share.stages - 1) / share.stages * turns;     // (0 or less: none)
        for (int u0 = 0; u0 < n; u0 += kBatch) {
            uint4 x[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; b++) {
                const int u = u0 + b, r = E2M1 ? w + (turns == 2 ? u & 1 : 0) * kLoadWarps : 2 * w + lane / 16;
                const int k = (from + (turns == 2 ? u >> 1 : u) * share.stages) * (E2M1 ? 256 : 128) + 8 * l;
                x[b] = make_uint4(0, 0, 0, 0);
                if (u < n && r < a.T && k < a.K) x[b] = *reinterpret_cast<const uint4*>(a.x + (size_t)r * a.K + k);
            }
#pragma unroll
            for (int b = 0; b < kBatch; b++) {
                const int u = u0 + b, half = turns == 2 ? u & 1 : 0, r = E2M1 ? w + half * kLoadWarps : 2 * w + lane / 16;
                if (u >= n) break;
                if (half == 0) {
                    const bool ok = mbar_wait_or_abort(&ctl.empty[slot], parity, &ctl.abort, a.wait_ns);
                    if (!__all_sync(0xFFFFFFFFu, ok)) return false;
                }
                uint8_t* st = ring + slot * p.stage;
                uint8_t* row = st + p.b + r * 128;
                uint8_t* atom = st + p.sfb + r * 16;
                int s;
                if (E2M1) {
                    const uint32_t c = e2m1_quantise(x[b], s);
                    if (r < a.T) {
                        *reinterpret_cast<uint32_t*>(row + ((l / 4 ^ (r & 7)) << 4) + l % 4 * 4) = c;
                        if (l % 4 == 0) atom[l / 16 * kLinAtom + l / 4 % 4] = (uint8_t)s;
                    }
                } else {
                    const uint2 c = e4m3_quantise(x[b], s);
                    if (r < a.T) {
                        *reinterpret_cast<uint2*>(row + ((l / 2 ^ (r & 7)) << 4) + l % 2 * 8) = c;
                        if (l == 0) *reinterpret_cast<uint32_t*>(atom) = (uint32_t)s * 0x01010101u;
                    }
                }
                if (half != turns - 1) continue;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0 && !(a.withhold && blockIdx.x == 0 && from == 0 && u < turns)) mbar_arrive(&ctl.full[slot]);
                slot += share.stages;
                if (slot >= (uint32_t)p.ring) {
                    slot -= p.ring;
                    parity ^= 1;
                }
            }
        }
        from += (n > 0 ? n / turns : 0) * share.stages - (k1 - k0);
    }
    return true;
}

// The MMA's thread: per stage the scales to tensor memory and four products.  Its
// instructions follow one another by few cycles only if little is computed between them:
// descriptors differ in their low words, by constants.  ATOMS: of 128 tokens' scales.
template <int E2M1, int ATOMS>
__device__ __forceinline__ bool multiply(const LinearArgs& a, const Plan& p, Control& ctl, uint8_t* ring, uint32_t tmem, int k0, int k1, int first,
                                         int tiles, int stride)
{
    constexpr int kHalves = E2M1 ? 2 : 1, kUnit = kLinAtom / 16;
    const uint64_t ad0 = desc_sw128(smem_u32(ring)), bd0 = ad0 + p.b / 16, sd0 = umma_desc(smem_u32(ring) + p.sfa, 16, 128);
    const uint32_t id = idesc<E2M1>(p.nt, 0), sf0 = tmem + p.nt + p.acc, stage = p.stage / 16, cols = p.sfcols;
    const int n = k1 - k0, depth = p.ring;
    uint32_t slot = 0, parity = 0, it = 0;
    for (int i = first; i < tiles; i += stride, it++) {
        const uint32_t buf = it & 1, acc = tmem + buf * p.acc;
        if (!mbar_wait_or_abort(&ctl.acc_empty[buf], (it >> 1 & 1) ^ 1, &ctl.abort, a.wait_ns)) return false;
        for (int k = 0; k < n; k++) {
            if (!mbar_wait_or_abort(&ctl.full[slot], parity, &ctl.abort, a.wait_ns)) return false;
            tc_fence_after();
            const uint64_t ad = ad0 + slot * stage, bd = bd0 + slot * stage, sd = sd0 + slot * stage;
            const uint32_t sfa = sf0 + slot * cols, sfb = sfa + 4 * kHalves;
#pragma unroll
            for (int h = 0; h < kHalves; h++) tc_cp_sf(sfa + 4 * h, sd + h * kUnit);
#pragma unroll
            for (int h = 0; h < kHalves * ATOMS; h++) tc_cp_sf(sfb + 4 * h, sd + (kHalves + h) * kUnit);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const uint32_t sf = E2M1 ? 2 * (j & 1) : j, h = E2M1 ? j / 2 : 0;
                mma<E2M1>(acc, ad + 2 * j, bd + 2 * j, id | (sf << 29) | (sf << 4), sfa + 4 * h, sfb + 4 * ATOMS * h, k > 0 || j > 0);
            }
            tc_commit(&ctl.empty[slot]);
            if (++slot == (uint32_t)depth) {
                slot = 0;
                parity ^= 1;
            }
        }
        tc_commit(&ctl.acc_full[buf]);
    }
    return true;
}

// QUANT: x is bf16, a few tokens, quantised here.
template <int E2M1, int QUANT>
__global__ void __launch_bounds__(kThreads, 2)
    k_linear(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap, LinearArgs a, Plan p)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    Control& ctl = *reinterpret_cast<Control*>(smem);
    uint8_t* ring = smem + sizeof(Control);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x < kRing) {
        mbar_init(&ctl.full[threadIdx.x], 1 + (QUANT ? QuantShare(E2M1, a.T, p.ring).rows : 1));
        mbar_init(&ctl.empty[threadIdx.x], 1);
        mbar_fence_init();
    } else if (threadIdx.x == 32) {
        for (int b = 0; b < 2; b++) {
            mbar_init(&ctl.acc_full[b], 1);
            mbar_init(&ctl.acc_empty[b], 4);
        }
        mbar_init(&ctl.drain, 1);
        mbar_init(&ctl.red, 1);
        ctl.abort = 0;
        mbar_fence_init();
    }
    if (warp == kWarpProd && elect_one()) {
        prefetch_map(&wmap);
        if (!QUANT) prefetch_map(&xmap);
    }
    if (warp == kWarpMma) tmem_alloc(&ctl.tmem, p.tmem);
    tc_fence_before();
    if (p.split > 1)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem;
    const uint32_t rank = p.split > 1 ? cluster_rank() : 0;
    const int k0 = p.steps * (int)rank / p.split, k1 = p.steps * ((int)rank + 1) / p.split;     // (at most 8192 stages)
    const int tiles = p.ttiles * p.rtiles, first = (int)blockIdx.x / p.split, stride = (int)gridDim.x / p.split;
    const int early = min(k1 - k0, p.ring);     // stages whose weights come first
    uint32_t c = 0, it = 0;
    pdl_trigger();
    if (warp == kWarpProd) {
        if (elect_one()) {
            bool ok = true, waited = false;
            uint32_t slot = 0, parity = 1;
            for (int i = first; i < tiles && ok; i += stride) {
                const int rt = i % p.rtiles, t0 = i / p.rtiles * p.nt;
                const uint8_t* scales = a.packed + (size_t)rt * p.units * kLinUnitBytes + kLinCodeBytes;
                // The weights of as many stages as there are come while the kernel before this
                // one still runs; their tokens the MMA's thread fetches after it.
                if (!waited)
                    for (int k = k0 + early; k < k1; k += E2M1 ? 1 : 2)
                        prefetch_l2(scales - kLinCodeBytes + (size_t)(E2M1 ? k : k / 2) * kLinUnitBytes, kLinUnitBytes);
                for (int k = k0; k < k1; k++, c++) {
                    if (k == k0 + early && !waited) {
                        pdl_wait();
                        waited = true;
                    }
                    if (!mbar_wait_or_abort(&ctl.empty[slot], parity, &ctl.abort, a.wait_ns)) {
                        give_up(a, &ctl.abort);
                        ok = false;
                        break;
                    }
                    uint8_t* st = ring + slot * p.stage;
                    uint64_t* bar = &ctl.full[slot];
                    const int u = E2M1 ? k : k / 2, half = E2M1 ? 0 : k & 1;
                    const uint32_t sf = E2M1 ? 2 * kLinAtom : kLinAtom;
                    // (expanded weights count as the bytes that were read)
                    mbar_arrive_expect_tx(bar, (E2M1 ? kLinCodeBytes : kLinCodeBytes / 2) + sf + (QUANT ? 0 : p.nt * 128));
                    tma_3d(st, &wmap, half * 128, 0, rt * p.units + u, bar);
                    bulk_g2s(st + p.sfa, scales + (size_t)u * kLinUnitBytes + half * kLinAtom, sf, bar);
                    if (!QUANT && waited) tma_2d(st + p.b, &xmap, k * 128, t0, bar);
                    if (++slot == (uint32_t)p.ring) {
                        slot = 0;
                        parity ^= 1;
                    }
                }
                if (!waited) pdl_wait();
                waited = true;
            }
            // no copy may be in flight into this CTA's memory at its end
            for (uint32_t m = c > (uint32_t)p.ring ? c - p.ring : 0; m < c; m++)
                if (!mbar_wait_or_abort(&ctl.full[m % p.ring], m / p.ring & 1, &ctl.abort, a.wait_ns))
                    mbar_wait_bounded(&ctl.full[m % p.ring], m / p.ring & 1, a.wait_ns / 64);
        }
    } else if (warp == kWarpMma) {
        if (elect_one()) {
            pdl_wait();     // (no limit runs while the kernel ahead does)
            if (!QUANT) {
                // (their bytes may be there before the weights' thread expects them: it is its
                // arrival that the barrier's phase waits for)
                for (int e = 0; e < early && first < tiles; e++)
                    tma_2d(ring + e * p.stage + p.b, &xmap, (k0 + e) * 128, first / p.rtiles * p.nt, &ctl.full[e]);
            }
            const bool ok = p.nt > 128 ? multiply<E2M1, 2>(a, p, ctl, ring, tmem, k0, k1, first, tiles, stride)
                                       : multiply<E2M1, 1>(a, p, ctl, ring, tmem, k0, k1, first, tiles, stride);
            if (!ok) {
                // (else the epilogue has waited for the last product)
                give_up(a, &ctl.abort);
                tc_commit(&ctl.drain);
                mbar_wait_bounded(&ctl.drain, 0, a.wait_ns);
            }
        }
    } else if (warp >= kWarpLoad) {
        pdl_wait();
        const bool ok = QUANT ? quantise_rows<E2M1>(a, p, ctl, ring, k0, k1, first, tiles, stride, warp - kWarpLoad, lane)
                              : gather_scales<E2M1>(a, p, ctl, ring, k0, k1, first, tiles, stride, warp - kWarpLoad, lane);
        if (!ok && lane == 0) give_up(a, &ctl.abort);
    } else {
        pdl_wait();
        for (int i = first; i < tiles; i += stride, it++) {
            const long long t0 = (long long)(i / p.rtiles) * p.nt, n = (long long)(i % p.rtiles) * kLinRows + 32 * warp + lane;
            const uint32_t buf = it & 1;
            bool ok = mbar_wait_or_abort(&ctl.acc_full[buf], it >> 1 & 1, &ctl.abort, a.wait_ns);
            // (the warps of a split tile meet below: all of them go on, or none)
            ok = p.split > 1 ? all_of(1, 128, ok) : __all_sync(0xFFFFFFFFu, ok);
            if (!ok) {
                if (lane == 0) give_up(a, &ctl.abort);
                break;
            }
            tc_fence_after();
            const int cols = (int)min((long long)p.nt, a.T - t0);
            const uint32_t from = tmem + buf * p.acc + ((uint32_t)(32 * warp) << 16);
            if (p.split > 1) {
                // CTA o adds up the columns o * width ..: every CTA sends it its own sums of them, by
                // way of its ring, which is free (every product is done), 32 columns or an owner's
                // at a time and its neighbour's first, so that copies and reads overlap.
                const int own = min(p.width, cols - (int)rank * p.width);
                if (warp == 0 && own > 0 && elect_one()) mbar_arrive_expect_tx(&ctl.red, p.split * own * kLinRows * 4);
                float* mine = reinterpret_cast<float*>(ring) + 32 * warp + lane;
                int turn = p.groups == 1 ? 0 : (int)rank / p.group;
                for (int d = 0; d < p.groups; d++) {
                    if (++turn >= p.groups) turn = 0;
                    const int o0 = turn * p.group, c1 = min(min(o0 + p.group, p.split) * p.width, cols);
                    if (o0 * p.width >= c1) continue;
                    for (int c0 = o0 * p.width; c0 < c1; c0 += 32) {
                        uint32_t r[2][16];
                        const int have = c1 - c0;
                        tc_ld16_nowait(from + c0, r[0]);
                        if (have > 16) tc_ld16_nowait(from + c0 + 16, r[1]);
                        tc_wait_ld();
                        tc_ld_fence_regs<16>(r[0]);
                        tc_ld_fence_regs<16>(r[1]);
#pragma unroll
                        for (int j = 0; j < 32; j++)
                            if (j < have) mine[(c0 + j) * kLinRows] = __uint_as_float(r[j / 16][j % 16]);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    named_sync(1, 128);
                    if (warp == 0 && elect_one())
                        for (int o = o0; o * p.width < c1; o++)
                            bulk_to_peer(smem_u32(smem + p.part) + rank * p.width * kLinRows * 4, smem_u32(ring) + o * p.width * kLinRows * 4,
                                         min(p.width, c1 - o * p.width) * kLinRows * 4, smem_u32(&ctl.red), o);
                }
            } else {
                // (a store a token: little is computed between them)
                const size_t size = a.out_f32 ? 4 : 2, next = a.N * size;
                uint8_t* to = (uint8_t*)a.y + ((size_t)t0 * a.N + n) * size;
                for (int c0 = 0; c0 < cols; c0 += 16) {
                    uint32_t r[16];
                    tc_ld16_nowait(from + c0, r);
                    tc_wait_ld();
                    tc_ld_fence_regs<16>(r);
                    if (n >= a.N) continue;
                    if (a.out_f32) {
#pragma unroll
                        for (int j = 0; j < 16; j++, to += next)
                            if (j < cols - c0) *reinterpret_cast<uint32_t*>(to) = r[j];
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; j++, to += next)
                            if (j < cols - c0) *reinterpret_cast<__nv_bfloat16*>(to) = __float2bfloat16_rn(__uint_as_float(r[j]));
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
        // One tile a cluster: its CTAs' sums are added in their order.
        const long long t0 = (long long)(first / p.rtiles) * p.nt, n0 = (long long)(first % p.rtiles) * kLinRows + 4 * lane;
        const int cols = (int)min((long long)p.nt, a.T - t0), here = min(p.width, cols - (int)rank * p.width);
        // (the producer's and the MMA's warps have no part in it)
        const int adder = warp < 4 ? warp : warp - 2, adders = 4 + kLoadWarps;
        if (here > adder && (warp < 4 || warp >= kWarpLoad)) {
            const bool ok = mbar_wait_bounded(&ctl.red, 0, a.wait_ns);
            if (!ok) give_up(a, &ctl.abort);
            const float4* part = reinterpret_cast<const float4*>(smem + p.part) + lane;
            for (int j = adder; j < here && ok; j += adders) {
                float4 w[kSplitMax], v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int r = 0; r < kSplitMax; r++)
                    if (r < p.split) w[r] = part[(r * p.width + j) * (kLinRows / 4)];
#pragma unroll
                for (int r = 0; r < kSplitMax; r++)
                    if (r < p.split) {
                        v.x += w[r].x;
                        v.y += w[r].y;
                        v.z += w[r].z;
                        v.w += w[r].w;
                    }
                store4(a, t0 + rank * p.width + j, n0, v);
            }
        }
        __syncwarp();
        cluster_meet();     // nobody's memory is still read
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWarpMma) tmem_dealloc(tmem, p.tmem);
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
// The driver's encoder of tensor maps, asked for once in a process; null if it has none.
EncodeTiled encoder()
{
    static const EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult got;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12080, cudaEnableDefault, &got);
        return e == cudaSuccess && got == cudaDriverEntryPointSuccess ? (EncodeTiled)p : (EncodeTiled) nullptr;
    }();
    return fn;
}

// Shared memory of an SM, and of it what each CTA takes beyond its own.
constexpr uint32_t kSmShared = 228 * 1024, kCtaReserved = 1024;
static_assert(kSmShared - kCtaReserved == kLinSmemMax, "a CTA with every column takes all of it");

long long tiles_of(const Plan& p) { return (long long)p.ttiles * p.rtiles; }

// Time of a product in microseconds, fitted to what was measured in CUDA graphs of products one
// after the other (K = 96 .. 8192, N = 300 .. 8192, T = 1 .. 3840): a start and end of 3.4, the
// longer of a CTA's stages (0.215, or 2.2 to 2.8 cycles a row of its TMA boxes) and of what all of
// them fetch through L2, and the output.  That is 0.006 a token of a single tile, 0.02 a token
// where CTAs send their sums to one another, and 0.5 and 0.0085 a token, a store each, beside
// the next tile's stages: what is longer of the two, and 0.3 of the other.
double tile_cost(const LinearArgs& a, const LinDevice& dev, const Plan& p)
{
    const long long tiles = tiles_of(p);
    const double waves = p.split > 1 ? 1.0 : (double)((tiles + dev.sms - 1) / dev.sms);
    const double stage = std::max(0.215, (kLinRows + p.nt) * (a.e2m1 ? 0.00145 : 0.00113));
    const double serial = ((p.steps + p.split - 1) / p.split) * stage, output = 0.5 + 0.0085 * p.nt;
    const double feed = (double)tiles * p.steps * ((a.e2m1 ? 17408 : 8704) + p.nt * 132) * 0.77e-7;
    if (p.split > 1) return 3.4 + std::max(serial, feed) + 0.02 * p.nt;
    if (waves == 1.0) return 3.4 + std::max(serial, feed) + 0.006 * p.nt;
    return 3.4 + std::max(waves * (std::max(serial, output) + 0.3 * std::min(serial, output)), feed);
}

// And of one on pairs of CTAs: 0.365 (E4M3 0.3) a stage and what of a tile's output does not
// overlap with them, or the output's time where that is longer.
double pair_cost(const LinearArgs& a, const LinDevice& dev, int steps)
{
    const double tiles = (double)((a.T + 255) / 256) * ((a.N + 255) / 256), waves = ceil(tiles / std::max(1, dev.pairs));
    const bool rows = a.N % (a.out_f32 ? 4 : 8) != 0;      // without TMA
    const double more = a.out_f32 ? (rows ? 2.0 : 0.5) : rows ? 1.0 : 0.0, output = a.out_f32 ? (rows ? 4.6 : 3.4) : rows ? 2.4 : 1.7;
    return 4.2 + waves * std::max(steps * (a.e2m1 ? 0.365 : 0.3) + more, output);
}

// Shared and tensor memory of a plan whose tile and split are set; false if it has no room.
bool lay_out(const LinearArgs& a, const LinDevice& dev, Plan& p)
{
    const int sf = p.nt > 128 ? 2 : 1, h = a.e2m1 ? 2 : 1, slice = (p.steps + p.split - 1) / p.split;
    p.b = kLinCodeBytes;
    p.sfa = p.b + p.nt * 128;
    p.sfb = p.sfa + h * kLinAtom;
    p.stage = (p.sfb + h * sf * kLinAtom + 1023) / 1024 * 1024;
    p.width = (p.nt + p.split - 1) / p.split;
    p.group = std::max(1, 32 / p.width);
    p.groups = (p.split + p.group - 1) / p.group;
    p.sfcols = 4 * h * (1 + sf);
    const uint32_t part = p.split > 1 ? p.split * p.width * kLinRows * 4 : 0, fixed = sizeof(Control) + part;
    const bool one = p.split > 1 || tiles_of(p) <= dev.sms;       // a CTA has one tile
    p.acc = one ? 0 : p.nt;
    p.ring = std::min({kRing, (int)((kLinSmemMax - fixed) / p.stage), (512 - p.nt - p.acc) / p.sfcols, one ? std::max(slice, 3) : kRing});
    // Where four stages fit half an SM and a CTA has no more than twice its stages, two CTAs share
    // one, so that a kernel can begin beside the one before it, each with at most half of the tensor
    // memory (one token by 4096 x 6144 6.5 us, before 6.8; their registers allow no third).  Else a
    // CTA has more than half of the shared memory, as its ring is made for.
    const int two = fixed < kLinSmemTwo ? (int)((kLinSmemTwo - fixed) / p.stage) : 0;
    const bool share = one && two >= 4 && slice <= 2 * two && p.nt + std::min(p.ring, two) * p.sfcols <= 256;
    if (share) p.ring = std::min(p.ring, two);
    p.loaders = std::min(kLoadWarps, p.ring);
    p.part = sizeof(Control) + p.ring * p.stage;
    p.smem = share ? p.part + part : std::max(p.part + part, kLinSmemMax / 2 + 4096);
    p.tmem = 32;
    while (p.tmem < p.nt + p.acc + p.ring * p.sfcols) p.tmem *= 2;
    // CTAs of a cluster wait for each other's tensor memory without a limit of time, and those of
    // products on two streams may meet on an SM: none of them may hold columns that another one
    // beside it lacks.  So each takes at least the share of the SM's shared memory that it takes of
    // its 512 columns, and what fits the one fits the other.  (CTAs without a cluster wait for
    // nobody that could wait for their columns.)
    if (p.split > 1) p.smem = std::max(p.smem, (uint32_t)((unsigned long long)kSmShared * p.tmem / 512 - kCtaReserved));
    // a split tile's sums are laid down in the ring
    return p.ring >= 3 && (p.split == 1 || p.ring * p.stage >= (uint32_t)p.nt * kLinRows * 4);
}

// The cheapest tile and split; no tile (nt = 0) where pairs of CTAs are cheaper.
Plan make_plan(const LinearArgs& a, const LinDevice& dev)
{
    Plan p{};
    p.rtiles = lin_tiles(a.N);
    p.steps = a.e2m1 ? lin_units(a.K) : (a.K + 127) / 128;
    p.units = lin_units(a.K);
    Plan best = p;
    double least = a.codes && a.T > 64 ? pair_cost(a, dev, p.steps) : HUGE_VAL;
    // Codes of more than 4096 tokens go to the pairs alone, which cut no K, so that there a feature's
    // sums are the same whatever T and N.  That costs time where tiles of 256 x 256 fit the sizes badly:
    // with tiles of one CTA looked at too, 216 products of 4200 to 16384 tokens by 24 to 4096 features
    // took from 0.59 (5000 by 256 x 1024 in E4M3 to fp32 10.2 us, so 6.0) to 1.21 (4200 by 4096 x 1024
    // 16.7, so 20.2) of theirs.
    const int widest = a.codes && a.T > 4096 ? 0 : std::min(kMaxNt, (a.T + 15) / 16 * 16);
    for (p.nt = widest; p.nt > 0; p.nt -= 16) {
        const int ttiles = (a.T + p.nt - 1) / p.nt;
        if (ttiles == p.ttiles) continue;
        p.ttiles = ttiles;
        Plan q = p;
        q.nt = ((a.T + ttiles - 1) / ttiles + 15) / 16 * 16;    // no more than so many tiles need
        const long long tiles = tiles_of(q);
        for (q.split = 1; q.split <= std::min(kSplitMax, q.steps); q.split++) {
            if (q.split > 1 && tiles * q.split > dev.sms) break;
            const double cost = tile_cost(a, dev, q);
            if (cost >= least || !lay_out(a, dev, q)) continue;
            // The clusters of a cut run at once: two CTAs an SM only where they share one (one token by
            // 4096 x 6144 in E4M3 from codes: 48 clusters of three, of which 46 ran, 11.8 us; so of two, 7.2).
            if (q.split > 1 && tiles > (long long)dev.clusters[q.split] * (q.smem <= kLinSmemTwo ? 2 : 1)) continue;
            least = cost;
            best = q;
        }
        if (tiles > 8 * dev.sms) break;
    }
    return best;
}

}  // namespace

cudaError_t linear_map(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* base, const cuuint64_t* dims,
                       const cuuint64_t* strides, const cuuint32_t* box)
{
    const cuuint32_t ones[3] = {1, 1, 1};
    return encoder()(map, type, (cuuint32_t)rank, (void*)base, dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

const void* const kKernels[4] = {(const void*)k_linear<0, 0>, (const void*)k_linear<1, 0>, (const void*)k_linear<0, 1>,
                                 (const void*)k_linear<1, 1>};

bool linear_takes_bf16(const LinearArgs& a0, const LinDevice& dev)
{
    // Every CTA quantises its slice of K, so that a kernel ahead, at 1.3 us and a launch, is saved
    // where a warp has few turns (16 rows, two stages a CTA 4.2 us, before 5.0; eight rows, six
    // stages 6.4, before 6.2; 16 rows in E2M1, six stages 8.4, before 6.5).
    if (a0.T > kQuantRows) return false;
    LinearArgs a = a0;
    a.codes = nullptr;
    const Plan p = make_plan(a, dev);
    const QuantShare q(a.e2m1, a.T, p.ring);
    return (p.steps + p.split - 1) / p.split * q.turns <= 6 * q.stages;
}

cudaError_t linear_init_device(LinDevice& dev)
{
    if (!encoder()) return cudaErrorNotSupported;
    for (const void* fn : kKernels) {
        const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kLinSmemMax);
        if (e != cudaSuccess) return e;
    }
    for (int split = 2; split <= kSplitMax; split++) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)split);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kLinSmemMax;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)split;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        const cudaError_t e = cudaOccupancyMaxActiveClusters(&dev.clusters[split], kKernels[0], &cfg);
        if (e != cudaSuccess) return e;
    }
    return linear_pair_init_device(dev);
}

void linear_plan(const LinearArgs& a, const LinDevice& dev, moe_lin_test_plan_t* plan)
{
    const Plan p = make_plan(a, dev);
    *plan = p.nt == 0 ? moe_lin_test_plan_t{0, 0, 0, 0, (int)linear_pair_smem(a.e2m1), 512}
                      : moe_lin_test_plan_t{p.nt, p.ttiles * p.rtiles, p.split, p.ring, (int)p.smem, p.tmem};
}

cudaError_t launch_linear(const LinearArgs& a0, const LinDevice& dev, cudaStream_t s)
{
    LinearArgs a = a0;
    Plan p = make_plan(a, dev);
    if (p.nt == 0) return launch_linear_pair(a, dev, s);
    CUtensorMap wmap, xmap{};
    const cuuint64_t wd[3] = {a.e2m1 ? 128u : 256u, kLinRows, (cuuint64_t)p.rtiles * p.units};
    const cuuint64_t ws[2] = {128, kLinUnitBytes};
    const cuuint32_t wb[3] = {128, kLinRows, 1};
    cudaError_t e = linear_map(&wmap, a.e2m1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 3, a.packed, wd, ws, wb);
    if (e != cudaSuccess) return e;
    const cuuint64_t width = a.e2m1 ? a.K / 2 : a.K;
    const cuuint64_t xd[2] = {width, (cuuint64_t)a.T}, xs[1] = {width};
    const cuuint32_t xb[2] = {128, (cuuint32_t)p.nt};
    if (a.codes) e = linear_map(&xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.codes, xd, xs, xb);
    if (e != cudaSuccess) return e;
    const long long tiles = (long long)p.ttiles * p.rtiles;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.split > 1 ? tiles * p.split : std::min(tiles, (long long)dev.sms)));
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
    return cudaLaunchKernelExC(&cfg, kKernels[(a.codes ? 0 : 2) + a.e2m1], args);
}

}  // namespace moe
