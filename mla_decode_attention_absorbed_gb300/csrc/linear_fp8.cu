// out = residual + act(x . W^T + bias) of E4M3 codes with a scale for each 128 values of a row of x
// and for each 128 x 128 values of W, on the 5th-generation tensor cores (tcgen05, kind::f8f6f4).
//
// With block b of K holding the values [128 b, 128 b + 128),
//   sum_k x[m, k] W[n, k] = sum_b sx[b, m] sw[n / 128, b] sum_{k in b} cx[m, k] cw[n, k],
// so the tensor cores' sum ends with each block: block b's product of the codes goes to one of two
// accumulators in tensor memory, and while the MMAs fill the other one, eight warps take it from
// there, times its scale, into the tile's fp32 sums, which stay in their registers.  The MMA's rows
// are the tokens and its columns those of the output: a lane then has one token, a warp's columns lie
// in one block of W (of a tile of 192 in one or two), and a value costs half an instruction (two fp32 multiply-adds each).
//
// A tile is 128 tokens x 64 or 128 columns on one CTA, or 256 x 192 or 256 on a pair of CTAs, each of
// which loads half of both operands and holds the sums of its 128 tokens.  K runs in blocks of 128
// through a ring of TMA stages.  The CTAs take whole tiles one after another; of a tile that is left (or of
// all, where there are few) the 2, 4 or 8 CTAs or pairs of a cluster take equal parts of K, exchange their
// sums through distributed shared memory and finish a share of the columns each.  Parts are added in the
// order of K, so results do not depend on timing.
//
// Warps: 0 issues the loads, 1 the MMAs, 2 moves residuals in and outputs out, 4-11 hold the sums.
//
// Measured (device time): 4096 x 16384 x 7168 in 320 to 330 us for a dozen calls = 2,900 to 3,000 TFLOP/s, 1.5
// times the measured bf16 rate (370 us = 2,600 in a long run of them, at the power limit): a block of a pair's
// tile takes 800 cycles where its MMAs alone take 560.  Copies of the kernel without one part or another: MMAs alone 226 us,
// loads alone 203, sums alone 270, loads and MMAs 269 (what comes in and what the MMAs read share the shared memory's
// ports), MMAs and sums 295, handshakes alone 166.  64 x 16384 x 7168 in 26.3 us: 117 MB of weights at 6.1 TB/s in 19 us,
// 2.7 of start and 4 of the wait for the other CTA, exchange and finish.  256 x 7168 x 24576 in 51 us, 333 x 1008 x 1544 in 6.4, a chain of latencies.
//
// What measured slower: arrivals across the pair that order memory (875 us when this took 488), clocks read
// before each wait, an epilogue turned over through shared memory (8 us a tile: 468), the scales' addresses
// worked out block by block (438), a commit for the sums and one for the stage (335 us, so 321), a block's sums in two
// halves with a commit each (336), waits of the sums' warps that poll (326).
#include <limits.h>

#include <atomic>

#include "layer.h"
#include "linear_common.cuh"
#include "tmap.h"

namespace mla {
namespace {

using namespace sm100;
using namespace product;

constexpr int kRows = 128;  // tokens a CTA
constexpr int kBK = 128;    // values, and bytes, of K a stage: a block
constexpr int kThreads = 384;
constexpr int kSumWarps = 8;  // two for each quarter of the tokens, half of the columns each
constexpr int kFirstSum = 4;  // the first of them
// Registers: the launch's 384 x 168 are dealt out anew, 128 of them a lane for the sums alone.
constexpr int kRegSum = 216, kRegOther = 72;
static_assert(2 * kRegSum + kRegOther == 3 * 168, "the split must equal the launch's total");

template <int kValue>
struct Value {
    static constexpr int value = kValue;
};

using Plan = LinearFp8Plan;

template <int kCols, bool kPair>
struct Smem {
    static constexpr int kXBytes = kRows * kBK;
    static constexpr int kWBytes = (kPair ? kCols / 2 : kCols) * kBK;
    static constexpr int kStage = kXBytes + kWBytes;
    static constexpr int kTile = kRows * kCols * 2;  // the output's tile: slabs of 64 columns, 128 bytes a token
    static constexpr int kStages = (227 * 1024 - 2048 - kTile) / kStage;
    static constexpr int kBytes = kStages * kStage + kTile + 1024 /* barriers */ + 1024 /* alignment */;
    static constexpr int kBufs = 512 / kCols;  // accumulators: a block of K each
    static constexpr int kWide = kCols / 2;    // columns of a warp's sums
    static constexpr bool kTwo = kBK % kWide != 0;  // which may lie in two blocks of W
    static_assert(kRows * kCols * 4 <= kStages * kStage, "a cluster's sums are exchanged in the ring");
    static_assert(kStages >= kBufs, "a stage's barrier tells the sums' warps, too, see the MMA warp");
    static_assert(kBytes <= 232448, "shared memory over the per-CTA limit");
};

// Instruction descriptor of kind::f8f6f4 with E4M3 A and B (formats 0), both K-major, fp32 D.
constexpr uint32_t idesc_e4m3(int M, int N) { return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24); }

template <bool kPair>
__device__ __forceinline__ void mma_codes(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    if (kPair)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
}

// Waits for the tensor-memory loads issued so far; r passes through it, so that no use of the
// loaded values can be moved before it.
__device__ __forceinline__ void tmem_ld_wait16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void fma2(float &a, float &b, uint32_t x, uint32_t y, float s) {
    asm("{\n\t.reg .b64 p, q, r;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\tmov.b64 r, {%4, %4};\n\tfma.rn.f32x2 p, q, r, p;\n\tmov.b64 {%0, %1}, p;\n\t}" : "+f"(a), "+f"(b) : "r"(x), "r"(y), "f"(s));
}
// sums *= f, a power of two.
template <int kWide>
__device__ __forceinline__ void times(float (&sums)[kWide], float f) {
    const float2 both = make_float2(f, f);
#pragma unroll
    for (int e = 0; e < kWide; e += 2) {
        const float2 p = mul2(make_float2(sums[e], sums[e + 1]), both);
        sums[e] = p.x;
        sums[e + 1] = p.y;
    }
}
// sums += scale * the kWide columns of tensor memory at taddr; the next 16 are on their way
// while 16 are added.  Columns from `before` on, a multiple of 32, are in the next block of W: scale2.
template <int kWide>
__device__ __forceinline__ void add_block(float (&sums)[kWide], uint32_t taddr, float scale1, float scale2, int before) {
    uint32_t r0[16], r1[16];
    tmem_ld16(taddr, r0);
#pragma unroll
    for (int c = 0; c < kWide; c += 32) {
        const float scale = c < before ? scale1 : scale2;
        tmem_ld_wait16(r0);
        tmem_ld16(taddr + c + 16, r1);
#pragma unroll
        for (int e = 0; e < 16; e += 2) fma2(sums[c + e], sums[c + e + 1], r0[e], r0[e + 1], scale);
        tmem_ld_wait16(r1);
        if (c + 32 < kWide) tmem_ld16(taddr + c + 32, r0);
#pragma unroll
        for (int e = 0; e < 16; e += 2) fma2(sums[c + 16 + e], sums[c + 17 + e], r1[e], r1[e + 1], scale);
    }
}

// The epilogue of 32 columns of a token, from its fp32 sums: `row` is the token's row of the slab
// that holds them (16-byte chunk c at c ^ swz), with the residual in it if there is one; the result
// takes its place.  n: the first column; columns at N and behind are not stored.
template <int kAct>
__device__ __forceinline__ void finish_columns(const LinearArgs &a, const float *sums, uint8_t *row, int first_chunk, int swz,
                                               int n) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        uint4 *at = reinterpret_cast<uint4 *>(row + (((first_chunk + g) ^ swz) << 4));
        float y[8], f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = sums[8 * g + e];
        if (a.bias && n + 8 * g < a.N) {
            Finish::unpack8(__ldg(reinterpret_cast<const uint4 *>(a.bias + n + 8 * g)), f);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] += f[e];
        }
        activate_all<kAct>(y);
        if (a.residual) {
            Finish::unpack8(*at, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] += f[e];
        }
        *at = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
    }
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, float a, float b, float c, float d) {
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *m, const void *src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(m)),
                 "r"(smem_u32(src)), "r"(x), "r"(y)
                 : "memory");
}

// "The accumulator was taken", across the pair.  Nothing in memory goes with it (what was read is in
// registers), so neither side orders memory: an arrival that does waits for all that the warp has under
// way (.release.cluster: 4096 x 16384 x 7168 875 us, without 488).
__device__ __forceinline__ void arrive_taken(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// Whether a phase is over: at once, or after the hardware's own short wait for it (which lasts longer than
// a limit of microseconds).  kCluster: of a barrier that arrive_taken arrives on.
template <bool kCluster>
__device__ __forceinline__ bool is_over(uint64_t *bar, uint32_t parity, bool at_once) {
    if (!kCluster) return at_once ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity);
    uint32_t ok;
    if (at_once)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.test_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
    return ok != 0;
}
// A whole warp's wait for work (see Patience), unless it is `done` already.  The clocks are read only
// once a first try has not been enough (read before it, as by warp_wait, they were part of every block's
// time).
template <bool kCluster = false>
__device__ __forceinline__ bool wait_for(bool done, uint64_t *bar, uint32_t parity, const Patience &p) {
    const bool at_once = p.ns < 1000000;
    if (__all_sync(~0u, done || is_over<kCluster>(bar, parity, at_once))) return true;
    const uint64_t t0 = globaltimer_ns();
    const long long c0 = clock64();
    for (uint32_t it = 0;; ++it) {
        if (__all_sync(~0u, is_over<kCluster>(bar, parity, at_once))) return true;
        if ((it & 15u) == 0 && __any_sync(~0u, p.over(t0, c0))) {
            *p.abort_flag = 1;
            return false;
        }
    }
}

// For what comes once the waits for work have ended, one way or the other (a whole warp); not if *lost.
__device__ __forceinline__ bool wait_beyond(uint64_t *bar, uint32_t parity, uint64_t wait_ns, volatile int *lost) {
    const uint64_t t0 = globaltimer_ns(), ns = wait_ns + 2 * kWaitLimitNs;
    const long long c0 = clock64();
    while (!__all_sync(~0u, mbar_try_wait(bar, parity)))
        if (__any_sync(~0u, *lost || globaltimer_ns() - t0 > ns || clock64() - c0 > (long long)(2 * ns))) return false;
    return !__any_sync(~0u, *lost);
}

// A CTA's work (a pair's, "unit"): whole tiles, then, for a cluster's units together, a share of one
// tile's K.
struct Segment {
    int m, n, k0, k1;  // m, n: the tile's place
    bool cut;
};
// The tiles go column by column through a band of this many tiles of tokens: the band's x stays in L2 while
// W passes.  4096 x 16384 x 7168 in a long run of calls 372 to 375 us, through all 16 tiles of tokens 380, through bands of 4 383.
constexpr int kBand = 8;
// A lane's sums and a block's scale x_scale * w_scale are held times kLift, so that a small scale keeps its bits: a
// block's codes sum to up to 128 * 448^2 < 2^25, and 2^25 times a scale below the normal numbers is one.  A
// lane that meets a scale past kMostLifted, held so (or an x_scale that passes fp32 so), puts its sums down for the rest of the tile (2^80 * 2^25
// in 2^13 blocks stays finite).  4096 x 16384 x 7168 321 us, without 319; 4096 x 512 x 7168 40.3, without 40.0.
constexpr float kLift = 0x1p64f, kMostLifted = 0x1p80f;
struct Walk {
    const Plan &p;
    int unit, units, tile, part;
    bool split;  // this cluster has a tile to share: the same for all its CTAs
    __device__ __forceinline__ Walk(const Plan &plan) : p(plan) {
        unit = tile = plan.pair ? blockIdx.x / 2 : blockIdx.x;
        units = plan.pair ? plan.grid / 2 : plan.grid;
        part = unit % plan.cluster;
        split = plan.cluster > 1 && plan.whole + unit / plan.cluster < plan.tiles_m * plan.tiles_n;
    }
    __device__ __forceinline__ bool next(Segment &s) {
        if (tile < p.whole) {
            s = Segment{0, 0, 0, p.nk, false};
            place(s, tile);
            tile += units;
            return true;
        }
        if (!split || tile == INT_MAX) return false;
        s = Segment{0, 0, p.nk * part / p.cluster, p.nk * (part + 1) / p.cluster, true};
        place(s, p.whole + unit / p.cluster);
        tile = INT_MAX;
        return true;
    }
    __device__ __forceinline__ void place(Segment &s, int t) {
        const int m0 = t / (kBand * p.tiles_n) * kBand, r = t - m0 * p.tiles_n, high = min(kBand, p.tiles_m - m0);
        s.m = m0 + r % high;
        s.n = r / high;
    }
};

template <int kCols, bool kPair>
__global__ void __launch_bounds__(kThreads, 1)
    linear_fp8_tc(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                  const __grid_constant__ CUtensorMap tm_out, const __grid_constant__ CUtensorMap tm_res,
                  const __grid_constant__ LinearFp8Args a, const __grid_constant__ Plan plan) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    using L = Smem<kCols, kPair>;
    uint64_t *taken = reinterpret_cast<uint64_t *>(smem + L::kStages * L::kStage + L::kTile);  // an accumulator, by the sums' warps
    uint64_t *full = taken + L::kBufs;  // a stage's copies have come
    uint64_t *spent = full + L::kStages;  // its MMAs are done: it is free, and their sums are there
    uint64_t *drain = spent + L::kStages;
    uint64_t *tile_free = drain + 1;  // the tile's memory holds the residual, or nothing that is needed
    uint64_t *tile_done = tile_free + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(tile_done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    // a pair's: whether some pair of the cluster gave up, and the stages the other CTA issued
    volatile int *gave_up = abort_flag + 1;
    volatile uint32_t *peer_issued = reinterpret_cast<volatile uint32_t *>(gave_up + 1);
    // some warp did not wait for the tile's memory: what lies there is not to be stored, of this tile or a later one
    volatile int *lost = reinterpret_cast<volatile int *>(peer_issued + 1);
    const Patience patience{a.wait_ns, abort_flag};
    const int warp = __shfl_sync(~0u, threadIdx.x / 32, 0), lane = threadIdx.x % 32;

    if (threadIdx.x == 0) {
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&spent[s], 1);
        }
        for (int i = 0; i < L::kBufs; ++i) mbar_init(&taken[i], (kPair ? 2 : 1) * kSumWarps);
        mbar_init(tile_free, 1);
        mbar_init(tile_done, kSumWarps);
        mbar_init(drain, 1);
        *abort_flag = *gave_up = *lost = 0;
        *peer_issued = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_x);
        tma_prefetch_desc(&tm_w);
    }
    if (warp == 1) {
        if (kPair) tmem_alloc_pair<512>(tmem_slot);
        else tmem_alloc<512>(tmem_slot);
    }
    tc_fence_before();
    __syncthreads();
    if (kPair) cluster_sync();  // the leader's barriers are ready for the other CTA
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // Launched while the grid before it ends, whose results are read from here on; the next one may
    // begin its setup, too (its tensor memory is another SM's: two of these do not fit one).
    pdl_launch_dependents();
    pdl_wait();
    constexpr int kTileM = kPair ? 2 * kRows : kRows;
    const int half = kPair ? (int)(blockIdx.x & 1) : 0;
    const uint32_t leader = kPair ? cluster_rank() & ~1u : 0, both = 3u << leader;
    Walk walk(plan);
    Segment seg;
    uint32_t issued = 0;  // the load warp's stages

    // The loads' and the MMAs' loops are run by whole warps on values that are the same in
    // every lane, and one elected lane issues: the operands stay in uniform registers.
    if (warp < kFirstSum) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegOther));
        if (warp == 0) {
            const uint32_t lead_full = kPair ? map_to_rank(smem_u32(full), leader) : 0;
            uint32_t s = 0, phase = 1;
            bool ok = true, free = mbar_test_wait(&spent[0], 1);
            while (ok && walk.next(seg)) {
                const int t0 = seg.m * kTileM + half * kRows;
                const int n0 = seg.n * kCols + half * (kCols / 2);
                for (int kc = seg.k0; kc < seg.k1; ++kc) {
                    // the first round's waits are for the phase before the barriers' first: over at once
                    if (!wait_for(free, &spent[s], phase, patience)) {
                        ok = false;
                        break;
                    }
                    uint8_t *st = smem + s * L::kStage;
                    uint64_t *bar = &full[s];
                    const uint32_t lead = lead_full + s * 8;
                    if (++s == L::kStages) {
                        s = 0;
                        phase ^= 1;
                    }
                    free = mbar_test_wait(&spent[s], phase);
                    if (elect_one()) {
                        if (kPair) {
                            if (half == 0) mbar_arrive_expect_tx(bar, 2 * L::kStage);
                            tma_load_2d_pair(st, &tm_x, lead, kc * kBK, t0);
                            tma_load_2d_pair(st + L::kXBytes, &tm_w, lead, kc * kBK, n0);
                        } else {
                            mbar_arrive_expect_tx(bar, plan.x_rows * kBK + L::kWBytes);
                            tma_load_2d(st, &tm_x, bar, kc * kBK, t0);
                            tma_load_2d(st + L::kXBytes, &tm_w, bar, kc * kBK, n0);
                        }
                    }
                    ++issued;
                }
            }
            // The copies in flight land in this CTA's shared memory.  A pair's are counted by the
            // leader, both halves of a stage together; where it does not see them all, the
            // cluster's CTAs settle it after their next barrier.
            const uint32_t tail = issued > L::kStages ? issued - L::kStages : 0;
            if (!kPair) {
                for (uint32_t i = tail; i < issued; ++i) ok &= mbar_wait(&full[i % L::kStages], (i / L::kStages) & 1);
                if (!ok) *abort_flag = 1;
            } else if (half == 0) {
                for (uint32_t i = tail; i < issued; ++i)
                    ok = ok && wait_for(false, &full[i % L::kStages], (i / L::kStages) & 1, patience);
                if (!ok && lane < 2 * plan.cluster) st_cluster_u32(map_to_rank(smem_u32((const void *)gave_up), lane), 1);
            } else if (lane == 0) {
                st_cluster_u32(map_to_rank(smem_u32((const void *)peer_issued), leader), issued);
            }
            __syncwarp();
        } else if (warp == 1 && half == 0) {
            // A commit takes some 200 cycles of the tensor pipe's time, so a block has one: its barrier tells the load
            // warp that the stage is free and the sums' warps that the accumulator is full.  They cannot miss a
            // phase of it: the stage's next MMAs come after kBufs or more others, and those wait for the sums' warps.
            constexpr uint32_t idesc = idesc_e4m3(kTileM, kCols);
            // descriptors of stage 0: a stage and a step of K move the start address (in 16 bytes)
            const uint64_t x_desc = smem_desc_sw128(smem_u32(smem), 16, 1024);
            const uint64_t w_desc = smem_desc_sw128(smem_u32(smem) + L::kXBytes, 16, 1024);
            const uint32_t acc0 = __shfl_sync(~0u, tmem, 0);
            uint32_t s = 0, phase = 0, n = 0;  // n: blocks issued
            bool ok = true, there = false;
            while (ok && walk.next(seg)) {
                for (int kc = seg.k0; ok && kc < seg.k1; ++kc, ++n) {
                    const uint32_t b = n % L::kBufs;
                    if (!wait_for(there, &full[s], phase, patience)) {
                        ok = false;
                        break;
                    }
                    const uint64_t dx = x_desc + (uint64_t)(s * (L::kStage >> 4)), dw = w_desc + (uint64_t)(s * (L::kStage >> 4));
                    uint64_t *bar = &spent[s];
                    if (++s == L::kStages) {
                        s = 0;
                        phase ^= 1;
                    }
                    there = mbar_test_wait(&full[s], phase);  // its answer comes while the MMAs are issued
                    if (n >= L::kBufs && !wait_for<true>(false, &taken[b], (n / L::kBufs - 1) & 1, patience)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < kBK / 32; ++kk)
                            mma_codes<kPair>(acc0 + b * kCols, dx + kk * (32 >> 4), dw + kk * (32 >> 4), idesc, kk > 0);
                        if (kPair) mma_commit_pair(bar, both);
                        else mma_commit(bar);
                    }
                }
            }
            __syncwarp();
            if (elect_one()) {  // waited for at the end
                if (kPair) mma_commit_pair(drain, both);
                else mma_commit(drain);
            }
            __syncwarp();
        } else if (warp == 2) {
            // The output's tiles: the residual comes to the tile's memory early (of a tile that a cluster
            // shares, the slabs with this CTA's columns), the sums' warps turn it into the result, and that is
            // copied out.  The wait for them is not one for work: they come whatever else happens.  Once one of them has
            // given up its wait for the tile's memory, that is offered no more, and the tiles that were not copied out yet become NaN
            // from here.  (What the sums' warps still do with it, and with the barriers, is then nobody's.)
            uint8_t *slabs = smem + L::kStages * L::kStage;
            bool ok = true;
            uint32_t offered = 0;  // tiles whose memory was
            while (walk.next(seg)) {
                const int t0 = seg.m * kTileM + half * kRows;
                int n0 = seg.n * kCols, used = kCols / 64;
                if (seg.cut) {
                    const int share = kCols / plan.cluster, first = walk.part * share / 64;
                    n0 += first * 64;
                    used = (walk.part * share + share - 1) / 64 - first + 1;
                }
                used = t0 < a.M && n0 < a.N ? min(used, (a.N - n0 + 63) / 64) : 0;
                if (ok) {
                    if (lane == 0) {
                        if (a.residual && used > 0) {
                            mbar_arrive_expect_tx(tile_free, used * (kRows * 128));
                            for (int j = 0; j < used; ++j)
                                tma_load_2d(slabs + j * (kRows * 128), &tm_res, tile_free, n0 + 64 * j, t0);
                        } else {
                            mbar_arrive(tile_free);
                        }
                    }
                    ++offered;
                }
                __syncwarp();
                if (seg.cut) break;
                ok = ok && wait_beyond(tile_done, (offered - 1) & 1, a.wait_ns, lost);
                if (!ok) {
                    if (used > 0 && n0 + 8 * lane < min(n0 + 64 * used, a.N)) {
                        uint4 *to = reinterpret_cast<uint4 *>(a.out + (long long)t0 * a.out_stride + n0 + 8 * lane);
                        uint4 *end = to + (long long)min(kRows, a.M - t0) * (a.out_stride / 8);
#pragma unroll 1
                        for (; to < end; to += a.out_stride / 8) *to = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
                    }
                } else if (lane == 0) {
                    for (int j = 0; j < used; ++j) tma_store_2d(&tm_out, slabs + j * (kRows * 128), n0 + 64 * j, t0);
                    bulk_commit();
                    bulk_wait_read_all();
                }
                __syncwarp();
            }
            if (lane == 0) bulk_wait_all();
            if (offered > 0) mbar_wait(tile_free, (offered - 1) & 1);  // no residual is on its way
            if (!ok) *abort_flag = 1;
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegSum));
        constexpr int kWide = L::kWide;
        const int q = warp & 3, cw = (warp - kFirstSum) / 4 * kWide;
        const uint32_t lead_taken = map_to_rank(smem_u32(taken), kPair ? leader : cluster_rank());
        uint8_t *tile_memory = smem + L::kStages * L::kStage;  // slabs of 64 columns, 128 bytes a token
        const uint32_t acc0 = __shfl_sync(~0u, tmem + tmem_lane_base(q) + cw, 0);
        bool ok = true;
        uint32_t b = 0, s = 0, phase = 0, done = 0;  // the next block's accumulator and stage; tiles taken
        for (; walk.next(seg); ++done) {
            const int k0 = seg.k0, k1 = seg.k1;
            const int t0 = seg.m * kTileM + half * kRows, n0 = seg.n * kCols;
            const int nt = min(kRows, a.M - t0);
            const bool active = q * 32 < nt && n0 + cw < a.N;
            float sums[kWide];
#pragma unroll
            for (int e = 0; e < kWide; ++e) sums[e] = 0.f;
            // the blocks' scales come four at a time, while the four before are at work
            const float *sx = a.x_scale + k0 * a.x_scale_stride + min(t0 + q * 32 + lane, a.M - 1);
            const int row = min(n0 + cw, a.N - 1) / kBK, before = L::kTwo ? kBK - (n0 + cw) % kBK : kWide;
            const float *sw = a.w_scale + (long long)row * plan.nk + k0;
            const int next = L::kTwo ? (min(n0 + cw + kWide, a.N) - 1) / kBK > row ? plan.nk : 0 : 0;
            float nx[4], nw[4] = {0.f, 0.f, 0.f, 0.f}, nw2[4] = {0.f, 0.f, 0.f, 0.f};
            auto load_scales = [&](int left) {  // the next `left` blocks', at most 4
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < left) {
                        nx[j] = __ldg(sx);
                        nw[j] = __ldg(sw + j);
                        if (L::kTwo) nw2[j] = __ldg(sw + next + j);
                        sx += a.x_scale_stride;
                    } else {
                        nx[j] = 0.f;
                    }
                sw += 4;
            };
            load_scales(k1 - k0);
            float lift = kLift;
#pragma unroll 1
            for (int kc = k0; ok && kc < k1; kc += 4) {
                float scale[4], scale2[4];
                bool lower = false;
                auto lift_scales = [&] {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float x = nx[e] * lift;
                        scale[e] = x * nw[e];
                        scale2[e] = L::kTwo ? x * nw2[e] : scale[e];
                        lower |= !(fabsf(scale[e]) <= kMostLifted && fabsf(scale2[e]) <= kMostLifted);  // a NaN, too
                    }
                };
                lift_scales();
                if (__any_sync(~0u, lower && lift > 1.f)) {
                    times(sums, lower && lift > 1.f ? 1.f / kLift : 1.f);
                    if (lower) lift = 1.f;
                    lift_scales();
                }
                load_scales(k1 - kc - 4);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (!ok || kc + j >= k1) continue;
                    ok = wait_for(false, &spent[s], phase, patience);
                    // a warp that gave up holds the accumulator: its arrivals, which wait for nothing, would
                    // stand for those of a warp that still reads
                    if (!ok) continue;
                    tc_fence_after();
                    if (active) add_block<kWide>(sums, acc0 + b * kCols, scale[j], scale2[j], before);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_taken(lead_taken + b * 8);
                    b = (b + 1) % L::kBufs;
                    if (++s == L::kStages) {
                        s = 0;
                        phase ^= 1;
                    }
                }
            }
            times(sums, lift > 1.f ? 1.f / kLift : 1.f);
            if (!ok) {
#pragma unroll
                for (int e = 0; e < kWide; ++e) sums[e] = __int_as_float(0x7fc00000);
            }
            if (!seg.cut) {
                const bool there = wait_for(false, tile_free, done & 1, patience);
                if (!there) *lost = 1;  // then warp 2 does not copy the tile out
                if (active) {
#pragma unroll
                    for (int c = 0; c < kWide; c += 32) {
                        const int column = cw + c;
                        uint8_t *row = tile_memory + (column / 64 * kRows + q * 32 + lane) * 128;
                        auto finish = [&](auto act) {
                            finish_columns<decltype(act)::value>(a, sums + c, row, column % 64 / 8, lane & 7, n0 + column);
                        };
                        switch (a.act) {
                            case MLA_ACT_RELU: finish(Value<MLA_ACT_RELU>()); break;
                            case MLA_ACT_SILU: finish(Value<MLA_ACT_SILU>()); break;
                            case MLA_ACT_GELU: finish(Value<MLA_ACT_GELU>()); break;
                            case MLA_ACT_GELU_TANH: finish(Value<MLA_ACT_GELU_TANH>()); break;
                            default: finish(Value<MLA_ACT_NONE>()); break;
                        }
                    }
                }
                fence_proxy_async_smem();  // the copy reads the tile through the async proxy
                __syncwarp();
                if (lane == 0) mbar_arrive(tile_done);
            } else {
                // Every CTA of the cluster holds its part of the tile.  The ring, idle once all of them
                // have, takes the parts of the columns this CTA finishes, one slot a rank.
                // parts: the cluster's, where it is known to the compiler, that does without thirty divisions then (64 x
                // 16384 x 7168 27.5 us, so 26.3; 2 x 1936 x 2352 6.9, so 5.9).  A pair's kernel that holds the code for 2 and
                // for 4 is 5 % slower at whole tiles.
                const int part = walk.part;
                auto exchange = [&](auto known) {
                    const int parts = decltype(known)::value ? decltype(known)::value : plan.cluster, share = kCols / parts;  // a multiple of 8
                    cluster_sync();
                    if (kPair && *gave_up) cluster_sync();  // the load warps settle it before this
                    // four columns of the tokens lie together, so that a warp writes and reads 512 bytes at a time
                    if (q * 32 + lane < nt) {
                        const uint32_t mine = smem_u32(smem) + (uint32_t)(part * (share / 4) * kRows + q * 32 + lane) * 16;
#pragma unroll
                        for (int e = 0; e < kWide / 4; ++e) {
                            const int c = cw + 4 * e, to = c / share;
                            const uint32_t at = mine + (uint32_t)(c % share / 4) * (kRows * 16);
                            if (to == part) st_shared_v4(at, sums[4 * e], sums[4 * e + 1], sums[4 * e + 2], sums[4 * e + 3]);
                            else st_cluster_v4(map_to_rank(at, kPair ? 2 * to + half : to), sums[4 * e], sums[4 * e + 1], sums[4 * e + 2], sums[4 * e + 3]);
                        }
                    }
                    __syncwarp();
                    const bool there = wait_for(false, tile_free, done & 1, patience) && !*lost;
                    cluster_sync();
                    // 32 tokens x 8 columns at a time, dealt out to the warps
                    const int runs = (nt + 31) / 32;
#pragma unroll 1
                    for (int i = warp - kFirstSum; i < runs * (share / 8); i += kSumWarps) {
                        const int g = i / runs, token = (i - g * runs) * 32 + lane;
                        const int at = part * share + 8 * g, n = n0 + at;  // in the tile, in the output
                        if (token >= nt || n >= a.N) continue;
                        const float4 *from = reinterpret_cast<const float4 *>(smem) + 2 * g * kRows + token;
                        float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, f[8];
#pragma unroll
                        for (int r = 0; r < parts; ++r) {
                            const float4 lo = from[r * (share / 4) * kRows], hi = from[(r * (share / 4) + 1) * kRows];
                            y[0] += lo.x; y[1] += lo.y; y[2] += lo.z; y[3] += lo.w;
                            y[4] += hi.x; y[5] += hi.y; y[6] += hi.z; y[7] += hi.w;
                        }
                        if (a.bias) {
                            Finish::unpack8(__ldg(reinterpret_cast<const uint4 *>(a.bias + n)), f);
#pragma unroll
                            for (int e = 0; e < 8; ++e) y[e] += f[e];
                        }
                        activate(a.act, y);
                        if (!there) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) y[e] = __int_as_float(0x7fc00000);
                        } else if (a.residual) {
                            const int in_slabs = at - part * share / 64 * 64, chunk = in_slabs % 64 / 8;
                            Finish::unpack8(*reinterpret_cast<const uint4 *>(tile_memory + (in_slabs / 64 * kRows + token) * 128 +
                                                                             ((chunk ^ (token & 7)) << 4)), f);
#pragma unroll
                            for (int e = 0; e < 8; ++e) y[e] += f[e];
                        }
                        *reinterpret_cast<uint4 *>(a.out + (long long)(t0 + token) * a.out_stride + n) = make_uint4(
                            pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
                    }
                };
                if (kPair) exchange(Value<0>());
                else if (plan.cluster == 2) exchange(Value<2>());
                else if (plan.cluster == 4) exchange(Value<4>());
                else exchange(Value<8>());
            }
        }
    }
    if (walk.split && warp < kFirstSum) {  // the barriers of the exchange
        __syncwarp();
        cluster_sync();
        if (kPair && *gave_up) {  // the same for every CTA of the cluster
            if (warp == 0 && half == 0 && !settle_pair<L::kStages, L::kStage>(full, issued, *peer_issued)) *abort_flag = 1;
            __syncwarp();
            cluster_sync();
        }
        cluster_sync();
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) set_status(a.status, MLA_ERR_TIMEOUT);
    // The MMAs end, and with them the arrivals on this CTA's barriers, before its memory is given
    // up.  They have ended where their results were waited for, and where that was given up
    // nobody reads what they still write.
    if (warp == 1) mbar_wait(drain, 0);
    __syncwarp();
    if (kPair) {
        cluster_sync();  // neither CTA's memory is used by the other any more
        if (!walk.split && *gave_up) {
            if (warp == 0 && half == 0) settle_pair<L::kStages, L::kStage>(full, issued, *peer_issued);
            __syncwarp();
            cluster_sync();
        }
    }
    if (warp == 1) {
        tc_fence_after();
        if (kPair) tmem_free_pair<512>(tmem);
        else tmem_free<512>(tmem);
    }
}

// A matrix of codes, 128-byte swizzle: `width` bytes a row, rows `stride` bytes apart (a multiple of 16),
// boxes of 128 bytes x box_rows.  Out-of-range elements read as zero.
bool encode_codes(CUtensorMap *m, const void *base, uint64_t width, uint64_t rows, uint64_t stride, uint32_t box_rows) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t gd[2] = {width, rows}, gs[1] = {stride};
    const cuuint32_t bd[2] = {kBK, box_rows}, es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), gd, gs, bd, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kCols, bool kPair = false>
cudaError_t launch(const LinearFp8Args &a, const Plan &p, cudaStream_t st) {
    CUtensorMap tm_x, tm_w;
    if (!encode_codes(&tm_x, a.x, a.K, a.M, a.x_stride, p.x_rows) ||
        !encode_codes(&tm_w, a.w, a.K, a.N, a.K, kPair ? kCols / 2 : kCols))
        return cudaErrorInvalidValue;
    // the output's map is for whole tiles alone, the residual's for a residual: else not read
    CUtensorMap tm_out = tm_x, tm_res = tm_x;
    const uint64_t dims[2] = {(uint64_t)a.N, (uint64_t)a.M}, out_stride = a.out_stride * 2, res_stride = a.residual_stride * 2;
    const uint32_t box[2] = {64, kRows};
    if ((p.whole > 0 && !encode_bf16_sw128(&tm_out, a.out, 2, dims, &out_stride, box)) ||
        (a.residual && !encode_bf16_sw128(&tm_res, a.residual, 2, dims, &res_stride, box)))
        return cudaErrorInvalidValue;
    const int smem = Smem<kCols, kPair>::kBytes;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
    static std::atomic<unsigned long long> ready{0};  // devices the kernel's shared memory is allowed on
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        const cudaError_t e = cudaFuncSetAttribute(linear_fp8_tc<kCols, kPair>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kPair ? 2 * p.cluster : p.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = kPair || p.cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, linear_fp8_tc<kCols, kPair>, tm_x, tm_w, tm_out, tm_res, a, p);
}

}  // namespace

// The plan with the shortest estimate, in SM cycles.  The parts' costs were fitted to timings of every form and
// cluster at 168 sizes (1 to 4096 tokens, K from 64 to 19000, 32 to 25000 columns): a block of a tile, a tile's
// epilogue, and of a shared tile the barriers, the sums sent and the finish.  (Of a long K a block takes 380, 480, 690
// and 770 cycles.)  The choice is within 0.6 % of the best form timed on average, within 5 % for all but six, and
// 12 % at most.  Both sides of it, the best of each:
//   64 x 16384 x 7168   26.3 us in clusters of 2, 31 in whole tiles of 64 columns, 36 of 128
//   64 x 7168 x 576     6.3 us in clusters of 8, 15 in whole tiles
//   256 x 7168 x 24576  51 us in pairs' tiles of 192 columns, 54 of 256, the last of them shared, 53 on single CTAs
//   512 x 7168 x 7168   28 us in pairs' tiles of 192 columns, 30 of 256, 32 on single CTAs
//   4096 x 16384 x 7168 321 us in pairs' tiles of 256 columns, 380 of 192, 399 on single CTAs
//   373 x 1792 x 4856   9.7 us on single CTAs, 13 in pairs' tiles of 192 columns
// Pairs' tiles of 128 columns were 9 % better than the best of these at one of 75 sizes, elsewhere 2 % at most.
LinearFp8Plan linear_fp8_plan(int M, int K, int N, int sms) {
    Plan best{};
    double best_cost = 0.0;
    const int nk = (K + kBK - 1) / kBK;
    for (int form = 0; form < 4; ++form) {
        Plan p;
        p.pair = form >= 2;
        p.columns = 64 * (form + 1);
        const int tile_m = p.pair ? 2 * kRows : kRows;
        if (p.pair && M <= kRows) break;
        // of a shorter x no more than it has, in whole groups of 8; the rest of a tile's rows is then whatever
        // shared memory held, and its sums are nobody's.  (With boxes of 128 rows on a tensor of fewer than 8,
        // 1 x 16384 x 7168 took 33 us, so 26.)
        p.x_rows = M < kRows ? (M + 7) / 8 * 8 : kRows;
        p.tiles_m = (M + tile_m - 1) / tile_m;
        p.tiles_n = (N + p.columns - 1) / p.columns;
        p.nk = nk;
        const long long tiles = (long long)p.tiles_m * p.tiles_n;
        if (tiles > (1ll << 28)) continue;
        const double block = form == 0 ? 430.0 : form == 1 ? 560.0 : form == 2 ? 720.0 : 870.0, epilogue = 1500.0 + 14.0 * p.columns;
        const int rows = M < kRows ? M : kRows;
        for (p.cluster = 1; p.cluster <= (p.pair ? 4 : 8); p.cluster *= 2) {
            const int ctas = p.pair ? 2 * p.cluster : p.cluster;
            // clusters that fit the SMs: fewer than an even share, as a cluster stays within one of
            // the groups the SMs are built in
            const int fit = ctas == 1 ? sms : ctas == 2 ? sms / 2 : ctas == 4 ? sms / 4 - 2 : sms / 8 - 4;
            if (fit < 1 || (p.cluster > 1 && nk < 2 * p.cluster)) break;
            double cost;
            if (p.cluster == 1) {
                p.whole = (int)tiles;
                p.grid = (int)(tiles < fit ? tiles : fit) * ctas;
                cost = (double)((tiles + fit - 1) / fit) * (nk * block + epilogue);
            } else {
                // rounds of whole tiles, one a unit, and at most one tile a cluster left
                const long long a_round = (long long)fit * p.cluster;
                p.whole = (int)(tiles / a_round * a_round);
                if (tiles - p.whole < 1 || tiles - p.whole > fit) continue;
                p.grid = (p.whole > 0 ? fit : (int)tiles) * ctas;
                const double sent = (double)rows * p.columns * 4 * (p.cluster - 1) / p.cluster;
                cost = (double)(p.whole / a_round) * (nk * block + epilogue) + (nk + p.cluster - 1) / p.cluster * block +
                       2000.0 + sent / 9.0 + 60.0 * rows * p.columns / p.cluster / 256.0;
            }
            if (best.grid == 0 || cost < best_cost) {
                best = p;
                best_cost = cost;
            }
        }
    }
    return best;
}

cudaError_t launch_linear_fp8(const LinearFp8Args &a, const LinearFp8Plan &p, cudaStream_t st) {
    if (p.pair) return p.columns == 256 ? launch<256, true>(a, p, st) : launch<192, true>(a, p, st);
    return p.columns == 128 ? launch<128>(a, p, st) : launch<64>(a, p, st);
}

}  // namespace mla
