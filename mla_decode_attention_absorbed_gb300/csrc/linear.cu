// out = residual + act(x . W + bias) on the 5th-generation tensor cores (tcgen05).
//
// The product is computed transposed: the MMA's rows are 128 columns n of W (as
// stored, so MN-major), its columns are BT tokens of x (K-major), D[n][token] in
// tensor memory.  A batch of a few tokens then costs an MMA of that width and a
// ring that is nearly all weights, and the epilogue's lanes are 32 neighbouring
// columns of one output row.
//
// K runs in chunks of 64 through a ring of TMA stages.  The work is tiles x chunks, cut
// in one of three ways:
//   whole    a CTA takes whole tiles;
//   cluster  2, 4 or 8 CTAs (or pairs, see below) of a cluster take a tile's K in equal
//            parts, exchange their accumulators through distributed shared memory and
//            finish a share of the tokens each;
//   runs     the tiles laid end to end are dealt out in equal runs of chunks, one a CTA:
//            the end of one tile, whole ones, the start of another.  The pieces of a cut
//            tile go to the workspace in fp32, and a second kernel joins them.
// Parts are always added in the order of K, so results do not depend on timing.
//
// Warps: 0 issues the loads, 1 the MMAs, 2-9 drain the accumulators (two of them, so
// that one tile's epilogue runs beside the next one's products).  The epilogue turns its
// 32 columns x 16 tokens over in shared memory, so that a lane has 8 columns of a token:
// residual and output move as 16 bytes a lane (column by column, 2 bytes a lane, a
// 256-token tile's epilogue took 36 us; it is the tail of the whole launch).
//
// With many tokens a tile is 256 columns x 256 tokens on a pair of CTAs: one MMA of 256 x 256
// x 16 over both, each holding half of both operands, so that an SM takes in 32 KB a chunk
// instead of 48 (with the tokens as the MMA's rows, and rows written as they come or turned
// over in bf16, 0 to 6 % slower).
//
// Measured (device time): 4096 x 16384 x 7168 in 494 to 508 us for a dozen calls = 1,894 to 1,948
// TFLOP/s, the measured bf16 rate (tiles of 128 x 256 on single CTAs: 560), bound by the tensor
// cores, and in a long run of calls, as a prompt's layers make them, in 541 to 576 us = 1,670 to
// 1,780 TFLOP/s, bound by the power limit, under which a library product sustains 1,713; 64 x
// 16384 x 7168 in 39 to 40 us, 235 MB of weights at 5.9 TB/s = 0.88 of the measured copy
// bandwidth, with 2 us of start and 4 of exchange and epilogue around the stream; 333 x 1000 x
// 1544 in 7.4 us, a chain of latencies: 1.4 us to the first chunk, 16 chunks of 0.21, 1.1 of
// epilogue.
#include <atomic>

#include "layer.h"
#include "sm100.cuh"
#include "tmap.h"

namespace mla {
namespace {

using namespace sm100;

constexpr int kBN = 128;  // columns of W a tile
constexpr int kBK = 64;
constexpr int kThreads = 320;
constexpr int kEpiWarps = 8;  // two for each quarter of an accumulator's rows
constexpr int kStep = 16;     // tokens an epilogue warp turns over at a time
constexpr int kPitch = 36;  // floats between the tokens of a turned tile: conflict-free columns, 16-byte rows
constexpr int kMinChunks = 4;  // chunks a CTA's run of a cut tile holds at least

using Plan = LinearPlan;

__host__ __device__ __forceinline__ long long run_start(const Plan &p, int g) {
    return (long long)p.tiles_m * p.tiles_n * p.nk * g / p.grid;
}

template <int BT, bool kPair>
struct Smem {
    static constexpr int kWBytes = kBN * kBK * 2;
    static constexpr int kXBytes = (kPair ? BT / 2 : BT) * kBK * 2;
    static constexpr int kStage = kWBytes + kXBytes;
    static constexpr int kStages = (200 * 1024) / kStage > 12 ? 12 : (200 * 1024) / kStage;
    static constexpr int kTurn = kEpiWarps * kStep * kPitch * 4;  // the epilogue warps' 16 tokens x 32 columns
    static constexpr int kBytes = kStages * kStage + kTurn + 1024 /* barriers */ + 1024 /* alignment */;
    static_assert(BT * kBN * 4 <= kStages * kStage, "a cluster's accumulators are exchanged in the ring");
    static constexpr uint32_t kTmemCols = 2 * BT < 32 ? 32 : 2 * BT;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The activations hold their relative error down to the smallest normal numbers: where they
// fall off, the power of two is taken as h^2 with h = 2^(half the exponent), and the value is
// multiplied by h twice, so that nothing on the way leaves the range of fp32.  (With 2^x in
// one piece SiLU was -0 below -87.3 and GELU below -13.1, where bf16 still holds the result.)

// v / (1 + 2^(-2 x)): v times the logistic function of 2 x ln 2.
__device__ __forceinline__ float times_logistic(float v, float x) {
    const float h = ex2(-fabsf(x)), s = v * rcp(fmaf(h, h, 1.f));
    return x < 0.f ? s * h * h : s;
}

// v Phi(v), Phi the normal distribution.  With z = |v| / sqrt 2 and t = 1 / (1 + z / 2) (the
// change of variable that Press et al., Numerical Recipes, use for erfc),
//   Phi(-|v|) = erfc(z) / 2 = t 2^(Q(t) - z^2 log2 e),
// Q a polynomial fitted to log2(erfc(z) exp(z^2) / (2 t)) on (0, 1] (worst error 3.5e-6), here
// halved: no cancellation on either side.  Relative error at most 2^-17.3 from v = -10 up and
// 2^-16.7 below, where the rounding of an exponent near -120 counts.  CUDA's erfcf in its
// place took a 1588 x 400 x 6072 product with bias and residual from 29 us to 41.
__device__ __forceinline__ float gelu(float v) {
    const float t = rcp(fmaf(fabsf(v), 0.35355339f, 1.f));
    float q = fmaf(t, 0.5f * -0.22946589f, 0.5f * 0.9304564f);
    q = fmaf(t, q, 0.5f * -1.2151098f);
    q = fmaf(t, q, 0.5f * 0.32995093f);
    q = fmaf(t, q, 0.5f * 0.014981962f);
    q = fmaf(t, q, 0.5f * 0.55273217f);
    q = fmaf(t, q, 0.5f * 1.4422023f);
    q = fmaf(t, q, 0.5f * -2.8257446f);
    const float h = ex2(fmaf(v * v, 0.5f * -0.72134752f, q)), th = t * h;
    return v < 0.f ? v * th * h : v * fmaf(-th, h, 1.f);
}

template <int kAct>
__device__ __forceinline__ float activate(float v) {
    if (kAct == MLA_ACT_RELU) return v < 0.f ? 0.f : v;  // NaN stays
    if (kAct == MLA_ACT_SILU) return times_logistic(v, v * 0.72134752f);  // 2^-17.1
    if (kAct == MLA_ACT_GELU) return gelu(v);
    // (1 + tanh z) / 2 is the logistic function of 2 z; 2^-16.3
    if (kAct == MLA_ACT_GELU_TANH) return times_logistic(v, v * fmaf(v * v, 0.05147162f, 1.1511041f));
    return v;
}
template <int kAct, int N>
__device__ __forceinline__ void activate_all(float (&v)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = activate<kAct>(v[e]);
}
template <int N>
__device__ __forceinline__ void activate(int act, float (&v)[N]) {
    switch (act) {
        case MLA_ACT_RELU: activate_all<MLA_ACT_RELU>(v); break;
        case MLA_ACT_SILU: activate_all<MLA_ACT_SILU>(v); break;
        case MLA_ACT_GELU: activate_all<MLA_ACT_GELU>(v); break;
        case MLA_ACT_GELU_TANH: activate_all<MLA_ACT_GELU_TANH>(v); break;
        default: break;
    }
}

// Cluster plans: CTAs of a tile (a cluster), and which part of K this one's are.
__device__ __forceinline__ int ctas_a_tile(const Plan &p) { return p.pair ? 2 * p.cluster : p.cluster; }
__device__ __forceinline__ int part_of_k(const Plan &p) {
    const int r = blockIdx.x % ctas_a_tile(p);
    return p.pair ? r / 2 : r;
}

// One segment of a CTA's work: chunks [k0, k1) of a tile.
struct Segment {
    int tile, k0, k1;
};
struct Walk {
    const Plan &p;
    long long u, end;
    __device__ __forceinline__ Walk(const Plan &plan, int g) : p(plan) {
        if (p.cluster > 1) {
            u = g / ctas_a_tile(p);
            end = u + 1;
            return;
        }
        u = p.pair ? g / 2 : p.whole ? g : run_start(p, g);
        end = p.whole ? (long long)p.tiles_m * p.tiles_n : run_start(p, g + 1);
    }
    __device__ __forceinline__ bool next(Segment &s) {
        if (u >= end) return false;
        if (p.cluster > 1) {
            const int rank = part_of_k(p);
            s = Segment{(int)u, p.nk * rank / p.cluster, p.nk * (rank + 1) / p.cluster};
            u = end;
            return true;
        }
        if (p.whole) {
            s = Segment{(int)u, 0, p.nk};
            u += p.pair ? p.grid / 2 : p.grid;
            return true;
        }
        s.tile = (int)(u / p.nk);
        s.k0 = (int)(u - (long long)s.tile * p.nk);
        s.k1 = (int)min((long long)p.nk, s.k0 + (end - u));
        u += s.k1 - s.k0;
        return true;
    }
};

// The epilogue of 8 columns of some of a tile's tokens.
struct Finish {
    int t0, n;  // the tile's first token, the first column
    float bias[8];
    uint4 res[2];

    __device__ __forceinline__ Finish(const LinearArgs &a, int t0, int n) : t0(t0), n(n) {
#pragma unroll
        for (int e = 0; e < 8; ++e) bias[e] = 0.f;
        if (a.bias && n < a.N) unpack8(*reinterpret_cast<const uint4 *>(a.bias + n), bias);
    }
    static __device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 p = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[e]));
            f[2 * e] = p.x;
            f[2 * e + 1] = p.y;
        }
    }
    // the residual of tokens t and t + 8 of the tile (those below nt).  out may be residual:
    // a value is loaded by the thread that stores it, before it does
    __device__ __forceinline__ void load_residual(const LinearArgs &a, int t, int nt) {
        if (!a.residual || n >= a.N) return;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (t + 8 * i < nt)
                res[i] = *reinterpret_cast<const uint4 *>(a.residual + (long long)(t0 + t + 8 * i) * a.residual_stride + n);
    }
    __device__ __forceinline__ void load_half(const LinearArgs &a, int t, int nt) {  // token t alone
        if (a.residual && n < a.N && t < nt)
            res[0] = *reinterpret_cast<const uint4 *>(a.residual + (long long)(t0 + t) * a.residual_stride + n);
    }
    // v: the products' sums of 8 columns of token t
    __device__ __forceinline__ void store(const LinearArgs &a, int t, int nt, const float *v, uint4 res) const {
        if (t >= nt || n >= a.N) return;
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = v[e] + bias[e];
        activate(a.act, y);
        if (a.residual) {
            float r[8];
            unpack8(res, r);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] += r[e];
        }
        *reinterpret_cast<uint4 *>(a.out + (long long)(t0 + t) * a.out_stride + n) =
            make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
    }
};

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// The waits for work, which end after ns nanoseconds (cycles: twice that) or when another
// warp of the CTA gave up.  A wait that runs out raises the CTA's flag; its other waits for
// work then end too, what was not computed is written as NaN, and the CTA leaves by the same
// barriers as always.  Copies and MMAs in flight are waited for whatever happened (mbar_wait,
// 2 s): nothing may land in memory that the next CTA holds.
struct Patience {
    uint64_t ns;
    volatile int *abort_flag;
    __device__ __forceinline__ bool over(uint64_t t0, long long c0) const {
        return *abort_flag || globaltimer_ns() - t0 > ns || clock64() - c0 > (long long)(2 * ns);
    }
};

// For a whole warp, unless it is `done` already: every lane gets the same answer.
template <bool kCluster = false>
__device__ __forceinline__ bool warp_wait(bool done, uint64_t *bar, uint32_t parity, const Patience &p) {
    if (__all_sync(~0u, done)) return true;
    const uint64_t t0 = globaltimer_ns();
    const long long c0 = clock64();
    for (uint32_t it = 0;; ++it) {
        if (__all_sync(~0u, kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity))) return true;
        if ((it & 15u) == 0 && __any_sync(~0u, p.over(t0, c0))) {
            *p.abort_flag = 1;
            return false;
        }
    }
}

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(p));
    return p != 0;
}

// ---- the pair's forms: one MMA of 256 x BT over both CTAs' shared and tensor memory,
// issued by the first of them (the leader)
template <uint32_t kCols>
__device__ __forceinline__ void tmem_alloc_pair(uint32_t *dst) {  // a whole warp in each CTA
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "n"(kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
template <uint32_t kCols>
__device__ __forceinline__ void tmem_free_pair(uint32_t taddr) {  // a whole warp in each CTA
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "n"(kCols) : "memory");
}
// A copy into this CTA's shared memory whose bytes count on a barrier of the leader's
// (a cluster address).
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const CUtensorMap *m, uint32_t bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], "
        "[%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y)
        : "memory");
}
__device__ __forceinline__ void mma_ss_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrives on `bar` of both CTAs (`pair`: their bits by rank in the cluster) when the MMAs
// issued so far have completed.
__device__ __forceinline__ void mma_commit_pair(uint64_t *bar, uint32_t pair) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)pair)
        : "memory");
}

__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// Counts `bytes` on this CTA's barrier as a copy would.
__device__ __forceinline__ void mbar_complete_tx(uint64_t *bar, uint32_t bytes) {
    asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes)
                 : "memory");
}
// After a pair gave up: the leader's load warp issued `mine` stages, the other's `theirs`, and
// every stage counts the bytes of both on the leader's barrier.  The leader counts what the
// other did not issue, arms the stages that only the other issued, and so sees the last
// copies of both land.  The two are at most a ring apart: a stage is issued again only
// after its last chunk, both halves of it, was multiplied.
template <int kStages, uint32_t kBytes>
__device__ __forceinline__ bool settle_pair(uint64_t *full, uint32_t mine, uint32_t theirs) {
    if (elect_one()) {
        for (uint32_t i = theirs; i < mine; ++i) mbar_complete_tx(&full[i % kStages], kBytes);
        for (uint32_t i = mine; i < theirs; ++i) mbar_arrive_expect_tx(&full[i % kStages], kBytes);
    }
    __syncwarp();
    const uint32_t last = max(mine, theirs);
    bool ok = true;
    for (uint32_t i = last > kStages ? last - kStages : 0; i < last; ++i)
        ok &= mbar_wait(&full[i % kStages], (i / kStages) & 1);
    return ok;
}

template <int BT, bool kPair>
__global__ void __launch_bounds__(kThreads, 1)
    linear_tc(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x, LinearArgs a, Plan plan) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    using L = Smem<BT, kPair>;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::kStages * L::kStage + L::kTurn);
    uint64_t *empty = full + L::kStages;
    uint64_t *acc_full = empty + L::kStages;
    uint64_t *acc_empty = acc_full + 2;
    uint64_t *drain = acc_empty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    // a pair's: whether some pair of the cluster gave up, and the stages the other CTA issued
    volatile int *gave_up = abort_flag + 1;
    volatile uint32_t *peer_issued = reinterpret_cast<volatile uint32_t *>(gave_up + 1);
    const Patience patience{a.wait_ns, abort_flag};
    const int warp = __shfl_sync(~0u, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    pdl_launch_dependents();

    if (threadIdx.x == 0) {
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], kPair ? 2 * kEpiWarps : kEpiWarps);
        }
        mbar_init(drain, 1);
        *abort_flag = *gave_up = 0;
        *peer_issued = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_w);
        tma_prefetch_desc(&tm_x);
    }
    if (warp == 1) {
        if (kPair) tmem_alloc_pair<L::kTmemCols>(tmem_slot);
        else tmem_alloc<L::kTmemCols>(tmem_slot);
    }
    tc_fence_before();
    __syncthreads();
    if (kPair) cluster_sync();  // the leader's barriers are ready for the other CTA
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // a tile's columns, and this CTA's part of them (and of its tokens' copies) in a pair
    constexpr int kTileN = kPair ? 2 * kBN : kBN;
    const int half = kPair ? (int)(blockIdx.x & 1) : 0;
    const uint32_t leader = kPair ? cluster_rank() & ~1u : 0, both = 3u << leader;
    Walk walk(plan, blockIdx.x);
    Segment seg;
    uint32_t issued = 0;  // the load warp's stages

    // The loads' and the MMAs' loops are run by whole warps on values that are the same in
    // every lane, and one elected lane issues: the operands stay in uniform registers.  (With
    // the loops in a single lane, a chunk took 583 cycles whatever its width, all of it
    // issue; the MMAs of the widest tile take 512.)
    if (warp == 0) {
        const uint32_t lead_full = kPair ? map_to_rank(smem_u32(full), leader) : 0;
        uint32_t s = 0, phase = 1;
        bool ok = true, free = mbar_test_wait(&empty[0], 1);
        while (ok && walk.next(seg)) {
            const int t0 = seg.tile % plan.tiles_m * BT + half * (BT / 2);
            const int n0 = seg.tile / plan.tiles_m * kTileN + half * kBN;
            for (int kc = seg.k0; kc < seg.k1; ++kc) {
                // the first round's waits are for the phase before the barriers' first: over at once
                if (!warp_wait(free, &empty[s], phase, patience)) {
                    ok = false;
                    break;
                }
                uint8_t *st = smem + s * L::kStage;
                uint64_t *bar = &full[s];
                if (++s == L::kStages) {
                    s = 0;
                    phase ^= 1;
                }
                free = mbar_test_wait(&empty[s], phase);
                if (kPair) {
                    const uint32_t lead = lead_full + (uint32_t)(reinterpret_cast<uint8_t *>(bar) - reinterpret_cast<uint8_t *>(full));
                    if (elect_one()) {
                        if (half == 0) mbar_arrive_expect_tx(bar, 2 * L::kStage);
                        tma_load_2d_pair(st, &tm_w, lead, n0, kc * kBK);
                        tma_load_2d_pair(st + L::kWBytes / 2, &tm_w, lead, n0 + 64, kc * kBK);
                        tma_load_2d_pair(st + L::kWBytes, &tm_x, lead, kc * kBK, t0);
                    }
                } else if (elect_one()) {
                    mbar_arrive_expect_tx(bar, L::kStage);
                    tma_load_2d(st, &tm_w, bar, n0, kc * kBK);
                    tma_load_2d(st + L::kWBytes / 2, &tm_w, bar, n0 + 64, kc * kBK);
                    tma_load_2d(st + L::kWBytes, &tm_x, bar, kc * kBK, t0);
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
                ok = ok && warp_wait(false, &full[i % L::kStages], (i / L::kStages) & 1, patience);
            if (!ok && lane < 2 * plan.cluster) st_cluster_u32(map_to_rank(smem_u32((const void *)gave_up), lane), 1);
        } else if (lane == 0) {
            st_cluster_u32(map_to_rank(smem_u32((const void *)peer_issued), leader), issued);
        }
        __syncwarp();
    } else if (warp == 1 && half == 0) {
        constexpr uint32_t idesc = idesc_bf16(kTileN, BT, true, false);
        // descriptors of stage 0: a stage and a step of K move the start address (in 16 bytes)
        const uint64_t w_desc = smem_desc_sw128(smem_u32(smem), 64 * 128, 1024);
        const uint64_t x_desc = smem_desc_sw128(smem_u32(smem) + L::kWBytes, 16, 1024);
        const uint32_t acc0 = __shfl_sync(~0u, tmem, 0);
        uint32_t s = 0, phase = 0, n_seg = 0;
        bool ok = true, there = false;
        for (; ok && walk.next(seg); ++n_seg) {
            const uint32_t b = n_seg & 1;
            if (n_seg >= 2 && !warp_wait<kPair>(false, &acc_empty[b], (n_seg / 2 - 1) & 1, patience)) break;
            tc_fence_after();
            const uint32_t d = acc0 + b * BT;
            for (int kc = seg.k0; kc < seg.k1; ++kc) {
                if (!warp_wait(there, &full[s], phase, patience)) {
                    ok = false;
                    break;
                }
                const uint64_t dw = w_desc + (uint64_t)(s * (L::kStage >> 4)), dx = x_desc + (uint64_t)(s * (L::kStage >> 4));
                uint64_t *bar = &empty[s];
                if (++s == L::kStages) {
                    s = 0;
                    phase ^= 1;
                }
                there = mbar_test_wait(&full[s], phase);  // its answer comes while the MMAs are issued
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk)
                        (kPair ? mma_ss_pair : mma_ss)(d, dw + kk * (16 * 128 >> 4), dx + kk * (32 >> 4), idesc,
                                                       kk > 0 || kc > seg.k0);
                    if (kPair) mma_commit_pair(bar, both);
                    else mma_commit(bar);
                    if (kc + 1 == seg.k1) {
                        if (kPair) mma_commit_pair(&acc_full[b], both);
                        else mma_commit(&acc_full[b]);
                    }
                }
            }
        }
        __syncwarp();
        if (elect_one()) {  // waited for at the end
            if (kPair) mma_commit_pair(drain, both);
            else mma_commit(drain);
        }
        __syncwarp();
    } else if (warp >= 2) {
        const int q = warp & 3, c0 = (warp - 2) / 4 * kStep;  // its rows, and its first tokens
        bool ok = true;
        bool first_seg = true;
        float *turn = reinterpret_cast<float *>(smem + L::kStages * L::kStage) + (warp - 2) * kStep * kPitch;
        for (uint32_t n_seg = 0; plan.cluster == 1 && walk.next(seg); ++n_seg) {
            const uint32_t b = n_seg & 1;
            const int t0 = seg.tile % plan.tiles_m * BT, n0 = seg.tile / plan.tiles_m * kTileN + half * kBN;
            const bool cut = !plan.whole && (seg.k0 > 0 || seg.k1 < plan.nk);
            const int nt = min(BT, a.M - t0);
            const uint32_t acc = tmem + tmem_lane_base(q) + b * BT;
            Finish fin(a, t0, n0 + q * 32 + lane % 4 * 8);
            if (!cut) fin.load_residual(a, c0 + lane / 4, nt);
            ok = ok && warp_wait(false, &acc_full[b], (n_seg / 2) & 1, patience);
            tc_fence_after();
            float *part = a.part + (2ll * blockIdx.x + (first_seg ? 0 : 1)) * (kBN * BT) + q * 32 + lane;
            for (int c = c0; c < nt; c += 2 * kStep) {
                uint32_t r[kStep];
                tmem_ld16(acc + c, r);
                tmem_ld_wait();
                if (!ok)
                    for (int e = 0; e < kStep; ++e) r[e] = 0x7fc00000u;
                if (cut) {
#pragma unroll
                    for (int e = 0; e < kStep; ++e)
                        if (c + e < nt) part[(c + e) * kBN] = __uint_as_float(r[e]);
                } else {
#pragma unroll
                    for (int e = 0; e < kStep; ++e) turn[e * kPitch + lane] = __uint_as_float(r[e]);
                    __syncwarp();
                    uint4 res = fin.res[0], res1 = fin.res[1];
                    fin.load_residual(a, c + 2 * kStep + lane / 4, nt);  // the next tokens', under way meanwhile
#pragma unroll 1
                    for (int t = lane / 4; t < kStep; t += 8, res = res1)
                        fin.store(a, c + t, nt, turn + t * kPitch + lane % 4 * 8, res);
                }
                __syncwarp();
            }
            tc_fence_before();
            __syncwarp();
            // a warp that gave up holds the accumulator: its arrivals, which wait for nothing, would
            // stand for those of a warp that still reads
            if (lane == 0 && ok) {
                if (half == 0) mbar_arrive(&acc_empty[b]);
                else mbar_arrive_remote(map_to_rank(smem_u32(&acc_empty[b]), leader));
            }
            first_seg = false;
        }
    }
    if (plan.cluster > 1) {
        // Every CTA of the cluster holds its part of the tile.  The ring, idle once all of them
        // have, takes the parts of the tokens this CTA finishes, one slot a rank.
        const int rank = part_of_k(plan), share = BT / plan.cluster;
        const int tile = blockIdx.x / ctas_a_tile(plan), t0 = tile % plan.tiles_m * BT;
        const int n0 = tile / plan.tiles_m * kTileN + half * kBN;
        const int nt = min(BT, a.M - t0), i0 = threadIdx.x - 64;  // 16 threads a token, 8 columns each
        const int first = rank * share, last = min(nt, first + share);
        Finish fin(a, t0, warp >= 2 ? n0 + i0 % 16 * 8 : a.N);
        bool ok = true;
        if (warp >= 2) {
            fin.load_half(a, first + i0 / 16, last);
            ok = warp_wait(false, &acc_full[0], 0, patience);
        }
        __syncwarp();
        cluster_sync();
        if (kPair && *gave_up) {  // the same for every CTA of the cluster
            if (warp == 0 && half == 0 && !settle_pair<L::kStages, L::kStage>(full, issued, *peer_issued)) *abort_flag = 1;
            __syncwarp();
            cluster_sync();
        }
        if (warp >= 2) {
            tc_fence_after();
            const int q = warp & 3;
            const uint32_t slot = smem_u32(smem) + (uint32_t)(rank * share * kBN + q * 32 + lane) * 4;
            const int step = share < 16 ? share : 16;
            // the quarter's two warps take every other run of 16 tokens
            for (int c = (warp - 2) / 4 * step; c < nt; c += 2 * step) {
                uint32_t r[16];
                tmem_ld16(tmem + tmem_lane_base(q) + c, r);
                tmem_ld_wait();
                const int to = c / share;
                const uint32_t at = map_to_rank(slot + (uint32_t)(c - to * share) * (kBN * 4), kPair ? 2 * to + half : to);
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (e < step) st_cluster_f32(at + e * (kBN * 4), ok ? __uint_as_float(r[e]) : __int_as_float(0x7fc00000));
            }
            tc_fence_before();
        }
        __syncwarp();
        cluster_sync();
        const float *mine = reinterpret_cast<const float *>(smem) + i0 % 16 * 8;
        // 16 tokens at a time, the next ones' residual under way meanwhile
        for (int t = i0 / 16; warp >= 2 && first + t < last; t += 16) {
            const uint4 res = fin.res[0];
            fin.load_half(a, first + t + 16, last);
            float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            for (int s = 0; s < plan.cluster; ++s) {
                const float4 *v = reinterpret_cast<const float4 *>(mine + (s * share + t) * kBN);
                const float4 lo = v[0], hi = v[1];
                sum[0] += lo.x; sum[1] += lo.y; sum[2] += lo.z; sum[3] += lo.w;
                sum[4] += hi.x; sum[5] += hi.y; sum[6] += hi.z; sum[7] += hi.w;
            }
            fin.store(a, first + t, last, sum, res);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) set_status(a.status, MLA_ERR_TIMEOUT);
    // The MMAs end, and with them the arrivals on this CTA's barriers, before its memory is given
    // up.  They have ended where their results were waited for, and where that was given up
    // nobody reads what they still write.  (Waited for in the MMA warp, before a cluster's
    // exchange: 1264 x 6792 x 416 19.6 us, so 19.4.)
    if (warp == 1) mbar_wait(drain, 0);
    __syncwarp();
    if (kPair) {
        cluster_sync();  // neither CTA's memory is used by the other any more
        if (plan.cluster == 1 && *gave_up) {
            if (warp == 0 && half == 0) settle_pair<L::kStages, L::kStage>(full, issued, *peer_issued);
            __syncwarp();
            cluster_sync();
        }
    }
    if (warp == 1) {
        tc_fence_after();
        if (kPair) tmem_free_pair<L::kTmemCols>(tmem);
        else tmem_free<L::kTmemCols>(tmem);
    }
}

// The cut tiles: pieces added in the order of K, then the epilogue.  A CTA takes 8
// tokens of a tile, a warp one of them, a lane 4 columns.
constexpr int kJoinTokens = 8;
__global__ void __launch_bounds__(32 * kJoinTokens) linear_join(LinearArgs a, Plan plan) {
    const int tile = blockIdx.x, t_in = blockIdx.y * kJoinTokens + threadIdx.x / 32, nl = threadIdx.x % 32 * 4;
    const long long t = (long long)(tile % plan.tiles_m) * plan.bt + t_in, n = (long long)(tile / plan.tiles_m) * kBN + nl;
    // the CTAs whose runs hold the tile's first and last chunk
    const long long u0 = (long long)tile * plan.nk, u1 = u0 + plan.nk - 1, units = (long long)plan.tiles_m * plan.tiles_n * plan.nk;
    auto owner = [&](long long u) {
        int g = (int)(u * plan.grid / units);
        while (g + 1 < plan.grid && run_start(plan, g + 1) <= u) ++g;
        while (g > 0 && run_start(plan, g) > u) --g;
        return g;
    };
    const int g0 = owner(u0), g1 = owner(u1);
    if (g0 == g1 || t >= a.M || n >= a.N) {
        // what follows this grid relies on the products' grid having completed, too
        pdl_wait();
        return;
    }
    float bias[4] = {0.f, 0.f, 0.f, 0.f}, res[4] = {0.f, 0.f, 0.f, 0.f};
    auto load4 = [](const __nv_bfloat16 *p, float (&f)[4]) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        const float2 lo = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&v.x));
        const float2 hi = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&v.y));
        f[0] = lo.x; f[1] = lo.y; f[2] = hi.x; f[3] = hi.y;
    };
    if (a.bias) load4(a.bias + n, bias);
    if (a.residual) load4(a.residual + t * a.residual_stride + n, res);
    // the first CTA's run may have begun with another tile, the others' begin with this one
    const int slot0 = run_start(plan, g0) < u0 ? 1 : 0;
    const float *piece = a.part + (2ll * g0 + slot0) * (kBN * plan.bt) + t_in * kBN + nl;
    pdl_wait();
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int g = g0; g <= g1; ++g) {
        const float4 v = *reinterpret_cast<const float4 *>(piece + (2ll * (g - g0) - (g > g0 ? slot0 : 0)) * (kBN * plan.bt));
        acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
    }
    float y[4] = {acc.x + bias[0], acc.y + bias[1], acc.z + bias[2], acc.w + bias[3]};
    activate(a.act, y);
    *reinterpret_cast<uint2 *>(a.out + t * a.out_stride + n) =
        make_uint2(pack_bf16x2(y[0] + res[0], y[1] + res[1]), pack_bf16x2(y[2] + res[2], y[3] + res[3]));
}

template <int BT, bool kPair = false>
cudaError_t launch_bt(const LinearArgs &a, const Plan &p, cudaStream_t st) {
    CUtensorMap tm_w, tm_x;
    const uint64_t wd[2] = {(uint64_t)a.N, (uint64_t)a.K}, ws[1] = {(uint64_t)a.N * 2};
    const uint64_t xd[2] = {(uint64_t)a.K, (uint64_t)a.M}, xs[1] = {(uint64_t)a.x_stride * 2};
    const uint32_t wb[2] = {64, kBK}, xb[2] = {kBK, kPair ? BT / 2 : BT};
    if (!encode_bf16_sw128(&tm_w, a.w, 2, wd, ws, wb) || !encode_bf16_sw128(&tm_x, a.x, 2, xd, xs, xb))
        return cudaErrorInvalidValue;
    const int smem = Smem<BT, kPair>::kBytes;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
    static std::atomic<unsigned long long> ready{0};  // devices the kernel's shared memory is allowed on
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        const cudaError_t e = cudaFuncSetAttribute(linear_tc<BT, kPair>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kPair ? 2 * p.cluster : p.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = kPair || p.cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, linear_tc<BT, kPair>, tm_w, tm_x, a, p);
}

}  // namespace

// The plan with the shortest estimate, in SM cycles.  What the parts were measured to take
// (clock traces at M = 64, 333, 2048 and 4096, K = 1000 to 16384):
//   a chunk of a tile   about 400 cycles for narrow tiles (waits and issue), 455 at 128 tokens,
//                       600 at 256 (the MMAs alone: 512); all chunks together at least what
//                       it takes the card to bring the weights, at 3500 bytes a cycle
//   a tile's epilogue   1000 cycles and 36 a token; only the last one is not hidden
//   a cluster's exchange  about 1000 cycles and 30 a token
//   a chunk of a pair's tile  530 cycles
//   the second kernel of runs  about 6000 cycles and 180 a piece of a tile, and the pieces'
//                       bytes there and back at half the card's rate
// E.g. 64 x 16384 x 7168: 40.3 us in clusters of 2, 43.7 in runs, 58.5 in whole tiles of 32
// tokens; 333 x 1000 x 1544: 7.7 us in whole tiles of 32, 8.8 of 64, 12.7 in clusters;
// 256 x 16384 x 7168: 51.8 us in clusters of two pairs, 60.2 in clusters of two CTAs, 59.2 in
// runs; 4096 x 7168 x 576: 40.9 us in pairs, 49.9 in runs; 4096 x 16384 x 7168: 482 to 510 us
// in pairs, 587 in whole tiles of 128 x 256.  Over 35 shapes from 1 x 7168 x 576 up the choice
// was within 12 % of the best plan timed, and within 5 % for all but four.
LinearPlan linear_plan(int M, int K, int N, int sms) {
    Plan best{};
    double best_cost = 0.0;
    const double weights = 2.0 * K * N / 3500.0;  // however they are dealt out
    for (int bt = 16; bt <= 256; bt *= 2) {
        if (bt > 16 && bt / 2 >= M) break;
        Plan p;
        p.bt = bt;
        p.tiles_m = (M + bt - 1) / bt;
        p.tiles_n = (N + kBN - 1) / kBN;
        p.nk = (K + kBK - 1) / kBK;
        const long long tiles = (long long)p.tiles_m * p.tiles_n;
        if (tiles > (1ll << 28)) continue;
        const double chunk = 390.0 + 0.5 * bt > 2.35 * bt ? 390.0 + 0.5 * bt : 2.35 * bt;
        // n tiles, `fit` at a time, each `cycles` long or what its share of the weights takes
        auto waves_of = [&](long long n, long long fit, double cycles) {
            auto wave = [&](long long at_work) {
                const double w = weights * at_work / n;
                return w > cycles ? w : cycles;
            };
            return n / fit * wave(fit) + (n % fit ? wave(n % fit) : 0.0);
        };
        auto keep = [&](double cost) {
            if (best.bt == 0 || cost < best_cost) {
                best = p;
                best_cost = cost;
            }
        };
        const double epilogue = 1000.0 + 36.0 * bt;
        p.pair = false;
        p.whole = true;
        for (p.cluster = 1; p.cluster <= 8; p.cluster *= 2) {
            if (p.cluster > 1 && (p.nk < 2 * p.cluster || tiles > sms)) break;
            // clusters that fit the SMs: fewer than an even share, as a cluster stays within one of
            // the groups the SMs are built in.  36 of 4 and 15 of 8 are what the occupancy query
            // answers for 152 SMs; a device with other groups would get a worse estimate here,
            // never a wrong result: clusters that do not fit wait for their turn
            const int fit = p.cluster == 1 ? sms : p.cluster == 2 ? sms / 2 : p.cluster == 4 ? sms / 4 - 2 : sms / 8 - 4;
            if (fit < 1) break;
            const long long waves = (tiles + fit - 1) / fit;
            p.grid = p.cluster > 1 ? (int)tiles * p.cluster : tiles < sms ? (int)tiles : sms;
            keep(waves_of(tiles, fit, (p.nk + p.cluster - 1) / p.cluster * chunk) + epilogue +
                 (p.cluster > 1 ? 1000.0 + 30.0 * bt + (waves - 1) * (epilogue + 3000.0) : 0.0));
        }
        p.cluster = 1;
        if (bt == 256) {
            p.pair = true;
            p.tiles_n = (N + 2 * kBN - 1) / (2 * kBN);
            const long long pairs = (long long)p.tiles_m * p.tiles_n;
            for (p.cluster = 1; p.cluster <= 4; p.cluster *= 2) {
                const int fit = p.cluster == 1 ? sms / 2 : p.cluster == 2 ? sms / 4 - 2 : sms / 8 - 4;
                if (p.cluster > 1 && (p.nk < 2 * p.cluster || pairs > fit)) break;
                p.grid = 2 * p.cluster * (int)(pairs < fit ? pairs : fit);
                keep(waves_of(pairs, fit, (p.nk + p.cluster - 1) / p.cluster * 530.0) + epilogue + 1000.0 +
                     (p.cluster > 1 ? 30.0 * bt : 0.0));
            }
            p.cluster = 1;
            p.pair = false;
            p.tiles_n = (N + kBN - 1) / kBN;
        }
        const long long most = (tiles * p.nk + kMinChunks - 1) / kMinChunks;
        p.grid = most < sms ? (int)most : sms;
        // equal runs of chunks are whole tiles; and over several waves whole tiles in order of
        // the tokens share their weights in L2, which runs of tiles of a CTA's own do not
        // (4096 x 16384 x 7168: 611 us whole, 775 us in runs)
        if (tiles % p.grid == 0 || tiles >= 2 * sms) continue;
        p.whole = false;
        const double run = (double)((tiles * p.nk + p.grid - 1) / p.grid) * chunk;
        const double pieces = p.grid < tiles ? 2.0 * p.grid : p.grid + tiles;
        keep((run > weights ? run : weights) + epilogue + 6000.0 + 180.0 * p.grid / tiles +
             4.0 * pieces * kBN * bt * 4 / 3500.0);
    }
    return best;
}

size_t linear_workspace_bytes(const LinearPlan &p) {
    return p.whole ? 256 : 2ull * p.grid * kBN * p.bt * sizeof(float);
}

cudaError_t launch_linear(const LinearArgs &a, const LinearPlan &p, cudaStream_t st) {
    cudaError_t e;
    switch (p.bt) {
        case 16: e = launch_bt<16>(a, p, st); break;
        case 32: e = launch_bt<32>(a, p, st); break;
        case 64: e = launch_bt<64>(a, p, st); break;
        case 128: e = launch_bt<128>(a, p, st); break;
        default: e = p.pair ? launch_bt<256, true>(a, p, st) : launch_bt<256>(a, p, st); break;
    }
    if (e != cudaSuccess || p.whole) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.tiles_m * p.tiles_n, (p.bt + kJoinTokens - 1) / kJoinTokens);
    cfg.blockDim = dim3(32 * kJoinTokens);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, linear_join, a, p);
}

}  // namespace mla
