// What the matrix products (bf16 and 8-bit) share: activations, the epilogue of 8 columns of a
// token, bounded waits, and the forms of the instructions that act on a pair of CTAs.
#pragma once

#include "layer.h"
#include "sm100.cuh"

namespace mla {
namespace product {

using namespace sm100;

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

}  // namespace product
}  // namespace mla
