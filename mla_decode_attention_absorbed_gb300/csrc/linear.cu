// out = residual + act(x . W + bias) on the 5th-generation tensor cores (tcgen05).
//
// The product is computed transposed: the MMA's rows are 128 columns n of W (as
// stored, so MN-major), its columns are BT tokens of x (K-major), D[n][token] in
// tensor memory.  A batch of a few tokens then costs an MMA of that width and a
// ring that is nearly all weights, and the epilogue's lanes are 32 neighbouring
// columns of one output row.
//
// K runs in chunks of 64 through a ring of TMA stages.  The work is tiles x chunks.
// With many tiles, a CTA takes whole tiles; with few, the tiles laid end to end are
// dealt out in equal runs of chunks, one a CTA: a run covers the end of one tile,
// whole ones, and the start of another.  A whole tile is finished in place; the
// pieces of a cut one go to the workspace in fp32, and a second kernel adds them in
// the order of K and applies the epilogue, so that results do not depend on which
// CTA was first.
//
// Warps: 0 issues the loads, 1 the MMAs, 2-5 drain the accumulators (two of them, so
// that one tile's epilogue runs beside the next one's products).
#include "layer.h"
#include "sm100.cuh"
#include "tmap.h"

namespace mla {
namespace {

using namespace sm100;

constexpr int kBN = 128;  // columns of W a tile
constexpr int kBK = 64;
constexpr int kThreads = 192;
constexpr int kMinChunks = 4;  // chunks a CTA's run holds at least

struct Plan {
    int bt;                // tokens a tile
    int tiles_m, tiles_n;  // tile t: tokens (t % tiles_m) * bt, columns (t / tiles_m) * 128
    int nk;                // chunks a tile
    int grid;
    bool whole;            // whole tiles, CTA g the tiles g, g + grid, ...; else runs of chunks
};

__host__ __device__ __forceinline__ long long run_start(const Plan &p, int g) {
    return (long long)p.tiles_m * p.tiles_n * p.nk * g / p.grid;
}

Plan make_plan(int M, int K, int N, int sms) {
    Plan p;
    p.bt = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : M <= 128 ? 128 : 256;
    p.tiles_m = (M + p.bt - 1) / p.bt;
    p.tiles_n = (N + kBN - 1) / kBN;
    p.nk = (K + kBK - 1) / kBK;
    const long long tiles = (long long)p.tiles_m * p.tiles_n;
    p.whole = tiles >= 2 * sms;
    const long long most = p.whole ? tiles : (tiles * p.nk + kMinChunks - 1) / kMinChunks;
    p.grid = most < sms ? (int)most : sms;
    if (tiles % p.grid == 0) p.whole = true;  // equal runs of chunks are whole tiles
    return p;
}

template <int BT>
struct Smem {
    static constexpr int kWBytes = kBN * kBK * 2;
    static constexpr int kXBytes = BT * kBK * 2;
    static constexpr int kStage = kWBytes + kXBytes;
    static constexpr int kStages = (200 * 1024) / kStage > 12 ? 12 : (200 * 1024) / kStage;
    static constexpr int kBytes = kStages * kStage + 1024 /* barriers */ + 1024 /* alignment */;
    static constexpr uint32_t kTmemCols = 2 * BT < 32 ? 32 : 2 * BT;
};

template <int kAct>
__device__ __forceinline__ float activate(float v) {
    if (kAct == MLA_ACT_RELU) return v < 0.f ? 0.f : v;  // NaN stays
    if (kAct == MLA_ACT_SILU) return v / (1.f + __expf(-v));
    // 1 + erf(z) = erfc(-z) and (1 + tanh z) / 2 = 1 / (1 + exp(-2 z)): no cancellation where they are small
    if (kAct == MLA_ACT_GELU) return 0.5f * v * erfcf(v * -0.70710678f);
    if (kAct == MLA_ACT_GELU_TANH) return v / (1.f + __expf(-1.59576912f * (v + 0.044715f * v * v * v)));
    return v;
}
__device__ __forceinline__ float activate(int act, float v) {
    switch (act) {
        case MLA_ACT_RELU: return activate<MLA_ACT_RELU>(v);
        case MLA_ACT_SILU: return activate<MLA_ACT_SILU>(v);
        case MLA_ACT_GELU: return activate<MLA_ACT_GELU>(v);
        case MLA_ACT_GELU_TANH: return activate<MLA_ACT_GELU_TANH>(v);
        default: return v;
    }
}

// One segment of a CTA's work: chunks [k0, k1) of a tile.
struct Segment {
    int tile, k0, k1;
};
struct Walk {
    const Plan &p;
    long long u, end;
    __device__ __forceinline__ Walk(const Plan &plan, int g) : p(plan) {
        u = p.whole ? g : run_start(p, g);
        end = p.whole ? (long long)p.tiles_m * p.tiles_n : run_start(p, g + 1);
    }
    __device__ __forceinline__ bool next(Segment &s) {
        if (u >= end) return false;
        if (p.whole) {
            s = Segment{(int)u, 0, p.nk};
            u += p.grid;
            return true;
        }
        s.tile = (int)(u / p.nk);
        s.k0 = (int)(u - (long long)s.tile * p.nk);
        s.k1 = (int)min((long long)p.nk, s.k0 + (end - u));
        u += s.k1 - s.k0;
        return true;
    }
};

// Bounded wait that also ends when another warp of the CTA gave up.
__device__ __forceinline__ bool wait_or_abort(uint64_t *bar, uint32_t parity, volatile int *abort_flag) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    const long long c0 = clock64();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 15u) == 0 && (*abort_flag || wait_expired(t0, c0))) {
            *abort_flag = 1;
            return false;
        }
    }
}

template <int BT>
__global__ void __launch_bounds__(kThreads, 1)
    linear_tc(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x, LinearArgs a, Plan plan) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    using L = Smem<BT>;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::kStages * L::kStage);
    uint64_t *empty = full + L::kStages;
    uint64_t *acc_full = empty + L::kStages;
    uint64_t *acc_empty = acc_full + 2;
    uint64_t *drain = acc_empty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    pdl_launch_dependents();

    if (threadIdx.x == 0) {
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 4);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_w);
        tma_prefetch_desc(&tm_x);
    }
    if (warp == 1) tmem_alloc<L::kTmemCols>(tmem_slot);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    Walk walk(plan, blockIdx.x);
    Segment seg;

    if (warp == 0 && lane == 0) {
        uint32_t it = 0;
        bool ok = true;
        while (ok && walk.next(seg)) {
            const int t0 = seg.tile % plan.tiles_m * BT, n0 = seg.tile / plan.tiles_m * kBN;
            for (int kc = seg.k0; kc < seg.k1; ++kc, ++it) {
                const uint32_t s = it % L::kStages;
                if (it >= L::kStages && !wait_or_abort(&empty[s], (it / L::kStages - 1) & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                uint8_t *st = smem + s * L::kStage;
                mbar_arrive_expect_tx(&full[s], L::kStage);
                tma_load_2d(st, &tm_w, &full[s], n0, kc * kBK);
                tma_load_2d(st + L::kWBytes / 2, &tm_w, &full[s], n0 + 64, kc * kBK);
                tma_load_2d(st + L::kWBytes, &tm_x, &full[s], kc * kBK, t0);
            }
        }
        // given up: the copies in flight still land in this CTA's shared memory
        if (!ok)
            for (uint32_t i = it > L::kStages ? it - L::kStages : 0; i < it; ++i)
                mbar_wait(&full[i % L::kStages], (i / L::kStages) & 1);
    } else if (warp == 1 && lane == 0) {
        constexpr uint32_t idesc = idesc_bf16(kBN, BT, true, false);
        uint32_t it = 0, n_seg = 0;
        bool ok = true;
        for (; ok && walk.next(seg); ++n_seg) {
            const uint32_t b = n_seg & 1;
            if (n_seg >= 2 && !wait_or_abort(&acc_empty[b], (n_seg / 2 - 1) & 1, abort_flag)) break;
            tc_fence_after();
            const uint32_t d = tmem + b * BT;
            for (int kc = seg.k0; kc < seg.k1; ++kc, ++it) {
                const uint32_t s = it % L::kStages;
                if (!wait_or_abort(&full[s], (it / L::kStages) & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t sw = smem_u32(smem + s * L::kStage), sx = sw + L::kWBytes;
#pragma unroll
                for (int kk = 0; kk < kBK / 16; ++kk)
                    mma_ss(d, smem_desc_sw128(sw + kk * 16 * 128, 64 * 128, 1024), smem_desc_sw128(sx + kk * 32, 16, 1024),
                           idesc, kc > seg.k0 || kk > 0);
                mma_commit(&empty[s]);
            }
            if (ok) mma_commit(&acc_full[b]);
        }
        if (*abort_flag) {  // let the MMAs in flight end before the memory they use is given up
            mma_commit(drain);
            mbar_wait(drain, 0);
        }
    } else if (warp >= 2) {
        const int q = warp & 3;
        const int nl = q * 32 + lane;
        bool ok = true;
        bool first_seg = true;
        for (uint32_t n_seg = 0; walk.next(seg); ++n_seg) {
            const uint32_t b = n_seg & 1;
            ok = ok && wait_or_abort(&acc_full[b], (n_seg / 2) & 1, abort_flag);
            tc_fence_after();
            const int t0 = seg.tile % plan.tiles_m * BT, n = seg.tile / plan.tiles_m * kBN + nl;
            const bool cut = seg.k0 > 0 || seg.k1 < plan.nk;
            float *part = a.part + (2ll * blockIdx.x + (first_seg ? 0 : 1)) * (kBN * BT) + nl;
            const float bias = a.bias && n < a.N ? __bfloat162float(a.bias[n]) : 0.f;
            const int nt = min(BT, a.M - t0);
            for (int c = 0; c < nt; c += 16) {
                uint32_t r[16];
                tmem_ld16(tmem + tmem_lane_base(q) + b * BT + c, r);
                tmem_ld_wait();
                if (!ok)
                    for (int e = 0; e < 16; ++e) r[e] = 0x7fc00000u;
                if (cut) {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (c + e < nt) part[(c + e) * kBN] = __uint_as_float(r[e]);
                } else if (n < a.N) {
                    // all the residual's loads before the first store (out may be residual)
                    __nv_bfloat16 res[16];
                    if (a.residual) {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (c + e < nt) res[e] = a.residual[(long long)(t0 + c + e) * a.residual_stride + n];
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        if (c + e >= nt) break;
                        float v = activate(a.act, __uint_as_float(r[e]) + bias);
                        if (a.residual) v += __bfloat162float(res[e]);
                        a.out[(long long)(t0 + c + e) * a.out_stride + n] = __float2bfloat16_rn(v);
                    }
                }
                __syncwarp();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[b]);
            first_seg = false;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_free<L::kTmemCols>(tmem);
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
    pdl_wait();
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int g = g0; g <= g1; ++g) {
        const int slot = run_start(plan, g) >= u0 ? 0 : run_start(plan, g) / plan.nk == tile ? 0 : 1;
        const float4 v = *reinterpret_cast<const float4 *>(a.part + (2ll * g + slot) * (kBN * plan.bt) + t_in * kBN + nl);
        acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
    }
    const float y[4] = {acc.x, acc.y, acc.z, acc.w};
    float o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = activate(a.act, y[e] + bias[e]) + res[e];
    *reinterpret_cast<uint2 *>(a.out + t * a.out_stride + n) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
}

template <int BT>
cudaError_t launch_bt(const LinearArgs &a, const Plan &p, cudaStream_t st) {
    CUtensorMap tm_w, tm_x;
    const uint64_t wd[2] = {(uint64_t)a.N, (uint64_t)a.K}, ws[1] = {(uint64_t)a.N * 2};
    const uint64_t xd[2] = {(uint64_t)a.K, (uint64_t)a.M}, xs[1] = {(uint64_t)a.x_stride * 2};
    const uint32_t wb[2] = {64, kBK}, xb[2] = {kBK, BT};
    if (!encode_bf16_sw128(&tm_w, a.w, 2, wd, ws, wb) || !encode_bf16_sw128(&tm_x, a.x, 2, xd, xs, xb))
        return cudaErrorInvalidValue;
    const int smem = Smem<BT>::kBytes;
    cudaError_t e = cudaFuncSetAttribute(linear_tc<BT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    linear_tc<BT><<<p.grid, kThreads, smem, st>>>(tm_w, tm_x, a, p);
    return cudaGetLastError();
}

}  // namespace

size_t linear_workspace_bytes(int M, int K, int N) {
    const Plan p = make_plan(M, K, N, layer_num_sms());
    return p.whole ? 256 : 2ull * p.grid * kBN * p.bt * sizeof(float);
}

cudaError_t launch_linear(const LinearArgs &a, cudaStream_t st) {
    const Plan p = make_plan(a.M, a.K, a.N, layer_num_sms());
    cudaError_t e;
    switch (p.bt) {
        case 16: e = launch_bt<16>(a, p, st); break;
        case 32: e = launch_bt<32>(a, p, st); break;
        case 64: e = launch_bt<64>(a, p, st); break;
        case 128: e = launch_bt<128>(a, p, st); break;
        default: e = launch_bt<256>(a, p, st); break;
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
