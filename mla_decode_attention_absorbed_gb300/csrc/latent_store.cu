// The new tokens' cache rows from their down-projection: RMS norm of the latent,
// rotation of the key, one rounding to the cache's format, written to the slots.
//
// One warp a token: a lane holds two 16-byte chunks of the latent (d_c <= 512) and
// two neighbouring values of the key (d_rope <= 64), so the row is read once, the mean
// square is one warp reduction, and nothing goes through shared memory.  In the half
// layout the two values belong to two pairs: lanes l and l + 16 hold values 2l, 2l + 1 of
// the first and of the second half, trade one each, turn a pair each, and trade back.
// A warp takes several tokens and has the next one's row under way.
//
// Bound by the rows' way through L2 with two of them under way a warp, not by HBM: of 32768
// rows of 576 values DRAM reads the 38 MB that come in, what is written stays in L2.  In turn
// over four sets of buffers (bf16, FP8; floors 11.1 and 8.3 us): 13.8 and 12.3 us with slots,
// 14.5 and 14.7 into a contiguous cache by the lengths, 15.7 and 16.0 into a paged one, where a
// row waits for its length and then for its page; the half layout 0.4 more.  On one set, in L2,
// 10.9 and 11.7.  64 rows: 2.3 us, a launch and a round trip.
#include "layer.h"
#include "rope.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

constexpr int kWarps = 4;  // warps a CTA
// As many as the 72 registers of each variant allow: 32768 rows in L2 10.9 us, with 6 11.1, with
// 8 11.9 (a second wave for the eighth), with 12 11.3, one warp a token without the loop 14.3.
constexpr int kCtasPerSm = 7;

// Two values as E4M3 codes (v0 in the low byte): nearest even, saturating at +-448.
__device__ __forceinline__ uint32_t e4m3x2(float v0, float v1) {
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(v1), "f"(v0));
    return r;
}

// What a warp reads of one token before it can compute: the row, and where it goes.
struct Row {
    uint4 c[2];   // 16-byte chunks lane and lane + 32 of the latent
    uint32_t k;   // the lane's two values of the key, bf16 x 2
    int slot;     // slots, else the sequence's length (which pos may need, too)
    int pos, len;
};

// The key's values at, at + 1 that a lane holds, and the pair it turns.
template <bool kHalf>
struct KeyLane {
    int at, pair;
    bool active;
    __device__ __forceinline__ KeyLane(int lane, int pairs) {
        const int l = lane & 15, upper = lane >> 4;
        at = kHalf ? upper * pairs + 2 * l : 2 * lane;
        pair = kHalf ? 2 * l + upper : lane;
        active = kHalf ? 2 * l < pairs : lane < pairs;
    }
    // the lane's two values <-> the pair it turns
    static __device__ __forceinline__ float2 trade(float2 k, int lane) {
        if (!kHalf) return k;
        const bool upper = lane & 16;
        const float got = __shfl_xor_sync(~0u, upper ? k.x : k.y, 16);
        return upper ? make_float2(got, k.y) : make_float2(k.x, got);
    }
};

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(r)
        : "l"(*reinterpret_cast<unsigned long long *>(&a)), "l"(*reinterpret_cast<unsigned long long *>(&b)),
          "l"(*reinterpret_cast<unsigned long long *>(&c)));
    return *reinterpret_cast<float2 *>(&r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(r)
        : "l"(*reinterpret_cast<unsigned long long *>(&a)), "l"(*reinterpret_cast<unsigned long long *>(&b)));
    return *reinterpret_cast<float2 *>(&r);
}

template <bool kHalf>
__device__ __forceinline__ Row load_row(const StoreArgs &a, int t, int lane) {
    Row r;
    const __nv_bfloat16 *src = a.x + t * a.token_stride;
    const int nc = a.d_c / 8;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        r.c[i] = make_uint4(0, 0, 0, 0);
        if (lane + 32 * i < nc) r.c[i] = *(reinterpret_cast<const uint4 *>(src) + lane + 32 * i);
    }
    r.k = 0;
    const KeyLane<kHalf> key(lane, a.d_rope / 2);
    if (key.active) r.k = *reinterpret_cast<const uint32_t *>(src + a.d_c + key.at);
    const bool by_lens = !a.slots || (a.rotate && !a.positions);
    r.len = by_lens ? __ldg(a.cache.seq_lens + (a.s_q == 1 ? t : t / a.s_q)) : 0;
    r.slot = a.slots ? __ldg(a.slots + t) : 0;
    r.pos = a.rotate && a.positions ? __ldg(a.positions + t) : 0;
    return r;
}

// Element offset in the cache of token t's row, or -1: skipped, or recorded in status.
__device__ __forceinline__ long long row_offset(const StoreArgs &a, Row &r, int t, int lane) {
    const AttnParams &c = a.cache;
    const long long W = a.d_c + a.d_rope;
    int error = 0;
    long long at = -1;
    if (a.slots && r.slot < 0) return -1;
    int b = t, j = 0;
    if (!a.slots || (a.rotate && !a.positions)) {  // where the lengths say
        b = a.s_q == 1 ? t : t / a.s_q;
        j = r.len - a.s_q + (t - b * a.s_q);
        if (!seq_len_ok(c, r.len)) error = MLA_ERR_SEQLEN;
        if (!a.positions) r.pos = j;
    }
    if (!error && a.rotate && r.pos < 0) return -1;
    if (error) {
    } else if (a.slots) {
        if (r.slot >= c.num_pages * c.page_size) error = MLA_ERR_PAGE;
        at = r.slot * W;
    } else if (c.block_table == nullptr) {
        at = (long long)b * c.seq_stride + j * W;
    } else {
        const int page = __ldg(c.block_table + (long long)b * c.max_pages + j / c.page_size);
        if (page < 0 || page >= c.num_pages) error = MLA_ERR_PAGE;
        at = ((long long)page * c.page_size + j % c.page_size) * W;
    }
    if (error) {
        if (lane == 0) set_status(a.status, error);
        return -1;
    }
    return at;
}

__device__ __forceinline__ float2 unpack(uint32_t v) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&v));
}

template <bool kFp8, bool kHalf>
__global__ void __launch_bounds__(32 * kWarps) latent_rows(const __grid_constant__ StoreArgs a) {
    const int lane = threadIdx.x % 32, nw = gridDim.x * kWarps;
    const int nc = a.d_c / 8;
    const KeyLane<kHalf> key(lane, a.d_rope / 2);
    int t = blockIdx.x * kWarps + threadIdx.x / 32;
    if (t >= a.tokens) return;
    Row row = load_row<kHalf>(a, t, lane);
    // FP8: value times 1 / kv_scale, last and by itself: the scale may be as small as 2^-126, and
    // taken together with a weight past 4 its inverse would be infinite, a latent of 0 NaN
    const float unit = kFp8 ? 1.f / a.cache.kv_scale : 1.f;
    const float2 unit2 = make_float2(unit, unit);
    float2 wt[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint4 v = make_uint4(0x3f803f80, 0x3f803f80, 0x3f803f80, 0x3f803f80);  // ones
        if (a.weight && lane + 32 * i < nc) v = __ldg(reinterpret_cast<const uint4 *>(a.weight) + lane + 32 * i);
        const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            wt[i][e] = unpack(w4[e]);
        }
    }
    const float part = 1.f / (float)a.d_c;
    const unsigned long long turn = a.rotate && key.active ? a.plan.turn[key.pair] : 0;
    while (true) {
        const int next = t + nw;
        const bool more = next < a.tokens;
        Row r = row;
        if (more) row = load_row<kHalf>(a, next, lane);  // on its way while this row is computed
        const long long at = row_offset(a, r, t, lane);
        if (at >= 0) {
            float2 f[2][4], sum2 = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t w4[4] = {r.c[i].x, r.c[i].y, r.c[i].z, r.c[i].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    f[i][e] = unpack(w4[e]);
                    sum2 = fma2(f[i][e], f[i][e], sum2);
                }
            }
            float2 inv = make_float2(1.f, 1.f);
            if (a.weight) {
                float sum = sum2.x + sum2.y;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
                inv.x = inv.y = rsqrtf(fmaf(sum, part, a.eps));
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    f[i][e] = mul2(mul2(f[i][e], inv), wt[i][e]);
                    if (kFp8) f[i][e] = mul2(f[i][e], unit2);
                }
            float2 k = unpack(r.k);
            if (a.rotate) {
                k = key.trade(k, lane);
                k = rope_turn(k.x, k.y, rope_cos_sin(turn, r.pos, a.plan.mscale, 1.f));
                k = key.trade(k, lane);
            }
            if (kFp8) {
                uint8_t *dst = const_cast<uint8_t *>(static_cast<const uint8_t *>(a.cache.kv)) + at;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int c = lane + 32 * i;
                    if (c < nc)
                        *(reinterpret_cast<uint2 *>(dst) + c) =
                            make_uint2(e4m3x2(f[i][0].x, f[i][0].y) | e4m3x2(f[i][1].x, f[i][1].y) << 16,
                                       e4m3x2(f[i][2].x, f[i][2].y) | e4m3x2(f[i][3].x, f[i][3].y) << 16);
                }
                if (key.active)
                    *reinterpret_cast<unsigned short *>(dst + a.d_c + key.at) = (unsigned short)e4m3x2(unit * k.x, unit * k.y);
            } else {
                __nv_bfloat16 *dst = const_cast<__nv_bfloat16 *>(static_cast<const __nv_bfloat16 *>(a.cache.kv)) + at;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int c = lane + 32 * i;
                    if (c < nc)
                        *(reinterpret_cast<uint4 *>(dst) + c) =
                            make_uint4(sm100::pack_bf16x2(f[i][0].x, f[i][0].y), sm100::pack_bf16x2(f[i][1].x, f[i][1].y),
                                       sm100::pack_bf16x2(f[i][2].x, f[i][2].y), sm100::pack_bf16x2(f[i][3].x, f[i][3].y));
                }
                if (key.active) *reinterpret_cast<uint32_t *>(dst + a.d_c + key.at) = sm100::pack_bf16x2(k.x, k.y);
            }
        }
        if (!more) return;
        t = next;
    }
}

}  // namespace

cudaError_t launch_latent_store(const StoreArgs &a, cudaStream_t st) {
    int grid = (a.tokens + kWarps - 1) / kWarps;
    if (grid > layer_num_sms() * kCtasPerSm) grid = layer_num_sms() * kCtasPerSm;
    const bool half = a.rotate && a.plan.layout == MLA_ROPE_HALF;
    if (a.cache.kv_fp8) {
        if (half) latent_rows<true, true><<<grid, 32 * kWarps, 0, st>>>(a);
        else latent_rows<true, false><<<grid, 32 * kWarps, 0, st>>>(a);
    } else {
        if (half) latent_rows<false, true><<<grid, 32 * kWarps, 0, st>>>(a);
        else latent_rows<false, false><<<grid, 32 * kWarps, 0, st>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace mla
