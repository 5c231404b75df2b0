// The new tokens' cache rows from their down-projection: RMS norm of the latent,
// rotation of the key, one rounding to the cache's format, written to the slots.
//
// One warp a token: a lane holds two 16-byte chunks of the latent (d_c <= 512) and
// one pair of the key (d_rope <= 64), so the row is read once, the mean square is
// one warp reduction, and nothing goes through shared memory.
#include "layer.h"
#include "rope.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

constexpr int kWarps = 4;  // warps a CTA
constexpr int kCtasPerSm = 8;

// Two values as E4M3 codes (v0 in the low byte): nearest even, saturating at +-448.
__device__ __forceinline__ uint32_t e4m3x2(float v0, float v1) {
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(v1), "f"(v0));
    return r;
}

// What a warp reads of one token before it can compute: the row, and where it goes.
struct Row {
    uint4 c[2];   // 16-byte chunks lane and lane + 32 of the latent
    uint32_t k;   // the lane's pair of the key, bf16 x 2
    int slot;     // slots, else the sequence's length (which pos may need, too)
    int pos, len;
};

template <bool kHalf>
__device__ __forceinline__ Row load_row(const StoreArgs &a, int t, int lane) {
    Row r;
    const __nv_bfloat16 *src = a.x + t * a.token_stride;
    const int nc = a.d_c / 8, nf = a.d_rope / 2;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        r.c[i] = make_uint4(0, 0, 0, 0);
        if (lane + 32 * i < nc) r.c[i] = *(reinterpret_cast<const uint4 *>(src) + lane + 32 * i);
    }
    r.k = 0;
    if (lane < nf) {
        const unsigned short *k = reinterpret_cast<const unsigned short *>(src + a.d_c);
        r.k = kHalf ? k[lane] | (uint32_t)k[lane + nf] << 16 : *reinterpret_cast<const uint32_t *>(k + 2 * lane);
    }
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
    const int nc = a.d_c / 8, nf = a.d_rope / 2;
    int t = blockIdx.x * kWarps + threadIdx.x / 32;
    if (t >= a.tokens) return;
    Row row = load_row<kHalf>(a, t, lane);
    float wt[2][8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (a.weight && lane + 32 * i < nc) v = __ldg(reinterpret_cast<const uint4 *>(a.weight) + lane + 32 * i);
        const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 p = unpack(w4[e]);
            wt[i][2 * e] = p.x;
            wt[i][2 * e + 1] = p.y;
        }
    }
    const float part = 1.f / (float)a.d_c;
    const unsigned long long turn = a.rotate && lane < nf ? a.plan.turn[lane] : 0;
    while (true) {
        const int next = t + nw;
        const bool more = next < a.tokens;
        Row r = row;
        if (more) row = load_row<kHalf>(a, next, lane);  // on its way while this row is computed
        const long long at = row_offset(a, r, t, lane);
        if (at >= 0) {
            float f[2][8], sum = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t w4[4] = {r.c[i].x, r.c[i].y, r.c[i].z, r.c[i].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 p = unpack(w4[e]);
                    f[i][2 * e] = p.x;
                    f[i][2 * e + 1] = p.y;
                    sum = fmaf(p.x, p.x, fmaf(p.y, p.y, sum));
                }
            }
            if (a.weight) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
                const float inv = rsqrtf(fmaf(sum, part, a.eps));
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[i][e] *= inv * wt[i][e];
            }
            float2 k = unpack(r.k);
            if (a.rotate) k = rope_turn(k.x, k.y, rope_cos_sin(turn, r.pos, a.plan.mscale, 1.f));
            if (kFp8) {
                uint8_t *dst = const_cast<uint8_t *>(static_cast<const uint8_t *>(a.cache.kv)) + at;
                const float s = a.cache.kv_scale;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int c = lane + 32 * i;
                    if (c < nc)
                        *(reinterpret_cast<uint2 *>(dst) + c) =
                            make_uint2(e4m3x2(f[i][0] / s, f[i][1] / s) | e4m3x2(f[i][2] / s, f[i][3] / s) << 16,
                                       e4m3x2(f[i][4] / s, f[i][5] / s) | e4m3x2(f[i][6] / s, f[i][7] / s) << 16);
                }
                if (lane < nf) {
                    const uint32_t code = e4m3x2(k.x / s, k.y / s);
                    dst += a.d_c;
                    if (kHalf) {
                        dst[lane] = (uint8_t)code;
                        dst[lane + nf] = (uint8_t)(code >> 8);
                    } else {
                        *reinterpret_cast<unsigned short *>(dst + 2 * lane) = (unsigned short)code;
                    }
                }
            } else {
                __nv_bfloat16 *dst = const_cast<__nv_bfloat16 *>(static_cast<const __nv_bfloat16 *>(a.cache.kv)) + at;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int c = lane + 32 * i;
                    if (c < nc)
                        *(reinterpret_cast<uint4 *>(dst) + c) =
                            make_uint4(sm100::pack_bf16x2(f[i][0], f[i][1]), sm100::pack_bf16x2(f[i][2], f[i][3]),
                                       sm100::pack_bf16x2(f[i][4], f[i][5]), sm100::pack_bf16x2(f[i][6], f[i][7]));
                }
                if (lane < nf) {
                    dst += a.d_c;
                    if (kHalf) {
                        dst[lane] = __float2bfloat16_rn(k.x);
                        dst[lane + nf] = __float2bfloat16_rn(k.y);
                    } else {
                        *reinterpret_cast<uint32_t *>(dst + 2 * lane) = sm100::pack_bf16x2(k.x, k.y);
                    }
                }
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
