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

constexpr int kWarps = 4;  // tokens a CTA

// Two values as E4M3 codes (v0 in the low byte): nearest even, saturating at +-448.
__device__ __forceinline__ uint32_t e4m3x2(float v0, float v1) {
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(v1), "f"(v0));
    return r;
}

// Row of the cache token t goes to, or -1: skipped, or recorded in status.
__device__ __forceinline__ long long store_row(const StoreArgs &a, int t, int lane, long long &at) {
    const AttnParams &c = a.cache;
    const long long W = a.d_c + a.d_rope;
    if (a.slots) {
        const int s = __ldg(a.slots + t);
        if (s < 0) return -1;
        if (s >= c.num_pages * c.page_size) {
            if (lane == 0) set_status(a.status, MLA_ERR_PAGE);
            return -1;
        }
        at = s * W;
        return s;
    }
    const int b = t / a.s_q, L = __ldg(c.seq_lens + b);
    if (!seq_len_ok(c, L)) {
        if (lane == 0) set_status(a.status, MLA_ERR_SEQLEN);
        return -1;
    }
    const int j = L - a.s_q + t % a.s_q;
    if (c.block_table == nullptr) {
        at = (long long)b * c.seq_stride + j * W;
        return j;
    }
    const int page = __ldg(c.block_table + (long long)b * c.max_pages + j / c.page_size);
    if (page < 0 || page >= c.num_pages) {
        if (lane == 0) set_status(a.status, MLA_ERR_PAGE);
        return -1;
    }
    at = ((long long)page * c.page_size + j % c.page_size) * W;
    return j;
}

template <bool kFp8, bool kHalf>
__global__ void __launch_bounds__(32 * kWarps) latent_rows(const __grid_constant__ StoreArgs a) {
    const int lane = threadIdx.x % 32, t = blockIdx.x * kWarps + threadIdx.x / 32;
    if (t >= a.tokens) return;
    const __nv_bfloat16 *src = a.x + t * a.token_stride;
    const int nc = a.d_c / 8;
    // the row's loads first: none of them waits for the slot, the position or the weight
    uint4 raw[2] = {}, wt[2] = {};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int c = lane + 32 * i;
        if (c < nc) {
            raw[i] = *(reinterpret_cast<const uint4 *>(src) + c);
            if (a.weight) wt[i] = __ldg(reinterpret_cast<const uint4 *>(a.weight) + c);
        }
    }
    const int nf = a.d_rope / 2;
    float u = 0.f, v = 0.f;
    if (lane < nf) {
        const __nv_bfloat16 *k = src + a.d_c;
        if (kHalf) {
            u = __bfloat162float(k[lane]);
            v = __bfloat162float(k[lane + nf]);
        } else {
            const float2 uv = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(k + 2 * lane));
            u = uv.x;
            v = uv.y;
        }
    }
    long long at = 0;
    if (store_row(a, t, lane, at) < 0) return;
    if (a.rotate) {
        int pos;
        if (a.positions) {
            pos = __ldg(a.positions + t);
        } else {
            const int L = __ldg(a.cache.seq_lens + t / a.s_q);
            pos = L - a.s_q + t % a.s_q;
            if (!seq_len_ok(a.cache, L)) {  // slots with the lengths' positions
                if (lane == 0) set_status(a.status, MLA_ERR_SEQLEN);
                return;
            }
        }
        if (pos < 0) return;
        if (lane < nf) {
            const float2 y = rope_turn(u, v, rope_cos_sin(a.plan.turn[lane], pos, a.plan.mscale, 1.f));
            u = y.x;
            v = y.y;
        }
    }
    float f[2][8], sum = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t w4[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 p = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w4[e]));
            f[i][2 * e] = p.x;
            f[i][2 * e + 1] = p.y;
            sum = fmaf(p.x, p.x, fmaf(p.y, p.y, sum));
        }
    }
    if (a.weight) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        const float r = 1.f / sqrtf(sum / (float)a.d_c + a.eps);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t w4[4] = {wt[i].x, wt[i].y, wt[i].z, wt[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 p = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w4[e]));
                f[i][2 * e] *= r * p.x;
                f[i][2 * e + 1] *= r * p.y;
            }
        }
    }
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
            const uint32_t k = e4m3x2(u / s, v / s);
            dst += a.d_c;
            if (kHalf) {
                dst[lane] = (uint8_t)k;
                dst[lane + nf] = (uint8_t)(k >> 8);
            } else {
                *reinterpret_cast<unsigned short *>(dst + 2 * lane) = (unsigned short)k;
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
                dst[lane] = __float2bfloat16_rn(u);
                dst[lane + nf] = __float2bfloat16_rn(v);
            } else {
                *reinterpret_cast<uint32_t *>(dst + 2 * lane) = sm100::pack_bf16x2(u, v);
            }
        }
    }
}

}  // namespace

cudaError_t launch_latent_store(const StoreArgs &a, cudaStream_t st) {
    const int grid = (a.tokens + kWarps - 1) / kWarps;
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
