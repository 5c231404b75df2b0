// Rotary positions of query or key rows, with the split of a projected query
// into the part that is not rotated and the part that is.
//
// Bound by memory: every value is read once and written once, 16 bytes an access; the
// angles are worked out once a token (a CTA's, in shared memory) and serve all of its
// heads.  8192 tokens x 128 heads x (128 + 64): 805 MB in 118.1 us = 6.82 TB/s, the measured
// copy bandwidth, with 128 rows a CTA and four copies under way a thread (one: 129.6, two:
// 120.6, eight: 134.8, for their registers; with one, 64 rows a CTA: 136.2, 256: 131.6, loads
// marked for early eviction: 133.7).  64 tokens x 128 heads take 3.1 us in groups of 16 rows
// (5.0 in groups of 128, on 64 of the 152 SMs): a launch and one memory round trip.
#include "layer.h"
#include "rope.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;
constexpr int kMaxTokens = 64;  // tokens a CTA holds the angles of (16 KB)

// i / d for i * d < 2^32 as one multiplication.
struct FastDiv {
    uint32_t d, m;
    explicit FastDiv(uint32_t n) : d(n), m((uint32_t)((0x100000000ull + n - 1) / n)) {}
    __device__ __forceinline__ uint32_t div(uint32_t i) const { return d == 1 ? i : __umulhi(i, m); }
};

__device__ __forceinline__ float2 unpack(uint32_t v) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&v));
}

// A CTA's rows: `tpb` whole tokens, or `hpb` of one token's heads.
__global__ void __launch_bounds__(kThreads)
    rope_rows(const __grid_constant__ RopeArgs a, int tpb, int hpb, FastDiv by_heads, FastDiv by_pass, FastDiv by_rope) {
    __shared__ float2 cs[kMaxTokens * 32];
    __shared__ int pos_s[kMaxTokens];
    const int t0 = blockIdx.x * tpb, h0 = blockIdx.y * hpb;
    const int nt = min(tpb, a.tokens - t0), nh = min(hpb, a.H - h0);
    const int nf = a.d_rope / 2;  // at most 32
    auto position = [&](int t) {
        if (a.positions) return __ldg(a.positions + t);
        const long long p = (long long)__ldg(a.seq_lens + t / a.s_q) - a.s_q + t % a.s_q;
        return p < 0 ? -1 : (int)p;
    };
    // a warp takes every 8th token, a lane a pair; the positions of all of a warp's tokens are
    // loaded at once (65536 keys of 64: 22.7 us one after another, 9.9 so)
    constexpr int kW = kThreads / 32;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (warp < nt) {
        const int mine = warp + kW * lane < nt ? position(t0 + warp + kW * lane) : 0;
        if (warp + kW * lane < nt) pos_s[warp + kW * lane] = mine;
        const unsigned long long turn = lane < nf ? a.plan.turn[lane] : 0;
        for (int t = warp, j = 0; t < nt; t += kW, ++j)
            cs[t * 32 + lane] = rope_cos_sin(turn, __shfl_sync(~0u, mine, j), a.plan.mscale, a.sign);
    }
    __syncthreads();
    const int rows = nt * nh;
    const int cp = a.d_pass / 8, ir = a.d_rope / 16;
    // kBatch loads before the first store, so that a thread has that many under way
    for (int i0 = threadIdx.x; i0 < rows * cp; i0 += kBatch * kThreads) {
        uint4 v[kBatch];
        __nv_bfloat16 *dst[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int i = i0 + j * kThreads;
            dst[j] = nullptr;
            if (i < rows * cp) {
                const int r = by_pass.div(i), c = i - r * cp;
                const int t = by_heads.div(r), h = h0 + r - t * nh;
                v[j] = *(reinterpret_cast<const uint4 *>(a.x + (t0 + t) * a.token_stride + h * a.head_stride) + c);
                if (pos_s[t] >= 0) dst[j] = a.pass_out + ((long long)(t0 + t) * a.H + h) * a.d_pass + 8 * c;
            }
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            if (dst[j]) *reinterpret_cast<uint4 *>(dst[j]) = v[j];
    }
    // an item is 16 values, 8 pairs: two neighbouring 16-byte chunks, or one of each half
    const bool half = a.plan.layout == MLA_ROPE_HALF;
    for (int i = threadIdx.x; i < rows * ir; i += kThreads) {
        const int r = by_rope.div(i), c = i - r * ir;
        const int t = by_heads.div(r), h = h0 + r - t * nh;
        const uint4 *src = reinterpret_cast<const uint4 *>(a.x + (t0 + t) * a.token_stride + h * a.head_stride + a.d_pass);
        const int c0 = half ? c : 2 * c, c1 = half ? c + ir : 2 * c + 1;
        const uint4 p = src[c0], q = src[c1];
        const uint32_t pw[4] = {p.x, p.y, p.z, p.w}, qw[4] = {q.x, q.y, q.z, q.w};
        uint32_t po[4], qo[4];
        const float2 *w = cs + t * 32 + 8 * c;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 u = unpack(pw[e]), v = unpack(qw[e]);
            if (half) {
                const float2 y0 = rope_turn(u.x, v.x, w[2 * e]), y1 = rope_turn(u.y, v.y, w[2 * e + 1]);
                po[e] = sm100::pack_bf16x2(y0.x, y1.x);
                qo[e] = sm100::pack_bf16x2(y0.y, y1.y);
            } else {
                const float2 y0 = rope_turn(u.x, u.y, w[e]), y1 = rope_turn(v.x, v.y, w[4 + e]);
                po[e] = sm100::pack_bf16x2(y0.x, y0.y);
                qo[e] = sm100::pack_bf16x2(y1.x, y1.y);
            }
        }
        if (pos_s[t] >= 0) {
            uint4 *dst = reinterpret_cast<uint4 *>(a.rope_out + ((long long)(t0 + t) * a.H + h) * a.d_rope);
            dst[c0] = make_uint4(po[0], po[1], po[2], po[3]);
            dst[c1] = make_uint4(qo[0], qo[1], qo[2], qo[3]);
        }
    }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, cudaStream_t st) {
    // Rows of one CTA: 128 where that makes four CTAs an SM, down to 16 where there are few.
    int rows = 128;
    const long long all = (long long)a.tokens * a.H;
    while (rows > 16 && all < 4ll * layer_num_sms() * rows) rows /= 2;
    int tpb = 1, hpb = a.H;
    if (a.H >= rows) {
        hpb = rows;
    } else {
        tpb = rows / a.H;
        if (tpb > kMaxTokens) tpb = kMaxTokens;
    }
    const dim3 grid((a.tokens + tpb - 1) / tpb, (a.H + hpb - 1) / hpb);
    rope_rows<<<grid, kThreads, 0, st>>>(a, tpb, hpb, FastDiv(hpb), FastDiv(a.d_pass ? a.d_pass / 8 : 1),
                                         FastDiv(a.d_rope / 16));
    return cudaGetLastError();
}

}  // namespace mla
