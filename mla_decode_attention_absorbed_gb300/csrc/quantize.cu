// Activations and weights as E4M3 codes with a scale for each block of 128 values of a row
// (activations), or of 128 x 128 (weights); activations on request after their RMS norm.
//
// Every value is read once, as 16 bytes a lane; 16 lanes hold 128 values of a row, so a
// row's block is a reduction over half a warp, and those of up to 8 blocks are one.  Each of the two divisions
// of a block is made once, by a lane that holds its maximum for the others (made by every lane: 4096 x 16384 43.0 us;
// by one, with a reduction for each block, 33.6; so 31.1).
//
// Measured (device time; copies at the card's measured rate): rows of 4096 x 16384 31.1 us against 29.9 of bytes, squares of
// 7168 x 16384 50.7 against 51.9, both bound by HBM; after the norm 4096 x 7168 20.0 against 13.1, bound by
// instructions, about 80 for a lane's 8 values (bf16 kept and normalised twice, for more CTAs an SM: 23.8; persistent
// CTAs that have the next rows on their way, to registers 20.9 when this took 20.8, to shared memory by cp.async 20.5, and
// 32.6 for 4096 x 12288, so 37.7, but 12.7 for 4096 x 4096, so 11.3, and 15.5 for 5120, so 14.3); 16384 x 512 6.9 against 3.7;
// 64 x 7168 2.6, a launch and a round trip.
#include "quantize.cuh"

namespace mla {
namespace {

using namespace quant;
using sm100::fma2;

constexpr int kThreads = 256;
constexpr int kMostThreads = 512;  // with the norm
constexpr int kRowsAWarp = 8;

// Without a norm the blocks have nothing to do with one another: a warp takes 8 rows of 256
// values, all of them under way before the first is used, and its scales leave as 8
// neighbouring values a block.
__global__ void __launch_bounds__(kThreads, 4) quantize_rows(const QuantizeArgs a, int wide) {
    sm100::pdl_launch_dependents();
    const int lane = threadIdx.x % 32;
    const long long item = (long long)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
    const int m0 = (int)(item / wide) * kRowsAWarp, k = (int)(item % wide) * 256 + lane * 8;
    if (m0 >= a.M) return;
    const int rows = min(kRowsAWarp, a.M - m0);
    uint4 v[kRowsAWarp];
#pragma unroll
    for (int r = 0; r < kRowsAWarp; ++r) {
        v[r] = make_uint4(0, 0, 0, 0);
        if (r < rows && k < a.K) v[r] = *reinterpret_cast<const uint4 *>(a.x + (m0 + r) * a.x_stride + k);
    }
    float top[kRowsAWarp];
#pragma unroll
    for (int r = 0; r < kRowsAWarp; ++r) top[r] = top8(v[r]);
    const float mine = unit_or_scale(tops16(top, lane), lane);
#pragma unroll
    for (int r = 0; r < kRowsAWarp; ++r) {
        float f[8];
        unpack8(v[r], f);
        const uint2 codes = codes8(f, unit_of<kRowsAWarp>(mine, lane, r));
        if (r < rows && k < a.K) *reinterpret_cast<uint2 *>(a.codes + (m0 + r) * a.code_stride + k) = codes;
    }
    const int row = (lane & 15) / (16 / kRowsAWarp);
    if (lane % 2 == 1 && row < rows && (k & ~(kBlock - 1)) < a.K)
        a.scales[(long long)(k / kBlock) * a.scale_stride + m0 + row] = mine;
}

// The sum over a CTA's warps, of any number up to kMostThreads / 32.
__device__ __forceinline__ float sum_of_warps(float sum) {
    __shared__ float part[kMostThreads / 32];
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = sum;
    __syncthreads();
    sum = 0.f;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) sum += part[w];
    return sum;
}

// With the norm: the row stays in registers between the sum and the codes, kParts times 8 values a
// thread.  A short row is a warp's (kWarp), a longer one a CTA's; one too long for that is read again,
// from L2, kParts at a time (kAgain).
template <int kParts, bool kWarp, bool kAgain>
__global__ void __launch_bounds__(kMostThreads, 2) quantize_normed(const QuantizeArgs a) {
    sm100::pdl_launch_dependents();
    const int lane = threadIdx.x % 32, t = kWarp ? lane : (int)threadIdx.x, step = kWarp ? 32 : (int)blockDim.x;
    const int m = kWarp ? (int)(blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32) : (int)blockIdx.x;
    if (kWarp && m >= a.M) return;
    const int nc = a.K / 8;
    const uint4 *src = reinterpret_cast<const uint4 *>(a.x + m * a.x_stride);
    const uint4 *weight = reinterpret_cast<const uint4 *>(a.weight);
    uint2 *dst = reinterpret_cast<uint2 *>(a.codes + m * a.code_stride);
    float y[kParts][8];
    auto load = [&](int c0) {
        uint4 v[kParts];
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            const int c = c0 + i * step + t;
            v[i] = c < nc ? src[c] : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kParts; ++i) unpack8(v[i], y[i]);
    };
    float2 sums = make_float2(0.f, 0.f);
    for (int c0 = 0; c0 < nc; c0 += kParts * step) {
        load(c0);
#pragma unroll
        for (int i = 0; i < kParts; ++i)
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const float2 p = make_float2(y[i][e], y[i][e + 1]);
                sums = fma2(p, p, sums);
            }
        if (!kAgain) break;
    }
    float sum = sums.x + sums.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    if (!kWarp) sum = sum_of_warps(sum);
    const float inv = rsqrtf(sum / (float)a.K + a.eps);
    for (int c0 = 0; c0 < nc; c0 += kParts * step) {
        if (kAgain) load(c0);
        // whole half warps are at work on a block, or beyond the row
        float top[kParts];
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            const int c = c0 + i * step + t;
            const uint4 w = c < nc ? __ldg(weight + c) : make_uint4(0, 0, 0, 0);
            const float2 inv2 = make_float2(inv, inv);
            float g[8];
            unpack8(w, g);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const float2 p = mul2(mul2(make_float2(y[i][e], y[i][e + 1]), inv2), make_float2(g[e], g[e + 1]));
                y[i][e] = p.x;
                y[i][e + 1] = p.y;
            }
            top[i] = top8(y[i]);
        }
        const float mine = unit_or_scale(tops16(top, lane), lane);
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            const int c = c0 + i * step + t;
            const uint2 codes = codes8(y[i], unit_of<kParts>(mine, lane, i));
            if (c < nc) dst[c] = codes;
        }
        // of a part's 16 / kParts lanes the second has its scale
        constexpr int kLanes = 16 / kParts;
        const int block = (c0 + (lane & 15) / kLanes * step + t - (lane & 15)) / 16;
        if (lane % kLanes == 1 && block * 16 < nc) a.scales[(long long)block * a.scale_stride + m] = mine;
        if (!kAgain) break;
    }
}

// A CTA a block of 128 x 128, 8 rows a thread.
__global__ void __launch_bounds__(kThreads, 4) quantize_squares(const QuantizeArgs a) {
    sm100::pdl_launch_dependents();
    __shared__ float part[kThreads / 32];
    const int k = blockIdx.x * kBlock + threadIdx.x % 16 * 8, m0 = blockIdx.y * kBlock + threadIdx.x / 16;
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = make_uint4(0, 0, 0, 0);
        if (m0 + 16 * i < a.M && k < a.K) v[i] = *reinterpret_cast<const uint4 *>(a.x + (m0 + 16 * i) * a.x_stride + k);
    }
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, top8(v[i]));
    top = top16(top);
    top = fmaxf(top, __shfl_xor_sync(~0u, top, 16));
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = top;
    __syncthreads();
    top = kLeast;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) top = fmaxf(top, part[w]);
    const float unit = __fdiv_rn(kTop, top);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float f[8];
        unpack8(v[i], f);
        if (m0 + 16 * i < a.M && k < a.K) *reinterpret_cast<uint2 *>(a.codes + (m0 + 16 * i) * a.code_stride + k) = codes8(f, unit);
    }
    if (threadIdx.x == 0) a.scales[blockIdx.y * a.scale_stride + blockIdx.x] = __fdiv_rn(top, kTop);
}

}  // namespace

cudaError_t launch_quantize(const QuantizeArgs &a, cudaStream_t st) {
    if (a.block_rows != 1) {
        quantize_squares<<<dim3((a.K + kBlock - 1) / kBlock, (a.M + kBlock - 1) / kBlock), kThreads, 0, st>>>(a);
    } else if (a.weight) {
        // a warp a row up to 1024 values (16384 rows of 512: 6.9 us, a CTA a row 17.6), then as many warps as
        // 1024 values each take, up to 16 (4096 rows of 2048, 5120 and 12288: 7.0, 14.0 and 37.7 us; with
        // 256 threads, past 8192 512, that hold less each or stand idle: 8.7, 18.4, 41.1)
        const int nc = a.K / 8;
        const unsigned grid = (a.M + kThreads / 32 - 1) / (kThreads / 32);
        if (nc <= 32) quantize_normed<1, true, false><<<grid, kThreads, 0, st>>>(a);
        else if (nc <= 64) quantize_normed<2, true, false><<<grid, kThreads, 0, st>>>(a);
        else if (nc <= 128) quantize_normed<4, true, false><<<grid, kThreads, 0, st>>>(a);
        else if (nc <= 4 * kMostThreads) quantize_normed<4, false, false><<<a.M, (nc + 127) / 128 * 32, 0, st>>>(a);
        else quantize_normed<4, false, true><<<a.M, kMostThreads, 0, st>>>(a);
    } else {
        const int wide = (a.K + 255) / 256;
        const long long warps = (long long)((a.M + kRowsAWarp - 1) / kRowsAWarp) * wide;
        quantize_rows<<<(unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32)), kThreads, 0, st>>>(a, wide);
    }
    return cudaGetLastError();
}

}  // namespace mla
