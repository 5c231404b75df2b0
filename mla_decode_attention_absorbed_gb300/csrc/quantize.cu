// Activations and weights as E4M3 codes with a scale for each block of 128 values of a row
// (activations), or of 128 x 128 (weights); activations on request after their RMS norm.
//
// Every value is read once, as 16 bytes a lane; 16 lanes hold 128 values of a row, so a
// row's block is one reduction over half a warp.
#include "quantize.cuh"

namespace mla {
namespace {

using namespace quant;

constexpr int kThreads = 256;
constexpr int kRowsAWarp = 8;

// Without a norm the blocks have nothing to do with one another: a warp takes 8 rows of 256
// values, all of them under way before the first is used, and its scales leave as 8
// neighbouring values a block.
__global__ void __launch_bounds__(kThreads) quantize_rows(const QuantizeArgs a, int wide) {
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
    float mine = 0.f;
#pragma unroll
    for (int r = 0; r < kRowsAWarp; ++r) {
        float f[8];
        unpack8(v[r], f);
        const float top = fmaxf(top16(top8(f)), kLeast);
        if (r < rows && k < a.K)
            *reinterpret_cast<uint2 *>(a.codes + (m0 + r) * a.code_stride + k) = codes8(f, __fdiv_rn(kTop, top));
        if ((lane & 15) == r) mine = top;
    }
    // lane r of a half holds row r's
    if ((lane & 15) < rows && (k & ~(kBlock - 1)) < a.K)
        a.scales[(long long)(k / kBlock) * a.scale_stride + m0 + (lane & 15)] = __fdiv_rn(mine, kTop);
}

// The norm's sum, over a CTA of any size up to kThreads.
__device__ __forceinline__ float sum_of_row(float sum) {
    __shared__ float part[kThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = sum;
    __syncthreads();
    sum = 0.f;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) sum += part[w];
    return sum;
}

// With the norm: a CTA a row, which stays in registers between the sum and the codes (kParts
// times 16 bytes a thread; 0: a row too long for that is read a second time, from L2).
template <int kParts>
__global__ void __launch_bounds__(kThreads) quantize_normed(const QuantizeArgs a) {
    const int m = blockIdx.x, nc = a.K / 8, step = blockDim.x;
    const uint4 *src = reinterpret_cast<const uint4 *>(a.x + m * a.x_stride);
    const uint4 *weight = reinterpret_cast<const uint4 *>(a.weight);
    uint2 *dst = reinterpret_cast<uint2 *>(a.codes + m * a.code_stride);
    auto add = [](uint4 v, float sum) {
        float f[8];
        unpack8(v, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(f[e], f[e], sum);
        return sum;
    };
    // chunk c (whole half warps are at work on a block, or beyond the row)
    auto finish = [&](uint4 v, uint4 g, int c, float inv) {
        float f[8], w[8];
        unpack8(v, f);
        unpack8(g, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = f[e] * inv * w[e];
        const float top = fmaxf(top16(top8(f)), kLeast);
        if (c < nc) {
            dst[c] = codes8(f, __fdiv_rn(kTop, top));
            if (threadIdx.x % 16 == 0) a.scales[(long long)(c / 16) * a.scale_stride + m] = __fdiv_rn(top, kTop);
        }
    };
    const uint4 zero = make_uint4(0, 0, 0, 0);
    float sum = 0.f;
    if (kParts > 0) {
        uint4 v[kParts > 0 ? kParts : 1], g[kParts > 0 ? kParts : 1];
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            const int c = i * step + threadIdx.x;
            v[i] = c < nc ? src[c] : zero;
        }
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            const int c = i * step + threadIdx.x;
            g[i] = c < nc ? __ldg(weight + c) : zero;
        }
#pragma unroll
        for (int i = 0; i < kParts; ++i) sum = add(v[i], sum);
        const float inv = rsqrtf(sum_of_row(sum) / (float)a.K + a.eps);
#pragma unroll
        for (int i = 0; i < kParts; ++i) finish(v[i], g[i], i * step + threadIdx.x, inv);
    } else {
        for (int c = threadIdx.x; c < nc; c += step) sum = add(src[c], sum);
        const float inv = rsqrtf(sum_of_row(sum) / (float)a.K + a.eps);
        for (int c0 = 0; c0 < nc; c0 += step) {
            const int c = c0 + threadIdx.x;
            finish(c < nc ? src[c] : zero, c < nc ? __ldg(weight + c) : zero, c, inv);
        }
    }
}

// A CTA a block of 128 x 128, 8 rows a thread.
__global__ void __launch_bounds__(kThreads) quantize_squares(const QuantizeArgs a) {
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
    for (int i = 0; i < 8; ++i) {
        float f[8];
        unpack8(v[i], f);
        top = fmaxf(top, top8(f));
    }
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
        const int nc = a.K / 8, threads = nc < kThreads ? (nc + 31) / 32 * 32 : kThreads, parts = (nc + threads - 1) / threads;
        if (parts <= 1) quantize_normed<1><<<a.M, threads, 0, st>>>(a);
        else if (parts <= 2) quantize_normed<2><<<a.M, threads, 0, st>>>(a);
        else if (parts <= 4) quantize_normed<4><<<a.M, threads, 0, st>>>(a);
        else if (parts <= 8) quantize_normed<8><<<a.M, threads, 0, st>>>(a);
        else quantize_normed<0><<<a.M, threads, 0, st>>>(a);
    } else {
        const int wide = (a.K + 255) / 256;
        const long long warps = (long long)((a.M + kRowsAWarp - 1) / kRowsAWarp) * wide;
        quantize_rows<<<(unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32)), kThreads, 0, st>>>(a, wide);
    }
    return cudaGetLastError();
}

}  // namespace mla
