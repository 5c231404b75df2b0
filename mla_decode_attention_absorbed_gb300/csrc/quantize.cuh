// Quantising by blocks of 128: the codes are OCP E4M3, each block has one fp32 scale.
//
//   A = max(max |y|, 2^-100),   scale = A / 448,   code = E4M3(y * (448 / A))
//
// 448 is the largest E4M3 value, so the block's largest value takes the last code and nothing
// saturates; both quotients are rounded once in fp32 (division, so that any program that divides so
// gives the same codes and scales; one that multiplies by a reciprocal, as torch does for 448.0 / t and for t / 448.0 on
// the GPU, has scales off in the last bit and at a tie the neighbouring code).  The 2^-100 keeps 448 / A finite for
// a block of zeros or of values that no result can show.  A NaN keeps its own code and leaves the
// rest of its block alone (fmaxf returns the other operand); an infinity makes A infinite and
// with it every value of the block NaN or 0 x infinity, so that it shows in what is computed.
#pragma once

#include "layer.h"
#include "sm100.cuh"

namespace mla {
namespace quant {

using sm100::mul2;

constexpr int kBlock = 128;
constexpr float kTop = 448.f;
constexpr float kLeast = 0x1p-100f;
constexpr int kScaleBytes = 16;  // of a cache row of blocks: four scales, whatever its width

// Two values as E4M3 codes (v0 in the low byte): nearest even, saturating at +-448.
__device__ __forceinline__ uint32_t e4m3x2(float v0, float v1) {
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(v1), "f"(v0));
    return r;
}
// Two E4M3 codes as values, exactly (every one of them is an fp16 number).
__device__ __forceinline__ float2 from_e4m3x2(uint32_t codes) {
    uint32_t h;
    asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(h) : "r"(codes));
    float2 f;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h));
    return f;
}

__device__ __forceinline__ float2 unpack(uint32_t v) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&v));
}
__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 p = unpack(w[e]);
        f[2 * e] = p.x;
        f[2 * e + 1] = p.y;
    }
}
__device__ __forceinline__ float top8(const float (&f)[8]) {
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[e]));
    return top;
}
// The same of 8 bf16 values as they come, two at a time (max.bf16x2 leaves a NaN out, too).
__device__ __forceinline__ float top8(uint4 v) {
    const uint32_t w[4] = {v.x & 0x7fff7fffu, v.y & 0x7fff7fffu, v.z & 0x7fff7fffu, v.w & 0x7fff7fffu};
    auto pair = [](uint32_t u) { return *reinterpret_cast<const __nv_bfloat162 *>(&u); };
    const float2 f = __bfloat1622float2(__hmax2(__hmax2(pair(w[0]), pair(w[1])), __hmax2(pair(w[2]), pair(w[3]))));
    return fmaxf(fmaxf(f.x, 0.f), f.y);
}
// The largest of 16 neighbouring lanes, which hold a block of 128 values, 8 each.
__device__ __forceinline__ float top16(float top) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    return top;
}
// The same for kN blocks, a power of two up to 8: lane l of the 16 gets that of block l / (16 / kN).  While
// blocks are left to part, lanes trade halves of them: kN = 8 takes 8 trades, one by one 32.
template <int kN>
__device__ __forceinline__ float tops16(float (&top)[kN], int lane) {
    int o = 8;
#pragma unroll
    for (int n = kN / 2; n > 0; n /= 2, o /= 2) {
        const bool upper = lane & o;
#pragma unroll
        for (int i = 0; i < n; ++i)
            top[i] = fmaxf(upper ? top[i + n] : top[i], __shfl_xor_sync(~0u, upper ? top[i] : top[i + n], o));
    }
#pragma unroll
    for (int p = 8 / kN; p > 0; p /= 2) top[0] = fmaxf(top[0], __shfl_xor_sync(~0u, top[0], p));
    return fmaxf(top[0], kLeast);
}
// A division takes as long as all the rest of a block's work for a lane, so each of a block's two is
// made once: of the 16 / kN lanes that have its A, the even ones make 448 / A, the odd ones A / 448.
__device__ __forceinline__ float unit_or_scale(float top, int lane) {
    return __fdiv_rn(lane & 1 ? top : kTop, lane & 1 ? kTop : top);
}
// 448 / A of block `which`, for all of its lanes.
template <int kN>
__device__ __forceinline__ float unit_of(float mine, int lane, int which) {
    return __shfl_sync(~0u, mine, (lane & 16) | which * (16 / kN));
}

__device__ __forceinline__ uint2 codes8(const float (&f)[8], float unit) {
    const float2 both = make_float2(unit, unit);
    uint32_t c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 p = mul2(make_float2(f[2 * e], f[2 * e + 1]), both);
        c[e] = e4m3x2(p.x, p.y);
    }
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

}  // namespace quant
}  // namespace mla
