// Rotary angles: cos and sin of position . frequency for positions below 2^31.
//
// The angle is taken in turns, as a 64-bit fraction: the plan holds each
// frequency as turn = f / (2 pi) in units of 2^-64, and position * turn modulo
// 2^64 is the fraction of a turn left after whole turns, exactly (integer
// multiplication wraps at one turn).  Its top 32 bits, signed, are the angle in
// [-pi, pi) to 2^-32 turns, the same for near and far positions; a float product
// position * f would be off by 2^-24 of the whole angle, 60 radians at 2^30.
#pragma once

#include "common.cuh"

namespace mla {

__device__ __forceinline__ float2 rope_cos_sin(unsigned long long turn, int position, float mscale, float sign) {
    const unsigned long long u = turn * (unsigned long long)(unsigned)position;
    const float x = (float)(int)(u >> 32) * 0x1p-31f;  // half turns in [-1, 1)
    float s, c;
    sincospif(x, &s, &c);
    return make_float2(mscale * c, sign * mscale * s);
}

__device__ __forceinline__ float2 rope_turn(float u, float v, float2 cs) {
    return make_float2(u * cs.x - v * cs.y, u * cs.y + v * cs.x);
}

}  // namespace mla
