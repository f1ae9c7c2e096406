// rope.cuh -- angles of the rotary positions, shared by the kernels that rotate.
//
// Pair i of a token at position p turns by p * f_i radians.  In 32-bit floats
// that product is wrong by whole turns' worth of rounding at far positions
// (p = 10^6 and f = 1 leave 0.06 rad), and 64-bit floats are slow here.  The
// plan therefore holds f_i / 2 pi as a 64-bit fraction of a turn: the product
// with the position, taken modulo 2^64, is the angle modulo one turn exactly,
// for any 32-bit position, in integer arithmetic (f_i itself is a 64-bit float's).  Read as a signed number it
// lies in [-1/2, 1/2) turns and is rounded once to 32 bits.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "libmla.h"

namespace mla {

// (cos, sin) of pair `i`'s angle at position `pos`, times the plan's factor.
static __device__ __forceinline__ float2 rope_cos_sin(uint64_t turns, int pos, float factor) {
    const int64_t t = (int64_t)(turns * (uint64_t)(int64_t)pos);
    float s, c;
    sincospif(__ll2float_rn(t) * 1.0842021724855044e-19f, &s, &c);   // 2^-63: half turns per unit
    return make_float2(c * factor, s * factor);
}

static __device__ __forceinline__ float to_float(float x) { return x; }
static __device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
static __device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

}  // namespace mla
