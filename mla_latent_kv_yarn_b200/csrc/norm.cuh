// Pieces of the root-mean-square norms: the norm factor of a vector held by a
// warp, and the rotation's cosine and sine in float32 from an exact position.
#pragma once

#include <cstdint>

#include "xmla_device.cuh"
#include "yarn.cuh"

namespace xmla {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// 1 / sqrt(mean of the squares + eps) of n values whose squares sum to sq (a
// float32 sum; correctly rounded root and quotients).
__device__ __forceinline__ float rms_factor(float sq, int n, float eps) {
  return 1.f / sqrtf(sq / (float)n + eps);
}

// Cosine and sine of pos * inv_freq, times the table's magnitude.  The angle in
// half turns and its remainder modulo a whole turn are formed in float64, so what
// float32 adds is the rounding of an angle in [-pi, pi] and of the result, some
// 2^-22, far below a bf16 step at any position.
__device__ __forceinline__ void rope_cos_sin(int64_t pos, double inv_freq, float magnitude,
                                             float* c, float* s) {
  const double half_turns = (double)pos * inv_freq * 0.3183098861837907;
  sincospif((float)fma(-2.0, rint(0.5 * half_turns), half_turns), s, c);
  *c *= magnitude;
  *s *= magnitude;
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(w[e] << 16);
    x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
    w[e] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// What a vector's values are to be multiplied by before they are squared, given the
// float32 sum sq of their plain squares: 1, unless that sum overflowed (|x| from
// 2^59 on) or mean and eps together are so small that squares were lost below the
// normal range.  bf16 values times 2^-70 are below 2^58, and 1024 squares of them
// below 2^126; values that take 2^90 (under 2^-45 for 1024 of them) stay below 2^45,
// and the smallest bf16 value becomes 2^-43.  The norm is then (x S) * (f w) with f =
// rms_factor(sum of (x S)^2, n, eps S S): the power of two cancels, and S = 1, the
// usual case, changes nothing.
__device__ __forceinline__ float rms_scale(float sq, int n, float eps) {
  const float v = sq / (float)n + eps;
  return v < 0x1p-100f ? 0x1p90f : v < INFINITY ? 1.f : 0x1p-70f;
}

}  // namespace xmla
