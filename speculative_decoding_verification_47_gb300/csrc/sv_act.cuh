// Activations of the products' epilogues.
#pragma once

#include "sv_common.cuh"
#include "sv_internal.h"

namespace sv {
namespace lin {

__device__ __forceinline__ float silu(float z) { return __fdividef(z, 1.f + __expf(-z)); }
// z times the normal distribution's mass below z, by its upper tail
//   1/2 erfc(a / sqrt 2) = exp(-a^2 / 2) t Q(t),  a = |z|, t = 1 / (1 + 0.3075914 a),
// Q of degree 7, fitted here to the least relative error (reweighted least squares over
// a = 0 .. 15.5: 1.3e-7).  A relative error, since a tail's error is one of the result
// where z is negative: a form whose error is absolute (3e-7) is off by 0.4% at z = -4.
// An infinite z has a tail of 0.
__device__ __forceinline__ float gelu(float z) {
  const float t = __fdividef(1.f, __fmaf_rn(0.30759143f, fabsf(z), 1.f));
  float p = __fmaf_rn(0.03628622f, t, -0.14713992f);
  p = __fmaf_rn(p, t, 0.16964923f);
  p = __fmaf_rn(p, t, -0.02564602f);
  p = __fmaf_rn(p, t, 0.11512012f);
  p = __fmaf_rn(p, t, 0.10576703f);
  p = __fmaf_rn(p, t, 0.12327711f);
  p = __fmaf_rn(p, t, 0.12268629f);
  const float tail = p * t * ex2(z * z * -0.72134752f);  // (log2(e) / 2)
  return z * (z > 0.f ? 1.f - tail : tail);
}
// z / 2 (1 + tanh u) = z / (1 + exp(-2u))
__device__ __forceinline__ float gelu_tanh(float z) {
  const float u = 0.79788456080286536f * (z + 0.044715f * z * z * z);
  return __fdividef(z, 1.f + __expf(-2.f * u));
}

// the activation of n values (one test of `act` for all of them)
template <int n>
__device__ __forceinline__ void activate(float (&z)[n], int act) {
  if (act == SV_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < n; ++i) z[i] = z[i] < 0.f ? 0.f : z[i];  // (a NaN stays)
  } else if (act == SV_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < n; ++i) z[i] = silu(z[i]);
  } else if (act == SV_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < n; ++i) z[i] = gelu(z[i]);
  } else if (act == SV_ACT_GELU_TANH) {
#pragma unroll
    for (int i = 0; i < n; ++i) z[i] = gelu_tanh(z[i]);
  }
}

}  // namespace lin
}  // namespace sv
