// The SwiGLU activation's sigmoid on the device.
#pragma once

#include "moe_internal.h"

namespace moe {

// 1 / (1 + e^-g) for g >= kFar. For bf16 results the hardware's exp2 and reciprocal (each within
// one unit of fp32, and the product with log2 e within |g| 2^-24) are far inside the result's
// rounding.
template <typename T>
__device__ __forceinline__ float sigmoid(float g) {
  if constexpr (sizeof(T) == 2) return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504088896f));
  else return 1.0f / (1.0f + expf(-g));
}

// Below kFar s = e^g leaves the normal fp32 numbers (2^-126 at g = -87.3): the reciprocal would flush
// it to 0 and, from -88.7 on, e^-g would overflow, however large the factors that s meets. There the
// products are taken in 64 bits and rounded to fp32 once, with s = (e^(g/4))^4: a quarter's power
// is a normal fp32 number down to g = -349, where s is under 2^-503 and every product with fp32
// factors is 0. One comparison per 8 elements where no g is that low; these results are stored over
// the ordinary ones, which need not wait for them then (65,536 rows of 2048 forward and back: 387.2 us
// without this, 388.0 with it, 389.4 where one store comes after the branch).
constexpr float kFar = -87.0f;
template <typename T>
__device__ __forceinline__ double far_sigmoid(float g) {
  // bf16: the hardware's exp2 and the product with log2 e leave s within 2^-15 of itself, inside the rounding
  const double q = sizeof(T) == 2 ? __builtin_amdgcn_exp2f(g * (0.25f * 1.44269504088896f)) : expf(0.25f * g);
  return (q * q) * (q * q);
}

}  // namespace moe
