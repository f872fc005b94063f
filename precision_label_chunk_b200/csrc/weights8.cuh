// weights8.cuh -- eight consecutive weights of a head as they are stored, and
// their values; kFormat is the head's format (elmo_dtype).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/elmo.h"
#include "elmo_common.cuh"

namespace elmo {

template <int kFormat> struct Raw8 { uint2 v; };
template <> struct Raw8<ELMO_BF16> { uint4 v; };

template <int kFormat>
__device__ __forceinline__ void values8(const Raw8<kFormat>& r, float (&w)[8]) {
  if constexpr (kFormat == ELMO_BF16) {
    const uint32_t v[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      w[2 * e] = __uint_as_float(v[e] << 16);
      w[2 * e + 1] = __uint_as_float(v[e] & 0xFFFF0000u);
    }
  } else {
    float a[4], b[4];
    if constexpr (kFormat == ELMO_FP8_E5M2) { e5m2x4_to_f32(r.v.x, a); e5m2x4_to_f32(r.v.y, b); }
    else { e4m3x4_to_f32(r.v.x, a); e4m3x4_to_f32(r.v.y, b); }
#pragma unroll
    for (int e = 0; e < 4; ++e) { w[e] = a[e]; w[4 + e] = b[e]; }
  }
}

}  // namespace elmo
