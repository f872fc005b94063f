// softmax.cuh -- the running softmax of a thread, shared by the kernels that
// form log probabilities from stored scores and from accumulators.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace elmo {

constexpr float kSoftFloor = -200.0f;     // z - m where e^(z - m) is 0 in fp32
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// max(a, b), NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// two fp32 operations an instruction
struct f2 { uint64_t v; };
__device__ __forceinline__ f2 pair(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(f2 p, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p.v)); }
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

__device__ __forceinline__ float max32(const float (&v)[32]) {
  float x[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) x[c] = fmaxf(fmaxf(v[c], v[c + 8]), fmaxf(v[c + 16], v[c + 24]));
  return fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
}

// Partial sums of a row's softmax: m its maximum, s = sum e^(z - m),
// t = sum e^(z - m)(z - m).
struct Stat { float m, s, t; };

// A thread's running m, s and t over values v whose scores are inv v; m and t
// are in the values' units (inv m, inv t are the scores').  About 4 issue
// slots a value (5 with kMasks), one of them for the exponential.
struct Soft {
  float m = -INFINITY, s = 0.0f, t = 0.0f;
  float c2, floor_v;                                   // inv log2(e); -200 / inv

  __device__ __forceinline__ explicit Soft(float inv) : c2(inv * kLog2e), floor_v(kSoftFloor / inv) {}

  __device__ __forceinline__ void raise(float to) {    // m <- to, to >= m
    if (m > -INFINITY) {
      const float dm = fmaxf(m - to, floor_v), c = ex2(dm * c2);
      t = c * fmaf(s, dm, t);
      s *= c;
    }
    m = to;
  }

  // 32 values with the maximum mx.  kMasks: values of -inf are ordinary (they
  // are cut at the floor, where e^ is 0); else they are rare, and a product 0
  // times infinity sends the 32 values through the sums again (add32_slow).
  template <bool kMasks>
  __device__ __forceinline__ void add32(const float (&v)[32], float mx) {
    if (mx > m) raise(mx);
    const float m0 = m > -INFINITY ? m : 0.0f;
    float ss, tt;
    sums32<kMasks>(v, m0, ss, tt);
    if (!kMasks && tt != tt) slow32(v, m0, ss, tt);
    s += ss;
    t += tt;
  }
  template <bool kMasks>
  __device__ __forceinline__ void sums32(const float (&v)[32], float m0, float& ss, float& tt) const {
    const f2 nm = pair(-m0, -m0);
    sums32_of([&](int c) {
      f2 d = add2(pair(v[2 * c], v[2 * c + 1]), nm);
      if (kMasks) {
        float a, b;
        unpair(d, a, b);
        d = pair(max_nan(a, floor_v), max_nan(b, floor_v));
      }
      return d;
    }, ss, tt);
  }
  // sums over the 16 pairs of differences v - m that diff(c) gives
  template <typename F>
  __device__ __forceinline__ void sums32_of(F diff, float& ss, float& tt) const {
    const f2 cc = pair(c2, c2);
    f2 ps[2] = {pair(0.0f, 0.0f), pair(0.0f, 0.0f)}, pt[2] = {pair(0.0f, 0.0f), pair(0.0f, 0.0f)};
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      const f2 d = diff(c);
      float a, b;
      unpair(mul2(d, cc), a, b);
      const f2 e = pair(ex2(a), ex2(b));
      ps[c & 1] = add2(ps[c & 1], e);
      pt[c & 1] = fma2(e, d, pt[c & 1]);
    }
    float s0, s1, t0, t1;
    unpair(add2(ps[0], ps[1]), s0, s1);
    unpair(add2(pt[0], pt[1]), t0, t1);
    ss = s0 + s1;
    tt = t0 + t1;
  }
  __device__ __forceinline__ void slow32(const float (&v)[32], float m0, float& ss, float& tt) const {
    ss = tt = 0.0f;
#pragma unroll
    for (int c = 0; c < 32; ++c) {
      const float d = max_nan(v[c] - m0, floor_v), e = ex2(d * c2);
      ss += e;
      tt = fmaf(e, d, tt);
    }
  }

  // the warp's sums in every lane
  __device__ __forceinline__ void join_warp() {
    float mx = m;
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
    if (mx > m) raise(mx);
    for (int o = 16; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
      t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    }
  }
};

}  // namespace elmo
