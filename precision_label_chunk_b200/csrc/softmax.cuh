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

// max of three in one instruction
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ float max32(const float (&v)[32]) {
  float x[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
  for (int c = 4; c < 28; c += 8)
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = max3(x[e], v[c + e], v[c + 4 + e]);
  return max3(max3(x[0], x[1], x[2]), max3(x[3], v[28], v[29]), fmaxf(v[30], v[31]));
}

// Partial sums of a row's softmax: m its maximum, s = sum e^(z - m),
// t = sum e^(z - m)(z - m).
struct Stat { float m, s, t; };

// A thread's running m, s and t over scores.  About 5 issue slots a score, one
// of them for the exponential.
struct Soft {
  float m = -INFINITY, s = 0.0f, t = 0.0f;

  __device__ __forceinline__ void raise(float to) {    // m <- to, to >= m
    if (m > -INFINITY) {
      const float dm = fmaxf(m - to, kSoftFloor), c = ex2(dm * kLog2e);
      t = c * fmaf(s, dm, t);
      s *= c;
    }
    m = to;
  }

  // 32 scores with the maximum mx; -inf is cut at the floor, where e^ is 0
  __device__ __forceinline__ void add32(const float (&v)[32], float mx) {
    if (mx > m) raise(mx);
    const float m0 = m > -INFINITY ? m : 0.0f;
    const f2 nm = pair(-m0, -m0);
    float ss, tt;
    sums32([&](int c) {
      float a, b;
      unpair(add2(pair(v[2 * c], v[2 * c + 1]), nm), a, b);
      return pair(max_nan(a, kSoftFloor), max_nan(b, kSoftFloor));
    }, ss, tt);
    if (tt != tt) slow32(v, m0, ss, tt);
    s += ss;
    t += tt;
  }
  // sums over the 16 pairs of differences z - m that diff(c) gives
  template <typename F>
  __device__ __forceinline__ void sums32(F diff, float& ss, float& tt) const {
    const f2 cc = pair(kLog2e, kLog2e);
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
  // one by one: scores of +inf count 1 each beside a maximum of +inf, so that only a NaN makes the sums NaN
  __device__ __forceinline__ void slow32(const float (&v)[32], float m0, float& ss, float& tt) const {
    ss = tt = 0.0f;
#pragma unroll
    for (int c = 0; c < 32; ++c) {
      const float d = v[c] == m0 ? 0.0f : max_nan(v[c] - m0, kSoftFloor), e = ex2(d * kLog2e);
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

// The same over accumulators v of scores inv v, in powers of two: with
// c2 = inv log2(e) and a reference r = fl(c2 max v),
//     s = sum 2^(c2 v - r),   t = sum 2^(c2 v - r)(c2 v - r),
// so that a value takes one multiply-add, the exponential, an addition and a
// multiply-add, two values an instruction but for the exponential.  The score
// that r stands for is r ln 2 without a rounding, whatever c2 max v rounded
// to; c2 v - r is rounded once, to within 2^-24 of its size: c2 itself is off
// by 2^-25, which moves a score by as much of itself, a quarter of what an
// accumulation in fp32 may.  Where |r| passes kFar that rounding of r would
// reach the exponentials' range: there the differences are taken first, one by
// one, and r stands for the maximum itself, to within 2^-24 of it.
struct Soft2 {
  static constexpr float kFar = 1048576.0f;

  float m = -INFINITY, r = 0.0f, s = 0.0f, t = 0.0f;
  float c2;

  __device__ __forceinline__ explicit Soft2(float inv) : c2(inv * kLog2e) {}

  __device__ __forceinline__ void raise(float mx) {    // m <- mx, mx > m
    const float to = mx * c2;
    if (m > -INFINITY) {
      const float d = fmaxf(fabsf(to) > kFar || fabsf(r) > kFar ? (m - mx) * c2 : r - to, -300.0f), c = ex2(d);
      t = c * fmaf(s, d, t);
      s *= c;
    }
    m = mx;
    r = to;
  }

  // 32 accumulators with the maximum mx.  Where one of them is NaN, repair(v) may
  // put others in their place, and says whether it did.
  template <typename F>
  __device__ __forceinline__ void add32(float (&v)[32], float mx, F repair) {
    if (mx > m) raise(mx);
    const f2 cc = pair(c2, c2), nr = pair(-r, -r);
    f2 ps[2] = {pair(0.0f, 0.0f), pair(0.0f, 0.0f)}, pt[2] = {pair(0.0f, 0.0f), pair(0.0f, 0.0f)};
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      const f2 d = fma2(pair(v[2 * c], v[2 * c + 1]), cc, nr);
      float a, b;
      unpair(d, a, b);
      const f2 e = pair(ex2(a), ex2(b));
      ps[c & 1] = add2(ps[c & 1], e);
      pt[c & 1] = fma2(e, d, pt[c & 1]);
    }
    float s0, s1, t0, t1;
    unpair(add2(ps[0], ps[1]), s0, s1);
    unpair(add2(pt[0], pt[1]), t0, t1);
    float ss = s0 + s1, tt = t0 + t1;
    if (tt != tt || fabsf(r) > kFar) {                 // also a score of -inf (0 times infinity), or a NaN
      if (tt != tt && repair(v)) {
        const float to = max32(v);
        if (to > m) raise(to);
      }
      const bool far = fabsf(r) > kFar;
      ss = tt = 0.0f;
      const float m0 = m > -INFINITY ? m : 0.0f;
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        // scores of +inf count 1 each beside a maximum of +inf, as in Soft
        const float d = far && v[c] == m0 ? 0.0f : max_nan(far ? (v[c] - m0) * c2 : fmaf(v[c], c2, -r), -300.0f);
        const float e = ex2(d);
        ss += e;
        tt = fmaf(e, d, tt);
      }
    }
    s += ss;
    t += tt;
  }
};

}  // namespace elmo
