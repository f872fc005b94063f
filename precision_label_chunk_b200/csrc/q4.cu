// q4.cu -- a head held in 4 bits: codes with a scale for every group of
// consecutive weights of a label, made from the head's weights, read back, and
// multiplied with a few queries.
//
// The classifier head dominates the model's memory ("ELMO: Efficiency via
// Low-precision and Peak Memory Optimization in Large Output Spaces",
// abstract); a query reads all of it, so the time of serving a few queries is
// that of reading the head, and a quarter of the bytes is a quarter of it.
//
// Format.  A group of G (32, 64 or 128) weights of one label has the bf16
// scale s = bf16(max|w| / 7) and codes u = rne(w / s) + 8, so that w stands
// for s (u - 8); two codes a byte, the even element in the low nibble.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "elmo_common.cuh"
#include "elmo_internal.h"
#include "elmo_operators.h"
#include "tc_ptx.cuh"
#include "weights8.cuh"

namespace elmo {
namespace {

using namespace tc;

// ---------------------------------------------------------------- pack, unpack
// Rows are whole groups, so the matrix is one run of groups: a thread takes
// eight consecutive weights, the G / 8 threads of a group share their maximum.
//
// w / s is rounded to the nearest whole number without a division: with
// r = 1 / s to within a few units in the last place, t = w r is near w / s,
// and w / s is either exactly k + 1/2 or at least 2^-9 away from it (w and s
// have 8-bit significands a 2^e and b 2^f; near k + 1/2 >= 1/2 they have
// e >= f - 1, so w / s - (k + 1/2) is a multiple of 1 / (2 b)).  Rounding t to
// a multiple of 2^-13 (the sum with 1.5 2^10) therefore restores exact ties
// and moves nothing else across one, and the sum that brings 1.5 2^23 + 8 into
// its place then rounds ties to even and leaves the code in the low byte.
// Likewise max / 7 rounds to bf16 as max times fl(1 / 7) does: 7 times a
// midpoint of that grid has more bits than max, so max / 7 stays 1 / 14 of a
// step away from every midpoint.  Scales below 2^-100, whose own rounding may
// be coarse, take the division.
//
// bf16 is HBM-bound: the bytes of W, half a byte a weight, the scales.  A thread has
// kPackAt vectors in flight, each warp access contiguous (16 weights a thread,
// two vectors apart, measured 214 us for 500K bf16 labels x 768).  On B200, for
// those in groups of 64: 162 us to pack (6.0 TB/s), 160 us to unpack (6.1 TB/s).
// 8-bit weights have half the bytes and more to do for each: E4M3 177 us (issue
// slots 82 % busy, ALU 70, DRAM 36), E5M2 152.
constexpr int kPackThreads = 256;
constexpr int kPackAt = 4;

// the largest magnitude's code of eight weights, and a code's value
template <int kFormat> __device__ __forceinline__ uint32_t code_max(const Raw8<kFormat>& r) {
  if constexpr (kFormat == ELMO_BF16) {
    constexpr uint32_t k = 0x7FFF7FFFu;
    const uint32_t m = __vmaxu2(__vmaxu2(r.v.x & k, r.v.y & k), __vmaxu2(r.v.z & k, r.v.w & k));
    return max(m & 0xFFFFu, m >> 16);
  } else {
    constexpr uint32_t k = 0x7F007F00u;
    const uint32_t m = __vmaxu2(__vmaxu2(r.v.x & k, (r.v.x << 8) & k), __vmaxu2(r.v.y & k, (r.v.y << 8) & k));
    return max(m & 0xFFFFu, m >> 16) >> 8;
  }
}
template <int kFormat> __device__ __forceinline__ float code_value(uint32_t m) {
  if constexpr (kFormat == ELMO_BF16) return bf16_to_f32((uint16_t)m);
  else if constexpr (kFormat == ELMO_FP8_E5M2) return e5m2_to_f32((uint8_t)m);
  else return e4m3_to_f32((uint8_t)m);
}

// sum over e of 16^e times the bits of 1.5 2^23 (0x4B400000), mod 2^32
constexpr uint32_t kCodeBits = 0x4B400000u * 0x11111111u;

// kLanes threads share a group.
template <int kFormat, int kLanes>
__global__ void __launch_bounds__(kPackThreads) q4_pack_kernel(const Raw8<kFormat>* __restrict__ W, int64_t n8,
                                                               uint32_t* __restrict__ codes,
                                                               uint16_t* __restrict__ scales) {
  // every thread of a warp stays for the shuffles; groups never straddle warps
  const int64_t stride = (int64_t)gridDim.x * kPackThreads * kPackAt;
  for (int64_t i0 = (int64_t)blockIdx.x * kPackThreads * kPackAt + threadIdx.x; i0 - threadIdx.x < n8; i0 += stride) {
    const int left = (int)min(n8 - i0, (int64_t)kPackThreads * kPackAt);   // vectors from this thread's first on
    const Raw8<kFormat>* from = W + i0;
    uint32_t* to = codes + i0;
    uint16_t* sc = scales + (uint64_t)i0 / kLanes;
    Raw8<kFormat> raw[kPackAt];
#pragma unroll
    for (int u = 0; u < kPackAt; ++u) {
      if (u * kPackThreads < left) raw[u].v = __ldcs(&from[u * kPackThreads].v);
      else raw[u] = Raw8<kFormat>{};
    }
#pragma unroll
    for (int u = 0; u < kPackAt; ++u) {
      float w[8];
      values8<kFormat>(raw[u], w);
      uint32_t m = code_max<kFormat>(raw[u]);          // magnitudes' codes order them, NaN above inf
#pragma unroll
      for (int o = kLanes >> 1; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      const float big = code_value<kFormat>(m);
      const uint16_t sb = big < INFINITY ? f32_to_bf16_rn(__fmul_rn(big, 1.0f / 7.0f)) : (uint16_t)0x7FC0u;
      const float s = bf16_to_f32(sb);
      uint32_t q = 0;
      if (s >= 0x1p-100f) {
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
#pragma unroll
        for (int e = 7; e >= 0; --e) {
          // |t| <= 7 (1 + 2^-8): the sum's bits are those of 1.5 2^23 plus the code
          const float t = __fadd_rn(__fmul_rn(w[e], r), 1536.0f);
          q = (q << 4) + __float_as_uint(__fadd_rn(t, 12582920.0f - 1536.0f));
        }
        q -= kCodeBits;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float t = s > 0.0f ? rintf(__fdiv_rn(w[e], s)) : 0.0f;   // NaN and zero scales: code 8
          t = fminf(fmaxf(t, -8.0f), 7.0f);
          q |= (uint32_t)((int)t + 8) << (4 * e);
        }
      }
      if (u * kPackThreads < left) {
        __stcs(to + u * kPackThreads, q);
        if (threadIdx.x % kLanes == 0) sc[u * (kPackThreads / kLanes)] = sb;
      }
    }
  }
}

// Eight codes -> eight values (u - 8) s in bf16, each rounded once: 0x4300 | u
// is the bf16 number 128 + u, 136 is subtracted exactly, and the product with
// the scale rounds.
__device__ __forceinline__ uint4 q4_values8(uint32_t c, __nv_bfloat162 s2) {
  const __nv_bfloat162 off = __halves2bfloat162(__ushort_as_bfloat16(0x4308), __ushort_as_bfloat16(0x4308));
  uint32_t o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t b = c >> (8 * e);
    const uint32_t v = 0x43004300u | (b & 0xFu) | ((b & 0xF0u) << 12);
    const __nv_bfloat162 q = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), off);
    const __nv_bfloat162 w = __hmul2(q, s2);
    o[e] = *reinterpret_cast<const uint32_t*>(&w);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

__global__ void __launch_bounds__(kPackThreads) q4_unpack_kernel(const uint32_t* __restrict__ codes,
                                                                 const uint16_t* __restrict__ scales, int64_t n8,
                                                                 int shift, uint4* __restrict__ W) {
  const int64_t stride = (int64_t)gridDim.x * kPackThreads * kPackAt;
  for (int64_t i0 = (int64_t)blockIdx.x * kPackThreads * kPackAt + threadIdx.x; i0 < n8; i0 += stride) {
    uint32_t c[kPackAt];
    uint16_t s[kPackAt];
#pragma unroll
    for (int u = 0; u < kPackAt; ++u) {
      const int64_t i = i0 + u * kPackThreads;
      if (i < n8) {
        c[u] = __ldcs(codes + i);
        s[u] = __ldg(scales + (i >> shift));
      }
    }
#pragma unroll
    for (int u = 0; u < kPackAt; ++u) {
      const int64_t i = i0 + u * kPackThreads;
      const __nv_bfloat16 one = __ushort_as_bfloat16(s[u]);
      if (i < n8) __stcs(W + i, q4_values8(c[u], __halves2bfloat162(one, one)));
    }
  }
}

int flat_grid(int64_t vectors) {
  const int64_t per = kPackThreads * kPackAt, want = (vectors + per - 1) / per, most = (int64_t)current_sms() * 32;
  return (int)(want < most ? want : most);
}

template <int kFormat>
cudaError_t run_pack(const void* W, int64_t n8, int32_t group, uint32_t* codes, uint16_t* scales, cudaStream_t s) {
  const Raw8<kFormat>* w = static_cast<const Raw8<kFormat>*>(W);
  const int grid = flat_grid(n8);
  if (group == 32) q4_pack_kernel<kFormat, 4><<<grid, kPackThreads, 0, s>>>(w, n8, codes, scales);
  else if (group == 64) q4_pack_kernel<kFormat, 8><<<grid, kPackThreads, 0, s>>>(w, n8, codes, scales);
  else q4_pack_kernel<kFormat, 16><<<grid, kPackThreads, 0, s>>>(w, n8, codes, scales);
  return cudaGetLastError();
}

// ---------------------------------------------------------------- scores
// Z[b, l] = sum_g s[l, g] sum_{j in g} x[b, j] (u[l, j] - 8).
//
// Warp w of a CTA owns 16 kMT labels of a tile as the M rows of m16n8k16
// matrix instructions (fp16 operands, fp32 sums), queries are the N columns.
// These instructions take A from registers, where the codes are unpacked; the
// tcgen05 ones would need them written back to shared memory at four times
// the bytes, and with at most a few dozen columns the tensor pipe is idle
// either way.
//
// Codes: a TMA ring of 128-byte boxes (256 codes of every label of the tile,
// 128-byte swizzle).  Thread (g, t) of a warp (g = lane / 4, t = lane % 4)
// holds, for its rows, the G / 4 consecutive codes t of each group: the K
// order inside a group is free as long as X follows it, and all K slots of an
// instruction lie in one group, so the group's sum comes out on its own in
// fp32 and is scaled in fp32.  The row of a tile that a fragment row stands
// for is chosen so that the shared loads have no bank conflicts.
//
// Codes to fp16 numbers: a nibble in bits 0-3 with 0x6400 is 1024 + u, in bits
// 4-7 it is 1024 + 16 u; one subtraction, or one multiply-add with 1/16, gives
// u - 8 exactly.  Nine instructions for eight codes.
//
// X: fp16 in fragment order, each query scaled by the power of two that puts
// its largest magnitude into [2^14, 2^15).  A bf16 number's 8 bits fit fp16's
// 11; numbers below 2^-31 of the query's largest are rounded, to within 2^-39
// of it, which is far below the fp32 sums' own rounding.
// The scaling is undone last, so that the sums may overflow where the score does
// not.  They stay below d 2^18 times the label's largest scale, so only scales of
// 2^97 and more can do that: q4_scores_again (3M labels x 768, all scales so
// large: 1.7 ms for 1 query, 37 for 32).  Where it stands matters, and that
// nothing of it lives on in the loop over the tiles: called from that loop it
// cost registers, 124 us for 500K labels and 32 queries in place of 109.
//
// Bound by no unit alone (1M labels, one query: issue slots 62 %, DRAM 57, ALU
// 49; seven queries much the same): on B200, 3M labels x 768 in groups of 64 and
// one query take 257 us in a loop (1.24 GB, 4.8 TB/s); the same ring with the
// arithmetic left out takes 203.  500K labels, groups of 128, seven queries: 48
// us; groups of 64, 32 queries: 107.
// Eight warps of labels in place of sixteen took 307 us against 237; 24 warps,
// larger requests and whole rows a stage changed nothing.
constexpr int kQKB = 128;                 // bytes of a box's row: 256 codes
constexpr int kQMaxStages = 8;
constexpr long long kQWait = 4000000000LL;
constexpr size_t kQSmem = 225 * 1024;     // of the 227 KB a CTA may have
constexpr uint32_t kQLarge = (97 + 127) << 7;   // 2^97 in bf16
constexpr int kQMaxNB = 4;                // 8-query column blocks of one pass

template <int kG> __device__ __forceinline__ int q4_row(int g) {
  // 16-byte loads go by quarter warps (rows g, g + 1), 8-byte loads by half warps (4 rows)
  if (kG == 128) return ((g & 1) << 2) | (g >> 1);
  if (kG == 64) return ((g & 3) << 1) | (g >> 2);
  return g;
}

template <int kWords> __device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&v)[kWords]);
template <> __device__ __forceinline__ void lds_words<1>(uint32_t addr, uint32_t (&v)[1]) {
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v[0]) : "r"(addr));
}
template <> __device__ __forceinline__ void lds_words<2>(uint32_t addr, uint32_t (&v)[2]) {
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(addr));
}
template <> __device__ __forceinline__ void lds_words<4>(uint32_t addr, uint32_t (&v)[4]) {
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr));
}

// (a & mask) | magic in one instruction: of two constants the compiler makes
// two, which kept the integer pipe 63 % busy (3M labels, one query: 286 us
// against 245), so the magic number comes in a register.
__device__ __forceinline__ uint32_t mask_or(uint32_t a, uint32_t mask, uint32_t magic) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(mask), "r"(magic));
  return r;
}
__device__ __forceinline__ uint32_t q4_magic() {
  uint32_t r;
  asm("mov.b32 %0, 0x64006400;" : "=r"(r));
  return r;
}

// 8 codes (elements 0..7, nibble i = element i) -> pairs (0,4), (1,5), (2,6), (3,7) of u - 8
__device__ __forceinline__ void q4_pairs(uint32_t c, uint32_t magic, uint32_t (&p)[4]) {
  const uint32_t hi = c >> 8;
  const __half2 m1032 = __half2half2(__ushort_as_half(0x6408));          // 1032
  const __half2 r16 = __half2half2(__ushort_as_half(0x2C00));            // 1 / 16
  const __half2 m72 = __half2half2(__ushort_as_half(0xD480));            // -72
  const uint32_t w[4] = {mask_or(c, 0x000F000Fu, magic), mask_or(c, 0x00F000F0u, magic),
                         mask_or(hi, 0x000F000Fu, magic), mask_or(hi, 0x00F000F0u, magic)};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __half2 v = *reinterpret_cast<const __half2*>(&w[e]);
    const __half2 q = (e & 1) ? __hfma2(v, r16, m72) : __hsub2(v, m1032);
    p[e] = *reinterpret_cast<const uint32_t*>(&q);
  }
}

// d = a b, and d += a b
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%10, %10, %10, %10};"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// 2^e as two factors that are normal numbers (|e| <= 250)
__device__ __forceinline__ void pow2_factors(int e, float& f0, float& f1) {
  f0 = __uint_as_float((uint32_t)(127 + e / 2) << 23);
  f1 = __uint_as_float((uint32_t)(127 + e - e / 2) << 23);
}

struct SmemQ {
  uint64_t full[kQMaxStages], empty[kQMaxStages];
  int32_t exponent[8 * kQMaxNB];
  int32_t finite[8 * kQMaxNB];          // whether the query is
  volatile int odd[17];                 // whether a warp has met a sum that is not finite
  int abort;
};

// Rows of a TMA box: at most 256.
constexpr int q4_box(int tile) { return tile / ((tile + 255) / 256); }

// Shared memory beside the ring: X's fragments, two tiles of scales.
template <int kMT, int kNB, int kWarps>
size_t q4_fixed(int d, int group) {
  return 1024 + (size_t)d * kNB * 16 + (size_t)4 * 16 * kMT * kWarps * (d / group) + sizeof(SmemQ);
}

struct Q4Args {
  const uint8_t* codes;
  const uint16_t* scales;
  const uint16_t* X;
  float* Z;
  int64_t L, ldz;
  int32_t d, B, stages;
};

// After the last tile, for a warp that has met a sum that is not finite: the
// scores of its labels with a scale of kQLarge or more that are not finite, of
// queries and scales that are, again in 64 bits.
template <int kG, int kRows, int kTile>
__device__ __noinline__ void q4_scores_again(const Q4Args A, const int32_t* finite, int queries) {
  const int lane = threadIdx.x & 31, b0 = blockIdx.y * queries;
  for (int64_t tile = (int64_t)blockIdx.x * kTile; tile < A.L; tile += (int64_t)gridDim.x * kTile) {
    const int64_t l = tile + (threadIdx.x >> 5) * kRows + lane % kRows;
    if (l >= A.L) continue;
    const uint8_t* codes = A.codes + l * (A.d / 2);
    const uint16_t* scales = A.scales + l * (A.d / kG);
    uint32_t most = 0;
    for (int g = 0; g < A.d / kG; ++g) most = max(most, scales[g] & 0x7FFFu);
    if (most < kQLarge || most >= 0x7F80u) continue;
    for (int n = lane / kRows; n < queries && b0 + n < A.B; n += 32 / kRows) {
      float* to = A.Z + (int64_t)(b0 + n) * A.ldz + l;
      if (!finite[n] || fabsf(*to) < INFINITY) continue;
      const uint16_t* x = A.X + (size_t)(b0 + n) * A.d;
      double z = 0.0;
      for (int g = 0; g < A.d / kG; ++g) {
        double sum = 0.0;
        for (int j = g * kG; j < (g + 1) * kG; j += 8) {
          const uint32_t u = __ldg(reinterpret_cast<const uint32_t*>(codes + j / 2));
          for (int e = 0; e < 8; ++e) sum += (double)bf16_to_f32(x[j + e]) * ((int)(u >> (4 * e) & 15u) - 8);
        }
        z += (double)bf16_to_f32(scales[g]) * sum;
      }
      *to = (float)z;
    }
  }
}

// kMT: 16-label blocks of a warp; kNB: 8-query blocks of this pass (grid.y
// walks over the batch 8 kNB queries at a time); kWarps warps of labels and
// one for the TMA.
template <int kG, int kMT, int kNB, int kWarps>
__global__ void __launch_bounds__(32 * (kWarps + 1), 1)
    q4_scores_kernel(const __grid_constant__ CUtensorMap tmQ, const Q4Args A) {
  constexpr int kRows = 16 * kMT;                    // labels of a warp
  constexpr int kTile = kRows * kWarps;              // labels of a tile
  constexpr uint32_t kStage = kTile * kQKB;
  constexpr int kBox = q4_box(kTile);
  constexpr int kWords = kG / 32;                    // words of 8 codes a thread has of a group and row
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int ng = A.d / kG;                           // groups of a label
  uint4* xs = reinterpret_cast<uint4*>(ring + (size_t)A.stages * kStage);          // [ng * kWords][kNB][32]
  uint16_t* sc = reinterpret_cast<uint16_t*>(xs + (size_t)ng * kWords * kNB * 32); // [2][kTile][ng]
  SmemQ* S = reinterpret_cast<SmemQ*>(sc + (size_t)2 * kTile * ng);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int b0 = blockIdx.y * 8 * kNB;
  const int64_t T = (A.L + kTile - 1) / kTile;
  const int nkb = (A.d / 2 + kQKB - 1) / kQKB;
  volatile int* abort = &S->abort;

  if (threadIdx.x == 0) {
    for (int s = 0; s < A.stages; ++s) { mbar_init(&S->full[s], 1); mbar_init(&S->empty[s], kWarps); }
    S->abort = 0;
    for (int w = 0; w <= kWarps; ++w) S->odd[w] = 0;
    fence_barrier_init();
  }
  __syncthreads();

  if (warp == kWarps) {
    if (elect_one()) {
      tma_prefetch_desc(&tmQ);
      uint32_t s = 0, ph = 1;
      for (int64_t tile = blockIdx.x; tile < T && !*abort; tile += gridDim.x) {
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(&S->empty[s], ph, abort, kQWait)) { *abort = 1; break; }
          mbar_arrive_expect_tx(&S->full[s], kStage);
          for (int r = 0; r < kTile; r += kBox)
            tma_load_2d(ring + (size_t)s * kStage + (size_t)r * kQKB, &tmQ, &S->full[s], kb * kQKB, (int32_t)(tile * kTile + r));
          if (++s == (uint32_t)A.stages) { s = 0; ph ^= 1; }
        }
      }
    }
  }

  // X into fragment order.  The exponents first: warp w takes queries w, w + kWarps, ...
  if (warp < kWarps) {
    for (int n = warp; n < 8 * kNB; n += kWarps) {
      uint32_t m = 0, most = 0;
      if (b0 + n < A.B) {
        const uint4* xr = reinterpret_cast<const uint4*>(A.X + (size_t)(b0 + n) * A.d);
        for (int j = lane; j < A.d / 8; j += 32) {
          const uint4 v = xr[j];
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t lo = w[e] & 0x7FFFu, hi = (w[e] >> 16) & 0x7FFFu;
            if (lo < 0x7F80u) m = max(m, lo);          // the largest finite magnitude
            if (hi < 0x7F80u) m = max(m, hi);
            most = max(most, max(lo, hi));
          }
        }
        for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      }
      most = __reduce_max_sync(0xFFFFFFFFu, most);
      if (lane == 0) {
        S->exponent[n] = m == 0 ? 0 : 141 - max((int)(m >> 7), 1);
        S->finite[n] = most < 0x7F80u;
      }
    }
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
    const int nf = ng * kWords * kNB * 32;
    for (int f = threadIdx.x; f < nf; f += 32 * kWarps) {
      const int ln = f & 31, nb = (f >> 5) % kNB, jw = (f >> 5) / kNB;
      const int j = jw / kWords, w = jw % kWords;
      const int n = nb * 8 + (ln >> 2);
      uint4 o = make_uint4(0u, 0u, 0u, 0u);
      if (b0 + n < A.B) {
        const int k = j * kG + (ln & 3) * (kG / 4) + 8 * w;
        const uint4 v = *reinterpret_cast<const uint4*>(A.X + (size_t)(b0 + n) * A.d + k);
        const uint32_t x[4] = {v.x, v.y, v.z, v.w};
        float f0, f1;
        pow2_factors(S->exponent[n], f0, f1);
        __half h[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          h[2 * i] = __float2half_rn(__uint_as_float(x[i] << 16) * f0 * f1);
          h[2 * i + 1] = __float2half_rn(__uint_as_float(x[i] & 0xFFFF0000u) * f0 * f1);
        }
        uint32_t p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __half2 q = __halves2half2(h[i], h[i + 4]);
          p[i] = *reinterpret_cast<const uint32_t*>(&q);
        }
        o = make_uint4(p[0], p[1], p[2], p[3]);
      }
      xs[f] = o;
    }
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");

    // the scales of this warp's labels of a tile: one run of 2 ng kRows bytes
    // (a multiple of 16, as its start is), cut at the matrix's end
    uint16_t* my_sc = sc + (size_t)warp * kRows * ng;
    auto fetch_scales = [&](int64_t tile, int buf) {
      const int64_t l0 = tile * kTile + (int64_t)warp * kRows;
      const int64_t end = A.L * ng * 2;
      const uint32_t dst = smem_u32(my_sc + (size_t)buf * kTile * ng);
      for (int c = lane; c < kRows * ng / 8; c += 32) {
        const int64_t off = l0 * ng * 2 + (int64_t)c * 16;
        const int64_t left = end - off;
        const uint32_t n = left >= 16 ? 16u : (left > 0 ? (uint32_t)left : 0u);
        cp_async16(dst + c * 16, reinterpret_cast<const uint8_t*>(A.scales) + (n ? off : 0), n);
      }
      cp_async_commit();
    };
    if ((int64_t)blockIdx.x < T) fetch_scales(blockIdx.x, 0);

    constexpr int kGroupsStage = 2 * kQKB / kG;
    const uint32_t magic = q4_magic();
    uint32_t s = 0, ph = 0;
    int buf = 0;
    const int row0 = warp * kRows + q4_row<kG>(g);     // of the tile: fragment rows g, g + 8 are rows row0, row0 + 8
    // byte t kG / 8 of a row's group j, swizzled; rows row0 + 8 i share row & 7
    const uint32_t mine = smem_u32(ring) + (uint32_t)row0 * kQKB, swz = (uint32_t)(row0 & 7) << 4;
    float odd = 0.0f;                                  // NaN from the first sum that is not finite on
    for (int64_t tile = blockIdx.x; tile < T; tile += gridDim.x, buf ^= 1) {
      cp_async_wait();
      __syncwarp();
      if (tile + gridDim.x < T) fetch_scales(tile + gridDim.x, buf ^ 1);
      float out[kMT][kNB][4];
#pragma unroll
      for (int m = 0; m < kMT; ++m)
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) out[m][nb][e] = 0.0f;
      const uint16_t* ts = sc + (size_t)buf * kTile * ng + (size_t)row0 * ng;
      const uint4* xp = xs + lane;
      bool ok = true;
      // one group: its sum in fp32, then times the labels' scales
      auto group = [&](uint32_t st, int j) {
        const uint32_t at = st + (((uint32_t)(j * (kG / 2) + t * (kG / 8))) ^ swz);
        float acc[kMT][kNB][4];
        uint32_t c[2 * kMT][kWords];
#pragma unroll
        for (int r = 0; r < 2 * kMT; ++r) lds_words<kWords>(at + (uint32_t)(r * 8 * kQKB), c[r]);
        float sl[kMT], sh[kMT];
#pragma unroll
        for (int m = 0; m < kMT; ++m) {
          sl[m] = bf16_to_f32(ts[(size_t)(16 * m) * ng + j]);
          sh[m] = bf16_to_f32(ts[(size_t)(16 * m + 8) * ng + j]);
        }
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          uint4 x[kNB];
#pragma unroll
          for (int nb = 0; nb < kNB; ++nb) x[nb] = xp[((j * kWords + w) * kNB + nb) * 32];
#pragma unroll
          for (int m = 0; m < kMT; ++m) {
            uint32_t p[4], q[4];
            q4_pairs(c[2 * m][w], magic, p);
            q4_pairs(c[2 * m + 1][w], magic, q);
#pragma unroll
            for (int nb = 0; nb < kNB; ++nb) {
              if (w == 0) mma_f16_zero(acc[m][nb], p[0], q[0], p[1], q[1], x[nb].x, x[nb].y);
              else mma_f16(acc[m][nb], p[0], q[0], p[1], q[1], x[nb].x, x[nb].y);
              mma_f16(acc[m][nb], p[2], q[2], p[3], q[3], x[nb].z, x[nb].w);
            }
          }
        }
#pragma unroll
        for (int m = 0; m < kMT; ++m)
#pragma unroll
          for (int nb = 0; nb < kNB; ++nb) {
            out[m][nb][0] = __fmaf_rn(sl[m], acc[m][nb][0], out[m][nb][0]);
            out[m][nb][1] = __fmaf_rn(sl[m], acc[m][nb][1], out[m][nb][1]);
            out[m][nb][2] = __fmaf_rn(sh[m], acc[m][nb][2], out[m][nb][2]);
            out[m][nb][3] = __fmaf_rn(sh[m], acc[m][nb][3], out[m][nb][3]);
          }
      };
      for (int left = ng; left > 0; left -= kGroupsStage) {
        if (!mbar_wait(&S->full[s], ph, abort, kQWait)) { *abort = 1; ok = false; break; }
        const uint32_t st = mine + s * kStage;
        if (left >= kGroupsStage) {
#pragma unroll
          for (int j = 0; j < kGroupsStage; ++j) group(st, j);
        } else {
#pragma unroll 1
          for (int j = 0; j < left; ++j) group(st, j);
        }
        ts += kGroupsStage;
        xp += kGroupsStage * kWords * kNB * 32;
        __syncwarp();
        if (lane == 0) mbar_arrive(&S->empty[s]);
        if (++s == (uint32_t)A.stages) { s = 0; ph ^= 1; }
      }
      if (!ok) {        // a wait ran out: no score of the tiles left is valid
        for (int64_t tl = tile; tl < T; tl += gridDim.x)
          for (int r = lane; r < kRows; r += 32)
            for (int n = b0; n < min(b0 + 8 * kNB, A.B); ++n)
              if (tl * kTile + warp * kRows + r < A.L) A.Z[(int64_t)n * A.ldz + tl * kTile + warp * kRows + r] = NAN;
        break;
      }
#pragma unroll
      for (int m = 0; m < kMT; ++m)
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb)
          odd = __fmaf_rn((out[m][nb][0] + out[m][nb][1]) + (out[m][nb][2] + out[m][nb][3]), 0.0f, odd);
#pragma unroll
      for (int nb = 0; nb < kNB; ++nb) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int n = nb * 8 + 2 * t + c;
          if (b0 + n >= A.B) continue;
          float f0, f1;
          pow2_factors(-S->exponent[n], f0, f1);
          float* z = A.Z + (int64_t)(b0 + n) * A.ldz + tile * kTile + row0;
          const int64_t left = A.L - tile * kTile - row0;
#pragma unroll
          for (int m = 0; m < kMT; ++m) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (16 * m + 8 * h < left) {
                __stcs(z + 16 * m + 8 * h, out[m][nb][2 * h + c] * f0 * f1);
              }
          }
        }
      }
    }
    if (odd != 0.0f) S->odd[warp] = 1;
  }
  __syncthreads();
  if (S->odd[warp] && !*abort) q4_scores_again<kG, kRows, kTile>(A, S->finite, 8 * kNB);
  if (*abort) __nanosleep(20000);       // copies still in flight land before the shared memory is given up
}

template <int kG, int kMT, int kNB, int kWarps>
cudaError_t run_q4(const uint8_t* codes, Q4Args A, int sms, cudaStream_t s) {
  constexpr int kTile = 16 * kMT * kWarps;
  constexpr size_t kStage = (size_t)kTile * kQKB;
  const size_t fixed = q4_fixed<kMT, kNB, kWarps>(A.d, kG);
  const int64_t T = (A.L + kTile - 1) / kTile;
  const int64_t boxes = (A.d / 2 + kQKB - 1) / kQKB * ((T + sms - 1) / sms);
  int stages = (int)((kQSmem - fixed) / kStage);
  if (stages > kQMaxStages) stages = kQMaxStages;
  if (stages > boxes) stages = (int)boxes;
  A.stages = stages;
  CUtensorMap tm;
  cudaError_t e = make_tma_map_2d(&tm, codes, 1, (uint64_t)A.d / 2, (uint64_t)A.L, (uint64_t)A.d / 2,
                                  q4_box(kTile));
  if (e != cudaSuccess) return e;
  auto k = q4_scores_kernel<kG, kMT, kNB, kWarps>;
  static std::atomic<uint64_t> seen{0};
  if ((e = allow_smem(k, (int)kQSmem, seen)) != cudaSuccess) return e;
  const dim3 grid((unsigned)(T < sms ? T : sms), (unsigned)((A.B + 8 * kNB - 1) / (8 * kNB)));
  k<<<grid, 32 * (kWarps + 1), fixed + (size_t)stages * kStage, s>>>(tm, A);
  return cudaGetLastError();
}

template <int kMT, int kNB, int kWarps>
bool q4_fits(int d, int group) {          // two stages at least
  return q4_fixed<kMT, kNB, kWarps>(d, group) + (size_t)2 * 16 * kMT * kWarps * kQKB <= kQSmem;
}

template <int kG>
cudaError_t run_q4_group(const uint8_t* codes, const Q4Args& A, cudaStream_t s) {
  const int sms = current_sms();
  const int nb = (A.B + 7) / 8;
  // as many queries to a pass over the codes as there are, up to 32
  if (nb > 2 && q4_fits<1, 4, 16>(A.d, kG)) return run_q4<kG, 1, 4, 16>(codes, A, sms, s);
  if (nb > 1 && q4_fits<1, 2, 16>(A.d, kG)) return run_q4<kG, 1, 2, 16>(codes, A, sms, s);
  // a few queries: two label blocks a warp share each read of X where there are tiles for every SM
  if (A.L >= (int64_t)sms * 512 && q4_fits<2, 1, 16>(A.d, kG)) return run_q4<kG, 2, 1, 16>(codes, A, sms, s);
  if (A.L >= (int64_t)sms * 256 && q4_fits<1, 1, 16>(A.d, kG)) return run_q4<kG, 1, 1, 16>(codes, A, sms, s);
  return run_q4<kG, 1, 1, 8>(codes, A, sms, s);
}

}  // namespace

cudaError_t launch_q4_pack(const void* W, int64_t L, int32_t d, int w_format, int32_t group, uint8_t* codes,
                           uint16_t* scales, cudaStream_t s) {
  const int64_t n8 = L * d / 8;
  uint32_t* c = reinterpret_cast<uint32_t*>(codes);
  if (w_format == ELMO_BF16) return run_pack<ELMO_BF16>(W, n8, group, c, scales, s);
  if (w_format == ELMO_FP8_E5M2) return run_pack<ELMO_FP8_E5M2>(W, n8, group, c, scales, s);
  return run_pack<ELMO_FP8_E4M3>(W, n8, group, c, scales, s);
}

cudaError_t launch_q4_unpack(const uint8_t* codes, const uint16_t* scales, int64_t L, int32_t d, int32_t group,
                             uint16_t* W, cudaStream_t s) {
  const int64_t n8 = L * d / 8;
  q4_unpack_kernel<<<flat_grid(n8), kPackThreads, 0, s>>>(reinterpret_cast<const uint32_t*>(codes), scales, n8,
                                                          group == 32 ? 2 : group == 64 ? 3 : 4,
                                                          reinterpret_cast<uint4*>(W));
  return cudaGetLastError();
}

cudaError_t launch_q4_scores(const uint8_t* codes, const uint16_t* scales, int64_t L, int32_t d, int32_t group,
                             const uint16_t* X, int32_t B, float* Z, int64_t ldz, cudaStream_t s) {
  const Q4Args A{codes, scales, X, Z, L, ldz, d, B, 0};
  if (group == 32) return run_q4_group<32>(codes, A, s);
  if (group == 64) return run_q4_group<64>(codes, A, s);
  return run_q4_group<128>(codes, A, s);
}

}  // namespace elmo
