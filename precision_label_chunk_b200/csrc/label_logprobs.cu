// label_logprobs.cu -- log probabilities of labels straight from the head:
// Z = X W^T on the tensor cores, and of Z only what the softmax needs is kept.
//
// For every query: lse, entropy, the log probabilities of given labels and the
// k best labels, as logprob.cu defines them for stored scores, over all labels
// of the head ("ELMO: Efficiency via Low-precision and Peak Memory
// Optimization in Large Output Spaces", "Approach": the label axis is
// processed in chunks so that no full logit matrix exists).
//
//   1. operands: bf16 heads multiply X as it is.  8-bit heads multiply
//      X = (hi + lo) / s_b: s_b a power of two for each query with
//      s_b max|x| in (224, 448] (s_b at most 2^60), hi = rne_e4m3(s_b x), lo = rne_e5m2(s_b x - hi).
//      A bf16 number has 8 significant bits, hi takes 4 and leaves at most 8
//      units of the last place, which E5M2's 3 bits hold exactly down to its
//      2^-16 spacing: only numbers below about 2^-15 of the query's largest
//      are rounded at all, to within 2^-23 of it.
//   2. score pass (tcgen05): 128 queries against a range of labels a CTA; each
//      epilogue thread has one query and keeps its running maximum m,
//      s = sum e^(z - m), t = sum e^(z - m)(z - m), and the kp > k best scores.
//   3. join: the ranges' sums in 64 bits, the given labels' scores recomputed
//      exactly (products exact, sums in 64 bits), and the k best labels: every
//      label outside the kept ones scores at most tau (the largest kept-list
//      minimum), so if the k-th best of the kept exceeds tau by more than twice
//      the error bound delta of the tensor-core scores, the k best are among
//      the kept ones within 2 delta of it, which are ranked by exact scores.
//   4. queries that this does not settle (ties within delta, weights that are
//      not finite) rank all labels by exact scores on the CUDA cores.
//
// delta = (gamma (n1 + r1) + r1) max|W|, n1 = sum_j (|hi| + |lo|) / s_b,
// r1 the sum of what hi and lo leave, gamma = nsteps 2^-22: each of the nsteps
// accumulating instructions is allowed 2^-22 of the magnitudes summed.  max|W|
// is read off the tiles in shared memory by two spare warps.
#include <cuda.h>
#include <float.h>

#include "elmo_common.cuh"
#include "elmo_internal.h"
#include "elmo_operators.h"
#include "tc_ptx.cuh"

namespace elmo {
namespace {

using namespace tc;

constexpr int kThreads = 256;             // warp 0 TMA, 1 MMA and TMEM, 2-5 epilogue, 6-7 max|W|
constexpr int kMaxStages = 16;
constexpr int kNBuf = 2;                  // accumulator buffers
constexpr uint32_t kAccCol = 384;         // first accumulator column where X lies in TMEM
constexpr long long kWait = 4000000000LL; // ~2 s
constexpr float kFloor = -200.0f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr size_t kSmemMost = 227 * 1024;
constexpr int kJoinThreads = 512;
constexpr int kMaxCand = 1024;            // kept scores that the join ranks
constexpr int kGroups = 128;
constexpr int kSegs = 74;                 // label segments of the exact path
constexpr int kExactThreads = 256;
constexpr int kExactChunk = 2048;

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// floats and doubles as whole numbers of the same order; 0 is below all
__device__ __forceinline__ uint32_t ord32(float f) {
  const uint32_t u = __float_as_uint(f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float ord32_value(uint32_t k) {
  return k == 0 ? -INFINITY : __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
// 0 for scores that are never listed (-inf, NaN); -0 and 0 are the same score
__device__ __forceinline__ uint64_t ord64(double f) {
  if (!(f > -INFINITY)) return 0ull;
  const uint64_t u = (uint64_t)__double_as_longlong(f + 0.0);
  return (u >> 63) ? ~u : (u | (1ull << 63));
}
__device__ __forceinline__ double ord64_value(uint64_t k) {
  return __longlong_as_double((long long)((k >> 63) ? (k & ~(1ull << 63)) : ~k));
}

struct Stat { float m, s, t; };

struct Args {
  const uint16_t* X;
  const uint8_t *xa, *xb;                 // 8-bit heads: hi and lo codes [B][d]
  const void* W;
  int64_t L, label_base, labels_total;
  int32_t d, B, G, k, kp, stages, nnz, fmt;
  float gamma;
  float *xinv, *n1, *r1;
  int32_t *rflag, *nfail, *fail;
  uint32_t *wmax, *tau;
  float* cand_v;                          // [B][G][kp]
  int32_t* cand_i;
  Stat* part;                             // [B][G]
  uint64_t* seg_key;                      // [B][kSegs][k]
  int32_t* seg_i;
  const int32_t *rowptr, *cols;
  float *logp, *lse, *entropy, *top_logp;
  int32_t* top_idx;
  double* rowstat;                        // [B][2] m and log s (for the exact path)
  int32_t* status;
};

// ---------------------------------------------------------------- 1. operands
constexpr int kPrepThreads = 128;

__device__ __forceinline__ float block_sum_up(float v, float* red) {
  for (int o = 16; o > 0; o >>= 1) v = __fadd_ru(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.0f;
  for (int i = 0; i < kPrepThreads / 32; ++i) t = __fadd_ru(t, red[i]);
  return t;
}

template <int kFp8>
__global__ void __launch_bounds__(kPrepThreads) label_prep_kernel(const Args A, uint8_t* xa, uint8_t* xb) {
  __shared__ float red[kPrepThreads / 32];
  __shared__ uint32_t mx;
  const int b = blockIdx.x, tid = threadIdx.x;
  if (tid == 0) {
    if (b == 0) { *A.wmax = 0; *A.nfail = 0; }
    A.tau[b] = 0;
    mx = 0;
  }
  __syncthreads();
  const uint32_t* xr = reinterpret_cast<const uint32_t*>(A.X + (size_t)b * A.d);
  uint32_t m = 0;
  for (int j = tid; j < A.d / 2; j += kPrepThreads) m = max(m, max(xr[j] & 0x7FFFu, (xr[j] >> 16) & 0x7FFFu));
  atomicMax(&mx, m);
  __syncthreads();
  m = mx;
  const bool bad = m >= 0x7F80u;
  float s = 1.0f;
  if (kFp8 && !bad && m != 0) {
    int e2;
    const float f = frexpf(__uint_as_float(m << 16), &e2);
    // 448 = 0.875 2^9; at most 2^60, so that the accumulators' -200 / inv stays finite
    s = ldexpf(1.0f, max(-126, min(60, f <= 0.875f ? 9 - e2 : 8 - e2)));
  }
  float n = 0.0f, r = 0.0f;
  for (int j = tid; j < A.d / 2; j += kPrepThreads) {
    const uint32_t w = xr[j];
    uint32_t hi2 = 0, lo2 = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float x = __uint_as_float(h ? w & 0xFFFF0000u : w << 16);
      if (kFp8) {
        const float v = __fmul_rn(x, s);
        const uint32_t ch = pack_e4m3x2(0.0f, v) & 0xFFu;
        const float hi = e4m3_to_f32((uint8_t)ch);
        const float left = __fsub_rn(v, hi);
        const uint32_t cl = pack_e5m2x2(0.0f, left) & 0xFFu;
        const float lo = e5m2_to_f32((uint8_t)cl);
        n = __fadd_ru(n, __fadd_ru(fabsf(hi), fabsf(lo)));
        r = __fadd_ru(r, fabsf(__fsub_rn(left, lo)));
        hi2 |= ch << (8 * h);
        lo2 |= cl << (8 * h);
      } else {
        n = __fadd_ru(n, fabsf(x));
      }
    }
    if (kFp8) {
      reinterpret_cast<uint16_t*>(xa + (size_t)b * A.d)[j] = (uint16_t)hi2;
      reinterpret_cast<uint16_t*>(xb + (size_t)b * A.d)[j] = (uint16_t)lo2;
    }
  }
  n = block_sum_up(n, red);
  r = block_sum_up(r, red);
  if (tid == 0) {
    const float inv = 1.0f / s;                              // exact
    A.xinv[b] = inv;
    A.n1[b] = __fmul_ru(n, inv);
    A.r1[b] = __fmul_ru(r, inv);
    A.rflag[b] = bad ? 1 : 0;
  }
}

// ---------------------------------------------------------------- 2. score pass
struct SmemP {
  uint64_t full[kMaxStages], empty[kMaxStages], tfull[kNBuf], tempty[kNBuf];
  uint32_t tmem_base;
  int abort;
};

__device__ __forceinline__ void record_timeout(int32_t* status, volatile int* abort, int site) {
  *abort = 1;
  if (atomicCAS(status, 0, (int)ELMO_ETIMEOUT) == 0) status[1] = site;
}

// The kept scores of column r of a CTA: a heap with the smallest on top,
// entry i at [i * 128 + r].
__device__ __forceinline__ void heap_down(float* hv, int32_t* hl, int r, int i, int n) {
  const float v = hv[i * 128 + r];
  const int32_t l = hl[i * 128 + r];
  for (int c = 2 * i + 1; c < n; c = 2 * i + 1) {
    float cv = hv[c * 128 + r];
    if (c + 1 < n && hv[(c + 1) * 128 + r] < cv) cv = hv[++c * 128 + r];
    if (!(cv < v)) break;
    hv[i * 128 + r] = cv;
    hl[i * 128 + r] = hl[c * 128 + r];
    i = c;
  }
  hv[i * 128 + r] = v;
  hl[i * 128 + r] = l;
}

// Adds a score to the n kept ones (of at most kp); the new lower limit.
__device__ __forceinline__ float heap_keep(float* hv, int32_t* hl, int r, int n, int kp, float v, int32_t l) {
  if (n < kp) {
    hv[n * 128 + r] = v;
    hl[n * 128 + r] = l;
    if (n + 1 < kp) return -INFINITY;
    for (int i = kp / 2 - 1; i >= 0; --i) heap_down(hv, hl, r, i, kp);
  } else {
    hv[r] = v;
    hl[r] = l;
    heap_down(hv, hl, r, 0, kp);
  }
  return hv[r];
}

// kFp8: 8-bit head (kW5: E5M2 weights).  kXs = 0: d <= 768, X (two 8-bit or
// one bf16 operand, 2 d bytes a query) stays in TMEM columns 0..383 and tiles
// are 64 labels with two accumulators in the rest; kXs = 1: wider heads, X
// comes through the ring with W, tiles are 128 labels.
template <int kFp8, int kW5, int kXs>
__global__ void __launch_bounds__(kThreads, 1)
    label_score_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA,
                       const __grid_constant__ CUtensorMap tmB, const Args A) {
  constexpr int kN = kXs ? 128 : 64;
  constexpr int kOps = kFp8 ? 2 : 1;
  constexpr uint32_t kWBytes = kN * 128;
  constexpr uint32_t kXBytes = kXs ? 128 * 128 * kOps : 0;
  constexpr uint32_t kStage = kWBytes + kXBytes;
  constexpr int kKE = kFp8 ? 128 : 64;                 // elements of a 128-byte k-block
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* zs = reinterpret_cast<float*>(ring + (size_t)A.stages * kStage);      // [32][128]
  float* hv = zs + 32 * 128;                                                   // [kp][128]
  int32_t* hl = reinterpret_cast<int32_t*>(hv + (size_t)A.kp * 128);
  SmemP* S = reinterpret_cast<SmemP*>(hl + (size_t)A.kp * 128);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int P = (A.B + 127) / 128;
  const int p = blockIdx.x % P, g = blockIdx.x / P;
  const int64_t T = (A.L + kN - 1) / kN;
  const int64_t t0 = T * g / A.G, t1 = T * (g + 1) / A.G;
  const int nkb = (A.d + kKE - 1) / kKE;
  const uint32_t opcols = (uint32_t)nkb * 32;
  volatile int* abort = &S->abort;
  const bool scan = p == 0 && A.kp > 0;                // this CTA's range is scanned for max|W|

  if (threadIdx.x == 0) {
    for (int s = 0; s < A.stages; ++s) { mbar_init(&S->full[s], 1); mbar_init(&S->empty[s], scan ? 3 : 1); }
    for (int i = 0; i < kNBuf; ++i) { mbar_init(&S->tfull[i], 1); mbar_init(&S->tempty[i], 4); }
    S->abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) { tmem_alloc(&S->tmem_base, 512); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S->tmem_base;

  if (!kXs) {
    if (warp >= 2 && warp < 6) {                       // query r of the panel into lane r
      const int q = warp & 3, row = p * 128 + q * 32 + lane;
      const size_t rowbytes = (size_t)A.d * (kFp8 ? 1 : 2);
      for (int op = 0; op < kOps; ++op) {
        const uint8_t* src = (kFp8 ? (op ? A.xb : A.xa) : reinterpret_cast<const uint8_t*>(A.X)) + (size_t)row * rowbytes;
        for (uint32_t c0 = 0; c0 < opcols; c0 += 32) {
          uint32_t v[32];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const size_t off = (size_t)(c0 + 4 * u) * 4;
            uint4 w4 = make_uint4(0u, 0u, 0u, 0u);
            if (row < A.B && off < rowbytes) w4 = *reinterpret_cast<const uint4*>(src + off);
            v[4 * u] = w4.x; v[4 * u + 1] = w4.y; v[4 * u + 2] = w4.z; v[4 * u + 3] = w4.w;
          }
          tmem_st32(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)op * opcols + c0, v);
        }
      }
      tmem_wait_st();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }

  if (warp == 0) {
    if (elect_one()) {
      tma_prefetch_desc(&tmW);
      uint32_t it = 0;
      for (int64_t t = t0; t < t1 && !*abort; ++t) {
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const uint32_t s = it % (uint32_t)A.stages, ph = (it / (uint32_t)A.stages) & 1;
          if (!mbar_wait(&S->empty[s], ph ^ 1, abort, kWait)) { record_timeout(A.status, abort, 71); break; }
          uint8_t* st = ring + (size_t)s * kStage;
          mbar_arrive_expect_tx(&S->full[s], kStage);
          tma_load_2d(st, &tmW, &S->full[s], kb * kKE, (int32_t)(t * kN));
          if (kXs) {
            tma_load_2d(st + kWBytes, &tmA, &S->full[s], kb * kKE, p * 128);
            if (kFp8) tma_load_2d(st + kWBytes + 16384, &tmB, &S->full[s], kb * kKE, p * 128);
          }
        }
      }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      // hi is E4M3 (format 0) and lo E5M2 (1); bf16 operands are format 1 of their kind
      const uint32_t idesc[2] = {kFp8 ? make_idesc(0, kW5, 0, 0, 128, kN) : make_idesc(1, 1, 0, 0, 128, kN),
                                 make_idesc(1, kW5, 0, 0, 128, kN)};
      uint32_t it = 0, n = 0;
      for (int64_t t = t0; t < t1 && !*abort; ++t, ++n) {
        const uint32_t buf = n % kNBuf, use = n / kNBuf;
        if (!mbar_wait(&S->tempty[buf], (use & 1) ^ 1, abort, kWait)) { record_timeout(A.status, abort, 72); break; }
        tc_fence_after();
        const uint32_t dcol = tmem + (kXs ? 0 : kAccCol) + buf * kN;
        bool ok = true;
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const uint32_t s = it % (uint32_t)A.stages, ph = (it / (uint32_t)A.stages) & 1;
          if (!mbar_wait(&S->full[s], ph, abort, kWait)) { record_timeout(A.status, abort, 73); ok = false; break; }
          tc_fence_after();
          const uint32_t ws = smem_u32(ring + (size_t)s * kStage);
#pragma unroll
          for (int op = 0; op < kOps; ++op) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {              // 32 bytes of K an instruction
              const uint64_t bd = sw128_desc(ws + k * 32, 16, 1024);
              const uint32_t more = (kb | op | k) != 0;
              if (kXs) {
                const uint64_t ad = sw128_desc(ws + kWBytes + op * 16384 + k * 32, 16, 1024);
                if (kFp8) mma_e4m3(dcol, ad, bd, idesc[op], more);
                else mma_bf16(dcol, ad, bd, idesc[0], more);
              } else {
                const uint32_t a = tmem + (uint32_t)op * opcols + (uint32_t)kb * 32 + (uint32_t)k * 8;
                if (kFp8) mma_e4m3_ts(dcol, a, bd, idesc[op], more);
                else mma_bf16_ts(dcol, a, bd, idesc[0], more);
              }
            }
          }
          mma_commit(&S->empty[s]);
        }
        if (!ok) break;
        mma_commit(&S->tfull[buf]);
      }
    }
  } else if (warp < 6) {
    const int q = warp & 3, r = q * 32 + lane, row = p * 128 + r;
    const bool live = row < A.B;
    const float inv = live ? A.xinv[row] : 1.0f;       // scores are inv times the accumulators
    const float c2 = inv * kLog2e, floor_v = kFloor / inv;
    float m = -INFINITY, s = 0.0f, t = 0.0f;
    float mine = -INFINITY;                            // the smallest kept score, once kp are kept
    int n = 0;
    uint32_t nt = 0;
    for (int64_t tile = t0; tile < t1 && !*abort; ++tile, ++nt) {
      const uint32_t buf = nt % kNBuf, use = nt / kNBuf;
      if (!mbar_wait(&S->tfull[buf], use & 1, abort, kWait)) { record_timeout(A.status, abort, 74); break; }
      tc_fence_after();
      float limit = A.kp > 0 && live ? fmaxf(mine, ord32_value(__ldcg(A.tau + row))) : INFINITY;
#pragma unroll 1
      for (int u = 0; u < kN / 64; ++u) {
        uint32_t v[2][32];
        const uint32_t at = tmem + ((uint32_t)(q * 32) << 16) + (kXs ? 0 : kAccCol) + buf * kN + u * 64;
        tmem_ld32(at, v[0]);
        tmem_ld32(at + 32, v[1]);
        tmem_wait_ld();
        if (u == kN / 64 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&S->tempty[buf]);
        }
        if (!live) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int64_t l0 = tile * kN + u * 64 + h * 32;
          if (l0 + 32 > A.L) {                         // labels past the end are no labels
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (l0 + c >= A.L) v[h][c] = 0xFF800000u;
          }
          float x[8];
#pragma unroll
          for (int c = 0; c < 8; ++c)
            x[c] = fmaxf(fmaxf(__uint_as_float(v[h][c]), __uint_as_float(v[h][c + 8])),
                         fmaxf(__uint_as_float(v[h][c + 16]), __uint_as_float(v[h][c + 24])));
          const float mx = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
          if (mx > m) {
            if (m > -INFINITY) {
              const float dm = fmaxf(m - mx, floor_v), c = ex2(dm * c2);
              t = c * fmaf(s, dm, t);
              s *= c;
            }
            m = mx;
          }
          const float m0 = m > -INFINITY ? m : 0.0f;
          float ps[4] = {0.0f, 0.0f, 0.0f, 0.0f}, pt[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float dz = max_nan(__uint_as_float(v[h][c]) - m0, floor_v);
            const float e = ex2(dz * c2);
            ps[c & 3] += e;
            pt[c & 3] = fmaf(e, dz, pt[c & 3]);
          }
          s += (ps[0] + ps[1]) + (ps[2] + ps[3]);
          t += (pt[0] + pt[1]) + (pt[2] + pt[3]);
          if (mx > limit) {
            uint32_t hit = 0;
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              zs[c * 128 + r] = __uint_as_float(v[h][c]);
              hit |= (uint32_t)(__uint_as_float(v[h][c]) > limit) << c;
            }
            while (hit) {
              const int c = __ffs((int)hit) - 1;
              hit &= hit - 1;
              const float z = zs[c * 128 + r];
              if (z > limit) {
                mine = heap_keep(hv, hl, r, n, A.kp, z, (int32_t)(l0 + c));
                n = min(n + 1, A.kp);
                if (mine > limit) {
                  limit = mine;
                  atomicMax(A.tau + row, ord32(mine));
                }
              }
            }
          }
        }
      }
    }
    if (live) {
      A.part[(size_t)row * A.G + g] = {m * inv, s, t * inv};
      const size_t o = ((size_t)row * A.G + g) * A.kp;
      for (int i = 0; i < A.kp; ++i) {
        A.cand_v[o + i] = i < n ? hv[i * 128 + r] : 0.0f;
        A.cand_i[o + i] = i < n ? hl[i * 128 + r] : -1;
      }
    }
  } else if (scan) {
    // magnitudes as whole numbers: 16 bits (bf16) or 8 (the bytes of each half in turn)
    const int id = (warp - 6) * 32 + lane;
    uint32_t mx = 0, it = 0;
    for (int64_t t = t0; t < t1 && !*abort; ++t) {
      for (int kb = 0; kb < nkb; ++kb, ++it) {
        const uint32_t s = it % (uint32_t)A.stages, ph = (it / (uint32_t)A.stages) & 1;
        if (!mbar_wait(&S->full[s], ph, abort, kWait)) { record_timeout(A.status, abort, 75); break; }
        const uint4* w = reinterpret_cast<const uint4*>(ring + (size_t)s * kStage);
#pragma unroll 4
        for (int i = id; i < (int)kWBytes / 16; i += 64) {
          const uint4 v = w[i];
          const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (kFp8) {
              mx = __vmaxu2(mx, x[e] & 0x7F007F00u);
              mx = __vmaxu2(mx, (x[e] << 8) & 0x7F007F00u);
            } else {
              mx = __vmaxu2(mx, x[e] & 0x7FFF7FFFu);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&S->empty[s]);
      }
    }
    mx = max(mx & 0xFFFFu, mx >> 16) >> (kFp8 ? 8 : 0);
    for (int o = 16; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
    if (lane == 0 && mx) atomicMax(A.wmax, mx);
  }
  __syncthreads();
  if (*abort) __nanosleep(20000);                      // copies in flight land before the memory is given up
  if (warp == 1) { tc_fence_after(); tmem_dealloc(tmem, 512); }
}

// ---------------------------------------------------------------- exact scores
// x . w_l with exact products and sums in 64 bits, by one warp, in an order
// that depends on d alone: equal rows have equal scores.
__device__ __forceinline__ double exact_score(const double* xs, const void* W, int fmt, int64_t l, int d, int lane) {
  double acc = 0.0;
  if (fmt == ELMO_BF16) {
    const uint4* w = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(W) + l * d);
    for (int c = lane; c < d / 8; c += 32) {
      const uint4 v = w[c];
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc = fma(xs[8 * c + 2 * e], (double)__uint_as_float(u[e] << 16), acc);
        acc = fma(xs[8 * c + 2 * e + 1], (double)__uint_as_float(u[e] & 0xFFFF0000u), acc);
      }
    }
  } else {
    const uint2* w = reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(W) + l * d);
    for (int c = lane; c < d / 8; c += 32) {
      const uint2 v = w[c];
      float f[8];
      float(&a)[4] = *reinterpret_cast<float(*)[4]>(f);
      float(&b)[4] = *reinterpret_cast<float(*)[4]>(f + 4);
      if (fmt == ELMO_FP8_E5M2) { e5m2x4_to_f32(v.x, a); e5m2x4_to_f32(v.y, b); }
      else { e4m3x4_to_f32(v.x, a); e4m3x4_to_f32(v.y, b); }
#pragma unroll
      for (int e = 0; e < 8; ++e) acc = fma(xs[8 * c + e], (double)f[e], acc);
    }
  }
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xFFFFFFFFu, acc, o);
  return acc;
}

__device__ __forceinline__ float max_weight(uint32_t code, int fmt) {
  if (fmt == ELMO_BF16) return code >= 0x7F80u ? NAN : bf16_to_f32((uint16_t)code);
  if (fmt == ELMO_FP8_E5M2) return code >= 0x7Cu ? NAN : e5m2_to_f32((uint8_t)code);
  return code >= 0x7Fu ? NAN : e4m3_to_f32((uint8_t)code);
}

// ---------------------------------------------------------------- 3. join
__global__ void __launch_bounds__(kJoinThreads) label_join_kernel(const Args A) {
  extern __shared__ double dyn[];
  double* xs = dyn;                                    // [d] the query
  __shared__ double ex[kMaxCand];                      // exact scores of the ones ranked
  __shared__ float cv[kMaxCand];                       // kept scores near the best
  __shared__ int32_t ci[kMaxCand];
  __shared__ double stat[2];
  __shared__ int count;
  __shared__ float kth, low;
  constexpr int kW = kJoinThreads / 32;
  const int b = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool bad = A.rflag[b] != 0;
  for (int j = tid; j < A.d; j += kJoinThreads) xs[j] = (double)bf16_to_f32(A.X[(size_t)b * A.d + j]);
  if (warp == 0) {
    const Stat* part = A.part + (size_t)b * A.G;
    float mf = -INFINITY;
    for (int i = lane; i < A.G; i += 32) mf = fmaxf(mf, part[i].m);
    for (int o = 16; o > 0; o >>= 1) mf = fmaxf(mf, __shfl_xor_sync(0xFFFFFFFFu, mf, o));
    double s = 0.0, t = 0.0;
    for (int i = lane; i < A.G; i += 32) {
      const Stat q = part[i];
      if (q.m == -INFINITY) { s += q.s; continue; }
      const double d = (double)q.m - (double)mf, c = q.m == mf ? 1.0 : exp(d);
      s += c * q.s;
      t += c * (q.t + (q.m == mf ? 0.0 : d * q.s));
    }
    for (int o = 16; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
      t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    }
    if (lane == 0) {
      double m = mf, logs = log(s), lse = m + logs, H = logs - t / s;
      if (mf == -INFINITY) {                           // no label has a finite score
        lse = s == 0.0 ? -INFINITY : NAN;
        H = s == 0.0 ? 0.0 : NAN;
        m = lse;
        logs = 0.0;
      } else if (mf == INFINITY) {
        lse = m;
        logs = 0.0;
      }
      if (bad) lse = H = m = NAN;
      A.lse[b] = (float)lse;
      A.entropy[b] = (float)H;
      stat[0] = m;
      stat[1] = logs;
      A.rowstat[2 * b] = m;
      A.rowstat[2 * b + 1] = logs;
    }
  }
  if (tid == 0) count = 0;
  __syncthreads();
  const double m = stat[0], logs = stat[1];

  const int e0 = max(A.rowptr[b], 0), e1 = min(A.rowptr[b + 1], A.nnz);
  for (int e = e0 + warp; e < e1; e += kW) {
    const int64_t id = A.cols[e], l = id - A.label_base;
    float r = NAN;
    if (id < 0 || id >= A.labels_total) {
      if (lane == 0 && atomicCAS(A.status, 0, (int)ELMO_EDATA) == 0) A.status[1] = e;
    } else if (l < 0 || l >= A.L) {
      r = -INFINITY;                                   // another device's label
    } else {
      const double z = exact_score(xs, A.W, A.fmt, l, A.d, lane);
      r = z == -INFINITY && !isnan(m + logs) ? -INFINITY : (float)(z - m - logs);
    }
    if (lane == 0) A.logp[e] = r;
  }

  if (A.k == 0) return;
  if (bad) {
    for (int i = tid; i < A.k; i += kJoinThreads) {
      A.top_idx[(size_t)b * A.k + i] = -1;
      A.top_logp[(size_t)b * A.k + i] = -INFINITY;
    }
    return;
  }
  const uint32_t tau_key = A.tau[b];
  const float tau = ord32_value(tau_key);
  const size_t base = (size_t)b * A.G * A.kp;
  const int nc = A.G * A.kp;
  const float inv = A.xinv[b];
  // 2 delta in the accumulators' units, rounded up; 2^-126 for subnormal partial sums
  float delta = __fmul_ru(A.gamma, __fadd_ru(A.n1[b], A.r1[b]));
  delta = __fmul_ru(__fadd_ru(delta, A.r1[b]), max_weight(*A.wmax, A.fmt));
  const float two = __fdiv_ru(__fmul_ru(2.0f, __fadd_ru(delta, 0x1p-126f)), inv);
  // of the ranges' lists, only what comes within 2 delta of the k-th best: the
  // k-th best of kGroups groups' best is at most that
  float best = -INFINITY;
  for (int i = tid; i < nc; i += kJoinThreads)
    if (A.cand_i[base + i] >= 0) best = fmaxf(best, A.cand_v[base + i]);
  for (int o = 1; o < kJoinThreads / kGroups; o <<= 1) best = fmaxf(best, __shfl_xor_sync(0xFFFFFFFFu, best, o));
  if (tid % (kJoinThreads / kGroups) == 0) cv[tid / (kJoinThreads / kGroups)] = best;
  if (tid == 0) low = -INFINITY;
  __syncthreads();
  if (tid < kGroups) {
    const float mine = cv[tid];
    int above = 0, same = 0;
    for (int j = 0; j < kGroups; ++j) { above += cv[j] > mine; same += cv[j] == mine; }
    if (above < A.k && above + same >= A.k) low = mine;
  }
  __syncthreads();
  const float from = __fsub_rd(low, two);
  for (int i = tid; i < nc; i += kJoinThreads) {
    const int32_t l = A.cand_i[base + i];
    if (l < 0) continue;
    const float v = A.cand_v[base + i];
    if (v >= from || !(two < INFINITY)) {
      const int at = atomicAdd(&count, 1);
      if (at < kMaxCand) { cv[at] = v; ci[at] = l; }
    }
  }
  if (tid == 0) kth = -INFINITY;
  __syncthreads();
  const int n = count;
  bool ok = n >= A.k && n <= kMaxCand;
  if (ok) {
    for (int i = tid; i < n; i += kJoinThreads) {      // the k-th best kept score, ties in any order
      const float v = cv[i];
      int above = 0, same = 0;
      for (int j = 0; j < n; ++j) { above += cv[j] > v; same += cv[j] == v; }
      if (above < A.k && above + same >= A.k) kth = v;
    }
  }
  __syncthreads();
  const float cut = __fsub_rd(kth, two);
  ok = ok && (tau_key == 0 || cut > tau) && two < INFINITY;           // NaN (weights that are not finite) fails too
  if (!ok) {
    if (tid == 0) A.fail[atomicAdd(A.nfail, 1)] = b;
    return;
  }
  for (int i = warp; i < n; i += kW) {
    double z = 0.0;
    const bool in = cv[i] >= cut;
    if (in) z = exact_score(xs, A.W, A.fmt, ci[i], A.d, lane);
    if (lane == 0) ex[i] = in ? z : -INFINITY;
  }
  __syncthreads();
  for (int i = tid; i < n; i += kJoinThreads) {
    if (!(cv[i] >= cut)) continue;
    const double z = ex[i];
    const int32_t l = ci[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += ex[j] > z || (ex[j] == z && ci[j] < l);
    if (rank < A.k) {
      A.top_idx[(size_t)b * A.k + rank] = (int32_t)(l + A.label_base);
      A.top_logp[(size_t)b * A.k + rank] = (float)(z - m - logs);
    }
  }
}

// ---------------------------------------------------------------- 4. exact path
__device__ __forceinline__ bool ranks_before(uint64_t ka, int32_t ia, uint64_t kb, int32_t ib) {
  return ka > kb || (ka == kb && ia < ib);
}

// The best entry of (key, index) pairs [0, n) that ranks after (last_k,
// last_i), by the whole CTA; key 0 if there is none.
template <typename F>
__device__ __forceinline__ void best_after(int n, F at, uint64_t last_k, int32_t last_i, uint64_t* rk, int32_t* ri,
                                           uint64_t& key, int32_t& idx) {
  uint64_t bk = 0;
  int32_t bi = 0x7FFFFFFF;
  for (int i = threadIdx.x; i < n; i += kExactThreads) {
    uint64_t k;
    int32_t l;
    at(i, k, l);
    if (k != 0 && ranks_before(last_k, last_i, k, l) && ranks_before(k, l, bk, bi)) { bk = k; bi = l; }
  }
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t ok = __shfl_xor_sync(0xFFFFFFFFu, bk, o);
    const int32_t oi = __shfl_xor_sync(0xFFFFFFFFu, bi, o);
    if (ranks_before(ok, oi, bk, bi)) { bk = ok; bi = oi; }
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) { rk[threadIdx.x >> 5] = bk; ri[threadIdx.x >> 5] = bi; }
  __syncthreads();
  key = 0;
  idx = 0x7FFFFFFF;
  for (int w = 0; w < kExactThreads / 32; ++w)
    if (ranks_before(rk[w], ri[w], key, idx)) { key = rk[w]; idx = ri[w]; }
}

// Work item (failed row, segment): the segment's k best labels.
__global__ void __launch_bounds__(kExactThreads) label_exact_kernel(const Args A) {
  extern __shared__ double dyn[];
  double* xs = dyn;
  __shared__ uint64_t key[kExactChunk + ELMO_MAX_TOPK];
  __shared__ uint64_t lk[ELMO_MAX_TOPK];
  __shared__ int32_t li[ELMO_MAX_TOPK];
  __shared__ int32_t old[ELMO_MAX_TOPK];
  __shared__ uint64_t rk[kExactThreads / 32];
  __shared__ int32_t ri[kExactThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nf = *A.nfail;
  for (int64_t item = blockIdx.x; item < (int64_t)nf * kSegs; item += gridDim.x) {
    const int r = (int)(item / kSegs), seg = (int)(item % kSegs);
    const int b = A.fail[r];
    const int64_t l0 = A.L * seg / kSegs, l1 = A.L * (seg + 1) / kSegs;
    __syncthreads();
    for (int j = tid; j < A.d; j += kExactThreads) xs[j] = (double)bf16_to_f32(A.X[(size_t)b * A.d + j]);
    if (tid < A.k) { lk[tid] = 0; li[tid] = 0x7FFFFFFF; }
    __syncthreads();
    for (int64_t a = l0; a < l1; a += kExactChunk) {
      const int n = (int)min((int64_t)kExactChunk, l1 - a);
      for (int i = warp; i < n; i += kExactThreads / 32) {
        const double z = exact_score(xs, A.W, A.fmt, a + i, A.d, lane);
        if (lane == 0) key[i] = ord64(z);
      }
      if (tid < A.k) { key[kExactChunk + tid] = lk[tid]; old[tid] = li[tid]; }
      __syncthreads();
      auto at = [&](int i, uint64_t& k, int32_t& l) {
        if (i < n) { k = key[i]; l = (int32_t)(a + i); }
        else { k = key[kExactChunk + i - n]; l = old[i - n]; }
      };
      uint64_t pk = ~0ull;
      int32_t pi = -1;
      for (int q = 0; q < A.k; ++q) {
        uint64_t k;
        int32_t l;
        best_after(n + A.k, at, pk, pi, rk, ri, k, l);
        if (tid == 0) { lk[q] = k; li[q] = l; }
        if (k == 0) {                                  // nothing left to list: the rest stays empty
          if (tid > q && tid < A.k) { lk[tid] = 0; li[tid] = 0x7FFFFFFF; }
          break;
        }
        pk = k;
        pi = l;
      }
      __syncthreads();
    }
    if (tid < A.k) {
      A.seg_key[((size_t)r * kSegs + seg) * A.k + tid] = lk[tid];
      A.seg_i[((size_t)r * kSegs + seg) * A.k + tid] = li[tid];
    }
  }
}

__global__ void __launch_bounds__(kExactThreads) label_exact_join_kernel(const Args A) {
  __shared__ uint64_t rk[kExactThreads / 32];
  __shared__ int32_t ri[kExactThreads / 32];
  const int nf = *A.nfail;
  for (int r = blockIdx.x; r < nf; r += gridDim.x) {
    const int b = A.fail[r];
    const double m = A.rowstat[2 * b], logs = A.rowstat[2 * b + 1];
    const uint64_t* sk = A.seg_key + (size_t)r * kSegs * A.k;
    const int32_t* si = A.seg_i + (size_t)r * kSegs * A.k;
    auto at = [&](int i, uint64_t& k, int32_t& l) { k = sk[i]; l = si[i]; };
    uint64_t pk = ~0ull;
    int32_t pi = -1;
    for (int q = 0; q < A.k; ++q) {
      uint64_t k = 0;
      int32_t l = 0;
      if (pk != 0) best_after(kSegs * A.k, at, pk, pi, rk, ri, k, l);
      if (threadIdx.x == 0) {
        A.top_idx[(size_t)b * A.k + q] = k ? (int32_t)(l + A.label_base) : -1;
        A.top_logp[(size_t)b * A.k + q] = k ? (float)(ord64_value(k) - m - logs) : -INFINITY;
      }
      pk = k;
      pi = l;
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- host
struct Layout {
  int G, kp;
  size_t xa, xb, xinv, n1, r1, rflag, wmax, nfail, fail, tau, cv, ci, part, sk, si, rowstat, total;
};

// Scores kept beyond k: enough that the k-th best clears the kp-th by more
// than 2 delta on ordinary rows.
int kept(int k) { return k == 0 ? 0 : (k + 11 + k / 12 + 7) / 8 * 8; }

Layout layout_of(const elmo_head* h, int32_t B, int32_t k) {
  Layout o{};
  const bool fp8 = h->dt != ELMO_BF16;
  const int P = (B + 127) / 128;
  const int64_t N = h->d <= 768 ? 64 : 128, T = (h->L + N - 1) / N;
  int64_t G = h->num_sms / P;
  if (G > T) G = T;
  if (G < 1) G = 1;
  o.G = (int)G;
  o.kp = kept(k);
  size_t off = 0;
  auto take = [&](size_t bytes) { const size_t at = off; off += (bytes + 255) / 256 * 256; return at; };
  o.xa = take(fp8 ? (size_t)B * h->d : 0);
  o.xb = take(fp8 ? (size_t)B * h->d : 0);
  o.xinv = take(4 * (size_t)B);
  o.n1 = take(4 * (size_t)B);
  o.r1 = take(4 * (size_t)B);
  o.rflag = take(4 * (size_t)B);
  o.wmax = take(4);
  o.nfail = take(4);
  o.fail = take(4 * (size_t)B);
  o.tau = take(4 * (size_t)B);
  o.cv = take(4 * (size_t)B * o.G * o.kp);
  o.ci = take(4 * (size_t)B * o.G * o.kp);
  o.part = take(sizeof(Stat) * (size_t)B * o.G);
  o.sk = take(8 * (size_t)B * kSegs * k);
  o.si = take(4 * (size_t)B * kSegs * k);
  o.rowstat = take(16 * (size_t)B);
  o.total = off;
  return o;
}

template <int kFp8, int kW5, int kXs>
cudaError_t run_pass(elmo_head* h, Args A, cudaStream_t s) {
  constexpr int kN = kXs ? 128 : 64;
  constexpr int kOps = kFp8 ? 2 : 1;
  constexpr size_t kStage = kN * 128 + (kXs ? 16384 * kOps : 0);
  const size_t fixed = 1024 + 4 * 32 * 128 + (size_t)A.kp * 128 * 8 + sizeof(SmemP);
  int stages = (int)((kSmemMost - fixed) / kStage);
  if (stages > kMaxStages) stages = kMaxStages;
  A.stages = stages;
  const int eb = kFp8 ? 1 : 2;
  CUtensorMap tmW, tmA, tmB;
  cudaError_t e = make_tma_map_2d(&tmW, h->W, eb, (uint64_t)h->d, (uint64_t)h->L, (uint64_t)h->d, kN);
  if (e != cudaSuccess) return e;
  tmA = tmB = tmW;
  if (kXs) {
    const void* a = kFp8 ? static_cast<const void*>(A.xa) : A.X;
    if ((e = make_tma_map_2d(&tmA, a, eb, (uint64_t)h->d, (uint64_t)A.B, (uint64_t)h->d, 128)) != cudaSuccess) return e;
    if (kFp8 && (e = make_tma_map_2d(&tmB, A.xb, eb, (uint64_t)h->d, (uint64_t)A.B, (uint64_t)h->d, 128)) != cudaSuccess)
      return e;
  }
  auto kern = label_score_kernel<kFp8, kW5, kXs>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMost);
  if (e != cudaSuccess) return e;
  const int P = (A.B + 127) / 128;
  kern<<<P * A.G, kThreads, fixed + stages * kStage, s>>>(tmW, tmA, tmB, A);
  return cudaGetLastError();
}

}  // namespace

size_t label_logprobs_workspace(const elmo_head* h, int32_t B, int32_t k) { return layout_of(h, B, k).total; }

cudaError_t launch_label_logprobs(elmo_head* h, const uint16_t* X, int32_t B, const int32_t* rowptr,
                                  const int32_t* cols, int32_t nnz, int32_t k, float* logp, float* lse, float* entropy,
                                  int32_t* top_idx, float* top_logp, void* work, cudaStream_t s) {
  const Layout o = layout_of(h, B, k);
  uint8_t* ws = static_cast<uint8_t*>(work);
  const bool fp8 = h->dt != ELMO_BF16;
  const bool wide = h->d > 768;
  Args A{};
  A.X = X;
  A.xa = ws + o.xa;
  A.xb = ws + o.xb;
  A.W = h->W;
  A.L = h->L;
  A.label_base = h->label_base;
  A.labels_total = h->labels_total;
  A.d = h->d; A.B = B; A.G = o.G; A.k = k; A.kp = o.kp; A.nnz = nnz;
  A.fmt = w_format(h);
  const int nsteps = (fp8 ? 2 : 1) * ((h->d * (fp8 ? 1 : 2) + 127) / 128) * 4;
  A.gamma = (float)nsteps * 0x1p-22f;
  A.xinv = reinterpret_cast<float*>(ws + o.xinv);
  A.n1 = reinterpret_cast<float*>(ws + o.n1);
  A.r1 = reinterpret_cast<float*>(ws + o.r1);
  A.rflag = reinterpret_cast<int32_t*>(ws + o.rflag);
  A.wmax = reinterpret_cast<uint32_t*>(ws + o.wmax);
  A.nfail = reinterpret_cast<int32_t*>(ws + o.nfail);
  A.fail = reinterpret_cast<int32_t*>(ws + o.fail);
  A.tau = reinterpret_cast<uint32_t*>(ws + o.tau);
  A.cand_v = reinterpret_cast<float*>(ws + o.cv);
  A.cand_i = reinterpret_cast<int32_t*>(ws + o.ci);
  A.part = reinterpret_cast<Stat*>(ws + o.part);
  A.seg_key = reinterpret_cast<uint64_t*>(ws + o.sk);
  A.seg_i = reinterpret_cast<int32_t*>(ws + o.si);
  A.rowstat = reinterpret_cast<double*>(ws + o.rowstat);
  A.rowptr = rowptr; A.cols = cols;
  A.logp = logp; A.lse = lse; A.entropy = entropy; A.top_idx = top_idx; A.top_logp = top_logp;
  A.status = h->status;
  cudaError_t e;
  {
    KernelScope sc(h, ELMO_K_PREP, s, 1);
    if (fp8) label_prep_kernel<1><<<B, kPrepThreads, 0, s>>>(A, ws + o.xa, ws + o.xb);
    else label_prep_kernel<0><<<B, kPrepThreads, 0, s>>>(A, nullptr, nullptr);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  {
    KernelScope sc(h, ELMO_K_TOPK_SCORE, s, 1);
    if (!fp8) e = wide ? run_pass<0, 0, 1>(h, A, s) : run_pass<0, 0, 0>(h, A, s);
    else if (h->w_e5m2) e = wide ? run_pass<1, 1, 1>(h, A, s) : run_pass<1, 1, 0>(h, A, s);
    else e = wide ? run_pass<1, 0, 1>(h, A, s) : run_pass<1, 0, 0>(h, A, s);
    if (e != cudaSuccess) return e;
  }
  KernelScope sc(h, ELMO_K_TOPK_MERGE, s, k > 0 ? 3 : 1);
  const size_t xbytes = sizeof(double) * (size_t)h->d;
  e = cudaFuncSetAttribute(label_join_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 4096 * 8);
  if (e != cudaSuccess) return e;
  label_join_kernel<<<B, kJoinThreads, xbytes, s>>>(A);
  if ((e = cudaGetLastError()) != cudaSuccess || k == 0) return e;
  e = cudaFuncSetAttribute(label_exact_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 4096 * 8);
  if (e != cudaSuccess) return e;
  label_exact_kernel<<<h->num_sms * 2, kExactThreads, xbytes, s>>>(A);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  label_exact_join_kernel<<<B < h->num_sms ? B : h->num_sms, kExactThreads, 0, s>>>(A);
  return cudaGetLastError();
}

}  // namespace elmo
