// logprob.cu -- log probabilities of labels from rows of scores, and their
// gradient.
//
// A row of scores z (one query against L labels) is read as the logits of a
// softmax over the labels.  With m = max z, s = sum e^(z - m) and
// t = sum e^(z - m) (z - m):
//     log sum exp  lse = m + log s,
//     entropy      H   = log s - t / s        (= -sum p log p, p = e^(z - lse))
//     log p_l          = (z_l - m) - log s,
// so one pass over the row with a running (m, s, t) gives everything but the
// k best labels, and those lie in the k blocks whose maxima rank first (by
// value, then by the lower block): each of k blocks ranked before an
// element's own block holds an element ranked before it.  The pass therefore
// stores the maximum of every block of 1024 scores, and a second look at a few
// blocks finds the best labels, at a cost that does not depend on how the
// scores are ordered.
//
// Masked labels are scores of -inf; a row may be all masked.
#include <cuda_bf16.h>

#include "elmo_common.cuh"
#include "elmo_internal.h"
#include "elmo_operators.h"
#include "tc_ptx.cuh"

namespace elmo {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBlock = 1024;              // scores of a block
constexpr float kFloor = -200.0f;         // z - m is cut here: e^-200 is 0 in fp32, and -inf 0 never forms
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxSplit = 512;

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

// A score's place in the order as a whole number: larger is better, 0 for a
// score that is never listed (-inf, NaN).  -0 and 0 are the same score.
__device__ __forceinline__ uint32_t order_of(float z) {
  if (!(z > -INFINITY)) return 0u;
  const uint32_t u = __float_as_uint(z + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
// (order, lower index first)
__device__ __forceinline__ uint64_t key_of(uint32_t order, uint32_t index) {
  return order ? ((uint64_t)order << 32) | (0xFFFFFFFFu - index) : 0ull;
}
__device__ __forceinline__ uint32_t index_of(uint64_t key) { return 0xFFFFFFFFu - (uint32_t)key; }

// Row statistics with the maximum: sums of e^(z - m) and e^(z - m)(z - m).
struct Stat { float m, s, t; };

template <typename T> __device__ __forceinline__ float score_at(const T* z, int64_t i);
template <> __device__ __forceinline__ float score_at<float>(const float* z, int64_t i) { return z[i]; }
template <> __device__ __forceinline__ float score_at<uint16_t>(const uint16_t* z, int64_t i) { return bf16_to_f32(z[i]); }

// Blocks are cut at 16-byte boundaries of the row's addresses: block j of a
// row whose first score lies `shift` elements past such a boundary holds
// scores [j kBlock - shift, (j + 1) kBlock - shift).  A thread has 32 of a
// warp's 1024: kV vectors of 16 bytes.
template <typename T> struct Vec { static constexpr int kE = 16 / sizeof(T); static constexpr int kV = 32 / kE; };

template <typename T>
__device__ __forceinline__ void load_block(const T* z, int64_t L, int shift, int64_t block, int lane, float (&v)[32]) {
  constexpr int kE = Vec<T>::kE, kV = Vec<T>::kV;
  const int64_t first = block * kBlock - shift;
  if (first >= 0 && first + kBlock <= L) {
    const uint4* p = reinterpret_cast<const uint4*>(z + first) + lane;
    uint4 q[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) q[i] = __ldg(p + 32 * i);
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (sizeof(T) == 4) {
          v[4 * i + e] = __uint_as_float(w[e]);
        } else {
          v[kE * i + 2 * e] = __uint_as_float(w[e] << 16);
          v[kE * i + 2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kV; ++i)
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const int64_t at = first + (32 * i + lane) * kE + e;
        v[kE * i + e] = at >= 0 && at < L ? score_at(z, at) : -INFINITY;
      }
  }
}
// the score's label of element e of load_block
template <typename T>
__device__ __forceinline__ int64_t label_of(int shift, int64_t block, int lane, int e) {
  constexpr int kE = Vec<T>::kE;
  return block * kBlock - shift + (32 * (e / kE) + lane) * kE + e % kE;
}

template <typename T> __host__ __device__ __forceinline__ int shift_of(const T* row) {
  return (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
}

struct Args {
  const void* Z;
  int64_t ldz, L;
  int32_t B, k, nnz, splits, nblk;
  const int32_t *rowptr, *cols;
  float *logp, *lse, *entropy, *top_logp;
  int32_t* top_idx;
  float* bmax;            // [B][nblk] block maxima
  Stat* part;             // [B][splits]
};

// The pass over the row: the CTA's warps take its blocks in turn.  HBM-bound:
// every score is read once, in 16-byte loads, 128 (fp32) or 64 (bf16) bytes
// of a thread in flight.
template <typename T>
__device__ __forceinline__ Stat scan_row(const Args& A, const T* z, int shift, int64_t b, int split, Stat* red) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float m = -INFINITY, s = 0.0f, t = 0.0f;
  for (int64_t blk = (int64_t)split * kWarps + warp; blk < A.nblk; blk += (int64_t)A.splits * kWarps) {
    float v[32];
    load_block(z, A.L, shift, blk, lane, v);
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = fmaxf(fmaxf(v[e], v[e + 8]), fmaxf(v[e + 16], v[e + 24]));
    float bm = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
    for (int o = 16; o > 0; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xFFFFFFFFu, bm, o));
    if (lane == 0) A.bmax[b * A.nblk + blk] = bm;
    if (bm > m) {
      if (m > -INFINITY) {
        const float d = fmaxf(m - bm, kFloor), c = ex2(d * kLog2e);
        t = c * fmaf(s, d, t);
        s *= c;
      }
      m = bm;
    }
    const float m0 = m > -INFINITY ? m : 0.0f;
    float ps[4] = {0.0f, 0.0f, 0.0f, 0.0f}, pt[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const float d = max_nan(v[e] - m0, kFloor);
      const float p = ex2(d * kLog2e);
      ps[e & 3] += p;
      pt[e & 3] = fmaf(p, d, pt[e & 3]);
    }
    s += (ps[0] + ps[1]) + (ps[2] + ps[3]);
    t += (pt[0] + pt[1]) + (pt[2] + pt[3]);
  }
  for (int o = 16; o > 0; o >>= 1) {      // a warp's lanes share m
    s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
  }
  if (lane == 0) red[warp] = {m, s, t};
  __syncthreads();
  Stat r{-INFINITY, 0.0f, 0.0f};
  for (int w = 0; w < kWarps; ++w) r.m = fmaxf(r.m, red[w].m);
  for (int w = 0; w < kWarps; ++w) {
    const Stat p = red[w];
    if (p.m == -INFINITY) { r.s += p.s; continue; }       // 0, or NaN where the warp saw nothing but NaN
    const float d = fmaxf(p.m - r.m, kFloor), c = ex2(d * kLog2e);
    r.s = fmaf(p.s, c, r.s);
    r.t = fmaf(c, fmaf(p.s, d, p.t), r.t);
  }
  return r;
}

// ---------------------------------------------------------------- the row's answers
constexpr int kGroups = 128;              // a lower bound on the k-th best block comes from the groups' best
constexpr int kCand = 4096;               // keys the selection holds
constexpr int kBatch = kThreads * 8;      // keys added between two looks at the room

struct SmemJ {
  uint64_t cand[kCand];
  uint64_t gbest[kGroups];
  uint64_t tau;
  int n;
  double red[3 * kWarps];
  Stat row[kWarps];
};

// The keys cand[0 .. n) into descending order (n <= kCand), the rest zero.
__device__ __forceinline__ void sort_desc(uint64_t* cand, int n) {
  int size2 = 1;
  while (size2 < n) size2 <<= 1;
  for (int i = n + threadIdx.x; i < size2; i += kThreads) cand[i] = 0;
  __syncthreads();
  for (int size = 2; size <= size2; size <<= 1) {
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      for (int i = threadIdx.x; i < size2 / 2; i += kThreads) {
        const int lo = 2 * i - (i & (stride - 1)), hi = lo + stride;
        const uint64_t a = cand[lo], c = cand[hi];
        if ((a < c) == ((lo & size) == 0)) { cand[lo] = c; cand[hi] = a; }
      }
      __syncthreads();
    }
  }
}

// Labels and log probabilities of the row's k best scores.  Every thread of
// the CTA calls it.
template <typename T>
__device__ __forceinline__ void best_labels(const Args& A, const T* z, int shift, int64_t b, double m, double logs,
                                            SmemJ* S) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int k = A.k;
  const float* bm = A.bmax + b * A.nblk;
  // tau: the k-th best of the groups' best blocks is at most the k-th best block
  if (A.nblk <= kGroups) {
    if (tid < kGroups) S->gbest[tid] = tid < A.nblk ? key_of(order_of(__ldcg(bm + tid)), (uint32_t)tid) : 0ull;
  } else {
    const int grp = tid / (kThreads / kGroups);
    uint64_t best = 0;
    for (int j = grp + kGroups * (tid % (kThreads / kGroups)); j < A.nblk; j += kThreads) {
      const uint64_t c = key_of(order_of(__ldcg(bm + j)), (uint32_t)j);
      best = c > best ? c : best;
    }
    const uint64_t other = __shfl_xor_sync(0xFFFFFFFFu, best, 1);
    best = other > best ? other : best;
    if (tid % 2 == 0) S->gbest[grp] = best;
  }
  if (tid == 0) { S->tau = 0; S->n = 0; }
  __syncthreads();
  if (tid < kGroups) {
    const uint64_t mine = S->gbest[tid];
    int rank = 0;
    for (int j = 0; j < kGroups; ++j) rank += S->gbest[j] > mine;
    if (mine && rank == k - 1) S->tau = mine;
  }
  __syncthreads();
  const uint64_t tau = S->tau;                       // 0: fewer than k groups hold a score
  // k scores are at least the score of tau's block
  uint64_t floor_key = tau & 0xFFFFFFFF00000000ull;
  // the blocks from tau's up, a warp each
  for (int j0 = 0; j0 < A.nblk; j0 += kWarps * 32) {
    const int j = j0 + warp * 32 + lane;
    const uint64_t key = j < A.nblk ? key_of(order_of(__ldcg(bm + j)), (uint32_t)j) : 0ull;
    uint32_t todo = __ballot_sync(0xFFFFFFFFu, key >= tau && key != 0);
    // every warp goes round as often as the one with most blocks
    while (__syncthreads_or(todo != 0)) {
      float v[32];
      int64_t blk = 0;
      const bool on = todo != 0;
      if (on) {
        blk = j0 + warp * 32 + (__ffs((int)todo) - 1);
        todo &= todo - 1;
        load_block(z, A.L, shift, blk, lane, v);
      }
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {                  // 8 scores of a thread at a time: at most 2048 keys
        if (on) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float x = q == 0 ? v[e] : q == 1 ? v[8 + e] : q == 2 ? v[16 + e] : v[24 + e];
            const uint64_t c = key_of(order_of(x), (uint32_t)label_of<T>(shift, blk, lane, 8 * q + e));
            if (c != 0 && c >= floor_key) {
              const int at = atomicAdd(&S->n, 1);
              S->cand[at] = c;
            }
          }
        }
        __syncthreads();
        const int n = S->n;                          // read by all before any thread adds to it again
        if (__syncthreads_or(n > kCand - kBatch)) {  // no room for another batch: keep the k best
          sort_desc(S->cand, n);
          if (tid == 0) S->n = n < k ? n : k;
          if (n >= k && S->cand[k - 1] > floor_key) floor_key = S->cand[k - 1];
          __syncthreads();
        }
      }
    }
  }
  __syncthreads();
  const int n = S->n;
  auto put = [&](int rank, uint64_t c) {
    const int64_t l = index_of(c);
    A.top_idx[b * k + rank] = (int32_t)l;
    A.top_logp[b * k + rank] = (float)((double)score_at(z, l) - m - logs);
  };
  if (n <= kThreads) {
    if (tid < n) {
      const uint64_t mine = S->cand[tid];
      int rank = 0;
      for (int j = 0; j < n; ++j) rank += S->cand[j] > mine;
      if (rank < k) put(rank, mine);
    }
  } else {
    sort_desc(S->cand, n);
    if (tid < k && tid < n) put(tid, S->cand[tid]);
  }
  for (int r = n + tid; r < k; r += kThreads) {      // fewer scores than places
    A.top_idx[b * k + r] = -1;
    A.top_logp[b * k + r] = -INFINITY;
  }
}

// All of a row's answers from its joined statistics (in 64 bits).
template <typename T>
__device__ __forceinline__ void finish_row(const Args& A, const T* z, int shift, int64_t b, double m, double s, double t,
                                           SmemJ* S) {
  double logs, lse, H;
  if (m == -INFINITY) {                              // nothing left: s is 0 (or NaN)
    logs = 0.0;
    lse = s == 0.0 ? -INFINITY : NAN;
    H = s == 0.0 ? 0.0 : NAN;
  } else {
    logs = log(s);
    lse = m == INFINITY ? (double)INFINITY : m + logs;
    H = logs - t / s;
  }
  const int tid = threadIdx.x;
  if (tid == 0) {
    A.lse[b] = (float)lse;
    A.entropy[b] = (float)H;
  }
  const double mm = m == -INFINITY || m == INFINITY ? lse : m, ll = m == -INFINITY || m == INFINITY ? 0.0 : logs;
  int e0 = A.rowptr[b], e1 = A.rowptr[b + 1];
  e0 = max(e0, 0);
  e1 = min(e1, A.nnz);
  for (int e = e0 + tid; e < e1; e += kThreads) {
    const int32_t l = A.cols[e];
    float r = NAN;
    if (l >= 0 && l < A.L) {
      const float x = score_at(z, l);
      r = x == -INFINITY && !isnan(lse) ? -INFINITY : (float)((double)x - mm - ll);
    }
    A.logp[e] = r;
  }
  if (A.k > 0) best_labels(A, z, shift, b, mm, ll, S);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) score_scan_kernel(const Args A) {
  __shared__ Stat red[kWarps];
  const int64_t b = blockIdx.y;
  const T* z = static_cast<const T*>(A.Z) + b * A.ldz;
  const Stat r = scan_row(A, z, shift_of(z), b, blockIdx.x, red);
  if (threadIdx.x == 0) A.part[b * A.splits + blockIdx.x] = r;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) score_join_kernel(const Args A) {
  __shared__ SmemJ S;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t b = blockIdx.x;
  const T* z = static_cast<const T*>(A.Z) + b * A.ldz;
  const Stat* part = A.part + b * A.splits;
  float mf = -INFINITY;
  for (int i = tid; i < A.splits; i += kThreads) mf = fmaxf(mf, part[i].m);
  for (int o = 16; o > 0; o >>= 1) mf = fmaxf(mf, __shfl_xor_sync(0xFFFFFFFFu, mf, o));
  if (lane == 0) S.row[warp].m = mf;
  __syncthreads();
  for (int w = 0; w < kWarps; ++w) mf = fmaxf(mf, S.row[w].m);
  const double m = mf;
  double s = 0.0, t = 0.0;
  for (int i = tid; i < A.splits; i += kThreads) {
    const Stat p = part[i];
    if (p.m == -INFINITY) { s += p.s; continue; }
    const double d = (double)p.m - m, c = p.m == mf ? 1.0 : exp(d);
    s += c * p.s;
    t += c * (p.t + (p.m == mf ? 0.0 : d * p.s));
  }
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
  }
  if (lane == 0) { S.red[warp] = s; S.red[kWarps + warp] = t; }
  __syncthreads();
  s = t = 0.0;
  for (int w = 0; w < kWarps; ++w) { s += S.red[w]; t += S.red[kWarps + w]; }
  finish_row(A, z, shift_of(z), b, m, s, t, &S);
}

// Short rows: the pass and the answers in one CTA.
template <typename T>
__global__ void __launch_bounds__(kThreads) score_row_kernel(const Args A) {
  __shared__ SmemJ S;
  const int64_t b = blockIdx.x;
  const T* z = static_cast<const T*>(A.Z) + b * A.ldz;
  const int shift = shift_of(z);
  const Stat r = scan_row(A, z, shift, b, 0, S.row);
  __syncthreads();
  finish_row(A, z, shift, b, r.m, r.s, r.t, &S);
}

// ---------------------------------------------------------------- gradient
// With g_i, g_lse and g_H the gradients of the row's log p of label c_i, lse
// and entropy H:
//     dz_l = sum_{i: c_i = l} g_i + p_l (g_lse - sum_i g_i - g_H (log p_l + H)).
// One pass that reads z and writes dz (HBM-bound); the CTA of a segment first
// gathers the segment's given labels into a row of addends, so that a label
// given twice gets the sum in the order of the list, each dz is rounded once,
// and dz may take z's place.
constexpr int kSeg = 4096;

struct BwdArgs {
  const void* Z;
  void* dZ;
  int64_t ldz, lddz, L;
  int32_t nnz;
  const int32_t *rowptr, *cols;
  const float *lse, *entropy, *g_logp, *g_lse, *g_entropy;
};

template <typename T> __device__ __forceinline__ void put_grad(T* p, float v);
template <> __device__ __forceinline__ void put_grad<float>(float* p, float v) { *p = v; }
template <> __device__ __forceinline__ void put_grad<uint16_t>(uint16_t* p, float v) { *p = f32_to_bf16_rn(v); }

template <typename T>
__global__ void __launch_bounds__(kThreads) score_backward_kernel(const BwdArgs A) {
  constexpr int kE = Vec<T>::kE;
  __shared__ float addend[kSeg];
  __shared__ int32_t ids[kThreads];
  __shared__ float gs[kThreads];
  __shared__ double red[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t b = blockIdx.y;
  const T* z = static_cast<const T*>(A.Z) + b * A.ldz;
  T* dz = static_cast<T*>(A.dZ) + b * A.lddz;
  const int shift = shift_of(z);
  const int64_t first = (int64_t)blockIdx.x * kSeg - shift;       // the segment's labels: [first, first + kSeg)
  const float lse = A.lse[b];
  const bool dead = isinf(lse);                                   // no label, or no softmax: no gradient

  double sum = 0.0;
  bool any = false;
  const int e0 = max(A.rowptr[b], 0), e1 = min(A.rowptr[b + 1], A.nnz);
  if (A.g_logp && !dead) {
    for (int e = e0 + tid; e < e1; e += kThreads) {
      const int32_t l = A.cols[e];
      if (l < 0 || l >= A.L) continue;
      sum += A.g_logp[e];
      any |= l >= first && l < first + kSeg;
    }
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane == 0) red[warp] = sum;
    any = __syncthreads_or(any);
    sum = 0.0;
    for (int w = 0; w < kWarps; ++w) sum += red[w];
  }
  if (any) {
    for (int i = tid; i < kSeg; i += kThreads) addend[i] = 0.0f;
    for (int base = e0; base < e1; base += kThreads) {
      const int e = base + tid;
      int32_t l = -1;
      if (e < e1) {
        l = A.cols[e];
        if (l < 0 || l >= A.L || l < first || l >= first + kSeg) l = -1;
      }
      if (!__syncthreads_or(l >= 0)) continue;                    // also: addend is clear, the last round's reads are done
      ids[tid] = l;
      if (l >= 0) gs[tid] = A.g_logp[e];
      __syncthreads();
      if (l >= 0) {
        bool mine = true;
        for (int j = 0; j < tid && mine; ++j) mine = ids[j] != l;
        if (mine) {
          float g = addend[l - first];
          for (int j = tid; j < kThreads && base + j < e1; ++j)
            if (ids[j] == l) g += gs[j];
          addend[l - first] = g;
        }
      }
    }
    __syncthreads();
  }

  const float gH = A.g_entropy ? A.g_entropy[b] : 0.0f;
  const float H = A.g_entropy ? A.entropy[b] : 0.0f;
  const float c0 = (float)((A.g_lse ? (double)A.g_lse[b] : 0.0) - sum - (double)gH * (double)H);
  auto grad = [&](float x, int i) {
    const float d = max_nan(x - lse, kFloor);
    const float r = ex2(d * kLog2e) * fmaf(-gH, d, c0);
    return dead ? 0.0f : any ? r + addend[i] : r;
  };
  if (shift_of(dz) == shift) {
#pragma unroll 2
    for (int i0 = tid * kE; i0 < kSeg; i0 += kThreads * kE) {
      const int64_t l = first + i0;
      if (l >= 0 && l + kE <= A.L) {
        const uint4 q = *reinterpret_cast<const uint4*>(z + l);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (sizeof(T) == 4) {
            o[e] = __float_as_uint(grad(__uint_as_float(w[e]), i0 + e));
          } else {
            const float lo = grad(__uint_as_float(w[e] << 16), i0 + 2 * e);
            const float hi = grad(__uint_as_float(w[e] & 0xFFFF0000u), i0 + 2 * e + 1);
            o[e] = pack_bf16x2(hi, lo);
          }
        }
        *reinterpret_cast<uint4*>(dz + l) = make_uint4(o[0], o[1], o[2], o[3]);
      } else {
        for (int e = 0; e < kE; ++e)
          if (l + e >= 0 && l + e < A.L) put_grad(dz + l + e, grad(score_at(z, l + e), i0 + e));
      }
    }
  } else {
    for (int i = tid; i < kSeg; i += kThreads) {
      const int64_t l = first + i;
      if (l >= 0 && l < A.L) put_grad(dz + l, grad(score_at(z, l), i));
    }
  }
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// blocks of a row, wherever its first score lies
int32_t blocks_of(int64_t L) { return (int32_t)((L + 7 + kBlock - 1) / kBlock); }

int sms_of_device() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 1;
  return n;
}

template <typename T>
cudaError_t run_scores(Args A, int sms, cudaStream_t s) {
  if (A.splits == 1) {
    score_row_kernel<T><<<A.B, kThreads, 0, s>>>(A);
    return cudaGetLastError();
  }
  score_scan_kernel<T><<<dim3(A.splits, A.B), kThreads, 0, s>>>(A);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  score_join_kernel<T><<<A.B, kThreads, 0, s>>>(A);
  return cudaGetLastError();
}

}  // namespace

size_t score_logprobs_workspace(int32_t B, int64_t L, int32_t k) {
  (void)k;
  return align256(sizeof(float) * (size_t)B * blocks_of(L)) + align256(sizeof(Stat) * (size_t)B * kMaxSplit);
}

cudaError_t launch_score_logprobs(const void* Z, bool bf16, int64_t ldz, int32_t B, int64_t L, const int32_t* rowptr,
                                  const int32_t* cols, int32_t nnz, int32_t k, float* logp, float* lse, float* entropy,
                                  int32_t* top_idx, float* top_logp, void* work, cudaStream_t s) {
  Args A{};
  A.Z = Z;
  A.ldz = ldz; A.L = L; A.B = B; A.k = k; A.nnz = nnz;
  A.rowptr = rowptr; A.cols = cols;
  A.logp = logp; A.lse = lse; A.entropy = entropy; A.top_idx = top_idx; A.top_logp = top_logp;
  A.nblk = blocks_of(L);
  A.bmax = static_cast<float*>(work);
  A.part = reinterpret_cast<Stat*>(static_cast<char*>(work) + align256(sizeof(float) * (size_t)B * A.nblk));
  const int sms = sms_of_device();
  // enough CTAs to fill the machine four deep, at least a block for every warp
  int64_t splits = ((int64_t)sms * 4 + B - 1) / B;
  const int64_t most = (A.nblk + kWarps - 1) / kWarps;
  if (splits > most) splits = most;
  if (splits > kMaxSplit) splits = kMaxSplit;
  if (A.nblk <= 4 * kWarps) splits = 1;
  A.splits = (int32_t)splits;
  return bf16 ? run_scores<uint16_t>(A, sms, s) : run_scores<float>(A, sms, s);
}

cudaError_t launch_score_backward(const void* Z, bool bf16, int64_t ldz, int32_t B, int64_t L, const int32_t* rowptr,
                                  const int32_t* cols, int32_t nnz, const float* lse, const float* entropy,
                                  const float* g_logp, const float* g_lse, const float* g_entropy, void* dZ,
                                  int64_t lddz, cudaStream_t s) {
  const BwdArgs A{Z, dZ, ldz, lddz, L, nnz, rowptr, cols, lse, entropy, g_logp, g_lse, g_entropy};
  const dim3 grid((unsigned)((L + 7 + kSeg - 1) / kSeg), (unsigned)B);
  if (bf16) score_backward_kernel<uint16_t><<<grid, kThreads, 0, s>>>(A);
  else score_backward_kernel<float><<<grid, kThreads, 0, s>>>(A);
  return cudaGetLastError();
}

}  // namespace elmo
