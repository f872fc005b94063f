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
#include "softmax.cuh"
#include "tc_ptx.cuh"

namespace elmo {
namespace {

using namespace tc;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBlock = 1024;              // scores of a block
constexpr int kMaxSplit = 512;

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

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Adds a thread's 32 scores of a block to its sums; returns their maximum.
//
// bf16: two scores an instruction as far as that goes, or the issue slots bind
// (256 rows of 500K: 70 us with seven and more a score, 56 with five and a half):
// the maximum of the pairs, and -inf raised to the lowest finite number, whose
// e^ is 0 and whose product with 0 is 0.  Where that number itself may be the
// row's maximum, and on infinities and NaN, the sums are formed one by one.
__device__ __forceinline__ float add_block(Soft& soft, const float* z, int64_t L, int shift, int64_t blk, int lane) {
  float v[32];
  load_block(z, L, shift, blk, lane, v);
  const float mx = max32(v);
  soft.add32<true>(v, mx);
  return mx;
}
__device__ __forceinline__ float add_block(Soft& soft, const uint16_t* z, int64_t L, int shift, int64_t blk, int lane) {
  const int64_t first = blk * kBlock - shift;
  float v[32];
  if (first < 0 || first + kBlock > L) {
    load_block(z, L, shift, blk, lane, v);
    const float mx = max32(v);
    soft.add32<true>(v, mx);
    return mx;
  }
  const uint4* p = reinterpret_cast<const uint4*>(z + first) + lane;
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 q = __ldg(p + 32 * i);
    w[4 * i] = q.x; w[4 * i + 1] = q.y; w[4 * i + 2] = q.z; w[4 * i + 3] = q.w;
  }
  uint32_t x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = max_bf16x2(max_bf16x2(w[i], w[i + 4]), max_bf16x2(w[i + 8], w[i + 12]));
  x[0] = max_bf16x2(max_bf16x2(x[0], x[1]), max_bf16x2(x[2], x[3]));
  // all NaN: the maximum is NaN, which raises nothing
  const float mx = fmaxf(fmaxf(__uint_as_float(x[0] << 16), __uint_as_float(x[0] & 0xFFFF0000u)), -INFINITY);
  if (mx > soft.m) soft.raise(mx);
  const float m0 = soft.m > -INFINITY ? soft.m : 0.0f;
  float ss, tt;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t u = max_nan_bf16x2(w[i], 0xFF7FFF7Fu);
    v[2 * i] = __uint_as_float(u << 16);
    v[2 * i + 1] = __uint_as_float(u & 0xFFFF0000u);
  }
  soft.sums32<false>(v, m0, ss, tt);
  if (tt != tt || m0 < -1.0e38f) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
    soft.slow32(v, m0, ss, tt);
  }
  soft.s += ss;
  soft.t += tt;
  return mx;
}

// The pass over a part of a row: the CTA's warps take its blocks in turn.
// HBM-bound: every score is read once, in 16-byte loads, 128 (fp32) or 64
// (bf16) bytes of a thread in flight.
template <typename T>
__device__ __forceinline__ Stat scan_row(const Args& A, const T* z, int shift, int64_t b, int64_t blk0, int64_t blk1,
                                         Stat* red) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Soft soft(1.0f);
  for (int64_t blk = blk0 + warp; blk < blk1; blk += kWarps) {
    float bm = add_block(soft, z, A.L, shift, blk, lane);
    if (A.k > 0) {
      for (int o = 16; o > 0; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xFFFFFFFFu, bm, o));
      if (lane == 0) A.bmax[b * A.nblk + blk] = bm;
    }
  }
  soft.join_warp();
  if (lane == 0) red[warp] = {soft.m, soft.s, soft.t};
  __syncthreads();
  const Stat q = red[lane % kWarps];
  Soft all(1.0f);
  if (lane < kWarps) { all.m = q.m; all.s = q.s; all.t = q.t; }
  all.join_warp();
  return {all.m, all.s, all.t};
}

// ---------------------------------------------------------------- the row's answers
constexpr int kGroups = 128;              // a lower bound on the k-th best block comes from the groups' best
constexpr int kCand = 4096;               // keys the selection holds
constexpr int kList = 512;                // blocks that may hold them
constexpr int kBatch = kThreads * 8;      // keys added between two looks at the room

struct SmemJ {
  uint64_t cand[kCand];
  uint64_t gbest[kGroups];
  uint64_t tau;
  int32_t blocks[kList];
  int n, nb;
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

// The scores from floor_key up of the blocks from tau up, where they are more
// than fit: in batches, of which the k best stay.
template <typename T>
__device__ __noinline__ void best_of_many(const Args& A, const T* z, int shift, int64_t b, uint64_t tau,
                                          uint64_t floor_key, SmemJ* S) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int k = A.k;
  const float* bm = A.bmax + b * A.nblk;
  __syncthreads();
  if (tid == 0) S->n = 0;
  __syncthreads();
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
  if (tid == 0) { S->tau = 0; S->n = S->nb = 0; }
  __syncthreads();
  auto kth_group = [&] {                             // tau <- the k-th best of the groups
    if (tid < kGroups) {
      const uint64_t mine = S->gbest[tid];
      int rank = 0;
      for (int j = 0; j < kGroups; ++j) rank += S->gbest[j] > mine;
      if (mine && rank == k - 1) S->tau = mine;
    }
    __syncthreads();
  };
  kth_group();
  const uint64_t tau = S->tau;                       // 0: fewer than k blocks hold a score
  // k scores are at least the score of tau's block
  uint64_t floor_key = tau & 0xFFFFFFFF00000000ull;
  if (tau == 0) {                                    // few blocks: groups of pairs of threads, a thread's best score
    uint64_t best = 0;
    for (int64_t blk = warp; blk < A.nblk; blk += kWarps) {
      if (order_of(__ldcg(bm + blk)) == 0) continue;
      float v[32];
      load_block(z, A.L, shift, blk, lane, v);
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const uint64_t c = key_of(order_of(v[e]), (uint32_t)label_of<T>(shift, blk, lane, e));
        best = c > best ? c : best;
      }
    }
    const uint64_t other = __shfl_xor_sync(0xFFFFFFFFu, best, 1);
    best = other > best ? other : best;
    if (tid % 2 == 0) S->gbest[tid / 2] = best;
    __syncthreads();
    kth_group();
    floor_key = S->tau;
  }
  // the blocks from tau's up, then their scores from the floor up
  for (int j = tid; j < A.nblk; j += kThreads) {
    const uint64_t key = key_of(order_of(__ldcg(bm + j)), (uint32_t)j);
    if (key >= tau && key != 0) {
      const int at = atomicAdd(&S->nb, 1);
      if (at < kList) S->blocks[at] = j;
    }
  }
  __syncthreads();
  const int nb = S->nb;
  if (nb <= kList) {
    for (int j = warp; j < nb; j += kWarps) {
      const int64_t blk = S->blocks[j];
      float v[32];
      load_block(z, A.L, shift, blk, lane, v);
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        if (order_of(v[e]) < (uint32_t)(floor_key >> 32)) continue;
        const uint64_t c = key_of(order_of(v[e]), (uint32_t)label_of<T>(shift, blk, lane, e));
        if (c != 0 && c >= floor_key) {
          const int at = atomicAdd(&S->n, 1);
          if (at < kCand) S->cand[at] = c;
        }
      }
    }
    __syncthreads();
  }
  if (nb > kList || S->n > kCand) best_of_many(A, z, shift, b, tau, floor_key, S);   // ties, or scores in order
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
  pdl_trigger();
  const int64_t n = A.nblk, i = blockIdx.x;
  const Stat r = scan_row(A, z, shift_of(z), b, n * i / A.splits, n * (i + 1) / A.splits, red);
  if (threadIdx.x == 0) A.part[b * A.splits + i] = r;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) score_join_kernel(const Args A) {
  __shared__ SmemJ S;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t b = blockIdx.x;
  const T* z = static_cast<const T*>(A.Z) + b * A.ldz;
  const Stat* part = A.part + b * A.splits;
  pdl_wait();
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
  const Stat r = scan_row(A, z, shift, b, 0, A.nblk, S.row);
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

  // the scores before anything that waits for the row's lists
  constexpr int kVecs = kSeg / (kThreads * kE);
  const bool whole = first >= 0 && first + kSeg <= A.L && shift_of(dz) == shift;
  uint4 q[kVecs];
  if (whole) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) q[i] = __ldcs(reinterpret_cast<const uint4*>(z + first) + i * kThreads + tid);
  }

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
  auto grad = [&](float x) {
    const float d = max_nan(x - lse, kSoftFloor);
    return ex2(d * kLog2e) * fmaf(-gH, d, c0);
  };
  auto grad2 = [&](float x0, float x1, float& r0, float& r1) {
    float d0, d1, a0, a1;
    unpair(add2(pair(x0, x1), pair(-lse, -lse)), d0, d1);
    const f2 d = pair(max_nan(d0, kSoftFloor), max_nan(d1, kSoftFloor));
    unpair(mul2(d, pair(kLog2e, kLog2e)), a0, a1);
    unpair(mul2(pair(ex2(a0), ex2(a1)), fma2(pair(-gH, -gH), d, pair(c0, c0))), r0, r1);
  };
  if (whole && !dead) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int i0 = (i * kThreads + tid) * kE;
      const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
      float r[kE];
#pragma unroll
      for (int e = 0; e < kE / 2; ++e) {
        if (sizeof(T) == 4) grad2(__uint_as_float(w[2 * e]), __uint_as_float(w[2 * e + 1]), r[2 * e], r[2 * e + 1]);
        else grad2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u), r[2 * e], r[2 * e + 1]);
      }
      if (any) {
#pragma unroll
        for (int e = 0; e < kE; ++e) r[e] += addend[i0 + e];
      }
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = sizeof(T) == 4 ? __float_as_uint(r[e]) : pack_bf16x2(r[(2 * e + 1) % kE], r[(2 * e) % kE]);
      __stcs(reinterpret_cast<uint4*>(dz + first) + i * kThreads + tid, make_uint4(o[0], o[1], o[2], o[3]));
    }
  } else {
    for (int i = tid; i < kSeg; i += kThreads) {
      const int64_t l = first + i;
      if (l < 0 || l >= A.L) continue;
      float r = dead ? 0.0f : grad(score_at(z, l));
      if (any) r += addend[i];
      put_grad(dz + l, r);
    }
  }
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// blocks of a row, wherever its first score lies
int32_t blocks_of(int64_t L) { return (int32_t)((L + 7 + kBlock - 1) / kBlock); }

template <typename T>
cudaError_t run_scores(const Args& A, cudaStream_t s) {
  if (A.splits == 1) {
    score_row_kernel<T><<<A.B, kThreads, 0, s>>>(A);
    return cudaGetLastError();
  }
  score_scan_kernel<T><<<dim3(A.splits, A.B), kThreads, 0, s>>>(A);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_after(score_join_kernel<T>, dim3(A.B), kThreads, 0, s, A);
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
  const int sms = current_sms();
  // about 32 CTAs an SM, so that the last ones to end leave little idle, of
  // whole rounds of a block a warp
  int64_t per = ((int64_t)A.nblk * B / ((int64_t)sms * 32) + kWarps - 1) / kWarps * kWarps;
  if (per < kWarps) per = kWarps;
  int64_t splits = (A.nblk + per - 1) / per;
  if (splits > kMaxSplit) splits = kMaxSplit;
  if (A.nblk <= 4 * kWarps) splits = 1;
  A.splits = (int32_t)splits;
  return bf16 ? run_scores<uint16_t>(A, s) : run_scores<float>(A, s);
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
