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
// blocks finds the best labels.  Where more blocks or scores come near the k-th
// best than are held, as in sorted rows or among many equal scores, one CTA goes
// through those blocks in turn: 256 rows of 500K bf16 scores, 10 best, take 66 us
// unordered, 0.64 ms if they ascend, 0.23 if they descend and 1.2 if all are
// equal; one row of 3M fp32, 5 best, 0.18, 0.06 and 1.8 ms in place of 14 us.
//
// Masked labels are scores of -inf; a row may be all masked.
//
// On B200: 256 rows of 500K bf16 scores, pass 55 us (4.7 TB/s) and answers 14
// behind it.  Nothing saturates in the pass: exponentials 61 %, issue slots 60,
// DRAM 59; the 64 registers leave four CTAs an SM, with one block a warp in
// flight.  256 rows of 500K fp32 scores 97 us (5.3 TB/s); one row of 3M 14 us in
// all, of which the pass is 7; 33 rows of 4099 in one launch 12 us; 4096 rows of
// 16,000 (0.87 TB/s) 300 us, between the barriers of a CTA a row.  Gradient of
// the 256 rows: 88 us (5.8 TB/s).
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
constexpr int kMaxParts = 1024;           // CTAs of the pass

// A score's place in the order as a whole number: larger is better, 0 for a
// score that is never listed (-inf, NaN).  -0 and 0 are the same score.
__device__ __forceinline__ uint32_t order_of(float z) {
  if (!(z > -INFINITY)) return 0u;
  const uint32_t u = __float_as_uint(z + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float score_of(uint32_t order) {
  return __uint_as_float((order & 0x80000000u) ? (order & 0x7FFFFFFFu) : ~order);
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
// scores [j kBlock - shift, (j + 1) kBlock - shift).  A lane of a warp has 32
// of its 1024: kV vectors of 16 bytes.
template <typename T> struct Vec { static constexpr int kE = 16 / sizeof(T); static constexpr int kV = 32 / kE; };

// The 16 bytes of scores at, at + 1, ... of which some lie outside [0, L): -inf for those.
template <typename T>
__device__ __noinline__ uint4 ragged_vector(const T* z, int64_t L, int64_t at) {
  uint32_t w[4];
  auto bits = [&](int64_t l) -> uint32_t {
    const uint32_t b = __float_as_uint(l < 0 || l >= L ? -INFINITY : score_at(z, l));
    return sizeof(T) == 4 ? b : b >> 16;
  };
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = sizeof(T) == 4 ? bits(at + e) : bits(at + 2 * e) | (bits(at + 2 * e + 1) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T>
__device__ __forceinline__ uint4 load_vector(const T* z, int64_t L, int64_t at) {
  if (at >= 0 && at + Vec<T>::kE <= L) return __ldg(reinterpret_cast<const uint4*>(z + at));
  return ragged_vector(z, L, at);
}

// Calls f(label, score) for the scores of a lane's i-th vector of a block, -inf for those that are none.
template <typename T, typename F>
__device__ __forceinline__ void visit_vector(const T* z, int64_t L, int shift, int64_t block, int i, int lane, F f) {
  const int64_t at = block * kBlock - shift + (32 * i + lane) * Vec<T>::kE;
  const uint4 q = load_vector(z, L, at);
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (sizeof(T) == 4) {
      f(at + e, __uint_as_float(w[e]));
    } else {
      f(at + 2 * e, __uint_as_float(w[e] << 16));
      f(at + 2 * e + 1, __uint_as_float(w[e] & 0xFFFF0000u));
    }
  }
}

template <typename T> __host__ __device__ __forceinline__ int shift_of(const T* row) {
  return (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
}

struct Args {
  const void* Z;
  int64_t ldz, L;
  int32_t B, k, nnz, nblk, parts;
  const int32_t *rowptr, *cols;
  float *logp, *lse, *entropy, *top_logp;
  int32_t* top_idx;
  float* bmax;            // [B][nblk] block maxima
  Stat* part;             // [parts + B] sums of each part of a row
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

// two bf16 numbers less an fp32 one
__device__ __forceinline__ f2 minus_f32(uint32_t w, float m) {
  float a, b;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tadd.rn.f32.bf16 %0, l, %3;\n\tadd.rn.f32.bf16 %1, h, %3;\n\t}"
      : "=f"(a), "=f"(b) : "r"(w), "f"(-m));
  return pair(a, b);
}

// A lane's 32 scores of a block as they are stored.
template <typename T> struct Raw { uint4 q[Vec<T>::kV]; };

template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* z, int64_t L, int64_t first, int lane) {
  Raw<T> r;
  if (first >= 0 && first + kBlock <= L) {
#pragma unroll
    for (int i = 0; i < Vec<T>::kV; ++i) r.q[i] = __ldg(reinterpret_cast<const uint4*>(z + first) + 32 * i + lane);
  } else {                                             // a row's first or last block
#pragma unroll
    for (int i = 0; i < Vec<T>::kV; ++i) r.q[i] = load_vector(z, L, first + (32 * i + lane) * Vec<T>::kE);
  }
  return r;
}

// Adds a lane's 32 scores to its sums; returns their maximum.
//
// bf16: two scores an instruction as far as that goes, which spares issue
// slots: the maximum of the pairs, and -inf raised to the lowest finite number,
// whose e^ is 0 and whose product with 0 is 0.  Where that number itself may be
// the row's maximum, and on infinities and NaN, the sums are formed one by one.
__device__ __forceinline__ float add_raw(Soft& soft, const Raw<float>& r) {
  float v[32];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[4 * i] = __uint_as_float(r.q[i].x);
    v[4 * i + 1] = __uint_as_float(r.q[i].y);
    v[4 * i + 2] = __uint_as_float(r.q[i].z);
    v[4 * i + 3] = __uint_as_float(r.q[i].w);
  }
  const float mx = max32(v);
  soft.add32(v, mx);
  return mx;
}
__device__ __forceinline__ float add_raw(Soft& soft, const Raw<uint16_t>& r) {
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[4 * i] = r.q[i].x;
    w[4 * i + 1] = r.q[i].y;
    w[4 * i + 2] = r.q[i].z;
    w[4 * i + 3] = r.q[i].w;
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
  soft.sums32([&](int c) { return minus_f32(max_nan_bf16x2(w[c], 0xFF7FFF7Fu), m0); }, ss, tt);
  if (tt != tt || m0 < -1.0e38f) {
    float v[32];
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

// The CTA's pass over blocks [blk0, blk1) of a row: the sums (in every thread)
// and, for the list, the maxima of the blocks.  Warps take the blocks in
// turn (not from a counter: the sums would depend on who came first).
// HBM-bound: every score is read once, in 16-byte loads, the next block's 128
// (fp32) or 64 (bf16) bytes of a lane in flight while this one's are added.
template <int kW> struct SmemS { Stat row[kW]; };

template <int kW, typename T>
__device__ __forceinline__ Stat scan_blocks(const Args& A, const T* z, int64_t b, int blk0, int blk1, SmemS<kW>* S) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int shift = shift_of(z);
  Soft soft;
  Raw<T> next;
  int blk = blk0 + warp;
  if (blk < blk1) next = load_raw(z, A.L, (int64_t)blk * kBlock - shift, lane);
  while (blk < blk1) {
    const Raw<T> now = next;
    const int then = blk + kW;
    if (then < blk1) next = load_raw(z, A.L, (int64_t)then * kBlock - shift, lane);
    float bm = add_raw(soft, now);
    if (A.k > 0) {
      for (int o = 16; o > 0; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xFFFFFFFFu, bm, o));
      if (lane == 0) A.bmax[b * A.nblk + blk] = bm;
    }
    blk = then;
  }
  soft.join_warp();
  __syncthreads();                                     // the last segment's sums are read
  if (lane == 0) S->row[warp] = {soft.m, soft.s, soft.t};
  __syncthreads();
  Soft all;
  if (lane < kW) { all.m = S->row[lane].m; all.s = S->row[lane].s; all.t = S->row[lane].t; }
  all.join_warp();
  return {all.m, all.s, all.t};
}

// All rows' blocks are one run, cut into equal parts for the CTAs that the
// machine holds: a part may cross rows, and its sums of row b go to slot
// part + b, which no other part has and which keeps a row's slots together.
__device__ __forceinline__ int64_t part_of(int64_t block, int64_t blocks, int64_t parts) {
  return ((block + 1) * parts - 1) / blocks;
}

// ---------------------------------------------------------------- the row's answers
constexpr int kJoinThreads = 512;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kGroups = 128;              // groups of blocks, whose best bound the k-th best block from below
constexpr int kHold = 8;                  // block maxima that a thread keeps
constexpr int kCand = 4096;               // scores that the selection holds
constexpr int kList = 512;                // blocks that may hold the k best

struct SmemJ {
  uint64_t cand[kCand];
  alignas(16) uint32_t gbest[kGroups];
  uint32_t tau;
  int32_t blocks[kList];
  int n, nb;
  double red[2 * kJoinWarps];
  float m[kJoinWarps];
};

// The keys cand[0 .. n) into descending order (n <= kCand), the rest zero.
__device__ __forceinline__ void sort_desc(uint64_t* cand, int n) {
  int size2 = 1;
  while (size2 < n) size2 <<= 1;
  for (int i = n + threadIdx.x; i < size2; i += kJoinThreads) cand[i] = 0;
  __syncthreads();
  for (int size = 2; size <= size2; size <<= 1) {
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      for (int i = threadIdx.x; i < size2 / 2; i += kJoinThreads) {
        const int lo = 2 * i - (i & (stride - 1)), hi = lo + stride;
        const uint64_t a = cand[lo], c = cand[hi];
        if ((a < c) == ((lo & size) == 0)) { cand[lo] = c; cand[hi] = a; }
      }
      __syncthreads();
    }
  }
}

// The k best of the blocks whose maximum has at least order tau, where the
// blocks or their scores are more than fit: a block at a time, and the k best
// stay when the room runs out.
template <typename T>
__device__ __noinline__ void best_of_many(const Args& A, const T* z, int shift, int64_t b, uint32_t tau, SmemJ* S) {
  constexpr int kV = Vec<T>::kV;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int k = A.k;
  const float* bm = A.bmax + b * A.nblk;
  uint64_t floor_key = (uint64_t)tau << 32;
  __syncthreads();
  if (tid == 0) S->n = 0;
  for (int j0 = 0; j0 < A.nblk; j0 += kJoinThreads) {
    __syncthreads();
    if (tid == 0) S->nb = 0;
    __syncthreads();
    const uint32_t o = j0 + tid < A.nblk ? order_of(__ldcg(bm + j0 + tid)) : 0u;
    if (o >= tau && o != 0) S->blocks[atomicAdd(&S->nb, 1)] = j0 + tid;
    __syncthreads();
    const int nb = S->nb;
    for (int i = 0; i < nb; ++i) {
      for (int v = warp; v < kV; v += kJoinWarps)
        visit_vector(z, A.L, shift, S->blocks[i], v, lane, [&](int64_t l, float x) {
          const uint64_t c = key_of(order_of(x), (uint32_t)l);
          if (c != 0 && c >= floor_key) S->cand[atomicAdd(&S->n, 1)] = c;
        });
      __syncthreads();
      const int n = S->n;                              // read by all before any thread adds to it again
      if (__syncthreads_or(n > kCand - kBlock)) {
        sort_desc(S->cand, n);
        if (tid == 0) S->n = n < k ? n : k;
        if (n >= k && S->cand[k - 1] > floor_key) floor_key = S->cand[k - 1];
        __syncthreads();
      }
    }
  }
  __syncthreads();
}

// tau <- the k-th best order of groups of neighbouring threads (0: fewer than
// k hold a score), each thread's best given.
__device__ __forceinline__ uint32_t kth_of_groups(uint32_t best, int k, SmemJ* S) {
  constexpr int kPer = kJoinThreads / kGroups;
  const int tid = threadIdx.x;
  for (int o = 1; o < kPer; o <<= 1) best = max(best, __shfl_xor_sync(0xFFFFFFFFu, best, o));
  __syncthreads();
  if (tid % kPer == 0) S->gbest[tid / kPer] = best;
  if (tid == 0) S->tau = 0;
  __syncthreads();
  if (tid < kGroups) {
    const uint32_t mine = S->gbest[tid];
    int above = 0, same = 0;
    for (int j = 0; j < kGroups; j += 4) {
      const uint4 o = *reinterpret_cast<const uint4*>(S->gbest + j);
      above += (o.x > mine) + (o.y > mine) + (o.z > mine) + (o.w > mine);
      same += (o.x == mine) + (o.y == mine) + (o.z == mine) + (o.w == mine);
    }
    if (above < k && above + same >= k) S->tau = mine;
  }
  __syncthreads();
  return S->tau;
}

// Labels and log probabilities of the row's k best scores.  Every thread of
// the CTA calls it.
template <typename T>
__device__ __forceinline__ void best_labels(const Args& A, const T* z, int shift, int64_t b, double m, double logs,
                                            SmemJ* S) {
  constexpr int kV = Vec<T>::kV;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int k = A.k;
  const float* bm = A.bmax + b * A.nblk;
  // the blocks' orders, the first kHold of a thread kept
  uint32_t held[kHold], best = 0;
#pragma unroll
  for (int i = 0; i < kHold; ++i) {
    const int j = tid + i * kJoinThreads;
    held[i] = j < A.nblk ? order_of(__ldcg(bm + j)) : 0u;
  }
#pragma unroll
  for (int i = 0; i < kHold; ++i) best = max(best, held[i]);
  for (int j = tid + kHold * kJoinThreads; j < A.nblk; j += kJoinThreads) best = max(best, order_of(__ldcg(bm + j)));
  if (tid == 0) S->n = S->nb = 0;
  // the k-th best of the groups' best is at most the k-th best block's
  uint32_t tau = kth_of_groups(best, k, S);
  auto list = [&](int j, uint32_t o) {
    if (o >= tau && o != 0) {
      const int at = atomicAdd(&S->nb, 1);
      if (at < kList) S->blocks[at] = j;
    }
  };
#pragma unroll
  for (int i = 0; i < kHold; ++i) list(tid + i * kJoinThreads, held[i]);
  for (int j = tid + kHold * kJoinThreads; j < A.nblk; j += kJoinThreads) list(j, order_of(__ldcg(bm + j)));
  __syncthreads();
  const int nb = S->nb;
  bool fits = nb <= kList;
  if (tau == 0 && fits) {                              // few blocks: the threads' best scores in their place
    best = 0;
#pragma unroll 2
    for (int it = warp; it < nb * kV; it += kJoinWarps)
      visit_vector(z, A.L, shift, S->blocks[it / kV], it % kV, lane,
                   [&](int64_t, float x) { best = max(best, order_of(x)); });
    tau = kth_of_groups(best, k, S);
  }
  if (fits) {                                          // k scores have at least order tau
#pragma unroll 2
    for (int it = warp; it < nb * kV; it += kJoinWarps) {
      visit_vector(z, A.L, shift, S->blocks[it / kV], it % kV, lane, [&](int64_t l, float x) {
        const uint32_t o = order_of(x);
        if (o >= tau && o != 0) {
          const int at = atomicAdd(&S->n, 1);
          if (at < kCand) S->cand[at] = key_of(o, (uint32_t)l);
        }
      });
    }
    __syncthreads();
    fits = S->n <= kCand;
  }
  if (!fits) best_of_many(A, z, shift, b, tau, S);     // ties, or scores in order
  const int n = S->n;
  auto put = [&](int rank, uint64_t c) {
    A.top_idx[b * k + rank] = (int32_t)index_of(c);
    A.top_logp[b * k + rank] = (float)((double)score_of((uint32_t)(c >> 32)) - m - logs);
  };
  if (n <= kJoinThreads) {
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
  for (int r = n + tid; r < k; r += kJoinThreads) {    // fewer scores than places
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
  } else if (m == INFINITY) {                        // s counts the infinities, a NaN makes it NaN
    logs = 0.0;
    lse = isnan(s) ? (double)NAN : (double)INFINITY;
    H = NAN;
  } else {
    logs = log(s);
    lse = m + logs;
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
  for (int e = e0 + tid; e < e1; e += kJoinThreads) {
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

// The CTAs of the pass that an SM holds.
template <typename T> constexpr int kResident = sizeof(T) == 4 ? 2 : 4;

template <typename T>
__global__ void __launch_bounds__(kThreads, kResident<T>) score_scan_kernel(const Args A) {
  __shared__ SmemS<kWarps> S;
  pdl_trigger();
  const int64_t w = blockIdx.x;
  const int64_t N = (int64_t)A.B * A.nblk, end = N * (w + 1) / A.parts;
  for (int64_t at = N * w / A.parts; at < end;) {
    const int64_t b = at / A.nblk, stop = min(end, (b + 1) * A.nblk);
    const Stat q = scan_blocks<kWarps>(A, static_cast<const T*>(A.Z) + b * A.ldz, b, (int)(at - b * A.nblk),
                               (int)(stop - b * A.nblk), &S);
    if (threadIdx.x == 0) A.part[w + b] = q;
    at = stop;
  }
}

template <typename T>
__global__ void __launch_bounds__(kJoinThreads) score_join_kernel(const Args A) {
  __shared__ SmemJ S;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t b = blockIdx.x;
  const T* z = static_cast<const T*>(A.Z) + b * A.ldz;
  const int64_t N = (int64_t)A.B * A.nblk;
  const int64_t w0 = part_of(b * A.nblk, N, A.parts), w1 = part_of((b + 1) * A.nblk - 1, N, A.parts);
  const Stat* part = A.part + w0 + b;
  const int n = (int)(w1 - w0 + 1);                    // at most kMaxParts: two of a thread
  pdl_wait();
  Stat q[2];
  float mf = -INFINITY;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    q[i] = tid + i * kJoinThreads < n ? part[tid + i * kJoinThreads] : Stat{-INFINITY, 0.0f, 0.0f};
    mf = fmaxf(mf, q[i].m);
  }
  for (int o = 16; o > 0; o >>= 1) mf = fmaxf(mf, __shfl_xor_sync(0xFFFFFFFFu, mf, o));
  if (lane == 0) S.m[warp] = mf;
  __syncthreads();
  for (int w = 0; w < kJoinWarps; ++w) mf = fmaxf(mf, S.m[w]);
  const double m = mf;
  double s = 0.0, t = 0.0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (q[i].m == -INFINITY) { s += q[i].s; continue; }
    const double d = (double)q[i].m - m, c = q[i].m == mf ? 1.0 : exp(d);
    s += c * q[i].s;
    t += c * (q[i].t + (q[i].m == mf ? 0.0 : d * q[i].s));
  }
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
  }
  if (lane == 0) { S.red[warp] = s; S.red[kJoinWarps + warp] = t; }
  __syncthreads();
  s = t = 0.0;
  for (int w = 0; w < kJoinWarps; ++w) { s += S.red[w]; t += S.red[kJoinWarps + w]; }
  finish_row(A, z, shift_of(z), b, m, s, t, &S);
}

// Short rows: the pass and the answers in one CTA.
template <typename T>
__global__ void __launch_bounds__(kJoinThreads) score_row_kernel(const Args A) {
  __shared__ SmemJ S;
  __shared__ SmemS<kJoinWarps> P;
  const int64_t b = blockIdx.x;
  const T* z = static_cast<const T*>(A.Z) + b * A.ldz;
  const Stat q = scan_blocks<kJoinWarps>(A, z, b, 0, A.nblk, &P);
  finish_row(A, z, shift_of(z), b, q.m, q.s, q.t, &S);
}

// ---------------------------------------------------------------- gradient
// With g_i, g_lse and g_H the gradients of the row's log p of label c_i, lse
// and entropy H:
//     dz_l = sum_{i: c_i = l} g_i + p_l (g_lse - sum_i g_i - g_H (log p_l + H)).
// One pass that reads z and writes dz (HBM-bound), a warp a segment: its scores
// are on their way while it goes through the row's list, and no warp waits for
// another (a CTA a segment of 4096, with barriers around the list, took 100 us
// for 256 rows of 500K bf16 scores).  The segment's given labels go into a row
// of addends first, so that a label given twice gets the sum in the order of
// the list, each dz is rounded once, and dz may take z's place.
// Every warp reads its row's whole list, and the part of it from its segment's
// labels in steps of 32: 256 rows of 500K bf16 scores take 82, 107, 382 and 3310
// us with 4, 100, 1000 and 10,000 given labels a row.
constexpr int kSeg = 1024;

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
__global__ void __launch_bounds__(kThreads, 5) score_backward_kernel(const BwdArgs A) {
  constexpr int kE = Vec<T>::kE, kV = Vec<T>::kV;
  __shared__ float addends[kWarps][kSeg];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* addend = addends[warp];
  const int64_t b = blockIdx.y;
  const T* z = static_cast<const T*>(A.Z) + b * A.ldz;
  T* dz = static_cast<T*>(A.dZ) + b * A.lddz;
  const int shift = shift_of(z);
  const int64_t first = ((int64_t)blockIdx.x * kWarps + warp) * kSeg - shift;   // the labels [first, first + kSeg)
  if (first >= A.L) return;
  const bool whole = first >= 0 && first + kSeg <= A.L && shift_of(dz) == shift;
  uint4 q[kV];
  if (whole) {
#pragma unroll
    for (int i = 0; i < kV; ++i) q[i] = __ldcs(reinterpret_cast<const uint4*>(z + first) + 32 * i + lane);
  }
  const float lse = A.lse[b];
  const bool dead = isinf(lse);                                   // no label, or no softmax: no gradient

  double sum = 0.0;
  bool any = false;
  const int e0 = min(max(A.rowptr[b], 0), A.nnz), e1 = min(A.rowptr[b + 1], A.nnz);
  if (A.g_logp && !dead) {
    for (int e = e0 + lane; e < e1; e += 32) {
      const int32_t l = A.cols[e];
      if (l < 0 || l >= A.L) continue;
      sum += A.g_logp[e];
      any |= l >= first && l < first + kSeg;
    }
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    any = __any_sync(0xFFFFFFFFu, any);
  }
  if (any) {
    for (int i = lane; i < kSeg; i += 32) addend[i] = 0.0f;
    for (int base = e0; base < e1; base += 32) {
      const int e = base + lane;
      int32_t l = -1;
      float g = 0.0f;
      if (e < e1) {
        l = A.cols[e];
        if (l < 0 || l >= A.L || l < first || l >= first + kSeg) l = -1;
        else g = A.g_logp[e];
      }
      if (!__any_sync(0xFFFFFFFFu, l >= 0)) continue;
      // the first lane that has a label adds those of all that have it, in order
      const uint32_t same = __match_any_sync(0xFFFFFFFFu, l);
      const bool leads = l >= 0 && (same & ((1u << lane) - 1u)) == 0;
      __syncwarp();
      float acc = leads ? addend[l - first] : 0.0f;
#pragma unroll 4
      for (int j = 0; j < 32; ++j) {
        const float gj = __shfl_sync(0xFFFFFFFFu, g, j);
        if ((same >> j) & 1u) acc += gj;
      }
      if (leads) addend[l - first] = acc;
    }
    __syncwarp();
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
    for (int i = 0; i < kV; ++i) {
      const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
      float r[kE];
#pragma unroll
      for (int e = 0; e < kE / 2; ++e) {
        if (sizeof(T) == 4) grad2(__uint_as_float(w[2 * e]), __uint_as_float(w[2 * e + 1]), r[2 * e], r[2 * e + 1]);
        else grad2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u), r[2 * e], r[2 * e + 1]);
      }
      if (any) {
#pragma unroll
        for (int e = 0; e < kE; ++e) r[e] += addend[(32 * i + lane) * kE + e];
      }
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = sizeof(T) == 4 ? __float_as_uint(r[e]) : pack_bf16x2(r[(2 * e + 1) % kE], r[(2 * e) % kE]);
      __stcs(reinterpret_cast<uint4*>(dz + first) + 32 * i + lane, make_uint4(o[0], o[1], o[2], o[3]));
    }
  } else {
    for (int i = lane; i < kSeg; i += 32) {
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
cudaError_t run_scores(Args A, cudaStream_t s) {
  // rows of up to two blocks a warp: one launch
  if (A.nblk <= 2 * kJoinWarps) {
    score_row_kernel<T><<<A.B, kJoinThreads, 0, s>>>(A);
    return cudaGetLastError();
  }
  const int64_t N = (int64_t)A.B * A.nblk;
  int64_t parts = (int64_t)current_sms() * kResident<T>;
  if (parts > kMaxParts) parts = kMaxParts;
  if (parts > N / kWarps) parts = N / kWarps;          // a block a warp at least
  A.parts = (int32_t)parts;
  score_scan_kernel<T><<<(unsigned)parts, kThreads, 0, s>>>(A);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_after(score_join_kernel<T>, dim3(A.B), kJoinThreads, 0, s, A);
}

}  // namespace

size_t score_logprobs_workspace(int32_t B, int64_t L, int32_t k) {
  (void)k;
  return align256(sizeof(float) * (size_t)B * blocks_of(L)) + align256(sizeof(Stat) * ((size_t)B + kMaxParts));
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
  return bf16 ? run_scores<uint16_t>(A, s) : run_scores<float>(A, s);
}

cudaError_t launch_score_backward(const void* Z, bool bf16, int64_t ldz, int32_t B, int64_t L, const int32_t* rowptr,
                                  const int32_t* cols, int32_t nnz, const float* lse, const float* entropy,
                                  const float* g_logp, const float* g_lse, const float* g_entropy, void* dZ,
                                  int64_t lddz, cudaStream_t s) {
  const BwdArgs A{Z, dZ, ldz, lddz, L, nnz, rowptr, cols, lse, entropy, g_logp, g_lse, g_entropy};
  const dim3 grid((unsigned)((L + 7 + kSeg * kWarps - 1) / (kSeg * kWarps)), (unsigned)B);
  if (bf16) score_backward_kernel<uint16_t><<<grid, kThreads, 0, s>>>(A);
  else score_backward_kernel<float><<<grid, kThreads, 0, s>>>(A);
  return cudaGetLastError();
}

}  // namespace elmo
