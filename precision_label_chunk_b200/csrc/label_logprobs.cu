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
//      s_b max|x| in (224, 448] (s_b at most 2^126), hi = rne_e4m3(s_b x), lo = rne_e5m2(s_b x - hi).
//      A bf16 number has 8 significant bits, hi takes 4 and leaves at most 8
//      units of the last place, which E5M2's 3 bits hold exactly.  Only below
//      E4M3's normal numbers, 2^-6 and so at most 2^-13 of the query's largest,
//      may more be left; lo is then at most 2^-10 and rounds to within 2^-14,
//      2^-21 of the largest.
//   2. score pass (tcgen05): 128 queries against a range of labels a CTA; an
//      epilogue thread has one query and keeps its running maximum m,
//      s = sum e^(z - m) and t = sum e^(z - m)(z - m).  For the list it only
//      notes the maximum of every block of labels, which the running maximum
//      needs anyway: keeping the best scores in the pass (a heap a query,
//      limits shared between the ranges) took 1841 us for 3M labels and 256
//      queries, where the pass now takes 1032 in a loop.
//   3. join: the ranges' sums in 64 bits; the given labels' scores recomputed
//      exactly (products exact, sums in 64 bits); and the k best labels.  Let
//      low be at most the k-th best block maximum.  k labels score at least
//      low on the tensor cores, so a label among the k best does so to within
//      2 delta, delta the error bound of those scores: the blocks with a
//      maximum of at least low - 2 delta hold all of the k best.  Their labels
//      are scored again in fp32, which narrows them down the same way, and
//      what is left is ranked by exact scores.  Heads of few labels keep all
//      their tensor-core scores in place of the maxima: with fewer blocks than
//      a few times k, most labels would be scored again (1571 labels, 180
//      queries, 5 best: 86 us).
//   4. queries with too many labels within 2 delta (ties), or with sums that
//      may leave fp32's range, or a head that is not finite, rank all labels
//      by exact scores on the CUDA cores: with all labels tied 0.35 ms for 500K
//      bf16 labels x 768 and one query, 0.87 for 4; 22 ms for 3M E4M3 labels
//      and 16.  One weight far above all others does that too (see delta).
//
// delta = (eps nw + r1) max|W|, r1 the sum of what hi and lo leave.  How the
// accumulating instructions round is documented nowhere.  Measured on B200, one
// cuts each product at 2^-25 of the largest addend, the sum so far among them,
// and the sum to fp32: crafted queries lost 2^-21.0 of the magnitudes summed an
// instruction of 16 products (16-bit operands) and 2^-20.0 of 32 (8-bit).  eps
// allows half as much again, 1.5 2^-25 a product (2^-22 an instruction puts such
// labels in the wrong order).  An element of X counts for the instructions
// from its own on, nw = sum_j (|hi| n(hi_j) + |lo| n(lo_j)) / s_b with n that
// number: a cut is one of the sum so far.  (Every element for every
// instruction, and as much for the fp32 scores, sent 64 queries against 1M
// E4M3 labels x 4096, 64 best, to the exact path: 61 ms in place of 1.6.)
// The fp32 scores are off by 2^-24 of the magnitudes for each addition of a
// chain: d / 32 products a lane and 5 joins.  max|W| is read off the tiles in
// shared memory by two spare warps.  One weight far above the others widens
// delta for every label, and from some hundred times their deviation on queries
// go to the exact path: with a deviation of 0.02, one weight of 8 costs 3M E4M3
// labels x 768 nothing, one of 448 takes 16 queries from 0.5 to 22 ms; x 2048,
// one of 4 takes 4 queries from 2.9 to 13 ms.
//
// Bounds and times on B200.  Few queries: the read of W; 500K bf16 labels x
// 768, 4 queries: pass 123 us (6.2 TB/s), all of it 158.  Many: the tensor pipe is
// the busiest unit (62 %, 500K E4M3 labels, 256 queries; issue slots 30, DRAM 29),
// and what it waits for is not measured: most likely the shared memory that the
// MMAs and the copies share, with 64 labels an instruction; 3M E4M3 labels, 256
// queries: pass 1032 us, 2.3 PFLOP/s of 8-bit products (two a weight), all of it
// 1175 in a loop, at the power limit and 1440 MHz; 1028 for single calls; 64 best
// in place of 5 take 1305.  E5M2 1204.  500K bf16, 256 queries 285.  Small heads:
// the launches; 20K bf16 labels x 256, 4 queries 31 us.  Narrow heads: the
// epilogue; 1M labels x 64, 128 queries: 70 us.
#include <cuda.h>
#include <float.h>

#include "elmo_common.cuh"
#include "elmo_internal.h"
#include "elmo_operators.h"
#include "softmax.cuh"
#include "tc_ptx.cuh"
#include "weights8.cuh"

namespace elmo {
namespace {

using namespace tc;

constexpr int kStreams = 4;               // groups of four epilogue warps: even or odd tiles, left or right half
constexpr int kEpi = 2 + 4 * kStreams;    // warp 0 TMA, 1 MMA and TMEM, 2 .. kEpi - 1 epilogue, then two for max|W|
constexpr int kThreads = 32 * (kEpi + 2);
constexpr int kMaxStages = 16;
constexpr int kMaxBufs = 4;               // accumulators
constexpr long long kWait = 4000000000LL; // ~2 s
constexpr size_t kSmemMost = 227 * 1024;
constexpr size_t kMaxima = size_t(256) << 20;   // bytes of block maxima, about
constexpr int64_t kKeepLabels = 16384;    // heads of up to so many labels keep every score instead,
constexpr size_t kKeepBytes = size_t(64) << 20;   // if they take no more than this
constexpr int kJoinThreads = 512;
constexpr int kGroups = 256;              // groups whose best give the lower bound on the k-th best
constexpr int kMaxBlocks = 2048;          // blocks that are scored again for a query,
constexpr int kMaxNear = 4096;            // of their labels the ones near the k-th best in fp32,
constexpr int kMaxExact = 1024;           // and of those the ones ranked by exact scores
constexpr int kNearThreads = 256;
constexpr int kNearAt = 8;                // labels that a warp scores at a time
constexpr int kExactThreads = 256;
constexpr int kExactChunk = 2048;
constexpr int kExactLabels = 4;         // labels of a warp at a time

// Doubles as whole numbers of the same order;
// 0 for scores that are never listed (-inf, NaN); -0 and 0 are the same score
__device__ __forceinline__ uint64_t ord64(double f) {
  if (!(f > -INFINITY)) return 0ull;
  const uint64_t u = (uint64_t)__double_as_longlong(f + 0.0);
  return (u >> 63) ? ~u : (u | (1ull << 63));
}
__device__ __forceinline__ double ord64_value(uint64_t k) {
  return __longlong_as_double((long long)((k >> 63) ? (k & ~(1ull << 63)) : ~k));
}

struct Counts { uint32_t wmax; int32_t nfail, nitems; };

struct Args {
  const uint16_t* X;
  const uint8_t *xa, *xb;                 // 8-bit heads: hi and lo codes [B][d]
  const void* W;
  int64_t L;
  int32_t d, B, G, k, nnz, fmt, segs;
  int32_t q, kbs, stages, kb3d;           // tiles and k-blocks of a stage; one TMA request for all of them
  int32_t nblk, nblkp, pairs;             // blocks of a stream, with padding; half tiles of a block
  int32_t streams;                        // kStreams; 0 where every label's score is kept: nblkp is their pitch
  float eps;                              // what an instruction may lose of the magnitudes it has summed
  float *xinv, *n1, *nw, *r1;
  int32_t *rflag, *fail;
  int32_t* done;                          // [B] segments of a failed query that are ranked
  Counts* counts;
  float* bmax;                            // [B][kStreams][nblkp] maxima of the accumulators over blocks, or [B][nblkp] of all
  int2* items;                            // (query, block) to be scored again, at most kMaxBlocks a query
  int32_t *listed, *nnear;                  // [B] whether the query's blocks are listed; labels found near
  float* near_v;                          // [B][kMaxNear] their fp32 scores
  int32_t* near_l;
  float* from;                            // [B] the fp32 score from which a label is near
  Stat* part;                             // [B][kStreams G] reference and sums in powers of two (Soft2)
  uint64_t* seg_key;                      // [B][segs][k]
  int32_t* seg_i;
  const int32_t *rowptr, *cols;
  float *logp, *lse, *entropy, *top_logp;
  int32_t* top_idx;
  double* rowstat;                        // [B][2] m and log s (for the exact path)
  int32_t* status;
};

// A tile's accumulators go to two groups of four epilogue warps, a half each;
// tiles of even and odd number have groups of their own.  Block i of stream
// 2 (tile & 1) + half is that half of the `pairs` tiles 2 (i pairs + r) +
// (tile & 1), and a range is a run of blocks of all streams.

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
  pdl_trigger();
  if (tid == 0) {
    if (b == 0) *A.counts = {0u, 0, 0};
    if (A.k > 0) A.done[b] = A.nnear[b] = 0;
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
    // 448 = 0.875 2^9; at most 2^126, so that 1 / s is a normal number
    s = ldexpf(1.0f, max(-126, min(126, f <= 0.875f ? 9 - e2 : 8 - e2)));
  }
  // 32 bytes of K an instruction: element k's hi is in instruction 4 ops (k / kKE) + k % kKE / (kKE / 4), its lo 4 later
  constexpr int kKE = kFp8 ? 128 : 64, kOps = kFp8 ? 2 : 1;
  const int steps = (A.d + kKE - 1) / kKE * 4 * kOps;
  float n = 0.0f, nw = 0.0f, r = 0.0f;
  for (int j = tid; j < A.d / 2; j += kPrepThreads) {
    const float from = (float)(steps - 2 * j / kKE * 4 * kOps - 2 * j % kKE / (kKE / 4));   // instructions from hi's own on
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
        nw = __fmaf_ru(fabsf(hi), from, __fmaf_ru(fabsf(lo), from - 4.0f, nw));
        r = __fadd_ru(r, fabsf(__fsub_rn(left, lo)));
        hi2 |= ch << (8 * h);
        lo2 |= cl << (8 * h);
      } else {
        n = __fadd_ru(n, fabsf(x));
        nw = __fmaf_ru(fabsf(x), from, nw);
      }
    }
    if (kFp8) {
      reinterpret_cast<uint16_t*>(xa + (size_t)b * A.d)[j] = (uint16_t)hi2;
      reinterpret_cast<uint16_t*>(xb + (size_t)b * A.d)[j] = (uint16_t)lo2;
    }
  }
  n = block_sum_up(n, red);
  nw = block_sum_up(nw, red);
  r = block_sum_up(r, red);
  if (tid == 0) {
    const float inv = 1.0f / s;                              // exact
    A.xinv[b] = inv;
    A.n1[b] = __fmul_ru(n, inv);
    A.nw[b] = __fmul_ru(nw, inv);
    A.r1[b] = __fmul_ru(r, inv);
    A.rflag[b] = bad ? 1 : 0;
  }
}

// ---------------------------------------------------------------- 2. score pass
struct SmemP {
  uint64_t full[kMaxStages], empty[kMaxStages], tfull[kMaxBufs], tempty[kMaxBufs];
  float win[8][32 * 4 * kStreams];
  uint32_t tmem_base;
  int abort;
};

__device__ __forceinline__ void record_timeout(int32_t* status, volatile int* abort, int site) {
  *abort = 1;
  if (atomicCAS(status, 0, (int)ELMO_ETIMEOUT) == 0) status[1] = site;
}

// Four MMAs along K, 32 bytes each (D += A B, the first D = A B unless `more`),
// A in tensor memory or in shared memory.  One thread issues them all; only the
// addresses move on between them, which is a little faster than a descriptor
// formed anew for each (300K labels x 1024: 276 to 268 us; x 768 unchanged).
#define ELMO_MMA4(KIND, A_OPERAND)                                                          \
  "tcgen05.mma.cta_group::1.kind::" KIND " [%0], " A_OPERAND("%1") ", %2, %3, p;\n\t"       \
  "tcgen05.mma.cta_group::1.kind::" KIND " [%0], " A_OPERAND("a1") ", b1, %3, q;\n\t"       \
  "tcgen05.mma.cta_group::1.kind::" KIND " [%0], " A_OPERAND("a2") ", b2, %3, q;\n\t"       \
  "tcgen05.mma.cta_group::1.kind::" KIND " [%0], " A_OPERAND("a3") ", b3, %3, q;\n\t}"
#define ELMO_MMA4_HEAD(A_BITS, A_STEP1, A_STEP2, A_STEP3)                                   \
  "{\n\t.reg .pred p, q;\n\t.reg .b64 b1, b2, b3;\n\t.reg .b" A_BITS " a1, a2, a3;\n\t"     \
  "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 q, 0, 0;\n\t"                                       \
  "add.u64 b1, %2, 2;\n\tadd.u64 b2, %2, 4;\n\tadd.u64 b3, %2, 6;\n\t"                      \
  "add.u" A_BITS " a1, %1, " A_STEP1 ";\n\tadd.u" A_BITS " a2, %1, " A_STEP2 ";\n\t"        \
  "add.u" A_BITS " a3, %1, " A_STEP3 ";\n\t"
#define ELMO_A_TMEM(R) "[" R "]"
#define ELMO_A_SMEM(R) R
template <int kFp8>
__device__ __forceinline__ void mma4_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t more) {
  if constexpr (kFp8)
    asm volatile(ELMO_MMA4_HEAD("32", "8", "16", "24") ELMO_MMA4("f8f6f4", ELMO_A_TMEM)
                 ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(more) : "memory");
  else
    asm volatile(ELMO_MMA4_HEAD("32", "8", "16", "24") ELMO_MMA4("f16", ELMO_A_TMEM)
                 ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(more) : "memory");
}
template <int kFp8>
__device__ __forceinline__ void mma4_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t more) {
  if constexpr (kFp8)
    asm volatile(ELMO_MMA4_HEAD("64", "2", "4", "6") ELMO_MMA4("f8f6f4", ELMO_A_SMEM)
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(more) : "memory");
  else
    asm volatile(ELMO_MMA4_HEAD("64", "2", "4", "6") ELMO_MMA4("f16", ELMO_A_SMEM)
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(more) : "memory");
}
#undef ELMO_MMA4
#undef ELMO_MMA4_HEAD
#undef ELMO_A_TMEM
#undef ELMO_A_SMEM

// The score of a label with a weight that is not finite, from its products with
// such weights alone: an infinity, or NaN.  In an E5M2 head the tensor cores'
// is no use: hi w + lo w of an infinite w is NaN wherever lo is zero or of the
// other sign.
__device__ __noinline__ float infinite_score(const uint16_t* x, const uint8_t* w, int d) {
  float z = 0.0f;
  for (int j = 0; j < d && z == z; j += 16) {
    const uint4 q = __ldg(reinterpret_cast<const uint4*>(w + j));
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if ((((u[i] & 0x7F7F7F7Fu) + 0x04040404u) & 0x80808080u) == 0) continue;    // magnitudes below 0x7C: all finite
      for (int e = 0; e < 4; ++e) {
        const uint32_t c = (u[i] >> (8 * e)) & 0xFFu;
        if ((c & 0x7Fu) >= 0x7Cu) z += bf16_to_f32(x[j + 4 * i + e]) * e5m2_to_f32((uint8_t)c);
      }
    }
  }
  return z == 0.0f ? NAN : z;
}

// kFp8: 8-bit head (kW5: E5M2 weights).  kXs = 0: d <= 768, X (two 8-bit or
// one bf16 operand, 2 d bytes a query) stays in the first TMEM columns, d / 2
// of the 512, and tiles are 64 labels; kXs = 1: wider heads, X comes through
// the ring with W, tiles are 128 labels.  The last columns hold four
// accumulators, two where X takes more than half: handing one over and back
// takes about 0.75 us, which two hide only behind a long tile (1M labels x
// 256, 105 queries: 87 us with two).
//
// A stage of the ring holds kbs 128-byte k-blocks of q tiles, up to 48 KB in
// one TMA request: the rate of the copies follows the number of requests (the
// 500K bf16 head streamed at 5.2 TB/s in 8 KB requests).
template <int kFp8, int kW5, int kXs>
__global__ void __launch_bounds__(kThreads, 1)
    label_score_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA,
                       const __grid_constant__ CUtensorMap tmB, const Args A) {
  constexpr int kN = kXs ? 128 : 64;
  constexpr int kOps = kFp8 ? 2 : 1;
  constexpr int kKE = kFp8 ? 128 : 64;                 // elements of a 128-byte k-block
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t slab = (uint32_t)A.q * kN * 128;      // a k-block of the stage's labels
  const uint32_t wbytes = slab * (uint32_t)A.kbs;
  const uint32_t stage = wbytes + (kXs ? (uint32_t)A.kbs * 16384u * kOps : 0u);
  SmemP* S = reinterpret_cast<SmemP*>(ring + (size_t)A.stages * stage);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int P = (A.B + 127) / 128;
  const int p = blockIdx.x % P, g = blockIdx.x / P;
  const int64_t T = (A.L + kN - 1) / kN;
  const int64_t nrange = (T + 2 * A.pairs - 1) / (2 * A.pairs);
  const int64_t blk0 = nrange * g / A.G, blk1 = nrange * (g + 1) / A.G;
  const int64_t t0 = 2 * blk0 * A.pairs, t1 = min(T, 2 * blk1 * A.pairs);
  const int nkb = (A.d + kKE - 1) / kKE;
  const int nst = (nkb + A.kbs - 1) / A.kbs;           // stages of a group of q tiles (1 where q > 1)
  const uint32_t opcols = (uint32_t)nkb * 32;
  const uint32_t nbuf = kXs || kOps * opcols <= 256 ? 4 : 2, acc0 = 512 - nbuf * kN;   // the accumulators' first column
  const uint32_t bufs = nbuf - 1, bufs_log = nbuf >> 1;                               // rel & bufs, rel >> bufs_log
  volatile int* abort = &S->abort;
  const bool scan = A.k > 0;                           // the ranges are scanned for max|W|

  if (threadIdx.x == 0) {
    for (int s = 0; s < A.stages; ++s) { mbar_init(&S->full[s], 1); mbar_init(&S->empty[s], scan ? 3 : 1); }
    for (int i = 0; i < kMaxBufs; ++i) { mbar_init(&S->tfull[i], 1); mbar_init(&S->tempty[i], 8); }
    S->abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) { tmem_alloc(&S->tmem_base, 512); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S->tmem_base;
  pdl_trigger();
  // W is no other kernel's here: its copies start while the operands are still
  // being formed, everything else waits for them
  if (warp != 0 || kXs) pdl_wait();

  if (!kXs) {
    if (warp >= 2 && warp < kEpi) {                    // query r of the panel into lane r, 32 columns at a time
      const int quad = warp & 3, row = p * 128 + quad * 32 + lane;
      const size_t rowbytes = (size_t)A.d * (kFp8 ? 1 : 2);
      // two pieces' loads in flight: one piece at a time kept the first MMA waiting for 10 us
#pragma unroll 2
      for (uint32_t piece = (warp - 2) >> 2; piece < (uint32_t)kOps * nkb; piece += kStreams) {
        const uint32_t op = piece / nkb, c0 = piece % nkb * 32;
        const uint8_t* src = (kFp8 ? (op ? A.xb : A.xa) : reinterpret_cast<const uint8_t*>(A.X)) + (size_t)row * rowbytes;
        uint32_t v[32];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const size_t off = (size_t)(c0 + 4 * u) * 4;
          uint4 w4 = make_uint4(0u, 0u, 0u, 0u);
          if (row < A.B && off < rowbytes) w4 = *reinterpret_cast<const uint4*>(src + off);
          v[4 * u] = w4.x; v[4 * u + 1] = w4.y; v[4 * u + 2] = w4.z; v[4 * u + 3] = w4.w;
        }
        tmem_st32(tmem + ((uint32_t)(quad * 32) << 16) + op * opcols + c0, v);
      }
      tmem_wait_st();
    }
    tc_fence_before();
    // the TMA warp does not come here: the others' barrier
    if (warp != 0) asm volatile("bar.sync 1, %0;" ::"n"(kThreads - 32) : "memory");
    tc_fence_after();
  }

  if (warp == 0) {
    if (elect_one()) {
      tma_prefetch_desc(&tmW);
      uint32_t s = 0, ph = 1;
      for (int64_t t = t0; t < t1 && !*abort; t += A.q) {
        for (int st = 0; st < nst; ++st) {
          if (!mbar_wait(&S->empty[s], ph, abort, kWait)) { record_timeout(A.status, abort, 71); break; }
          uint8_t* at = ring + (size_t)s * stage;
          uint64_t* bar = &S->full[s];
          const int kb0 = st * A.kbs;
          mbar_arrive_expect_tx(bar, stage);
          if (A.kb3d) {
            tma_load_3d(at, &tmW, bar, 0, (int32_t)(t * kN), kb0);
            if (kXs) {
              tma_load_3d(at + wbytes, &tmA, bar, 0, p * 128, kb0);
              if (kFp8) tma_load_3d(at + wbytes + A.kbs * 16384, &tmB, bar, 0, p * 128, kb0);
            }
          } else {
            for (int j = 0; j < A.kbs; ++j) {
              tma_load_2d(at + j * slab, &tmW, bar, (kb0 + j) * kKE, (int32_t)(t * kN));
              if (kXs) {
                tma_load_2d(at + wbytes + j * 16384, &tmA, bar, (kb0 + j) * kKE, p * 128);
                if (kFp8) tma_load_2d(at + wbytes + (A.kbs + j) * 16384, &tmB, bar, (kb0 + j) * kKE, p * 128);
              }
            }
          }
          if (++s == (uint32_t)A.stages) { s = 0; ph ^= 1; }
        }
      }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      // hi is E4M3 (format 0) and lo E5M2 (1); bf16 operands are format 1 of their kind
      const uint32_t idesc[2] = {kFp8 ? make_idesc(0, kW5, 0, 0, 128, kN) : make_idesc(1, 1, 0, 0, 128, kN),
                                 make_idesc(1, kW5, 0, 0, 128, kN)};
      uint32_t s = 0, ph = 0;
      bool ok = true;
      for (int64_t t = t0; t < t1 && ok && !*abort; t += A.q) {
        for (int st = 0; st < nst && ok; ++st) {
          if (!mbar_wait(&S->full[s], ph, abort, kWait)) { record_timeout(A.status, abort, 73); ok = false; break; }
          tc_fence_after();
          // descriptors advance by their start addresses, in units of 16 bytes
          const uint64_t wd = sw128_desc(smem_u32(ring + (size_t)s * stage), 16, 1024), xd = wd + (wbytes >> 4);
          for (int j = 0; j < A.q && t + j < t1; ++j) {
            const uint32_t rel = (uint32_t)(t + j - t0), buf = rel & bufs;
            if (st == 0) {
              if (!mbar_wait(&S->tempty[buf], ((rel >> bufs_log) & 1) ^ 1, abort, kWait)) {
                record_timeout(A.status, abort, 72);
                ok = false;
                break;
              }
              tc_fence_after();
            }
            const uint32_t dcol = tmem + acc0 + buf * kN;
            for (int i = 0; i < A.kbs && st * A.kbs + i < nkb; ++i) {
              const int kb = st * A.kbs + i;
              const uint64_t bd = wd + (((uint32_t)i * slab + (uint32_t)j * (kN * 128)) >> 4);
#pragma unroll
              for (int op = 0; op < kOps; ++op) {      // four instructions of 32 bytes of K
                const uint32_t more = (kb | op) != 0;
                if (kXs) mma4_ss<kFp8>(dcol, xd + (uint32_t)(op * A.kbs + i) * (16384 >> 4), bd, idesc[op], more);
                else mma4_ts<kFp8>(dcol, tmem + (uint32_t)op * opcols + (uint32_t)kb * 32, bd, idesc[op], more);
              }
            }
            if (st == nst - 1) mma_commit(&S->tfull[buf]);
          }
          if (!ok) break;
          mma_commit(&S->empty[s]);
          if (++s == (uint32_t)A.stages) { s = 0; ph ^= 1; }
        }
      }
    }
  } else if (warp < kEpi) {
    // The score of a query and label costs some 7 issue slots and one
    // exponential, and a warp on its own starts an instruction every 6 cycles:
    // four warps a scheduler bring the epilogue below the other bounds (two
    // took 93 us for 1M labels x 256 and 105 queries).
    const int stream = (warp - 2) >> 2, par = stream >> 1, half = stream & 1;   // t0 is even
    const int quad = warp & 3, r = quad * 32 + lane, row = p * 128 + r;
    const bool live = row < A.B;
    const float inv = live ? A.xinv[row] : 1.0f;       // scores are inv times the accumulators
    const bool finite = kW5 && live && A.rflag[row] == 0;
    Soft2 soft(inv);
    const bool keep = A.k > 0 && A.streams == 0, lists = A.k > 0 && !keep && live;
    float* bm = A.bmax + (keep ? (size_t)row : (size_t)row * kStreams + stream) * A.nblkp;
    // maxima of the aligned eight blocks under way, a column of shared memory a thread
    float* win = S->win[0] + (warp - 2) * 32 + lane;
    const int L = (int)A.L, last = (int)t1;
    uint32_t rel = par;
    bool ok = true;
    int tile = (int)t0 + par;
    for (int blk = (int)blk0; blk < (int)blk1 && ok; ++blk) {
      float best = -INFINITY;
      for (int i = 0; i < A.pairs && tile < last; ++i, tile += 2, rel += 2) {
        const uint32_t buf = rel & bufs;
        if (!mbar_wait(&S->tfull[buf], (rel >> bufs_log) & 1, abort, kWait)) {
          record_timeout(A.status, abort, 74);
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll 1
        for (int u = 0; u < kN / 64; ++u) {
          __syncwarp();
          uint32_t raw[32];
          tmem_ld32(tmem + ((uint32_t)(quad * 32) << 16) + acc0 + buf * kN + half * (kN / 2) + u * 32, raw);
          tmem_wait_ld();
          if (u == kN / 64 - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S->tempty[buf]);
          }
          const int l0 = tile * kN + half * (kN / 2) + u * 32;
          if (!live || l0 >= L) continue;
          float v[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) v[c] = __uint_as_float(raw[c]);
          if (l0 + 32 > L) {                           // past the end there are no labels
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (l0 + c >= L) v[c] = -INFINITY;
          }
          const float mx = max32(v);
          best = fmaxf(best, mx);
          soft.add32(v, mx, [&](float (&bad)[32]) {
            if constexpr (kW5) {
              if (!finite) return false;
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (bad[c] != bad[c])
                  bad[c] = infinite_score(A.X + (size_t)row * A.d, static_cast<const uint8_t*>(A.W) + (size_t)(l0 + c) * A.d, A.d);
              return true;
            }
            return false;
          });
          if (keep) {
#pragma unroll
            for (int c = 0; c < 32; c += 4)
              if (l0 + c < A.nblkp) *reinterpret_cast<float4*>(bm + l0 + c) = make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]);
          }
        }
      }
      if (lists) {
        const int j = blk & 7;
        win[j * 32 * 4 * kStreams] = best;
        if (j == 7 || blk + 1 == (int)blk1) {
          const bool end = blk + 1 == A.nblk;          // of the row: the padding holds nothing
          const int first = blk - j;
          float w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = e <= j ? win[e * 32 * 4 * kStreams] : -INFINITY;
          if (first >= (int)blk0 && (j == 7 || end)) {
            reinterpret_cast<float4*>(bm + first)[0] = make_float4(w[0], w[1], w[2], w[3]);
            reinterpret_cast<float4*>(bm + first)[1] = make_float4(w[4], w[5], w[6], w[7]);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if ((e <= j || end) && first + e >= (int)blk0) bm[first + e] = w[e];
          }
        }
      }
    }
    if (live)
      A.part[((size_t)row * A.G + g) * kStreams + stream] = {soft.m > -INFINITY ? soft.r : -INFINITY, soft.s, soft.t};
  } else if (scan) {
    // bf16 magnitudes by 16-bit maxima, two instructions for two weights.  Of
    // 8-bit magnitudes x, x + (0x7F - m) carries into the sign bit exactly
    // where x exceeds the largest so far, m: two and a half for four, and m
    // seldom moves.  Panels of one range take its stages in turn.
    const int id = (warp - kEpi) * 32 + lane;
    uint32_t mx = 0, s = 0, ph = 0, turn = 0;
    bool ok = true;
    for (int64_t t = t0; t < t1 && ok && !*abort; t += A.q) {
      for (int st = 0; st < nst; ++st) {
        if (!mbar_wait(&S->full[s], ph, abort, kWait)) { record_timeout(A.status, abort, 75); ok = false; break; }
        if (turn == (uint32_t)p) {
          const uint4* w = reinterpret_cast<const uint4*>(ring + (size_t)s * stage);
          for (uint32_t i = id; i < wbytes / 16; i += 64 * 8) {      // stages are multiples of 8 KB
            uint4 v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = w[i + 64 * e];
            if constexpr (!kFp8) {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                mx = __vmaxu2(__vmaxu2(__vmaxu2(mx, v[e].x & 0x7FFF7FFFu), __vmaxu2(v[e].y & 0x7FFF7FFFu, v[e].z & 0x7FFF7FFFu)),
                              v[e].w & 0x7FFF7FFFu);
            } else {
              const uint32_t add = 0x7F7F7F7Fu - mx * 0x01010101u;
              uint32_t any = 0;
#pragma unroll
              for (int e = 0; e < 8; ++e)
                any |= ((v[e].x & 0x7F7F7F7Fu) + add) | ((v[e].y & 0x7F7F7F7Fu) + add) | ((v[e].z & 0x7F7F7F7Fu) + add) |
                       ((v[e].w & 0x7F7F7F7Fu) + add);
              if (__any_sync(0xFFFFFFFFu, any & 0x80808080u)) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const uint32_t x[4] = {v[e].x, v[e].y, v[e].z, v[e].w};
#pragma unroll
                  for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int h = 0; h < 32; h += 8) mx = max(mx, (x[c] >> h) & 0x7Fu);
                }
                mx = __reduce_max_sync(0xFFFFFFFFu, mx);
              }
            }
          }
        }
        if (++turn == (uint32_t)P) turn = 0;
        __syncwarp();
        if (lane == 0) mbar_arrive(&S->empty[s]);
        if (++s == (uint32_t)A.stages) { s = 0; ph ^= 1; }
      }
    }
    if (!kFp8) mx = __reduce_max_sync(0xFFFFFFFFu, max(mx & 0xFFFFu, mx >> 16));
    if (lane == 0 && mx) atomicMax(&A.counts->wmax, mx);
  }
  __syncthreads();
  if (*abort) __nanosleep(20000);                      // copies in flight land before the memory is given up
  if (warp == 1) { tc_fence_after(); tmem_dealloc(tmem, 512); }
}

// ---------------------------------------------------------------- exact scores
// Eight weights of a label from element 8 c on, as they are stored: a loop's
// loads all start before the first is used.
template <int kFormat>
__device__ __forceinline__ Raw8<kFormat> load8(const void* W, int64_t l, int d, int c) {
  Raw8<kFormat> r;
  if constexpr (kFormat == ELMO_BF16) r.v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(W) + l * d) + c);
  else r.v = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(W) + l * d) + c);
  return r;
}
// x . w_l with exact products and sums in 64 bits, by one warp, in an order
// that depends on d alone: equal rows have equal scores.
template <int kFormat>
__device__ __forceinline__ double exact_score(const float* xs, const void* W, int64_t l, int d, int lane) {
  double acc = 0.0;
#pragma unroll 4
  for (int c = lane; c < d / 8; c += 32) {
    float f[8];
    values8<kFormat>(load8<kFormat>(W, l, d, c), f);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc = fma((double)xs[8 * c + e], (double)f[e], acc);
  }
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xFFFFFFFFu, acc, o);
  return acc;
}

// The same for kM labels from l on, whose loads are in flight together; each sum
// in exact_score's order.  Labels beyond `end` are read as `end`.
template <int kFormat, int kM>
__device__ __forceinline__ void exact_scores(const float* xs, const void* W, int64_t l, int64_t end, int d, int lane,
                                             double (&acc)[kM]) {
#pragma unroll
  for (int m = 0; m < kM; ++m) acc[m] = 0.0;
  // two steps: one spills at 64 registers (500K bf16 labels tied, 4 queries: 1350 us against 865)
#pragma unroll 2
  for (int c = lane; c < d / 8; c += 32) {
    Raw8<kFormat> r[kM];
#pragma unroll
    for (int m = 0; m < kM; ++m) r[m] = load8<kFormat>(W, min(l + m, end), d, c);
    double x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (double)xs[8 * c + e];
#pragma unroll
    for (int m = 0; m < kM; ++m) {
      float f[8];
      values8<kFormat>(r[m], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[m] = fma(x[e], (double)f[e], acc[m]);
    }
  }
#pragma unroll
  for (int m = 0; m < kM; ++m)
    for (int o = 16; o > 0; o >>= 1) acc[m] += __shfl_xor_sync(0xFFFFFFFFu, acc[m], o);
}

// The same in fp32 for kM labels at a time.
template <int kFormat, int kM>
__device__ __forceinline__ void near_scores(const uint16_t* X, const void* W, const int64_t (&l)[kM], int d, int lane,
                                            float (&acc)[kM]) {
#pragma unroll
  for (int m = 0; m < kM; ++m) acc[m] = 0.0f;
#pragma unroll 3
  for (int c = lane; c < d / 8; c += 32) {
    Raw8<kFormat> r[kM];
#pragma unroll
    for (int m = 0; m < kM; ++m) r[m] = load8<kFormat>(W, l[m], d, c);
    float x[8];
    values8<ELMO_BF16>(load8<ELMO_BF16>(X, 0, d, c), x);
#pragma unroll
    for (int m = 0; m < kM; ++m) {
      float f[8];
      values8<kFormat>(r[m], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[m] = fmaf(x[e], f[e], acc[m]);
    }
  }
#pragma unroll
  for (int m = 0; m < kM; ++m)
    for (int o = 16; o > 0; o >>= 1) acc[m] += __shfl_xor_sync(0xFFFFFFFFu, acc[m], o);
}

__device__ __forceinline__ float max_weight(uint32_t code, int fmt) {
  if (fmt == ELMO_BF16) return code >= 0x7F80u ? NAN : bf16_to_f32((uint16_t)code);
  if (fmt == ELMO_FP8_E5M2) return code >= 0x7Cu ? NAN : e5m2_to_f32((uint8_t)code);
  return code >= 0x7Fu ? NAN : e4m3_to_f32((uint8_t)code);
}

// ---------------------------------------------------------------- 3. join
struct SmemB {
  alignas(16) float gbest[kGroups];
  float low;
};

// low = a lower bound on the k-th best of values of which each thread has seen
// the best of its own: the k-th best of the groups of kPer neighbouring
// threads (-inf where fewer groups hold a value).
template <int kThr>
__device__ __forceinline__ float lower_bound_kth(SmemB* S, float best, int k) {
  constexpr int kPer = kThr / kGroups;
  const int tid = threadIdx.x;
  for (int o = 1; o < kPer; o <<= 1) best = fmaxf(best, __shfl_xor_sync(0xFFFFFFFFu, best, o));
  __syncthreads();
  if (tid % kPer == 0) S->gbest[tid / kPer] = best;
  if (tid == 0) S->low = -INFINITY;
  __syncthreads();
  if (tid < kGroups) {
    const float mine = S->gbest[tid];
    int above = 0, same = 0;
    for (int j = 0; j < kGroups; j += 4) {
      const float4 o = *reinterpret_cast<const float4*>(S->gbest + j);
      above += (o.x > mine) + (o.y > mine) + (o.z > mine) + (o.w > mine);
      same += (o.x == mine) + (o.y == mine) + (o.z == mine) + (o.w == mine);
    }
    if (above < k && above + same >= k) S->low = mine;
  }
  __syncthreads();
  return S->low;
}

// The error bounds of a query's scores, rounded up; 2^-126 for subnormal partial
// sums: `tensor` of the tensor cores', `near` of the fp32 ones.  Infinite where
// the weights are not finite or a sum may leave fp32's range on its way (to an
// infinity or a NaN that no bound holds for).
struct Deltas { float tensor, near; };
__device__ __forceinline__ Deltas deltas_of(const Args& A, int b) {
  const float r = A.r1[b], n = __fadd_ru(A.n1[b], r), w = max_weight(A.counts->wmax, A.fmt);
  const float all = __fmul_ru(n, w);
  if (!(all < 0x1p126f)) return {INFINITY, INFINITY};
  const float chain = (float)((A.d + 255) / 256 * 8 + 6) * 0x1p-24f;     // an addition more for what the others' rounding adds
  return {__fadd_ru(__fmul_ru(__fmaf_ru(A.eps, A.nw[b], r), w), 0x1p-126f), __fadd_ru(__fmul_ru(chain, all), 0x1p-126f)};
}

// Ranks a query's `near` labels near the k-th best by exact scores, or lists the
// query for the exact path; their scores in near_v are off by `delta` at most.
// The whole CTA.
struct SmemR {
  double ex[kMaxExact];
  int32_t el[kMaxExact];
  int nexact;
};

template <int kFormat, int kThr>
__device__ __forceinline__ void rank_near(const Args& A, int b, const float* xs, int near, float delta, double m, double logs,
                                          SmemB* S, SmemR* R) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  bool ok = near >= A.k && near <= kMaxNear;
  const float* nv = A.near_v + (size_t)b * kMaxNear;
  if (tid == 0) R->nexact = 0;
  if (ok) {
    float best = -INFINITY;
    for (int i = tid; i < near; i += kThr) best = fmaxf(best, nv[i]);
    const float cut = __fsub_rd(lower_bound_kth<kThr>(S, best, A.k), __fmul_ru(2.0f, delta));
    for (int i = tid; i < near; i += kThr) {
      if (nv[i] >= cut) {
        const int at = atomicAdd(&R->nexact, 1);
        if (at < kMaxExact) R->el[at] = A.near_l[(size_t)b * kMaxNear + i];
      }
    }
    __syncthreads();
    ok = R->nexact <= kMaxExact;
  }
  if (!ok) {
    if (tid == 0) A.fail[atomicAdd(&A.counts->nfail, 1)] = b;
    return;
  }
  const int n = R->nexact;
  for (int i = warp; i < n; i += kThr / 32) {
    const double z = exact_score<kFormat>(xs, A.W, R->el[i], A.d, lane);
    if (lane == 0) R->ex[i] = z;
  }
  __syncthreads();
  for (int i = tid; i < n; i += kThr) {
    const double z = R->ex[i];
    const int32_t l = R->el[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += R->ex[j] > z || (R->ex[j] == z && R->el[j] < l);
    if (rank < A.k) {
      A.top_idx[(size_t)b * A.k + rank] = l;
      A.top_logp[(size_t)b * A.k + rank] = (float)(z - m - logs);
    }
  }
}

// A query as fp32 numbers in shared memory.
template <int kThr>
__device__ __forceinline__ void load_query(const Args& A, int b, float* xs) {
  for (int j = threadIdx.x; j < A.d / 2; j += kThr) {
    const uint32_t w = reinterpret_cast<const uint32_t*>(A.X + (size_t)b * A.d)[j];
    xs[2 * j] = __uint_as_float(w << 16);
    xs[2 * j + 1] = __uint_as_float(w & 0xFFFF0000u);
  }
}

// Statistics of a query, log p of its given labels, and the blocks that may
// hold its k best labels.
template <int kFormat>
__global__ void __launch_bounds__(kJoinThreads) label_join_kernel(const Args A) {
  extern __shared__ __align__(16) uint8_t dyn[];
  float* xs = reinterpret_cast<float*>(dyn);           // [d] the query
  __shared__ SmemB S;
  __shared__ union { SmemR rank; int32_t blocks[kMaxBlocks]; } U;   // one or the other
  constexpr int kW = kJoinThreads / 32;
  constexpr int kEarly = 512;
  __shared__ double stat[2], ws[kW], wt[kW], early[kEarly];
  __shared__ float wm[kW];
  __shared__ int nblocks, at0;
  const int b = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  load_query<kJoinThreads>(A, b, xs);
  if (tid == 0) nblocks = 0;
  __syncthreads();
  // the given labels' scores need only X and W: the first kEarly of them while
  // the score pass still runs elsewhere
  const int e0 = min(max(A.rowptr[b], 0), A.nnz), e1 = min(A.rowptr[b + 1], A.nnz), ee = min(e1, e0 + kEarly);
  auto given = [&](int e) {
    const int64_t l = A.cols[e];
    return l >= 0 && l < A.L ? exact_score<kFormat>(xs, A.W, l, A.d, lane) : 0.0;
  };
  for (int e = e0 + warp; e < ee; e += kW) {
    const double z = given(e);
    if (lane == 0) early[e - e0] = z;
  }
  pdl_wait();
  pdl_trigger();
  const bool bad = A.rflag[b] != 0;
  {
    // at most two partial sums of a thread: kStreams G, G at most the SMs
    const int n = kStreams * A.G;
    const Stat* part = A.part + (size_t)b * n;
    Stat q[2];
    float mf = -INFINITY;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      q[i] = tid + i * kJoinThreads < n ? part[tid + i * kJoinThreads] : Stat{-INFINITY, 0.0f, 0.0f};
      mf = fmaxf(mf, q[i].m);
    }
    for (int o = 16; o > 0; o >>= 1) mf = fmaxf(mf, __shfl_xor_sync(0xFFFFFFFFu, mf, o));
    if (lane == 0) wm[warp] = mf;
    __syncthreads();
    for (int w = 0; w < kW; ++w) mf = fmaxf(mf, wm[w]);
    double s = 0.0, t = 0.0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (q[i].m == -INFINITY) { s += q[i].s; continue; }
      const double d = (double)q[i].m - (double)mf, c = q[i].m == mf ? 1.0 : exp2(d);
      s += c * q[i].s;
      t += c * (q[i].t + (q[i].m == mf ? 0.0 : d * q[i].s));
    }
    for (int o = 16; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
      t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    }
    if (lane == 0) { ws[warp] = s; wt[warp] = t; }
    __syncthreads();
    if (tid == 0) {
      s = t = 0.0;
      for (int w = 0; w < kW; ++w) { s += ws[w]; t += wt[w]; }
      constexpr double kLn2 = 0.693147180559945309417;
      double m = mf * kLn2, logs = log(s), lse = m + logs, H = logs - t / s * kLn2;
      if (mf == -INFINITY) {                           // no label has a finite score
        lse = s == 0.0 ? -INFINITY : NAN;
        H = s == 0.0 ? 0.0 : NAN;
        m = lse;
        logs = 0.0;
      } else if (mf == INFINITY) {                     // s counts the infinities, a NaN makes it NaN
        lse = m = isnan(s) ? NAN : m;
        H = NAN;
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
  __syncthreads();
  const double m = stat[0], logs = stat[1];

  if (A.k > 0) {
    const Deltas delta = deltas_of(A, b);
    const float two = __fmul_ru(2.0f, delta.tensor), inv = A.xinv[b];
    if (bad || (A.n1[b] == 0.0f && A.r1[b] == 0.0f && two < INFINITY)) {
      // no list, or that of a query of zeros (as padding is): every label's score is 0
      if (tid == 0) A.listed[b] = 0;
      for (int i = tid; i < A.k; i += kJoinThreads) {
        A.top_idx[(size_t)b * A.k + i] = bad ? -1 : i;
        A.top_logp[(size_t)b * A.k + i] = bad ? -INFINITY : (float)(0.0 - m - logs);
      }
    } else {
      bool ok = two < INFINITY;                        // not so for weights that are not finite, or sums that overflow
      // n maxima, -inf in the padding between streams; or all the labels' scores
      const bool keep = A.streams == 0;
      const float* bm = A.bmax + (size_t)b * (keep ? 1 : kStreams) * A.nblkp;
      const int n = keep ? (int)A.L : kStreams * A.nblkp;
      auto each = [&](auto f) {
        if (n <= kGroups) {                            // one to a group
          if (tid % (kJoinThreads / kGroups) == 0 && tid / (kJoinThreads / kGroups) < n) {
            const int i = tid / (kJoinThreads / kGroups);
            f(i, __ldcg(bm + i));
          }
        } else if (n <= 4 * kJoinThreads) {
          float v[4];
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (tid + u * kJoinThreads < n) v[u] = __ldcg(bm + tid + u * kJoinThreads);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int i = tid + u * kJoinThreads;
            if (i < n) f(i, v[u]);
          }
        } else {
          const int n4 = (n + 3) / 4;
          for (int i0 = tid; i0 < n4; i0 += 8 * kJoinThreads) {
            float4 v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
              if (i0 + u * kJoinThreads < n4) v[u] = __ldcg(reinterpret_cast<const float4*>(bm) + i0 + u * kJoinThreads);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const int i = 4 * (i0 + u * kJoinThreads);
              const float w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (i + e < n) f(i + e, w[e]);
            }
          }
        }
      };
      float best = -INFINITY;
      if (ok) each([&](int, float v) { best = fmaxf(best, v); });
      const float low = lower_bound_kth<kJoinThreads>(&S, best, A.k);
      const float from = __fsub_rd(low, __fdiv_ru(two, inv));
      if (ok && best >= from)                          // a thread that has seen none has none to list
        each([&](int i, float v) {
          if (v >= from && v > -INFINITY) {
            const int at = atomicAdd(&nblocks, 1);
            if (keep) {
              if (at < kMaxNear) {
                A.near_v[(size_t)b * kMaxNear + at] = __fmul_rn(v, inv);
                A.near_l[(size_t)b * kMaxNear + at] = i;
              }
            } else if (at < kMaxBlocks) {
              U.blocks[at] = i;
            }
          }
        });
      __syncthreads();
      const int found = nblocks;
      ok = ok && found > 0 && found <= (keep ? kMaxNear : kMaxBlocks);
      if (tid == 0) {
        A.listed[b] = ok;
        if (!ok) {
          A.fail[atomicAdd(&A.counts->nfail, 1)] = b;
        } else if (!keep) {
          at0 = atomicAdd(&A.counts->nitems, found);
          A.from[b] = __fsub_rd(__fmul_rd(low, inv), __fadd_ru(delta.tensor, delta.near));
        }
      }
      __syncthreads();
      if (ok && keep) rank_near<kFormat, kJoinThreads>(A, b, xs, found, delta.tensor, m, logs, &S, &U.rank);
      else if (ok)
        for (int i = tid; i < found; i += kJoinThreads) A.items[at0 + i] = make_int2(b, U.blocks[i]);
    }
  }

  auto put = [&](int e, double z) {
    const int32_t l = A.cols[e];
    float r = (float)(z - m - logs);
    if (l < 0 || l >= A.L) {
      r = NAN;
      if (atomicCAS(A.status, 0, (int)ELMO_EDATA) == 0) A.status[1] = e;
    } else if (z == -INFINITY && !isnan(m + logs)) {
      r = -INFINITY;                                   // a masked label
    }
    A.logp[e] = r;
  };
  for (int e = e0 + tid; e < ee; e += kJoinThreads) put(e, early[e - e0]);
  for (int e = e0 + kEarly + warp; e < e1; e += kW) {
    const double z = given(e);
    if (lane == 0) put(e, z);
  }
}

// The labels of the listed blocks again, in fp32, kNearAt of a block to a
// warp.  Bound by the read of the blocks where there are many (256 queries'
// 64 best among 3M 8-bit labels: 0.9 GB), by latency else: every load of a
// step starts before the first is used, and the query comes from L1.
template <int kFormat>
__global__ void __launch_bounds__(kNearThreads, 2) label_near_kernel(const Args A, int tile) {
  const int lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  const int block = tile / 2, per = A.pairs * block / kNearAt;     // labels of half a tile; warps' shares of a block
  const int64_t work = (int64_t)A.counts->nitems * per;
  for (int64_t w = (int64_t)blockIdx.x * (kNearThreads / 32) + (threadIdx.x >> 5); w < work;
       w += (int64_t)gridDim.x * (kNearThreads / 32)) {
    const int2 it = A.items[w / per];
    const int b = it.x, in = (int)(w % per) * kNearAt;
    const int stream = it.y / A.nblkp;
    const int64_t pair0 = (int64_t)(it.y % A.nblkp) * A.pairs;
    const int64_t l0 = (2 * (pair0 + in / block) + (stream >> 1)) * tile + (stream & 1) * block + in % block;
    if (l0 >= A.L) continue;
    int64_t l[kNearAt];
    float z[kNearAt];
#pragma unroll
    for (int c = 0; c < kNearAt; ++c) l[c] = min(l0 + c, A.L - 1);
    near_scores<kFormat, kNearAt>(A.X + (size_t)b * A.d, A.W, l, A.d, lane, z);
    float mine = z[0];
#pragma unroll
    for (int c = 1; c < kNearAt; ++c) mine = lane == c ? z[c] : mine;
    if (lane < kNearAt && l0 + lane < A.L && mine >= A.from[b]) {
      const int at = atomicAdd(A.nnear + b, 1);
      if (at < kMaxNear) {
        A.near_v[(size_t)b * kMaxNear + at] = mine;
        A.near_l[(size_t)b * kMaxNear + at] = (int32_t)(l0 + lane);
      }
    }
  }
}

// A query's k best of the labels near the k-th best, by exact scores.
template <int kFormat>
__global__ void __launch_bounds__(kNearThreads) label_rank_kernel(const Args A) {
  extern __shared__ __align__(16) uint8_t dyn[];
  float* xs = reinterpret_cast<float*>(dyn);           // [d]
  __shared__ SmemB S;
  __shared__ SmemR R;
  const int b = blockIdx.x;
  load_query<kNearThreads>(A, b, xs);
  pdl_wait();
  pdl_trigger();
  if (A.listed[b] == 0) return;                        // answered, or a failed query already
  rank_near<kFormat, kNearThreads>(A, b, xs, A.nnear[b], deltas_of(A, b).near, A.rowstat[2 * b], A.rowstat[2 * b + 1],
                                   &S, &R);
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

// Work item (failed query, segment): the segment's k best labels; the CTA that
// does a query's last segment joins them.
template <int kFormat>
__global__ void __launch_bounds__(kExactThreads) label_exact_kernel(const Args A) {
  extern __shared__ __align__(16) uint8_t dyn[];
  float* xs = reinterpret_cast<float*>(dyn);
  __shared__ uint64_t key[kExactChunk + ELMO_MAX_TOPK];
  __shared__ uint64_t lk[ELMO_MAX_TOPK];
  __shared__ int32_t li[ELMO_MAX_TOPK];
  __shared__ int32_t old[ELMO_MAX_TOPK];
  __shared__ uint64_t rk[kExactThreads / 32];
  __shared__ int32_t ri[kExactThreads / 32];
  __shared__ int last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  const int nf = A.counts->nfail;
  for (int64_t item = blockIdx.x; item < (int64_t)nf * A.segs; item += gridDim.x) {
    const int r = (int)(item / A.segs), seg = (int)(item % A.segs);
    const int b = A.fail[r];
    const int64_t l0 = A.L * seg / A.segs, l1 = A.L * (seg + 1) / A.segs;
    __syncthreads();
    for (int j = tid; j < A.d; j += kExactThreads) xs[j] = bf16_to_f32(A.X[(size_t)b * A.d + j]);
    if (tid < A.k) { lk[tid] = 0; li[tid] = 0x7FFFFFFF; }
    __syncthreads();
    for (int64_t a = l0; a < l1; a += kExactChunk) {
      const int n = (int)min((int64_t)kExactChunk, l1 - a);
      for (int i = warp * kExactLabels; i < n; i += kExactThreads / 32 * kExactLabels) {
        double z[kExactLabels];
        exact_scores<kFormat, kExactLabels>(xs, A.W, a + i, l1 - 1, A.d, lane, z);
#pragma unroll
        for (int m = 0; m < kExactLabels; ++m)
          if (lane == m && i + m < n) key[i + m] = ord64(z[m]);
      }
      if (tid < A.k) { key[kExactChunk + tid] = lk[tid]; old[tid] = li[tid]; }
      __syncthreads();
      int enters = 0;                                  // of labels that all tie only the first chunk's do
      for (int i = tid; i < n; i += kExactThreads)
        enters |= key[i] != 0 && ranks_before(key[i], (int32_t)(a + i), lk[A.k - 1], li[A.k - 1]);
      if (!__syncthreads_or(enters)) continue;
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
    uint64_t* sk = A.seg_key + (size_t)r * A.segs * A.k;
    int32_t* si = A.seg_i + (size_t)r * A.segs * A.k;
    if (tid < A.k) {
      __stcg(reinterpret_cast<unsigned long long*>(sk) + seg * A.k + tid, (unsigned long long)lk[tid]);
      __stcg(si + seg * A.k + tid, li[tid]);
    }
    __threadfence();
    __syncthreads();
    if (tid == 0) last = atomicAdd(A.done + r, 1) == A.segs - 1;
    __syncthreads();
    if (!last) continue;
    __threadfence();
    const double m = A.rowstat[2 * b], logs = A.rowstat[2 * b + 1];
    auto at = [&](int i, uint64_t& k, int32_t& l) {
      k = __ldcg(reinterpret_cast<const unsigned long long*>(sk) + i);
      l = __ldcg(si + i);
    };
    uint64_t pk = ~0ull;
    int32_t pi = -1;
    for (int q = 0; q < A.k; ++q) {
      uint64_t k = 0;
      int32_t l = 0;
      if (pk != 0) best_after(A.segs * A.k, at, pk, pi, rk, ri, k, l);
      if (tid == 0) {
        A.top_idx[(size_t)b * A.k + q] = k ? l : -1;
        A.top_logp[(size_t)b * A.k + q] = k ? (float)(ord64_value(k) - m - logs) : -INFINITY;
      }
      pk = k;
      pi = l;
    }
  }
}

// ---------------------------------------------------------------- host
struct Layout {
  int G, nblk, nblkp, pairs, streams;
  size_t xa, xb, xinv, n1, nw, r1, rflag, counts, fail, done, bmax, items, listed, nnear, near_v, near_l, from, part, sk, si,
      rowstat, total;
};

// Label segments of a query on the exact path, a CTA each: 74 fill the GPU from
// four queries on (two CTAs an SM).  Fewer queries take four times as many where
// the scan is long against the join of segs x k entries, k times over (all
// labels tied, one query: 500K bf16 labels, 5 best 788 -> 347 us, but 64 best
// 1169 -> 1506; 3M E4M3 labels, 64 best 8.0 -> 2.7 ms).
int exact_segments(int64_t L, int32_t B, int32_t k) { return B < 4 && L >= (int64_t)k << 15 ? 296 : 74; }

int tile_labels(const elmo_head* h) { return h->d <= 768 ? 64 : 128; }

Layout layout_of(const elmo_head* h, int32_t B, int32_t k) {
  Layout o{};
  const bool fp8 = h->dt != ELMO_BF16;
  const int P = (B + 127) / 128;
  const int64_t N = tile_labels(h), T = (h->L + N - 1) / N;
  o.pairs = 1;
  o.streams = k > 0 && h->L <= kKeepLabels && (size_t)B * h->L * 4 <= kKeepBytes ? 0 : kStreams;
  if (k > 0 && o.streams)
    while ((size_t)B * (2 * T / o.pairs) * 4 > kMaxima) o.pairs *= 2;
  o.nblk = (int)((T + 2 * o.pairs - 1) / (2 * o.pairs));
  int64_t G = h->num_sms / P;
  if (G > o.nblk) G = o.nblk;
  if (o.streams == 0) o.nblk = (int)h->L;
  o.nblkp = (o.nblk + 7) / 8 * 8;
  if (G < 1) G = 1;
  o.G = (int)G;
  size_t off = 0;
  auto take = [&](size_t bytes) { const size_t at = off; off += (bytes + 255) / 256 * 256; return at; };
  o.xa = take(fp8 ? (size_t)B * h->d : 0);
  o.xb = take(fp8 ? (size_t)B * h->d : 0);
  o.xinv = take(4 * (size_t)B);
  o.n1 = take(4 * (size_t)B);
  o.nw = take(4 * (size_t)B);
  o.r1 = take(4 * (size_t)B);
  o.rflag = take(4 * (size_t)B);
  o.counts = take(sizeof(Counts));
  const size_t lists = k > 0 ? (size_t)B : 0;
  o.fail = take(4 * lists);
  o.done = take(4 * lists);
  o.items = take(sizeof(int2) * lists * kMaxBlocks);
  o.listed = take(4 * lists);
  o.nnear = take(4 * lists);
  o.near_v = take(4 * lists * kMaxNear);
  o.near_l = take(4 * lists * kMaxNear);
  o.from = take(4 * lists);
  o.bmax = take(k > 0 ? 4 * (size_t)(o.streams ? o.streams : 1) * B * o.nblkp : 0);
  o.part = take(sizeof(Stat) * (size_t)B * kStreams * o.G);
  o.sk = take(8 * (size_t)B * exact_segments(h->L, B, k) * k);
  o.si = take(4 * (size_t)B * exact_segments(h->L, B, k) * k);
  o.rowstat = take(16 * (size_t)B);
  o.total = off;
  return o;
}

template <int kFp8, int kW5, int kXs>
cudaError_t run_pass(elmo_head* h, Args A, cudaStream_t s) {
  constexpr int kN = kXs ? 128 : 64;
  constexpr int kOps = kFp8 ? 2 : 1;
  const int eb = kFp8 ? 1 : 2;
  const int nkb = (A.d * eb + 127) / 128;
  // up to 48 KB of W a stage (32 KB beside X), boxes of at most 256 labels
  A.kbs = kXs ? 2 : (nkb + (nkb + 5) / 6 - 1) / ((nkb + 5) / 6);
  A.q = kXs ? 1 : 6 / A.kbs < 4 ? 6 / A.kbs : 4;
  if (nkb > A.kbs) A.q = 1;
  A.kb3d = A.d * eb % 128 == 0;
  const size_t stage = (size_t)A.kbs * (A.q * kN * 128 + (kXs ? 16384 * kOps : 0));
  const size_t fixed = 1024 + sizeof(SmemP);
  int stages = (int)((kSmemMost - fixed) / stage);
  A.stages = stages < kMaxStages ? stages : kMaxStages;
  CUtensorMap tmW, tmA, tmB;
  auto map = [&](CUtensorMap* m, const void* p, int64_t rows, int box) {
    return A.kb3d ? make_tma_map_kb3d(m, p, eb, (uint64_t)A.d, (uint64_t)rows, (uint32_t)box, (uint32_t)A.kbs)
                  : make_tma_map_2d(m, p, eb, (uint64_t)A.d, (uint64_t)rows, (uint64_t)A.d, (uint32_t)box);
  };
  cudaError_t e = map(&tmW, h->W, h->L, A.q * kN);
  if (e != cudaSuccess) return e;
  tmA = tmB = tmW;
  if (kXs) {
    if ((e = map(&tmA, kFp8 ? static_cast<const void*>(A.xa) : A.X, A.B, 128)) != cudaSuccess) return e;
    if (kFp8 && (e = map(&tmB, A.xb, A.B, 128)) != cudaSuccess) return e;
  }
  auto kern = label_score_kernel<kFp8, kW5, kXs>;
  static std::atomic<uint64_t> seen{0};
  if ((e = allow_smem(kern, (int)kSmemMost, seen)) != cudaSuccess) return e;
  const int P = (A.B + 127) / 128;
  return launch_after(kern, dim3(P * A.G), kThreads, fixed + A.stages * stage, s, tmW, tmA, tmB, A);
}

template <int kFormat>
cudaError_t run_join(elmo_head* h, const Args& A, cudaStream_t s) {
  const size_t xbytes = sizeof(float) * (size_t)h->d;
  cudaError_t e = launch_after(label_join_kernel<kFormat>, dim3(A.B), kJoinThreads, xbytes, s, A);
  if (e != cudaSuccess || A.k == 0) return e;
  if (A.streams != 0) {
    e = launch_after(label_near_kernel<kFormat>, dim3(h->num_sms * 4), kNearThreads, 0, s, A, tile_labels(h));
    if (e != cudaSuccess) return e;
    e = launch_after(label_rank_kernel<kFormat>, dim3(A.B), kNearThreads, xbytes, s, A);
    if (e != cudaSuccess) return e;
  }
  return launch_after(label_exact_kernel<kFormat>, dim3(h->num_sms * 2), kExactThreads, xbytes, s, A);
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
  A.d = h->d; A.B = B; A.G = o.G; A.k = k; A.nnz = nnz;
  A.nblk = o.nblk; A.nblkp = o.nblkp; A.pairs = o.pairs; A.streams = o.streams;
  A.fmt = w_format(h);
  A.segs = exact_segments(h->L, B, k);
  A.eps = 1.5f * (fp8 ? 32.0f : 16.0f) * 0x1p-25f;
  A.xinv = reinterpret_cast<float*>(ws + o.xinv);
  A.n1 = reinterpret_cast<float*>(ws + o.n1);
  A.nw = reinterpret_cast<float*>(ws + o.nw);
  A.r1 = reinterpret_cast<float*>(ws + o.r1);
  A.rflag = reinterpret_cast<int32_t*>(ws + o.rflag);
  A.counts = reinterpret_cast<Counts*>(ws + o.counts);
  A.fail = reinterpret_cast<int32_t*>(ws + o.fail);
  A.done = reinterpret_cast<int32_t*>(ws + o.done);
  A.items = reinterpret_cast<int2*>(ws + o.items);
  A.listed = reinterpret_cast<int32_t*>(ws + o.listed);
  A.nnear = reinterpret_cast<int32_t*>(ws + o.nnear);
  A.near_v = reinterpret_cast<float*>(ws + o.near_v);
  A.near_l = reinterpret_cast<int32_t*>(ws + o.near_l);
  A.from = reinterpret_cast<float*>(ws + o.from);
  A.bmax = reinterpret_cast<float*>(ws + o.bmax);
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
    KernelScope sc(h, ELMO_K_LOGPROB_SCORE, s, 1);
    if (!fp8) e = wide ? run_pass<0, 0, 1>(h, A, s) : run_pass<0, 0, 0>(h, A, s);
    else if (h->w_e5m2) e = wide ? run_pass<1, 1, 1>(h, A, s) : run_pass<1, 1, 0>(h, A, s);
    else e = wide ? run_pass<1, 0, 1>(h, A, s) : run_pass<1, 0, 0>(h, A, s);
    if (e != cudaSuccess) return e;
  }
  KernelScope sc(h, ELMO_K_LOGPROB_JOIN, s, k == 0 ? 1 : A.streams ? 4 : 2);
  if (A.fmt == ELMO_BF16) return run_join<ELMO_BF16>(h, A, s);
  if (A.fmt == ELMO_FP8_E5M2) return run_join<ELMO_FP8_E5M2>(h, A, s);
  return run_join<ELMO_FP8_E4M3>(h, A, s);
}

}  // namespace elmo
