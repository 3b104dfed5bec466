// jf_beam.cu -- beam search over a paged cache: the best (beam, token) pairs of a step, and
// the fork of the surviving beams' block tables.
#include <algorithm>
#include <cmath>

#include "jf_common.cuh"
#include "jf_sm100.cuh"

namespace jf {
namespace {

constexpr int kPage = 16;
constexpr int kMaxK = 64;                 // most beams, and most continuations
constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------------------ scan
//
// The K best pairs of a prompt lie in few places.  The scan streams the logits once and
// keeps, for every block of logits (1024 in bf16; fewer where a prompt has few), only the
// greatest, beside the slice's maximum and sum of exponentials for the log-sum-exp.  The K-th best of the blocks' best pairs
// bounds the K-th best pair from below, so the merge reads again only the blocks that reach
// it: about K of them.  The scan has no barrier, no shared memory and no candidates; HBM
// bounds it.  (Collecting candidates while streaming cost a threshold, a compaction and a
// ranking per slice: 36 us with a CTA a slice, 50 us with a warp a slice, on 256 rows of
// 151,936 bf16 logits, whose bytes take 11.7 us.)
constexpr int kScanThreads = 128;
constexpr int kScanWarps = kScanThreads / 32;
constexpr int kStep = 4;                       // 16-byte vectors a lane holds at a time
constexpr int kStepVecs = 32 * kStep;          // vectors of a warp's step
constexpr uint32_t kNegInfKey = 0x007fffffu;   // logit_key(-inf)

// Orders as the value does; NaN lowest, -0 == +0.
__device__ __forceinline__ uint32_t logit_key(float x) {
  uint32_t u = __float_as_uint(x);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0u;
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  if (k == 0u) return -INFINITY;
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

template <typename T>
struct Row;
template <>
struct Row<uint16_t> {                    // bf16
  static constexpr int kN = 8;            // logits of a 16-byte vector
  static constexpr uint32_t kNone = 0xff80ff80u;   // -inf, -inf
  static __device__ __forceinline__ float get(const uint4& v, int c) {
    const uint32_t w = (&v.x)[c >> 1];
    return __uint_as_float((c & 1) ? (w & 0xffff0000u) : (w << 16));
  }
  static __device__ __forceinline__ void put(uint4& v, int c, uint16_t x) {
    uint32_t& w = (&v.x)[c >> 1];
    w = (c & 1) ? ((w & 0xffffu) | (static_cast<uint32_t>(x) << 16)) : ((w & 0xffff0000u) | x);
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ float vmax(const uint4& v) {
    const uint32_t m = max2(max2(v.x, v.y), max2(v.z, v.w));
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
};
template <>
struct Row<float> {
  static constexpr int kN = 4;
  static constexpr uint32_t kNone = 0xff800000u;
  static __device__ __forceinline__ float get(const uint4& v, int c) { return __uint_as_float((&v.x)[c]); }
  static __device__ __forceinline__ void put(uint4& v, int c, float x) { (&v.x)[c] = __float_as_uint(x); }
  static __device__ __forceinline__ float vmax(const uint4& v) {
    return fmaxf(fmaxf(get(v, 0), get(v, 1)), fmaxf(get(v, 2), get(v, 3)));
  }
};

__device__ __forceinline__ float to_float(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }
__device__ __forceinline__ float to_float(float x) { return x; }

struct BeamParams {
  const void* logits;
  const float* score;
  const int32_t* finished;
  int32_t* parent;
  int32_t* token;
  float* new_score;
  int32_t* new_finished;
  float2* stats;          // [rows][slices]: maximum, sum of exp(x - maximum)
  uint32_t* best;         // [rows][blocks]: key of a block's greatest logit
  int W, V, K, eos;
  int slices, slice_steps;    // slices of a row (a warp each), steps of a slice
  int steps;                  // steps of a row
  int blocks, block_vecs;     // blocks of a row, 16-byte vectors of a block
  int total;                  // rows * slices
};

// A row as 16-byte vectors, the first of which starts at the boundary at or below the row's
// first logit: logit e of the row is element e + off of the vectors.  Vectors that reach
// over either end of the row are read logit by logit.
template <typename T>
struct RowVecs {
  const T* x;
  int off, V;
  __device__ RowVecs(const void* logits, int row, int V_) : x(static_cast<const T*>(logits) + static_cast<size_t>(row) * V_), V(V_) {
    off = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
  }
  __device__ __forceinline__ int first(int vec) const { return vec * Row<T>::kN - off; }
  __device__ __forceinline__ uint4 load(int vec) const;
};

// A vector that reaches over an end of its row: the logits inside, -inf for the others.
template <typename T>
__device__ __noinline__ uint4 row_end(const T* x, int at, int V) {
  using R = Row<T>;
  uint4 r = make_uint4(R::kNone, R::kNone, R::kNone, R::kNone);
#pragma unroll
  for (int c = 0; c < R::kN; ++c)
    if (at + c >= 0 && at + c < V) R::put(r, c, x[at + c]);
  return r;
}

template <typename T>
__device__ __forceinline__ uint4 RowVecs<T>::load(int vec) const {
  const int at = first(vec);
  if (at >= 0 && at + Row<T>::kN <= V) return __ldg(reinterpret_cast<const uint4*>(x + at));
  return row_end(x, at, V);
}

template <typename T, bool SMALL>       // SMALL: blocks of part of a step's vectors
__global__ void __launch_bounds__(kScanThreads, 8) beam_scan_kernel(const BeamParams p) {
  using R = Row<T>;
  constexpr int VN = R::kN;
  grid_dependency_wait();
  grid_dependents_launch();               // the merge's blocks may take their places; it waits for this grid
  const int lane = threadIdx.x & 31, slice = blockIdx.x * kScanWarps + (threadIdx.x >> 5);
  const int row = slice / p.slices, part = slice - row * p.slices;
  // (the merge makes the pairs of beams that are not live itself)
  if (slice >= p.total || (p.finished != nullptr && p.finished[row] != 0) || p.score[row] == -INFINITY) {
    return;
  }
  const RowVecs<T> r(p.logits, row, p.V);
  const int step0 = part * p.slice_steps, steps = min(p.slice_steps, p.steps - step0);
  const int vec0 = step0 * kStepVecs + lane;
  // (a slice holds whole blocks)
  const int block_steps = max(1, p.block_vecs / kStepVecs);
  uint32_t* best = p.best + static_cast<size_t>(row) * p.blocks;
  int block = step0 / block_steps;
  float m = -INFINITY, sum = 0.f;         // of this lane
  uint32_t greatest = 0u;                 // of this lane, in the block
  uint4 next[kStep];
#pragma unroll
  for (int u = 0; u < kStep; ++u) next[u] = r.load(vec0 + u * 32);
#pragma unroll 1
  for (int i = 0, left = block_steps; i < steps; ++i) {
    uint4 v[kStep];
#pragma unroll
    for (int u = 0; u < kStep; ++u) v[u] = next[u];
    if (i + 1 < steps) {
#pragma unroll
      for (int u = 0; u < kStep; ++u) next[u] = r.load(vec0 + (i + 1) * kStepVecs + u * 32);
    }
    const float mine = fmaxf(fmaxf(R::vmax(v[0]), R::vmax(v[1])), fmaxf(R::vmax(v[2]), R::vmax(v[3])));
    if constexpr (SMALL) {                // 32, 8 or 1 vectors
#pragma unroll
      for (int u = 0; u < kStep; ++u) {
        uint32_t top = logit_key(R::vmax(v[u]));
        for (int o = 1; o < p.block_vecs; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int at = (vec0 + i * kStepVecs + u * 32) / p.block_vecs;
        if ((lane & (p.block_vecs - 1)) == 0 && at < p.blocks) best[at] = top;
      }
    } else {
      greatest = max(greatest, logit_key(mine));
      if (--left == 0) {
        const uint32_t top = __reduce_max_sync(0xffffffffu, greatest);
        if (lane == 0) best[block] = top;
        ++block;
        greatest = 0u;
        left = block_steps;
      }
    }
    const float up = fmaxf(m, mine), ref = up == -INFINITY ? 0.f : up;
    if (up > m) sum *= fast_exp2((m - ref) * kLog2e);
    m = up;
    const uint64_t neg = f2(-ref, -ref), l2e = f2(kLog2e, kLog2e);
    uint64_t acc = 0ull, acc1 = 0ull;
#pragma unroll
    for (int u = 0; u < kStep; ++u)
#pragma unroll
      for (int c = 0; c < VN; c += 4) {
        float a, b, d, e;
        f2_split(fmul2(fadd2(f2(R::get(v[u], c), R::get(v[u], c + 1)), neg), l2e), a, b);
        f2_split(fmul2(fadd2(f2(R::get(v[u], c + 2), R::get(v[u], c + 3)), neg), l2e), d, e);
        acc = fadd2(acc, f2(fast_exp2(a), fast_exp2(b)));
        acc1 = fadd2(acc1, f2(fast_exp2(d), fast_exp2(e)));
      }
    float a, b;
    f2_split(fadd2(acc, acc1), a, b);
    sum += a + b;
  }
  float M = m;
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  sum *= m == -INFINITY ? 0.f : fast_exp2((m - M) * kLog2e);
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) p.stats[slice] = make_float2(M, sum);
}

// ------------------------------------------------------------------------ merge

// A pair's rank: score (as ordered 64 bits), then the lower flat index w * V + v.
struct Pair {
  uint64_t key;
  uint32_t flat;
};
__device__ __forceinline__ bool before(const Pair& a, const Pair& b) {
  return a.key > b.key || (a.key == b.key && a.flat < b.flat);
}
__device__ __forceinline__ uint64_t score_key(double s) {
  if (!(s == s)) return 0ull;
  uint64_t u = static_cast<uint64_t>(__double_as_longlong(s));
  if (u == 0x8000000000000000ull) u = 0ull;
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ double key_score(uint64_t k) {
  if (k == 0ull) return -INFINITY;
  return __longlong_as_double(static_cast<long long>((k >> 63) ? (k & 0x7fffffffffffffffull) : ~k));
}

constexpr int kMergeThreads = 512;
constexpr int kMergeWarps = kMergeThreads / 32;
constexpr int kMergeBlocks = 8192;        // blocks of a prompt: 8 bytes of shared memory each
constexpr int kBins = 1024;
constexpr int kListCap = kMaxK + 32;      // pairs a warp collects before it cuts back to K

__device__ __forceinline__ void two_sum(float& hi, float& lo, float x, float x_lo) {
  const float s = hi + x, t = s - hi;
  lo += x_lo + ((hi - (s - t)) + (x - t));
  hi = s;
}

// log(z), z >= 1, to about 1e-11: one Newton step y + (z e^-y - 1) from the fp32 logarithm,
// with e^-y = 2^k e^r, |r| <= 0.35, and the Taylor series of e^r to the ninth power in
// Estrin's order.  A dependent fp64 instruction takes some 100 cycles here, so the chain's
// length (13) is what counts; the library's exp and log took 11,000 cycles together.
__device__ __forceinline__ double log_fp64(double z) {
  const float y = logf(static_cast<float>(z));
  const float k = rintf(y * 1.44269504f);
  const double r = fma(static_cast<double>(k), 0.69314718055994530942, -static_cast<double>(y));
  const double r2 = r * r, r4 = r2 * r2;
  const double a = fma(r, 1.0, 1.0), b = fma(r, 1.0 / 6, 1.0 / 2), c = fma(r, 1.0 / 120, 1.0 / 24),
               d = fma(r, 1.0 / 5040, 1.0 / 720), e = fma(r, 1.0 / 362880, 1.0 / 40320);
  const double lo = fma(r2, b, a), hi = fma(r2, d, c);
  const double er = fma(r4, fma(r4, e, hi), lo);
  const double back = z * __hiloint2double((1023 - static_cast<int>(k)) << 20, 0);   // z 2^-k
  return static_cast<double>(y) + fma(back, er, -1.0);
}

// Sorts a warp's n <= kListCap pairs and keeps the first K; returns their number.
__device__ __noinline__ int cut_back(uint64_t* key, uint32_t* flat, int n, int K) {
  const int lane = threadIdx.x & 31;
  constexpr int kMine = kListCap / 32;
  Pair e[kMine];
  int r[kMine];
#pragma unroll
  for (int u = 0; u < kMine; ++u) {
    const int i = u * 32 + lane;
    e[u] = i < n ? Pair{key[i], flat[i]} : Pair{0ull, 0u};
    r[u] = 0;
  }
  for (int j = 0; j < n; ++j) {
    const Pair x{key[j], flat[j]};
#pragma unroll
    for (int u = 0; u < kMine; ++u) r[u] += before(x, e[u]);
  }
  __syncwarp();
#pragma unroll
  for (int u = 0; u < kMine; ++u)
    if (u * 32 + lane < n && r[u] < K) {
      key[r[u]] = e[u].key;
      flat[r[u]] = e[u].flat;
    }
  __syncwarp();
  return min(n, K);
}

// A pair's score is off + (x - M), with its beam's off = score - log(sum exp(x - M)) and greatest
// logit M: x - M is small where it counts, however far from zero the logits are.  (With M in off
// instead, a beam whose tokens are all masked with the type's lowest value loses its score and its
// logarithm to the rounding of M, and outranks the others.)  Here in fp32, as an ordered word.
__device__ __forceinline__ uint32_t score_word(float off, float M, float x) { return logit_key(off + (x - M)); }

// One CTA per prompt: the log-sum-exp of every beam, the bound from the blocks' best pairs,
// the pairs of the blocks that reach it, their ranking.  A chain of small dependent steps
// bounds the call, so half the warps form the bound from fp32 scores while the others take
// the fp64 logarithms that the ranking wants.  An fp32 score s is off by 2^-24 times the sizes
// of what is rounded (off, x - M, which is at most |off| + |s|, and s) and 2^-19 for logf (below
// 25): in all 2^-23 (|off| + |s|) + 2^-19.  A pair among the K best may stand below the K-th
// block's word by twice that, so the bound is lowered by 2^-22 (|score| + 32 + |off| + |s|) and
// a little more.
constexpr int kBoundThreads = kMergeThreads / 2;
template <typename T>
__global__ void __launch_bounds__(kMergeThreads) beam_merge_kernel(const BeamParams p) {
  using R = Row<T>;
  constexpr int VN = R::kN;
  extern __shared__ uint32_t s_dyn[];     // [heads]: score words, then [heads]: blocks that pass
  __shared__ double s_off[kMaxK];         // score - log of the sum
  __shared__ float s_off32[kMaxK], s_mag[kMaxK];
  __shared__ float s_stat[3][kMaxK];      // maximum (0 without logits above -inf), sum of exponentials in two parts
  __shared__ int s_kind[kMaxK];           // 0 live, 1 finished, 2 without a score
  __shared__ uint32_t s_hist[kBins];
  __shared__ uint64_t s_key[kMergeWarps][kListCap];
  __shared__ uint32_t s_flat[kMergeWarps][kListCap];
  __shared__ uint64_t s_all_key[kMergeWarps * kMaxK + kMaxK];
  __shared__ __align__(16) uint32_t s_all_hi[kMergeWarps * kMaxK + kMaxK];
  __shared__ uint32_t s_all_flat[kMergeWarps * kMaxK + kMaxK];
  __shared__ uint32_t s_range[2], s_warp[kBoundThreads / 32];
  __shared__ int s_bin, s_pass, s_n;
  grid_dependency_wait();
  const int b = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int W = p.W, K = p.K, heads = W * p.blocks;
  uint32_t* s_word = s_dyn;
  uint32_t* s_list = s_dyn + heads;
  const uint32_t* best = p.best + static_cast<size_t>(b) * heads;
#pragma unroll 1
  for (int i = tid; i < heads; i += kMergeThreads)    // (those of beams that are not live are not used)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(s_word + i)), "l"(best + i) : "memory");
  for (int w = warp; w < W; w += kMergeWarps) {
    const int row = b * W + w;
    // (asked for together; those of a beam that is not live are not used)
    const float2* st = p.stats + static_cast<size_t>(row) * p.slices;
    const float2 mine = lane < p.slices ? st[lane] : make_float2(-INFINITY, 0.f);
    const float sc = p.score[row];
    const bool over = p.finished != nullptr && p.finished[row] != 0;
    float M = -INFINITY, hi = 0.f, lo = 0.f, off = sc, mag = 0.f;
    if (!over && sc != -INFINITY) {
      M = mine.x;
      for (int c = lane + 32; c < p.slices; c += 32) M = fmaxf(M, st[c].x);
#pragma unroll
      for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      if (M != -INFINITY) {
        hi = mine.y * expf(mine.x - M);
        for (int c = lane + 32; c < p.slices; c += 32) two_sum(hi, lo, st[c].y * expf(st[c].x - M), 0.f);
#pragma unroll
        for (int o = 16; o; o >>= 1) {
          const float x = __shfl_xor_sync(0xffffffffu, hi, o), y = __shfl_xor_sync(0xffffffffu, lo, o);
          two_sum(hi, lo, x, y);
        }
        off = sc - logf(hi);
        mag = fabsf(sc) + 32.f;
      }
    }
    if (lane == 0) {
      s_kind[w] = over ? 1 : (sc == -INFINITY ? 2 : 0);
      s_off32[w] = off;
      s_mag[w] = mag;
      s_stat[0][w] = M == -INFINITY ? 0.f : M;
      s_stat[1][w] = hi;
      s_stat[2][w] = lo;
    }
  }
  if (tid == 0) {
    s_range[0] = 0xffffffffu;
    s_range[1] = 0u;
    s_pass = 0;
    s_n = 0;
    s_bin = -1;
  }
  for (int i = tid; i < kBins; i += kMergeThreads) s_hist[i] = 0u;
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  if (tid >= kBoundThreads) {
    // fp64 offsets; a finished beam's only pair goes straight into the final list.
    for (int w = warp - kBoundThreads / 32; w < W; w += kMergeWarps / 2)
      if (lane == 0) {
        double off = p.score[b * W + w];
        if (s_kind[w] == 0 && s_stat[1][w] != 0.f)
          off -= log_fp64(static_cast<double>(s_stat[1][w]) + s_stat[2][w]);
        s_off[w] = off;
        if (s_kind[w] == 1 && off != -INFINITY) {
          const int n = atomicAdd(&s_n, 1);
          s_all_key[n] = score_key(off);
          s_all_hi[n] = static_cast<uint32_t>(s_all_key[n] >> 32);
          s_all_flat[n] = static_cast<uint32_t>(w) * static_cast<uint32_t>(p.V) + static_cast<uint32_t>(p.eos);
        }
      }
  } else {
    // Score words of the blocks' best pairs; 0 where a block has no pair above -inf.
    // i / blocks for i < 2^13: the product's excess, i (recip - 2^32 / blocks), stays below
    // 2^32 / blocks.  (This and the loops left rolled, since every step's code is fetched and
    // run once: 14.9 -> 14.3 us a call on 1 x 4 x 151936.)
    const uint32_t recip = 0xffffffffu / static_cast<uint32_t>(p.blocks) + 1u;
    uint32_t low = 0xffffffffu, high = 0u;
#pragma unroll 1
    for (int i = tid; i < heads; i += kBoundThreads) {
      const int w = p.blocks == 1 ? i : static_cast<int>(__umulhi(static_cast<uint32_t>(i), recip));
      const uint32_t k = s_word[i];
      uint32_t word = 0u;
      if (s_kind[w] == 0 && k > kNegInfKey) {
        word = score_word(s_off32[w], s_stat[0][w], key_logit(k));
        if (word != 0u) {
          low = min(low, word);
          high = max(high, word);
        }
      }
      s_word[i] = word;
    }
    float most = 0.f;                     // greatest sum of what is rounded, of a live beam
    for (int w = lane; w < W; w += 32) most = fmaxf(most, s_mag[w] + fabsf(s_kind[w] == 0 ? s_off32[w] : 0.f));
#pragma unroll
    for (int o = 16; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    low = __reduce_min_sync(0xffffffffu, low);
    high = __reduce_max_sync(0xffffffffu, high);
    if (lane == 0) {
      atomicMin(&s_range[0], low);
      atomicMax(&s_range[1], high);
    }
    named_bar(1, kBoundThreads);
    // The K-th greatest word's step of a histogram over their range; its lower end is the
    // bound.  With fewer than K words everything passes.
    low = s_range[0];
    high = s_range[1];
    uint32_t bound = 1u;
    if (low <= high) {
      constexpr int kMine = kBins / kBoundThreads;
      const int shift = max(0, 32 - __clz(high - low) - 10);
#pragma unroll 1
      for (int i = tid; i < heads; i += kBoundThreads)
        if (s_word[i] != 0u) atomicAdd(&s_hist[(s_word[i] - low) >> shift], 1u);
      named_bar(1, kBoundThreads);
      const int top = kBins - 1 - kMine * tid;
      uint32_t c[kMine], all = 0u;
#pragma unroll
      for (int i = 0; i < kMine; ++i) all += c[i] = s_hist[top - i];
      uint32_t incl = all;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      if (lane == 31) s_warp[warp] = incl;
      named_bar(1, kBoundThreads);
      uint32_t above = incl - all;
      for (int v = 0; v < warp; ++v) above += s_warp[v];
      const uint32_t want = static_cast<uint32_t>(K);
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        if (above < want && above + c[i] >= want) s_bin = top - i;
        above += c[i];
      }
      named_bar(1, kBoundThreads);
      if (s_bin >= 0) {
        const float at = key_logit(low + (static_cast<uint32_t>(s_bin) << shift));
        bound = max(1u, logit_key(at - 2.3841858e-7f * (most + fabsf(at)) - 9.5367432e-7f));
      }
    }
#pragma unroll 1
    for (int i = tid; i < heads; i += kBoundThreads)
      if (s_word[i] >= bound) s_list[atomicAdd(&s_pass, 1)] = i;
    if (tid == 0) s_range[0] = bound;
  }
  __syncthreads();
  const uint32_t bound = s_range[0];
  const int pass = s_pass;
  uint64_t* key = s_key[warp];
  uint32_t* flat = s_flat[warp];
  int n = 0;
  Pair last{0ull, 0xffffffffu};           // the K-th pair so far: what does not rank before it is out
  for (int i = warp; i < pass; i += kMergeWarps) {
    const int id = s_list[i], w = id / p.blocks, block = id - w * p.blocks;
    const double off = s_off[w];
    const float off32 = s_off32[w], M = s_stat[0][w];
    const RowVecs<T> r(p.logits, b * W + w, p.V);
    for (int v0 = 0; v0 < p.block_vecs; v0 += kStepVecs) {
      uint4 v[kStep];
#pragma unroll
      for (int u = 0; u < kStep; ++u) {
        const int i_vec = v0 + u * 32 + lane;
        v[u] = make_uint4(R::kNone, R::kNone, R::kNone, R::kNone);
        if (i_vec < p.block_vecs) v[u] = r.load(block * p.block_vecs + i_vec);
      }
#pragma unroll
      for (int u = 0; u < kStep; ++u) {
        const float most = R::vmax(v[u]);
        const int first = r.first(block * p.block_vecs + v0 + u * 32 + lane);
        bool look = score_word(off32, M, most) >= bound;
        if (look && last.key != 0ull)         // (many equal logits: nothing here ranks before the K-th)
          look = before(Pair{score_key(off + (static_cast<double>(most) - M)),
                             static_cast<uint32_t>(w) * static_cast<uint32_t>(p.V) + static_cast<uint32_t>(max(first, 0))}, last);
        uint32_t some = __ballot_sync(0xffffffffu, look);
        // One passing vector (there are few) after the other, a lane a logit.
        for (; some != 0u; some &= some - 1u) {
          const int src = __ffs(some) - 1;
          uint4 t;
          t.x = __shfl_sync(0xffffffffu, v[u].x, src);
          t.y = __shfl_sync(0xffffffffu, v[u].y, src);
          t.z = __shfl_sync(0xffffffffu, v[u].z, src);
          t.w = __shfl_sync(0xffffffffu, v[u].w, src);
          const int token = __shfl_sync(0xffffffffu, first, src) + lane;
          float x = -INFINITY;
#pragma unroll
          for (int c = 0; c < VN; ++c)
            if (lane == c) x = R::get(t, c);
          bool in = x != -INFINITY && score_word(off32, M, x) >= bound && token >= 0 && token < p.V;
          Pair e{0ull, 0u};
          if (in) {
            e = Pair{score_key(off + (static_cast<double>(x) - M)), static_cast<uint32_t>(w) * static_cast<uint32_t>(p.V) + static_cast<uint32_t>(token)};
            in = before(e, last);
          }
          if (n + VN > kListCap) {
            n = cut_back(key, flat, n, K);
            last = Pair{key[K - 1], flat[K - 1]};      // (n was above kMaxK)
            in = in && before(e, last);
          }
          const uint32_t ms = __ballot_sync(0xffffffffu, in);
          if (in) {
            const int to = n + __popc(ms & ((1u << lane) - 1u));
            key[to] = e.key;
            flat[to] = e.flat;
          }
          n += __popc(ms);
          __syncwarp();
        }
      }
    }
  }
  if (n > K) n = cut_back(key, flat, n, K);
  if (n > 0) {
    int at = 0;
    if (lane == 0) at = atomicAdd(&s_n, n);
    at = __shfl_sync(0xffffffffu, at, 0);
    for (int i = lane; i < n; i += 32) {
      s_all_key[at + i] = key[i];
      s_all_hi[at + i] = static_cast<uint32_t>(key[i] >> 32);
      s_all_flat[at + i] = flat[i];
    }
  }
  __syncthreads();
  const int all = s_n;
  auto put = [&](int rank, uint32_t flat_at, float score) {
    const int w = static_cast<int>(flat_at / static_cast<uint32_t>(p.V));
    const int v = static_cast<int>(flat_at - static_cast<uint32_t>(w) * static_cast<uint32_t>(p.V));
    const size_t o = static_cast<size_t>(b) * K + rank;
    p.parent[o] = w;
    p.token[o] = v;
    p.new_score[o] = score;
    if (p.new_finished != nullptr) p.new_finished[o] = (s_kind[w] == 1 || v == p.eos) ? 1 : 0;
  };
  for (int i = tid; i < all; i += kMergeThreads) {
    const uint32_t hi = s_all_hi[i];
    int rank = 0, equal = 0;
#pragma unroll 1
    for (int j = 0; j < all / 4; ++j) {
      const uint4 h = reinterpret_cast<const uint4*>(s_all_hi)[j];
      rank += (h.x > hi) + (h.y > hi) + (h.z > hi) + (h.w > hi);
      equal += (h.x == hi) + (h.y == hi) + (h.z == hi) + (h.w == hi);
    }
    for (int j = all / 4 * 4; j < all; ++j) {
      rank += s_all_hi[j] > hi;
      equal += s_all_hi[j] == hi;
    }
    if (rank >= K) continue;
    const Pair mine{s_all_key[i], s_all_flat[i]};
    if (equal > 1)
      for (int j = 0; j < all; ++j) rank += s_all_hi[j] == hi && before(Pair{s_all_key[j], s_all_flat[j]}, mine);
    if (rank < K) put(rank, mine.flat, static_cast<float>(key_score(mine.key)));
  }
  // Fewer than K pairs above -inf: the rest are the first pairs at -inf (each live beam has
  // fewer than K others, so they come early).
  if (all < K && warp == 0) {
    int at = all;
    for (int w = 0; w < W && at < K; ++w) {
      const T* x = static_cast<const T*>(p.logits) + static_cast<size_t>(b * W + w) * p.V;
      for (int t0 = 0; t0 < p.V && at < K; t0 += 32) {
        const int t = t0 + lane;
        bool none = t < p.V;
        if (s_kind[w] == 0) none = none && to_float(x[t]) == -INFINITY;
        else if (s_kind[w] == 1) none = none && (t != p.eos || s_off[w] == -INFINITY);
        const uint32_t ms = __ballot_sync(0xffffffffu, none);
        const int rank = at + __popc(ms & ((1u << lane) - 1u));
        if (none && rank < K) put(rank, static_cast<uint32_t>(w) * static_cast<uint32_t>(p.V) + static_cast<uint32_t>(t), -INFINITY);
        at += __popc(ms);
      }
    }
    // (left only where NaN or +inf took a beam's pairs away: nothing stale is left behind)
    for (int rank = at + lane; rank < K; rank += 32) put(rank, 0u, __int_as_float(0x7fffffff));
  }
  grid_dependents_launch();
}

// ------------------------------------------------------------------------ fork

constexpr int kForkThreads = 256;

// The first slots of a page are one run of bytes (all kv-heads of slot 0, then slot 1, ..),
// so a partial page is one contiguous copy.  blockIdx.y: K or V, and a part of the run; the
// CTA of K's first part also writes the beam's block-table row.
__global__ void __launch_bounds__(kForkThreads)
    fork_kernel(uint16_t* k_cache, uint16_t* v_cache, const int32_t* __restrict__ block_table,
                const int32_t* __restrict__ prefix_len, const int32_t* __restrict__ parent,
                const int32_t* __restrict__ fresh_page, int W, int K, int row_vecs, int max_pages,
                int num_pages, int parts, int32_t* __restrict__ new_table,
                int32_t* __restrict__ new_len, int32_t* dev_err) {
  grid_dependency_wait();
  const int j = blockIdx.x, b = j / K, tid = threadIdx.x;
  const int part = blockIdx.y % parts;
  const bool is_v = static_cast<int>(blockIdx.y) >= parts;
  const bool lead = blockIdx.y == 0;
  const int w = parent[j];
  int32_t* nt = new_table + static_cast<size_t>(j) * max_pages;
  int bits = 0, len = 0;
  if (w < 0 || w >= W) bits = JF_DEVERR_BAD_PATH;
  else {
    len = prefix_len[static_cast<size_t>(b) * W + w];
    if (len < 0 || len > max_pages * kPage) bits = JF_DEVERR_BAD_PREFIX;
  }
  if (bits) {
    if (lead) {
      if (tid == 0) {
        report(dev_err, bits);
        new_len[j] = 0;
      }
      for (int i = tid; i < max_pages; i += kForkThreads) nt[i] = -1;
    }
    grid_dependents_launch();
    return;
  }
  const int32_t* bt = block_table + (static_cast<size_t>(b) * W + w) * max_pages;
  const int full = len / kPage, slots = len % kPage;
  const int fresh = fresh_page[j];
  const int from = full < max_pages && slots > 0 ? bt[full] : 0;
  auto bad = [&](int page) { return page < 0 || page >= num_pages; };
  const bool stop = full < max_pages && (bad(fresh) || bad(from));
  if (lead) {
    bool wrong = stop;
    for (int i = tid; i < max_pages; i += kForkThreads) {
      const int page = i < full ? bt[i] : (i == full ? fresh : -1);
      wrong |= i < full && bad(page);
      nt[i] = page;
    }
    wrong = __syncthreads_or(wrong);
    if (wrong)                            // as for a bad parent: nothing that a later call could read
      for (int i = tid; i < max_pages; i += kForkThreads) nt[i] = -1;
    if (tid == 0) {
      if (wrong) report(dev_err, JF_DEVERR_BAD_PAGE);
      new_len[j] = wrong ? 0 : len;
    }
  }
  if (full < max_pages && !stop && slots > 0) {
    const int n = slots * row_vecs, span = (n + parts - 1) / parts;
    const int lo = min(n, part * span), hi = min(n, lo + span);
    uint16_t* cache = is_v ? v_cache : k_cache;
    const uint4* src = reinterpret_cast<const uint4*>(cache) + static_cast<size_t>(from) * kPage * row_vecs;
    uint4* dst = reinterpret_cast<uint4*>(cache) + static_cast<size_t>(fresh) * kPage * row_vecs;
    for (int i0 = lo + tid; i0 < hi; i0 += kForkThreads * 4) {
      uint4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i0 + u * kForkThreads < hi) v[u] = src[i0 + u * kForkThreads];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i0 + u * kForkThreads < hi) dst[i0 + u * kForkThreads] = v[u];
    }
  }
  grid_dependents_launch();
}

// ------------------------------------------------------------------------ host

struct BeamPlan {
  int blocks, block_vecs;     // blocks of a row, vectors of a block
  int steps;                  // 128-vector steps of a row (whole blocks)
  int slices, slice_steps;    // slices of a row (a warp each), steps of a slice
};

// A block is one step of a warp, 128 vectors; more where a prompt would have more than
// kMergeBlocks, and 32, 8 or 1 vectors where it would have fewer than 8 K, since the bound
// comes from the K-th best block (4 prompts of 3 x 6000 bf16 logits, K = 20: 17 us, against
// 170 us with blocks of 1024 logits, where the merge has to look at every logit).  A slice is eight steps while that gives every SM 16
// warps; with few rows, shorter ones spread a row over more SMs.  One vector more than the
// logits fill: a row may start inside one.
void plan_beam(long long rows, int W, int V, int K, int dtype, int sms, BeamPlan* pl) {
  const int vn = dtype == JF_DTYPE_BF16 ? 8 : 4;
  const long long vecs = (static_cast<long long>(V) + vn - 1) / vn + 1;
  auto blocks_of = [&](int block_vecs) { return (vecs + block_vecs - 1) / block_vecs; };
  pl->block_vecs = kStepVecs;
  while (W * blocks_of(pl->block_vecs) > kMergeBlocks) pl->block_vecs *= 2;
  while (pl->block_vecs > 1 && pl->block_vecs <= kStepVecs && W * blocks_of(pl->block_vecs) < 8ll * K)
    pl->block_vecs = pl->block_vecs > 8 ? pl->block_vecs / 4 : 1;
  pl->blocks = static_cast<int>(blocks_of(pl->block_vecs));
  const int block_steps = std::max(1, pl->block_vecs / kStepVecs);
  pl->steps = static_cast<int>((vecs + kStepVecs - 1) / kStepVecs + block_steps - 1) / block_steps * block_steps;
  for (pl->slice_steps = 8 * block_steps; pl->slice_steps > block_steps; pl->slice_steps /= 2)
    if (rows * ((pl->steps + pl->slice_steps - 1) / pl->slice_steps) >= 16ll * sms) break;
  pl->slices = (pl->steps + pl->slice_steps - 1) / pl->slice_steps;
}

bool beam_sizes_ok(int32_t B, int32_t W, int32_t V, int32_t K) {
  return B >= 1 && W >= 1 && V >= 1 && K >= 1;
}
bool beam_supported(int32_t B, int32_t W, int32_t V, int32_t K) {
  return K <= kMaxK && W <= kMaxK && static_cast<long long>(W) * V <= (1ll << 26) &&
         static_cast<long long>(K) <= static_cast<long long>(W) * V &&
         static_cast<long long>(B) * W < (1ll << 20);
}

size_t beam_workspace(const BeamPlan& pl, long long rows) {
  return static_cast<size_t>(rows) * (pl.slices * sizeof(float2) + pl.blocks * sizeof(uint32_t));
}

template <typename T>
cudaError_t launch_beam(const BeamParams& p, int B, cudaStream_t s) {
  static SmemAttr attr;
  if (!attr.ensure(beam_merge_kernel<T>, 2 * sizeof(uint32_t) * kMergeBlocks)) return cudaErrorUnknown;
  const dim3 grid(static_cast<unsigned>((p.total + kScanWarps - 1) / kScanWarps));
  const cudaError_t e = p.block_vecs < kStepVecs
                            ? launch_pdl(beam_scan_kernel<T, true>, grid, dim3(kScanThreads), 0, s, p)
                            : launch_pdl(beam_scan_kernel<T, false>, grid, dim3(kScanThreads), 0, s, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(beam_merge_kernel<T>, dim3(static_cast<unsigned>(B)), dim3(kMergeThreads),
                    2 * sizeof(uint32_t) * p.W * p.blocks, s, p);
}

}  // namespace
}  // namespace jf

extern "C" size_t jf_beam_select_workspace_size(int32_t B, int32_t W, int32_t V, int32_t K,
                                                int32_t dtype) {
  using namespace jf;
  if (!beam_sizes_ok(B, W, V, K) || !beam_supported(B, W, V, K) ||
      (dtype != JF_DTYPE_BF16 && dtype != JF_DTYPE_F32))
    return static_cast<size_t>(-1);
  const int sms = current_sm_count();
  if (sms <= 0) return static_cast<size_t>(-1);
  BeamPlan pl;
  plan_beam(static_cast<long long>(B) * W, W, V, K, dtype, sms, &pl);
  return beam_workspace(pl, static_cast<long long>(B) * W);
}

extern "C" jf_status jf_beam_select(const void* logits, int32_t dtype, const float* score,
                                    const int32_t* finished, int32_t eos_token, int32_t B,
                                    int32_t W, int32_t V, int32_t K, int32_t* parent,
                                    int32_t* token, float* new_score, int32_t* new_finished,
                                    void* workspace, size_t workspace_bytes, jf_stream_t stream) {
  using namespace jf;
  if (logits == nullptr || score == nullptr || parent == nullptr || token == nullptr ||
      new_score == nullptr || workspace == nullptr)
    return JF_ERR_INVALID_ARGUMENT;
  if ((dtype != JF_DTYPE_BF16 && dtype != JF_DTYPE_F32) || !beam_sizes_ok(B, W, V, K))
    return JF_ERR_INVALID_ARGUMENT;
  if (eos_token < -1 || eos_token >= V || (finished != nullptr && eos_token < 0))
    return JF_ERR_INVALID_ARGUMENT;
  if (!beam_supported(B, W, V, K)) return JF_ERR_UNSUPPORTED;
  // (one prompt's block writes while another's still reads)
  const size_t beams = sizeof(int32_t) * static_cast<size_t>(B) * W, pairs = sizeof(int32_t) * static_cast<size_t>(B) * K;
  if (overlap(new_score, pairs, score, beams) ||
      (finished != nullptr && new_finished != nullptr && overlap(new_finished, pairs, finished, beams)))
    return JF_ERR_INVALID_ARGUMENT;
  if (!aligned_to(logits, dtype == JF_DTYPE_BF16 ? 2 : 4) || !aligned_to(workspace, 8)) return JF_ERR_MISALIGNED;
  const int sms = current_sm_count();
  if (sms <= 0) return JF_ERR_CUDA;
  const long long rows = static_cast<long long>(B) * W;
  BeamPlan pl;
  plan_beam(rows, W, V, K, dtype, sms, &pl);
  if (rows * pl.slices >= (1ll << 31)) return JF_ERR_UNSUPPORTED;
  if (workspace_bytes < beam_workspace(pl, rows)) return JF_ERR_WORKSPACE_TOO_SMALL;
  BeamParams p;
  p.logits = logits;
  p.score = score;
  p.finished = finished;
  p.parent = parent;
  p.token = token;
  p.new_score = new_score;
  p.new_finished = new_finished;
  p.stats = static_cast<float2*>(workspace);
  p.best = reinterpret_cast<uint32_t*>(p.stats + static_cast<size_t>(rows) * pl.slices);
  p.W = W;
  p.V = V;
  p.K = K;
  p.eos = eos_token;
  p.slices = pl.slices;
  p.slice_steps = pl.slice_steps;
  p.steps = pl.steps;
  p.blocks = pl.blocks;
  p.block_vecs = pl.block_vecs;
  p.total = static_cast<int>(rows * pl.slices);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == JF_DTYPE_BF16 ? launch_beam<uint16_t>(p, B, s) : launch_beam<float>(p, B, s);
  return e == cudaSuccess ? JF_OK : JF_ERR_CUDA;
}

extern "C" jf_status jf_beam_fork_kv(void* k_cache, void* v_cache, const int32_t* block_table,
                                     const int32_t* prefix_len, const int32_t* parent,
                                     const int32_t* fresh_page, int32_t B, int32_t W, int32_t K,
                                     int32_t Hkv, int32_t D, int32_t page_size, int32_t max_pages,
                                     int32_t num_pages, int32_t* new_block_table,
                                     int32_t* new_prefix_len, int32_t* dev_err,
                                     jf_stream_t stream) {
  using namespace jf;
  if (k_cache == nullptr || v_cache == nullptr || block_table == nullptr || prefix_len == nullptr ||
      parent == nullptr || fresh_page == nullptr || new_block_table == nullptr || new_prefix_len == nullptr)
    return JF_ERR_INVALID_ARGUMENT;
  if (B < 1 || W < 1 || K < 1 || Hkv < 1 || max_pages < 1 || num_pages < 1) return JF_ERR_INVALID_ARGUMENT;
  if ((D != 64 && D != 128) || page_size != kPage || Hkv > 65535 || max_pages > (1 << 26)) return JF_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * std::max(W, K) >= (1ll << 31)) return JF_ERR_UNSUPPORTED;
  // (one beam's blocks write while another's still read)
  const size_t olds = sizeof(int32_t) * static_cast<size_t>(B) * W, news = sizeof(int32_t) * static_cast<size_t>(B) * K;
  if (overlap(new_block_table, news * max_pages, block_table, olds * max_pages) ||
      overlap(new_prefix_len, news, prefix_len, olds))
    return JF_ERR_INVALID_ARGUMENT;
  if (!aligned_to(k_cache, 16) || !aligned_to(v_cache, 16)) return JF_ERR_MISALIGNED;
  const int sms = current_sm_count();
  if (sms <= 0) return JF_ERR_CUDA;
  const int row_vecs = Hkv * D / 8;
  int parts = 1;
  while (parts < 8 && static_cast<long long>(B) * K * 2 * parts < 2 * sms && kPage * row_vecs > parts * kForkThreads) parts *= 2;
  const cudaError_t e = launch_pdl(
      fork_kernel, dim3(static_cast<unsigned>(B * K), static_cast<unsigned>(2 * parts)), dim3(kForkThreads), 0,
      reinterpret_cast<cudaStream_t>(stream), static_cast<uint16_t*>(k_cache), static_cast<uint16_t*>(v_cache),
      block_table, prefix_len, parent, fresh_page, W, K, row_vecs, max_pages, num_pages, parts, new_block_table,
      new_prefix_len, dev_err);
  return e == cudaSuccess ? JF_OK : JF_ERR_CUDA;
}
