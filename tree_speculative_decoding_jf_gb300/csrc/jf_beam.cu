// jf_beam.cu -- beam search over a paged cache: the best (beam, token) pairs of a step, and
// the fork of the surviving beams' block tables.
#include <algorithm>
#include <cmath>

#include "jf_common.cuh"
#include "jf_sm100.cuh"

namespace jf {
namespace {

constexpr int kPage = 16;
constexpr int kMaxK = 64;

// ------------------------------------------------------------------------ candidates
//
// Within a beam the pairs rank as the logits do, so a slice of a row contributes at most
// its K greatest logits.  A thread's 16-byte vectors stay packed in registers: the slice's
// maximum, its sum of exponentials and its candidates come from one read of the logits,
// which is all that bounds the call (bytes / HBM bandwidth).  The K-th greatest of 32 (or,
// for K > 16, 256) groups' maxima is a value that K logits of the slice reach, so only
// vectors that reach it are looked at logit by logit.
constexpr int kScanThreads = 256;
constexpr int kScanWarps = kScanThreads / 32;
constexpr int kCandCap = 512;
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
  float2* stats;          // [rows][chunks]: maximum, sum of exp(x - maximum)
  uint64_t* cand;         // [rows][chunks][K]: logit key << 32 | ~token, descending; 0 = none
  int W, V, K, eos, chunks, chunk_vecs;
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

template <typename T, int NV>
__global__ void __launch_bounds__(kScanThreads, 4) beam_scan_kernel(const BeamParams p) {
  using R = Row<T>;
  constexpr int VN = R::kN;
  __shared__ uint32_t s_max[kScanThreads];
  __shared__ float s_sum[kScanWarps];
  __shared__ int s_n;
  __shared__ uint64_t s_cand[kCandCap];
  __shared__ uint64_t s_best[kScanWarps];
  grid_dependency_wait();
  const int chunk = blockIdx.x % p.chunks, row = blockIdx.x / p.chunks;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, K = p.K;
  uint64_t* out = p.cand + (static_cast<size_t>(row) * p.chunks + chunk) * K;
  if ((p.finished != nullptr && p.finished[row] != 0) || p.score[row] == -INFINITY) {
    grid_dependents_launch();
    return;                               // the merge makes this beam's pairs itself
  }
  // Vectors start at the 16-byte boundary at or below the row's first logit: logit e of the
  // row is element e + off of the vectors.  Vectors that reach over either end of the row
  // are read logit by logit.
  const T* x = static_cast<const T*>(p.logits) + static_cast<size_t>(row) * p.V;
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
  const int vec0 = chunk * p.chunk_vecs;
  auto first_of = [&](int i) { return (vec0 + i * kScanThreads + tid) * VN - off; };
  auto load = [&](int i) -> uint4 {
    const int at = first_of(i);
    if (i * kScanThreads + tid >= p.chunk_vecs) return make_uint4(R::kNone, R::kNone, R::kNone, R::kNone);
    if (at >= 0 && at + VN <= p.V) return __ldg(reinterpret_cast<const uint4*>(x + at));
    return row_end(x, at, p.V);
  };
  uint4 v[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = load(i);
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < NV; ++i) m = fmaxf(m, R::vmax(v[i]));
  const uint32_t best = logit_key(m);
  s_max[tid] = best;
  if (tid == 0) s_n = 0;
  __syncthreads();
  // Every warp: the slice's maximum and the K-th greatest group maximum to 16 bits (a lower
  // bound), bit by bit.
  uint32_t mx[kScanWarps], gmax = 0u;
#pragma unroll
  for (int i = 0; i < kScanWarps; ++i) {
    mx[i] = s_max[i * 32 + lane];
    gmax = max(gmax, mx[i]);
  }
  const uint32_t top = __reduce_max_sync(0xffffffffu, gmax);
  uint32_t thr = 0u;
  if (K <= 16) {
#pragma unroll
    for (int bit = 31; bit >= 16; --bit) {
      const uint32_t at = thr | (1u << bit);
      if (__popc(__ballot_sync(0xffffffffu, gmax >= at)) >= K) thr = at;
    }
  } else {
    for (int bit = 31; bit >= 16; --bit) {
      const uint32_t at = thr | (1u << bit);
      int n = 0;
#pragma unroll
      for (int i = 0; i < kScanWarps; ++i) n += mx[i] >= at;
      if (__reduce_add_sync(0xffffffffu, n) >= K) thr = at;
    }
  }
  // A bound of -inf (a slice with few allowed tokens): collect what lies above it, the rest
  // of the list is the first tokens at -inf.
  const bool sparse = thr <= kNegInfKey;
  if (sparse) thr = kNegInfKey + 1u;
  const float M = key_logit(top), ref = M == -INFINITY ? 0.f : M;
  const uint64_t neg = f2(-ref, -ref), l2e = f2(1.4426950408889634f, 1.4426950408889634f);
  uint64_t acc = 0ull, acc1 = 0ull;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int c = 0; c < VN; c += 4) {
      float a, b, d, e;
      f2_split(fmul2(fadd2(f2(R::get(v[i], c), R::get(v[i], c + 1)), neg), l2e), a, b);
      f2_split(fmul2(fadd2(f2(R::get(v[i], c + 2), R::get(v[i], c + 3)), neg), l2e), d, e);
      acc = fadd2(acc, f2(fast_exp2(a), fast_exp2(b)));
      acc1 = fadd2(acc1, f2(fast_exp2(d), fast_exp2(e)));
    }
  float a, b;
  f2_split(fadd2(acc, acc1), a, b);
  float sum = a + b;
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) s_sum[warp] = sum;
  // The few threads that reach the bound read their vectors again (from L2): unrolled over
  // the registers this code was most of the kernel's, and fetching it held up every warp.
  if (best >= thr) {
#pragma unroll 1
    for (int i = 0; i < NV; ++i) {
      const uint4 w = load(i);
      if (logit_key(R::vmax(w)) < thr) continue;
#pragma unroll
      for (int c = 0; c < VN; ++c) {
        const int at = first_of(i) + c;
        const uint32_t key = logit_key(R::get(w, c));
        if (key < thr || at < 0 || at >= p.V) continue;
        const int n = atomicAdd(&s_n, 1);
        if (n < kCandCap) s_cand[n] = (static_cast<uint64_t>(key) << 32) | (0xffffffffu - static_cast<uint32_t>(at));
      }
    }
  }
  __syncthreads();
  const int n = s_n;
  if (tid == 0) {
    float t = 0.f;
    for (int i = 0; i < kScanWarps; ++i) t += s_sum[i];
    p.stats[static_cast<size_t>(row) * p.chunks + chunk] = make_float2(M, t);
  }
  if (n <= kCandCap) {
    for (int i = tid; i < n; i += kScanThreads) {
      const uint64_t mine = s_cand[i];
      int r = 0;
      for (int j = 0; j < n; ++j) r += s_cand[j] > mine;
      if (r < K) out[r] = mine;
    }
    if (n < K) {                          // sparse, or a slice shorter than K
      const int lo = max(0, vec0 * VN - off), hi = min(p.V, (vec0 + p.chunk_vecs) * VN - off);
      if (warp == 0) {
        int at = n;
        for (int t0 = lo; t0 < hi && at < K && sparse; t0 += 32) {
          const int t = t0 + lane;
          const bool none = t < hi && to_float(x[t]) == -INFINITY;
          const uint32_t ms = __ballot_sync(0xffffffffu, none);
          const int r = at + __popc(ms & ((1u << lane) - 1u));
          if (none && r < K)
            out[r] = (static_cast<uint64_t>(kNegInfKey) << 32) | (0xffffffffu - static_cast<uint32_t>(t));
          at += __popc(ms);
        }
        for (int r = min(at, K) + lane; r < K; r += 32) out[r] = 0ull;
      }
    }
  } else {                                // many equal logits: K rounds over the whole slice
    const int lo = max(0, vec0 * VN - off), hi = min(p.V, (vec0 + p.chunk_vecs) * VN - off);
    uint64_t last = ~0ull;
    for (int r = 0; r < K; ++r) {
      uint64_t most = 0ull;
      for (int t = lo + tid; t < hi; t += kScanThreads) {
        const uint64_t e = (static_cast<uint64_t>(logit_key(to_float(x[t]))) << 32) | (0xffffffffu - static_cast<uint32_t>(t));
        if (e < last && e > most) most = e;
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
      if (lane == 0) s_best[warp] = most;
      __syncthreads();
      for (int i = 0; i < kScanWarps; ++i) most = max(most, s_best[i]);
      if (tid == 0) out[r] = most;
      last = most;
      __syncthreads();
    }
  }
  grid_dependents_launch();
}

// ------------------------------------------------------------------------ merge

// A pair's rank: score (as ordered 64 bits), then the lower flat index.
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
constexpr int kMergeCand = 4096;          // candidates held on chip when they fit
constexpr int kSpare = 8;                 // lists over K that may pass the bound

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

// One CTA per prompt.  A list is a slice's candidates in descending order.  The lists' first
// `first` entries (their heads) bound the K-th best pair from below: a value that at least K
// heads reach, found on the upper 32 bits of their keys, passes few lists, and only those
// are looked at further.  The call is a chain of small dependent steps; each is spread over
// a warp's lanes.
__global__ void __launch_bounds__(kMergeThreads) beam_merge_kernel(const BeamParams p) {
  extern __shared__ uint64_t s_dyn[];
  __shared__ int s_n, s_reach;
  __shared__ uint32_t s_thr;
  __shared__ Pair s_bound;
  grid_dependency_wait();
  const int b = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int W = p.W, K = p.K, lists = W * p.chunks;
  const int first = min(K, (K + lists - 1) / lists), heads = lists * first;
  const bool held = static_cast<long long>(lists) * K <= kMergeCand;
  const int room = (K + kSpare) * K;
  double* s_off = reinterpret_cast<double*>(s_dyn);                // [W]: score - lse
  int* s_kind = reinterpret_cast<int*>(s_off + W);                 // [W]: 0 live, 1 finished, 2 dead
  uint64_t* s_cand = reinterpret_cast<uint64_t*>(s_off + W + (W + 1) / 2);
  uint64_t* s_head = s_cand + (held ? lists * K : 0);              // [heads]
  uint64_t* s_key = s_head + heads;                                // [room]: survivors
  // Upper words of the keys, padded with 0 to whole 16-byte vectors.
  uint32_t* s_hhi = reinterpret_cast<uint32_t*>((reinterpret_cast<uintptr_t>(s_key + room) + 15) & ~static_cast<uintptr_t>(15));
  uint32_t* s_hi = s_hhi + (heads + 3) / 4 * 4;
  uint32_t* s_hflat = s_hi + (room + 3) / 4 * 4;                   // [heads]
  uint32_t* s_flat = s_hflat + heads;                              // [room]
  const uint64_t* cand = p.cand + static_cast<size_t>(b) * lists * K;
  if (held)                               // (lists of beams that are not live are not used)
    for (int i = tid; i < lists * K; i += kMergeThreads)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(s_cand + i)), "l"(cand + i) : "memory");
  for (int w = warp; w < W; w += kMergeWarps) {
    const int row = b * W + w;
    // (asked for together; those of a beam that is not live are not used)
    const float2* st = p.stats + static_cast<size_t>(row) * p.chunks;
    const float2 mine = lane < p.chunks ? st[lane] : make_float2(-INFINITY, 0.f);
    const float sc = p.score[row];
    const bool over = p.finished != nullptr && p.finished[row] != 0;
    double off = sc;
    if (!over && sc != -INFINITY) {
      float M = mine.x;
      for (int c = lane + 32; c < p.chunks; c += 32) M = fmaxf(M, st[c].x);
#pragma unroll
      for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      if (M != -INFINITY) {
        float hi = mine.y * expf(mine.x - M), lo = 0.f;
        for (int c = lane + 32; c < p.chunks; c += 32) two_sum(hi, lo, st[c].y * expf(st[c].x - M), 0.f);
#pragma unroll
        for (int o = 16; o; o >>= 1) {
          const float x = __shfl_xor_sync(0xffffffffu, hi, o), y = __shfl_xor_sync(0xffffffffu, lo, o);
          two_sum(hi, lo, x, y);
        }
        off -= static_cast<double>(M) + log_fp64(static_cast<double>(hi) + lo);
      }
    }
    if (lane == 0) {
      s_kind[w] = over ? 1 : (sc == -INFINITY ? 2 : 0);
      s_off[w] = off;
    }
  }
  if (tid == 0) {
    s_n = 0;
    s_thr = 0xffffffffu;
    s_reach = 0;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  // Entry j of a list.  Beams that are not live offer their pairs in the first chunk's list:
  // a finished one its end token at its own score, then tokens at -inf in rising order.
  auto entry = [&](int list, int j, Pair& e) -> bool {
    const int w = list / p.chunks, c = list - w * p.chunks;
    const uint32_t base = static_cast<uint32_t>(w) * static_cast<uint32_t>(p.V);
    if (s_kind[w] == 0) {
      const uint64_t r = held ? s_cand[list * K + j] : cand[static_cast<size_t>(list) * K + j];
      if (r == 0ull) return false;
      const float x = key_logit(static_cast<uint32_t>(r >> 32));
      e.key = score_key(x == -INFINITY ? -INFINITY : s_off[w] + static_cast<double>(x));
      e.flat = base + (0xffffffffu - static_cast<uint32_t>(r));
      return true;
    }
    if (c != 0) return false;
    if (s_kind[w] == 1) {
      if (j == 0) {
        e.key = score_key(s_off[w]);
        e.flat = base + static_cast<uint32_t>(p.eos);
        return true;
      }
      const int v = j - 1 + (j - 1 >= p.eos ? 1 : 0);
      if (v >= p.V) return false;
      e.key = score_key(-INFINITY);
      e.flat = base + static_cast<uint32_t>(v);
      return true;
    }
    if (j >= p.V) return false;
    e.key = score_key(-INFINITY);
    e.flat = base + static_cast<uint32_t>(j);
    return true;
  };
  // s_head is 0 where a list has no such entry: no pair's key is 0 (that of NaN).
  for (int i = tid; i < (heads + 3) / 4 * 4; i += kMergeThreads) {
    Pair e;
    const bool ok = i < heads && entry(i / first, i % first, e);
    const uint64_t k = ok ? (e.key == 0ull ? 1ull : e.key) : 0ull;
    s_hhi[i] = static_cast<uint32_t>(k >> 32);
    if (i < heads) {
      s_head[i] = k;
      s_hflat[i] = ok ? e.flat : 0xffffffffu;
    }
  }
  __syncthreads();
  // Upper words of the array above x, and equal to it.
  auto count = [&](const uint32_t* hi, int n, uint32_t x, int& above, int& equal) {
    above = equal = 0;
#pragma unroll 4
    for (int j = 0; j < (n + 3) / 4; ++j) {
      const uint4 h = reinterpret_cast<const uint4*>(hi)[j];
      above += (h.x > x) + (h.y > x) + (h.z > x) + (h.w > x);
      equal += (h.x == x) + (h.y == x) + (h.z == x) + (h.w == x);
    }
  };
  // The K-th greatest upper word of the heads; 0 with fewer than K of them: all pass.
  for (int i = tid; i < heads; i += kMergeThreads) {
    if (s_head[i] == 0ull) continue;
    int above, equal;
    count(s_hhi, heads, s_hhi[i], above, equal);
    if (above < K && above + equal >= K) {
      s_thr = s_hhi[i];                   // (the same value from each that writes)
      s_reach = above + equal;
    }
  }
  __syncthreads();
  const uint32_t thr = s_reach == 0 ? 0u : s_thr;
  const bool exact = s_reach > K + kSpare;   // the bound is s_bound, not thr
  if (exact) {                            // many equal heads: the K-th itself
    for (int i = warp; i < heads; i += kMergeWarps) {
      const Pair mine{s_head[i], s_hflat[i]};
      int r = 0;
      for (int j = lane; j < heads; j += 32) r += before(Pair{s_head[j], s_hflat[j]}, mine);
      r = __reduce_add_sync(0xffffffffu, r);
      if (r == K - 1 && mine.key != 0ull && lane == 0) s_bound = mine;
    }
    __syncthreads();
  }
  const Pair bound = exact ? s_bound : Pair{static_cast<uint64_t>(thr) << 32, 0xffffffffu};
  for (int l = warp; l < lists; l += kMergeWarps) {
    const uint64_t h = s_head[l * first];
    if (h == 0ull || before(bound, Pair{h, s_hflat[l * first]})) continue;
    for (int j0 = 0; j0 < K; j0 += 32) {
      Pair e;
      const int j = j0 + lane;
      const bool in = j < K && entry(l, j, e) && !before(bound, Pair{e.key == 0ull ? 1ull : e.key, e.flat});
      const uint32_t ms = __ballot_sync(0xffffffffu, in);
      int at = 0;
      if (lane == 0 && ms != 0u) at = atomicAdd(&s_n, __popc(ms));
      at = __shfl_sync(0xffffffffu, at, 0) + __popc(ms & ((1u << lane) - 1u));
      if (in && at < room) {
        s_key[at] = e.key;
        s_flat[at] = e.flat;
        s_hi[at] = static_cast<uint32_t>(e.key >> 32);
      }
      if (ms != 0xffffffffu) break;       // a list descends
    }
  }
  __syncthreads();
  const int n = min(s_n, room);
  for (int i = tid; i < n; i += kMergeThreads) {
    int r, equal;
    const uint32_t hi = s_hi[i];
    count(s_hi, n / 4 * 4, hi, r, equal);
    for (int j = n / 4 * 4; j < n; ++j) {
      r += s_hi[j] > hi;
      equal += s_hi[j] == hi;
    }
    if (r >= K) continue;
    const Pair mine{s_key[i], s_flat[i]};
    if (equal > 1)
      for (int j = 0; j < n; ++j) r += s_hi[j] == hi && before(Pair{s_key[j], s_flat[j]}, mine);
    if (r >= K) continue;
    const int w = static_cast<int>(mine.flat / static_cast<uint32_t>(p.V));
    const int v = static_cast<int>(mine.flat - static_cast<uint32_t>(w) * static_cast<uint32_t>(p.V));
    const size_t o = static_cast<size_t>(b) * K + r;
    p.parent[o] = w;
    p.token[o] = v;
    p.new_score[o] = static_cast<float>(key_score(mine.key));
    if (p.new_finished != nullptr) p.new_finished[o] = (s_kind[w] == 1 || v == p.eos) ? 1 : 0;
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
  if (lead) {
    for (int i = tid; i < max_pages; i += kForkThreads) nt[i] = i < full ? bt[i] : (i == full ? fresh : -1);
    if (tid == 0) new_len[j] = len;
  }
  if (full < max_pages) {
    const int from = slots > 0 ? bt[full] : 0;
    if (fresh < 0 || fresh >= num_pages || from < 0 || from >= num_pages) {
      if (lead && tid == 0) report(dev_err, JF_DEVERR_BAD_PAGE);
    } else if (slots > 0) {
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
  }
  grid_dependents_launch();
}

// ------------------------------------------------------------------------ host

struct BeamPlan {
  int nv;                  // vectors a thread holds
  int chunks, chunk_vecs;  // slices of a row, 16-byte vectors of a slice
};

// Eight vectors a thread (16,384 bf16 logits a CTA) while that gives every SM a CTA; with
// few rows, shorter slices spread a row over more SMs.  Slices of a row are equally long.
// One vector more than the logits fill: a row may start inside one.
void plan_beam(long long rows, int V, int dtype, int sms, BeamPlan* pl) {
  const int vn = dtype == JF_DTYPE_BF16 ? 8 : 4;
  const long long vecs = (static_cast<long long>(V) + vn - 1) / vn + 1;
  for (int nv = 8; nv >= 1; nv /= 2) {
    pl->nv = nv;
    pl->chunks = static_cast<int>((vecs + nv * kScanThreads - 1) / (nv * kScanThreads));
    pl->chunk_vecs = static_cast<int>((vecs + pl->chunks - 1) / pl->chunks);
    if (rows * pl->chunks >= sms) break;
  }
}

bool beam_sizes_ok(int32_t B, int32_t W, int32_t V, int32_t K) {
  return B >= 1 && W >= 1 && V >= 1 && K >= 1;
}
bool beam_supported(int32_t B, int32_t W, int32_t V, int32_t K) {
  return K <= kMaxK && W <= kMaxK && static_cast<long long>(W) * V <= (1ll << 26) &&
         static_cast<long long>(K) <= static_cast<long long>(W) * V &&
         static_cast<long long>(B) * W < (1ll << 20);
}

size_t beam_workspace(const BeamPlan& pl, long long rows, int K) {
  return static_cast<size_t>(rows) * pl.chunks * (sizeof(float2) + sizeof(uint64_t) * K);
}

template <typename T>
cudaError_t launch_scan(const BeamParams& p, int nv, unsigned grid, cudaStream_t s) {
  switch (nv) {
    case 8: return launch_pdl(beam_scan_kernel<T, 8>, dim3(grid), dim3(kScanThreads), 0, s, p);
    case 4: return launch_pdl(beam_scan_kernel<T, 4>, dim3(grid), dim3(kScanThreads), 0, s, p);
    case 2: return launch_pdl(beam_scan_kernel<T, 2>, dim3(grid), dim3(kScanThreads), 0, s, p);
    default: return launch_pdl(beam_scan_kernel<T, 1>, dim3(grid), dim3(kScanThreads), 0, s, p);
  }
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
  plan_beam(static_cast<long long>(B) * W, V, dtype, sms, &pl);
  return beam_workspace(pl, static_cast<long long>(B) * W, K);
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
  if (new_score == score || (finished != nullptr && new_finished == finished)) return JF_ERR_INVALID_ARGUMENT;
  if (!beam_supported(B, W, V, K)) return JF_ERR_UNSUPPORTED;
  if (!aligned_to(logits, dtype == JF_DTYPE_BF16 ? 2 : 4) || !aligned_to(workspace, 8)) return JF_ERR_MISALIGNED;
  const int sms = current_sm_count();
  if (sms <= 0) return JF_ERR_CUDA;
  const long long rows = static_cast<long long>(B) * W;
  BeamPlan pl;
  plan_beam(rows, V, dtype, sms, &pl);
  if (rows * pl.chunks >= (1ll << 31)) return JF_ERR_UNSUPPORTED;
  if (workspace_bytes < beam_workspace(pl, rows, K)) return JF_ERR_WORKSPACE_TOO_SMALL;
  BeamParams p;
  p.logits = logits;
  p.score = score;
  p.finished = finished;
  p.parent = parent;
  p.token = token;
  p.new_score = new_score;
  p.new_finished = new_finished;
  p.cand = static_cast<uint64_t*>(workspace);
  p.stats = reinterpret_cast<float2*>(p.cand + static_cast<size_t>(rows) * pl.chunks * K);
  p.W = W;
  p.V = V;
  p.K = K;
  p.eos = eos_token;
  p.chunks = pl.chunks;
  p.chunk_vecs = pl.chunk_vecs;
  const int lists = W * pl.chunks, first = std::min(K, (K + lists - 1) / lists);
  const size_t room = static_cast<size_t>(lists) * first + static_cast<size_t>(K + kSpare) * K;
  const size_t held = static_cast<long long>(lists) * K <= kMergeCand ? static_cast<size_t>(lists) * K : 0;
  const size_t smem = sizeof(double) * (W + (W + 1) / 2) + held * sizeof(uint64_t) +
                      room * (sizeof(uint64_t) + 2 * sizeof(uint32_t)) + 64;
  static SmemAttr attr;
  if (!attr.ensure(beam_merge_kernel, 220 * 1024)) return JF_ERR_CUDA;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>(rows * pl.chunks);
  cudaError_t e = dtype == JF_DTYPE_BF16 ? launch_scan<uint16_t>(p, pl.nv, grid, s)
                                         : launch_scan<float>(p, pl.nv, grid, s);
  if (e == cudaSuccess)
    e = launch_pdl(beam_merge_kernel, dim3(static_cast<unsigned>(B)), dim3(kMergeThreads), smem, s, p);
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
  if (new_block_table == block_table || new_prefix_len == prefix_len) return JF_ERR_INVALID_ARGUMENT;
  if ((D != 64 && D != 128) || page_size != kPage || Hkv > 65535 || max_pages > (1 << 26)) return JF_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * std::max(W, K) >= (1ll << 31)) return JF_ERR_UNSUPPORTED;
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
