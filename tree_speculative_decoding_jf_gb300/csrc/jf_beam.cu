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
// its K greatest logits.  A thread's 16-byte vectors stay in registers: the slice's maximum,
// its sum of exponentials and its candidates come from one read.  The K-th greatest of the
// 256 threads' maxima is a value that K logits of the slice reach, so only logits at or
// above it are looked at again.
constexpr int kScanThreads = 256;
constexpr int kScanWarps = kScanThreads / 32;
constexpr int kCandCap = 512;

template <typename T>
struct Vec;
template <>
struct Vec<uint16_t> {
  static constexpr int kN = 8;
};
template <>
struct Vec<float> {
  static constexpr int kN = 4;
};

__device__ __forceinline__ float logit(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }
__device__ __forceinline__ float logit(float x) { return x; }

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
  int W, V, K, eos, chunks, chunk_len;
};

template <typename T, int NV>
__global__ void __launch_bounds__(kScanThreads) beam_scan_kernel(const BeamParams p) {
  constexpr int VN = Vec<T>::kN;
  __shared__ uint32_t s_max[kScanThreads];
  __shared__ float s_f[kScanWarps];
  __shared__ float s_sum[kScanWarps];
  __shared__ uint32_t s_thr;
  __shared__ int s_n;
  __shared__ uint64_t s_cand[kCandCap];
  __shared__ uint64_t s_best[kScanWarps];
  grid_dependency_wait();
  const int chunk = blockIdx.x % p.chunks, row = blockIdx.x / p.chunks;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* out = p.cand + (static_cast<size_t>(row) * p.chunks + chunk) * p.K;
  if ((p.finished != nullptr && p.finished[row] != 0) || p.score[row] == -INFINITY) {
    grid_dependents_launch();
    return;                               // the merge makes this beam's pairs itself
  }
  const T* x = static_cast<const T*>(p.logits) + static_cast<size_t>(row) * p.V;
  const int v_lo = chunk * p.chunk_len, v_hi = min(p.V, v_lo + p.chunk_len);

  float v[NV][VN];
  const bool vec_ok = (reinterpret_cast<uintptr_t>(x) & 15u) == 0;
  float m = -INFINITY;
  uint32_t best = 0u;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = v_lo + (i * kScanThreads + tid) * VN;
    if (vec_ok && at + VN <= v_hi) {
      const uint4 raw = *reinterpret_cast<const uint4*>(x + at);
      const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
      for (int c = 0; c < VN; ++c) v[i][c] = logit(e[c]);
    } else {
#pragma unroll
      for (int c = 0; c < VN; ++c) v[i][c] = at + c < v_hi ? logit(x[at + c]) : -INFINITY;
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int c = 0; c < VN; ++c) m = fmaxf(m, v[i][c]);
  best = logit_key(m);
  s_max[tid] = best;
  float wm = m;
#pragma unroll
  for (int o = 16; o; o >>= 1) wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, o));
  if (lane == 0) s_f[warp] = wm;
  if (tid == 0) s_n = 0;
  __syncthreads();
  float M = s_f[0];
  for (int i = 1; i < kScanWarps; ++i) M = fmaxf(M, s_f[i]);
  const float ref = M == -INFINITY ? 0.f : M;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float part = 0.f;
#pragma unroll
    for (int c = 0; c < VN; ++c) part += exp2f((v[i][c] - ref) * 1.4426950408889634f);
    sum += part;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) s_sum[warp] = sum;
  // The K-th greatest thread maximum, bit by bit (warp 0, eight maxima a lane).
  if (warp == 0) {
    uint32_t mx[kScanWarps];
#pragma unroll
    for (int i = 0; i < kScanWarps; ++i) mx[i] = s_max[i * 32 + lane];
    uint32_t thr = 0u;
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t tryv = thr | (1u << bit);
      int n = 0;
#pragma unroll
      for (int i = 0; i < kScanWarps; ++i) n += mx[i] >= tryv;
      if (__reduce_add_sync(0xffffffffu, n) >= p.K) thr = tryv;
    }
    if (lane == 0) s_thr = thr;
  }
  __syncthreads();
  const uint32_t thr = s_thr;
  if (tid == 0) {
    float s = 0.f;
    for (int i = 0; i < kScanWarps; ++i) s += s_sum[i];
    p.stats[static_cast<size_t>(row) * p.chunks + chunk] = make_float2(M, s);
  }
  if (best >= thr) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int c = 0; c < VN; ++c) {
        const int at = v_lo + (i * kScanThreads + tid) * VN + c;
        const uint32_t key = logit_key(v[i][c]);
        if (key >= thr && at < v_hi) {
          const int n = atomicAdd(&s_n, 1);
          if (n < kCandCap) s_cand[n] = (static_cast<uint64_t>(key) << 32) | (0xffffffffu - static_cast<uint32_t>(at));
        }
      }
  }
  __syncthreads();
  const int n = s_n;
  if (n <= kCandCap) {
    for (int i = tid; i < max(n, p.K); i += kScanThreads) {
      if (i >= n) {
        out[i] = 0ull;                    // a slice shorter than K
        continue;
      }
      const uint64_t mine = s_cand[i];
      int r = 0;
      for (int j = 0; j < n; ++j) r += s_cand[j] > mine;
      if (r < p.K) out[r] = mine;
    }
  } else {                                // ties: K rounds over the whole slice
    uint64_t last = ~0ull;
    for (int r = 0; r < p.K; ++r) {
      uint64_t top = 0ull;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int c = 0; c < VN; ++c) {
          const int at = v_lo + (i * kScanThreads + tid) * VN + c;
          const uint64_t e = (static_cast<uint64_t>(logit_key(v[i][c])) << 32) | (0xffffffffu - static_cast<uint32_t>(at));
          if (at < v_hi && e < last && e > top) top = e;
        }
#pragma unroll
      for (int o = 16; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (lane == 0) s_best[warp] = top;
      __syncthreads();
      for (int i = 0; i < kScanWarps; ++i) top = max(top, s_best[i]);
      if (tid == 0) out[r] = top;
      last = top;
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

constexpr int kMergeThreads = 256;

// One CTA per prompt.  A list is a slice's candidates in descending order.  The K-th best
// of the lists' first `first` entries bounds the K-th best pair from below; since pairs
// rank strictly, at most K lists reach the bound, so the survivors are at most K * K.
__global__ void __launch_bounds__(kMergeThreads) beam_merge_kernel(const BeamParams p) {
  extern __shared__ uint64_t s_raw[];
  __shared__ int s_n;
  __shared__ Pair s_bound;
  grid_dependency_wait();
  const int b = blockIdx.x, tid = threadIdx.x;
  const int W = p.W, K = p.K, lists = W * p.chunks;
  const int first = min(K, (K + lists - 1) / lists), heads = lists * first;
  double* s_off = reinterpret_cast<double*>(s_raw);                // [W]: score - lse
  int* s_kind = reinterpret_cast<int*>(s_off + W);                 // [W]: 0 live, 1 finished, 2 dead
  uint64_t* s_key = reinterpret_cast<uint64_t*>(s_off + W + (W + 1) / 2);
  const int room = max(heads, K * K);
  uint32_t* s_flat = reinterpret_cast<uint32_t*>(s_key + room);
  for (int w = tid; w < W; w += kMergeThreads) {
    const int row = b * W + w;
    const float sc = p.score[row];
    if (p.finished != nullptr && p.finished[row] != 0) {
      s_kind[w] = 1;
      s_off[w] = sc;
    } else if (sc == -INFINITY) {
      s_kind[w] = 2;
      s_off[w] = -INFINITY;
    } else {
      const float2* st = p.stats + static_cast<size_t>(row) * p.chunks;
      float M = -INFINITY;
      for (int c = 0; c < p.chunks; ++c) M = fmaxf(M, st[c].x);
      double Z = 0.0;
      if (M != -INFINITY)
        for (int c = 0; c < p.chunks; ++c) Z += static_cast<double>(st[c].y) * exp(static_cast<double>(st[c].x) - M);
      s_kind[w] = 0;
      s_off[w] = static_cast<double>(sc) - (M == -INFINITY ? 0.0 : static_cast<double>(M) + log(Z));
    }
  }
  if (tid == 0) s_n = 0;
  __syncthreads();
  // Entry j of a list.  Beams that are not live offer their pairs in the first chunk's list:
  // a finished one its end token at its own score, then tokens at -inf in rising order.
  auto entry = [&](int list, int j, Pair& e) -> bool {
    const int w = list / p.chunks, c = list % p.chunks;
    const uint32_t base = static_cast<uint32_t>(w) * static_cast<uint32_t>(p.V);
    if (s_kind[w] == 0) {
      const uint64_t r = p.cand[(static_cast<size_t>(b) * lists + list) * K + j];
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
  for (int i = tid; i < heads; i += kMergeThreads) {
    Pair e;
    const bool ok = entry(i / first, i % first, e);
    s_key[i] = ok ? e.key : 0ull;
    s_flat[i] = ok ? e.flat : 0xffffffffu;
  }
  if (tid == 0) s_bound = Pair{0ull, 0xffffffffu};      // fewer than K heads: everything passes
  __syncthreads();
  for (int i = tid; i < heads; i += kMergeThreads) {
    const Pair mine{s_key[i], s_flat[i]};
    if (mine.flat == 0xffffffffu) continue;
    int r = 0;
    for (int j = 0; j < heads; ++j) r += before(Pair{s_key[j], s_flat[j]}, mine);
    if (r == K - 1) s_bound = mine;
  }
  __syncthreads();
  const Pair bound = s_bound;
  __syncthreads();
  for (int l = tid; l < lists; l += kMergeThreads)
    for (int j = 0; j < K; ++j) {
      Pair e;
      if (!entry(l, j, e) || before(bound, e)) break;
      const int n = atomicAdd(&s_n, 1);
      if (n < room) {
        s_key[n] = e.key;
        s_flat[n] = e.flat;
      }
    }
  __syncthreads();
  const int n = min(s_n, room);
  for (int i = tid; i < n; i += kMergeThreads) {
    const Pair mine{s_key[i], s_flat[i]};
    int r = 0;
    for (int j = 0; j < n; ++j) r += before(Pair{s_key[j], s_flat[j]}, mine);
    if (r >= K) continue;
    const int w = static_cast<int>(mine.flat / static_cast<uint32_t>(p.V));
    const int v = static_cast<int>(mine.flat % static_cast<uint32_t>(p.V));
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
  int nv;          // vectors a thread holds
  int chunks, chunk_len;
};

// Sixteen vectors a thread hide the most latency per CTA; with few rows shorter slices
// spread one row over more SMs.
bool plan_beam(long long rows, int V, int dtype, int sms, BeamPlan* pl) {
  const int vn = dtype == JF_DTYPE_BF16 ? 8 : 4;
  pl->nv = 8;
  for (int nv = 8; nv >= 2; nv /= 2) {
    pl->nv = nv;
    pl->chunk_len = nv * kScanThreads * vn;
    pl->chunks = static_cast<int>((static_cast<long long>(V) + pl->chunk_len - 1) / pl->chunk_len);
    if (rows * pl->chunks >= sms) break;
  }
  return true;
}

bool beam_sizes_ok(int32_t B, int32_t W, int32_t V, int32_t K) {
  return B >= 1 && W >= 1 && V >= 1 && K >= 1;
}
bool beam_supported(int32_t B, int32_t W, int32_t V, int32_t K) {
  return K <= kMaxK && W <= kMaxK && static_cast<long long>(W) * V < (1ll << 31) &&
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
    default: return launch_pdl(beam_scan_kernel<T, 2>, dim3(grid), dim3(kScanThreads), 0, s, p);
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
  BeamPlan pl;
  if (sms <= 0 || !plan_beam(static_cast<long long>(B) * W, V, dtype, sms, &pl)) return static_cast<size_t>(-1);
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
  p.chunk_len = pl.chunk_len;
  const int lists = W * pl.chunks, first = std::min(K, (K + lists - 1) / lists);
  const size_t room = std::max(static_cast<size_t>(lists) * first, static_cast<size_t>(K) * K);
  const size_t smem = sizeof(double) * (W + (W + 1) / 2) + room * (sizeof(uint64_t) + sizeof(uint32_t));
  if (smem > 200 * 1024) return JF_ERR_UNSUPPORTED;
  static SmemAttr attr;
  if (!attr.ensure(beam_merge_kernel, 200 * 1024)) return JF_ERR_CUDA;
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
